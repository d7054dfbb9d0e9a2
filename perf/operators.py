"""What the serving operators next to the W4A16 linear layer are measured on.

One verification step of speculative decoding uses them one after another: rotary positions, the
quantised paged cache (written with the rotation fused, read back), the attention of a tree of drafted
tokens over that cache, and the log probabilities of the drafted tokens. With ``own`` false ``run``
computes them from elementary torch operations in 32 bits; with ``own`` true it calls the library.

The head counts are those of the layers that the benchmark and the tests time: 7168 output columns
of the 5120-wide layer are (40 + 2 * 8) heads of 128, 3840 of the 2560-wide one (20 + 2 * 5) heads of 128.

Cache layout (uint8 [pages, kv_heads, page_size / 16, tile_bytes]); a tile holds 16 tokens of one head:
K codes [16][D * bits / 8], V codes [16][D * bits / 8], K parameters [16] and V parameters [16] of 32 bits
each (scale bits in the low half, zero point in the high half). 4-bit codes: element 2i in the low
nibble of byte i, element 2i + 1 in the high one. Value = (code - zero) * scale.
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_TINY = 1.1754943508222875e-38  # smallest normal float32


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one drafted chain of a single user: a handful of tokens, latency is all there is
        dict(name="rope_step", op="rope", T=5, H=30, D=128, rot=128, inter=False, dtype="bf16", offset=70000),
        # a prompt's queries and keys, rotated half of each head in the interleaved layout, odd length
        dict(name="rope_prompt", op="rope", T=8191, H=48, D=128, rot=64, inter=True, dtype="f16", offset=0),
        # one step of four users with four drafted tokens each, into a 4-bit cache
        dict(name="cache_step", op="write", T=16, Hq=20, Hkv=5, D=128, rot=128, inter=False, bits=4, page=16, pages=256,
             dtype="bf16"),
        # a long prompt into an 8-bit cache
        dict(name="cache_prompt", op="write", T=8192, Hq=40, Hkv=8, D=128, rot=128, inter=False, bits=8, page=64, pages=256,
             dtype="f16"),
        # a cached prefix read back for a path that wants dense keys and values
        dict(name="cache_read", op="read", T=50001, Hkv=8, D=128, bits=4, page=64, pages=1024, dtype="bf16"),
        # a short chat of one user, one token a step
        dict(name="attend_one", op="attend", B=1, n=1, L=517, Hq=20, Hkv=5, D=128, bits=4, page=16, dtype="bf16",
             ragged=False, tree=False),
        # a full batch of users at different lengths, one token each
        dict(name="attend_batch", op="attend", B=48, n=1, L=6001, Hq=40, Hkv=8, D=128, bits=4, page=64, dtype="f16",
             ragged=True, tree=False),
        # one user with a very long document
        dict(name="attend_long", op="attend", B=1, n=1, L=131073, Hq=40, Hkv=8, D=128, bits=8, page=128, dtype="bf16",
             ragged=False, tree=False),
        # small trees of drafted tokens, wide heads
        dict(name="attend_drafts", op="attend", B=12, n=13, L=8200, Hq=8, Hkv=4, D=256, bits=8, page=32, dtype="f16",
             ragged=True, tree=True),
        # the largest trees, where the products of the scores and the values are the work
        dict(name="attend_tree", op="attend", B=6, n=64, L=20000, Hq=40, Hkv=8, D=128, bits=4, page=64, dtype="bf16",
             ragged=False, tree=True),
        # verifying one user's drafted chain
        dict(name="logprobs_step", op="logprobs", T=5, V=32003, n=1, k=5, dtype="bf16"),
        # scoring a prompt over a large vocabulary, with alternatives
        dict(name="logprobs_prompt", op="logprobs", T=1024, V=128007, n=2, k=20, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attend", "attend", "attend", "logprobs", "logprobs"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 256])
        H = rng.randint(1, 64)
        rot = 2 * rng.randint(4, D // 2) if rng.random() < 0.3 else rng.choice([D, D // 2, D // 4])
        T = _log(rng, 1, max(2, 8191 * 48 * 128 // (H * D)))
        return dict(op=op, T=T, H=H, D=D, rot=rot, inter=rng.random() < 0.5, dtype=dtype, offset=rng.randint(0, 100000))
    if op in ("write", "read"):
        D, bits, page = rng.choice([64, 128, 256]), rng.choice([4, 8]), rng.choice([16, 32, 64, 128])
        Hkv = rng.randint(1, 8)
        top = 50001 * 8 * 128 if op == "read" else 8192 * 56 * 128
        G = 0 if op == "read" else rng.choice([1, 2, 4, 5, 8])
        T = _log(rng, 1, top // (D * Hkv * (G + 2 if G else 1)))
        c = dict(op=op, T=T, Hkv=Hkv, D=D, bits=bits, page=page, pages=T // page + rng.randint(2, 50), dtype=dtype)
        if op == "write":
            c.update(Hq=Hkv * G, rot=rng.choice([D, D // 2]), inter=rng.random() < 0.5)
        return c
    if op == "attend":
        D, bits, page = rng.choice([64, 128, 128, 256]), rng.choice([4, 8]), rng.choice([16, 32, 64, 128])
        Hkv, G = rng.randint(1, 8), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        n = 1 if rng.random() < 0.4 else rng.randint(2, 64)
        B = _log(rng, 1, 64)
        # at most the largest listed case's products, and the long case's tokens of one head
        most = min(6 * 64 * 40 * 20000 * 128 // (n * Hkv * G * D), 131073 * 8 * 128 * 2 // (Hkv * D)) // B
        L = max(1, min(131073, _log(rng, min(16, max(1, most)), max(17, most))))
        return dict(op=op, B=B, n=n, L=L, Hq=Hkv * G, Hkv=Hkv, D=D, bits=bits, page=page, dtype=dtype,
                    ragged=rng.random() < 0.7, tree=rng.random() < 0.7)
    T = _log(rng, 1, 1024)
    V = _log(rng, 1000, min(260000, 1024 * 128007 // T))
    dtype = rng.choice(["f16", "bf16", "f32"])
    return dict(op=op, T=T if dtype != "f32" else max(1, T // 2), V=V, n=rng.randint(1, 4), k=rng.randint(0, 32), dtype=dtype)


def _lens(c):
    """Cached tokens (the drafted ones among them) and drafted tokens of each sequence."""
    B, L, n = c["B"], c["L"], c["n"]
    if not c["ragged"]:
        return [L] * B, [n] * B
    lens = [max(1, int(L * (1.0 - 0.95 * ((b * 0.6180339887498949) % 1.0)))) for b in range(B)]
    if B > 3:
        lens[B - 1] = 0  # a sequence that has nothing cached: its rows are empty
    return lens, [max(1, n - (5 * b) % n) for b in range(B)]


def work(c):
    T = c.get("T", 0)
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rope":
        return dict(bytes=2 * T * c["H"] * c["D"] * e + T * (4 * c["rot"] + 8), flops=3 * T * c["H"] * c["rot"])
    tok = 2 * c["D"] * c["bits"] // 8 + 8 if "bits" in c else 0  # cache bytes of one token of one head
    if c["op"] == "write":  # written, and read back
        heads = 2 * c["Hq"] + 4 * c["Hkv"]
        return dict(bytes=T * (heads * c["D"] * e + 2 * c["Hkv"] * tok + 4 * c["rot"] + 24),
                    flops=3 * T * (c["Hq"] + c["Hkv"]) * c["rot"] + 8 * T * c["Hkv"] * c["D"])
    if c["op"] == "read":
        return dict(bytes=T * (c["Hkv"] * (tok + 2 * c["D"] * e) + 8), flops=4 * T * c["Hkv"] * c["D"])
    if c["op"] == "attend":
        lens, ns = _lens(c)
        rows = sum(ns) * c["Hq"]
        return dict(bytes=sum(lens) * c["Hkv"] * tok + rows * (2 * c["D"] * e + 4),
                    flops=4 * sum(m * l for m, l in zip(ns, lens)) * c["Hq"] * c["D"])
    return dict(bytes=T * (c["V"] * e + 12 * c["n"] + 4 + 12 * c["k"]), flops=5 * T * c["V"])


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _table(n, rot, dev):
    """cos and sin of every position, positions interpolated by 4 for a long context: [n, rot], cos then sin."""
    f = 500000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot) / 4.0
    a = torch.arange(n, device=dev, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _activations(g, dev, *shape):
    """Normal values with a few channels that are several times larger, as keys have them."""
    x = torch.randn(*shape, generator=g, device=dev)
    return x * (1.0 + 5.0 * (torch.rand(shape[-1], generator=g, device=dev) > 0.96))


def _quantise(x, bits, dtype):
    """x float32 [..., D] -> codes, scale (as float32), zero point; the rounding steps of the definition."""
    top = 2 ** bits - 1
    c = torch.tensor(1.0 / top, dtype=torch.float32, device=x.device)
    lo, hi = x.amin(-1).clamp(max=0.0), x.amax(-1).clamp(min=0.0)
    s = (hi * c - lo * c).to(dtype).float()
    bad = ~torch.isfinite(lo) | ~torch.isfinite(hi)
    s = torch.where(s < _TINY, torch.zeros_like(s), s)
    inv = torch.where((s > 0) & ~bad, torch.reciprocal(s), torch.zeros_like(s))
    z = torch.round(torch.where(bad, torch.zeros_like(lo), -lo) * inv).clamp(0, top)
    u = (torch.round(torch.where(bad[..., None], torch.zeros_like(x), x) * inv[..., None]) + z[..., None]).clamp(0, top)
    return u, torch.where(bad, torch.full_like(s, math.nan), s), z


def _bytes_of(u, bits):
    u = u.to(torch.uint8)
    return u if bits == 8 else u[..., 0::2] | (u[..., 1::2] << 4)


def _params_of(s, z, dtype):
    w = (s.to(dtype).view(torch.int16).to(torch.int32) & 0xFFFF) | (z.to(torch.int32) << 16)
    return w.contiguous().view(torch.uint8)


def _fill(g, dev, pages, heads, D, bits, page, dtype):
    """A cache whose every slot holds the quantised form of random keys and values."""
    data = torch.empty(pages, heads, page // 16, 4 * D * bits + 128, dtype=torch.uint8, device=dev)
    step = max(1, (1 << 27) // (heads * page * D))
    for p in range(0, pages, step):
        part = data[p:p + step]
        m, rb = part.shape[0], 2 * D * bits
        for j in range(2):
            x = _activations(g, dev, m, heads, page // 16, 16, D).to(dtype).float()
            u, s, z = _quantise(x, bits, dtype)
            part[..., j * rb:(j + 1) * rb] = _bytes_of(u, bits).flatten(-2)
            part[..., 2 * rb + 64 * j:2 * rb + 64 * (j + 1)] = _params_of(s, z, dtype)
    return data


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DT[c["dtype"]]
    st = dict(c=c, dtype=dt)
    if c["op"] == "rope":
        st["x"] = _activations(g, dev, c["T"], c["H"], c["D"]).to(dt)
        st["table"] = _table(c["offset"] + c["T"], c["rot"], dev)
        st["positions"] = torch.arange(c["offset"], c["offset"] + c["T"], device=dev)
    elif c["op"] == "write":
        # q, k and v are parts of the projection's output, as the linear layer writes it
        heads = c["Hq"] + 2 * c["Hkv"]
        qkv = _activations(g, dev, c["T"], heads, c["D"]).to(dt)
        st["q"], st["k"], st["v"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], 1)
        st["slots"] = torch.randperm(c["pages"] * c["page"], generator=g, device=dev)[:c["T"]].contiguous()
        st["positions"] = torch.arange(c["T"], device=dev) + 100
        st["table"] = _table(c["T"] + 100, c["rot"], dev)
        st["cache"] = torch.zeros(c["pages"], c["Hkv"], c["page"] // 16, 4 * c["D"] * c["bits"] + 128,
                                  dtype=torch.uint8, device=dev)
    elif c["op"] == "read":
        st["cache"] = _fill(g, dev, c["pages"], c["Hkv"], c["D"], c["bits"], c["page"], dt)
        order = torch.randperm(c["pages"], generator=g, device=dev)
        st["slots"] = (order[:, None] * c["page"] + torch.arange(c["page"], device=dev)).flatten()[:c["T"]].contiguous()
    elif c["op"] == "attend":
        lens, ns = _lens(c)
        cols = max(1, -(-max(lens) // c["page"]))
        held = [-(-l // c["page"]) for l in lens]
        pages = sum(held) + 3
        st["cache"] = _fill(g, dev, pages, c["Hkv"], c["D"], c["bits"], c["page"], dt)
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        at = torch.tensor([sum(held[:b]) for b in range(c["B"])], device=dev)
        st["page_table"] = order[(at[:, None] + torch.arange(cols, device=dev)).clamp(max=pages - 1)].contiguous()
        st["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        starts = [sum(ns[:b]) for b in range(c["B"] + 1)]
        st["q_start"] = torch.tensor(starts, dtype=torch.int32, device=dev) if c["n"] > 1 else None
        st["max_q"] = max(ns)
        r = torch.Generator()
        r.manual_seed(seed)
        st["tree_mask"] = None
        if c["tree"]:
            words = []
            for m in ns:
                parents = torch.rand(m, generator=r).tolist()
                row = []
                for i in range(m):
                    up = row[int(parents[i] * i)] if i else 0
                    row.append(up | (1 << i))
                words += [w - (1 << 64) if w >> 63 else w for w in row]
            st["tree_mask"] = torch.tensor(words, dtype=torch.int64, device=dev)
        st["q"] = (torch.randn(starts[-1], c["Hq"], c["D"], generator=g, device=dev) * 1.5).to(dt)
        st["scale"] = c["D"] ** -0.5
    else:
        x = torch.randn(c["T"], c["V"], generator=g, device=dev) * 2.0
        peaks = torch.randint(0, c["V"], (c["T"], 8), generator=g, device=dev)
        x.scatter_add_(1, peaks, torch.rand(c["T"], 8, generator=g, device=dev) * 15.0)
        x[:, torch.randint(0, c["V"], (c["V"] // 50,), generator=g, device=dev)] = -math.inf  # forbidden tokens
        st["logits"] = x.to(dt)
        tokens = torch.randint(0, c["V"], (c["T"], c["n"]), generator=g, device=dev)
        tokens[:, 0] = peaks[:, 0]
        st["tokens"] = tokens
    return st


# ---------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------
def _rotate(x, positions, table, inter):
    rot = table.shape[1]
    t = table[positions][:, None, :]
    cos, sin = t[..., :rot // 2], t[..., rot // 2:]
    x = x.float()
    y = x.clone()
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    return y


def _codes(raw, D, bits):
    raw = raw.unflatten(-1, (16, D * bits // 8))
    return raw.float() if bits == 8 else torch.stack([raw & 15, raw >> 4], -1).flatten(-2).float()


def _values(tiles, D, bits, dtype, j):
    """Keys (j = 0) or values (j = 1) of tiles [..., tile_bytes] as float32 [..., 16, D]."""
    rb = 2 * D * bits
    w = tiles[..., 2 * rb + 64 * j:2 * rb + 64 * (j + 1)].contiguous().view(torch.int32)
    s = (w & 0xFFFF).to(torch.int16).view(dtype).float()
    z = ((w >> 16) & 0xFFFF).float()
    return (_codes(tiles[..., j * rb:(j + 1) * rb], D, bits) - z[..., None]) * s[..., None]


def _plain_read(cache, slots, D, bits, dtype):
    rb, page = 2 * D * bits, cache.shape[2] * 16
    p, t, row = slots // page, slots % page // 16, slots % 16
    codes = cache[..., :2 * rb].unflatten(-1, (2, 16, rb // 16))[p, :, t, :, row]  # [T, heads, 2, bytes of a row]
    w = cache[..., 2 * rb:].unflatten(-1, (2, 16, 4))[p, :, t, :, row].contiguous().view(torch.int32)
    codes = codes.float() if bits == 8 else torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    s = (w & 0xFFFF).to(torch.int16).view(dtype).float()
    return tuple(((codes - ((w >> 16) & 0xFFFF).float()) * s).to(dtype).unbind(2))


def _plain_write(st):
    c, dt = st["c"], st["dtype"]
    q = _rotate(st["q"], st["positions"], st["table"], c["inter"]).to(dt)
    k = _rotate(st["k"], st["positions"], st["table"], c["inter"]).to(dt)
    cache, slots, page = st["cache"], st["slots"], c["page"]
    rb, per = 2 * c["D"] * c["bits"], c["D"] * c["bits"] // 8
    p, t, row = slots // page, slots % page // 16, slots % 16
    for j, x in enumerate((k, st["v"])):
        u, s, z = _quantise(x.float(), c["bits"], dt)
        at = (j * rb + row * per)[:, None] + torch.arange(per, device=row.device)
        heads = torch.arange(c["Hkv"], device=row.device)
        cache[p[:, None, None], heads[:, None], t[:, None, None], at[:, None, :]] = _bytes_of(u, c["bits"])
        at = (2 * rb + 64 * j + 4 * row)[:, None] + torch.arange(4, device=row.device)
        words = _params_of(s, z, dt).view(c["T"], c["Hkv"], 4)
        cache[p[:, None, None], heads[:, None], t[:, None, None], at[:, None, :]] = words
    return q


def _plain_attend(st):
    c, dt, dev = st["c"], st["dtype"], st["q"].device
    B, D, Hkv, G = c["B"], c["D"], c["Hkv"], c["Hq"] // c["Hkv"]
    tiles = st["cache"][st["page_table"].long()]  # [B, pages, heads, tiles, bytes]
    k, v = (_values(tiles, D, c["bits"], dt, j).permute(0, 2, 1, 3, 4, 5).reshape(B, Hkv, -1, D) for j in range(2))
    total, n, L = st["q"].shape[0], st["max_q"], k.shape[2]
    start = st["q_start"].long() if st["q_start"] is not None else torch.arange(B + 1, device=dev)
    count = start[1:] - start[:-1]
    seq = torch.searchsorted(start, torch.arange(total, device=dev), right=True) - 1
    i = torch.arange(total, device=dev) - start[seq]
    q = torch.zeros(B, n, Hkv, G, D, device=dev)
    q[seq, i] = st["q"].float().view(total, Hkv, G, D)
    words = torch.zeros(B, n, dtype=torch.int64, device=dev)
    words[seq, i] = st["tree_mask"] if st["tree_mask"] is not None else -1
    first = st["kv_lens"].long() - count  # where the drafted tokens begin
    place = torch.arange(L, device=dev)
    draft = (place - first[:, None])[:, None, :]  # [B, 1, L]
    bit = (words[:, :, None] >> draft.clamp(0, 63)) & 1
    seen = (draft < 0) | ((bit == 1) if st["tree_mask"] is not None else (draft <= torch.arange(n, device=dev)[:, None]))
    seen &= (place < st["kv_lens"][:, None])[:, None, :]
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D) * st["scale"]
    s = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, n, G, L)
    s = s.masked_fill(~seen[:, None, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
    total_p = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, n * G, L), v).view(B, Hkv, n, G, D)
    o = torch.where(total_p > 0, o / total_p, torch.zeros_like(o))
    lse = (m + torch.log(total_p)).squeeze(-1)
    return o.permute(0, 2, 1, 3, 4)[seq, i].reshape(total, -1, D).to(dt), lse.permute(0, 2, 1, 3)[seq, i].reshape(total, -1)


def _plain_logprobs(st):
    x, k = st["logits"].float(), st["c"]["k"]
    m = x.amax(-1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    s = e.sum(-1, keepdim=True)
    logs = torch.log(s)
    lp = torch.gather(d, 1, st["tokens"]) - logs
    entropy = (logs - torch.where(e > 0, d * e, torch.zeros_like(e)).sum(-1, keepdim=True) / s).squeeze(-1)
    # a whole number that orders by value and, among equal values, by the lower index
    b = (x + 0.0).view(torch.int32).long()
    key = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
    key = key * (1 << 20) + ((1 << 20) - 1 - torch.arange(x.shape[1], device=x.device))
    top = torch.topk(key, k, dim=1).values
    ids = (1 << 20) - 1 - (top & ((1 << 20) - 1))
    return lp, entropy, ids, torch.gather(d, 1, ids) - logs


def run(st):
    op, c = st["c"]["op"], st["c"]
    if own:
        import w4a16_int4_weight_group_gb300 as w4
        if op == "rope":
            return w4.w4a16_rope(st["x"], st["positions"], st["table"], interleaved=c["inter"])
        if op == "write":
            q = w4.w4a16_kv_write(st["k"], st["v"], st["cache"], st["slots"], q=st["q"], positions=st["positions"],
                                  table=st["table"], interleaved=c["inter"])
            return (q,) + tuple(w4.w4a16_kv_read(st["cache"], st["slots"], c["D"], st["dtype"]))
        if op == "read":
            return w4.w4a16_kv_read(st["cache"], st["slots"], c["D"], st["dtype"])
        if op == "attend":
            return w4.w4a16_tree_attention(st["q"], st["cache"], st["page_table"], st["kv_lens"], q_start=st["q_start"],
                                           tree_mask=st["tree_mask"], softmax_scale=st["scale"], max_q=st["max_q"],
                                           return_lse=True)
        return w4.w4a16_token_logprobs(st["logits"], st["tokens"], top_k=c["k"])
    if op == "rope":
        return _rotate(st["x"], st["positions"], st["table"], c["inter"]).to(st["dtype"])
    if op == "write":
        q = _plain_write(st)
        return (q,) + _plain_read(st["cache"], st["slots"], c["D"], c["bits"], st["dtype"])
    if op == "read":
        return _plain_read(st["cache"], st["slots"], c["D"], c["bits"], st["dtype"])
    if op == "attend":
        return _plain_attend(st)
    return _plain_logprobs(st)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _turn64(x, positions, table, inter):
    """The rotation as a product of complex numbers."""
    R = table.shape[1]
    turn = torch.complex(table[positions, :R // 2].double(), table[positions, R // 2:].double())[:, None]
    x = x.double()
    if inter:
        z = torch.complex(x[..., 0:R:2].contiguous(), x[..., 1:R:2].contiguous()) * turn
        y = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * turn
        y = torch.cat([z.real, z.imag], -1)
    return torch.cat([y, x[..., R:]], -1)


def _grid64(x, bits, dtype):
    """x rounded to the grid that its token and head get: zero among its points, scale in the dtype."""
    top = 2.0 ** bits - 1.0
    low = torch.minimum(x.min(-1, keepdim=True).values, torch.zeros((), dtype=x.dtype, device=x.device))
    high = torch.maximum(x.max(-1, keepdim=True).values, torch.zeros((), dtype=x.dtype, device=x.device))
    s = ((high - low) / top).to(dtype).double()
    safe = torch.where(s > 0, s, torch.ones_like(s))
    z = torch.clamp(torch.round(-low / safe), 0, top)
    return torch.where(s > 0, (torch.clamp(torch.round(x / safe) + z, 0, top) - z) * s, torch.zeros_like(x))


def _slot64(cache, slots, D, bits, dtype):
    """Keys and values [tokens, heads, D] at `slots`, decoded byte by byte of each token's own row."""
    pages, heads, tiles, width = cache.shape
    flat = cache.view(pages, heads, tiles * width)
    page, place = slots // (tiles * 16), slots % (tiles * 16)
    base = (place // 16) * width
    per = D * bits // 8
    got = []
    for j in range(2):
        at = base + j * 16 * per + (place % 16) * per
        raw = flat[page[:, None], :, at[:, None] + torch.arange(per, device=at.device)].transpose(1, 2)  # [T, heads, per]
        if bits == 4:
            both = torch.empty(*raw.shape[:2], D, dtype=torch.uint8, device=raw.device)
            both[..., 0::2], both[..., 1::2] = raw % 16, raw // 16
            raw = both
        at = base + 32 * per + 64 * j + 4 * (place % 16)
        par = flat[page[:, None], :, at[:, None] + torch.arange(4, device=at.device)].transpose(1, 2).contiguous()
        s = par[..., :2].contiguous().view(dtype).double()
        z = par[..., 2:3].double() + 256.0 * par[..., 3:4].double()
        got.append((raw.double() - z) * s)
    return got


def exact(c, seed):
    st = prepare(c, seed)
    dt = st["dtype"]
    if c["op"] == "rope":
        return _turn64(st["x"], st["positions"], st["table"], c["inter"])
    if c["op"] == "write":
        k = _turn64(st["k"], st["positions"], st["table"], c["inter"]).to(dt).double()
        return (_turn64(st["q"], st["positions"], st["table"], c["inter"]), _grid64(k, c["bits"], dt),
                _grid64(st["v"].double(), c["bits"], dt))
    if c["op"] == "read":
        return tuple(_slot64(st["cache"], st["slots"], c["D"], c["bits"], dt))
    if c["op"] == "attend":
        lens, ns = _lens(c)
        G, outs, lses, at = c["Hq"] // c["Hkv"], [], [], 0
        for b, (L, n) in enumerate(zip(lens, ns)):
            q = st["q"][at:at + n].double().view(n, c["Hkv"], G, c["D"])
            if L == 0:
                outs.append(torch.zeros(n, c["Hq"], c["D"], dtype=torch.float64, device=q.device))
                lses.append(torch.full((n, c["Hq"]), -math.inf, dtype=torch.float64, device=q.device))
                at += n
                continue
            place = torch.arange(L, device=q.device)
            slots = st["page_table"][b, place // c["page"]].long() * c["page"] + place % c["page"]
            k, v = _slot64(st["cache"], slots, c["D"], c["bits"], dt)
            see = torch.zeros(n, L, dtype=torch.bool, device=q.device)
            see[:, :max(0, L - n)] = True
            for i in range(n):
                w = int(st["tree_mask"][at + i]) if c["tree"] else (1 << (i + 1)) - 1
                cols = [L - n + j for j in range(n) if (w >> j) & 1 and L - n + j >= 0]
                see[i, cols] = True
            s = torch.einsum("nhgd,lhd->nhgl", q, k) * st["scale"]
            s = s.masked_fill(~see[:, None, None, :], -math.inf)
            lse = torch.logsumexp(s, -1)
            p = torch.where(torch.isfinite(lse)[..., None], torch.exp(s - lse[..., None]), torch.zeros_like(s))
            outs.append(torch.einsum("nhgl,lhd->nhgd", p, v).reshape(n, c["Hq"], c["D"]))
            lses.append(lse.reshape(n, c["Hq"]))
            at += n
        return torch.cat(outs), torch.cat(lses)
    lp, entropy = [], []
    for x, t in zip(st["logits"].split(64), st["tokens"].split(64)):
        y = x.double()
        y = y - torch.logsumexp(y, -1, keepdim=True)
        p = torch.exp(y)
        lp.append(y.gather(1, t))
        entropy.append(-torch.where(p > 0, y * p, torch.zeros_like(p)).sum(-1))
    lp, entropy = torch.cat(lp), torch.cat(entropy)
    # alternatives: a stable sort keeps equal logits in the order of their indices
    ids = torch.cat([torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :c["k"]]
                     for x in st["logits"].split(64)])
    top = torch.cat([(x.double() - torch.logsumexp(x.double(), -1, keepdim=True)).gather(1, i)
                     for x, i in zip(st["logits"].split(64), ids.split(64))])
    return lp, entropy, ids, top
