"""What the operators around a verification step of many users are measured on.

Beside the projections: low-rank adapters, another one for each user, added to what the shared 4-bit layer gives.
After the head: which drafted tokens stand, from given random numbers, and the token after them. Then the cache: the
accepted tokens' rows moved together, pages shared by forked sequences, copied before they are written, given back.
With ``own`` false ``run`` computes them from elementary torch operations in 32 bits; with ``own`` true it calls
the library.

The layers' sizes are those that the benchmark and the tests time (5120 -> 7168, 2560 -> 3840, 2112 -> 1152). The cache is uint8
[layers, pages, kv_heads, page_size / 16, tile_bytes]; a tile holds 16 tokens of one head: K codes [16][D * bits / 8], V codes
[16][D * bits / 8], K parameters [16] and V parameters [16] of 4 bytes each.
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one user's next token: the smallest layer of the tests, latency is all there is
        dict(name="lora_one", op="lora", T=1, K=2112, N=1152, r=8, n=4, mix="each", dtype="bf16"),
        # a step of 48 users, one token each, most with an adapter of their own and some with none
        dict(name="lora_batch", op="lora", T=48, K=5120, N=7168, r=16, n=32, mix="each", dtype="bf16"),
        # a verification step of 40 users with 13 drafted tokens each, wide adapters
        dict(name="lora_drafts", op="lora", T=520, K=2560, N=3840, r=64, n=24, mix="runs", dtype="f16"),
        # prompts of several users in one batch
        dict(name="lora_prompt", op="lora", T=8191, K=5120, N=7168, r=32, n=12, mix="runs", dtype="bf16"),
        # one user, four tokens drawn by a draft model
        dict(name="verify_chain", op="verify", B=1, n=5, V=32003, tree=False, dtype="bf16"),
        # 64 users, seven drafted tokens each, large vocabulary
        dict(name="verify_chains", op="verify", B=64, n=8, V=128007, tree=False, dtype="bf16"),
        # trees of the likeliest guesses of a few users
        dict(name="verify_trees", op="verify", B=6, n=25, V=32003, tree=True, dtype="f16"),
        # the largest trees, logits that the head left in 32 bits
        dict(name="verify_forest", op="verify", B=8, n=64, V=65537, tree=True, dtype="f32"),
        # accepted tokens of four users put together in one layer's cache
        dict(name="compact_step", op="compact", L=1, B=4, n=8, len=300, Hkv=5, D=128, bits=4, page=16),
        # the same for a full batch and all layers at once
        dict(name="compact_layers", op="compact", L=16, B=64, n=16, len=230, Hkv=8, D=128, bits=8, page=64),
        # a prompt continued by eight beams, one token further
        dict(name="fork_beams", op="fork", L=1, B=1, new=8, len=1500, grow=1, Hkv=5, D=128, bits=4, page=16),
        # four answers to each of 32 prompts, in every layer's cache
        dict(name="fork_samples", op="fork", L=8, B=32, new=128, len=500, grow=200, Hkv=8, D=128, bits=8, page=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "lora", "lora", "verify", "verify", "verify", "compact", "fork"])
    if op == "lora":
        K, N = 8 * _log(rng, 32, 1100), 8 * _log(rng, 32, 1100)
        r = 8 * _log(rng, 1, 16)
        n = _log(rng, 1, max(2, min(64, 300_000_000 // (r * (K + N) * 2))))
        most = min(8191 * (5120 + 2 * 7168) // (K + 2 * N), 8191 * 12288 * 32 // ((K + N) * r))
        return dict(op=op, T=_log(rng, 1, max(2, min(16000, most))), K=K, N=N, r=r, n=n, mix=rng.choice(["each", "runs", "one"]),
                    dtype=rng.choice(["f16", "bf16"]))
    if op == "verify":
        V, dtype = _log(rng, 500, 260000), rng.choice(["f16", "bf16", "f32"])
        rows = min(512, 64 * 8 * 128007 // V // (2 if dtype == "f32" else 1))
        n = rng.randint(1, 16) if rng.random() < 0.6 else rng.randint(1, 64)
        n = max(1, min(n, rows))
        return dict(op=op, B=_log(rng, 1, max(1, min(64, rows // n))), n=n, V=V, tree=rng.random() < 0.5, dtype=dtype)
    L, Hkv, D, bits = rng.randint(1, 8), rng.randint(1, 8), rng.choice([64, 128, 256]), rng.choice([4, 8])
    page = rng.choice([16, 32, 64, 128])
    token = L * Hkv * (2 * D * bits // 8 + 8)
    if op == "compact":
        B, n = _log(rng, 1, 64), rng.randint(1, 64)
        most = 550_000_000 // (token * B) - page  # the cache of the largest listed one
        n = max(1, min(n, most // 2, 16 * 64 * 16 * 8 * 264 // (token * B)))
        return dict(op=op, L=L, B=B, n=n, len=n + rng.randint(0, max(1, min(1000, most - n))), Hkv=Hkv, D=D, bits=bits, page=page)
    B, each = _log(rng, 1, 32), rng.randint(1, 8)
    most = 800_000_000 // (token * page)  # pages
    B = max(1, min(B, most // 40))
    new = max(1, min(B * each, most // 4))
    len_ = rng.randint(1, max(1, min(2000, (most // 4) * page // B)))
    return dict(op=op, L=L, B=B, new=new, len=len_, grow=rng.randint(1, max(1, min(300, (most // 8) * page // new))), Hkv=Hkv, D=D, bits=bits, page=page)


def _lens(c):
    """Cached tokens (the drafted ones among them) and drafted tokens of each sequence of a compaction."""
    ns = [max(1, c["n"] - (5 * b) % c["n"]) for b in range(c["B"])]
    return [max(ns[b], int(c["len"] * (1.0 - 0.5 * ((b * 0.6180339887498949) % 1.0)))) for b in range(c["B"])], ns


def _counts(c):
    """Drafted tokens of each sequence of a verification, the root among them."""
    return [max(1, c["n"] - (3 * b) % c["n"]) for b in range(c["B"])]


def _fork_lens(c):
    return [max(1, int(c["len"] * (1.0 - 0.4 * ((b * 0.6180339887498949) % 1.0)))) for b in range(c["B"])]


def work(c):
    if c["op"] == "lora":
        used = min(c["n"], c["T"])
        return dict(bytes=2 * (c["T"] * (c["K"] + 2 * c["N"]) + used * c["r"] * (c["K"] + c["N"])) + 4 * c["T"],
                    flops=2 * c["T"] * c["r"] * (c["K"] + c["N"]))
    if c["op"] == "verify":
        rows, e = sum(_counts(c)), 4 if c["dtype"] == "f32" else 2
        return dict(bytes=rows * c["V"] * e + c["B"] * c["V"] * (4 if c["tree"] else 8), flops=4 * rows * c["V"])
    token = c["L"] * c["Hkv"] * (2 * c["D"] * c["bits"] // 8 + 8)
    if c["op"] == "compact":  # about half of the drafted tokens stand, and most of those move
        return dict(bytes=sum(_lens(c)[1]) * token, flops=0)
    lens = _fork_lens(c)  # every new sequence copies its parent's last page, unless that is full
    copied = c["new"] * sum(n % c["page"] != 0 for n in lens) / len(lens)
    return dict(bytes=2 * copied * token * c["page"] + 8 * c["new"] * (-(-c["len"] // c["page"])), flops=0)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _signed(w):
    return w - (1 << 64) if w >> 63 else w


def _random_tree(n, r):
    """Parents of a tree of n nodes (node 0 the root): wide near the root."""
    return [0] + [int(r.random() ** 1.5 * i) for i in range(1, n)]


def prepare(c, seed):
    import random
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = random.Random(seed)
    st = dict(c=c)
    if c["op"] == "lora":
        dt, T, K, N, n = _DT[c["dtype"]], c["T"], c["K"], c["N"], c["n"]
        loud = 1.0 + 5.0 * (torch.rand(K, generator=g, device=dev) > 0.97)
        st["x"] = (torch.randn(T, K, generator=g, device=dev) * loud).to(dt)
        st["a"] = (torch.randn(n, c["r"], K, generator=g, device=dev) * K ** -0.5).to(dt)
        st["b"] = (torch.randn(n, N, c["r"], generator=g, device=dev) * 0.3).to(dt)
        st["scales"] = 16.0 / c["r"] * (0.5 + torch.rand(n, generator=g, device=dev))
        st["base"] = torch.randn(T, N, generator=g, device=dev).to(dt)
        if c["mix"] == "each":
            ids = torch.randint(-1 if T > 1 else 0, n, (T,), generator=g, device=dev)  # -1: a user without an adapter
        elif c["mix"] == "one":
            ids = torch.full((T,), r.randrange(n), device=dev)
        else:  # runs of tokens of one request
            cut = torch.rand(T, generator=g, device=dev) < 3.0 * n / (2 * T + n)
            ids = torch.randint(0, n, (T + 1,), generator=g, device=dev)[cut.cumsum(0)]
        st["ids"] = ids.to(torch.int32)
    elif c["op"] == "verify":
        dt, B, V, ns = _DT[c["dtype"]], c["B"], c["V"], _counts(c)
        start = [sum(ns[:b]) for b in range(B + 1)]
        total = start[-1]
        x = torch.randn(total, V, generator=g, device=dev)
        peaks = torch.randint(0, V, (total, 6), generator=g, device=dev)
        x.scatter_add_(1, peaks, 4.0 + torch.rand(total, 6, generator=g, device=dev) * 10.0)
        x[:, torch.randint(0, V, (V // 50,), generator=g, device=dev)] = -math.inf  # forbidden tokens
        st["logits"] = x.to(dt)
        st["q_start"] = torch.tensor(start, dtype=torch.int32, device=dev)
        st["max_q"] = max(ns)
        st["uniforms"] = torch.rand(total, generator=g, device=dev)
        st["noise"] = torch.empty(B, V, device=dev).exponential_(generator=g)
        temps = [(0.0, 0.7, 1.0, 1.3)[(b + seed) % 4] for b in range(B)]
        st["temperature"] = torch.tensor(temps, device=dev)
        st["tree_mask"] = st["draft_probs"] = None
        if c["tree"]:
            # a node's guesses are its likeliest tokens, as another model sees them
            words, parents, order = [], [], []
            for b, m in enumerate(ns):
                up, seen, row = _random_tree(m, r), {}, []
                for i in range(m):
                    row.append((row[up[i]] if i else 0) | (1 << i))
                    parents.append(start[b] + up[i])
                    order.append(seen.get(up[i], 0))
                    seen[up[i]] = order[-1] + 1
                words += [_signed(w) for w in row]
            near = x + torch.randn(total, V, generator=g, device=dev)
            best = torch.topk(near, min(V, 64), dim=1).indices
            parents, order = torch.tensor(parents, device=dev), torch.tensor(order, device=dev)
            st["tokens"] = best[parents, order % best.shape[1]].contiguous()
            st["tree_mask"] = torch.tensor(words, dtype=torch.int64, device=dev)
        else:
            q = torch.softmax(x + 0.7 * torch.randn(total, V, generator=g, device=dev), -1)
            drawn = (q / torch.empty(total, V, device=dev).exponential_(generator=g)).argmax(1)
            st["draft_probs"] = q
            st["tokens"] = torch.cat([drawn[:1], drawn[:-1]])  # row i's draft is token i + 1
    else:
        page, L, Hkv = c["page"], c["L"], c["Hkv"]
        tile = 4 * c["D"] * c["bits"] + 128
        if c["op"] == "compact":
            lens, ns = _lens(c)
            held = [-(-n // page) for n in lens]
            pages, rows = sum(held) + 3, c["B"]
            start = [sum(ns[:b]) for b in range(rows + 1)]
            st["q_start"] = torch.tensor(start, dtype=torch.int32, device=dev)
            path = []
            for m in ns:  # a path down a random tree
                up, kept = _random_tree(m, r), [0]
                for i in range(1, m):
                    if up[i] == kept[-1] and r.random() < 0.8:
                        kept.append(i)
                path.append(kept + [-1] * (max(ns) - len(kept)))
            st["path"] = torch.tensor(path, dtype=torch.int32, device=dev)
        else:
            lens = _fork_lens(c)
            held = [-(-n // page) for n in lens]
            rows = c["B"]
            pages = sum(held) + c["new"] * (2 + -(-c["grow"] // page)) + 3
            st["parents"] = torch.tensor([i % rows if i < rows else r.randrange(rows) for i in range(c["new"])], dtype=torch.int32, device=dev)
            st["grow"] = torch.tensor([r.randint(1, c["grow"]) for _ in range(c["new"])], dtype=torch.int32, device=dev)
        st["cache"] = torch.randint(0, 256, (L, pages, Hkv, page // 16, tile), generator=g, device=dev, dtype=torch.uint8)
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        cols = -(-max(lens) // page) + (-(-c["grow"] // page) + 1 if c["op"] == "fork" else 0)
        at = torch.tensor([sum(held[:b]) for b in range(rows)], device=dev)
        spread = torch.arange(cols, device=dev)
        table = order[(at[:, None] + spread).clamp(max=pages - 1)]
        st["page_table"] = torch.where(spread < torch.tensor(held, device=dev)[:, None], table, torch.full_like(table, -1)).contiguous()
        st["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        if c["op"] == "fork":
            st["refs"] = torch.zeros(pages, dtype=torch.int32, device=dev)
            st["refs"][order[:sum(held)].long()] = 1
    return st


# ---------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------
def _plain_lora(st):
    x, a, b, ids = st["x"].float(), st["a"], st["b"], st["ids"].long()
    n, r, K = a.shape
    has = ((ids >= 0) & (ids < n))[:, None]
    at = ids.clamp(0, n - 1)
    s = torch.where(has, st["scales"][at][:, None], torch.zeros_like(has, dtype=torch.float32))
    if x.shape[0] <= 64:  # few tokens: each with its adapter's matrices beside it
        h = torch.matmul(a[at].float(), x[:, :, None])[:, :, 0] * s
        y = torch.matmul(b[at].float(), h[:, :, None])[:, :, 0]
    else:  # all adapters side by side, and of each token's products those of its own
        h = torch.matmul(x, a.reshape(n * r, K).float().t()).view(-1, n, r)
        mine = torch.arange(n, device=x.device) == at[:, None]
        h = torch.where(mine[:, :, None], h * s[:, :, None], torch.zeros_like(h)).view(-1, n * r)
        y = torch.matmul(h, b.float().permute(0, 2, 1).reshape(n * r, -1))
    return (st["base"].float() + y).to(st["base"].dtype)


def _first_of_largest(x):
    at = torch.arange(x.shape[-1], device=x.device)
    return torch.where(x == x.amax(-1, keepdim=True), at, torch.full_like(at, x.shape[-1])).amin(-1)


def _plain_verify(st):
    l, q = st["logits"].float(), st["draft_probs"]
    total, V = l.shape
    dev, m = l.device, st["max_q"]
    start = st["q_start"].long()
    count, B = start[1:] - start[:-1], start.shape[0] - 1
    seq = torch.searchsorted(start, torch.arange(total, device=dev), right=True) - 1
    i = torch.arange(total, device=dev) - start[seq]
    t = st["temperature"][seq][:, None]
    e = torch.exp((l - l.amax(-1, keepdim=True)) / torch.where(t > 0, t, torch.ones_like(t)))
    p = e / e.sum(-1, keepdim=True)
    p = torch.where(t > 0, p, (torch.arange(V, device=dev) == _first_of_largest(l)[:, None]).float())
    # [sequence, token]
    tok, u, words = (torch.zeros(B, m, dtype=x.dtype, device=dev) for x in (st["tokens"], st["uniforms"], st["tokens"]))
    tok[seq, i], u[seq, i] = st["tokens"], st["uniforms"]
    words[seq, i] = st["tree_mask"] if st["tree_mask"] is not None else -torch.ones_like(i)
    j = torch.arange(m, device=dev)
    below = ((words[:, :, None] >> j) & 1).bool() & (j < j[:, None])  # [B, i, j]: j is an ancestor of i
    parent = torch.where(below, j, torch.zeros_like(j)).amax(-1)
    valid = (j > 0) & (j < count[:, None]) & below.any(-1) & (tok >= 0) & (tok < V)
    row = (start[:-1, None] + parent).clamp(max=total - 1)
    pd = p[row, tok.clamp(0, V - 1)]
    if q is not None:
        passed = valid & (u * q[row, tok.clamp(0, V - 1)] < pd)
        chosen = passed
    else:
        before = valid[:, :, None] & valid[:, None, :] & (parent[:, :, None] == parent[:, None, :]) & (j < j[:, None])
        again = (before & (tok[:, :, None] == tok[:, None, :])).any(-1)
        pd = torch.where(again, torch.zeros_like(pd), pd)
        left = 1.0 - torch.where(before, pd[:, None, :], torch.zeros_like(pd)[:, None, :]).sum(-1)
        passed = valid & (u * left < pd)
        chosen = passed & ~(before & passed[:, None, :]).any(-1)
    stands = chosen & (~below | chosen[:, None, :] | (j == 0)).all(-1)
    stands[:, 0] = count > 0
    path = torch.where(stands, j, torch.full_like(j, m)).sort(-1).values
    last = torch.where(stands, j, torch.zeros_like(j)).amax(-1)
    at = start[:-1] + last
    probs, p = p, p[at]
    kids = valid & (parent == last[:, None])
    if q is not None:
        r = torch.where(kids.any(-1)[:, None], (p - q[at]).clamp(min=0), p)
    else:
        gone = torch.zeros(B, V + 1, dtype=torch.bool, device=dev)
        gone.scatter_(1, torch.where(kids, tok, torch.full_like(tok, V)), True)
        r = torch.where(gone[:, :V], torch.zeros_like(p), p)
    r = torch.where((r > 0).any(-1, keepdim=True), r, p)
    new = _first_of_largest(torch.where(r > 0, r / st["noise"], torch.full_like(r, -1.0)))
    accepted = stands.sum(-1) - 1
    follow = torch.gather(tok, 1, torch.cat([path[:, 1:], path[:, :1]], 1).clamp(max=m - 1))
    out = torch.where(j < accepted[:, None], follow, torch.where(j == accepted[:, None], new[:, None], torch.full_like(tok, -1)))
    # the target's probability of each of them
    probs = probs[(start[:-1, None] + path).clamp(max=total - 1), out.clamp(min=0)]
    probs = torch.where(out >= 0, probs, torch.zeros_like(probs))
    return accepted.to(torch.int32), torch.where(path < m, path, torch.full_like(path, -1)).to(torch.int32), out, probs


def _plain_compact(st):
    c, cache, table = st["c"], st["cache"], st["page_table"].long()
    page, per = c["page"], c["D"] * c["bits"] // 8
    path, lens = st["path"].long(), st["kv_lens"].long()
    start = st["q_start"].long()
    first = (lens - (start[1:] - start[:-1]))[:, None]
    to = torch.arange(path.shape[1], device=path.device)
    b, k = torch.nonzero((path >= 0) & (path != to), as_tuple=True)
    src, dst = first[b, 0] + path[b, k], first[b, 0] + k
    at = torch.arange(per, device=src.device)
    # bytes of a token's row in its tile: K codes, V codes, K parameter, V parameter
    row = torch.cat([at, 16 * per + at, 32 * per + at[:4], 32 * per + 64 + at[:4]])
    step = torch.cat([torch.full_like(at, per), torch.full_like(at, per), torch.full((8,), 4, device=at.device)])

    def place(x):
        return table[b, x // page][:, None], (x % page // 16)[:, None], row + step * (x % 16)[:, None]

    (p0, t0, y0), (p1, t1, y1) = place(src), place(dst)
    moved = cache[:, p0, :, t0, y0]  # [tokens, bytes, layers, heads]: all read before any is written
    cache[:, p1, :, t1, y1] = moved
    return cache, (first[:, 0] + (path >= 0).sum(1)).to(torch.int32)


def _plain_fork(st):
    c, refs, cache = st["c"], st["refs"], st["cache"]
    page, up = c["page"], st["parents"].long()
    table, lens = st["page_table"].long()[up], st["kv_lens"].long()[up]
    dev, cols = table.device, table.shape[1]
    col = torch.arange(cols, device=dev)
    have = (lens + page - 1) // page
    owned = col < have[:, None]
    table = torch.where(owned, table, torch.full_like(table, -1))
    refs.index_add_(0, table.clamp(min=0).flatten(), owned.flatten().to(torch.int32))
    # room for the tokens to come: shared partial pages are copied (the last holder keeps its page), new ones added
    new_lens = lens + st["grow"]
    want = ((new_lens + page - 1) // page).clamp(max=cols)
    tail = torch.gather(table, 1, (have - 1).clamp(min=0)[:, None])[:, 0]
    shared = (lens % page != 0) & (refs[tail.clamp(min=0)] > 1)
    n = torch.arange(len(lens), device=dev)
    earlier = (shared[:, None] & shared & (tail[:, None] == tail) & (n < n[:, None])).sum(1)
    cow = (shared & (earlier < refs[tail.clamp(min=0)] - 1)).long()
    need = cow + (want - have).clamp(min=0)
    first = need.cumsum(0) - need
    free = torch.argsort((refs != 0).to(torch.int32), stable=True)
    room = (refs == 0).sum()
    number = first[:, None] + cow[:, None] + (col - have[:, None])
    fresh = (col >= have[:, None]) & (col < want[:, None]) & (number < room)
    table = torch.where(fresh, free[number.clamp(0, len(refs) - 1)], table)
    got = (cow == 1) & (first < room)
    dst = free[first.clamp(max=len(refs) - 1)]
    table = torch.where(got[:, None] & (col == (have - 1)[:, None]), dst[:, None], table)
    refs.index_add_(0, tail.clamp(min=0), -got.to(torch.int32))
    mine = fresh | (got[:, None] & (col == (have - 1)[:, None]))
    refs.index_add_(0, table.clamp(min=0).flatten(), mine.flatten().to(torch.int32))
    held = torch.minimum(new_lens, (owned | fresh).sum(1) * page)
    held = torch.where((cow == 1) & ~got, lens, held)
    copies = torch.where(got[:, None], torch.stack([tail, dst], 1), torch.full_like(dst, -1)[:, None])
    two = copies[copies[:, 0] >= 0]
    cache[:, two[:, 1]] = cache[:, two[:, 0]]
    kept = refs.clone()
    # the new sequences end: their pages go back
    used = (col < ((held + page - 1) // page)[:, None]).flatten()
    refs.index_add_(0, table.clamp(min=0).flatten(), -used.to(torch.int32))
    return table.to(torch.int32), held.to(torch.int32), copies.to(torch.int32), kept, refs, cache


def run(st):
    op = st["c"]["op"]
    if own:
        import w4a16_int4_weight_group_gb300 as w4
        if op == "lora":
            return w4.w4a16_lora(st["x"], st["a"], st["b"], st["ids"], st["base"], scales=st["scales"])
        if op == "verify":
            return w4.w4a16_verify_drafts(st["logits"], st["tokens"], st["uniforms"], st["noise"], q_start=st["q_start"],
                                          tree_mask=st["tree_mask"], draft_probs=st["draft_probs"], temperature=st["temperature"],
                                          max_q=st["max_q"])
        c = st["c"]
        if op == "compact":
            lens = w4.w4a16_kv_compact(st["cache"], c["D"], st["page_table"], st["kv_lens"], st["path"], q_start=st["q_start"])
            return st["cache"], lens
        table, lens = w4.w4a16_kv_fork(st["refs"], st["page_table"], st["kv_lens"], st["parents"], c["page"])
        held, copies = w4.w4a16_kv_reserve(st["refs"], table, lens, lens + st["grow"], c["page"])
        w4.w4a16_kv_copy(st["cache"], copies)
        given, kept = table.clone(), st["refs"].clone()
        w4.w4a16_kv_free(st["refs"], table, held, c["page"])
        return given, held, copies, kept, st["refs"], st["cache"]
    if op == "lora":
        return _plain_lora(st)
    if op == "verify":
        return _plain_verify(st)
    return _plain_compact(st) if op == "compact" else _plain_fork(st)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _exact_lora(st):
    y = st["base"].double()
    for k in range(st["a"].shape[0]):
        rows = torch.nonzero(st["ids"] == k)[:, 0]
        h = torch.einsum("tk,rk->tr", st["x"][rows].double(), st["a"][k].double())
        y[rows] += float(st["scales"][k]) * torch.einsum("tr,nr->tn", h, st["b"][k].double())
    return y


def _exact_verify(st):
    """The walk down each tree, one node after another."""
    start, V, m = st["q_start"].tolist(), st["logits"].shape[1], st["max_q"]
    tok, u, temps = st["tokens"].tolist(), st["uniforms"].double().tolist(), st["temperature"].tolist()
    words = None if st["tree_mask"] is None else [w & (2 ** 64 - 1) for w in st["tree_mask"].tolist()]
    counts, paths, outs, probs = [], [], [], []
    for b in range(len(start) - 1):
        s, n = start[b], start[b + 1] - start[b]
        up = [-1] + [(i if words is None else (words[s + i] & ((1 << i) - 1)).bit_length()) - 1 for i in range(1, n)]
        path, token, given = [0], None, []
        while token is None:
            at = s + path[-1]
            l = st["logits"][at].double()
            if temps[b] > 0:
                p = torch.softmax(l / float(st["temperature"][b]), 0)
            else:
                p = torch.zeros_like(l)
                p[int(torch.nonzero(l == l.max())[0])] = 1.0
            q = None if st["draft_probs"] is None else st["draft_probs"][at].double()
            r = p.clone()
            for i in [i for i in range(1, n) if up[i] == path[-1]]:
                d = tok[s + i]
                if q is not None and u[s + i] * float(q[d]) < float(p[d]):
                    path.append(i)
                    given.append(float(p[d]))
                    break
                if q is not None:
                    r = torch.clamp(p - q, min=0)
                    continue
                if u[s + i] * float(r.sum()) < float(r[d]):
                    path.append(i)
                    given.append(float(p[d]))
                    break
                r[d] = 0.0
            else:
                r = r if bool((r > 0).any()) else p
                score = torch.where(r > 0, r / st["noise"][b].double(), torch.full_like(r, -1.0))
                token = int(torch.nonzero(score == score.max())[0])
                given.append(float(p[token]))
        k = len(path) - 1
        counts.append(k)
        paths.append(path + [-1] * (m - k - 1))
        outs.append([tok[s + i] for i in path[1:]] + [token] + [-1] * (m - k - 1))
        probs.append(given + [0.0] * (m - k - 1))
    dev = st["logits"].device
    return tuple(torch.tensor(x, dtype=t, device=dev)
                 for x, t in ((counts, torch.int32), (paths, torch.int32), (outs, torch.int64), (probs, torch.float64)))


def exact(c, seed):
    if c["op"] not in ("lora", "verify"):
        return None  # nothing is computed: bytes are moved and pages counted
    st = prepare(c, seed)
    return _exact_lora(st) if c["op"] == "lora" else _exact_verify(st)
