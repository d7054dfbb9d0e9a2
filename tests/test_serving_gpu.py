"""The serving operators on the GPU against plain 64-bit implementations (tests/_serving.py).

Tolerances. Rotation: one rounding to the dtype, plus three fp32 roundings of the two terms. Cache: bytes are
equal (the definition fixes every rounding). Attention: scores are fp32 sums of exact products, off by at most
e = (D + 8) 2^-24 sum |q| |k| scale, and the probabilities are rounded to 11 bits, so a result is off by at most
(2^-11 + 2 e + N 2^-23) sum p |v| plus one rounding to the dtype; lse by e + N 2^-23. Log probabilities: sums of V
fp32 terms over 512 threads, each with a few roundings: (V / 512 + 64) 2^-24 (1 + |value|), four times that for the
entropy, whose terms carry the distance to the maximum.
"""
import math

import numpy as np
import pytest
import torch

from tests import _serving as plain
from tests._serving import DT, HALF_ULP, TINY

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_weight_group_gb300 import build
    build.build()
    import w4a16_int4_weight_group_gb300 as mod
    mod.lib()
    return mod


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dtype="bf16"):
    x = torch.randn(*shape, generator=g)
    x = x * (1 + 5 * (torch.rand(shape[-1], generator=g) > 0.9))
    return x.to(DT[dtype])


def table_for(w, n, rot, **kw):
    return w.w4a16_rope_table(n, rot, device="cpu", **kw)


# ------------------------------------------------------------------------------------------------- rotation
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 128, 128), (7, 5, 128, 64), (3, 2, 80, 20), (5, 3, 64, 62), (2, 3, 6, 2),
                                       (130, 9, 256, 256), (3, 40, 96, 96)])
def test_rope(w, T, H, D, rot, dtype, interleaved):
    g = gen(T * 1000 + rot)
    x = normal(g, T, H, D, dtype=dtype)
    pos = torch.randint(0, 3000, (T,), generator=g)
    table = table_for(w, 3000, rot, base=10000.0, scaling="linear", factor=4.0)
    y = w.w4a16_rope(x.cuda(), pos.cuda(), table.cuda(), interleaved).cpu().double()
    ref, mag = plain.rotate(x.double(), pos, table, interleaved)
    tol = HALF_ULP[dtype] * ref.abs() + 3 * 2.0 ** -24 * mag * (1 + HALF_ULP[dtype]) + TINY[dtype]
    assert ((y - ref).abs() <= tol).all()
    assert torch.equal(y[..., rot:], x.double()[..., rot:])


def test_rope_in_place_strided_and_unaligned(w):
    g = gen(5)
    for rot, off in ((128, 0), (64, 0), (128, 1)):  # off: elements that the rows start past a 16-byte boundary
        buf = normal(g, 6, 12, 136)
        x = buf[:, 2:9, off:off + 128]
        pos, table = torch.arange(6) * 11, table_for(w, 100, rot)
        ref = plain.rotate32(x, pos, table, False).to(torch.bfloat16)
        dev = buf.cuda()
        xd = dev[:, 2:9, off:off + 128]
        assert w.w4a16_rope(xd, pos.cuda(), table.cuda(), out=xd) is xd
        assert torch.equal(xd.cpu(), ref)
        keep = dev.cpu()
        keep[:, 2:9, off:off + 128] = x
        assert torch.equal(keep, buf)  # nothing else was written
        # the same strided input to a new tensor
        assert torch.equal(w.w4a16_rope(buf.cuda()[:, 2:9, off:off + 128], pos.cuda(), table.cuda()).cpu(), ref)


def test_rope_positions_outside_the_table_give_nan(w):
    x = normal(gen(1), 4, 3, 128)
    pos = torch.tensor([2, -1, 10, 9])
    table = table_for(w, 10, 64)
    y = w.w4a16_rope(x.cuda(), pos.cuda(), table.cuda()).cpu()
    assert torch.isnan(y[1:3, :, :64]).all() and torch.equal(y[1:3, :, 64:], x[1:3, :, 64:])
    assert torch.isfinite(y[[0, 3]]).all()


def test_rope_of_nothing(w):
    t = table_for(w, 10, 64).cuda()
    for shape in ((0, 4, 64), (3, 0, 64)):
        x = torch.empty(shape, dtype=torch.float16, device="cuda")
        assert w.w4a16_rope(x, torch.zeros(shape[0], dtype=torch.int64, device="cuda"), t).shape == x.shape


# ------------------------------------------------------------------------------------------------- cache
@pytest.mark.parametrize("rot,interleaved", [(0, False), (0.5, False), (1, True), (1, False), (0.25, True)])
@pytest.mark.parametrize("D,bits,page,Hk,G,dtype", [(64, 4, 16, 1, 1, "bf16"), (128, 4, 48, 5, 4, "f16"), (256, 8, 32, 2, 3, "bf16"),
                                                    (128, 8, 16, 3, 8, "f16"), (64, 8, 128, 4, 2, "f16"), (256, 4, 16, 1, 5, "f16")])
def test_cache_write_and_read(w, D, bits, page, Hk, G, dtype, rot, interleaved):
    g = gen(D + bits + Hk)
    T, pages, Hq = 37, 6, Hk * G
    dt = DT[dtype]
    qkv = normal(g, T, Hq + 2 * Hk, D, dtype=dtype)
    q, k, v = qkv.split([Hq, Hk, Hk], 1)
    v = v.clone()
    v[3] = 0                                    # a row of zeros
    v[4] = v[4].abs()                           # no negative element
    k[5, 0] = -k[5, 0].abs()                    # no positive element
    v[6] *= 1e-7 if dtype == "f16" else 1e-39   # scales that round to zero or a subnormal number
    v[7, 0, 1], k[8, 0, 3] = math.inf, math.nan
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[9], slots[10] = -1, pages * page      # not stored
    cache = w.w4a16_kv_cache(pages, Hk, D, page, bits)
    cache.random_(0, 256)
    ref = cache.cpu()
    R = int(D * rot)
    kw, kr, qr = {}, k, None
    if R:
        pos, table = torch.randint(0, 500, (T,), generator=g), table_for(w, 500, R)
        kw = dict(q=q.cuda(), positions=pos.cuda(), table=table.cuda(), interleaved=interleaved)
        kr = plain.rotate32(k, pos, table, interleaved).to(dt)
        qr = plain.rotate32(q, pos, table, interleaved).to(dt)
    q_out = w.w4a16_kv_write(qkv.cuda()[:, Hq:Hq + Hk] if R == 0 else k.cuda(), v.cuda(), cache, slots.cuda(), **kw)
    plain.put(ref, slots, kr, v, bits, dt)
    assert torch.equal(cache.cpu(), ref)
    if R:
        assert torch.equal(q_out.cpu(), qr)
    else:
        assert q_out is None
    got_k, got_v = w.w4a16_kv_read(cache, slots.cuda(), D, dt)
    good = [t for t in range(T) if t not in (9, 10)]
    ek, ev = plain.get(ref, slots[good].tolist(), D, bits, dt)
    for got, want in ((got_k, ek), (got_v, ev)):
        assert torch.equal(torch.nan_to_num(got.cpu()[good].double(), 777.0), torch.nan_to_num(want.to(dt).double(), 777.0))
        assert (got[[9, 10]] == 0).all()
    assert torch.isnan(got_v[7, 0]).all() and torch.isnan(got_k[8, 0]).all() and (got_v[3] == 0).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_cache_error_is_at_most_half_a_step(w, bits):
    x = normal(gen(3), 64, 4, 128, dtype="f16").cuda()
    cache = w.w4a16_kv_cache(4, 4, 128, 16, bits)
    slots = torch.arange(64, device="cuda")
    w.w4a16_kv_write(x, x, cache, slots)
    k, v = w.w4a16_kv_read(cache, slots, 128, torch.float16)
    assert torch.equal(k, v)
    span = x.double().amax(-1).clamp(min=0) - x.double().amin(-1).clamp(max=0)
    step = span / (2 ** bits - 1)
    # half a step, half a step for the rounded zero point at the ends of the range, the scale's and the result's rounding
    assert ((k.double() - x.double()).abs() <= step[..., None] * 1.01 + 2.0 ** -10 * x.double().abs().amax(-1, keepdim=True)).all()


def test_cache_of_nothing(w):
    cache = w.w4a16_kv_cache(2, 2, 64, 16, 8)
    e = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    s = torch.empty(0, dtype=torch.int64, device="cuda")
    assert w.w4a16_kv_write(e, e, cache, s) is None
    k, v = w.w4a16_kv_read(cache, s, 64, torch.float16)
    assert k.shape == v.shape == (0, 2, 64)
    assert (cache == 0).all()


# ------------------------------------------------------------------------------------------------- attention
def random_tree(r, n):
    row = []
    for i in range(n):
        up = row[int(torch.randint(0, i, (1,), generator=r))] if i else 0
        row.append(up | (1 << i))
    return row


def signed(words):
    return torch.tensor([x - (1 << 64) if x >> 63 else x for x in words], dtype=torch.int64)


def make_attention(w, D, bits, dtype, page, Hk, G, lens, ns, tree, seed=0, extra_pages=2, q_scale=1.5):
    """Inputs whose unseen cache slots hold garbage (random bytes: scales among them that are NaN or infinite)."""
    g = gen(seed)
    B, dt = len(lens), DT[dtype]
    cols = max(1, max(-(-l // page) for l in lens))
    pages = sum(-(-l // page) for l in lens) + extra_pages
    cache = w.w4a16_kv_cache(pages, Hk, D, page, bits)
    cache.random_(0, 256)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    pt, at = torch.full((B, cols), -1, dtype=torch.int32), 0
    for b, l in enumerate(lens):
        m = -(-l // page)
        pt[b, :m] = order[at:at + m]
        at += m
        if l:
            k, v = normal(g, l, Hk, D, dtype=dtype), normal(g, l, Hk, D, dtype=dtype)
            t = torch.arange(l)
            w.w4a16_kv_write(k.cuda(), v.cuda(), cache, (pt[b, t // page].long() * page + t % page).cuda())
    total = sum(ns)
    q = (torch.randn(total, Hk * G, D, generator=g) * q_scale).to(dt)
    mask = signed([x for n in ns for x in random_tree(g, n)]) if tree else None
    start = torch.tensor([sum(ns[:b]) for b in range(B + 1)], dtype=torch.int32)
    return dict(q=q, cache=cache, page_table=pt, kv_lens=torch.tensor(lens, dtype=torch.int32), q_start=start, tree_mask=mask,
                max_q=max(ns)), (D, bits, dt, page)


def check_attention(w, a, meta, dtype, scale=None, **kw):
    D, bits, dt, page = meta
    scale = D ** -0.5 if scale is None else scale
    dev = {n: (x.cuda() if isinstance(x, torch.Tensor) else x) for n, x in a.items()}
    out, lse = w.w4a16_tree_attention(softmax_scale=scale, return_lse=True, **{**dev, **kw})
    torch.cuda.synchronize()
    assert w.w4a16_get_device_error() == 0
    ref, rl, mag, dots = plain.attend(a["q"], a["cache"].cpu(), a["page_table"], a["kv_lens"], a["q_start"], a["tree_mask"], scale,
                                      D, bits, dt, page)
    N = max(1, int(a["kv_lens"].max()))
    e = (D + 8) * 2.0 ** -24 * dots
    tol = (2.0 ** -11 + 2 * e + N * 2.0 ** -23)[..., None] * mag + HALF_ULP[dtype] * ref.abs() + TINY[dtype]
    o, l = out.cpu().double(), lse.cpu().double()
    empty = torch.isinf(rl)
    assert (o[empty] == 0).all() and torch.equal(torch.isinf(l), empty) and (l[empty] < 0).all()
    assert ((o - ref).abs() <= tol).all(), float(((o - ref).abs() / tol.clamp(min=1e-30)).max())
    assert ((l - rl).abs()[~empty] <= (e + N * 2.0 ** -23 + 2.0 ** -23 * rl.abs())[~empty] + 1e-6).all()
    return out, lse


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G,Hk", [(1, 1, 2), (1, 5, 3), (1, 16, 1), (3, 4, 2), (2, 5, 1), (7, 4, 2), (13, 3, 1), (16, 8, 1), (64, 2, 1)])
def test_attention_shapes(w, D, bits, dtype, n, G, Hk):
    page = 16 if n % 2 else 32
    lens = [n, n + 1, 15 + n, 16 + n, 17 + n, 130 + n, 300]
    a, meta = make_attention(w, D, bits, dtype, page, Hk, G, lens, [n] * len(lens), tree=n > 1, seed=n * G)
    check_attention(w, a, meta, dtype)


@pytest.mark.parametrize("n,G,D,bits", [(1, 4, 128, 4), (4, 4, 128, 8), (12, 8, 64, 4), (40, 4, 128, 8), (9, 2, 256, 4)])
def test_attention_ragged_with_empty_rows(w, n, G, D, bits):
    # lengths of zero and one, fewer cached than query tokens, sequences of one to n query tokens
    lens = [0, 1, n, max(0, n - 1), 1000, 33, 500, 0]
    ns = [n, n, n, n, 1, max(1, n // 2), n, 1]
    a, meta = make_attention(w, D, bits, "bf16", 48, 2, G, lens, ns, tree=False, seed=3)
    check_attention(w, a, meta, "bf16")
    words = [0 if i % 3 == 0 else (1 << (i % n)) for i in range(sum(ns))]  # some see no drafted token, not even themselves
    a["tree_mask"] = signed(words)
    check_attention(w, a, meta, "bf16")
    a["tree_mask"] = signed([2 ** 64 - 1] * sum(ns))
    check_attention(w, a, meta, "bf16")


@pytest.mark.parametrize("bits,dtype,n", [(4, "bf16", 1), (8, "f16", 1), (4, "f16", 6), (8, "bf16", 30)])
def test_attention_over_a_long_context_is_split_and_repeatable(w, bits, dtype, n):
    a, meta = make_attention(w, 128, bits, dtype, 64, 1, 4, [5003], [n], tree=n > 1, seed=8)
    o1, l1 = check_attention(w, a, meta, dtype)
    for _ in range(3):
        o2, l2 = check_attention(w, a, meta, dtype)
        assert torch.equal(o1, o2) and torch.equal(l1, l2)


def test_attention_peaked_and_large_scores(w):
    # one token that takes everything, scores of several hundred, and a negative scale
    a, meta = make_attention(w, 128, 8, "bf16", 32, 2, 4, [700, 90], [2, 3], tree=True, seed=4, q_scale=40.0)
    check_attention(w, a, meta, "bf16")
    check_attention(w, a, meta, "bf16", scale=-0.05)
    check_attention(w, a, meta, "bf16", scale=0.0)


def test_attention_value_scales_of_very_different_size(w):
    D, page = 128, 16
    g = gen(9)
    cache = w.w4a16_kv_cache(8, 1, D, page, 4)
    k, v = normal(g, 100, 1, D, dtype="bf16"), normal(g, 100, 1, D, dtype="bf16")
    v = (v.float() * torch.logspace(-20, 20, 100)[torch.randperm(100, generator=g)][:, None, None]).to(torch.bfloat16)
    w.w4a16_kv_write(k.cuda(), v.cuda(), cache, torch.arange(100, device="cuda"))
    for n in (1, 20):
        a = dict(q=normal(g, n, 8, D), cache=cache, page_table=torch.arange(8, dtype=torch.int32)[None],
                 kv_lens=torch.tensor([100], dtype=torch.int32), q_start=torch.tensor([0, n], dtype=torch.int32), tree_mask=None, max_q=n)
        check_attention(w, a, (D, 4, torch.bfloat16, page), "bf16")


def test_attention_pages_outside_the_cache_are_not_seen(w):
    for n in (1, 20):
        a, meta = make_attention(w, 128, 4, "bf16", 16, 1, 4, [200, 60], [n, n], tree=False, seed=6)
        pt = a["page_table"]
        pt[0, 3], pt[0, 5], pt[1, 0] = -7, 2 ** 31 - 1, pt.max() + 50
        check_attention(w, a, meta, "bf16")
        pt[1, :] = -1
        check_attention(w, a, meta, "bf16")
        # a length past the page table counts as the table's end
        a, meta = make_attention(w, 128, 4, "bf16", 16, 1, 4, [64], [n], tree=False, seed=6)
        a["kv_lens"][0] = 100000
        check_attention(w, a, meta, "bf16")


def test_attention_nan_stays_in_its_own_rows(w):
    D, page = 128, 16
    g = gen(2)
    for n in (1, 24):
        cache = w.w4a16_kv_cache(8, 2, D, page, 8)
        k, v = normal(g, 100, 2, D, dtype="f16"), normal(g, 100, 2, D, dtype="f16")
        v[50, 0, 3] = math.nan
        w.w4a16_kv_write(k.cuda(), v.cuda(), cache, torch.arange(100, device="cuda"))
        q = normal(g, n, 8, D, dtype="f16")
        q[0, 5, 0] = math.nan
        out, lse = w.w4a16_tree_attention(q.cuda(), cache, torch.arange(8, dtype=torch.int32, device="cuda")[None],
                                          torch.tensor([100], dtype=torch.int32, device="cuda"),
                                          q_start=torch.tensor([0, n], dtype=torch.int32, device="cuda"), max_q=n, return_lse=True)
        assert torch.isnan(out[:, :4]).all() and torch.isfinite(lse[:, :4]).all()   # heads of the first cache head
        assert torch.isnan(out[0, 5]).all() and torch.isnan(lse[0, 5])
        ok = torch.ones(n, 8, dtype=torch.bool)
        ok[:, :4], ok[0, 5] = False, False
        assert torch.isfinite(out[ok.cuda()]).all()


def test_attention_strided_queries_another_stream_and_a_graph(w):
    a, meta = make_attention(w, 128, 4, "bf16", 32, 2, 4, [333, 64, 2000], [3, 1, 4], tree=True, seed=1)
    want, _ = check_attention(w, a, meta, "bf16")
    dev = {n: (x.cuda() if isinstance(x, torch.Tensor) else x) for n, x in a.items()}
    wide = torch.zeros(8, 16, 136, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:11, :128] = dev["q"]
    dev["q"] = wide[:, 3:11, :128]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = w.w4a16_tree_attention(**dev)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        w.w4a16_tree_attention(out=out, **dev)
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            w.w4a16_tree_attention(out=out, **dev)
    out.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_attention_without_workspace(w):
    """The C entry point with a NULL workspace gives the layer's result (nothing is split)."""
    import ctypes
    a, meta = make_attention(w, 128, 4, "bf16", 32, 2, 4, [3000], [1], tree=False, seed=1)
    want, _ = check_attention(w, a, meta, "bf16")
    from w4a16_int4_weight_group_gb300 import serving
    d = {n: (x.cuda() if isinstance(x, torch.Tensor) else x) for n, x in a.items()}
    c = serving._cache(d["cache"], 128)
    out = torch.empty_like(want)
    st = w.lib().w4a16_tree_attention(ctypes.byref(c), d["q"].data_ptr(), d["q"].stride(0), d["q"].stride(1), 8, 1, None, 1, 1,
                                      d["kv_lens"].data_ptr(), d["page_table"].data_ptr(), d["page_table"].shape[1], None, 128 ** -0.5,
                                      out.data_ptr(), None, 1, None, 0, None)
    assert st == 0, w.last_error()
    torch.cuda.synchronize()
    assert ((out.double() - want.double()).abs() <= 2.0 ** -7 * want.double().abs() + 2.0 ** -10).all()


def test_attention_offsets_past_32_bits(w):
    """Pages more than 2^32 bytes into the cache."""
    D, page, Hk, bits = 128, 128, 8, 8
    pages = (1 << 32) // (Hk * page * 264) + 40
    cache = torch.empty(pages, Hk, page // 16, int(w.lib().w4a16_kv_tile_bytes(D, bits)), dtype=torch.uint8, device="cuda")
    g = gen(12)
    L = 300
    pt = torch.tensor([[pages - 1, 3, pages - 7]], dtype=torch.int32)
    t = torch.arange(L)
    slots = pt[0, t // page].long() * page + t % page
    k, v = normal(g, L, Hk, D), normal(g, L, Hk, D)
    w.w4a16_kv_write(k.cuda(), v.cuda(), cache, slots.cuda())
    small = cache[[pages - 1, 3, pages - 7]].cpu()
    ref = torch.zeros_like(small)
    plain.put(ref, t, k, v, bits, torch.bfloat16)
    rk, rv = plain.get(ref, range(L), D, bits, torch.bfloat16)
    gk, gv = w.w4a16_kv_read(cache, slots.cuda(), D, torch.bfloat16)
    assert torch.equal(gk.cpu().double(), rk.to(torch.bfloat16).double()) and torch.equal(gv.cpu().double(), rv.to(torch.bfloat16).double())
    for n in (1, 20):
        q = normal(g, n, Hk * 4, D)
        out = w.w4a16_tree_attention(q.cuda(), cache, pt.cuda(), torch.tensor([L], dtype=torch.int32, device="cuda"),
                                     q_start=torch.tensor([0, n], dtype=torch.int32, device="cuda"), max_q=n).cpu().double()
        want, _, mag, dots = plain.attend(q, small, torch.tensor([[0, 1, 2]]), torch.tensor([L]), torch.tensor([0, n]), None, D ** -0.5,
                                          D, bits, torch.bfloat16, page)
        tol = (2.0 ** -11 + 2 * (D + 8) * 2.0 ** -24 * dots + L * 2.0 ** -23)[..., None] * mag + HALF_ULP["bf16"] * want.abs()
        assert ((out - want).abs() <= tol).all()


# ------------------------------------------------------------------------------------------------- log probabilities
def check_logprobs(w, x, tokens, k):
    lp, h, ids, top = w.w4a16_token_logprobs(x, tokens, k)
    V = x.shape[1]
    y = torch.log_softmax(x.cpu().double(), -1)
    p = y.exp()
    H = -torch.where(p > 0, p * y, torch.zeros_like(p)).sum(-1)
    t = tokens.cpu() if tokens.dim() == 2 else tokens.cpu()[:, None]
    want = y.gather(1, t).view(lp.shape)
    unit = (V / 512 + 64) * 2.0 ** -24

    def near(a, b, f=1.0):
        a, b = a.cpu().double(), b.double()
        fin = torch.isfinite(b)
        assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a[~fin & ~torch.isnan(b)], b[~fin & ~torch.isnan(b)])
        assert ((a - b).abs()[fin] <= f * unit * (1 + b.abs()[fin])).all(), float(((a - b).abs()[fin] / (f * unit * (1 + b.abs()[fin]))).max())

    near(lp, want)
    near(h, H, 4.0)
    order = torch.sort(x.cpu().double(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.cpu(), order)
    near(top, y.gather(1, order))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,V,n,k", [(1, 1, 1, 1), (3, 2, 2, 2), (2, 33, 1, 32), (5, 1000, 3, 7), (1, 4097, 1, 20), (4, 32003, 2, 5), (2, 70001, 1, 32),
                                        (170, 2050, 1, 3), (400, 16390, 0, 1), (3, 16384, 1, 0)])
def test_logprobs(w, dtype, rows, V, n, k):
    g = gen(V + k)
    x = (torch.randn(rows, V, generator=g) * 3).to({**DT, "f32": torch.float32}[dtype]).cuda()
    check_logprobs(w, x, torch.randint(0, V, (rows, n), generator=g).cuda(), k)


def test_logprobs_masked_tied_and_sorted_rows(w):
    V, k = 20011, 20
    g = gen(7)
    x = torch.randn(9, V, generator=g)
    x[0] = 1.25                                   # every logit the same
    x[1, :] = -math.inf
    x[1, 17777:17780] = torch.tensor([0.5, 2.0, 0.5])   # three tokens allowed
    x[2] = torch.finfo(torch.bfloat16).min        # all at the type's lowest value
    x[3] = torch.finfo(torch.bfloat16).min
    x[3, 19] = 3.0
    x[4] = torch.linspace(-50, 50, V)             # rising: every step holds larger ones
    x[5] = torch.linspace(50, -50, V)
    x[6] = (torch.arange(V) % 3).float()          # thousands of ties at the top
    x[7, ::2], x[7, 1::2] = 0.0, -0.0
    x[8] = -math.inf
    x[8, V - 1] = -1e30
    for dt in (torch.bfloat16, torch.float32):
        y = x.to(dt).cuda()
        check_logprobs(w, y, torch.randint(0, V, (9, 2), generator=g).cuda(), k)
    for rows in (200,):                           # as above with one CTA a row
        y = x[4:5].expand(rows, V).to(torch.bfloat16).contiguous().cuda()
        check_logprobs(w, y, torch.zeros(rows, dtype=torch.int64, device="cuda"), k)


def test_logprobs_rows_without_a_distribution(w):
    V = 9001
    x = torch.randn(5, V, generator=gen(1))
    x[0] = -math.inf
    x[1, 77] = math.nan
    x[2, 78] = math.inf
    for dt in (torch.float16, torch.float32):
        lp, h, ids, top = w.w4a16_token_logprobs(x.to(dt).cuda(), torch.tensor([5, 6, 7, -1, V], device="cuda"), 4)
        assert torch.isnan(lp).all()              # rows 3 and 4: tokens outside the vocabulary
        assert torch.isnan(h[:3]).all() and torch.isfinite(h[3:]).all()
        assert ((ids >= -1) & (ids < V)).all()
        y = torch.log_softmax(x[3:].to(dt).double(), -1).topk(4).values
        assert ((top[3:].cpu().double() - y).abs() < 1e-4).all()


def test_logprobs_row_stride_and_unaligned_rows(w):
    g = gen(4)
    wide = torch.randn(7, 5003, generator=g).to(torch.bfloat16).cuda()
    for a, b in ((0, 5000), (1, 4999), (3, 4100), (8, 8 + 4096)):
        check_logprobs(w, wide[:, a:b], torch.randint(0, b - a, (7,), generator=g).cuda(), 9)


def test_logprobs_of_nothing(w):
    lp, h, ids, top = w.w4a16_token_logprobs(torch.empty(0, 100, dtype=torch.float16, device="cuda"), None, 3)
    assert lp.shape == (0, 0) and h.shape == (0,) and ids.shape == (0, 3) and top.shape == (0, 3)
