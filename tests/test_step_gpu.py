"""The operators around a step of many users against plain 64-bit implementations (GB300)."""
import math

import pytest
import torch

from tests import _step as plain
from tests._serving import DT, HALF_ULP

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


# ------------------------------------------------------------------------------------------------- adapters
def make_lora(T, K, N, r, n, dtype, seed, ids=None):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, K, generator=g) * (1 + 5 * (torch.rand(K, generator=g) > 0.95))).to(DT[dtype])
    a = (torch.randn(n, r, K, generator=g) * K ** -0.5).to(DT[dtype])
    b = (torch.randn(n, N, r, generator=g) * 0.3).to(DT[dtype])
    base = torch.randn(T, N, generator=g).to(DT[dtype])
    scales = 0.5 + torch.rand(n, generator=g)
    if ids is None:
        ids = torch.randint(-1, n + 1, (T,), generator=g)  # -1 and n: no adapter
    return dict(x=x, a=a, b=b, ids=torch.as_tensor(ids, dtype=torch.int32), base=base, scales=scales)


def check_lora(w, c, dtype, out):
    ref, mag, mag1 = plain.lora(c["x"], c["a"], c["b"], c["ids"], c["scales"], c["base"])
    K, r = c["a"].shape[2], c["a"].shape[1]
    # first product: K fp32 additions and one product with the scale (2^-23 each bounds an addition of either rounding mode),
    # second: r of both parts and the base; h kept with 15 bits at least (bf16: truncated to 8, the rest rounded to 8: 2^-7 2^-9 = 2^-16;
    # fp16 has more); one rounding of the result
    tol = (K + 2) * 2.0 ** -23 * mag1 + ((2 * r + 2) * 2.0 ** -23 + 2.0 ** -15) * mag + 2.0 ** -23 * c["base"].double().abs()
    tol = tol * (1 + HALF_ULP[dtype]) + HALF_ULP[dtype] * ref.abs() + 2.0 ** -24
    err = (out.cpu().double() - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())


def cuda(c):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,K,N,r,n", [(1, 2112, 1152, 8, 4), (1, 8, 8, 8, 1), (7, 200, 40, 24, 3), (9, 520, 264, 16, 1), (33, 1000, 136, 32, 5),
                                       (48, 640, 1160, 64, 48), (64, 264, 72, 128, 7), (256, 72, 96, 48, 2), (257, 136, 104, 16, 3),
                                       (300, 264, 200, 8, 300), (333, 520, 328, 40, 2), (400, 200, 264, 72, 9), (600, 328, 136, 128, 4), (1000, 64, 32, 32, 1),
                                       (1024, 72, 40, 8, 512), (270, 72, 40, 24, 513), (1025, 136, 72, 32, 4), (2049, 64, 40, 16, 30), (2100, 72, 96, 64, 2),
                                       (2500, 64, 72, 128, 3), (2200, 2600, 200, 40, 3), (3000, 1032, 520, 72, 40), (2049, 8, 8, 48, 700), (2500, 712, 1160, 104, 1), (1100, 5120, 264, 64, 3),
                                       (300, 4000, 136, 72, 2), (641, 200, 3904, 128, 40), (640, 4096, 40, 96, 8), (700, 64, 72, 80, 600),
                                       (2100, 4032, 72, 64, 2), (2500, 64, 4072, 128, 3), (1281, 8, 4088, 40, 20), (1300, 4104, 8, 48, 20), (2600, 1000, 3104, 104, 81),
                                       (2600, 1000, 3104, 104, 82), (2570, 520, 3608, 64, 41), (257, 72, 4024, 128, 1), (2400, 136, 3968, 72, 48)])
def test_lora(w, T, K, N, r, n, dtype):
    c = make_lora(T, K, N, r, n, dtype, seed=T + r)
    d = cuda(c)
    out = w.w4a16_lora(**d)
    check_lora(w, c, dtype, out)
    assert torch.equal(d["base"].cpu(), c["base"])
    none = (c["ids"] < 0) | (c["ids"] >= n)
    assert torch.equal(out.cpu()[none], c["base"][none])
    same = w.w4a16_lora(**d, out=d["base"])  # in place
    assert same is d["base"] and torch.equal(same, out)


@pytest.mark.parametrize("T,r", [(20, 16), (500, 16), (1300, 16), (2200, 48), (2200, 80)])
def test_lora_strided_rows_and_no_scales(w, T, r):
    c = make_lora(T, 264, 136, r, 3, "bf16", seed=1)
    c["scales"] = None
    d = cuda(c)
    wide = torch.zeros(T, 512, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:272] = d["x"]
    qkv = torch.full((T, 600), 7.0, dtype=torch.bfloat16, device="cuda")
    part = qkv[:, 160:296]
    part.copy_(d["base"])
    d["x"], d["base"] = wide[:, 8:272], part
    w.w4a16_lora(**d, out=part)
    check_lora(w, c, "bf16", part)
    assert (qkv[:, :160] == 7.0).all() and (qkv[:, 296:] == 7.0).all()


@pytest.mark.parametrize("T,r,N", [(30, 32, 264), (700, 32, 264), (1500, 32, 264), (2300, 32, 264), (2300, 40, 264), (2300, 96, 264), (2300, 40, 3656),
                                   (2300, 96, 3656)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_lora_of_a_token_does_not_depend_on_its_neighbours(w, T, r, N, dtype):
    """The same token, among others in another order, on all ways of finding tiles: the same bits."""
    c = make_lora(T, 520, N, r, 4, dtype, seed=3, ids=[i % 4 for i in range(T)])
    d = cuda(c)
    first = w.w4a16_lora(**d)
    order = torch.randperm(T, generator=torch.Generator().manual_seed(5)).cuda()
    e = dict(d, x=d["x"][order].contiguous(), ids=d["ids"][order].contiguous(), base=d["base"][order].contiguous())
    assert torch.equal(w.w4a16_lora(**e), first[order])
    for _ in range(3):
        assert torch.equal(w.w4a16_lora(**d), first)


@pytest.mark.parametrize("T,r", [(6, 16), (2100, 40)])
def test_lora_large_and_non_finite_values(w, T, r):
    """float16: sums past its range between the products; an infinite or NaN input stays in its own row."""
    c = make_lora(T, 512, 64, r, 2, "f16", seed=4, ids=[0, 1, 0, 1, 0, 0] + [1] * (T - 6))
    c["x"][:2] *= 300.0
    c["a"] *= 100.0
    c["b"] *= 2.0 ** -12
    d = cuda(c)
    out = w.w4a16_lora(**d)
    h = c["x"][0].double() @ c["a"][0].double().T
    assert h.abs().max() > 65504
    check_lora(w, c, "f16", out)
    for dtype in ("f16", "bf16"):
        c = make_lora(T, 512, 64, r, 2, dtype, seed=4, ids=[0] * T)
        fine = w.w4a16_lora(**cuda(c))
        c["x"][1, 3] = math.inf
        c["x"][2, 4] = math.nan
        out = w.w4a16_lora(**cuda(c))
        rest = [0] + list(range(3, T))
        assert torch.equal(out[rest], fine[rest])
        assert not torch.isfinite(out[1:3]).any()


def test_lora_of_no_tokens(w):
    c = cuda(make_lora(4, 64, 32, 8, 2, "bf16", seed=1))
    out = w.w4a16_lora(c["x"][:0], c["a"], c["b"], c["ids"][:0], c["base"][:0])
    assert out.shape == (0, 32)


# ------------------------------------------------------------------------------------------------- verification
def make_verify(counts, V, dtype, tree, draft, seed, temps=None, sharp=8.0):
    g = torch.Generator().manual_seed(seed)
    B, total = len(counts), sum(counts)
    x = torch.randn(total, V, generator=g)
    x.scatter_add_(1, torch.randint(0, V, (total, 4), generator=g), sharp * torch.rand(total, 4, generator=g))
    if V > 50:
        x[:, torch.randint(0, V, (V // 20,), generator=g)] = -math.inf
    x = x.to(DT.get(dtype, torch.float32))
    start = [sum(counts[:b]) for b in range(B + 1)]
    words, tokens = [], torch.zeros(total, dtype=torch.int64)
    q = torch.softmax(x.float() + 0.5 * torch.randn(total, V, generator=g), -1)
    for b, n in enumerate(counts):
        row = []
        for i in range(n):
            up = 0 if i == 0 else int(torch.rand(1, generator=g) ** 1.5 * i) if tree else i - 1
            row.append((row[up] if i else 0) | (1 << i))
            if i:
                at = start[b] + up
                if draft:
                    tokens[start[b] + i] = torch.multinomial(q[at], 1, generator=g)[0]
                else:
                    tokens[start[b] + i] = int(torch.topk(x[at].float(), min(3, V)).indices[int(torch.randint(0, min(3, V), (1,), generator=g))])
        words += [v - (1 << 64) if v >> 63 else v for v in row]
    return dict(logits=x, tokens=tokens, uniforms=torch.rand(total, generator=g), noise=torch.empty(B, V).exponential_(generator=g),
                q_start=torch.tensor(start, dtype=torch.int32), tree_mask=torch.tensor(words, dtype=torch.int64) if tree else None,
                draft_probs=q if draft else None, temperature=None if temps is None else torch.tensor(temps, dtype=torch.float32),
                max_q=max(max(counts), 1))


def check_verify(w, c, out=None):
    out = w.w4a16_verify_drafts(**cuda(c)) if out is None else out
    (k, path, toks, p), close = plain.verify(**c)
    # fp32 sums of up to 2^17 terms and exponentials: decisions nearer than this to their border are not the test's inputs
    assert close > 2.0 ** -16, "the inputs are next to a border: take another seed"
    assert out[0].tolist() == k
    assert out[1].tolist() == path
    assert out[2].tolist() == toks
    ref = torch.tensor(p, dtype=torch.float64)
    got = out[3].cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    # exponent (x - m) / T of up to 50 with four roundings of 2^-24 relative, the exponentials' 2^-22, a sum of the row in parts
    assert ((got - ref).abs() <= 2.0 ** -14 * ref).logical_or(torch.isnan(ref)).all()
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("counts,V,tree,draft", [([5], 32003, False, True), ([1, 4, 8, 2], 1001, False, True), ([8, 3, 1], 20011, False, False),
                                                 ([25, 7, 1, 12], 4099, True, False), ([64, 33], 999, True, False), ([64], 130001, False, True),
                                                 ([2, 2, 2], 1, False, True), ([3, 5], 7, True, False), ([4, 4], 17, False, True)])
def test_verify(w, counts, V, tree, draft, dtype):
    temps = [(1.0, 0.7, 0.0, 1.3)[i % 4] for i in range(len(counts))]
    c = make_verify(counts, V, dtype, tree, draft, seed=V + len(counts), temps=temps)
    out = check_verify(w, c)
    for _ in range(2):
        again = w.w4a16_verify_drafts(**cuda(c))
        assert all(torch.equal(x, y) for x, y in zip(out, again))
    if temps.count(0.0):
        c["temperature"] = None
        check_verify(w, c)


def test_verify_many_sequences(w):
    g = torch.Generator().manual_seed(0)
    counts = torch.randint(0, 5, (300,), generator=g).tolist()
    c = make_verify(counts, 211, "bf16", False, True, seed=12, temps=[1.0] * 300)
    check_verify(w, c)


def test_plain_sampling_and_padded_batches(w):
    c = make_verify([1] * 9, 5003, "bf16", False, False, seed=3, temps=[0.5] * 9)
    c["q_start"], c["max_q"] = None, 1
    check_verify(w, c)
    c = make_verify([6, 9, 4], 1009, "f16", True, False, seed=4)
    c["max_q"] = 5                                       # tokens past the fifth do not count
    check_verify(w, c)
    c["q_start"] = torch.tensor([2, 8, 8, 12], dtype=torch.int32)  # rows in front, behind, and a sequence of nothing
    c["max_q"] = 6
    check_verify(w, c)


def test_verify_strided_rows(w):
    c = make_verify([4, 6], 1003, "bf16", False, True, seed=5)
    d = cuda(c)
    for name in ("logits", "noise", "draft_probs"):
        t = d[name]
        pad = torch.zeros(t.shape[0], t.shape[1] + 13, dtype=t.dtype, device="cuda")
        pad[:, 5:5 + t.shape[1]] = t
        d[name] = pad[:, 5:5 + t.shape[1]]
    check_verify(w, c, w.w4a16_verify_drafts(**d))


def test_verify_rows_without_probabilities(w):
    for bad in (math.nan, math.inf, None):
        for temps in (None, [0.0, 0.0]):
            c = make_verify([3, 4], 700, "f32", False, False, seed=6, temps=temps)
            if bad is None:
                c["logits"][0] = -math.inf
            else:
                c["logits"][0, 699] = bad
            out = check_verify(w, c)
            assert out[0][0] == 0 and out[2][0, 0] == -1


def test_temperatures_out_of_range(w):
    c = make_verify([3, 2, 4, 2], 900, "bf16", False, False, seed=8, temps=[-1.0, math.nan, 1e-30, 0.0])
    out = w.w4a16_verify_drafts(**cuda(c))
    assert out[2][:2, 0].tolist() == [-1, -1] and out[0][:2].tolist() == [0, 0] and torch.isnan(out[3][:2, 0]).all()
    best = c["logits"][5].float()
    assert int(out[2][2, 0]) == int((best == best.max()).nonzero()[0]) or int(out[0][2]) > 0  # a tiny one is as good as none


def test_verify_borders(w):
    V = 600
    c = make_verify([3, 3], V, "f32", False, False, seed=7)
    c["uniforms"][:] = 0.0                               # accepted wherever p > 0
    check_verify(w, c)
    c["tokens"][1], c["tokens"][4] = -1, V               # no tokens of the vocabulary: they do not stand
    out = check_verify(w, c)
    assert out[0].tolist() == [0, 0]
    # equal logits, equal noise, the lowest index; masked by the type's lowest value and by -inf
    for dtype, low in (("f32", -3.4028234663852886e38), ("bf16", -3.3895313892515355e38), ("f16", -65504.0)):
        c = make_verify([1, 1], V, dtype, False, False, seed=8, temps=[0.0, 1.0])
        c["logits"][:] = low
        c["logits"][:, 300:] = -math.inf
        c["logits"][:, [77, 200]] = 3.0
        c["noise"][:] = 0.5
        out = w.w4a16_verify_drafts(**cuda(c))
        assert out[2].flatten().tolist() == [77, 77]
        assert abs(float(out[3][1, 0]) - 0.5) < 1e-6 and float(out[3][0, 0]) == 1.0
    # nothing of p is left once the guesses are rejected: the draw is from p
    c = make_verify([3], V, "f32", True, False, seed=9)
    c["logits"][:] = -math.inf
    c["logits"][:, 5], c["logits"][:, 6] = 0.0, 0.0
    c["tree_mask"] = torch.tensor([1, 3, 5])
    c["tokens"] = torch.tensor([0, 5, 6])
    c["uniforms"][:] = 1.0                               # (outside its range: rejects all)
    out = w.w4a16_verify_drafts(**cuda(c))
    assert out[0].tolist() == [0] and int(out[2][0, 0]) in (5, 6)
    # a guess repeated at the same token
    c["tokens"] = torch.tensor([0, 5, 5])
    c["uniforms"] = torch.tensor([0.0, 0.75, 0.25])
    out = check_verify(w, c)
    assert out[0].tolist() == [0] and int(out[2][0, 0]) == 6


def test_a_repeated_guess_does_not_stand_for_rounding(w):
    """All tokens of a small vocabulary guessed and rejected: what is left of 1 may be less than nothing, the repeated guess has no weight."""
    B, V = 3000, 3
    g = torch.Generator().manual_seed(4)
    tokens = torch.tensor([0, 0, 1, 2, 0]).repeat(B)
    mask = torch.tensor([1, 3, 5, 9, 17]).repeat(B)
    out = w.w4a16_verify_drafts(torch.randn(5 * B, V, generator=g).cuda(), tokens.cuda(), torch.ones(5 * B).cuda(),
                                torch.empty(B, V).exponential_(generator=g).cuda(), q_start=(torch.arange(B + 1) * 5).to(torch.int32).cuda(),
                                tree_mask=mask.cuda(), max_q=5)
    assert not (out[1] == 4).any() and (out[2][:, 0] >= 0).all()


def test_verify_draws_from_the_targets_distribution(w):
    """Frequencies of the first token that comes out, for a sampled chain and for two guesses: those of p."""
    B, V = 20000, 6
    g = torch.Generator().manual_seed(1)
    l = torch.tensor([1.0, 0.0, -1.0, 2.0, -math.inf, 0.5])
    p = torch.softmax(l.double(), 0)
    q = torch.tensor([0.3, 0.3, 0.1, 0.1, 0.1, 0.1])
    for tree in (False, True):
        n = 3 if tree else 2
        tokens = torch.zeros(B, n, dtype=torch.int64)
        tokens[:, 1] = 3 if tree else torch.multinomial(q, B, True, generator=g)
        if tree:
            tokens[:, 2] = 0
        out = w.w4a16_verify_drafts(l.expand(B * n, V).contiguous().cuda(), tokens.flatten().cuda(), torch.rand(B * n, generator=g).cuda(),
                                    torch.empty(B, V).exponential_(generator=g).cuda(), q_start=(torch.arange(B + 1) * n).to(torch.int32).cuda(),
                                    tree_mask=torch.tensor([1, 3, 5]).repeat(B).cuda() if tree else None,
                                    draft_probs=None if tree else q.expand(B * n, V).contiguous().cuda(), max_q=n)
        f = torch.bincount(out[2][:, 0].cpu(), minlength=V).double() / B
        assert ((f - p).abs() <= 5 * (p * (1 - p) / B).sqrt() + 1e-9).all()  # five standard deviations of a fixed seed's draw


# ------------------------------------------------------------------------------------------------- pages
def make_pool(seed, B, cols, page, pages, lens):
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=g).tolist()
    table, refs = [], [0] * pages
    for n in lens:
        row = [order.pop() for _ in range(plain.pages_of(n, page, cols))]
        for q in row:
            refs[q] = 1
        table.append(row + [-1] * (cols - len(row)))
    return refs, table


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B,page,cols,pages,rows", [(1, 16, 4, 20, 8), (3, 32, 9, 60, 12), (40, 16, 6, 400, 130), (2, 64, 3, 9, 6), (5, 16, 0, 7, 4),
                                                    (700, 16, 2, 5000, 1500)])
def test_fork_reserve_free(w, B, page, cols, pages, rows):
    g = torch.Generator().manual_seed(B)
    lens = [min(int(n), cols * page) for n in torch.randint(0, max(1, min(cols, pages // (2 * B) if B else 1) * page + 1), (B,), generator=g)]
    refs, table = make_pool(B, B, cols, page, pages, lens)
    parents = torch.randint(-1, B + 1, (rows,), generator=g).tolist()
    tr, tt = i32(refs), torch.tensor(table, dtype=torch.int32, device="cuda").view(B, cols)
    nt, nl = w.w4a16_kv_fork(tr, tt, i32(lens), i32(parents), page)
    refs, rt, rl = plain.fork(refs, table, lens, parents, page)
    rt = torch.tensor(rt, dtype=torch.int32).view(rows, cols)
    assert tr.tolist() == refs and torch.equal(nt.cpu(), rt) and nl.tolist() == rl
    # every sequence grows by another number of tokens, some by none, some by fewer (the pages run out in some of the cases)
    more = [n + int(x) for n, x in zip(rl, torch.randint(-3, 2 * page, (rows,), generator=g))]
    held, copies = w.w4a16_kv_reserve(tr, nt, nl, i32(more), page)
    refs, rt2, rh, rc = plain.reserve(refs, rt.tolist(), rl, more, page)
    assert tr.tolist() == refs
    assert torch.equal(nt.cpu(), torch.tensor(rt2, dtype=torch.int32).view(rows, cols))
    assert held.tolist() == rh and copies.tolist() == [list(x) for x in rc]
    keep = [max(0, n // 2 - 1) for n in rh]
    for kp in (keep, None):
        w.w4a16_kv_free(tr, nt, i32(rh), page, keep=None if kp is None else i32(kp))
        refs, rt2 = plain.free(refs, rt2, rh, kp, page)
        assert tr.tolist() == refs and torch.equal(nt.cpu(), torch.tensor(rt2, dtype=torch.int32).view(rows, cols))
    w.w4a16_kv_free(tr, tt, i32(lens), page)
    assert not tr.any()


def test_pages_out_of_range_and_freed_twice(w):
    refs = i32([1, 0, 3, 0])
    table = i32([[0, 9, -5, 2], [2, 2, 7, 7]])
    nt, nl = w.w4a16_kv_fork(refs, table, i32([64, -3]), i32([0, 1, 5, -1]), 16)
    assert refs.tolist() == [2, 0, 4, 0] and nl.tolist() == [64, 0, 0, 0]
    assert nt.tolist() == [[0, 9, -5, 2]] + [[-1] * 4] * 3
    w.w4a16_kv_free(refs, table, i32([1000, 20]), 16)
    assert refs.tolist() == [1, 0, 1, 0] and table.tolist() == [[-1] * 4, [-1, -1, 7, 7]]
    w.w4a16_kv_free(refs, table, i32([1000, 20]), 16)
    w.w4a16_kv_free(refs, i32([[0, 0, 0]]), i32([48]), 16)
    assert refs.tolist() == [0, 0, 1, 0]
    # a shared page outside the cache is not copied; lengths past the table have no pages
    refs = i32([0, 0, 0])
    table = i32([[5, -1], [-1, -1]])
    held, copies = w.w4a16_kv_reserve(refs, table, i32([10, 0]), i32([40, 1000]), 16)
    assert held.tolist() == [32, 32] and copies.tolist() == [[-1, -1]] * 2
    assert table.tolist() == [[5, 0], [1, 2]] and refs.tolist() == [1, 1, 1]


@pytest.mark.parametrize("D,bits,page,heads,layers", [(64, 4, 16, 1, 1), (128, 8, 64, 3, 2), (256, 4, 32, 2, 3), (256, 8, 128, 1, 1)])
def test_copy(w, D, bits, page, heads, layers):
    g = torch.Generator().manual_seed(D)
    cache = torch.randint(0, 256, (layers, 12, heads, page // 16, 4 * D * bits + 128), generator=g, dtype=torch.uint8)
    pairs = [(3, 7), (-1, -1), (0, 1), (11, 12), (5, 2), (12, 9), (3, 8), (4, 4)]
    d = cache.cuda()
    w.w4a16_kv_copy(d, i32(pairs))
    for a, z in ((3, 7), (0, 1), (5, 2), (3, 8)):
        cache[:, z] = cache[:, a]
    assert torch.equal(d.cpu(), cache)
    one = cache[0].contiguous().cuda()
    w.w4a16_kv_copy(one, i32([(9, 10)]))
    cache[0, 10] = cache[0, 9]
    assert torch.equal(one.cpu(), cache[0])
    w.w4a16_kv_copy(one, i32([]).view(0, 2))


@pytest.mark.parametrize("layers", [1, 3])
@pytest.mark.parametrize("D,bits,page,heads,counts,lens", [(64, 4, 16, 1, [8], [300]), (128, 8, 64, 3, [16, 5, 1, 0], [70, 5, 40, 33]),
                                                           (256, 8, 32, 2, [64, 64], [200, 64]), (128, 4, 16, 5, [33, 40], [900, 41])])
def test_compact(w, D, bits, page, heads, counts, lens, layers):
    g = torch.Generator().manual_seed(D + layers)
    B, cols = len(lens), max(-(-n // page) for n in lens) + 1
    pages = sum(-(-n // page) for n in lens) + 4
    _, table = make_pool(1, B, cols, page, pages, lens)
    cache = torch.randint(0, 256, (layers, pages, heads, page // 16, 4 * D * bits + 128), generator=g, dtype=torch.uint8)
    start = [sum(counts[:b]) for b in range(B + 1)]
    m = max(counts)
    path = []
    for b, n in enumerate(counts):
        row = sorted(torch.randperm(n, generator=g)[:max(1, n // 2)].tolist()) if n else []
        if b == 1:
            row = row[::-1]  # any order: all are read before one is written
        path.append(row + [-1] * (m - len(row)))
    d = cache.cuda() if layers > 1 else cache[0].contiguous().cuda()
    out = w.w4a16_kv_compact(d, D, i32(table), i32(lens), i32(path), q_start=i32(start))
    ref = plain.compact(cache, D, bits, table, lens, path, start)
    assert out.tolist() == ref and torch.equal(d.cpu().view_as(cache), cache)


def test_compact_out_of_range(w):
    D, bits, page = 64, 8, 16
    g = torch.Generator().manual_seed(2)
    cache = torch.randint(0, 256, (1, 6, 2, 1, 4 * D * bits + 128), generator=g, dtype=torch.uint8)
    table = [[0, 1, 9], [2, -1, 3], [4, 5, -1], [0, 0, 0]]
    lens, start = [40, 48, 2, 5000], [0, 12, 44, 48, 48]
    path = [[0, 3, 11, -1], [0, 16, 31, 40], [3, 2, -1, 1], [2, 1, -1, -1]]
    d = cache.cuda()
    out = w.w4a16_kv_compact(d, D, i32(table), i32(lens), i32(path), q_start=i32(start))
    ref = plain.compact(cache, D, bits, table, lens, path, start)
    assert out.tolist() == ref and torch.equal(d.cpu(), cache)
