"""The operators around a step of many users together, in CUDA graphs, on streams, and as library ops (GB300)."""
import importlib.util
import os

import pytest
import torch

from tests.test_serving_gpu import make_attention
from tests.test_step_gpu import check_lora, check_verify, cuda, i32, make_lora, make_pool, make_verify

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def w():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_weight_group_gb300 import build
    build.build()
    import w4a16_int4_weight_group_gb300 as mod
    mod.lib()
    return mod


@pytest.fixture(scope="module")
def example(w):
    spec = importlib.util.spec_from_file_location("sampled_decode", os.path.join(ROOT, "examples", "sampled_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_trees_of_guesses_give_the_tokens_of_decoding_one_by_one(w, example):
    """Temperature 0: users with and without an adapter, two answers each on shared pages; the guesses that stand are the tokens that
    a model without guesses finds (or within rounding of its best), and all pages come back."""
    g = torch.Generator().manual_seed(3)
    prompts, users = [torch.randint(0, 2048, (n,), generator=g).tolist() for n in (37, 80, 16)], [2, -1, 0]
    server = example.Server(seed=4)
    plain, none = example.decode(server, prompts, users, 1, 16, lambda tokens: [], temperature=0.0)
    assert none == 0 and not server.refs.any()
    following = {tuple(o[:i]): o[i] for p, o in zip(prompts, plain) for i in range(len(p), len(o))}

    def draft(tokens):
        tree, parent, seen = [], -1, list(tokens)
        for _ in range(4):
            t = following.get(tuple(seen))
            if t is None:
                break
            tree += [(parent, (t + 5) % 2048), (parent, t), (parent, (t + 9) % 2048)]
            parent = len(tree) - 2
            seen.append(t)
        return tree

    fast, accepted = example.decode(server, prompts, users, 2, 16, draft, temperature=0.0)
    assert accepted >= 40 and not server.refs.any()
    check = example.Server(seed=4)
    for i, o in enumerate(fast):
        p, user = prompts[i // 2], users[i // 2]
        assert o[:len(p)] == p and len(o) >= len(p) + 16
        table, lens = check.read(p, user)
        for at in range(len(p) - 1, len(o) - 1):
            one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
            logits, lens = check.step(table, lens, torch.tensor([user], dtype=torch.int32, device="cuda"), torch.tensor([o[at]], device="cuda"),
                                      torch.tensor([at], device="cuda"), one, None, 1)
            lp, _, _, top = w.w4a16_token_logprobs(logits, torch.tensor([o[at + 1]], device="cuda"), 1)
            assert float(top[0, 0] - lp[0]) < 0.1
        w.w4a16_kv_free(check.refs, table, lens, check.page)
    assert not check.refs.any() and w.w4a16_get_device_error() == 0


def test_sampled_answers_differ_and_give_their_pages_back(w, example):
    server = example.Server(seed=5)
    prompts = [list(range(40)), list(range(100, 150))]
    a, _ = example.decode(server, prompts, [0, 1], 3, 8, lambda t: [(-1, (t[-1] + 1) % 2048), (0, 7)], temperature=1.0, seed=1)
    b, _ = example.decode(server, prompts, [0, 1], 3, 8, lambda t: [(-1, (t[-1] + 1) % 2048), (0, 7)], temperature=1.0, seed=1)
    assert a == b and len({tuple(x) for x in a}) == 6 and not server.refs.any()


def cases():
    lora = [cuda(make_lora(T, 520, 264, 16, 5, "bf16", seed=T)) for T in (6, 1500, 700)]
    verify = [cuda(make_verify([4, 9, 2], 3001, "bf16", True, False, seed=4, temps=[1.0, 0.0, 0.8])),
              cuda(make_verify([5, 1, 3], 40001, "f16", False, True, seed=5))]
    refs, table = make_pool(1, 3, 6, 16, 40, [40, 16, 90])
    cache = torch.randint(0, 256, (2, 40, 2, 1, 1152), generator=torch.Generator().manual_seed(1), dtype=torch.uint8).cuda()
    return lora, verify, i32(refs), i32(table), cache


def everything(w, lora, verify, refs, table, cache):
    out = [w.w4a16_lora(**c) for c in lora]
    for c in verify:
        out += w.w4a16_verify_drafts(**c)
    nt, nl = w.w4a16_kv_fork(refs, table, i32_cached([40, 16, 90]), i32_cached([0, 2, 2, 1]), 16)
    held, copies = w.w4a16_kv_reserve(refs, nt, nl, i32_cached([50, 95, 100, 40]), 16)
    w.w4a16_kv_copy(cache, copies)
    lens = w.w4a16_kv_compact(cache, 64, nt, held, i32_cached([[0, 2, 4], [0, 1, -1], [3, 2, 1], [0, -1, -1]]), q_start=i32_cached([0, 5, 8, 12, 13]))
    w.w4a16_kv_free(refs, nt, held, 16, keep=lens)
    return out + [nt, nl, held, copies, lens]


_kept = {}


def i32_cached(x):
    key = repr(x)
    if key not in _kept:
        _kept[key] = i32(x)
    return _kept[key]


def test_everything_captured_without_a_warm_up_and_replayed(w):
    lora, verify, refs, table, cache = cases()
    refs2, cache2 = refs.clone(), cache.clone()
    for x in ([40, 16, 90], [0, 2, 2, 1], [50, 95, 100, 40], [[0, 2, 4], [0, 1, -1], [3, 2, 1], [0, -1, -1]], [0, 5, 8, 12, 13]):
        i32_cached(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = everything(w, lora, verify, refs, table, cache)
    want = everything(w, lora, verify, refs2, table, cache2)
    for _ in range(3):  # the eager calls' buffers are others
        w.w4a16_lora(**cuda(make_lora(3000, 64, 64, 8, 900, "bf16", seed=1)))
    first = refs.clone()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert torch.equal(refs, refs2) and torch.equal(cache, cache2) and not torch.equal(refs, first)
    # other inputs in the same places
    other = make_lora(1500, 520, 264, 16, 5, "bf16", seed=77)
    for name in ("x", "a", "b", "ids", "base", "scales"):
        lora[1][name].copy_(other[name])
    v = make_verify([4, 9, 2], 3001, "bf16", True, False, seed=41, temps=[0.6, 1.0, 0.0])
    for name in ("logits", "tokens", "uniforms", "noise", "tree_mask", "temperature"):
        verify[0][name].copy_(v[name])
    g.replay()
    torch.cuda.synchronize()
    check_lora(w, other, "bf16", got[1])
    check_verify(w, v, got[3:7])


def test_two_streams_at_once_and_between_attention_calls(w):
    """The stream's buffer serves the layer, the attention, the adapters and the verification in turn."""
    a, _ = make_attention(w, 128, 4, "bf16", 64, 2, 4, [3000], [5], tree=True, seed=6)
    a = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in a.items()}
    c = [make_lora(1200, 264, 520, 32, 7, "f16", seed=s) for s in (1, 2)]
    v = [make_verify([8, 5], 20003, "f16", False, True, seed=s) for s in (3, 5)]
    dc, dv = [cuda(x) for x in c], [cuda(x) for x in v]
    want = w.w4a16_tree_attention(**a)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = [w.w4a16_lora(**dc[i]), w.w4a16_tree_attention(**a), w.w4a16_verify_drafts(**dv[i]), w.w4a16_tree_attention(**a)]
    torch.cuda.synchronize()
    for i in range(2):
        check_lora(w, c[i], "f16", got[i][0])
        check_verify(w, v[i], got[i][2])
        assert torch.equal(got[i][1], want) and torch.equal(got[i][3], want)
    for ws in w._workspaces.values():
        assert (ws[:4096] == 0).all()
    assert w.w4a16_get_device_error() == 0


def test_a_workspace_of_the_callers_own(w):
    c = cuda(make_lora(1100, 264, 136, 16, 30, "bf16", seed=9))
    need = w.w4a16_lora_workspace_size(1100, 16, 30)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(w.w4a16_lora(**c, workspace=ws), w.w4a16_lora(**c))
    assert (ws[:4096] == 255).all()
    with pytest.raises(w.W4A16Error, match="needed"):
        w.w4a16_lora(**c, workspace=ws[:need - 256])
    v = cuda(make_verify([3, 4], 9001, "bf16", False, False, seed=10))
    need = w.w4a16_verify_drafts_workspace_size(7, 9001)
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")
    out = w.w4a16_verify_drafts(**v, workspace=ws[:need])
    assert all(torch.equal(x, y) for x, y in zip(out, w.w4a16_verify_drafts(**v)))
    assert (ws[:4096] == 255).all() and (ws[need:] == 255).all()
    with pytest.raises(w.W4A16Error, match="needed"):
        w.w4a16_verify_drafts(**v, workspace=ws[:need - 256])


@pytest.mark.parametrize("backend", ["eager", "aot_eager"])
def test_a_compiled_step_keeps_one_graph(w, backend):
    from w4a16_int4_weight_group_gb300 import ops
    lora, verify, refs, table, cache = cases()
    v = verify[0]
    lens, parents = i32([40, 16, 90]), i32([2, 0])

    def fn(x, a, b, ids, base, scales, refs, table, cache):
        y = ops.lora(x, a, b, ids, base, scales)
        acc, path, toks, p = ops.verify_drafts(v["logits"], v["tokens"], v["uniforms"], v["noise"], 9, v["q_start"], v["tree_mask"], None, v["temperature"])
        nt, nl = ops.kv_fork(refs, table, lens, parents, 16)
        held, copies = ops.kv_reserve(refs, nt, nl, nl + 3, 16)
        ops.kv_copy(cache, copies)
        short = ops.kv_compact(cache, 64, nt, held, path[:2].contiguous(), v["q_start"][:3].contiguous())
        ops.kv_free(refs, nt, held, 16, short)
        return y, acc, path, toks, p, nt, nl, held, copies, short

    args = [lora[0][k] for k in ("x", "a", "b", "ids", "base", "scales")]
    r1, c1, r2, c2 = refs.clone(), cache.clone(), refs.clone(), cache.clone()
    want = fn(*args, r1, table, c1)
    got = torch.compile(fn, backend=backend, fullgraph=True)(*args, r2, table, c2)
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(r1, r2) and torch.equal(c1, c2)


def test_ordinary_calls_and_the_bindings_own_agree(w, monkeypatch):
    """The module of ordinary calls makes the same calls as the binding, and leaves it those that it has something to say about."""
    from w4a16_int4_weight_group_gb300 import step
    if not step._bind_fast():
        pytest.skip("the module of ordinary calls was not built")
    made = []

    class Count:
        def __getattr__(self, name):
            def call(*a):
                out = getattr(fast, name)(*a)
                made.append((name, out is not None))
                return out
            return call

    fast = step._fast
    lora, verify, refs, table, cache = cases()
    r1, c1, r2, c2 = refs.clone(), cache.clone(), refs.clone(), cache.clone()
    monkeypatch.setattr(step, "_fast", Count())
    got = everything(w, lora, verify, r1, table, c1)
    # 1500 tokens need a workspace, which is the binding's
    assert made == [("lora", True), ("lora", False), ("lora", True), ("verify_drafts", True), ("verify_drafts", True), ("kv_fork", True),
                    ("kv_reserve", True), ("kv_copy", True), ("kv_compact", True), ("kv_free", True)]
    monkeypatch.setattr(step, "_fast", False)
    want = everything(w, lora, verify, r2, table, c2)
    assert all(torch.equal(x, y) and x.dtype == y.dtype and x.stride() == y.stride() for x, y in zip(got, want))
    assert torch.equal(r1, r2) and torch.equal(c1, c2)
    monkeypatch.setattr(step, "_fast", fast)
    c = lora[0]
    before = w.w4a16_debug_launch_count()
    for kw, error in ((dict(ids=c["ids"].long()), ValueError), (dict(x=c["x"].t().contiguous().t()), ValueError), (dict(a=c["a"][:, :4].contiguous()), ValueError),
                      (dict(out=c["base"][:2]), ValueError), (dict(out=c["x"][:, :264]), w.W4A16Error), (dict(scales=c["scales"].double()), ValueError),
                      (dict(base=c["base"].cpu()), ValueError), (dict(x=c["x"].float()), w.W4A16Error)):
        with pytest.raises(error):
            w.w4a16_lora(**{**c, **kw})
    v = verify[0]
    for kw, error in ((dict(max_q=65), w.W4A16Error), (dict(max_q=2 ** 40), w.W4A16Error), (dict(tokens=v["tokens"].int()), ValueError),
                      (dict(draft_probs=torch.zeros_like(v["logits"], dtype=torch.float32)), w.W4A16Error), (dict(noise=v["noise"][:2]), ValueError)):
        with pytest.raises(error):
            w.w4a16_verify_drafts(**{**v, **kw})
    for fn, args in ((w.w4a16_kv_fork, (refs, table, table[:, 0].contiguous(), table[0], 0)), (w.w4a16_kv_reserve, (refs, table, refs[:3], refs[:3], 2 ** 33)),
                     (w.w4a16_kv_free, (refs, table.t(), refs[:6], 16)), (w.w4a16_kv_copy, (cache, table[:, :3])),
                     (w.w4a16_kv_compact, (cache, 256, table, refs[:3], table))):
        with pytest.raises((ValueError, w.W4A16Error)):
            fn(*args)
    assert w.w4a16_debug_launch_count() == before


FRESH = """
import torch
import w4a16_int4_weight_group_gb300 as w
from tests.test_step_together import cases, everything, i32_cached
lora, verify, refs, table, cache = cases()
for x in ([40, 16, 90], [0, 2, 2, 1], [50, 95, 100, 40], [[0, 2, 4], [0, 1, -1], [3, 2, 1], [0, -1, -1]], [0, 5, 8, 12, 13]):
    i32_cached(x)
refs2, cache2 = refs.clone(), cache.clone()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = everything(w, lora, verify, refs, table, cache)
g.replay()
torch.cuda.synchronize()
want = everything(w, lora, verify, refs2, table, cache2)
assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(refs, refs2) and torch.equal(cache, cache2)
print("equal")
"""


def test_the_first_calls_of_a_process_may_be_captured(w):
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", FRESH], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stdout + r.stderr


def test_two_threads_at_once(w):
    """Host threads with a stream each, first calls of their shapes among them."""
    import threading
    c = [make_lora(T, 136, 264, 24, 4, "bf16", seed=T) for T in (3, 130, 300, 1100)]
    dc = [cuda(x) for x in c]
    v = make_verify([4, 5], 5001, "bf16", False, True, seed=5)
    dv = cuda(v)
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    got[i] = w.w4a16_lora(**dc[i]), w.w4a16_verify_drafts(**dv)
            s.synchronize()
        except Exception as e:  # (told by the main thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for i in range(4):
        check_lora(w, c[i], "bf16", got[i][0])
        check_verify(w, v, got[i][1])


def test_bounded_waits_of_the_adapters_report_timeout_and_recover(w):
    """No MMA is issued, so the waits for them run out: the status says so, and the next call is right."""
    for r in (40, 128):
        c = make_lora(2100, 200, 3960, r, 2, "bf16", seed=r)
        d = cuda(c)
        assert w.w4a16_get_device_error() == 0
        try:
            w.w4a16_debug_set_wait_limit_ns(5_000_000)
            w.w4a16_debug_inject_stall(True)
            w.w4a16_lora(**d)
            torch.cuda.synchronize()
            assert w.w4a16_get_device_error() == 5  # W4A16_ERR_TIMEOUT
        finally:
            w.w4a16_debug_inject_stall(False)
            w.w4a16_debug_set_wait_limit_ns(0)
        assert w.w4a16_get_device_error() == 0
        check_lora(w, c, "bf16", w.w4a16_lora(**d))
