"""The serving operators in CUDA graphs: every graph has a workspace of its own, whatever is captured, run and replayed
around it. Results are compared with the same calls outside of graphs, bit for bit (they do not depend on timing)."""
import pytest
import torch

from tests.test_serving_gpu import make_attention

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


def attention_case(w, n, seed, D=128):
    """One sequence long enough to be split over many CTAs: n drafted tokens of 4 query heads a cache head."""
    a, _ = make_attention(w, D, 4, "bf16", 64, 2, 4, [3000], [n], tree=n > 1, seed=seed)
    return {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in a.items()}


def captured(w, dev, **kw):
    out = torch.empty_like(dev["q"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, **kw):
        w.w4a16_tree_attention(out=out, **dev)
    return g, out


def test_graphs_captured_without_a_stream_replay_in_any_order(w):
    """No warm-up on the capture's stream: its first call is the captured one."""
    small, large = attention_case(w, 1, 1), attention_case(w, 40, 2)
    want = [w.w4a16_tree_attention(**small), w.w4a16_tree_attention(**large)]
    torch.cuda.synchronize()
    graphs = [captured(w, small), captured(w, large), captured(w, small)]
    for order in ((2, 1, 0), (1, 0, 2), (0, 2, 1)):
        for i in order:
            g, out = graphs[i]
            out.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[i % 2]), (order, i)
    assert w.w4a16_get_device_error() == 0


def test_a_graph_survives_eager_calls_that_need_more(w):
    small, large = attention_case(w, 1, 3), attention_case(w, 40, 4)
    want = w.w4a16_tree_attention(**small)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        w.w4a16_tree_attention(**small)  # the stream's own buffer, of the small call's size
    s.synchronize()
    g, out = captured(w, small, stream=s)
    with torch.cuda.stream(s):
        big = w.w4a16_tree_attention(**large)  # grows the stream's buffer
        s.synchronize()
        # whatever was freed goes to these
        others = [torch.full((1 << 18,), 5, dtype=torch.int32, device="cuda") for _ in range(64)]
        s.synchronize()
        for _ in range(3):
            out.fill_(7.0)
            g.replay()
        s.synchronize()
    assert torch.equal(out, want)
    assert all((x == 5).all() for x in others)
    assert torch.equal(big, w.w4a16_tree_attention(**large))


def test_graphs_of_one_stream_may_run_side_by_side(w):
    a, b = attention_case(w, 1, 5), attention_case(w, 5, 6)
    want = [w.w4a16_tree_attention(**a), w.w4a16_tree_attention(**b)]
    torch.cuda.synchronize()
    graphs = [captured(w, a), captured(w, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(50):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (g, out), ref in zip(graphs, want):
        assert torch.equal(out, ref)


def test_layer_and_attention_in_one_graph(w):
    """A stream-K product and the attention captured together, then eager calls of both, then the replay."""
    import synth
    from tests._util import case_tensors
    c = synth.make_case(512, 4096, 1024, 128, "bf16", asym=True, seed=2)
    t = case_tensors(c)
    dev = attention_case(w, 40, 7)
    first = w.w4a16_gemm(t["a"], t["b_q"], t["scales"], t["qzeros"], c.G, 8)
    want = w.w4a16_tree_attention(**dev)
    out = torch.empty_like(first)
    att = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(2):
            w.w4a16_gemm(t["a"], t["b_q"], t["scales"], t["qzeros"], c.G, 8, out=out)
            w.w4a16_tree_attention(out=att, **dev)
    for _ in range(3):
        out.zero_()
        att.zero_()
        assert torch.equal(w.w4a16_tree_attention(**dev), want)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(att, want)


@pytest.mark.parametrize("n", [1, 40])
def test_a_workspace_of_the_caller(w, n):
    dev = attention_case(w, n, 8)
    want = w.w4a16_tree_attention(**dev)
    need = w.w4a16_tree_attention_workspace_size(dev["max_q"], 8, 2, 128)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert torch.equal(w.w4a16_tree_attention(workspace=ws, **dev), want)
        assert (ws[:4096] == 0).all()
    with pytest.raises(ValueError, match="workspace"):
        w.w4a16_tree_attention(workspace=ws.view(torch.int32), **dev)


FRESH = """
import sys
import torch
import w4a16_int4_weight_group_gb300 as w
T, HQ, HK, D = 5, 8, 2, {D}
g = torch.Generator().manual_seed(0)
qkv = torch.randn(T, HQ + 2 * HK, D, generator=g).to(torch.bfloat16).cuda()
q, k, v = qkv.split([HQ, HK, HK], 1)
cache = w.w4a16_kv_cache(8, HK, D, 64, 4)
slots, pos, table = torch.arange(T, device="cuda") + 400, torch.arange(T, device="cuda"), w.w4a16_rope_table(16, D)
pages = torch.arange(8, dtype=torch.int32, device="cuda")[None]
lens, start = torch.tensor([405], dtype=torch.int32, device="cuda"), torch.tensor([0, T], dtype=torch.int32, device="cuda")
logits = torch.randn(T, 5000, generator=g).cuda()
def step():
    x = w.w4a16_rope(q, pos, table)
    y = w.w4a16_kv_write(k, v, cache, slots, q=q, positions=pos, table=table)
    a, l = w.w4a16_tree_attention(y, cache, pages, lens, q_start=start, max_q={max_q}, return_lse=True)
    return [x, y, a, l, *w.w4a16_kv_read(cache, slots, D, torch.bfloat16), *w.w4a16_token_logprobs(logits, pos, 3)]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
kept, want = cache.clone(), step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(kept, cache) and w.w4a16_get_device_error() == 0
print("equal")
"""


@pytest.mark.parametrize("D,max_q", [(64, 5), (128, 5), (256, 5), (64, 40), (128, 40)])
def test_the_first_calls_of_a_process_may_be_captured(w, D, max_q):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FRESH.format(D=D, max_q=max_q)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stdout + r.stderr
