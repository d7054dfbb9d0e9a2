"""The adapters' form on tcgen05 in CUDA graphs, as a process's first call, on streams beside other kernels with tensor memory, from
several host threads, and in a workspace of the caller's (GB300)."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from tests.test_serving_gpu import make_attention
from tests.test_step_gpu import check_lora, cuda, make_lora

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# tokens, K, N, rank, adapters: one piece of 64 ranks and two, K split over a cluster and not
SIZES = [(1500, 520, 3608, 40, 5, "bf16"), (700, 200, 3904, 128, 3, "bf16"), (1300, 2600, 1504, 64, 2, "f16"), (300, 4104, 136, 72, 2, "f16")]


@pytest.fixture(scope="module")
def w():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_weight_group_gb300 import build
    build.build()
    import w4a16_int4_weight_group_gb300 as mod
    mod.lib()
    return mod


def inputs(seed=0):
    return [make_lora(*size, seed=seed + i) for i, size in enumerate(SIZES)]


def captured(w, calls):
    """The outputs' places and the graph of the calls, whose first ones these may be."""
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = [w.w4a16_lora(**c) for c in calls]
    return g, out


def test_captured_and_replayed_with_other_inputs(w):
    c = inputs()
    d = [cuda(x) for x in c]
    g, got = captured(w, d)
    for _ in range(2):  # the eager calls' buffers are others
        w.w4a16_lora(**cuda(make_lora(3000, 64, 4040, 48, 9, "bf16", seed=1)))
    g.replay()
    torch.cuda.synchronize()
    for x, size, y in zip(c, SIZES, got):
        check_lora(w, x, size[5], y)
    for x, y in zip(inputs(seed=50), d):
        for name, t in y.items():
            t.copy_(x[name])
    # a second graph, replayed in turn with the first: each has a workspace of its own
    h, others = captured(w, [cuda(x) for x in c])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for s, graph in zip(streams, (g, h)):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for x, size, y in zip(inputs(seed=50), SIZES, got):
        check_lora(w, x, size[5], y)
    for x, size, y in zip(c, SIZES, others):
        check_lora(w, x, size[5], y)
    assert w.w4a16_get_device_error() == 0


FRESH = """
import torch
import w4a16_int4_weight_group_gb300 as w
from tests.test_step_gpu import cuda
from tests.test_step_tcgen05 import captured, inputs
d = [cuda(x) for x in inputs()]
g, got = captured(w, d)
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(x, w.w4a16_lora(**c)) for x, c in zip(got, d)) and w.w4a16_get_device_error() == 0
print("equal")
"""


def test_the_first_calls_of_a_process_may_be_captured(w):
    r = subprocess.run([sys.executable, "-c", FRESH], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stdout + r.stderr


def test_streams_beside_attention_and_the_layer(w):
    """Kernels that hold tensor memory, on three streams at once: each takes what the others leave, and nothing waits for good."""
    a, _ = make_attention(w, 128, 8, "bf16", 128, 2, 16, [700, 300], [64, 30], tree=True, seed=6)
    a = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in a.items()}
    M, K, N, group = 600, 2048, 1536, 128
    g = torch.Generator().manual_seed(1)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).cuda()
    q = torch.randint(0, 16, (K, N), generator=g, dtype=torch.uint8).cuda()
    layer = w.W4A16Linear(w.w4a16_pack(q), (torch.rand(K // group, N, generator=g) / 64).to(torch.bfloat16).cuda(), None, group)
    c = inputs()
    d = [cuda(v) for v in c]
    want = w.w4a16_tree_attention(**a), layer(x)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], [None] * 3
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = [w.w4a16_lora(**v) if j % 2 else (w.w4a16_tree_attention(**a), w.w4a16_lora(**v), layer(x))[1] for j, v in enumerate(d)]
                got[i] += [w.w4a16_tree_attention(**a), layer(x)]
    torch.cuda.synchronize()
    for out in got:
        assert torch.equal(out[-2], want[0]) and torch.equal(out[-1], want[1])
        assert all(torch.equal(y, z) for y, z in zip(out, got[0]))
    for v, size, y in zip(c, SIZES, got[0]):
        check_lora(w, v, size[5], y)
    assert w.w4a16_get_device_error() == 0


def test_host_threads(w):
    c = inputs(seed=7)
    d = [cuda(x) for x in c]
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got[i] = w.w4a16_lora(**d[i])
            s.synchronize()
        except Exception as e:  # (told by the main thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(d))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for i, size in enumerate(SIZES):
        check_lora(w, c[i], size[5], got[i])


@pytest.mark.parametrize("size", SIZES)
def test_a_workspace_of_exactly_what_is_needed(w, size):
    c = cuda(make_lora(*size, seed=9))
    need = w.w4a16_lora_workspace_size(size[0], size[3], size[4])
    ws = torch.full((need + 1024,), 255, dtype=torch.uint8, device="cuda")
    out = w.w4a16_lora(**c, workspace=ws[:need])
    assert torch.equal(out, w.w4a16_lora(**c))
    assert (ws[:4096] == 255).all() and (ws[need:] == 255).all()
    with pytest.raises(w.W4A16Error, match="needed"):
        w.w4a16_lora(**c, workspace=ws[:need - 1])
