"""The attention of many rows between layer calls whose kernel allocates tensor memory before it waits for its predecessor: long
chains on one stream, launched without a wait in between, outside of graphs and in one."""
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


@pytest.mark.parametrize("D,G,lens", [(64, 4, [900, 300, 4000]), (128, 4, [900]), (64, 2, [40] * 8)])
def test_attention_and_layer_in_turn(w, D, G, lens):
    import synth
    from tests._util import case_tensors
    n, Hk = 32, 2
    a, _ = make_attention(w, D, 4, "bf16", 32, Hk, G, lens, [n] * len(lens), tree=True, seed=3)
    dev = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in a.items()}
    rows = n * len(lens)
    c = synth.make_case(rows, Hk * G * D, 512, 64, "bf16", asym=True, seed=2)
    t = case_tensors(c)
    layer = w.W4A16Linear(t["b_q"], t["scales"], t["qzeros"], c.G)
    att = w.w4a16_tree_attention(**dev)
    want = layer(att.view(rows, -1))
    torch.cuda.synchronize()

    def chain():
        y = None
        for _ in range(20):
            y = layer(w.w4a16_tree_attention(**dev).view(rows, -1))
        return y

    for _ in range(5):
        assert torch.equal(chain(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = chain()
    for _ in range(5):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert w.w4a16_get_device_error() == 0
