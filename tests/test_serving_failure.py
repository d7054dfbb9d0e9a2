"""Bounded waits of the attention that run out while a CTA holds parts of several sequences: the status is reported, every
CTA ends, and the calls after it are right. (The waits run out on a barrier that nothing arrives on; no GPU fault.)"""
import pytest
import torch

from tests.test_serving_gpu import check_attention, make_attention

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


@pytest.mark.parametrize("n,G,D,bits", [(20, 4, 128, 4), (20, 4, 64, 8), (2, 4, 128, 8)])
@pytest.mark.parametrize("workspace", [True, False])
def test_attention_gives_up_shares_of_many_segments(w, n, G, D, bits, workspace):
    # 16 sequences of up to seven units of 128 tokens on 4 heads: about three units a CTA, so that its share begins and ends
    # inside a sequence's tokens and holds the whole of others
    lens = [(37 * i) % 800 + 60 for i in range(16)]
    a, meta = make_attention(w, D, bits, "bf16", 32, 4, G, lens, [n] * 16, tree=True, seed=9)
    dev = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in a.items()}
    kw = {} if workspace else dict(workspace=torch.zeros(0, dtype=torch.uint8, device="cuda"))
    want = w.w4a16_tree_attention(**dev, **kw)
    torch.cuda.synchronize()
    assert w.w4a16_get_device_error() == 0
    try:
        w.w4a16_debug_set_wait_limit_ns(2_000_000)
        w.w4a16_debug_inject_stall(True)
        for _ in range(3):
            w.w4a16_tree_attention(**dev, **kw)
        torch.cuda.synchronize()
        assert w.w4a16_get_device_error() == 5  # W4A16_ERR_TIMEOUT
    finally:
        w.w4a16_debug_inject_stall(False)
        w.w4a16_debug_set_wait_limit_ns(0)
    assert w.w4a16_get_device_error() == 0
    assert torch.equal(w.w4a16_tree_attention(**dev, **kw), want)
    check_attention(w, a, meta, "bf16", **kw)
