"""Strides of dimensions of one element, which a view may have at any value: the results of contiguous tensors, bit for bit."""
import pytest
import torch

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


def odd(x, stride):
    """x with `stride` for its dimensions of one element."""
    return x.as_strided(x.shape, [stride if n == 1 else s for n, s in zip(x.shape[:2], x.stride()[:2])] + [1])


@pytest.mark.parametrize("T,H", [(5, 1), (1, 4), (1, 1)])
@pytest.mark.parametrize("stride", [0, 3, 129])
def test_odd_strides_of_one_element(w, T, H, stride):
    g = torch.Generator().manual_seed(T + H)
    x = torch.randn(T, H, 128, generator=g).to(torch.bfloat16).cuda()
    pos, table = torch.arange(T, device="cuda") + 2, w.w4a16_rope_table(20, 128)
    want = w.w4a16_rope(x, pos, table)
    assert torch.equal(w.w4a16_rope(odd(x, stride), pos, table), want)
    y = odd(x.clone(), stride)
    assert torch.equal(w.w4a16_rope(y, pos, table, out=odd(y, stride + 1)), want)  # in place: only the strides that count
    slots = torch.arange(T, device="cuda")
    caches = [w.w4a16_kv_cache(1, H, 128, 16, 4) for _ in range(2)]
    qs = [w.w4a16_kv_write(k, k, c, slots, q=k, positions=pos, table=table) for k, c in ((x, caches[0]), (odd(x, stride), caches[1]))]
    assert torch.equal(*caches) and torch.equal(*qs) and torch.equal(qs[0], want)
    args = (caches[0], torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.full((T,), T, dtype=torch.int32, device="cuda"))
    assert torch.equal(w.w4a16_tree_attention(odd(x, stride), *args), w.w4a16_tree_attention(x, *args))
