"""The adapters' products between which sums cancel: what the second product takes of h has to hold all of its bits (GB300)."""
import pytest
import torch

from tests._serving import DT

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


def cancelling(T, K, N, r, n, dtype, seed):
    """h of an adapter: a 20-bit number in one place, and less its upper 12 bits, apart, in two others; B gives them the same weight, so that
    the lowest byte is left. Every product and every partial sum, in any order, is a whole number below 2^22 (with the weights and
    scales), which fp32 holds exactly: nothing may be off, whatever the order or the rounding of the sums."""
    g = torch.Generator().manual_seed(seed)
    ks, rs = [0, K // 2, K - 1], torch.stack([torch.randperm(r, generator=g)[:3] for _ in range(n)])
    high, mid, low = torch.randint(8, 16, (n,), generator=g), torch.randint(128, 256, (n,), generator=g), torch.randint(1, 256, (n,), generator=g)
    x, a, b = torch.zeros(T, K), torch.zeros(n, r, K), torch.zeros(n, N, r)
    x[:, ks[0]], x[:, ks[1:]] = 256.0, 1.0
    weight = torch.randint(-1, 2, (n, N), generator=g).float()
    for i in range(n):
        a[i, rs[i, 0], ks] = torch.stack([high[i] * 256, mid[i] * 256, low[i]]).float()
        a[i, rs[i, 1], ks[0]] = -256.0 * high[i]
        a[i, rs[i, 2], ks[1]] = -256.0 * mid[i]
        b[i][:, rs[i]] = weight[i][:, None].expand(N, 3)
    scales = torch.tensor([1.0, 2.0])[torch.randint(0, 2, (n,), generator=g)]
    ids = torch.randint(-1, n, (T,), generator=g)
    out = torch.where((ids >= 0)[:, None], (weight * (low.float() * scales)[:, None])[ids.clamp(min=0)], torch.zeros(T, N))
    d = lambda t: t.to(DT[dtype]).cuda()  # noqa: E731
    return dict(x=d(x), a=d(a), b=d(b), ids=ids.to(torch.int32).cuda(), base=d(torch.zeros(T, N)), scales=scales.cuda()), out


# every way of finding tiles and every part of the rank: ranked, counted and listed tokens, tcgen05 up to rank 64 and past it
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,K,N,r,n", [(5, 64, 72, 8, 2), (40, 2056, 136, 32, 3), (100, 200, 40, 64, 4), (70, 1000, 520, 128, 2), (300, 264, 72, 16, 5),
                                       (500, 72, 264, 32, 600), (900, 520, 136, 56, 3), (400, 264, 72, 104, 2), (1300, 72, 136, 24, 4),
                                       (1500, 264, 72, 64, 40), (1200, 200, 264, 72, 3), (2500, 136, 72, 16, 3), (3000, 264, 200, 32, 7),
                                       (1500, 4008, 136, 40, 3), (2100, 200, 3912, 64, 5), (300, 4040, 72, 72, 2), (2300, 136, 3976, 96, 3),
                                       (700, 3000, 1160, 128, 4)])
def test_h_keeps_its_bits(w, T, K, N, r, n, dtype):
    c, want = cancelling(T, K, N, r, n, dtype, seed=T + r)
    assert torch.equal(w.w4a16_lora(**c).cpu().float(), want)
