"""Lengths of the attention's sequences at and past their limits. A length past the page table counts as the table's end, so that
the query tokens are the last tokens of its pages (the definition in the C header)."""
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


@pytest.mark.parametrize("past", [1, 15, 16, 17, 1000, 2 ** 31 - 1 - 96])
@pytest.mark.parametrize("n,G,D,bits", [(1, 4, 128, 4), (5, 2, 64, 8), (20, 4, 128, 8), (9, 4, 256, 4)])
def test_a_length_past_the_page_table_is_its_end(w, n, G, D, bits, past):
    for tree in (False, n > 1):
        a, meta = make_attention(w, D, bits, "bf16", 48, 2, G, [96, 70], [n, n], tree=tree, seed=6)
        want, lse = check_attention(w, a, meta, "bf16")
        a["kv_lens"][0] = 96 + past
        got, other = check_attention(w, a, meta, "bf16")
        assert torch.equal(got, want) and torch.equal(other, lse)


def test_a_negative_length_is_zero(w):
    for n in (1, 20):
        a, _ = make_attention(w, 128, 4, "bf16", 16, 2, 4, [40, 60], [n, n], tree=False, seed=6)
        dev = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in a.items()}
        dev["kv_lens"][0] = -7
        out, lse = w.w4a16_tree_attention(return_lse=True, **dev)
        assert (out[:n] == 0).all() and (lse[:n] == -float("inf")).all()
        assert torch.isfinite(lse[n:]).all() and (out[n:] != 0).any()


@pytest.mark.parametrize("n", [1, 40])
def test_the_longest_sequences(w, n):
    """Lengths around 2^31, made of one page of 2^20 tokens that the table holds 2048 times: every token of the page counts 2048
    times (the last 256 of them 2047 times). The sums over so many tokens are long: `adds` fp32 sums one after the other in a
    row's longest chain, each off by at most 2^-23 of the sum so far (the tensor cores truncate)."""
    D, G, size, copies = 64, 4, 1 << 20, 2048
    g = torch.Generator(device="cuda").manual_seed(3)
    cache = w.w4a16_kv_cache(1, 1, D, size, 4)
    slots = torch.arange(size, device="cuda")
    for at in range(0, size, 1 << 17):
        k = torch.randn(1 << 17, 1, D, generator=g, device="cuda").to(torch.bfloat16)
        v = (torch.randn(1 << 17, 1, D, generator=g, device="cuda") + 1.0).to(torch.bfloat16)
        w.w4a16_kv_write(k, v, cache, slots[at:at + (1 << 17)])
    q = torch.randn(n, G, D, generator=g, device="cuda").to(torch.bfloat16)
    table = torch.zeros(1, copies, dtype=torch.int32, device="cuda")
    k, v = (x[:, 0].double() for x in w.w4a16_kv_read(cache, slots, D, torch.bfloat16))
    count = torch.full((size,), float(copies), dtype=torch.float64, device="cuda")
    count[-256:] -= 1
    s = q.double().view(-1, D) @ k.T * D ** -0.5 + count.log()
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    want, mag = (p @ v).view(n, G, D), (p @ v.abs()).view(n, G, D)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    # streaming: 2 CTAs of 8 warps an SM, a sum for each 16 tokens of a warp; tiles: a CTA an SM, two groups, two sums for each 16
    adds = (1 << 31) / 16 / (2 * sms * 8) if n == 1 else (1 << 31) / 16 / sms
    for length in (2 ** 31 - 1, 2 ** 31 - 130, 2 ** 31 - 256, 2 ** 31 - 257):
        out, got = w.w4a16_tree_attention(q, cache, table, torch.tensor([length], dtype=torch.int32, device="cuda"),
                                          q_start=torch.tensor([0, n], dtype=torch.int32, device="cuda"), max_q=n, return_lse=True)
        assert w.w4a16_get_device_error() == 0
        assert ((out.double() - want).abs() <= (2.0 ** -11 + 2 * adds * 2.0 ** -23) * mag + 2.0 ** -8 * want.abs()).all()
        assert ((got.double() - lse.view(n, G)).abs() <= 2 * adds * 2.0 ** -23 + 1e-5).all()
