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
