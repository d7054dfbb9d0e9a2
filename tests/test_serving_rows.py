"""Rows of the attention's outputs that no sequence computes: NaN in tensors that the call makes, untouched in given ones."""
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


def run(w, dev, computed, **kw):
    """Calls with outputs of the call's own, over memory that held zeros, and with given ones: the same bits in the rows that are
    computed, in the others NaN and what was there."""
    total, Hq, _ = dev["q"].shape
    given = torch.full_like(dev["q"], 3.0)
    w.w4a16_tree_attention(out=given, **dev, **kw)
    zeros = [torch.zeros_like(dev["q"]), torch.zeros(total, Hq, device="cuda")]
    del zeros  # the allocator hands these out next
    out, lse = w.w4a16_tree_attention(return_lse=True, **dev, **kw)
    torch.cuda.synchronize()
    assert w.w4a16_get_device_error() == 0
    rows = torch.zeros(total, dtype=torch.bool)
    rows[computed] = True
    assert torch.equal(out[rows], given[rows]) and torch.isfinite(out[rows]).all() and torch.isfinite(lse[rows]).all()
    assert torch.isnan(out[~rows]).all() and torch.isnan(lse[~rows]).all()
    assert (given[~rows] == 3.0).all()


def inputs(w, lens, ns, total, starts, D=128, bits=4, G=4):
    a, _ = make_attention(w, D, bits, "bf16", 16, 2, G, lens, ns, tree=False, seed=5)
    dev = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in a.items()}
    dev["q"] = torch.randn(total, 2 * G, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    dev["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    return dev


@pytest.mark.parametrize("D,bits", [(64, 8), (128, 4), (256, 8)])
def test_more_query_tokens_than_a_call_takes(w, D, bits):
    dev = inputs(w, [200, 90, 150], [70, 3, 66], 139, [0, 70, 73, 139], D, bits)
    del dev["max_q"]  # 64 unless given
    run(w, dev, [*range(64), *range(70, 73), *range(73, 137)])


@pytest.mark.parametrize("max_q", [1, 3, 20])
@pytest.mark.parametrize("G", [1, 4])
def test_rows_outside_the_sequences(w, max_q, G):
    dev = inputs(w, [50, 60, 33], [4, 1, 7], 17, [2, 6, 7, 14], G=G)
    dev["max_q"] = max_q
    run(w, dev, [*range(2, 2 + min(4, max_q)), 6, *range(7, 7 + min(7, max_q))])


def test_sequences_whose_ends_are_no_rows(w):
    dev = inputs(w, [50, 60], [5, 5], 9, [0, 5, 30])
    dev["max_q"] = 5
    run(w, dev, range(5))
    dev["q_start"] = torch.tensor([-4, 5, 9], dtype=torch.int32, device="cuda")
    run(w, dev, range(5, 9))


def test_more_sequences_than_ctas(w):
    ns = [1 + i % 3 for i in range(400)]
    starts = [sum(ns[:i]) for i in range(401)]
    dev = inputs(w, [20] * 400, ns, starts[-1] + 5, starts, D=64)
    dev["max_q"] = 2
    run(w, dev, [r for i, n in enumerate(ns) for r in range(starts[i], starts[i] + min(n, 2))])


def test_no_sequences_at_all(w):
    dev = inputs(w, [20], [3], 3, [0])
    dev["page_table"], dev["kv_lens"] = dev["page_table"][:0], dev["kv_lens"][:0]
    dev["max_q"] = 3
    run(w, dev, [])


def test_without_q_start_every_row_is_computed(w):
    dev = inputs(w, [20, 40, 60], [1, 1, 1], 3, [0, 1, 2, 3])
    dev["q_start"], dev["max_q"] = None, None
    run(w, dev, range(3))


@pytest.mark.parametrize("max_q", [2, 64])
def test_a_prompt_that_is_far_too_long(w, max_q):
    dev = inputs(w, [20000], [1], 20000, [0, 20000])
    dev["max_q"] = max_q
    run(w, dev, range(max_q))
