"""The attention of many query rows, and that of few, with more sequences than a warp has lanes and than a CTA has threads, and
without a workspace (every sequence whole on one CTA)."""
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


def no_workspace():
    return dict(workspace=torch.zeros(0, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("D,bits", [(64, 8), (128, 4), (128, 8), (64, 4)])
@pytest.mark.parametrize("workspace", [True, False])
def test_many_rows_of_forty_sequences(w, D, bits, workspace):
    # 80 rows a cache head; lengths from nothing to three units; each CTA's share holds several sequences
    lens = [(53 * i) % 330 for i in range(40)]
    ns = [20 if i % 3 else 1 + i % 20 for i in range(40)]
    a, meta = make_attention(w, D, bits, "bf16", 16, 2, 4, lens, ns, tree=True, seed=4)
    check_attention(w, a, meta, "bf16", **({} if workspace else no_workspace()))


@pytest.mark.parametrize("n,G,D,bits", [(20, 4, 128, 4), (20, 4, 64, 8), (64, 3, 128, 8), (2, 4, 128, 4), (9, 2, 256, 8)])
def test_without_a_workspace_several_sequences_and_heads(w, n, G, D, bits):
    lens = [1500, 0, 129, 700, 5, 1023]
    a, meta = make_attention(w, D, bits, "f16", 32, 3, G, lens, [n] * 6, tree=True, seed=2)
    check_attention(w, a, meta, "f16", **no_workspace())


@pytest.mark.parametrize("workspace", [True, False])
def test_many_rows_of_more_sequences_than_threads(w, workspace):
    g = torch.Generator().manual_seed(11)
    lens = torch.randint(0, 40, (700,), generator=g).tolist()
    a, meta = make_attention(w, 64, 8, "f16", 16, 1, 4, lens, [10] * 700, tree=False, seed=7)
    check_attention(w, a, meta, "f16", **({} if workspace else no_workspace()))
