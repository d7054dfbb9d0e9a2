"""Verification at high temperatures over rows masked with finite values far below the others (GB300)."""
import math

import pytest
import torch

from tests._serving import DT
from tests.test_step_gpu import check_verify, make_verify

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


@pytest.mark.parametrize("temperature", [0.7, 150.0, 1000.0, 3.0e4, 1.0e6, 1.0e30])
@pytest.mark.parametrize("dtype,low", [("f16", -65504.0), ("bf16", -1.0e9), ("f32", -1.0e5), ("f32", torch.finfo(torch.float32).min), ("f32", -math.inf)])
def test_masked_blocks_count_what_they_weigh(w, dtype, low, temperature):
    """All but a few tokens of a row are masked, whole blocks in front, so that most threads' running maximum starts there: in the row's
    probabilities they count exp(low / T), next to nothing or next to one. (check_verify's tolerance: exponents, sums and products of
    fp32, whatever the temperature.)"""
    for V, at in ((60000, slice(-50, None)), (20011, slice(11000, 11040)), (700, slice(3, 40))):
        c = make_verify([3, 1], V, dtype, False, False, seed=V + 1, temps=[temperature, temperature])
        keep = torch.randn(4, 50, generator=torch.Generator().manual_seed(V))
        c["logits"][:] = torch.tensor(low).to(DT.get(dtype, torch.float32))
        part = c["logits"][:, at]
        part.copy_(3 * keep[:, :part.shape[1]])
        c["tokens"] = torch.tensor([0, V - 1 if at.start < 0 else at.start, V - 2 if at.start < 0 else at.start + 1, 0])
        check_verify(w, c)
