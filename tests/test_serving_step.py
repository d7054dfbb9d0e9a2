"""The serving operators together: decoding with trees of drafted tokens gives the tokens of decoding one by one, and
failure detection of the attention kernels' bounded waits (no GPU fault: a wait on a barrier that nothing arrives on
runs out and is reported)."""
import importlib.util
import os

import pytest
import torch

from tests import _serving as plain
from tests.test_serving_gpu import check_attention, make_attention

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def w():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_weight_group_gb300 import build
    build.build()
    import w4a16_int4_weight_group_gb300 as mod
    mod.lib()
    return mod


@pytest.fixture(scope="module")
def example(w):
    spec = importlib.util.spec_from_file_location("speculative_decode", os.path.join(ROOT, "examples", "speculative_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_tree_decoding_agrees_with_decoding_one_by_one(w, example):
    prompt = torch.randint(0, 2048, (70,), generator=torch.Generator().manual_seed(3)).tolist()
    one, none = example.decode(example.Decoder(seed=4), prompt, 24, lambda tokens: [])
    assert none == [0] * 24

    def draft(tokens):
        tree, parent = [], -1
        for t in one[len(tokens):len(tokens) + 5]:
            tree += [(parent, (t + 1) % 2048), (parent, t), (parent, (t + 7) % 2048)]
            parent = len(tree) - 2
        return tree

    model = example.Decoder(seed=4)
    fast, accepted = example.decode(model, prompt, 24, draft)
    assert len(accepted) <= 8 and sum(accepted) >= 16
    # greedy choices may differ only where two logits nearly tie: the tokens are the best ones, or within rounding of them,
    # of a model that reads them one by one
    check = example.Decoder(seed=4)
    for at in range(len(prompt) - 1):
        check.step(torch.tensor([fast[at]], device="cuda"), torch.tensor([at], device="cuda"), at, None)
    for at in range(len(prompt) - 1, len(fast) - 1):
        logits, _ = check.step(torch.tensor([fast[at]], device="cuda"), torch.tensor([at], device="cuda"), at, None)
        lp, _, _, top = w.w4a16_token_logprobs(logits, torch.tensor([fast[at + 1]], device="cuda"), 1)
        assert float(top[0, 0] - lp[0]) < 0.1
    assert w.w4a16_get_device_error() == 0


@pytest.mark.parametrize("n,G,D,bits", [(1, 4, 128, 4), (3, 8, 64, 8), (40, 4, 128, 4)])
def test_attention_bounded_wait_reports_timeout_and_recovers(w, n, G, D, bits):
    a, meta = make_attention(w, D, bits, "bf16", 32, 2, G, [900, 70], [n, n], tree=n > 1, seed=5)
    dev = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in a.items()}
    assert w.w4a16_get_device_error() == 0
    try:
        w.w4a16_debug_set_wait_limit_ns(5_000_000)
        w.w4a16_debug_inject_stall(True)
        w.w4a16_tree_attention(**dev)
        torch.cuda.synchronize()
        assert w.w4a16_get_device_error() == 5        # W4A16_ERR_TIMEOUT
    finally:
        w.w4a16_debug_inject_stall(False)
        w.w4a16_debug_set_wait_limit_ns(0)
    assert w.w4a16_get_device_error() == 0
    check_attention(w, a, meta, "bf16")


def test_attention_shares_its_workspace_with_the_layer(w):
    """Calls of the linear layer (stream-K, which keeps flags in the workspace) and of the attention in turn on one stream."""
    import synth
    from tests._util import case_tensors
    c = synth.make_case(512, 4096, 1024, 128, "bf16", asym=True, seed=2)
    t = case_tensors(c)
    a, meta = make_attention(w, 128, 4, "bf16", 32, 2, 4, [1500, 700], [3, 30], tree=True, seed=6)
    first = w.w4a16_gemm(t["a"], t["b_q"], t["scales"], t["qzeros"], c.G, 8)
    o1, _ = check_attention(w, a, meta, "bf16")
    for _ in range(3):
        assert torch.equal(w.w4a16_gemm(t["a"], t["b_q"], t["scales"], t["qzeros"], c.G, 8), first)
        o2, _ = check_attention(w, a, meta, "bf16")
        assert torch.equal(o1, o2)
    for ws in w._workspaces.values():
        assert (ws[:4096] == 0).all()


def test_attention_of_many_sequences(w):
    """More sequences than threads of a CTA, lengths from nothing to a few pages, shares that span many of them."""
    g = torch.Generator().manual_seed(11)
    lens = torch.randint(0, 40, (700,), generator=g).tolist()
    a, meta = make_attention(w, 64, 8, "f16", 16, 1, 2, lens, [1] * 700, tree=False, seed=7)
    check_attention(w, a, meta, "f16")
    a["q_start"] = None
    a["max_q"] = 1
    D, bits, dt, page = meta
    dev = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in a.items()}
    out = w.w4a16_tree_attention(**dev)
    ref, _, mag, _ = plain.attend(a["q"], a["cache"].cpu(), a["page_table"], a["kv_lens"], None, None, D ** -0.5, D, bits, dt, page)
    assert ((out.cpu().double() - ref).abs() <= 2.0 ** -9 * mag + 2.0 ** -20).all()


def test_attention_query_tokens_past_max_q_and_unowned_rows_stay(w):
    a, meta = make_attention(w, 128, 4, "bf16", 16, 1, 4, [50, 60], [5, 2], tree=False, seed=8)
    dev = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in a.items()}
    dev["q_start"] = torch.tensor([0, 5, 6], dtype=torch.int32, device="cuda")  # row 6 belongs to no sequence
    out = torch.full_like(dev["q"], 7.0)
    dev["max_q"] = 3
    w.w4a16_tree_attention(out=out, **dev)
    assert (out[3:5] == 7.0).all() and (out[6] == 7.0).all()
    D, bits, dt, page = meta
    ref, _, mag, dots = plain.attend(a["q"], a["cache"].cpu(), a["page_table"], a["kv_lens"], torch.tensor([0, 5, 6]), None, D ** -0.5, D,
                                     bits, dt, page)
    tol = (2.0 ** -11 + 2 * (D + 8) * 2.0 ** -24 * dots + 60 * 2.0 ** -23)[..., None] * mag + plain.HALF_ULP["bf16"] * ref.abs()
    rows = [0, 1, 2, 5]
    assert ((out.cpu().double() - ref).abs() <= tol)[rows].all()
