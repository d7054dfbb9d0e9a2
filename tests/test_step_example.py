"""The example of sampled decoding where its pool of pages is too small (GB300)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_weight_group_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("sampled_decode", os.path.join(ROOT, "examples", "sampled_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def nothing(tokens):
    return []


@pytest.mark.parametrize("prompts,answers,steps", [([20], 8, 4),       # 2 pages, and 7 copies of the second one
                                                   ([20, 30], 2, 12),  # enough at first, not for the tokens that come
                                                   ([20, 17, 30, 33], 1, 2), ([20, 500], 1, 2)])  # a prompt that does not fit, or not in the table
def test_answers_that_do_not_fit_are_refused_and_their_pages_come_back(example, prompts, answers, steps):
    """No answer is told to go on over pages that others hold: the call says so, and the pool is as it was."""
    g = torch.Generator().manual_seed(1)
    make = lambda: example.Server(pages=8, seed=2)  # noqa: E731  (tables of 2 pages of 16 tokens)
    texts = [torch.randint(0, 2048, (n,), generator=g).tolist() for n in prompts]
    server = make()
    with pytest.raises(MemoryError, match="no room"):
        example.decode(server, texts, [0] * len(texts), answers, steps, nothing)
    assert not server.refs.any()
    small = [texts[0][:18]]
    got, _ = example.decode(server, small, [1], 3, 6, nothing, seed=3)
    want, _ = example.decode(make(), small, [1], 3, 6, nothing, seed=3)
    assert got == want and not server.refs.any()
