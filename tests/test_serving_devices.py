"""The serving operators' calls run with their tensors' device as the current one (host-side logic with a recorder in the
place of the library's calls, no GPU)."""
import contextlib

import pytest
import torch

HERE = -1  # what CPU tensors say of their device


@pytest.fixture
def s(monkeypatch):
    from w4a16_int4_weight_group_gb300 import build
    build.build()
    import w4a16_int4_weight_group_gb300 as mod
    mod.lib()
    from w4a16_int4_weight_group_gb300 import serving

    class State:
        current, entered, calls, sizes = 5, [], [], []

    @contextlib.contextmanager
    def device(d):
        before, State.current = State.current, d
        State.entered.append(d)
        try:
            yield
        finally:
            State.current = before

    class Calls:
        def __getattr__(self, name):
            def call(*a):
                State.calls.append((name, State.current))
                return 0
            return call

    def size(*a):
        State.sizes.append(State.current)
        return 64

    State.entered, State.calls, State.sizes = [], [], []
    monkeypatch.setattr(serving, "_device", lambda t: t.get_device())
    monkeypatch.setattr(serving, "_current_device", lambda: State.current, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(serving, "_calls", Calls())
    monkeypatch.setattr(serving, "_current_stream", lambda dev: 0)
    monkeypatch.setattr(serving, "w4a16_tree_attention_workspace_size", size)
    monkeypatch.setattr(serving, "workspace_for", lambda device, stream, n: torch.zeros(n, dtype=torch.uint8))
    monkeypatch.setattr(serving, "_attention_ws", {})
    serving.state = State
    return serving


def arguments(s):
    x = torch.zeros(3, 2, 64, dtype=torch.float16)
    pos = torch.zeros(3, dtype=torch.int64)
    cache = torch.zeros(2, 2, 1, 1152, dtype=torch.uint8)
    return [
        (s.w4a16_rope, "rope", (x, pos, torch.zeros(8, 64)), {}),
        (s.w4a16_kv_write, "kv_write", (x, x, cache, pos), {}),
        (s.w4a16_kv_write, "kv_write", (x, x, cache, pos), dict(q=x, positions=pos, table=torch.zeros(8, 64))),
        (s.w4a16_kv_read, "kv_read", (cache, pos, 64, torch.float16), {}),
        (s.w4a16_tree_attention, "tree_attention", (x, cache, torch.zeros(3, 1, dtype=torch.int32), torch.ones(3, dtype=torch.int32)),
         dict(return_lse=True)),
        (s.w4a16_token_logprobs, "token_logprobs", (torch.zeros(2, 10, dtype=torch.float16), torch.zeros(2, dtype=torch.int64), 3), {}),
    ]


@pytest.mark.parametrize("i", range(6))
def test_calls_run_on_the_tensors_device(s, i):
    fn, name, args, kw = arguments(s)[i]
    fn(*args, **kw)  # device 5 is the current one
    assert s.state.calls == [(name, HERE)] and s.state.entered == [HERE] and s.state.current == 5
    assert all(d == HERE for d in s.state.sizes)
    s.state.current = HERE
    fn(*args, **kw)  # nothing to change
    assert s.state.calls == [(name, HERE)] * 2 and s.state.entered == [HERE]


def test_results_pass_through(s):
    fn, _, args, kw = arguments(s)[4]
    out, lse = fn(*args, **kw)
    assert out.shape == (3, 2, 64) and lse.shape == (3, 2)
    out = torch.zeros(3, 2, 64, dtype=torch.float16)
    x, pos, table = arguments(s)[0][2]
    assert s.w4a16_rope(x, pos, table, out=out) is out
