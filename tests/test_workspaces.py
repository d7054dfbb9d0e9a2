"""Workspaces that the binding keeps: calls under capture have one of their own (host-side logic, no GPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def w():
    from w4a16_int4_weight_group_gb300 import build
    build.build()
    import w4a16_int4_weight_group_gb300 as mod
    mod.lib()
    return mod


@pytest.fixture
def capture(w, monkeypatch):
    """Sets which capture the streams are said to be in; the module's buffers are put back afterwards."""
    now = {}
    monkeypatch.setattr(w, "_capture_id", lambda stream: now.get(stream, 0), raising=False)
    monkeypatch.setattr(w, "_workspaces", {})
    monkeypatch.setattr(w, "_captured", {}, raising=False)
    return now


CPU = torch.device("cpu")


def test_eager_calls_share_a_stream_s_buffer(w, capture):
    a = w.workspace_for(CPU, 7, 100)
    assert w.workspace_for(CPU, 7, 1 << 20) is a and w.workspace_for(CPU, 8, 100) is not a
    b = w.workspace_for(CPU, 7, 3 << 20)
    assert b.numel() == 3 << 20 and (b == 0).all() and w.workspace_for(CPU, 7, 100) is b


def test_every_capture_has_a_buffer_of_its_own(w, capture):
    eager = w.workspace_for(CPU, 7, 100)
    eager.fill_(1)  # (what is in it must not matter to a graph)
    capture[7] = 41
    first = w.workspace_for(CPU, 7, 100)
    assert first is not eager and (first[:4096] == 0).all()
    assert w.workspace_for(CPU, 7, 1 << 20) is first  # the same for all calls of the capture
    grown = w.workspace_for(CPU, 7, 2 << 20)
    assert grown is not first and grown.numel() == 2 << 20 and (grown[:4096] == 0).all()
    capture[7] = 42
    second = w.workspace_for(CPU, 7, 100)
    assert second is not grown and second is not first and (second[:4096] == 0).all()
    capture[9] = 42  # another stream that takes part in the capture
    assert w.workspace_for(CPU, 9, 100) is not second and w.workspace_for(CPU, 7, 100) is second
    capture.clear()
    assert w.workspace_for(CPU, 7, 100) is eager  # captures left the eager calls' buffer alone


def test_an_eager_call_never_replaces_a_captured_buffer(w, capture):
    capture[7] = 5
    held = w.workspace_for(CPU, 7, 100)
    del capture[7]
    small = w.workspace_for(CPU, 7, 100)
    large = w.workspace_for(CPU, 7, 8 << 20)
    assert held is not small and held is not large
    capture[7] = 5
    assert w.workspace_for(CPU, 7, 100) is held


def test_capture_number_without_a_capture(w):
    assert w._capture_id(0) == 0 and w._capture_id(1) == 0  # (1: the handle of the legacy default stream)
    assert [f[0] for f in w.SIGNATURES].count("w4a16_stream_capture_id") == 1
    mod = pytest.importorskip("w4a16_int4_weight_group_gb300._w4a16_call")
    with pytest.raises(TypeError):
        mod.capture_id("one")
    with pytest.raises(ValueError):
        mod.bind_capture(0)
