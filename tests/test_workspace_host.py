"""Default and explicit workspaces, without a GPU."""
import weakref

import pytest

import paged_varlen_attention_attn_gb300 as pa


@pytest.mark.parametrize("captured", [False, True])
def test_a_buffer_in_a_captured_graph_is_not_given_back(monkeypatch, captured):
    """The graph's replays write to its address after a larger call has replaced it."""
    ws = pa.Workspace()
    first = weakref.ref(ws.get(1000, "cpu"))
    monkeypatch.setattr(pa, "_capturing", lambda raw: captured, raising=False)
    ws.used_on(0)
    monkeypatch.setattr(pa, "_capturing", lambda raw: False, raising=False)
    ws.used_on(0)
    second = weakref.ref(ws.get(5000, "cpu"))
    assert ws.buf.numel() >= 5000
    assert (first() is not None) == captured
    ws.get(9000, "cpu")
    assert second() is None  # no graph has used this one
    assert (first() is not None) == captured
    del ws
    assert first() is None
