"""Default and explicit workspaces, without a GPU."""
import threading
import time
import weakref

import pytest
import torch

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


def test_host_threads_have_default_workspaces_of_their_own():
    """Two threads' calls on one stream interleave their launches."""
    device, stream, got = torch.device("cuda", 0), 4096, []
    work = threading.Event()

    def call():
        got.append(pa._workspace(None, device, stream))
        work.wait(30)

    threads = [threading.Thread(target=call) for _ in range(2)]
    for t in threads:
        t.start()
    while len(got) < 2:
        time.sleep(0.001)
    mine = [pa._workspace(None, device, stream) for _ in range(2)]
    work.set()
    for t in threads:
        t.join()
    assert mine[0] is mine[1]
    assert len({id(w) for w in (got[0], got[1], mine[0])}) == 3
    own = pa.Workspace()
    assert pa._workspace(own, device, stream) is own


def test_default_workspaces_can_be_released():
    ws = pa._workspace(None, torch.device("cuda", 0), 4096)
    buf = weakref.ref(ws.get(1000, "cpu"))
    del ws
    assert buf() is not None
    pa.release_workspaces()
    assert buf() is None


def test_a_release_by_another_thread_disturbs_no_call(monkeypatch):
    class Released(dict):
        def __contains__(self, key):  # it is there, and gone at the next look
            return True
    monkeypatch.setattr(pa, "_default_ws", Released())
    assert isinstance(pa._workspace(None, torch.device("cuda", 0), 4096), pa.Workspace)
