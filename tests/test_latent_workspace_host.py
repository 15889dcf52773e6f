"""The workspace of the latent attentions, without a GPU."""
import types
import weakref

import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
from paged_varlen_attention_attn_gb300 import latent

CPU = torch.device("cpu")
STREAM = types.SimpleNamespace(cuda_stream=0)


@pytest.fixture
def plain_memory(monkeypatch):
    monkeypatch.setattr(pa, "_empty", lambda n, dtype, dev, stream: torch.empty(n, dtype=dtype, device=dev))


def test_a_replaced_buffer_is_given_back(plain_memory):
    """Another operator's larger call has replaced it: nothing holds it any longer."""
    ws = pa.Workspace()
    at, size, raw, ext = latent._scratch(ws, 1000, CPU, STREAM)
    assert (at, size, raw) == (ws.buf.data_ptr(), 1000, 0)
    assert latent._scratch(ws, 900, CPU, STREAM)[3] is ext  # looked up once
    first = weakref.ref(ws.buf)
    ws.get(5000, CPU, STREAM)
    assert first() is not None  # (the call's status may still be asked for)
    del ext
    assert first() is None
    at, size, _, ext = latent._scratch(ws, 900, CPU, STREAM)
    assert (at, size) == (ws.buf.data_ptr(), 5000)
    assert ext.workspace == at and ext.workspace_bytes == size


def test_a_call_on_another_stream_has_its_own(plain_memory, monkeypatch):
    monkeypatch.setattr(pa, "_capturing", lambda raw: False)
    ws = pa.Workspace()
    first = latent._scratch(ws, 1000, CPU, STREAM)[3]
    other = latent._scratch(ws, 1000, CPU, types.SimpleNamespace(cuda_stream=4096))[3]
    assert (first.stream, other.stream) == (None, 4096)
    assert first.workspace == other.workspace and ws._held
