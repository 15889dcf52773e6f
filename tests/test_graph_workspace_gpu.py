"""A graph captured with the default workspace, replayed after larger calls on the
same stream have replaced that workspace."""
import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
from test_call_streams_gpu import DEV, LARGE, SMALL, batch, built  # noqa: F401

pytestmark = pytest.mark.gpu


def _forward(args, kw, out):
    pa.forward(*args, out=out, **kw)


def _cascade(args, kw, out):
    pa.cascade_forward(*args, out=out, common_prefix_len=32, **kw)


@pytest.mark.parametrize("call", [_forward, _cascade])
@pytest.mark.parametrize("warm", [True, False])  # False: the capture allocates it
def test_replay_after_the_default_workspace_has_grown(call, warm):
    pa._default_ws.clear()
    s = torch.cuda.Stream(DEV)
    args, kw = batch(SMALL)
    kw["num_splits"] = 4
    out = torch.empty_like(args[0])
    big, big_kw = batch(LARGE, seed=2)
    call(args, kw, out)  # (on another stream: the library's one-time set-up)
    want = out.clone()
    torch.cuda.synchronize()
    if warm:
        with torch.cuda.stream(s):
            call(args, kw, out)
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(args, kw, out)
    captured = pa.forward.last_ext
    at, size = captured.workspace, captured.workspace_bytes
    del captured  # (it holds the buffer too)
    with torch.cuda.stream(s):
        big_out = torch.empty_like(big[0])
        call(big, big_kw, big_out)
        assert pa.forward.last_ext.workspace != at
        # what the allocator hands out next
        others = [torch.full((size,), 0x5A, dtype=torch.uint8, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    assert not [x for x in others if x.data_ptr() < at + size and at < x.data_ptr() + size]
    for _ in range(3):
        out.fill_(float("nan"))
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all(bool((x == 0x5A).all()) for x in others)
