"""``stream=``: what a call allocates belongs to the stream that it runs on, so
that the allocator orders the memory's next use behind the call."""
import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H, HKV, D, BS, NB = 8, 2, 128, 16, 64


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_varlen_attention_attn_gb300 import _build
    _build.build()
    pa.load()


def owner(address):
    """The stream whose pool of torch's allocator holds a device address."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= address < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not an address of the allocator's")


def batch(reqs, seed=1):
    """Tensors and arguments of an attention call over requests (q, s)."""
    g = torch.Generator().manual_seed(seed)
    T = sum(q for q, _ in reqs)
    width = max((s + BS - 1) // BS for _, s in reqs)
    bt = torch.stack([torch.randperm(NB, generator=g)[:width] for _ in reqs]).int()
    bt[:, :2] = bt[0, :2]  # a shared prefix, for the cascade
    args = [torch.randn(T, H, D, generator=g).bfloat16(),
            torch.randn(2, NB, BS, HKV, D, generator=g).bfloat16(), bt,
            torch.tensor([s for _, s in reqs], dtype=torch.int32),
            torch.tensor([0] + [q for q, _ in reqs], dtype=torch.int32).cumsum(0).int()]
    kw = dict(scale=D ** -0.5, num_heads=H, num_kv_heads=HKV, head_size=D, block_size=BS,
              max_query_len=max(q for q, _ in reqs), max_seq_len=max(s for _, s in reqs))
    return [x.to(DEV) for x in args], kw


SMALL = [(1, 100), (3, 90)]
LARGE = [(1, 700)] * 20 + [(40, 600)] * 3


def side_stream():
    s = torch.cuda.Stream(DEV)
    s.wait_stream(torch.cuda.current_stream())
    assert s != torch.cuda.current_stream()
    return s


def call_forward(stream, reqs=SMALL, **kw):
    args, base = batch(reqs)
    return [pa.forward(*args, stream=stream, **base, **kw)]


def call_cascade(stream, reqs=SMALL, **kw):
    args, base = batch(reqs)
    return [pa.cascade_forward(*args, common_prefix_len=2 * BS, stream=stream, **base, **kw)]


def call_rope(stream):
    g = torch.Generator().manual_seed(3)
    q, k, v = torch.randn(5, H + 2 * HKV, D, generator=g).bfloat16().to(DEV).split([H, HKV, HKV], 1)
    cache = torch.zeros(2, NB, BS, HKV, D, dtype=torch.bfloat16, device=DEV)
    at = torch.arange(5, device=DEV)
    return [pa.rope_and_cache(q, k, v, cache, at, at, torch.ones(8, D, device=DEV), block_size=BS,
                              stream=stream)]


def call_gather(stream):
    cache = torch.ones(2, NB, BS, HKV, D, dtype=torch.bfloat16, device=DEV)
    bt = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    return list(pa.gather_cache(cache, bt, torch.tensor([0, 20, 30], dtype=torch.int32, device=DEV),
                                num_rows=30, block_size=BS, stream=stream))


@pytest.mark.parametrize("call", [call_forward, call_cascade, call_rope, call_gather])
def test_outputs_belong_to_the_calls_stream(call):
    s = side_stream()
    got = call(s)
    s.synchronize()
    assert [owner(x.data_ptr()) for x in got] == [s.cuda_stream] * len(got)
    for x, y in zip(got, call(None)):
        assert owner(y.data_ptr()) == torch.cuda.current_stream().cuda_stream
        assert torch.equal(x, y)


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("call", [call_forward, call_cascade])
def test_a_workspace_belongs_to_the_calls_stream_also_when_it_grows(call, own):
    s = side_stream()
    kw = {"workspace": pa.Workspace()} if own else {}
    pa._default_ws.clear()  # (the stream may have served another test)
    before = 0
    for reqs in (SMALL, LARGE):
        got = call(s, reqs, **kw)
        s.synchronize()
        ext = pa.forward.last_ext
        assert owner(ext.workspace) == s.cuda_stream
        assert ext.workspace_bytes > before
        before = ext.workspace_bytes
        assert torch.equal(got[0], call(None, reqs)[0])


def test_a_workspace_of_several_streams_keeps_the_buffer_it_replaces():
    """Its memory is no other tensor's while a call on the second stream may use it."""
    ws = pa.Workspace()
    call_forward(None, workspace=ws)
    a, size = ws.buf.data_ptr(), ws.buf.numel()
    call_forward(side_stream(), workspace=ws)
    assert ws.buf.data_ptr() == a
    call_forward(None, LARGE, workspace=ws)
    b = ws.buf.data_ptr()
    assert b != a
    others = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(8)]
    assert a not in [x.data_ptr() for x in others]
    torch.cuda.synchronize()
