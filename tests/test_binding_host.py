"""The binding's handling of its arguments, with a library that records its calls
(no GPU)."""
import ctypes
import weakref

import numpy as np
import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa

NEED = 4096


class Library:
    """Answers like libpattn's entry points and keeps what it was called with."""

    def __init__(self):
        self.calls = []

    def pattn_workspace_bytes(self, *args):
        self.calls.append(("pattn_workspace_bytes", args))
        return NEED

    def pattn_varlen_fwd(self, *args):
        self.calls.append(("pattn_varlen_fwd", args))
        return 0 if args[-1].workspace_bytes >= NEED else 3


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(pa, "load", lambda path=None: lib)
    monkeypatch.setattr(pa, "_raw_stream", lambda stream, dev: 0 if stream is None else stream.cuda_stream)
    monkeypatch.setattr(pa, "_call_on", lambda dev, fn, *args: fn(*args))
    return lib


def _forward(**kw):
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    args = (q, torch.zeros(2, 5, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 3, dtype=torch.int32),
            torch.ones(2, dtype=torch.int32), torch.tensor([0, 1, 3], dtype=torch.int32))
    base = dict(scale=1.0, num_heads=4, num_kv_heads=2, head_size=64, block_size=16, max_query_len=2,
                max_seq_len=40, workspace=pa.Workspace())
    return pa.forward(*args, **{**base, **kw})


@pytest.mark.parametrize("kind", [int, float, torch.tensor, lambda x: torch.tensor(float(x))])
def test_sizes_may_be_any_number(lib, kind):
    """As int() takes them: a maximum of a float tensor, a quotient."""
    _forward(max_query_len=kind(2), max_seq_len=kind(40), num_splits=kind(3), head_size_v=kind(0))
    ext = lib.calls[-1][1][-1]
    assert (ext.max_query_len, ext.max_seq_len, ext.num_splits, ext.head_size_v) == (2, 40, 3, 0)
    assert (ext.num_seqs, ext.num_tokens, ext.max_blocks_per_seq, ext.num_blocks) == (2, 3, 3, 5)


def test_sizes_past_32_bits_are_refused(lib):
    with pytest.raises(pa.PattnError) as e:
        _forward(max_seq_len=1 << 31)
    assert e.value.status == 1


def _rope(lib, **kw):
    seen = []
    lib.pattn_rope_and_cache = lambda args: seen.append(pa.RopeArgs.from_buffer_copy(args)) or 0
    T, H, Hkv, D, NB = 4, 4, 2, 64, 3
    t = dict(q=torch.zeros(T, H, D).bfloat16(), key=torch.zeros(T, Hkv, D).bfloat16(),
             value=torch.zeros(T, Hkv, D).bfloat16(), kv_cache=torch.zeros(2, NB, 16, Hkv, D).bfloat16(),
             slot_mapping=torch.arange(T), positions=torch.arange(T), cos_sin=torch.zeros(8, D),
             block_size=16)
    pa.rope_and_cache(**{**t, **kw})
    return seen[0]


def test_rotary_sizes_may_be_any_number(lib):
    a = _rope(lib, block_size=16.0, norm_eps=1, interleaved=True)
    assert (a.block_size, a.norm_eps, a.interleaved, a.num_tokens) == (16, 1.0, 1, 4)


def test_a_norm_eps_past_fp32_arrives_as_an_infinity(lib):
    # (which the library refuses, as it does a NaN)
    assert _rope(lib, norm_eps=1e300).norm_eps == float("inf")


class _Stream:
    cuda_stream = 0


def _row_write(lib):
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pa.reshape_and_cache(x, x, torch.zeros(2, 5, 16, 2, 64, dtype=torch.bfloat16),
                         torch.zeros(3, dtype=torch.int64), block_size=16, stream=_Stream())


def _diffkv_write(lib):
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pa.reshape_and_cache_diffkv(x, x, torch.zeros(5, 16, 2, 128, dtype=torch.bfloat16),
                                torch.zeros(3, dtype=torch.int64), block_size=16, stream=_Stream())


def _cascade(lib):
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    pa.cascade_forward(q, torch.zeros(2, 5, 16, 2, 64, dtype=torch.bfloat16),
                       torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32),
                       torch.tensor([0, 1, 3], dtype=torch.int32), scale=1.0, num_heads=4,
                       num_kv_heads=2, head_size=64, block_size=16, common_prefix_len=16,
                       max_query_len=2, max_seq_len=40, workspace=pa.Workspace(), stream=_Stream())


@pytest.mark.parametrize("call,names", [
    (lambda lib: _forward(stream=_Stream()), ["pattn_workspace_bytes", "pattn_varlen_fwd"]),
    (_cascade, ["pattn_cascade_workspace_bytes", "pattn_cascade_fwd"]),
    (_row_write, ["pattn_reshape_and_cache"]),
    (_diffkv_write, ["pattn_reshape_and_cache_diffkv"])],
    ids=["forward", "cascade", "row write", "DiffKV write"])
def test_every_call_runs_with_the_tensors_device_current(lib, monkeypatch, call, names):
    """Launches, and the sizes that depend on the device's SM count."""
    current, seen = [], []

    def call_on(dev, fn, *args):
        current.append(dev)
        try:
            return fn(*args)
        finally:
            current.pop()

    def entry(name, status):
        def run(*args):
            seen.append((name, list(current)))
            return status
        return run

    monkeypatch.setattr(pa, "_call_on", call_on)
    for name in names:
        setattr(lib, name, entry(name, NEED if name.endswith("_bytes") else 0))
    call(lib)
    assert seen == [(name, [torch.device("cpu")]) for name in names]


@pytest.mark.parametrize("kind", [list, tuple, torch.tensor, np.array, lambda x: np.array(x, np.uint8),
                                  lambda x: np.array(x, np.int32)])
def test_pair_axis_may_be_any_sequence(lib, kind):
    axes = [0] * 10 + [1] * 12 + [2] * 10
    lib.pattn_rope_and_cache = lambda args: got.append(
        ctypes.string_at(pa.RopeArgs.from_buffer_copy(args).pair_axis, 32)) or 0
    got = []
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pa.rope_and_cache(x, None, None, None, None, torch.zeros(3, 4, dtype=torch.int64),
                      torch.zeros(8, 64), block_size=16, pair_axis=kind(axes))
    assert got == [bytes(axes)]
    for bad in ([0] * 31 + [-1], [0] * 31 + [256], [0] * 31):
        with pytest.raises(ValueError):
            pa.rope_and_cache(x, None, None, None, None, torch.zeros(3, 4, dtype=torch.int64),
                              torch.zeros(8, 64), block_size=16, pair_axis=bad)


@pytest.mark.parametrize("kw", [dict(key=None), dict(q=None, q_out=torch.zeros(4, 4, 64).bfloat16())])
def test_half_a_rotary_call_is_refused(lib, kw):
    # (as the C entry does: the value would not be written, the output not filled)
    with pytest.raises(ValueError, match="goes with"):
        _rope(lib, **kw)
    assert _rope(lib, key=None, value=None).key is None
    assert _rope(lib, q=None).q is None


@pytest.mark.parametrize("cascade", [False, True])
def test_a_calls_status_outlives_its_workspace(lib, cascade):
    """pattn_read_device_status reads and clears a word of the call's own buffer,
    also when a larger call has replaced it since."""
    ws, need = pa.Workspace(), [NEED]
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    args = (q, torch.zeros(2, 5, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 3, dtype=torch.int32),
            torch.ones(2, dtype=torch.int32), torch.tensor([0, 1, 3], dtype=torch.int32))
    kw = dict(scale=1.0, num_heads=4, num_kv_heads=2, head_size=64, block_size=16, max_query_len=2,
              max_seq_len=40, workspace=ws)
    lib.pattn_workspace_bytes = lambda *args: need[0]
    lib.pattn_varlen_fwd = lambda *args: 0 if args[-1].workspace_bytes >= need[0] else 3
    lib.pattn_cascade_workspace_bytes = lambda *args: need[0]
    lib.pattn_cascade_fwd = lambda *args: 0
    if cascade:
        pa.cascade_forward(*args, common_prefix_len=16, stream=_Stream(), **kw)
    else:
        pa.forward(*args, **kw)
    ext, buf = pa.forward.last_ext, weakref.ref(ws.buf)
    need[0] = 2 * NEED
    pa.forward(*args, **kw)
    assert ws.buf.numel() >= 2 * NEED and pa.forward.last_ext is not ext
    assert buf() is not None and buf().data_ptr() == ext.workspace
    del ext
    assert buf() is None


@pytest.mark.parametrize("shape", [(2, 16, 2, 2), (2, 2, 1, 2, 16), (2, 1, 2, 16, 2), (128,)])
def test_row_scales_of_another_layout_are_refused(lib, shape):
    """As many numbers, but not where the kernels read them."""
    assert torch.Size(shape).numel() == torch.Size(pa.row_scales_shape(2, 16, 2)).numel()
    scales = torch.ones(shape)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 2, 16, 2, 64, dtype=torch.uint8)
    row = dict(block_size=16, kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=scales)
    slots, bt = torch.arange(3), torch.zeros(1, 2, dtype=torch.int32)
    qsl, sl = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([3], dtype=torch.int32)
    att = dict(scale=1.0, num_heads=2, num_kv_heads=2, head_size=64, max_query_len=3, max_seq_len=32, **row)
    for call in (lambda: pa.reshape_and_cache(x, x, cache, slots, **row),
                 lambda: pa.rope_and_cache(x, x, x, cache, slots, None, None, **row),
                 lambda: pa.gather_cache(cache, bt, qsl, num_rows=3, **row),
                 lambda: pa.forward(x, cache, bt, sl, qsl, **att),
                 lambda: pa.cascade_forward(x, cache, bt, sl, qsl, common_prefix_len=16, **att)):
        with pytest.raises(ValueError, match="row_scales_shape"):
            call()
