"""Python binding of libpattn -- paged variable-length attention for GB300.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libpattn.so`` (built by ``_build.build()``).  There is no CPU or
PyTorch fallback; if the library is missing, ``load()`` raises.

``stream=`` of a call is the torch stream it runs on (default: the current one);
an output that the call allocates belongs to that stream, as if it were
allocated under ``torch.cuda.stream(stream)``.

The names follow the C ABI in ``include/pattn.h``:
``pattn_varlen_fwd``, ``pattn_workspace_bytes``, ``pattn_decode_splits``,
``pattn_read_device_status``, ``pattn_status_string``, ``pattn_version``.
``forward(...)`` is a convenience wrapper for torch tensors that fills the
extension struct from the tensors' shapes and allocates the workspace with
torch (plumbing; the library itself allocates nothing).
"""
import ctypes
import os
import struct
import threading

from . import _build

KV_BF16 = 0
KV_FP8_E4M3 = 1
KV_F16 = 2  # f16 cache; q and out are f16 too
KV_FP8_E4M3_ROW = 3  # e4m3 cache with one fp32 scale per (token, KV head) row
MAX_SPLITS = 64

STATUS = {0: "PATTN_OK", 1: "PATTN_ERR_INVALID_ARGUMENT", 2: "PATTN_ERR_UNSUPPORTED",
          3: "PATTN_ERR_WORKSPACE_TOO_SMALL", 4: "PATTN_ERR_CUDA",
          5: "PATTN_ERR_BAD_METADATA", 6: "PATTN_ERR_DEVICE_TIMEOUT"}

EXPORTS = ("pattn_varlen_fwd", "pattn_workspace_bytes", "pattn_decode_splits",
           "pattn_read_device_status", "pattn_status_string", "pattn_version",
           "pattn_decode_fwd_static", "pattn_reshape_and_cache",
           "pattn_reshape_and_cache_diffkv", "pattn_cascade_fwd",
           "pattn_cascade_workspace_bytes", "pattn_reshape_and_cache_rows",
           "pattn_rope_and_cache", "pattn_gather_cache")
STATIC_SCRATCH_BYTES = 32 << 20


class PattnError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}" if what else STATUS.get(status, str(status)))


class Ext(ctypes.Structure):
    """pattn_ext_t"""
    _fields_ = [("struct_size", ctypes.c_size_t), ("num_seqs", ctypes.c_int),
                ("num_tokens", ctypes.c_int), ("max_blocks_per_seq", ctypes.c_int),
                ("num_blocks", ctypes.c_int), ("max_query_len", ctypes.c_int),
                ("max_seq_len", ctypes.c_int), ("num_splits", ctypes.c_int),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("stream", ctypes.c_void_p),
                ("timing_events", ctypes.POINTER(ctypes.c_void_p)),
                ("sinks", ctypes.c_void_p), ("head_size_v", ctypes.c_int)]


class RopeArgs(ctypes.Structure):
    """pattn_rope_t"""
    _fields_ = ([("struct_size", ctypes.c_size_t)] +
                [(n, ctypes.c_void_p) for n in ("q", "q_out", "key", "value")] +
                [(n, ctypes.c_longlong) for n in ("q_stride", "q_out_stride", "key_stride",
                                                  "value_stride")] +
                [("cos_sin", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                 ("positions_stride", ctypes.c_longlong)] +
                [(n, ctypes.c_void_p) for n in ("pair_axis", "q_norm", "k_norm", "kv_cache",
                                                "row_scales", "kv_scale", "slot_mapping",
                                                "device_status", "stream")] +
                [("norm_eps", ctypes.c_float)] +
                [(n, ctypes.c_int) for n in ("num_tokens", "num_heads", "num_kv_heads",
                                             "head_size", "rot_dim", "interleaved", "num_axes",
                                             "max_position", "kv_dtype", "block_size",
                                             "num_blocks")])


def _packer(cls):
    """struct.Struct with a ctypes structure's layout: building a call's arguments
    in one step costs a quarter of setting the fields one by one."""
    codes = {ctypes.c_size_t: "N", ctypes.c_longlong: "q", ctypes.c_float: "f", ctypes.c_int: "i"}
    fmt = "@" + "".join(codes.get(t, "P") for _, t in cls._fields_)
    pad = ctypes.sizeof(cls) - struct.calcsize(fmt)
    return struct.Struct(fmt + "x" * pad)


def _pack(packer, what, *values):
    """The structure's bytes; sizes that its fields do not hold are invalid."""
    try:
        return packer.pack(*values)
    except (struct.error, OverflowError):
        raise PattnError(1, what) from None


_ROPE_PACK = _packer(RopeArgs)
_EXT_PACK = _packer(Ext)

PHASES = ("plan", "prefill", "decode", "combine")


_lib = None


def library_path():
    return _build.LIB


def load(path=None):
    """Open libpattn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB
    if not os.path.exists(p):
        raise PattnError(4, f"{p} is missing; build it with __graft_entry__.build()")
    lib = ctypes.CDLL(p)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.pattn_varlen_fwd.restype = i
    lib.pattn_varlen_fwd.argtypes = [vp, vp, vp, vp, vp, vp, f, i, i, i, i, i, i, i, vp,
                                     ctypes.POINTER(Ext)]
    lib.pattn_workspace_bytes.restype = ctypes.c_size_t
    lib.pattn_workspace_bytes.argtypes = [ctypes.POINTER(Ext), i, i, i, i]
    lib.pattn_decode_splits.restype = i
    lib.pattn_decode_splits.argtypes = [ctypes.POINTER(Ext), i, i, i, i]
    lib.pattn_read_device_status.restype = i
    lib.pattn_read_device_status.argtypes = [ctypes.POINTER(Ext)]
    lib.pattn_status_string.restype = ctypes.c_char_p
    lib.pattn_status_string.argtypes = [i]
    lib.pattn_version.restype = i
    lib.pattn_version.argtypes = []
    lib.pattn_decode_fwd_static.restype = i
    lib.pattn_decode_fwd_static.argtypes = [vp, vp, vp, vp, vp, vp, f, i, i, i, i, i, i, i, vp,
                                            i, i, i, i, i, i, vp]
    lib.pattn_cascade_fwd.restype = i
    lib.pattn_cascade_fwd.argtypes = [vp, vp, vp, vp, vp, vp, f, i, i, i, i, i, i, i, vp, i,
                                      ctypes.POINTER(Ext)]
    lib.pattn_cascade_workspace_bytes.restype = ctypes.c_size_t
    lib.pattn_cascade_workspace_bytes.argtypes = [ctypes.POINTER(Ext), i, i, i, i, i]
    lib.pattn_reshape_and_cache.restype = i
    lib.pattn_reshape_and_cache.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, vp, vp, vp]
    lib.pattn_reshape_and_cache_diffkv.restype = i
    lib.pattn_reshape_and_cache_diffkv.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, vp, vp]
    lib.pattn_reshape_and_cache_rows.restype = i
    lib.pattn_reshape_and_cache_rows.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, vp, vp]
    lib.pattn_rope_and_cache.restype = i
    lib.pattn_rope_and_cache.argtypes = [vp]  # a RopeArgs by reference, or its bytes
    lib.pattn_gather_cache.restype = i
    lib.pattn_gather_cache.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, vp, vp, vp]
    if path is None:
        _lib = lib
    return lib


def _scale_arg(kv_dtype, kv_scale):
    """kv_scale as the C ABI takes it: host float[2], or for KV_FP8_E4M3_ROW the
    device address of the row scales (a tensor or its address)."""
    if kv_scale is None:
        return None
    if kv_dtype == KV_FP8_E4M3_ROW:
        return kv_scale if isinstance(kv_scale, int) else kv_scale.data_ptr()
    return (ctypes.c_float * 2)(float(kv_scale[0]), float(kv_scale[1]))


def row_scales_shape(num_blocks, block_size, num_kv_heads):
    """Shape of the fp32 row scales of a KV_FP8_E4M3_ROW cache: slot i of block b
    is scaled by scales[b, i // 16, head, 0 (K) or 1 (V), i % 16]."""
    return (num_blocks, block_size // 16, num_kv_heads, 2, 16)


def _check_row_scales(scales, num_blocks, block_size, num_kv_heads, device):
    import torch
    if (not isinstance(scales, torch.Tensor) or scales.dtype != torch.float32 or
            scales.device != device or not scales.is_contiguous() or
            scales.shape != row_scales_shape(num_blocks, block_size, num_kv_heads)):
        raise ValueError("kv_scale of a KV_FP8_E4M3_ROW cache must be a contiguous fp32 tensor of "
                         "shape row_scales_shape(...) on the cache's device")


def pattn_reshape_and_cache(key, value, kv_cache, slot_mapping, num_tokens, num_kv_heads,
                            head_size, block_size, num_blocks, kv_dtype, kv_scale,
                            device_status, stream, lib=None):
    """Raw call of the KV-cache write with integer device pointers; returns
    the status code."""
    lib = lib or load()
    ks = _scale_arg(kv_dtype, kv_scale)
    return lib.pattn_reshape_and_cache(key, value, kv_cache, slot_mapping, int(num_tokens),
                                       int(num_kv_heads), int(head_size), int(block_size),
                                       int(num_blocks), int(kv_dtype), ks,
                                       int(device_status) or None, int(stream) or None)


def reshape_and_cache(key, value, kv_cache, slot_mapping, *, block_size, kv_dtype=KV_BF16,
                      kv_scale=None, device_status=None, stream=None):
    """pattn_reshape_and_cache on torch tensors: key/value bf16 [T, Hkv, d],
    kv_cache [2, num_blocks, block_size, Hkv, d] (bf16, or uint8 e4m3 codes),
    slot_mapping int64 [T].  ``device_status``: optional int32/uint32 tensor of
    one element that collects the out-of-pool bit.  With KV_FP8_E4M3_ROW
    ``kv_scale`` is the cache's row-scale tensor, updated as well
    (pattn_reshape_and_cache_rows).  Raises PattnError."""
    import torch
    if kv_dtype == KV_FP8_E4M3_ROW:
        _check_row_scales(kv_scale, kv_cache.shape[1], block_size, key.shape[1], kv_cache.device)
        T, Hkv, D = key.shape
        dev, NB = key.device, kv_cache.shape[1]
        for name, x, shape, types in (
                ("key", key, (T, Hkv, D), (torch.bfloat16,)),
                ("value", value, (T, Hkv, D), (torch.bfloat16,)),
                ("kv_cache", kv_cache, (2, NB, block_size, Hkv, D),
                 (torch.uint8, torch.float8_e4m3fn)),
                ("slot_mapping", slot_mapping, (T,), (torch.int64,))):
            if x.shape != shape or x.dtype not in types or x.device != dev or not x.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {types[0]} tensor of shape {shape}")
        status_at = _status_at(device_status, dev)
        if T == 0:  # (an empty tensor has no address)
            return kv_cache
        st = _call_on(
            dev, load().pattn_reshape_and_cache_rows, key.data_ptr(), value.data_ptr(),
            kv_cache.data_ptr(), kv_scale.data_ptr(), slot_mapping.data_ptr(), T, Hkv, D,
            int(block_size), NB, status_at or None, _raw_stream(stream, dev))
        if st != 0:
            raise PattnError(st, "pattn_reshape_and_cache_rows")
        return kv_cache
    st = _call_on(key.device, pattn_reshape_and_cache, key.data_ptr(), value.data_ptr(),
                  kv_cache.data_ptr(), slot_mapping.data_ptr(), key.shape[0], key.shape[1],
                  key.shape[2], block_size, kv_cache.shape[1], kv_dtype, kv_scale,
                  0 if device_status is None else device_status.data_ptr(),
                  _raw_stream(stream, key.device))
    if st != 0:
        raise PattnError(st, "pattn_reshape_and_cache")
    return kv_cache


def reshape_and_cache_diffkv(key, value, kv_cache, slot_mapping, *, block_size,
                             kv_dtype=KV_BF16, device_status=None, stream=None):
    """pattn_reshape_and_cache_diffkv on torch tensors: key 16-bit [T, Hkv, dk],
    value [T, Hkv, dv], kv_cache [num_blocks, block_size, Hkv, dk + dv],
    slot_mapping int64 [T].  Raises PattnError."""
    st = _call_on(
        key.device, load().pattn_reshape_and_cache_diffkv, key.data_ptr(), value.data_ptr(),
        kv_cache.data_ptr(), slot_mapping.data_ptr(), int(key.shape[0]), int(key.shape[1]),
        int(key.shape[2]), int(value.shape[2]), int(block_size), int(kv_cache.shape[0]),
        int(kv_dtype), None if device_status is None else device_status.data_ptr(),
        _raw_stream(stream, key.device))
    if st != 0:
        raise PattnError(st, "pattn_reshape_and_cache_diffkv")
    return kv_cache


def rope_pair_axis(sections, interleaved=False):
    """The axis of each rotary pair, for rope_and_cache.  ``sections``: pairs per
    axis, e.g. (16, 24, 24).  In order, or ``interleaved``: the axes take turns
    (0, 1, 2, 0, 1, 2, ...) while each still has pairs left and pairs without a
    partner go to the first axis."""
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    n_axes, total = len(sections), sum(sections)
    out = [0] * total
    for a in range(1, n_axes):
        for p in list(range(a, total, n_axes))[:sections[a]]:
            out[p] = a
    if [out.count(a) for a in range(n_axes)] != list(sections):
        raise ValueError("sections cannot take turns")
    return out


_torch_c = None


def _torch():
    """torch's C module (bound once: torch is imported by the first call that needs
    it, and an import statement per call costs as much as a check or two)."""
    global _torch_c
    if _torch_c is None:
        from torch import _C
        _torch_c = _C
    return _torch_c


def _raw_stream(stream, dev):
    """The cudaStream_t of ``stream``, or of the device's current stream (read
    without building a Stream object: 2 us less per call)."""
    if stream is not None:
        return stream.cuda_stream
    return (_torch_c or _torch())._cuda_getCurrentRawStream(dev.index)


def _empty(shape, dtype, dev, stream):
    """torch.empty from the pool of the stream the call runs on (None: the device's
    current one), so that the allocator hands the memory to nobody before the call
    is done with it.  From another stream's pool nothing would order the two."""
    import torch
    if stream is None or stream.cuda_stream == _raw_stream(None, dev):
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):  # any object with the handle
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


_driver = None


def _capturing(raw_stream):
    """Whether a graph is being captured from a cudaStream_t.  (Asked of the driver,
    which answers for any stream, current or not, in 0.45 us.)"""
    global _driver
    if not raw_stream:  # the legacy default stream cannot be captured
        return False
    if _driver is None:
        _driver = ctypes.CDLL("libcuda.so.1")
        _driver.cuStreamIsCapturing.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int)]
    status = ctypes.c_int(0)
    return _driver.cuStreamIsCapturing(raw_stream, status) == 0 and status.value != 0


def _call_on(dev, fn, *args):
    """fn(*args) with ``dev`` the current device, as the library's launches need."""
    if dev.index == (_torch_c or _torch())._cuda_getDevice():
        return fn(*args)
    import torch
    with torch.cuda.device(dev):
        return fn(*args)


def _rows_of(x, name, dtype, dev):
    """(address, elements between tokens, shape) of a [T, heads, head_size] tensor
    whose token rows are contiguous."""
    shape = x.shape
    if len(shape) != 3 or x.dtype != dtype or x.device != dev:
        raise ValueError(f"{name} must be a {dtype} tensor [num_tokens, heads, head_size] on one device")
    T, H, D = shape
    st, sh, sd = x.stride()
    if (sh != D and H > 1) or (sd != 1 and D > 1):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return x.data_ptr(), st if T > 1 else H * D, shape


def _status_at(status, dev):
    """Address of a device_status tensor, 0 for None."""
    if status is None:
        return 0
    import torch
    if (status.device != dev or status.dtype not in (torch.int32, torch.uint32) or
            status.numel() < 1):
        raise ValueError("device_status must be an int32 or uint32 tensor of one element on the "
                         "call's device")
    return status.data_ptr()


def _norm_at(w, name, dtype, dev, D):
    if w.dtype != dtype or w.shape != (D,) or w.device != dev or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} [head_size] tensor")
    return w.data_ptr()


def rope_and_cache(q, key, value, kv_cache, slot_mapping, positions, cos_sin, *, block_size,
                   kv_dtype=KV_BF16, kv_scale=None, interleaved=False, pair_axis=None,
                   q_norm=None, k_norm=None, norm_eps=1e-6, q_out=None, device_status=None,
                   stream=None):
    """pattn_rope_and_cache on torch tensors: rotates q and k, writes q to
    ``q_out`` (default: a new tensor; ``q`` itself for in place) and k and v into
    the cache.

    q [T, H, d], key and value [T, Hkv, d], each with contiguous token rows at
    any token stride (views of one packed projection); q or key with value may
    be None.  kv_cache, ``kv_dtype``, ``kv_scale``: as for ``forward``
    (KV_FP8_E4M3_ROW: the row scales, updated too).  positions: int64 [T], or
    [axes, T] with ``pair_axis`` the axis of each rotary pair (see
    ``rope_pair_axis``), or None for no rotation.  cos_sin: fp32
    [max_position, rot_dim], cosines then sines.  ``q_norm``, ``k_norm``: [d]
    weights of a root-mean-square norm per head.  ``device_status``: optional
    int32/uint32 tensor of one element that collects bit 1 for slots past the
    pool and positions outside the table.  Returns ``q_out``; raises PattnError
    or ValueError."""
    import torch
    x = q if q is not None else key
    if x is None:
        raise ValueError("rope_and_cache needs q or key")
    if (key is None and value is not None) or (q is None and q_out is not None):
        raise ValueError("value goes with key and q_out with q")
    dt = torch.float16 if kv_dtype == KV_F16 else torch.bfloat16
    dev = x.device
    q_at = qo_at = k_at = v_at = q_st = qo_st = k_st = v_st = 0
    H = Hkv = NB = cache_at = slots_at = rows_at = scale_at = 0
    if q is not None:
        q_at, q_st, shape = _rows_of(q, "q", dt, dev)
        T, H, D = shape
        if q_out is None:
            q_out = _empty(shape, dt, dev, stream)
        qo_at, qo_st, out_shape = _rows_of(q_out, "q_out", dt, dev)
        if out_shape != shape:
            raise ValueError("q_out must have q's shape")
    if key is not None:
        if value is None:
            raise ValueError("key needs a value")
        k_at, k_st, shape = _rows_of(key, "key", dt, dev)
        v_at, v_st, v_shape = _rows_of(value, "value", dt, dev)
        if v_shape != shape or (q is not None and (shape[0] != T or shape[2] != D)):
            raise ValueError("key and value must be [num_tokens, num_kv_heads, head_size] like q")
        T, Hkv, D = shape
        quantised = kv_dtype == KV_FP8_E4M3_ROW or kv_dtype == KV_FP8_E4M3
        cache_shape = kv_cache.shape
        if (len(cache_shape) != 5 or cache_shape != (2, cache_shape[1], block_size, Hkv, D) or
                not kv_cache.is_contiguous() or kv_cache.device != dev or
                kv_cache.element_size() != (1 if quantised else 2)):
            raise ValueError("kv_cache must be a contiguous [2, num_blocks, block_size, "
                             "num_kv_heads, head_size] tensor of the cache's type")
        if (slot_mapping.dtype != torch.int64 or slot_mapping.shape != (T,) or
                slot_mapping.device != dev or not slot_mapping.is_contiguous()):
            raise ValueError("slot_mapping must be a contiguous int64 [num_tokens] tensor")
        NB = cache_shape[1]
        cache_at, slots_at = kv_cache.data_ptr(), slot_mapping.data_ptr()
        if kv_dtype == KV_FP8_E4M3_ROW:
            _check_row_scales(kv_scale, NB, block_size, Hkv, dev)
            rows_at = kv_scale.data_ptr()
        elif quantised and kv_scale is not None:
            scale = _scale_arg(kv_dtype, kv_scale)
            scale_at = ctypes.addressof(scale)
    pos_at = pos_st = table_at = axes_at = axes = max_pos = rot = 0
    if positions is not None:
        pos_shape = positions.shape
        axes = 1 if len(pos_shape) == 1 else pos_shape[0]
        if (positions.dtype != torch.int64 or not 1 <= len(pos_shape) <= 2 or axes < 1 or
                pos_shape[-1] != T or
                positions.device != dev or (T > 1 and positions.stride(-1) != 1)):
            raise ValueError("positions must be int64 [num_tokens] or [axes, num_tokens]")
        if (cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or cos_sin.device != dev or
                not cos_sin.is_contiguous()):
            raise ValueError("cos_sin must be a contiguous fp32 [max_position, rot_dim] tensor")
        pos_at, table_at = positions.data_ptr(), cos_sin.data_ptr()
        max_pos, rot = cos_sin.shape
        if axes > 1:
            pos_st = positions.stride(0)
            if pair_axis is None or len(pair_axis) != rot // 2:
                raise ValueError("positions of several axes need pair_axis with rot_dim / 2 entries")
            pairs = ctypes.c_char_p(bytes(list(pair_axis)))  # (not an array's own bytes)
            axes_at = ctypes.cast(pairs, ctypes.c_void_p).value
    qn_at = 0 if q_norm is None else _norm_at(q_norm, "q_norm", dt, dev, D)
    kn_at = 0 if k_norm is None else _norm_at(k_norm, "k_norm", dt, dev, D)
    status_at = _status_at(device_status, dev)
    if T == 0:  # (an empty tensor has no address)
        return q_out
    args = _pack(
        _ROPE_PACK, "pattn_rope_and_cache", _ROPE_PACK.size, q_at, qo_at, k_at, v_at, q_st, qo_st,
        k_st, v_st, table_at, pos_at, pos_st, axes_at, qn_at, kn_at, cache_at, rows_at, scale_at,
        slots_at, status_at, _raw_stream(stream, dev),
        float(norm_eps), T, H, Hkv, D, rot, int(interleaved), axes, max_pos, int(kv_dtype),
        int(block_size), NB)
    st = _call_on(dev, load().pattn_rope_and_cache, args)
    if st != 0:
        raise PattnError(st, "pattn_rope_and_cache")
    return q_out


def gather_cache(kv_cache, block_table, out_start_loc, *, num_rows, block_size, kv_dtype=KV_BF16,
                 kv_scale=None, key_starts=None, key_out=None, value_out=None,
                 device_status=None, stream=None):
    """pattn_gather_cache on torch tensors: the keys and values of request r's
    positions key_starts[r] (default 0), ... into rows out_start_loc[r] ...
    out_start_loc[r + 1] of ``key_out`` and ``value_out`` [num_rows, Hkv, d]
    (default: new tensors; bf16, f16 for KV_F16).  kv_cache, ``kv_dtype``,
    ``kv_scale``: as for ``forward``.  Returns (key_out, value_out); raises
    PattnError or ValueError."""
    import torch
    dev = kv_cache.device
    cache_shape = kv_cache.shape
    if (len(cache_shape) != 5 or cache_shape[0] != 2 or cache_shape[2] != block_size or
            not kv_cache.is_contiguous()):
        raise ValueError("kv_cache must be a contiguous [2, num_blocks, block_size, num_kv_heads, "
                         "head_size] tensor")
    _, NB, _, Hkv, D = cache_shape
    quantised = kv_dtype == KV_FP8_E4M3_ROW or kv_dtype == KV_FP8_E4M3
    if kv_cache.element_size() != (1 if quantised else 2):
        raise ValueError("kv_cache must be of the cache's type")
    B, mbps = block_table.shape
    i32 = torch.int32
    if (block_table.dtype != i32 or block_table.device != dev or not block_table.is_contiguous() or
            out_start_loc.dtype != i32 or out_start_loc.shape != (B + 1,) or
            out_start_loc.device != dev or not out_start_loc.is_contiguous()):
        raise ValueError("block_table and out_start_loc must be contiguous int32 tensors "
                         "[num_seqs, blocks] and [num_seqs + 1]")
    starts_at = 0
    if key_starts is not None:
        if (key_starts.dtype != i32 or key_starts.shape != (B,) or key_starts.device != dev or
                not key_starts.is_contiguous()):
            raise ValueError("key_starts must be a contiguous int32 [num_seqs] tensor")
        starts_at = key_starts.data_ptr()
    if kv_dtype == KV_FP8_E4M3_ROW:
        _check_row_scales(kv_scale, NB, block_size, Hkv, dev)
    dt = torch.float16 if kv_dtype == KV_F16 else torch.bfloat16
    shape = (num_rows, Hkv, D)
    outs = []
    for x in (key_out, value_out):
        if x is None:
            x = _empty(shape, dt, dev, stream)
        elif x.shape != shape or x.dtype != dt or x.device != dev or not x.is_contiguous():
            raise ValueError(f"key_out and value_out must be contiguous {dt} tensors of shape {shape}")
        outs.append(x)
    key_out, value_out = outs
    status_at = _status_at(device_status, dev)
    if num_rows == 0 or B == 0:  # (an empty tensor has no address)
        return key_out, value_out
    st = _call_on(
        dev, load().pattn_gather_cache, kv_cache.data_ptr(), block_table.data_ptr(),
        starts_at or None, out_start_loc.data_ptr(),
        key_out.data_ptr(), value_out.data_ptr(), B, int(num_rows), mbps, NB, Hkv, D,
        int(block_size), int(kv_dtype),
        _scale_arg(kv_dtype, kv_scale), status_at or None, _raw_stream(stream, dev))
    if st != 0:
        raise PattnError(st, "pattn_gather_cache")
    return key_out, value_out


def pattn_cascade_workspace_bytes(ext, num_heads, num_kv_heads, head_size, block_size,
                                  common_prefix_len, lib=None):
    lib = lib or load()
    return lib.pattn_cascade_workspace_bytes(ctypes.byref(ext), int(num_heads), int(num_kv_heads),
                                             int(head_size), int(block_size),
                                             int(common_prefix_len))


def cascade_forward(q, kv_cache, block_table, seq_lens, query_start_loc, *, scale, num_heads,
                    num_kv_heads, head_size, block_size, common_prefix_len, window=0, causal=1,
                    kv_dtype=KV_BF16, kv_scale=None, max_query_len, max_seq_len, num_splits=0,
                    out=None, workspace=None, stream=None, sinks=None):
    """pattn_cascade_fwd on torch tensors: pattn_varlen_fwd for a batch whose
    requests share their first common_prefix_len keys (same blocks).
    ``sinks``: optional fp32 [num_heads] device tensor of attention-sink logits.
    ``kv_scale``: (k_scale, v_scale), or the row-scale tensor of a
    KV_FP8_E4M3_ROW cache.  Returns ``out``; raises PattnError."""
    import torch
    dev = q.device
    T = q.shape[0]
    if kv_dtype == KV_FP8_E4M3_ROW:
        _check_row_scales(kv_scale, kv_cache.shape[1], block_size, num_kv_heads, dev)
    if out is None:
        odt = torch.float16 if kv_dtype == KV_F16 else torch.bfloat16
        out = _empty((T, num_heads, head_size), odt, dev, stream)
    raw_stream = _raw_stream(stream, dev)
    ext = make_ext(num_seqs=seq_lens.shape[0], num_tokens=T,
                   max_blocks_per_seq=block_table.shape[1], num_blocks=kv_cache.shape[1],
                   max_query_len=max_query_len, max_seq_len=max_seq_len,
                   num_splits=num_splits, stream=raw_stream,
                   sinks=_sinks_ptr(sinks, num_heads, dev))
    need = _call_on(dev, pattn_cascade_workspace_bytes, ext, num_heads, num_kv_heads, head_size,
                    block_size, common_prefix_len)
    if need == 0:
        raise PattnError(1, "pattn_cascade_workspace_bytes")
    ws = _workspace(workspace, dev, raw_stream)
    buf = ws.get(need, dev, stream)
    ws.used_on(raw_stream)
    ext.workspace = buf.data_ptr()
    ext.workspace_bytes = buf.numel()
    st = _call_on(dev, load().pattn_cascade_fwd, q.data_ptr(), kv_cache.data_ptr(),
                  block_table.data_ptr(), seq_lens.data_ptr(), query_start_loc.data_ptr(),
                  out.data_ptr(), float(scale), int(num_heads), int(num_kv_heads), int(head_size),
                  int(block_size), int(window), int(causal), int(kv_dtype),
                  _scale_arg(kv_dtype, kv_scale), int(common_prefix_len), ctypes.byref(ext))
    if st != 0:
        raise PattnError(st, "pattn_cascade_fwd")
    ext._workspace_keepalive = buf
    forward.last_ext = ext
    return out


def make_ext(*, num_seqs, num_tokens, max_blocks_per_seq, num_blocks, max_query_len,
             max_seq_len, num_splits=0, workspace=0, workspace_bytes=0, stream=0,
             timing_events=None, sinks=0, head_size_v=0):
    e = Ext()
    e.struct_size = ctypes.sizeof(Ext)
    e.num_seqs, e.num_tokens = int(num_seqs), int(num_tokens)
    e.max_blocks_per_seq, e.num_blocks = int(max_blocks_per_seq), int(num_blocks)
    e.max_query_len, e.max_seq_len = int(max_query_len), int(max_seq_len)
    e.num_splits = int(num_splits)
    e.workspace = int(workspace) or None
    e.workspace_bytes = int(workspace_bytes)
    e.stream = int(stream) or None
    e.sinks = int(sinks) or None
    e.head_size_v = int(head_size_v)
    if timing_events is not None:
        arr = (ctypes.c_void_p * 8)(*[int(x) for x in timing_events])
        e._events_keepalive = arr
        e.timing_events = ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p))
    return e


def pattn_varlen_fwd(q, kv_cache, block_table, seq_lens, query_start_loc, out, scale,
                     num_heads, num_kv_heads, head_size, block_size, window, causal,
                     kv_dtype, kv_scale, ext, lib=None):
    """Raw call with integer device pointers; returns the status code."""
    lib = lib or load()
    ks = _scale_arg(kv_dtype, kv_scale)
    return lib.pattn_varlen_fwd(q, kv_cache, block_table, seq_lens, query_start_loc, out,
                                float(scale), int(num_heads), int(num_kv_heads),
                                int(head_size), int(block_size), int(window), int(causal),
                                int(kv_dtype), ks, ctypes.byref(ext))


def pattn_decode_fwd_static(q, kv_cache, block_table, seq_lens, query_start_loc, out, scale,
                            num_heads, num_kv_heads, head_size, block_size, window, causal,
                            kv_dtype, kv_scale, num_seqs, num_tokens, max_blocks_per_seq,
                            num_blocks, max_seq_len, num_splits, stream, lib=None):
    """Raw call of the workspace-free decode entry point; returns the status.
    For callers that cannot allocate device memory (see include/pattn.h)."""
    lib = lib or load()
    ks = _scale_arg(kv_dtype, kv_scale)
    return lib.pattn_decode_fwd_static(q, kv_cache, block_table, seq_lens, query_start_loc,
                                       out, float(scale), int(num_heads), int(num_kv_heads),
                                       int(head_size), int(block_size), int(window),
                                       int(causal), int(kv_dtype), ks, int(num_seqs),
                                       int(num_tokens), int(max_blocks_per_seq),
                                       int(num_blocks), int(max_seq_len), int(num_splits),
                                       int(stream) or None)


def pattn_workspace_bytes(ext, num_heads, num_kv_heads, head_size, block_size, lib=None):
    return (lib or load()).pattn_workspace_bytes(ctypes.byref(ext), num_heads, num_kv_heads,
                                                 head_size, block_size)


def pattn_decode_splits(ext, num_heads, num_kv_heads, block_size, window, lib=None):
    return (lib or load()).pattn_decode_splits(ctypes.byref(ext), num_heads, num_kv_heads,
                                               block_size, window)


def pattn_read_device_status(ext, lib=None):
    return (lib or load()).pattn_read_device_status(ctypes.byref(ext))


def pattn_status_string(status, lib=None):
    return (lib or load()).pattn_status_string(int(status)).decode()


def pattn_version(lib=None):
    return (lib or load()).pattn_version()


class Workspace:
    """A torch-allocated device workspace, grown on demand (plumbing only).

    A buffer comes from the pool of the stream whose call needed it, and one that
    is replaced goes back there, where the next use is ordered behind the calls.
    A buffer that calls on another stream have used too, or that is part of a
    captured graph (its replays write to the address that the capture saw), is not
    given back before the Workspace is: keep an explicit Workspace as long as a
    graph captured with it."""

    def __init__(self):
        self.buf = None
        self._stream = None  # whose pool the buffer is from (cudaStream_t)
        self._held = False   # not to be given back when it is replaced
        self._replaced = []

    def current(self, device):
        """The buffer it has on ``device``, or None."""
        return self.buf if self.buf is not None and self.buf.device == device else None

    def get(self, nbytes, device, stream=None):
        """A buffer of at least ``nbytes`` for a call on ``stream`` (default: the
        device's current one)."""
        import torch
        nbytes = max(256, int(nbytes))
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        if self.buf is None or self.buf.numel() < nbytes or self.buf.device != device:
            buf = _empty(nbytes, torch.uint8, device, stream)
            if self._held:
                self._replaced.append(self.buf)
            self.buf, self._held = buf, False
            self._stream = _raw_stream(stream, device) if device.type == "cuda" else 0
        return self.buf

    def used_on(self, raw_stream):
        """Notes that a call on a cudaStream_t is about to use the buffer."""
        if not self._held and (raw_stream != self._stream or _capturing(raw_stream)):
            self._held = True


_default_ws = {}  # (device index, cudaStream_t, host thread) -> Workspace


def _workspace(workspace, dev, raw_stream):
    """The caller's Workspace, or the stream's own: a thread's calls on one stream
    run one after the other and may share scratch.  Calls on two streams may not,
    nor two threads' calls on one, whose launches interleave.  (Nor may two captured
    graphs that run at once: they need a Workspace each.)"""
    if workspace is not None:
        return workspace
    key = (dev.index, raw_stream, threading.get_ident())
    ws = _default_ws.get(key)
    if ws is None:
        ws = _default_ws[key] = Workspace()
    return ws


def release_workspaces():
    """Gives every default workspace back to torch's allocator (each stream and host
    thread keeps its largest one otherwise).  Not while a graph captured with one
    may still be replayed."""
    _default_ws.clear()


def _sinks_ptr(sinks, num_heads, device):
    """Device pointer of an fp32 [num_heads] sink tensor (0 for None)."""
    if sinks is None:
        return 0
    import torch
    if (sinks.dtype != torch.float32 or sinks.device != torch.device(device) or
            sinks.numel() != num_heads or not sinks.is_contiguous()):
        raise ValueError("sinks must be a contiguous fp32 [num_heads] tensor on q's device")
    return sinks.data_ptr()


def forward(q, kv_cache, block_table, seq_lens, query_start_loc, *, scale, num_heads,
            num_kv_heads, head_size, block_size, window=0, causal=1, kv_dtype=KV_BF16,
            kv_scale=None, max_query_len, max_seq_len, num_splits=0, out=None,
            workspace=None, stream=None, timing_events=None, sinks=None, head_size_v=0,
            check=True, lib=None):
    """pattn_varlen_fwd on torch tensors (all on one CUDA device).

    max_query_len / max_seq_len are host ints (as in FlashAttentionMetadata):
    the library never reads device memory on the host.  ``kv_scale``: (k_scale,
    v_scale) of an e4m3 cache, or the row-scale tensor of a KV_FP8_E4M3_ROW cache
    (see ``row_scales_shape``).  ``workspace``: a Workspace (default: one per
    stream and host thread; two graphs that may run at once need one each, and a
    Workspace serves one thread at a time).  ``timing_events``:
    optional 8 raw cudaEvent_t handles (see pattn_ext_t).  ``sinks``: optional
    fp32 [num_heads] device tensor of attention-sink logits.  ``head_size_v``:
    > 0 selects the DiffKV cache layout [num_blocks, block_size, num_kv_heads,
    head_size + head_size_v] and an output of head size head_size_v (see
    pattn_ext_t).  ``lib``: a library handle from ``load(path)`` (default: the
    built libpattn.so).  Returns ``out``.
    """
    import torch
    dev = q.device
    T = q.shape[0]
    if out is None:
        odt = torch.float16 if kv_dtype == KV_F16 else torch.bfloat16
        out = _empty((T, num_heads, head_size_v or head_size), odt, dev, stream)
    num_blocks = kv_cache.shape[0] if head_size_v else kv_cache.shape[1]
    if kv_dtype == KV_FP8_E4M3_ROW:
        _check_row_scales(kv_scale, num_blocks, block_size, num_kv_heads, dev)
    mbps = block_table.shape[1]
    raw_stream = _raw_stream(stream, dev)
    events = None
    if timing_events is not None:
        events = (ctypes.c_void_p * 8)(*[int(x) for x in timing_events])
    ws = _workspace(workspace, dev, raw_stream)
    buf = ws.current(dev)
    ext = Ext.from_buffer_copy(_pack(
        _EXT_PACK, "pattn_varlen_fwd", _EXT_PACK.size, seq_lens.shape[0], T, mbps, num_blocks,
        int(max_query_len), int(max_seq_len), int(num_splits),
        0 if buf is None else buf.data_ptr(), 0 if buf is None else buf.numel(), raw_stream,
        0 if events is None else ctypes.addressof(events), _sinks_ptr(sinks, num_heads, dev),
        int(head_size_v)))
    ext._events_keepalive = events
    run = (lib or load()).pattn_varlen_fwd
    args = (q.data_ptr(), kv_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
            query_start_loc.data_ptr(), out.data_ptr(), float(scale), int(num_heads),
            int(num_kv_heads), int(head_size), int(block_size), int(window), int(causal),
            int(kv_dtype), _scale_arg(kv_dtype, kv_scale), ext)
    # the library itself says when the workspace is missing or too small
    st = 3
    if buf is not None:
        ws.used_on(raw_stream)
        st = _call_on(dev, run, *args)
    if st != 0:
        need = _call_on(dev, pattn_workspace_bytes, ext, num_heads, num_kv_heads, head_size,
                        block_size, lib)
        if need == 0:
            raise PattnError(1, "pattn_workspace_bytes")
        if st == 3:
            buf = ws.get(need, dev, stream)
            ws.used_on(raw_stream)
            ext.workspace, ext.workspace_bytes = buf.data_ptr(), buf.numel()
            st = _call_on(dev, run, *args)
    if check and st != 0:
        raise PattnError(st, "pattn_varlen_fwd")
    ext._workspace_keepalive = buf  # (its status word may be read after a larger call)
    forward.last_ext = ext
    return out
