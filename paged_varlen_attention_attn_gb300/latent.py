"""Attention with keys and values from one shared latent vector a token.

The cache holds one row per token, [latent | rotary key], shared by all heads:
[num_blocks, block_size, latent_size + rope_size], bf16 (KV_BF16) or f16
(KV_F16).  ``latent_rope_and_cache`` writes it, ``latent_forward`` attends it
as it is (the absorbed form), ``gather_latent`` reads it back and
``latent_expanded_forward`` attends keys and values that were projected up to a
pair per head (the expanded form).  Argument marshalling only, as in the
package's other wrappers; the calls are declared in ``include/pattn.h``.
"""
import ctypes

from . import (_EXT_PACK, KV_BF16, KV_F16, Ext, PattnError, _call_on, _empty, _norm_at, _pack,
               _packer, _raw_stream, _status_at, _workspace, load)

_PTR, _I64 = ctypes.c_void_p, ctypes.c_longlong


class LatentRopeArgs(ctypes.Structure):
    """pattn_latent_rope_t"""
    _fields_ = ([("struct_size", ctypes.c_size_t)] +
                [(n, _PTR) for n in ("q", "q_out", "latent", "k_rope", "row_out")] +
                [(n, _I64) for n in ("q_stride", "q_head_stride", "q_out_stride",
                                     "q_out_head_stride", "latent_stride", "k_rope_stride",
                                     "row_out_stride")] +
                [(n, _PTR) for n in ("latent_norm", "cos_sin", "positions", "kv_cache",
                                     "slot_mapping", "device_status", "stream")] +
                [("norm_eps", ctypes.c_float)] +
                [(n, ctypes.c_int) for n in ("num_tokens", "num_heads", "latent_size", "rope_size",
                                             "interleaved", "max_position", "kv_dtype",
                                             "block_size", "num_blocks")])


class LatentArgs(ctypes.Structure):
    """pattn_latent_t"""
    _fields_ = ([("struct_size", ctypes.c_size_t)] +
                [(n, _PTR) for n in ("q", "kv_cache", "out", "block_table", "seq_lens",
                                     "query_start_loc", "workspace")] +
                [("workspace_bytes", ctypes.c_size_t), ("stream", _PTR), ("scale", ctypes.c_float)] +
                [(n, ctypes.c_int) for n in ("causal", "kv_dtype", "num_seqs", "num_tokens",
                                             "num_heads", "latent_size", "rope_size", "block_size",
                                             "max_blocks_per_seq", "num_blocks", "max_query_len")])


class LatentExpandedArgs(ctypes.Structure):
    """pattn_latent_expanded_t"""
    _fields_ = ([("struct_size", ctypes.c_size_t)] +
                [(n, _PTR) for n in ("q", "k_nope", "k_rope", "value", "out")] +
                [(n, _I64) for n in ("q_stride", "q_head_stride", "k_stride", "k_head_stride",
                                     "k_rope_stride", "v_stride", "v_head_stride")] +
                [(n, _PTR) for n in ("query_start_loc", "key_start_loc", "workspace")] +
                [("workspace_bytes", ctypes.c_size_t), ("stream", _PTR), ("scale", ctypes.c_float)] +
                [(n, ctypes.c_int) for n in ("causal", "kv_dtype", "num_seqs", "num_tokens",
                                             "num_keys", "num_heads", "nope_size", "rope_size",
                                             "value_size")])


_ROPE_PACK, _ATTEND_PACK, _EXPANDED_PACK = (_packer(c) for c in (LatentRopeArgs, LatentArgs,
                                                                 LatentExpandedArgs))


_types = {}  # kv_dtype -> torch dtype; the index tensors' types by their C names


def _type_of(kv_dtype):
    dt = _types.get(kv_dtype)
    if dt is None:
        if kv_dtype not in (KV_BF16, KV_F16):
            raise PattnError(2, "a cache of latent rows is KV_BF16 or KV_F16")
        import torch
        _types.update({KV_BF16: torch.bfloat16, KV_F16: torch.float16, "int32": torch.int32,
                       "int64": torch.int64, "float": torch.float32})
        dt = _types[kv_dtype]
    return dt


def _heads(x, name, dtype, dev):
    """(address, elements between tokens, between heads) of a [tokens, heads, size]
    tensor whose last axis is contiguous.  (The stride of an axis of length 1 means
    nothing: the one that a dense tensor would have.)"""
    shape = x.shape
    if len(shape) != 3 or x.dtype != dtype or x.device != dev:
        raise ValueError(f"{name} must be a {dtype} tensor of three axes on one device")
    T, H, D = shape
    st, sh, sd = x.stride()
    if sd != 1 and D > 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    if H == 1:
        sh = D
    return x.data_ptr(), st if T > 1 else max(H * sh, D), sh


def _rows(x, name, dtype, dev):
    """(address, elements between rows) of a [tokens, size] tensor."""
    if x.dim() != 2 or x.dtype != dtype or x.device != dev:
        raise ValueError(f"{name} must be a {dtype} tensor of two axes on one device")
    st, sd = x.stride()
    if sd != 1 and x.shape[1] > 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    return x.data_ptr(), st if x.shape[0] > 1 else x.shape[1]


def _cache(kv_cache, dtype, block_size):
    if (kv_cache.dim() != 3 or kv_cache.shape[1] != block_size or kv_cache.dtype != dtype or
            not kv_cache.is_contiguous()):
        raise ValueError(f"kv_cache must be a contiguous {dtype} [num_blocks, block_size, "
                         "latent_size + rope_size] tensor")
    return kv_cache.shape[0], kv_cache.shape[2]


def _index(x, name, dtype, shape, dev):
    if x.dtype != dtype or x.shape != shape or x.device != dev or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    return x.data_ptr()


def _out(x, name, dtype, shape, dev, stream):
    """(tensor, address) of a contiguous output: x if it is one, or a new one."""
    if x is None:
        x = _empty(shape, dtype, dev, stream)
        return x, x.data_ptr()
    return x, _index(x, name, dtype, shape, dev)


def _length(x, what):
    """Refuses a length that no batch has (None: not given)."""
    if x is not None and not int(x) >= 0:
        raise PattnError(1, what)


def latent_rope_and_cache(q, latent, k_rope, kv_cache, slot_mapping, positions, cos_sin, *,
                          block_size, kv_dtype=KV_BF16, interleaved=False, latent_norm=None,
                          norm_eps=1e-6, q_out=None, row_out=None, device_status=None,
                          stream=None):
    """pattn_latent_rope_and_cache on torch tensors: norms the latents (``latent_norm``:
    [latent_size] weight, or None), rotates the rotary parts of q and of the shared
    key, and writes [latent | key] to each token's cache slot.

    q [T, H, rope_size] with any token and head strides (a view of the heads' last
    elements, say) or None; latent [T, latent_size] and k_rope [T, rope_size] at any
    token stride (views of one projection).  positions: int64 [T], or None for no
    rotation; cos_sin: fp32 [max_position, rope_size], cosines then sines.
    slot_mapping: int64 [T].  ``q_out``: as q (default: a new tensor; ``q`` itself for
    in place).  ``row_out``: optional [T, latent_size + rope_size] tensor that gets
    the rows as well; it may be the tensor that latent and k_rope are the parts of.
    ``device_status``: optional int32/uint32 tensor of one element that collects
    bit 1 for slots past the pool and positions outside the table.  Returns
    ``q_out``; raises PattnError or ValueError."""
    dt = _type_of(kv_dtype)
    dev = kv_cache.device
    NB, row = _cache(kv_cache, dt, block_size)
    lat_at, lat_st = _rows(latent, "latent", dt, dev)
    kr_at, kr_st = _rows(k_rope, "k_rope", dt, dev)
    T, dc = latent.shape
    dr = k_rope.shape[1]
    if k_rope.shape[0] != T or dc + dr != row:
        raise ValueError("latent and k_rope must be [num_tokens, latent_size] and [num_tokens, "
                         "rope_size], the parts of a cache row")
    q_at = q_st = q_sh = o_at = o_st = o_sh = H = row_at = row_st = 0
    if q is not None:
        q_at, q_st, q_sh = _heads(q, "q", dt, dev)
        H = q.shape[1]
        if q.shape[0] != T or q.shape[2] != dr:
            raise ValueError("q must be [num_tokens, heads, rope_size]")
        if q_out is None:
            q_out = _empty(q.shape, dt, dev, stream)
            o_at, o_st, o_sh = q_out.data_ptr(), H * dr, dr
        else:
            o_at, o_st, o_sh = _heads(q_out, "q_out", dt, dev)
            if q_out.shape != q.shape:
                raise ValueError("q_out must have q's shape")
    elif q_out is not None:
        raise ValueError("q_out goes with q")
    if row_out is not None:
        row_at, row_st = _rows(row_out, "row_out", dt, dev)
        if row_out.shape != (T, row):
            raise ValueError("row_out must be [num_tokens, latent_size + rope_size]")
    slots_at = _index(slot_mapping, "slot_mapping", _types["int64"], (T,), dev)
    pos_at = table_at = max_pos = 0
    if positions is not None:
        pos_at = _index(positions, "positions", _types["int64"], (T,), dev)
        if (cos_sin is None or cos_sin.dtype != _types["float"] or cos_sin.dim() != 2 or cos_sin.shape[1] != dr or
                cos_sin.device != dev or not cos_sin.is_contiguous()):
            raise ValueError("cos_sin must be a contiguous fp32 [max_position, rope_size] tensor")
        table_at, max_pos = cos_sin.data_ptr(), cos_sin.shape[0]
    norm_at = 0 if latent_norm is None else _norm_at(latent_norm, "latent_norm", dt, dev, dc)
    status_at = _status_at(device_status, dev)
    if T == 0 or (q is not None and H == 0):  # (an empty tensor has no address)
        if T == 0:
            return q_out
        raise PattnError(1, "pattn_latent_rope_and_cache")
    args = _pack(
        _ROPE_PACK, "pattn_latent_rope_and_cache", _ROPE_PACK.size, q_at, o_at, lat_at, kr_at,
        row_at, q_st, q_sh, o_st, o_sh, lat_st, kr_st, row_st, norm_at, table_at, pos_at,
        kv_cache.data_ptr(), slots_at, status_at, _raw_stream(stream, dev), float(norm_eps), T, H,
        dc, dr, int(interleaved), max_pos, int(kv_dtype), int(block_size), NB)
    st = _call_on(dev, load().pattn_latent_rope_and_cache, args)
    if st != 0:
        raise PattnError(st, "pattn_latent_rope_and_cache")
    return q_out


def gather_latent(kv_cache, block_table, out_start_loc, *, num_rows, latent_size, block_size,
                  kv_dtype=KV_BF16, key_starts=None, latent_out=None, rope_out=None,
                  device_status=None, stream=None):
    """pattn_gather_latent on torch tensors: the cached rows of request r's positions
    key_starts[r] (default 0), ... into rows out_start_loc[r] ... out_start_loc[r + 1]
    of ``latent_out`` [num_rows, latent_size] and ``rope_out`` [num_rows, rope_size]
    (default: new tensors).  Returns (latent_out, rope_out); raises PattnError or
    ValueError."""
    dt = _type_of(kv_dtype)
    dev = kv_cache.device
    NB, row = _cache(kv_cache, dt, block_size)
    dr = row - latent_size
    B, mbps = block_table.shape
    i32 = _types["int32"]
    bt_at = _index(block_table, "block_table", i32, (B, mbps), dev)
    osl_at = _index(out_start_loc, "out_start_loc", i32, (B + 1,), dev)
    ks_at = 0 if key_starts is None else _index(key_starts, "key_starts", i32, (B,), dev)
    if latent_size <= 0 or dr <= 0 or num_rows < 0:
        raise PattnError(1, "pattn_gather_latent")
    latent_out, lat_at = _out(latent_out, "latent_out", dt, (num_rows, latent_size), dev, stream)
    rope_out, rope_at = _out(rope_out, "rope_out", dt, (num_rows, dr), dev, stream)
    status_at = _status_at(device_status, dev)
    if num_rows == 0 or B == 0:  # (an empty tensor has no address)
        return latent_out, rope_out
    st = _call_on(dev, load().pattn_gather_latent, kv_cache.data_ptr(), bt_at, ks_at or None,
                  osl_at, lat_at, rope_at, B, int(num_rows), mbps, NB, int(latent_size), dr,
                  int(block_size), int(kv_dtype), status_at or None, _raw_stream(stream, dev))
    if st != 0:
        raise PattnError(st, "pattn_gather_latent")
    return latent_out, rope_out


_sizes = {}  # workspace bytes by (name, device index, sizes)


def _workspace_bytes(name, dev, *sizes):
    key = (name, dev.index, sizes)
    need = _sizes.get(key)
    if need is None:
        need = _call_on(dev, getattr(load(), name), *sizes)
        if need == 0:
            raise PattnError(1, name)
        if len(_sizes) > 4096:
            _sizes.clear()
        _sizes[key] = need
    return need


def _scratch(workspace, need, dev, stream):
    """(address, bytes, raw stream, Ext for pattn_read_device_status) of a call's
    workspace of at least ``need`` bytes.  (The Ext lasts as long as the buffer: a
    Workspace drops it with the buffer that it replaces.)"""
    raw = _raw_stream(stream, dev)
    ws = _workspace(workspace, dev, raw)
    ext = ws._ext
    if ext is None or ext._bytes < need or ext._raw != raw or ext._device != dev:
        buf = ws.get(need, dev, stream)
        at, size = buf.data_ptr(), buf.numel()
        ext = Ext.from_buffer_copy(_pack(_EXT_PACK, "workspace", _EXT_PACK.size, 0, 0, 0, 0, 0, 0, 0,
                                         at, size, raw, 0, 0, 0))
        ext._at, ext._bytes, ext._raw, ext._device = at, size, raw, dev
        ext._workspace_keepalive = buf  # (its status word may be read after a larger call)
        ws._ext = ext
    ws.used_on(raw)
    return ext._at, ext._bytes, raw, ext


def latent_forward(q, kv_cache, block_table, seq_lens, query_start_loc, *, scale, latent_size,
                   block_size, causal=1, kv_dtype=KV_BF16, max_query_len, max_seq_len=None,
                   out=None, workspace=None, stream=None):
    """pattn_latent_fwd on torch tensors (all on one CUDA device): every head of q
    [T, H, latent_size + rope_size] attends the cached rows of its request, whose
    first latent_size elements are the values.  Returns ``out`` [T, H, latent_size].

    block_table int32 [B, blocks], seq_lens int32 [B], query_start_loc int32 [B + 1]
    as for ``forward``; ``max_query_len``: host int, at least every query length (1
    selects the layout for single tokens).  ``max_seq_len``: as for ``forward``, whose
    callers have it; it chooses nothing here and is checked for its sign only.  ``workspace``: a Workspace (default: one per
    stream and host thread).  ``latent_forward.last_ext`` serves
    pattn_read_device_status, which tells (and clears) the status of the latest call
    on that workspace, of whichever operator.  Raises PattnError or ValueError."""
    dt = _type_of(kv_dtype)
    dev = q.device
    NB, row = _cache(kv_cache, dt, block_size)
    if (q.dim() != 3 or q.dtype != dt or q.shape[2] != row or not q.is_contiguous() or
            kv_cache.device != dev):
        raise ValueError(f"q must be a contiguous {dt} [num_tokens, heads, latent_size + rope_size] "
                         "tensor on the cache's device")
    T, H, _ = q.shape
    B, mbps = block_table.shape
    i32 = _types["int32"]
    bt_at = _index(block_table, "block_table", i32, (B, mbps), dev)
    sl_at = _index(seq_lens, "seq_lens", i32, (B,), dev)
    qsl_at = _index(query_start_loc, "query_start_loc", i32, (B + 1,), dev)
    latent_size = int(latent_size)
    if not 0 < latent_size < row:
        raise PattnError(1, "pattn_latent_fwd")
    _length(max_query_len, "pattn_latent_fwd")
    _length(max_seq_len, "pattn_latent_fwd")
    out, out_at = _out(out, "out", dt, (T, H, latent_size), dev, stream)
    if T == 0 or B == 0:  # (an empty tensor has no address)
        return out
    need = _workspace_bytes("pattn_latent_workspace_bytes", dev, B, H, latent_size)
    at, size, raw, ext = _scratch(workspace, need, dev, stream)
    args = _pack(_ATTEND_PACK, "pattn_latent_fwd", _ATTEND_PACK.size, q.data_ptr(),
                 kv_cache.data_ptr(), out_at, bt_at, sl_at, qsl_at, at, size, raw, float(scale),
                 int(causal), int(kv_dtype), B, T, H, latent_size, row - latent_size,
                 int(block_size), mbps, NB, int(max_query_len))
    st = _call_on(dev, load().pattn_latent_fwd, args)
    if st != 0:
        raise PattnError(st, "pattn_latent_fwd")
    latent_forward.last_ext = ext
    return out


def latent_expanded_forward(q, k_nope, k_rope, value, query_start_loc, key_start_loc, *, scale,
                            causal=1, kv_dtype=KV_BF16, max_query_len=None, max_key_len=None,
                            out=None, workspace=None, stream=None):
    """pattn_latent_expanded_fwd on torch tensors (all on one CUDA device): ragged
    attention of q [T, H, nope + rope] over k_nope [K, H, nope], k_rope [K, rope]
    (shared by the heads) and value [K, H, nope]; request r owns q rows
    query_start_loc[r] ... and keys key_start_loc[r] ....  Any token and head strides
    that are multiples of 8 elements (k_nope and value may be views of one
    up-projection).  Returns ``out`` [T, H, nope].  ``max_query_len`` and
    ``max_key_len`` choose nothing (the kernel plans from the device's own lengths) and
    are checked for their signs only.
    ``latent_expanded_forward.last_ext`` serves pattn_read_device_status, as for
    ``latent_forward``.  Raises PattnError or ValueError."""
    dt = _type_of(kv_dtype)
    dev = q.device
    q_at, q_st, q_sh = _heads(q, "q", dt, dev)
    k_at, k_st, k_sh = _heads(k_nope, "k_nope", dt, dev)
    v_at, v_st, v_sh = _heads(value, "value", dt, dev)
    r_at, r_st = _rows(k_rope, "k_rope", dt, dev)
    T, H, D = q.shape
    K, _, dn = k_nope.shape
    dr, dv = k_rope.shape[1], value.shape[2]
    if (k_nope.shape[1] != H or value.shape[:2] != (K, H) or k_rope.shape[0] != K or
            D != dn + dr):
        raise ValueError("q, k_nope, k_rope and value must be [num_tokens, heads, nope + rope], "
                         "[num_keys, heads, nope], [num_keys, rope] and [num_keys, heads, value]")
    _length(max_query_len, "pattn_latent_expanded_fwd")
    _length(max_key_len, "pattn_latent_expanded_fwd")
    B = query_start_loc.numel() - 1
    if B < 0:
        raise ValueError("query_start_loc must hold num_seqs + 1 numbers")
    qsl_at = _index(query_start_loc, "query_start_loc", _types["int32"], (B + 1,), dev)
    ksl_at = _index(key_start_loc, "key_start_loc", _types["int32"], (B + 1,), dev)
    out, out_at = _out(out, "out", dt, (T, H, dv), dev, stream)
    if T == 0 or B == 0:  # (an empty tensor has no address)
        return out
    if K == 0:  # (likewise: no key is read)
        k_at = v_at = r_at = q_at
        k_st, k_sh, v_st, v_sh, r_st = H * dn, dn, H * dv, dv, dr
    need = load().pattn_latent_expanded_workspace_bytes(B, T)
    at, size, raw, ext = _scratch(workspace, need, dev, stream)
    args = _pack(_EXPANDED_PACK, "pattn_latent_expanded_fwd", _EXPANDED_PACK.size, q_at, k_at, r_at,
                 v_at, out_at, q_st, q_sh, k_st, k_sh, r_st, v_st, v_sh, qsl_at, ksl_at, at, size,
                 raw, float(scale), int(causal), int(kv_dtype), B, T, K, H, dn, dr, dv)
    st = _call_on(dev, load().pattn_latent_expanded_fwd, args)
    if st != 0:
        raise PattnError(st, "pattn_latent_expanded_fwd")
    latent_expanded_forward.last_ext = ext
    return out
