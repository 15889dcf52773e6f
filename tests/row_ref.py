"""Plain definitions in 64 bits for the row-scaled e4m3 cache: rotary embedding,
row quantisation, cache write and read-back, attention (inputs only on the CPU)."""
import math

import numpy as np
import torch

E4M3_MAX = 448.0
ROW_MIN, ROW_MAX = 2.0 ** -60, 2.0 ** 60


def f64(x):
    """A 16-bit, fp32 or e4m3-byte (uint8) tensor as float64 on the CPU."""
    x = x.detach().cpu()
    if x.dtype == torch.uint8:
        x = x.view(torch.float8_e4m3fn)
    return x.to(torch.float32).double()


def cos_sin_table(max_pos, rot, base=10000.0):
    """(fp32 table [max_pos, rot], its angles in float64 [max_pos, rot / 2])"""
    freq = base ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], 1).float(), ang


def rotate(x, table, positions, *, interleaved=False, pair_axis=None, weight=None, eps=0.0):
    """x [T, h, d] float64 normed and rotated by the fp32 table's own values."""
    x = x.clone()
    d = x.shape[-1]
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + eps) * f64(weight)
    if positions is None:
        return x
    rot = table.shape[1]
    pos = positions.view(-1, x.shape[0])
    for p in range(rot // 2):
        at = pos[pair_axis[p] if pair_axis is not None else 0]
        c, s = table[at, p].double()[:, None], table[at, rot // 2 + p].double()[:, None]
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)
        a, b = x[..., i].clone(), x[..., j].clone()
        x[..., i], x[..., j] = a * c - b * s, b * c + a * s
    return x


def row_scale(x):
    """The scale of each row of x [..., d] in 64 bits (NaN elements do not count)."""
    m = torch.nan_to_num(x.abs(), nan=0.0, posinf=float(torch.finfo(torch.float32).max) * 2).amax(-1)
    return (m / E4M3_MAX).clamp(ROW_MIN, ROW_MAX)


def row_codes_fp32(x):
    """(codes uint8, scales) of 16-bit rows x [..., d] by the written steps in fp32:
    scale = max / 448 clamped, code = e4m3(x / scale)."""
    x = x.detach().cpu().float()
    m = torch.nan_to_num(x.abs(), nan=0.0, posinf=math.inf).amax(-1)
    s = (m / torch.tensor(E4M3_MAX)).clamp(ROW_MIN, ROW_MAX)
    y = x / s[..., None]
    codes = y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = torch.where(torch.isnan(x), torch.full_like(codes, 0x7F), codes)
    return codes, s


def scales_at(scales, slots):
    """[len(slots), Hkv, 2] scales of cache slots from the cache's scale tensor."""
    s = scales.detach().cpu().double()
    nb, groups = s.shape[:2]
    flat = s.permute(0, 1, 4, 2, 3).reshape(nb * groups * 16, s.shape[2], 2)
    return flat[slots]


def dense(kv_cache, scales):
    """[2, NB, bs, Hkv, d] float64 values of a row-scaled cache."""
    x = f64(kv_cache)
    nb, bs = x.shape[1:3]
    s = scales.detach().cpu().double().permute(3, 0, 1, 4, 2).reshape(2, nb, bs, -1)
    return x * s[..., None]


def attention(q, dense_kv, block_table, seq_lens, qsl, *, scale, window=0, causal=1, sinks=None):
    """out [T, H, d] float64 (rows of tokens outside every request stay NaN)."""
    Q = f64(q).numpy()
    T, H, D = Q.shape
    KV = dense_kv.numpy()
    bs, Hkv = KV.shape[2], KV.shape[3]
    bt, sl, qs = (x.detach().cpu().numpy() for x in (block_table, seq_lens, qsl))
    out = np.full((T, H, D), np.nan)
    for r in range(len(sl)):
        t0, t1 = int(qs[r]), int(qs[r + 1])
        n, s = t1 - t0, int(sl[r])
        if n == 0:
            continue
        blocks = bt[r, :(s + bs - 1) // bs]
        K = KV[0][blocks].reshape(-1, Hkv, D)[:s]
        V = KV[1][blocks].reshape(-1, Hkv, D)[:s]
        pos = (s - n + np.arange(n))[:, None]
        key = np.arange(s)[None]
        seen = np.ones((n, s), bool)
        if causal:
            seen &= key <= pos
        if window > 0:
            seen &= pos - key < window
        for h in range(H):
            g = h // (H // Hkv)
            x = np.where(seen, float(np.float32(scale)) * (Q[t0:t1, h] @ K[:, g].T), -np.inf)
            m = x.max(1, keepdims=True)
            e = np.exp(x - m)
            den = e.sum(1, keepdims=True)
            if sinks is not None:
                den = den + np.exp(float(sinks[h]) - m)
            out[t0:t1, h] = e @ V[:, g] / den
    return out
