"""Long contexts whose values tell which keys were added up: the keys of a run of 16 share
one dim of the latent, in which the others hold zero.  A dim of the output is then the
weight of a few runs (two or three at 20000 keys and 512 dims), and a tile that is lost,
or taken twice, moves it by a third or more of itself, where roundings move it by half
a percent."""
import math

import torch

from latent_ref import DTYPES, Paged

RUN = 16


def planted(seed, lens, *, H, dc, dr, bs, kv_dtype, device):
    """A Paged batch with such latents; scores come from the rotary parts too."""
    c = Paged(seed, lens, H=H, dc=dc, dr=dr, bs=bs, kv_dtype=kv_dtype, device=device, spread=0.0)
    g = torch.Generator().manual_seed(seed + 1)
    for r, (_, s) in enumerate(lens):
        key = torch.arange(s)
        value = 1 + torch.rand(s, generator=g)
        lat = torch.zeros(s, dc).scatter_(1, (key // RUN % dc)[:, None], value[:, None])
        key = key.to(device)
        c.cache[c.table[r][key // bs].long(), key % bs, :dc] = lat.to(DTYPES[kv_dtype]).to(device)
    return c


def weights(c, r, causal=1):
    """Of request r's rows, in 64 bits: (exp(score - largest) [n, H, s], the largest sum
    of |q k| a row has [n, H])."""
    n, s = c.lens[r]
    t = sum(m for m, _ in c.lens[:r])
    q, rows = c.q[t:t + n].double(), c.rows(r).double()
    x = torch.einsum("nhd,sd->nhs", q, rows) * c.scale
    if causal:
        at = torch.arange(s, device=x.device)
        x = x.masked_fill((at[None] > at[s - n:, None])[:, None], -math.inf)
    size = torch.einsum("nhd,sd->nhs", q.abs(), rows.abs()).amax(-1)
    return torch.exp(x - x.amax(-1, keepdim=True)), size


def bound(c, r, w, size):
    """How far the kernels' output may be from sum w v / sum w, dim by dim.

    Half a step u for each weight and for the result; scores, O and the normaliser are
    fp32 sums, each addition off by 2^-23 of the sum of magnitudes at most; exp2 and the
    scale by 2^-21.  An f16 weight is at least w of the largest one (the reference that it
    is taken against is at most the largest score): only where w is below 2^-14 may it be
    subnormal, and then it is off by 2^-25 of the largest weight."""
    dt = c.q.dtype
    u = torch.finfo(dt).eps / 2
    s = c.lens[r][1]
    v = c.rows(r)[:, :c.dc].double()
    total = w.sum(-1, keepdim=True)
    out = torch.einsum("nhs,sd->nhd", w, v) / total  # (no value is negative)
    shift = c.scale * size[..., None] * (c.dc + c.dr) * 2.0 ** -23 + 2.0 ** -21 + s * 2.0 ** -23
    off = (2 * u + 2 * shift) * out + 1e-30
    if dt == torch.float16:
        # (and a result below f16's normal range is off by half of its smallest step)
        off += 2.0 ** -25 * torch.einsum("nhs,sd->nhd", (w < 2.0 ** -14).double(), v) / total + 2.0 ** -25
    return out, off


def check(c, got, causal=1):
    t = 0
    for r, (n, _) in enumerate(c.lens):
        w, size = weights(c, r, causal)
        out, off = bound(c, r, w, size)
        x = ((got[t:t + n].double() - out).abs() / off).max().item()
        assert x <= 1, (r, x)
        t += n
