"""Plain definitions in 64 bits of attention over one shared latent vector a token,
random cases of it, and how far a kernel of 16-bit operands may be off."""
import math

import torch

import paged_varlen_attention_attn_gb300 as pa
from row_ref import cos_sin_table

DTYPES = {pa.KV_BF16: torch.bfloat16, pa.KV_F16: torch.float16}


def attend(q, k, v, scale, causal):
    """Rows q [n, H, d] at the end of keys k [s, H or 1, d], values v [s, H or 1, dv], in
    64 bits: (out, sum of |weight * value|, largest sum of |q k| a row has)."""
    q, k, v = q.double(), k.double(), v.double()
    n, s = q.shape[0], k.shape[0]
    H = q.shape[1]
    k, v = k.expand(s, H, -1), v.expand(s, H, -1)
    x = torch.einsum("nhd,shd->nhs", q, k) * scale
    if causal:
        hidden = torch.arange(s, device=q.device)[None] > torch.arange(s - n, s, device=q.device)[:, None]
        x = x.masked_fill(hidden[:, None], -math.inf)
    p = torch.softmax(x, -1)
    size = torch.einsum("nhd,shd->nhs", q.abs(), k.abs()).amax(-1)
    return (torch.einsum("nhs,shd->nhd", p, v), torch.einsum("nhs,shd->nhd", p, v.abs()), size)


def bound(out, weighted, size, scale, depth, keys, most, dtype):
    """How far an element of the kernels' output may be from ``out``.

    Weights and result are rounded to dtype (half a step u each); scores are fp32
    sums of ``depth`` exact products, each addition off by 2^-23 of the sum of
    magnitudes at most, which moves a weight and the normaliser by the same factor,
    exp2 and the scale by 2^-21 more; O and the sum are fp32 sums over the keys;
    an f16 weight below 2^-14 is off by 2^-25 (the largest weight is 1 or more)."""
    u = torch.finfo(dtype).eps / 2
    shift = scale * size[..., None] * depth * 2.0 ** -23 + 2.0 ** -21 + keys * 2.0 ** -23
    tiny = keys * 2.0 ** -25 * most if dtype == torch.float16 else 0.0
    return (u + 2 * shift) * weighted + u * out.abs() + tiny + 1e-30


def assert_close(got, ref, weighted, size, *, scale, depth, keys, most, dtype, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), what
    off = (got - ref).abs() / bound(ref, weighted, size, scale, depth, keys, most, dtype)
    assert off.max() <= 1, (what, off.max().item())


class Paged:
    """A batch [(new tokens, keys)] over a shuffled pool of latent rows."""

    def __init__(self, seed, lens, *, H, dc, dr, bs, kv_dtype=pa.KV_BF16, device="cpu", spread=0.3,
                 spare=2, poison=False):
        g = torch.Generator().manual_seed(seed)
        dt = DTYPES[kv_dtype]
        self.lens, self.H, self.dc, self.dr, self.bs, self.kv_dtype = lens, H, dc, dr, bs, kv_dtype
        need = [(s + bs - 1) // bs for _, s in lens]
        self.nb = sum(need) + spare
        perm = torch.randperm(self.nb, generator=g).int()
        self.table = torch.full((len(lens), max(need + [1]) + 1), -7, dtype=torch.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = perm[at:at + n]
            at += n
        cache = torch.randn(self.nb, bs, dc + dr, generator=g)
        self.cache = (cache * torch.exp(spread * torch.randn(self.nb, bs, 1, generator=g))).to(dt)
        if poison:  # every slot that holds no key of the batch
            used = torch.zeros(self.nb, bs, dtype=torch.bool)
            for r, (_, s) in enumerate(lens):
                key = torch.arange(s)
                used[self.table[r][key // bs].long(), key % bs] = True
            bad = torch.tensor([math.nan, math.inf, -math.inf])[torch.arange(self.nb * bs) % 3]
            self.cache[~used] = bad.view(self.nb, bs)[~used][:, None].to(dt)
        self.T = sum(n for n, _ in lens)
        self.q = torch.randn(self.T, H, dc + dr, generator=g).to(dt)
        self.seq_lens = torch.tensor([s for _, s in lens], dtype=torch.int32)
        self.starts = torch.tensor([0] + [n for n, _ in lens]).cumsum(0).int()
        self.scale = 1 / math.sqrt(128 + dr)
        self.max_q = max([n for n, _ in lens] + [0])
        for name in ("table", "cache", "q", "seq_lens", "starts"):
            setattr(self, name, getattr(self, name).to(device))

    def rows(self, r):
        s = self.lens[r][1]
        key = torch.arange(s, device=self.cache.device)
        return self.cache[self.table[r][key // self.bs].long(), key % self.bs]

    def run(self, causal=1, **kw):
        kw.setdefault("max_query_len", self.max_q)
        return pa.latent_forward(self.q, self.cache, self.table, self.seq_lens, self.starts,
                                 scale=self.scale, latent_size=self.dc, block_size=self.bs,
                                 causal=causal, kv_dtype=self.kv_dtype, **kw)

    def check(self, got, causal=1, requests=None):
        t = 0
        for r, (n, s) in enumerate(self.lens):
            if n > 0 and (requests is None or r in requests):
                rows = self.rows(r)[:, None]
                ref, w, size = attend(self.q[t:t + n], rows, rows[..., :self.dc], self.scale, causal)
                assert_close(got[t:t + n], ref, w, size, scale=self.scale, depth=self.dc + self.dr,
                             keys=s, most=rows.abs().max().double(), dtype=self.q.dtype,
                             what=(r, n, s))
            t += n


class Dense:
    """Ragged requests [(rows, keys)] of the expanded form; k_nope and value are views
    of one projection."""

    def __init__(self, seed, lens, *, H, dn, dr, kv_dtype=pa.KV_BF16, device="cpu"):
        g = torch.Generator().manual_seed(seed)
        dt = DTYPES[kv_dtype]
        self.lens, self.kv_dtype = lens, kv_dtype
        T, K = sum(n for n, _ in lens), sum(s for _, s in lens)
        self.q = torch.randn(T, H, dn + dr, generator=g).to(dt).to(device)
        self.up = torch.randn(K, H, 2 * dn, generator=g).to(dt).to(device)
        self.k_nope, self.value = self.up.split([dn, dn], 2)
        self.k_rope = torch.randn(K, dr, generator=g).to(dt).to(device)
        self.starts = torch.tensor([0] + [n for n, _ in lens]).cumsum(0).int().to(device)
        self.key_starts = torch.tensor([0] + [s for _, s in lens]).cumsum(0).int().to(device)
        self.scale = 1 / math.sqrt(dn + dr)

    def run(self, causal=1, **kw):
        return pa.latent_expanded_forward(self.q, self.k_nope, self.k_rope, self.value, self.starts,
                                          self.key_starts, scale=self.scale, causal=causal,
                                          kv_dtype=self.kv_dtype, **kw)

    def check(self, got, causal=1, requests=None):
        H, dn = self.k_nope.shape[1:]
        t = k = 0
        for r, (n, s) in enumerate(self.lens):
            if n > 0 and (requests is None or r in requests):
                if s == 0:
                    assert (got[t:t + n] == 0).all()
                else:
                    keys = torch.cat([self.k_nope[k:k + s], self.k_rope[k:k + s, None].expand(s, H, -1)], -1)
                    for i in range(0, n, 512):  # (a piece of the rows at a time)
                        m = min(512, n - i)
                        seen = s - n + i + m if causal else s
                        ref, w, size = attend(self.q[t + i:t + i + m], keys[:seen],
                                              self.value[k:k + seen], self.scale, causal)
                        assert_close(got[t + i:t + i + m], ref, w, size, scale=self.scale,
                                     depth=keys.shape[-1], keys=s, most=self.value.abs().max().double(),
                                     dtype=self.q.dtype, what=(r, n, s, i))
            t, k = t + n, k + s


def turned(x, table, positions, interleaved):
    """x [T, h, dr] in 64 bits, turned by the fp32 table's own values."""
    x = x.double()
    dr = x.shape[-1]
    c, s = table[positions].double()[:, None].chunk(2, -1)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)
    y, z = a * c - b * s, b * c + a * s
    return torch.stack([y, z], -1).flatten(-2) if interleaved else torch.cat([y, z], -1)


def normed(x, weight, eps):
    x = x.double()
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double()


__all__ = ["Paged", "Dense", "attend", "bound", "assert_close", "turned", "normed", "cos_sin_table",
           "DTYPES"]
