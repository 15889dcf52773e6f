"""A layer's run of the latent operators, each step held to its own definition: the
cached rows and the turned q to the inputs, each attention to the rows or projections
that it was given, and the absorbed form, projected up, to the layer's formula.

``Layer.run(ops)`` takes the operators from ``ops``: the package's, or the definitions
with a fault planted in them (which the checks have to find)."""
import math

import torch

import paged_varlen_attention_attn_gb300 as pa
from latent_ref import assert_close, attend, cos_sin_table, normed, turned

H, DC, DN, DR, BS = 16, 512, 128, 64, 16
U = 2.0 ** -8  # half a step of bf16


class Package:
    """The operators under test."""

    def write(self, s, q, down, slots, pos):
        rows = torch.empty_like(down)
        q_rope = None if q is None else q[..., DN:]
        pa.latent_rope_and_cache(q_rope, down[:, :DC], down[:, DC:], s.cache, slots, pos, s.cos_sin,
                                 block_size=BS, interleaved=True, latent_norm=s.norm, q_out=q_rope,
                                 row_out=rows)
        return rows

    def absorbed(self, s, q):
        return pa.latent_forward(q, s.cache, s.table, s.seq_lens, s.starts, scale=s.scale,
                                 latent_size=DC, block_size=BS, max_query_len=max(s.new))

    def read_back(self, s):
        return pa.gather_latent(s.cache, s.table, s.key_starts, num_rows=sum(s.lens), latent_size=DC,
                                block_size=BS)

    def expanded(self, s, q, up, kr):
        return pa.latent_expanded_forward(q, up[..., :DN], kr, up[..., DN:], s.starts, s.key_starts,
                                          scale=s.scale)


def _weigh(q, k, v, scale, causal, dropped=()):
    """The attention as a kernel computes it: weights rounded, their sum not."""
    n, s = q.shape[0], k.shape[0]
    k, v = k.double().expand(s, q.shape[1], -1), v.double().expand(s, q.shape[1], -1)
    x = torch.einsum("nhd,shd->nhs", q.double(), k) * scale
    if causal:
        x = x.masked_fill((torch.arange(s)[None] > torch.arange(s - n, s)[:, None])[:, None], -math.inf)
    x[..., list(dropped)] = -math.inf
    w = torch.exp(x - x.amax(-1, keepdim=True))
    return (torch.einsum("nhs,shd->nhd", w.bfloat16().double(), v) / w.sum(-1)[..., None]).bfloat16()


class Definition:
    """The operators from their formulas on the CPU.  ``fault``: what the absorbed form
    does wrong."""

    def __init__(self, fault=None):
        self.fault = fault

    def write(self, s, q, down, slots, pos):
        if q is not None:
            q[..., DN:] = turned(q[..., DN:], s.cos_sin, pos, True).bfloat16()
        key = turned(down[:, None, DC:], s.cos_sin, pos, True)[:, 0]
        rows = torch.cat([normed(down[:, :DC], s.norm, 1e-6), key], 1).bfloat16()
        if self.fault == "rows not turned":
            rows[:, DC:] = down[:, DC:]
        s.cache.view(-1, DC + DR)[slots] = rows
        return rows

    def absorbed(self, s, q):
        out, t = torch.empty(q.shape[0], H, DC, dtype=torch.bfloat16), 0
        for r, (n, keys) in enumerate(zip(s.new, s.lens)):
            rows = s.cached(r)[:, None]
            mine = q[t:t + n].clone()
            if self.fault == "no rotary part":
                mine[..., DC:] = 0
            drop = range(keys // 2, keys // 2 + 16) if self.fault == "16 keys lost" and keys > 40 else ()
            out[t:t + n] = _weigh(mine, rows, rows[..., :DC], s.scale, self.fault != "no causal mask", drop)
            if self.fault == "uniform weights":
                out[t:t + n] = rows[..., :DC].double().mean(0).bfloat16()
            t += n
        return out

    def read_back(self, s):
        return torch.cat([s.cached(r) for r in range(len(s.lens))]).split([DC, DR], 1)

    def expanded(self, s, q, up, kr):
        out, t, k = torch.empty(q.shape[0], H, DN, dtype=torch.bfloat16), 0, 0
        for n, keys in zip(s.new, s.lens):
            full = torch.cat([up[k:k + keys, :, :DN], kr[k:k + keys, None].expand(keys, H, DR)], -1)
            out[t:t + n] = _weigh(q[t:t + n], full, up[k:k + keys, :, DN:], s.scale, True)
            t, k = t + n, k + keys
        return out


def _near(got, ref, size):
    """A few fp32 operations rounded once: half a step and 2^-21 of the operands' size,
    and the norm's sum of 512 terms of one sign, 2^-16 of it."""
    off = (got.double() - ref).abs() - (U * ref.abs() + (2.0 ** -21 + 2.0 ** -16) * size)
    assert off.max() <= 0, off.max().item()


class Layer:
    """Chunks and single tokens on cached context, one of a single key."""

    def __init__(self, device):
        g = torch.Generator().manual_seed(1)

        def randn(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g) * scale).bfloat16().to(device)

        self.ctx, self.new = [100, 37, 300, 64, 0], [20, 33, 1, 1, 1]
        self.lens = [a + b for a, b in zip(self.ctx, self.new)]
        need = [(s + BS - 1) // BS for s in self.lens]
        perm = torch.randperm(sum(need) + 2, generator=g).int()
        table = torch.zeros(len(need), max(need), dtype=torch.int32)
        at = 0
        for r, n in enumerate(need):
            table[r, :n] = perm[at:at + n]
            at += n
        self.table = table.to(device)
        self.cache = torch.full((sum(need) + 2, BS, DC + DR), math.nan, dtype=torch.bfloat16, device=device)
        self.cos_sin = cos_sin_table(512, DR)[0].to(device)
        self.norm = (1 + 0.1 * torch.randn(DC, generator=g)).bfloat16().to(device)
        self.w_k, self.w_v = randn(H, DN, DC, scale=DC ** -0.5), randn(H, DN, DC, scale=DC ** -0.5)
        self.down = [randn(n, DC + DR) for n in self.lens]  # by request
        self.q = randn(sum(self.new), H, DN + DR)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=device)
        self.starts = torch.tensor([0] + self.new).cumsum(0).int().to(device)
        self.key_starts = torch.tensor([0] + self.lens).cumsum(0).int().to(device)
        self.scale = (DN + DR) ** -0.5
        self.device = device

    def cached(self, r):
        key = torch.arange(self.lens[r], device=self.device)
        return self.cache[self.table[r][key // BS].long(), key % BS]

    def _step(self, ops, q, spans):
        key = [torch.arange(a, b, device=self.device) for _, a, b in spans]
        slots = torch.cat([self.table[r][k // BS].long() * BS + k % BS for (r, _, _), k in zip(spans, key)])
        down = torch.cat([self.down[r][a:b] for r, a, b in spans])
        return ops.write(self, q, down, slots, torch.cat(key))

    def run(self, ops):
        self._step(ops, None, [(r, 0, n) for r, n in enumerate(self.ctx)])
        self.q_in = self.q.clone()
        spans = [(r, c, c + n) for r, (c, n) in enumerate(zip(self.ctx, self.new))]
        self.rows = self._step(ops, self.q, spans)
        self.absorbed_q = torch.cat([
            torch.einsum("thd,hde->the", self.q[..., :DN].double(), self.w_k.double()).bfloat16(),
            self.q[..., DN:]], -1)
        self.latent = ops.absorbed(self, self.absorbed_q)
        self.c, self.kr = ops.read_back(self)
        self.up = torch.cat([torch.einsum("ke,hde->khd", self.c.double(), w.double())
                             for w in (self.w_k, self.w_v)], -1).bfloat16()
        self.expanded = ops.expanded(self, self.q, self.up, self.kr)

    # ---------------------------------------------------------------- the checks

    def check_rows(self):
        pos = torch.cat([torch.arange(n, device=self.device) for n in self.lens])
        down = torch.cat(self.down)
        lat = normed(down[:, :DC], self.norm, 1e-6)
        _near(self.c, lat, lat.abs())
        _near(self.kr, turned(down[:, None, DC:], self.cos_sin, pos, True)[:, 0],
              2 * down[:, DC:].double().abs().amax(-1, keepdim=True))
        mine = torch.cat([torch.arange(c, c + n, device=self.device) for c, n in zip(self.ctx, self.new)])
        _near(self.q[..., DN:], turned(self.q_in[..., DN:], self.cos_sin, mine, True),
              2 * self.q_in[..., DN:].double().abs().amax(-1, keepdim=True))
        assert torch.equal(self.q[..., :DN], self.q_in[..., :DN])
        at = 0
        for r, (c, n) in enumerate(zip(self.ctx, self.new)):
            assert torch.equal(self.rows[at:at + n], self.cached(r)[c:])
            at += n

    def _requests(self):
        t = k = 0
        for n, s in zip(self.new, self.lens):
            yield slice(t, t + n), slice(k, k + s), n, s
            t, k = t + n, k + s

    def check_absorbed(self):
        """In the latents' own space, on the rows that are in the cache."""
        for ts, ks, n, s in self._requests():
            rows = torch.cat([self.c[ks], self.kr[ks]], 1)[:, None]
            out, w, size = attend(self.absorbed_q[ts], rows, rows[..., :DC], self.scale, 1)
            assert_close(self.latent[ts], out, w, size, scale=self.scale, depth=DC + DR, keys=s,
                         most=1.0, dtype=torch.bfloat16, what=(n, s))

    def check_expanded(self):
        for ts, ks, n, s in self._requests():
            keys = torch.cat([self.up[ks, :, :DN], self.kr[ks, None].expand(s, H, DR)], -1)
            out, w, size = attend(self.q[ts], keys, self.up[ks, :, DN:], self.scale, 1)
            assert_close(self.expanded[ts], out, w, size, scale=self.scale, depth=DN + DR, keys=s,
                         most=1.0, dtype=torch.bfloat16, what=(n, s))

    def check_formula(self):
        """Both forms, projected up, against the layer's formula in 64 bits.

        Independent roundings of up to u |x_e| each in a sum over e exceed 8 u ||x||
        with a probability below 2 exp(-32) (Hoeffding), which no test meets.  So a
        score is off by 8 u scale ||q_e k_e|| for rounded operands, a weight by twice
        that (itself and the normaliser) and by u for its own rounding, and a result by
        8 u ||.|| of the rounded terms that it is a sum of.  The fp32 sums add 2^-10 of
        the weighted values, far more than the attentions' own checks allow."""
        for ts, ks, n, s in self._requests():
            c = self.c[ks].double()
            k_n = torch.einsum("ke,hde->khd", c, self.w_k.double())
            v = torch.einsum("ke,hde->khd", c, self.w_v.double())
            keys = torch.cat([k_n, self.kr[ks, None].double().expand(s, H, DR)], -1)
            ref, weighted, _ = attend(self.q[ts], keys, v, self.scale, 1)

            def slack(moved, last):
                return (U + torch.expm1(2 * moved) + 2.0 ** -10) * weighted + last

            aq = self.absorbed_q[ts][..., :DC].double()
            moved = 8 * U * self.scale * torch.einsum("the,ke->thk", aq ** 2, c ** 2).amax(-1).sqrt()[..., None]
            lat = self.latent[ts].double()
            last = 8 * U * torch.einsum("the,hde->thd", lat ** 2, self.w_v.double() ** 2).sqrt()
            got = torch.einsum("the,hde->thd", lat, self.w_v.double())
            assert ((got - ref).abs() <= slack(moved, last)).all(), (n, s)
            q = self.q[ts][..., :DN].double()
            moved = 8 * U * self.scale * torch.einsum("thd,khd->thk", q ** 2, k_n ** 2).amax(-1).sqrt()[..., None]
            # (a rounded value's error is at most u |v|: u of the weighted values)
            off = (self.expanded[ts].double() - ref).abs()
            assert (off <= slack(moved, U * weighted + U * ref.abs())).all(), (n, s)
