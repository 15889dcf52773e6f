"""The operators around a cache of 8-bit rows, each with what it has to do.

A serving step over a paged cache whose keys and values are held as e4m3 codes
with one fp32 scale per (token, KV head) row takes three kinds of call:

  rope_cache  rotates the step's q and k heads (one position per token, or a
              time / height / width position per rotary pair; optionally a
              root-mean-square norm per head first) and writes k and v into
              the cache, quantised on the way;
  read_back   gathers ranges of cached keys and values of many requests into
              contiguous 16-bit rows;
  attend      attention of single tokens and of chunks of new tokens over the
              cache.

``own`` False computes them with elementary torch operations in fp32, rounded
once; ``own`` True calls this repository's package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
SCALE_MIN, SCALE_MAX = 2.0 ** -60, 2.0 ** 60
NORM_EPS = 1e-6
ROPE_BASE = 10000.0


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one new token of one request, heads of the decode benchmark: latency
        dict(name="rope_one_token", op="rope_cache", tokens=1, heads=32, kv_heads=8, head_size=128,
             rot_dim=128, axes=1, adjacent=False, norm=False, cache="rows", block_size=16,
             positions=32768),
        # all tokens of the mixed benchmark step (4 chunks of 2048 and 192 decodes)
        dict(name="rope_mixed_step", op="rope_cache", tokens=8384, heads=64, kv_heads=8,
             head_size=128, rot_dim=128, axes=1, adjacent=False, norm=False, cache="rows",
             block_size=16, positions=32768),
        # a video prompt: time, height and width positions, normed heads
        dict(name="rope_video", op="rope_cache", tokens=5003, heads=32, kv_heads=4, head_size=128,
             rot_dim=128, axes=3, adjacent=False, norm=True, cache="rows", block_size=64,
             positions=8192),
        # a small model that rotates half of each head, adjacent pairs, bf16 cache
        dict(name="rope_half_rotated", op="rope_cache", tokens=777, heads=16, kv_heads=2,
             head_size=64, rot_dim=32, axes=1, adjacent=True, norm=False, cache="bf16",
             block_size=16, positions=4096),
        # a few short prefixes taken out of the cache
        dict(name="read_back_short", op="read_back", seqs=4, lo=1, hi=90, kv_heads=8,
             head_size=128, block_size=16, cache="rows", lengths=11),
        # every key of the decode benchmark's batch, to hand it to another instance
        dict(name="read_back_batch", op="read_back", seqs=64, lo=512, hi=4096, kv_heads=8,
             head_size=128, block_size=16, cache="rows", lengths=12),
        # the tiny batch: one prefill of 8 tokens beside one decode
        dict(name="attend_tiny", op="attend", chunks=1, chunk_lo=8, chunk_hi=8, ctx_lo=0, ctx_hi=0,
             decodes=1, key_lo=40, key_hi=40, heads=4, kv_heads=2, head_size=64, block_size=16,
             window=0, lengths=21),
        # a decode batch: the benchmark's 64 requests
        dict(name="attend_decode", op="attend", chunks=0, chunk_lo=0, chunk_hi=0, ctx_lo=0,
             ctx_hi=0, decodes=64, key_lo=512, key_hi=4096, heads=32, kv_heads=8, head_size=128,
             block_size=16, window=0, lengths=22),
        # few requests with long contexts: the keys are split over the GPU
        dict(name="attend_long", op="attend", chunks=0, chunk_lo=0, chunk_hi=0, ctx_lo=0, ctx_hi=0,
             decodes=8, key_lo=120001, key_hi=131072, heads=64, kv_heads=8, head_size=128,
             block_size=64, window=0, lengths=23),
        # chunks of 2048 new tokens on a context, sliding window
        dict(name="attend_chunks", op="attend", chunks=4, chunk_lo=2048, chunk_hi=2048,
             ctx_lo=6144, ctx_hi=6144, decodes=0, key_lo=0, key_hi=0, heads=64, kv_heads=8,
             head_size=128, block_size=16, window=4096, lengths=24),
        # ragged whole prompts
        dict(name="attend_prompts", op="attend", chunks=8, chunk_lo=512, chunk_hi=4096, ctx_lo=0,
             ctx_hi=0, decodes=0, key_lo=0, key_hi=0, heads=32, kv_heads=8, head_size=128,
             block_size=16, window=0, lengths=25),
        # a serving step: chunks of prompts beside decodes
        dict(name="attend_step", op="attend", chunks=3, chunk_lo=300, chunk_hi=1024, ctx_lo=0,
             ctx_hi=5000, decodes=96, key_lo=200, key_hi=8192, heads=32, kv_heads=4,
             head_size=128, block_size=16, window=0, lengths=26),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_cache", "read_back", "attend", "attend"])
    heads, kv_heads = rng.choice([(4, 2), (6, 2), (16, 2), (28, 4), (32, 4), (32, 8), (8, 8), (64, 8)])
    block_size = rng.choice([16, 16, 32, 64, 128])
    if op == "rope_cache":
        head_size = rng.choice([64, 96, 128, 128, 256])
        return dict(op=op, tokens=_log_int(rng, 1, 4000), heads=heads, kv_heads=kv_heads,
                    head_size=head_size, rot_dim=rng.choice([head_size, head_size, head_size // 2]),
                    axes=rng.choice([1, 1, 3]), adjacent=rng.random() < 0.3,
                    norm=rng.random() < 0.4, cache=rng.choice(["rows", "rows", "e4m3", "bf16"]),
                    block_size=block_size, positions=_log_int(rng, 1000, 40000))
    if op == "read_back":
        lo = _log_int(rng, 1, 1500)
        return dict(op=op, seqs=_log_int(rng, 1, 64), lo=lo, hi=lo + _log_int(rng, 1, 2500),
                    kv_heads=kv_heads, head_size=rng.choice([64, 128]), block_size=block_size,
                    cache=rng.choice(["rows", "rows", "e4m3", "bf16"]),
                    lengths=rng.randrange(1 << 20))
    case = dict(op=op, chunks=0, chunk_lo=0, chunk_hi=0, ctx_lo=0, ctx_hi=0, decodes=0, key_lo=0,
                key_hi=0, heads=heads, kv_heads=kv_heads, head_size=rng.choice([64, 128, 128]),
                block_size=block_size, window=rng.choice([0, 0, 0, _log_int(rng, 60, 4000)]),
                lengths=rng.randrange(1 << 20))
    kind = rng.choice(["decode", "chunk", "both"])
    if kind != "decode":
        lo = _log_int(rng, 2, 900)
        ctx = rng.choice([0, _log_int(rng, 1, 3000)])
        case.update(chunks=rng.randint(1, 4), chunk_lo=lo, chunk_hi=lo + _log_int(rng, 1, 900),
                    ctx_lo=ctx // 2, ctx_hi=ctx)
    if kind != "chunk":
        lo = _log_int(rng, 1, 12000)
        case.update(decodes=_log_int(rng, 1, 96), key_lo=lo, key_hi=lo + _log_int(rng, 1, 6000))
    return case


def _lengths(c):
    """[(new tokens, keys)] of the batch's requests, from the case alone."""
    r = random.Random(c["lengths"])
    if c["op"] == "read_back":
        return [(0, r.randint(c["lo"], c["hi"])) for _ in range(c["seqs"])]
    out = []
    for _ in range(c["chunks"]):
        n = r.randint(c["chunk_lo"], c["chunk_hi"])
        out.append((n, n + r.randint(c["ctx_lo"], c["ctx_hi"])))
    return out + [(1, r.randint(c["key_lo"], c["key_hi"])) for _ in range(c["decodes"])]


def _visible(q, s, w):
    """Visible (row, key) pairs of one head of a request, and its visible keys."""
    ctx = s - q
    if w <= 0:
        return q * ctx + q * (q + 1) // 2, s
    grow = max(0, min(q, w - ctx))  # rows whose window still reaches key 0
    pairs = grow * ctx + grow * (grow + 1) // 2 + (q - grow) * w
    return pairs, min(s, q + w - 1)


def work(c):
    d, g = c["head_size"], c["kv_heads"]
    row = {"rows": d + 4, "e4m3": d, "bf16": 2 * d}[c.get("cache", "rows")]  # a stored row's bytes
    if c["op"] == "rope_cache":
        t, h = c["tokens"], c["heads"]
        table = 4 * c["rot_dim"] * min(t * min(c["axes"], 3), c["positions"])
        data = t * (2 * h * d * 2 + 2 * g * d * 2 + 2 * g * row + 8 * c["axes"] + 8)
        flops = t * ((h + g) * c["rot_dim"] * 3 + (4 * (h + g) * d if c["norm"] else 0) + 2 * g * d)
        return {"bytes": data + table, "flops": flops}
    lens = _lengths(c)
    if c["op"] == "read_back":
        keys = sum(s for _, s in lens)
        return {"bytes": keys * 2 * g * (row + 2 * d) + 4 * keys // c["block_size"], "flops": keys * 2 * g * d}
    seen = [_visible(q, s, c["window"]) for q, s in lens]
    return {"bytes": sum(2 * g * row * k for _, k in seen) + 4 * sum(k for _, k in seen) // c["block_size"]
            + sum(4 * c["heads"] * d * q for q, _ in lens),
            "flops": 4 * d * c["heads"] * sum(p for p, _ in seen)}


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _quantised_pool(g, blocks, c):
    """A filled cache [2, blocks, bs, Hkv, d] and what its codes are scaled by."""
    bs, hkv, d = c["block_size"], c["kv_heads"], c["head_size"]
    kind = c.get("cache", "rows")
    cache = torch.empty((2, blocks, bs, hkv, d), device=DEV,
                        dtype=torch.bfloat16 if kind == "bf16" else torch.uint8)
    scales = torch.empty((blocks, bs // 16, hkv, 2, 16), device=DEV)
    tensor_scale = (4.0 / E4M3_MAX, 5.0 / E4M3_MAX)
    for kv in range(2):
        # rows of uneven size, as heads and tokens of a model have
        x = _randn(g, blocks, bs, hkv, d) * torch.exp(0.4 * _randn(g, blocks, bs, hkv, 1))
        if kind == "bf16":
            cache[kv] = x.bfloat16()
        elif kind == "e4m3":
            cache[kv] = (x / tensor_scale[kv]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            s = x.abs().amax(-1, keepdim=True) / E4M3_MAX
            cache[kv] = (x / s).to(torch.float8_e4m3fn).view(torch.uint8)
            scales[:, :, :, kv] = s.view(blocks, bs // 16, 16, hkv).transpose(2, 3)
        del x
    return cache, scales if kind == "rows" else tensor_scale if kind == "e4m3" else None


def _tables(g, lens, bs):
    """A block table over a permuted pool, the pool's size and the widest row."""
    need = [(s + bs - 1) // bs for _, s in lens]
    blocks = sum(need) + 3
    perm = torch.randperm(blocks, generator=g, device=DEV).int()
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    return table, blocks


def _starts(counts):
    return torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).int().to(DEV)


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = dict(case=c)
    d, hkv, bs = c["head_size"], c["kv_heads"], c["block_size"]
    if c["op"] == "rope_cache":
        t, h, rot = c["tokens"], c["heads"], c["rot_dim"]
        blocks = (t + bs - 1) // bs * 2 + 8
        # q, k and v side by side, as one projection leaves them
        st["qkv"] = _randn(g, t, (h + 2 * hkv) * d).bfloat16()
        st["q_out"] = torch.zeros((t, h, d), dtype=torch.bfloat16, device=DEV)
        if c["axes"] == 1:
            first = torch.randint(0, max(1, c["positions"] - t), (1,), generator=g, device=DEV)
            st["positions"] = (first + torch.arange(t, device=DEV)) % c["positions"]
            st["pair_axis"] = None
        else:
            st["positions"] = torch.randint(0, c["positions"], (c["axes"], t), generator=g, device=DEV)
            # a quarter of the pairs by time, the rest by height and width
            a = rot // 8
            b = (rot // 2 - a) // 2
            st["pair_axis"] = [0] * a + [1] * b + [2] * (rot // 2 - a - b)
        freq = ROPE_BASE ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) * 2 / rot)
        angle = torch.arange(c["positions"], device=DEV, dtype=torch.float64)[:, None] * freq
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        st["q_norm"] = (1 + 0.1 * _randn(g, d)).bfloat16() if c["norm"] else None
        st["k_norm"] = (1 + 0.1 * _randn(g, d)).bfloat16() if c["norm"] else None
        slots = torch.randperm(blocks * bs, generator=g, device=DEV)[:t]
        slots[torch.rand(t, generator=g, device=DEV) < 0.01] = -1  # a few padding tokens
        st["slots"] = slots
        st["cache"], st["scale"] = _quantised_pool(g, blocks, c)
        return st
    lens = _lengths(c)
    st["table"], blocks = _tables(g, lens, bs)
    st["cache"], st["scale"] = _quantised_pool(g, blocks, c)
    st["max_s"] = max(s for _, s in lens)
    if c["op"] == "read_back":
        st["starts"] = _starts([s for _, s in lens])
        st["rows"] = sum(s for _, s in lens)
        return st
    st["seq_lens"] = torch.tensor([s for _, s in lens], dtype=torch.int32, device=DEV)
    st["starts"] = _starts([q for q, _ in lens])
    st["max_q"] = max(q for q, _ in lens)
    st["q"] = _randn(g, sum(q for q, _ in lens), c["heads"], d).bfloat16()
    # requests that are served together: the chunks, then the single tokens
    st["groups"] = [(a, b, max(q for q, _ in lens[a:b]), max(s for _, s in lens[a:b]))
                    for a, b in ((0, c["chunks"]), (c["chunks"], len(lens))) if b > a]
    return st


# ---------------------------------------------------------------- plain forms

def _stored(st, cache, which, index):
    """Rows of the cache as fp32 values: cache[which] viewed by block and slot."""
    kind = st["case"].get("cache", "rows")
    blk, slot = index
    rows = cache[which][blk, slot]
    if kind == "bf16":
        return rows.float()
    rows = rows.view(torch.float8_e4m3fn).float()
    if kind == "e4m3":
        return rows * st["scale"][which]
    return rows * st["scale"][blk, slot // 16, :, which, slot % 16][..., None]


def _rms(x, weight):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + NORM_EPS) * weight.float()


def _turned(x, cos, sin, rot, adjacent):
    head, rest = x[..., :rot], x[..., rot:]
    if adjacent:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _plain_rope(st):
    c = st["case"]
    t, h, hkv, d, rot, bs = (c[k] for k in ("tokens", "heads", "kv_heads", "head_size", "rot_dim", "block_size"))
    x = st["qkv"].float().view(t, h + 2 * hkv, d)
    q, k, v = x[:, :h], x[:, h:h + hkv], x[:, h + hkv:]
    if c["norm"]:
        q, k = _rms(q, st["q_norm"]), _rms(k, st["k_norm"])
    pair = torch.arange(rot // 2, device=DEV)
    if st["pair_axis"] is None:
        pos = st["positions"][:, None].expand(t, rot // 2)
    else:
        pos = st["positions"][torch.tensor(st["pair_axis"], device=DEV)].t()
    cos, sin = st["cos_sin"][pos, pair][:, None], st["cos_sin"][pos, pair + rot // 2][:, None]
    q, k = _turned(q, cos, sin, rot, c["adjacent"]), _turned(k, cos, sin, rot, c["adjacent"])
    st["q_out"].copy_(q)
    keep = st["slots"] >= 0
    slot = st["slots"][keep]
    blk, off = slot // bs, slot % bs
    for which, rows in ((0, k[keep]), (1, v[keep])):
        if c["cache"] == "bf16":
            st["cache"][which][blk, off] = rows.bfloat16()
            continue
        if c["cache"] == "e4m3":
            code = rows / st["scale"][which]
        else:
            s = (rows.abs().amax(-1) / E4M3_MAX).clamp(SCALE_MIN, SCALE_MAX)
            st["scale"][blk, off // 16, :, which, off % 16] = s
            code = rows / s[..., None]
        st["cache"][which][blk, off] = code.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_read_back(st):
    bs = st["case"]["block_size"]
    row = torch.arange(st["rows"], device=DEV)
    req = torch.searchsorted(st["starts"], row, right=True) - 1
    key = row - st["starts"][req]
    at = st["table"][req, key // bs].long(), key % bs
    return [_stored(st, st["cache"], kv, at).bfloat16() for kv in (0, 1)]


def _plain_attend(st):
    c = st["case"]
    h, hkv, d, bs, w = c["heads"], c["kv_heads"], c["head_size"], c["block_size"], c["window"]
    out = torch.zeros_like(st["q"])
    for a, b, most_q, most_s in st["groups"]:  # chunks and single tokens: two padded batches
        n = b - a
        first, s = st["starts"][a:b, None].long(), st["seq_lens"][a:b, None].long()
        count = st["starts"][a + 1:b + 1, None].long() - first
        i, key = torch.arange(most_q, device=DEV)[None], torch.arange(most_s, device=DEV)[None]
        live = i < count
        row = torch.where(live, first + i, 0)
        q = st["q"][row].float().view(n, most_q, hkv, h // hkv, d)
        at = st["table"][a:b, :(most_s + bs - 1) // bs].long()[:, key[0] // bs], (key % bs).expand(n, -1)
        k, v = _stored(st, st["cache"], 0, at), _stored(st, st["cache"], 1, at)
        v = v.masked_fill((key >= s)[..., None, None], 0.0)
        p = torch.einsum("nqhgd,nkhd->nhgqk", q, k).mul_(1.0 / math.sqrt(d))
        pos = (s - count + i)[:, :, None]
        seen = (key[:, None] <= pos) & (key[:, None] < s[..., None])
        if w > 0:
            seen = seen & (pos - key[:, None] < w)
        p.masked_fill_(~seen[:, None, None], -math.inf)
        p.sub_(p.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
        o = torch.einsum("nhgqk,nkhd->nqhgd", p, v)
        o = o / p.sum(-1).permute(0, 3, 1, 2)[..., None]
        out[row[live]] = o.reshape(n, most_q, h, d)[live].bfloat16()
        del p
    return out


# --------------------------------------------------------------------- a pass

def _rope_outputs(st):
    """q, the cache as the values of its codes, and their scales."""
    cache = st["cache"]
    out = {"q": st["q_out"], "cache": cache if cache.dtype == torch.bfloat16 else cache.view(torch.float8_e4m3fn)}
    if st["case"]["cache"] == "rows":
        out["scales"] = st["scale"]
    return out


def run(state):
    st = state
    c = st["case"]
    if not own:
        if c["op"] == "rope_cache":
            _plain_rope(st)
            return _rope_outputs(st)
        return _plain_read_back(st) if c["op"] == "read_back" else _plain_attend(st)
    import paged_varlen_attention_attn_gb300 as pa
    kind = {"bf16": pa.KV_BF16, "e4m3": pa.KV_FP8_E4M3, "rows": pa.KV_FP8_E4M3_ROW}[c.get("cache", "rows")]
    if c["op"] == "rope_cache":
        h, hkv, d = c["heads"], c["kv_heads"], c["head_size"]
        q, k, v = st["qkv"].view(c["tokens"], h + 2 * hkv, d).split([h, hkv, hkv], 1)
        pa.rope_and_cache(q, k, v, st["cache"], st["slots"], st["positions"], st["cos_sin"],
                          block_size=c["block_size"], kv_dtype=kind, kv_scale=st["scale"],
                          interleaved=c["adjacent"], pair_axis=st["pair_axis"],
                          q_norm=st["q_norm"], k_norm=st["k_norm"], norm_eps=NORM_EPS,
                          q_out=st["q_out"])
        return _rope_outputs(st)
    if c["op"] == "read_back":
        return list(pa.gather_cache(st["cache"], st["table"], st["starts"], num_rows=st["rows"],
                                    block_size=c["block_size"], kv_dtype=kind, kv_scale=st["scale"]))
    return pa.forward(st["q"], st["cache"], st["table"], st["seq_lens"], st["starts"],
                      scale=1.0 / math.sqrt(c["head_size"]), num_heads=c["heads"],
                      num_kv_heads=c["kv_heads"], head_size=c["head_size"],
                      block_size=c["block_size"], window=c["window"], kv_dtype=kind,
                      kv_scale=st["scale"], max_query_len=st["max_q"], max_seq_len=st["max_s"])


# ---------------------------------------------------------------- in 64 bits

def _dense64(st, r, n):
    """Keys and values 0 .. n - 1 of request r in 64 bits, [2, n, Hkv, d]."""
    c = st["case"]
    bs, kind = c["block_size"], c.get("cache", "rows")
    blocks = st["table"][r, :(n + bs - 1) // bs].long()
    x = st["cache"][:, blocks]
    if kind == "bf16":
        return x.double().flatten(1, 2)[:, :n]
    x = x.view(torch.float8_e4m3fn).to(torch.float32).double()
    if kind == "e4m3":
        s = torch.tensor(st["scale"], dtype=torch.float32, device=DEV).double()[:, None, None, None, None]
    else:  # [block, group, head, 2, 16] -> [2, block, slot, head, 1]
        s = st["scale"][blocks].double().permute(3, 0, 1, 4, 2).flatten(2, 3)[..., None]
    return (x * s).flatten(1, 2)[:, :n]


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    d, hkv, bs = c["head_size"], c["kv_heads"], c["block_size"]
    if c["op"] == "read_back":
        rows = torch.cat([_dense64(st, r, s) for r, (_, s) in enumerate(_lengths(c))], 1)
        return [rows[0], rows[1]]
    if c["op"] == "rope_cache":
        t, h, rot = c["tokens"], c["heads"], c["rot_dim"]
        q, k, v = st["qkv"].double().view(t, -1, d).split([h, hkv, hkv], 1)
        # each pair is a complex number that turns by its angle
        freq = ROPE_BASE ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) * 2 / rot)
        pos = st["positions"].double().view(-1, t)
        axis = torch.tensor(st["pair_axis"] or [0] * (rot // 2), device=DEV)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos[axis].t() * freq)[:, None]

        def spin(x, weight):
            x = x.clone()
            if weight is not None:
                x = x / (x.pow(2).sum(-1, keepdim=True) / d + NORM_EPS).sqrt() * weight.double()
            first, second = (slice(0, rot, 2), slice(1, rot, 2)) if c["adjacent"] else (slice(0, rot // 2), slice(rot // 2, rot))
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            return x

        q, k = spin(q, st["q_norm"]), spin(k, st["k_norm"])
        cache = st["cache"].double() if c["cache"] == "bf16" else st["cache"].view(torch.float8_e4m3fn).to(torch.float32).double()
        flat = cache.view(2, -1, hkv, d)
        live = (st["slots"] >= 0).nonzero()[:, 0]
        at = st["slots"][live]
        out = {"q": q, "cache": cache}
        if c["cache"] == "rows":
            out["scales"] = st["scale"].double()
        for which, rows in enumerate((k[live], v[live])):
            if c["cache"] == "e4m3":
                rows = rows / st["scale"][which]
            elif c["cache"] == "rows":
                s = rows.abs().amax(-1) / E4M3_MAX
                rows = rows / s[..., None]
                out["scales"][at // bs, at % bs // 16, :, which, at % 16] = s
            flat[which, at] = rows if c["cache"] == "bf16" else rows.clamp(-E4M3_MAX, E4M3_MAX)
        return out
    h, w = c["heads"], c["window"]
    group = h // hkv
    out, t0 = [], 0
    for r, (n, s) in enumerate(_lengths(c)):
        kv = _dense64(st, r, s)
        q = st["q"][t0:t0 + n].double()
        t0 += n
        o = torch.empty((n, h, d), dtype=torch.float64, device=DEV)
        for i0 in range(0, n, 1024):
            i1 = min(n, i0 + 1024)
            hi = s - n + i1
            lo = max(0, s - n + i0 - w + 1) if w > 0 else 0
            at = torch.arange(s - n + i0, hi, device=DEV)[:, None] - torch.arange(lo, hi, device=DEV)[None]
            hidden = (at < 0) | (at >= w) if w > 0 else at < 0
            for g in range(hkv):
                k, v = kv[0, lo:hi, g], kv[1, lo:hi, g]
                x = q[i0:i1, g * group:(g + 1) * group].transpose(0, 1) @ k.t() / math.sqrt(d)
                x = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
                o[i0:i1, g * group:(g + 1) * group] = (x @ v).transpose(0, 1)
        out.append(o)
    return torch.cat(out)
