"""Attention with keys and values from one shared latent vector a token.

A model of this kind caches, for each token, one latent vector and one rotary
key that all heads share.  A serving step takes four kinds of call:

  write      norms the step's latents, rotates the rotary parts of q and of the
             shared key, and writes latent and key as one row of the paged cache;
  read_back  gathers cached rows of many requests into dense latents and keys
             (what the up-projection of the expanded form takes);
  absorbed   attention of single tokens and chunks over the cached rows
             themselves: every head reads the row, its first part is the value;
  expanded   attention of prompts over keys and values that were projected up to
             a pair per head, with the shared rotary key beside them.

``own`` False computes them with elementary torch operations in fp32, rounded
once; ``own`` True calls this repository's package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
NORM_EPS = 1e-6
ROPE_BASE = 10000.0


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one new token of one request: latency
        dict(name="write_one_token", op="write", dtype="bf16", tokens=1, heads=16, latent=512,
             rope=64, adjacent=True, norm=True, dense=False, block_size=64, positions=32768),
        # all tokens of the mixed benchmark step (4 chunks of 2048 and 192 decodes)
        dict(name="write_mixed_step", op="write", dtype="bf16", tokens=8384, heads=64, latent=512,
             rope=64, adjacent=True, norm=True, dense=True, block_size=16, positions=32768),
        # a few short prefixes taken out of the cache
        dict(name="read_back_short", op="read_back", dtype="f16", seqs=4, lo=1, hi=90, latent=512,
             rope=64, block_size=16, lengths=11),
        # every key of the decode benchmark's batch, to project it up again
        dict(name="read_back_batch", op="read_back", dtype="bf16", seqs=64, lo=512, hi=4096,
             latent=512, rope=64, block_size=64, lengths=12),
        # the tiny batch: one prefill of 8 tokens beside one decode, a small latent
        dict(name="absorbed_tiny", op="absorbed", dtype="bf16", chunks=1, chunk_lo=8, chunk_hi=8,
             ctx_lo=0, ctx_hi=0, decodes=1, key_lo=40, key_hi=40, heads=4, latent=128, rope=32,
             block_size=16, lengths=21),
        # the decode benchmark's 64 requests on one share of a model's heads
        dict(name="absorbed_decode", op="absorbed", dtype="bf16", chunks=0, chunk_lo=0, chunk_hi=0,
             ctx_lo=0, ctx_hi=0, decodes=64, key_lo=512, key_hi=4096, heads=16, latent=512, rope=64,
             block_size=16, lengths=22),
        # the same requests with all heads of a large model
        dict(name="absorbed_decode_heads", op="absorbed", dtype="bf16", chunks=0, chunk_lo=0,
             chunk_hi=0, ctx_lo=0, ctx_hi=0, decodes=64, key_lo=512, key_hi=4096, heads=128,
             latent=512, rope=64, block_size=64, lengths=23),
        # few requests with long contexts: the keys are split over the GPU
        dict(name="absorbed_long", op="absorbed", dtype="f16", chunks=0, chunk_lo=0, chunk_hi=0,
             ctx_lo=0, ctx_hi=0, decodes=8, key_lo=120001, key_hi=131072, heads=32, latent=512,
             rope=64, block_size=64, lengths=24),
        # a step that checks several drafted tokens per request, beside a chunk of a prompt
        dict(name="absorbed_step", op="absorbed", dtype="bf16", chunks=24, chunk_lo=2, chunk_hi=40,
             ctx_lo=300, ctx_hi=6000, decodes=40, key_lo=200, key_hi=8192, heads=32, latent=512,
             rope=64, block_size=16, lengths=25),
        # short ragged prompts
        dict(name="expanded_short", op="expanded", dtype="bf16", chunks=6, chunk_lo=1, chunk_hi=130,
             ctx_lo=0, ctx_hi=50, heads=16, nope=128, rope=64, value=128, lengths=31),
        # ragged whole prompts
        dict(name="expanded_prompts", op="expanded", dtype="bf16", chunks=8, chunk_lo=1024,
             chunk_hi=8192, ctx_lo=0, ctx_hi=0, heads=32, nope=128, rope=64, value=128, lengths=32),
        # chunks of 2048 new tokens on 6144 keys that were read back
        dict(name="expanded_chunks", op="expanded", dtype="f16", chunks=4, chunk_lo=2048,
             chunk_hi=2048, ctx_lo=6144, ctx_hi=6144, heads=16, nope=128, rope=64, value=128,
             lengths=33),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read_back", "absorbed", "absorbed", "expanded", "expanded"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16"]))
    if op in ("write", "read_back", "absorbed"):
        case.update(latent=rng.choice([128, 256, 384, 512, 512, 512]),
                    rope=rng.choice([16, 32, 64, 64, 64]), block_size=rng.choice([16, 16, 32, 64, 128]))
    if op == "write":
        case.update(tokens=_log_int(rng, 1, 6000), heads=rng.choice([1, 4, 10, 16, 32, 40, 64, 128]),
                    adjacent=rng.random() < 0.5, norm=rng.random() < 0.7, dense=rng.random() < 0.4,
                    positions=_log_int(rng, 1000, 40000))
        case["tokens"] = min(case["tokens"], 8384 * 64 // case["heads"])
        return case
    if op == "read_back":
        lo = _log_int(rng, 1, 1500)
        case.update(seqs=_log_int(rng, 1, 64), lo=lo, hi=lo + _log_int(rng, 1, 2500),
                    lengths=rng.randrange(1 << 20))
        return case
    case.update(chunks=0, chunk_lo=0, chunk_hi=0, ctx_lo=0, ctx_hi=0, lengths=rng.randrange(1 << 20))
    if op == "expanded":
        lo = _log_int(rng, 1, 1500)
        ctx = rng.choice([0, _log_int(rng, 1, 4000)])
        nope = rng.choice([64, 128, 128])
        case.update(chunks=rng.randint(1, 5), chunk_lo=lo, chunk_hi=lo + _log_int(rng, 1, 1500),
                    ctx_lo=ctx // 2, ctx_hi=ctx, heads=rng.choice([1, 5, 8, 16, 20, 32]), nope=nope,
                    rope=rng.choice([16, 32, 64, 64]), value=nope)
        return case
    case.update(decodes=0, key_lo=0, key_hi=0, heads=rng.choice([1, 4, 10, 16, 20, 32, 40, 64, 128]))
    kind = rng.choice(["decode", "decode", "chunk", "both"])
    if kind != "decode":
        lo = _log_int(rng, 2, 60)
        ctx = rng.choice([0, _log_int(rng, 1, 3000)])
        case.update(chunks=rng.randint(1, 6), chunk_lo=lo, chunk_hi=lo + _log_int(rng, 1, 60),
                    ctx_lo=ctx // 2, ctx_hi=ctx)
    if kind != "chunk":
        lo = _log_int(rng, 1, 12000)
        case.update(decodes=_log_int(rng, 1, 64), key_lo=lo, key_hi=lo + _log_int(rng, 1, 6000))
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
    return out + [(1, r.randint(c["key_lo"], c["key_hi"])) for _ in range(c.get("decodes", 0))]


def work(c):
    if c["op"] == "write":
        t, h, row = c["tokens"], c["heads"], c["latent"] + c["rope"]
        data = t * (2 * 2 * h * c["rope"] + 2 * row * (3 if c["dense"] else 2) + 16)
        return {"bytes": data + 4 * c["rope"] * min(t, c["positions"]),
                "flops": t * (3 * (h + 1) * c["rope"] + (4 * c["latent"] if c["norm"] else 0))}
    lens = _lengths(c)
    keys, new = sum(s for _, s in lens), sum(q for q, _ in lens)
    pairs = sum(q * (s - q) + q * (q + 1) // 2 for q, s in lens)
    if c["op"] == "read_back":
        return {"bytes": keys * 4 * (c["latent"] + c["rope"]) + 4 * keys // c["block_size"], "flops": 0}
    h = c["heads"]
    if c["op"] == "absorbed":
        dc, dr = c["latent"], c["rope"]
        return {"bytes": 2 * keys * (dc + dr) + 4 * keys // c["block_size"] + 2 * new * h * (2 * dc + dr),
                "flops": 2 * h * (2 * dc + dr) * pairs}
    dk, dv, dr = c["nope"] + c["rope"], c["value"], c["rope"]
    return {"bytes": 2 * keys * (h * (c["nope"] + dv) + dr) + 2 * new * h * (dk + dv),
            "flops": 2 * h * (dk + dv) * pairs}


# ------------------------------------------------------------------ the inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _dtype(c):
    return torch.float16 if c["dtype"] == "f16" else torch.bfloat16


def _pool(g, blocks, c):
    """A filled cache [blocks, bs, latent + rope]: rows of uneven size, as tokens have."""
    out = torch.empty((blocks, c["block_size"], c["latent"] + c["rope"]), device=DEV, dtype=_dtype(c))
    for a in range(0, blocks, 4096):
        n = min(4096, blocks - a)
        out[a:a + n] = _randn(g, n, *out.shape[1:]) * torch.exp(0.3 * _randn(g, n, c["block_size"], 1))
    return out


def _tables(g, lens, bs):
    """A block table over a permuted pool, and the pool's size."""
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
    c, g = case, torch.Generator(device=DEV).manual_seed(seed)
    st = dict(case=c)
    dt = _dtype(c)
    if c["op"] == "write":
        t, h, dc, dr, bs = c["tokens"], c["heads"], c["latent"], c["rope"], c["block_size"]
        blocks = (t + bs - 1) // bs * 2 + 8
        # the rotary parts of q lie behind each head's other part, as the projection leaves them
        st["q"] = _randn(g, t, h, 2 * dr).to(dt)[..., dr:]
        st["q_out"] = torch.zeros((t, h, dr), dtype=dt, device=DEV)
        # latent and shared key side by side, from one projection
        st["down"] = _randn(g, t, dc + dr).mul_(torch.exp(0.3 * _randn(g, t, 1))).to(dt)
        st["norm"] = (1 + 0.1 * _randn(g, dc)).to(dt) if c["norm"] else None
        first = torch.randint(0, max(1, c["positions"] - t), (1,), generator=g, device=DEV)
        st["positions"] = (first + torch.arange(t, device=DEV)) % c["positions"]
        freq = ROPE_BASE ** (-torch.arange(dr // 2, device=DEV, dtype=torch.float64) * 2 / dr)
        angle = torch.arange(c["positions"], device=DEV, dtype=torch.float64)[:, None] * freq
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        slots = torch.randperm(blocks * bs, generator=g, device=DEV)[:t]
        slots[torch.rand(t, generator=g, device=DEV) < 0.01] = -1  # a few padding tokens
        st["slots"] = slots
        st["cache"] = _pool(g, blocks, c)
        st["dense"] = torch.zeros((t, dc + dr), dtype=dt, device=DEV) if c["dense"] else None
        return st
    lens = _lengths(c)
    st["max_q"], st["max_s"] = max(q for q, _ in lens), max(s for _, s in lens)
    if c["op"] == "expanded":
        keys, new, h = sum(s for _, s in lens), sum(q for q, _ in lens), c["heads"]
        st["q"] = _randn(g, new, h, c["nope"] + c["rope"]).to(dt)
        # keys and values of a head side by side, as one up-projection leaves them
        st["up"] = _randn(g, keys, h, c["nope"] + c["value"]).to(dt)
        st["k_rope"] = _randn(g, keys, c["rope"]).to(dt)
        st["starts"] = _starts([q for q, _ in lens])
        st["key_starts"] = _starts([s for _, s in lens])
        # requests that are served together: all where their scores take little room
        small = len(lens) * h * st["max_q"] * st["max_s"] < 1 << 28
        st["groups"] = [(0, len(lens), st["max_q"], st["max_s"])] if small else [
            (r, r + 1, q, s) for r, (q, s) in enumerate(lens)]
        return st
    st["table"], blocks = _tables(g, lens, c["block_size"])
    st["cache"] = _pool(g, blocks, c)
    if c["op"] == "read_back":
        st["starts"], st["rows"] = _starts([s for _, s in lens]), sum(s for _, s in lens)
        return st
    st["seq_lens"] = torch.tensor([s for _, s in lens], dtype=torch.int32, device=DEV)
    st["starts"] = _starts([q for q, _ in lens])
    st["q"] = _randn(g, sum(q for q, _ in lens), c["heads"], c["latent"] + c["rope"]).to(dt)
    # requests that are served together: the chunks, then the single tokens
    st["groups"] = [(a, b, max(q for q, _ in lens[a:b]), max(s for _, s in lens[a:b]))
                    for a, b in ((0, c["chunks"]), (c["chunks"], len(lens))) if b > a]
    return st


def _scale(c):
    # of the head size that the scores had before they were absorbed
    return 1.0 / math.sqrt(c["nope"] + c["rope"]) if c["op"] == "expanded" else 1.0 / math.sqrt(128 + c["rope"])


# ---------------------------------------------------------------- plain forms

def _turned(x, cos, sin, adjacent):
    if adjacent:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_write(st):
    c = st["case"]
    dc, bs, dt = c["latent"], c["block_size"], _dtype(c)
    cos, sin = st["cos_sin"][st["positions"]].chunk(2, -1)
    st["q_out"].copy_(_turned(st["q"].float(), cos[:, None], sin[:, None], c["adjacent"]))
    row = st["down"].float()
    latent, key = row[:, :dc], row[:, dc:]
    if c["norm"]:
        latent = latent * torch.rsqrt(latent.square().mean(-1, keepdim=True) + NORM_EPS) * st["norm"].float()
    row = torch.cat([latent, _turned(key, cos, sin, c["adjacent"])], -1).to(dt)
    keep = st["slots"] >= 0
    slot = st["slots"][keep]
    st["cache"][slot // bs, slot % bs] = row[keep]
    if c["dense"]:
        st["dense"].copy_(row)


def _plain_read_back(st):
    bs, dc = st["case"]["block_size"], st["case"]["latent"]
    row = torch.arange(st["rows"], device=DEV)
    req = torch.searchsorted(st["starts"], row, right=True) - 1
    key = row - st["starts"][req]
    rows = st["cache"][st["table"][req, key // bs].long(), key % bs]
    return [rows[:, :dc].contiguous(), rows[:, dc:].contiguous()]


def _softmax(x, hidden):
    x = x.masked_fill_(hidden, -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    return x.div_(x.sum(-1, keepdim=True))


def _plain_absorbed(st):
    c = st["case"]
    h, dc, bs = c["heads"], c["latent"], c["block_size"]
    out = torch.zeros((st["q"].shape[0], h, dc), dtype=_dtype(c), device=DEV)
    for a, b, most_q, most_s in st["groups"]:  # chunks and single tokens: two padded batches
        n = b - a
        first, s = st["starts"][a:b, None].long(), st["seq_lens"][a:b, None].long()
        count = st["starts"][a + 1:b + 1, None].long() - first
        i, key = torch.arange(most_q, device=DEV)[None], torch.arange(most_s, device=DEV)[None]
        live = i < count
        q = st["q"][torch.where(live, first + i, 0)].float().flatten(1, 2)
        rows = st["cache"][st["table"][a:b].long()[:, key[0] // bs], (key % bs).expand(n, -1)].float()
        rows = rows.masked_fill_((key >= s)[..., None], 0.0)
        hidden = key[:, None] > (s - count + i)[:, :, None]
        x = torch.bmm(q, rows.transpose(1, 2)).mul_(_scale(c)).view(n, most_q, h, most_s)
        x = _softmax(x, hidden[:, :, None])
        o = torch.bmm(x.view(n, most_q * h, most_s), rows[..., :dc]).view(n, most_q, h, dc)
        out[(first + i)[live]] = o[live].to(out.dtype)
        del x, rows
    return out


def _plain_expanded(st):
    c = st["case"]
    h, dn = c["heads"], c["nope"]
    out = torch.zeros((st["q"].shape[0], h, c["value"]), dtype=_dtype(c), device=DEV)
    for a, b, most_q, most_s in st["groups"]:  # one padded batch, or a large request at a time
        n = b - a
        first, at = st["starts"][a:b, None].long(), st["key_starts"][a:b, None].long()
        count, s = st["starts"][a + 1:b + 1, None].long() - first, st["key_starts"][a + 1:b + 1, None].long() - at
        i, key = torch.arange(most_q, device=DEV)[None], torch.arange(most_s, device=DEV)[None]
        live, there = i < count, key < s
        q = st["q"][torch.where(live, first + i, 0)].float().transpose(1, 2).flatten(0, 1)
        row = torch.where(there, at + key, 0)
        up = st["up"][row].float().masked_fill_(~there[..., None, None], 0.0).transpose(1, 2).flatten(0, 1)
        kr = st["k_rope"][row].float()
        x = torch.bmm(q[..., :dn], up[..., :dn].transpose(1, 2)).view(n, h * most_q, most_s)
        x = torch.baddbmm(x, q[..., dn:].reshape(n, h * most_q, -1), kr.transpose(1, 2)).mul_(_scale(c))
        hidden = key[:, None] > (s - count + i)[:, :, None]
        x = _softmax(x.view(n, h, most_q, most_s), hidden[:, None]).view(n * h, most_q, most_s)
        o = torch.bmm(x, up[..., dn:]).view(n, h, most_q, -1).transpose(1, 2)
        out[(first + i)[live]] = o[live].to(out.dtype)
        del x, up
    return out


# --------------------------------------------------------------------- a pass

def _written(st):
    out = {"q": st["q_out"], "cache": st["cache"]}
    if st["dense"] is not None:
        out["dense"] = st["dense"]
    return out


def run(state):
    st = state
    c = st["case"]
    if not own:
        if c["op"] == "write":
            _plain_write(st)
            return _written(st)
        return {"read_back": _plain_read_back, "absorbed": _plain_absorbed,
                "expanded": _plain_expanded}[c["op"]](st)
    import paged_varlen_attention_attn_gb300 as pa
    kind = pa.KV_F16 if c["dtype"] == "f16" else pa.KV_BF16
    if c["op"] == "write":
        latent, key = st["down"].split([c["latent"], c["rope"]], 1)
        pa.latent_rope_and_cache(st["q"], latent, key, st["cache"], st["slots"], st["positions"],
                                 st["cos_sin"], block_size=c["block_size"], kv_dtype=kind,
                                 interleaved=c["adjacent"], latent_norm=st["norm"],
                                 norm_eps=NORM_EPS, q_out=st["q_out"], row_out=st["dense"])
        return _written(st)
    if c["op"] == "read_back":
        return list(pa.gather_latent(st["cache"], st["table"], st["starts"], num_rows=st["rows"],
                                     latent_size=c["latent"], block_size=c["block_size"],
                                     kv_dtype=kind))
    if c["op"] == "absorbed":
        return pa.latent_forward(st["q"], st["cache"], st["table"], st["seq_lens"], st["starts"],
                                 scale=_scale(c), latent_size=c["latent"],
                                 block_size=c["block_size"], kv_dtype=kind,
                                 max_query_len=st["max_q"], max_seq_len=st["max_s"])
    k_nope, value = st["up"].split([c["nope"], c["value"]], 2)
    return pa.latent_expanded_forward(st["q"], k_nope, st["k_rope"], value, st["starts"],
                                      st["key_starts"], scale=_scale(c), kv_dtype=kind,
                                      max_query_len=st["max_q"], max_key_len=st["max_s"])


# ---------------------------------------------------------------- in 64 bits

def _attend64(q, k, v, scale, first):
    """Rows of q [n, d] at positions first .. over keys k [s, d], in 64 bits."""
    n, s = q.shape[0], k.shape[0]
    at = torch.arange(s, device=DEV)[None] - torch.arange(n, device=DEV)[:, None]
    return torch.softmax((q @ k.t() * scale).masked_fill(at > first, -math.inf), -1) @ v


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    if c["op"] == "write":
        t, dc, dr, bs = c["tokens"], c["latent"], c["rope"], c["block_size"]
        # each pair is a complex number that turns by its angle
        freq = ROPE_BASE ** (-torch.arange(dr // 2, device=DEV, dtype=torch.float64) * 2 / dr)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), st["positions"].double()[:, None] * freq)

        def spin(x, turn):
            y = torch.empty_like(x)
            first, second = (slice(0, dr, 2), slice(1, dr, 2)) if c["adjacent"] else (slice(0, dr // 2), slice(dr // 2, dr))
            z = torch.complex(x[..., first], x[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            return y

        row = st["down"].double()
        if c["norm"]:
            size = (row[:, :dc].pow(2).sum(-1, keepdim=True) / dc + NORM_EPS).sqrt()
            row[:, :dc] = row[:, :dc] / size * st["norm"].double()
        row[:, dc:] = spin(row[:, dc:].contiguous(), turn)
        cache = st["cache"].double()
        live = (st["slots"] >= 0).nonzero()[:, 0]
        cache.view(-1, dc + dr)[st["slots"][live]] = row[live]
        out = {"q": spin(st["q"].double().contiguous(), turn[:, None]), "cache": cache}
        if c["dense"]:
            out["dense"] = row
        return out
    scale = _scale(c)
    if c["op"] == "expanded":
        out = torch.empty((st["q"].shape[0], c["heads"], c["value"]), dtype=torch.float64, device=DEV)
        q0 = k0 = 0
        for n, s in _lengths(c):
            for h in range(c["heads"]):
                k = torch.cat([st["up"][k0:k0 + s, h, :c["nope"]], st["k_rope"][k0:k0 + s]], -1).double()
                v = st["up"][k0:k0 + s, h, c["nope"]:].double()
                for i in range(0, n, 2048):
                    m = min(2048, n - i)
                    seen = s - n + i + m
                    out[q0 + i:q0 + i + m, h] = _attend64(st["q"][q0 + i:q0 + i + m, h].double(), k[:seen],
                                                          v[:seen], scale, s - n + i)
            q0, k0 = q0 + n, k0 + s
        return out
    bs, dc = c["block_size"], c["latent"]
    dense = [st["cache"][st["table"][r, :(s + bs - 1) // bs].long()].flatten(0, 1)[:s].double()
             for r, (_, s) in enumerate(_lengths(c))]
    if c["op"] == "read_back":
        rows = torch.cat(dense)
        return [rows[:, :dc], rows[:, dc:]]
    out, q0 = [], 0
    for (n, s), rows in zip(_lengths(c), dense):
        for i in range(q0, q0 + n):
            seen = s - n + 1 + i - q0
            x = torch.softmax(st["q"][i].double() @ rows[:seen].t() * scale, -1)
            out.append(x @ rows[:seen, :dc])
        q0 += n
    return torch.stack(out)
