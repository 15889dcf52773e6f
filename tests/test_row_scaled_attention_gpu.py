"""Attention over a cache of e4m3 rows with a scale per (token, KV head)
(PATTN_KV_FP8_E4M3_ROW) against the definition in 64 bits.

Tolerance.  out = sum p v / sum p.  With A = sum p |v| / sum p: the weights are
rounded to f16 (2^-11), the prefill kernel's V rows are f16 products of a code
and a scale rounded to f16 (2^-11 each), so the sum is within 3 * 2^-11 A; the
scores are fp32 sums of exact products (and of a q whose entries below 2^-9 of
the row's largest lose under 2^-16 of it), which moves a weight by less than
2^-10: together under 1.5 * 2^-9 A.  Weights below f16's normal range are off by
2^-25 of the largest weight times its scale each: n 2^-25 B, with B the sum A
for rows of the largest code.  The output is rounded to bf16 (2^-8 of it).
"""
import numpy as np
import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
import row_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_varlen_attention_attn_gb300 import _build
    _build.build()
    pa.load()


class Case:
    def __init__(self, seed, reqs, H, Hkv, D, bs, spread=0.5, q_mul=1.0):
        g = torch.Generator().manual_seed(seed)
        self.H, self.Hkv, self.D, self.bs = H, Hkv, D, bs
        self.reqs = reqs
        need = [(s + bs - 1) // bs for _, s in reqs]
        self.NB = sum(need) + 2
        perm = torch.randperm(self.NB, generator=g).int()
        self.bt = torch.zeros((len(reqs), max(need)), dtype=torch.int32)
        at = 0
        for r, n in enumerate(need):
            self.bt[r, :n] = perm[at:at + n]
            at += n
        self.sl = torch.tensor([s for _, s in reqs], dtype=torch.int32)
        self.qsl = torch.tensor([0] + [q for q, _ in reqs], dtype=torch.int32).cumsum(0).int()
        self.T = int(self.qsl[-1])
        self.q = (torch.randn(self.T, H, D, generator=g) * q_mul).bfloat16()
        x = torch.randn(2, self.NB, bs, Hkv, D, generator=g)
        x = x * torch.exp2(spread * torch.randn(2, self.NB, bs, Hkv, 1, generator=g))
        codes, s = R.row_codes_fp32(x.bfloat16())
        self.cache = codes
        self.scales = torch.empty(pa.row_scales_shape(self.NB, bs, Hkv))
        for kv in range(2):
            self.scales[:, :, :, kv] = s[kv].view(self.NB, bs // 16, 16, Hkv).transpose(2, 3)
        self.scale = float(torch.tensor(D ** -0.5, dtype=torch.float32))

    def spread_scales(self, lo, hi, seed, which=(0, 1)):
        g = torch.Generator().manual_seed(seed)
        for kv in which:
            e = torch.randint(lo, hi + 1, self.scales[:, :, :, kv].shape, generator=g)
            self.scales[:, :, :, kv] = torch.exp2(e.float()) * (1 + torch.rand(e.shape, generator=g))

    def args(self):
        return (self.q.to(DEV), self.cache.to(DEV), self.bt.to(DEV), self.sl.to(DEV), self.qsl.to(DEV))

    def kw(self, **kw):
        base = dict(scale=self.scale, num_heads=self.H, num_kv_heads=self.Hkv, head_size=self.D,
                    block_size=self.bs, kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=self.scales.to(DEV),
                    max_query_len=max(q for q, _ in self.reqs), max_seq_len=max(s for _, s in self.reqs))
        base.update(kw)
        return base

    def run(self, expect=0, **kw):
        out = torch.full((self.T, self.H, self.D), float("nan"), dtype=torch.bfloat16, device=DEV)
        pa.forward(*self.args(), out=out, **self.kw(**kw))
        st = pa.pattn_read_device_status(pa.forward.last_ext)
        torch.cuda.synchronize()
        assert st == expect, pa.pattn_status_string(st)
        return out

    def reference(self, **kw):
        """(out, what it may be off by)"""
        kv = R.dense(self.cache, self.scales)
        a = (self.q,)
        b = (self.bt, self.sl, self.qsl)
        kw = dict(scale=self.scale, **kw)
        ref = R.attention(*a, kv, *b, **kw)
        A = R.attention(*a, torch.stack([kv[0], kv[1].abs()]), *b, **kw)
        s = self.scales.double().permute(3, 0, 1, 4, 2).reshape(2, self.NB, self.bs, self.Hkv)[1]
        B = R.attention(*a, torch.stack([kv[0], (448 * s)[..., None].expand_as(kv[1])]), *b, **kw)
        n = max(x for _, x in self.reqs)
        return ref, 2.0 ** -8 * np.abs(ref) + 1.5 * 2.0 ** -9 * A + n * 2.0 ** -25 * B

    def check(self, out, rows=slice(None), **kw):
        ref, tol = self.reference(**kw)
        got = R.f64(out).numpy()[rows]
        assert np.isfinite(got).all()
        bad = np.abs(got - ref[rows]) > tol[rows]
        assert not bad.any(), (int(bad.sum()), bad.size, np.abs(got - ref[rows]).max())


BATCHES = {
    "decode": [(1, 1), (1, 2), (1, 16), (1, 17), (1, 129), (1, 700)],
    "chunk": [(5, 5), (130, 300), (2, 2), (64, 257), (33, 401)],
    "mixed": [(1, 300), (70, 70), (0, 40), (1, 15), (129, 500), (1, 513), (2, 130)],
}


@pytest.mark.parametrize("batch", sorted(BATCHES))
@pytest.mark.parametrize("H,Hkv,D,bs,window", [
    (8, 2, 128, 16, 0), (6, 2, 64, 16, 0), (4, 4, 128, 64, 0), (16, 1, 128, 16, 90), (12, 4, 128, 128, 0),
    (8, 8, 64, 128, 0), (8, 2, 64, 32, 50), (6, 2, 128, 32, 130), (32, 8, 128, 16, 0), (5, 1, 128, 256, 7),
    (28, 4, 64, 16, 1)])
def test_batches(batch, H, Hkv, D, bs, window):
    c = Case(H + D + bs + window, BATCHES[batch], H, Hkv, D, bs)
    c.check(c.run(window=window), window=window)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("splits", [1, 3, 16])
def test_partitions(D, splits):
    c = Case(70 + D, [(1, 900), (1, 33), (1, 2000)], 8, 4, D, 16)
    c.check(c.run(num_splits=splits))


@pytest.mark.parametrize("window", [0, 300])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (32, 8)])
@pytest.mark.parametrize("most", [1, 63, 64, 145, 579, 1601, 4096])
def test_the_chosen_partition_count(most, H, Hkv, window):
    # from one partition over a few keys to fifteen, and what each merges to by force
    c = Case(75 + most + window, [(1, most), (1, max(1, most // 3)), (1, 1)], H, Hkv, 128, 16)
    out = c.run(window=window)
    c.check(out, window=window)
    visible = min(most, window) if window else most
    bound = max(1, int((visible / 16) ** 0.5) - 1)
    forced = c.run(window=window, num_splits=bound)
    assert torch.equal(out, forced)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("splits", [2, 5, 7, 33, 63, 64])
def test_merges_of_every_remainder(D, splits):
    c = Case(78 + D, [(1, 900), (1, 33), (1, 2000)], 8, 4, D, 16)
    c.check(c.run(num_splits=splits))


@pytest.mark.parametrize("D", [64, 128])
def test_sinks(D):
    c = Case(80 + D, BATCHES["mixed"], 8, 2, D, 16)
    sinks = torch.linspace(-3.0, 6.0, 8)
    sinks[2] = -float("inf")
    c.check(c.run(sinks=sinks.to(DEV)), sinks=sinks)
    c.check(c.run(sinks=sinks.to(DEV), num_splits=4), sinks=sinks)


@pytest.mark.parametrize("D", [64, 128])
def test_not_causal(D):
    c = Case(90 + D, BATCHES["mixed"], 8, 2, D, 16)
    c.check(c.run(causal=0), causal=0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("batch", ["decode", "chunk", "mixed"])
@pytest.mark.parametrize("lo,hi", [(-12, 12), (-30, 30), (-58, -50), (50, 58)])
def test_value_scales_far_apart(batch, D, lo, hi):
    c = Case(100 + D, BATCHES[batch], 8, 2, D, 16)
    c.spread_scales(lo, hi, 5, which=(1,))
    c.check(c.run())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("batch", ["decode", "mixed"])
def test_key_scales_far_apart(batch, D):
    # scores of very different sizes: from nothing to a few hundred
    c = Case(110 + D, BATCHES[batch], 8, 2, D, 16, q_mul=0.25)
    c.spread_scales(-30, -5, 6, which=(0,))
    c.check(c.run())


@pytest.mark.parametrize("D", [64, 128])
def test_a_dominant_key_with_a_tiny_value(D):
    """The first key takes nearly all the weight and has a value far smaller than
    the others', as an attention sink's: the others' small weights decide."""
    c = Case(120 + D, [(1, 600), (100, 600), (1, 40)], 8, 2, D, 16)
    c.q[:] = c.q.abs()
    for r in range(3):
        b = int(c.bt[r, 0])
        c.cache[0, b, 0] = 0x70           # a key along every q, 128 per element
        c.scales[b, 0, :, 0, 0] = 0.012
        c.scales[b, 0, :, 1, 0] = 1e-9
    c.check(c.run())


def test_nothing_past_the_end_or_below_the_window_is_used():
    for window in (0, 37):
        c = Case(130, BATCHES["mixed"], 8, 2, 128, 16)
        ref, tol = c.reference(window=window)
        used = torch.zeros(c.NB * 16, dtype=torch.bool)
        for r, (q, s) in enumerate(c.reqs):
            if q == 0:
                continue
            lo = max(0, s - q - window + 1) if window else 0
            key = torch.arange(lo, s)
            used[c.bt[r][key // 16].long() * 16 + key % 16] = True
        flat = c.cache.view(2, -1, 2, 128)
        flat[:, ~used] = 0x7F  # NaN
        g = torch.Generator().manual_seed(1)
        junk = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -1.0, 3e38])
        s = c.scales.permute(0, 1, 4, 2, 3).reshape(-1, 2, 2).clone()
        s[~used] = junk[torch.randint(0, 6, (int((~used).sum()), 2, 2), generator=g)]
        c.scales = s.view(c.NB, 1, 16, 2, 2).permute(0, 1, 3, 4, 2).contiguous()
        got = R.f64(c.run(window=window)).numpy()
        assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("D", [64, 128])
def test_q_rows_of_very_different_magnitudes(D):
    c = Case(140 + D, BATCHES["mixed"], 8, 2, D, 16)
    g = torch.Generator().manual_seed(2)
    e = torch.randint(-40, 4, (c.T, 8, 1), generator=g).float()
    c.q = (c.q.float() * torch.exp2(e)).bfloat16()
    c.check(c.run())


def test_nan_codes_reach_the_rows_that_see_them():
    c = Case(150, [(1, 64), (1, 70)], 4, 2, 128, 16)
    b = int(c.bt[0, 1])
    c.cache[1, b, 3, 1, 5] = 0x7F
    out = R.f64(c.run())
    assert torch.isnan(out[0, 2:, 5]).all() and not torch.isnan(out[1]).any()
    assert not torch.isnan(out[0, :2]).any()


@pytest.mark.parametrize("batch", ["decode", "mixed"])
def test_bad_blocks_are_reported_and_stay_in_bounds(batch):
    c = Case(160, BATCHES[batch], 8, 2, 128, 16)
    bad = 5
    c.bt[bad, 3] = c.NB + 1000
    out = c.run(expect=5)
    a, b = int(c.qsl[bad]), int(c.qsl[bad + 1])
    assert torch.isfinite(out[a:b].float()).all()
    rows = np.r_[0:a, b:c.T]
    c.bt[bad, 3] = 0
    c.check(out, rows=rows)


@pytest.mark.parametrize("reqs", [[(1, 200), (1, 500), (1, 333)], [(40, 200), (1, 300), (130, 400)]])
def test_cascade(reqs):
    c = Case(170, reqs, 8, 2, 128, 16)
    c.bt[1:, :6] = c.bt[0, :6]
    out = pa.cascade_forward(*c.args(), common_prefix_len=96, **c.kw())
    assert pa.pattn_read_device_status(pa.forward.last_ext) == 0
    c.check(out)


def test_the_workspace_free_decode():
    c = Case(180, BATCHES["mixed"], 8, 2, 128, 16)
    q, cache, bt, sl, qsl = c.args()
    scales = c.scales.to(DEV)
    out = torch.full((c.T, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    st = pa.pattn_decode_fwd_static(
        q.data_ptr(), cache.data_ptr(), bt.data_ptr(), sl.data_ptr(), qsl.data_ptr(), out.data_ptr(),
        c.scale, 8, 2, 128, 16, 0, 1, pa.KV_FP8_E4M3_ROW, scales, len(c.reqs), c.T, bt.shape[1], c.NB,
        600, 0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0
    rows = np.array([int(c.qsl[r]) for r, (n, _) in enumerate(c.reqs) if n == 1])
    c.check(out, rows=rows)
    rest = np.setdiff1d(np.arange(c.T), rows)
    assert (out[rest] == 7.0).all()


def test_captured_and_replayed_on_another_stream():
    a, b = (Case(s, BATCHES["mixed"], 8, 2, 128, 16) for s in (190, 191))
    bufs = [x.clone() for x in a.args()]
    scales = a.scales.to(DEV)
    out = torch.empty(a.T, 8, 128, dtype=torch.bfloat16, device=DEV)
    kw = a.kw(kv_scale=scales, workspace=pa.Workspace(), out=out)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        pa.forward(*bufs, **kw)
    torch.cuda.synchronize()
    a.check(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pa.forward(*bufs, **kw)
    for c in (b, a):
        for x, y in zip(bufs, c.args()):
            x.copy_(y)
        scales.copy_(c.scales)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        c.check(out)


def test_row_scales_all_equal_match_the_tensor_scaled_cache():
    c = Case(200, BATCHES["mixed"], 8, 2, 128, 16)
    c.scales[:, :, :, 0] = 0.0078125
    c.scales[:, :, :, 1] = 0.03125
    rows = c.run()
    tensor = c.run(kv_dtype=pa.KV_FP8_E4M3, kv_scale=(0.0078125, 0.03125))
    c.check(rows)
    c.check(tensor)


def test_write_attend_and_read_back_over_steps():
    """What a serving loop does: a prompt chunk, then single tokens, each step
    rotated and written by rope_and_cache and attended; at the end the cache is
    read back.  The reference follows the cache's own contents."""
    H, Hkv, D, bs, NB = 8, 2, 128, 16, 24
    g = torch.Generator().manual_seed(210)
    table, _ = R.cos_sin_table(512, D)
    cache = torch.full((2, NB, bs, Hkv, D), 0x7F, dtype=torch.uint8, device=DEV)
    scales = torch.full(pa.row_scales_shape(NB, bs, Hkv), float("nan"), device=DEV)
    bt = torch.randperm(NB, generator=g).int()[:20].view(2, 10)
    lens = [0, 0]
    for step, news in enumerate([(70, 33), (1, 40), (1, 1), (20, 1), (1, 1)]):
        T = sum(news)
        pos = torch.cat([torch.arange(n) + s for n, s in zip(news, lens)])
        req = torch.tensor([0] * news[0] + [1] * news[1])
        slots = bt[req, pos // bs].long() * bs + pos % bs
        qkv = torch.randn(T, (H + 2 * Hkv) * D, generator=g).bfloat16()
        q, k, v = qkv.to(DEV).view(T, -1, D).split([H, Hkv, Hkv], 1)
        qr = pa.rope_and_cache(q, k, v, cache, slots.to(DEV), pos.to(DEV), table.to(DEV),
                               block_size=bs, kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=scales)
        lens = [s + n for n, s in zip(news, lens)]
        c = Case.__new__(Case)
        c.H, c.Hkv, c.D, c.bs, c.NB, c.T = H, Hkv, D, bs, NB, T
        c.reqs = list(zip(news, lens))
        c.q, c.cache, c.scales, c.bt = qr.cpu(), cache.cpu(), scales.cpu(), bt
        c.sl = torch.tensor(lens, dtype=torch.int32)
        c.qsl = torch.tensor([0, news[0], T], dtype=torch.int32)
        c.scale = float(torch.tensor(D ** -0.5, dtype=torch.float32))
        c.check(c.run())
        at = R.f64(R.f64(q.cpu()).float())
        ref = R.rotate(at, table, pos)
        assert ((R.f64(qr) - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -17 * ref.abs().amax(-1, keepdim=True)).all()
    osl = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32)
    ko, vo = pa.gather_cache(cache, bt.to(DEV), osl.to(DEV), num_rows=sum(lens), block_size=bs,
                             kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=scales)
    kv = R.dense(cache, scales)
    for r in range(2):
        key = torch.arange(lens[r])
        for got, x in ((ko, kv[0]), (vo, kv[1])):
            ref = x[bt[r, key // bs].long(), key % bs]
            d = (R.f64(got[int(osl[r]):int(osl[r + 1])]) - ref).abs()
            assert (d <= (2.0 ** -8 + 2.0 ** -23) * ref.abs()).all()


def test_a_cache_past_32_bit_offsets():
    """Blocks at the end of a pool of 2.6e9 code elements: written, attended and
    read back like any other."""
    H, Hkv, D, bs = 8, 8, 128, 64
    NB = 20000
    cache = torch.empty(2, NB, bs, Hkv, D, dtype=torch.uint8, device=DEV)
    scales = torch.empty(pa.row_scales_shape(NB, bs, Hkv), device=DEV)
    small = Case(220, [(1, 200), (90, 90)], H, Hkv, D, bs)
    where = torch.arange(NB - small.NB, NB)
    cache[:, where] = small.cache.to(DEV)
    scales[where] = small.scales.to(DEV)
    q, _, bt, sl, qsl = small.args()
    out = pa.forward(q, cache, bt + NB - small.NB, sl, qsl, **small.kw(kv_scale=scales))
    ko, vo = pa.gather_cache(cache, bt + NB - small.NB, torch.tensor([0, 200, 290], dtype=torch.int32, device=DEV),
                             num_rows=290, block_size=bs, kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=scales)
    want = pa.gather_cache(small.cache.to(DEV), bt, torch.tensor([0, 200, 290], dtype=torch.int32, device=DEV),
                           num_rows=290, block_size=bs, kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=small.scales.to(DEV))
    torch.cuda.synchronize()
    small.check(out)
    assert torch.equal(ko, want[0]) and torch.equal(vo, want[1])
    k = torch.randn(3, Hkv, D, device=DEV).bfloat16()
    slots = torch.tensor([NB * bs - 1, (NB - 1) * bs, 0], device=DEV)
    pa.reshape_and_cache(k, k, cache, slots, block_size=bs, kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=scales)
    torch.cuda.synchronize()
    codes, s = R.row_codes_fp32(k)
    for i, at in enumerate(slots.tolist()):
        assert torch.equal(cache[0, at // bs, at % bs].cpu(), codes[i])
        assert torch.equal(cache[1, at // bs, at % bs].cpu(), codes[i])
        assert torch.equal(scales[at // bs, at % bs // 16, :, 1, at % 16].cpu(), s[i])


def test_decode_over_blocks_that_are_no_power_of_two():
    c = Case(230, [(1, 5), (1, 48), (1, 49), (1, 700)], 8, 2, 128, 48)
    c.check(c.run())
    c.check(c.run(window=60), window=60)


def test_calls_on_two_streams_at_once_do_not_share_scratch():
    """Default workspaces: two streams' calls, each with partitions, interleaved."""
    a = Case(240, [(1, 3000), (1, 2500)], 8, 2, 128, 16)
    b = Case(241, [(1, 2800), (40, 300), (1, 900)], 8, 2, 128, 16)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    prepared = [(c.args(), c.kw(num_splits=8)) for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(pa.forward(*prepared[i][0], **prepared[i][1]))
    torch.cuda.synchronize()
    for c, got in zip((a, b), outs):
        c.check(got[0])
        assert all(torch.equal(x, got[0]) for x in got)


def test_repeated_calls_give_the_same_bits():
    c = Case(250, BATCHES["mixed"] + [(1, 4000)], 8, 2, 128, 16)
    prepared, kw = c.args(), c.kw(num_splits=6)
    first = pa.forward(*prepared, **kw)
    for _ in range(5):
        assert torch.equal(pa.forward(*prepared, **kw), first)


def test_rows_outside_the_batch_stay():
    """A padded batch: q and out have rows before and behind the requests'."""
    c = Case(260, BATCHES["mixed"], 8, 2, 128, 16)
    q, cache, bt, sl, qsl = c.args()
    wide = torch.full((c.T + 9, 8, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[4:4 + c.T] = q
    out = torch.full_like(wide, 7.0)
    pa.forward(wide, cache, bt, sl, qsl + 4, out=out, **c.kw())
    torch.cuda.synchronize()
    c.check(out[4:4 + c.T])
    assert (out[:4] == 7.0).all() and (out[4 + c.T:] == 7.0).all()
