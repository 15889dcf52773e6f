"""pattn_rope_and_cache and pattn_reshape_and_cache_rows against plain
definitions in 64 bits.

Tolerances.  The kernel rounds once: a 16-bit output is within half a step,
eps / 2 of the value (bf16 2^-8, f16 2^-11).  Before that it computes in fp32:
a rotated element is a c - b s with three roundings of terms no larger than
|a| + |b| <= sqrt(2) row norms of the pair, and the norm adds the error of a sum
of d <= 256 squares, a reciprocal square root (2^-22) and two products: together
under 2^-18 of the row's largest pair, which is at most sqrt(2) of the rotated
row's largest magnitude: 2^-17 of that magnitude is allowed.  An e4m3 code is
within half a step: 2^-4 of the value, or 2^-10 of the scale among subnormals.
"""
import pytest
import torch

import oracle
import paged_varlen_attention_attn_gb300 as pa
import row_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_varlen_attention_attn_gb300 import _build
    _build.build()
    pa.load()


def make(seed, T, H, Hkv, D, rot, bs, *, kind, axes=1, norm=False, max_pos=4096, pad=True):
    g = torch.Generator().manual_seed(seed)
    dt = torch.float16 if kind == pa.KV_F16 else torch.bfloat16
    c = dict(kind=kind, T=T, H=H, Hkv=Hkv, D=D, rot=rot, bs=bs, NB=(T + bs - 1) // bs + 3)
    c["qkv"] = (torch.randn(T, (H + 2 * Hkv) * D, generator=g) * 2).to(dt).to(DEV)
    c["table"], _ = R.cos_sin_table(max_pos, rot)
    c["pos"] = torch.randint(0, max_pos, (axes, T) if axes > 1 else (T,), generator=g)
    c["slots"] = torch.randperm(c["NB"] * bs, generator=g)[:T]
    if pad:
        c["slots"][2::7] = -1
    c["qn"] = (1 + 0.3 * torch.randn(D, generator=g)).to(dt).to(DEV) if norm else None
    c["kn"] = (1 + 0.3 * torch.randn(D, generator=g)).to(dt).to(DEV) if norm else None
    shape = (2, c["NB"], bs, Hkv, D)
    if kind in (pa.KV_FP8_E4M3, pa.KV_FP8_E4M3_ROW):
        c["cache"] = torch.randint(0, 127, shape, generator=g, dtype=torch.uint8).to(DEV)
    else:
        c["cache"] = torch.randn(shape, generator=g).to(dt).to(DEV)
    c["scale"] = {pa.KV_FP8_E4M3: (0.03, 0.02)}.get(kind)
    if kind == pa.KV_FP8_E4M3_ROW:
        c["scale"] = torch.rand(pa.row_scales_shape(c["NB"], bs, Hkv), generator=g).to(DEV)
    return c


def parts(c):
    return c["qkv"].view(c["T"], c["H"] + 2 * c["Hkv"], c["D"]).split([c["H"], c["Hkv"], c["Hkv"]], 1)


def call(c, *, axis=None, interleaved=False, q_out=None, status=None, **kw):
    q, k, v = parts(c)
    return pa.rope_and_cache(q, k, v, c["cache"], c["slots"].to(DEV), c["pos"].to(DEV),
                             c["table"].to(DEV), block_size=c["bs"], kv_dtype=c["kind"],
                             kv_scale=c["scale"], interleaved=interleaved, pair_axis=axis,
                             q_norm=c["qn"], k_norm=c["kn"], norm_eps=1e-5, q_out=q_out,
                             device_status=status, **kw)


def near16(got, ref, dt):
    rowmax = ref.abs().amax(-1, keepdim=True)
    tol = torch.finfo(dt).eps / 2 * ref.abs() + 2.0 ** -17 * rowmax
    bad = (R.f64(got) - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), (R.f64(got) - ref).abs().max())


def near_codes(codes, scale, ref):
    """codes float64 code values [..., d], scale [..., 1], ref the unrounded rows."""
    rowmax = ref.abs().amax(-1, keepdim=True)
    half = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * scale)
    over = (ref.abs() - E4M3_MAX_OF(scale)).clamp_min(0)  # saturated values
    bad = (codes * scale - ref).abs() > half * (1 + 2.0 ** -12) + 2.0 ** -17 * rowmax + over
    assert not bad.any(), int(bad.sum())


def E4M3_MAX_OF(scale):
    return R.E4M3_MAX * scale


def check(c, before, q_out, axis=None, interleaved=False):
    q, k, v = (R.f64(x) for x in parts(c))
    kw = dict(interleaved=interleaved, pair_axis=axis, eps=1e-5)
    dt = c["qkv"].dtype
    near16(q_out, R.rotate(q, c["table"], c["pos"], weight=c["qn"], **kw), dt)
    k = R.rotate(k, c["table"], c["pos"], weight=c["kn"], **kw)
    live = c["slots"] >= 0
    at = c["slots"][live]
    got = c["cache"].cpu()
    flat = got.reshape(2, -1, c["Hkv"], c["D"])
    old = before.cpu().reshape(flat.shape)
    rest = torch.ones(flat.shape[1], dtype=torch.bool)
    rest[at] = False
    assert torch.equal(flat[:, rest].view(torch.uint8), old[:, rest].view(torch.uint8))
    for kv, ref in ((0, k[live]), (1, v[live])):
        rows = R.f64(flat[kv, at])
        if c["kind"] in (pa.KV_BF16, pa.KV_F16):
            near16(flat[kv, at], ref, dt)
        elif c["kind"] == pa.KV_FP8_E4M3:
            near_codes(rows, torch.full((1,), float(torch.tensor(c["scale"][kv]))).double(), ref)
        else:
            s = R.scales_at(c["scale"], at)[:, :, kv]
            want = R.row_scale(ref)
            assert ((s - want).abs() <= 2.0 ** -17 * want).all()
            near_codes(rows, s[..., None], ref)


@pytest.mark.parametrize("kind", [pa.KV_BF16, pa.KV_FP8_E4M3, pa.KV_F16, pa.KV_FP8_E4M3_ROW])
@pytest.mark.parametrize("T,H,Hkv,D,rot,bs,axes,norm,interleaved", [
    (1, 8, 2, 128, 128, 16, 1, False, False),
    (37, 6, 2, 64, 64, 16, 1, True, True),
    (130, 32, 8, 128, 128, 64, 3, True, False),
    (61, 7, 7, 96, 48, 32, 1, False, False),
    (19, 4, 1, 256, 64, 16, 2, False, True),
    (301, 3, 1, 80, 80, 16, 4, True, False),
    (5, 2, 2, 16, 16, 16, 1, False, True),
    (2050, 16, 2, 128, 64, 128, 1, False, True),
    # many tokens, short rows
    (1300, 6, 2, 64, 64, 16, 1, True, True),
    (3001, 7, 7, 96, 48, 32, 1, False, False),
    # long calls of long rows: the streaming kernel
    (2400, 32, 8, 128, 128, 64, 3, True, False),
    (3333, 64, 4, 64, 64, 16, 1, True, True),
    (2500, 16, 4, 256, 64, 16, 2, False, True),
    (3100, 48, 8, 80, 80, 16, 4, True, False),
    (4001, 31, 3, 96, 48, 32, 1, False, False),
    (1500, 64, 8, 128, 64, 16, 1, False, False),
    (1000, 128, 8, 128, 128, 16, 1, False, False),   # three stages do not fit: one warp per step
])
def test_matches_the_definition(kind, T, H, Hkv, D, rot, bs, axes, norm, interleaved):
    c = make(7 * T + D + rot + kind, T, H, Hkv, D, rot, bs, kind=kind, axes=axes, norm=norm)
    axis = None
    if axes > 1:  # a mix whose groups of four pairs do not share an axis
        g = torch.Generator().manual_seed(T)
        axis = torch.randint(0, axes, (rot // 2,), generator=g).tolist()
    before = c["cache"].clone()
    scales = c["scale"].clone() if kind == pa.KV_FP8_E4M3_ROW else None
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = call(c, axis=axis, interleaved=interleaved, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    check(c, before, out, axis, interleaved)
    if scales is not None:  # the scales of slots that were not written stay
        flat = lambda s: s.cpu().permute(0, 1, 4, 2, 3).reshape(-1, Hkv, 2)
        rest = torch.ones(c["NB"] * bs, dtype=torch.bool)
        rest[c["slots"][c["slots"] >= 0]] = False
        assert torch.equal(flat(c["scale"])[rest], flat(scales)[rest])


def test_sections_in_order_and_in_turns():
    for inter in (False, True):
        c = make(400 + inter, 77, 8, 2, 128, 128, 16, kind=pa.KV_FP8_E4M3_ROW, axes=3)
        axis = pa.rope_pair_axis((24, 20, 20), interleaved=inter)
        before = c["cache"].clone()
        out = call(c, axis=axis)
        torch.cuda.synchronize()
        check(c, before, out, axis)


def test_in_place_and_strided_q():
    c = make(410, 53, 8, 2, 128, 128, 16, kind=pa.KV_FP8_E4M3_ROW)
    ref = call(c)
    d = make(410, 53, 8, 2, 128, 128, 16, kind=pa.KV_FP8_E4M3_ROW)
    q = parts(d)[0]
    kept = d["qkv"][:, 8 * 128:].clone()
    got = call(d, q_out=q)
    torch.cuda.synchronize()
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, ref)
    assert torch.equal(d["qkv"][:, 8 * 128:], kept)
    assert torch.equal(c["cache"], d["cache"]) and torch.equal(c["scale"], d["scale"])


def test_q_alone_and_keys_alone():
    c = make(420, 40, 8, 2, 128, 128, 16, kind=pa.KV_FP8_E4M3_ROW)
    ref = call(c)
    d = make(420, 40, 8, 2, 128, 128, 16, kind=pa.KV_FP8_E4M3_ROW)
    q, k, v = parts(d)
    rest = (d["slots"].to(DEV), d["pos"].to(DEV), d["table"].to(DEV))
    kw = dict(block_size=16, kv_dtype=d["kind"])
    only_q = pa.rope_and_cache(q, None, None, None, None, *rest[1:], **kw)
    assert pa.rope_and_cache(None, k, v, d["cache"], *rest, kv_scale=d["scale"], **kw) is None
    torch.cuda.synchronize()
    assert torch.equal(only_q, ref)
    assert torch.equal(c["cache"], d["cache"]) and torch.equal(c["scale"], d["scale"])


def test_padding_and_positions_outside_the_table():
    c = make(430, 30, 8, 2, 64, 64, 16, kind=pa.KV_FP8_E4M3_ROW, axes=3, max_pos=100, pad=False)
    axis = pa.rope_pair_axis((8, 12, 12))
    c["pos"][0, 4] = -1       # padding: silent
    c["pos"][2, 4] = 1 << 40
    before, scales = c["cache"].clone(), c["scale"].clone()
    marked = torch.full((30, 8, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = call(c, axis=axis, q_out=marked, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0 and (out[4] == 7.0).all()
    at = int(c["slots"][4])
    assert torch.equal(c["cache"][:, at // 16, at % 16], before[:, at // 16, at % 16])
    for bad in (100, 1 << 40, (1 << 63) - 1):  # reported, nothing of the token written
        c["pos"][1, 9] = bad
        c["cache"].copy_(before)
        c["scale"].copy_(scales)
        marked.fill_(7.0)
        status.zero_()
        call(c, axis=axis, q_out=marked, status=status)
        torch.cuda.synchronize()
        at = int(c["slots"][9])
        assert int(status) == 1 and (marked[9] == 7.0).all() and not (marked[8] == 7.0).all()
        assert torch.equal(c["cache"][:, at // 16, at % 16], before[:, at // 16, at % 16])


def test_slot_past_the_pool_is_reported_and_its_q_is_rotated():
    c = make(440, 30, 4, 2, 64, 64, 16, kind=pa.KV_FP8_E4M3_ROW, pad=False)
    ok = make(440, 30, 4, 2, 64, 64, 16, kind=pa.KV_FP8_E4M3_ROW, pad=False)
    ok["slots"][11] = -1
    c["slots"][11] = c["NB"] * 16
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, ref = call(c, status=status), call(ok)
    torch.cuda.synchronize()
    assert int(status) == 1 and torch.equal(out, ref)
    assert torch.equal(c["cache"], ok["cache"]) and torch.equal(c["scale"], ok["scale"])


@pytest.mark.parametrize("T,Hkv,D,bs", [(1, 1, 16, 16), (77, 4, 128, 16), (400, 8, 64, 64),
                                        (33, 3, 256, 32), (50, 2, 112, 16)])
def test_rows_are_quantised_bit_for_bit(T, Hkv, D, bs):
    g = torch.Generator().manual_seed(500 + T)
    x = torch.randn(2, T, Hkv, D, generator=g) * torch.exp2(
        torch.randint(-40, 40, (2, T, Hkv, 1), generator=g).float())
    x[0, 0, 0] = 0.0
    if T > 4:
        x[0, 1, 0, 3], x[1, 2, 0, 5], x[0, 3, 0, 1] = float("nan"), float("inf"), -float("inf")
        x[1, 4, 0] = float("nan")
        x[0, 4, 0] = 1e-38
        x[0, 5, 0] = 3e38
    x = x.bfloat16()
    nb = (T + bs - 1) // bs + 2
    slots = torch.randperm(nb * bs, generator=g)[:T]
    if T > 1:
        slots[1::9] = -1
    cache = torch.zeros(2, nb, bs, Hkv, D, dtype=torch.uint8, device=DEV)
    scales = torch.full(pa.row_scales_shape(nb, bs, Hkv), -1.0, device=DEV)
    pa.reshape_and_cache(x[0].to(DEV), x[1].to(DEV), cache, slots.to(DEV), block_size=bs,
                         kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=scales)
    torch.cuda.synchronize()
    codes, s = R.row_codes_fp32(x)
    live = slots >= 0
    flat = cache.cpu().reshape(2, -1, Hkv, D)
    assert torch.equal(flat[:, slots[live]], codes[:, live])
    assert torch.equal(R.scales_at(scales, slots[live]).permute(2, 0, 1), s[:, live].double())
    rest = torch.ones(nb * bs, dtype=torch.bool)
    rest[slots[live]] = False
    assert (flat[:, rest] == 0).all()
    every = scales.cpu().permute(0, 1, 4, 2, 3).reshape(-1, Hkv, 2)
    assert (every[rest] == -1).all()


@pytest.mark.parametrize("T,H", [(40, 8), (1300, 8), (3400, 64)])
def test_skipped_tokens_of_every_sort(T, H):
    """Padding, bad positions, negative slots and slots past the pool scattered
    over a batch: the others are as if those were not there."""
    kind = pa.KV_FP8_E4M3_ROW
    make_it = lambda: make(600 + T, T, H, 2, 64, 64, 16, kind=kind, axes=3, max_pos=300, pad=False)
    c, ok = make_it(), make_it()
    axis = pa.rope_pair_axis((8, 12, 12))
    for i in range(0, T, 10):
        c["pos"][0, i] = -7
        c["pos"][2, i + 1] = 300
        c["slots"][i + 2] = -9
        c["slots"][i + 3] = c["NB"] * 16 + i
        c["pos"][1, i + 4] = -1
    ref = call(ok, axis=axis)
    marked = torch.full((T, H, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    before, scales = c["cache"].clone(), c["scale"].clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = call(c, axis=axis, q_out=marked, status=status)
    torch.cuda.synchronize()
    assert int(status) == 1
    i = torch.arange(T) % 10
    gone, kv_gone = (i == 0) | (i == 1) | (i == 4), (i < 5)
    assert (out[gone.to(DEV)] == 7.0).all() and torch.equal(out[~gone.to(DEV)], ref[~gone.to(DEV)])
    flat = lambda x: x.reshape(2, -1, 2, 64)
    flat_s = lambda x: x.permute(0, 1, 4, 2, 3).reshape(-1, 2, 2)
    at = ok["slots"].to(DEV)
    live, dead = at[~kv_gone.to(DEV)], at[kv_gone.to(DEV)]
    assert torch.equal(flat(c["cache"])[:, live], flat(ok["cache"])[:, live])
    assert torch.equal(flat_s(c["scale"])[live], flat_s(ok["scale"])[live])
    assert torch.equal(flat(c["cache"])[:, dead], flat(before)[:, dead])
    assert torch.equal(flat_s(c["scale"])[dead], flat_s(scales)[dead])


@pytest.mark.parametrize("T,H,Hkv", [(1999, 8, 2), (2999, 40, 16)])
def test_many_tokens_in_place_alone_and_without_rotation(T, H, Hkv):
    kind = pa.KV_FP8_E4M3_ROW
    c, d, e = (make(620, T, H, Hkv, 128, 128, 16, kind=kind) for _ in range(3))
    ref = call(c)
    rest = (d["slots"].to(DEV), d["pos"].to(DEV), d["table"].to(DEV))
    q, k, v = parts(d)
    kw = dict(block_size=16, kv_dtype=kind)
    pa.rope_and_cache(None, k, v, d["cache"], *rest, kv_scale=d["scale"], **kw)
    pa.rope_and_cache(q, None, None, None, None, *rest[1:], q_out=q, **kw)
    torch.cuda.synchronize()
    assert torch.equal(q, ref)
    assert torch.equal(c["cache"], d["cache"]) and torch.equal(c["scale"], d["scale"])
    q, k, v = parts(e)
    pa.reshape_and_cache(k.contiguous(), v.contiguous(), e["cache"], rest[0], block_size=16,
                         kv_dtype=kind, kv_scale=e["scale"])
    torch.cuda.synchronize()
    codes, s = R.row_codes_fp32(torch.stack([k, v]))
    live = e["slots"] >= 0
    at = e["slots"][live]
    assert torch.equal(e["cache"].cpu().reshape(2, -1, Hkv, 128)[:, at], codes[:, live])
    assert torch.equal(R.scales_at(e["scale"], at).permute(2, 0, 1), s[:, live].double())


def test_the_tensor_scaled_write_without_rotation_is_the_plain_write():
    c = make(520, 90, 4, 4, 128, 128, 16, kind=pa.KV_FP8_E4M3)
    _, k, v = parts(c)
    other = c["cache"].clone()
    pa.rope_and_cache(None, k, v, c["cache"], c["slots"].to(DEV), None, None, block_size=16,
                      kv_dtype=pa.KV_FP8_E4M3, kv_scale=c["scale"])
    pa.reshape_and_cache(k.contiguous(), v.contiguous(), other, c["slots"].to(DEV), block_size=16,
                         kv_dtype=pa.KV_FP8_E4M3, kv_scale=c["scale"])
    torch.cuda.synchronize()
    assert torch.equal(c["cache"], other)


def test_no_tokens_and_a_captured_call():
    c = make(530, 64, 8, 2, 128, 128, 16, kind=pa.KV_FP8_E4M3_ROW)
    q, k, v = parts(c)
    e = lambda x: x[:0]
    pos, slots, table = c["pos"].to(DEV), c["slots"].to(DEV), c["table"].to(DEV)
    out = pa.rope_and_cache(e(q), e(k), e(v), c["cache"], e(slots), e(pos), table, block_size=16,
                            kv_dtype=c["kind"], kv_scale=c["scale"])
    assert out.shape == (0, 8, 128)
    q_out = torch.zeros(64, 8, 128, dtype=torch.bfloat16, device=DEV)

    def step():
        pa.rope_and_cache(q, k, v, c["cache"], slots, pos, table, block_size=16,
                          kv_dtype=c["kind"], kv_scale=c["scale"], q_out=q_out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (531, 532):  # new contents in the captured buffers
        d = make(seed, 64, 8, 2, 128, 128, 16, kind=pa.KV_FP8_E4M3_ROW)
        for name in ("qkv", "cache", "scale"):
            c[name].copy_(d[name])
        pos.copy_(d["pos"])
        slots.copy_(d["slots"])
        c["pos"], c["slots"] = d["pos"], d["slots"]
        before = d["cache"]
        graph.replay()
        torch.cuda.synchronize()
        check(c, before, q_out)


def test_e4m3_decoder_agrees_with_the_oracle():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    mine = R.f64(codes)
    for i in range(256):
        o = oracle.e4m3_to_double(i)
        assert (o != o and mine[i] != mine[i]) or o == float(mine[i])


def test_one_call_and_its_parts_give_the_same_bits():
    """The streaming kernel on a whole batch, one warp per step on its parts."""
    c, d = (make(640, 2600, 32, 8, 128, 128, 16, kind=pa.KV_FP8_E4M3_ROW, norm=True) for _ in range(2))
    ref = call(c)
    q, k, v = parts(d)
    pos, slots, table = d["pos"].to(DEV), d["slots"].to(DEV), d["table"].to(DEV)
    outs = []
    for a in range(0, 2600, 400):
        b = a + 400
        outs.append(pa.rope_and_cache(q[a:b], k[a:b], v[a:b], d["cache"], slots[a:b], pos[a:b], table,
                                      block_size=16, kv_dtype=d["kind"], kv_scale=d["scale"],
                                      q_norm=d["qn"], k_norm=d["kn"], norm_eps=1e-5))
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(outs), ref)
    assert torch.equal(c["cache"], d["cache"]) and torch.equal(c["scale"], d["scale"])
