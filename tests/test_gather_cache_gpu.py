"""pattn_gather_cache against the definition: 16-bit caches are copied bit for
bit; a code of an e4m3 cache times its scale is a product of a 4-bit and a
24-bit significand rounded to fp32 and then to bf16, so the result is within
2^-8 (half a bf16 step) and 2^-24 of the 64-bit product."""
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


def make(seed, lens, Hkv, D, bs, kind):
    g = torch.Generator().manual_seed(seed)
    need = [(n + bs - 1) // bs for n in lens]
    nb = sum(need) + 2
    perm = torch.randperm(nb, generator=g).int()
    table = torch.full((len(lens), max(need + [1])), -5, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    shape = (2, nb, bs, Hkv, D)
    scale = None
    if kind in (pa.KV_FP8_E4M3, pa.KV_FP8_E4M3_ROW):
        cache = torch.randint(0, 256, shape, generator=g, dtype=torch.int32)
        cache = torch.where(cache % 128 == 127, cache - 1, cache).to(torch.uint8)
        scale = (0.37, 1.93)
        if kind == pa.KV_FP8_E4M3_ROW:
            scale = torch.exp2(torch.rand(pa.row_scales_shape(nb, bs, Hkv), generator=g) * 40 - 20)
    else:
        dt = torch.float16 if kind == pa.KV_F16 else torch.bfloat16
        cache = torch.randn(shape, generator=g).to(dt)
    return cache, table, scale


def expected(cache, table, scale, lens, starts, bs, kind):
    rows = []
    for r, n in enumerate(lens):
        key = torch.arange(starts[r], starts[r] + n)
        blk, off = table[r][key // bs].long(), key % bs
        x = cache[:, blk, off]
        if kind == pa.KV_FP8_E4M3:
            x = R.f64(x) * torch.tensor(scale, dtype=torch.float32).double()[:, None, None, None]
        elif kind == pa.KV_FP8_E4M3_ROW:
            x = R.f64(x) * R.scales_at(scale, blk * bs + off).permute(2, 0, 1)[..., None]
        rows.append(x)
    return torch.cat(rows, 1)


@pytest.mark.parametrize("kind", [pa.KV_BF16, pa.KV_FP8_E4M3, pa.KV_F16, pa.KV_FP8_E4M3_ROW])
@pytest.mark.parametrize("lens,Hkv,D,bs", [
    ([1], 1, 16, 16), ([5, 0, 0, 3, 17], 2, 64, 16), ([130, 33, 257, 1], 8, 128, 64),
    ([0, 0, 40], 3, 80, 32), ([1000] * 3 + [7] * 30, 2, 128, 128), ([9, 6], 1, 24, 48)])
@pytest.mark.parametrize("offset", [0, 3])
def test_matches_the_definition(kind, lens, Hkv, D, bs, offset):
    # the first `offset` keys of each request are skipped
    cache, table, scale = make(sum(lens) + D + kind, [n + offset for n in lens], Hkv, D, bs, kind)
    osl = torch.tensor([2] + [0] * len(lens), dtype=torch.int32)
    osl[1:] = 2 + torch.tensor(lens).cumsum(0)
    total = int(osl[-1]) + 3
    dt = torch.float16 if kind == pa.KV_F16 else torch.bfloat16
    ko, vo = (torch.full((total, Hkv, D), 9.0, dtype=dt, device=DEV) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dev_scale = scale.to(DEV) if torch.is_tensor(scale) else scale
    starts = torch.full((len(lens),), offset, dtype=torch.int32, device=DEV) if offset else None
    pa.gather_cache(cache.to(DEV), table.to(DEV), osl.to(DEV), num_rows=total, block_size=bs,
                    kv_dtype=kind, kv_scale=dev_scale, key_starts=starts, key_out=ko,
                    value_out=vo, device_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    ref = expected(cache, table, scale, lens, [offset] * len(lens), bs, kind)
    got = torch.stack([ko, vo]).cpu()
    assert (got[:, :2] == 9.0).all() and (got[:, total - 3:] == 9.0).all()
    got = got[:, 2:total - 3]
    if kind in (pa.KV_BF16, pa.KV_F16):
        assert torch.equal(got.view(torch.int16), ref.view(torch.int16))
    else:
        assert ((R.f64(got) - ref).abs() <= (2.0 ** -8 + 2.0 ** -23) * ref.abs()).all()


def test_bad_blocks_and_keys_are_reported_and_zeroed():
    cache, table, scale = make(90, [40, 40], 2, 64, 16, pa.KV_FP8_E4M3_ROW)
    osl = torch.tensor([0, 40, 80], dtype=torch.int32)
    args = dict(num_rows=80, block_size=16, kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=scale.to(DEV))
    good = [x.cpu() for x in pa.gather_cache(cache.to(DEV), table.to(DEV), osl.to(DEV), **args)]
    for block in (-1, cache.shape[1], 1 << 30):
        t = table.clone()
        t[1, 1] = block
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = pa.gather_cache(cache.to(DEV), t.to(DEV), osl.to(DEV), device_status=status, **args)
        torch.cuda.synchronize()
        assert int(status) == 1
        for x, y in zip(got, good):
            assert (x[56:72] == 0).all()
            x = x.cpu()
            x[56:72] = y[56:72]
            assert torch.equal(x, y)
    # a range past the block table's row, and one that starts before key 0
    for start, zero in ((16, slice(72, 80)), (-4, slice(40, 44))):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = pa.gather_cache(cache.to(DEV), table.to(DEV), osl.to(DEV), device_status=status,
                              key_starts=torch.tensor([0, start], dtype=torch.int32, device=DEV), **args)
        torch.cuda.synchronize()
        assert int(status) == 1
        for x in got:
            assert (x[zero] == 0).all()


def test_rows_past_num_rows_are_not_written():
    cache, table, scale = make(91, [50], 2, 64, 16, pa.KV_FP8_E4M3_ROW)
    big = torch.full((60, 2, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    out = big[:33]
    other = torch.empty_like(out)
    pa.gather_cache(cache.to(DEV), table.to(DEV), torch.tensor([0, 50], dtype=torch.int32, device=DEV),
                    num_rows=33, block_size=16, kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=scale.to(DEV),
                    key_out=out, value_out=other)
    torch.cuda.synchronize()
    assert (big[33:] == 9.0).all() and not (big[32] == 9.0).all()


def test_no_requests_and_no_rows():
    cache, table, scale = make(92, [50], 2, 64, 16, pa.KV_FP8_E4M3_ROW)
    k, v = pa.gather_cache(cache.to(DEV), table.to(DEV), torch.zeros(2, dtype=torch.int32, device=DEV),
                           num_rows=0, block_size=16, kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=scale.to(DEV))
    assert k.shape == (0, 2, 64) == v.shape


def test_what_was_written_is_read_back():
    """Written with row scales and read back: within the quantisation's half step
    (2^-4 of the value, 2^-10 of the scale among subnormals) and bf16's."""
    g = torch.Generator().manual_seed(93)
    T, Hkv, D, bs, nb = 200, 4, 128, 16, 20
    k, v = (torch.randn(T, Hkv, D, generator=g).bfloat16() for _ in range(2))
    table = torch.randperm(nb, generator=g)[:13].int()[None]
    key = torch.arange(T)
    slots = table[0, key // bs].long() * bs + key % bs
    cache = torch.zeros(2, nb, bs, Hkv, D, dtype=torch.uint8, device=DEV)
    scales = torch.ones(pa.row_scales_shape(nb, bs, Hkv), device=DEV)
    pa.reshape_and_cache(k.to(DEV), v.to(DEV), cache, slots.to(DEV), block_size=bs,
                         kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=scales)
    ko, vo = pa.gather_cache(cache, table.to(DEV), torch.tensor([0, T], dtype=torch.int32, device=DEV),
                             num_rows=T, block_size=bs, kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=scales)
    torch.cuda.synchronize()
    for x, y in ((k, ko), (v, vo)):
        x, y = R.f64(x), R.f64(y)
        s = R.row_scale(x)[..., None]
        half = torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * s)
        assert ((x - y).abs() <= half * (1 + 2.0 ** -10) + 2.0 ** -8 * (x.abs() + half)).all()
