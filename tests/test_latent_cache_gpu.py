"""The write and the read-back of a cache of latent rows against the definition.

A copied value is exact.  A turned or normed one is a few fp32 operations rounded
once: within half a step u of the 16-bit type and 2^-21 of the pair's (the
value's) magnitude; the norm's sum has at most 512 terms of one sign, so it is
off by 512 * 2^-24 at most, half of that under the root."""
import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
from latent_ref import DTYPES, cos_sin_table, normed, turned

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_varlen_attention_attn_gb300 import _build
    _build.build()
    pa.load()


def randn(g, *shape, dt):
    return torch.randn(*shape, generator=g).to(dt).to(DEV)


def near(got, ref, size, dt):
    u = torch.finfo(dt).eps / 2
    least = 2.0 ** -25 if dt == torch.float16 else 0.0  # half a step below f16's normal range
    off = (got.double() - ref).abs() - (u * ref.abs() + (2.0 ** -21 + 2.0 ** -16) * size + least)
    assert off.max() <= 0, off.max().item()


@pytest.mark.parametrize("T,H", [(1, 1), (1, 16), (7, 9), (33, 128), (1500, 40), (4100, 16)])
@pytest.mark.parametrize("dc,dr,bs", [(512, 64, 16), (128, 16, 48), (256, 32, 64), (384, 48, 16)])
@pytest.mark.parametrize("kv_dtype,interleaved,norm,dense", [
    (pa.KV_BF16, False, True, False), (pa.KV_F16, True, True, True), (pa.KV_BF16, True, False, True)])
def test_write(T, H, dc, dr, bs, kv_dtype, interleaved, norm, dense):
    dt = DTYPES[kv_dtype]
    g = torch.Generator().manual_seed(T + H + dc)
    wide = randn(g, T, H, 3 * dr, dt=dt)
    q = wide[..., dr:2 * dr]
    down = randn(g, T, dc + dr, dt=dt)
    w = randn(g, dc, dt=dt) if norm else None
    table, _ = cos_sin_table(500, dr)
    table = table.to(DEV)
    pos = torch.randint(0, 500, (T,), generator=g).to(DEV)
    nb = T // bs + 3
    slots = torch.randperm(nb * bs, generator=g)[:T].to(DEV)
    if T > 5:
        slots[3], pos[4] = -1, -1
    cache = randn(g, nb, bs, dc + dr, dt=dt)
    before = cache.clone()
    row_out = torch.full((T, dc + dr), 7.0, dtype=dt, device=DEV) if dense else None
    q_out = torch.full((T, H, dr), 7.0, dtype=dt, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = pa.latent_rope_and_cache(q, down[:, :dc], down[:, dc:], cache, slots, pos, table,
                                   block_size=bs, kv_dtype=kv_dtype, interleaved=interleaved,
                                   latent_norm=w, q_out=q_out, row_out=row_out, device_status=status)
    assert got is q_out and status.item() == 0
    live = pos >= 0
    at = pos.clamp_min(0)
    keep = live & (slots >= 0)
    flat, old = cache.view(-1, dc + dr), before.view(-1, dc + dr)
    size = q.double().abs().view(T, H, dr).amax(-1, keepdim=True) * 2
    near(q_out[live], turned(q, table, at, interleaved)[live], size[live], dt)
    assert (q_out[~live] == 7).all()
    lat = normed(down[:, :dc], w, 1e-6) if norm else down[:, :dc].double()
    key = turned(down[:, None, dc:], table, at, interleaved)[:, 0]
    key_size = down[:, dc:].double().abs().amax(-1, keepdim=True) * 2
    for rows, on in ((flat[slots[keep]], keep), (row_out[live] if dense else None, live)):
        if rows is None:
            continue
        if norm:
            near(rows[:, :dc], lat[on], lat[on].abs(), dt)
        else:
            assert torch.equal(rows[:, :dc], down[on][:, :dc])
        near(rows[:, dc:], key[on], key_size[on], dt)
    other = torch.ones(nb * bs, dtype=torch.bool, device=DEV)
    other[slots[keep]] = False
    assert torch.equal(flat[other], old[other])
    if dense:
        assert (row_out[~live] == 7).all()


def test_in_place_and_without_rotation():
    g = torch.Generator().manual_seed(1)
    q, down = randn(g, 50, 6, 64, dt=torch.bfloat16), randn(g, 50, 192, dt=torch.bfloat16)
    table = cos_sin_table(64, 64)[0].to(DEV)
    pos, slots = torch.arange(50, device=DEV), torch.arange(50, device=DEV)
    cache = torch.zeros(4, 16, 192, dtype=torch.bfloat16, device=DEV)
    apart = pa.latent_rope_and_cache(q, down[:, :128], down[:, 128:], cache, slots, pos, table,
                                     block_size=16)
    q2, down2, cache2 = q.clone(), down.clone(), torch.zeros_like(cache)
    assert pa.latent_rope_and_cache(q2, down2[:, :128], down2[:, 128:], cache2, slots, pos, table,
                                    block_size=16, q_out=q2, row_out=down2) is q2
    assert torch.equal(apart, q2) and torch.equal(cache, cache2)
    assert torch.equal(down2, cache.view(-1, 192)[:50])
    assert pa.latent_rope_and_cache(None, down[:, :128], down[:, 128:], cache, slots, None, None,
                                    block_size=16) is None
    assert torch.equal(cache.view(-1, 192)[:50], down)


@pytest.mark.parametrize("fault", ["slot", "position"])
def test_faults_are_reported(fault):
    g = torch.Generator().manual_seed(2)
    q, down = randn(g, 5, 3, 32, dt=torch.float16), randn(g, 5, 160, dt=torch.float16)
    table = cos_sin_table(10, 32)[0].to(DEV)
    pos, slots = torch.arange(5, device=DEV), torch.arange(5, device=DEV)
    (slots if fault == "slot" else pos)[2] = 16 if fault == "slot" else 10
    cache = torch.zeros(1, 16, 160, dtype=torch.float16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.latent_rope_and_cache(q, down[:, :128], down[:, 128:], cache, slots, pos, table,
                             block_size=16, kv_dtype=pa.KV_F16, device_status=status)
    assert status.item() == 1
    assert (cache[0, 2] == 0).all() and (cache[0, :5] != 0).any(-1).sum() == 4


@pytest.mark.parametrize("dc,dr,bs", [(512, 64, 16), (128, 16, 48), (384, 64, 64)])
@pytest.mark.parametrize("kv_dtype", [pa.KV_BF16, pa.KV_F16])
def test_read_back(dc, dr, bs, kv_dtype):
    lens, first = [70, 0, 1, 200, 33], [5, 3, 0, 17, 64]
    g = torch.Generator().manual_seed(dc)
    nb = 40
    cache = randn(g, nb, bs, dc + dr, dt=DTYPES[kv_dtype])
    table = torch.randperm(nb, generator=g)[:35].view(5, 7).int()
    wide = torch.full((5, 16), -3, dtype=torch.int32)
    wide[:, :7] = table
    wide[3, 7:] = torch.randint(0, nb, (9,), generator=g).int()
    wide = wide.to(DEV)
    starts = torch.tensor([0] + lens).cumsum(0).int().to(DEV) + 2
    out = [torch.full((320, w), 9.0, dtype=cache.dtype, device=DEV) for w in (dc, dr)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = pa.gather_latent(cache, wide, starts, num_rows=320, latent_size=dc, block_size=bs,
                           kv_dtype=kv_dtype, key_starts=torch.tensor(first, dtype=torch.int32, device=DEV),
                           latent_out=out[0], rope_out=out[1], device_status=status)
    assert status.item() == 0
    rows = torch.cat([cache[wide[r][k // bs].long(), k % bs] for r, n in enumerate(lens)
                      for k in [torch.arange(first[r], first[r] + n, device=DEV)]])
    for x, want in zip(got, rows.split([dc, dr], 1)):
        assert torch.equal(x[2:2 + len(rows)], want)
        assert (x[:2] == 9).all() and (x[2 + len(rows):] == 9).all()


def test_read_back_of_bad_blocks():
    cache = torch.ones(4, 16, 144, dtype=torch.bfloat16, device=DEV)
    table = torch.tensor([[1, 9], [2, -1]], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 20, 70], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lat, rope = pa.gather_latent(cache, table, starts, num_rows=70, latent_size=128, block_size=16,
                                 device_status=status)
    assert status.item() == 1
    good = torch.zeros(70, dtype=torch.bool, device=DEV)
    good[:16] = good[20:36] = True
    assert (lat[good] == 1).all() and (lat[~good] == 0).all()
    assert (rope[good] == 1).all() and (rope[~good] == 0).all()
