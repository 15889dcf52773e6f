"""Attention over a paged cache of latent rows (the absorbed form) against the
definition in 64 bits: head counts around the row tiles of 16, 32 and 64, lengths
around the tiles of 64 keys, pages that end inside a tile, rows of several tokens,
keys cut over the GPU, and what lies behind a request's keys."""
import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
from latent_ref import Paged

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_varlen_attention_attn_gb300 import _build
    _build.build()
    pa.load()


def status():
    return pa.pattn_read_device_status(pa.latent_forward.last_ext)


@pytest.mark.parametrize("H", [1, 3, 16, 17, 32, 40, 64, 65, 128])
@pytest.mark.parametrize("kv_dtype", [pa.KV_BF16, pa.KV_F16])
def test_single_tokens(H, kv_dtype):
    lens = [(1, s) for s in (1, 2, 16, 63, 64, 65, 127, 128, 200, 513)]
    c = Paged(H, lens, H=H, dc=512, dr=64, bs=16, kv_dtype=kv_dtype, device=DEV, poison=True)
    out = c.run()
    assert status() == 0
    c.check(out)


@pytest.mark.parametrize("dc,dr", [(128, 16), (128, 32), (256, 64), (384, 48), (512, 16)])
@pytest.mark.parametrize("H", [4, 20, 64])
def test_sizes_of_the_row(dc, dr, H):
    lens = [(1, 700), (3, 90), (1, 64), (5, 5), (0, 10), (1, 1)]
    c = Paged(dc + dr, lens, H=H, dc=dc, dr=dr, bs=32, device=DEV, poison=True)
    out = c.run()
    assert status() == 0
    c.check(out)


@pytest.mark.parametrize("bs", [16, 32, 48, 64, 80, 128, 192])
def test_block_sizes(bs):
    lens = [(1, 1000), (2, 129), (7, 300), (1, 47), (1, 64)]
    c = Paged(bs, lens, H=16, dc=512, dr=64, bs=bs, device=DEV, poison=True)
    c.check(c.run())


@pytest.mark.parametrize("H", [1, 5, 16, 24, 128])
@pytest.mark.parametrize("causal", [1, 0])
def test_chunks(H, causal):
    lens = [(70, 70), (33, 500), (2, 2), (1, 300), (64, 128), (130, 1000)]
    c = Paged(7 * H + causal, lens, H=H, dc=512, dr=64, bs=16, device=DEV, poison=True)
    out = c.run(causal=causal)
    assert status() == 0
    c.check(out, causal)


@pytest.mark.parametrize("lens", [[(1, 20000)], [(1, 9000), (1, 3), (1, 17000)], [(2, 12000)] * 3])
@pytest.mark.parametrize("H", [8, 32, 128])
def test_keys_cut_over_the_gpu(lens, H):
    c = Paged(H + len(lens), lens, H=H, dc=512, dr=64, bs=64, kv_dtype=pa.KV_F16, device=DEV)
    c.check(c.run())


@pytest.mark.parametrize("H", [16, 40])
def test_lengths_around_the_tiles_of_48_keys(H):
    lens = [(1, s) for s in (47, 48, 49, 95, 96, 97, 143, 144, 145, 191, 193)]
    c = Paged(H, lens, H=H, dc=256, dr=64, bs=16, device=DEV, poison=True)
    c.check(c.run())


@pytest.mark.parametrize("H", [100, 512, 513, 1000])
def test_single_tokens_of_many_heads(H):
    c = Paged(H, [(1, 5), (0, 3), (1, 900), (1, 64)], H=H, dc=128, dr=16, bs=16, device=DEV, poison=True)
    c.check(c.run())
    assert status() == 0


@pytest.mark.parametrize("H", [16, 128])
def test_longest_row_given_too_long_or_too_short(H):
    c = Paged(8, [(1, 90), (3, 200), (1, 30)], H=H, dc=128, dr=64, bs=16, device=DEV)
    c.check(c.run(max_query_len=77))
    assert status() == 0
    out = torch.full((5, H, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    c.run(out=out, max_query_len=1)  # with single tokens' layout the chunk is refused
    if H == 128:
        assert status() == 5 and (out[1:4] == 0).all()
    c.check(out, requests=[0, 2])


def test_many_requests():
    lens = [(1, 1 + (37 * i) % 400) for i in range(1500)]
    c = Paged(5, lens, H=16, dc=128, dr=64, bs=16, device=DEV)
    c.check(c.run(), requests=range(0, 1500, 97))


def test_scores_that_grow_along_the_keys():
    """The reference max moves at almost every tile."""
    c = Paged(9, [(1, 1500), (4, 900)], H=16, dc=512, dr=64, bs=16, device=DEV)
    rise = torch.linspace(0.05, 3.0, 1500, device=DEV)
    for r, (_, s) in enumerate(c.lens):
        key = torch.arange(s, device=DEV)
        at = (c.table[r][key // 16].long(), key % 16)
        c.cache[at] = (c.cache[at].float().abs() * rise[:s, None]).bfloat16()
    c.q = c.q.abs() * 0.25
    c.check(c.run())


def test_rows_outside_the_requests_are_left():
    c = Paged(3, [(2, 40), (1, 7)], H=5, dc=128, dr=16, bs=16, device=DEV)
    c.q = torch.cat([c.q, c.q[:2], c.q[:2]])
    out = torch.full((7, 5, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    c.starts = c.starts + 2
    c.q[2:5] = c.q[:3].clone()
    c.run(out=out)
    assert (out[:2] == 3).all() and (out[5:] == 3).all()
    c.q = c.q[2:5]
    c.check(out[2:5])


def test_results_repeat_bit_for_bit():
    c = Paged(4, [(1, 5000), (1, 700), (3, 2000)], H=32, dc=512, dr=64, bs=16, device=DEV)
    first = c.run()
    for _ in range(5):
        assert torch.equal(first, c.run())


@pytest.mark.parametrize("fault", ["block", "length", "query", "table"])
@pytest.mark.parametrize("H", [16, 128])
def test_bad_metadata_is_reported_and_kept_apart(fault, H):
    c = Paged(6, [(1, 300), (1, 200), (1, 100)], H=H, dc=256, dr=64, bs=16, device=DEV)
    out = torch.full((3, H, 256), float("nan"), dtype=torch.bfloat16, device=DEV)
    if fault == "block":
        c.table[1, 3] = c.nb + 5
    elif fault == "length":
        c.seq_lens[1] = c.table.shape[1] * 16 + 1
    elif fault == "query":
        c.seq_lens[1] = 0
    else:
        c.table[1, 0] = -1
    c.run(out=out)
    assert status() == 5
    assert torch.isfinite(out.float()).all()
    c.check(out, requests=[0, 2])
    assert status() == 0  # read and cleared
