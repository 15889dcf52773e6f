"""Ragged attention over keys and values projected up from latents (the expanded
form) against the definition in 64 bits."""
import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
from latent_ref import Dense

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_varlen_attention_attn_gb300 import _build
    _build.build()
    pa.load()


def status():
    return pa.pattn_read_device_status(pa.latent_expanded_forward.last_ext)


@pytest.mark.parametrize("dn,dr", [(128, 64), (64, 64), (128, 16), (64, 32), (128, 48)])
@pytest.mark.parametrize("kv_dtype", [pa.KV_BF16, pa.KV_F16])
@pytest.mark.parametrize("causal", [1, 0])
def test_ragged_batch(dn, dr, kv_dtype, causal):
    lens = [(1, 1), (2, 130), (0, 40), (128, 128), (129, 129), (257, 400), (64, 64), (1, 300),
            (300, 300)]
    c = Dense(dn + dr, lens, H=5, dn=dn, dr=dr, kv_dtype=kv_dtype, device=DEV)
    out = c.run(causal)
    assert status() == 0
    c.check(out, causal)


@pytest.mark.parametrize("H", [1, 2, 16])
@pytest.mark.parametrize("lens", [[(700, 700)], [(5, 2000), (600, 1500)], [(1, 1)], [(1200, 1200), (3, 3)]])
def test_heads_and_lengths(H, lens):
    c = Dense(H, lens, H=H, dn=128, dr=64, device=DEV)
    c.check(c.run())


def test_many_items():
    """More items than the GPU has SMs: the item ring and the claims at work."""
    lens = [(100 + 37 * i % 600, 100 + 37 * i % 600 + 50 * (i % 3)) for i in range(40)]
    c = Dense(1, lens, H=16, dn=128, dr=64, kv_dtype=pa.KV_F16, device=DEV)
    c.check(c.run(), requests=range(0, 40, 3))


def test_many_requests():
    lens = [(1 + 5 * (i % 7 == 3), 6 + 11 * i % 90) for i in range(700)]
    c = Dense(7, lens, H=2, dn=64, dr=16, device=DEV)
    c.check(c.run(), requests=range(0, 700, 41))
    assert status() == 0


def test_requests_without_keys():
    c = Dense(2, [(3, 0), (4, 9), (2, 0)], H=3, dn=64, dr=32, device=DEV)
    c.check(c.run(causal=0), causal=0)
    assert status() == 0


def test_scores_that_grow_along_the_keys():
    c = Dense(3, [(300, 900)], H=2, dn=128, dr=64, device=DEV)
    rise = torch.linspace(0.05, 3.0, 900, device=DEV)[:, None]
    c.up[..., :128] = (c.up[..., :128].float().abs() * rise[..., None]).bfloat16()
    c.k_rope[:] = (c.k_rope.float().abs() * rise).bfloat16()
    c.q.abs_().mul_(0.25)
    c.check(c.run())


def test_strides_and_rows_outside_the_requests():
    """Heads before tokens, rows inside wider tensors, q and keys that no request owns."""
    c = Dense(4, [(40, 60), (7, 90)], H=4, dn=64, dr=32, device=DEV)
    T, K = 47, 150
    nan = float("nan")

    def inside(x, before, after):
        shape = (x.shape[0] + before + after,) + tuple(x.shape[1:-1]) + (x.shape[-1] + 24,)
        wide = torch.full(shape, nan, dtype=x.dtype, device=DEV)
        if x.dim() == 3:
            wide = wide.transpose(0, 1).contiguous().transpose(0, 1)
        view = wide[..., 8:8 + x.shape[-1]]
        view[before:before + x.shape[0]] = x
        return view

    q, kn, kr, v = inside(c.q, 3, 2), inside(c.k_nope, 5, 1), inside(c.k_rope, 5, 1), inside(c.value, 5, 1)
    out = torch.full((T + 5, 4, 64), 2.0, dtype=torch.bfloat16, device=DEV)
    pa.latent_expanded_forward(q, kn, kr, v, c.starts + 3, c.key_starts + 5, scale=c.scale, out=out)
    assert status() == 0
    assert (out[:3] == 2).all() and (out[T + 3:] == 2).all()
    c.check(out[3:T + 3])


def test_results_repeat_bit_for_bit():
    c = Dense(5, [(900, 900), (300, 2000)], H=8, dn=128, dr=64, device=DEV)
    first = c.run()
    for _ in range(4):
        assert torch.equal(first, c.run())


@pytest.mark.parametrize("fault", ["more rows than keys", "rows", "keys", "backwards"])
def test_bad_metadata_is_reported_and_kept_apart(fault):
    c = Dense(6, [(30, 50), (20, 40), (10, 10)], H=3, dn=128, dr=64, device=DEV)
    out = torch.full((60, 3, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    good = [0, 1]
    if fault == "more rows than keys":
        c.key_starts[3] = c.key_starts[2] + 9
    elif fault == "rows":
        c.starts[3] = 61
    elif fault == "keys":
        c.key_starts[3] = 101
    else:
        c.key_starts[3] = c.key_starts[2] - 1
    c.run(out=out)
    assert status() == 5
    assert torch.isfinite(out.float()).all()
    c.check(out, requests=good)
    assert (out[50:] == 0).all()
