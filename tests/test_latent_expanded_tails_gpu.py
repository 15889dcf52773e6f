"""The last key tile of a request in the expanded form: its rows behind the request are
cleared once, before either of an item's two sub-tiles of 128 rows reads them."""
import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
from latent_ref import Dense

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BATCHES = {
    # a tile an item, so that the stages' phases run ahead of each other: one sub-tile or
    # both, the tail's tile seen by the second one alone or by both
    "short": [(r, s) for r in (1, 128, 129, 200, 256) for s in (1, 17, 63, 64)],
    "one sub-tile": [(1 + 7 * i % 128, 128 + i) for i in range(60)],
    "two sub-tiles": [(129 + 3 * i % 128, 257 + 5 * i) for i in range(60)],
    "both": [(100 + 37 * i % 700, 800 + 11 * i) for i in range(40)],
}


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_varlen_attention_attn_gb300 import _build
    _build.build()
    pa.load()


@pytest.mark.parametrize("name", sorted(BATCHES))
@pytest.mark.parametrize("causal", [1, 0])
@pytest.mark.parametrize("dn", [64, 128])
def test_what_lies_behind_a_request_is_cleared_for_both_sub_tiles(name, causal, dn):
    lens = [(n, s) for n, s in BATCHES[name] if not causal or n <= s]
    gap = 64  # rows of NaN behind every request's keys
    H = 8
    c = Dense(len(lens) + dn, lens, H=H, dn=dn, dr=64, device=DEV)
    want = c.run(causal)
    wide = [torch.full((c.up.shape[0] + gap * len(lens),) + x.shape[1:], float("nan"), dtype=x.dtype,
                       device=DEV) for x in (c.up, c.k_rope)]
    # (each request's keys, then the NaN: requests one at a time, so that the tail's tile
    # is followed by them)
    k0 = 0
    for r, (n, s) in enumerate(lens):
        at = k0 + gap * r
        for w, x in zip(wide, (c.up, c.k_rope)):
            w[at:at + s] = x[k0:k0 + s]
        k0 += s
    begins = c.key_starts[:-1] + gap * torch.arange(len(lens), dtype=torch.int32, device=DEV)
    ends = begins + (c.key_starts[1:] - c.key_starts[:-1])
    # requests as pairs of (its keys, an empty row range over the gap)
    keys = torch.stack([begins, ends], 1).flatten()
    keys = torch.cat([keys, keys[-1:] + gap]).int()
    rows = torch.stack([c.starts[:-1], c.starts[1:]], 1).flatten()
    rows = torch.cat([rows, rows[-1:]]).int()
    k_nope, value = wide[0].split([dn, dn], 2)
    for _ in range(4):
        got = pa.latent_expanded_forward(c.q, k_nope, wide[1], value, rows, keys, scale=c.scale,
                                         causal=causal)
        assert pa.pattn_read_device_status(pa.latent_expanded_forward.last_ext) == 0
        assert torch.equal(got, want)
    c.check(want, causal, requests=range(0, len(lens), 7))
