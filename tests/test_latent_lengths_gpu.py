"""Lengths that a block-table row could hold and 32 bits cannot count in tiles."""
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


@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 50, 0x7fffff01])
def test_a_length_at_the_end_of_32_bits_is_refused(H, length):
    bs = 192
    c = Paged(H, [(1, 300), (1, 200), (1, 100)], H=H, dc=256, dr=64, bs=bs, device=DEV)
    wide = torch.zeros(3, 2 ** 31 // bs + 1, dtype=torch.int32, device=DEV)
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    c.seq_lens[1] = length
    out = torch.full((3, H, 256), float("nan"), dtype=torch.bfloat16, device=DEV)
    c.run(out=out)
    assert pa.pattn_read_device_status(pa.latent_forward.last_ext) == 5
    assert (out[1] == 0).all()
    c.check(out, requests=[0, 2])
