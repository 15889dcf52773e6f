"""That a tile lost or taken twice anywhere in a long context is outside the bound that
the kernels are held to."""
import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
from latent_runs import bound, planted, weights


@pytest.mark.parametrize("kv_dtype", [pa.KV_BF16, pa.KV_F16])
@pytest.mark.parametrize("lens,H", [([(1, 20000)], 8), ([(1, 9000), (1, 17000)], 3), ([(2, 12000)], 3)])
@pytest.mark.parametrize("keys", [48, 64])
def test_every_tile_is_missed(kv_dtype, lens, H, keys):
    c = planted(H, lens, H=H, dc=512, dr=64, bs=64, kv_dtype=kv_dtype, device="cpu")
    for r, (n, s) in enumerate(lens):
        w, size = weights(c, r)
        out, off = bound(c, r, w, size)
        v, total = c.rows(r)[:, :512].double(), w.sum(-1, keepdim=True)
        for k0 in range(0, s, keys):
            part = w[..., k0:k0 + keys]
            mine = torch.einsum("nhs,sd->nhd", part, v[k0:k0 + keys])
            weight = part.sum(-1, keepdim=True)
            for times in (-1, 1):  # lost, or taken twice, in the values and in the sum or there alone
                for in_sum in (0, 1):
                    wrong = (out * total + times * mine) / (total + times * in_sum * weight)
                    assert ((wrong - out).abs() > off).any(), (r, k0, times, in_sum)
