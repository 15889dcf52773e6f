"""Keys cut over the GPU, with values that tell which of them were added up
(latent_runs.py): no tile at a share's border or in a merge is lost or taken twice."""
import pytest

import paged_varlen_attention_attn_gb300 as pa
from latent_runs import check, planted

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_varlen_attention_attn_gb300 import _build
    _build.build()
    pa.load()


@pytest.mark.parametrize("lens", [[(1, 20000)], [(1, 9000), (1, 3), (1, 17000)], [(2, 12000)] * 3,
                                  [(1, 700 + 41 * i) for i in range(64)], [(5, 3000), (1, 8000), (40, 2100)]])
@pytest.mark.parametrize("H", [8, 32, 128])
@pytest.mark.parametrize("kv_dtype", [pa.KV_BF16, pa.KV_F16])
def test_every_run_of_keys_is_in_the_output_once(lens, H, kv_dtype):
    c = planted(H + len(lens), lens, H=H, dc=512, dr=64, bs=64, kv_dtype=kv_dtype, device=DEV)
    check(c, c.run())
    assert pa.pattn_read_device_status(pa.latent_forward.last_ext) == 0


@pytest.mark.parametrize("dc,dr,bs", [(128, 16, 16), (256, 64, 32), (384, 32, 80)])
@pytest.mark.parametrize("H", [4, 40, 100])
def test_other_rows(dc, dr, bs, H):
    c = planted(dc + H, [(1, 9000), (1, 3), (7, 5000), (1, 16)], H=H, dc=dc, dr=dr, bs=bs,
                kv_dtype=pa.KV_F16, device=DEV)
    check(c, c.run())
