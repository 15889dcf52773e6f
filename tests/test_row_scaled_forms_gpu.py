"""Forms of attention over a row-scaled e4m3 cache in combination: value scales
far apart with windows, sinks and odd head groups; cascade and the
workspace-free decode at head size 64.  Definition and tolerance as in
test_row_scaled_attention_gpu."""
import numpy as np
import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
from test_row_scaled_attention_gpu import BATCHES, DEV, Case, built  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv,bs", [(8, 2, 16), (6, 2, 32), (5, 1, 128), (16, 1, 64), (7, 7, 16)])
@pytest.mark.parametrize("window", [0, 1, 90, 257])
def test_value_scales_far_apart_under_a_window(D, H, Hkv, bs, window):
    c = Case(300 + D + H + window, BATCHES["mixed"], H, Hkv, D, bs)
    c.spread_scales(-30, 30, 7, which=(1,))
    c.check(c.run(window=window), window=window)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (6, 2)])
@pytest.mark.parametrize("lo,hi", [(-30, 30), (-58, -50), (50, 58)])
def test_value_scales_far_apart_with_sinks(D, H, Hkv, lo, hi):
    c = Case(310 + D + H, BATCHES["mixed"], H, Hkv, D, 16)
    c.spread_scales(lo, hi, 8, which=(1,))
    sinks = torch.linspace(-3.0, 6.0, H)
    sinks[1] = -float("inf")
    c.check(c.run(sinks=sinks.to(DEV)), sinks=sinks)
    c.check(c.run(sinks=sinks.to(DEV), num_splits=5, window=200), sinks=sinks, window=200)


@pytest.mark.parametrize("D", [64, 128])
def test_some_tiles_far_apart_and_some_not(D):
    """Long rows whose tiles take both paths in turn."""
    c = Case(320 + D, [(200, 900), (1, 1500), (130, 1300), (257, 257)], 8, 4, D, 16)
    g = torch.Generator().manual_seed(9)
    some = torch.rand(c.NB, generator=g) < 0.05
    e = torch.randint(-30, 31, c.scales[some][:, :, :, 1].shape, generator=g).float()
    s = c.scales[some]
    s[:, :, :, 1] = torch.exp2(e)
    c.scales[some] = s
    c.check(c.run())
    c.check(c.run(window=333), window=333)


@pytest.mark.parametrize("H,Hkv", [(8, 2), (6, 2), (16, 1)])
@pytest.mark.parametrize("reqs", [[(1, 200), (1, 500), (1, 333)], [(40, 200), (1, 300), (130, 400)],
                                  [(1, 700)]])
@pytest.mark.parametrize("wide", [False, True])
def test_cascade_at_head_size_64(reqs, H, Hkv, wide):
    c = Case(330 + H, reqs, H, Hkv, 64, 16)
    if wide:
        c.spread_scales(-20, 20, 10, which=(1,))
    c.bt[1:, :6] = c.bt[0, :6]
    out = pa.cascade_forward(*c.args(), common_prefix_len=96, **c.kw())
    assert pa.pattn_read_device_status(pa.forward.last_ext) == 0
    c.check(out)


@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 64), (6, 2, 64), (16, 1, 64), (6, 2, 128)])
@pytest.mark.parametrize("window", [0, 60])
def test_the_workspace_free_decode(H, Hkv, D, window):
    c = Case(340 + H + D, BATCHES["mixed"], H, Hkv, D, 16)
    q, cache, bt, sl, qsl = c.args()
    scales = c.scales.to(DEV)
    out = torch.full((c.T, H, D), 7.0, dtype=torch.bfloat16, device=DEV)
    st = pa.pattn_decode_fwd_static(
        q.data_ptr(), cache.data_ptr(), bt.data_ptr(), sl.data_ptr(), qsl.data_ptr(), out.data_ptr(),
        c.scale, H, Hkv, D, 16, window, 1, pa.KV_FP8_E4M3_ROW, scales, len(c.reqs), c.T, bt.shape[1],
        c.NB, 600, 0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0
    rows = np.array([int(c.qsl[r]) for r, (n, _) in enumerate(c.reqs) if n == 1])
    c.check(out, rows=rows, window=window)
    rest = np.setdiff1d(np.arange(c.T), rows)
    assert (out[rest] == 7.0).all()
