"""Bounded waits of the latent attentions: a copy that is never issued is reported as a
timeout, and the next call is right.  With the wait-test build, as in
test_wait_timeout_gpu.py: a 10 ms limit, and CTA 0 posts no bytes for its first key
tile, a barrier phase that nothing then completes."""
import ctypes

import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
from latent_ref import Dense, Paged

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TIMEOUT = 6  # PATTN_ERR_DEVICE_TIMEOUT


@pytest.fixture
def wlib(monkeypatch):
    from paged_varlen_attention_attn_gb300 import _build
    lib = pa.load(_build.build_wait_test())
    lib.pattn_test_set_wait_skip.argtypes = [ctypes.c_int]
    lib.pattn_test_set_wait_skip.restype = None
    monkeypatch.setattr("paged_varlen_attention_attn_gb300.latent.load", lambda: lib)
    yield lib
    lib.pattn_test_set_wait_skip(0)


def _absorbed(H):
    return Paged(1, [(1, 900), (3, 400)], H=H, dc=512, dr=64, bs=16, device=DEV)


def _expanded(heads):
    return Dense(2, [(300, 700), (20, 20)], H=heads, dn=128, dr=64, device=DEV)


@pytest.mark.parametrize("make,op,mode", [
    (lambda: _absorbed(8), "latent_forward", 3), (lambda: _absorbed(64), "latent_forward", 3),
    (lambda: _expanded(2), "latent_expanded_forward", 4),
    (lambda: _expanded(100), "latent_expanded_forward", 4)])
def test_a_copy_that_never_comes(wlib, make, op, mode):
    c = make()
    wlib.pattn_test_set_wait_skip(mode)
    try:
        c.run()
        status = pa.pattn_read_device_status(getattr(pa, op).last_ext, lib=wlib)
    finally:
        wlib.pattn_test_set_wait_skip(0)
    torch.cuda.synchronize()
    assert status == TIMEOUT
    c.check(c.run())
    assert pa.pattn_read_device_status(getattr(pa, op).last_ext, lib=wlib) == 0
