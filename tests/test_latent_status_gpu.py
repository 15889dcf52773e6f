"""The status of a call in which one CTA gives up on a wait while the first one, which
clears the call's status, has not begun.  With the wait-test build, as in
test_latent_waits_gpu.py: a 10 ms limit, a first CTA that sleeps for 40 ms, and a copy of
the last CTA's that is never issued."""
import ctypes

import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
from latent_ref import Dense, Paged

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TIMEOUT = 6  # PATTN_ERR_DEVICE_TIMEOUT
BAD = 5      # PATTN_ERR_BAD_METADATA
FEW = dict(lens=[(300, 700), (20, 20)], H=2)    # an item a CTA at most
MANY = dict(lens=[(300, 700), (20, 20)], H=100)


@pytest.fixture
def wlib(monkeypatch):
    from paged_varlen_attention_attn_gb300 import _build
    lib = pa.load(_build.build_wait_test())
    lib.pattn_test_set_wait_skip.argtypes = [ctypes.c_int]
    lib.pattn_test_set_wait_skip.restype = None
    monkeypatch.setattr("paged_varlen_attention_attn_gb300.latent.load", lambda: lib)
    yield lib
    lib.pattn_test_set_wait_skip(0)


def _status(lib, op="latent_expanded_forward"):
    return pa.pattn_read_device_status(getattr(pa, op).last_ext, lib=lib)


@pytest.mark.parametrize("size", [FEW, MANY], ids=["few", "many"])
def test_a_timeout_before_the_first_cta_begins_is_reported(wlib, size):
    c = Dense(2, dn=128, dr=64, device=DEV, **size)
    wlib.pattn_test_set_wait_skip(5)
    try:
        c.run()
        status = _status(wlib)
    finally:
        wlib.pattn_test_set_wait_skip(0)
    torch.cuda.synchronize()
    assert status == TIMEOUT
    assert _status(wlib) == 0  # read and cleared
    c.check(c.run())
    assert _status(wlib) == 0


def test_a_timeout_does_not_stay_behind_for_other_calls(wlib):
    """Calls on the same workspace, none of whose CTAs give up."""
    few, many = (Dense(3, dn=128, dr=64, device=DEV, **s) for s in (FEW, MANY))
    absorbed = Paged(4, [(1, 300), (3, 90)], H=16, dc=256, dr=64, bs=16, device=DEV)
    ws = pa.Workspace()
    for run, op in ((few.run, "latent_expanded_forward"), (many.run, "latent_expanded_forward"),
                    (absorbed.run, "latent_forward")):
        wlib.pattn_test_set_wait_skip(5)
        try:
            few.run(workspace=ws)
            torch.cuda.synchronize()
        finally:
            wlib.pattn_test_set_wait_skip(0)
        run(workspace=ws)
        assert _status(wlib, op) == 0


def test_the_status_of_part_of_a_workspace_is_refused():
    c = Dense(6, dn=128, dr=64, device=DEV, **FEW)
    c.run()
    whole = pa.latent_expanded_forward.last_ext
    part = pa.Ext.from_buffer_copy(whole)
    part.workspace_bytes = 256
    assert pa.pattn_read_device_status(part) == 1
    assert pa.pattn_read_device_status(whole) == 0


def test_bad_metadata_of_few_items():
    c = Dense(5, dn=128, dr=64, device=DEV, **FEW)
    c.key_starts[2] += 1
    c.run()
    assert pa.pattn_read_device_status(pa.latent_expanded_forward.last_ext) == BAD
    assert pa.pattn_read_device_status(pa.latent_expanded_forward.last_ext) == 0
