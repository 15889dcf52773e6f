"""Host-side checks of the rotary cache write, the row-scaled write and the
read-back (no GPU): the argument struct's layout, refusals before any CUDA call,
and the binding's own checks."""
import ctypes
import os
import subprocess

import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
from paged_varlen_attention_attn_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # aligned and never dereferenced by these calls


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load()


def test_struct_layout_matches_c(tmp_path):
    names = [f[0] for f in pa.RopeArgs._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "pattn.h"\nint main(void) {\n' + "".join(
        f'printf("%zu\\n", offsetof(pattn_rope_t, {n}));\n' for n in names) +
        'printf("%zu\\n", sizeof(pattn_rope_t));\nreturn 0; }\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(pa.RopeArgs, n).offset for n in names] + [ctypes.sizeof(pa.RopeArgs)]


def _rope(lib, pair_axis=None, kv_scale=None, **kw):
    a = pa.RopeArgs()
    a.struct_size = ctypes.sizeof(a)
    base = dict(q=FAKE, q_out=FAKE, key=FAKE, value=FAKE, q_stride=1024, q_out_stride=1024,
                key_stride=256, value_stride=256, cos_sin=FAKE, positions=FAKE, kv_cache=FAKE,
                row_scales=FAKE, slot_mapping=FAKE, num_tokens=0, num_heads=8, num_kv_heads=2,
                head_size=128, rot_dim=128, num_axes=1, max_position=10, kv_dtype=3,
                block_size=16, num_blocks=4)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    keep = None
    if pair_axis is not None:
        keep = ctypes.create_string_buffer(bytes(pair_axis), len(pair_axis))
        a.pair_axis = ctypes.addressof(keep)
    if kv_scale is not None:
        ks = (ctypes.c_float * 2)(*kv_scale)
        a.kv_scale = ctypes.addressof(ks)
    return lib.pattn_rope_and_cache(ctypes.byref(a))


@pytest.mark.parametrize("kw,status", [
    ({}, 0),                                        # no tokens: nothing to do
    (dict(q=0, q_out=0), 0),                        # keys alone
    (dict(key=0, value=0, kv_cache=0, slot_mapping=0, row_scales=0), 0),  # q alone
    (dict(num_axes=0, cos_sin=0, positions=0), 0),  # no rotation
    (dict(num_axes=3, pair_axis=[0, 1, 2, 0] * 16), 0),
    (dict(q_norm=FAKE, k_norm=FAKE, norm_eps=1e-6), 0),
    (dict(struct_size=8), 1),
    (dict(q=0, q_out=0, key=0, value=0), 1),        # nothing to do at all
    (dict(q_out=0), 1),
    (dict(value=0), 1),
    (dict(num_tokens=-1), 1),
    (dict(num_heads=0), 1),
    (dict(num_kv_heads=0), 1),
    (dict(kv_cache=0), 1),
    (dict(slot_mapping=0), 1),
    (dict(row_scales=0), 1),
    (dict(row_scales=FAKE + 4), 1),
    (dict(kv_dtype=1), 1),                          # e4m3 without scales
    (dict(kv_dtype=1, kv_scale=(1.0, 0.0)), 1),
    (dict(kv_dtype=1, kv_scale=(1.0, float("nan"))), 1),
    (dict(kv_dtype=1, kv_scale=(1.0, 2.0)), 0),
    (dict(kv_dtype=4), 2),
    (dict(block_size=24), 1),
    (dict(num_blocks=-1), 1),
    (dict(head_size=120), 2),
    (dict(head_size=272), 2),
    (dict(rot_dim=40), 2),
    (dict(rot_dim=144), 1),
    (dict(rot_dim=0), 1),
    (dict(cos_sin=0), 1),
    (dict(positions=0), 1),
    (dict(max_position=0), 1),
    (dict(num_axes=5, pair_axis=[0] * 64), 1),
    (dict(num_axes=-1), 1),
    (dict(num_axes=2), 1),                          # several axes need pair_axis
    (dict(num_axes=2, pair_axis=[0, 2] * 32), 1),   # an axis that is not there
    (dict(interleaved=2), 1),
    (dict(q_norm=FAKE, norm_eps=-1.0), 1),
    (dict(q_norm=FAKE, norm_eps=float("nan")), 1),
    (dict(q_norm=FAKE + 2), 1),
    (dict(q_stride=1020), 1),
    (dict(q_stride=1016), 1),                       # a token's row reaches into the next
    (dict(q_out_stride=0), 1),
    (dict(key_stride=248), 1),
    (dict(value=FAKE + 8), 1),
    (dict(cos_sin=FAKE + 4), 1),
])
def test_rope_arguments_are_checked_on_the_host(lib, kw, status):
    assert _rope(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(key=0), 1), (dict(value=0), 1), (dict(cache=0), 1), (dict(scales=0), 1),
    (dict(slots=0), 1), (dict(T=-1), 1), (dict(Hkv=0), 1), (dict(D=72), 2), (dict(bs=20), 1),
    (dict(scales=FAKE + 8), 1), (dict(NB=-1), 1)])
def test_row_write_arguments_are_checked_on_the_host(lib, kw, status):
    a = dict(key=FAKE, value=FAKE, cache=FAKE, scales=FAKE, slots=FAKE, T=0, Hkv=2, D=128, bs=16, NB=4)
    a.update(kw)
    assert lib.pattn_reshape_and_cache_rows(a["key"], a["value"], a["cache"], a["scales"], a["slots"],
                                            a["T"], a["Hkv"], a["D"], a["bs"], a["NB"], None, None) == status


@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(cache=0), 1), (dict(bt=0), 1), (dict(osl=0), 1), (dict(ko=0), 1), (dict(vo=0), 1),
    (dict(B=-1), 1), (dict(rows=-1), 1), (dict(mbps=-1), 1), (dict(NB=-1), 1), (dict(Hkv=0), 1),
    (dict(D=12), 2), (dict(bs=8), 1), (dict(kind=9), 2), (dict(kind=3, scale=0), 1),
    (dict(kind=1, scale=0), 1), (dict(ko=FAKE + 8), 1)])
def test_gather_arguments_are_checked_on_the_host(lib, kw, status):
    a = dict(cache=FAKE, bt=FAKE, osl=FAKE, ko=FAKE, vo=FAKE, B=2, rows=0, mbps=4, NB=4, Hkv=2, D=64,
             bs=16, kind=3, scale=FAKE)
    a.update(kw)
    assert lib.pattn_gather_cache(a["cache"], a["bt"], None, a["osl"], a["ko"], a["vo"], a["B"], a["rows"],
                                  a["mbps"], a["NB"], a["Hkv"], a["D"], a["bs"], a["kind"],
                                  a["scale"] or None, None, None) == status


def test_pair_axis_of_sections():
    assert pa.rope_pair_axis((2, 1, 1)) == [0, 0, 1, 2]
    assert pa.rope_pair_axis((2, 1, 1), interleaved=True) == [0, 1, 2, 0]
    assert pa.rope_pair_axis((4, 2, 2), interleaved=True) == [0, 1, 2, 0, 1, 2, 0, 0]
    mixed = pa.rope_pair_axis((24, 20, 20), interleaved=True)
    assert [mixed.count(a) for a in range(3)] == [24, 20, 20] and mixed[:6] == [0, 1, 2, 0, 1, 2]
    with pytest.raises(ValueError):
        pa.rope_pair_axis((1, 30, 1), interleaved=True)


def _tensors(T=3, H=4, Hkv=2, D=64, kind=pa.KV_FP8_E4M3_ROW):
    bf = torch.bfloat16
    return dict(q=torch.zeros(T, H, D, dtype=bf), key=torch.zeros(T, Hkv, D, dtype=bf),
                value=torch.zeros(T, Hkv, D, dtype=bf),
                kv_cache=torch.zeros(2, 2, 16, Hkv, D, dtype=torch.uint8),
                slot_mapping=torch.zeros(T, dtype=torch.int64),
                positions=torch.zeros(T, dtype=torch.int64), cos_sin=torch.zeros(8, D),
                block_size=16, kv_dtype=kind, kv_scale=torch.zeros(pa.row_scales_shape(2, 16, Hkv)))


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(3, 4, 64)),                                     # fp32 q
    dict(q=torch.zeros(4, 3, 64, dtype=torch.bfloat16).transpose(0, 1)),  # heads not contiguous
    dict(key=torch.zeros(4, 2, 64, dtype=torch.bfloat16)),             # another token count
    dict(value=torch.zeros(3, 2, 32, dtype=torch.bfloat16)),
    dict(value=None),
    dict(kv_cache=torch.zeros(2, 2, 16, 2, 64, dtype=torch.bfloat16)),  # 16-bit cache for codes
    dict(kv_cache=torch.zeros(2, 2, 32, 2, 64, dtype=torch.uint8)),
    dict(slot_mapping=torch.zeros(3, dtype=torch.int32)),
    dict(slot_mapping=torch.zeros(2, dtype=torch.int64)),
    dict(positions=torch.zeros(3, dtype=torch.int32)),
    dict(positions=torch.zeros(4, dtype=torch.int64)),
    dict(positions=torch.zeros(2, 3, dtype=torch.int64)),              # axes without pair_axis
    dict(cos_sin=torch.zeros(8, 64, dtype=torch.bfloat16)),
    dict(kv_scale=None),
    dict(kv_scale=torch.zeros(2, 1, 2, 2, 8)),
    dict(q_norm=torch.ones(64)),
    dict(q_out=torch.zeros(3, 4, 32, dtype=torch.bfloat16)),
    dict(q=None, key=None, value=None),
])
def test_the_binding_refuses_tensors_that_do_not_fit(kw):
    a = _tensors()
    a.update(kw)
    with pytest.raises(ValueError):
        pa.rope_and_cache(stream=None, **a)


def test_the_binding_refuses_gather_tensors_that_do_not_fit():
    ok = dict(kv_cache=torch.zeros(2, 2, 16, 2, 64, dtype=torch.uint8),
              block_table=torch.zeros(2, 2, dtype=torch.int32),
              out_start_loc=torch.zeros(3, dtype=torch.int32), num_rows=4, block_size=16,
              kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=torch.zeros(pa.row_scales_shape(2, 16, 2)))
    for kw in (dict(block_table=torch.zeros(2, 2, dtype=torch.int64)),
               dict(out_start_loc=torch.zeros(2, dtype=torch.int32)),
               dict(key_starts=torch.zeros(3, dtype=torch.int32)),
               dict(kv_cache=torch.zeros(2, 2, 16, 2, 64, dtype=torch.bfloat16)),
               dict(block_size=32), dict(kv_scale=torch.zeros(2, 16)),
               dict(key_out=torch.zeros(3, 2, 64, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            pa.gather_cache(**{**ok, **kw})


def test_the_binding_refuses_rows_that_do_not_fit():
    bf = torch.bfloat16
    ok = dict(key=torch.zeros(3, 2, 64, dtype=bf), value=torch.zeros(3, 2, 64, dtype=bf),
              kv_cache=torch.zeros(2, 2, 16, 2, 64, dtype=torch.uint8),
              slot_mapping=torch.zeros(3, dtype=torch.int64), block_size=16,
              kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=torch.zeros(pa.row_scales_shape(2, 16, 2)))
    for kw in (dict(key=torch.zeros(3, 4, 64, dtype=bf)[:, ::2]), dict(value=torch.zeros(3, 2, 64)),
               dict(value=torch.zeros(2, 2, 64, dtype=bf)), dict(slot_mapping=torch.zeros(3, dtype=torch.int32)),
               dict(kv_cache=torch.zeros(2, 2, 16, 2, 64, dtype=bf)), dict(kv_scale=(1.0, 1.0)),
               dict(kv_scale=torch.zeros(2, 2, 16, 2, 2).transpose(0, 1))):
        with pytest.raises(ValueError):
            pa.reshape_and_cache(**{**ok, **kw})


def test_attention_refuses_row_scales_that_do_not_fit():
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    args = (q, torch.zeros(2, 2, 16, 2, 64, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.int32),
            torch.ones(1, dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32))
    kw = dict(scale=1.0, num_heads=4, num_kv_heads=2, head_size=64, block_size=16,
              kv_dtype=pa.KV_FP8_E4M3_ROW, max_query_len=1, max_seq_len=16)
    for scales in (None, (1.0, 1.0), torch.zeros(2, 1, 2, 2, 8), torch.zeros(pa.row_scales_shape(2, 16, 2)).double()):
        with pytest.raises(ValueError):
            pa.forward(*args, kv_scale=scales, **kw)
        with pytest.raises(ValueError):
            pa.cascade_forward(*args, kv_scale=scales, common_prefix_len=16, **kw)


@pytest.mark.parametrize("kw,status", [(dict(ks=None), 1), (dict(ks=FAKE + 4), 1), (dict(ks=FAKE, hv=64), 2)])
def test_row_scaled_attention_arguments_are_checked_on_the_host(lib, kw, status):
    ext = pa.make_ext(num_seqs=2, num_tokens=9, max_blocks_per_seq=3, num_blocks=8, max_query_len=8,
                      max_seq_len=40, workspace=FAKE, workspace_bytes=1 << 30, head_size_v=kw.get("hv", 0))
    assert pa.pattn_varlen_fwd(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, 4, 2, 64, 16, 0, 1,
                               pa.KV_FP8_E4M3_ROW, kw["ks"], ext, lib=lib) == status
    if "hv" not in kw:
        assert pa.pattn_decode_fwd_static(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, 4, 2, 64, 16, 0, 1,
                                          pa.KV_FP8_E4M3_ROW, kw["ks"], 2, 2, 3, 8, 40, 0, 0, lib=lib) == status


@pytest.mark.parametrize("hq,hkv,bs,splits", [(5, 2, 16, 0), (4, 2, 0, 0), (4, 0, 16, 0), (4, 2, 16, -1)])
def test_workspace_free_decode_of_row_scales_refuses_what_it_refuses_of_other_caches(lib, hq, hkv, bs, splits):
    def call(kind):
        return pa.pattn_decode_fwd_static(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, hq, hkv, 64, bs, 0, 1,
                                          kind, FAKE if kind else None, 2, 2, 3, 8, 40, splits, 0, lib=lib)
    assert call(pa.KV_BF16) != 0
    assert call(pa.KV_FP8_E4M3_ROW) == call(pa.KV_BF16)


def _rope_tensors(**kw):
    T, H, Hkv, D, NB = 4, 4, 2, 64, 3
    t = dict(q=torch.zeros(T, H, D).bfloat16(), key=torch.zeros(T, Hkv, D).bfloat16(),
             value=torch.zeros(T, Hkv, D).bfloat16(), kv_cache=torch.zeros(2, NB, 16, Hkv, D).bfloat16(),
             slot_mapping=torch.arange(T), positions=torch.arange(T), cos_sin=torch.zeros(8, 64))
    t.update(kw)
    return t


@pytest.mark.parametrize("status", [torch.zeros(1, dtype=torch.int32, device="meta"),
                                    torch.zeros(1, dtype=torch.int64), torch.zeros(1),
                                    torch.zeros(0, dtype=torch.int32)])
def test_a_status_word_elsewhere_or_of_another_type_is_refused(lib, status):
    t = _rope_tensors()
    with pytest.raises(ValueError, match="device_status"):
        pa.rope_and_cache(**t, block_size=16, device_status=status)
    with pytest.raises(ValueError, match="device_status"):
        pa.reshape_and_cache(t["key"], t["value"], torch.zeros(2, 3, 16, 2, 64, dtype=torch.uint8),
                             t["slot_mapping"], block_size=16, kv_dtype=pa.KV_FP8_E4M3_ROW,
                             kv_scale=torch.zeros(pa.row_scales_shape(3, 16, 2)), device_status=status)
    with pytest.raises(ValueError, match="device_status"):
        pa.gather_cache(t["kv_cache"], torch.zeros(1, 2, dtype=torch.int32),
                        torch.tensor([0, 4], dtype=torch.int32), num_rows=4, block_size=16,
                        device_status=status)


def test_positions_without_an_axis_are_refused(lib):
    with pytest.raises(ValueError, match="positions"):
        pa.rope_and_cache(**_rope_tensors(positions=torch.zeros(0, 4, dtype=torch.int64)), block_size=16)


def test_read_back_of_half_a_cache_is_refused(lib):
    with pytest.raises(ValueError, match="kv_cache"):
        pa.gather_cache(torch.zeros(1, 3, 16, 2, 64).bfloat16(), torch.zeros(1, 2, dtype=torch.int32),
                        torch.tensor([0, 4], dtype=torch.int32), num_rows=4, block_size=16)


def test_read_back_of_misaligned_row_scales_is_refused(lib):
    assert lib.pattn_gather_cache(FAKE, FAKE, None, FAKE, FAKE, FAKE, 1, 0, 2, 3, 2, 64, 16,
                                  pa.KV_FP8_E4M3_ROW, FAKE + 4, None, None) == 1
