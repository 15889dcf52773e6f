"""Host-side checks of the latent operators (no GPU): the argument structs' layouts,
refusals before any CUDA call, the binding's own checks, and the definitions that
the GPU tests hold the kernels to."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
from latent_ref import attend, bound, cos_sin_table, normed, turned
from paged_varlen_attention_attn_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # 256-aligned and never dereferenced by these calls
STRUCTS = {"pattn_latent_rope_t": pa.LatentRopeArgs, "pattn_latent_t": pa.LatentArgs,
           "pattn_latent_expanded_t": pa.LatentExpandedArgs}


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load()


@pytest.mark.parametrize("name", sorted(STRUCTS))
def test_struct_layout_matches_c(tmp_path, name):
    cls = STRUCTS[name]
    names = [f[0] for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "pattn.h"\nint main(void) {\n' + "".join(
        f'printf("%zu\\n", offsetof({name}, {n}));\n' for n in names) +
        f'printf("%zu\\n", sizeof({name}));\nreturn 0; }}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(cls, n).offset for n in names] + [ctypes.sizeof(cls)]


def _call(fn, cls, base, kw):
    a = cls()
    a.struct_size = ctypes.sizeof(a)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return fn(ctypes.byref(a))


ROPE = dict(q=FAKE, q_out=FAKE, latent=FAKE, k_rope=FAKE, q_stride=1024, q_head_stride=64,
            q_out_stride=1024, q_out_head_stride=64, latent_stride=576, k_rope_stride=576,
            cos_sin=FAKE, positions=FAKE, kv_cache=FAKE, slot_mapping=FAKE, norm_eps=1e-6,
            num_tokens=0, num_heads=16, latent_size=512, rope_size=64, max_position=10,
            block_size=16, num_blocks=4)


@pytest.mark.parametrize("kw,status", [
    ({}, 0),                                       # (no tokens: nothing is done)
    (dict(struct_size=8), 1), (dict(latent=0), 1), (dict(kv_cache=0), 1), (dict(slot_mapping=0), 1),
    (dict(q_out=0), 1), (dict(q=0), 1), (dict(q=0, q_out=0), 0),
    (dict(latent_size=96), 2), (dict(latent_size=640), 2), (dict(latent_size=0), 1),
    (dict(rope_size=24), 2), (dict(rope_size=80), 2), (dict(block_size=24), 1),
    (dict(kv_dtype=pa.KV_FP8_E4M3), 2), (dict(interleaved=2), 1), (dict(num_tokens=-1), 1),
    (dict(cos_sin=0), 1), (dict(max_position=0), 1), (dict(positions=0, cos_sin=0), 0),
    (dict(latent_stride=580), 1), (dict(q_stride=-8), 1), (dict(latent=FAKE + 8), 1),
    (dict(latent_norm=FAKE, norm_eps=-1.0), 1), (dict(latent_norm=FAKE, norm_eps=math.nan), 1),
    (dict(num_tokens=2, q_out_head_stride=32), 1),        # heads that reach into each other
    (dict(num_tokens=2, q_out_stride=512), 1),            # and tokens
    (dict(num_tokens=2, row_out=FAKE, row_out_stride=512), 1),
])
def test_write_arguments_are_refused_on_the_host(lib, kw, status):
    assert _call(lib.pattn_latent_rope_and_cache, pa.LatentRopeArgs, ROPE, kw) == status


ATTEND = dict(q=FAKE, kv_cache=FAKE, out=FAKE, block_table=FAKE, seq_lens=FAKE, query_start_loc=FAKE,
              workspace=FAKE, workspace_bytes=1 << 40, scale=0.1, causal=1, num_seqs=0, num_tokens=0,
              num_heads=16, latent_size=512, rope_size=64, block_size=16, max_blocks_per_seq=4,
              num_blocks=9, max_query_len=1)


@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(struct_size=8), 1), (dict(q=0), 1), (dict(out=0), 1), (dict(workspace=0), 1),
    (dict(workspace=FAKE + 16), 1), (dict(workspace_bytes=1000), 3), (dict(q=FAKE + 8), 1),
    (dict(scale=-1.0), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1), (dict(causal=2), 1),
    (dict(num_heads=0), 1), (dict(latent_size=192), 2), (dict(rope_size=72), 2),
    (dict(block_size=8), 1), (dict(kv_dtype=pa.KV_FP8_E4M3_ROW), 2), (dict(max_query_len=-1), 1),
    (dict(num_tokens=1 << 24, num_heads=128), 2), (dict(num_blocks=1 << 28), 2),
    (dict(num_seqs=1, num_tokens=1, num_blocks=0), 1),
])
def test_absorbed_arguments_are_refused_on_the_host(lib, kw, status):
    assert _call(lib.pattn_latent_fwd, pa.LatentArgs, ATTEND, kw) == status


EXPANDED = dict(q=FAKE, k_nope=FAKE, k_rope=FAKE, value=FAKE, out=FAKE, q_stride=768, q_head_stride=192,
                k_stride=1024, k_head_stride=256, k_rope_stride=64, v_stride=1024, v_head_stride=256,
                query_start_loc=FAKE, key_start_loc=FAKE, workspace=FAKE, workspace_bytes=1 << 40,
                scale=0.1, causal=1, num_seqs=0, num_tokens=0, num_keys=0, num_heads=4, nope_size=128,
                rope_size=64, value_size=128)


@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(struct_size=8), 1), (dict(value=0), 1), (dict(nope_size=96, value_size=96), 2),
    (dict(value_size=64), 2), (dict(rope_size=8), 2), (dict(rope_size=0), 1),
    (dict(kv_dtype=pa.KV_FP8_E4M3), 2), (dict(k_stride=0), 1), (dict(v_head_stride=100), 1),
    (dict(q_stride=-768), 1), (dict(scale=-0.5), 1), (dict(causal=-1), 1), (dict(num_keys=-1), 1),
    (dict(workspace_bytes=0), 3), (dict(k_rope=FAKE + 2), 1), (dict(num_heads=0), 1),
])
def test_expanded_arguments_are_refused_on_the_host(lib, kw, status):
    assert _call(lib.pattn_latent_expanded_fwd, pa.LatentExpandedArgs, EXPANDED, kw) == status


def test_read_back_arguments_are_refused_on_the_host(lib):
    def call(**kw):
        a = dict(cache=FAKE, bt=FAKE, ks=None, osl=FAKE, lat=FAKE, rope=FAKE, B=1, rows=0, mbps=2, NB=4,
                 dc=512, dr=64, bs=16, kind=0)
        a.update(kw)
        return lib.pattn_gather_latent(a["cache"], a["bt"], a["ks"], a["osl"], a["lat"], a["rope"],
                                       a["B"], a["rows"], a["mbps"], a["NB"], a["dc"], a["dr"],
                                       a["bs"], a["kind"], None, None)
    assert call() == 0
    for kw, status in ((dict(cache=None), 1), (dict(rope=None), 1), (dict(B=-1), 1), (dict(rows=-2), 1),
                       (dict(dc=500), 2), (dict(dr=100), 2), (dict(bs=20), 1), (dict(kind=1), 2),
                       (dict(lat=FAKE + 4), 1)):
        assert call(**kw) == status, kw


def test_workspace_sizes(lib):
    assert lib.pattn_latent_workspace_bytes(64, 16, 512) > 0
    for bad in ((-1, 16, 512), (1, 0, 512), (1, 16, 500), (1, 16, 640)):
        assert lib.pattn_latent_workspace_bytes(*bad) == 0
    small, large = (lib.pattn_latent_expanded_workspace_bytes(4, t) for t in (10, 100000))
    assert 0 < small < large
    assert lib.pattn_latent_expanded_workspace_bytes(-1, 5) == 0


# ------------------------------------------------------ the binding's own checks

def _write(**kw):
    bf = torch.bfloat16
    a = dict(q=torch.zeros(3, 2, 32, dtype=bf), latent=torch.zeros(3, 128, dtype=bf),
             k_rope=torch.zeros(3, 32, dtype=bf), kv_cache=torch.zeros(2, 16, 160, dtype=bf),
             slot_mapping=torch.zeros(3, dtype=torch.int64), positions=torch.zeros(3, dtype=torch.int64),
             cos_sin=torch.zeros(9, 32))
    more = {k: kw.pop(k) for k in list(kw) if k not in a}
    a.update(kw)
    return pa.latent_rope_and_cache(*a.values(), block_size=16, **more)


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(3, 2, 16, dtype=torch.bfloat16)), dict(q=torch.zeros(2, 2, 32, dtype=torch.bfloat16)),
    dict(q=torch.zeros(3, 2, 32)), dict(latent=torch.zeros(3, 144, dtype=torch.bfloat16)),
    dict(k_rope=torch.zeros(2, 32, dtype=torch.bfloat16)),
    dict(kv_cache=torch.zeros(2, 32, 160, dtype=torch.bfloat16)),
    dict(kv_cache=torch.zeros(2, 16, 320, dtype=torch.bfloat16)[..., ::2]),
    dict(slot_mapping=torch.zeros(3, dtype=torch.int32)), dict(positions=torch.zeros(4, dtype=torch.int64)),
    dict(cos_sin=None), dict(cos_sin=torch.zeros(9, 16)), dict(cos_sin=torch.zeros(9, 32).double()),
    dict(latent_norm=torch.zeros(64, dtype=torch.bfloat16)),
    dict(q_out=torch.zeros(3, 1, 32, dtype=torch.bfloat16)), dict(q=None, q_out=torch.zeros(3, 2, 32)),
    dict(row_out=torch.zeros(3, 128, dtype=torch.bfloat16)),
    dict(device_status=torch.zeros(1)),
    dict(q=torch.zeros(3, 2, 64, dtype=torch.bfloat16)[..., ::2]),
])
def test_write_tensors_are_refused(kw):
    with pytest.raises(ValueError):
        _write(**kw)


def test_other_caches_are_refused():
    for kind in (pa.KV_FP8_E4M3, pa.KV_FP8_E4M3_ROW, 9):
        with pytest.raises(pa.PattnError):
            _write(kv_dtype=kind)


def _absorbed(**kw):
    bf, i32 = torch.bfloat16, torch.int32
    a = dict(q=torch.zeros(3, 2, 160, dtype=bf), kv_cache=torch.zeros(4, 16, 160, dtype=bf),
             block_table=torch.zeros(2, 2, dtype=i32), seq_lens=torch.zeros(2, dtype=i32),
             query_start_loc=torch.zeros(3, dtype=i32))
    out = kw.pop("out", None)
    a.update(kw)
    return pa.latent_forward(*a.values(), scale=1.0, latent_size=128, block_size=16, max_query_len=1,
                             out=out)


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(3, 2, 128, dtype=torch.bfloat16)), dict(q=torch.zeros(3, 2, 160)),
    dict(q=torch.zeros(2, 3, 160, dtype=torch.bfloat16).transpose(0, 1)),
    dict(seq_lens=torch.zeros(3, dtype=torch.int32)), dict(seq_lens=torch.zeros(2, dtype=torch.int64)),
    dict(query_start_loc=torch.zeros(2, dtype=torch.int32)),
    dict(block_table=torch.zeros(2, 4, dtype=torch.int32)[:, ::2]),
    dict(out=torch.zeros(3, 2, 160, dtype=torch.bfloat16)),
])
def test_absorbed_tensors_are_refused(kw):
    with pytest.raises(ValueError):
        _absorbed(**kw)


def _expanded(**kw):
    bf, i32 = torch.bfloat16, torch.int32
    a = dict(q=torch.zeros(3, 2, 96, dtype=bf), k_nope=torch.zeros(5, 2, 64, dtype=bf),
             k_rope=torch.zeros(5, 32, dtype=bf), value=torch.zeros(5, 2, 64, dtype=bf),
             query_start_loc=torch.zeros(3, dtype=i32), key_start_loc=torch.zeros(3, dtype=i32))
    out = kw.pop("out", None)
    a.update(kw)
    return pa.latent_expanded_forward(*a.values(), scale=1.0, out=out)


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(3, 2, 64, dtype=torch.bfloat16)), dict(k_nope=torch.zeros(5, 3, 64, dtype=torch.bfloat16)),
    dict(k_rope=torch.zeros(4, 32, dtype=torch.bfloat16)), dict(value=torch.zeros(4, 2, 64, dtype=torch.bfloat16)),
    dict(value=torch.zeros(5, 2, 64)), dict(key_start_loc=torch.zeros(2, dtype=torch.int32)),
    dict(query_start_loc=torch.zeros(3, dtype=torch.int64)),
    dict(out=torch.zeros(3, 2, 96, dtype=torch.bfloat16)),
    dict(k_nope=torch.zeros(5, 2, 128, dtype=torch.bfloat16)[..., ::2]),
])
def test_expanded_tensors_are_refused(kw):
    with pytest.raises(ValueError):
        _expanded(**kw)


# ------------------------------------------------------------------ the definitions

def test_definition_of_the_attention():
    """Against sums written out: shared keys, a causal chunk at the end of its keys."""
    g = torch.Generator().manual_seed(1)
    q, rows = torch.randn(2, 3, 6, generator=g), torch.randn(5, 1, 6, generator=g)
    out, weighted, size = attend(q, rows, rows[..., :4], 0.3, 1)
    for i in range(2):
        for h in range(3):
            seen = 5 - 2 + i + 1
            w = [math.exp(0.3 * sum(q[i, h, e].item() * rows[k, 0, e].item() for e in range(6)))
                 for k in range(seen)]
            for e in range(4):
                want = sum(x * rows[k, 0, e].item() for k, x in enumerate(w)) / sum(w)
                assert abs(out[i, h, e].item() - want) < 1e-12
                assert weighted[i, h, e] >= abs(want) - 1e-12
    assert size.shape == (2, 3) and (size > 0).all()
    assert (bound(out, weighted, size, 0.3, 6, 5, 3.0, torch.bfloat16) >= out.abs() * 2.0 ** -8).all()


def test_absorbed_and_expanded_forms_agree():
    """q_n . (W_k c) = (W_k^T q_n) . c, and sum p (W_v c) = W_v sum p c."""
    g = torch.Generator().manual_seed(2)
    c, kr = torch.randn(9, 8, generator=g).double(), torch.randn(9, 4, generator=g).double()
    wk, wv = torch.randn(3, 5, 8, generator=g).double(), torch.randn(3, 5, 8, generator=g).double()
    qn, qr = torch.randn(4, 3, 5, generator=g).double(), torch.randn(4, 3, 4, generator=g).double()
    up = [torch.einsum("hde,ke->khd", w, c) for w in (wk, wv)]
    keys = torch.cat([up[0], kr[:, None].expand(9, 3, 4)], -1)
    expanded = attend(torch.cat([qn, qr], -1), keys, up[1], 0.2, 1)[0]
    rows = torch.cat([c, kr], -1)[:, None]
    q = torch.cat([torch.einsum("thd,hde->the", qn, wk), qr], -1)
    absorbed = attend(q, rows, rows[..., :8], 0.2, 1)[0]
    assert torch.allclose(expanded, torch.einsum("the,hde->thd", absorbed, wv))


@pytest.mark.parametrize("interleaved", [False, True])
def test_definition_of_the_rotation(interleaved):
    table, angle = cos_sin_table(30, 8)
    x = torch.randn(5, 2, 8, generator=torch.Generator().manual_seed(3)).double()
    pos = torch.tensor([0, 1, 7, 29, 3])
    got = turned(x, table, pos, interleaved)
    first, second = (slice(0, 8, 2), slice(1, 8, 2)) if interleaved else (slice(0, 4), slice(4, 8))
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones(()).double(), angle[pos])[:, None]
    assert torch.allclose(got[..., first], z.real, atol=1e-6)
    assert torch.allclose(got[..., second], z.imag, atol=1e-6)
    w = torch.randn(8, generator=torch.Generator().manual_seed(4))
    y = normed(x[:, 0], w, 0.0)
    assert torch.allclose((y / w.double()).square().mean(-1), torch.ones(5).double())
