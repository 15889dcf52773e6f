"""Calls from several host threads at once: none may refuse or disturb another's."""
import ctypes
import threading

import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
import row_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_varlen_attention_attn_gb300 import _build
    _build.build()
    pa.load()


def test_streamed_rotary_calls_of_two_shapes_from_two_threads():
    """Two models' calls run the same kernel with rings of different sizes: each
    thread's launches are accepted whatever the other's are."""
    lib = pa.load()
    table, _ = R.cos_sin_table(4096, 128)
    table = table.to(DEV)
    refused, keep, want = [[], []], [], []

    def prepared(T, H, Hkv, seed):
        g = torch.Generator().manual_seed(seed)
        NB = T // 16 + 2
        qkv = torch.randn(T, H + 2 * Hkv, 128, generator=g).bfloat16().to(DEV)
        q, k, v = qkv.split([H, Hkv, Hkv], 1)
        pos = torch.arange(T, device=DEV)
        cache = torch.zeros(2, NB, 16, Hkv, 128, dtype=torch.uint8, device=DEV)
        scales = torch.zeros(pa.row_scales_shape(NB, 16, Hkv), device=DEV)
        out = pa.rope_and_cache(q, k, v, cache, pos, pos, table, block_size=16,
                                kv_dtype=pa.KV_FP8_E4M3_ROW, kv_scale=scales)
        again = torch.zeros_like(out)
        stream = torch.cuda.Stream(DEV)
        stream.wait_stream(torch.cuda.current_stream())
        a = pa.RopeArgs(struct_size=ctypes.sizeof(pa.RopeArgs), q=q.data_ptr(), q_out=again.data_ptr(),
                        key=k.data_ptr(), value=v.data_ptr(), q_stride=q.stride(0),
                        q_out_stride=H * 128, key_stride=k.stride(0), value_stride=v.stride(0),
                        cos_sin=table.data_ptr(), positions=pos.data_ptr(), kv_cache=cache.data_ptr(),
                        row_scales=scales.data_ptr(), slot_mapping=pos.data_ptr(),
                        stream=stream.cuda_stream, num_tokens=T, num_heads=H, num_kv_heads=Hkv,
                        head_size=128, rot_dim=128, num_axes=1, max_position=4096,
                        kv_dtype=pa.KV_FP8_E4M3_ROW, block_size=16, num_blocks=NB)
        keep.append((qkv, pos, cache, scales, stream, again))
        want.append((out, again))
        return a

    args = [prepared(1500, 64, 8, 1), prepared(2500, 32, 8, 2)]
    torch.cuda.synchronize()
    start = threading.Barrier(2)

    def work(i):
        torch.cuda.set_device(0)
        start.wait()
        for _ in range(6000):
            st = lib.pattn_rope_and_cache(ctypes.byref(args[i]))
            if st != 0:
                refused[i].append(st)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused[0] and not refused[1], (len(refused[0]), len(refused[1]))
    for a, b in want:
        assert torch.equal(a, b)


def test_attention_calls_of_two_threads_on_one_stream():
    """Default workspaces: partitioned decodes and chunks, all on one stream."""
    from test_row_scaled_attention_gpu import Case
    cases = [Case(400, [(1, 3000), (1, 2500)], 8, 2, 128, 16),
             Case(401, [(1, 2800), (140, 300), (1, 900)], 8, 2, 128, 16)]
    calls = [(c.args(), c.kw(num_splits=8)) for c in cases]
    want = [pa.forward(*a, **kw) for a, kw in calls]
    outs = [[torch.empty_like(w) for _ in range(200)] for w in want]
    torch.cuda.synchronize()
    start = threading.Barrier(2)

    def work(i):
        start.wait()
        for out in outs[i]:
            pa.forward(*calls[i][0], out=out, **calls[i][1])

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for c, w, got in zip(cases, want, outs):
        c.check(w)
        assert all(torch.equal(x, w) for x in got)
