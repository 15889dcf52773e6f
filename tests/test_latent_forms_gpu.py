"""The latent operators as a program uses them: a layer's run of them, streams, graphs,
host threads, a cache whose offsets pass 32 bits."""
import threading

import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
from latent_ref import Dense, Paged, attend, cos_sin_table
from test_call_streams_gpu import owner, side_stream

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_varlen_attention_attn_gb300 import _build
    _build.build()
    pa.load()


def test_a_layer_in_both_forms():
    """Two chunks on cached context and three single tokens: projections, the write,
    the absorbed form over the cache, and the expanded form over rows read back."""
    H, dc, dn, dr, bs = 16, 512, 128, 64, 16
    g = torch.Generator().manual_seed(1)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).bfloat16().to(DEV)

    ctx, new = [100, 37, 300, 64, 1], [20, 33, 1, 1, 1]
    lens = [a + b for a, b in zip(ctx, new)]
    need = [(s + bs - 1) // bs for s in lens]
    perm = torch.randperm(sum(need) + 2, generator=g).int()
    table = torch.zeros(5, max(need), dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    cache = torch.full((sum(need) + 2, bs, dc + dr), float("nan"), dtype=torch.bfloat16, device=DEV)
    cos_sin = cos_sin_table(512, dr)[0].to(DEV)
    norm = (1 + 0.1 * torch.randn(dc, generator=g)).bfloat16().to(DEV)
    w_k, w_v = randn(H, dn, dc, scale=dc ** -0.5), randn(H, dn, dc, scale=dc ** -0.5)

    def slots(r, a, b):
        key = torch.arange(a, b)
        return (table[r, key // bs].long() * bs + key % bs)

    def step(spans, q):
        """Writes the tokens of spans [(request, first, last)]."""
        T = sum(b - a for _, a, b in spans)
        down = randn(T, dc + dr)
        pos = torch.cat([torch.arange(a, b) for _, a, b in spans]).to(DEV)
        slot = torch.cat([slots(*s) for s in spans]).to(DEV)
        rows = torch.empty(T, dc + dr, dtype=torch.bfloat16, device=DEV)
        pa.latent_rope_and_cache(None if q is None else q[..., dn:], down[:, :dc], down[:, dc:], cache,
                                 slot, pos, cos_sin, block_size=bs, interleaved=True, latent_norm=norm,
                                 q_out=None if q is None else q[..., dn:], row_out=rows)
        return rows

    step([(r, 0, n) for r, n in enumerate(ctx)], None)
    T = sum(new)
    q = randn(T, H, dn + dr)
    step([(r, c, c + n) for r, (c, n) in enumerate(zip(ctx, new))], q)  # (q turned in place)
    table = table.to(DEV)
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    starts = torch.tensor([0] + new).cumsum(0).int().to(DEV)
    key_starts = torch.tensor([0] + lens).cumsum(0).int().to(DEV)
    scale = (dn + dr) ** -0.5
    absorbed_q = torch.cat([torch.einsum("thd,hde->the", q[..., :dn].float(), w_k.float()).bfloat16(),
                            q[..., dn:]], -1)
    latent = pa.latent_forward(absorbed_q, cache, table, seq_lens, starts, scale=scale, latent_size=dc,
                               block_size=bs, max_query_len=max(new))
    absorbed = torch.einsum("the,hde->thd", latent.float(), w_v.float())
    c, kr = pa.gather_latent(cache, table, key_starts, num_rows=sum(lens), latent_size=dc, block_size=bs)
    up = torch.cat([torch.einsum("ke,hde->khd", c.float(), w.float()) for w in (w_k, w_v)], -1).bfloat16()
    expanded = pa.latent_expanded_forward(q, up[..., :dn], kr, up[..., dn:], starts, key_starts,
                                          scale=scale).float()
    # both against the formula on the cached rows; each rounds its weights, its
    # operands and its result to bf16, whose half step is 2^-8
    t = k = 0
    for n, s in zip(new, lens):
        keys = torch.cat([torch.einsum("ke,hde->khd", c[k:k + s].double(), w_k.double()),
                          kr[k:k + s, None].double().expand(s, H, dr)], -1)
        vals = torch.einsum("ke,hde->khd", c[k:k + s].double(), w_v.double())
        ref, weighted, size = attend(q[t:t + n], keys, vals, scale, 1)
        # an operand rounded by 2^-8 moves a score by 2^-8 of the sum of magnitudes at most
        slack = 2.0 ** -8 * (4 * weighted + ref.abs()) + 2 * 2.0 ** -8 * scale * size[..., None] * weighted
        assert ((expanded[t:t + n].double() - ref).abs() <= slack).all()
        # (and the absorbed form's output passes through w_v: 512 rounded terms)
        through = torch.einsum("the,hde->thd", latent[t:t + n].double().abs() + 0.1, w_v.double().abs())
        q_size = torch.einsum("the,ke->thk", absorbed_q[t:t + n].double().abs(),
                              torch.cat([c, kr], -1)[k:k + s].double().abs()).amax(-1)
        slack = 2.0 ** -8 * 2 * through + 2 * 2.0 ** -8 * scale * q_size[..., None] * through
        assert ((absorbed[t:t + n].double() - ref).abs() <= slack).all()
        t, k = t + n, k + s


def _absorbed():
    c = Paged(1, [(1, 700), (5, 300), (1, 64), (1, 3000)], H=16, dc=256, dr=64, bs=16, device=DEV)
    return c, lambda **kw: c.run(**kw)


def _expanded():
    c = Dense(2, [(70, 200), (300, 300), (1, 40)], H=4, dn=128, dr=64, device=DEV)
    return c, lambda **kw: c.run(**kw)


def _expanded_many():
    c = Dense(3, [(300, 300)] * 30, H=8, dn=64, dr=32, device=DEV)
    return c, lambda **kw: c.run(**kw)


CALLS = [_absorbed, _expanded, _expanded_many]


@pytest.mark.parametrize("make", CALLS)
def test_outputs_belong_to_the_stream(make):
    _, call = make()
    want = call()
    s = side_stream()
    got = call(stream=s)
    assert owner(got.data_ptr()) == s.cuda_stream
    s.synchronize()
    assert torch.equal(got, want)


def test_cache_operators_on_a_stream():
    s = side_stream()
    cache = torch.randn(8, 16, 160, device=DEV).bfloat16()
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(1, 8)
    starts = torch.tensor([0, 100], dtype=torch.int32, device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    lat, rope = pa.gather_latent(cache, table, starts, num_rows=100, latent_size=128, block_size=16, stream=s)
    assert owner(lat.data_ptr()) == owner(rope.data_ptr()) == s.cuda_stream
    q = torch.randn(4, 3, 32, device=DEV).bfloat16()
    slots = torch.arange(4, device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    out = pa.latent_rope_and_cache(q, lat[:4], rope[:4], cache, slots, None, None, block_size=16, stream=s)
    assert owner(out.data_ptr()) == s.cuda_stream
    s.synchronize()
    assert torch.equal(out, q) and torch.equal(torch.cat([lat, rope], 1), cache.view(-1, 160)[:100])


@pytest.mark.parametrize("make", CALLS)
def test_captured_and_replayed_on_other_inputs(make):
    """Two graphs with a workspace each, replayed at once on two streams."""
    c, call = make()
    graphs = []
    for k in range(2):
        ws, s = pa.Workspace(), side_stream()
        out = torch.empty_like(call())
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            call(out=out, workspace=ws)
        graphs.append((graph, s, out, ws))
    c.q.mul_(-0.5)
    want = call()
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, s, out, _ in graphs:
            with torch.cuda.stream(s):
                out.fill_(float("nan"))
                graph.replay()
    torch.cuda.synchronize()
    for _, _, out, _ in graphs:
        assert torch.equal(out, want)


@pytest.mark.parametrize("make", CALLS)
def test_replay_after_a_larger_call_took_another_workspace(make):
    pa.release_workspaces()
    _, call = make()
    want = call()
    s = side_stream()
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        call(out=out)
    with torch.cuda.stream(s):
        Dense(5, [(1, 1)] * 50000, H=1, dn=64, dr=16, device=DEV).run()
        Paged(6, [(1, 100)], H=64, dc=512, dr=64, bs=16, device=DEV).run()
        junk = [torch.full((1 << 22,), 90, dtype=torch.uint8, device=DEV) for _ in range(12)]
        out.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all((x == 90).all() for x in junk)
    pa.release_workspaces()


def test_calls_back_to_back_wait_for_each_other():
    """Each call reads what the call before wrote, or writes what it read, with nothing
    between them; the kernels may be launched while the one before still runs."""
    T, H, dc, dr, bs = 2048, 16, 512, 64, 16
    c = Paged(8, [(1, 2048)] * 4, H=H, dc=dc, dr=dr, bs=bs, device=DEV)
    slots = (c.table[:, :128].long().repeat_interleave(bs, 1) * bs + torch.arange(2048, device=DEV) % bs).flatten()
    starts = torch.arange(0, 4 * T + 1, T, dtype=torch.int32, device=DEV)
    size = dict(latent_size=dc, block_size=bs)
    g = torch.Generator().manual_seed(2)
    rows = [torch.randn(4 * T, dc + dr, generator=g).bfloat16().to(DEV) for _ in range(2)]

    def steps(wait):
        got = []
        for i in range(12):
            latent, key = rows[i % 2].split([dc, dr], 1)
            pa.latent_rope_and_cache(None, latent, key, c.cache, slots, None, None, block_size=bs)
            wait()
            out = c.run()
            wait()
            back = pa.gather_latent(c.cache, c.table, starts, num_rows=4 * T, **size)
            wait()
            # the rows read back, turned over, overwrite the cache that both have read
            pa.latent_rope_and_cache(None, back[0], back[1], c.cache, slots.flip(0), None, None, block_size=bs)
            wait()
            got += [out, c.run(), *back]
            wait()
        torch.cuda.synchronize()
        return got

    for x, y in zip(steps(torch.cuda.synchronize), steps(lambda: None)):
        assert torch.equal(x, y)


def test_calls_from_two_threads():
    calls = [make()[1] for make in CALLS]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    failed = []

    def work(order):
        try:
            for _ in range(15):
                for i in order:
                    if not torch.equal(calls[i](), want[i]):
                        failed.append(i)
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=(o,)) for o in ([0, 1, 2], [2, 1, 0])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_offsets_that_pass_32_bits():
    """A pool of 4.4 GB; the rows used lie at its end."""
    nb, bs, dc, dr = 60000, 64, 512, 64
    cache = torch.empty(nb, bs, dc + dr, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(8)
    T, H = 200, 16
    down = torch.randn(T, dc + dr, generator=g).bfloat16().to(DEV)
    slots = torch.arange(nb * bs - 4 * bs, nb * bs - 4 * bs + T, device=DEV)
    pa.latent_rope_and_cache(None, down[:, :dc], down[:, dc:], cache, slots, None, None, block_size=bs)
    assert torch.equal(cache.view(-1, dc + dr)[-4 * bs:][:T], down)
    table = torch.arange(nb - 4, nb, dtype=torch.int32, device=DEV).view(1, 4)
    lat, rope = pa.gather_latent(cache, table, torch.tensor([0, T], dtype=torch.int32, device=DEV),
                                 num_rows=T, latent_size=dc, block_size=bs)
    assert torch.equal(torch.cat([lat, rope], 1), down)
    c = Paged(9, [(1, T)], H=H, dc=dc, dr=dr, bs=bs, device=DEV)
    c.cache, c.table = cache, table
    c.check(c.run())


def test_a_padded_batch():
    """Requests without tokens, block-table rows wider than any request, a batch whose
    last requests are empty, rows behind the last request."""
    lens = [(0, 50), (1, 33), (0, 0), (1, 200), (0, 0)]
    c = Paged(10, lens, H=16, dc=512, dr=64, bs=16, device=DEV, poison=True)
    c.q = torch.cat([c.q, torch.full_like(c.q, float("nan"))])
    out = torch.full((4, 16, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    c.run(out=out)
    assert (out[2:] == 7).all()
    c.q = c.q[:2]
    c.check(out[:2])
    d = Dense(11, [(0, 5), (40, 60), (0, 0), (0, 0)], H=3, dn=128, dr=64, device=DEV)
    d.check(d.run())


def test_non_finite_values_behind_a_request_stay_there():
    """Keys of the next request and of the tail of the last tile hold NaN."""
    d = Dense(12, [(30, 100), (20, 70), (64, 90)], H=4, dn=128, dr=64, device=DEV)
    clean = d.run()
    d.up[100:170] = float("nan")
    d.k_rope[100:170] = float("inf")
    got = d.run()
    assert torch.equal(got[:30], clean[:30]) and torch.equal(got[50:], clean[50:])
    assert not torch.isfinite(got[30:50].float()).any()
