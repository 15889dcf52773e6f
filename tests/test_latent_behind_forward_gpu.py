"""Latent operators right behind ``forward`` on a batch of prompts and single tokens,
whose two kernels overlap and whose last one has far less to do: on the default
workspace that both calls take, and on memory that ``forward`` still reads or writes.
Each against the same calls with a synchronisation between them."""
import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
from latent_ref import Dense, Paged
from test_call_streams_gpu import side_stream

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H, HKV, D, BS = 32, 8, 128, 16
DC, DR = 512, 64


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_varlen_attention_attn_gb300 import _build
    _build.build()
    pa.load()


class Mixed:
    """A chunk of 4096 tokens behind 4096 keys and six decodes of 40 keys."""

    def __init__(self):
        g = torch.Generator().manual_seed(1)
        reqs = [(4096, 8192)] + [(1, 40)] * 6
        width = 8192 // BS
        self.nb = width + 6 * 3
        perm = torch.randperm(self.nb, generator=g).int()
        table = torch.zeros(len(reqs), width, dtype=torch.int32)
        table[0] = perm[:width]
        table[1:, :3] = perm[width:].view(6, 3)
        T = sum(n for n, _ in reqs)
        self.master = [torch.randn(T, H, D, generator=g).bfloat16().to(DEV),
                       torch.randn(2, self.nb, BS, HKV, D, generator=g).bfloat16().to(DEV)]
        self.q, self.kv = (torch.empty_like(x) for x in self.master)
        self.out = torch.empty_like(self.q)
        self.args = [table.to(DEV), torch.tensor([s for _, s in reqs], dtype=torch.int32, device=DEV),
                     torch.tensor([0] + [n for n, _ in reqs], dtype=torch.int32).cumsum(0).int().to(DEV)]
        self.reset()

    def reset(self):
        self.q.copy_(self.master[0])
        self.kv.copy_(self.master[1])
        self.out.fill_(float("nan"))

    def run(self):
        return pa.forward(self.q, self.kv, *self.args, scale=D ** -0.5, num_heads=H, num_kv_heads=HKV,
                          head_size=D, block_size=BS, max_query_len=4096, max_seq_len=8192, out=self.out)

    def memory(self, which, *shape):
        """A tensor over the first bytes of one of forward's."""
        n = 1
        for x in shape:
            n *= x
        return getattr(self, which).view(-1)[:n].view(shape)


def _rows(n, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, DC + DR, generator=g).bfloat16().to(DEV).split([DC, DR], 1)


def absorbed(m):
    """On the workspace that forward's items lie in, many requests."""
    c = Paged(2, [(1, 1 + 13 * i % 700) for i in range(400)], H=16, dc=256, dr=64, bs=16, device=DEV)
    return lambda: [c.run()]


def absorbed_over_q(m):
    c = Paged(3, [(1, 900), (5, 300), (1, 64)], H=16, dc=DC, dr=DR, bs=16, device=DEV)
    out = m.memory("q", 7, 16, DC)
    return lambda: [c.run(out=out)]


def expanded(m):
    """With the list of its items in the workspace."""
    c = Dense(4, [(200 + 30 * i, 300 + 40 * i) for i in range(20)], H=16, dn=64, dr=32, device=DEV)
    return lambda: [c.run()]


def expanded_over_the_cache(m):
    c = Dense(5, [(100, 130), (20, 20)], H=8, dn=128, dr=64, device=DEV)
    out = m.memory("kv", 120, 8, 128)
    return lambda: [c.run(out=out)]


def write_over_the_cache(m):
    blocks = 1000
    cache = m.memory("kv", blocks, 16, DC + DR)
    latent, key = _rows(blocks * 16, 6)
    slots = torch.randperm(blocks * 16, generator=torch.Generator().manual_seed(7)).to(DEV)

    def call():
        pa.latent_rope_and_cache(None, latent, key, cache, slots, None, None, block_size=16)
        return [cache]
    return call


def read_back_over(which):
    def make(m):
        latent, key = _rows(64 * 16, 8)
        cache = torch.cat([latent, key], 1).view(64, 16, DC + DR)
        table = torch.randint(0, 64, (40, 30), generator=torch.Generator().manual_seed(9)).int().to(DEV)
        starts = torch.arange(0, 40 * 480 + 1, 480, dtype=torch.int32, device=DEV)
        lat = m.memory(which, 40 * 480, DC)

        def call():
            return list(pa.gather_latent(cache, table, starts, num_rows=40 * 480, latent_size=DC,
                                         block_size=16, latent_out=lat))
        return call
    make.__name__ = f"read_back_over_{which}"
    return make


OPS = [absorbed, absorbed_over_q, expanded, expanded_over_the_cache, write_over_the_cache,
       read_back_over("q"), read_back_over("out")]


@pytest.fixture(scope="module")
def mixed():
    return Mixed()


def _all(m, got):
    torch.cuda.synchronize()
    return [x.clone() for x in [m.q, m.kv, m.out, *got]]


def _same(got, want):
    return all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, want))


@pytest.mark.parametrize("make", OPS, ids=lambda f: f.__name__)
def test_a_latent_call_behind_a_mixed_batch(mixed, make):
    m = mixed
    call = make(m)
    m.reset()
    call()  # (workspaces and outputs that the timed calls would allocate)
    m.reset()
    torch.cuda.synchronize()
    m.run()
    torch.cuda.synchronize()
    want = _all(m, call())
    for _ in range(3):
        m.reset()
        torch.cuda.synchronize()
        m.run()
        got = _all(m, call())
        assert _same(got, want)


@pytest.mark.parametrize("make", OPS, ids=lambda f: f.__name__)
def test_captured_behind_a_mixed_batch(mixed, make):
    """In a graph a node waits for the nodes it depends on alone."""
    m = mixed
    call = make(m)
    s = side_stream()
    m.reset()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        m.run()
        torch.cuda.synchronize()
        want = _all(m, call())
    graph = torch.cuda.CUDAGraph()
    m.reset()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        m.run()
        got = call()
    for _ in range(3):
        m.reset()
        torch.cuda.synchronize()
        graph.replay()
        assert _same(_all(m, got), want)


def test_an_ordinary_kernel_captured_behind_a_mixed_batch(mixed):
    m = mixed
    s = side_stream()
    m.reset()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        m.run()
    torch.cuda.synchronize()
    want = m.out.clone()
    graph, copy = torch.cuda.CUDAGraph(), torch.empty_like(m.out)
    with torch.cuda.graph(graph, stream=s):
        m.run()
        torch.mul(m.out, 1, out=copy)
        m.kv.zero_()
    for _ in range(3):
        m.reset()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert _same([copy, m.out], [want, want])
        assert not m.kv.any()
