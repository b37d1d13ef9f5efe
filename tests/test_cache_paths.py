"""GPU tests of the paged 8-bit cache as a serving step runs it: layers, pages
and attention together, captured and replayed, on other streams, beside other
kernels of the library, and twice with the same bits."""
import math

import pytest
import torch

from gather_matmul_b200 import _lib, ops
from gather_matmul_b200.layers import AttentionInputs, CachedAttention
from test_base_ops import make
from test_cache_ops import BF16, F16, FP8, TYPES, Cache, Pool, check_attention, gen, ints, rows, starts_of, up

pytestmark = pytest.mark.gpu


class Model:
    """Layers of attention over one pool of pages."""

    def __init__(self, layers, hq, hk, dim, page, P, B, M, K=256, dtype=BF16, seed=0, max_tokens=256):
        g = gen(seed)
        self.hq, self.hk, self.dim, self.page, self.K, self.dtype, self.L, self.P = hq, hk, dim, page, K, dtype, layers, P
        N, S, r = (hq + 2 * hk) * dim, 3, 16
        self.cache = torch.full((layers, P, 2, hk, page, dim), math.nan, device="cuda").to(FP8)
        self.scale = torch.full((layers, P, 2, hk), math.nan, device="cuda")
        self.tables = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
        self.lengths, self.refs = ints([0] * B), ints([0] * P)
        self.work = ops.cache_workspace(P, dim)
        f, m = ops.rope_frequencies(dim)
        self.layers = []
        for i in range(layers):
            W, ws = torch.empty(N, K, dtype=FP8, device="cuda"), torch.empty(up(N, 128), up(K, 128), device="cuda")
            ops.quantize_fp8((0.1 * torch.randn(N, K, generator=g, device="cuda")).to(dtype), W, ws, block_rows=128)
            A = [(0.1 * torch.randn(S, r, K, generator=g, device="cuda")).to(dtype)]
            Bs = [(0.1 * torch.randn(S, h * dim, r, generator=g, device="cuda")).to(dtype) for h in (hq, hk, hk)]
            inputs = AttentionInputs(W, ws, A, Bs, hq, hk, dim, f, max_tokens=max_tokens, attn_scale=m)
            self.layers.append(CachedAttention(inputs, self.cache[i], self.scale[i], self.work))

    def extend(self):
        ops.pages_extend(self.tables, self.lengths, self.refs, self.page, self.work)

    def buffers(self, T):
        N = (self.hq + 2 * self.hk) * self.dim
        return [(torch.empty(T, N, dtype=self.dtype, device="cuda"), torch.empty(T, self.hq * self.dim, dtype=self.dtype, device="cuda"))
                for _ in range(self.L)]

    def run(self, x, idx, positions, buf, starts=None):
        for layer, (y, out) in zip(self.layers, buf):
            layer(x, idx, positions, self.tables, self.lengths, y, out, starts=starts)

    def view(self, i):
        """Layer i's cache as the reference takes it."""
        c = Cache.__new__(Cache)
        c.lens, c.H, c.dim, c.page, c.B = self.lengths.tolist(), self.hk, self.dim, self.page, len(self.lengths)
        c.cache, c.scale, c.tables, c.lengths, c.work = self.cache[i], self.scale[i], self.tables, self.lengths, self.work
        return c


@pytest.mark.parametrize("hq,hk,dim,page", [(8, 2, 64, 16), (6, 1, 128, 32), (4, 4, 80, 64)])
def test_prompts_tokens_branches_ends_and_moves(hq, hk, dim, page):
    B, g = 6, gen(1)
    m = Model(2, hq, hk, dim, page, P=60 * 16 // page + 8, B=B, M=20 * 16 // page + 2)
    pool = Pool(m.tables, m.lengths, m.refs, page)

    def step(news, seed):
        """New tokens of every sequence (0: none), through all layers, and the reference of each."""
        T = sum(news)
        m.lengths += ints(news)
        pool.n = [a + b for a, b in zip(pool.n, news)]
        assert pool.extend() == 0
        m.extend()
        pool.check(m.tables, m.lengths, m.refs)
        x = torch.randn(T, m.K, generator=g, device="cuda").to(m.dtype)
        idx = torch.randint(-1, 3, (T,), generator=g, device="cuda").to(torch.int32)
        pos = torch.cat([torch.arange(n - k, n, device="cuda") for n, k in zip(pool.n, news)])
        buf = m.buffers(T)
        m.run(x, idx, pos, buf, None if news == [1] * B else starts_of(news))
        for i, (y, out) in enumerate(buf):
            check_attention(m.view(i), y[:, :hq * dim], out, news)
        return buf
    step([37, 0, 5, 16, 0, 0], 1)                            # prompts
    step([1, 40, 1, 1, 0, 0], 2)                             # a prompt among single tokens
    src, dst = [0, 1], [4, 5]
    copies, missed = pool.fork(src, dst)
    assert missed == 0
    ops.pages_fork(m.tables, m.lengths, m.refs, ints(src), ints(dst), m.cache, m.scale, m.work)
    pool.check(m.tables, m.lengths, m.refs)
    a, b = step([1] * B, 3), None                            # branches go their own ways
    assert not torch.equal(a[1][1][0], a[1][1][4])
    pool.free([0, 2])
    ops.pages_free(m.tables, m.lengths, m.refs, ints([0, 2]), m.work)
    q = torch.randn(B, hq * dim, generator=g, device="cuda").to(m.dtype)

    def look():
        out = [torch.empty_like(q) for _ in range(m.L)]
        for i in range(m.L):
            ops.cache_attention(q, m.cache[i], m.scale[i], m.tables, m.lengths, out[i], m.work)
        return out
    before = look()
    moves, live = pool.compact()
    n = ints([0])
    ops.pages_compact(m.tables, m.refs, m.cache, m.scale, m.work, n_live=n)
    pool.check(m.tables, m.lengths, m.refs)
    assert int(n) == live and len(moves) > 0
    for a, b in zip(before, look()):
        assert torch.equal(a, b) and (a[0] == 0).all() and (a[2] == 0).all()
    step([3, 1, 21, 1, 1, 1], 4)                             # freed rows begin anew
    assert ops.check_errors(m.work) == _lib.LORA_OK


def test_a_captured_decode_step_replayed_as_lengths_grow():
    B = 5
    m, e = Model(2, 8, 2, 64, 16, 64, B, 12, seed=3), Model(2, 8, 2, 64, 16, 64, B, 12, seed=3)
    g = gen(4)
    xs = [torch.randn(B, m.K, generator=g, device="cuda").to(m.dtype) for _ in range(40)]
    idx = ints([-1, 0, 1, 2, -1])
    x, pos, one = torch.empty_like(xs[0]), torch.zeros(B, dtype=torch.int64, device="cuda"), ints([1, 1, 0, 1, 1])
    bufs = {id(m): m.buffers(B), id(e): e.buffers(B)}

    def step(mm):
        mm.lengths += one                                    # row 2 of the batch stays empty
        mm.extend()
        mm.run(x, idx, pos, bufs[id(mm)])
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    kept = m.lengths.clone(), m.tables.clone(), m.refs.clone()
    x.copy_(xs[0])
    with torch.cuda.stream(stream):
        step(m)
    torch.cuda.synchronize()
    for a, b in zip((m.lengths, m.tables, m.refs), kept):
        a.copy_(b)
    with torch.cuda.graph(graph, stream=stream):
        step(m)
    for i, xi in enumerate(xs):
        x.copy_(xi)
        pos.fill_(i)
        graph.replay()
        step(e)
        for (y, out), (ye, oute) in zip(bufs[id(m)], bufs[id(e)]):
            assert torch.equal(out, oute) and torch.equal(y, ye), i
    assert m.lengths.tolist() == [40, 40, 0, 40, 40] and torch.equal(m.tables, e.tables)
    assert (out[2] == 0).all() and torch.isfinite(out).all()
    assert ops.check_errors(m.work) == _lib.LORA_OK


@pytest.mark.parametrize("news", [None, [1, 300, 2, 90]], ids=["single", "chunks"])
@pytest.mark.parametrize("dtype", TYPES)
def test_the_same_bits_every_time_and_on_every_stream(news, dtype):
    c = Cache([9000, 300, 5000, 1111], 2, 128, 64, seed=5)
    q = rows(4 if news is None else sum(news), 8 * 128, dtype, gen(5))
    starts = None if news is None else starts_of(news)
    want = torch.empty_like(q)
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, want, c.work, starts=starts)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for i in range(30):
        y = torch.full_like(q, math.nan)
        if i % 3 == 0:
            ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, y, c.work, starts=starts)
        elif i % 3 == 1:
            other.wait_stream(torch.cuda.current_stream())
            ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, y, c.work, starts=starts, stream=other)
            torch.cuda.current_stream().wait_stream(other)
        else:
            other.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(other):
                ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, y, c.work, starts=starts)
            torch.cuda.current_stream().wait_stream(other)
        assert torch.equal(y, want), i


def test_two_graphs_share_a_workspace_one_after_another():
    a, b = Cache([5000, 70], 2, 128, 16, seed=6), Cache([40, 9000], 2, 64, 64, seed=7)
    work = ops.cache_workspace(max(a.P, b.P), 128)
    news = [1, 200]
    q = [rows(sum(news), 8 * 128, BF16, gen(8)), rows(2, 8 * 64, F16, gen(9))]
    y = [torch.empty_like(v) for v in q]

    def run(i):
        c = (a, b)[i]
        ops.cache_attention(q[i], c.cache, c.scale, c.tables, c.lengths, y[i], work, starts=starts_of(news) if i == 0 else None)
    starts = starts_of(news)
    runs = [lambda: ops.cache_attention(q[0], a.cache, a.scale, a.tables, a.lengths, y[0], work, starts=starts),
            lambda: ops.cache_attention(q[1], b.cache, b.scale, b.tables, b.lengths, y[1], work)]
    graphs, stream = [], torch.cuda.Stream()
    for f in runs:
        with torch.cuda.stream(stream):
            f()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            f()
    want = [v.clone() for v in y]
    check_attention(a, q[0], want[0], news)
    check_attention(b, q[1], want[1], [1, 1])
    for i in range(20):
        for v in y:
            v.fill_(math.nan)
        for k in ((0, 1), (1, 0), (0, 0, 1), (1, 1, 0))[i % 4]:
            graphs[k].replay()
        assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])


@pytest.mark.parametrize("replayed", [False, True], ids=["eager", "graphs"])
def test_attention_beside_the_products_on_streams_of_their_own(replayed):
    """Tensor memory of an SM is divided between kernels that know nothing of each other."""
    c = [Cache([3000, 200, 4000], 2, 128, 64, seed=i) for i in range(3)]
    news = [1, 200, 150]
    starts = starts_of(news)
    q = [rows(sum(news), 8 * 128, BF16, gen(10)), rows(sum(news), 8 * 128, F16, gen(11)), rows(3, 8 * 128, BF16, gen(12))]
    y = [torch.empty_like(v) for v in q]
    wide, narrow = make(700, 6000, 512, BF16, 1), make(60, 19200, 512, F16, 2)
    jobs = [lambda: ops.cache_attention(q[0], c[0].cache, c[0].scale, c[0].tables, c[0].lengths, y[0], c[0].work, starts=starts),
            lambda: ops.cache_attention(q[1], c[1].cache, c[1].scale, c[1].tables, c[1].lengths, y[1], c[1].work, starts=starts),
            lambda: ops.cache_attention(q[2], c[2].cache, c[2].scale, c[2].tables, c[2].lengths, y[2], c[2].work),
            lambda: ops.matmul_fp8(*wide[:5]), lambda: ops.matmul_fp8(*narrow[:5])]
    results = [*y, wide[4], narrow[4]]
    want = []
    for job, res in zip(jobs, results):
        job()
        torch.cuda.synchronize()
        want.append(res.clone())
    streams = [torch.cuda.Stream() for _ in jobs]
    if replayed:
        graphs = []
        for job, s in zip(jobs, streams):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=s):
                for _ in range(4):
                    job()
        jobs = [gr.replay for gr in graphs]
    for res in results:
        res.zero_()
    torch.cuda.synchronize()
    for _ in range(30):
        for job, s in zip(jobs, streams):
            with torch.cuda.stream(s):
                job()
    torch.cuda.synchronize()
    for i, (res, w) in enumerate(zip(results, want)):
        assert torch.equal(res, w), i
    assert all(v.errors() == _lib.LORA_OK for v in c)


def test_write_and_attention_follow_each_other_without_waiting():
    """Each call reads what the one before it wrote, 60 times over."""
    c = Cache([1, 1, 1], 2, 128, 16, seed=13, spare=40, more_places=12)
    g = gen(13)
    k = [rows(3, 256, BF16, g) for _ in range(60)]
    q = rows(3, 8 * 128, BF16, g)
    ys = [torch.empty_like(q) for _ in range(60)]
    for i in range(60):
        c.lengths += 1
        ops.pages_extend(c.tables, c.lengths, c.refs, 16, c.work)
        ops.cache_write(k[i], k[i], c.cache, c.scale, c.tables, c.lengths, c.work)
        ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, ys[i], c.work)
    torch.cuda.synchronize()
    c.lens = c.lengths.tolist()
    check_attention(c, q, ys[-1], [1, 1, 1])
    assert c.lens == [61] * 3 and c.errors() == _lib.LORA_OK


def test_layer_refusals():
    m = Model(1, 4, 2, 64, 16, 8, 2, 4)
    inputs = m.layers[0].inputs
    with pytest.raises(ValueError):
        CachedAttention(inputs, m.cache[0][:, :, :1].contiguous(), m.scale[0])
    with pytest.raises(ValueError):
        CachedAttention(inputs, m.cache, m.scale)
    with pytest.raises(ValueError):
        CachedAttention(inputs, m.cache[0].cpu(), m.scale[0])
    small = ops.cache_workspace(4, 64)
    q = torch.zeros(2, 256, dtype=BF16, device="cuda")
    with pytest.raises(ops.LoraError):                       # a workspace of fewer pages
        ops.cache_attention(q, m.cache[0], m.scale[0], m.tables, m.lengths, torch.empty_like(q), small[:small.numel() - 256])
    with pytest.raises(ops.LoraError):                       # y over q
        ops.cache_attention(q, m.cache[0], m.scale[0], m.tables, m.lengths, q, m.work)
