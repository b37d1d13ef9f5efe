"""GPU tests of the 8-bit products among the other kernels of the library: right
behind the adapters' tensor-core kernels on one stream, with nothing waited for
in between, and beside them on other streams, eager and replayed.  Tensor memory
and shared memory of an SM are then divided between kernels that know nothing of
each other.  Every result must have the bits that it has when each call is waited
for."""
import pytest
import torch

from gather_matmul_b200 import _lib, ops
from test_base_ops import BF16, F16, assert_product, gen, make, product

pytestmark = pytest.mark.gpu


class Adapters:
    """One batch's LoRA delta on y, from scratch each time."""

    def __init__(self, T, S, r, D, widths, dtype, seed):
        g = gen(seed)
        self.x = torch.randn(T, D, generator=g, device="cuda").to(dtype)
        self.A = [(0.05 * torch.randn(S, r, D, generator=g, device="cuda")).to(dtype) for _ in widths]
        self.B = [(0.05 * torch.randn(S, w, r, generator=g, device="cuda")).to(dtype) for w in widths]
        self.idx = torch.randint(-1, S, (T,), generator=g, device="cuda").to(torch.int32)
        self.y0 = torch.randn(T, sum(widths), generator=g, device="cuda").to(dtype)
        self.y, self.buf = self.y0.clone(), torch.empty(len(widths), T, r, device="cuda")
        self.meta, self.S = ops.workspace(T, S), S

    def start(self):
        self.y.copy_(self.y0)
        ops.group(self.idx, self.S, self.meta)

    def shrink(self, laned=False):
        (ops.shrink_laned if laned else ops.shrink)(self.x, self.A, self.idx, self.buf, self.meta)

    def expand(self):
        ops.expand(self.buf, self.B, self.idx, self.y, self.meta, 0.5)


@pytest.mark.parametrize("laned", [False, True], ids=["grouped", "laned"])
@pytest.mark.parametrize("r", [16, 32, 64])
@pytest.mark.parametrize("T,N,K", [(60, 19200, 512), (64, 4096, 1024), (200, 4096, 1024), (300, 6000, 512), (700, 6000, 512)])
def test_products_right_behind_the_adapters_kernels(laned, r, T, N, K):
    a = Adapters(T, 2, r, 1024, [1024, 512], BF16, 7 + r)
    q, qs, W, ws, y, _ = make(T, N, K, BF16, T + N)
    y2 = torch.empty(T, N, dtype=BF16, device="cuda") if N % 8 == 0 else y.clone()

    def step(wait):
        sync = torch.cuda.synchronize if wait else lambda: None
        a.start(), sync()
        a.shrink(laned), sync()
        ops.matmul_fp8(q, qs, W, ws, y), sync()
        a.expand(), sync()
        ops.matmul_fp8(q, qs, W, ws, y2), sync()
    step(True)
    assert_product(y, *product(q, qs, W, ws), K)
    want = a.y.clone(), y.clone(), y2.clone()
    assert not torch.equal(a.y, a.y0)
    for _ in range(20):
        y.zero_(), y2.zero_()
        step(False)
        assert torch.equal(a.y, want[0]) and torch.equal(y, want[1]) and torch.equal(y2, want[2])
    assert ops.check_errors(a.meta) == _lib.LORA_OK


@pytest.mark.parametrize("replayed", [False, True], ids=["eager", "graphs"])
def test_products_adapters_and_rotation_on_streams_of_their_own(replayed):
    g = gen(5)
    a = [Adapters(300, 2, r, 1024, [2048, 512], dt, 3) for r, dt in ((64, F16), (16, BF16))]
    wide, narrow = make(700, 6000, 512, BF16, 1), make(60, 19200, 512, F16, 2)
    W, ws = wide[2], wide[3]
    x = torch.randn(300, 512, generator=g, device="cuda").to(BF16)
    y, work = torch.empty(300, 6000, dtype=BF16, device="cuda"), ops.linear_fp8_workspace(300, 512)
    h, out = torch.randn(900, 768, generator=g, device="cuda").to(F16), torch.empty(900, 768, dtype=F16, device="cuda")
    pos, f = torch.arange(900, device="cuda"), ops.rope_frequencies(128)[0]

    def adapters(b):
        b.start(), b.shrink(), b.expand()
    jobs = [lambda: ops.matmul_fp8(*wide[:5]), lambda: ops.matmul_fp8(*narrow[:5]), lambda: adapters(a[0]),
            lambda: adapters(a[1]), lambda: ops.linear_fp8(x, W, ws, y, work), lambda: ops.rope(h, out, [6], 128, pos, f)]
    results = [wide[4], narrow[4], a[0].y, a[1].y, y, out]
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
    for b in a:
        assert ops.check_errors(b.meta) == _lib.LORA_OK
