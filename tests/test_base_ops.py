"""GPU tests of the operators around a LoRA-wrapped projection, each against its
formula in 64 bits on the same bits.

Tolerances, from the arithmetic (u = half a step of the output's type, relative:
2^-8 bf16, 2^-11 fp16):

  quantiser   none: the value is the rounded real quotient, the scale the
              rounded a / 448.
  product     every product of two e4m3 values is exact in fp32; a sum of n
              fp32 terms, each step off by at most 2^-23 (truncated), is off by
              n 2^-23 of the sum of magnitudes.  A block of 128, KB blocks and
              two scale products: (128 + KB + 4) 2^-23 sum |terms|, then u |y|.
  rotation    the angle, reduced in turns to [-1/2, 1/2] in fp64 and rounded to
              fp32, is off by pi 2^-25 at most; sine and cosine by 2 units of
              2^-24 more, the products and the sum by 3 half steps: under
              2^-21 (|a| + |b|) m, then u |y|.
  norm        dim squares summed in fp32, a division, a root, a reciprocal and
              two products: (dim + 8) 2^-24 relative, before the rotation.

fp16 results below its normal range round to steps of 2^-24: 2^-25 is added.
"""
import math

import pytest
import torch

from gather_matmul_b200 import _lib, ops

pytestmark = pytest.mark.gpu

F16, BF16, FP8 = torch.float16, torch.bfloat16, torch.float8_e4m3fn
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8}
TYPES = [pytest.param(F16, id="f16"), pytest.param(BF16, id="bf16")]


def up(n, m):
    return -(-n // m) * m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def strided(T, K, multiple, dtype, fill=None, extra=0):
    """A [T, K] view of rows `multiple`-aligned and `extra` longer, and the whole."""
    whole = torch.zeros(T, up(K, multiple) + extra, device="cuda").to(dtype)
    if fill is not None:
        whole.view(torch.uint8).fill_(fill)
    return whole[:, :K], whole


# ---------------------------------------------------------------- 64-bit forms
def grid():
    return torch.tensor([m * 2.0 ** -9 for m in range(8)] +
                        [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64)


def round_e4m3(v):
    """Nearest e4m3 value, ties to the even code; NaN stays NaN."""
    g = grid().to(v.device)
    mid = (g[1:] + g[:-1]) / 2
    lo, hi = torch.bucketize(v.abs(), mid), torch.bucketize(v.abs(), mid, right=True)
    code = torch.where(lo != hi, lo + lo % 2, lo)
    return torch.where(v.isnan(), v, torch.copysign(g[code], v))


def quantized(x, block_rows=1):
    """Values and scales of a finite x, by the formula."""
    T, K = x.shape
    p = torch.zeros(up(T, block_rows), up(K, 128), dtype=torch.float64, device=x.device)
    p[:T, :K] = x.double()
    b = p.view(-1, block_rows, p.shape[1] // 128, 128)
    a = b.abs().amax((1, 3)).clamp_min(2.0 ** -100)
    q = round_e4m3(b * 448 / a[:, None, :, None]).view(p.shape)[:T, :K]
    return q, (a / 448).float()


def product(q, qs, W, ws):
    """The formula in 64 bits, and the sum of the terms' magnitudes."""
    T, K = q.shape
    N = W.shape[0]
    l = q.double() * qs.double().repeat_interleave(128, 1)[:, :K]
    r = W.double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return l @ r.t(), l.abs() @ r.abs().t()


def assert_product(y, ref, mag, K):
    tol = (128 + -(-K // 128) + 4) * 2.0 ** -23 * mag + U[y.dtype] * 1.001 * ref.abs() + 2.0 ** -25
    err = (y.double() - ref).abs()
    assert torch.isfinite(y).all()
    assert (err <= tol).all(), f"{int((err > tol).sum())} off, worst {float((err / tol).max()):.3g} of the tolerance"


def rotated(x, heads, dim, positions, f, m, inter, off, weights=None, eps=0.0):
    """Slices of heads by the formula: list of [T, heads, dim] and their tolerances."""
    out = []
    rot = 2 * f.numel()
    ang = positions.double()[:, None] * f[None]
    c, s = (torch.cos(ang) * m)[:, None], (torch.sin(ang) * m)[:, None]
    for i, (h, o) in enumerate(zip(heads, off)):
        v = x[:, o:o + h * dim].double().view(x.shape[0], h, dim)
        rel = 0.0
        if weights is not None and weights[i] is not None:
            v = v * weights[i].double() / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)
            rel = (dim + 8) * 2.0 ** -24
        a, b = (v[..., 0:rot:2], v[..., 1:rot:2]) if inter else (v[..., :rot // 2], v[..., rot // 2:rot])
        ra, rb = a * c - b * s, b * c + a * s
        mag = (a.abs() + b.abs()) * abs(m)
        r = torch.cat([torch.stack([ra, rb], -1).flatten(-2) if inter else torch.cat([ra, rb], -1), v[..., rot:]], -1)
        g = torch.cat([torch.stack([mag, mag], -1).flatten(-2) if inter else torch.cat([mag, mag], -1), v[..., rot:].abs()], -1)
        tol = (2.0 ** -21 + rel) * g + U[x.dtype] * 1.001 * r.abs() + 2.0 ** -25
        out.append((r, tol))
    return out


# ---------------------------------------------------------------- the quantiser
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("T,K", [(1, 1), (1, 128), (1, 14336), (3, 127), (5, 129), (130, 1000), (257, 2056), (64, 8), (300, 4096)])
def test_quantize(dtype, rows, T, K):
    x, _ = strided(T, K, 8, dtype, extra=16)
    x.copy_(torch.randn(T, K, generator=gen(T + K), device="cuda") * torch.exp(2 * torch.randn(K, generator=gen(1), device="cuda")))
    x[T // 2] = 0
    q, whole = strided(T, K, 16, FP8, fill=0x55, extra=32)
    n = -(-T // rows)
    guard = torch.full((n * -(-K // 128) + 8,), 7.0, device="cuda")
    s = guard[:-8].view(n, -1)
    ops.quantize_fp8(x, q, s, block_rows=rows)
    rq, rs = quantized(x, rows)
    assert torch.equal(q.double(), rq) and torch.equal(s, rs)
    assert (whole[:, K:].view(torch.uint8) == 0x55).all() and (guard[-8:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_every_value_against_every_scale(dtype):
    """All finite values of the type in groups of many maxima, ties among them."""
    v = torch.arange(0, 1 << 15, device="cuda", dtype=torch.int32).to(torch.int16).view(dtype)
    v = v[torch.isfinite(v)]
    g = gen(3)
    a = v[torch.randint(1, v.numel(), (600,), generator=g, device="cuda")]
    x = v[torch.randint(0, v.numel(), (600, 128), generator=g, device="cuda")]
    # near values as well: within 2^10 of the group's maximum, where the 8-bit values lie
    near = a[:, None].float() * torch.rand(600, 128, generator=g, device="cuda") ** 3
    x = torch.where(torch.rand(600, 128, generator=g, device="cuda") < 0.8, near, x.float()).to(dtype)
    x = torch.minimum(x, a[:, None]).contiguous()
    x[:, 5] = a
    x = torch.where(torch.rand(600, 128, generator=g, device="cuda") < 0.5, -x, x)
    q, s = torch.empty(600, 128, dtype=FP8, device="cuda"), torch.empty(600, 1, device="cuda")
    ops.quantize_fp8(x, q, s)
    rq, rs = quantized(x)
    assert torch.equal(q.double(), rq) and torch.equal(s, rs)


def test_quantize_exact_ties():
    # a = 21: 448 x / 21 = 64 x / 3, a border for x = 3 m with odd m of 5 bits and its halves
    x = torch.zeros(1, 128, dtype=BF16, device="cuda")
    m = torch.arange(17, 32, 2, device="cuda")
    x[0, :8] = (3 * m).to(BF16) / 8
    x[0, 8:16] = -(3 * m).to(BF16) / 64
    x[0, 127] = 21
    q, s = torch.empty(1, 128, dtype=FP8, device="cuda"), torch.empty(1, 1, device="cuda")
    ops.quantize_fp8(x, q, s)
    assert torch.equal(q.double(), quantized(x)[0])
    want = (m // 2 + (m // 2) % 2) * 2.0        # the even neighbour
    assert torch.equal(q[0, :8].double(), want.double() * 8)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_infinities_and_nans_reach_their_group_only(dtype):
    x = torch.randn(4, 384, generator=gen(5), device="cuda").to(dtype)
    clean = x.clone()
    x[1, 130], x[2, 383] = math.inf, math.nan
    q, s = torch.empty(4, 384, dtype=FP8, device="cuda"), torch.empty(4, 3, device="cuda")
    ops.quantize_fp8(x, q, s)
    rq, rs = quantized(clean)
    assert math.isinf(s[1, 1]) and math.isnan(s[2, 2])
    ok = torch.ones(4, 3, dtype=torch.bool, device="cuda")
    ok[1, 1] = ok[2, 2] = False
    assert torch.equal(s[ok], rs[ok])
    assert torch.equal(q.double()[ok.repeat_interleave(128, 1)], rq[ok.repeat_interleave(128, 1)])
    W = torch.randn(32, 384, generator=gen(6), device="cuda").to(FP8)
    y = ops.matmul_fp8(q, s, W, torch.ones(1, 3, device="cuda"), torch.empty(4, 32, dtype=dtype, device="cuda"))
    assert torch.isfinite(y[[0, 3]]).all() and torch.isnan(y[[1, 2]]).all()


# ---------------------------------------------------------------- the product
SHAPES = [(1, 1, 1), (1, 128, 128), (1, 4096, 4096), (2, 64, 14336), (3, 129, 257), (7, 1000, 640), (16, 256, 4096),
          (17, 1501, 1000), (31, 384, 130), (32, 6144, 512), (33, 200, 2048), (48, 64, 16), (64, 2048, 2048),
          (65, 300, 384), (77, 1501, 1000), (128, 128, 8192), (129, 257, 513), (200, 513, 255), (256, 4096, 1024),
          (300, 72, 4104), (512, 1024, 896), (1000, 640, 1111), (1025, 1153, 200), (2048, 2304, 384),
          # more of the tiles and parts of K that the host chooses (all: test_base_paths.py)
          (4, 1024, 4096), (5, 4000, 2050), (20, 4000, 2050), (24, 4000, 300), (130, 2000, 6200), (70, 4000, 300),
          (200, 4000, 300), (70, 10000, 200), (64, 19100, 200), (128, 19100, 200), (300, 6000, 300),
          (300, 4000, 5300), (700, 6000, 200)]


def make(T, N, K, dtype, seed, extra=0, ints=False):
    g = gen(seed)
    q, _ = strided(T, K, 16, FP8, extra=extra, fill=0x7f)        # NaN past the rows' ends
    W, _ = strided(N, K, 16, FP8, extra=extra, fill=0x7f)
    KB, NB = -(-K // 128), -(-N // 128)
    if ints:
        q.copy_(torch.randint(-4, 5, (T, K), generator=g, device="cuda").float())
        W.copy_(torch.randint(-4, 5, (N, K), generator=g, device="cuda").float())
        qs = 2.0 ** torch.randint(-2, 3, (T, KB), generator=g, device="cuda").float()
        ws = 2.0 ** torch.randint(-2, 3, (NB, KB), generator=g, device="cuda").float()
    else:
        q.copy_((torch.randn(T, K, generator=g, device="cuda") * 100).clamp(-448, 448))
        W.copy_((torch.randn(N, K, generator=g, device="cuda") * 100).clamp(-448, 448))
        qs = torch.exp(torch.randn(T, KB, generator=g, device="cuda")) * 0.01
        ws = torch.exp(torch.randn(NB, KB, generator=g, device="cuda")) * 0.0005
    y, whole = strided(T, N, 8, dtype, fill=0x3c, extra=extra)
    return q, qs, W, ws, y, whole


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_matmul(dtype, T, N, K):
    q, qs, W, ws, y, whole = make(T, N, K, dtype, T + N + K, extra=48)
    ops.matmul_fp8(q, qs, W, ws, y)
    ref, mag = product(q, qs, W, ws)
    assert_product(y, ref, mag, K)
    assert (whole[:, N:].contiguous().view(torch.uint8) == 0x3c).all()      # columns past N untouched
    first = y.clone()
    ops.matmul_fp8(q, qs, W, ws, y)
    assert torch.equal(first, y)                                            # the same bits every time


@pytest.mark.parametrize("T,N,K", [(1, 256, 4096), (24, 300, 1024), (100, 128, 640), (513, 400, 2048), (1100, 1100, 512)])
def test_matmul_exact_on_integers(T, N, K):
    # small integers and power-of-two scales: every partial sum is a multiple of
    # 2^-4 below 2^20 in magnitude, exact in 24 bits, so only the last rounding is left
    q, qs, W, ws, y, _ = make(T, N, K, BF16, 7, ints=True)
    ops.matmul_fp8(q, qs, W, ws, y)
    assert torch.equal(y, product(q, qs, W, ws)[0].to(torch.float32).to(BF16))


def test_matmul_nan_values_reach_their_rows_and_columns_only():
    for T in (5, 70, 300):
        q, qs, W, ws, y, _ = make(T, 200, 300, BF16, 11)
        q[3, 299] = math.nan
        W[130, 0] = math.nan
        ops.matmul_fp8(q, qs, W, ws, y)
        bad = torch.zeros(T, 200, dtype=torch.bool, device="cuda")
        bad[3] = True
        bad[:, 130] = True
        assert torch.equal(torch.isnan(y), bad)


def test_matmul_zero_scales_and_no_tokens():
    q, qs, W, ws, y, _ = make(40, 136, 256, F16, 12)
    qs[:, 1] = 0
    ws[1] = 0
    ops.matmul_fp8(q, qs, W, ws, y)
    ref, mag = product(q, qs, W, ws)
    assert_product(y, ref, mag, 256)
    assert (y[:, 128:] == 0).all()
    before = ops.launch_count()
    ops.matmul_fp8(q[:0], qs[:0], W, ws, y[:0])
    ops.quantize_fp8(torch.empty(0, 256, dtype=F16, device="cuda"), q[:0], qs[:0])
    assert ops.launch_count() == before


def test_matmul_rows_past_2_31():
    """Outputs whose element offsets pass 2^31."""
    T, ld = 2100, 1 << 20
    whole = torch.empty(T, ld, dtype=BF16, device="cuda")
    q, qs, W, ws, _, _ = make(T, 72, 256, BF16, 13)
    y = whole[:, ld - 72:]
    y.fill_(3)
    whole[:, ld - 80:ld - 72] = 5
    ops.matmul_fp8(q, qs, W, ws, y)
    assert_product(y, *product(q, qs, W, ws), 256)
    assert (whole[:, ld - 80:ld - 72] == 5).all()
    x = whole[:, ld - 72:]
    f = ops.rope_frequencies(24)[0]
    pos = torch.arange(T, device="cuda")
    (r, tol), = rotated(x, [3], 24, pos, f, 1.0, False, [0])
    ops.rope(x, x, [3], 24, pos, f)
    assert ((x.double().view(T, 3, 24) - r).abs() <= tol).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,N,K", [(1, 4096, 4096), (5, 300, 1000), (33, 1024, 14336), (256, 640, 2056), (600, 1000, 520)])
def test_linear_is_quantize_then_matmul(dtype, T, N, K):
    g = gen(T)
    x, _ = strided(T, K, 8, dtype, extra=8)
    x.copy_(torch.randn(T, K, generator=g, device="cuda"))
    wide = (torch.randn(N, K, generator=g, device="cuda") * 0.02).to(dtype)
    W, _ = strided(N, K, 16, FP8)
    ws = torch.empty(-(-N // 128), -(-K // 128), device="cuda")
    if K % 8 == 0:
        ops.quantize_fp8(wide, W, ws, block_rows=128)
    y, _ = strided(T, N, 8, dtype)
    work = ops.linear_fp8_workspace(T, K)
    ops.linear_fp8(x, W, ws, y, work)
    rq, rs = quantized(x)
    assert_product(y, *product(rq, rs, W, ws), K)
    q, _ = strided(T, K, 16, FP8)
    s = torch.empty(T, -(-K // 128), device="cuda")
    ops.quantize_fp8(x, q, s)
    y2, _ = strided(T, N, 8, dtype)
    ops.matmul_fp8(q, s, W, ws, y2)
    assert torch.equal(y, y2)
    # and near the product of the unquantised values: two roundings of e4m3 (2^-4 each) per term
    full, mag = x.double() @ wide.double().t(), x.double().abs() @ wide.double().abs().t()
    assert ((y.double() - full).abs() <= (2.1 * 2.0 ** -4 + 0.01) * mag + 0.02).all()


# ---------------------------------------------------------------- rotation
HEADS = [  # heads per slice, dim, rot
    ([4, 2], 128, 128), ([32, 8], 128, 64), ([1], 64, 64), ([3, 1, 2], 80, 80), ([5], 96, 48), ([2, 2], 256, 256),
    ([7], 80, 20), ([9, 1], 64, 2), ([2], 8, 8), ([3], 24, 6), ([71], 192, 192), ([130], 256, 64), ([2], 256, 14)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("heads,dim,rot", HEADS, ids=[f"{'+'.join(map(str, h))}x{d}r{r}" for h, d, r in HEADS])
@pytest.mark.parametrize("T", [1, 2, 37])
@pytest.mark.parametrize("norm", [False, True], ids=["rope", "norm"])
def test_rope(dtype, inter, heads, dim, rot, T, norm):
    g = gen(T + dim + rot)
    n = sum(heads) * dim
    x, _ = strided(T, n + 40, 8, dtype, extra=24)
    x.copy_(torch.randn(T, n + 40, generator=g, device="cuda") * 3)
    pos = torch.randint(-5000, 1 << 20, (T,), generator=g, device="cuda")
    f, m = ops.rope_frequencies(rot, 500000.0, "yarn", 4.0, 32768.0)
    xo, yo, c = [], [], n
    for h in heads:                         # the slices from column 8 of x on, in reverse order in y
        xo.append(8 + (xo[-1] - 8 + prev * dim if xo else 0))
        c -= h * dim
        yo.append(c + 16)
        prev = h
    y, whole = strided(T, n + 32, 8, dtype, fill=0x3c, extra=8)
    w = [(1 + 0.3 * torch.randn(dim, generator=g, device="cuda")).to(dtype) if i != 1 or len(heads) != 2 else None
         for i in range(len(heads))]
    x[0, 8:8 + dim] = 0                     # a head of zeros
    kw = dict(x_col_off=xo, y_col_off=yo, interleaved=inter, attn_scale=m)
    if norm:
        ops.norm_rope(x, w, y, heads, dim, pos, f, eps=1e-5, **kw)
    else:
        ops.rope(x, y, heads, dim, pos, f, **kw)
    for (r, tol), h, o in zip(rotated(x, heads, dim, pos, f, m, inter, xo, w if norm else None, 1e-5), heads, yo):
        err = (y[:, o:o + h * dim].double().view(T, h, dim) - r).abs()
        assert (err <= tol).all(), f"worst {float((err / tol).max()):.3g} of the tolerance"
    rest = whole.clone()
    for h, o in zip(heads, yo):
        rest[:, o:o + h * dim] = whole[0, -1]
    assert (rest.view(torch.uint8) == 0x3c).all()         # other columns untouched
    # in place, the same bits
    z = x.clone(memory_format=torch.contiguous_format) if x.shape[1] % 8 == 0 else None
    if z is not None:
        before = z.clone()
        kw["y_col_off"] = xo
        (ops.norm_rope(z, w, z, heads, dim, pos, f, eps=1e-5, **kw) if norm else ops.rope(z, z, heads, dim, pos, f, **kw))
        for h, o, p in zip(heads, xo, yo):
            assert torch.equal(z[:, o:o + h * dim], y[:, p:p + h * dim])
            before[:, o:o + h * dim] = z[:, o:o + h * dim]
        assert torch.equal(before, z)


def test_rope_far_positions_and_turning_back():
    """Positions up to 2^53: the angle mod 2 pi in exact integers and 64 bits; a
    negative position turns back."""
    f = torch.tensor([2 * math.pi / 4, 2 * math.pi / 8], dtype=torch.float64, device="cuda")  # quarter, eighth turns
    x = torch.zeros(4, 8, dtype=BF16, device="cuda")
    x[:, 0], x[:, 1] = 1, 1
    pos = torch.tensor([(1 << 20) * 8 + 1, -1, (1 << 33) * 8 + 3, 0], device="cuda")
    y = ops.rope(x, torch.empty_like(x), [1], 8, pos, f)
    for t, p in enumerate((1, -1, 3, 0)):
        for i, turn in enumerate((4, 8)):
            assert abs(float(y[t, i]) - math.cos(2 * math.pi * p / turn)) < 2.0 ** -8
            assert abs(float(y[t, i + 2]) - math.sin(2 * math.pi * p / turn)) < 2.0 ** -8
    g = gen(2)
    x = torch.randn(9, 640, generator=g, device="cuda").to(F16)
    pos = torch.randint(0, 1 << 20, (9,), generator=g, device="cuda")
    f = ops.rope_frequencies(128)[0]
    z = ops.rope(ops.rope(x, torch.empty_like(x), [5], 128, pos, f), torch.empty_like(x), [5], 128, -pos, f)
    # two roundings of at most 2^-11 of a pair's length each
    length = torch.sqrt(x.double().view(9, 5, 2, 64).square().sum(2, keepdim=True)).expand(9, 5, 2, 64).reshape(9, 640)
    assert ((z.double() - x.double()).abs() <= 2.5 * 2.0 ** -11 * length + 2.0 ** -24).all()


def test_norm_rope_infinities_and_nans_stay_in_their_head():
    x = torch.randn(3, 4 * 64, generator=gen(4), device="cuda").to(BF16)
    x[1, 64 + 7], x[2, 130] = math.inf, math.nan
    w = [torch.ones(64, dtype=BF16, device="cuda")]
    y = ops.norm_rope(x, w, torch.empty_like(x), [4], 64, torch.arange(3, device="cuda"), ops.rope_frequencies(64)[0])
    bad = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    bad[1, 1] = bad[2, 2] = True
    assert torch.isfinite(y.view(3, 4, 64)[~bad]).all()
    assert torch.isnan(y.view(3, 4, 64)[bad]).any(-1).all()


def test_rope_many_tokens():
    T = 8192 + 3
    x = torch.randn(T, 6 * 128, generator=gen(8), device="cuda").to(BF16)
    w = [torch.randn(128, generator=gen(9 + i), device="cuda").to(BF16) for i in range(2)]
    pos = torch.arange(T, device="cuda") + 100000
    f, m = ops.rope_frequencies(128, 1e6, "linear", 4.0)
    y = ops.norm_rope(x, w, torch.empty_like(x), [4, 2], 128, pos, f, attn_scale=m)
    got = [y[:, :512], y[:, 512:]]
    for (r, tol), v in zip(rotated(x, [4, 2], 128, pos, f, m, False, [0, 512], w, 1e-6), got):
        assert ((v.double().reshape(r.shape) - r).abs() <= tol).all()


# ---------------------------------------------------------------- streams and graphs
def test_calls_on_another_stream_and_in_a_graph():
    T, N, K = 40, 640, 1024
    q, qs, W, ws, y, _ = make(T, N, K, BF16, 21)
    x = torch.randn(T, K, generator=gen(22), device="cuda").to(BF16)
    f = ops.rope_frequencies(64)[0]
    pos = torch.arange(T, device="cuda")
    work = ops.linear_fp8_workspace(T, K)
    out = torch.empty(T, N, dtype=BF16, device="cuda")

    def step():
        ops.linear_fp8(x, W, ws, y, work)
        ops.rope(y, out, [N // 64], 64, pos, f)
    step()
    want = out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(torch.randn(T, K, generator=gen(23), device="cuda"))
    pos.add_(1000)
    graph.replay()
    got = out.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(got, out) and not torch.equal(got, want)


@pytest.mark.parametrize("T", [3, 100, 300, 700])
def test_linear_sees_what_was_written_just_before(T):
    """The product reads its first weight tiles before the quantiser of the same
    call has ended: weights, inputs and outputs that change from call to call
    on one stream, without a wait between, must still be each call's own."""
    N, K = 640, 1024
    g = gen(41)
    wides = [(0.05 * torch.randn(N, K, generator=g, device="cuda")).to(BF16) for _ in range(4)]
    xs = [torch.randn(T, K, generator=g, device="cuda").to(BF16) for _ in range(4)]
    W, ws = torch.empty(N, K, dtype=FP8, device="cuda"), torch.empty(N // 128, K // 128, device="cuda")
    x, y = torch.empty(T, K, dtype=BF16, device="cuda"), torch.empty(T, N, dtype=BF16, device="cuda")
    work = ops.linear_fp8_workspace(T, K)

    def call(i, wait):
        ops.quantize_fp8(wides[i], W, ws, block_rows=128)
        if wait:
            torch.cuda.synchronize()
        ops.linear_fp8(xs[i], W, ws, y, work)
        if wait:
            torch.cuda.synchronize()
    want = []
    for i in range(4):
        call(i, True)
        want.append(y.clone())
    got = []
    for j in range(24):
        call(j % 4, False)
        got.append(y.clone())
    x.copy_(xs[2])
    ops.linear_fp8(x, W, ws, y, work)          # behind a torch kernel that wrote x
    x.fill_(float("nan"))                      # and before one that overwrites it
    torch.cuda.synchronize()
    for j, v in enumerate(got):
        assert torch.equal(v, want[j % 4]), j
    ops.linear_fp8(xs[2], W, ws, got[0], work)
    assert torch.equal(y, got[0])


def test_two_streams_with_a_workspace_each():
    T, N, K = 200, 768, 2048
    g = gen(51)
    x = [torch.randn(T, K, generator=g, device="cuda").to(F16) for _ in range(2)]
    q, qs, W, ws, _, _ = make(T, N, K, F16, 52)
    work = [ops.linear_fp8_workspace(T, K) for _ in range(2)]
    want = [ops.linear_fp8(x[i], W, ws, torch.empty(T, N, dtype=F16, device="cuda"), work[i]) for i in range(2)]
    out = [torch.empty(T, N, dtype=F16, device="cuda") for _ in range(2)]
    st = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(st[i]):
                ops.linear_fp8(x[i], W, ws, out[i], work[i])
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("norms", [True, False], ids=["norms", "plain"])
@pytest.mark.parametrize("T", [1, 9, 130])
def test_attention_inputs(norms, T):
    """The base product, the adapters' delta and the rotation as one layer makes
    them, against the formulas in 64 bits on the values each step received."""
    from gather_matmul_b200.graphs import LoraGraphSet
    from gather_matmul_b200.layers import AttentionInputs
    hq, hk, dim, K, S, r = 4, 2, 64, 512, 3, 16
    widths = [hq * dim, hk * dim, hk * dim]
    N, g = sum(widths), gen(31 + T)
    wide = (torch.randn(N, K, generator=g, device="cuda") * 0.05).to(BF16)
    W, ws = torch.empty(N, K, dtype=FP8, device="cuda"), torch.empty(N // 128, K // 128, device="cuda")
    ops.quantize_fp8(wide, W, ws, block_rows=128)
    A = [(0.05 * torch.randn(S, r, K, generator=g, device="cuda")).to(BF16) for _ in range(3)]
    B = [(0.05 * torch.randn(S, w, r, generator=g, device="cuda")).to(BF16) for w in widths]
    f, m = ops.rope_frequencies(dim)
    nw = [torch.rand(dim, generator=g, device="cuda").to(BF16) for _ in range(2)] if norms else [None, None]
    layer = AttentionInputs(W, ws, A, B, hq, hk, dim, f, max_tokens=max(T, 16), scale=0.5, attn_scale=m,
                            q_norm=nw[0], k_norm=nw[1])
    x = torch.randn(T, K, generator=g, device="cuda").to(BF16)
    idx = torch.randint(-1, S, (T,), generator=g, device="cuda").to(torch.int32)
    pos = torch.randint(0, 4096, (T,), generator=g, device="cuda")
    y = torch.empty(T, N, dtype=BF16, device="cuda")
    layer(x, idx, pos, y)
    assert ops.check_errors(layer.meta) == _lib.LORA_OK

    # 64 bits, with the roundings of y between the steps left out: each is 2^-8 of |y|
    rq, rs = quantized(x)
    base, mag = product(rq, rs, W, ws)
    ref, c = base.clone(), 0
    for a, b, w in zip(A, B, widths):
        for t in range(T):
            if idx[t] >= 0:
                ref[t, c:c + w] += 0.5 * (b[idx[t]].double() @ (a[idx[t]].double() @ x[t].double()))
        c += w
    step_err = 2.0 ** -8 * (base.abs() + ref.abs()) * 1.01 + 1e-3 * (ref - base).abs() + 2.0 ** -15 * mag + 1e-6
    v = y[:, widths[0] + widths[1]:].double()
    assert ((v - ref[:, -widths[2]:]).abs() <= step_err[:, -widths[2]:]).all()
    off = [0, widths[0]]
    for i, (h, o) in enumerate(zip([hq, hk], off)):
        t = ref[:, o:o + h * dim].view(T, h, dim)
        e = step_err[:, o:o + h * dim].view(T, h, dim)
        if norms:
            inv = 1 / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-6)
            # the head's size moves by at most the root mean square of its elements' errors
            de = torch.sqrt(e.square().mean(-1, keepdim=True))
            e = nw[i].double().abs() * (e * inv + t.abs() * inv * inv * de) * 1.1
            t = t * nw[i].double() * inv
        ang = pos.double()[:, None, None] * f
        a, b = t[..., :dim // 2], t[..., dim // 2:]
        want = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
        pair = (e[..., :dim // 2] + e[..., dim // 2:]).repeat(1, 1, 2)
        got = y[:, o:o + h * dim].double().view(T, h, dim)
        assert ((got - want).abs() <= pair + 2.0 ** -8 * want.abs() + 1e-5).all()

    # the same step captured twice, with and without the adapters' work, in the framework's graph set
    want = y.clone()
    gs = LoraGraphSet(lambda has: layer(x, idx, pos, y, has_lora=has)).capture()
    y.zero_()
    gs.replay(True)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    idx.fill_(-1)
    gs.replay(True)
    torch.cuda.synchronize()
    none = y.clone()
    y.zero_()
    gs.replay(False)
    torch.cuda.synchronize()
    assert torch.equal(y, none)


def test_attention_inputs_refusals():
    from gather_matmul_b200.layers import AttentionInputs
    W = torch.zeros(256, 128, device="cuda").to(FP8)
    ws = torch.ones(2, 1, device="cuda")
    A = [torch.zeros(2, 8, 128, dtype=BF16, device="cuda")]
    B = [torch.zeros(2, w, 8, dtype=BF16, device="cuda") for w in (128, 64, 64)]
    f = ops.rope_frequencies(64)[0]
    layer = AttentionInputs(W, ws, A, B, 2, 1, 64, f, max_tokens=8)
    with pytest.raises(ValueError):
        AttentionInputs(W, ws, A, B, 1, 1, 64, f, max_tokens=8)
    with pytest.raises(ValueError):
        AttentionInputs(W, ws, [A[0][:, :, :64].contiguous()], B, 2, 1, 64, f, max_tokens=8)   # another K
    with pytest.raises(ValueError):
        AttentionInputs(W, ws, A, [b[:1].contiguous() for b in B], 2, 1, 64, f, max_tokens=8)  # another S
    none = torch.empty(0, 128, dtype=BF16, device="cuda")
    before = ops.launch_count()
    layer(none, torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"),
          torch.empty(0, 256, dtype=BF16, device="cuda"))
    assert ops.launch_count() == before
    x = torch.zeros(9, 128, dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        layer(x, torch.zeros(9, dtype=torch.int32, device="cuda"), torch.zeros(9, dtype=torch.int64, device="cuda"),
              torch.empty(9, 256, dtype=BF16, device="cuda"))
