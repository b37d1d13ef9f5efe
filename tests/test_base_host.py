"""The host side of the operators around a LoRA-wrapped projection, without a
GPU: exported symbols, workspace sizes, refusals (no call here launches), the
rotary frequencies against their formulas in Python's own arithmetic, and the
argument proof of the quantiser's rounding by exhaustion."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from gather_matmul_b200 import _lib, build, ops

HEADER = os.path.join(os.path.dirname(__file__), "..", "include", "lora.h")
FAKE = 0x10000   # a 256-byte aligned non-null address; never dereferenced
INV, UNS, MIS = _lib.LORA_ERR_INVALID_ARG, _lib.LORA_ERR_UNSUPPORTED, _lib.LORA_ERR_MISALIGNED


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.load()


def test_every_declared_function_is_exported_and_bound(L):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(lora_[a-z0-9_]+)\s*\(", src))
    for n in ("lora_quantize_fp8", "lora_matmul_fp8", "lora_linear_fp8", "lora_rope",
              "lora_norm_rope", "lora_rope_frequencies", "lora_linear_fp8_workspace_bytes"):
        assert n in names
    assert names == set(_lib.SIGNATURES)
    for n in names:
        assert hasattr(L, n)
    for c in ("LORA_FP8_BLOCK", "LORA_MAX_HEAD_DIM", "LORA_MAX_HEADS"):
        assert int(re.search(rf"#define {c} (\d+)", src).group(1)) == getattr(_lib, c)


def test_linear_workspace_bytes(L):
    def a256(v):
        return (v + 255) // 256 * 256
    for T, K in [(0, 1), (1, 1), (1, 4096), (77, 1000), (8192, 14336), (1 << 22, 1 << 20)]:
        rows, up = max(T, 1), -(-K // 16) * 16
        assert L.lora_linear_fp8_workspace_bytes(T, K) == \
            a256(rows * up) + a256(4 * rows * -(-K // 128))
    for T, K in [(-1, 4), (4, 0), ((1 << 22) + 1, 4), (4, (1 << 20) + 1)]:
        assert L.lora_linear_fp8_workspace_bytes(T, K) == 0


def _quant(L, dt=0, T=8, K=200, rows=1, x=FAKE, ldx=200, q=FAKE, ldq=208, s=FAKE):
    return L.lora_quantize_fp8(dt, T, K, rows, x, ldx, q, ldq, s, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), INV), (dict(T=-1), INV), (dict(K=0), INV), (dict(x=0), INV), (dict(q=0), INV),
    (dict(s=0), INV), (dict(ldx=192), INV), (dict(ldq=192), INV), (dict(rows=64), UNS),
    (dict(rows=0), UNS), (dict(T=(1 << 22) + 1), UNS), (dict(K=(1 << 20) + 1), UNS),
    (dict(ldx=204), MIS), (dict(ldq=200), MIS), (dict(x=FAKE + 8), MIS), (dict(q=FAKE + 8), MIS),
    (dict(s=FAKE + 2), MIS), (dict(T=0, x=0, q=0, s=0), 0),
])
def test_quantize_refusals(L, kw, status):
    assert _quant(L, **kw) == status


def _matmul(L, dt=1, T=8, N=100, K=200, q=FAKE, ldq=208, qs=FAKE, W=FAKE, ldw=208, ws=FAKE, y=FAKE,
            ldy=104):
    return L.lora_matmul_fp8(dt, T, N, K, q, ldq, qs, W, ldw, ws, y, ldy, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=-1), INV), (dict(T=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(q=0), INV),
    (dict(W=0), INV), (dict(y=0), INV), (dict(qs=0), INV), (dict(ws=0), INV),
    (dict(ldq=192), INV), (dict(ldw=192), INV), (dict(ldy=96), INV),
    (dict(ldq=200), MIS), (dict(ldw=200), MIS), (dict(ldy=100), MIS), (dict(q=FAKE + 8), MIS),
    (dict(W=FAKE + 8), MIS), (dict(y=FAKE + 8), MIS), (dict(qs=FAKE + 1), MIS),
    (dict(N=(1 << 20) + 1), UNS), (dict(T=0, q=0, y=0), 0),
])
def test_matmul_refusals(L, kw, status):
    assert _matmul(L, **kw) == status


def _linear(L, dt=1, T=8, N=100, K=200, x=FAKE, ldx=200, W=FAKE, ldw=208, ws=FAKE, y=FAKE, ldy=104,
            work=FAKE, nb=None):
    nb = L.lora_linear_fp8_workspace_bytes(T, K) if nb is None else nb
    return L.lora_linear_fp8(dt, T, N, K, x, ldx, W, ldw, ws, y, ldy, work, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(work=0), INV), (dict(nb=100), INV), (dict(work=FAKE + 128), MIS), (dict(x=0), INV),
    (dict(ldx=196), INV), (dict(ldx=204), MIS), (dict(ws=0), INV), (dict(y=0), INV),
    (dict(K=0), INV), (dict(T=(1 << 22) + 1, nb=1 << 40), UNS), (dict(T=0, x=0), 0),
])
def test_linear_refusals(L, kw, status):
    assert _linear(L, **kw) == status


def _rope(L, dt=1, T=8, dim=64, rot=64, heads=(4, 2), x=FAKE, ldx=512, xo=(0, 256), y=1 << 24, ldy=384,
          yo=(0, 256), pos=FAKE, f=FAKE, attn=1.0, n=None, w=None, eps=None):
    n = len(heads) if n is None else n
    h = (ctypes.c_int32 * len(heads))(*heads)
    a, b = (ctypes.c_int64 * len(xo))(*xo), (ctypes.c_int64 * len(yo))(*yo)
    if w is None and eps is None:
        return L.lora_rope(dt, T, dim, rot, n, h, x, ldx, a, y, ldy, b, pos, f, attn, 0, None)
    ws = (ctypes.c_void_p * len(heads))(*(w or (FAKE, FAKE)))
    return L.lora_norm_rope(dt, T, dim, rot, n, h, x, ldx, a, ws, 1e-6 if eps is None else eps, y,
                            ldy, b, pos, f, attn, 0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), INV), (dict(T=-1), INV), (dict(dim=0), INV), (dict(rot=0), INV), (dict(rot=63), INV),
    (dict(rot=66), INV), (dict(dim=60, rot=60), UNS), (dict(dim=264), UNS), (dict(n=0), UNS),
    (dict(n=9), UNS), (dict(heads=(4, 0)), INV), (dict(xo=(0, 257)), MIS), (dict(yo=(0, 260)), INV),
    (dict(xo=(0, 388)), INV), (dict(xo=(0, -8)), INV), (dict(yo=(0, 248)), INV),   # overlap in y
    (dict(x=0), INV), (dict(y=0), INV), (dict(pos=0), INV), (dict(f=0), INV), (dict(pos=FAKE + 4), MIS),
    (dict(f=FAKE + 4), MIS), (dict(ldx=516), MIS), (dict(x=FAKE + 2), MIS), (dict(attn=math.inf), INV),
    (dict(attn=math.nan), INV), (dict(heads=(4096, 1), ldx=1 << 20, ldy=1 << 20, xo=(0, 262144), yo=(0, 262144)), UNS),
    (dict(eps=0.0), INV), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV), (dict(w=(FAKE, FAKE + 8)), MIS),
    # y over x: another offset, another row stride, one row further
    (dict(y=FAKE, ldy=512, yo=(64, 320)), INV), (dict(y=FAKE), INV),
    (dict(y=FAKE + 2 * 512, ldy=512), INV), (dict(T=0, x=0, y=0, pos=0), 0),
])
def test_rope_refusals(L, kw, status):
    assert _rope(L, **kw) == status


def _freq(L, rot=64, base=10000.0, kind=0, factor=4.0, orig=4096.0, fast=32.0, slow=1.0):
    out, attn = (ctypes.c_double * 128)(), ctypes.c_float()
    st = L.lora_rope_frequencies(rot, base, kind, factor, orig, fast, slow, out, ctypes.byref(attn))
    return st, list(out)[:rot // 2], attn.value


@pytest.mark.parametrize("kw,status", [
    (dict(rot=0), INV), (dict(rot=7), INV), (dict(rot=258), UNS), (dict(base=1.0), INV),
    (dict(base=math.nan), INV), (dict(base=math.inf), INV), (dict(kind=5), INV), (dict(kind=-1), INV),
    (dict(kind=1, factor=0.0), INV), (dict(kind=2, rot=2), INV), (dict(kind=3, orig=0.0), INV),
    (dict(kind=4, fast=1.0), INV), (dict(kind=4, slow=0.0), INV), (dict(kind=0, factor=0.0), 0),
])
def test_frequency_refusals(L, kw, status):
    assert _freq(L, **kw)[0] == status


@pytest.mark.parametrize("rot,base,orig", [(2, 10000.0, 2048.0), (64, 10000.0, 4096.0), (128, 500000.0, 8192.0),
                                           (40, 1e6, 32768.0), (256, 10000.0, 100.0)])
@pytest.mark.parametrize("factor", [1.0, 4.0, 0.5, 40.0])
def test_frequencies(L, rot, base, orig, factor):
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    close = lambda a, b: np.testing.assert_allclose(a, b, rtol=1e-12)   # noqa: E731
    assert _freq(L, rot, base, 0)[1:] == (_freq(L, rot, base, 0)[1], 1.0)
    close(_freq(L, rot, base, 0)[1], f)
    close(_freq(L, rot, base, 1, factor)[1], [v / factor for v in f])
    if rot >= 4:
        b2 = base * factor ** (rot / (rot - 2))
        close(_freq(L, rot, base, 2, factor)[1], [b2 ** (-2 * i / rot) for i in range(rot // 2)])
        # the slowest pair is stretched by exactly the factor
        close(_freq(L, rot, base, 2, factor)[1][-1], f[-1] / factor)
    st, got, attn = _freq(L, rot, base, 4, factor, orig)
    for v, g in zip(f, got):
        turns = orig * v / (2 * math.pi)
        u = min(max((turns - 1) / 31, 0), 1)
        close(g, ((1 - u) / factor + u) * v)
    assert attn == 1.0
    st, got, attn = _freq(L, rot, base, 3, factor, orig)
    assert abs(attn - (0.1 * math.log(factor) + 1 if factor > 1 else 1)) < 1e-6
    at = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))   # noqa: E731
    low, high = max(math.floor(at(32)), 0), min(math.ceil(at(1)), rot - 1)
    for i, (v, g) in enumerate(zip(f, got)):
        u = min(max((i - low) / max(high - low, 1e-3), 0), 1)
        close(g, v / factor * u + v * (1 - u))


def test_binding_refusals_on_cpu_tensors():
    q = torch.zeros(4, 256).to(torch.float8_e4m3fn)
    x, s = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, 2)
    W, ws, y = torch.zeros(64, 256).to(torch.float8_e4m3fn), torch.zeros(1, 2), torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current CUDA device"):
        ops.quantize_fp8(x, q, s)
    with pytest.raises(ValueError, match="current CUDA device"):
        ops.matmul_fp8(q, s, W, ws, y)
    with pytest.raises(ValueError, match="current CUDA device"):
        ops.linear_fp8(x, W, ws, y, torch.zeros(1 << 16, dtype=torch.uint8))
    with pytest.raises(TypeError):
        ops.quantize_fp8(x, x, s)                              # q of another type
    with pytest.raises(TypeError):
        ops.quantize_fp8(x, q, s.double())
    with pytest.raises(TypeError):
        ops.quantize_fp8(x, q, torch.zeros(4, 3))              # one scale too many
    with pytest.raises(ValueError):
        ops.quantize_fp8(x.t(), q, s)                          # columns apart
    with pytest.raises(ValueError):
        ops.quantize_fp8(x, q[:2], s)
    with pytest.raises(ValueError):
        ops.matmul_fp8(q, s, W[:, :128], ws, y)
    with pytest.raises(TypeError):
        ops.matmul_fp8(q, s, W, torch.zeros(2, 2), y)
    with pytest.raises(TypeError):
        ops.linear_fp8(x, W, ws, y.half(), torch.zeros(1 << 16, dtype=torch.uint8))
    pos, f = torch.zeros(4, dtype=torch.int64), torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="current CUDA device"):
        ops.rope(x, x, [4], 64, pos, f)
    with pytest.raises(TypeError):
        ops.rope(x, x, [4], 64, pos.int(), f)
    with pytest.raises(TypeError):
        ops.rope(x, x, [4], 64, pos, f.float())
    with pytest.raises(TypeError):
        ops.norm_rope(x, [torch.ones(64)], x, [4], 64, pos, f)
    with pytest.raises(ValueError):
        ops.norm_rope(x, [], x, [4], 64, pos, f)
    with pytest.raises(ValueError):
        ops.rope_frequencies(64, kind="other", device="cpu")
    with pytest.raises(ops.LoraError):
        ops.rope_frequencies(63, device="cpu")
    with pytest.raises(ops.LoraError):
        ops.linear_fp8_workspace(4, 0, device="cpu")


def test_slices_past_the_last_column_are_refused():
    x = torch.zeros(4, 512, dtype=torch.bfloat16)[:, :248]
    with pytest.raises(ValueError, match="past the last column"):
        ops._offsets(x, [4], 64, None)
    with pytest.raises(ValueError, match="past the last column"):
        ops._offsets(x, [1], 64, [192])
    assert list(ops._offsets(x, [1, 2], 64, None)[1]) == [0, 64]
    with pytest.raises(ValueError, match="one column offset"):
        ops._offsets(x, [1, 2], 64, [0])


# ---------------------------------------------------------------- the quantiser's rounding
def e4m3_grid():
    return np.array([m * 2.0 ** -9 for m in range(8)] +
                    [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def test_product_with_the_reciprocal_then_18_bits_rounds_as_the_quotient_does():
    """For every pair of 8-bit significands (all of bf16's) and a sample of
    11-bit ones (fp16's), x * rn(448 / a) in fp32, rounded to 18 bits, rounds to
    the same e4m3 value (ties to even) as the real quotient 448 x / a."""
    grid = e4m3_grid()
    border = (grid[1:] + grid[:-1]) / 2

    def check(X, A):
        x, a = X.astype(np.float32), A.astype(np.float32)
        r = np.float32(448) / a
        t = x * r
        u = (t.astype(np.float64) * 65).astype(np.float32)         # one rounding
        h = (u.astype(np.float64) - 64 * t.astype(np.float64)).astype(np.float32)
        # 448 x / a against border m / 1024 (m whole): 448 * 1024 * X against m * A, in integers
        m = np.round(border * 1024).astype(np.int64)
        assert np.array_equal(m / 1024, border)
        lhs = 448 * 1024 * X.astype(np.int64)
        got = np.searchsorted(border, h.astype(np.float64), "left"), np.searchsorted(border, h.astype(np.float64), "right")
        at = np.searchsorted(m, lhs / A, "left")              # near; settled in integers below
        want_l, want_r = np.zeros_like(at), np.zeros_like(at)
        for d in (-1, 0, 1):
            j = np.clip(at + d, 0, len(m) - 1)
            want_l = np.maximum(want_l, np.where(m[j] * A < lhs, j + 1, 0))
            want_r = np.maximum(want_r, np.where(m[j] * A <= lhs, j + 1, 0))
        even = lambda lo, hi: np.where(lo != hi, lo + lo % 2, lo)     # noqa: E731
        assert np.array_equal(even(*got), even(want_l, want_r))

    sig = np.arange(128, 256, dtype=np.int64)
    for shift in range(0, 20):
        A, X = np.meshgrid(sig << 19, sig << (19 - shift))
        keep = X <= A
        check(X[keep], A[keep])
    rng = np.random.default_rng(1)
    A = rng.integers(1024, 2048, 400000) << 19
    X = rng.integers(1024, 2048, 400000) << (19 - rng.integers(0, 20, 400000))
    check(X[X <= A], A[X <= A])
