"""GPU tests that reach every form of the kernels around a LoRA-wrapped
projection that the host chooses between, each with enough work to go round its
rings of buffers: a product's stages hold up to 11 blocks of 128 columns, its
scale slots 16, a wide CTA pair works on several tiles in turn from 75 tiles on;
the quantiser takes four groups to a half-warp from 32768 groups on, the rotation
two tokens to a thread from 568320 lanes on.  Which kernel ran, on how many CTAs,
is read from the profiler.  Tolerances as in test_base_ops.py."""
import json
import math
import re

import pytest
import torch

from gather_matmul_b200 import ops
from test_base_ops import (BF16, F16, FP8, TYPES, assert_product, gen, make, product, quantized, rotated, strided,
                           up)

pytestmark = pytest.mark.gpu


def kernels(call, tmp_path):
    """(name, CTAs) of every kernel that the call launches; none where the
    profiler records none (another one may be attached to the process)."""
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
        call()
        torch.cuda.synchronize()
    path = tmp_path / "trace.json"
    p.export_chrome_trace(str(path))
    return [(e["name"], math.prod(e["args"]["grid"])) for e in json.loads(path.read_text())["traceEvents"]
            if e.get("cat") == "kernel"]


def flag(text):
    return text.strip().replace("(bool)", "") in ("1", "true")


# (form, T, N, K): narrow forms as (tokens per tile, deep, parts of K), wide ones as (parts of K,)
PATHS = [((16, False, 1), 3, 20001, 4100), ((16, False, 2), 9, 14333, 6200), ((16, False, 2), 1, 14336, 8192),
         ((16, False, 4), 16, 4001, 8300), ((16, False, 8), 7, 1001, 14336), ((32, False, 1), 70, 10001, 2700),
         ((32, False, 2), 130, 2001, 6200), ((32, False, 4), 31, 4001, 8300), ((32, True, 1), 70, 4001, 4100),
         ((64, False, 1), 64, 19101, 2700), ((64, True, 1), 200, 4001, 4100), ((128, True, 1), 300, 6001, 2700),
         ((1,), 700, 6001, 2700), ((1,), 700, 6003, 2560), ((1,), 2600, 4101, 2700), ((1,), 2500, 4096, 2560),
         ((1,), 5000, 2301, 130), ((2,), 300, 4001, 5300), ((2,), 300, 4003, 5200)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("form,T,N,K", PATHS, ids=[f"{'wide' if len(f) == 1 else 'narrow'}{'-'.join(str(int(v)) for v in f)}"
                                                   f"-{T}x{N}x{K}" for f, T, N, K in PATHS])
def test_product_paths(dtype, form, T, N, K, tmp_path):
    q, qs, W, ws, y, whole = make(T, N, K, dtype, T + N + K, extra=48)
    ops.matmul_fp8(q, qs, W, ws, y)
    assert_product(y, *product(q, qs, W, ws), K)
    assert (whole[:, N:].contiguous().view(torch.uint8) == 0x3c).all()
    first = y.clone()
    ran = kernels(lambda: ops.matmul_fp8(q, qs, W, ws, y), tmp_path)
    assert torch.equal(first, y)
    if not ran or torch.cuda.get_device_properties(0).multi_processor_count != 148:
        return                                             # the choice goes by CTAs per SM
    (name, ctas), = ran
    if len(form) == 3:
        m = re.search(r"narrow_kernel<[^,]+, (?:\(int\))?(\d+), ([^>]+)>", name)
        assert m, name
        got = int(m[1]), flag(m[2]), ctas // (-(-N // 128) * -(-T // int(m[1])))
    else:
        assert "wide_kernel" in name
        tiles = -(-N // 256) * -(-T // 256)
        got = (ctas // (2 * tiles),) if 2 * tiles <= 74 else (1,) if ctas == 2 * min(tiles, 74) else None
    assert got == form


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,N,K", [(700, 6008, 1304), (2600, 4104, 2704)], ids=["one tile a pair", "several"])
def test_linear_on_the_wide_kernel_sees_what_was_written_just_before(dtype, T, N, K, tmp_path):
    """Weights and inputs that change from call to call on one stream: the wide
    kernel too reads weight tiles before the quantiser of its call has ended."""
    g = gen(81)
    wides = [(0.05 * torch.randn(N, K, generator=g, device="cuda")).to(dtype) for _ in range(3)]
    xs = [torch.randn(T, K, generator=g, device="cuda").to(dtype) for _ in range(3)]
    W, ws = strided(N, K, 16, FP8)[0], torch.empty(-(-N // 128), -(-K // 128), device="cuda")
    y, work = torch.empty(T, N, dtype=dtype, device="cuda"), ops.linear_fp8_workspace(T, K)

    def call(i):
        ops.quantize_fp8(wides[i], W, ws, block_rows=128)
        return ops.linear_fp8(xs[i], W, ws, y, work)
    want = []
    for i in range(3):
        call(i)
        torch.cuda.synchronize()
        q, s = quantized(xs[i])
        assert_product(y, *product(q, s, *quantized(wides[i], 128)), K)
        want.append(y.clone())
    got = []
    for j in range(12):
        call(j % 3)
        got.append(y.clone())
    torch.cuda.synchronize()
    for j, v in enumerate(got):
        assert torch.equal(v, want[j % 3]), j
    ran = kernels(lambda: call(0), tmp_path)
    assert not ran or any("wide_kernel" in n for n, _ in ran)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K", [(1100, 4100), (1100, 4103), (8193, 520), (2341, 1800), (8200, 512), (300, 14336)])
def test_quantize_four_groups_to_a_half_warp(dtype, T, K, tmp_path):
    g = gen(T + K)
    x, _ = strided(T, K, 8, dtype, extra=16)
    x.copy_(torch.randn(T, K, generator=g, device="cuda") * torch.exp(2 * torch.randn(K, generator=g, device="cuda")))
    x[T // 2] = 0
    q, whole = strided(T, K, 16, FP8, fill=0x55, extra=32)
    KB = -(-K // 128)
    guard = torch.full((T * KB + 8,), 7.0, device="cuda")
    s = guard[:-8].view(T, KB)
    ran = kernels(lambda: ops.quantize_fp8(x, q, s), tmp_path)
    rq, rs = quantized(x)
    assert torch.equal(q.double(), rq) and torch.equal(s, rs)
    assert (whole[:, K:].view(torch.uint8) == 0x55).all() and (guard[-8:] == 7).all()
    assert all(re.search(r"quant_rows_kernel<[^,]+, (?:\(int\))?4>", name) for name, _ in ran), ran
    # a NaN and an infinity reach their own groups only
    x[1, K - 1], x[T - 1, 130] = math.nan, math.inf
    ops.quantize_fp8(x, q, s)
    assert math.isnan(s[1, KB - 1]) and math.isinf(s[T - 1, 1])
    ok = torch.ones(T, KB, dtype=torch.bool, device="cuda")
    ok[1, KB - 1] = ok[T - 1, 1] = False
    assert torch.equal(s[ok], rs[ok])
    ok = ok.repeat_interleave(128, 1)[:, :K]
    assert torch.equal(q.double()[ok], rq[ok])


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_many_blocks(dtype):
    T, K = 3001, 4103
    x, _ = strided(T, K, 8, dtype)
    x.copy_(torch.randn(T, K, generator=gen(91), device="cuda"))
    q, s = strided(T, K, 16, FP8)[0], torch.empty(up(T, 128) // 128, up(K, 128) // 128, device="cuda")
    ops.quantize_fp8(x, q, s, block_rows=128)
    rq, rs = quantized(x, 128)
    assert torch.equal(q.double(), rq) and torch.equal(s, rs)


# vector length, heads per slice, dim, rot
WIDE = [(8, [7, 2], 128, 128), (8, [9], 128, 64), (8, [3, 2], 256, 256), (4, [8, 1], 72, 72), (4, [9], 80, 40),
        (2, [5, 3], 80, 20), (1, [8, 1], 64, 2), (1, [40], 16, 6)]


@pytest.mark.parametrize("dtype,inter", [(BF16, False), (F16, True), (BF16, True), (F16, False)],
                         ids=["bf16-halves", "f16-interleaved", "bf16-interleaved", "f16-halves"])
@pytest.mark.parametrize("norm", [False, True], ids=["rope", "norm"])
@pytest.mark.parametrize("V,heads,dim,rot", WIDE, ids=[f"{'+'.join(map(str, h))}x{d}r{r}" for _, h, d, r in WIDE])
def test_rotation_two_tokens_to_a_thread(dtype, inter, norm, V, heads, dim, rot, tmp_path):
    T, n, g = 8195, sum(heads) * dim, gen(dim + rot)
    x, _ = strided(T, n + 8, 8, dtype, extra=16)
    x.copy_(torch.randn(T, n + 8, generator=g, device="cuda") * 3)
    pos = torch.randint(-5000, 1 << 20, (T,), generator=g, device="cuda")
    f, m = ops.rope_frequencies(rot, 500000.0, "yarn", 4.0, 32768.0)
    w = [(1 + 0.3 * torch.randn(dim, generator=g, device="cuda")).to(dtype) if i == 0 else None for i in range(len(heads))]
    off = [8 + dim * sum(heads[:i]) for i in range(len(heads))]
    y, whole = strided(T, n + 8, 8, dtype, fill=0x3c, extra=8)

    def call(y):
        kw = dict(x_col_off=off, y_col_off=off, interleaved=inter, attn_scale=m)
        return (ops.norm_rope(x, w, y, heads, dim, pos, f, eps=1e-5, **kw) if norm
                else ops.rope(x, y, heads, dim, pos, f, **kw))
    ran = kernels(lambda: call(y), tmp_path)
    for (r, tol), h, o in zip(rotated(x, heads, dim, pos, f, m, inter, off, w if norm else None, 1e-5), heads, off):
        err = (y[:, o:o + h * dim].double().reshape(T, h, dim) - r).abs()
        assert (err <= tol).all(), f"worst {float((err / tol).max()):.3g} of the tolerance"
    rest = whole.clone()
    rest[:, 8:8 + n] = whole[0, -1]
    assert (rest.view(torch.uint8) == 0x3c).all()
    for name, _ in ran:
        t = re.search(r"rope_kernel<[^,]+, (?:\(int\))?(\d+), (?:\(int\))?\d+, (?:\(int\))?(\d+), ([^,]+), ([^>]+)>", name)
        assert t and (int(t[1]), int(t[2]), flag(t[3]), flag(t[4])) == (V, 2, inter, norm), name
    before = x.clone()
    call(x)                                                # in place, the same bits
    assert torch.equal(x[:, 8:8 + n], y[:, 8:8 + n]) and torch.equal(x[:, :8], before[:, :8])
