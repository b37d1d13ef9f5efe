"""GPU tests of the paged 8-bit cache, each against its formula in 64 bits (or in
whole numbers) on the same bits.

Tolerances, from the arithmetic (u = half a step of the output's type, relative:
2^-8 bf16, 2^-11 fp16):

  write       none: powers of two as scales, values rounded once (begun pages:
              once more).
  pages       none.
  attention   a logit is a sum of dim products in fp32, each step off by at most
              2^-23 (truncated): (dim + 8) 2^-23 c sum |q k|, and three roundings
              of it and of the running maximum, 2^-22 of the largest magnitude
              each in units of its logarithm; 2^-18 for the exponential (the
              polynomial that some are formed by is off by 2.6e-6).  Call the
              sum of these e: a weight is off by the factor 1 +- 2 e, numerator and
              denominator alike, so 4 e covers their quotient.  Weights round to
              fp16, 2^-11, or by 2^-25 absolutely where they are small: the
              largest weight is at least 2^6, so 2^-31 of it each.  The sums over
              n tokens: (n / 8 + 64) 2^-23 of the sum of magnitudes.  Then u |y|.

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
    return -(-n // m)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Cache:
    """One layer's cache: sequences of the given lengths on shuffled pages; every
    place that holds no token is NaN, and so is the scale of every free page."""

    def __init__(self, lens, H, dim, page, seed=0, spare=3, more_places=1, fill=True, scales=(-9, -5)):
        g = gen(seed)
        self.lens, self.H, self.dim, self.page = list(lens), H, dim, page
        need = [up(max(n, 0), page) for n in lens]
        self.B, self.M, self.P = len(lens), max(max(need, default=0), 1) + more_places, sum(need) + spare
        order = torch.randperm(self.P, generator=g, device="cuda").to(torch.int32)
        self.tables = torch.full((self.B, self.M), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(self.P, dtype=torch.int32, device="cuda")
        self.cache = torch.full((self.P, 2, H, page, dim), math.nan, device="cuda").to(FP8)
        self.scale = torch.full((self.P, 2, H), math.nan, device="cuda")
        at = 0
        for b, k in enumerate(need):
            pages = order[at:at + k]
            at += k
            self.tables[b, :k] = pages
            self.refs[pages.long()] = 1
            if fill and k:
                v = (torch.randn(k, 2, H, page, dim, generator=g, device="cuda") * 100).clamp(-448, 448)
                place = torch.arange(k * page, device="cuda").view(k, 1, 1, page, 1)
                self.cache[pages.long()] = torch.where(place < lens[b], v, math.nan).to(FP8)
                self.scale[pages.long()] = torch.exp2(torch.randint(*scales, (k, 2, H), generator=g, device="cuda").float())
        self.lengths = ints(list(lens))
        self.work = ops.cache_workspace(self.P, dim)

    def errors(self):
        return ops.check_errors(self.work)

    def kv(self, b, h):
        """k and v of a sequence's head in 64 bits."""
        n = self.lens[b]
        pages = self.tables[b, :up(n, self.page)].long()
        return [(self.cache[pages, a, h].double() * self.scale[pages, a, h].double()[:, None, None]).reshape(-1, self.dim)[:n]
                for a in (0, 1)]


def starts_of(news):
    s = [0]
    for n in news:
        s.append(s[-1] + n)
    return ints(s)


def rows(T, width, dtype, g, extra=0, more=0, std=1.0):
    """[T, width] columns of a longer matrix, `more` rows behind them."""
    whole = (torch.randn(T + more, width + extra, generator=g, device="cuda") * std).to(dtype)
    return whole[:, :width] if extra else whole


def check_attention(c, q, y, news, softmax_scale=None, window=0):
    sm = c.dim ** -0.5 if softmax_scale is None else softmax_scale
    group, t = q.shape[1] // (c.H * c.dim), 0
    for b, n in enumerate(news):
        length = c.lens[b]
        for h in range(c.H):
            if n == 0:
                continue
            k, v = c.kv(b, h)
            cols = slice(h * group * c.dim, (h + 1) * group * c.dim)
            qq = q[t:t + n, cols].double().reshape(n * group, c.dim)
            got = y[t:t + n, cols].reshape(n * group, c.dim)
            if length == 0:
                assert torch.equal(got, torch.zeros_like(got))
                continue
            i = (length - n + torch.arange(n, device="cuda"))[:, None, None]
            j = torch.arange(length, device="cuda")
            seen = (j <= i) & ((j > i - window) if window else (j >= 0))
            seen = seen.expand(n, group, length).reshape(n * group, length)
            a = ((qq @ k.t()) * sm).masked_fill(~seen, -math.inf)
            empty = ~seen.any(1)
            p = torch.softmax(a, 1).masked_fill(empty[:, None], 0.0)
            ref, mag = p @ v, p @ v.abs()
            big = ((qq.abs() @ k.abs().t()) * sm).masked_fill(~seen, 0.0).amax(1, keepdim=True)
            logs = (big + 40) * 2.0 ** -22
            e = (c.dim + 8) * 2.0 ** -23 * big + 3 * logs + 2.0 ** -18
            tol = mag * (4 * e + 2.0 ** -11 + (length / 8 + 64) * 2.0 ** -23) + \
                length * 2.0 ** -31 * v.abs().max() + U[y.dtype] * 1.001 * ref.abs() + 2.0 ** -25
            err = (got.double() - ref).abs()
            assert torch.isfinite(got).all(), (b, h)
            assert (err <= tol).all(), \
                f"seq {b} head {h}: {int((err > tol).sum())} off, worst {float((err / tol).max()):.3g} of the tolerance"
            assert torch.equal(got[empty], torch.zeros_like(got[empty]))
        t += n
    return t


def attend(c, q, y, news, **kw):
    starts = None if news is None else starts_of(news)
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, y, c.work, starts=starts, **kw)
    torch.cuda.synchronize()
    check_attention(c, q, y, [1] * c.B if news is None else news, kw.get("softmax_scale"), kw.get("window", 0))
    assert c.errors() == _lib.LORA_OK


# ---------------------------------------------------------------- single tokens
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 112, 128, 160, 192, 208, 256])
@pytest.mark.parametrize("page,H,group", [(16, 2, 4), (32, 3, 1), (64, 1, 8), (128, 2, 3)])
def test_decode_heads_and_pages(dtype, dim, page, H, group):
    c = Cache([1, 0, 15, 16, 17, 63, 64, 65, 300, 2 * page], H, dim, page, seed=dim + page)
    q = rows(c.B, H * group * dim, dtype, gen(1), extra=8)
    attend(c, q, torch.full_like(q.contiguous(), math.nan), None)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [1, 2, 5, 7, 8, 9, 12, 16, 17, 24, 40, 64])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_decode_groups(dtype, group, dim):
    c = Cache([333, 1, 0, 1000], 2, dim, 32, seed=group)
    q = rows(c.B, 2 * group * dim, dtype, gen(2))
    attend(c, q, torch.full_like(q, math.nan), None)


@pytest.mark.parametrize("lens", [[1], [40000], [20011, 3], [5000, 1, 0, 77, 4096, 64, 8191, 2]], ids=str)
@pytest.mark.parametrize("H,group", [(1, 1), (8, 4)])
def test_decode_long_sequences_are_shared_by_many_ctas(lens, H, group):
    c = Cache(lens, H, 128, 64, seed=len(lens))
    q = rows(c.B, H * group * 128, BF16, gen(3))
    attend(c, q, torch.full_like(q, math.nan), None)


def test_decode_many_ragged_sequences():
    g = torch.Generator().manual_seed(4)
    lens = [int(2 ** (torch.rand(1, generator=g) * 11)) if i % 7 else 0 for i in range(600)]
    c = Cache(lens, 2, 64, 16, seed=4)
    q = rows(c.B, 8 * 64, F16, gen(4))
    attend(c, q, torch.full_like(q, math.nan), None)


# ---------------------------------------------------------------- several tokens
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 80, 128, 192, 256])
@pytest.mark.parametrize("page,H,group", [(16, 2, 4), (128, 1, 7)])
@pytest.mark.parametrize("window", [0, 33])
def test_ragged_chunks(dtype, dim, page, H, group, window):
    news = [5, 0, 1, 130, 33, 0, 257, 2, 64]
    lens = [5, 0, 700, 131, 500, 90, 257, 2, 64]
    c = Cache(lens, H, dim, page, seed=dim)
    q = rows(sum(news), H * group * dim, dtype, gen(5), extra=16)
    attend(c, q, torch.full_like(q.contiguous(), math.nan), news, window=window)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 176, 256])
@pytest.mark.parametrize("B,H,group", [(70, 2, 2), (400, 3, 16), (300, 4, 3)])
@pytest.mark.parametrize("window", [0, 50])
def test_batches_for_both_kernels(dtype, dim, B, H, group, window):
    """Many sequences, most of them of few rows, some longer, some empty: each kernel takes its own."""
    g = torch.Generator().manual_seed(B + dim)
    news = [int(v) for v in torch.randint(0, 3, (B,), generator=g)]
    news[3], news[B // 2], news[B - 1] = (20, 16 // group, 7) if group == 16 else (200, 16 // group + 1, 90)
    lens = [n + int(v) if i % 5 else n for i, (n, v) in enumerate(zip(news, torch.randint(0, 150, (B,), generator=g)))]
    c = Cache(lens, H, dim, 16, seed=B)
    q = rows(sum(news), H * group * dim, dtype, gen(31))
    assert B * H > 128 and (B * H > 8 * 148 or sum(news) * group <= 16 * B)
    before = ops.launch_count()
    attend(c, q, torch.full_like(q, math.nan), news, window=window)
    assert ops.launch_count() - before == 2


@pytest.mark.parametrize("window", [1, 16, 64, 100, 5000])
@pytest.mark.parametrize("news", [None, [3, 200, 1, 65]], ids=["single", "chunks"])
def test_windows(window, news):
    c = Cache([900, 200, 2049, 65], 2, 128, 16, seed=window)
    q = rows(4 if news is None else sum(news), 8 * 128, BF16, gen(6))
    attend(c, q, torch.full_like(q, math.nan), news, window=window)


def test_more_new_tokens_than_the_length():
    c = Cache([3, 40], 2, 64, 16)
    news = [9, 41]
    q = rows(sum(news), 4 * 64, F16, gen(7))
    attend(c, q, torch.full_like(q, math.nan), news)


@pytest.mark.parametrize("news", [None, [2, 70]], ids=["single", "chunks"])
def test_rows_behind_the_last_sequence_are_left(news):
    c = Cache([100, 90], 2, 64, 16)
    T = 2 if news is None else sum(news)
    q = rows(T, 4 * 64, BF16, gen(8), more=5)
    y = torch.full_like(q, 7.0)
    if news is None:
        ops.cache_attention(q[:T], c.cache, c.scale, c.tables, c.lengths, y[:T], c.work)
    else:
        ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, y, c.work, starts=starts_of(news))
    check_attention(c, q, y, news or [1, 1])
    assert (y[T:] == 7).all()


def test_columns_of_one_matrix():
    c = Cache([100, 33], 2, 64, 16)
    whole = rows(2, 1024, BF16, gen(9))
    before = whole.clone()
    q, y = whole[:, 64:320], whole[:, 512:768]
    attend(c, q, y, None)
    assert torch.equal(whole[:, :512], before[:, :512]) and torch.equal(whole[:, 768:], before[:, 768:])


@pytest.mark.parametrize("sm", [1e-3, 1.0, 30.0])
@pytest.mark.parametrize("news", [None, [1, 30, 200]], ids=["single", "chunks"])
def test_sharp_and_flat_softmax(sm, news):
    c = Cache([500, 700, 200], 2, 64, 16, seed=11)
    q = rows(3 if news is None else sum(news), 4 * 64, F16, gen(11))
    attend(c, q, torch.full_like(q, math.nan), news, softmax_scale=sm)


@pytest.mark.parametrize("jump", [20.0, 60.0, 88.0, 150.0, 1000.0])
@pytest.mark.parametrize("news", [None, [20] * 40], ids=["single", "chunks"])
def test_a_score_far_above_all_before_it(jump, news):
    """One key among zeros, at another place in each sequence: its weight is 2^(1.44 jump) times the others'."""
    c = Cache([160] * 40, 1, 64, 16, seed=24)
    c.cache[:, 0] = 0.0
    c.scale[:, 0] = torch.where(c.scale[:, 0].isnan(), math.nan, 1.0)
    for b in range(40):
        at = 60 + 2 * b
        c.cache[int(c.tables[b, at // 16]), 0, 0, at % 16, 7] = 16.0
    q = torch.zeros(40 if news is None else sum(news), 2 * 64, device="cuda")
    q[:, 7] = jump / 16
    q[:, 64 + 7] = -jump / 16
    attend(c, q.to(BF16), torch.full(q.shape, math.nan, dtype=BF16, device="cuda"), news, softmax_scale=1.0)


@pytest.mark.parametrize("dtype,std", [(F16, 1e-6), (F16, 8000.0), (BF16, 1e-30), (BF16, 1e30)])
@pytest.mark.parametrize("news", [None, [1, 30, 200]], ids=["single", "chunks"])
def test_queries_of_all_sizes(dtype, std, news):
    c = Cache([500, 700, 200], 2, 64, 16, seed=12)
    q = rows(3 if news is None else sum(news), 4 * 64, dtype, gen(12), std=std)
    attend(c, q, torch.full_like(q, math.nan), news, softmax_scale=0.1 / std)


@pytest.mark.parametrize("news", [None, [2, 60]], ids=["single", "chunks"])
def test_scales_from_the_smallest_to_the_largest(news):
    c = Cache([600, 600], 1, 64, 16, seed=13)
    # values of one page are 2^64 times those of the next; logits stay small
    c.scale[:, 1] = torch.where(c.scale[:, 1].isnan(), math.nan, torch.exp2((torch.arange(c.P, device="cuda") % 2 * 64 - 32).float())[:, None])
    q = rows(2 if news is None else sum(news), 64, BF16, gen(13))
    attend(c, q, torch.full_like(q, math.nan), news)


def test_factors_that_are_no_powers_of_two():
    c = Cache([600, 90], 2, 128, 16, seed=14)
    c.scale *= torch.rand(c.scale.shape, generator=gen(14), device="cuda") + 0.5
    q = rows(2, 8 * 128, F16, gen(15))
    attend(c, q, torch.full_like(q, math.nan), None)


@pytest.mark.parametrize("news", [None, [1, 40]], ids=["single", "chunks"])
def test_a_nan_scale_spoils_its_head_alone(news):
    c = Cache([200, 200], 2, 64, 16)
    bad = int(c.tables[1, 3])
    c.scale[bad, 1, 1] = math.nan
    q = rows(2 if news is None else sum(news), 4 * 64, BF16, gen(16))
    y = torch.zeros_like(q)
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, y, c.work, starts=None if news is None else starts_of(news))
    nan = y.isnan().view(-1, 4, 64)
    assert nan[1:, 2:].all() and not nan[:1].any() and not nan[:, :2].any()


@pytest.mark.parametrize("group", [100, 256, 300, 700])
def test_one_head_of_k_for_hundreds_of_q(group):
    c = Cache([333, 0, 70], 1, 64, 16, seed=group)
    q = rows(c.B, group * 64, BF16, gen(25))
    attend(c, q, torch.full_like(q, math.nan), None)
    q = rows(5, group * 64, F16, gen(26))
    attend(c, q, torch.full_like(q, math.nan), [2, 0, 3])


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("news", [None, [30, 1]], ids=["single", "chunks"])
def test_a_query_of_no_number_spoils_its_row_alone(what, news):
    c = Cache([500, 90], 2, 64, 16, seed=27)
    T = 2 if news is None else sum(news)
    q, starts = rows(T, 4 * 64, BF16, gen(27)), None if news is None else starts_of(news)
    y, z = torch.empty_like(q), torch.empty_like(q)
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, y, c.work, starts=starts)
    q[0, 70] = what                                          # head 1 of the first token
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, z, c.work, starts=starts)
    assert z[0, 64:128].isnan().all()
    z[0, 64:128] = y[0, 64:128]
    assert torch.equal(y, z)


@pytest.mark.parametrize("what", [0x7F, 0xFF])
@pytest.mark.parametrize("news", [None, [40, 30]], ids=["single", "chunks"])
def test_values_behind_the_last_token_may_be_anything(what, news):
    """NaN there, in the places of the last page and in pages that are held and not needed."""
    c = Cache([83, 33], 2, 128, 16, seed=28, spare=8, more_places=3)
    q, starts = rows(2 if news is None else sum(news), 4 * 128, F16, gen(28)), None if news is None else starts_of(news)
    y, z = torch.empty_like(q), torch.empty_like(q)
    for b, n in enumerate(c.lens):
        c.cache[int(c.tables[b, n // 16]), :, :, n % 16:] = 0.0
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, y, c.work, starts=starts)
    for b, n in enumerate(c.lens):
        c.cache.view(torch.uint8)[int(c.tables[b, n // 16]), :, :, n % 16:] = what
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, z, c.work, starts=starts)
    assert torch.equal(y, z) and torch.isfinite(y).all()


def test_offsets_past_32_bits():
    """A cache of 5 GB whose last pages are in use, written, read and moved."""
    P, H, page, dim = 40000, 8, 64, 128
    c = Cache([1], H, dim, page)
    c.cache = torch.zeros(P, 2, H, page, dim, dtype=torch.uint8, device="cuda").view(FP8)
    assert c.cache.numel() > 1 << 32
    c.scale, c.P, c.B, c.M = torch.ones(P, 2, H, device="cuda"), P, 3, 4
    c.tables = ints([[P - 1, P - 3, P - 2, -1], [P - 4, -1, -1, -1], [P - 5, P - 6, -1, -1]])
    c.refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    c.refs[P - 6:] = 1
    c.lens, c.work = [150, 1, 100], ops.cache_workspace(P, dim)
    c.lengths = ints(c.lens)
    x = rows(251, 2 * H * dim, BF16, gen(29))
    ops.cache_write(x[:, :H * dim], x[:, H * dim:], c.cache, c.scale, c.tables, c.lengths, c.work, starts=starts_of(c.lens))
    c.lens = [151, 2, 101]
    c.lengths += 1
    ops.cache_write(x[:3, :H * dim], x[:3, H * dim:], c.cache, c.scale, c.tables, c.lengths, c.work)
    k, v = c.kv(0, 5)
    assert (k[:150] - x[:150, 5 * dim:6 * dim].double()).abs().max() <= 2.0 ** -4 * 8 and k.abs().max() > 1
    for news in (None, [40, 2, 9]):
        q = rows(3 if news is None else sum(news), 2 * H * dim, BF16, gen(30))
        attend(c, q, torch.full_like(q, math.nan), news)
    y, z = torch.empty_like(q[:3]), torch.empty_like(q[:3])
    ops.cache_attention(q[:3], c.cache, c.scale, c.tables, c.lengths, y, c.work)
    ops.pages_compact(c.tables, c.refs, c.cache[None], c.scale[None], c.work)
    assert sorted(c.tables[c.tables >= 0].tolist()) == [0, 1, 2, 3, 4, 5]
    ops.cache_attention(q[:3], c.cache, c.scale, c.tables, c.lengths, z, c.work)
    assert torch.equal(y, z) and c.errors() == _lib.LORA_OK


@pytest.mark.parametrize("entry", [-1, 10 ** 6, -2 ** 31])
@pytest.mark.parametrize("news", [None, [1, 40]], ids=["single", "chunks"])
def test_a_missing_page_is_left_out_and_counted(entry, news):
    c = Cache([200, 200], 2, 64, 16)
    q = rows(2 if news is None else sum(news), 4 * 64, BF16, gen(17))
    y, want = torch.zeros_like(q), torch.zeros_like(q)
    starts = None if news is None else starts_of(news)
    kept = c.tables.clone()
    c.tables[1, 3] = entry
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, y, c.work, starts=starts)
    assert c.errors() == _lib.LORA_ERR_BAD_INDEX and c.errors() == _lib.LORA_OK
    # as if the page's keys were far below all others: scores of -inf by a window of its own
    c.tables.copy_(kept)
    group = 2
    t = 0
    for b, n in enumerate([1, 1] if news is None else news):
        for h in range(2):
            k, v = c.kv(b, h)
            j = torch.arange(200, device="cuda")
            qq = q[t:t + n, h * group * 64:(h + 1) * group * 64].double().reshape(n, group, 64)
            a = torch.einsum("ngd,jd->ngj", qq, k) / 8
            i = 200 - n + torch.arange(n, device="cuda")[:, None, None]
            hide = (j > i) | ((j // 16 == 3) & (b == 1))
            o = torch.softmax(a.masked_fill(hide, -math.inf), -1) @ v
            err = (y[t:t + n, h * group * 64:(h + 1) * group * 64].double().reshape(n, group, 64) - o).abs().max()
            assert err < 0.02 * o.abs().max()
        t += n


def test_a_length_past_the_table_is_cut():
    c = Cache([64, 30], 1, 64, 16, more_places=0)
    q = rows(2, 64, BF16, gen(18))
    y, z = torch.zeros_like(q), torch.zeros_like(q)
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, y, c.work)
    c.lengths[0] = 2 ** 31 - 1
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, z, c.work)
    assert torch.equal(y, z)
    c.lengths[0] = -5
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, z, c.work)
    assert (z[0] == 0).all() and torch.equal(y[1], z[1])


@pytest.mark.parametrize("starts", [[0, 3, 2, 9], [-4, 3, 5, 9], [0, 4, 6, 1000], [5, 5, 5, 5], [9, 0, 9, 0]], ids=str)
def test_starts_out_of_order_stay_in_bounds(starts):
    c = Cache([50, 60, 70], 2, 64, 16)
    whole = torch.full((40, 256), 3.0, dtype=BF16, device="cuda")
    q, y = rows(9, 256, BF16, gen(19)), whole[16:25]
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, y, c.work, starts=ints(starts))
    torch.cuda.synchronize()
    assert (whole[:16] == 3).all() and (whole[25:] == 3).all()
    ops.cache_write(q[:, :128], q[:, 128:], c.cache, c.scale, c.tables, c.lengths, c.work, starts=ints(starts))
    torch.cuda.synchronize()


@pytest.mark.parametrize("group", [1, 4])
def test_descending_starts_of_many_rows_end_and_are_counted(group):
    """Sequences of many tiles, whose places a bisection and a walk would not agree on."""
    B, T = 12, 4000
    c = Cache([900] * B, 2, 64, 16)
    whole = torch.full((T + 32, 2 * group * 64), 3.0, dtype=BF16, device="cuda")
    q, y = rows(T, 2 * group * 64, BF16, gen(20)), whole[16:T + 16]
    order = [0, 500, 100, 700, 300, 2000, 900, 3100, 1500, 3900, 2500, 4000, 3300]
    for starts in (order, order[::-1], [0, 2, 1, 3, 2, 4, 3, 5, 4, 4000, 10, 4000, 0]):
        ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, y, c.work, starts=ints(starts))
        torch.cuda.synchronize()
        assert ops.check_errors(c.work) == _lib.LORA_ERR_BAD_INDEX
        assert (whole[:16] == 3).all() and (whole[T + 16:] == 3).all()
        # the workspace is as it was: a good call's results hold
        news = [9] * B
        z = torch.empty(9 * B, 2 * group * 64, dtype=BF16, device="cuda")
        ops.cache_attention(q[:9 * B], c.cache, c.scale, c.tables, c.lengths, z, c.work, starts=starts_of(news))
        assert ops.check_errors(c.work) == _lib.LORA_OK
        one = torch.empty_like(z)
        ops.cache_attention(q[:9 * B], c.cache, c.scale, c.tables, c.lengths, one,
                            ops.cache_workspace(c.cache.shape[0], 64), starts=starts_of(news))
        assert torch.equal(z, one)


# ---------------------------------------------------------------- the write
def grid():
    return torch.tensor([m * 2.0 ** -9 for m in range(8)] +
                        [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1], dtype=torch.float64, device="cuda")


def round_e4m3(v):
    g = grid()
    mid = (g[1:] + g[:-1]) / 2
    lo, hi = torch.bucketize(v.abs(), mid), torch.bucketize(v.abs(), mid, right=True)
    code = torch.where(lo != hi, lo + lo % 2, lo)
    return torch.where(v.isnan(), v, torch.copysign(g[code], v))


def write_by_hand(c, k, v, news):
    """The cache and scales after the write, by the formula, token by token."""
    cache, scale = c.cache.double(), c.scale.double()
    x = torch.stack([k, v], 1).double().view(-1, 2, c.H, c.dim)
    t = 0
    for b, n in enumerate(news):
        length = max(c.lens[b], 0)
        for at in range(max(length - n, 0) // c.page, up(length, c.page)):
            first, last = max(at * c.page, length - n, 0), min((at + 1) * c.page, length)
            if first >= last:
                continue
            p = int(c.tables[b, at])
            new = x[t + first - (length - n):t + last - (length - n)].permute(1, 2, 0, 3)
            a = new.abs().amax((2, 3))
            s = torch.exp2(torch.ceil(torch.log2(a.clamp_min(2.0 ** -80) / 448)).clamp(-32, 32))
            s = torch.where((a <= 448 * s / 2) & (s > 2.0 ** -32), s / 2, torch.where((a > 448 * s) & (s < 2.0 ** 32), s * 2, s))
            s = torch.where(a.isfinite(), s, math.nan)
            begun = first - at * c.page
            if begun:
                old = scale[p]
                s = torch.where(old.isnan() | s.isnan(), math.nan, torch.maximum(old, s))
                redo = round_e4m3(cache[p, :, :, :begun] * (old / s)[..., None, None])
                cache[p, :, :, :begun] = torch.where((s == old)[..., None, None] | s.isnan()[..., None, None], cache[p, :, :, :begun], redo)
            scale[p] = s
            q = new / s[..., None, None]
            cache[p, :, :, begun:begun + last - first] = round_e4m3(q.clamp(-448, 448))
        t += n
    return cache, scale


def same(a, b):
    return torch.equal(a.double().nan_to_num(12345.0), b.nan_to_num(12345.0))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [16, 64, 80, 96, 128, 176, 256])
@pytest.mark.parametrize("page,H", [(16, 2), (32, 3), (64, 1), (128, 5)])
@pytest.mark.parametrize("news", [None, [1, 0, 15, 1, 100, 17, 33, 128, 2, 1]], ids=["single", "chunks"])
def test_write(dtype, dim, page, H, news):
    lens = [1, 0, 15, 16, 300, 17, 33, 128, 130, 2 * page + 1]
    c = Cache(lens, H, dim, page, seed=dim + H, scales=(-14, 2))
    T = len(lens) if news is None else sum(news)
    x = rows(T, 2 * H * dim, dtype, gen(20), extra=24, more=0 if news is None else 3)
    x = (x.float() * torch.exp(torch.randn(x.shape[0], 1, generator=gen(21), device="cuda"))).to(dtype)
    k, v = x[:, :H * dim], x[:, H * dim:2 * H * dim]
    want = write_by_hand(c, k, v, [1] * len(lens) if news is None else news)
    ops.cache_write(k, v, c.cache, c.scale, c.tables, c.lengths, c.work, starts=None if news is None else starts_of(news))
    assert same(c.scale, want[1]) and same(c.cache, want[0])
    assert c.errors() == _lib.LORA_OK


@pytest.mark.parametrize("dtype", TYPES)
def test_write_scales_at_their_borders(dtype):
    """Maxima at and next to 448 times a power of two, zeros, the type's ends."""
    vals = [0.0, 448.0, 449.0 if dtype is F16 else 450.0, 447.5 if dtype is F16 else 446.0, 1.75, 1.7510 if dtype is F16 else 1.7578125, 2.0 ** -20,
            torch.finfo(dtype).max, torch.finfo(dtype).tiny, torch.finfo(dtype).smallest_normal / 4, 896.0, 3.5, 1e-7]
    c = Cache([1] * len(vals), 1, 16, 16, fill=False)
    k = torch.zeros(len(vals), 16, device="cuda")
    k[:, 3], k[:, 5] = torch.tensor(vals, device="cuda"), -torch.tensor(vals, device="cuda") / 3
    k = k.to(dtype)
    want = write_by_hand(c, k, k, [1] * len(vals))
    ops.cache_write(k, k.clone(), c.cache, c.scale, c.tables, c.lengths, c.work)
    assert same(c.scale, want[1]) and same(c.cache, want[0])


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_write_of_no_number_spoils_its_scale_alone(what):
    c = Cache([40, 40], 2, 64, 16)
    k = rows(6, 128, BF16, gen(22))
    k[1, 70] = what                                     # sequence 0, head 1
    want = write_by_hand(c, k, k, [3, 3])
    ops.cache_write(k, k, c.cache, c.scale, c.tables, c.lengths, c.work, starts=ints([0, 3, 6]))
    assert same(c.scale, want[1])
    p = int(c.tables[0, 2])
    assert c.scale[p, :, 1].isnan().all() and not c.scale[p, :, 0].isnan().any()
    good = torch.ones(c.P, dtype=torch.bool, device="cuda")
    good[p] = False
    assert same(c.cache[good], want[0][good])
    c.lens = [41, 41]                                   # a NaN stays
    c.lengths += 1
    ops.cache_write(k[4:], k[4:], c.cache, c.scale, c.tables, c.lengths, c.work)
    assert c.scale[p, :, 1].isnan().all()


def test_write_again_after_a_shorter_length():
    """Tokens that were taken back are written over; the scale does not shrink."""
    c = Cache([20], 1, 64, 16, fill=False)
    big, small = torch.full((20, 64), 100.0, dtype=BF16, device="cuda"), torch.ones(3, 64, dtype=BF16, device="cuda")
    ops.cache_write(big, big, c.cache, c.scale, c.tables, c.lengths, c.work, starts=ints([0, 20]))
    c.lengths.fill_(19)
    ops.cache_write(small, small, c.cache, c.scale, c.tables, c.lengths, c.work, starts=ints([0, 2]))
    p = int(c.tables[0, 1])
    assert (c.scale[p] == 0.25).all()                   # 100 / 448 < 2^-2
    got = c.cache[p, 0, 0].float() * 0.25
    # 400 lies halfway between 384 = 12 * 32 and 416 = 13 * 32: to the even one
    assert (got[0] == 96).all() and (got[1:3] == 1).all()


def test_write_without_its_page_is_left_out_and_counted():
    c = Cache([40, 40], 2, 64, 16)
    k = rows(2, 128, BF16, gen(23))
    c.tables[0, 2] = -1
    before = c.cache.clone(), c.scale.clone()
    want = write_by_hand(c, k[1:], k[1:], [0, 1])
    ops.cache_write(k, k, c.cache, c.scale, c.tables, c.lengths, c.work)
    assert c.errors() == _lib.LORA_ERR_BAD_INDEX
    assert same(c.cache, want[0]) and same(c.scale, want[1]) and not same(c.scale, before[1].double())
    c.tables[0, 2] = c.P
    ops.cache_write(k, k, c.cache, c.scale, c.tables, c.lengths, c.work)
    c.lengths[0] = 1000                                 # past the table
    ops.cache_write(k, k, c.cache, c.scale, c.tables, c.lengths, c.work)
    assert c.errors() == _lib.LORA_ERR_BAD_INDEX


# ---------------------------------------------------------------- pages
class Pool:
    """The pages' bookkeeping by hand."""

    def __init__(self, tables, lengths, refs, page):
        self.t, self.n, self.r, self.page, self.M = tables.tolist(), lengths.tolist(), refs.tolist(), page, tables.shape[1]

    def free_pages(self):
        return [p for p, r in enumerate(self.r) if r <= 0]

    def extend(self):
        free, missed = self.free_pages(), 0
        for b, n in enumerate(self.n):
            need = up(max(n, 0), self.page)
            held = next((i for i, p in enumerate(self.t[b]) if p < 0), self.M)
            missed += max(need - self.M, 0)
            for i in range(held, min(need, self.M)):
                if free:
                    self.t[b][i] = free.pop(0)
                    self.r[self.t[b][i]] = 1
                else:
                    missed += 1
        return missed

    def free(self, seqs):
        for b in seqs:
            for p in self.t[b]:
                if p >= 0:
                    self.r[p] -= 1
            self.t[b], self.n[b] = [-1] * self.M, 0

    def fork(self, src, dst):
        free, copies, missed, begun_n = self.free_pages(), [], 0, list(self.n)
        for s, d in zip(src, dst):
            if not (0 <= s < len(self.n) and 0 <= d < len(self.n)) or s == d or begun_n[d] or self.t[d][0] >= 0 or self.n[d]:
                missed += 1
                continue
            full, begun = divmod(begun_n[s], self.page)
            if begun and not free:
                missed += 1
                continue
            self.t[d][:full] = self.t[s][:full]
            for p in self.t[s][:full]:
                self.r[p] += 1
            if begun:
                p = free.pop(0)
                copies.append((self.t[s][full], p))
                self.t[d][full], self.r[p] = p, 1
            self.n[d] = begun_n[s]
        return copies, missed

    def compact(self):
        live = [p for p, r in enumerate(self.r) if r > 0]
        n = len(live)
        holes, high = [p for p in range(n) if self.r[p] <= 0], [p for p in reversed(live) if p >= n]
        moves = list(zip(high, holes))
        names = dict(moves)
        self.t = [[names.get(p, p) for p in row] for row in self.t]
        for s, d in moves:
            self.r[d], self.r[s] = self.r[s], 0
        self.r = [max(r, 0) for r in self.r]
        return moves, n

    def check(self, tables, lengths, refs):
        assert tables.tolist() == self.t
        assert refs.tolist() == self.r
        if lengths is not None:
            assert lengths.tolist() == self.n


def layers(L, P, H, page, dim, seed=0):
    g = gen(seed)
    cache = torch.randint(0, 256, (L, P, 2, H, page, dim), dtype=torch.uint8, generator=g, device="cuda").view(FP8)
    return cache, torch.randn(L, P, 2, H, generator=g, device="cuda")


def moved(cache, scale, moves):
    cache, scale = cache.view(torch.uint8).clone(), scale.clone()
    old_c, old_s = cache.clone(), scale.clone()
    for s, d in moves:
        cache[:, d], scale[:, d] = old_c[:, s], old_s[:, s]
    return cache, scale


def bookkeeping(lens, P, page, M, seed=0, share=0.0):
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(P, generator=g).tolist()
    t, r = [[-1] * M for _ in lens], [0] * P
    for b, n in enumerate(lens):
        for i in range(up(n, page)):
            t[b][i] = order.pop()
            r[t[b][i]] = 1
    return ints(t), ints(lens), ints(r)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("P,lens,more", [
    (5, [0, 0], [1, 1]), (64, [3, 0, 17, 16, 15], [4, 40, 17, 17, 31]), (1, [0], [16]), (4096, [100] * 70, [900] * 70),
    (30011, [0, 5] * 300, [700, 6] * 300), (10000, [1] * 5000, [17] * 5000), (9000, [0, 0, 0], [30000, 1, 50000])])
def test_extend(page, P, lens, more):
    M = up(max(more), 16) + 1
    tables, lengths, refs = bookkeeping(lens, P, page, M, seed=P)
    lengths = ints(more)
    work = ops.cache_workspace(P, 64)
    pool = Pool(tables, lengths, refs, page)
    missed = pool.extend()
    ops.pages_extend(tables, lengths, refs, page, work)
    pool.check(tables, lengths, refs)
    assert ops.check_errors(work) == (_lib.LORA_ERR_BAD_INDEX if missed else _lib.LORA_OK)
    ops.pages_extend(tables, lengths, refs, page, work)   # nothing lacks, or nothing is left
    pool.check(tables, lengths, refs)


def test_extend_when_pages_or_places_run_out():
    tables, lengths, refs = bookkeeping([0, 0, 0], 7, 16, 3)
    lengths.copy_(ints([33, 200, 64]))                  # 3; 13 in 3 places; 4 in 3 places: 9 of 7
    work = ops.cache_workspace(7, 64)
    pool = Pool(tables, lengths, refs, 16)
    assert pool.extend() > 0
    ops.pages_extend(tables, lengths, refs, 16, work)
    pool.check(tables, lengths, refs)
    assert ops.check_errors(work) == _lib.LORA_ERR_BAD_INDEX


@pytest.mark.parametrize("seqs", [[0], [4, 1], [2, 2, 2], [0, 1, 2, 3, 4], [3]])
def test_free(seqs):
    tables, lengths, refs = bookkeeping([40, 100, 16, 0, 7], 40, 16, 9)
    tables[1, 0] = tables[0, 0]                         # shared
    refs[tables[0, 0].long()] = 2
    pool = Pool(tables, lengths, refs, 16)
    pool.free(seqs)
    work = ops.cache_workspace(40, 64)
    ops.pages_free(tables, lengths, refs, ints(seqs), work)
    pool.check(tables, lengths, refs)
    assert ops.check_errors(work) == _lib.LORA_OK


def test_free_of_no_such_row_or_uncounted_pages():
    tables, lengths, refs = bookkeeping([40, 100], 40, 16, 9)
    work = ops.cache_workspace(40, 64)
    before = tables.clone()
    ops.pages_free(tables, lengths, refs, ints([-1, 2, 2 ** 31 - 1]), work)
    assert torch.equal(tables, before) and ops.check_errors(work) == _lib.LORA_ERR_BAD_INDEX
    refs[tables[0, 0].long()] = 0
    ops.pages_free(tables, lengths, refs, ints([0]), work)
    assert ops.check_errors(work) == _lib.LORA_ERR_BAD_INDEX and int(refs.min()) == 0
    tables[1, 1] = 40
    ops.pages_free(tables, lengths, refs, ints([1]), work)
    assert ops.check_errors(work) == _lib.LORA_ERR_BAD_INDEX and (tables == -1).all()


@pytest.mark.parametrize("L,H,page,dim", [(1, 1, 16, 16), (3, 2, 32, 80), (2, 3, 128, 64)])
@pytest.mark.parametrize("lens,src,dst", [
    ([20, 0], [0], [1]), ([32, 0], [0], [1]), ([1, 0, 0, 0], [0, 0, 0], [3, 1, 2]), ([0, 0], [0], [1]),
    ([100, 50, 0, 0, 0, 0, 128], [0, 1, 6, 0], [5, 2, 4, 3]),
    ([20, 30, 0], [0, 1], [2, 2]),                       # one row twice: the first pair has it
    ([20, 30, 0], [0, 1, 5, -1, 0], [0, 0, 2, 2, 7]),    # itself, a row that holds something, no such rows
    ([20, 0, 0], [0, 1], [1, 2]),                        # a row that another pair fills is still empty
], ids=str)
def test_fork(L, H, page, dim, lens, src, dst):
    P = sum(up(n, page) for n in lens) + 5
    tables, lengths, refs = bookkeeping(lens, P, page, up(max(lens), page) + 1, seed=len(lens))
    cache, scale = layers(L, P, H, page, dim)
    pool = Pool(tables, lengths, refs, page)
    copies, missed = pool.fork(src, dst)
    want = moved(cache, scale, copies)
    work = ops.cache_workspace(P, dim)
    ops.pages_fork(tables, lengths, refs, ints(src), ints(dst), cache, scale, work)
    pool.check(tables, lengths, refs)
    assert torch.equal(cache.view(torch.uint8), want[0]) and torch.equal(scale, want[1])
    assert ops.check_errors(work) == (_lib.LORA_ERR_BAD_INDEX if missed else _lib.LORA_OK)


def test_fork_when_pages_run_out():
    lens = [20, 32, 0, 0, 0, 0]
    tables, lengths, refs = bookkeeping(lens, 5, 16, 3)
    cache, scale = layers(2, 5, 1, 16, 16)
    pool = Pool(tables, lengths, refs, 16)
    src, dst = [0, 0, 1, 0], [2, 3, 4, 5]                # one page is free; the one that shares only still goes
    copies, missed = pool.fork(src, dst)
    assert missed == 2
    want = moved(cache, scale, copies)
    work = ops.cache_workspace(5, 16)
    ops.pages_fork(tables, lengths, refs, ints(src), ints(dst), cache, scale, work)
    pool.check(tables, lengths, refs)
    assert torch.equal(cache.view(torch.uint8), want[0]) and ops.check_errors(work) == _lib.LORA_ERR_BAD_INDEX


def test_fork_of_many_pairs():
    lens = [37 * i % 300 + 1 for i in range(50)] + [0] * 1500
    P = sum(up(n, 16) for n in lens) + 1600
    tables, lengths, refs = bookkeeping(lens, P, 16, 20, seed=5)
    cache, scale = layers(1, P, 1, 16, 16)
    src, dst = [i * 7 % 50 for i in range(1500)], [50 + (i * 11) % 1500 for i in range(1500)]
    pool = Pool(tables, lengths, refs, 16)
    copies, missed = pool.fork(src, dst)
    assert missed == 0
    want = moved(cache, scale, copies)
    work = ops.cache_workspace(P, 16)
    ops.pages_fork(tables, lengths, refs, ints(src), ints(dst), cache, scale, work)
    pool.check(tables, lengths, refs)
    assert torch.equal(cache.view(torch.uint8), want[0]) and torch.equal(scale, want[1])


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
@pytest.mark.parametrize("P,lens", [(1, [0]), (1, [5]), (10, [160]), (10, [0, 0]), (64, [100, 3, 0, 60]), (5000, [33] * 700),
                                    (4096, [16] * 2048), (9001, [100] * 1000)], ids=lambda v: str(v)[:20])
def test_compact(in_place, P, lens):
    L, H, page, dim = 2, 2, 16, 48
    tables, lengths, refs = bookkeeping(lens, P, page, up(max(lens), page) + 1, seed=P)
    if lens[0] and len(lens) > 1:                        # a shared page
        tables[1, 0] = tables[0, 0]
        refs = torch.bincount(tables[tables >= 0].long(), minlength=P).to(torch.int32)
    cache, scale = layers(L, P, H, page, dim)
    pool = Pool(tables, lengths, refs, page)
    moves, n = pool.compact()
    want = moved(cache, scale, moves)
    work, live = ops.cache_workspace(P, dim), ints([-7])
    kept = tables.clone(), refs.clone()
    ot, o = (tables, refs) if in_place else (torch.full_like(tables, 99), torch.full_like(refs, 99))
    if in_place:
        ops.pages_compact(tables, refs, cache, scale, work)
    else:
        ops.pages_compact(tables, refs, cache, scale, work, out_tables=ot, out_refs=o, n_live=live)
        assert int(live) == n and torch.equal(tables, kept[0]) and torch.equal(refs, kept[1])
    pool.check(ot, None, o)
    assert torch.equal(cache.view(torch.uint8), want[0]) and torch.equal(scale, want[1])
    assert ops.check_errors(work) == _lib.LORA_OK


def test_compact_of_an_entry_that_nobody_counts():
    tables, lengths, refs = bookkeeping([40], 10, 16, 4)
    free = [p for p in range(10) if int(refs[p]) == 0]
    tables[0, 3] = free[0]
    cache, scale = layers(1, 10, 1, 16, 16)
    work = ops.cache_workspace(10, 16)
    ops.pages_compact(tables, refs, cache, scale, work)
    assert int(tables[0, 3]) == -1 and sorted(tables[0, :3].tolist()) == [0, 1, 2]
    assert ops.check_errors(work) == _lib.LORA_ERR_BAD_INDEX
    tables[0, 3] = 10
    ops.pages_compact(tables, refs, cache, scale, work)
    assert ops.check_errors(work) == _lib.LORA_ERR_BAD_INDEX


@pytest.mark.parametrize("L,P,H,page,dim,n", [(1, 2, 1, 16, 16, 1), (4, 40, 3, 16, 80, 17), (2, 64, 8, 128, 128, 30), (32, 16, 1, 32, 256, 8)])
def test_copy(L, P, H, page, dim, n):
    cache, scale = layers(L, P, H, page, dim, seed=n)
    order = torch.randperm(P, generator=gen(n), device="cuda").to(torch.int32)
    src, dst = order[:n].contiguous(), order[n:2 * n].contiguous()
    src[:n // 2] = src[0].clone()                        # one source many times
    want = moved(cache, scale, list(zip(src.tolist(), dst.tolist())))
    work = ops.cache_workspace(P, dim)
    ops.pages_copy(cache, scale, src, dst, work)
    assert torch.equal(cache.view(torch.uint8), want[0]) and torch.equal(scale, want[1])
    bad = ints([-1, 0, P, 1, 0])
    ops.pages_copy(cache, scale, bad, ints([0, P, 1, -5, 0]), work)   # no pages; a page onto itself
    assert torch.equal(cache.view(torch.uint8), want[0]) and ops.check_errors(work) == _lib.LORA_ERR_BAD_INDEX
