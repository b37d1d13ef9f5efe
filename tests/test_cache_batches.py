"""GPU tests of the cache's attention by what a batch is made of: long and short
sequences side by side, so that a CTA goes through dozens of items of different
sizes.  References and tolerances are those of test_cache_ops."""
import math
import random

import pytest
import torch

from gather_matmul_b200 import _lib, ops
from test_cache_ops import BF16, F16, Cache, attend, check_attention, gen, rows, starts_of
from test_cache_paths import Model

pytestmark = pytest.mark.gpu


def uniform(n, top, seed):
    r = random.Random(seed)
    return [r.randint(1, top) for _ in range(n)]


# Batches in which a CTA meets dozens of items of at most 128 rows (queries times the heads that share
# a k/v head) behind one of more: new tokens, lengths, k/v heads, q heads of each.
MIXED = {
    "prompts of 300": ([300] * 128, [300] * 128, 32, 1),
    "prompts of up to 256": (uniform(200, 256, 1), None, 32, 1),
    "prompts of up to 64": (uniform(1024, 64, 2), None, 8, 4),
    "a chunk, then 5 tokens": ([2048] + [1] * 5, [16384] + [100] * 5, 8, 4),
    "a chunk, then 12 tokens": ([2048] + [1] * 12, [16384] + [100] * 12, 8, 4),
}


@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("batch", list(MIXED))
def test_many_small_items_behind_a_large_one(batch, dim, dtype):
    news, lens, H, group = MIXED[batch]
    c = Cache(news if lens is None else lens, H, dim, 64, seed=dim)
    q = rows(sum(news), H * group * dim, dtype, gen(41))
    y = torch.full_like(q, math.nan)
    attend(c, q, y, news)
    # the workspace is as it was: the same bits again, and in one that is new
    for work in (c.work, ops.cache_workspace(c.P, dim)):
        z = torch.full_like(q, math.nan)
        ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, z, work, starts=starts_of(news))
        assert torch.equal(y, z) and ops.check_errors(work) == _lib.LORA_OK
    # sequences that many CTAs share, joined by counters in the same workspace
    d = Cache([9000, 700], H, dim, 64, seed=42)
    assert d.P <= c.P
    d.work = c.work
    q = rows(300, H * group * dim, dtype, gen(42))
    attend(d, q, torch.full_like(q, math.nan), [290, 10])


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, F16)])
def test_thousands_of_steps_without_a_second_tile(dim, dtype):
    """Most items have rows for one tile only, now and then one has for both: the warp that issues the
    second tile's products runs through the plan with nothing to wait for but the keys."""
    r = random.Random(45)
    news = [r.randint(20, 32) if i % 23 else r.randint(65, 80) for i in range(700)]
    lens = [n + r.randint(0, 600) for n in news]
    c = Cache(lens, 4, dim, 32, seed=45)
    q = rows(sum(news), 16 * dim, dtype, gen(45))
    y = torch.full_like(q, math.nan)
    attend(c, q, y, news)
    starts = starts_of(news)
    for _ in range(10):
        z = torch.full_like(q, math.nan)
        ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, z, c.work, starts=starts)
        assert torch.equal(y, z)
    assert c.errors() == _lib.LORA_OK


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("softmax_scale", [None, 1e-20, 3.0])
@pytest.mark.parametrize("news", [None, [300, 7, 1, 64]], ids=["single", "chunks"])
def test_zeros_give_the_mean_of_the_values(news, softmax_scale, dim):
    """Rows of zeros over keys of zeros, whose factors are the smallest there are: every score is 0, masked or not."""
    c = Cache([300, 500, 129, 64], 2, dim, 16, seed=43)
    held = c.refs.bool()
    c.cache.view(torch.uint8)[held, 0] = 0
    c.scale[held, 0] = 2.0 ** -32
    T = 4 if news is None else sum(news)
    q = torch.zeros(T, 4 * dim, dtype=BF16, device="cuda")
    attend(c, q, torch.full_like(q, math.nan), news, softmax_scale=softmax_scale)
    q[::3] = rows(len(q[::3]), 4 * dim, BF16, gen(43))        # some rows of numbers among them
    attend(c, q, torch.full_like(q, math.nan), news, softmax_scale=softmax_scale)
    attend(c, q, torch.full_like(q, math.nan), news, softmax_scale=softmax_scale, window=50)


def test_a_layer_s_step_on_zeros_gives_zeros():
    """As a server warms up: x = 0 gives q = k = v = 0."""
    m = Model(1, 8, 2, 128, 16, 64, 3, 12, seed=9)
    news = [100, 3, 40]
    m.lengths += torch.tensor(news, dtype=torch.int32, device="cuda")
    m.extend()
    T = sum(news)
    buf = m.buffers(T)
    m.run(torch.zeros(T, m.K, dtype=m.dtype, device="cuda"), torch.full((T,), -1, dtype=torch.int32, device="cuda"),
          torch.arange(T, device="cuda"), buf, starts_of(news))
    assert (buf[0][0] == 0).all() and (buf[0][1] == 0).all()
    assert ops.check_errors(m.work) == _lib.LORA_OK


@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("news,lens,window,place", [
    ([5, 3], [99, 40], 0, 6),                   # few rows: positions 94 and 95 come before page 6
    ([5, 3], [101, 40], 20, 4),                 # 99 and 100 are past the window of page 4
    ([300, 7], [300, 90], 0, 12),               # many: the first 192 rows of a prompt
    ([300, 7], [400, 90], 64, 10),              # before the page, and past its window
    ([1, 200], [200, 200], 0, 12),              # the other sequence's last page
], ids=str)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_page_of_nan_spoils_only_the_queries_that_see_it(news, lens, window, place, side, dim):
    c = Cache(lens, 2, dim, 16, seed=46)
    q, starts = rows(sum(news), 4 * dim, BF16, gen(46)), starts_of(news)
    y = torch.full_like(q, math.nan)
    attend(c, q, y, news, window=window)
    b = 0 if place * 16 < lens[0] and news[0] > 1 else 1
    page = int(c.tables[b, place])
    kept = c.cache.view(torch.uint8)[page, side, 1].clone(), c.scale[page, side, 1].clone()
    c.cache.view(torch.uint8)[page, side, 1] = 0x7F
    c.scale[page, side, 1] = math.nan
    z = torch.full_like(q, 7.0)
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, z, c.work, starts=starts, window=window)
    i = lens[b] - news[b] + torch.arange(news[b], device="cuda")
    last = torch.minimum(i, torch.tensor(place * 16 + 15, device="cuda"))
    sees = (last >= place * 16) & ((last > i - window) if window else (i >= 0))
    assert sees.any() and (not sees.all() or news[0] == 1)
    first = sum(news[:b])
    want = torch.zeros(sum(news), 4, dtype=torch.bool, device="cuda")
    want[first:first + news[b], 2:] = sees[:, None]
    bad = z.view(-1, 4, dim).isnan()
    assert torch.equal(bad.any(2), want) and torch.equal(bad.all(2), want)
    # all others are right
    c.cache.view(torch.uint8)[page, side, 1], c.scale[page, side, 1] = kept
    check_attention(c, q, torch.where(z.isnan(), y, z), news, window=window)
    assert c.errors() == _lib.LORA_OK


@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_a_token_of_no_number_leaves_the_tokens_before_its_page(what):
    """Written and attended over in one step, as a prompt is."""
    n, at, H, dim = 200, 150, 2, 128
    c = Cache([n], H, dim, 16, seed=47)
    x = rows(n, 2 * H * dim, BF16, gen(47))
    q = rows(n, 4 * dim, BF16, gen(48))
    x[at, H * dim + 3] = what                                # v of head 0
    x[at + 20, dim + 5] = what                               # k of head 1
    ops.cache_write(x[:, :H * dim], x[:, H * dim:], c.cache, c.scale, c.tables, c.lengths, c.work, starts=starts_of([n]))
    y = torch.empty_like(q)
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, y, c.work, starts=starts_of([n]))
    bad = y.view(n, 4, dim).isnan()
    assert bad[at // 16 * 16:, :2].all() and not bad[:at // 16 * 16, :2].any()
    assert bad[(at + 20) // 16 * 16:, 2:].all() and not bad[:(at + 20) // 16 * 16, 2:].any()


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 40, 2 ** 30, 41, 3])
@pytest.mark.parametrize("news,lens", [([9, 41, 200, 12], [3, 40, 150, 0]), ([7], [2]), ([300, 4], [299, 1])], ids=str)
@pytest.mark.parametrize("dim,group", [(64, 2), (128, 1), (192, 4)])
def test_windows_of_any_size_over_fewer_tokens_than_are_new(window, news, lens, dim, group):
    """2^31 - 1 is a caller's "no window"; queries before the first token see nothing and get zeros."""
    c = Cache(lens, 2, dim, 16, seed=49)
    q = rows(sum(news), 2 * group * dim, F16, gen(49))
    attend(c, q, torch.full_like(q, math.nan), news, window=window)
    if window >= 2 ** 30:
        y, z = torch.empty_like(q), torch.full_like(q, math.nan)
        ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, y, c.work, starts=starts_of(news))
        ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, z, c.work, starts=starts_of(news), window=window)
        assert torch.equal(y, z)


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("past", [1, 37, 300, 2 ** 30])
@pytest.mark.parametrize("news", [None, [2, 3], [300, 2]], ids=["single", "few", "chunks"])
def test_a_length_past_the_table_is_counted_and_its_queries_keep_their_positions(news, past, window):
    """The tokens behind the table are left out; the new ones are the length's last, not the table's."""
    dim, held = 64, 320
    c = Cache([held, 50], 2, dim, 16, seed=50, more_places=0)
    assert c.M * 16 == held
    T = 2 if news is None else sum(news)
    q = rows(T, 4 * dim, BF16, gen(50))
    y = torch.full_like(q, math.nan)
    starts = None if news is None else starts_of(news)
    c.lengths[0] = held + past
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, y, c.work, starts=starts, window=window)
    assert c.errors() == _lib.LORA_ERR_BAD_INDEX and c.errors() == _lib.LORA_OK
    n = 1 if news is None else news[0]
    i = held + past - n + torch.arange(n, device="cuda")[:, None, None]
    j = torch.arange(held, device="cuda")
    seen = (j <= i) & ((j > i - window) if window else (j >= 0))
    for h in range(2):
        k, v = c.kv(0, h)
        qq = q[:n, 2 * h * dim:2 * (h + 1) * dim].double().view(n, 2, dim)
        a = (torch.einsum("ngd,jd->ngj", qq, k) * dim ** -0.5).masked_fill(~seen, -math.inf)
        p = torch.softmax(a, -1).masked_fill(~seen.any(-1, keepdim=True), 0.0)
        want, got = p @ v, y[:n, 2 * h * dim:2 * (h + 1) * dim].double().view(n, 2, dim)
        # bf16 results; weights 2^-11; logits' sums, maxima and exponentials, 4 e of test_cache_ops: below 2^-10,
        # as sum |q k| / 8 is below 20
        tol = 2.0 ** -8 * 1.001 * want.abs() + (2.0 ** -11 + 2.0 ** -10) * (p @ v.abs()) + 2.0 ** -25
        assert (torch.einsum("ngd,jd->ngj", qq.abs(), k.abs()) / 8).max() < 20
        assert ((got - want).abs() <= tol).all()
    # the other sequence is as without
    c.lengths[0] = held
    z = torch.full_like(q, math.nan)
    ops.cache_attention(q, c.cache, c.scale, c.tables, c.lengths, z, c.work, starts=starts, window=window)
    assert c.errors() == _lib.LORA_OK
    check_attention(c, q, z, [1, 1] if news is None else news, window=window)
    c.lens[0] = 0                                            # looked at above
    check_attention(c, q, torch.cat([torch.zeros_like(y[:n]), y[n:]]), [1, 1] if news is None else news, window=window)


@pytest.mark.parametrize("new", [3, 40, 300])
@pytest.mark.parametrize("at", ["first", "last", "between"])
def test_sequences_without_new_tokens_have_no_places(new, at):
    """The division among CTAs passes over them: many, with tokens of their own, around two that have new ones."""
    none = [0] * 200
    news = {"first": none + [new, new], "last": [new, new] + none, "between": [new] + none + [new]}[at]
    c = Cache([900 if n else 33 for n in news], 2, 64, 16, seed=51)
    q = rows(sum(news), 8 * 64, F16, gen(51))
    y = torch.full_like(q, math.nan)
    attend(c, q, y, news)
    two = [i for i, n in enumerate(news) if n]
    z = torch.full_like(q, math.nan)
    ops.cache_attention(q, c.cache, c.scale, c.tables[two].contiguous(), c.lengths[two].contiguous(), z, c.work,
                        starts=starts_of([new, new]))
    check_attention(c, q, z, news)


@pytest.mark.parametrize("news", [None, [2, 9]], ids=["single", "chunks"])
@pytest.mark.parametrize("s", [7, 13, 15, 41, 47, 51, 55, 61, 63])
def test_write_to_pages_begun_with_a_factor_that_is_no_power_of_two(s, news):
    """Halfway values: s (17 .. 31) / s lies between two codes, and goes to the even one; x (1 / s) in fp32 may lie beside it."""
    dim = 64
    c = Cache([30, 43], 1, dim, 16, seed=52)
    at = [int(c.tables[0, 1]), int(c.tables[1, 2])]
    c.scale[at] = 2.0 ** -4 * s
    old = c.cache.clone()
    T = 2 if news is None else sum(news)
    m = torch.arange(17, 33, 2, device="cuda").repeat(T, dim // 8).double()
    x = (m * s / 16).to(F16)
    x[:, 1::2] *= -1
    assert torch.equal(x.double().abs(), m * s / 16)
    ops.cache_write(x, x, c.cache, c.scale, c.tables, c.lengths, c.work, starts=None if news is None else starts_of(news))
    assert (c.scale[at] == 2.0 ** -4 * s).all()
    # m = 16 + 2 i + 1 lies between 16 + 2 i and 16 + 2 i + 2: the multiple of 4
    want = torch.where(m % 4 == 1, m - 1, m + 1)
    want[:, 1::2] *= -1
    t = 0
    for b, n in enumerate([1, 1] if news is None else news):
        first = c.lens[b] - n
        for k in range(n):
            page, place = int(c.tables[b, (first + k) // 16]), (first + k) % 16
            if page == at[b]:
                assert torch.equal(c.cache[page, :, 0, place].double(), want[t + k].expand(2, dim)), (b, k)
        begun = first % 16
        assert torch.equal(c.cache.view(torch.uint8)[at[b], :, :, :begun], old.view(torch.uint8)[at[b], :, :, :begun])
        t += n
    assert c.errors() == _lib.LORA_OK


def test_extend_counts_lengths_past_their_tables_whatever_they_add_up_to():
    """64 sequences that lack 2^26 places each: 2^32 in all."""
    B, M, page = 64, 4, 16
    tables = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(B * M, dtype=torch.int32, device="cuda")
    lengths = torch.full((B,), ((1 << 26) + M) * page, dtype=torch.int32, device="cuda")
    work = ops.cache_workspace(B * M, 64)
    ops.pages_extend(tables, lengths, refs, page, work)
    assert torch.equal(tables.flatten(), torch.arange(B * M, dtype=torch.int32, device="cuda")) and (refs == 1).all()
    assert ops.check_errors(work) == _lib.LORA_ERR_BAD_INDEX
    ops.pages_extend(tables, lengths, refs, page, work)
    assert ops.check_errors(work) == _lib.LORA_ERR_BAD_INDEX


@pytest.mark.parametrize("dim,dtype", [(64, F16), (80, BF16), (128, F16), (256, BF16)])
@pytest.mark.parametrize("news", [None, [3, 2], [40, 60], [1, 300]], ids=["single", "few", "chunks", "mixed"])
def test_any_factors_in_both_kernels(news, dim, dtype):
    """Factors that are no powers of two, of k and of v, over a range of 2^20."""
    c = Cache([600, 301], 2, dim, 16, seed=53, scales=(-16, 4))
    c.scale *= torch.rand(c.scale.shape, generator=gen(53), device="cuda") + 0.5
    c.scale[:, 0] = (c.scale[:, 0].log2() / 4 - 6).exp2()     # logits of moderate size
    q = rows(2 if news is None else sum(news), 6 * dim, dtype, gen(54))
    attend(c, q, torch.full_like(q, math.nan), news)
    attend(c, q, torch.full_like(q, math.nan), news, window=100)
