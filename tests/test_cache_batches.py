"""GPU tests of the cache's attention by what a batch is made of: long and short
sequences side by side, so that a CTA goes through dozens of items of different
sizes.  References and tolerances are those of test_cache_ops."""
import math
import random

import pytest
import torch

from gather_matmul_b200 import _lib, ops
from test_cache_ops import BF16, F16, Cache, attend, gen, rows, starts_of

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
