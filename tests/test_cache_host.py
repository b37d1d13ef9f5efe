"""The host side of the paged 8-bit cache, without a GPU: workspace sizes and
refusals (no call here launches)."""
import math
import os
import re

import pytest
import torch

from gather_matmul_b200 import _lib, build, ops

HEADER = os.path.join(os.path.dirname(__file__), "..", "include", "lora.h")
FAKE = 0x10000   # a 256-byte aligned non-null address; never dereferenced
FAR = 1 << 40    # another, far from the first
INV, UNS, MIS = _lib.LORA_ERR_INVALID_ARG, _lib.LORA_ERR_UNSUPPORTED, _lib.LORA_ERR_MISALIGNED
BIG = 1 << 62


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.load()


def test_limits_are_the_header_s():
    src = open(HEADER).read()
    for name in ("LORA_MAX_PAGES", "LORA_MAX_SEQS", "LORA_MAX_FORKS"):
        text = re.search(rf"#define {name} (.+)", src).group(1)
        assert eval(text) == getattr(_lib, name)


def test_workspace_bytes(L):
    sizes = [L.lora_cache_workspace_bytes(p, 128) for p in (1, 64, 1000, 1 << 22)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    # three integers for each page, beside what does not depend on them
    assert abs(sizes[3] - sizes[2] - 12 * ((1 << 22) - 1000)) <= 3 * 256
    assert L.lora_cache_workspace_bytes(64, 256) > L.lora_cache_workspace_bytes(64, 64)
    for p, d in [(0, 128), (-1, 128), ((1 << 22) + 1, 128), (64, 0), (64, 24), (64, 272)]:
        assert L.lora_cache_workspace_bytes(p, d) == 0


def _write(L, dt=1, T=8, B=8, H=4, dim=64, page=16, P=100, M=9, k=FAKE, ldk=256, v=FAKE, ldv=256, cache=FAKE,
           scale=FAKE, tables=FAKE, lengths=FAKE, starts=None, work=FAKE, nb=BIG):
    return L.lora_cache_write(dt, T, B, H, dim, page, P, M, k, ldk, v, ldv, cache, scale, tables, lengths, starts,
                              work, nb, None)


SHAPES = [
    (dict(dt=2), INV), (dict(T=-1), INV), (dict(B=-1), INV), (dict(H=0), INV), (dict(dim=0), INV), (dict(page=0), INV),
    (dict(P=0), INV), (dict(M=0), INV), (dict(dim=40), UNS), (dict(dim=272), UNS), (dict(page=24), UNS), (dict(page=8), UNS),
    (dict(page=256), UNS), (dict(H=4097), UNS), (dict(P=(1 << 22) + 1), UNS), (dict(B=(1 << 16) + 1), UNS), (dict(M=1 << 24), UNS), (dict(M=1 << 23), UNS),
    (dict(T=7), INV),                                    # without starts, a row for each sequence
    (dict(T=(1 << 22) + 1, starts=FAKE), UNS),
    (dict(cache=0), INV), (dict(scale=0), INV), (dict(tables=0), INV), (dict(lengths=0), INV), (dict(work=0), INV),
    (dict(nb=1000), INV), (dict(work=FAKE + 128), MIS), (dict(cache=FAKE + 8), MIS), (dict(scale=FAKE + 2), MIS),
    (dict(tables=FAKE + 1), MIS), (dict(lengths=FAKE + 2), MIS), (dict(starts=FAKE + 2), MIS),
]


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict(k=0), INV), (dict(v=0), INV), (dict(ldk=248), INV), (dict(ldv=248), INV), (dict(ldk=260), MIS), (dict(ldv=260), MIS),
    (dict(k=FAKE + 8), MIS), (dict(v=FAKE + 2), MIS), (dict(T=0, B=0, k=0, cache=0), 0),
])
def test_write_refusals(L, kw, status):
    assert _write(L, **kw) == status


def _attend(L, dt=1, T=8, B=8, Hq=8, H=4, dim=64, page=16, P=100, M=9, q=FAKE, ldq=512, cache=FAKE, scale=FAKE, tables=FAKE,
            lengths=FAKE, starts=None, c=0.125, window=0, y=FAR, ldy=512, work=FAKE, nb=BIG):
    return L.lora_cache_attention(dt, T, B, Hq, H, dim, page, P, M, q, ldq, cache, scale, tables, lengths, starts, c, window,
                                  y, ldy, work, nb, None)


@pytest.mark.parametrize("kw,status", [(k, s) for k, s in SHAPES if "H" not in k] + [
    (dict(H=0), INV), (dict(Hq=0), INV), (dict(Hq=7), INV), (dict(Hq=8192, H=4096, ldq=1 << 20, ldy=1 << 20), UNS),
    (dict(c=0.0), INV), (dict(c=-1.0), INV), (dict(c=math.nan), INV), (dict(c=math.inf), INV), (dict(window=-1), INV),
    (dict(T=1 << 22, starts=FAKE, Hq=256, H=4), UNS),
    (dict(q=0), INV), (dict(y=0), INV), (dict(ldq=504), INV), (dict(ldy=504), INV), (dict(ldq=516), MIS), (dict(ldy=516), MIS),
    (dict(q=FAKE + 8), MIS), (dict(y=FAR + 8), MIS),
    # y over q: the same columns, neighbouring ones that overlap, another stride
    (dict(y=FAKE), INV), (dict(y=FAKE + 512, ldq=1024, ldy=1024), INV), (dict(y=FAKE + 1024, ldq=1024, ldy=1032), INV),
    (dict(y=FAKE + 16, T=1, B=1), INV), (dict(T=0, B=0, q=0, cache=0), 0),
])
def test_attention_refusals(L, kw, status):
    assert _attend(L, **kw) == status


def _extend(L, B=8, M=9, page=16, P=100, t=FAKE, n=FAKE, r=FAKE, work=FAKE, nb=BIG):
    return L.lora_pages_extend(B, M, page, P, t, n, r, work, nb, None)


def _free(L, B=8, M=9, P=100, t=FAKE, n=FAKE, r=FAKE, seqs=FAKE, k=3, work=FAKE, nb=BIG):
    return L.lora_pages_free(B, M, P, t, n, r, seqs, k, work, nb, None)


def _fork(L, B=8, M=9, layers=2, H=4, dim=64, page=16, P=100, t=FAKE, n=FAKE, r=FAKE, src=FAKE, dst=FAKE, k=3, cache=FAKE,
          scale=FAKE, work=FAKE, nb=BIG):
    return L.lora_pages_fork(B, M, layers, H, dim, page, P, t, n, r, src, dst, k, cache, scale, work, nb, None)


def _compact(L, B=8, M=9, layers=2, H=4, dim=64, page=16, P=100, t=FAKE, r=FAKE, ot=FAKE, o=FAKE, live=None, cache=FAKE,
             scale=FAKE, work=FAKE, nb=BIG):
    return L.lora_pages_compact(B, M, layers, H, dim, page, P, t, r, ot, o, live, cache, scale, work, nb, None)


def _copy(L, layers=2, H=4, dim=64, page=16, P=100, cache=FAKE, scale=FAKE, src=FAKE, dst=FAKE, k=3, work=FAKE, nb=BIG):
    return L.lora_pages_copy(layers, H, dim, page, P, cache, scale, src, dst, k, work, nb, None)


PLAN = [(dict(B=-1), INV), (dict(M=0), INV), (dict(P=0), INV), (dict(P=(1 << 22) + 1), UNS), (dict(B=(1 << 16) + 1), UNS),
        (dict(t=0), INV), (dict(r=0), INV), (dict(t=FAKE + 2), MIS), (dict(r=FAKE + 1), MIS), (dict(work=0), INV),
        (dict(nb=64), INV), (dict(work=FAKE + 64), MIS)]
LAYERS = [(dict(layers=0), INV), (dict(H=0), INV), (dict(dim=24), UNS), (dict(page=48), UNS), (dict(cache=0), INV),
          (dict(scale=0), INV), (dict(cache=FAKE + 4), MIS), (dict(scale=FAKE + 2), MIS)]


@pytest.mark.parametrize("call,kw,status", [
    *[(_extend, k, s) for k, s in PLAN + [(dict(n=0), INV), (dict(n=FAKE + 2), MIS), (dict(page=17), UNS), (dict(B=0, t=0), 0)]],
    *[(_free, k, s) for k, s in PLAN + [(dict(n=0), INV), (dict(seqs=0), INV), (dict(seqs=FAKE + 2), MIS), (dict(k=-1), INV),
                                        (dict(k=(1 << 16) + 1), UNS), (dict(k=0, seqs=0), 0)]],
    *[(_fork, k, s) for k, s in PLAN + LAYERS + [(dict(n=0), INV), (dict(src=0), INV), (dict(dst=0), INV), (dict(src=FAKE + 2), MIS),
                                                 (dict(k=-1), INV), (dict(k=4097), UNS), (dict(k=0, src=0), 0)]],
    *[(_compact, k, s) for k, s in PLAN + LAYERS + [(dict(ot=0), INV), (dict(o=0), INV), (dict(live=FAKE + 2), MIS)]],
    *[(_copy, k, s) for k, s in LAYERS + [(dict(src=0), INV), (dict(dst=0), INV), (dict(dst=FAKE + 2), MIS), (dict(k=-1), INV),
                                          (dict(k=(1 << 22) + 1), UNS), (dict(work=0), INV), (dict(nb=64), INV), (dict(k=0, src=0), 0)]],
])
def test_page_refusals(L, call, kw, status):
    assert call(L, **kw) == status


@pytest.mark.parametrize("call", [_write, _attend, _extend, _free, _fork, _compact])
def test_tables_of_more_places_than_ranks_have(call, L):
    assert call(L, B=1 << 10, M=1 << 21, **(dict(T=1 << 10) if call in (_write, _attend) else {})) == UNS
    assert call(L, B=1 << 16, M=1 << 15, **(dict(T=1 << 16) if call in (_write, _attend) else {})) == UNS
    # one place fewer is refused for what comes next
    small = dict(T=1 << 10, work=FAKE + 128) if call in (_write, _attend) else dict(work=FAKE + 64)
    assert call(L, B=1 << 10, M=(1 << 21) - 1, **small) == MIS


def test_binding_refusals_on_cpu_tensors():
    P, H, page, dim, B, M = 10, 2, 16, 64, 3, 4
    cache, scale = torch.zeros(P, 2, H, page, dim).to(torch.float8_e4m3fn), torch.ones(P, 2, H)
    tables, lengths, refs = torch.zeros(B, M, dtype=torch.int32), torch.ones(B, dtype=torch.int32), torch.zeros(P, dtype=torch.int32)
    k, q = torch.zeros(B, H * dim, dtype=torch.bfloat16), torch.zeros(B, 2 * H * dim, dtype=torch.bfloat16)
    work, y, i = torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros_like(q), torch.zeros(2, dtype=torch.int32)
    all_l, all_s = cache[None], scale[None]
    for f in (lambda: ops.cache_write(k, k, cache, scale, tables, lengths, work),
              lambda: ops.cache_attention(q, cache, scale, tables, lengths, y, work),
              lambda: ops.pages_extend(tables, lengths, refs, page, work),
              lambda: ops.pages_free(tables, lengths, refs, i, work),
              lambda: ops.pages_fork(tables, lengths, refs, i, i, all_l, all_s, work),
              lambda: ops.pages_compact(tables, refs, all_l, all_s, work),
              lambda: ops.pages_copy(all_l, all_s, i, i, work)):
        with pytest.raises(ValueError, match="current CUDA device"):
            f()
    bad = [
        (TypeError, lambda: ops.cache_write(k, k, all_l, all_s, tables, lengths, work)),       # all layers
        (TypeError, lambda: ops.cache_write(k, k, cache.float(), scale, tables, lengths, work)),
        (TypeError, lambda: ops.cache_write(k, k, cache, scale[:, :1], tables, lengths, work)),
        (TypeError, lambda: ops.cache_write(k, k, cache, scale.double(), tables, lengths, work)),
        (TypeError, lambda: ops.cache_write(k, k, cache.transpose(0, 3), scale, tables, lengths, work)),
        (TypeError, lambda: ops.cache_write(k, k, cache, scale, tables.long(), lengths, work)),
        (TypeError, lambda: ops.cache_write(k, k, cache, scale, tables.t(), lengths, work)),
        (TypeError, lambda: ops.cache_write(k, k, cache, scale, tables, lengths[:2], work)),
        (TypeError, lambda: ops.cache_write(k, k.half(), cache, scale, tables, lengths, work)),
        (ValueError, lambda: ops.cache_write(k[:, :64], k, cache, scale, tables, lengths, work)),
        (ValueError, lambda: ops.cache_write(k[:2], k[:2], cache, scale, tables, lengths, work)),  # a row too few
        (TypeError, lambda: ops.cache_write(k, k, cache, scale, tables, lengths, work, starts=lengths)),
        (ValueError, lambda: ops.cache_attention(q[:, :192], cache, scale, tables, lengths, y[:, :192], work)),
        (ValueError, lambda: ops.cache_attention(q, cache, scale, tables, lengths, y[:, :128], work)),
        (TypeError, lambda: ops.cache_attention(q, cache, scale, tables, lengths, y.half(), work)),
        (ValueError, lambda: ops.cache_attention(q.t(), cache, scale, tables, lengths, y, work)),
        (TypeError, lambda: ops.pages_fork(tables, lengths, refs, i, i, cache, scale, work)),  # one layer
        (TypeError, lambda: ops.pages_fork(tables, lengths, refs[:5], i, i, all_l, all_s, work)),
        (TypeError, lambda: ops.pages_fork(tables, lengths, refs, i, i[:1], all_l, all_s, work)),
        (TypeError, lambda: ops.pages_free(tables, lengths, refs, i.long(), work)),
        (TypeError, lambda: ops.pages_compact(tables, refs, all_l, all_s, work, out_tables=tables[:2])),
        (TypeError, lambda: ops.pages_compact(tables, refs, all_l, all_s, work, n_live=i)),
        (ops.LoraError, lambda: ops.cache_workspace(0, 128, device="cpu")),
        (ops.LoraError, lambda: ops.cache_workspace(4, 40, device="cpu")),
        (ops.LoraError, lambda: ops.cache_workspace(1 << 33, 64, device="cpu")),
        (ops.LoraError, lambda: ops.pages_extend(tables, lengths, refs, 1 << 32, work)),
    ]
    for error, f in bad:
        with pytest.raises(error):
            f()
