"""Python binding of the multi-LoRA shrink / expand C ABI.

Argument marshalling only: each function reads shapes, strides and device
pointers off torch tensors, passes them to liblora_b200.so on the current
torch CUDA stream, and raises LoraError on a non-OK status.  Every step of the
computation runs in the library's CUDA kernels; torch supplies device memory
and streams.

  group(idx, S, meta)                          per-batch group-by-slot metadata
  shrink(x, A, idx, buf, meta)                 buf[i] = per-token x . A_i[idx]^T
  expand(buf, B, idx, y, meta, scale)          y[:, slice_i] += scale buf_i . B_i[idx]^T
  bgmv(x, A, B, idx, y, buf, meta, scale)      group + shrink + expand in one call
  shrink_segment / expand_segment              the same with segments
  check_errors(meta)                           device-side bad-index report
  quantize_fp8 / matmul_fp8 / linear_fp8       the base product y = x W^T in block-scaled e4m3
  rope / norm_rope / rope_frequencies          rotation (and norms) of q and k head slices
  cache_write / cache_attention                a paged 8-bit k/v cache: its write, attention over it
  pages_extend / _fork / _free / _compact / _copy   its pages

has_active: the per-token calls take the host flag of the C ABI.  Left as
None, it is derived from `idx_host` (a host copy of the batch's indices, as a
serving loop has before it moves them to the device) when one is given: no
index in [0, S) means no LoRA work at all, so nothing is enqueued.  Without a
host copy the call runs, and the kernels skip tokens without an adapter.
"""
import ctypes
import functools
from typing import Optional, Sequence

import torch

from . import _lib

_DT = {torch.float16: _lib.LORA_F16, torch.bfloat16: _lib.LORA_BF16}


class LoraError(RuntimeError):
    def __init__(self, call, status):
        self.status = status
        super().__init__(f"{call} failed: {_lib.status_string(status)} ({status})")


def _check(call, status):
    if status != _lib.LORA_OK:
        raise LoraError(call, status)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr() if t is not None else 0)


def _ptrs(ts):
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


def _dtype(t):
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}; fp16 or bf16")
    return _DT[t.dtype]


def active_from_host(idx_host, S: int) -> bool:
    """Whether any index of a host copy of a batch's indices selects a slot
    in [0, S)."""
    if isinstance(idx_host, torch.Tensor):
        if idx_host.is_cuda:
            raise ValueError("idx_host must be a host tensor or array")
        idx_host = idx_host.numpy()
    import numpy as np
    a = np.asarray(idx_host)
    return bool(np.any((a >= 0) & (a < S)))


def _active(has_active, idx_host, S):
    if has_active is not None:
        return int(bool(has_active))
    if idx_host is not None:
        return int(active_from_host(idx_host, S))
    return 1


def _check_idx(idx, T):
    if idx.dtype != torch.int32 or not idx.is_contiguous() or idx.numel() != T:
        raise TypeError("idx must be a contiguous int32 tensor of one index per token")


def workspace_bytes(T: int, S: int) -> int:
    return _lib.load().lora_workspace_bytes(int(T), int(S))


def workspace(T: int, S: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace ("meta") for batches of up to T tokens over S slots."""
    n = workspace_bytes(T, S)
    if n == 0:
        raise LoraError("lora_workspace_bytes", _lib.LORA_ERR_UNSUPPORTED)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def set_slot_ranks(ranks: Optional[torch.Tensor], S: int, meta: torch.Tensor, stream=None):
    """Record each slot's own rank (device int32 [S]; None clears) in the
    workspace: the kernels then skip the zero padding of smaller-rank slots."""
    if ranks is not None:
        if ranks.dtype != torch.int32 or not ranks.is_contiguous() or ranks.numel() != S:
            raise TypeError("ranks must be a contiguous int32 tensor of one rank per slot")
    _check("lora_set_slot_ranks", _lib.load().lora_set_slot_ranks(
        int(S), _ptr(ranks), _ptr(meta), meta.numel(), _stream(stream)))


def group(idx: torch.Tensor, S: int, meta: torch.Tensor, stream=None):
    """Group-by-slot metadata of one batch's int32 adapter indices (-1 = none)."""
    _check_idx(idx, idx.numel())
    _check("lora_group", _lib.load().lora_group(idx.numel(), int(S), _ptr(idx), _ptr(meta),
                                                meta.numel(), _stream(stream)))


def _xinfo(x):
    if x.dim() != 2 or (x.numel() > 0 and x.stride(1) != 1):
        raise ValueError("x must be [T, D] with unit column stride")
    return x.shape[0], x.shape[1], (x.stride(0) if x.numel() > 0 else x.shape[1])


def shrink(x: torch.Tensor, A: Sequence[torch.Tensor], idx: torch.Tensor, buf: torch.Tensor,
           meta: torch.Tensor, has_active: Optional[bool] = None, idx_host=None,
           stream=None) -> torch.Tensor:
    """buf[i, t, :] = x[t] . A[i][idx[t]]^T (0 for tokens without an adapter).

    A: list of [S, r, D] stacks; idx: the device int32 indices that group()
    grouped into meta; buf: float32 [len(A), T, r]."""
    T, D, ldx = _xinfo(x)
    S, r, _ = A[0].shape
    _check_idx(idx, T)
    _check("lora_shrink", _lib.load().lora_shrink(
        _dtype(x), T, D, r, S, len(A), _ptr(x), ldx, _ptrs(A), _ptr(idx), _ptr(buf),
        _active(has_active, idx_host, S), _ptr(meta), meta.numel(), _stream(stream)))
    return buf


def shrink_laned(x: torch.Tensor, A: Sequence[torch.Tensor], idx: torch.Tensor,
                 buf: torch.Tensor, meta: torch.Tensor, has_active: Optional[bool] = None,
                 idx_host=None, stream=None) -> torch.Tensor:
    """shrink() without a grouping: every slot's lanes in one dense tensor-core
    contraction, each token keeping its own slot's r lanes.  meta only
    collects the error counters (group() is not needed)."""
    T, D, ldx = _xinfo(x)
    S, r, _ = A[0].shape
    _check_idx(idx, T)
    _check("lora_shrink_laned", _lib.load().lora_shrink_laned(
        _dtype(x), T, D, r, S, len(A), _ptr(x), ldx, _ptrs(A), _ptr(idx), _ptr(buf),
        _active(has_active, idx_host, S), _ptr(meta), meta.numel(), _stream(stream)))
    return buf


def _expand_common(buf, B, y, y_col_off, buf_slice_stride):
    if y.dim() != 2 or (y.numel() > 0 and y.stride(1) != 1):
        raise ValueError("y must be [T, ldy] with unit column stride")
    T, ldy = y.shape[0], (y.stride(0) if y.numel() > 0 else y.shape[1])
    S, _, r = B[0].shape
    n = len(B)
    d_out = (ctypes.c_int32 * n)(*[b.shape[1] for b in B])
    if y_col_off is None:
        offs, c = [], 0
        for b in B:
            offs.append(c)
            c += b.shape[1]
        y_col_off = offs
    off = (ctypes.c_int64 * n)(*[int(v) for v in y_col_off])
    if buf_slice_stride is None:
        buf_slice_stride = 0 if buf.dim() == 2 else buf.stride(0)
    return T, ldy, S, r, n, d_out, off, int(buf_slice_stride)


def expand(buf: torch.Tensor, B: Sequence[torch.Tensor], idx: torch.Tensor, y: torch.Tensor,
           meta: torch.Tensor, scale: float = 1.0, y_col_off=None, buf_slice_stride=None,
           has_active: Optional[bool] = None, idx_host=None, stream=None) -> torch.Tensor:
    """y[t, off_i:off_i+D_out_i] += scale * buf[i, t] . B[i][idx[t]]^T, in place.

    B: list of [S, D_out_i, r]; idx as for shrink(); buf: float32 [n, T, r]
    (or [T, r] shared by every slice); y: [T, >= sum D_out] fp16/bf16."""
    T, ldy, S, r, n, d_out, off, stride = _expand_common(buf, B, y, y_col_off, buf_slice_stride)
    _check_idx(idx, T)
    _check("lora_expand", _lib.load().lora_expand(
        _dtype(y), T, r, S, n, _ptr(buf), stride, _ptrs(B), d_out, _ptr(idx),
        ctypes.c_float(scale), _ptr(y), ldy, off, _active(has_active, idx_host, S), _ptr(meta),
        meta.numel(), _stream(stream)))
    return y


def bgmv(x: torch.Tensor, A: Sequence[torch.Tensor], B: Sequence[torch.Tensor], idx: torch.Tensor,
         y: torch.Tensor, buf: torch.Tensor, meta: torch.Tensor, scale: float = 1.0,
         y_col_off=None, has_active: Optional[bool] = None, idx_host=None,
         pdl_early: bool = False, grouped: bool = False, stream=None):
    """group + shrink + expand of one batch in one call (one launch when the
    shape fits the fused kernel).  A: one stack per slice of B, or a single
    stack shared by every slice; buf: float32 [len(A), T, r] receives the
    intermediate; y is updated in place.  pdl_early=True promises that A, B
    and idx are not written by the kernel launched just before on the stream;
    grouped=True that meta already holds this idx's grouping (group(), or an
    earlier bgmv of the batch): no grouping launch."""
    T, D, ldx = _xinfo(x)
    S, r, _ = A[0].shape
    n = len(B)
    shared = len(A) == 1 and n > 1
    if not shared and len(A) != n:
        raise ValueError("A must hold one stack per slice, or one shared stack")
    _, ldy, _, _, _, d_out, off, _ = _expand_common(buf, B, y, y_col_off, None)
    _check_idx(idx, T)
    flags = (_lib.LORA_FLAG_PDL_EARLY if pdl_early else 0) | \
        (_lib.LORA_FLAG_GROUPED if grouped else 0)
    _check("lora_bgmv", _lib.load().lora_bgmv(
        _dtype(x), T, D, r, S, n, _ptr(x), ldx, _ptrs(A), int(shared), _ptrs(B), d_out,
        ctypes.c_float(scale), _ptr(y), ldy, off, _ptr(buf), _ptr(idx),
        _active(has_active, idx_host, S), flags, _ptr(meta), meta.numel(), _stream(stream)))
    return y


def bgmv_launches(dtype, T: int, D: int, r: int, S: int, d_out) -> int:
    """Kernel launches bgmv() makes for this shape: 1 (fused) or 3."""
    dt = _DT[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    arr = (ctypes.c_int32 * len(d_out))(*[int(v) for v in d_out])
    return _lib.load().lora_bgmv_launches(dt, int(T), int(D), int(r), int(S), len(d_out), arr)


def shrink_segment(x, A, seg_starts, seg_adapter, buf, meta, has_active=True, stream=None):
    """shrink() with adapters given by segments (int32 CSR starts [n+1], adapters [n])."""
    T, D, ldx = _xinfo(x)
    S, r, _ = A[0].shape
    _check("lora_shrink_segment", _lib.load().lora_shrink_segment(
        _dtype(x), T, D, r, S, len(A), _ptr(x), ldx, _ptrs(A), _ptr(seg_starts),
        _ptr(seg_adapter), seg_adapter.numel(), _ptr(buf), int(bool(has_active)), _ptr(meta),
        meta.numel(), _stream(stream)))
    return buf


def expand_segment(buf, B, seg_starts, seg_adapter, y, meta, scale=1.0, y_col_off=None,
                   buf_slice_stride=None, has_active=True, stream=None):
    """expand() with adapters given by segments."""
    T, ldy, S, r, n, d_out, off, stride = _expand_common(buf, B, y, y_col_off, buf_slice_stride)
    _check("lora_expand_segment", _lib.load().lora_expand_segment(
        _dtype(y), T, r, S, n, _ptr(buf), stride, _ptrs(B), d_out, _ptr(seg_starts),
        _ptr(seg_adapter), seg_adapter.numel(), ctypes.c_float(scale), _ptr(y), ldy, off,
        int(bool(has_active)), _ptr(meta), meta.numel(), _stream(stream)))
    return y


def sgmv(x: torch.Tensor, A: Sequence[torch.Tensor], B: Sequence[torch.Tensor],
         seg_starts: torch.Tensor, seg_adapter: torch.Tensor, y: torch.Tensor, buf: torch.Tensor,
         meta: torch.Tensor, scale: float = 1.0, y_col_off=None, has_active: bool = True,
         stream=None):
    """shrink_segment() + expand_segment() of one prefill batch in one call
    (the expand starts while the shrink finishes).  A: one stack per slice of
    B, or a single stack shared by every slice; buf: float32 [len(A), T, r]."""
    T, D, ldx = _xinfo(x)
    S, r, _ = A[0].shape
    n = len(B)
    shared = len(A) == 1 and n > 1
    if not shared and len(A) != n:
        raise ValueError("A must hold one stack per slice, or one shared stack")
    _, ldy, _, _, _, d_out, off, _ = _expand_common(buf, B, y, y_col_off, None)
    _check("lora_sgmv", _lib.load().lora_sgmv(
        _dtype(x), T, D, r, S, n, _ptr(x), ldx, _ptrs(A), int(shared), _ptrs(B), d_out,
        ctypes.c_float(scale), _ptr(y), ldy, off, _ptr(buf), _ptr(seg_starts), _ptr(seg_adapter),
        seg_adapter.numel(), int(bool(has_active)), _ptr(meta), meta.numel(), _stream(stream)))
    return y


def shrink_noalloc(x: torch.Tensor, A: Sequence[torch.Tensor], idx: torch.Tensor,
                   buf: torch.Tensor, has_active: bool = True, stream=None) -> torch.Tensor:
    """group() + shrink() in one call that needs no workspace: the library keeps
    the grouping scratch in a fixed device array.  For callers that cannot
    allocate; calls that overlap on the GPU race on that array."""
    T, D, ldx = _xinfo(x)
    S, r, _ = A[0].shape
    _check_idx(idx, T)
    _check("lora_shrink_noalloc", _lib.load().lora_shrink_noalloc(
        _dtype(x), T, D, r, S, len(A), _ptr(x), ldx, _ptrs(A), _ptr(idx), _ptr(buf),
        int(bool(has_active)), _stream(stream)))
    return buf


# ---------------------------------------------------------------------------
# Around a LoRA-wrapped projection: the 8-bit base product, and the rotation
# (and norms) of the query and key heads.  Tensors must lie on the current
# CUDA device.
# ---------------------------------------------------------------------------
_FP8 = torch.float8_e4m3fn
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# The C calls take sizes as int, and ctypes cuts a larger number down to its
# low 32 bits without a word: such numbers are refused here.
_INT_MAX = 0x7fffffff


def _int(call, v):
    v = int(v)
    if not -_INT_MAX <= v <= _INT_MAX:
        raise LoraError(call, _lib.LORA_ERR_UNSUPPORTED)
    return v


def _here(stream, *tensors):
    """The stream handle to launch on, once every tensor lies on the current device."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev:
            dev = -1
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError("tensors must lie on the current CUDA device")
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(dev) if _raw_stream else torch.cuda.current_stream().cuda_stream


def _rows(t, name, dtype=None):
    """Row stride of a 2-D tensor with unit column stride."""
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1 and shape[0] > 0):
        raise ValueError(f"{name} must be 2-D with unit column stride")
    if shape[0] > _INT_MAX or shape[1] > _INT_MAX:
        raise ValueError(f"{name} must have less than 2^31 rows and columns")
    # a single row has no next one: any stride that the alignment rules take
    return stride[0] if shape[0] > 1 else -(-max(shape[1], 1) // 16) * 16


def _scales(t, name, rows, K):
    if t.dtype is not torch.float32 or not t.is_contiguous() or t.shape != (rows, -(-K // 128)):
        raise TypeError(f"{name} must be a contiguous float32 tensor of {rows} x {-(-K // 128)}")


def quantize_fp8(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, block_rows: int = 1,
                 stream=None):
    """q, scale = x in e4m3 with one fp32 scale per group of 128 columns of a
    row (block_rows=1, activations) or per 128 x 128 block (block_rows=128,
    weights): scale = max|x| / 448, q = x / scale rounded once.

    x: fp16/bf16 [T, K]; q: float8_e4m3fn [T, K] whose rows start at multiples
    of 16; scale: float32 [ceil(T / block_rows), ceil(K / 128)]."""
    ldx, ldq = _rows(x, "x"), _rows(q, "q", _FP8)
    T, K = x.shape
    if q.shape != x.shape:
        raise ValueError("q must have the shape of x")
    if block_rows != 1:
        block_rows = _int("lora_quantize_fp8", block_rows)
    _scales(scale, "scale", -(-T // block_rows) if block_rows > 0 else 0, K)
    st = _here(stream, x, q, scale)
    _check("lora_quantize_fp8", _lib.load().lora_quantize_fp8(
        _dtype(x), T, K, block_rows, x.data_ptr(), ldx, q.data_ptr(), ldq, scale.data_ptr(), st))
    return q, scale


def matmul_fp8(q: torch.Tensor, q_scale: torch.Tensor, W: torch.Tensor, w_scale: torch.Tensor,
               y: torch.Tensor, stream=None) -> torch.Tensor:
    """y = (q * q_scale) (W * w_scale)^T: products and sums in fp32, rounded
    once to y's fp16/bf16.  q, q_scale as quantize_fp8(x, ...) writes them, W
    [N, K] and w_scale as quantize_fp8(..., block_rows=128) does; y: [T, N]."""
    ldq, ldw, ldy = _rows(q, "q", _FP8), _rows(W, "W", _FP8), _rows(y, "y")
    T, K = q.shape
    N = W.shape[0]
    if W.shape[1] != K or y.shape[0] != T or y.shape[1] != N:
        raise ValueError("shapes must be q [T, K], W [N, K], y [T, N]")
    _scales(q_scale, "q_scale", T, K)
    _scales(w_scale, "w_scale", -(-N // 128), K)
    st = _here(stream, q, q_scale, W, w_scale, y)
    _check("lora_matmul_fp8", _lib.load().lora_matmul_fp8(
        _dtype(y), T, N, K, q.data_ptr(), ldq, q_scale.data_ptr(), W.data_ptr(), ldw,
        w_scale.data_ptr(), y.data_ptr(), ldy, st))
    return y


def linear_fp8_workspace(T: int, K: int, device="cuda") -> torch.Tensor:
    """A workspace for linear_fp8() of up to T tokens of K columns."""
    call = "lora_linear_fp8_workspace_bytes"
    n = _lib.load().lora_linear_fp8_workspace_bytes(_int(call, T), _int(call, K))
    if n == 0:
        raise LoraError(call, _lib.LORA_ERR_UNSUPPORTED)
    return torch.empty(n, dtype=torch.uint8, device=device)


def linear_fp8(x: torch.Tensor, W: torch.Tensor, w_scale: torch.Tensor, y: torch.Tensor,
               work: torch.Tensor, stream=None) -> torch.Tensor:
    """y = x (W * w_scale)^T with x quantised per token and 128 columns:
    quantize_fp8 into the workspace and matmul_fp8 in one call.  x, y:
    fp16/bf16 [T, K], [T, N] of one dtype; work: linear_fp8_workspace(T, K),
    one for each stream that such calls run on."""
    ldx, ldw, ldy = _rows(x, "x"), _rows(W, "W", _FP8), _rows(y, "y", x.dtype)
    T, K = x.shape
    N = W.shape[0]
    if W.shape[1] != K or y.shape[0] != T or y.shape[1] != N:
        raise ValueError("shapes must be x [T, K], W [N, K], y [T, N]")
    _scales(w_scale, "w_scale", -(-N // 128), K)
    if not work.is_contiguous():
        raise ValueError("work must be contiguous")
    st = _here(stream, x, W, w_scale, y, work)
    _check("lora_linear_fp8", _lib.load().lora_linear_fp8(
        _dtype(x), T, N, K, x.data_ptr(), ldx, W.data_ptr(), ldw, w_scale.data_ptr(), y.data_ptr(),
        ldy, work.data_ptr(), work.numel() * work.element_size(), st))
    return y


def rope_frequencies(rot: int, base: float = 10000.0, kind: str = "none", factor: float = 1.0,
                     original_length: float = 0.0, beta_fast: float = 32.0,
                     beta_slow: float = 1.0, device="cuda"):
    """(inv_freq, attn_scale) for rope(): radians per position of the rot / 2
    pairs (float64 tensor) and the factor on cos and sin.  kind: "none",
    "linear", "ntk", "yarn" or "bands" (see lora_rope_frequencies)."""
    if kind not in _lib.ROPE_KINDS:
        raise ValueError(f"kind must be one of {sorted(_lib.ROPE_KINDS)}")
    rot = _int("lora_rope_frequencies", rot)
    out = (ctypes.c_double * max(min(rot, _lib.LORA_MAX_HEAD_DIM) // 2, 1))()
    attn = ctypes.c_float()
    _check("lora_rope_frequencies", _lib.load().lora_rope_frequencies(
        rot, float(base), _lib.ROPE_KINDS[kind], float(factor), float(original_length),
        float(beta_fast), float(beta_slow), out, ctypes.byref(attn)))
    return torch.tensor(list(out), dtype=torch.float64, device=device), attn.value


@functools.lru_cache(maxsize=256)
def _layout(heads, dim, col_off):
    """(heads, first columns, past-the-end column) of a tuple of slices, as the
    C call takes them; a pure function of its arguments."""
    if col_off is None:
        col_off, c = [], 0
        for h in heads:
            col_off.append(c)
            c += h * dim
    if len(col_off) != len(heads):
        raise ValueError("one column offset per slice")
    if dim <= 0 or any(h <= 0 for h in heads) or any(c < 0 for c in col_off):
        raise LoraError("lora_rope", _lib.LORA_ERR_INVALID_ARG)
    end = max([c + h * dim for h, c in zip(heads, col_off)], default=0)
    return ((ctypes.c_int32 * len(heads))(*heads), (ctypes.c_int64 * len(heads))(*col_off), end)


def _offsets(t, heads, dim, col_off):
    h, off, end = _layout(tuple(heads), dim, None if col_off is None else tuple(col_off))
    if end > t.shape[1]:
        raise ValueError("a slice's heads reach past the last column")
    return h, off


def _rope_args(x, y, heads, head_dim, positions, inv_freq, x_col_off, y_col_off):
    ldx, ldy = _rows(x, "x"), _rows(y, "y", x.dtype)
    T = x.shape[0]
    if y.shape[0] != T:
        raise ValueError("x and y must have the same rows")
    if positions.dtype is not torch.int64 or not positions.is_contiguous() or \
            positions.numel() != T:
        raise TypeError("positions must be a contiguous int64 tensor of one position per token")
    if inv_freq.dtype is not torch.float64 or not inv_freq.is_contiguous() or inv_freq.dim() != 1:
        raise TypeError("inv_freq must be a contiguous float64 tensor of one frequency per pair")
    rot = 2 * inv_freq.numel()
    if rot > _INT_MAX:
        raise LoraError("lora_rope", _lib.LORA_ERR_INVALID_ARG)
    h, xo = _offsets(x, heads, head_dim, x_col_off)
    _, yo = _offsets(y, heads, head_dim, y_col_off)
    head = (_dtype(x), T, head_dim, rot, len(h), h, x.data_ptr(), ldx, xo)
    return head, (y.data_ptr(), ldy, yo, positions.data_ptr(), inv_freq.data_ptr())


def rope(x: torch.Tensor, y: torch.Tensor, heads: Sequence[int], head_dim: int,
         positions: torch.Tensor, inv_freq: torch.Tensor, x_col_off=None, y_col_off=None,
         interleaved: bool = False, attn_scale: float = 1.0, stream=None) -> torch.Tensor:
    """Rotary positions of head slices: slice i is heads[i] heads of head_dim
    columns from x_col_off[i] of x, written from y_col_off[i] of y (both side
    by side from column 0 by default).  The first 2 * len(inv_freq) elements
    of each head are rotated by positions[t] * inv_freq[pair], pairs split in
    halves or interleaved; the rest are copied.  y may be x with the same
    offsets (in place).  positions: int64 [T]; inv_freq, attn_scale from
    rope_frequencies()."""
    head, tail = _rope_args(x, y, heads, head_dim, positions, inv_freq, x_col_off, y_col_off)
    st = _here(stream, x, y, positions, inv_freq)
    _check("lora_rope", _lib.load().lora_rope(*head, *tail, attn_scale, bool(interleaved), st))
    return y


def norm_rope(x: torch.Tensor, weights, y: torch.Tensor, heads: Sequence[int], head_dim: int,
              positions: torch.Tensor, inv_freq: torch.Tensor, eps: float = 1e-6, x_col_off=None,
              y_col_off=None, interleaved: bool = False, attn_scale: float = 1.0,
              stream=None) -> torch.Tensor:
    """rope() with a root-mean-square norm of each head before it, in one
    pass: weights holds one tensor [head_dim] of x's dtype per slice, or None
    for a slice without a norm."""
    head, tail = _rope_args(x, y, heads, head_dim, positions, inv_freq, x_col_off, y_col_off)
    if len(weights) != len(heads):
        raise ValueError("one weight (or None) per slice")
    given = [w for w in weights if w is not None]
    for w in given:
        if w.dtype is not x.dtype or not w.is_contiguous() or w.numel() != head_dim:
            raise TypeError("a weight must be a contiguous tensor of head_dim elements of x's dtype")
    st = _here(stream, x, y, positions, inv_freq, *given)
    ws = (ctypes.c_void_p * len(weights))(*[None if w is None else w.data_ptr() for w in weights])
    _check("lora_norm_rope", _lib.load().lora_norm_rope(
        *head, ws, eps, *tail, attn_scale, bool(interleaved), st))
    return y


# ---------------------------------------------------------------------------
# Behind the attention inputs: a paged key/value cache in 8 bits.  cache:
# float8_e4m3fn [P, 2, kv_heads, page_tokens, head_dim] of one layer, scale:
# float32 [P, 2, kv_heads]; the moves of pages take those of all layers, with a
# leading dimension.  tables: int32 [B, pages of a sequence], -1 = none;
# lengths: int32 [B]; refs: int32 [P].  Tensors must lie on the current CUDA
# device.
# ---------------------------------------------------------------------------
def _ints(t, name, shape):
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)}")


def _list(t, name):
    if t.dtype is not torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor of one dimension")
    return _int(name, t.shape[0])


def _cache(cache, scale, layers):
    """The cache's dimensions: [layers,] pages, 2, kv_heads, page_tokens, head_dim."""
    shape = cache.shape
    if cache.dtype is not _FP8 or len(shape) != 5 + layers or shape[1 + layers] != 2 or \
            not cache.is_contiguous():
        raise TypeError("cache must be a contiguous float8_e4m3fn tensor of " +
                        ("layers x " if layers else "") + "pages x 2 x kv_heads x page_tokens x head_dim")
    if scale.dtype is not torch.float32 or scale.shape != shape[:3 + layers] or not scale.is_contiguous():
        raise TypeError("scale must be a contiguous float32 tensor of the cache's first dimensions")
    if max(shape) > _INT_MAX:
        raise LoraError("lora_cache", _lib.LORA_ERR_UNSUPPORTED)
    return shape


def _seqs(tables, lengths=None):
    shape = tables.shape
    if tables.dtype is not torch.int32 or len(shape) != 2 or not tables.is_contiguous():
        raise TypeError("tables must be a contiguous int32 tensor of sequences x pages")
    if max(shape) > _INT_MAX:
        raise LoraError("lora_cache", _lib.LORA_ERR_UNSUPPORTED)
    if lengths is not None and (lengths.dtype is not torch.int32 or lengths.shape != shape[:1] or
                                not lengths.is_contiguous()):
        raise TypeError("lengths must be a contiguous int32 tensor of one length per sequence")
    return shape


def _work(work):
    if not work.is_contiguous():
        raise ValueError("work must be contiguous")
    return work.data_ptr(), work.numel() * work.element_size()


def cache_workspace(n_pages: int, head_dim: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for the calls on a cache of n_pages pages; one
    for each stream that such calls run on."""
    call = "lora_cache_workspace_bytes"
    n = _lib.load().lora_cache_workspace_bytes(_int(call, n_pages), _int(call, head_dim))
    if n == 0:
        raise LoraError(call, _lib.LORA_ERR_UNSUPPORTED)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _new_rows(t, name, width, starts, B, T=None, dtype=None):
    ld = _rows(t, name, dtype)
    if t.shape[1] != width or (T is not None and t.shape[0] != T):
        raise ValueError(f"{name} must be [T, heads * head_dim] = [{t.shape[0] if T is None else T}, {width}]")
    if starts is None and t.shape[0] != B:
        raise ValueError("without starts there is one row for each sequence")
    return ld


def cache_write(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, scale: torch.Tensor,
                tables: torch.Tensor, lengths: torch.Tensor, work: torch.Tensor,
                starts: Optional[torch.Tensor] = None, stream=None):
    """Put the new tokens' keys and values (fp16/bf16 [T, kv_heads * head_dim],
    columns of one matrix or not) into their sequences' pages in e4m3, with one
    power of two as scale for each (page, k or v, head).

    lengths: tokens of each sequence, the new ones counted in; starts: int32
    [B + 1], the new tokens of sequence b are rows starts[b] .. starts[b+1]
    (None: one row each); the pages must be there (pages_extend)."""
    P, _, H, page, dim = _cache(cache, scale, 0)
    B, M = _seqs(tables, lengths)
    T = k.shape[0]
    ldk = _new_rows(k, "k", H * dim, starts, B)
    ldv = _new_rows(v, "v", H * dim, starts, B, T, k.dtype)
    given = () if starts is None else (starts,)
    if starts is not None:
        _ints(starts, "starts", (B + 1,))
    wp, wn = _work(work)
    st = _here(stream, k, v, cache, scale, tables, lengths, work, *given)
    _check("lora_cache_write", _lib.load().lora_cache_write(
        _dtype(k), T, B, H, dim, page, P, M, k.data_ptr(), ldk, v.data_ptr(), ldv, cache.data_ptr(),
        scale.data_ptr(), tables.data_ptr(), lengths.data_ptr(),
        None if starts is None else starts.data_ptr(), wp, wn, st))


def cache_attention(q: torch.Tensor, cache: torch.Tensor, scale: torch.Tensor, tables: torch.Tensor,
                    lengths: torch.Tensor, y: torch.Tensor, work: torch.Tensor,
                    starts: Optional[torch.Tensor] = None, softmax_scale: Optional[float] = None,
                    window: int = 0, stream=None) -> torch.Tensor:
    """y = softmax(softmax_scale q k^T) v of the new tokens' queries over the
    tokens of their sequences up to themselves (the last `window` of them only,
    if window > 0).  q, y: fp16/bf16 [T, q_heads * head_dim]; lengths, starts as
    for cache_write, which comes first; softmax_scale: 1 / sqrt(head_dim) by
    default.  Queries that see nothing get zeros."""
    P, _, H, page, dim = _cache(cache, scale, 0)
    B, M = _seqs(tables, lengths)
    T, width = q.shape[0], q.shape[1] if q.dim() == 2 else -1
    if width <= 0 or width % (H * dim):
        raise ValueError("q must hold a multiple of the cache's heads")
    ldq = _new_rows(q, "q", width, starts, B)
    ldy = _new_rows(y, "y", width, starts, B, T, q.dtype)
    given = () if starts is None else (starts,)
    if starts is not None:
        _ints(starts, "starts", (B + 1,))
    wp, wn = _work(work)
    st = _here(stream, q, cache, scale, tables, lengths, y, work, *given)
    _check("lora_cache_attention", _lib.load().lora_cache_attention(
        _dtype(q), T, B, width // dim, H, dim, page, P, M, q.data_ptr(), ldq, cache.data_ptr(),
        scale.data_ptr(), tables.data_ptr(), lengths.data_ptr(),
        None if starts is None else starts.data_ptr(),
        dim ** -0.5 if softmax_scale is None else softmax_scale, _int("window", window),
        y.data_ptr(), ldy, wp, wn, st))
    return y


def pages_extend(tables: torch.Tensor, lengths: torch.Tensor, refs: torch.Tensor, page_tokens: int,
                 work: torch.Tensor, stream=None):
    """Free pages, lowest first, for the places of each sequence's table that
    its length needs and that hold none yet."""
    B, M = _seqs(tables, lengths)
    P, page_tokens = _list(refs, "refs"), _int("lora_pages_extend", page_tokens)
    wp, wn = _work(work)
    st = _here(stream, tables, lengths, refs, work)
    _check("lora_pages_extend", _lib.load().lora_pages_extend(
        B, M, page_tokens, P, tables.data_ptr(), lengths.data_ptr(),
        refs.data_ptr(), wp, wn, st))


def pages_free(tables: torch.Tensor, lengths: torch.Tensor, refs: torch.Tensor, seqs: torch.Tensor,
               work: torch.Tensor, stream=None):
    """The listed sequences (int32 [n]) end: their pages' counts go down by one,
    their rows become -1 and their lengths 0."""
    B, M = _seqs(tables, lengths)
    P, n = _list(refs, "refs"), _list(seqs, "seqs")
    wp, wn = _work(work)
    st = _here(stream, tables, lengths, refs, seqs, work)
    _check("lora_pages_free", _lib.load().lora_pages_free(
        B, M, P, tables.data_ptr(), lengths.data_ptr(), refs.data_ptr(), seqs.data_ptr(), n, wp, wn,
        st))


def pages_fork(tables: torch.Tensor, lengths: torch.Tensor, refs: torch.Tensor, src: torch.Tensor,
               dst: torch.Tensor, cache: torch.Tensor, scale: torch.Tensor, work: torch.Tensor,
               stream=None):
    """Each empty row dst[i] becomes a copy of the sequence src[i] (int32 [n]):
    full pages are shared, the begun last one is copied in all layers."""
    B, M = _seqs(tables, lengths)
    L, P, _, H, page, dim = _cache(cache, scale, 1)
    _ints(refs, "refs", (P,))
    n = _list(src, "src")
    _ints(dst, "dst", (n,))
    wp, wn = _work(work)
    st = _here(stream, tables, lengths, refs, src, dst, cache, scale, work)
    _check("lora_pages_fork", _lib.load().lora_pages_fork(
        B, M, L, H, dim, page, P, tables.data_ptr(), lengths.data_ptr(), refs.data_ptr(),
        src.data_ptr(), dst.data_ptr(), n, cache.data_ptr(), scale.data_ptr(), wp, wn, st))


def pages_compact(tables: torch.Tensor, refs: torch.Tensor, cache: torch.Tensor, scale: torch.Tensor,
                  work: torch.Tensor, out_tables: Optional[torch.Tensor] = None,
                  out_refs: Optional[torch.Tensor] = None, n_live: Optional[torch.Tensor] = None,
                  stream=None):
    """Move the live pages to the front of the pool in all layers; the tables
    and counts follow, in place or into out_tables and out_refs.  n_live: int32
    [1], receives the number of live pages."""
    B, M = _seqs(tables)
    L, P, _, H, page, dim = _cache(cache, scale, 1)
    _ints(refs, "refs", (P,))
    out_tables = tables if out_tables is None else out_tables
    out_refs = refs if out_refs is None else out_refs
    _ints(out_tables, "out_tables", (B, M))
    _ints(out_refs, "out_refs", (P,))
    given = () if n_live is None else (n_live,)
    if n_live is not None:
        _ints(n_live, "n_live", (1,))
    wp, wn = _work(work)
    st = _here(stream, tables, refs, cache, scale, work, out_tables, out_refs, *given)
    _check("lora_pages_compact", _lib.load().lora_pages_compact(
        B, M, L, H, dim, page, P, tables.data_ptr(), refs.data_ptr(), out_tables.data_ptr(),
        out_refs.data_ptr(), None if n_live is None else n_live.data_ptr(), cache.data_ptr(),
        scale.data_ptr(), wp, wn, st))


def pages_copy(cache: torch.Tensor, scale: torch.Tensor, src: torch.Tensor, dst: torch.Tensor,
               work: torch.Tensor, stream=None):
    """Copy page src[i] to page dst[i] (int32 [n]) in all layers, with its
    scales.  No page may be the target of two pairs, or target and source."""
    L, P, _, H, page, dim = _cache(cache, scale, 1)
    n = _list(src, "src")
    _ints(dst, "dst", (n,))
    wp, wn = _work(work)
    st = _here(stream, cache, scale, src, dst, work)
    _check("lora_pages_copy", _lib.load().lora_pages_copy(
        L, H, dim, page, P, cache.data_ptr(), scale.data_ptr(), src.data_ptr(), dst.data_ptr(), n,
        wp, wn, st))


def check_errors(meta: torch.Tensor, stream=None) -> int:
    """Synchronise and return the library status for device-detected bad
    indices / segments since the last check (0 = LORA_OK); clears them."""
    return _lib.load().lora_check_errors(_ptr(meta), meta.numel(), _stream(stream))


def build_info() -> str:
    return _lib.load().lora_build_info().decode()


def launch_count() -> int:
    """Kernel launches the library has made in this process (a launch recorded
    into a stream capture counts once)."""
    return int(_lib.load().lora_launch_count())
