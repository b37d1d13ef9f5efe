// extern "C" entry points of the operators around a LoRA-wrapped projection
// (8-bit base product, rotary positions, head norms): host-side argument
// checks and dispatch.  See include/lora.h for the contract of each call.
#include <math.h>

#include "common.cuh"
#include "internal.h"

using namespace lora;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

lora_status from_cuda(cudaError_t e) { return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA; }

size_t a256(size_t v) { return (v + 255) & ~size_t(255); }
int64_t up16(int64_t v) { return (v + 15) & ~int64_t(15); }
int blocks(int n) { return (n + LORA_FP8_BLOCK - 1) / LORA_FP8_BLOCK; }

// dtype and sizes shared by the 8-bit calls (n = 1 for the quantiser)
lora_status check_sizes(lora_dtype dt, int T, int n, int K) {
  if (dt != LORA_F16 && dt != LORA_BF16) return LORA_ERR_INVALID_ARG;
  if (T < 0 || n <= 0 || K <= 0) return LORA_ERR_INVALID_ARG;
  if (T > LORA_MAX_TOKENS || n > LORA_MAX_WIDTH || K > LORA_MAX_WIDTH) return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

// a row-major operand: non-null, 16-byte aligned, rows of at least `width`
// elements that start at multiples of `mult` elements
lora_status check_rows(const void* p, int64_t ld, int64_t width, int64_t mult) {
  if (p == nullptr || ld < width) return LORA_ERR_INVALID_ARG;
  if (ld > (int64_t)1 << 38) return LORA_ERR_UNSUPPORTED;   // a tensor map's stride
  if (!aligned(p, 16) || ld % mult != 0) return LORA_ERR_MISALIGNED;
  return LORA_OK;
}

lora_status check_scale(const float* p) {
  if (p == nullptr) return LORA_ERR_INVALID_ARG;
  return aligned(p, 4) ? LORA_OK : LORA_ERR_MISALIGNED;
}

// Whether two row-major regions of `rows` rows (start address, width and row
// stride in bytes) share memory.  Regions of one matrix (equal strides) may
// interleave without sharing; otherwise their spans must be apart.
bool share(const char* p, int64_t wp, int64_t ldp, const char* q, int64_t wq, int64_t ldq,
           int64_t rows) {
  const char* pe = p + (rows - 1) * ldp + wp;
  const char* qe = q + (rows - 1) * ldq + wq;
  if (pe <= q || qe <= p) return false;
  if (ldp != ldq || rows == 1) return true;
  const int64_t d = ((q - p) % ldp + ldp) % ldp;     // q's column seen from p
  return d < wp || ldp - d < wq;
}

lora_status rope_impl(lora_dtype dtype, int T, int dim, int rot, int n_slices,
                      const int32_t* heads, const void* x, int64_t ldx, const int64_t* x_col_off,
                      const void* const* weight, float eps, bool norm, void* y, int64_t ldy,
                      const int64_t* y_col_off, const int64_t* positions, const double* inv_freq,
                      float attn_scale, int interleaved, lora_stream_t stream) {
  if (dtype != LORA_F16 && dtype != LORA_BF16) return LORA_ERR_INVALID_ARG;
  if (T < 0 || dim <= 0 || rot <= 0 || n_slices < 0) return LORA_ERR_INVALID_ARG;
  if (T > LORA_MAX_TOKENS || dim > LORA_MAX_HEAD_DIM || dim % 8 != 0 || n_slices < 1 ||
      n_slices > LORA_MAX_SLICES)
    return LORA_ERR_UNSUPPORTED;
  if (rot > dim || rot % 2 != 0) return LORA_ERR_INVALID_ARG;
  if (heads == nullptr || x_col_off == nullptr || y_col_off == nullptr) return LORA_ERR_INVALID_ARG;
  if (!isfinite(attn_scale)) return LORA_ERR_INVALID_ARG;
  if (norm && (weight == nullptr || !isfinite(eps) || eps <= 0.f)) return LORA_ERR_INVALID_ARG;
  RopeArgs a = {};
  int64_t total = 0;
  for (int i = 0; i < n_slices; ++i) {
    if (heads[i] <= 0 || x_col_off[i] < 0 || y_col_off[i] < 0) return LORA_ERR_INVALID_ARG;
    total += heads[i];
    if (total > LORA_MAX_HEADS) return LORA_ERR_UNSUPPORTED;
    const int64_t w = (int64_t)heads[i] * dim;
    if (x_col_off[i] > ldx - w || y_col_off[i] > ldy - w) return LORA_ERR_INVALID_ARG;
    if (x_col_off[i] % 8 != 0 || y_col_off[i] % 8 != 0) return LORA_ERR_MISALIGNED;
    a.head_end[i] = (int)total;
    a.x_off[i] = x_col_off[i];
    a.y_off[i] = y_col_off[i];
    a.weight[i] = norm ? weight[i] : nullptr;
    if (!aligned(a.weight[i], 16)) return LORA_ERR_MISALIGNED;
  }
  if (T == 0) return LORA_OK;
  lora_status s = check_rows(x, ldx, 1, 8);
  if (s == LORA_OK) s = check_rows(y, ldy, 1, 8);
  if (s != LORA_OK) return s;
  if (positions == nullptr || inv_freq == nullptr) return LORA_ERR_INVALID_ARG;
  if (!aligned(positions, 8) || !aligned(inv_freq, 8)) return LORA_ERR_MISALIGNED;
  for (int i = 0; i < n_slices; ++i) {
    const char* yi = static_cast<const char*>(y) + 2 * y_col_off[i];
    const int64_t wi = 2 * (int64_t)heads[i] * dim;
    for (int j = 0; j < n_slices; ++j) {
      const char* xj = static_cast<const char*>(x) + 2 * x_col_off[j];
      const char* yj = static_cast<const char*>(y) + 2 * y_col_off[j];
      const int64_t wj = 2 * (int64_t)heads[j] * dim;
      // a single row has no next one, so its strides need not agree
      const bool in_place = i == j && yi == xj && (ldx == ldy || T == 1);
      if (!in_place && share(yi, wi, 2 * ldy, xj, wj, 2 * ldx, T)) return LORA_ERR_INVALID_ARG;
      if (j < i && share(yi, wi, 2 * ldy, yj, wj, 2 * ldy, T)) return LORA_ERR_INVALID_ARG;
    }
  }
  a.x = x;
  a.ldx = ldx;
  a.y = y;
  a.ldy = ldy;
  a.n_slices = n_slices;
  a.T = T;
  a.dim = dim;
  a.rot = rot;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.attn_scale = attn_scale;
  a.eps = eps;
  a.inv_dim = 1.f / (float)dim;
  a.interleaved = interleaved != 0;
  cudaGetLastError();
  return from_cuda(launch_rope(dtype, a, norm, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

lora_status lora_quantize_fp8(lora_dtype dtype, int T, int K, int block_rows, const void* x,
                              int64_t ldx, void* q, int64_t ldq, float* scale,
                              lora_stream_t stream) {
  lora_status s = check_sizes(dtype, T, 1, K);
  if (s != LORA_OK) return s;
  if (block_rows != 1 && block_rows != LORA_FP8_BLOCK) return LORA_ERR_UNSUPPORTED;
  if (T == 0) return LORA_OK;
  s = check_rows(x, ldx, K, 8);
  if (s == LORA_OK) s = check_rows(q, ldq, K, 16);
  if (s == LORA_OK) s = check_scale(scale);
  if (s != LORA_OK) return s;
  const QuantArgs a = {x, ldx, q, ldq, scale, T, K, block_rows};
  cudaGetLastError();
  return from_cuda(launch_quantize_fp8(dtype, a, (cudaStream_t)stream));
}

lora_status lora_matmul_fp8(lora_dtype dtype, int T, int N, int K, const void* q, int64_t ldq,
                            const float* q_scale, const void* W, int64_t ldw,
                            const float* w_scale, void* y, int64_t ldy, lora_stream_t stream) {
  lora_status s = check_sizes(dtype, T, N, K);
  if (s != LORA_OK) return s;
  if (T == 0) return LORA_OK;
  s = check_rows(q, ldq, K, 16);
  if (s == LORA_OK) s = check_rows(W, ldw, K, 16);
  if (s == LORA_OK) s = check_rows(y, ldy, N, 8);
  if (s == LORA_OK) s = check_scale(q_scale);
  if (s == LORA_OK) s = check_scale(w_scale);
  if (s != LORA_OK) return s;
  const MatmulFp8Args a = {q, ldq, q_scale, W, ldw, w_scale, y, ldy, T, N, K, 0};
  cudaGetLastError();
  return from_cuda(launch_matmul_fp8(dtype, a, (cudaStream_t)stream));
}

size_t lora_linear_fp8_workspace_bytes(int T, int K) {
  if (T < 0 || T > LORA_MAX_TOKENS || K < 1 || K > LORA_MAX_WIDTH) return 0;
  const size_t rows = T > 0 ? T : 1;
  return a256(rows * up16(K)) + a256(sizeof(float) * rows * blocks(K));
}

lora_status lora_linear_fp8(lora_dtype dtype, int T, int N, int K, const void* x, int64_t ldx,
                            const void* W, int64_t ldw, const float* w_scale, void* y,
                            int64_t ldy, void* work, size_t work_bytes, lora_stream_t stream) {
  lora_status s = check_sizes(dtype, T, N, K);
  if (s != LORA_OK) return s;
  if (work == nullptr || work_bytes < lora_linear_fp8_workspace_bytes(T, K))
    return LORA_ERR_INVALID_ARG;
  if (!aligned(work, 256)) return LORA_ERR_MISALIGNED;
  if (T == 0) return LORA_OK;
  s = check_rows(x, ldx, K, 8);
  if (s == LORA_OK) s = check_rows(W, ldw, K, 16);
  if (s == LORA_OK) s = check_rows(y, ldy, N, 8);
  if (s == LORA_OK) s = check_scale(w_scale);
  if (s != LORA_OK) return s;
  float* scale = reinterpret_cast<float*>(static_cast<char*>(work) + a256((size_t)T * up16(K)));
  const QuantArgs qa = {x, ldx, work, up16(K), scale, T, K, 1};
  const MatmulFp8Args ma = {work, up16(K), scale, W, ldw, w_scale, y, ldy, T, N, K, 1};
  cudaGetLastError();
  cudaError_t e = launch_quantize_fp8(dtype, qa, (cudaStream_t)stream);
  if (e == cudaSuccess) e = launch_matmul_fp8(dtype, ma, (cudaStream_t)stream);
  return from_cuda(e);
}

lora_status lora_rope_frequencies(int rot, double base, lora_rope_kind kind, double factor,
                                  double original_length, double beta_fast, double beta_slow,
                                  double* inv_freq, float* attn_scale) {
  const double two_pi = 6.283185307179586477;
  if (rot < 2 || rot % 2 != 0 || inv_freq == nullptr || attn_scale == nullptr)
    return LORA_ERR_INVALID_ARG;
  if (rot > LORA_MAX_HEAD_DIM) return LORA_ERR_UNSUPPORTED;
  if (!(base > 1.0) || !isfinite(base)) return LORA_ERR_INVALID_ARG;
  if (kind < LORA_ROPE_NONE || kind > LORA_ROPE_BANDS) return LORA_ERR_INVALID_ARG;
  if (kind != LORA_ROPE_NONE && (!(factor > 0.0) || !isfinite(factor))) return LORA_ERR_INVALID_ARG;
  if (kind == LORA_ROPE_NTK && rot < 4) return LORA_ERR_INVALID_ARG;
  const bool by_turns = kind == LORA_ROPE_YARN || kind == LORA_ROPE_BANDS;
  if (by_turns && (!(original_length > 0.0) || !isfinite(original_length) || !(beta_slow > 0.0) ||
                   !(beta_fast > beta_slow) || !isfinite(beta_fast)))
    return LORA_ERR_INVALID_ARG;
  if (kind == LORA_ROPE_NTK) base *= pow(factor, (double)rot / (rot - 2));
  double low = 0, high = 0;
  if (kind == LORA_ROPE_YARN) {
    // the (real) pair index that makes `turns` turns over the original length
    const double c = rot / (2.0 * log(base));
    low = fmax(floor(c * log(original_length / (beta_fast * two_pi))), 0.0);
    high = fmin(ceil(c * log(original_length / (beta_slow * two_pi))), (double)rot - 1);
  }
  *attn_scale = kind == LORA_ROPE_YARN && factor > 1.0 ? (float)(0.1 * log(factor) + 1.0) : 1.f;
  for (int i = 0; i < rot / 2; ++i) {
    double f = pow(base, -2.0 * i / rot);
    if (kind == LORA_ROPE_LINEAR) f /= factor;
    if (kind == LORA_ROPE_YARN) {
      const double u = fmin(fmax((i - low) / fmax(high - low, 1e-3), 0.0), 1.0);
      f = f / factor * u + f * (1.0 - u);
    }
    if (kind == LORA_ROPE_BANDS) {
      const double turns = original_length * f / two_pi;
      const double u =
          fmin(fmax((turns - beta_slow) / (beta_fast - beta_slow), 0.0), 1.0);
      f = (1.0 - u) * f / factor + u * f;
    }
    inv_freq[i] = f;
  }
  return LORA_OK;
}

lora_status lora_rope(lora_dtype dtype, int T, int head_dim, int rot, int n_slices,
                      const int32_t* heads, const void* x, int64_t ldx, const int64_t* x_col_off,
                      void* y, int64_t ldy, const int64_t* y_col_off, const int64_t* positions,
                      const double* inv_freq, float attn_scale, int interleaved,
                      lora_stream_t stream) {
  return rope_impl(dtype, T, head_dim, rot, n_slices, heads, x, ldx, x_col_off, nullptr, 1.f,
                   false, y, ldy, y_col_off, positions, inv_freq, attn_scale, interleaved, stream);
}

lora_status lora_norm_rope(lora_dtype dtype, int T, int head_dim, int rot, int n_slices,
                           const int32_t* heads, const void* x, int64_t ldx,
                           const int64_t* x_col_off, const void* const* weight, float eps, void* y,
                           int64_t ldy, const int64_t* y_col_off, const int64_t* positions,
                           const double* inv_freq, float attn_scale, int interleaved,
                           lora_stream_t stream) {
  return rope_impl(dtype, T, head_dim, rot, n_slices, heads, x, ldx, x_col_off, weight, eps, true,
                   y, ldy, y_col_off, positions, inv_freq, attn_scale, interleaved, stream);
}

}  // extern "C"
