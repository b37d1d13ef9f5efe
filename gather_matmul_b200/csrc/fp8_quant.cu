// Quantise fp16/bf16 to e4m3 with one fp32 scale per group of 128 columns of a
// row, or per 128 x 128 block:
//   a = max(max |x|, 2^-100),  scale = rn(a / 448),  q = rn_e4m3(448 x / a).
//
// q is the real quotient rounded once, without a division per element.  With
// r = rn(448 / a) and t = rn(x r), t is within 2^-23 (relative) of the
// quotient v = 448 x / a.  x and a have at most 11 significant bits, and a
// border between two e4m3 values is m 2^k with m < 2^5, so v is either exactly
// a border or at least 2^-16 (relative) away from every border:
// |7 X 2^p - m A| / (m A) >= 1 / (m A) for the integer significands X, A.
// Rounding t to 18 bits therefore puts it exactly on the border in the first
// case and, moving it by at most 2^-18, leaves it on its side in the second;
// the conversion's own rounding then decides as for v itself.
//
// Bound: memory (2 bytes read and 1 written per element).
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

namespace {

constexpr int kQThreads = 256;
constexpr int kQGroups = kQThreads / 16;   // 16 lanes x 8 elements = one group of 128
constexpr float kQTiny = 7.888609052210118e-31f;   // 2^-100

// Largest magnitude of 8 packed elements; a NaN stays one.
template <typename E>
__device__ __forceinline__ float absmax8(const float* f) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = fabsf(f[i]);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(v));
  }
  return m;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
  return a;
}

// x * r rounded to 18 significant bits (Veltkamp's splitting with 2^6 + 1);
// the intrinsics keep the compiler from contracting the steps.
__device__ __forceinline__ float scaled18(float x, float r) {
  const float t = __fmul_rn(x, r);
  const float c = __fmul_rn(t, 65.f);
  return __fsub_rn(c, __fsub_rn(c, t));
}

__device__ __forceinline__ uint32_t to_e4m3x4(const float* f, float r) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(scaled18(f[0], r), scaled18(f[1], r)),
                                               __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(scaled18(f[2], r), scaled18(f[3], r)),
                                               __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// 8 elements from column c of a row of K columns, 0 past the row's end.
template <typename E>
__device__ __forceinline__ void load8(const E* row, int c, int K, float* f) {
  if (c + 8 <= K) {
    Elem<E>::to_f32(ldg_stream(row + c), f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = c + i < K ? Elem<E>::to_f32(reinterpret_cast<const uint16_t*>(row)[c + i]) : 0.f;
  }
}

__device__ __forceinline__ void store8(uint8_t* row, int c, int K, uint32_t a, uint32_t b) {
  if (c + 8 <= K) {
    *reinterpret_cast<uint2*>(row + c) = make_uint2(a, b);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < K) row[c + i] = (uint8_t)((i < 4 ? a : b) >> (8 * (i & 3)));
  }
}

// One half-warp per group of 128 columns of one row.  cw (a power of two, at
// most 16) half-warps of a CTA lie side by side in a row, the rest in the
// following rows; each half-warp takes G groups, cw apart.
template <typename E, int G>
__global__ void __launch_bounds__(kQThreads)
quant_rows_kernel(const E* x, int64_t ldx, uint8_t* q, int64_t ldq, float* scale, int T, int K,
                  int KB, int cw) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  const int hw = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int row = blockIdx.x * (kQGroups / cw) + hw / cw;
  const int kb0 = blockIdx.y * (cw * G) + hw % cw;
  float f[G][8], m[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c = (kb0 + g * cw) * LORA_FP8_BLOCK + l * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[g][i] = 0.f;
    if (row < T && c < K) load8(x + row * ldx, c, K, f[g]);
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    m[g] = absmax8<E>(f[g]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m[g] = max_nan(m[g], __shfl_xor_sync(~0u, m[g], o));
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int kb = kb0 + g * cw;
    const int c = kb * LORA_FP8_BLOCK + l * 8;
    const float a = max_nan(m[g], kQTiny);
    const float r = __fdiv_rn(448.f, a);
    if (row < T && c < K) {
      store8(q + row * ldq, c, K, to_e4m3x4(f[g], r), to_e4m3x4(f[g] + 4, r));
      if (l == 0) scale[(int64_t)row * KB + kb] = __fdiv_rn(a, 448.f);
    }
  }
}

// One CTA per 128 x 128 block, 8 rows per half-warp.
template <typename E>
__global__ void __launch_bounds__(kQThreads)
quant_blocks_kernel(const E* x, int64_t ldx, uint8_t* q, int64_t ldq, float* scale, int T, int K,
                    int KB) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  __shared__ float part[kQThreads / 32];
  const int hw = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int c = blockIdx.y * LORA_FP8_BLOCK + l * 8;
  float f[8][8], m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int row = blockIdx.x * 128 + j * kQGroups + hw;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[j][i] = 0.f;
    if (row < T && c < K) load8(x + row * ldx, c, K, f[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max_nan(m, absmax8<E>(f[j]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(~0u, m, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQThreads / 32; ++w) m = max_nan(m, part[w]);
  const float a = max_nan(m, kQTiny);
  const float r = __fdiv_rn(448.f, a);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int row = blockIdx.x * 128 + j * kQGroups + hw;
    if (row < T && c < K)
      store8(q + row * ldq, c, K, to_e4m3x4(f[j], r), to_e4m3x4(f[j] + 4, r));
  }
  if (threadIdx.x == 0) scale[(int64_t)blockIdx.x * KB + blockIdx.y] = __fdiv_rn(a, 448.f);
}

template <typename E>
cudaError_t quant_launch(const QuantArgs& a, cudaStream_t st) {
  const int KB = (a.K + LORA_FP8_BLOCK - 1) / LORA_FP8_BLOCK;
  const E* x = static_cast<const E*>(a.x);
  uint8_t* q = static_cast<uint8_t*>(a.q);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kQThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.block_rows != 1) {
    cfg.gridDim = dim3((a.T + 127) / 128, KB, 1);
    return counted_launch(cudaLaunchKernelEx(&cfg, quant_blocks_kernel<E>, x, a.ldx, q, a.ldq,
                                             a.scale, a.T, a.K, KB));
  }
  int cw = 1;
  while (cw < kQGroups && cw < KB) cw *= 2;
  const unsigned gx = (a.T + kQGroups / cw - 1) / (kQGroups / cw);
  cfg.gridDim = dim3(gx, (KB + cw - 1) / cw, 1);
  return counted_launch(cudaLaunchKernelEx(&cfg, quant_rows_kernel<E, 1>, x, a.ldx, q, a.ldq,
                                           a.scale, a.T, a.K, KB, cw));
}

}  // namespace

cudaError_t launch_quantize_fp8(lora_dtype dt, const QuantArgs& a, cudaStream_t st) {
  return dt == LORA_BF16 ? quant_launch<__nv_bfloat16>(a, st) : quant_launch<__half>(a, st);
}

}  // namespace lora
