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
// the conversion's own rounding then decides as for v itself.  (One border is a
// power of two, 2^-10 between 0 and the smallest value.  A t just below it may
// stay below: both that and the tie round to 0.)
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

// Largest magnitudes of two packed elements, and of two such pairs; a NaN stays one.
template <typename E> struct Pair;
template <> struct Pair<__half> {
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return a;
  }
};
template <> struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return a;
  }
};
template <typename E>
__device__ __forceinline__ uint32_t absmax8(const uint4& v) {
  constexpr uint32_t m = 0x7fff7fffu;
  return Pair<E>::max(Pair<E>::max(v.x & m, v.y & m), Pair<E>::max(v.z & m, v.w & m));
}
// The larger of the two halves of a pair, as fp32.
template <typename E>
__device__ __forceinline__ float larger(uint32_t v) {
  return Elem<E>::to_f32((uint16_t)Pair<E>::max(v, v >> 16));
}
__device__ __forceinline__ float max_nan(float a, float b) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
  return a;
}

// Two values times r, rounded to 18 significant bits and packed to e4m3.  For
// t = rn(x r), u = rn(65 t) has the step of 2^6 t, so u - 64 t, which is exact,
// is t rounded to 24 - 6 bits.  Two values per instruction: 71.6 us at 8192 x
// 14336 against 77.1 with a scalar product and the rounding in integer steps.
__device__ __forceinline__ uint32_t scaled2(float x0, float x1, uint64_t r2) {
  const uint64_t k64 = 0x4280000042800000ull, km64 = 0xc2800000c2800000ull;   // 64, -64
  const uint64_t t = ptx::fmul2(ptx::pack2(x0, x1), r2);
  const uint64_t h = ptx::ffma2(t, km64, ptx::ffma2(t, k64, t));
  return __nv_cvt_float2_to_fp8x2(make_float2(ptx::lo32(h), ptx::hi32(h)), __NV_SATFINITE,
                                  __NV_E4M3);
}

// 8 elements from column c of a row of K columns, 0 past the row's end.
template <typename E>
__device__ __forceinline__ uint4 load8(const E* row, int c, int K) {
  if (c + 8 <= K) return ldg_stream(row + c);
  const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < K) w[i / 2] |= (uint32_t)p[c + i] << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 values scaled by r to column c of a row of K columns.
template <typename E>
__device__ __forceinline__ void store8(uint8_t* row, int c, int K, const uint4& v, float r) {
  float f[8];
  Elem<E>::to_f32(v, f);
  const uint64_t r2 = ptx::pack2(r, r);
  const uint32_t a = scaled2(f[0], f[1], r2) | (scaled2(f[2], f[3], r2) << 16);
  const uint32_t b = scaled2(f[4], f[5], r2) | (scaled2(f[6], f[7], r2) << 16);
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
// following rows; each half-warp takes G groups, cw apart, whose loads are all
// in flight at once and whose divisions G lanes make together.
template <typename E, int G>
__global__ void __launch_bounds__(kQThreads, 6)
quant_rows_kernel(const E* x, int64_t ldx, uint8_t* q, int64_t ldq, float* scale, int T, int K,
                  int KB, int cw) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  const int hw = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int row = blockIdx.x * (kQGroups / cw) + hw / cw;
  const int kb0 = blockIdx.y * (cw * G) + hw % cw;
  uint4 v[G];
  uint32_t m[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c = (kb0 + g * cw) * LORA_FP8_BLOCK + l * 8;
    v[g] = make_uint4(0, 0, 0, 0);
    if (row < T && c < K) v[g] = load8(x + row * ldx, c, K);
  }
  float mine = 0.f;          // the largest magnitude of group l % G
#pragma unroll
  for (int g = 0; g < G; ++g) {
    m[g] = absmax8<E>(v[g]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m[g] = Pair<E>::max(m[g], __shfl_xor_sync(~0u, m[g], o));
    if (l % G == g) mine = larger<E>(m[g]);
  }
  const float a = max_nan(mine, kQTiny);
  const float r = __fdiv_rn(448.f, a);
  if (l < G && row < T && kb0 + l * cw < KB)
    scale[(int64_t)row * KB + kb0 + l * cw] = __fdiv_rn(a, 448.f);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c = (kb0 + g * cw) * LORA_FP8_BLOCK + l * 8;
    const float rg = __shfl_sync(~0u, r, (threadIdx.x & 16) + g);
    if (row < T && c < K) store8<E>(q + row * ldq, c, K, v[g], rg);
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
  uint4 v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int row = blockIdx.x * 128 + j * kQGroups + hw;
    v[j] = make_uint4(0, 0, 0, 0);
    if (row < T && c < K) v[j] = load8(x + row * ldx, c, K);
  }
  uint32_t mm = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) mm = Pair<E>::max(mm, absmax8<E>(v[j]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mm = Pair<E>::max(mm, __shfl_xor_sync(~0u, mm, o));
  float m = larger<E>(mm);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQThreads / 32; ++w) m = max_nan(m, part[w]);
  const float a = max_nan(m, kQTiny);
  const float r = __fdiv_rn(448.f, a);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int row = blockIdx.x * 128 + j * kQGroups + hw;
    if (row < T && c < K) store8<E>(q + row * ldq, c, K, v[j], r);
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
  // four groups per half-warp once there are enough to fill the device (71.6 us
  // against 93 with one at 8192 x 14336, 67.8 with six CTAs per SM; one token of
  // 4096: 2.1 us against 1.6)
  const int G = KB >= 4 && (int64_t)a.T * KB >= 32768 ? 4 : 1;
  int cw = 1;
  while (cw < kQGroups && cw * G < KB) cw *= 2;
  const unsigned gx = (a.T + kQGroups / cw - 1) / (kQGroups / cw);
  cfg.gridDim = dim3(gx, (KB + cw * G - 1) / (cw * G), 1);
  return counted_launch(G == 4 ? cudaLaunchKernelEx(&cfg, quant_rows_kernel<E, 4>, x, a.ldx, q,
                                                    a.ldq, a.scale, a.T, a.K, KB, cw)
                               : cudaLaunchKernelEx(&cfg, quant_rows_kernel<E, 1>, x, a.ldx, q,
                                                    a.ldq, a.scale, a.T, a.K, KB, cw));
}

}  // namespace

cudaError_t launch_quantize_fp8(lora_dtype dt, const QuantArgs& a, cudaStream_t st) {
  return dt == LORA_BF16 ? quant_launch<__nv_bfloat16>(a, st) : quant_launch<__half>(a, st);
}

}  // namespace lora
