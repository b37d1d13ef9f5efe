// Block-scaled e4m3 matrix product:
//   y[t][n] = sum_b q_scale[t][b] w_scale[n/128][b] sum_{k in b} q[t][k] W[n][k]
// with fp32 products and sums and one rounding.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

namespace {

constexpr int kMT = 64, kMN = 64, kMThreads = 256;

__device__ __forceinline__ void e4m3x16(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
    const float2 p = __half22float2(__half2(h));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

// 16 values from column c of a row of K columns, 0 past its end.
__device__ __forceinline__ uint4 load16(const uint8_t* row, int c, int K) {
  if (c + 16 <= K) return *reinterpret_cast<const uint4*>(row + c);
  uint32_t w[4] = {0, 0, 0, 0};
  for (int i = 0; i < 16; ++i)
    if (c + i < K) w[i / 4] |= (uint32_t)row[c + i] << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 64 x 64 outputs per CTA, 4 x 4 per thread, 32 columns of K at a time.
template <typename E>
__global__ void __launch_bounds__(kMThreads) matmul_fp8_kernel(MatmulFp8Args a) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  __shared__ float sq[32][kMT + 4], sw[32][kMN + 4];
  const int t0 = blockIdx.x * kMT, n0 = blockIdx.y * kMN;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int KB = (a.K + LORA_FP8_BLOCK - 1) / LORA_FP8_BLOCK;
  float acc[4][4] = {};
  for (int b = 0; b < KB; ++b) {
    float part[4][4] = {};
    for (int k0 = b * LORA_FP8_BLOCK; k0 < min(a.K, (b + 1) * LORA_FP8_BLOCK); k0 += 32) {
      __syncthreads();
      const int r = (threadIdx.x & 127) >> 1, c = (threadIdx.x & 1) * 16;
      const bool left = threadIdx.x < 128;
      const bool in = left ? t0 + r < a.T : n0 + r < a.N;
      float f[16] = {};
      if (in && k0 + c < a.K)
        e4m3x16(left ? load16(static_cast<const uint8_t*>(a.q) + (t0 + r) * a.ldq, k0 + c, a.K)
                     : load16(static_cast<const uint8_t*>(a.W) + (n0 + r) * a.ldw, k0 + c, a.K),
                f);
      for (int i = 0; i < 16; ++i) (left ? sq[c + i] : sw[c + i])[r] = f[i];
      __syncthreads();
      for (int k = 0; k < 32; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            part[i][j] = fmaf(sq[k][ty * 4 + i], sw[k][tx * 4 + j], part[i][j]);
    }
    const float ws = a.w_scale[(int64_t)(n0 / LORA_FP8_BLOCK) * KB + b];
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + ty * 4 + i;
      const float s = t < a.T ? a.q_scale[(int64_t)t * KB + b] * ws : 0.f;
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(s, part[i][j], acc[i][j]);
    }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t t = t0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (t < a.T && n < a.N)
        static_cast<uint16_t*>(a.y)[t * a.ldy + n] = Elem<E>::from_f32(acc[i][j]);
    }
}

}  // namespace

cudaError_t launch_matmul_fp8(lora_dtype dt, const MatmulFp8Args& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kMThreads, 1, 1);
  cfg.gridDim = dim3((a.T + kMT - 1) / kMT, (a.N + kMN - 1) / kMN, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return counted_launch(dt == LORA_BF16
                            ? cudaLaunchKernelEx(&cfg, matmul_fp8_kernel<__nv_bfloat16>, a)
                            : cudaLaunchKernelEx(&cfg, matmul_fp8_kernel<__half>, a));
}

}  // namespace lora
