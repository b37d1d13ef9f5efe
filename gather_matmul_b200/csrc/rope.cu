// Rotary positions on head slices, with or without the norm of each head:
//   n = x w / sqrt(mean(x^2) + eps),   (a, b) -> m (a cos - b sin, b cos + a sin)
// at the angle positions[t] * inv_freq[i].
//
// The angle is formed in turns in fp64 and reduced to [-1/2, 1/2] there (a
// position of 2^20 and a frequency of 1 leave fp32 no bits below 2^-4 of a
// radian); sine and cosine are then taken in fp32.  Each CTA does that once
// per token for all its heads, into shared memory, while its loads of the
// heads are in flight.
//
// Bound: memory (2 bytes read and 2 written per element).  A group of L lanes
// holds one head: each lane the two vectors of V elements that its pairs join,
// so a half-split rotation needs no exchange between lanes, and the norm needs
// one sum over the L lanes.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

namespace {

template <int V> struct Vec;
template <> struct Vec<8> { typedef uint4 type; };
template <> struct Vec<4> { typedef uint2 type; };
template <> struct Vec<2> { typedef uint32_t type; };
template <> struct Vec<1> { typedef uint16_t type; };

template <typename E, int V>
__device__ __forceinline__ void unpack(const typename Vec<V>::type& v, float* f) {
  const uint16_t* h = reinterpret_cast<const uint16_t*>(&v);
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = Elem<E>::to_f32(h[i]);
}
template <typename E, int V>
__device__ __forceinline__ typename Vec<V>::type pack(const float* f) {
  typename Vec<V>::type v;
  if constexpr (V == 1) {
    v = Elem<E>::from_f32(f[0]);
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = Elem<E>::pack2(f[2 * i], f[2 * i + 1]);
  }
  return v;
}

constexpr int kRThreads = 512;   // most threads of a CTA

struct RopeGrid {
  int L;            // lanes per head, a power of two up to 32
  int heads_cta;    // heads per CTA and token
  int tokens_cta;   // tokens per CTA
};

// ITEMS pair vectors per lane: units of V pairs u, u + L, ... of the head's
// dim / 2 / V; the first rot / 2 / V of them are rotated.
template <typename E, int V, int ITEMS, bool INTER, bool NORM>
__global__ void __launch_bounds__(kRThreads) rope_kernel(const RopeArgs a, const RopeGrid G) {
  typedef typename Vec<V>::type vec;
  extern __shared__ float2 cs[];          // [tokens_cta][rot / 2]
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  const int h = a.rot / 2, pass = (a.dim - a.rot) / 2;
  const int units = a.dim / 2 / V, turned = h / V;
  const int n_heads = a.head_end[a.n_slices - 1];
  const int slot = threadIdx.x / G.L, l = threadIdx.x % G.L;
  const int tok = slot / G.heads_cta;
  const int64_t t0 = (int64_t)blockIdx.x * G.tokens_cta;
  const int64_t t = t0 + tok;
  const int head = blockIdx.y * G.heads_cta + slot % G.heads_cta;
  const bool active = tok < G.tokens_cta && t < a.T && head < n_heads;
  int s = 0, in_slice = head;
  if (active) {
    while (head >= a.head_end[s]) ++s;
    in_slice = head - (s > 0 ? a.head_end[s - 1] : 0);
  }
  const E* x = static_cast<const E*>(a.x) + t * a.ldx + a.x_off[s] + (int64_t)in_slice * a.dim;
  vec va[ITEMS], vb[ITEMS];
  int ea[ITEMS], eb[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int u = l + i * G.L;
    if constexpr (INTER) {
      ea[i] = 2 * V * u;
      eb[i] = ea[i] + V;
    } else {
      ea[i] = u < turned ? u * V : a.rot + (u - turned) * V;
      eb[i] = ea[i] + (u < turned ? h : pass);
    }
    va[i] = vec();
    vb[i] = vec();
    if (active && u < units) {
      va[i] = *reinterpret_cast<const vec*>(x + ea[i]);
      vb[i] = *reinterpret_cast<const vec*>(x + eb[i]);
    }
  }
  for (int i = threadIdx.x; i < G.tokens_cta * h; i += blockDim.x) {
    const int64_t tt = t0 + i / h;
    if (tt >= a.T) break;
    const double turns = (double)a.positions[tt] * (a.inv_freq[i % h] * 0.15915494309189533577);
    float sn, c;
    sincospif(2.f * (float)(turns - rint(turns)), &sn, &c);
    cs[i] = make_float2(c * a.attn_scale, sn * a.attn_scale);
  }
  __syncthreads();
  float fa[ITEMS][V], fb[ITEMS][V];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    unpack<E, V>(va[i], fa[i]);
    unpack<E, V>(vb[i], fb[i]);
  }
  if constexpr (NORM) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) sum = fmaf(fa[i][j], fa[i][j], fmaf(fb[i][j], fb[i][j], sum));
    for (int o = G.L >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    const E* w = static_cast<const E*>(a.weight[s]);
    if (active && w != nullptr) {
      const float inv = 1.f / sqrtf(sum / (float)a.dim + a.eps);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        if (l + i * G.L < units) {
          float wa[V], wb[V];
          unpack<E, V>(*reinterpret_cast<const vec*>(w + ea[i]), wa);
          unpack<E, V>(*reinterpret_cast<const vec*>(w + eb[i]), wb);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            fa[i][j] *= inv * wa[j];
            fb[i][j] *= inv * wb[j];
          }
        }
      }
    }
  }
  if (!active) return;
  E* y = static_cast<E*>(a.y) + t * a.ldy + a.y_off[s] + (int64_t)in_slice * a.dim;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int u = l + i * G.L;
    if (u < units) {
      if (u < turned) {
        const float2* c = cs + tok * h + u * V;
        if constexpr (INTER && V > 1) {
          // pairs lie inside each vector: V / 2 in va, V / 2 in vb
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            const float2 p = c[j], q = c[j + V / 2];
            const float a0 = fa[i][2 * j], a1 = fa[i][2 * j + 1];
            const float b0 = fb[i][2 * j], b1 = fb[i][2 * j + 1];
            fa[i][2 * j] = a0 * p.x - a1 * p.y;
            fa[i][2 * j + 1] = a1 * p.x + a0 * p.y;
            fb[i][2 * j] = b0 * q.x - b1 * q.y;
            fb[i][2 * j + 1] = b1 * q.x + b0 * q.y;
          }
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float2 p = c[j];
            const float u0 = fa[i][j], u1 = fb[i][j];
            fa[i][j] = u0 * p.x - u1 * p.y;
            fb[i][j] = u1 * p.x + u0 * p.y;
          }
        }
      }
      *reinterpret_cast<vec*>(y + ea[i]) = pack<E, V>(fa[i]);
      *reinterpret_cast<vec*>(y + eb[i]) = pack<E, V>(fb[i]);
    }
  }
}

template <typename E, int V, int ITEMS, bool INTER>
cudaError_t rope_launch(const RopeArgs& a, bool norm, cudaStream_t st) {
  const int units = a.dim / 2 / V, n_heads = a.head_end[a.n_slices - 1];
  RopeGrid G;
  G.L = 1;
  while (G.L < 32 && G.L < units) G.L *= 2;
  const int slots = kRThreads / G.L;
  const int chunks = (n_heads + slots - 1) / slots;
  G.heads_cta = (n_heads + chunks - 1) / chunks;
  G.tokens_cta = chunks > 1 ? 1 : min(max(256 / G.L / n_heads, 1), a.T);
  const int threads = (G.heads_cta * G.tokens_cta * G.L + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.T + G.tokens_cta - 1) / G.tokens_cta, chunks, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = sizeof(float2) * (size_t)G.tokens_cta * (a.rot / 2);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return counted_launch(
      norm ? cudaLaunchKernelEx(&cfg, rope_kernel<E, V, ITEMS, INTER, true>, a, G)
           : cudaLaunchKernelEx(&cfg, rope_kernel<E, V, ITEMS, INTER, false>, a, G));
}

template <typename E, int V, int ITEMS>
cudaError_t rope_layout(const RopeArgs& a, bool norm, cudaStream_t st) {
  return a.interleaved ? rope_launch<E, V, ITEMS, true>(a, norm, st)
                       : rope_launch<E, V, ITEMS, false>(a, norm, st);
}

// The widest vector whose length divides both the rotated pairs and the rest:
// every access is then aligned (columns and rows are multiples of 8 elements).
template <typename E>
cudaError_t rope_width(const RopeArgs& a, bool norm, cudaStream_t st) {
  const int both = (a.rot / 2) | ((a.dim - a.rot) / 2);
  if (both % 8 == 0) return rope_layout<E, 8, 1>(a, norm, st);
  if (both % 4 == 0) return rope_layout<E, 4, 1>(a, norm, st);
  if (both % 2 == 0) return rope_layout<E, 2, 2>(a, norm, st);
  return rope_layout<E, 1, 4>(a, norm, st);
}

}  // namespace

cudaError_t launch_rope(lora_dtype dt, const RopeArgs& a, bool norm, cudaStream_t st) {
  return dt == LORA_BF16 ? rope_width<__nv_bfloat16>(a, norm, st)
                         : rope_width<__half>(a, norm, st);
}

}  // namespace lora
