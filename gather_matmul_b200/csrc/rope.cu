// Rotary positions on head slices, with or without the norm of each head:
//   n = x w / sqrt(mean(x^2) + eps),   (a, b) -> m (a cos - b sin, b cos + a sin)
// at the angle positions[t] * inv_freq[i].
//
// The angle is formed in turns in fp64, with what the products round off carried
// along, and reduced to about [-1/2, 1/2] there (a position of 2^20 and a
// frequency of 1 leave fp32 no bits below 2^-4 of a radian; plain fp64 is off by
// 2e-8 turns at 2^30 and by 0.2 at 2^53); sine and cosine are then taken in fp32.
// Each CTA does that once per token for all its heads, into shared memory, while
// its loads of the heads are in flight.
//
// Bound: memory (2 bytes read and 2 written per element; 28.1 us at 8192 tokens
// of 32 + 8 heads of 128, 6.0 TB/s), with norms nearly as much by the issue of
// instructions (36.4 us; packed fp32 arithmetic needed more registers: 42.6).  A
// group of L lanes holds one head: each lane the two vectors of V elements that its
// pairs join, so a half-split rotation needs no exchange between lanes, and the
// norm needs one sum over the L lanes.
// The order of the table decides much: with (cos, sin) pairs in the order of the
// pairs, lanes read it with 4-way bank conflicts, and the same call took 35 us.
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

template <int W> struct Floats;
template <> struct Floats<4> { typedef float4 type; };
template <> struct Floats<2> { typedef float2 type; };
template <> struct Floats<1> { typedef float type; };

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

// Most threads of a CTA: with 512 the rotation took 29.9 us (38.2 with norms) at
// 8192 tokens of 32 + 8 heads of 128, with 128 30.4 (42.5).
constexpr int kRThreads = 256;

// The registers of a thread, as CTAs per SM of so many threads.  Without norms 48,
// in which the two-token kernels spill 12 to 32 bytes (8 elements to a vector; up
// to 96 with single elements): 28.1 us at 8192 tokens of 40 heads of 128.  64 leave
// 27.8 there, but 32.3 against 29.3 at 2048 tokens of 72 heads of 80.  With norms
// 64, which spill next to nothing: 3.5 us at 512 tokens (4.0 with 48); two tokens
// with 8 elements to a vector 56 (4 to 36 bytes spilled): 36.4 us at 8192 tokens,
// 37.3 with 64, 38.1 with 48.
constexpr int rope_threads(int V, int TPT, bool norm) {
  return norm && V == 8 && TPT == 2 ? 288 : kRThreads;
}
constexpr int rope_ctas(bool norm) { return norm ? 4 : 5; }

// position * f / (2 pi) less a whole number near it.  g + gl are the turns per
// position to a part in 2^104, and position * g - n is rounded once, as a whole:
// |position| < 2^53 and f up to 1 leave the result within 5/8 and off by 2^-52 at
// most (of its own size, in the usual positions).
__device__ __forceinline__ float turn(int64_t position, double f) {
  constexpr double kInv = 0x1.45f306dc9c883p-3, kRest = -0x1.6b01ec5417056p-57;   // 1 / (2 pi)
  const double x = (double)position, g = f * kInv, gl = fma(f, kRest, fma(f, kInv, -g));
  const double n = rint(x * g);
  return (float)fma(x, gl, fma(x, g, -n));
}

struct RopeGrid {
  int L;            // lanes per head, a power of two up to 32
  int heads_cta;    // heads per CTA and token
  int slots;        // groups of TPT tokens per CTA
};

// ITEMS pair vectors per lane: units of V pairs u, u + L, ... of the head's
// dim / 2 / V; the first rot / 2 / V of them are rotated.  TPT consecutive
// tokens per thread, all of whose loads are in flight at once.
template <typename E, int V, int ITEMS, int TPT, bool INTER, bool NORM>
__global__ void __launch_bounds__(rope_threads(V, TPT, NORM), rope_ctas(NORM))
    rope_kernel(const RopeArgs a, const RopeGrid G) {
  typedef typename Vec<V>::type vec;
  extern __shared__ float4 cs4[];         // [slots * TPT][rot]
  float* cs = reinterpret_cast<float*>(cs4);
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  const int h = a.rot / 2, pass = (a.dim - a.rot) / 2;
  const int units = a.dim / 2 / V, turned = h / V;
  // A token's table: the W cosines (then sines) of a unit that one access takes lie
  // side by side, units next to each other, so that lanes read without conflicts.
  constexpr int W = V < 4 ? V : 4;
  const auto put = [&](float* t, int i, float c, float sn) {
    const int u = i / V, j = i % V;
    t[((j / W) * turned + u) * W + j % W] = c;
    t[((V / W + j / W) * turned + u) * W + j % W] = sn;
  };
  const auto get = [&](const float* t, int u, float* c, float* sn) {
    typedef typename Floats<W>::type vf;
#pragma unroll
    for (int q = 0; q < V / W; ++q) {
      *reinterpret_cast<vf*>(c + q * W) = *reinterpret_cast<const vf*>(t + (q * turned + u) * W);
      *reinterpret_cast<vf*>(sn + q * W) =
          *reinterpret_cast<const vf*>(t + ((V / W + q) * turned + u) * W);
    }
  };
  const int n_heads = a.head_end[a.n_slices - 1];
  const int place = threadIdx.x / G.L, l = threadIdx.x % G.L;
  const int slot = place / G.heads_cta;
  const int64_t first = (int64_t)blockIdx.x * G.slots * TPT;
  const int64_t t0 = first + slot * TPT;
  const int head = blockIdx.y * G.heads_cta + place % G.heads_cta;
  const bool active = slot < G.slots && t0 < a.T && head < n_heads;
  int s = 0, in_slice = head;
  if (active) {
    while (head >= a.head_end[s]) ++s;
    in_slice = head - (s > 0 ? a.head_end[s - 1] : 0);
  }
  const E* x = static_cast<const E*>(a.x) + t0 * a.ldx + a.x_off[s] + (int64_t)in_slice * a.dim;
  const E* w = NORM ? static_cast<const E*>(a.weight[s]) : nullptr;
  vec va[TPT][ITEMS], vb[TPT][ITEMS], wa[ITEMS], wb[ITEMS];
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
#pragma unroll
    for (int k = 0; k < TPT; ++k) {
      va[k][i] = vec();
      vb[k][i] = vec();
      if (active && u < units && t0 + k < a.T) {
        va[k][i] = *reinterpret_cast<const vec*>(x + k * a.ldx + ea[i]);
        vb[k][i] = *reinterpret_cast<const vec*>(x + k * a.ldx + eb[i]);
      }
    }
    if constexpr (NORM) {
      wa[i] = vec();
      wb[i] = vec();
      if (active && w != nullptr && u < units) {
        wa[i] = *reinterpret_cast<const vec*>(w + ea[i]);
        wb[i] = *reinterpret_cast<const vec*>(w + eb[i]);
      }
    }
  }
  for (int i = threadIdx.x; i < G.slots * TPT * h; i += blockDim.x) {
    const int64_t tt = first + i / h;
    if (tt >= a.T) break;
    float sn, c;
    sincospif(2.f * turn(a.positions[tt], a.inv_freq[i % h]), &sn, &c);
    put(cs + (i / h) * a.rot, i % h, c * a.attn_scale, sn * a.attn_scale);
  }
  __syncthreads();
  E* y = static_cast<E*>(a.y) + t0 * a.ldy + a.y_off[s] + (int64_t)in_slice * a.dim;
#pragma unroll
  for (int k = 0; k < TPT; ++k) {
    float fa[ITEMS][V], fb[ITEMS][V];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      unpack<E, V>(va[k][i], fa[i]);
      unpack<E, V>(vb[k][i], fb[i]);
    }
    if constexpr (NORM) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) sum = fmaf(fa[i][j], fa[i][j], fmaf(fb[i][j], fb[i][j], sum));
      for (int o = G.L >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
      if (w != nullptr) {
        const float inv = rsqrtf(fmaf(sum, a.inv_dim, a.eps));
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          float ga[V], gb[V];
          unpack<E, V>(wa[i], ga);
          unpack<E, V>(wb[i], gb);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            fa[i][j] *= inv * ga[j];
            fb[i][j] *= inv * gb[j];
          }
        }
      }
    }
    if (!active || t0 + k >= a.T) continue;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int u = l + i * G.L;
      if (u < units) {
        if (u < turned) {
          alignas(16) float co[V], si[V];
          get(cs + (slot * TPT + k) * a.rot, u, co, si);
          if constexpr (INTER && V > 1) {
            // pairs lie inside each vector: V / 2 in va, V / 2 in vb
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
              const float a0 = fa[i][2 * j], a1 = fa[i][2 * j + 1];
              const float b0 = fb[i][2 * j], b1 = fb[i][2 * j + 1];
              fa[i][2 * j] = a0 * co[j] - a1 * si[j];
              fa[i][2 * j + 1] = a1 * co[j] + a0 * si[j];
              fb[i][2 * j] = b0 * co[j + V / 2] - b1 * si[j + V / 2];
              fb[i][2 * j + 1] = b1 * co[j + V / 2] + b0 * si[j + V / 2];
            }
          } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
              const float u0 = fa[i][j], u1 = fb[i][j];
              fa[i][j] = u0 * co[j] - u1 * si[j];
              fb[i][j] = u1 * co[j] + u0 * si[j];
            }
          }
        }
        *reinterpret_cast<vec*>(y + k * a.ldy + ea[i]) = pack<E, V>(fa[i]);
        *reinterpret_cast<vec*>(y + k * a.ldy + eb[i]) = pack<E, V>(fb[i]);
      }
    }
  }
}

template <typename E, int V, int ITEMS, int TPT, bool INTER>
cudaError_t rope_launch(const RopeArgs& a, bool norm, cudaStream_t st) {
  const int units = a.dim / 2 / V, n_heads = a.head_end[a.n_slices - 1];
  RopeGrid G;
  G.L = 1;
  while (G.L < 32 && G.L < units) G.L *= 2;
  const int places = kRThreads / G.L;
  const int chunks = (n_heads + places - 1) / places;
  G.heads_cta = (n_heads + chunks - 1) / chunks;
  const int groups = (a.T + TPT - 1) / TPT;
  G.slots = chunks > 1 ? 1 : min(max(256 / G.L / n_heads, 1), groups);
  const int threads = (G.heads_cta * G.slots * G.L + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((groups + G.slots - 1) / G.slots, chunks, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = sizeof(float2) * (size_t)G.slots * TPT * (a.rot / 2);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return counted_launch(
      norm ? cudaLaunchKernelEx(&cfg, rope_kernel<E, V, ITEMS, TPT, INTER, true>, a, G)
           : cudaLaunchKernelEx(&cfg, rope_kernel<E, V, ITEMS, TPT, INTER, false>, a, G));
}

template <typename E, int V, int ITEMS, int TPT>
cudaError_t rope_tokens(const RopeArgs& a, bool norm, cudaStream_t st) {
  return a.interleaved ? rope_launch<E, V, ITEMS, TPT, true>(a, norm, st)
                       : rope_launch<E, V, ITEMS, TPT, false>(a, norm, st);
}

// Two tokens per thread from 3840 lanes for each of the 148 SMs on, enough to fill
// them with half the threads: at 40 heads of 128, 14.1 us against 16.1 at 3750
// tokens (17.9 against 20.2 with norms), 8.1 against 8.7 at 1776, but 4.9 against
// 4.7 at 937 and 4.6 against 3.8 at 625.  Four tokens were slower than two (31.0 us
// against 30.0 at 8192 tokens in the form of then).
constexpr int64_t kTwoTokenLanes = 148 * 3840;

template <typename E, int V, int ITEMS>
cudaError_t rope_layout(const RopeArgs& a, bool norm, cudaStream_t st) {
  const int64_t lanes = (int64_t)a.T * a.head_end[a.n_slices - 1] * (a.dim / 2 / V / ITEMS);
  return lanes >= kTwoTokenLanes ? rope_tokens<E, V, ITEMS, 2>(a, norm, st)
                                    : rope_tokens<E, V, ITEMS, 1>(a, norm, st);
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
