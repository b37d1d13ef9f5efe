// Attention of many queries over the paged 8-bit cache (lora_cache_attention):
// prompts and chunks of prompts, where the kernel is bound by the products and by
// the exponentials between them.  The mathematics (weights that carry the v scales,
// a running maximum that is raised late) is that of cache_attn.cu.
//
// Products run on tcgen05: S = Q K^T into tensor memory, the weights P back into
// tensor memory as fp16, O += P V with P from there.  A CTA holds two tiles of 128
// rows (for heads of up to 128 elements), so that one tile's products run while the
// other's softmax does, and a step of 128 tokens serves both:
//
//   softmax warpgroups (one for each tile, a thread for each row): S from tensor
//     memory, weights back, the running sums; q into shared memory and the tile's
//     results out of tensor memory between items
//   conversion warpgroup: k and v from global memory (two tiles ahead in
//     registers), e4m3 to fp16, into the swizzled layout that the products read
//   one thread issues the products
//
// e4m3 is converted once for 256 rows; as fp16 operands q, k, v keep all their bits.
#include <cfloat>
#include <type_traits>

#include "cache_attn.cuh"
#include "internal.h"

namespace lora {

namespace {

using namespace attn;

constexpr int kN = 128;                       // tokens of a step (and of a unit)
constexpr float kShift = 6.f, kSlack = 8.f;
constexpr int kBlock = 4, kBlocks = 4;        // steps that are planned at once, and such blocks in shared memory
constexpr int kRing = kBlock * kBlocks;

template <int D> struct Many {
  static constexpr int kTiles = D <= 128 ? 2 : 1;
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kBufs = D <= 128 ? 2 : 1;        // of k, and of v
  // warpgroups: softmax of each tile, conversion of k, of v, products and plan; what
  // they do with the registers that the block is launched with
  static constexpr int kThreads = 128 * (kTiles + 3);
  static constexpr int kSoftRegs = kTiles == 2 ? 160 : 184, kConvRegs = kTiles == 2 ? 64 : 128, kOtherRegs = kTiles == 2 ? 32 : 56;
  static constexpr int kTileBytes = kN * D * 2;         // 128 rows of fp16
  static constexpr int kSmem = kTileBytes * (kTiles + 2 * kBufs) + 1024;
  static constexpr int kPieces = D / 16;                // 16 bytes of e4m3 each, of a conversion thread
  static constexpr int kCols = 512;                          // tensor memory: S of each tile, O of each tile
};

// What the other roles need to know of a step, by groups of 16 tokens (which lie
// in one page): where a group's k begins in the cache (negative: nowhere, or not
// visible), and (k scale * c, log2 v scale, 1 / v scale).
struct Step {
  float4 scale[8];
  int64_t at[8];
  int visible;                                // tokens of the step below the last visible one
  uint32_t flags;                             // kFirst, kLast: of its item here; kSecond: so has the second tile rows
  int item;
};
constexpr uint32_t kFirst = 1, kLast = 2, kSecond = 4;
// What the softmax needs to know of an item.  A slot is written again kItems items
// later, when the softmax has long passed all steps of the first one.
constexpr int kItems = 2 * kRing;
struct Item {
  int q0, r0, rows, base;                     // row r: query q0 + r / group, at position base + r / group
  int head, tok, steps;                       // k/v head; first token and number of steps here
  int first_cta, last_cta, which;             // CTAs that share it; which of this CTA's parts it is, -1: it is whole
};

struct ManyShared {
  Shared div;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], o_empty[2], plan_full[kBlocks], plan_empty[kBlocks], done;
  uint32_t tmem;
  int stop;
  int flag[2];
  Step step[kRing];
  Item item[kItems];
};

// The items of a CTA's share, one after another.
struct Cursor {
  unsigned long long w, w1, off;
  int64_t slot;
  int seq, h, ua, nu;
  unsigned long long item0, item1;
  Tile t;
  template <int R>
  __device__ __forceinline__ bool next(const AttnArgs& a) {
    if (w >= w1) return false;
    for (;;) {
      while (seq + 1 < a.B && slot_of<R>(a, seq + 1) <= slot) ++seq;
      tile_of<R, kN>(a, seq, slot, t);
      const unsigned long long slot_units = (unsigned long long)t.units * a.Hk;
      if (off < slot_units) break;
      off -= slot_units;
      ++slot;
    }
    h = (int)(off / t.units);
    ua = (int)(off - (unsigned long long)h * t.units);
    nu = (int)min((unsigned long long)(t.units - ua), w1 - w);
    item0 = w - ua;
    item1 = item0 + t.units;
    w += nu;
    off += nu;
    return true;
  }
};

__device__ __forceinline__ uint32_t halves_lo(uint32_t two) {
  uint32_t h;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(h) : "r"(two));
  return h;
}
__device__ __forceinline__ uint32_t halves_hi(uint32_t two) {
  uint32_t h;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}" : "=r"(h) : "r"(two));
  return h;
}
// {x, y} = {x, y} * s + l, and {x, y} += l
__device__ __forceinline__ void fma2(float& x, float& y, uint64_t s, uint64_t l) {
  asm("{\n .reg .b64 t;\n mov.b64 t, {%0, %1};\n fma.rn.f32x2 t, t, %2, %3;\n mov.b64 {%0, %1}, t;\n}"
      : "+f"(x), "+f"(y) : "l"(s), "l"(l));
}
__device__ __forceinline__ void add2(float& x, float& y, uint64_t l) {
  asm("{\n .reg .b64 t;\n mov.b64 t, {%0, %1};\n add.rn.f32x2 t, t, %2;\n mov.b64 {%0, %1}, t;\n}"
      : "+f"(x), "+f"(y) : "l"(l));
}
__device__ __forceinline__ uint64_t twice(float x) { return ptx::pack2(x, x); }

__device__ __forceinline__ void group_sync(int id) {
  asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}

// Sums of a tile's row that several CTAs share: [which][tile]: [D / 4][128] of
// four values, then [128] of (maximum, sum).
template <int D>
__device__ __forceinline__ float* part_of(const AttnArgs& a, int cta, int which, int tile) {
  return a.part + ((size_t)(2 * cta + which) * Many<D>::kTiles + tile) * 128 * (D + 2);
}

template <int D, typename E>
__global__ void __launch_bounds__(Many<D>::kThreads, 1)
attention_many_kernel(const __grid_constant__ AttnArgs a) {
  using M = Many<D>;
  extern __shared__ uint8_t raw[];
  __shared__ ManyShared sm;
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t q_at = ptx::smem_u32(smem), k_at = q_at + M::kTiles * M::kTileBytes, v_at = k_at + M::kBufs * M::kTileBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = tid >> 7;
  const uint32_t stop = ptx::smem_u32(&sm.stop);

  if (warp == 0) ptx::tmem_alloc(&sm.tmem, M::kCols);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sm.k_full[i], 128);
      ptx::mbar_init(&sm.v_full[i], 128);
      ptx::mbar_init(&sm.k_empty[i], 1);
      ptx::mbar_init(&sm.v_empty[i], 1);
      ptx::mbar_init(&sm.q_full[i], 128);
      ptx::mbar_init(&sm.s_full[i], 1);
      ptx::mbar_init(&sm.p_full[i], 128);
      ptx::mbar_init(&sm.o_full[i], 1);
      ptx::mbar_init(&sm.o_empty[i], 128);
    }
    for (int i = 0; i < kBlocks; ++i) {
      ptx::mbar_init(&sm.plan_full[i], 1);
      ptx::mbar_init(&sm.plan_empty[i], 4 * (M::kTiles + 2));
    }
    ptx::mbar_init(&sm.done, 1);
    sm.stop = 0;
    ptx::fence_mbar_init();
  }
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  ptx::tc_fence_before();
  unsigned long long w0, w1, all;
  int ctas;
  divide<M::kRows, kN>(a, sm.div, 2, w0, w1, all, ctas);   // __syncthreads
  ptx::tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const int steps = (int)(w1 - w0);
  const uint32_t s_col = 0, o_col = M::kTiles * kN;

  if (wg < M::kTiles) {
    // ------------------------------------------------------------ softmax
    ptx::reg_inc<M::kSoftRegs>();
    const int row = tid & 127, tile = wg;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t S = tmem + lanes + s_col + tile * kN, O = tmem + lanes + o_col + tile * D;
    float cs = 0.f;
    int st = 0, n_s = 0, n_items = 0;
    auto planned = [&]() {
      ptx::mbar_wait_asm(ptx::smem_u32(&sm.plan_full[st / kBlock % kBlocks]), (st / kRing) & 1, stop);
    };
    auto pass = [&]() {                       // step st is done with
      if (st % kBlock == kBlock - 1 && lane == 0) ptx::mbar_arrive(&sm.plan_empty[st / kBlock % kBlocks]);
      ++st;
    };
    // the next item in which this tile has rows, or -1
    auto seek = [&]() -> int {
      while (st < steps) {
        planned();
        const int item = sm.step[st % kRing].item;
        if (sm.item[item].rows > 128 * tile) return item;
        for (int n = sm.item[item].steps; n > 0; --n) {
          planned();
          pass();
        }
      }
      return -1;
    };
    // where this thread's row of an item lies in q and y
    auto find = [&](const Item& it, int& line, int& col) -> bool {
      const int r = it.r0 + 128 * tile + row;
      const bool in = 128 * tile + row < it.rows;
      const int i = in ? r / a.group : 0;
      line = it.q0 + i;
      col = (it.head * a.group + (in ? r - i * a.group : 0)) * a.dim;
      return in;
    };
    // its q into shared memory
    auto load_q = [&](int item) {
      int line, col;
      const bool in = find(sm.item[item], line, col);
      const E* src = static_cast<const E*>(a.q) + (int64_t)line * a.ldq + col;
      // the row's largest element to 2^7 .. 2^8 by a power of two; read twice, 64 elements
      // at a time, rather than held
      float top = 0.f;
#pragma unroll 1
      for (int j = 0; j < D / 64; ++j) {
        uint4 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = in && 64 * j + 8 * e < a.dim ? ldg_nc(src + 64 * j + 8 * e) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float f[8];
          Elem<E>::to_f32(v[e], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
        }
      }
      const int k = min(max(7 + 127 - (int)(__float_as_uint(top) >> 23), -120), 120);
      const float up = __uint_as_float((uint32_t)(127 + k) << 23);
      cs = __uint_as_float((uint32_t)(127 - k) << 23);
      uint8_t* dst = smem + (size_t)tile * M::kTileBytes + row * 128;
#pragma unroll 1
      for (int j = 0; j < D / 64; ++j) {
        uint4 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = in && 64 * j + 8 * e < a.dim ? ldg_nc(src + 64 * j + 8 * e) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float f[8];
          Elem<E>::to_f32(v[e], f);
          uint4 w;
          w.x = Elem<__half>::pack2(f[0] * up, f[1] * up);
          w.y = Elem<__half>::pack2(f[2] * up, f[3] * up);
          w.z = Elem<__half>::pack2(f[4] * up, f[5] * up);
          w.w = Elem<__half>::pack2(f[6] * up, f[7] * up);
          *reinterpret_cast<uint4*>(dst + j * (kN * 128) + (e ^ (row & 7)) * 16) = w;
        }
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(&sm.q_full[tile]);
    };
    int item = seek();
    if (item >= 0) load_q(item);
    while (item >= 0) {
      int line, col, pos, from, pos_low, pos_high, tok, n_steps, first_cta, last_cta, which;
      bool in;
      {
        const Item& it = sm.item[item];
        in = find(it, line, col);
        pos = in ? it.base + (line - it.q0) : -1;
        from = a.window > 0 ? pos - a.window : -1;           // visible: from < token <= pos
        pos_low = it.base + (it.r0 + 128 * tile) / a.group;
        pos_high = it.base + (it.r0 + min(it.rows, 128 * tile + 128) - 1) / a.group;
        tok = it.tok;
        n_steps = it.steps;
        first_cta = it.first_cta;
        last_cta = it.last_cta;
        which = it.which;
      }
      float m = -FLT_MAX, l = 0.f;
      for (int i = 0; i < n_steps; ++i, tok += kN) {
        planned();
        const Step& step = sm.step[st % kRing];
        ptx::mbar_wait_asm(ptx::smem_u32(&sm.s_full[tile]), n_s & 1, stop);
        ++n_s;
        ptx::tc_fence_after();
        float x[kN];
#pragma unroll
        for (int j = 0; j < kN / 32; ++j) ptx::tc_ld32(S + 32 * j, reinterpret_cast<uint32_t*>(x) + 32 * j);
#pragma unroll
        for (int j = 0; j < kN / 32; ++j) ptx::tc_wait_ld32(reinterpret_cast<uint32_t*>(x) + 32 * j);
        if (tok + kN - 1 > pos_low || (a.window > 0 && tok <= pos_high - a.window)) {
          const int hi = pos - tok, lo = from - tok;                   // visible: lo < j <= hi
#pragma unroll
          for (int j = 0; j < kN; ++j)
            if (j > hi || j <= lo) x[j] = -INFINITY;
        }
        // factors are positive: the largest score of 16 tokens gives their largest t
        float tops[8];
#pragma unroll
        for (int gq = 0; gq < 8; ++gq) {
          const float* y = x + 16 * gq;
          float t0 = fmaxf(y[0], fmaxf(y[1], y[2])), t1 = fmaxf(y[3], fmaxf(y[4], y[5]));
          t0 = fmaxf(t0, fmaxf(y[6], y[7]));
          t1 = fmaxf(t1, fmaxf(y[8], y[9]));
          t0 = fmaxf(t0, fmaxf(y[10], y[11]));
          t1 = fmaxf(t1, fmaxf(y[12], y[13]));
          t0 = fmaxf(t0, fmaxf(y[14], y[15]));
          tops[gq] = fmaf(fmaxf(t0, t1), step.scale[gq].x * cs, step.scale[gq].y);
        }
        const float top = fmaxf(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])),
                                fmaxf(fmaxf(tops[4], tops[5]), fmaxf(tops[6], tops[7])));
        // the products of the step before are complete: S came after them
        if (__any_sync(~0u, top > m + kSlack)) {
          const float n = fmaxf(m, top), f = exp2_fast(m - n);
          m = n;
          l *= f;
          if (i > 0) {
#pragma unroll 1
            for (int j = 0; j < D; j += 16) {
              uint32_t o[16];
              ptx::tc_ld16(O + j, o);
              ptx::tc_wait_ld16(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              ptx::tc_st16(O + j, o);
            }
          }
        }
        const float off = kShift - m;
#pragma unroll
        for (int gq = 0; gq < 8; gq += 2) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float* y = x + 16 * (gq + e);
            const float4 sc = step.scale[gq + e];
            const uint64_t s2 = twice(sc.x * cs), l2 = twice(sc.y + off);
#pragma unroll
            for (int j = 0; j < 16; j += 2) fma2(y[j], y[j + 1], s2, l2);
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              y[j] = exp2_fast(y[j]);
              y[j + 1] = exp2_fast(y[j + 1]);
              add2(s0, s1, ptx::pack2(y[j], y[j + 1]));
              p[8 * e + j / 2] = Elem<__half>::pack2(y[j], y[j + 1]);
            }
            l = fmaf(s0 + s1, sc.z, l);
          }
          ptx::tc_st16(S + 8 * gq, p);
        }
        ptx::tc_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&sm.p_full[tile]);
        pass();
      }
      // q of the next item, while this one's last products run
      item = seek();
      if (item >= 0) load_q(item);
      ptx::mbar_wait_asm(ptx::smem_u32(&sm.o_full[tile]), n_items & 1, stop);
      ++n_items;
      ptx::tc_fence_after();
      E* out = static_cast<E*>(a.y) + (int64_t)line * a.ldy + col;
      if (which < 0) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int j = 0; j < D; j += 32) {
          float o[32];
          ptx::tc_ld32(O + j, reinterpret_cast<uint32_t*>(o));
          ptx::tc_wait_ld32(reinterpret_cast<uint32_t*>(o));
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            if (in && j + e < a.dim) {
              uint4 v;
              v.x = Elem<E>::pack2(o[e] * inv, o[e + 1] * inv);
              v.y = Elem<E>::pack2(o[e + 2] * inv, o[e + 3] * inv);
              v.z = Elem<E>::pack2(o[e + 4] * inv, o[e + 5] * inv);
              v.w = Elem<E>::pack2(o[e + 6] * inv, o[e + 7] * inv);
              *reinterpret_cast<uint4*>(out + j + e) = v;
            }
          }
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(&sm.o_empty[tile]);
      } else {
        float* part = part_of<D>(a, blockIdx.x, which, tile);
#pragma unroll
        for (int j = 0; j < D; j += 32) {
          float o[32];
          ptx::tc_ld32(O + j, reinterpret_cast<uint32_t*>(o));
          ptx::tc_wait_ld32(reinterpret_cast<uint32_t*>(o));
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            __stcg(reinterpret_cast<float4*>(part) + (size_t)((j + e) / 4) * 128 + row,
                   make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]));
        }
        __stcg(reinterpret_cast<float2*>(part + 128 * D) + row, make_float2(m, l));
        ptx::tc_fence_before();
        ptx::mbar_arrive(&sm.o_empty[tile]);
        __threadfence();
        group_sync(1 + tile);
        if (row == 0) {
          int* join = a.join + 2 * first_cta + tile;
          sm.flag[tile] = atomicAdd(join, 1) == last_cta - first_cta;
          if (sm.flag[tile]) *join = 0;                   // as the next call finds it
        }
        group_sync(1 + tile);
        if (sm.flag[tile]) {
          __threadfence();
          float top = -FLT_MAX, sum = 0.f;
          for (int k = first_cta; k <= last_cta; ++k) {
            const float2 ms = __ldcg(reinterpret_cast<const float2*>(part_of<D>(a, k, k == first_cta ? 1 : 0, tile) + 128 * D) + row);
            const float up = fmaxf(top, ms.x);
            sum = sum * exp2_fast(top - up) + ms.y * exp2_fast(ms.x - up);
            top = up;
          }
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          for (int j = 0; j < a.dim; j += 16) {
            float o[16] = {};
            for (int k = first_cta; k <= last_cta; ++k) {
              const float* pk = part_of<D>(a, k, k == first_cta ? 1 : 0, tile);
              const float f = exp2_fast(__ldcg(reinterpret_cast<const float2*>(pk + 128 * D) + row).x - top) * inv;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(pk) + (size_t)(j / 4 + e) * 128 + row);
                o[4 * e] = fmaf(v.x, f, o[4 * e]);
                o[4 * e + 1] = fmaf(v.y, f, o[4 * e + 1]);
                o[4 * e + 2] = fmaf(v.z, f, o[4 * e + 2]);
                o[4 * e + 3] = fmaf(v.w, f, o[4 * e + 3]);
              }
            }
            if (in) {
#pragma unroll
              for (int e = 0; e < 16; e += 8) {
                uint4 v;
                v.x = Elem<E>::pack2(o[e], o[e + 1]);
                v.y = Elem<E>::pack2(o[e + 2], o[e + 3]);
                v.z = Elem<E>::pack2(o[e + 4], o[e + 5]);
                v.w = Elem<E>::pack2(o[e + 6], o[e + 7]);
                *reinterpret_cast<uint4*>(out + j + e) = v;
              }
            }
          }
        }
      }
    }
  } else if (wg < M::kTiles + 2) {
    // ------------------------------------------------------------ conversion
    ptx::reg_dec<M::kConvRegs>();
    const int ct = tid & 127;
    const bool is_v = wg == M::kTiles + 1;
    const int64_t side = is_v ? ((int64_t)a.Hk * a.dim) << a.page_log : 0;
    const uint8_t* const base = a.cache + side;
    const uint32_t tiles_at = is_v ? v_at : k_at;
    uint64_t *const full = is_v ? sm.v_full : sm.k_full, *const empty = is_v ? sm.v_empty : sm.k_empty;
    uint4 r[M::kPieces];
    // A thread's pieces of 16 bytes: four lanes take 64 bytes of a row, the next four
    // of the row behind it, so that the halves they store hit different banks.
    auto place = [&](int k, int& row, int& e) {
      const int i = ct + 128 * k, rest = i >> 3;
      e = 64 * (rest % (D / 64)) + 16 * (i & 3);
      row = 2 * (rest / (D / 64)) + ((i >> 2) & 1);
    };
    auto load = [&](int st) {
      ptx::mbar_wait_asm(ptx::smem_u32(&sm.plan_full[st / kBlock % kBlocks]), (st / kRing) & 1, stop);
      const Step& step = sm.step[st % kRing];
      const int visible = is_v ? step.visible : kN;         // v behind the last visible token may be
#pragma unroll                                              // anything: zeros in its place
      for (int k = 0; k < M::kPieces; ++k) {
        int row, e;
        place(k, row, e);
        const int64_t at = step.at[row >> 4];
        r[k] = make_uint4(0, 0, 0, 0);
        if (at >= 0 && e < a.dim && row < visible) r[k] = ldg_stream(base + at + (row & 15) * a.dim + e);
      }
      // this step's entries are not looked at again
      if (st % kBlock == kBlock - 1) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.plan_empty[st / kBlock % kBlocks]);
      }
    };
    if (steps > 0) load(0);
    for (int st = 0; st < steps; ++st) {
      const int buf = st % M::kBufs, use = st / M::kBufs;
      if (use > 0) ptx::mbar_wait_asm(ptx::smem_u32(&empty[buf]), (use - 1) & 1, stop);
      const uint32_t dst = tiles_at + buf * M::kTileBytes;
#pragma unroll
      for (int k = 0; k < M::kPieces; ++k) {
        int row, e;
        place(k, row, e);
        const uint32_t at = dst + (e / 64) * (kN * 128) + row * 128, c0 = ((e & 63) >> 3) ^ (row & 7);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + (c0 << 4)), "r"(halves_lo(r[k].x)), "r"(halves_hi(r[k].x)),
                     "r"(halves_lo(r[k].y)), "r"(halves_hi(r[k].y)) : "memory");
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + ((c0 ^ 1) << 4)), "r"(halves_lo(r[k].z)), "r"(halves_hi(r[k].z)),
                     "r"(halves_lo(r[k].w)), "r"(halves_hi(r[k].w)) : "memory");
      }
      if (st + 1 < steps) load(st + 1);
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(&full[buf]);
    }
  } else {
    // ------------------------------------------------------------ products
    ptx::reg_dec<M::kOtherRegs>();
    if (warp == 4 * (M::kTiles + 2)) {
      // Whatever an instruction's operands or the loop depend on goes through a warp
      // reduction, whose result the compiler knows to be the same in all lanes: it
      // keeps it in uniform registers, as these instructions want it (moving it there
      // for each one made an issue of 16 take 1050 cycles).
      const bool one = ptx::elect_one();
      const uint32_t tm = __reduce_or_sync(~0u, tmem);
      const int n_steps = (int)__reduce_max_sync(~0u, (unsigned)steps);
      constexpr uint32_t id_s = ptx::umma_idesc_f16(false, 128, kN);
      constexpr uint32_t id_o = ptx::umma_idesc_f16(false, 128, D) | ptx::kIdescNMajorB;
      const uint64_t q_desc = ptx::umma_desc_kmajor(q_at, 128), k_desc = ptx::umma_desc_kmajor(k_at, 128);
      const uint64_t v_desc = ptx::umma_desc_nmajor(v_at, kN * 128);
      constexpr uint64_t kTile16 = M::kTileBytes >> 4;
      uint32_t n_q0 = 0, n_q1 = 0, n_p0 = 0, n_p1 = 0, n_o0 = 0, n_o1 = 0;
      auto flags = [&](int st) -> uint32_t {
        ptx::mbar_wait_asm(ptx::smem_u32(&sm.k_full[st % M::kBufs]), (st / M::kBufs) & 1, stop);
        return __reduce_or_sync(~0u, sm.step[st % kRing].flags);
      };
      auto scores = [&](auto tile, int st, uint32_t f) {
        constexpr int t = decltype(tile)::value;
        uint32_t& n_q = t ? n_q1 : n_q0;
        if (f & kFirst) {
          ptx::mbar_wait_asm(ptx::smem_u32(&sm.q_full[t]), n_q & 1, stop);
          ++n_q;
        }
        ptx::tc_fence_after();
        if (one) {
          const uint64_t k = k_desc + (uint32_t)(st % M::kBufs) * kTile16;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const uint32_t off = ((j / 4) * (kN * 128) + (j % 4) * 32) >> 4;
            ptx::tc_mma_f16(tm + s_col + t * kN, q_desc + t * kTile16 + off, k + off, id_s, j > 0);
          }
          ptx::tc_commit(&sm.s_full[t]);
        }
        __syncwarp();
      };
      auto sums = [&](auto tile, int st, uint32_t f) {
        constexpr int t = decltype(tile)::value;
        uint32_t &n_p = t ? n_p1 : n_p0, &n_o = t ? n_o1 : n_o0;
        ptx::mbar_wait_asm(ptx::smem_u32(&sm.p_full[t]), n_p & 1, stop);
        ++n_p;
        if (f & kFirst) {
          if (n_o > 0) ptx::mbar_wait_asm(ptx::smem_u32(&sm.o_empty[t]), (n_o - 1) & 1, stop);
          ++n_o;
        }
        ptx::tc_fence_after();
        if (one) {
          const uint64_t v = v_desc + (uint32_t)(st % M::kBufs) * kTile16;
#pragma unroll
          for (int j = 0; j < kN / 16; ++j)
            ptx::tc_mma_f16_ts(tm + o_col + t * D, tm + s_col + t * kN + 8 * j, v + j * (2048 >> 4), id_o, j > 0 || !(f & kFirst));
          if (f & kLast) ptx::tc_commit(&sm.o_full[t]);
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t* bar) {
        if (one) ptx::tc_commit(bar);
        __syncwarp();
      };
      constexpr std::integral_constant<int, 0> t0{};
      constexpr std::integral_constant<int, M::kTiles - 1> t1{};
      uint32_t now = 0;
      if (n_steps > 0) {
        now = flags(0);
        scores(t0, 0, now);
        if (now & kSecond) scores(t1, 0, now);
        commit(&sm.k_empty[0]);
      }
      for (int st = 0; st < n_steps; ++st) {
        const int buf = st % M::kBufs;
        const bool go_on = st + 1 < n_steps;
        const uint32_t then = go_on ? flags(st + 1) : 0;
        ptx::mbar_wait_asm(ptx::smem_u32(&sm.v_full[buf]), (st / M::kBufs) & 1, stop);
        if (!(now & kLast)) {
          sums(t0, st, now);
          scores(t0, st + 1, then);
          if (now & kSecond) {
            sums(t1, st, now);
            scores(t1, st + 1, then);
          }
          commit(&sm.v_empty[buf]);
          commit(&sm.k_empty[(st + 1) % M::kBufs]);
        } else {
          sums(t0, st, now);
          if (now & kSecond) sums(t1, st, now);
          commit(&sm.v_empty[buf]);
          if (go_on) {
            scores(t0, st + 1, then);
            if (then & kSecond) scores(t1, st + 1, then);
            commit(&sm.k_empty[(st + 1) % M::kBufs]);
          }
        }
        now = then;
      }
      // nothing is in flight when tensor memory goes back
      commit(&sm.done);
      ptx::mbar_wait_asm(ptx::smem_u32(&sm.done), 0, stop);
    } else if (warp == 4 * (M::kTiles + 2) + 1) {
      // ---------------------------------------------------------- plan
      // four steps at a time, eight lanes for the groups of each
      const int64_t head_bytes = (int64_t)a.dim << a.page_log;
      Cursor cur;
      cur.w = w0;
      cur.w1 = w1;
      cur.off = sm.div.off;
      cur.slot = sm.div.slot;
      cur.seq = sm.div.seq;
      cur.nu = 0;
      int u = 0, item = -1;
      for (int st = 0; st < steps; st += kBlock) {
        const int block = st / kBlock % kBlocks, use = st / kRing;
        if (use > 0) ptx::mbar_wait_asm(ptx::smem_u32(&sm.plan_empty[block]), (use - 1) & 1, stop);
        int64_t entry = -1;                   // of the table, for this lane's group
        int at = 0, head = 0;
        for (int i = 0; i < kBlock && st + i < steps; ++i, ++u) {
          if (u == cur.nu) {
            cur.next<M::kRows>(a);
            u = 0;
            item = (item + 1) % kItems;
            if (lane == 0) {
              Item& it = sm.item[item];
              it.q0 = cur.t.q0;
              it.r0 = cur.t.r0;
              it.rows = cur.t.rows;
              it.base = cur.t.len - cur.t.n;
              it.head = cur.h;
              it.tok = (cur.t.u0 + cur.ua) * kN;
              it.steps = cur.nu;
              it.first_cta = owner(cur.item0, all, ctas);
              it.last_cta = owner(cur.item1 - 1, all, ctas);
              // begun here and not ended: this CTA's last
              it.which = cur.nu == cur.t.units ? -1 : (cur.ua == 0 ? 1 : 0);
            }
          }
          const int tok = (cur.t.u0 + cur.ua + u) * kN;
          if (lane >> 3 == i) {
            at = tok + 16 * (lane & 7);
            head = cur.h;
            if (at < cur.t.hi && at + 16 > cur.t.lo) entry = (int64_t)cur.t.b * a.M + (at >> a.page_log);
          }
          if (lane == 0) {
            Step& step = sm.step[(st + i) % kRing];
            step.visible = cur.t.hi - tok;
            step.flags = (u == 0 ? kFirst : 0) | (u == cur.nu - 1 ? kLast : 0) | (cur.t.rows > 128 ? kSecond : 0);
            step.item = item;
          }
        }
        int64_t where = -1;
        float4 scale = make_float4(1.f, -INFINITY, 0.f, 0.f);         // weights of 0, for scores of -inf too
        if (entry >= 0) {
          const int pid = a.tables[entry];
          if (pid < 0 || pid >= a.P) {
            atomicAdd(a.bad, 1);
          } else {
            const int64_t page = (int64_t)pid * 2 * a.Hk + head;
            const float ks = a.scale[page], vs = a.scale[page + a.Hk];
            scale = make_float4(ks * a.c, log2f(vs), 1.f / vs, 0.f);
            where = page * head_bytes + (int64_t)(at & ((1 << a.page_log) - 1)) * a.dim;
          }
        }
        if (st + (lane >> 3) < steps) {
          Step& step = sm.step[(st + (lane >> 3)) % kRing];
          step.scale[lane & 7] = scale;
          step.at[lane & 7] = where;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.plan_full[block]);
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 0) {
    ptx::tmem_relinquish();
    ptx::tmem_dealloc(tmem, M::kCols);
  }
  if (tid == 0 && sm.stop) atomicAdd(a.bad + 1, 1);         // a wait gave up
}

template <int D, typename E>
cudaError_t many_launch(const AttnArgs& a, cudaStream_t st) {
  using M = Many<D>;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(attention_many_kernel<D, E>, cudaFuncAttributeMaxDynamicSharedMemorySize, M::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(148, 1, 1);
  cfg.blockDim = dim3(M::kThreads, 1, 1);
  cfg.dynamicSmemBytes = M::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return counted_launch(cudaLaunchKernelEx(&cfg, attention_many_kernel<D, E>, a));
}

template <typename E>
cudaError_t many_width(const AttnArgs& a, cudaStream_t st) {
  if (a.dim <= 64) return many_launch<64, E>(a, st);
  if (a.dim <= 128) return many_launch<128, E>(a, st);
  if (a.dim <= 192) return many_launch<192, E>(a, st);
  return many_launch<256, E>(a, st);
}

}  // namespace

cudaError_t launch_attention_many(lora_dtype dt, const AttnArgs& a, cudaStream_t st) {
  return dt == LORA_BF16 ? many_width<__nv_bfloat16>(a, st) : many_width<__half>(a, st);
}

}  // namespace lora
