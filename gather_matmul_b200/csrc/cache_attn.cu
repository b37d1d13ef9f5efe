// Attention of few queries over the paged 8-bit cache (lora_cache_attention):
// single tokens, where every k and v byte is used by one sequence's rows only and
// the kernel is bound by reading them.
//
//   s_rj = c q_r . k_j,   o_r = sum_j 2^(s_rj - m) v_j / sum_j 2^(s_rj - m)
//
// with c = softmax scale * log2 e.  A page's v scale enters as its logarithm: with
// t = s + log2 v_scale the numerators' weights 2^(t - m) are at most 2^kShift, so
// that they round to fp16 as they are (11 bits), whatever the scales, and the
// denominators' terms are 2^(t - m) / v_scale in fp32.  m is a running maximum of t
// that is only raised when a term would pass 2^(kShift + kSlack).
//
// Products run on mma.sync with the tokens (k) and the head's elements (v) on the
// wide side, M = 16, and the rows on the narrow one, N = 8: a tile of 8 rows costs
// half of what it would cost as M = 16.  e4m3 becomes fp16 exactly, in registers.
// The order of the products' inner indices is free, so every thread loads 16-byte
// pieces and needs no others: no transposes, no barriers, no shared memory before a
// warp's sums are done.  The next group of tokens is loaded into the registers that the
// products have just read.  q's rows are brought to fp16 by powers of two (their largest
// elements to 2^7 .. 2^8), which costs less than the rounding of the sums.
//
// 128 sequences of 4096 tokens, 32 heads on 8 of 128: 200 us, 5.4 TB/s, 0.82 of the
// measured copy rate; 512 ragged ones of up to 8192: 231 us, 0.74 (through stages in
// shared memory, by cp.async: 407 before the idle units below, 352 in registers).  Between
// two items of a CTA (about seven of the ragged batch) loads stop, until the warps' sums
// have met and the next item's pages are known.  9 to 16 rows spill registers (280 bytes of
// a thread at heads of 128, 640 at 256) and are not bound by memory: 128 heads on 8 over
// the same 128 sequences 292 us, 0.56; over 64, heads of 256, 128 on 8 410 us, 0.40, where
// 64 on 8 take 217, 0.75.
#include <cfloat>

#include "cache_attn.cuh"
#include "internal.h"

namespace lora {

namespace {

using namespace attn;

constexpr int kFThreads = 128, kFWarps = 4;
constexpr int kFUnit = 64;                  // tokens of a unit: 16 for each warp
// What an item costs beside its tokens, in units: CTAs of many short sequences get
// fewer.  The ragged batch above: 0 units 352 us, 1 264, 2 231, 4 250, 8 264.
constexpr int kIdle = 2;
constexpr float kShift = 6.f, kSlack = 8.f;

// Four CTAs share an SM where their registers do.  A second group in flight for each
// warp leaves room for three: 367 us against 352 (the ragged batch, in the form of then).
template <int D, int NT> constexpr int few_ctas() { return D <= 128 ? (NT == 1 ? 4 : 3) : 2; }

// 16 or 8 bytes, or zeros; no branch, so that loads follow one another
__device__ __forceinline__ uint4 load16(const void* p, bool in) {
  uint4 v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n mov.b32 %0, 0;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n mov.b32 %3, 0;\n"
      " @p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w) : "l"(p), "r"((uint32_t)in));
  return v;
}
__device__ __forceinline__ uint2 load8(const void* p, bool in) {
  uint2 v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %3, 0;\n mov.b32 %0, 0;\n mov.b32 %1, 0;\n"
      " @p ld.global.nc.v2.u32 {%0, %1}, [%2];\n}"
      : "=&r"(v.x), "=&r"(v.y) : "l"(p), "r"((uint32_t)in));
  return v;
}
__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float inverse_fast(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two e4m3 codes (low byte first) to two halves
__device__ __forceinline__ uint32_t halves(uint32_t two) {
  uint32_t h;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(h) : "r"(two));
  return h;
}
__device__ __forceinline__ uint32_t halves_hi(uint32_t two) {
  uint32_t h;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}" : "=r"(h) : "r"(two));
  return h;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Partial sums of a row tile: [R][D] weighted values, then [R][2] maximum and sum.
template <int D, int NT>
__device__ __forceinline__ float* part_of(const AttnArgs& a, int cta, int which) {
  return a.part + (size_t)(2 * cta + which) * (8 * NT) * (D + 2);
}

// dims d, d + 1 of a row of y
template <typename E>
__device__ __forceinline__ void put_row(const AttnArgs& a, const Tile& t, int h, int row, int d, float x, float y) {
  const int r = t.r0 + row, i = r / a.group;
  E* out = static_cast<E*>(a.y) + (int64_t)(t.q0 + i) * a.ldy + ((int64_t)h * a.group + (r - i * a.group)) * a.dim + d;
  *reinterpret_cast<uint32_t*>(out) = Elem<E>::pack2(x, y);
}

template <int D, int NT, typename E>
__global__ void __launch_bounds__(kFThreads, few_ctas<D, NT>())
attention_few_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int R = 8 * NT;
  constexpr int KT = D / 64;               // 16-byte pieces of k of a token that a thread holds (of 2 tokens)
  constexpr int MT = D / 16;               // m-tiles of the v product, and words of k of a token
  constexpr int VB = D / 8;                // bytes of v of one token (4 tokens), in pieces of PW
  constexpr int PW = VB % 16 == 0 ? 16 : 8;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  __shared__ float stat[kFWarps][R][2];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;

  unsigned long long w0, w1, all;
  int ctas;
  divide<R, kFUnit, kIdle>(a, sh, 2, w0, w1, all, ctas);
  if (w0 >= w1) return;
  int64_t slot = sh.slot;
  int seq = sh.seq;
  unsigned long long off = sh.off, w = w0;
  const int page = 1 << a.page_log;
  const int64_t head_bytes = (int64_t)a.dim << a.page_log;

  while (w < w1) {
    Tile t;
    while (seq + 1 < a.B && slot_of<R>(a, seq + 1) <= slot) ++seq;
    tile_of<R, kFUnit, kIdle>(a, seq, slot, t);
    const unsigned long long slot_units = (unsigned long long)t.units * a.Hk;
    if (off >= slot_units) {                // this slot is done (or holds no rows)
      off -= slot_units;
      ++slot;
      continue;
    }
    const int h = (int)(off / t.units), from = (int)(off - (unsigned long long)h * t.units);
    const int share = (int)min((unsigned long long)(t.units - from), w1 - w);
    // of the units that have tokens
    const int ua = max(from - kIdle, 0), nu = from + share - kIdle - ua;
    const unsigned long long item0 = w - from + kIdle, item1 = w - from + t.units;
    const bool begins = from <= kIdle;
    w += share;
    off += share;
    if (nu <= 0) continue;

    // ---- copies: iteration it of this warp takes tokens tok0 + it * kFUnit .. + 16
    const int tok0 = (t.u0 + ua) * kFUnit + warp * 16;
    const uint8_t* base = a.cache + (int64_t)h * head_bytes;
    const int64_t v_off = (int64_t)a.Hk * head_bytes, page_bytes = 2 * v_off;
    int pids = -1;
    auto fetch_pids = [&](int it) {
      const int tok = tok0 + (it + lane) * kFUnit;
      pids = -1;
      if (it + lane < nu && tok < t.hi && tok + 16 > t.lo) {
        pids = a.tables[(int64_t)t.b * a.M + (tok >> a.page_log)];
        if (pids < 0 || pids >= a.P) {
          atomicAdd(a.bad, 1);
          pids = -1;
        }
      }
    };
    // A group in registers: k of tokens g and g + 8, 16 of each 64 elements from 16 c on; v
    // of tokens 2c, 2c + 1, 2c + 8, 2c + 9, PW of each 8 PW elements from PW g on (a load's
    // neighbouring lanes have neighbouring pieces); the scales.
    struct Group {
      uint4 k[2 * KT];
      uint32_t v[4][VB / 4];
      float ks, vs;
      const uint8_t* at;                    // its k in the cache, or null
    };
    const int k_lane = g * a.dim + 16 * c, v_lane = 2 * c * a.dim + PW * g;
    auto load_k = [&](Group& r, int it) {
      if ((it & 31) == 0) fetch_pids(it);
      const int pid = __shfl_sync(~0u, pids, it & 31);
      const bool in = it < nu && pid >= 0;
      const int tok = tok0 + it * kFUnit;
      r.at = in ? base + (int64_t)pid * page_bytes + (int64_t)(tok & (page - 1)) * a.dim : nullptr;
#pragma unroll
      for (int j = 0; j < KT; ++j) {
        const bool ok = in && 64 * j + 16 * c < a.dim;
        r.k[j] = load16(r.at + k_lane + 64 * j, ok);
        r.k[KT + j] = load16(r.at + k_lane + 8 * a.dim + 64 * j, ok);
      }
      r.ks = r.vs = 1.f;
      if (in) {
        const float* sp = a.scale + (int64_t)pid * 2 * a.Hk + h;
        r.ks = __ldg(sp);
        r.vs = __ldg(sp + a.Hk);
      }
    };
    auto load_v = [&](Group& r, int it) {
      const uint8_t* v = r.at + v_off + v_lane;
      const int left = r.at ? t.hi - (tok0 + it * kFUnit) - 2 * c : 0;   // what lies behind may be anything: zeros in its place
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tk = (i & 1) + 8 * (i >> 1);
        if constexpr (VB % 16 == 0) {
#pragma unroll
          for (int j = 0; j < VB / 16; ++j) {
            const uint4 x = load16(v + tk * a.dim + 128 * j, tk < left && 128 * j + 16 * g < a.dim);
            r.v[i][4 * j] = x.x, r.v[i][4 * j + 1] = x.y, r.v[i][4 * j + 2] = x.z, r.v[i][4 * j + 3] = x.w;
          }
        } else {
#pragma unroll
          for (int j = 0; j < VB / 8; ++j) {
            const uint2 x = load8(v + tk * a.dim + 64 * j, tk < left && 64 * j + 8 * g < a.dim);
            r.v[i][2 * j] = x.x, r.v[i][2 * j + 1] = x.y;
          }
        }
      }
    };
    Group r;
    load_k(r, 0);
    load_v(r, 0);

    // ---- q: row 8 nt + g of the tile, the elements that this thread has of k
    uint32_t q[NT][MT][2];
    float cs[NT][2];                        // c * the power of two, of rows 2c and 2c + 1
    int pos[NT][2];                         // their positions; -1: no such row
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = 8 * nt + g, r = t.r0 + row, i = r / a.group;
      const bool in = row < t.rows;
      const E* src = static_cast<const E*>(a.q) + (int64_t)(t.q0 + (in ? i : 0)) * a.ldq +
                     ((int64_t)h * a.group + (in ? r - i * a.group : 0)) * a.dim + 16 * c;
      uint4 v[2 * KT];
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < 2 * KT; ++j) {
        v[j] = make_uint4(0, 0, 0, 0);
        const int e = 64 * (j / 2) + 8 * (j & 1);
        if (in && 16 * c + e < a.dim) v[j] = ldg_nc(src + e);
        float f[8];
        Elem<E>::to_f32(v[j], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
      }
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
      // 2^k brings the largest element to 2^7 .. 2^8
      const int k = min(max(7 + 127 - (int)(__float_as_uint(top) >> 23), -120), 120);
      const float up = __uint_as_float((uint32_t)(127 + k) << 23), down = __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
      for (int j = 0; j < 2 * KT; ++j) {
        float f[8];
        Elem<E>::to_f32(v[j], f);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          q[nt][2 * j + e / 2][e & 1] = Elem<__half>::pack2(f[2 * e] * up, f[2 * e + 1] * up);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row2 = 8 * nt + 2 * c + e;
        cs[nt][e] = a.c * __shfl_sync(~0u, down, (2 * c + e) * 4);
        pos[nt][e] = row2 < t.rows ? position(a, t.len - t.n, t.r0 + row2) : -1;
      }
    }
    const int pos_low = position(a, t.len - t.n, t.r0), pos_high = position(a, t.len - t.n, t.r0 + t.rows - 1);

    float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      m[nt][0] = m[nt][1] = -FLT_MAX;
      l[nt][0] = l[nt][1] = 0.f;
    }

    // group it, whose registers then take the next one
    auto group = [&](int it) {
      const int tok = tok0 + it * kFUnit;
      const bool have = r.at != nullptr;
      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
      if (have) {
#pragma unroll
        for (int j = 0; j < KT; ++j) {
          const uint32_t wl[4] = {r.k[j].x, r.k[j].y, r.k[j].z, r.k[j].w};
          const uint32_t wh[4] = {r.k[KT + j].x, r.k[KT + j].y, r.k[KT + j].z, r.k[KT + j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t af[4] = {halves(wl[i]), halves(wh[i]), halves_hi(wl[i]), halves_hi(wh[i])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              ptx::mma_16816<false>(sc[nt], af, q[nt][4 * j + i][0], q[nt][4 * j + i][1]);
          }
        }
      }
      const float ks = r.ks, lv = log2_fast(r.vs);
      float inv = inverse_fast(r.vs);
      load_k(r, it + 1);                 // (r.at is the next group's from here on)
      if (!have) {
        load_v(r, it + 1);
        return;
      }
      const bool edge = tok + 15 > pos_low || (a.window > 0 && tok <= pos_high - a.window);
      // A NaN scale spoils the rows that see its page and no others: their weights of 0 meet
      // numbers, in the denominator and in the product.  (On every group, edge or not, it
      // cost the decode batch 2 %.)
      if (edge && lv != lv) {
        inv = 1.f;
#pragma unroll
        for (int j = 0; j < VB / 4; ++j) r.v[0][j] = r.v[1][j] = r.v[2][j] = r.v[3][j] = 0;
      }
      uint32_t p[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = fmaf(sc[nt][i], ks * cs[nt][i & 1], lv);
        if (edge) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = tok + g + 8 * (i >> 1), at = pos[nt][i & 1];
            if (j > at || (a.window > 0 && j <= at - a.window)) x[i] = -INFINITY;
          }
        }
        const float t0 = fmaxf(x[0], x[2]), t1 = fmaxf(x[1], x[3]);
        if (__any_sync(~0u, t0 > m[nt][0] + kSlack || t1 > m[nt][1] + kSlack)) {
          float n0 = fmaxf(m[nt][0], t0), n1 = fmaxf(m[nt][1], t1);
#pragma unroll
          for (int d = 4; d < 32; d *= 2) {
            n0 = fmaxf(n0, __shfl_xor_sync(~0u, n0, d));
            n1 = fmaxf(n1, __shfl_xor_sync(~0u, n1, d));
          }
          const float f0 = exp2_fast(m[nt][0] - n0), f1 = exp2_fast(m[nt][1] - n1);
          m[nt][0] = n0;
          m[nt][1] = n1;
          l[nt][0] *= f0;
          l[nt][1] *= f1;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            o[nt][i][0] *= f0;
            o[nt][i][1] *= f1;
            o[nt][i][2] *= f0;
            o[nt][i][3] *= f1;
          }
        }
        const float b0 = m[nt][0] - kShift, b1 = m[nt][1] - kShift;
        const float e0 = exp2_fast(x[0] - b0), e1 = exp2_fast(x[1] - b1);
        const float e2 = exp2_fast(x[2] - b0), e3 = exp2_fast(x[3] - b1);
        l[nt][0] = fmaf(e0 + e2, inv, l[nt][0]);
        l[nt][1] = fmaf(e1 + e3, inv, l[nt][1]);
        p[nt][0] = transpose8x8(Elem<__half>::pack2(e0, e1));
        p[nt][1] = transpose8x8(Elem<__half>::pack2(e2, e3));
      }
      // v: words of 4 elements of the 4 tokens -> pairs of tokens of one element
#pragma unroll
      for (int j = 0; j < VB / 4; ++j) {
        const uint32_t x0 = __byte_perm(r.v[0][j], r.v[1][j], 0x5140), x1 = __byte_perm(r.v[0][j], r.v[1][j], 0x7362);
        const uint32_t y0 = __byte_perm(r.v[2][j], r.v[3][j], 0x5140), y1 = __byte_perm(r.v[2][j], r.v[3][j], 0x7362);
        const uint32_t a0[4] = {halves(x0), halves_hi(x0), halves(y0), halves_hi(y0)};
        const uint32_t a1[4] = {halves(x1), halves_hi(x1), halves(y1), halves_hi(y1)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          ptx::mma_16816<false>(o[nt][2 * j], a0, p[nt][0], p[nt][1]);
          ptx::mma_16816<false>(o[nt][2 * j + 1], a1, p[nt][0], p[nt][1]);
        }
      }
      load_v(r, it + 1);
    };
    for (int it = 0; it < nu; ++it) group(it);

    // ---- the warps' sums meet in shared memory.  What lane g has of m-tile mt lies at
    // 16 mt + 2 g: neighbouring lanes write neighbouring words.
    constexpr int LD = D + 8;
    __syncthreads();
    float* acc = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nt][e];
#pragma unroll
        for (int d = 4; d < 32; d *= 2) sum += __shfl_xor_sync(~0u, sum, d);
        const int row = 8 * nt + 2 * c + e;
        if (g == 0) {
          stat[warp][row][0] = m[nt][e];
          stat[warp][row][1] = sum;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
          *reinterpret_cast<float2*>(acc + ((size_t)warp * R + row) * LD + 16 * i + 2 * g) =
              make_float2(o[nt][i][e], o[nt][i][2 + e]);
      }
    }
    __syncthreads();
    const bool whole = begins && w == item1;
    const int which = begins ? 1 : 0;       // an item begun here and not ended is this CTA's last
    float* part = part_of<D, NT>(a, blockIdx.x, which);
    for (int i = tid; i < t.rows * (D / 2); i += kFThreads) {
      const int row = i / (D / 2), pr = i % (D / 2), d = 2 * pr;
      const int gg = d % (8 * PW) / PW, mt = d / (8 * PW) * (PW / 2) + d % PW / 2;
      float top = stat[0][row][0];
#pragma unroll
      for (int k = 1; k < kFWarps; ++k) top = fmaxf(top, stat[k][row][0]);
      float x = 0.f, y = 0.f, sum = 0.f;
#pragma unroll
      for (int k = 0; k < kFWarps; ++k) {
        const float f = exp2_fast(stat[k][row][0] - top);
        const float2 v = *reinterpret_cast<const float2*>(acc + ((size_t)k * R + row) * LD + 16 * mt + 2 * gg);
        x = fmaf(v.x, f, x);
        y = fmaf(v.y, f, y);
        sum = fmaf(stat[k][row][1], f, sum);
      }
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (d < a.dim) put_row<E>(a, t, h, row, d, x * inv, y * inv);
      } else {
        __stcg(reinterpret_cast<float2*>(part + (size_t)row * D + d), make_float2(x, y));
        if (pr == 0) __stcg(reinterpret_cast<float2*>(part + (size_t)R * D + 2 * row), make_float2(top, sum));
      }
    }
    if (!whole) {
      const int first = owner(item0, all, ctas), last = owner(item1 - 1, all, ctas);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int come = atomicAdd(a.join + first, 1);
        sh.flag = come == last - first;
        if (sh.flag) a.join[first] = 0;     // as the next call finds it
      }
      __syncthreads();
      if (sh.flag) {
        __threadfence();
        for (int i = tid; i < t.rows * (D / 2); i += kFThreads) {
          const int row = i / (D / 2), d = 2 * (i % (D / 2));
          if (d >= a.dim) continue;
          float top = -FLT_MAX, x = 0.f, y = 0.f, sum = 0.f;
          for (int k = first; k <= last; ++k) {
            const float* pk = part_of<D, NT>(a, k, k == first ? 1 : 0);
            const float2 ms = __ldcg(reinterpret_cast<const float2*>(pk + (size_t)R * D + 2 * row));
            const float2 v = __ldcg(reinterpret_cast<const float2*>(pk + (size_t)row * D + d));
            const float up = fmaxf(top, ms.x), f0 = exp2_fast(top - up), f1 = exp2_fast(ms.x - up);
            x = x * f0 + v.x * f1;
            y = y * f0 + v.y * f1;
            sum = sum * f0 + ms.y * f1;
            top = up;
          }
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          put_row<E>(a, t, h, row, d, x * inv, y * inv);
        }
      }
    }
    __syncthreads();                        // shared memory is free again
  }
}

template <int D, int NT, typename E>
cudaError_t few_launch(const AttnArgs& a, cudaStream_t st) {
  constexpr int smem = kFWarps * 8 * NT * (D + 8) * 4;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(attention_few_kernel<D, NT, E>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(148 * few_ctas<D, NT>(), 1, 1);
  cfg.blockDim = dim3(kFThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return counted_launch(cudaLaunchKernelEx(&cfg, attention_few_kernel<D, NT, E>, a));
}

template <int D, typename E>
cudaError_t few_rows(const AttnArgs& a, cudaStream_t st) {
  return a.starts == nullptr && a.group <= 8 ? few_launch<D, 1, E>(a, st) : few_launch<D, 2, E>(a, st);
}

template <typename E>
cudaError_t few_width(const AttnArgs& a, cudaStream_t st) {
  if (a.dim <= 64) return few_rows<64, E>(a, st);
  if (a.dim <= 128) return few_rows<128, E>(a, st);
  if (a.dim <= 192) return few_rows<192, E>(a, st);
  return few_rows<256, E>(a, st);
}

}  // namespace

// two parts of each CTA, of the kernel that needs more room
size_t CacheWork::part_floats(int dim) {
  const int D = (dim + 63) / 64 * 64;
  const size_t few = (size_t)148 * 4 * kFewRows, many = (size_t)148 * (D <= 128 ? kManyRows : kManyRows / 2);
  return 2 * (few > many ? few : many) * (D + 2);
}

cudaError_t launch_attention_few(lora_dtype dt, const AttnArgs& a, cudaStream_t st) {
  return dt == LORA_BF16 ? few_width<__nv_bfloat16>(a, st) : few_width<__half>(a, st);
}

}  // namespace lora
