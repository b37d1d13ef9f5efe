// Attention of many queries over the paged 8-bit cache (lora_cache_attention):
// prompts and chunks of prompts.  The mathematics (weights that carry the v scales,
// a running maximum that is raised late) is that of cache_attn.cu.
//
// Products run on tcgen05: S = Q K^T into tensor memory, the weights P back into
// tensor memory as fp16, O += P V with P from there.  A CTA holds two tiles of 128
// rows (one for heads of more than 128 elements), so that k and v are converted once
// for 256 rows; as fp16 operands k and v keep all their bits, and q, whose rows a power of
// two brings to 2^7 .. 2^8, what is above 2^-32 of the row's largest element.  It goes
// through its items in steps of 128 tokens:
//
//   a warpgroup for each tile's softmax, a thread for each row: scores of 64 tokens
//     from tensor memory, their weights back, the running sums; the products of one
//     half of a step run while the weights of the other are formed.  Between items it
//     brings q in and results out, through shared memory, rows side by side
//   a warpgroup each for k and v: the next tile from global memory in registers, e4m3
//     to fp16, into the swizzled layouts that the products read
//   a warp for each tile that issues its products, and one that plans: it looks up
//     pages and scales of the next steps, four steps at a time, and divides the items
//
// 8 x 1024 queries of 32 heads of 128 behind 7168 tokens each: 1200 to 1230 us in a loop of
// calls, 850 TFLOP/s, 0.52 of the measured rate of a 16-bit product, at the clock that the
// power limit leaves; 1090 us, 0.58, where calls lie apart (a CTA's step 4800 cycles at two
// tiles).  4 x 1024 queries, each the last of 4096 tokens, apart: 32 heads of 128 on 8 307
// us, 0.48, on 32 319 us, 0.46; with one tile and one buffer of k and v, 32 heads of 192
// on 8 521 us, 0.42, 16 of 256 on 4 387 us, 0.38.  No unit is full: the tensor pipe is
// busy 53 % of the time, issue slots 54 %, special functions 33 %. Scores are there
// before the softmax asks for them; it forms the weights of 64 tokens in 1250 cycles
// alone and in up to 2800 beside the other tile's, most of it waiting for shared and
// tensor memory, which the operands of the products (q and k 1536 cycles of a step, v
// 512, at 128 bytes a cycle), the converted tiles (512) and the scores and weights
// themselves keep busy.  Measured otherwise: one warpgroup that converts k, then v 1310;
// scores of 128 tokens at once, which have room for one buffer, 1235; q as an operand
// from tensor memory, which leaves room for one buffer of 64, 1370; two softmax
// warpgroups a tile, half of the columns each, 1255.
#include <cfloat>
#include <type_traits>

#include "cache_attn.cuh"
#include "internal.h"

namespace lora {

namespace {

using namespace attn;

constexpr int kN = 128, kHalf = 64;           // tokens of a step (and of a unit), and that a softmax takes at once
constexpr float kShift = 6.f, kMost = 32768.f;
// A denominator below this comes from rows that see nothing: the largest weight of
// others is at least 2^kShift / 2^32.
constexpr float kNothing = 0x1p-60f;
// Of each 8 pairs of weights, those whose exponentials are formed on the FMA pipe:
// the special function unit gives 16 a cycle and SM.  None of 8 1230 us, one 1140, two
// 1120, three 1170 (the case above).
constexpr uint32_t kPolyPairs = 0x12;
constexpr int kBlock = 4, kBlocks = 4;        // steps that are planned at once, and such blocks in shared memory
constexpr int kRing = kBlock * kBlocks;
// What an item costs beside its steps, in steps (q in, results out, the first scores:
// 9 us).  37 chunks and tokens with a window, and the case above: 1 step 92 and 1102 us,
// 3 90 and 1100, 5 92 and 1094.
constexpr int kIdle = 3;

template <int D> struct Many {
  static constexpr int kTiles = D <= 128 ? 2 : 1;
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kBufs = D <= 128 ? 2 : 1;        // of k, and of v
  // warpgroups: the softmax of each tile, the conversion of k, of v, products and plan
  static constexpr int kThreads = 128 * (kTiles + 3);
  // Registers of a thread at launch (checked before the first one), and the shares: the
  // softmax takes what the others give back, no more, and those can only give.
  static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
  static constexpr int kSoftRegs = kTiles == 2 ? 152 : 144, kConvRegs = kTiles == 2 ? 56 : 128, kOtherRegs = kTiles == 2 ? 56 : 96;
  static_assert(kTiles * kSoftRegs + 2 * kConvRegs + kOtherRegs <= (kTiles + 3) * kLaunchRegs, "more registers than the launch has");
  static_assert(kSoftRegs > kLaunchRegs && kConvRegs <= kLaunchRegs && kOtherRegs < kLaunchRegs, "setmaxnreg in its direction");
  static constexpr int kTileBytes = kN * D * 2;         // 128 rows of fp16
  static constexpr int kSmem = kTileBytes * (kTiles + 2 * kBufs) + 1024;
  static constexpr int kPieces = D / 16;                // 16 bytes of e4m3 each, of a conversion thread
  static constexpr int kCols = 512;                     // tensor memory: scores and O of each tile
};

// What the other roles need to know of a step, by groups of 16 tokens (which lie
// in one page): where a group's k and v begin in the cache behind their first page
// (kNowhere: no page, or not visible; kNaN), and (k scale, log2 v scale, 1 / v scale).
// A page whose k or v scale is NaN spoils the rows that see it and no others: its k are
// read as NaN, which masks take out of a score, its v as zeros and its scales as 1, so
// that weights of 0 add nothing.
constexpr int64_t kNowhere = -1, kNaN = -2;
struct Step {
  float4 scale[8];
  int64_t at[2][8];
  int visible;                                // tokens of the step below the last visible one
  uint32_t flags;                             // kFirst, kLast: of its item here; kSecond: so has the second tile rows
  int item;
};
constexpr uint32_t kFirst = 1, kLast = 2, kSecond = 4;
// What the softmax needs to know of an item.  The plan is at most kRing steps ahead of
// what each softmax has passed, so an item's slot, written again kItems items later, holds
// it until its steps are passed.  Its results come later still: the second tile's softmax
// passes the steps of all items without rows for it before it writes them.  What an item's
// steps and results need is in the tile's own copy.
constexpr int kItems = 2 * kRing;
struct Item {
  int q0, r0, rows, base;                     // row r: query q0 + r / group; the sequence's first is at position base
  int head, tok, steps;                       // k/v head; first token and number of steps here
  int first_cta, last_cta, which;             // CTAs that share it; which of this CTA's parts it is, -1: it is whole
};

struct ManyShared {
  Shared div;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t q_full[2], s_full[2][2], p_full[2][2], o_full[2][2], o_empty[2], plan_items[kBlocks], plan_full[kBlocks], plan_empty[kBlocks], meet[2], done[2];
  uint32_t tmem;
  int stop;
  int flag[2];
  float q_scale[2][128];                      // of a tile's rows
  Step step[kRing];
  Item item[kItems];
  Item own[2];                                // the one that a tile's softmax is at
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
    do {
      for (;;) {
        while (seq + 1 < a.B && slot_of<R>(a, seq + 1) <= slot) ++seq;
        tile_of<R, kN, kIdle>(a, seq, slot, t);
        const unsigned long long slot_units = (unsigned long long)t.units * a.Hk;
        if (off < slot_units) break;
        off -= slot_units;
        ++slot;
      }
      h = (int)(off / t.units);
      const int from = (int)(off - (unsigned long long)h * t.units);
      const int share = (int)min((unsigned long long)(t.units - from), w1 - w);
      // of the units that have tokens
      ua = max(from - kIdle, 0);
      nu = from + share - kIdle - ua;
      item0 = w - from + kIdle;
      item1 = w - from + t.units;
      w += share;
      off += share;
    } while (nu <= 0 && w < w1);
    return nu > 0;
  }
};

__device__ __forceinline__ int same(int x) { return __reduce_max_sync(~0u, x); }
__device__ __forceinline__ uint32_t same(uint32_t x) { return __reduce_max_sync(~0u, x); }

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
// {x, y} = {x, y} * s + l
__device__ __forceinline__ void fma2(float& x, float& y, uint64_t s, uint64_t l) {
  asm("{\n .reg .b64 t;\n mov.b64 t, {%0, %1};\n fma.rn.f32x2 t, t, %2, %3;\n mov.b64 {%0, %1}, t;\n}"
      : "+f"(x), "+f"(y) : "l"(s), "l"(l));
}
__device__ __forceinline__ uint64_t twice(float x) { return ptx::pack2(x, x); }
// 2^x and 2^y on the FMA pipe, arguments past 127 as 127 (a weight that large is seen
// to be too large whatever it is) and below -126 as -126: x = n + f with n the nearest
// whole number (it is left in the low bits of x + 1.5 2^23), 2^f by the polynomial of
// degree 4 whose relative error over |f| <= 1/2 is least (2.6e-6; fitted by
// reweighted least squares), times 2^n made from bits.  NaN stays NaN.
__device__ __forceinline__ void exp2_fma(float& x, float& y) {
  constexpr float kMagic = 12582912.f;
  uint64_t v, r, f, p;
  asm("max.NaN.f32 %0, %0, %1;\n min.NaN.f32 %0, %0, %2;" : "+f"(x) : "f"(-126.f), "f"(127.f));
  asm("max.NaN.f32 %0, %0, %1;\n min.NaN.f32 %0, %0, %2;" : "+f"(y) : "f"(-126.f), "f"(127.f));
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(v), "l"(twice(kMagic)));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(r), "l"(twice(-kMagic)));
  f = ptx::ffma2(p, twice(-1.f), v);
  p = ptx::ffma2(f, twice(0.009570102207362652f), twice(0.05591786280274391f));
  p = ptx::ffma2(p, f, twice(0.240247443318367f));
  p = ptx::ffma2(p, f, twice(0.6931217908859253f));
  p = ptx::ffma2(p, f, twice(0.9999992847442627f));
  const uint32_t nx = ((uint32_t)r << 23) + 0x3f800000u, ny = ((uint32_t)(r >> 32) << 23) + 0x3f800000u;
  asm("{\n .reg .b64 n;\n mov.b64 n, {%2, %3};\n mul.rn.f32x2 n, n, %4;\n mov.b64 {%0, %1}, n;\n}"
      : "=f"(x), "=f"(y) : "r"(nx), "r"(ny), "l"(p));
}

// 16 bytes, or what stands for them: no branch, so that the loads of a loop follow one another
__device__ __forceinline__ uint4 load_if(const void* p, bool in, uint32_t other = 0) {
  uint4 v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n mov.b32 %0, %6;\n mov.b32 %1, %6;\n mov.b32 %2, %6;\n mov.b32 %3, %6;\n"
      " @p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w) : "l"(p), "r"((uint32_t)in), "r"(other));
  return v;
}
// One arrival for the warp: hundreds of them a step, each a write to shared memory,
// would be in the way of the products' operands.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(bar);
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
  // Numbers that are the same in all lanes of a warp go through a warp reduction where
  // the compiler cannot see that they are: its result is in a uniform register, and so is
  // what follows from it (registers of the lanes are what this kernel is short of).
  const int tid = threadIdx.x, lane = tid & 31, warp = same(tid >> 5), wg = warp >> 2;
  const uint32_t stop = ptx::smem_u32(&sm.stop);

  if (warp == 0) ptx::tmem_alloc(&sm.tmem, M::kCols);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sm.k_full[i], 4);
      ptx::mbar_init(&sm.v_full[i], 4);
      ptx::mbar_init(&sm.k_empty[i], M::kTiles);
      ptx::mbar_init(&sm.v_empty[i], M::kTiles);
      ptx::mbar_init(&sm.q_full[i], 4);
      ptx::mbar_init(&sm.s_full[i][0], 1);
      ptx::mbar_init(&sm.s_full[i][1], 1);
      ptx::mbar_init(&sm.p_full[i][0], 4);
      ptx::mbar_init(&sm.p_full[i][1], 4);
      ptx::mbar_init(&sm.o_full[i][0], 1);
      ptx::mbar_init(&sm.o_full[i][1], 1);
      ptx::mbar_init(&sm.o_empty[i], 4);
    }
    for (int i = 0; i < kBlocks; ++i) {
      ptx::mbar_init(&sm.plan_items[i], 1);
      ptx::mbar_init(&sm.plan_full[i], 1);
      ptx::mbar_init(&sm.plan_empty[i], 4 * (M::kTiles + 2) + M::kTiles);   // softmax and conversion, issuing warps
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sm.meet[i], 4);
      ptx::mbar_init(&sm.done[i], 1);
    }
    sm.stop = 0;
    ptx::fence_mbar_init();
  }
  // Waits that give up let everyone run on, with plans that may be another step's: loops
  // end all the same, nothing is read or written where these plans say, and a call that
  // met this is counted (its workspace is then to be filled with zeros again).
  if (tid < kRing) {
    for (int i = 0; i < 16; ++i) sm.step[tid].at[i / 8][i % 8] = kNowhere;
    sm.step[tid].item = 0;
    sm.step[tid].flags = 0;
  }
  if (tid < kItems) sm.item[tid] = {0, 0, 0, 0, 0, 0, 1, 0, 0, -1};
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  ptx::tc_fence_before();
  unsigned long long w0, w1, all;
  int ctas;
  divide<M::kRows, kN, kIdle>(a, sm.div, 2, w0, w1, all, ctas);   // __syncthreads
  ptx::tc_fence_after();
  const uint32_t tmem = same(sm.tmem);
  const int steps = same(sm.div.real);
  const uint32_t s_col = 0, o_col = M::kTiles * kN;

  if (wg < M::kTiles) {
    // ------------------------------------------------------------ softmax
    ptx::reg_inc<M::kSoftRegs>();
    const int row = tid & 127, tile = wg;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t S = tmem + lanes + s_col + tile * kN, O = tmem + lanes + o_col + tile * D;
    float cs = 0.f;
    int st = 0, n_s = 0, met = 0;
    // the threads of a tile, as a barrier that a wait can leave
    auto tile_sync = [&]() {
      warp_arrive(&sm.meet[tile], lane);
      ptx::mbar_wait_asm(ptx::smem_u32(&sm.meet[tile]), met & 1, stop);
      ++met;
    };
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
        ptx::mbar_wait_asm(ptx::smem_u32(&sm.plan_items[st / kBlock % kBlocks]), (st / kRing) & 1, stop);
        const int item = same(sm.step[st % kRing].item);
        if (same(sm.item[item].rows) > 128 * tile) return item;
        for (int n = same(sm.item[item].steps); n > 0 && st < steps; --n) {
          planned();
          pass();
        }
      }
      return -1;
    };
    // Between global memory and registers a row goes through kLanes neighbouring lanes, 16
    // bytes each: a thread for each row would touch as many lines as it has lanes.
    constexpr int kLanes = D <= 64 ? 8 : D <= 128 ? 16 : 32, kApart = 128 / kLanes, kPasses = 128 / kApart;
    const int tt = tid & 127, piece = tt % kLanes;
    const int step_line = kApart / a.group, step_head = kApart % a.group;
    // the offset of this thread's piece of a row in q or y, pass after pass, and whether
    // there is such a row
    struct Walk {
      int line, head, left;
    };
    auto walk = [&](const Item& it) -> Walk {
      const int k = 128 * tile + tt / kLanes, r = it.r0 + k;
      const Walk w = {it.q0 + r / a.group, r % a.group, 8 * piece < a.dim ? it.rows - k : 0};
      __threadfence_block();                  // the item has been read
      return *const_cast<volatile int*>(&sm.stop) ? Walk{0, 0, 0} : w;
    };
    auto place = [&](const Item& it, const Walk& w, int64_t ld) -> int64_t {
      return (int64_t)w.line * ld + (it.head * a.group + w.head) * a.dim + 8 * piece;
    };
    auto on = [&](Walk& w) {
      w.line += step_line;
      w.head += step_head;
      if (w.head >= a.group) w.head -= a.group, ++w.line;
      w.left -= kApart;
    };
    // the tile's rows in shared memory, as the products read q; y goes through the same place
    uint8_t* const stage = smem + (size_t)tile * M::kTileBytes;
    auto chunk = [&](int k, int p) -> uint4* {
      return reinterpret_cast<uint4*>(stage + (p / 8) * (kN * 128) + k * 128 + (((p & 7) ^ (k & 7)) << 4));
    };
    // q of the next item waits in registers, where there is room for a tile of it
    constexpr int kGroup = kPasses <= 16 ? kPasses : 8;
    uint4 v[kGroup];
    Walk q_walk;
    auto load_group = [&](const Item& it) {
#pragma unroll
      for (int k = 0; k < kGroup; ++k, on(q_walk))
        v[k] = load_if(static_cast<const E*>(a.q) + place(it, q_walk, a.ldq), q_walk.left > 0);
    };
    auto load_q = [&](int item) {
      if constexpr (kGroup == kPasses) {
        q_walk = walk(sm.item[item]);
        load_group(sm.item[item]);
      }
    };
    auto put_q = [&](int item) {
      if constexpr (kGroup < kPasses) q_walk = walk(sm.item[item]);
#pragma unroll 1
      for (int first = 0; first < kPasses; first += kGroup) {
        if constexpr (kGroup < kPasses) load_group(sm.item[item]);
#pragma unroll
        for (int k = 0; k < kGroup; ++k) {
          const int at = tt / kLanes + kApart * (first + k);
          float f[8], top = 0.f;
          Elem<E>::to_f32(v[k], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
#pragma unroll
          for (int d = 1; d < kLanes; d *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
          // the row's largest element to 2^7 .. 2^8 by a power of two
          const int n = min(max(7 + 127 - (int)(__float_as_uint(top) >> 23), -120), 120);
          const float up = __uint_as_float((uint32_t)(127 + n) << 23);
          uint4 w;
          w.x = Elem<__half>::pack2(f[0] * up, f[1] * up);
          w.y = Elem<__half>::pack2(f[2] * up, f[3] * up);
          w.z = Elem<__half>::pack2(f[4] * up, f[5] * up);
          w.w = Elem<__half>::pack2(f[6] * up, f[7] * up);
          if (piece < D / 8) *chunk(at, piece) = w;
          if (piece == 0) sm.q_scale[tile][at] = __uint_as_float((uint32_t)(127 - n) << 23);
        }
      }
      if (row == 0) sm.own[tile] = sm.item[item];
      ptx::fence_proxy_async_smem();
      tile_sync();
      // The factor of a score is a page's (at least 2^-32) times this one.  It stays off zero,
      // since masked scores are -inf before it: a row of zeros has the scale 2^-120.  Where
      // the bound is met the scores are below 2^-30, and no weight changes.
      cs = fmaxf(sm.q_scale[tile][row] * a.c, 0x1p-90f);
      warp_arrive(&sm.q_full[tile], lane);
    };
    int item = seek();
    if (item >= 0) {
      load_q(item);
      put_q(item);
    }
    while (item >= 0) {
      const Item& it = sm.own[tile];
      int pos, pos_low, pos_high, tok, n_steps;
      {
        pos = 128 * tile + row < it.rows ? position(a, it.base, it.r0 + 128 * tile + row) : -1;
        pos_low = same(position(a, it.base, it.r0 + 128 * tile));
        pos_high = same(position(a, it.base, it.r0 + min(it.rows, 128 * tile + 128) - 1));
        tok = same(it.tok);
        n_steps = same(it.steps);
      }
      float m = -FLT_MAX, l = 0.f;
      for (int i = 0; i < n_steps; ++i) {
        if (i == 0 || st % kBlock == 0) planned();
        const Step& step = sm.step[st % kRing];
        // 64 tokens at a time: the products of one half run while the other half's weights
        // are formed
#pragma unroll 1
        for (int half = 0; half < 2; ++half, tok += kHalf) {
          const uint32_t Sh = S + kHalf * half;
          float4 sc[4];                     // read before the wait: shared memory is busy
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            sc[g] = step.scale[4 * half + g];
            sc[g].x *= cs;
          }
          ptx::mbar_wait_asm(ptx::smem_u32(&sm.s_full[tile][half]), n_s & 1, stop);
          ptx::tc_fence_after();
          const bool edge = tok + kHalf - 1 > pos_low || (a.window > 0 && tok <= pos_high - a.window);
          // 32 scores, asked for and taken
          auto ask = [&](int j, float* x) { ptx::tc_ld32(Sh + j, reinterpret_cast<uint32_t*>(x)); };
          auto take = [&](int j, float* x) {
            ptx::tc_wait_ld32(reinterpret_cast<uint32_t*>(x));
            if (edge) {
              // visible: lo < e <= hi; behind the last visible token lo may wrap, hi hides all
              const int hi = pos - (tok + j), lo = a.window > 0 ? (int)((uint32_t)hi - (uint32_t)a.window) : -1;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e > hi || e <= lo) x[e] = -INFINITY;
            }
          };
          auto raise = [&]() {
            float top = m;
#pragma unroll 1
            for (int j = 0; j < kHalf; j += 32) {
              float x[32];
              ask(j, x);
              take(j, x);
#pragma unroll
              for (int e = 0; e < 32; e += 16) {
                // factors are positive: the largest score of 16 tokens gives their largest t
                float t = x[e];
#pragma unroll
                for (int i = 1; i < 16; ++i) t = fmaxf(t, x[e + i]);
                const float4 s4 = step.scale[4 * half + (j + e) / 16];
                top = fmaxf(top, fmaf(t, s4.x * cs, s4.y));
              }
            }
            const float f = exp2_fast(m - top);
            m = top;
            l *= f;
            if (i > 0 || half > 0) {
              // once the products of all weights so far are in
              ptx::mbar_wait_asm(ptx::smem_u32(&sm.o_full[tile][half ^ 1]), (n_s + half + 1) & 1, stop);
              ptx::tc_fence_after();
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
          };
          // The weights of an item's first tokens need their maximum.  Later ones are formed
          // with the maximum so far, and again with the new one where they show to be too
          // large for fp16: where the sum of 16 of them passes kMost.
          if (i == 0 && half == 0) raise();
          uint32_t p[kHalf / 2];
          for (int again = 0;; ++again) {
            const float off = kShift - m;
            float sum = 0.f, most = 0.f, x[2][32];
            ask(0, x[0]);
#pragma unroll
            for (int h = 0; h < kHalf; h += 16) {
              float* y = x[h / 32 & 1] - h / 32 * 32;
              if (h % 32 == 0) {
                take(h, y + h);
                if (h + 32 < kHalf) ask(h + 32, x[(h / 32 + 1) & 1]);
              }
              const uint64_t s2 = twice(sc[h / 16].x), l2 = twice(sc[h / 16].y + off);
              float s0 = 0.f, s1 = 0.f;
#pragma unroll
              for (int e = h; e < h + 16; e += 2) {
                fma2(y[e], y[e + 1], s2, l2);
                if ((kPolyPairs >> (e / 2 % 8)) & 1) {
                  exp2_fma(y[e], y[e + 1]);
                } else {
                  y[e] = exp2_fast(y[e]);
                  y[e + 1] = exp2_fast(y[e + 1]);
                }
                s0 += y[e];
                s1 += y[e + 1];
                p[e / 2] = Elem<__half>::pack2(y[e], y[e + 1]);
              }
              s0 += s1;
              most = fmaxf(most, s0);
              sum = fmaf(s0, sc[h / 16].z, sum);
            }
            if (!__any_sync(~0u, most > kMost) || again) {   // with a new maximum none is too large
              l += sum;
              break;
            }
            raise();
          }
#pragma unroll
          for (int j = 0; j < kHalf / 2; j += 16) ptx::tc_st16(Sh + j, p + j);
          ptx::tc_wait_st();
          ptx::tc_fence_before();
          warp_arrive(&sm.p_full[tile][half], lane);
        }
        ++n_s;
        pass();
      }
      // q of the next item into registers, while this one's last products run
      item = seek();
      if (item >= 0) load_q(item);
      ptx::mbar_wait_asm(ptx::smem_u32(&sm.o_full[tile][1]), (n_s + 1) & 1, stop);   // the last half's products
      ptx::tc_fence_after();
      // the thread's row, into the place of q
      const int which = same(it.which);
      auto put = [&](int j, const float* o) {
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
          uint4 w;
          w.x = Elem<E>::pack2(o[e], o[e + 1]);
          w.y = Elem<E>::pack2(o[e + 2], o[e + 3]);
          w.z = Elem<E>::pack2(o[e + 4], o[e + 5]);
          w.w = Elem<E>::pack2(o[e + 6], o[e + 7]);
          *chunk(row, (j + e) / 8) = w;
        }
      };
      bool out = which < 0;
      if (which < 0) {
        const float inv = l < kNothing ? 0.f : 1.f / l;
#pragma unroll 1
        for (int j = 0; j < D; j += 16) {
          float o[16];
          ptx::tc_ld16(O + j, reinterpret_cast<uint32_t*>(o));
          ptx::tc_wait_ld16(reinterpret_cast<uint32_t*>(o));
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] *= inv;
          put(j, o);
        }
        ptx::tc_fence_before();
        warp_arrive(&sm.o_empty[tile], lane);
      } else {
        const int first_cta = same(it.first_cta), last_cta = same(it.last_cta);
        float* part = part_of<D>(a, blockIdx.x, which, tile);
#pragma unroll 1
        for (int j = 0; j < D; j += 16) {
          float o[16];
          ptx::tc_ld16(O + j, reinterpret_cast<uint32_t*>(o));
          ptx::tc_wait_ld16(reinterpret_cast<uint32_t*>(o));
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            __stcg(reinterpret_cast<float4*>(part) + (size_t)((j + e) / 4) * 128 + row,
                   make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]));
        }
        __stcg(reinterpret_cast<float2*>(part + 128 * D) + row, make_float2(m, l));
        ptx::tc_fence_before();
        warp_arrive(&sm.o_empty[tile], lane);
        __threadfence();
        tile_sync();
        if (row == 0) {
          int* join = a.join + 2 * first_cta + tile;
          sm.flag[tile] = atomicAdd(join, 1) == last_cta - first_cta;
          if (sm.flag[tile]) *join = 0;                   // as the next call finds it
        }
        tile_sync();
        out = same(sm.flag[tile]);
        if (out) {
          __threadfence();
          float top = -FLT_MAX, sum = 0.f;
          for (int k = first_cta; k <= last_cta; ++k) {
            const float2 ms = __ldcg(reinterpret_cast<const float2*>(part_of<D>(a, k, k == first_cta ? 1 : 0, tile) + 128 * D) + row);
            const float up = fmaxf(top, ms.x);
            sum = sum * exp2_fast(top - up) + ms.y * exp2_fast(ms.x - up);
            top = up;
          }
          const float inv = sum < kNothing ? 0.f : 1.f / sum;
#pragma unroll 1
          for (int j = 0; j < D; j += 16) {
            float o[16] = {};
            for (int k = first_cta; k <= last_cta; ++k) {
              const float* pk = part_of<D>(a, k, k == first_cta ? 1 : 0, tile);
              const float f = exp2_fast(__ldcg(reinterpret_cast<const float2*>(pk + 128 * D) + row).x - top) * inv;
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const float4 x = __ldcg(reinterpret_cast<const float4*>(pk) + (size_t)((j + e) / 4) * 128 + row);
                o[e] = fmaf(x.x, f, o[e]);
                o[e + 1] = fmaf(x.y, f, o[e + 1]);
                o[e + 2] = fmaf(x.z, f, o[e + 2]);
                o[e + 3] = fmaf(x.w, f, o[e + 3]);
              }
            }
            put(j, o);
          }
        }
      }
      if (out) {
        tile_sync();
        Walk w = walk(it);
#pragma unroll 1
        for (int k = tt / kLanes; k < 128 && w.left > 0; k += kApart, on(w))
          *reinterpret_cast<uint4*>(static_cast<E*>(a.y) + place(it, w, a.ldy)) = *chunk(k, piece);
        tile_sync();
      }
      if (item >= 0) put_q(item);
    }
  } else if (wg < M::kTiles + 2) {
    // ------------------------------------------------------------ conversion
    if constexpr (M::kConvRegs < M::kLaunchRegs) ptx::reg_dec<M::kConvRegs>();
    const int ct = tid & 127;
    const bool is_v = wg == M::kTiles + 1;
    const int64_t side = is_v ? ((int64_t)a.Hk * a.dim) << a.page_log : 0;
    const uint8_t* const base = a.cache + side;
    const uint32_t tiles_at = is_v ? v_at : k_at;
    uint64_t *const full = is_v ? sm.v_full : sm.k_full, *const empty = is_v ? sm.v_empty : sm.k_empty;
    uint4 r[M::kPieces];
    // A thread's pieces of 16 bytes: the same 16 of each 64-byte column, of every 32nd
    // row.  Four lanes take 64 bytes of a row, the next four of the row behind it, so that
    // the halves they store hit different banks; what depends on the lane is the same for
    // all pieces, the rest is known to the compiler.
    constexpr int A = D / 64;
    const int row0 = 2 * (ct >> 3) + ((ct >> 2) & 1), e0 = 16 * (ct & 3);
    const int64_t lane_at = (row0 & 15) * a.dim + e0;
    const uint32_t lane_sm = row0 * 128 + (((2 * (ct & 3)) ^ (row0 & 7)) << 4);
    auto load = [&](int st) {
      if (st % kBlock == 0)
        ptx::mbar_wait_asm(ptx::smem_u32(&sm.plan_full[st / kBlock % kBlocks]), (st / kRing) & 1, stop);
      const Step& step = sm.step[st % kRing];
      const int visible = is_v ? step.visible : kN;         // v behind the last visible token may be
#pragma unroll                                              // anything: zeros in its place
      for (int g = 0; g < 4; ++g) {
        const int64_t at = step.at[is_v][2 * g + (row0 >> 4)];
        const uint8_t* src = base + at + lane_at;
        const bool in = at >= 0 && row0 + 32 * g < visible;
        const uint32_t other = at == kNaN ? 0x7f7f7f7fu : 0u;
#pragma unroll
        for (int c = 0; c < A; ++c) r[g * A + c] = load_if(src + 64 * c, in && e0 + 64 * c < a.dim, other);
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
      const uint32_t dst = tiles_at + buf * M::kTileBytes + lane_sm, dst2 = dst ^ 16;
#pragma unroll
      for (int k = 0; k < M::kPieces; ++k) {
        const uint32_t at = (k % A) * (kN * 128) + (k / A) * (32 * 128);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + at), "r"(halves_lo(r[k].x)), "r"(halves_hi(r[k].x)),
                     "r"(halves_lo(r[k].y)), "r"(halves_hi(r[k].y)) : "memory");
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst2 + at), "r"(halves_lo(r[k].z)), "r"(halves_hi(r[k].z)),
                     "r"(halves_lo(r[k].w)), "r"(halves_hi(r[k].w)) : "memory");
      }
      ptx::fence_proxy_async_smem();        // before the next loads: it would wait for them
      warp_arrive(&full[buf], lane);
      if (st + 1 < steps) load(st + 1);
    }
  } else {
    // ------------------------------------------------------------ products
    ptx::reg_dec<M::kOtherRegs>();
    const int role = warp - 4 * (M::kTiles + 2);
    // One warp issues a tile's products, so that one waits while the other's run.
    auto issue = [&](auto tile) {
      constexpr int t = decltype(tile)::value;
      // operands of these instructions are wanted in uniform registers; moving them there
      // for each one made an issue of 16 take 1050 cycles
      const bool one = ptx::elect_one();
      constexpr uint32_t id_s = ptx::umma_idesc_f16(false, 128, kHalf);
      constexpr uint32_t id_o = ptx::umma_idesc_f16(false, 128, D) | ptx::kIdescNMajorB;
      const uint64_t q_desc = ptx::umma_desc_kmajor(q_at, 128), k_desc = ptx::umma_desc_kmajor(k_at, 128);
      const uint64_t v_desc = ptx::umma_desc_nmajor(v_at, kN * 128);
      constexpr uint64_t kTile16 = M::kTileBytes >> 4;
      uint32_t n_q = 0, n_p = 0, n_o = 0;
      auto flags = [&](int st) -> uint32_t {
        ptx::mbar_wait_asm(ptx::smem_u32(&sm.k_full[st % M::kBufs]), (st / M::kBufs) & 1, stop);
        const uint32_t f = same(sm.step[st % kRing].flags);
        // the block is written again when this warp has read it too: nothing else says so
        // in steps without rows for its tile
        if (st % kBlock == kBlock - 1) {
          __syncwarp();
          if (one) ptx::mbar_arrive(&sm.plan_empty[st / kBlock % kBlocks]);
          __syncwarp();
        }
        return f;
      };
      auto scores = [&](auto half, int st, uint32_t f) {
        constexpr int h = decltype(half)::value;
        if (h == 0 && (f & kFirst)) {
          ptx::mbar_wait_asm(ptx::smem_u32(&sm.q_full[t]), n_q & 1, stop);
          ++n_q;
        }
        ptx::tc_fence_after();
        if (one) {
          const uint64_t k = k_desc + (uint32_t)(st % M::kBufs) * kTile16 + h * (kHalf * 128 >> 4);
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const uint32_t off = ((j / 4) * (kN * 128) + (j % 4) * 32) >> 4;
            ptx::tc_mma_f16(tmem + s_col + t * kN + h * kHalf, q_desc + t * kTile16 + off, k + off, id_s, j > 0);
          }
          ptx::tc_commit(&sm.s_full[t][h]);
        }
        __syncwarp();
      };
      auto sums = [&](auto half, int st, uint32_t f) {
        constexpr int h = decltype(half)::value;
        ptx::mbar_wait_asm(ptx::smem_u32(&sm.p_full[t][h]), n_p & 1, stop);
        if (h == 1) ++n_p;
        if (h == 0 && (f & kFirst)) {
          if (n_o > 0) ptx::mbar_wait_asm(ptx::smem_u32(&sm.o_empty[t]), (n_o - 1) & 1, stop);
          ++n_o;
        }
        ptx::tc_fence_after();
        if (one) {
          const uint64_t v = v_desc + (uint32_t)(st % M::kBufs) * kTile16 + h * (kHalf * 128 >> 4);
#pragma unroll
          for (int j = 0; j < kHalf / 16; ++j)
            ptx::tc_mma_f16_ts(tmem + o_col + t * D, tmem + s_col + t * kN + h * kHalf + 8 * j, v + j * (2048 >> 4), id_o,
                               h > 0 || j > 0 || !(f & kFirst));
          ptx::tc_commit(&sm.o_full[t][h]);
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t* bar) {
        if (one) ptx::tc_commit(bar);
        __syncwarp();
      };
      constexpr std::integral_constant<int, 0> h0{};
      constexpr std::integral_constant<int, 1> h1{};
      // a step in which the tile has no rows: its buffer's use is over for this warp
      auto skip = [&](uint64_t* bar) {
        if (one) ptx::mbar_arrive(bar);
        __syncwarp();
      };
      const uint32_t mine = t == 0 ? 0 : kSecond;               // the flag of items with rows for this tile
      auto all_scores = [&](int st, uint32_t f) {
        uint64_t* bar = &sm.k_empty[st % M::kBufs];
        if ((f & mine) != mine) return skip(bar);
        scores(h0, st, f);
        scores(h1, st, f);
        commit(bar);
      };
      uint32_t now = 0;
      if (steps > 0) {
        now = flags(0);
        all_scores(0, now);
      }
      for (int st = 0; st < steps; ++st) {
        const int buf = st % M::kBufs;
        const bool go_on = st + 1 < steps;
        const uint32_t then = go_on ? flags(st + 1) : 0;
        ptx::mbar_wait_asm(ptx::smem_u32(&sm.v_full[buf]), (st / M::kBufs) & 1, stop);
        if ((now & mine) != mine) {
          skip(&sm.v_empty[buf]);
          if (go_on) all_scores(st + 1, then);
        } else if (!(now & kLast)) {
          // within an item each half's scores of the next step follow its sums of this one
          sums(h0, st, now);
          scores(h0, st + 1, then);
          sums(h1, st, now);
          scores(h1, st + 1, then);
          commit(&sm.v_empty[buf]);
          commit(&sm.k_empty[(st + 1) % M::kBufs]);
        } else {
          sums(h0, st, now);
          sums(h1, st, now);
          commit(&sm.v_empty[buf]);
          if (go_on) all_scores(st + 1, then);
        }
        now = then;
      }
      // nothing is in flight when tensor memory goes back
      commit(&sm.done[t]);
      ptx::mbar_wait(&sm.done[t], 0);         // whatever other waits did
    };
    if (role < M::kTiles) {
      if (role == 0) issue(std::integral_constant<int, 0>{});
      else issue(std::integral_constant<int, M::kTiles - 1>{});
    } else if (role == M::kTiles) {
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
              it.which = cur.nu == cur.t.units - kIdle ? -1 : (cur.ua == 0 ? 1 : 0);
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
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.plan_items[block]);       // q can be fetched meanwhile
        int64_t k_where = kNowhere, v_where = kNowhere;
        float4 scale = make_float4(1.f, -INFINITY, 0.f, 0.f);         // weights of 0, for scores of -inf too
        if (entry >= 0) {
          const int pid = a.tables[entry];
          if (pid < 0 || pid >= a.P) {
            atomicAdd(a.bad, 1);
          } else {
            const int64_t page = (int64_t)pid * 2 * a.Hk + head;
            const float ks = a.scale[page], vs = a.scale[page + a.Hk];
            if (ks != ks || vs != vs) {
              scale = make_float4(1.f, 0.f, 1.f, 0.f);
              k_where = kNaN;
            } else {
              scale = make_float4(ks, log2f(vs), 1.f / vs, 0.f);
              k_where = v_where = page * head_bytes + (int64_t)(at & ((1 << a.page_log) - 1)) * a.dim;
            }
          }
        }
        if (st + (lane >> 3) < steps) {
          Step& step = sm.step[(st + (lane >> 3)) % kRing];
          step.scale[lane & 7] = scale;
          step.at[0][lane & 7] = k_where;
          step.at[1][lane & 7] = v_where;
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
    cudaFuncAttributes f;
    e = cudaFuncGetAttributes(&f, attention_many_kernel<D, E>);
    if (e == cudaSuccess && f.numRegs != M::kLaunchRegs) e = cudaErrorInvalidConfiguration;   // the shares would not fit
    if (e == cudaSuccess)
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
