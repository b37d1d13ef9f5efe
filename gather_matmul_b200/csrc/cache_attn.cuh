// What the two attention kernels over the paged cache share: how the work of a
// batch whose lengths only the device knows is divided, and how the parts of a
// row that several CTAs computed are joined.
//
// A row is one query of one head.  The rows of a sequence that share a k/v head
// (its queries times `group` heads, queries outer) are cut into tiles of R rows;
// an item is (row tile, k/v head); a unit is U of the item's visible tokens, or one of
// `C` idle ones that stand for what an item costs beside its tokens.  All units, item
// after item, are divided evenly among the CTAs, so a batch of ragged lengths and a
// single long sequence fill the GPU alike.  Every CTA finds its own
// share from the lengths.  A CTA whose share ends inside an item leaves the sums
// of its part in the workspace; the last of an item's CTAs to come adds the parts
// in order, so results do not depend on which one that is.
#pragma once

#include "cache.h"
#include "common.cuh"
#include "ptx.cuh"

namespace lora {
namespace attn {

// A row tile of a sequence: rows r0 .. r0 + rows of the sequence's n * group,
// queries in rows q0 .. q0 + n of q, tokens [lo, hi) visible to at least one row.
struct Tile {
  int b, q0, n, len, r0, rows, lo, hi, u0, units;   // units: with the idle ones, which come first
  bool past;                                  // the sequence's first tile, and its length is past its table
};

// Slots of row tiles: the one of a sequence of few rows is the sequence's number, the
// tiles of longer ones begin at this.
template <int R>
__host__ __device__ __forceinline__ constexpr bool one_tile() { return R <= kFewRows; }
template <int R>
__device__ __forceinline__ int64_t slot_of(const AttnArgs& a, int b) {
  if constexpr (one_tile<R>()) return b;
  if (a.starts == nullptr) return (int64_t)b * ((a.group + R - 1) / R);
  return ((int64_t)a.starts[b] * a.group) / R + b;
}
template <int R>
__device__ __forceinline__ int64_t slots_of(const AttnArgs& a) {
  if constexpr (one_tile<R>()) return a.B;
  if (a.starts == nullptr) return (int64_t)a.B * ((a.group + R - 1) / R);
  return ((int64_t)a.T * a.group) / R + a.B;
}
// the sequence whose slots hold this one
template <int R>
__device__ __forceinline__ int seq_of(const AttnArgs& a, int64_t slot) {
  if constexpr (one_tile<R>()) return (int)slot;
  if (a.starts == nullptr) return (int)min(slot / ((a.group + R - 1) / R), (int64_t)a.B - 1);
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (slot_of<R>(a, mid) <= slot) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Position of a row's query, the sequence's first one being at `base`.  Queries before the
// first token (more new tokens than the length) see nothing wherever they are: at -1, from
// which any window can be taken.
__device__ __forceinline__ int position(const AttnArgs& a, int base, int row) { return max(base + row / a.group, -1); }

// units == 0: the slot holds no rows
template <int R, int U, int C>
__device__ __forceinline__ void tile_of(const AttnArgs& a, int b, int64_t slot, Tile& t) {
  t.b = b;
  t.q0 = b;
  t.n = 1;
  if (a.starts != nullptr) {
    t.q0 = min(max(a.starts[b], 0), a.T);
    t.n = min(max(a.starts[b + 1], t.q0), a.T) - t.q0;
  }
  const int64_t at = slot - slot_of<R>(a, b), all = (int64_t)t.n * a.group;
  t.units = 0;
  t.past = false;
  if (at < 0 || at * R >= all || all < a.min_rows || all > a.max_rows) return;
  t.len = max(a.lengths[b], 0);
  const int places = a.M << a.page_log;       // tokens that the table has room for
  t.past = at == 0 && t.len > places;
  t.r0 = (int)(at * R);
  t.rows = (int)min((int64_t)R, all - t.r0);
  const int p0 = position(a, t.len - t.n, t.r0), p1 = position(a, t.len - t.n, t.r0 + t.rows - 1);
  t.hi = min(p1 + 1, places);                 // what lies behind the table is left out
  t.lo = a.window > 0 ? min(max(p0 - a.window + 1, 0), t.hi) : 0;
  t.u0 = t.lo / U;
  t.units = C + max((t.hi + U - 1) / U - t.u0, 1);   // one even where nothing is visible: its rows are zero
}

struct Shared {
  unsigned long long warp[32];
  int slot, seq;
  unsigned long long off;
  int real;                                   // units of this CTA's share that have tokens
  int flag;
};

// This CTA's share [w0, w1) of all units, and the first one's slot, sequence and
// place among the slot's units (of all k/v heads).  Every thread calls it.  CTAs
// past `ctas` get nothing, and none does where starts descend: a slot's sequence is
// found by bisection here and by walking on elsewhere, which agree in ascending starts.
template <int R, int U, int C>
__device__ __forceinline__ void divide(const AttnArgs& a, Shared& sm, int min_units, unsigned long long& w0,
                                       unsigned long long& w1, unsigned long long& all, int& ctas) {
  const int64_t slots = slots_of<R>(a);
  const int64_t each = (slots + blockDim.x - 1) / blockDim.x;
  const int64_t s0 = min((int64_t)threadIdx.x * each, slots), s1 = min(s0 + each, slots);
  unsigned long long mine = 0;
  const int first = s0 < s1 ? seq_of<R>(a, s0) : 0;
  int b = first;
  Tile t;
  for (int64_t s = s0; s < s1; ++s) {
    while (b + 1 < a.B && slot_of<R>(a, b + 1) <= s) ++b;
    tile_of<R, U, C>(a, b, s, t);
    mine += (unsigned long long)t.units * a.Hk;
    if (blockIdx.x == 0 && t.past) atomicAdd(a.bad, 1);
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long in = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const unsigned long long v = __shfl_up_sync(~0u, in, d);
    if (lane >= d) in += v;
  }
  if (lane == 31) sm.warp[warp] = in;
  if (threadIdx.x == 0) sm.real = 0;
  bool descends = false;
  if (a.starts != nullptr && (!one_tile<R>() || blockIdx.x == 0)) {
    for (int i = threadIdx.x; i < a.B; i += blockDim.x) {
      const int q0 = a.starts[i], q1 = a.starts[i + 1];
      descends |= q1 < q0;
      if (blockIdx.x == 0 && (q0 < 0 || q1 < q0 || q1 > a.T)) atomicAdd(a.bad + 1, 1);
    }
  }
  descends = __syncthreads_or(descends) && !one_tile<R>();
  unsigned long long base = 0;
  all = 0;
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) {
    if (i == warp) base = all;
    all += sm.warp[i];
  }
  if (descends) all = 0;
  ctas = (int)min((unsigned long long)gridDim.x, max(all / min_units, 1ull));
  if ((int)blockIdx.x >= ctas) {
    w0 = w1 = 0;
  } else {
    w0 = all * blockIdx.x / ctas;
    w1 = all * (blockIdx.x + 1) / ctas;
  }
  const unsigned long long begin = base + in - mine;
  if (begin < w1 && w0 < begin + mine) {
    unsigned long long at = begin;
    int real = 0;
    b = first;
    for (int64_t s = s0; s < s1 && at < w1; ++s) {
      while (b + 1 < a.B && slot_of<R>(a, b + 1) <= s) ++b;
      tile_of<R, U, C>(a, b, s, t);
      const unsigned long long u = (unsigned long long)t.units * a.Hk;
      if (u > 0 && w0 < at + u) {             // a slot without rows has no places
        if (w0 >= at) {
          sm.slot = (int)s;
          sm.seq = b;
          sm.off = w0 - at;
        }
        // idle units before place x of the slot
        const auto idle = [&](unsigned long long x) { return (int)(x / t.units) * C + (int)min((unsigned long long)C, x % t.units); };
        const unsigned long long from = max(w0, at) - at, to = min(w1, at + u) - at;
        real += (int)(to - from) - (idle(to) - idle(from));
      }
      at += u;
    }
    atomicAdd(&sm.real, real);
  }
  __syncthreads();
}

// the CTA whose share holds unit u
__device__ __forceinline__ int owner(unsigned long long u, unsigned long long all, int ctas) {
  return (int)(((u + 1) * ctas - 1) / all);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace attn
}  // namespace lora
