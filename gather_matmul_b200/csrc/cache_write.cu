// Keys and values of new tokens into the paged 8-bit cache (lora_cache_write).
//
// A scale belongs to one (page, k or v, head): the smallest power of two s with
// max |x| <= 448 s over the page's tokens.  Powers of two cost e4m3 nothing (its
// relative step is the same over 15 binades) and make the change of a page's
// scale exact but for values that fall below its normal range: a page that is
// begun already keeps its scale or, when a new token needs a larger one, its
// values are divided by the quotient of the two and rounded once more.
//
// Several tokens: one warp holds 16 tokens of one head of k or v in registers (read
// once), page / 16 warps meet in shared memory for the maximum.  Bound by memory, two
// bytes read and one written for each element, and by the chain from a slot to its
// sequence, its page and its scale, which values are loaded beside, and which each of two
// waves of CTAs pays.  8 x 1024 tokens of 8 heads of 128: 15.3 us, 3.3 TB/s, 0.50 of the
// measured copy rate (three CTAs to an SM instead of four 18).  512 single tokens 5 us; in
// the kernel of several 15.
#include "cache.h"
#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

namespace {

constexpr int kWThreads = 256;

// the e4m3 codes of two floats, a in the low byte; past +-448 to +-448, NaN to NaN
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    const uint16_t two = (uint16_t)(w >> (16 * i));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    out |= e4m3x2(f.x * r, f.y * r) << (16 * i);
  }
  return out;
}

// The smallest power of two, within 2^-32 and 2^32, that is at least a / 448;
// NaN for an infinity or a NaN.  448 = 1.75 * 2^8.
__device__ __forceinline__ float power_scale(float a) {
  const uint32_t u = __float_as_uint(a);
  if (u >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, -32), 32);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// With a power of two the product with 1 / s is the quotient; a page that is begun may have
// another factor, not of lora_cache_write's making.
__device__ __forceinline__ bool power_of_two(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0; }

// the e4m3 codes of 8 elements' quotients
template <typename E, typename F>
__device__ __forceinline__ uint2 codes8(const uint4& x, F quotient) {
  float f[8];
  Elem<E>::to_f32(x, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = quotient(f[i]);
  return make_uint2(e4m3x2(f[0], f[1]) | (e4m3x2(f[2], f[3]) << 16), e4m3x2(f[4], f[5]) | (e4m3x2(f[6], f[7]) << 16));
}

// NC: 16-byte pieces (8 elements) that a lane holds of its warp's 16 tokens, at most
template <typename E, int NC>
__global__ void __launch_bounds__(kWThreads, NC <= 8 ? 4 : 2)
cache_write_kernel(const __grid_constant__ CacheWriteArgs a) {
  __shared__ uint32_t warp_max[kWThreads / 32];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int page = 1 << a.page_log, wpu = page >> 4;       // warps of a unit
  const int sub = warp & (wpu - 1);
  const int64_t unit = ((int64_t)blockIdx.x * (kWThreads / 32) + warp) / wpu;
  const int sides = 2 * a.Hk;
  const int64_t slot = unit / sides;
  const int side = (int)(unit - slot * sides);             // k heads, then v heads

  // the slot's sequence and page: sequence b owns the slots from starts[b] / page + 2 b,
  // as many as its new tokens can touch pages
  int lo = 0, hi = a.B;                                     // first slot of lo <= slot < that of hi
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool below = at < hi && (int64_t)(a.starts[at] >> a.page_log) + 2 * at <= slot;
    const int k = max(31 - __clz(__ballot_sync(~0u, below)), 0);
    lo += k * step;
    hi = min(hi, lo + step);
  }
  const int b = lo;
  const int s0 = a.starts[b], s1 = a.starts[b + 1], len = a.lengths[b];
  int row0 = min(max(s0, 0), a.T);
  const int n = min(max(s1, row0), a.T) - row0;
  if ((s0 < 0 || s1 < s0 || s1 > a.T) && side == 0 && sub == 0 && lane == 0) atomicAdd(a.bad + 1, 1);
  const int64_t t = slot - (s0 >> a.page_log) - 2 * (int64_t)b;
  bool live = t >= 0 && t < 0x7fffffff;
  const int touch = live ? (int)t : 0;
  int first = 0, last = 0, page_at = 0, begun = 0;          // new positions [first, last) of this page
  int64_t pid = -1;
  if (live) {
    const int p0 = max(len - n, 0);
    const int64_t pi = (int64_t)(p0 >> a.page_log) + touch;
    live = len > 0 && n > 0 && (pi << a.page_log) < len;
    if (live) {
      page_at = (int)(pi << a.page_log);
      first = max(p0, page_at);
      last = (int)min((int64_t)len, (int64_t)page_at + page);
      begun = first - page_at;
      row0 += first - (len - n);
      pid = pi < a.M ? a.tables[(int64_t)b * a.M + pi] : -1;
    }
  }
  const bool is_v = side >= a.Hk;
  const E* x = static_cast<const E*>(is_v ? a.v : a.k);
  const int64_t ld = is_v ? a.ldv : a.ldk;
  x += (int64_t)(is_v ? side - a.Hk : side) * a.dim;
  const int per_row = a.dim >> 3, nc = a.dim >> 4;          // pieces of a token, and of a lane
  const int inv_row = (65535 + per_row) / per_row;          // i / per_row, exact for i < 512
  const int t0 = page_at + sub * 16;

  uint4 r[NC];
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    r[k] = make_uint4(0, 0, 0, 0);
    if (k < nc && live) {
      const int i = lane + 32 * k, row = i * inv_row >> 16, t = t0 + row;
      if (t >= first && t < last)
        r[k] = ldg_stream(x + (int64_t)(row0 + t - first) * ld + 8 * (i - row * per_row));
    }
  }
  if (live && (pid < 0 || pid >= a.P)) {                    // looked at once x is on its way
    if (side == 0 && sub == 0 && lane == 0) atomicAdd(a.bad, 1);
    live = false;
  }
  const int64_t place = pid * sides + side;
  float before = 0.f;
  if (live && begun) before = a.scale[place];
  // 16-bit magnitudes order as their bits do; infinities and NaN come out on top
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const uint32_t m = __vmaxu2(__vmaxu2(r[k].x & 0x7fff7fffu, r[k].y & 0x7fff7fffu),
                                __vmaxu2(r[k].z & 0x7fff7fffu, r[k].w & 0x7fff7fffu));
    top = __vmaxu2(top, m);
  }
  top = max(top & 0xffffu, top >> 16);
  top = __reduce_max_sync(~0u, top);
  if (wpu > 1) {
    if (lane == 0) warp_max[warp] = top;
    __syncthreads();
    for (int i = 0; i < wpu; ++i) top = max(top, warp_max[(warp & ~(wpu - 1)) + i]);
  }
  if (!live) return;
  float s = power_scale(Elem<E>::to_f32((uint16_t)top));
  if (begun) s = before >= s ? before : (before < s ? s : before + s);   // NaN stays NaN
  else before = s;
  if (wpu > 1) {
    // every warp has read the old scale; the barrier counts the unit's own warps only
    asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / wpu), "r"(wpu * 32) : "memory");
  }
  uint8_t* out = a.cache + (place << a.page_log) * a.dim;
  if (before != s && before == before && s == s) {
    const float ratio = before / s;
    const int pieces = a.dim >> 4;                          // 16 bytes each
    for (int i = lane; i < 16 * pieces; i += 32) {
      const int row = sub * 16 + i / pieces;
      if (row < begun) {
        uint4* p = reinterpret_cast<uint4*>(out + (int64_t)row * a.dim + 16 * (i % pieces));
        uint4 v = *p;
        v = make_uint4(rescale4(v.x, ratio), rescale4(v.y, ratio), rescale4(v.z, ratio), rescale4(v.w, ratio));
        *p = v;
      }
    }
  }
  if (sub == 0 && lane == 0) a.scale[place] = s;
  const auto store = [&](auto quotient) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      if (k < nc) {
        const int i = lane + 32 * k, row = i * inv_row >> 16, t = t0 + row;
        if (t >= first && t < last)
          *reinterpret_cast<uint2*>(out + (int64_t)(t - page_at) * a.dim + 8 * (i - row * per_row)) = codes8<E>(r[k], quotient);
      }
    }
  };
  const float inv = 1.f / s;
  // one branch for all (a branch in each piece 17.4 us)
  if (power_of_two(s)) store([=](float f) { return f * inv; });
  else store([=](float f) { return f / s; });
}

// Single tokens: LANES lanes, of 8 elements each, for a head of k or v; little to hold
// for each, so that all of a decode batch is on the GPU at once.
template <typename E, int LANES>
__global__ void __launch_bounds__(kWThreads)
cache_write_single_kernel(const __grid_constant__ CacheWriteArgs a) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  const int sides = 2 * a.Hk, lane = threadIdx.x & (LANES - 1);
  const int64_t unit = ((int64_t)blockIdx.x * kWThreads + threadIdx.x) / LANES;
  const int64_t seq = unit / sides;
  const int side = (int)(unit - seq * sides), b = (int)min(seq, (int64_t)a.B - 1);
  const int len = a.lengths[b];
  bool live = seq < a.B && len > 0;
  const int at = max(len - 1, 0), page = 1 << a.page_log, begun = at & (page - 1);
  int64_t pid = -1;
  if (live && at >> a.page_log < a.M) pid = a.tables[(int64_t)b * a.M + (at >> a.page_log)];
  const bool is_v = side >= a.Hk;
  const E* x = static_cast<const E*>(is_v ? a.v : a.k) + (int64_t)b * (is_v ? a.ldv : a.ldk) +
               (int64_t)(is_v ? side - a.Hk : side) * a.dim;
  uint4 r = make_uint4(0, 0, 0, 0);
  if (live && 8 * lane < a.dim) r = ldg_stream(x + 8 * lane);
  if (live && (pid < 0 || pid >= a.P)) {
    if (side == 0 && lane == 0) atomicAdd(a.bad, 1);
    live = false;
  }
  const int64_t place = pid * sides + side;
  float before = 0.f;
  if (live && begun) before = a.scale[place];
  const uint32_t m = __vmaxu2(__vmaxu2(r.x & 0x7fff7fffu, r.y & 0x7fff7fffu), __vmaxu2(r.z & 0x7fff7fffu, r.w & 0x7fff7fffu));
  uint32_t top = max(m & 0xffffu, m >> 16);
#pragma unroll
  for (int d = 1; d < LANES; d *= 2) top = max(top, __shfl_xor_sync(~0u, top, d));
  if (!live) return;
  float s = power_scale(Elem<E>::to_f32((uint16_t)top));
  if (begun) s = before >= s ? before : (before < s ? s : before + s);   // NaN stays NaN
  else before = s;
  uint8_t* out = a.cache + (place << a.page_log) * a.dim;
  if (before != s && before == before && s == s) {
    const float ratio = before / s;
    for (int i = lane; i < begun * (a.dim >> 4); i += LANES) {
      uint4* p = reinterpret_cast<uint4*>(out) + i;
      uint4 v = *p;
      v = make_uint4(rescale4(v.x, ratio), rescale4(v.y, ratio), rescale4(v.z, ratio), rescale4(v.w, ratio));
      *p = v;
    }
  }
  if (lane == 0) a.scale[place] = s;
  if (8 * lane < a.dim) {
    const float inv = 1.f / s;
    *reinterpret_cast<uint2*>(out + (int64_t)begun * a.dim + 8 * lane) =
        power_of_two(s) ? codes8<E>(r, [=](float f) { return f * inv; }) : codes8<E>(r, [=](float f) { return f / s; });
  }
}

template <typename K>
cudaError_t launch_ctas(K kernel, const CacheWriteArgs& a, int64_t ctas, cudaStream_t st) {
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(kWThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return counted_launch(cudaLaunchKernelEx(&cfg, kernel, a));
}

template <typename E, int LANES>
cudaError_t single_launch(const CacheWriteArgs& a, cudaStream_t st) {
  return launch_ctas(cache_write_single_kernel<E, LANES>, a, ((int64_t)a.B * 2 * a.Hk * LANES + kWThreads - 1) / kWThreads, st);
}

template <typename E, int NC>
cudaError_t write_launch(const CacheWriteArgs& a, cudaStream_t st) {
  const int64_t slots = (int64_t)(a.T >> a.page_log) + 2 * (int64_t)a.B;
  const int64_t warps = (slots * 2 * a.Hk) << (a.page_log - 4);
  return launch_ctas(cache_write_kernel<E, NC>, a, (warps + kWThreads / 32 - 1) / (kWThreads / 32), st);
}

template <typename E>
cudaError_t write_width(const CacheWriteArgs& a, cudaStream_t st) {
  if (a.starts == nullptr) {
    if (a.dim <= 64) return single_launch<E, 8>(a, st);
    if (a.dim <= 128) return single_launch<E, 16>(a, st);
    return single_launch<E, 32>(a, st);
  }
  if (a.dim <= 64) return write_launch<E, 4>(a, st);
  if (a.dim <= 128) return write_launch<E, 8>(a, st);
  return write_launch<E, 16>(a, st);
}

}  // namespace

cudaError_t launch_cache_write(lora_dtype dt, const CacheWriteArgs& a, cudaStream_t st) {
  return dt == LORA_BF16 ? write_width<__nv_bfloat16>(a, st) : write_width<__half>(a, st);
}

}  // namespace lora
