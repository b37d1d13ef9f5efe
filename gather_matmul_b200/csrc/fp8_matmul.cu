// Block-scaled e4m3 matrix product on tcgen05:
//   y[t][n] = sum_b q_scale[t][b] w_scale[n/128][b] sum_{k in b} q[t][k] W[n][k]
//
// One scale block is 128 columns = one 128-byte swizzled row of a K-major
// operand tile = four kind::f8f6f4 MMAs of K = 32.  The scales are arbitrary
// fp32 numbers that change with every block, so no accumulator can live in
// tensor memory across blocks: each block's product goes to a tensor-memory
// buffer of its own, and warps beside the pipeline read it and add it, times
// its scale, to fp32 sums in registers ("promotion") while the tensor core
// works on the next block in another buffer.
//
// Two kernels, wide for many tokens and narrow for few (below).
//
// A wait that runs out (up to a second; never in a sound run) ends the kernel and
// makes its outputs NaN.
//
// Tensor memory is allocated before the wait for the previous kernel, which may not
// have allocated its own yet (the adapters' kernels let their successors start
// first).  No CTA is starved by that, on this stream or another: a CTA that takes all
// 512 columns fills its SM's shared memory, and of those that take up to 256 an SM
// holds two.
#include <string.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

namespace {

constexpr int kBlockK = LORA_FP8_BLOCK;

__device__ __forceinline__ char* align1024(char* p) {
  return reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// After a timed-out wait: let copies in flight into this CTA's shared memory
// land before it exits (10 ms, a bound and not a measure).
__device__ __forceinline__ void drain_copies() {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (ptx::globaltimer_ns() - t0 < 10000000ull) __nanosleep(100000);
}

// ---------------------------------------------------------------------------
// Wide: 256 tokens x 256 outputs per pair of CTAs (cta_group::2), tokens on the
// MMA's M side, so that a thread's tensor-memory lane is one token and a block's
// scale one number per thread and half of the tile.
//
// 256 x 256 is the largest tile whose fp32 sums fit the registers (128 a thread in
// eight warps of each CTA), and reads the fewest operand bytes per MMA: 64 KB per
// block of 512 MMA clocks and pair.  Tensor memory then holds two blocks.
//
// What bounds it: the hand-over MMA -> promotion -> MMA, two blocks deep, whose
// steps take 150 to 200 clocks each beside the copies; the tensor pipe is busy 65 %
// of the time at 4096 x 8192 x 4096.  At 8192 x 28672 x 4096: 792 to 830 us (2.3 to
// 2.4 PFLOP/s) at full clocks, 966 to 984 us in a long run, which stands at the power
// limit at 1.49 GHz.  An earlier form took 750 without the promotion's arithmetic and
// 508 without the MMAs.
// ---------------------------------------------------------------------------
constexpr int kWTile = 256;                 // tokens and outputs per pair
constexpr int kWHalf = 128;                 // rows of A and of B that one CTA loads
constexpr int kWStages = 5;
constexpr int kWBufs = 4;                   // tensor-memory buffers of 128 columns
constexpr int kWPromote = 8;                // promotion warps
constexpr int kWSlots = 4;                  // groups of 4 blocks whose scales are in shared memory
constexpr int kWThreads = 32 * (kWPromote + 4);
// registers: 168 a thread at launch (384 threads); 2 x 232 + 40 = 3 x 168
constexpr int kWRegsPromote = 232, kWRegsRest = 40;

struct WideSmem {
  static constexpr int kOperand = kWHalf * kBlockK;             // 16 KB
  static constexpr int kStage = 2 * kOperand;
  static constexpr int kOut = kWStages * kStage;                // 3 x 2 KB per promotion warp
  static constexpr int kScale = kOut + kWPromote * 6144;        // per slot: 4 of 128 tokens, 4 of 2 of W
  static constexpr int kSlot = 16 * (kWHalf + 2);
  static constexpr int kBar = kScale + kWSlots * kSlot;
  static constexpr int kTotal = kBar + 8 * 2 * (kWStages + kWBufs + kWSlots) + 64 + 1024;
};
static_assert(WideSmem::kTotal <= 227 * 1024, "one CTA per SM");

struct WideParams {
  CUtensorMap tmQ, tmW, tmY;     // boxes {128, 128}, {128, 64} bytes; y {32, 32} elements
  const float* q_scale;
  const float* w_scale;
  uint16_t* y;
  int64_t ldy;
  int T, N, KB, NB, KS;
  int m_tiles, n_tiles;
  int w_early;                   // W is not written by the previous launch
};

// Tile order: groups of 8 token tiles, output tiles within a group, so that the
// CTAs of one wave share few rows of x and of W.
__device__ __forceinline__ void wide_tile(const WideParams& P, int tile, int& m0, int& n0) {
  const int per = 8 * P.n_tiles;
  const int g = tile / per, r = tile % per;
  const int gm = min(8, P.m_tiles - 8 * g);
  m0 = (8 * g + r % gm) * kWTile;
  n0 = (r / gm) * kWTile;
}

template <typename E>
__global__ void __launch_bounds__(kWThreads, 1)
matmul_fp8_wide_kernel(const __grid_constant__ WideParams P) {
  using L = WideSmem;
  constexpr uint32_t kIdesc = ptx::umma_idesc_e4m3(kWTile, kWHalf);
  extern __shared__ char smem_raw[];
  char* smem = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* empty = full + kWStages;
  uint64_t* tfull = empty + kWStages;
  uint64_t* tempty = tfull + kWBufs;
  uint64_t* sfull = tempty + kWBufs;
  uint64_t* sempty = sfull + kWSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sempty + kWSlots);
  volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t stop_at = ptx::smem_u32(tmem_slot + 1);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);     // uniform in the warp
  const uint32_t rank = ptx::cluster_rank(), half = rank & 1, leader = rank & ~1u;
  const int KS = P.KS, part = (int)(rank >> 1);
  const int n_tiles = P.m_tiles * P.n_tiles;
  const int first = blockIdx.x / (2 * KS), stride = gridDim.x / (2 * KS);
  const int kb0 = part * P.KB / KS, kb1 = (part + 1) * P.KB / KS;

  if (tid == 0) {
    for (int s = 0; s < kWStages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 2);             // both issuing warps
    }
    for (int b = 0; b < kWBufs; ++b) {
      ptx::mbar_init(&tfull[b], 1);
      ptx::mbar_init(&tempty[b], kWPromote);    // half of them, in both CTAs
    }
    for (int s = 0; s < kWSlots; ++s) {
      ptx::mbar_init(&sfull[s], 32);
      ptx::mbar_init(&sempty[s], kWPromote);
    }
    ptx::fence_mbar_init();
    *stop = 0;
    ptx::prefetch_tensormap(&P.tmQ);
    ptx::prefetch_tensormap(&P.tmW);
    ptx::prefetch_tensormap(&P.tmY);
  }
  if (warp == kWPromote + 1) {
    ptx::tmem_alloc_pair(tmem_slot, 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_arrive();
  ptx::cluster_wait();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // W's tiles of the first stages before the wait for the previous kernel (the
  // quantiser of the same call, which writes q and its scales only)
  const int early = P.w_early && first < n_tiles ? min(kWStages, kb1 - kb0) : 0;
  if (warp == kWPromote && lane == 0 && early > 0) {
    int m0, n0;
    wide_tile(P, first, m0, n0);
    for (int i = 0; i < early; ++i) {
      if (half == 0) ptx::mbar_arrive_expect_tx(&full[i], 2 * L::kStage);
      for (int h = 0; h < 2; ++h)
        ptx::tma_load_2d_pair(smem + i * L::kStage + L::kOperand + h * 64 * kBlockK, &P.tmW,
                              (kb0 + i) * kBlockK, n0 + h * kWHalf + (int)half * 64,
                              ptx::map_rank(&full[i], leader));
    }
  }
  __syncwarp();
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();

  if (warp >= kWPromote) {
    ptx::reg_dec<kWRegsRest>();
    if (warp == kWPromote) {
      // operand tiles of this CTA's half
      if (lane == 0) {
        int it = 0;
        const uint32_t bar0 = ptx::map_rank(full, leader), em = ptx::smem_u32(empty);
        for (int tile = first; tile < n_tiles && !*stop; tile += stride) {
          int m0, n0;
          wide_tile(P, tile, m0, n0);
          for (int kb = kb0; kb < kb1; ++kb, ++it) {
            const int s = it % kWStages;
            if (it >= kWStages && !ptx::mbar_wait_asm(em + 8 * s, (it / kWStages - 1) & 1, stop_at))
              break;
            char* st = smem + s * L::kStage;
            const uint32_t bar = bar0 + 8 * s;
            if (half == 0 && it >= early) ptx::mbar_arrive_expect_tx(&full[s], 2 * L::kStage);
            ptx::tma_load_2d_pair(st, &P.tmQ, kb * kBlockK, m0 + (int)half * kWHalf, bar);
            if (it < early) continue;
            // W's rows in two boxes of 64: the MMA of output half h takes rows
            // h * 64 .. of either CTA, which then are h * 128 + half * 64 .. of the tile
            ptx::tma_load_2d_pair(st + L::kOperand, &P.tmW, kb * kBlockK, n0 + (int)half * 64, bar);
            ptx::tma_load_2d_pair(st + L::kOperand + 64 * kBlockK, &P.tmW, kb * kBlockK,
                                  n0 + kWHalf + (int)half * 64, bar);
          }
        }
        // the last stages' release: no signal may arrive after this CTA has left
        for (int i = max(it - kWStages, 0); i < it; ++i)
          if (!ptx::mbar_wait_asm(em + 8 * (i % kWStages), (i / kWStages) & 1, stop_at)) break;
      }
    } else if (warp == kWPromote + 2) {
      // scales, in groups of 4 blocks: 128 of this CTA's tokens and two of W
      const bool wide16 = P.KB % 4 == 0 && kb0 % 4 == 0 &&
                          ((reinterpret_cast<uintptr_t>(P.q_scale) |
                            reinterpret_cast<uintptr_t>(P.w_scale)) & 15) == 0;
      const uint32_t sf = ptx::smem_u32(sfull), se = ptx::smem_u32(sempty);
      int g = 0;
      for (int tile = first; tile < n_tiles && !*stop; tile += stride) {
        int m0, n0;
        wide_tile(P, tile, m0, n0);
        m0 += (int)half * kWHalf;
        const float* src[5];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          src[i] = P.q_scale + (int64_t)min(m0 + i * 32 + lane, P.T - 1) * P.KB;
        src[4] = P.w_scale + (int64_t)min(n0 / kBlockK + (lane & 1), P.NB - 1) * P.KB;
        for (int kb = kb0; kb < kb1; kb += 4, ++g) {
          const int s = g % kWSlots;
          if (g >= kWSlots && !ptx::mbar_wait_asm(se + 8 * s, (g / kWSlots - 1) & 1, stop_at)) break;
          float* dst = reinterpret_cast<float*>(smem + L::kScale + s * L::kSlot);
          const int n = min(4, kb1 - kb);
          if (wide16 && n == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) ptx::cp_async16(dst + 4 * (i * 32 + lane), src[i] + kb);
            if (lane < 2) ptx::cp_async16(dst + 4 * (kWHalf + lane), src[4] + kb);
          } else {
            for (int j = 0; j < n; ++j) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                ptx::cp_async4(dst + 4 * (i * 32 + lane) + j, src[i] + kb + j);
              if (lane < 2) ptx::cp_async4(dst + 4 * (kWHalf + lane) + j, src[4] + kb + j);
            }
          }
          ptx::cp_async_arrive(&sfull[s]);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (half == 0) {
      // the pair's even CTA issues, one warp for each 128-column half of the tile:
      // a half's buffer goes to its four promotion warps and back without waiting
      // for the other half (66.4 us against 69.4 at 2048 x 8192 x 4096 with MMAs of
      // 256 columns); the whole warp runs the loop, an elected thread the
      // instructions
      const int h = warp == kWPromote + 1 ? 0 : 1;
      const bool one = ptx::elect_one();
      const uint32_t fu = ptx::smem_u32(full), te = ptx::smem_u32(tempty + h);
      const uint64_t dq = ptx::umma_desc_kmajor(ptx::smem_u32(smem), 128);
      const uint64_t dw = dq + ((L::kOperand + h * 64 * kBlockK) >> 4);
      const uint16_t mask = (uint16_t)(3u << leader);
      const int total = ((n_tiles - first + stride - 1) / stride) * (kb1 - kb0);
      for (int it = 0; it < total; ++it) {
        const int s = it % kWStages, b = it & 1;
        bool ok = ptx::mbar_wait_asm(fu + 8 * s, (it / kWStages) & 1, stop_at);
        ok &= ptx::mbar_wait_asm(te + 16 * b, (it / 2 + 1) & 1, stop_at);
        if (!__all_sync(~0u, ok)) break;
        ptx::tc_fence_after();
        if (one) {
          const uint32_t d = tmem + (2 * b + h) * kWHalf;
          const uint64_t qa = dq + (uint32_t)(s * (L::kStage >> 4));
          const uint64_t wa = dw + (uint32_t)(s * (L::kStage >> 4));
#pragma unroll
          for (int k = 0; k < kBlockK / 32; ++k)
            ptx::tc_mma_f8_pair(d, qa + k * 2, wa + k * 2, kIdesc, k > 0);
          ptx::tc_commit_pair(&tfull[2 * b + h], mask);
          ptx::tc_commit_pair(&empty[s], mask);
        }
        __syncwarp();
      }
    }
    __syncwarp();
  } else {
    ptx::reg_inc<kWRegsPromote>();
    // promotion: thread = token row; one 128-column half of the tile (one block
    // of W) per four warps
    const int quad = warp & 3, wh = warp >> 2, col = wh * kWHalf, row = quad * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16) + col;
    const uint32_t te = ptx::map_rank(&tempty[wh], leader);
    const uint32_t tf = ptx::smem_u32(tfull + wh), sf = ptx::smem_u32(sfull);
    char* out = smem + L::kOut + warp * 6144;
    const int nkb = kb1 - kb0, groups = (nkb + 3) / 4;
    const int all_groups = (n_tiles - first + stride - 1) / stride * groups;
    int it = 0, g = 0, box = 0;
    bool ok = true;
    // A group's scales (4 blocks) are read while the group before is worked on:
    // a wait and a read here take 300 clocks beside the copies and the MMAs.
    float4 q4, w4;
    const auto scales = [&](int group, uint32_t ready) {
      const int sl = group % kWSlots;
      ok &= ptx::mbar_wait_asm(sf + 8 * sl, (group / kWSlots) & 1, stop_at, ready);
      const float4* sc = reinterpret_cast<const float4*>(smem + L::kScale + sl * L::kSlot);
      q4 = sc[row];
      w4 = sc[kWHalf + wh];
    };
    if (all_groups > 0) scales(0, 0);
    for (int tile = first; tile < n_tiles; tile += stride) {
      uint64_t acc[2][32];
      // 32 columns at a time: the next ones are on their way from tensor memory
      // while the sums of these are formed
      uint32_t r0[32], r1[32];
      ok &= ptx::mbar_wait_asm(tf + 16 * (it & 1), (it / 2) & 1, stop_at);
      __syncwarp();
      ptx::tc_fence_after();
      ptx::tc_ld32(trow + (it & 1) * kWTile, r0);
      float4 s4;
      uint32_t sready = 0;
      bool pending = false;
      const auto block = [&](auto start, int j) {
        const auto add = [&](uint64_t* sums, uint64_t s2, const uint32_t* r) {
          if constexpr (decltype(start)::value) ptx::fmul2_set16(sums, s2, r);
          else ptx::ffma2_acc16(sums, s2, r);
        };
        if ((j & 3) == 0)
          s4 = make_float4(q4.x * w4.x, q4.y * w4.y, q4.z * w4.z, q4.w * w4.w);
        const int b = it & 1;
        const uint32_t t0 = trow + b * kWTile;
        const uint64_t s2 = ptx::pack2(s4.x, s4.x);
        s4.x = s4.y; s4.y = s4.z; s4.z = s4.w;
        const bool more = j + 1 < nkb;
        ptx::tc_wait_ld32(r0);
        ptx::tc_ld32(t0 + 32, r1);
        add(acc[0], s2, r0);
        ptx::tc_wait_ld32(r1);
        ptx::tc_ld32(t0 + 64, r0);
        add(acc[0] + 16, s2, r1);
        ptx::tc_wait_ld32(r0);
        ptx::tc_ld32(t0 + 96, r1);
        // the buffer goes back, and the next one is looked at, before the last two
        // quarters are added (63.9 us against 66.4 at 2048 x 8192 x 4096)
        ptx::tc_wait_ld32(r1);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(te + 16 * b);
        const uint32_t ready = ptx::mbar_test(tf + 16 * (b ^ 1), ((it + 1) / 2) & 1);
        add(acc[1], s2, r0);
        if ((j & 3) == 0) {
          if (lane == 0) ptx::mbar_arrive(&sempty[g % kWSlots]);
          ++g;
          pending = g < all_groups;
          sready = pending ? ptx::mbar_test(sf + 8 * (g % kWSlots), (g / kWSlots) & 1) : 0;
        } else if (pending) {
          scales(g, sready);
          pending = false;
        }
        if (more) {
          ok &= ptx::mbar_wait_asm(tf + 16 * (b ^ 1), ((it + 1) / 2) & 1, stop_at, ready);
          __syncwarp();
          ptx::tc_fence_after();
          ptx::tc_ld32(trow + (b ^ 1) * kWTile, r0);
        }
        add(acc[1] + 16, s2, r1);
        ++it;
      };
      block(std::true_type{}, 0);
      for (int j = 1; j < nkb; ++j) block(std::false_type{}, j);
      if (pending) scales(g, 0);
      int m0, n0;
      wide_tile(P, tile, m0, n0);
      m0 += (int)half * kWHalf;
      const int t = m0 + row;
      if (!ok) {
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i / 32][i % 32] = 0x7fffffff7fffffffull;
      }
      if (KS == 1) {
        // 32 rows x 32 columns at a time through a ring of three boxes in shared
        // memory, in the 64-byte swizzle the tensor map expects, and out by TMA.
        // TMA clips at T, but in a row only at whole 16 bytes: the map ends at N
        // rounded down to 8, and the last columns are stored one by one
        const int n8 = P.N & ~7;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if (lane == 0) ptx::bulk_wait_read<2>();    // the copy three boxes ago has left
          __syncwarp();
          char* o = out + box * 2048;
          char* mine = o + lane * 64;
          box = box == 2 ? 0 : box + 1;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4 v;
            uint32_t* w = &v.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint64_t u = acc[h / 2][(h % 2) * 16 + j * 4 + i];
              w[i] = Elem<E>::pack2(ptx::lo32(u), ptx::hi32(u));
            }
            *reinterpret_cast<uint4*>(mine + ((j ^ ((lane >> 1) & 3)) << 4)) = v;
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          const int mr = m0 + quad * 32, nc = n0 + col + h * 32;
          if (lane == 0) {
            if (mr < P.T && nc < n8) ptx::tma_store_2d(&P.tmY, nc, mr, o);
            ptx::bulk_commit();
          }
          if (n8 >= nc && n8 < nc + 32 && t < P.T) {
            const uint16_t* v =
                reinterpret_cast<const uint16_t*>(mine + ((((n8 - nc) >> 3) ^ ((lane >> 1) & 3)) << 4));
            for (int n = n8; n < P.N; ++n) P.y[(int64_t)t * P.ldy + n] = v[n - n8];
          }
        }
      } else {
        // one tile per cluster: part p of K hands each other part its share of a
        // thread's 128 columns (32 vectors of 4), through the drained stages, and
        // each adds the KS shares in rank order
        ptx::cluster_arrive();
        ptx::cluster_wait();
        const int sh = 6 - __ffs(KS), share = 1 << sh;      // 32 / KS; KS is a power of two
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const uint64_t u = acc[j / 16][(j % 16) * 2], v = acc[j / 16][(j % 16) * 2 + 1];
          ptx::st_cluster_v4(ptx::map_rank(smem, (uint32_t)(j >> sh) * 2 + half) +
                                 16 * ((part * share + (j & (share - 1))) * 32 * kWPromote + tid),
                             ptx::lo32(u), ptx::hi32(u), ptx::lo32(v), ptx::hi32(v));
        }
        ptx::cluster_arrive();
        ptx::cluster_wait();
        const float4* recv = reinterpret_cast<const float4*>(smem);
        for (int j = 0; j < share; ++j) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int p = 0; p < KS; ++p) {
            const float4 u = recv[(p * share + j) * 32 * kWPromote + tid];
            v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
          }
          const int jj = part * share + j;
          const int n = n0 + col + jj * 4;
          uint16_t* y = P.y + (int64_t)t * P.ldy + n;
          if (t < P.T && n + 4 <= P.N) {
            *reinterpret_cast<uint2*>(y) =
                make_uint2(Elem<E>::pack2(v.x, v.y), Elem<E>::pack2(v.z, v.w));
          } else if (t < P.T) {
            if (n < P.N) y[0] = Elem<E>::from_f32(v.x);
            if (n + 1 < P.N) y[1] = Elem<E>::from_f32(v.y);
            if (n + 2 < P.N) y[2] = Elem<E>::from_f32(v.z);
          }
        }
      }
    }
    if (lane == 0) ptx::bulk_wait_all();
    __syncwarp();
  }
  if (KS > 1 && warp >= kWPromote) {
    // the promotion warps' two cluster barriers
    ptx::cluster_arrive();
    ptx::cluster_wait();
    ptx::cluster_arrive();
    ptx::cluster_wait();
  }
  if (*stop && tid == 0) drain_copies();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_arrive();     // no CTA leaves while a peer may still signal it
  ptx::cluster_wait();
  if (warp == kWPromote + 1) ptx::tmem_dealloc_pair(tmem, 512);
}

// ---------------------------------------------------------------------------
// Narrow: 128 outputs x TN tokens per CTA, weights on the M side (a full M at any
// number of tokens), K split over a cluster where the tiles leave SMs idle.  A
// thread's lane is one output, its columns are tokens: the tokens' scales, times
// the tile's one scale of W, come through shared memory.
//
// What bounds it: one or a few tokens, reading W (12.7 us for 58.7 MB at 1 x 4096 x
// 14336, 4.6 TB/s); up to 256 tokens, the hand-over of each block between copies,
// MMA and promotion, 0.2 us with 32 tokens (10.0 us at 128 x 4096 x 4096) and
// 0.3 with 64 (13.3 us at 256 x 4096 x 4096), which CTAs beside each other hide.
// ---------------------------------------------------------------------------
constexpr int kNRows = 128;
constexpr int kNBufs = 4;           // tensor-memory buffers
constexpr int kLongK = 48;          // blocks: a K that two parts shorten enough
constexpr int kNSlots = 4;          // groups of 4 blocks whose scales are in shared memory

// Two CTAs per SM of up to 64 tokens, or one with twice the stages (DEEP).
template <int TN, bool DEEP>
struct NarrowShape {
  // promotion warps, as many as registers allow: 13.3 us with 16, 13.5 with 8, 15.1
  // with 4 at 256 x 4096 x 4096 (64 tokens, deep)
  static constexpr int kPromote = TN == 16 || (TN == 64 && !DEEP) ? 4 : (TN == 32 ? 8 : 16);
  static constexpr int kCols = TN / (kPromote / 4);                 // columns of each
  static constexpr int kCtas = DEEP ? 1 : 2;                        // per SM
  static constexpr int kIssue = TN == 64 && !DEEP ? 1 : 2;          // issuing warps (registers)
  static constexpr int kThreads = 32 * (kPromote + 2 + kIssue);
  static constexpr int kW = kNRows * kBlockK;
  static constexpr int kStage = kW + TN * kBlockK;
  static constexpr int kSlot = 4 * 4 * TN;                          // scales [4][TN]
  // as many stages as fit beside the scales and barriers (under 1.5 KB)
  static constexpr int kStages =
      (227 * 1024 / kCtas - 3584 - kNSlots * kSlot) / kStage;
  static constexpr int kTmem = TN * kNBufs;
  static constexpr int kScale = kStages * kStage;
  static constexpr int kBar = kScale + kNSlots * kSlot;
  static constexpr int kTotal = kBar + 8 * 2 * (kStages + kNBufs + kNSlots) + 64 + 1024;
  static_assert(kCtas * (kTotal + 1024) <= 228 * 1024, "CTAs per SM");
};

struct NarrowParams {
  CUtensorMap tmQ, tmW;     // boxes {128, TN}, {128, 128} bytes
  const float* q_scale;
  const float* w_scale;
  uint16_t* y;
  int64_t ldy;
  int T, N, KB, KS, n_tiles;
  int w_early;              // W is not written by the previous launch
};

template <typename E, int TN, bool DEEP>
__global__ void __launch_bounds__(NarrowShape<TN, DEEP>::kThreads, NarrowShape<TN, DEEP>::kCtas)
matmul_fp8_narrow_kernel(const __grid_constant__ NarrowParams P) {
  using L = NarrowShape<TN, DEEP>;
  constexpr int kS = L::kStages, kB = kNBufs, kPW = L::kPromote, kC = L::kCols;
  constexpr int kChunk = kC < 32 ? kC : 32;
  constexpr bool kAhead = DEEP && TN <= 64;
  constexpr uint32_t kIdesc = ptx::umma_idesc_e4m3(kNRows, TN);
  extern __shared__ char smem_raw[];
  char* smem = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* empty = full + kS;
  uint64_t* tfull = empty + kS;
  uint64_t* tempty = tfull + kB;
  uint64_t* sfull = tempty + kB;
  uint64_t* sempty = sfull + kNSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sempty + kNSlots);
  volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t stop_at = ptx::smem_u32(tmem_slot + 1);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);     // uniform in the warp
  const int KS = P.KS, part = (int)ptx::cluster_rank();
  const int unit = blockIdx.x / KS;
  const int n0 = (unit % P.n_tiles) * kNRows, t0 = (unit / P.n_tiles) * TN;
  const int kb0 = part * P.KB / KS, nkb = (part + 1) * P.KB / KS - kb0;

  if (tid == 0) {
    for (int s = 0; s < kS; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kB; ++b) {
      ptx::mbar_init(&tfull[b], 1);
      ptx::mbar_init(&tempty[b], kPW);
    }
    for (int s = 0; s < kNSlots; ++s) {
      ptx::mbar_init(&sfull[s], 32);
      ptx::mbar_init(&sempty[s], kPW);
    }
    ptx::fence_mbar_init();
    *stop = 0;
    ptx::prefetch_tensormap(&P.tmQ);
    ptx::prefetch_tensormap(&P.tmW);
  }
  if (warp == kPW + 1) {
    ptx::tmem_alloc(tmem_slot, L::kTmem);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // W's tiles of the first stages before the wait for the previous kernel (the
  // quantiser of the same call, which writes q and its scales only)
  const int early = P.w_early ? min(kS, nkb) : 0;
  if (warp == kPW && lane == 0)
    for (int i = 0; i < early; ++i) {
      ptx::mbar_arrive_expect_tx(&full[i], L::kStage);
      ptx::tma_load_2d(smem + i * L::kStage, &P.tmW, (kb0 + i) * kBlockK, n0, &full[i]);
    }
  __syncwarp();
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();

  // promotion: thread = output row, columns = tokens: 32 * (warp % 4) + lane and
  // kC columns per four warps
  const int row = (warp & 3) * 32 + lane, c0 = (warp >> 2) * kC;
  uint64_t acc[kC / 2];
  if (warp == kPW) {
    if (lane == 0) {
      const uint32_t em = ptx::smem_u32(empty);
      for (int i = 0; i < nkb; ++i) {
        const int s = i % kS;
        if (i >= kS && !ptx::mbar_wait_asm(em + 8 * s, (i / kS - 1) & 1, stop_at)) break;
        char* st = smem + s * L::kStage;
        if (i >= early) {
          ptx::mbar_arrive_expect_tx(&full[s], L::kStage);
          ptx::tma_load_2d(st, &P.tmW, (kb0 + i) * kBlockK, n0, &full[s]);
        }
        ptx::tma_load_2d(st + L::kW, &P.tmQ, (kb0 + i) * kBlockK, t0, &full[s]);
      }
      // the last stages' release: no signal may arrive after this CTA has left
      for (int i = max(nkb - kS, 0); i < nkb; ++i)
        if (!ptx::mbar_wait_asm(em + 8 * (i % kS), (i / kS) & 1, stop_at)) break;
    }
    __syncwarp();
  } else if (warp == kPW + 1 || warp == kPW + 3) {
    // two issuing warps take the blocks in turn (one waits while the other
    // issues); the whole warp runs the loop, an elected thread the instructions
    const bool one = ptx::elect_one();
    const uint32_t fu = ptx::smem_u32(full), te = ptx::smem_u32(tempty);
    const uint64_t dw = ptx::umma_desc_kmajor(ptx::smem_u32(smem), 128);
    for (int i = warp == kPW + 1 ? 0 : 1; i < nkb; i += L::kIssue) {
      const int s = i % kS, b = i % kB;
      bool ok = ptx::mbar_wait_asm(te + 8 * b, (i / kB + 1) & 1, stop_at);
      ok &= ptx::mbar_wait_asm(fu + 8 * s, (i / kS) & 1, stop_at);
      if (!__all_sync(~0u, ok)) break;
      ptx::tc_fence_after();
      if (one) {
        const uint64_t wa = dw + (uint32_t)(s * (L::kStage >> 4)), qa = wa + (L::kW >> 4);
#pragma unroll
        for (int k = 0; k < kBlockK / 32; ++k)
          ptx::tc_mma_f8(tmem + b * TN, wa + k * 2, qa + k * 2, kIdesc, k > 0);
        ptx::tc_commit(&tfull[b]);
        ptx::tc_commit(&empty[s]);
      }
      __syncwarp();
    }
  } else if (warp == kPW + 2) {
    // scales of the tile's tokens, each times the tile's one scale of W, in
    // groups of 4 blocks
    constexpr int kPer = (TN + 31) / 32;
    const uint32_t se = ptx::smem_u32(sempty);
    const float* ws = P.w_scale + (int64_t)(n0 / kBlockK) * P.KB + kb0;
    const float* qs[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      qs[i] = P.q_scale + (int64_t)min(t0 + i * 32 + lane, P.T - 1) * P.KB + kb0;
    for (int kb = 0, g = 0; kb < nkb; kb += 4, ++g) {
      const int s = g % kNSlots, n = min(4, nkb - kb);
      float v[4][kPer];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) {
          const float w = ws[kb + j];
#pragma unroll
          for (int i = 0; i < kPer; ++i) v[j][i] = qs[i][kb + j] * w;
        }
      if (g >= kNSlots && !ptx::mbar_wait_asm(se + 8 * s, (g / kNSlots - 1) & 1, stop_at)) break;
      float* dst = reinterpret_cast<float*>(smem + L::kScale + s * L::kSlot);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (j < n && i * 32 + lane < TN) dst[j * TN + i * 32 + lane] = v[j][i];
      ptx::mbar_arrive(&sfull[s]);
    }
    __syncwarp();
  } else {
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16) + c0;
    const uint32_t tf = ptx::smem_u32(tfull), sf = ptx::smem_u32(sfull);
#pragma unroll
    for (int j = 0; j < kC / 2; ++j) acc[j] = 0;
    bool ok = true;
    for (int kb = 0, g = 0; kb < nkb; kb += 4, ++g) {
      const int sl = g % kNSlots, n = min(4, nkb - kb);
      ok &= ptx::mbar_wait_asm(sf + 8 * sl, (g / kNSlots) & 1, stop_at);
      const char* sc = smem + L::kScale + sl * L::kSlot + c0 * 4;
      for (int j = 0; j < n; ++j, sc += 4 * TN) {
        const int b = (kb + j) % kB;
        const ulonglong2* s2 = reinterpret_cast<const ulonglong2*>(sc);
        // With registers to spare the scales are read before the block's sums are
        // awaited, behind the wait's own latency: 10.4 us against 11.2 at 128 x
        // 4096 x 4096 (elsewhere it spills: 43 us against 40 with 128 tokens).
        ulonglong2 sv[kAhead ? kC / 4 : 1];
        if constexpr (kAhead) {
#pragma unroll
          for (int i = 0; i < kC / 4; ++i) sv[i] = s2[i];
        }
        ok &= ptx::mbar_wait_asm(tf + 8 * b, ((kb + j) / kB) & 1, stop_at);
        __syncwarp();
        ptx::tc_fence_after();
        const uint32_t ta = trow + b * TN;
#pragma unroll
        for (int c = 0; c < kC / kChunk; ++c) {
          uint32_t r[kChunk];
          if constexpr (kChunk == 32) {
            ptx::tc_ld32(ta + c * 32, r);
            ptx::tc_wait_ld32(r);
          } else {
            ptx::tc_ld16(ta + c * 16, r);
            ptx::tc_wait_ld16(r);
          }
          if (c == kC / kChunk - 1) {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&tempty[b]);
          }
#pragma unroll
          for (int i = 0; i < kChunk / 4; ++i) {
            const int at = c * (kChunk / 4) + i;
            const ulonglong2 v = kAhead ? sv[kAhead ? at : 0] : s2[at];
            ptx::ffma2_acc(acc[2 * at], v.x, r[4 * i], r[4 * i + 1]);
            ptx::ffma2_acc(acc[2 * at + 1], v.y, r[4 * i + 2], r[4 * i + 3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sempty[sl]);
    }
    if (!ok) {
#pragma unroll
      for (int j = 0; j < kC / 2; ++j) acc[j] = 0x7fffffff7fffffffull;
    }
  }
  const int n = n0 + row;
  if (DEEP || KS == 1) {
    if (warp < kPW && n < P.N) {
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        const int t = t0 + c0 + j;
        if (t < P.T)
          P.y[(int64_t)t * P.ldy + n] =
              Elem<E>::from_f32(j & 1 ? ptx::hi32(acc[j / 2]) : ptx::lo32(acc[j / 2]));
      }
    }
  } else if constexpr (!DEEP) {
    // part p of K hands every other part its share of the tokens (TN / KS),
    // through the drained stages; each adds the KS shares in rank order
    const int sh = __ffs(TN) - __ffs(KS), share = 1 << sh;   // TN / KS; both powers of two
    ptx::cluster_arrive();
    ptx::cluster_wait();
    if (warp < kPW) {
#pragma unroll
      for (int j = 0; j < kC; ++j)
        ptx::st_cluster_f32(ptx::map_rank(smem, (uint32_t)((c0 + j) >> sh)) +
                                4 * ((part * share + ((c0 + j) & (share - 1))) * kNRows + row),
                            j & 1 ? ptx::hi32(acc[j / 2]) : ptx::lo32(acc[j / 2]));
    }
    ptx::cluster_arrive();
    ptx::cluster_wait();
    const float* recv = reinterpret_cast<const float*>(smem);
    if (warp < kPW && n < P.N) {
      for (int j = warp >> 2; j < share; j += kPW / 4) {
        const int t = t0 + part * share + j;
        if (t >= P.T) break;
        float v = 0.f;
        for (int p = 0; p < KS; ++p) v += recv[(p * share + j) * kNRows + row];
        P.y[(int64_t)t * P.ldy + n] = Elem<E>::from_f32(v);
      }
    }
  }
  if (*stop && tid == 0) drain_copies();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kPW + 1) ptx::tmem_dealloc(tmem, L::kTmem);
}

int sm_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (cache[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      n = 148;
    cache[dev] = n;
  }
  return cache[dev];
}

template <auto kKernel, typename Params>
cudaError_t cluster_launch(const Params& P, unsigned grid, unsigned cluster,
                           unsigned threads, size_t smem, cudaStream_t st) {
  // the shared-memory limit is a property of the kernel on a device: set it on
  // the first launch there only
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit) || bit == 0) {
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = pdl_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return counted_launch(cudaLaunchKernelEx(&cfg, kKernel, P));
}

template <typename E>
cudaError_t wide_launch(lora_dtype dt, const MatmulFp8Args& a, cudaStream_t st) {
  WideParams P;
  memset(&P, 0, sizeof(P));
  cudaError_t e = encode_tmap_2d_bytes(&P.tmQ, a.q, a.K, a.T, a.ldq, kBlockK, kWHalf, 128);
  if (e == cudaSuccess) e = encode_tmap_2d_bytes(&P.tmW, a.W, a.K, a.N, a.ldw, kBlockK, 64, 128);
  if (e == cudaSuccess) e = encode_tmap_2d(&P.tmY, dt, a.y, a.N < 8 ? 8 : a.N & ~7, a.T,
                                           (uint64_t)a.ldy * 2, 32, 32, 64);
  if (e != cudaSuccess) return e;
  P.q_scale = a.q_scale;
  P.w_scale = a.w_scale;
  P.y = static_cast<uint16_t*>(a.y);
  P.ldy = a.ldy;
  P.T = a.T;
  P.N = a.N;
  P.KB = (a.K + kBlockK - 1) / kBlockK;
  P.w_early = a.w_early;
  P.NB = (a.N + kBlockK - 1) / kBlockK;
  P.m_tiles = (a.T + kWTile - 1) / kWTile;
  P.n_tiles = (a.N + kWTile - 1) / kWTile;
  const int tiles = P.m_tiles * P.n_tiles, pairs = sm_count() / 2;
  // Two pairs per tile where at most half of them would work: 18.2 us against
  // 19.6 at 256 x 4096 x 4096, 37.5 against 54.6 at 512 x 4096 x 14336.  The
  // exchange of a tile's sums costs about 8 us, so not for short K (7.3 us
  // against 12 at 8192 x 128 x 512), and four parts never pay (29 against 18 us
  // at 4096 x 256 x 4096).
  const int KS = tiles * 2 <= pairs && P.KB >= 16 ? 2 : 1;
  P.KS = KS;
  const int clusters = KS > 1 ? tiles : (tiles < pairs ? tiles : pairs);
  return cluster_launch<matmul_fp8_wide_kernel<E>>(P, clusters * 2 * KS, 2 * KS, kWThreads,
                                                   WideSmem::kTotal, st);
}

template <typename E, int TN, bool DEEP>
cudaError_t narrow_launch(const MatmulFp8Args& a, cudaStream_t st) {
  NarrowParams P;
  memset(&P, 0, sizeof(P));
  cudaError_t e = encode_tmap_2d_bytes(&P.tmQ, a.q, a.K, a.T, a.ldq, kBlockK, TN, 128);
  if (e == cudaSuccess) e = encode_tmap_2d_bytes(&P.tmW, a.W, a.K, a.N, a.ldw, kBlockK, kNRows, 128);
  if (e != cudaSuccess) return e;
  P.q_scale = a.q_scale;
  P.w_scale = a.w_scale;
  P.y = static_cast<uint16_t*>(a.y);
  P.ldy = a.ldy;
  P.T = a.T;
  P.N = a.N;
  P.KB = (a.K + kBlockK - 1) / kBlockK;
  P.w_early = a.w_early;
  P.n_tiles = (a.N + kNRows - 1) / kNRows;
  const int units = P.n_tiles * ((a.T + TN - 1) / TN);
  // Parts of K.  Few CTAs are split in 8 or 4 (K = 4096, us: 4 x 1024, 8 CTAs, 7.4
  // in 2, 5.3 in 4, 4.3 in 8; 64 x 4096, 64 CTAs, 11.7 in 1, 10.7 in 2, 9.4 in 4;
  // but 1 x 4096, 32 CTAs, 6.2 in 4, 6.8 in 8), a short K only as far as one CTA
  // per SM (77 x 1504 x 1008, 60 CTAs, 4.2 in 1, 5.3 in 4).  Two parts hardly
  // repay the exchange: only of a long K (256 x 2048 x 8192: 18.8, 20.9 in 1).
  // Deep CTAs are chosen where they fill the device unsplit.
  const int sms = sm_count();
  int KS = 1;
  if constexpr (!DEEP) {
    if (P.KB >= 8 && 8 * units <= sms) KS = 8;
    else if (P.KB >= 4 && 4 * units <= (P.KB >= 16 ? 2 * sms : sms)) KS = 4;
    else if (P.KB >= kLongK && units <= sms) KS = 2;
  }
  P.KS = KS;
  return cluster_launch<matmul_fp8_narrow_kernel<E, TN, DEEP>>(
      P, units * KS, KS, NarrowShape<TN, DEEP>::kThreads, NarrowShape<TN, DEEP>::kTotal, st);
}

template <typename E>
cudaError_t matmul_launch(lora_dtype dt, const MatmulFp8Args& a, cudaStream_t st) {
  // The tile by how many CTAs it makes.  Measured (us, K = 4096 unless given,
  // the better of a tile's two depths):
  //   T x N           16     32     64    128    256 (wide)
  //   1 x 4096        6.3    6.9    8.3   15     25
  //   64 x 8192      12.7   10.7   12.6   17.4   31
  //   64 x 28672     60.3   35.7   25.8   35.1   68
  //   128 x 4096     12.3   10.1   12.3   18.4   21
  //   128 x 14336    43.4   29.1   25.2   20.3   31
  //   128 x 28672   109     66.2   47.8   37.9   49
  //   256 x 4096     23.1   15.6   13.4   18.8   17.1
  //   256 x 8192     44.0   29.3   24.7   19.9   19.3
  //   160 x 8192            23.9          19.5   25.3
  //   256 x 14336    75.4   50.4   47.0   37.4   19.5
  //   512 x 4096 x 14336    82.6   65.9   50.8   34.7
  // Tiles of 32 tokens are the best while one CTA per SM holds them all (in deep
  // CTAs, unless K is split: 10.0 at 128 x 4096, 10.6 at 64 x 8192), then 64 with
  // one deep CTA per SM (13.3 at 256 x 4096), then 32 with two, 128 with one (the wide
  // kernel is level there with full tiles only); past
  // that only the wide kernel's reuse of both operands keeps up.  Few tiles
  // of a long K go to the wide kernel, whose two parts of K then fill the device.
  // 16 tokens also where they leave CTAs to spare: 5.7 against 6.2 at 64 x 1024,
  // 4.0 against 4.5 at 128 x 1024 x 1024.
  const int sms = sm_count(), n = (a.N + kNRows - 1) / kNRows;
  const auto units = [&](int tn) { return (int64_t)n * ((a.T + tn - 1) / tn); };
  const int64_t tiles = (int64_t)((a.N + kWTile - 1) / kWTile) * ((a.T + kWTile - 1) / kWTile);
  const int KB = (a.K + kBlockK - 1) / kBlockK;
  if (a.T <= 16 || units(16) * (KB >= 16 ? 4 : 1) <= sms) return narrow_launch<E, 16, false>(a, st);
  if (a.T <= 32 || 2 * units(32) <= sms) return narrow_launch<E, 32, false>(a, st);
  if (units(32) <= sms)
    return KB < kLongK ? narrow_launch<E, 32, true>(a, st) : narrow_launch<E, 32, false>(a, st);
  if (a.T > 128 && 4 * tiles <= sms && a.K >= 40 * kBlockK) return wide_launch<E>(dt, a, st);
  if (units(64) <= sms) return narrow_launch<E, 64, true>(a, st);
  if (units(32) <= 2 * sms) return narrow_launch<E, 32, false>(a, st);
  if (a.T <= 64) return narrow_launch<E, 64, false>(a, st);
  if (a.T <= 128 || units(128) <= sms) return narrow_launch<E, 128, true>(a, st);
  return wide_launch<E>(dt, a, st);
}

}  // namespace

cudaError_t launch_matmul_fp8(lora_dtype dt, const MatmulFp8Args& a, cudaStream_t st) {
  return dt == LORA_BF16 ? matmul_launch<__nv_bfloat16>(dt, a, st)
                         : matmul_launch<__half>(dt, a, st);
}

}  // namespace lora
