// Pages of the cache: taking, sharing, returning and moving them
// (lora_pages_extend / _fork / _free / _compact / _copy).
//
// What page goes where depends on counts over all pages, so one cluster of
// kPlanCtas CTAs decides it: every thread counts a run of consecutive pages
// (and of sequences), one exchange through distributed shared memory turns the
// counts into ranks, and the k-th free page meets the k-th place that wants one.
// That is a chain of latencies: 4 to 6 us for a pool of 1024 or 16 000 pages, 10 for the
// fork of 128 branches (15 with each pair's row copied by its own thread's warp).  The
// bytes are moved by a second kernel over all SMs, in pieces of 4 KB a warp, at the speed
// of a plain copy: 200 MB in 70 us, 6.0 TB/s, 0.92 of the measured rate.
#include <cooperative_groups.h>

#include "cache.h"
#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace lora {

namespace {

constexpr int kPThreads = 512;
constexpr int kPAll = kPlanCtas * kPThreads;
constexpr int kCThreads = 256;

struct PlanShared {
  int2 warp[kPThreads / 32];
  int2 cta[kPlanCtas];
};

// Exclusive ranks of two counts over the cluster's threads in order, and the
// totals.  Every thread of the cluster calls it, once it knows that the cluster's
// CTAs have all begun: their shared memory is written.
__device__ __forceinline__ void cluster_ranks(PlanShared& sm, int2 mine, int2& before, int2& total) {
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 in = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int x = __shfl_up_sync(~0u, in.x, d), y = __shfl_up_sync(~0u, in.y, d);
    if (lane >= d) in.x += x, in.y += y;
  }
  if (lane == 31) sm.warp[warp] = in;
  __syncthreads();
  int2 base = make_int2(0, 0), sum = make_int2(0, 0);
  for (int i = 0; i < kPThreads / 32; ++i) {
    if (i == warp) base = sum;
    sum.x += sm.warp[i].x;
    sum.y += sm.warp[i].y;
  }
  if (threadIdx.x < kPlanCtas) cl.map_shared_rank(sm.cta, threadIdx.x)[cl.block_rank()] = sum;
  cl.sync();
  total = make_int2(0, 0);
  for (int i = 0; i < kPlanCtas; ++i) {
    if (i == (int)cl.block_rank()) base.x += total.x, base.y += total.y;
    total.x += sm.cta[i].x;
    total.y += sm.cta[i].y;
  }
  before = make_int2(base.x + in.x - mine.x, base.y + in.y - mine.y);
  cl.sync();                                    // sm may be written again
}

__device__ __forceinline__ int plan_thread() {
  return (int)cg::this_cluster().block_rank() * kPThreads + threadIdx.x;
}

// [begin, end) of this thread's share of n things
__device__ __forceinline__ void share_of(int n, int& begin, int& end) {
  const int each = (n + kPAll - 1) / kPAll;
  begin = (int)min((int64_t)plan_thread() * each, (int64_t)n);
  end = min(begin + each, n);
}

__device__ __forceinline__ int count_free(const int32_t* refs, int begin, int end) {
  int n = 0;
#pragma unroll 4
  for (int p = begin; p < end; ++p) n += refs[p] <= 0;
  return n;
}

// the free pages of ranks below `wanted` into list
__device__ __forceinline__ void list_free(const int32_t* refs, int begin, int end, int rank, int wanted, int32_t* list) {
  if (rank >= wanted) return;
  for (int p = begin; p < end && rank < wanted; ++p)
    if (refs[p] <= 0) list[rank++] = p;
}

// ---------------------------------------------------------------- extend
// The pages that a sequence lacks, [held, need): its held pages come first, so a
// row that lacks none shows it at its last needed place, others are bisected.
__device__ __forceinline__ void lacking(const PagePlanArgs& a, int b, int& held, int& need) {
  const int page = 1 << a.page_log, len = max(a.lengths[b], 0);
  need = (int)(((int64_t)len + page - 1) >> a.page_log);
  if (need > a.M) {
    atomicAdd(a.bad, 1);                        // once: the missing places of many could add up to 0
    need = a.M;
  }
  const int32_t* row = a.tables + (int64_t)b * a.M;
  held = need;
  if (need == 0 || row[need - 1] >= 0) return;
  int lo = 0, hi = need - 1;                    // row[lo - 1] >= 0, row[hi] < 0
  if (hi > 0 && row[hi - 1] >= 0) lo = hi;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (row[mid] < 0) hi = mid;
    else lo = mid + 1;
  }
  held = lo;
}

__global__ void __launch_bounds__(kPThreads) pages_extend_kernel(const __grid_constant__ PagePlanArgs a) {
  __shared__ PlanShared sm;
  ptx::cluster_arrive();
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  int p0, p1, b0, b1;
  share_of(a.P, p0, p1);
  share_of(a.B, b0, b1);
  int want = 0, held = 0, need = 0;
  for (int b = b0; b < b1; ++b) {
    lacking(a, b, held, need);
    want += need - held;
  }
  __syncwarp();
  ptx::cluster_wait();
  int2 before, total;
  cluster_ranks(sm, make_int2(count_free(a.refs, p0, p1), want), before, total);
  if (total.y == 0) return;                     // the same for the whole cluster
  list_free(a.refs, p0, p1, before.x, total.y, a.list_dst);
  cg::this_cluster().sync();
  // a warp serves its 32 threads' sequences one after another
  const int lane = threadIdx.x & 31;
  int rank = before.y;
  const int most = (a.B + kPAll - 1) / kPAll;
  for (int i = 0; i < most; ++i) {
    const int b = b0 + i;
    if (most > 1 || want == 0) held = need = 0;
    if (most > 1 && b < b1) lacking(a, b, held, need);
    for (unsigned todo = __ballot_sync(~0u, need > held); todo; todo &= todo - 1) {
      const int l = __ffs(todo) - 1;
      const int sb = __shfl_sync(~0u, b, l), sh = __shfl_sync(~0u, held, l), sn = __shfl_sync(~0u, need, l);
      const int sr = __shfl_sync(~0u, rank, l);
      for (int j = sh + lane; j < sn; j += 32) {
        const int r = sr + j - sh;
        int32_t* at = a.tables + (int64_t)sb * a.M + j;
        if (r >= total.x) atomicAdd(a.bad, 1);
        else if (*at < 0) {
          const int p = a.list_dst[r];
          *at = p;
          a.refs[p] = 1;
        }
      }
    }
    rank += need - held;
  }
}

// ---------------------------------------------------------------- free
__global__ void __launch_bounds__(kCThreads)
pages_free_kernel(const __grid_constant__ PagePlanArgs a, const int32_t* seqs) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  const int b = seqs[blockIdx.x];
  if (b < 0 || b >= a.B) {
    if (threadIdx.x == 0) atomicAdd(a.bad, 1);
    return;
  }
  // taken out of the row by an exchange: a sequence that is listed twice
  // gives its pages back once
  for (int j = threadIdx.x; j < a.M; j += kCThreads) {
    int32_t* at = a.tables + (int64_t)b * a.M + j;
    if (*at == -1) continue;
    const int p = atomicExch(at, -1);
    if (p < 0) continue;
    if (p >= a.P) atomicAdd(a.bad, 1);
    else if (atomicSub(a.refs + p, 1) <= 0) {   // held by a table, counted by none
      atomicAdd(a.refs + p, 1);
      atomicAdd(a.bad + 1, 1);
    }
  }
  if (threadIdx.x == 0) a.lengths[b] = 0;
}

// ---------------------------------------------------------------- fork
__global__ void __launch_bounds__(kPThreads) pages_fork_kernel(const __grid_constant__ PagePlanArgs a) {
  __shared__ PlanShared sm;
  __shared__ int3 rows[kPThreads];              // source, target, full pages of this CTA's pairs
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  cg::cluster_group cl = cg::this_cluster();
  // thread i serves pair i (n <= kPAll)
  const int i = plan_thread(), lane = threadIdx.x & 31, page = 1 << a.page_log;
  int s = -1, d = -1, len = 0;
  bool ok = false;
  if (i < a.n) {
    s = a.src[i];
    d = a.dst[i];
    ok = s >= 0 && s < a.B && d >= 0 && d < a.B && s != d;
    if (ok) {
      len = max(a.lengths[s], 0);
      ok = ((int64_t)len + page - 1) >> a.page_log <= a.M && a.lengths[d] == 0 && a.tables[(int64_t)d * a.M] < 0;
    }
  }
  cl.sync();                                    // lengths read before any is claimed
  if (ok) atomicMin(a.lengths + d, i - kPAll);  // the first pair of an empty row has it
  cl.sync();
  if (ok) ok = atomicAdd(a.lengths + d, 0) == i - kPAll;
  if (i < a.n && !ok) atomicAdd(a.bad, 1);
  const int full = ok ? len >> a.page_log : 0;
  int last = -1;
  if (ok && (len & (page - 1))) {
    last = a.tables[(int64_t)s * a.M + full];
    if (last < 0 || last >= a.P) {
      atomicAdd(a.bad, 1);
      last = -2;                                // the source lacks the page: so does the copy
    }
  }
  int p0, p1;
  share_of(a.P, p0, p1);
  int2 before, total;
  cluster_ranks(sm, make_int2(count_free(a.refs, p0, p1), last >= 0), before, total);
  list_free(a.refs, p0, p1, before.x, total.y, a.list_dst);
  cl.sync();
  int fresh = -1;
  if (last >= 0) {
    if (before.y < total.x) {
      fresh = a.list_dst[before.y];
      a.list_src[before.y] = last;
      a.refs[fresh] = 1;
    } else {                                    // no page is left: the row stays empty
      atomicAdd(a.bad, 1);
      ok = false;
    }
  }
  if (i == 0) *a.count = min(total.x, total.y);
  rows[threadIdx.x] = make_int3(s, d, ok ? full : 0);
  cl.sync();                                    // every claim has been read, every row is known
  if (d >= 0 && d < a.B && i < a.n) {
    if (ok) {
      a.lengths[d] = len;
      if (fresh >= 0) a.tables[(int64_t)d * a.M + full] = fresh;
    } else if (last >= 0) {
      a.lengths[d] = 0;
    }
  }
  // the shared pages: pair after pair over all warps of the cluster
  for (int k = i >> 5; k < a.n; k += kPAll / 32) {
    const int3 r = cl.map_shared_rank(rows, k / kPThreads)[k % kPThreads];
    for (int j = lane; j < r.z; j += 32) {
      const int p = a.tables[(int64_t)r.x * a.M + j];
      if (p < 0 || p >= a.P) {
        atomicAdd(a.bad, 1);
        continue;
      }
      a.tables[(int64_t)r.y * a.M + j] = p;
      atomicAdd(a.refs + p, 1);
    }
  }
  cl.sync();                                    // nobody leaves while its rows are read
}

// ---------------------------------------------------------------- compact
// n live pages; the k-th highest of those at n or above goes to the k-th lowest
// hole below n.  Refs may be rewritten in place: holes read the counts of pages
// at n or above, which are cleared after everyone has read them.
__global__ void __launch_bounds__(kPThreads) pages_compact_kernel(const __grid_constant__ PagePlanArgs a) {
  __shared__ PlanShared sm;
  ptx::cluster_arrive();
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  cg::cluster_group cl = cg::this_cluster();
  int p0, p1;
  share_of(a.P, p0, p1);
  const int live = p1 - p0 - count_free(a.refs, p0, p1);
  __syncwarp();
  ptx::cluster_wait();
  int2 before, total;
  cluster_ranks(sm, make_int2(live, 0), before, total);
  const int n = total.x;
  int rank = before.x;                          // live pages before p
  for (int p = p0; p < p1; ++p) {
    const bool used = a.refs[p] > 0;
    if (used && p >= n) a.list_src[n - 1 - rank] = p;
    if (!used && p < n) a.list_dst[p - rank] = p;
    if (!used || p < n) a.names[p] = used ? p : -1;
    rank += used;
  }
  cl.sync();
  rank = before.x;
  for (int p = p0; p < min(p1, n); ++p) {
    const int r = a.refs[p];
    if (r > 0) {
      a.out_refs[p] = r;
      ++rank;
    } else {
      const int from = a.list_src[p - rank];
      a.names[from] = p;
      a.out_refs[p] = a.refs[from];
    }
  }
  if (p0 <= n && n < p1) *a.count = n - rank;   // holes below n
  if (plan_thread() == 0) {
    if (n == a.P) *a.count = 0;
    if (a.n_live) *a.n_live = n;
  }
  cl.sync();
  for (int p = max(p0, n); p < p1; ++p) a.out_refs[p] = 0;
}

// ---------------------------------------------------------------- copy
// A warp moves 4 KB of one page of one layer at a time, eight 16-byte loads in
// flight a lane.
__global__ void __launch_bounds__(kCThreads) page_copy_kernel(const __grid_constant__ PageCopyArgs a) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch_dependents();
  const int lane = threadIdx.x & 31;
  if (a.names) {
    for (int64_t i = (int64_t)blockIdx.x * kCThreads + threadIdx.x; i < a.entries; i += (int64_t)gridDim.x * kCThreads) {
      const int p = a.tables[i];
      int q = p;
      if (p >= 0) {
        if (p < a.P) q = a.names[p];
        if (p >= a.P || q < 0) atomicAdd(a.bad, 1);   // no page, or one that nobody counts
      }
      a.out_tables[i] = q;
    }
  }
  const int n = a.count ? *a.count : a.n;
  const int64_t pieces = (a.page_bytes + 4095) >> 12;
  const int64_t units = pieces * a.layers * n;
  const int64_t warps = (int64_t)gridDim.x * (kCThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kCThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
    const int64_t rest = u / pieces;
    const int64_t at = (u - rest * pieces) << 12;
    const int k = (int)(rest / a.layers), l = (int)(rest - (int64_t)k * a.layers);
    const int s = a.src[k], d = a.dst[k];
    if (s < 0 || s >= a.P || d < 0 || d >= a.P) {
      if (at == 0 && l == 0 && lane == 0) atomicAdd(a.bad, 1);
      continue;
    }
    if (s == d) continue;
    const int64_t base = (int64_t)l * a.P;
    const uint8_t* from = a.cache + (base + s) * a.page_bytes + at;
    uint8_t* to = a.cache + (base + d) * a.page_bytes + at;
    const int64_t left = a.page_bytes - at;
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (16 * (lane + 32 * i) < left) v[i] = *reinterpret_cast<const uint4*>(from + 16 * (lane + 32 * i));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (16 * (lane + 32 * i) < left) *reinterpret_cast<uint4*>(to + 16 * (lane + 32 * i)) = v[i];
    if (at == 0)
      for (int i = lane; i < a.scales; i += 32) a.scale[(base + d) * a.scales + i] = a.scale[(base + s) * a.scales + i];
  }
}

template <typename F>
cudaError_t plan_launch(F kernel, const PagePlanArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanCtas, 1, 1);
  cfg.blockDim = dim3(kPThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[2] = {pdl_attribute()};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kPlanCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return counted_launch(cudaLaunchKernelEx(&cfg, kernel, a));
}

}  // namespace

cudaError_t launch_pages_extend(const PagePlanArgs& a, cudaStream_t st) {
  return plan_launch(pages_extend_kernel, a, st);
}
cudaError_t launch_pages_fork(const PagePlanArgs& a, cudaStream_t st) {
  return plan_launch(pages_fork_kernel, a, st);
}
cudaError_t launch_pages_compact(const PagePlanArgs& a, cudaStream_t st) {
  return plan_launch(pages_compact_kernel, a, st);
}

cudaError_t launch_pages_free(const PagePlanArgs& a, const int32_t* seqs, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.n, 1, 1);
  cfg.blockDim = dim3(kCThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return counted_launch(cudaLaunchKernelEx(&cfg, pages_free_kernel, a, seqs));
}

cudaError_t launch_page_copy(const PageCopyArgs& a, cudaStream_t st) {
  const int64_t pieces = (a.page_bytes + 4095) >> 12;
  // moves of pages (at most a.n) and table entries; 8 CTAs of 8 warps fill an SM
  const int64_t ctas = max((pieces * a.layers * a.n + 7) / 8, (a.entries + kCThreads - 1) / kCThreads);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)max((int64_t)1, min(ctas, (int64_t)148 * 8)), 1, 1);
  cfg.blockDim = dim3(kCThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return counted_launch(cudaLaunchKernelEx(&cfg, page_copy_kernel, a));
}

}  // namespace lora
