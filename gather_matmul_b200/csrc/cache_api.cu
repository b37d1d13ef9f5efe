// extern "C" entry points of the paged 8-bit key/value cache: host-side
// argument checks and dispatch.  See include/lora.h for the contract of each call.
#include <limits.h>

#include "cache.h"
#include "common.cuh"
#include "internal.h"

using namespace lora;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

lora_status from_cuda(cudaError_t e) { return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA; }

int log2_of(int page) {
  switch (page) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
  }
  return -1;
}

// shape of a cache of one layer
lora_status check_cache(int pages, int kv_heads, int page_tokens, int dim) {
  if (pages <= 0 || kv_heads <= 0 || page_tokens <= 0 || dim <= 0) return LORA_ERR_INVALID_ARG;
  if (pages > LORA_MAX_PAGES || kv_heads > LORA_MAX_HEADS || log2_of(page_tokens) < 0 ||
      dim > LORA_MAX_HEAD_DIM || dim % 16 != 0)
    return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

// tables of n sequences of up to m pages; ranks of places are 32-bit numbers
lora_status check_seqs(int n, int m) {
  if (n < 0 || m <= 0) return LORA_ERR_INVALID_ARG;
  if (n > LORA_MAX_SEQS || (int64_t)m * 128 > INT_MAX / 2 || (int64_t)n * m > INT_MAX)
    return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

lora_status check_ptr(const void* p, uintptr_t align) {
  if (p == nullptr) return LORA_ERR_INVALID_ARG;
  return aligned(p, align) ? LORA_OK : LORA_ERR_MISALIGNED;
}

lora_status check_all(const void* const* p, int n, uintptr_t align) {
  for (int i = 0; i < n; ++i) {
    const lora_status s = check_ptr(p[i], align);
    if (s != LORA_OK) return s;
  }
  return LORA_OK;
}

lora_status check_rows(const void* p, int64_t ld, int64_t width) {
  if (p == nullptr || ld < width) return LORA_ERR_INVALID_ARG;
  if (ld > (int64_t)1 << 38) return LORA_ERR_UNSUPPORTED;
  if (!aligned(p, 16) || ld % 8 != 0) return LORA_ERR_MISALIGNED;
  return LORA_OK;
}

lora_status check_work(const void* work, size_t bytes, size_t need) {
  if (work == nullptr || bytes < need) return LORA_ERR_INVALID_ARG;
  return aligned(work, 256) ? LORA_OK : LORA_ERR_MISALIGNED;
}

template <typename T>
T* at(void* work, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(work) + off); }

#define TRY(expr)                            \
  do {                                       \
    const lora_status s_ = (expr);           \
    if (s_ != LORA_OK) return s_;            \
  } while (0)

}  // namespace

extern "C" {

size_t lora_cache_workspace_bytes(int n_pages, int head_dim) {
  if (check_cache(n_pages, 1, 16, head_dim) != LORA_OK) return 0;
  return CacheWork(n_pages, head_dim).total;
}

lora_status lora_cache_write(lora_dtype dtype, int T, int n_seqs, int kv_heads, int head_dim,
                             int page_tokens, int n_pages, int max_pages, const void* k,
                             int64_t ldk, const void* v, int64_t ldv, void* cache, float* scale,
                             const int32_t* tables, const int32_t* lengths, const int32_t* starts,
                             void* work, size_t work_bytes, lora_stream_t stream) {
  if ((dtype != LORA_F16 && dtype != LORA_BF16) || T < 0) return LORA_ERR_INVALID_ARG;
  TRY(check_cache(n_pages, kv_heads, page_tokens, head_dim));
  TRY(check_seqs(n_seqs, max_pages));
  if (T > LORA_MAX_TOKENS) return LORA_ERR_UNSUPPORTED;
  if (starts == nullptr && T != n_seqs) return LORA_ERR_INVALID_ARG;
  TRY(check_work(work, work_bytes, CacheWork(n_pages, head_dim).total));
  if (T == 0 || n_seqs == 0) return LORA_OK;
  const int64_t width = (int64_t)kv_heads * head_dim;
  TRY(check_rows(k, ldk, width));
  TRY(check_rows(v, ldv, width));
  TRY(check_ptr(cache, 16));
  const void* ints[4] = {scale, tables, lengths, starts ? starts : lengths};
  TRY(check_all(ints, 4, 4));
  CacheWriteArgs a = {};
  a.k = k;
  a.v = v;
  a.ldk = ldk;
  a.ldv = ldv;
  a.cache = static_cast<uint8_t*>(cache);
  a.scale = scale;
  a.tables = tables;
  a.lengths = lengths;
  a.starts = starts;
  a.bad = at<int>(work, 0);
  a.T = T;
  a.B = n_seqs;
  a.Hk = kv_heads;
  a.dim = head_dim;
  a.page_log = log2_of(page_tokens);
  a.P = n_pages;
  a.M = max_pages;
  // eight warps of 16 tokens of a head in a CTA: the grid's limit
  const int64_t slots = starts ? (int64_t)(T >> a.page_log) + 2 * (int64_t)n_seqs : n_seqs;
  if (((slots * 2 * kv_heads) << (a.page_log - 4)) / 8 >= INT_MAX) return LORA_ERR_UNSUPPORTED;
  cudaGetLastError();
  return from_cuda(launch_cache_write(dtype, a, (cudaStream_t)stream));
}

lora_status lora_cache_attention(lora_dtype dtype, int T, int n_seqs, int q_heads, int kv_heads,
                                 int head_dim, int page_tokens, int n_pages, int max_pages,
                                 const void* q, int64_t ldq, const void* cache,
                                 const float* scale, const int32_t* tables,
                                 const int32_t* lengths, const int32_t* starts,
                                 float softmax_scale, int window, void* y, int64_t ldy, void* work,
                                 size_t work_bytes, lora_stream_t stream) {
  if ((dtype != LORA_F16 && dtype != LORA_BF16) || T < 0 || q_heads <= 0 || window < 0)
    return LORA_ERR_INVALID_ARG;
  // its product with log2 e is a number too
  if (!(softmax_scale > 0.f && softmax_scale < 0x1p127f)) return LORA_ERR_INVALID_ARG;
  TRY(check_cache(n_pages, kv_heads, page_tokens, head_dim));
  TRY(check_seqs(n_seqs, max_pages));
  if (q_heads > LORA_MAX_HEADS || T > LORA_MAX_TOKENS || (int64_t)T * q_heads > INT_MAX / 2)
    return LORA_ERR_UNSUPPORTED;
  if (q_heads % kv_heads != 0 || (starts == nullptr && T != n_seqs)) return LORA_ERR_INVALID_ARG;
  const CacheWork L(n_pages, head_dim);
  TRY(check_work(work, work_bytes, L.total));
  if (T == 0 || n_seqs == 0) return LORA_OK;
  const int64_t width = (int64_t)q_heads * head_dim;
  TRY(check_rows(q, ldq, width));
  TRY(check_rows(y, ldy, width));
  TRY(check_ptr(cache, 16));
  const void* ints[4] = {scale, tables, lengths, starts ? starts : lengths};
  TRY(check_all(ints, 4, 4));
  // q is read while other CTAs write y
  const char *q0 = static_cast<const char*>(q), *y0 = static_cast<const char*>(y);
  if (q0 < y0 + 2 * ((T - 1) * ldy + width) && y0 < q0 + 2 * ((T - 1) * ldq + width)) {
    // rows of one matrix may lie side by side
    const int64_t d = ((y0 - q0) % (2 * ldq) + 2 * ldq) % (2 * ldq);
    if (T == 1 || ldq != ldy || d < 2 * width || 2 * ldq - d < 2 * width) return LORA_ERR_INVALID_ARG;
  }
  AttnArgs a = {};
  a.q = q;
  a.ldq = ldq;
  a.y = y;
  a.ldy = ldy;
  a.cache = static_cast<const uint8_t*>(cache);
  a.scale = scale;
  a.tables = tables;
  a.lengths = lengths;
  a.starts = starts;
  a.bad = at<int>(work, 0);
  a.join = at<int>(work, L.off_join);
  a.part = at<float>(work, L.off_part);
  a.T = T;
  a.B = n_seqs;
  a.Hk = kv_heads;
  a.group = q_heads / kv_heads;
  a.dim = head_dim;
  a.page_log = log2_of(page_tokens);
  a.P = n_pages;
  a.M = max_pages;
  a.window = window;
  a.c = (float)((double)softmax_scale * 1.4426950408889634);
  cudaGetLastError();
  // Sequences of up to kFewRows rows and others have kernels of their own; only the device
  // knows them where starts is given.  The kernel for many rows takes all, slower for few
  // (at half the speed where there is much to read); a second launch costs up to 20 us, most
  // of it the kernel's way to its first products.  Items (sequences x k/v heads) are what
  // the host knows:
  //   up to 128, one for each CTA at most: one kernel.  12 sequences of up to 8 tokens over
  //     12 000 on 4 heads 43 us, in two kernels 75; 16 of up to 200 over 2000 38 and 60; 16
  //     of up to 8 over 16 000 on 8 heads 66 and 91.  It loses where all have one or two
  //     tokens: 16 over 16 000 on 8 heads 66 and 56, 8 over 30 000 51 and 42, 4 over 2000
  //     21 and 24; 128 over 8000 on 1 head 53 and 56; 36 of up to 4 over 30 000 on 4 heads
  //     (144 items) 99 and 91
  //   up to 8 for each CTA: one, unless the rows say that most sequences are short.  64 of
  //     up to 200 over 8000 94 us and 122; 64 of up to 4 over 8000 66 and 61
  //   more: two.  300 of up to 16 over 8000 on 8 heads 326 us and 305; 150 of up to 64
  //     (1200 items) 218 and 220
  const int64_t rows = starts ? (int64_t)T * a.group : a.group, items = (int64_t)n_seqs * kv_heads;
  const bool one = !starts || items <= 128 || (items <= 8 * 148 && rows > (int64_t)kFewRows * n_seqs);
  const bool many = rows > kFewRows, few = !many || !one;
  cudaError_t e = cudaSuccess;
  if (many) {
    a.min_rows = few ? kFewRows + 1 : 1;
    a.max_rows = INT_MAX;
    e = launch_attention_many(dtype, a, (cudaStream_t)stream);
  }
  if (few && e == cudaSuccess) {
    a.min_rows = 1;
    a.max_rows = kFewRows;
    e = launch_attention_few(dtype, a, (cudaStream_t)stream);
  }
  return from_cuda(e);
}

static lora_status plan_args(PagePlanArgs& a, int n_seqs, int max_pages, int page_tokens, int n_pages, void* work,
                             size_t work_bytes) {
  TRY(check_cache(n_pages, 1, page_tokens, 16));
  TRY(check_seqs(n_seqs, max_pages));
  // the least of the workspaces of that many pages holds the plan
  TRY(check_work(work, work_bytes, CacheWork(n_pages, 16).total));
  const CacheWork L(n_pages, 16);
  a.list_src = at<int32_t>(work, L.off_src);
  a.list_dst = at<int32_t>(work, L.off_dst);
  a.names = at<int32_t>(work, L.off_name);
  a.count = at<int32_t>(work, L.off_count);
  a.bad = at<int>(work, 0);
  a.B = n_seqs;
  a.M = max_pages;
  a.P = n_pages;
  a.page_log = log2_of(page_tokens);
  return LORA_OK;
}

static lora_status copy_args(PageCopyArgs& c, int layers, int n_pages, int kv_heads, int page_tokens, int head_dim,
                             void* cache, float* scale, int* bad) {
  TRY(check_cache(n_pages, kv_heads, page_tokens, head_dim));
  if (layers <= 0) return LORA_ERR_INVALID_ARG;
  TRY(check_ptr(cache, 16));
  TRY(check_ptr(scale, 4));
  c.cache = static_cast<uint8_t*>(cache);
  c.scale = scale;
  c.layers = layers;
  c.P = n_pages;
  c.scales = 2 * kv_heads;
  c.page_bytes = (int64_t)2 * kv_heads * page_tokens * head_dim;
  c.bad = bad;
  return LORA_OK;
}

lora_status lora_pages_extend(int n_seqs, int max_pages, int page_tokens, int n_pages,
                              int32_t* tables, const int32_t* lengths, int32_t* refs, void* work,
                              size_t work_bytes, lora_stream_t stream) {
  PagePlanArgs a = {};
  TRY(plan_args(a, n_seqs, max_pages, page_tokens, n_pages, work, work_bytes));
  if (n_seqs == 0) return LORA_OK;
  const void* ints[3] = {tables, lengths, refs};
  TRY(check_all(ints, 3, 4));
  a.tables = tables;
  a.lengths = const_cast<int32_t*>(lengths);
  a.refs = refs;
  cudaGetLastError();
  return from_cuda(launch_pages_extend(a, (cudaStream_t)stream));
}

lora_status lora_pages_free(int n_seqs, int max_pages, int n_pages, int32_t* tables,
                            int32_t* lengths, int32_t* refs, const int32_t* seqs, int n,
                            void* work, size_t work_bytes, lora_stream_t stream) {
  PagePlanArgs a = {};
  TRY(plan_args(a, n_seqs, max_pages, 16, n_pages, work, work_bytes));
  if (n < 0) return LORA_ERR_INVALID_ARG;
  if (n > LORA_MAX_SEQS) return LORA_ERR_UNSUPPORTED;
  if (n == 0) return LORA_OK;
  const void* ints[4] = {tables, lengths, refs, seqs};
  TRY(check_all(ints, 4, 4));
  a.tables = tables;
  a.lengths = lengths;
  a.refs = refs;
  a.n = n;
  cudaGetLastError();
  return from_cuda(launch_pages_free(a, seqs, (cudaStream_t)stream));
}

lora_status lora_pages_fork(int n_seqs, int max_pages, int layers, int kv_heads, int head_dim,
                            int page_tokens, int n_pages, int32_t* tables, int32_t* lengths,
                            int32_t* refs, const int32_t* src, const int32_t* dst, int n,
                            void* cache, float* scale, void* work, size_t work_bytes,
                            lora_stream_t stream) {
  PagePlanArgs a = {};
  TRY(plan_args(a, n_seqs, max_pages, page_tokens, n_pages, work, work_bytes));
  PageCopyArgs c = {};
  TRY(copy_args(c, layers, n_pages, kv_heads, page_tokens, head_dim, cache, scale, a.bad));
  if (n < 0) return LORA_ERR_INVALID_ARG;
  if (n > LORA_MAX_FORKS) return LORA_ERR_UNSUPPORTED;
  if (n == 0) return LORA_OK;
  const void* ints[5] = {tables, lengths, refs, src, dst};
  TRY(check_all(ints, 5, 4));
  a.tables = tables;
  a.lengths = lengths;
  a.refs = refs;
  a.src = src;
  a.dst = dst;
  a.n = n;
  c.src = a.list_src;
  c.dst = a.list_dst;
  c.count = a.count;
  c.n = n;
  cudaGetLastError();
  cudaError_t e = launch_pages_fork(a, (cudaStream_t)stream);
  if (e == cudaSuccess) e = launch_page_copy(c, (cudaStream_t)stream);
  return from_cuda(e);
}

lora_status lora_pages_compact(int n_seqs, int max_pages, int layers, int kv_heads, int head_dim,
                               int page_tokens, int n_pages, const int32_t* tables,
                               const int32_t* refs, int32_t* out_tables, int32_t* out_refs,
                               int32_t* n_live, void* cache, float* scale, void* work,
                               size_t work_bytes, lora_stream_t stream) {
  PagePlanArgs a = {};
  TRY(plan_args(a, n_seqs, max_pages, page_tokens, n_pages, work, work_bytes));
  PageCopyArgs c = {};
  TRY(copy_args(c, layers, n_pages, kv_heads, page_tokens, head_dim, cache, scale, a.bad));
  const void* ints[5] = {refs, out_refs, n_seqs ? tables : refs, n_seqs ? out_tables : refs, n_live ? n_live : refs};
  TRY(check_all(ints, 5, 4));
  a.refs = const_cast<int32_t*>(refs);
  a.out_refs = out_refs;
  a.n_live = n_live;
  c.src = a.list_src;
  c.dst = a.list_dst;
  c.count = a.count;
  c.n = n_pages / 2;                      // a move needs a live page and a hole
  c.names = a.names;
  c.tables = tables;
  c.out_tables = out_tables;
  c.entries = (int64_t)n_seqs * max_pages;
  cudaGetLastError();
  cudaError_t e = launch_pages_compact(a, (cudaStream_t)stream);
  if (e == cudaSuccess) e = launch_page_copy(c, (cudaStream_t)stream);
  return from_cuda(e);
}

lora_status lora_pages_copy(int layers, int kv_heads, int head_dim, int page_tokens, int n_pages,
                            void* cache, float* scale, const int32_t* src, const int32_t* dst,
                            int n, void* work, size_t work_bytes, lora_stream_t stream) {
  TRY(check_cache(n_pages, kv_heads, page_tokens, head_dim));
  TRY(check_work(work, work_bytes, CacheWork(n_pages, 16).total));
  if (n < 0) return LORA_ERR_INVALID_ARG;
  if (n > LORA_MAX_PAGES) return LORA_ERR_UNSUPPORTED;
  PageCopyArgs c = {};
  TRY(copy_args(c, layers, n_pages, kv_heads, page_tokens, head_dim, cache, scale, at<int>(work, 0)));
  if (n == 0) return LORA_OK;
  TRY(check_ptr(src, 4));
  TRY(check_ptr(dst, 4));
  c.src = src;
  c.dst = dst;
  c.n = n;
  cudaGetLastError();
  return from_cuda(launch_page_copy(c, (cudaStream_t)stream));
}

}  // extern "C"
