// Launch arguments of the paged 8-bit cache's kernels, between the C ABI
// (cache_api.cu) and the kernel files.  Not part of the public interface.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "lora.h"

namespace lora {

constexpr int kPlanCtas = 8;          // one cluster plans the moves of pages
constexpr int kMaxAttnCtas = 1024;    // CTAs of an attention launch, at most
// rows (queries x heads that share a k/v head) of a tile of the two kernels
constexpr int kFewRows = 16, kManyRows = 256;

// Workspace: header (the error counters of common.cuh), one join counter for
// each attention CTA (0 between calls), the plan of a move (source and
// destination pages, new names, their number), the parts of rows that
// attention CTAs share.
struct CacheWork {
  size_t off_join, off_count, off_src, off_dst, off_name, off_part, total;
  static size_t a256(size_t v) { return (v + 255) & ~size_t(255); }
  static size_t part_floats(int dim);
  CacheWork(int P, int dim) {
    off_join = 256;
    off_count = off_join + a256(sizeof(int) * kMaxAttnCtas);
    off_src = off_count + 256;
    off_dst = off_src + a256(sizeof(int) * (size_t)P);
    off_name = off_dst + a256(sizeof(int) * (size_t)P);
    off_part = off_name + a256(sizeof(int) * (size_t)P);
    total = off_part + a256(sizeof(float) * part_floats(dim));
  }
};

struct CacheWriteArgs {
  const void *k, *v;
  int64_t ldk, ldv;
  uint8_t* cache;
  float* scale;
  const int32_t *tables, *lengths, *starts;   // starts null: one row for each sequence
  int* bad;                                   // the header's counters
  int T, B, Hk, dim, page_log, P, M;
};

struct AttnArgs {
  const void* q;
  int64_t ldq;
  void* y;
  int64_t ldy;
  const uint8_t* cache;
  const float* scale;
  const int32_t *tables, *lengths, *starts;   // starts null: one row for each sequence
  int* bad;
  int* join;
  float* part;
  int T, B, Hk, group, dim, page_log, P, M, window;
  int min_rows, max_rows;                     // sequences of other numbers of rows are left out
  float c;                                    // softmax scale * log2 e
};

struct PageCopyArgs {
  uint8_t* cache;
  float* scale;
  const int32_t *src, *dst;
  const int* count;                           // null: n pairs
  int n, layers, P, scales;                   // scales: of a page of a layer
  int64_t page_bytes;
  int* bad;
  // compaction: names of the pages after the move, and the tables they go into
  const int32_t* names;
  const int32_t* tables;
  int32_t* out_tables;
  int64_t entries;
};

struct PagePlanArgs {
  int32_t* tables;
  int32_t* lengths;
  int32_t* refs;
  const int32_t *src, *dst;                   // fork: pairs of sequences
  int32_t *out_refs, *n_live;                 // compaction
  int32_t *list_src, *list_dst, *names, *count;
  int* bad;
  int n, B, M, P, page_log;
};

cudaError_t launch_cache_write(lora_dtype dt, const CacheWriteArgs& a, cudaStream_t st);
cudaError_t launch_attention_few(lora_dtype dt, const AttnArgs& a, cudaStream_t st);
cudaError_t launch_attention_many(lora_dtype dt, const AttnArgs& a, cudaStream_t st);
cudaError_t launch_page_copy(const PageCopyArgs& a, cudaStream_t st);
cudaError_t launch_pages_extend(const PagePlanArgs& a, cudaStream_t st);
cudaError_t launch_pages_fork(const PagePlanArgs& a, cudaStream_t st);
cudaError_t launch_pages_compact(const PagePlanArgs& a, cudaStream_t st);
cudaError_t launch_pages_free(const PagePlanArgs& a, const int32_t* seqs, cudaStream_t st);

}  // namespace lora
