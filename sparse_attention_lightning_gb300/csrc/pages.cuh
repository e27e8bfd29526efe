// Pages of a cache, forked, reserved, freed and compacted: what the kernels and the host code share.
#pragma once

#include "cache_ops.cuh"

namespace dsa {

constexpr int kMaxCaches = 8;

struct PageCaches {
  int n;
  char* base[kMaxCaches];
  int64_t row_bytes[kMaxCaches];
  int seg0[kMaxCaches + 1];  // of a page's pieces, the first of each cache (set by the launcher)
};

struct PagesArgs {
  int32_t* table;      // [rows, ld_table]
  int rows, width;
  int64_t ld_table;
  int32_t* refs;       // [num_pages] holders of a page
  int num_pages, page_size;
  int n;               // entries of the call
  const int32_t* src;  // fork
  const int32_t* dst;  // fork: destination rows; free, reserve: the rows
  const int32_t* lens;
  const int32_t* new_lens;
  int32_t* held;       // reserve
  int32_t* moved;      // compact: [num_pages]
  int32_t* live;       // compact: [1]
  PageCaches caches;
  uint32_t* status;
  int32_t* scratch;
};
size_t reserve_scratch_bytes(int rows, int n, int num_pages);
size_t compact_scratch_bytes(int num_pages);
int launch_fork_pages(const PagesArgs& a, cudaStream_t stream);
int launch_free_pages(const PagesArgs& a, cudaStream_t stream);
int launch_reserve_pages(const PagesArgs& a, cudaStream_t stream);
int launch_compact_pages(const PagesArgs& a, cudaStream_t stream);

}  // namespace dsa
