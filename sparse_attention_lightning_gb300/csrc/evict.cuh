// Cache eviction: what its kernels and its host code share.
#pragma once

#include "cache_ops.cuh"

namespace dsa {

struct EvictArgs {
  Seqs seqs;
  const float* acc;      // [B, ld_acc]
  int64_t ld_acc;
  int budget, sink, recent;
  int32_t* kept;         // [B, budget]
  int32_t* cu_k_out;     // [B + 1]
  float* acc_out;        // [B, ld_acc_out] or null
  int64_t ld_acc_out;
  const void* src[3];    // kv, k_idx, k_scale
  void* dst[3];
  int row_bytes[3];      // 0: not moved
  const int32_t* table_out;  // [B, max_pages_out], or null: packed destination rows
  int max_pages_out, num_pages_out;
  int64_t rows_out;
  uint32_t* status;
  bool moves;            // there is something to move (set by launch_evict)
};

int launch_evict(EvictArgs a, cudaStream_t stream);

}  // namespace dsa
