// Shared-prefix attention: what its kernels and its host code share.
#pragma once

#include "cache_ops.cuh"

namespace dsa {

struct PrefixArgs {
  Seqs seqs;
  int max_q_len, h, d_c, d_rope, kv_dtype, out_dtype;
  float scale_log2;            // softmax scale · log2(e)
  int prefix_len;              // P
  const void* prefix_kv;       // [P, D], or null: prefix rows through prefix_table
  const int32_t* prefix_table; // [ceil(P / page_size)] pages of the prefix
  const void* q;
  const void* kv;
  void* out;
  float* lse;
  uint32_t* status;
  int splits;                  // pieces a row's keys are cut into
  float* part_o;               // [pieces][total_q · h][d_c] unnormalised partial outputs
  float2* part_ml;             // [pieces][total_q · h] (max in log2 units, sum); sum 0: no keys
};

struct SeqInfo {
  int b, q0, T, k0, L;
};

// Sequence b's rows; false (and flagged) when cu_q/cu_k are inconsistent with the descriptor.
__device__ __forceinline__ bool prefix_seq(const PrefixArgs& a, int b, SeqInfo& i) {
  const Seqs& s = a.seqs;
  const int q0 = s.cu_q[b], q1 = s.cu_q[b + 1];
  const int k0 = s.cu_k[b], k1 = s.cu_k[b + 1];
  i = SeqInfo{b, q0, q1 - q0, k0, k1 - k0};
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= s.total_q && k0 >= 0 && k1 >= k0 &&
                  k1 <= s.total_k && i.T <= i.L && i.L <= s.max_k_len && i.T <= a.max_q_len;
  if (!ok) atomicOr(a.status, DSA_FLAG_BAD_SEQS);
  return ok;
}

// The key at position x of [prefix | suffix of sequence b]; null when its page is outside the cache.
__device__ __forceinline__ const void* prefix_key(const PrefixArgs& a, int b, int k0, int x) {
  const int64_t bytes = (int64_t)(a.d_c + a.d_rope) * (a.kv_dtype == DSA_BF16 ? 2 : 4);
  int64_t row;
  const char* base = static_cast<const char*>(a.kv);
  if (x >= a.prefix_len) {
    row = cache_row(a.seqs, b, k0, x - a.prefix_len);
  } else if (a.prefix_kv) {
    base = static_cast<const char*>(a.prefix_kv);
    row = x;
  } else {
    const int sh = __ffs(a.seqs.page_size) - 1;
    const int pg = a.prefix_table[x >> sh];
    row = (unsigned)pg < (unsigned)a.seqs.num_pages
              ? ((int64_t)pg << sh) | (x & (a.seqs.page_size - 1)) : -1;
  }
  return row < 0 ? nullptr : base + row * bytes;
}

// Which pieces of part_o and part_ml a row has.
constexpr int kMaxLines = 192;
struct PrefixMerge {
  int pieces;        // of every row (table = 0); otherwise the number of piece slots
  int table = 0;     // pieces go by line: the block of 128 rows that attended together
  int fblk, nblk;    // blocks over the prefix alone (0: none; one key axis), blocks of a sequence
  int base;          // slot of a sequence block's first piece
  uint8_t np[kMaxLines];  // pieces of a line, the prefix's blocks first
};

inline int prefix_simt_blocks(int max_q_len, int h) {
  return (int)(((int64_t)max_q_len * h + 15) / 16);
}

// tcgen05 path (bf16, 64 <= D <= 576, d_c <= 512): the most pieces it cuts rows into (the workspace's size).
bool prefix_tc_eligible(const PrefixArgs& a);
int prefix_tc_most_pieces(const PrefixArgs& a);
int launch_prefix_tc(const PrefixArgs& a, cudaStream_t stream);

int launch_prefix_simt(const PrefixArgs& a, cudaStream_t stream);
int launch_prefix_merge(const PrefixArgs& a, const PrefixMerge& m, cudaStream_t stream);

}  // namespace dsa
