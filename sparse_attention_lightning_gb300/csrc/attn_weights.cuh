// Accumulated attention weight: what its kernels and its host code share.
#pragma once

#include "cache_ops.cuh"

namespace dsa {

struct WeightArgs {
  Seqs seqs;
  int h, d, top_k, kv_dtype, max_q_len;
  float scale_log2;     // softmax scale · log2(e)
  const void* q;
  const void* kv;
  const int32_t* idx;
  const float* lse;
  float* acc;           // [B, ld_acc]
  int64_t ld_acc;
  long long* fx;        // [B, max_k_len] fixed-point sums, or null (one query a sequence at most)
  double fx_scale;      // fx counts units of 1 / fx_scale (a power of two)
  uint32_t* status;
};

// Add the weight w (a sum of probabilities over the heads) to position pos of sequence b.
__device__ __forceinline__ void add_weight(const WeightArgs& a, int b, int pos, float w) {
  if (!dsa_check(pos >= 0 && pos < a.seqs.max_k_len && b >= 0 && b < a.seqs.B, a.status)) return;
  float* acc = a.acc + (int64_t)b * a.ld_acc + pos;
  if (!a.fx) {
    atomicAdd(acc, w);
  } else if (w <= 2.f * a.h) {
    // w is at most h (probabilities; the factor 2 covers their rounding), and fx_scale leaves
    // room for max_q_len such sums (a query's repeated entries share its h); rounded to half a unit, which a weight of
    // 2^-20 of a head still has 22 bits above at 128 heads x 4096 queries
    atomicAdd(reinterpret_cast<unsigned long long*>(a.fx + (int64_t)b * a.seqs.max_k_len + pos),
              (unsigned long long)__double2ll_rn((double)w * a.fx_scale));
  } else {
    atomicAdd(acc, w);  // infinite, NaN, or an lse that is not the attention's
  }
}

// tcgen05 path (bf16, 64 <= D <= 576, up to 128 heads).
bool attn_weights_tc_eligible(const WeightArgs& a);
int launch_attn_weights_tc(const WeightArgs& a, cudaStream_t stream);

int launch_attn_weights(const WeightArgs& a, cudaStream_t stream);

}  // namespace dsa
