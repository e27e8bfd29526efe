// dsa_accumulate_attn_weights: the attention weight each cached position received, added up
// over heads and queries.
//
//   acc[b, idx[t,i]] += Σ_h exp(scale · q[t,h,:]·kv[row_i,:] − lse[t,h])
//
// A query's weights are probabilities (the lse is the attention's), so the sum needs no running
// max.  One CTA = one query × 16 of its selected positions; the CUDA cores compute in fp32
// (the generic path: any type and width).
//
// Order.  Where no sequence has more than one query, a position receives additions of one value
// only (a repeated index adds the same weight again), so plain fp32 atomics give the same bytes
// in every order.  Otherwise the queries' weights are first added in 64-bit fixed point, whose
// sums do not depend on the order, and then once to acc.
#include "attn_weights.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 16;    // selected positions a CTA takes
constexpr int kHeads = 16;   // heads at a time

// 16 bytes of TK as floats to shared memory (zeros where src is null).
__device__ __forceinline__ void copy16(float* dst, const float* src) {
  const float4 v = src ? __ldg(reinterpret_cast<const float4*>(src)) : make_float4(0.f, 0.f, 0.f, 0.f);
  *reinterpret_cast<float4*>(dst) = v;
}
__device__ __forceinline__ void copy16(float* dst, const __nv_bfloat16* src) {
  const uint4 v = src ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0u, 0u, 0u, 0u);
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<float4*>(dst + 4 * i) =
        make_float4(__uint_as_float(u[2 * i] << 16), __uint_as_float(u[2 * i] & 0xffff0000u),
                    __uint_as_float(u[2 * i + 1] << 16), __uint_as_float(u[2 * i + 1] & 0xffff0000u));
}

// A thread a (head, key) pair, 16 x 16 of them; rows are four floats longer than their columns in shared
// memory, which spreads 16-byte loads over the banks.
template <typename TK>
__global__ void __launch_bounds__(kThreads) attn_weights_simt_kernel(WeightArgs a) {
  extern __shared__ __align__(16) float smem[];
  constexpr int V = 16 / (int)sizeof(TK);
  const int D = a.d, DP = D + 4;
  const int t = blockIdx.x, tid = threadIdx.x;
  float* ks = smem;                  // [kKeys][D + 4]
  float* qs = ks + kKeys * DP;       // [kHeads][D + 4]
  float* red = qs + kHeads * DP;     // [kHeads][kKeys]
  __shared__ int row_s[kKeys];
  RowInfo r;
  if (!query_row_info(a.seqs, t, r, a.status)) return;
  if (__ldg(a.seqs.cu_q + r.b + 1) - __ldg(a.seqs.cu_q + r.b) > a.max_q_len) {
    atomicOr(a.status, DSA_FLAG_BAD_SEQS);  // the order of additions and fx_scale rest on max_q_len
    return;
  }
  const TK* q = static_cast<const TK*>(a.q) + (int64_t)t * a.h * D;
  const TK* kv = static_cast<const TK*>(a.kv);
  const int hh = tid / kKeys, kk = tid % kKeys;
  int pos = -1;  // threads 0..15: their key's position
  if (tid < kKeys) {
    const int i = blockIdx.y * kKeys + tid;
    const int v = i < a.top_k ? a.idx[(int64_t)t * a.top_k + i] : -1;
    int row = -1;
    if (v >= 0 && v <= r.pos) row = key_row(a.seqs, r.b, r.k0, v);
    if (row < 0 && v != -1) atomicOr(a.status, DSA_FLAG_BAD_INDEX);
    if (!dsa_check(row < a.seqs.cache_rows(), a.status)) row = -1;
    pos = row < 0 ? -1 : v;
    row_s[tid] = row;
  }
  if (!__syncthreads_or(pos >= 0)) return;  // padding only
  {
    const int row = row_s[hh];  // 16 threads a key
    for (int i = kk * V; i < D; i += 16 * V)
      copy16(ks + hh * DP + i, row >= 0 ? kv + (int64_t)row * D + i : static_cast<const TK*>(nullptr));
  }
  float w = 0.f;
  for (int h0 = 0; h0 < a.h; h0 += kHeads) {
    __syncthreads();
    const bool head = h0 + hh < a.h;
    for (int i = kk * V; i < D; i += 16 * V)
      copy16(qs + hh * DP + i, head ? q + (int64_t)(h0 + hh) * D + i : static_cast<const TK*>(nullptr));
    const float lse = head ? a.lse[(int64_t)t * a.h + h0 + hh] : -INFINITY;
    __syncthreads();
    float dot = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      const float4 x = *reinterpret_cast<const float4*>(qs + hh * DP + c);
      const float4 y = *reinterpret_cast<const float4*>(ks + kk * DP + c);
      dot = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, dot))));
    }
    // lse = -inf: the attention had no valid entry, so nothing received weight
    if (lse != -INFINITY) w += exp2f(fmaf(dot, a.scale_log2, -lse * kLog2e));
  }
  red[hh * kKeys + kk] = w;
  __syncthreads();
  if (pos >= 0) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < kHeads; ++j) s += red[j * kKeys + tid];
    add_weight(a, r.b, pos, s);
  }
}

// Zero the fixed-point sums.  The kernel that adds to them is set up meanwhile, and gathers its first rows.
__global__ void __launch_bounds__(256) attn_weights_clear_kernel(long long* fx, int64_t n) {
  griddep_launch();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) fx[i] = 0;
}

// acc += the fixed-point sums of the positions a sequence holds.
__global__ void __launch_bounds__(256) attn_weights_finish_kernel(WeightArgs a, int per) {
  griddep_wait();
  const int b = blockIdx.x / per, j = blockIdx.x - b * per;
  const int L = min(__ldg(a.seqs.cu_k + b + 1) - __ldg(a.seqs.cu_k + b), a.seqs.max_k_len);
  const float unit = (float)(1.0 / a.fx_scale);
  for (int s = j * 256 + threadIdx.x; s < L; s += per * 256) {
    const long long v = a.fx[(int64_t)b * a.seqs.max_k_len + s];
    if (v) a.acc[(int64_t)b * a.ld_acc + s] += (float)v * unit;
  }
}

template <typename TK>
int launch_typed(const WeightArgs& a, cudaStream_t stream) {
  auto bytes = [](int D) constexpr { return (int)sizeof(float) * ((kKeys + kHeads) * (D + 4) + kHeads * kKeys); };
  const int smem = bytes(a.d);
  auto kern = attn_weights_simt_kernel<TK>;
  static std::atomic<bool> allowed[64];
  const int rc = allow_smem<bytes(kMaxWidth)>(kern, allowed, "attn_weights_simt: smem attribute");
  if (rc != DSA_OK) return rc;
  dim3 grid((unsigned)a.seqs.total_q, (unsigned)((a.top_k + kKeys - 1) / kKeys));
  DSA_LAUNCH("attn_weights_simt", stream, kern<<<grid, kThreads, smem, stream>>>(a));
  return check_launch("attn_weights_simt");
}

}  // namespace

int launch_attn_weights_simt(const WeightArgs& a, cudaStream_t stream) {
  return a.kv_dtype == DSA_F32 ? launch_typed<float>(a, stream)
                               : launch_typed<__nv_bfloat16>(a, stream);
}

int launch_attn_weights(const WeightArgs& a, cudaStream_t stream) {
  if (a.fx) {
    const int64_t n = (int64_t)a.seqs.B * a.seqs.max_k_len, blocks = (n + 1023) / 1024;
    const unsigned grid = (unsigned)(blocks < 1 ? 1 : blocks < 4 * num_sms() ? blocks : 4 * num_sms());
    DSA_LAUNCH("attn_weights_clear", stream, attn_weights_clear_kernel<<<grid, 256, 0, stream>>>(a.fx, n));
    const int rc = check_launch("attn_weights_clear");
    if (rc != DSA_OK) return rc;
  }
  const int rc = attn_weights_tc_eligible(a) ? launch_attn_weights_tc(a, stream)
                                             : launch_attn_weights_simt(a, stream);
  if (rc != DSA_OK || !a.fx) return rc;
  const int64_t want = (a.seqs.max_k_len + 1023) / 1024, most = 0x7fffffff / a.seqs.B;
  const int per = (int)(want < 64 ? (want < most ? want : most) : (64 < most ? 64 : most));
  cudaError_t e = cudaSuccess;
  DSA_LAUNCH("attn_weights_finish", stream,
             e = launch_pdl(attn_weights_finish_kernel, dim3((unsigned)per * a.seqs.B), dim3(256), 0, stream, a, per));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "attn_weights_finish: %s", cudaGetErrorString(e));
  return check_launch("attn_weights_finish");
}

}  // namespace dsa
