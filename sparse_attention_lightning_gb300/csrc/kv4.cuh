// The latent cache in 4 bits: its row layout and arithmetic, and what its kernels and its host code share.
//
// A row of d_c latent and d_rope rope columns, kv4_row_bytes() bytes, in this order:
//   d_c / 2   codes: E2M1 (sign, magnitude 0 .5 1 1.5 2 3 4 6), eight columns a 32-bit word
//   2·d_rope  the rope columns in bf16
//   d_c / 16  scales: one UE5M3 byte for 16 columns
//   zeros up to a multiple of 16
// and column c is code[c] · scale[c / 16].
//
// A scale byte is an fp16 number without its sign and its seven lowest bits (five bits of exponent with bias 15, three
// of mantissa, subnormal steps of 2^-17, 0xf8 and above not finite): a scale has no sign, and the bit buys the range, 2^-17 to
// 61440, that an E4M3 scale would need a second, per-row scale for.  Codes have two significant bits and scales four, so
// every value is a bf16 number exactly.
//
// In a word column 2k of eight is the nibble at bit 4k and column 2k + 1 the one at bit 16 + 4k: a shift and two masks
// turn a nibble in each half into a pair of bf16.
#pragma once

#include "cache_ops.cuh"

namespace dsa {

__host__ __device__ constexpr int kv4_rope_at(int d_c) { return d_c / 2; }
__host__ __device__ constexpr int kv4_scale_at(int d_c, int d_rope) { return d_c / 2 + 2 * d_rope; }
__host__ __device__ constexpr int kv4_row_bytes(int d_c, int d_rope) {
  return (kv4_scale_at(d_c, d_rope) + d_c / 16 + 15) / 16 * 16;
}

// A scale byte in fp32.  (byte << 20 is its exponent and mantissa in fp32's places, 112 too low in the exponent; a
// subnormal one is a subnormal fp32 number there, so both come right by one multiplication.)
__device__ __forceinline__ float kv4_scale(uint32_t byte) {
  return byte >= 0xf8u ? __uint_as_float(0x7fffffffu) : __uint_as_float(byte << 20) * 0x1p112f;
}

// Pair k (columns 2k and 2k + 1) of a word of codes as two bf16 numbers, 2^-126 times their value: the magnitude's exponent and
// mantissa bits at the lower end of bf16's, where E2M1's subnormal 0.5 is a subnormal too.
template <int K>
__device__ __forceinline__ uint32_t kv4_pair(uint32_t w) {
  const uint32_t s = K == 3 ? w : w << (12 - 4 * K);
  const uint32_t m = K < 2 ? w << (6 - 4 * K) : w >> (4 * K - 6);
  return (s & 0x80008000u) | (m & 0x01c001c0u);
}

// Product of two pairs of bf16 (subnormal operands count; products that are bf16 numbers are exact).
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Eight columns of a word in fp32, from their scale.
__device__ __forceinline__ void kv4_widen8(uint32_t w, float scale, float (&f)[8]) {
  const uint32_t p[4] = {kv4_pair<0>(w), kv4_pair<1>(w), kv4_pair<2>(w), kv4_pair<3>(w)};
#pragma unroll
  for (int k = 0; k < 4; ++k) {  // (times 2^126, then the scale: their product would overflow)
    f[2 * k] = __uint_as_float(p[k] << 16) * 0x1p126f * scale;
    f[2 * k + 1] = __uint_as_float(p[k] & 0xffff0000u) * 0x1p126f * scale;
  }
}

// The query row t's place in its sequence, by ordinary loads; false (and flagged) when cu_q/cu_k are inconsistent with the
// descriptor.
__device__ __forceinline__ bool kv4_query_row(const Seqs& s, int max_q_len, int t, RowInfo& r, uint32_t* status) {
  int lo = 0, hi = s.B - 1;
  while (lo < hi) {  // last b with cu_q[b] <= t
    const int mid = (lo + hi + 1) >> 1;
    if (s.cu_q[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int q0 = s.cu_q[lo], q1 = s.cu_q[lo + 1], k0 = s.cu_k[lo], k1 = s.cu_k[lo + 1];
  const int T = q1 - q0, L = k1 - k0;
  if (!(t >= q0 && t < q1 && T <= L && k0 >= 0 && k1 <= s.total_k && L <= s.max_k_len && q0 >= 0 &&
        q1 <= s.total_q && T <= max_q_len)) {
    atomicOr(status, DSA_FLAG_BAD_SEQS);
    return false;
  }
  r = RowInfo{lo, L - T + (t - q0), k0, L};
  return true;
}

struct Kv4Rows {
  Seqs seqs;
  int max_q_len, d_c, d_rope, dtype;
  const void* latent;   // write: [total_q, d_c], rows ld_latent elements apart
  int64_t ld_latent;
  const void* k_rope;   // [total_q, d_rope], rows ld_rope apart
  int64_t ld_rope;
  uint8_t* kv4;         // the cache
  void* out;            // read: [total_k, d_c + d_rope]
  uint32_t* status;
};
int launch_write_kv4(const Kv4Rows& a, cudaStream_t stream);
int launch_read_kv4(const Kv4Rows& a, cudaStream_t stream);

struct Attn4Args {
  Seqs seqs;
  int max_q_len, h, d_c, d_rope, top_k, kv_dtype, out_dtype;
  float scale_log2;    // softmax scale · log2(e)
  const void* q;
  const uint8_t* kv4;
  const int32_t* idx;
  void* out;
  float* lse;
  uint32_t* status;
  int splits;          // pieces a row's entries are cut into that leave partial outputs
  int cluster;         // tcgen05 path: or CTAs of a cluster that share a row's entries
  float* part_o;       // [pieces][total_q · h][d_c] unnormalised partial outputs
  float2* part_ml;     // [pieces][total_q · h] (max in log2 units, sum)
  uint8_t* scratch;    // tcgen05 path: attn4_tc_scratch() bytes
};
// tcgen05 path (bf16, 512 + 64 columns; a build whose registers do not suffice for its roles takes the other one).
bool attn4_tc_eligible(const Attn4Args& a);
void attn4_tc_plan(Attn4Args& a);  // sets splits, cluster
size_t attn4_tc_scratch(const Attn4Args& a);
int launch_attn4_tc(const Attn4Args& a, cudaStream_t stream);
int attn4_simt_splits(const Attn4Args& a);
int launch_attn4_simt(const Attn4Args& a, cudaStream_t stream);
int launch_attn4_merge(const Attn4Args& a, cudaStream_t stream);

}  // namespace dsa
