// Sparse attention over the 4-bit latent cache on the CUDA cores, and the merge of rows attended in pieces (both paths
// use it).
//
//   S_i = scale · q[t,h,:]·kv[row_i, :],  out = Σ softmax(S)_i · kv[row_i, :d_c],  lse = log Σ exp S_i
//
// over the valid entries of idx[t, :], with a running max and sum, so each selected row is read and decoded once for 16
// heads.  This is the generic path (all widths, fp32 and bf16 queries); it computes in fp32 on the decoded values, which
// are exact.
//
// One CTA = one query × 16 heads × one share of the entries; 16 threads a head: two entries each for the logits,
// four columns in 64 each for the values, by 16-byte loads of shared memory (a decoded row is four floats longer than its columns,
// which spreads it over the banks).  Bound by latency for few queries and by shared-memory loads for many: 32 queries of 2,048
// entries and 128 heads, 512 + 64 columns in fp32 1,386 us (13 TFLOP/s), 256 + 64 in bf16 824.
#include <float.h>

#include "kv4.cuh"
#include "prefix_attn.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 16;

// KC entries a step (16 or 32); NJ: 64-column groups of the values (d_c <= 64 · NJ).
template <typename TK, typename TO, int KC, int NJ>
__global__ void __launch_bounds__(kThreads) attn4_simt_kernel(const __grid_constant__ Attn4Args a) {
  griddep_wait();
  if (a.splits > 1) griddep_launch();  // the merge may be set up meanwhile; it waits for this grid to end
  extern __shared__ __align__(16) float smem[];
  const int D = a.d_c + a.d_rope, DP = D + 4, dc = a.d_c, H = a.h;
  const int blocks = (H + kHeads - 1) / kHeads;
  const int t = blockIdx.x / blocks, h0 = (blockIdx.x - t * blocks) * kHeads, split = blockIdx.y;
  const int tid = threadIdx.x;
  float* qs = smem;                // [kHeads][D]
  float* ks = qs + kHeads * D;     // [KC][D + 4]
  float* P = ks + KC * DP;         // [kHeads][KC]
  __shared__ int rows[KC];         // cache rows, -1: skipped

  RowInfo r;
  if (!kv4_query_row(a.seqs, a.max_q_len, t, r, a.status)) return;
  const int nch = (a.top_k + KC - 1) / KC;
  const int c0 = (int)((int64_t)nch * split / a.splits), c1 = (int)((int64_t)nch * (split + 1) / a.splits);

  // a thread's head (heads past the last repeat it) and place among the head's 16 threads
  const int row = tid >> 4, place = tid & 15;
  const int h = min(h0 + row, H - 1);
  const int64_t flat = (int64_t)t * H + h;
  const TK* q = static_cast<const TK*>(a.q) + flat * D;
  for (int i = place; i < D; i += 16) qs[row * D + i] = to_f32(q[i]);
  const int rb = kv4_row_bytes(dc, a.d_rope), scale_at = kv4_scale_at(dc, a.d_rope);
  const int lats = dc / 8, units = D / 8;
  float m = -INFINITY, l = 0.f;
  float4 acc[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);

  for (int c = c0; c < c1; ++c) {
    __syncthreads();
    int found = -1;
    if (tid < KC) {
      const int i = c * KC + tid;
      const int v = i < a.top_k ? a.idx[(int64_t)t * a.top_k + i] : -1;
      if (v >= 0 && v <= r.pos) found = cache_row(a.seqs, r.b, r.k0, v);
      if (found < 0 && v != -1) atomicOr(a.status, DSA_FLAG_BAD_INDEX);
      if (!dsa_check(found < a.seqs.cache_rows(), a.status)) found = -1;
      rows[tid] = found;
    }
    if (!__syncthreads_or(found >= 0)) continue;  // a step of padding
    {
      constexpr int kT = kThreads / KC;  // threads that decode a row, 8 columns at a time
      const int k = tid / kT, from = rows[k];
      const uint8_t* src = a.kv4 + (int64_t)from * rb;
      for (int u = tid % kT; u < units; u += kT) {
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (from >= 0 && u < lats) {
          kv4_widen8(*reinterpret_cast<const uint32_t*>(src + 4 * u), kv4_scale(src[scale_at + u / 2]), f);
        } else if (from >= 0) {
          const uint2* v = reinterpret_cast<const uint2*>(src + kv4_rope_at(dc) + 16 * (u - lats));
          const uint2 x = v[0], y = v[1];
          const uint32_t w[4] = {x.x, x.y, y.x, y.y};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(w[j] << 16);
            f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
          }
        }
        float4* o = reinterpret_cast<float4*>(ks + k * DP + 8 * u);
        o[0] = make_float4(f[0], f[1], f[2], f[3]);
        o[1] = make_float4(f[4], f[5], f[6], f[7]);
      }
    }
    __syncthreads();
    float dot[KC / 16];
#pragma unroll
    for (int j = 0; j < KC / 16; ++j) dot[j] = 0.f;
    const float* qr = qs + row * D;
#pragma unroll 4
    for (int e = 0; e < D; e += 4) {
      const float4 x = *reinterpret_cast<const float4*>(qr + e);
#pragma unroll
      for (int j = 0; j < KC / 16; ++j) {
        const float4 y = *reinterpret_cast<const float4*>(ks + (place + 16 * j) * DP + e);
        dot[j] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, dot[j]))));
      }
    }
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < KC / 16; ++j) {
      dot[j] = rows[place + 16 * j] >= 0 ? dot[j] * a.scale_log2 : -INFINITY;
      mx = fmaxf(mx, dot[j]);
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float m_new = fmaxf(m, mx), ref = m_new == -INFINITY ? 0.f : m_new;  // -inf: nothing visible so far
    float sum = 0.f;
    __syncwarp();  // the last step's P has been read
#pragma unroll
    for (int j = 0; j < KC / 16; ++j) {
      const float e = exp2f(dot[j] - ref);
      P[row * KC + place + 16 * j] = e;
      sum += e;
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float alpha = exp2f(m - ref);
    l = fmaf(l, alpha, sum);
    m = m_new;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      acc[j].x *= alpha; acc[j].y *= alpha; acc[j].z *= alpha; acc[j].w *= alpha;
    }
    // (a skipped entry's row is zeros and its P is 0)
#pragma unroll 4
    for (int k = 0; k < KC; ++k) {
      const float pk = P[row * KC + k];
      const float* v = ks + k * DP + place * 4;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (place * 4 + 64 * j < dc) {
          const float4 y = *reinterpret_cast<const float4*>(v + 64 * j);
          acc[j].x = fmaf(pk, y.x, acc[j].x); acc[j].y = fmaf(pk, y.y, acc[j].y);
          acc[j].z = fmaf(pk, y.z, acc[j].z); acc[j].w = fmaf(pk, y.w, acc[j].w);
        }
    }
  }
  if (h0 + row >= H) return;
  const int64_t all = (int64_t)a.seqs.total_q * H;
  const bool last = a.splits == 1;
  const float inv = last ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int col = place * 4 + 64 * j;
    if (col >= dc) continue;
    const float f[4] = {acc[j].x * inv, acc[j].y * inv, acc[j].z * inv, acc[j].w * inv};
    if (last) {
      TO* o = static_cast<TO*>(a.out) + flat * dc + col;
#pragma unroll
      for (int i = 0; i < 4; ++i) store_f32(o + i, f[i]);
    } else {
      *reinterpret_cast<float4*>(a.part_o + ((int64_t)split * all + flat) * dc + col) =
          make_float4(f[0], f[1], f[2], f[3]);
    }
  }
  if (place == 0) {
    if (!last) a.part_ml[(int64_t)split * all + flat] = make_float2(fmaxf(m, -FLT_MAX), l);
    else if (a.lse) a.lse[flat] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

template <typename TK, typename TO, int KC, int NJ>
int launch_typed(const Attn4Args& a, cudaStream_t stream) {
  auto bytes = [](int D) constexpr { return (int)sizeof(float) * (kHeads * D + KC * (D + 4) + kHeads * KC); };
  const int smem = bytes(a.d_c + a.d_rope);
  auto kern = attn4_simt_kernel<TK, TO, KC, NJ>;
  static std::atomic<bool> allowed[64];
  const int rc = smem <= 40960 ? DSA_OK : allow_smem<bytes(KC == 16 ? kMaxWidth : 1024)>(kern, allowed, "attn4_simt: smem attribute");
  if (rc != DSA_OK) return rc;
  const int64_t blocks = (int64_t)a.seqs.total_q * ((a.h + kHeads - 1) / kHeads);
  if (blocks > 0x7fffffff) return set_error(DSA_ERR_UNSUPPORTED, "attn4: too many (query, head) rows");
  cudaError_t e = cudaSuccess;
  DSA_LAUNCH("attn4_simt", stream,
             e = launch_pdl(kern, dim3((unsigned)blocks, (unsigned)a.splits), dim3(kThreads), smem, stream, a));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "attn4_simt: %s", cudaGetErrorString(e));
  return check_launch("attn4_simt");
}

// 32 entries a step (16 where rows are wider than 1024: they would not fit the shared memory).
template <typename TK, typename TO>
int launch_dims(const Attn4Args& a, cudaStream_t stream) {
  if (a.d_c + a.d_rope > 1024) return launch_typed<TK, TO, 16, 16>(a, stream);
  return a.d_c <= 64    ? launch_typed<TK, TO, 32, 1>(a, stream)
         : a.d_c <= 512 ? launch_typed<TK, TO, 32, 8>(a, stream)
                        : launch_typed<TK, TO, 32, 16>(a, stream);
}

}  // namespace

// Pieces a row's entries are cut into, so that few rows still fill the SMs (three blocks fit one): at least 64 entries a
// piece.
int attn4_simt_splits(const Attn4Args& a) {
  const int64_t blocks = (int64_t)a.seqs.total_q * ((a.h + kHeads - 1) / kHeads);
  if (blocks == 0) return 1;
  int64_t s = 3 * (int64_t)num_sms() / blocks;
  const int64_t most = (a.top_k + 63) / 64;
  if (s > most) s = most;
  return (int)(s < 1 ? 1 : s);
}

int launch_attn4_simt(const Attn4Args& a, cudaStream_t stream) {
  const bool kf = a.kv_dtype == DSA_F32, of = a.out_dtype == DSA_F32;
  const int rc = kf ? (of ? launch_dims<float, float>(a, stream) : launch_dims<float, __nv_bfloat16>(a, stream))
                    : (of ? launch_dims<__nv_bfloat16, float>(a, stream)
                          : launch_dims<__nv_bfloat16, __nv_bfloat16>(a, stream));
  if (rc != DSA_OK || a.splits == 1) return rc;
  return launch_attn4_merge(a, stream);
}

int launch_attn4_merge(const Attn4Args& a, cudaStream_t stream) {
  PrefixArgs p{};
  p.seqs = a.seqs;
  p.max_q_len = a.max_q_len;
  p.h = a.h;
  p.d_c = a.d_c;
  p.d_rope = a.d_rope;
  p.kv_dtype = a.kv_dtype;
  p.out_dtype = a.out_dtype;
  p.out = a.out;
  p.lse = a.lse;
  p.status = a.status;
  p.part_o = a.part_o;
  p.part_ml = a.part_ml;
  PrefixMerge m{};
  m.pieces = m.base = a.splits;
  return launch_prefix_merge(p, m, stream);
}

}  // namespace dsa
