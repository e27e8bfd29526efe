// Dense attention over the MLA latent cache for a batch that shares a prefix, on the CUDA cores,
// and the merge of rows attended in pieces (both paths use it).
//
// Every query sees the prefix's keys and, causally, its own sequence's: for query row t, head h,
// over the keys x of [prefix | suffix of its sequence] up to its own position,
//   S_x = scale · q[t,h,:]·key_x,   out = Σ softmax(S)_x · key_x[0:d_c],   lse = log Σ exp S_x
// with a running max and sum, so each key is read once per block of rows.
//
// One CTA = 16 of a sequence's (token, head) rows × one share of their keys: every row attends
// over the same latent keys, so a key loaded to shared memory serves 16 rows.  This is the
// generic fp32/bf16 path (all dims); it computes in fp32.
#include "prefix_attn.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;

template <typename TK, typename TO, int KC>
__global__ void __launch_bounds__(kThreads) prefix_simt_kernel(PrefixArgs a, int nblk) {
  griddep_launch();  // the merge may be set up meanwhile; it waits for this grid to end
  extern __shared__ float smem[];
  const int D = a.d_c + a.d_rope, DP = D + 1, dc = a.d_c, H = a.h;
  const int b = blockIdx.x / nblk, blk = blockIdx.x - b * nblk, split = blockIdx.y;
  const int tid = threadIdx.x;
  float* qs = smem;                 // [kRows][D]
  float* ks = qs + kRows * D;       // [KC][D + 1]
  float* acc = ks + KC * DP;        // [kRows][dc]
  float* P = acc + kRows * dc;      // [kRows][KC]
  float* m_s = P + kRows * KC;      // [kRows]
  float* l_s = m_s + kRows;
  float* al_s = l_s + kRows;
  __shared__ uint32_t okmask;

  SeqInfo s;
  if (!prefix_seq(a, b, s)) return;
  const int64_t r0 = (int64_t)blk * kRows, nrow = (int64_t)s.T * H;
  if (r0 >= nrow) return;
  const int R = (int)min((int64_t)kRows, nrow - r0);
  const int64_t flat0 = (int64_t)s.q0 * H + r0;  // first (token, head) row of the block
  // keys row i of the block sees: the prefix and its sequence up to its token
  auto visible = [&](int i) { return a.prefix_len + s.L - s.T + (int)((r0 + i) / H) + 1; };
  const int nvis = visible(R - 1);
  const int nch = (nvis + KC - 1) / KC;
  const int c0 = (int)((int64_t)nch * split / a.splits), c1 = (int)((int64_t)nch * (split + 1) / a.splits);

  const TK* q = static_cast<const TK*>(a.q) + flat0 * D;
  for (int i = tid; i < R * D; i += kThreads) qs[i] = to_f32(q[i]);
  for (int i = tid; i < R * dc; i += kThreads) acc[i] = 0.f;
  if (tid < kRows) { m_s[tid] = -INFINITY; l_s[tid] = 0.f; }

  for (int c = c0; c < c1; ++c) {
    const int x0 = c * KC, cn = min(KC, nvis - x0);
    __syncthreads();
    if (tid < 32) {
      // a key on a page outside the cache is skipped (and reported)
      const bool in = tid < cn;
      const bool ok = in && prefix_key(a, s.b, s.k0, x0 + tid) != nullptr;
      if (in && !ok) atomicOr(a.status, DSA_FLAG_BAD_INDEX);
      const unsigned bal = __ballot_sync(0xffffffffu, ok);
      if (tid == 0) okmask = bal;
    }
    for (int i = tid; i < KC * D; i += kThreads) {
      const int k = i / D, col = i - k * D;
      const TK* src = k < cn ? static_cast<const TK*>(prefix_key(a, s.b, s.k0, x0 + k)) : nullptr;
      ks[k * DP + col] = src ? to_f32(src[col]) : 0.f;
    }
    __syncthreads();
    const uint32_t ok = okmask;
    for (int i = tid; i < kRows * KC; i += kThreads) {
      const int r = i / KC, k = i - r * KC;
      if (r >= R) continue;
      const float* qr = qs + r * D;
      const float* kr = ks + k * DP;
      float dot = 0.f;
      for (int e = 0; e < D; ++e) dot = fmaf(qr[e], kr[e], dot);
      P[i] = ((ok >> k) & 1u) && x0 + k < visible(r) ? dot * a.scale_log2 : -INFINITY;
    }
    __syncthreads();
    for (int r = tid >> 5; r < R; r += kThreads / 32) {  // a warp per row, KC <= 32
      const int lane = tid & 31;
      const bool in = lane < KC && ((ok >> lane) & 1u) && x0 + lane < visible(r);
      const float v = in ? P[r * KC + lane] : -INFINITY;
      float mx = v;
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m_old = m_s[r], m_new = fmaxf(m_old, mx);
      const float ref = m_new == -INFINITY ? 0.f : m_new;  // nothing visible so far
      const float e = in ? exp2f(v - ref) : 0.f;
      if (lane < KC) P[r * KC + lane] = e;
      float sum = e;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) {
        const float alpha = exp2f(m_old - ref);
        al_s[r] = alpha;
        l_s[r] = l_s[r] * alpha + sum;
        m_s[r] = m_new;
      }
    }
    __syncthreads();
    for (int i = tid; i < R * dc; i += kThreads) {
      const int r = i / dc, col = i - r * dc;
      const float* pr = P + r * KC;
      // only keys the row sees: a masked key's values (whatever they are) add nothing
      const int n = min(cn, visible(r) - x0);
      float v = acc[i] * al_s[r];
      for (int k = 0; k < n; ++k) v = fmaf(pr[k], ks[k * DP + col], v);
      acc[i] = v;
    }
  }
  __syncthreads();
  if (a.splits == 1) {
    TO* o = static_cast<TO*>(a.out) + flat0 * dc;
    for (int i = tid; i < R * dc; i += kThreads) {
      const float l = l_s[i / dc];
      store_f32(o + i, l == 0.f ? 0.f : acc[i] / l);
    }
    if (a.lse && tid < R)
      a.lse[flat0 + tid] = l_s[tid] == 0.f ? -INFINITY : (m_s[tid] + log2f(l_s[tid])) * kLn2;
    return;
  }
  const int64_t rows = (int64_t)a.seqs.total_q * H;
  float* o = a.part_o + ((int64_t)split * rows + flat0) * dc;
  for (int i = tid; i < R * dc; i += kThreads) o[i] = acc[i];
  if (tid < R) a.part_ml[(int64_t)split * rows + flat0 + tid] = make_float2(m_s[tid], l_s[tid]);
}

// out = Σ_j w_j O_j / Σ_j w_j l_j, w_j = 2^(m_j - max m) over the row's pieces, O added in piece order.  A block a
// row, four columns a thread.  All it costs is latency: the row is looked up before the pieces' grid has
// ended, each lane takes two pieces' (max, sum), and eight pieces' outputs are loaded before the first is
// added.  (One load after another, for 9 pieces of 64 rows: 12 us; so: 4.)  A piece without keys has l = 0
// and its O is not read.
constexpr int kMaxPieces = 128;
template <typename TO>
__global__ void __launch_bounds__(128, 8) prefix_merge_kernel(PrefixArgs a, int pieces) {
  const int64_t rows = (int64_t)a.seqs.total_q * a.h, row = blockIdx.x;
  const int lane = threadIdx.x & 31;
  RowInfo ri;
  SeqInfo si;  // the pieces of a row whose sequence is inconsistent were not written
  const bool ok = query_row_info(a.seqs, (int)(row / a.h), ri, a.status) && prefix_seq(a, ri.b, si);
  griddep_wait();
  if (!ok) return;
  float m[kMaxPieces / 32], w[kMaxPieces / 32], M = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxPieces / 32; ++i) {
    const int j = i * 32 + lane;
    const float2 v = j < pieces ? __ldcg(a.part_ml + j * rows + row) : make_float2(-INFINITY, 0.f);
    m[i] = v.x;
    w[i] = v.y;
    if (v.y != 0.f) M = fmaxf(M, v.x);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
  for (int i = 0; i < kMaxPieces / 32; ++i) {
    const float f = w[i] == 0.f ? 0.f : exp2f(m[i] - ref);
    l = fmaf(f, w[i], l);
    w[i] = f;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  TO* o = static_cast<TO*>(a.out) + row * a.d_c;
  const float* po = a.part_o + row * a.d_c;
  const int64_t stride = rows * a.d_c;
  for (int c0 = 0; c0 < a.d_c; c0 += 512) {
    const int c = c0 + (int)threadIdx.x * 4;
    const bool in = c < a.d_c;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kMaxPieces / 32; ++i) {
      if (i * 32 >= pieces) break;
      for (int j0 = 0; j0 < 32 && i * 32 + j0 < pieces; j0 += 8) {
        float4 x[8];
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[j] = __shfl_sync(0xffffffffu, w[i], j0 + j);  // 0 past the last piece
          x[j] = in && f[j] != 0.f
                     ? __ldcg(reinterpret_cast<const float4*>(po + (i * 32 + j0 + j) * stride + c))
                     : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s.x = fmaf(f[j], x[j].x, s.x); s.y = fmaf(f[j], x[j].y, s.y);
          s.z = fmaf(f[j], x[j].z, s.z); s.w = fmaf(f[j], x[j].w, s.w);
        }
      }
    }
    if (!in) continue;
    if (sizeof(TO) == 4) {
      *reinterpret_cast<float4*>(o + c) = make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
    } else {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x * inv, s.y * inv);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(s.z * inv, s.w * inv);
      *reinterpret_cast<uint2*>(o + c) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
  }
  if (a.lse && threadIdx.x == 0) a.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
}

template <typename TK, typename TO, int KC>
int launch_typed(const PrefixArgs& a, cudaStream_t stream) {
  const int D = a.d_c + a.d_rope;
  const size_t smem = sizeof(float) * ((size_t)kRows * D + (size_t)KC * (D + 1) +
                                       (size_t)kRows * a.d_c + kRows * KC + 3 * kRows);
  auto kern = prefix_simt_kernel<TK, TO, KC>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
      cudaSuccess)
    return check_launch("prefix_simt: smem attribute");
  const int nblk = prefix_simt_blocks(a.max_q_len, a.h);
  dim3 grid((unsigned)(a.seqs.B * nblk), (unsigned)a.splits);
  DSA_LAUNCH("prefix_simt", stream, kern<<<grid, kThreads, smem, stream>>>(a, nblk));
  return check_launch("prefix_simt");
}

template <typename TK, typename TO>
int launch_dims(const PrefixArgs& a, cudaStream_t stream) {
  // 32 keys a step where they fit the shared memory beside the widest rows, else 16
  return a.d_c + a.d_rope <= 640 ? launch_typed<TK, TO, 32>(a, stream)
                                 : launch_typed<TK, TO, 16>(a, stream);
}

}  // namespace

int launch_prefix_simt(const PrefixArgs& a, cudaStream_t stream) {
  const bool kf = a.kv_dtype == DSA_F32, of = a.out_dtype == DSA_F32;
  const int rc = kf ? (of ? launch_dims<float, float>(a, stream)
                          : launch_dims<float, __nv_bfloat16>(a, stream))
                    : (of ? launch_dims<__nv_bfloat16, float>(a, stream)
                          : launch_dims<__nv_bfloat16, __nv_bfloat16>(a, stream));
  if (rc != DSA_OK || a.splits == 1) return rc;
  return launch_prefix_merge(a, a.splits, stream);
}

int launch_prefix_merge(const PrefixArgs& a, int pieces, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.seqs.total_q * a.h;
  auto kern = a.out_dtype == DSA_F32 ? prefix_merge_kernel<float> : prefix_merge_kernel<__nv_bfloat16>;
  cudaError_t e = cudaSuccess;
  DSA_LAUNCH("prefix_merge", stream, e = launch_pdl(kern, dim3((unsigned)rows), dim3(128), 0, stream, a, pieces));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "prefix_merge: %s", cudaGetErrorString(e));
  return check_launch("prefix_merge");
}

}  // namespace dsa
