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
//
// Bound by latency (few rows) and by shared-memory loads.  16 threads take a row: two keys each for the
// logits, four columns in 64 each for the values, both by 16-byte loads (a row of keys is four floats longer
// than its columns, which spreads it over the banks); max and sum stay within the 16, so a chunk of 32
// keys needs two block barriers.  One thread a dot, scalar loads and the softmax through shared memory took
// 45 us for 3 sequences of up to 40 tokens x 8 heads over 256 + 130 keys of 80 columns; this way it is 16.
#include <float.h>

#include "prefix_attn.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;

// 16 bytes of keys or queries as floats.
__device__ __forceinline__ void widen16(const uint4& v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void widen16(const uint4& v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
template <typename TK>
__device__ __forceinline__ void copy16(float* dst, const TK* src) {
  constexpr int V = 16 / (int)sizeof(TK);
  float f[V];
  widen16(src ? *reinterpret_cast<const uint4*>(src) : make_uint4(0u, 0u, 0u, 0u), f);
#pragma unroll
  for (int i = 0; i < V; i += 4)
    *reinterpret_cast<float4*>(dst + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
}

// KC keys a step (16 or 32); NJ: 64-column groups of the values (d_c <= 64 · NJ).
template <typename TK, typename TO, int KC, int NJ>
__global__ void __launch_bounds__(kThreads) prefix_simt_kernel(PrefixArgs a, int nblk) {
  griddep_wait();
  if (a.splits > 1) griddep_launch();  // the merge may be set up meanwhile; it waits for this grid to end
  extern __shared__ __align__(16) float smem[];
  constexpr int V = 16 / (int)sizeof(TK);
  const int D = a.d_c + a.d_rope, DP = D + 4, dc = a.d_c, H = a.h;
  const int b = blockIdx.x / nblk, blk = blockIdx.x - b * nblk, split = blockIdx.y;
  const int tid = threadIdx.x;
  float* qs = smem;                 // [kRows][D]
  float* ks = qs + kRows * D;       // [KC][D + 4]
  float* P = ks + KC * DP;          // [kRows][KC]
  __shared__ const TK* keys[KC];    // null: masked

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

  // a thread's row (rows past the block repeat its last) and place among the row's 16 threads
  const int row = tid >> 4, place = tid & 15;
  const int r = min(row, R - 1), vis = visible(r);
  const TK* q = static_cast<const TK*>(a.q) + (flat0 + r) * D;
  for (int i = place * V; i < D; i += 16 * V) copy16(qs + row * D + i, q + i);
  float m = -INFINITY, l = 0.f;
  float4 acc[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);

  for (int c = c0; c < c1; ++c) {
    const int x0 = c * KC, cn = min(KC, nvis - x0);
    __syncthreads();
    if (tid < KC) {
      const void* k = tid < cn ? prefix_key(a, s.b, s.k0, x0 + tid) : nullptr;
      // a key on a page outside the cache is skipped (and reported)
      if (tid < cn && !k) atomicOr(a.status, DSA_FLAG_BAD_INDEX);
      keys[tid] = static_cast<const TK*>(k);
    }
    __syncthreads();
    {
      // 256 / KC threads load a key
      constexpr int kT = kThreads / KC;
      const int k = tid / kT;
      const TK* src = keys[k];
      for (int i = (tid % kT) * V; i < D; i += kT * V) copy16(ks + k * DP + i, src ? src + i : nullptr);
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
      const int k = place + 16 * j;
      dot[j] = keys[k] && x0 + k < vis ? dot[j] * a.scale_log2 : -INFINITY;
      mx = fmaxf(mx, dot[j]);
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float m_new = fmaxf(m, mx), ref = m_new == -INFINITY ? 0.f : m_new;  // -inf: nothing visible so far
    float sum = 0.f;
    __syncwarp();  // the last chunk's P has been read
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
    // only keys the row sees: a masked key's values (whatever they are) add nothing
    const int n = min(cn, vis - x0);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
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
  if (row >= R) return;
  const int64_t rows = (int64_t)a.seqs.total_q * H, flat = flat0 + row;
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
      *reinterpret_cast<float4*>(a.part_o + ((int64_t)split * rows + flat) * dc + col) =
          make_float4(f[0], f[1], f[2], f[3]);
    }
  }
  if (place == 0) {
    if (!last) a.part_ml[(int64_t)split * rows + flat] = make_float2(c0 < c1 ? fmaxf(m, -FLT_MAX) : m, l);
    else if (a.lse) a.lse[flat] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// out = Σ_j w_j O_j / Σ_j w_j l_j, w_j = 2^(m_j - max m) over the row's pieces, O added in piece order.  A block a
// row, four columns a thread.  All it costs is latency: the row is looked up before the pieces' grid has
// ended, each lane takes up to four pieces' (max, sum), and U pieces' outputs are loaded before the first is
// added: 8 where all blocks run at once, 4 (and twice the blocks on an SM) for more rows: 4096 rows of 2 to 4 pieces
// take 2 us less that way, 64 rows of 9 pieces 1 us more.  One load after another, those 64 rows took 12 us;
// so they take 4.  A piece without keys has m = -inf and its O is not read; one whose weight is 0 is: 0 times a NaN
// in it is NaN, as in a row attended whole.
constexpr int kMaxPieces = 128;
template <typename TO, int U>
__global__ void __launch_bounds__(128, 64 / U) prefix_merge_kernel(const __grid_constant__ PrefixArgs a, const __grid_constant__ PrefixMerge mg) {
  const int64_t rows = (int64_t)a.seqs.total_q * a.h, row = blockIdx.x;
  const int lane = threadIdx.x & 31;
  RowInfo ri;
  SeqInfo si;  // the pieces of a row whose sequence is inconsistent were not written
  const bool ok = query_row_info(a.seqs, (int)(row / a.h), ri, a.status) && prefix_seq(a, ri.b, si);
  // its pieces: slots [0, n0) and [base, base + n1)
  int n0 = mg.pieces, n1 = 0, pieces = mg.pieces;
  if (mg.table && ok) {
    const int line = mg.fblk + ri.b * mg.nblk + (int)((row - (int64_t)si.q0 * a.h) >> 7);
    n0 = mg.fblk ? mg.np[row >> 7] : 0;
    n1 = mg.np[line];
    pieces = mg.base + n1;
  }
  griddep_wait();
  if (!ok || (mg.table && !mg.fblk && n1 == 1)) return;  // (a line that was not cut wrote its output)
  float m[kMaxPieces / 32], w[kMaxPieces / 32], M = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxPieces / 32; ++i) {
    const int j = i * 32 + lane;
    const float2 v = j < n0 || (j >= mg.base && j < mg.base + n1) ? __ldcg(a.part_ml + j * rows + row) : make_float2(-INFINITY, 0.f);
    m[i] = v.x;
    w[i] = v.y;
    if (v.y != 0.f) M = fmaxf(M, v.x);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
  for (int i = 0; i < kMaxPieces / 32; ++i) {
    float f = w[i] == 0.f ? 0.f : exp2f(m[i] - ref);
    l = fmaf(f, w[i], l);
    if (f == 0.f) f = m[i] == -INFINITY ? 0.f : -0.f;  // +0: not read
    w[i] = f;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (l < 0.f) return;  // (the pieces' grid found the row's sequence inconsistent)
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
      for (int j0 = 0; j0 < 32 && i * 32 + j0 < pieces; j0 += U) {
        float4 x[U];
        float f[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
          f[j] = __shfl_sync(0xffffffffu, w[i], j0 + j);  // 0 past the last piece
          x[j] = in && __float_as_uint(f[j]) != 0u
                     ? __ldcg(reinterpret_cast<const float4*>(po + (i * 32 + j0 + j) * stride + c))
                     : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
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

template <typename TK, typename TO, int KC, int NJ>
int launch_typed(const PrefixArgs& a, cudaStream_t stream) {
  auto bytes = [](int D) constexpr { return (int)sizeof(float) * (kRows * D + KC * (D + 4) + kRows * KC); };
  const int smem = bytes(a.d_c + a.d_rope);
  auto kern = prefix_simt_kernel<TK, TO, KC, NJ>;
  static std::atomic<bool> allowed[64];
  const int rc = smem <= 40960 ? DSA_OK : allow_smem<bytes(KC == 16 ? kMaxWidth : 1024)>(kern, allowed, "prefix_simt: smem attribute");
  if (rc != DSA_OK) return rc;
  const int nblk = prefix_simt_blocks(a.max_q_len, a.h);
  dim3 grid((unsigned)(a.seqs.B * nblk), (unsigned)a.splits);
  cudaError_t e = cudaSuccess;
  DSA_LAUNCH("prefix_simt", stream, e = launch_pdl(kern, grid, dim3(kThreads), smem, stream, a, nblk));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "prefix_simt: %s", cudaGetErrorString(e));
  return check_launch("prefix_simt");
}

// 32 keys a step (16 where rows are wider than 1024: they would not fit the shared memory).
template <typename TK, typename TO>
int launch_dims(const PrefixArgs& a, cudaStream_t stream) {
  if (a.d_c + a.d_rope > 1024) return launch_typed<TK, TO, 16, 16>(a, stream);
  return a.d_c <= 64    ? launch_typed<TK, TO, 32, 1>(a, stream)
         : a.d_c <= 512 ? launch_typed<TK, TO, 32, 8>(a, stream)
                        : launch_typed<TK, TO, 32, 16>(a, stream);
}

}  // namespace

int launch_prefix_simt(const PrefixArgs& a, cudaStream_t stream) {
  const bool kf = a.kv_dtype == DSA_F32, of = a.out_dtype == DSA_F32;
  const int rc = kf ? (of ? launch_dims<float, float>(a, stream)
                          : launch_dims<float, __nv_bfloat16>(a, stream))
                    : (of ? launch_dims<__nv_bfloat16, float>(a, stream)
                          : launch_dims<__nv_bfloat16, __nv_bfloat16>(a, stream));
  if (rc != DSA_OK || a.splits == 1) return rc;
  PrefixMerge m{};
  m.pieces = m.base = a.splits;
  return launch_prefix_merge(a, m, stream);
}

int launch_prefix_merge(const PrefixArgs& a, const PrefixMerge& m, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.seqs.total_q * a.h;
  const bool few = rows <= 8 * (int64_t)num_sms();
  auto kern = a.out_dtype == DSA_F32
                  ? (few ? prefix_merge_kernel<float, 8> : prefix_merge_kernel<float, 4>)
                  : (few ? prefix_merge_kernel<__nv_bfloat16, 8> : prefix_merge_kernel<__nv_bfloat16, 4>);
  cudaError_t e = cudaSuccess;
  DSA_LAUNCH("prefix_merge", stream, e = launch_pdl(kern, dim3((unsigned)rows), dim3(128), 0, stream, a, m));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "prefix_merge: %s", cudaGetErrorString(e));
  return check_launch("prefix_merge");
}

}  // namespace dsa
