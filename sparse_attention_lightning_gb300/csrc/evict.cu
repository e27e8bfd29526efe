// dsa_evict: the positions of a cache to keep, by accumulated attention weight, and their move
// to a smaller cache.
//
// Of a sequence with L positions and a budget n < L, the first `sink` and the last `recent`
// positions stay, and of those between the budget - sink - recent with the largest acc (ties: the
// smaller position).  Kept positions keep their order.
//
// Two kernels.  Select: one CTA a sequence finds the exact threshold by radix select (four
// passes of 8 bits over order-preserving keys, counted in shared memory) and writes the kept
// positions in ascending order by a block scan.  Move: rows are independent, so the whole
// grid copies them, a warp a row, 16 bytes a lane.
#include "evict.cuh"

namespace dsa {
namespace {

constexpr int kSel = 1024;

__device__ __forceinline__ int seq_keep(const EvictArgs& a, int b, int& L) {
  const int k0 = __ldg(a.seqs.cu_k + b), k1 = __ldg(a.seqs.cu_k + b + 1);
  L = k1 - k0;
  if (k0 < 0 || L < 0 || k1 > a.seqs.total_k || L > a.seqs.max_k_len) {
    atomicOr(a.status, DSA_FLAG_BAD_SEQS);
    L = 0;
  }
  return min(L, a.budget);
}

// Exclusive prefix sum of v over the block; total in `sum`.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int w = warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  sum = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return x - v + (warp ? before : 0);
}

__global__ void __launch_bounds__(kSel) evict_select_kernel(EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int warp_sums[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int b = blockIdx.x, tid = threadIdx.x;
  int L;
  const int n = seq_keep(a, b, L);
  if (b == 0) {  // the kept lengths' prefix sums
    int run = 0;
    for (int i0 = 0; i0 < a.seqs.B; i0 += kSel) {
      int Li = 0, tot;
      const int v = i0 + tid < a.seqs.B ? seq_keep(a, i0 + tid, Li) : 0;
      const int ex = block_scan(v, warp_sums, tot);
      if (i0 + tid < a.seqs.B) a.cu_k_out[i0 + tid] = run + ex;
      run += tot;
    }
    if (tid == 0) a.cu_k_out[a.seqs.B] = run;
  }
  int32_t* kept = a.kept + (int64_t)b * a.budget;
  for (int i = n + tid; i < a.budget; i += kSel) kept[i] = -1;
  if (n == L) {
    for (int i = tid; i < n; i += kSel) kept[i] = i;
    return;
  }
  const float* acc = a.acc + (int64_t)b * a.ld_acc;
  const int lo = a.sink, hi = L - a.recent;
  // the (budget - sink - recent)-th largest key of [lo, hi), digit by digit; `need` counts how
  // many of the keys equal to the prefix so far are still to be taken
  uint32_t prefix = 0, mask = 0;
  int need = a.budget - a.sink - a.recent;
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int i = lo + tid; i < hi; i += kSel) {
        const uint32_t k = order_key(acc[i]);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int d = 255, left = need;
        while (d > 0 && hist[d] < left) left -= hist[d--];
        s_prefix = prefix | (uint32_t)d << shift;
        s_need = left;
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
      mask |= 255u << shift;
    }
  }
  // kept: sinks, recent ones, keys above the threshold, and the first `need` equal to it
  int out = 0, ties = 0;
  const bool any = a.budget - a.sink - a.recent > 0;
  for (int i0 = 0; i0 < L; i0 += kSel) {
    const int i = i0 + tid;
    bool keep = i < L && (i < lo || i >= hi);
    bool tie = false;
    if (any && i >= lo && i < hi) {
      const uint32_t k = order_key(acc[i]);
      keep = k > prefix;
      tie = k == prefix;
    }
    int tt, tk;
    const int tb = block_scan(tie, warp_sums, tt);
    keep |= tie && ties + tb < need;
    const int at = block_scan(keep, warp_sums, tk);
    if (keep) kept[out + at] = i;
    ties += tt;
    out += tk;
  }
}

struct Row {
  int64_t src, dst;  // cache rows, -1: not moved
};

__device__ __forceinline__ Row move_row(const EvictArgs& a, int b, int slot, int pos) {
  Row r{-1, -1};
  r.src = key_row(a.seqs, b, __ldg(a.seqs.cu_k + b), pos);
  if (a.table_out) {
    const int sh = __ffs(a.seqs.page_size) - 1;
    const int ps = slot >> sh;
    const int pg = ps < a.max_pages_out ? __ldg(a.table_out + (int64_t)b * a.max_pages_out + ps) : -1;
    if ((unsigned)pg < (unsigned)a.num_pages_out)
      r.dst = ((int64_t)pg << sh) | (slot & (a.seqs.page_size - 1));
  } else {
    r.dst = a.cu_k_out[b] + slot;
    if (r.dst >= a.rows_out) r.dst = -1;
  }
  if (r.src < 0 || r.dst < 0) {
    atomicOr(a.status, DSA_FLAG_BAD_SEQS);
    r.src = r.dst = -1;
  }
  return r;
}

__global__ void __launch_bounds__(256) evict_move_kernel(EvictArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t total = (int64_t)a.seqs.B * a.budget;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < total; w += step) {
    const int b = (int)(w / a.budget), slot = (int)(w - (int64_t)b * a.budget);
    const int pos = a.kept[w];
    if (pos < 0) continue;
    const Row r = move_row(a, b, slot, pos);
    if (r.src < 0) continue;
#pragma unroll
    for (int c = 0; c < 3; ++c) {
      const int nb = a.row_bytes[c];
      if (!nb) continue;
      const char* s = static_cast<const char*>(a.src[c]) + r.src * nb;
      char* d = static_cast<char*>(a.dst[c]) + r.dst * nb;
      if (nb % 16 == 0)
        for (int i = lane * 16; i < nb; i += 512)
          *reinterpret_cast<uint4*>(d + i) = *reinterpret_cast<const uint4*>(s + i);
      else if (lane < nb)
        d[lane] = s[lane];
    }
  }
}

// acc of the kept positions, zero behind them (positions appended later start from nothing).
__global__ void __launch_bounds__(256) evict_acc_kernel(EvictArgs a, int per) {
  const int b = blockIdx.x / per, j = blockIdx.x - b * per;
  for (int64_t i = j * 256 + threadIdx.x; i < a.ld_acc_out; i += (int64_t)per * 256) {
    const int pos = i < a.budget ? a.kept[(int64_t)b * a.budget + i] : -1;
    a.acc_out[(int64_t)b * a.ld_acc_out + i] = pos >= 0 ? a.acc[(int64_t)b * a.ld_acc + pos] : 0.f;
  }
}

}  // namespace

int launch_evict(const EvictArgs& a, cudaStream_t stream) {
  DSA_LAUNCH("evict_select", stream, evict_select_kernel<<<a.seqs.B, kSel, 0, stream>>>(a));
  int rc = check_launch("evict_select");
  if (rc != DSA_OK) return rc;
  if (a.row_bytes[0] || a.row_bytes[1] || a.row_bytes[2]) {
    const int64_t warps = (int64_t)a.seqs.B * a.budget;
    const int64_t most = (int64_t)num_sms() * 8;
    const int64_t blocks = (warps + 7) / 8;
    DSA_LAUNCH("evict_move", stream,
               evict_move_kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, stream>>>(a));
    rc = check_launch("evict_move");
    if (rc != DSA_OK) return rc;
  }
  if (a.acc_out) {
    const int64_t want = (a.ld_acc_out + 255) / 256, most = 0x7fffffff / a.seqs.B;
    const int per = (int)(want < 64 ? (want < most ? want : most) : (64 < most ? 64 : most));
    DSA_LAUNCH("evict_acc", stream,
               evict_acc_kernel<<<(unsigned)per * a.seqs.B, 256, 0, stream>>>(a, per));
    rc = check_launch("evict_acc");
  }
  return rc;
}

}  // namespace dsa
