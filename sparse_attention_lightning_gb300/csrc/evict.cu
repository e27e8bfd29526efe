// dsa_evict: the positions of a cache to keep, by accumulated attention weight, and their move
// to a smaller cache.
//
// Of a sequence with L positions and a budget n < L, the first `sink` and the last `recent`
// positions stay, and of those between the budget - sink - recent with the largest acc (ties: the
// smaller position).  Kept positions keep their order.
//
// Select: one CTA a sequence.  Its order-preserving keys are read once into shared memory (up to
// 48K positions; longer histories are read again each pass).  The exact threshold comes from three
// radix passes of 11, 11 and 10 bits (a first digit of sign, exponent and two mantissa bits spreads
// weights over many bins; with 8-bit digits their exponents share a few, and the counts serialise).
// Then each thread takes one contiguous run: it counts its keys above and at the threshold, two scans
// give it its first slot and its share of the ties, and it writes its kept positions in order.
//
// Move: rows are independent.  A thread takes a row: one bulk copy a cache into its slot of shared
// memory, one out of it; 128 rows (164 KB) are in flight on an SM and no piece of them passes through
// registers.  It is launched while Select runs and waits for it on the device.
#include "evict.cuh"
#include "tc_sm100.cuh"

namespace dsa {
namespace {

constexpr int kSel = 1024;
constexpr int kWarps = kSel / 32;
constexpr int kBins = 2048;
constexpr int kSmemKeys = 49152;

__device__ __forceinline__ int seq_keep(const EvictArgs& a, int b, int& L) {
  const int k0 = a.seqs.cu_k[b], k1 = a.seqs.cu_k[b + 1];
  L = k1 - k0;
  if (k0 < 0 || L < 0 || k1 > a.seqs.total_k || L > a.seqs.max_k_len) {
    atomicOr(a.status, DSA_FLAG_BAD_SEQS);
    L = 0;
  }
  return min(L, a.budget);
}

// order_key with every NaN, whatever its sign and payload, above all numbers.
__device__ __forceinline__ uint32_t weight_key(float f) { return f != f ? 0xffffffffu : order_key(f); }

__device__ __forceinline__ int warp_scan(int v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// Exclusive prefix sum of v over the block; total in `sum`.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int x = warp_scan(v, lane);
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  const int w = warp_scan(warp_sums[lane], lane);
  sum = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return x - v + (warp ? before : 0);
}

// SMEM: the keys of [0, L) are held in shared memory (max_k_len <= kSmemKeys).
template <bool SMEM>
__global__ void __launch_bounds__(kSel) evict_select_kernel(EvictArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ int hist[kBins];
  __shared__ int warp_sums[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  griddep_wait();
  if (a.moves) griddep_launch();  // the move may be set up meanwhile; it waits for this grid to end
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  auto key = [&](int i) { return SMEM ? keys[i] : weight_key(acc[i]); };
  int need = a.budget - a.sink - a.recent;
  const bool any = need > 0;
  uint32_t prefix = 0;
  // the (budget - sink - recent)-th largest key of [lo, hi), digit by digit; `need` counts how many of
  // the keys equal to the digits so far are still to be taken
  for (int pass = 0; any && pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
    const int bins = pass == 2 ? 1024 : kBins;
    for (int i = tid; i < kBins; i += kSel) hist[i] = 0;
    __syncthreads();
    if (SMEM && pass == 0) {
      constexpr int kFly = 16;  // loads in flight: with 4, 32K positions took 8 round trips to memory
      for (int i = lo + tid; i < hi; i += kFly * kSel) {
        float f[kFly];
#pragma unroll
        for (int j = 0; j < kFly; ++j) f[j] = i + j * kSel < hi ? acc[i + j * kSel] : 0.f;
#pragma unroll
        for (int j = 0; j < kFly; ++j)
          if (i + j * kSel < hi) {
            const uint32_t k = weight_key(f[j]);
            keys[i + j * kSel] = k;
            atomicAdd(&hist[k >> 21], 1);
          }
      }
    } else {
      for (int i = lo + tid; i < hi; i += kSel) {
        const uint32_t k = key(i);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
      }
    }
    __syncthreads();
    // thread i holds bins bins-1-2i and bins-2-2i: the first whose running count from the top reaches need
    const int d0 = bins - 1 - 2 * tid, d1 = d0 - 1;
    const int h0 = d0 >= 0 ? hist[d0] : 0, h1 = d1 >= 0 ? hist[d1] : 0;
    int tot;
    const int before = block_scan(h0 + h1, warp_sums, tot);
    if (before < need && need <= before + h0 + h1) {
      const bool first = need <= before + h0;
      s_prefix = prefix | (uint32_t)(first ? d0 : d1) << shift;
      s_need = need - before - (first ? 0 : h0);
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // kept: sinks, recent ones, keys above the threshold, and the first `need` equal to it.  A thread takes
  // one contiguous run; its odd length spreads the lanes over the banks.
  const int per = ((L + kSel - 1) / kSel) | 1;
  const int i0 = min(tid * per, L), i1 = min(i0 + per, L);
  // 1: above the threshold, 2: equal to it
  auto judge = [&](int i) {
    if (i < lo || i >= hi) return 1;
    if (!any) return 0;
    const uint32_t k = key(i);
    return k > prefix ? 1 : k == prefix ? 2 : 0;
  };
  int above = 0, ties = 0;
  for (int i = i0; i < i1; ++i) {
    const int j = judge(i);
    above += j & 1;
    ties += j >> 1;
  }
  int tot;
  int tie = block_scan(ties, warp_sums, tot);
  const int taken = min(tie + ties, need) - min(tie, need);
  int out = block_scan(above + taken, warp_sums, tot);
  for (int i = i0; i < i1; ++i) {
    const int j = judge(i);
    if (j == 1 || (j == 2 && tie < need)) kept[out++] = i;
    tie += j >> 1;
  }
}

// The destination's cache row of a slot, -1 outside it.
__device__ __forceinline__ int64_t dst_row(const EvictArgs& a, int b, int slot) {
  if (!a.table_out) {
    const int64_t r = __ldcg(a.cu_k_out + b) + (int64_t)slot;
    return r < a.rows_out ? r : -1;
  }
  const int sh = __ffs(a.seqs.page_size) - 1, ps = slot >> sh;
  const int pg = ps < a.max_pages_out ? __ldg(a.table_out + (int64_t)b * a.max_pages_out + ps) : -1;
  return (unsigned)pg < (unsigned)a.num_pages_out
             ? ((int64_t)pg << sh) | (slot & (a.seqs.page_size - 1)) : -1;
}

constexpr int kMoveSmem = 200 * 1024;  // row slots of an SM

__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                   reinterpret_cast<uint64_t>(dst)),
               "r"(tc::smem_u32(src)), "r"(bytes)
               : "memory");
}

// A thread per row, each with a slot of shared memory and a barrier of its own.  Half of a warp's lanes work:
// lanes of a warp wait for the slowest of their rows, and 8 warps of 16 rows move 680 MB in 120 us where 4 warps of
// 32 took 135 (16 of 8 or 32 of 4: 122).
constexpr int kMoveLanes = 16;
__global__ void __launch_bounds__(256) evict_move_kernel(EvictArgs a) {
  extern __shared__ __align__(128) uint8_t slots[];
  __shared__ uint64_t bars[128];
  __shared__ int abort_flag;
  const int rb0 = a.row_bytes[0], rb1 = a.row_bytes[1], nsc = a.row_bytes[2];
  const bool on = (threadIdx.x & 31) < kMoveLanes;
  const int me = on ? (int)(threadIdx.x >> 5) * kMoveLanes + (int)(threadIdx.x & 31) : 0;
  const int rows = (int)(blockDim.x >> 5) * kMoveLanes;  // at most 128
  uint64_t* bar = &bars[me];
  uint8_t* slot_mem = slots + (int64_t)me * (rb0 + rb1);
  if (on) tc::mbar_init(bar, 1);
  if (threadIdx.x == 0) abort_flag = 0;
  tc::fence_barrier_init();
  __syncthreads();
  griddep_wait();
  if (!on) return;
  const int64_t total = (int64_t)a.seqs.B * a.budget;
  uint32_t phase = 0;
  for (int64_t w = (int64_t)blockIdx.x * rows + me; w < total;
       w += (int64_t)gridDim.x * rows) {
    const int b = (int)(w / a.budget), slot = (int)(w - (int64_t)b * a.budget);
    const int pos = __ldcg(a.kept + w);
    int64_t src = -1, dst = -1;
    if (pos >= 0) {
      src = key_row(a.seqs, b, __ldg(a.seqs.cu_k + b), pos);
      dst = dst_row(a, b, slot);
      if ((src < 0 || dst < 0) && rb0 + rb1 + nsc) {
        atomicOr(a.status, DSA_FLAG_BAD_SEQS);
        src = dst = -1;
      }
    }
    const bool move = src >= 0 && rb0 + rb1;
    if (move) {
      tc::mbar_arrive_expect_tx(bar, (uint32_t)(rb0 + rb1));
      if (rb0) tc::bulk_load(slot_mem, static_cast<const char*>(a.src[0]) + src * rb0, rb0, bar);
      if (rb1) tc::bulk_load(slot_mem + rb0, static_cast<const char*>(a.src[1]) + src * rb1, rb1, bar);
    }
    // acc of the kept positions, zero behind them (positions appended later start from nothing)
    if (a.acc_out) a.acc_out[b * a.ld_acc_out + slot] = pos >= 0 ? __ldg(a.acc + b * a.ld_acc + pos) : 0.f;
    if (src >= 0 && nsc) {  // 4 bytes, or up to 8 of E8M0
      const char* s = static_cast<const char*>(a.src[2]) + src * nsc;
      char* d = static_cast<char*>(a.dst[2]) + dst * nsc;
      if (nsc == 4) *reinterpret_cast<uint32_t*>(d) = *reinterpret_cast<const uint32_t*>(s);
      else
        for (int i = 0; i < nsc; ++i) d[i] = s[i];
    }
    if (move) {
      if (!tc::mbar_wait(bar, phase, &abort_flag, a.status, DSA_FLAG_TIMEOUT)) {
        tc::mbar_wait_drain(bar, phase);
        break;
      }
      phase ^= 1;
      if (rb0) bulk_store(static_cast<char*>(a.dst[0]) + dst * rb0, slot_mem, rb0);
      if (rb1) bulk_store(static_cast<char*>(a.dst[1]) + dst * rb1, slot_mem + rb0, rb1);
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the slot may be filled again
    }
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

}  // namespace

int launch_evict(EvictArgs a, cudaStream_t stream) {
  a.moves = a.row_bytes[0] || a.row_bytes[1] || a.row_bytes[2] || a.acc_out;
  cudaError_t e = cudaSuccess;
  if (a.seqs.max_k_len <= kSmemKeys) {
    const int smem = a.seqs.max_k_len * 4;
    static std::atomic<bool> allowed[64];
    const int rc = smem + 16384 <= 49152 ? DSA_OK
                                         : allow_smem<kSmemKeys * 4>(evict_select_kernel<true>, allowed, "evict_select: smem attribute");
    if (rc != DSA_OK) return rc;
    DSA_LAUNCH("evict_select", stream, e = launch_pdl(evict_select_kernel<true>, dim3(a.seqs.B), dim3(kSel), smem, stream, a));
  } else {
    DSA_LAUNCH("evict_select", stream, e = launch_pdl(evict_select_kernel<false>, dim3(a.seqs.B), dim3(kSel), 0, stream, a));
  }
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "evict_select: %s", cudaGetErrorString(e));
  const int rc = check_launch("evict_select");
  if (rc != DSA_OK) return rc;
  if (!a.moves) return DSA_OK;
  // row slots a block, blocks an SM: as many row slots as fit kMoveSmem (rows are at most 6 KB)
  const int64_t total = (int64_t)a.seqs.B * a.budget;
  const int rb = a.row_bytes[0] + a.row_bytes[1];
  int thr = 128;
  while (thr > kMoveLanes && thr * rb > kMoveSmem) thr -= kMoveLanes;
  const int smem = thr * rb, per_sm = rb ? kMoveSmem / smem : 8;
  const int64_t most = (int64_t)num_sms() * (per_sm < 8 ? per_sm : 8), blocks = (total + thr - 1) / thr;
  static std::atomic<bool> allowed[64];
  const int rc2 = smem <= 40960 ? DSA_OK : allow_smem<kMoveSmem>(evict_move_kernel, allowed, "evict_move: smem attribute");
  if (rc2 != DSA_OK) return rc2;
  DSA_LAUNCH("evict_move", stream,
             e = launch_pdl(evict_move_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(thr / kMoveLanes * 32), smem,
                            stream, a));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "evict_move: %s", cudaGetErrorString(e));
  return check_launch("evict_move");
}

}  // namespace dsa
