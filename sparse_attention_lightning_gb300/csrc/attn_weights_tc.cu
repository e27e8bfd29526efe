// dsa_accumulate_attn_weights on tcgen05 tensor cores (bf16, 64 <= D <= 576, up to 128 heads).
//
//   w[i] = Σ_h exp(scale · q[t,h,:]·kv[row_i,:] − lse[t,h])
//
// Bound by the gather (1152 B a selected row from anywhere in the cache), so shared memory is left to it: the
// query's heads are the MMA's M = 128 and live in tensor memory (288 columns), and three chunks of 64
// gathered rows (216 KB) are in flight on an SM.  (With the keys as M and the query in shared memory, 64 KB
// were: 34 us for the decode step below.)  The sum over heads is then one
// over lanes: a thread takes one head's 64 exponentials (of fp32 logits · scale − lse in one rounding, by the
// hardware's 2^x: some 2^-20 of a weight in all, for logits in the tens), 62 shuffles a warp transpose and add them, and
// the four warps' sums meet in shared memory.
//
// Per chunk of 64 selected rows: four producer warps gather them by TMA, four rows x 128 bytes a copy, into the
// swizzled operand layout; one thread issues S = Q·Kᵀ (M=128, N=64, K=D, A from tensor memory: 33 clocks a
// K-step); four warps take the exponentials from two logit buffers in turn.  The query block comes through
// the same ring as one or two chunks of 64 heads and is copied to tensor memory from there: read row by row
// from global memory (a thread a head, 1152 bytes apart) it took 16,000 clocks before the first MMA.
// Every CTA takes a contiguous share of all queries' chunks, so that few queries fill the SMs;
// where a share crosses queries, the query block is loaded again (see the launcher).  Every wait is bounded (DSA_FLAG_TIMEOUT).
// Decode step of 32 queries x 2048 rows of 1152 B, 128 heads: 18.7 us, 75.5 MB gathered at 5.9 TB/s once rows arrive;
// before that the first indices and the row's lookup (1.6 us), the query block and the first rows (2.4 us).  Prefetching
// the next chunk's rows to L2 while the query block has the ring did not change it.
#include "attn_weights.cuh"
#include "tc_sm100.cuh"

namespace dsa {
namespace {

using namespace tc;

constexpr int kN = 64;                 // selected rows of a chunk
constexpr int kTile = kN * 128;        // 8 KB: 64 rows x 64 columns
constexpr int kMaxTiles = 9;
constexpr int kStages = 3;
constexpr int kProducers = 4;          // warps
constexpr int kThreads = 32 * (kProducers + 1 + 4);
constexpr int kSums = 4;               // chunks whose sums the weights warps hold: buffers, and a barrier each
constexpr int kMetaBytes = kSums * 4 * kN * 4 + 256; // the warps' sums, barriers
constexpr int kSCol = 0, kQCol = 128;  // tensor memory: 2 x 64 logit columns, 288 query columns

constexpr int smem_bytes(int ntile) { return kStages * ntile * kTile + kMetaBytes + 1024; }

struct Params {
  WeightArgs a;
  uint32_t chunks; // of a query
  int ntile;       // column tiles
  uint32_t split;  // units a query's chunks are split into
  uint32_t per;    // consecutive units of a CTA
};

// Rows r0..r3, 64 columns from column c, to four consecutive 128-byte rows of shared memory.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* m, uint64_t* bar, int c, int r0, int r1,
                                            int r2, int r3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(smem_u32(bar))
      : "memory");
}

// The k-th piece of this CTA's units: chunks [c0, c1) of query row t; false past the end.
struct Piece {
  int t, c0, c1;
};
__device__ __forceinline__ bool piece_at(const Params& p, int k, Piece& pc) {
  // (32 bits: the launcher keeps the units below 2^31; 64-bit divisions took 0.6 us ahead of the first copy)
  const uint32_t tot = (uint32_t)p.a.seqs.total_q * p.split;
  const uint32_t x0 = blockIdx.x * (uint32_t)p.per, x1 = min(x0 + p.per, tot);
  const uint32_t t = x0 / p.split + k, r0 = t * p.split;
  if (r0 >= x1) return false;
  pc.t = (int)t;
  pc.c0 = k == 0 ? (int)((x0 - r0) * p.chunks / p.split) : 0;
  pc.c1 = (int)(min((uint32_t)p.split, x1 - r0) * p.chunks / p.split);
  return true;
}

// query_row_info by a whole warp: a 32-way search over cu_q, whose last round loads all that is needed of
// the sequence (one round of loads up to 32 sequences).
__device__ __forceinline__ bool warp_row_info(const WeightArgs& a, int t, int lane, RowInfo& r) {
  const Seqs& s = a.seqs;
  int lo = 0, hi = s.B;  // the last b with cu_q[b] <= t is in [lo, hi)
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32;
    const int probe = lo + lane * step;
    const bool le = probe < hi && (lane == 0 || s.cu_q[probe] <= t);
    const int m = 31 - __clz(__ballot_sync(0xffffffffu, le));
    lo += m * step;
    hi = min(hi, lo + step);
  }
  const int b = min(lo + lane, hi - 1);
  int q0 = s.cu_q[b], q1 = s.cu_q[b + 1], k0 = s.cu_k[b], k1 = s.cu_k[b + 1];
  const unsigned le = __ballot_sync(0xffffffffu, lo + lane < hi && (lane == 0 || q0 <= t));
  const int m = 31 - __clz(le);
  q0 = __shfl_sync(0xffffffffu, q0, m);
  q1 = __shfl_sync(0xffffffffu, q1, m);
  k0 = __shfl_sync(0xffffffffu, k0, m);
  k1 = __shfl_sync(0xffffffffu, k1, m);
  const int T = q1 - q0, L = k1 - k0;
  if (!(t >= q0 && t < q1 && T <= L && k0 >= 0 && k1 <= s.total_k && L <= s.max_k_len && q1 <= s.total_q &&
        T <= a.max_q_len)) {  // (the order of additions and fx_scale rest on max_q_len)
    atomicOr(a.status, DSA_FLAG_BAD_SEQS);
    return false;
  }
  r = RowInfo{lo + m, L - T + (t - q0), k0, L};
  return true;
}

// v[i] of all lanes added up for i = 0..31: lane l gets the sum of v[l] (31 shuffles: each step a lane
// keeps the half its bit selects).  The tree is the same for every i.
__device__ __forceinline__ float transpose_add(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o];
      const float keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return v[0];
}

__global__ void __launch_bounds__(kThreads, 1)
attn_weights_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap qmap,
                       const __grid_constant__ CUtensorMap kvmap) {
  // With sums, the kernel before this one clears them (waited for ahead of the first addition), and the one behind
  // it, which adds them to acc, may be set up meanwhile: it waits for this grid to end.  A caller's next
  // kernel may not: it may read what comes before it without waiting.
  if (p.a.fx) griddep_launch();
  else griddep_wait();
  const WeightArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* ring = smem;                                   // [3][ntile][64][128 B]
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + kStages * p.ntile * kTile);
  uint64_t* k_full = bars;          // [3] 4 producer warps, and their bytes
  uint64_t* k_empty = bars + 3;     // [3]
  uint64_t* s_full = bars + 6;      // [2]
  uint64_t* s_empty = bars + 8;     // [2] 4 warps
  uint64_t* q_full = bars + 10;     // 4 warps have stored the query
  uint64_t* drain = bars + 11;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 12);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 13);
  // [kSums] 4 warps have stored a chunk's sums.  A warp frees a chunk's logits before it stores its sums, so one that reads
  // none may be two chunks ahead of a reader that has yet to arrive for its own: with two barriers it would arrive in
  // that reader's place.  With four it comes back to the same one for chunk n + 4, whose logits need chunk
  // n + 2's freed by every warp, each of which has then passed chunk n.
  uint64_t* red_full = bars + 14;
  float* red = reinterpret_cast<float*>(bars + 14 + kSums);  // [kSums][4][64] the warps' sums

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) { mbar_init(&k_full[i], kProducers); mbar_init(&k_empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], 4); }
    mbar_init(q_full, 4);
    for (int i = 0; i < kSums; ++i) mbar_init(&red_full[i], 4);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kProducers) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int D = a.d;
  const int stage_bytes = p.ntile * kTile;
  const int qchunks = a.h > 64 ? 2 : 1;  // ring chunks of a query block

  if (warp < kProducers) {
    // ---------------- producers: 16 rows of a chunk each, four rows x 128 bytes a copy ----------------
    int slot = 0, phase = 1, n = 0;
    bool stop = false;
    Piece pc;
    for (int k = 0; !stop && piece_at(p, k, pc); ++k) {
      RowInfo ri;
      // lanes 0..15: this warp's entries, read two chunks ahead, and their pages, one chunk ahead
      auto load_idx = [&](int c) {
        const int i = c * kN + warp * 16 + lane;
        return lane < 16 && i < a.top_k ? a.idx[(int64_t)pc.t * a.top_k + i] : -1;
      };
      int v0 = load_idx(pc.c0), v1 = load_idx(pc.c0 + 1);
      // the query block, 64 heads a chunk of the ring (ahead of the row's lookup: it is consumed in any case)
      for (int c = 0; c < qchunks && !stop; ++c, ++n) {
        if (!__all_sync(0xffffffffu, mbar_wait(&k_empty[slot], phase, abort_flag, a.status, DSA_FLAG_TIMEOUT))) {
          stop = true;
          break;
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(&k_full[slot], (uint32_t)((p.ntile + 3 - warp) / kProducers * kTile));
          for (int t = warp; t < p.ntile; t += kProducers)
            tma_load_2d(ring + slot * stage_bytes + t * kTile, &qmap, &k_full[slot], t * 64, pc.t * a.h + c * kN);
        }
        __syncwarp();
        if (++slot == kStages) { slot = 0; phase ^= 1; }
      }
      if (stop) break;
      if (!warp_row_info(a, pc.t, lane, ri)) continue;
      const bool paged = a.seqs.paged();
      const int sh = paged ? __ffs(a.seqs.page_size) - 1 : 0;
      const int32_t* table = a.seqs.block_table + (int64_t)ri.b * a.seqs.max_pages;
      auto load_page = [&](int v) { return paged && v >= 0 && v <= ri.pos ? table[v >> sh] : 0; };
      int pg = load_page(v0);
      for (int c = pc.c0; c < pc.c1; ++c, ++n) {
        int row = -1;
        if (v0 >= 0 && v0 <= ri.pos) {
          if (!paged) row = ri.k0 + v0;
          else if ((unsigned)pg < (unsigned)a.seqs.num_pages) row = (pg << sh) | (v0 & (a.seqs.page_size - 1));
        }
        if (!dsa_check(row < a.seqs.cache_rows(), a.status)) row = -1;
        v0 = v1;
        pg = load_page(v0);
        v1 = load_idx(c + 2);
        // Four entries a copy.  Skipped entries repeat another of their four (their weight is dropped), and four
        // skipped ones copy nothing: standing in for padding with one fixed row made every SM ask for the same
        // lines (43 us instead of 21 for 86 queries, half of whose 500 entries were padding).
        const unsigned ok = __ballot_sync(0xffffffffu, row >= 0) & 0xffffu;
        const unsigned four = (ok >> (lane & 12)) & 15u;
        const int other = __shfl_sync(0xffffffffu, row, (lane & 12) + (four ? __ffs(four) - 1 : 0));
        if (row < 0) row = other;
        const int copies = __popc((ok | ok >> 1 | ok >> 2 | ok >> 3) & 0x1111u);
        int r[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = __shfl_sync(0xffffffffu, row, i);
        if (!__all_sync(0xffffffffu, mbar_wait(&k_empty[slot], phase, abort_flag, a.status, DSA_FLAG_TIMEOUT))) {
          stop = true;
          break;
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(&k_full[slot], (uint32_t)(copies * p.ntile * 512));
          uint8_t* dst = ring + slot * stage_bytes + warp * 16 * 128;
#pragma unroll
          for (int t = 0; t < kMaxTiles; ++t) {
            if (t >= p.ntile) break;
#pragma unroll
            for (int g = 0; g < 4; ++g)
              if ((ok >> (4 * g)) & 15u)
                tma_gather4(dst + t * kTile + g * 512, &kvmap, &k_full[slot], t * 64, r[4 * g], r[4 * g + 1],
                          r[4 * g + 2], r[4 * g + 3]);
          }
        }
        __syncwarp();
        if (++slot == kStages) { slot = 0; phase ^= 1; }
      }
    }
    // every copy issued has landed before the CTA may exit
    for (int i = max(0, n - kStages); i < n; ++i) mbar_wait_drain(&k_full[i % kStages], (i / kStages) & 1);
  } else if (warp == kProducers) {
    // ---------------- MMA issue: the warp walks the pieces, one lane issues ----------------
    const uint32_t idesc = idesc_bf16(128, kN);
    const uint64_t kd0 = sdesc_sw128(smem_u32(ring), 16, 1024);
    int slot = 0, phase = 0, n = 0, qn = 0;
    bool stop = false;
    Piece pc;
    for (int k = 0; !stop && piece_at(p, k, pc); ++k) {
      RowInfo ri;
      const bool ok = warp_row_info(a, pc.t, lane, ri);
      if (!__all_sync(0xffffffffu, mbar_wait(q_full, qn & 1, abort_flag, a.status, DSA_FLAG_TIMEOUT))) break;
      ++qn;
      for (int c = 0; c < qchunks; ++c) {  // the query has left the ring for tensor memory
        if (lane == 0) mbar_arrive(&k_empty[slot]);
        if (++slot == kStages) { slot = 0; phase ^= 1; }
      }
      for (int c = pc.c0; ok && c < pc.c1; ++c, ++n) {
        if (!__all_sync(0xffffffffu,
                        mbar_wait(&s_empty[n & 1], ((n >> 1) & 1) ^ 1, abort_flag, a.status, DSA_FLAG_TIMEOUT) &&
                            mbar_wait(&k_full[slot], phase, abort_flag, a.status, DSA_FLAG_TIMEOUT))) {
          stop = true;
          break;
        }
        if (elect_one()) {
          tc_fence_after();
          const uint32_t d = tmem + kSCol + (n & 1) * kN;
          const uint64_t kd = kd0 + (uint64_t)(slot * (stage_bytes >> 4));
#pragma unroll
          for (int t = 0; t < kMaxTiles; ++t) {
            if (t * 64 >= D) break;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (t * 64 + i * 16 < D)
                mma_bf16_ts(d, tmem + kQCol + t * 32 + i * 8, kd + (uint64_t)(t * (kTile >> 4) + i * 2), idesc,
                            t || i ? 1u : 0u);
          }
          mma_commit(&k_empty[slot]);
          mma_commit(&s_full[n & 1]);
        }
        __syncwarp();
        if (++slot == kStages) { slot = 0; phase ^= 1; }
      }
    }
    if (elect_one()) {
      mma_commit(drain);
      mbar_wait_drain(drain, 0);
    }
    __syncwarp();
  } else {
    // ---------------- weights: thread = head ----------------
    const int quarter = warp & 3, h = quarter * 32 + lane;
    const int et = threadIdx.x - 32 * (kProducers + 1);  // 0..127
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    int n = 0, slot = 0, phase = 0;
    bool stop = false;
    Piece pc;
    for (int k = 0; !stop && piece_at(p, k, pc); ++k) {
      RowInfo ri;
      const bool ok = warp_row_info(a, pc.t, lane, ri);
      // this warp's 32 heads of the query block, from the ring to tensor memory (the previous piece's
      // logits are complete: its last chunk has been read)
      const int qc = quarter >> 1;
      int qslot = slot + qc, qphase = phase;
      if (qslot >= kStages) { qslot -= kStages; qphase ^= 1; }
      if (qc < qchunks) {
        if (!__all_sync(0xffffffffu, mbar_wait(&k_full[qslot], qphase, abort_flag, a.status, DSA_FLAG_TIMEOUT))) break;
        const int r = (quarter & 1) * 32 + lane;  // row of the chunk
        const uint8_t* from = ring + qslot * stage_bytes + r * 128;
#pragma unroll 3
        for (int t = 0; t < p.ntile; ++t) {
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(from + t * kTile + ((i ^ (r & 7)) * 16));
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
          }
          tmem_st32(lane_base + kQCol + t * 32, w);
        }
      }
      int lslot = slot + qchunks - 1, lphase = phase;  // the query block's last chunk
      if (lslot >= kStages) { lslot -= kStages; lphase ^= 1; }
      slot += qchunks + (ok ? pc.c1 - pc.c0 : 0);  // the piece's place in the ring is passed
      phase ^= (slot / kStages) & 1;
      slot %= kStages;
      const int64_t flat = (int64_t)pc.t * a.h + min(h, a.h - 1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      if (!ok) {
        // No logits follow to wait for, and a warp that went on could arrive for the next query before the others
        // have for this one: the MMA warp releases the block once all four have.
        if (!__all_sync(0xffffffffu, mbar_wait(&k_empty[lslot], lphase, abort_flag, a.status, DSA_FLAG_TIMEOUT))) break;
        continue;
      }
      griddep_wait();  // the sums are zero (and written: the kernels behind this one wait for it alone)
      const float lse = h < a.h ? a.lse[flat] : -INFINITY;
      const bool dead = lse == -INFINITY;  // no such head, or it attended to nothing: it adds nothing
      const float lse2 = dead ? 0.f : lse * kLog2e;
      for (int c = pc.c0; c < pc.c1; ++c, ++n) {
        // threads 0..63 add up and store one selected position each
        int pos = -1;
        if (et < kN) {
          const int i = c * kN + et;
          const int v = i < a.top_k ? a.idx[(int64_t)pc.t * a.top_k + i] : -1;
          if (v >= 0 && v <= ri.pos && cache_row(a.seqs, ri.b, ri.k0, v) >= 0) pos = v;
          else if (v != -1) atomicOr(a.status, DSA_FLAG_BAD_INDEX);
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&s_full[n & 1], (n >> 1) & 1, abort_flag, a.status,
                                               DSA_FLAG_TIMEOUT))) { stop = true; break; }
        tc_fence_after();
        float* mine = red + (n % kSums) * (4 * kN) + quarter * kN;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t s[32];
          __syncwarp();
          tmem_ld32(lane_base + kSCol + (n & 1) * kN + half * 32, s);
          if (half == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[n & 1]);
          }
          float x[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float e = ex2(fmaf(__uint_as_float(s[i]), a.scale_log2, -lse2));
            x[i] = dead ? 0.f : e;
          }
          mine[half * 32 + lane] = transpose_add(x, lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&red_full[n % kSums]);
        if (et >= kN) continue;
        if (!__all_sync(0xffffffffu, mbar_wait(&red_full[n % kSums], (n / kSums) & 1, abort_flag, a.status,
                                               DSA_FLAG_TIMEOUT))) { stop = true; break; }
        if (pos >= 0) {
          const float* r = red + (n % kSums) * (4 * kN) + et;
          add_weight(a, ri.b, pos, (r[0] + r[kN]) + (r[2 * kN] + r[3 * kN]));
        }
      }
    }
    griddep_wait();
  }
  tc_fence_before();
  cta_sync();
  if (warp == kProducers) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

bool attn_weights_tc_eligible(const WeightArgs& a) {
  return a.kv_dtype == DSA_BF16 && a.d >= 64 && a.d <= 64 * kMaxTiles && a.h <= 128;
}

int launch_attn_weights_tc(const WeightArgs& a, cudaStream_t stream) {
  Params p{};
  p.a = a;
  p.ntile = (a.d + 63) / 64;
  // Shares.  A query block costs about two chunks each time a CTA loads one (it comes through the ring).  So queries
  // are split into units, and a CTA takes `per` consecutive ones: the fewest chunks and query blocks a CTA.
  // (Contiguous equal shares of all chunks: 32 queries x 32 chunks on 152 SMs are 7 chunks and two queries for 31 of
  // them, which end 3 us behind the others; 4 CTAs a query with 8 chunks each end together.)
  const int64_t chunks = (a.top_k + kN - 1) / kN;
  int64_t best = -1;
  for (int64_t s = 1; s <= chunks; ++s) {
    const int64_t units = a.seqs.total_q * s, n = (units + num_sms() - 1) / num_sms();
    if (s > 1 && units >= int64_t(1) << 30) break;
    const int64_t blocks = s % n == 0 ? 1 : n % s == 0 ? n / s : (n - 2) / s + 2;
    const int64_t cost = (n * chunks + s - 1) / s + 2 * blocks;
    if (best < 0 || cost < best) {
      best = cost;
      p.split = (uint32_t)s;
      p.per = (uint32_t)n;
    }
  }
  p.chunks = (uint32_t)chunks;
  const int grid = (int)(((int64_t)a.seqs.total_q * p.split + p.per - 1) / p.per);
  const int smem = smem_bytes(p.ntile);
  CUtensorMap qmap, kvmap;
  int rc = make_tmap_2d(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, (uint64_t)a.d,
                        (uint64_t)a.seqs.total_q * a.h, (uint64_t)a.d * 2, 64, kN);
  if (rc != DSA_OK) return rc;
  rc = make_tmap_2d(&kvmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv, (uint64_t)a.d,
                        (uint64_t)a.seqs.cache_rows(), (uint64_t)a.d * 2, 64, 1);
  if (rc != DSA_OK) return rc;
  static std::atomic<bool> allowed[64];
  rc = allow_smem<smem_bytes(kMaxTiles)>(attn_weights_tc_kernel, allowed, "attn_weights_tc: smem attribute");
  if (rc != DSA_OK) return rc;
  cudaError_t e = cudaSuccess;
  DSA_LAUNCH("attn_weights_tc", stream,
             e = launch_pdl(attn_weights_tc_kernel, dim3(grid), dim3(kThreads), smem, stream, p, qmap, kvmap));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "attn_weights_tc: %s", cudaGetErrorString(e));
  return check_launch("attn_weights_tc");
}

}  // namespace dsa
