// Sparse attention over the 4-bit latent cache on tcgen05 tensor cores (bf16 queries, 512 + 64 columns, up to 128 heads).
//
//   S_i = scale · q[t,h,:]·kv[row_i, :],  out = Σ softmax(S)_i · kv[row_i, :512],  lse = log Σ exp S_i
//
// A query's heads are the MMA's M = 128 rows.  A 128 x 512 fp32 accumulator is all of the tensor memory, so a CTA accumulates
// 256 output columns, two CTAs a query, each with the whole logits: 576 + 256 columns of MMA a CTA where 544 would do, without
// an exchange between SMs.  The twin finds the rows in L2.  Few queries are cut into pieces of their entries, merged
// afterwards.
//
// Eight warps gather and decode.  A row is 416 bytes, so the gather is a third of what bf16 rows take and goes through
// registers, kAhead chunks of 64 entries ahead: a lane takes one row (eight rows a warp) and, of it, 16-byte pieces 64 bytes apart,
// and stores what they decode to in the MMA's operand layout.  A quarter warp's eight lanes hold eight different rows, whose 16-byte
// stores the 128-byte swizzle spreads over all banks.  Decoding is two shifts, two logical operations and a product for
// a pair of columns (kv4.cuh): the operand is the value times 2^-16, exactly, which the logits' scale and the output make good;
// rope columns get the same factor.  Some 400 instructions a lane and chunk, 800 of a scheduler's ~2,100 clocks.
//
// Shared memory: five query tiles (80 KB) and two chunks of nine tiles of [64 keys x 64 columns] (144 KB).  A chunk's
// five "K tiles" (the other half's columns and the rope) are free again once its logits are done, its four "V tiles" (the CTA's own
// columns) after P·V, half a chunk later.  Tensor memory: O (256 columns), two logit buffers (64; P, as bf16 pairs, overwrites
// the first half of its own logits), the query columns that match the V tiles (128).
//
// One thread issues S(g) over the K tiles and half the V tiles, P(g-1)·V, and the other half of S(g): softmax has the
// first part to finish in, and the last hides the wait for P·V before the next chunk overwrites its P.  Four softmax warps, a
// thread a head: the running max moves only when a row's grows by more than 2^8 (O is then rescaled), the sum is in fp32 of
// the unrounded p.  P is rounded to bf16, which the MMA wants beside bf16 values: 2^-8 of each p at most, in either
// direction.  Every wait is bounded (DSA_FLAG_TIMEOUT).
#include <float.h>

#include "kv4.cuh"
#include "tc_sm100.cuh"

namespace dsa {
namespace {

using namespace tc;

constexpr int kM = 128;                    // heads
constexpr int kN = 64;                     // entries of a chunk
constexpr int kTile = kN * 128;            // 8 KB: 64 keys x 64 columns
constexpr int kQTile = kM * 128;           // 16 KB
constexpr int kVT = 4, kKT = 5;            // V and K tiles of a chunk
constexpr int kSlot = (kVT + kKT) * kTile; // 72 KB
constexpr int kDecoders = 8;               // warps
constexpr int kSoftWarps = 4;
constexpr int kThreads = 32 * (kSoftWarps + kDecoders + 1);
constexpr int kMmaWarp = kSoftWarps + kDecoders;
constexpr int kAhead = 1;                  // chunks whose rows are in flight ahead of the one being decoded
constexpr int kBarBytes = 512;
constexpr int kSmem = kKT * kQTile + 2 * kSlot + kBarBytes + 1024;
constexpr int kOCol = 0, kSCol = 256, kQCol = 384;
constexpr int kDc = 512, kDr = 64, kD = kDc + kDr;
constexpr int kRow = kv4_row_bytes(kDc, kDr);
constexpr int kRopeAt = kv4_rope_at(kDc), kScaleAt = kv4_scale_at(kDc, kDr);
constexpr float kRescaleLog2 = 8.0f;
static_assert(kSmem <= 232448, "shared memory");
static_assert(kVT * kQTile <= kSlot, "the query passes through the second chunk's tiles");
static_assert(kM * (256 * 4 + 16) <= 2 * kSlot, "the output leaves through the key tiles");

struct Params {
  Attn4Args a;
  int chunks;  // of a query
};

// kv4_query_row by a whole warp: a 32-way search over cu_q, whose last round loads all that is needed of the
// sequence (one round of loads up to 32 sequences).
__device__ __forceinline__ bool warp_query_row(const Attn4Args& a, int t, int lane, RowInfo& r) {
  const Seqs& s = a.seqs;
  int lo = 0, hi = s.B;  // the last b with cu_q[b] <= t is in [lo, hi)
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32, probe = lo + lane * step;
    const bool le = probe < hi && (lane == 0 || s.cu_q[probe] <= t);
    lo += (31 - __clz(__ballot_sync(0xffffffffu, le))) * step;
    hi = min(hi, lo + step);
  }
  const int b = min(lo + lane, hi - 1);
  int q0 = s.cu_q[b], q1 = s.cu_q[b + 1], k0 = s.cu_k[b], k1 = s.cu_k[b + 1];
  const int m = 31 - __clz(__ballot_sync(0xffffffffu, lo + lane < hi && (lane == 0 || q0 <= t)));
  q0 = __shfl_sync(0xffffffffu, q0, m);
  q1 = __shfl_sync(0xffffffffu, q1, m);
  k0 = __shfl_sync(0xffffffffu, k0, m);
  k1 = __shfl_sync(0xffffffffu, k1, m);
  const int T = q1 - q0, L = k1 - k0;
  if (!(t >= q0 && t < q1 && T <= L && k0 >= 0 && k1 <= s.total_k && L <= s.max_k_len && q0 >= 0 &&
        q1 <= s.total_q && T <= a.max_q_len)) {
    atomicOr(a.status, DSA_FLAG_BAD_SEQS);
    return false;
  }
  r = RowInfo{lo + m, L - T + (t - q0), k0, L};
  return true;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// A lane's share of one row: of the K and the V columns two pieces of 32 columns with their scales each, and two pieces of 8 rope
// columns.
struct Share {
  uint4 k[2], v[2], rope[2];
  uint16_t ks[2], vs[2];
  bool ok;
};

// 32 columns into four 16-byte pieces of a tile row, from logical piece c on.
__device__ __forceinline__ void decode32(uint8_t* row, int c, int x, const uint4& w, uint32_t scales) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  const uint32_t s[2] = {kv4_scale_pair(scales & 0xffu), kv4_scale_pair(scales >> 8)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t f = s[i >> 1];
    *reinterpret_cast<uint4*>(row + (((c + i) ^ x) * 16)) =
        make_uint4(mul_bf16x2(kv4_pair<0>(u[i]), f), mul_bf16x2(kv4_pair<1>(u[i]), f),
                   mul_bf16x2(kv4_pair<2>(u[i]), f), mul_bf16x2(kv4_pair<3>(u[i]), f));
  }
}

// 64 consecutive tensor-memory columns of this warp's 32 lanes.
__device__ __forceinline__ void load_row(uint32_t taddr, float (&s)[kN]) {
  uint32_t r[32];
  tmem_ld32(taddr, r);
#pragma unroll
  for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(r[i]);
  tmem_ld32(taddr + 32, r);
#pragma unroll
  for (int i = 0; i < 32; ++i) s[32 + i] = __uint_as_float(r[i]);
}

__global__ void __launch_bounds__(kThreads, 1)
attn4_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap qmap) {
  griddep_wait();
  const Attn4Args& a = p.a;
  if (a.splits > 1) griddep_launch();  // the merge may be set up meanwhile; it waits for this grid to end
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = blockIdx.x & 1, piece = (int)((blockIdx.x >> 1) % (uint32_t)a.splits);
  const int t = (int)((blockIdx.x >> 1) / (uint32_t)a.splits);
  const int64_t rows_all = (int64_t)a.seqs.total_q * a.h, row0 = (int64_t)t * a.h;
  const bool split = a.splits > 1;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* qs = smem;                           // [5][128][128 B]
  uint8_t* slots = qs + kKT * kQTile;           // [2][4 V tiles, 5 K tiles]
  uint64_t* bars = reinterpret_cast<uint64_t*>(slots + 2 * kSlot);
  uint64_t* k_full = bars;         // [2] 8 warps have stored the K tiles
  uint64_t* k_empty = bars + 2;    // [2] multiplied
  uint64_t* v_full = bars + 4;     // [2]
  uint64_t* v_empty = bars + 6;    // [2]
  uint64_t* s_full = bars + 8;     // [2] logits of the buffer's chunk complete
  uint64_t* p_full = bars + 10;    // [2] the softmax warps have written P
  uint64_t* pv_done = bars + 12;   // [2]
  uint64_t* q_full = bars + 14;    // the query tiles in shared memory
  uint64_t* q_staged = bars + 15;  // those on their way to tensor memory
  uint64_t* qt_full = bars + 16;   // the query columns in tensor memory
  uint64_t* drain = bars + 17;
  uint8_t* valid = reinterpret_cast<uint8_t*>(bars + 18);  // [2][8] a bit an entry that is not skipped
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 20);
  int* last_chunk = reinterpret_cast<int*>(bars + 21);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 22);

  const int live_warps = (a.h + 31) / 32;  // of the softmax: the others' rows are no head's
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], kDecoders);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], kDecoders);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], live_warps);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_staged, 1);
    mbar_init(qt_full, live_warps);
    mbar_init(drain, 1);
    *last_chunk = -1;
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  RowInfo ri;
  const bool good = warp_query_row(a, t, lane, ri);
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int c0 = (int)((int64_t)p.chunks * piece / a.splits), c1 = (int)((int64_t)p.chunks * (piece + 1) / a.splits);
  const int32_t* idx = a.idx + (int64_t)t * a.top_k;
  const int end = min(a.top_k, c1 * kN);
  if (good) {
    // the piece ends with its last chunk that is not all padding (a short history's row is mostly -1)
    int last = -1;
    for (int i = c0 * kN + (int)threadIdx.x; i < end; i += kThreads)
      if (idx[i] != -1) last = i / kN;
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0 && last >= 0) atomicMax(last_chunk, last);
  }
  cta_sync();
  const int nch = good ? max(0, *last_chunk + 1 - c0) : 0;

  // half h: its V tiles are column tiles 4h .. 4h + 3; the K tiles the other four and the rope's
  const int vt0 = half * kVT;
  auto ktile = [&](int j) { return j < vt0 ? j : j + kVT; };
  if (nch == 0) {
    // no entries: nothing, or zeros
    for (int i = threadIdx.x; good && i < a.h; i += kThreads) {
      if (half) continue;
      if (split) a.part_ml[(int64_t)piece * rows_all + row0 + i] = make_float2(-INFINITY, 0.f);
      else if (a.lse) a.lse[row0 + i] = -INFINITY;
    }
    const int per = a.out_dtype == DSA_F32 ? 64 : 32;  // 16-byte pieces of the row's half
    for (int i = threadIdx.x; good && !split && i < a.h * per; i += kThreads)
      reinterpret_cast<uint4*>(a.out)[(row0 + i / per) * (2 * per) + half * per + i % per] = make_uint4(0u, 0u, 0u, 0u);
  } else if (warp == kMmaWarp) {
    // ---------------- query loads, MMA issue ----------------
    if (elect_one()) {
      mbar_arrive_expect_tx(q_staged, kVT * kQTile);
      for (int j = 0; j < kVT; ++j) tma_load_2d(slots + kSlot + j * kQTile, &qmap, q_staged, (vt0 + j) * 64, (int)row0);
      mbar_arrive_expect_tx(q_full, kKT * kQTile);
      for (int j = 0; j < kKT; ++j) tma_load_2d(qs + j * kQTile, &qmap, q_full, ktile(j) * 64, (int)row0);
      const uint32_t idesc_s = idesc_bf16(kM, kN), idesc_pv = idesc_bf16(kM, 256, false, true);
      const uint64_t qd = sdesc_sw128(smem_u32(qs), 16, 1024);
      const uint64_t vd0 = sdesc_sw128(smem_u32(slots), 16, 1024);
      const uint64_t kd0 = sdesc_sw128(smem_u32(slots) + kVT * kTile, 16, 1024);
      const uint64_t pd0 = sdesc_sw128(smem_u32(slots), kTile, 1024);  // V tiles as P·V reads them
      bool stop = !mbar_wait(qt_full, 0, abort_flag, a.status, DSA_FLAG_TIMEOUT) ||
                  !mbar_wait(q_full, 0, abort_flag, a.status, DSA_FLAG_TIMEOUT);
      tc_fence_after();
      // a barrier is tested ahead of the MMAs that come before its use, and waited for only where it was not complete
      auto test = [&](uint64_t* bar, uint32_t parity) { return mbar_test(smem_u32(bar), parity); };
      auto sure = [&](bool ready, uint64_t* bar, uint32_t parity) {
        return ready || mbar_wait(bar, parity, abort_flag, a.status, DSA_FLAG_TIMEOUT);
      };
      auto pv = [&](int g, bool ready) -> bool {
        const int s = g & 1;
        if (!sure(ready, &p_full[s], (g >> 1) & 1)) return false;
        tc_fence_after();
        const uint32_t pa = tmem + kSCol + s * kN;
        const uint64_t b0 = pd0 + (uint64_t)(s * (kSlot >> 4));
        const uint32_t acc = g > 0;
#pragma unroll
        for (int kk = 0; kk < kN / 16; ++kk)
          mma_bf16_ts(tmem + kOCol, pa + kk * 8, b0 + (uint64_t)(kk * 128), idesc_pv, kk ? 1u : acc);
        mma_commit(&v_empty[s]);
        mma_commit(&pv_done[s]);
        return true;
      };
      for (int g = 0; g < nch && !stop; ++g) {
        const int s = g & 1;
        const uint32_t par = (g >> 1) & 1;
        bool ready = test(&k_full[s], par);
        // the buffer's last P (chunk g - 2) has been read
        if (g >= 2 && !mbar_wait(&pv_done[s], par ^ 1, abort_flag, a.status, DSA_FLAG_TIMEOUT)) break;
        if (!sure(ready, &k_full[s], par)) break;
        tc_fence_after();
        ready = test(&v_full[s], par);
        const uint32_t d = tmem + kSCol + s * kN;
        const uint64_t kd = kd0 + (uint64_t)(s * (kSlot >> 4)), vd = vd0 + (uint64_t)(s * (kSlot >> 4));
#pragma unroll
        for (int j = 0; j < kKT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_bf16(d, qd + (uint64_t)(j * (kQTile >> 4) + i * 2), kd + (uint64_t)(j * (kTile >> 4) + i * 2), idesc_s,
                     j || i ? 1u : 0u);
        mma_commit(&k_empty[s]);
        if (!sure(ready, &v_full[s], par)) break;
        tc_fence_after();
        ready = g > 0 && test(&p_full[s ^ 1], ((g - 1) >> 1) & 1);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_bf16_ts(d, tmem + kQCol + j * 32 + i * 8, vd + (uint64_t)(j * (kTile >> 4) + i * 2), idesc_s, 1u);
        if (g > 0 && !pv(g - 1, ready)) break;
#pragma unroll
        for (int j = 2; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_bf16_ts(d, tmem + kQCol + j * 32 + i * 8, vd + (uint64_t)(j * (kTile >> 4) + i * 2), idesc_s, 1u);
        mma_commit(&s_full[s]);
        if (g == nch - 1) pv(g, false);
      }
      mma_commit(drain);
      mbar_wait_drain(drain, 0);
      // every copy issued has landed before the CTA may exit
      mbar_wait_drain(q_staged, 0);
      mbar_wait_drain(q_full, 0);
    }
  } else if (warp >= kSoftWarps) {
    // ---------------- gather and decode ----------------
    const int w = warp - kSoftWarps, x = lane & 7, sub = lane >> 3;  // row of the chunk w · 8 + x
    const int r = w * 8 + x;
    const bool paged = a.seqs.paged();
    const int sh = paged ? __ffs(a.seqs.page_size) - 1 : 0;
    const int32_t* table = a.seqs.block_table + (int64_t)ri.b * a.seqs.max_pages;
    auto load_idx = [&](int g) {
      const int i = (c0 + g) * kN + r;
      return i < end ? idx[i] : -1;
    };
    auto load_page = [&](int v) { return paged && v >= 0 && v <= ri.pos ? table[v >> sh] : 0; };
    // the row of chunk g's entry v with its page pg, and its loads
    auto fetch = [&](int v, int pg, Share& f) {
      int row = -1;
      if (v >= 0 && v <= ri.pos) {
        if (!paged) row = ri.k0 + v;
        else if ((unsigned)pg < (unsigned)a.seqs.num_pages) row = (pg << sh) | (v & (a.seqs.page_size - 1));
      }
      if (row < 0 && v != -1) atomicOr(a.status, DSA_FLAG_BAD_INDEX);
      if (!dsa_check(row < a.seqs.cache_rows(), a.status)) row = -1;
      f.ok = row >= 0;
      if (!f.ok) {  // zeros: its P is 0, and its columns have to be finite
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          f.k[i] = f.v[i] = f.rope[i] = make_uint4(0u, 0u, 0u, 0u);
          f.ks[i] = f.vs[i] = 0;
        }
        return;
      }
      const uint8_t* src = a.kv4 + (int64_t)row * kRow;
      const int kp = (1 - half) * 8 + sub, vp = half * 8 + sub;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f.k[i] = *reinterpret_cast<const uint4*>(src + (kp + 4 * i) * 16);
        f.ks[i] = *reinterpret_cast<const uint16_t*>(src + kScaleAt + (kp + 4 * i) * 2);
        f.rope[i] = *reinterpret_cast<const uint4*>(src + kRopeAt + (sub + 4 * i) * 16);
        f.v[i] = *reinterpret_cast<const uint4*>(src + (vp + 4 * i) * 16);
        f.vs[i] = *reinterpret_cast<const uint16_t*>(src + kScaleAt + (vp + 4 * i) * 2);
      }
    };
    Share f[kAhead + 1];
    int v1 = load_idx(0), v2 = load_idx(1);  // (past the piece: -1)
    int pg1 = load_page(v1);
    static_assert(kAhead == 1, "");
    fetch(v1, pg1, f[0]);
    v1 = v2;
    pg1 = load_page(v1);
    v2 = load_idx(2);
    bool stop = false;
    for (int g0 = 0; g0 < nch && !stop; g0 += kAhead + 1) {
#pragma unroll
      for (int u = 0; u <= kAhead; ++u) {
        const int g = g0 + u;
        if (g >= nch) break;
        const Share& now = f[u];
        // the next chunk's rows, the pages of the one after it, the entries of the one after that
        if (g + kAhead < nch) fetch(v1, pg1, f[(u + kAhead) % (kAhead + 1)]);
        v1 = v2;
        pg1 = load_page(v1);
        v2 = load_idx(g + kAhead + 2);
        const int s = g & 1;
        const uint32_t par = (g >> 1) & 1;
        uint8_t* tiles = slots + s * kSlot;
        // (the second chunk's tiles bring the query first)
        if (!__all_sync(0xffffffffu, (g != 1 || mbar_wait(qt_full, 0, abort_flag, a.status, DSA_FLAG_TIMEOUT)) &&
                                         mbar_wait(&k_empty[s], par ^ 1, abort_flag, a.status, DSA_FLAG_TIMEOUT))) {
          stop = true;
          break;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          decode32(tiles + (kVT + 2 * i + (sub >> 1)) * kTile + r * 128, (sub & 1) * 4, x, now.k[i], now.ks[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          constexpr uint32_t kShrink = 0x37803780u;  // 2^-16 twice
          *reinterpret_cast<uint4*>(tiles + (kVT + kKT - 1) * kTile + r * 128 + (((sub + 4 * i) ^ x) * 16)) =
              make_uint4(mul_bf16x2(now.rope[i].x, kShrink), mul_bf16x2(now.rope[i].y, kShrink),
                         mul_bf16x2(now.rope[i].z, kShrink), mul_bf16x2(now.rope[i].w, kShrink));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[s]);
        if (!__all_sync(0xffffffffu, mbar_wait(&v_empty[s], par ^ 1, abort_flag, a.status, DSA_FLAG_TIMEOUT))) {
          stop = true;
          break;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          decode32(tiles + (2 * i + (sub >> 1)) * kTile + r * 128, (sub & 1) * 4, x, now.v[i], now.vs[i]);
        const uint32_t m = __ballot_sync(0xffffffffu, now.ok);
        if (lane == 0) valid[s * 8 + w] = (uint8_t)m;  // (softmax has read the chunk before's: its P has been multiplied)
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[s]);
      }
    }
  } else if (warp < live_warps) {
    // ---------------- softmax: thread = head ----------------
    const int r = warp * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    bool stop = !__all_sync(0xffffffffu, mbar_wait(q_staged, 0, abort_flag, a.status, DSA_FLAG_TIMEOUT));
    if (!stop) {
#pragma unroll
      for (int j = 0; j < kVT; ++j) {
        const uint8_t* from = slots + kSlot + j * kQTile + r * 128;
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(from + ((i ^ (r & 7)) * 16));
          w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
        tmem_st32(lane_base + kQCol + j * 32, w);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(qt_full);
    }
    const float scale = a.scale_log2 * (1.f / kKv4Shrink);
    float m = -INFINITY, l = 0.f;  // the reference (log2 units) and the sum relative to it
    for (int g = 0; g < nch && !stop; ++g) {
      const int s = g & 1;
      const uint32_t par = (g >> 1) & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&s_full[s], par, abort_flag, a.status, DSA_FLAG_TIMEOUT) &&
                                       mbar_wait(&v_full[s], par, abort_flag, a.status, DSA_FLAG_TIMEOUT))) {
        stop = true;
        break;
      }
      tc_fence_after();
      const uint64_t see = *reinterpret_cast<volatile uint64_t*>(valid + s * 8);
      const uint32_t sbuf = lane_base + kSCol + s * kN;
      float z[kN];
      load_row(sbuf, z);
      if (see != ~0ull) {
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (!((see >> i) & 1)) z[i] = -INFINITY;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < kN; ++i) mx[i & 3] = fmaxf(mx[i & 3], z[i]);
      const float mc = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
      const bool grow = mc > m + kRescaleLog2;  // the first entries always (m = -inf)
      if (__any_sync(0xffffffffu, grow)) {
        const float m_new = grow ? mc : m;
        const float factor = grow ? ex2(m - m_new) : 1.f;
        l *= factor;
        if (g > 0) {
          // O holds the chunks before g at the old reference: rescale it once P·V(g - 1) is in
          if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[s ^ 1], ((g - 1) >> 1) & 1, abort_flag, a.status,
                                                 DSA_FLAG_TIMEOUT))) { stop = true; break; }
          tc_fence_after();
          __syncwarp();
          for (int b = 0; b < 8; ++b) {
            uint32_t o[32];
            tmem_ld32(lane_base + kOCol + 32 * b, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
            tmem_st32(lane_base + kOCol + 32 * b, o);
          }
        }
        m = m_new;
      }
      const float ref = m == -INFINITY ? 0.f : m;  // nothing visible so far
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t pk[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float p0 = ex2(fmaf(z[2 * i], scale, -ref));
        const float p1 = ex2(fmaf(z[2 * i + 1], scale, -ref));
        sum[(2 * i) & 3] += p0;
        sum[(2 * i + 1) & 3] += p1;
        pk[i] = bf16x2(p0, p1);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      __syncwarp();
      tmem_st32(sbuf, pk);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[s]);
    }
    if (!stop)
      stop = !__all_sync(0xffffffffu, mbar_wait(&pv_done[(nch - 1) & 1], ((nch - 1) >> 1) & 1, abort_flag, a.status,
                                                DSA_FLAG_TIMEOUT));
    if (!stop) {
      tc_fence_after();
      // O goes out through the key tiles (all of them have been multiplied): a thread writes its row there, 16 bytes more
      // than its length apart from the next, and sends it with one bulk copy
      const bool live = r < a.h;
      const float inv = (split ? 1.f : (l == 0.f ? 0.f : 1.f / l)) * (1.f / kKv4Shrink);
      const bool f32 = split || a.out_dtype == DSA_F32;
      const int row_bytes = 256 * (f32 ? 4 : 2);
      uint8_t* mine = slots + r * (row_bytes + 16);
      for (int b = 0; b < 8; ++b) {
        uint32_t o[32];
        __syncwarp();  // the load is the whole warp's
        tmem_ld32(lane_base + kOCol + 32 * b, o);
        if (f32) {
          float4* dst = reinterpret_cast<float4*>(mine) + 8 * b;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(__uint_as_float(o[4 * i]) * inv, __uint_as_float(o[4 * i + 1]) * inv,
                                 __uint_as_float(o[4 * i + 2]) * inv, __uint_as_float(o[4 * i + 3]) * inv);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(mine) + 4 * b;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = bf16x2(__uint_as_float(o[8 * i + 2 * e]) * inv, __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
            dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      fence_proxy_async_smem();  // our writes, seen by the bulk copy
      if (live) {
        const int64_t at = (row0 + r) * kDc + half * 256;
        void* dst = split ? static_cast<void*>(a.part_o + (int64_t)piece * rows_all * kDc + at)
                    : f32 ? static_cast<void*>(static_cast<float*>(a.out) + at)
                          : static_cast<void*>(static_cast<__nv_bfloat16*>(a.out) + at);
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                         reinterpret_cast<uint64_t>(dst)), "r"(smem_u32(mine)), "r"(row_bytes)
                     : "memory");
        if (half == 0) {
          if (split) a.part_ml[(int64_t)piece * rows_all + row0 + r] = make_float2(fmaxf(m, -FLT_MAX), l);
          else if (a.lse) a.lse[row0 + r] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
      }
      asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
    }
  }
  tc_fence_before();
  cta_sync();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr double kStart = 4;  // a CTA's start and end, in chunks
constexpr size_t kMostPartial = size_t(1) << 30;

}  // namespace

bool attn4_tc_eligible(const Attn4Args& a) {
  return a.kv_dtype == DSA_BF16 && a.d_c == kDc && a.d_rope == kDr && a.h <= kM;
}

// Pieces a query's entries are cut into: a wave ends with its longest CTA, and merging costs a launch (about
// three chunks) and the partial outputs' traffic (at 4 TB/s, a chunk being about a microsecond).
int attn4_tc_splits(const Attn4Args& a) {
  const int64_t items = 2 * (int64_t)a.seqs.total_q, chunks = (a.top_k + kN - 1) / kN;
  if (items == 0) return 1;
  const double row_cost = (double)a.seqs.total_q * a.h * a.d_c * 8 / 4e6;
  int best = 1;
  double cost = 1e30;
  for (int s = 1; s <= chunks; ++s) {
    if (s > 1 && (size_t)s * a.seqs.total_q * a.h * (a.d_c * 4 + 8) > kMostPartial) break;
    const int64_t waves = (items * s + num_sms() - 1) / num_sms();
    const double c = waves * ((double)((chunks + s - 1) / s) + kStart) + (s > 1 ? 3 + s * row_cost : 0);
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}

int launch_attn4_tc(const Attn4Args& a, cudaStream_t stream) {
  Params p{};
  p.a = a;
  p.chunks = (a.top_k + kN - 1) / kN;
  const int64_t items = 2 * (int64_t)a.seqs.total_q * a.splits;
  if (items > 0x7fffffff) return set_error(DSA_ERR_UNSUPPORTED, "attn4: grid too large");
  CUtensorMap qmap;
  int rc = make_tmap_2d(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, kD, (uint64_t)a.seqs.total_q * a.h, kD * 2, 64, kM);
  if (rc != DSA_OK) return rc;
  static std::atomic<bool> allowed[64];
  rc = allow_smem<kSmem>(attn4_tc_kernel, allowed, "attn4_tc: smem attribute");
  if (rc != DSA_OK) return rc;
  cudaError_t e = cudaSuccess;
  DSA_LAUNCH("attn4_tc", stream,
             e = launch_pdl(attn4_tc_kernel, dim3((unsigned)items), dim3(kThreads), kSmem, stream, p, qmap));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "attn4_tc: %s", cudaGetErrorString(e));
  rc = check_launch("attn4_tc");
  if (rc != DSA_OK || a.splits == 1) return rc;
  return launch_attn4_merge(a, stream);
}

}  // namespace dsa
