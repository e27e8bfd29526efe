// Dense attention over the MLA latent cache for a batch that shares a prefix, on tcgen05 tensor
// cores (bf16, 64 <= D <= 576, d_c <= 512, any number of heads).
//
//   S[r, x] = scale · q[r,:]·key_x,  out[r,:] = Σ_x softmax(S[r,:])_x · key_x[0:d_c]
//
// All heads of all queries attend over the same latent keys, so the MMA's M = 128 rows are any 128
// (token, head) rows.  Rows of different sequences share a block where only the prefix is attended
// (few rows a sequence): the prefix is then computed once for the batch, 128 rows at a time,
// and each sequence's own keys in blocks of its own rows, and the pieces are merged.  Where a
// sequence fills blocks by itself, its blocks run over prefix and suffix as one key axis.
//
// Why value halves.  A 128 x 512 fp32 output accumulator is all of the tensor memory.  So a CTA
// accumulates at most 256 output columns, and d_c = 512 takes two CTAs a block, each with the
// whole logits: 576 + 256 columns of MMA instead of 576 + 512 split in two (544), but no exchange of
// partial logits between SMs (that link moves ~12 B a clock: 16 KB for a 64-key chunk would
// take longer than the duplicate MMAs).  The twin CTA finds the keys in L2.
//
// Tensor memory: O (256 columns) | two logit buffers (64 each; P, as bf16 pairs, overwrites the
// first half of its own logits) | the query columns that match the CTA's value tiles (128).  Shared
// memory: the other query columns (80 KB) and 18 tiles of [64 keys x 64 columns]: the CTA's own value
// columns ("V tiles") are held until P·V (3 chunks of 32 KB for d_c = 512), the others ("K tiles")
// only until the logits.
//
// Per chunk of 64 keys: the producer thread loads tiles by TMA; the MMA thread issues
// S(g) = Q·Kᵀ (M=128, N=64, K=D) and O += P(g-1)·V (M=128, N=256, K=64; P from tensor memory);
// four softmax warps, a thread a row, take the running max (it moves only when a row's max grows
// by more than 2^8; O is then rescaled), the sum in fp32 of the unrounded p, and write P.  P is rounded to bf16 there, the
// type that the MMA wants beside bf16 values: each p is off by 2^-8 of it at most, in either direction, and the output by
// less than its own rounding to bf16 (against 64 bits: 1.0 to 1.3 times the error of fp32 p and a rounded output).
// Order of the MMAs: S over the K tiles (their buffers are refilled meanwhile), over half the V tiles, P·V
// of the chunk before, the other half: softmax has the first part to finish in, and the last part hides the
// wait for P·V before the next chunk overwrites its P.
// Every wait is bounded (DSA_FLAG_TIMEOUT).
#include <float.h>

#include "prefix_attn.cuh"
#include "tc_sm100.cuh"

namespace dsa {
namespace {

using namespace tc;

constexpr int kM = 128;                 // rows of a block
constexpr int kN = 64;                  // keys of a chunk
constexpr int kTile = kN * 128;         // 8 KB: 64 keys x 64 columns
constexpr int kQTile = kM * 128;        // 16 KB: 128 rows x 64 columns
constexpr int kQTmemTiles = 4;          // query column tiles in tensor memory
constexpr int kQSmemTiles = 5;
constexpr int kTiles = 18;              // key tiles in flight
constexpr int kVSlots = 3, kKSlots = 3; // at most: chunks whose V, K tiles are in flight
constexpr int kThreads = 192;           // producer, MMA, 4 softmax warps
constexpr int kBarBytes = 512;
constexpr int kSmem = kQSmemTiles * kQTile + kTiles * kTile + kBarBytes + 1024;
constexpr int kOCol = 0, kSCol = 256, kQCol = 384;
constexpr float kRescaleLog2 = 8.0f;
static_assert(kSmem <= 232448, "shared memory");
static_assert(kM * (256 * 4 + 16) <= kTiles * kTile, "the output leaves through the key tiles");

struct Params {
  PrefixArgs a;
  int nblk;        // blocks of a sequence
  int fblk;        // blocks of all rows end to end (prefix items), 0: one key axis
  int sp, ss;      // pieces of the prefix alone / of a sequence's keys
  int halves;      // value column halves
  int prefix_items;
  int chunk_rows;  // cache rows a tile is loaded in
  int nseg;        // cuts: segments (0: every line in equal pieces, sp or ss)
  int ns;          // cuts: length of a line of a sequence's block, as the segments count it
  bool merged;     // a merge of pieces follows
};

// One CTA's (with halves, two CTAs') part of a line: the key chunks [a, b) of a block of rows.  Lines: the
// blocks of all rows over the prefix (fblk of them), then the sequences' blocks.
struct Seg {
  uint32_t a, b;
  uint16_t line, piece;
};
constexpr int kMaxSegs = 288;
struct Cuts {
  Seg seg[kMaxSegs];
};

struct Item {
  int half, piece, b;        // b < 0: prefix only
  bool split;                // the rows have other pieces: partial outputs
  int64_t row0;              // first flat (token, head) row
  int rows;
  int c0, c1;                // chunks [c0, c1) of the item's key axis
  int ncp;                   // prefix chunks on the axis
  int k0, pos0;              // suffix: first key row, position of the block's first token
  int hoff;                  // head of the block's first row
};

// floor(n · a / of), a <= of (in 32 bits where it fits: with 64-bit divisions here 64 sequences' call took 0.6 us more).
__device__ __forceinline__ int part(int n, uint32_t a, int of) {
  if (n < 65536 && of < 65536) return (int)((uint32_t)n * a / (uint32_t)of);
  return (int)((int64_t)n * a / of);
}

// False: nothing to do (a block past its sequence's rows, an inconsistent sequence).
__device__ __forceinline__ bool item_at(const Params& p, const Cuts& cuts, int i, Item& it) {
  const int pch = (p.a.prefix_len + kN - 1) / kN;
  it.half = i % p.halves;
  i /= p.halves;
  int line, split = 0;  // line: block, counted over the prefix's, then the sequences'
  Seg sg{};
  if (p.nseg) {
    sg = cuts.seg[i];
    line = sg.line;
    it.piece = sg.piece;
  } else if (i < p.prefix_items) {
    line = i % p.fblk;
    it.piece = split = i / p.fblk;
  } else {
    i -= p.prefix_items;
    const int blocks = p.a.seqs.B * p.nblk;
    line = p.fblk + i % blocks;
    split = i / blocks;
    it.piece = split + (p.fblk ? p.sp : 0);
  }
  if (line < p.fblk) {
    it.split = true;
    it.row0 = (int64_t)line * kM;
    it.b = -1;
    it.rows = (int)min((int64_t)kM, (int64_t)p.a.seqs.total_q * p.a.h - it.row0);
    it.ncp = pch;
    it.c0 = p.nseg ? (int)sg.a : part(pch, split, p.sp);
    it.c1 = p.nseg ? (int)sg.b : part(pch, split + 1, p.sp);
    it.k0 = it.pos0 = it.hoff = 0;
    return true;
  }
  const int blk = line - p.fblk;
  it.b = blk / p.nblk;
  it.split = p.fblk || (p.nseg ? sg.a > 0 || (int)sg.b < p.ns : p.ss > 1);
  SeqInfo s;
  if (!prefix_seq(p.a, it.b, s)) return false;
  // (32 bits: total_q · h is below 2^31)
  const uint32_t h = p.a.h, r0 = (uint32_t)(blk - it.b * p.nblk) * kM, nrow = s.T * h;
  if (r0 >= nrow) return false;
  it.row0 = (int64_t)s.q0 * p.a.h + r0;
  it.rows = (int)min((uint32_t)kM, nrow - r0);
  it.ncp = p.fblk ? 0 : pch;
  it.k0 = s.k0;
  it.pos0 = s.L - s.T + (int)(r0 / h);
  it.hoff = (int)(r0 % h);
  const int last = s.L - s.T + (int)((r0 + it.rows - 1) / h);
  const int n = it.ncp + last / kN + 1;
  it.c0 = p.nseg ? part(n, sg.a, p.ns) : part(n, split, p.ss);
  it.c1 = p.nseg ? part(n, sg.b, p.ns) : part(n, split + 1, p.ss);
  return true;
}

// 64 consecutive tensor-memory columns of this warp's 32 lanes (two loads, one wait each).
__device__ __forceinline__ void load_row(uint32_t taddr, float (&s)[kN]) {
  uint32_t r[32];
  tmem_ld32(taddr, r);
#pragma unroll
  for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(r[i]);
  tmem_ld32(taddr + 32, r);
#pragma unroll
  for (int i = 0; i < 32; ++i) s[32 + i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Zero the infinities and NaNs among 8 bf16 values; whether there were any.
__device__ __forceinline__ bool finite8(uint4& v) {
  uint32_t u[4] = {v.x, v.y, v.z, v.w};
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((u[i] & 0x7f80u) == 0x7f80u) { u[i] &= 0xffff0000u; any = true; }
    if ((u[i] & 0x7f800000u) == 0x7f800000u) { u[i] &= 0xffffu; any = true; }
  }
  v = make_uint4(u[0], u[1], u[2], u[3]);
  return any;
}

// NaN in those of a row's n output columns from column c (at `out`, f32 or bf16) in which one of the keys at positions
// [x0, x1) of its sequence holds an infinity or a NaN.  (Read from the cache: the tile's were zeroed.)
__device__ __noinline__ void spoil(const PrefixArgs& a, int b, int k0, int x0, int x1, int c, int n, bool f32, uint8_t* out) {
  for (int x = x0; x < x1; ++x) {
    const int row = cache_row(a.seqs, b, k0, x);
    if (row < 0) continue;
    const uint16_t* v = static_cast<const uint16_t*>(a.kv) + (int64_t)row * (a.d_c + a.d_rope) + c;
    for (int i = 0; i < n; ++i) {
      if ((v[i] & 0x7f80u) != 0x7f80u) continue;
      if (f32) reinterpret_cast<uint32_t*>(out)[i] = 0x7fffffffu;
      else reinterpret_cast<uint16_t*>(out)[i] = 0x7fffu;
    }
  }
}

// Box of kN (or a page's) rows x 64 columns x 4 column tiles into four consecutive tiles.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

struct Maps {
  CUtensorMap q;           // [rows, D], box 128 x 64
  CUtensorMap pre, key;    // prefix and cache rows, box chunk_rows x 64
  CUtensorMap pre4, key4;  // the same as [tiles][rows][64], box 4 x chunk_rows x 64
};

// NK > 0: 512 value columns and NK K tiles in both halves (d_rope = 64: 5, d_rope = 0: 4), everything unrolled, V
// tiles loaded four at a time, a barrier a K tile.  NK = 0: any widths, a barrier a chunk's K tiles.  One thread issues
// all MMAs and one all copies, and their scalar code is what counts: with the counts known only at run time
// (and divided by, for a slot and a phase) the issue took 4,600 clocks a chunk of 512 + 64 columns where
// the tensor pipe needs 1,980 (36 MMAs of N = 64 and 4 of N = 256); unrolled it takes 2,170.  Without
// divisions the general form takes 2,530 for 512 + 0 columns (NK = 4: 2,130), 1,950 for 256 + 32, 1,430 for 128 + 64
// and 1,340 for 64 + 16, the last two bound by softmax; a barrier a K tile there cost 100 to 700 clocks more.
template <int NK>
__global__ void __launch_bounds__(kThreads, 1)
prefix_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps,
                 const __grid_constant__ Cuts cuts) {
  constexpr bool FIXED = NK > 0;
  griddep_wait();
  if (p.merged) griddep_launch();  // the merge may be set up meanwhile; it waits for this grid to end
  Item it;
  if (!item_at(p, cuts, blockIdx.x, it)) return;
  const PrefixArgs& a = p.a;
  const int64_t rows_all = (int64_t)a.seqs.total_q * a.h;
  const int nch = it.c1 - it.c0;
  const bool split = it.split;
  if (nch == 0) {  // a piece without keys
    if (split && it.half == 0)
      for (int i = threadIdx.x; i < it.rows; i += kThreads)
        a.part_ml[(int64_t)it.piece * rows_all + it.row0 + i] = make_float2(-INFINITY, 0.f);
    return;
  }

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* qs = smem;                               // [5][128][128 B]
  uint8_t* vs = qs + kQSmemTiles * kQTile;          // [vslots][nvt][64][128 B], then the K tiles
  uint64_t* bars = reinterpret_cast<uint64_t*>(vs + kTiles * kTile);
  uint64_t* v_full = bars;            // [3]
  uint64_t* v_empty = bars + 3;       // [3]
  uint64_t* k_full = bars + 6;        // [3] a chunk's K tiles; NK > 0: [NK] a K tile
  uint64_t* k_empty = bars + 12;
  uint64_t* s_full = bars + 18;       // [2] logits of the buffer's chunk complete
  uint64_t* p_full = bars + 20;       // [2] its 4 softmax warps have written P
  uint64_t* pv_done = bars + 22;      // [2] its P·V complete
  uint64_t* q_full = bars + 24;       // the query tiles in shared memory
  uint64_t* qt_full = bars + 25;      // the query columns in tensor memory (4 warps)
  uint64_t* drain = bars + 26;
  uint64_t* badkeys = bars + 27;      // [3] keys of a chunk on pages outside the cache, a bit each
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 30);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 31);
  uint64_t* q_staged = bars + 32;     // query tiles on their way to tensor memory

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int D = a.d_c + a.d_rope;
  const int ntile = (D + 63) / 64;
  const int vcol0 = it.half * 256;
  const int ncol = FIXED ? 256 : min(256, a.d_c - vcol0);         // this CTA's output columns (a multiple of 16)
  const int vt0 = it.half * 4, nvt = FIXED ? 4 : (ncol + 63) / 64;
  const int nkt = FIXED ? NK : ntile - nvt;          // at most 8
  // 3 chunks of V tiles always fit beside one of K tiles (3·4 + 5, or nvt < 4: 3·3 + 8 of 18)
  const int kslots = FIXED ? 1 : nkt ? min(kKSlots, (kTiles - kVSlots * nvt) / nkt) : 0;
  uint8_t* ks = vs + kVSlots * nvt * kTile;         // [kslots][nkt][64][128 B]
  // Column tile of K tile j, and where the query columns that match a tile are: V tile j in tensor
  // memory at tile j; K tile j after them while there is room (4 tiles), then in shared memory.
  auto ktile = [&](int j) { return j < vt0 ? j : j + nvt; };
  const int nkq = FIXED ? 0 : min(nkt, kQTmemTiles - nvt);  // K tiles whose query columns are in tensor memory
  // The query tiles for tensor memory come by TMA into key tiles that no chunk uses yet (NK > 0: those of
  // chunks 1 and 2; otherwise the first, and no key is loaded before they have left).
  uint8_t* qstage = vs + (FIXED ? 4 * kTile : 0);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kVSlots; ++i) { mbar_init(&v_full[i], 1); mbar_init(&v_empty[i], 1); }
    for (int i = 0; i < 2 * kKSlots; ++i) { mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_staged, 1);
    mbar_init(qt_full, 4);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ---------------- producer ----------------
    if (elect_one()) {
      const int nqs = nkt - nkq, nqt = nvt + nkq;
      mbar_arrive_expect_tx(q_staged, (uint32_t)(nqt * kQTile));
      for (int t = 0; t < nqt; ++t)
        tma_load_2d(qstage + t * kQTile, &maps.q, q_staged, (t < nvt ? vt0 + t : ktile(t - nvt)) * 64, (int)it.row0);
      if (nqs) {
        mbar_arrive_expect_tx(q_full, (uint32_t)(nqs * kQTile));
        for (int j = 0; j < nqs; ++j)
          tma_load_2d(qs + j * kQTile, &maps.q, q_full, ktile(nkq + j) * 64, (int)it.row0);
      }
      int g = 0, kn = 0;  // chunks whose V tiles, chunks (NK > 0: tiles) whose K tiles have been issued
      int kslot = 0, kphase = 0;
      auto stage_free = [&]() { return mbar_wait(qt_full, 0, abort_flag, a.status, DSA_FLAG_TIMEOUT); };
      const int stop_at = FIXED || stage_free() ? nch : 0;
      for (; g < stop_at; ++g) {
        const int c = it.c0 + g, vslot = g % kVSlots;
        // the cache rows of the chunk's keys: one run, or one a page
        const bool pre = c < it.ncp;
        const int x0 = (pre ? c : c - it.ncp) * kN;
        const CUtensorMap* map = pre ? &maps.pre : &maps.key;
        const CUtensorMap* map4 = pre ? &maps.pre4 : &maps.key4;
        const bool paged = a.seqs.paged() && !(pre && a.prefix_kv);  // a paged cache's prefix may be packed
        int run[kN / 16];
        uint64_t bad = 0;
        const int cr = p.chunk_rows, nrun = kN / cr;
        if (!paged) {
#pragma unroll
          for (int j = 0; j < kN / 16; ++j) run[j] = (pre ? x0 : it.k0 + x0) + j * cr;
        } else {
          const int sh = __ffs(a.seqs.page_size) - 1;
          const int pages = pre ? (a.prefix_len + a.seqs.page_size - 1) >> sh : a.seqs.max_pages;
          const int32_t* table = pre ? a.prefix_table : a.seqs.block_table + (int64_t)it.b * a.seqs.max_pages;
#pragma unroll
          for (int j = 0; j < kN / 16; ++j) {
            if (j >= nrun) break;
            const int x = x0 + j * cr, slot = x >> sh;
            const int pg = slot < pages ? table[slot] : -1;
            const bool ok = (unsigned)pg < (unsigned)a.seqs.num_pages;
            // keys of a page outside the cache are masked; page 0 stands in for their rows
            if (!ok) bad |= (cr == 64 ? ~0ull : ((1ull << cr) - 1)) << (j * cr);
            run[j] = ok ? (pg << sh) | (x & (a.seqs.page_size - 1)) : 0;
          }
        }
        auto load = [&](uint8_t* dst, uint64_t* bar, int tile) {
#pragma unroll
          for (int j = 0; j < kN / 16; ++j) {
            if (j >= nrun) break;
            tma_load_2d(dst + j * cr * 128, map, bar, tile * 64, run[j]);
          }
        };
        auto load4 = [&](uint8_t* dst, uint64_t* bar, int tile) {
#pragma unroll
          for (int j = 0; j < kN / 16; ++j) {
            if (j >= nrun) break;
            if (cr == kN) {
              tma_load_3d(dst, map4, bar, 0, run[j], tile);
            } else {  // a page's rows of each tile: the tiles are kTile apart, not the box's size
              for (int t = 0; t < 4; ++t) tma_load_2d(dst + t * kTile + j * cr * 128, map, bar, (tile + t) * 64, run[j]);
            }
          }
        };
        // K tiles first: the MMAs start with them
        bool stop = false;
        if constexpr (FIXED) {
          for (int j = 0; j < NK; ++j) {
            if (!mbar_wait(&k_empty[j], (g & 1) ^ 1, abort_flag, a.status, DSA_FLAG_TIMEOUT)) { stop = true; break; }
            mbar_arrive_expect_tx(&k_full[j], kTile);
            load(ks + j * kTile, &k_full[j], ktile(j));
            ++kn;
          }
          if (g == 1 && !stop) stop = !stage_free();
        } else if (nkt) {
          stop = !mbar_wait(&k_empty[kslot], kphase ^ 1, abort_flag, a.status, DSA_FLAG_TIMEOUT);
          if (!stop) {
            mbar_arrive_expect_tx(&k_full[kslot], (uint32_t)(nkt * kTile));
            for (int j = 0; j < nkt; ++j) load(ks + (kslot * nkt + j) * kTile, &k_full[kslot], ktile(j));
            ++kn;
            if (++kslot == kslots) { kslot = 0; kphase ^= 1; }
          }
        }
        if (stop || !mbar_wait(&v_empty[vslot], ((g / kVSlots) & 1) ^ 1, abort_flag, a.status, DSA_FLAG_TIMEOUT))
          break;
        badkeys[vslot] = bad;
        mbar_arrive_expect_tx(&v_full[vslot], (uint32_t)(nvt * kTile));
        if (FIXED) {
          load4(vs + vslot * 4 * kTile, &v_full[vslot], vt0);
        } else {
          for (int t = 0; t < nvt; ++t) load(vs + (vslot * nvt + t) * kTile, &v_full[vslot], vt0 + t);
        }
      }
      // every copy issued has landed before the CTA may exit
      mbar_wait_drain(q_staged, 0);
      if (nqs) mbar_wait_drain(q_full, 0);
      for (int i = max(0, g - kVSlots); i < g; ++i)
        mbar_wait_drain(&v_full[i % kVSlots], (i / kVSlots) & 1);
      if constexpr (FIXED) {
        for (int i = max(0, kn - NK); i < kn; ++i) mbar_wait_drain(&k_full[i % NK], (i / NK) & 1);
      } else {
        for (int i = max(0, kn - kslots); i < kn; ++i) mbar_wait_drain(&k_full[i % kslots], (i / kslots) & 1);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    // elect.sync and unrolled K-steps keep the operands in uniform registers: an M=128, N=64, K=16
    // MMA with A in tensor memory then issues every 33 clocks (the pipe's own rate), with A in shared
    // memory every 49 (6 KB of operands at 128 B a clock); under lane == 0 and a counted loop it was 164.
    if (elect_one()) {
      const uint32_t idesc_s = idesc_bf16(kM, kN);
      const uint32_t idesc_pv = idesc_bf16(kM, ncol, false, true);
      const uint32_t q0 = smem_u32(qs), v0 = smem_u32(vs), k0 = smem_u32(ks);
      bool stop = !mbar_wait(qt_full, 0, abort_flag, a.status, DSA_FLAG_TIMEOUT);
      if (!stop && nkt > nkq) stop = !mbar_wait(q_full, 0, abort_flag, a.status, DSA_FLAG_TIMEOUT);
      tc_fence_after();
      const uint64_t qd = sdesc_sw128(q0, 16, 1024);
      if constexpr (FIXED) {
        const uint64_t kd = sdesc_sw128(k0, 16, 1024);
        int vslot = 0, vphase = 0;           // of chunk g
        uint64_t pvd = 0;                    // V tiles of chunk g - 1, as P·V reads them
        uint64_t* pv_empty = nullptr;
        // A barrier is tested before the MMAs that come ahead of its use are issued, so that the test's own latency
        // passes beside them (a wait that finds its barrier complete still takes ~100 clocks, and eight of them
        // a chunk were the issuing thread's time); only where it was not complete yet is it waited for.
        auto test = [&](uint64_t* bar, uint32_t parity) { return mbar_test(smem_u32(bar), parity); };
        auto sure = [&](bool ready, uint64_t* bar, uint32_t parity) {
          return ready || mbar_wait(bar, parity, abort_flag, a.status, DSA_FLAG_TIMEOUT);
        };
        auto pv_fixed = [&](int g, bool ready) -> bool {
          if (!sure(ready, &p_full[g & 1], (g >> 1) & 1)) return false;
          tc_fence_after();
          const uint32_t pa = tmem + kSCol + (g & 1) * kN;
          const uint32_t acc = g > 0;
#pragma unroll
          for (int kk = 0; kk < kN / 16; ++kk)
            mma_bf16_ts(tmem + kOCol, pa + kk * 8, pvd + (uint64_t)(kk * 128), idesc_pv, kk ? 1u : acc);
          mma_commit(pv_empty);
          mma_commit(&pv_done[g & 1]);
          return true;
        };
        for (int g = 0; g < nch && !stop; ++g) {
          bool ready = test(&k_full[0], g & 1);
          if (g >= 2 && !mbar_wait(&pv_done[g & 1], ((g >> 1) & 1) ^ 1, abort_flag, a.status, DSA_FLAG_TIMEOUT))
            break;
          const uint32_t d = tmem + kSCol + (g & 1) * kN;
          // a barrier a tile: each is refilled while the others and the V tiles are multiplied
#pragma unroll
          for (int j = 0; j < NK; ++j) {
            if (!sure(ready, &k_full[j], g & 1)) { stop = true; break; }
            tc_fence_after();
            ready = j + 1 < NK ? test(&k_full[j + 1], g & 1) : test(&v_full[vslot], vphase);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_bf16(d, qd + (uint64_t)(j * (kQTile >> 4) + i * 2), kd + (uint64_t)(j * (kTile >> 4) + i * 2),
                       idesc_s, j || i ? 1u : 0u);
            mma_commit(&k_empty[j]);
          }
          if (stop || !sure(ready, &v_full[vslot], vphase)) break;
          tc_fence_after();
          ready = g > 0 && test(&p_full[(g - 1) & 1], ((g - 1) >> 1) & 1);
          const uint64_t vd = sdesc_sw128(v0 + vslot * (4 * kTile), 16, 1024);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_bf16_ts(d, tmem + kQCol + t * 32 + i * 8, vd + (uint64_t)(t * (kTile >> 4) + i * 2), idesc_s, 1u);
          if (g > 0 && !pv_fixed(g - 1, ready)) { stop = true; break; }
#pragma unroll
          for (int t = 2; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_bf16_ts(d, tmem + kQCol + t * 32 + i * 8, vd + (uint64_t)(t * (kTile >> 4) + i * 2), idesc_s, 1u);
          mma_commit(&s_full[g & 1]);
          pvd = sdesc_sw128(v0 + vslot * (4 * kTile), kTile, 1024);
          pv_empty = &v_empty[vslot];
          if (++vslot == kVSlots) { vslot = 0; vphase ^= 1; }
          if (g == nch - 1 && !pv_fixed(g, false)) stop = true;
        }
      } else {
        // The logits' K-steps of one tile: A = tile qt of the query in tensor memory, or (qt >= 4) tile qt - 4 of
        // it in shared memory; the last tile may have fewer than four steps.
        const int tail = D % 64 / 16;
        uint32_t acc = 0;
        auto qk_tile = [&](uint32_t d, int qt, int t, uint64_t b0) {
          const uint64_t a0 = qd + (uint64_t)((qt - kQTmemTiles) * (kQTile >> 4));
          const uint32_t at = tmem + kQCol + qt * 32;
          if (tail == 0 || t + 1 < ntile) {
            if (qt < kQTmemTiles) {
              mma_bf16_ts(d, at, b0, idesc_s, acc);
#pragma unroll
              for (int i = 1; i < 4; ++i) mma_bf16_ts(d, at + i * 8, b0 + (uint64_t)(i * 2), idesc_s, 1u);
            } else {
              mma_bf16(d, a0, b0, idesc_s, acc);
#pragma unroll
              for (int i = 1; i < 4; ++i) mma_bf16(d, a0 + (uint64_t)(i * 2), b0 + (uint64_t)(i * 2), idesc_s, 1u);
            }
          } else {
            for (int i = 0; i < tail; ++i) {
              if (qt < kQTmemTiles) mma_bf16_ts(d, at + i * 8, b0 + (uint64_t)(i * 2), idesc_s, i ? 1u : acc);
              else mma_bf16(d, a0 + (uint64_t)(i * 2), b0 + (uint64_t)(i * 2), idesc_s, i ? 1u : acc);
            }
          }
          acc = 1;
        };
        const uint64_t kd = sdesc_sw128(k0, 16, 1024), vd = sdesc_sw128(v0, 16, 1024);
        const uint64_t pvd = sdesc_sw128(v0, kTile, 1024);
        int kslot = 0, kphase = 0, vslot = 0, vphase = 0, pslot = 0;  // pslot: V slot of chunk g - 1
        auto pv = [&](int g) -> bool {
          if (!mbar_wait(&p_full[g & 1], (g >> 1) & 1, abort_flag, a.status, DSA_FLAG_TIMEOUT)) return false;
          tc_fence_after();
          const uint64_t b0 = pvd + (uint64_t)(pslot * nvt * (kTile >> 4));
          const uint32_t pa = tmem + kSCol + (g & 1) * kN;
#pragma unroll
          for (int kk = 0; kk < kN / 16; ++kk)
            mma_bf16_ts(tmem + kOCol, pa + kk * 8, b0 + (uint64_t)(kk * 128), idesc_pv, (g > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&v_empty[pslot]);
          mma_commit(&pv_done[g & 1]);
          return true;
        };
        // P·V waits for softmax (~800 clocks after its logits): with few column tiles the next logits come whole
        // before it, or softmax would wait for them in turn (64 + 16 columns: 1,535 clocks a chunk with
        // P·V in their middle, 1,340 so)
        const int mid = ntile > 5 ? nvt / 2 : nvt;
        for (int g = 0; g < nch && !stop; ++g) {
          // the buffer's last P (chunk g - 2) has been read
          if (g >= 2 && !mbar_wait(&pv_done[g & 1], ((g >> 1) & 1) ^ 1, abort_flag, a.status, DSA_FLAG_TIMEOUT))
            break;
          const uint32_t d = tmem + kSCol + (g & 1) * kN;
          acc = 0;
          if (nkt) {
            if (!mbar_wait(&k_full[kslot], kphase, abort_flag, a.status, DSA_FLAG_TIMEOUT)) break;
            tc_fence_after();
            uint64_t b0 = kd + (uint64_t)(kslot * nkt * (kTile >> 4));
            for (int j = 0; j < nkt; ++j, b0 += kTile >> 4)
              qk_tile(d, j < nkq ? nvt + j : kQTmemTiles + j - nkq, ktile(j), b0);
            mma_commit(&k_empty[kslot]);
            if (++kslot == kslots) { kslot = 0; kphase ^= 1; }
          }
          if (!mbar_wait(&v_full[vslot], vphase, abort_flag, a.status, DSA_FLAG_TIMEOUT)) break;
          tc_fence_after();
          uint64_t b0 = vd + (uint64_t)(vslot * nvt * (kTile >> 4));
          for (int t = 0; t < mid; ++t, b0 += kTile >> 4) qk_tile(d, t, vt0 + t, b0);
          if (g > 0 && !pv(g - 1)) { stop = true; break; }
          for (int t = mid; t < nvt; ++t, b0 += kTile >> 4) qk_tile(d, t, vt0 + t, b0);
          mma_commit(&s_full[g & 1]);
          pslot = vslot;
          if (++vslot == kVSlots) { vslot = 0; vphase ^= 1; }
          if (g == nch - 1 && !pv(g)) stop = true;
        }
      }
      mma_commit(drain);
      mbar_wait_drain(drain, 0);
    }
  } else {
    // ---------------- softmax: thread = row ----------------
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    const int64_t flat = it.row0 + min(r, it.rows - 1);  // rows past the block repeat its last
    // this row's last visible suffix position
    const int pos = it.pos0 + (it.hoff + min(r, it.rows - 1)) / a.h;
    {
      const bool ok = __all_sync(0xffffffffu, mbar_wait(q_staged, 0, abort_flag, a.status, DSA_FLAG_TIMEOUT));
      for (int t = 0; ok && t < nvt + nkq; ++t) {
        const uint8_t* from = qstage + t * kQTile + r * 128;
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(from + ((i ^ (r & 7)) * 16));
          w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
        tmem_st32(lane_base + kQCol + t * 32, w);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(qt_full);
    }
    float m = -INFINITY, l = 0.f;  // the reference (log2 units) and the sum relative to it
    bool spoilt = false;           // this row sees a key that may have been zeroed for others
    bool stop = false;
    for (int g = 0; g < nch; ++g) {
      const int c = it.c0 + g;
      // keys of the chunk this row sees, and the block's first row
      const bool pre = c < it.ncp;
      const int x0 = (pre ? c : c - it.ncp) * kN;
      const int lim = pre ? min(kN, a.prefix_len - x0) : max(0, min(kN, pos + 1 - x0));
      const int lim0 = pre ? lim : max(0, min(kN, it.pos0 + 1 - x0));
      if (!__all_sync(0xffffffffu, mbar_wait(&s_full[g & 1], (g >> 1) & 1, abort_flag, a.status,
                                             DSA_FLAG_TIMEOUT))) { stop = true; break; }
      tc_fence_after();
      uint64_t bad = 0;
      if (a.seqs.paged()) {
        if (!__all_sync(0xffffffffu, mbar_wait(&v_full[g % kVSlots], (g / kVSlots) & 1, abort_flag,
                                               a.status, DSA_FLAG_TIMEOUT))) { stop = true; break; }
        bad = *const_cast<volatile uint64_t*>(&badkeys[g % kVSlots]);
      }
      const uint32_t sbuf = lane_base + kSCol + (g & 1) * kN;
      float s[kN];
      load_row(sbuf, s);
      if (lim0 < kN || bad) {
        // some row does not see some key.  Its p is 0, but 0 times an infinity or a NaN in the
        // key's value columns would not be: those are zeroed in the tile, which the logits have read
        // already.  A row that does see such a key has a logit that is not finite (the value columns are columns of
        // the key): NaN or +inf, and its whole output is NaN; or -inf, and where the zeroed ones would have
        // made its output NaN (0 times them) NaN is written in the end
        if (!a.seqs.paged() &&
            !__all_sync(0xffffffffu, mbar_wait(&v_full[g % kVSlots], (g / kVSlots) & 1, abort_flag,
                                               a.status, DSA_FLAG_TIMEOUT))) { stop = true; break; }
        bool any = false;
        uint8_t* vt = vs + (g % kVSlots) * nvt * kTile;
        for (int i0 = r; i0 < nvt * kN * 8; i0 += 4 * kM) {  // 16-byte pieces, four loads in flight; a row of the
          uint4 v[4];                                       // tile is a key, in whatever order its pieces are
          bool look[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * kM, key = (i >> 3) & (kN - 1);
            look[j] = i < nvt * kN * 8 && (key >= lim0 || ((bad >> key) & 1));
            if (look[j]) v[j] = reinterpret_cast<const uint4*>(vt)[i];
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (look[j] && finite8(v[j])) { reinterpret_cast<uint4*>(vt)[i0 + j * kM] = v[j]; any = true; }
        }
        if (any) fence_proxy_async_smem();
        const uint64_t in = (lim >= kN ? ~0ull : (1ull << lim) - 1);
        if ((bad & in) && it.half == 0) atomicOr(a.status, DSA_FLAG_BAD_INDEX);
        const uint64_t see = in & ~bad;
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (!((see >> i) & 1)) s[i] = -INFINITY;
        if (lim > lim0) {  // it sees keys that the first row does not
          uint32_t none[2] = {0u, 0u};
#pragma unroll
          for (int i = 0; i < kN; ++i) none[i >> 5] |= s[i] == -INFINITY ? 1u << (i & 31) : 0u;
          spoilt |= (see & ((uint64_t)none[1] << 32 | none[0])) != 0;
        }
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < kN; ++i) mx[i & 3] = fmaxf(mx[i & 3], s[i]);
      const float mc = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
      const bool grow = mc > m + kRescaleLog2;  // the first keys always (m = -inf)
      if (__any_sync(0xffffffffu, grow)) {
        const float m_new = grow ? mc : m;
        const float factor = grow ? ex2(m - m_new) : 1.f;
        l *= factor;
        if (g > 0) {
          // O holds the chunks before g at the old reference: rescale it once P·V(g - 1) is in
          if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag,
                                                 a.status, DSA_FLAG_TIMEOUT))) { stop = true; break; }
          tc_fence_after();
          __syncwarp();
          for (int b = 0; b < (ncol + 31) / 32; ++b) {
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
        const float p0 = ex2(fmaf(s[2 * i], a.scale_log2, -ref));
        const float p1 = ex2(fmaf(s[2 * i + 1], a.scale_log2, -ref));
        sum[(2 * i) & 3] += p0;
        sum[(2 * i + 1) & 3] += p1;
        pk[i] = bf16x2(p0, p1);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      __syncwarp();
      tmem_st32(sbuf, pk);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[g & 1]);
    }
    if (!stop)
      stop = !__all_sync(0xffffffffu, mbar_wait(&pv_done[(nch - 1) & 1], ((nch - 1) >> 1) & 1, abort_flag,
                                                a.status, DSA_FLAG_TIMEOUT));
    if (!stop) {
      tc_fence_after();
      // O goes out through the key tiles (all of them have been multiplied): a thread writes its row there and
      // sends it with one bulk copy.  Stored from registers, 16 bytes of 32 different rows at a time, the
      // rows took 2.5 us.  Rows are 16 bytes more than their length apart, which spreads them over the banks.
      const bool live = r < it.rows;
      const float inv = split ? 1.f : (l == 0.f ? 0.f : 1.f / l);
      const bool f32 = split || a.out_dtype == DSA_F32;
      const int row_bytes = ncol * (f32 ? 4 : 2);
      uint8_t* mine = vs + r * (row_bytes + 16);
      for (int b = 0; b < (ncol + 31) / 32; ++b) {
        uint32_t o[32];
        __syncwarp();  // the load is the whole warp's
        tmem_ld32(lane_base + kOCol + 32 * b, o);
        const int n = min(32, ncol - 32 * b);  // 16 or 32 columns
        if (f32) {
          float4* dst = reinterpret_cast<float4*>(mine) + 8 * b;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (4 * i < n)
              dst[i] = make_float4(__uint_as_float(o[4 * i]) * inv, __uint_as_float(o[4 * i + 1]) * inv,
                                   __uint_as_float(o[4 * i + 2]) * inv, __uint_as_float(o[4 * i + 3]) * inv);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(mine) + 4 * b;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (8 * i < n) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = bf16x2(__uint_as_float(o[8 * i + 2 * e]) * inv,
                              __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
              dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
      }
      // the keys that the row sees and the block's first row does not, in this item's chunks
      if (spoilt)
        spoil(a, it.b, it.k0, max(it.pos0 + 1, (it.c0 - it.ncp) * kN), min(pos + 1, (it.c1 - it.ncp) * kN), vcol0, ncol,
              f32, mine);
      fence_proxy_async_smem();  // our writes, seen by the bulk copy
      if (live) {
        const int64_t at = flat * a.d_c + vcol0;
        void* dst = split ? static_cast<void*>(a.part_o + (int64_t)it.piece * rows_all * a.d_c + at)
                    : f32 ? static_cast<void*>(static_cast<float*>(a.out) + at)
                          : static_cast<void*>(static_cast<__nv_bfloat16*>(a.out) + at);
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                         reinterpret_cast<uint64_t>(dst)), "r"(smem_u32(mine)), "r"(row_bytes)
                     : "memory");
      }
      if (live && it.half == 0) {
        // (m = -inf is a piece without keys, whose output the merge does not read)
        if (split) a.part_ml[(int64_t)it.piece * rows_all + flat] = make_float2(fmaxf(m, -FLT_MAX), l);
        else if (a.lse) a.lse[flat] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
      asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
    }
  }
  tc_fence_before();
  cta_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// How the rows and their keys are cut (all from the descriptor's sizes and the prefix's length): into
// equal pieces (sp, ss), or into segments.
struct Plan {
  int nblk, fblk, sp, ss, halves;
  int nseg = 0, ns = 0;
  PrefixMerge merge;
  Cuts cuts;
};

// Most pieces a row is cut into: about four waves of CTAs.
int most_pieces(int64_t blocks, int halves) {
  const int64_t s = 4 * (int64_t)num_sms() / (blocks * halves > 0 ? blocks * halves : 1);
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

constexpr size_t kMostPartial = size_t(1) << 30;
size_t partial_bytes(const PrefixArgs& a, int pieces) {
  return pieces > 1 ? (size_t)pieces * a.seqs.total_q * a.h * (a.d_c * 4 + 8) : 0;
}

void blocks_of(const PrefixArgs& a, Plan& pl) {
  pl.halves = (a.d_c + 255) / 256;
  pl.nblk = (int)(((int64_t)a.max_q_len * a.h + kM - 1) / kM);
  pl.fblk = (int)(((int64_t)a.seqs.total_q * a.h + kM - 1) / kM);
}

constexpr double kStart = 4;   // a CTA's start and end, in chunks
constexpr int kShort = 3;      // chunks of the shortest segment (but for a line's own length)

// Cut the lines, laid end to end, into one share a machine (an SM, or one a half) of at most C chunks' time.
// False if they do not fit.  `round` counts a machine's segments.
bool cut(int fblk, int pch, int lines, int ns, int machines, double C, Seg* seg, uint8_t* round, uint8_t* np,
         int& nseg) {
  int m = 0, r = 0, n = 0;
  double used = 0;
  for (int line = 0; line < lines; ++line) {
    const int len = line < fblk ? pch : ns;
    int at = 0, k = 0;
    while (at < len) {
      int take = (int)(C - used - kStart);
      if (take >= len - at) take = len - at;
      else if (len - at - take < kShort) take = len - at - kShort;
      if (take < kShort && take < len - at) {
        if (r == 0 || ++m >= machines) return false;
        used = 0;
        r = 0;
        continue;
      }
      if (n >= kMaxSegs || k >= 64) return false;
      seg[n] = Seg{(uint32_t)at, (uint32_t)(at + take), (uint16_t)line, (uint16_t)k++};
      round[n++] = (uint8_t)r++;
      used += take + kStart;
      at += take;
    }
    np[line] = (uint8_t)k;
  }
  nseg = n;
  return true;
}

// Segments of equal shares, in launch order: every machine's first, then the others, longest first (a
// machine that ends its first segment early then takes what its own share had left, or as much).  Returns
// the time in chunks, or 1e30.
double cut_equal(const PrefixArgs& a, int fblk, Plan& pl) {
  const int pch = (a.prefix_len + kN - 1) / kN;
  const int sch = (int)(((int64_t)a.seqs.total_k / a.seqs.B + kN - 1) / kN);
  const int64_t lines = fblk + (int64_t)a.seqs.B * pl.nblk;
  const int ns = (fblk ? 0 : pch) + (sch > 0 ? sch : 1), machines = num_sms() / pl.halves;
  if (lines > kMaxLines) return 1e30;
  const double total = (double)fblk * (pch + kStart) + (double)(lines - fblk) * (ns + kStart);
  if (total < 8.0 * machines) return 1e30;  // little to balance
  Seg seg[kMaxSegs];
  uint8_t round[kMaxSegs];
  int n = 0;
  double C = total / machines + kStart * 0.8;
  bool fits = false;
  for (int i = 0; i < 16 && !fits; ++i, C *= 1.015)
    fits = cut(fblk, pch, (int)lines, ns, machines, C, seg, round, pl.merge.np, n);
  // segments of a sequence's block are the same parts of its own length: with very different lengths, equal
  // pieces in several waves even out better
  if (!fits || (double)a.seqs.max_k_len / kN - sch > 0.2 * C) return 1e30;
  int most[2] = {0, 0}, order[kMaxSegs], k = 0;
  for (int i = 0; i < (int)lines; ++i) {
    int& x = most[i < fblk ? 0 : 1];
    if (pl.merge.np[i] > x) x = pl.merge.np[i];
  }
  if (most[0] + most[1] > prefix_tc_most_pieces(a)) return 1e30;
  for (int i = 0; i < n; ++i)
    if (round[i] == 0) order[k++] = i;
  const int first = k;
  for (int i = 0; i < n; ++i) {
    if (round[i] == 0) continue;
    int j = k++;
    for (; j > first && seg[order[j - 1]].b - seg[order[j - 1]].a < seg[i].b - seg[i].a; --j) order[j] = order[j - 1];
    order[j] = i;
  }
  for (int i = 0; i < n; ++i) {
    Seg& t = pl.cuts.seg[i];
    t = seg[order[i]];
    if (t.line >= fblk) t.piece = (uint16_t)(t.piece + most[0]);
  }
  pl.nseg = n;
  pl.ns = ns;
  pl.merge.table = 1;
  pl.merge.fblk = fblk;
  pl.merge.nblk = pl.nblk;
  pl.merge.base = most[0];
  pl.merge.pieces = most[0] + most[1];
  return C;
}

// Time model in units of a chunk: a CTA's start and end cost about four chunks, a wave ends
// with its longest CTA, and merging costs a launch (about three chunks) and the partial outputs' traffic.
void plan_of(const PrefixArgs& a, Plan& out) {
  blocks_of(a, out);
  const int halves = out.halves, fblk = out.fblk;
  const int sms = num_sms();
  const int64_t seq_blocks = (int64_t)a.seqs.B * out.nblk;
  const double pch = (a.prefix_len + kN - 1) / kN;
  const double sch = 0.5 + (double)a.seqs.total_k / a.seqs.B / kN;  // a sequence's own chunks, on average
  const double row_cost = (double)a.seqs.total_q * a.h * a.d_c * 8 / 4e6;  // partials of a piece: us at 4 TB/s
  double best = 1e30;
  // one key axis
  for (int s = 1; s <= most_pieces(seq_blocks, halves); ++s) {
    const double len = (pch + sch) / s;
    if (s > 1 && (len < 2 || partial_bytes(a, s) > kMostPartial)) break;
    const int64_t items = seq_blocks * halves * s;
    const double waves = (double)((items + sms - 1) / sms);
    const double cost = waves * (ceil(len) + kStart) + (s > 1 ? 3 + s * row_cost : 0);
    if (cost < best) {
      best = cost;
      out.fblk = 0; out.sp = 0; out.ss = s;
    }
  }
  // the prefix by blocks of all rows, the sequences' own keys apart
  const bool apart = a.prefix_len > 0 && fblk < seq_blocks;
  for (int s = 1; apart && s <= most_pieces(fblk, halves); ++s) {
    const double len = pch / s;
    if (s > 1 && len < 2) break;
    int ss = (int)(sch / (len > 2 ? len : 2) + 0.5);
    const int most = most_pieces(seq_blocks, halves);
    ss = ss < 1 ? 1 : ss > most ? most : ss;
    if (partial_bytes(a, s + ss) > kMostPartial) break;
    const double work = halves * (fblk * (pch + s * kStart) + seq_blocks * (sch + ss * kStart));
    const double longest = ceil(len) + kStart;
    const double items = (double)halves * fblk * s;
    const double waves = ceil(items / sms) * longest;
    const double cost = (work / sms > waves ? work / sms + 0.3 * longest : waves) + 3 + (s + ss) * row_cost;
    if (cost < best) {
      best = cost;
      out.fblk = fblk; out.sp = s; out.ss = ss;
    }
  }
  out.merge.table = 0;
  out.merge.base = 0;
  out.merge.pieces = out.fblk ? out.sp + out.ss : out.ss;
  // equal shares, cut anywhere
  for (int f = 0; f <= (apart ? 1 : 0); ++f) {
    Plan t;
    t.halves = halves;
    t.nblk = out.nblk;
    const double time = cut_equal(a, f ? fblk : 0, t);
    if (time >= 1e30) continue;
    const double lines = (double)seq_blocks + (f ? fblk : 0);
    const double cost = time + 3 + (f ? 2 : 1) * (t.nseg / lines) * row_cost;
    if (cost < best) {
      best = cost;
      t.fblk = f ? fblk : 0;
      t.sp = t.ss = 0;
      out = t;
    }
  }
}

}  // namespace

bool prefix_tc_eligible(const PrefixArgs& a) {
  const int D = a.d_c + a.d_rope;
  return a.kv_dtype == DSA_BF16 && a.d_c <= 512 && D >= 64 && D <= 576;
}

// Pieces the workspace has room for, whatever the prefix's length.
int prefix_tc_most_pieces(const PrefixArgs& a) {
  Plan pl;
  blocks_of(a, pl);
  const int64_t seq_blocks = (int64_t)a.seqs.B * pl.nblk;
  if (pl.fblk == 0 || seq_blocks == 0) return 1;
  const int one = most_pieces(seq_blocks, pl.halves);
  const int two = pl.fblk < seq_blocks ? most_pieces(pl.fblk, pl.halves) + one : 1;
  int n = one > two ? one : two;
  while (n > 1 && partial_bytes(a, n) > kMostPartial) --n;
  return n;
}

int launch_prefix_tc(const PrefixArgs& a, cudaStream_t stream) {
  Plan pl;
  plan_of(a, pl);
  Params p{};
  p.a = a;
  p.nblk = pl.nblk;
  p.fblk = pl.fblk;
  p.sp = pl.sp;
  p.ss = pl.ss;
  p.halves = pl.halves;
  p.nseg = pl.nseg;
  p.ns = pl.ns;
  p.merged = pl.merge.pieces > 1;
  p.prefix_items = pl.fblk * pl.sp;
  p.chunk_rows = a.seqs.paged() && a.seqs.page_size < kN ? a.seqs.page_size : kN;
  const int64_t items =
      (pl.nseg ? pl.nseg : p.prefix_items + (int64_t)a.seqs.B * pl.nblk * pl.ss) * pl.halves;
  if (items > 0x7fffffff) return set_error(DSA_ERR_UNSUPPORTED, "prefix attention: grid too large");
  const uint64_t D = a.d_c + a.d_rope, keys = (uint64_t)a.seqs.cache_rows();
  const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int nk = a.d_c == 512 && (a.d_rope == 64 || a.d_rope == 0) ? (a.d_rope ? 5 : 4) : 0;
  const bool fixed = nk > 0;
  Maps m;
  int rc = make_tmap_2d(&m.q, bf, a.q, D, (uint64_t)a.seqs.total_q * a.h, D * 2, 64, kM);
  if (rc == DSA_OK) rc = make_tmap_2d(&m.key, bf, a.kv, D, keys, D * 2, 64, (uint32_t)p.chunk_rows);
  m.key4 = m.key;
  if (rc == DSA_OK && fixed && p.chunk_rows == kN) rc = make_tmap_tiles(&m.key4, bf, a.kv, D / 64, keys, D * 2, 4, kN);
  m.pre = m.key;
  m.pre4 = m.key4;
  if (a.prefix_kv) {
    const uint64_t n = (uint64_t)a.prefix_len;
    if (rc == DSA_OK) rc = make_tmap_2d(&m.pre, bf, a.prefix_kv, D, n, D * 2, 64, (uint32_t)p.chunk_rows);
    if (rc == DSA_OK && fixed) rc = make_tmap_tiles(&m.pre4, bf, a.prefix_kv, D / 64, n, D * 2, 4, kN);
  }
  if (rc != DSA_OK) return rc;
  auto kern = nk == 5 ? prefix_tc_kernel<5> : nk == 4 ? prefix_tc_kernel<4> : prefix_tc_kernel<0>;
  static std::atomic<bool> allowed[6][64];
  rc = allow_smem<kSmem>(kern, allowed[nk], "prefix_tc: smem attribute");
  if (rc != DSA_OK) return rc;
  cudaError_t e = cudaSuccess;
  DSA_LAUNCH("prefix_tc", stream,
             e = launch_pdl(kern, dim3((unsigned)items), dim3(kThreads), kSmem, stream, p, m, pl.cuts));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "prefix_tc: %s", cudaGetErrorString(e));
  rc = check_launch("prefix_tc");
  if (rc != DSA_OK || !p.merged) return rc;
  return launch_prefix_merge(a, pl.merge, stream);
}

}  // namespace dsa
