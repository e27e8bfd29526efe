// Sparse attention over the 4-bit latent cache on tcgen05 tensor cores (bf16 queries, 512 + 64 columns, up to 128 heads).
//
//   S_i = scale · q[t,h,:]·kv[row_i, :],  out = Σ softmax(S)_i · kv[row_i, :512],  lse = log Σ exp S_i
//
// A query's heads are the MMA's M = 128 rows, a CTA takes a query (or a piece of its entries, joined afterwards), and
// goes over its entries twice, 64 at a time:
//   phase 1, logits:  S = Q·Kᵀ (M=128, N=64, K=576), p = 2^(S − m) to a scratch of the CTA (16 KB a chunk, in L2)
//   phase 2, values:  O += P·V (M=128, N=2·256, K=64)
// Why twice.  A 128 x 512 fp32 accumulator is all of the tensor memory, so logits and values do not fit it together.  (The first
// form was one pass by two CTAs a query, each with half the values, both with the whole logits from a query of which five
// ninths were in shared memory: 3,500 clocks a chunk in each of the two.)  Apart, the query's 288 columns and three logit buffers fill the
// tensor memory in phase 1, the accumulator does in phase 2, and nothing is multiplied twice: 2,212 clocks of MMAs a chunk.  The
// price is that rows are copied and decoded twice and P goes through L2.
//
// What bounds it: not the MMAs (taking all but one of a chunk's out changes nothing), but the way of a chunk through
// gather, decoding, softmax and their hand-overs, some 4,200 clocks for both phases: instructions (54 % of the issue slots), 1,152
// clocks of operand stores, and the chains of waits between the roles.  1,024 queries of 2,048 entries, 128 heads: 541 us
// (0.57 of the MMAs' floor), with one pass 890.  Steps on the way there: rows gathered by TMA, four 416-byte rows a copy (87
// clocks each: 730), by 16-byte asynchronous copies of the decoding warps (662), scales two at a time (618), fp16 logits (591), decoding in two groups
// (538).  Loads straight to registers took 843: a warp's loads and its index loads wait for each other.  32 queries of 2,048 entries: 36.8 us
// of four CTAs each, of which the first MMA comes after 13,000 clocks, eight chunks take 31,000 and O's way out 22,000.
//
// The running maximum m of a head only decides the scale of p: it starts as the first chunk's, rounded up to a whole number (of log2), moves
// by whole numbers when a chunk's maximum is more than 2^8 above it, and phase 2 brings a chunk's p to the last m by a power of two, which
// is exact, instead of rescaling O.  (Whole numbers stay whole in fp32 at any size; a sum with a fraction would be rounded, and the step
// from one m to the next would be no power of two: of logits about 2^17, sums of p were off by up to 1.4 of its roundings.)
// The sum is in fp32 of the unrounded p.  P is rounded to bf16, which the MMA wants beside bf16 values: 2^-8 of each p at
// most, in either direction, whatever the output's type (bf16 outputs are 0.0020 to 0.0021 off the 64-bit result, relative to its size, where
// rounding them alone gives 0.0017).
//
// Roles of a CTA's 24 warps: four take the softmax, a thread a head; sixteen gather and decode, in two groups that take
// the chunks in turn; one issues the MMAs (its warp group's other three only look up entries).  The CTAs are persistent, one an SM.  An item begins
// with its entries looked up by all warps (cache rows, without skipped entries, to a list in L2) while its query is loaded.
//
// Shared memory: two chunks of nine tiles of [64 keys x 64 columns] in phase 1, four halves of a chunk and two P tiles in
// phase 2; a stage of gathered rows a group.  Every wait is bounded (DSA_FLAG_TIMEOUT).
//
// Pieces of a query in a cluster: each CTA tells the others its heads' (m, l) after phase 1, brings its O to the common m and sum on
// its way from tensor to shared memory, and sums up its share of the columns of all pieces from there, in their order, at 16
// bytes a clock and CTA (192 KB: 12,000 clocks; half as fast in shares of 128 bytes; loads for several rows at once, shares kept together and a
// share's sums while the next columns are put there were no faster).  Partial outputs through L2 and a merge in their place took 42 us
// (the merge 13), but suit pieces shorter than a quarter.
#include <float.h>

#include <type_traits>

#include "kv4.cuh"
#include "tc_sm100.cuh"

namespace dsa {
namespace {

using namespace tc;

constexpr int kM = 128;                    // heads
constexpr int kN = 64;                     // entries of a chunk
constexpr int kTile = kN * 128;            // 8 KB: 64 keys x 64 columns
constexpr int kQTile = kM * 128;           // 16 KB: 128 heads x 64 columns, or a chunk's P
constexpr int kDc = 512, kDr = 64, kD = kDc + kDr;
constexpr int kTiles = kD / 64, kVTiles = kDc / 64;
constexpr int kRow = kv4_row_bytes(kDc, kDr), kRaw = kN * kRow;  // a gathered chunk: 26 KB
constexpr int kKSlots = 2, kKSlot = kTiles * kTile;              // phase 1: 2 x 72 KB
constexpr int kVSlots = 4, kVSlot = kVTiles / 2 * kTile;         // phase 2: 4 x 32 KB (half the columns of a chunk)
constexpr int kPSlots = 2;                                       //   and 2 x 16 KB
constexpr int kSBufs = 3;                  // logit buffers
constexpr int kSoftWarps = 4;
constexpr int kGroups = 2, kDecoders = 8;  // groups of decoding warps, which take the chunks in turn
constexpr int kMmaWarp = kSoftWarps + kGroups * kDecoders;
constexpr int kThreads = 32 * (kMmaWarp + 4);  // (whole groups of four warps: their registers are set together)
constexpr int kParts = (kSoftWarps + kGroups * kDecoders) / 4;  // warps that take a quarter of the heads to tensor memory
// Registers a thread of softmax, of the decoders, of the MMA's four warps; together at most what the block is launched with (a build with
// fewer would wait forever for those that softmax asks for).  `regs`: what the compiler reports, of which a warp gets whole eights.
constexpr int kSoftRegs = 136, kDecodeRegs = 72, kMmaRegs = 56;
constexpr bool registers_suffice(int regs) {
  const int held = (regs + 7) / 8 * 8;
  return held >= kDecodeRegs && held <= kSoftRegs &&
         128 * kSoftRegs + 32 * kGroups * kDecoders * kDecodeRegs + 128 * kMmaRegs <= kThreads * held;
}
static_assert(registers_suffice(80) && registers_suffice(73) && !registers_suffice(72) && !registers_suffice(137), "registers");
constexpr int kRing = kVSlots * kVSlot + kPSlots * kQTile;
constexpr int kBarBytes = 512, kTopBytes = 2 * kM * 4;
constexpr int kMostPieces = 4;             // of a query: CTAs of a cluster
constexpr int kSumBytes = kMostPieces * kM * 8;
constexpr int kSmem = kRing + kGroups * kRaw + kBarBytes + kTopBytes + kSumBytes + 1024;
constexpr int kQCol = 0, kSCol = kD / 2;   // tensor memory of phase 1: 288 query columns, the logits; of phase 2: O
constexpr int kRopeAt = kv4_rope_at(kDc), kScaleAt = kv4_scale_at(kDc, kDr);
constexpr float kGrowLog2 = 8.0f;
constexpr int kNoQuery = 1 << 20;
constexpr int kMostRows = 2048;            // entries of a query
constexpr int64_t kPBytes = kM * kN * 2, kRefBytes = kM * 4, kListBytes = kN * 4;  // scratch of a chunk
static_assert(kSmem <= 232448, "shared memory");
static_assert(kSCol + kSBufs * kN <= 512, "tensor memory");
static_assert(kKSlots * kKSlot <= kRing, "phase 1's ring");
static_assert(kTiles * kQTile <= kRing, "the query passes through the ring");
constexpr int kOutRow = 1024;              // the output leaves through the ring, 256 fp32 columns of 128 heads at a time
static_assert(kM * kOutRow <= kVSlots * kVSlot, "the output's way through the ring");

struct Params {
  Attn4Args a;
  int chunks;     // of a query
  int items;      // queries, or pieces of all of them that leave partial outputs
  int most;       // chunks of the longest piece
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

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// 16 bytes to shared memory, asynchronously.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Phase 1's operand: fp16, 2^-3 times the value.  A code's two bits and a scale's four, from 2^-17 · 0.5 to 61440 · 6, are fp16
// numbers exactly that way, subnormal ones among them, and the conversion is the hardware's: two instructions a pair instead of
// five.  It takes a byte, two neighbouring nibbles: pairs of columns (0, 2), (4, 6), (1, 3), (5, 7) of eight, so the
// query's columns stand in that order too.
constexpr float kShrinkK = 0x1p-3f;
constexpr uint32_t kShrinkKf16 = 0x30003000u, kShrinkKbf16 = 0x3e003e00u;  // 2^-3 twice
// Phase 2's: bf16 beside P's (an fp16 P would lose what is 2^-39 of a row's largest), 2^-14 times the value: kv4_pair() times the scale
// times 2^112, which is within bf16's range for every scale and brings the first one that is none (0xf8) to infinity.
constexpr float kShrinkV = 0x1p-14f;
constexpr uint32_t kUp112 = 0x77807780u;  // 2^112 twice in bf16

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 32 columns (a gathered row's 16-byte piece and their two scales) into the four 16-byte pieces of an operand row from logical piece c
// on, XOR-ed with x.  Both scales are decoded at once (their exponent and mantissa go to fp16's or bf16's places); infinity times 0,
// added, makes a scale that is not a number one.
__device__ __forceinline__ void decode32_k(uint8_t* row, int c, int x, const uint4& w, uint32_t scales) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t two = mul_f16x2(__byte_perm(scales, 0u, 0x4140) << 7, kShrinkKf16);
  asm("fma.rn.f16x2 %0, %0, %1, %0;" : "+r"(two) : "r"(0u));
  const uint32_t s[2] = {__byte_perm(two, two, 0x1010), __byte_perm(two, two, 0x3232)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t o[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(u[i]));
    const uint32_t f = s[i >> 1];
    *reinterpret_cast<uint4*>(row + (((c + i) ^ x) * 16)) =
        make_uint4(mul_f16x2(o[0], f), mul_f16x2(o[1], f), mul_f16x2(o[2], f), mul_f16x2(o[3], f));
  }
}
__device__ __forceinline__ void decode32_v(uint8_t* row, int c, int x, const uint4& w, uint32_t scales) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t two = mul_bf16x2(mul_bf16x2(__byte_perm(scales, 0u, 0x4140) << 4, kUp112), kUp112);
  asm("fma.rn.bf16x2 %0, %0, %1, %0;" : "+r"(two) : "r"(0u));
  const uint32_t s[2] = {__byte_perm(two, two, 0x1010), __byte_perm(two, two, 0x3232)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t f = s[i >> 1];
    *reinterpret_cast<uint4*>(row + (((c + i) ^ x) * 16)) =
        make_uint4(mul_bf16x2(kv4_pair<0>(u[i]), f), mul_bf16x2(kv4_pair<1>(u[i]), f),
                   mul_bf16x2(kv4_pair<2>(u[i]), f), mul_bf16x2(kv4_pair<3>(u[i]), f));
  }
}

// kind::f16 with both operands fp16 (format 0), fp32 accumulate, K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The larger of pairs of bf16 (a NaN is passed over).
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// A pair of bf16 magnitudes with 0 for an infinity or a NaN.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
  return w;
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

// The block's barrier, which each role meets in its own code.  (Warp-aligned, as those of the cluster: each reconverges the warp first,
// whose lanes may come apart from a role's loop.)
__device__ __forceinline__ void block_sync() {
  __syncwarp();
  asm volatile("barrier.cta.sync.aligned 0;" ::: "memory");
}

// The cluster's barrier in two halves, and its shared memory (addresses of mapa()).
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float x, float y) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

struct Item {
  bool good;  // the query belongs to a sequence
  int piece, nch, total;
  int64_t row0;
};

template <int S>
__global__ void __cluster_dims__(S, 1, 1) __launch_bounds__(kThreads, 1)
attn4_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap qmap) {
  const Attn4Args& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = S > 1 ? (int)cluster_ctarank() : 0;
  const int64_t rows_all = (int64_t)a.seqs.total_q * a.h;
  const bool partial = S == 1 && a.splits > 1;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* ptiles = ring + kVSlots * kVSlot;
  uint8_t* raw = ring + kRing;     // [2][64][416]
  uint64_t* bars = reinterpret_cast<uint64_t*>(raw + kGroups * kRaw);
  uint64_t* k_full = bars;         // [2] 8 warps have stored a chunk's tiles
  uint64_t* k_empty = bars + 2;    // [2] multiplied
  uint64_t* s_full = bars + 4;     // [3] logits complete
  uint64_t* s_empty = bars + 7;    // [3] read
  uint64_t* v_full = bars + 10;    // [4]
  uint64_t* v_empty = bars + 14;   // [4]
  uint64_t* p_full = bars + 18;    // [2]
  uint64_t* p_empty = bars + 20;   // [2]
  uint64_t* q_staged = bars + 22;  // the query on its way to tensor memory
  uint64_t* qt_full = bars + 23;   // there
  uint64_t* o_full = bars + 24;    // O complete
  constexpr int kBars = 25;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + kBars + 1);
  int* counts = reinterpret_cast<int*>(bars + kBars + 2);  // [warps] entries of a warp's share
  uint32_t* tops = reinterpret_cast<uint32_t*>(bars + kBarBytes / 8);  // [2][128] largest magnitude of a head's latent, rope columns
  int* holds = counts + kThreads / 32;                     // [pieces] entries of a piece
  float2* sums = reinterpret_cast<float2*>(tops + 2 * kM);  // [pieces][128] a piece's (m, l)
  static_assert((kBars + 2) * 8 + (kThreads / 32 + kMostPieces) * 4 <= kBarBytes, "barriers");

  const int live_warps = (a.h + 31) / 32;  // of the softmax: the others' rows are no head's
  if (warp == kMmaWarp) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKSlots; ++i) { mbar_init(&k_full[i], kDecoders); mbar_init(&k_empty[i], 1); }
    for (int i = 0; i < kSBufs; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], live_warps); }
    for (int i = 0; i < kVSlots; ++i) { mbar_init(&v_full[i], kDecoders); mbar_init(&v_empty[i], 1); }
    for (int i = 0; i < kPSlots; ++i) { mbar_init(&p_full[i], live_warps); mbar_init(&p_empty[i], 1); }
    mbar_init(q_staged, 1);
    mbar_init(qt_full, live_warps * kParts);
    mbar_init(o_full, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  uint8_t* const scratch = a.scratch + (int64_t)blockIdx.x * p.most * (kPBytes + kRefBytes + kListBytes);
  float* const refs = reinterpret_cast<float*>(scratch + (int64_t)p.most * kPBytes);  // [chunk][128]
  int32_t* const list = reinterpret_cast<int32_t*>(refs + (int64_t)p.most * kM);  // cache rows of the entries, without those skipped
  tc_fence_before();
  if (S > 1) cluster_sync();  // (the others' shared memory is written from the first item on)
  else block_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Barriers and tensor memory are set up beside the kernel before; what a caller wrote is read from here on.  Only the merge, which reads
  // offsets ahead of its own wait, may start early, and not before this wait (a caller's next kernel may read what this one waits for).
  griddep_wait();
  if (partial) griddep_launch();
  // The barriers' phases go on from item to item: chunks so far, the parity of the items and of those that had any.
  uint32_t done = 0, turn = 0, full_turn = 0;
  // An item's query, its entries' chunks.
  auto begin = [&](int item, Item& it) {
    const int t = S > 1 ? item : item / a.splits, pieces = S > 1 ? S : a.splits;
    it.piece = S > 1 ? rank : item - t * a.splits;
    it.row0 = (int64_t)t * a.h;
    // The query comes while the entries are looked up (the ring is free: all roles have left the item before).
    if (warp == kMmaWarp && elect_one()) {
      mbar_arrive_expect_tx(q_staged, kTiles * kQTile);
      for (int j = 0; j < kTiles; ++j) tma_load_2d(ring + j * kQTile, &qmap, q_staged, j * 64, (int)it.row0);
    }
    __syncwarp();
    const int c0 = p.chunks * it.piece / pieces, c1 = p.chunks * (it.piece + 1) / pieces;
    const int32_t* idx = a.idx + (int64_t)t * a.top_k;
    const int end = min(a.top_k, c1 * kN);
    // The piece's entries as cache rows, without the skipped ones (a short history's row is mostly -1): a warp takes
    // consecutive ones, all its loads at once, ahead of the row's lookup.
    constexpr int kWarps = kThreads / 32, kMine = (kMostRows + 32 * kWarps - 1) / (32 * kWarps);
    const int per_warp = (end - c0 * kN + 32 * kWarps - 1) / (32 * kWarps);  // at most kMine
    int row[kMine], mine = 0;
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int e = c0 * kN + (warp * per_warp + j) * 32 + lane;
      row[j] = j < per_warp && e < end ? idx[e] : -1;
    }
    if (threadIdx.x < 2 * kM) tops[threadIdx.x] = 0u;
    RowInfo ri;
    const bool good = warp_query_row(a, t, lane, ri);
    if (good) {
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const int v = row[j];
        row[j] = v >= 0 && v <= ri.pos ? cache_row(a.seqs, ri.b, ri.k0, v) : -1;
        if (row[j] < 0 && v != -1) atomicOr(a.status, DSA_FLAG_BAD_INDEX);
        if (!dsa_check(row[j] < a.seqs.cache_rows(), a.status)) row[j] = -1;
        mine += __popc(__ballot_sync(0xffffffffu, row[j] >= 0));
      }
      if (lane == 0) counts[warp] = mine;
    }
    tc_fence_before();
    block_sync();
    tc_fence_after();
    int total = 0;
    if (good) {
      const int c = lane < kWarps ? counts[lane] : 0;
      int at = __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
      total = __reduce_add_sync(0xffffffffu, c);
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const uint32_t m = __ballot_sync(0xffffffffu, row[j] >= 0);
        if (row[j] >= 0) list[at + __popc(m & ((1u << lane) - 1u))] = row[j];
        at += __popc(m);
      }
    }
    block_sync();
    it.good = good;
    it.total = total;
    it.nch = (total + kN - 1) / kN;
  };
  // The query to tensor memory, by all warps but the MMA's: those of a quarter of the heads (each warp can write to one) take a few
  // of the column tiles each.  The latent columns go to fp16, times the power of two that brings the head's largest finite one into
  // [2^14, 2^15): a column is off by at most 2^-39 of it, so those below 2^-29 of it lose bits and those below 2^-39 are 0.  (That is below
  // the rounding of a logit to which the largest column adds; where a key's code in that column is 0 it is not.)  The rope columns get the
  // same factor, which is held where they stay within bf16's range.  The factor's exponent, or kNoQuery (a wait was given up).
  auto stage_query = [&](int quarter, int part) -> int {
    const int r = quarter * 32 + lane;
    const bool ok = __all_sync(0xffffffffu, mbar_wait(q_staged, turn, abort_flag, a.status, DSA_FLAG_TIMEOUT));
    const bool mine = ok && quarter < live_warps;
    const uint8_t* const row = ring + r * 128;
    auto piece = [&](int j, int i) { return *reinterpret_cast<const uint4*>(row + j * kQTile + ((i ^ (r & 7)) * 16)); };
    for (int j = part; mine && j < kTiles; j += kParts) {
      uint32_t t = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 v = piece(j, i);
        t = max_bf16x2(max_bf16x2(t, v.x & 0x7fff7fffu),
                       max_bf16x2(v.y & 0x7fff7fffu, max_bf16x2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
      }
      if (__any_sync(0xffffffffu, finite_pair(t) != t)) {  // infinities: once more without them (the maximum passes NaNs over)
        t = 0u;
        for (int i = 0; i < 8; ++i) {
          const uint4 v = piece(j, i);
          t = max_bf16x2(t, max_bf16x2(max_bf16x2(finite_pair(v.x & 0x7fff7fffu), finite_pair(v.y & 0x7fff7fffu)),
                                       max_bf16x2(finite_pair(v.z & 0x7fff7fffu), finite_pair(v.w & 0x7fff7fffu))));
        }
      }
      atomicMax(&tops[(j == kVTiles ? kM : 0) + r], max(t & 0x7fffu, t >> 16 & 0x7fffu));
    }
    __syncwarp();
    asm volatile("barrier.cta.sync.aligned 1, %0;" ::"n"(32 * kMmaWarp) : "memory");
    if (!ok) return kNoQuery;
    const int e0 = (int)(tops[r] >> 7) - 127, e1 = (int)(tops[kM + r] >> 7) - 127;  // (0 and subnormal: -127)
    const int shift = min(max(e0 == -127 ? 0 : e0 - 14, max(e1 - 100, -100)), 113);
    const float down = __uint_as_float((uint32_t)(127 - shift) << 23);
    const uint32_t two = (uint32_t)(127 - shift) * 0x00800080u;  // the same twice in bf16
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    for (int j = part; mine && j < kTiles; j += kParts) {
      uint32_t w[32];
      if (j < kVTiles) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = piece(j, i);
          auto lo = [&](uint32_t u) { return __uint_as_float(u << 16) * down; };
          auto hi = [&](uint32_t u) { return __uint_as_float(u & 0xffff0000u) * down; };
          w[4 * i] = f16x2(lo(v.x), lo(v.y));
          w[4 * i + 1] = f16x2(lo(v.z), lo(v.w));
          w[4 * i + 2] = f16x2(hi(v.x), hi(v.y));
          w[4 * i + 3] = f16x2(hi(v.z), hi(v.w));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = piece(j, i);
          w[4 * i] = mul_bf16x2(v.x, two); w[4 * i + 1] = mul_bf16x2(v.y, two);
          w[4 * i + 2] = mul_bf16x2(v.z, two); w[4 * i + 3] = mul_bf16x2(v.w, two);
        }
      }
      __syncwarp();
      tmem_st32(lane_base + kQCol + j * 32, w);
    }
    tc_fence_before();
    __syncwarp();
    if (mine && lane == 0) mbar_arrive(qt_full);
    return shift;
  };
  auto sync = [&] {
    if (S > 1) cluster_sync();
    else block_sync();
  };
  // The item's end, of all roles: O, scaled, to shared memory and from there, summed over the query's pieces, to the output: 256
  // columns at a time (pieces of up to 64 heads: all), of which each CTA of the cluster takes its share of all heads.  False: a wait was given up.
  auto finish = [&](const Item& it) -> bool {
    // (Without entries nobody else waited for the query, and where a wait was given up it may still be on its way.)
    if (warp == kMmaWarp) mbar_wait_drain(q_staged, turn);
    if (S > 1) cluster_wait();  // the pieces' sums are there
    else block_sync();
    bool stopped = false;
    if (it.good) {
      const bool stages = warp >= kSoftWarps && warp < kMmaWarp && (warp & 3) < live_warps && it.nch;
      const int r = (warp & 3) * 32 + lane;
      float factor = 0.f;
      if (warp < kMmaWarp) {
        float top = -FLT_MAX, sum = 0.f;
#pragma unroll
        for (int c = 0; c < S; ++c) top = fmaxf(top, sums[c * kM + r].x);
#pragma unroll
        for (int c = 0; c < S; ++c) sum += sums[c * kM + r].y * ex2(sums[c * kM + r].x - top);
        factor = sum == 0.f ? 0.f : ex2(sums[rank * kM + r].x - top) / sum * (1.f / kShrinkV);
        if (partial) {
          factor = 1.f / kShrinkV;
          if (warp < kSoftWarps && r < a.h) a.part_ml[it.piece * rows_all + it.row0 + r] = sums[r];
        } else if (a.lse && warp < kSoftWarps && rank == 0 && r < a.h) {
          a.lse[it.row0 + r] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
        }
      }
      if (stages) {
        mbar_wait(o_full, full_turn, abort_flag, a.status, DSA_FLAG_TIMEOUT);
        tc_fence_after();
      }
      auto put_out = [&](auto columns) {
        constexpr int kCols = decltype(columns)::value;
#pragma unroll
        for (int half = 0; half < kDc / kCols; ++half) {
          if (stages) {
#pragma unroll 1
            for (int c = (warp - kSoftWarps) / 4; c < kCols / 32; c += kGroups * kDecoders / 4) {
              uint32_t o[32];
              __syncwarp();  // the load is the whole warp's
              tmem_ld32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * kCols + c * 32, o);
              uint8_t* const to = ring + r * (kCols * 4) + c * 128;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float4*>(to + ((i ^ (r & 7)) * 16)) =
                    make_float4(__uint_as_float(o[4 * i]) * factor, __uint_as_float(o[4 * i + 1]) * factor,
                                __uint_as_float(o[4 * i + 2]) * factor, __uint_as_float(o[4 * i + 3]) * factor);
            }
            tc_fence_before();
            fence_proxy_async_smem();  // the next query comes to the same place
          }
          sync();
          constexpr int kPer = kCols / 4 / S;  // 16-byte pieces of a row that are this CTA's
          for (int i = threadIdx.x; i < a.h * kPer; i += kThreads) {
            const int row = i / kPer, k = rank * kPer + i % kPer;
            const uint32_t at = smem_u32(ring) + row * (kCols * 4) + ((k ^ (row & 7)) * 16);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            constexpr int kAtOnce = S < 4 ? S : 4;
#pragma unroll
            for (int c0 = 0; c0 < S; c0 += kAtOnce) {
              float4 v[kAtOnce];
#pragma unroll
              for (int c = 0; c < kAtOnce; ++c)
                v[c] = holds[c0 + c] == 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : ld_cluster4(S > 1 ? mapa(at, c0 + c) : at);
#pragma unroll
              for (int c = 0; c < kAtOnce; ++c) o = make_float4(o.x + v[c].x, o.y + v[c].y, o.z + v[c].z, o.w + v[c].w);
            }
            const int64_t to = (it.row0 + row) * kDc + half * kCols + k * 4;
            if (partial) *reinterpret_cast<float4*>(a.part_o + it.piece * rows_all * kDc + to) = o;
            else if (a.out_dtype == DSA_F32) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + to) = o;
            else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + to) = make_uint2(bf16x2(o.x, o.y), bf16x2(o.z, o.w));
          }
          // (all pieces stop together: none writes to what another has left)
          if (S > 1 && half == kDc / kCols - 1)
            stopped = __any_sync(0xffffffffu, ld_cluster(mapa(smem_u32(const_cast<int*>(abort_flag)), lane % S)) != 0);
          sync();
        }
      };
      if (S > 1 && a.h <= 64) put_out(std::integral_constant<int, 512>());
      else put_out(std::integral_constant<int, 256>());
    }
    turn ^= 1;
    if (it.nch) full_turn ^= 1;
    done += it.nch;
    if (S == 1) {
      if (!it.good) block_sync();
      // (of offsets that do not rise the merge's search may find another sequence, a consistent one)
      if (partial && !it.good && threadIdx.x < a.h) a.part_ml[it.piece * rows_all + it.row0 + threadIdx.x] = make_float2(0.f, -1.f);
      stopped = *abort_flag != 0;
    } else if (!it.good) {
      cluster_sync();
    }
    return !stopped;
  };
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
    for (int item = blockIdx.x / S; item < p.items; item += gridDim.x / S) {
      Item it;
      begin(item, it);
      const int nch = it.nch;
      if (S > 1) cluster_arrive();
      if (nch && warp == kMmaWarp) {
        // ---------------- query loads, MMA issue ----------------
        if (elect_one()) {
          const uint32_t idesc_s = idesc_f16(kM, kN), idesc_r = idesc_bf16(kM, kN), idesc_pv = idesc_bf16(kM, 256, false, true);
          const uint64_t kd0 = sdesc_sw128(smem_u32(ring), 16, 1024);
          const uint64_t vd0 = sdesc_sw128(smem_u32(ring), kTile, 1024);  // V tiles as P·V reads them
          const uint64_t pd0 = sdesc_sw128(smem_u32(ptiles), 16, 1024);
          bool stop = !mbar_wait(qt_full, full_turn, abort_flag, a.status, DSA_FLAG_TIMEOUT);
          for (int g = 0; g < nch && !stop; ++g) {
            const uint32_t n = done + g, ks = n % kKSlots, sb = n % kSBufs;
            if (!mbar_wait(&s_empty[sb], ((n / kSBufs) & 1) ^ 1, abort_flag, a.status, DSA_FLAG_TIMEOUT) ||
                !mbar_wait(&k_full[ks], (n / kKSlots) & 1, abort_flag, a.status, DSA_FLAG_TIMEOUT)) {
              stop = true;
              break;
            }
            tc_fence_after();
            const uint32_t d = tmem + kSCol + sb * kN;
            const uint64_t kd = kd0 + (uint64_t)(ks * (kKSlot >> 4));
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mma_bf16_ts(d, tmem + kQCol + j * 32 + i * 8, kd + (uint64_t)(j * (kTile >> 4) + i * 2), j < kVTiles ? idesc_s : idesc_r,
                            j || i ? 1u : 0u);
            mma_commit(&k_empty[ks]);
            mma_commit(&s_full[sb]);
          }
          for (int g = 0; g < 2 * nch && !stop; ++g) {  // half g & 1 of the columns
            const uint32_t n = done + (g >> 1), vn = 2 * done + g, vs = vn % kVSlots, ps = n % kPSlots;
            if (!mbar_wait(&v_full[vs], (vn / kVSlots) & 1, abort_flag, a.status, DSA_FLAG_TIMEOUT) ||
                ((g & 1) == 0 && !mbar_wait(&p_full[ps], (n / kPSlots) & 1, abort_flag, a.status, DSA_FLAG_TIMEOUT)))
              break;
            tc_fence_after();
            const uint64_t vd = vd0 + (uint64_t)(vs * (kVSlot >> 4)), pd = pd0 + (uint64_t)(ps * (kQTile >> 4));
            const uint32_t acc = g > 1;
#pragma unroll
            for (int kk = 0; kk < kN / 16; ++kk)
              mma_bf16(tmem + (g & 1) * 256, pd + (uint64_t)(kk * 2), vd + (uint64_t)(kk * 128), idesc_pv, kk ? 1u : acc);
            mma_commit(&v_empty[vs]);
            if (g & 1) mma_commit(&p_empty[ps]);
          }
          mma_commit(o_full);
          mbar_wait_drain(o_full, full_turn);
        }
      }
      if (!finish(it)) break;
    }
  } else if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDecodeRegs));
    for (int item = blockIdx.x / S; item < p.items; item += gridDim.x / S) {
      Item it;
      begin(item, it);
      const int nch = it.nch, total = it.total;
      if (S > 1) cluster_arrive();
      if (nch) {
        // ---------------- gather and decode: the chunks of phase 1, then the same again for phase 2 ----------------
        // The two groups take the chunks in turn: a chunk is a chain of waits and latencies as long as its work, which the other
        // group's work fills.  A warp takes eight rows: their 16-byte pieces are copied to its part of the group's stage and
        // come to registers from there, when the copies of the group's next chunk begin.  Eight neighbouring lanes read pieces of four rows (8 banks
        // apart) and two pieces each, and store what they decode to at eight different places of the swizzle: no bank is
        // asked for twice.
        const int w = (warp - kSoftWarps) % kDecoders, group = (warp - kSoftWarps) / kDecoders;
        const int pair = (lane >> 2) & 1, grp = lane >> 4;
        const int r = w * 8 + ((lane >> 3) & 1) * 4 + (lane & 3), x = r & 7;  // row of the chunk
        // the group's chunks, and its steps: its chunks of phase 1, then the same again
        const int count = (nch - group + kGroups - 1) / kGroups, steps = 2 * count;
        auto chunk_of = [&](int i) { return group + kGroups * (i < count ? i : i - count); };
        // Lane l holds the cache row of the warp's row l & 7, read a step ahead of its copy.  Behind the last entry the last
        // one is repeated: its P is 0 there, and what its columns hold the query attends to anyway.
        auto load_row_of = [&](int i) { return __ldcg(list + min(chunk_of(i) * kN + w * 8 + (lane & 7), total - 1)); };
        constexpr int kPieces = kRow / 16, kCopies = (8 * kPieces + 31) / 32;
        uint8_t* const mine_raw = raw + group * kRaw + w * 8 * kRow;
        int next_row = load_row_of(0);
        auto gather = [&](int i) {
          const int row_of = next_row;
          next_row = load_row_of(i + 1);
          const uint32_t dst = smem_u32(mine_raw) + lane * 16;
#pragma unroll
          for (int c = 0; c < kCopies; ++c) {
            const int f = c * 32 + lane, j = f / kPieces;  // piece f of the warp's rows, in row j
            const int from = __shfl_sync(0xffffffffu, row_of, j & 7);
            if (f < 8 * kPieces) copy16_async(dst + c * 512, a.kv4 + (int64_t)from * kRow + (f - j * kPieces) * 16);
          }
        };
        if (steps) gather(0);
        bool stop = stage_query(warp & 3, 1 + (warp - kSoftWarps) / 4) == kNoQuery;
        for (int i = 0; !stop && i < steps; ++i) {
          const int n = i < count ? chunk_of(i) : nch + chunk_of(i);  // phase 1: [0, nch), phase 2: [nch, 2 nch)
          asm volatile("cp.async.wait_all;" ::: "memory");
          __syncwarp();
          const uint8_t* src = raw + group * kRaw + r * kRow;
          uint4 v[4], rope[2];  // piece j: columns 32 (2 (2 j + grp) + pair) ..
          uint32_t sc[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = 2 * (2 * j + grp) + pair;
            v[j] = *reinterpret_cast<const uint4*>(src + 16 * k);
            sc[j] = *reinterpret_cast<const uint16_t*>(src + kScaleAt + 2 * k);
          }
          if (n < nch) {
#pragma unroll
            for (int j = 0; j < 2; ++j) rope[j] = *reinterpret_cast<const uint4*>(src + kRopeAt + 16 * (2 * j + grp + 4 * pair));
          }
          __syncwarp();  // the stage has been read (a warp's loads of shared memory are served in order, ahead of the copies)
          if (i + 1 < steps) gather(i + 1);
          if (n < nch) {
            const uint32_t kn = done + n, ks = kn % kKSlots;
            // (the query passes through the tiles first)
            if (!__all_sync(0xffffffffu,
                            (n >= kKSlots || mbar_wait(qt_full, full_turn, abort_flag, a.status, DSA_FLAG_TIMEOUT)) &&
                                mbar_wait(&k_empty[ks], ((kn / kKSlots) & 1) ^ 1, abort_flag, a.status, DSA_FLAG_TIMEOUT)))
              break;
            uint8_t* tiles = ring + ks * kKSlot;
#pragma unroll
            for (int i = 0; i < 4; ++i) decode32_k(tiles + (2 * i + grp) * kTile + r * 128, 4 * pair, x, v[i], sc[i]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              *reinterpret_cast<uint4*>(tiles + kVTiles * kTile + r * 128 + (((2 * i + grp + 4 * pair) ^ x) * 16)) =
                  make_uint4(mul_bf16x2(rope[i].x, kShrinkKbf16), mul_bf16x2(rope[i].y, kShrinkKbf16), mul_bf16x2(rope[i].z, kShrinkKbf16),
                             mul_bf16x2(rope[i].w, kShrinkKbf16));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&k_full[ks]);
          } else {
            const int g = n - nch;
            // (the first tiles are some of phase 1's: its last MMAs are done)
            const uint32_t lg = done + nch - 1;
            bool ok = g >= kGroups || mbar_wait(&s_full[lg % kSBufs], (lg / kSBufs) & 1, abort_flag, a.status, DSA_FLAG_TIMEOUT);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t vn = 2 * (done + g) + h, vs = vn % kVSlots;
              ok = ok && mbar_wait(&v_empty[vs], ((vn / kVSlots) & 1) ^ 1, abort_flag, a.status, DSA_FLAG_TIMEOUT);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              uint8_t* tiles = ring + vs * kVSlot;
#pragma unroll
              for (int i = 0; i < 2; ++i)
                decode32_v(tiles + (2 * i + grp) * kTile + r * 128, 4 * pair, x, v[2 * h + i], sc[2 * h + i]);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&v_full[vs]);
            }
            if (!ok) break;
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");  // every copy has landed before the CTA goes on
      }
      if (!finish(it)) break;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    for (int item = blockIdx.x / S; item < p.items; item += gridDim.x / S) {
      Item it;
      begin(item, it);
      const int nch = it.nch, total = it.total;
      const int r = warp * 32 + lane;
      // The head's sum goes to all pieces' CTAs, which take O together.
      auto give = [&](float m, float l) {
        if (S == 1) {
          sums[r] = make_float2(fmaxf(m, -FLT_MAX), l);
          if (r == 0) holds[0] = total;
        } else {
#pragma unroll
          for (int c = 0; c < S; ++c) {
            st_cluster(mapa(smem_u32(&sums[rank * kM + r]), c), fmaxf(m, -FLT_MAX), l);
            if (r == 0) st_cluster(mapa(smem_u32(&holds[rank]), c), total);
          }
          cluster_arrive();
        }
      };
      if (nch == 0) give(-INFINITY, 0.f);
      if (nch) {
        // ---------------- softmax: thread = head ----------------
        const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
        const int shift = stage_query(warp & 3, 0);  // the row's logits are 2^shift times what its operands say
        bool stop = shift == kNoQuery || warp >= live_warps;  // (the others' rows are no head's)
        const float scale = a.scale_log2 * (1.f / kShrinkK) * __uint_as_float((uint32_t)(127 + shift) << 23);
        float m = -INFINITY, l = 0.f;  // the reference (log2 units) and the sum relative to it
        uint4* const pbuf = reinterpret_cast<uint4*>(scratch) + r;  // piece i of chunk g at [(8 g + i) · 128]
        for (int g = 0; g < nch && !stop; ++g) {
          const uint32_t n = done + g, sb = n % kSBufs;
          if (!__all_sync(0xffffffffu, mbar_wait(&s_full[sb], (n / kSBufs) & 1, abort_flag, a.status, DSA_FLAG_TIMEOUT))) {
            stop = true;
            break;
          }
          tc_fence_after();
          float z[kN];
          load_row(lane_base + kSCol + sb * kN, z);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[sb]);
          if (g == nch - 1) {  // behind the last entry
            const int n_in = total - g * kN;
#pragma unroll
            for (int i = 0; i < kN; ++i)
              if (i >= n_in) z[i] = -INFINITY;
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < kN; ++i) mx[i & 3] = fmaxf(mx[i & 3], z[i]);
          const float mc = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
          if (mc > m + kGrowLog2) {  // the first entries always (m = -inf)
            const float m_new = m == -INFINITY ? ceilf(mc) : m + ceilf(mc - m);
            l *= ex2(m - m_new);
            m = m_new;
          }
          const float ref = m == -INFINITY ? 0.f : m;  // nothing visible so far
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t pk[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p0 = ex2(fmaf(z[8 * i + 2 * e], scale, -ref));
              const float p1 = ex2(fmaf(z[8 * i + 2 * e + 1], scale, -ref));
              sum[(2 * e) & 3] += p0;
              sum[(2 * e + 1) & 3] += p1;
              pk[e] = bf16x2(p0, p1);
            }
            __stcg(pbuf + (8 * g + i) * kM, make_uint4(pk[0], pk[1], pk[2], pk[3]));
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          __stcg(refs + g * kM + r, m);
        }
        give(m, l);
        // phase 2: this thread's row of P, relative to the last m (a power of two: exact)
        uint4 pk[8];
        float ref = 0.f;
        auto load_p = [&](int g) {
#pragma unroll
          for (int i = 0; i < 8; ++i) pk[i] = __ldcg(pbuf + (8 * g + i) * kM);
          ref = __ldcg(refs + g * kM + r);
        };
        if (!stop) load_p(0);
        for (int g = 0; g < nch && !stop; ++g) {
          const uint32_t n = done + g, ps = n % kPSlots;
          // (phase 1's MMAs are done with the tiles: softmax has read their last logits)
          if (!__all_sync(0xffffffffu, mbar_wait(&p_empty[ps], ((n / kPSlots) & 1) ^ 1, abort_flag, a.status, DSA_FLAG_TIMEOUT))) {
            stop = true;
            break;
          }
          if (__any_sync(0xffffffffu, ref != m)) {
            const float f = ref == m ? 1.f : ex2(ref - m);
            const uint32_t ff = bf16x2(f, f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              pk[i] = make_uint4(mul_bf16x2(pk[i].x, ff), mul_bf16x2(pk[i].y, ff), mul_bf16x2(pk[i].z, ff),
                                 mul_bf16x2(pk[i].w, ff));
          }
          uint8_t* to = ptiles + ps * kQTile + r * 128;
#pragma unroll
          for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(to + ((i ^ (r & 7)) * 16)) = pk[i];
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[ps]);
          if (g + 1 < nch) load_p(g + 1);
        }
      }
      if (!finish(it)) break;
    }
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, 512);
  }
}

// In times of a chunk (both phases; 1.9 us): an item's start and end, the merge's launch, a partial output of 128 heads on its way through
// L2, and what a cluster's CTAs take to join an output.  Least squares' and then the choices' best fit of 110 sizes (1 to 608 queries, 16, 64
// and 128 heads, 512 to 2,048 entries) in every form: the rule's form takes 0.3 % longer than the fastest one on average, 9 % at most.
constexpr double kStart = 4.5, kMerge = 1.25, kPartial = 0.035;
double joining(int cluster, double heads) { return cluster > 1 ? (0.4 + 0.6 * heads) * (1 + cluster / 2) : 0; }
constexpr size_t kMostPartial = size_t(1) << 30;

int chunks_of(const Attn4Args& a) { return (a.top_k + kN - 1) / kN; }
// Clusters that are at work at once (a processing cluster's SMs are cut into them).
int clusters_of(int pieces) { return pieces == 1 ? num_sms() : pieces == 2 ? num_sms() / 2 : num_sms() * 9 / 38; }
int64_t ctas_of(const Attn4Args& a) {
  const int64_t items = (int64_t)a.seqs.total_q * a.splits, most = clusters_of(a.cluster);
  return (items < most ? items : most) * a.cluster;
}

// Whether the kernels were built with the registers that their roles are given: 1 or -1, asked of the runtime once; 0 where it has no
// device to ask (a workspace's size).
int built_to_run() {
  static std::atomic<int> known{0};
  const int k = known.load(std::memory_order_relaxed);
  if (k != 0) return k;
  bool ok = true;
  for (auto kern : {attn4_tc_kernel<1>, attn4_tc_kernel<2>, attn4_tc_kernel<4>}) {
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, kern) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    ok = ok && registers_suffice(attr.numRegs);
  }
  known.store(ok ? 1 : -1, std::memory_order_relaxed);
  return ok ? 1 : -1;
}

template <int S>
int launch_pieces(const Params& p, const CUtensorMap& qmap, cudaStream_t stream) {
  static std::atomic<bool> allowed[64];
  int rc = allow_smem<kSmem>(attn4_tc_kernel<S>, allowed, "attn4_tc: smem attribute");
  if (rc != DSA_OK) return rc;
  cudaError_t e = cudaSuccess;
  DSA_LAUNCH("attn4_tc", stream,
             e = launch_pdl(attn4_tc_kernel<S>, dim3((unsigned)ctas_of(p.a)), dim3(kThreads), kSmem, stream, p, qmap));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "attn4_tc: %s", cudaGetErrorString(e));
  return check_launch("attn4_tc");
}

}  // namespace

bool attn4_tc_eligible(const Attn4Args& a) {
  return a.kv_dtype == DSA_BF16 && a.d_c == kDc && a.d_rope == kDr && a.h <= kM && built_to_run() >= 0;
}

// Few queries are cut into pieces to fill the SMs: a round of items ends with its longest.  Either a cluster of 2 or 4 CTAs takes a
// query and joins its pieces in shared memory, or any number of CTAs leave partial outputs for a merge: a launch and their way
// through L2 more, but pieces of any length.  2,048 entries, us, clusters (CTAs) | partial outputs (pieces): 128 heads, 1 query 34.7 (4) | 20.3 (32),
// 12 queries 35.1 (4) | 29.2 (8), 24 queries 35.5 (4) | 35.9 (6), 32 queries 36.9 (4) | 40.4 (4), 64 queries 52.0 (2) | 67.7 (2); 16 heads, 4 queries
// 26.2 (4) | 17.7 (16), 18 queries 26.5 (4) | 21.9 (8), 48 queries 40.3 (2) | 33.9 (3), 64 queries 40.8 (2) | 42.5 (2).  (Clusters of 8 were the
// fastest form of one size in 110, by 1 %.)
void attn4_tc_plan(Attn4Args& a) {
  const int chunks = chunks_of(a);
  const int64_t queries = a.seqs.total_q;
  const double heads = a.h / 128.0;
  double best = 1e30;
  auto consider = [&](int cluster, int splits) {
    const int64_t rounds = (queries * splits + clusters_of(cluster) - 1) / clusters_of(cluster);
    const int pieces = cluster * splits, longest = (chunks + pieces - 1) / pieces;
    const double cost = rounds * (longest + kStart + joining(cluster, heads)) +
                        (splits > 1 ? kMerge + kPartial * heads * queries * splits : 0);
    if (cost >= best) return;
    best = cost;
    a.cluster = cluster;
    a.splits = splits;
  };
  for (int c = 1; c <= kMostPieces && c <= chunks && clusters_of(c) > 0; c *= 2) consider(c, 1);
  for (int n = 2; n <= chunks && n * queries * a.h * (a.d_c * 4 + 8) <= (int64_t)kMostPartial; ++n) consider(1, n);
}

size_t attn4_tc_scratch(const Attn4Args& a) {
  return (size_t)ctas_of(a) * ((chunks_of(a) + a.cluster * a.splits - 1) / (a.cluster * a.splits)) * (kPBytes + kRefBytes + kListBytes);
}

int launch_attn4_tc(const Attn4Args& a, cudaStream_t stream) {
  if (built_to_run() != 1) return set_error(DSA_ERR_CUDA, "attn4_tc: the kernel's attributes are not to be had");
  Params p{};
  p.a = a;
  p.chunks = chunks_of(a);
  p.most = (p.chunks + a.cluster * a.splits - 1) / (a.cluster * a.splits);
  const int64_t items = (int64_t)a.seqs.total_q * a.splits;
  if (items > 0x3fffffff) return set_error(DSA_ERR_UNSUPPORTED, "attn4: too many queries");
  p.items = (int)items;
  CUtensorMap qmap;
  int rc = make_tmap_2d(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, kD, (uint64_t)a.seqs.total_q * a.h, kD * 2, 64, kM);
  if (rc != DSA_OK) return rc;
  switch (a.cluster) {
    case 1: rc = launch_pieces<1>(p, qmap, stream); break;
    case 2: return launch_pieces<2>(p, qmap, stream);
    default: return launch_pieces<4>(p, qmap, stream);
  }
  return rc != DSA_OK || a.splits == 1 ? rc : launch_attn4_merge(a, stream);
}

}  // namespace dsa

