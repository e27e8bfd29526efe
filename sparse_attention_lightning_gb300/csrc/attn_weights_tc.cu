// dsa_accumulate_attn_weights on tcgen05 tensor cores (bf16, 64 <= D <= 576, up to 128 heads).
//
//   w[i] = Σ_h exp(scale · q[t,h,:]·kv[row_i,:] − lse[t,h])
//
// The sum runs over heads, so the selected keys are the MMA's M = 128 (a tensor-memory lane a key) and the
// heads its N: a thread holds one key's logits of all heads and adds their exponentials without any
// exchange.  The query's heads stay in shared memory (D x 128 heads: 144 KB); gathered rows come
// through a ring of four [128 keys x 64 columns] tiles.
//
// Bound by the gather: 1152 B a selected row, and ~2,300 clocks of MMA and ~1,500 of exponentials per 128 keys that
// overlap with it.  Four producer warps copy with cp.async, eight lanes a 128-byte row piece, straight
// into the swizzled operand layout (64 KB in flight an SM); one thread issues the MMAs; four warps
// take the exponentials from two logit buffers in turn.  A CTA takes one query and a share of its
// selected positions, so that few queries still fill the SMs.  Every wait is bounded (DSA_FLAG_TIMEOUT).
#include "attn_weights.cuh"
#include "tc_sm100.cuh"

namespace dsa {
namespace {

using namespace tc;

constexpr int kM = 128;               // keys of a chunk
constexpr int kTile = kM * 128;       // 16 KB
constexpr int kSlots = 4;
constexpr int kProducers = 4;         // warps
constexpr int kThreads = 32 * (kProducers + 1 + 4);
constexpr int kMetaBytes = 1024;      // barriers, lse

struct Params {
  WeightArgs a;
  int splits;   // CTAs of a query
  int chunks;   // of a query
  int n;        // MMA N: heads rounded up to 16
  int ntile;    // column tiles
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive_noinc(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
attn_weights_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap qmap) {
  const WeightArgs& a = p.a;
  const int t = blockIdx.x / p.splits, split = blockIdx.x - t * p.splits;
  const int c0 = (int)((int64_t)p.chunks * split / p.splits);
  const int nch = (int)((int64_t)p.chunks * (split + 1) / p.splits) - c0;
  RowInfo ri;
  if (!query_row_info(a.seqs, t, ri, a.status) || nch == 0) return;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* ring = smem;                                   // [4][128][128 B]
  uint8_t* qs = ring + kSlots * kTile;                    // [ntile][n][128 B]
  uint64_t* bars = reinterpret_cast<uint64_t*>(qs + p.ntile * p.n * 128);
  uint64_t* a_full = bars;          // [4] 128 producer threads (cp.async completion)
  uint64_t* a_empty = bars + 4;     // [4]
  uint64_t* s_full = bars + 8;      // [2]
  uint64_t* s_empty = bars + 10;    // [2] 4 warps
  uint64_t* q_full = bars + 12;
  uint64_t* drain = bars + 13;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 14);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 15);
  float* lse2 = reinterpret_cast<float*>(bars + 16);      // [128] lse in log2 units, +inf: no weight

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) { mbar_init(&a_full[i], 32 * kProducers); mbar_init(&a_empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], 4); }
    mbar_init(q_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (threadIdx.x < 128) {
    float v = INFINITY;
    if ((int)threadIdx.x < a.h) {
      v = a.lse[(int64_t)t * a.h + threadIdx.x];
      v = v == -INFINITY ? INFINITY : v * kLog2e;
    }
    lse2[threadIdx.x] = v;
  }
  if (warp == kProducers) { tmem_alloc(tmem_slot, 256); tmem_relinquish(); }
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int D = a.d;

  if (warp < kProducers) {
    // ---------------- producers: 8 lanes a row piece of 128 bytes, 4 rows a step and warp ----------------
    const int piece = lane & 7, rsub = warp * 4 + (lane >> 3);
    const __nv_bfloat16* kv = static_cast<const __nv_bfloat16*>(a.kv);
    // this thread's 8 cache rows of chunk c (row 0 in place of entries that are skipped: their weight
    // is dropped)
    int row[8];
    auto load_rows = [&](int c) {
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const int i = c * kM + g * 16 + rsub;
        const int v = i < a.top_k ? __ldg(a.idx + (int64_t)t * a.top_k + i) : -1;
        int r = -1;
        if (v >= 0 && v <= ri.pos) r = key_row(a.seqs, ri.b, ri.k0, v);
        row[g] = r < 0 ? 0 : r;
      }
    };
    load_rows(c0);
    int n = 0;
    bool stop = false;
    for (int c = 0; c < nch && !stop; ++c) {
      const char* src[8];
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        if (!dsa_check(row[g] < a.seqs.cache_rows(), a.status)) row[g] = 0;
        src[g] = reinterpret_cast<const char*>(kv + (int64_t)row[g] * D) + piece * 16;
      }
      if (c + 1 < nch) load_rows(c0 + c + 1);
      for (int tile = 0; tile < p.ntile; ++tile, ++n) {
        const int slot = n % kSlots;
        if (!__all_sync(0xffffffffu, mbar_wait(&a_empty[slot], ((n / kSlots) & 1) ^ 1, abort_flag, a.status,
                                               DSA_FLAG_TIMEOUT))) { stop = true; break; }
        const uint32_t dst = smem_u32(ring + slot * kTile) + rsub * 128;
        if (tile * 64 + piece * 8 < D) {  // D is a multiple of 16: a piece is inside or outside
#pragma unroll
          for (int g = 0; g < 8; ++g)
            // rows g·16 + rsub: their place in the 8-row swizzle is rsub's
            cp_async16(dst + g * 2048 + ((piece ^ (rsub & 7)) * 16), src[g] + tile * 128);
        }
        cp_async_arrive_noinc(&a_full[slot]);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // landed before the CTA may exit
  } else if (warp == kProducers) {
    // ---------------- the query's heads, MMA issue ----------------
    if (elect_one()) {
      mbar_arrive_expect_tx(q_full, (uint32_t)(p.ntile * p.n * 128));
      for (int j = 0; j < p.ntile; ++j)
        tma_load_2d(qs + j * p.n * 128, &qmap, q_full, j * 64, t * a.h);
      const uint32_t idesc = idesc_bf16(kM, p.n);
      const uint64_t ad0 = sdesc_sw128(smem_u32(ring), 16, 1024), bd0 = sdesc_sw128(smem_u32(qs), 16, 1024);
      const uint32_t bstep = (uint32_t)(p.n * 128) >> 4;
      bool stop = !mbar_wait(q_full, 0, abort_flag, a.status, DSA_FLAG_TIMEOUT);
      uint32_t slot = 0, phase = 0;
      for (int c = 0; c < nch && !stop; ++c) {
        if (!mbar_wait(&s_empty[c & 1], ((c >> 1) & 1) ^ 1, abort_flag, a.status, DSA_FLAG_TIMEOUT)) break;
        const uint32_t d = tmem + (c & 1) * 128;
        uint64_t bd = bd0;
        for (int tile = 0; tile < p.ntile; ++tile) {
          if (!mbar_wait(&a_full[slot], phase, abort_flag, a.status, DSA_FLAG_TIMEOUT)) { stop = true; break; }
          fence_proxy_async_smem();  // the cp.async writes, seen by the tensor core
          tc_fence_after();
          const uint64_t ad = ad0 + (uint64_t)(slot * (kTile >> 4));
          if (tile * 64 + 64 <= D) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_bf16(d, ad + (uint64_t)(i * 2), bd + (uint64_t)(i * 2), idesc, tile || i ? 1u : 0u);
          } else {
            for (int i = 0; i < (D - tile * 64) / 16; ++i)
              mma_bf16(d, ad + (uint64_t)(i * 2), bd + (uint64_t)(i * 2), idesc, tile || i ? 1u : 0u);
          }
          mma_commit(&a_empty[slot]);
          bd += bstep;
          if (++slot == kSlots) { slot = 0; phase ^= 1; }
        }
        if (!stop) mma_commit(&s_full[c & 1]);
      }
      mma_commit(drain);
      mbar_wait_drain(drain, 0);
      mbar_wait_drain(q_full, 0);
    }
  } else {
    // ---------------- weights: thread = key ----------------
    const int quarter = warp & 3;
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    for (int c = 0; c < nch; ++c) {
      const int i = (c0 + c) * kM + quarter * 32 + lane;
      const int v = i < a.top_k ? __ldg(a.idx + (int64_t)t * a.top_k + i) : -1;
      const bool valid = v >= 0 && v <= ri.pos && key_row(a.seqs, ri.b, ri.k0, v) >= 0;
      if (!valid && v != -1) atomicOr(a.status, DSA_FLAG_BAD_INDEX);
      if (!__all_sync(0xffffffffu, mbar_wait(&s_full[c & 1], (c >> 1) & 1, abort_flag, a.status,
                                             DSA_FLAG_TIMEOUT))) break;
      tc_fence_after();
      float w[4] = {0.f, 0.f, 0.f, 0.f};
      for (int h0 = 0; h0 < a.h; h0 += 32) {
        uint32_t s[32];
        __syncwarp();
        tmem_ld32(lane_base + (c & 1) * 128 + h0, s);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 l4 = *reinterpret_cast<const float4*>(lse2 + h0 + j);
          const float l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // +inf: no such head, or it attended to nothing; whatever its logit is, it adds nothing
            const float x = ex2(fmaf(__uint_as_float(s[j + e]), a.scale_log2, -l[e]));
            w[e] += l[e] == INFINITY ? 0.f : x;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_empty[c & 1]);
      if (valid) add_weight(a, ri.b, v, (w[0] + w[1]) + (w[2] + w[3]));
    }
  }
  tc_fence_before();
  cta_sync();
  if (warp == kProducers) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

}  // namespace

bool attn_weights_tc_eligible(const WeightArgs& a) {
  return a.kv_dtype == DSA_BF16 && a.d >= 64 && a.d <= 576 && a.h <= 128;
}

int launch_attn_weights_tc(const WeightArgs& a, cudaStream_t stream) {
  Params p{};
  p.a = a;
  p.n = (a.h + 15) / 16 * 16;
  p.ntile = (a.d + 63) / 64;
  p.chunks = (a.top_k + kM - 1) / kM;
  // CTAs of a query: fewest waves of its chunks, with about one and a half chunks' time for a CTA's start
  const int sms = num_sms();
  double best = 1e30;
  p.splits = 1;
  for (int s = 1; s <= p.chunks; ++s) {
    const int64_t ctas = (int64_t)a.seqs.total_q * s;
    const double cost = (double)((ctas + sms - 1) / sms) * ((p.chunks + s - 1) / s + 1.5);
    if (cost < best) { best = cost; p.splits = s; }
  }
  const int64_t grid = (int64_t)a.seqs.total_q * p.splits;
  if (grid > 0x7fffffff) return set_error(DSA_ERR_UNSUPPORTED, "attention weights: grid too large");
  CUtensorMap qmap;
  int rc = make_tmap_2d(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, (uint64_t)a.d,
                              (uint64_t)a.seqs.total_q * a.h, (uint64_t)a.d * 2, 64, (uint32_t)p.n);
  if (rc != DSA_OK) return rc;
  const int smem = kSlots * kTile + p.ntile * p.n * 128 + kMetaBytes + 1024;
  static int allowed[64];
  rc = allow_smem(attn_weights_tc_kernel, smem, allowed, "attn_weights_tc: smem attribute");
  if (rc != DSA_OK) return rc;
  DSA_LAUNCH("attn_weights_tc", stream,
             attn_weights_tc_kernel<<<(unsigned)grid, kThreads, smem, stream>>>(p, qmap));
  return check_launch("attn_weights_tc");
}

}  // namespace dsa
