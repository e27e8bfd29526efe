// dsa_add_rmsnorm: the residual's addition, the root-mean-square norm and, optionally, its
// output in 8 bits, one pass over each row ("Day0 Inference Adaptation and Performance
// Optimization for New-Architecture LLMs", §4.2: the indexer's preprocessing normalises the K
// side before it is quantised and scored; §5.1: the index side is kept in MXFP8).
//
//   h = x + residual                        (fp32, stored rounded to the input type)
//   y = (h · rsqrt(mean(h²) + eps)) · w     (fp32, from the unrounded h)
//   E4M3:  scale = max|y| / 448 a row, codes = E4M3(y · (1 / scale)): a product an element instead of a division,
//          off by fp32 roundings like y itself
//   MXFP8: 2^e a group of 32, the smallest with max|y| <= 448·2^e, codes = E4M3(y / 2^e)
//
// Bound by memory (8192 x 7168 bf16 with a residual: 470 MB in 68 us, 6.9 TB/s), for few rows by the
// launch: a row is read once and held in registers as 16-byte vectors between the
// statistics and the output.  Short rows take 8, 16 or 32 lanes each (several rows a warp: indexer
// keys are 128 wide); longer rows take a block.  Rows without 16-byte alignment go element by element.  Both
// statistics a row needs (the sum of squares and max |h·w|, from which max |y| follows by the
// factor rsqrt(...)) are reduced together, so a row costs one reduction.
#include <cuda_fp8.h>
#include <float.h>

#include "cache_ops.cuh"

namespace dsa {
namespace {

struct NormParams {
  const void* x;
  const void* res;  // or null
  const void* w;
  void* h;          // or null
  void* y;          // or null
  uint8_t* codes;   // or null
  void* scale;
  int64_t rows, ld_x, ld_res;
  int d, nvec, quant;
  float eps;
  int lanes;        // lanes of a row (rows that share a warp)
};

// V consecutive elements of T as one load or store.
template <typename T, int V>
struct Vec;
template <>
struct Vec<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ void get(const Raw& r, float (&f)[4]) {
    f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
  }
  static __device__ __forceinline__ Raw put(const float (&f)[4]) {
    return make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct Vec<float, 1> {
  using Raw = float;
  static __device__ __forceinline__ void get(const Raw& r, float (&f)[1]) { f[0] = r; }
  static __device__ __forceinline__ Raw put(const float (&f)[1]) { return f[0]; }
};
template <>
struct Vec<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ void get(const Raw& r, float (&f)[8]) {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ Raw put(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Vec<__nv_bfloat16, 1> {
  using Raw = __nv_bfloat16;
  static __device__ __forceinline__ void get(const Raw& r, float (&f)[1]) {
    f[0] = __bfloat162float(r);
  }
  static __device__ __forceinline__ Raw put(const float (&f)[1]) {
    return __float2bfloat16_rn(f[0]);
  }
};

// The E4M3 codes of V values (round to nearest even, saturating; NaN stays NaN).
template <int V>
__device__ __forceinline__ void store_codes(uint8_t* dst, const float (&f)[V]) {
  if constexpr (V == 1) {
    *dst = __nv_cvt_float_to_fp8(f[0], __NV_SATFINITE, __NV_E4M3);
  } else {
    uint32_t u[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i], f[4 * i + 1]),
                                                   __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2], f[4 * i + 3]),
                                                   __NV_SATFINITE, __NV_E4M3);
      u[i] = lo | hi << 16;
    }
    if constexpr (V == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(u[0], u[1]);
    else *reinterpret_cast<uint32_t*>(dst) = u[0];
  }
}

// BLOCK: a block per row; otherwise p.lanes lanes of a warp per row.  C: vectors a thread holds;
// 0: the row does not fit the registers and is read twice.
template <typename T, int V, int C, bool BLOCK>
__global__ void __launch_bounds__(!BLOCK ? 256 : C == 4 ? 512 : 1024) add_rmsnorm_kernel(NormParams p) {
  using Raw = typename Vec<T, V>::Raw;
  griddep_wait();
  const int nthr = BLOCK ? (int)blockDim.x : p.lanes;
  const int me = BLOCK ? (int)threadIdx.x : (int)threadIdx.x & (p.lanes - 1);
  const int64_t row = BLOCK ? (int64_t)blockIdx.x
                            : ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / p.lanes;
  // lanes past the last row repeat it up to the stores (they take part in the shuffles)
  const bool live = row < p.rows;
  const int64_t r = live ? row : p.rows - 1;
  const Raw* xr = reinterpret_cast<const Raw*>(static_cast<const T*>(p.x) + r * p.ld_x);
  const Raw* rr = p.res ? reinterpret_cast<const Raw*>(static_cast<const T*>(p.res) + r * p.ld_res)
                        : nullptr;
  const Raw* wr = static_cast<const Raw*>(p.w);
  const bool e4m3 = p.quant == DSA_FP8_E4M3;

  auto load_h = [&](int v, float (&f)[V]) {
    Vec<T, V>::get(xr[v], f);
    if (rr) {
      float g[V];
      Vec<T, V>::get(rr[v], g);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] += g[i];
    }
  };
  float ss = 0.f, mx = 0.f;
  auto stats = [&](const float (&f)[V], const Raw& rw) {
#pragma unroll
    for (int i = 0; i < V; ++i) ss = fmaf(f[i], f[i], ss);
    if (e4m3) {
      float w[V];
      Vec<T, V>::get(rw, w);
#pragma unroll
      for (int i = 0; i < V; ++i) mx = fmaxf(mx, fabsf(f[i] * w[i]));
    }
  };

  // the weight's vectors are read ahead of the stores, which the compiler would not move loads across
  float hv[C > 0 ? C : 1][V];
  Raw rw[C > 0 ? C : 1];
  if constexpr (C > 0) {
    Raw rx[C], rs[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int v = me + c * nthr;
      if (v < p.nvec) rx[c] = xr[v];
    }
    if (rr) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int v = me + c * nthr;
        if (v < p.nvec) rs[c] = rr[v];
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int v = me + c * nthr;
      if (v < p.nvec) rw[c] = wr[v];
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int v = me + c * nthr;
      if (v < p.nvec) {
        Vec<T, V>::get(rx[c], hv[c]);
        if (rr) {
          float g[V];
          Vec<T, V>::get(rs[c], g);
#pragma unroll
          for (int i = 0; i < V; ++i) hv[c][i] += g[i];
        }
        stats(hv[c], rw[c]);
      }
    }
  } else {
    for (int v = me; v < p.nvec; v += nthr) {
      load_h(v, hv[0]);
      stats(hv[0], wr[v]);
    }
  }

  // the row's sum of squares and max
  const int width = BLOCK ? 32 : p.lanes;
  for (int o = width >> 1; o; o >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  if constexpr (BLOCK) {
    __shared__ float2 red[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) red[warp] = make_float2(ss, mx);
    __syncthreads();
    const float2 o = lane < nw ? red[lane] : make_float2(0.f, 0.f);
    ss = o.x;
    mx = o.y;
#pragma unroll
    for (int k = 16; k; k >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, k);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    }
  }
  const float rstd = rsqrtf(ss / (float)p.d + p.eps);
  float inv = 1.f;
  if (e4m3) {
    // a row whose scale would not be a normal number (an all-zero one) is stored with scale 1
    float scale = mx * rstd / 448.f;
    if (scale < FLT_MIN) scale = 1.f;
    inv = 1.f / scale;
    if (me == 0 && live) static_cast<float*>(p.scale)[row] = scale;
  }

  Raw* ho = p.h ? reinterpret_cast<Raw*>(static_cast<T*>(p.h) + r * p.d) : nullptr;
  Raw* yo = p.y ? reinterpret_cast<Raw*>(static_cast<T*>(p.y) + r * p.d) : nullptr;
  auto finish = [&](int v, const float (&f)[V], const Raw& rw, bool in) {
    float y[V];
    if (in) {
      float w[V];
      Vec<T, V>::get(rw, w);
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = f[i] * rstd * w[i];
      if (live) {
        if (ho) ho[v] = Vec<T, V>::put(f);
        if (yo) yo[v] = Vec<T, V>::put(y);
      }
    }
    if (p.quant == DSA_MXFP8_E4M3) {
      // 32/V neighbouring threads hold a group; rows are whole groups, so all of them are in
      float m = 0.f;
      if (in) {
#pragma unroll
        for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(y[i]));
      }
#pragma unroll
      for (int o = 32 / V / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      // m = f·2^k with 1 <= f < 2, 448 = 1.75·2^8: e = k - 8, one more where f > 1.75
      const uint32_t b = __float_as_uint(m);
      int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
      e = m > 0.f ? max(e, -127) : 0;
      if (in && live) {
        const float up = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] *= up;
        store_codes<V>(p.codes + r * p.d + (int64_t)v * V, y);
        if (v % (32 / V) == 0)
          static_cast<uint8_t*>(p.scale)[r * (p.d >> 5) + v / (32 / V)] = (uint8_t)(e + 127);
      }
    } else if (e4m3 && in && live) {
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] *= inv;
      store_codes<V>(p.codes + r * p.d + (int64_t)v * V, y);
    }
  };
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int v = me + c * nthr;
      finish(v, hv[c], rw[c], v < p.nvec);
    }
  } else {
    for (int v0 = 0; v0 < p.nvec; v0 += nthr) {  // whole warps take part in the group shuffles
      const int v = v0 + me;
      if (v < p.nvec) {
        load_h(v, hv[0]);
        rw[0] = wr[v];
      }
      finish(v, hv[0], rw[0], v < p.nvec);
    }
  }
}

template <typename T, int V>
cudaError_t launch(NormParams p, cudaStream_t s) {
  p.nvec = p.d / V;
  constexpr int kMinLanes = V == 1 ? 32 : 8;  // a group of 32 stays inside a row's lanes
  const bool few = p.rows <= 4 * num_sms();
  // Lanes of a warp for rows of up to 32 vectors, and of up to 128 where there are many (64 rows x 512 bf16: a block
  // 1.6 us, a warp 2.0; 2,000 rows: 2.8 and 2.5; 16384 rows x 101 fp32: 14.7 and 8.8); as few lanes as there are
  // vectors (65536 rows x 128 bf16 to MXFP8: 16 lanes 9.7 us, 32 lanes 18.1, a block a row 34.8).
  if (p.nvec <= 32 || (p.nvec <= 128 && !few)) {
    int lanes = kMinLanes;
    while (lanes < 32 && lanes < p.nvec) lanes *= 2;
    p.lanes = lanes;
    const int rows = 256 / lanes;
    const unsigned grid = (unsigned)((p.rows + rows - 1) / rows);
    if (p.nvec <= lanes) return launch_pdl(add_rmsnorm_kernel<T, V, 1, false>, dim3(grid), dim3(256), 0, s, p);
    return launch_pdl(add_rmsnorm_kernel<T, V, 4, false>, dim3(grid), dim3(256), 0, s, p);
  }
  // A block a row.  Few rows: as many threads as there are vectors (64 rows x 1024 bf16: 1.6 us, 4 vectors a thread 2.2);
  // many: 4 vectors a thread (512 threads at most, 128 registers each; 8192 rows x 7168: 68 us, 1 vector 89).  Single elements
  // 8 a thread up to 4096, and up to 8192 where there are few rows (4096 rows x 3001 fp32: 46 us, read twice 73; x 5001: 93
  // and 92); longer rows are read twice, the second time from L2.
  const int C = p.nvec <= 1024 && few ? 1
                : p.nvec <= 2048      ? 4
                : V == 1 && p.nvec <= (few ? 8192 : 4096) ? 8 : 0;
  const int thr = C ? ((p.nvec + C - 1) / C + 31) / 32 * 32 : 1024;
  const dim3 grid((unsigned)p.rows);
  if constexpr (V == 1)
    if (C == 8) return launch_pdl(add_rmsnorm_kernel<T, V, 8, true>, grid, dim3(thr), 0, s, p);
  switch (C) {
    case 1: return launch_pdl(add_rmsnorm_kernel<T, V, 1, true>, grid, dim3(thr), 0, s, p);
    case 4: return launch_pdl(add_rmsnorm_kernel<T, V, 4, true>, grid, dim3(thr), 0, s, p);
    default: return launch_pdl(add_rmsnorm_kernel<T, V, 0, true>, grid, dim3(thr), 0, s, p);
  }
}

bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  if (!a || !b) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

}  // namespace
}  // namespace dsa

extern "C" int dsa_add_rmsnorm(int64_t rows, int32_t d, int32_t dtype, int32_t quant, float eps,
                               const void* x, int64_t ld_x, const void* residual, int64_t ld_res,
                               const void* weight, void* h_out, void* y, uint8_t* codes,
                               void* scale, void* stream) {
  using namespace dsa;
  if (rows < 0 || d < 1) return set_error(DSA_ERR_INVALID_ARG, "rows = %lld, d = %d", (long long)rows, d);
  if (dtype != DSA_F32 && dtype != DSA_BF16)
    return set_error(DSA_ERR_UNSUPPORTED, "dtype = %d (F32 or BF16)", dtype);
  if (quant != 0 && quant != DSA_FP8_E4M3 && quant != DSA_MXFP8_E4M3)
    return set_error(DSA_ERR_INVALID_ARG, "quant = %d (0, FP8_E4M3 or MXFP8_E4M3)", quant);
  if (quant == DSA_MXFP8_E4M3 && d % 32)
    return set_error(DSA_ERR_UNSUPPORTED, "MXFP8 needs d a multiple of 32 (d = %d)", d);
  if (!(eps >= 0.f) || eps > FLT_MAX)
    return set_error(DSA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (rows > 0x7fffffff || d > (1 << 24))
    return set_error(DSA_ERR_UNSUPPORTED, "rows = %lld, d = %d too large", (long long)rows, d);
  if (rows == 0) return DSA_OK;  // nothing to do; the pointers may be NULL
  if (!x || !weight) return set_error(DSA_ERR_INVALID_ARG, "x or weight is NULL");
  if ((residual != nullptr) != (h_out != nullptr))
    return set_error(DSA_ERR_INVALID_ARG, "residual and h_out go together");
  if (quant ? (!codes || !scale) : !y)
    return set_error(DSA_ERR_INVALID_ARG, quant ? "codes/scale is NULL" : "y is NULL");
  if (!quant) { codes = nullptr; scale = nullptr; }
  if (ld_x < d || (residual && ld_res < d))
    return set_error(DSA_ERR_INVALID_ARG, "ld_x = %lld, ld_res = %lld below d = %d",
                     (long long)ld_x, (long long)ld_res, d);
  const int es = dtype == DSA_BF16 ? 2 : 4;
  if (ld_x > (int64_t(1) << 40) / rows || (residual && ld_res > (int64_t(1) << 40) / rows))
    return set_error(DSA_ERR_UNSUPPORTED, "row stride too large");
  if (!al(x, es) || !al(residual, es) || !al(weight, es) || !al(h_out, es) || !al(y, es) ||
      (quant == DSA_FP8_E4M3 && !al(scale, 4)))
    return set_error(DSA_ERR_INVALID_ARG, "a pointer is not aligned to its element");
  // an output may be an input (row by row, a thread reads an element before it writes it);
  // any other overlap would let one row's store reach another row's load
  const int64_t nx = ((rows - 1) * ld_x + d) * es, nr = ((rows - 1) * ld_res + d) * es;
  const int64_t no = rows * (int64_t)d * es;
  const int64_t nc = codes ? rows * (int64_t)d : 0;
  const int64_t ns = quant == DSA_FP8_E4M3 ? rows * 4 : quant ? rows * (int64_t)(d / 32) : 0;
  const bool bad_h = (overlap(h_out, no, x, nx) && !(h_out == x && ld_x == d)) ||
                     (overlap(h_out, no, residual, nr) && !(h_out == residual && ld_res == d));
  const bool bad_y = (overlap(y, no, x, nx) && !(y == x && ld_x == d)) ||
                     (overlap(y, no, residual, nr) && !(y == residual && ld_res == d)) ||
                     overlap(y, no, h_out, no);
  const void* q[2] = {codes, scale};
  const int64_t nq[2] = {nc, ns};
  bool bad_q = overlap(codes, nc, scale, ns);
  for (int i = 0; i < 2; ++i)
    bad_q |= overlap(q[i], nq[i], x, nx) || overlap(q[i], nq[i], residual, nr) ||
             overlap(q[i], nq[i], h_out, no) || overlap(q[i], nq[i], y, no) ||
             overlap(q[i], nq[i], weight, (int64_t)d * es);
  if (bad_h || bad_y || bad_q || overlap(h_out, no, weight, (int64_t)d * es) ||
      overlap(y, no, weight, (int64_t)d * es))
    return set_error(DSA_ERR_INVALID_ARG, "an output overlaps an input or another output");

  NormParams p{};
  p.x = x; p.res = residual; p.w = weight; p.h = h_out; p.y = y; p.codes = codes; p.scale = scale;
  p.rows = rows; p.ld_x = ld_x; p.ld_res = residual ? ld_res : 0;
  p.d = d; p.quant = quant; p.eps = eps;
  // 16-byte vectors where every row starts on one (8 or 4 bytes of codes), single elements otherwise
  const int V = 16 / es;
  const bool vec = d % V == 0 && ld_x % V == 0 && p.ld_res % V == 0 && al(x, 16) &&
                   al(residual, 16) && al(weight, 16) && al(h_out, 16) && al(y, 16) && al(codes, V);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  DSA_LAUNCH("add_rmsnorm", s,
             e = dtype == DSA_BF16 ? (vec ? launch<__nv_bfloat16, 8>(p, s) : launch<__nv_bfloat16, 1>(p, s))
                                   : (vec ? launch<float, 4>(p, s) : launch<float, 1>(p, s)));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "add_rmsnorm: %s", cudaGetErrorString(e));
  return DSA_OK;
}
