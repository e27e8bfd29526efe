// Rotary positions with several axes, on the rope columns of queries or keys.
//
//   pair i of a row, (a, b):  φ = positions[axis_i, t] · f_i,  (a, b) -> (a cos φ − b sin φ, a sin φ + b cos φ)
//
// The angle.  φ / 2π is wanted modulo one turn, for positions of up to 31 bits: in fp32 a position of a million has
// an angle off by 0.03.  So a pair's turns a position are a 64-bit fixed-point fraction, and the product with the position,
// in 64-bit integers, wraps modulo one turn by itself: off by 2^-65 turns a position.  Its upper 32 bits, signed, are the angle in
// units of 2^-31 half turns, for sincospi.
//
// Bound by HBM for many rows: 2 · 16 bytes of every 8 bf16 columns.  A thread takes 8 columns (4 pairs side by side,
// or, where a pair's two columns are half a row apart, 16: 8 of each half) of up to 8 heads of a token, so that
// the sines (30 to 40 instructions a pair) are shared by the heads and the heads' loads are in flight together.
// 8,192 tokens of 128 heads, 64 of 576 columns in place: 46.5 us, 5.8 TB/s (0.85 of a copy's rate: 128 bytes of every 1,152).
// One token of 128 heads: 2.1 us.
#include "rotary.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;

// Eight columns as they are in memory: a 16-byte vector of bf16, two of fp32.
template <typename T>
struct Eight {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
  }
  __device__ __forceinline__ void widen(float (&f)[8]) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t u[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(u[j] << 16);
        f[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(v[i].x); f[4 * i + 1] = __uint_as_float(v[i].y);
        f[4 * i + 2] = __uint_as_float(v[i].z); f[4 * i + 3] = __uint_as_float(v[i].w);
      }
    }
  }
  __device__ __forceinline__ void narrow(const float (&f)[8]) {
    if constexpr (sizeof(T) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
      v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                          __float_as_uint(f[4 * i + 3]));
    }
  }
};

__device__ __forceinline__ void sine(const RotaryArgs& a, int pair, int64_t t, float& s, float& c) {
  const int64_t p = a.pos[a.axis[pair] * a.ld_pos + t];
  const int32_t hi = (int32_t)(((uint64_t)p * a.turn[pair] + 0x80000000u) >> 32);  // nearest
  sincospif((float)hi * 0x1p-31f, &s, &c);
  if (a.inverse) s = -s;
}

// NH heads a thread: heads h, h + step, ...; `tokens` tokens a block, or `parts` blocks a token.
struct Cut {
  int step, slots, tokens, parts;
};
template <typename T, bool INTERLEAVED, int NH>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a, const Cut k) {
  griddep_wait();
  const uint32_t group = blockIdx.x / (uint32_t)k.parts, part = blockIdx.x - group * k.parts;
  const uint32_t per = (uint32_t)(k.step * k.slots);  // threads a token
  const uint32_t i = k.tokens > 1 ? threadIdx.x : part * kThreads + threadIdx.x;
  const uint32_t tt = k.tokens > 1 ? i / per : 0u, rest = i - tt * per;
  const int h0 = (int)(rest / (uint32_t)k.slots), s = (int)(rest - h0 * k.slots);
  const int64_t t = (int64_t)group * k.tokens + tt;
  if (rest >= per || (int)tt >= k.tokens || t >= a.tokens) return;
  constexpr int NP = INTERLEAVED ? 4 : 8, NV = INTERLEAVED ? 1 : 2;
  const int c0 = s * 8, p0 = s * NP, half = a.d / 2;
  const T* x = static_cast<const T*>(a.x) + t * a.xt + c0;
  T* o = static_cast<T*>(a.out) + t * a.ot + c0;
  Eight<T> e[NH][NV];
#pragma unroll
  for (int j = 0; j < NH; ++j) {
    const int h = h0 + j * k.step;
    if (h >= a.heads) break;
#pragma unroll
    for (int v = 0; v < NV; ++v) e[j][v].load(x + h * a.xh + v * half);
  }
  float sn[NP], cs[NP];
#pragma unroll
  for (int q = 0; q < NP; ++q) sine(a, p0 + q, t, sn[q], cs[q]);
#pragma unroll
  for (int j = 0; j < NH; ++j) {
    const int h = h0 + j * k.step;
    if (h >= a.heads) break;
    float f[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) e[j][v].widen(f[v]);
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      float& u = INTERLEAVED ? f[0][2 * q] : f[0][q];
      float& w = INTERLEAVED ? f[0][2 * q + 1] : f[NV - 1][q];
      const float y = u * cs[q] - w * sn[q], z = u * sn[q] + w * cs[q];
      u = y;
      w = z;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      e[j][v].narrow(f[v]);
      e[j][v].store(o + h * a.oh + v * half);
    }
  }
}

// Any width and alignment: a thread a pair, with 2- or 4-byte accesses and a sine of its own for every head (8,192 tokens of 128 heads, rows of 64
// columns 2 bytes off: 462 us, ten times the kernel above).
template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_pairs_kernel(const __grid_constant__ RotaryArgs a) {
  griddep_wait();
  const int pairs = a.d / 2;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t rest = i / pairs;
  const int k = (int)(i - rest * pairs);
  const int64_t t = rest / a.heads;
  const int h = (int)(rest - t * a.heads);
  if (t >= a.tokens) return;
  const int cu = a.interleaved ? 2 * k : k, cv = a.interleaved ? 2 * k + 1 : k + pairs;
  const T* x = static_cast<const T*>(a.x) + t * a.xt + h * a.xh;
  T* o = static_cast<T*>(a.out) + t * a.ot + h * a.oh;
  float s, c;
  sine(a, k, t, s, c);
  const float u = to_f32(x[cu]), v = to_f32(x[cv]);
  store_f32(o + cu, u * c - v * s);
  store_f32(o + cv, u * s + v * c);
}

template <typename K, typename... A>
int launch_blocks(K kern, int64_t blocks, cudaStream_t stream, const A&... args) {
  if (blocks > 0x7fffffff) return set_error(DSA_ERR_UNSUPPORTED, "rotary: too many rows");
  cudaError_t e = cudaSuccess;
  DSA_LAUNCH("rotary", stream, e = launch_pdl(kern, dim3((unsigned)blocks), dim3(kThreads), 0, stream, args...));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "rotary: %s", cudaGetErrorString(e));
  return check_launch("rotary");
}

template <typename T, bool INTERLEAVED, int NH>
int launch_heads(const RotaryArgs& a, cudaStream_t stream) {
  Cut k;
  k.slots = a.d / (INTERLEAVED ? 8 : 16);
  k.step = (a.heads + NH - 1) / NH;
  const int64_t per = (int64_t)k.step * k.slots;
  if (per > 0x7fffffff / 2) return set_error(DSA_ERR_UNSUPPORTED, "rotary: too many heads");
  k.tokens = per < kThreads ? (int)(kThreads / per) : 1;
  k.parts = (int)((per + kThreads - 1) / kThreads);
  return launch_blocks(rotary_kernel<T, INTERLEAVED, NH>, (a.tokens + k.tokens - 1) / k.tokens * k.parts, stream, a, k);
}

template <typename T, bool INTERLEAVED>
int launch_wide(const RotaryArgs& a, cudaStream_t stream) {
  // Heads a thread: 8 where that leaves every SM 1024 threads, fewer otherwise.
  const int64_t rows = a.tokens * a.heads * (a.d / (INTERLEAVED ? 8 : 16)), fill = 1024 * (int64_t)num_sms();
  if (a.heads >= 8 && rows / 8 >= fill) return launch_heads<T, INTERLEAVED, 8>(a, stream);
  if (a.heads >= 2 && rows / 2 >= fill) return launch_heads<T, INTERLEAVED, 2>(a, stream);
  return launch_heads<T, INTERLEAVED, 1>(a, stream);
}

}  // namespace

int launch_rotary(const RotaryArgs& a, cudaStream_t stream) {
  const int64_t size = a.dtype == DSA_F32 ? 4 : 2;
  const uintptr_t at = (uintptr_t)a.x | (uintptr_t)a.out | (uintptr_t)(a.xt * size) | (uintptr_t)(a.xh * size) |
                       (uintptr_t)(a.ot * size) | (uintptr_t)(a.oh * size);
  const bool wide = at % 16 == 0 && a.d % (a.interleaved ? 8 : 16) == 0;
  const int64_t pairs = (a.tokens * a.heads * (a.d / 2) + kThreads - 1) / kThreads;  // blocks of them
  if (a.dtype == DSA_F32) {
    if (!wide) return launch_blocks(rotary_pairs_kernel<float>, pairs, stream, a);
    return a.interleaved ? launch_wide<float, true>(a, stream) : launch_wide<float, false>(a, stream);
  }
  if (!wide) return launch_blocks(rotary_pairs_kernel<__nv_bfloat16>, pairs, stream, a);
  return a.interleaved ? launch_wide<__nv_bfloat16, true>(a, stream) : launch_wide<__nv_bfloat16, false>(a, stream);
}

}  // namespace dsa
