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
#include "rotary.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(u[j] << 16);
      f[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

__device__ __forceinline__ void sine(const RotaryArgs& a, int pair, int64_t t, float& s, float& c) {
  const int64_t p = a.pos[a.axis[pair] * a.ld_pos + t];
  const int32_t hi = (int32_t)(((uint64_t)p * a.turn[pair] + 0x80000000u) >> 32);  // nearest
  sincospif((float)hi * 0x1p-31f, &s, &c);
  if (a.inverse) s = -s;
}

// NH heads a thread: heads h, h + step, ...
template <typename T, bool INTERLEAVED, int NH>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a, int step) {
  griddep_wait();
  const int slots = a.d / (INTERLEAVED ? 8 : 16);
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t rest = i / slots;
  const int s = (int)(i - rest * slots);
  const int64_t t = rest / step;
  const int h0 = (int)(rest - t * step);
  if (t >= a.tokens) return;
  constexpr int NP = INTERLEAVED ? 4 : 8;
  const int c0 = s * 8, p0 = s * NP, half = a.d / 2;
  const T* x = static_cast<const T*>(a.x) + t * a.xt + c0;
  T* o = static_cast<T*>(a.out) + t * a.ot + c0;
  float f[NH][INTERLEAVED ? 1 : 2][8];
#pragma unroll
  for (int j = 0; j < NH; ++j) {
    const int h = h0 + j * step;
    if (h >= a.heads) break;
    load8(x + h * a.xh, f[j][0]);
    if constexpr (!INTERLEAVED) load8(x + h * a.xh + half, f[j][1]);
  }
  float sn[NP], cs[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) sine(a, p0 + k, t, sn[k], cs[k]);
#pragma unroll
  for (int j = 0; j < NH; ++j) {
    const int h = h0 + j * step;
    if (h >= a.heads) break;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      float& u = INTERLEAVED ? f[j][0][2 * k] : f[j][0][k];
      float& v = INTERLEAVED ? f[j][0][2 * k + 1] : f[j][INTERLEAVED ? 0 : 1][k];
      const float p = u * cs[k] - v * sn[k], q = u * sn[k] + v * cs[k];
      u = p;
      v = q;
    }
    store8(o + h * a.oh, f[j][0]);
    if constexpr (!INTERLEAVED) store8(o + h * a.oh + half, f[j][1]);
  }
}

// Any width and alignment: a thread a pair.
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
int launch_blocks(K kern, int64_t threads, cudaStream_t stream, const A&... args) {
  const int64_t blocks = (threads + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return set_error(DSA_ERR_UNSUPPORTED, "rotary: too many rows");
  cudaError_t e = cudaSuccess;
  DSA_LAUNCH("rotary", stream, e = launch_pdl(kern, dim3((unsigned)blocks), dim3(kThreads), 0, stream, args...));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "rotary: %s", cudaGetErrorString(e));
  return check_launch("rotary");
}

template <typename T, bool INTERLEAVED>
int launch_wide(const RotaryArgs& a, cudaStream_t stream) {
  const int64_t slots = a.d / (INTERLEAVED ? 8 : 16);
  // Heads a thread: 8 where that leaves every SM 1024 threads, fewer otherwise.
  const int64_t rows = a.tokens * slots;
  const int64_t fill = 1024 * (int64_t)num_sms();
  if (a.heads >= 8 && rows * a.heads / 8 >= fill) {
    const int step = (a.heads + 7) / 8;
    return launch_blocks(rotary_kernel<T, INTERLEAVED, 8>, rows * step, stream, a, step);
  }
  if (a.heads >= 2 && rows * a.heads / 2 >= fill) {
    const int step = (a.heads + 1) / 2;
    return launch_blocks(rotary_kernel<T, INTERLEAVED, 2>, rows * step, stream, a, step);
  }
  return launch_blocks(rotary_kernel<T, INTERLEAVED, 1>, rows * a.heads, stream, a, a.heads);
}

}  // namespace

int launch_rotary(const RotaryArgs& a, cudaStream_t stream) {
  const int64_t size = a.dtype == DSA_F32 ? 4 : 2;
  const uintptr_t at = (uintptr_t)a.x | (uintptr_t)a.out | (uintptr_t)(a.xt * size) | (uintptr_t)(a.xh * size) |
                       (uintptr_t)(a.ot * size) | (uintptr_t)(a.oh * size);
  const bool wide = at % 16 == 0 && a.d % (a.interleaved ? 8 : 16) == 0;
  if (a.dtype == DSA_F32) {
    if (!wide) return launch_blocks(rotary_pairs_kernel<float>, a.tokens * a.heads * (a.d / 2), stream, a);
    return a.interleaved ? launch_wide<float, true>(a, stream) : launch_wide<float, false>(a, stream);
  }
  if (!wide) return launch_blocks(rotary_pairs_kernel<__nv_bfloat16>, a.tokens * a.heads * (a.d / 2), stream, a);
  return a.interleaved ? launch_wide<__nv_bfloat16, true>(a, stream) : launch_wide<__nv_bfloat16, false>(a, stream);
}

}  // namespace dsa
