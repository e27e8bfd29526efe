// Rows of the 4-bit latent cache: written (quantised) from new tokens' latent and rope columns, and read back.
//
//   scale = UE5M3(max|x| / 6),  code = E2M1(x / scale)   over 16 columns, both to nearest, ties to even
//
// Both are decided by the exact quotients: the divisions are IEEE's in fp32, and a quotient whose exact value is not a
// tie of the target's does not round to one (ties of E2M1 and UE5M3 have at most five significant bits, and
// x / scale next to a tie differs from it by more than half a unit of fp32).  A reciprocal's product would miss ties, which bf16
// inputs meet often.
//
// Bound by HBM where there is work enough: a thread takes 16 latent columns (32 or 64 bytes in, 8 and 1 out) or 8 rope
// columns, and a row's threads are neighbours.  Below some thousand rows it is the launch.  8,192 rows of 512 + 64 bf16
// columns: written in 10.0 us and read back in 8.4 from HBM (1.3 and 1.5 TB/s), 6.1 and 4.6 where they are in L2: latencies in a chain (a row's
// place by its sequence and page, its data) with scattered 8- and 16-byte pieces behind them.
#include "kv4.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;

// N consecutive elements in fp32; VEC: 16-byte loads (the address is a multiple of 16).
template <typename T, int N, bool VEC>
__device__ __forceinline__ void load_f32(const T* p, float (&f)[N]) {
  if constexpr (VEC && sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[8 * i + 2 * j] = __uint_as_float(u[j] << 16);
        f[8 * i + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      }
    }
  } else if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 v = reinterpret_cast<const float4*>(p)[i];
      f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f32(p[i]);
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// 16 columns: their codes and scale byte.
__device__ __forceinline__ uint2 quantise16(const float (&x)[16], uint32_t& scale_byte) {
  float amax = 0.f;
  bool odd = false;  // an infinity or a NaN: the group is NaN
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    amax = fmaxf(amax, fabsf(x[i]));
    odd |= !(fabsf(x[i]) <= 3.402823466e38f);
  }
  if (odd) {
    scale_byte = 0xffu;
    return make_uint2(0u, 0u);
  }
  // four significant bits, to nearest even; steps of 2^-17 below 2^-14
  const float raw = fminf(__fdiv_rn(amax, 6.f), 61440.f);
  uint32_t b;
  if (raw < 0x1p-14f) {
    b = (uint32_t)__float2int_rn(raw * 0x1p17f);  // 8 is the smallest normal one's byte
  } else {
    const uint32_t u = __float_as_uint(raw);
    b = ((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - (112u << 3);
  }
  scale_byte = b;
  if (b == 0u) return make_uint2(0u, 0u);
  const float s = kv4_scale(b);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {  // pairs: column 2k at bit 4k, column 2k + 1 at bit 16 + 4k
    uint16_t two;
    const float lo = __fdiv_rn(x[2 * i], s), hi = __fdiv_rn(x[2 * i + 1], s);
    asm("{\n\t.reg .b8 e;\n\tcvt.rn.satfinite.e2m1x2.f32 e, %1, %2;\n\tcvt.u16.u8 %0, e;\n\t}" : "=h"(two) : "f"(hi), "f"(lo));
    const uint32_t v = two;
    w[i >> 2] |= (v & 15u) << (4 * (i & 3)) | (v >> 4 & 15u) << (16 + 4 * (i & 3));
  }
  return make_uint2(w[0], w[1]);
}

// Units of a row: its 16-column groups, its groups of 8 rope columns, the zeros behind the scales.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) write_kv4_kernel(const __grid_constant__ Kv4Rows a, int units) {
  griddep_wait();
  const int groups = a.d_c / 16, ropes = a.d_rope / 8, rb = kv4_row_bytes(a.d_c, a.d_rope);
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t t = i / units;
  const int u = (int)(i - t * units);
  if (t >= a.seqs.total_q) return;
  RowInfo r;
  if (!kv4_query_row(a.seqs, a.max_q_len, (int)t, r, a.status)) return;
  const int row = cache_row(a.seqs, r.b, r.k0, r.pos);
  if (row < 0) {
    if (u == 0) atomicOr(a.status, DSA_FLAG_BAD_SEQS);
    return;
  }
  uint8_t* dst = a.kv4 + (int64_t)row * rb;
  const int scale_at = kv4_scale_at(a.d_c, a.d_rope);
  if (u < groups) {
    float x[16];
    load_f32<T, 16, VEC>(static_cast<const T*>(a.latent) + t * a.ld_latent + u * 16, x);
    uint32_t b;
    const uint2 w = quantise16(x, b);
    *reinterpret_cast<uint2*>(dst + u * 8) = w;
    dst[scale_at + u] = (uint8_t)b;
  } else if (u < groups + ropes) {
    const int c = (u - groups) * 8;
    float x[8];
    load_f32<T, 8, VEC>(static_cast<const T*>(a.k_rope) + t * a.ld_rope + c, x);
    // (rows of an odd number of 16-column groups leave the rope columns 8-byte aligned)
    uint2* o = reinterpret_cast<uint2*>(dst + kv4_rope_at(a.d_c) + 2 * c);
    o[0] = make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]));
    o[1] = make_uint2(bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
  } else {
    for (int j = scale_at + groups; j < rb; ++j) dst[j] = 0;
  }
}

__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {  // (the values are bf16 numbers)
  *reinterpret_cast<uint4*>(p) =
      make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}

// A thread reads 8 columns: 4 bytes of codes or 16 of rope, and writes 16 or 32.  (16 columns a thread would store 32
// bytes apart, half of each sector at a time.)
template <typename T>
__global__ void __launch_bounds__(kThreads) read_kv4_kernel(const __grid_constant__ Kv4Rows a, int units) {
  griddep_wait();
  const int lats = a.d_c / 8, D = a.d_c + a.d_rope, rb = kv4_row_bytes(a.d_c, a.d_rope);
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t x = i / units;  // packed row
  const int u = (int)(i - x * units);
  const Seqs& s = a.seqs;
  if (x >= s.total_k) return;
  int lo = 0, hi = s.B - 1;
  while (lo < hi) {  // last b with cu_k[b] <= x
    const int mid = (lo + hi + 1) >> 1;
    if (s.cu_k[mid] <= x) lo = mid; else hi = mid - 1;
  }
  const int k0 = s.cu_k[lo], k1 = s.cu_k[lo + 1];
  if (!(x >= k0 && x < k1 && k0 >= 0 && k1 <= s.total_k && k1 - k0 <= s.max_k_len)) {
    atomicOr(a.status, DSA_FLAG_BAD_SEQS);
    return;
  }
  const int row = cache_row(s, lo, k0, (int)x - k0);
  if (row < 0) {
    atomicOr(a.status, DSA_FLAG_BAD_INDEX);
    return;
  }
  const uint8_t* src = a.kv4 + (int64_t)row * rb;
  float f[8];
  if (u < lats) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(src + 4 * u);
    kv4_widen8(w, kv4_scale(src[kv4_scale_at(a.d_c, a.d_rope) + u / 2]), f);
  } else {
    const uint2* v = reinterpret_cast<const uint2*>(src + kv4_rope_at(a.d_c) + 16 * (u - lats));
    const uint2 p = v[0], q = v[1];
    const uint32_t w[4] = {p.x, p.y, q.x, q.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
  store8(static_cast<T*>(a.out) + x * D + 8 * u, f);
}

template <typename K>
int launch_units(const char* name, K kern, const Kv4Rows& a, int64_t rows, int units, cudaStream_t stream) {
  const int64_t blocks = (rows * units + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return set_error(DSA_ERR_UNSUPPORTED, "%s: too many rows", name);
  cudaError_t e = cudaSuccess;
  DSA_LAUNCH(name, stream, e = launch_pdl(kern, dim3((unsigned)blocks), dim3(kThreads), 0, stream, a, units));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
  return check_launch(name);
}

}  // namespace

int launch_write_kv4(const Kv4Rows& a, cudaStream_t stream) {
  const int size = a.dtype == DSA_F32 ? 4 : 2, scale_end = kv4_scale_at(a.d_c, a.d_rope) + a.d_c / 16;
  const int units = a.d_c / 16 + a.d_rope / 8 + (scale_end < kv4_row_bytes(a.d_c, a.d_rope) ? 1 : 0);
  auto al = [&](const void* p, int64_t ld) { return ((uintptr_t)p | (uintptr_t)(ld * size)) % 16 == 0; };
  const bool vec = al(a.latent, a.ld_latent) && (a.d_rope == 0 || al(a.k_rope, a.ld_rope));
  auto kern = a.dtype == DSA_F32 ? (vec ? write_kv4_kernel<float, true> : write_kv4_kernel<float, false>)
                                 : (vec ? write_kv4_kernel<__nv_bfloat16, true> : write_kv4_kernel<__nv_bfloat16, false>);
  return launch_units("write_kv4", kern, a, a.seqs.total_q, units, stream);
}

int launch_read_kv4(const Kv4Rows& a, cudaStream_t stream) {
  auto kern = a.dtype == DSA_F32 ? read_kv4_kernel<float> : read_kv4_kernel<__nv_bfloat16>;
  return launch_units("read_kv4", kern, a, a.seqs.total_k, (a.d_c + a.d_rope) / 8, stream);
}

}  // namespace dsa
