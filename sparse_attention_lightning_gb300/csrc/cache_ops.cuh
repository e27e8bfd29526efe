// What the operators around the caches share: constants, tensor maps of column tiles, shared-memory limits.
#pragma once

#include <atomic>

#include "dsa_internal.cuh"

namespace dsa {

constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxWidth = 1024 + 256;  // of a latent row (d_c + d_rope)

// Kernels launched with launch_pdl read what the kernels before them wrote by ordinary loads, behind
// griddep_wait(): the read-only path (__ldg) is for data that nobody changes while the grid runs, and its loads may
// be moved ahead of the wait.  Those that begin an operator wait at their very start (the launch itself
// then passes beside the kernel before: a call of 20 to 140 us is 2 to 3 us shorter in a row of calls), and let only
// their own operator's next kernel start early, as a caller's next one may read its inputs ahead of its wait.

// 2^x by the special-function unit (relative error about 2^-22; results below the normal numbers are 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// key_row by ordinary loads.
__device__ __forceinline__ int cache_row(const Seqs& s, int b, int k0, int pos) {
  if (!s.paged()) return k0 + pos;
  const int sh = __ffs(s.page_size) - 1;
  const int pg = s.block_table[(int64_t)b * s.max_pages + (pos >> sh)];
  return (unsigned)pg < (unsigned)s.num_pages ? (pg << sh) | (pos & (s.page_size - 1)) : -1;
}

// 16-bit rows as [tiles][rows][64 columns] (rows of tiles · 64 elements): a box is box_tiles tiles of
// box_rows rows, each tile as make_tmap_2d's box of 64 columns would store it.
int make_tmap_tiles(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t tiles,
                    uint64_t rows, uint64_t row_bytes, uint32_t box_tiles, uint32_t box_rows);

// Allow `kern` BYTES of dynamic shared memory, the most that any of its launches asks for: launches of other host
// threads, with other sizes, then never find a smaller limit.  Asked of the runtime once for a kernel (its slot:
// one static array a kernel) and device.
template <int BYTES, typename K>
inline int allow_smem(K kern, std::atomic<bool> (&slot)[64], const char* what) {
  static_assert(BYTES <= 232448, "shared memory");
  int dev = 0;
  cudaGetDevice(&dev);
  const bool keep = dev >= 0 && dev < 64;
  if (keep && slot[dev].load(std::memory_order_acquire)) return DSA_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES) != cudaSuccess)
    return check_launch(what);
  if (keep) slot[dev].store(true, std::memory_order_release);
  return DSA_OK;
}

}  // namespace dsa
