// What the operators around the caches share: constants, tensor maps of column tiles, shared-memory limits.
#pragma once

#include "dsa_internal.cuh"

namespace dsa {

constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;

// 16-bit rows as [tiles][rows][64 columns] (rows of tiles · 64 elements): a box is box_tiles tiles of
// box_rows rows, each tile as make_tmap_2d's box of 64 columns would store it.
int make_tmap_tiles(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t tiles,
                    uint64_t rows, uint64_t row_bytes, uint32_t box_tiles, uint32_t box_rows);

// Allow `kern` `bytes` of dynamic shared memory; asked of the runtime once for a kernel (its slot:
// one static array a kernel), device and size.
template <typename K>
inline int allow_smem(K kern, int bytes, int (&slot)[64], const char* what) {
  int dev = 0;
  cudaGetDevice(&dev);
  const bool keep = dev >= 0 && dev < 64;
  if (keep && slot[dev] >= bytes) return DSA_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return check_launch(what);
  if (keep) slot[dev] = bytes;
  return DSA_OK;
}

}  // namespace dsa
