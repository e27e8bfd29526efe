// Rotary positions with several axes: what the kernel and its host code share.
#pragma once

#include "cache_ops.cuh"

namespace dsa {

constexpr int kMaxPairs = 128;  // d <= 256

struct RotaryArgs {
  int64_t tokens;
  int heads, d, dtype;
  bool interleaved, inverse;
  const int32_t* pos;          // [axes, ld_pos]
  int64_t ld_pos;
  const void* x;               // element (t, h, c) at t · xt + h · xh + c
  int64_t xt, xh;
  void* out;
  int64_t ot, oh;
  uint64_t turn[kMaxPairs];    // of a pair: 2^64 times the turns of one position
  uint8_t axis[kMaxPairs];
};
int launch_rotary(const RotaryArgs& a, cudaStream_t stream);

}  // namespace dsa
