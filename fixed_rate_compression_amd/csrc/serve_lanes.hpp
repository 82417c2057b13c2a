// Values moved between the lanes of a wave, as appending to and reading from the serving caches
// need them.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cgs {

__device__ __forceinline__ void swap32(float &a, float &b) {  // a's upper lanes and b's lower ones
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap16(float &a, float &b) {  // the same within each half
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}

// register e of quarter q of the wave <-> register q of quarter e
__device__ __forceinline__ void transpose(float &a, float &b, float &c, float &d) {
  swap32(a, c);
  swap32(b, d);
  swap16(a, b);
  swap16(c, d);
}

// Register 4 r + e of quarter q holds channel 8 q + 4 r + e of 32; transposed four by four, the one of channel
// 16 g + 4 s + quarter, what the matrix cores multiply in step s of group g, is this
constexpr int turned(int g, int s) { return 4 * (s & 1) + 2 * g + (s >> 1); }

}  // namespace cgs
