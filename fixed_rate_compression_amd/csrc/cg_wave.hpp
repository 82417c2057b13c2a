// Sums over a wave without LDS.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cgw {

// sum over the lanes up to this one
template <int N>
__device__ __forceinline__ int shr16(int v) {  // from the lane N before it in its 16, else 0
  return __builtin_amdgcn_update_dpp(0, v, 0x110 + N, 0xf, 0xf, true);
}
__device__ __forceinline__ int wave_scan(int v) {
  v += shr16<1>(v);
  v += shr16<2>(v);
  v += shr16<4>(v);
  v += shr16<8>(v);
  const int lane = threadIdx.x & 63;
  const int s0 = __builtin_amdgcn_readlane(v, 15), s1 = __builtin_amdgcn_readlane(v, 31), s2 = __builtin_amdgcn_readlane(v, 47);
  return v + (lane >= 16 ? s0 : 0) + (lane >= 32 ? s1 : 0) + (lane >= 48 ? s2 : 0);
}

}  // namespace cgw
