// Device pieces of attention over the 4-bit cache.  Not part of the public ABI.
#pragma once

#include "attend.hpp"

namespace cga {

constexpr int HALF_D = D / 2;  // bytes of a row of codes
constexpr uint32_t INF = 0x7f800000u;

// the largest bit pattern over a wave, of magnitudes
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, false));
  const auto x = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(x[0], x[1]);
  const auto y = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(y[0], y[1]);
}
__device__ __forceinline__ uint32_t range_bits(float2 m) {  // of the larger end of a range; a NaN is the largest
  const uint32_t a = __float_as_uint(m.x) & 0x7fffffffu, b = __float_as_uint(__builtin_fmaf(15.0f, m.y, m.x)) & 0x7fffffffu;
  return max(a, b);
}
// smallest E with |x| < 2^E, of the largest magnitude's bits
__device__ __forceinline__ int exponent_of(uint32_t bits) { return (int)(bits >> 23) - 126; }

// How a row's sums leave its wave.  Sums of weights (the largest 1) times values of 2^64 and more are kept 2^-32 of
// themselves beside a maximum 32 higher, and so is the sum of the weights: over 2^31 tokens at most they then stay
// below the largest value, and 2^up, which may be 2^128, is not formed alone.
struct FarSums {
  bool is;
  float up, less, shift;  // log2 of the sums' scale, what is taken off it (18 with the weights' and values' own), and the maximum's
  __device__ __forceinline__ FarSums(float m, float mo) {
    up = m > -INFINITY ? mo - m : 0.0f;
    is = up > 64.0f;
    shift = is ? 32.0f : 0.0f;
    less = is ? 50.0f : 0.0f;
  }
};

}  // namespace cga
