// Device pieces of many-row attention that both caches' kernels use.  Not part of the
// public ABI.
#pragma once

#include "attend.hpp"

namespace cga {

constexpr int WROWS = 32;  // query rows of a wave
constexpr int KP = 2 * D + 16;        // LDS pitch of a token's keys, fp16: 16 tokens' 16-byte pieces in all 64 banks
constexpr int VP = 2 * D + 64;        // of its values: 4 tokens' 64-byte pieces in all 64 banks
constexpr int KBYTES = UNIT * KP, VBYTES = UNIT * VP;

typedef float f16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f16_t mfma32(h8_t a, h8_t b, f16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// the sums of a unit's weights, of each of its NB ranges
template <int NB>
__device__ __forceinline__ void sum_weights(const float (&p)[16], float (&ps)[NB]) {
  float h[2];
#pragma unroll
  for (int u = 0; u < 2; u++) {
    const float *x = p + 8 * u;
    h[u] = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
  }
  if constexpr (NB == 2) {
    ps[0] = h[0];
    ps[1] = h[1];
  } else {
    ps[0] = h[0] + h[1];
  }
}

__device__ __forceinline__ float pair_max(float v) { return fmaxf(v, __shfl_xor(v, 32)); }

// a unit's weights as operands (tokens 16 x + ..)
template <bool BF16>
struct UnitOperands {
  h8_t hi[2], lo[2];  // lo: fp32 storage only
};

template <bool BF16>
__device__ __forceinline__ void pack_weights(const float (&p)[16], UnitOperands<BF16> &P) {
#pragma unroll
  for (int x = 0; x < 2; x++) {
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const float a = p[8 * x + 2 * k], b = p[8 * x + 2 * k + 1];
      ph[k] = pack_f16x2(a, b);
      if constexpr (!BF16) {
        const f2_t hh = unpack_f16x2(ph[k]);
        pl[k] = pack_f16x2(a - hh.x, b - hh.y);
      }
    }
    P.hi[x] = as_h8(ph[0], ph[1], ph[2], ph[3]);
    if constexpr (!BF16) P.lo[x] = as_h8(pl[0], pl[1], pl[2], pl[3]);
  }
}

// 4 tokens x 16 channels of fp16 values as an operand half: lane n of 16 names
// 4 channels of token n / 4 and receives the 4 tokens of channel n
// (transposing LDS read)
typedef short s4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ s4_t transposed(const unsigned char *p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4_t *)p);
}

}  // namespace cga
