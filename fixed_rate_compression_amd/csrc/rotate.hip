// Norm of each query and key head and the rotation by its row's position, in one pass:
//   x <- w x / sqrt(mean x^2 + eps),   (x_a, x_b) <- (x_a cos - x_b sin, x_b cos + x_a sin)
// with the angle position * freq of the pair, the position that of the pair's axis.
//
// A workgroup takes some heads of one row, 16 lanes and 16 bytes a lane to a head (fp32: 32
// bytes); the row's sines and cosines are formed once for all of them.  An angle is
// a product of far positions, so it is taken in fp64, in turns, and only what is left of
// whole turns goes on in fp32.  The other half of a pair comes from another lane's
// registers, a row rotation where all 128 channels turn.
#include "cg_tile.hpp"
#include "rotate.hpp"

namespace cgr {

using cgk::D;
constexpr int NTH = 256;

template <int N>
__device__ __forceinline__ float ror16(float v) {  // from the lane N further round in its 16
  return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), 0x120 + N, 0xf, 0xf, false));
}

// the axis whose position turns pair i
__device__ __forceinline__ int axis_of(const RotateArgs &a, int i) {
  if (a.axes == 1) return 0;
  if (a.dealt) {
    const int x = i % a.axes;
    return x == 0 || i < a.axes * a.sections[x] ? x : 0;
  }
  int x = 0, end = a.sections[0];
#pragma unroll
  for (int k = 1; k < 4; k++) {
    if (k < a.axes && i >= end) x = k;
    end += k < a.axes ? a.sections[k] : 0;
  }
  return x;
}

template <bool BF16>
__global__ __launch_bounds__(NTH) void k_rotate(const RotateArgs a) {
  __shared__ __align__(16) float2 cs[D / 2];
  constexpr int ESZ = BF16 ? 2 : 4;
  const uint32_t row = blockIdx.x / (uint32_t)a.chunks;
  const int chunk = (int)(blockIdx.x - row * a.chunks);
  const int b = (int)(row / (uint32_t)a.n), i = (int)(row - (uint32_t)b * a.n);
  const int64_t len = a.lengths ? min(max((int64_t)a.lengths[b], (int64_t)0), a.tokens) : a.tokens;
  const int64_t pos = (a.starts ? (int64_t)a.starts[b] : len - a.n) + i;
  if (pos < 0 || pos >= len) return;
  const int half = a.dim >> 1;
  if ((int)threadIdx.x < half) {
    const int k = threadIdx.x;
    const int64_t at = a.positions ? (int64_t)a.positions[((int64_t)axis_of(a, k) * a.batch + b) * a.n + i] : pos;
    double turn = (double)at * ((double)a.freq[k] * 0.15915494309189533576888);
    turn -= rint(turn);
    float s, c;
    sincospif(2.0f * (float)turn, &s, &c);
    cs[k] = make_float2(c * a.magnitude, s * a.magnitude);
  }
  __syncthreads();
  const int l = threadIdx.x & 15, total = a.r[0].heads + a.r[1].heads;
  const int h1 = min((chunk + 1) * a.each, total);
  for (int hh = chunk * a.each + (int)(threadIdx.x >> 4); hh < h1; hh += NTH / 16) {  // 16 lanes go together
    const bool key = hh >= a.r[0].heads;
    const Rows &r = a.r[key];
    const int h = key ? hh - a.r[0].heads : hh;
    const char *in = (const char *)r.in + ((int64_t)b * r.ibs + (int64_t)i * r.irs + (int64_t)h * D + 8 * l) * ESZ;
    float x[8];
    if (BF16) {
      const uint4 w = *(const uint4 *)in;
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; k++) {
        x[2 * k] = cgk::bf16lo(u[k]);
        x[2 * k + 1] = cgk::bf16hi(u[k]);
      }
    } else {
      const float4 u = ((const float4 *)in)[0], v = ((const float4 *)in)[1];
      x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
      x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    }
    if (r.weight) {
      float ss = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; k++) ss = __builtin_fmaf(x[k], x[k], ss);
      ss += ror16<8>(ss);
      ss += ror16<4>(ss);
      ss += ror16<2>(ss);
      ss += ror16<1>(ss);
      const float f = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
      const float4 u = ((const float4 *)(r.weight + 8 * l))[0], v = ((const float4 *)(r.weight + 8 * l))[1];
      const float w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 8; k++) x[k] = x[k] * f * w[k];
    }
    float y[8];
    if (a.interleaved) {
      if (8 * l < a.dim) {
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const float2 t = cs[4 * l + k];
          y[2 * k] = x[2 * k] * t.x - x[2 * k + 1] * t.y;
          y[2 * k + 1] = x[2 * k + 1] * t.x + x[2 * k] * t.y;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; k++) y[k] = x[k];
      }
    } else {
      const int lanes = a.dim >> 4;  // of half the turned channels
      const bool second = l >= lanes, turns = l < 2 * lanes;
      const int other = (threadIdx.x & 48) + (second ? l - lanes : l + lanes);
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const float o = a.dim == D ? ror16<8>(x[k]) : __shfl(x[k], turns ? other : (int)(threadIdx.x & 63));
        const float2 t = turns ? cs[8 * (second ? l - lanes : l) + k] : make_float2(1.0f, 0.0f);
        y[k] = turns ? x[k] * t.x + (second ? o : -o) * t.y : x[k];
      }
    }
    char *out = (char *)r.out + ((int64_t)b * r.obs + (int64_t)i * r.ors + (int64_t)h * D + 8 * l) * ESZ;
    if (BF16) {
      *(uint4 *)out = make_uint4(cgk::pack_bf16x2(y[0], y[1]), cgk::pack_bf16x2(y[2], y[3]), cgk::pack_bf16x2(y[4], y[5]),
                                 cgk::pack_bf16x2(y[6], y[7]));
    } else {
      ((float4 *)out)[0] = make_float4(y[0], y[1], y[2], y[3]);
      ((float4 *)out)[1] = make_float4(y[4], y[5], y[6], y[7]);
    }
  }
}

hipError_t rotate_launch(const RotateArgs &a0, bool bf16, hipStream_t s) {
  RotateArgs a = a0;
  const int64_t rows = (int64_t)a.batch * a.n;
  const int total = a.r[0].heads + a.r[1].heads;
  a.each = 16;
  a.chunks = (total + a.each - 1) / a.each;
  const dim3 grid((unsigned)(rows * a.chunks)), block(NTH);
  if (bf16) hipLaunchKernelGGL(k_rotate<true>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(k_rotate<false>, grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace cgr
