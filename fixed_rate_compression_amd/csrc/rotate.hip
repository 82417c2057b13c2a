// Norm of each query and key head and the rotation by its row's position, in one pass:
//   x <- w x / sqrt(mean x^2 + eps),   (x_a, x_b) <- (x_a cos - x_b sin, x_b cos + x_a sin)
// with the angle position * freq of the pair, the position that of the pair's axis.
//
// A row's query heads, and its key heads, go in groups of PER; 16 lanes take a group, 16 bytes a lane to a
// head (fp32: 32 bytes), and a workgroup 16 groups.  The loads are asked for before the sines and cosines of
// the rows are formed, and those go into one pair of factors a channel with the norm's weights, once a group.
// An angle is a product of far positions, so it is taken in fp64, in turns, and only what is left of whole
// turns goes on in fp32.  The other half of a pair comes from another lane's registers, a row rotation where
// all 128 channels turn.  Squares are summed in fp32: a head whose sum passes it (values of 1e19) is zeros.
//
// Bound by memory traffic where there are many rows: 4000 rows of 2 sequences, 32 + 8 heads, three axes, both
// norms (164 MB) take 34.5 us, 4750 GB/s, where a copy of the same size runs at 5100.  With factors formed a
// head and not a group it took 59 us, the vector instructions its bound.  A row of 64 sequences takes 4.1 us
// on the device, a launch and three loads that follow one another.
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
struct Eight {  // channels of a head
  uint4 w[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const char *p) {
    w[0] = *(const uint4 *)p;
    if constexpr (!BF16) w[1] = *(const uint4 *)(p + 16);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
    if constexpr (BF16) {
#pragma unroll
      for (int k = 0; k < 4; k++) {
        x[2 * k] = cgk::bf16lo(u[k]);
        x[2 * k + 1] = cgk::bf16hi(u[k]);
      }
    } else {
      const uint32_t v[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int k = 0; k < 4; k++) {
        x[k] = __uint_as_float(u[k]);
        x[4 + k] = __uint_as_float(v[k]);
      }
    }
  }
};

template <bool BF16>
__device__ __forceinline__ void store8(char *p, const float (&y)[8]) {
  if constexpr (BF16) {
    *(uint4 *)p = make_uint4(cgk::pack_bf16x2(y[0], y[1]), cgk::pack_bf16x2(y[2], y[3]), cgk::pack_bf16x2(y[4], y[5]),
                             cgk::pack_bf16x2(y[6], y[7]));
  } else {
    ((float4 *)p)[0] = make_float4(y[0], y[1], y[2], y[3]);
    ((float4 *)p)[1] = make_float4(y[4], y[5], y[6], y[7]);
  }
}

// v of the lane that holds the other half of this lane's pairs
template <bool FULL>
__device__ __forceinline__ float partner(float v, int lane) {
  if constexpr (FULL) return ror16<8>(v);
  else return __shfl(v, lane);
}

// y_k = u_k A_k + (the pair's other)_k B_k for the PER heads of a lane group, u the normed head without its weights
template <bool BF16, int PER, int MODE>  // 0: halves of 128 channels, 1: halves of fewer, 2: neighbours
__device__ __forceinline__ void turn(const Eight<BF16> (&in)[PER], char *out, int heads, bool norm, float eps,
                                     const float (&A)[8], const float (&B)[8], int other, bool turns) {
#pragma unroll
  for (int x = 0; x < PER; x++) {
    if (x >= heads) break;  // 16 lanes go together
    float v[8], y[8];
    in[x].get(v);
    if (norm) {
      float ss = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; k++) ss = __builtin_fmaf(v[k], v[k], ss);
      ss += ror16<8>(ss);
      ss += ror16<4>(ss);
      ss += ror16<2>(ss);
      ss += ror16<1>(ss);
      const float f = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
      for (int k = 0; k < 8; k++) v[k] *= f;
    }
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const float o = MODE == 2 ? v[k ^ 1] : partner<MODE == 0>(v[k], other);
      y[k] = __builtin_fmaf(o, B[k], v[k] * A[k]);
      if (MODE != 0 && !turns) y[k] = v[k] * A[k];
    }
    store8<BF16>(out + x * (int)(D * (BF16 ? 2 : 4)), y);
  }
}

template <bool BF16, int PER>
__global__ __launch_bounds__(NTH) void k_rotate(const RotateArgs a) {
  extern __shared__ __align__(16) float2 cs[];  // [row of the workgroup's][dim / 2]
  constexpr int ESZ = BF16 ? 2 : 4;
  const int half = a.dim >> 1;
  const uint32_t uq = (uint32_t)(a.r[0].heads + PER - 1) / PER, units = uq + (uint32_t)(a.r[1].heads + PER - 1) / PER;
  const uint32_t all = (uint32_t)a.batch * a.n, row0 = blockIdx.x * 16u / units;
  const int l = threadIdx.x & 15, g = threadIdx.x >> 4;
  const uint32_t unit = blockIdx.x * 16u + g, row = unit / units;
  const bool key = unit - row * units >= uq;
  const int h0 = (int)(unit - row * units - (key ? uq : 0u)) * PER;  // its first head
  Eight<BF16> in[PER];
  char *out = nullptr;
  int heads = 0;  // it has; none where there is no row, or padding
  const float *weight = key ? a.r[1].weight : a.r[0].weight;
  float A[8], B[8];
#pragma unroll
  for (int k = 0; k < 8; k++) A[k] = 1.0f;
  if (row < all) {
    const int b = (int)(row / (uint32_t)a.n), i = (int)(row - (uint32_t)b * a.n);
    const int64_t len = a.lengths ? min(max((int64_t)a.lengths[b], (int64_t)0), a.tokens) : a.tokens;
    const int64_t pos = (a.starts ? (int64_t)a.starts[b] : len - a.n) + i;
    if (pos >= 0 && pos < len) {
      heads = min(PER, (key ? a.r[1].heads : a.r[0].heads) - h0);
      const int64_t at = (int64_t)h0 * D + 8 * l;
      const char *src = (const char *)(key ? a.r[1].in : a.r[0].in) +
                        ((int64_t)b * (key ? a.r[1].ibs : a.r[0].ibs) + (int64_t)i * (key ? a.r[1].irs : a.r[0].irs) + at) * ESZ;
      out = (char *)(key ? a.r[1].out : a.r[0].out) +
            ((int64_t)b * (key ? a.r[1].obs : a.r[0].obs) + (int64_t)i * (key ? a.r[1].ors : a.r[0].ors) + at) * ESZ;
#pragma unroll
      for (int x = 0; x < PER; x++)
        if (x < heads) in[x].load(src + x * D * ESZ);
      if (weight) {
        const float4 u0 = ((const float4 *)(weight + 8 * l))[0], u1 = ((const float4 *)(weight + 8 * l))[1];
        const float w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
        for (int k = 0; k < 8; k++) A[k] = w[k];
      }
    }
  }
  const uint32_t rows = min((blockIdx.x * 16u + 15u) / units + 1, all) - row0;
  for (uint32_t k = threadIdx.x; k < rows * half; k += NTH) {
    const uint32_t dr = k / (uint32_t)half, r = row0 + dr;
    const int pair = (int)(k - dr * half), b = (int)(r / (uint32_t)a.n), i = (int)(r - (uint32_t)b * a.n);
    int64_t at;
    if (a.positions) {
      at = a.positions[((int64_t)axis_of(a, pair) * a.batch + b) * a.n + i];
    } else {
      const int64_t len = a.lengths ? min(max((int64_t)a.lengths[b], (int64_t)0), a.tokens) : a.tokens;
      at = (a.starts ? (int64_t)a.starts[b] : len - a.n) + i;
    }
    double turn = (double)at * ((double)a.freq[pair] * 0.15915494309189533576888);
    turn -= rint(turn);
    float s, c;
    sincospif(2.0f * (float)turn, &s, &c);
    cs[k] = make_float2(c * a.magnitude, s * a.magnitude);
  }
  __syncthreads();
  const float2 *t = cs + (row - row0) * half;
  if (a.interleaved) {
    const bool turns = 8 * l < a.dim;
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const float2 e = turns && heads ? t[4 * l + k / 2] : make_float2(1.0f, 0.0f);
      B[k] = -A[k + 1] * e.y;
      B[k + 1] = A[k] * e.y;
      A[k] *= e.x;
      A[k + 1] *= e.x;
    }
    turn<BF16, PER, 2>(in, out, heads, weight, a.eps, A, B, 0, turns);
  } else if (a.dim == D) {
    const float sign = l >= 8 ? 1.0f : -1.0f;
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const float2 e = heads ? t[8 * (l & 7) + k] : make_float2(1.0f, 0.0f);
      B[k] = partner<true>(A[k], 0) * (sign * e.y);
      A[k] *= e.x;
    }
    turn<BF16, PER, 0>(in, out, heads, weight, a.eps, A, B, 0, true);
  } else {
    const int lanes = a.dim >> 4;  // of half the turned channels
    const bool second = l >= lanes, turns = l < 2 * lanes;
    const int other = (int)(threadIdx.x & 48) + (!turns ? l : second ? l - lanes : l + lanes);
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const float2 e = turns && heads ? t[8 * (second ? l - lanes : l) + k] : make_float2(1.0f, 0.0f);
      B[k] = partner<false>(A[k], other) * (second ? e.y : -e.y);
      A[k] *= e.x;
    }
    turn<BF16, PER, 1>(in, out, heads, weight, a.eps, A, B, other, turns);
  }
}

template <bool BF16, int PER>
static hipError_t launch(const RotateArgs &a, hipStream_t s) {
  const int64_t units = (a.r[0].heads + PER - 1) / PER + (a.r[1].heads + PER - 1) / PER;
  const dim3 grid((unsigned)(((int64_t)a.batch * a.n * units + 15) / 16)), block(NTH);
  const int64_t rows = 14 / units + 2;  // that a workgroup's heads may be of
  hipLaunchKernelGGL((k_rotate<BF16, PER>), grid, block, (unsigned)(rows * (a.dim / 2) * sizeof(float2)), s, a);
  return hipGetLastError();
}

hipError_t rotate_launch(const RotateArgs &a, bool bf16, hipStream_t s) {
  // One head to a lane group while that leaves compute units free, four where they share the factors: 2560
  // heads 4.1 us and 4.7, 20480 heads 5.9 and 5.6, 32000 7.5 and 6.2, 128000 18.9 and 13.6.
  const bool few = (int64_t)a.batch * a.n * (a.r[0].heads + a.r[1].heads) <= 16 * 512;
  if (bf16) return few ? launch<true, 1>(a, s) : launch<true, 4>(a, s);
  return few ? launch<false, 1>(a, s) : launch<false, 4>(a, s);
}

}  // namespace cgr
