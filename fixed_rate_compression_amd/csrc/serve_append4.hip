// New K/V rows into the 4-bit KIVI-style cache: gauge, ranges and codes of the blocks of 32 tokens that they
// fall in, every sequence at its own position.
//
// A key's range is that of 32 tokens of its channel, a value's that of 32 channels of its token; the block
// that receives a row is encoded again from the raw rows (kept beside the cache, `tail`) and the new ones, as
// in the 8-bit cache.  Rows that are not there yet take no part in a range and their codes are not written.
//
// What bounds it is the chain of a call's loads and steps, so a workgroup takes one block of one (K/V,
// sequence, head), each of its four waves 32 channels from the load to the store, and no wave waits for
// another.  A lane loads eight channels of a row; 4 x 4 transpositions over a row's lanes give the
// matrix cores' operands (the gauge's are loaded in whole lines too and transposed likewise: in single
// values they took 128 of a wave's 350 cycles at the first cache).  The gauge is the encoder's chains of
// fused multiply-adds (cg_tile.hpp); its result has a lane hold 8 rows of two channels: a key's range is
// the lane's own and three other lanes', a value's that of 16 lanes.  Lanes side by side have the codes
// of a byte; a 4 x 4 transposition of bytes over four such pairs gives each lane a row's dword.
// The raw rows of the last block are stored by the wave that reads those of the first, after its reads.
//
// A token for 64 sequences of 8 heads 7.1 us on the device (rows in LDS, 64 to a workgroup whose waves
// met four times: 9.5), of which a single workgroup takes 4; prompts of up to 2000 tokens for 4 sequences 13.4
// (19.6), fp32 15.3.  Workgroups that take several blocks, the next one's rows on their way: 12.5 to 14.2, and
// a token 8.0 for the registers.
#include "cg_tile.hpp"
#include "quant_kernels.hpp"
#include "serve.hpp"

namespace cgs {

using namespace cgk;

template <int CTRL>
__device__ __forceinline__ uint32_t lanes(uint32_t v) {  // of another lane of the same 16
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ float lanes(float v) {
  return __uint_as_float(lanes<CTRL>(__float_as_uint(v)));
}
constexpr int XOR1 = 0xB1, XOR2 = 0x4E, XOR3 = 0x1B, MIRROR8 = 0x141, TURN8 = 0x128;

typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef float gauge4_t __attribute__((ext_vector_type(4), aligned(4)));  // gauges are aligned as floats are

// 8 of 32 channels of a row: bf16 8 q .. + 7 of quarter q of the wave, fp32 4 q .. + 3 and 16 + 4 q .. + 3
template <bool BF16>
struct Part {
  u4_t w[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const char *row, int q) {
    w[0] = *(const u4_t *)(row + 16 * q);
    if constexpr (!BF16) w[1] = *(const u4_t *)(row + 64 + 16 * q);
  }
  __device__ __forceinline__ void store(char *row, int q) const {
    *(u4_t *)(row + 16 * q) = w[0];
    if constexpr (!BF16) *(u4_t *)(row + 64 + 16 * q) = w[1];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const uint32_t u = w[0][k];
      if constexpr (BF16) {
        x[2 * k] = bf16lo(u);
        x[2 * k + 1] = bf16hi(u);
      } else {
        const uint32_t v = w[1][k];
        x[k] = __uint_as_float(u);
        x[4 + k] = __uint_as_float(v);
      }
    }
  }
};

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

// smallest (MAX: largest) of 8 rows over a lane's 16; v[4 p + j] is row 16 p + 4 (lane / 16) + j's.  Half of
// the rows go on in each step, so a lane is left with one: p its bit 3, j its bits 2 and 1
template <bool MAX>
__device__ __forceinline__ float of_rows(const float (&v)[8], int n) {
  const auto better = [](float x, float y) { return MAX ? fmaxf(x, y) : fminf(x, y); };
  float a[4], b[2];
#pragma unroll
  for (int j = 0; j < 4; j++) a[j] = better(n & 8 ? v[4 + j] : v[j], lanes<TURN8>(n & 8 ? v[j] : v[4 + j]));
#pragma unroll
  for (int j = 0; j < 2; j++) b[j] = better(n & 4 ? a[2 + j] : a[j], lanes<MIRROR8>(n & 4 ? a[j] : a[2 + j]));
  const float c = better(n & 2 ? b[1] : b[0], lanes<XOR2>(n & 2 ? b[0] : b[1]));
  return better(c, lanes<XOR1>(c));
}

// rint((x - mn) inv) between 0 and 15 in the low bits, 0 where it is not a number: the float 1.5 2^23 + q
__device__ __forceinline__ uint32_t code(float x, float mn, float inv) {
  const float p = (x - mn) * inv;
  return __float_as_uint(fminf(fmaxf(p, 0.0f), 15.0f) + 12582912.0f);
}

template <bool BF16, int G>
__global__ __launch_bounds__(NT, G == 128 ? 2 : G == 32 && !BF16 ? 4 : 8) void k_append4(const AppendArgs a) {
  constexpr int PIECES = G == 128 ? 4 : 1;  // of 32 channels, that a wave reads
  constexpr int ESZ = BF16 ? 2 : 4, XP = 36;
  __shared__ float2 vrange[4][32];                                // a wave's own: (minimum, 1 / step) of the rows
  __shared__ __align__(16) float rows[G == 0 ? 4 * 32 * XP : 1];  // no gauge: a wave's own rows, to be turned round
  const uint32_t q1 = a.by_tiles(blockIdx.x), q2 = a.by_heads(q1);
  const int strip = (int)(blockIdx.x - q1 * a.tiles), h = (int)(q1 - q2 * a.heads);
  const int kind = (int)q2 >= a.batch, b = (int)q2 - (kind ? a.batch : 0);
  const int64_t f = q1;  // (kind, b, h)
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, n = lane & 15, kr = lane >> 4;
  const int32_t *any = (const int32_t *)a.k;  // both loads at once, from a place that is there where an array is not
  const int32_t ln = *(a.lengths ? a.lengths + b : any), sn = *(a.starts ? a.starts + b : any);
  MfmaGaugeFrags<G ? G : 16> fr;  // fr.b[nb][4 k + e]: channel 16 k + 4 kr + e of row 16 nb + n, until it is transposed
  const float *gf = G ? a.gauges + (int64_t)(kind * a.heads + h) * (D * G) : nullptr;
  if constexpr (G == 8) {
    load_mfma_gauge<G, false>(gf, fr);
  } else if constexpr (G != 0) {
#pragma unroll
    for (int nb = 0; nb < 2; nb++) {
      const float *row = gf + (32 * w + 16 * nb + n) * G + 4 * kr;  // the groups follow one another
#pragma unroll
      for (int k = 0; k < G / 16; k++) {
        const gauge4_t g = *(const gauge4_t *)(row + 16 * k);
        fr.b[nb][4 * k] = g.x;
        fr.b[nb][4 * k + 1] = g.y;
        fr.b[nb][4 * k + 2] = g.z;
        fr.b[nb][4 * k + 3] = g.w;
      }
    }
  }
  const int64_t len = a.lengths ? min(max((int64_t)ln, (int64_t)0), a.tokens) : a.tokens;
  const int64_t start = a.starts ? (int64_t)sn : len - a.n;
  const int64_t p0 = max(start, (int64_t)0), p1 = min(start + a.n, len);  // positions of the new rows
  if (p1 <= p0) return;
  const int64_t head = p0 & ~(int64_t)31, tb = head + (int64_t)strip * 32;
  if (tb >= p1) return;
  const int there = (int)min((int64_t)32, p1 - tb), old = (int)max(p0 - tb, (int64_t)0);  // rows of the block
  // src: as if position `tb` of the head's rows were row 0
  const int64_t rs = a.row_stride * ESZ;
  const char *src = (const char *)(kind ? a.v : a.k) + ((int64_t)b * a.batch_stride + (int64_t)h * D) * ESZ + (tb - start) * rs;
  char *tail = (char *)a.tail + f * (32 * D * ESZ);
  Part<BF16> in[2][PIECES], raw[2];
#pragma unroll
  for (int p = 0; p < 2; p++) {
    const int r = 16 * p + n;
#pragma unroll
    for (int k = 0; k < PIECES; k++) {
      in[p][k].w[0] = u4_t(0u);
      if constexpr (!BF16) in[p][k].w[1] = u4_t(0u);
    }
    if (r < there) {
      const char *row = (r < old ? tail + r * (D * ESZ) : src + r * rs) + (G == 128 ? 0 : 32 * ESZ * w);
#pragma unroll
      for (int k = 0; k < PIECES; k++) in[p][k].load(row + 32 * ESZ * k, kr);
    }
  }
  // new rows of the last block, which strip 0 keeps
  const int last = (int)(((p1 - 1) & ~(int64_t)31) - tb), keep0 = max(old, last), keep1 = (int)(p1 - tb);
  if (strip == 0) {
#pragma unroll
    for (int p = 0; p < 2; p++) {
      const int r = last + 16 * p + n;
      if (r >= keep0 && r < keep1) raw[p].load(src + r * rs + 32 * ESZ * w, kr);
    }
  }

  if constexpr (G == 128)  // here the waves read one another's channels of the old rows
    if (strip == 0) {
#pragma unroll
      for (int p = 0; p < 2; p++)
#pragma unroll
        for (int k = 0; k < PIECES; k++) {
          asm volatile("" ::"v"(in[p][k].w[0]));  // the rows have come
          if constexpr (!BF16) asm volatile("" ::"v"(in[p][k].w[1]));
        }
      __syncthreads();
    }

  // y[p][nb][j]: row 16 p + 4 kr + j, channel 32 w + 16 nb + n
  float y[2][2][4];
  if constexpr (G == 0) {
    float *x = rows + w * 32 * XP;
#pragma unroll
    for (int p = 0; p < 2; p++) {
      float v[8];
      in[p][0].get(v);
#pragma unroll
      for (int k = 0; k < 2; k++)
        *(float4 *)(x + (16 * p + n) * XP + (BF16 ? 8 * kr + 4 * k : 16 * k + 4 * kr)) =
            make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int p = 0; p < 2; p++)
#pragma unroll
      for (int k = 0; k < 2; k++)
#pragma unroll
        for (int j = 0; j < 4; j++) y[p][k][j] = x[(16 * p + 4 * kr + j) * XP + 16 * k + n];
  } else {
    if constexpr (G >= 16)
#pragma unroll
      for (int nb = 0; nb < 2; nb++)
#pragma unroll
        for (int k = 0; k < G / 16; k++)
          transpose(fr.b[nb][4 * k], fr.b[nb][4 * k + 1], fr.b[nb][4 * k + 2], fr.b[nb][4 * k + 3]);
    cg_f32x4_t acc[2][2], other[2][2];  // other: groups of 8, the second of 16 channels
#pragma unroll
    for (int p = 0; p < 2; p++)
#pragma unroll
      for (int nb = 0; nb < 2; nb++) acc[p][nb] = other[p][nb] = cg_f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < PIECES; k++)
#pragma unroll
      for (int p = 0; p < 2; p++) {
        // transposed, register e of quarter kr is of 4 e + kr in 16 channels; of bf16's, whose quarters are
        // eight channels apart, 8 (e & 1) + 4 (register / 4) + kr of group e / 2
        float x[8];
        in[p][k].get(x);
        transpose(x[0], x[1], x[2], x[3]);
        transpose(x[4], x[5], x[6], x[7]);
#pragma unroll
        for (int g16 = 0; g16 < 2; g16++)
#pragma unroll
          for (int s = 0; s < 4; s++) {
            const float v = BF16 ? x[4 * (s & 1) + 2 * g16 + (s >> 1)] : x[4 * g16 + s];
#pragma unroll
            for (int nb = 0; nb < 2; nb++) {
              if (G <= 16 && nb != g16) continue;
              cg_f32x4_t &c = G == 8 && s >= 2 ? other[p][nb] : acc[p][nb];
              const int e = G == 8 ? s & 1 : G == 16 ? s : 8 * k + 4 * g16 + s;
              c = __builtin_amdgcn_mfma_f32_16x16x4f32(v, fr.b[nb][e], c, 0, 0, 0);
            }
          }
      }
#pragma unroll
    for (int p = 0; p < 2; p++)
#pragma unroll
      for (int nb = 0; nb < 2; nb++)
#pragma unroll
        for (int j = 0; j < 4; j++) y[p][nb][j] = G == 8 && n >= 8 ? other[p][nb][j] : acc[p][nb][j];
  }
  if (strip == 0) {
#pragma unroll
    for (int p = 0; p < 2; p++) {
      const int r = last + 16 * p + n;
      if (r >= keep0 && r < keep1) raw[p].store(tail + (16 * p + n) * (D * ESZ) + 32 * ESZ * w, kr);
    }
  }

  float2 *meta = (float2 *)a.meta + 4 * f * a.tcap;
  uint32_t word[2][2];  // codes of 4 rows, a byte each
  const auto put = [&](int p, int nb, const uint32_t (&q)[4]) {
    constexpr uint32_t M = 0x4B400000u;  // of 1.5 2^23
    word[p][nb] = (q[0] + (q[1] << 8)) + ((q[2] << 16) + (q[3] << 24)) - (M + (M << 8) + (M << 16) + (M << 24));
  };
  if (kind == 0) {
    float mn[2], mx[2];
#pragma unroll
    for (int nb = 0; nb < 2; nb++) {
      mn[nb] = INFINITY;
      mx[nb] = -INFINITY;
#pragma unroll
      for (int p = 0; p < 2; p++)
#pragma unroll
        for (int j = 0; j < 4; j++)
          if (16 * p + 4 * kr + j < there) {
            mn[nb] = fminf(mn[nb], y[p][nb][j]);
            mx[nb] = fmaxf(mx[nb], y[p][nb][j]);
          }
    }
    // over the four lanes of a channel: both channels' of half the lanes, then one's
    swap32(mn[0], mn[1]);
    swap32(mx[0], mx[1]);
    float lo = fminf(mn[0], mn[1]), hi = fmaxf(mx[0], mx[1]);  // lanes below 32: channel 0's, above: 1's
    {
      float l2 = lo, h2 = hi;
      swap16(lo, l2);
      swap16(hi, h2);
      lo = fminf(lo, l2);
      hi = fmaxf(hi, h2);
    }
    const cgq::Range r = cgq::make_range(lo, hi, 15);
    if (!(kr & 1)) meta[(tb >> 5) * D + 32 * w + 16 * (kr >> 1) + n] = make_float2(r.mn, r.scale);
    float m0 = r.mn, m1 = r.mn, i0 = r.zero ? 0.0f : r.inv, i1 = i0;
    swap32(m0, m1);
    swap32(i0, i1);
#pragma unroll
    for (int p = 0; p < 2; p++)
#pragma unroll
      for (int nb = 0; nb < 2; nb++) {
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; j++) q[j] = code(y[p][nb][j], nb ? m1 : m0, nb ? i1 : i0);
        put(p, nb, q);
      }
  } else {
    float mn[8], mx[8];
#pragma unroll
    for (int k = 0; k < 8; k++) {
      mn[k] = fminf(y[k >> 2][0][k & 3], y[k >> 2][1][k & 3]);
      mx[k] = fmaxf(y[k >> 2][0][k & 3], y[k >> 2][1][k & 3]);
    }
    const cgq::Range r = cgq::make_range(of_rows<false>(mn, n), of_rows<true>(mx, n), 15);
    const int at = 2 * (n & 8) + 4 * kr + ((n >> 1) & 3);  // the row that this lane is left with
    if (!(n & 1)) {
      vrange[w][at] = make_float2(r.mn, r.zero ? 0.0f : r.inv);
      if (at < there) meta[(tb + at) * 4 + w] = make_float2(r.mn, r.scale);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int p = 0; p < 2; p++) {
      uint32_t q0[4], q1[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float2 m = vrange[w][16 * p + 4 * kr + j];
        q0[j] = code(y[p][0][j], m.x, m.y);
        q1[j] = code(y[p][1][j], m.x, m.y);
      }
      put(p, 0, q0);
      put(p, 1, q1);
    }
  }

  // bytes of two channels: even lanes the first group's, odd lanes the second's; then a row's four of them
  const uint32_t sa = n & 2 ? 0x03070105u : 0x06020400u, sb = n & 4 ? 0x03020706u : 0x05040100u;
#pragma unroll
  for (int p = 0; p < 2; p++) {
    const uint32_t own = n & 1 ? word[p][1] : word[p][0], got = lanes<XOR1>(n & 1 ? word[p][0] : word[p][1]);
    uint32_t x = n & 1 ? got | own << 4 : own | got << 4;
    x = __builtin_amdgcn_perm(lanes<XOR2>(x), x, sa);
    x = __builtin_amdgcn_perm(lanes<XOR3>(lanes<MIRROR8>(x)), x, sb);
    const int row = 16 * p + 4 * kr + ((n >> 1) & 3);
    if (row < there)
      *(uint32_t *)(a.payload + (f * a.tcap + tb + row) * (D / 2) + 16 * w + 8 * (n & 1) + (n >> 3) * 4) = x;
  }
}

hipError_t append4_launch(const AppendArgs &a, bool bf16, int g, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)2 * a.batch * a.heads * a.tiles)), block(NT);
#define CG_A(BF, GG)                                               \
  if (bf16 == BF && g == GG) {                                     \
    hipLaunchKernelGGL((k_append4<BF, GG>), grid, block, 0, s, a); \
    return hipGetLastError();                                      \
  }
  CG_A(true, 0) CG_A(true, 8) CG_A(true, 16) CG_A(true, 32) CG_A(true, 128)
  CG_A(false, 0) CG_A(false, 8) CG_A(false, 16) CG_A(false, 32) CG_A(false, 128)
#undef CG_A
  return hipErrorInvalidValue;
}

}  // namespace cgs
