// Attention over the 8-bit block-uniform cache: launch interface and the
// device pieces its kernels share.  Not part of the public ABI.
//
// With k'_t = mk_b + sk_b code_t and v'_t = mv_b + sv_b code_t (block b of
// token t), a gauged query row q' = G_K q and c = scale log2(e):
//   s_t = c (q' . k'_t) = (c sk_b) (q' . code_t) + (c sum q') mk_b
//   u   = sum_t p_t v'_t = sum_t (p_t sv_b) code_t + sum_t p_t mv_b,  p_t = 2^(s_t - m)
//   out = G_V^T u / sum_t p_t
// so both products run on the codes themselves and the ranges are applied to
// scores and weights.  For the values the code is taken less 128 and the
// minimum plus 128 sv_b: the matrix cores' fp32 sums then hold the values'
// deviations and not 128 times the sum of the weights, against which a mean
// over many tokens is small (uncentred, 262144 tokens lose 2^-9 of the output).  A code c = 0 .. 255 placed in the low byte of an fp16
// is the subnormal c 2^-24, which the matrix cores multiply exactly: widening
// a dword of codes costs two byte permutes and no conversion.
//
// Query rows: a KV head's rows are (query i, head j of the group), row
// i ratio + j; a row tile is 16 of them.  q' is scaled by a power of two that
// puts the row's largest magnitude in [2^13, 2^14) and held in two fixed-point
// parts, hi a multiple of 2^4 and lo of 2^-7 (2^-22 of the largest): each
// part's sum over 128 centred codes is a whole number of at most 2^24 units,
// so the matrix cores, which round their fp32 sums towards zero, add it
// without a rounding (as two floating parts in one sum, fp32 outputs were off
// by 1e-5, now by 1e-6).  sum q' is that of the parts, so a rounding of q'
// perturbs the query and not the balance of the two terms of s_t.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cg_tile.hpp"

namespace cga {

using cgk::D;
using cgk::PITCH;

constexpr int ROWS = 16;  // query rows of a row tile (one matrix-core operand)
constexpr int UNIT = 32;  // tokens of a unit of work
constexpr int NTH = 256;  // threads of a workgroup
constexpr int MERGE_SPLITS = 1024;  // splits at most

struct AttendArgs {
  const uint8_t *kpay, *vpay;    // codes of the layer's key / value fields, field (b, h) at (b heads + h) tcap 128
  const float2 *kmeta, *vmeta;   // (minimum, step) of the layer's blocks, [b][h][nblk]
  const int32_t *lengths;        // [batch] or null (tokens)
  const int32_t *starts;         // [batch] or null (lengths - n)
  const float *gk, *gv;          // the layer's gauges [heads][128 g], ignored when g == 0
  const void *q;                 // storage format
  void *out;
  float *lse;                    // [batch][n][q_heads] or null
  float *mass;                   // the layer's [b][h][nblk] or null
  float *part_o;                 // [b][h][split][rows][128] sums of a split
  float2 *part_ml;               // [b][h][split][rows] (maximum, sum of weights)
  float2 *bsum;                  // [b][h][entry][rows] (block sum, its maximum)
  float *lse2;                   // [b][h][rows] log2 of the row's sum (many rows with mass)
  float *mpart;                  // [part][b][h][nblk] parts of the blocks' weights (many rows)
  uint4 *qfrag;                  // [b][h][tile][hi/lo][step][lane] fp16 query operands
  float2 *qrow;                  // [b][h][16 tiles] (score factor, minimum factor)
  int64_t tcap, tokens, nblk;
  int64_t q_bs, q_ts;            // query strides (elements)
  int64_t entries;               // block-sum entries of a field
  int32_t batch, heads, ratio, n, rows, tiles;  // rows = n ratio, tiles = ceil(rows / 16)
  int32_t g, bshift, causal, splits, mparts;
  float c;                       // scale log2(e)
};

// rows [0, rows) of every field over its tokens, one workgroup per (field,
// row tile, split); splits > 1 leaves parts for merge_launch
hipError_t rows_launch(const AttendArgs &a, bool bf16, hipStream_t s);
// the same for many rows, one workgroup per (field, 128 rows, split),
// after one that lays the gauged queries out (qfrag, qrow)
hipError_t tile_launch(const AttendArgs &a, bool bf16, hipStream_t s);
hipError_t merge_launch(const AttendArgs &a, bool bf16, hipStream_t s);
// block weights: few rows from the attention's block sums, many rows from a
// second pass over the keys with the rows' sums known
hipError_t mass_finish_launch(const AttendArgs &a, hipStream_t s);
hipError_t mass_many_launch(const AttendArgs &a, hipStream_t s);

// ---------------------------------------------------------------------------
// device pieces
// ---------------------------------------------------------------------------

typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef float f2_t __attribute__((ext_vector_type(2)));
typedef float f4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f4_t mfma(h8_t a, h8_t b, f4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const f2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, h2_t));
}

__device__ __forceinline__ f2_t unpack_f16x2(uint32_t w) {
  return __builtin_convertvector(__builtin_bit_cast(h2_t, w), f2_t);
}

__device__ __forceinline__ h8_t as_h8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint4 v = make_uint4(a, b, c, d);
  return __builtin_bit_cast(h8_t, v);
}

// bytes J and J + 1 of a dword as the halves (J even)
template <int J>
__device__ __forceinline__ uint32_t bytes2(uint32_t w) {
  return __builtin_amdgcn_perm(0u, w, 0x0c000c00u | ((J + 1) << 16) | J);
}

// codes as subnormals -> (code - 128) 2^-9, one packed multiply-add, exact.  The
// matrix cores align the products of a sum by their exponent fields and cut
// what lies below: with subnormal operands, whose significands begin with
// zeros, sums of weights of unlike sizes kept 17 bits, with these 24.
__device__ __forceinline__ uint32_t centred(uint32_t w) {
  const h2_t up = {(_Float16)32768.0f, (_Float16)32768.0f}, c = {(_Float16)-0.25f, (_Float16)-0.25f};
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(h2_t, w), up, c));
}
constexpr float kCodeUnit = 16777216.0f;  // 2^24: codes as they are
constexpr float kCentredUnit = 512.0f;    // 2^9: centred codes

// 8 consecutive codes (two dwords) as fp16 subnormals, CENTRED: less 128
template <bool CENTRED>
__device__ __forceinline__ h8_t codes8(uint32_t a, uint32_t b) {
  if constexpr (CENTRED)
    return as_h8(centred(bytes2<0>(a)), centred(bytes2<2>(a)), centred(bytes2<0>(b)), centred(bytes2<2>(b)));
  else
    return as_h8(bytes2<0>(a), bytes2<2>(a), bytes2<0>(b), bytes2<2>(b));
}

// byte J of two dwords as the halves (lo of w0)
template <int J>
__device__ __forceinline__ uint32_t byte_pair(uint32_t w0, uint32_t w1) {
  return __builtin_amdgcn_perm(w1, w0, 0x0c000c00u | ((J + 4) << 16) | J);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// sum / maximum over the four lanes of one row (lane, lane ^ 16, ^ 32, ^ 48)
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}

// tokens of sequence b
__device__ __forceinline__ int seq_length(const AttendArgs &a, int b) {
  const int64_t n = a.lengths ? (int64_t)a.lengths[b] : a.tokens;
  return (int)min(max(n, (int64_t)0), a.tokens);
}

// tokens query i of sequence b sees: none unless it stands inside the sequence
__device__ __forceinline__ int query_limit(const AttendArgs &a, int b, int len, int i) {
  const int64_t pos = (a.starts ? (int64_t)a.starts[b] : (int64_t)len - a.n) + i;
  if (pos < 0 || pos >= len) return 0;
  return a.causal ? (int)pos + 1 : len;
}

// the largest limit of queries [i0, i1]
__device__ __forceinline__ int limit_of(const AttendArgs &a, int b, int len, int i0, int i1) {
  const int64_t p0 = a.starts ? (int64_t)a.starts[b] : (int64_t)len - a.n;
  const int64_t lo = max(p0 + i0, (int64_t)0), hi = min(p0 + i1, (int64_t)len - 1);
  if (lo > hi) return 0;
  return a.causal ? (int)hi + 1 : len;
}

// this thread's 8 channels of one of the query rows [r0, r0 + 16) of (b, h) as
// fp32; rows past the last one are zero
struct RowPart {
  f4_t lo, hi;
};

template <bool BF16>
__device__ __forceinline__ RowPart load_row_part(const AttendArgs &a, int b, int h, int r0) {
  const int r = r0 + (threadIdx.x >> 4), c = (threadIdx.x & 15) * 8;
  RowPart p;
  p.lo = p.hi = f4_t{0.f, 0.f, 0.f, 0.f};
  if (r < a.rows) {
    const int i = r / a.ratio, j = r - i * a.ratio;
    const int64_t off = (int64_t)b * a.q_bs + (int64_t)i * a.q_ts + (int64_t)(h * a.ratio + j) * D + c;
    if (BF16) {
      const uint4 w = *(const uint4 *)((const uint16_t *)a.q + off);
      p.lo = f4_t{cgk::bf16lo(w.x), cgk::bf16hi(w.x), cgk::bf16lo(w.y), cgk::bf16hi(w.y)};
      p.hi = f4_t{cgk::bf16lo(w.z), cgk::bf16hi(w.z), cgk::bf16lo(w.w), cgk::bf16hi(w.w)};
    } else {
      const f4_t *x = (const f4_t *)((const float *)a.q + off);
      p.lo = x[0];
      p.hi = x[1];
    }
  }
  return p;
}

// into xs [16][PITCH]
__device__ __forceinline__ void put_row_part(float *xs, const RowPart &p) {
  float *d = xs + (threadIdx.x >> 4) * PITCH + (threadIdx.x & 15) * 8;
  *(f4_t *)d = p.lo;
  *(f4_t *)(d + 4) = p.hi;
}

// y = G x (INV: G^T x) for rows of xs [NR][PITCH], fmaf chains over a group's
// channels in index order; thread (c, half) owns channel c of rows half,
// half + 2, ...  The first 32 weights of the thread's chain are loaded apart
// from their use, so that they travel beside other loads.
constexpr int GCHUNK = 32;
struct GaugeWeights {
  float w[GCHUNK];
};

template <bool INV>
__device__ __forceinline__ void load_gauge(const float *__restrict__ gh, int g, int k0, GaugeWeights &x) {
  if (g == 0) return;
  const int c = threadIdx.x & (D - 1), cg = c & (g - 1);  // g is a power of two
  const float *gp = gh + (int64_t)(c - cg) * g + (INV ? cg : cg * g);
#pragma unroll
  for (int k = 0; k < GCHUNK; k += 8) {
    if (k0 + k < g) {
#pragma unroll
      for (int e = 0; e < 8; e++) x.w[k + e] = gp[INV ? (k0 + k + e) * g : k0 + k + e];
    }
  }
}

// gw: load_gauge's for k0 = 0; emit(row, c, value) takes the results of rows < nr
template <bool INV, int NR, typename Emit>
__device__ __forceinline__ void gauge_rows(const float *xs, int nr, const float *__restrict__ gh, int g,
                                           const GaugeWeights &first, Emit emit) {
  const int c = threadIdx.x & (D - 1), half = threadIdx.x >> 7;
  if (g == 0) {
    for (int r = half; r < nr; r += 2) emit(r, c, xs[r * PITCH + c]);
    return;
  }
  const int base = c - (c & (g - 1));
  float acc[NR / 2];
#pragma unroll
  for (int r = 0; r < NR / 2; r++) acc[r] = 0.0f;
  GaugeWeights x = first;
  for (int k0 = 0; k0 < g; k0 += GCHUNK) {
    if (k0) load_gauge<INV>(gh, g, k0, x);
#pragma unroll
    for (int k = 0; k < GCHUNK; k += 8) {
      if (k0 + k < g) {
        const float *w = x.w + k;
#pragma unroll
        for (int r = 0; r < NR / 2; r++) {
          if (half + 2 * r < nr) {
            const float *p = xs + (half + 2 * r) * PITCH + base + k0 + k;
            const f4_t u = *(const f4_t *)p, v = *(const f4_t *)(p + 4);
            float t = acc[r];
            t = __builtin_fmaf(w[0], u[0], t); t = __builtin_fmaf(w[1], u[1], t);
            t = __builtin_fmaf(w[2], u[2], t); t = __builtin_fmaf(w[3], u[3], t);
            t = __builtin_fmaf(w[4], v[0], t); t = __builtin_fmaf(w[5], v[1], t);
            t = __builtin_fmaf(w[6], v[2], t); t = __builtin_fmaf(w[7], v[3], t);
            acc[r] = t;
          }
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < NR / 2; r++)
    if (half + 2 * r < nr) emit(half + 2 * r, c, acc[r]);
}

// The fp16 operands of 16 gauged rows xs [16][PITCH]: lane (row = lane % 16,
// grp = lane / 16) holds 8 channels of its row at step s: BYTES: 64 (s / 2) +
// 16 grp + 8 (s % 2) + 0 .. 7, the order in which 16-byte loads of key codes
// arrive; else 32 s + 8 grp + 0 .. 7.
struct QueryFrags {
  h8_t hi[4], lo[4];
  float ca, cq;  // score = (sum of q' code) step ca + minimum cq
};

// TWO: two fixed-point parts; else one fp16 part, each channel rounded to 2^-11
template <bool TWO, bool BYTES>
__device__ __forceinline__ void make_frags(const float *xs, float c, QueryFrags &f) {
  const int lane = threadIdx.x & 63, row = lane & 15, grp = lane >> 4;
  float x[4][8];
  float mx = 0.0f;
#pragma unroll
  for (int s = 0; s < 4; s++) {
    const float *p = xs + row * PITCH + (BYTES ? 64 * (s >> 1) + 16 * grp + 8 * (s & 1) : 32 * s + 8 * grp);
    const float4 u = *(const float4 *)p, v = *(const float4 *)(p + 4);
    x[s][0] = u.x; x[s][1] = u.y; x[s][2] = u.z; x[s][3] = u.w;
    x[s][4] = v.x; x[s][5] = v.y; x[s][6] = v.z; x[s][7] = v.w;
#pragma unroll
    for (int k = 0; k < 8; k++) mx = fmaxf(mx, fabsf(x[s][k]));
  }
  mx = row_max(mx);
  // power-of-two factor that puts the row's maximum into [2^13, 2^14)
  const int ex = mx > 0.0f ? (int)(__float_as_uint(mx) >> 23) - 127 : 0;
  const int sh = min(max(13 - ex, -100), 100);
  const float up = __builtin_ldexpf(1.0f, sh);
  float sum = 0.0f;
#pragma unroll
  for (int s = 0; s < 4; s++) {
    uint32_t wh[4], wl[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const float p = x[s][2 * k] * up, q = x[s][2 * k + 1] * up;
      if constexpr (TWO) {
        const float ph = rintf(p * 0.0625f) * 16.0f, qh = rintf(q * 0.0625f) * 16.0f;
        const float pl = rintf((p - ph) * 128.0f) * 0.0078125f, ql = rintf((q - qh) * 128.0f) * 0.0078125f;
        wh[k] = pack_f16x2(ph, qh);  // both parts are exact in fp16
        wl[k] = pack_f16x2(pl, ql);
        sum += (ph + pl) + (qh + ql);
      } else {
        wh[k] = pack_f16x2(p, q);
        wl[k] = 0u;
        const f2_t h = unpack_f16x2(wh[k]);
        sum += h.x + h.y;
      }
    }
    f.hi[s] = as_h8(wh[0], wh[1], wh[2], wh[3]);
    f.lo[s] = as_h8(wl[0], wl[1], wl[2], wl[3]);
  }
  const float down = c * __builtin_ldexpf(1.0f, -sh);
  f.ca = down;
  f.cq = down * row_sum(sum);
}

// one output row element (b, query row r of head h, channel c)
template <bool BF16>
__device__ __forceinline__ void store_out(const AttendArgs &a, int b, int h, int r, int c, float v) {
  const int i = r / a.ratio, j = r - i * a.ratio;
  const int64_t off = (((int64_t)b * a.n + i) * a.heads * a.ratio + h * a.ratio + j) * D + c;
  if (BF16) ((uint16_t *)a.out)[off] = (uint16_t)cgk::bf16_rne(v);
  else ((float *)a.out)[off] = v;
}

__device__ __forceinline__ void store_lse(const AttendArgs &a, int b, int h, int r, float m, float l) {
  const int i = r / a.ratio, j = r - i * a.ratio;
  // natural logarithm of the row's sum of exp(score)
  a.lse[((int64_t)b * a.n + i) * a.heads * a.ratio + h * a.ratio + j] =
      l > 0.0f ? (m + __builtin_log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace cga
