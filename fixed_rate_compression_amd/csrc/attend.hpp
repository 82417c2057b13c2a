// Attention over the serving caches (8-bit block-uniform, 4-bit KIVI-style): launch
// interface and the device pieces its kernels share.  Not part of the public ABI.
//
// 8 bits:
//
// With k'_t = mk_b + sk_b code_t and v'_t = mv_b + sv_b code_t (block b of
// token t), a gauged query row q' = G_K q and c = scale log2(e):
//   s_t = c (q' . k'_t) = (c sk_b) (q' . code_t) + (c sum q') mk_b
//   u   = sum_t p_t v'_t = sum_t (p_t sv_b) code_t + sum_t p_t mv_b,  p_t = 2^(s_t - m)
//   out = G_V^T u / sum_t p_t
// so both products run on the codes themselves and the ranges are applied to
// scores and weights.  For the values the code is taken less a centre z and the
// minimum plus z sv_b: the matrix cores' fp32 sums then hold the values'
// deviations and not z times the sum of the weights, against which a mean
// over many tokens is small (uncentred, 262144 tokens lose 2^-9 of the output).  z is
// 128 for bf16 storage and the code of the value 0 for fp32 storage, there for the keys
// as well (see Centre).  A code c = 0 .. 255 placed in the low byte of an fp16
// is the subnormal c 2^-24, which the matrix cores multiply exactly: widening
// a dword of codes costs two byte permutes and no conversion.
//
// Query rows: a KV head's rows are (query i, head j of the group), row
// i ratio + j; a row tile is 16 of them.  q' is scaled by a power of two that
// puts the row's largest magnitude in [2^13, 2^14) and held in two fp16 parts: hi, a
// multiple of 2^3, and lo, what is left of it (2^2 at most, so off by 2^-10: 2^-23 of
// the largest; a channel below 2^-11 of that by 2^-12 of itself).  The sum of hi over 128
// centred codes is a whole number of units, 2^26 at most and hardly ever beyond 2^24, so
// the matrix cores, which round their fp32 sums towards zero, add it without a
// rounding; that of lo is 2^-11 of it (as two floating parts in one sum, fp32 outputs
// were off by 1e-5; with lo in fixed point, 2^-21 of the largest, log-sums of 45 and 5
// tokens by 1.3e-7 and 3.0e-7, now by 0.6e-7 and 1.2e-7).  sum q' is that of the parts,
// so a rounding of q' perturbs the query and not the balance of the two terms of s_t.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cg_tile.hpp"
#include "cg_wave.hpp"

namespace cga {

using cgk::D;
using cgk::PITCH;

constexpr int ROWS = 16;  // query rows of a row tile (one matrix-core operand)
constexpr int FEW_TILES = 4;  // at most of the few-row form
constexpr int UNIT = 32;  // tokens of a unit of work
constexpr int NTH = 256;  // threads of a workgroup
constexpr int MERGE_SPLITS = 1024;  // splits at most

struct AttendArgs {
  const uint8_t *kpay, *vpay;    // codes of the layer's key / value fields, field (b, h) at (b heads + h) tcap 128
                                 // (4 bits: tcap 64)
  const float2 *kmeta, *vmeta;   // (minimum, step) of the layer's blocks, [b][h][nblk]; 4 bits: of keys
                                 // [b][h][nblk][128], of values [b][h][tcap][4]
  const int32_t *lengths;        // [batch] or null (tokens)
  const int32_t *starts;         // [batch] or null (lengths - n)
  const float *gk, *gv;          // the layer's gauges [heads][128 g], ignored when g == 0
  const void *q;                 // storage format
  void *out;
  float *lse;                    // [batch][n][q_heads] or null
  float *mass;                   // the layer's [b][h][nblk] or null
  float *part_o;                 // [b][h][split][rows][128] sums of a split
  float2 *part_ml;               // [b][h][split][rows] (maximum, sum of weights)
  int2 *dealt;                   // [b] (first slot, slots) of sequences of unlike lengths
  float2 *bsum;                  // [b][h][entry][rows] (block sum, its maximum)
  float *lse2;                   // [b][h][rows] log2 of the row's sum (many rows with mass)
  int64_t tcap, tokens, nblk;
  int64_t q_bs, q_ts;            // query strides (elements)
  int64_t entries;               // block-sum entries of a field
  int32_t batch, heads, ratio, n, rows, tiles;  // rows = n ratio, tiles = ceil(rows / 16)
  int32_t n_all, first;          // queries of the call, the first of these n (q, out and lse point at it)
  int32_t g, bshift, causal, splits, few;
  int32_t waves;  // of a few-row workgroup: 4 or 8
  int32_t ragged, slots, least;  // few rows of sequences of unlike lengths: see Slot
  float c;                       // scale log2(e)
  // many rows over the 4-bit cache: what ranges4_launch leaves of every block of the tokens' bound
  uint8_t *ranges;               // [b][h][block] scaled ranges
  void *units;                   // [b][h][block] powers of two
  int32_t two;                   // keys in two parts
};

// rows [0, rows) of every field over its tokens, one workgroup per (field,
// row tile, split); splits > 1 leaves parts for merge_launch
hipError_t rows_launch(const AttendArgs &a, bool bf16, hipStream_t s);
// the same over the 4-bit cache
hipError_t rows4_launch(const AttendArgs &a, bool bf16, hipStream_t s);
// the same for many rows, one workgroup per (field, 128 rows, split)
hipError_t tile_launch(const AttendArgs &a, bool bf16, hipStream_t s);
// and over the 4-bit cache, one per (field, 128 or 256 rows, split), after ranges4_launch
int ranges4_bytes(bool bf16);  // of a block, at most
int units4_bytes();
hipError_t ranges4_launch(const AttendArgs &a, bool bf16, hipStream_t s);
hipError_t tile4_launch(const AttendArgs &a, bool bf16, hipStream_t s);
hipError_t merge_launch(const AttendArgs &a, bool bf16, hipStream_t s);
// block weights from the attention's block sums, of few rows and of many
hipError_t mass_finish_launch(const AttendArgs &a, hipStream_t s);
hipError_t mass_rows_launch(const AttendArgs &a, hipStream_t s);

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
// c: the centre times -2^-9, in both halves.
constexpr uint32_t kMiddle = 0xb400b400u;  // 128
__device__ __forceinline__ uint32_t centred(uint32_t w, uint32_t c) {
  const h2_t up = {(_Float16)32768.0f, (_Float16)32768.0f};
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(h2_t, w), up, __builtin_bit_cast(h2_t, c)));
}
constexpr float kCodeUnit = 16777216.0f;  // 2^24: codes as they are
constexpr float kCentredUnit = 512.0f;    // 2^9: centred codes

// fp32 storage: a block's codes less the one nearest to the value 0, so that products are
// with the values themselves.  Around the middle of a range that lies to one side of 0 the
// two terms of a score or an output nearly cancel, and the larger one's rounding stays:
// equal weights over 58 values of ranges around 0 were off by 2.5e-6, by fp32 products
// 0.25e-6.  The differences, at most 255, have 9 bits.
struct Centre {
  float mid;   // the value of the centre: half a step from 0, or the end of the range
  uint32_t c;
};
__device__ __forceinline__ Centre centre_of(float2 m) {  // of a (minimum, step), whatever they are: 0 .. 255
  const float z = fminf(fmaxf(rintf(-m.x * __builtin_amdgcn_rcpf(m.y)), 0.0f), 255.0f);
  return Centre{__builtin_fmaf(z, m.y, m.x), pack_f16x2(z * -0x1p-9f, z * -0x1p-9f)};
}

// 8 consecutive codes (two dwords) as fp16 subnormals, CENTRED: less a centre
template <bool CENTRED>
__device__ __forceinline__ h8_t codes8(uint32_t a, uint32_t b, uint32_t c = kMiddle) {
  if constexpr (CENTRED)
    return as_h8(centred(bytes2<0>(a), c), centred(bytes2<2>(a), c), centred(bytes2<0>(b), c), centred(bytes2<2>(b), c));
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
  const uint32_t a = __float_as_uint(v);
  const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const uint32_t b = __float_as_uint(__uint_as_float(x[0]) + __uint_as_float(x[1]));
  const auto y = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __uint_as_float(y[0]) + __uint_as_float(y[1]);
}
__device__ __forceinline__ float row_max(float v) {
  const uint32_t a = __float_as_uint(v);
  const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const uint32_t b = __float_as_uint(fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])));
  const auto y = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
}

// sum / maximum over a wave's 64 lanes, without LDS
template <int N>
__device__ __forceinline__ float ror16(float v) {  // from the lane N further round in its 16
  return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), 0x120 + N, 0xf, 0xf, false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += ror16<8>(v);
  v += ror16<4>(v);
  v += ror16<2>(v);
  v += ror16<1>(v);
  return row_sum(v);
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, ror16<8>(v));
  v = fmaxf(v, ror16<4>(v));
  v = fmaxf(v, ror16<2>(v));
  v = fmaxf(v, ror16<1>(v));
  return row_max(v);
}

// a sequence's length and the position of the first of these queries, loaded once
struct Sequence {
  int len;
  int64_t start;
};
// from what the arrays hold (anything where there is none)
__device__ __forceinline__ Sequence sequence_of(const AttendArgs &a, int32_t n, int32_t p) {
  Sequence s;
  s.len = a.lengths ? (int)min(max((int64_t)n, (int64_t)0), a.tokens) : (int)a.tokens;
  s.start = (a.starts ? (int64_t)p : (int64_t)s.len - a.n_all) + a.first;
  return s;
}

__device__ __forceinline__ Sequence load_sequence(const AttendArgs &a, int b) {
  // both loads at once, from a place that is there where an array is not
  const int32_t *any = (const int32_t *)a.q;
  const int32_t n = *(a.lengths ? a.lengths + b : any), p = *(a.starts ? a.starts + b : any);
  return sequence_of(a, n, p);
}

// Few rows of sequences of unlike lengths: `slots` workgroups a head and row tile are
// dealt to the sequences by their lengths, a sequence of u units has max(ceil(u / t),
// 1) of them.  t is the first of five growing sizes (at least `least`) with which they
// suffice: ceil(sum u / (slots - k batch / 4)), k = 0 .. 4; with the last, the
// sum of u / t + 1 over the sequences is no more than slots.  Equal lengths take the
// first, a whole number of slots each.  Parts are laid out by slot, [head][slot][rows].
struct Slot {
  int b, first, count;  // sequence (batch: none), its first slot and how many it has
  int32_t n, p;         // what lengths and starts hold for it
};

// the sequence that slot j belongs to; a wave's lanes are the sequences (at most 64,
// with fewer than 2^31 units in all)
__device__ __forceinline__ Slot find_slot(const AttendArgs &a, int j) {
  const int lane = threadIdx.x & 63;
  const bool there = lane < a.batch;
  const int32_t len = there ? a.lengths[lane] : 0, start = there && a.starts ? a.starts[lane] : 0;
  const uint32_t u = there ? (uint32_t)((min(max((int64_t)len, (int64_t)0), a.tokens) + UNIT - 1) / UNIT) : 0u;
  const uint32_t sum = (uint32_t)__builtin_amdgcn_readlane(cgw::wave_scan((int)u), 63);
  int n, end;
  for (int k = 0; k < 5; k++) {
    const uint32_t shares = (uint32_t)(a.slots - k * a.batch / 4);
    const uint32_t t = max((sum + (shares - 1)) / shares, (uint32_t)a.least);
    n = there ? max((int)((u + t - 1) / t), 1) : 0;
    end = cgw::wave_scan(n);  // slots up to this sequence's last
    if (__builtin_amdgcn_readlane(end, 63) <= a.slots) break;
  }
  const int l = __popcll(__ballot(end <= j));
  if (l >= a.batch) return Slot{a.batch, 0, 0, 0, 0};
  const int count = __builtin_amdgcn_readlane(n, l);
  return Slot{l, __builtin_amdgcn_readlane(end, l) - count, count, __builtin_amdgcn_readlane(len, l),
              __builtin_amdgcn_readlane(start, l)};
}

// tokens query i sees: none unless it stands inside the sequence
__device__ __forceinline__ int query_limit(const AttendArgs &a, const Sequence &q, int i) {
  const int64_t pos = q.start + i;
  if (pos < 0 || pos >= q.len) return 0;
  return a.causal ? (int)pos + 1 : q.len;
}

// first unit of part `part` of `parts` nearly equal ones
__device__ __forceinline__ int split_begin(int units, int part, int parts) {
  const int each = (int)((uint32_t)units / (uint32_t)parts), more = units - each * parts;
  return each * part + min(part, more);
}

// the largest limit of queries [i0, i1]
__device__ __forceinline__ int limit_of(const AttendArgs &a, const Sequence &q, int i0, int i1) {
  const int64_t lo = max(q.start + i0, (int64_t)0), hi = min(q.start + i1, (int64_t)q.len - 1);
  if (lo > hi) return 0;
  return a.causal ? (int)hi + 1 : q.len;
}

// this thread's 8 channels of one of the query rows [r0, r0 + 16) of (b, h) as
// fp32, four waves to the 16; rows past the last one are zero
struct RowPart {
  f4_t lo, hi;
};

template <bool BF16>
__device__ __forceinline__ RowPart load_row_part(const AttendArgs &a, int b, int h, int r0) {
  const int r = r0 + ((threadIdx.x >> 4) & 15), c = (threadIdx.x & 15) * 8;
  RowPart p;
  p.lo = p.hi = f4_t{0.f, 0.f, 0.f, 0.f};
  if (r < a.rows) {
    const int i = (int)((uint32_t)r / (uint32_t)a.ratio), j = r - i * a.ratio;
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
  float *d = xs + ((threadIdx.x >> 4) & 15) * PITCH + (threadIdx.x & 15) * 8;
  *(f4_t *)d = p.lo;
  *(f4_t *)(d + 4) = p.hi;
}

// y = G x (INV: G^T x) for 16-row tiles in LDS, on the matrix cores: an fp32
// 16x16x4 product adds its four terms as fused multiply-adds, so the result is
// a chain of them over a group's channels (groups of 8 run as 16 with zeros).
// Wave w owns channels 32 w .. + 31; the weights are loaded apart from their
// use, beside other loads.  On the vector units the same for four rows and
// groups of 16 took 2000 cycles, most of it waiting.
struct GaugeFrag {
  f4_t b[2][2];  // output block nb, terms 16 (s0 + s) + 4 (lane / 16) + 0 .. 3 for channel lane % 16
};

template <bool INV>
__device__ __forceinline__ void load_gauge(const float *__restrict__ gh, int g, int s0, GaugeFrag &f) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3;
  const int lane = threadIdx.x & 63, kr = lane >> 4, n = lane & 15;
  const int ge = max(g, 16);
  if (g == 0) return;
#pragma unroll
  for (int s = 0; s < 2; s++) {
    if (16 * (s0 + s) < ge) {
#pragma unroll
      for (int nb = 0; nb < 2; nb++) {
        const int col = 32 * wave + 16 * nb + n, base = col & ~(ge - 1);  // sizes are powers of two
        const int c = col & (g - 1), k = base + 16 * (s0 + s) + 4 * kr, kk = k & (g - 1);
        const float *gp = gh + (int64_t)(col - c) * g;
        f4_t w;
        if constexpr (INV) {
#pragma unroll
          for (int e = 0; e < 4; e++) w[e] = gp[(kk + e) * g + c];
        } else {
          w = f4_t{gp[c * g + kk], gp[c * g + kk + 1], gp[c * g + kk + 2], gp[c * g + kk + 3]};
        }
        f.b[nb][s] = g >= 16 || (k ^ col) < 8 ? w : f4_t{0.f, 0.f, 0.f, 0.f};
      }
    }
  }
}

// tiles [0, T) of xs -> ys, both [16 T][PITCH]; first: load_gauge's for s0 = 0.
// IN_PLACE: the workgroup meets between the reads and the writes (ys == xs).
// The caller's barriers stand before and after.
template <bool INV, int T, bool IN_PLACE>
__device__ __forceinline__ void gauge_tiles(const float *xs, float *ys, const float *__restrict__ gh, int g,
                                            const GaugeFrag &first) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3;
  const int lane = threadIdx.x & 63, kr = lane >> 4, n = lane & 15;
  const int ge = max(g, 16);
  f4_t acc[T][2];
#pragma unroll
  for (int t = 0; t < T; t++) acc[t][0] = acc[t][1] = f4_t{0.f, 0.f, 0.f, 0.f};
  GaugeFrag f = first, nx = first;
#pragma unroll 1
  for (int s0 = 0; 16 * s0 < ge; s0 += 2) {
    if (16 * (s0 + 2) < ge) load_gauge<INV>(gh, g, s0 + 2, nx);
#pragma unroll
    for (int s = 0; s < 2; s++) {
      if (16 * (s0 + s) < ge) {
#pragma unroll
        for (int t = 0; t < T; t++) {
          const float *row = xs + (16 * t + n) * PITCH + 16 * (s0 + s) + 4 * kr;
#pragma unroll
          for (int nb = 0; nb < 2; nb++) {
            const f4_t x = *(const f4_t *)(row + ((32 * wave + 16 * nb) & ~(ge - 1)));
#pragma unroll
            for (int e = 0; e < 4; e++)
              acc[t][nb] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], f.b[nb][s][e], acc[t][nb], 0, 0, 0);
          }
        }
      }
    }
    f = nx;
  }
  if (IN_PLACE) __syncthreads();
#pragma unroll
  for (int t = 0; t < T; t++)
#pragma unroll
    for (int nb = 0; nb < 2; nb++)
#pragma unroll
      for (int j = 0; j < 4; j++) ys[(16 * t + 4 * kr + j) * PITCH + 32 * wave + 16 * nb + n] = acc[t][nb][j];
}

// power-of-two factor that puts a row's largest magnitude into [2^13, 2^14), and back
struct FragScale {
  float up, un;
};
__device__ __forceinline__ FragScale frag_scale(float mx) {
  const int ex = mx > 0.0f ? (int)(__float_as_uint(mx) >> 23) - 127 : 0;
  const int sh = min(13 - ex, 126);  // -115 (an infinity) at least; both factors are normal numbers
  return FragScale{__uint_as_float((uint32_t)(127 + sh) << 23), __uint_as_float((uint32_t)(127 - sh) << 23)};
}

// 8 channels u, v of a row as fp16 operands, their sum added to `sum`.  TWO: two
// parts as above; else one, each channel rounded to 2^-11.
template <bool TWO>
__device__ __forceinline__ void frag_parts(f4_t u, f4_t v, float up, h8_t &hi, h8_t &lo, float &sum) {
  constexpr float H = 1.5f * 67108864.0f;  // x + H - H rounds to multiples of 2^3
  uint32_t wh[4], wl[4];
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const float x = (k < 2 ? u[2 * k] : v[2 * k - 4]) * up, y = (k < 2 ? u[2 * k + 1] : v[2 * k - 3]) * up;
    if constexpr (TWO) {
      const float xh = (x + H) - H, yh = (y + H) - H;
      wh[k] = pack_f16x2(xh, yh);  // exact
      wl[k] = pack_f16x2(x - xh, y - yh);
      const f2_t l = unpack_f16x2(wl[k]);
      sum += (xh + l.x) + (yh + l.y);
    } else {
      wh[k] = pack_f16x2(x, y);
      wl[k] = 0u;
      const f2_t h = unpack_f16x2(wh[k]);
      sum += h.x + h.y;
    }
  }
  hi = as_h8(wh[0], wh[1], wh[2], wh[3]);
  lo = as_h8(wl[0], wl[1], wl[2], wl[3]);
}

// The fp16 operands, step s, of 16 gauged rows xs [16][PITCH]: lane (row = lane %
// 16, grp = lane / 16) holds channels 64 (s / 2) + 16 grp + 8 (s % 2) + 0 .. 7 of its
// row, the order in which 16-byte loads of key codes arrive.  cq is this step's
// part of the minimum's factor.
struct QueryFrags {
  h8_t hi[4], lo[4];
  float ca, cq;  // score = (sum of q' code) step ca + minimum cq
};

__device__ __forceinline__ void make_frags(const float *xs, float c, int s, h8_t &hi, h8_t &lo, float &ca, float &cq) {
  const int lane = threadIdx.x & 63, row = lane & 15, grp = lane >> 4;
  const float *rp = xs + row * PITCH;
  float mx = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; k++) {  // the row's largest magnitude, a quarter of the row to a lane
    const f4_t u = *(const f4_t *)(rp + 32 * grp + 4 * k);
    mx = fmaxf(fmaxf(mx, fabsf(u[0])), fmaxf(fabsf(u[1]), fmaxf(fabsf(u[2]), fabsf(u[3]))));
  }
  const FragScale sc = frag_scale(row_max(mx));
  const float *p = rp + 64 * (s >> 1) + 16 * grp + 8 * (s & 1);
  float sum = 0.0f;
  frag_parts<true>(*(const f4_t *)p, *(const f4_t *)(p + 4), sc.up, hi, lo, sum);
  ca = c * sc.un;
  cq = ca * row_sum(sum);
}

// one output element (b, query row r of head h, channel c)
template <bool BF16>
__device__ __forceinline__ void store_out(const AttendArgs &a, int b, int h, int r, int c, float v) {
  const int i = r / a.ratio, j = r - i * a.ratio;
  const int64_t off = (((int64_t)b * a.n_all + i) * a.heads * a.ratio + h * a.ratio + j) * D + c;
  if (BF16) ((uint16_t *)a.out)[off] = (uint16_t)cgk::bf16_rne(v);
  else ((float *)a.out)[off] = v;
}

// rows [r0, r0 + nr) of (b, h) from LDS [][PITCH], 16 bytes (8 values) a thread
template <bool BF16, int NT = NTH>
__device__ __forceinline__ void store_rows(const AttendArgs &a, int b, int h, int r0, int nr, const float *ys) {
  for (int x = threadIdx.x; x < nr * 16; x += NT) {
    const int r = r0 + (x >> 4), c = 8 * (x & 15);
    const float *y = ys + (x >> 4) * PITCH + c;
    const f4_t lo = *(const f4_t *)y, hi = *(const f4_t *)(y + 4);
    const int i = (int)((uint32_t)r / (uint32_t)a.ratio), j = r - i * a.ratio;
    const int64_t off = (((int64_t)b * a.n_all + i) * a.heads * a.ratio + h * a.ratio + j) * D + c;
    if (BF16) {
      *(uint4 *)((uint16_t *)a.out + off) = make_uint4(cgk::pack_bf16x2(lo[0], lo[1]), cgk::pack_bf16x2(lo[2], lo[3]),
                                                       cgk::pack_bf16x2(hi[0], hi[1]), cgk::pack_bf16x2(hi[2], hi[3]));
    } else {
      *(f4_t *)((float *)a.out + off) = lo;
      *(f4_t *)((float *)a.out + off + 4) = hi;
    }
  }
}

__device__ __forceinline__ void store_lse(const AttendArgs &a, int b, int h, int r, float m, float l) {
  const int i = r / a.ratio, j = r - i * a.ratio;
  // natural logarithm of the row's sum of exp(score); a NaN stays one
  a.lse[((int64_t)b * a.n_all + i) * a.heads * a.ratio + h * a.ratio + j] =
      l != 0.0f ? (m + __builtin_log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace cga
