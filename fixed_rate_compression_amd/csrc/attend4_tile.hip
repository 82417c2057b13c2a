// Attention of many query rows over the 4-bit cache: prompts, chunks of them and drafted
// tokens.  The walk is that of the 8-bit cache's form (attend_tile.hip): 32 rows to
// a wave, 32 tokens a turn laid in LDS as fp16 for all waves, scores and weights of the
// next unit beside the value product of the present one.
//
// Keys and values are widened to what they stand for, since their ranges differ along the
// contraction (keys: by channel) or along both axes (values): two packed fp16
// multiply-adds a pair of codes, once for all rows, or in fp32 and in two parts (keys where
// log-sums or weights are asked for, both for fp32 storage).  A power of two brings a unit's
// largest value to [2^8, 2^9), so that halves keep 2^-33 of it.  That and the ranges in the
// form in which they are used come from a launch before (k_ranges4): the vector units bound
// this kernel, and forming them at every use took 64 of its 235 vector instructions a wave and unit.
//
// 2048 queries over 8192 tokens, 8 KV heads, four query heads each: 292 us, 825 TFLOP/s (a library product of 8192^3
// 1221 in fp16): matrix cores 38 % of the cycles, vector instructions 41 %, hardly at once.  With log-sums, keys and
// queries in two parts, 501; fp32 storage 701.
#include <type_traits>

#include "attend.hpp"
#include "attend4.hpp"
#include "attend_tile.hpp"

namespace cga {

typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

constexpr int kTop = 9;        // widened keys and values are below 2^9

// LDS of a workgroup's token loop; two parts of the keys (P2), of the values (V2)
template <bool P2, bool V2, int NW>
struct Lds4 {
  static constexpr int K = 0, KLO = 2 * KBYTES, V = KLO + (P2 ? 2 * KBYTES : 0), VLO = V + 3 * VBYTES;
  static constexpr int QLO = VLO + (V2 ? 3 * VBYTES : 0), LOOP = QLO + (P2 ? NW * 8192 : 0);
  static constexpr int END = NW * WROWS * PITCH * 4, SIZE = LOOP > END ? LOOP : END;
};

// What the tiles need of a block's ranges, formed once for all of them (k_ranges4): powers of
// two that keys and values are below, value ranges that are not numbers (bit 4 token + group, of the first and
// the last 16 tokens), and the ranges themselves, scaled, as they are used.  Keys in one part: for 8
// channels the steps times 2^9, then the centres, as halves in the order of centred8; in two parts:
// (minimum, step) in fp32.  Values likewise, a pair a token and group.
struct Unit4 {
  int ek, ev;
  uint32_t bad;  // whether there is such a range
  uint64_t bad0, bad1;
};
template <bool P2, bool V2>
struct Ranges4 {
  static constexpr int K = P2 ? 1024 : 512, V = V2 ? 1024 : 512, BYTES = K + V;
};

// One wave to a block of a sequence's tokens.
template <bool P2, bool V2>
__global__ __launch_bounds__(NTH) void k_ranges4(const AttendArgs a, int blocks) {
  using R = Ranges4<P2, V2>;
  const int lane = threadIdx.x & 63;
  const int64_t at = (int64_t)blockIdx.x * (NTH / 64) + (threadIdx.x >> 6);  // (b, h, block)
  const int64_t bh = at / blocks;
  const int blk = (int)(at - bh * blocks);
  if (bh >= (int64_t)a.batch * a.heads) return;
  const Sequence sq = load_sequence(a, (int)(bh / a.heads));
  if (blk * UNIT >= sq.len) return;
  const float2 *km = a.kmeta + (bh * a.tcap + (int64_t)blk * UNIT) * 4, *vm = a.vmeta + (bh * a.tcap + (int64_t)blk * UNIT) * 4;
  const int c0 = 8 * (lane >> 2) + (lane & 3);  // this lane's channels: c0 and c0 + 4
  float2 k[2] = {km[c0], km[c0 + 4]}, v[2] = {vm[lane], vm[lane + 64]};  // values: token, group of entry 4 token + group
  // ranges behind the sequence's end are whatever they are; one that gives a NaN or an infinity for some
  // code (15 steps alone may) counts as zeros and is marked
  uint64_t bad[2];
#pragma unroll
  for (int x = 0; x < 2; x++) {
    const bool there = blk * UNIT + 16 * x + (lane >> 2) < sq.len;
    const bool b = there && max(range_bits(v[x]), __float_as_uint(v[x].y) & 0x7fffffffu) >= INF;
    bad[x] = __ballot(b);
    if (!there || b) v[x] = make_float2(0.f, 0.f);
  }
  const int ek = exponent_of(wave_umax(max(range_bits(k[0]), range_bits(k[1]))));
  const int ev = exponent_of(wave_umax(max(range_bits(v[0]), range_bits(v[1]))));
  if (lane == 0) ((Unit4 *)a.units)[at] = Unit4{ek, ev, bad[0] | bad[1] ? 1u : 0u, bad[0], bad[1]};
  uint8_t *o = a.ranges + at * R::BYTES;
#pragma unroll
  for (int x = 0; x < 2; x++) {
    k[x] = make_float2(__builtin_ldexpf(k[x].x, kTop - ek), __builtin_ldexpf(k[x].y, kTop - ek));
    v[x] = make_float2(__builtin_ldexpf(v[x].x, kTop - ev), __builtin_ldexpf(v[x].y, kTop - ev));
  }
  if constexpr (P2) {
    ((float2 *)o)[c0] = k[0];
    ((float2 *)o)[c0 + 4] = k[1];
  } else {
    uint32_t *p = (uint32_t *)(o + 32 * (lane >> 2)) + (lane & 3);
    p[0] = pack_f16x2(512.0f * k[0].y, 512.0f * k[1].y);  // 35000 at most
    p[4] = pack_f16x2(__builtin_fmaf(8.0f, k[0].y, k[0].x), __builtin_fmaf(8.0f, k[1].y, k[1].x));
  }
#pragma unroll
  for (int x = 0; x < 2; x++) {
    if constexpr (V2) ((float2 *)(o + R::K))[lane + 64 * x] = v[x];
    else ((uint32_t *)(o + R::K))[lane + 64 * x] = pack_f16x2(512.0f * v[x].y, __builtin_fmaf(8.0f, v[x].y, v[x].x));
  }
}

// A unit's codes and ranges on their way: N = 16 or 8 values of the keys and of the values to a thread.
// Keys: channels 8 (i % 16) .. + 7 of tokens i / 16, + 16; values: N channels of a token.
template <bool P2, bool V2, int N>
struct Regs4 {
  uint32_t k[N / 8], v[N / 8];
  u4_t mk[P2 ? 4 : 2];
  uint32_t mv[V2 ? 2 : 1];
};

struct Place4 {
  const uint8_t *kf, *vf, *ranges;
  const Unit4 *units;
  int last;  // of the blocks that the tokens' bound has
};

template <bool P2, bool V2, int N>
__device__ __forceinline__ void fetch4(const Place4 &p, int un, Regs4<P2, V2, N> &s) {
  using R = Ranges4<P2, V2>;
  const uint32_t i = threadIdx.x;
  const int64_t u = min(un, p.last);
  constexpr uint32_t VT = D / N;  // threads to a token's values
  const uint8_t *kc = p.kf + u * (UNIT * HALF_D), *vc = p.vf + u * (UNIT * HALF_D), *r = p.ranges + u * R::BYTES;
#pragma unroll
  for (uint32_t x = 0; x < N / 8; x++) s.k[x] = *(const uint32_t *)(kc + ((i >> 4) * HALF_D + 4 * (i & 15)) + x * 16 * HALF_D);
#pragma unroll
  for (uint32_t x = 0; x < N / 8; x++) s.v[x] = *(const uint32_t *)(vc + ((i / VT) * HALF_D + N / 2 * (i % VT)) + 4 * x);
#pragma unroll
  for (uint32_t x = 0; x < (P2 ? 4 : 2); x++) s.mk[x] = *(const u4_t *)(r + (P2 ? 64 : 32) * (i & 15) + 16 * x);
  const uint32_t *mv = (const uint32_t *)(r + R::K + (V2 ? 8 : 4) * ((i / VT) * 4 + N * (i % VT) / 32));
#pragma unroll
  for (int x = 0; x < (V2 ? 2 : 1); x++) s.mv[x] = mv[x];
}

// Eight codes as halves, less 8 and times 2^-9: pairs (0, 4), (1, 5), (2, 6), (3, 7).  The low ones of
// a byte's are multiples of 2^-24 as they stand, the high ones of 2^-20.
__device__ __forceinline__ void centred8(uint32_t w, h2_t (&c)[4]) {
  const h2_t up = {(_Float16)32768.0f, (_Float16)32768.0f}, up16 = {(_Float16)2048.0f, (_Float16)2048.0f};
  const h2_t mid = {(_Float16)-0x1p-6f, (_Float16)-0x1p-6f};
  const uint32_t x = w >> 8;
  c[0] = __builtin_elementwise_fma(__builtin_bit_cast(h2_t, w & 0x000f000fu), up, mid);
  c[1] = __builtin_elementwise_fma(__builtin_bit_cast(h2_t, w & 0x00f000f0u), up16, mid);
  c[2] = __builtin_elementwise_fma(__builtin_bit_cast(h2_t, x & 0x000f000fu), up, mid);
  c[3] = __builtin_elementwise_fma(__builtin_bit_cast(h2_t, x & 0x00f000f0u), up16, mid);
}

__device__ __forceinline__ h2_t pack2(float a, float b) {
  const f2_t v = {a, b};
  return __builtin_convertvector(v, h2_t);
}

// the values themselves, in the order of centred8, from a step (times 2^9) and a centre a pair
__device__ __forceinline__ void put_centred(unsigned char *p, uint32_t w, const h2_t (&st)[4], const h2_t (&mid)[4]) {
  h2_t c[4];
  centred8(w, c);
#pragma unroll
  for (int k = 0; k < 4; k++) c[k] = __builtin_elementwise_fma(c[k], st[k], mid[k]);
  *(h8_t *)p = as_h8(__builtin_bit_cast(uint32_t, c[0]), __builtin_bit_cast(uint32_t, c[1]), __builtin_bit_cast(uint32_t, c[2]),
                     __builtin_bit_cast(uint32_t, c[3]));
}

// in two parts, formed in fp32, in the order of the channels
__device__ __forceinline__ void put_two(unsigned char *p, int lo, uint32_t w, const float (&st)[8], const float (&m)[8]) {
  const uint32_t e = w & 0x0f0f0f0fu, o = (w >> 4) & 0x0f0f0f0fu;
  uint32_t h[4], l[4];
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const float x = __builtin_fmaf((float)((e >> 8 * k) & 0xffu), st[2 * k], m[2 * k]);
    const float y = __builtin_fmaf((float)((o >> 8 * k) & 0xffu), st[2 * k + 1], m[2 * k + 1]);
    h[k] = pack_f16x2(x, y);
    const f2_t hh = unpack_f16x2(h[k]);
    l[k] = pack_f16x2(x - hh.x, y - hh.y);
  }
  *(h8_t *)p = as_h8(h[0], h[1], h[2], h[3]);
  *(h8_t *)(p + lo) = as_h8(l[0], l[1], l[2], l[3]);
}

// A unit into LDS in steps, to be taken between matrix instructions
template <typename L, bool P2, bool V2, int N>
struct Put4 {
  static constexpr int VT = D / N;
  const Regs4<P2, V2, N> &s;
  unsigned char *k, *v;

  __device__ __forceinline__ Put4(unsigned char *lds, int un, const Regs4<P2, V2, N> &regs) : s(regs) {
    const int i = threadIdx.x;
    k = lds + L::K + (un & 1) * KBYTES + (i >> 4) * KP + 16 * (i & 15);
    v = lds + L::V + (un % 3) * VBYTES + (i / VT) * VP + 2 * N * (i % VT);
  }
  template <int S>
  __device__ __forceinline__ void step() {
    if constexpr (S < N / 8) {
      if constexpr (P2) {
        float m[8], st[8];
#pragma unroll
        for (int c = 0; c < 8; c++) {
          m[c] = __uint_as_float(s.mk[c >> 1][2 * (c & 1)]);
          st[c] = __uint_as_float(s.mk[c >> 1][2 * (c & 1) + 1]);
        }
        put_two(k + 16 * S * KP, L::KLO - L::K, s.k[S], st, m);
      } else {
        h2_t hs[4], hm[4];
#pragma unroll
        for (int x = 0; x < 4; x++) {
          const uint32_t a = s.mk[0][x], c = s.mk[1][x];  // (a bit cast of a vector's element takes its first)
          hs[x] = __builtin_bit_cast(h2_t, a);
          hm[x] = __builtin_bit_cast(h2_t, c);
        }
        put_centred(k + 16 * S * KP, s.k[S], hs, hm);
      }
    } else if constexpr (S < N / 4) {
      constexpr int T = S - N / 8;
      if constexpr (V2) {
        float ms[8], sts[8];
#pragma unroll
        for (int c = 0; c < 8; c++) {
          ms[c] = __uint_as_float(s.mv[0]);
          sts[c] = __uint_as_float(s.mv[1]);
        }
        put_two(v + 16 * T, L::VLO - L::V, s.v[T], sts, ms);
      } else {
        const h2_t m = __builtin_bit_cast(h2_t, s.mv[0]);
        const h2_t st = {m.x, m.x}, mid = {m.y, m.y};
        const h2_t hs[4] = {st, st, st, st}, hm[4] = {mid, mid, mid, mid};
        put_centred(v + 16 * T, s.v[T], hs, hm);
      }
    }
  }
  __device__ __forceinline__ void all() {
    step<0>();
    step<1>();
    step<2>();
    step<3>();
  }
};

// a lane's row (the same in lanes l and l + 32 but for l), as in attend_tile.hip; mu is -inf while the
// row has seen nothing, f the log2 of the factor to the values' power of two
struct State4 {
  float m, mu, mo, f, l;
  uint32_t poison;  // groups of channels of which the row has seen a value that is not a number
};

struct Queries4 {
  h8_t hi[8];
  float ca;
};

template <bool TWO>
__device__ __forceinline__ void tile_queries4(const float *xs, float c, Queries4 &q, h8_t (&lo)[8]) {
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const float *rp = xs + (lane & 31) * PITCH + 8 * half;
  f4_t x[16];
  float mx = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; k++) {
    x[k] = *(const f4_t *)(rp + 16 * (k >> 1) + 4 * (k & 1));
    mx = fmaxf(fmaxf(mx, fmaxf(fabsf(x[k][0]), fabsf(x[k][1]))), fmaxf(fabsf(x[k][2]), fabsf(x[k][3])));
  }
  mx = fmaxf(mx, __shfl_xor(mx, 32));
  const FragScale sc = frag_scale(mx);
#pragma unroll
  for (int s = 0; s < 8; s++) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      // one part: in the order of centred8
      const float u = (TWO ? x[2 * s + (k >> 1)][2 * (k & 1)] : x[2 * s][k]) * sc.up;
      const float v = (TWO ? x[2 * s + (k >> 1)][2 * (k & 1) + 1] : x[2 * s + 1][k]) * sc.up;
      h[k] = pack_f16x2(u, v);
      if constexpr (TWO) {
        const f2_t hh = unpack_f16x2(h[k]);
        l[k] = pack_f16x2(u - hh.x, v - hh.y);
      }
    }
    q.hi[s] = as_h8(h[0], h[1], h[2], h[3]);
    if constexpr (TWO) lo[s] = as_h8(l[0], l[1], l[2], l[3]);
  }
  q.ca = __builtin_fmaf(mx, 0.0f, c * sc.un);  // an infinity: NaN for the row
}

// scores of a unit: z = K Q^T, z[r] that of token 8 (r / 4) + 4 half + r % 4
template <bool P2>
__device__ __forceinline__ void scores4(const unsigned char *kb, int klo, const Queries4 &q, const unsigned char *lo, f16_t &z) {
  f16_t zl;
#pragma unroll
  for (int r = 0; r < 16; r++) z[r] = zl[r] = 0.0f;
#pragma unroll
  for (int s = 0; s < 8; s++) {
    const h8_t c = *(const h8_t *)(kb + 32 * s);
    z = mfma32(c, q.hi[s], z);
    if constexpr (P2) {
      zl = mfma32(c, *(const h8_t *)(lo + 1024 * s), zl);
      zl = mfma32(*(const h8_t *)(kb + klo + 32 * s), q.hi[s], zl);
    }
  }
  if constexpr (P2) z += zl;
}

// a unit's weights (times the values' factor) and the sum of those without it
struct Weights4 {
  float p[16], ps;
};

// raise the row's maximum to the unit's scores, rescale what was summed, and form the
// unit's weights again (rare: the scores are not kept for it)
template <bool P2>
__device__ __forceinline__ void raise4(const unsigned char *kb, int klo, const unsigned char *lo, float A, float lv,
                                       const Queries4 &q, int vis, State4 &st, f16_t (&acc)[4], Weights4 &o) {
  f16_t z;
  uint32_t again = 0;  // unknown to the compiler: the operands of the rare second product are not kept for it
  asm volatile("" : "+v"(again));
  scores4<P2>(kb + again, klo, q, lo + again, z);
  float mx = -INFINITY;
#pragma unroll
  for (int r = 0; r < 16; r++) {
    o.p[r] = 8 * (r >> 2) + (r & 3) < vis ? z[r] * A : -INFINITY;
    mx = fmaxf(mx, o.p[r]);
  }
  const float tm = pair_max(mx), mn = fmaxf(st.m, tm);
  float on = fmaxf(st.mo, tm + lv);
  const bool some = mn > -INFINITY;
  if (some) on = fmaxf(on, mn - 126.0f);  // keeps 2^(mo - m) a normal number beside weights that vanish
  const float al = st.m > -INFINITY ? exp2_fast(st.m - mn) : 0.0f;
  const float ao = st.mo > -INFINITY ? exp2_fast(st.mo - on) : 0.0f;
  st.l *= al;
#pragma unroll
  for (int j = 0; j < 4; j++) acc[j] *= ao;
  st.m = st.mu = mn;
  st.mo = on;
  st.f = some ? mn - on + 9.0f : 0.0f;
  const float lw = fmaxf(lv + st.f, -60.0f), up = lw - (some ? mn : 0.0f);
#pragma unroll
  for (int r = 0; r < 16; r++) o.p[r] = exp2_fast(o.p[r] + up);
  float sum[1];
  sum_weights<1>(o.p, sum);
  o.ps = sum[0] * exp2_fast(-lw);
}

// acc += V^T P^T of a unit; acc[j][r]: channel 32 j + 8 (r / 4) + 4 half + r % 4
template <bool V2>
__device__ __forceinline__ void values4(const unsigned char *vb, int vlo, const UnitOperands<!V2> &P, f16_t (&acc)[4]) {
#pragma unroll
  for (int x = 0; x < 2; x++)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const auto at = [&](const unsigned char *p) {
        const s4_t a = transposed(p + 16 * x * VP + 64 * j), b = transposed(p + (16 * x + 8) * VP + 64 * j);
        return __builtin_bit_cast(h8_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
      };
      const h8_t vj = at(vb);
      acc[j] = mfma32(vj, P.hi[x], acc[j]);
      if constexpr (V2) {
        acc[j] = mfma32(vj, P.lo[x], acc[j]);
        acc[j] = mfma32(at(vb + vlo), P.hi[x], acc[j]);
      }
    }
}

// P2: keys and queries in two fp16 parts (fp32 storage, or where log-sums or weights are asked
// for), else one each.  SUMS: the rows' sums of every unit are kept.
template <bool BF16, bool P2, bool SUMS, int NW>
__global__ __launch_bounds__(64 * NW, 2) void k_attend4_tile(const AttendArgs a) {
  static_assert(BF16 || P2, "fp32 storage takes both parts");
  constexpr bool V2 = !BF16;
  constexpr int NT = 64 * NW, N = UNIT * D / NT, TROWS = NW * WROWS;
  using L = Lds4<P2, V2, NW>;
  __shared__ __align__(16) unsigned char lds[L::SIZE];
  const int lane = threadIdx.x & 63, row = lane & 31, half = lane >> 5, n = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fields = a.batch * a.heads, groups = (a.rows + TROWS - 1) / TROWS;
  const uint32_t q1 = blockIdx.x / (uint32_t)fields, q2 = q1 / (uint32_t)a.splits;
  const int bh = (int)(blockIdx.x - q1 * fields);  // a head's workgroups share an XCD's L2 where the heads are a multiple of 8
  const int split = (int)(q1 - q2 * a.splits);
  // the longest first; where all are resident at once the second half runs from the
  // shortest up, beside the first half's longest
  const int turn_of = (int)q2, first = (groups + 1) / 2;
  const bool paired = (int64_t)gridDim.x <= 2048 / NW && a.splits == 1;
  const int grpi = paired && turn_of >= first ? turn_of - first : groups - 1 - turn_of;
  const int h = bh % a.heads, b = bh / a.heads;
  const int r0 = grpi * TROWS, nr = min(TROWS, a.rows - r0);
  const Sequence sq = load_sequence(a, b);
  const int blocks = (int)((a.tokens + UNIT - 1) / UNIT);
  const Place4 place{a.kpay + (int64_t)bh * a.tcap * HALF_D, a.vpay + (int64_t)bh * a.tcap * HALF_D,
                     a.ranges + (int64_t)bh * blocks * Ranges4<P2, V2>::BYTES, (const Unit4 *)a.units + (int64_t)bh * blocks,
                     blocks - 1};
  const int tmax = limit_of(a, sq, r0 / a.ratio, (r0 + nr - 1) / a.ratio);
  const int units = (tmax + UNIT - 1) / UNIT;
  const int u0 = split_begin(units, split, a.splits), u1 = split_begin(units, split + 1, a.splits);
  // codes on their way, of units at even and odd distance from the first (with two parts, whose
  // operands take registers, of one)
  constexpr int SETS = P2 ? 1 : 2;
  using In = Regs4<P2, V2, N>;
  In nx[SETS];
  if (u0 < u1)
#pragma unroll
    for (int x = 0; x < SETS; x++) fetch4(place, u0 + x, nx[x]);

  // gauged queries as operands
  Queries4 q;
  unsigned char *const lo = lds + L::QLO + wave * 8192 + lane * 16;
  const int wr = r0 + wave * WROWS + row;  // the lane's row
  {
    float *xs = (float *)lds + (wave >> 2) * 128 * PITCH;  // of four waves
    const float *gk = a.gk + (int64_t)h * D * a.g;
    GaugeFrag gw;
    load_gauge<false>(gk, a.g, 0, gw);
    RowPart p[8];
#pragma unroll
    for (int t = 0; t < 8; t++) p[t] = load_row_part<BF16>(a, b, h, r0 + (wave >> 2) * 128 + t * ROWS);
#pragma unroll
    for (int t = 0; t < 8; t++) put_row_part(xs + t * ROWS * PITCH, p[t]);
    __syncthreads();
    if (a.g) {
      gauge_tiles<false, 8, true>(xs, xs, gk, a.g, gw);
      __syncthreads();
    }
    h8_t part[8];
    tile_queries4<P2>((float *)lds + wave * WROWS * PITCH, a.c, q, part);
    __syncthreads();  // the rows have been read
    if constexpr (P2)
#pragma unroll
      for (int s = 0; s < 8; s++) *(h8_t *)(lo + s * 1024) = part[s];
  }
  // A wave without rows widens the units with the others, no more: 68 rows with log-sums 83 us, so 64.
  // In one part, which fewer waves take, the test cost more than it saved (a prompt of 1000 36 us, 40).
  const bool mine = !P2 || wave * WROWS < nr;
  // what the row sees; rows that are not there see everything
  const int lim = wr < a.rows ? query_limit(a, sq, (int)((uint32_t)wr / (uint32_t)a.ratio)) : tmax;
  int all = lim;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) all = min(all, __shfl_xor(all, k));
  all = __builtin_amdgcn_readfirstlane(all);

  State4 st;
  st.m = st.mo = st.mu = -INFINITY;
  st.l = st.f = 0.0f;
  st.poison = 0u;
  f16_t acc[4];
#pragma unroll
  for (int j = 0; j < 4; j++)
#pragma unroll
    for (int r = 0; r < 16; r++) acc[j][r] = 0.0f;
  constexpr int klo = L::KLO - L::K, vlo = L::VLO - L::V;
  const auto keys_at = [&](int un) { return lds + L::K + (un & 1) * KBYTES + row * KP + 16 * half; };
  const auto values_at = [&](int un) {
    return lds + L::V + (un % 3) * VBYTES + (4 * half + (n >> 2)) * VP + 32 * ((lane >> 4) & 1) + 8 * (n & 3);
  };
  // a unit's powers of two, loaded a turn before they are used
  int4 un_head;
  const auto fetch_head = [&](int un) { un_head = *(const int4 *)(place.units + min(un, place.last)); };
  // the row's factor of a unit's scores and the log2 of its values' power of two; marks the rows that see
  // a value that is not a number
  const auto factors = [&](int un, float &A, float &lv) {
    const int4 e = un_head;
    A = __builtin_ldexpf(q.ca, e.x - kTop);
    lv = (float)e.y;
    if (__builtin_amdgcn_readfirstlane(e.z)) {
      const Unit4 *u = place.units + un;
      const int vis = min(max(lim - un * UNIT, 0), UNIT), v0 = min(vis, 16), v1 = vis - v0;
      uint64_t x = (v0 < 16 ? u->bad0 & ((1ull << 4 * v0) - 1) : u->bad0) | (v1 < 16 ? u->bad1 & ((1ull << 4 * v1) - 1) : u->bad1);
#pragma unroll
      for (int k = 32; k >= 4; k >>= 1) x |= x >> k;
      st.poison |= (uint32_t)x & 15u;
    }
  };

  if (u0 < u1) {
    Weights4 o;
    UnitOperands<BF16> P;
    Put4<L, P2, V2, N>(lds, u0, nx[0]).all();
    fetch4(place, u0 + SETS, nx[0]);  // units past the last are fetched (blocks that exist), put and not used
    fetch_head(u0);
    Put4<L, P2, V2, N>(lds, u0 + 1, nx[SETS - 1]).all();
    fetch4(place, u0 + 1 + SETS, nx[SETS - 1]);
    __syncthreads();
    float A, lv;
    factors(u0, A, lv);
    fetch_head(u0 + 1);
    if (mine) raise4<P2>(keys_at(u0), klo, lo, A, lv, q, lim - u0 * UNIT - 4 * half, st, acc, o);
    const auto store_sum = [&](int un) {
      const uint32_t x = __float_as_uint(o.ps);
      const auto y = __builtin_amdgcn_permlane32_swap(x, x, false, false);
      const float v = __uint_as_float(y[0]) + __uint_as_float(y[1]);
      if (half == 0 && wr < a.rows) a.bsum[((int64_t)bh * a.entries + un) * a.rows + wr] = make_float2(v, st.mu);
    };
    if constexpr (SUMS)
      if (mine) store_sum(u0);
    const auto turn = [&](int un, auto masked, In &in) {
      __syncthreads();  // unit un + 1 is there, unit un - 1 is done with
      if (!mine) {
        Put4<L, P2, V2, N>(lds, un + 2, in).all();
        fetch4(place, un + 2 + SETS, in);
        return;
      }
      float A, lv;
      factors(un + 1, A, lv);
      fetch_head(un + 2);
      // One block from here on, in the order in which it is to be issued: a matrix instruction runs
      // for 32 cycles beside what follows it.  The scores' products, with the next unit's
      // widening between them, then the values', with the weights between them.
      const int vis = lim - (un + 1) * UNIT - 4 * half;
      const unsigned char *kb = keys_at(un + 1), *vb = values_at(un);
      Put4<L, P2, V2, N> put(lds, un + 2, in);
      f16_t z, zl;
#pragma unroll
      for (int r = 0; r < 16; r++) z[r] = zl[r] = 0.0f;
      h8_t kc[2] = {*(const h8_t *)kb, *(const h8_t *)(kb + 32)};
      const auto score = [&](auto step) {
        constexpr int S = decltype(step)::value;
        z = mfma32(kc[S & 1], q.hi[S], z);
        if constexpr (P2) {
          zl = mfma32(kc[S & 1], *(const h8_t *)(lo + 1024 * S), zl);
          zl = mfma32(*(const h8_t *)(kb + klo + 32 * S), q.hi[S], zl);
        }
        if constexpr (S < 6) kc[S & 1] = *(const h8_t *)(kb + 32 * (S + 2));
        put.template step<S>();
        if constexpr (S == 4) pack_weights<BF16>(o.p, P);
        if constexpr (S == 5) fetch4(place, un + 2 + SETS, in);
        __builtin_amdgcn_sched_barrier(0);
      };
      score(std::integral_constant<int, 0>{});
      score(std::integral_constant<int, 1>{});
      score(std::integral_constant<int, 2>{});
      score(std::integral_constant<int, 3>{});
      score(std::integral_constant<int, 4>{});
      score(std::integral_constant<int, 5>{});
      score(std::integral_constant<int, 6>{});
      score(std::integral_constant<int, 7>{});
      st.l += o.ps;
      const float lw = fmaxf(lv + st.f, -60.0f), iw = exp2_fast(-lw), B = lw - st.mu;
      const auto at = [&](const unsigned char *p, int x, int j) {
        const s4_t a = transposed(p + 16 * x * VP + 64 * j), b = transposed(p + (16 * x + 8) * VP + 64 * j);
        return __builtin_bit_cast(h8_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
      };
      h8_t vc[2] = {at(vb, 0, 0), at(vb, 0, 1)};
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (P2) z += zl;
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const int x = k >> 2, j = k & 3;
        acc[j] = mfma32(vc[k & 1], P.hi[x], acc[j]);
        if constexpr (V2) {
          acc[j] = mfma32(vc[k & 1], P.lo[x], acc[j]);
          acc[j] = mfma32(at(vb + vlo, x, j), P.hi[x], acc[j]);
        }
        if (k < 6) vc[k & 1] = at(vb, (k + 2) >> 2, (k + 2) & 3);
#pragma unroll
        for (int r = 2 * k; r < 2 * k + 2; r++) {
          const float s = __builtin_fmaf(z[r], A, B);
          o.p[r] = exp2_fast(decltype(masked)::value && 8 * (r >> 2) + (r & 3) >= vis ? -INFINITY : s);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      float sum[1];
      sum_weights<1>(o.p, sum);
      o.ps = sum[0] * iw;
      // some weight is too large for its scale, or infinite: a row that has seen nothing yet
      const bool up = fmaxf(sum[0], o.ps * 128.0f) > 32768.0f;
      if (__any(up)) raise4<P2>(keys_at(un + 1), klo, lo, A, lv, q, vis, st, acc, o);
      if constexpr (SUMS) store_sum(un + 1);
    };
    // units that every row of the wave sees whole, then the others
    const int ua = min(u1 - 1, max(all / UNIT - 1, u0));
    int un = u0;
    for (; un + SETS <= ua; un += SETS) {
      turn(un, std::false_type{}, nx[0]);
      if constexpr (SETS == 2) turn(un + 1, std::false_type{}, nx[1]);
    }
    for (; un + 1 < u1; un += SETS) {
      turn(un, std::true_type{}, nx[0]);
      if constexpr (SETS == 2)
        if (un + 2 < u1) turn(un + 1, std::true_type{}, nx[1]);
    }
    if (mine) {
      st.l += o.ps;
      pack_weights<BF16>(o.p, P);
      values4<V2>(values_at(u1 - 1), vlo, P, acc);
    }
  }
  __syncthreads();

  // rows' sums, scaled as they stand, into LDS; then parts or outputs
  const float *gv = a.gv + (int64_t)h * D * a.g;
  GaugeFrag gw;
  load_gauge<true>(gv, a.g, 0, gw);
  float *us = (float *)lds;
  {
    const int rr = wave * WROWS + row;
    const float Ls = st.l + __shfl_xor(st.l, 32);
    const bool some = st.m > -INFINITY;
    const float inv = a.splits > 1 ? 1.0f : Ls > 0.0f ? 1.0f / Ls : 0.0f;
    const FarSums far(st.m, st.mo);  // one split: divided by the sum of the weights already
    const float less = !far.is || a.splits > 1 ? far.less : far.less - far.shift;
    const float ks = some ? inv * exp2_fast(far.up - less) : 0.0f, kv = far.is ? 1.0f : 0x1p-18f;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const float k = (st.poison >> j) & 1u ? NAN : 0.0f;  // a group of 32 channels
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        f4_t v;
#pragma unroll
        for (int x = 0; x < 4; x++) v[x] = __builtin_fmaf(acc[j][r + x] * kv, ks, k);  // 2^9 of the values, 2^9 of f
        float *o = us + rr * PITCH + 32 * j + 2 * r;
        if constexpr (V2) {
          *(f4_t *)(o + 4 * half) = v;
        } else {  // the order of centred8
          *(float2 *)(o + 2 * half) = make_float2(v[0], v[2]);
          *(float2 *)(o + 2 * half + 4) = make_float2(v[1], v[3]);
        }
      }
    }
    if (half == 0 && rr < nr) {
      if (a.splits > 1) {
        a.part_ml[((int64_t)bh * a.splits + split) * a.rows + wr] = make_float2(st.m + far.shift, far.is ? Ls * 0x1p-32f : Ls);
      } else {
        if (a.lse) store_lse(a, b, h, wr, st.m, Ls);
        if (a.lse2) a.lse2[(int64_t)bh * a.rows + wr] = Ls != 0.0f ? st.m + __builtin_log2f(Ls) : INFINITY;
      }
    }
  }
  __syncthreads();
  if (a.splits > 1) {
    float *po = a.part_o + (((int64_t)bh * a.splits + split) * a.rows + r0) * D;
    for (int i = threadIdx.x; i < nr * (D / 4); i += NT)
      *(float4 *)(po + 4 * (int64_t)i) = *(const float4 *)(us + (i / (D / 4)) * PITCH + 4 * (i % (D / 4)));
    return;
  }
  if (a.g) {
    float *xs = us + (wave >> 2) * 128 * PITCH;
    gauge_tiles<true, 8, true>(xs, xs, gv, a.g, gw);
    __syncthreads();
  }
  store_rows<BF16, NT>(a, b, h, r0, nr, us);
}

int ranges4_bytes(bool bf16) { return bf16 ? Ranges4<true, false>::BYTES : Ranges4<true, true>::BYTES; }
int units4_bytes() { return (int)sizeof(Unit4); }

hipError_t ranges4_launch(const AttendArgs &a, bool bf16, hipStream_t s) {
  const int64_t blocks = (a.tokens + UNIT - 1) / UNIT, all = (int64_t)a.batch * a.heads * blocks;
  if (all == 0) return hipSuccess;
  const dim3 grid((unsigned)((all + NTH / 64 - 1) / (NTH / 64))), block(NTH);
  if (!bf16) hipLaunchKernelGGL((k_ranges4<true, true>), grid, block, 0, s, a, (int)blocks);
  else if (a.two) hipLaunchKernelGGL((k_ranges4<true, false>), grid, block, 0, s, a, (int)blocks);
  else hipLaunchKernelGGL((k_ranges4<false, false>), grid, block, 0, s, a, (int)blocks);
  return hipGetLastError();
}

hipError_t tile4_launch(const AttendArgs &a, bool bf16, hipStream_t s) {
  const bool p2 = a.two, sums = a.bsum != nullptr;
  // Eight waves widen a unit for twice the rows, where that still gives every compute unit a workgroup:
  // 2048 queries over 8192 tokens (256 workgroups) 309 us, by four 316; a prompt of 4000 196 and 209, of
  // 1000 (128 workgroups) 51 and 42; and where there are rows for them: 68 rows a head of 8 sequences of
  // 4096 tokens 57 us, by four 35.  Two parts take most of a compute unit's LDS either way.
  const int64_t wide = (int64_t)a.batch * a.heads * ((a.rows + 255) / 256) * a.splits;
  const int nw = p2 || (wide >= 256 && a.rows > 4 * WROWS) ? 8 : 4;
  const int64_t groups = (a.rows + nw * WROWS - 1) / (nw * WROWS);
  const dim3 grid((unsigned)((int64_t)a.batch * a.heads * groups * a.splits)), block(64 * nw);
#define CG_T(BF, P2, SUMS, NW)                                                             \
  if (bf16 == BF && p2 == P2 && sums == SUMS && nw == NW) {                                \
    hipLaunchKernelGGL((k_attend4_tile<BF, P2, SUMS, NW>), grid, block, 0, s, a);          \
    return hipGetLastError();                                                              \
  }
  CG_T(true, false, false, 4) CG_T(true, false, false, 8)
  CG_T(true, true, false, 8) CG_T(true, true, true, 8) CG_T(false, true, false, 8) CG_T(false, true, true, 8)
#undef CG_T
  return hipErrorInvalidValue;
}

}  // namespace cga
