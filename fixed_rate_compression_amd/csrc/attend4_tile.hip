// Attention of many query rows over the 4-bit cache: prompts, chunks of them and drafted
// tokens.  The walk is that of the 8-bit cache's form (attend_tile.hip): 32 rows to
// a wave, 32 tokens a turn laid in LDS as fp16 for all waves, scores and weights of the
// next unit beside the value product of the present one.
//
// Keys and values are widened to what they stand for, since their ranges differ along the
// contraction (keys: by channel) or along both axes (values): two packed fp16
// multiply-adds a pair of codes, once for all rows, or in fp32 and in two parts (keys where
// log-sums or weights are asked for, both for fp32 storage).  Where a unit's values leave
// fp16's range a power of two brings them back; the units' largest magnitudes are found
// from their ranges every fourth turn, a unit to a wave, four to seven turns ahead.
#include <type_traits>

#include "attend.hpp"
#include "attend_tile.hpp"

namespace cga {

typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

constexpr int HALF_D = D / 2;  // bytes of a row of codes
constexpr int kTop = 9;        // widened keys and values are below 2^9

// LDS of a workgroup's token loop; two parts of the keys (P2), of the values (V2)
template <bool P2, bool V2, int NW>
struct Lds4 {
  static constexpr int K = 0, KLO = 2 * KBYTES, V = KLO + (P2 ? 2 * KBYTES : 0), VLO = V + 3 * VBYTES;
  static constexpr int TOPS = VLO + (V2 ? 3 * VBYTES : 0);  // [8]: Unit4 of units that come
  static constexpr int QLO = TOPS + 8 * 32, LOOP = QLO + (P2 ? NW * 8192 : 0);
  static constexpr int END = NW * WROWS * PITCH * 4, SIZE = LOOP > END ? LOOP : END;
};

// What a unit's ranges say: powers of two that keys and values are below, value ranges that are
// not numbers (bit 2 token + group / 2 of groups 0 and 2, of groups 1 and 3)
struct Unit4 {
  int ek;
  int ev;
  uint32_t some, none;  // whether there is such a range
  uint64_t bad0, bad1;
};

// A unit's codes and ranges on their way: N = 16 or 8 values of the keys and of the values to a thread.
// Keys: channels 8 (i % 16) .. + 7 of tokens i / 16, + 16; values: N channels of a token.
template <int N>
struct Regs4 {
  uint32_t k[N / 8], v[N / 8];
  f4_t mk[4];
  float2 mv;
};

struct Place4 {
  const uint8_t *kf, *vf;
  const float2 *km, *vm;
  int last;  // block of the capacity
};

template <int N>
__device__ __forceinline__ void fetch4(const Place4 &p, int un, Regs4<N> &s) {
  const uint32_t i = threadIdx.x;
  const int64_t u = min(un, p.last);
  constexpr uint32_t VT = D / N;  // threads to a token's values
  const uint8_t *kc = p.kf + u * (UNIT * HALF_D), *vc = p.vf + u * (UNIT * HALF_D);
  const uint8_t *km = (const uint8_t *)(p.km + u * 128), *vm = (const uint8_t *)(p.vm + u * 128);
#pragma unroll
  for (uint32_t x = 0; x < N / 8; x++) s.k[x] = *(const uint32_t *)(kc + ((i >> 4) * HALF_D + 4 * (i & 15)) + x * 16 * HALF_D);
#pragma unroll
  for (uint32_t x = 0; x < N / 8; x++) s.v[x] = *(const uint32_t *)(vc + ((i / VT) * HALF_D + N / 2 * (i % VT)) + 4 * x);
#pragma unroll
  for (uint32_t x = 0; x < 4; x++) s.mk[x] = *(const f4_t *)(km + 64 * (i & 15) + 16 * x);
  s.mv = *(const float2 *)(vm + (i / VT) * 32 + 8 * (N * (i % VT) / 32));
}

__device__ __forceinline__ float range_top(float2 m) { return fmaxf(fabsf(m.x), fabsf(__builtin_fmaf(15.0f, m.y, m.x))); }
// whether a value range gives no number for some code
__device__ __forceinline__ bool bad_range(float2 m) {
  return !(range_top(m) + fabsf(m.x) < INFINITY && m.y < INFINITY);
}
// A power of two above x: 2^9, which asks for no scaling, where x is in [2^-3, 2^8), so that small values keep
// 2^-22 of the largest; else the smallest
__device__ __forceinline__ int exponent_of(float x) {
  const int e = (int)(__float_as_uint(x) >> 23) - 126;
  return e >= -2 && e <= 8 ? kTop : e;
}

// a wave's unit: two ranges of keys and of values to a lane
struct Tops4 {
  f4_t k, v;
};
__device__ __forceinline__ void fetch_tops(const Place4 &p, int un, Tops4 &s) {
  const int lane = threadIdx.x & 63;
  const int64_t u = min(un, p.last);
  s.k = *(const f4_t *)((const uint8_t *)(p.km + u * 128) + 16u * lane);
  s.v = *(const f4_t *)((const uint8_t *)(p.vm + u * 128) + 16u * lane);
}
template <typename L>
__device__ __forceinline__ void put_tops(unsigned char *lds, int un, int len, const Tops4 &s) {
  const int lane = threadIdx.x & 63;
  const float tk = wave_max(fmaxf(range_top(make_float2(s.k[0], s.k[1])), range_top(make_float2(s.k[2], s.k[3]))));
  const bool there = un * UNIT + (lane >> 1) < len;  // ranges behind the sequence's end are whatever they are
  const float2 m0 = make_float2(s.v[0], s.v[1]), m1 = make_float2(s.v[2], s.v[3]);
  const bool bad0 = there && bad_range(m0), bad1 = there && bad_range(m1);
  const uint64_t b0 = __ballot(bad0), b1 = __ballot(bad1);
  const float tv = wave_max(fmaxf(there && !bad0 ? range_top(m0) : 0.0f, there && !bad1 ? range_top(m1) : 0.0f));
  if (lane == 0) {
    Unit4 *u = (Unit4 *)(lds + L::TOPS) + (un & 7);
    *u = Unit4{exponent_of(tk), exponent_of(tv), (b0 | b1) ? 1u : 0u, 0u, b0, b1};
  }
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

template <typename L, bool P2, bool V2, int N>
__device__ __forceinline__ void put4(unsigned char *lds, int un, int len, const Regs4<N> &s) {
  const int i = threadIdx.x;
  constexpr int VT = D / N;
  const Unit4 *u = (const Unit4 *)(lds + L::TOPS) + (un & 7);
  const int sk = kTop - __builtin_amdgcn_readfirstlane(u->ek), sv = kTop - __builtin_amdgcn_readfirstlane(u->ev);
  {
    float m[8], st[8];
#pragma unroll
    for (int k = 0; k < 8; k++) {
      m[k] = s.mk[k >> 1][2 * (k & 1)];
      st[k] = s.mk[k >> 1][2 * (k & 1) + 1];
    }
    if (sk != 0) {
#pragma unroll
      for (int k = 0; k < 8; k++) {
        m[k] = __builtin_ldexpf(m[k], sk);
        st[k] = __builtin_ldexpf(st[k], sk);
      }
    }
    unsigned char *k = lds + L::K + (un & 1) * KBYTES + (i >> 4) * KP + 16 * (i & 15);
    if constexpr (P2) {
#pragma unroll
      for (int t = 0; t < N / 8; t++) put_two(k + 16 * t * KP, L::KLO - L::K, s.k[t], st, m);
    } else {
      h2_t hs[4], hm[4];
#pragma unroll
      for (int x = 0; x < 4; x++) {
        hs[x] = pack2(st[x], st[x + 4]) * (_Float16)512.0f;  // 35000 at most
        hm[x] = pack2(__builtin_fmaf(8.0f, st[x], m[x]), __builtin_fmaf(8.0f, st[x + 4], m[x + 4]));
      }
#pragma unroll
      for (int t = 0; t < N / 8; t++) put_centred(k + 16 * t * KP, s.k[t], hs, hm);
    }
  }
  {
    const bool there = un * UNIT + i / VT < len && !bad_range(s.mv);
    const float m = there ? __builtin_ldexpf(s.mv.x, sv) : 0.0f, st = there ? __builtin_ldexpf(s.mv.y, sv) : 0.0f;
    unsigned char *v = lds + L::V + (un % 3) * VBYTES + (i / VT) * VP + 2 * N * (i % VT);
    if constexpr (V2) {
      float ms[8], sts[8];
#pragma unroll
      for (int k = 0; k < 8; k++) {
        ms[k] = m;
        sts[k] = st;
      }
#pragma unroll
      for (int t = 0; t < N / 8; t++) put_two(v + 16 * t, L::VLO - L::V, s.v[t], sts, ms);
    } else {
      const float c = __builtin_fmaf(8.0f, st, m);
      const h2_t a = pack2(st, st) * (_Float16)512.0f, z = pack2(c, c);
      const h2_t hs[4] = {a, a, a, a}, hm[4] = {z, z, z, z};
#pragma unroll
      for (int t = 0; t < N / 8; t++) put_centred(v + 16 * t, s.v[t], hs, hm);
    }
  }
}

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

struct Weights4 {
  float p[16], ps;
};

// weights of a unit; vis: tokens of the unit, less 4 half, that the lane's row sees (MASKED).
// Returns whether some weight is too large for its scale (or infinite: a row that has seen nothing yet).
template <bool MASKED>
__device__ __forceinline__ bool weights4(float A, float lv, const f16_t &z, int vis, const State4 &st, Weights4 &o) {
  const float lw = fmaxf(lv + st.f, -60.0f), iw = exp2_fast(-lw), B = lw - st.mu;
#pragma unroll
  for (int r = 0; r < 16; r++) {
    const float s = __builtin_fmaf(z[r], A, B);
    o.p[r] = exp2_fast(MASKED && 8 * (r >> 2) + (r & 3) >= vis ? -INFINITY : s);
  }
  float sum[1];
  sum_weights<1>(o.p, sum);
  o.ps = sum[0] * iw;
  return fmaxf(sum[0], o.ps * 128.0f) > 32768.0f;
}

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
  const Place4 place{a.kpay + (int64_t)bh * a.tcap * HALF_D, a.vpay + (int64_t)bh * a.tcap * HALF_D,
                     a.kmeta + (int64_t)bh * a.tcap * 4, a.vmeta + (int64_t)bh * a.tcap * 4, (int)a.nblk - 1};
  const int tmax = limit_of(a, sq, r0 / a.ratio, (r0 + nr - 1) / a.ratio);
  const int units = (tmax + UNIT - 1) / UNIT;
  const int u0 = split_begin(units, split, a.splits), u1 = split_begin(units, split + 1, a.splits);
  Regs4<N> nx;
  Tops4 tops;  // a wave's own of four units: a workgroup's first four waves find them every fourth turn
  if (u0 < u1) {
    fetch4(place, u0, nx);
    if (wave < 4) fetch_tops(place, u0 + wave, tops);
  }

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
  // the row's factor of a unit's scores and the log2 of its values' power of two; marks the rows that see
  // a value that is not a number
  const auto factors = [&](int un, float &A, float &lv) {
    const Unit4 *u = (const Unit4 *)(lds + L::TOPS) + (un & 7);
    const int4 e = *(const int4 *)u;
    A = __builtin_ldexpf(q.ca, e.x - kTop);
    lv = (float)e.y;
    if (__builtin_amdgcn_readfirstlane(e.z)) {
      const int vis = min(max(lim - un * UNIT, 0), UNIT);
      const uint64_t see = vis < 32 ? (1ull << 2 * vis) - 1 : ~0ull;
      const uint64_t b0 = u->bad0 & see, b1 = u->bad1 & see;
      constexpr uint64_t EVEN = 0x5555555555555555ull;
      st.poison |= (b0 & EVEN ? 1u : 0u) | (b1 & EVEN ? 2u : 0u) | (b0 & ~EVEN ? 4u : 0u) | (b1 & ~EVEN ? 8u : 0u);
    }
  };

  if (u0 < u1) {
    Weights4 o;
    UnitOperands<BF16> P;
    if (wave < 4) {
      put_tops<L>(lds, u0 + wave, sq.len, tops);
      fetch_tops(place, u0 + 4 + wave, tops);
    }
    __syncthreads();
    put4<L, P2, V2>(lds, u0, sq.len, nx);
    fetch4(place, u0 + 1, nx);  // units past the last are fetched (rows that exist) and not used
    if (u0 + 1 < u1) put4<L, P2, V2>(lds, u0 + 1, sq.len, nx);
    fetch4(place, u0 + 2, nx);
    __syncthreads();
    float A, lv;
    factors(u0, A, lv);
    raise4<P2>(keys_at(u0), klo, lo, A, lv, q, lim - u0 * UNIT - 4 * half, st, acc, o);
    const auto store_sum = [&](int un) {
      const uint32_t x = __float_as_uint(o.ps);
      const auto y = __builtin_amdgcn_permlane32_swap(x, x, false, false);
      const float v = __uint_as_float(y[0]) + __uint_as_float(y[1]);
      if (half == 0 && wr < a.rows) a.bsum[((int64_t)bh * a.entries + un) * a.rows + wr] = make_float2(v, st.mu);
    };
    if constexpr (SUMS) store_sum(u0);
    const auto turn = [&](int un, auto masked) {
      __syncthreads();  // unit un + 1 is there, unit un - 1 is done with
      if (un + 2 < u1) put4<L, P2, V2>(lds, un + 2, sq.len, nx);
      fetch4(place, un + 3, nx);
      if (((un - u0) & 3) == 0 && wave < 4) {
        put_tops<L>(lds, un + 4 + wave, sq.len, tops);
        fetch_tops(place, un + 8 + wave, tops);
      }
      const int vis = lim - (un + 1) * UNIT - 4 * half;
      st.l += o.ps;
      pack_weights<BF16>(o.p, P);
      float A, lv;
      factors(un + 1, A, lv);
      f16_t z;
      scores4<P2>(keys_at(un + 1), klo, q, lo, z);
      values4<V2>(values_at(un), vlo, P, acc);
      const bool up = weights4<decltype(masked)::value>(A, lv, z, vis, st, o);
      if (__any(up)) raise4<P2>(keys_at(un + 1), klo, lo, A, lv, q, vis, st, acc, o);
      if constexpr (SUMS) store_sum(un + 1);
    };
    // units that every row of the wave sees whole, then the others
    const int ua = min(u1 - 1, max(all / UNIT - 1, u0));
    for (int un = u0; un < ua; un++) turn(un, std::false_type{});
    for (int un = max(ua, u0); un + 1 < u1; un++) turn(un, std::true_type{});
    st.l += o.ps;
    pack_weights<BF16>(o.p, P);
    values4<V2>(values_at(u1 - 1), vlo, P, acc);
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
    const float ks = some ? inv * exp2_fast(st.mo - st.m) : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const float k = (st.poison >> j) & 1u ? NAN : 0.0f;  // a group of 32 channels
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        f4_t v;
#pragma unroll
        for (int x = 0; x < 4; x++) v[x] = __builtin_fmaf(acc[j][r + x] * 0x1p-18f, ks, k);  // 2^9 of the values, 2^9 of f
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
        a.part_ml[((int64_t)bh * a.splits + split) * a.rows + wr] = make_float2(st.m, Ls);
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

hipError_t tile4_launch(const AttendArgs &a, bool bf16, hipStream_t s) {
  const bool p2 = !bf16 || a.lse || a.mass, sums = a.bsum != nullptr;
  const int nw = p2 ? 8 : 4;
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
