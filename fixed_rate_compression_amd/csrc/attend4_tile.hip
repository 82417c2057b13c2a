// Attention of many query rows over the 4-bit cache: prompts, chunks of them and drafted
// tokens.  The walk is that of the 8-bit cache's form (attend_tile.hip): 32 rows to
// a wave, 32 tokens a turn laid in LDS as fp16 for all waves, scores and weights of the
// next unit beside the value product of the present one.
//
// Keys and values are widened to what they stand for, since their ranges differ along the
// contraction (keys: by channel) or along both axes (values): one multiply-add a code in
// fp32, rounded to fp16 once for all rows, in two parts where log-sums or
// weights are asked for or the storage is fp32.  A power of two a unit keeps either in fp16's
// range; it is found from the unit's 256 ranges two turns before the codes are
// widened, a range to a thread.
#include <type_traits>

#include "attend.hpp"
#include "attend_tile.hpp"

namespace cga {

typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

constexpr int HALF_D = D / 2;  // bytes of a row of codes
constexpr int kTop = 14;       // widened keys and values are below 2^14

// LDS of a workgroup's token loop; two parts of the keys (P2), of the values (V2)
template <bool P2, bool V2, int NW>
struct Lds4 {
  static constexpr int K = 0, KLO = 2 * KBYTES, V = KLO + (P2 ? 2 * KBYTES : 0), VLO = V + 3 * VBYTES;
  static constexpr int TOPS = VLO + (V2 ? 3 * VBYTES : 0);  // [4][4]: largest magnitudes, of the keys by waves 0 and 1, of the values by 2 and 3
  static constexpr int BAD = TOPS + 64;                     // [4][2]: value ranges that are not numbers, bit 4 token + group
  static constexpr int QLO = BAD + 64, LOOP = QLO + (P2 ? NW * 8192 : 0);
  static constexpr int END = NW * WROWS * PITCH * 4, SIZE = LOOP > END ? LOOP : END;
};

// A unit's codes and ranges on their way: N = 16 or 8 values of the keys and of the values to a thread.
// Keys: channels 8 (i % 16) .. + 7 of tokens i / 16, + 16; values: N channels of a token.
template <int N>
struct Regs4 {
  uint32_t k[N / 8], v[N / 8];
  f4_t mk[4];
  float2 mv;
  float2 top;  // one of the 256 ranges of the unit two further
};

template <int N>
struct Place4 {
  const uint8_t *kf, *vf;
  const float2 *km, *vm;
  int last;  // block of the capacity
};

template <int N>
__device__ __forceinline__ void fetch4(const Place4<N> &p, int un, Regs4<N> &s) {
  const int i = threadIdx.x;
  const int64_t t0 = (int64_t)min(un, p.last) * UNIT;
  constexpr int VT = D / N;  // threads to a token's values
#pragma unroll
  for (int x = 0; x < N / 8; x++) s.k[x] = *(const uint32_t *)(p.kf + (t0 + (i >> 4) + 16 * x) * HALF_D + 4 * (i & 15));
  const uint32_t *v = (const uint32_t *)(p.vf + (t0 + i / VT) * HALF_D + N / 2 * (i % VT));
#pragma unroll
  for (int x = 0; x < N / 8; x++) s.v[x] = v[x];
  const f4_t *m = (const f4_t *)(p.km + t0 * 4 + 8 * (i & 15));
#pragma unroll
  for (int x = 0; x < 4; x++) s.mk[x] = m[x];
  s.mv = p.vm[(t0 + i / VT) * 4 + N * (i % VT) / 32];
}

template <int N>
__device__ __forceinline__ void fetch_top(const Place4<N> &p, int un, Regs4<N> &s) {
  const int i = threadIdx.x & 255;  // the same for both halves of eight waves
  s.top = (i < 128 ? p.km : p.vm - 128)[(int64_t)min(un, p.last) * 128 + i];
}

__device__ __forceinline__ float range_top(float2 m) { return fmaxf(fabsf(m.x), fabsf(__builtin_fmaf(15.0f, m.y, m.x))); }
// whether a value range gives no number for some code
__device__ __forceinline__ bool bad_range(float2 m) {
  return !(range_top(m) + fabsf(m.x) < INFINITY && m.y < INFINITY);
}
// smallest E with |x| < 2^E
__device__ __forceinline__ int exponent_of(float x) { return (int)(__float_as_uint(x) >> 23) - 126; }

// the unit's largest magnitudes, and its value ranges that are not numbers; `len`: rows of the
// sequence, `tmax`: tokens that some row of the workgroup sees
template <typename L, int N>
__device__ __forceinline__ void put_top(unsigned char *lds, int un, int len, int tmax, const Regs4<N> &s) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (wave >= 4) return;
  const bool there = wave < 2 ? un * UNIT < tmax : un * UNIT + 16 * (wave & 1) + (lane >> 2) < len;
  const float2 m = there ? s.top : make_float2(0.f, 0.f);
  const bool bad = wave >= 2 && bad_range(m);
  const uint64_t all = __ballot(bad);
  const float t = wave_max(bad ? 0.0f : range_top(m));
  if (lane == 0) {
    *(float *)(lds + L::TOPS + 16 * (un & 3) + 4 * wave) = t;
    if (wave >= 2) *(uint64_t *)(lds + L::BAD + 16 * (un & 3) + 8 * (wave & 1)) = all;
  }
}

struct Exponents {
  int k, v;
};
template <typename L>
__device__ __forceinline__ Exponents exponents_at(const unsigned char *lds, int un) {
  const f4_t t = *(const f4_t *)(lds + L::TOPS + 16 * (un & 3));
  return Exponents{exponent_of(fmaxf(t[0], t[1])), exponent_of(fmaxf(t[2], t[3]))};
}

// eight codes as floats
__device__ __forceinline__ void codes_f32(uint32_t w, float (&c)[8]) {
  const uint32_t e = w & 0x0f0f0f0fu, o = (w >> 4) & 0x0f0f0f0fu;
#pragma unroll
  for (int k = 0; k < 4; k++) {
    c[2 * k] = (float)((e >> 8 * k) & 0xffu);
    c[2 * k + 1] = (float)((o >> 8 * k) & 0xffu);
  }
}

// 8 values as fp16, what is left of them in `lo` (TWO)
template <bool TWO>
__device__ __forceinline__ void put8(unsigned char *p, int lo, const float (&x)[8]) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int k = 0; k < 4; k++) {
    h[k] = pack_f16x2(x[2 * k], x[2 * k + 1]);
    if constexpr (TWO) {
      const f2_t hh = unpack_f16x2(h[k]);
      l[k] = pack_f16x2(x[2 * k] - hh.x, x[2 * k + 1] - hh.y);
    }
  }
  *(h8_t *)p = as_h8(h[0], h[1], h[2], h[3]);
  if constexpr (TWO) *(h8_t *)(p + lo) = as_h8(l[0], l[1], l[2], l[3]);
}

template <typename L, bool P2, bool V2, int N>
__device__ __forceinline__ void put4(unsigned char *lds, int un, int len, int tmax, const Regs4<N> &s) {
  const int i = threadIdx.x;
  constexpr int VT = D / N;
  const Exponents e = exponents_at<L>(lds, un);
  float c[8], x[8];
  {
    const bool there = un * UNIT < tmax;  // a block that holds no row yet is not looked at
    float m[8], st[8];
#pragma unroll
    for (int k = 0; k < 8; k++) {
      m[k] = there ? __builtin_ldexpf(s.mk[k >> 1][2 * (k & 1)], kTop - e.k) : 0.0f;
      st[k] = there ? __builtin_ldexpf(s.mk[k >> 1][2 * (k & 1) + 1], kTop - e.k) : 0.0f;
    }
    unsigned char *k = lds + L::K + (un & 1) * KBYTES + (i >> 4) * KP + 16 * (i & 15);
#pragma unroll
    for (int t = 0; t < N / 8; t++) {
      codes_f32(s.k[t], c);
#pragma unroll
      for (int j = 0; j < 8; j++) x[j] = __builtin_fmaf(c[j], st[j], m[j]);
      put8<P2>(k + 16 * t * KP, L::KLO - L::K, x);
    }
  }
  {
    const bool there = un * UNIT + i / VT < len && !bad_range(s.mv);
    const float m = there ? __builtin_ldexpf(s.mv.x, kTop - e.v) : 0.0f, st = there ? __builtin_ldexpf(s.mv.y, kTop - e.v) : 0.0f;
    unsigned char *v = lds + L::V + (un % 3) * VBYTES + (i / VT) * VP + 2 * N * (i % VT);
#pragma unroll
    for (int t = 0; t < N / 8; t++) {
      codes_f32(s.v[t], c);
#pragma unroll
      for (int j = 0; j < 8; j++) x[j] = __builtin_fmaf(c[j], st, m);
      put8<V2>(v + 16 * t, L::VLO - L::V, x);
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
      const float u = x[2 * s + (k >> 1)][2 * (k & 1)] * sc.up, v = x[2 * s + (k >> 1)][2 * (k & 1) + 1] * sc.up;
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
  const Place4<N> place{a.kpay + (int64_t)bh * a.tcap * HALF_D, a.vpay + (int64_t)bh * a.tcap * HALF_D,
                        a.kmeta + (int64_t)bh * a.tcap * 4, a.vmeta + (int64_t)bh * a.tcap * 4, (int)a.nblk - 1};
  const int tmax = limit_of(a, sq, r0 / a.ratio, (r0 + nr - 1) / a.ratio);
  const int units = (tmax + UNIT - 1) / UNIT;
  const int u0 = split_begin(units, split, a.splits), u1 = split_begin(units, split + 1, a.splits);
  Regs4<N> nx, ny;
  if (u0 < u1) {
    fetch4(place, u0, nx);
    fetch_top(place, u0, nx);
    fetch_top(place, u0 + 1, ny);
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
    const Exponents e = exponents_at<L>(lds, un);
    A = __builtin_ldexpf(q.ca, e.k - kTop);
    lv = (float)e.v;
    const uint64_t *bad = (const uint64_t *)(lds + L::BAD + 16 * (un & 3));
    const uint64_t b0 = bad[0], b1 = bad[1];
    if (__builtin_amdgcn_readfirstlane((uint32_t)(b0 | b0 >> 32 | b1 | b1 >> 32))) {
      const int vis = min(max(lim - un * UNIT, 0), UNIT), v0 = min(vis, 16), v1 = vis - v0;
      uint64_t x = (v0 < 16 ? b0 & ((1ull << 4 * v0) - 1) : b0) | (v1 < 16 ? b1 & ((1ull << 4 * v1) - 1) : b1);
#pragma unroll
      for (int k = 32; k >= 4; k >>= 1) x |= x >> k;
      st.poison |= (uint32_t)x & 15u;
    }
  };

  if (u0 < u1) {
    Weights4 o;
    UnitOperands<BF16> P;
    put_top<L>(lds, u0, sq.len, tmax, nx);
    put_top<L>(lds, u0 + 1, sq.len, tmax, ny);
    fetch_top(place, u0 + 2, nx);
    __syncthreads();
    put4<L, P2, V2>(lds, u0, sq.len, tmax, nx);
    fetch4(place, u0 + 1, nx);  // units past the last are fetched (rows that exist) and not used
    put_top<L>(lds, u0 + 2, sq.len, tmax, nx);
    put4<L, P2, V2>(lds, u0 + 1, sq.len, tmax, nx);
    fetch4(place, u0 + 2, nx);
    fetch_top(place, u0 + 3, nx);
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
      put4<L, P2, V2>(lds, un + 2, sq.len, tmax, nx);
      put_top<L>(lds, un + 3, sq.len, tmax, nx);
      fetch4(place, un + 3, nx);
      fetch_top(place, un + 4, nx);
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
        for (int x = 0; x < 4; x++) v[x] = __builtin_fmaf(acc[j][r + x] * 0x1p-23f, ks, k);  // 2^14 of the values, 2^9 of f
        *(f4_t *)(us + rr * PITCH + 32 * j + 2 * r + 4 * half) = v;
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
  const int nw = p2 || a.rows > 128 ? 8 : 4;
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
