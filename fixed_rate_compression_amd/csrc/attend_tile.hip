// Attention of many query rows over the 8-bit cache: prompts, chunks of them
// and drafted tokens, bound by the vector units that make the weights.
//
// A workgroup takes 128 query rows of one KV head, 32 to each of its four
// waves, gauges them in LDS (in a launch of their own, through memory, 13 us for
// 64000 rows and 5 more here), and walks the tokens 32 at a time: a unit's codes go
// through registers, are widened to centred fp16 once for the four waves and
// laid in LDS while another unit is worked on, one barrier a unit.  Widening
// at the use, from codes in LDS, took 96 of 244 vector instructions a wave
// and unit.  Keys are read as rows, values transposed by the LDS; the row
// pitches spread both over the banks.  The products are 32 x 32 (tokens x rows,
// channels x rows), which leaves a lane one row: half the matrix instructions
// and half the arithmetic on a row's state of 16 x 16 ones.
//
// The running maximum is not looked for: a lane's sum of weights tells whether
// one of them has outgrown its scale, and only then (and where a row sees its
// first token) the scores are formed again and the maximum raised.
//
// 2048 queries x 4 heads over 8192 tokens of 8 KV heads: the whole call 265 to
// 280 us, 890 TFLOP/s (with log-sums 348, fp32 storage 431); the matrix cores work 40 %
// of the cycles and the vector units 48 %, hardly at once.  Two prompts to 1000 tokens with both query parts and every row's
// sum of every unit kept for the blocks' weights (1.5 us): 55 us, the last rows'
// workgroups, which see all tokens, on their own at the end.  Value stores free of
// the bank conflicts they have (8 bytes of two rows a thread) changed nothing.
#include <type_traits>

#include "attend.hpp"

namespace cga {

constexpr int TROWS = 128;            // query rows of a workgroup
constexpr int WROWS = 32;             // of a wave
constexpr int KP = 2 * D + 16;        // LDS pitch of a token's keys, fp16: 16 tokens' 16-byte pieces in all 64 banks
constexpr int VP = 2 * D + 64;        // of its values: 4 tokens' 64-byte pieces in all 64 banks
constexpr int KBYTES = UNIT * KP, VBYTES = UNIT * VP;
// LDS of the token loop: a unit's keys are read a turn before its values
constexpr int KBUF = 0, VBUF = 2 * KBYTES, MBUF = VBUF + 3 * VBYTES, LOBUF = MBUF + 3 * 32;

typedef float f16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f16_t mfma32(h8_t a, h8_t b, f16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

typedef uint32_t u4_t __attribute__((ext_vector_type(4)));  // stays in registers through a loop (a uint4 member did not)

template <bool BF16>
struct UnitRegs {
  u4_t k, v;
  float2 m[BF16 ? 1 : 2];
};

// a unit's codes into registers: 16 bytes of a key and a value row to a thread;
// tokens past the capacity repeat its last row
template <bool BF16>
__device__ __forceinline__ void fetch_unit(const AttendArgs &a, const uint8_t *kf, const uint8_t *vf,
                                           const float2 *km, const float2 *vm, int un, UnitRegs<BF16> &s) {
  const int i = threadIdx.x;
  const int64_t t = min((int64_t)un * UNIT + (i >> 3), a.tcap - 1);
  s.k = *(const u4_t *)(kf + t * D + 16 * (i & 7));
  s.v = *(const u4_t *)(vf + t * D + 16 * (i & 7));
  // two 16-token tiles: key ranges, value ranges (lanes 0 .. 3 store them); fp32
  // storage: those of the thread's token, whose codes they centre
  const int64_t blk = min(((int64_t)un * UNIT + (BF16 ? 16 * (i & 1) : (i >> 3) & 16)) >> a.bshift, a.nblk - 1);
  if constexpr (BF16) {
    s.m[0] = ((i & 2) ? vm : km)[blk];
  } else {
    s.m[0] = km[blk];
    s.m[1] = vm[blk];
  }
}

// widened into LDS, once for the four waves (keys centred where both query
// parts take part; around the value 0 for fp32 storage)
template <bool BF16, bool LO>
__device__ __forceinline__ void put_unit(unsigned char *lds, int un, int tmax, const UnitRegs<BF16> &s) {
  const int i = threadIdx.x;
  unsigned char *k = lds + KBUF + (un & 1) * KBYTES + (i >> 3) * KP + 32 * (i & 7);
  unsigned char *v = lds + VBUF + (un % 3) * VBYTES + (i >> 3) * VP + 32 * (i & 7);
  // the range that this thread stores (entries: keys of both tiles, values of both) and
  // the value of its centre
  Centre ck{0.0f, kMiddle}, cv = ck;
  int e;
  float2 m;
  float mid;
  bool mine;
  if constexpr (BF16) {
    e = i;
    mine = i < 4;
    m = s.m[0];
    mid = LO || (i & 2) ? __builtin_fmaf(128.0f, m.y, m.x) : m.x;
  } else {
    ck = centre_of(s.m[0]);
    cv = centre_of(s.m[1]);
    e = 2 * (i & 1) + (i >> 7);
    mine = (i & 127) < 2;
    m = i & 1 ? s.m[1] : s.m[0];
    mid = i & 1 ? cv.mid : ck.mid;
  }
  *(h8_t *)k = codes8<LO>(s.k.x, s.k.y, ck.c);
  *(h8_t *)(k + 16) = codes8<LO>(s.k.z, s.k.w, ck.c);
  *(h8_t *)v = codes8<true>(s.v.x, s.v.y, cv.c);
  *(h8_t *)(v + 16) = codes8<true>(s.v.z, s.v.w, cv.c);
  if (mine) {
    const bool there = un * UNIT + 16 * (e & 1) < tmax;  // a block that holds no row yet is not looked at
    const float st = there ? m.y : 0.0f;
    *(float2 *)(lds + MBUF + (un % 3) * 32 + 8 * e) =
        make_float2(there ? mid : 0.0f, (e & 2) ? fminf(fmaxf(__builtin_amdgcn_logf(st), -200.0f), 128.0f) : st);  // values: log2 of the step
  }
}

// a lane's row (the same in lanes l and l + 32 but for l and mv), as in
// attend_rows.hip, but mu is -inf while the row has seen nothing
struct TileState {
  float m, mu, mo, f, l, mv;  // f: log2 of the values' scale
};

// the queries of a wave: channels 16 s + 8 half + 0 .. 7 of row lane % 32 at step s
struct TileQueries {
  h8_t hi[8];
  float ca, cq;
};

// The fp16 operands of a wave's 32 gauged rows xs [32][PITCH]: the scale and the two
// parts of make_frags, or one part (a channel rounded to 2^-11).
template <bool TWO>
__device__ __forceinline__ void tile_queries(const float *xs, float c, TileQueries &q, h8_t (&lo)[8]) {
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const float *rp = xs + (lane & 31) * PITCH + 8 * half;
  f4_t x[16];
  float mx = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; k++) {
    x[k] = *(const f4_t *)(rp + 16 * (k >> 1) + 4 * (k & 1));
    mx = fmaxf(fmaxf(mx, fmaxf(fabsf(x[k][0]), fabsf(x[k][1]))), fmaxf(fabsf(x[k][2]), fabsf(x[k][3])));
  }
  const FragScale sc = frag_scale(fmaxf(mx, __shfl_xor(mx, 32)));
  float sum = 0.0f;
#pragma unroll
  for (int s = 0; s < 8; s++) frag_parts<TWO>(x[2 * s], x[2 * s + 1], sc.up, q.hi[s], lo[s], sum);
  // an infinity: NaN for the row, as its difference from its first part is with two (alone it
  // can make every score -inf, whose weights would all be 0)
  if constexpr (!TWO) sum = __builtin_fmaf(mx, 0.0f, sum);
  q.ca = c * sc.un;
  q.cq = q.ca * (sum + __shfl_xor(sum, 32));
}

// the weights of a unit, p_t sv_b f, and what goes with them; NB ranges to a
// unit (two where blocks have 16 tokens).  The values' factor is added to the
// exponent: sums of p itself are those of the weights over the factor.  Where it
// is below 2^-60 the weights vanish in fp16 either way and 2^-60 stands for it
// (a constant block has factor 0, its rows still count).
template <int NB>
struct UnitWeights {
  float p[16];
  float ps[NB], mid[NB];  // sums of p_t, values of the centres
};

// scores of a unit: z = K Q^T, z[r] that of token 8 (r / 4) + 4 half + r % 4,
// from the keys at kb (this lane's token and piece)
template <bool LO>
__device__ __forceinline__ void unit_scores(const unsigned char *kb, const TileQueries &q, const unsigned char *lo,
                                            f16_t &z) {
  f16_t zl;
#pragma unroll
  for (int r = 0; r < 16; r++) z[r] = zl[r] = 0.0f;
#pragma unroll
  for (int s = 0; s < 8; s++) {
    const h8_t c = *(const h8_t *)(kb + 32 * s);
    z = mfma32(c, q.hi[s], z);
    if constexpr (LO) zl = mfma32(c, *(const h8_t *)(lo + 1024 * s), zl);
  }
  if constexpr (LO) z += zl;
}

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

// whether the lane's row sees none of range u's tokens: the values' range, which
// may hold a NaN of a later token, is then left out
template <int NB>
__device__ __forceinline__ bool unseen(int u, int vis) {
  return vis + (int)((threadIdx.x & 32) >> 3) <= (NB == 2 ? 16 * u : 0);
}

// weights of a unit; vis: tokens of the unit, less 4 half, that the lane's row
// sees (MASKED).  Returns whether some weight is too large for its scale (or
// infinite: a row that has seen nothing yet).
template <bool MASKED, int NB>
__device__ __forceinline__ bool unit_weights(const float2 *mt, const TileQueries &q, const f16_t &z, int vis,
                                             const TileState &st, UnitWeights<NB> &o) {
  float iw[NB], sum[NB], over = 0.0f;
#pragma unroll
  for (int u = 0; u < NB; u++) {
    const float2 mk = mt[u], mv = mt[2 + u];
    o.mid[u] = MASKED && unseen<NB>(u, vis) ? 0.0f : mv.x;
    const float lw = fmaxf(mv.y + st.f, -60.0f);
    iw[u] = exp2_fast(-lw);
    const float A = mk.y * q.ca, B = __builtin_fmaf(mk.x, q.cq, lw - st.mu);
#pragma unroll
    for (int k = 0; k < 16 / NB; k++) {
      const int r = 16 / NB * u + k;
      const float s = __builtin_fmaf(z[r], A, B);
      o.p[r] = exp2_fast(MASKED && 8 * (r >> 2) + (r & 3) >= vis ? -INFINITY : s);
    }
  }
  sum_weights<NB>(o.p, sum);
#pragma unroll
  for (int u = 0; u < NB; u++) {
    o.ps[u] = sum[u] * iw[u];
    over = fmaxf(over, fmaxf(sum[u], o.ps[u] * 128.0f));
  }
  return over > 32768.0f;
}

__device__ __forceinline__ float pair_max(float v) { return fmaxf(v, __shfl_xor(v, 32)); }

// raise the row's maximum to the unit's scores, rescale what was summed, and
// form the unit's weights again (rare: the scores are not kept for it)
template <bool LO, int NB>
__device__ __forceinline__ void raise(const unsigned char *kb, const unsigned char *lo, const float2 *mt,
                                      const TileQueries &q, int vis, TileState &st, f16_t (&acc)[4],
                                      UnitWeights<NB> &o) {
  f16_t z;
  uint32_t again = 0;  // unknown to the compiler: the operands of the rare second product are not kept for it
  asm volatile("" : "+v"(again));
  unit_scores<LO>(kb + again, q, lo + again, z);
  float mx = -INFINITY, mv = -INFINITY;
#pragma unroll
  for (int u = 0; u < NB; u++) {
    const float2 mk = mt[u];
    const float A = mk.y * q.ca, B = mk.x * q.cq;
    float t = -INFINITY;
#pragma unroll
    for (int k = 0; k < 16 / NB; k++) {
      const int r = 16 / NB * u + k;
      o.p[r] = 8 * (r >> 2) + (r & 3) < vis ? __builtin_fmaf(z[r], A, B) : -INFINITY;
      t = fmaxf(t, o.p[r]);
    }
    mx = fmaxf(mx, t);
    mv = fmaxf(mv, t + mt[2 + u].y);
  }
  const float mn = fmaxf(st.m, pair_max(mx));
  float on = fmaxf(st.mo, pair_max(mv));
  const bool some = mn > -INFINITY;
  if (some) on = fmaxf(on, mn - 80.0f);  // keeps 2^(m - mo) finite beside weights that vanish
  const float al = st.m > -INFINITY ? exp2_fast(st.m - mn) : 0.0f;
  const float ao = st.mo > -INFINITY ? exp2_fast(st.mo - on) : 0.0f;
  st.l *= al;
  st.mv *= al;
#pragma unroll
  for (int j = 0; j < 4; j++) acc[j] *= ao;
  st.m = st.mu = mn;
  st.mo = on;
  st.f = some ? mn - on + 9.0f : 0.0f;
  const float mu = some ? mn : 0.0f;
  float iw[NB], sum[NB];
#pragma unroll
  for (int u = 0; u < NB; u++) {
    const float lw = fmaxf(mt[2 + u].y + st.f, -60.0f);
    iw[u] = exp2_fast(-lw);
#pragma unroll
    for (int k = 0; k < 16 / NB; k++) {
      const int r = 16 / NB * u + k;
      o.p[r] = exp2_fast(o.p[r] + (lw - mu));
    }
  }
  sum_weights<NB>(o.p, sum);
#pragma unroll
  for (int u = 0; u < NB; u++) {
    o.ps[u] = sum[u] * iw[u];
    o.mid[u] = unseen<NB>(u, vis) ? 0.0f : mt[2 + u].x;
  }
}

// a unit's weights as operands (tokens 16 x + ..), its sums into the row's state
template <bool BF16>
struct UnitOperands {
  h8_t hi[2], lo[2];  // lo: fp32 storage only
};

template <bool BF16, int NB>
__device__ __forceinline__ void take_weights(const UnitWeights<NB> &o, TileState &st, UnitOperands<BF16> &P) {
#pragma unroll
  for (int u = 0; u < NB; u++) {
    st.l += o.ps[u];
    st.mv = __builtin_fmaf(o.mid[u], o.ps[u], st.mv);
  }
#pragma unroll
  for (int x = 0; x < 2; x++) {
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const float a = o.p[8 * x + 2 * k], b = o.p[8 * x + 2 * k + 1];
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

// acc += V^T P^T of a unit, from the values at vb (this lane's token and piece);
// acc[j][r]: channel 32 j + 8 (r / 4) + 4 half + r % 4
template <bool BF16>
__device__ __forceinline__ void unit_values(const unsigned char *vb, const UnitOperands<BF16> &P, f16_t (&acc)[4]) {
#pragma unroll
  for (int x = 0; x < 2; x++)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const s4_t a = transposed(vb + 16 * x * VP + 64 * j), b = transposed(vb + (16 * x + 8) * VP + 64 * j);
      const h8_t vj = __builtin_bit_cast(h8_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
      acc[j] = mfma32(vj, P.hi[x], acc[j]);
      if constexpr (!BF16) acc[j] = mfma32(vj, P.lo[x], acc[j]);
    }
}

// a row's sum of a unit's weights and the maximum it stands on, for the blocks' weights
template <int NB>
__device__ __forceinline__ void store_sums(const AttendArgs &a, int bh, int un, int wr, int half,
                                           const UnitWeights<NB> &o, float mu) {
  const int64_t e = (int64_t)un * NB;
  float2 *p = a.bsum + ((int64_t)bh * a.entries + e) * a.rows + wr;
#pragma unroll
  for (int u = 0; u < NB; u++) {
    const uint32_t x = __float_as_uint(o.ps[u]);
    const auto y = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    const float v = __uint_as_float(y[0]) + __uint_as_float(y[1]);
    if (half == 0 && wr < a.rows && (u == 0 || e + u < a.entries)) p[(int64_t)u * a.rows] = make_float2(v, mu);
  }
}

// LO: the queries' second fp16 part takes part (fp32 storage, or where log-sums
// or weights are asked for); else a query is rounded to 2^-11 of a channel.
// NB: ranges to a unit of 32 tokens.  SUMS: the rows' sums of every unit are kept.
template <bool BF16, bool LO, int NB, bool SUMS>
__global__ __launch_bounds__(NTH, 2) void k_attend_tile(const AttendArgs a) {
  static_assert(BF16 || LO, "fp32 storage takes both parts");
  constexpr int LOOP_LDS = LOBUF + (LO ? 4 * 8192 : 0), END_LDS = TROWS * PITCH * 4;
  __shared__ __align__(16) unsigned char lds[LOOP_LDS > END_LDS ? LOOP_LDS : END_LDS];
  const int lane = threadIdx.x & 63, row = lane & 31, half = lane >> 5, n = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fields = a.batch * a.heads, groups = (a.rows + TROWS - 1) / TROWS;
  const uint32_t q1 = blockIdx.x / (uint32_t)fields, q2 = q1 / (uint32_t)a.splits;
  const int bh = (int)(blockIdx.x - q1 * fields);  // a head's workgroups share an XCD's L2 where the heads are a multiple of 8
  const int split = (int)(q1 - q2 * a.splits);
  // the longest first; where all are resident at once (two to a compute unit) the
  // second half runs from the shortest up, beside the first half's longest
  const int turn_of = (int)q2, first = (groups + 1) / 2;
  const bool paired = (int64_t)gridDim.x <= 512 && a.splits == 1;
  const int grpi = paired && turn_of >= first ? turn_of - first : groups - 1 - turn_of;
  const int h = bh % a.heads, b = bh / a.heads;
  const int r0 = grpi * TROWS, nr = min(TROWS, a.rows - r0);
  const Sequence sq = load_sequence(a, b);

  const uint8_t *kf = a.kpay + (int64_t)bh * a.tcap * D, *vf = a.vpay + (int64_t)bh * a.tcap * D;
  const float2 *km = a.kmeta + (int64_t)bh * a.nblk, *vm = a.vmeta + (int64_t)bh * a.nblk;
  const int tmax = limit_of(a, sq, r0 / a.ratio, (r0 + nr - 1) / a.ratio);
  const int units = (tmax + UNIT - 1) / UNIT;
  const int u0 = split_begin(units, split, a.splits), u1 = split_begin(units, split + 1, a.splits);
  UnitRegs<BF16> nx;
  if (u0 < u1) fetch_unit<BF16>(a, kf, vf, km, vm, u0, nx);

  // gauged queries as operands
  TileQueries q;
  unsigned char *const lo = lds + LOBUF + wave * 8192 + lane * 16;
  const int wr = r0 + wave * WROWS + row;  // the lane's row
  {
    float *xs = (float *)lds;
    const float *gk = a.gk + (int64_t)h * D * a.g;
    GaugeFrag gw;
    load_gauge<false>(gk, a.g, 0, gw);
    RowPart p[TROWS / ROWS];
#pragma unroll
    for (int t = 0; t < TROWS / ROWS; t++) p[t] = load_row_part<BF16>(a, b, h, r0 + t * ROWS);
#pragma unroll
    for (int t = 0; t < TROWS / ROWS; t++) put_row_part(xs + t * ROWS * PITCH, p[t]);
    __syncthreads();
    if (a.g) {
      gauge_tiles<false, TROWS / ROWS, true>(xs, xs, gk, a.g, gw);
      __syncthreads();
    }
    h8_t part[8];
    tile_queries<LO>(xs + wave * WROWS * PITCH, a.c, q, part);
    __syncthreads();  // the rows have been read
    q.ca *= LO ? kCentredUnit : kCodeUnit;
    if constexpr (LO)
#pragma unroll
      for (int s = 0; s < 8; s++) *(h8_t *)(lo + s * 1024) = part[s];
  }
  // what the row sees; rows that are not there see everything
  const int lim = wr < a.rows ? query_limit(a, sq, (int)((uint32_t)wr / (uint32_t)a.ratio)) : tmax;
  int all = lim;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) all = min(all, __shfl_xor(all, k));
  all = __builtin_amdgcn_readfirstlane(all);

  TileState st;
  st.m = st.mo = st.mu = -INFINITY;
  st.l = st.mv = 0.0f;
  st.f = 0.0f;
  f16_t acc[4];
#pragma unroll
  for (int j = 0; j < 4; j++)
#pragma unroll
    for (int r = 0; r < 16; r++) acc[j][r] = 0.0f;
  const auto keys_at = [&](int un) { return lds + KBUF + (un & 1) * KBYTES + row * KP + 16 * half; };
  const auto values_at = [&](int un) {
    return lds + VBUF + (un % 3) * VBYTES + (4 * half + (n >> 2)) * VP + 32 * ((lane >> 4) & 1) + 8 * (n & 3);
  };
  const auto ranges_at = [&](int un) { return (const float2 *)(lds + MBUF + (un % 3) * 32); };

  // One unit ahead: a turn forms the scores and weights of the next unit beside
  // the value product of the present one, so matrix and vector work of both
  // lie in one block for the scheduler.
  if (u0 < u1) {
    UnitWeights<NB> o;
    UnitOperands<BF16> P;
    put_unit<BF16, LO>(lds, u0, tmax, nx);
    fetch_unit<BF16>(a, kf, vf, km, vm, u0 + 1, nx);  // units past the last are fetched (rows that exist) and not used
    put_unit<BF16, LO>(lds, u0 + 1, tmax, nx);
    fetch_unit<BF16>(a, kf, vf, km, vm, u0 + 2, nx);
    __syncthreads();
    raise<LO, NB>(keys_at(u0), lo, ranges_at(u0), q, lim - u0 * UNIT - 4 * half, st, acc, o);
    if constexpr (SUMS) store_sums<NB>(a, bh, u0, wr, half, o, st.mu);
    const auto turn = [&](int un, auto masked) {
      __syncthreads();  // unit un + 1 is there, unit un - 1 is done with
      put_unit<BF16, LO>(lds, un + 2, tmax, nx);
      fetch_unit<BF16>(a, kf, vf, km, vm, un + 3, nx);
      const float2 *mt = ranges_at(un + 1);
      const int vis = lim - (un + 1) * UNIT - 4 * half;
      take_weights<BF16, NB>(o, st, P);
      f16_t z;
      unit_scores<LO>(keys_at(un + 1), q, lo, z);
      unit_values<BF16>(values_at(un), P, acc);
      const bool up = unit_weights<decltype(masked)::value, NB>(mt, q, z, vis, st, o);
      if (__any(up)) raise<LO, NB>(keys_at(un + 1), lo, mt, q, vis, st, acc, o);
      if constexpr (SUMS) store_sums<NB>(a, bh, un + 1, wr, half, o, st.mu);
    };
    // units that every row of the wave sees whole, then the others
    const int ua = min(u1 - 1, max(all / UNIT - 1, u0));
    for (int un = u0; un < ua; un++) turn(un, std::false_type{});
    for (int un = max(ua, u0); un + 1 < u1; un++) turn(un, std::true_type{});
    take_weights<BF16, NB>(o, st, P);
    unit_values<BF16>(values_at(u1 - 1), P, acc);
  }
  __syncthreads();

  // rows' sums, scaled as they stand, into LDS; then parts or outputs
  const float *gv = a.gv + (int64_t)h * D * a.g;
  GaugeFrag gw;
  load_gauge<true>(gv, a.g, 0, gw);
  float *us = (float *)lds;
  {
    const int rr = wave * WROWS + row;
    const float L = st.l + __shfl_xor(st.l, 32), mvs = st.mv + __shfl_xor(st.mv, 32);
    const bool some = st.m > -INFINITY;
    const float inv = a.splits > 1 ? 1.0f : L > 0.0f ? 1.0f / L : 0.0f;
    const float ks = some ? inv * exp2_fast(st.mo - st.m) : 0.0f;
    const float k = some ? inv * mvs : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        *(float4 *)(us + rr * PITCH + 32 * j + 2 * r + 4 * half) =
            make_float4(__builtin_fmaf(acc[j][r], ks, k), __builtin_fmaf(acc[j][r + 1], ks, k),
                        __builtin_fmaf(acc[j][r + 2], ks, k), __builtin_fmaf(acc[j][r + 3], ks, k));
    if (half == 0 && rr < nr) {
      if (a.splits > 1) {
        a.part_ml[((int64_t)bh * a.splits + split) * a.rows + wr] = make_float2(st.m, L);
      } else {
        if (a.lse) store_lse(a, b, h, wr, st.m, L);
        if (a.lse2) a.lse2[(int64_t)bh * a.rows + wr] = L != 0.0f ? st.m + __builtin_log2f(L) : INFINITY;
      }
    }
  }
  __syncthreads();
  if (a.splits > 1) {
    float *po = a.part_o + (((int64_t)bh * a.splits + split) * a.rows + r0) * D;
    for (int i = threadIdx.x; i < nr * (D / 4); i += NTH)
      *(float4 *)(po + 4 * (int64_t)i) = *(const float4 *)(us + (i / (D / 4)) * PITCH + 4 * (i % (D / 4)));
    return;
  }
  if (a.g) {
    gauge_tiles<true, TROWS / ROWS, true>(us, us, gv, a.g, gw);
    __syncthreads();
  }
  store_rows<BF16>(a, b, h, r0, nr, us);
}

hipError_t tile_launch(const AttendArgs &a, bool bf16, hipStream_t s) {
  const int64_t groups = (a.rows + TROWS - 1) / TROWS;
  const dim3 grid((unsigned)((int64_t)a.batch * a.heads * groups * a.splits)), block(NTH);
#define CG_T(BF, LO, NB, SUMS)                                                                 \
  if (bf16 == BF && lo == LO && nb == NB && sums == SUMS) {                                    \
    hipLaunchKernelGGL((k_attend_tile<BF, LO, NB, SUMS>), grid, block, 0, s, a);               \
    return hipGetLastError();                                                                  \
  }
  const bool lo = !bf16 || a.lse || a.mass, sums = a.bsum != nullptr;
  const int nb = a.bshift == 4 ? 2 : 1;  // ranges to a unit
  CG_T(true, false, 1, false) CG_T(true, false, 2, false)
  CG_T(true, true, 1, false) CG_T(true, true, 2, false) CG_T(false, true, 1, false) CG_T(false, true, 2, false)
  CG_T(true, true, 1, true) CG_T(true, true, 2, true) CG_T(false, true, 1, true) CG_T(false, true, 2, true)
#undef CG_T
  return hipErrorInvalidValue;
}

}  // namespace cga
