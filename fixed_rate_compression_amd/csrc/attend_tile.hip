// Attention of many query rows over the 8-bit cache: prompts, chunks of them
// and drafted tokens, bound by the vector units that make the weights.
//
// A workgroup takes 128 query rows of one KV head, 32 to each of its four
// waves (two row tiles), and walks the tokens 64 at a time: the codes and
// ranges of a stage go through registers into LDS while another is worked on,
// one barrier a stage.  The products are those of the
// few-row kernel (attend_rows.hip) with the codes read from LDS and each
// widened operand used for both row tiles.  Rows of 16-byte pieces are stored
// with piece ^ (row % 8), so the 16 rows that a key operand's lanes read at
// one piece lie in different banks.
//
// The running maximum is not looked for: a lane's sum of weights tells whether
// one of them has outgrown its scale, and only then (and where a row sees its
// first token) the scores are formed again and the maximum raised.
#include <type_traits>

#include "attend.hpp"

namespace cga {

constexpr int STAGE = 64;        // tokens of a stage
constexpr int TROWS = 128;       // query rows of a workgroup
constexpr int WT = 2;            // row tiles of a wave
constexpr int CODES = STAGE * D; // bytes of a stage's key (value) codes

typedef uint32_t u4_t __attribute__((ext_vector_type(4)));  // stays in registers through a loop (a uint4 member did not)

struct StageRegs {
  u4_t k0, k1, v0, v1;
  float2 m;
};

// stage tokens [t0, t0 + 64) into registers; tokens past the capacity repeat
// its last rows
__device__ __forceinline__ void fetch_stage(const AttendArgs &a, const uint8_t *kf, const uint8_t *vf,
                                            const float2 *km, const float2 *vm, int t0, StageRegs &s) {
  const int i = threadIdx.x;
  const int64_t ta = min((int64_t)t0 + (i >> 3), a.tcap - 1), tb = min((int64_t)t0 + 32 + (i >> 3), a.tcap - 1);
  s.k0 = *(const u4_t *)(kf + ta * D + 16 * (i & 7));
  s.k1 = *(const u4_t *)(kf + tb * D + 16 * (i & 7));
  s.v0 = *(const u4_t *)(vf + ta * D + 16 * (i & 7));
  s.v1 = *(const u4_t *)(vf + tb * D + 16 * (i & 7));
  // four 16-token tiles: key ranges, value ranges (lanes 0 .. 7 store them)
  const int64_t blk = min(((int64_t)t0 + 16 * (i & 3)) >> a.bshift, a.nblk - 1);
  s.m = ((i & 4) ? vm : km)[blk];
}

// LDS of the token loop: a stage's keys are read from one unit before its
// values, so values take three buffers and keys two
constexpr int KBUF = 0, VBUF = 2 * CODES, MBUF = VBUF + 3 * CODES, LOBUF = MBUF + 3 * 64;

template <bool CENTRE_K>
__device__ __forceinline__ void put_stage(unsigned char *lds, int stage, int tmax, const StageRegs &s) {
  const int i = threadIdx.x;
  const int r = i >> 3, off = r * D + 16 * ((i & 7) ^ (r & 7));  // the same piece order 32 rows on
  unsigned char *k = lds + KBUF + (stage & 1) * CODES, *v = lds + VBUF + (stage % 3) * CODES;
  *(u4_t *)(k + off) = s.k0;
  *(u4_t *)(k + 32 * D + off) = s.k1;
  *(u4_t *)(v + off) = s.v0;
  *(u4_t *)(v + 32 * D + off) = s.v1;
  if (i < 8) {
    float2 m = s.m;
    if ((i & 4) || CENTRE_K) m.x = __builtin_fmaf(128.0f, m.y, m.x);  // the value of code 128
    if (stage * STAGE + 16 * (i & 3) >= tmax) m = make_float2(0.f, 0.f);  // a block that holds no row yet
    *(float2 *)(lds + MBUF + (stage % 3) * 64 + 8 * i) = m;
  }
}

struct TileState {
  float m, mu, mo, f, l, mv;  // as in attend_rows.hip, but mu is -inf while the row has seen nothing
};

// the weights of a unit and what goes with them
struct UnitWeights {
  float p[WT][2][4], ps[WT][2], w[WT][2];  // weights, their sums, value factors
  float mid[2];                            // the tiles' values of code 128
};

template <int J>
__device__ __forceinline__ h8_t value_frag(const uint2 (&v)[2][4]) {
  constexpr int B = J & 3;
  uint32_t w[2][4];
#pragma unroll
  for (int t = 0; t < 2; t++)
#pragma unroll
    for (int i = 0; i < 4; i++) w[t][i] = J < 4 ? v[t][i].x : v[t][i].y;
  return as_h8(centred(byte_pair<B>(w[0][0], w[0][1])), centred(byte_pair<B>(w[0][2], w[0][3])),
               centred(byte_pair<B>(w[1][0], w[1][1])), centred(byte_pair<B>(w[1][2], w[1][3])));
}

// scores of a unit: z = K Q^T from the key codes at kb
template <bool BF16, bool LO>
__device__ __forceinline__ void unit_scores(const unsigned char *kb, const QueryFrags (&q)[WT], const unsigned char *lo,
                                            f4_t (&z)[WT][2]) {
  const int lane = threadIdx.x & 63, row = lane & 15, grp = lane >> 4;
#pragma unroll
  for (int u = 0; u < 2; u++) {
    f4_t zl[WT];
#pragma unroll
    for (int t = 0; t < WT; t++) zl[t] = z[t][u] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < 2; x++) {
      const uint4 w = *(const uint4 *)(kb + (16 * u + row) * D + 16 * ((4 * x + grp) ^ (row & 7)));
      const h8_t c0 = codes8<!BF16>(w.x, w.y), c1 = codes8<!BF16>(w.z, w.w);
#pragma unroll
      for (int t = 0; t < WT; t++) {
        z[t][u] = mfma(c0, q[t].hi[2 * x], z[t][u]);
        z[t][u] = mfma(c1, q[t].hi[2 * x + 1], z[t][u]);
        if constexpr (LO) {
          zl[t] = mfma(c0, *(const h8_t *)(lo + (4 * t + 2 * x) * 1024), zl[t]);
          zl[t] = mfma(c1, *(const h8_t *)(lo + (4 * t + 2 * x + 1) * 1024), zl[t]);
        }
      }
    }
    if constexpr (LO) {
#pragma unroll
      for (int t = 0; t < WT; t++) z[t][u] += zl[t];
    }
  }
}

// weights of a unit; vis[t]: tokens of the unit, less 4 grp, that this lane's row
// sees (MASKED).  Returns whether some weight is too large for its scale (or
// infinite: a row that has seen nothing yet).
template <bool MASKED>
__device__ __forceinline__ bool unit_weights(const float2 *mt, const QueryFrags (&q)[WT], const f4_t (&z)[WT][2],
                                             const int (&vis)[WT], const TileState (&st)[WT], UnitWeights &o) {
  float over = 0.0f;
  float2 mk[2], mv[2];
#pragma unroll
  for (int u = 0; u < 2; u++) {
    mk[u] = mt[u];
    mv[u] = mt[4 + u];
    o.mid[u] = mv[u].x;
  }
#pragma unroll
  for (int t = 0; t < WT; t++) {
#pragma unroll
    for (int u = 0; u < 2; u++) {
      const float A = mk[u].y * q[t].ca, B = __builtin_fmaf(mk[u].x, q[t].cq, -st[t].mu);
#pragma unroll
      for (int r = 0; r < 4; r++) {
        const float s = __builtin_fmaf(z[t][u][r], A, B);
        o.p[t][u][r] = exp2_fast(MASKED && 16 * u + r >= vis[t] ? -INFINITY : s);
      }
      o.ps[t][u] = (o.p[t][u][0] + o.p[t][u][1]) + (o.p[t][u][2] + o.p[t][u][3]);
      o.w[t][u] = mv[u].y * st[t].f;
    }
    over = fmaxf(fmaxf(over, (o.ps[t][0] + o.ps[t][1]) * 128.0f),
                 fmaxf(o.ps[t][0] * o.w[t][0], o.ps[t][1] * o.w[t][1]));
  }
  return over > 32768.0f;
}

// raise the rows' maxima to the unit's scores, rescale what was summed, and
// form the unit's weights again (rare: the scores are not kept for it)
template <bool BF16, bool LO>
__device__ __forceinline__ void raise(const unsigned char *kb, const unsigned char *lo, const float2 *mt,
                                      const QueryFrags (&q)[WT], const int (&vis)[WT], TileState (&st)[WT],
                                      f4_t (&acc)[WT][8], UnitWeights &o) {
  f4_t z[WT][2];
  uint32_t again = 0;  // unknown to the compiler: the operands of the rare second product are not kept for it
  asm volatile("" : "+v"(again));
  unit_scores<BF16, LO>(kb + again, q, lo + again, z);
  o.mid[0] = mt[4].x;
  o.mid[1] = mt[5].x;
#pragma unroll
  for (int t = 0; t < WT; t++) {
    float s[2][4], mx[2], lv[2];
#pragma unroll
    for (int u = 0; u < 2; u++) {
      const float A = mt[u].y * q[t].ca, B = mt[u].x * q[t].cq;
#pragma unroll
      for (int r = 0; r < 4; r++) s[u][r] = 16 * u + r < vis[t] ? __builtin_fmaf(z[t][u][r], A, B) : -INFINITY;
      mx[u] = fmaxf(fmaxf(s[u][0], s[u][1]), fmaxf(s[u][2], s[u][3]));
      lv[u] = __builtin_amdgcn_logf(mt[4 + u].y);
    }
    const float mn = fmaxf(st[t].m, row_max(fmaxf(mx[0], mx[1])));
    float on = fmaxf(st[t].mo, row_max(fmaxf(mx[0] + lv[0], mx[1] + lv[1])));
    const bool some = mn > -INFINITY;
    if (some) on = fmaxf(on, mn - 80.0f);
    const float al = st[t].m > -INFINITY ? exp2_fast(st[t].m - mn) : 0.0f;
    const float ao = st[t].mo > -INFINITY ? exp2_fast(st[t].mo - on) : 0.0f;
    st[t].l *= al;
    st[t].mv *= al;
#pragma unroll
    for (int j = 0; j < 8; j++) acc[t][j] *= ao;
    st[t].m = st[t].mu = mn;
    st[t].mo = on;
    st[t].f = some ? exp2_fast(mn - on + 9.0f) : 1.0f;
    const float mu = some ? mn : 0.0f;
#pragma unroll
    for (int u = 0; u < 2; u++) {
#pragma unroll
      for (int r = 0; r < 4; r++) o.p[t][u][r] = exp2_fast(s[u][r] - mu);
      o.ps[t][u] = (o.p[t][u][0] + o.p[t][u][1]) + (o.p[t][u][2] + o.p[t][u][3]);
      o.w[t][u] = mt[4 + u].y * st[t].f;
    }
  }
}

// a unit's weights as operands, its sums into the rows' state
template <bool BF16>
struct UnitOperands {
  h8_t hi[WT], lo[WT];  // lo: fp32 storage only
};

template <bool BF16>
__device__ __forceinline__ void take_weights(const UnitWeights &o, TileState (&st)[WT], UnitOperands<BF16> &P) {
#pragma unroll
  for (int t = 0; t < WT; t++) {
    uint32_t ph[2][2], pl[2][2];
    st[t].l += o.ps[t][0] + o.ps[t][1];
#pragma unroll
    for (int u = 0; u < 2; u++) {
      st[t].mv = __builtin_fmaf(o.mid[u], o.ps[t][u], st[t].mv);
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const float x = o.p[t][u][2 * k] * o.w[t][u], y = o.p[t][u][2 * k + 1] * o.w[t][u];
        ph[u][k] = pack_f16x2(x, y);
        if constexpr (!BF16) {
          const f2_t hh = unpack_f16x2(ph[u][k]);
          pl[u][k] = pack_f16x2(x - hh.x, y - hh.y);
        }
      }
    }
    P.hi[t] = as_h8(ph[0][0], ph[0][1], ph[1][0], ph[1][1]);
    if constexpr (!BF16) P.lo[t] = as_h8(pl[0][0], pl[0][1], pl[1][0], pl[1][1]);
  }
}

// acc += V^T P^T of a unit, from the value codes at vl[i] (lane offsets of tokens
// 4 grp + i; the second tile 16 rows on)
template <bool BF16>
__device__ __forceinline__ void unit_values(const unsigned char *vb, const int (&vl)[4], const UnitOperands<BF16> &P,
                                            f4_t (&acc)[WT][8]) {
  uint2 v[2][4];
#pragma unroll
  for (int u = 0; u < 2; u++)
#pragma unroll
    for (int i = 0; i < 4; i++) v[u][i] = *(const uint2 *)(vb + vl[i] + 16 * D * u);
#define CG_PV(J)                                                   \
  {                                                                \
    const h8_t vj = value_frag<J>(v);                              \
    _Pragma("unroll") for (int t = 0; t < WT; t++) {               \
      acc[t][J] = mfma(vj, P.hi[t], acc[t][J]);                       \
      if constexpr (!BF16) acc[t][J] = mfma(vj, P.lo[t], acc[t][J]); \
    }                                                              \
  }
  CG_PV(0) CG_PV(1) CG_PV(2) CG_PV(3) CG_PV(4) CG_PV(5) CG_PV(6) CG_PV(7)
#undef CG_PV
}

// LO: the queries' second fp16 part takes part (fp32 storage, or where log-sums
// or weights are asked for); else a query is rounded to 2^-11 of a channel
template <bool BF16, bool LO>
__global__ __launch_bounds__(NTH, 2) void k_attend_tile(const AttendArgs a) {
  static_assert(BF16 || LO, "fp32 storage takes both parts");
  constexpr int LOOP_LDS = LOBUF + (LO ? 4 * WT * 4096 : 0), END_LDS = TROWS * PITCH * 4;
  __shared__ __align__(16) unsigned char lds[LOOP_LDS > END_LDS ? LOOP_LDS : END_LDS];
  const int lane = threadIdx.x & 63, row = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fields = a.batch * a.heads, groups = (a.rows + TROWS - 1) / TROWS;
  int64_t id = blockIdx.x;
  const int bh = (int)(id % fields);  // a head's workgroups share an XCD's L2 where the heads are a multiple of 8
  id /= fields;
  const int split = (int)(id % a.splits);
  const int grpi = groups - 1 - (int)(id / a.splits);  // the longest first
  const int h = bh % a.heads, b = bh / a.heads;
  const int r0 = grpi * TROWS, nr = min(TROWS, a.rows - r0);
  const int len = seq_length(a, b);

  const uint8_t *kf = a.kpay + (int64_t)bh * a.tcap * D, *vf = a.vpay + (int64_t)bh * a.tcap * D;
  const float2 *km = a.kmeta + (int64_t)bh * a.nblk, *vm = a.vmeta + (int64_t)bh * a.nblk;
  const int tmax = limit_of(a, b, len, r0 / a.ratio, (r0 + nr - 1) / a.ratio);
  const int stages = (tmax + STAGE - 1) / STAGE;
  const int s0 = (int)((int64_t)stages * split / a.splits), s1 = (int)((int64_t)stages * (split + 1) / a.splits);
  StageRegs nx;
  if (s0 < s1) fetch_stage(a, kf, vf, km, vm, s0 * STAGE, nx);

  // gauged queries as operands (a wave past the last tile takes the last one's)
  QueryFrags q[WT];
#pragma unroll
  for (int t = 0; t < WT; t++) {
    const int tile = min((r0 >> 4) + wave * WT + t, a.tiles - 1);
    const uint4 *f = a.qfrag + ((int64_t)bh * a.tiles + tile) * 8 * 64 + lane;
    const float2 x = a.qrow[((int64_t)bh * a.tiles + tile) * ROWS + row];
    q[t].ca = x.x * (BF16 ? kCodeUnit : kCentredUnit);
    q[t].cq = x.y;
#pragma unroll
    for (int s = 0; s < 4; s++) {
      q[t].hi[s] = __builtin_bit_cast(h8_t, f[s * 64]);
      if constexpr (LO) *(uint4 *)(lds + LOBUF + ((wave * WT + t) * 4 + s) * 1024 + lane * 16) = f[(4 + s) * 64];
    }
  }
  int lim[WT], all = tmax;  // what the lane's rows see; rows that are not there see everything
#pragma unroll
  for (int t = 0; t < WT; t++) {
    const int r = r0 + (wave * WT + t) * ROWS + row;
    lim[t] = r < a.rows ? query_limit(a, b, len, r / a.ratio) : tmax;
    all = min(all, lim[t]);
  }
#pragma unroll
  for (int k = 1; k < 16; k <<= 1) all = min(all, __shfl_xor(all, k));
  all = __builtin_amdgcn_readfirstlane(all);

  TileState st[WT];
  f4_t acc[WT][8];
#pragma unroll
  for (int t = 0; t < WT; t++) {
    st[t].m = st[t].mo = st[t].mu = -INFINITY;
    st[t].l = st[t].mv = 0.0f;
    st[t].f = 1.0f;
#pragma unroll
    for (int j = 0; j < 8; j++) acc[t][j] = f4_t{0.f, 0.f, 0.f, 0.f};
  }
  const unsigned char *lo = lds + LOBUF + wave * WT * 4096 + lane * 16;
  int vl[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int r = 4 * grp + i;
    vl[i] = r * D + 16 * ((row >> 1) ^ (r & 7)) + 8 * (row & 1);
  }
  const auto keys_at = [&](int un) { return lds + KBUF + ((un >> 1) & 1) * CODES + (un & 1) * UNIT * D; };
  const auto values_at = [&](int un) { return lds + VBUF + ((un >> 1) % 3) * CODES + (un & 1) * UNIT * D; };
  const auto ranges_at = [&](int un) { return (const float2 *)(lds + MBUF + ((un >> 1) % 3) * 64) + (un & 1) * 2; };

  // One unit ahead: a turn forms the scores and weights of the next unit beside
  // the value product of the present one, so matrix and vector work of both
  // lie in one block for the scheduler.
  if (s0 < s1) {
    const int u0 = 2 * s0, u1 = min(2 * s1, (tmax + UNIT - 1) / UNIT);
    UnitWeights o;
    UnitOperands<BF16> P;
    int vis[WT];
    put_stage<!BF16>(lds, s0, tmax, nx);
    if (s0 + 1 < s1) fetch_stage(a, kf, vf, km, vm, (s0 + 1) * STAGE, nx);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < WT; t++) vis[t] = lim[t] - u0 * UNIT - 4 * grp;
    raise<BF16, LO>(keys_at(u0), lo, ranges_at(u0), q, vis, st, acc, o);
    const auto turn = [&](int un, auto masked) {
      if (un & 1) {
        __syncthreads();  // the next stage is there
      } else {
        const int sg = un >> 1;
        if (sg + 1 < s1) put_stage<!BF16>(lds, sg + 1, tmax, nx);
        if (sg + 2 < s1) fetch_stage(a, kf, vf, km, vm, (sg + 2) * STAGE, nx);
      }
      const float2 *mt = ranges_at(un + 1);
#pragma unroll
      for (int t = 0; t < WT; t++) vis[t] = lim[t] - (un + 1) * UNIT - 4 * grp;
      take_weights<BF16>(o, st, P);
      f4_t z[WT][2];
      unit_scores<BF16, LO>(keys_at(un + 1), q, lo, z);
      unit_values<BF16>(values_at(un), vl, P, acc);
      const bool up = unit_weights<decltype(masked)::value>(mt, q, z, vis, st, o);
      if (__any(up)) raise<BF16, LO>(keys_at(un + 1), lo, mt, q, vis, st, acc, o);
    };
    // units that every row of the wave sees whole, then the others
    const int ua = min(u1 - 1, max(all / UNIT - 1, u0));
    for (int un = u0; un < ua; un++) turn(un, std::false_type{});
    for (int un = max(ua, u0); un + 1 < u1; un++) turn(un, std::true_type{});
    take_weights<BF16>(o, st, P);
    unit_values<BF16>(values_at(u1 - 1), vl, P, acc);
  }
  __syncthreads();

  // rows' sums, scaled as they stand, into LDS; then parts or outputs
  float *us = (float *)lds;
#pragma unroll
  for (int t = 0; t < WT; t++) {
    const int rr = (wave * WT + t) * ROWS + row;
    const float L = row_sum(st[t].l), mvs = row_sum(st[t].mv);
    const bool some = st[t].m > -INFINITY;
    const float inv = a.splits > 1 ? 1.0f : L > 0.0f ? 1.0f / L : 0.0f;
    const float ks = some ? inv * exp2_fast(st[t].mo - st[t].m) : 0.0f;
    const float k = some ? inv * mvs : 0.0f;
#pragma unroll
    for (int r = 0; r < 4; r++) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; j++) v[j] = __builtin_fmaf(acc[t][j][r], ks, k);
      float *o = us + rr * PITCH + 8 * (4 * grp + r);
      *(float4 *)o = make_float4(v[0], v[1], v[2], v[3]);
      *(float4 *)(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
    if (grp == 0 && rr < nr) {
      if (a.splits > 1) {
        a.part_ml[((int64_t)bh * a.splits + split) * a.rows + r0 + rr] = make_float2(st[t].m, L);
      } else {
        if (a.lse) store_lse(a, b, h, r0 + rr, st[t].m, L);
        if (a.lse2) a.lse2[(int64_t)bh * a.rows + r0 + rr] = L > 0.0f ? st[t].m + __builtin_log2f(L) : INFINITY;
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
  for (int t = 0; t * ROWS < nr; t++)
    gauge_rows<true>(us + t * ROWS * PITCH, min(ROWS, nr - t * ROWS), a.gv + (int64_t)h * D * a.g, a.g,
                     [&](int r, int c, float v) { store_out<BF16>(a, b, h, r0 + t * ROWS + r, c, v); });
}

// One workgroup per four row tiles: gauge, split into the operands' parts and
// store in operand order, with each row's factors.
template <bool BF16, bool LO>
__global__ __launch_bounds__(NTH) void k_attend_prepare(const AttendArgs a) {
  __shared__ __align__(16) float xs[4][ROWS * PITCH], ys[4][ROWS * PITCH];
  const int quads = (a.tiles + 3) / 4;
  const int64_t id = blockIdx.x;
  const int tile0 = (int)(id % quads) * 4, bh = (int)(id / quads);
  const int h = bh % a.heads, b = bh / a.heads;
#pragma unroll
  for (int t = 0; t < 4; t++) load_rows<BF16>(a, b, h, (tile0 + t) * ROWS, xs[t]);
  __syncthreads();
#pragma unroll 1
  for (int t = 0; t < 4; t++)
    gauge_rows<false>(xs[t], ROWS, a.gk + (int64_t)h * D * a.g, a.g,
                      [&](int r, int c, float v) { ys[t][r * PITCH + c] = v; });
  __syncthreads();
  const int lane = threadIdx.x & 63, tile = tile0 + (int)(threadIdx.x >> 6);
  if (tile >= a.tiles) return;
  QueryFrags q;
  make_frags<LO>(ys[threadIdx.x >> 6], a.c, q);
  uint4 *d = a.qfrag + ((int64_t)bh * a.tiles + tile) * 8 * 64 + lane;
#pragma unroll
  for (int s = 0; s < 4; s++) {
    d[s * 64] = __builtin_bit_cast(uint4, q.hi[s]);
    if constexpr (LO) d[(4 + s) * 64] = __builtin_bit_cast(uint4, q.lo[s]);
  }
  if (lane < ROWS) a.qrow[((int64_t)bh * a.tiles + tile) * ROWS + lane] = make_float2(q.ca, q.cq);
}

hipError_t tile_launch(const AttendArgs &a, bool bf16, hipStream_t s) {
  const int64_t groups = (a.rows + TROWS - 1) / TROWS;
  const dim3 grid((unsigned)((int64_t)a.batch * a.heads * groups * a.splits)), block(NTH);
  const dim3 pre((unsigned)((int64_t)a.batch * a.heads * ((a.tiles + 3) / 4)));
  if (!bf16) {
    hipLaunchKernelGGL((k_attend_prepare<false, true>), pre, block, 0, s, a);
    hipLaunchKernelGGL((k_attend_tile<false, true>), grid, block, 0, s, a);
  } else if (a.lse || a.mass) {
    hipLaunchKernelGGL((k_attend_prepare<true, true>), pre, block, 0, s, a);
    hipLaunchKernelGGL((k_attend_tile<true, true>), grid, block, 0, s, a);
  } else {
    hipLaunchKernelGGL((k_attend_prepare<true, false>), pre, block, 0, s, a);
    hipLaunchKernelGGL((k_attend_tile<true, false>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace cga
