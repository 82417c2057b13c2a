// Attention of up to 16 query rows (a row tile) over the 8-bit cache, split
// along the tokens: the form for single tokens and few drafted ones, bound by
// the memory traffic of the codes.
//
// A workgroup takes one part of one field pair's tokens for one row tile; its
// four waves take the part's 32-token units in turn and join at the end.  Per
// unit a wave computes S^T = K Q^T (tokens x rows), turns its scores into
// weights in registers and feeds them as they lie to O^T = V^T P^T: lane
// (row = lane % 16, grp = lane / 16) holds the scores of tokens 4 grp + 0..3
// of both 16-token tiles, which are the eight contraction slots of that lane
// in the second product once V's tokens are numbered the same way.  All of a
// row's state is in the four lanes of that row, so the running maximum needs
// no exchange until it is raised: it is raised only when a score passes it by
// more than 2^8 (weights stay within fp16 either way), which is rare after
// the first units.
//
// V's weights are p_t sv_b in fp16.  Their scale is kept apart from the sum's:
// `m` follows the scores, `mo` the scores plus log2 sv_b, so that blocks of
// unlike steps keep 11 significant bits each.  The largest weight lies between
// 2^9 and 2^15: below 2^-14 a weight is rounded to multiples of 2^-24, which
// is 2^-33 of the largest.
#include "attend.hpp"

namespace cga {

struct RawUnit {
  uint4 k[2][2];  // [tile][half row]: token 16 tile + lane % 16, codes 64 x + 16 grp ..
  uint2 v[2][4];  // [tile][i]: token 16 tile + 4 grp + i, codes 8 (lane % 16) ..
  float2 km[2], vm[2];
};

__device__ __forceinline__ void load_unit(const AttendArgs &a, const uint8_t *kf, const uint8_t *vf,
                                          const float2 *km, const float2 *vm, int t0, RawUnit &u) {
  const int lane = threadIdx.x & 63, n = lane & 15, grp = lane >> 4;
  const uint8_t *kb = kf + (int64_t)t0 * D, *vb = vf + (int64_t)t0 * D;
  if ((int64_t)t0 + UNIT <= a.tcap) {
#pragma unroll
    for (int t = 0; t < 2; t++) {
#pragma unroll
      for (int x = 0; x < 2; x++) u.k[t][x] = *(const uint4 *)(kb + (16 * t + n) * D + 64 * x + 16 * grp);
#pragma unroll
      for (int i = 0; i < 4; i++) u.v[t][i] = *(const uint2 *)(vb + (16 * t + 4 * grp + i) * D + 8 * n);
    }
  } else {  // 16-token blocks: the capacity ends after the unit's first tile
#pragma unroll
    for (int t = 0; t < 2; t++) {
#pragma unroll
      for (int x = 0; x < 2; x++) u.k[t][x] = *(const uint4 *)(kb + n * D + 64 * x + 16 * grp);
#pragma unroll
      for (int i = 0; i < 4; i++) u.v[t][i] = *(const uint2 *)(vb + (4 * grp + i) * D + 8 * n);
    }
  }
#pragma unroll
  for (int t = 0; t < 2; t++) {
    const int64_t blk = min((int64_t)(t0 + 16 * t) >> a.bshift, a.nblk - 1);
    u.km[t] = km[blk];
    u.vm[t] = vm[blk];
  }
}

template <int J>
__device__ __forceinline__ h8_t value_frag(const RawUnit &u) {
  constexpr int B = J & 3;
  uint32_t w[2][4];
#pragma unroll
  for (int t = 0; t < 2; t++)
#pragma unroll
    for (int i = 0; i < 4; i++) w[t][i] = J < 4 ? u.v[t][i].x : u.v[t][i].y;
  return as_h8(centred(byte_pair<B>(w[0][0], w[0][1])), centred(byte_pair<B>(w[0][2], w[0][3])),
               centred(byte_pair<B>(w[1][0], w[1][1])), centred(byte_pair<B>(w[1][2], w[1][3])));
}

// a row's running state, the same in its four lanes but for l and mv
struct RowState {
  float m, mu, mo, f;   // maximum, the one used (0 while none), value scale, 2^(mu - mo + 9)
  float l, mv;          // this lane's part of the sums of p and of p mv_b
};

// fp32 storage: the weights in two fp16 parts, the keys' codes centred like the
// values' (scores to 2^-22 of the sum of |q'| 255 step; uncentred 10 times
// that).  bf16 storage: the weights are one fp16 part (2^-11 of a weight).
template <bool BF16, bool MASS>
__global__ __launch_bounds__(NTH) void k_attend_rows(const AttendArgs a) {
  __shared__ __align__(16) float lds[4 * ROWS * PITCH];
  __shared__ float2 ml[4][ROWS];
  const int lane = threadIdx.x & 63, row = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t id = blockIdx.x;
  const int split = (int)(id % a.splits);
  id /= a.splits;
  const int tile = (int)(id % a.tiles);
  id /= a.tiles;
  const int h = (int)(id % a.heads), b = (int)(id / a.heads);
  const int bh = b * a.heads + h;
  const int r0 = tile * ROWS, nr = min(ROWS, a.rows - r0);
  // on their way first: what does not wait for the sequence's length
  const float *gk = a.gk + (int64_t)h * D * a.g;
  const RowPart qp = load_row_part<BF16>(a, b, h, r0);
  GaugeWeights gw;
  load_gauge<false>(gk, a.g, 0, gw);
  const int len = seq_length(a, b);
  const int tmax = limit_of(a, b, len, r0 / a.ratio, (r0 + nr - 1) / a.ratio);
  const int units = (tmax + UNIT - 1) / UNIT;
  const int u0 = (int)((int64_t)units * split / a.splits), u1 = (int)((int64_t)units * (split + 1) / a.splits);

  const uint8_t *kf = a.kpay + (int64_t)bh * a.tcap * D, *vf = a.vpay + (int64_t)bh * a.tcap * D;
  const float2 *km = a.kmeta + (int64_t)bh * a.nblk, *vm = a.vmeta + (int64_t)bh * a.nblk;

  RawUnit nx;
  if (u0 + wave < u1) load_unit(a, kf, vf, km, vm, (u0 + wave) * UNIT, nx);

  // gauged query rows
  float *xs = lds, *ys = lds + ROWS * PITCH;
  put_row_part(xs, qp);
  if (nr < ROWS)
    for (int i = threadIdx.x; i < (ROWS - nr) * D; i += NTH) ys[(nr + (i >> 7)) * PITCH + (i & 127)] = 0.0f;
  __syncthreads();
  gauge_rows<false, ROWS>(xs, nr, gk, a.g, gw, [&](int r, int c, float v) { ys[r * PITCH + c] = v; });
  __syncthreads();
  QueryFrags q;
  make_frags<true, true>(ys, a.c, q);
  q.ca *= BF16 ? kCodeUnit : kCentredUnit;
  __syncthreads();

  // what this lane's row sees; rows that are not there see everything, and
  // are never stored
  const int lim = row < nr ? query_limit(a, b, len, (r0 + row) / a.ratio) : tmax;
  int all = lim;
#pragma unroll
  for (int k = 1; k < 16; k <<= 1) all = min(all, __shfl_xor(all, k));
  all = __builtin_amdgcn_readfirstlane(all);  // every row sees the tokens before it

  RowState st;
  st.m = st.mo = -INFINITY;
  st.mu = 0.0f;
  st.f = 1.0f;
  st.l = st.mv = 0.0f;
  f4_t acc[8];
#pragma unroll
  for (int j = 0; j < 8; j++) acc[j] = f4_t{0.f, 0.f, 0.f, 0.f};

  for (int un = u0 + wave; un < u1; un += 4) {
    const RawUnit u = nx;
    const int t0 = un * UNIT;
    if (un + 4 < u1) load_unit(a, kf, vf, km, vm, t0 + 4 * UNIT, nx);
    float s[2][4];
#pragma unroll
    for (int t = 0; t < 2; t++) {
      f4_t z = f4_t{0.f, 0.f, 0.f, 0.f}, zl = z;
#pragma unroll
      for (int x = 0; x < 2; x++) {
        const h8_t c0 = codes8<!BF16>(u.k[t][x].x, u.k[t][x].y), c1 = codes8<!BF16>(u.k[t][x].z, u.k[t][x].w);
        z = mfma(c0, q.hi[2 * x], z);
        z = mfma(c1, q.hi[2 * x + 1], z);
        zl = mfma(c0, q.lo[2 * x], zl);
        zl = mfma(c1, q.lo[2 * x + 1], zl);
      }
      z += zl;
      const float A = u.km[t].y * q.ca, Bm = (BF16 ? u.km[t].x : __builtin_fmaf(128.0f, u.km[t].y, u.km[t].x)) * q.cq;
#pragma unroll
      for (int r = 0; r < 4; r++) s[t][r] = __builtin_fmaf(z[r], A, Bm);
    }
    float vst[2], vmn[2];
#pragma unroll
    for (int t = 0; t < 2; t++) {
      vst[t] = u.vm[t].y;
      vmn[t] = __builtin_fmaf(128.0f, u.vm[t].y, u.vm[t].x);  // the value of code 128
    }
    if (t0 + UNIT > all) {
#pragma unroll
      for (int t = 0; t < 2; t++) {
        if (t0 + 16 * t >= tmax) vst[t] = vmn[t] = 0.0f;  // a block that holds no row yet
#pragma unroll
        for (int r = 0; r < 4; r++)
          s[t][r] = t0 + 16 * t + 4 * grp + r < lim ? s[t][r] : -INFINITY;
      }
    }
    float mx[2], lv[2];
#pragma unroll
    for (int t = 0; t < 2; t++) {
      mx[t] = fmaxf(fmaxf(s[t][0], s[t][1]), fmaxf(s[t][2], s[t][3]));
      lv[t] = __builtin_amdgcn_logf(vst[t]);  // log2; -inf for a constant block
    }
    const float top = fmaxf(mx[0], mx[1]), topv = fmaxf(mx[0] + lv[0], mx[1] + lv[1]);
    if (__any(top > st.m + 8.0f || topv > st.mo + 6.0f)) {
      const float mn = fmaxf(st.m, row_max(top));
      float on = fmaxf(st.mo, row_max(topv));
      const bool some = mn > -INFINITY;
      if (some) on = fmaxf(on, mn - 80.0f);  // keeps 2^(m - mo) finite beside weights that vanish
      const float mu = some ? mn : 0.0f;
      const float al = st.m > -INFINITY ? exp2_fast(st.m - mn) : 0.0f;
      const float ao = st.mo > -INFINITY ? exp2_fast(st.mo - on) : 0.0f;
      st.l *= al;
      st.mv *= al;
#pragma unroll
      for (int j = 0; j < 8; j++) acc[j] *= ao;
      st.m = mn;
      st.mo = on;
      st.mu = mu;
      st.f = some ? exp2_fast(mn - on + 9.0f) : 1.0f;
    }
    uint32_t ph[2][2], pl[2][2];
    float bs[2];
#pragma unroll
    for (int t = 0; t < 2; t++) {
      float p[4];
#pragma unroll
      for (int r = 0; r < 4; r++) p[r] = exp2_fast(s[t][r] - st.mu);
      bs[t] = (p[0] + p[1]) + (p[2] + p[3]);
      st.l += bs[t];
      st.mv = __builtin_fmaf(vmn[t], bs[t], st.mv);
      const float w = vst[t] * st.f;
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const float x = p[2 * k] * w, y = p[2 * k + 1] * w;
        ph[t][k] = pack_f16x2(x, y);
        if constexpr (!BF16) {
          const f2_t hh = unpack_f16x2(ph[t][k]);
          pl[t][k] = pack_f16x2(x - hh.x, y - hh.y);
        }
      }
    }
    if constexpr (MASS) {
      if (a.bshift == 4) {
#pragma unroll
        for (int t = 0; t < 2; t++) {
          const float v = row_sum(bs[t]);
          const int64_t e = (t0 >> 4) + t;
          if (grp == 0 && row < nr && e < a.entries)
            a.bsum[((int64_t)bh * a.entries + e) * a.rows + r0 + row] = make_float2(v, st.mu);
        }
      } else {
        const float v = row_sum(bs[0] + bs[1]);
        if (grp == 0 && row < nr)
          a.bsum[((int64_t)bh * a.entries + (t0 >> 5)) * a.rows + r0 + row] = make_float2(v, st.mu);
      }
    }
    const h8_t P = as_h8(ph[0][0], ph[0][1], ph[1][0], ph[1][1]);
    h8_t Pl;
    if constexpr (!BF16) Pl = as_h8(pl[0][0], pl[0][1], pl[1][0], pl[1][1]);
#define CG_PV(J)                                        \
  {                                                     \
    const h8_t vj = value_frag<J>(u);                   \
    acc[J] = mfma(vj, P, acc[J]);                       \
    if constexpr (!BF16) acc[J] = mfma(vj, Pl, acc[J]); \
  }
    CG_PV(0) CG_PV(1) CG_PV(2) CG_PV(3) CG_PV(4) CG_PV(5) CG_PV(6) CG_PV(7)
#undef CG_PV
  }

  // join the waves: rows' sums relative to the workgroup's maximum
  const float l = row_sum(st.l), mv = row_sum(st.mv);
  if (grp == 0) ml[wave][row] = make_float2(st.m, l);
  __syncthreads();
  float M = -INFINITY, Lw = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; w++) M = fmaxf(M, ml[w][row].x);
#pragma unroll
  for (int w = 0; w < 4; w++) Lw += ml[w][row].x > -INFINITY ? ml[w][row].y * exp2_fast(ml[w][row].x - M) : 0.0f;
  {
    const bool some = st.m > -INFINITY;
    const float k = some ? exp2_fast(st.m - M) : 0.0f;
    // true sums: acc 2^9 / f (the codes' and the weights' scales)
    const float ks = some ? k * exp2_fast(st.mo - st.m) : 0.0f;
    float *o = lds + (wave * ROWS + row) * PITCH;
#pragma unroll
    for (int r = 0; r < 4; r++) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; j++) v[j] = acc[j][r] * ks + mv * k;
      *(float4 *)(o + 8 * (4 * grp + r)) = make_float4(v[0], v[1], v[2], v[3]);
      *(float4 *)(o + 8 * (4 * grp + r) + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
  __syncthreads();
  if (wave == 0 && grp == 0 && row < nr) {
    const int64_t pr = ((int64_t)bh * a.splits + split) * a.rows + r0 + row;
    if (a.part_ml) a.part_ml[pr] = make_float2(M, Lw);
    if (a.splits == 1 && a.lse) store_lse(a, b, h, r0 + row, M, Lw);
    if (a.splits == 1 && a.lse2) a.lse2[(int64_t)bh * a.rows + r0 + row] = Lw > 0.0f ? M + __builtin_log2f(Lw) : INFINITY;
    ml[0][row] = make_float2(M, Lw);
  }
  if (a.splits > 1) {
    for (int i = threadIdx.x; i < nr * (D / 4); i += NTH) {
      const int r = i / (D / 4), c = 4 * (i % (D / 4));
      float4 v = *(const float4 *)(lds + r * PITCH + c);
#pragma unroll
      for (int w = 1; w < 4; w++) {
        const float4 x = *(const float4 *)(lds + (w * ROWS + r) * PITCH + c);
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      }
      *(float4 *)(a.part_o + (((int64_t)bh * a.splits + split) * a.rows + r0 + r) * D + c) = v;
    }
    return;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nr * (D / 4); i += NTH) {
    const int r = i / (D / 4), c = 4 * (i % (D / 4));
    const float ll = ml[0][r].y;
    const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
    float4 v = *(const float4 *)(lds + r * PITCH + c);
#pragma unroll
    for (int w = 1; w < 4; w++) {
      const float4 x = *(const float4 *)(lds + (w * ROWS + r) * PITCH + c);
      v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
    }
    v.x *= inv; v.y *= inv; v.z *= inv; v.w *= inv;
    *(float4 *)(lds + r * PITCH + c) = v;  // this thread alone reads row r's channels c .. c + 3
  }
  const float *gv = a.gv + (int64_t)h * D * a.g;
  load_gauge<true>(gv, a.g, 0, gw);
  __syncthreads();
  gauge_rows<true, ROWS>(lds, nr, gv, a.g, gw, [&](int r, int c, float v) { store_out<BF16>(a, b, h, r0 + r, c, v); });
}

// Joins the splits of one row, a workgroup to a row: 2^(m_s - M) of every
// split, eight groups of 32 lanes adding every eighth split's sums, then the
// inverse gauge.  For few rows with many splits.
template <bool BF16>
__global__ __launch_bounds__(NTH) void k_attend_merge(const AttendArgs a) {
  __shared__ __align__(16) float part[8][D];
  __shared__ __align__(16) float us[PITCH];
  __shared__ float wt[MERGE_SPLITS];
  __shared__ float2 red[4];
  const int64_t id = blockIdx.x;
  const int r = (int)(id % a.rows), bh = (int)(id / a.rows);
  const int h = bh % a.heads, b = bh / a.heads;
  const float2 *pm = a.part_ml + (int64_t)bh * a.splits * a.rows + r;
  const float *po = a.part_o + ((int64_t)bh * a.splits * a.rows + r) * D;
  const int S = a.splits, t = threadIdx.x;
  // this thread's part of G_V, on its way while the sums are joined
  const float *gv = a.gv + (int64_t)h * D * a.g;
  GaugeWeights gw;
  load_gauge<true>(gv, a.g, 0, gw);
  float M = -INFINITY;
  for (int s = t; s < S; s += NTH) M = fmaxf(M, pm[(int64_t)s * a.rows].x);
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) M = fmaxf(M, __shfl_xor(M, k));
  if ((t & 63) == 0) red[t >> 6].x = M;
  __syncthreads();
  M = fmaxf(fmaxf(red[0].x, red[1].x), fmaxf(red[2].x, red[3].x));
  float L = 0.0f;
  for (int s = t; s < S; s += NTH) {
    const float2 x = pm[(int64_t)s * a.rows];
    const float k = x.x > -INFINITY ? exp2_fast(x.x - M) : 0.0f;
    wt[s] = k;
    L += x.y * k;
  }
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) L += __shfl_xor(L, k);
  if ((t & 63) == 0) red[t >> 6].y = L;
  __syncthreads();
  L = (red[0].y + red[1].y) + (red[2].y + red[3].y);
  const int grp = t >> 5, c4 = 4 * (t & 31);
  float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = grp; s < S; s += 8) {
    const float k = wt[s];
    const float4 x = *(const float4 *)(po + (int64_t)s * a.rows * D + c4);
    u.x += x.x * k; u.y += x.y * k; u.z += x.z * k; u.w += x.w * k;
  }
  *(float4 *)&part[grp][c4] = u;
  __syncthreads();
  if (t == 0 && a.lse) store_lse(a, b, h, r, M, L);
  if (t < D) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k++) v += part[k][t];
    us[t] = L > 0.0f ? v / L : 0.0f;
  }
  __syncthreads();
  gauge_rows<true, 2>(us, 1, gv, a.g, gw, [&](int, int cc, float v) { store_out<BF16>(a, b, h, r, cc, v); });
}

// The same for many rows with few splits: 16 rows to a workgroup, a row to a
// wave at a time.
template <bool BF16>
__global__ __launch_bounds__(NTH) void k_attend_merge_many(const AttendArgs a) {
  __shared__ __align__(16) float us[ROWS * PITCH];
  const int64_t id = blockIdx.x;
  const int r0 = (int)(id % a.tiles) * ROWS, bh = (int)(id / a.tiles);
  const int h = bh % a.heads, b = bh / a.heads, nr = min(ROWS, a.rows - r0);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float *gv = a.gv + (int64_t)h * D * a.g;
  GaugeWeights gw;
  load_gauge<true>(gv, a.g, 0, gw);
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int rr = wave + 4 * i, r = min(r0 + rr, a.rows - 1);
    const float2 *pm = a.part_ml + (int64_t)bh * a.splits * a.rows + r;
    const float *po = a.part_o + ((int64_t)bh * a.splits * a.rows + r) * D + 2 * lane;
    float M = -INFINITY, L = 0.0f;
    for (int s = 0; s < a.splits; s++) M = fmaxf(M, pm[(int64_t)s * a.rows].x);
    float2 u = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < a.splits; s++) {
      const float2 x = pm[(int64_t)s * a.rows], y = *(const float2 *)(po + (int64_t)s * a.rows * D);
      const float k = x.x > -INFINITY ? exp2_fast(x.x - M) : 0.0f;
      L += x.y * k;
      u.x += y.x * k;
      u.y += y.y * k;
    }
    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
    *(float2 *)(us + rr * PITCH + 2 * lane) = make_float2(u.x * inv, u.y * inv);
    if (lane == 0 && rr < nr) {
      if (a.lse) store_lse(a, b, h, r, M, L);
      if (a.lse2) a.lse2[(int64_t)bh * a.rows + r] = L > 0.0f ? M + __builtin_log2f(L) : INFINITY;
    }
  }
  __syncthreads();
  gauge_rows<true, ROWS>(us, nr, gv, a.g, gw, [&](int r, int cc, float v) { store_out<BF16>(a, b, h, r0 + r, cc, v); });
}

// Block weights of few rows from the sums the attention left: mass[block] +=
// sum over rows of sum_t 2^(s_t - m) 2^(m - log2 sum)
__global__ __launch_bounds__(NTH) void k_mass_finish(const AttendArgs a) {
  __shared__ float lse2[ROWS];
  const int chunks = (int)((a.nblk + NTH - 1) / NTH);
  const int64_t id = blockIdx.x;
  const int bh = (int)(id / chunks), b = bh / a.heads;
  const int64_t blk = (id % chunks) * NTH + threadIdx.x;
  const int len = seq_length(a, b);
  const int tmax = limit_of(a, b, len, 0, a.n - 1);
  if ((int)threadIdx.x < a.rows) {
    const float2 *pm = a.part_ml + (int64_t)bh * a.splits * a.rows + threadIdx.x;
    float M = -INFINITY, L = 0.0f;
    for (int s = 0; s < a.splits; s++) M = fmaxf(M, pm[(int64_t)s * a.rows].x);
    for (int s = 0; s < a.splits; s++) {
      const float2 x = pm[(int64_t)s * a.rows];
      L += x.x > -INFINITY ? x.y * exp2_fast(x.x - M) : 0.0f;
    }
    lse2[threadIdx.x] = L > 0.0f ? M + __builtin_log2f(L) : INFINITY;
  }
  __syncthreads();
  if (blk >= a.nblk || (blk << a.bshift) >= tmax) return;
  const int per = a.bshift == 6 ? 2 : 1;
  float w = 0.0f;
  for (int k = 0; k < per; k++) {
    const int64_t e = blk * per + k;
    if (a.bshift != 4 && e * UNIT >= tmax) break;  // the unit was not visited
    const float2 *p = a.bsum + ((int64_t)bh * a.entries + e) * a.rows;
    for (int r = 0; r < a.rows; r++)
      if (p[r].x > 0.0f && lse2[r] < INFINITY) w += p[r].x * exp2_fast(p[r].y - lse2[r]);
  }
  a.mass[(int64_t)bh * a.nblk + blk] += w;
}

hipError_t rows_launch(const AttendArgs &a, bool bf16, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.batch * a.heads * a.tiles * a.splits)), block(NTH);
  const bool mass = a.mass && a.bsum;
  if (bf16 && mass) hipLaunchKernelGGL((k_attend_rows<true, true>), grid, block, 0, s, a);
  else if (bf16) hipLaunchKernelGGL((k_attend_rows<true, false>), grid, block, 0, s, a);
  else if (mass) hipLaunchKernelGGL((k_attend_rows<false, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_attend_rows<false, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t merge_launch(const AttendArgs &a, bool bf16, hipStream_t s) {
  const int64_t fields = (int64_t)a.batch * a.heads;
  if (a.tiles > 1) {
    const dim3 grid((unsigned)(fields * a.tiles)), block(NTH);
    if (bf16) hipLaunchKernelGGL(k_attend_merge_many<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_attend_merge_many<false>, grid, block, 0, s, a);
  } else {
    const dim3 grid((unsigned)(fields * a.rows)), block(NTH);
    if (bf16) hipLaunchKernelGGL(k_attend_merge<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_attend_merge<false>, grid, block, 0, s, a);
  }
  return hipGetLastError();
}

hipError_t mass_finish_launch(const AttendArgs &a, hipStream_t s) {
  const int64_t chunks = (a.nblk + NTH - 1) / NTH;
  const dim3 grid((unsigned)((int64_t)a.batch * a.heads * chunks)), block(NTH);
  hipLaunchKernelGGL(k_mass_finish, grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace cga
