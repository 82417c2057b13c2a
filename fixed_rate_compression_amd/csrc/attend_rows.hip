// Attention of few query rows (up to four row tiles of 16) over the 8-bit
// cache, split along the tokens: the form for single tokens and few drafted
// ones, bound by the memory traffic of the codes (of which the other
// tiles find most in the caches).
//
// A workgroup takes one part of one field pair's tokens for one row tile; its
// waves (four, or eight where that saves the splits) take the part's 32-token
// units in turn and join at the end.  Per
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
//
// 262144 tokens of 8 KV heads: 95 us, 5.6 TB/s of the 5.97 that a plain sum of the
// same bytes reaches, the codes read once.  16 sequences of 0 .. 8192 tokens 23 us
// (5.2 TB/s), with block sums 8 sequences of 0 .. 16384 31 us (4.5 TB/s: two
// workgroups a compute unit for the registers, three spill), one sequence of 1024
// tokens 11.3 us, all of it latency.
#include "attend.hpp"
#include "attend_few.hpp"

namespace cga {

// a unit's codes as they are loaded; the keys of the next unit are asked for as
// soon as this one's are used, and so the values
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));
struct RawKeys {
  u4_t k[2][2];  // [tile][half row]: token 16 tile + lane % 16, codes 64 x + 16 grp ..
  float2 m[2];
};
struct RawValues {
  u2_t v[2][4];  // [tile][i]: token 16 tile + 4 grp + i, codes 8 (lane % 16) ..
  float2 m[2];
};

// with 16-token blocks the capacity may end after the unit's first tile: its
// second then repeats the first
__device__ __forceinline__ void load_keys(const AttendArgs &a, const uint8_t *kf, const float2 *km, int t0, RawKeys &u) {
  const int lane = threadIdx.x & 63, n = lane & 15, grp = lane >> 4;
  const int second = (int64_t)t0 + UNIT <= a.tcap ? 16 : 0;
  const uint8_t *k0 = kf + (int64_t)t0 * D, *k1 = k0 + second * D;
#pragma unroll
  for (int x = 0; x < 2; x++) {
    u.k[0][x] = *(const u4_t *)(k0 + n * D + 64 * x + 16 * grp);
    u.k[1][x] = *(const u4_t *)(k1 + n * D + 64 * x + 16 * grp);
  }
  u.m[0] = km[(int64_t)t0 >> a.bshift];
  u.m[1] = km[((int64_t)t0 + second) >> a.bshift];
}

__device__ __forceinline__ void load_values(const AttendArgs &a, const uint8_t *vf, const float2 *vm, int t0, RawValues &u) {
  const int lane = threadIdx.x & 63, n = lane & 15, grp = lane >> 4;
  const int second = (int64_t)t0 + UNIT <= a.tcap ? 16 : 0;
  const uint8_t *v0 = vf + (int64_t)t0 * D, *v1 = v0 + second * D;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    u.v[0][i] = *(const u2_t *)(v0 + (4 * grp + i) * D + 8 * n);
    u.v[1][i] = *(const u2_t *)(v1 + (4 * grp + i) * D + 8 * n);
  }
  u.m[0] = vm[(int64_t)t0 >> a.bshift];
  u.m[1] = vm[((int64_t)t0 + second) >> a.bshift];
}

// c: the centres of the two tiles
template <int J>
__device__ __forceinline__ h8_t value_frag(const RawValues &u, const uint32_t (&c)[2]) {
  constexpr int B = J & 3;
  uint32_t w[2][4];
#pragma unroll
  for (int t = 0; t < 2; t++)
#pragma unroll
    for (int i = 0; i < 4; i++) w[t][i] = J < 4 ? u.v[t][i].x : u.v[t][i].y;
  return as_h8(centred(byte_pair<B>(w[0][0], w[0][1]), c[0]), centred(byte_pair<B>(w[0][2], w[0][3]), c[0]),
               centred(byte_pair<B>(w[1][0], w[1][1]), c[1]), centred(byte_pair<B>(w[1][2], w[1][3]), c[1]));
}

// a row's running state, the same in its four lanes but for l and mv
struct RowState {
  float m, mu, mo, f;   // maximum, the one used (0 while none), value scale, 2^(mu - mo + 9)
  float l, mv;          // this lane's part of the sums of p and of p mv_b
};

// fp32 storage: the weights in two fp16 parts, keys' and values' codes around the value 0
// (scores to 2^-22 of the sum of |q' k'|; with codes as they are 10 times that of
// |q'| 255 step).  bf16 storage: the weights are one fp16 part (2^-11 of a weight),
// the values' codes less 128.
template <bool BF16, bool MASS, int NW>
__global__ __launch_bounds__(64 * NW, NW == 4 && !MASS ? 3 : 2) void k_attend_rows(const AttendArgs a) {
  __shared__ __align__(16) float lds[NW * ROWS * PITCH];
  __shared__ float2 ml[NW][ROWS];
  const int lane = threadIdx.x & 63, row = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // 32-bit divisions: a 64-bit one takes longer than a unit of work
  const uint32_t id = blockIdx.x;
  int b, h, tile, slot = 0, split = 0, splits = a.splits;
  int64_t part;  // where this part's row 0 goes
  if (a.ragged) {  // row tiles of a slot and head on one XCD where the heads are a multiple of 8
    const uint32_t q1 = id / (uint32_t)a.heads, q2 = q1 / (uint32_t)a.tiles;
    h = (int)(id - q1 * a.heads);
    tile = (int)(q1 - q2 * a.tiles);
    slot = (int)q2;
    b = (int)(q2 * (uint32_t)a.batch / (uint32_t)a.slots);  // with equal lengths; found out below
    part = ((int64_t)h * a.slots + slot) * a.rows;
  } else {
    const uint32_t q1 = id / (uint32_t)splits;
    split = (int)(id - q1 * splits);
    const int f = a.tiles == 1 ? (int)q1 : (int)(q1 / (uint32_t)a.tiles);
    tile = (int)q1 - f * a.tiles;
    b = (int)((uint32_t)f / (uint32_t)a.heads);
    h = f - b * a.heads;
    part = ((int64_t)f * splits + split) * a.rows;
  }
  const int r0 = tile * ROWS, nr = min(ROWS, a.rows - r0);
  // on their way first: what does not wait for the sequence's length
  const float *gk = a.gk + (int64_t)h * D * a.g;
  const bool front = NW == 4 || wave < 4;  // the first four waves gauge the queries, and the outputs
  RowPart qp;
  GaugeFrag gw;
  if (front) {
    qp = load_row_part<BF16>(a, b, h, r0);
    load_gauge<false>(gk, a.g, 0, gw);
  }
  Sequence sq;
  if (a.ragged) {
    const Slot sl = find_slot(a, slot);
    if (sl.b >= a.batch) return;
    if (front && sl.b != b) qp = load_row_part<BF16>(a, sl.b, h, r0);
    b = sl.b;
    split = slot - sl.first;
    splits = sl.count;
    sq = sequence_of(a, sl.n, sl.p);
  }
  const FewPlace fp{b, h, tile, slot, split, splits, part, r0, nr};
  const int bh = b * a.heads + h;
  const uint8_t *kf = a.kpay + (int64_t)bh * a.tcap * D, *vf = a.vpay + (int64_t)bh * a.tcap * D;
  const float2 *km = a.kmeta + (int64_t)bh * a.nblk, *vm = a.vmeta + (int64_t)bh * a.nblk;
  RawKeys uk;
  RawValues uv;
  // nor do the first units of a sequence that is not split (rows of the capacity, used
  // or not; 200 tokens 8.3 us, behind the length 8.6)
  if (splits == 1 && wave * UNIT < a.tcap) {
    load_keys(a, kf, km, wave * UNIT, uk);
    load_values(a, vf, vm, wave * UNIT, uv);
  }
  if (!a.ragged) sq = load_sequence(a, b);
  const int tmax = limit_of(a, sq, r0 / a.ratio, (r0 + nr - 1) / a.ratio);
  const int units = (tmax + UNIT - 1) / UNIT;
  const int u0 = split_begin(units, split, splits), u1 = split_begin(units, split + 1, splits);
  if (splits > 1 && u0 + wave < u1) {
    load_keys(a, kf, km, (u0 + wave) * UNIT, uk);
    load_values(a, vf, vm, (u0 + wave) * UNIT, uv);
  }

  // gauged query rows
  float *xs = lds, *ys = lds + ROWS * PITCH;
  if (front) put_row_part(xs, qp);
  __syncthreads();
  if (a.g) {
    if (front) gauge_tiles<false, 1, false>(xs, ys, gk, a.g, gw);
    __syncthreads();
  } else {
    ys = xs;
  }
  // the operands, a step to a wave, and from LDS to all (each wave for itself:
  // 400 vector instructions instead of 130)
  QueryFrags q;
  {
    unsigned char *fs = (unsigned char *)(lds + 2 * ROWS * PITCH);  // [hi, lo][step][lane]
    float *qs = (float *)(fs + 8192);  // [step][row] parts of the minimum's factor, then the score's factor
    if (front) {
      h8_t hi, lo;
      float ca, cq;
      make_frags(ys, a.c, wave, hi, lo, ca, cq);
      *(h8_t *)(fs + wave * 1024 + lane * 16) = hi;
      *(h8_t *)(fs + 4096 + wave * 1024 + lane * 16) = lo;
      if (grp == 0) {
        qs[wave * ROWS + row] = cq;
        qs[(4 + wave) * ROWS + row] = ca;
      }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 4; s++) {
      q.hi[s] = *(const h8_t *)(fs + s * 1024 + lane * 16);
      q.lo[s] = *(const h8_t *)(fs + 4096 + s * 1024 + lane * 16);
    }
    q.cq = (qs[row] + qs[ROWS + row]) + (qs[2 * ROWS + row] + qs[3 * ROWS + row]);
    q.ca = qs[4 * ROWS + row] * (BF16 ? kCodeUnit : kCentredUnit);
  }

  // what this lane's row sees; rows that are not there see everything, and
  // are never stored
  const int lim = row < nr ? query_limit(a, sq, (int)((uint32_t)(r0 + row) / (uint32_t)a.ratio)) : tmax;
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

  for (int un = u0 + wave; un < u1; un += NW) {
    const int t0 = un * UNIT;
    const bool more = un + NW < u1;
    float s[2][4];
#pragma unroll
    for (int t = 0; t < 2; t++) {
      f4_t z = f4_t{0.f, 0.f, 0.f, 0.f}, zl = z;
      Centre ck{uk.m[t].x, 0u};
      if constexpr (!BF16) ck = centre_of(uk.m[t]);
#pragma unroll
      for (int x = 0; x < 2; x++) {
        const h8_t c0 = codes8<!BF16>(uk.k[t][x].x, uk.k[t][x].y, ck.c), c1 = codes8<!BF16>(uk.k[t][x].z, uk.k[t][x].w, ck.c);
        z = mfma(c0, q.hi[2 * x], z);
        z = mfma(c1, q.hi[2 * x + 1], z);
        zl = mfma(c0, q.lo[2 * x], zl);
        zl = mfma(c1, q.lo[2 * x + 1], zl);
      }
      z += zl;
      const float A = uk.m[t].y * q.ca, Bm = ck.mid * q.cq;
#pragma unroll
      for (int r = 0; r < 4; r++) s[t][r] = __builtin_fmaf(z[r], A, Bm);
    }
    if (more) load_keys(a, kf, km, t0 + NW * UNIT, uk);
    float vst[2], vmn[2];
    uint32_t vc[2];
#pragma unroll
    for (int t = 0; t < 2; t++) {
      Centre cv{__builtin_fmaf(128.0f, uv.m[t].y, uv.m[t].x), kMiddle};
      if constexpr (!BF16) cv = centre_of(uv.m[t]);
      vst[t] = uv.m[t].y;
      vmn[t] = cv.mid;  // the value of the centre
      vc[t] = cv.c;
    }
    if (t0 + UNIT > all) {
#pragma unroll
      for (int t = 0; t < 2; t++) {
        if (t0 + 16 * t >= lim) vst[t] = vmn[t] = 0.0f;  // nothing this row sees: perhaps not a number
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
    const h8_t P = as_h8(ph[0][0], ph[0][1], ph[1][0], ph[1][1]);
    h8_t Pl;
    if constexpr (!BF16) Pl = as_h8(pl[0][0], pl[0][1], pl[1][0], pl[1][1]);
#define CG_PV(J)                                        \
  {                                                     \
    const h8_t vj = value_frag<J>(uv, vc);              \
    acc[J] = mfma(vj, P, acc[J]);                       \
    if constexpr (!BF16) acc[J] = mfma(vj, Pl, acc[J]); \
  }
    CG_PV(0) CG_PV(1) CG_PV(2) CG_PV(3) CG_PV(4) CG_PV(5) CG_PV(6) CG_PV(7)
#undef CG_PV
    if (more) load_values(a, vf, vm, t0 + NW * UNIT, uv);
    if constexpr (MASS) {  // block sums over the row's lanes; behind the loads: waiting for those does not wait for a store
      const int64_t e = t0 >> min(a.bshift, 5);
      float2 *p = a.bsum + ((int64_t)bh * a.entries + e) * a.rows + r0 + row;
      const bool two = a.bshift == 4;
      const float v0 = row_sum(two ? bs[0] : bs[0] + bs[1]), v1 = two ? row_sum(bs[1]) : 0.0f;
      if (grp == 0 && row < nr) {
        *p = make_float2(v0, st.mu);
        if (two && e + 1 < a.entries) p[a.rows] = make_float2(v1, st.mu);
      }
    }
  }

  const float *gv = a.gv + (int64_t)h * D * a.g;
  if (splits == 1 && front) load_gauge<true>(gv, a.g, 0, gw);
  const float mv = row_sum(st.mv);
  // true sums: acc 2^9 / f (the codes' and the weights' scales)
  const float ks = st.m > -INFINITY ? exp2_fast(st.mo - st.m) : 0.0f;
  finish_few<BF16, NW>(a, fp, lds, ml, gv, gw, front, st.m, st.l, ks, mv, acc);
}

// the parts of (b, h): the first one's number and how many there are
struct Parts {
  int64_t first;
  int count;
};
__device__ __forceinline__ Parts parts_of(const AttendArgs &a, int b, int h) {
  if (!a.ragged) return Parts{((int64_t)b * a.heads + h) * a.splits, a.splits};
  const int2 x = a.dealt[b];
  return Parts{(int64_t)h * a.slots + x.x, x.y};
}

// Block weights of few rows from the sums the attention left, 256 blocks to a
// workgroup: mass[block] += sum over rows of sum_t 2^(s_t - m) 2^(m - log2 sum)
__device__ __forceinline__ void finish_mass(const AttendArgs &a, uint32_t id) {
  __shared__ float lse2[FEW_TILES * ROWS];
  __shared__ int lim[FEW_TILES * ROWS];
  const uint32_t chunks = (uint32_t)((a.nblk + NTH - 1) / NTH);
  const int bh = (int)(id / chunks), b = bh / a.heads;
  const int64_t blk = (int64_t)(id - bh * chunks) * NTH + threadIdx.x;
  const Sequence sq = load_sequence(a, b);
  const int j = threadIdx.x & 15;  // 16 lanes to a row's splits
  const Parts ps = parts_of(a, b, bh - b * a.heads);
  for (int row = threadIdx.x >> 4; row < a.rows; row += NTH / 16) {
    const float2 *pm = a.part_ml + ps.first * a.rows + row;
    float M = -INFINITY, L = 0.0f;
    for (int s = j; s < ps.count; s += 16) {
      const float2 x = pm[(int64_t)s * a.rows];
      const float m = fmaxf(M, x.x);
      L = m > -INFINITY ? L * exp2_fast(M - m) + x.y * exp2_fast(x.x - m) : L + x.y;
      M = m;
    }
#pragma unroll
    for (int k = 8; k >= 1; k >>= 1) {
      const float m2 = __shfl_xor(M, k), l2 = __shfl_xor(L, k), m = fmaxf(M, m2);
      L = m > -INFINITY ? L * exp2_fast(M - m) + l2 * exp2_fast(m2 - m) : L + l2;
      M = m;
    }
    if (j == 0) {
      lse2[row] = M + __builtin_log2f(L);
      lim[row] = L != 0.0f ? query_limit(a, sq, (int)((uint32_t)row / (uint32_t)a.ratio)) : 0;
    }
  }
  __syncthreads();
  if (blk >= a.nblk || (blk << a.bshift) >= limit_of(a, sq, 0, a.n - 1)) return;
  const int per = a.bshift == 6 ? 2 : 1, esh = min(a.bshift, 5);
  float w = 0.0f;
  for (int k = 0; k < per; k++) {
    const int64_t e = blk * per + k;
    const float2 *p = a.bsum + ((int64_t)bh * a.entries + e) * a.rows;
#pragma unroll 4
    for (int r = 0; r < a.rows; r++) {
      if ((e << esh) >= lim[r]) continue;  // nothing for this row: perhaps nobody wrote its sum
      const float2 x = p[r];
      if (x.x != 0.0f) w += x.x * exp2_fast(x.y - lse2[r]);
    }
  }
  a.mass[(int64_t)bh * a.nblk + blk] += w;
}

__global__ __launch_bounds__(NTH) void k_mass_finish(const AttendArgs a) { finish_mass(a, blockIdx.x); }

// Joins the splits of one row, a workgroup to a row: 2^(m_s - M) of every
// split, eight groups of 32 lanes adding every eighth split's sums, then the
// inverse gauge.  Up to 128 splits each wave forms all factors for itself, beside
// the loads of the sums: 32 rows of 32 splits 4.0 us, through LDS and two more
// barriers 5.0; 3200 rows of 3 splits 8.5 and 10.0; 32 rows of 96 5.3 and 8.0.  For few rows with many splits; workgroups past the last row
// finish the blocks' weights (MASS), which need no more than the rows do.
template <bool BF16, bool MASS>
__global__ __launch_bounds__(NTH) void k_attend_merge(const AttendArgs a) {
  __shared__ __align__(16) float part[8][D];
  __shared__ __align__(16) float us[PITCH];
  __shared__ float wt[MERGE_SPLITS];
  __shared__ float2 red[4];
  const uint32_t id = blockIdx.x;
  if constexpr (MASS) {
    const uint32_t merging = (uint32_t)(a.batch * a.heads * a.rows);
    if (id >= merging) {
      finish_mass(a, id - merging);
      return;
    }
  }
  const int bh = (int)(id / (uint32_t)a.rows), r = (int)id - bh * a.rows;
  const int b = (int)((uint32_t)bh / (uint32_t)a.heads), h = bh - b * a.heads;
  const Parts ps = parts_of(a, b, h);
  if (a.ragged && ps.count == 1) return;  // the attention has stored the row
  const float2 *pm = a.part_ml + ps.first * a.rows + r;
  const float *po = a.part_o + (ps.first * a.rows + r) * D;
  const int S = ps.count, t = threadIdx.x;
  const int lane = t & 63, grp = t >> 5, c4 = 4 * (t & 31);
  // on their way first, in the order of their use: the splits' maxima and sums, the
  // first rows of sums, this thread's part of G_V (the two halves of the
  // workgroup take half of a channel's chain each)
  constexpr int HEAD = 4;
  float2 ml = make_float2(-INFINITY, 0.0f), mh = ml;
  f4_t head[HEAD];
  if (S <= 128) {
    if (lane < S) ml = pm[(int64_t)lane * a.rows];
    if (lane + 64 < S) mh = pm[(int64_t)(lane + 64) * a.rows];
#pragma unroll
    for (int k = 0; k < HEAD; k++)
      head[k] = grp + 8 * k < S ? *(const f4_t *)(po + (int64_t)(grp + 8 * k) * a.rows * D + c4) : f4_t{0.f, 0.f, 0.f, 0.f};
  }
  const int c = t & (D - 1), cg = c & (a.g - 1), gh = a.g >> 1, k0 = (t >> 7) * gh;
  const float *gp = a.gv + (int64_t)h * D * a.g + (int64_t)(c - cg) * a.g + (int64_t)k0 * a.g + cg;
  float gw[16];
#pragma unroll
  for (int k = 0; k < 16; k++) gw[k] = k < gh ? gp[(int64_t)k * a.g] : 0.0f;
  float M = -INFINITY, L = 0.0f;
  f4_t u = f4_t{0.f, 0.f, 0.f, 0.f};
  if (S <= 128) {
    M = wave_max(fmaxf(ml.x, mh.x));
    const float w = ml.x > -INFINITY ? exp2_fast(ml.x - M) : 0.0f, wh = mh.x > -INFINITY ? exp2_fast(mh.x - M) : 0.0f;
    L = wave_sum(__builtin_fmaf(mh.y, wh, ml.y * w));
#pragma unroll
    for (int k = 0; k < HEAD; k++) u += head[k] * __shfl(w, grp + 8 * k);
    const auto more = [&](float f, int first) {  // four more, side by side
      f4_t v[4];
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const int x = first + grp + 8 * k;
        v[k] = x < S ? *(const f4_t *)(po + (int64_t)x * a.rows * D + c4) : f4_t{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int k = 0; k < 4; k++) u += v[k] * __shfl(f, (first + grp + 8 * k) & 63);
    };
    if (S > 32) more(w, 32);
    if (S > 64) more(wh, 64);
    if (S > 96) more(wh, 96);
  } else {
    for (int s = t; s < S; s += NTH) M = fmaxf(M, pm[(int64_t)s * a.rows].x);
    M = wave_max(M);
    if (lane == 0) red[t >> 6].x = M;
    __syncthreads();
    M = fmaxf(fmaxf(red[0].x, red[1].x), fmaxf(red[2].x, red[3].x));
    for (int s = t; s < S; s += NTH) {
      const float2 x = pm[(int64_t)s * a.rows];
      const float k = x.x > -INFINITY ? exp2_fast(x.x - M) : 0.0f;
      wt[s] = k;
      L += x.y * k;
    }
    L = wave_sum(L);
    if (lane == 0) red[t >> 6].y = L;
    __syncthreads();
    L = (red[0].y + red[1].y) + (red[2].y + red[3].y);
    for (int s = grp; s < S; s += 64) {
      f4_t v[8];
#pragma unroll
      for (int k = 0; k < 8; k++)
        v[k] = s + 8 * k < S ? *(const f4_t *)(po + (int64_t)(s + 8 * k) * a.rows * D + c4) : f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 8; k++) u += v[k] * (s + 8 * k < S ? wt[s + 8 * k] : 0.0f);
    }
  }
  *(f4_t *)&part[grp][c4] = u;
  __syncthreads();
  if (t == 0) {
    if (a.lse) store_lse(a, b, h, r, M, L);
    if (a.lse2) a.lse2[(int64_t)bh * a.rows + r] = L != 0.0f ? M + __builtin_log2f(L) : INFINITY;
  }
  if (t < D) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k++) v += part[k][t];
    us[t] = L != 0.0f ? v / L : 0.0f;
  }
  __syncthreads();
  if (a.g == 0) {
    if (t < D) store_out<BF16>(a, b, h, r, t, us[t]);
    return;
  }
  const float *x = us + (c - cg) + k0;
  float v = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; k++)
    if (k < gh) v = __builtin_fmaf(gw[k], x[k], v);
#pragma unroll 16
  for (int k = 16; k < gh; k++) v = __builtin_fmaf(gp[(int64_t)k * a.g], x[k], v);
  part[t >> 7][c] = v;
  __syncthreads();
  if (t < D) store_out<BF16>(a, b, h, r, t, part[0][t] + part[1][t]);
}

// The same for many rows with few splits: 16 rows to a workgroup, a row to a
// wave at a time.
template <bool BF16>
__global__ __launch_bounds__(NTH) void k_attend_merge_many(const AttendArgs a) {
  __shared__ __align__(16) float us[ROWS * PITCH];
  const uint32_t id = blockIdx.x;
  const int bh = (int)(id / (uint32_t)a.tiles), r0 = (int)(id - bh * a.tiles) * ROWS;
  const int h = bh % a.heads, b = bh / a.heads, nr = min(ROWS, a.rows - r0);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float *gv = a.gv + (int64_t)h * D * a.g;
  GaugeFrag gw;
  load_gauge<true>(gv, a.g, 0, gw);
  // four rows a wave, side by side
  int r[4];
  float M[4], L[4];
  float2 u[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    r[i] = min(r0 + wave + 4 * i, a.rows - 1);
    M[i] = -INFINITY;
    L[i] = 0.0f;
    u[i] = make_float2(0.f, 0.f);
  }
  const Parts ps = parts_of(a, b, h);
  if (a.ragged && ps.count == 1) return;
  const float2 *pm = a.part_ml + ps.first * a.rows;
  const float *po = a.part_o + ps.first * a.rows * D + 2 * lane;
  for (int s = 0; s < ps.count; s++)
#pragma unroll
    for (int i = 0; i < 4; i++) M[i] = fmaxf(M[i], pm[(int64_t)s * a.rows + r[i]].x);
#pragma unroll 2
  for (int s = 0; s < ps.count; s++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float2 x = pm[(int64_t)s * a.rows + r[i]], y = *(const float2 *)(po + ((int64_t)s * a.rows + r[i]) * D);
      const float k = x.x > -INFINITY ? exp2_fast(x.x - M[i]) : 0.0f;
      L[i] += x.y * k;
      u[i].x += y.x * k;
      u[i].y += y.y * k;
    }
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int rr = wave + 4 * i;
    const float inv = L[i] > 0.0f ? 1.0f / L[i] : 0.0f;
    *(float2 *)(us + rr * PITCH + 2 * lane) = make_float2(u[i].x * inv, u[i].y * inv);
    if (lane == 0 && rr < nr) {
      if (a.lse) store_lse(a, b, h, r[i], M[i], L[i]);
      if (a.lse2) a.lse2[(int64_t)bh * a.rows + r[i]] = L[i] != 0.0f ? M[i] + __builtin_log2f(L[i]) : INFINITY;
    }
  }
  __syncthreads();
  if (a.g) {
    gauge_tiles<true, 1, true>(us, us, gv, a.g, gw);
    __syncthreads();
  }
  store_rows<BF16>(a, b, h, r0, nr, us);
}

hipError_t rows_launch(const AttendArgs &a, bool bf16, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.heads * a.tiles * a.slots));
  const bool mass = a.mass && a.bsum;
#define CG_R(BF, MA, NW)                                                                       \
  if (bf16 == BF && mass == MA && a.waves == NW) {                                             \
    hipLaunchKernelGGL((k_attend_rows<BF, MA, NW>), grid, dim3(64 * NW), 0, s, a);             \
    return hipGetLastError();                                                                  \
  }
  CG_R(true, false, 4) CG_R(true, true, 4) CG_R(false, false, 4) CG_R(false, true, 4)
  CG_R(true, false, 8) CG_R(true, true, 8) CG_R(false, false, 8) CG_R(false, true, 8)
#undef CG_R
  return hipErrorInvalidValue;
}

hipError_t merge_launch(const AttendArgs &a, bool bf16, hipStream_t s) {
  const int64_t fields = (int64_t)a.batch * a.heads;
  const bool mass = a.mass && a.bsum && a.tokens > 0 && a.few;
  const dim3 block(NTH);
  // a workgroup a row while they fit the machine twice over (1024 rows of 64
  // splits: 8.6 us, by sixteens 58), else sixteen rows (9600 rows of 3: 13 and 26)
  if (fields * a.rows > 4096) {
    const dim3 grid((unsigned)(fields * a.tiles));
    if (bf16) hipLaunchKernelGGL(k_attend_merge_many<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_attend_merge_many<false>, grid, block, 0, s, a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess && mass ? mass_finish_launch(a, s) : e;
  }
  const dim3 grid((unsigned)(fields * a.rows + (mass ? fields * ((a.nblk + NTH - 1) / NTH) : 0)));
  if (bf16 && mass) hipLaunchKernelGGL((k_attend_merge<true, true>), grid, block, 0, s, a);
  else if (bf16) hipLaunchKernelGGL((k_attend_merge<true, false>), grid, block, 0, s, a);
  else if (mass) hipLaunchKernelGGL((k_attend_merge<false, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_attend_merge<false, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t mass_finish_launch(const AttendArgs &a, hipStream_t s) {
  const int64_t chunks = (a.nblk + NTH - 1) / NTH;
  const dim3 grid((unsigned)((int64_t)a.batch * a.heads * chunks)), block(NTH);
  hipLaunchKernelGGL(k_mass_finish, grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace cga
