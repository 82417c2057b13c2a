// Attention of query rows over the 4-bit cache, 16 rows to a workgroup, split along the
// tokens like the form of the 8-bit cache (attend_rows.hip).
//
// Keys have a range for 32 tokens of a channel, values one for 32 channels of a token:
//   s_t = c ( sum_c (q'_c sk_c) a_tc + sum_c q'_c mk_c ),   out = sum_t p_t (mv_tg + sv_tg b_tc) / sum_t p_t
// A wave takes units of 32 tokens, a key range's, in turn.  The key steps go to the queries:
// 128 products a row and unit, each lane those of two channels for all rows, which reach the
// matrix cores' operand layout through the wave's own LDS; the codes are multiplied as they
// are.  The values are widened to v' itself, since their ranges differ along both
// axes of the second product: one packed multiply-add turns two codes into
// fp16 values of a power-of-two scale that the unit's weights carry.
//
// Precision of a score: a unit's power of two 2^E bounds |mk| and |mk + 15 sk|; the products
// q'_c sk_c stand in two fp16 parts, a multiple of 2^3 and what is left, where q's
// largest is in [2^13, 2^14) and sk in units of 2^(E - 2): off by 2^-23 of the
// largest |q'| times the largest |k'|.  The matrix cores add the first part's products without
// a rounding (128 multiples of 2^3 below 2^14, times 15).  For fp32 storage, log-sums and weights
// there is a part between the two, a multiple of 2^-8, added exactly too (2^-34; in two parts
// fp32 outputs of 4000 tokens were off by 1.4e-6, log-sums of 28 tokens by 1.35e-6, by fp32
// products 0.4e-6 and 0.08e-6).  Values: the step and the centre of a range and the value
// rounded to fp16 each, around the code 8 (2^-12 of themselves, 2^-34 of the largest of the unit's
// 32 tokens), for fp32 storage in two parts.  With the code as it stands and the minimum, a third
// of this work less, bf16 outputs were off by 1.95e-3 of themselves, by 1.72e-3 around the
// centre, and 1.66e-3 is their own rounding; 262144 tokens took 86.5 us for 87.7.
//
// 262144 tokens of 8 KV heads, four query heads each: 80 us (4.9 TB/s, a sum of as many bytes 5.9; 412 vector
// instructions a unit) and a merge of 5; 16 sequences of up to 8192 with log-sums 26 (13 of them units, 5
// the query's way into its operands) and 4.8.  Up to 1024 tokens in one workgroup of eight waves 13.9: its
// chain takes 8, four units a wave 1.5 each; sixteen waves 15.4 (spills).  Two units' keys in flight: the same.
// Rows beyond 4 and 8 have forms of their own, whose queries take as much work: eight query heads and
// 262144 tokens 96 us, in the form of 16 rows 106; five, 16 sequences with log-sums 28 and 44.
#include "attend.hpp"
#include "attend4.hpp"
#include "attend_few.hpp"

namespace cga {

typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

// orders a wave's LDS accesses for the compiler (the hardware keeps them in order)
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

constexpr float kKeyUnit = 1.5f * 67108864.0f;  // x + u - u rounds to multiples of 2^3

// A unit as it is loaded.  Keys: token 16 t + lane % 16, channels 32 (lane / 16) .. + 31, and
// the ranges of this lane's two channels; values: tokens 16 t + 4 grp + i, channels 8
// (lane % 16) .. + 7, and the ranges of group lane / 16 of tokens 2 (lane % 16), + 1.
struct Keys4 {
  u4_t k[2];
  float2 m[2];
};
struct Values4 {
  uint32_t v[2][4];
  float2 m[2];
};

__device__ __forceinline__ int key_channel() {  // this lane's first channel; its second is 4 further
  const int lane = threadIdx.x & 63;
  return 8 * (lane >> 2) + (lane & 3);
}

__device__ __forceinline__ void load_keys4(const uint8_t *kf, const float2 *km, int t0, Keys4 &u) {
  const int lane = threadIdx.x & 63, n = lane & 15, grp = lane >> 4;
  const uint8_t *k = kf + (int64_t)(t0 + n) * HALF_D + 16 * grp;
  u.k[0] = *(const u4_t *)k;
  u.k[1] = *(const u4_t *)(k + 16 * HALF_D);
  const float2 *m = km + (int64_t)t0 * 4 + key_channel();  // 128 ranges for 32 tokens
  u.m[0] = m[0];
  u.m[1] = m[4];
}

__device__ __forceinline__ void load_values4(const uint8_t *vf, const float2 *vm, int t0, Values4 &u) {
  const int lane = threadIdx.x & 63, n = lane & 15, grp = lane >> 4;
  const uint8_t *v = vf + (int64_t)(t0 + 4 * grp) * HALF_D + 4 * n;
#pragma unroll
  for (int t = 0; t < 2; t++)
#pragma unroll
    for (int i = 0; i < 4; i++) u.v[t][i] = *(const uint32_t *)(v + (16 * t + i) * HALF_D);
  const float2 *m = vm + ((int64_t)t0 + 2 * n) * 4 + grp;
  u.m[0] = m[0];
  u.m[1] = m[4];
}

// eight codes of a dword as halves: pairs (0, 4), (1, 5), (2, 6), (3, 7); the odd ones 16 times
// themselves, which their queries make up for
__device__ __forceinline__ h8_t nibbles8(uint32_t w) {
  const uint32_t x = w >> 8;
  return as_h8(w & 0x000f000fu, w & 0x00f000f0u, x & 0x000f000fu, x & 0x00f000f0u);
}

// codes of two tokens' channels 2 B and 2 B + 1 of a dword, less 8, times 2^-9
template <int B>
__device__ __forceinline__ void centred4(uint32_t w0, uint32_t w1, uint32_t &even, uint32_t &odd) {
  const h2_t up = {(_Float16)32768.0f, (_Float16)32768.0f}, up16 = {(_Float16)2048.0f, (_Float16)2048.0f};
  const h2_t mid = {(_Float16)-0x1p-6f, (_Float16)-0x1p-6f};
  const uint32_t x = byte_pair<B>(w0, w1);
  even = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(h2_t, x & 0x000f000fu), up, mid));
  odd = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(h2_t, x & 0x00f000f0u), up16, mid));
}

struct RowState4 {
  float m, mu, mo, f;   // maximum, the one used (-inf while none), value scale, log2 of the weights' factor
  float l;
  uint32_t poison;      // groups of channels of which the row has seen a value that is not a number
};

// P3: three parts of a query times a key step (fp32 storage, or where log-sums or weights are
// asked for), else two.  NR: rows that get key operands; the others read those of row % NR
template <bool BF16, bool P3, bool MASS, int NW, int NR>
__global__ __launch_bounds__(64 * NW, NW == 4 && !MASS ? 3 : 2) void k_attend4_rows(const AttendArgs a) {
  // a wave's own: key operands [part][step][row][grp][8], the rows' sums with the minima, the
  // values' centres and steps [4][32]
  static_assert(P3 || (BF16 && !MASS), "two parts for bf16 outputs alone");
  constexpr int PARTS = P3 ? 3 : 2;
  // 64 bytes between the steps: other banks.  Half of them for 16 rows in three parts, for a third workgroup on a
  // compute unit (4 queries of 16 sequences of up to 8192 with log-sums 37 us for 41)
  constexpr int STEP = NR * 64 + (BF16 && P3 && NR == 16 && !MASS ? 32 : 64), KOPS = 4 * PARTS * STEP, VB = BF16 ? 2 : 4, VR = 32 * VB;
  constexpr int WAVE = KOPS + 64 + 8 * VR, JOIN = ROWS * PITCH * 4;
  constexpr int PER = WAVE > JOIN ? WAVE : JOIN;
  static_assert(PER * NW >= 3 * ROWS * PITCH * 4, "gauged rows and their factors");
  __shared__ __align__(16) unsigned char lds8[NW * PER];
  __shared__ float2 ml[NW][ROWS];
  float *lds = (float *)lds8;
  const int lane = threadIdx.x & 63, row = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t id = blockIdx.x;
  int b, h, tile, slot = 0, split = 0, splits = a.splits;
  int64_t part;  // where this part's row 0 goes
  if (a.ragged) {
    const uint32_t q1 = id / (uint32_t)a.heads, q2 = q1 / (uint32_t)a.tiles;
    h = (int)(id - q1 * a.heads);
    tile = (int)(q1 - q2 * a.tiles);
    slot = (int)q2;
    b = (int)(q2 * (uint32_t)a.batch / (uint32_t)a.slots);
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
  const float *gk = a.gk + (int64_t)h * D * a.g;
  const bool front = NW == 4 || wave < 4;
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
  const uint8_t *kf = a.kpay + (int64_t)bh * a.tcap * HALF_D, *vf = a.vpay + (int64_t)bh * a.tcap * HALF_D;
  const float2 *km = a.kmeta + (int64_t)bh * a.tcap * 4, *vm = a.vmeta + (int64_t)bh * a.tcap * 4;
  Keys4 uk;
  Values4 uv;
  if (splits == 1 && wave * UNIT < a.tcap) {
    load_keys4(kf, km, wave * UNIT, uk);
    load_values4(vf, vm, wave * UNIT, uv);
  }
  if (!a.ragged) sq = load_sequence(a, b);
  const int tmax = limit_of(a, sq, r0 / a.ratio, (r0 + nr - 1) / a.ratio);
  const int units = (tmax + UNIT - 1) / UNIT;
  const int u0 = split_begin(units, split, splits), u1 = split_begin(units, split + 1, splits);
  if (splits > 1 && u0 + wave < u1) {
    load_keys4(kf, km, (u0 + wave) * UNIT, uk);
    load_values4(vf, vm, (u0 + wave) * UNIT, uv);
  }

  // gauged query rows, each lane's two channels of them scaled; odd channels less the 16
  // that their codes carry
  float *xs = lds, *ys = lds + ROWS * PITCH;
  float2 *fac = (float2 *)(lds + 2 * ROWS * PITCH);  // [row] (factor, its inverse)
  if (front) put_row_part(xs, qp);
  __syncthreads();
  if (a.g) {
    if (front) gauge_tiles<false, 1, false>(xs, ys, gk, a.g, gw);
    __syncthreads();
  } else {
    ys = xs;
  }
  if (front) {
    const float *rp = ys + (threadIdx.x >> 4) * PITCH + 8 * (threadIdx.x & 15);
    float mx = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k++) mx = fmaxf(mx, fabsf(rp[k]));
    mx = fmaxf(mx, ror16<8>(mx));
    mx = fmaxf(mx, ror16<4>(mx));
    mx = fmaxf(mx, ror16<2>(mx));
    mx = fmaxf(mx, ror16<1>(mx));
    const FragScale sc = frag_scale(mx);
    if ((threadIdx.x & 15) == 0) fac[threadIdx.x >> 4] = make_float2(sc.up, sc.un);
  }
  __syncthreads();
  const int ch = key_channel();
  const bool odd = lane & 1;
  const float unit = odd ? kKeyUnit / 16.0f : kKeyUnit;
  const int msh = odd ? 4 : 0;
  float q[NR][2];
#pragma unroll
  for (int r = 0; r < NR; r++) {
    const float up = fac[r].x * (odd ? 0.0625f : 1.0f);
    q[r][0] = ys[r * PITCH + ch] * up;
    q[r][1] = ys[r * PITCH + ch + 4] * up;
  }
  const float ca = a.c * fac[row].y;
  __syncthreads();  // the rows have been read
  unsigned char *const wl = lds8 + wave * PER;
  // this lane's dword of row 0's operands, and what it reads of them
  unsigned char *const kput = wl + ((lane >> 2) & 3) * STEP + (lane >> 4) * 16 + 4 * (lane & 3);
  const unsigned char *const kget = wl + (row & (NR - 1)) * 64 + grp * 16;
  float *const msum = (float *)(wl + KOPS);
  unsigned char *const vput = wl + KOPS + 64 + grp * VR + 2 * row * VB;
  const unsigned char *const vget = wl + KOPS + 64 + (row >> 2) * VR + 4 * grp * VB;

  const int lim = row < nr ? query_limit(a, sq, (int)((uint32_t)(r0 + row) / (uint32_t)a.ratio)) : tmax;
  int all = lim;
#pragma unroll
  for (int k = 1; k < 16; k <<= 1) all = min(all, __shfl_xor(all, k));
  all = __builtin_amdgcn_readfirstlane(all);  // every row sees the tokens before it

  RowState4 st;
  st.m = st.mu = st.mo = -INFINITY;
  st.f = 0.0f;
  st.l = 0.0f;
  st.poison = 0u;
  f4_t acc[8];
#pragma unroll
  for (int j = 0; j < 8; j++) acc[j] = f4_t{0.f, 0.f, 0.f, 0.f};

  for (int un = u0 + wave; un < u1; un += NW) {
    const int t0 = un * UNIT;
    const bool more = un + NW < u1;
    // key steps into the queries
    const int ek = exponent_of(__builtin_amdgcn_readfirstlane(wave_umax(max(range_bits(uk.m[0]), range_bits(uk.m[1])))));
    {
      const float s0 = __builtin_ldexpf(uk.m[0].y, 2 - ek), s1 = __builtin_ldexpf(uk.m[1].y, 2 - ek);
      const float m0 = __builtin_ldexpf(uk.m[0].x, msh - ek), m1 = __builtin_ldexpf(uk.m[1].x, msh - ek);
      float v[NR];
#pragma unroll
      for (int r = 0; r < NR; r++) {
        const float x = q[r][0] * s0, y = q[r][1] * s1;
        const float xh = (x + unit) - unit, yh = (y + unit) - unit;
        *(uint32_t *)(kput + 64 * r) = pack_f16x2(xh, yh);  // exact
        float xl = x - xh, yl = y - yh;
        if constexpr (P3) {
          const float xm = (xl + unit * 0x1p-11f) - unit * 0x1p-11f, ym = (yl + unit * 0x1p-11f) - unit * 0x1p-11f;
          *(uint32_t *)(kput + 8 * STEP + 64 * r) = pack_f16x2(xm, ym);  // exact
          xl -= xm;
          yl -= ym;
        }
        *(uint32_t *)(kput + 4 * STEP + 64 * r) = pack_f16x2(xl, yl);
        v[r] = __builtin_fmaf(q[r][0], m0, q[r][1] * m1);
      }
      // the rows' sums over the lanes, four rows at once: row 4 k + (0, 2, 1, 3)[grp]
#pragma unroll
      for (int r = 0; r < NR; r += 4) {
        const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[r]), __float_as_uint(v[r + 1]), false, false);
        const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[r + 2]), __float_as_uint(v[r + 3]), false, false);
        const float a0 = __uint_as_float(x[0]) + __uint_as_float(x[1]), a1 = __uint_as_float(y[0]) + __uint_as_float(y[1]);
        const auto z = __builtin_amdgcn_permlane16_swap(__float_as_uint(a0), __float_as_uint(a1), false, false);
        float s = __uint_as_float(z[0]) + __uint_as_float(z[1]);
        s += ror16<8>(s);
        s += ror16<4>(s);
        s += ror16<2>(s);
        s += ror16<1>(s);
        if (row == 0) msum[r + ((grp & 1) << 1) + (grp >> 1)] = s;
      }
    }
    // value ranges: those behind the sequence's end are whatever they are
    float2 vr[2] = {uv.m[0], uv.m[1]};
    if (t0 + UNIT > sq.len) {
      if (t0 + 2 * row >= sq.len) vr[0] = make_float2(0.f, 0.f);
      if (t0 + 2 * row + 1 >= sq.len) vr[1] = make_float2(0.f, 0.f);
    }
    const uint32_t x0 = range_bits(vr[0]), x1 = range_bits(vr[1]);
    uint32_t tv = __builtin_amdgcn_readfirstlane(wave_umax(max(x0, x1)));
    if (tv >= INF) {
      // a range that is not a number: its tokens count as zeros, and the rows that see them are marked
      const bool bad0 = x0 >= INF, bad1 = x1 >= INF;
      const uint64_t e = __ballot(bad0), o = __ballot(bad1);  // tokens 2 i and 2 i + 1 of group g: bit 16 g + i
      const int vis = min(max(lim - t0, 0), UNIT);
      const uint32_t se = (1u << ((vis + 1) >> 1)) - 1u, so = (1u << (vis >> 1)) - 1u;
#pragma unroll
      for (int g = 0; g < 4; g++)
        if (((uint32_t)(e >> 16 * g) & se) | ((uint32_t)(o >> 16 * g) & so)) st.poison |= 1u << g;
      if (bad0) vr[0] = make_float2(0.f, 0.f);
      if (bad1) vr[1] = make_float2(0.f, 0.f);
      tv = __builtin_amdgcn_readfirstlane(wave_umax(max(bad0 ? 0u : x0, bad1 ? 0u : x1)));
    }
    const int ev = exponent_of(tv);
    {
      // values below 2^9; the steps times the 2^9 that centred codes lack (34953 at most)
      const float s0 = __builtin_ldexpf(vr[0].y, 18 - ev), s1 = __builtin_ldexpf(vr[1].y, 18 - ev);
      const float c0 = __builtin_ldexpf(__builtin_fmaf(8.0f, vr[0].y, vr[0].x), 9 - ev);
      const float c1 = __builtin_ldexpf(__builtin_fmaf(8.0f, vr[1].y, vr[1].x), 9 - ev);
      if constexpr (BF16) {
        *(uint32_t *)vput = pack_f16x2(s0, s1);
        *(uint32_t *)(vput + 4 * VR) = pack_f16x2(c0, c1);
      } else {
        *(float2 *)vput = make_float2(s0, s1);
        *(float2 *)(vput + 4 * VR) = make_float2(c0, c1);
      }
    }
    wave_sync();
    // scores: fma(z, A, Bm)
    f4_t z[2];
    {
      f4_t zl[2];
#pragma unroll
      for (int t = 0; t < 2; t++) z[t] = zl[t] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < 4; x++) {
        const h8_t hi = *(const h8_t *)(kget + x * STEP), lo = *(const h8_t *)(kget + (4 + x) * STEP);
#pragma unroll
        for (int t = 0; t < 2; t++) {
          const h8_t c = nibbles8(uk.k[t][x]);
          z[t] = mfma(c, hi, z[t]);
          if constexpr (P3) {
            zl[t] = mfma(c, *(const h8_t *)(kget + (8 + x) * STEP), zl[t]);
            zl[t] = mfma(c, lo, zl[t]);
          } else {
            z[t] = mfma(c, lo, z[t]);
          }
        }
      }
      if constexpr (P3)
#pragma unroll
        for (int t = 0; t < 2; t++) z[t] += zl[t];
    }
    const float A = __builtin_ldexpf(ca, ek + 22), Bm = __builtin_ldexpf(ca, ek) * msum[row & (NR - 1)];
    if (more) load_keys4(kf, km, t0 + NW * UNIT, uk);
    const bool masked = t0 + UNIT > all;
    const auto unseen = [&](int t, int r) { return masked && t0 + 16 * t + 4 * grp + r >= lim; };
    // weights times their factor, with the maximum as it stands; a lane's sum tells whether one of them has
    // outgrown its scale, or is infinite: a row that has seen nothing yet
    float p[2][4], lw, sum, bs;
    const auto weigh = [&](float B) {
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int r = 0; r < 4; r++) p[t][r] = exp2_fast(unseen(t, r) ? -INFINITY : __builtin_fmaf(z[t][r], A, B));
      sum = ((p[0][0] + p[0][1]) + (p[0][2] + p[0][3])) + ((p[1][0] + p[1][1]) + (p[1][2] + p[1][3]));
      bs = sum * exp2_fast(-lw);
    };
    const float lv = (float)ev;
    lw = fmaxf(lv + st.f, -60.0f);  // below 2^-60 the weights vanish either way
    weigh(Bm + (lw - st.mu));
    if (__any(fmaxf(sum, bs * 256.0f) > 32768.0f)) {
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int r = 0; r < 4; r++) top = fmaxf(top, unseen(t, r) ? -INFINITY : __builtin_fmaf(z[t][r], A, Bm));
      const float tm = row_max(top), mn = fmaxf(st.m, tm);
      float on = fmaxf(st.mo, tm + lv);
      const bool some = mn > -INFINITY;
      if (some) on = fmaxf(on, mn - 126.0f);  // keeps 2^(mo - m) a normal number beside weights that vanish
      const float al = st.m > -INFINITY ? exp2_fast(st.m - mn) : 0.0f;
      const float ao = st.mo > -INFINITY ? exp2_fast(st.mo - on) : 0.0f;
      st.l *= al;
#pragma unroll
      for (int j = 0; j < 8; j++) acc[j] *= ao;
      st.m = st.mu = mn;
      st.mo = on;
      st.f = some ? mn - on + 9.0f : 0.0f;
      lw = fmaxf(lv + st.f, -60.0f);
      weigh(Bm + (lw - (some ? mn : 0.0f)));
    }
    st.l += bs;
    uint32_t ph[2][2], pl[2][2];
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const float x = p[t][2 * k], y = p[t][2 * k + 1];
        ph[t][k] = pack_f16x2(x, y);
        if constexpr (!BF16) {
          const f2_t hh = unpack_f16x2(ph[t][k]);
          pl[t][k] = pack_f16x2(x - hh.x, y - hh.y);
        }
      }
    const h8_t P = as_h8(ph[0][0], ph[0][1], ph[1][0], ph[1][1]);
    if constexpr (BF16) {
      h2_t vs[2][2], vc[2][2];
#pragma unroll
      for (int t = 0; t < 2; t++) {
        const uint2 x = *(const uint2 *)(vget + 16 * t * VB), y = *(const uint2 *)(vget + 4 * VR + 16 * t * VB);
        vs[t][0] = __builtin_bit_cast(h2_t, x.x);
        vs[t][1] = __builtin_bit_cast(h2_t, x.y);
        vc[t][0] = __builtin_bit_cast(h2_t, y.x);
        vc[t][1] = __builtin_bit_cast(h2_t, y.y);
      }
#define CG_PV(B)                                                                                             \
  {                                                                                                          \
    uint32_t e[2][2], o[2][2];                                                                               \
    _Pragma("unroll") for (int t = 0; t < 2; t++) _Pragma("unroll") for (int i = 0; i < 2; i++) {            \
      uint32_t ce, co;                                                                                       \
      centred4<B>(uv.v[t][2 * i], uv.v[t][2 * i + 1], ce, co);                                               \
      e[t][i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(h2_t, ce), vs[t][i], vc[t][i])); \
      o[t][i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(h2_t, co), vs[t][i], vc[t][i])); \
    }                                                                                                        \
    acc[2 * B] = mfma(as_h8(e[0][0], e[0][1], e[1][0], e[1][1]), P, acc[2 * B]);                             \
    acc[2 * B + 1] = mfma(as_h8(o[0][0], o[0][1], o[1][0], o[1][1]), P, acc[2 * B + 1]);                     \
  }
      CG_PV(0) CG_PV(1) CG_PV(2) CG_PV(3)
#undef CG_PV
    } else {
      const h8_t Pl = as_h8(pl[0][0], pl[0][1], pl[1][0], pl[1][1]);
      f4_t vs[2], vc[2];
#pragma unroll
      for (int t = 0; t < 2; t++) {
        vs[t] = *(const f4_t *)(vget + 16 * t * VB);
        vc[t] = *(const f4_t *)(vget + 4 * VR + 16 * t * VB);
      }
#define CG_PV(B)                                                                                             \
  {                                                                                                          \
    uint32_t vh[2][2][2], vl[2][2][2];                                                                       \
    _Pragma("unroll") for (int t = 0; t < 2; t++) _Pragma("unroll") for (int i = 0; i < 2; i++) {            \
      uint32_t c[2];                                                                                         \
      centred4<B>(uv.v[t][2 * i], uv.v[t][2 * i + 1], c[0], c[1]);                                           \
      _Pragma("unroll") for (int k = 0; k < 2; k++) {                                                        \
        const f2_t x = unpack_f16x2(c[k]);                                                                   \
        const float y0 = __builtin_fmaf(x.x, vs[t][2 * i], vc[t][2 * i]);                                    \
        const float y1 = __builtin_fmaf(x.y, vs[t][2 * i + 1], vc[t][2 * i + 1]);                            \
        vh[k][t][i] = pack_f16x2(y0, y1);                                                                    \
        const f2_t hh = unpack_f16x2(vh[k][t][i]);                                                           \
        vl[k][t][i] = pack_f16x2(y0 - hh.x, y1 - hh.y);                                                      \
      }                                                                                                      \
    }                                                                                                        \
    _Pragma("unroll") for (int k = 0; k < 2; k++) {                                                          \
      const h8_t H = as_h8(vh[k][0][0], vh[k][0][1], vh[k][1][0], vh[k][1][1]);                              \
      acc[2 * B + k] = mfma(H, P, acc[2 * B + k]);                                                           \
      acc[2 * B + k] = mfma(H, Pl, acc[2 * B + k]);                                                          \
      acc[2 * B + k] = mfma(as_h8(vl[k][0][0], vl[k][0][1], vl[k][1][0], vl[k][1][1]), P, acc[2 * B + k]);   \
    }                                                                                                        \
  }
      CG_PV(0) CG_PV(1) CG_PV(2) CG_PV(3)
#undef CG_PV
    }
    if (more) load_values4(vf, vm, t0 + NW * UNIT, uv);
    wave_sync();  // the unit's LDS has been read
    if constexpr (MASS) {
      const float v = row_sum(bs);
      if (grp == 0 && row < nr) a.bsum[((int64_t)bh * a.entries + un) * a.rows + r0 + row] = make_float2(v, st.mu);
    }
  }

  const float *gv = a.gv + (int64_t)h * D * a.g;
  if (splits == 1 && front) load_gauge<true>(gv, a.g, 0, gw);
  // true sums: acc 2^(mo - m) less the 2^9 of the weights and of the values; a lane's channels are of group grp
  const FarSums far(st.m, st.mo);
#pragma unroll
  for (int j = 0; j < 8; j++) acc[j] *= far.is ? 1.0f : 0x1p-18f;
  const float ks = st.m > -INFINITY ? exp2_fast(far.up - far.less) : 0.0f;
  st.m += far.shift;
  st.l *= far.is ? 0x1p-32f : 1.0f;
  finish_few<BF16, NW>(a, fp, lds, ml, gv, gw, front, st.m, st.l, ks, (st.poison >> grp) & 1u ? NAN : 0.0f, acc);
}

hipError_t rows4_launch(const AttendArgs &a, bool bf16, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.heads * a.tiles * a.slots));
  const bool mass = a.mass && a.bsum, p3 = !bf16 || mass || a.lse;
  const int nr = a.rows <= 4 ? 4 : a.rows <= 8 ? 8 : 16;
#define CG_R(BF, P3, MA, NW, NR)                                                                 \
  if (bf16 == BF && p3 == P3 && mass == MA && a.waves == NW && nr == NR) {                       \
    hipLaunchKernelGGL((k_attend4_rows<BF, P3, MA, NW, NR>), grid, dim3(64 * NW), 0, s, a);      \
    return hipGetLastError();                                                                    \
  }
#define CG_RR(BF, P3, MA)                                                                        \
  CG_R(BF, P3, MA, 4, 4) CG_R(BF, P3, MA, 8, 4) CG_R(BF, P3, MA, 4, 8) CG_R(BF, P3, MA, 8, 8)    \
  CG_R(BF, P3, MA, 4, 16) CG_R(BF, P3, MA, 8, 16)
  CG_RR(true, false, false) CG_RR(true, true, false) CG_RR(true, true, true) CG_RR(false, true, false) CG_RR(false, true, true)
#undef CG_RR
#undef CG_R
  return hipErrorInvalidValue;
}

}  // namespace cga
