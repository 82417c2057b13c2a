// Attention of many query rows over the 8-bit cache: prompts, chunks of them
// and drafted tokens, bound by the vector units that make the weights.
//
// A workgroup takes 128 query rows of one KV head, 32 to each of its four
// waves (two row tiles), and walks the tokens 64 at a time: the codes and
// ranges of a stage go through registers into one of two LDS buffers while the
// other is worked on, one barrier a stage.  The products are those of the
// few-row kernel (attend_rows.hip) with the codes read from LDS and each
// widened operand used for both row tiles.  Rows of 16-byte pieces are stored
// with piece ^ (row % 8), so the 16 rows that a key operand's lanes read at
// one piece lie in different banks.
//
// The running maximum is not looked for: a lane's sum of weights tells whether
// one of them has outgrown its scale, and only then (and where a row sees its
// first token) the scores are formed again and the maximum raised.
#include "attend.hpp"

namespace cga {

constexpr int STAGE = 64;        // tokens of a stage
constexpr int TROWS = 128;       // query rows of a workgroup
constexpr int WT = 2;            // row tiles of a wave
constexpr int CODES = STAGE * D; // bytes of a stage's key (value) codes

struct StageRegs {
  uint4 k[2], v[2];
  float2 m;
};

// stage tokens [t0, t0 + 64) into registers; tokens past the capacity repeat
// its last rows
__device__ __forceinline__ void fetch_stage(const AttendArgs &a, const uint8_t *kf, const uint8_t *vf,
                                            const float2 *km, const float2 *vm, int t0, StageRegs &s) {
  const int i = threadIdx.x;
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const int64_t t = min((int64_t)t0 + 32 * k + (i >> 3), a.tcap - 1);
    s.k[k] = *(const uint4 *)(kf + t * D + 16 * (i & 7));
    s.v[k] = *(const uint4 *)(vf + t * D + 16 * (i & 7));
  }
  if (i < 8) {  // four 16-token tiles: key ranges, value ranges
    const int64_t blk = min(((int64_t)t0 + 16 * (i & 3)) >> a.bshift, a.nblk - 1);
    s.m = (i < 4 ? km : vm)[blk];
  }
}

__device__ __forceinline__ void put_stage(unsigned char *buf, const StageRegs &s) {
  const int i = threadIdx.x;
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const int r = 32 * k + (i >> 3), off = r * D + 16 * ((i & 7) ^ (r & 7));
    *(uint4 *)(buf + off) = s.k[k];
    *(uint4 *)(buf + CODES + off) = s.v[k];
  }
  if (i < 8) *(float2 *)(buf + 2 * CODES + 8 * i) = s.m;
}

constexpr int STAGE_LDS = 2 * CODES + 64;

struct TileState {
  float m, mu, mo, f, l, mv;
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

// LO: the queries' second fp16 part takes part (fp32 storage, or where log-sums
// or weights are asked for); else a query is rounded to 2^-11 of a channel
template <bool BF16, bool LO>
__global__ __launch_bounds__(NTH, 2) void k_attend_tile(const AttendArgs a) {
  static_assert(BF16 || LO, "fp32 storage takes both parts");
  __shared__ __align__(16) unsigned char lds[(TROWS + ROWS) * PITCH * 4];
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

  // gauged queries as operands of the wave that owns them
  QueryFrags q[WT];
  {
    float *xs = (float *)lds, *ys = xs + TROWS * PITCH;
#pragma unroll
    for (int t = 0; t < TROWS / ROWS; t++) load_rows<BF16>(a, b, h, r0 + t * ROWS, xs + t * ROWS * PITCH);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; w++)
#pragma unroll
      for (int t = 0; t < WT; t++) {
        gauge_rows<false>(xs + (w * WT + t) * ROWS * PITCH, ROWS, a.gk + (int64_t)h * D * a.g, a.g,
                          [&](int r, int c, float v) { ys[r * PITCH + c] = v; });
        __syncthreads();
        if (wave == w) make_frags<LO>(ys, a.c, q[t]);
        __syncthreads();
      }
  }
  int lim[WT], all = tmax, top = 0;
#pragma unroll
  for (int t = 0; t < WT; t++) {
    const int r = r0 + (wave * WT + t) * ROWS + row;
    lim[t] = r < a.rows ? query_limit(a, b, len, r / a.ratio) : 0;
    all = min(all, r < a.rows ? lim[t] : tmax);
    top = max(top, lim[t]);
    if (a.qfrag && split == 0) {  // for the pass that gives the blocks' weights
      const int64_t tile = (int64_t)bh * a.tiles + (r0 >> 4) + wave * WT + t;
      if (r0 + (wave * WT + t) * ROWS < a.rows) {
        uint4 *d = a.qfrag + tile * 8 * 64 + lane;
#pragma unroll
        for (int s = 0; s < 4; s++) {
          d[s * 64] = __builtin_bit_cast(uint4, q[t].hi[s]);
          d[(4 + s) * 64] = __builtin_bit_cast(uint4, q[t].lo[s]);
        }
        if (grp == 0) a.qrow[tile * ROWS + row] = make_float4(q[t].ca * kCentredUnit, q[t].cq, __int_as_float(lim[t]), 0.0f);
      }
    }
    q[t].ca *= BF16 ? kCodeUnit : kCentredUnit;
  }
#pragma unroll
  for (int k = 1; k < 16; k <<= 1) {
    all = min(all, __shfl_xor(all, k));
    top = max(top, __shfl_xor(top, k));
  }
  all = __builtin_amdgcn_readfirstlane(all);
  top = __builtin_amdgcn_readfirstlane(top);

  TileState st[WT];
  f4_t acc[WT][8];
#pragma unroll
  for (int t = 0; t < WT; t++) {
    st[t].m = st[t].mo = -INFINITY;
    st[t].mu = st[t].l = st[t].mv = 0.0f;
    st[t].f = 1.0f;
#pragma unroll
    for (int j = 0; j < 8; j++) acc[t][j] = f4_t{0.f, 0.f, 0.f, 0.f};
  }

  if (s0 < s1) put_stage(lds + (s0 & 1) * STAGE_LDS, nx);
  if (s0 + 1 < s1) fetch_stage(a, kf, vf, km, vm, (s0 + 1) * STAGE, nx);
  for (int sg = s0; sg < s1; sg++) {
    __syncthreads();
    if (sg + 1 < s1) put_stage(lds + ((sg + 1) & 1) * STAGE_LDS, nx);
    if (sg + 2 < s1) fetch_stage(a, kf, vf, km, vm, (sg + 2) * STAGE, nx);
    const unsigned char *buf = lds + (sg & 1) * STAGE_LDS;
#pragma unroll 1
    for (int half = 0; half < 2; half++) {
      const int t0 = sg * STAGE + half * UNIT;
      if (t0 >= top) break;
      const unsigned char *kb = buf + half * UNIT * D, *vb = kb + CODES;
      const float2 *mt = (const float2 *)(buf + 2 * CODES) + half * 2;
      f4_t z[WT][2];
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
              zl[t] = mfma(c0, q[t].lo[2 * x], zl[t]);
              zl[t] = mfma(c1, q[t].lo[2 * x + 1], zl[t]);
            }
          }
        }
        if constexpr (LO) {
#pragma unroll
          for (int t = 0; t < WT; t++) z[t][u] += zl[t];
        }
      }
      float2 mk[2], mv[2];
#pragma unroll
      for (int u = 0; u < 2; u++) {
        mk[u] = mt[u];
        mv[u] = mt[4 + u];
        if (!BF16) mk[u].x = __builtin_fmaf(128.0f, mk[u].y, mk[u].x);
        if (t0 + 16 * u >= tmax) mv[u] = make_float2(0.f, 0.f);  // a block that holds no row yet
        else mv[u].x = __builtin_fmaf(128.0f, mv[u].y, mv[u].x);
      }
      const bool masked = t0 + UNIT > all;
      float p[WT][2][4], ps[WT][2];
      bool up = false;
#pragma unroll
      for (int t = 0; t < WT; t++) {
#pragma unroll
        for (int u = 0; u < 2; u++) {
          const float A = mk[u].y * q[t].ca, B = mk[u].x * q[t].cq - st[t].mu;
#pragma unroll
          for (int r = 0; r < 4; r++) p[t][u][r] = __builtin_fmaf(z[t][u][r], A, B);
          if (masked) {
#pragma unroll
            for (int r = 0; r < 4; r++) p[t][u][r] = t0 + 16 * u + 4 * grp + r < lim[t] ? p[t][u][r] : -INFINITY;
          }
#pragma unroll
          for (int r = 0; r < 4; r++) p[t][u][r] = exp2_fast(p[t][u][r]);
          ps[t][u] = (p[t][u][0] + p[t][u][1]) + (p[t][u][2] + p[t][u][3]);
        }
        const float big = fmaxf(ps[t][0] * mv[0].y, ps[t][1] * mv[1].y) * st[t].f;
        up = up || ps[t][0] + ps[t][1] > 256.0f || big > 32768.0f || (st[t].m == -INFINITY && t0 < lim[t]);
      }
      if (__any(up)) {
#pragma unroll
        for (int t = 0; t < WT; t++) {
          float s[2][4], mx[2];
#pragma unroll
          for (int u = 0; u < 2; u++) {
            const float A = mk[u].y * q[t].ca, B = mk[u].x * q[t].cq;
#pragma unroll
            for (int r = 0; r < 4; r++)
              s[u][r] = t0 + 16 * u + 4 * grp + r < lim[t] ? __builtin_fmaf(z[t][u][r], A, B) : -INFINITY;
            mx[u] = fmaxf(fmaxf(s[u][0], s[u][1]), fmaxf(s[u][2], s[u][3]));
          }
          const float mn = fmaxf(st[t].m, row_max(fmaxf(mx[0], mx[1])));
          float on = fmaxf(st[t].mo, row_max(fmaxf(mx[0] + __builtin_amdgcn_logf(mv[0].y), mx[1] + __builtin_amdgcn_logf(mv[1].y))));
          const bool some = mn > -INFINITY;
          if (some) on = fmaxf(on, mn - 80.0f);
          const float al = st[t].m > -INFINITY ? exp2_fast(st[t].m - mn) : 0.0f;
          const float ao = st[t].mo > -INFINITY ? exp2_fast(st[t].mo - on) : 0.0f;
          st[t].l *= al;
          st[t].mv *= al;
#pragma unroll
          for (int j = 0; j < 8; j++) acc[t][j] *= ao;
          st[t].m = mn;
          st[t].mo = on;
          st[t].mu = some ? mn : 0.0f;
          st[t].f = some ? exp2_fast(mn - on + 9.0f) : 1.0f;
#pragma unroll
          for (int u = 0; u < 2; u++) {
#pragma unroll
            for (int r = 0; r < 4; r++) p[t][u][r] = exp2_fast(s[u][r] - st[t].mu);
            ps[t][u] = (p[t][u][0] + p[t][u][1]) + (p[t][u][2] + p[t][u][3]);
          }
        }
      }
      h8_t P[WT], Pl[WT];
#pragma unroll
      for (int t = 0; t < WT; t++) {
        uint32_t ph[2][2], pl[2][2];
#pragma unroll
        for (int u = 0; u < 2; u++) {
          st[t].l += ps[t][u];
          st[t].mv = __builtin_fmaf(mv[u].x, ps[t][u], st[t].mv);
          const float w = mv[u].y * st[t].f;
#pragma unroll
          for (int k = 0; k < 2; k++) {
            const float x = p[t][u][2 * k] * w, y = p[t][u][2 * k + 1] * w;
            ph[u][k] = pack_f16x2(x, y);
            if constexpr (!BF16) {
              const f2_t hh = unpack_f16x2(ph[u][k]);
              pl[u][k] = pack_f16x2(x - hh.x, y - hh.y);
            }
          }
        }
        P[t] = as_h8(ph[0][0], ph[0][1], ph[1][0], ph[1][1]);
        if constexpr (!BF16) Pl[t] = as_h8(pl[0][0], pl[0][1], pl[1][0], pl[1][1]);
      }
      uint2 v[2][4];
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int r = 16 * u + 4 * grp + i;
          v[u][i] = *(const uint2 *)(vb + r * D + 16 * ((row >> 1) ^ (r & 7)) + 8 * (row & 1));
        }
#define CG_PV(J)                                                     \
  {                                                                  \
    const h8_t vj = value_frag<J>(v);                                \
    _Pragma("unroll") for (int t = 0; t < WT; t++) {                 \
      acc[t][J] = mfma(vj, P[t], acc[t][J]);                         \
      if constexpr (!BF16) acc[t][J] = mfma(vj, Pl[t], acc[t][J]);   \
    }                                                                \
  }
      CG_PV(0) CG_PV(1) CG_PV(2) CG_PV(3) CG_PV(4) CG_PV(5) CG_PV(6) CG_PV(7)
#undef CG_PV
    }
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

hipError_t tile_launch(const AttendArgs &a, bool bf16, hipStream_t s) {
  const int64_t groups = (a.rows + TROWS - 1) / TROWS;
  const dim3 grid((unsigned)((int64_t)a.batch * a.heads * groups * a.splits)), block(NTH);
  if (!bf16) hipLaunchKernelGGL((k_attend_tile<false, true>), grid, block, 0, s, a);
  else if (a.lse || a.mass) hipLaunchKernelGGL((k_attend_tile<true, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_attend_tile<true, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace cga
