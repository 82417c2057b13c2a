// The weight each block of the 8-bit cache received from many query rows: a
// second pass over the keys with the queries' operands and the rows' log-sums
// that the attention left.
#include "attend.hpp"

namespace cga {

// A wave owns 32 tokens (64 where a block has 64: twice 32) of one field, holds
// their codes as operands and walks the row tiles: weights 2^(s - log2 sum),
// summed over rows and tokens of a block in a fixed order by their one owner.
__global__ __launch_bounds__(NTH) void k_mass_many(const AttendArgs a, int64_t groups) {
  const int lane = threadIdx.x & 63, row = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t wgs = (groups + 3) / 4;
  const int bh = (int)(blockIdx.x / wgs);
  const int64_t grpi = (blockIdx.x % wgs) * 4 + wave;
  const int b = bh / a.heads;
  const int len = seq_length(a, b);
  const int tmax = limit_of(a, b, len, 0, a.n - 1);
  const int per = a.bshift == 6 ? 2 : 1;
  if (grpi * per * UNIT >= tmax) return;
  const uint8_t *kf = a.kpay + (int64_t)bh * a.tcap * D;
  const float2 *km = a.kmeta + (int64_t)bh * a.nblk;
  float total[2] = {0.0f, 0.0f};
  for (int half = 0; half < per; half++) {
    const int t0 = (int)(grpi * per + half) * UNIT;
    if (t0 >= tmax) break;
    h8_t kc[2][4];
    float2 m[2];
#pragma unroll
    for (int t = 0; t < 2; t++) {
      const int64_t tt = min((int64_t)t0 + 16 * t, a.tcap - 16);  // 16-token blocks: the capacity may end here
#pragma unroll
      for (int x = 0; x < 4; x++) {
        const uint2 w = *(const uint2 *)(kf + (tt + row) * D + 32 * x + 8 * grp);
        kc[t][x] = codes8<true>(w.x, w.y);
      }
      m[t] = km[tt >> a.bshift];
    }
    float sum[2] = {0.0f, 0.0f};
    for (int tile = 0; tile < a.tiles; tile++) {
      const int r1 = min(a.rows, (tile + 1) * ROWS) - 1;
      if (limit_of(a, b, len, tile * ROWS / a.ratio, r1 / a.ratio) <= t0) continue;
      const int64_t id = (int64_t)bh * a.tiles + tile;
      const uint4 *qf = a.qfrag + id * 8 * 64 + lane;
      const float2 qr = a.qrow[id * ROWS + row];
      const int r = tile * ROWS + row;
      const int lim = r < a.rows ? query_limit(a, b, len, r / a.ratio) : 0;
      const float lse2 = r < a.rows ? a.lse2[(int64_t)bh * a.rows + r] : INFINITY;
      const f4_t none = f4_t{0.f, 0.f, 0.f, 0.f};
      f4_t z[2] = {none, none}, zl[2] = {none, none};
#pragma unroll
      for (int s = 0; s < 4; s++) {
        const h8_t qh = __builtin_bit_cast(h8_t, qf[s * 64]), ql = __builtin_bit_cast(h8_t, qf[(4 + s) * 64]);
#pragma unroll
        for (int t = 0; t < 2; t++) {
          z[t] = mfma(kc[t][s], qh, z[t]);
          zl[t] = mfma(kc[t][s], ql, zl[t]);
        }
      }
      z[0] += zl[0];
      z[1] += zl[1];
#pragma unroll
      for (int t = 0; t < 2; t++) {
        const float A = m[t].y * qr.x * kCentredUnit, Bm = __builtin_fmaf(128.0f, m[t].y, m[t].x) * qr.y - lse2;
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const float s = __builtin_fmaf(z[t][k], A, Bm);
          sum[t] += t0 + 16 * t + 4 * grp + k < lim ? exp2_fast(s) : 0.0f;
        }
      }
    }
    total[0] += sum[0];
    total[1] += sum[1];
  }
#pragma unroll
  for (int t = 0; t < 2; t++)
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) total[t] += __shfl_xor(total[t], k);
  if (lane) return;
  float *out = a.mass + (int64_t)bh * a.nblk;
  if (a.bshift == 4) {
    out[2 * grpi] += total[0];
    if (2 * grpi + 1 < a.nblk) out[2 * grpi + 1] += total[1];
  } else {
    out[grpi] += total[0] + total[1];
  }
}

hipError_t mass_many_launch(const AttendArgs &a, hipStream_t s) {
  const int64_t span = a.bshift == 6 ? 2 * UNIT : UNIT, groups = (a.tokens + span - 1) / span;
  const dim3 grid((unsigned)((int64_t)a.batch * a.heads * ((groups + 3) / 4))), block(NTH);
  hipLaunchKernelGGL(k_mass_many, grid, block, 0, s, a, groups);
  return hipGetLastError();
}

}  // namespace cga
