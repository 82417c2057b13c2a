// The weight each block of the 8-bit cache received from many query rows: a
// second pass over the keys with the queries' operands and the rows' log-sums
// that the attention left.  No row's state is carried, so the work splits over
// tokens and rows alike; a workgroup's share of a block's sum goes to a slot of
// its own and the slots are added in order (no atomics: the same bits every time).
// Bound like the attention by matrix and vector work that hardly overlap: two
// products and an exponential a score.  2048 queries x 4 heads over 8192 tokens of 8
// KV heads 265 us, two prompts to 1000 tokens 34 us and 4.6 to add the slots.
#include "attend.hpp"

namespace cga {

typedef float f16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

constexpr int QT = 32;                  // query rows of a step
constexpr int QBYTES = 2 * 8 * 64 * 16; // their operands, two row tiles
constexpr int QSTEP = QBYTES + QT * 16; // and (score factor, minimum factor, log-sum, limit) of each row

struct QueryRegs {
  u4_t q0, q1, q2, q3;
  float4 r;
};

__device__ __forceinline__ void fetch_queries(const AttendArgs &a, int bh, const Sequence &sq, int step, QueryRegs &s) {
  const int i = threadIdx.x;
  const int64_t t0 = (int64_t)bh * a.tiles + min(2 * step, a.tiles - 1);
  const int64_t t1 = (int64_t)bh * a.tiles + min(2 * step + 1, a.tiles - 1);
  const u4_t *p0 = (const u4_t *)(a.qfrag + t0 * 512), *p1 = (const u4_t *)(a.qfrag + t1 * 512);
  s.q0 = p0[i];
  s.q1 = p0[256 + i];
  s.q2 = p1[i];
  s.q3 = p1[256 + i];
  const int row = i & (QT - 1), r = step * QT + row, rr = min(r, a.rows - 1);
  const float2 f = a.qrow[(int64_t)bh * a.tiles * ROWS + rr];
  s.r = make_float4(f.x * kCentredUnit, f.y, a.lse2[(int64_t)bh * a.rows + rr],
                    __int_as_float(r < a.rows ? query_limit(a, sq, (int)((uint32_t)r / (uint32_t)a.ratio)) : 0));
}

__device__ __forceinline__ void put_queries(unsigned char *buf, const QueryRegs &s) {
  u4_t *d = (u4_t *)buf;
  const int i = threadIdx.x;
  d[i] = s.q0;
  d[256 + i] = s.q1;
  d[512 + i] = s.q2;
  d[768 + i] = s.q3;
  if (i < QT) *(float4 *)(buf + QBYTES + 16 * i) = s.r;
}

// A workgroup: 256 tokens of a field, 64 to a wave (held as operands), against
// a part of the query rows, 32 at a time through LDS.  NB: blocks to 32 tokens
// (one also where a block has 64).
template <int NB>
__global__ __launch_bounds__(NTH, 2) void k_mass_many(const AttendArgs a) {
  __shared__ __align__(16) unsigned char lds[2 * QSTEP];
  const int lane = threadIdx.x & 63, row = lane & 31, half = lane >> 5, n = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fields = a.batch * a.heads;
  const uint32_t q1 = blockIdx.x / (uint32_t)fields;
  const int bh = (int)(blockIdx.x - q1 * fields);
  const int tg = (int)(q1 / (uint32_t)a.mparts), part = (int)q1 - tg * a.mparts;
  const int b = bh / a.heads;
  const Sequence sq = load_sequence(a, b);
  const int tmax = limit_of(a, sq, 0, a.n - 1);
  const int w0 = tg * 256;
  if (w0 >= tmax) return;
  // the row steps that see one of these tokens, this workgroup's part of them
  const int64_t i0 = a.causal ? max((int64_t)w0 - sq.start, (int64_t)0) : 0;
  const int steps = (a.rows + QT - 1) / QT;
  const int s_lo = (int)min(i0 * a.ratio / QT, (int64_t)steps);
  const int s0 = s_lo + split_begin(steps - s_lo, part, a.mparts), s1 = s_lo + split_begin(steps - s_lo, part + 1, a.mparts);
  const int t0 = w0 + 64 * wave;

  const uint8_t *kf = a.kpay + (int64_t)bh * a.tcap * D;
  const float2 *km = a.kmeta + (int64_t)bh * a.nblk;
  QueryRegs nx;
  if (s0 < s1) fetch_queries(a, bh, sq, s0, nx);
  h8_t kc[2][8];
  float2 m[2][NB];
#pragma unroll
  for (int u = 0; u < 2; u++) {
    const int64_t t = min((int64_t)t0 + 32 * u + row, a.tcap - 1);  // tokens past the capacity repeat its last row
#pragma unroll
    for (int s = 0; s < 8; s++) {
      const uint2 w = *(const uint2 *)(kf + t * D + 16 * s + 8 * half);
      kc[u][s] = codes8<true>(w.x, w.y);
    }
#pragma unroll
    for (int k = 0; k < NB; k++) {
      const int64_t tt = (int64_t)t0 + 32 * u + 16 * k;
      float2 x = km[min(tt >> a.bshift, a.nblk - 1)];
      x.x = __builtin_fmaf(128.0f, x.y, x.x);
      m[u][k] = tt < tmax ? x : make_float2(0.f, 0.f);  // a block that holds no row yet
    }
  }
  float sum[2][NB];
#pragma unroll
  for (int u = 0; u < 2; u++)
#pragma unroll
    for (int k = 0; k < NB; k++) sum[u][k] = 0.0f;
  if (s0 < s1) put_queries(lds, nx);
  if (s0 + 1 < s1) fetch_queries(a, bh, sq, s0 + 1, nx);
  for (int st = s0; st < s1; st++) {
    __syncthreads();
    const unsigned char *buf = lds + ((st - s0) & 1) * QSTEP;
    if (st + 1 < s1) put_queries(lds + ((st + 1 - s0) & 1) * QSTEP, nx);
    if (st + 2 < s1) fetch_queries(a, bh, sq, st + 2, nx);
    const unsigned char *qb = buf + (row >> 4) * 8192 + 16 * n;
    f16_t z[2], zl[2];
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
      for (int r = 0; r < 16; r++) z[u][r] = zl[u][r] = 0.0f;
#pragma unroll
    for (int s = 0; s < 8; s++) {
      const int c = 2 * s + half, at = ((c >> 2) * 64 + (c & 3) * 16) * 16;
      const h8_t qh = *(const h8_t *)(qb + at), ql = *(const h8_t *)(qb + 4096 + at);
#pragma unroll
      for (int u = 0; u < 2; u++) {
        z[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kc[u][s], qh, z[u], 0, 0, 0);
        zl[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kc[u][s], ql, zl[u], 0, 0, 0);
      }
    }
    const float4 rp = *(const float4 *)(buf + QBYTES + 16 * row);
    const int lim = __float_as_int(rp.w) - t0 - 4 * half;
    const bool masked = __any(lim < 64 - 4 * half);  // some row does not see all of the wave's tokens
#pragma unroll
    for (int u = 0; u < 2; u++) {
      z[u] += zl[u];
#pragma unroll
      for (int k = 0; k < NB; k++) {
        const float A = m[u][k].y * rp.x, B = __builtin_fmaf(m[u][k].x, rp.y, -rp.z);
        float p[16 / NB];
#pragma unroll
        for (int e = 0; e < 16 / NB; e++) p[e] = __builtin_fmaf(z[u][16 / NB * k + e], A, B);
        if (masked) {
#pragma unroll
          for (int e = 0; e < 16 / NB; e++) {
            const int r = 16 / NB * k + e;
            p[e] = 32 * u + 8 * (r >> 2) + (r & 3) < lim ? p[e] : -INFINITY;
          }
        }
#pragma unroll
        for (int e = 0; e < 16 / NB; e++) p[e] = exp2_fast(p[e]);
#pragma unroll
        for (int w = 8 / NB; w >= 1; w >>= 1)
#pragma unroll
          for (int e = 0; e < w; e++) p[e] += p[e + w];
        sum[u][k] += p[0];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < 2; u++)
#pragma unroll
    for (int k = 0; k < NB; k++)
#pragma unroll
      for (int x = 1; x < 64; x <<= 1) sum[u][k] += __shfl_xor(sum[u][k], x);
  if (lane) return;
  float *out = a.mpart + ((int64_t)part * fields + bh) * a.nblk;
  if (a.bshift == 6) {
    if (t0 < tmax) out[t0 >> 6] = sum[0][0] + sum[1][0];
    return;
  }
#pragma unroll
  for (int u = 0; u < 2; u++)
#pragma unroll
    for (int k = 0; k < NB; k++) {
      const int t = t0 + 32 * u + 16 * k;
      if (t < tmax) out[t >> a.bshift] = sum[u][k];
    }
}

__global__ __launch_bounds__(NTH) void k_mass_add(const AttendArgs a) {
  const int fields = a.batch * a.heads;
  const uint32_t chunks = (uint32_t)((a.nblk + NTH - 1) / NTH);
  const int bh = (int)(blockIdx.x / chunks), b = bh / a.heads;
  const int64_t blk = (int64_t)(blockIdx.x - bh * chunks) * NTH + threadIdx.x;
  if (blk >= a.nblk || (blk << a.bshift) >= limit_of(a, load_sequence(a, b), 0, a.n - 1)) return;
  float w = 0.0f;
#pragma unroll 8
  for (int p = 0; p < a.mparts; p++) w += a.mpart[((int64_t)p * fields + bh) * a.nblk + blk];
  a.mass[(int64_t)bh * a.nblk + blk] += w;
}

hipError_t mass_many_launch(const AttendArgs &a, hipStream_t s) {
  const int64_t fields = (int64_t)a.batch * a.heads, tg = (a.tokens + 255) / 256;
  const dim3 grid((unsigned)(fields * tg * a.mparts)), block(NTH);
  if (a.bshift == 4) hipLaunchKernelGGL(k_mass_many<2>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(k_mass_many<1>, grid, block, 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_mass_add, dim3((unsigned)(fields * ((a.nblk + NTH - 1) / NTH))), block, 0, s, a);
  return hipGetLastError();
}

}  // namespace cga
