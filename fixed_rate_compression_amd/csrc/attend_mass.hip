// The weight each block of the 8-bit cache received from many query rows.  The
// attention has left, for every row and unit of tokens, the sum of 2^(score - m) and
// the m it stands on; with the row's log-sum each becomes a weight, and a block's
// are added up over its rows:
//   mass[block] += sum over rows of sum_t 2^(s_t - m) 2^(m - log2 sum)
// One wave to a block (four for many rows), its rows side by side, in a fixed order.
//
// Bound by the memory traffic of the sums: 8 bytes a row and 32 tokens, written
// once and read once.  2048 queries x 4 heads over 8192 tokens of 8 KV heads
// (134 MB): 23 us, prompts of 2 x 1000 tokens 6 us; a second pass over the keys with
// the log-sums known, the scores formed again, took 265 and 39.
#include "attend.hpp"

namespace cga {

template <int W>
__global__ __launch_bounds__(NTH) void k_mass_rows(const AttendArgs a, int groups) {
  __shared__ float red[NTH / 64];
  constexpr int PER = NTH / 64 / W;  // blocks to a workgroup
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int bh = (int)(blockIdx.x / (uint32_t)groups), b = bh / a.heads;
  const Sequence sq = load_sequence(a, b);
  const int tmax = limit_of(a, sq, 0, a.n - 1);
  // the same number of turns for all waves of a block
  for (int64_t blk = (int64_t)((int)blockIdx.x - bh * groups) * PER + wave / W; blk << a.bshift < tmax;
       blk += (int64_t)groups * PER) {
    const int64_t t0 = blk << a.bshift;
    float w = 0.0f;
    const int per = a.bshift == 6 ? 2 : 1, esh = min(a.bshift, 5);
    for (int k = 0; k < per; k++) {
      const int64_t te = t0 + ((int64_t)k << esh);
      // queries inside the sequence that see one of these tokens
      const int64_t i0 = max((a.causal ? te : 0) - sq.start, (int64_t)0);
      const int64_t i1 = te < tmax ? min((int64_t)a.n, (int64_t)sq.len - sq.start) : 0;
      const int r1 = (int)max(i1, (int64_t)0) * a.ratio;
      const float2 *p = a.bsum + ((int64_t)bh * a.entries + blk * per + k) * a.rows;
      const float *ls = a.lse2 + (int64_t)bh * a.rows;
#pragma unroll 8
      for (int r = (int)min(i0, (int64_t)a.n) * a.ratio + (wave % W) * 64 + lane; r < r1; r += 64 * W) {
        const float2 x = p[r];
        w = __builtin_fmaf(x.x, exp2_fast(x.y - ls[r]), w);
      }
    }
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1) w += __shfl_xor(w, k);
    if constexpr (W > 1) {
      if (lane == 0) red[wave] = w;
      __syncthreads();
      w = (red[0] + red[1]) + (red[2] + red[3]);
      __syncthreads();
    }
    if (lane == 0 && wave % W == 0) a.mass[(int64_t)bh * a.nblk + blk] += w;
  }
}

hipError_t mass_rows_launch(const AttendArgs &a, hipStream_t s) {
  // a wave to a block of few rows; 16 workgroups a compute unit at most, which take a
  // field's blocks in turn: the capacity may be far beyond what is there
  const int64_t fields = (int64_t)a.batch * a.heads, per = a.rows <= 512 ? 4 : 1;
  const int64_t most = (((a.tokens - 1) >> a.bshift) + per) / per, fit = (4096 + fields - 1) / fields;
  const int groups = (int)(most < fit ? most : fit);
  const dim3 grid((unsigned)(fields * groups));
  if (per == 4) hipLaunchKernelGGL(k_mass_rows<1>, grid, dim3(NTH), 0, s, a, groups);
  else hipLaunchKernelGGL(k_mass_rows<4>, grid, dim3(NTH), 0, s, a, groups);
  return hipGetLastError();
}

}  // namespace cga
