// How a workgroup of few-row attention ends, whatever the cache's format: its waves'
// sums joined, and parts for a merge or outputs.  Not part of the public ABI.
#pragma once

#include "attend.hpp"

namespace cga {

// the workgroup's rows [r0, r0 + nr) of (b, h) and its share of the tokens
struct FewPlace {
  int b, h, tile, slot, split, splits;
  int64_t part;  // where this part's row 0 goes
  int r0, nr;
};

// A wave's lane (row = lane % 16, grp = lane / 16) brings the maximum m (the same in a
// row's four lanes), its part l of the sum of weights and the sums of channels
// 8 (4 grp + r) + j, ks acc[j][r] + mv.  lds: NW ROWS PITCH floats, free once the waves
// have met; gv, gw: the inverse gauge, loaded where there is one split.
template <bool BF16, int NW>
__device__ __forceinline__ void finish_few(const AttendArgs &a, const FewPlace &p, float *lds, float2 (*ml)[ROWS],
                                           const float *gv, const GaugeFrag &gw, bool front, float m, float lsum,
                                           float ks, float mv, const f4_t (&acc)[8]) {
  const int lane = threadIdx.x & 63, row = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = p.b, h = p.h, splits = p.splits, r0 = p.r0, nr = p.nr;
  // join the waves: each leaves its sums relative to its own maximum
  __syncthreads();  // the operands have been read
  const float l = row_sum(lsum);
  if (grp == 0) ml[wave][row] = make_float2(m, l);
  {
    float *o = lds + (wave * ROWS + row) * PITCH;
#pragma unroll
    for (int r = 0; r < 4; r++) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; j++) v[j] = __builtin_fmaf(acc[j][r], ks, mv);
      *(float4 *)(o + 8 * (4 * grp + r)) = make_float4(v[0], v[1], v[2], v[3]);
      *(float4 *)(o + 8 * (4 * grp + r) + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
  __syncthreads();
  // for the merge (a store before the loop turns its scalar loads into vector ones)
  if (a.ragged && h == 0 && p.tile == 0 && p.split == 0 && threadIdx.x == 0)
    a.dealt[b] = make_int2(p.slot, splits);
  for (int i = threadIdx.x; i < ROWS * (D / 4); i += 64 * NW) {  // also rows that are not there: none is left undefined
    const int r = i / (D / 4), c = 4 * (i % (D / 4));
    float M = -INFINITY;
#pragma unroll
    for (int k = 0; k < NW; k++) M = fmaxf(M, ml[k][r].x);
    float L = 0.0f;
    f4_t v = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NW; k++) {
      const float2 w = ml[k][r];
      const float f = w.x > -INFINITY ? exp2_fast(w.x - M) : 0.0f;
      L += w.y * f;
      v += *(const f4_t *)(lds + (k * ROWS + r) * PITCH + c) * f;
    }
    const int64_t pr = p.part + r0 + r;
    if (c == 0 && r < nr) {
      if (a.part_ml) a.part_ml[pr] = make_float2(M, L);
      if (splits == 1 && a.lse) store_lse(a, b, h, r0 + r, M, L);
    }
    if (splits > 1) {
      if (r < nr) *(f4_t *)(a.part_o + pr * D + c) = v;
    } else {
      *(f4_t *)(lds + r * PITCH + c) = v * (L > 0.0f ? 1.0f / L : 0.0f);  // this thread alone reads these channels of row r
    }
  }
  if (splits > 1) return;
  __syncthreads();
  float *os = lds;
  if (a.g) {
    os = lds + ROWS * PITCH;
    if (front) gauge_tiles<true, 1, false>(lds, os, gv, a.g, gw);
    __syncthreads();
  }
  if (front) store_rows<BF16>(a, b, h, r0, nr, os);
}

}  // namespace cga
