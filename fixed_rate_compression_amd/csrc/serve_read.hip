// Rows of a serving cache read back: decoded, turned by the inverse gauge and rounded
// to the storage format, each sequence's from its own position on.
//
// One workgroup takes 64 rows of one (K/V, sequence, head), wherever in a block they begin.
// Codes go from memory to a thread's 32 channels of a row; the ranges of 4-bit
// keys, one for a channel and 32 tokens, through LDS, since every row of a block reads them
// all.  The inverse gauge is the decoders': fmaf chains, or for bf16 storage and groups of
// 16 and 32 split bf16 products (split_gauge.hpp).
//
// 131072 rows of 8 heads in 8 bits 183 us (805 MB, 4.4 TB/s; a copy runs at 5.1), 1000 of 3 sequences in 4
// bits 7.7, which is a launch, the lengths, the codes and the gauge one after another.  Waves that keep 32
// channels of 32 rows in registers from the codes to the outputs took 258 and 8.8: 64-byte pieces of rows.
#include "cg_tile.hpp"
#include "quant_kernels.hpp"
#include "serve.hpp"
#include "split_gauge.hpp"

namespace cgs {

using namespace cgk;

template <bool BF16, int G, bool KIVI>
__global__ __launch_bounds__(NT) void k_read(const ReadArgs a) {
  constexpr bool SPLIT = BF16 && (G == 16 || G == 32);
  __shared__ __align__(16) float xs[TILE_T * PITCH];
  __shared__ __align__(16) float2 kr[KIVI ? 3 * D : 1];
  constexpr size_t ESZ = BF16 ? 2 : 4;
  // heads side by side: their rows lie next to one another in the output
  const uint32_t q1 = a.by_heads(blockIdx.x), q2 = a.by_tiles(q1), q3 = q2 / 2;
  const int h = (int)(blockIdx.x - q1 * a.heads), strip = (int)(q1 - q2 * a.tiles), kind = (int)(q2 & 1), b = (int)q3;
  uint8_t *dst = (uint8_t *)(kind ? a.v : a.k);
  if (!dst) return;
  const int32_t *any = (const int32_t *)a.payload;
  const int32_t ln = *(a.lengths ? a.lengths + b : any), sn = *(a.starts ? a.starts + b : any);
  const int64_t len = a.lengths ? min(max((int64_t)ln, (int64_t)0), a.tokens) : a.tokens;
  const int64_t start = a.starts ? (int64_t)sn : len - a.n;
  const int64_t i0 = (int64_t)strip * TILE_T, nrows = min((int64_t)TILE_T, a.n - i0);
  const int64_t p0 = start + i0, lo = max(p0, (int64_t)0), hi = min(p0 + nrows, len);  // positions that are there
  if (lo >= hi) return;
  const int64_t f = ((int64_t)kind * a.batch + b) * a.heads + h;
  const int t = threadIdx.x >> 2, j = threadIdx.x & 3;
  const int64_t p = p0 + t;
  const bool there = p >= lo && p < hi;
  const float *gf = G ? a.gauges + ((int64_t)kind * a.heads + h) * D * G : nullptr;
  TileGauge<SPLIT ? 0 : G, true> tg;
  SplitGaugeFrags<SPLIT ? G : 16> sg;
  if constexpr (SPLIT) load_split_gauge<G>(gf, sg);
  else if constexpr (G != 0) tg.load(gf);

  float v[32];
#pragma unroll
  for (int k = 0; k < 32; k++) v[k] = 0.0f;
  if constexpr (KIVI) {
    const float2 *mf = a.meta + f * 4 * a.tcap;
    uint32_t wd[4], q[32];
    if (there) cgq::load_words<4>(a.payload + (f * a.tcap + p) * (D / 2) + 16 * j, wd);
    float2 m = make_float2(0.f, 0.f);
    if (kind) {
      if (there) m = mf[p * 4 + j];
    } else {
      const int64_t b0 = lo >> 5, nb = ((hi - 1) >> 5) - b0 + 1;  // three blocks at most
      for (int i = threadIdx.x; i < (int)nb * D; i += NT) kr[i] = mf[b0 * D + i];
      __syncthreads();
    }
    if (there) {
      cgq::unpack32<4>(wd, q);
      if (kind) {
#pragma unroll
        for (int k = 0; k < 32; k++) v[k] = cgq::dequant1(q[k], m.x, m.y);
      } else {
        const float2 *r = kr + ((p >> 5) - (lo >> 5)) * D + 32 * j;
#pragma unroll
        for (int k = 0; k < 32; k++) v[k] = cgq::dequant1(q[k], r[k].x, r[k].y);
      }
    }
  } else if (there) {
    uint32_t wd[8], q[32];
    cgq::load_words<8>(a.payload + (f * a.tcap + p) * D + 32 * j, wd);
    const float2 m = a.meta[f * a.nblk + (p >> a.bshift)];
    cgq::unpack32<8>(wd, q);
#pragma unroll
    for (int k = 0; k < 32; k++) v[k] = cgq::dequant1(q[k], m.x, m.y);
  }
  if constexpr (SPLIT) {
    split_store32((unsigned char *)xs, t, j, v);
    __syncthreads();
    gauge_tile_split<G>((unsigned char *)xs, TILE_T, sg);
  } else {
    cgq::write32(xs, t, j, v);
    __syncthreads();
    if constexpr (G != 0) tg.apply(xs, TILE_T);
  }
  __syncthreads();
  constexpr int PER = (int)(D * ESZ / 16);  // 16-byte pieces of a row
  dst += ((int64_t)b * a.batch_stride + i0 * a.row_stride + (int64_t)h * D) * ESZ;
  for (int i = (int)(lo - p0) * PER + threadIdx.x; i < (int)(hi - p0) * PER; i += NT) {
    const int r = i / PER, c = i % PER;
    uint4 *o = (uint4 *)(dst + (int64_t)r * a.row_stride * ESZ + 16 * c);
    if (BF16) {
      const float *s = xs + r * PITCH + 8 * c;
      const float4 x = *(const float4 *)s, y = *(const float4 *)(s + 4);
      *o = make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    } else {
      *o = *(const uint4 *)(xs + r * PITCH + 4 * c);
    }
  }
}

hipError_t read_launch(const ReadArgs &a, bool bf16, int g, bool kivi, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)2 * a.batch * a.heads * a.tiles)), block(NT);
#define CG_R(BF, GG)                                                                \
  if (bf16 == BF && g == GG) {                                                      \
    if (kivi) hipLaunchKernelGGL((k_read<BF, GG, true>), grid, block, 0, s, a);     \
    else hipLaunchKernelGGL((k_read<BF, GG, false>), grid, block, 0, s, a);         \
    return hipGetLastError();                                                       \
  }
  CG_R(true, 0) CG_R(true, 8) CG_R(true, 16) CG_R(true, 32) CG_R(true, 128)
  CG_R(false, 0) CG_R(false, 8) CG_R(false, 16) CG_R(false, 32) CG_R(false, 128)
#undef CG_R
  return hipErrorInvalidValue;
}

}  // namespace cgs
