// Eviction by accumulated attention weight: which blocks of a head stay, and
// the cache's compaction.
//
// Blocks, not tokens, leave: a block's codes share one range, so whole blocks
// move as they are and nothing is quantized a second time.
#include "serve.hpp"

namespace cgs {

constexpr int ST = 1024;       // threads of a selecting workgroup
constexpr int SW = ST / 64;
constexpr int MT = 256;        // threads of a moving workgroup
constexpr int STEP = 4;        // 16-byte pieces a moving thread holds

// weights in an unsigned order: NaN below everything, -0 equal to +0
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int lanes_below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
}

// One workgroup per (layer, sequence, head).  The smallest kept weight is
// found eight bits at a time from the top (a radix selection: four counting
// passes over the weights, which stay in the L2), then one ordered pass
// writes the kept blocks' numbers and weights; blocks of that smallest weight
// stay in index order until the budget is met.
__global__ __launch_bounds__(ST) void k_evict_select(const EvictArgs a) {
  __shared__ int hist[SW][256];
  __shared__ int cnt[SW][2];
  __shared__ int pick[2];
  const int64_t id = blockIdx.x;
  const int b = (int)(id / a.heads % a.batch);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t len = min(max(a.lengths ? (int64_t)a.lengths[b] : a.tokens, (int64_t)0), a.tokens);
  const int n = (int)((len + a.block - 1) / a.block);
  const float *mass = a.mass + id * a.nblk;
  float *mo = a.mass_out + id * a.nblk_out;
  int32_t *kept = a.kept + id * a.budget;
  const bool all = n <= a.budget;
  const int lo = a.sink, hi = n - a.recent;  // blocks that compete
  uint32_t key = 0;
  int need = all ? 0 : a.budget - a.sink - a.recent;
  if (!all && need > 0) {
    for (int sft = 24; sft >= 0; sft -= 8) {
      for (int i = threadIdx.x; i < SW * 256; i += ST) (&hist[0][0])[i] = 0;
      __syncthreads();
      for (int i = lo + threadIdx.x; i < hi; i += ST) {
        const uint32_t k = order_key(mass[i]);
        if (sft == 24 || (k >> (sft + 8)) == (key >> (sft + 8))) atomicAdd(&hist[wave][(k >> sft) & 255], 1);
      }
      __syncthreads();
      if (threadIdx.x < 256) {
        int c = 0;
        for (int w = 0; w < SW; w++) c += hist[w][threadIdx.x];
        hist[0][threadIdx.x] = c;
      }
      __syncthreads();
      if (wave == 0) {  // lane l: bins 255 - 4 l .. 252 - 4 l, from the top
        int c[4], s = 0;
        for (int k = 0; k < 4; k++) {
          c[k] = hist[0][255 - 4 * lane - k];
          s += c[k];
        }
        int before = s;
        for (int k = 1; k < 64; k <<= 1) {
          const int o = __shfl_up(before, k);
          if (lane >= k) before += o;
        }
        before -= s;
        for (int k = 0; k < 4; k++) {
          if (before < need && before + c[k] >= need) {
            pick[0] = 255 - 4 * lane - k;
            pick[1] = need - before;
          }
          before += c[k];
        }
      }
      __syncthreads();
      key |= (uint32_t)pick[0] << sft;
      need = pick[1];
      __syncthreads();
    }
  }
  // need: how many blocks of weight `key` stay
  int out = 0, ties = 0;
  for (int i0 = 0; i0 < n; i0 += ST) {
    const int i = i0 + threadIdx.x;
    const float x = i < n ? mass[i] : 0.0f;
    bool stay = false, tie = false;
    if (i < n) {
      if (all || i < lo || i >= hi) {
        stay = true;
      } else if (a.budget > a.sink + a.recent) {
        const uint32_t k = order_key(x);
        stay = k > key;
        tie = k == key;
      }
    }
    const uint64_t mt = __ballot(tie);
    if (lane == 0) cnt[wave][1] = __popcll(mt);
    __syncthreads();
    int tr = ties + lanes_below(mt);
    for (int w = 0; w < SW; w++) {
      if (w < wave) tr += cnt[w][1];
      ties += cnt[w][1];
    }
    if (tie && tr < need) stay = true;
    const uint64_t ms = __ballot(stay);
    if (lane == 0) cnt[wave][0] = __popcll(ms);
    __syncthreads();
    int at = out + lanes_below(ms);
    for (int w = 0; w < SW; w++) {
      if (w < wave) at += cnt[w][0];
      out += cnt[w][0];
    }
    if (stay) {  // at <= i, and this pass has read its weights: mass_out may be mass
      kept[at] = i;
      mo[at] = x;
    }
    __syncthreads();
  }
  for (int i = out + threadIdx.x; i < a.budget; i += ST) kept[i] = -1;
  for (int64_t i = out + threadIdx.x; i < a.nblk_out; i += ST) mo[i] = 0.0f;
}

// Kept blocks to their places.  In place one workgroup walks a field in
// order: a block moves to a lower or equal number, so once a piece has been
// read by all threads everything up to it may be overwritten.  Into another
// cache the field is cut into `chunks`.
__global__ __launch_bounds__(MT) void k_evict_move(const EvictArgs a, int chunks) {
  const int64_t f = blockIdx.x / chunks;  // (layer, kind, b, h)
  const int chunk = (int)(blockIdx.x % chunks);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.batch; b += MT) {
      const int64_t len = min(max(a.lengths ? (int64_t)a.lengths[b] : a.tokens, (int64_t)0), a.tokens);
      const int64_t n = (len + a.block - 1) / a.block;
      a.lengths_out[b] = (int32_t)(n > a.budget ? len - (n - a.budget) * a.block : len);
    }
  const int64_t bh = f % ((int64_t)a.batch * a.heads), layer = f / ((int64_t)2 * a.batch * a.heads);
  const int32_t *kept = a.kept + (layer * a.batch * a.heads + bh) * a.budget;
  const float2 *ms = a.meta + f * a.nblk;
  float2 *md = a.meta_out + f * a.nblk_out;
  const int64_t bytes = (int64_t)a.block * 128;
  const uint8_t *src = a.payload + f * a.nblk * bytes;
  uint8_t *dst = a.payload_out + f * a.nblk_out * bytes;
  const int per = (int)(bytes / 16);  // 16-byte pieces of a block
  const int b0 = (int)((int64_t)a.budget * chunk / chunks), b1 = (int)((int64_t)a.budget * (chunk + 1) / chunks);
  for (int j0 = b0; j0 < b1; j0 += MT) {
    const int j = j0 + (int)threadIdx.x;
    const int s = j < b1 ? kept[j] : -1;
    float2 m = make_float2(0.f, 0.f);
    if (s >= 0) m = ms[s];
    if (a.in_place) __syncthreads();
    if (s >= 0) md[j] = m;
    if (a.in_place) __syncthreads();
  }
  const int64_t p0 = (int64_t)b0 * per, p1 = (int64_t)b1 * per;
  for (int64_t p = p0; p < p1; p += MT * STEP) {
    uint4 v[STEP];
    int s[STEP];
#pragma unroll
    for (int k = 0; k < STEP; k++) {
      const int64_t x = p + (int64_t)k * MT + threadIdx.x;
      s[k] = x < p1 ? kept[x / per] : -1;
      if (s[k] >= 0) v[k] = *(const uint4 *)(src + s[k] * bytes + (x % per) * 16);
    }
    if (a.in_place) __syncthreads();
#pragma unroll
    for (int k = 0; k < STEP; k++) {
      const int64_t x = p + (int64_t)k * MT + threadIdx.x;
      if (s[k] >= 0) *(uint4 *)(dst + x * 16) = v[k];
    }
    if (a.in_place) __syncthreads();
  }
}

hipError_t evict_launch(const EvictArgs &a, hipStream_t s) {
  const int64_t heads = (int64_t)a.layers * a.batch * a.heads;
  hipLaunchKernelGGL(k_evict_select, dim3((unsigned)heads), dim3(ST), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  int64_t chunks = 1;
  if (!a.in_place) {  // four workgroups a compute unit, 16 KB at least to each
    const int64_t bytes = (int64_t)a.budget * a.block * 128;
    chunks = (1024 + 2 * heads - 1) / (2 * heads);
    if (chunks > (bytes + 16383) / 16384) chunks = (bytes + 16383) / 16384;
    if (chunks > a.budget) chunks = a.budget;
  }
  hipLaunchKernelGGL(k_evict_move, dim3((unsigned)(2 * heads * chunks)), dim3(MT), 0, s, a, (int)chunks);
  return hipGetLastError();
}

}  // namespace cgs
