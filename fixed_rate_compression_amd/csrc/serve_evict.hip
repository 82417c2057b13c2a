// Eviction by accumulated attention weight: which blocks of a head stay, and
// the cache's compaction.
//
// Blocks, not tokens, leave: a block's codes share one range, so whole blocks
// move as they are and nothing is quantized a second time.
#include "cg_wave.hpp"
#include "serve.hpp"

namespace cgs {

constexpr int ST = 1024;       // threads of a selecting workgroup
constexpr int SW = ST / 64;
constexpr int MT = 256;        // threads of a moving workgroup
constexpr int STEP = 8;        // 16-byte pieces a moving thread holds
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));  // an array of these stays in registers (of uint4 it did not)

// weights in an unsigned order: NaN below everything, -0 equal to +0
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int lanes_below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
}

// Up to 4096 blocks a head: their weights stay in registers, K to a thread, block e
// 256 + thread.  The smallest kept weight is built from its top bit down, each bit
// by a count of the weights at or above it, until the count is the number to keep
// or the bits end; then one ordered pass writes the kept blocks' numbers and
// weights, blocks of that smallest weight in index order until the budget is met.
// 256 heads of 256 blocks 5.6 us, by the four counting passes below 8.5; 128 heads of
// 2500 10.9 and 11.8, of 4096 12.9 and 14.8.
constexpr int PT = 256, PW = PT / 64;
template <int K>
__global__ __launch_bounds__(PT) void k_evict_pick(const EvictArgs a) {
  __shared__ int cnt[2][PW];
  __shared__ int part[2][K * PW > 64 ? K * PW : 64];  // ties, kept blocks of (e, wave)
  const int64_t id = blockIdx.x;
  const int b = (int)(blockIdx.x / (uint32_t)a.heads % (uint32_t)a.batch);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t len = min(max(a.lengths ? (int64_t)a.lengths[b] : a.tokens, (int64_t)0), a.tokens);
  const int n = (int)((len + a.block - 1) / a.block);
  const float *mass = a.mass + id * a.nblk;
  float *mo = a.mass_out + id * a.nblk_out;
  int32_t *kept = a.kept + id * a.budget;
  const bool all = n <= a.budget;
  const int lo = a.sink, hi = n - a.recent;  // blocks that compete
  float x[K];
  uint32_t key[K];  // 0: not competing, or NaN
#pragma unroll
  for (int e = 0; e < K; e++) {
    const int i = e * PT + (int)threadIdx.x;
    x[e] = i < n ? mass[i] : 0.0f;
  }
#pragma unroll
  for (int e = 0; e < K; e++) {
    const int i = e * PT + (int)threadIdx.x;
    key[e] = i >= lo && i < hi ? order_key(x[e]) : 0u;
  }
  const int want = all ? 0 : a.budget - a.sink - a.recent;
  // count of the competing weights of at least c (> 0); one barrier, `turn` alternates
  const auto at_least = [&](uint32_t c, int turn) {
    int m = 0;
#pragma unroll
    for (int e = 0; e < K; e++) m += __popcll(__ballot(key[e] >= c));
    if (lane == 0) cnt[turn & 1][wave] = m;
    __syncthreads();
    return (cnt[turn & 1][0] + cnt[turn & 1][1]) + (cnt[turn & 1][2] + cnt[turn & 1][3]);
  };
  // the largest `least` that `want` weights reach; `above`: how many pass it for certain
  uint32_t least = 0;
  int above = 0;
  bool exact = want == 0;  // all that reach `least` stay
  if (want > 0) {
    for (int bit = 31; bit >= 0; bit--) {
      const uint32_t c = least | 1u << bit;
      const int m = at_least(c, bit);
      if (m >= want) least = c;
      else above = m;
      if (m == want) {
        exact = true;
        break;
      }
    }
  }
  const int need = want - above;  // how many of weight `least` stay (where not exact)
  uint64_t stay[K], tie[K];
#pragma unroll
  for (int e = 0; e < K; e++) {
    const int i = e * PT + (int)threadIdx.x;
    const bool mid = i >= lo && i < hi && !all;
    stay[e] = __ballot(i < n && (!mid || (want > 0 && (exact ? key[e] >= least : key[e] > least))));
    tie[e] = exact ? 0ull : __ballot(mid && key[e] == least);
  }
  // positions: entry (e, wave) of part begins where the entries before it end
  if (!exact) {
#pragma unroll
    for (int e = 0; e < K; e++)
      if (lane == e) part[0][e * PW + wave] = __popcll(tie[e]);
    __syncthreads();
    const int v = lane < K * PW ? part[0][lane] : 0, end = cgw::wave_scan(v);
#pragma unroll
    for (int e = 0; e < K; e++) {
      const int before = __builtin_amdgcn_readlane(end - v, e * PW + wave);
      const bool mine = (tie[e] >> lane & 1) && before + lanes_below(tie[e]) < need;
      stay[e] |= __ballot(mine);
    }
  }
#pragma unroll
  for (int e = 0; e < K; e++)
    if (lane == e) part[1][e * PW + wave] = __popcll(stay[e]);
  __syncthreads();  // every weight has been read: mass_out may be mass
  const int v = lane < K * PW ? part[1][lane] : 0, end = cgw::wave_scan(v);
  const int out = __builtin_amdgcn_readlane(end, 63);
#pragma unroll
  for (int e = 0; e < K; e++) {
    const int at = __builtin_amdgcn_readlane(end - v, e * PW + wave) + lanes_below(stay[e]);
    if (stay[e] >> lane & 1) {
      kept[at] = e * PT + (int)threadIdx.x;
      mo[at] = x[e];
    }
  }
  for (int i = out + (int)threadIdx.x; i < a.budget; i += PT) kept[i] = -1;
  for (int64_t i = out + (int)threadIdx.x; i < a.nblk_out; i += PT) mo[i] = 0.0f;
}

// More: one workgroup per (layer, sequence, head).  The smallest kept weight is found
// eight bits at a time from the top: four counting passes over weights held in
// registers (past 8192 blocks: read again).  Then the ordered pass, as above.  128
// heads of 8192 blocks 21 us.
constexpr int HELD = 8;
__global__ __launch_bounds__(ST) void k_evict_select(const EvictArgs a) {
  __shared__ int hist[SW][256];
  __shared__ int cnt[SW][2];
  __shared__ int pick[2];
  const int64_t id = blockIdx.x;
  const int b = (int)(blockIdx.x / (uint32_t)a.heads % (uint32_t)a.batch);
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
    uint32_t held[HELD];
#pragma unroll
    for (int e = 0; e < HELD; e++) {
      const int i = threadIdx.x + e * ST;
      held[e] = i >= lo && i < hi ? order_key(mass[i]) : 0u;
    }
    for (int sft = 24; sft >= 0; sft -= 8) {
      for (int i = threadIdx.x; i < SW * 256; i += ST) (&hist[0][0])[i] = 0;
      __syncthreads();
      const auto count = [&](uint32_t k) {
        if (sft == 24 || (k >> (sft + 8)) == (key >> (sft + 8))) atomicAdd(&hist[wave][(k >> sft) & 255], 1);
      };
#pragma unroll
      for (int e = 0; e < HELD; e++) {
        const int i = threadIdx.x + e * ST;
        if (i >= lo && i < hi) count(held[e]);
      }
      for (int i = threadIdx.x + HELD * ST; i < hi; i += ST)
        if (i >= lo) count(order_key(mass[i]));
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
// cache the field is cut into `chunks`.  Half of 32 layers x 8 heads x 8192 tokens
// (269 MB each way): 106 us, 4.9 TB/s, a large copy's 5.1.
// KIVI: a block's ranges move as its codes do (half of 32 layers x 8 heads x 8192 tokens, 201 MB each way:
// 79 us of 85, 5.1 TB/s).
template <bool KIVI>
__global__ __launch_bounds__(MT) void k_evict_move(const EvictArgs a, int chunks) {
  const uint32_t f32 = blockIdx.x / (uint32_t)chunks, heads = (uint32_t)(a.batch * a.heads);
  const int chunk = (int)(blockIdx.x - f32 * chunks);
  const int64_t f = f32;  // (layer, kind, b, h)
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.batch; b += MT) {
      const int64_t len = min(max(a.lengths ? (int64_t)a.lengths[b] : a.tokens, (int64_t)0), a.tokens);
      const int64_t n = (len + a.block - 1) / a.block;
      a.lengths_out[b] = (int32_t)(n > a.budget ? len - (n - a.budget) * a.block : len);
    }
  const uint32_t layer = f32 / (2 * heads), bh = f32 % heads;
  const int32_t *kept = a.kept + ((int64_t)layer * heads + bh) * a.budget;
  const int each = (a.budget + chunks - 1) / chunks, b0 = min(chunk * each, a.budget), b1 = min(b0 + each, a.budget);
  __shared__ int32_t from[MT];  // former numbers of the blocks [j0, j0 + MT)
  for (int j0 = b0; j0 < b1; j0 += MT) {
    const int j = j0 + (int)threadIdx.x;
    const int s = j < b1 ? kept[j] : -1;
    __syncthreads();
    from[threadIdx.x] = s;
    if constexpr (KIVI) {
      __syncthreads();
    } else {
      const float2 *ms = a.meta + f * a.nblk;
      float2 *md = a.meta_out + f * a.nblk_out;
      float2 m = make_float2(0.f, 0.f);
      if (s >= 0) m = ms[s];
      __syncthreads();
      if (s >= 0) md[j] = m;  // in place: at or below any number that is still to be read
    }
    // blocks of 1 << sh pieces
    const auto move = [&](const void *from_field, void *to_field, int sh) {
      const int per = 1 << sh, np = min(MT, b1 - j0) << sh;
      const u4_t *src = (const u4_t *)from_field + f * a.nblk * per;
      u4_t *dst = (u4_t *)to_field + f * a.nblk_out * per;
      for (int p = 0; p < np; p += MT * STEP) {
        u4_t v[STEP];
        int s[STEP];
#pragma unroll
        for (int k = 0; k < STEP; k++) {
          const int x = p + k * MT + (int)threadIdx.x;
          s[k] = x < np ? from[x >> sh] : -1;
          if (a.in_place && s[k] == j0 + (x >> sh)) s[k] = -1;  // stays where it is
          if (s[k] >= 0) v[k] = src[(int64_t)s[k] * per + (x & (per - 1))];
        }
        if (a.in_place) __syncthreads();
#pragma unroll
        for (int k = 0; k < STEP; k++)
          if (s[k] >= 0) __builtin_nontemporal_store(v[k], &dst[((int64_t)j0 << sh) + p + k * MT + (int)threadIdx.x]);
        if (a.in_place) __syncthreads();
      }
    };
    move(a.payload, a.payload_out, a.pshift);
    if constexpr (KIVI) move(a.meta, a.meta_out, a.mshift);
    if (from[0] < 0) return;  // blocks behind the last kept one
  }
}

hipError_t evict_launch(const EvictArgs &a, hipStream_t s) {
  const int64_t heads = (int64_t)a.layers * a.batch * a.heads;
  const int64_t blocks = (a.tokens + a.block - 1) / a.block;
  const dim3 grid((unsigned)heads);
  if (blocks <= PT) hipLaunchKernelGGL(k_evict_pick<1>, grid, dim3(PT), 0, s, a);
  else if (blocks <= 4 * PT) hipLaunchKernelGGL(k_evict_pick<4>, grid, dim3(PT), 0, s, a);
  else if (blocks <= 16 * PT) hipLaunchKernelGGL(k_evict_pick<16>, grid, dim3(PT), 0, s, a);
  else hipLaunchKernelGGL(k_evict_select, grid, dim3(ST), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  int64_t chunks = 1;
  if (!a.in_place) {  // eight workgroups a compute unit, 16 KB at least to each
    const int64_t bytes = (int64_t)a.budget * 16 * ((1 << a.pshift) + (a.mshift < 0 ? 0 : 1 << a.mshift));
    chunks = (2048 + 2 * heads - 1) / (2 * heads);
    if (chunks > (bytes + 16383) / 16384) chunks = (bytes + 16383) / 16384;
    if (chunks > a.budget) chunks = a.budget;
  }
  const dim3 moves((unsigned)(2 * heads * chunks));
  if (a.mshift < 0) hipLaunchKernelGGL(k_evict_move<false>, moves, dim3(MT), 0, s, a, (int)chunks);
  else hipLaunchKernelGGL(k_evict_move<true>, moves, dim3(MT), 0, s, a, (int)chunks);
  return hipGetLastError();
}

}  // namespace cgs
