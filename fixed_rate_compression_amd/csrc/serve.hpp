// Appending to, reading from and evicting from the serving caches (8-bit
// block-uniform, 4-bit KIVI-style): launch interface.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cgs {

// x / d for x below 2^31: two scalar instructions, where a division takes some thirty
struct Div {
  uint32_t mul = 0, shift = 0;
  Div() = default;
  explicit Div(uint32_t d) {  // 2^(shift - 1) < d <= 2^shift
    while (shift < 31 && (uint32_t)1 << shift < d) shift++;
    mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - d)) / d + 1);
  }
  __host__ __device__ uint32_t operator()(uint32_t x) const {
    return ((uint32_t)(((uint64_t)x * mul) >> 32) + x) >> shift;
  }
};

struct AppendArgs {
  uint8_t *payload;        // the layer's fields, (kind, b, h) at ((kind batch + b) heads + h) tcap 128 (4 bits: 64)
  float *meta;             // the layer's (minimum, step) pairs, nblk a field (4 bits: 4 tcap)
  void *tail;              // the layer's raw rows [kind][b][h][block][128]
  const void *k, *v;       // new rows [b][n][h][128], storage format
  int64_t batch_stride, row_stride;  // of k and v (elements)
  const int32_t *lengths, *starts;
  const float *gauges;     // the layer's [kind][heads][128 g]
  int64_t tcap, tokens, nblk;
  int32_t batch, heads, n, block, bshift, tiles;  // tiles: 64-row (4 bits: 32-row) strips of a sequence at most
  Div by_tiles, by_heads;
};
hipError_t append_launch(const AppendArgs &a, bool bf16, int g, hipStream_t s);
hipError_t append4_launch(const AppendArgs &a, bool bf16, int g, hipStream_t s);

struct ReadArgs {
  const uint8_t *payload;  // as above
  const float2 *meta;
  void *k, *v;             // rows [b][n][h][128], storage format, or null
  int64_t batch_stride, row_stride;  // of k and v (elements)
  const int32_t *lengths, *starts;
  const float *gauges;     // the layer's [kind][heads][128 g]
  int64_t tcap, tokens, nblk;
  int32_t batch, heads, n, bshift, tiles;  // tiles: 64-row strips of the rows
  Div by_tiles, by_heads;
};
hipError_t read_launch(const ReadArgs &a, bool bf16, int g, bool kivi, hipStream_t s);

struct EvictArgs {
  const uint8_t *payload;
  const float2 *meta;
  const float *mass;       // [layers][b][h][nblk]
  const int32_t *lengths;  // or null (tokens)
  uint8_t *payload_out;
  float2 *meta_out;
  float *mass_out;         // [layers][b][h][nblk_out]
  int32_t *kept;           // [layers][b][h][budget]
  int32_t *lengths_out;
  int64_t tokens, nblk, nblk_out;
  int32_t layers, batch, heads, block, budget, sink, recent;
  int32_t in_place;
  int32_t pshift;          // log2 of a block's 16-byte pieces of codes
  int32_t mshift;          // 4 bits: of ranges; 8 bits: -1, one range a block
};
hipError_t evict_launch(const EvictArgs &a, hipStream_t s);

}  // namespace cgs
