// Appending to, reading from and evicting from the serving caches (8-bit
// block-uniform, 4-bit KIVI-style): launch interface.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cgs {

struct AppendArgs {
  uint8_t *payload;        // the layer's fields, (kind, b, h) at ((kind batch + b) heads + h) tcap 128 (4 bits: 64)
  float *meta;             // the layer's (minimum, step) pairs, nblk a field (4 bits: 4 tcap)
  void *tail;              // the layer's raw rows [kind][b][h][block][128]
  const void *k, *v;       // new rows [b][n][h][128], storage format
  int64_t batch_stride, row_stride;  // of k and v (elements)
  const int32_t *lengths, *starts;
  const float *gauges;     // the layer's [kind][heads][128 g]
  int64_t tcap, tokens, nblk;
  int32_t batch, heads, n, block, bshift, tiles;  // tiles: 64-row strips of a sequence at most
};
hipError_t append_launch(const AppendArgs &a, bool bf16, int g, bool kivi, hipStream_t s);

struct ReadArgs {
  const uint8_t *payload;  // as above
  const float2 *meta;
  void *k, *v;             // rows [b][n][h][128], storage format, or null
  int64_t batch_stride, row_stride;  // of k and v (elements)
  const int32_t *lengths, *starts;
  const float *gauges;     // the layer's [kind][heads][128 g]
  int64_t tcap, tokens, nblk;
  int32_t batch, heads, n, bshift, tiles;  // tiles: 64-row strips of the rows
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
