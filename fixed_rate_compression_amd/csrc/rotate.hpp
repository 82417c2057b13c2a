// Norm and rotation of query and key heads: launch interface.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cgr {

struct Rows {
  const void *in;  // [batch][n][heads][128], heads contiguous
  void *out;
  int64_t ibs, irs, obs, ors;  // elements between sequences and rows
  const float *weight;         // [128] or null: no norm
  int32_t heads;               // 0: nothing to do
};

struct RotateArgs {
  Rows r[2];  // queries, keys
  const float *freq;           // [dim / 2]
  const int32_t *positions;    // [axes][batch][n] or null
  const int32_t *lengths, *starts;
  int64_t tokens;
  int32_t batch, n, dim, axes, interleaved, dealt;
  int32_t sections[4];
  float eps, magnitude;
};
hipError_t rotate_launch(const RotateArgs &a, bool bf16, hipStream_t s);

}  // namespace cgr
