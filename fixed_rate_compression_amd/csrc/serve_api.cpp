// cg_append and cg_evict: argument checks and launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/codec_gauge.h"
#include "cg_check.hpp"
#include "serve.hpp"

using cgh::error;

namespace {

bool overlap(const void *a, uint64_t na, const void *b, uint64_t nb) {
  return (const char *)a < (const char *)b + nb && (const char *)b < (const char *)a + na;
}

}  // namespace

extern "C" {

int cg_append(const cg_shape *shape, const cg_gauge *gauge, const cg_codec *codec, int32_t layer,
              int32_t n_new, const void *k_new, const void *v_new, int64_t batch_stride,
              int64_t row_stride, const int32_t *lengths, const int32_t *starts, void *tail,
              void *payload, uint64_t payload_cap, void *meta, uint64_t meta_cap, void *stream) {
  cgh::set_error("");
  if (!gauge) return error(CG_E_INVAL, "gauge is NULL");
  int rc = cgh::check_cache8(shape, gauge, codec, payload, payload_cap, meta, meta_cap);
  if (rc) return rc;
  if (layer < 0 || layer >= shape->layers) return error(CG_E_SHAPE, "layer outside the cache shape");
  if (n_new < 0) return error(CG_E_SHAPE, "n_new < 0");
  if (n_new == 0) return CG_OK;
  if (!k_new || !v_new || !tail) return error(CG_E_INVAL, "k_new, v_new or tail is NULL");
  if (((uintptr_t)k_new | (uintptr_t)v_new | (uintptr_t)tail) & 15u)
    return error(CG_E_INVAL, "k_new, v_new and tail must be 16-byte aligned");
  if (((uintptr_t)lengths | (uintptr_t)starts) & 3u)
    return error(CG_E_INVAL, "lengths and starts must be 4-byte aligned");
  const int64_t row = (int64_t)shape->heads * shape->head_dim;
  const int64_t rs = row_stride ? row_stride : row, bs = batch_stride ? batch_stride : row * n_new;
  const int64_t unit = shape->dtype == CG_DTYPE_BF16 ? 8 : 4, far = (int64_t)1 << 40;
  if (rs < 0 || bs < 0 || rs % unit || bs % unit || rs > far || bs > far)
    return error(CG_E_INVAL, "row strides must be multiples of 16 bytes and not negative");
  cgs::AppendArgs a{};
  const int64_t fields = (int64_t)2 * shape->batch * shape->heads, f0 = layer * fields;
  // strips of 64 rows from the block of the first new row on
  const int64_t tiles = ((int64_t)n_new + codec->block_tokens - 1 + 63) / 64;
  if (fields * tiles >= (int64_t)1 << 31) return error(CG_E_SHAPE, "too many rows for one launch");
  const uint64_t esz = shape->dtype == CG_DTYPE_BF16 ? 2 : 4;
  const uint64_t in = cgh::reach(shape->batch, bs, n_new, rs, row) * esz;
  if (!in) return error(CG_E_INVAL, "row strides reach too far");
  const uint64_t tb = (uint64_t)fields * codec->block_tokens * shape->head_dim * esz;
  char *t0 = (char *)tail + (uint64_t)layer * tb;
  if (overlap(k_new, in, t0, tb) || overlap(v_new, in, t0, tb))
    return error(CG_E_INVAL, "new rows and tail overlap");
  a.tcap = shape->token_capacity;
  a.tokens = shape->tokens;
  a.nblk = a.tcap / codec->block_tokens;
  a.payload = (uint8_t *)payload + f0 * a.tcap * shape->head_dim;
  a.meta = (float *)meta + 2 * f0 * a.nblk;
  a.tail = t0;
  a.k = k_new;
  a.v = v_new;
  a.batch_stride = bs;
  a.row_stride = rs;
  a.lengths = lengths;
  a.starts = starts;
  a.gauges = gauge->group ? gauge->G + (int64_t)layer * 2 * shape->heads * shape->head_dim * gauge->group : nullptr;
  a.batch = shape->batch;
  a.heads = shape->heads;
  a.n = n_new;
  a.block = codec->block_tokens;
  a.bshift = a.block == 16 ? 4 : a.block == 32 ? 5 : 6;
  a.tiles = (int32_t)tiles;
  hipError_t e = cgs::append_launch(a, shape->dtype == CG_DTYPE_BF16, gauge->group, (hipStream_t)stream);
  return e == hipSuccess ? CG_OK : cgh::hip_error(e, "cg_append launch");
}

int cg_evict(const cg_shape *shape, const cg_codec *codec, int32_t budget, int32_t sink, int32_t recent,
             const float *mass, const void *payload, uint64_t payload_cap, const void *meta,
             uint64_t meta_cap, const int32_t *lengths, const cg_shape *out_shape, void *payload_out,
             uint64_t payload_out_cap, void *meta_out, uint64_t meta_out_cap, float *mass_out,
             int32_t *kept, int32_t *lengths_out, void *stream) {
  cgh::set_error("");
  int rc = cgh::check_cache8(shape, nullptr, codec, payload, payload_cap, meta, meta_cap);
  if (rc) return rc;
  if ((rc = cgh::check_cache8(out_shape, nullptr, codec, payload_out, payload_out_cap, meta_out, meta_out_cap)))
    return rc;
  if (out_shape->layers != shape->layers || out_shape->batch != shape->batch || out_shape->heads != shape->heads)
    return error(CG_E_SHAPE, "the caches differ in layers, batch or heads");
  if (sink < 0 || recent < 1 || (int64_t)sink + recent > budget)
    return error(CG_E_SHAPE, "need sink >= 0, recent >= 1 and sink + recent <= budget");
  const int64_t nblk = shape->token_capacity / codec->block_tokens, nout = out_shape->token_capacity / codec->block_tokens;
  if (budget > nout) return error(CG_E_SHAPE, "the output cache holds fewer blocks than the budget");
  if (!mass || !mass_out || !kept || !lengths_out) return error(CG_E_INVAL, "mass, mass_out, kept or lengths_out is NULL");
  if (((uintptr_t)mass | (uintptr_t)mass_out | (uintptr_t)kept | (uintptr_t)lengths | (uintptr_t)lengths_out) & 3u)
    return error(CG_E_INVAL, "mass, kept and lengths must be 4-byte aligned");
  const int64_t heads = (int64_t)shape->layers * shape->batch * shape->heads;
  if (2 * heads * (int64_t)1024 >= (int64_t)1 << 31) return error(CG_E_SHAPE, "too many heads for one launch");
  const uint64_t pb = (uint64_t)2 * heads * shape->token_capacity * shape->head_dim, mb = (uint64_t)2 * heads * nblk * 8;
  const uint64_t po = (uint64_t)2 * heads * out_shape->token_capacity * shape->head_dim, mo = (uint64_t)2 * heads * nout * 8;
  const uint64_t wb = (uint64_t)heads * nblk * 4, wo = (uint64_t)heads * nout * 4;
  const bool in_place = payload_out == payload;
  if (in_place) {
    if (meta_out != meta || nout != nblk || mass_out != mass)
      return error(CG_E_INVAL, "in place: payload, meta, mass and the capacity must all be the same");
  } else if (overlap(payload, pb, payload_out, po) || overlap(meta, mb, meta_out, mo) || overlap(mass, wb, mass_out, wo)) {
    return error(CG_E_INVAL, "the caches overlap");
  }
  if (lengths != lengths_out && lengths && overlap(lengths, 4u * shape->batch, lengths_out, 4u * shape->batch))
    return error(CG_E_INVAL, "lengths and lengths_out overlap in part");
  cgs::EvictArgs a{};
  a.payload = (const uint8_t *)payload;
  a.meta = (const float2 *)meta;
  a.mass = mass;
  a.lengths = lengths;
  a.payload_out = (uint8_t *)payload_out;
  a.meta_out = (float2 *)meta_out;
  a.mass_out = mass_out;
  a.kept = kept;
  a.lengths_out = lengths_out;
  a.tokens = shape->tokens;
  a.nblk = nblk;
  a.nblk_out = nout;
  a.layers = shape->layers;
  a.batch = shape->batch;
  a.heads = shape->heads;
  a.block = codec->block_tokens;
  a.budget = budget;
  a.sink = sink;
  a.recent = recent;
  a.in_place = in_place ? 1 : 0;
  a.pshift = codec->block_tokens == 16 ? 7 : codec->block_tokens == 32 ? 8 : 9;
  hipError_t e = cgs::evict_launch(a, (hipStream_t)stream);
  return e == hipSuccess ? CG_OK : cgh::hip_error(e, "cg_evict launch");
}

}  // extern "C"
