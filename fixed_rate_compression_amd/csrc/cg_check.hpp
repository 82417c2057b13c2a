// Host-side checks and error reporting shared by the entry points of the
// serving operators (defined in codec_gauge_api.cpp).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/codec_gauge.h"

namespace cgh {

void set_error(const char *msg);
int error(int code, const char *msg);                // records msg, returns code
int hip_error(hipError_t e, const char *what);       // CG_E_HIP with HIP's message
// elements from the first to behind the last of `batch` x `n` rows of `row` elements
// that lie bs and rs apart; 0 if they reach past 2^60
inline uint64_t reach(int64_t batch, int64_t bs, int64_t n, int64_t rs, int64_t row) {
  const unsigned __int128 e = (unsigned __int128)(batch - 1) * bs + (unsigned __int128)(n - 1) * rs + row;
  return e >> 60 ? 0 : (uint64_t)e;
}
// whether rows of w elements at b bs + i rs (b < batch, i < n; strides that reach() takes) lie apart: the smaller stride
// passes a row, the larger one all rows of the smaller.  The stride of a single row or sequence is not looked at.
inline bool rows_apart(int64_t batch, int64_t bs, int64_t n, int64_t rs, int64_t w) {
  if (batch == 1 || n == 1) return (n == 1 || rs >= w) && (batch == 1 || bs >= w);
  return (rs >= w && bs >= rs * (n - 1) + w) || (bs >= w && rs >= bs * (batch - 1) + w);
}
int check_shape_of(const cg_shape *s);
// a K/V cache in 8-bit block-uniform or 4-bit KIVI-style form with its buffers (gauge
// may be NULL: not looked at)
int check_cache(const cg_shape *s, const cg_gauge *g, const cg_codec *c, const void *payload,
                 uint64_t payload_cap, const void *meta, uint64_t meta_cap);

inline bool is_kivi4(const cg_codec *c) { return c->backend == CG_BACKEND_KIVI; }  // of a cache that passed
// bytes of a field of tcap rows: codes, (minimum, step) pairs
inline int64_t payload_field(const cg_codec *c, int64_t tcap) { return is_kivi4(c) ? tcap * 64 : tcap * 128; }
inline int64_t meta_field(const cg_codec *c, int64_t tcap) { return is_kivi4(c) ? tcap * 32 : tcap / c->block_tokens * 8; }

}  // namespace cgh
