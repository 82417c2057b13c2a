// Host-side checks and error reporting shared by the entry points of the
// serving operators (defined in codec_gauge_api.cpp).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

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
// whether rows of wa elements, laid out so that rows of one of the widths lie apart, and rows of wb elements laid out
// alike d elements further on share memory.  Two rows' distance is d + x so + y si, x below the larger stride's
// count and y below the smaller's; few x bring them near one another.
inline bool rows_meet(int64_t batch, int64_t bs, int64_t n, int64_t rs, int64_t d, int64_t wa, int64_t wb) {
  const bool by_row = batch == 1 || (n > 1 && rs > bs);  // the larger stride is that of the rows
  const int64_t co = by_row ? n : batch, so = by_row ? rs : bs, ci = by_row ? batch : n, si = by_row ? bs : rs;
  const int64_t all = ci > 1 ? (ci - 1) * si : 0;
  const auto down = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
  // y with -wb < e + y s < wa, |y| < count
  const auto first = [&](int64_t e, int64_t w, int64_t s, int64_t count) { return std::max(1 - count, down(-w - e, s) + 1); };
  const auto last = [&](int64_t e, int64_t w, int64_t s, int64_t count) { return std::min(count - 1, down(w - e - 1, s)); };
  for (int64_t x = co > 1 ? first(d, wb + all, so, co) : 0; x <= (co > 1 ? last(d, wa + all, so, co) : 0); x++) {
    const int64_t e = d + (co > 1 ? x * so : 0);
    if (ci > 1 ? first(e, wb, si, ci) <= last(e, wa, si, ci) : e > -wb && e < wa) return true;
  }
  return false;
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
