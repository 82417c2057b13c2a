// Host-side checks and error reporting shared by the entry points of the 8-bit
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
// a K/V cache in 8-bit block-uniform form with its buffers (gauge may be NULL:
// not looked at)
int check_cache8(const cg_shape *s, const cg_gauge *g, const cg_codec *c, const void *payload,
                 uint64_t payload_cap, const void *meta, uint64_t meta_cap);

}  // namespace cgh
