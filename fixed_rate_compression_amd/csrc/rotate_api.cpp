// cg_rotate: argument checks and launch.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/codec_gauge.h"
#include "cg_check.hpp"
#include "rotate.hpp"

using cgh::error;

namespace {

struct Span {
  const char *at;
  uint64_t bytes;
  int64_t bs, rs;
};

// whether rows of the two (wa and wb elements) may share memory; parts of the same rows, side by side, do not
bool clash(const cg_shape *s, int32_t n, const Span &a, int64_t wa, const Span &b, int64_t wb, int64_t esz) {
  if (a.at >= b.at + b.bytes || b.at >= a.at + a.bytes) return false;
  if (a.rs != b.rs || a.bs != b.bs) return true;
  return cgh::rows_meet(s->batch, a.bs, n, a.rs, (b.at - a.at) / esz, wa, wb);
}

// rows of `heads` heads; 0 strides: dense
int span_of(const cg_rows *r, const cg_shape *s, int32_t n, int32_t heads, bool written, Span *o) {
  const int64_t row = (int64_t)heads * s->head_dim, unit = s->dtype == CG_DTYPE_BF16 ? 8 : 4, far = (int64_t)1 << 40;
  if (!r->data) return error(CG_E_INVAL, "rows are NULL");
  if ((uintptr_t)r->data & 15u) return error(CG_E_INVAL, "rows must be 16-byte aligned");
  o->at = (const char *)r->data;
  o->rs = r->row_stride ? r->row_stride : row;
  o->bs = r->batch_stride ? r->batch_stride : row * n;
  if (o->rs < 0 || o->bs < 0 || o->rs % unit || o->bs % unit || o->rs > far || o->bs > far)
    return error(CG_E_INVAL, "row strides must be multiples of 16 bytes and not negative");
  o->bytes = cgh::reach(s->batch, o->bs, n, o->rs, row) * (s->dtype == CG_DTYPE_BF16 ? 2 : 4);
  if (!o->bytes) return error(CG_E_INVAL, "row strides reach too far");
  // one row a sequence: the sequences are the rows; one sequence: it has no next
  if (n == 1 && s->batch > 1) o->rs = o->bs;
  if (s->batch == 1) o->bs = o->rs * n;
  if (written && !cgh::rows_apart(s->batch, o->bs, n, o->rs, row)) return error(CG_E_INVAL, "rows of an output overlap");
  return CG_OK;
}

}  // namespace

extern "C" int cg_rotate(const cg_shape *shape, const cg_rotary *rotary, int32_t q_heads, int32_t n,
                         const int32_t *positions, const int32_t *lengths, const int32_t *starts, const cg_rows *q,
                         const cg_rows *k, const cg_rows *q_out, const cg_rows *k_out, void *stream) {
  cgh::set_error("");
  int rc = cgh::check_shape_of(shape);
  if (rc) return rc;
  if (!rotary) return error(CG_E_INVAL, "rotary is NULL");
  const cg_rotary &t = *rotary;
  if (t.dim < 0 || t.dim > shape->head_dim || t.dim % 16)
    return error(CG_E_UNSUPPORTED, "dim must be a multiple of 16, head_dim at most");
  if (t.axes < 1 || t.axes > 4) return error(CG_E_SHAPE, "axes must be 1 to 4");
  if ((t.interleaved != 0 && t.interleaved != 1) || (t.dealt != 0 && t.dealt != 1))
    return error(CG_E_INVAL, "interleaved and dealt must be 0 or 1");
  if (t.axes > 1) {
    int64_t pairs = 0;
    for (int i = 0; i < t.axes; i++) {
      if (t.sections[i] < 0) return error(CG_E_SHAPE, "sections must not be negative");
      pairs += t.sections[i];
      if (i && t.dealt && (int64_t)t.axes * t.sections[i] > t.dim / 2 + t.axes - 1 - i)
        return error(CG_E_SHAPE, "an axis is dealt more pairs than come to it");
    }
    if (pairs != t.dim / 2) return error(CG_E_SHAPE, "the sections must have dim / 2 pairs in all");
    if (!positions) return error(CG_E_INVAL, "several axes need positions");
  }
  if (t.dim && !t.freq) return error(CG_E_INVAL, "freq is NULL");
  if (!(t.eps >= 0.0f) || !isfinite(t.eps) || !isfinite(t.magnitude))
    return error(CG_E_INVAL, "eps must be finite and not negative, magnitude finite");
  if (((uintptr_t)t.freq | (uintptr_t)positions | (uintptr_t)lengths | (uintptr_t)starts) & 3u)
    return error(CG_E_INVAL, "freq, positions, lengths and starts must be 4-byte aligned");
  if (((uintptr_t)t.q_weight | (uintptr_t)t.k_weight) & 15u)
    return error(CG_E_INVAL, "norm weights must be 16-byte aligned");
  if (n < 0) return error(CG_E_SHAPE, "n < 0");
  if (!q != !q_out || !k != !k_out || (!q && !k)) return error(CG_E_INVAL, "queries or keys, each with its output, are needed");
  if (q && (q_heads <= 0 || q_heads > (1 << 20))) return error(CG_E_SHAPE, "q_heads must be 1 to 2^20");
  if (n == 0) return CG_OK;
  const int64_t heads = (q ? q_heads : 0) + (k ? (int64_t)shape->heads : 0);
  if (heads > (1 << 21) || (int64_t)shape->batch * n * heads >= (int64_t)1 << 31)
    return error(CG_E_SHAPE, "too many rows for one launch");

  cgr::RotateArgs a{};
  const cg_rows *in[2] = {q, k}, *out[2] = {q_out, k_out};
  const int32_t hs[2] = {q ? q_heads : 0, k ? shape->heads : 0};
  Span si[2] = {}, so[2] = {};
  bool inplace[2] = {};
  for (int x = 0; x < 2; x++) {
    if (!in[x]) continue;
    if ((rc = span_of(in[x], shape, n, hs[x], false, &si[x]))) return rc;
    if ((rc = span_of(out[x], shape, n, hs[x], true, &so[x]))) return rc;
    inplace[x] = si[x].at == so[x].at;
    if (inplace[x] && (si[x].rs != so[x].rs || si[x].bs != so[x].bs)) return error(CG_E_INVAL, "in place: the strides must be the same");
  }
  // rows are written where others are read only in place
  const int64_t esz = shape->dtype == CG_DTYPE_BF16 ? 2 : 4;
  const int64_t w[2] = {(int64_t)hs[0] * shape->head_dim, (int64_t)hs[1] * shape->head_dim};
  for (int x = 0; x < 2; x++)
    for (int y = 0; y < 2; y++)
      if (in[x] && in[y] && (x != y || !inplace[x]) && clash(shape, n, so[x], w[x], si[y], w[y], esz))
        return error(CG_E_INVAL, "an output overlaps an input");
  if (q && k && clash(shape, n, so[0], w[0], so[1], w[1], esz)) return error(CG_E_INVAL, "the outputs overlap");
  for (int x = 0; x < 2; x++) {
    if (!in[x]) continue;
    a.r[x] = cgr::Rows{si[x].at, (void *)so[x].at, si[x].bs, si[x].rs, so[x].bs, so[x].rs, x ? t.k_weight : t.q_weight, hs[x]};
  }
  a.freq = t.freq;
  a.positions = positions;
  a.lengths = lengths;
  a.starts = starts;
  a.tokens = shape->tokens;
  a.batch = shape->batch;
  a.n = n;
  a.dim = t.dim;
  a.axes = t.axes;
  a.interleaved = t.interleaved;
  a.dealt = t.dealt;
  for (int i = 0; i < 4; i++) a.sections[i] = t.sections[i];
  a.eps = t.eps;
  a.magnitude = t.magnitude;
  const hipError_t e = cgr::rotate_launch(a, shape->dtype == CG_DTYPE_BF16, (hipStream_t)stream);
  return e == hipSuccess ? CG_OK : cgh::hip_error(e, "cg_rotate launch");
}
