// cg_attend and its workspace: argument checks, the choice of splits, launches.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/codec_gauge.h"
#include "attend.hpp"
#include "cg_check.hpp"

namespace {

using cgh::error;

struct Plan {
  int64_t rows, tiles;
  int n;  // queries of a sequence that are taken at once
  int splits, waves, ragged, slots, least;
  bool merge;
  bool few;  // few row tiles: block sums come with the attention
  int64_t entries;
  size_t o_bytes, ml_bytes, dealt_bytes, bsum_bytes, lse2_bytes;
  size_t total() const { return o_bytes + ml_bytes + dealt_bytes + bsum_bytes + lse2_bytes; }
};

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Splits of the few-row form.  256 compute units hold `kResident` of its
// workgroups at once (three on each; two where block sums are gathered: more
// registers).  A round of them takes about 6 us for what does not depend on the
// tokens, plus each workgroup's tokens at its share of 5.5 TB/s, at best 12.5 ns a
// token; a merge takes about 4.5 us.  Of one split and the most that one, two,
// three or four rounds hold the fastest by that sum is taken, with at least 256
// tokens (two units a wave) to a workgroup.  80 KV heads of 3000 tokens: 9 splits
// (one round) 19 us, 10 splits 24; 200 heads of 4000 tokens: one split 55 us, 3
// splits and merge 49; 800 heads: 171 and 162; 300 heads of 8000 tokens: one split
// 121, 2 splits 130; 131072 tokens with sums by 512 workgroups 54 us, by 768 66.
constexpr int64_t kResident = 768, kResidentSums = 512, kMinTokens = 256;

int64_t few_splits(int64_t work, int64_t tokens, int64_t resident) {
  const int64_t most = (tokens + kMinTokens - 1) / kMinTokens;
  int64_t best = 1;
  double best_us = 0.0;
  for (int k = 0; k <= 4; k++) {
    int64_t sp = k ? k * resident / work : 1;
    if (sp > most) sp = most;
    if (sp > cga::MERGE_SPLITS) sp = cga::MERGE_SPLITS;
    if (sp < 1) sp = 1;
    // whole rounds, then what is left, at its share of the bandwidth
    const int64_t groups = work * sp, full = groups / resident, rest = groups % resident;
    const double each = (double)tokens / sp, whole = resident * 256.0 / 5.5e6;
    const double part = whole * rest / resident;
    const double us = full * (6.0 + each * (whole > 0.0125 ? whole : 0.0125)) +
                      (rest ? 6.0 + each * (part > 0.0125 ? part : 0.0125) : 0.0) + (sp > 1 ? 4.5 : 0.0);
    if (k == 0 || us < best_us) {
      best = sp;
      best_us = us;
    }
  }
  return best;
}

// Splits of 128-row tiles.  A workgroup takes 24 ns a token on a compute unit of
// its own and 36 beside another (512 at once), after about 6 us; a merge moves
// every split's sums twice (5 us and 4.5 TB/s).  8 KV heads x 4 query heads, whole
// calls: a prompt of 300 / 500 / 1000 tokens 18.7 / 23 / 35 us, in two splits 25 / 31 /
// 45, in four 32 / 38 / 60; 512 queries over 2048 and 8192 tokens: 56 and 183 us, in two
// splits 49 and 113, in four 49 and 100; 1024 over 8192: 186, in two 169, in four 181.
constexpr int64_t kTargetTiles = 512;

int64_t tile_splits(int64_t work, int64_t rows, int64_t tokens) {
  const int64_t most = (tokens + kMinTokens - 1) / kMinTokens;
  int64_t best = 1;
  double best_us = 0.0;
  for (int64_t sp = 1; sp == 1 || (sp <= most && work * sp <= kTargetTiles && sp <= cga::MERGE_SPLITS); sp *= 2) {
    const double each = (double)tokens / sp * (work * sp <= kTargetTiles / 2 ? 0.024 : 0.036);
    const double us = 6.0 + each + (sp > 1 ? 5.0 + (double)rows * sp * cga::D * 4 / 4.5e6 : 0.0);
    if (sp == 1 || us < best_us) {
      best = sp;
      best_us = us;
    }
  }
  return best;
}

// Block weights of many rows need 8 bytes a row and 32 tokens of the capacity.
// Where that would pass 1 GiB the queries are taken in turn, 128 rows a KV head
// at least (a full tile: fewer would leave waves without rows), so a large batch and
// capacity pass it all the same.
constexpr uint64_t kMaxSums = (uint64_t)1 << 30;

Plan make_plan(const cg_shape *s, const cg_codec *c, const cg_attn *t, bool mass) {
  Plan p{};
  const int64_t fields = (int64_t)s->batch * s->heads, ratio = t->q_heads / s->heads;
  const int64_t nblk = s->token_capacity / c->block_tokens;
  p.entries = c->block_tokens == 64 ? 2 * nblk : nblk;
  p.n = t->n_queries;
  if (mass && p.n * ratio > (int64_t)cga::FEW_TILES * cga::ROWS) {
    int64_t rows = p.entries ? (int64_t)(kMaxSums / 8) / (fields * p.entries) : p.n * ratio;
    if (rows < 128) rows = 128;
    const int64_t each = rows < ratio ? 1 : rows / ratio, turns = (p.n + each - 1) / each;
    p.n = (int)((p.n + turns - 1) / turns);
  }
  p.rows = p.n * ratio;
  p.tiles = (p.rows + cga::ROWS - 1) / cga::ROWS;
  // 8 KV heads x 4096 tokens with 32, 48 and 64 rows a head: one sequence 14, 17 and 17
  // us by row tiles of 16, 21, 22 and 23 by tiles of 128 (merges with them), 8
  // sequences 31, 37 and 45 against 40, 45 and 47
  p.few = p.tiles <= cga::FEW_TILES;
  const int64_t work = fields * (p.few ? p.tiles : (p.rows + 127) / 128);
  int64_t sp = 1;
  if (work > 0 && p.few) {
    sp = few_splits(work, s->tokens, mass ? kResidentSums : kResident);
  } else if (work > 0) {
    sp = tile_splits(work, fields * p.rows, s->tokens);
  }
  // Short histories: eight waves to a workgroup, one to a compute unit, in place
  // of splits and their merge.  8 KV heads x 4 query heads, one sequence of 512
  // tokens: 9.3 us, by four waves 10.0; of 1000 and 2048: 11.7 and 16.4, with
  // splits 12.2 and 12.5; 16 sequences of 2048: 19.2 and 20.4; 32 of 1024 and of
  // 2048: 16.4 and 29.1, by four waves 17.7 and 33.1; 40 of 1024, past one to a
  // unit: 25.7 and 21.0.
  p.waves = 4;
  if (p.few && work <= 256 && s->tokens > kMinTokens && s->tokens <= (work >= 128 ? 2048 : 1024)) {
    p.waves = 8;
    sp = 1;
  }
  p.splits = (int)sp;
  // Sequences of unlike lengths: splits dealt by length (see Slot), with one split
  // half as many more for the longest.  8 KV heads, 8 sequences of 0 .. 16384 tokens
  // with sums 31 us, equal splits 37; 16 of 0 .. 8192 23 and 26 (all of 8192: 53 and 51);
  // 32 sequences of 2000 tokens but one of 131072: the whole call 72 and 428; 64 of
  // 16000 in one split each, with a merge that finds nothing to do: 390 and 389.
  // (The workspace is the same with and without lengths.)
  const bool may = p.few && p.waves == 4 && s->batch > 1 && s->batch <= 64 &&
                   s->tokens > (p.splits > 1 ? 2048 : 16384) && s->tokens < (int64_t)1 << 30;
  p.ragged = may && t->lengths;
  const int64_t more = may && p.splits == 1 ? s->batch / 2 : 0, slots = (int64_t)s->batch * p.splits;
  p.slots = (int)(slots + (p.ragged ? more : 0));
  p.least = (int)((s->tokens + cga::UNIT - 1) / cga::UNIT / cga::MERGE_SPLITS + 1);
  if (p.least < kMinTokens / cga::UNIT) p.least = kMinTokens / cga::UNIT;
  const int64_t parts = (slots + more) * s->heads * p.rows;
  p.merge = p.splits > 1 || p.ragged;
  p.o_bytes = p.merge || may ? up256((size_t)parts * cga::D * 4) : 0;
  p.ml_bytes = p.merge || may || (mass && p.few) ? up256((size_t)parts * 8) : 0;
  if (may) p.dealt_bytes = up256((size_t)s->batch * 8);
  if (mass) p.bsum_bytes = up256((size_t)(fields * p.entries * p.rows) * 8);
  if (mass && !p.few) p.lse2_bytes = up256((size_t)(fields * p.rows) * 4);
  return p;
}

// factor of the scores, which are powers of two
float log2_scale(const cg_attn *t) { return (float)((double)t->scale * 1.4426950408889634074); }

int check_attn(const cg_shape *s, const cg_attn *t) {
  if (!t) return error(CG_E_INVAL, "attn is NULL");
  if (t->layer < 0 || t->layer >= s->layers) return error(CG_E_SHAPE, "layer outside the cache shape");
  if (t->q_heads <= 0 || t->q_heads % s->heads) return error(CG_E_SHAPE, "q_heads must be a positive multiple of heads");
  if (t->n_queries < 0) return error(CG_E_SHAPE, "n_queries < 0");
  if (t->causal != 0 && t->causal != 1) return error(CG_E_INVAL, "causal must be 0 or 1");
  if (!isfinite(t->scale) || !isfinite(log2_scale(t))) return error(CG_E_INVAL, "scale or scale log2(e) is not finite");
  if (((uintptr_t)t->lengths | (uintptr_t)t->starts) & 3u)
    return error(CG_E_INVAL, "lengths and starts must be 4-byte aligned");
  const int64_t token = (int64_t)t->q_heads * s->head_dim;
  const int64_t ts = t->q_token_stride ? t->q_token_stride : token;
  const int64_t bs = t->q_batch_stride ? t->q_batch_stride : token * t->n_queries;
  const int64_t unit = s->dtype == CG_DTYPE_BF16 ? 8 : 4, far = (int64_t)1 << 40;
  if (ts < 0 || bs < 0 || ts % unit || bs % unit || ts > far || bs > far)
    return error(CG_E_INVAL, "query strides must be multiples of 16 bytes and not negative");
  // bounds of the launches and of the workspace's sizes
  const int64_t rows = (int64_t)t->n_queries * (t->q_heads / s->heads);
  if (rows > (int64_t)1 << 26 || (int64_t)s->batch * s->heads > (int64_t)1 << 22 ||
      (rows + 15) / 16 * s->batch * s->heads > (int64_t)1 << 27)
    return error(CG_E_SHAPE, "too many query rows");
  if ((int64_t)s->batch * s->heads * ((s->token_capacity + 15) / 16) >= (int64_t)1 << 31)
    return error(CG_E_SHAPE, "too many tokens for one launch");
  return CG_OK;
}

}  // namespace

extern "C" {

int cg_attend_workspace_bytes(const cg_shape *shape, const cg_gauge *gauge, const cg_codec *codec,
                              const cg_attn *attn, int32_t with_mass, size_t *bytes) {
  cgh::set_error("");
  if (!bytes) return error(CG_E_INVAL, "bytes is NULL");
  if (!gauge) return error(CG_E_INVAL, "gauge is NULL");
  alignas(16) static const char any[16] = {};
  int rc = cgh::check_cache8(shape, gauge, codec, any, UINT64_MAX, any, UINT64_MAX);
  if (rc) return rc;
  if ((rc = check_attn(shape, attn))) return rc;
  *bytes = make_plan(shape, codec, attn, with_mass != 0).total();
  return CG_OK;
}

int cg_attend(const cg_shape *shape, const void *payload, uint64_t payload_cap, const void *meta,
              uint64_t meta_cap, const cg_gauge *gauge, const cg_codec *codec, const cg_attn *attn,
              const void *q, void *out, float *lse, float *mass, void *workspace, size_t ws_bytes,
              void *stream) {
  cgh::set_error("");
  if (!gauge) return error(CG_E_INVAL, "gauge is NULL");
  int rc = cgh::check_cache8(shape, gauge, codec, payload, payload_cap, meta, meta_cap);
  if (rc) return rc;
  if ((rc = check_attn(shape, attn))) return rc;
  if (attn->n_queries == 0) return CG_OK;
  if (!q || !out) return error(CG_E_INVAL, "q or out is NULL");
  if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15u)
    return error(CG_E_INVAL, "q, out and workspace must be 16-byte aligned");
  if (((uintptr_t)lse | (uintptr_t)mass) & 3u) return error(CG_E_INVAL, "lse and mass must be 4-byte aligned");
  const int64_t esz = shape->dtype == CG_DTYPE_BF16 ? 2 : 4;
  const int64_t token = (int64_t)attn->q_heads * shape->head_dim;
  const int64_t ts = attn->q_token_stride ? attn->q_token_stride : token;
  const int64_t bs = attn->q_batch_stride ? attn->q_batch_stride : token * attn->n_queries;
  const char *q0 = (const char *)q, *o0 = (const char *)out;
  const int64_t qb = (int64_t)cgh::reach(shape->batch, bs, attn->n_queries, ts, token) * esz;
  if (!qb) return error(CG_E_INVAL, "query strides reach too far");
  const int64_t ob = (int64_t)shape->batch * attn->n_queries * token * esz;
  if (q0 < o0 + ob && o0 < q0 + qb) return error(CG_E_INVAL, "q and out overlap");
  const Plan p = make_plan(shape, codec, attn, mass != nullptr);
  if (p.total() && (!workspace || ws_bytes < p.total()))
    return error(CG_E_SIZE, "workspace missing or smaller than cg_attend_workspace_bytes");

  cga::AttendArgs a{};
  const int64_t fields = (int64_t)shape->batch * shape->heads, d = shape->head_dim;
  const int64_t kf = (int64_t)attn->layer * 2 * fields, vf = kf + fields;
  a.tcap = shape->token_capacity;
  a.tokens = shape->tokens;
  a.nblk = a.tcap / codec->block_tokens;
  a.kpay = (const uint8_t *)payload + kf * a.tcap * d;
  a.vpay = (const uint8_t *)payload + vf * a.tcap * d;
  a.kmeta = (const float2 *)meta + kf * a.nblk;
  a.vmeta = (const float2 *)meta + vf * a.nblk;
  a.lengths = attn->lengths;
  a.starts = attn->starts;
  a.g = gauge->group;
  a.gk = gauge->group ? gauge->G + (int64_t)attn->layer * 2 * shape->heads * d * gauge->group : nullptr;
  a.gv = gauge->group ? a.gk + (int64_t)shape->heads * d * gauge->group : nullptr;
  a.mass = mass ? mass + (int64_t)attn->layer * fields * a.nblk : nullptr;
  a.q_bs = bs;
  a.q_ts = ts;
  a.batch = shape->batch;
  a.heads = shape->heads;
  a.ratio = attn->q_heads / shape->heads;
  a.n_all = attn->n_queries;
  a.bshift = codec->block_tokens == 16 ? 4 : codec->block_tokens == 32 ? 5 : 6;
  a.causal = attn->causal;
  a.splits = p.splits;
  a.few = p.few;
  a.ragged = p.ragged;
  a.slots = p.slots;
  a.least = p.least;
  a.waves = p.waves;
  a.entries = p.entries;
  a.c = log2_scale(attn);
  char *w = (char *)workspace;
  auto take = [&w](size_t n) { char *r = n ? w : nullptr; w += n; return r; };
  a.part_o = (float *)take(p.o_bytes);
  a.part_ml = (float2 *)take(p.ml_bytes);
  a.dealt = (int2 *)take(p.dealt_bytes);
  a.bsum = (float2 *)take(p.bsum_bytes);
  a.lse2 = (float *)take(p.lse2_bytes);

  const bool bf16 = shape->dtype == CG_DTYPE_BF16;
  hipStream_t st = (hipStream_t)stream;
  for (int32_t first = 0; first < attn->n_queries; first += p.n) {
    a.first = first;
    a.n = attn->n_queries - first < p.n ? attn->n_queries - first : p.n;
    a.rows = a.n * a.ratio;
    a.tiles = (a.rows + cga::ROWS - 1) / cga::ROWS;
    a.q = (const char *)q + (int64_t)first * ts * esz;
    a.out = (char *)out + (int64_t)first * token * esz;
    a.lse = lse ? lse + (int64_t)first * attn->q_heads : nullptr;
    hipError_t e = p.few ? cga::rows_launch(a, bf16, st) : cga::tile_launch(a, bf16, st);
    if (e != hipSuccess) return cgh::hip_error(e, "cg_attend launch");
    if (p.merge && (e = cga::merge_launch(a, bf16, st)) != hipSuccess)
      return cgh::hip_error(e, "cg_attend merge launch");
    if (mass && shape->tokens > 0) {
      // the merge of few rows has finished the weights
      e = !p.few ? cga::mass_rows_launch(a, st) : p.merge ? hipSuccess : cga::mass_finish_launch(a, st);
      if (e != hipSuccess) return cgh::hip_error(e, "cg_attend mass launch");
    }
  }
  return CG_OK;
}

}  // extern "C"
