// C-ABI entry points of the token operators: argument validation, workspace
// layout and launches. Declared (with their contracts) in include/gs.h.
#include <math.h>

#include "tokens_common.h"

hipError_t gs_launch_dropout(DropK p, int dtype, hipStream_t st);
hipError_t gs_launch_qk_fwd(const QkK &p, int dtype, hipStream_t st);
hipError_t gs_launch_qk_bwd(const QkK &p, int dtype, hipStream_t st);
int gs_qk_bwd_blocks(int64_t batch, int64_t tokens, int q_heads, int k_heads, int lanes);
void gs_attn_plan(AttnK *p);
void gs_attn_bwd_plan(AttnK *p, bool masked);
hipError_t gs_launch_attn_fwd(AttnK p, int dtype, hipStream_t st);
hipError_t gs_launch_attn_bwd(AttnK p, int dtype, hipStream_t st);

namespace {

constexpr int64_t LIMIT = (int64_t)1 << 30;     // tokens, heads, batch entries
constexpr int64_t THREADS = (int64_t)1 << 32;   // of a launch, never so many
constexpr int64_t TOKEN_STRIDE = (int64_t)1 << 23;  // 64 rows within 32-bit byte offsets

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }
int32_t hip_status(hipError_t e) { return e == hipSuccess ? GS_OK : GS_ERR_HIP; }

int type_bytes(int32_t dtype) {
  return dtype == GS_F32 ? 4 : dtype == GS_BF16 || dtype == GS_F16 ? 2 : 0;
}

// A tensor of batch x tokens x heads rows: present, on 16-byte boundaries with all
// its rows, and, where it is written, with rows that do not overlap each other.
int32_t take(const gs_tokens *t, int64_t batch, int64_t tokens, int64_t heads, int64_t dim,
             int bytes, bool written, TokK *out) {
  *out = {nullptr, 0, 0, 0};
  if (batch == 0 || tokens == 0 || heads == 0) return GS_OK;
  if (!t || !t->data || !aligned(t->data, 16)) return GS_ERR_INVALID_ARGUMENT;
  const int64_t s[3] = {t->batch_stride, t->token_stride, t->head_stride};
  const int64_t n[3] = {batch, tokens, heads};
  for (int i = 0; i < 3; i++) {
    if (n[i] == 1) continue;
    if (s[i] < 0 || s[i] * bytes % 16 != 0) return GS_ERR_INVALID_ARGUMENT;
    if (written && s[i] < dim) return GS_ERR_INVALID_ARGUMENT;
  }
  if (tokens > 1 && s[1] >= TOKEN_STRIDE) return GS_ERR_UNSUPPORTED;
  *out = {t->data, batch > 1 ? s[0] : 0, tokens > 1 ? s[1] : 0, heads > 1 ? s[2] : 0};
  return GS_OK;
}

#define GS_TRY(call)                      \
  do {                                    \
    const int32_t gs_try_status = (call); \
    if (gs_try_status != GS_OK) return gs_try_status; \
  } while (0)

// ---------------------------------------------------------------- norm and rotation

int32_t qk_shape(const gs_qk_shape *s, QkK *k) {
  if (!s || s->batch < 0 || s->tokens < 0 || s->q_heads < 0 || s->k_heads < 0 || s->dim <= 0 ||
      s->rot_dim < 0 || s->rot_dim > s->dim || s->n_positions < 0 || !type_bytes(s->dtype) ||
      (s->neighbours != 0 && s->neighbours != 1) || !isfinite(s->eps) || s->eps < 0.0f ||
      s->positions_stride < 0)
    return GS_ERR_INVALID_ARGUMENT;
  if (s->dim % 8 || s->dim > 256 || s->rot_dim % 8 || s->batch >= LIMIT || s->tokens >= LIMIT ||
      s->q_heads > 65535 || s->k_heads > 65535 ||
      (int64_t)s->batch * s->tokens >= LIMIT)
    return GS_ERR_UNSUPPORTED;
  int lanes = 1;  // of a row of one head
  while (lanes * 8 < s->dim) lanes *= 2;
  const int chunks = (s->q_heads + 3) / 4 + (s->k_heads + 3) / 4;
  if ((int64_t)s->batch * s->tokens * chunks * lanes > THREADS - 256) return GS_ERR_UNSUPPORTED;
  *k = {};
  k->batch = s->batch;
  k->tokens = s->tokens;
  k->q_heads = s->q_heads;
  k->k_heads = s->k_heads;
  k->dim = s->dim;
  k->rot = s->rot_dim;
  k->neighbours = s->neighbours;
  k->n_positions = s->n_positions;
  k->eps = s->eps;
  k->pos_stride = s->positions_stride;
  k->lanes = lanes;
  k->blocks = gs_qk_bwd_blocks(s->batch, s->tokens, s->q_heads, s->k_heads, k->lanes);
  return GS_OK;
}

int32_t qk_args(const gs_qk_shape *s, QkK *k, const gs_tokens *q, const gs_tokens *kk,
                const float *q_weight, const float *k_weight, const float *cos_sin,
                const int32_t *positions) {
  GS_TRY(qk_shape(s, k));
  const int bytes = type_bytes(s->dtype);
  GS_TRY(take(q, s->batch, s->tokens, s->q_heads, s->dim, bytes, false, &k->q));
  GS_TRY(take(kk, s->batch, s->tokens, s->k_heads, s->dim, bytes, false, &k->k));
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(cos_sin, 16) ||
      !aligned(positions, 4))
    return GS_ERR_INVALID_ARGUMENT;
  if (s->rot_dim && s->n_positions && !cos_sin) return GS_ERR_INVALID_ARGUMENT;
  if (s->rot_dim && !positions && s->n_positions < s->tokens) return GS_ERR_INVALID_ARGUMENT;
  k->qw = q_weight;
  k->kw = k_weight;
  k->cos_sin = cos_sin;
  k->positions = positions;
  return GS_OK;
}

// ---------------------------------------------------------------- attention

int32_t attn_shape(const gs_attn_shape *s, AttnK *p) {
  if (!s || s->batch < 0 || s->q_tokens < 0 || s->kv_tokens < 0 || s->q_heads <= 0 ||
      s->kv_heads <= 0 || s->q_heads % s->kv_heads || s->dim <= 0 || !type_bytes(s->dtype) ||
      (s->causal != 0 && s->causal != 1) || !isfinite(s->scale) || !(s->scale > 0.0f) ||
      s->spans_stride < 0)
    return GS_ERR_INVALID_ARGUMENT;
  // (lse / scale, where the backward's scores start, and scale log2 e stay within 32 bits)
  if (s->dtype == GS_F32 || s->dim % 8 || s->dim > 128 || s->q_heads > 65535 ||
      s->q_tokens >= LIMIT || s->kv_tokens >= LIMIT || s->scale < 0x1p-100f ||
      s->scale > 0x1p100f)
    return GS_ERR_UNSUPPORTED;
  // A launch has fewer than 2^32 threads: 512 for every 64 rows of queries and of keys.
  const int64_t bh = (int64_t)s->batch * s->q_heads, bk = (int64_t)s->batch * s->kv_heads;
  const int64_t tiles = THREADS / 512 - 64;  // (some are launched past the last one)
  if (bh >= LIMIT || bh * ((s->q_tokens + 63) / 64) + bk * ((s->kv_tokens + 63) / 64) > tiles)
    return GS_ERR_UNSUPPORTED;
  *p = {};
  p->batch = s->batch;
  p->q_heads = s->q_heads;
  p->kv_heads = s->kv_heads;
  p->share = s->q_heads / s->kv_heads;
  p->q_len = s->q_tokens;
  p->kv_len = s->kv_tokens;
  p->dim = s->dim;
  p->causal = s->causal;
  p->scale = s->scale;
  p->scale_log2 = (float)((double)s->scale * 1.4426950408889634);
  p->span_stride = s->spans_stride;
  return GS_OK;
}

// Workspace of the forward's split form: o, then m and l of every part and row. (Spans
// may choose between forms without one, not its size.)
size_t attn_layout(AttnK *p, void *ws) {
  gs_attn_plan(p);
  if (p->splits <= 1) return 0;
  const size_t slots = (size_t)p->splits * p->batch * p->q_heads * p->q_len;
  const size_t o = round256(slots * p->dim * 4);
  p->part_o = (float *)ws;
  p->part_ml = (float *)((char *)ws + o);
  return o + round256(slots * 8);
}

size_t attn_bwd_layout(AttnK *p, bool masked, void *ws) {
  const size_t qt = (p->q_len + 63) / 64, b = p->batch;
  char *at = (char *)ws;
  size_t total = 0;
  auto part = [&](size_t bytes) {
    char *r = at + total;
    total += round256(bytes);
    return r;
  };
  p->q_pad = (int)(qt * 64);
  p->row_lse = (float *)part(b * p->q_heads * p->q_pad * 4);
  p->row_delta = (float *)part(b * p->q_heads * p->q_pad * 4);
  p->row_spans = (int2 *)part(masked ? b * p->q_pad * 8 : 0);
  char *spans = part(masked ? b * qt * 16 : 0);
  p->tile_spans = masked ? (int4 *)spans : nullptr;
  gs_attn_bwd_plan(p, masked);
  const size_t q = b * p->q_heads * p->q_len * p->dim * 4, k = b * p->kv_heads * p->kv_len * p->dim * 4;
  p->part_q = (float *)part(p->q_parts > 1 ? q * p->q_parts : 0);
  p->part_k = (float *)part(p->kv_parts > 1 ? k * p->kv_parts : 0);
  p->part_v = (float *)part(p->kv_parts > 1 ? k * p->kv_parts : 0);
  return total;
}

int32_t attn_inputs(const gs_attn_shape *s, AttnK *p, const gs_tokens *q, const gs_tokens *k,
                    const gs_tokens *v, const int32_t *spans) {
  GS_TRY(attn_shape(s, p));
  GS_TRY(take(q, s->batch, s->q_tokens, s->q_heads, s->dim, 2, false, &p->q));
  GS_TRY(take(k, s->batch, s->kv_tokens, s->kv_heads, s->dim, 2, false, &p->k));
  GS_TRY(take(v, s->batch, s->kv_tokens, s->kv_heads, s->dim, 2, false, &p->v));
  if (!aligned(spans, 8)) return GS_ERR_INVALID_ARGUMENT;
  p->spans = (const int2 *)spans;
  return GS_OK;
}

}  // namespace

extern "C" {

size_t gs_qk_workspace_size(const gs_qk_shape *shape) {
  QkK k;
  if (qk_shape(shape, &k) != GS_OK) return 0;
  return round256((size_t)2 * k.blocks * k.dim * 4);
}

int32_t gs_qk_norm_rope(const gs_qk_shape *shape, const gs_tokens *q, const gs_tokens *k,
                        const float *q_weight, const float *k_weight, const float *cos_sin,
                        const int32_t *positions, const gs_tokens *q_out, const gs_tokens *k_out,
                        void *stream) {
  QkK p;
  GS_TRY(qk_args(shape, &p, q, k, q_weight, k_weight, cos_sin, positions));
  const int bytes = type_bytes(shape->dtype);
  GS_TRY(take(q_out, shape->batch, shape->tokens, shape->q_heads, shape->dim, bytes, true, &p.qo));
  GS_TRY(take(k_out, shape->batch, shape->tokens, shape->k_heads, shape->dim, bytes, true, &p.ko));
  if (p.batch == 0 || p.tokens == 0 || p.q_heads + p.k_heads == 0) return GS_OK;
  return hip_status(gs_launch_qk_fwd(p, shape->dtype, (hipStream_t)stream));
}

int32_t gs_qk_norm_rope_bwd(const gs_qk_shape *shape, const gs_tokens *dL_dq_out,
                            const gs_tokens *dL_dk_out, const gs_tokens *q, const gs_tokens *k,
                            const float *q_weight, const float *k_weight, const float *cos_sin,
                            const int32_t *positions, const gs_tokens *dL_dq,
                            const gs_tokens *dL_dk, float *dL_dq_weight, float *dL_dk_weight,
                            void *workspace, size_t workspace_bytes, void *stream) {
  QkK p;
  GS_TRY(qk_args(shape, &p, q, k, q_weight, k_weight, cos_sin, positions));
  const int bytes = type_bytes(shape->dtype);
  const int64_t B = shape->batch, n = shape->tokens;
  GS_TRY(take(dL_dq_out, B, n, shape->q_heads, shape->dim, bytes, false, &p.qg));
  GS_TRY(take(dL_dk_out, B, n, shape->k_heads, shape->dim, bytes, false, &p.kg));
  GS_TRY(take(dL_dq, B, n, shape->q_heads, shape->dim, bytes, true, &p.qo));
  GS_TRY(take(dL_dk, B, n, shape->k_heads, shape->dim, bytes, true, &p.ko));
  if (!aligned(dL_dq_weight, 4) || !aligned(dL_dk_weight, 4)) return GS_ERR_INVALID_ARGUMENT;
  p.dqw = dL_dq_weight;
  p.dkw = dL_dk_weight;
  if (p.dqw || p.dkw) {
    if (workspace_bytes < gs_qk_workspace_size(shape)) return GS_ERR_WORKSPACE;
    if (p.blocks && (!workspace || !aligned(workspace, 256))) return GS_ERR_INVALID_ARGUMENT;
    p.partial = (float *)workspace;
  } else if (p.blocks == 0) {
    return GS_OK;
  }
  return hip_status(gs_launch_qk_bwd(p, shape->dtype, (hipStream_t)stream));
}

size_t gs_attention_workspace_size(const gs_attn_shape *shape) {
  AttnK p;
  if (attn_shape(shape, &p) != GS_OK) return 0;
  return attn_layout(&p, nullptr);
}

size_t gs_attention_bwd_workspace_size(const gs_attn_shape *shape) {
  AttnK p;
  if (attn_shape(shape, &p) != GS_OK) return 0;
  // with spans or without: the larger
  AttnK n = p;
  const size_t a = attn_bwd_layout(&p, true, nullptr);
  const size_t c = attn_bwd_layout(&n, false, nullptr);
  return a > c ? a : c;
}

int32_t gs_attention(const gs_attn_shape *shape, const gs_tokens *q, const gs_tokens *k,
                     const gs_tokens *v, const int32_t *spans, const gs_tokens *o, float *lse,
                     void *workspace, size_t workspace_bytes, void *stream) {
  AttnK p;
  GS_TRY(attn_inputs(shape, &p, q, k, v, spans));
  GS_TRY(take(o, shape->batch, shape->q_tokens, shape->q_heads, shape->dim, 2, true, &p.o));
  if (p.batch == 0 || p.q_len == 0) return GS_OK;
  if (!lse || !aligned(lse, 4)) return GS_ERR_INVALID_ARGUMENT;
  p.lse = lse;
  const size_t need = attn_layout(&p, workspace);
  if (workspace_bytes < need) return GS_ERR_WORKSPACE;
  if (need && (!workspace || !aligned(workspace, 256))) return GS_ERR_INVALID_ARGUMENT;
  return hip_status(gs_launch_attn_fwd(p, shape->dtype, (hipStream_t)stream));
}

int32_t gs_attention_bwd(const gs_attn_shape *shape, const gs_tokens *dL_do, const gs_tokens *q,
                         const gs_tokens *k, const gs_tokens *v, const int32_t *spans,
                         const gs_tokens *o, const float *lse, const gs_tokens *dL_dq,
                         const gs_tokens *dL_dk, const gs_tokens *dL_dv, void *workspace,
                         size_t workspace_bytes, void *stream) {
  AttnK p;
  GS_TRY(attn_inputs(shape, &p, q, k, v, spans));
  const int64_t B = shape->batch, nq = shape->q_tokens, nk = shape->kv_tokens;
  GS_TRY(take(o, B, nq, shape->q_heads, shape->dim, 2, false, &p.o));
  GS_TRY(take(dL_do, B, nq, shape->q_heads, shape->dim, 2, false, &p.d_o));
  GS_TRY(take(dL_dq, B, nq, shape->q_heads, shape->dim, 2, true, &p.dq));
  GS_TRY(take(dL_dk, B, nk, shape->kv_heads, shape->dim, 2, true, &p.dk));
  GS_TRY(take(dL_dv, B, nk, shape->kv_heads, shape->dim, 2, true, &p.dv));
  if (p.batch == 0 || (nq == 0 && nk == 0)) return GS_OK;
  if ((nq && !lse) || !aligned(lse, 4)) return GS_ERR_INVALID_ARGUMENT;
  p.lse = (float *)lse;
  const size_t need = gs_attention_bwd_workspace_size(shape);
  if (workspace_bytes < need) return GS_ERR_WORKSPACE;
  if (need && (!workspace || !aligned(workspace, 256))) return GS_ERR_INVALID_ARGUMENT;
  attn_bwd_layout(&p, spans != nullptr || p.causal, workspace);
  return hip_status(gs_launch_attn_bwd(p, shape->dtype, (hipStream_t)stream));
}

int32_t gs_dropout(int64_t rows, int64_t cols, int32_t dtype, const void *x, int64_t x_stride,
                   const void *residual, int64_t residual_stride, void *y, int64_t y_stride,
                   double p, uint64_t seed, uint64_t offset, int32_t per_row, void *stream) {
  const int bytes = type_bytes(dtype);
  if (rows < 0 || cols < 0 || !bytes || !(p >= 0.0 && p < 1.0) || (per_row != 0 && per_row != 1))
    return GS_ERR_INVALID_ARGUMENT;
  if (rows == 0 || cols == 0) return GS_OK;
  const int64_t most = (int64_t)1 << 40;
  if (rows > most || cols > most || rows > most / cols) return GS_ERR_UNSUPPORTED;
  if (!x || !y || !aligned(x, bytes) || !aligned(residual, bytes) || !aligned(y, bytes))
    return GS_ERR_INVALID_ARGUMENT;
  if (rows > 1 && (x_stride < 0 || (residual && residual_stride < 0) || y_stride < cols))
    return GS_ERR_INVALID_ARGUMENT;
  DropK k = {};
  k.rows = rows;
  k.cols = cols;
  k.x = x;
  k.res = residual;
  k.y = y;
  k.x_stride = x_stride;
  k.res_stride = residual_stride;
  k.y_stride = y_stride;
  k.seed = seed;
  k.offset = offset;
  const double below = nearbyint(p * 4294967296.0);  // p < 1 may round up to 2^32
  k.drop_below = below >= 4294967295.0 ? 0xffffffffu : (uint32_t)below;
  k.scale = (float)(1.0 / (1.0 - p));
  k.per_row = per_row;
  return hip_status(gs_launch_dropout(k, dtype, (hipStream_t)stream));
}

}  // extern "C"
