// C entry points of the operators that feed the non-matrix parameters:
// argument checks, launch shapes and workspace layout.  Nothing is uploaded and
// nothing is kept between calls, so every call may be recorded into a graph.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <string>

#include "api_checks.hpp"
#include "ops.hpp"

namespace dmuon {
namespace {

// ---------------------------------------------------------------- embedding plan
struct PlanLayout {
  int passes, bits, items, blocks;
  size_t off_key[2], off_idx[2], off_counts, off_heads, total;
};
PlanLayout plan_layout(int64_t n, int64_t vocab) {
  PlanLayout l{};
  int need = 1;
  while ((int64_t{1} << need) <= vocab) ++need;   // the value `vocab` stands for an unknown token
  l.passes = (need + 8) / 9;
  l.bits = (need + l.passes - 1) / l.passes;
  if (n <= kPlanSmall) return l;
  l.items = static_cast<int>((n + int64_t{kPlanThreads} * kPlanMaxBlocks - 1) / (int64_t{kPlanThreads} * kPlanMaxBlocks)) *
            kPlanThreads;
  l.blocks = static_cast<int>((n + l.items - 1) / l.items);
  size_t off = 0;
  for (int k = 0; k < 2; ++k) {
    l.off_key[k] = off;
    off = align_up(off + sizeof(unsigned) * n);
    l.off_idx[k] = off;
    off = align_up(off + sizeof(int) * n);
  }
  l.off_counts = off;
  off = align_up(off + sizeof(int) * l.blocks * (size_t{1} << l.bits));
  l.off_heads = off;
  off = align_up(off + sizeof(int) * l.blocks);
  l.total = off;
  return l;
}

int check_tokens(int64_t n, int64_t vocab) {
  DMUON_TRY(check_range(n, 0, DMUON_MAX_TOKENS, "n"));
  return check_range(vocab, 1, DMUON_MAX_VOCAB, "vocab");
}

// ---------------------------------------------------------------- embedding gradient
// Sorted positions per chunk: long chunks leave fewer unfinished sums, short
// ones give a small batch enough blocks (a block covers 256 16-byte columns).
int egrad_chunk(int64_t n, int64_t dim, int dout_dtype) {
  const int64_t c = dout_dtype == kBF16 ? 8 : 4;
  const int64_t tiles = ((dim + c - 1) / c + kEgThreads - 1) / kEgThreads;
  int chunk = 32;
  while (chunk > 8 && (n + chunk - 1) / chunk * tiles < 2048) chunk /= 2;
  return chunk;
}

// ---------------------------------------------------------------- AdamW rows
int check_adamw_rows(const void* param, const void* grad_rows, int64_t n_grad_rows, const int32_t* row_index,
                     const float* exp_avg, const float* exp_avg_sq, int64_t rows, int64_t dim, int dtype, int step,
                     float lr, float beta1, float beta2, float eps, float weight_decay) {
  DMUON_TRY(check_float(dtype, "dtype"));
  DMUON_TRY(check_range(rows, 1, DMUON_MAX_VOCAB, "rows"));
  DMUON_TRY(check_range(dim, 1, DMUON_MAX_DIM, "dim"));
  DMUON_TRY(check_range(n_grad_rows, 0, DMUON_MAX_TOKENS, "n_grad_rows"));
  if (step < 1) return invalid("step counts from 1");
  if (!std::isfinite(lr) || !std::isfinite(weight_decay) || !std::isfinite(eps) || eps < 0.0f)
    return invalid("lr and weight_decay must be finite, eps finite and >= 0");
  if (!(beta1 >= 0.0f && beta1 < 1.0f) || !(beta2 >= 0.0f && beta2 < 1.0f)) return invalid("betas must lie in [0, 1)");
  const int64_t es = size_of(dtype), numel = rows * dim;
  const Buf bufs[] = {flat("param", param, numel * es, es, true), flat("exp_avg", exp_avg, numel * 4, 4, true),
                      flat("exp_avg_sq", exp_avg_sq, numel * 4, 4, true),
                      flat("grad_rows", grad_rows, n_grad_rows * dim * es, es, false),
                      flat("row_index", row_index, rows * 4, 4, false)};
  return check_bufs(bufs, 5);
}

// ---------------------------------------------------------------- distillation
constexpr int64_t kDistillPartBytes = 8 * sizeof(float);
// Blocks per row, for a few long rows (at least 8192 elements each); 0: a
// block takes a whole row, in one launch.
int distill_slices(int64_t n, int64_t vocab) {
  if (n > 128 || vocab <= 65536) return 0;
  return static_cast<int>(std::min<int64_t>({(1024 + n - 1) / std::max<int64_t>(n, 1), (vocab + 8191) / 8192, 64}));
}

// ---------------------------------------------------------------- query / key norm
int check_qk(const dmuon_qk_shape* s) {
  if (!s) return invalid("shape is NULL");
  DMUON_TRY(check_float(s->dtype, "dtype"));
  DMUON_TRY(check_float(s->weight_dtype, "weight_dtype"));
  DMUON_TRY(check_range(s->tokens, 0, DMUON_MAX_TOKENS, "tokens"));
  DMUON_TRY(check_range(s->q_heads, 0, DMUON_MAX_HEADS, "q_heads"));
  DMUON_TRY(check_range(s->k_heads, 0, DMUON_MAX_HEADS, "k_heads"));
  if (s->q_heads + s->k_heads == 0) return invalid("q_heads and k_heads are both 0");
  DMUON_TRY(check_range(s->head_dim, 1, DMUON_MAX_HEAD_DIM, "head_dim"));
  DMUON_TRY(check_range(s->rot_dim, 0, s->head_dim, "rot_dim"));
  if (s->rot_dim % 2) return invalid("rot_dim must be even");
  if (!(std::isfinite(s->eps) && s->eps >= 0.0f)) return invalid("eps must be finite and >= 0");
  if (!std::isfinite(s->weight_offset)) return invalid("weight_offset must be finite");
  if (s->rot_dim > 0) {
    DMUON_TRY(check_index(s->pos_dtype, "pos_dtype"));
    DMUON_TRY(check_range(s->max_pos, 1, int64_t{1} << 31, "max_pos"));
  }
  return DMUON_OK;
}

// Token rows of one tensor of `heads` heads.
int qk_buf(const dmuon_qk_shape& s, const char* name, const void* p, int64_t stride, int heads, bool written, Buf* out) {
  const int64_t es = size_of(s.dtype), width = static_cast<int64_t>(heads) * s.head_dim;
  *out = Buf{name, p, heads > 0 ? s.tokens : 0, width * es, stride * es, es, written};
  if (heads > 0 && s.tokens > 1 && (stride < width || stride > (int64_t{1} << 31)))
    return invalid(std::string(name) + "'s stride " + std::to_string(stride) + " is shorter than its " +
                   std::to_string(width) + " elements per token, or over 2^31");
  return DMUON_OK;
}

// Blocks of the backward pass for one tensor: each leaves one row of gain
// sums.  At least 32 heads a block, and no more than eight blocks a CU in all.
int qk_grad_blocks(const dmuon_qk_shape& s, int heads) {
  const int64_t want = (s.tokens * heads + 31) / 32, all = s.q_heads + s.k_heads;
  return static_cast<int>(std::min<int64_t>(want, std::max<int64_t>(1, int64_t{2048} * heads / all)));
}

// Pairs that a lane holds: 16 bytes of each half.  By type and shape alone, so
// that strides and alignment do not change the order of a sum.
int qk_pairs(const dmuon_qk_shape& s) {
  return s.dtype == DMUON_BF16 && s.head_dim % 16 == 0 && s.rot_dim % 16 == 0 ? 8 : 4;
}
// Those pairs can be loaded at once: whole, aligned runs in every row.
bool qk_vec(const dmuon_qk_shape& s, std::initializer_list<const Buf*> bufs, std::initializer_list<const void*> gains) {
  const int pairs = qk_pairs(s);
  if (s.head_dim % (2 * pairs) || s.rot_dim % (2 * pairs)) return false;
  const int64_t run = pairs * size_of(s.dtype), gain_run = std::min<int64_t>(16, pairs * size_of(s.weight_dtype));
  for (const Buf* b : bufs)
    if (!b->empty() && (!aligned(b->p, run) || (b->rows > 1 && b->pitch % run))) return false;
  for (const void* w : gains)
    if (w && !aligned(w, gain_run)) return false;
  return true;
}

void fill_qk(const dmuon_qk_shape& s, const float* rope, QkArgs* a) {
  a->n = s.tokens;
  a->heads[0] = s.q_heads;
  a->heads[1] = s.k_heads;
  a->dim = s.head_dim;
  a->rot = s.rot_dim;
  a->interleaved = s.interleaved ? 1 : 0;
  a->max_pos = s.rot_dim ? s.max_pos : INT64_MAX;   // no table, none to be behind
  a->eps = s.eps;
  a->offset = s.weight_offset;
  a->pos64 = s.pos_dtype == DMUON_I64;
  a->pairs = qk_pairs(s);
  a->rope_vec = aligned(rope, 16) && s.rot_dim % 8 == 0;
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" {

int dmuon_embedding_forward(const void* table, int64_t vocab, int64_t dim, int table_dtype, const void* tokens,
                            int64_t n, int token_dtype, float scale, void* out, int out_dtype, void* hip_stream) {
  return guarded([&]() -> int {
    DMUON_TRY(check_float(table_dtype, "table_dtype"));
    DMUON_TRY(check_float(out_dtype, "out_dtype"));
    DMUON_TRY(check_index(token_dtype, "token_dtype"));
    DMUON_TRY(check_tokens(n, vocab));
    DMUON_TRY(check_range(dim, 1, DMUON_MAX_DIM, "dim"));
    if (!std::isfinite(scale)) return invalid("scale must be finite");
    const int64_t ts = size_of(table_dtype), os = size_of(out_dtype), ks = size_of(token_dtype);
    const Buf bufs[] = {flat("out", out, n * dim * os, os, true), flat("table", table, n ? vocab * dim * ts : 0, ts, false),
                        flat("tokens", tokens, n * ks, ks, false)};
    DMUON_TRY(check_bufs(bufs, 3));
    bool capturing = false;
    DMUON_TRY(check_device(hip_stream, &capturing));
    if (n == 0) return DMUON_OK;
    EmbedArgs a{};
    a.table = table;
    a.tokens = tokens;
    a.out = out;
    a.n = n;
    a.vocab = vocab;
    a.dim = dim;
    a.scale = scale;
    a.tok64 = token_dtype == DMUON_I64;
    return launched("embedding", kKEmbed, 0.0, static_cast<double>(n) * dim * (ts + os), hip_stream, capturing,
                    [&] { return launch_embed(table_dtype, out_dtype, a, static_cast<hipStream_t>(hip_stream)); });
  });
}

int dmuon_embedding_plan_workspace_bytes(int64_t n, int64_t vocab, size_t* bytes_out) {
  return guarded([&]() -> int {
    if (!bytes_out) return invalid("bytes_out is NULL");
    DMUON_TRY(check_tokens(n, vocab));
    *bytes_out = plan_layout(n, vocab).total;
    return DMUON_OK;
  });
}

int dmuon_embedding_plan(const void* tokens, int64_t n, int token_dtype, int64_t vocab, int32_t* order, int32_t* slot,
                         int32_t* rows, int32_t* row_index, int32_t* count, void* workspace, size_t workspace_bytes,
                         void* hip_stream) {
  return guarded([&]() -> int {
    DMUON_TRY(check_index(token_dtype, "token_dtype"));
    DMUON_TRY(check_tokens(n, vocab));
    const PlanLayout l = plan_layout(n, vocab);
    const int64_t cap = std::min(n, vocab), ks = size_of(token_dtype);
    DMUON_TRY(check_workspace(workspace, workspace_bytes, l.total));
    const Buf bufs[] = {flat("tokens", tokens, n * ks, ks, false), flat("order", order, n * 4, 4, true),
                        flat("slot", slot, n * 4, 4, true), flat("rows", rows, cap * 4, 4, true),
                        flat("row_index", row_index, vocab * 4, 4, true), flat("count", count, 4, 4, true),
                        flat("workspace", workspace, static_cast<int64_t>(l.total), 1, true)};
    DMUON_TRY(check_bufs(bufs, 7));
    bool capturing = false;
    DMUON_TRY(check_device(hip_stream, &capturing));
    char* ws = static_cast<char*>(workspace);
    PlanArgs a{};
    a.tokens = tokens;
    a.vocab = vocab;
    a.n = static_cast<int>(n);
    a.tok64 = token_dtype == DMUON_I64;
    a.cap = static_cast<int>(cap);
    a.bits = l.bits;
    a.passes = l.passes;
    a.items = l.items;
    a.blocks = l.blocks;
    a.order = order;
    a.slot = slot;
    a.rows = rows;
    a.row_index = row_index;
    a.count = count;
    if (l.total > 0) {
      for (int k = 0; k < 2; ++k) {
        a.key[k] = reinterpret_cast<unsigned*>(ws + l.off_key[k]);
        a.idx[k] = reinterpret_cast<int*>(ws + l.off_idx[k]);
      }
      a.counts = reinterpret_cast<int*>(ws + l.off_counts);
      a.heads = reinterpret_cast<int*>(ws + l.off_heads);
    }
    return launched("embedding plan", kKEmbedPlan, 0.0, static_cast<double>(n) * (ks + 8) + 4.0 * vocab, hip_stream,
                    capturing, [&] { return launch_embed_plan(a, static_cast<hipStream_t>(hip_stream)); });
  });
}

int dmuon_embedding_backward_workspace_bytes(int64_t n, int64_t dim, int dout_dtype, size_t* bytes_out) {
  return guarded([&]() -> int {
    if (!bytes_out) return invalid("bytes_out is NULL");
    DMUON_TRY(check_float(dout_dtype, "dout_dtype"));
    DMUON_TRY(check_range(n, 0, DMUON_MAX_TOKENS, "n"));
    DMUON_TRY(check_range(dim, 1, DMUON_MAX_DIM, "dim"));
    const int64_t chunk = egrad_chunk(n, dim, dout_dtype), chunks = (n + chunk - 1) / chunk;
    *bytes_out = chunks < 2 ? 0 : align_up(sizeof(float) * 2 * chunks * dim);
    return DMUON_OK;
  });
}

int dmuon_embedding_backward(const void* dout, int64_t n, int64_t dim, int dout_dtype, float scale,
                             const int32_t* order, const int32_t* slot, const int32_t* rows,
                             const int32_t* row_index, const int32_t* count, int64_t vocab, int form, void* grad,
                             int grad_dtype, void* workspace, size_t workspace_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    DMUON_TRY(check_float(dout_dtype, "dout_dtype"));
    DMUON_TRY(check_float(grad_dtype, "grad_dtype"));
    DMUON_TRY(check_tokens(n, vocab));
    DMUON_TRY(check_range(dim, 1, DMUON_MAX_DIM, "dim"));
    DMUON_TRY(check_range(form, DMUON_EMBED_DENSE, DMUON_EMBED_ROWS, "form"));
    if (!std::isfinite(scale)) return invalid("scale must be finite");
    size_t need = 0;
    DMUON_TRY(dmuon_embedding_backward_workspace_bytes(n, dim, dout_dtype, &need));
    DMUON_TRY(check_workspace(workspace, workspace_bytes, need));
    const int64_t cap = std::min(n, vocab), ds = size_of(dout_dtype), gs = size_of(grad_dtype);
    const int64_t grad_rows = form == DMUON_EMBED_ROWS ? cap : vocab;
    const Buf bufs[] = {flat("grad", grad, grad_rows * dim * gs, gs, true), flat("dout", dout, n * dim * ds, ds, false),
                        flat("order", order, n * 4, 4, false), flat("slot", slot, n * 4, 4, false),
                        flat("rows", rows, cap * 4, 4, false), flat("row_index", row_index, vocab * 4, 4, false),
                        flat("count", count, 4, 4, false),
                        flat("workspace", workspace, static_cast<int64_t>(need), 1, true)};
    DMUON_TRY(check_bufs(bufs, 8));
    bool capturing = false;
    DMUON_TRY(check_device(hip_stream, &capturing));
    EmbedGradArgs a{};
    a.dout = dout;
    a.order = order;
    a.slot = slot;
    a.rows = rows;
    a.row_index = row_index;
    a.count = count;
    a.grad = grad;
    a.part = static_cast<float*>(workspace);
    a.n = n;
    a.vocab = vocab;
    a.dim = dim;
    a.scale = scale;
    a.cap = static_cast<int>(cap);
    a.form = form;
    a.chunk = egrad_chunk(n, dim, dout_dtype);
    a.chunks = static_cast<int>((n + a.chunk - 1) / a.chunk);
    const double out_rows = form == DMUON_EMBED_ADD ? 2.0 * cap : static_cast<double>(grad_rows);
    return launched("embedding gradient", kKEmbedGrad, static_cast<double>(n) * dim,
                    static_cast<double>(dim) * (static_cast<double>(n) * ds + out_rows * gs), hip_stream, capturing,
                    [&] { return launch_embed_grad(dout_dtype, grad_dtype, a, static_cast<hipStream_t>(hip_stream)); });
  });
}

int dmuon_adamw_rows_check(const void* param, const void* grad_rows, int64_t n_grad_rows, const int32_t* row_index,
                           const float* exp_avg, const float* exp_avg_sq, int64_t rows, int64_t dim, int dtype,
                           int step, float lr, float beta1, float beta2, float eps, float weight_decay) {
  return guarded([&]() -> int {
    return check_adamw_rows(param, grad_rows, n_grad_rows, row_index, exp_avg, exp_avg_sq, rows, dim, dtype, step, lr,
                            beta1, beta2, eps, weight_decay);
  });
}

int dmuon_adamw_rows_step(void* param, const void* grad_rows, int64_t n_grad_rows, const int32_t* row_index,
                          float* exp_avg, float* exp_avg_sq, int64_t rows, int64_t dim, int dtype, int step, float lr,
                          float beta1, float beta2, float eps, float weight_decay, void* hip_stream) {
  return guarded([&]() -> int {
    DMUON_TRY(check_adamw_rows(param, grad_rows, n_grad_rows, row_index, exp_avg, exp_avg_sq, rows, dim, dtype, step, lr,
                               beta1, beta2, eps, weight_decay));
    const int64_t es = size_of(dtype), numel = rows * dim;
    bool capturing = false;
    DMUON_TRY(check_device(hip_stream, &capturing));
    AdamRowsArgs a{};
    a.p = param;
    a.g = grad_rows;
    a.row_index = row_index;
    a.m = exp_avg;
    a.v = exp_avg_sq;
    a.rows = rows;
    a.dim = dim;
    a.n_grad_rows = n_grad_rows;
    a.hp = adam_args(step, lr, beta1, beta2, eps, weight_decay);
    const double bytes = static_cast<double>(numel) * (2.0 * es + 16.0) +
                         static_cast<double>(std::min(n_grad_rows, rows)) * dim * es;
    return launched("AdamW rows", kKAdamwRows, 0.0, bytes, hip_stream, capturing,
                    [&] { return launch_adamw_rows(dtype, a, static_cast<hipStream_t>(hip_stream)); });
  });
}

int dmuon_distill_loss_workspace_bytes(int64_t n, int64_t vocab, size_t* bytes_out) {
  return guarded([&]() -> int {
    if (!bytes_out) return invalid("bytes_out is NULL");
    DMUON_TRY(check_tokens(n, vocab));
    *bytes_out = align_up(static_cast<size_t>(n * distill_slices(n, vocab) * kDistillPartBytes));
    return DMUON_OK;
  });
}

int dmuon_distill_loss(const void* logits, int64_t n, int64_t vocab, int64_t logits_stride, int dtype,
                       const void* teacher_index, int index_dtype, const float* teacher_logits, int k,
                       const void* labels, float temperature, float kd_weight, float ce_weight,
                       const float* row_weight, float grad_scale, float* losses, void* dlogits,
                       int64_t dlogits_stride, void* workspace, size_t workspace_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    DMUON_TRY(check_float(dtype, "dtype"));
    DMUON_TRY(check_index(index_dtype, "index_dtype"));
    DMUON_TRY(check_tokens(n, vocab));
    DMUON_TRY(check_range(k, 0, DMUON_MAX_TEACHER_K, "k"));
    // log2(e) / T is then a normal float, and its product with a logit at most overflows to infinity
    if (!(temperature >= 1e-6f && temperature <= 1e6f)) return invalid("temperature must lie in [1e-6, 1e6]");
    if (!std::isfinite(kd_weight) || !std::isfinite(ce_weight) || !std::isfinite(grad_scale))
      return invalid("kd_weight, ce_weight and grad_scale must be finite");
    if (k == 0 && kd_weight != 0.0f) return invalid("kd_weight must be 0 without teacher entries");
    if (!labels && ce_weight != 0.0f) return invalid("ce_weight must be 0 without labels");
    const int64_t most = int64_t{1} << 31;
    if (n > 1) {
      DMUON_TRY(check_range(logits_stride, vocab, most, "logits_stride"));
      if (dlogits) DMUON_TRY(check_range(dlogits_stride, vocab, most, "dlogits_stride"));
    }
    size_t need = 0;
    DMUON_TRY(dmuon_distill_loss_workspace_bytes(n, vocab, &need));
    DMUON_TRY(check_workspace(workspace, workspace_bytes, need));
    const int64_t es = size_of(dtype), is = size_of(index_dtype);
    const Buf bufs[] = {Buf{"logits", logits, n, vocab * es, logits_stride * es, es, false},
                        Buf{"dlogits", dlogits, dlogits ? n : 0, vocab * es, dlogits_stride * es, es, true},
                        flat("losses", losses, n * 4, 4, true),
                        flat("teacher_index", teacher_index, n * k * is, is, false),
                        flat("teacher_logits", teacher_logits, n * k * 4, 4, false),
                        flat("labels", labels, labels ? n * is : 0, is, false),
                        flat("row_weight", row_weight, row_weight ? n * 4 : 0, 4, false),
                        flat("workspace", workspace, static_cast<int64_t>(need), 1, true)};
    const int in_place[1][2] = {{0, 1}};
    DMUON_TRY(check_bufs(bufs, 8, in_place, 1));
    bool capturing = false;
    DMUON_TRY(check_device(hip_stream, &capturing));
    if (n == 0) return DMUON_OK;
    DistillArgs a{};
    a.logits = logits;
    a.index = teacher_index;
    a.teacher = teacher_logits;
    a.labels = labels;
    a.row_weight = row_weight;
    a.losses = losses;
    a.dlogits = dlogits;
    a.part = static_cast<float*>(workspace);
    a.n = n;
    a.vocab = vocab;
    a.stride = logits_stride;
    a.dstride = dlogits_stride;
    a.k = k;
    a.idx64 = index_dtype == DMUON_I64;
    a.slices = distill_slices(n, vocab);
    if (a.slices > 0) a.slice_len = ((vocab + a.slices - 1) / a.slices + 7) / 8 * 8;
    a.temperature = temperature;
    a.kd = kd_weight;
    a.ce = ce_weight;
    a.grad_scale = grad_scale;
    const double elems = static_cast<double>(n) * vocab;
    return launched("distillation loss", kKDistill, (dlogits ? 8.0 : 4.0) * elems, elems * es * (dlogits ? 2.0 : 1.0),
                    hip_stream, capturing,
                    [&] { return launch_distill(dtype, a, static_cast<hipStream_t>(hip_stream)); });
  });
}

int dmuon_qk_norm_rope_forward(const dmuon_qk_shape* shape, const void* q, int64_t q_stride, const void* k,
                               int64_t k_stride, const void* q_weight, const void* k_weight, const void* positions,
                               const float* rope, void* q_out, int64_t q_out_stride, void* k_out,
                               int64_t k_out_stride, void* hip_stream) {
  return guarded([&]() -> int {
    DMUON_TRY(check_qk(shape));
    const dmuon_qk_shape& s = *shape;
    if (positions) DMUON_TRY(check_index(s.pos_dtype, "pos_dtype"));
    const int64_t ws = size_of(s.weight_dtype), ps = size_of(s.pos_dtype);
    Buf b[8];
    DMUON_TRY(qk_buf(s, "q", q, q_stride, s.q_heads, false, &b[0]));
    DMUON_TRY(qk_buf(s, "k", k, k_stride, s.k_heads, false, &b[1]));
    DMUON_TRY(qk_buf(s, "q_out", q_out, q_out_stride, s.q_heads, true, &b[2]));
    DMUON_TRY(qk_buf(s, "k_out", k_out, k_out_stride, s.k_heads, true, &b[3]));
    b[4] = flat("q_weight", q_weight, q_weight ? s.head_dim * ws : 0, ws, false);
    b[5] = flat("k_weight", k_weight, k_weight ? s.head_dim * ws : 0, ws, false);
    b[6] = flat("positions", positions, s.rot_dim || positions ? s.tokens * ps : 0, ps, false);
    b[7] = flat("rope", rope, s.rot_dim && s.tokens ? s.max_pos * s.rot_dim * 4 : 0, 4, false);
    const int in_place[2][2] = {{0, 2}, {1, 3}};
    DMUON_TRY(check_bufs(b, 8, in_place, 2));
    bool capturing = false;
    DMUON_TRY(check_device(hip_stream, &capturing));
    if (s.tokens == 0) return DMUON_OK;
    QkArgs a{};
    fill_qk(s, rope, &a);
    a.x[0] = q;
    a.x[1] = k;
    a.x_stride[0] = q_stride;
    a.x_stride[1] = k_stride;
    a.out[0] = q_out;
    a.out[1] = k_out;
    a.out_stride[0] = q_out_stride;
    a.out_stride[1] = k_out_stride;
    a.w[0] = q_weight;
    a.w[1] = k_weight;
    a.positions = positions;
    a.rope = rope;
    a.vec = qk_vec(s, {&b[0], &b[1], &b[2], &b[3]}, {q_weight, k_weight});
    const double elems = static_cast<double>(s.tokens) * (s.q_heads + s.k_heads) * s.head_dim;
    return launched("q/k norm", kKQkNorm, 8.0 * elems, 2.0 * elems * size_of(s.dtype), hip_stream, capturing, [&] {
      return launch_qk_norm(s.dtype, s.weight_dtype, a, static_cast<hipStream_t>(hip_stream));
    });
  });
}

int dmuon_qk_norm_rope_backward_workspace_bytes(const dmuon_qk_shape* shape, size_t* bytes_out) {
  return guarded([&]() -> int {
    if (!bytes_out) return invalid("bytes_out is NULL");
    DMUON_TRY(check_qk(shape));
    const size_t blocks = qk_grad_blocks(*shape, shape->q_heads) + qk_grad_blocks(*shape, shape->k_heads);
    *bytes_out = align_up(sizeof(float) * shape->head_dim * blocks);
    return DMUON_OK;
  });
}

int dmuon_qk_norm_rope_backward(const dmuon_qk_shape* shape, const void* dq_out, int64_t dq_out_stride,
                                const void* dk_out, int64_t dk_out_stride, const void* q, int64_t q_stride,
                                const void* k, int64_t k_stride, const void* q_weight, const void* k_weight,
                                const void* positions, const float* rope, void* dq, int64_t dq_stride, void* dk,
                                int64_t dk_stride, void* dq_weight, void* dk_weight, void* workspace,
                                size_t workspace_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    DMUON_TRY(check_qk(shape));
    const dmuon_qk_shape& s = *shape;
    if (positions) DMUON_TRY(check_index(s.pos_dtype, "pos_dtype"));
    size_t need = 0;
    DMUON_TRY(dmuon_qk_norm_rope_backward_workspace_bytes(shape, &need));
    if (!dq_weight && !dk_weight) need = 0;   // no sums over tokens are asked for
    DMUON_TRY(check_workspace(workspace, workspace_bytes, need));
    const int64_t ws = size_of(s.weight_dtype), ps = size_of(s.pos_dtype);
    Buf b[13];
    DMUON_TRY(qk_buf(s, "dq_out", dq_out, dq_out_stride, s.q_heads, false, &b[0]));
    DMUON_TRY(qk_buf(s, "dk_out", dk_out, dk_out_stride, s.k_heads, false, &b[1]));
    DMUON_TRY(qk_buf(s, "q", q, q_stride, s.q_heads, false, &b[2]));
    DMUON_TRY(qk_buf(s, "k", k, k_stride, s.k_heads, false, &b[3]));
    DMUON_TRY(qk_buf(s, "dq", dq, dq_stride, s.q_heads, true, &b[4]));
    DMUON_TRY(qk_buf(s, "dk", dk, dk_stride, s.k_heads, true, &b[5]));
    b[6] = flat("q_weight", q_weight, q_weight ? s.head_dim * ws : 0, ws, false);
    b[7] = flat("k_weight", k_weight, k_weight ? s.head_dim * ws : 0, ws, false);
    b[8] = flat("positions", positions, s.rot_dim || positions ? s.tokens * ps : 0, ps, false);
    b[9] = flat("rope", rope, s.rot_dim && s.tokens ? s.max_pos * s.rot_dim * 4 : 0, 4, false);
    b[10] = flat("dq_weight", dq_weight, dq_weight ? s.head_dim * ws : 0, ws, true);
    b[11] = flat("dk_weight", dk_weight, dk_weight ? s.head_dim * ws : 0, ws, true);
    b[12] = flat("workspace", workspace, static_cast<int64_t>(need), 1, true);
    const int in_place[4][2] = {{0, 4}, {1, 5}, {2, 4}, {3, 5}};
    DMUON_TRY(check_bufs(b, 13, in_place, 4));
    bool capturing = false;
    DMUON_TRY(check_device(hip_stream, &capturing));
    QkArgs a{};
    fill_qk(s, rope, &a);
    a.x[0] = q;
    a.x[1] = k;
    a.x_stride[0] = q_stride;
    a.x_stride[1] = k_stride;
    a.dy[0] = dq_out;
    a.dy[1] = dk_out;
    a.dy_stride[0] = dq_out_stride;
    a.dy_stride[1] = dk_out_stride;
    a.out[0] = dq;
    a.out[1] = dk;
    a.out_stride[0] = dq_stride;
    a.out_stride[1] = dk_stride;
    a.w[0] = q_weight;
    a.w[1] = k_weight;
    a.dw[0] = dq_weight;
    a.dw[1] = dk_weight;
    a.positions = positions;
    a.rope = rope;
    a.blocks[0] = qk_grad_blocks(s, s.q_heads);
    a.blocks[1] = qk_grad_blocks(s, s.k_heads);
    a.part = need ? static_cast<float*>(workspace) : nullptr;
    a.vec = qk_vec(s, {&b[0], &b[1], &b[2], &b[3], &b[4], &b[5]}, {q_weight, k_weight});
    const double elems = static_cast<double>(s.tokens) * (s.q_heads + s.k_heads) * s.head_dim;
    return launched("q/k norm gradient", kKQkNormGrad, 16.0 * elems, 3.0 * elems * size_of(s.dtype), hip_stream, capturing,
                    [&] { return launch_qk_norm_grad(s.dtype, s.weight_dtype, a, static_cast<hipStream_t>(hip_stream)); });
  });
}

}  // extern "C"
