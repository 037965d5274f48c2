// C entry points of the operators between a decoder block's projections:
// argument checks, launch shapes and workspace layout.  Nothing is uploaded and
// nothing is kept between calls, so every call may be recorded into a graph.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "api_checks.hpp"
#include "block.hpp"

namespace dmuon {
namespace {

constexpr int64_t kMaxStride = int64_t{1} << 31;

// `rows` rows of `width` elements, `stride` elements apart.
int row_buf(const char* name, const void* p, int64_t rows, int64_t width, int64_t stride, int dtype, bool written,
            Buf* out) {
  const int64_t es = size_of(dtype);
  *out = Buf{name, p, rows, width * es, stride * es, es, written};
  if (rows > 1 && (stride < width || stride > kMaxStride))
    return invalid(std::string(name) + "'s stride " + std::to_string(stride) + " is shorter than its rows of " +
                   std::to_string(width) + " elements, or over 2^31");
  return DMUON_OK;
}

// ---------------------------------------------------------------- norms around a block
int check_bn(const dmuon_block_norm_shape* s) {
  if (!s) return invalid("shape is NULL");
  DMUON_TRY(check_float(s->dtype, "dtype"));
  DMUON_TRY(check_float(s->branch_dtype, "branch_dtype"));
  DMUON_TRY(check_float(s->weight_dtype, "weight_dtype"));
  DMUON_TRY(check_range(s->rows, 0, DMUON_MAX_TOKENS, "rows"));
  DMUON_TRY(check_range(s->dim, 1, DMUON_MAX_DIM, "dim"));
  if (!(std::isfinite(s->eps) && s->eps >= 0.0f)) return invalid("eps must be finite and >= 0");
  if (!std::isfinite(s->residual_scale) || !std::isfinite(s->weight_offset))
    return invalid("residual_scale and weight_offset must be finite");
  return DMUON_OK;
}

// Blocks of the backward pass, each leaving one row of sums: as many as are at
// work at once, and, since a row of sums is moved twice, four runs of rows each
// where that leaves a block a CU (fp32, in calls from Python: 1024 x 4096 27 us,
// without that 33; 2048 x 1024 26, 29; 8192 x 512 27, 29; 777 x 1001 26 either way,
// of which the kernels take 17).  Wide rows: blocks of the pass over columns.
int bn_grad_blocks(const dmuon_block_norm_shape& s) {
  if (s.dim > kBnMaxFused) {
    const int64_t per = std::max<int64_t>(64, (s.rows + 4095) / 4096);
    return static_cast<int>((s.rows + per - 1) / per);
  }
  const int64_t once = bn_rows_at_once(s.dim), most = s.dim <= 512 ? 1024 : s.dim <= 1024 ? 2048 : s.dim <= 2048 ? 1024 : 512;
  const int64_t runs = (s.rows + once - 1) / once;
  return static_cast<int>(std::min<int64_t>(runs, std::min<int64_t>(most, std::max<int64_t>(256, runs / 4))));
}

struct BnLayout { size_t part, total; };
BnLayout bn_layout(const dmuon_block_norm_shape& s) {
  BnLayout l{};
  l.part = s.dim > kBnMaxFused ? align_up(sizeof(float) * 3 * s.rows) : 0;   // the stats come first
  l.total = l.part + align_up(sizeof(float) * 2 * s.dim * bn_grad_blocks(s));
  return l;
}

void fill_bn(const dmuon_block_norm_shape& s, const void* pre, const void* post, const void* gate, BlockNormArgs* a) {
  a->rows = s.rows;
  a->dim = static_cast<int>(s.dim);
  a->post_norm = s.post_norm ? 1 : 0;
  a->w_bf16 = s.weight_dtype == DMUON_BF16;
  a->eps = s.eps;
  a->scale = s.residual_scale;
  a->offset = s.weight_offset;
  a->w[0] = pre;
  a->w[1] = post;
  a->w[2] = gate;
}

// ---------------------------------------------------------------- attention
int check_attn(const dmuon_attention_shape* s) {
  if (!s) return invalid("shape is NULL");
  DMUON_TRY(check_float(s->dtype, "dtype"));
  DMUON_TRY(check_range(s->q_tokens, 0, DMUON_MAX_TOKENS, "q_tokens"));
  DMUON_TRY(check_range(s->k_tokens, 0, DMUON_MAX_TOKENS, "k_tokens"));
  DMUON_TRY(check_range(s->sequences, 1, DMUON_MAX_TOKENS, "sequences"));
  DMUON_TRY(check_range(s->q_heads, 1, DMUON_MAX_HEADS, "q_heads"));
  DMUON_TRY(check_range(s->k_heads, 1, DMUON_MAX_HEADS, "k_heads"));
  if (s->q_heads % s->k_heads) return invalid("q_heads must be a multiple of k_heads");
  DMUON_TRY(check_range(s->head_dim, 1, DMUON_MAX_ATTENTION_DIM, "head_dim"));
  DMUON_TRY(check_range(s->window, 0, int64_t{1} << 30, "window"));
  if (s->window && !s->causal) return invalid("a window needs causal");
  // the kernels' exponentials are base 2
  if (!(std::isfinite(s->scale * 1.4426950408889634f) && s->scale > 0.0f)) return invalid("scale times log2(e) must be finite and > 0");
  return check_range(s->q_tokens * (s->q_heads / s->k_heads), 0, int64_t{1} << 30, "q_tokens * q_heads / k_heads");
}

// Blocks of a launch stay below the limit of its grid.
int64_t attn_q_slots(const dmuon_attention_shape& s) {
  return attn_slots(s.q_tokens * (s.q_heads / s.k_heads), s.sequences);
}
int check_attn_grid(const dmuon_attention_shape& s) {
  const int64_t slots = std::max(attn_q_slots(s), attn_slots(s.k_tokens, s.sequences));
  return check_range(slots * s.k_heads, 0, (int64_t{1} << 24) - 1, "tiles (tokens / 128 + sequences, times k_heads)");
}

// Parts of a tile's keys: where the tiles alone leave CUs idle and the
// sequences have keys to share out, at least 512 a part.  In us, in slices and
// not: a token over 1024 keys 19, 26; 8 over 16384 21, 49; 8 over 65536 49, 179;
// 31 over 126976 28, 92; 2048 queries on 2048 keys 33, 55; 512 on 512 14 either way.
// The keys are shared out by their mean: a sequence far longer than the others is
// cut no finer than they are.
// No more sequences than there are queries have any; the others, such as the room
// behind a growing cache, have places for tiles and leave them at once (a token of
// 16 sequences over 4096 keys each, as many again as room: 53; counted as sequences
// with queries 92; without room 48).  Both kinds take workspace, which 2048 parts bound.
int attn_slices(const dmuon_attention_shape& s) {
  const int64_t active = std::max<int64_t>(1, std::min(s.sequences, s.q_tokens)), all = attn_q_slots(s) * s.k_heads;
  const int64_t tiles = attn_slots(s.q_tokens * (s.q_heads / s.k_heads), active) * s.k_heads, keys = s.k_tokens / active;
  if (tiles >= 256 || keys < 1024) return 1;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({1024 / tiles, 2048 / all, keys / 512, 64})));
}
int64_t attn_part_bytes(const dmuon_attention_shape& s) {
  const int64_t slices = attn_slices(s);
  if (slices <= 1) return 0;
  return attn_q_slots(s) * s.k_heads * slices * kAttnTile * (attn_padded(s.head_dim) + 2) * int64_t{4};
}

// Two numbers a row.
size_t attn_stat_bytes(const dmuon_attention_shape& s) {
  return align_up(2 * sizeof(float) * static_cast<size_t>(s.q_tokens) * s.q_heads);
}

int head_buf(const dmuon_attention_shape& s, const char* name, const void* p, int64_t tokens, int64_t heads,
             int64_t stride, bool written, Buf* out) {
  return row_buf(name, p, tokens, heads * s.head_dim, stride, s.dtype, written, out);
}

// Every 16-byte run of every head lies at a multiple of 16 bytes, and a tile
// within 32 bits of offset.
bool attn_vec(const dmuon_attention_shape& s, std::initializer_list<const Buf*> bufs) {
  if (s.head_dim * size_of(s.dtype) % 16) return false;
  for (const Buf* b : bufs)
    if (!b->empty() && (!aligned(b->p, 16) || (b->rows > 1 && (b->pitch % 16 || b->pitch > (int64_t{1} << 23))))) return false;
  return true;
}

int check_offsets(const int32_t* q, const int32_t* k, int64_t sequences) {
  if (!q != !k) return invalid("q_offsets and k_offsets come together");
  if (!q && sequences != 1) return invalid("several sequences need offsets");
  return DMUON_OK;
}

void fill_attn(const dmuon_attention_shape& s, AttnArgs* a) {
  a->q_tokens = static_cast<int>(s.q_tokens);
  a->k_tokens = static_cast<int>(s.k_tokens);
  a->sequences = static_cast<int>(s.sequences);
  a->q_heads = s.q_heads;
  a->k_heads = s.k_heads;
  a->group = s.q_heads / s.k_heads;
  a->group_inv = static_cast<unsigned>(((uint64_t{1} << 32) + a->group - 1) / a->group);
  a->dim = s.head_dim;
  a->causal = s.causal ? 1 : 0;
  a->window = s.window;
  a->scale = s.scale;
  a->slots = static_cast<int>(attn_q_slots(s));
}

// What a call has to compute and move, with all sequences equally long: the offsets
// are the device's.  A sequence of lq queries and lk keys: the last query sees up to
// lk keys, each one before it one fewer, and none more than the window.
struct AttnWork { double pairs, query_elems, key_elems, seen_elems; };   // seen: of the keys that any query sees
AttnWork attn_work(const dmuon_attention_shape& s) {
  const double seqs = static_cast<double>(s.sequences), lq = s.q_tokens / seqs, lk = s.k_tokens / seqs;
  const double most = s.window ? std::min<double>(s.window, lk) : lk;
  auto sum = [&](double n) { return n <= most ? n * (n + 1.0) / 2.0 : most * (most + 1.0) / 2.0 + (n - most) * most; };   // of min(1..n, most)
  const double pairs = s.causal ? sum(lk) - sum(std::max(lk - lq, 0.0)) : lq * lk;
  const double seen = s.window ? std::min(lk, lq + s.window - 1.0) : lk;
  const double heads = static_cast<double>(s.k_heads) * s.head_dim;
  return AttnWork{seqs * pairs * s.q_heads, static_cast<double>(s.q_tokens) * s.q_heads * s.head_dim, s.k_tokens * heads, seqs * seen * heads};
}

// ---------------------------------------------------------------- gated feed-forward
int check_ffn(const dmuon_gated_ffn_shape* s) {
  if (!s) return invalid("shape is NULL");
  DMUON_TRY(check_float(s->dtype, "dtype"));
  DMUON_TRY(check_range(s->tokens, 0, DMUON_MAX_TOKENS, "tokens"));
  DMUON_TRY(check_range(s->dim, 1, DMUON_MAX_DIM, "dim"));
  DMUON_TRY(check_range(s->hidden, 1, DMUON_MAX_DIM, "hidden"));
  return check_range(s->activation, DMUON_ACT_SILU, DMUON_ACT_GELU, "activation");
}

// Threads of a launch fit 32 bits: 512 to a 256 x 256 tile of bf16, 256 to a 64 x 64
// one of fp32 (of the hidden width half of that, twice).
int check_ffn_grid(const dmuon_gated_ffn_shape& s, bool back) {
  const int64_t tile = s.dtype == DMUON_BF16 ? 256 : 64, most = s.dtype == DMUON_BF16 ? int64_t{1} << 23 : int64_t{1} << 24;
  auto up = [](int64_t v, int64_t t) { return v / t + 1; };
  const int64_t rows = up(s.tokens, tile), gated = rows * up(s.hidden, tile / 2), dx = back ? rows * up(s.dim, tile) : 0;
  return check_range(std::max(gated, dx), 0, most - 1, "tiles (tokens times hidden or dim)");
}

int64_t whole_stages(int64_t v) { return (v + kFfnStage - 1) / kFfnStage * kFfnStage; }

void fill_ffn(const dmuon_gated_ffn_shape& s, FfnArgs* a) {
  a->n = s.tokens;
  a->mid_rows = whole_stages(s.tokens);
  a->dim = static_cast<int>(s.dim);
  a->kdim = static_cast<int>(s.dtype == DMUON_BF16 ? whole_stages(s.dim) : s.dim);
  a->hidden = static_cast<int>(s.hidden);
  a->hp = static_cast<int>(whole_stages(s.hidden));
  a->act = s.activation;
  a->ws = s.dim;
}

// The projections' gradients and the slices' sums (backward), and padded copies
// of the operands.  dx is done with its slices before the weights' begin.
struct FfnLayout { size_t off_part, off_x, off_g, off_u, total; bool copies; };
FfnLayout ffn_layout(const dmuon_gated_ffn_shape& s, bool back, bool in_place) {
  FfnLayout l{};
  const int64_t es = size_of(s.dtype);
  FfnArgs a{};
  fill_ffn(s, &a);
  if (back) {
    l.off_part = align_up(static_cast<size_t>(a.mid_rows * 2 * a.hp * es));
    ffn_slices(s.dtype, &a);
    const int64_t dx = a.dx_slices > 1 ? a.dx_slices * s.tokens : 0, dw = a.dw_slices > 1 ? a.dw_slices * 2 * s.hidden : 0;
    l.total = l.off_part + align_up(static_cast<size_t>(std::max(dx, dw) * ((s.dim + 3) / 4 * 4) * int64_t{4}));
  }
  l.copies = s.dtype == DMUON_BF16 && !(in_place && s.dim % kFfnStage == 0) && (back || !ffn_few(s.dtype, s.tokens, s.dim, s.hidden));
  if (l.copies) {
    l.off_x = l.total;
    l.off_g = l.off_x + align_up(static_cast<size_t>(s.tokens * a.kdim * es));
    l.off_u = l.off_g + align_up(static_cast<size_t>(s.hidden * a.kdim * es));
    l.total = l.off_u + align_up(static_cast<size_t>(s.hidden * a.kdim * es));
  }
  return l;
}

bool ffn_vec(std::initializer_list<const Buf*> bufs) {
  for (const Buf* b : bufs)
    if (!b->empty() && (!aligned(b->p, 16) || (b->rows > 1 && b->pitch % 16))) return false;
  return true;
}
// The bf16 tiles read the operands in place when their rows are whole stages at
// multiples of 16 bytes, and 256 of them lie within 32 bits of offset.  Copies
// of all three add 0.09 ms to 8192 tokens' 1.50 ms at 4096 -> 14336.
bool ffn_in_place(const Buf& x, const Buf& wg, const Buf& wu) {
  return ffn_vec({&x, &wg, &wu}) && (x.rows <= 1 || x.pitch <= (int64_t{1} << 23));
}

// Sets the operands of the tile kernels, behind copies where they cannot be read in place.
hipError_t ffn_operands(const dmuon_gated_ffn_shape& s, const FfnLayout& l, void* workspace, FfnArgs* a, hipStream_t stream) {
  if (!l.copies) return hipSuccess;
  char* ws = static_cast<char*>(workspace);
  const int dim = static_cast<int>(s.dim);
  hipError_t e = launch_ffn_pad(a->x, a->xs, ws + l.off_x, s.tokens, dim, a->kdim, stream);
  if (e == hipSuccess) e = launch_ffn_pad(a->wg, s.dim, ws + l.off_g, s.hidden, dim, a->kdim, stream);
  if (e == hipSuccess) e = launch_ffn_pad(a->wu, s.dim, ws + l.off_u, s.hidden, dim, a->kdim, stream);
  a->x = ws + l.off_x;
  a->wg = ws + l.off_g;
  a->wu = ws + l.off_u;
  a->xs = a->ws = a->kdim;
  return e;
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" {

int dmuon_block_norm_forward(const dmuon_block_norm_shape* shape, const void* x, int64_t x_stride, const void* h,
                             int64_t h_stride, const void* pre, const void* post, const void* gate, void* x_out,
                             int64_t x_out_stride, void* y, int64_t y_stride, void* hip_stream) {
  return guarded([&]() -> int {
    DMUON_TRY(check_bn(shape));
    const dmuon_block_norm_shape& s = *shape;
    if (post && !s.post_norm) return invalid("post is given without post_norm");
    const int64_t ws = size_of(s.weight_dtype);
    Buf b[7];
    DMUON_TRY(row_buf("x", x, s.rows, s.dim, x_stride, s.dtype, false, &b[0]));
    DMUON_TRY(row_buf("h", h, s.rows, s.dim, h_stride, s.branch_dtype, false, &b[1]));
    DMUON_TRY(row_buf("x_out", x_out, s.rows, s.dim, x_out_stride, s.dtype, true, &b[2]));
    DMUON_TRY(row_buf("y", y, s.rows, s.dim, y_stride, s.branch_dtype, true, &b[3]));
    b[4] = flat("pre", pre, pre ? s.dim * ws : 0, ws, false);
    b[5] = flat("post", post, post ? s.dim * ws : 0, ws, false);
    b[6] = flat("gate", gate, gate ? s.dim * ws : 0, ws, false);
    const int in_place[2][2] = {{0, 2}, {1, 3}};
    DMUON_TRY(check_bufs(b, 7, in_place, 2));
    bool capturing = false;
    DMUON_TRY(check_device(hip_stream, &capturing));
    if (s.rows == 0) return DMUON_OK;
    BlockNormArgs a{};
    fill_bn(s, pre, post, gate, &a);
    a.x = x;
    a.h = h;
    a.x_out = x_out;
    a.in_place = x_out == x;
    a.y = y;
    a.xs = x_stride;
    a.hs = h_stride;
    a.xos = x_out_stride;
    a.ys = y_stride;
    const double elems = static_cast<double>(s.rows) * s.dim;
    return launched("block norm", kKBlockNorm, 10.0 * elems, 2.0 * elems * (size_of(s.dtype) + size_of(s.branch_dtype)),
                    hip_stream, capturing, [&] {
                      return launch_block_norm(s.dtype, s.branch_dtype, a, static_cast<hipStream_t>(hip_stream));
                    });
  });
}

int dmuon_block_norm_backward_workspace_bytes(const dmuon_block_norm_shape* shape, size_t* bytes_out) {
  return guarded([&]() -> int {
    if (!bytes_out) return invalid("bytes_out is NULL");
    DMUON_TRY(check_bn(shape));
    *bytes_out = bn_layout(*shape).total;
    return DMUON_OK;
  });
}

int dmuon_block_norm_backward(const dmuon_block_norm_shape* shape, const void* dx_out, int64_t dx_out_stride,
                              const void* dy, int64_t dy_stride, const void* x_out, int64_t x_out_stride,
                              const void* h, int64_t h_stride, const void* pre, const void* post, const void* gate,
                              void* dx, int64_t dx_stride, void* dh, int64_t dh_stride, void* dpre, void* dpost,
                              void* dgate, void* workspace, size_t workspace_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    DMUON_TRY(check_bn(shape));
    const dmuon_block_norm_shape& s = *shape;
    if ((post || dpost) && !s.post_norm) return invalid("post or dpost is given without post_norm");
    const BnLayout l = bn_layout(s);
    const size_t need = dpre || dpost || dgate ? l.total : 0;   // no sums over rows are asked for
    DMUON_TRY(check_workspace(workspace, workspace_bytes, need));
    const int64_t ws = size_of(s.weight_dtype);
    Buf b[13];
    DMUON_TRY(row_buf("dx_out", dx_out, dx_out ? s.rows : 0, s.dim, dx_out_stride, s.dtype, false, &b[0]));
    DMUON_TRY(row_buf("dy", dy, s.rows, s.dim, dy_stride, s.branch_dtype, false, &b[1]));
    DMUON_TRY(row_buf("x_out", x_out, s.rows, s.dim, x_out_stride, s.dtype, false, &b[2]));
    DMUON_TRY(row_buf("h", h, s.rows, s.dim, h_stride, s.branch_dtype, false, &b[3]));
    DMUON_TRY(row_buf("dx", dx, s.rows, s.dim, dx_stride, s.dtype, true, &b[4]));
    DMUON_TRY(row_buf("dh", dh, s.rows, s.dim, dh_stride, s.branch_dtype, true, &b[5]));
    b[6] = flat("pre", pre, pre ? s.dim * ws : 0, ws, false);
    b[7] = flat("post", post, post ? s.dim * ws : 0, ws, false);
    b[8] = flat("gate", gate, gate ? s.dim * ws : 0, ws, false);
    b[9] = flat("dpre", dpre, dpre ? s.dim * ws : 0, ws, true);
    b[10] = flat("dpost", dpost, dpost ? s.dim * ws : 0, ws, true);
    b[11] = flat("dgate", dgate, dgate ? s.dim * ws : 0, ws, true);
    b[12] = flat("workspace", workspace, static_cast<int64_t>(need), 1, true);
    const int in_place[1][2] = {{0, 4}};
    DMUON_TRY(check_bufs(b, 13, in_place, 1));
    bool capturing = false;
    DMUON_TRY(check_device(hip_stream, &capturing));
    BlockNormArgs a{};
    fill_bn(s, pre, post, gate, &a);
    a.x = x_out;
    a.h = h;
    a.dx_out = dx_out;
    a.dy = dy;
    a.x_out = dx;
    a.in_place = dx == dx_out;
    a.y = dh;
    a.xs = x_out_stride;
    a.hs = h_stride;
    a.dxs = dx_out_stride;
    a.dys = dy_stride;
    a.xos = dx_stride;
    a.ys = dh_stride;
    a.dw[0] = dpre;
    a.dw[1] = dpost;
    a.dw[2] = dgate;
    a.blocks = bn_grad_blocks(s);
    a.col_rows = std::max<int64_t>(64, (s.rows + 4095) / 4096);
    a.stats = static_cast<float*>(workspace);
    a.part = need ? reinterpret_cast<float*>(static_cast<char*>(workspace) + l.part) : nullptr;
    const double elems = static_cast<double>(s.rows) * s.dim;
    return launched("block norm gradient", kKBlockNormGrad, 24.0 * elems,
                    elems * ((dx_out ? 3.0 : 2.0) * size_of(s.dtype) + 3.0 * size_of(s.branch_dtype)), hip_stream,
                    capturing, [&] {
                      return launch_block_norm_grad(s.dtype, s.branch_dtype, a, static_cast<hipStream_t>(hip_stream));
                    });
  });
}

int dmuon_attention_workspace_bytes(const dmuon_attention_shape* shape, size_t* bytes_out) {
  return guarded([&]() -> int {
    if (!bytes_out) return invalid("bytes_out is NULL");
    DMUON_TRY(check_attn(shape));
    *bytes_out = align_up(static_cast<size_t>(attn_part_bytes(*shape)));
    return DMUON_OK;
  });
}

int dmuon_attention_forward(const dmuon_attention_shape* shape, const void* q, int64_t q_stride, const void* k,
                            int64_t k_stride, const void* v, int64_t v_stride, const int32_t* q_offsets,
                            const int32_t* k_offsets, void* out, int64_t out_stride, float* lse, void* workspace,
                            size_t workspace_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    DMUON_TRY(check_attn(shape));
    const dmuon_attention_shape& s = *shape;
    DMUON_TRY(check_attn_grid(s));
    DMUON_TRY(check_offsets(q_offsets, k_offsets, s.sequences));
    const int64_t part = attn_part_bytes(s);
    DMUON_TRY(check_workspace(workspace, workspace_bytes, align_up(static_cast<size_t>(part))));
    Buf b[8];
    DMUON_TRY(head_buf(s, "q", q, s.q_tokens, s.q_heads, q_stride, false, &b[0]));
    DMUON_TRY(head_buf(s, "k", k, s.k_tokens, s.k_heads, k_stride, false, &b[1]));
    DMUON_TRY(head_buf(s, "v", v, s.k_tokens, s.k_heads, v_stride, false, &b[2]));
    DMUON_TRY(head_buf(s, "out", out, s.q_tokens, s.q_heads, out_stride, true, &b[3]));
    b[4] = flat("lse", lse, s.q_tokens * s.q_heads * 4, 4, true);
    b[5] = flat("q_offsets", q_offsets, q_offsets ? (s.sequences + 1) * 4 : 0, 4, false);
    b[6] = flat("k_offsets", k_offsets, k_offsets ? (s.sequences + 1) * 4 : 0, 4, false);
    b[7] = flat("workspace", workspace, part, 1, true);
    DMUON_TRY(check_bufs(b, 8));
    bool capturing = false;
    DMUON_TRY(check_device(hip_stream, &capturing));
    if (s.q_tokens == 0) return DMUON_OK;
    AttnArgs a{};
    fill_attn(s, &a);
    a.q = q;
    a.k = k;
    a.v = v;
    a.o = out;
    a.lse = lse;
    a.q_off = q_offsets;
    a.k_off = k_offsets;
    a.qs = q_stride;
    a.ks = k_stride;
    a.vs = v_stride;
    a.os = out_stride;
    a.part = static_cast<float*>(workspace);
    a.slices = attn_slices(s);
    a.vec = attn_vec(s, {&b[0], &b[1], &b[2], &b[3]});
    const AttnWork w = attn_work(s);
    return launched("attention", kKAttention, 4.0 * w.pairs * s.head_dim, 2.0 * (w.query_elems + w.seen_elems) * size_of(s.dtype),
                    hip_stream, capturing,
                    [&] { return launch_attention(s.dtype, a, static_cast<hipStream_t>(hip_stream)); });
  });
}

int dmuon_attention_backward_workspace_bytes(const dmuon_attention_shape* shape, size_t* bytes_out) {
  return guarded([&]() -> int {
    if (!bytes_out) return invalid("bytes_out is NULL");
    DMUON_TRY(check_attn(shape));
    *bytes_out = attn_stat_bytes(*shape);
    return DMUON_OK;
  });
}

int dmuon_attention_backward(const dmuon_attention_shape* shape, const void* dout, int64_t dout_stride, const void* q,
                             int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             const void* out, int64_t out_stride, const float* lse, const int32_t* q_offsets,
                             const int32_t* k_offsets, void* dq, int64_t dq_stride, void* dk, int64_t dk_stride,
                             void* dv, int64_t dv_stride, void* workspace, size_t workspace_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    DMUON_TRY(check_attn(shape));
    const dmuon_attention_shape& s = *shape;
    DMUON_TRY(check_attn_grid(s));
    DMUON_TRY(check_offsets(q_offsets, k_offsets, s.sequences));
    const size_t need = attn_stat_bytes(s);
    DMUON_TRY(check_workspace(workspace, workspace_bytes, need));
    Buf b[12];
    DMUON_TRY(head_buf(s, "dout", dout, s.q_tokens, s.q_heads, dout_stride, false, &b[0]));
    DMUON_TRY(head_buf(s, "q", q, s.q_tokens, s.q_heads, q_stride, false, &b[1]));
    DMUON_TRY(head_buf(s, "k", k, s.k_tokens, s.k_heads, k_stride, false, &b[2]));
    DMUON_TRY(head_buf(s, "v", v, s.k_tokens, s.k_heads, v_stride, false, &b[3]));
    DMUON_TRY(head_buf(s, "out", out, s.q_tokens, s.q_heads, out_stride, false, &b[4]));
    DMUON_TRY(head_buf(s, "dq", dq, s.q_tokens, s.q_heads, dq_stride, true, &b[5]));
    DMUON_TRY(head_buf(s, "dk", dk, s.k_tokens, s.k_heads, dk_stride, true, &b[6]));
    DMUON_TRY(head_buf(s, "dv", dv, s.k_tokens, s.k_heads, dv_stride, true, &b[7]));
    b[8] = flat("lse", lse, s.q_tokens * s.q_heads * 4, 4, false);
    b[9] = flat("q_offsets", q_offsets, q_offsets ? (s.sequences + 1) * 4 : 0, 4, false);
    b[10] = flat("k_offsets", k_offsets, k_offsets ? (s.sequences + 1) * 4 : 0, 4, false);
    b[11] = flat("workspace", workspace, static_cast<int64_t>(need), 1, true);
    DMUON_TRY(check_bufs(b, 12));
    bool capturing = false;
    DMUON_TRY(check_device(hip_stream, &capturing));
    if (s.q_tokens == 0 && s.k_tokens == 0) return DMUON_OK;
    AttnArgs a{};
    fill_attn(s, &a);
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.dout = dout;
    a.lse = const_cast<float*>(lse);
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.q_off = q_offsets;
    a.k_off = k_offsets;
    a.qs = q_stride;
    a.ks = k_stride;
    a.vs = v_stride;
    a.os = out_stride;
    a.dos = dout_stride;
    a.dqs = dq_stride;
    a.dks = dk_stride;
    a.dvs = dv_stride;
    a.stats = static_cast<float*>(workspace);
    a.slices = 1;
    a.vec = attn_vec(s, {&b[0], &b[1], &b[2], &b[3], &b[4], &b[5], &b[6], &b[7]});
    const int k_slots = static_cast<int>(attn_slots(s.k_tokens, s.sequences));
    const AttnWork w = attn_work(s);
    return launched("attention gradient", kKAttentionGrad, 10.0 * w.pairs * s.head_dim,
                    (4.0 * w.query_elems + 2.0 * (w.seen_elems + w.key_elems)) * size_of(s.dtype), hip_stream, capturing,
                    [&] { return launch_attention_grad(s.dtype, a, k_slots, static_cast<hipStream_t>(hip_stream)); });
  });
}

int dmuon_gated_ffn_workspace_bytes(const dmuon_gated_ffn_shape* shape, int is_aligned, size_t* bytes_out) {
  return guarded([&]() -> int {
    if (!bytes_out) return invalid("bytes_out is NULL");
    DMUON_TRY(check_ffn(shape));
    *bytes_out = ffn_layout(*shape, false, is_aligned != 0).total;
    return DMUON_OK;
  });
}

int dmuon_gated_ffn_forward(const dmuon_gated_ffn_shape* shape, const void* x, int64_t x_stride, const void* w_gate,
                            const void* w_up, void* h, int64_t h_stride, void* workspace, size_t workspace_bytes,
                            void* hip_stream) {
  return guarded([&]() -> int {
    DMUON_TRY(check_ffn(shape));
    const dmuon_gated_ffn_shape& s = *shape;
    DMUON_TRY(check_ffn_grid(s, false));
    const int64_t es = size_of(s.dtype), wbytes = s.tokens ? s.hidden * s.dim * es : 0;
    Buf b[5];
    DMUON_TRY(row_buf("x", x, s.tokens, s.dim, x_stride, s.dtype, false, &b[0]));
    DMUON_TRY(row_buf("h", h, s.tokens, s.hidden, h_stride, s.dtype, true, &b[1]));
    b[2] = flat("w_gate", w_gate, wbytes, es, false);
    b[3] = flat("w_up", w_up, wbytes, es, false);
    const Buf wg{"w_gate", w_gate, s.hidden, s.dim * es, s.dim * es, es, false};
    const Buf wu{"w_up", w_up, s.hidden, s.dim * es, s.dim * es, es, false};
    const FfnLayout l = ffn_layout(s, false, ffn_in_place(b[0], wg, wu));
    DMUON_TRY(check_workspace(workspace, workspace_bytes, l.total));
    b[4] = flat("workspace", workspace, static_cast<int64_t>(l.total), 1, true);
    DMUON_TRY(check_bufs(b, 5));
    bool capturing = false;
    DMUON_TRY(check_device(hip_stream, &capturing));
    if (s.tokens == 0) return DMUON_OK;
    FfnArgs a{};
    fill_ffn(s, &a);
    a.x = x;
    a.xs = x_stride;
    a.wg = w_gate;
    a.wu = w_up;
    a.out = h;
    a.outs = h_stride;
    a.vec = ffn_vec({&b[0], &wg, &wu});
    const double flops = 4.0 * s.tokens * s.dim * s.hidden;
    const double bytes = static_cast<double>(es) * (s.tokens * (s.dim + s.hidden) + 2 * s.hidden * s.dim);
    hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    return launched("gated feed-forward", kKFfn, flops, bytes, hip_stream, capturing, [&] {
      if (ffn_few(s.dtype, s.tokens, s.dim, s.hidden)) return launch_ffn_few(s.dtype, a, stream);
      const hipError_t e = ffn_operands(s, l, workspace, &a, stream);
      return e != hipSuccess ? e : launch_ffn(s.dtype, kFfnOut, a, stream);
    });
  });
}

int dmuon_gated_ffn_backward_workspace_bytes(const dmuon_gated_ffn_shape* shape, int is_aligned, size_t* bytes_out) {
  return guarded([&]() -> int {
    if (!bytes_out) return invalid("bytes_out is NULL");
    DMUON_TRY(check_ffn(shape));
    *bytes_out = ffn_layout(*shape, true, is_aligned != 0).total;
    return DMUON_OK;
  });
}

int dmuon_gated_ffn_backward(const dmuon_gated_ffn_shape* shape, const void* dh, int64_t dh_stride, const void* x,
                             int64_t x_stride, const void* w_gate, const void* w_up, void* dx, int64_t dx_stride,
                             void* dw_gate, void* dw_up, void* workspace, size_t workspace_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    DMUON_TRY(check_ffn(shape));
    const dmuon_gated_ffn_shape& s = *shape;
    DMUON_TRY(check_ffn_grid(s, true));
    const int64_t es = size_of(s.dtype), wbytes = s.hidden * s.dim * es;
    Buf b[8];
    DMUON_TRY(row_buf("dh", dh, s.tokens, s.hidden, dh_stride, s.dtype, false, &b[0]));
    DMUON_TRY(row_buf("x", x, s.tokens, s.dim, x_stride, s.dtype, false, &b[1]));
    DMUON_TRY(row_buf("dx", dx, s.tokens, s.dim, dx_stride, s.dtype, true, &b[2]));
    b[3] = flat("w_gate", w_gate, s.tokens ? wbytes : 0, es, false);
    b[4] = flat("w_up", w_up, s.tokens ? wbytes : 0, es, false);
    b[5] = flat("dw_gate", dw_gate, wbytes, es, true);
    b[6] = flat("dw_up", dw_up, wbytes, es, true);
    const Buf wg{"w_gate", w_gate, s.hidden, s.dim * es, s.dim * es, es, false};
    const Buf wu{"w_up", w_up, s.hidden, s.dim * es, s.dim * es, es, false};
    const FfnLayout l = ffn_layout(s, true, ffn_in_place(b[1], wg, wu));
    DMUON_TRY(check_workspace(workspace, workspace_bytes, l.total));
    b[7] = flat("workspace", workspace, static_cast<int64_t>(l.total), 1, true);
    DMUON_TRY(check_bufs(b, 8));
    bool capturing = false;
    DMUON_TRY(check_device(hip_stream, &capturing));
    FfnArgs a{};
    fill_ffn(s, &a);
    a.x = x;
    a.xs = x_stride;
    a.wg = w_gate;
    a.wu = w_up;
    a.dh = dh;
    a.dhs = dh_stride;
    a.out = dx;
    a.outs = dx_stride;
    a.dwg = dw_gate;
    a.dwu = dw_up;
    a.mid = workspace;
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + l.off_part);
    ffn_slices(s.dtype, &a);
    a.vec = ffn_vec({&b[1], &wg, &wu});
    const double flops = 12.0 * s.tokens * s.dim * s.hidden;
    const double bytes = static_cast<double>(es) * (s.tokens * (2 * s.dim + s.hidden) + 4 * s.hidden * s.dim);
    hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    return launched("gated feed-forward gradient", kKFfnGrad, flops, bytes, hip_stream, capturing, [&] {
      hipError_t e = hipSuccess;
      if (s.tokens > 0) {
        e = ffn_operands(s, l, workspace, &a, stream);
        if (e == hipSuccess) e = launch_ffn(s.dtype, kFfnMid, a, stream);
        if (e == hipSuccess) e = launch_ffn(s.dtype, kFfnDx, a, stream);
      }
      return e != hipSuccess ? e : launch_ffn(s.dtype, kFfnDw, a, stream);
    });
  });
}

}  // extern "C"
