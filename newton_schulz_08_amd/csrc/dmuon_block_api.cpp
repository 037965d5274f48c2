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

// Blocks of the backward pass, each leaving one row of sums: three a CU, and
// no more than there are runs of rows.  Wide rows: blocks of the pass over columns.
int bn_grad_blocks(const dmuon_block_norm_shape& s) {
  if (s.dim > kBnMaxFused) {
    const int64_t per = std::max<int64_t>(64, (s.rows + 4095) / 4096);
    return static_cast<int>((s.rows + per - 1) / per);
  }
  const int64_t once = bn_rows_at_once(s.dim);
  return static_cast<int>(std::min<int64_t>((s.rows + once - 1) / once, 768));
}

struct BnLayout { size_t part, total; };
BnLayout bn_layout(const dmuon_block_norm_shape& s) {
  BnLayout l{};
  l.part = s.dim > kBnMaxFused ? align_up(sizeof(float) * 3 * s.rows) : 0;   // the stats come first
  l.total = l.part + align_up(sizeof(float) * 3 * s.dim * bn_grad_blocks(s));
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

}  // extern "C"
