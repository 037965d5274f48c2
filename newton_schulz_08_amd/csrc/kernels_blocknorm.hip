// The norms around a block with its gate and residual scale, in one pass, and
// their gradients, on gfx950 (HBM-bound).
//
// For every row, with the block's output h, the residual stream x, the gains
// (offset + w) of both norms, a gate per column and the residual scale s:
//
//   b  = h rh (offset + w_post)      rh = 1 / sqrt(mean(h^2) + eps)   (or b = h)
//   x' = x + s gate b
//   y  = x' rx (offset + w_pre)      rx = 1 / sqrt(mean(x'^2) + eps)
//
// y reads x' as it was stored.  With t the whole gradient of x':
//
//   t   = dx' + rx (dy g_pre - xh mean(dy g_pre xh)),   xh = x' rx
//   dx  = t,   db = s gate t
//   dh  = rh (db g_post - hh mean(db g_post hh)),       hh = h rh
//   dw_pre = sum dy xh,  dw_post = sum s gate t hh,  dgate = sum s t g_post hh
//
// A row is held in registers by one wave (up to 1024 elements), by four, or by
// sixteen, in runs of eight elements, so every tensor moves once.  The
// backward pass strides over the rows and keeps its columns' three sums beside
// the row; each block leaves one row of sums for a second launch that adds
// them in a fixed order.  Rows beyond 8192 elements leave no registers for the
// sums (24 a run of eight): a first pass over the rows then stores both
// reciprocal lengths and the mean, a pass over columns forms the sums, and a
// second pass over the rows the gradients.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "block.hpp"

namespace dmuon {
namespace {

// Eight consecutive elements as they lie in memory; `dim` bounds the last run.
template <int DT> struct Run {
  using T = typename OpElem<DT>::T;
  typedef T V __attribute__((ext_vector_type(8)));
  V v;
  __device__ __forceinline__ void load(const T* row, int e, int dim) {
    if (e + 8 <= dim) {
      constexpr int M = 16 / sizeof(T);
      using L = typename Loose<T, M>::V;
#pragma unroll
      for (int k = 0; k < 8 / M; ++k) {
        const L x = *reinterpret_cast<gptr<const L>>(gmem(row + e + M * k));
#pragma unroll
        for (int i = 0; i < M; ++i) v[M * k + i] = x[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = e + i < dim ? gmem(row)[e + i] : static_cast<T>(0.0f);
    }
  }
  __device__ __forceinline__ float operator[](int i) const { return static_cast<float>(v[i]); }
};
template <typename T> __device__ __forceinline__ void put(T* row, int e, int dim, const float* v) {
  if (e + 8 <= dim) {
    store_any<8>(row + e, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i < dim) gmem(row)[e + i] = static_cast<T>(v[i]);
  }
}
__device__ __forceinline__ void gain(const void* w, int bf16, float offset, int e, int dim, float* g) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    g[i] = 1.0f;
    if (w && e + i < dim)
      g[i] = offset + (bf16 ? static_cast<float>(gmem(static_cast<const __bf16*>(w))[e + i])
                            : gmem(static_cast<const float*>(w))[e + i]);
  }
}

// Sums of N values over the T threads of a row.  T > 64: through `red`, which
// holds two sets so that one barrier per sum is enough.
template <int T, int N> struct RowSum {
  float* red;   // 2 x (T / 64) x N
  int turn = 0;
  __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], o, 64);
    if constexpr (T > 64) {
      constexpr int kW = T / 64;
      float* at = red + turn * kW * N;
      turn ^= 1;
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) at[(threadIdx.x >> 6) * N + k] = v[k];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < N; ++k) {
        float s = at[k];
#pragma unroll
        for (int w = 1; w < kW; ++w) s += at[w * N + k];
        v[k] = s;
      }
    }
  }
};

// T threads a row, C runs of eight a thread.
template <int XDT, int BDT, int T, int C>
__global__ __launch_bounds__(T > 256 ? T : 256) void block_norm_kernel(BlockNormArgs a) {
  using X = typename OpElem<XDT>::T;
  using B = typename OpElem<BDT>::T;
  constexpr int kRows = T == 64 ? 4 : 1;
  __shared__ float red[2 * (T / 64) * 1];
  const int t = threadIdx.x % T;
  const float inv = 1.0f / static_cast<float>(a.dim);
  float gpre[C][8], gb[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = (c * T + t) * 8;
    float gate[8];
    gain(a.w[0], a.w_bf16, a.offset, e, a.dim, gpre[c]);
    gain(a.w[1], a.w_bf16, a.offset, e, a.dim, gb[c]);
    gain(a.w[2], a.w_bf16, 0.0f, e, a.dim, gate);
#pragma unroll
    for (int i = 0; i < 8; ++i) gb[c][i] *= gate[i] * a.scale;
  }
  RowSum<T, 1> sum{red};
  const X* x = static_cast<const X*>(a.x);
  const B* h = static_cast<const B*>(a.h);
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + (T == 64 ? threadIdx.x >> 6 : 0);
  Run<XDT> nx[C];
  Run<BDT> nh[C];
  auto ahead = [&](int64_t r) {
    if (r < a.rows)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        nx[c].load(x + r * a.xs, (c * T + t) * 8, a.dim);
        nh[c].load(h + r * a.hs, (c * T + t) * 8, a.dim);
      }
  };
  ahead(row);
  for (; row < a.rows; row += static_cast<int64_t>(gridDim.x) * kRows) {
    float v[C][8], b[C][8];
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][i] = nx[c][i];
        b[c][i] = nh[c][i];
        s[0] += b[c][i] * b[c][i];
      }
    ahead(row + static_cast<int64_t>(gridDim.x) * kRows);
    float rh = 1.0f;
    if (a.post_norm) {
      sum(s);
      rh = 1.0f / sqrtf(s[0] * inv + a.eps);
    }
    s[0] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // rounded as it is stored
        v[c][i] = static_cast<float>(static_cast<X>(fmaf(b[c][i] * rh, gb[c][i], v[c][i])));
        s[0] += v[c][i] * v[c][i];
      }
      put(static_cast<X*>(a.x_out) + row * a.xos, (c * T + t) * 8, a.dim, v[c]);
    }
    sum(s);
    const float rx = 1.0f / sqrtf(s[0] * inv + a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * rx * gpre[c][i];
      put(static_cast<B*>(a.y) + row * a.ys, (c * T + t) * 8, a.dim, v[c]);
    }
  }
}

// SUMS: the gains' and the gate's sums stay in registers.  Else they are
// bn_columns_kernel's, and a launch with stats_only leaves it each row's
// reciprocal lengths and mean.
template <int XDT, int BDT, int T, int C, bool SUMS>
__global__ __launch_bounds__(T > 256 ? T : 256) void block_norm_grad_kernel(BlockNormArgs a) {
  using X = typename OpElem<XDT>::T;
  using B = typename OpElem<BDT>::T;
  constexpr int kRows = T == 64 ? 4 : 1;
  __shared__ float red3[2 * (T / 64) * 3], red1[2 * (T / 64)];
  __shared__ float join[T == 64 ? 4 * 64 * C * 8 : 1];
  const int t = threadIdx.x % T;
  const float inv = 1.0f / static_cast<float>(a.dim);
  float acc[SUMS ? 3 : 1][C][8] = {};
  RowSum<T, 3> sum3{red3};
  RowSum<T, 1> sum1{red1};
  const X* x = static_cast<const X*>(a.x);
  const X* dx = static_cast<const X*>(a.dx_out);
  const B* h = static_cast<const B*>(a.h);
  const B* dy = static_cast<const B*>(a.dy);
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + (T == 64 ? threadIdx.x >> 6 : 0);
  for (; row < a.rows; row += static_cast<int64_t>(gridDim.x) * kRows) {
    Run<XDT> rx_[C], rd[C];
    Run<BDT> rh_[C], ry[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = (c * T + t) * 8;
      rx_[c].load(x + row * a.xs, e, a.dim);
      ry[c].load(dy + row * a.dys, e, a.dim);
      rh_[c].load(h + row * a.hs, e, a.dim);
      if (dx) rd[c].load(dx + row * a.dxs, e, a.dim);
    }
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float g[8];
      gain(a.w[0], a.w_bf16, a.offset, (c * T + t) * 8, a.dim, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[0] += rx_[c][i] * rx_[c][i];
        s[1] += ry[c][i] * g[i] * rx_[c][i];
        s[2] += rh_[c][i] * rh_[c][i];
      }
    }
    sum3(s);
    const float rx = 1.0f / sqrtf(s[0] * inv + a.eps);
    const float rh = a.post_norm ? 1.0f / sqrtf(s[2] * inv + a.eps) : 1.0f;
    const float along = s[1] * rx * inv;   // mean(dy g xh)
    if (!SUMS && a.stats_only) {
      if (t == 0) {
        gmem(a.stats)[3 * row] = rx;
        gmem(a.stats)[3 * row + 1] = rh;
        gmem(a.stats)[3 * row + 2] = along;
      }
      continue;
    }
    float d[C][8];
    float u[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = (c * T + t) * 8;
      float gpre[8], gpost[8], gate[8];
      gain(a.w[0], a.w_bf16, a.offset, e, a.dim, gpre);
      gain(a.w[1], a.w_bf16, a.offset, e, a.dim, gpost);
      gain(a.w[2], a.w_bf16, 0.0f, e, a.dim, gate);
      float out[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = rx_[c][i] * rx, hh = rh_[c][i] * rh;
        const float tt = rx * (ry[c][i] * gpre[i] - xh * along) + (dx ? rd[c][i] : 0.0f);
        out[i] = tt;
        const float st = a.scale * tt, db = st * gate[i];
        if constexpr (SUMS) {
          acc[0][c][i] += ry[c][i] * xh;
          acc[1][c][i] += db * hh;
          acc[2][c][i] += st * gpost[i] * hh;
        }
        d[c][i] = db * gpost[i];
        u[0] += d[c][i] * hh;
      }
      put(static_cast<X*>(a.x_out) + row * a.xos, e, a.dim, out);
    }
    float mean = 0.0f;
    if (a.post_norm) {
      sum1(u);
      mean = u[0] * inv;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (a.post_norm)
#pragma unroll
        for (int i = 0; i < 8; ++i) d[c][i] = rh * (d[c][i] - rh_[c][i] * rh * mean);
      put(static_cast<B*>(a.y) + row * a.ys, (c * T + t) * 8, a.dim, d[c]);
    }
  }
  if constexpr (SUMS) {
    if (!a.part) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      float* out = a.part + (static_cast<int64_t>(blockIdx.x) * 3 + k) * a.dim;
      if constexpr (T == 64) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) join[((threadIdx.x >> 6) * 64 * C + c * 64 + t) * 8 + i] = acc[k][c][i];
        __syncthreads();
        for (int e = threadIdx.x; e < a.dim; e += 256) {
          float v = 0.0f;
#pragma unroll
          for (int w = 0; w < 4; ++w) v += join[w * 64 * C * 8 + e];
          gmem(out)[e] = v;
        }
      } else {
#pragma unroll
        for (int c = 0; c < C; ++c) put(out, (c * T + t) * 8, a.dim, acc[k][c]);
      }
    }
  }
}

// Wide rows: sums of each thread's column over col_rows rows.
template <int XDT, int BDT>
__global__ __launch_bounds__(256) void bn_columns_kernel(BlockNormArgs a) {
  using X = typename OpElem<XDT>::T;
  using B = typename OpElem<BDT>::T;
  const int e = blockIdx.x * 256 + threadIdx.x;
  if (e >= a.dim) return;
  auto one = [&](const void* w, float offset) {
    if (!w) return 1.0f;
    return offset + (a.w_bf16 ? static_cast<float>(gmem(static_cast<const __bf16*>(w))[e])
                              : gmem(static_cast<const float*>(w))[e]);
  };
  const float gpre = one(a.w[0], a.offset), gpost = one(a.w[1], a.offset), gate = one(a.w[2], 0.0f);
  float acc[3] = {0.0f, 0.0f, 0.0f};
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * a.col_rows, r1 = least(r0 + a.col_rows, a.rows);
  for (int64_t r = r0; r < r1; ++r) {
    const float x = static_cast<float>(gmem(static_cast<const X*>(a.x))[r * a.xs + e]);
    const float h = static_cast<float>(gmem(static_cast<const B*>(a.h))[r * a.hs + e]);
    const float dy = static_cast<float>(gmem(static_cast<const B*>(a.dy))[r * a.dys + e]);
    const float dx = a.dx_out ? static_cast<float>(gmem(static_cast<const X*>(a.dx_out))[r * a.dxs + e]) : 0.0f;
    const float rx = gmem(a.stats)[3 * r], rh = gmem(a.stats)[3 * r + 1], along = gmem(a.stats)[3 * r + 2];
    const float t = rx * (dy * gpre - x * rx * along) + dx;   // unrounded, as the narrower rows sum it
    acc[0] += dy * (x * rx);
    acc[1] += a.scale * t * gate * (h * rh);
    acc[2] += a.scale * t * gpost * (h * rh);
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) gmem(a.part)[(static_cast<int64_t>(blockIdx.y) * 3 + k) * a.dim + e] = acc[k];
}

// Adds the blocks' rows of sums: 64 columns a block, 16 runs of rows, joined in order.
constexpr int kJoinRuns = 16;
__global__ __launch_bounds__(64 * kJoinRuns) void bn_join_kernel(BlockNormArgs a) {
  __shared__ float run[kJoinRuns][64];
  const int k = blockIdx.y, lane = threadIdx.x & 63, r = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  void* out = k == 0 ? a.dw[0] : k == 1 ? a.dw[1] : a.dw[2];
  if (!out) return;
  const int per = (a.blocks + kJoinRuns - 1) / kJoinRuns;
  float s = 0.0f;
  if (e < a.dim)
    for (int b = r * per; b < least((r + 1) * per, a.blocks); ++b)
      s += gmem(a.part)[(static_cast<int64_t>(b) * 3 + k) * a.dim + e];
  run[r][lane] = s;
  __syncthreads();
  if (r > 0 || e >= a.dim) return;
  for (int i = 1; i < kJoinRuns; ++i) s += run[i][lane];
  if (a.w_bf16) gmem(static_cast<__bf16*>(out))[e] = static_cast<__bf16>(s);
  else gmem(static_cast<float*>(out))[e] = s;
}

constexpr int kBnBlocks = 2048;   // blocks of the forward pass: eight a CU stride over the rows

template <int XDT, int BDT, int T, int C> void forward(const BlockNormArgs& a, hipStream_t stream) {
  const int64_t rows = T == 64 ? (a.rows + 3) / 4 : a.rows;
  block_norm_kernel<XDT, BDT, T, C>
      <<<dim3(static_cast<unsigned>(std::min<int64_t>(rows, kBnBlocks))), dim3(T > 256 ? T : 256), 0, stream>>>(a);
}
template <int XDT, int BDT> void forward_any(const BlockNormArgs& a, hipStream_t s) {
  const int d = a.dim;
  if (d <= 512) forward<XDT, BDT, 64, 1>(a, s);
  else if (d <= 1024) forward<XDT, BDT, 64, 2>(a, s);
  else if (d <= 2048) forward<XDT, BDT, 256, 1>(a, s);
  else if (d <= 4096) forward<XDT, BDT, 256, 2>(a, s);
  else if (d <= 8192) forward<XDT, BDT, 1024, 1>(a, s);
  else if (d <= 16384) forward<XDT, BDT, 1024, 2>(a, s);
  else if (d <= 32768) forward<XDT, BDT, 1024, 4>(a, s);
  else forward<XDT, BDT, 1024, 8>(a, s);
}
template <int XDT, int BDT, int T, int C, bool SUMS> void backward(const BlockNormArgs& a, int64_t blocks, hipStream_t s) {
  block_norm_grad_kernel<XDT, BDT, T, C, SUMS>
      <<<dim3(static_cast<unsigned>(blocks)), dim3(T > 256 ? T : 256), 0, s>>>(a);
}
template <int XDT, int BDT> void backward_any(const BlockNormArgs& a, hipStream_t s) {
  const int d = a.dim;
  if (d <= 512) backward<XDT, BDT, 64, 1, true>(a, a.blocks, s);
  else if (d <= 1024) backward<XDT, BDT, 64, 2, true>(a, a.blocks, s);
  else if (d <= 2048) backward<XDT, BDT, 256, 1, true>(a, a.blocks, s);
  else if (d <= 4096) backward<XDT, BDT, 256, 2, true>(a, a.blocks, s);
  else if (d <= 8192) backward<XDT, BDT, 1024, 1, true>(a, a.blocks, s);
  else {
    auto rows = [&](const BlockNormArgs& r) {
      const int64_t blocks = std::min<int64_t>(a.rows, 1024);
      if (d <= 16384) backward<XDT, BDT, 1024, 2, false>(r, blocks, s);
      else if (d <= 32768) backward<XDT, BDT, 1024, 4, false>(r, blocks, s);
      else backward<XDT, BDT, 1024, 8, false>(r, blocks, s);
    };
    if (a.part) {   // the sums first: dx may take dx_out's place
      BlockNormArgs r = a;
      r.stats_only = 1;
      rows(r);
      bn_columns_kernel<XDT, BDT><<<dim3((d + 255) / 256, static_cast<unsigned>(a.blocks)), dim3(256), 0, s>>>(a);
    }
    rows(a);
  }
}

}  // namespace

hipError_t launch_block_norm(int dt, int bdt, const BlockNormArgs& a, hipStream_t stream) {
  if (dt == kF32) bdt == kF32 ? forward_any<kF32, kF32>(a, stream) : forward_any<kF32, kBF16>(a, stream);
  else bdt == kF32 ? forward_any<kBF16, kF32>(a, stream) : forward_any<kBF16, kBF16>(a, stream);
  return hipGetLastError();
}

hipError_t launch_block_norm_grad(int dt, int bdt, const BlockNormArgs& a, hipStream_t stream) {
  if (a.rows > 0) {
    if (dt == kF32) bdt == kF32 ? backward_any<kF32, kF32>(a, stream) : backward_any<kF32, kBF16>(a, stream);
    else bdt == kF32 ? backward_any<kBF16, kF32>(a, stream) : backward_any<kBF16, kBF16>(a, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.dw[0] || a.dw[1] || a.dw[2])
    bn_join_kernel<<<dim3((a.dim + 63) / 64, 3), dim3(64 * kJoinRuns), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace dmuon
