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
// A lane holds eight elements of a row, so that rows up to 8192 elements stay
// in the registers of one to sixteen waves and every tensor moves once; the
// next row's loads are under way while a row is reduced.  The backward pass
// strides over the rows and keeps two sums per column beside the row, since
//
//   dw_post = gate Q,  dgate = g_post Q,   Q = sum s t hh;
//
// each block leaves one row of them for a second launch that adds them in a
// fixed order.  Wider rows are swept several times, out of the caches, and
// their column sums are a launch of its own behind one that stores each row's
// lengths and mean.
//
// Measured, fp32 stream and bf16 branch: backward of 32768 x 4096 455 to 490 us and
// of 32768 x 8192 885, 5.0 to 5.5 TB/s of the bytes it cannot do without (a copy
// of 1 GiB moves 5.2); forward 308 and 615, 5.2.  bf16: backward 311 and 642 us,
// 5.2 and 5.0 TB/s, forward 211 and 410.  Forward of 16 x 4096 3.8 us, which is
// latency.  Two runs of eight a lane, and half the threads, take 852 us backward
// at 4096; loads behind branches 1247.  Rows over 8192 are swept: 8192 x 16384
// forward 412 us and backward 1255 (statistics 228, columns 285, rows 735) where
// the bytes would take 311 and 466; bf16 321 and 950.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "block.hpp"

namespace dmuon {
namespace {

// Eight consecutive elements as they lie in memory.  Every lane loads, from the
// row's last eight if its own reach behind them, and land() moves those into
// place with zeros behind the row: a branch around a load would make the next
// one wait for it.
template <int DT> struct Run {
  using T = typename OpElem<DT>::T;
  typedef T V __attribute__((ext_vector_type(8)));
  V v;
  __device__ __forceinline__ void load(const T* row, int e, int dim) {
    if (dim >= 8) {
      const T* p = row + (e < dim - 8 ? e : dim - 8);
      constexpr int M = 16 / sizeof(T);
      using L = typename Loose<T, M>::V;
#pragma unroll
      for (int k = 0; k < 8 / M; ++k) {
        const L x = *reinterpret_cast<gptr<const L>>(gmem(p + M * k));
#pragma unroll
        for (int i = 0; i < M; ++i) v[M * k + i] = x[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = gmem(row)[i < dim ? i : dim - 1];
    }
  }
  // The lane's own elements and no other's, landed: of a row that is being stored to.
  __device__ __forceinline__ void load_own(const T* row, int e, int dim) {
    if (e + 8 <= dim) {
      load(row, e, dim);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = e + i < dim ? gmem(row)[e + i] : static_cast<T>(0.0f);
    }
  }
  __device__ __forceinline__ void land(int e, int dim) {
    const T zero = static_cast<T>(0.0f);
    if (dim % 8 == 0) {
      if (e >= dim) v = V{};
    } else if (dim >= 8) {
      const int by = e - dim + 8;   // > 0: the elements lie that far up
      if (by >= 8) v = V{};
#pragma unroll
      for (int b = 4; b > 0; b >>= 1)
        if (by > 0 && (by & b))
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = i + b < 8 ? v[i + b < 8 ? i + b : 0] : zero;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = e + i < dim ? v[i] : zero;
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
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = 1.0f;
  } else if (bf16) {
    Run<kBF16> r;
    r.load(static_cast<const __bf16*>(w), e, dim);
    r.land(e, dim);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = offset + r[i];
  } else {
    Run<kF32> r;
    r.load(static_cast<const float*>(w), e, dim);
    r.land(e, dim);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = offset + r[i];
  }
}

__device__ __forceinline__ float one_gain(const void* w, int bf16, float offset, int e) {
  if (!w) return 1.0f;
  return offset + (bf16 ? static_cast<float>(gmem(static_cast<const __bf16*>(w))[e]) : gmem(static_cast<const float*>(w))[e]);
}
// v as it is stored in a tensor of T.
template <typename T> __device__ __forceinline__ float stored(float v) { return static_cast<float>(static_cast<T>(v)); }

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

// Rows of a block: four of one wave each, or one of T threads.
template <int T> constexpr int kRowsAtOnce = T == 64 ? 4 : 1;
template <int T> constexpr int kBlock = T == 64 ? 256 : T;

// In front of a store over what was loaded: the last lane's load reaches into
// the elements of the lane before it, which another wave may own.
template <int T> __device__ __forceinline__ void row_loaded(const BlockNormArgs& a) {
  if (T > 64 && a.in_place && a.dim % 8 != 0) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  }
}

template <int XDT, int BDT, int T> __global__ __launch_bounds__(kBlock<T>) void block_norm_kernel(BlockNormArgs a) {
  using X = typename OpElem<XDT>::T;
  using B = typename OpElem<BDT>::T;
  __shared__ float red[2 * (T / 64)];
  const int e = threadIdx.x % T * 8;
  const float inv = 1.0f / static_cast<float>(a.dim);
  float gpre[8], gb[8], gate[8];
  gain(a.w[0], a.w_bf16, a.offset, e, a.dim, gpre);
  gain(a.w[1], a.w_bf16, a.offset, e, a.dim, gb);
  gain(a.w[2], a.w_bf16, 0.0f, e, a.dim, gate);
#pragma unroll
  for (int i = 0; i < 8; ++i) gb[i] *= gate[i] * a.scale;
  RowSum<T, 1> sum{red};
  const X* x = static_cast<const X*>(a.x);
  const B* h = static_cast<const B*>(a.h);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRowsAtOnce<T>;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsAtOnce<T> + threadIdx.x / T;
  Run<XDT> nx;
  Run<BDT> nh;
  if (row < a.rows) {
    nx.load(x + row * a.xs, e, a.dim);
    nh.load(h + row * a.hs, e, a.dim);
  }
  for (; row < a.rows; row += step) {
    nx.land(e, a.dim);
    nh.land(e, a.dim);
    float v[8], b[8], s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = nx[i];
      b[i] = nh[i];
      s[0] += b[i] * b[i];
    }
    if (row + step < a.rows) {
      nx.load(x + (row + step) * a.xs, e, a.dim);
      nh.load(h + (row + step) * a.hs, e, a.dim);
    }
    float rh = 1.0f;
    if (a.post_norm) {
      sum(s);
      rh = 1.0f / sqrtf(s[0] * inv + a.eps);
    }
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = stored<X>(fmaf(b[i] * rh, gb[i], v[i]));
      s[0] += v[i] * v[i];
    }
    row_loaded<T>(a);
    put(static_cast<X*>(a.x_out) + row * a.xos, e, a.dim, v);
    sum(s);
    const float rx = 1.0f / sqrtf(s[0] * inv + a.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * rx * gpre[i];
    put(static_cast<B*>(a.y) + row * a.ys, e, a.dim, v);
  }
}

template <int XDT, int BDT, int T> __global__ __launch_bounds__(kBlock<T>) void block_norm_grad_kernel(BlockNormArgs a) {
  using X = typename OpElem<XDT>::T;
  using B = typename OpElem<BDT>::T;
  __shared__ float red3[2 * (T / 64) * 3], red1[2 * (T / 64)];
  __shared__ float join[T == 64 ? 4 * 512 : 1];
  const int e = threadIdx.x % T * 8;
  const float inv = 1.0f / static_cast<float>(a.dim);
  float gpre[8], gd[8], gate[8];
  gain(a.w[0], a.w_bf16, a.offset, e, a.dim, gpre);
  gain(a.w[1], a.w_bf16, a.offset, e, a.dim, gd);
  gain(a.w[2], a.w_bf16, 0.0f, e, a.dim, gate);
#pragma unroll
  for (int i = 0; i < 8; ++i) gd[i] *= gate[i];
  // Sixteen waves leave 128 registers to each.  The next row beside this one does
  // not fit them: a row of over 4096 is under way as a whole instead, and the
  // gains are kept in LDS, each lane its own (32768 x 8192: 884 us; with the next
  // row and the gains in registers, up to 122 of which spill, 1779).
  constexpr bool kAhead = T < 1024;
  __shared__ f32v4 kept[kAhead ? 1 : 4][kAhead ? 1 : T];
  if constexpr (!kAhead)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      kept[k][threadIdx.x] = f32v4{gpre[4 * k], gpre[4 * k + 1], gpre[4 * k + 2], gpre[4 * k + 3]};
      kept[2 + k][threadIdx.x] = f32v4{gd[4 * k], gd[4 * k + 1], gd[4 * k + 2], gd[4 * k + 3]};
    }
  auto pre_gain = [&](int i) { if constexpr (kAhead) return gpre[i]; else return kept[i >> 2][threadIdx.x][i & 3]; };
  auto post_gain = [&](int i) { if constexpr (kAhead) return gd[i]; else return kept[2 + (i >> 2)][threadIdx.x][i & 3]; };
  float acc[2][8] = {};
  RowSum<T, 3> sum3{red3};
  RowSum<T, 1> sum1{red1};
  const X* x = static_cast<const X*>(a.x);
  const X* dx = static_cast<const X*>(a.dx_out);
  const B* h = static_cast<const B*>(a.h);
  const B* dy = static_cast<const B*>(a.dy);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRowsAtOnce<T>;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsAtOnce<T> + threadIdx.x / T;
  Run<XDT> nx, nd;
  Run<BDT> nh, ny;
  nd.v = {};
  auto ahead = [&](int64_t r) {
    if (r >= a.rows) return;
    nx.load(x + r * a.xs, e, a.dim);
    ny.load(dy + r * a.dys, e, a.dim);
    nh.load(h + r * a.hs, e, a.dim);
    if (dx) nd.load(dx + r * a.dxs, e, a.dim);
  };
  if (kAhead) ahead(row);
  for (; row < a.rows; row += step) {
    if (!kAhead) ahead(row);
    nx.land(e, a.dim);
    ny.land(e, a.dim);
    nh.land(e, a.dim);
    nd.land(e, a.dim);
    const Run<XDT> cx = nx, cd = nd;
    const Run<BDT> ch = nh, cy = ny;
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[0] += cx[i] * cx[i];
      s[1] += cy[i] * pre_gain(i) * cx[i];
      s[2] += ch[i] * ch[i];
    }
    if (kAhead) ahead(row + step);
    sum3(s);
    const float rx = 1.0f / sqrtf(s[0] * inv + a.eps);
    const float rh = a.post_norm ? 1.0f / sqrtf(s[2] * inv + a.eps) : 1.0f;
    const float along = s[1] * rx * inv;   // mean(dy g xh)
    float out[8], d[8], u[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float xh = cx[i] * rx, hh = ch[i] * rh;
      out[i] = rx * (cy[i] * pre_gain(i) - xh * along) + cd[i];
      const float st = a.scale * out[i];
      acc[0][i] += cy[i] * xh;
      acc[1][i] += st * hh;
      d[i] = st * post_gain(i);
      u[0] += d[i] * hh;
    }
    row_loaded<T>(a);
    put(static_cast<X*>(a.x_out) + row * a.xos, e, a.dim, out);
    if (a.post_norm) {
      sum1(u);
      const float mean = u[0] * inv;
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = rh * (d[i] - ch[i] * rh * mean);
    }
    put(static_cast<B*>(a.y) + row * a.ys, e, a.dim, d);
  }
  if (!a.part) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float* out = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + k) * a.dim;
    if constexpr (T == 64) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) join[(threadIdx.x >> 6) * 512 + e + i] = acc[k][i];
      __syncthreads();
      for (int c = threadIdx.x; c < a.dim; c += 256) gmem(out)[c] = join[c] + join[512 + c] + join[1024 + c] + join[1536 + c];
    } else {
      put(out, e, a.dim, acc[k]);
    }
  }
}

// ---------------------------------------------------------------- wide rows
constexpr int kWide = 1024;   // threads of a row

template <int XDT, int BDT> __global__ __launch_bounds__(kWide) void bn_wide_kernel(BlockNormArgs a) {
  using X = typename OpElem<XDT>::T;
  using B = typename OpElem<BDT>::T;
  __shared__ float red[2 * (kWide / 64)];
  RowSum<kWide, 1> sum{red};
  const float inv = 1.0f / static_cast<float>(a.dim);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const X* x = static_cast<const X*>(a.x) + row * a.xs;
    const B* h = static_cast<const B*>(a.h) + row * a.hs;
    X* xo = static_cast<X*>(a.x_out) + row * a.xos;
    float s[1] = {0.0f}, rh = 1.0f;
    if (a.post_norm) {
      for (int e = threadIdx.x * 8; e < a.dim; e += kWide * 8) {
        Run<BDT> ch;
        ch.load(h, e, a.dim);
        ch.land(e, a.dim);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += ch[i] * ch[i];
      }
      sum(s);
      rh = 1.0f / sqrtf(s[0] * inv + a.eps);
      s[0] = 0.0f;
    }
    for (int e = threadIdx.x * 8; e < a.dim; e += kWide * 8) {
      Run<XDT> cx;
      Run<BDT> ch;
      cx.load_own(x, e, a.dim);
      ch.load(h, e, a.dim);
      ch.land(e, a.dim);
      float gpost[8], gate[8], v[8];
      gain(a.w[1], a.w_bf16, a.offset, e, a.dim, gpost);
      gain(a.w[2], a.w_bf16, 0.0f, e, a.dim, gate);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = stored<X>(fmaf(ch[i] * rh, gpost[i] * (gate[i] * a.scale), cx[i]));
        s[0] += v[i] * v[i];
      }
      put(xo, e, a.dim, v);
    }
    sum(s);
    const float rx = 1.0f / sqrtf(s[0] * inv + a.eps);
    for (int e = threadIdx.x * 8; e < a.dim; e += kWide * 8) {   // what this thread has stored
      Run<XDT> cx;
      cx.load_own(xo, e, a.dim);
      float g[8], v[8];
      gain(a.w[0], a.w_bf16, a.offset, e, a.dim, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = cx[i] * rx * g[i];
      put(static_cast<B*>(a.y) + row * a.ys, e, a.dim, v);
    }
  }
}

// stats_only: stores both reciprocal lengths and the mean of a row, and nothing else.
template <int XDT, int BDT> __global__ __launch_bounds__(kWide) void bn_wide_grad_kernel(BlockNormArgs a) {
  using X = typename OpElem<XDT>::T;
  using B = typename OpElem<BDT>::T;
  __shared__ float red3[2 * (kWide / 64) * 3], red1[2 * (kWide / 64)];
  RowSum<kWide, 3> sum3{red3};
  RowSum<kWide, 1> sum1{red1};
  const float inv = 1.0f / static_cast<float>(a.dim);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const X* x = static_cast<const X*>(a.x) + row * a.xs;
    const X* dx = a.dx_out ? static_cast<const X*>(a.dx_out) + row * a.dxs : nullptr;
    const B* h = static_cast<const B*>(a.h) + row * a.hs;
    const B* dy = static_cast<const B*>(a.dy) + row * a.dys;
    float s[3] = {0.0f, 0.0f, 0.0f};
    for (int e = threadIdx.x * 8; e < a.dim; e += kWide * 8) {
      Run<XDT> cx;
      Run<BDT> ch, cy;
      cx.load(x, e, a.dim);
      cy.load(dy, e, a.dim);
      ch.load(h, e, a.dim);
      cx.land(e, a.dim);
      cy.land(e, a.dim);
      ch.land(e, a.dim);
      float g[8];
      gain(a.w[0], a.w_bf16, a.offset, e, a.dim, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[0] += cx[i] * cx[i];
        s[1] += cy[i] * g[i] * cx[i];
        s[2] += ch[i] * ch[i];
      }
    }
    sum3(s);
    const float rx = 1.0f / sqrtf(s[0] * inv + a.eps);
    const float rh = a.post_norm ? 1.0f / sqrtf(s[2] * inv + a.eps) : 1.0f;
    const float along = s[1] * rx * inv;
    if (a.stats_only) {
      if (threadIdx.x == 0) {
        gmem(a.stats)[3 * row] = rx;
        gmem(a.stats)[3 * row + 1] = rh;
        gmem(a.stats)[3 * row + 2] = along;
      }
      continue;
    }
    // t and db g_post of a run, formed once for the mean and once more for the results
    auto run = [&](int e, float* t, float* d, float* hh) {
      Run<XDT> cx, cd;
      Run<BDT> ch, cy;
      cx.load(x, e, a.dim);
      cy.load(dy, e, a.dim);
      ch.load(h, e, a.dim);
      cd.v = {};
      if (dx) cd.load_own(dx, e, a.dim);
      cx.land(e, a.dim);
      cy.land(e, a.dim);
      ch.land(e, a.dim);
      float gpre[8], gpost[8], gate[8];
      gain(a.w[0], a.w_bf16, a.offset, e, a.dim, gpre);
      gain(a.w[1], a.w_bf16, a.offset, e, a.dim, gpost);
      gain(a.w[2], a.w_bf16, 0.0f, e, a.dim, gate);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t[i] = rx * (cy[i] * gpre[i] - cx[i] * rx * along) + cd[i];
        d[i] = a.scale * t[i] * (gpost[i] * gate[i]);
        hh[i] = ch[i] * rh;
      }
    };
    float t[8], d[8], hh[8], u[1] = {0.0f};
    if (a.post_norm) {
      for (int e = threadIdx.x * 8; e < a.dim; e += kWide * 8) {
        run(e, t, d, hh);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[0] += d[i] * hh[i];
      }
      sum1(u);
    }
    const float mean = u[0] * inv;
    for (int e = threadIdx.x * 8; e < a.dim; e += kWide * 8) {
      run(e, t, d, hh);
      put(static_cast<X*>(a.x_out) + row * a.xos, e, a.dim, t);
      if (a.post_norm)
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = rh * (d[i] - hh[i] * mean);
      put(static_cast<B*>(a.y) + row * a.ys, e, a.dim, d);
    }
  }
}

// Both sums of each thread's column over col_rows rows.
template <int XDT, int BDT> __global__ __launch_bounds__(256) void bn_columns_kernel(BlockNormArgs a) {
  using X = typename OpElem<XDT>::T;
  using B = typename OpElem<BDT>::T;
  const int e = blockIdx.x * 256 + threadIdx.x;
  if (e >= a.dim) return;
  const float gpre = one_gain(a.w[0], a.w_bf16, a.offset, e);
  float acc[2] = {0.0f, 0.0f};
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * a.col_rows, r1 = least(r0 + a.col_rows, a.rows);
  for (int64_t r = r0; r < r1; ++r) {
    const float x = static_cast<float>(gmem(static_cast<const X*>(a.x))[r * a.xs + e]);
    const float h = static_cast<float>(gmem(static_cast<const B*>(a.h))[r * a.hs + e]);
    const float dy = static_cast<float>(gmem(static_cast<const B*>(a.dy))[r * a.dys + e]);
    const float dx = a.dx_out ? static_cast<float>(gmem(static_cast<const X*>(a.dx_out))[r * a.dxs + e]) : 0.0f;
    const float rx = gmem(a.stats)[3 * r], rh = gmem(a.stats)[3 * r + 1], along = gmem(a.stats)[3 * r + 2];
    const float t = rx * (dy * gpre - x * rx * along) + dx;
    acc[0] += dy * (x * rx);
    acc[1] += a.scale * t * (h * rh);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) gmem(a.part)[(static_cast<int64_t>(blockIdx.y) * 2 + k) * a.dim + e] = acc[k];
}

// Adds the blocks' rows of sums: 64 columns a block, 16 runs of rows, joined in order.
constexpr int kJoinRuns = 16;
__global__ __launch_bounds__(64 * kJoinRuns) void bn_join_kernel(BlockNormArgs a) {
  __shared__ float run[kJoinRuns][64];
  const int k = blockIdx.y, lane = threadIdx.x & 63, r = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  const int per = (a.blocks + kJoinRuns - 1) / kJoinRuns;
  float s = 0.0f;
  if (e < a.dim)
#pragma unroll 8
    for (int b = r * per; b < least((r + 1) * per, a.blocks); ++b)
      s += gmem(a.part)[(static_cast<int64_t>(b) * 2 + k) * a.dim + e];
  run[r][lane] = s;
  __syncthreads();
  if (r > 0 || e >= a.dim) return;
  for (int i = 1; i < kJoinRuns; ++i) s += run[i][lane];
  auto write = [&](void* out, float v) {
    if (!out) return;
    if (a.w_bf16) gmem(static_cast<__bf16*>(out))[e] = static_cast<__bf16>(v);
    else gmem(static_cast<float*>(out))[e] = v;
  };
  if (k == 0) {
    write(a.dw[0], s);
  } else {
    write(a.dw[1], s * one_gain(a.w[2], a.w_bf16, 0.0f, e));
    write(a.dw[2], s * one_gain(a.w[1], a.w_bf16, a.offset, e));
  }
}

constexpr int kBnBlocks = 2048;   // blocks of the forward pass: eight a CU stride over the rows

template <int XDT, int BDT, int T> void forward(const BlockNormArgs& a, hipStream_t stream) {
  const int64_t runs = (a.rows + kRowsAtOnce<T> - 1) / kRowsAtOnce<T>;
  block_norm_kernel<XDT, BDT, T>
      <<<dim3(static_cast<unsigned>(std::min<int64_t>(runs, kBnBlocks))), dim3(kBlock<T>), 0, stream>>>(a);
}
template <int XDT, int BDT> void forward_any(const BlockNormArgs& a, hipStream_t s) {
  const int d = a.dim;
  if (d <= 512) forward<XDT, BDT, 64>(a, s);
  else if (d <= 1024) forward<XDT, BDT, 128>(a, s);
  else if (d <= 2048) forward<XDT, BDT, 256>(a, s);
  else if (d <= 4096) forward<XDT, BDT, 512>(a, s);
  else if (d <= kBnMaxFused) forward<XDT, BDT, 1024>(a, s);
  else
    bn_wide_kernel<XDT, BDT>
        <<<dim3(static_cast<unsigned>(std::min<int64_t>(a.rows, kBnBlocks))), dim3(kWide), 0, s>>>(a);
}
template <int XDT, int BDT, int T> void backward(const BlockNormArgs& a, hipStream_t s) {
  block_norm_grad_kernel<XDT, BDT, T><<<dim3(static_cast<unsigned>(a.blocks)), dim3(kBlock<T>), 0, s>>>(a);
}
template <int XDT, int BDT> void backward_any(const BlockNormArgs& a, hipStream_t s) {
  const int d = a.dim;
  if (d <= 512) backward<XDT, BDT, 64>(a, s);
  else if (d <= 1024) backward<XDT, BDT, 128>(a, s);
  else if (d <= 2048) backward<XDT, BDT, 256>(a, s);
  else if (d <= 4096) backward<XDT, BDT, 512>(a, s);
  else if (d <= kBnMaxFused) backward<XDT, BDT, 1024>(a, s);
  else {
    const dim3 blocks(static_cast<unsigned>(std::min<int64_t>(a.rows, kBnBlocks)));
    if (a.part) {   // the sums first: dx may take dx_out's place
      BlockNormArgs r = a;
      r.stats_only = 1;
      bn_wide_grad_kernel<XDT, BDT><<<blocks, dim3(kWide), 0, s>>>(r);
      bn_columns_kernel<XDT, BDT><<<dim3((d + 255) / 256, static_cast<unsigned>(a.blocks)), dim3(256), 0, s>>>(a);
    }
    bn_wide_grad_kernel<XDT, BDT><<<blocks, dim3(kWide), 0, s>>>(a);
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
    bn_join_kernel<<<dim3((a.dim + 63) / 64, 2), dim3(64 * kJoinRuns), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace dmuon
