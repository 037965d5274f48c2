// Norms of queries and keys per head with the position rotation in the same
// pass, forward and backward, on gfx950 (HBM-bound).
//
// For every token and head of width D, with gain w and rotation R(pos):
//
//   r   = 1 / sqrt(mean(x^2) + eps)
//   out = R n,   n = x r (offset + w)
//
// and, with dn = R^T dout, xh = x r, g = dn (offset + w):
//
//   dx = r (g - xh mean(g xh)),     dw = sum over tokens and heads of dn xh
//
// R turns `rot` / 2 pairs by the angles of the token's position: elements
// (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved; the elements behind
// `rot` stay.  A negative position marks a padding token: zeros, and no part
// in dw.  A position behind the table gives NaN.
//
// A lane holds four pairs of one head (a "unit" of eight elements), so both
// halves of a rotation meet in one lane; the smallest power of two of lanes
// that covers D holds a head, and a wave works on 64 / that many heads of one
// token at once.  The cosines and sines are read once per token.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops.hpp"

namespace dmuon {
namespace {

constexpr int kQkThreads = 256;
constexpr int kQkWaves = kQkThreads / 64;

// The query's or the key's entry: a select, where an index would go through memory.
template <typename V> __device__ __forceinline__ V pick(const V (&v)[2], int which) { return which ? v[1] : v[0]; }

// Elements of pair p; the second is D when there is none.
__device__ __forceinline__ void pair_elems(const QkArgs& a, int p, int* e0, int* e1) {
  const int half = a.rot / 2;
  if (a.interleaved || p >= half) {
    *e0 = 2 * p;   // behind the rotated part both layouts count on: rot + 2 (p - half) = 2 p
    *e1 = 2 * p + 1;
  } else {
    *e0 = p;
    *e1 = half + p;
  }
}

template <int DT, bool VEC>
__device__ __forceinline__ void load_unit(const QkArgs& q, const typename OpElem<DT>::T* p, int t, float* a, float* b) {
  if constexpr (VEC) {
    float lo[4], hi[4];
    const int half = q.rot / 2;
    const bool split = !q.interleaved && 4 * t < half;
    load_n<4>(p + (split ? 4 * t : 8 * t), lo);
    load_n<4>(p + (split ? half + 4 * t : 8 * t + 4), hi);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = i < 2 ? lo[2 * i] : hi[2 * i - 4], y = i < 2 ? lo[2 * i + 1] : hi[2 * i - 3];
      a[i] = split ? lo[i] : x;
      b[i] = split ? hi[i] : y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int e0, e1;
      pair_elems(q, 4 * t + i, &e0, &e1);
      a[i] = e0 < q.dim ? static_cast<float>(gmem(p)[e0]) : 0.0f;
      b[i] = e1 < q.dim ? static_cast<float>(gmem(p)[e1]) : 0.0f;
    }
  }
}

template <int DT, bool VEC>
__device__ __forceinline__ void store_unit(const QkArgs& q, typename OpElem<DT>::T* p, int t, const float* a, const float* b) {
  using T = typename OpElem<DT>::T;
  if constexpr (VEC) {
    const int half = q.rot / 2;
    const bool split = !q.interleaved && 4 * t < half;
    const float lo[4] = {a[0], split ? a[1] : b[0], split ? a[2] : a[1], split ? a[3] : b[1]};
    const float hi[4] = {split ? b[0] : a[2], split ? b[1] : b[2], split ? b[2] : a[3], b[3]};
    store_n<4>(p + (split ? 4 * t : 8 * t), lo);
    store_n<4>(p + (split ? half + 4 * t : 8 * t + 4), hi);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int e0, e1;
      pair_elems(q, 4 * t + i, &e0, &e1);
      if (e0 < q.dim) gmem(p)[e0] = static_cast<T>(a[i]);
      if (e1 < q.dim) gmem(p)[e1] = static_cast<T>(b[i]);
    }
  }
}

__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Cosines and sines of a lane's four pairs at the token's position, and how
// the token is treated: 0 padding, 1 rotated, 2 behind the table.
__device__ __forceinline__ int token_angles(const QkArgs& a, int64_t token, int t, float* c, float* s) {
  int64_t pos = 0;
  if (a.rot > 0) pos = load_index(a.positions, token, a.pos64);
  const int kind = pos < 0 ? 0 : a.rot > 0 && pos >= a.max_pos ? 2 : 1;
  const int half = a.rot / 2;
  const float* row = a.rope + (kind == 1 ? pos : 0) * a.rot;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = 4 * t + i;
    const bool turn = kind == 1 && p < half;
    c[i] = turn ? gmem(row)[p] : 1.0f;
    s[i] = turn ? gmem(row)[half + p] : 0.0f;
  }
  return kind;
}

template <int WDT, bool VEC>
__device__ __forceinline__ void load_gain(const QkArgs& q, int which, int t, float* wa, float* wb) {
  using W = typename OpElem<WDT>::T;
  const W* w = static_cast<const W*>(pick(q.w, which));
  if (!w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) wa[i] = wb[i] = 1.0f;
    return;
  }
  load_unit<WDT, VEC>(q, w, t, wa, wb);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    wa[i] += q.offset;
    wb[i] += q.offset;
  }
}

template <int DT, int WDT, bool VEC>
__global__ __launch_bounds__(kQkThreads) void qk_norm_kernel(QkArgs a, int log_lanes, int heads_per_item) {
  using T = typename OpElem<DT>::T;
  const int lanes = 1 << log_lanes, lane = threadIdx.x & 63;
  const int t = lane & (lanes - 1), sub = lane >> log_lanes, per = 64 >> log_lanes;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kQkWaves + (threadIdx.x >> 6);
  if (token >= a.n) return;
  const bool any = 8 * t < a.dim;
  float c[4], s[4];
  const int kind = token_angles(a, token, any ? t : 0, c, s);
  const int all = a.heads[0] + a.heads[1];
  const int h0 = static_cast<int>(blockIdx.y) * heads_per_item;
  const int h1 = min(all, h0 + heads_per_item);
  for (int hb = h0; hb < h1; hb += per) {
    const int h = hb + sub;
    const bool on = any && h < h1;
    const int which = h >= a.heads[0] ? 1 : 0;
    const int64_t head = which ? h - a.heads[0] : h;
    float x[4] = {}, y[4] = {};
    if (on && kind != 0)
      load_unit<DT, VEC>(a, static_cast<const T*>(pick(a.x, which)) + token * pick(a.x_stride, which) + head * a.dim, t, x, y);
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) ss += x[i] * x[i] + y[i] * y[i];
    ss = group_sum(ss, lanes);
    float r = 1.0f / sqrtf(ss / static_cast<float>(a.dim) + a.eps);
    if (kind == 2) r = NAN;
    if (!on) continue;
    float wa[4], wb[4];
    load_gain<WDT, VEC>(a, which, t, wa, wb);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float na = x[i] * r * wa[i], nb = y[i] * r * wb[i];
      x[i] = kind == 0 ? 0.0f : na * c[i] - nb * s[i];
      y[i] = kind == 0 ? 0.0f : nb * c[i] + na * s[i];
    }
    store_unit<DT, VEC>(a, static_cast<T*>(pick(a.out, which)) + token * pick(a.out_stride, which) + head * a.dim, t, x, y);
  }
}

template <int DT, int WDT, bool VEC>
__global__ __launch_bounds__(kQkThreads) void qk_norm_grad_kernel(QkArgs a, int log_lanes) {
  using T = typename OpElem<DT>::T;
  extern __shared__ float sum[];   // kQkWaves x 2 x dim
  const int lanes = 1 << log_lanes, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = lane & (lanes - 1), sub = lane >> log_lanes, per = 64 >> log_lanes;
  const bool any = 8 * t < a.dim;
  const int all = a.heads[0] + a.heads[1];
  float dwa[2][4] = {}, dwb[2][4] = {};
  const int64_t waves = static_cast<int64_t>(gridDim.x) * kQkWaves;
  for (int64_t token = static_cast<int64_t>(blockIdx.x) * kQkWaves + wave; token < a.n; token += waves) {
    float c[4], s[4];
    const int kind = token_angles(a, token, any ? t : 0, c, s);
    for (int hb = 0; hb < all; hb += per) {
      const int h = hb + sub;
      const bool on = any && h < all;
      const int which = h >= a.heads[0] ? 1 : 0;
      const int64_t head = which ? h - a.heads[0] : h;
      float x[4] = {}, y[4] = {}, u[4] = {}, v[4] = {};
      if (on && kind != 0) {
        load_unit<DT, VEC>(a, static_cast<const T*>(pick(a.x, which)) + token * pick(a.x_stride, which) + head * a.dim, t, x, y);
        load_unit<DT, VEC>(a, static_cast<const T*>(pick(a.dy, which)) + token * pick(a.dy_stride, which) + head * a.dim, t, u, v);
      }
      float wa[4] = {}, wb[4] = {};
      if (on) load_gain<WDT, VEC>(a, which, t, wa, wb);
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) ss += x[i] * x[i] + y[i] * y[i];
      ss = group_sum(ss, lanes);
      float r = 1.0f / sqrtf(ss / static_cast<float>(a.dim) + a.eps);
      r = kind == 2 ? NAN : kind == 0 ? 0.0f : r;
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float da = u[i] * c[i] + v[i] * s[i], db = v[i] * c[i] - u[i] * s[i];
        x[i] *= r;
        y[i] *= r;
        const float ga = da * x[i], gb = db * y[i];
        dwa[0][i] += on && !which ? ga : 0.0f;
        dwb[0][i] += on && !which ? gb : 0.0f;
        dwa[1][i] += on && which ? ga : 0.0f;
        dwb[1][i] += on && which ? gb : 0.0f;
        dot += ga * wa[i] + gb * wb[i];
        u[i] = da * wa[i];
        v[i] = db * wb[i];
      }
      dot = group_sum(dot, lanes) / static_cast<float>(a.dim);
      if (!on) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u[i] = kind == 0 ? 0.0f : r * (u[i] - x[i] * dot);
        v[i] = kind == 0 ? 0.0f : r * (v[i] - y[i] * dot);
      }
      store_unit<DT, VEC>(a, static_cast<T*>(pick(a.out, which)) + token * pick(a.out_stride, which) + head * a.dim, t, u, v);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      for (int o = 32; o >= lanes; o >>= 1) {
        dwa[k][i] += __shfl_xor(dwa[k][i], o, 64);
        dwb[k][i] += __shfl_xor(dwb[k][i], o, 64);
      }
      if (sub == 0) {
        int e0, e1;
        pair_elems(a, 4 * t + i, &e0, &e1);
        if (e0 < a.dim) sum[(wave * 2 + k) * a.dim + e0] = dwa[k][i];
        if (e1 < a.dim) sum[(wave * 2 + k) * a.dim + e1] = dwb[k][i];
      }
    }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * a.dim; e += kQkThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kQkWaves; ++w) v += sum[w * 2 * a.dim + e];
    gmem(a.part)[static_cast<int64_t>(blockIdx.x) * 2 * a.dim + e] = v;
  }
}

// dw = sum of the blocks' parts, in a fixed order.
template <int WDT>
__global__ __launch_bounds__(kQkThreads) void qk_gain_kernel(QkArgs a) {
  using W = typename OpElem<WDT>::T;
  __shared__ float red[kQkWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  float v = 0.0f;
  if (e < 2 * a.dim)
    for (int b = wave; b < a.blocks; b += kQkWaves) v += gmem(a.part)[static_cast<int64_t>(b) * 2 * a.dim + e];
  red[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && e < 2 * a.dim) {
    float r = 0.0f;
#pragma unroll
    for (int w = 0; w < kQkWaves; ++w) r += red[w][lane];
    const int which = e >= a.dim ? 1 : 0;
    W* dw = static_cast<W*>(a.dw[which]);
    if (dw) gmem(dw)[e - which * a.dim] = static_cast<W>(r);
  }
}

int log_lanes_of(int dim) {
  int l = 0;
  while ((8 << l) < dim) ++l;
  return l;
}

template <typename F> void by_types(int dt, int w_dt, int vec, F&& f) {
  auto w = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (w_dt == kBF16) {
      if (vec) f(std::integral_constant<int, D>{}, std::integral_constant<int, kBF16>{}, std::true_type{});
      else f(std::integral_constant<int, D>{}, std::integral_constant<int, kBF16>{}, std::false_type{});
    } else {
      if (vec) f(std::integral_constant<int, D>{}, std::integral_constant<int, kF32>{}, std::true_type{});
      else f(std::integral_constant<int, D>{}, std::integral_constant<int, kF32>{}, std::false_type{});
    }
  };
  if (dt == kBF16) w(std::integral_constant<int, kBF16>{});
  else w(std::integral_constant<int, kF32>{});
}

}  // namespace

hipError_t launch_qk_norm(int dt, int w_dt, const QkArgs& a, hipStream_t stream) {
  if (a.n == 0) return hipSuccess;
  const int ll = log_lanes_of(a.dim), per = 64 >> ll;
  const int all = a.heads[0] + a.heads[1];
  // few tokens: one pass of heads per wave; many: up to eight passes share a token's angles
  const int passes = (all + per - 1) / per;
  const int item_passes = a.n >= 4096 ? (passes < 8 ? passes : 8) : 1;
  const int hp = item_passes * per;
  const dim3 grid(static_cast<unsigned>((a.n + kQkWaves - 1) / kQkWaves), static_cast<unsigned>((all + hp - 1) / hp));
  by_types(dt, w_dt, a.vec, [&](auto d, auto w, auto v) {
    hipLaunchKernelGGL((qk_norm_kernel<decltype(d)::value, decltype(w)::value, decltype(v)::value>), grid,
                       dim3(kQkThreads), 0, stream, a, ll, hp);
  });
  return hipGetLastError();
}

hipError_t launch_qk_norm_grad(int dt, int w_dt, const QkArgs& a, hipStream_t stream) {
  const int ll = log_lanes_of(a.dim);
  if (a.n > 0) {
    by_types(dt, w_dt, a.vec, [&](auto d, auto w, auto v) {
      hipLaunchKernelGGL((qk_norm_grad_kernel<decltype(d)::value, decltype(w)::value, decltype(v)::value>),
                         dim3(a.blocks), dim3(kQkThreads), sizeof(float) * kQkWaves * 2 * a.dim, stream, a, ll);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.dw[0] && !a.dw[1]) return hipSuccess;
  const dim3 grid((2 * a.dim + 63) / 64);
  if (w_dt == kBF16) hipLaunchKernelGGL(qk_gain_kernel<kBF16>, grid, dim3(kQkThreads), 0, stream, a);
  else hipLaunchKernelGGL(qk_gain_kernel<kF32>, grid, dim3(kQkThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace dmuon
