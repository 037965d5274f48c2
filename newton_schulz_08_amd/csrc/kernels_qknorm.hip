// Norms of queries and keys per head with the position rotation in the same
// pass, forward and backward, on gfx950 (HBM-bound).  Measured at 32768 tokens of
// 40 bf16 heads of 128: forward 128 us (0.67 GB, 5.2 TB/s), backward 206 us (1.0
// GB, 5.0 TB/s).
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
// A lane holds P pairs of one head, so both halves of a rotation meet in one
// lane; the smallest power of two of lanes that covers D holds a head.  P = 8
// makes every access of a bf16 head 16 bytes wide; P = 4 does so for fp32 and
// serves bf16 heads whose halves are no multiple of 8.  The queries and the
// keys are worked on by different blocks (one gain, one set of gain sums in
// registers); a wave takes as many heads of a token at once as it has groups
// of lanes, or several tokens where a token has fewer heads, and keeps the
// token's cosines and sines over all of its heads.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops.hpp"

namespace dmuon {
namespace {

constexpr int kQkThreads = 256;
constexpr int kQkWaves = kQkThreads / 64;

// The query's or the key's entry: a select, where an index would go through memory.
template <typename V> __device__ __forceinline__ V pick(const V (&v)[2], int which) { return which ? v[1] : v[0]; }

// Elements of pair p (the second is >= D when there is none).
__device__ __forceinline__ void pair_elems(const QkArgs& a, int p, int* e0, int* e1) {
  const int half = a.rot / 2;
  if (a.interleaved || p >= half) {
    *e0 = 2 * p;   // behind the rotated part: rot + 2 (p - half) = 2 p
    *e1 = 2 * p + 1;
  } else {
    *e0 = p;
    *e1 = half + p;
  }
}

// A lane's P pairs (a[i], b[i]), the t-th such run of the head.  VEC: the run
// is either two runs of P elements half a rotation apart, or 2 P consecutive
// ones; `Raw` keeps it as loaded, so that a load can run ahead of its use.
template <int DT, int P, bool VEC> struct Raw {
  using T = typename OpElem<DT>::T;
  using V = T __attribute__((ext_vector_type(P)));
  V lo, hi;
  template <bool STREAM> __device__ __forceinline__ void load(const QkArgs& q, const T* p, int t) {
    const int half = q.rot / 2;
    const bool split = !q.interleaved && P * t < half;
    const auto pl = reinterpret_cast<gptr<const V>>(gmem(p + (split ? P * t : 2 * P * t)));
    const auto ph = reinterpret_cast<gptr<const V>>(gmem(p + (split ? half + P * t : 2 * P * t + P)));
    if constexpr (STREAM) {
      lo = __builtin_nontemporal_load(pl);
      hi = __builtin_nontemporal_load(ph);
    } else {
      lo = *pl;
      hi = *ph;
    }
  }
  __device__ __forceinline__ void clear() { lo = hi = V{}; }
  __device__ __forceinline__ void pairs(const QkArgs& q, int t, float* a, float* b) const {
    const bool split = !q.interleaved && P * t < q.rot / 2;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const T x = i < P / 2 ? lo[2 * i] : hi[2 * i - P], y = i < P / 2 ? lo[2 * i + 1] : hi[2 * i + 1 - P];
      a[i] = static_cast<float>(split ? lo[i] : x);
      b[i] = static_cast<float>(split ? hi[i] : y);
    }
  }
};
template <int DT, int P> struct Raw<DT, P, false> {
  using T = typename OpElem<DT>::T;
  T x[P], y[P];
  template <bool STREAM> __device__ __forceinline__ void load(const QkArgs& q, const T* p, int t) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      int e0, e1;
      pair_elems(q, P * t + i, &e0, &e1);
      x[i] = e0 < q.dim ? gmem(p)[e0] : static_cast<T>(0.0f);
      y[i] = e1 < q.dim ? gmem(p)[e1] : static_cast<T>(0.0f);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = y[i] = static_cast<T>(0.0f);
  }
  __device__ __forceinline__ void pairs(const QkArgs&, int, float* a, float* b) const {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      a[i] = static_cast<float>(x[i]);
      b[i] = static_cast<float>(y[i]);
    }
  }
};

template <int DT, int P, bool VEC, bool STREAM>
__device__ __forceinline__ void store_unit(const QkArgs& q, typename OpElem<DT>::T* p, int t, const float* a, const float* b) {
  using T = typename OpElem<DT>::T;
  if constexpr (VEC) {
    const int half = q.rot / 2;
    const bool split = !q.interleaved && P * t < half;
    float lo[P], hi[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int l = i / 2, h = (P + i) / 2;   // pair that the i-th element of each run belongs to, side by side
      lo[i] = split ? a[i] : i % 2 ? b[l] : a[l];
      hi[i] = split ? b[i] : i % 2 ? b[h] : a[h];
    }
    store_n<P, STREAM>(p + (split ? P * t : 2 * P * t), lo);
    store_n<P, STREAM>(p + (split ? half + P * t : 2 * P * t + P), hi);
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      int e0, e1;
      pair_elems(q, P * t + i, &e0, &e1);
      if (e0 < q.dim) gmem(p)[e0] = static_cast<T>(a[i]);
      if (e1 < q.dim) gmem(p)[e1] = static_cast<T>(b[i]);
    }
  }
}

__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Cosines and sines of a lane's pairs at the token's position, and how the
// token is treated: 0 padding, 1 rotated, 2 behind the table.
template <int P, bool VEC>
__device__ __forceinline__ int token_angles(const QkArgs& a, int64_t token, int t, float* c, float* s) {
  if (!a.positions) {   // no rotation and no padding; without a rotation alone, every run below stays as it is
#pragma unroll
    for (int i = 0; i < P; ++i) {
      c[i] = 1.0f;
      s[i] = 0.0f;
    }
    return 1;
  }
  const int64_t pos = load_index(a.positions, token, a.pos64);
  const int kind = pos < 0 ? 0 : pos >= a.max_pos ? 2 : 1;
  const int half = a.rot / 2;
  const float* row = a.rope + (kind == 1 ? pos : 0) * a.rot;
  if (VEC && a.rope_vec) {   // a run is turned or not as a whole
    const bool turn = kind == 1 && P * t < half;
    if (turn) {
      load_n<P>(row + P * t, c);
      load_n<P>(row + half + P * t, s);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      c[i] = turn ? c[i] : 1.0f;
      s[i] = turn ? s[i] : 0.0f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = P * t + i;
      const bool turn = kind == 1 && p < half;
      c[i] = turn ? gmem(row)[p] : 1.0f;
      s[i] = turn ? gmem(row)[half + p] : 0.0f;
    }
  }
  return kind;
}

template <int WDT, int P, bool VEC>
__device__ __forceinline__ void load_gain(const QkArgs& q, int which, int t, float* wa, float* wb) {
  using W = typename OpElem<WDT>::T;
  const W* w = static_cast<const W*>(pick(q.w, which));
  if (!w) {
#pragma unroll
    for (int i = 0; i < P; ++i) wa[i] = wb[i] = 1.0f;
    return;
  }
  if constexpr (VEC) {
    // fp32 gains of eight pairs are wider than one load
    float lo[P], hi[P];
    const int half = q.rot / 2;
    const bool split = !q.interleaved && P * t < half;
    load_n<P>(w + (split ? P * t : 2 * P * t), lo);
    load_n<P>(w + (split ? half + P * t : 2 * P * t + P), hi);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float x = i < P / 2 ? lo[2 * i] : hi[2 * i - P], y = i < P / 2 ? lo[2 * i + 1] : hi[2 * i + 1 - P];
      wa[i] = split ? lo[i] : x;
      wb[i] = split ? hi[i] : y;
    }
  } else {
    Raw<WDT, P, false> r;
    r.template load<false>(q, w, t);
    r.pairs(q, t, wa, wb);
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    wa[i] += q.offset;
    wb[i] += q.offset;
  }
}

// What a wave's lanes do: lane group `head` of `heads_at_once`, token `tok` of
// the wave's tokens, t-th run of the head.
struct Place {
  int which, t, head, tok, heads_at_once, tokens_at_once;
  int64_t block;   // among the blocks of its tensor
  bool any;        // the lane has elements
};
template <int P>
__device__ __forceinline__ Place place(const QkArgs& a, int log_lanes, int blocks_q) {
  Place p;
  const int lane = threadIdx.x & 63;
  p.which = static_cast<int>(blockIdx.x) >= blocks_q ? 1 : 0;
  p.block = static_cast<int64_t>(blockIdx.x) - (p.which ? blocks_q : 0);
  p.t = lane & ((1 << log_lanes) - 1);
  p.any = 2 * P * p.t < a.dim;
  const int group = lane >> log_lanes, log_groups = 6 - log_lanes;
  const int lh = least(pick(a.log_heads, p.which), log_groups);
  p.heads_at_once = 1 << lh;
  p.tokens_at_once = 1 << (log_groups - lh);
  p.head = group & (p.heads_at_once - 1);
  p.tok = group >> lh;
  return p;
}

// blockIdx.y takes `passes` runs of heads of a token.
template <int DT, int WDT, int P, bool VEC, bool STREAM>
__global__ __launch_bounds__(kQkThreads) void qk_norm_kernel(QkArgs a, int log_lanes, int blocks_q, int passes) {
  using T = typename OpElem<DT>::T;
  const Place p = place<P>(a, log_lanes, blocks_q);
  const int heads = pick(a.heads, p.which);
  const int64_t token = (p.block * kQkWaves + (threadIdx.x >> 6)) * p.tokens_at_once + p.tok;
  const int h0 = static_cast<int>(blockIdx.y) * passes * p.heads_at_once;
  if (h0 >= heads || (p.block * kQkWaves + (threadIdx.x >> 6)) * p.tokens_at_once >= a.n) return;
  const bool here = p.any && token < a.n;
  const T* src = static_cast<const T*>(pick(a.x, p.which)) + token * pick(a.x_stride, p.which);
  T* dst = static_cast<T*>(pick(a.out, p.which)) + token * pick(a.out_stride, p.which);
  // the first heads are on their way while the position leads to its angles
  Raw<DT, P, VEC> next;
  next.clear();
  if (here && h0 + p.head < heads) next.template load<STREAM>(a, src + static_cast<int64_t>(h0 + p.head) * a.dim, p.t);
  float c[P], s[P], wa[P], wb[P];
  const int kind = token_angles<P, VEC>(a, least(token, a.n - 1), p.any ? p.t : 0, c, s);
  load_gain<WDT, P, VEC>(a, p.which, p.any ? p.t : 0, wa, wb);
  for (int k = 0; k < passes; ++k) {
    const int h = h0 + k * p.heads_at_once + p.head;
    const bool on = here && h < heads;
    float x[P], y[P];
    next.pairs(a, p.t, x, y);
    if (k + 1 < passes && here && h + p.heads_at_once < heads)
      next.template load<STREAM>(a, src + static_cast<int64_t>(h + p.heads_at_once) * a.dim, p.t);
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) ss += x[i] * x[i] + y[i] * y[i];
    ss = group_sum(ss, 1 << log_lanes);
    float r = 1.0f / sqrtf(ss / static_cast<float>(a.dim) + a.eps);
    if (kind == 2) r = NAN;
    if (!on) continue;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float na = x[i] * r * wa[i], nb = y[i] * r * wb[i];
      x[i] = kind == 0 ? 0.0f : na * c[i] - nb * s[i];
      y[i] = kind == 0 ? 0.0f : nb * c[i] + na * s[i];
    }
    store_unit<DT, P, VEC, STREAM>(a, dst + static_cast<int64_t>(h) * a.dim, p.t, x, y);
  }
}

// The blocks of a tensor stride over its tokens and keep the gain's sums in
// registers; each leaves one row of sums in `part`.
template <int DT, int WDT, int P, bool VEC, bool STREAM>
__global__ __launch_bounds__(kQkThreads) void qk_norm_grad_kernel(QkArgs a, int log_lanes) {
  using T = typename OpElem<DT>::T;
  extern __shared__ float sum[];   // kQkWaves x dim
  const int lanes = 1 << log_lanes, wave = threadIdx.x >> 6;
  const Place p = place<P>(a, log_lanes, a.blocks[0]);
  const int heads = pick(a.heads, p.which);
  float dwa[P] = {}, dwb[P] = {}, wa[P], wb[P];
  load_gain<WDT, P, VEC>(a, p.which, p.any ? p.t : 0, wa, wb);
  const float inv_dim = 1.0f / static_cast<float>(a.dim);
  const int64_t step = static_cast<int64_t>(pick(a.blocks, p.which)) * kQkWaves * p.tokens_at_once;
  const T* xp = static_cast<const T*>(pick(a.x, p.which));
  const T* dyp = static_cast<const T*>(pick(a.dy, p.which));
  T* op = static_cast<T*>(pick(a.out, p.which));
  const int64_t xs = pick(a.x_stride, p.which), dys = pick(a.dy_stride, p.which), os = pick(a.out_stride, p.which);
  // one run of heads ahead: its loads cover the angles of its token and the sums of the run before
  Raw<DT, P, VEC> nx, ny;
  auto ahead = [&](int64_t token, int h) {
    nx.clear();
    ny.clear();
    if (p.any && token < a.n && h < heads) {
      nx.template load<STREAM>(a, xp + token * xs + static_cast<int64_t>(h) * a.dim, p.t);
      ny.template load<STREAM>(a, dyp + token * dys + static_cast<int64_t>(h) * a.dim, p.t);
    }
  };
  int64_t t0 = (p.block * kQkWaves + wave) * p.tokens_at_once;
  ahead(t0 + p.tok, p.head);
  for (; t0 < a.n; t0 += step) {
    const int64_t token = t0 + p.tok;
    const bool here = p.any && token < a.n;
    float c[P], s[P];
    const int kind = token_angles<P, VEC>(a, least(token, a.n - 1), p.any ? p.t : 0, c, s);
    for (int h = p.head; h - p.head < heads; h += p.heads_at_once) {
      const bool on = here && h < heads;
      float x[P], y[P], u[P], v[P];
      nx.pairs(a, p.t, x, y);
      ny.pairs(a, p.t, u, v);
      const int hn = h + p.heads_at_once;
      if (hn - p.head < heads) ahead(token, hn);
      else ahead(token + step, p.head);
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (kind == 0) x[i] = y[i] = u[i] = v[i] = 0.0f;   // whatever a padding token holds
        ss += x[i] * x[i] + y[i] * y[i];
      }
      ss = group_sum(ss, lanes);
      float r = 1.0f / sqrtf(ss / static_cast<float>(a.dim) + a.eps);
      r = kind == 2 ? NAN : kind == 0 ? 0.0f : r;
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float da = u[i] * c[i] + v[i] * s[i], db = v[i] * c[i] - u[i] * s[i];
        x[i] *= r;
        y[i] *= r;
        const float ga = da * x[i], gb = db * y[i];
        dwa[i] += on ? ga : 0.0f;
        dwb[i] += on ? gb : 0.0f;
        dot += ga * wa[i] + gb * wb[i];
        u[i] = da * wa[i];
        v[i] = db * wb[i];
      }
      dot = group_sum(dot, lanes) * inv_dim;
      if (!on) continue;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        u[i] = kind == 0 ? 0.0f : r * (u[i] - x[i] * dot);
        v[i] = kind == 0 ? 0.0f : r * (v[i] - y[i] * dot);
      }
      store_unit<DT, P, VEC, STREAM>(a, op + token * os + static_cast<int64_t>(h) * a.dim, p.t, u, v);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    for (int o = 32; o >= lanes; o >>= 1) {
      dwa[i] += __shfl_xor(dwa[i], o, 64);
      dwb[i] += __shfl_xor(dwb[i], o, 64);
    }
    if ((threadIdx.x & 63) < lanes) {
      int e0, e1;
      pair_elems(a, P * p.t + i, &e0, &e1);
      if (e0 < a.dim) sum[wave * a.dim + e0] = dwa[i];
      if (e1 < a.dim) sum[wave * a.dim + e1] = dwb[i];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.dim; e += kQkThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kQkWaves; ++w) v += sum[w * a.dim + e];
    gmem(a.part)[static_cast<int64_t>(blockIdx.x) * a.dim + e] = v;
  }
}

// dw = sum of the blocks' rows, in a fixed order: 16 columns a block, every
// 64th row to one of 64 threads per column, then a tree.
constexpr int kGainThreads = 1024;
template <int WDT>
__global__ __launch_bounds__(kGainThreads) void qk_gain_kernel(QkArgs a) {
  using W = typename OpElem<WDT>::T;
  __shared__ float red[64][17];
  const int which = blockIdx.y;
  W* dw = static_cast<W*>(pick(a.dw, which));
  if (!dw) return;
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4, e = blockIdx.x * 16 + col;
  const float* part = a.part + static_cast<int64_t>(which ? a.blocks[0] : 0) * a.dim;
  const int rows = pick(a.blocks, which);
  float v = 0.0f;
  if (e < a.dim) {
    for (int b0 = row; b0 < rows; b0 += 64 * 8) {
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = b0 + 64 * k < rows ? gmem(part)[static_cast<int64_t>(b0 + 64 * k) * a.dim + e] : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) v += w[k];
    }
  }
  red[row][col] = v;
  __syncthreads();
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    if (row < o) red[row][col] += red[row + o][col];
    __syncthreads();
  }
  if (row == 0 && e < a.dim) gmem(dw)[e] = static_cast<W>(red[0][col]);
}

int log2_ceil(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

// f(element type, gain type, pairs per lane, vector path, streaming accesses).
// Passes over more than the 256 MB of the memory-side cache leave it alone:
// non-temporal accesses took the 32768-token bf16 backward pass (1.0 GB) from
// 228 to 215 us.  Smaller ones find their inputs there, just written by what
// ran before (8191 fp32 tokens forward, 168 MB: 37 us, 40 non-temporal).  Only
// where one access of a wave covers whole cache lines, that is for split pairs:
// interleaved ones (two accesses to each line) went from 248 to 285 us at
// 16384 tokens of 24 fp32 heads of 256.
template <typename F> void by_types(int dt, int w_dt, const QkArgs& a, int tensors, F&& f) {
  using B = std::integral_constant<int, kBF16>;
  using S = std::integral_constant<int, kF32>;
  using P4 = std::integral_constant<int, 4>;
  using P8 = std::integral_constant<int, 8>;
  const double bytes = static_cast<double>(a.n) * (a.heads[0] + a.heads[1]) * a.dim * (dt == kBF16 ? 2 : 4) * tensors;
  auto v = [&](auto d, auto w, auto p) {
    if (a.vec && bytes > 256e6 && !a.interleaved && a.rot == a.dim) f(d, w, p, std::true_type{}, std::true_type{});
    else if (a.vec) f(d, w, p, std::true_type{}, std::false_type{});
    else f(d, w, p, std::false_type{}, std::false_type{});
  };
  auto w = [&](auto d, auto p) {
    if (w_dt == kBF16) v(d, B{}, p);
    else v(d, S{}, p);
  };
  if (dt == kF32) w(S{}, P4{});
  else if (a.pairs == 8) w(B{}, P8{});
  else w(B{}, P4{});
}

}  // namespace

hipError_t launch_qk_norm(int dt, int w_dt, const QkArgs& in, hipStream_t stream) {
  if (in.n == 0) return hipSuccess;
  QkArgs a = in;
  const int pairs = a.pairs;
  const int ll = log2_ceil((a.dim + 2 * pairs - 1) / (2 * pairs)), groups = 6 - ll;
  // few tokens: every wave one run of heads; many: up to four share a token's angles
  int blocks[2], most = 1;
  const int share = a.n >= 4096 ? 4 : 1;
  for (int k = 0; k < 2; ++k) {
    a.log_heads[k] = log2_ceil(a.heads[k]);
    const int lh = a.log_heads[k] < groups ? a.log_heads[k] : groups;
    const int64_t tokens = int64_t{kQkWaves} << (groups - lh);
    blocks[k] = a.heads[k] ? static_cast<int>((a.n + tokens - 1) / tokens) : 0;
    const int runs = (a.heads[k] + (1 << lh) - 1) >> lh;
    most = runs > most ? runs : most;
  }
  const int passes = most < share ? most : share;
  const dim3 grid(static_cast<unsigned>(blocks[0] + blocks[1]), static_cast<unsigned>((most + passes - 1) / passes));
  by_types(dt, w_dt, a, 2, [&](auto d, auto w, auto p, auto v, auto st) {
    hipLaunchKernelGGL((qk_norm_kernel<decltype(d)::value, decltype(w)::value, decltype(p)::value, decltype(v)::value,
                                       decltype(st)::value>), grid,
                       dim3(kQkThreads), 0, stream, a, ll, blocks[0], passes);
  });
  return hipGetLastError();
}

hipError_t launch_qk_norm_grad(int dt, int w_dt, const QkArgs& in, hipStream_t stream) {
  QkArgs a = in;
  const int pairs = a.pairs;
  const int ll = log2_ceil((a.dim + 2 * pairs - 1) / (2 * pairs));
  for (int k = 0; k < 2; ++k) a.log_heads[k] = log2_ceil(a.heads[k]);
  if (a.blocks[0] + a.blocks[1] > 0) {
    by_types(dt, w_dt, a, 3, [&](auto d, auto w, auto p, auto v, auto st) {
      hipLaunchKernelGGL((qk_norm_grad_kernel<decltype(d)::value, decltype(w)::value, decltype(p)::value,
                                              decltype(v)::value, decltype(st)::value>),
                         dim3(a.blocks[0] + a.blocks[1]), dim3(kQkThreads), sizeof(float) * kQkWaves * a.dim, stream, a, ll);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.dw[0] && !a.dw[1]) return hipSuccess;
  const dim3 grid((a.dim + 15) / 16, 2);
  if (w_dt == kBF16) hipLaunchKernelGGL(qk_gain_kernel<kBF16>, grid, dim3(kGainThreads), 0, stream, a);
  else hipLaunchKernelGGL(qk_gain_kernel<kF32>, grid, dim3(kGainThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace dmuon
