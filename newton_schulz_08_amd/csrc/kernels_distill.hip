// Distillation from a teacher's top logits, loss and gradient, on gfx950.
//
// Per row, with q = softmax(y / T) over the teacher's valid entries and
// lse_T = log sum_i exp(z_i / T) over the student's whole row:
//
//   KD   = T^2 sum_j q_j (log q_j - z_j / T + lse_T)
//   CE   = lse_1 - z_label
//   loss = w (kd KD + ce CE)
//   dz_i = gs w (kd T (exp(z_i / T - lse_T) - q_i) + ce (exp(z_i - lse_1) - [i = label]))
//
// HBM-bound: one or two exponentials per element against 2 or 4 bytes each way.
// Measured: 8192 x 128256 bf16 with labels at T = 2, a tenth of the rows masked,
// 811 us a call (4.0 GB that it cannot do without, 4.9 TB/s); the loss alone of
// as many unmasked rows 353 us (5.9 TB/s).
//
// Exponentials are taken in base 2 against an integer reference: with
// s2 = log2(e) / T and M = ceil(max z s2), exp2(z s2 - M) is one fused
// multiply-add (its only rounding is relative to the small difference) and one
// v_exp_f32, and moving a sum to another reference multiplies it by an exact
// power of two.  Where the label's term has another exponent than the
// teacher's, T = 2 or 4 squares the first exponential (M doubles with it)
// instead of taking a second one.  M is the ceiling of a rounded product, which
// below 2^22 is within 1/4 of the exact one; further out the difference would
// overflow the exponential.  So M stops at -+ 2^22: elements further down than
// that (finite masks) come out as 0, and a row whose maximum lies beyond it on
// either side subtracts the maximum first.
//
// Sums of exponentials are fp32; the few scalars of a row are joined in fp64
// and counted from the row's maximum, so that the loss is exact to the fp32 sums
// although it is a difference of terms that grow with the vocabulary and with
// the logits.
//
// Many rows: a block takes a row, reads it once from HBM for its sums and a
// second time, now from the memory-side cache, for the gradient.  Few rows:
// a row is cut into slices over several blocks, one launch for the sums of the
// slices and one that joins them and writes the gradient.  Either way the
// softmax terms of all elements are written first and, behind a barrier, the
// at most k + 1 elements that the teacher or the label name are rewritten.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops.hpp"

namespace dmuon {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.6931471805599453094;
constexpr float kFar = 4194304.0f;   // 2^22, of z s2
// Vectors of a long row's thread that are kept between the two passes, in
// registers and behind them in LDS (128256 bf16, 31 vectors: 892 us for 8192
// rows with none, 854 with 12 + 0, 811 with 12 + 3, 817 with 12 + 6; 790 were
// the second pass to read nothing).
constexpr int kHeld = 12, kStash = 3;

template <int N> using Int = std::integral_constant<int, N>;

// How the exponents of a row's two terms hang together.
enum DistillMode { kOne = 0, kTwo = 1, kSquare = 2, kFourth = 3 };

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}
template <typename F> __device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Scalars of a row (or of a slice of one).
struct Sums {
  float top = -INFINITY;             // largest logit
  float st = 0.0f, s1 = 0.0f;        // sums of exponentials, against the references of `top`
  float ytop = -INFINITY;            // largest teacher logit
  double ysum = 0.0;                 // sum of e_j = exp((y_j - ytop) / T)
  double dot = 0.0;                  // sum of e_j (z_j - origin(top)), over the entries in the slice
  float part = 0.0f;                 // sum of their e_j (what it scales adds up without cancelling)
  double ent = 0.0;                  // sum of e_j (y_j - ytop) / T
};

// PER: named elements per thread, THREADS x PER > k.
template <int THREADS, int PER> struct Shared {
  static constexpr int kWaves = THREADS / 64, kNamed = THREADS * PER;
  float top[kWaves], ytop[kWaves], st[kWaves], s1[kWaves];
  float part[kWaves];
  double ysum[kWaves], dot[kWaves], ent[kWaves];
  int idx[kNamed];                   // elements named by the teacher (label last), or -1
  float e[kNamed];
  float z[kNamed];
};

// What logits are counted from: the largest one, if that is a number to subtract.
__device__ __forceinline__ float origin(float top) { return isfinite(top) ? top : 0.0f; }

// Exponentials of one row: exponents s2 and, in kTwo, log2(e).
template <int MODE> struct Expo {
  float s2, m0, m1, top;
  bool far;   // the maximum is beyond the fused form, in one exponent or the other
  __device__ __forceinline__ static float reference(float top, float s2) {
    return ceilf(fminf(fmaxf(top * s2, -kFar), kFar));
  }
  __device__ __forceinline__ void set(float t, float scale) {
    s2 = scale;
    top = t;
    far = !(fabsf(t) * (MODE == kOne ? s2 : fmaxf(s2, kLog2e)) < kFar);
    m0 = reference(t, s2);
    m1 = MODE == kTwo ? reference(t, kLog2e) : MODE == kSquare ? 2.0f * m0 : 4.0f * m0;
  }
  // What the sums' exponentials are relative to, in units of the exponent s2
  // (`second`: the label's), exactly: products of two floats fit a double.
  __device__ __forceinline__ double zero(bool second) const {
    const bool one = second && MODE != kOne;
    return far ? static_cast<double>(top) * (one ? kLog2e : s2) : static_cast<double>(one ? m1 : m0);
  }
  // ... and behind the maximum
  __device__ __forceinline__ double behind(bool second) const {
    return far ? 0.0 : zero(second) - static_cast<double>(top) * (second && MODE != kOne ? kLog2e : s2);
  }
  // FAR: the slow form
  template <bool FAR> __device__ __forceinline__ void both(float v, float* et, float* e1) const {
    if constexpr (FAR) {
      const float d = v - top;
      *et = __builtin_amdgcn_exp2f(d * s2);
      if constexpr (MODE != kOne) *e1 = __builtin_amdgcn_exp2f(d * kLog2e);
    } else {
      *et = __builtin_amdgcn_exp2f(fmaf(v, s2, -m0));
      if constexpr (MODE == kTwo) *e1 = __builtin_amdgcn_exp2f(fmaf(v, kLog2e, -m1));
      if constexpr (MODE == kSquare) *e1 = *et * *et;
      if constexpr (MODE == kFourth) *e1 = (*et * *et) * (*et * *et);
    }
  }
};

__device__ __forceinline__ float scale_of(const DistillArgs& a) {
  return a.kd != 0.0f ? kLog2e / a.temperature : kLog2e;
}

// f(vector of C logits, first element, how many) over elements [from, i1),
// `from` a multiple of C behind i0.
template <typename T, int THREADS, int U, typename F>
__device__ __forceinline__ void sweep(const T* z, int64_t from, int64_t i1, F&& f) {
  constexpr int C = 16 / sizeof(T);
  const int64_t whole = from + most<int64_t>(i1 - from, 0) / C * C;
  int64_t i = from + threadIdx.x * C;
  for (; i + (U - 1) * THREADS * C < whole; i += U * THREADS * C) {
    float v[U][C];
#pragma unroll
    for (int u = 0; u < U; ++u) load_any<C>(z + i + u * THREADS * C, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) f(v[u], i + u * THREADS * C, Int<C>{});
  }
  if (i < whole) {   // the last group, as far as it goes: its loads go out together as well
    float v[U][C];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * THREADS * C < whole) load_any<C>(z + i + u * THREADS * C, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * THREADS * C < whole) f(v[u], i + u * THREADS * C, Int<C>{});
  }
  for (i = whole + threadIdx.x; i < i1; i += THREADS) {
    const float v = static_cast<float>(gmem(z)[i]);
    f(&v, i, Int<1>{});
  }
}

// The first vectors of a thread's share of a row, kept as they were loaded, so
// that the gradient need not read them again: R in registers, L in LDS.
template <typename T, int THREADS, int R, int L> struct Held {
  static constexpr int C = 16 / sizeof(T);
  using V = typename Loose<T, C>::V;
  V raw[R > 0 ? R : 1];
  uint4* stash = nullptr;   // L x THREADS
};
// As sweep; KEPT: the held vectors are there from an earlier sweep.
template <bool KEPT, typename T, int THREADS, int R, int L, typename F>
__device__ __forceinline__ void sweep_held(const T* z, int64_t i0, int64_t i1, Held<T, THREADS, R, L>& held, F&& f) {
  using H = Held<T, THREADS, R, L>;
  constexpr int C = H::C;
  const int64_t whole = i0 + (i1 - i0) / C * C;
  const int64_t first = i0 + threadIdx.x * C;
  auto at = [&](int r) { return first + r * THREADS * C; };
  auto fetch = [&](int r) { return *reinterpret_cast<gptr<const typename H::V>>(gmem(z + at(r))); };
  auto use = [&](const typename H::V& x, int r) {
    float v[C];
#pragma unroll
    for (int e = 0; e < C; ++e) v[e] = static_cast<float>(x[e]);
    f(v, at(r), Int<C>{});
  };
  constexpr int U = 4;
  static_assert(R % U == 0, "registers are filled in groups");
#pragma unroll
  for (int r = 0; r < R; r += U) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (!KEPT && at(r + u) < whole) held.raw[r + u] = fetch(r + u);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (at(r + u) < whole) use(held.raw[r + u], r + u);
  }
  if constexpr (L > 0) {
    union Word {
      typename H::V v;
      uint4 w;
    } x[L];
#pragma unroll
    for (int l = 0; l < L; ++l)
      if (at(R + l) < whole) {
        if constexpr (KEPT) x[l].w = held.stash[l * THREADS + threadIdx.x];
        else x[l].v = fetch(R + l);
      }
#pragma unroll
    for (int l = 0; l < L; ++l)
      if (at(R + l) < whole) {
        if constexpr (!KEPT) held.stash[l * THREADS + threadIdx.x] = x[l].w;   // this thread's own place
        use(x[l].v, R + l);
      }
  }
  sweep<T, THREADS, U>(z, least(whole, i0 + (R + L) * THREADS * C), i1, f);
}

// The sums of [i0, i1) of a row, and of the teacher's entries that lie in it
// (its own sums are over all entries).  Ends behind a barrier, with the entries
// in `sh` and everything in `s` of every thread; s.part only with PART.
template <int DT, int MODE, int THREADS, int PER, bool PART, int R, int L>
__device__ __forceinline__ void row_sums(const DistillArgs& a, int64_t row, int64_t i0, int64_t i1,
                                         Shared<THREADS, PER>& sh, Sums& s,
                                         Held<typename OpElem<DT>::T, THREADS, R, L>& held) {
  using T = typename OpElem<DT>::T;
  constexpr int kPer = PER;
  const T* z = static_cast<const T*>(a.logits) + row * a.stride;
  const int tid = threadIdx.x, wave = tid >> 6;
  // named elements: the indices are waited for (whether they lie in the row
  // decides what is loaded); the teacher's logits travel while the row is swept,
  // the student's while its maximum is found
  float y[kPer], zj[kPer];
  int idx[kPer];
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int j = tid + p * THREADS;
    idx[p] = -1;
    y[p] = -INFINITY;
    if (j < a.k && a.kd != 0.0f) {
      const int64_t i = load_index(a.index, row * a.k + j, a.idx64);
      if (i >= 0 && i < a.vocab) {
        idx[p] = static_cast<int>(i);
        y[p] = gmem(a.teacher)[row * a.k + j];
      }
    } else if (j == a.k && a.labels && a.ce != 0.0f) {
      const int64_t i = load_index(a.labels, row, a.idx64);
      if (i >= 0 && i < a.vocab) idx[p] = static_cast<int>(i);
    }
  }
  const float s2 = scale_of(a);
  Expo<MODE> x;
  x.set(-INFINITY, s2);
  float top = -INFINITY, st = 0.0f, s1 = 0.0f;
  sweep_held<false>(z, i0, i1, held, [&](const float* v, int64_t, auto count) {
    constexpr int N = decltype(count)::value;
    float t = v[0];
#pragma unroll
    for (int e = 1; e < N; ++e) t = fmaxf(t, v[e]);
    if (t > top) {   // rare once a few vectors are in
      const float old0 = x.m0, old1 = x.m1;
      top = t;
      x.set(t, s2);
      st *= __builtin_amdgcn_exp2f(old0 - x.m0);
      if constexpr (MODE != kOne) s1 *= __builtin_amdgcn_exp2f(old1 - x.m1);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
      float et, e1;
      x.template both<false>(v[e], &et, &e1);
      st += et;
      if constexpr (MODE != kOne) s1 += e1;
    }
  });
  float ytop = -INFINITY;
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    zj[p] = idx[p] >= i0 && idx[p] < i1 ? static_cast<float>(gmem(z)[idx[p]]) : 0.0f;
    ytop = fmaxf(ytop, y[p]);
  }
  {
    const float m = wave_max(top), n = wave_max(ytop);
    if ((tid & 63) == 0) {
      sh.top[wave] = m;
      sh.ytop[wave] = n;
    }
  }
  __syncthreads();
  s.top = sh.top[0];
  s.ytop = sh.ytop[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) {
    s.top = fmaxf(s.top, sh.top[w]);
    s.ytop = fmaxf(s.ytop, sh.ytop[w]);
  }
  Expo<MODE> all;
  all.set(s.top, s2);
  if (all.far) {   // out of the fused form's range: the maximum is subtracted first
    st = s1 = 0.0f;
    sweep<T, THREADS, 1>(z, i0, i1, [&](const float* v, int64_t, auto count) {
#pragma unroll
      for (int e = 0; e < decltype(count)::value; ++e) {
        float et, e1;
        all.template both<true>(v[e], &et, &e1);
        // nothing but -inf (whose difference is no number) sums to 0, unless a NaN is among it
        if (s.top == -INFINITY) et = e1 = v[e] == -INFINITY ? 0.0f : v[e];
        st += et;
        if constexpr (MODE != kOne) s1 += e1;
      }
    });
  } else {
    st *= __builtin_amdgcn_exp2f(x.m0 - all.m0);
    if constexpr (MODE != kOne) s1 *= __builtin_amdgcn_exp2f(x.m1 - all.m1);
  }
  const double from = origin(s.top);
  float part = 0.0f;
  double ysum = 0.0, dot = 0.0, ent = 0.0;
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int j = tid + p * THREADS;
    float e = 0.0f;
    if (y[p] != -INFINITY) {
      const float d = (y[p] - s.ytop) / a.temperature;
      e = expf(d);
      ysum += e;
      if (e != 0.0f) {
        ent += static_cast<double>(e) * d;
        if (idx[p] >= i0 && idx[p] < i1) {
          dot += e * (zj[p] - from);
          if constexpr (PART) part += e;
        }
      }
    }
    if (j <= a.k) {
      sh.idx[j] = idx[p];
      sh.z[j] = zj[p];
      sh.e[j] = e;
    }
  }
  st = wave_sum(st);
  if constexpr (MODE != kOne) s1 = wave_sum(s1);
  if (a.kd != 0.0f) {
    ysum = wave_sum(ysum);
    dot = wave_sum(dot);
    if constexpr (PART) part = wave_sum(part);
    ent = wave_sum(ent);
  }
  if ((tid & 63) == 0) {
    sh.st[wave] = st;
    sh.s1[wave] = s1;
    sh.ysum[wave] = ysum;
    sh.dot[wave] = dot;
    if constexpr (PART) sh.part[wave] = part;
    sh.ent[wave] = ent;
  }
  __syncthreads();
  s.st = s.s1 = 0.0f;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    s.st += sh.st[w];
    s.s1 += MODE != kOne ? sh.s1[w] : sh.st[w];
    s.ysum += sh.ysum[w];
    s.dot += sh.dot[w];
    if constexpr (PART) s.part += sh.part[w];
    s.ent += sh.ent[w];
  }
}

// The row's loss from its sums; s.dot over all entries, z_label the label's
// logit.  Log-sums and logits are both taken from the row's maximum: their
// difference then keeps its digits however far the row lies from zero.
template <int MODE>
__device__ __forceinline__ float row_loss(const DistillArgs& a, const Sums& s, const Expo<MODE>& x, double st, double s1,
                                          bool has_kd, bool has_ce, float z_label, float w) {
  double loss = 0.0;
  if (has_kd)
    loss += a.kd * static_cast<double>(a.temperature) * a.temperature *
            (s.ent / s.ysum - log(s.ysum) + kLn2 * (x.behind(false) + log2(st) - s.dot / s.ysum * x.s2));
  if (has_ce)
    loss += a.ce * kLn2 * (x.behind(true) + log2(s1) - (static_cast<double>(z_label) - origin(s.top)) * kLog2e);
  return static_cast<float>(w * loss);
}

// Zeros for a row that has nothing to say.
template <int DT, int THREADS, bool STREAM>
__device__ __forceinline__ void zero_row(const DistillArgs& a, int64_t row, int64_t i0, int64_t i1) {
  using T = typename OpElem<DT>::T;
  constexpr int C = 16 / sizeof(T);
  if (i0 == 0 && threadIdx.x == 0) gmem(a.losses)[row] = 0.0f;
  if (!a.dlogits) return;
  T* dz = static_cast<T*>(a.dlogits) + row * a.dstride;
  const int64_t whole = i0 + (i1 - i0) / C * C;
  const float none[C] = {};
  for (int64_t i = i0 + threadIdx.x * C; i < whole; i += THREADS * C) store_any<C, STREAM>(dz + i, none);
  for (int64_t i = whole + threadIdx.x; i < i1; i += THREADS) gmem(dz)[i] = static_cast<T>(0.0f);
}

// The gradient of [i0, i1) of a row.  `sh` holds the named elements' indices,
// weights and, for those in [i0, i1), logits (dlogits may overwrite them).
template <int DT, int MODE, int THREADS, bool STREAM, int PER, int R, int L>
__device__ __forceinline__ void row_grad(const DistillArgs& a, int64_t row, int64_t i0, int64_t i1,
                                         const Shared<THREADS, PER>& sh, const Expo<MODE>& x, double st, double s1,
                                         double ysum, bool has_kd, bool has_ce, float w,
                                         Held<typename OpElem<DT>::T, THREADS, R, L>& held) {
  using T = typename OpElem<DT>::T;
  const T* z = static_cast<const T*>(a.logits) + row * a.stride;
  T* dz = static_cast<T*>(a.dlogits) + row * a.dstride;
  const float scale = a.grad_scale * w;
  const float kdt = has_kd ? scale * a.kd * a.temperature : 0.0f;
  const float cew = has_ce ? scale * a.ce : 0.0f;
  // one coefficient serves both terms when they share the exponent
  const float ct = MODE == kOne ? static_cast<float>((static_cast<double>(kdt) + cew) / st)
                   : has_kd     ? static_cast<float>(kdt / st)
                                : 0.0f;
  const float c1 = MODE != kOne && has_ce ? static_cast<float>(cew / s1) : 0.0f;
  auto soft = [&](float v, auto far) {
    float et, e1;
    x.template both<decltype(far)::value>(v, &et, &e1);
    if constexpr (MODE == kOne) return ct * et;
    else return fmaf(c1, e1, ct * et);
  };
  auto write = [&](auto far) {
    return [&](const float* v, int64_t i, auto count) {
      constexpr int N = decltype(count)::value;
      float g[N];
#pragma unroll
      for (int e = 0; e < N; ++e) g[e] = soft(v[e], decltype(far){});
      if constexpr (N > 1) store_any<N, STREAM>(dz + i, g);
      else gmem(dz)[i] = static_cast<T>(g[0]);
    };
  };
  if (x.far) sweep<T, THREADS, 1>(z, i0, i1, write(std::true_type{}));
  else sweep_held<true>(z, i0, i1, held, write(std::false_type{}));
  __syncthreads();
  // named elements: the first entry that names one collects all that do
  for (int j = threadIdx.x; j <= a.k; j += THREADS) {
    const int i = sh.idx[j];
    if (i < i0 || i >= i1) continue;
    bool first = true;
    for (int h = 0; h < j && first; ++h) first = sh.idx[h] != i;
    if (!first) continue;
    double q = 0.0;
    for (int h = j; h < a.k; ++h)
      if (sh.idx[h] == i) q += sh.e[h];
    const float off = (has_kd ? kdt * static_cast<float>(q / ysum) : 0.0f) + (has_ce && sh.idx[a.k] == i ? cew : 0.0f);
    const float g = x.far ? soft(sh.z[j], std::true_type{}) : soft(sh.z[j], std::false_type{});
    gmem(dz)[i] = static_cast<T>(g - off);
  }
}

__device__ __forceinline__ float weight_of(const DistillArgs& a, int64_t row) {
  return a.row_weight ? gmem(a.row_weight)[row] : 1.0f;
}

// One block, one row.
template <int DT, int MODE, int THREADS, bool STREAM, int PER, int R>
__global__ __launch_bounds__(THREADS, 4) void distill_row_kernel(DistillArgs a) {
  __shared__ Shared<THREADS, PER> sh;
  const int64_t row = blockIdx.x;
  const float w = weight_of(a, row);
  if (w == 0.0f) {
    zero_row<DT, THREADS, STREAM>(a, row, 0, a.vocab);
    return;
  }
  constexpr int L = THREADS == 512 && R > 0 ? kStash : 0;
  __shared__ uint4 stash[L > 0 ? L * THREADS : 1];
  Held<typename OpElem<DT>::T, THREADS, R, L> held;
  held.stash = stash;
  Sums s;
  row_sums<DT, MODE, THREADS, PER, false>(a, row, 0, a.vocab, sh, s, held);
  const bool has_kd = a.kd != 0.0f && !(s.ysum == 0.0), has_ce = sh.idx[a.k] >= 0;
  if (!has_kd && !has_ce) {
    zero_row<DT, THREADS, STREAM>(a, row, 0, a.vocab);
    return;
  }
  Expo<MODE> x;
  x.set(s.top, scale_of(a));
  if (threadIdx.x == 0) gmem(a.losses)[row] = row_loss(a, s, x, s.st, s.s1, has_kd, has_ce, sh.z[a.k], w);
  if (a.dlogits)
    row_grad<DT, MODE, THREADS, STREAM, PER>(a, row, 0, a.vocab, sh, x, s.st, s.s1, s.ysum, has_kd, has_ce, w, held);
}

// Words of a slice's sums.
enum { kPmMax = 0, kPmSumT, kPmSum1, kPmDotHi, kPmDotLo, kPmPart, kPmLabel, kPmWords = 8 };
constexpr int kSliceThreads = 256, kSlicePer = kDistillMaxK / kSliceThreads + 1;

template <int DT, int MODE>
__global__ __launch_bounds__(kSliceThreads) void distill_slice_kernel(DistillArgs a) {
  __shared__ Shared<kSliceThreads, kSlicePer> sh;
  const int64_t row = blockIdx.x / a.slices;
  const int slice = static_cast<int>(blockIdx.x - row * a.slices);
  if (weight_of(a, row) == 0.0f) return;
  const int64_t i0 = least(a.vocab, slice * a.slice_len), i1 = least(a.vocab, i0 + a.slice_len);
  Sums s;
  Held<typename OpElem<DT>::T, kSliceThreads, 0, 0> none;
  row_sums<DT, MODE, kSliceThreads, kSlicePer, true>(a, row, i0, i1, sh, s, none);
  if (threadIdx.x == 0) {
    float* p = a.part + blockIdx.x * static_cast<int64_t>(kPmWords);
    p[kPmMax] = s.top;
    p[kPmSumT] = s.st;
    p[kPmSum1] = s.s1;
    const float hi = static_cast<float>(s.dot);
    p[kPmDotHi] = hi;
    p[kPmDotLo] = isfinite(hi) ? static_cast<float>(s.dot - hi) : 0.0f;
    p[kPmPart] = s.part;
    p[kPmLabel] = sh.z[a.k];   // 0 outside this slice
  }
}

// Joins a row's slices, writes the loss (first slice) and this slice's gradient.
template <int DT, int MODE>
__global__ __launch_bounds__(kSliceThreads) void distill_join_kernel(DistillArgs a) {
  using T = typename OpElem<DT>::T;
  __shared__ Shared<kSliceThreads, kSlicePer> sh;
  const int64_t row = a.dlogits ? blockIdx.x / a.slices : blockIdx.x;
  const int slice = a.dlogits ? static_cast<int>(blockIdx.x - row * a.slices) : 0;
  const int64_t i0 = least(a.vocab, slice * a.slice_len), i1 = least(a.vocab, i0 + a.slice_len);
  const float w = weight_of(a, row);
  if (w == 0.0f) {
    zero_row<DT, kSliceThreads, false>(a, row, i0, i1);
    return;
  }
  // the teacher's entries again: sums over no elements
  Sums s;
  Held<T, kSliceThreads, 0, 0> none;
  row_sums<DT, MODE, kSliceThreads, kSlicePer, false>(a, row, 0, 0, sh, s, none);
  const bool has_kd = a.kd != 0.0f && !(s.ysum == 0.0), has_ce = sh.idx[a.k] >= 0;
  if (!has_kd && !has_ce) {
    zero_row<DT, kSliceThreads, false>(a, row, i0, i1);
    return;
  }
  const T* z = static_cast<const T*>(a.logits) + row * a.stride;
  if (a.dlogits)   // before dlogits (which may be logits) is written
    for (int j = threadIdx.x; j <= a.k; j += kSliceThreads)
      if (sh.idx[j] >= i0 && sh.idx[j] < i1) sh.z[j] = static_cast<float>(gmem(z)[sh.idx[j]]);
  // a lane per slice (at most 64), the same in every wave
  const int lane = threadIdx.x & 63;
  const float* p = a.part + (row * a.slices + least(lane, a.slices - 1)) * kPmWords;
  const bool on = lane < a.slices;
  const float top = on ? gmem(p)[kPmMax] : -INFINITY;
  s.top = wave_max(top);
  Expo<MODE> x, y;
  x.set(s.top, scale_of(a));
  y.set(top, x.s2);
  // from a slice's references to the row's; either may be in either form
  float ft = 0.0f, f1 = 0.0f;   // a slice of nothing but -inf
  if (top != -INFINITY) {
    ft = __builtin_amdgcn_exp2f(static_cast<float>(y.zero(false) - x.zero(false)));
    f1 = MODE == kOne ? ft : __builtin_amdgcn_exp2f(static_cast<float>(y.zero(true) - x.zero(true)));
  }
  const double st = wave_sum(on ? static_cast<double>(gmem(p)[kPmSumT]) * ft : 0.0);
  const double s1 = wave_sum(on ? static_cast<double>(gmem(p)[kPmSum1]) * f1 : 0.0);
  s.dot = wave_sum(on ? static_cast<double>(gmem(p)[kPmDotHi]) + static_cast<double>(gmem(p)[kPmDotLo]) +
                            gmem(p)[kPmPart] * (static_cast<double>(origin(top)) - origin(s.top))   // to the row's origin
                      : 0.0);
  const float z_label = wave_sum(on ? gmem(p)[kPmLabel] : 0.0f);
  if (slice == 0 && threadIdx.x == 0) gmem(a.losses)[row] = row_loss(a, s, x, st, s1, has_kd, has_ce, z_label, w);
  if (!a.dlogits) return;
  __syncthreads();   // every named logit is read
  row_grad<DT, MODE, kSliceThreads, false, kSlicePer>(a, row, i0, i1, sh, x, st, s1, s.ysum, has_kd, has_ce, w, none);
}

}  // namespace

hipError_t launch_distill(int dt, const DistillArgs& a, hipStream_t stream) {
  if (a.n == 0) return hipSuccess;
  const bool two = a.kd != 0.0f && a.ce != 0.0f && a.temperature != 1.0f;
  const int mode = !two ? kOne : a.temperature == 2.0f ? kSquare : a.temperature == 4.0f ? kFourth : kTwo;
  const double row_bytes = static_cast<double>(a.vocab) * (dt == kBF16 ? 2 : 4);
  const bool streams = a.dlogits && row_bytes * a.n * 2 > 256e6;
  // Threads of a row's block.  Rows of up to 12 KB: one wave, which needs no
  // barriers (8192 rows of 4001 bf16: 40 us, 53 with 256 threads); up to 64 KB:
  // 256, most of the row in registers (16000 bf16: 111 us, 126 without); longer
  // ones: 512 and two blocks to a CU, so that the rows in work stay in the 256 MB
  // memory-side cache for their second reading (50257 bf16: 209 us for 4000 rows,
  // 240 with 256 threads; 128256 fp32: 911 us for 4096 rows, 925 with 1024).  Few
  // rows alone on the chip take 1024 early.
  const int threads = a.n <= 128 ? (row_bytes > 16384.0 ? 1024 : 256)
                      : row_bytes <= 12288.0 && a.k < 256 ? 64 : row_bytes <= 65536.0 ? 256 : 512;
  auto launch = [&](auto d, auto m) {
    constexpr int D = decltype(d)::value, M = decltype(m)::value;
    if (a.slices > 0) {
      const dim3 grid(static_cast<unsigned>(a.n * a.slices));
      hipLaunchKernelGGL((distill_slice_kernel<D, M>), grid, dim3(kSliceThreads), 0, stream, a);
      hipLaunchKernelGGL((distill_join_kernel<D, M>), a.dlogits ? grid : dim3(static_cast<unsigned>(a.n)),
                         dim3(kSliceThreads), 0, stream, a);
    } else {
      const dim3 grid(static_cast<unsigned>(a.n));
      auto rows = [&](auto t, auto st, auto per, auto r) {
        constexpr int N = decltype(t)::value;
        hipLaunchKernelGGL((distill_row_kernel<D, M, N, decltype(st)::value, decltype(per)::value, decltype(r)::value>),
                           grid, dim3(N), 0, stream, a);
      };
      auto by_stream = [&](auto t, auto per, auto r) {
        if (streams) rows(t, std::true_type{}, per, r);
        else rows(t, std::false_type{}, per, r);
      };
      // without a gradient nothing is read again: no vectors held, more rows in flight
      if (threads == 1024) rows(Int<1024>{}, std::false_type{}, Int<2>{}, Int<0>{});
      else if (!a.dlogits && threads == 512) rows(Int<512>{}, std::false_type{}, Int<3>{}, Int<0>{});
      else if (!a.dlogits && threads == 256) rows(Int<256>{}, std::false_type{}, Int<5>{}, Int<0>{});
      else if (!a.dlogits) rows(Int<64>{}, std::false_type{}, Int<4>{}, Int<0>{});
      else if (threads == 512) by_stream(Int<512>{}, Int<3>{}, Int<kHeld>{});
      else if (threads == 256 && row_bytes > 36e3) by_stream(Int<256>{}, Int<5>{}, Int<kHeld>{});
      else if (threads == 256) by_stream(Int<256>{}, Int<5>{}, Int<8>{});
      else if (row_bytes > 4096.0) by_stream(Int<64>{}, Int<4>{}, Int<kHeld>{});
      else by_stream(Int<64>{}, Int<4>{}, Int<4>{});
    }
  };
  auto by_mode = [&](auto d) {
    if (mode == kOne) launch(d, std::integral_constant<int, kOne>{});
    else if (mode == kTwo) launch(d, std::integral_constant<int, kTwo>{});
    else if (mode == kSquare) launch(d, std::integral_constant<int, kSquare>{});
    else launch(d, std::integral_constant<int, kFourth>{});
  };
  if (dt == kBF16) by_mode(std::integral_constant<int, kBF16>{});
  else by_mode(std::integral_constant<int, kF32>{});
  return hipGetLastError();
}

}  // namespace dmuon
