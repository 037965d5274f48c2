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
// A row is cut into slices.  distill_stats_kernel reads each slice once and
// leaves its running maximum, its sums of exponentials relative to that maximum
// and its part of sum_j e_j z_j; distill_grad_kernel joins the slices of its
// row, writes the loss, and rewrites its slice as the gradient: first the
// softmax terms of every element, then, behind a barrier, the at most k + 1
// elements that the teacher or the label name.  HBM-bound: one or two
// exponentials per element against 2 or 4 bytes each way.
//
// Sums of exponentials are fp32; the few scalars of a row are joined in fp64,
// so that the loss is exact to the fp32 sums although it is a difference of
// terms that grow with the vocabulary.
#include <hip/hip_runtime.h>

#include "ops.hpp"

namespace dmuon {
namespace {

constexpr int kDsThreads = 256;
constexpr int kDsWaves = kDsThreads / 64;
constexpr float kLog2e = 1.4426950408889634f;

// Words of a slice's partial result.
enum { kPmMax = 0, kPmSumT, kPmSum1, kPmDotHi, kPmDotLo, kPmLabel, kPmWords = 8 };

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

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
__device__ __forceinline__ float block_max(float v, float* red) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = red[0];
#pragma unroll
  for (int w = 1; w < kDsWaves; ++w) r = fmaxf(r, red[w]);
  __syncthreads();
  return r;
}
template <typename F> __device__ __forceinline__ F block_sum(F v, F* red) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  F r = red[0];
#pragma unroll
  for (int w = 1; w < kDsWaves; ++w) r += red[w];
  __syncthreads();
  return r;
}

// exp((a - b) s) where an empty sum has maximum -inf
__device__ __forceinline__ float rescale(float a, float b, float s2) {
  return a == -INFINITY ? 0.0f : exp2_fast((a - b) * s2);
}

// The teacher's entries of one row: indices (or -1), unnormalised weights
// e_j = exp((y_j - max) / T) and their sum.
struct Teacher {
  int64_t idx[kDistillMaxK];
  float e[kDistillMaxK];
};
__device__ __forceinline__ void load_teacher(const DistillArgs& a, int64_t row, Teacher& t, float* red, double* dred,
                                             float* top, double* sum) {
  float m = -INFINITY;
  for (int j = threadIdx.x; j < a.k; j += kDsThreads) {
    const int64_t i = load_index(a.index, row * a.k + j, a.idx64);
    const float y = gmem(a.teacher)[row * a.k + j];
    const bool ok = i >= 0 && i < a.vocab;
    t.idx[j] = ok ? i : -1;
    t.e[j] = ok ? y : -INFINITY;
    // a NaN has to reach the sum
    if (ok) m = fmaxf(m, y);
  }
  m = block_max(m, red);
  double s = 0.0;
  for (int j = threadIdx.x; j < a.k; j += kDsThreads) {
    const float e = t.e[j] == -INFINITY ? 0.0f : expf((t.e[j] - m) / a.temperature);
    t.e[j] = e;
    s += e;
  }
  *sum = block_sum(s, dred);   // its barriers also publish t
  *top = m;
}

template <int DT, bool DUAL>
__global__ __launch_bounds__(kDsThreads) void distill_stats_kernel(DistillArgs a) {
  using T = typename OpElem<DT>::T;
  constexpr int C = DT == kBF16 ? 8 : 4;
  constexpr int U = 4;
  __shared__ Teacher teacher;
  __shared__ float red[kDsWaves];
  __shared__ double dred[kDsWaves];
  const int64_t row = blockIdx.x / a.slices;
  const int slice = static_cast<int>(blockIdx.x - row * a.slices);
  if (a.row_weight && gmem(a.row_weight)[row] == 0.0f) return;
  const T* z = static_cast<const T*>(a.logits) + row * a.stride;
  const int64_t i0 = slice * a.slice_len, i1 = min(a.vocab, i0 + a.slice_len);
  const float s2t = kLog2e / a.temperature;
  const float s2 = a.kd != 0.0f ? s2t : kLog2e;   // the only scale unless DUAL
  float m = -INFINITY, st = 0.0f, s1 = 0.0f;
  auto add = [&](const float* v, int count) {
    float top = m;
    for (int e = 0; e < count; ++e) top = fmaxf(top, v[e]);
    if (top > m) {
      st *= rescale(m, top, s2);
      if (DUAL) s1 *= rescale(m, top, kLog2e);
      m = top;
    }
    for (int e = 0; e < count; ++e) {
      // nothing to add for -inf: (-inf) - (-inf) is no number
      const float d = v[e] == -INFINITY ? -INFINITY : v[e] - m;
      st += exp2_fast(d * s2);
      if (DUAL) s1 += exp2_fast(d * kLog2e);
    }
  };
  if (a.vec) {
    const int64_t whole = i0 + (i1 - i0) / C * C;
    for (int64_t i = i0 + threadIdx.x * C; i < whole; i += kDsThreads * C * U) {
      float v[U][C];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t p = i + static_cast<int64_t>(u) * kDsThreads * C;
        if (p < whole) load_n<C>(z + p, v[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + static_cast<int64_t>(u) * kDsThreads * C < whole) add(v[u], C);
    }
    for (int64_t i = whole + threadIdx.x; i < i1; i += kDsThreads) {
      const float v = static_cast<float>(gmem(z)[i]);
      add(&v, 1);
    }
  } else {
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kDsThreads) {
      const float v = static_cast<float>(gmem(z)[i]);
      add(&v, 1);
    }
  }
  const float top = block_max(m, red);
  st = block_sum(st * rescale(m, top, s2), red);
  if (DUAL) s1 = block_sum(s1 * rescale(m, top, kLog2e), red);
  double dot = 0.0;
  if (a.kd != 0.0f) {
    float ymax;
    double ysum;
    load_teacher(a, row, teacher, red, dred, &ymax, &ysum);
    for (int j = threadIdx.x; j < a.k; j += kDsThreads) {
      const int64_t i = teacher.idx[j];
      if (i >= i0 && i < i1 && teacher.e[j] != 0.0f)
        dot += static_cast<double>(teacher.e[j]) * static_cast<double>(static_cast<float>(gmem(z)[i]));
    }
    dot = block_sum(dot, dred);
  }
  if (threadIdx.x == 0) {
    float* p = a.part + blockIdx.x * static_cast<int64_t>(kPmWords);
    const int64_t label = a.labels ? load_index(a.labels, row, a.idx64) : -1;
    p[kPmMax] = top;
    p[kPmSumT] = st;
    p[kPmSum1] = DUAL ? s1 : st;
    const float hi = static_cast<float>(dot);
    p[kPmDotHi] = hi;
    p[kPmDotLo] = isfinite(hi) ? static_cast<float>(dot - hi) : 0.0f;
    p[kPmLabel] = label >= i0 && label < i1 ? static_cast<float>(gmem(z)[label]) : 0.0f;
  }
}

template <int DT, bool DUAL>
__global__ __launch_bounds__(kDsThreads) void distill_grad_kernel(DistillArgs a) {
  using T = typename OpElem<DT>::T;
  constexpr int C = DT == kBF16 ? 8 : 4;
  __shared__ Teacher teacher;
  __shared__ float red[kDsWaves];
  __shared__ double dred[kDsWaves];
  __shared__ float zsel[kDistillMaxK + 1];
  const int64_t row = blockIdx.x / a.slices;
  const int slice = static_cast<int>(blockIdx.x - row * a.slices);
  const float w = a.row_weight ? gmem(a.row_weight)[row] : 1.0f;
  const int64_t i0 = slice * a.slice_len, i1 = min(a.vocab, i0 + a.slice_len);
  const T* z = static_cast<const T*>(a.logits) + row * a.stride;
  T* dz = a.dlogits ? static_cast<T*>(a.dlogits) + row * a.dstride : nullptr;
  const int tid = threadIdx.x;

  auto zero_row = [&]() {
    if (slice == 0 && tid == 0) gmem(a.losses)[row] = 0.0f;
    if (!dz) return;
    const int64_t whole = a.vec ? i0 + (i1 - i0) / C * C : i0;
    const float none[C] = {};
    for (int64_t i = i0 + tid * C; i < whole; i += kDsThreads * C) store_n<C>(dz + i, none);
    for (int64_t i = whole + tid; i < i1; i += kDsThreads) gmem(dz)[i] = static_cast<T>(0.0f);
  };
  if (w == 0.0f) {
    zero_row();
    return;
  }
  float ymax = -INFINITY;
  double ysum = 0.0;
  if (a.kd != 0.0f) load_teacher(a, row, teacher, red, dred, &ymax, &ysum);
  const bool has_kd = a.kd != 0.0f && !(ysum == 0.0);
  const int64_t label = a.labels ? load_index(a.labels, row, a.idx64) : -1;
  const bool has_ce = a.ce != 0.0f && label >= 0 && label < a.vocab;
  if (!has_kd && !has_ce) {   // neither term has anything to say about this row
    zero_row();
    return;
  }
  // join the slices of this row
  float m = -INFINITY, zl = 0.0f;
  const float* part = a.part + row * a.slices * kPmWords;
  for (int s = 0; s < a.slices; ++s) m = fmaxf(m, gmem(part)[s * kPmWords + kPmMax]);
  const float s2t = kLog2e / a.temperature;
  const float s2 = a.kd != 0.0f ? s2t : kLog2e;
  double st = 0.0, s1 = 0.0, dot = 0.0;
  for (int s = 0; s < a.slices; ++s) {
    const float* p = part + s * kPmWords;
    const float ms = gmem(p)[kPmMax];
    st += static_cast<double>(gmem(p)[kPmSumT]) * rescale(ms, m, s2);
    s1 += static_cast<double>(gmem(p)[kPmSum1]) * rescale(ms, m, DUAL ? kLog2e : s2);
    dot += static_cast<double>(gmem(p)[kPmDotHi]) + static_cast<double>(gmem(p)[kPmDotLo]);
    zl += gmem(p)[kPmLabel];
  }
  if (slice == 0) {
    double loss = 0.0;
    if (has_kd) {
      const double temp = a.temperature;
      double h = 0.0;
      for (int j = tid; j < a.k; j += kDsThreads)
        if (teacher.e[j] != 0.0f) h += static_cast<double>(teacher.e[j]) * log(static_cast<double>(teacher.e[j]) / ysum);
      h = block_sum(h, dred) / ysum;
      loss += a.kd * temp * temp * (h - dot / (ysum * temp) + static_cast<double>(m) / temp + log(st));
    }
    if (has_ce) loss += a.ce * (static_cast<double>(m) + log(s1) - static_cast<double>(zl));
    if (tid == 0) gmem(a.losses)[row] = static_cast<float>(w * loss);
  }
  if (!dz) return;
  const float scale = a.grad_scale * w;
  const float kdt = has_kd ? scale * a.kd * a.temperature : 0.0f;
  const float cew = has_ce ? scale * a.ce : 0.0f;
  // one coefficient serves both terms when they share the exponent
  const float ct = DUAL ? (has_kd ? static_cast<float>(kdt / st) : 0.0f) : static_cast<float>((static_cast<double>(kdt) + cew) / st);
  const float c1 = DUAL && has_ce ? static_cast<float>(cew / s1) : 0.0f;
  auto soft = [&](float v) {
    const float d = v - m;
    float g = ct == 0.0f ? 0.0f : ct * exp2_fast(d * s2);
    if (DUAL && c1 != 0.0f) g = fmaf(c1, exp2_fast(d * kLog2e), g);
    return g;
  };
  // the named elements' logits, before dlogits (which may be logits) is written
  const int entries = a.k + 1;
  for (int j = tid; j < entries; j += kDsThreads) {
    const int64_t i = j < a.k ? (has_kd ? teacher.idx[j] : -1) : (has_ce ? label : -1);
    zsel[j] = i >= i0 && i < i1 ? static_cast<float>(gmem(z)[i]) : 0.0f;
  }
  __syncthreads();
  const int64_t whole = a.vec ? i0 + (i1 - i0) / C * C : i0;
  for (int64_t i = i0 + tid * C; i < whole; i += kDsThreads * C) {
    float v[C];
    load_n<C>(z + i, v);
#pragma unroll
    for (int e = 0; e < C; ++e) v[e] = soft(v[e]);
    store_n<C>(dz + i, v);
  }
  for (int64_t i = whole + tid; i < i1; i += kDsThreads) gmem(dz)[i] = static_cast<T>(soft(static_cast<float>(gmem(z)[i])));
  __syncthreads();
  // named elements: the first entry that names one collects all that do
  auto entry = [&](int j) -> int64_t { return j < a.k ? (has_kd ? teacher.idx[j] : -1) : (has_ce ? label : -1); };
  for (int j = tid; j < entries; j += kDsThreads) {
    const int64_t i = entry(j);
    if (i < i0 || i >= i1) continue;
    bool first = true;
    for (int h = 0; h < j && first; ++h) first = entry(h) != i;
    if (!first) continue;
    double q = 0.0;
    for (int h = j; h < a.k; ++h)
      if (entry(h) == i) q += teacher.e[h];
    const float off = (has_kd ? kdt * static_cast<float>(q / ysum) : 0.0f) + (has_ce && label == i ? cew : 0.0f);
    gmem(dz)[i] = static_cast<T>(soft(zsel[j]) - off);
  }
}

}  // namespace

hipError_t launch_distill(int dt, const DistillArgs& a, hipStream_t stream) {
  if (a.n == 0) return hipSuccess;
  const bool dual = a.kd != 0.0f && a.ce != 0.0f && a.temperature != 1.0f;
  const dim3 grid(static_cast<unsigned>(a.n * a.slices));
  auto go = [&](auto stats, auto grad) {
    hipLaunchKernelGGL(stats, grid, dim3(kDsThreads), 0, stream, a);
    hipLaunchKernelGGL(grad, grid, dim3(kDsThreads), 0, stream, a);
  };
  if (dt == kBF16) {
    if (dual) go(distill_stats_kernel<kBF16, true>, distill_grad_kernel<kBF16, true>);
    else go(distill_stats_kernel<kBF16, false>, distill_grad_kernel<kBF16, false>);
  } else {
    if (dual) go(distill_stats_kernel<kF32, true>, distill_grad_kernel<kF32, true>);
    else go(distill_stats_kernel<kF32, false>, distill_grad_kernel<kF32, false>);
  }
  return hipGetLastError();
}

}  // namespace dmuon
