// Shared definitions for the fused multi-tensor AdamW step (host planner and kernel).
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.hpp"

namespace dmuon {

constexpr int kAdamChunk = 4;                                   // consecutive elements per lane and load
constexpr int kAdamChunks = 4;                                  // chunks per lane and tile
constexpr int kAdamThreads = 256;
constexpr int kAdamTile = kAdamThreads * kAdamChunk * kAdamChunks;  // 4096 elements

// One parameter tensor; lives in the workspace.
struct alignas(16) AdamDesc {
  void* p;          // device, numel contiguous elements of the parameter dtype
  const void* g;    // device, same dtype and size as p
  float* m;         // device, numel floats (first moment)
  float* v;         // device, numel floats (second moment)
  int64_t numel;
  int vec_ok;       // 1 when p and g hold whole aligned chunks and m, v are 16-byte aligned
  int pad_;
};
static_assert(sizeof(AdamDesc) == 48, "AdamDesc layout");

// Per-call constants, formed on the host from the step counter and hyper-parameters.
struct AdamArgs {
  float decay;         // 1 - lr * weight_decay
  float beta1, one_minus_beta1;
  float beta2, one_minus_beta2;
  float step_size;     // lr / (1 - beta1^t)
  float inv_bc2_sqrt;  // 1 / sqrt(1 - beta2^t)
  float eps;
};

// Bias corrections and the decay factor in double, each rounded once.
inline AdamArgs adam_args(int step, float lr, float beta1, float beta2, float eps, float weight_decay) {
  const double t = static_cast<double>(step);
  AdamArgs a{};
  a.decay = static_cast<float>(1.0 - static_cast<double>(lr) * static_cast<double>(weight_decay));
  a.beta1 = beta1;
  a.one_minus_beta1 = static_cast<float>(1.0 - static_cast<double>(beta1));
  a.beta2 = beta2;
  a.one_minus_beta2 = static_cast<float>(1.0 - static_cast<double>(beta2));
  a.step_size = static_cast<float>(static_cast<double>(lr) / (1.0 - pow(static_cast<double>(beta1), t)));
  a.inv_bc2_sqrt = static_cast<float>(1.0 / sqrt(1.0 - pow(static_cast<double>(beta2), t)));
  a.eps = eps;
  return a;
}

#if defined(__HIPCC__)
// One element's step, shared by the dense step and the step on row gradients.
__device__ __forceinline__ void adamw_elem(float& p, float g, float& m, float& v, const AdamArgs& a) {
  p *= a.decay;
  m = fmaf(a.beta1, m, a.one_minus_beta1 * g);
  v = fmaf(a.beta2, v, (a.one_minus_beta2 * g) * g);
  const float denom = fmaf(sqrtf(v), a.inv_bc2_sqrt, a.eps);
  p = fmaf(-a.step_size, m / denom, p);
}
#endif

hipError_t launch_adamw(int dt, const AdamDesc* descs, const int* tile_prefix, int n, int total_tiles,
                        const AdamArgs& args, int grid, hipStream_t stream);

}  // namespace dmuon
