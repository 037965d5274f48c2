// Shared definitions between the host entry points (dmuon_ops_api.cpp) and the
// kernels of the operators beside the optimizer step: embedding, row-gradient
// AdamW, distillation loss, query/key norm with rotation.
//
// Every argument travels by value in the kernel's argument block: nothing is
// uploaded, so these launches can be recorded into a graph.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "adamw.hpp"
#include "common.hpp"

namespace dmuon {

// ---------------------------------------------------------------- embedding
struct EmbedArgs {
  const void* table;
  const void* tokens;
  void* out;
  int64_t n, vocab, dim;
  float scale;
  int tok64;   // tokens are int64 (else int32)
};
hipError_t launch_embed(int table_dt, int out_dt, const EmbedArgs& a, hipStream_t stream);

// Stable sort of the tokens and the row lists derived from it.
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanMaxDigits = 512;      // 9 bits a pass
constexpr int kPlanSmall = 4096;         // tokens sorted by one block in LDS
constexpr int kPlanMaxBlocks = 128;

struct PlanArgs {
  const void* tokens;
  int64_t vocab;
  int n, tok64;
  int cap;              // min(n, vocab): length of rows
  int bits;             // digit width of a pass
  int passes;
  int items;            // tokens per block (multiple of kPlanThreads)
  int blocks;
  int* order;
  int* slot;
  int* rows;
  int* row_index;
  int* count;
  // workspace
  unsigned* key[2];
  int* idx[2];
  int* counts;          // blocks x 2^bits
  int* heads;           // blocks
};
hipError_t launch_embed_plan(const PlanArgs& a, hipStream_t stream);

enum EmbedGradForm : int { kGradDense = 0, kGradAdd = 1, kGradRows = 2 };
constexpr int kEgThreads = 256;
constexpr int kEgZeroRows = 4;   // rows a zero-filling block looks after

struct EmbedGradArgs {
  const void* dout;
  const int* order;
  const int* slot;
  const int* rows;
  const int* row_index;
  const int* count;
  void* grad;
  float* part;          // 2 x chunks x dim: a chunk's first and last unfinished sums
  int64_t n, vocab, dim;
  float scale;
  int cap;
  int form;
  int chunk;            // sorted positions per chunk
  int chunks;
};
hipError_t launch_embed_grad(int dout_dt, int grad_dt, const EmbedGradArgs& a, hipStream_t stream);

// ---------------------------------------------------------------- AdamW, gradient as rows
struct AdamRowsArgs {
  void* p;
  const void* g;
  const int* row_index;
  float* m;
  float* v;
  int64_t rows, dim, n_grad_rows;
  AdamArgs hp;
};
hipError_t launch_adamw_rows(int dt, const AdamRowsArgs& a, hipStream_t stream);

// ---------------------------------------------------------------- distillation loss
constexpr int kDistillMaxK = 1024;
struct DistillArgs {
  const void* logits;
  const void* index;
  const float* teacher;
  const void* labels;      // nullptr: no labels
  const float* row_weight; // nullptr: 1
  float* losses;
  void* dlogits;           // nullptr: loss only
  float* part;             // n x slices x 8 (slices > 0)
  int64_t n, vocab, stride, dstride;
  int k, idx64;
  int slices;              // 0: a block takes a whole row; else blocks per row
  int64_t slice_len;
  float temperature, kd, ce, grad_scale;
};
hipError_t launch_distill(int dt, const DistillArgs& a, hipStream_t stream);

// ---------------------------------------------------------------- query / key norm with rotation
struct QkArgs {
  const void* x[2];        // q, k
  const void* dy[2];       // backward: gradients of the outputs
  void* out[2];            // forward: outputs; backward: gradients of the inputs
  const void* w[2];        // gains or nullptr
  void* dw[2];             // backward: gradients of the gains, or nullptr
  int64_t x_stride[2], dy_stride[2], out_stride[2];   // elements between tokens
  int heads[2];
  const void* positions;   // nullptr: rot is 0 and no token is padding
  const float* rope;       // max_pos x rot: cosines, then sines
  float* part;             // backward: (blocks[0] + blocks[1]) x head_dim
  int64_t n, max_pos;
  int dim, rot, interleaved, pos64;
  float eps, offset;
  int pairs;               // pairs of a head that a lane holds: 8 or 4, by type and shape alone
  int vec;                 // ... loaded at once (else one element at a time)
  int rope_vec;            // the table's rows hold aligned runs of four
  int blocks[2];           // backward: blocks of each tensor
  int log_heads[2];        // set by the launch: log2 of the heads, rounded up
};
hipError_t launch_qk_norm(int dt, int w_dt, const QkArgs& a, hipStream_t stream);
hipError_t launch_qk_norm_grad(int dt, int w_dt, const QkArgs& a, hipStream_t stream);

#if defined(__HIPCC__)
// Of integers of one type: `min` and `max` of 64-bit integers may go through floating point.
template <typename T> __device__ __forceinline__ T least(T a, T b) { return a < b ? a : b; }
template <typename T> __device__ __forceinline__ T most(T a, T b) { return a > b ? a : b; }

// An index array's entry, int32 or int64.
__device__ __forceinline__ int64_t load_index(const void* p, int64_t i, int is64) {
  return is64 ? gmem(static_cast<const int64_t*>(p))[i] : static_cast<int64_t>(gmem(static_cast<const int*>(p))[i]);
}

template <int DT> struct OpElem;
template <> struct OpElem<kBF16> { using T = __bf16; };
template <> struct OpElem<kF32> { using T = float; };

typedef __bf16 bf16v8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16v4 __attribute__((ext_vector_type(4)));

// N consecutive elements (N = 4 or 8) to and from fp32.  load_n and store_n:
// the address is aligned to the whole (fp32: to 16 bytes).  load_any and
// store_any: aligned to one element; gfx950's global accesses take any address,
// at the price of a second cache line now and then.
template <typename T, int N> struct Loose {
  typedef T V __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};
// STREAM: non-temporal, for what does not fit the caches anyway.
template <int N, bool STREAM = false, typename T> __device__ __forceinline__ void load_any(const T* p, float* v) {
  constexpr int M = 16 / sizeof(T) < N ? 16 / sizeof(T) : N;
  using V = typename Loose<T, M>::V;
#pragma unroll
  for (int h = 0; h < N / M; ++h) {
    const auto q = reinterpret_cast<gptr<const V>>(gmem(p + M * h));
    V x;
    if constexpr (STREAM) x = __builtin_nontemporal_load(q);
    else x = *q;
#pragma unroll
    for (int e = 0; e < M; ++e) v[M * h + e] = static_cast<float>(x[e]);
  }
}
template <int N, bool STREAM = false, typename T> __device__ __forceinline__ void store_any(T* p, const float* v) {
  constexpr int M = 16 / sizeof(T) < N ? 16 / sizeof(T) : N;
  using V = typename Loose<T, M>::V;
#pragma unroll
  for (int h = 0; h < N / M; ++h) {
    V x;
#pragma unroll
    for (int e = 0; e < M; ++e) x[e] = static_cast<T>(v[M * h + e]);
    if constexpr (STREAM) __builtin_nontemporal_store(x, reinterpret_cast<gptr<V>>(gmem(p + M * h)));
    else *reinterpret_cast<gptr<V>>(gmem(p + M * h)) = x;
  }
}
template <int N> __device__ __forceinline__ void load_n(const float* p, float* v) {
#pragma unroll
  for (int h = 0; h < N / 4; ++h) {
    const f32v4 x = *reinterpret_cast<gptr<const f32v4>>(gmem(p + 4 * h));
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * h + e] = x[e];
  }
}
template <int N> __device__ __forceinline__ void load_n(const __bf16* p, float* v) {
  if constexpr (N == 8) {
    const bf16v8 x = *reinterpret_cast<gptr<const bf16v8>>(gmem(p));
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = static_cast<float>(x[e]);
  } else {
    const bf16v4 x = *reinterpret_cast<gptr<const bf16v4>>(gmem(p));
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(x[e]);
  }
}
// STREAM: non-temporal, for results that do not fit the caches anyway.
template <bool STREAM, typename V> __device__ __forceinline__ void store_vec(gptr<V> p, V x) {
  if constexpr (STREAM) __builtin_nontemporal_store(x, p);
  else *p = x;
}
template <int N, bool STREAM = false> __device__ __forceinline__ void store_n(float* p, const float* v) {
#pragma unroll
  for (int h = 0; h < N / 4; ++h)
    store_vec<STREAM>(reinterpret_cast<gptr<f32v4>>(gmem(p + 4 * h)), f32v4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]});
}
template <int N, bool STREAM = false> __device__ __forceinline__ void store_n(__bf16* p, const float* v) {
  typedef __bf16 V __attribute__((ext_vector_type(N)));
  V x;
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = static_cast<__bf16>(v[e]);
  store_vec<STREAM>(reinterpret_cast<gptr<V>>(gmem(p)), x);
}
#endif

}  // namespace dmuon
