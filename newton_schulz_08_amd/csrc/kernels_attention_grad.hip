// Gradients of attention over packed sequences, on gfx950 (MFMA-bound).
//
// With the forward's lse, the probabilities are formed again, tile by tile:
//
//   p  = exp(scale q . k - lse),       delta = dout . out  of each row
//   ds = p (dout . v - delta) scale
//   dq = sum over keys of ds k,   dk = sum over rows of ds q,   dv = sum of p dout
//
// Three launches.  The first forms delta and puts it beside lse.  dq's blocks keep
// a tile of rows (queries x the heads that share a key head) and pass over the
// keys; dk's and dv's keep a tile of keys and pass over the rows, those of all heads that
// share it, so a shared head's gradient is one sum in one block.  Each forms
// the scores for itself: seven products in all instead of five, but every sum
// has one owner and one order, with no atomics and no partial results in
// memory.
//
// Measured, 32 heads over 8 key heads of 128 bf16, causal, two sequences of 8192
// tokens: 4.2 to 4.75 ms on different cards (dk and dv 2.2 to 2.5, dq 2.0 to 2.2,
// statistics 0.055), 0.58 to 0.65 PFLOP/s of five products; with the two that are formed twice and dq's
// second operand 1.0.  In dk and dv a wave reads 368 LDS cycles a step of 32
// rows beside 1024 of matrix instructions, eight waves to one LDS: without
// barriers, exponentials or later loads it would still take 1.9 ms.  Eight
// waves on 256 keys with three buffers take 2.45 ms; 64 keys a wave, which would
// halve the reads, spill (13 ms).  Heads of 64 2.85 ms, of 192 13.1, of 256 36.2
// (151 registers of dk and dv spill: 29.6 of it).  fp32, 4096 tokens in two
// sequences: heads of 64 1.8 ms, of 128 3.6, of 192 11.8, of 256 21 (both with
// spills).
//
// Rows without visible keys (lse -infinity) take lse = +infinity, which makes
// their probabilities exp2(-infinity) = 0.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attention.hpp"

namespace dmuon {
namespace attn {
namespace {

// Where a row's base-2 log-sum-exp and delta lie: in the order of a key head's
// rows (token, head of the group), so that a tile's are one run.
__device__ __forceinline__ int64_t stat_of(const AttnArgs& a, int head, int64_t token, int g) {
  return 2 * ((static_cast<int64_t>(head) * a.q_tokens + token) * a.group + g);
}

// Runs of 16 bytes of (token, query head) rows; LANES lanes a row.
template <int DT, int LANES, bool VEC> __global__ __launch_bounds__(kThreads) void attention_stats_kernel(AttnArgs a) {
  using T = typename OpElem<DT>::T;
  constexpr int M = 16 / static_cast<int>(sizeof(T));
  typedef T V __attribute__((ext_vector_type(M)));
  const int64_t row = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * (kThreads / LANES) + threadIdx.x / LANES;
  const int64_t token = row / a.q_heads;
  const int h = static_cast<int>(row - token * a.q_heads), d = threadIdx.x % LANES * M;
  if (token >= a.q_tokens) return;
  const T* o = static_cast<const T*>(a.out) + token * a.os + static_cast<int64_t>(h) * a.dim;
  const T* g = static_cast<const T*>(a.dout) + token * a.dos + static_cast<int64_t>(h) * a.dim;
  float s = 0.0f;
  if constexpr (VEC) {
    if (d < a.dim) {
      const V x = *reinterpret_cast<gptr<const V>>(gmem(o + d)), y = *reinterpret_cast<gptr<const V>>(gmem(g + d));
#pragma unroll
      for (int i = 0; i < M; ++i) s += static_cast<float>(x[i]) * static_cast<float>(y[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < M; ++i)
      if (d + i < a.dim) s += static_cast<float>(gmem(o)[d + i]) * static_cast<float>(gmem(g)[d + i]);
  }
#pragma unroll
  for (int x = LANES / 2; x > 0; x >>= 1) s += __shfl_xor(s, x, 64);
  if (threadIdx.x % LANES) return;
  const float lse = gmem(a.lse)[static_cast<int64_t>(h) * a.q_tokens + token];
  const int head = h / a.group;
  float* at = a.stats + stat_of(a, head, token, h - head * a.group);
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  *reinterpret_cast<gptr<f32x2>>(gmem(at)) = f32x2{lse == -INFINITY ? INFINITY : lse * kLog2e, s};
}

template <int DT, int DP, bool VEC>
__global__ __launch_bounds__(kThreads, DT == kBF16 && DP <= 128 ? 2 : 1) void attention_dq_kernel(AttnArgs a) {
  using S = Shape<DT, DP>;
  using T = typename S::T;
  constexpr int kKeys = S::kPitch <= 256 ? 64 : 32;
  constexpr int kTileBytes = kKeys * S::kPitch;
  __shared__ __attribute__((aligned(16))) char shared[4 * kTileBytes];   // K, V; twice
  const lds_t lds = (lds_t)shared;

  const int head = blockIdx.x % a.k_heads, rest = blockIdx.x / a.k_heads;
  const Place p = place(a, a.slots - 1 - rest, false);
  if (!p.any) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int shift = p.lk - p.lq;
  const int last = (p.rows < p.row0 + kAttnTile ? p.rows : p.row0 + kAttnTile) - 1;
  int end = p.lk, begin = 0;
  if (a.causal) end = min(end, query_of(a, last) + shift + 1);
  if (a.window) begin = max(0, query_of(a, p.row0) + shift - a.window + 1) / kKeys * kKeys;
  const int tiles = end > begin ? (end - begin + kKeys - 1) / kKeys : 0;

  const int row = p.row0 + wave * 32 + (lane & 31);
  const bool any = row < p.rows;
  const int qi = query_of(a, any ? row : last), g = (any ? row : last) - qi * a.group;
  const int64_t token = p.q0 + qi;
  const int qh = head * a.group + g;
  const int hi = a.causal ? min(qi + shift, p.lk - 1) : p.lk - 1, lo = a.window ? qi + shift - a.window + 1 : 0;
  const int w0 = p.row0 + wave * 32;
  const bool wave_any = w0 < p.rows;
  const int wlo = query_of(a, min(w0, last)), whi = query_of(a, min(w0 + 31, last));

  const T* qrow = static_cast<const T*>(a.q) + token * a.qs + static_cast<int64_t>(qh) * a.dim;
  const T* drow = static_cast<const T*>(a.dout) + token * a.dos + static_cast<int64_t>(qh) * a.dim;
  Frag<DT> qf[S::kSteps], df[S::kSteps];
#pragma unroll
  for (int s = 0; s < S::kSteps; ++s) {
    qf[s] = frag_global<DT, VEC>(qrow, s, a.dim);
    df[s] = frag_global<DT, VEC>(drow, s, a.dim);
  }
  const float* stat = a.stats + stat_of(a, head, token, g);
  const float lse = any ? gmem(stat)[0] : INFINITY, delta = gmem(stat)[1];

  const T* kbase = static_cast<const T*>(a.k) + p.k0 * a.ks + static_cast<int64_t>(head) * a.dim;
  const T* vbase = static_cast<const T*>(a.v) + p.k0 * a.vs + static_cast<int64_t>(head) * a.dim;
  Filler<DT, DP, kKeys, VEC> fill_k, fill_v;
  fill_k.init(a.dim, [&](int r) { return static_cast<uint32_t>(r) * static_cast<uint32_t>(a.ks * S::kElem); });
  fill_v.init(a.dim, [&](int r) { return static_cast<uint32_t>(r) * static_cast<uint32_t>(a.vs * S::kElem); });
  auto fetch = [&](int tile) {
    const lds_t to = lds + (tile & 1) * 2 * kTileBytes;
    const int key0 = begin + tile * kKeys;
    if constexpr (VEC)
      if (key0 + kKeys <= p.lk) {
        fill_k.whole(to, kbase + key0 * a.ks, a.dim);
        fill_v.whole(to + kTileBytes, vbase + key0 * a.vs, a.dim);
        return;
      }
    fill_k.any(to, a.dim, [&](int r) { return kbase + min(key0 + r, p.lk - 1) * a.ks; });
    fill_v.any(to + kTileBytes, a.dim, [&](int r) { return vbase + min(key0 + r, p.lk - 1) * a.vs; });
  };
  f32x16 dq[S::kBlocks];
#pragma unroll
  for (int b = 0; b < S::kBlocks; ++b) dq[b] = f32x16{};
  const float c = a.scale * kLog2e;
  if (tiles > 0) {
    if (VEC && a.dim < DP) {
      clear_tiles(lds, 4 * kTileBytes);
      __syncthreads();
    }
    fetch(0);
    tiles_landed();
  }
  for (int tile = 0; tile < tiles; ++tile) {
    if (tile + 1 < tiles) fetch(tile + 1);
    const lds_t kt = lds + (tile & 1) * 2 * kTileBytes;
    const lds_t vt = kt + kTileBytes;
#pragma unroll 1
    for (int kb = 0; kb < kKeys; kb += 32) {
      const int key0 = begin + tile * kKeys + kb;
      const bool see = wave_any && key0 < p.lk && (!a.causal || key0 <= whi + shift) &&
                       (!a.window || key0 + 32 > wlo + shift - a.window + 1);
      if (!see) continue;
      f32x16 s{}, dp{};
#pragma unroll
      for (int st = 0; st < S::kSteps; ++st) s = mma(frag_rows<DT, DP>(kt, kb, st), qf[st], s);
#pragma unroll
      for (int st = 0; st < S::kSteps; ++st) dp = mma(frag_rows<DT, DP>(vt, kb, st), df[st], dp);
      const bool mask = key0 + 32 > p.lk || (a.causal && key0 + 31 > wlo + shift) ||
                        (a.window && key0 < whi + shift - a.window + 1);
      if (mask) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = key0 + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
          if (key > hi || key < lo) s[i] = -INFINITY;
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) dp[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -lse)) * (dp[i] - delta);
      // A row's ds add up to 0, so what its keys have in common cancels in dq, but
      // not in the errors of rounding ds to bf16: with those alone dq of trained
      // keys is half as far off again as its own rounding.  The product takes ds
      // as two bf16 numbers, from the same fragments of the keys (0.5 ms of the
      // 16384-token batch; the relative error of dq falls from 2.5e-3 to 1.7e-3, all but its own rounding).
      Frag<DT> ds[2], low[2];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        ds[i >> 3].set(i & 7, dp[i]);
        if constexpr (DT == kBF16) low[i >> 3].set(i & 7, dp[i] - static_cast<float>(ds[i >> 3].v[i & 7]));
      }
#pragma unroll
      for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const Frag<DT> k = frag_cols<DT, DP>(kt, kb + 16 * h, b);
          dq[b] = mma(k, ds[h], dq[b]);
          if constexpr (DT == kBF16) dq[b] = mma(k, low[h], dq[b]);
        }
    }
    tiles_landed();
  }
  if (any)
    store_row<DT, DP, VEC>(static_cast<T*>(a.dq) + token * a.dqs + static_cast<int64_t>(qh) * a.dim, dq, a.scale, a.dim);
}

// Where the tile's keys and values stay: their fragments in registers, or, where
// two sums of a head fill those, the values in LDS (bf16 from 128 on), or both in
// memory and read again for every tile of rows (fp32 beyond 128).  With the
// values in LDS 256 registers hold a wave and two share a SIMD: the 16384-token
// batch in 4.24 ms, and in 6.8 with one wave.
template <int DT, int DP> struct Held {
  static constexpr bool kMemory = DT == kF32 && DP > 128;
  static constexpr bool kValuesLds = DT == kBF16 && DP >= 128;
};

template <int DT, int DP, bool VEC>
__global__ __launch_bounds__(kThreads, DT == kBF16 && DP <= 128 ? 2 : 1) void attention_dkv_kernel(AttnArgs a) {
  using S = Shape<DT, DP>;
  using T = typename S::T;
  using H = Held<DT, DP>;
  constexpr int kTileBytes = 32 * S::kPitch, kValues = H::kValuesLds ? kAttnTile * S::kPitch : 0;
  constexpr int kStats = 4 * kTileBytes;   // lse, delta of 32 rows; twice
  __shared__ __attribute__((aligned(16))) char shared[kStats + 512 + kValues];   // Q, dout; twice
  const lds_t lds = (lds_t)shared;

  const int head = blockIdx.x % a.k_heads;
  const Place p = place(a, blockIdx.x / a.k_heads, true);
  if (!p.any) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, hf = lane >> 5;
  const int shift = p.lk - p.lq;
  const int last = min(p.lk, p.row0 + kAttnTile) - 1;
  // rows that see any of the tile's keys
  int first_q = 0, end_q = p.lq;
  if (a.causal) first_q = max(0, p.row0 - shift);
  if (a.window) end_q = max(0, min(end_q, last - shift + a.window));   // times the group it stays within 32 bits
  const int begin = first_q * a.group, end = end_q * a.group;
  const int tiles = end > begin ? (end - begin + 31) / 32 : 0;

  const int w0 = p.row0 + wave * 32, w1 = min(w0 + 32, p.lk) - 1;   // this wave's keys
  const bool wave_any = w0 < p.lk;
  const int key = w0 + (lane & 31);
  const T* kbase = static_cast<const T*>(a.k) + p.k0 * a.ks + static_cast<int64_t>(head) * a.dim;
  const T* vbase = static_cast<const T*>(a.v) + p.k0 * a.vs + static_cast<int64_t>(head) * a.dim;
  const T* krow = kbase + min(key, last) * a.ks;
  const T* vrow = vbase + min(key, last) * a.vs;
  Frag<DT> kf[H::kMemory ? 1 : S::kSteps], vf[H::kMemory || H::kValuesLds ? 1 : S::kSteps];
  if constexpr (!H::kMemory)
#pragma unroll
    for (int s = 0; s < S::kSteps; ++s) {
      kf[s] = frag_global<DT, VEC>(krow, s, a.dim);
      if constexpr (!H::kValuesLds) vf[s] = frag_global<DT, VEC>(vrow, s, a.dim);
    }
  const lds_t values = lds + kStats + 512;
  auto key_frag = [&](int st) {
    if constexpr (H::kMemory) return frag_global<DT, VEC>(krow, st, a.dim);
    else return kf[st];
  };
  auto value_frag = [&](int st) {
    if constexpr (H::kMemory) return frag_global<DT, VEC>(vrow, st, a.dim);
    else if constexpr (H::kValuesLds) return frag_rows<DT, DP>(values, wave * 32, st);
    else return vf[st];
  };

  const T* qbase = static_cast<const T*>(a.q) + p.q0 * a.qs + static_cast<int64_t>(head) * a.group * a.dim;
  const T* dbase = static_cast<const T*>(a.dout) + p.q0 * a.dos + static_cast<int64_t>(head) * a.group * a.dim;
  const float* sbase = a.stats + stat_of(a, head, p.q0, 0);
  // whole tiles begin with a query's first head where the group divides 32
  Filler<DT, DP, 32, VEC> fill_q, fill_d;
  const bool even = 32 % a.group == 0;
  auto at = [&](int r, int64_t stride) {
    const int i = query_of(a, r);
    return i * stride + static_cast<int64_t>(r - i * a.group) * a.dim;
  };
  fill_q.init(a.dim, [&](int r) { return static_cast<uint32_t>(at(r, a.qs) * S::kElem); });
  fill_d.init(a.dim, [&](int r) { return static_cast<uint32_t>(at(r, a.dos) * S::kElem); });
  auto fetch = [&](int tile) {
    const lds_t to = lds + (tile & 1) * 2 * kTileBytes;
    const int r0 = begin + tile * 32;
    // 32 rows' pairs; behind the last row, the last one's
    if (wave == 0)
      lds_dma4(uniform_ptr(sbase + 2 * static_cast<int64_t>(r0)), static_cast<uint32_t>(8 * min(lane >> 1, end - 1 - r0) + 4 * (lane & 1)),
           __builtin_amdgcn_readfirstlane(lds_address(lds + kStats)) + (tile & 1) * 256);
    if constexpr (VEC)
      if (even && r0 + 32 <= end) {
        fill_q.whole(to, qbase + at(r0, a.qs), a.dim);
        fill_d.whole(to + kTileBytes, dbase + at(r0, a.dos), a.dim);
        return;
      }
    fill_q.any(to, a.dim, [&](int r) { return qbase + at(min(r0 + r, end - 1), a.qs); });
    fill_d.any(to + kTileBytes, a.dim, [&](int r) { return dbase + at(min(r0 + r, end - 1), a.dos); });
  };
  f32x16 dk[S::kBlocks], dv[S::kBlocks];
#pragma unroll
  for (int b = 0; b < S::kBlocks; ++b) dk[b] = dv[b] = f32x16{};
  const float c = a.scale * kLog2e;
  if (tiles > 0) {
    if (VEC && a.dim < DP) {
      clear_tiles(lds, sizeof(shared));
      __syncthreads();
    }
    if constexpr (H::kValuesLds) {
      Filler<DT, DP, kAttnTile, VEC> fill_v;
      fill_v.any(values, a.dim, [&](int r) { return vbase + min(p.row0 + r, last) * a.vs; });
    }
    fetch(0);
    tiles_landed();
  }
  for (int tile = 0; tile < tiles; ++tile) {
    if (tile + 1 < tiles) fetch(tile + 1);
    const lds_t qt = lds + (tile & 1) * 2 * kTileBytes;
    const lds_t dt = qt + kTileBytes;
    const int r0 = begin + tile * 32, r1 = min(r0 + 31, end - 1);
    const int qlo = query_of(a, r0), qhi = query_of(a, r1);
    const bool see = wave_any && (!a.causal || w0 <= qhi + shift) && (!a.window || w1 > qlo + shift - a.window);
    if (see) {
      f32x16 s{}, dp{};
#pragma unroll
      for (int st = 0; st < S::kSteps; ++st) s = mma(frag_rows<DT, DP>(qt, 0, st), key_frag(st), s);
#pragma unroll
      for (int st = 0; st < S::kSteps; ++st) dp = mma(frag_rows<DT, DP>(dt, 0, st), value_frag(st), dp);
      const bool mask = r0 + 32 > end || (a.causal && w1 > qlo + shift) || (a.window && w0 <= qhi + shift - a.window);
      if (mask) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = r0 + 8 * (i >> 2) + 4 * hf + (i & 3), q = query_of(a, r) + shift;
          if (r >= end || (a.causal && key > q) || (a.window && key <= q - a.window)) s[i] = -INFINITY;
        }
      }
      const lptr<const float> stat = reinterpret_cast<lptr<const float>>(lds + kStats + (tile & 1) * 256) + 8 * hf;
      // P and dS are rounded once, as bf16 operands: what they are summed with, dout
      // and q, has no common part that would have to cancel as the keys' has in dq.
      // dk and dv of the 16384-token batch are 2.3e-3 off (relative, of the whole), of
      // which their own rounding is 1.7e-3; two numbers each would double the matrix
      // instructions of this phase, and its registers.
      Frag<DT> pf[2], ds[2];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = 8 * (i >> 2) + (i & 3);
        const float e = __builtin_amdgcn_exp2f(fmaf(s[i], c, -stat[2 * r]));
        pf[i >> 3].set(i & 7, e);
        ds[i >> 3].set(i & 7, e * (dp[i] - stat[2 * r + 1]));
      }
#pragma unroll
      for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          dv[b] = mma(frag_cols<DT, DP>(dt, 16 * h, b), pf[h], dv[b]);
          dk[b] = mma(frag_cols<DT, DP>(qt, 16 * h, b), ds[h], dk[b]);
        }
    }
    tiles_landed();
  }
  if (key >= p.lk) return;
  const int64_t token = p.k0 + key;
  store_row<DT, DP, VEC>(static_cast<T*>(a.dk) + token * a.dks + static_cast<int64_t>(head) * a.dim, dk, a.scale, a.dim);
  store_row<DT, DP, VEC>(static_cast<T*>(a.dv) + token * a.dvs + static_cast<int64_t>(head) * a.dim, dv, 1.0f, a.dim);
}

constexpr int64_t kGridLine = int64_t{1} << 20;   // blocks along a grid's first axis; the rows' come in lines of it

template <int DT, int DP, bool VEC> hipError_t run(const AttnArgs& a, int k_slots, hipStream_t stream) {
  if (a.q_tokens > 0) {
    constexpr int kLanes = Shape<DT, DP>::kPitch / 16;
    const int64_t per = kThreads / kLanes, blocks = (static_cast<int64_t>(a.q_tokens) * a.q_heads + per - 1) / per;
    const int64_t cols = std::min<int64_t>(blocks, kGridLine);
    attention_stats_kernel<DT, kLanes, VEC><<<dim3(static_cast<unsigned>(cols), static_cast<unsigned>((blocks + cols - 1) / cols)),
                                              dim3(kThreads), 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    attention_dq_kernel<DT, DP, VEC><<<dim3(static_cast<unsigned>(a.slots) * a.k_heads), dim3(kThreads), 0, stream>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (a.k_tokens > 0)
    attention_dkv_kernel<DT, DP, VEC>
        <<<dim3(static_cast<unsigned>(k_slots) * a.k_heads), dim3(kThreads), 0, stream>>>(a);
  return hipGetLastError();
}
template <int DT, int DP> hipError_t run(const AttnArgs& a, int k_slots, hipStream_t stream) {
  return a.vec ? run<DT, DP, true>(a, k_slots, stream) : run<DT, DP, false>(a, k_slots, stream);
}
template <int DT> hipError_t run_any(const AttnArgs& a, int k_slots, hipStream_t stream) {
  switch (attn_padded(a.dim)) {
    case 64: return run<DT, 64>(a, k_slots, stream);
    case 96: return run<DT, 96>(a, k_slots, stream);
    case 128: return run<DT, 128>(a, k_slots, stream);
    case 192: return run<DT, 192>(a, k_slots, stream);
    default: return run<DT, 256>(a, k_slots, stream);
  }
}

}  // namespace
}  // namespace attn

hipError_t launch_attention_grad(int dt, const AttnArgs& a, int k_slots, hipStream_t stream) {
  return dt == kF32 ? attn::run_any<kF32>(a, k_slots, stream) : attn::run_any<kBF16>(a, k_slots, stream);
}

}  // namespace dmuon
