// Attention over packed sequences, forward, on gfx950 (MFMA-bound for long
// sequences, HBM-bound for single queries).
//
// Of a sequence with lq queries and lk keys, query i sees key j when
// j <= i + lk - lq (causal) and j > i + lk - lq - window (with a window).  With
// s = scale q . k, one pass over the keys keeps the maximum m and the sum l of
// exp(s - m) of every row:
//
//   out = sum exp(s - m) v / l,    lse = m + log l
//
// A row without visible keys has out 0 and lse -infinity.
//
// The rows of a tile are a key head's (query, query head) pairs, so the heads
// that share keys read them once, and a single query still fills rows.  Each
// wave keeps 32 rows: S^T = K Q^T puts a row's scores into one pair of lanes,
// maximum and sum need one exchange, and P^T is the next product's operand
// where it lies (attention.hpp).  K and V tiles go straight to LDS, one tile
// ahead.  Exponentials are base 2 with log2(e) folded into the scale.
//
// Few tiles (single queries): a tile's keys are cut into slices, each leaving its
// unnormed sum, maximum and weight; a second launch joins them.
//
// Measured, 32 heads over 8 key heads of 128 bf16, causal: two sequences of 8192
// tokens 1.10 to 1.23 ms on different cards, 0.90 to 1.00 PFLOP/s of the visible
// half (the matrix pipe is busy for 47% of it, the vector pipe for 57%:
// exponentials, maxima, conversions); one new token of 8 sequences over 65536 keys
// in all 49 us with the join's 4.8, 5.5 TB/s out of the memory-side cache in part,
// 50 with as many keys again as room behind the caches; a fresh cache 63, 4.2 TB/s.
// Heads of 64 0.62 to 0.68 ms, of 192 2.9, of 256 3.3 (one wave a SIMD).
// fp32, 4096 tokens in two sequences: heads of 64 0.34 ms, of 128 0.63 (0.11
// PFLOP/s), of 192 1.1, of 256 2.3 (86 registers spill).  The 8 tokens over 65536
// fp32 keys 308 us, 1.7 TB/s: of a block's four waves one has rows, and its chain
// of fp32 matrix instructions is the time.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attention.hpp"

namespace dmuon {
namespace attn {
namespace {

constexpr float kNone = -INFINITY;
// Two blocks a CU where their tiles fit its LDS and 256 registers hold a wave:
// one's softmax runs beside the other's matrix instructions.  Heads over 128 bf16
// (64 fp32) need more of both.
template <int DT, int DP> constexpr int waves_per_simd() { return Shape<DT, DP>::kPitch <= 256 ? 2 : 1; }
// A row's sums are scaled to a new maximum only when it lies this far (a factor
// of 2^8) above the one they were formed with: fp32 has room for that, and the
// result does not depend on which maximum was taken off.  The 16384-token batch:
// 1.14 ms; with an exchange between the half rows in every tile 1.16.
constexpr float kSlack = 8.0f;

// Unnormed sums of a slice: rows x DP, then maximum and weight of each row.
__host__ __device__ constexpr int64_t slice_floats(int dp) { return static_cast<int64_t>(kAttnTile) * (dp + 2); }

// lse of a row with maximum m (base 2) and weight l.
__device__ __forceinline__ float row_lse(float m, float l) {
  return l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : l == 0.0f ? kNone : l;
}

template <int DT, int DP, bool VEC>
__global__ __launch_bounds__(kThreads, (waves_per_simd<DT, DP>())) void attention_kernel(AttnArgs a) {
  using S = Shape<DT, DP>;
  using T = typename S::T;
  constexpr int kKeys = S::kPitch <= 512 ? 64 : 32;          // of a tile
  constexpr int kKb = kKeys / 32;
  constexpr int kTileBytes = kKeys * S::kPitch;
  __shared__ __attribute__((aligned(16))) char shared[4 * kTileBytes];   // K, V; twice
  const lds_t lds = (lds_t)shared;

  // heads vary fastest: the blocks of one XCD share few heads' keys.  The last
  // tiles of a causal sequence have the most keys: they start first.  A tile's
  // slices come together: with empty places between the tiles (room behind caches)
  // the CUs are then filled evenly (8 tokens over 65536 keys, each cache with room
  // behind it, 50 us; with the places one after another 66).
  const int head = blockIdx.x % a.k_heads, rest = blockIdx.x / a.k_heads;
  const int slot = a.slots - 1 - rest / a.slices, slice = rest % a.slices;
  const Place p = place(a, slot, false);
  if (!p.any) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int shift = p.lk - p.lq;
  const int last = (p.rows < p.row0 + kAttnTile ? p.rows : p.row0 + kAttnTile) - 1;

  // keys that any row of the tile sees, whole tiles of them, this slice's share
  int end = p.lk, begin = 0;
  if (a.causal) end = min(end, query_of(a, last) + shift + 1);
  if (a.window) begin = max(0, query_of(a, p.row0) + shift - a.window + 1) / kKeys * kKeys;
  int tiles = end > begin ? (end - begin + kKeys - 1) / kKeys : 0;
  if (a.slices > 1) {
    const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * slice / a.slices);
    const int t1 = static_cast<int>(static_cast<int64_t>(tiles) * (slice + 1) / a.slices);
    begin += t0 * kKeys;
    tiles = t1 - t0;
  }

  // this lane's row
  const int row = p.row0 + wave * 32 + (lane & 31);
  const bool any = row < p.rows;
  const int qi = query_of(a, any ? row : last), g = (any ? row : last) - qi * a.group;
  const int64_t token = p.q0 + qi;
  const int qh = head * a.group + g;
  const T* qrow = static_cast<const T*>(a.q) + token * a.qs + static_cast<int64_t>(qh) * a.dim;
  const int hi = a.causal ? min(qi + shift, p.lk - 1) : p.lk - 1, lo = a.window ? qi + shift - a.window + 1 : 0;
  // this wave's rows
  const int w0 = p.row0 + wave * 32;
  const bool wave_any = w0 < p.rows;
  const int wlo = query_of(a, min(w0, last)), whi = query_of(a, min(w0 + 31, last));

  Frag<DT> qf[S::kSteps];
#pragma unroll
  for (int s = 0; s < S::kSteps; ++s) qf[s] = frag_global<DT, VEC>(qrow, s, a.dim);

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

  f32x16 o[S::kBlocks];
#pragma unroll
  for (int b = 0; b < S::kBlocks; ++b) o[b] = f32x16{};
  float m = kNone, l = 0.0f;   // l: this lane's half of the row
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
    const int key0 = begin + tile * kKeys;
    const bool see = wave_any && (!a.causal || key0 <= whi + shift) && (!a.window || key0 + kKeys > wlo + shift - a.window + 1);
    if (see) {
      f32x16 s[kKb];
#pragma unroll
      for (int kb = 0; kb < kKb; ++kb) {
        s[kb] = f32x16{};
#pragma unroll
        for (int st = 0; st < S::kSteps; ++st) s[kb] = mma(frag_rows<DT, DP>(kt, 32 * kb, st), qf[st], s[kb]);
      }
      const bool mask = key0 + kKeys > p.lk || (a.causal && key0 + kKeys - 1 > wlo + shift) ||
                        (a.window && key0 < whi + shift - a.window + 1);
      if (mask) {
#pragma unroll
        for (int kb = 0; kb < kKb; ++kb)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = key0 + 32 * kb + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
            if (key > hi || key < lo) s[kb][i] = kNone;
          }
      }
      float top = s[0][0];
#pragma unroll
      for (int kb = 0; kb < kKb; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[kb][i]);
      // m is the row's, the same in both lanes that share it; the lanes' own maxima
      // decide whether it still serves.  Nothing visible so far: any finite
      // maximum will do, exp2(-inf) is 0.
      if (__any(top * c > m + kSlack)) {
        top = fmaxf(top, other_half(top)) * c;
        const float mn = fmaxf(m, top), by = __builtin_amdgcn_exp2f(m - (mn == kNone ? 0.0f : mn));
        m = mn;
        l *= by;
#pragma unroll
        for (int b = 0; b < S::kBlocks; ++b) o[b] *= by;
      }
      const float ms = m == kNone ? 0.0f : m;
      // For bf16 the probabilities are rounded to it as operands of their product;
      // l, which norms them, adds them as they are.  out of the 16384-token batch is
      // then 2.2e-3 off (relative, of the whole), of which its own rounding is 1.6e-3.
      // Two bf16 numbers each would take that product's matrix instructions, half of
      // all, twice.
      Frag<DT> pf[kKb][2];
#pragma unroll
      for (int kb = 0; kb < kKb; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float e = __builtin_amdgcn_exp2f(fmaf(s[kb][i], c, -ms));
          l += e;
          pf[kb][i >> 3].set(i & 7, e);
        }
#pragma unroll
      for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
        for (int kb = 0; kb < kKb; ++kb)
#pragma unroll
          for (int h = 0; h < 2; ++h) o[b] = mma(frag_cols<DT, DP>(vt, 32 * kb + 16 * h, b), pf[kb][h], o[b]);
    }
    tiles_landed();
  }

  l += other_half(l);
  if (a.slices > 1) {
    if (!any) return;
    float* part = a.part + (static_cast<int64_t>(blockIdx.x)) * slice_floats(DP);
    const int r = wave * 32 + (lane & 31);
    store_row<kF32, DP, true>(part + static_cast<int64_t>(r) * DP, o, 1.0f, DP);
    if (lane < 32) {
      gmem(part)[static_cast<int64_t>(kAttnTile) * DP + 2 * r] = m;
      gmem(part)[static_cast<int64_t>(kAttnTile) * DP + 2 * r + 1] = l;
    }
    return;
  }
  if (!any) return;
  store_row<DT, DP, VEC>(static_cast<T*>(a.o) + token * a.os + static_cast<int64_t>(qh) * a.dim, o, l > 0.0f ? 1.0f / l : l, a.dim);
  if (lane < 32) gmem(a.lse)[static_cast<int64_t>(qh) * a.q_tokens + token] = row_lse(m, l);
}

// Joins a tile's slices: one wave a row, in the slices' order.  The slices' maxima
// and weights are loaded by a lane each, their sums eight at a time.
template <int DT, int DP> __global__ __launch_bounds__(64) void attention_join_kernel(AttnArgs a) {
  using T = typename OpElem<DT>::T;
  constexpr int kRun = (DP + 63) / 64;
  const int head = blockIdx.x % a.k_heads, rest = blockIdx.x / a.k_heads;
  const Place p = place(a, a.slots - 1 - rest, false);
  const int r = blockIdx.y, lane = threadIdx.x, row = p.row0 + r;
  if (!p.any || row >= p.rows) return;
  const int64_t step = static_cast<int64_t>(a.k_heads) * slice_floats(DP);
  const float* part = a.part + (static_cast<int64_t>(rest) * a.slices * a.k_heads + head) * slice_floats(DP);
  const float* ml = part + static_cast<int64_t>(kAttnTile) * DP + 2 * r;
  part += static_cast<int64_t>(r) * DP;
  const bool mine = lane < a.slices;   // at most 64
  float m = mine ? gmem(ml)[lane * step] : kNone, l = mine ? gmem(ml)[lane * step + 1] : 0.0f;
  float top = m;
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor(top, x, 64));
  const float by = mine ? __builtin_amdgcn_exp2f(m - (top == kNone ? 0.0f : top)) : 0.0f;
  l *= by;
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) l += __shfl_xor(l, x, 64);
  float o[kRun] = {};
  for (int s0 = 0; s0 < a.slices; s0 += 8) {
    float v[8][kRun];
#pragma unroll
    for (int s = 0; s < 8; ++s)
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        const int64_t at = least(s0 + s, a.slices - 1) * step;   // every lane loads
        v[s][k] = gmem(part)[at + (64 * k + lane < DP ? 64 * k + lane : 0)];
      }
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const float w = __shfl(by, s0 + s, 64);                  // 0 behind the last slice
#pragma unroll
      for (int k = 0; k < kRun; ++k) o[k] = w == 0.0f ? o[k] : o[k] + w * v[s][k];
    }
  }
  const int qi = query_of(a, row), qh = head * a.group + row - qi * a.group;
  const int64_t token = p.q0 + qi;
  T* out = static_cast<T*>(a.o) + token * a.os + static_cast<int64_t>(qh) * a.dim;
  const float inv = l > 0.0f ? 1.0f / l : l;
#pragma unroll
  for (int k = 0; k < kRun; ++k)
    if (64 * k + lane < a.dim) gmem(out)[64 * k + lane] = static_cast<T>(o[k] * inv);
  if (lane == 0) gmem(a.lse)[static_cast<int64_t>(qh) * a.q_tokens + token] = row_lse(top, l);
}

template <int DT, int DP> hipError_t run(const AttnArgs& a, hipStream_t stream) {
  const unsigned tiles = static_cast<unsigned>(a.slots) * a.k_heads;
  const dim3 blocks(tiles * a.slices);
  if (a.vec) attention_kernel<DT, DP, true><<<blocks, dim3(kThreads), 0, stream>>>(a);
  else attention_kernel<DT, DP, false><<<blocks, dim3(kThreads), 0, stream>>>(a);
  if (a.slices > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // no tile has more rows than there are
    const int rows = static_cast<int>(std::min<int64_t>(kAttnTile, static_cast<int64_t>(a.q_tokens) * a.group));
    attention_join_kernel<DT, DP><<<dim3(tiles, rows), dim3(64), 0, stream>>>(a);
  }
  return hipGetLastError();
}
template <int DT> hipError_t run_any(const AttnArgs& a, hipStream_t stream) {
  switch (attn_padded(a.dim)) {
    case 64: return run<DT, 64>(a, stream);
    case 96: return run<DT, 96>(a, stream);
    case 128: return run<DT, 128>(a, stream);
    case 192: return run<DT, 192>(a, stream);
    default: return run<DT, 256>(a, stream);
  }
}

}  // namespace
}  // namespace attn

hipError_t launch_attention(int dt, const AttnArgs& a, hipStream_t stream) {
  return dt == kF32 ? attn::run_any<kF32>(a, stream) : attn::run_any<kBF16>(a, stream);
}

}  // namespace dmuon
