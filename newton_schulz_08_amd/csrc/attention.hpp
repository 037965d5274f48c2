// What the attention kernels share: tiles in LDS, matrix fragments, and where a
// tile lies in the packed sequences.
//
// All products run on 32 x 32 blocks, v_mfma_f32_32x32x16_bf16 or eight
// v_mfma_f32_32x32x2_f32, with 16 contraction steps a fragment: lane l holds
// row (or column) l & 31 and eight steps, those of half l >> 5.  A result block
// has lane l in column l & 31 and, in register i, row 8 (i / 4) + 4 (l >> 5) +
// i % 4: registers 8 h .. 8 h + 7 are a fragment again, of the 16 steps
//
//   16 h + {0..3, 8..11} + 4 (l >> 5),
//
// so a block of probabilities enters the next product from the registers it
// was formed in, and the other operand is read in that order of steps.
//
// A tile's row of `Pitch` bytes (a power of two) holds 16-byte chunk c at
// c ^ swizzle(row): rows read together, along a row or across rows, lie in
// distinct banks.
#pragma once

#include "block.hpp"
#include "lds_fill.hpp"

namespace dmuon {
namespace attn {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
// LDS is addressed as such throughout: a cast from a general pointer would test it for null.
template <typename T> using lptr = __attribute__((address_space(3))) T*;
typedef lptr<char> lds_t;

template <int DT, int DP> struct Shape {
  using T = typename OpElem<DT>::T;
  static constexpr int kElem = DT == kBF16 ? 2 : 4;
  static constexpr int kRow = DP * kElem;                       // bytes of a padded head
  static constexpr int kPitch = kRow <= 128 ? 128 : kRow <= 256 ? 256 : kRow <= 512 ? 512 : 1024;
  static constexpr int kChunks = kPitch / 16;
  static constexpr int kSteps = DP / 16;                        // fragments of a head
  static constexpr int kBlocks = DP / 32;                       // result blocks of a head
  __device__ static __forceinline__ int swizzle(int r) {
    if constexpr (kPitch == 128) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
    else if constexpr (DT == kBF16) return ((r & 3) << 2) | ((r >> 2) & 3);
    else return (((r >> 2) & 1) << 3) | (((r >> 3) & 1) << 2) | (r & 3);
  }
};

template <int DT> struct Frag;
template <> struct Frag<kBF16> {
  bf16x8 v;
  __device__ __forceinline__ void set(int i, float x) { v[i] = static_cast<__bf16>(x); }
};
template <> struct Frag<kF32> {
  float v[8];
  __device__ __forceinline__ void set(int i, float x) { v[i] = x; }
};
__device__ __forceinline__ f32x16 mma(const Frag<kBF16>& a, const Frag<kBF16>& b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(const Frag<kF32>& a, const Frag<kF32>& b, f32x16 c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}

// Fragment `step` of a tile's rows row0 .. row0 + 31, steps along the head.
template <int DT, int DP> __device__ __forceinline__ Frag<DT> frag_rows(lds_t tile, int row0, int step) {
  using S = Shape<DT, DP>;
  const int lane = threadIdx.x & 63, row = row0 + (lane & 31), hf = lane >> 5, sw = S::swizzle(lane & 31);
  const lds_t at = tile + row * S::kPitch;
  Frag<DT> f;
  if constexpr (DT == kBF16) {
    f.v = *reinterpret_cast<lptr<const bf16x8>>(at + (((2 * step + hf) ^ sw) << 4));
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32v4 x = *reinterpret_cast<lptr<const f32v4>>(at + (((4 * step + 2 * hf + h) ^ sw) << 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) f.v[4 * h + i] = x[i];
    }
  }
  return f;
}
// Fragment of columns 32 block .. + 31 of the head, steps along the tile's
// rows: the 16 from row0 on, in the order of a result block's registers.
template <int DT, int DP> __device__ __forceinline__ Frag<DT> frag_cols(lds_t tile, int row0, int block) {
  using S = Shape<DT, DP>;
  const int lane = threadIdx.x & 63, hf = lane >> 5;
  Frag<DT> f;
  if constexpr (DT == kBF16) {
    // a transposing read: in each group of 16 lanes, lane 4 t + a points at row t, columns 4 a .. + 3,
    // and receives column (lane & 15) of the four rows
    const int t = (lane >> 2) & 3, a = lane & 3, g = (lane >> 4) & 1;
    bf16x4 part[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = row0 + 8 * h + 4 * hf + t;
      const lds_t at = tile + row * S::kPitch + (((4 * block + 2 * g + (a >> 1)) ^ S::swizzle(row)) << 4) + 8 * (a & 1);
      part[h] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(reinterpret_cast<lptr<bf16x4>>(at));
    }
    f.v = __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    const int col = 32 * block + (lane & 31);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = row0 + 8 * (i >> 2) + 4 * hf + (i & 3);
      f.v[i] = *reinterpret_cast<lptr<const float>>(tile + row * S::kPitch + (((col >> 2) ^ S::swizzle(row)) << 4) + 4 * (col & 3));
    }
  }
  return f;
}
// The 16 bytes from element d of a head on, wherever it lies, zeros behind it.
// Every lane loads, from the head's last 16 bytes if its own reach behind them,
// and moves those into place: a branch around a load would make the next one
// wait for it.
template <typename T> using Chunk = T __attribute__((ext_vector_type(16 / sizeof(T))));
template <typename T> __device__ __forceinline__ Chunk<T> chunk_of(const T* head, int d, int dim) {
  constexpr int M = 16 / static_cast<int>(sizeof(T));
  const T zero = static_cast<T>(0.0f);
  Chunk<T> x;
  if (dim >= M) {
    using L = typename Loose<T, M>::V;
    const L v = *reinterpret_cast<gptr<const L>>(gmem(head + min(d, dim - M)));
#pragma unroll
    for (int i = 0; i < M; ++i) x[i] = v[i];
    const int by = d - (dim - M);   // > 0: the elements lie that far up
    if (by >= M) x = Chunk<T>{};
#pragma unroll
    for (int b = M / 2; b > 0; b >>= 1)
      if (by > 0 && (by & b))
#pragma unroll
        for (int i = 0; i < M; ++i) x[i] = i + b < M ? x[i + b < M ? i + b : 0] : zero;
  } else {
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const T v = gmem(head)[min(d + i, dim - 1)];
      x[i] = d + i < dim ? v : zero;
    }
  }
  return x;
}
// Fragment `step` of one row in memory, zeros behind the head.  VEC: runs of 16
// bytes are aligned and whole.
template <int DT, bool VEC> __device__ __forceinline__ Frag<DT> frag_global(const void* row, int step, int dim) {
  using T = typename OpElem<DT>::T;
  constexpr int M = 16 / static_cast<int>(sizeof(T));
  typedef T V __attribute__((ext_vector_type(M)));
  const int d0 = 16 * step + 8 * ((threadIdx.x & 63) >> 5);
  const T* p = static_cast<const T*>(row);
  Frag<DT> f;
#pragma unroll
  for (int h = 0; h < 8 / M; ++h) {
    const int d = d0 + M * h;
    V x;
    if constexpr (VEC) {   // every lane loads, so that no load waits for another
      x = *reinterpret_cast<gptr<const V>>(gmem(p + (d < dim ? d : 0)));
      if (d >= dim) x = V{};
    } else {
      x = chunk_of(p, d, dim);
    }
#pragma unroll
    for (int i = 0; i < M; ++i) f.v[M * h + i] = x[i];
  }
  return f;
}

// Row r of a sequence's (query, head of the group) rows.
__device__ __forceinline__ int query_of(const AttnArgs& a, int r) {
  int i = static_cast<int>(__umulhi(static_cast<unsigned>(r), a.group_inv));
  if (a.group == 1) i = r;                  // 2^32 does not fit the factor
  else if (i * a.group > r) --i;            // the factor is rounded up: at most one too many
  return i;
}

// Everything that the block has on its way into LDS is there behind this.
__device__ __forceinline__ void tiles_landed() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

// Fills tiles of R rows, straight to LDS (VEC; the padding behind a head is left
// alone, clear_tiles) or through registers, 16 bytes at a time.
template <int DT, int DP, int R, bool VEC> struct Filler {
  using S = Shape<DT, DP>;
  using T = typename S::T;
  static constexpr int kLoads = R * S::kChunks / 64 / kWaves;   // of 1 KB, per wave
  static_assert(R * S::kChunks % (64 * kWaves) == 0, "whole loads for every wave");
  static constexpr uint32_t kNone = 0xFFFFFFFFu;
  uint32_t off[VEC ? kLoads : 1];

  __device__ static __forceinline__ int row_of(int u) {
    return ((u * kWaves + static_cast<int>(threadIdx.x >> 6)) * 64 + static_cast<int>(threadIdx.x & 63)) / S::kChunks;
  }
  // offset(row): bytes from the tile's first row to this one; every row's are
  // the same in every whole tile.
  template <typename Offset> __device__ __forceinline__ void init(int dim, Offset&& offset) {
    if constexpr (VEC)
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int row = row_of(u), chunk = (static_cast<int>(threadIdx.x & 63) % S::kChunks) ^ S::swizzle(row);
        off[u] = chunk * 16 < dim * S::kElem ? offset(row) + chunk * 16 : kNone;
      }
  }
  __device__ static __forceinline__ void move(const char* base, uint32_t voff, uint32_t lds, int u, bool full) {
    const uint32_t dst = lds + static_cast<uint32_t>(u * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * 1024;
    if (full) lds_dma16(base, voff, dst);
    else if (voff != kNone) lds_dma16(base, voff, dst);
  }
  // A whole tile whose first row begins at `first`.
  __device__ __forceinline__ void whole(lds_t tile, const void* first, int dim) const {
    static_assert(VEC, "through registers: any()");
    const char* base = uniform_ptr(first);
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_address(tile));
    const bool full = dim * S::kElem == S::kPitch;
#pragma unroll
    for (int u = 0; u < kLoads; ++u) move(base, off[u], lds, u, full);
  }
  // Any tile: address(row) is where the row's head begins; rows that do not
  // exist take one that does.
  template <typename Address> __device__ __forceinline__ void any(lds_t tile, int dim, Address&& address) const {
    if constexpr (VEC) {
      const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_address(tile));
      const char* base = uniform_ptr(address(0));
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int row = row_of(u), chunk = (static_cast<int>(threadIdx.x & 63) % S::kChunks) ^ S::swizzle(row);
        const uint32_t at = static_cast<uint32_t>(reinterpret_cast<const char*>(address(row)) - base) + chunk * 16;
        move(base, chunk * 16 < dim * S::kElem ? at : kNone, lds, u, false);
      }
    } else {
      constexpr int kC = S::kRow / 16, kAll = R * kC, kAtOnce = 4;   // chunks under way in a thread
#pragma unroll 1
      for (int e0 = threadIdx.x; e0 < kAll; e0 += kAtOnce * kThreads) {
        Chunk<T> x[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const int e = min(e0 + u * kThreads, kAll - 1);
          x[u] = chunk_of(address(e / kC), e % kC * (16 / S::kElem), dim);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const int e = e0 + u * kThreads, row = e / kC;
          if (e < kAll) *reinterpret_cast<lptr<Chunk<T>>>(tile + row * S::kPitch + ((e % kC ^ S::swizzle(row)) << 4)) = x[u];
        }
      }
    }
  }
};
__device__ __forceinline__ void clear_tiles(lds_t lds, int bytes) {
  for (int i = threadIdx.x * 16; i < bytes; i += blockDim.x * 16) *reinterpret_cast<lptr<f32v4>>(lds + i) = f32v4{};
}

// A block's place: sequence, tile of it, and the sequence's extent.
struct Place {
  int q0, lq, k0, lk;   // first token and tokens of the sequence's queries and keys
  int row0, rows;       // first row of the tile, rows of the sequence
  bool any;
};
__device__ __forceinline__ int offset(const int* off, int i, int tokens) {
  const int v = gmem(off)[i];
  return v < 0 ? 0 : v > tokens ? tokens : v;   // whatever the offsets say, rows stay within the tensor
}
// The tile of `slot`; by: rows of a token on the side that is tiled (the group, or 1 for keys).
__device__ __forceinline__ Place place(const AttnArgs& a, int slot, bool keys) {
  Place p;
  int tile;
  const int64_t by = keys ? 1 : a.group;
  if (!a.q_off) {
    p.q0 = p.k0 = 0;
    p.lq = a.q_tokens;
    p.lk = a.k_tokens;
    tile = slot;
  } else {
    const int* off = keys ? a.k_off : a.q_off;
    const int tokens = keys ? a.k_tokens : a.q_tokens;
    auto first = [&](int i) { return static_cast<int>(offset(off, i, tokens) * by / kAttnTile) + i; };
    int lo = 0, hi = a.sequences;     // first(lo) <= slot
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first(mid) <= slot) lo = mid;
      else hi = mid;
    }
    tile = slot - first(lo);
    p.q0 = offset(a.q_off, lo, a.q_tokens);
    p.lq = offset(a.q_off, lo + 1, a.q_tokens) - p.q0;
    p.k0 = offset(a.k_off, lo, a.k_tokens);
    p.lk = offset(a.k_off, lo + 1, a.k_tokens) - p.k0;
    if (p.lq < 0) p.lq = 0;
    if (p.lk < 0) p.lk = 0;
  }
  p.rows = static_cast<int>(keys ? p.lk : p.lq * by);
  p.any = tile >= 0 && tile < (p.rows + kAttnTile - 1) / kAttnTile;
  p.row0 = tile * kAttnTile;
  return p;
}

// The value of the lane in the other half of the wave.
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32, 64); }

// One lane's row of a result: four elements at a time, scaled.
template <int DT, int DP, bool VEC>
__device__ __forceinline__ void store_row(void* row, const f32x16 (&o)[DP / 32], float by, int dim) {
  using T = typename OpElem<DT>::T;
  T* p = static_cast<T*>(row);
  const int hf = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int b = 0; b < DP / 32; ++b)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int d = 32 * b + 8 * g + 4 * hf;
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = o[b][4 * g + i] * by;
      if constexpr (VEC) {
        if (d < dim) store_n<4>(p + d, x);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (d + i < dim) gmem(p)[d + i] = static_cast<T>(x[i]);
      }
    }
}

}  // namespace attn
}  // namespace dmuon
