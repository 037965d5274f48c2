// The gated feed-forward product and its gradients, on gfx950 (MFMA-bound for
// batches, HBM-bound for few tokens).
//
//   g = x Wg^T,  u = x Wu^T,  h = act(g) u                     (forward)
//   dg = dh u act'(g),  du = dh act(g)                         (backward)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// act is silu, g s(g), or gelu in its tanh form, which is g s(2 y) with
// y = sqrt(2 / pi) (g + 0.044715 g^3); s is the logistic function.  The backward
// pass forms both projections again (nothing but the inputs is kept between the
// passes), stores dg and du side by side, rounded to the inputs' type for the
// products that read them, and runs those two products.
//
// bf16 batches: 256 x 256 tiles on v_mfma_f32_16x16x32_bf16, eight waves of
// 128 x 64, stages of 64 contraction steps double-buffered in LDS (2 x 64 KB),
// filled straight from memory while the stage before is multiplied, in the
// manner of the Newton-Schulz products.  The forward's Q panel takes 32 rows
// of Wg and 32 of Wu by turns, so a lane holds g and u of the same elements and
// the epilogue needs no exchange.  An operand lies with its contraction steps
// along a row, or (Q of dx, both of dW) with one step a row, and is then read
// from LDS through transposing reads: no matrix is transposed in memory.
//
// fp32: 64 x 64 tiles on v_mfma_f32_16x16x4_f32, loaded through registers: every
// thread loads, from the last line or run that exists if it has none of its own,
// and zeros take their place on the way to LDS.  Products with few tiles cut their contraction into
// slices, whose sums another launch adds in order.
//
// Few tokens: the weights are read once, straight into fragments, by waves
// that split the contraction; at most 64 tokens a wave.
//
// Measured, 4096 -> 14336 bf16: 8192 tokens 1.45 to 1.53 ms, 1.26 to 1.30 PFLOP/s
// (a library product of 8192 on each side reaches 1.38); gradient 4.5 to 4.6 ms,
// 1.28 (projections again 1.67, dx 1.40, weights 1.49); 1 to 4 tokens 43 us, 5.5
// TB/s of the weights as they lie in the memory-side cache (fresh ones 48), 32
// tokens 61, 64 to 256 tokens 77 to 86 (one row of tiles on 112 CUs), 512 95 to
// 100.  fp32: 1 to 4 tokens 105 to 135 us, 3.5 to 4.5 TB/s, 64 tokens 165 to 187,
// 65 twice that (two rows of tiles).  512 -> 2048 fp32, gradient of 1001 tokens:
// 149 to 167 us on different cards, three products of 48 to 54 and a join of 5,
// where 27 would be the matrix pipe's time; of 4096 tokens 536 to 610, where 328
// would be.  Of those, the loads cost 27 and moving them on to LDS 80; the rest is
// what two waves a SIMD leave open around each stage's barrier.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "block.hpp"
#include "lds_fill.hpp"

namespace dmuon {
namespace ffn {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) bf16x4* lds_bf16x4_t;

constexpr float kLog2e = 1.4426950408889634f;

// act(g) and act'(g).  e = exp(-2 y) is held below 2^126, so that e s(2 y),
// which is 1 - s(2 y), stays a number; there s(2 y) is 0.  gelu is 0 or g beyond
// 30 on either side, so its polynomials stop there (a NaN goes on).
__device__ __forceinline__ void activate(int kind, float g, float* a, float* da) {
  float y2 = g, gdy2 = g;
  if (kind == kGelu) {
    constexpr float c = 1.5957691216057308f, k = 0.044715f;   // 2 sqrt(2 / pi)
    const float near = g > 30.0f ? 30.0f : g < -30.0f ? -30.0f : g;
    y2 = c * (near + k * near * near * near);
    gdy2 = near * (c * (1.0f + 3.0f * k * near * near));
  }
  const float t = -y2 * kLog2e;
  const float e = __builtin_amdgcn_exp2f(fminf(t, 126.0f));
  const float s = t > 126.0f ? 0.0f : 1.0f / (1.0f + e);
  *a = g * s;
  *da = s + gdy2 * s * (e * s);
}

// Four consecutive elements of a row, as far as it reaches, whatever its alignment.
template <typename T> __device__ __forceinline__ void load4(const T* row, int c, int cols, float* v) {
  if (c + 4 <= cols) {
    load_any<4>(row + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = c + i < cols ? static_cast<float>(gmem(row)[c + i]) : 0.0f;
  }
}
template <typename T> __device__ __forceinline__ void store4(T* row, int c, int cols, const float* v) {
  if (c + 4 <= cols) {
    store_any<4>(row + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < cols) gmem(row)[c + i] = static_cast<T>(v[i]);
  }
}

// What becomes of four elements of row r: both projections' (kFfnOut, kFfnMid), at
// columns f .. f + 3 of the hidden width.
template <int DT, int MODE> __device__ __forceinline__ void finish_gated(const FfnArgs& a, int64_t r, int f, const float* g, const float* u) {
  using T = typename OpElem<DT>::T;
  float act[4], dact[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) activate(a.act, g[i], act + i, dact + i);
  if constexpr (MODE == kFfnOut) {
    if (r >= a.n) return;
    float h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = act[i] * u[i];
    store4(static_cast<T*>(a.out) + r * a.outs, f, a.hidden, h);
  } else {
    // rows and columns up to whole stages take zeros: they enter sums
    if (r >= a.mid_rows || f >= a.hp) return;
    float dh[4] = {}, dg[4], du[4];
    if (r < a.n) load4(static_cast<const T*>(a.dh) + r * a.dhs, f, a.hidden, dh);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = r < a.n && f + i < a.hidden;
      dg[i] = in ? dh[i] * u[i] * dact[i] : 0.0f;
      du[i] = in ? dh[i] * act[i] : 0.0f;
    }
    // rounded to T, once, as operands of the next two products: dx and the weights'
    // gradients of 8192 bf16 tokens, 4096 -> 14336, are 2.35e-3 off (relative, of the
    // whole), of which their own rounding is 1.66e-3.  In fp32 those would be fp32
    // products, at a tenth of the rate.
    T* mid = static_cast<T*>(a.mid) + r * (2 * static_cast<int64_t>(a.hp));
    store_n<4>(mid + f, dg);
    store_n<4>(mid + a.hp + f, du);
  }
}
// ... and of one product's (kFfnDx: row r of dx; kFfnDw: row r of the gradient of
// weight `which`), columns c .. c + 3; of a slice, the partial sums.
template <int DT, int MODE>
__device__ __forceinline__ void finish_plain(const FfnArgs& a, int which, int slice, int64_t r, int c, const float* v) {
  using T = typename OpElem<DT>::T;
  const int64_t rows = MODE == kFfnDx ? a.n : a.hidden;
  if (r >= rows || c >= a.dim) return;
  if (a.slices > 1) {
    const int64_t line = MODE == kFfnDx ? slice * rows + r : (2 * static_cast<int64_t>(slice) + which) * rows + r;
    store_n<4>(a.part + line * ((a.dim + 3) / 4 * 4) + c, v);
  } else if constexpr (MODE == kFfnDx) {
    store4(static_cast<T*>(a.out) + r * a.outs, c, a.dim, v);
  } else {
    store4(static_cast<T*>(which ? a.dwu : a.dwg) + r * a.dim, c, a.dim, v);
  }
}

// Tiles of a launch: rows x cols, and, for dW, both weights one behind the other.
struct Grid { int rows, cols, all; };
template <int MODE> __host__ __device__ Grid grid_of(const FfnArgs& a, int tile) {
  auto up = [&](int64_t v, int t) { return static_cast<int>((v + t - 1) / t); };
  Grid g{};
  if (MODE == kFfnOut || MODE == kFfnMid) {
    g.rows = up(MODE == kFfnMid ? a.mid_rows : a.n, tile);
    g.cols = up(MODE == kFfnMid ? a.hp : a.hidden, tile / 2);
  } else if (MODE == kFfnDx) {
    g.rows = up(a.n, tile);
    g.cols = up(a.dim, tile);
  } else {
    g.rows = 2 * up(a.hidden, tile);
    g.cols = up(a.dim, tile);
  }
  g.all = g.rows * g.cols;
  return g;
}
// Contraction stages of a launch.
template <int MODE> __host__ __device__ int64_t stages_of(const FfnArgs& a, int step) {
  const int64_t steps = MODE == kFfnDx ? 2 * static_cast<int64_t>(a.hp) : MODE == kFfnDw ? a.n : a.kdim;
  return (steps + step - 1) / step;
}
// Blocks go round-robin over the eight XCDs.  In each round of 256 an XCD takes 32
// consecutive tiles, a compact patch of the grid (groups of eight tile rows,
// column by column), whose operand panels its L2 holds.
__device__ __forceinline__ void tile_of(const Grid& g, int block, int* ti, int* tj) {
  const int base = g.all >> 8 << 8;
  int t = block;
  if (block < base) {
    t = (block & ~255) + (block & 7) * 32 + ((block >> 3) & 31);
  } else {
    const int n = g.all - base, l = block - base, x = l & 7, each = n >> 3, more = n & 7;
    t = base + x * each + (x < more ? x : more) + (l >> 3);
  }
  constexpr int kGroup = 8;
  const int per = kGroup * g.cols, first = t / per * kGroup, within = t % per;
  const int h = g.rows - first < kGroup ? g.rows - first : kGroup;
  *ti = first + within % h;
  *tj = within / h;
}

// ---------------------------------------------------------------- bf16 tiles
constexpr int kTileThreads = 512;
constexpr int kOperandBytes = 32768, kStageBytes = 65536;

// One operand's 256 rows (or columns) of a tile.
//
// Steps along a row: stage row r (128 bytes: 64 steps) keeps 16-byte chunk c
// at c ^ (r & 7) ^ ((r >> 3) & 1).  Rows behind the last take the last one's.
// Steps as rows (TR): stage row k (512 bytes: 256 columns) keeps chunk c at
// c ^ 4 (k & 3) ^ 2 ((k >> 4) & 1); columns behind the last take the last
// aligned eight's, steps behind the last the last one's (the other operand
// holds zeros there).  Both orders keep the reads below in distinct banks.
template <bool TR> struct Operand {
  const char* base;     // of the tile's first row, or of the steps' first row at the tile's first column
  uint32_t off[4];
  uint32_t pitch;       // bytes
  int lane, wave;
  uint32_t col;         // TR: this lane's bytes along a row, loads 0, 2 and 1, 3
  uint32_t col1;

  // rows: rows that exist from the tile's first on (TR: columns)
  __device__ __forceinline__ void init(const void* p, uint32_t pitch_bytes, int rows) {
    base = uniform_ptr(p);
    pitch = pitch_bytes;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if constexpr (TR) {
      const int k = 8 * wave + (lane >> 5), pc = lane & 31, most_ = rows / 8 - 1;   // load u: row k + 2 u
      auto at = [&](int row) { return static_cast<uint32_t>(min(pc ^ (4 * (row & 3)) ^ (2 * ((row >> 4) & 1)), most_)) * 16; };
      col = at(k);
      col1 = at(k + 2);
      steps(64);
    } else {
      const int r = lane >> 3;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int row = wave * 32 + u * 8 + r;
        off[u] = static_cast<uint32_t>(min(row, rows - 1)) * pitch + (((lane & 7) ^ r ^ (u & 1)) << 4);
      }
    }
  }
  // TR: a stage of `left` steps (at least one).
  __device__ __forceinline__ void steps(int left) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      off[u] = static_cast<uint32_t>(min(8 * wave + (lane >> 5) + 2 * u, left - 1)) * pitch + ((u & 1) ? col1 : col);
  }
  __device__ __forceinline__ void load(const char* at, uint32_t lds, int u) const {
    lds_dma16(at, off[u], lds + static_cast<uint32_t>(wave) * 4096 + u * 1024);
  }
};

// Fragment reads.  Lane l holds row (column) l & 15 of a block and, of the 32
// steps of a sub-step, octet k = (0, 2, 1, 3)[l >> 4], the same for both operands.
template <bool TR> struct Reader {
  int at;
  int sw;
  int lk;
  __device__ __forceinline__ void init() {
    const int lane = threadIdx.x & 63, l16 = lane & 15, lq = lane >> 4;
    lk = ((lq & 1) << 1) | (lq >> 1);
    if constexpr (TR) {
      // in each group of 16 lanes, lane 4 t + a points at step t, columns 4 a .. + 3,
      // and receives column (lane & 15) of four steps
      const int t = (lane >> 2) & 3;
      sw = (4 * t) ^ (2 * ((lk >> 1) & 1));
      at = (8 * lk + t) * 512 + 8 * (lane & 1);
    } else {
      sw = (l16 & 7) ^ ((l16 >> 3) & 1);
      at = l16 * 128;
    }
  }
  __device__ __forceinline__ bf16x8 read(const char* operand, int sub, int block) const {
    if constexpr (TR) {
      const int a = threadIdx.x & 3, ch = 2 * block + (a >> 1);
      const char* p = operand + at + ((ch ^ sw) << 4) + 32 * sub * 512;
      const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(reinterpret_cast<lds_bf16x4_t>((lds_ptr_t)p));
      const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(reinterpret_cast<lds_bf16x4_t>((lds_ptr_t)(p + 4 * 512)));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      return *reinterpret_cast<const bf16x8*>(operand + at + (((4 * sub + lk) ^ sw) << 4) + block * 16 * 128);
    }
  }
};

// acc[mi][ni] of wave (wr, wc): row 16 mi + (l & 15) of its 128, columns
// 16 ni + 4 (l >> 4) .. + 3 of its 64.  stage(kt) gives a stage's addresses
// and sets the operands' offsets for it.
template <bool PT, bool QT, typename Stage>
__device__ __forceinline__ void product(Operand<PT>& P, Operand<QT>& Q, int nk, char* lds, f32x4 (&acc)[8][4], Stage&& stage) {
  if (nk <= 0) return;   // no tokens: the sums are empty, and there is nothing to load
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wr = wave >> 2, wc = wave & 3;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_address(lds));
  Reader<PT> rp;
  Reader<QT> rq;
  rp.init();
  rq.init();
  bf16x8 fa[2][4], fb[2][4];
  auto read_p = [&](int b, int sub, int h, int i) { fa[h][i] = rp.read(lds + b * kStageBytes, sub, wr * 8 + 4 * h + i); };
  auto read_q = [&](int b, int sub, int i) { fb[sub][i] = rq.read(lds + b * kStageBytes + kOperandBytes, sub, wc * 4 + i); };
  // A stage is four quarter-steps of 16 MFMAs: (sub-step s, half h of the P
  // blocks); each reads what the next one needs, one read behind each of its
  // first MFMAs, and the last spreads the loads of the stage after the next.
  auto quarter = [&](int s, int h, auto&& rd, int nr, auto&& dma, int nd) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int mi = 4 * h + j / 4, ni = j % 4;
      acc[mi][ni] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[s][ni], fa[h][j / 4], acc[mi][ni], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (j < nr) rd(j);
#pragma unroll
      for (int i = j * nd / 16; i < (j + 1) * nd / 16; ++i) dma(i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto none = [](int) {};
  auto fetch = [&](int kt, int i, const char* p, const char* q) {
    const uint32_t at = lds0 + (kt & 1) * kStageBytes;
    if (i & 1) Q.load(q, at + kOperandBytes, i >> 1);
    else P.load(p, at, i >> 1);
  };
  const char *p, *q;
  stage(0, &p, &q);
#pragma unroll
  for (int i = 0; i < 8; ++i) fetch(0, i, p, q);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (nk > 1) {
    stage(1, &p, &q);
#pragma unroll
    for (int i = 0; i < 8; ++i) fetch(1, i, p, q);
  }
  auto first = [&](int b) { return [&, b](int i) { if (i < 4) read_q(b, 0, i); else read_p(b, 0, 0, i - 4); }; };
#pragma unroll
  for (int i = 0; i < 8; ++i) first(0)(i);
  __builtin_amdgcn_sched_barrier(0);
  auto most_of = [&](int b) {
    quarter(0, 0, [&](int i) { read_p(b, 0, 1, i); }, 4, none, 0);
    quarter(0, 1, [&](int i) { if (i < 4) read_q(b, 1, i); else read_p(b, 1, 0, i - 4); }, 8, none, 0);
    quarter(1, 0, [&](int i) { read_p(b, 1, 1, i); }, 4, none, 0);
    // the next stage has landed, and every read of this buffer is done
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  };
  for (int kt = 0; kt < nk - 2; ++kt) {
    most_of(kt & 1);
    stage(kt + 2, &p, &q);
    quarter(1, 1, first((kt & 1) ^ 1), 8, [&](int i) { fetch(kt, i, p, q); }, 8);
  }
  // the last two stages (or the only one); behind the last the other buffer is read and not used
#pragma unroll 1
  for (int kt = nk > 1 ? nk - 2 : 0; kt < nk; ++kt) {
    most_of(kt & 1);
    quarter(1, 1, first((kt & 1) ^ 1), 8, none, 0);
  }
}

template <int MODE> __global__ __launch_bounds__(kTileThreads, 2) void ffn_tile_kernel(FfnArgs a) {
  constexpr bool kPT = MODE == kFfnDw, kQT = MODE == kFfnDx || MODE == kFfnDw;
  constexpr bool kGated = MODE == kFfnOut || MODE == kFfnMid;
  __shared__ __attribute__((aligned(16))) char lds[2 * kStageBytes];
  const Grid grid = grid_of<MODE>(a, 256);
  int ti, tj;
  tile_of(grid, blockIdx.x / a.slices, &ti, &tj);
  const int slice = blockIdx.x % a.slices;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t all = stages_of<MODE>(a, kFfnStage);
  const int first = static_cast<int>(all * slice / a.slices), count = static_cast<int>(all * (slice + 1) / a.slices) - first;
  f32x4 acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{};
  const char* x = static_cast<const char*>(a.x);
  const char* mid = static_cast<const char*>(a.mid);
  const uint32_t xp = static_cast<uint32_t>(a.xs * 2), wp = static_cast<uint32_t>(a.ws * 2), mp = static_cast<uint32_t>(a.hp) * 4;
  Operand<kPT> P;
  Operand<kQT> Q;
  int which = 0;
  if constexpr (kGated) {
    const int64_t r0 = static_cast<int64_t>(ti) * 256;
    P.init(x + r0 * xp, xp, static_cast<int>(least<int64_t>(a.n - r0, 256)));
    // this wave's 32 stage rows: 32 of one weight, for columns 32 (wave / 2) .. of the tile's 128
    const int f0 = tj * 128 + (wave >> 1) * 32;
    const char* w = static_cast<const char*>((wave & 1) ? a.wu : a.wg);
    // the offsets count from the wave's own rows; Operand::init's from a tile's 256
    Q.pitch = wp;
    Q.lane = lane;
    Q.wave = wave;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = lane >> 3, row = min(f0 + u * 8 + r, a.hidden - 1) - min(f0, a.hidden - 1);
      Q.off[u] = static_cast<uint32_t>(row) * wp + (((lane & 7) ^ r ^ (u & 1)) << 4);
    }
    Q.base = uniform_ptr(w + static_cast<int64_t>(min(f0, a.hidden - 1)) * wp);
    product<kPT, kQT>(P, Q, count, lds, acc, [&](int kt, const char** p, const char** q) {
      *p = P.base + kt * (kFfnStage * 2);
      *q = Q.base + kt * (kFfnStage * 2);
    });
  } else if constexpr (MODE == kFfnDx) {
    const int64_t r0 = static_cast<int64_t>(ti) * 256;
    P.init(mid + r0 * mp, mp, static_cast<int>(least<int64_t>(a.n - r0, 256)));
    Q.init(a.wg, wp, a.kdim - tj * 256);
    const int half = a.hp / kFfnStage;
    product<kPT, kQT>(P, Q, count, lds, acc, [&](int kt, const char** p, const char** q) {
      kt += first;
      *p = P.base + kt * (kFfnStage * 2);
      const int k = (kt < half ? kt : kt - half) * kFfnStage;
      *q = uniform_ptr(static_cast<const char*>(kt < half ? a.wg : a.wu) + static_cast<int64_t>(k) * wp + tj * 512);
      if (a.hidden < a.hp) Q.steps(min(a.hidden - k, kFfnStage));
    });
  } else {
    const int per = grid.rows / 2;
    which = ti >= per;
    const int f0 = (ti - which * per) * 256;
    P.init(mid + (static_cast<int64_t>(which) * a.hp + f0) * 2, mp, a.hp - f0);
    Q.init(x + tj * 512, xp, a.kdim - tj * 256);
    product<kPT, kQT>(P, Q, count, lds, acc, [&](int kt, const char** p, const char** q) {
      kt += first;
      *p = P.base + static_cast<int64_t>(kt) * kFfnStage * mp;
      *q = Q.base + static_cast<int64_t>(kt) * kFfnStage * xp;
      if (a.n < a.mid_rows) Q.steps(static_cast<int>(least<int64_t>(a.n - static_cast<int64_t>(kt) * kFfnStage, kFfnStage)));
    });
    ti -= which * per;
  }
  const int wr = wave >> 2, wc = wave & 3;
#pragma unroll
  for (int mi = 0; mi < 8; ++mi) {
    const int64_t r = static_cast<int64_t>(ti) * 256 + wr * 128 + 16 * mi + (lane & 15);
    if constexpr (kGated) {
#pragma unroll
      for (int ni = 0; ni < 2; ++ni) {
        float g[4], u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = acc[mi][ni][i];
          u[i] = acc[mi][ni + 2][i];
        }
        finish_gated<kBF16, MODE>(a, r, tj * 128 + wc * 32 + 16 * ni + 4 * (lane >> 4), g, u);
      }
    } else {
#pragma unroll
      for (int ni = 0; ni < 4; ++ni) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = acc[mi][ni][i];
        finish_plain<kBF16, MODE>(a, which, slice, r, tj * 256 + wc * 64 + 16 * ni + 4 * (lane >> 4), v);
      }
    }
  }
}

// ---------------------------------------------------------------- fp32 tiles
// 64 x 64, four waves of 16 x 64 on v_mfma_f32_16x16x4_f32, stages of 64 steps
// in two LDS buffers, the next stage's loads under way in registers.  At 32
// cycles a matrix instruction the LDS reads need a third of its bandwidth, so
// small tiles cost little and give small matrices enough blocks.
constexpr int kTile32 = 64, kStep32 = 64;
constexpr int kPitch32 = 68;   // floats: reads along a row and across rows start in different banks

// Part of one operand's stage that a thread moves: 64 rows x 64 steps, zero
// outside.  In LDS as in memory: rows of steps, or (TR) steps of rows.  VEC: runs
// of four are whole and aligned; otherwise element by element.  Every thread
// loads, from the last line and run (element) if it has none of its own, and
// store() writes zeros for it: a branch around a load, or between two ways to
// load, would make the next load wait for it.
template <bool TR, bool VEC> struct Stage32 {
  f32x4 v[4];
  // base(u): where the lines of load u count from, row(line): rows behind it,
  // stride elements apart.  VEC: all within 32 bits of offset, which keeps the
  // addresses' arithmetic short.
  template <typename Base, typename Row>
  __device__ __forceinline__ void load(Base&& base, Row&& row, int64_t stride, int64_t lines, int64_t line0, int cols, int col0) {
    const int last = static_cast<int>(least<int64_t>(lines - line0, 64)) - 1;
    const int col = col0 + (threadIdx.x & 15) * 4;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = row(min(u * 16 + static_cast<int>(threadIdx.x >> 4), last));
      if constexpr (VEC) {
        const uint32_t at = (static_cast<uint32_t>(r) * static_cast<uint32_t>(stride) + min(col, cols - 4)) * 4;
        v[u] = *reinterpret_cast<gptr<const f32x4>>(gmem(reinterpret_cast<const char*>(base(u)) + at));
      } else {
        const float* p = base(u) + r * stride;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = gmem(p)[min(col + i, cols - 1)];
      }
    }
  }
  __device__ __forceinline__ void store(float* lds, int64_t lines, int64_t line0, int cols, int col0) const {
    const int count = static_cast<int>(least<int64_t>(lines - line0, 64));
    const int left = cols - col0 - static_cast<int>(threadIdx.x & 15) * 4;   // elements of the run that exist
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int line = u * 16 + (threadIdx.x >> 4);
      f32x4 x = line < count && left > 0 ? v[u] : f32x4{};
      if constexpr (!VEC)
#pragma unroll
        for (int i = 1; i < 4; ++i) x[i] = i < left ? x[i] : 0.0f;
      *reinterpret_cast<f32x4*>(lds + line * kPitch32 + (threadIdx.x & 15) * 4) = x;
    }
  }
  // Steps 16 s + 4 oct .. + 3 of row (block, l & 15).
  __device__ static __forceinline__ f32x4 read(const float* lds, int s, int block) {
    const int l16 = threadIdx.x & 15, oct = (threadIdx.x >> 4) & 3;
    if constexpr (!TR) {
      return *reinterpret_cast<const f32x4*>(lds + (16 * block + l16) * kPitch32 + 16 * s + 4 * oct);
    } else {
      f32x4 x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = lds[(16 * s + 4 * oct + e) * kPitch32 + 16 * block + l16];
      return x;
    }
  }
};

// VEC: of x and the weights (what the kernels themselves stored is always whole runs).
template <int MODE, bool VEC> __global__ __launch_bounds__(256, 2) void ffn_tile32_kernel(FfnArgs a) {
  constexpr bool kGated = MODE == kFfnOut || MODE == kFfnMid, kPT = MODE == kFfnDw, kQT = !kGated;
  __shared__ __attribute__((aligned(16))) float lds[2][2][64 * kPitch32];
  const Grid grid = grid_of<MODE>(a, kTile32);
  int ti, tj;
  tile_of(grid, blockIdx.x / a.slices, &ti, &tj);
  const int slice = blockIdx.x % a.slices;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float *x = static_cast<const float*>(a.x), *wg = static_cast<const float*>(a.wg), *wu = static_cast<const float*>(a.wu);
  const float* mid = static_cast<const float*>(a.mid);
  const int64_t mp = 2 * static_cast<int64_t>(a.hp);
  int which = 0;
  if constexpr (MODE == kFfnDw) {
    const int per = grid.rows / 2;
    which = ti >= per;
    ti -= which * per;
  }
  const int64_t r0 = static_cast<int64_t>(ti) * kTile32;
  const int c0 = tj * (kGated ? kTile32 / 2 : kTile32);
  const int64_t all = stages_of<MODE>(a, kStep32);
  const int64_t first = all * slice / a.slices, end = all * (slice + 1) / a.slices;
  Stage32<kPT, VEC || !kGated> p;
  Stage32<kQT, VEC> q;
  auto load = [&](int64_t stage) {
    const int64_t k0 = stage * kStep32;
    auto same = [](int line) { return line; };
    if constexpr (kGated) {
      p.load([&](int) { return x + r0 * a.xs; }, same, a.xs, a.n, r0, a.dim, static_cast<int>(k0));
      // 32 rows of one weight, then the same of the other
      const int f0 = min(c0, a.hidden - 1);
      q.load([&](int u) { return (u & 2 ? wu : wg) + f0 * a.ws; }, [&](int line) { return min(c0 + (line & 31), a.hidden - 1) - f0; }, a.ws,
             64, 0, a.dim, static_cast<int>(k0));
    } else if constexpr (MODE == kFfnDx) {
      const bool second = k0 >= a.hp;   // hp holds whole stages
      const int64_t k = k0 - (second ? a.hp : 0);
      p.load([&](int) { return mid + r0 * mp; }, same, mp, a.n, r0, 2 * a.hp, static_cast<int>(k0));
      q.load([&](int) { return (second ? wu : wg) + k * a.ws; }, same, a.ws, a.hidden, k, a.dim, c0);
    } else {
      p.load([&](int) { return mid + k0 * mp + (which ? a.hp : 0); }, same, mp, a.n, k0, a.hp, static_cast<int>(r0));
      q.load([&](int) { return x + k0 * a.xs; }, same, a.xs, a.n, k0, a.dim, c0);
    }
  };
  auto store = [&](int b, int64_t stage) {
    const int64_t k0 = stage * kStep32;
    if constexpr (kGated) {
      p.store(lds[b][0], a.n, r0, a.dim, static_cast<int>(k0));
      q.store(lds[b][1], 64, 0, a.dim, static_cast<int>(k0));
    } else if constexpr (MODE == kFfnDx) {
      p.store(lds[b][0], a.n, r0, 2 * a.hp, static_cast<int>(k0));
      q.store(lds[b][1], a.hidden, k0 - (k0 >= a.hp ? a.hp : 0), a.dim, c0);
    } else {
      p.store(lds[b][0], a.n, k0, a.hp, static_cast<int>(r0));
      q.store(lds[b][1], a.n, k0, a.dim, c0);
    }
  };
  f32x4 acc[4] = {};
  if (first < end) {
    load(first);
    store(0, first);
  }
  __syncthreads();
  for (int64_t st = first; st < end; ++st) {
    const int b = static_cast<int>(st - first) & 1;
    if (st + 1 < end) load(st + 1);
    // a stage's sum is added as a whole: the roundings of a long contraction then
    // grow with its stages, not with its steps
    f32x4 part[4] = {};
    // fragments are read one sub-step ahead of their products: left alone, the
    // compiler reads them right in front of those and waits (4096 tokens, 512 ->
    // 2048: the gradient 595 us instead of 586; 560 with whole runs' loads free of
    // branches, 536 with their offsets in 32 bits)
    f32x4 fp[2], fq[2][4];
    auto read = [&](int s) {
      fp[s & 1] = decltype(p)::read(lds[b][0], s, wave);
#pragma unroll
      for (int j = 0; j < 4; ++j) fq[s & 1][j] = decltype(q)::read(lds[b][1], s, j);
    };
    read(0);
#pragma unroll
    for (int s = 0; s < kStep32 / 16; ++s) {
      if (s + 1 < kStep32 / 16) read(s + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fq[s & 1][j][e], fp[s & 1][e], part[j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += part[j];
    if (st + 1 < end) store(b ^ 1, st + 1);
    __syncthreads();
  }
  // lane l: row l & 15 of the wave's 16, columns 16 j + 4 (l >> 4) .. + 3
  const int64_t r = r0 + wave * 16 + (lane & 15);
  const int c = c0 + 4 * (lane >> 4);
  if constexpr (kGated) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float g[4] = {acc[j][0], acc[j][1], acc[j][2], acc[j][3]};
      const float u[4] = {acc[j + 2][0], acc[j + 2][1], acc[j + 2][2], acc[j + 2][3]};
      finish_gated<kF32, MODE>(a, r, c + 16 * j, g, u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v[4] = {acc[j][0], acc[j][1], acc[j][2], acc[j][3]};
      finish_plain<kF32, MODE>(a, which, slice, r, c + 16 * j, v);
    }
  }
}

// ---------------------------------------------------------------- joining slices
// Adds the slices of dx (kFfnDx) or of both weights' gradients, in order.
template <int DT, int MODE> __global__ __launch_bounds__(256) void ffn_join_kernel(FfnArgs a) {
  const int per = (a.dim + 3) / 4;
  const int64_t rows = MODE == kFfnDx ? a.n : 2 * static_cast<int64_t>(a.hidden);
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, r = id / per;
  const int c = static_cast<int>(id % per) * 4;
  if (r >= rows) return;
  const int64_t pitch = 4 * static_cast<int64_t>(per);
  float v[4] = {};
  for (int s = 0; s < a.slices; ++s) {
    const f32x4 x = *reinterpret_cast<gptr<const f32x4>>(gmem(a.part + (s * rows + r) * pitch + c));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += x[i];
  }
  const int which = MODE == kFfnDw && r >= a.hidden;
  FfnArgs one = a;
  one.slices = 1;
  finish_plain<DT, MODE>(one, which, 0, r - (which ? a.hidden : 0), c, v);
}

// ---------------------------------------------------------------- few tokens
template <int DT> struct Oct;   // eight consecutive steps of a row
template <> struct Oct<kBF16> { bf16x8 v; };
template <> struct Oct<kF32> { f32x4 v[2]; };

template <int DT> __device__ __forceinline__ Oct<DT> octet(const void* row, bool any, int k, int dim, int vec) {
  using T = typename OpElem<DT>::T;
  const T* p = static_cast<const T*>(row);
  Oct<DT> o{};
  if (!any || k >= dim) return o;
  if (vec && k + 8 <= dim) {
    if constexpr (DT == kBF16) {
      o.v = *reinterpret_cast<gptr<const bf16x8>>(gmem(p + k));
    } else {
      o.v[0] = *reinterpret_cast<gptr<const f32x4>>(gmem(p + k));
      o.v[1] = *reinterpret_cast<gptr<const f32x4>>(gmem(p + k + 4));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const T x = k + i < dim ? gmem(p)[k + i] : static_cast<T>(0.0f);
      if constexpr (DT == kBF16) o.v[i] = x;
      else o.v[i >> 2][i & 3] = x;
    }
  }
  return o;
}
__device__ __forceinline__ f32x4 mma(const Oct<kBF16>& a, const Oct<kBF16>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Oct<kF32>& a, const Oct<kF32>& b, f32x4 c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i >> 2][i & 3], b.v[i >> 2][i & 3], c, 0, 0, 0);
  return c;
}

constexpr int kFewWaves = 4;

// Eight steps from k on of a row whose runs of 16 bytes are whole and aligned:
// every lane loads, so that no load waits for another.
template <int DT> __device__ __forceinline__ Oct<DT> whole_octet(const void* row, int k, int dim) {
  using T = typename OpElem<DT>::T;
  const T* p = static_cast<const T*>(row) + (k < dim ? k : 0);
  Oct<DT> o;
  if constexpr (DT == kBF16) {
    o.v = *reinterpret_cast<gptr<const bf16x8>>(gmem(p));
  } else {
    o.v[0] = *reinterpret_cast<gptr<const f32x4>>(gmem(p));
    o.v[1] = *reinterpret_cast<gptr<const f32x4>>(gmem(p + 4));
  }
  if (k >= dim) o = Oct<DT>{};
  return o;
}

// 16 rows of both weights a block, up to 16 G tokens; the waves take the steps by
// turns, 32 U at a time, and their sums meet in LDS in the waves' order.
template <int DT, int G, int U, bool VEC> __global__ __launch_bounds__(64 * kFewWaves) void ffn_few_kernel(FfnArgs a) {
  using T = typename OpElem<DT>::T;
  constexpr int kSums = 2 * G;   // of each weight with each 16 tokens
  __shared__ f32x4 sums[kFewWaves - 1][kSums][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, oct = lane >> 4;
  const int f0 = blockIdx.x * 16, f = f0 + l16;
  const bool any = f < a.hidden;
  const int64_t row = static_cast<int64_t>(any ? f : a.hidden - 1) * a.ws;
  const T* w[2] = {static_cast<const T*>(a.wg) + row, static_cast<const T*>(a.wu) + row};
  const T* x[G];
  bool has[G];
#pragma unroll
  for (int t = 0; t < G; ++t) {
    has[t] = 16 * t + l16 < a.n;
    x[t] = static_cast<const T*>(a.x) + (has[t] ? 16 * t + l16 : a.n - 1) * a.xs;
  }
  f32x4 acc[kSums] = {};
  for (int k0 = wave * 32 * U; k0 < a.dim; k0 += 32 * U * kFewWaves) {
    Oct<DT> ow[U][2], ox[U][G];
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const int k = k0 + 32 * n + 8 * oct;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if constexpr (VEC) ow[n][r] = whole_octet<DT>(w[r], k, a.dim);
        else ow[n][r] = octet<DT>(w[r], any, k, a.dim, a.vec);
      }
#pragma unroll
      for (int t = 0; t < G; ++t) {
        if constexpr (VEC) ox[n][t] = whole_octet<DT>(x[t], k, a.dim);
        else ox[n][t] = octet<DT>(x[t], has[t], k, a.dim, a.vec);
      }
    }
    f32x4 part[kSums] = {};   // added as a whole, as the fp32 tiles' stages are
#pragma unroll
    for (int n = 0; n < U; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int t = 0; t < G; ++t) part[r * G + t] = mma(ow[n][r], ox[n][t], part[r * G + t]);
#pragma unroll
    for (int s = 0; s < kSums; ++s) acc[s] += part[s];
  }
  if (wave > 0)
#pragma unroll
    for (int s = 0; s < kSums; ++s) sums[wave - 1][s][lane] = acc[s];
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int s = 0; s < kSums; ++s)
#pragma unroll
    for (int v = 0; v < kFewWaves - 1; ++v) acc[s] += sums[v][s][lane];
#pragma unroll
  for (int t = 0; t < G; ++t) {
    const float g[4] = {acc[t][0], acc[t][1], acc[t][2], acc[t][3]};
    const float u[4] = {acc[G + t][0], acc[G + t][1], acc[G + t][2], acc[G + t][3]};
    // lane l: token l & 15, rows 4 (l >> 4) .. + 3 of the weights
    finish_gated<DT, kFfnOut>(a, 16 * t + l16, f0 + 4 * oct, g, u);
  }
}

// ---------------------------------------------------------------- padding
__global__ __launch_bounds__(256) void ffn_pad_kernel(const __bf16* src, int64_t stride, __bf16* dst, int64_t rows, int width, int padded) {
  const int per = padded / 8;
  const int64_t id = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  const int64_t r = id / per;
  const int c = static_cast<int>(id % per) * 8;
  if (r >= rows) return;
  const __bf16* s = src + r * stride;
  float v[8];
  if (c + 8 <= width) load_any<8>(s + c, v);
  else
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < width ? static_cast<float>(gmem(s)[c + i]) : 0.0f;
  store_n<8>(dst + r * padded + c, v);
}

template <int DT, int MODE> hipError_t run(const FfnArgs& args, hipStream_t stream) {
  FfnArgs a = args;
  if (MODE == kFfnOut || MODE == kFfnMid) a.slices = 1;
  else a.slices = MODE == kFfnDx ? a.dx_slices : a.dw_slices;
  if constexpr (DT == kBF16) {
    const unsigned blocks = static_cast<unsigned>(grid_of<MODE>(a, 256).all) * a.slices;
    ffn_tile_kernel<MODE><<<dim3(blocks), dim3(kTileThreads), 0, stream>>>(a);
  } else {
    const unsigned blocks = static_cast<unsigned>(grid_of<MODE>(a, kTile32).all) * a.slices;
    // a tile's rows lie within 32 bits of offset (the weights' always do)
    if (a.vec && a.dim % 4 == 0 && a.xs < int64_t{1} << 22) ffn_tile32_kernel<MODE, true><<<dim3(blocks), dim3(256), 0, stream>>>(a);
    else ffn_tile32_kernel<MODE, false><<<dim3(blocks), dim3(256), 0, stream>>>(a);
  }
  if constexpr (MODE == kFfnDx || MODE == kFfnDw) {
    if (a.slices > 1) {
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      const int64_t units = (MODE == kFfnDx ? a.n : 2 * static_cast<int64_t>(a.hidden)) * ((a.dim + 3) / 4);
      ffn_join_kernel<DT, MODE><<<dim3(static_cast<unsigned>((units + 255) / 256)), dim3(256), 0, stream>>>(a);
    }
  }
  return hipGetLastError();
}
template <int DT> hipError_t run_any(int mode, const FfnArgs& a, hipStream_t stream) {
  switch (mode) {
    case kFfnOut: return run<DT, kFfnOut>(a, stream);
    case kFfnMid: return run<DT, kFfnMid>(a, stream);
    case kFfnDx: return run<DT, kFfnDx>(a, stream);
    default: return run<DT, kFfnDw>(a, stream);
  }
}
// Slices of a product's contraction: where its tiles alone leave CUs idle, at
// least eight stages each.  Gradients in us, with slices and without:
//   fp32, 512 -> 2048:  256 tokens 56, 149;  1001 tokens 149, 210
//   bf16, 1024 -> 4096: 512 tokens 87, 211;  2048 tokens 147, 245;  8192 tokens 426, 465
template <int DT, int MODE> int slices_of(const FfnArgs& a) {
  const int64_t tiles = grid_of<MODE>(a, DT == kBF16 ? 256 : kTile32).all;
  if (tiles == 0 || tiles > 128) return 1;
  const int64_t most_ = stages_of<MODE>(a, kFfnStage) / 8;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({(DT == kBF16 ? 256 : 512) / tiles, most_, 16})));
}
template <int DT, int G, int U> void few_any(const FfnArgs& a, hipStream_t stream) {
  const dim3 blocks((a.hidden + 15) / 16), threads(64 * kFewWaves);
  if (a.vec && a.dim % 8 == 0) ffn_few_kernel<DT, G, U, true><<<blocks, threads, 0, stream>>>(a);
  else ffn_few_kernel<DT, G, U, false><<<blocks, threads, 0, stream>>>(a);
}
template <int DT> hipError_t few(const FfnArgs& a, hipStream_t stream) {
  if (a.n <= 16) few_any<DT, 1, 4>(a, stream);
  else if (a.n <= 32) few_any<DT, 2, 4>(a, stream);
  else few_any<DT, 4, 2>(a, stream);
  return hipGetLastError();
}

}  // namespace
}  // namespace ffn

void ffn_slices(int dt, FfnArgs* a) {
  a->dx_slices = dt == kF32 ? ffn::slices_of<kF32, kFfnDx>(*a) : ffn::slices_of<kBF16, kFfnDx>(*a);
  a->dw_slices = dt == kF32 ? ffn::slices_of<kF32, kFfnDw>(*a) : ffn::slices_of<kBF16, kFfnDw>(*a);
}
hipError_t launch_ffn(int dt, int mode, const FfnArgs& a, hipStream_t stream) {
  return dt == kF32 ? ffn::run_any<kF32>(mode, a, stream) : ffn::run_any<kBF16>(mode, a, stream);
}
hipError_t launch_ffn_few(int dt, const FfnArgs& a, hipStream_t stream) {
  return dt == kF32 ? ffn::few<kF32>(a, stream) : ffn::few<kBF16>(a, stream);
}
hipError_t launch_ffn_pad(const void* src, int64_t stride, void* dst, int64_t rows, int width, int padded, hipStream_t stream) {
  const int64_t all = (rows * (padded / 8) + 255) / 256, cols = std::min<int64_t>(all, int64_t{1} << 20);
  const dim3 blocks(static_cast<unsigned>(cols), static_cast<unsigned>((all + cols - 1) / cols));
  ffn::ffn_pad_kernel<<<blocks, dim3(256), 0, stream>>>(static_cast<const __bf16*>(src), stride, static_cast<__bf16*>(dst), rows, width, padded);
  return hipGetLastError();
}

}  // namespace dmuon
