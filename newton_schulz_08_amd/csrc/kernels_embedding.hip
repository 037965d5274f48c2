// Embedding lookup with scaling, and its gradient by sorted tokens, on gfx950.
//
//   out[t, :]    = scale * table[tok[t], :]
//   dtable[v, :] = scale * sum over t with tok[t] = v of dout[t, :]
//
// A token outside [0, vocab) names no row: its output is zero and it gives no
// gradient.  All of it is bound by HBM: one read of the rows and one write.
//
// The gradient needs no atomics.  The plan sorts the tokens stably (an LSD
// radix sort of (token, position) pairs), so equal tokens lie next to each
// other in their order of occurrence.  The sum of a run of equal tokens is then
// formed in fp32 in that order, a long run's in pieces cut at fixed sorted
// positions and added up afterwards: the same batch gives the same bits.
//
// Measured: lookup of 65536 x 4096, fp32 to bf16, 175 us (0.86 GB that it cannot
// do without, 4.9 TB/s).  Gradient with its plan, 65536 x 4096 bf16 to one row
// per distinct token, 252-256 us over three batches in turn (1.06 GB, 4.2 TB/s; 231
// for one batch again and again, part of which the memory-side cache then
// holds), of which the sort takes 34 us; 16384 x 2048 fp32 to a dense 32000-row
// gradient 111 us (0.40 GB; 93 again and again), the sums 61.
#include <hip/hip_runtime.h>

#include "ops.hpp"

namespace dmuon {
namespace {

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }
__device__ __forceinline__ int popc_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<unsigned>(mask >> 32),
                                   __builtin_amdgcn_mbcnt_lo(static_cast<unsigned>(mask), 0));
}

// ---------------------------------------------------------------- lookup
// 2^log_tpr threads take a row, 16 bytes of the output each at a time.  STREAM:
// an output larger than the memory-side cache passes it by, which keeps the
// table's frequent rows there (65536 x 4096 fp32 to bf16: 187 -> 176 us).
template <int TDT, int ODT, bool STREAM>
__global__ __launch_bounds__(256) void embed_kernel(EmbedArgs a, int log_tpr) {
  using T = typename OpElem<TDT>::T;
  using O = typename OpElem<ODT>::T;
  constexpr int C = ODT == kBF16 ? 8 : 4;
  constexpr int U = 2;
  const int tpr = 1 << log_tpr;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) << (8 - log_tpr)) + (threadIdx.x >> log_tpr);
  const int lane = threadIdx.x & (tpr - 1);
  if (row >= a.n) return;
  const int64_t tok = load_index(a.tokens, row, a.tok64);
  const bool known = tok >= 0 && tok < a.vocab;
  const T* src = static_cast<const T*>(a.table) + (known ? tok : 0) * a.dim;
  O* dst = static_cast<O*>(a.out) + row * a.dim;
  const int64_t nch = a.dim / C;
  for (int64_t c0 = lane; c0 < nch; c0 += tpr * U) {
    float v[U][C] = {};
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * tpr < nch && known) load_any<C>(src + (c0 + u * tpr) * C, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int e = 0; e < C; ++e) v[u][e] *= a.scale;
      if (c0 + u * tpr < nch) store_any<C, STREAM>(dst + (c0 + u * tpr) * C, v[u]);
    }
  }
  for (int64_t e = nch * C + lane; e < a.dim; e += tpr)
    gmem(dst)[e] = static_cast<O>(known ? static_cast<float>(gmem(src)[e]) * a.scale : 0.0f);
}

// ---------------------------------------------------------------- plan
__device__ __forceinline__ unsigned plan_key(const PlanArgs& a, int i) {
  const int64_t t = load_index(a.tokens, i, a.tok64);
  return static_cast<unsigned>(t >= 0 && t < a.vocab ? t : a.vocab);   // unknown tokens sort to the end
}

// Lanes of the wave with the same digit as this lane (among `valid` lanes).
__device__ __forceinline__ uint64_t same_digit(unsigned d, int bits, bool valid) {
  uint64_t peers = __ballot(valid);
  for (int b = 0; b < bits; ++b) {
    const bool one = (d >> b) & 1;
    const uint64_t m = __ballot(one);
    peers &= one ? m : ~m;
  }
  return peers;
}

// Inclusive scan over a block of WAVES waves of one value per thread; total in *sum.
template <int WAVES> __device__ __forceinline__ int block_scan(int v, int* wave_tot, int* sum) {
  const int w = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(v, o, 64);
    if (lane_id() >= o) v += t;
  }
  if (lane_id() == 63) wave_tot[w] = v;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int k = 0; k < WAVES; ++k) {
    const int t = wave_tot[k];
    before += k < w ? t : 0;
    all += t;
  }
  __syncthreads();
  *sum = all;
  return v + before;
}

// p[0 .. n) = -1 by `threads` threads.
__device__ __forceinline__ void fill_minus_one(int* p, int64_t n, int64_t thread, int64_t threads) {
  using V = Loose<int, 4>::V;
  for (int64_t i = thread; i < n / 4; i += threads) *reinterpret_cast<gptr<V>>(gmem(p + 4 * i)) = V{-1, -1, -1, -1};
  for (int64_t i = n / 4 * 4 + thread; i < n; i += threads) gmem(p)[i] = -1;
}

// All of the plan in one block: up to 64 WAVES PER tokens, whose pairs stay in
// LDS.  A wave owns 64 PER consecutive ones.
template <int WAVES, int PER>
__global__ __launch_bounds__(64 * WAVES) void plan_small_kernel(PlanArgs a) {
  constexpr int kThreads = 64 * WAVES, kMost = kThreads * PER;
  constexpr int kDigits = kPlanMaxDigits > kThreads ? kPlanMaxDigits / kThreads : 1;   // consecutive ones per thread
  __shared__ unsigned key[2][kMost];
  __shared__ uint16_t idx[2][kMost];
  __shared__ uint16_t cnt[WAVES][kPlanMaxDigits];
  __shared__ int wave_tot[WAVES];
  const int tid = threadIdx.x, w = tid >> 6, lane = lane_id();
  const unsigned mask = (1u << a.bits) - 1;
  unsigned mine[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = (w * PER + j) * 64 + lane;
    mine[j] = i < a.n ? plan_key(a, i) : 0;
  }
  fill_minus_one(a.row_index, a.vocab, tid, kThreads);
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = (w * PER + j) * 64 + lane;
    key[0][i] = mine[j];
    idx[0][i] = static_cast<uint16_t>(i);
  }
  int cur = 0;
  for (int pass = 0; pass < a.passes; ++pass, cur ^= 1) {
    const int shift = pass * a.bits;
    for (int i = tid; i < WAVES * kPlanMaxDigits / 2; i += kThreads) reinterpret_cast<unsigned*>(&cnt[0][0])[i] = 0;
    __syncthreads();
    int rank[PER];
    unsigned k[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = (w * PER + j) * 64 + lane;
      const bool valid = i < a.n;
      k[j] = key[cur][i];
      if ((w * PER + j) * 64 >= a.n) break;   // nothing left in this wave
      const unsigned d = (k[j] >> shift) & mask;
      const uint64_t peers = same_digit(d, a.bits, valid);
      const int below = popc_below(peers);
      const int base = valid ? cnt[w][d] : 0;
      __builtin_amdgcn_wave_barrier();
      if (valid && below == 0) cnt[w][d] = static_cast<uint16_t>(base + __popcll(peers));
      __builtin_amdgcn_wave_barrier();
      rank[j] = base + below;
    }
    __syncthreads();
    // counts -> first places: over the waves of a digit, over the digits
    int c[kDigits][WAVES], total = 0;
#pragma unroll
    for (int g = 0; g < kDigits; ++g)
#pragma unroll
      for (int v = 0; v < WAVES; ++v) c[g][v] = tid * kDigits + g < kPlanMaxDigits ? cnt[v][tid * kDigits + g] : 0;
#pragma unroll
    for (int g = 0; g < kDigits; ++g)
#pragma unroll
      for (int v = 0; v < WAVES; ++v) total += c[g][v];
    int all;
    int run = block_scan<WAVES>(total, wave_tot, &all) - total;
#pragma unroll
    for (int g = 0; g < kDigits; ++g)
#pragma unroll
      for (int v = 0; v < WAVES; ++v) {
        if (tid * kDigits + g < kPlanMaxDigits) cnt[v][tid * kDigits + g] = static_cast<uint16_t>(run);
        run += c[g][v];
      }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = (w * PER + j) * 64 + lane;
      if (i < a.n) {
        const int pos = cnt[w][(k[j] >> shift) & mask] + rank[j];
        key[cur ^ 1][pos] = k[j];
        idx[cur ^ 1][pos] = idx[cur][i];
      }
    }
    __syncthreads();
  }
  // runs of equal tokens
  const unsigned none = static_cast<unsigned>(a.vocab);
  uint64_t heads[PER];
  int here = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = (w * PER + j) * 64 + lane;
    const bool head = i < a.n && key[cur][i] != none && (i == 0 || key[cur][i - 1] != key[cur][i]);
    heads[j] = __ballot(head);
    here += __popcll(heads[j]);
  }
  if (lane == 0) wave_tot[w] = here;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int k = 0; k < WAVES; ++k) {
    base += k < w ? wave_tot[k] : 0;
    all += wave_tot[k];
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = (w * PER + j) * 64 + lane;
    if (i < a.n) {
      const unsigned kv = key[cur][i];
      const bool head = (heads[j] >> lane) & 1;
      const int s = kv == none ? -1 : base + popc_below(heads[j]) + (head ? 0 : -1);
      gmem(a.order)[i] = idx[cur][i];
      gmem(a.slot)[i] = s;
      if (head) {
        gmem(a.rows)[s] = static_cast<int>(kv);
        gmem(a.row_index)[kv] = s;   // behind the clearing: barriers lie between
      }
    }
    base += __popcll(heads[j]);
  }
  for (int i = all + tid; i < a.cap; i += kThreads) gmem(a.rows)[i] = -1;
  if (tid == 0) gmem(a.count)[0] = all;
}

// Digit counts of one block's tokens.
__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(PlanArgs a, int pass) {
  __shared__ int hist[kPlanMaxDigits];
  const int digits = 1 << a.bits, shift = pass * a.bits;
  const int tid = threadIdx.x;
  if (tid < digits) hist[tid] = 0;
  if (pass == 0) {
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
    fill_minus_one(a.row_index, a.vocab, first, step);
    fill_minus_one(a.rows, a.cap, first, step);
  }
  __syncthreads();
  const int i0 = blockIdx.x * a.items;
  const int i1 = least(a.n, i0 + a.items);
  for (int i = i0 + tid; i < i1; i += kPlanThreads) {
    const unsigned k = pass == 0 ? plan_key(a, i) : gmem(a.key[(pass + 1) & 1])[i];
    atomicAdd(&hist[(k >> shift) & (digits - 1)], 1);
  }
  __syncthreads();
  if (tid < digits) gmem(a.counts)[blockIdx.x * digits + tid] = hist[tid];
}

// Stable scatter of one pass: every wave ranks its own consecutive tokens, the
// block adds the counts of the waves and blocks before it.  Up to 64 kHold
// tokens a wave stay in registers between the ranking and the scatter; more
// are ranked a second time.
constexpr int kHold = 4;
__global__ __launch_bounds__(kPlanThreads) void plan_scatter_kernel(PlanArgs a, int pass) {
  __shared__ int cnt[kPlanWaves][kPlanMaxDigits];
  __shared__ int part[2][kPlanThreads];
  __shared__ int wave_tot[kPlanWaves];
  const int tid = threadIdx.x, w = tid >> 6, lane = lane_id();
  const int digits = 1 << a.bits, shift = pass * a.bits;
  const unsigned mask = digits - 1;
  const unsigned* kin = a.key[(pass + 1) & 1];
  const int* iin = a.idx[(pass + 1) & 1];
  unsigned* kout = a.key[pass & 1];
  int* iout = a.idx[pass & 1];
  const int per_wave = a.items / kPlanWaves;   // a multiple of 64
  const int64_t w0 = static_cast<int64_t>(blockIdx.x) * a.items + w * per_wave + lane;
  auto load_key = [&](int64_t i) {
    return i >= a.n ? 0u : pass == 0 ? plan_key(a, static_cast<int>(i)) : gmem(kin)[i];
  };
  auto load_idx = [&](int64_t i) { return i >= a.n ? 0 : pass == 0 ? static_cast<int>(i) : gmem(iin)[i]; };
  // rank of this lane's token among the wave's earlier ones of its digit, counted on
  auto rank = [&](unsigned k, bool valid) {
    const unsigned d = (k >> shift) & mask;
    const uint64_t peers = same_digit(d, a.bits, valid);
    const int below = popc_below(peers);
    const int base = valid ? cnt[w][d] : 0;
    __builtin_amdgcn_wave_barrier();
    if (valid && below == 0) cnt[w][d] = base + __popcll(peers);
    __builtin_amdgcn_wave_barrier();
    return base + below;
  };
  // tokens and their positions, and the counts of all blocks, on their way together
  const bool hold = per_wave <= 64 * kHold;
  unsigned key[kHold];
  int idx[kHold], at[kHold];
#pragma unroll
  for (int h = 0; h < kHold; ++h) {
    key[h] = hold && 64 * h < per_wave ? load_key(w0 + 64 * h) : 0;
    idx[h] = hold && 64 * h < per_wave ? load_idx(w0 + 64 * h) : 0;
  }
  // tokens of each digit in all blocks and in the ones before: as many threads
  // per digit as there are, each on every `groups`-th block
  const int groups = kPlanThreads >> a.bits, digit = tid & (digits - 1), group = tid >> a.bits;
  int before = 0, total = 0;
#pragma unroll 8
  for (int b = group; b < a.blocks; b += groups) {
    const int c = gmem(a.counts)[b * digits + digit];
    before += b < static_cast<int>(blockIdx.x) ? c : 0;
    total += c;
  }
  part[0][tid] = before;
  part[1][tid] = total;
  for (int i = tid; i < kPlanWaves * digits; i += kPlanThreads) cnt[i >> a.bits][i & mask] = 0;
  __syncthreads();
  if (hold) {
#pragma unroll
    for (int h = 0; h < kHold; ++h)
      if (64 * h < per_wave) at[h] = rank(key[h], w0 + 64 * h < a.n);
  } else {
    for (int j = 0; j < per_wave; j += 64) rank(load_key(w0 + j), w0 + j < a.n);
  }
  before = total = 0;
  if (tid < digits)
    for (int g = 0; g < groups; ++g) {
      before += part[0][g * digits + tid];
      total += part[1][g * digits + tid];
    }
  int all;
  const int first = block_scan<kPlanWaves>(total, wave_tot, &all) - total;   // its barriers also end the ranking
  if (tid < digits) {
    int run = first + before;
    for (int k = 0; k < kPlanWaves; ++k) {
      const int t = cnt[k][tid];
      cnt[k][tid] = run;
      run += t;
    }
  }
  __syncthreads();
  if (hold) {
#pragma unroll
    for (int h = 0; h < kHold; ++h)
      if (64 * h < per_wave && w0 + 64 * h < a.n) {
        const int pos = cnt[w][(key[h] >> shift) & mask] + at[h];
        gmem(kout)[pos] = key[h];
        gmem(iout)[pos] = idx[h];
      }
  } else {
    for (int j = 0; j < per_wave; j += 64) {
      const unsigned k = load_key(w0 + j);
      const int pos = rank(k, w0 + j < a.n);   // the counters now start at the wave's first place
      if (w0 + j < a.n) {
        gmem(kout)[pos] = k;
        gmem(iout)[pos] = load_idx(w0 + j);
      }
    }
  }
}

__device__ __forceinline__ bool plan_head(const unsigned* key, int64_t i, unsigned none) {
  const unsigned k = gmem(key)[i];
  return k != none && (i == 0 || gmem(key)[i - 1] != k);
}

// Run heads of one block's sorted tokens.
__global__ __launch_bounds__(kPlanThreads) void plan_heads_kernel(PlanArgs a) {
  __shared__ int wave_tot[kPlanWaves];
  const unsigned* key = a.key[(a.passes + 1) & 1];
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * a.items;
  int mine = 0;
  for (int j = threadIdx.x; j < a.items; j += kPlanThreads)
    if (i0 + j < a.n && plan_head(key, i0 + j, static_cast<unsigned>(a.vocab))) ++mine;
  int all;
  block_scan<kPlanWaves>(mine, wave_tot, &all);
  if (threadIdx.x == 0) gmem(a.heads)[blockIdx.x] = all;
}

// Numbers the runs, behind the heads of the blocks before.
__global__ __launch_bounds__(kPlanThreads) void plan_rows_kernel(PlanArgs a) {
  __shared__ int wave_tot[kPlanWaves];
  const unsigned* key = a.key[(a.passes + 1) & 1];
  const int* idx = a.idx[(a.passes + 1) & 1];
  const unsigned none = static_cast<unsigned>(a.vocab);
  const int tid = threadIdx.x;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * a.items;
  const int mine = tid < static_cast<int>(blockIdx.x) ? gmem(a.heads)[tid] : 0;
  int before;
  block_scan<kPlanWaves>(mine, wave_tot, &before);
  for (int j = 0; j < a.items; j += kPlanThreads) {
    const int64_t i = i0 + j + tid;
    const bool head = i < a.n && plan_head(key, i, none);
    int here;
    const int s = before + block_scan<kPlanWaves>(head ? 1 : 0, wave_tot, &here) - 1;
    if (i < a.n) {
      const unsigned k = gmem(key)[i];
      gmem(a.order)[i] = gmem(idx)[i];
      gmem(a.slot)[i] = k == none ? -1 : s;
      if (head) {
        gmem(a.rows)[s] = static_cast<int>(k);
        gmem(a.row_index)[k] = s;
      }
    }
    before += here;
  }
  if (blockIdx.x == gridDim.x - 1 && tid == 0) gmem(a.count)[0] = before;
}

// ---------------------------------------------------------------- gradient
// The sorted positions are cut into chunks of equal length, so that work is
// even however often a token occurs.  A thread owns one 16-byte column chunk
// and walks its chunk's positions, adding rows of dout; where the run of a
// token ends it writes the row.  A run that crosses a chunk's edge is short when
// it covers no chunk whole: the chunk in which it begins then walks on to its
// end, and the next one starts behind it.  A longer run is cut at the edges and
// leaves fp32 sums in `part` (index 2c: of the run that began before chunk c;
// 2c + 1: of one that goes on behind it), which egrad_join_kernel adds up.
struct Edges {
  int first, last;            // slots of the chunk's first and last position
  bool inherited, crossing;   // the first run began before, the last one goes on behind
  bool cut_before, cut_behind;// ... and is cut there
};
__device__ __forceinline__ Edges chunk_edges(const EmbedGradArgs& a, int64_t chunk) {
  const int64_t p0 = chunk * a.chunk, p1 = least(a.n, p0 + a.chunk);
  const int far_before = p0 >= a.chunk ? gmem(a.slot)[p0 - a.chunk] : -1;
  const int before = p0 > 0 ? gmem(a.slot)[p0 - 1] : -1;
  const int behind = p1 < a.n ? gmem(a.slot)[p1] : -1;
  const int far_behind = p1 + a.chunk <= a.n ? gmem(a.slot)[p1 + a.chunk - 1] : -1;
  Edges e;
  e.first = gmem(a.slot)[p0];
  e.last = gmem(a.slot)[p1 - 1];
  const bool whole = p1 - p0 == a.chunk && e.first == e.last;   // one run covers this chunk
  e.inherited = e.first >= 0 && before == e.first;
  e.crossing = e.last >= 0 && behind == e.last;
  e.cut_before = e.inherited && (far_before == e.first || whole);
  e.cut_behind = e.crossing && (whole || far_behind == e.last);
  return e;
}

// Writes C columns from `col` of a slot's row, without the first `skip` (which
// another thread owns); cols < C only where the row is shorter than C.
template <int GDT, int C>
__device__ __forceinline__ void grad_write(const EmbedGradArgs& a, int slot, int64_t col, int skip, int cols, float* v) {
  using G = typename OpElem<GDT>::T;
  if (slot >= a.cap) return;   // not a slot of this plan
  const int64_t row = a.form == kGradRows ? slot : gmem(a.rows)[slot];
  if (row < 0 || row >= (a.form == kGradRows ? static_cast<int64_t>(a.cap) : a.vocab)) return;
  G* dst = static_cast<G*>(a.grad) + row * a.dim + col;
  if (skip == 0 && cols == C) {
    if (a.form == kGradAdd) {
      float old[C];
      load_any<C>(dst, old);
#pragma unroll
      for (int e = 0; e < C; ++e) v[e] = fmaf(v[e], a.scale, old[e]);
    } else {
#pragma unroll
      for (int e = 0; e < C; ++e) v[e] *= a.scale;
    }
    store_any<C>(dst, v);
  } else {
#pragma unroll
    for (int e = 0; e < C; ++e)
      if (e >= skip && e < cols) {
        const float old = a.form == kGradAdd ? static_cast<float>(gmem(dst)[e]) : 0.0f;
        gmem(dst)[e] = static_cast<G>(a.form == kGradAdd ? fmaf(v[e], a.scale, old) : v[e] * a.scale);
      }
  }
}

// STREAM: dout is larger than the memory-side cache and leaves it alone
// (65536 x 4096 bf16: 294 -> 281 us in all; 8192 rows, which it holds, 64 -> 77).
template <int DT, int GDT, bool STREAM>
__global__ __launch_bounds__(kEgThreads) void egrad_kernel(EmbedGradArgs a, int log_tpr, int col_tiles,
                                                           int64_t sum_blocks) {
  using T = typename OpElem<DT>::T;
  using G = typename OpElem<GDT>::T;
  constexpr int C = DT == kBF16 ? 8 : 4;
  constexpr int U = 4;
  const int tid = threadIdx.x;
  if (static_cast<int64_t>(blockIdx.x) >= sum_blocks) {
    // rows that no token names: of the table, or behind the last distinct token
    const int64_t r0 = (blockIdx.x - sum_blocks) * kEgZeroRows;
    const int64_t rows = a.form == kGradRows ? a.cap : a.vocab;
    const int used = a.form == kGradRows ? gmem(a.count)[0] : 0;
    constexpr int Z = GDT == kBF16 ? 8 : 4;
    const float zero[Z] = {};
    for (int r = 0; r < kEgZeroRows; ++r) {
      const int64_t row = r0 + r;
      if (row >= rows) break;
      if (a.form == kGradRows ? row < used : gmem(a.row_index)[row] >= 0) continue;
      G* dst = static_cast<G*>(a.grad) + row * a.dim;
      const int64_t whole = a.dim / Z * Z;
      // non-temporal: zeros that nothing reads soon need no place in the caches
      // (65536 x 4096 bf16 rows: 309 -> 294 us in all, 32000 x 2048 fp32 dense: 131 -> 115)
      for (int64_t e = tid * Z; e < whole; e += kEgThreads * Z) store_any<Z, true>(dst + e, zero);
      for (int64_t e = whole + tid; e < a.dim; e += kEgThreads) gmem(dst)[e] = static_cast<G>(0.0f);
    }
    return;
  }
  const int tpr = 1 << log_tpr;
  const int64_t group = blockIdx.x / col_tiles;
  const int ct = static_cast<int>(blockIdx.x - group * col_tiles);
  const int64_t chunk = (group << (8 - log_tpr)) + (tid >> log_tpr);
  int64_t col = (static_cast<int64_t>(ct) * tpr + (tid & (tpr - 1))) * C;
  if (chunk >= a.chunks) return;
  const bool mine = col < a.dim;   // lanes without columns still help to find the runs' ends
  // the last columns of a row that is no multiple of C: a whole chunk that
  // reaches back over columns of the thread before, and writes only its own
  const int cols = static_cast<int>(least<int64_t>(C, a.dim));
  const int skip = static_cast<int>(most<int64_t>(0, col + cols - a.dim));
  col -= skip;
  const Edges edges = chunk_edges(a, chunk);
  if (edges.first < 0) return;
  // length of the run of `slot` from position p on, known to be below a chunk
  auto run = [&](int64_t p, int slot) -> int64_t {
    if (log_tpr >= 6) {   // the wave works on one chunk: a lane a position (a chunk has at most 64)
      const int64_t q = p + lane_id();
      return __popcll(__ballot(lane_id() < a.chunk && q < a.n && gmem(a.slot)[least(q, a.n - 1)] == slot));
    }
    int64_t k = 0;
    while (p + k < a.n && gmem(a.slot)[p + k] == slot) ++k;
    return k;
  };
  int64_t p0 = chunk * a.chunk, p1 = least(a.n, p0 + a.chunk);
  const int last = edges.last;
  if (edges.inherited && !edges.cut_before) p0 += run(p0, edges.first);
  if (edges.crossing && !edges.cut_behind && p0 < p1) p1 += run(p1, last);
  if (p0 >= p1 || !mine) return;
  const T* dout = static_cast<const T*>(a.dout) + col;
  int cur = gmem(a.slot)[p0];
  if (cur < 0) return;
  bool began_before = edges.cut_before;
  float acc[C];
#pragma unroll
  for (int e = 0; e < C; ++e) acc[e] = 0.0f;
  auto flush = [&](bool at_end) {
    const bool goes_on = at_end && edges.cut_behind && cur == last;
    if (began_before || goes_on) {
      float* dst = a.part + (2 * chunk + (began_before ? 0 : 1)) * a.dim + col;
      if (skip == 0 && cols == C) {
        store_any<C>(dst, acc);
      } else {
#pragma unroll
        for (int e = 0; e < C; ++e)
          if (e >= skip && e < cols) gmem(dst)[e] = acc[e];
      }
    } else {
      grad_write<GDT, C>(a, cur, col, skip, cols, acc);
    }
    began_before = false;
#pragma unroll
    for (int e = 0; e < C; ++e) acc[e] = 0.0f;
  };
  using V = typename Loose<T, C>::V;
  // slots and positions are read one step ahead of the rows they lead to
  // (65536 x 4096 bf16 rows: 274 us with neither, 254 with bf16 kept as loaded, 236 with both)
  int sn[U], tn[U];
  auto ahead = [&](int64_t p) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t q = least(p + u, p1 - 1);
      sn[u] = gmem(a.slot)[q];
      tn[u] = gmem(a.order)[q];
    }
  };
  ahead(p0);
  for (int64_t p = p0; p < p1; p += U) {
    int s[U];
    V raw[U];   // bf16 is converted where it is added: 57 registers instead of 76, eight waves a SIMD
#pragma unroll
    for (int u = 0; u < U; ++u) {
      s[u] = sn[u];
      const int t = tn[u];
      if (p + u >= p1 || static_cast<unsigned>(t) >= a.n) s[u] = -1;
      if (s[u] >= 0) {
        const T* src = dout + t * a.dim;
        if (cols == C) {
          const auto r = reinterpret_cast<gptr<const V>>(gmem(src));
          if constexpr (STREAM) raw[u] = __builtin_nontemporal_load(r);
          else raw[u] = *r;
        } else {
#pragma unroll
          for (int e = 0; e < C; ++e) raw[u][e] = e < cols ? gmem(src)[e] : static_cast<T>(0.0f);
        }
      }
    }
    ahead(least(p + U, p1 - 1));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s[u] < 0) continue;
      if (s[u] != cur) {
        flush(false);
        cur = s[u];
      }
#pragma unroll
      for (int e = 0; e < C; ++e) acc[e] += static_cast<float>(raw[u][e]);
    }
  }
  flush(true);
}

// Sums of the runs that were cut.  A block looks through kJoinChunks chunks for
// those in which such a run begins, and adds up the run's pieces in its 256
// columns: four waves take every fourth piece, then the four sums are joined in
// order.
constexpr int kJoinChunks = 8;
template <int GDT>
__global__ __launch_bounds__(kEgThreads) void egrad_join_kernel(EmbedGradArgs a) {
  __shared__ float red[4][256];
  const int lane = lane_id(), w = threadIdx.x >> 6;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kJoinChunks;
  bool owner = false;
  int owner_slot = -1;
  if (lane < kJoinChunks && c0 + lane < a.chunks) {
    const Edges e = chunk_edges(a, c0 + lane);
    owner = e.cut_behind && !(e.cut_before && e.first == e.last);
    owner_slot = e.last;
  }
  const int64_t col0 = static_cast<int64_t>(blockIdx.y) * 256 + lane * 4;
  const int cols = static_cast<int>(least<int64_t>(4, a.dim));
  const int skip = static_cast<int>(least<int64_t>(4, most<int64_t>(0, col0 + cols - a.dim)));
  const int64_t col = col0 - skip;   // as in egrad_kernel; skip == cols: nothing of the row is left
  const bool on = col0 < a.dim;
  for (uint64_t owners = __ballot(owner); owners; owners &= owners - 1) {
    const int64_t chunk = c0 + __builtin_ctzll(owners);
    const int seg = __shfl(owner_slot, static_cast<int>(chunk - c0), 64);
    // pieces: the chunks behind this one that begin inside the run
    int64_t last = chunk + 1;
    while (true) {
      const int64_t k = last + lane;
      const uint64_t in =
          __ballot(k < a.chunks && gmem(a.slot)[least(k, static_cast<int64_t>(a.chunks) - 1) * a.chunk] == seg);
      const int m = in == ~0ull ? 64 : __builtin_ctzll(~in);
      last += m;
      if (m < 64) break;
    }
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    auto load = [&](int64_t index, float* v) {
      const float* p = a.part + index * a.dim + col;
      if (cols == 4) {
        load_any<4>(p, v);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = e < cols ? gmem(p)[e] : 0.0f;
      }
    };
    if (on) {
      for (int64_t k0 = chunk + 1 + w; k0 < last; k0 += 4 * 8) {
        float v[8][4] = {};
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (k0 + 4 * u < last) load(2 * (k0 + 4 * u), v[u]);
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] += v[u][e];
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) red[w][lane * 4 + e] = acc[e];
    __syncthreads();
    if (w == 0 && on) {
      float v[4];
      load(2 * chunk + 1, v);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[e] += red[k][lane * 4 + e];
      grad_write<GDT, 4>(a, seg, col, skip, cols, v);
    }
  }
}

int log2_ceil(int64_t v, int most) {
  int l = 0;
  while (l < most && (int64_t{1} << l) < v) ++l;
  return l;
}

}  // namespace

hipError_t launch_embed(int table_dt, int out_dt, const EmbedArgs& a, hipStream_t stream) {
  if (a.n == 0) return hipSuccess;
  const int c = out_dt == kBF16 ? 8 : 4;
  const int log_tpr = log2_ceil((a.dim + c - 1) / c, 8);
  const int64_t rpb = 256 >> log_tpr;
  const dim3 grid(static_cast<unsigned>((a.n + rpb - 1) / rpb));
  const bool streams = static_cast<double>(a.n) * a.dim * (out_dt == kBF16 ? 2 : 4) > 256e6;
  auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, a, log_tpr); };
  auto go = [&](auto cached, auto streamed) {
    if (streams) launch(streamed);
    else launch(cached);
  };
  if (table_dt == kBF16) {
    if (out_dt == kBF16) go(embed_kernel<kBF16, kBF16, false>, embed_kernel<kBF16, kBF16, true>);
    else go(embed_kernel<kBF16, kF32, false>, embed_kernel<kBF16, kF32, true>);
  } else {
    if (out_dt == kBF16) go(embed_kernel<kF32, kBF16, false>, embed_kernel<kF32, kBF16, true>);
    else go(embed_kernel<kF32, kF32, false>, embed_kernel<kF32, kF32, true>);
  }
  return hipGetLastError();
}

hipError_t launch_embed_plan(const PlanArgs& a, hipStream_t stream) {
  if (a.n <= kPlanSmall) {
    // four waves rank up to 1024 tokens, each alone on its SIMD
    if (a.n <= 1024) hipLaunchKernelGGL((plan_small_kernel<4, 4>), dim3(1), dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((plan_small_kernel<16, 4>), dim3(1), dim3(kPlanThreads), 0, stream, a);
    return hipGetLastError();
  }
  for (int pass = 0; pass < a.passes; ++pass) {
    hipLaunchKernelGGL(plan_count_kernel, dim3(a.blocks), dim3(kPlanThreads), 0, stream, a, pass);
    hipLaunchKernelGGL(plan_scatter_kernel, dim3(a.blocks), dim3(kPlanThreads), 0, stream, a, pass);
  }
  hipLaunchKernelGGL(plan_heads_kernel, dim3(a.blocks), dim3(kPlanThreads), 0, stream, a);
  hipLaunchKernelGGL(plan_rows_kernel, dim3(a.blocks), dim3(kPlanThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_embed_grad(int dout_dt, int grad_dt, const EmbedGradArgs& a, hipStream_t stream) {
  const int c = dout_dt == kBF16 ? 8 : 4;
  const int64_t nch = (a.dim + c - 1) / c;
  const int log_tpr = log2_ceil(nch, 8);
  const int tpr = 1 << log_tpr;
  const int col_tiles = static_cast<int>((nch + tpr - 1) / tpr);
  const int sub = kEgThreads / tpr;
  const int64_t sum_blocks = (static_cast<int64_t>(a.chunks) + sub - 1) / sub * col_tiles;
  const int64_t zero_rows = a.form == kGradAdd ? 0 : a.form == kGradRows ? a.cap : a.vocab;
  const int64_t blocks = sum_blocks + (zero_rows + kEgZeroRows - 1) / kEgZeroRows;
  if (blocks == 0) return hipSuccess;
  const bool stream_in = static_cast<double>(a.n) * a.dim * (dout_dt == kBF16 ? 2 : 4) > 256e6;
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kEgThreads), 0, stream, a, log_tpr, col_tiles,
                       sum_blocks);
  };
  auto go = [&](auto cached, auto streamed) {
    if (stream_in) launch(streamed);
    else launch(cached);
  };
  if (dout_dt == kBF16) {
    if (grad_dt == kBF16) go(egrad_kernel<kBF16, kBF16, false>, egrad_kernel<kBF16, kBF16, true>);
    else go(egrad_kernel<kBF16, kF32, false>, egrad_kernel<kBF16, kF32, true>);
  } else {
    if (grad_dt == kBF16) go(egrad_kernel<kF32, kBF16, false>, egrad_kernel<kF32, kBF16, true>);
    else go(egrad_kernel<kF32, kF32, false>, egrad_kernel<kF32, kF32, true>);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.chunks < 2) return e;
  const dim3 jgrid(static_cast<unsigned>((a.chunks + kJoinChunks - 1) / kJoinChunks), static_cast<unsigned>((a.dim + 255) / 256));
  if (grad_dt == kBF16)
    hipLaunchKernelGGL(egrad_join_kernel<kBF16>, jgrid, dim3(kEgThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(egrad_join_kernel<kF32>, jgrid, dim3(kEgThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace dmuon
