// Shared definitions between the host entry points (dmuon_block_api.cpp) and the
// kernels of the operators between a decoder block's projections: norms around
// the block, attention, gated feed-forward.
//
// Every argument travels by value in the kernel's argument block: nothing is
// uploaded, so these launches can be recorded into a graph.
#pragma once

#include "ops.hpp"

namespace dmuon {

// ---------------------------------------------------------------- norms around a block
struct BlockNormArgs {
  const void* x;           // forward: the stream before the block; backward: behind it
  const void* h;           // the block's output
  const void* dx_out;      // backward: gradient of the stream behind the block, or nullptr
  const void* dy;          // backward
  void* x_out;             // forward: the stream behind the block; backward: its gradient before the block
  void* y;                 // forward: the normed stream; backward: gradient of h
  const void* w[3];        // pre, post, gate; nullptr: 1
  void* dw[3];             // their gradients, or nullptr
  int64_t xs, hs, dxs, dys, xos, ys;   // elements between rows
  int64_t rows;
  int dim, post_norm, w_bf16;
  int in_place;            // x_out is x (backward: dx_out)
  float eps, scale, offset;
  float* part;             // backward: blocks x 2 x dim
  float* stats;            // backward, wide rows: rows x 3, the reciprocal lengths of x and h, and mean(dy g_pre xh)
  int stats_only;          // set by the launch: a pass over wide rows that only fills `stats`
  int64_t col_rows;        // backward, wide rows: rows of a block of the pass over columns
  int blocks;              // backward: rows of `part`
};
hipError_t launch_block_norm(int dt, int branch_dt, const BlockNormArgs& a, hipStream_t stream);
hipError_t launch_block_norm_grad(int dt, int branch_dt, const BlockNormArgs& a, hipStream_t stream);
constexpr int kBnMaxFused = 8192;   // widest row whose column sums stay in registers beside the row
// Rows that a block of the backward pass works on at once.
inline int bn_rows_at_once(int64_t dim) { return dim <= 512 ? 4 : 1; }

// ---------------------------------------------------------------- attention over packed sequences
constexpr int kAttnTile = 128;       // rows of a block: queries x the heads that share a key head, or keys
struct AttnArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* out;         // backward: the forward's result
  const void* dout;        // backward
  const int* q_off;        // sequences + 1, or nullptr: one sequence of all tokens
  const int* k_off;
  void* o;                 // forward: out
  float* lse;              // forward: written; backward: read
  void* dq;
  void* dk;
  void* dv;
  float* stats;            // backward: base-2 lse and dout . out of every row, in the rows' order
  float* part;             // forward in slices: per tile, slice and row the sum, then maximum and weight
  int64_t qs, ks, vs, os, dos, dqs, dks, dvs;   // elements between tokens
  int q_tokens, k_tokens, sequences;
  int q_heads, k_heads, group, dim;   // group: query heads of a key head
  unsigned group_inv;                 // ceil(2^32 / group), for rows / group
  int causal, window;
  float scale;
  int vec;                 // every run of 16 bytes of a head is aligned (the 16384-token batch 1.16 ms; otherwise 2.5)
  int slots;               // tiles' places over all sequences, of queries or of keys
  int slices;              // forward: parts of a tile's keys
};
hipError_t launch_attention(int dt, const AttnArgs& a, hipStream_t stream);
hipError_t launch_attention_grad(int dt, const AttnArgs& a, int k_slots, hipStream_t stream);
// Places for tiles of kAttnTile rows: sequence i's begin at floor(first row / tile) + i.
inline int64_t attn_slots(int64_t rows, int64_t sequences) { return rows / kAttnTile + sequences; }
// Head sizes that have kernels; a smaller head is padded with zeros.
inline int attn_padded(int dim) { return dim <= 64 ? 64 : dim <= 96 ? 96 : dim <= 128 ? 128 : dim <= 192 ? 192 : 256; }

// ---------------------------------------------------------------- gated feed-forward
enum Activation : int { kSilu = 0, kGelu = 1 };
// What a launch of the products computes.
enum FfnMode : int {
  kFfnOut = 0,    // h = act(x Wg^T) * (x Wu^T)
  kFfnMid = 1,    // both projections again; their gradients from dh
  kFfnDx = 2,     // dx = dg Wg + du Wu
  kFfnDw = 3,     // dWg = dg^T x, dWu = du^T x
};
struct FfnArgs {
  const void* x;           // tokens x dim, xs apart
  const void* wg;          // hidden x dim, ws apart
  const void* wu;
  const void* dh;          // backward: tokens x hidden
  void* out;               // forward: h; backward: dx
  void* dwg;               // backward: hidden x dim
  void* dwu;
  void* mid;               // backward: mid_rows x 2 hp, the projections' gradients side by side
  int64_t xs, ws, dhs, outs;
  int64_t n, mid_rows;     // tokens; rounded up to whole contraction stages
  int dim, kdim;           // kdim: dim, or for bf16 rounded up to whole stages (zeros)
  int hidden, hp;          // hp: hidden rounded up to whole stages
  int act;
  int vec;                 // the runs of 16 bytes of x and the weights are aligned (dh and results may lie anywhere)
  int dx_slices, dw_slices;   // parts of those products' contractions
  int slices;              // set by the launch: its own
  float* part;             // slices x rows x dim rounded up to four: their sums
};
// Sets both slices, from the sizes alone.
void ffn_slices(int dt, FfnArgs* a);
constexpr int kFfnStage = 64;      // contraction steps of a bf16 stage
// Most tokens that the forward pass takes without tiles: beyond, a wave's sums
// would not fit its registers.
constexpr int kFfnFewTokens = 64;
// Whether it does.  Without tiles the time grows with the weights and the tokens;
// tiles of few rows take the same time for 1 to 64 tokens and, up to a tile a CU,
// for every hidden width.  In us, without and with:
//   bf16, 4096 -> 8192   32 tokens 33, 76;  48 42, 76;  64 47, 76
//         4096 -> 14336  32 tokens 62, 76;  48 78, 76;  64 89, 77
//         4096 -> 28672  16 tokens 108, 118;  24 125, 118;  32 136, 118;  64 189, 119
//         1024 -> 14336  64 tokens 26, 26;  512 -> 14336  64 tokens 15, 18;  512 -> 28672  64 tokens 24, 20
//   fp32, 4096 -> 4096   32 tokens 43, 97;  33 66, 97;  64 70, 97
//         4096 -> 8192   32 tokens 66, 97;  33 100, 97;  64 107, 98
//         4096 -> 14336  32 tokens 155, 164;  33 194, 164;  64 211, 165
inline bool ffn_few(int dt, int64_t tokens, int64_t dim, int64_t hidden) {
  if (tokens > kFfnFewTokens) return false;
  if (dt == kF32) return tokens <= 32 || hidden < 8192;
  return dim < 1024 || tokens * hidden <= 3 << 18;
}
hipError_t launch_ffn_few(int dt, const FfnArgs& a, hipStream_t stream);
hipError_t launch_ffn(int dt, int mode, const FfnArgs& a, hipStream_t stream);
// Copies bf16 rows of `width` elements to rows of `padded`, zeros behind them.
hipError_t launch_ffn_pad(const void* src, int64_t stride, void* dst, int64_t rows, int width, int padded, hipStream_t stream);

}  // namespace dmuon
