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
  float eps, scale, offset;
  float* part;             // backward: blocks x 3 x dim
  float* stats;            // backward, wide rows: rows x 3, the reciprocal lengths of x and h, and mean(dy g_pre xh)
  int stats_only;          // set by the launch: a pass over wide rows that only fills `stats`
  int64_t col_rows;        // backward, wide rows: rows of a block of the pass over columns
  int blocks;              // backward: rows of `part`
};
hipError_t launch_block_norm(int dt, int branch_dt, const BlockNormArgs& a, hipStream_t stream);
hipError_t launch_block_norm_grad(int dt, int branch_dt, const BlockNormArgs& a, hipStream_t stream);
constexpr int kBnMaxFused = 8192;   // widest row whose column sums stay in registers beside the row
// Rows that a block of the backward pass works on at once.
inline int bn_rows_at_once(int64_t dim) { return dim <= 1024 ? 4 : 1; }

}  // namespace dmuon
