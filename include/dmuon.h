/*
 * dmuon.h -- batched Muon optimizer step for AMD Instinct MI355X (gfx950).
 *
 * One call runs the Muon update over a whole set of 2-D weight matrices on one
 * GPU stream:
 *
 *   buf <- mu * buf + grad                          momentum (fp32 state)
 *   Y   <- grad + mu * buf   (Nesterov)  or  buf    Newton-Schulz input
 *   U   <- NS_k(Y)                                  numel >= 100000
 *   U   <- Y                                        numel <  100000
 *   p   <- p - lr * lr_scale_i * U
 *
 * where NS_k normalises by the Frobenius norm (+1e-7), iterates on the wide
 * orientation (the transpose when rows > cols) and applies k times the cubic
 * map X <- 1.5 X - 0.5 (X X^T) X, or a custom odd polynomial (dmuon_ns_config).
 * With weight decay wd the update is p <- p (1 - lr wd) - lr s_i U.
 *
 * Sources: DMuon blog post "DMuon：让矩阵正交化优化器达到接近 AdamW 的分布式训练开销",
 * sections "Muon 核心：Newton-Schulz 迭代" (normalisation, cubic map, transpose
 * to the wide side) and "代码实现" (VanillaMuon: momentum, non-matrix branch,
 * update); DMuon training guide "训练指南", table "超参数指南" (lr, momentum,
 * ns_steps, nesterov: ns_input = grad + mu * buf) and section "编写 Predicate"
 * (numel < 100_000 is too small for NS).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Matrices are dense, row-major, contiguous: element (r, c) of matrix i is at
 *   offset r * cols[i] + c.  rows[i], cols[i] >= 1 and <= DMUON_MAX_DIM.
 * - Tensor pointers are device pointers; the pointer arrays themselves, the
 *   shape arrays and lr_scale are host arrays, read only during the call.
 * - All tensors and the workspace are owned by the caller.  The library
 *   allocates no device memory at run time; its only device memory is the
 *   static scratch of dmuon_muon_step_noalloc, which comes with the library's
 *   code on each GPU.  It keeps no state between calls other than per-device
 *   capability checks, the scratch addresses and the optional profiler record.
 * - Work is enqueued on `hip_stream` (a hipStream_t; NULL = the null stream)
 *   and the call returns without synchronising.  Inputs must stay valid and
 *   unmodified until the stream reaches the end of the enqueued work.
 * - The workspace must hold at least the queried number of bytes and must not
 *   be used by anything else until the enqueued work completes.  Two calls may
 *   run concurrently only with distinct workspaces and disjoint outputs.
 * - The calls cannot be recorded into a HIP graph: each uploads its
 *   descriptors from host memory that lives only for the call.  A call on a
 *   stream that is capturing returns DMUON_ERR_INVALID_ARG.  (The operators
 *   from dmuon_embedding_forward on upload nothing and can be recorded.)
 * - Argument errors are detected before anything is enqueued; nothing is
 *   modified in that case.  A later DMUON_ERR_HIP means a launch failed and the
 *   outputs are unspecified.
 * - Results are bitwise reproducible for the same inputs, and a matrix's result
 *   does not depend on the other matrices in the batch or their order.
 * - Environment (read at each call): DMUON_NS_KERNEL=gemm selects the
 *   DMUON_NS_DIRECT backend whatever ns_config says: every tile of each Gram
 *   product instead of its lower triangle plus a mirrored copy.  It is a
 *   measurement ablation that shows what the triangle saves; results match the
 *   default to rounding.  Every other value, or no value, changes nothing.
 */
#ifndef DMUON_H
#define DMUON_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of gradients, parameters and Newton-Schulz operands.  The blog's
 * newton_schulz accepts float32 or bfloat16.  Momentum is always float32. */
#define DMUON_F32 0
#define DMUON_BF16 1

/* Status codes. */
#define DMUON_OK 0
#define DMUON_ERR_INVALID_ARG 1        /* bad count, shape, pointer, step count, ... */
#define DMUON_ERR_UNSUPPORTED_DTYPE 2  /* dtype is neither DMUON_F32 nor DMUON_BF16 */
#define DMUON_ERR_WORKSPACE 3          /* workspace NULL or smaller than the query */
#define DMUON_ERR_NO_DEVICE 4          /* no HIP device visible */
#define DMUON_ERR_UNSUPPORTED_ARCH 5   /* current device is not gfx950 */
#define DMUON_ERR_HIP 6                /* a HIP runtime call or launch failed */

/* Training guide, "编写 Predicate": matrices with numel < 100_000 skip NS. */
#define DMUON_MIN_NS_NUMEL 100000
/* Largest accepted rows or cols. */
#define DMUON_MAX_DIM 65536
/* Largest accepted ns_steps. */
#define DMUON_MAX_NS_STEPS 64

/*
 * Newton-Schulz configuration: the training guide's `ns_backend` ("超参数指南":
 * "gram" or "direct", or a NewtonSchulz object with custom coefficients; the
 * pages print no coefficients).  Each step maps the iterate X (wide side) to
 *
 *   X <- c0 X + c1 A X + c2 A^2 X,    A = X X^T,
 *
 * an odd polynomial in X; (c0, c1) = (1.5, -0.5) with no c2 is the blog's
 * cubic map ("Muon 核心：Newton-Schulz 迭代").  A NULL config pointer means
 * { DMUON_NS_GRAM, 0, 0, NULL }.
 */
#define DMUON_NS_GRAM 0       /* Gram products on lower-triangle tiles, mirrored (default) */
#define DMUON_NS_DIRECT 1     /* Gram products on every tile */
#define DMUON_MAX_NS_TERMS 3  /* c0, c1, c2 */
typedef struct {
    int backend;          /* DMUON_NS_GRAM or DMUON_NS_DIRECT */
    int num_terms;        /* 0: the cubic map (1.5, -0.5); 2 or 3: coefficients from `coeffs` */
    int per_step;         /* 0: one coefficient set for every step; 1: one set per step (ns_steps sets) */
    const float* coeffs;  /* host; sets of num_terms floats (c0 first), one after another; read during
                             the call; every value finite.  Ignored when num_terms is 0. */
} dmuon_ns_config;

/* Learning-rate scale modes of dmuon_muon_step (s_i below). */
#define DMUON_LR_SCALE_ONE 0        /* s_i = lr_scale[i], or 1 when lr_scale is NULL */
#define DMUON_LR_SCALE_MOONLIGHT 1  /* s_i = 0.2 * sqrt(max(rows_i, cols_i)) * (lr_scale[i], or 1) --
                                       the training guide's per-parameter scaling ("超参数指南", lr) */

/*
 * Workspace size for dmuon_ns_batched over the given shapes and configuration
 * (NULL = default), in bytes.  The blog post's "什么时候用 / 不用？" notes that
 * Newton-Schulz needs temporary matrices; here they are the iterate (two
 * operand copies plus, for bf16, its low half) and the m' x m' Gram matrix per
 * matrix, in the caller's workspace.  Writes *bytes_out and returns DMUON_OK,
 * or an argument error (the shape rules of dmuon_ns_batched, whose
 * newton_schulz in "代码实现" accepts 2-D matrices only).  Needs no GPU.  A
 * three-term polynomial needs an extra m' x m' buffer per matrix.
 */
int dmuon_ns_workspace_bytes(int count, const int64_t* rows, const int64_t* cols, int dtype,
                             const dmuon_ns_config* ns_config, size_t* bytes_out);

/*
 * Newton-Schulz orthogonalisation of `count` independent matrices
 * (blog post, "Muon 核心：Newton-Schulz 迭代" and the newton_schulz listing of
 * "代码实现"):
 *
 *   out_i = NS_{ns_steps}(x_i)
 *
 * x_in[i]  : device, rows[i] x cols[i], `dtype`, read only.
 * x_out[i] : device, rows[i] x cols[i], `dtype`, written (RNE for bf16).  May
 *            equal x_in[i]; must not overlap any other input or output.
 * ns_steps : 0 .. DMUON_MAX_NS_STEPS; 0 returns the normalised input.
 * ns_config: NULL (the cubic map, gram backend) or a host configuration, read
 *            during the call; the workspace must be sized for the same one.
 * Every matrix is orthogonalised, whatever its size.  bf16 inputs run the
 * contractions on bf16 operands with fp32 accumulation; between steps the
 * iterate is kept as a bf16 pair hi + lo (16 significant bits), and all
 * epilogue arithmetic is fp32.
 */
int dmuon_ns_batched(int count, const void* const* x_in, void* const* x_out,
                     const int64_t* rows, const int64_t* cols, int dtype, int ns_steps,
                     const dmuon_ns_config* ns_config,
                     void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * Workspace size for dmuon_muon_step over the given shapes and Newton-Schulz
 * configuration (NULL = default), in bytes: the Newton-Schulz temporaries of
 * the matrices that take that route (blog post, "什么时候用 / 不用？"; matrices
 * below DMUON_MIN_NS_NUMEL need none), plus descriptors and the per-block norm
 * partials.  Same errors as dmuon_ns_workspace_bytes.  Needs no GPU.
 */
int dmuon_muon_step_workspace_bytes(int count, const int64_t* rows, const int64_t* cols, int dtype,
                                    const dmuon_ns_config* ns_config, size_t* bytes_out);

/*
 * One Muon step over `count` matrices (blog post VanillaMuon.step with the
 * training guide's Nesterov input; equations at the top of this header).
 *
 * params[i]     : device, rows x cols, `dtype`; updated in place (RNE for bf16).
 * grads[i]      : device, rows x cols, `dtype`; read only.
 * momentum[i]   : device, rows x cols, float32; updated in place.  Start from
 *                 zeros for a fresh optimizer.
 * mu            : momentum coefficient (0.95 in the pages' defaults).
 * nesterov      : nonzero -> Y = grad + mu * buf (with the updated buf).
 * ns_steps      : 0 .. DMUON_MAX_NS_STEPS (5 in the pages' defaults).
 * ns_config     : NULL (cubic map, gram backend) or a host configuration; the
 *                 workspace must be sized for the same one.
 * lr            : learning rate (0.02 in the pages' defaults).
 * weight_decay  : decoupled decay (training guide, creating the optimizer:
 *                 `weight_decay`, default 0): p <- p (1 - lr wd) - lr s_i U,
 *                 with the unscaled lr in the decay.  Finite.
 * lr_scale_mode : DMUON_LR_SCALE_ONE or DMUON_LR_SCALE_MOONLIGHT.
 * lr_scale      : host array of `count` finite floats multiplying lr per
 *                 matrix, or NULL for 1.0.
 * update_out    : NULL, or a host array of `count` device pointers (entries
 *                 may be NULL) receiving U_i as float32, rows x cols.
 * norms_out     : NULL, or a device float32 array of `count` entries receiving
 *                 ||Y_i||_F.
 * params, grads, momentum and non-NULL update_out entries must be distinct
 * non-overlapping buffers.
 * Range: the 1/(||Y|| + 1e-7) scale is folded into the first Newton-Schulz
 * step, whose Gram product accumulates the unnormalised Y Y^T in fp32.  A
 * matrix with ||Y||_F >= 2^63 (about 9.2e18; its norms_out entry may be inf)
 * is outside that range and gets a NaN update, as a non-finite gradient does;
 * the other matrices of the call are unaffected.
 */
int dmuon_muon_step(int count, void* const* params, const void* const* grads, float* const* momentum,
                    const int64_t* rows, const int64_t* cols, int dtype,
                    int ns_steps, const dmuon_ns_config* ns_config,
                    float mu, int nesterov, float lr, float weight_decay,
                    int lr_scale_mode, const float* lr_scale,
                    float* const* update_out, float* norms_out,
                    void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * Workspace size for dmuon_muon_step_clipped, in bytes: that of
 * dmuon_muon_step for the same shapes and configuration, plus the clip's
 * per-tile partial sums and per-segment coefficients.  Needs no GPU.
 */
int dmuon_muon_step_clip_workspace_bytes(int count, const int64_t* rows, const int64_t* cols, int dtype,
                                         const dmuon_ns_config* ns_config, int num_segments, size_t* bytes_out);

/*
 * dmuon_muon_step with per-segment global p-norm gradient clipping folded in
 * (training guide, "梯度裁剪": the Muon clip runs on the reduced gradients
 * before momentum and Newton-Schulz; "regular / Muon / AdamW 的融合 CUDA 裁剪":
 * per-segment norms and coefficients computed in one fused pass).  The clip is
 * dmuon_clip_grad_norm's rule with the matrices as its tensors:
 *
 *   total_s = || gradients of segment s ||_p
 *   coef_s  = min(max_norm[s] / (total_s + 1e-6), 1)
 *
 * and the step then runs on coef_{segment[i]} * grads[i], formed in fp32 as
 * each gradient element is read and never rounded to the gradient dtype.  The
 * caller's gradients are not rewritten (unlike dmuon_clip_grad_norm), which
 * saves that pass: clipping costs one extra read of the gradients.
 *
 * segment[i]   : host, the clipping segment of matrix i, in [0, num_segments).
 * num_segments, max_norm (host, finite, >= 0), norm_type (p > 0 or +inf),
 * totals_out (NULL or device float32[num_segments]): as in
 * dmuon_clip_grad_norm.  Every other argument as in dmuon_muon_step; the
 * workspace is sized by dmuon_muon_step_clip_workspace_bytes.  A segment whose
 * coefficient is 1 gets bitwise the result of dmuon_muon_step.
 */
int dmuon_muon_step_clipped(int count, void* const* params, const void* const* grads, float* const* momentum,
                            const int64_t* rows, const int64_t* cols, int dtype,
                            int ns_steps, const dmuon_ns_config* ns_config,
                            float mu, int nesterov, float lr, float weight_decay,
                            int lr_scale_mode, const float* lr_scale,
                            float* const* update_out, float* norms_out,
                            const int* segment, int num_segments, const float* max_norm, float norm_type,
                            float* totals_out, void* workspace, size_t workspace_bytes, void* hip_stream);

/* Scratch held by the library for dmuon_muon_step_noalloc: 64 MiB on each GPU
 * the library is loaded on, from the load until the process ends. */
#define DMUON_NOALLOC_SCRATCH_BYTES 67108864

/*
 * dmuon_muon_step for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid allocation.
 * Same arguments and results as dmuon_muon_step (bitwise: the same kernels),
 * but the scratch is the library's own static device array of
 * DMUON_NOALLOC_SCRATCH_BYTES per GPU instead of a caller workspace; the call
 * allocates nothing.  A set whose dmuon_muon_step_workspace_bytes exceeds
 * DMUON_NOALLOC_SCRATCH_BYTES is rejected with DMUON_ERR_WORKSPACE before
 * anything is enqueued.  Every call on one GPU shares that GPU's array: calls
 * that overlap on one GPU (other streams or threads) race and give undefined
 * results; calls ordered on one stream are safe.  The array needs no clearing
 * between calls (every stage writes what it later reads).  The stream-capture
 * restriction of dmuon_muon_step applies as well (host-side descriptors).
 */
int dmuon_muon_step_noalloc(int count, void* const* params, const void* const* grads, float* const* momentum,
                            const int64_t* rows, const int64_t* cols, int dtype,
                            int ns_steps, const dmuon_ns_config* ns_config,
                            float mu, int nesterov, float lr, float weight_decay,
                            int lr_scale_mode, const float* lr_scale,
                            float* const* update_out, float* norms_out, void* hip_stream);

/*
 * Workspace size for dmuon_clip_grad_norm, in bytes.  Needs no GPU.
 */
int dmuon_clip_grad_norm_workspace_bytes(int count, const int64_t* numel, int num_segments, size_t* bytes_out);

/*
 * Per-segment global p-norm gradient clipping, in place (training guide,
 * "梯度裁剪": the Muon clip before momentum and Newton-Schulz, and the fused
 * bucketed clip that keeps per-segment semantics; the rule of PyTorch's
 * clip_grad_norm_, which the guide names for the other parameters):
 *
 *   total_s = (sum over i with segment[i] == s of sum |g_i|^p)^(1/p)   (max |g_i| for p = +inf)
 *   coef_s  = min(max_norm[s] / (total_s + 1e-6), 1)
 *   g_i    <- coef_s * g_i     (a segment with coef_s == 1 is not rewritten)
 *
 * grads[i]     : device, numel[i] contiguous elements of `dtype`, updated in
 *                place (RNE for bf16); distinct buffers.
 * numel[i]     : >= 0 (0 = an empty tensor, ignored).
 * segment[i]   : host, in [0, num_segments).
 * max_norm[s]  : host, finite, >= 0.
 * norm_type    : p > 0 or +inf.  Totals accumulate in fp32 in a fixed order,
 *                so results are bitwise reproducible.  A non-finite total
 *                gives a coefficient of 0 (total +inf) or NaN (total NaN),
 *                as the reference rule does.
 * totals_out   : NULL or device float32[num_segments] receiving total_s.
 * count == 0 enqueues nothing.
 */
int dmuon_clip_grad_norm(int count, void* const* grads, const int64_t* numel, int dtype, const int* segment,
                         int num_segments, const float* max_norm, float norm_type, float* totals_out,
                         void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * Workspace size for dmuon_adamw_step, in bytes.  Needs no GPU.
 */
int dmuon_adamw_step_workspace_bytes(int count, const int64_t* numel, size_t* bytes_out);

/*
 * One AdamW step over `count` non-matrix parameters, in place (training
 * guide, "第 4 步：创建优化器": the parameters Muon does not take form a
 * standard AdamW group with adamw_lr, adamw_betas, adamw_eps and
 * adamw_weight_decay; blog post, section "为什么需要矩阵感知优化器": the
 * update subtracts alpha m_hat / (sqrt(v_hat) + eps) with bias-corrected
 * moments).  Read as PyTorch's AdamW, per element in fp32:
 *
 *   p <- p (1 - lr weight_decay)
 *   m <- beta1 m + (1 - beta1) g
 *   v <- beta2 v + (1 - beta2) g^2
 *   p <- p - (lr / (1 - beta1^step)) m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 *
 * params[i]     : device, numel[i] contiguous elements of `dtype`; updated in
 *                 place (RNE for bf16).
 * grads[i]      : device, numel[i] elements of `dtype`; read only.
 * exp_avg[i], exp_avg_sq[i] : device, numel[i] float32 moments, updated in
 *                 place.  Start both from zeros.
 * numel[i]      : >= 0 (0 = an empty tensor, ignored; its pointers may be NULL).
 * step          : the step counter t >= 1 of this update (1 on the first call).
 * lr, weight_decay : finite.  beta1, beta2 in [0, 1).  eps finite, >= 0.
 *                 The pages' defaults: lr 1e-3, betas (0.9, 0.999), eps 1e-8,
 *                 weight_decay 0.01.
 * All buffers must be distinct and aligned to their element size; 16-byte
 * alignment (8-byte for bf16 parameters and gradients) takes the vector path.
 * The bias corrections and 1 - lr weight_decay are formed in double on the
 * host and rounded to float once.  count == 0 enqueues nothing.
 */
int dmuon_adamw_step(int count, void* const* params, const void* const* grads, float* const* exp_avg,
                     float* const* exp_avg_sq, const int64_t* numel, int dtype, int step, float lr, float beta1,
                     float beta2, float eps, float weight_decay, void* workspace, size_t workspace_bytes,
                     void* hip_stream);

/* ------------------------------------------------------------------------
 * Operators that feed the non-matrix parameters of a training step: the
 * embedding table, the norm gains and the output head, which the training
 * guide ("第 4 步：创建优化器") leaves to the AdamW group.
 *
 * They keep the conventions above, with these additions:
 * - Every argument travels with the launch, nothing is uploaded: these calls
 *   may be recorded into a HIP graph (kernel timing is off while a stream
 *   captures).  Workspaces are then the graph's: two graphs, or a graph and
 *   eager calls, share one only if they never overlap in time.
 * - All pointers belong to the current device.
 * - Any pointer aligned to its element size is accepted; 16-byte aligned rows are
 *   the fastest.
 * - bf16 results are rounded once (RNE) from fp32.
 * - The same inputs in the same shapes give the same bits, whatever their
 *   addresses and strides.  The order of a sum may follow the shape of the call
 *   (the number of rows or tokens in it), never what other rows hold; but in
 *   dmuon_embedding_backward it follows the batch's tokens, whose sorted order
 *   decides where a long run of one token is cut.
 * ------------------------------------------------------------------------ */

/* Types of token, index and position arrays. */
#define DMUON_I32 2
#define DMUON_I64 3

#define DMUON_MAX_TOKENS 4194304    /* tokens or rows per call */
#define DMUON_MAX_VOCAB 16777216    /* rows of a table, length of a row of logits */
#define DMUON_MAX_HEAD_DIM 512
#define DMUON_MAX_HEADS 1024
#define DMUON_MAX_TEACHER_K 1024    /* teacher entries per row */

/*
 * Embedding lookup with scaling: out[t, :] = scale * table[tokens[t], :].
 *
 * table  : device, vocab x dim, table_dtype, read only.
 * tokens : device, n entries of token_dtype (DMUON_I32 or DMUON_I64).  A token
 *          outside [0, vocab) names no row: its output row is zero.
 * out    : device, n x dim, out_dtype; must not overlap table or tokens.
 * scale  : finite (sqrt(dim) in models that scale their embeddings).
 */
int dmuon_embedding_forward(const void* table, int64_t vocab, int64_t dim, int table_dtype, const void* tokens,
                            int64_t n, int token_dtype, float scale, void* out, int out_dtype, void* hip_stream);

/*
 * Sorted order of a batch's tokens, which dmuon_embedding_backward sums along
 * and dmuon_adamw_rows_step looks rows up in.  With U distinct tokens inside
 * [0, vocab) and cap = min(n, vocab):
 *
 * order[n]         : positions of the batch, sorted by token (stable); positions
 *                    of tokens outside [0, vocab) come last.
 * slot[n]          : slot[i] = number of the distinct token of position order[i]
 *                    (0 .. U - 1, ascending), or -1 outside [0, vocab).
 * rows[cap]        : the distinct tokens, ascending; -1 from U on.
 * row_index[vocab] : the inverse: the number of a distinct token, or -1.
 * count[1]         : U.
 * All are device int32 and written whole.
 */
int dmuon_embedding_plan_workspace_bytes(int64_t n, int64_t vocab, size_t* bytes_out);
int dmuon_embedding_plan(const void* tokens, int64_t n, int token_dtype, int64_t vocab, int32_t* order, int32_t* slot,
                         int32_t* rows, int32_t* row_index, int32_t* count, void* workspace, size_t workspace_bytes,
                         void* hip_stream);

/* Forms of the embedding gradient. */
#define DMUON_EMBED_DENSE 0   /* grad is vocab x dim, written whole: zero rows for tokens not in the batch */
#define DMUON_EMBED_ADD 1     /* grad is vocab x dim: the batch's rows are added to, the others left as they are */
#define DMUON_EMBED_ROWS 2    /* grad is cap x dim: row i belongs to token rows[i]; zero rows from U on */

/*
 * Gradient of dmuon_embedding_forward with respect to the table:
 *
 *   grad[v, :] = scale * sum over t with tokens[t] = v of dout[t, :]
 *
 * Sums are fp32, a token's positions in their order in the batch, cut into
 * pieces at fixed sorted positions: the same inputs give the same bits.
 *
 * dout      : device, n x dim, dout_dtype.  Rows of tokens outside [0, vocab)
 *             are not read.
 * order, slot, rows, row_index, count : as dmuon_embedding_plan wrote them for
 *             the same n and vocab.
 * grad      : device, grad_dtype; with DMUON_EMBED_ADD the sum is fp32 and
 *             rounded once.
 */
int dmuon_embedding_backward_workspace_bytes(int64_t n, int64_t dim, int dout_dtype, size_t* bytes_out);
int dmuon_embedding_backward(const void* dout, int64_t n, int64_t dim, int dout_dtype, float scale,
                             const int32_t* order, const int32_t* slot, const int32_t* rows,
                             const int32_t* row_index, const int32_t* count, int64_t vocab, int form, void* grad,
                             int grad_dtype, void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * dmuon_adamw_step for one table whose gradient comes as rows.  Row r of the
 * table has the gradient grad_rows[row_index[r], :], or zero where
 * row_index[r] is outside [0, n_grad_rows); every element of the table takes
 * the AdamW update (the moments of rows without a gradient decay as they would
 * under a zero gradient).  Bitwise the result of dmuon_adamw_step on the dense
 * gradient, which is never formed.
 *
 * param     : device, rows x dim, `dtype`; updated in place.
 * grad_rows : device, n_grad_rows x dim, `dtype` (the DMUON_EMBED_ROWS form);
 *             may be NULL when n_grad_rows is 0.
 * row_index : device, int32[rows].
 * exp_avg, exp_avg_sq : device, rows x dim float32; updated in place.
 * Other arguments as in dmuon_adamw_step.
 */
int dmuon_adamw_rows_step(void* param, const void* grad_rows, int64_t n_grad_rows, const int32_t* row_index,
                          float* exp_avg, float* exp_avg_sq, int64_t rows, int64_t dim, int dtype, int step, float lr,
                          float beta1, float beta2, float eps, float weight_decay, void* hip_stream);
/* The argument checks of that step alone, without a device: for a caller that
 * has several steps to take, all or none. */
int dmuon_adamw_rows_check(const void* param, const void* grad_rows, int64_t n_grad_rows, const int32_t* row_index,
                           const float* exp_avg, const float* exp_avg_sq, int64_t rows, int64_t dim, int dtype,
                           int step, float lr, float beta1, float beta2, float eps, float weight_decay);

/*
 * Distillation from a teacher's top logits, loss and gradient in one call.
 * With q = softmax(teacher / T) over a row's valid teacher entries and z the
 * student's row:
 *
 *   KD     = T^2 sum_j q_j (log q_j - log softmax(z / T)[index_j])
 *   CE     = -log softmax(z)[label]
 *   losses = row_weight (kd_weight KD + ce_weight CE)
 *   dlogits = grad_scale * d losses / dz
 *
 * logits    : device, n rows of vocab elements of `dtype`, logits_stride
 *             elements apart (>= vocab).
 * teacher_index  : device, n x k, index_dtype.  An entry outside [0, vocab) is
 *             left out (rows with fewer entries are padded with -1); entries
 *             that name the same element add up.
 * teacher_logits : device, n x k float32; any constant per row cancels, so log
 *             probabilities serve as well.  -inf gives q = 0.
 * labels    : NULL (then ce_weight must be 0), or device, n entries of
 *             index_dtype.  A label outside [0, vocab) leaves CE out of its row.
 * k         : 0 .. DMUON_MAX_TEACHER_K; 0 needs kd_weight = 0.
 * temperature : T in [1e-6, 1e6].  kd_weight, ce_weight, grad_scale: finite.
 * row_weight : NULL (1), or device float32[n].  A row of weight 0 is not read:
 *             its loss and gradient are 0 whatever it holds.  A row without a
 *             valid teacher entry and without a label is read, but to no effect:
 *             both are 0 whatever it holds, too.
 * losses    : device float32[n].
 * dlogits   : NULL (loss only), or device, n rows of vocab elements of
 *             `dtype`, dlogits_stride apart.  May equal logits with the same
 *             stride (in place); must not overlap it otherwise.  Elements
 *             between the rows are left as they are.
 * -inf logits are masked elements (probability 0), and so are finite ones as
 * far below the row's largest as masks lie.  Only differences within a row count,
 * wherever it lies: one that holds a single value throughout is an even
 * distribution.  A row of nothing but -inf has no distribution and gets NaN.
 */
int dmuon_distill_loss_workspace_bytes(int64_t n, int64_t vocab, size_t* bytes_out);
int dmuon_distill_loss(const void* logits, int64_t n, int64_t vocab, int64_t logits_stride, int dtype,
                       const void* teacher_index, int index_dtype, const float* teacher_logits, int k,
                       const void* labels, float temperature, float kd_weight, float ce_weight,
                       const float* row_weight, float grad_scale, float* losses, void* dlogits,
                       int64_t dlogits_stride, void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * Shape and types of dmuon_qk_norm_rope_forward and _backward.
 */
typedef struct {
    int64_t tokens;       /* 0 .. DMUON_MAX_TOKENS */
    int q_heads, k_heads; /* 0 .. DMUON_MAX_HEADS; not both 0 */
    int head_dim;         /* D, 1 .. DMUON_MAX_HEAD_DIM */
    int rot_dim;          /* rotated elements of a head: even, 0 .. D; 0 = norm only */
    int interleaved;      /* 0: pairs (i, i + rot_dim / 2); 1: pairs (2 i, 2 i + 1) */
    int64_t max_pos;      /* rows of the rotation table */
    float eps;            /* finite, >= 0 */
    float weight_offset;  /* finite; 1 for gains stored around zero */
    int dtype;            /* queries, keys, outputs and their gradients */
    int weight_dtype;     /* gains and their gradients */
    int pos_dtype;        /* DMUON_I32 or DMUON_I64 */
} dmuon_qk_shape;

/*
 * Root-mean-square norm of every query and key head, then the rotation by the
 * token's position:
 *
 *   n = x / sqrt(mean(x^2) + eps) * (weight_offset + w),   out = R(position) n
 *
 * q, k       : device; token t's heads are contiguous (heads x D) at element
 *              t * stride: a packed projection's output is read in place.
 * q_weight, k_weight : device, D entries of weight_dtype, or NULL for no gain.
 * positions  : device, tokens entries.  A negative position marks a padding
 *              token: its outputs are zero whatever its inputs hold.  A
 *              position >= max_pos gives NaN.  When rot_dim is 0 only the sign
 *              counts, and NULL means that no token is padding.
 * rope       : device float32, max_pos x rot_dim: a position's rot_dim / 2
 *              cosines, then its sines.  NULL when rot_dim is 0.
 * q_out, k_out : device; may equal q and k with the same stride (in place).
 * Pointers of a tensor with 0 heads are ignored.  The sum of a head's squares
 * is formed in float32 and has to be finite (and, when eps is 0, normal).
 */
int dmuon_qk_norm_rope_forward(const dmuon_qk_shape* shape, const void* q, int64_t q_stride, const void* k,
                               int64_t k_stride, const void* q_weight, const void* k_weight, const void* positions,
                               const float* rope, void* q_out, int64_t q_out_stride, void* k_out,
                               int64_t k_out_stride, void* hip_stream);

/*
 * Gradients of dmuon_qk_norm_rope_forward: dq, dk from dq_out, dk_out and the
 * forward's inputs, and the gains' gradients, summed over tokens and heads in
 * fp32 in a fixed order.  Padding tokens get zeros and add nothing to the gains.
 *
 * dq, dk may equal dq_out, dk_out or q, k with the same stride.
 * dq_weight, dk_weight : device, D entries of weight_dtype, or NULL.
 */
int dmuon_qk_norm_rope_backward_workspace_bytes(const dmuon_qk_shape* shape, size_t* bytes_out);
int dmuon_qk_norm_rope_backward(const dmuon_qk_shape* shape, const void* dq_out, int64_t dq_out_stride,
                                const void* dk_out, int64_t dk_out_stride, const void* q, int64_t q_stride,
                                const void* k, int64_t k_stride, const void* q_weight, const void* k_weight,
                                const void* positions, const float* rope, void* dq, int64_t dq_stride, void* dk,
                                int64_t dk_stride, void* dq_weight, void* dk_weight, void* workspace,
                                size_t workspace_bytes, void* hip_stream);

/*
 * Shape and types of dmuon_block_norm_forward and _backward.
 */
typedef struct {
    int64_t rows;         /* 0 .. DMUON_MAX_TOKENS */
    int64_t dim;          /* 1 .. DMUON_MAX_DIM */
    int post_norm;        /* 1: the block's output is normed before it is added */
    float eps;            /* finite, >= 0 */
    float residual_scale; /* s, finite */
    float weight_offset;  /* finite; 1 for gains stored around zero (not for the gate) */
    int dtype;            /* the residual stream and its gradients */
    int branch_dtype;     /* the block's output, the normed stream and their gradients */
    int weight_dtype;     /* gains, gate and their gradients */
} dmuon_block_norm_shape;

/*
 * What lies between two blocks: the norm of a block's output h, its gate and
 * scale, the residual sum, and the norm in front of the next block:
 *
 *   b     = h / sqrt(mean(h^2) + eps) * (weight_offset + post)    or b = h
 *   x_out = x + s * gate * b
 *   y     = x_out / sqrt(mean(x_out^2) + eps) * (weight_offset + pre)
 *
 * y reads x_out as it is stored.  pre, post, gate: device, dim entries of
 * weight_dtype, or NULL for a factor of 1; post is NULL without post_norm.
 * Row r of a tensor begins at element r * stride.  x_out may equal x, and y
 * may equal h, with the same stride.  The sums of a row's squares are formed in
 * float32 and have to be finite (and, when eps is 0, normal).
 */
int dmuon_block_norm_forward(const dmuon_block_norm_shape* shape, const void* x, int64_t x_stride, const void* h,
                             int64_t h_stride, const void* pre, const void* post, const void* gate, void* x_out,
                             int64_t x_out_stride, void* y, int64_t y_stride, void* hip_stream);

/*
 * Gradients of dmuon_block_norm_forward: dx and dh from dx_out, dy, the stream
 * behind the block and the block's output; the gains' and the gate's
 * gradients, summed over rows in fp32 in a fixed order.
 *
 * dx_out     : device, gradient of x_out by its other readers, or NULL for none.
 * dx         : device; may equal dx_out with the same stride.
 * dpre, dpost, dgate : device, dim entries of weight_dtype, or NULL.  dpost is
 *              NULL without post_norm.
 */
int dmuon_block_norm_backward_workspace_bytes(const dmuon_block_norm_shape* shape, size_t* bytes_out);
int dmuon_block_norm_backward(const dmuon_block_norm_shape* shape, const void* dx_out, int64_t dx_out_stride,
                              const void* dy, int64_t dy_stride, const void* x_out, int64_t x_out_stride,
                              const void* h, int64_t h_stride, const void* pre, const void* post, const void* gate,
                              void* dx, int64_t dx_stride, void* dh, int64_t dh_stride, void* dpre, void* dpost,
                              void* dgate, void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * Shape and types of dmuon_attention_forward and _backward.
 */
#define DMUON_MAX_ATTENTION_DIM 256
typedef struct {
    int64_t q_tokens;     /* 0 .. DMUON_MAX_TOKENS; times q_heads / k_heads at most 2^30 */
    int64_t k_tokens;     /* 0 .. DMUON_MAX_TOKENS */
    int64_t sequences;    /* 1 .. DMUON_MAX_TOKENS */
    int q_heads, k_heads; /* 1 .. DMUON_MAX_HEADS; q_heads a multiple of k_heads */
    int head_dim;         /* D, 1 .. DMUON_MAX_ATTENTION_DIM */
    int causal;           /* 1: a query sees no key behind it */
    int window;           /* with causal: the keys a query sees at most; 0 = no limit */
    float scale;          /* of q . k; > 0, and finite times log2(e), as the scores have to be */
    int dtype;            /* queries, keys, values, outputs and their gradients */
} dmuon_attention_shape;
/* A call takes less than 2^24 tiles: of 128 (query, head) rows, and of 128 keys,
 * a key head, one more of each a sequence. */

/*
 * Attention over packed sequences:
 *
 *   out = softmax(scale q . k over the visible keys) v,
 *   lse = log of the sum of exp(scale q . k) over them.
 *
 * Sequence b has the queries q_offsets[b] .. q_offsets[b + 1] - 1 and the keys
 * k_offsets[b] .. k_offsets[b + 1] - 1.  Query i of its lq sees key j of its lk
 * when, with causal, j <= i + lk - lq, and, with a window too,
 * j > i + lk - lq - window: the last query stands at the last key, so one call
 * serves whole sequences and single new tokens behind a cache.  Caches that grow
 * in place have room behind them, which a sequence without queries takes: with
 * room for C keys each and n0, n1 in use, q_offsets 0, 1, 1, 2, 2 and k_offsets
 * 0, n0, C, C + n1, 2 C; from token to token only the offsets change.  A query that
 * sees no key has out 0 and lse -infinity.  Query head h reads key head
 * h / (q_heads / k_heads).
 *
 * q, k, v, out : device; token t's heads are contiguous (heads x D) at element
 *              t * stride: a packed projection's output is read in place.
 * q_offsets, k_offsets : device int32, sequences + 1 entries that do not
 *              decrease, from 0 to at most the tokens.  Both NULL for one
 *              sequence of all tokens.  Rows of out and lse behind the last
 *              sequence are left as they were.
 * lse        : device float32, q_heads x q_tokens.
 * workspace  : as queried; 0 unless few tiles of queries meet many keys.
 * Scores, their maximum and sum are float32; for DMUON_BF16 the probabilities
 * are rounded to bf16 in front of their product with v.  Numbers that no query
 * of a sequence may see are not kept from it: an infinity or NaN in a key or
 * value can reach any query of its sequence, but no other sequence.
 */
int dmuon_attention_workspace_bytes(const dmuon_attention_shape* shape, size_t* bytes_out);
int dmuon_attention_forward(const dmuon_attention_shape* shape, const void* q, int64_t q_stride, const void* k,
                            int64_t k_stride, const void* v, int64_t v_stride, const int32_t* q_offsets,
                            const int32_t* k_offsets, void* out, int64_t out_stride, float* lse, void* workspace,
                            size_t workspace_bytes, void* hip_stream);

/*
 * Gradients of dmuon_attention_forward: dq, dk, dv from dout, the forward's
 * inputs and its out and lse.  The probabilities are formed again from lse; a
 * key head's gradients are summed over the query heads that share it, in fp32,
 * in a fixed order.  Rows behind the last sequence are left as they were.  An
 * infinity or NaN in any operand can reach every gradient of its sequence, and
 * none of another's.
 */
int dmuon_attention_backward_workspace_bytes(const dmuon_attention_shape* shape, size_t* bytes_out);
int dmuon_attention_backward(const dmuon_attention_shape* shape, const void* dout, int64_t dout_stride, const void* q,
                             int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             const void* out, int64_t out_stride, const float* lse, const int32_t* q_offsets,
                             const int32_t* k_offsets, void* dq, int64_t dq_stride, void* dk, int64_t dk_stride,
                             void* dv, int64_t dv_stride, void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * Shape and types of dmuon_gated_ffn_forward and _backward.
 */
#define DMUON_ACT_SILU 0   /* g / (1 + exp(-g)) */
#define DMUON_ACT_GELU 1   /* g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2 */
typedef struct {
    int64_t tokens;       /* 0 .. DMUON_MAX_TOKENS */
    int64_t dim;          /* 1 .. DMUON_MAX_DIM */
    int64_t hidden;       /* 1 .. DMUON_MAX_DIM */
    int activation;       /* DMUON_ACT_SILU or DMUON_ACT_GELU */
    int dtype;            /* inputs, weights, output and their gradients */
} dmuon_gated_ffn_shape;
/* A call takes less than 2^32 threads: 512 to 256 tokens x 128 of the hidden width
 * (backward, also x 256 of dim) for DMUON_BF16, 256 to 64 x 32 (x 64) for DMUON_F32. */

/*
 * The gated half of a feed-forward block: both projections, the activation and
 * the product in one pass,
 *
 *   h = act(x Wg^T) * (x Wu^T).
 *
 * x      : device, tokens x dim, row r at element r * x_stride.
 * w_gate, w_up : device, hidden x dim, contiguous.
 * h      : device, tokens x hidden, row r at element r * h_stride.
 * Sums are float32, and so is everything up to h.  workspace: for DMUON_BF16
 * it takes padded copies of the operands unless dim is a multiple of 64 and they
 * are aligned: x, w_gate and w_up at multiples of 16 bytes, rows of x a
 * multiple of 16 bytes apart and at most 8 MiB.  The query is told whether they
 * are; a call needs no more than that.
 */
int dmuon_gated_ffn_workspace_bytes(const dmuon_gated_ffn_shape* shape, int is_aligned, size_t* bytes_out);
int dmuon_gated_ffn_forward(const dmuon_gated_ffn_shape* shape, const void* x, int64_t x_stride, const void* w_gate,
                            const void* w_up, void* h, int64_t h_stride, void* workspace, size_t workspace_bytes,
                            void* hip_stream);

/*
 * Gradients of dmuon_gated_ffn_forward from dh and its inputs: dx, and the
 * weights' gradients as the Muon step takes them.  Both projections are formed
 * again; their gradients are rounded to dtype once, as operands of the products
 * that give the results, whose sums are float32 in a fixed order.
 *
 * dw_gate, dw_up : device, hidden x dim, contiguous.
 */
int dmuon_gated_ffn_backward_workspace_bytes(const dmuon_gated_ffn_shape* shape, int is_aligned, size_t* bytes_out);
int dmuon_gated_ffn_backward(const dmuon_gated_ffn_shape* shape, const void* dh, int64_t dh_stride, const void* x,
                             int64_t x_stride, const void* w_gate, const void* w_up, void* dx, int64_t dx_stride,
                             void* dw_gate, void* dw_up, void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * The plan of a call as text: routes (numel < DMUON_MIN_NS_NUMEL goes
 * elementwise when muon_step is nonzero), shape groups with their transposed
 * count, tiles and K slices, launches per Newton-Schulz step, algorithmic
 * flops and the workspace size -- the analogue of the training guide's INFO
 * summary of how parameters were assigned ("日志与调试", "验证参数分配").
 * Writes at most buf_len bytes including the terminating NUL (buf may be NULL
 * when buf_len is 0) and sets *needed (if not NULL) to the full length + 1.
 * Needs no GPU.  With the environment variable DMUON_LOG set (to anything but
 * "" or "0"), every call prints this text to stderr when its plan differs from
 * the last one printed.
 */
int dmuon_plan_summary(int count, const int64_t* rows, const int64_t* cols, int dtype,
                       const dmuon_ns_config* ns_config, int ns_steps, int muon_step, char* buf, size_t buf_len,
                       size_t* needed);

/* Static text for a status code.  The codes translate the pages' error
 * conventions to return values: the blog's newton_schulz asserts a 2-D input
 * ("代码实现", and "常见错误" 2: a bias vector must not reach NS) and accepts
 * float32 or bfloat16 only; the training guide's optimizer rejects bad
 * parameter lists when it is built ("第 4 步：创建优化器"). */
const char* dmuon_status_string(int status);

/* Details of the last error returned on the calling thread ("" if none). */
const char* dmuon_last_error(void);

/* Build and kernel description, the analogue of the pages' get_ns_backend()
 * string (training guide, "检查 NS 后端"). */
const char* dmuon_backend_info(void);

/*
 * Kernel-level timing.  While enabled, every kernel the library enqueues is
 * bracketed by a pair of HIP events on its stream.  dmuon_profile_read waits
 * for those events, returns per-kernel totals and clears the record.  Attention
 * counts the visible pairs of queries and keys of sequences that share the tokens
 * equally: the offsets are not read on the host.
 */
typedef struct {
    char name[40];      /* kernel family, e.g. "ns_gemm" */
    int64_t launches;   /* launches recorded */
    double total_ms;    /* sum of event-measured launch durations */
    double flops;       /* algorithmic flops summed over those launches */
    double bytes;       /* algorithmic HBM bytes summed over those launches */
} dmuon_kernel_stat;

int dmuon_profile_enable(int on);
/* Fills up to `max_stats` entries and sets *n_stats; returns a status. */
int dmuon_profile_read(dmuon_kernel_stat* stats, int max_stats, int* n_stats);

#ifdef __cplusplus
}
#endif

#endif /* DMUON_H */
