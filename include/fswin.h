/*
 * fswin — fused Swin windowed self-attention with window-local learnable 2D RoPE
 * on B200 (sm_100a): forward and backward behind a plain C ABI.
 *
 * The operation is the one the FlashSwin paper introduces ("FLASHSWIN: Unlocking
 * Large Windows and Dense Tokens in Swin Vision Transformers with Memory Efficient
 * Attention"; arxivdaily.com/papers/2610.04664, English abstract; and
 * thelatestinai.com/papers/2610.04664, Figure 1B and Figure S4): exact softmax
 * attention inside every M x M window of a cyclically shifted token grid, computed
 * without materialising the M^2 x M^2 score matrix, with queries and keys rotated
 * by a window-local 2D RoPE whose inverse frequencies theta are learnable.
 *
 * Conventions (readings of the paper where it is silent):
 *  - tensors q, k, v, o, dout, dq, dk, dv are bf16, contiguous [B, H, W, heads, d]
 *    (d = 32 or 64), 16-byte aligned, in DEVICE memory;
 *  - theta and dtheta are fp32 [heads, 2, d/4]; axis 0 (x) rotates channel pairs
 *    (2k, 2k+1) of the first d/2 channels by j * theta[h][0][k], axis 1 (y) the pairs
 *    of the last d/2 channels by i * theta[h][1][k], where (i, j) is the token's
 *    row and column inside its window (0 .. M-1, in the rolled frame);
 *  - H or W that is not a multiple of M is padded at the bottom and right to
 *    Hp = ceil(H/M)*M, Wp = ceil(W/M)*M with zero tokens, as a Swin layer pads its
 *    input before the shift; everything below then refers to the padded grid
 *    (Hp = H, Wp = W for multiples), padded tokens take part in the softmax, and
 *    only the H x W real tokens are read or written;
 *  - the shift takes rolled token (r, c) from original position ((r+s) mod Hp,
 *    (c+s) mod Wp); outputs are written back at original positions;
 *  - with s > 0 a query attends a key of its window only when both carry the same
 *    Swin shift-region label, built from the row/column slices [0, Hp-M),
 *    [Hp-M, Hp-s), [Hp-s, Hp); masked scores are -infinity;
 *  - softmax scale 1/sqrt(d); lse is the natural-log log-sum-exp per query, fp32
 *    [B, H, W, heads];
 *  - gradients are those of sum(o * dout).
 *
 * Ownership and ordering: the caller owns every buffer.  The library never
 * allocates device memory and never synchronises; all work is enqueued on the
 * given stream (a cudaStream_t; NULL is the legacy default stream).
 *
 * Per-device state (the device status word's address, the kernels' shared-memory
 * opt-in) is set up on the first call on each device and kept for the life of the
 * process, so the library must not be used on a device after cudaDeviceReset.
 *
 * Errors: invalid arguments return a status and launch nothing.  A kernel whose
 * internal wait runs past its time limit stops and records FS_ERR_TIMEOUT in a
 * device status word that fs_device_status() reads (after the stream is
 * synchronised by the caller).
 */
#ifndef FSWIN_H
#define FSWIN_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FS_API __attribute__((visibility("default")))
#else
#define FS_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FS_OK = 0,
    FS_ERR_NULL = 1,      /* a required pointer is NULL */
    FS_ERR_SHAPE = 2,     /* unsupported or inconsistent shape (see fs_winattn_shape) */
    FS_ERR_ALIGN = 3,     /* a pointer is not 16-byte aligned */
    FS_ERR_WORKSPACE = 4, /* workspace missing, misaligned or too small */
    FS_ERR_CUDA = 5,      /* a CUDA runtime/driver call failed */
    FS_ERR_TIMEOUT = 6,   /* a device-side wait ran out of time */
    FS_ERR_ARCH = 7       /* the current device is not sm_100 */
} fs_status;

/*
 * Problem shape.  Supported: d == 32 or d == 64; M in {4, 8, 16, 32, 64}; H >= M and W >= M
 * (not necessarily multiples of M: the grid is then padded, see above; a grid
 * smaller than the window is the caller's to clamp, as Swin clamps the window);
 * 0 <= s < M with s a multiple of 4; heads >= 1; B >= 0 (B == 0 is a valid empty
 * problem).  Anything else returns FS_ERR_SHAPE.
 * Heads of d = 64 (16 RoPE pairs per axis) run their own kernels, plain
 * one-tile pipelines; their backward's workspace holds an fp32 dQ accumulator
 * (256 bytes per token-head) besides the d theta partials.
 */
typedef struct {
    int B, H, W, heads, d, M, s;
} fs_winattn_shape;

typedef struct CUstream_st* fs_stream_t; /* same type as cudaStream_t */

/* Returns FS_OK when the shape is supported, without touching the device. */
FS_API fs_status fs_winattn_check_shape(const fs_winattn_shape* shape);

/*
 * Forward.  In: q, k, v (bf16 [B,H,W,heads,d]), theta (fp32 [heads,2,d/4]).
 * Out: o (bf16 [B,H,W,heads,d]) and lse (fp32 [B,H,W,heads], natural log);
 * both overwritten.  lse may be NULL: an inference forward that writes o only
 * (the workload of FlashSwin's inference-throughput figure, thelatestinai.com
 * Fig. S1); the backward needs lse, so a training forward passes it.
 * Exact softmax attention per window, with no score matrix in device memory
 * (the FlashSwin abstract).
 */
FS_API fs_status fs_winattn_fwd(const fs_winattn_shape* shape, const void* q, const void* k, const void* v,
                         const float* theta, void* o, float* lse, fs_stream_t stream);

/*
 * Forward of the whole window-attention block of a Swin layer, for inference
 * (the attention module of a FlashSwin block, thelatestinai.com 2610.04664,
 * Figure 1B, with its two linear maps):
 *   qkv = x W_qkv^T + b_qkv, split in (3, heads, d) along the channels;
 *   o = fs_winattn_fwd's attention of (q, k, v) with theta, M, s;
 *   y = o W_o^T + b_o, o taken as [B,H,W,C].
 * In: x bf16 [B,H,W,C] with C = heads * d; w_qkv bf16 [3C, C] (output channels
 * q of every head, then k, then v); b_qkv fp32 [3C]; w_o bf16 [C, C]; b_o
 * fp32 [C]; theta fp32 [heads,2,d/4].  Out: y bf16 [B,H,W,C], overwritten.  d == 32 only.
 * q, k, v and o never reach device memory.  Supported: the shapes of
 * fs_winattn_check_shape with M*M < 128 (windows inside one 128-token tile)
 * and heads <= 3; anything else returns FS_ERR_SHAPE.  On a padded grid (H or W
 * not a multiple of M) the padded tokens of x are zero, as the Swin layer pads x
 * before its qkv map, so their q, k, v equal the bias.  x, w_qkv, w_o, y
 * 16-byte aligned (FS_ERR_ALIGN); no pointer may be NULL (FS_ERR_NULL).
 */
FS_API fs_status fs_winattn_block_fwd(const fs_winattn_shape* shape, const void* x, const void* w_qkv,
                               const float* b_qkv, const void* w_o, const float* b_o, const float* theta,
                               void* y, fs_stream_t stream);

/*
 * Workspace the backward needs, in bytes.  It depends on the token count of the
 * padded grid, B*Hp*Wp*heads, only: for H and W multiples of M it does not depend
 * on the window size (memory flat in M, FlashSwin Table S1).
 */
FS_API size_t fs_winattn_bwd_workspace_bytes(const fs_winattn_shape* shape);

/*
 * Backward (recompute-based: the probabilities are rebuilt from lse, never stored).
 * In: q, k, v, o (the forward output), dout, lse, theta.  Out: dq, dk, dv (bf16
 * [B,H,W,heads,d]) and dtheta (fp32 [heads,2,d/4]); all overwritten.  workspace:
 * device scratch of at least fs_winattn_bwd_workspace_bytes(shape) bytes, 256-byte
 * aligned; its contents on entry are ignored.
 */
FS_API fs_status fs_winattn_bwd(const fs_winattn_shape* shape, const void* q, const void* k, const void* v,
                         const void* o, const void* dout, const float* lse, const float* theta, void* dq,
                         void* dk, void* dv, float* dtheta, void* workspace, size_t workspace_bytes,
                         fs_stream_t stream);

/*
 * Windowed attention with a low-rank additive bias (the FlashBias-T variant of
 * the same pages: thelatestinai.com 2610.04664, Table 2 and Table S1 captions,
 * a trainable rank-16 factorization of an additive attention bias whose
 * parameters grow with M).  Reading where the pages are silent: per head h the
 * bias of a window's (query position t, key position u) pair is
 * U[h][t] . W[h][u], t = i*M + j the window-local position in the rolled frame,
 * the same for every window of the batch, added to the scaled score before the
 * shift mask:  S_tu = q'_t . k'_u / sqrt(d) + U[h][t] . W[h][u].
 *
 * Shapes: those of fs_winattn_check_shape with d == 32 (else FS_ERR_SHAPE);
 * rank == 16 (else FS_ERR_SHAPE).  u, w: fp32 [heads][M*M][16], 16-byte aligned.
 * theta may be NULL: no rotation (q' = q, k' = k), and the backward then takes
 * dtheta == NULL too; with theta the RoPE of fs_winattn_fwd applies.  Other
 * arguments, layouts, ownership and errors as fs_winattn_fwd / fs_winattn_bwd.
 *
 * Forward: o and lse (lse may be NULL: inference), overwritten.
 * Backward: dq, dk, dv, dtheta (when theta is given), du and dw (fp32
 * [heads][M*M][16], the gradients summed over every window of the batch, in a
 * fixed order), all overwritten.  dq, du and the query side of dtheta are
 * accumulated in fp32 with vector reductions whose order varies from run to
 * run; dk, dv and dw do not vary.  workspace: at least fs_winattn_lrbias_bwd_workspace_bytes(shape)
 * bytes, 256-byte aligned (about 276 bytes per token-head on the padded grid,
 * plus a few KB per head).  The kernels are plain one-tile pipelines.
 */
FS_API fs_status fs_winattn_lrbias_fwd(const fs_winattn_shape* shape, const void* q, const void* k, const void* v,
                                       const float* theta, const float* u, const float* w, int rank, void* o,
                                       float* lse, fs_stream_t stream);
FS_API size_t fs_winattn_lrbias_bwd_workspace_bytes(const fs_winattn_shape* shape);
FS_API fs_status fs_winattn_lrbias_bwd(const fs_winattn_shape* shape, const void* q, const void* k, const void* v,
                                       const void* o, const void* dout, const float* lse, const float* theta,
                                       const float* u, const float* w, int rank, void* dq, void* dk, void* dv,
                                       float* dtheta, float* du, float* dw, void* workspace, size_t workspace_bytes,
                                       fs_stream_t stream);

/*
 * Windowed attention with a learned relative position bias by buckets (the
 * additive bias of a Swin layer, which the FlashSwin pages replace by RoPE): per
 * head h and pair of window positions
 *   S_tu = q_t . k_u / sqrt(d) + table[h][b],
 *   b = buckets[(i_t - i_u + M - 1) (2M - 1) + (j_t - j_u + M - 1)],
 * (i, j) the row and column inside the window (rolled frame), the same for every
 * window, added before the shift mask.  No rotation.
 *
 * Shapes: those of fs_winattn_check_shape with d == 32 (else FS_ERR_SHAPE).
 * table: bf16 [heads][n_buckets], 2-byte aligned, 1 <= n_buckets <= 2^20.
 * buckets: int32 [(2M-1)^2] in DEVICE memory, or NULL: the displacement index is
 * the bucket and n_buckets must be (2M-1)^2 (else FS_ERR_SHAPE).  A bucket outside
 * [0, n_buckets) adds no bias and takes no gradient.  An entry of -inf keeps its
 * pairs apart; a query left without a key has o = 0, lse = -inf and no gradient.
 * Finite entries beyond 8.5e37 in magnitude act as that value.  A query whose every
 * key has a large entry (the type's lowest value as a mask, say) has the softmax of its
 * biased scores as fp32 holds them, the uniform one where a step of fp32 exceeds the
 * scores (from about 1e9 on), forward and backward alike.  (The backward forms such a
 * row's maximum and sum again, key by key, which is slow.)  Where, at M >= 8, the scores
 * q . k alone make a log-sum-exp beyond 2800 in magnitude, the gradient carries fp32's step there
 * (2^-11 of a probability, growing with it), and has no part of the query beyond 7e29.
 *
 * Forward: o and lse (lse may be NULL: inference), overwritten.
 * Backward: dq, dk, dv and dtable (bf16 [heads][n_buckets]: the gradient summed in
 * fp32 over every window of the batch and every pair of the bucket, in a fixed
 * order; at M >= 16 each pair's term is rounded to bf16 first, as dq and dk take it),
 * all overwritten.  At M >= 16 dq is accumulated in fp32 with bulk
 * reductions whose order varies from run to run; everything else, and at M <= 8
 * every output, is the same from run to run.  workspace: at least
 * fs_winattn_relbias_bwd_workspace_bytes(shape) bytes, 256-byte aligned (M >= 16:
 * 145 bytes per token-head on the padded grid; and 4 bytes a displacement for
 * every head and CTA).  Other arguments, layouts, ownership and errors as
 * fs_winattn_fwd / fs_winattn_bwd.  At M = 8 and M = 4, where windows share a
 * tile, values that are not finite stay inside their own window.
 */
FS_API fs_status fs_winattn_relbias_fwd(const fs_winattn_shape* shape, const void* q, const void* k, const void* v,
                                        const void* table, const int* buckets, int n_buckets, void* o, float* lse,
                                        fs_stream_t stream);
FS_API size_t fs_winattn_relbias_bwd_workspace_bytes(const fs_winattn_shape* shape);
FS_API fs_status fs_winattn_relbias_bwd(const fs_winattn_shape* shape, const void* q, const void* k, const void* v,
                                        const void* o, const void* dout, const float* lse, const void* table,
                                        const int* buckets, int n_buckets, void* dq, void* dk, void* dv, void* dtable,
                                        void* workspace, size_t workspace_bytes, fs_stream_t stream);

/*
 * The residual step between the blocks of a Swin layer, row by row over the
 * channels (a row is a token):
 *   y = post(f);  r = x + gate[b] * (scale o drop(y));  n = pre(r)
 * post and pre: FS_NORM_NONE, FS_NORM_LAYER ((v - mean) / sqrt(var + eps), times
 * weight, plus bias) or FS_NORM_RMS (v / sqrt(mean(v^2) + eps), times weight, plus
 * bias).  A pre-norm layer has pre, a post-norm layer (Swin V2) post.
 *  - gate: one value a sample (stochastic depth, or a learned gate).  A sample whose
 *    gate is zero takes nothing from f, whatever f holds, and gives it no gradient;
 *  - scale: one value a channel (layer scale);
 *  - drop: element e of the whole tensor is kept, times 1 / (1 - drop_p), when word
 *    e mod 4 of Philox4x32-10 with counter (e / 4, rng[1]) and key rng[0] is at least
 *    floor(drop_p 2^32), else replaced by zero.  The mask is never stored: the
 *    backward draws it again from the same rng.
 * Types: x, r, dr, dx and every parameter and parameter gradient are of the stream
 * type (bf16, or fp32 with stream_f32); f, n, dn, df are bf16.  Sums, means and
 * deviations are fp32; n is the norm of r before r is rounded, and the backward
 * forms it again from the stored r.
 * Layout: x, f, r, n and their gradients [samples, tokens, channels], contiguous,
 * any alignment of their element (16-byte aligned tensors take 16-byte accesses, but
 * for the ends of rows whose channels are no multiple of 8); gate [samples]; parameters [channels]; rng: int64
 * [2] in DEVICE memory, read when the kernel runs.  r may be x, n may be f, dx may
 * be dr, df may be dn (the same buffer, not a shifted one).
 * Shapes: 1 <= channels <= 8192, samples * tokens < 2^31 (both >= 0), eps >= 0 and
 * finite, 0 <= drop_p < 1; else FS_ERR_SHAPE, as for the weight or bias of a norm
 * that is FS_NORM_NONE.  gate, scale, weights and biases may be NULL; rng may be
 * NULL when drop_p == 0; n is required with pre and not written without.
 *
 * Backward: gradients of sum(r * dr) + sum(n * dn); dr or dn may be NULL (zero).  f is
 * required; dgate, dscale and the parameter gradients may each be NULL (not
 * wanted), and are ignored where their parameter is NULL.  Results do not vary from
 * run to run.  workspace: at least fs_resnorm_bwd_workspace_bytes(shape) bytes,
 * 256-byte aligned.
 */
typedef enum { FS_NORM_NONE = 0, FS_NORM_LAYER = 1, FS_NORM_RMS = 2 } fs_norm;
typedef struct {
    long long samples, tokens;
    int channels;
    int stream_f32; /* 0: bf16 stream, 1: fp32 */
    int pre, post;  /* fs_norm */
    float eps;
    double drop_p;
} fs_resnorm_shape;
FS_API fs_status fs_resnorm_fwd(const fs_resnorm_shape* shape, const void* x, const void* f, const void* gate,
                                const void* scale, const void* post_w, const void* post_b, const void* pre_w,
                                const void* pre_b, const long long* rng, void* r, void* n, fs_stream_t stream);
FS_API size_t fs_resnorm_bwd_workspace_bytes(const fs_resnorm_shape* shape);
FS_API fs_status fs_resnorm_bwd(const fs_resnorm_shape* shape, const void* dr, const void* dn, const void* r,
                                const void* f, const void* gate, const void* scale, const void* post_w,
                                const void* post_b, const void* pre_w, const void* pre_b, const long long* rng,
                                void* dx, void* df, void* dgate, void* dscale, void* dpost_w, void* dpost_b,
                                void* dpre_w, void* dpre_b, void* workspace, size_t workspace_bytes,
                                fs_stream_t stream);

/*
 * Gated feed-forward block of a layer:
 *   h = act(x W_gate^T + b_gate) o (x W_up^T + b_up);  y = h W_down^T + b_down
 * act: FS_ACT_SILU (g sigmoid(g)) or FS_ACT_GELU (g Phi(g), the exact one).  All bf16:
 * x, y [tokens, channels]; w_gate, w_up [hidden, channels]; w_down [channels, hidden];
 * b_gate, b_up [hidden] and b_down [channels], each of which may be NULL.  Products and
 * the activation are fp32; h is rounded to bf16 between the two products.
 * Shapes: 0 <= tokens < 2^31 - 256, channels 8 .. 16384 and hidden 8 .. 65536, both
 * multiples of 8, and fewer than 2^31 tiles of 128 tokens by 64 channels of the wider
 * of the two (else FS_ERR_SHAPE); every pointer 16-byte aligned (FS_ERR_ALIGN).
 *
 * Backward: gradients of sum(y * dy), from x and the weights (h is formed again).  dx and
 * the weight gradients are bf16 like what they belong to; a NULL bias gradient is not
 * computed.  Weight and bias gradients are summed over the tokens in fp32 in a fixed
 * order: results do not vary from run to run.
 * workspace: at least fs_gated_mlp_{fwd,bwd}_workspace_bytes(shape) bytes, 256-byte
 * aligned (forward 2 bytes a token and hidden channel, or 256 in all where the weights
 * fit into an SM's shared memory; backward 6 bytes a token and hidden channel, and 12 a
 * weight of one matrix for each part, of 1 to 16, in which the tokens are summed: one up
 * to 384 tokens, and about one where the weights alone give every SM work).
 */
typedef enum { FS_ACT_SILU = 0, FS_ACT_GELU = 1 } fs_act;
typedef struct {
    long long tokens;
    int channels, hidden, act; /* act: fs_act */
} fs_mlp_shape;
FS_API size_t fs_gated_mlp_fwd_workspace_bytes(const fs_mlp_shape* shape);
FS_API fs_status fs_gated_mlp_fwd(const fs_mlp_shape* shape, const void* x, const void* w_gate, const void* w_up,
                                  const void* w_down, const void* b_gate, const void* b_up, const void* b_down, void* y,
                                  void* workspace, size_t workspace_bytes, fs_stream_t stream);
FS_API size_t fs_gated_mlp_bwd_workspace_bytes(const fs_mlp_shape* shape);
FS_API fs_status fs_gated_mlp_bwd(const fs_mlp_shape* shape, const void* dy, const void* x, const void* w_gate,
                                  const void* w_up, const void* w_down, const void* b_gate, const void* b_up, void* dx,
                                  void* dw_gate, void* dw_up, void* dw_down, void* db_gate, void* db_up, void* db_down,
                                  void* workspace, size_t workspace_bytes, fs_stream_t stream);

/*
 * Training pair.  fs_winattn_fwd_train is fs_winattn_fwd (lse required) that
 * also leaves, in `workspace` (the backward's: at least
 * fs_winattn_bwd_workspace_bytes(shape) bytes, 256-byte aligned), the rotated
 * q', k' tiles the backward needs; fs_winattn_bwd_train is fs_winattn_bwd that
 * takes them from there instead of rotating q and k again.  The forward of
 * windows of >= 128 tokens (d == 32) then reads its Q', K' tiles from those
 * images, rotating each row once instead of once per query tile of the window.
 * Same results as fs_winattn_fwd / fs_winattn_bwd.  Contract: the backward gets
 * the workspace of the training forward of the same shape, q, k and theta,
 * unchanged in between (otherwise its gradients are wrong; nothing checks it).
 * For windows of fewer than 128 tokens and for d == 64 the pair behaves as
 * fs_winattn_fwd / fs_winattn_bwd (the forward writes nothing to the workspace).
 * Errors as those of fs_winattn_fwd and fs_winattn_bwd; the forward also
 * returns FS_ERR_WORKSPACE for a missing, misaligned or short workspace.
 */
FS_API fs_status fs_winattn_fwd_train(const fs_winattn_shape* shape, const void* q, const void* k, const void* v,
                                      const float* theta, void* o, float* lse, void* workspace,
                                      size_t workspace_bytes, fs_stream_t stream);
FS_API fs_status fs_winattn_bwd_train(const fs_winattn_shape* shape, const void* q, const void* k, const void* v,
                                      const void* o, const void* dout, const float* lse, const float* theta,
                                      void* dq, void* dk, void* dv, float* dtheta, void* workspace,
                                      size_t workspace_bytes, fs_stream_t stream);

/* Human-readable name of a status. */
FS_API const char* fs_status_string(fs_status status);

/*
 * Reads and clears the device status word of the current device.  *code receives 0
 * when no kernel reported a failure, else (status << 24) | where.  Synchronous.
 */
FS_API fs_status fs_device_status(unsigned int* code);

/* Time limit of every device-side wait, in nanoseconds (default 10 s). */
FS_API fs_status fs_set_wait_limit_ns(uint64_t limit_ns);

/*
 * Self-test of the bounded-wait path: launches one CTA that waits on a barrier no
 * thread ever arrives on, with the given limit.  Afterwards (stream synchronised)
 * fs_device_status() reports FS_ERR_TIMEOUT.  The GPU context stays usable.
 */
FS_API fs_status fs_selftest_bounded_wait(uint64_t limit_ns, fs_stream_t stream);

/*
 * Backward that allocates nothing and takes no workspace (the paper has no
 * counterpart; this is a convenience of this library).  For callers that cannot
 * allocate device memory when they call the backward, for example code that
 * runs inside a memory pool that is already fully handed out, or a runtime that
 * forbids cudaMalloc after start-up.  The scratch is one array inside the
 * library, fs_winattn_bwd_noalloc_max_bytes() bytes (64 MiB) on every GPU that
 * loads the library, held until the process exits.  Problems whose
 * fs_winattn_bwd_workspace_bytes() exceeds that size return FS_ERR_WORKSPACE and
 * launch nothing.  Arguments and results are those of fs_winattn_bwd.
 *
 * The first call on a device looks up the array's device address (once per
 * device).  All calls on a device share the array: calls whose kernels may overlap on the GPU (other
 * streams or host threads without ordering between them) race on it.
 * The address is kept for the life of the process: do not use this entry point
 * (or any other of this library, whose device status word is looked up the same
 * way) on a device after cudaDeviceReset.
 */
FS_API fs_status fs_winattn_bwd_noalloc(const fs_winattn_shape* shape, const void* q, const void* k, const void* v,
                                        const void* o, const void* dout, const float* lse, const float* theta,
                                        void* dq, void* dk, void* dv, float* dtheta, fs_stream_t stream);

/* Size of the scratch array fs_winattn_bwd_noalloc uses, in bytes. */
FS_API size_t fs_winattn_bwd_noalloc_max_bytes(void);

/*
 * Profiling hook.  events: `n` caller-created cudaEvent_t handles (as void*), or
 * n == 0 to switch the hook off.  While set, fs_winattn_fwd records events[0]
 * before and events[1] after its kernel (n >= 2), and fs_winattn_bwd records
 * events[0] before its first kernel and events[1 + i] after its kernel i
 * (prep, main, post, dtheta reduction; n >= 5), on the call's stream; the
 * low-rank-bias entry points record the same marks (the backward's last one
 * after the dtheta, du and dw sums).  The
 * handles are kept by value; the hook is process-wide and not thread-safe.
 */
FS_API fs_status fs_set_phase_events(void* const* events, int n);

#ifdef __cplusplus
}
#endif

#endif /* FSWIN_H */
