/*
 * mamba3_ssm.h -- C ABI of the MI355X (gfx950) Mamba-3 SSM layer core.
 *
 * Five operations of the layer core, three of the residual block around it
 * and three of an attention layer beside it, all asynchronous on a caller-given
 * HIP stream:
 *
 *   mamba3_ssm_chunked_fwd   whole-sequence forward (prefill / training
 *                            forward) by the chunked parallel form;
 *   mamba3_ssm_chunked_bwd   its backward (training);
 *   mamba3_ssm_decode_step   one-token state update (generation);
 *   mamba3_rope_bc           the cumulative-angle rotation of B and C;
 *   mamba3_bc_prologue       the projection to B and C with their
 *                            normalisation, bias and rotation fused;
 *   mamba3_layer_norm_*      layer norm over the model width;
 *   mamba3_linear_*          a matrix product with bias, activation and
 *                            residual;
 *   mamba3_gated_ffn_*       both projections of a gated feed-forward, its
 *                            activation and product (each of the three with
 *                            its backward; their own conventions stand with
 *                            them, below the core's);
 *   mamba3_qk_norm_rope_*    norms of queries and keys for each head and their
 *                            rotation by position;
 *   mamba3_window_attn_*     causal attention over a sliding window with first
 *                            tokens that stay visible, its backward, and the
 *                            same for new tokens over a cache (at the end).
 *
 * What the core computes (pages cited by title and section):
 *
 *  - linkstar.cloud/article/869, "第一刀：指数梯形离散化": with
 *    alpha_t = exp(dt_t A_t), beta_t = (1 - lam_t) dt_t alpha_t and
 *    gamma_t = lam_t dt_t,
 *        h_t = alpha_t h_{t-1} + beta_t B_{t-1} x_{t-1}^T + gamma_t B_t x_t^T;
 *    the same section gives the parallel form (a 1-semiseparable decay matrix
 *    times a 2-band matrix) that the chunked forward evaluates per chunk.
 *  - same page, "第二刀：复值状态空间": the complex state is a real state whose
 *    transition holds 2x2 rotations R(w) = [[cos w, -sin w], [sin w, cos w]]
 *    with w = dt_t theta_t[k] on pair (2k, 2k+1); equivalently the rotations
 *    move onto B and C as cumulative angles phi_t = sum_{s<=t} dt_s theta_s
 *    (B~ = R(-phi) B, C~ = R(-phi) C: a data-dependent RoPE).
 *  - same page, "第三刀：多输入多输出": B_t is N x R, x_t is P x R, the input
 *    term is the rank-R product B_t x_t^T, and y_t = C_t^T h_t is R x P.
 *  - yetianai.com/news/16273, "榨干硬件算力": chunks are computed in parallel
 *    internally and pass the state from chunk to chunk in order.
 *
 * Notation per (batch b, head h): L tokens, P head dim, N state size (even,
 * N/2 rotation pairs), R MIMO rank, Q chunk length in tokens.
 *
 * Layouts: row-major, contiguous, no strides.
 *   x, y            (B, L, H, R, P)   io dtype
 *   B, C            (B, L, H, R, N)   io dtype
 *   dt, A, lam      (B, L, H)         fp32 (dt > 0, already post-softplus)
 *   theta           (B, L, H, N/2)    fp32, one angle rate per pair
 *   h0, h_final     (B, H, N, P)      fp32, un-rotated ("true") frame
 *   prev_B          (B, H, R, N)      io dtype: raw B of the token before x[:,0]
 *   prev_x          (B, H, R, P)      io dtype: x of that token
 *   angle0/final    (B, H, N/2)       fp32
 *   decode: x, y (B, H, R, P); B, C, prev_B (B, H, R, N); prev_x (B, H, R, P);
 *           dt, A, lam (B, H); theta (B, H, N/2); state (B, H, N, P) fp32.
 * Pair (2k, 2k+1) of B, C and of the state rows is (real, imaginary) of
 * complex component k.
 *
 * Ownership: the caller owns every buffer (device memory unless stated).  The
 * library allocates nothing and, apart from the fixed per-GPU array of
 * mamba3_ssm_chunked_fwd_noalloc, keeps no mutable global state: every other
 * call is reentrant and may run on concurrent streams when its buffers are
 * disjoint from the other calls' buffers.  Alignment: x, B, C, theta, y and the workspace of chunked_fwd,
 * B, C, B_rot and C_rot of rope_bc, and the state of decode_step must be
 * 16-byte aligned; every other pointer must be aligned to its element size.
 *
 * Errors: every entry point validates its arguments on the host and returns a
 * status before any HIP call; nothing is launched on error.  M3_ERR_HIP
 * reports a failed launch.  Device-side faults surface, as usual in HIP, at
 * the caller's next synchronisation.
 *
 * Supported sizes: N in {16,32,64,128}; P in {16,32,64,128}; R in {1,2,4};
 * Q in {16,32,64}; io dtype fp32 or bf16: every combination, for the chunked
 * forward and the backward alike; M3_ERR_UNSUPPORTED outside it.  Where a
 * chunk's tiles would not fit in the 160 KiB of LDS of one compute unit
 * (fp32 io with Q*R = 256, N = P = 128 with long chunks) the chunked forward
 * walks each chunk as 2, 4 or 8 shorter pieces: the chunked form is exact for
 * any split (linkstar.cloud/article/869, "第一刀"), so only the rounding order
 * changes.  batch, seqlen and nheads may be 0 (empty input: nothing is read;
 * h_final receives h0, or zeros).  Size limits (M3_ERR_UNSUPPORTED beyond
 * them): batch and nheads at most 65535 each; the chunked forward and the
 * backward run one block of up to 512 threads per (b, h, segment) and the
 * decode step one of 256 threads per (b, h), and a launch holds fewer than
 * 2^32 threads, so batch * nheads * segments is at most 8,388,607 (16,777,215
 * for decode_step); split larger batches over several calls.
 */
#ifndef MAMBA3_SSM_H
#define MAMBA3_SSM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MAMBA3_ABI_VERSION 1

typedef enum {
  M3_OK = 0,
  M3_ERR_NULL = 1,        /* a required pointer is NULL, or only one of prev_B/prev_x is given */
  M3_ERR_SHAPE = 2,       /* a negative size, or an odd dstate */
  M3_ERR_UNSUPPORTED = 3, /* size outside the supported set listed above */
  M3_ERR_ALIGN = 4,       /* a pointer breaks the alignment rule above */
  M3_ERR_WORKSPACE = 5,   /* workspace NULL or smaller than the queried size */
  M3_ERR_HIP = 6          /* a kernel launch failed */
} m3_status;

typedef enum { M3_F32 = 0, M3_BF16 = 1 } m3_dtype;

typedef struct {
  int64_t batch;    /* B */
  int64_t seqlen;   /* L (ignored by decode_step) */
  int64_t nheads;   /* H */
  int64_t headdim;  /* P */
  int64_t dstate;   /* N, even */
  int64_t rank;     /* R */
  int64_t chunk;    /* Q tokens per chunk (chunked_fwd only).  For bf16 io
                       with P = 64 and N = 64 (Q in {32, 64}) or N = 128
                       (R in {2, 4}) the library walks each chunk as 32- or
                       16-token sub-chunks (the chunked form is exact for
                       any split); segments and workspace follow Q.  At
                       N = 64 a chunk of 16 is walked (and segmented) as
                       chunks of 32.  Where Q's tiles do not fit the LDS the
                       walk (and with it segments and workspace) uses Q/2,
                       Q/4 or Q/8. */
  int32_t io_dtype; /* m3_dtype of x, B, C, y, prev_B, prev_x, B_rot, C_rot */
  int32_t flags;    /* chunked_fwd: bits 0..15 = number of sequence segments
                       walked in parallel per (b,h) (0 = chosen by the
                       library: more than one only for bf16 io when B*H <
                       256); M3_FLAG_CHUNK_WALK or M3_FLAG_TOKEN_PATH;
                       other bits must be 0.
                       Segments > 1 need bf16 io and B*H <= 65535.
                       chunked_bwd: bits 0..15 = number of sequence
                       segments (0 = chosen by the library: more than one
                       only when B*H < 256); other bits must be 0.  Other
                       entry points: must be 0. */
} m3_dims;

/* chunked_fwd: short calls (e.g. verifying k draft tokens of a decoder, with
 * the decode state as h0 and h_final) read the state once and write it once.
 * For bf16 io with P = 64 and N = 64 or 128, a call of at most
 * M3_TOKEN_PATH_MAX_L tokens runs as one chunk of the chunked form on bf16
 * MFMAs (two 8-token pieces for R = 4 past 8 tokens).  Other sizes run token
 * by token with the state held on chip (the one-token update of decode_step
 * applied to each token) for seqlen <= M3_TOKEN_PATH_SUBWALK_L when the
 * sub-chunk walker covers the sizes and seqlen <= M3_TOKEN_PATH_MAX_L
 * otherwise.  M3_FLAG_CHUNK_WALK forces the chunk walk; M3_FLAG_TOKEN_PATH
 * forces the token-by-token path (seqlen <= M3_TOKEN_PATH_MAX_L, else
 * M3_ERR_UNSUPPORTED); not both.  Every path computes the same function (the
 * chunked ones to the rounding of their bf16 products). */
#define M3_FLAG_CHUNK_WALK 0x10000
#define M3_FLAG_TOKEN_PATH 0x20000
#define M3_TOKEN_PATH_MAX_L 16
#define M3_TOKEN_PATH_SUBWALK_L 8

/* Whole-sequence forward.
 *   y_t = C_t^T h_t for every token, and h_final = h_L.
 * h0: nullable, the state before x[:,0] (true frame); NULL means zero.
 * prev_B, prev_x: nullable pair, the raw B and x of the token before x[:,0]
 *   (its trapezoid term enters the first update); NULL means none.
 * y: written (must not alias an input).  h_final: nullable; may alias h0.
 * workspace: device scratch of at least
 *   mamba3_ssm_chunked_fwd_workspace_size(d) bytes (may be NULL when that is 0);
 *   its contents on entry do not matter.  It is non-zero only when the
 *   sequence is walked as several segments (see flags): the segments are
 *   walked from a zero state in parallel, then a segment scan supplies the
 *   true incoming states and their contribution is added to y (linearity of
 *   the recurrence).
 * To continue a sequence, pass h_final as h0 and the last token's raw B and x
 * as prev_B / prev_x. */
m3_status mamba3_ssm_chunked_fwd(const m3_dims* d,
                                 const void* x, const void* B, const void* C,
                                 const float* dt, const float* A, const float* lam, const float* theta,
                                 const float* h0, const void* prev_B, const void* prev_x,
                                 void* y, float* h_final,
                                 void* workspace, size_t workspace_bytes, void* stream);
size_t mamba3_ssm_chunked_fwd_workspace_size(const m3_dims* d);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, serving loops that must not call hipMalloc, harnesses that forbid
 * it): mamba3_ssm_chunked_fwd with no workspace argument.  The workspace comes
 * from a fixed array of M3_NOALLOC_SCRATCH_BYTES that the library holds on
 * every GPU it runs on, until the process ends; this call allocates nothing.
 * Sizes whose workspace (mamba3_ssm_chunked_fwd_workspace_size) exceeds it
 * return M3_ERR_WORKSPACE before any HIP call (48 MiB covers, e.g., one
 * 65,536-token sequence of 32 heads at N = 128, P = 64, R = 4 walked as
 * segments).  Every call on one GPU shares that GPU's array: calls that
 * overlap in time on one GPU (concurrent streams, or several host threads)
 * race on it and must be serialised by the caller.  The array used is that of
 * the calling thread's current device (hipGetDevice), which must be the
 * device that stream belongs to.  The array's contents carry over between
 * calls; the forward needs none on entry.  Results are those of
 * mamba3_ssm_chunked_fwd with the same arguments. */
#define M3_NOALLOC_SCRATCH_BYTES (48u << 20)
m3_status mamba3_ssm_chunked_fwd_noalloc(const m3_dims* d,
                                         const void* x, const void* B, const void* C,
                                         const float* dt, const float* A, const float* lam, const float* theta,
                                         const float* h0, const void* prev_B, const void* prev_x,
                                         void* y, float* h_final, void* stream);

/* Backward of mamba3_ssm_chunked_fwd: the gradients of
 *     l = sum_t <dy_t, y_t> + <dh_final, h_final>
 * with respect to every input of the forward (the chain rule of the chunked
 * form, chunks walked in reverse order; same pages as the forward).
 *   dy: (B, L, H, R, P) io dtype.  dh_final: nullable (B, H, N, P) fp32; NULL
 *       means zero.
 *   dx (B, L, H, R, P), dB, dC (B, L, H, R, N): io dtype, written.
 *   ddt, dA, dlam (B, L, H), dtheta (B, L, H, N/2): fp32, written.
 *   dh0: nullable (B, H, N, P) fp32, written when given (also when h0 is NULL:
 *        the gradient with respect to a zero initial state).
 *   dprev_B (B, H, R, N), dprev_x (B, H, R, P): nullable pair, io dtype,
 *        written when prev_B/prev_x are given.
 * Supported: N and P in {16, 32, 64, 128}, R in {1, 2, 4}, io fp32 or bf16;
 * d->chunk must be a supported chunk length but the backward walks chunks of
 * its own: 16 tokens, 8 when N or P is 128 and R = 4, 16 / R when both are
 * 128 (the chunked form is exact for any split); nheads
 * at most 65536 (M3_ERR_UNSUPPORTED otherwise: offsets inside a chunk are
 * 32-bit).  Products: fp32 for fp32 io; bf16 MFMAs with fp32 accumulation
 * for bf16 io (operands rounded to bf16; the state product of the checkpoint
 * walk takes w B~ as bf16 hi + lo parts), with fp32 state checkpoints.
 * Segments (flags bits 0..15, for few long sequences): each sequence is cut
 * into runs of whole chunks that separate blocks walk at once.  The states at
 * segment starts come from walks from a zero state and the forward's segment
 * scan; the state adjoints at segment ends from walks of the adjoint from zero
 * and a reverse scan (the adjoint recurrence is linear too); the first token
 * of each segment takes the parts of its dt and lam gradients that the
 * previous segment computes.  The result is the same function; only rounding
 * differs.  The library picks ceil(512 / (B*H)) segments (at most a quarter
 * of the chunks) when B*H < 256 and one otherwise; a count above the number
 * of chunks is clamped to it.
 * workspace: at least
 * mamba3_ssm_chunked_bwd_workspace_size(d) bytes (the states at every chunk
 * start, and with segments four (B, H, S, N, P) fp32 arrays and small
 * per-segment records); its contents on entry do not matter.  Outputs must
 * not alias inputs.
 * Alignment: x, B, C, dy, dx, dB, dC, theta, dtheta and the workspace 16-byte;
 * the others their element size. */
m3_status mamba3_ssm_chunked_bwd(const m3_dims* d,
                                 const void* x, const void* B, const void* C,
                                 const float* dt, const float* A, const float* lam, const float* theta,
                                 const float* h0, const void* prev_B, const void* prev_x,
                                 const void* dy, const float* dh_final,
                                 void* dx, void* dB, void* dC,
                                 float* ddt, float* dA, float* dlam, float* dtheta,
                                 float* dh0, void* dprev_B, void* dprev_x,
                                 void* workspace, size_t workspace_bytes, void* stream);
size_t mamba3_ssm_chunked_bwd_workspace_size(const m3_dims* d);

/* One-token update, in place on the fp32 true-frame state:
 *   h <- alpha R(dt theta) [h + eps prev_B^T prev_x] + gamma B^T x,
 *   y  = C^T h (new state),  eps = (1 - lam) dt.
 * prev_B, prev_x: nullable pair (NULL: no previous token, e.g. the very first
 * token of a sequence).  seqlen and chunk of d are ignored.  y must not alias
 * any input. */
m3_status mamba3_ssm_decode_step(const m3_dims* d, float* state,
                                 const void* x, const void* B, const void* C,
                                 const float* dt, const float* A, const float* lam, const float* theta,
                                 const void* prev_B, const void* prev_x,
                                 void* y, void* stream);

/* Cumulative-angle rotation:
 *   phi_t = angle0 + sum_{s<=t} dt_s theta_s (per pair), B_rot = R(-phi_t) B_t,
 *   C_rot = R(-phi_t) C_t, angle_final = phi_L.
 * angle0, angle_final: nullable.  B_rot / C_rot must not alias B / C.
 * workspace: at least mamba3_rope_bc_workspace_size(d) bytes: the angle
 * totals of every 64-token chunk, which a first pass writes and the rotating
 * pass scans, so that every chunk of a long sequence is rotated in parallel.
 * The library allocates nothing, so the caller provides this array.  chunk
 * of d is ignored.  seqlen is limited to
 * 65535 * 64 tokens (M3_ERR_UNSUPPORTED). */
m3_status mamba3_rope_bc(const m3_dims* d, const void* B, const void* C,
                         const float* dt, const float* theta, const float* angle0,
                         void* B_rot, void* C_rot, float* angle_final,
                         void* workspace, size_t workspace_bytes, void* stream);
size_t mamba3_rope_bc_workspace_size(const m3_dims* d);

/* B/C prologue: the projection of the token activations to B and C with the
 * normalisation, bias and rotation applied on the way out, so that B_rot and
 * C_rot are written once (the input projection of the block,
 * papers.ananclaw.com/promo/explainers__2603-15569, "关键公式与“伪代码”"; RMS
 * normalisation and bias of B and C, linkstar.cloud/article/869,
 * "架构上的其他改动"; the rotation fused with the projection, same page,
 * "第二刀"):
 *   p_t = W u_t  (features ordered (B or C, head, rank, n)),
 *   v = p / sqrt(mean_n p^2 + eps) * gain + bias  (per (token, B or C, head,
 *       rank) vector of N entries),
 *   B_rot, C_rot = R(-phi_t) v with phi_t = angle0 + sum_{s<=t} dt_s theta_s
 *       (as mamba3_rope_bc), angle_final = phi_L.
 * B_rot and C_rot are in the frame that chunked_fwd expects when it is given
 * theta = 0 (then its h_final is in that frame too).
 *   d: batch, seqlen, nheads, dstate (N), rank (R) as for the core; headdim and
 *      chunk are ignored; io_dtype must be M3_BF16; flags 0.
 *   d_model: D, a positive multiple of 64 and at most 2^20
 *      (M3_ERR_UNSUPPORTED otherwise).
 *   u: (B, L, D) bf16.  W: (2*H*R*N, D) bf16, row-major: the H*R*N rows of
 *      W_B, then those of W_C.
 *   gain, bias: nullable (2, H, R, N) fp32 (NULL: 1 and 0).
 *   eps: >= 0 and finite (M3_ERR_UNSUPPORTED otherwise).  With eps = 0 an
 *      all-zero projected vector gives NaN, as the formula does.
 *   dt (B, L, H), theta (B, L, H, N/2), angle0 nullable (B, H, N/2): fp32.
 *   B_rot, C_rot: (B, L, H, R, N) bf16, written (must not alias inputs).
 *   angle_final: nullable (B, H, N/2) fp32, written.
 *   workspace: at least mamba3_bc_prologue_workspace_size(d) bytes (the fp32
 *      angle totals of every 64-token chunk, then the cosine and sine of every
 *      token's angles as fp16 pairs, 4 bytes per (token, head, pair));
 *      contents on entry do not matter.
 * Products: bf16 MFMAs with fp32 accumulation; normalisation, bias and
 * rotation in fp32; outputs rounded to bf16 (nearest even).
 * Alignment: u, W, B_rot, C_rot, gain, bias and the workspace 16-byte; the
 * others 4-byte.  seqlen is limited to 65535 * 64 tokens and 2*H*R*N to
 * 134,213,632 features (M3_ERR_UNSUPPORTED); any number of tokens B*L is taken (the
 * library launches the product in token slices that keep each launch under
 * 2^32 work-items). */
m3_status mamba3_bc_prologue(const m3_dims* d, int64_t d_model, const void* u, const void* W,
                             const float* gain, const float* bias, float eps,
                             const float* dt, const float* theta, const float* angle0,
                             void* B_rot, void* C_rot, float* angle_final,
                             void* workspace, size_t workspace_bytes, void* stream);
size_t mamba3_bc_prologue_workspace_size(const m3_dims* d);

/* ---------------------------------------------------------------------------
 * The residual block around the core: norm, products, gated feed-forward.
 *
 * A row is one token's vector; every operand below is a matrix of rows.
 * Row-major; io operands (x, W, residual, y, pre, dy, dx, dW) are fp32 or bf16,
 * all of one call the same type.  gain, bias, mean, rstd, dgain, dbias are
 * fp32.  Sums, statistics and activations are held in fp32; bf16 outputs are
 * rounded once (nearest even); the backward's products take
 * dP (below) rounded to bf16 when io is bf16.
 *
 * Strides: x, y (or dy) and residual (or dskip) may have rows further apart
 * than they are wide (a column slice of a wider matrix): the stride fields
 * count elements from row to row, 0 stands for contiguous rows, and a stride
 * below the width is M3_ERR_SHAPE.  Every other operand is contiguous.
 *
 * Any row count from 0, any width from 1, odd ones included.  The products
 * read x, W and dy (as dP) 16 bytes at a time; where a width or stride of them
 * is no multiple of 16 bytes they are first copied into the workspace, so such
 * sizes cost a pass over those operands.  Alignment: x and W, and dy of
 * linear_bwd with M3_ACT_NONE, 16 bytes where their rows lie on 16 bytes,
 * unless flags holds M3_FLAG_UNALIGNED, which makes the call copy them (the
 * workspace queries count it in); every other pointer its element's size,
 * the workspaces 16.  Limits
 * (M3_ERR_UNSUPPORTED): widths and strides at most 2^20, rows at most 2^24 - 1,
 * and at most 2^24 - 1 tiles of 64 x 64 outputs in any product of a call.
 * With rows = 0 nothing is read and no row written; gradients summed over the
 * rows (dW, dgain, dbias) are written as zeros.
 *
 * Outputs must not alias inputs, save y over residual and dx over dskip (same
 * strides).  Results do not depend on the launch's timing: every sum is taken
 * in a fixed order. */
#define M3_FLAG_UNALIGNED 0x40000
typedef enum {
  M3_ACT_NONE = 0,
  M3_ACT_RELU = 1,      /* max(z, 0); derivative 0 at 0 */
  M3_ACT_SILU = 2,      /* z sigmoid(z) */
  M3_ACT_GELU = 3,      /* z Phi(z), Phi the normal distribution function */
  M3_ACT_GELU_TANH = 4, /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
  M3_ACT_SIGMOID = 5
} m3_act;

typedef struct {
  int64_t rows;
  int64_t width;       /* D */
  int64_t x_stride;    /* of x */
  int64_t y_stride;    /* of y (forward) or dy (backward) */
  int64_t skip_stride; /* of dskip (backward) and dx; ignored forward */
  int32_t io_dtype;
  int32_t flags;       /* must be 0 */
} m3_norm_dims;

/* y = (x - mean) rstd gain + bias with mean and rstd = 1/sqrt(var + eps) of
 * each row (var about the mean, divided by D).
 * gain, bias: nullable (D) (NULL: 1 and 0).  eps: >= 0 and finite
 * (M3_ERR_UNSUPPORTED otherwise).  mean, rstd: nullable pair (rows), written
 * when given (the backward takes them). */
m3_status mamba3_layer_norm_fwd(const m3_norm_dims* d, const void* x, const float* gain, const float* bias,
                                float eps, void* y, float* mean, float* rstd, void* stream);

/* Its backward: with xh = (x - mean) rstd and a = dy gain,
 *   dx = rstd (a - mean_D(a) - xh mean_D(a xh)) + dskip,
 *   dgain = sum over rows of dy xh,  dbias = sum over rows of dy.
 * dskip: nullable, the gradient that reaches x past the norm (the residual
 * path), with row stride skip_stride, which is dx's too.  dx: nullable.
 * dgain, dbias: nullable, each by itself.  workspace: at least
 * mamba3_layer_norm_bwd_workspace_size(d) bytes (partial column sums), needed
 * when dgain or dbias is given; contents on entry do not matter. */
m3_status mamba3_layer_norm_bwd(const m3_norm_dims* d, const void* x, const float* gain, const float* mean,
                                const float* rstd, const void* dy, const void* dskip, void* dx, float* dgain,
                                float* dbias, void* workspace, size_t workspace_bytes, void* stream);
size_t mamba3_layer_norm_bwd_workspace_size(const m3_norm_dims* d);

typedef struct {
  int64_t rows;            /* M */
  int64_t d_in;            /* K: width of x */
  int64_t d_out;           /* N: width of y (gated_ffn: F, of h) */
  int64_t x_stride;        /* of x */
  int64_t y_stride;        /* of y or h (forward), dy or dh (backward) */
  int64_t residual_stride; /* of residual (linear_fwd only) */
  int32_t io_dtype;
  int32_t act;             /* m3_act */
  int32_t flags;           /* 0 or M3_FLAG_UNALIGNED */
  int32_t reserved;        /* must be 0 */
} m3_linear_dims;

/* pre = x W^T + bias, y = act(pre) + residual.
 * W: (N, K).  bias: nullable (N).  residual: nullable (M, N).
 * pre: nullable (M, N), written when given (the backward takes it for any
 * activation but M3_ACT_NONE).
 * workspace: at least mamba3_linear_fwd_workspace_size(d) bytes (copies of x
 * and W where their rows need them, fp32 partial sums of tiles whose K is
 * split over several blocks; may be 0); contents on entry do not matter. */
m3_status mamba3_linear_fwd(const m3_linear_dims* d, const void* x, const void* W, const float* bias,
                            const void* residual, void* y, void* pre, void* workspace, size_t workspace_bytes,
                            void* stream);
size_t mamba3_linear_fwd_workspace_size(const m3_linear_dims* d);

/* Its backward: dP = dy act'(pre), dx = dP W, dW = dP^T x, dbias = sum over
 * rows of dP (the residual's gradient is dy itself).
 * pre: required unless act is M3_ACT_NONE (then ignored).  dx (M, K), dW
 * (N, K), dbias (N): nullable, each by itself; x is needed for dW, W for dx.
 * workspace: at least mamba3_linear_bwd_workspace_size(d) bytes (dP, copies,
 * partial sums), whichever gradients are asked for; a call that asks for none
 * returns after its checks and needs none. */
m3_status mamba3_linear_bwd(const m3_linear_dims* d, const void* x, const void* W, const void* pre, const void* dy,
                            void* dx, void* dW, float* dbias, void* workspace, size_t workspace_bytes,
                            void* stream);
size_t mamba3_linear_bwd_workspace_size(const m3_linear_dims* d);

/* Gated feed-forward: pre = [g u] = x W^T + bias, h = act(g) u (entry by
 * entry).  W: (2F, K), the F rows of the gate's projection, then the F of the
 * other.  bias: nullable (2F), in the same order.  pre: nullable (M, 2F), g
 * then u in each row, written when given (the backward takes it). */
m3_status mamba3_gated_ffn_fwd(const m3_linear_dims* d, const void* x, const void* W, const float* bias, void* h,
                               void* pre, void* workspace, size_t workspace_bytes, void* stream);
size_t mamba3_gated_ffn_fwd_workspace_size(const m3_linear_dims* d);

/* Its backward: dP = [dh u act'(g), dh act(g)], dx = dP W, dW = dP^T x,
 * dbias = sum over rows of dP.  pre is required; the rest as linear_bwd with
 * 2F rows of W. */
m3_status mamba3_gated_ffn_bwd(const m3_linear_dims* d, const void* x, const void* W, const void* pre,
                               const void* dh, void* dx, void* dW, float* dbias, void* workspace,
                               size_t workspace_bytes, void* stream);
size_t mamba3_gated_ffn_bwd_workspace_size(const m3_linear_dims* d);

/* ---------------------------------------------------------------------------
 * An attention layer beside the core: norms of queries and keys with their
 * rotation, windowed attention with sinks, and that over a cache.
 *
 * A row is one token: its heads side by side, head_dim entries each (queries
 * q_heads of them, keys and values kv_heads).  The stride fields count elements
 * from token to token, so that queries, keys and values may be slices of one
 * projection's rows; 0 stands for contiguous rows, and a stride below a row's
 * width is M3_ERR_SHAPE.  io operands are fp32 or bf16, all of one call the
 * same type.  Sums, softmax statistics and angles' reductions are held in fp32
 * (angles in fp64) and outputs rounded once (nearest even); for bf16 io the
 * softmax weights p and the scores' gradients ds are rounded to bf16 as
 * operands of the products that take them, one rounding each as the outputs'.
 *
 * Limits (M3_ERR_UNSUPPORTED beyond them): strides and rows' widths at most
 * 2^20, tokens of a call at most 2^24 - 1.  Outputs must not alias inputs
 * unless stated.  Results do not depend on the launch's timing. */
#define M3_FLAG_ROPE_HALVES 0x80000  /* qk_norm_rope: pairs (j, j + rope_dim/2) rather than (2j, 2j + 1) */
#define M3_FLAG_PACKED 0x100000      /* window_attn: sequences of any lengths, given by starts */

typedef struct {
  int64_t rows;          /* tokens */
  int64_t seqlen;        /* without pos, row r stands at position r mod seqlen (0: r) */
  int64_t q_heads, k_heads;  /* either may be 0: its pointers are ignored */
  int64_t head_dim;      /* D, 1 to 256 */
  int64_t rope_dim;      /* the first entries, which are rotated: even, 0 to D */
  int64_t q_stride, k_stride;          /* of q and k */
  int64_t q_out_stride, k_out_stride;  /* of q_out and k_out (forward), of their gradients (backward) */
  int64_t dq_stride, dk_stride;        /* of dq and dk (backward) */
  int32_t io_dtype;
  int32_t flags;         /* 0 or M3_FLAG_ROPE_HALVES */
} m3_norm_rope_dims;

/* For every head x of q and k: z = x / sqrt(mean x^2 + eps) gain, then every
 * pair (a, b) of z's first rope_dim entries turned by the angle w = pos
 * theta[pair]: (a cos w - b sin w, a sin w + b cos w).
 * gain_q, gain_k: nullable (D) (NULL: 1).  eps: >= 0 and finite.
 * theta: (rope_dim/2) fp32 angle rates, required unless rope_dim is 0.
 * pos: nullable (rows) positions, any sign.  Angles are taken in fp64, squares
 * summed in fp32: entries should lie below about 2^60 (a sum that overflows
 * gives a head of zeros) and, without eps, above 2^-60.
 * q_out and k_out may be q and k themselves (same strides).
 * Alignment: an element's size (pos 8). */
m3_status mamba3_qk_norm_rope_fwd(const m3_norm_rope_dims* d, const void* q, const void* k, const float* gain_q,
                                  const float* gain_k, float eps, const float* theta, const int64_t* pos,
                                  void* q_out, void* k_out, void* stream);

/* Its backward from q, k and the gradients dq_out, dk_out of the results: with
 * r = 1 / sqrt(mean x^2 + eps), xh = x r, dz the incoming gradient turned back
 * and a = dz gain,
 *   dx = r (a - xh mean(a xh)),  dgain = sum over tokens and heads of dz xh.
 * dq, dk: written (may be dq_out, dk_out themselves with the same strides).
 * dgain_q, dgain_k: nullable (D) fp32, each by itself; zeros where its heads
 * or the rows are 0.
 * workspace: at least mamba3_qk_norm_rope_bwd_workspace_size(d) bytes (partial
 * sums), needed when dgain_q or dgain_k is given. */
m3_status mamba3_qk_norm_rope_bwd(const m3_norm_rope_dims* d, const void* q, const void* k, const void* dq_out,
                                  const void* dk_out, const float* gain_q, const float* gain_k, float eps,
                                  const float* theta, const int64_t* pos, void* dq, void* dk, float* dgain_q,
                                  float* dgain_k, void* workspace, size_t workspace_bytes, void* stream);
size_t mamba3_qk_norm_rope_bwd_workspace_size(const m3_norm_rope_dims* d);

typedef struct {
  int64_t batch;           /* sequences */
  int64_t q_len, kv_len;   /* of each sequence; ignored when packed */
  int64_t rows;            /* packed: tokens in all; else ignored */
  int64_t kv_rows;         /* rows of k and v from sequence to sequence (0: kv_len; at least that), e.g. a
                              cache's capacity; ignored when packed */
  int64_t q_heads, kv_heads;  /* kv_heads divides q_heads: head i of q uses head i / (q_heads / kv_heads) */
  int64_t head_dim;        /* D: a multiple of 8, 8 to 128 */
  int64_t window;          /* 0: none */
  int64_t sinks;           /* first tokens that stay visible behind the window */
  int64_t q_stride, k_stride, v_stride, o_stride;
  int64_t do_stride, dq_stride, dk_stride, dv_stride;  /* backward */
  float scale;             /* of the scores: > 0, at most 2.35e38 */
  int32_t io_dtype;
  int32_t flags;           /* 0 or M3_FLAG_PACKED */
  int32_t reserved;        /* must be 0 */
} m3_attn_dims;

/* Query i of a sequence stands at position p = kv_len - q_len + i and sees key
 * j (at position j) if j <= p and, with a window, p - j < window or j < sinks:
 *   s_j = scale q k_j over what is seen,  lse = log sum exp s,
 *   o = sum_j exp(s_j - lse) v_j.
 * A query that sees nothing (p < 0) gets o = 0 and lse = -inf.  What a query
 * does not see may hold anything finite; rows of other sequences, and rows of
 * k and v past kv_len, anything at all.
 * Without M3_FLAG_PACKED: q and o are (batch, q_len) rows, k and v (batch,
 * kv_rows) rows of which the first kv_len are keys; starts is ignored.  With it:
 * q, k, v and o have `rows` rows, sequence b those from starts[b] to
 * starts[b + 1] - 1 (batch + 1 entries, rising, on the device; queries and keys
 * have the same); rows of no sequence are not written, and what they hold does
 * not matter.  Starts that do not rise, or lie past the rows, give undefined
 * results, but no access outside the operands and the workspace.
 * lse: nullable (tokens, q_heads) fp32, written when given (the backward takes
 * it).
 * Alignment: io pointers, and rows (strides), 16 bytes; starts 8.
 * Limits (M3_ERR_UNSUPPORTED beyond them), n being 2^24 - 1:
 *   equal lengths: batch q_len, batch kv_len and q_heads batch ceil(q_len / 128)
 *   at most n, kv_heads batch ceil(kv_len / 128) at most n - 2^15, kv_rows at
 *   most 2^40;
 *   packed: q_heads (rows / 128 + the smaller of batch and rows) at most n - 2^15. */
m3_status mamba3_window_attn_fwd(const m3_attn_dims* d, const void* q, const void* k, const void* v,
                                 const int64_t* starts, void* o, float* lse, void* stream);

/* Its backward: with p = exp(s - lse), dp = do v^T and delta = sum over D of
 * do o (o and lse as the forward gave them),
 *   ds = p (dp - delta),  dq = scale ds k,  dk = scale ds^T q,  dv = p^T do,
 * dk and dv summed over the query heads that share a head.  dq, dk, dv:
 * nullable, each by itself.  Keys that no query sees get zeros.  dk and dv lie
 * as k and v do: with kv_rows above kv_len their rows past kv_len are not
 * written.
 * Beside the forward's limits, tokens times ceil(q_heads / 16) is at most
 * 2^24 - 1 (with 32 heads, half of the forward's tokens).
 * workspace: at least mamba3_window_attn_bwd_workspace_size(d) bytes (per query
 * and head two fp32 statistics, and partial sums of the sinks' keys, which
 * whole sequences see: those are summed in pieces of at least 256 queries side
 * by side, 1024 D bytes for each piece, 32 keys with sinks among them and head of
 * keys, 8192 such sums at most).  16-byte aligned, as every io pointer. */
m3_status mamba3_window_attn_bwd(const m3_attn_dims* d, const void* q, const void* k, const void* v, const void* o,
                                 const float* lse, const void* dout, const int64_t* starts, void* dq, void* dk,
                                 void* dv, void* workspace, size_t workspace_bytes, void* stream);
size_t mamba3_window_attn_bwd_workspace_size(const m3_attn_dims* d);

typedef struct {
  int64_t batch;
  int64_t tokens;          /* T new tokens of each sequence, 1 to 16 (several: drafted tokens to verify) */
  int64_t capacity;        /* slots of each sequence's cache, at most 2^30 */
  int64_t q_heads, kv_heads, head_dim, window, sinks;  /* as above */
  int64_t q_stride, k_stride, v_stride, o_stride;      /* of the new tokens */
  int64_t k_cache_stride, v_cache_stride;              /* from slot to slot */
  float scale;
  int32_t io_dtype;
  int32_t flags;           /* must be 0 */
  int32_t reserved;        /* must be 0 */
} m3_attn_decode_dims;

/* The same for T new tokens of each sequence over a cache that it writes them
 * to first.  The token at position p lies in slot p if p < sinks, and in slot
 * sinks + (p - sinks) mod (capacity - sinks) otherwise: the sinks stay, the
 * rest is a ring (a cache longer than the sequence never wraps).
 * q, o: (batch, T) rows; k, v: (batch, T) rows of the new tokens, rotated
 * already; k_cache, v_cache: (batch, capacity) rows, updated in place.
 * lens: (batch) tokens in the cache before the call, on the device; a negative
 * one marks an idle sequence: its cache is left alone and its o set to 0.
 * Slots that hold no token yet may hold anything.
 * With a window, capacity - sinks is at least window + T - 1 (M3_ERR_SHAPE
 * otherwise); without one, at least T, and every token sees all earlier ones
 * that the cache holds after the write.
 * The last of the new tokens may be dropped (drafted ones that were refused) by a
 * lens that does not count them: the next call writes over them.  The older
 * tokens that they had overwritten are behind every later token's window; without
 * a window this holds until the cache wraps, and not from then on: a dropped
 * token would be seen at the position of the one it overwrote.
 * workspace: at least mamba3_window_attn_decode_workspace_size(d) bytes
 * (results of parts of a long cache; may be 0).
 * Alignment: io pointers, strides and the workspace 16 bytes, lens 8. */
m3_status mamba3_window_attn_decode(const m3_attn_decode_dims* d, const void* q, const void* k, const void* v,
                                    void* k_cache, void* v_cache, const int64_t* lens, void* o, void* workspace,
                                    size_t workspace_bytes, void* stream);
size_t mamba3_window_attn_decode_workspace_size(const m3_attn_decode_dims* d);

const char* mamba3_status_string(m3_status s);
int mamba3_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA3_SSM_H */
