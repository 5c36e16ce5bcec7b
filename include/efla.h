/*
 * efla.h - C ABI of the EFLA (Exact Flow Linear Attention) token mixer for
 * NVIDIA B200 (sm_100a).
 *
 * The method ("Exact Flow Linear Attention: Exact Solution from
 * Continuous-Time Dynamics", papernotes.org summary of arXiv 2512.12602):
 *
 *   lambda_t = ||k_t||^2                                   (关键设计 2)
 *   alpha_t  = (1 - e^{-beta_t lambda_t}) / lambda_t       (关键设计 2)
 *            = -expm1(-beta_t lc) / lc, lc = max(lambda_t, 1e-12), in fp32
 *                                                          (损失函数 / 训练策略)
 *   S_t      = (I - alpha_t k_t k_t^T) S_{t-1} + alpha_t k_t v_t^T
 *   o_t      = S_t^T q_t                (post-update state; 整体框架 flowchart)
 *
 * EFLA_MODE_EULER replaces alpha_t by beta_t, which is the DeltaNet
 * (explicit Euler) update of section 关键设计 1; everything else is shared.
 *
 * Conventions for every call:
 *  - All tensor pointers are DEVICE pointers owned by the caller.  The
 *    library allocates nothing; efla_chunk_fwd takes caller-owned scratch.
 *  - Layouts are dense row-major (C-contiguous):
 *      q, k      [B][H][L][d_k]       v, o      [B][H][L][d_v]
 *      beta, alpha, lambda [B][H][L]  (fp32)
 *      S0, S_L, S          [B][H][d_k][d_v] (fp32)
 *    For decode L is absent: q,k [B][H][d_k], v,o [B][H][d_v], beta [B][H].
 *  - q, k and v share one storage dtype (`dtype`); the output o has its
 *    own dtype (`o_dtype`, fp32 or bf16); beta, alpha, lambda and every
 *    state are fp32.  Arithmetic is fp32 throughout (the bf16 chunk path
 *    feeds bf16 operands to tensor-core products that accumulate in fp32;
 *    the state is kept in fp32).  A bf16 o adds its own rounding (up to
 *    2^-8 relative per element) on top of the arithmetic error.
 *  - Supported head sizes: d_k == d_v in {32, 64, 128}; anything else
 *    returns EFLA_ERR_UNSUPPORTED.  B, H >= 0; L >= 0 (L = 0 copies S0 to
 *    S_L); L need not be a multiple of the internal chunk size.
 *  - Every pointer must be 16-byte aligned (EFLA_ERR_ALIGN otherwise).
 *  - Validation is synchronous and happens before anything is enqueued; on
 *    any error nothing is launched.  Work is enqueued on `stream` and runs
 *    asynchronously.  Launch failures return EFLA_ERR_CUDA.  Faults that
 *    happen later on the device surface through efla_last_error() or the
 *    caller's next synchronising CUDA call.
 *  - beta may be any real number; NaN and Inf propagate into the outputs
 *    and are not reported as errors.
 *  - The calls are thread-safe and keep no host state between calls except
 *    the sticky device error word read by efla_last_error().
 */
#ifndef EFLA_H
#define EFLA_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t / CUstream.  NULL selects the legacy default stream. */
typedef struct CUstream_st *efla_stream_t;

typedef enum {
    EFLA_OK = 0,
    EFLA_ERR_NULL = 1,        /* a required pointer is NULL                        */
    EFLA_ERR_SHAPE = 2,       /* a negative size, or an overflowing element count  */
    EFLA_ERR_DTYPE = 3,       /* unknown efla_dtype_t / efla_mode_t                */
    EFLA_ERR_ALIGN = 4,       /* a pointer is not 16-byte aligned                  */
    EFLA_ERR_UNSUPPORTED = 5, /* head size outside {32,64,128} or d_k != d_v       */
    EFLA_ERR_CUDA = 6,        /* a CUDA runtime call or kernel launch failed       */
    EFLA_ERR_TIMEOUT = 7,     /* a device-side bounded wait gave up (sticky word)  */
    EFLA_ERR_WORKSPACE = 8,   /* workspace missing or smaller than required        */
    EFLA_ERR_ALIAS = 9        /* an output overlaps an input it must not overlap   */
} efla_status_t;

typedef enum { EFLA_F32 = 0, EFLA_BF16 = 1 } efla_dtype_t;

typedef enum {
    EFLA_MODE_EXACT = 0, /* exact-flow gate alpha_t (EFLA)                 */
    EFLA_MODE_EULER = 1  /* alpha_t = beta_t (DeltaNet / explicit Euler)   */
} efla_mode_t;

/* Human-readable name of a status code (static storage, never NULL). */
const char *efla_status_string(efla_status_t status);

/* Library version as 10000*major + 100*minor + patch. */
int efla_version(void);

/*
 * Sticky device error word of the current device.  Synchronises the
 * current device, returns EFLA_ERR_TIMEOUT if a kernel's bounded wait gave
 * up since the last call (and clears the word), EFLA_ERR_CUDA if the CUDA
 * context holds an error, else EFLA_OK.
 */
efla_status_t efla_last_error(void);

/*
 * Diagnostic: launch one CTA that waits on an mbarrier nothing ever arrives
 * on, through the same clock-bounded wait the prefill kernel uses, with a
 * limit of `limit_cycles` SM clock cycles.  The wait gives up, the kernel
 * sets the sticky error word and returns; the next efla_last_error()
 * reports EFLA_ERR_TIMEOUT and the CUDA context stays usable.  Exists so the
 * failure path can be tested without faulting or hanging a GPU.
 */
efla_status_t efla_diag_wait_timeout(long long limit_cycles, efla_stream_t stream);

/*
 * efla_gate - the exact-flow gate (关键设计 2; numerics per 损失函数 /
 * 训练策略): for every row t of k,
 *     lambda[t] = sum_i k[t][i]^2                (fp32 accumulation, unclamped)
 *     alpha[t]  = -expm1(-beta[t]*lc)/lc,  lc = max(lambda[t], 1e-12)
 * (alpha[t] = beta[t] in EFLA_MODE_EULER).
 *   k      [B][H][L][d_k], dtype `dtype`            (input)
 *   beta   [B][H][L] fp32                            (input)
 *   alpha  [B][H][L] fp32                            (output)
 *   lambda [B][H][L] fp32                            (output; may be NULL)
 * alpha must not overlap k or beta.
 */
efla_status_t efla_gate(const void *k, efla_dtype_t dtype, efla_mode_t mode,
                        const float *beta, float *alpha, float *lambda,
                        int B, int H, int L, int d_k, efla_stream_t stream);

/*
 * Bytes of scratch efla_chunk_fwd needs for these sizes (0 if none).  The
 * value depends only on the arguments.
 */
size_t efla_chunk_fwd_workspace_size(efla_dtype_t dtype, int B, int H, int L,
                                     int d_k, int d_v);

/*
 * efla_chunk_fwd - prefill over a whole sequence: runs the recurrence above
 * for t = 0..L-1 from S0 and writes every o_t and the final state.  It
 * evaluates the recurrence chunk by chunk in the UT form of the chunked
 * scheme the pages cite (整体框架: "WY / UT" chunk-parallel products):
 *     A = strictly-lower(diag(alpha) K K^T),  T = (I + A)^{-1},
 *     W = T diag(alpha) K,  U = T diag(alpha) V,
 *     D = U - W S,  O = Q S + lower-incl-diag(Q K^T) D,  S <- S + K^T D,
 * which equals the token-by-token recurrence up to rounding.
 *   q, k  [B][H][L][d_k]   v [B][H][L][d_v]   dtype `dtype`   (inputs)
 *   beta  [B][H][L] fp32                                        (input)
 *   S0    [B][H][d_k][d_v] fp32, or NULL for the zero state     (input)
 *   o     [B][H][L][d_v] dtype `o_dtype`                        (output)
 *   S_L   [B][H][d_k][d_v] fp32, or NULL if not wanted          (output)
 *   workspace / workspace_bytes: caller-owned device scratch of at least
 *     efla_chunk_fwd_workspace_size(...) bytes (may be NULL when that is 0);
 *     its contents on entry are ignored and on exit undefined.
 * S_L may be the same pointer as S0 (in-place state update).  o must not
 * overlap any input; S_L must not overlap q, k, v, beta or o.
 */
efla_status_t efla_chunk_fwd(const void *q, const void *k, const void *v,
                             efla_dtype_t dtype, efla_mode_t mode,
                             const float *beta, const float *S0, void *o,
                             efla_dtype_t o_dtype, float *S_L, int B, int H,
                             int L, int d_k, int d_v,
                             void *workspace, size_t workspace_bytes,
                             efla_stream_t stream);

/*
 * efla_decode_step - one token of the recurrence for B*H independent
 * states, updated in place:
 *     S <- (I - alpha k k^T) S + alpha k v^T,   o = S^T q  (updated S)
 *   q, k [B][H][d_k]   v [B][H][d_v]   dtype `dtype`   (inputs)
 *   beta [B][H] fp32                                    (input)
 *   S    [B][H][d_k][d_v] fp32                          (input/output)
 *   o    [B][H][d_v] dtype `o_dtype`                    (output)
 * o must not overlap S or any input.
 */
efla_status_t efla_decode_step(const void *q, const void *k, const void *v,
                               efla_dtype_t dtype, efla_mode_t mode,
                               const float *beta, float *S, void *o,
                               efla_dtype_t o_dtype, int B, int H, int d_k,
                               int d_v, efla_stream_t stream);

/*
 * efla_prefill_bwd - reverse-mode derivative of efla_chunk_fwd.  The pages
 * train with this mixer but print no backward; it is derived from the
 * recurrence of 关键设计 2 (S_t = S_{t-1} + alpha_t k_t e_t^T with
 * e_t = v_t - S_{t-1}^T k_t, o_t = S_t^T q_t) and the gate of 关键设计 2 /
 * 损失函数 (d alpha/d beta = e^{-beta lambda}, d alpha/d lambda =
 * (beta lambda e^{-beta lambda} - (1 - e^{-beta lambda})) / lambda^2, zero
 * where lambda <= 1e-12).  For the loss sum(dO * o) + sum(dSL * S_L) it
 * returns the gradients with respect to every input:
 *   q, k [B][H][L][d]  v [B][H][L][d]  dtype `dtype`    (forward inputs)
 *   beta [B][H][L] fp32, S0 [B][H][d][d] fp32 or NULL (zero state)
 *   dO [B][H][L][d] fp32; dSL [B][H][d][d] fp32 or NULL (zero)
 *   dq, dk, dv [B][H][L][d] fp32; dbeta [B][H][L] fp32; dS0 [B][H][d][d] fp32
 *   workspace / workspace_bytes: caller-owned device scratch of at least
 *     efla_prefill_bwd_workspace_size(...) bytes.
 * d = d_k = d_v in {32, 64, 128}.  Exact fp32 arithmetic, one CTA per (b,h)
 * walking the sequence three times (forward, backward, forward).  Outputs
 * must not overlap inputs or each other.  Asynchronous on `stream`.
 */
size_t efla_prefill_bwd_workspace_size(int B, int H, int L, int d_k, int d_v);
efla_status_t efla_prefill_bwd(const void *q, const void *k, const void *v, efla_dtype_t dtype, efla_mode_t mode,
                               const float *beta, const float *S0, const float *dO, const float *dSL,
                               float *dq, float *dk, float *dv, float *dbeta, float *dS0,
                               int B, int H, int L, int d_k, int d_v,
                               void *workspace, size_t workspace_bytes, efla_stream_t stream);

/*
 * efla_state_affine - one step of composing the state maps of consecutive
 * sequence segments: for every (b, h),
 *     out = (SI - SZ) X + SZ
 * The state after a segment is affine in the state before it (the
 * recurrence of 关键设计 2 is linear in S): S_out = M S_in + S_Z, where
 * S_Z is the final state from S_in = 0, S_I the final state from the
 * identity and M = S_I - S_Z.  With SI = S_I, SZ = S_Z and X a segment's
 * true initial state, `out` is the next segment's true initial state.  The
 * pages have no such call; sequence-parallel prefill (across GPUs or SMs)
 * is built on it.
 *   SI, SZ, X, out [B][H][d][d] fp32, d = d_k = d_v in {32, 64, 128}.
 *   out must not overlap SI, SZ or X.  Asynchronous on `stream`.
 */
efla_status_t efla_state_affine(const float *SI, const float *SZ, const float *X, float *out,
                                int B, int H, int d, efla_stream_t stream);

/*
 * efla_chunk_fwd_noalloc - the same prefill as efla_chunk_fwd, for callers
 * that cannot allocate device memory.  The pages describe no such call; it
 * exists for this library's users.  Some hosts (inference engines and
 * plugins that budget every byte of GPU memory through their own pool, or
 * latency-critical loops where cudaMalloc/cudaFree would synchronise the
 * device) cannot hand this library a scratch buffer or let it allocate one.
 * This entry point takes no workspace and allocates nothing: its scratch is
 * a fixed array of EFLA_NOALLOC_SCRATCH_BYTES (32 MiB) that the library
 * places in device memory of every GPU on which it is loaded and keeps until
 * the process exits.
 *   Arguments, layouts and results are those of efla_chunk_fwd.  It always
 *   runs the CUDA-core (exact fp32) chunked kernels, for every dtype and head
 *   size.  Problems whose scratch would not fit
 *   (efla_chunk_fwd_workspace_size_simt > EFLA_NOALLOC_SCRATCH_BYTES, e.g.
 *   more than 409 head-chunks of 64 tokens at d = 128) return
 *   EFLA_ERR_WORKSPACE before anything is launched.
 *   The first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress); make that first call before capturing a stream
 *   into a CUDA graph.
 *   Every call on a device shares the one array and leaves its contents
 *   behind; nothing in it needs to start zeroed.  Calls whose kernels overlap
 *   on the GPU (other streams, other host threads) race on it: serialise them.
 */
#define EFLA_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)

/* Scratch bytes the CUDA-core chunked kernels need for these sizes. */
size_t efla_chunk_fwd_workspace_size_simt(int B, int H, int L, int d_k, int d_v);

efla_status_t efla_chunk_fwd_noalloc(const void *q, const void *k, const void *v,
                                     efla_dtype_t dtype, efla_mode_t mode,
                                     const float *beta, const float *S0,
                                     void *o, efla_dtype_t o_dtype, float *S_L,
                                     int B, int H, int L, int d_k, int d_v,
                                     efla_stream_t stream);

/* ---------------------------------------------------------------------------
 * The operators around the mixer.  A block has the norm of the residual
 * stream in front of its projections, the short convolution on what they
 * give (the pages' layer has one of width 4, jsqmd.com blog 4.1), the mixer
 * (or, in layers that mix the two, a selective state space scan), and the
 * norm of the mixer's output per head.  The pages print no formulas for
 * these; they are the usual ones, written below.
 *
 * Conventions beyond those above: activations are [B][L][channels]
 * (channels-last) in `dtype`; parameters and recurrent states are fp32,
 * except the convolution's state, which is the last inputs themselves and has
 * their dtype.  Where a call takes a row stride (ld...), in elements, token
 * (b, t) is at base + (b * L + t) * ld, so a column slice of a wider
 * projection can be passed as it is; such a base needs the alignment of its
 * element alone (16-byte aligned rows of whole vectors are faster).  All
 * other pointers are 16-byte aligned and dense.  `lengths` [B] (int32,
 * device; NULL: all L) is each sequence's number of tokens, taken into
 * [0, L]: tokens from there on are padding, which is not read into any
 * result; their outputs and gradients are zeros.  L is at most 0x7fff0000.
 * Workspaces, as large as the call's _workspace_size says for its sizes, hold
 * nothing between calls.  Outputs must not overlap
 * inputs or each other, except where a call says so.  Gradients of
 * activations have the activations' dtype, gradients of parameters are fp32.
 * Every sum is taken in fp32 in a fixed order: the same call gives the same
 * bits.
 */

/*
 * efla_norm_fwd - root-mean-square norm of rows, with the residual's addition:
 *     h = x + res,  y = h / sqrt(mean(h^2) + eps) * weight,  res_out = h
 *   x [rows][C] dtype `dtype`; res, res_out [rows][C] dtype `res_dtype` (the
 *   dtype of x, or fp32), or both NULL; res_out may be NULL
 *   weight [C] fp32
 *   y [rows][C] dtype `dtype`, or NULL
 *   y8 [rows][C] e4m3, scale [rows][ceil(C / group)] fp32, or both NULL:
 *     scale = max(max |y| / 448, 2^-126) over each group of columns,
 *     y8 = y / scale rounded to e4m3 (y from the fp32 value, not its rounding; the
 *     quotient in fp32, so that one within 11 2^-24 of the border between two
 *     values of e4m3 may become either)
 *   group: 128, or 0 for one scale a row.  C <= 16384.
 * At least one of y and y8.  In place: res_out may be res; y or res_out may
 * be x (res_out only where the dtypes agree).  Fewer than 2^31 rows.  Squares
 * are summed in fp32: a row whose mean square passes its range (values from
 * 10^19 on) is normed to zeros.
 */
efla_status_t efla_norm_fwd(const void *x, efla_dtype_t dtype, const void *res, efla_dtype_t res_dtype,
                            const float *weight, float eps, void *y, void *y8, float *scale, int group, void *res_out,
                            long long rows, int C, efla_stream_t stream);

/*
 * efla_norm_bwd - its backward pass.  With h the sum that was normed
 * (res_out, or x), dy the gradient of y and dres_out that of res_out (NULL: 0):
 *     u = weight dy,  dh = (u - h mean(u h) / (mean(h^2) + eps)) / sqrt(mean(h^2) + eps) + dres_out
 *     dweight = sum over rows of dy h / sqrt(mean(h^2) + eps)
 *   dy [rows][C] `dtype`; h, dres_out [rows][C] `h_dtype` (the dtype of dy, or fp32)
 *   dx [rows][C] `dtype` and dres [rows][C] `h_dtype` are dh; either may be NULL
 *   dweight [C] fp32
 */
size_t efla_norm_bwd_workspace_size(long long rows, int C);
efla_status_t efla_norm_bwd(const void *dy, efla_dtype_t dtype, const void *h, efla_dtype_t h_dtype,
                            const float *weight, float eps, const void *dres_out, void *dx, void *dres, float *dweight,
                            long long rows, int C, void *workspace, size_t workspace_bytes, efla_stream_t stream);

/*
 * efla_conv_fwd - short causal convolution along the sequence, a filter of
 * K = 2, 3 or 4 taps a channel, with SiLU if `silu`:
 *     y_t = act(bias + sum_j weight[j] x_{t-K+1+j}),  j = 0 .. K-1
 *   x [B][L][C] rows `ldx` apart; weight [C][K], bias [C] (or NULL) fp32
 *   state [B][K-1][C] `dtype`: the K-1 inputs before x, oldest first (NULL: 0)
 *   state_out [B][K-1][C]: the last K-1 inputs of each sequence (or NULL); may be `state`
 *   y: [B][L][C] where heads is 0, else [B][heads][L][C / heads], the layout
 *     of the mixer's q, k and v
 * C <= 2097120, B ceil(L / 32) <= 0x7fff0000.
 */
efla_status_t efla_conv_fwd(const void *x, long long ldx, efla_dtype_t dtype, const float *weight, const float *bias,
                            const void *state, const int *lengths, int silu, void *y, int heads, void *state_out,
                            int B, int L, int C, int K, efla_stream_t stream);

/*
 * efla_conv_bwd - its backward pass.  dy has the layout of y; dstate_out is
 * the gradient of state_out (NULL: 0).  dx [B][L][C] dense; dweight [C][K],
 * dbias [C] (or NULL), dstate [B][K-1][C] `dtype` (or NULL).
 */
size_t efla_conv_bwd_workspace_size(int B, int L, int C, int K);
efla_status_t efla_conv_bwd(const void *dy, const void *x, long long ldx, efla_dtype_t dtype, const float *weight,
                            const float *bias, const void *state, const int *lengths, int silu, int heads,
                            const void *dstate_out, void *dx, float *dweight, float *dbias, void *dstate, int B, int L,
                            int C, int K, void *workspace, size_t workspace_bytes, efla_stream_t stream);

/*
 * efla_conv_step - one token: x [B][C] rows `ldx` apart, state [B][K-1][C]
 * updated in place, y [B][C].
 */
efla_status_t efla_conv_step(const void *x, long long ldx, efla_dtype_t dtype, void *state, const float *weight,
                             const float *bias, int silu, void *y, int B, int C, int K, efla_stream_t stream);

/*
 * Diagnostic: tokens of a thread's run in efla_conv_fwd (backward = 0) or
 * efla_conv_bwd where a thread has `channels` neighbouring channels: forward 4,
 * backward 2, or 1 where rows or heads are not aligned for that; lengths: whether
 * the call has some.  0 for other arguments.  For tests that mean to reach a run
 * of some length.
 */
int efla_diag_conv_run(int B, int L, int C, int channels, int backward, int lengths);

/*
 * efla_scan_fwd - selective state space scan, N state values a channel:
 *     D_t = softplus(dt_t + dt_bias)   (dt_t + dt_bias where `softplus` is 0)
 *     h_t = exp(D_t A) h_{t-1} + D_t x_t B_t,   y_t = (<C_t, h_t> + D x_t) silu(z_t)
 *   x, dt, z [B][L][C] rows ldx, lddt, ldz apart (z may be NULL: no gate)
 *   Bm, Cm [B][L][G][N] tokens ldb, ldc apart; channel c reads group c / (C / G)
 *   A [C][N] fp32, finite; D [C], dt_bias [C] fp32 (or NULL: 0)
 *   h0 [B][C][N] fp32 (NULL: 0); h_L [B][C][N] fp32 (or NULL); h_L may be h0
 *   y [B][L][C]
 * N in {8, 16, 32, 64}; G divides C.  C N is below 2^31; the blocks of a pass,
 * each of at least 8 channels (or a narrower group) of a sequence, are at most
 * 0x7fff0000.
 */
size_t efla_scan_fwd_workspace_size(int B, int L, int C, int G, int N);
efla_status_t efla_scan_fwd(const void *x, long long ldx, const void *dt, long long lddt, const float *A,
                            const void *Bm, long long ldb, const void *Cm, long long ldc, const float *D, const void *z,
                            long long ldz, const float *dt_bias, const float *h0, const int *lengths,
                            efla_dtype_t dtype, int softplus, void *y, float *h_L, int B, int L, int C, int G, int N,
                            void *workspace, size_t workspace_bytes, efla_stream_t stream);

/*
 * efla_scan_bwd - its backward pass, from dy [B][L][C] and dh_L [B][C][N]
 * (NULL: 0): dx, ddt, dz [B][L][C] (dz where there is z), dB, dC
 * [B][L][G][N], all dense in `dtype`; dA [C][N], dD [C] (or NULL), ddt_bias
 * [C] (or NULL), dh0 [B][C][N] (or NULL) fp32.  Nothing of the forward pass
 * is kept for it: the states are recomputed, from checkpoints in the workspace
 * every few tokens.  With them and the blocks' shares of dB and dC it is large:
 * some 1.25 N bytes (N = 8 to 32; 1.5 N for 64) for every token and channel, 336
 * MB for 8 x 2048 x 1024 x 16.
 */
size_t efla_scan_bwd_workspace_size(int B, int L, int C, int G, int N);
efla_status_t efla_scan_bwd(const void *dy, const void *x, long long ldx, const void *dt, long long lddt,
                            const float *A, const void *Bm, long long ldb, const void *Cm, long long ldc,
                            const float *D, const void *z, long long ldz, const float *dt_bias, const float *h0,
                            const int *lengths, const float *dh_L, efla_dtype_t dtype, int softplus, void *dx,
                            void *ddt, float *dA, void *dB, void *dC, float *dD, void *dz, float *ddt_bias, float *dh0,
                            int B, int L, int C, int G, int N, void *workspace, size_t workspace_bytes,
                            efla_stream_t stream);

/*
 * Diagnostic: how efla_scan_fwd (backward = 0) or efla_scan_bwd cuts a call of
 * these sizes: plan[0] state values of a lane in each of its plan[1] channels,
 * plan[2] segments of plan[3] tokens, plan[4] channel tiles of a group.  For
 * tests that mean to reach a variant.
 */
efla_status_t efla_diag_scan_plan(int B, int L, int C, int G, int N, int backward, int plan[5]);

/*
 * efla_scan_step - one token: x, dt, z [B][C], Bm, Cm [B][G][N] (rows ld...
 * apart), h [B][C][N] fp32 updated in place, y [B][C].  B <= 65535.
 */
efla_status_t efla_scan_step(const void *x, long long ldx, const void *dt, long long lddt, const float *A,
                             const void *Bm, long long ldb, const void *Cm, long long ldc, const float *D,
                             const void *z, long long ldz, const float *dt_bias, efla_dtype_t dtype, int softplus,
                             float *h, void *y, int B, int C, int G, int N, efla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EFLA_H */
