/*
 * ssmscan.h -- C ABI of the MI355X (gfx950) selective state-space scan library.
 *
 * The library computes the input-dependent linear recurrence
 *
 *     h_t = A_t h_{t-1} + b_t,      y_t = C_t . h_t,      t = 0 .. L-1,  h_{-1} = h0,
 *
 * over many independent sequences, forward and backward, for three kinds of
 * transition A_t:
 *
 *   - diagonal real.  SSM_REAL_SELECTIVE forms a_t = exp(delta_t * A) and the
 *     Euler input term b_t = delta_t * x_t * B_t (or the zero-order-hold term
 *     (exp(delta_t A) - 1) / A * x_t * B_t) from a step size delta, as in the
 *     selection-and-discretisation step of the lpnh.cn page "Selective State
 *     Space Models (S3M)", section 1.1.  SSM_REAL_DENSE takes a_t and b_t as
 *     given tensors.
 *   - diagonal complex with shared controls (SPARC page, abstract): two
 *     per-step scalars, retention r_t and phase phi_t, drive every complex mode
 *     m through a_{t,m} = exp(r_t ln(lambda_m) + i phi_t theta_m), with
 *     b_t = u_t and the real readout y_t = Re sum_m c_m h_{t,m}.
 *     SSM_COMPLEX_DENSE takes the complex a_{t,m} as a given tensor (same
 *     recurrence and readout).
 *   - PD (Flash PD-SSM page, section "Neuer Selektionsmechanismus"): per step,
 *     argmax over K scores picks one column-one-hot matrix P from a per-head
 *     dictionary; A_t = P diag(d_t), i.e. h_t[i] = b_t[i] + sum over the
 *     columns j whose one sits in row i of d_t[j] h_{t-1}[j].
 *
 * The scan runs as a chunked (tiled) three-phase computation -- local scans
 * inside chunks, a prefix over chunk summaries, a carry correction -- as the
 * Flash PD-SSM page describes under "Hardwarebewusste Implementierung".  The
 * forward leaves the state entering every chunk of chunk_len steps (the
 * checkpoints); the backward recomputes states tile by tile from them, so the
 * on-chip working set is one chunk and nothing of size O(L * state) is stored
 * (PGF page, abstract: exact analytical derivatives by tiled operator-space
 * evolution instead of a materialised graph).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  Memory.   Every pointer is a device pointer the caller owns, except where
 *            noted.  Tensors are dense, row-major, in the shapes stated, with
 *            no padding (the last dimension is contiguous), unless the call's
 *            ssm_layout describes them as strided views.  The library never
 *            allocates device memory; scratch memory is the caller's workspace
 *            `ws` of at least ssm_workspace_bytes() bytes (256-byte aligned),
 *            used only during the call's stream work.  No pointer is kept
 *            after return.
 *  Streams.  All work is enqueued on `stream` (a hipStream_t; NULL is the
 *            legacy default stream).  There is no host synchronisation and no
 *            host<->device copy.  Buffers must stay valid until the stream
 *            work completes.  Calls on different streams must use different
 *            workspaces and outputs.
 *  Outputs.  Outputs are overwritten, never accumulated.  A NULL output (or
 *            gradient) is not computed.  Outputs must not overlap inputs or
 *            each other.
 *  Types.    Accumulation is float32 everywhere.  For SSM_REAL_SELECTIVE the
 *            streamed tensors (delta, x, Bm, C, y, gy and their gradients)
 *            share `dtype` (SSM_F32 or SSM_BF16, bf16 rounded to nearest even
 *            on output); A, h0, h_last, checkpoints and gA are float32.  All
 *            other modes are float32 (complex64 = interleaved float32 re, im).
 *  Errors.   0 (SSM_OK) on success, a negative SSM_ERR_* code otherwise.  The
 *            arguments are validated completely before anything is enqueued;
 *            on error nothing is written.  ssm_last_error_detail() returns a
 *            thread-local description of the last error.  Device faults are
 *            asynchronous and surface at the caller's next synchronisation.
 *  Results.  Mathematically independent of chunk_len; bitwise deterministic
 *            run to run (no floating-point atomics).
 */
#ifndef SSMSCAN_H
#define SSMSCAN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Entry points added since with structs of their own leave the version as it is:
 * the gated recurrence (ssm_gated_*, ssm_tokens_gated), the group norm
 * (ssm_group_norm_*) and products in 8-bit integers (ssm_tokens_pack8, _mm8).
 * An older library of version 8 has not got these symbols, so what calls them does
 * not link or load with it; where they are looked up at run time, the symbol tells, or
 * ssm_workspace_bytes of SSM_OP_GATED_FWD, which it answers with SSM_ERR_UNSUPPORTED.
 * 8: adds the short causal convolution (ssm_conv_*), 8-bit activation
 * checkpoints (ssm_ckpt8_*) and the serving forms over packed rows
 * (ssm_tokens_*); structs of 7 unchanged.  7 added SSM_HEAD_SCALAR
 * (head_dim field); 6 added strided views (ssm_layout, the layout fields of ssm_scan_args and
 * pd_scan_args) and the ZOH discretisation (discretization field); 5 added
 * ssm_scan_fwd_noalloc and ssm_roof_probe; 4 added SSM_COMPLEX_DENSE; 3 added
 * ssm_sensitivity_rows and SSM_OP_SENS_ROWS; struct layouts as in 2 */
#define SSM_ABI_VERSION 8

/* status codes */
#define SSM_OK               0
#define SSM_ERR_NULL        -1  /* a required pointer is NULL */
#define SSM_ERR_SHAPE       -2  /* a size is < 1 or inconsistent, K or N out of range */
#define SSM_ERR_DTYPE       -3  /* unknown or unsupported element type for the mode */
#define SSM_ERR_LAYOUT      -4  /* misaligned pointer, or an output overlapping another buffer */
#define SSM_ERR_WORKSPACE   -5  /* workspace NULL or smaller than ssm_workspace_bytes() */
#define SSM_ERR_UNSUPPORTED -6  /* valid request this build does not implement (e.g. chunk_len) */
#define SSM_ERR_DEVICE      -7  /* HIP reported an error while enqueuing */

/* element types of streamed tensors */
#define SSM_F32  0
#define SSM_BF16 1

/* transition kinds of ssm_scan_* */
#define SSM_REAL_SELECTIVE 0
#define SSM_REAL_DENSE     1
#define SSM_COMPLEX_SHARED 2
#define SSM_COMPLEX_DENSE  3  /* complex a_t given; f32 only */
#define SSM_HEAD_SCALAR    4  /* one scalar transition per head of head_dim channels (below) */

/* operation ids for ssm_workspace_bytes */
#define SSM_OP_SCAN_FWD 0
#define SSM_OP_SCAN_BWD 1
#define SSM_OP_IMPULSE  2
#define SSM_OP_PD_FWD   3
#define SSM_OP_PD_BWD   4
#define SSM_OP_COMPLEX_RTRL 5
#define SSM_OP_OUTPUT_SENS  6
#define SSM_OP_SENS_ROWS    7
#define SSM_OP_CONV_FWD     8   /* ssm_conv_args: no workspace             */
#define SSM_OP_CONV_BWD     9   /* ssm_conv_args                           */
#define SSM_OP_TOKENS_CONV 10   /* ssm_tokens_conv_args: no workspace      */
#define SSM_OP_TOKENS_SCAN 11   /* ssm_tokens_scan_args                    */
#define SSM_OP_GATED_FWD   12   /* ssm_gated_args: no workspace            */
#define SSM_OP_GATED_BWD   13   /* ssm_gated_args                          */
#define SSM_OP_TOKENS_GATED 14  /* ssm_tokens_gated_args                   */
#define SSM_OP_GROUP_NORM_BWD 15 /* ssm_group_norm_args                    */

/* discretisations of SSM_REAL_SELECTIVE (S3M page, section 1.1) */
#define SSM_EULER 0   /* b_t = delta_t x_t B_t (the default)                               */
#define SSM_ZOH   1   /* zero-order hold: b_t[n] = (exp(delta_t A[d,n]) - 1) / A[d,n] x_t B_t[n],
                         delta_t x_t B_t[n] where A[d,n] = 0 (the limit)                     */

/*
 * Strided views.  By default every tensor is dense and row-major in the shape
 * stated for it.  A caller whose tensors are views -- slices of a larger
 * buffer, or inputs expanded (broadcast) along a dimension -- passes an
 * ssm_layout: for every tensor role r whose bit (1 << r) is set in `given`,
 * stride[r] holds the element strides of the role's dimensions, outermost
 * first (entries past the role's rank are ignored); other roles stay dense.
 * Rules (checked before anything is enqueued):
 *   - the innermost stride must be 1 (rank-1 inputs excepted: the per-head
 *     A may have any stride, 0 included), strides are >= 0 -> SSM_ERR_LAYOUT;
 *   - stride 0 (broadcast) is allowed on inputs only; an output's strides
 *     must give distinct elements                        -> SSM_ERR_LAYOUT;
 *   - a role the mode or entry point does not take as a view -> SSM_ERR_UNSUPPORTED.
 * Gradients of a broadcast input are returned per broadcast position (in the
 * expanded shape); the caller sums them over the broadcast dimension.
 *
 * Roles of ssm_scan_args.layout (logical shape; dense strides):
 *   SSM_REAL_SELECTIVE, every entry point:
 *     SSM_V_DELTA, SSM_V_X  (B,D,L)    inputs; any batch / channel stride
 *     SSM_V_A               (D,N)      channel stride 0: one A row for every channel
 *     SSM_V_BM, SSM_V_C     (B,D,L,N)  dense = (L*N, 0, N, 1): B_t, C_t shared by the
 *                                      channels.  A nonzero channel stride (on either)
 *                                      gives every channel its own B_t / C_t
 *                                      (ssm_scan_fwd / _bwd only); gBm and gC are then
 *                                      both (B,D,L,N) dense, per channel, not sums over
 *                                      channels.  Batch stride 0: shared by the batch
 *                                      rows (gBm / gC stay per batch row).
 *   SSM_REAL_SELECTIVE, ssm_scan_fwd / ssm_scan_bwd:
 *     SSM_V_Y, SSM_V_GY, SSM_V_GDELTA, SSM_V_GX (B,D,L) outputs / upstream gradient
 *   SSM_COMPLEX_SHARED, ssm_scan_fwd / ssm_scan_bwd / ssm_complex_rtrl:
 *     SSM_V_R, SSM_V_PHI    (B,H,L)    head stride 0: one control signal for all heads
 *     SSM_V_U               (B,H,L,M)  complex elements (one (re, im) pair = 1)
 *     SSM_V_LAM, SSM_V_THETA, SSM_V_CC (H,M) head stride 0: shared per-mode parameters
 * Roles of pd_scan_args.layout:
 *     SSM_V_LOGITS          (B,H,L,K)
 *     SSM_V_PD_D, SSM_V_PD_B, SSM_V_PD_C (B,H,L,N)
 *     SSM_V_DICT            (H,K,N)    head stride 0: one dictionary for every head
 */
#define SSM_V_DELTA   0
#define SSM_V_X       1
#define SSM_V_A       2
#define SSM_V_BM      3
#define SSM_V_C       4
#define SSM_V_Y       5
#define SSM_V_GY      6
#define SSM_V_GDELTA  7
#define SSM_V_GX      8
#define SSM_V_R       9
#define SSM_V_PHI    10
#define SSM_V_U      11
#define SSM_V_LAM    12
#define SSM_V_THETA  13
#define SSM_V_CC     14
#define SSM_V_LOGITS 15
#define SSM_V_PD_D   16
#define SSM_V_PD_B   17
#define SSM_V_PD_C   18
#define SSM_V_DICT   19
#define SSM_V_COUNT  20
typedef struct {
    uint64_t given;                    /* bit r: stride[r] describes role r */
    int64_t  stride[SSM_V_COUNT][4];   /* element strides, outermost dimension first */
} ssm_layout;

/*
 * Arguments of the diagonal scans.  Sizes: batch = B; channels = D (real) or
 * H heads (complex); length = L; state = N (real, 1..16) or M complex modes
 * per head (complex, 1..64).  chunk_len = checkpoint interval T in steps:
 * 0 picks the default (256 selective, 32 dense and complex); the selective
 * mode accepts 64, 128 or 256, the dense and complex modes 32.
 * n_chunks = ceil(L / T).  batch, channels and length may be 0 (an empty
 * problem): nothing is read, outputs with no elements are not touched (their
 * pointers may be NULL), h_last becomes h0 (or 0), gh0 becomes gh_last (or 0)
 * and the parameter gradients 0 (gBm and gC, sums over channels, are zero when
 * channels is 0 and batch, length are not); the sensitivity calls still need
 * 0 <= t_out < L.  state must be >= 1.
 */
typedef struct {
    int32_t mode;      /* SSM_REAL_SELECTIVE, SSM_REAL_DENSE, SSM_COMPLEX_SHARED or SSM_COMPLEX_DENSE */
    int32_t dtype;     /* SSM_F32 or SSM_BF16 (bf16: SSM_REAL_SELECTIVE and SSM_COMPLEX_SHARED) */
    int64_t batch, channels, length, state, chunk_len;
    /* SSM_REAL_SELECTIVE */
    const void*  delta;  /* (B,D,L) dtype, step sizes                      */
    const void*  x;      /* (B,D,L) dtype, inputs                          */
    const float* A;      /* (D,N)  f32, continuous-time diagonal (A < 0)   */
    const void*  Bm;     /* (B,L,N) dtype, input projection B_t (shared over D) */
    /* SSM_REAL_DENSE */
    const float* a;      /* (B,D,L,N) f32, transition diagonal a_t;
                            SSM_COMPLEX_DENSE: (B,H,L,M) complex64 a_{t,m}  */
    const float* b;      /* (B,D,L,N) f32, input term b_t                   */
    /* both real modes */
    const void*  C;      /* (B,L,N) dtype (f32 for dense), readout C_t (shared over D) */
    /* SSM_COMPLEX_SHARED (SSM_COMPLEX_DENSE reads u, c and a instead of r, phi, lam, theta) */
    const void*  r;      /* (B,H,L) dtype retention control r_t            */
    const void*  phi;    /* (B,H,L) dtype phase control phi_t              */
    const float* lam;    /* (H,M) baseline rate, 0 < lambda <= 1           */
    const float* theta;  /* (H,M) baseline frequency                       */
    const void*  u;      /* (B,H,L,M) input b_t = u_t: (re, im) pairs of dtype (complex64 for f32) */
    const float* c;      /* (H,M) complex64 readout                        */
    /* all modes */
    const float* h0;     /* nullable initial state (B,D,N) f32 / (B,H,M) complex64; NULL = 0 */
    /* SSM_REAL_SELECTIVE: step sizes from the input projection, with the
     * discretisation merged into the scan (S3M page, sections 1.1 and 4.1):
     * when delta_bias is non-NULL or delta_softplus is 1, delta holds the
     * projection output z and the scan uses delta = softplus(z + delta_bias[d])
     * (softplus(v) = log(1 + e^v)), or z + delta_bias[d] without softplus;
     * gdelta is then the gradient w.r.t. z.  Both off: delta is used as given. */
    const float* delta_bias;  /* nullable (D) f32 */
    int32_t delta_softplus;   /* 0 or 1 */
    int32_t discretization;   /* SSM_REAL_SELECTIVE: SSM_EULER (0) or SSM_ZOH (ssm_scan_fwd,
                                 ssm_scan_bwd, ssm_scan_fwd_noalloc); other modes: 0 */
    const ssm_layout* layout; /* nullable: strided views (above); NULL = every tensor dense */
    /* SSM_HEAD_SCALAR: channels per head P (16, 32, 48 or 64; channels = H * P).
     * The selective scan with one scalar transition per head, as in the S3M
     * page's matrix form (section 4.1): head h owns channels d = h*P .. h*P+P-1,
     *   a_t = exp(delta[b,h,t] * A[h]),  h_t[d,n] = a_t h_{t-1}[d,n] + delta[b,h,t] x[b,d,t] Bm[b,t,n],
     *   y[b,d,t] = sum_n C[b,t,n] h_t[d,n].
     * Tensors: delta (B,H,L) dtype, x (B,D,L) dtype, A (H) f32, Bm, C (B,L,N)
     * dtype (shared by the channels), h0 (B,D,N); state N in {16, 32, 48, 64};
     * chunk_len 0 or 64.  Forward and backward run the chunked matrix form on
     * the matrix cores (the backward is its exact adjoint, from the 64-step
     * checkpoints or a recompute of them).  Gradients: gdelta
     * (B,H,L) dtype, gx (B,D,L), gA (H) f32, gBm, gC (B,L,N), gh0.  Views:
     * SSM_V_DELTA is (B,H,L), SSM_V_A (H); Bm and C are shared by the channels.
     * No step-size transform, no ZOH.  Other modes: 0. */
    int64_t head_dim;
} ssm_scan_args;

typedef struct {
    void*  y;        /* nullable (B,D,L) dtype (dense: f32)                                */
    float* h_last;   /* nullable h_{L-1}: (B,D,N) f32 / (B,H,M) complex64                  */
    float* ckpt;     /* nullable (B,D,n_chunks,N) f32 / (B,H,n_chunks,M) complex64:
                        ckpt[.., c, :] = state entering chunk c (h_{cT-1}; c = 0 holds h0) */
} ssm_scan_fwd_out;

typedef struct {
    const void*  gy;       /* (B,D,L) dtype (dense: f32): dLoss/dy                        */
    const float* gh_last;  /* nullable dLoss/dh_{L-1}, same layout as h_last; NULL = 0    */
    const float* ckpt;     /* nullable checkpoints from ssm_scan_fwd with the same args;
                              NULL = recomputed into the workspace                         */
} ssm_scan_bwd_in;

/* Gradients of Loss = sum_t <gy_t, y_t> + <gh_last, h_{L-1}>; every pointer
 * nullable.  Complex gradients use the real-pair convention
 * g = dLoss/dRe + i dLoss/dIm (interleaved).  SSM_COMPLEX_DENSE writes ga,
 * gu, gc and gh0 only (the other pointers are ignored). */
typedef struct {
    void*  gdelta;  /* selective (B,D,L) dtype; SSM_HEAD_SCALAR (B,H,L) */
    void*  gx;      /* selective (B,D,L) dtype                  */
    float* gA;      /* selective (D,N) f32 (sum over b and t); SSM_HEAD_SCALAR (H) */
    void*  gBm;     /* selective (B,L,N) dtype (sum over d); (B,D,L,N) for a per-channel Bm */
    float* ga;      /* dense (B,D,L,N) f32; complex dense (B,H,L,M) complex64 */
    float* gb;      /* dense (B,D,L,N) f32                      */
    void*  gC;      /* real (B,L,N) dtype (sum over d); (B,D,L,N) for a per-channel C */
    void*  gu;      /* complex (B,H,L,M) (re, im) pairs of dtype */
    void*  gr;      /* complex (B,H,L) dtype                    */
    void*  gphi;    /* complex (B,H,L) dtype                    */
    float* glam;    /* complex (H,M) f32 (sum over b and t)     */
    float* gtheta;  /* complex (H,M) f32 (sum over b and t)     */
    float* gc;      /* complex (H,M) complex64                  */
    float* gh0;     /* (B,D,N) f32 / (B,H,M) complex64          */
    float* gdelta_bias;  /* selective (D) f32, sum over b and t (bias taken as 0 if delta_bias is NULL) */
} ssm_scan_grads;

/* Arguments of the PD scan.  N = state (1..16), K = dictionary size (1..64).
 * chunk_len: 0 = default 64; only 64 is accepted.  dtype: element type of the
 * streams (logits, d, b, C, and gy, ste_logits, y, gd, gb, gC, glogits of the
 * calls below), SSM_F32 or SSM_BF16; h0, h_last, gh_last, gh0 and checkpoints
 * are always f32, and the recurrence runs in fp32 either way.  batch, heads and
 * length may be 0 (an empty problem: h_last = h0 or 0, gh0 = gh_last or 0,
 * nothing else is touched). */
typedef struct {
    int64_t batch, heads, length, state, dict_size, chunk_len;
    const void*    logits; /* (B,H,L,K) dtype selection scores; may be NULL if sel is given */
    const int32_t* sel;    /* (B,H,L) selected entries; input alternative to logits (used
                              when logits is NULL); values must lie in [0,K) (values outside
                              are a precondition violation: every pass clamps them to
                              [0,K), and pd_scan_fwd reports the clamped selection)        */
    const int32_t* dict;   /* (H,K,N): dict[h,k,j] = row of the one in column j of entry k,
                              values in [0,N) (outside: clamped to [0,N) by every pass)    */
    const void*  d;        /* (B,H,L,N) dtype diagonal d_t                                  */
    const void*  b;        /* (B,H,L,N) dtype input term b_t                                */
    const void*  C;        /* (B,H,L,N) dtype readout C_t                                   */
    const float* h0;       /* nullable (B,H,N) f32                                          */
    int32_t dtype;         /* SSM_F32 or SSM_BF16                                           */
    const ssm_layout* layout;  /* nullable: strided views (roles above); NULL = dense       */
} pd_scan_args;

typedef struct {
    void*    y;       /* nullable (B,H,L) dtype                                         */
    int32_t* sel;     /* nullable (B,H,L): argmax_k logits (lowest index among ties)    */
    float*   h_last;  /* nullable (B,H,N)                                               */
    float*   ckpt;    /* nullable (B,H,n_chunks,N): state entering each chunk           */
} pd_scan_fwd_out;

typedef struct {
    const void*  gy;       /* (B,H,L) dtype                                             */
    const float* gh_last;  /* nullable (B,H,N)                                          */
    const float* ckpt;     /* nullable checkpoints from pd_scan_fwd; NULL = recomputed  */
    const void*  ste_logits; /* (B,H,L,K) dtype selection scores for glogits; required
                                when glogits is wanted, ignored otherwise                */
    float tau;             /* softmax temperature of glogits (> 0, finite)              */
} pd_scan_bwd_in;

/* Gradients with the selection held fixed (argmax is piecewise constant), and
 * optionally the straight-through surrogate gradient of the selection scores
 * (Flash PD-SSM page, gradient propagation: hard argmax in the forward pass, a
 * tempered softmax in its place in the backward pass).  Reading: the
 * transition is sum_k w_k P_k diag(d_t) with w one-hot at the selected entry;
 *   gw[t,k] = dLoss/dw_{t,k} = sum_j lambda_t[dict[h,k,j]] d_t[j] h_{t-1}[j]
 * (lambda_t = dLoss/dh_t of the hard forward) and
 *   glogits[t,k] = (1/tau) s_k (gw[t,k] - sum_i s_i gw[t,i]),
 *   s = softmax(ste_logits[t,:] / tau). */
typedef struct {
    void*  gd;       /* (B,H,L,N) dtype */
    void*  gb;       /* (B,H,L,N) dtype */
    void*  gC;       /* (B,H,L,N) dtype */
    float* gh0;      /* (B,H,N) f32     */
    void*  glogits;  /* (B,H,L,K) dtype surrogate gradient of the scores; NULL = not wanted
                        (with bf16 streams: K <= 16)                                    */
} pd_scan_grads;

/* Workspace size in bytes for operation `op` (SSM_OP_*) with `args`
 * (ssm_scan_args* for the ssm_* scan ops, pd_scan_args* for the pd_* ops, the
 * struct of their own for the convolution and the packed-row ops).
 * Host-only; enqueues nothing.  Errors as for the operation itself. */
int ssm_workspace_bytes(int op, const void* args, size_t* out_bytes);

/* Forward scan: y, h_last and checkpoints (each nullable). */
int ssm_scan_fwd(const ssm_scan_args* args, const ssm_scan_fwd_out* out,
                 void* ws, size_t ws_bytes, void* stream);

/* Allocation-free variant of ssm_scan_fwd, for callers that cannot allocate
 * device memory or pass a workspace (code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc).  Same arguments, outputs,
 * results (bit for bit) and errors as ssm_scan_fwd, with the workspace taken
 * from a static device array of SSM_NOALLOC_SCRATCH_BYTES bytes that every
 * device the library runs on holds until the process ends.  Every diagonal,
 * dense and complex forward fits it (at most about 25 MB: complex mode,
 * M = 64, a few thousand sequences).  The SSM_HEAD_SCALAR forward keeps its
 * chunk states there, 4 * B * D * N * ceil(L / 64) bytes plus
 * 4 * B * H * ceil(L / 64): a need beyond the array is refused with
 * SSM_ERR_WORKSPACE before anything is enqueued.  The call allocates nothing.  Calls that overlap on
 * one device (different streams, or different threads) share the array and
 * race: serialise them.  On first use on a device the call looks up the
 * array's device address (hipGetSymbolAddress). */
#define SSM_NOALLOC_SCRATCH_BYTES (32 * 1024 * 1024)
int ssm_scan_fwd_noalloc(const ssm_scan_args* args, const ssm_scan_fwd_out* out, void* stream);

/* Exact backward of ssm_scan_fwd by tiled recompute from the checkpoints and a
 * reverse adjoint scan lambda_t = C_t gy_t + A_{t+1}^T lambda_{t+1}. */
int ssm_scan_bwd(const ssm_scan_args* args, const ssm_scan_bwd_in* in,
                 const ssm_scan_grads* grads, void* ws, size_t ws_bytes, void* stream);

/* Impulse-response sensitivity of a selective real scan (PGF page, abstract:
 * sensitivity analysis on a 128,000-step impulse-response benchmark):
 *   s[b,d,t] = d y[b,d,t_out] / d x[b,d,t]
 *            = delta_t sum_n Bm[b,t,n] C[b,t_out,n] exp(A[d,n] sum_{s=t+1..t_out} delta_s)
 * for t <= t_out and 0 for t > t_out, by reverse costate evolution in tiles
 * (workspace O(n_chunks), no checkpoints).  t_out in [0,L); -1 means L-1.
 * y (nullable, (B,D,L) dtype) additionally receives the forward output.
 * s is (B,D,L) dtype.  SSM_REAL_SELECTIVE only. */
int ssm_impulse_sensitivity(const ssm_scan_args* args, int64_t t_out, void* y, void* s,
                            void* ws, size_t ws_bytes, void* stream);

/* Forward-mode (real-time recurrent) gradients of the complex mode w.r.t. its
 * per-mode parameters (SPARC page, abstract: exact structured real-time
 * recurrent learning for online credit assignment).  Carries the state
 * sensitivities S^lambda_t = dh_t/dlambda and S^theta_t = dh_t/dtheta forward
 * with the state:
 *   S^lambda_t = a_t S^lambda_{t-1} + (r_t / lambda) a_t h_{t-1},
 *   S^theta_t  = a_t S^theta_{t-1}  + i phi_t a_t h_{t-1}   (S_{-1} = 0),
 * and accumulates, for Loss = sum_t gy_t y_t + <gh_last, h_{L-1}>,
 *   glam[h,m]   = sum_{b,t} gy_t Re(c_m S^lambda_t) + <gh_last, S^lambda_{L-1}>,
 *   gtheta[h,m] = the same with S^theta.
 * The results equal ssm_scan_bwd's glam and gtheta up to rounding; no
 * checkpoints or reverse pass.  args: mode SSM_COMPLEX_SHARED (the
 * ssm_scan_fwd argument rules).  gy: (B,H,L) dtype, required.  gh_last:
 * nullable (B,H,M) complex64, real-pair convention.  y: nullable (B,H,L) dtype,
 * receives the forward output.  glam, gtheta: nullable (H,M) f32, overwritten.
 * Segments of the sequence run in parallel (workspace from
 * ssm_workspace_bytes(SSM_OP_COMPLEX_RTRL, ...)).  Errors as for ssm_scan_fwd;
 * SSM_ERR_UNSUPPORTED for another mode. */
int ssm_complex_rtrl(const ssm_scan_args* args, const void* gy, const float* gh_last, void* y,
                     float* glam, float* gtheta, void* ws, size_t ws_bytes, void* stream);

/* Sensitivity of one output of a selective real scan to the inputs and to the
 * step sizes (PGF page, abstract: sensitivities of the SSM dynamics), with the
 * reverse costate mu_t = C[b,t_out,:] prod_{s=t+1..t_out} a_s in closed form:
 *   s_x[b,d,t]     = d y[b,d,t_out] / d x[b,d,t]     = delta_t sum_n Bm[b,t,n] mu_t[n],
 *   s_delta[b,d,t] = d y[b,d,t_out] / d delta[b,d,t]
 *                  = sum_n mu_t[n] (A[d,n] a_t[n] h_{t-1}[n] + x_t Bm[b,t,n]),
 * t <= t_out, 0 after; h_{t-1} are the forward states (from h0).  With N = 16,
 * the Euler term, shared Bm and C and a sequence the call cuts into segments
 * the forward's main pass forms both sensitivities from the states it re-runs
 * (workspace as for ssm_impulse_sensitivity); otherwise a separate pass
 * recomputes the states per tile from checkpoints the call writes into its
 * workspace (O(n_chunks * N) per sequence).  t_out in [0,L); -1 means
 * L-1.  y, s_x nullable, s_delta required; all (B,D,L) dtype.  With delta_bias or
 * delta_softplus set, s_delta is the sensitivity to the projection output z.
 * SSM_REAL_SELECTIVE only; workspace from ssm_workspace_bytes(SSM_OP_OUTPUT_SENS, ...). */
int ssm_output_sensitivity(const ssm_scan_args* args, int64_t t_out, void* y, void* s_x, void* s_delta,
                           void* ws, size_t ws_bytes, void* stream);

/* Rows of the input Jacobian of the selective scan (PGF page, abstract:
 * sensitivities of outputs to inputs by reverse costate evolution, O(chunk)
 * working memory).  For the R consecutive output steps tau_r = t_out0 + r:
 *   s[r,b,d,t] = d y[b,d,tau_r] / d x[b,d,t]
 *              = delta_t sum_n B_t[n] C_{tau_r}[n] prod_{t < u <= tau_r} a_u[n]  (t <= tau_r), 0 after,
 * i.e. per channel the (R x L) block of the Jacobian.  One call costs one
 * exp per (t, n) for all R rows: the product is split at t_out0 into the
 * costate of row t_out0 and a per-row weight.  s[r] equals
 * ssm_impulse_sensitivity's s at t_out = tau_r up to rounding.
 * args: mode SSM_REAL_SELECTIVE, chunk_len 0 or 64 (64-step tiles); the step
 * transform (delta_bias, delta_softplus) applies as in ssm_scan_fwd, and s is
 * then still the sensitivity to x.  rows in [1, 16]; 0 <= t_out0 and
 * t_out0 + rows <= L.  s: (rows,B,D,L) dtype, required, every element written.
 * Workspace from ssm_workspace_bytes(SSM_OP_SENS_ROWS, ...) (sized for 16
 * rows).  Errors: SSM_ERR_SHAPE for rows or t_out0 out of range,
 * SSM_ERR_UNSUPPORTED for another mode or chunk_len, otherwise as for
 * ssm_scan_fwd. */
int ssm_sensitivity_rows(const ssm_scan_args* args, int64_t t_out0, int32_t rows, void* s,
                         void* ws, size_t ws_bytes, void* stream);

/* PD forward: selection (argmax of logits unless sel is given), scan, readout. */
int pd_scan_fwd(const pd_scan_args* args, const pd_scan_fwd_out* out,
                void* ws, size_t ws_bytes, void* stream);

/* PD backward with the selection from args->sel (or recomputed from logits). */
int pd_scan_bwd(const pd_scan_args* args, const pd_scan_bwd_in* in,
                const pd_scan_grads* grads, void* ws, size_t ws_bytes, void* stream);

/*
 * Short causal convolution (training form).  The depthwise convolution along
 * the sequence in front of a selective scan, with the bias and activation of
 * its layer.  With e = the W-1 inputs before step 0 followed by x,
 *   p[b,d,t] = bias[d] + sum_{k<W} w[d,k] e[b,d,t+k],
 *   y = p, or p * sigmoid(p) with silu = 1,
 *   last[b,d,:] = e[b,d,L..L+W-2]   (what a following segment takes as init).
 * The backward recomputes p from its input.  The input is x, or x's 8-bit
 * checkpoint (below) in place of x: the values it stands for then are the
 * input, widened to float32.
 * Roles of `layout`: SSM_V_X, SSM_V_GY inputs, SSM_V_Y, SSM_V_GX outputs, all
 * (B,D,L).  An 8-bit checkpoint is dense.  batch, channels and length may be 0:
 * tensors with no elements are not touched; with length 0 last is init (or 0)
 * and ginit is glast (or 0); gw and gbias are 0.
 * Errors: SSM_ERR_UNSUPPORTED for a width other than 2, 3 or 4; SSM_ERR_SHAPE
 * where batch * length reaches 2^33.
 */
typedef struct {
    int32_t dtype;           /* of x, y, init, last and their gradients: SSM_F32 or SSM_BF16 */
    int32_t silu;            /* 0 or 1                                                       */
    int64_t batch, channels, length, width;
    const void*   x;         /* (B,D,L) dtype; exactly one of x and x8 is given              */
    const int8_t* x8;        /* (B,D,L) 8-bit checkpoint of the input                        */
    const float*  x8_scale;  /* (B,D,ceil(L/SSM_CKPT8_BLOCK)), with x8                       */
    const float*  w;         /* (D,W) f32, w[d,W-1] for the step itself                      */
    const float*  bias;      /* nullable (D) f32                                             */
    const void*   init;      /* nullable (B,D,W-1) dtype: the inputs before step 0 (0)       */
    const ssm_layout* layout;
} ssm_conv_args;

typedef struct {
    void*   y;         /* nullable (B,D,L) dtype                                              */
    void*   last;      /* nullable (B,D,W-1) dtype                                            */
    int8_t* x8;        /* nullable (B,D,L): 8-bit checkpoint of x, written in the same pass
                          (needs args->x); together with x8_scale                            */
    float*  x8_scale;
} ssm_conv_fwd_out;

typedef struct {
    void*  gx;         /* nullable (B,D,L) dtype                                              */
    float* gw;         /* nullable (D,W)                                                      */
    float* gbias;      /* nullable (D)                                                        */
    void*  ginit;      /* nullable (B,D,W-1) dtype                                            */
} ssm_conv_grads;

int ssm_conv_fwd(const ssm_conv_args* args, const ssm_conv_fwd_out* out, void* stream);
/* Gradients of Loss = sum <gy, y> + <glast, last> (gy (B,D,L), glast nullable (B,D,W-1), dtype). */
int ssm_conv_bwd(const ssm_conv_args* args, const void* gy, const void* glast, const ssm_conv_grads* grads,
                 void* ws, size_t ws_bytes, void* stream);

/*
 * 8-bit activation checkpoints.  A stream (B,D,L) kept for the backward pass in
 * one signed byte an element and one float32 scale for every SSM_CKPT8_BLOCK
 * steps of a row, in place of its 2 or 4 bytes an element.  Per block, in
 * float32 (each operation rounded to nearest even):
 *   amax = max |x|,  scale = amax / 127,  q = rint(x * (127 / amax)),
 * with a scale of at most 0x1.020406p+121, the largest whose product with 127 is
 * finite (only the largest float's exceeds it).  The block stands for q * scale:
 * off by at most (1/2 + 2^-15) scale, as the reciprocal step, the product, the
 * scale and the value are each off by up to 2^-24 of at most 127 scales.  A block
 * whose amax is below 2^-100 is all zeros (scale 0); a block that holds a NaN or
 * an infinity stands for NaN throughout.  ssm_conv_fwd writes it in the pass that
 * reads x; ssm_conv_fwd and ssm_conv_bwd take it in place of x; ssm_ckpt8_unpack
 * rounds it to a stream that ssm_scan_bwd takes.
 */
#define SSM_CKPT8_BLOCK 64
typedef struct {
    int32_t dtype;             /* of the stream                                              */
    int64_t batch, channels, length;
    const ssm_layout* layout;  /* ssm_ckpt8_pack: role SSM_V_X; ssm_ckpt8_unpack: role SSM_V_Y */
} ssm_ckpt8_args;
int ssm_ckpt8_pack(const ssm_ckpt8_args* args, const void* x, int8_t* x8, float* x8_scale, void* stream);
int ssm_ckpt8_unpack(const ssm_ckpt8_args* args, const int8_t* x8, const float* x8_scale, void* y, void* stream);

/*
 * Serving forms: the convolution and the selective scan over packed rows.  The
 * tokens of all sequences of a call are rows of one matrix, as the projections
 * around them read and write them: sequence s owns rows seq_start[s] ..
 * seq_start[s+1]-1 (ascending), in order.  seq_start NULL is the step form:
 * one row a sequence (tokens == sequences).  What a sequence carries from call to
 * call lies in a pool of slots; sequence s begins with the state in slot[s] (or
 * with zeros where fresh[s] is not 0: its slot is not read) and leaves its
 * state there.
 *  - A sequence with no rows leaves its slot as it was, fresh or not.
 *  - slot[s] outside [0, slots) marks an empty place of a padded batch: its rows
 *    of y and every slot stay as they were.  So does a sequence whose slot an
 *    earlier sequence of the call has (each slot has one sequence a call), and
 *    rows that no sequence owns.
 *  - seq_start, slot and fresh are device memory and are not checked on the
 *    host: values out of range are never followed out of the buffers, but rows
 *    of sequences that overlap or descend have unspecified results.
 *  - Rows: row strides in elements; the row itself is contiguous.  Inputs may be
 *    slices of wider rows (any stride from 0 to 2^40 - 1; to 2^26 - 1 in
 *    ssm_tokens_scan with seq_start), y's stride is at least its row.  The
 *    stride of a single row is not used.
 *  - pool_stride: elements from one slot to the next, at least a slot's own.
 *  - pool is read and written; it must not overlap any other buffer.
 */
typedef struct {
    int32_t dtype;             /* of x, y and the pool                                       */
    int32_t silu;              /* 0 or 1                                                     */
    int64_t tokens, channels, width, sequences, slots;
    const void*  x;            /* (T,D) dtype                                                */
    const float* w;            /* (D,W) f32, width 2, 3 or 4                                 */
    const float* bias;         /* nullable (D) f32                                           */
    const int32_t* seq_start;  /* nullable (sequences + 1)                                   */
    const int32_t* slot;       /* nullable (sequences); NULL: sequence s has slot s          */
    const uint8_t* fresh;      /* nullable (sequences); NULL: every sequence has a state     */
    void* pool;                /* (slots,D,W-1) dtype: the last W-1 inputs, oldest first     */
    void* y;                   /* (T,D) dtype                                                */
    int64_t x_stride, y_stride, pool_stride;
} ssm_tokens_conv_args;

/* y[t] = act(bias + sum_k w[:,k] e[t+k]), as ssm_conv_fwd with init = the slot and last = the slot. */
int ssm_tokens_conv(const ssm_tokens_conv_args* args, void* stream);

typedef struct {
    int32_t dtype;             /* of delta, x, Bm, C, z and y                                */
    int32_t delta_softplus;    /* as in ssm_scan_args                                        */
    int64_t tokens, channels, state, sequences, slots;   /* state N in 1..16                 */
    const void*  delta;        /* (T,D)                                                      */
    const void*  x;            /* (T,D)                                                      */
    const float* A;            /* (D,N) f32 (A < 0)                                          */
    const void*  Bm;           /* (T,N)                                                      */
    const void*  C;            /* (T,N)                                                      */
    const float* delta_bias;   /* nullable (D) f32                                           */
    const float* skip;         /* nullable (D) f32                                           */
    const void*  z;            /* nullable (T,D) gate                                        */
    const int32_t* seq_start;  /* as above                                                   */
    const int32_t* slot;
    const uint8_t* fresh;
    float* pool;               /* (slots,D,N) f32: the state h                               */
    void*  y;                  /* (T,D)                                                      */
    int64_t delta_stride, x_stride, Bm_stride, C_stride, z_stride, y_stride, pool_stride;
} ssm_tokens_scan_args;

/* The selective scan (SSM_REAL_SELECTIVE, Euler input term) with its layer's skip and gate:
 *   h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,
 *   y_t = (C_t . h_t + skip x_t) * z_t sigmoid(z_t)     (skip, z: where given).
 * The states are float32.  The workspace (SSM_OP_TOKENS_SCAN) holds the states that cross from one
 * range of rows to the next; the step form needs none.  Ranges are joined by exp(A sum delta), several
 * of them at once, which has to be a finite float32: a sequence that grows by more than e^88 over a
 * call (A delta > 0) is out of reach of the packed form, though not of single steps. */
int ssm_tokens_scan(const ssm_tokens_scan_args* args, void* ws, size_t ws_bytes, void* stream);

/*
 * Gated linear recurrence.  A state for each channel whose decay and input are
 * opened by gates of their own (the scan without a state expansion):
 *   rho = sigmoid(r + r_bias),  iota = sigmoid(i + i_bias),
 *   q = power * softplus(lam) * rho,  a = exp(-q),
 *   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) iota_t x_t,   y_t = h_t,   h_{-1} = h0.
 * The states and everything that forms them are float32.  Where a gate's input
 * lies below about -87 its sigmoid is 0.  power * softplus(lam) is to stay below
 * 2^64 and the states below 2^60: past them products of float32 overflow.
 * Strides are in elements: batch, then
 * channel; steps are contiguous; 0 (broadcast) for inputs only, whose gradients
 * come back for every position.  batch, channels and length may be 0 (h_last is
 * then h0 or 0, gh0 is gh_last or 0, parameter gradients are 0).  SSM_ERR_SHAPE for
 * a batch of more than 65535, as in the other calls over streams, for 2^24 channels,
 * 2^31 - 2^16 steps or 2^28 - 64 rows (batch times channels) and more.
 */
#define SSM_GATED_CHUNK 128
typedef struct {
    int32_t dtype;           /* of x, r, i, y and their gradients: SSM_F32 or SSM_BF16       */
    float   power;           /* > 0: the decay of a wide open gate is exp(-power softplus(lam)) */
    int64_t batch, channels, length;
    const void*  x;          /* (B,D,L) input                                                */
    const void*  r;          /* (B,D,L) decay gate, before its sigmoid                       */
    const void*  i;          /* (B,D,L) input gate, before its sigmoid                       */
    const float* lam;        /* (D) f32                                                      */
    const float* r_bias;     /* nullable (D) f32                                             */
    const float* i_bias;     /* nullable (D) f32                                             */
    const float* h0;         /* nullable (B,D) f32                                           */
    int64_t x_stride[2], r_stride[2], i_stride[2];
} ssm_gated_args;

typedef struct {
    void*  y;                /* nullable (B,D,L) dtype                                       */
    float* h_last;           /* nullable (B,D)                                               */
    float* ckpt;             /* nullable (B,D,ceil(L/SSM_GATED_CHUNK)): the state that every
                                SSM_GATED_CHUNK steps begin with, for the backward           */
    int64_t y_stride[2];
} ssm_gated_fwd_out;

typedef struct {
    const void*  gy;         /* (B,D,L) dtype                                                */
    const float* gh_last;    /* nullable (B,D)                                               */
    const float* ckpt;       /* nullable: formed again in the workspace (the same bits)      */
    int64_t gy_stride[2];
} ssm_gated_bwd_in;

typedef struct {
    void  *gx, *gr, *gi;     /* nullable (B,D,L) dtype                                       */
    float *glam, *gr_bias, *gi_bias;   /* nullable (D)                                       */
    float* gh0;              /* nullable (B,D)                                               */
    int64_t gx_stride[2], gr_stride[2], gi_stride[2];
} ssm_gated_grads;

int ssm_gated_fwd(const ssm_gated_args* args, const ssm_gated_fwd_out* out, void* stream);
/* Gradients of Loss = sum <gy, y> + <gh_last, h_last>. */
int ssm_gated_bwd(const ssm_gated_args* args, const ssm_gated_bwd_in* in, const ssm_gated_grads* grads,
                  void* ws, size_t ws_bytes, void* stream);

/* The gated recurrence over packed rows, with sequences, pool and rows as in ssm_tokens_conv above.  The workspace
 * (SSM_OP_TOKENS_GATED) holds what one tile of rows hands on to the next; the step form needs none.  Of calls that
 * overlap in time each needs a workspace of its own: in one that another call writes to meanwhile the wait for the tile
 * before is bounded and ends in NaN, and no access leaves the buffers. */
typedef struct {
    int32_t dtype;             /* of x, r, i and y                                           */
    float   power;
    int64_t tokens, channels, sequences, slots;
    const void*  x;            /* (T,D)                                                      */
    const void*  r;            /* (T,D)                                                      */
    const void*  i;            /* (T,D)                                                      */
    const float* lam;          /* (D)                                                        */
    const float* r_bias;       /* nullable (D)                                               */
    const float* i_bias;       /* nullable (D)                                               */
    const int32_t* seq_start;
    const int32_t* slot;
    const uint8_t* fresh;
    float* pool;               /* (slots,D) f32: the state h                                 */
    void*  y;                  /* (T,D)                                                      */
    int64_t x_stride, r_stride, i_stride, y_stride, pool_stride;
} ssm_tokens_gated_args;
int ssm_tokens_gated(const ssm_tokens_gated_args* args, void* ws, size_t ws_bytes, void* stream);

/*
 * Group norm of rows, channels last, with activation and gate.  The channels of
 * a row are `groups` groups of consecutive ones; statistics are those of one
 * group of one row, so none crosses from token to token:
 *   xh = (x - mean) / sqrt(var + eps),  v = xh w + bias,
 *   u = v, or v sigmoid(v) with silu = 1,   y = u, or u z sigmoid(z) with z.
 * The backward forms the statistics again from x.  Row strides as in the packed
 * forms above.  The statistics are float32: the values of a group are to stay below
 * 2^114, their differences to the mean below 2^57, and var + eps is to be at least
 * 2^-126 (with eps = 0 a group without spread has no value: NaN).  rows may be 0
 * (gw, gbias are then 0).  Errors: SSM_ERR_SHAPE where groups does not divide channels, SSM_ERR_UNSUPPORTED for groups of more than 8192
 * channels.
 */
typedef struct {
    int32_t dtype;             /* of x, z, y and their gradients                             */
    int32_t silu;              /* 0 or 1                                                     */
    int64_t rows, channels, groups;
    const void*  x;            /* (T,C)                                                      */
    const void*  z;            /* nullable (T,C) gate                                        */
    const float* w;            /* nullable (C) f32 (1)                                       */
    const float* bias;         /* nullable (C) f32 (0)                                       */
    int64_t x_stride, z_stride;
    float eps;                 /* >= 0                                                       */
} ssm_group_norm_args;

typedef struct {
    void  *gx, *gz;            /* nullable (T,C) dtype                                       */
    float *gw, *gbias;         /* nullable (C)                                               */
    int64_t gx_stride, gz_stride;
} ssm_group_norm_grads;

int ssm_group_norm_fwd(const ssm_group_norm_args* args, void* y, int64_t y_stride, void* stream);
int ssm_group_norm_bwd(const ssm_group_norm_args* args, const void* gy, int64_t gy_stride,
                       const ssm_group_norm_grads* grads, void* ws, size_t ws_bytes, void* stream);

/*
 * Products in 8-bit integers.  ssm_tokens_pack8 holds each row in signed bytes
 * and one float32 scale, in the format of the 8-bit checkpoints above with a row
 * in place of a block of steps.  ssm_tokens_mm8 multiplies such rows with weights
 * that have a scale for each output:
 *   y[t][n] = x8_scale[t] w8_scale[n] sum_k x8[t][k] w8[n][k] + bias[n].
 * The sums are whole numbers in 32 bits (inputs below 2^17: they cannot overflow),
 * rounded once to float32 before the scales, whose product is formed first: where that leaves float32's range y is
 * infinite or NaN, and where it falls below it bias.  Rows may have any stride from 0 (inputs) or their own width
 * (outputs) to 2^40 - 1.  With no inputs y is bias (where the scales' product is finite).  SSM_ERR_SHAPE for 2^17 inputs, 2^24 tokens or 2^26 outputs and more.
 */
typedef struct {
    int32_t dtype;             /* of x                                                       */
    int64_t tokens, channels;
    const void* x;             /* (T,K)                                                      */
    int8_t* x8;                /* (T,K)                                                      */
    float*  x8_scale;          /* (T)                                                        */
    int64_t x_stride, x8_stride;
} ssm_tokens_pack8_args;
int ssm_tokens_pack8(const ssm_tokens_pack8_args* args, void* stream);

typedef struct {
    int32_t dtype;             /* of y                                                       */
    int64_t tokens, inputs, outputs;
    const int8_t* x8;          /* (T,K)                                                      */
    const float*  x8_scale;    /* (T)                                                        */
    const int8_t* w8;          /* (N,K)                                                      */
    const float*  w8_scale;    /* (N)                                                        */
    const float*  bias;        /* nullable (N)                                               */
    void* y;                   /* (T,N)                                                      */
    int64_t x8_stride, w8_stride, y_stride;
} ssm_tokens_mm8_args;
int ssm_tokens_mm8(const ssm_tokens_mm8_args* args, void* stream);

/* Diagnostics: per-kernel timing with HIP events.  After ssm_profile_begin(n)
 * every kernel the entry points enqueue from this thread is bracketed by two
 * HIP events recorded on the same stream (at most n kernels; later ones are
 * not recorded).  ssm_profile_end waits for the last event, writes up to
 * `capacity` per-kernel durations in milliseconds and static kernel names,
 * sets *n_launches to the number recorded, and stops recording.  The events
 * are created by the library and kept for reuse until the process ends. */
int ssm_profile_begin(int max_launches);
int ssm_profile_end(int* n_launches, float* ms, const char** names, int capacity);

/* Diagnostics: issue rate of one VALU instruction class, measured on the
 * device (the arithmetic ceiling the scan kernels' roofline is taken against).
 * Launches `waves` one-wave workgroups (waves / (4 x compute units) waves per
 * SIMD), every lane running `chains` (4 or 8) independent dependency chains of
 * iters x 8 instructions of class `kind`: 0 v_fma_f32 (VOP3), 1 v_mul_f32,
 * 2 v_exp_f32, 3 v_fmac_f32 with a DPP row_shr source (4 chains only),
 * 4 v_permlane32_swap, 5 v_permlane16_swap, 6 v_add_f32, 7 v_fmac_f32 (VOP2,
 * accumulating into its addend; 8 chains only).  Times the launch
 * with two HIP events on `stream`, waits for it, and writes lane operations
 * per second (64 x waves x instructions per lane / seconds).  `sink` is a
 * device buffer of waves x 64 floats that is never written in practice (it
 * keeps the chains live).  Synchronises with the stream. */
int ssm_roof_probe(int kind, int chains, int waves, int iters, float* sink, double* lane_ops_per_s,
                   void* stream);

const char* ssm_status_string(int status);   /* static string for a status code */
const char* ssm_last_error_detail(void);     /* thread-local detail of the last error */
int ssm_abi_version(void);                   /* SSM_ABI_VERSION of the built library */

#ifdef __cplusplus
}
#endif

#endif /* SSMSCAN_H */
