/*
 * ssm.h -- C ABI of the MI355X (gfx950) selective-scan library.
 *
 * The library computes the Mamba-1 selective state-space layer (S6) on one
 * GPU with hand-written HIP kernels:
 *   - ssm_selective_scan_fwd: the whole-sequence scan (prefill), optionally
 *     with a fused depthwise causal conv1d + SiLU prologue and a final-state
 *     output;
 *   - ssm_state_update: one recurrent (decode) step on a resident state;
 *   - ssm_causal_conv1d_silu: the conv prologue on its own;
 *   - ssm_selective_scan_bwd: the gradients of the scan (training);
 *   - ssm_block_fwd: a whole Mamba block around the scan (with a plan);
 *   - ssm_ssd_fwd: the SSD (Mamba-2) layer, chunked on the matrix cores;
 *   - ssm_ssd_step: one decode step of that layer on a resident state;
 *   - ssm_gated_scan_fwd, _bwd, _step: a gated linear recurrence, whose decay
 *     is itself an input, with its gradients and its decode step;
 *   - ssm_add_rmsnorm_fwd, _bwd: the residual sum and the RMSNorm between two
 *     blocks in one pass, with its gradients;
 *   - ssm_gated_rmsnorm_fwd, _bwd: the RMSNorm of a gated layer output over
 *     groups of channels, with its gradients;
 *   - ssm_gated_delta_fwd, _bwd, _step: the gated delta rule, a matrix state
 *     per head that forgets what it holds for a key before it takes up the
 *     key's new value, with its gradients and its decode step;
 *   - ssm_add_rmsnorm_fp8, ssm_quantize_fp8, ssm_matmul_fp8: the norm between
 *     two blocks with its output in 8 bits, the quantising of any matrix, and
 *     the product of two such matrices.
 *
 * The operations are defined on these pages (cited by title and section):
 *   [P1] "Mamba: Linear-Time Sequence Modeling with Selective State Spaces"
 *        (paper summary page): sec. 4a (Mamba block: Conv1d -> SiLU -> SSM,
 *        output x SiLU(gate)), sec. 4b eq. (1a)/(1b), eq. (4) (ZOH),
 *        eq. (2a)/(2b) (recurrence), Algorithm 2 (S6 shapes), sec. 4d (A
 *        diagonal and real, N = 16, E = 2).
 *   [P2] "2. Mamba 상세" (EulerStack mixer tutorial): d_conv: 4 and the
 *        ssm_state kept between inference steps.
 *   [P4] "14.1 SSM(State Space Models)과 Mamba 아키텍처의 부상": sec. 3.1
 *        (y = C h + D x, the D skip), sec. 3.2 (ZOH), sec. 4.1 (Delta =
 *        softplus(parameter + projection)), sec. 5.1/5.2 (SSD, chunks).
 *
 * Conventions common to every entry point
 *   - Every tensor pointer is a DEVICE pointer into memory the caller owns
 *     (e.g. a torch tensor's data_ptr()).  The library allocates no device
 *     memory of its own, keeps no state between calls and never frees caller
 *     memory; the one exception is the block plan (ssm_block_plan_create),
 *     which holds a hipBLASLt handle until ssm_block_plan_destroy.
 *   - Tensors are dense and row-major with the last index fastest; element
 *     strides are implied by the shapes.  Pointers must be aligned to their
 *     element size (2 bytes for bf16, 4 for fp32).
 *   - `stream` is a hipStream_t passed as void*; NULL means the default
 *     stream.  Calls are asynchronous with respect to the host: they enqueue
 *     kernels on `stream` and return.  Faults inside a kernel surface at the
 *     caller's next synchronisation on that stream.
 *   - Argument checking is complete before any HIP call: on an error the
 *     function returns a status other than SSM_OK, enqueues nothing and
 *     writes nothing.  ssm_last_error_message() then describes the failure
 *     (per calling thread).  After launching, a launch failure reported by
 *     the runtime returns SSM_ERR_HIP.
 *   - No C++ exception crosses this interface.  All entry points are
 *     re-entrant and thread-safe; calls that write the same output memory
 *     concurrently race, as with any kernel.
 *   - Sizes: a batch or sequence length of 0 is a valid empty call and
 *     returns SSM_OK without launching (the final state, if requested, is
 *     then a copy of h0, or zeros).  Negative sizes give SSM_ERR_BAD_SHAPE.
 *   - Arithmetic is fp32 throughout, on fp32 or bf16 inputs; bf16 results
 *     are rounded to nearest even.  State, A, D, bias and conv weights are
 *     always fp32.
 */
#ifndef SSM_MI355X_H
#define SSM_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_ABI_VERSION 12
#define SSM_MAX_DSTATE 16 /* largest N the kernels hold in registers */
#define SSM_MAX_CONV_K 4  /* largest conv1d kernel width */

typedef enum ssm_status {
    SSM_OK = 0,
    SSM_ERR_NULL_ARG = 1,    /* a required pointer is NULL                   */
    SSM_ERR_BAD_SHAPE = 2,   /* a negative or inconsistent size              */
    SSM_ERR_BAD_DTYPE = 3,   /* io_dtype is not one of ssm_dtype_t           */
    SSM_ERR_UNSUPPORTED = 4, /* N or K above the compiled maximum, bad flags */
    SSM_ERR_ALIAS = 5,       /* an output overlaps an input or another output*/
    SSM_ERR_WORKSPACE = 6,   /* workspace missing, too small or misaligned  */
    SSM_ERR_HIP = 7,         /* the HIP runtime reported an error            */
    SSM_ERR_ALIGN = 8        /* a pointer is not aligned to its element size */
} ssm_status_t;

typedef enum ssm_dtype {
    SSM_F32 = 0, /* IEEE binary32 */
    SSM_BF16 = 1 /* bfloat16 (upper half of a binary32) */
} ssm_dtype_t;

/*
 * Arguments of the selective scan, [P1] Algorithm 2 with the gate of sec. 4a
 * and the skip of [P4] sec. 3.1.  Per batch b, channel d and state index n:
 *
 *   u[b,t,d]   = x[b,t,d], or, when conv_w != NULL, the fused prologue
 *                silu(sum_{k<K} conv_w[d,k] x[b,t-(K-1)+k,d] + conv_b[d])
 *                ([P1] sec. 4a, [P2] d_conv), where x at negative times
 *                comes from conv_state_in, or is 0 without it.
 *   dt[b,t,d]  = delta[b,t,d], or softplus(delta[b,t,d] + delta_bias[d])
 *                when delta_softplus != 0 ([P1] Algorithm 2).
 *   Abar       = exp(dt A[d,n])                                 (eq. 4)
 *   Bbar       = (dt A[d,n])^-1 (exp(dt A[d,n]) - 1) dt Bm[b,t,n]  (eq. 4),
 *                = dt Bm[b,t,n] where A[d,n] == 0 (the limit)
 *   h[b,d,n]   = Abar h[b,d,n] + Bbar u[b,t,d], from h0 (or 0)  (eq. 2a)
 *   y[b,t,d]   = (sum_n Cm[b,t,n] h[b,d,n] + Dskip[d] u[b,t,d])
 *                * silu(z[b,t,d])                               (eq. 2b, 4a)
 *   h_final    = h after the last time step.
 *
 * Conv state (the prefill -> decode handoff of the conv window, kept between
 * inference calls like the SSM state of [P2]): a (B, K-1, D) io_dtype tensor
 * holding, for every batch row and channel, the K-1 most recent inputs x,
 * oldest first (row k is time -(K-1)+k relative to the next token).
 * conv_state_in gives x at times -(K-1)..-1 of this call; conv_state_out
 * receives x at times L-(K-1)..L-1 (from conv_state_in, or 0, where that time
 * is negative), which is the window ssm_state_update expects for the next
 * token.  Both are raw copies of the inputs, bit for bit.
 */
typedef struct ssm_scan_args {
    int64_t batch;          /* B >= 0                                         */
    int64_t seqlen;         /* L >= 0                                         */
    int64_t dim;            /* D >= 1 (channels, E*d_model in the block)      */
    int64_t dstate;         /* N, 1 <= N <= SSM_MAX_DSTATE                    */
    int32_t io_dtype;       /* ssm_dtype_t of x, delta, Bm, Cm, z and y       */
    int32_t delta_softplus; /* 0: delta is the step; 1: softplus(delta+bias) */
    int64_t conv_k;         /* 0: no prologue; 1..SSM_MAX_CONV_K: fused conv  */
    const void *x;          /* (B,L,D) io_dtype, required                     */
    const void *delta;      /* (B,L,D) io_dtype, required                     */
    const void *Bm;         /* (B,L,N) io_dtype, required; shared by channels */
    const void *Cm;         /* (B,L,N) io_dtype, required; shared by channels */
    const void *z;          /* (B,L,D) io_dtype gate, or NULL (no gate)       */
    const float *A;         /* (D,N) fp32, required; any finite value         */
    const float *Dskip;     /* (D) fp32, or NULL (no skip term)               */
    const float *delta_bias;/* (D) fp32, or NULL (= 0); used with softplus    */
    const float *conv_w;    /* (D,conv_k) fp32; required iff conv_k > 0       */
    const float *conv_b;    /* (D) fp32, or NULL (= 0)                        */
    const float *h0;        /* (B,D,N) fp32 initial state, or NULL (= 0)      */
    void *y;                /* (B,L,D) io_dtype output; required              */
    float *h_final;         /* (B,D,N) fp32 output, or NULL (not written)     */
    void *workspace;        /* device scratch of workspace_bytes, 256-aligned */
    size_t workspace_bytes; /* >= ssm_selective_scan_workspace_size(args)     */
    const void *conv_state_in; /* (B,K-1,D) io_dtype, or NULL (= 0); only with conv_k > 0 */
    void *conv_state_out;   /* (B,K-1,D) io_dtype output, or NULL; only with conv_k > 0;
                               may be exactly conv_state_in (updated in place)    */
    float *checkpoints;     /* (ceil(L/SSM_SCAN_BLOCK), B, D, SSM_MAX_DSTATE) fp32
                               output, or NULL: see below                         */
} ssm_scan_args_t;

/*
 * Checkpoints (for training: the forward hands them to the backward, which
 * then does not recompute them).  checkpoints[j][b][d][n] is the state
 * h[b,d,n] entering time step SSM_SCAN_BLOCK * j (the state after step
 * SSM_SCAN_BLOCK * j - 1, or h0 for j = 0), for n < N; entries n >= N are 0.
 * Where the scan splits a long sequence into segments run at the same time,
 * each segment but the first is scanned from a zero state and its first
 * blocks again from its true entering state, up to the block after which
 * exp(A times the segment's sum of dt) is below 2^-160 for every entry; the
 * states from there on are the zero-start ones, which differ from the true
 * states by that factor times the entering state.  Must not overlap any
 * other argument or the workspace.
 */
#define SSM_SCAN_BLOCK 16

/*
 * Bytes of device workspace ssm_selective_scan_fwd needs for these sizes and
 * options (0 when none is needed; only the size fields, io_dtype and the
 * optional-output flags are read, pointers may be NULL).  The workspace holds
 * per-chunk carries of the split sequence; its contents on entry do not
 * matter and on return are unspecified.  Two calls in flight at once need
 * two workspaces.  Returns (size_t)-1 for invalid sizes.
 */
size_t ssm_selective_scan_workspace_size(const ssm_scan_args_t *args);

/*
 * Enqueue the selective scan described above on `stream`.
 * y must not overlap any input; h_final must not overlap any input or y.
 * h0 may be NULL; when given it may not overlap h_final (copy first to scan
 * in place).  conv_state_out must not overlap any other argument except that
 * it may be the same tensor as conv_state_in.  Returns SSM_OK or an error
 * status (see the conventions).
 */
ssm_status_t ssm_selective_scan_fwd(const ssm_scan_args_t *args, void *stream);

/* Bytes of the device scratch array behind ssm_selective_scan_fwd_noalloc (32 MiB). */
#define SSM_NOALLOC_SCRATCH_BYTES (32u << 20)

/*
 * ssm_selective_scan_fwd for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  It computes exactly what ssm_selective_scan_fwd computes, with
 * the same kernels, but its workspace is a device array of
 * SSM_NOALLOC_SCRATCH_BYTES that the library holds on each device it runs on
 * until the process ends (a 1M-token sequence at D = 1024 needs about 2 MiB).
 * args->workspace must be NULL and args->workspace_bytes 0.  The caller still
 * passes every input and output.
 *
 * Errors: besides those of ssm_selective_scan_fwd, SSM_ERR_WORKSPACE when
 * ssm_selective_scan_workspace_size(args) exceeds SSM_NOALLOC_SCRATCH_BYTES
 * (before any HIP call) or a workspace is passed; SSM_ERR_HIP if the array's
 * address cannot be obtained on the stream's device.  The call allocates
 * nothing; the first call on a device looks up the array's address there.
 *
 * Every call on one device shares that device's array, and the array keeps
 * whatever the last call left in it (no call depends on its contents on
 * entry).  Calls that may overlap in time on one device -- on different
 * streams, or from different threads without ordering -- race on it: order
 * them on one stream, or use ssm_selective_scan_fwd with separate workspaces.
 */
ssm_status_t ssm_selective_scan_fwd_noalloc(const ssm_scan_args_t *args, void *stream);

/*
 * Depthwise causal conv1d + SiLU, the prologue of [P1] sec. 4a with the
 * width of [P2] (d_conv: 4):
 *   u[b,t,d] = silu(sum_{k<K} w[d,k] x[b,t-(K-1)+k,d] + bias[d]),
 * x at negative times taken as 0 (zero left padding; w[d,K-1] weighs the
 * current token).  x and u: (B,L,D) of io_dtype; w: (D,K) fp32; bias: (D)
 * fp32 or NULL.  1 <= K <= SSM_MAX_CONV_K.  u must not overlap x.
 */
ssm_status_t ssm_causal_conv1d_silu(int64_t batch, int64_t seqlen, int64_t dim, int64_t k,
                                    int32_t io_dtype, const void *x, const float *w,
                                    const float *bias, void *u, void *stream);

/*
 * One decode step, [P1] eq. (2a)/(2b) in recurrent mode on a state kept
 * between calls ([P2] ssm_state), for every batch row b and channel d:
 *   u           = x[b,d], or with conv_k > 0 the prologue of [P1] sec. 4a on
 *                 the window (conv_state[b,0..K-2,d], x[b,d]):
 *                 silu(sum_{k<K-1} conv_w[d,k] conv_state[b,k,d]
 *                      + conv_w[d,K-1] x[b,d] + conv_b[d]);
 *                 the window then drops its oldest row and appends x[b,d]
 *   dt          = delta[b,d] or softplus(delta[b,d] + delta_bias[d])
 *   state[b,d,n] <- exp(dt A[d,n]) state[b,d,n] + Bbar(dt, A[d,n], Bm[b,n]) u
 *   y[b,d]      = (sum_n Cm[b,n] state[b,d,n] + Dskip[d] u) * silu(z[b,d])
 * with Bbar as in the scan.  The state and the conv state are read and
 * written IN PLACE; the conv state has the layout of the scan's
 * conv_state_out, so a prefill hands over to decode directly.
 */
typedef struct ssm_state_update_args {
    int64_t batch;          /* B >= 0                                     */
    int64_t dim;            /* D >= 1                                     */
    int64_t dstate;         /* N, 1 <= N <= SSM_MAX_DSTATE                */
    int32_t io_dtype;       /* ssm_dtype_t of x, delta, z, Bm, Cm, y      */
    int32_t delta_softplus; /* as in ssm_scan_args                        */
    float *state;           /* (B,D,N) fp32, updated in place; required   */
    const void *x;          /* (B,D) io_dtype, required                   */
    const void *delta;      /* (B,D) io_dtype, required                   */
    const void *z;          /* (B,D) io_dtype, or NULL (no gate)          */
    const void *Bm;         /* (B,N) io_dtype, required                   */
    const void *Cm;         /* (B,N) io_dtype, required                   */
    const float *A;         /* (D,N) fp32, required                       */
    const float *Dskip;     /* (D) fp32, or NULL                          */
    const float *delta_bias;/* (D) fp32, or NULL                          */
    void *y;                /* (B,D) io_dtype output; must not overlap any input or the state */
    int64_t conv_k;         /* 0: no prologue; 1..SSM_MAX_CONV_K: causal conv1d + SiLU on x
                               (then D <= 2^28, else SSM_ERR_UNSUPPORTED) */
    const float *conv_w;    /* (D,conv_k) fp32; required iff conv_k > 0   */
    const float *conv_b;    /* (D) fp32, or NULL (= 0)                    */
    void *conv_state;       /* (B,conv_k-1,D) io_dtype, updated in place; required iff
                               conv_k > 1; must not overlap any other argument */
} ssm_state_update_args_t;

ssm_status_t ssm_state_update(const ssm_state_update_args_t *args, void *stream);

/*
 * Backward pass of the selective scan: the gradients of a scalar loss with
 * dL/dy = dy and dL/dh_final = dh_final through the forward defined above
 * ([P1] eq. (4), (2a)/(2b), sec. 4a; the states are recomputed from
 * checkpoints instead of stored, as [P1] sec. 4c does).  With
 * lambda_t = dL/dh_t and gy_t = dy_t silu(z_t):
 *   lambda_t = C_t gy_t + exp(dt_{t+1} A) lambda_{t+1}  (lambda_{L-1} adds dh_final)
 *   dx       = sum_n lambda Bbar + Dskip gy;   ddelta by the chain rule through
 *              exp(dt A), Bbar and the softplus;   dz = dy (C h + D u) silu'(z);
 *   dA, dDskip, ddelta_bias summed over batch and time; dBm, dCm summed over
 *   channels; dh0 = exp(dt_0 A) lambda_0;
 *   with the conv prologue (u = silu(c), c the causal conv of x): dc = du
 *   silu'(c), dx = the conv's transpose applied to dc, dconv_w and dconv_b
 *   summed over batch and time; with a conv state entering the sequence
 *   (the forward's conv_state_in) its rows are read at negative times and
 *   dconv_state_in is the conv's transpose at those times.
 * 1 <= N <= SSM_MAX_DSTATE.  The kernels hold 16 state entries per channel;
 * for N < 16 the workspace also holds 16-wide copies of Bm, Cm, A, h0 and
 * dh_final (extra entries B = C = 0, h0 = dh_final = 0, A = -1, whose state
 * and adjoint stay 0) and of the gradients dA, dBm, dCm and dh0, which are
 * copied back to N-wide rows.  The forward's input fields have the same
 * meaning and shapes as in ssm_scan_args_t.
 */
typedef struct ssm_scan_bwd_args {
    int64_t batch, seqlen, dim, dstate; /* as in ssm_scan_args_t (1 <= N <= 16) */
    int32_t io_dtype;       /* of x, delta, Bm, Cm, z, dy, dx, ddelta, dz      */
    int32_t delta_softplus; /* as in ssm_scan_args_t                           */
    int64_t conv_k;         /* 0 or 1..SSM_MAX_CONV_K, as in ssm_scan_args_t   */
    const void *x, *delta, *Bm, *Cm, *z;            /* forward inputs            */
    const float *A, *Dskip, *delta_bias, *conv_w, *conv_b, *h0;
    const void *dy;         /* (B,L,D) io_dtype, required                      */
    const float *dh_final;  /* (B,D,N) fp32, or NULL (= 0)                     */
    void *dx;               /* (B,L,D) io_dtype output, required               */
    void *ddelta;           /* (B,L,D) io_dtype output (w.r.t. the raw delta)  */
    void *dz;               /* (B,L,D) io_dtype output; required iff z         */
    float *dA;              /* (D,N) fp32 output, required                     */
    float *dBm, *dCm;       /* (B,L,N) fp32 outputs, required                  */
    float *dDskip;          /* (D) fp32 output, or NULL (not written)          */
    float *ddelta_bias;     /* (D) fp32 output, or NULL; 0 without softplus    */
    float *dconv_w;         /* (D,conv_k) fp32 output; required iff conv_k > 0 */
    float *dconv_b;         /* (D) fp32 output, or NULL; only with conv_k > 0  */
    float *dh0;             /* (B,D,N) fp32 output, or NULL                    */
    void *workspace;        /* device scratch, 256-aligned                     */
    size_t workspace_bytes; /* >= ssm_selective_scan_bwd_workspace_size(args)  */
    const void *conv_state_in; /* (B,K-1,D) io_dtype: the inputs before t = 0 the
                                  forward's conv read (its conv_state_in), or
                                  NULL (= 0); only with conv_k > 1          */
    void *dconv_state_in;   /* (B,K-1,D) io_dtype output: its gradient, or NULL;
                               only with conv_k > 1                            */
    const float *checkpoints; /* (ceil(L/SSM_SCAN_BLOCK), B, D, SSM_MAX_DSTATE) fp32: the
                                 checkpoints an ssm_selective_scan_fwd call wrote for the
                                 same x, delta, A, Bm, h0, delta options, conv weights
                                 and conv_state_in; or NULL, and the backward computes
                                 them (in its workspace, which is then larger) */
} ssm_scan_bwd_args_t;

/* Workspace bytes ssm_selective_scan_bwd needs ((size_t)-1 for invalid sizes). */
size_t ssm_selective_scan_bwd_workspace_size(const ssm_scan_bwd_args_t *args);

/*
 * Enqueue the backward pass on `stream`.  Outputs must not overlap any input,
 * each other or the workspace.  Every output given is overwritten.  Returns
 * SSM_OK or an error status (see the conventions).
 */
ssm_status_t ssm_selective_scan_bwd(const ssm_scan_bwd_args_t *args, void *stream);

/*
 * One Mamba block with its pre-norm residual, the block of [P1] sec. 4a (the
 * table of tensor shapes: RMSNorm, the expanding Linear to x and the gate z,
 * Conv1d -> SiLU, the selective SSM, x SiLU(z), the output Linear, + input),
 * with the projections of [P1] Algorithm 2 (s_B, s_C = Linear_N, s_Delta a
 * low-rank Linear of rank R followed by Linear_D; the page's Linear_1 +
 * Broadcast_D is R = 1 with W_dt = 1) and tau_Delta = softplus:
 *   hn = RMSNorm(h) (eps = norm_eps, weight norm_w)
 *   x = hn W_in[0:D]^T, z = hn W_in[D:2D]^T, u = silu(conv1d(x))
 *   dt_low = u W_x[0:R]^T, B = u W_x[R:R+N]^T, C = u W_x[R+N:R+2N]^T
 *   delta = dt_low W_dt^T;  y = S6(u, softplus(delta + dt_bias), A, B, C, D) * silu(z)
 *   h_out = h + y W_out^T
 * I/O and intermediates are bf16 (products accumulate in fp32; the step
 * softplus(delta + dt_bias) is formed in fp32 and stored in bf16); norm_w,
 * conv weights, dt_bias, A and Dskip are fp32.  in_proj, x_proj and out_proj
 * run in hipBLASLt, dt_proj in the library's own kernel.
 *
 * Usage: create a plan for the sizes (this creates a hipBLASLt handle and
 * picks the GEMM algorithms; host memory only, needs the GPU), query its
 * device workspace size, call ssm_block_fwd any number of times, destroy.
 */
typedef struct ssm_block_dims {
    int64_t batch, seqlen;  /* B >= 1, L >= 1                                  */
    int64_t d_model;        /* model width, a multiple of 8                    */
    int64_t d_inner;        /* D = E * d_model (SSM channels), a multiple of 8 */
    int64_t dstate;         /* N, 1 <= N <= SSM_MAX_DSTATE                     */
    int64_t dt_rank;        /* R >= 1                                          */
    int64_t conv_k;         /* 1..SSM_MAX_CONV_K                               */
} ssm_block_dims_t;

typedef struct ssm_block_weights {
    const float *norm_w;    /* (d_model) fp32                                  */
    const void *w_in;       /* (2 D, d_model) bf16: rows of x, then of z       */
    const float *conv_w;    /* (D, conv_k) fp32                                */
    const float *conv_b;    /* (D) fp32, or NULL                               */
    const void *w_x;        /* (R + 2N, D) bf16: rows of dt_low, B, C          */
    const void *w_dt;       /* (D, R) bf16                                     */
    const float *dt_bias;   /* (D) fp32                                        */
    const float *A;         /* (D, N) fp32                                     */
    const float *Dskip;     /* (D) fp32, or NULL                               */
    const void *w_out;      /* (d_model, D) bf16                               */
    float norm_eps;         /* > 0, e.g. 1e-5                                  */
} ssm_block_weights_t;

typedef struct ssm_block_plan ssm_block_plan_t;

/*
 * Plan for these sizes.  Returns SSM_OK and *plan, or an error and *plan =
 * NULL: SSM_ERR_NULL_ARG, SSM_ERR_BAD_SHAPE (a size < 1, dt_rank > d_inner,
 * B*L >= 2^30), SSM_ERR_UNSUPPORTED (dstate, conv_k or a width not a multiple
 * of 8; or hipBLASLt offers no algorithm), SSM_ERR_HIP (no device, or the
 * handle could not be created).  The plan belongs to the device current at
 * creation.
 */
ssm_status_t ssm_block_plan_create(const ssm_block_dims_t *dims, ssm_block_plan_t **plan);

/* Device workspace bytes ssm_block_fwd needs with this plan (0 for NULL). */
size_t ssm_block_workspace_size(const ssm_block_plan_t *plan);

/*
 * h_out = the block applied to h_in, both (B, L, d_model) bf16.  h_out may be
 * h_in itself (updated in place) but may not overlap it otherwise or any
 * weight; nothing may overlap the workspace (256-aligned, >=
 * ssm_block_workspace_size).  bf16 tensors (h_in, h_out, w_in, w_x, w_dt,
 * w_out), norm_w and dt_bias must be 16-byte aligned, the other fp32 ones
 * 4-byte aligned.  The plan may be
 * shared by calls on different streams only with separate workspaces.
 * Errors: SSM_ERR_NULL_ARG (plan, h_in, h_out or a required weight NULL),
 * SSM_ERR_BAD_SHAPE (norm_eps <= 0), SSM_ERR_ALIGN, SSM_ERR_WORKSPACE,
 * SSM_ERR_ALIAS, SSM_ERR_HIP (a launch or hipBLASLt call failed).
 */
ssm_status_t ssm_block_fwd(const ssm_block_plan_t *plan, const ssm_block_weights_t *weights,
                           const void *h_in, void *h_out, void *workspace, size_t workspace_bytes,
                           void *stream);

/* Release a plan (NULL is ignored). */
void ssm_block_plan_destroy(ssm_block_plan_t *plan);

/*
 * The SSD (Mamba-2) layer: [P4] sec. 5.1 restricts the state matrix to a
 * scalar times the identity per step and head, A_t = a_t I, which makes the
 * layer the masked product Y = (L o (C B^T)) X with L the causal mask of
 * cumulative decays; sec. 5.2 evaluates it chunk by chunk (the quadratic form
 * inside a chunk on the matrix cores, the recurrence between chunks).  With
 * the ZOH rule of [P1] eq. (4) for A = a I, per batch b, head h, head channel
 * p, state entry n and step t (g = h / (H / G) the head's group):
 *   dt      = delta[b,t,h], or softplus(delta[b,t,h] + delta_bias[h])
 *   S[p,n] <- exp(dt A[h]) S[p,n] + (exp(dt A[h]) - 1) / A[h] Bm[b,t,g,n] x[b,t,h,p]
 *             (the weight is dt where dt A[h] == 0), from h0 (or 0)
 *   y[b,t,h,p] = (sum_n Cm[b,t,g,n] S[p,n] + Dskip[h] x[b,t,h,p]) * silu(z[b,t,h,p])
 * The state layout (B, H, P, N) is the scan's (B, D, N) with D = H P.
 * This version: headdim P a multiple of 32 up to 4096, dstate N in
 * {16, 32, 64, 128}, batch * nheads * P / 32 <= 2^23; other values give
 * SSM_ERR_UNSUPPORTED.  bf16 I/O runs the chunked form below.  fp32 I/O runs
 * the recurrent form (the same map, [P4] sec. 5.1) sequentially in time with
 * the state in registers, in fp32 throughout, and needs no workspace; its
 * Bm, Cm, h0 and h_final must be 16-byte aligned.  Products run in bf16 on the matrix
 * cores with fp32 accumulation; the state is fp32 (its bf16 copy feeds the
 * product with C).
 */
typedef struct ssm_ssd_args {
    int64_t batch, seqlen;  /* B >= 0, L >= 0                                  */
    int64_t nheads;         /* H >= 1                                          */
    int64_t headdim;        /* P, a multiple of 32 (<= 4096)                   */
    int64_t ngroups;        /* G >= 1, divides H: heads of a group share B, C  */
    int64_t dstate;         /* N (16, 32, 64 or 128)                           */
    int32_t io_dtype;       /* of x, delta, Bm, Cm, z, y: SSM_BF16 or SSM_F32  */
    int32_t delta_softplus; /* 0: delta is the step; 1: softplus(delta + bias) */
    const void *x;          /* (B,L,H,P) io_dtype, required                    */
    const void *delta;      /* (B,L,H) io_dtype, required                      */
    const float *A;         /* (H) fp32, required; any finite value            */
    const void *Bm, *Cm;    /* (B,L,G,N) io_dtype, required                    */
    const float *Dskip;     /* (H) fp32, or NULL                               */
    const void *z;          /* (B,L,H,P) io_dtype gate, or NULL                */
    const float *delta_bias;/* (H) fp32, or NULL                               */
    const float *h0;        /* (B,H,P,N) fp32 initial state, or NULL (= 0)     */
    void *y;                /* (B,L,H,P) io_dtype output, required             */
    float *h_final;         /* (B,H,P,N) fp32 output, or NULL                  */
    void *workspace;        /* device scratch of workspace_bytes, 256-aligned  */
    size_t workspace_bytes; /* >= ssm_ssd_workspace_size(args)                 */
} ssm_ssd_args_t;

/*
 * Bytes of device workspace ssm_ssd_fwd needs (0 when none; only the size
 * fields are read).  With few (batch, head) pairs the sequence is cut into
 * segments that run at once: each segment's end state from a zero start,
 * then the entering states by the recurrence over segments, then each
 * segment's outputs from its entering state.  The workspace holds those
 * states; its contents on entry do not matter.  (size_t)-1 for invalid sizes.
 */
size_t ssm_ssd_workspace_size(const ssm_ssd_args_t *args);

/*
 * Enqueue the SSD layer on `stream`.  x, Bm, Cm, z and y must be 16-byte
 * aligned, delta 2-byte, the fp32 tensors 4-byte.  y, h_final and the
 * workspace must not overlap any input or each other.  L == 0 copies h0 (or zeros) to h_final;
 * the (B,L,...) pointers may then be NULL.
 */
ssm_status_t ssm_ssd_fwd(const ssm_ssd_args_t *args, void *stream);

/*
 * One decode step of the SSD layer: the recurrence above ([P4] sec. 5.1, the
 * state matrix a_t I per step; the recurrent mode of [P1] sec. 4b used for
 * decoding) for a single token on a state kept between calls (updated IN
 * PLACE), for every batch b, head h, head channel p and state entry n
 * (g = h / (H / G)):
 *   dt = delta[b,h] (or softplus(delta[b,h] + delta_bias[h]))
 *   state[b,h,p,n] <- exp(dt A[h]) state[b,h,p,n] + w(dt, A[h]) Bm[b,g,n] x[b,h,p]
 *   y[b,h,p] = (sum_n Cm[b,g,n] state[b,h,p,n] + Dskip[h] x[b,h,p]) * silu(z[b,h,p])
 * with w the ZOH weight of ssm_ssd_fwd; the state layout is that function's
 * h0/h_final, so a prefill hands over to decode directly.  bf16 I/O; any
 * head dim; dstate a power of two from 4 to 256.
 */
typedef struct ssm_ssd_step_args {
    int64_t batch, nheads, headdim, ngroups, dstate; /* B >= 0, H, P, G | H, N */
    int32_t io_dtype;       /* of x, delta, Bm, Cm, z, y: SSM_BF16 or SSM_F32  */
    int32_t delta_softplus; /* as in ssm_ssd_args_t                            */
    float *state;           /* (B,H,P,N) fp32, updated in place; 16-byte aligned */
    const void *x;          /* (B,H,P) bf16, required                          */
    const void *delta;      /* (B,H) bf16, required                            */
    const float *A;         /* (H) fp32, required                              */
    const void *Bm, *Cm;    /* (B,G,N) bf16, required; 8-byte aligned          */
    const float *Dskip;     /* (H) fp32, or NULL                               */
    const void *z;          /* (B,H,P) bf16 gate, or NULL                      */
    const float *delta_bias;/* (H) fp32, or NULL                               */
    void *y;                /* (B,H,P) bf16 output; must not overlap any input or the state */
} ssm_ssd_step_args_t;

ssm_status_t ssm_ssd_step(const ssm_ssd_step_args_t *args, void *stream);

/*
 * The gated linear recurrence: one state per channel, whose decay a_t is an
 * input of every step rather than exp(dt A).  Per batch row b and channel d,
 *   h_t = a_t h_{t-1} + b_t, from h0 (or 0);   y_t = h_t;   h_final = h_{L-1}
 * with a_t and b_t formed from the inputs by `mode` (sig the logistic
 * function; a bias that is not given is 0):
 *   SSM_GATE_DECAY    a = gate,            b = x
 *   SSM_GATE_SIGMOID  s = sig(gate + gate_bias),  a = 1 - s,  b = s x
 *                     ([P1] Theorem 1, the gated RNN the scan reduces to)
 *   SSM_GATE_RATE     r = sig(gate + gate_bias),  a = exp(A r),
 *                     b = sqrt(1 - a^2) sig(in_gate + in_bias) x
 *                     (without in_gate: b = sqrt(1 - a^2) x).  A <= 0: the
 *                     input weight keeps a unit-variance input's state at unit
 *                     variance; where A > 0 it is 0.
 * Where reset[b,t] != 0 the state is dropped before step t (h_t = b_t,
 * whatever h_{t-1} was, an infinity or a NaN included): sequences packed one
 * behind the other in a row come out as in calls of their own, and a row
 * padded on the left resets at its first token.
 *
 * The decays are meant to lie in [-1, 1]: in SSM_GATE_DECAY as they are given, in
 * SSM_GATE_RATE by A <= 0.  Others are computed too, but the products of up to
 * SSM_GATED_TILE decays formed inside (in the backward too) must stay below 2^127:
 * growth beyond it gives an infinity or a NaN also where the states themselves
 * stay finite.  In SSM_GATE_RATE a state of 0 stays 0 all the same where each
 * decay is finite, and so do the gradients through it where each lambda, formed
 * from such products, is.
 *
 * Arithmetic is fp32 (the hardware's exponential, reciprocal and square root,
 * 1 ulp); y is rounded once.  Results do not change from run to run.
 *
 * A call is several launches on its stream, and its workspace carries data from
 * one to the next: calls enqueued one after the other on a stream may use the
 * same workspace, calls from several host threads at once, also on one stream,
 * may not.
 */
typedef enum ssm_gate_mode {
    SSM_GATE_DECAY = 0,
    SSM_GATE_SIGMOID = 1,
    SSM_GATE_RATE = 2
} ssm_gate_mode_t;

#define SSM_GATED_BLOCK 128 /* steps between two checkpoints of the gated scan */
#define SSM_GATED_TILE 256  /* most steps whose decays are multiplied together */

typedef struct ssm_gated_scan_args {
    int64_t batch, seqlen;  /* B >= 0, L >= 0                                  */
    int64_t dim;            /* D, 1 <= D <= 2^20; B ceil(L/128) ceil(D/32) < 2^23 */
    int32_t io_dtype;       /* ssm_dtype_t of x, gate, in_gate and y           */
    int32_t mode;           /* ssm_gate_mode_t                                 */
    const void *x;          /* (B,L,D) io_dtype, required                      */
    const void *gate;       /* (B,L,D) io_dtype, required                      */
    const void *in_gate;    /* (B,L,D) io_dtype, or NULL; SSM_GATE_RATE only   */
    const float *A;         /* (D) fp32; required with SSM_GATE_RATE, else NULL */
    const float *gate_bias; /* (D) fp32, or NULL; not with SSM_GATE_DECAY      */
    const float *in_bias;   /* (D) fp32, or NULL; only with in_gate            */
    const uint8_t *reset;   /* (B,L) bytes, or NULL (no resets)                */
    const float *h0;        /* (B,D) fp32 initial state, or NULL (= 0)         */
    void *y;                /* (B,L,D) io_dtype output, required               */
    float *h_final;         /* (B,D) fp32 output, or NULL                      */
    float *checkpoints;     /* (ceil(L/SSM_GATED_BLOCK), B, D) fp32 output, or NULL:
                               the state entering step SSM_GATED_BLOCK * j, before
                               a reset there (h0 or 0 for j = 0)               */
    void *workspace;        /* device scratch of workspace_bytes, 256-aligned  */
    size_t workspace_bytes; /* >= ssm_gated_scan_workspace_size(args)          */
} ssm_gated_scan_args_t;

/* Bytes of device workspace ssm_gated_scan_fwd needs (only the size fields and
 * io_dtype are read); its contents on entry do not matter.  (size_t)-1 for
 * invalid sizes. */
size_t ssm_gated_scan_workspace_size(const ssm_gated_scan_args_t *args);

/* Enqueue the recurrence.  Outputs must not overlap any input, each other or
 * the workspace.  L == 0 copies h0 (or zeros) to h_final. */
ssm_status_t ssm_gated_scan_fwd(const ssm_gated_scan_args_t *args, void *stream);

/*
 * Gradients of the recurrence for dL/dy = dy and dL/dh_final = dh_final:
 *   lambda_t = dy_t + a_{t+1} lambda_{t+1}  (0 through a reset at t + 1;
 *              lambda_{L-1} adds dh_final)
 *   da_t = lambda_t h_{t-1} (0 at a reset), db_t = lambda_t, and the chain rule
 *   through a and b above;  dA, dgate_bias, din_bias summed over batch and
 *   time;  dh0 = a_0 lambda_0 (0 with a reset at 0).
 * The states are recomputed in fp32 from the forward's checkpoints (which the
 * backward computes itself when none are given).  Where 1 - a^2 is 0 or below
 * 2^-126, the derivative of its root is taken as 0.  Steps ahead of a reset take
 * part in the sums dA, dgate_bias and din_bias also where their dy is 0, so the
 * inputs in a row's left padding have to be finite.
 */
typedef struct ssm_gated_scan_bwd_args {
    int64_t batch, seqlen, dim; /* as in ssm_gated_scan_args_t                 */
    int32_t io_dtype;       /* of x, gate, in_gate, dy, dx, dgate, din_gate    */
    int32_t mode;           /* as in ssm_gated_scan_args_t                     */
    const void *x, *gate, *in_gate;                       /* forward inputs    */
    const float *A, *gate_bias, *in_bias;
    const uint8_t *reset;
    const float *h0;
    const void *dy;         /* (B,L,D) io_dtype, required                      */
    const float *dh_final;  /* (B,D) fp32, or NULL (= 0)                       */
    const float *checkpoints; /* of an ssm_gated_scan_fwd call on the same inputs, or NULL */
    void *dx, *dgate;       /* (B,L,D) io_dtype outputs, required              */
    void *din_gate;         /* (B,L,D) io_dtype output; required iff in_gate   */
    float *dA;              /* (D) fp32 output; required iff SSM_GATE_RATE     */
    float *dgate_bias;      /* (D) fp32 output, or NULL; not with SSM_GATE_DECAY */
    float *din_bias;        /* (D) fp32 output, or NULL; only with in_gate     */
    float *dh0;             /* (B,D) fp32 output, or NULL                      */
    void *workspace;        /* device scratch, 256-aligned                     */
    size_t workspace_bytes; /* >= ssm_gated_scan_bwd_workspace_size(args)      */
} ssm_gated_scan_bwd_args_t;

/* Workspace bytes ssm_gated_scan_bwd needs: the size fields, io_dtype, mode and
 * whether checkpoints are given are read.  (size_t)-1 for invalid sizes. */
size_t ssm_gated_scan_bwd_workspace_size(const ssm_gated_scan_bwd_args_t *args);

/* Enqueue the backward pass.  Outputs must not overlap any input, each other
 * or the workspace; every output given is overwritten. */
ssm_status_t ssm_gated_scan_bwd(const ssm_gated_scan_bwd_args_t *args, void *stream);

/*
 * One decode step of the recurrence on a state kept between calls:
 *   state[b,d] <- a state[b,d] + b (state taken as 0 where reset[b] != 0);
 *   y[b,d] = state[b,d]
 * The state is read and written IN PLACE; it is h_final of a prefill.
 */
typedef struct ssm_gated_step_args {
    int64_t batch, dim;     /* B >= 0, 1 <= D <= 2^20; B ceil(D/32) < 2^23     */
    int32_t io_dtype, mode; /* as in ssm_gated_scan_args_t                     */
    float *state;           /* (B,D) fp32, updated in place; required          */
    const void *x, *gate;   /* (B,D) io_dtype, required                        */
    const void *in_gate;    /* (B,D) io_dtype, or NULL; SSM_GATE_RATE only     */
    const float *A, *gate_bias, *in_bias; /* as in ssm_gated_scan_args_t       */
    const uint8_t *reset;   /* (B) bytes, or NULL                              */
    void *y;                /* (B,D) io_dtype output, required                 */
} ssm_gated_step_args_t;

/* y must not overlap any input or the state, nor the state an input. */
ssm_status_t ssm_gated_scan_step(const ssm_gated_step_args_t *args, void *stream);

/*
 * The boundary between two pre-norm residual blocks in one pass over the rows
 * ([P1] sec. 4a: the block's output is added to its input, the next block
 * begins with the norm).  Per row, with RMS(v) = v / sqrt(mean(v^2) + eps):
 *   u       = x, or RMS(x) * post_w when post_w is given (a norm behind the
 *             block as well)
 *   res_out = residual + scale * u   (residual NULL: 0; scale NULL: 1)
 *   y       = RMS(res_out) * w       (of the sum before its rounding)
 */
typedef struct ssm_add_norm_args {
    int64_t rows;           /* >= 0                                            */
    int64_t dim;            /* D, 1 <= D <= 2^20                               */
    int32_t io_dtype;       /* ssm_dtype_t of x and y                          */
    int32_t res_dtype;      /* ssm_dtype_t of residual and res_out             */
    const void *x;          /* (rows,D) io_dtype, required                     */
    const void *residual;   /* (rows,D) res_dtype, or NULL                     */
    const float *scale;     /* (D) fp32, or NULL                               */
    const float *post_w;    /* (D) fp32, or NULL                               */
    const float *w;         /* (D) fp32, required                              */
    void *res_out;          /* (rows,D) res_dtype output, or NULL; may be exactly residual */
    void *y;                /* (rows,D) io_dtype output, required              */
    float eps;              /* > 0                                             */
} ssm_add_norm_args_t;

/* Outputs must not overlap an input (but res_out may be residual) or each other. */
ssm_status_t ssm_add_rmsnorm_fwd(const ssm_add_norm_args_t *args, void *stream);

/*
 * Its gradients for dL/dy = dy and dL/dres_out = dres_out.  The forward's
 * inputs are read again and every intermediate is recomputed in fp32 from
 * them, so the sums dw, dscale and dpost_w do not see a rounded stream.
 */
typedef struct ssm_add_norm_bwd_args {
    int64_t rows, dim;
    int32_t io_dtype;       /* of x, dy, dx                                    */
    int32_t res_dtype;      /* of residual, dres_out, dresidual                */
    const void *x, *residual;               /* forward inputs (before an in-place update) */
    const float *scale, *post_w, *w;
    const void *dy;         /* (rows,D) io_dtype, required                     */
    const void *dres_out;   /* (rows,D) res_dtype, or NULL (= 0)               */
    void *dx;               /* (rows,D) io_dtype output, required              */
    void *dresidual;        /* (rows,D) res_dtype output, or NULL; only with residual */
    float *dw;              /* (D) fp32 output, required                       */
    float *dscale;          /* (D) fp32 output, or NULL; only with scale       */
    float *dpost_w;         /* (D) fp32 output, or NULL; only with post_w      */
    void *workspace;        /* device scratch, 256-aligned                     */
    size_t workspace_bytes; /* >= ssm_add_rmsnorm_bwd_workspace_size(args)     */
    float eps;              /* > 0                                             */
} ssm_add_norm_bwd_args_t;

/* Workspace bytes (the size fields and types and whether scale and post_w are given
 * are read); (size_t)-1 for invalid sizes. */
size_t ssm_add_rmsnorm_bwd_workspace_size(const ssm_add_norm_bwd_args_t *args);

/* Outputs must not overlap an input, each other or the workspace, except that
 * dresidual may be exactly dres_out. */
ssm_status_t ssm_add_rmsnorm_bwd(const ssm_add_norm_bwd_args_t *args, void *stream);

/*
 * RMSNorm of a gated layer output (the output of ssm_ssd_fwd or
 * ssm_gated_scan_fwd ahead of the output projection), over `groups` groups of
 * D / groups consecutive channels each.  With g = SiLU(z):
 *   gate_first = 1:  v = x g,  y = v / sqrt(mean_group(v^2) + eps) * w
 *   gate_first = 0:  y = x / sqrt(mean_group(x^2) + eps) * w * g
 */
typedef struct ssm_gated_norm_args {
    int64_t rows;           /* >= 0                                            */
    int64_t dim;            /* D, 1 <= D <= 2^20                               */
    int64_t groups;         /* G >= 1, divides D                               */
    int32_t io_dtype;       /* ssm_dtype_t of x, z and y                       */
    int32_t gate_first;     /* 0 or 1                                          */
    const void *x, *z;      /* (rows,D) io_dtype, required                     */
    const float *w;         /* (D) fp32, required                              */
    void *y;                /* (rows,D) io_dtype output, required              */
    float eps;              /* > 0                                             */
} ssm_gated_norm_args_t;

/* y must not overlap an input, except that it may be exactly x or z. */
ssm_status_t ssm_gated_rmsnorm_fwd(const ssm_gated_norm_args_t *args, void *stream);

typedef struct ssm_gated_norm_bwd_args {
    int64_t rows, dim, groups;
    int32_t io_dtype, gate_first;
    const void *x, *z;      /* forward inputs                                  */
    const float *w;
    const void *dy;         /* (rows,D) io_dtype, required                     */
    void *dx, *dz;          /* (rows,D) io_dtype outputs, required             */
    float *dw;              /* (D) fp32 output, required                       */
    void *workspace;        /* device scratch, 256-aligned                     */
    size_t workspace_bytes; /* >= ssm_gated_rmsnorm_bwd_workspace_size(args)   */
    float eps;              /* > 0                                             */
} ssm_gated_norm_bwd_args_t;

/* Workspace bytes (the size fields and io_dtype are read); (size_t)-1 for invalid sizes. */
size_t ssm_gated_rmsnorm_bwd_workspace_size(const ssm_gated_norm_bwd_args_t *args);

/* Outputs must not overlap an input, each other or the workspace. */
ssm_status_t ssm_gated_rmsnorm_bwd(const ssm_gated_norm_bwd_args_t *args, void *stream);

/*
 * The gated delta rule: per batch row b and value head h a state S of
 * (kdim, vdim), read by a query and written by a key.  Per step t
 *   S' = e^{g_t} S_{t-1}                     (0 where reset[b,t] != 0)
 *   e_t = v_t - S'^T k_t                     what the state has wrong for k_t
 *   S_t = S' + beta_t k_t e_t^T,   o_t = scale S_t^T q_t
 * from S = h0 (or 0); h_final is the state after the last step.  Value head h
 * uses q and k of head h / (heads / kheads).  With l2norm, q and k stand for
 * q / sqrt(sum q^2 + 1e-6) and k / sqrt(sum k^2 + 1e-6) over a head's channels.
 *
 * g is the log of the decay: usually <= 0, or above as long as e^g is finite in
 * fp32; a step with g < SSM_DELTA_FORGET (e^g is 0 in fp32; -infinity is one) is
 * a reset, with dg = 0.  The state settles for beta |k|^2 in (0, 2); beyond, it
 * grows as the formulas say.  Decays that grow: a head in which those of some
 * steps of a chunk multiply to more than e is computed one step after another
 * (backwards: all heads of its key head), far slower, as the 64 steps of a chunk
 * at once would lose what such a product exceeds the state by.
 * A reset drops the state whatever it held, an infinity or a NaN included; the
 * inputs themselves have to be finite, in a row's left padding too (the 64 steps
 * of a chunk are computed together).
 *
 * Arithmetic is fp32: bf16 tensors run on the bf16 matrix cores, with what was
 * computed carried through the products as the sum of three bf16 numbers (two,
 * 16 bits, where only bf16 outputs follow: o, and dq and dk, with l2norm ahead of
 * the norm's gradient, which takes their part along q and k out); outputs are
 * rounded once.  Results
 * do not change from run to run.  Long sequences of few heads run as parallel
 * segments, in other places for another length: a sequence in two calls gives
 * what one call does to rounding.  kdim: a multiple of 8 up to SSM_DELTA_MAX_KDIM;
 * vdim: a multiple of 8 up to SSM_DELTA_MAX_VDIM; kheads divides heads <= 65535;
 * batch <= 65535; seqlen < 2^30; heads * vdim and kheads * kdim < 2^24;
 * (batch * heads + 8) * ceil(vdim / 16) < 2^23.
 *
 * q, k and v may be parts of a wider tensor: x_token is the distance of two steps
 * and x_batch that of two batch rows, in elements; x_token 0: dense.  A head's
 * channels and a step's heads are always consecutive.  Strides are not negative,
 * x_token < 2^24 and x_batch <= 2^40.  q and k lie at 16-byte boundaries, with
 * strides that keep them there (ssm_gated_delta_step: at their elements').
 *
 * A call is several launches and its workspace carries data between them: as
 * with ssm_gated_scan_fwd.
 */
#define SSM_DELTA_CHUNK 64
#define SSM_DELTA_MAX_KDIM 128
#define SSM_DELTA_MAX_VDIM 1024
#define SSM_DELTA_FORGET (-104.0f)

typedef struct ssm_gated_delta_args {
    int64_t batch, seqlen;  /* B >= 0, L >= 0                                  */
    int64_t kheads, heads;  /* Hk >= 1, H: a multiple of it                    */
    int64_t kdim, vdim;     /* K, V                                            */
    int32_t io_dtype;       /* ssm_dtype_t of q, k, v, beta and o              */
    int32_t l2norm;         /* 0 or 1                                          */
    const void *q, *k;      /* (B,L,Hk,K) io_dtype, required                   */
    const void *v;          /* (B,L,H,V) io_dtype, required                    */
    const float *g;         /* (B,L,H) fp32, required                          */
    const void *beta;       /* (B,L,H) io_dtype, required                      */
    const uint8_t *reset;   /* (B,L) bytes, or NULL (no resets)                */
    const float *h0;        /* (B,H,K,V) fp32 initial state, or NULL (= 0)     */
    void *o;                /* (B,L,H,V) io_dtype output, required             */
    float *h_final;         /* (B,H,K,V) fp32 output, or NULL                  */
    float *checkpoints;     /* (ceil(L/SSM_DELTA_CHUNK), B, H, K + SSM_DELTA_CHUNK, V) fp32
                               output, 16-byte aligned, or NULL: for each chunk the state
                               entering it, and e_t of its steps (0 behind the last) */
    int64_t q_token, q_batch, k_token, k_batch, v_token, v_batch;
    void *workspace;        /* device scratch of workspace_bytes, 256-aligned  */
    size_t workspace_bytes; /* >= ssm_gated_delta_workspace_size(args)         */
    float scale;            /* of the outputs; finite                          */
} ssm_gated_delta_args_t;

/* Workspace bytes (the size fields and io_dtype are read); (size_t)-1 for invalid sizes. */
size_t ssm_gated_delta_workspace_size(const ssm_gated_delta_args_t *args);

/* Outputs must not overlap any input, each other or the workspace.  L == 0 copies
 * h0 (or zeros) to h_final. */
ssm_status_t ssm_gated_delta_fwd(const ssm_gated_delta_args_t *args, void *stream);

/*
 * Its gradients for dL/do = dout and dL/dh_final = dh_final.  The chunks' inner
 * matrices are formed again; states and errors come from the forward's
 * checkpoints (computed once more when none are given).  Gradients of shared
 * heads are summed in a fixed order; dense outputs.
 */
typedef struct ssm_gated_delta_bwd_args {
    int64_t batch, seqlen, kheads, heads, kdim, vdim; /* as in ssm_gated_delta_args_t */
    int32_t io_dtype, l2norm;
    const void *q, *k, *v;  /* forward inputs                                  */
    const float *g;
    const void *beta;
    const uint8_t *reset;
    const float *h0;
    const void *dout;       /* (B,L,H,V) io_dtype, dense, required             */
    const float *dh_final;  /* (B,H,K,V) fp32, or NULL (= 0)                   */
    const float *checkpoints; /* of an ssm_gated_delta_fwd call on the same inputs, 16-byte
                                 aligned, or NULL                              */
    void *dq, *dk;          /* (B,L,Hk,K) io_dtype outputs, required           */
    void *dv;               /* (B,L,H,V) io_dtype output, required             */
    float *dg;              /* (B,L,H) fp32 output, required                   */
    void *dbeta;            /* (B,L,H) io_dtype output, required               */
    float *dh0;             /* (B,H,K,V) fp32 output, or NULL                  */
    int64_t q_token, q_batch, k_token, k_batch, v_token, v_batch;
    void *workspace;
    size_t workspace_bytes; /* >= ssm_gated_delta_bwd_workspace_size(args)     */
    float scale;
} ssm_gated_delta_bwd_args_t;

/* Workspace bytes (the size fields, io_dtype and whether checkpoints are given are read);
 * (size_t)-1 for invalid sizes. */
size_t ssm_gated_delta_bwd_workspace_size(const ssm_gated_delta_bwd_args_t *args);

/* Outputs must not overlap any input, each other or the workspace; every output
 * given is overwritten. */
ssm_status_t ssm_gated_delta_bwd(const ssm_gated_delta_bwd_args_t *args, void *stream);

/*
 * One decode step on a state kept between calls (h_final of a prefill), advanced
 * IN PLACE; a row with reset[b] != 0 begins anew.  x_batch: distance of two batch
 * rows of q, k or v, < 2^24; 0 for dense ones.
 */
typedef struct ssm_gated_delta_step_args {
    int64_t batch, kheads, heads, kdim, vdim;
    int32_t io_dtype, l2norm;
    float *state;           /* (B,H,K,V) fp32, 16-byte aligned, required       */
    const void *q, *k;      /* (B,Hk,K) io_dtype, required                     */
    const void *v;          /* (B,H,V) io_dtype, required                      */
    const float *g;         /* (B,H) fp32, required                            */
    const void *beta;       /* (B,H) io_dtype, required                        */
    const uint8_t *reset;   /* (B) bytes, or NULL                              */
    void *o;                /* (B,H,V) io_dtype output, required               */
    int64_t q_batch, k_batch, v_batch;
    float scale;
} ssm_gated_delta_step_args_t;

/* o must not overlap any input or the state, nor the state an input. */
ssm_status_t ssm_gated_delta_step(const ssm_gated_delta_step_args_t *args, void *stream);

/*
 * 8-bit values (OCP e4m3: 3 bits behind the leading one, up to 448, no infinity)
 * with a scale for each block of SSM_FP8_BLOCK consecutive columns and one row, or
 * as many rows.  For a block with largest magnitude m:
 *   scale = max(m, 2^-100) / 448,   q = e4m3(x / scale), to nearest even
 * so q * scale stands for x.  A block that holds an infinity or a NaN has a scale
 * that is none either, and all of it stands for NaN.  The last blocks of a matrix
 * may be shorter.
 */
#define SSM_FP8_BLOCK 128

typedef struct ssm_quantize_fp8_args {
    int64_t rows;           /* M >= 0; M * ceil(D/128) < 2^28                  */
    int64_t dim;            /* D: a multiple of 16, 16 <= D <= 2^20            */
    int64_t block_rows;     /* 1, or SSM_FP8_BLOCK                             */
    int32_t io_dtype;       /* ssm_dtype_t of x                                */
    const void *x;          /* (M,D) io_dtype, required                        */
    void *q;                /* (M,D) e4m3 bytes, 16-byte aligned, required     */
    float *scales;          /* (ceil(M/block_rows), ceil(D/128)) fp32, required */
} ssm_quantize_fp8_args_t;

/* Outputs must not overlap x or each other. */
ssm_status_t ssm_quantize_fp8(const ssm_quantize_fp8_args_t *args, void *stream);

/*
 * ssm_add_rmsnorm_fwd with y quantised as by ssm_quantize_fp8 with block_rows 1,
 * from its fp32 values: q (rows,D) e4m3 bytes and scales (rows, ceil(D/128)) fp32.
 * `norm` is that function's struct with y NULL, and a dim that is a multiple of 16;
 * rows * ceil(D/128) < 2^28.
 */
typedef struct ssm_add_norm_fp8_args {
    ssm_add_norm_args_t norm;
    void *q;                /* 16-byte aligned, required                       */
    float *scales;          /* required                                        */
} ssm_add_norm_fp8_args_t;

/* Outputs must not overlap an input (but res_out may be residual) or each other. */
ssm_status_t ssm_add_rmsnorm_fp8(const ssm_add_norm_fp8_args_t *args, void *stream);

/*
 * The product of 8-bit matrices, y = x w^T:
 *   y[m,n] = sum_j x_scales[m,j] w_scales[n/128,j] sum_{k in block j} xq[m,k] wq[n,k]
 * Sums are fp32; y is rounded once.  x is quantised by rows of 1, w by rows of 128.
 * For a bf16 y a block's 128 terms are summed by the 8-bit matrix instruction, which
 * aligns eight products at a time to the largest and drops what lies 2^14 below it:
 * beside its rounding y is off by less than 7 * 2^-14 sum |x w|.  For random data
 * that is 1.5e-5 of y, where the rounding is 2e-3; where large terms cancel, or one
 * channel stands far above the others, it may be more than the rounding.  For an
 * fp32 y the terms are summed in fp32 and nothing is dropped.
 * A block's two scales are multiplied first, in fp32: a product below 2^-126 loses
 * digits of the block's part, one of 2^128 or more is infinite.
 */
typedef struct ssm_matmul_fp8_args {
    int64_t m, n, k;        /* M >= 0; 1 <= N < 2^24; K: a multiple of 16 up to 2^20;
                               ceil(M/256) * ceil(N/256) < 2^22                */
    int32_t out_dtype;      /* ssm_dtype_t of y                                */
    const void *xq;         /* (M,K) e4m3 bytes, 16-byte aligned, required     */
    const float *x_scales;  /* (M, ceil(K/128)) fp32, required                 */
    const void *wq;         /* (N,K) e4m3 bytes, 16-byte aligned, required     */
    const float *w_scales;  /* (ceil(N/128), ceil(K/128)) fp32, required       */
    void *y;                /* (M,N) out_dtype, required                       */
} ssm_matmul_fp8_args_t;

/* y must not overlap an input. */
ssm_status_t ssm_matmul_fp8(const ssm_matmul_fp8_args_t *args, void *stream);

/* Static description of a status code (never NULL). */
const char *ssm_status_string(ssm_status_t status);

/* Description of the last failure returned on the calling thread ("" if none). */
const char *ssm_last_error_message(void);

/* SSM_ABI_VERSION of the built library. */
int ssm_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SSM_MI355X_H */
