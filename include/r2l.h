/*
 * r2l.h — C ABI of libr2l, the B200 (sm_100a) R2L sidecar forward.
 *
 * The operation is the reverse-direction Mamba stream of "Bifocal Diffusion
 * Language Models: Asymmetric Bidirectional Context for Parallel Generation"
 * (arXiv 2606.27732v1), §3.4 "R2LM Architecture", steps ❶–❹: for hidden
 * states h ∈ R^{B×L×d},
 *
 *     h⁺ = h + tanh(s) · LN( flip( Mamba( flip(h) ) ) )
 *
 * where Mamba is the Mamba-1 selective-scan block (step ❷; d_state = 16,
 * d_conv = 4, expand 2 per §4.1) and LN is a LayerNorm local to the stream
 * (step ❸).  With flip applied per sequence to its valid prefix, the block
 * runs from each sequence's last valid token to its first:
 *
 *     [x | z] = h·W_inᵀ
 *     u_i     = SiLU(conv_b + Σ_{k=0..3} conv_w[:, 3-k] ⊙ x_{i+k})   (x_j = 0, j ≥ len)
 *     [Δr | B | C]_i = u_i·W_xᵀ
 *     Δ_i     = softplus(Δr_i·W_dtᵀ + dt_b)
 *     H_i     = exp(Δ_i ⊗ A) ⊙ H_{i+1} + (Δ_i ⊙ u_i) ⊗ B_i,   H_len = 0,  A = -exp(A_log)
 *     y_i     = (H_i·C_i + D ⊙ u_i) ⊙ SiLU(z_i)
 *     o_i     = y_i·W_outᵀ
 *     h_i    += tanh(s) · (γ ⊙ (o_i − mean) / sqrt(var + 1e-5) + β)      (0 ≤ i < len)
 *
 * Conventions (all entry points):
 *   - Every pointer in a forward call is a DEVICE pointer owned by the caller,
 *     except the r2l_dims / r2l_weights / r2l_debug_out structs themselves,
 *     which are host memory read during the call only.  The library never
 *     allocates, frees or synchronises on the forward path.
 *   - Work is enqueued on `stream` (a cudaStream_t passed as void*; NULL is
 *     the legacy default stream) and runs asynchronously.  Errors found on the
 *     host are returned as r2l_status before anything is enqueued; nothing is
 *     thrown and nothing is printed.
 *   - Matrices are row-major, nn.Linear convention W[out][in].
 *   - The library holds no mutable global state; calls on different streams
 *     with different workspaces may run concurrently.  Two calls that share a
 *     workspace must be ordered by the caller.
 */
#ifndef R2L_H
#define R2L_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define R2L_ABI_VERSION 1

#if defined(__GNUC__)
#define R2L_API __attribute__((visibility("default")))
#else
#define R2L_API
#endif

typedef enum {
  R2L_OK = 0,
  R2L_ERR_INVALID_ARG = 1,   /* null pointer, non-positive size, bad enum */
  R2L_ERR_UNSUPPORTED = 2,   /* d_state != 16, d_conv != 4, or a size the kernels do not tile */
  R2L_ERR_ALIGNMENT = 3,     /* a pointer is not 16-byte aligned */
  R2L_ERR_WORKSPACE = 4,     /* workspace NULL or smaller than r2l_workspace_size() */
  R2L_ERR_CUDA = 5,          /* a CUDA runtime call or launch failed */
  R2L_ERR_DEVICE_CHECK = 6   /* r2l_get_device_status found a device-side flag */
} r2l_status;

typedef enum {
  R2L_BF16 = 0,   /* bf16 activations and GEMM weights, fp32 accumulation and state */
  R2L_FP32 = 1    /* fp32 everywhere, true fp32 arithmetic (no TF32) */
} r2l_dtype;

/* r2l_dims.flags
 *
 * The scan's power path (bf16 path only).  When A is the S4D-real
 * initialisation A[c][m] = -(m+1), the 16 decays exp(Δ·A[c][m]) of a (position,
 * channel) are the powers r, r², …, r¹⁶ of r = exp(-Δ), so the scan needs one
 * reciprocal instead of 16 exponentials.  The choice is made once per call
 * (per hook of r2l_sidecar_stack), on the device, by an exact test: the power
 * path is taken when every A_log[c][m] equals, bit for bit, the float nearest
 * ln(m+1), and the scan then uses A[c][m] = -(m+1) exactly (it differs from
 * -exp(A_log[c][m]) by less than 2e-7 relative).  Any other A_log, even one
 * entry, sends the whole call down the general path (one exponential per
 * state).  R2L_FLAG_GENERAL_A skips the test and always takes the general
 * path.  The fp32 path always evaluates exp(Δ·A) directly.                   */
#define R2L_FLAG_GENERAL_A 0x1u     /* never take the A = -(1..16) power fast path of the scan    */
#define R2L_FLAG_FORWARD_SCAN 0x2u  /* run the block left to right instead: causal conv and a
                                       forward scan (the "L2R Mamba" control of Table 4); every
                                       other step is unchanged                                    */
#define R2L_FLAG_SAVED_FORWARD 0x4u /* r2l_sidecar_backward only: the workspace holds this hook's
                                       forward from r2l_sidecar_forward_train, so the forward is
                                       not recomputed                                             */
#define R2L_FLAG_ACT8 0x8u          /* r2l_gated_scan_train and its gradient only: the checkpoint also
                                       keeps x, r and g, in 8 bits (see r2l_act8_pack)            */
/* Device status bits, reported by r2l_get_device_status(). */
#define R2L_DEVFLAG_LENGTH_CLAMPED 0x1u   /* a lengths[b] was outside [0, L] and was clamped */
#define R2L_DEVFLAG_TIMEOUT 0x2u          /* a kernel gave up waiting on a pipeline barrier (results invalid) */

typedef struct {
  int d_model;       /* d: hidden width of the backbone                             */
  int d_inner;       /* E: expanded width (2·d_model in the paper's setup)         */
  int d_state;       /* N: SSM state size; must be 16                              */
  int dt_rank;       /* R: rank of the Δ projection                                */
  int d_conv;        /* W: depthwise conv width; must be 4                         */
  r2l_dtype dtype;   /* activation / GEMM-weight storage type                      */
  unsigned flags;    /* R2L_FLAG_* bits, 0 by default                              */
} r2l_dims;

/* One hook's parameters.  Device pointers, read-only, 16-byte aligned.
 * "act" = bf16 for R2L_BF16, fp32 for R2L_FP32.                               */
typedef struct {
  const void  *in_proj_w;   /* act  [2E, d]   rows 0..E-1 produce x, rows E..2E-1 produce z */
  const float *conv_w;      /* fp32 [E, W]    tap W-1 multiplies the current token          */
  const float *conv_b;      /* fp32 [E]                                                      */
  const void  *x_proj_w;    /* act  [R+2N, E] output rows ordered Δr | B | C                 */
  const void  *dt_proj_w;   /* act  [E, R]                                                   */
  const float *dt_proj_b;   /* fp32 [E]                                                      */
  const float *A_log;       /* fp32 [E, N]    A = -exp(A_log)                                */
  const float *D;           /* fp32 [E]                                                      */
  const void  *out_proj_w;  /* act  [d, E]                                                   */
  const float *ln_w;        /* fp32 [d]  LayerNorm γ; ln_w = ln_b = NULL: no LayerNorm       */
  const float *ln_b;        /* fp32 [d]  LayerNorm β                                         */
} r2l_weights;

/* Optional intermediates for testing (device pointers, NULL = not wanted).
 * Row b·L + i holds position i of sequence b; rows with i ≥ len_b hold
 * unspecified values, except in hhat where they are not written.             */
typedef struct {
  void  *x;        /* act  [B·L, E]      in_proj, first half                  */
  void  *z;        /* act  [B·L, E]      in_proj, second half                 */
  void  *u;        /* act  [B·L, E]      conv + SiLU                          */
  float *dbc;      /* fp32 [B·L, R+2N]   x_proj output Δr | B | C             */
  void  *y;        /* act  [B·L, E]      scan output after the SiLU(z) gate   */
  void  *o;        /* act  [B·L, d]      out_proj output                      */
  float *hhat;     /* fp32 [B·L, d]      LayerNorm output (pre-gate)          */
} r2l_debug_out;

/* ABI version of the loaded library (R2L_ABI_VERSION at build time). */
R2L_API int r2l_abi_version(void);

/* Human-readable name of a status code; never NULL, static storage. */
R2L_API const char *r2l_status_string(r2l_status status);

/* Bytes of device workspace a forward call on a [B, L] batch needs.  Returns 0
 * for invalid dims or sizes.  The size depends only on (dims, B, L).          */
R2L_API size_t r2l_workspace_size(const r2l_dims *dims, int B, int L);

/* The sidecar forward of §3.4 on hidden [B, L, d_model] (act dtype), updated in
 * place: rows i < len_b become h⁺, rows i ≥ len_b are neither read nor written.
 *
 *   lengths   device int32 [B] of valid lengths, or NULL for all L.  Values
 *             outside [0, L] are clamped on the device and flagged
 *             (R2L_DEVFLAG_LENGTH_CLAMPED, see r2l_get_device_status).
 *   s         the hook's scalar gate; g = tanh(s) is formed in double on the
 *             host and rounded to float.  If g == 0 the call returns R2L_OK
 *             without enqueuing anything (the identity at initialisation, §3.4 ❹).
 *   workspace device scratch of at least r2l_workspace_size(dims, B, L) bytes,
 *             16-byte aligned, caller-owned; its contents on entry do not
 *             matter and on return are unspecified (the device status word
 *             lives at its start).
 * Checks on the host: non-null pointers, positive sizes, d_state == 16,
 * d_conv == 4, 16-byte alignment, workspace size, supported tiling.  On any
 * error nothing is enqueued.                                                   */
R2L_API r2l_status r2l_sidecar_forward(void *hidden, const r2l_weights *weights, const r2l_dims *dims,
                               float s, int B, int L, const int32_t *lengths,
                               void *workspace, size_t workspace_bytes, void *stream);

/* Same as r2l_sidecar_forward, and also copies the intermediates requested in
 * *debug (non-NULL fields) into the caller's buffers.  For tests.  Unlike the
 * forward call it runs the layer even when tanh(s) == 0.                       */
R2L_API r2l_status r2l_sidecar_forward_debug(void *hidden, const r2l_weights *weights, const r2l_dims *dims,
                                     float s, int B, int L, const int32_t *lengths,
                                     void *workspace, size_t workspace_bytes, void *stream,
                                     const r2l_debug_out *debug);

/* n_hooks sidecar layers applied one after another to the same hidden tensor
 * (§4.1: a hook after every 4th decoder layer; here the backbone between hooks
 * is whatever the caller does between calls, i.e. nothing).  weights and s are
 * host arrays of n_hooks entries.  Same contract as r2l_sidecar_forward.      */
R2L_API r2l_status r2l_sidecar_stack(void *hidden, const r2l_weights *weights, const float *s, int n_hooks,
                             const r2l_dims *dims, int B, int L, const int32_t *lengths,
                             void *workspace, size_t workspace_bytes, void *stream);

/* Stages of one hook, in launch order, for r2l_sidecar_forward_profiled. */
typedef enum {
  R2L_STAGE_IN_PROJ = 0,      /* [x | z] = h·W_inᵀ                              */
  R2L_STAGE_CONV = 1,         /* u = SiLU(anti-causal conv(x))                  */
  R2L_STAGE_X_PROJ = 2,       /* [Δr | B | C] = u·W_xᵀ                          */
  R2L_STAGE_DT_PROJ = 3,      /* Δr·W_dtᵀ                                       */
  R2L_STAGE_SCAN = 4,         /* reverse selective scan and SiLU(z) gate        */
  R2L_STAGE_OUT_PROJ = 5,     /* o = y·W_outᵀ                                   */
  R2L_STAGE_LN_RESIDUAL = 6,  /* LayerNorm and tanh(s)-gated residual           */
  R2L_NUM_STAGES = 7
} r2l_stage;

/* Same as r2l_sidecar_forward, and also records events[k] on `stream` just
 * before stage k starts and events[R2L_NUM_STAGES] after the last stage.
 * events: host array of n_events cudaEvent_t handles (passed as void*),
 * created and owned by the caller; n_events must be R2L_NUM_STAGES + 1.  A
 * stage that is fused into its neighbour shows zero time.  *launches (if not
 * NULL) receives the number of kernels the call enqueued.  For measurement.  */
R2L_API r2l_status r2l_sidecar_forward_profiled(void *hidden, const r2l_weights *weights,
                                        const r2l_dims *dims, float s, int B, int L,
                                        const int32_t *lengths, void *workspace,
                                        size_t workspace_bytes, void *stream,
                                        void *const *events, int n_events, int *launches);

/* Bytes of device workspace r2l_reverse_scan needs for a [B, L] batch split
 * into chunks of chunk_tokens tokens (0 = automatic).  0 for invalid input. */
R2L_API size_t r2l_reverse_scan_workspace_size(const r2l_dims *dims, int B, int L, int chunk_tokens);

/* The selective scan of §3.4 step ❷ on its own (the Mamba-1 scan, run from
 * each sequence's last valid token to its first) followed by the SiLU(z) gate:
 *
 *     Δ_i = softplus(dt_raw_i + dt_b);  H_i = exp(Δ_i ⊗ A) ⊙ H_{i+1} + (Δ_i ⊙ u_i) ⊗ B_i;
 *     y_i = (H_i·C_i + D ⊙ u_i) ⊙ SiLU(z_i),   H entering position len_b − 1 is 0.
 *
 *   u        act  [B·L, E]     (row stride E)
 *   z        act  [B·L, ldz]   first E columns are z
 *   dt_raw   act  [B·L, E]     Δr·W_dtᵀ, before bias and softplus
 *   bc       fp32 [B·L, ldbc]  B in columns 0..15, C in columns 16..31
 *   A_log    fp32 [E, 16],  D, dt_b  fp32 [E]
 *   y        act  [B·L, E]     output; rows i ≥ len_b are not written
 *   lengths  as for r2l_sidecar_forward
 *   chunk_tokens  bf16 path: tokens per chunk when sequences are split for
 *            parallelism (rounded up to a multiple of 16; 0 = automatic).
 *            Ignored by the fp32 path, which scans each sequence whole.
 *   workspace  ≥ r2l_reverse_scan_workspace_size(dims, B, L, chunk_tokens) bytes,
 *            16-byte aligned (chunk carries and the device status word).
 * Device pointers, 16-byte aligned; ldz a multiple of 8 and ldbc of 4.        */
R2L_API r2l_status r2l_reverse_scan(const void *u, const void *z, int ldz, const void *dt_raw,
                                    const float *bc, int ldbc, const float *A_log, const float *D,
                                    const float *dt_b, void *y, const r2l_dims *dims, int B, int L,
                                    const int32_t *lengths, int chunk_tokens, void *workspace,
                                    size_t workspace_bytes, void *stream);

/* Capacity, in bytes, of the scratch array behind r2l_reverse_scan_noalloc. */
#define R2L_NOALLOC_SCRATCH_BYTES (16u << 20)

/* r2l_reverse_scan without a workspace argument, for callers that cannot
 * allocate device memory while they run: for example a serving runtime that
 * reserves all device memory when it starts and forbids allocation while it
 * handles requests, or a plug-in whose host program owns the CUDA context and
 * its allocator.  It computes exactly what r2l_reverse_scan computes.  (The
 * paper has no counterpart; this entry point exists for such callers only.)
 *
 * Its scratch (status word, clamped lengths, chunk carries) is a fixed array
 * of R2L_NOALLOC_SCRATCH_BYTES that the library's device code declares; every
 * device that loads the library holds it until the process exits.  The entry
 * point calls no cudaMalloc, cudaFree or other allocating routine.
 *   - Every call looks up the array's device address in the current device's
 *     context (cudaGetSymbolAddress; nothing is allocated), so the address
 *     stays right after cudaDeviceReset.  The first call on a device also
 *     loads the library's device image into that context; make that first
 *     call before any stream capture.
 *   - All calls share the one array, which keeps the last call's contents
 *     (each call rewrites what it reads).  Calls whose work overlaps on the
 *     GPU (for instance on two streams) race on it; order them.
 *   - A request that needs more scratch than the array holds
 *     (r2l_reverse_scan_workspace_size() > R2L_NOALLOC_SCRATCH_BYTES) returns
 *     R2L_ERR_WORKSPACE and enqueues nothing.  A smaller chunk count (larger
 *     chunk_tokens) needs less scratch; one chunk per sequence needs almost none.
 * r2l_get_device_status cannot read this scratch; use r2l_reverse_scan when
 * device-side flags matter.  Other arguments and errors as r2l_reverse_scan. */
R2L_API r2l_status r2l_reverse_scan_noalloc(const void *u, const void *z, int ldz, const void *dt_raw,
                                            const float *bc, int ldbc, const float *A_log, const float *D,
                                            const float *dt_b, void *y, const r2l_dims *dims, int B, int L,
                                            const int32_t *lengths, int chunk_tokens, void *stream);

/* Bytes of device workspace r2l_reverse_scan_backward needs for a [B, L]
 * batch split into chunks of chunk_tokens positions (0 = automatic, 16).
 * 0 for invalid or unsupported input (see r2l_reverse_scan_backward).       */
R2L_API size_t r2l_reverse_scan_backward_workspace_size(const r2l_dims *dims, int B, int L, int chunk_tokens);

/* Gradient of r2l_reverse_scan (the scan of §3.4 step ❷ with its softplus(Δ)
 * input and SiLU(z) gate), the step that training the sidecar alone
 * back-propagates through.  For dy = ∂L/∂y it returns, with the forward's
 * notation (a_i = exp(Δ_i A), G_i = ∂L/∂H_i = a_{i-1} ⊙ G_{i-1} + dp_i C_i,
 * dp_i = dy_i ⊙ SiLU(z_i)):
 *
 *   du      [B·L, E]   D ⊙ dp_i + Δ_i ⊙ Σ_m G_i[:,m] B_i[m]
 *   ddt_raw [B·L, E]   (Σ_m G_i ⊙ H_{i+1} ⊙ a_i ⊙ A + u_i ⊙ Σ_m G_i B_i) ⊙ softplus'(dt_raw_i + dt_b)
 *   dz      [B·L, ld_dz] first E columns: dy_i ⊙ p_i ⊙ SiLU'(z_i), p_i = H_i·C_i + D ⊙ u_i
 *   dbc     [B·L, ld_dbc] columns 0..15 dB_i = Σ_e G_i Δ_i u_i, 16..31 dC_i = Σ_e dp_i H_i
 *   dA_log  [E, 16]    A ⊙ Σ_i Δ_i ⊙ G_i ⊙ H_{i+1} ⊙ a_i   (summed over the batch)
 *   dD, ddt_b [E]      Σ_i dp_i ⊙ u_i,  Σ_i ddt_raw_i        (summed over the batch)
 *
 * Rows i ≥ len_b of du, ddt_raw, dz and dbc are written with zeros.  Inputs
 * are those of r2l_reverse_scan (u, z, dt_raw, bc, A_log, D, dt_b, lengths)
 * plus dy [B·L, E].  Every reduction runs in a fixed order: the results are
 * bitwise reproducible for a given chunk_tokens.
 *
 * Supported: dims->dtype R2L_FP32 (every array fp32) or R2L_BF16 (u and z
 * bf16 as the bf16 forward stores them, every other array fp32), d_state == 16, d_inner a multiple of 64, B and L up to 65535 with
 * B·⌈L / chunk⌉ ≤ 2,097,120 (grid limits), the right-to-left block (the
 * R2L_FLAG_FORWARD_SCAN flag returns R2L_ERR_UNSUPPORTED); ldz, ld_dz and
 * ldbc multiples of 4.  chunk_tokens: positions per chunk (1 … 32; larger values are
 * clamped to 32; 0 = 16).  workspace ≥
 * r2l_reverse_scan_backward_workspace_size(dims, B, L, chunk_tokens) bytes,
 * 16-byte aligned; its first 16 bytes are the device status word that
 * r2l_get_device_status reads.  Device pointers, 16-byte aligned.          */
R2L_API r2l_status r2l_reverse_scan_backward(const void *u, const void *z, int ldz, const void *dt_raw,
                                             const float *bc, int ldbc, const float *A_log, const float *D,
                                             const float *dt_b, const void *dy, void *du, void *dz, int ld_dz,
                                             void *ddt_raw, float *dbc, int ld_dbc, float *dA_log, float *dD,
                                             float *ddt_b, const r2l_dims *dims, int B, int L,
                                             const int32_t *lengths, int chunk_tokens, void *workspace,
                                             size_t workspace_bytes, void *stream);

/* Gradients of one hook's parameters: fp32 device arrays, 16-byte aligned,
 * caller-owned, each shaped like the matching field of r2l_weights (in_proj_w
 * [2E, d], conv_w [E, W], conv_b [E], x_proj_w [R+2N, E], dt_proj_w [E, R],
 * dt_proj_b [E], A_log [E, N], D [E], out_proj_w [d, E], ln_w and ln_b [d]).
 * ln_w / ln_b may be NULL when the hook has no LayerNorm.  Every array is
 * written in full (not accumulated into).                                    */
typedef struct {
  float *in_proj_w, *conv_w, *conv_b, *x_proj_w, *dt_proj_w, *dt_proj_b, *A_log, *D, *out_proj_w, *ln_w, *ln_b;
} r2l_grads;

/* Bytes of device workspace r2l_sidecar_backward needs for a [B, L] batch;
 * 0 for invalid or unsupported input.                                        */
R2L_API size_t r2l_sidecar_backward_workspace_size(const r2l_dims *dims, int B, int L);

/* The gradient of one hook (§3.4 steps ❶–❹), the step that training the
 * sidecar alone (the paper's R2LM-PI setting, §3.4 and §4.1) back-propagates
 * through.  For the hook's input hidden [B, L, d] (act dtype, as given to
 * r2l_sidecar_forward) and dh_out = ∂L/∂h⁺ (fp32 [B, L, d]) it writes
 *
 *   dh    fp32 [B, L, d]  ∂L/∂h: dh_out on padding rows (the hook neither reads
 *                          nor writes them), dh_out + ∂L/∂h through the sidecar
 *                          on valid rows
 *   *ds   fp32 scalar     ∂L/∂s = (1 − tanh²(s)) Σ dh_out ⊙ ĥ (device pointer)
 *   grads                 ∂L/∂(every parameter), summed over the batch
 *
 * The forward is recomputed into the workspace (unless R2L_FLAG_SAVED_FORWARD
 * says r2l_sidecar_forward_train left it there), then the chain rule runs in
 * reverse: gate, LayerNorm, out_proj, the scan (bf16 u and z, fp32 state),
 * dt_proj, x_proj, conv + SiLU, in_proj.  GEMM operands are bf16 (gradients
 * rounded once to bf16 where they feed a GEMM), accumulation fp32; every
 * reduction over positions runs in a fixed order, so results are bitwise
 * reproducible.
 *
 * Supported: dims->dtype R2L_BF16, d_state 16, d_conv 4, d_model and dt_rank
 * multiples of 8, d_inner a multiple of 64, the right-to-left block
 * (R2L_FLAG_FORWARD_SCAN returns R2L_ERR_UNSUPPORTED).  workspace ≥
 * r2l_sidecar_backward_workspace_size(dims, B, L) bytes, 16-byte aligned; its
 * first 16 bytes are the status word r2l_get_device_status reads.  Other
 * arguments, conventions and errors as r2l_sidecar_forward; hidden is not
 * written.                                                                     */
R2L_API r2l_status r2l_sidecar_backward(const void *hidden, const r2l_weights *weights, const r2l_dims *dims,
                                        float s, int B, int L, const int32_t *lengths, const float *dh_out,
                                        float *dh, float *ds, const r2l_grads *grads, void *workspace,
                                        size_t workspace_bytes, void *stream);

/* The hook's forward for training (the R2LM-PI setting, §3.4 and §4.1):
 * out = h⁺ = h + tanh(s)·ĥ as r2l_sidecar_forward computes it, written to
 * `out` (act dtype [B, L, d], 16-byte aligned, not aliasing hidden: padding
 * rows are copied from hidden; hidden is not written, since the gradient reads
 * it again), and everything r2l_sidecar_backward needs left in `workspace`
 * (≥ r2l_sidecar_backward_workspace_size(dims, B, L) bytes): the forward's
 * intermediates, dt_raw in fp32, and the H checkpoints of its scan gradient
 * (every 16 positions, for sequences whose length is a multiple of 16, with
 * dt_rank 128).  A later r2l_sidecar_backward with R2L_FLAG_SAVED_FORWARD in
 * dims->flags and the same hidden, weights, other dims, s, B, L, lengths and
 * workspace (untouched in between) skips its recomputation of the forward.
 * Supported shapes and errors as r2l_sidecar_backward; out == hidden returns
 * R2L_ERR_INVALID_ARG.  Runs the layer even when tanh(s) == 0 (the gradient
 * needs ĥ for ds).                                                            */
R2L_API r2l_status r2l_sidecar_forward_train(const void *hidden, void *out, const r2l_weights *weights,
                                             const r2l_dims *dims, float s, int B, int L, const int32_t *lengths,
                                             void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * A gated linear recurrence: one state per channel, whose decay and input are
 * gated position by position by two projections of the layer's input.  For an
 * input x, a recurrence gate r and an input gate g (all before the sigmoid) and
 * a decay parameter lam per channel, at position k of the scan order,
 *
 *     log a_k = -R2L_GATED_RATE · softplus(lam) · σ(r_k)
 *     h_k     = a_k ⊙ h_{k-1} + sqrt(1 − a_k²) ⊙ σ(g_k) ⊙ x_k,      y_k = h_k
 *
 * The scan runs from each sequence's last valid position to its first, as
 * r2l_reverse_scan does, or the other way with R2L_FLAG_FORWARD_SCAN.  A state
 * may enter (h0) and leave (h_last), so a sequence can be scanned in pieces, a
 * piece of one position being one step of decoding.  r = −∞ closes the
 * recurrence gate: a_k = 1, and the position, its x being finite, leaves the
 * state as it was (0 times an infinity or a NaN is NaN here as elsewhere).
 * lam = −∞ keeps the state throughout, lam = +∞ forgets it at any gate that is
 * not closed (softplus(lam) is held to 2^124, and a σ(r) below 2^-126 may count
 * as closed).  State, gates and sums are fp32 for both dtypes.
 *
 * r2l_dims: d_inner is the number of channels E (any positive number), dtype
 * the type of the [B·L, ·] arrays, flags R2L_FLAG_FORWARD_SCAN and
 * R2L_FLAG_ACT8; the other fields are not read.
 *
 * Arrays of rows have a row stride (ld…) in elements, at least E, so that they
 * can be columns of a wider array; row b·L + i is position i of sequence b.
 * Pointers need the alignment of their element type only; a call whose arrays
 * of rows all start on 16-byte boundaries with strides that are multiples of
 * 16 bytes runs faster.  Between the start of an array's first row and the
 * end of its last one, up to 15 bytes beside a row's E columns may be read
 * (nothing depends on them); they are never written.  No output may overlap an
 * input, except h_last = h0 and dh0 = dh_last.  lengths as for
 * r2l_sidecar_forward (clamped to [0, L]; a sequence of length 0 passes its
 * state through).  E and L up to 2^30 and B · L · E up to 2^50; more returns
 * R2L_ERR_UNSUPPORTED.
 * ------------------------------------------------------------------------- */
#define R2L_GATED_RATE 8.0f
#define R2L_GATED_TILE 64   /* positions between two states of a checkpoint */

typedef struct {
  const void *x;      /* act  [B·L, ldx]                                        */
  const void *r;      /* act  [B·L, ldr]  recurrence gate, before the sigmoid   */
  const void *g;      /* act  [B·L, ldg]  input gate, before the sigmoid        */
  int ldx, ldr, ldg;
  const float *lam;   /* fp32 [E]                                               */
  const float *h0;    /* fp32 [B, E] state that enters the scan, NULL: 0        */
} r2l_gated_in;

typedef struct {
  void *dx, *dr, *dg;           /* act [B·L, ld…]; rows i ≥ len_b are written with zeros  */
  int ld_dx, ld_dr, ld_dg;
  float *dlam;                  /* fp32 [E], summed over the batch                        */
  float *dh0;                   /* fp32 [B, E], or NULL: not wanted                       */
} r2l_gated_grads;

/* The recurrence.  y: act [B·L, ldy], rows i ≥ len_b are not written.  h_last:
 * fp32 [B, E], the state that leaves the scan, or NULL; it may be in->h0.
 * status: device word that receives the R2L_DEVFLAG_* bits of this call (what
 * r2l_get_device_status reads), or NULL.  No workspace is needed, and nothing
 * is enqueued on an error.  A sequence's result does not depend on the other
 * sequences' values; it is bitwise reproducible for given B, L and E and
 * lengths given or not, which choose how the work is cut.                    */
R2L_API r2l_status r2l_gated_scan(const r2l_gated_in *in, void *y, int ldy, float *h_last, const r2l_dims *dims,
                                  int B, int L, const int32_t *lengths, uint32_t *status, void *stream);

/* Bytes of the checkpoint that r2l_gated_scan_train writes; 0 for invalid
 * input.  Without R2L_FLAG_ACT8 it holds the state that enters every
 * R2L_GATED_TILE-th position of the scan order (fp32, 1/16 byte per position
 * and channel); with it also x, r and g as r2l_act8_pack packs them (3 + 3/64
 * bytes per position and channel), after the same states; but an r or g counts
 * for its scale up to ±256 only, and what lies beyond, infinite or finite, is
 * kept as a value from ±256 to ±448, which closes or opens that gate just the
 * same.  Channels are rounded up to R2L_ACT8_GROUP.                          */
R2L_API size_t r2l_gated_scan_checkpoint_size(const r2l_dims *dims, int B, int L);

/* r2l_gated_scan for training: also writes `checkpoint`
 * (≥ r2l_gated_scan_checkpoint_size(dims, B, L) bytes, 16-byte aligned,
 * caller-owned), which r2l_gated_scan_backward reads.                        */
R2L_API r2l_status r2l_gated_scan_train(const r2l_gated_in *in, void *y, int ldy, float *h_last, const r2l_dims *dims,
                                        int B, int L, const int32_t *lengths, void *checkpoint,
                                        size_t checkpoint_bytes, uint32_t *status, void *stream);

/* Bytes of workspace of r2l_gated_scan_backward; 0 for invalid input. */
R2L_API size_t r2l_gated_scan_backward_workspace_size(const r2l_dims *dims, int B, int L);

/* Gradient of r2l_gated_scan.  For dy = ∂L/∂y (act [B·L, ld_dy]) and dh_last =
 * ∂L/∂h_last (fp32 [B, E], NULL: 0), with G_k = ∂L/∂h_k = dy_k + a_{k+1} G_{k+1}
 * and β = sqrt(1 − a²):
 *
 *   dx = G ⊙ β ⊙ σ(g)                    dg = G ⊙ β ⊙ x ⊙ σ(g)(1 − σ(g))
 *   d(log a) = G ⊙ (a ⊙ h_{k-1} − σ(g) ⊙ x ⊙ a²/β)       (0 where log a = 0)
 *   dr = d(log a) ⊙ log a ⊙ (1 − σ(r))   dlam = Σ d(log a) ⊙ σ(r) · (−R2L_GATED_RATE σ(lam))
 *   dh0 = a_0 ⊙ G_0
 *
 * in: x, r, g and lam as given to the forward (h0 is not read: the checkpoint
 * has it).  With R2L_FLAG_ACT8 x, r and g are not read either and may be NULL;
 * the gradient is then the formula at the values that the checkpoint's 8 bits
 * stand for, each tile's states recomputed from its exact first one.
 * dims, B, L and lengths as given to r2l_gated_scan_train; dims->flags too.
 * Every sum runs in a fixed order: results are bitwise reproducible (with
 * lengths and without, a call may be cut differently).  dr and dlam need
 * σ(g) x a σ(r) / β within fp32's range before G multiplies it (|x| up to 1e37
 * where a memory is of 1000 positions).
 * workspace ≥ r2l_gated_scan_backward_workspace_size(dims, B, L) bytes,
 * 16-byte aligned; its first word is the device status word.                 */
R2L_API r2l_status r2l_gated_scan_backward(const r2l_gated_in *in, const void *dy, int ld_dy, const float *dh_last,
                                           const r2l_gated_grads *grads, const r2l_dims *dims, int B, int L,
                                           const int32_t *lengths, const void *checkpoint, size_t checkpoint_bytes,
                                           void *workspace, size_t workspace_bytes, void *stream);

/* Activation checkpoints in 8 bits: what a training step keeps of an
 * activation between its forward and its gradient (a hook's hidden state for
 * r2l_sidecar_backward, which recomputes the hook's forward from it) in half
 * the bytes of bf16.  A row is cut into groups of R2L_ACT8_GROUP channels (the
 * last one may be shorter).  A group holds x / 2^k rounded to the nearest e4m3
 * value, ties to even, and the byte k + 127, with k ≥ −126 the least integer
 * for which every finite |x| of the group is ≤ 448 · 2^k.  The scale being a
 * power of two, a value that e4m3's 4 significant bits hold comes back as it
 * was, and packing what was unpacked changes nothing.  An infinity or a NaN
 * comes back as NaN; |x| from 248 · 2^120 on, whose nearest value would be
 * 2^128, is held as 240 · 2^120, so that finite values come back finite.     */
#define R2L_ACT8_GROUP 64

/* Packs x (dtype, [B·L, ldx], its first `cols` columns) into q ([B·L, ldq]
 * bytes, e4m3) and scales ([B·L, ⌈cols / R2L_ACT8_GROUP⌉] bytes).  lengths as
 * for r2l_sidecar_forward (NULL: all rows); rows i ≥ len_b are neither read
 * nor written.  The output may not overlap the input, here or in unpacking.  */
R2L_API r2l_status r2l_act8_pack(const void *x, int ldx, r2l_dtype dtype, int B, int L, int cols,
                                 const int32_t *lengths, uint8_t *q, int ldq, uint8_t *scales, void *stream);

/* The values that q and scales stand for, into out (dtype, [B·L, ldo]),
 * rounded to nearest where dtype needs it.  Arguments as r2l_act8_pack.      */
R2L_API r2l_status r2l_act8_unpack(const uint8_t *q, int ldq, const uint8_t *scales, r2l_dtype dtype, int B, int L,
                                   int cols, const int32_t *lengths, void *out, int ldo, void *stream);

/* Synchronises `stream`, then reads the device status word that the last
 * forward call on `workspace` wrote.  *flags_out receives the R2L_DEVFLAG_*
 * bits.  Returns R2L_ERR_DEVICE_CHECK if any bit is set, R2L_ERR_CUDA if the
 * stream reported an error, R2L_OK otherwise.  Not for the hot path.          */
R2L_API r2l_status r2l_get_device_status(const void *workspace, void *stream, uint32_t *flags_out);

#ifdef __cplusplus
}
#endif

#endif /* R2L_H */
