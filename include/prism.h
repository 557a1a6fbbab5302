/*
 * prism.h - C ABI of the PRISM sequence-mixer scan for NVIDIA B200 (sm_100a).
 *
 * The operation (forward only), per batch row b and head h, with the state
 * S in R^{d_v x d_k} (S0, or zeros), m = L - 1 residual steps and a ShortConv of
 * width W:
 *
 *   a_t     = sum_{i<W} conv_w[h,:,i] * v_{t-i}      depthwise causal ShortConv anchor
 *   r_{t,0} = v_t - a_t                               anchor residual
 *   r_{t,l} = (1 - gain_{t,l}) * r_{t,l-1}            linearised residual chain, l = 1..m
 *   S_t     = gamma_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
 *             + sum_l alpha_{t,l} r_{t,l} u_{t,l}^T    gated-delta write + rank-m residual write
 *   o_t     = S_t q_t                                 post-update readout
 *
 * Sources (web pages on PRISM, Parallel Residual Iterative Sequence Model):
 *   - "ICML 2026 | 当线性注意力学会"写入前思考"：并行化的多步记忆写入" (Tencent Ads
 *     write-up): section 核心迭代形式 (the step-size x residual x direction write),
 *     消除 Token 间串行 (forget path kept as GDN, ShortConv anchor replaces the
 *     global state), 消除 Step 间串行 (closed-form element-wise residual chain),
 *     架构形式 (write = GDN write + low-rank residual; L = 1 is exactly GDN),
 *     混合架构是必然 (the anchor window covers the last 3-4 tokens).
 *   - "PRISM: Parallel Residual Iterative Sequence Model" technical summary,
 *     sections 2.1 (S_t = S_{t-1} A_t + B_t, A_t the rank-1 gated-delta
 *     transition) and 2.2 (two-stage proxy: anchor from a short convolution,
 *     then L parallel refinement steps with gain, residual and direction).
 *   - ICML 2026 poster abstract of the same paper (short-convolution anchor,
 *     rank-L accumulation).
 *
 * Conventions shared by every entry point:
 *   - All tensor pointers are DEVICE pointers (except in prism_scan_fwd_host),
 *     owned by the caller.  The library never allocates or frees device memory
 *     and never synchronises, except prism_stream_status.  Work is enqueued on
 *     `stream` (0 = legacy default stream).
 *   - Layouts are dense, row-major, token-major:
 *       q, k    [B, T, H, d_k]          dtype
 *       v       [B, T, H, d_v]          dtype
 *       gamma   [B, T, H]               fp32, decay gate in (0, 1]
 *       beta    [B, T, H]               fp32, delta-rule step size
 *       u       [B, T, H, L-1, d_k]     dtype, residual-write directions (NULL iff L == 1)
 *       alpha   [B, T, H, L-1]          fp32, residual step sizes        (NULL iff L == 1)
 *       gain    [B, T, H, L-1, d_v]     dtype, per-channel gains g       (NULL iff L == 1)
 *       conv_w  [H, d_v, W]             fp32, ShortConv taps, tap i multiplies v_{t-i}
 *       S0      [B, H, d_v, d_k]        fp32 or NULL (zeros)
 *       lengths [B]                     int32 or NULL (every row has T valid steps);
 *                                       right padding: steps t >= lengths[b] leave S
 *                                       unchanged and write o_t = 0
 *       o       [B, T, H, d_v]          dtype (output)
 *       S_final [B, H, d_v, d_k]        fp32 (output) or NULL: state after the last
 *                                       valid step of each row
 *     dtype is PRISM_BF16 (bfloat16) or PRISM_FP32.  Arithmetic is fp32 with an
 *     fp32 state; bf16 outputs are rounded to nearest even.
 *   - Every device pointer must be 16-byte aligned.
 *   - Return value: PRISM_OK or a PRISM_ERR_* code.  All argument checks run
 *     before anything is enqueued; on an error nothing is launched and the
 *     outputs are untouched.  Launch failures return PRISM_ERR_CUDA.  Device-side
 *     errors (a bounded wait that expired) are recorded in a per-device status
 *     word that prism_stream_status reports.
 */
#ifndef PRISM_H_
#define PRISM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* prism_stream_t; /* same type as cudaStream_t */

#define PRISM_VERSION_MAJOR 0
#define PRISM_VERSION_MINOR 1
#define PRISM_VERSION_PATCH 0

enum prism_dtype {
  PRISM_BF16 = 0,
  PRISM_FP32 = 1
};

/* Residual chain step.  Exact: gist.science PRISM explainer, 2.2 Input-Anchored Loop
 * Unrolling (Residual Update).  Linearised: ICML 2026 PRISM write-up, 消除 Step 间串行. */
enum prism_chain {
  PRISM_CHAIN_LINEAR = 0, /* r_l = (1 - g_l) * r_{l-1}: the linearised chain (default) */
  PRISM_CHAIN_GELU = 1    /* r_l = r_{l-1} - GELU(g_l * r_{l-1}), GELU(x) = x Phi(x) (erf form) */
};

/* Activation of the gated norm's gate: g sigmoid(g), or sigmoid(g). */
enum prism_act {
  PRISM_ACT_SILU = 0,
  PRISM_ACT_SIGMOID = 1
};

enum prism_status {
  PRISM_OK = 0,
  PRISM_ERR_INVALID_ARG = 1, /* NULL where required, non-positive size, L < 1, W < 1, ... */
  PRISM_ERR_UNSUPPORTED = 2, /* valid but not implemented: head size, width, alignment, device */
  PRISM_ERR_WORKSPACE = 3,   /* workspace smaller than the call's workspace_size query */
  PRISM_ERR_CUDA = 4,        /* a CUDA runtime call or kernel launch failed */
  PRISM_ERR_TIMEOUT = 5,     /* a bounded device-side wait expired (from prism_stream_status) */
  PRISM_ERR_BOUNDS = 6       /* an id outside the table of prism_embed_fwd / prism_embed_bwd, or,
                                in the debug build, a kernel index outside its buffer; the kernel
                                recorded it and skipped the access (from prism_stream_status) */
};

/* Limits of this build (checked; larger values return PRISM_ERR_UNSUPPORTED). */
#define PRISM_MAX_HEAD_DIM 128 /* d_k, d_v in {16, 32, 64, 128} */
#define PRISM_MAX_L 16         /* 1 <= L <= 16 */
#define PRISM_MAX_W 8          /* 1 <= W <= 8 */
#define PRISM_MAX_WIDTH 8192   /* row width D of the block norm and the embedding */

/*
 * prism_scan_fwd - the whole mixer forward: ShortConv anchor, residual chain,
 * rank-(L-1) residual write and gated-delta write inside one scan, readout.
 * Defined by the sources above (write-up 核心迭代形式 / 架构形式, summary 2.1-2.2).
 *
 * chunk: chunk length of the chunkwise-parallel evaluation, a power of two in
 *   [16, 64].  The result does not depend on it beyond rounding.  The bf16
 *   tensor-core path runs chunk == 64 with d_k == d_v in {64, 128}.  fp32 with
 *   d_k == d_v in {16, 32, 64} runs the same chunk decomposition in fp32 FMAs on
 *   CUDA cores (one launch, chunk length `chunk`).  Every other supported shape runs
 *   the fp32 CUDA-core path that evaluates the recurrence token by token.
 * workspace / workspace_bytes: device scratch of at least
 *   prism_scan_fwd_workspace_size(...) bytes (may be NULL when that is 0), 16-byte
 *   aligned, owned by the caller, contents undefined on return.  The tensor-core
 *   path writes there, in one launch over all chunks before the scan, the residual
 *   write vectors alpha_{t,l} r_{t,l} of every token, scaled for the chunk form, as
 *   bf16 in the layout of gain (B * T * H * (L - 1) * d_v * 2 bytes, rounded up to
 *   256); a sequence cut into segments (long sequences over few (batch row, head)
 *   chains) adds three fp32 d_v x d_k states per segment, and a scan run in two halves
 *   (chains that leave SMs idle) adds two fp32 d_v x d_k states per chain.  The CUDA-core paths
 *   need none.  Too small or NULL: PRISM_ERR_WORKSPACE, before any launch.
 * Errors: PRISM_ERR_INVALID_ARG, PRISM_ERR_UNSUPPORTED, PRISM_ERR_WORKSPACE,
 *   PRISM_ERR_CUDA, as described above.
 */
int prism_scan_fwd(const void* q, const void* k, const void* v,
                   const float* gamma, const float* beta,
                   const void* u, const float* alpha, const void* gain,
                   const float* conv_w, const float* S0, const int32_t* lengths,
                   int B, int T, int H, int d_k, int d_v, int L, int W, int chunk,
                   int dtype, void* o, float* S_final,
                   void* workspace, size_t workspace_bytes, prism_stream_t stream);

/*
 * prism_scan_fwd_ex - prism_scan_fwd with the residual chain selected by `chain`
 * (PRISM_CHAIN_LINEAR or PRISM_CHAIN_GELU; any other value is PRISM_ERR_INVALID_ARG),
 * and the ShortConv history of the sequences in `conv_state`.
 * For PRISM_CHAIN_GELU the `gain` tensor holds the predictor output p of the exact
 * refinement step r <- r - GELU(p * r) (gist.science PRISM explainer, 2.2), any real value.
 * conv_state [B,H,W-1,d_v] dtype (device, 16-byte aligned; NULL: zeros): v_{-W+1}, ...,
 *   v_{-1}, oldest first, the values of v before token 0 that the ShortConv anchors of
 *   the first W - 1 tokens read (ICML 2026 PRISM write-up, 消除 Token 间串行: the anchor
 *   reads the last few tokens).  A sequence scanned in two calls, the second with
 *   S0 = the first's S_final and conv_state = the first's last W - 1 rows of v, gives
 *   the result of one call over the whole sequence (the layout of prism_decode_step's
 *   conv_state).  Ignored when W == 1.
 * prism_scan_fwd is prism_scan_fwd_ex with PRISM_CHAIN_LINEAR and no history.
 */
int prism_scan_fwd_ex(const void* q, const void* k, const void* v,
                      const float* gamma, const float* beta,
                      const void* u, const float* alpha, const void* gain,
                      const float* conv_w, const float* S0, const int32_t* lengths,
                      int B, int T, int H, int d_k, int d_v, int L, int W, int chunk,
                      int dtype, void* o, float* S_final,
                      void* workspace, size_t workspace_bytes, prism_stream_t stream, int chain,
                      const void* conv_state);

/* Bytes of device workspace prism_scan_fwd needs for these sizes (0 if none).
 * Returns 0 for invalid sizes as well; prism_scan_fwd reports those. */
size_t prism_scan_fwd_workspace_size(int B, int T, int H, int d_k, int d_v, int L,
                                     int W, int chunk, int dtype);

/*
 * prism_scan_bwd - gradients of the scan (the training pass): for the cotangents dO of o
 * and (optionally) dS_final of S_final, the gradients of L = <o, dO> + <S_final, dS_final>
 * with respect to every input of prism_scan_fwd_ex with the same arguments.  Reverse-mode
 * differentiation of the recurrence defined above (ICML 2026 PRISM write-up, 核心迭代形式 /
 * 架构形式; PRISM explainer 2.1-2.2).
 *
 * Inputs: as prism_scan_fwd_ex (q, k, v, gamma, beta, u, alpha, gain, conv_w, S0, lengths,
 *   chain), plus dO [B,T,H,d_v] (dtype) and dS_final [B,H,d_v,d_k] fp32 or NULL (zero).
 * Outputs (fp32, device, caller-owned, same shapes as the inputs): dq, dk [B,T,H,d_k];
 *   dv [B,T,H,d_v]; dgamma, dbeta [B,T,H]; du [B,T,H,L-1,d_k], dalpha [B,T,H,L-1],
 *   dgain [B,T,H,L-1,d_v] (all three NULL iff L == 1); dconv_w [H,d_v,W]; dS0 [B,H,d_v,d_k]
 *   (the gradient with respect to the initial state, zeros or S0).  Padded steps get zero
 *   gradients.
 * Two algorithms, chosen by shape; both compute in fp32 and are deterministic:
 *   chunked (d_k = d_v in {64, 128}, L <= 4): a token-by-token forward records S at every
 *     64-token chunk boundary and v_t - gamma_t S_{t-1} k_t; a reverse token-by-token
 *     launch runs the adjoint recurrence G_t = dO_t q_t^T + gamma_{t+1} G_{t+1}
 *     (I - beta_{t+1} k_{t+1} k_{t+1}^T) and records G_t k_t, G_t u_{t,l}, the gradient
 *     entering every chunk end and its inner product with the state there; one launch
 *     per chunk then forms every gradient of the chunk's tokens from those records; a
 *     last launch adds the per-chunk dconv_w partials in a fixed order.  Workspace
 *     (fp32): B*H*(2*NC+1)*d*d for the boundary states and gradients (NC = ceil(T/64)),
 *     B*T*H*(L+1)*d for the per-token records, plus small per-chunk partials.
 *   token-by-token (every other shape): a forward records every state S_t
 *     (B*H*T*d_v*d_k fp32), a reverse launch walks the tokens, two launches reduce the
 *     per-row-block partial sums (of 32 rows; 64 for d_k = 16) of the gradients that
 *     are sums over rows (dq, dk, du, dgamma, dbeta, dalpha) and dconv_w.
 * workspace: prism_scan_bwd_workspace_size() bytes (the chunked form: 0.54 GB for the
 *   130M-LM layer, B=16 T=2048 H=6 d=128 L=4, against 12.9 GB token by token).
 * Sizes as prism_scan_fwd.  Four launches on `stream` after memsets of the outputs; no
 * synchronisation.
 */
size_t prism_scan_bwd_workspace_size(int B, int T, int H, int d_k, int d_v, int L, int W, int dtype);

int prism_scan_bwd(const void* q, const void* k, const void* v,
                   const float* gamma, const float* beta,
                   const void* u, const float* alpha, const void* gain,
                   const float* conv_w, const float* S0, const int32_t* lengths,
                   const void* dO, const float* dS_final,
                   int B, int T, int H, int d_k, int d_v, int L, int W, int dtype, int chain,
                   float* dq, float* dk, float* dv, float* dgamma, float* dbeta,
                   float* du, float* dalpha, float* dgain, float* dconv_w, float* dS0,
                   void* workspace, size_t workspace_bytes, prism_stream_t stream);

/*
 * prism_state_affine - out = S M + N for every (batch, head): the composition step of
 * per-segment state maps.  The state update is affine in the state (see the recurrence
 * above), so a run over a segment of tokens maps a start state S to S M + N, with
 * M [d_k, d_k] the ordered product of the transitions gamma_t (I - beta_t k_t k_t^T) and
 * N [d_v, d_k] the segment's end state from a zero start.  Sequence sharding folds the
 * maps of earlier segments into a segment's start state with this call.
 *
 * S, N, out: [BH, d_v, d_k] fp32; M: [BH, d_k, d_k] fp32; device, caller-owned.  N may
 * be NULL (zero).  out may be exactly S or exactly N; any other overlap of out with S, M
 * or N returns PRISM_ERR_INVALID_ARG before any launch.  d_k, d_v in
 * {16, 32, 64, 128}; 1 <= BH <= 65535.  fp32, fixed summation order (deterministic).
 * One launch on `stream`, no synchronisation.
 */
int prism_state_affine(const float* S, const float* M, const float* N, float* out, int BH, int d_v, int d_k,
                       prism_stream_t stream);

/* Size of the device-global scratch behind prism_scan_fwd_static. */
#define PRISM_STATIC_WORKSPACE_BYTES (192u << 20)

/*
 * prism_scan_fwd_static - prism_scan_fwd_ex without a caller-supplied workspace and
 * without any allocation (an entry point of this library; the PRISM write-ups describe
 * no counterpart): the scratch is a file-scope device array of
 * PRISM_STATIC_WORKSPACE_BYTES (192 MiB, 256-byte aligned) inside the library, one per
 * device.  The first call on a device looks its address up with cudaGetSymbolAddress
 * (make that first call before any stream capture); later calls reuse it.  The array
 * sits in a module of its own: with lazy module loading (the default of CUDA 12, and
 * what PyTorch sets) it is held, until the process exits, on each device where this
 * entry point has run; with CUDA_MODULE_LOADING=EAGER, on every device where the
 * library is loaded.  Results are bit-for-bit those of prism_scan_fwd_ex with a
 * workspace.  Sizes whose
 * prism_scan_fwd_workspace_size() exceeds PRISM_STATIC_WORKSPACE_BYTES return
 * PRISM_ERR_WORKSPACE before any launch (the 130M-LM layer, B=16 T=2048 H=6 d=128
 * L=4, needs 144 MiB; a 65536-token sequence over 8 heads with L=8 needs more and is
 * refused).  Because the scratch is shared, calls on one device must not overlap
 * in time: issue them on one stream or order them; calls on one stream may follow each
 * other freely.  Other arguments, conventions and errors as for prism_scan_fwd_ex.
 */
int prism_scan_fwd_static(const void* q, const void* k, const void* v,
                          const float* gamma, const float* beta,
                          const void* u, const float* alpha, const void* gain,
                          const float* conv_w, const float* S0, const int32_t* lengths,
                          int B, int T, int H, int d_k, int d_v, int L, int W, int chunk,
                          int dtype, void* o, float* S_final, prism_stream_t stream, int chain,
                          const void* conv_state);

/*
 * prism_scan_fwd_host - the same operation on HOST buffers: copies every input
 * from host memory into the caller's device buffers, runs prism_scan_fwd on
 * them, and copies o (and S_final if both pointers are given) back to host
 * memory, all enqueued on `stream` with cudaMemcpyAsync (pinned host memory
 * makes the copies asynchronous).  host_* are host pointers with the layouts
 * above, dev_* the device buffers of the same sizes; dk, dv are d_k, d_v.  The
 * call returns once the work is enqueued; synchronise `stream` before reading
 * host_o / host_S_final.
 */
int prism_scan_fwd_host(const void* host_q, const void* host_k, const void* host_v,
                        const float* host_gamma, const float* host_beta,
                        const void* host_u, const float* host_alpha, const void* host_gain,
                        const float* host_conv_w, const float* host_S0, const int32_t* host_lengths,
                        void* dev_q, void* dev_k, void* dev_v, float* dev_gamma, float* dev_beta,
                        void* dev_u, float* dev_alpha, void* dev_gain, float* dev_conv_w,
                        float* dev_S0, int32_t* dev_lengths,
                        int B, int T, int H, int dk, int dv, int L, int W, int chunk,
                        int dtype, void* dev_o, float* dev_S_final, void* host_o, float* host_S_final,
                        void* workspace, size_t workspace_bytes, prism_stream_t stream);

/*
 * prism_prologue_fwd - steps before the scan, on their own: the ShortConv
 * anchor, the anchor residual and the closed-form residual chain, giving the
 * residual-write vectors rho_{t,l} = alpha_{t,l} r_{t,l} (write-up 消除 Step
 * 间串行: the chain is element-wise and linear, so it has a closed form).
 * Inputs as for prism_scan_fwd (L >= 2); lengths may be NULL.
 * rho_out: [B, T, H, L-1, d_v] fp32 device buffer; rows t >= lengths[b] are
 * written as 0.  Errors as for prism_scan_fwd.
 */
int prism_prologue_fwd(const void* v, const float* alpha, const void* gain,
                       const float* conv_w, const int32_t* lengths,
                       int B, int T, int H, int d_v, int L, int W, int dtype,
                       float* rho_out, prism_stream_t stream);

/* 1 if prism_scan_fwd runs these sizes on the tcgen05 tensor-core chunk
 * kernel, 0 if on a CUDA-core kernel (the fp32 chunk form or token by token;
 * sizes as for prism_scan_fwd; unsupported sizes also give 0). */
int prism_scan_fwd_uses_tensor_cores(int d_k, int d_v, int L, int W, int chunk, int dtype);

/* Number of kernel launches one prism_scan_fwd call with these sizes issues (0 for
 * invalid sizes).  Tensor-core path: the residual-write launch when L > 1, then one
 * scan launch, or four (three scans and a fold) when a long sequence over few
 * (batch row, head) chains is cut into segments; when the chains leave at least 24 of
 * a B200's SMs idle, L > 1 and the sequence has at least 8 chunks, four: the scan runs
 * in two halves, and the second half's residual write runs beside the first half's
 * scan (on an internal stream of the device, forked from and joined back into the
 * call's stream).  CUDA-core paths: 1. */
int prism_scan_fwd_launches(int B, int T, int H, int d_k, int d_v, int L, int W, int chunk, int dtype);

/* Chunks (of 64 tokens) in the first of the two scan launches when prism_scan_fwd runs
 * these sizes in two halves (see prism_scan_fwd_launches); 0 when it does not, or for
 * invalid sizes.  The cut is placed so that the second half's residual write, on the SMs
 * the chains leave idle, ends about when the first scan does: with x = 0.28 chains /
 * idle SMs, ceil(NC x / (1 + x)) chunks, clamped to [ceil(NC / 4), NC - 1] (11 of 32 for
 * the 130M-LM layer, B=16 T=2048 H=6).  A measurement aid; results do not depend on it
 * beyond rounding. */
int prism_scan_fwd_split_chunks(int B, int T, int H, int d_k, int d_v, int L, int W, int chunk, int dtype);

/* prism_prologue_fwd with the residual chain selected by `chain` (see prism_scan_fwd_ex). */
int prism_prologue_fwd_ex(const void* v, const float* alpha, const void* gain,
                          const float* conv_w, const int32_t* lengths,
                          int B, int T, int H, int d_v, int L, int W, int dtype,
                          float* rho_out, prism_stream_t stream, int chain);

/*
 * prism_decode_step - one recurrent step of the scan for every (b, h): the O(1)-state
 * inference form of the recurrence above (ICML 2026 PRISM write-up, 背景 and
 * Rank-1 写入瓶颈: a linear-attention layer keeps a fixed-size state and updates it
 * once per token).  For one token t and each (b, h):
 *   a = w[h,:,0] v_t + sum_{i=1}^{W-1} w[h,:,i] v_{t-i}   (v_{t-i} taken from conv_state)
 *   r_0 = v_t - a;  r_l = chain step of r_{l-1} with gain g_l (see prism_scan_fwd_ex)
 *   S <- gamma S (I - beta k k^T) + beta v_t k^T + sum_l alpha_l r_l u_l^T;   o = S q
 * Decoding tokens one at a time from S0 and a zero history gives what prism_scan_fwd
 * gives for the whole sequence; decoding after prism_scan_fwd continues that sequence
 * when S = its S_final and conv_state = its last W-1 values of v.
 *
 * Inputs (device pointers, contiguous, 16-byte aligned):
 *   q, k        [B,H,d_k]      dtype
 *   v           [B,H,d_v]      dtype
 *   gamma, beta [B,H]          fp32
 *   u           [B,H,L-1,d_k]  dtype   (NULL iff L == 1)
 *   alpha       [B,H,L-1]      fp32    (NULL iff L == 1)
 *   gain        [B,H,L-1,d_v]  dtype   (NULL iff L == 1)
 *   conv_w      [H,d_v,W]      fp32
 * In/out, updated in place:
 *   conv_state  [B,H,W-1,d_v]  dtype   v_{t-W+1}, ..., v_{t-1}, oldest first (zeros at the
 *                                      start of a sequence); becomes v_{t-W+2}, ..., v_t.
 *                                      NULL iff W == 1.
 *   S           [B,H,d_v,d_k]  fp32    the state before the token; becomes the state after it.
 * Output:
 *   o           [B,H,d_v]      dtype
 * d_k, d_v in {16, 32, 64, 128} (independently); 1 <= L <= PRISM_MAX_L; 1 <= W <= PRISM_MAX_W;
 * chain is PRISM_CHAIN_LINEAR or PRISM_CHAIN_GELU.  Enqueued on `stream`; allocates nothing;
 * no synchronisation.  Errors as for prism_scan_fwd, returned before any launch.
 */
int prism_decode_step(const void* q, const void* k, const void* v,
                      const float* gamma, const float* beta,
                      const void* u, const float* alpha, const void* gain,
                      const float* conv_w, void* conv_state, float* S,
                      int B, int H, int d_k, int d_v, int L, int W, int dtype, int chain,
                      void* o, prism_stream_t stream);

/*
 * The operators around the mixer.  A layer of a model normalises the residual stream before
 * the mixer, gates and normalises the mixer's readout, and adds its output back to the
 * stream; before the first layer stands the embedding, behind the backward pass the optimiser.
 * They follow the conventions above: dense device buffers, 16-byte aligned, no allocation and
 * no synchronisation, statistics and sums in fp32, each output rounded once.  Rows of padding
 * (t >= lengths[b]) are not read; their outputs are written as zero, whatever the weights hold, and
 * they add nothing to the gradients of weights.  Every result is the same bit for bit on every run.  Weights and
 * their gradients are fp32; activations and their gradients have the dtype of the call.  A
 * buffer that a call writes may overlap no other buffer of the call, except where an argument
 * below says that it may be exactly another one (PRISM_ERR_INVALID_ARG otherwise).
 */

/*
 * prism_gated_norm_fwd - the norm of the mixer's readout with its output gate, one row per
 * (token, head):  y = o / sqrt(mean(o^2) + eps) * weight * act(gate),  mean over d.
 *   o       [B,T,H,d] dtype     (prism_decode_step's o: T = 1)
 *   gate    [B,T,H,d] dtype or NULL (no gate).  The H * d values of one token are dense; tokens
 *           are gate_stride elements apart (H * d when dense; more for a slice of a wider
 *           projection; a multiple of 16 bytes; ignored when gate is NULL)
 *   weight  [d] fp32, shared by the heads
 *   y       [B,T,H,d] dtype (output); may be o
 * d in {16, 32, 64, 128}; eps > 0; act is a prism_act.  One launch.
 * With PRISM_BF16 the sigmoid is taken from the hardware's approximate exponential and reciprocal, here
 * and in the backward (d_weight among them): relative error below (2 + 1.2 |gate|) 2^-23 and 2^-22, and
 * a sigmoid below 2^-126 is zero.  With PRISM_FP32 it is computed with expf and a division.
 */
int prism_gated_norm_fwd(const void* o, const void* gate, const float* weight, const int32_t* lengths,
                         int B, int T, int H, int d, long long gate_stride, float eps, int act, int dtype,
                         void* y, prism_stream_t stream);

/*
 * prism_gated_norm_bwd - gradients of <y, dy>:  d_o, d_gate (dense; NULL iff gate is NULL)
 * [B,T,H,d] dtype and d_weight [d] fp32.  d_o may be dy; it is what prism_scan_bwd takes as dO.
 * The statistics are computed again from o.  workspace: at least
 * prism_gated_norm_bwd_workspace_size() bytes.  Two launches, or one for few rows.
 */
size_t prism_gated_norm_bwd_workspace_size(int B, int T, int H, int d);

int prism_gated_norm_bwd(const void* o, const void* gate, const float* weight, const void* dy,
                         const int32_t* lengths, int B, int T, int H, int d, long long gate_stride, float eps,
                         int act, int dtype, void* d_o, void* d_gate, float* d_weight,
                         void* workspace, size_t workspace_bytes, prism_stream_t stream);

/*
 * prism_block_norm_fwd - the border between two blocks of the residual stream: the block's
 * output y joins the stream x, and the next block's input is normalised.
 *   z = y, or y / sqrt(mean(y^2) + eps) * post_weight where post_weight is given
 *   x_out = x + res_scale * scale * z;   h = x_out / sqrt(mean(x_out^2) + eps) * weight
 * (means over D; h is computed from x_out before its rounding)
 *   x, x_out  [B,T,D] x_dtype; x_out may be x.  y NULL: x_out is not written, h is the norm of x
 *   y, h      [B,T,D] dtype
 *   weight, post_weight (or NULL), scale (or NULL: 1)  [D] fp32
 * 1 <= D <= PRISM_MAX_WIDTH (any width; multiples of 8, of 4 with an
 * fp32 stream, take wide accesses); B T <= 2e9 for D > 256.  x_dtype and
 * dtype: both PRISM_BF16, both PRISM_FP32, or an fp32 stream with bf16 blocks.  One launch.
 */
int prism_block_norm_fwd(const void* x, const void* y, const float* post_weight, const float* scale,
                         const float* weight, const int32_t* lengths, int B, int T, int D,
                         float res_scale, float eps, int x_dtype, int dtype,
                         void* x_out, void* h, prism_stream_t stream);

/*
 * prism_block_norm_bwd - gradients of <x_out, dx_out> + <h, dh>, from the stored x_out (x
 * itself when y is NULL) and y.
 *   dh [B,T,D] dtype; dx_out [B,T,D] x_dtype or NULL (zero)
 *   dx [B,T,D] x_dtype, may be dx_out; dy [B,T,D] dtype (NULL iff y is NULL)
 *   d_weight, and where their vectors are given d_post_weight and d_scale: [D] fp32
 * workspace: at least prism_block_norm_bwd_workspace_size() bytes.  Two launches, or one for few rows.
 */
size_t prism_block_norm_bwd_workspace_size(int B, int T, int D);

int prism_block_norm_bwd(const void* x_out, const void* y, const float* post_weight, const float* scale,
                         const float* weight, const void* dh, const void* dx_out, const int32_t* lengths,
                         int B, int T, int D, float res_scale, float eps, int x_dtype, int dtype,
                         void* dx, void* dy, float* d_weight, float* d_post_weight, float* d_scale,
                         void* workspace, size_t workspace_bytes, prism_stream_t stream);

/*
 * prism_embed_fwd - out[b,t] = scale * table[ids[b,t]].
 *   ids    [B,T] int32 or int64 (ids_bits 32 or 64)
 *   table  [V,D] table_dtype;  out [B,T,D] dtype (table_dtype, or bf16 of an fp32 table)
 * An id outside [0, V) at a valid step reads nothing: its row is zero, and PRISM_ERR_BOUNDS is
 * recorded in the status word.  1 <= D <= PRISM_MAX_WIDTH, V <= 2^30, B T < 2^31.  One launch.
 */
int prism_embed_fwd(const void* ids, const void* table, const int32_t* lengths, int B, int T, int V, int D,
                    float scale, int ids_bits, int table_dtype, int dtype, void* out, prism_stream_t stream);

/*
 * prism_embed_bwd - the table's gradient:  d_table[v] = scale * sum of d_out[b,t] over the
 * tokens with ids[b,t] = v, summed in fp32 in the order of the tokens.
 *   d_out [B,T,D] dtype;  d_table [V,D] fp32
 *   accumulate 0: every row of d_table is written (zero where no token names it); otherwise
 *   the sums are added to what d_table holds and only the rows that a token names are touched
 * Ids outside [0, V) give no gradient and are recorded as in prism_embed_fwd.  workspace: at
 * least prism_embed_bwd_workspace_size() bytes (16 bytes a token for the sorted ids, up to 2 MB
 * of counts, a bit per table row, and 8 D bytes for each chunk of 16 to 128 tokens).  Two or three
 * launches for up to 32768 tokens (up to 8192 where the device has no place for a cluster of sixteen
 * blocks), else five to thirteen.
 */
size_t prism_embed_bwd_workspace_size(int B, int T, int V, int D);

int prism_embed_bwd(const void* ids, const void* d_out, const int32_t* lengths, int B, int T, int V, int D,
                    float scale, int ids_bits, int dtype, int accumulate, float* d_table,
                    void* workspace, size_t workspace_bytes, prism_stream_t stream);

/* Test hook, process-wide: with `on` not 0 the sort of prism_embed_bwd takes no cluster of more than
 * eight blocks, as where the device has no place for one (more than 8192 tokens are then sorted
 * by tiles).  The results are the same bit for bit. */
void prism_set_portable_clusters(int on);

/* One parameter tensor of prism_adamw_step: n elements at each of the device pointers. */
typedef struct prism_adamw_tensor {
  void* param;            /* p_dtype, updated in place */
  const void* grad;       /* g_dtype */
  void* exp_avg;          /* first moment: fp32, or e4m3 codes (one byte) */
  void* exp_avg_sq;       /* second moment: fp32, or the e4m3 codes of its square root */
  float* exp_avg_scale;   /* 8-bit states: [ceil(n / 256)], value = code * scale; NULL with 32 bits */
  float* exp_avg_sq_scale;
  void* copy;             /* bf16 copy of an fp32 parameter, written; or NULL */
  long long n;            /* 0: the tensor is skipped */
  double weight_decay;
} prism_adamw_tensor;

/*
 * prism_adamw_step - one AdamW step over `count` tensors.  `tensors` is a HOST array, read
 * during the call only (a captured graph holds its contents).
 *   g = grad_scale * grad;  m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^step) m / (sqrt(v / (1 - beta2^step)) + eps)
 *   step      counts from 1; step_dev, when given, is read on the device instead (below 1 counts as 1)
 *   lr        likewise lr_dev; both let a captured graph be replayed along a schedule
 *   grad_scale  device scalar (such as a clipping factor) or NULL (1)
 *   state_bits  32: fp32 moments.  8: blocks of 256 consecutive elements of a tensor hold their
 *             moments as e4m3 codes times one scale, the block's largest magnitude / 448 (at
 *             least 2^-126); the second moment is held as its square root, and one that is not
 *             zero is never held as zero.  The update takes the moments before that rounding.
 *             Zeros are a valid first state.  An infinity or NaN in a gradient makes its block
 *             NaN.  The quotient of the update is taken by the approximate reciprocal (relative error
 *             2^-23; with 32 bits it is a division).
 * The decay lr * weight_decay * p and the update are summed before they are subtracted from p, so that a
 * decay far below 2^-24 is not lost to the rounding of 1 - lr * weight_decay.
 * All parameters share p_dtype and all gradients g_dtype.  The scalars and the scales are
 * 4-byte aligned.  One launch for up to 440 tensors.
 */
int prism_adamw_step(const prism_adamw_tensor* tensors, int count, int step, const int32_t* step_dev, double lr,
                     const float* lr_dev, double beta1, double beta2, double eps, const float* grad_scale,
                     int p_dtype, int g_dtype, int state_bits, prism_stream_t stream);

/* A tensor as DLPack describes it (the layout of DLTensor, DLPack 1). */
typedef struct prism_dl_tensor {
  void* data;
  int32_t device_type; /* 2: CUDA */
  int32_t device_id;
  int32_t ndim;
  uint8_t type_code; /* 2: float, 4: bfloat, 10: e4m3 (fn) */
  uint8_t type_bits;
  uint16_t type_lanes;
  int64_t* shape;
  int64_t* strides; /* NULL: dense */
  uint64_t byte_offset;
} prism_dl_tensor;

/* DLPack's exchange function of a framework: views `object` as a tensor; 0 on success. */
typedef int (*prism_dl_from_object)(void* object, prism_dl_tensor* out);

/* What the tensors of one field are: type_code 0 leaves the field out. */
typedef struct prism_dl_field {
  int type_code;
  int type_bits;
  int block; /* 0: the shapes of the first field; else as many elements as those have blocks of `block` */
} prism_dl_field;

/*
 * prism_dl_pointers - the data pointers of a framework's tensors for a host array of structs,
 * such as prism_adamw_step's (host only, no CUDA call; a binding's loop over hundreds of
 * tensors).  objects holds n tensors for each of the `fields` fields that is not left out, one
 * field after the other; from_object views each.  Every object has to be a dense tensor of its
 * field's type on CUDA device `device`, and (behind the first field) to match the first field's
 * tensor of the same place.  The pointer of field f, place i goes to out + i * stride + 8 f, the
 * first field's numbers of elements (long long) to out + i * stride + count_offset.
 * views: room for n prism_dl_tensor.  Returns -1, or the index in objects of the first object
 * that is not as described.
 */
int prism_dl_pointers(int fields, const prism_dl_field* spec, int n, void* const* objects,
                      prism_dl_from_object from_object, int device, prism_dl_tensor* views, void* out, size_t stride,
                      size_t count_offset);

/* Synchronises `stream`, then returns and clears the device status word of the
 * current device: PRISM_OK, PRISM_ERR_TIMEOUT, PRISM_ERR_BOUNDS, or
 * PRISM_ERR_CUDA if the synchronisation itself failed. */
int prism_stream_status(prism_stream_t stream);

/* Test hook: the spin limit of the device-side bounded waits (0 restores the
 * default).  A tiny limit makes those waits give up and record
 * PRISM_ERR_TIMEOUT instead of waiting, which tests the error path without
 * hanging a GPU.  Host-side setting; applies to launches made after the call. */
void prism_set_spin_limit(long long limit);

/* Measurement hook: `event` (a cudaEvent_t, or NULL to clear) is recorded on the
 * stream of the next prism_scan_fwd call that runs the tensor-core path with L > 1,
 * after its (first) residual-write launch, and is then forgotten.  Events recorded by
 * the caller before and after that call then time that launch and the rest apart.  Process-wide; set it from the thread that makes the call. */
void prism_set_split_event(void* event);

/* Static description of a status code; never NULL. */
const char* prism_status_string(int code);

/* (major << 16) | (minor << 8) | patch */
int prism_version(void);

/* 1 in the debug build of this library (libprism_debug.so, compiled with
 * PRISM_DEBUG_BOUNDS), 0 in the release build (libprism.so).  Both export the same
 * functions and compute the same results bit for bit.  In the debug build the kernels
 * check the global indices they compute against the extents of their buffers (and the
 * innermost coordinate of every TMA copy against the 16-byte rule); a failed check
 * records PRISM_ERR_BOUNDS in the device status word and skips the access. */
int prism_debug_bounds(void);

/* Test hook of the debug build: one launch on `stream` that runs the device-side check
 * of index i against extent n (no memory is accessed at that index), so that
 * prism_stream_status then reports PRISM_ERR_BOUNDS exactly when i is outside [0, n).
 * PRISM_ERR_UNSUPPORTED in the release build; PRISM_ERR_CUDA if the launch fails. */
int prism_debug_bounds_probe(long long i, long long n, prism_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PRISM_H_ */
