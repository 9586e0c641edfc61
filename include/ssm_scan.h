/*
 * ssm_scan.h — C ABI of the MI355X (gfx950) selective state-space scan library, libssmscan.so.
 *
 * The operation (sources: page "State Space Models（SSM）とMamba" §2.1–§2.2 and §4.2; page
 * "Mambaとは？Transformer以外の系列モデル", sections 状態空間モデルを一つの式から理解する,
 * Mambaの核心は入力依存のDelta、B、C, Selective Scanは選択機構そのものではない, Mamba blockの
 * architecture and training、prefill、decodeでは計算の姿が違う):
 *
 *   for every batch row b and channel d, with a diagonal continuous-time A[d][·] and per-token
 *   step Δ_t, input matrices B_t and C_t (shared by all channels of the batch row):
 *     Ā_t[n] = exp(Δ_t · A[d][n])                        zero-order hold
 *     B̄_t[n] = (exp(Δ_t · A[d][n]) − 1) / A[d][n] · B_t[n]   (Δ_t · B_t[n] at A = 0, the limit)
 *     h_t[n] = Ā_t[n] · h_{t−1}[n] + B̄_t[n] · x_t         the recurrence (h_{−1} = 0 in prefill)
 *     y_t    = Σ_n C_t[n] · h_t[n] + D[d] · x_t            readout with the updated state + skip
 *     y_t    ← y_t · z_t · σ(z_t)                           optional SiLU gate
 *
 * Prefill (ssm_scan_fwd) evaluates the whole sequence; decode (ssm_scan_step) advances a stored
 * state by one token. Both compute in fp32 with an fp32 state.
 *
 * Conventions shared by every entry point
 *   - Pointers to tensors are DEVICE pointers owned by the caller; the library never frees them.
 *     All tensors are dense, row-major, with no padding:
 *       x, delta, z, y : [b][d][L]        (decode: [b][d])
 *       A              : [d][N]  fp32
 *       B, C           : [b][L][N]        (decode: [b][N])
 *       D              : [d]     fp32
 *       states         : [b][d][N] fp32
 *     `dtype` is the storage type of x, delta, z, B, C and y (SSM_F32 = float, SSM_BF16 = bf16 bit
 *     patterns, rounded to nearest-even on output). A, D and states are always fp32.
 *   - delta is used as given (a positive step; no softplus or bias is applied here).
 *   - Arguments are validated on the host before any launch; a failed check returns a non-zero
 *     status and launches nothing. Work is enqueued on `stream` (0 = the null stream) and the call
 *     returns without synchronising. Asynchronous device faults surface at the caller's next
 *     synchronisation of that stream.
 *   - Calls are reentrant: the library keeps no per-call global state. Calls on different streams
 *     may run concurrently. Calls that need scratch (a prefill split into time segments, the
 *     gradient pass, ssm_lti_fwd, ssm_ssd_fwd except bf16 with N of 64 or 128 and b·H at least
 *     twice the device's compute units) take it stream-ordered on `stream` from a memory pool the
 *     library creates on the current device at its first such call, and return it there at the
 *     end of the call. That pool keeps freed scratch (its release threshold is at the maximum), so
 *     repeated calls reuse it; it lives until the process ends. The device's default pool is not
 *     touched. ssm_scan_fwd_noalloc takes no scratch from any pool (see there).
 *   - NaN and Inf inputs propagate; nothing is clamped.
 */
#ifndef SSM_SCAN_H
#define SSM_SCAN_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_ABI_VERSION 1
#define SSM_MAX_N 64

/* Exported symbols (the library is built with hidden visibility by default). */
#if defined(__GNUC__)
#define SSM_API __attribute__((visibility("default")))
#else
#define SSM_API
#endif
/* The *_MAX_ENUM members are not values: they give both enums a 32-bit range, so any int a C or FFI
 * caller passes is a representable value of the type (and is then rejected or named "unknown"). */
typedef enum { SSM_F32 = 0, SSM_BF16 = 1, SSM_DTYPE_MAX_ENUM = 0x7fffffff } ssm_dtype_t;

typedef enum {
    SSM_OK = 0,
    SSM_ERR_NULL = 1,        /* a required pointer is NULL                                   */
    SSM_ERR_SHAPE = 2,       /* a size is out of range (b, d, N < 1; L < 0; overflow)         */
    SSM_ERR_UNSUPPORTED = 3, /* N > SSM_MAX_N, unknown dtype, or an option value not accepted */
    SSM_ERR_HIP = 4,         /* a HIP runtime call or a launch failed                          */
    SSM_ERR_ALIAS = 5,       /* an output overlaps an input or another output                 */
    SSM_ERR_SCRATCH = 6,     /* ssm_scan_fwd_noalloc: the plan needs more than its fixed scratch;
                                a caller's workspace is smaller than the call needs            */
    SSM_STATUS_MAX_ENUM = 0x7fffffff
} ssm_status_t;

/*
 * Prefill: the selective scan over a whole sequence (the parallel "prefill" mode), h_{−1} = 0.
 *   x, delta   [b][d][L] dtype      required
 *   A          [d][N] fp32          required; any finite value, A = 0 takes the ZOH limit
 *   B, C       [b][L][N] dtype      required
 *   D          [d] fp32             optional (NULL = no skip term)
 *   z          [b][d][L] dtype      optional (NULL = no gate)
 *   y          [b][d][L] dtype      required output; must not overlap any input
 *   final_state[b][d][N] fp32       optional output h_{L−1} (NULL = not written)
 *   b, d, N >= 1; L >= 0; N <= SSM_MAX_N. With L = 0 the call writes zeros to final_state (with
 *   ssm_scan_fwd_ex's initial_state: a copy of it) and touches nothing else, so x, delta, A, B, C, y may
 *   then be NULL.
 *   Errors: SSM_ERR_NULL, SSM_ERR_SHAPE, SSM_ERR_UNSUPPORTED, SSM_ERR_ALIAS (nothing launched);
 *   SSM_ERR_HIP when scratch allocation or a launch fails (work already enqueued may have run).
 */
SSM_API ssm_status_t ssm_scan_fwd(const void *x, const void *delta, const float *A, const void *B,
                          const void *C, const float *D, const void *z, void *y,
                          float *final_state, int64_t b, int64_t d, int64_t L, int64_t N,
                          ssm_dtype_t dtype, hipStream_t stream);

/*
 * Decode: one recurrent step per (b, d) on a state kept in HBM (the recurrent "decode" mode).
 *   state      [b][d][N] fp32       required, in/out: read as h_{t−1}, overwritten with h_t
 *   x, delta   [b][d] dtype         required
 *   A          [d][N] fp32          required
 *   B, C       [b][N] dtype         required
 *   D          [d] fp32             optional
 *   z          [b][d] dtype         optional
 *   y          [b][d] dtype         required output
 *   b, d, N >= 1; N <= SSM_MAX_N; b * d < 2^31 (SSM_ERR_SHAPE otherwise). The state is read and
 *   written in place (it may not overlap any other argument). Errors as for ssm_scan_fwd.
 */
SSM_API ssm_status_t ssm_scan_step(float *state, const void *x, const void *delta, const float *A,
                           const void *B, const void *C, const float *D, const void *z, void *y,
                           int64_t b, int64_t d, int64_t N, ssm_dtype_t dtype, hipStream_t stream);

/*
 * Gradients of the prefill scan (ssm_scan_fwd with an optional initial state) for an upstream
 * gradient dy on y and, optionally, d_final_state on the final state. The forward map is the one
 * ssm_scan_fwd computes (page "Mambaとは？Transformer以外の系列モデル", section 状態空間モデルを一つの
 * 式から理解する); its derivatives follow by the chain rule in reverse time, and the forward states are
 * recomputed rather than stored (same page, section hardware-awareとは memory trafficまで設計すること).
 *   inputs            as for ssm_scan_fwd (x, delta, A, B, C, D, z), initial_state [b][d][N] fp32
 *                     or NULL (zeros)
 *   dy                [b][d][L] dtype, required
 *   d_final_state     [b][d][N] fp32 or NULL (zeros)
 *   dx, ddelta        [b][d][L] dtype, required outputs
 *   dz                [b][d][L] dtype; required when z is given, ignored otherwise
 *   dA                [d][N] fp32, required (summed over b and t)
 *   dB, dC            [b][L][N] fp32, required (summed over d)
 *   dD                [d] fp32 or NULL (summed over b and t; defined also when D is NULL)
 *   d_initial_state   [b][d][N] fp32 or NULL
 * The sums dA, dB, dC, dD are accumulated with float atomics, so their last bits can differ from
 * run to run; everything else is deterministic. Scratch (checkpoints every max(4, 32/states_per_lane) steps
 * and the segment aggregates) is taken stream-ordered from `stream` and returned. Outputs may not
 * overlap inputs or each other. b, d, N >= 1, L >= 1, N <= SSM_MAX_N. Errors as for ssm_scan_fwd.
 */
SSM_API ssm_status_t ssm_scan_bwd(const void *x, const void *delta, const float *A, const void *B,
                                  const void *C, const float *D, const void *z,
                                  const float *initial_state, const void *dy, const float *d_final_state,
                                  void *dx, void *ddelta, float *dA, float *dB, float *dC, float *dD,
                                  void *dz, float *d_initial_state, int64_t b, int64_t d, int64_t L,
                                  int64_t N, ssm_dtype_t dtype, hipStream_t stream);

/*
 * The short causal depthwise Conv1D (+ SiLU) of the Mamba block's main branch, which produces the
 * scan's x (page "Mambaとは？Transformer以外の系列モデル", section Mamba blockのarchitecture), and its
 * decode step with the per-layer Conv1D state (same page, section training、prefill、decodeでは計算の
 * 姿が違う). Per channel d with taps w[d][0..W) and bias c_d:
 *     u_t = c_d + Σ_{k<W} w[d][k] · xin_{t−(W−1)+k},   x_t = silu(u_t) if apply_silu, else u_t,
 * the inputs before t = 0 taken from state_in (zeros when NULL).
 *   xin, x_out        [b][d][L] dtype (x_out may not overlap xin)
 *   w                 [d][W] fp32, 1 <= W <= SSM_MAX_CONV_W
 *   bias              [d] fp32 or NULL
 *   state_in          [b][d][W−1] fp32 or NULL: the W−1 inputs before the sequence, oldest first
 *   state_out         [b][d][W−1] fp32 or NULL: the last W−1 inputs after it (may equal state_in)
 * b, d >= 1, L >= 0. Errors as for ssm_scan_fwd.
 */
#define SSM_MAX_CONV_W 8
SSM_API ssm_status_t ssm_conv1d_fwd(const void *xin, const float *w, const float *bias, const float *state_in,
                                    void *x_out, float *state_out, int64_t b, int64_t d, int64_t L, int64_t W,
                                    int32_t apply_silu, ssm_dtype_t dtype, hipStream_t stream);

/* Decode: one new input per (b, d). state [b][d][W−1] fp32 is read and shifted in place (the new
 * input enters last); xin, x_out [b][d] dtype. Other arguments as for ssm_conv1d_fwd. */
SSM_API ssm_status_t ssm_conv1d_step(float *state, const void *xin, const float *w, const float *bias,
                                     void *x_out, int64_t b, int64_t d, int64_t W, int32_t apply_silu,
                                     ssm_dtype_t dtype, hipStream_t stream);

/*
 * The main branch of the Mamba block from the Conv1D's input to y in one pass: the Conv1D + SiLU of
 * ssm_conv1d_fwd (apply_silu on) and the scan of ssm_scan_fwd, with the parameter preprocessing folded
 * into the scan's tile staging (page "Mambaとは？Transformer以外の系列モデル", section hardware-awareとは
 * memory trafficまで設計すること: parameter generation, discretisation and scan in one kernel, only the
 * outputs going back to memory; section Mamba blockのarchitecture: Conv1D, SiLU, then the selective SSM).
 * Per (b, d) and t:
 *     x_t = silu(c_d + Σ_{k<W} conv_w[d][k] · xin_{t−(W−1)+k})        (inputs before t = 0 from
 *                                                                     conv_state_in, else zeros)
 *     Δ_t = softplus(delta_t + delta_bias[d]) if delta_softplus, else delta_t + delta_bias[d]
 * then the scan of ssm_scan_fwd on x, Δ from initial_state (zeros when NULL). The convolved x is kept in
 * fp32 inside the kernel (it is not rounded to the storage type before the scan); x_out, when given,
 * receives it rounded to the storage type (for the caller's projections of x).
 *   xin                [b][d][L] dtype, required
 *   conv_w             [d][W] fp32, required, 1 <= W <= SSM_MAX_FUSED_CONV_W (SSM_ERR_UNSUPPORTED above)
 *   conv_bias          [d] fp32 or NULL
 *   conv_state_in      [b][d][W−1] fp32 or NULL: the W−1 inputs before the sequence, oldest first
 *   delta              [b][d][L] dtype, required: Δ before its bias and softplus
 *   delta_bias         [d] fp32 or NULL
 *   A, B, C, D, z      as for ssm_scan_fwd; initial_state [b][d][N] fp32 or NULL
 *   y, final_state     as for ssm_scan_fwd
 *   conv_state_out     [b][d][W−1] fp32 or NULL: the last W−1 inputs after the sequence (must not
 *                      overlap conv_state_in; copy it back for the next call)
 *   x_out              [b][d][L] dtype or NULL
 * Scratch as for ssm_scan_fwd. No output may overlap an input or another output. Errors as for
 * ssm_scan_fwd.
 */
#define SSM_MAX_FUSED_CONV_W 4
SSM_API ssm_status_t ssm_scan_fwd_conv(const void *xin, const float *conv_w, const float *conv_bias,
                                       const float *conv_state_in, int64_t W, const void *delta,
                                       const float *delta_bias, int32_t delta_softplus, const float *A,
                                       const void *B, const void *C, const float *D, const void *z,
                                       const float *initial_state, void *y, float *final_state,
                                       float *conv_state_out, void *x_out, int64_t b, int64_t d, int64_t L,
                                       int64_t N, ssm_dtype_t dtype, hipStream_t stream);

/*
 * One decode step of the same branch in one launch (page "Mambaとは？Transformer以外の系列モデル", section
 * training、prefill、decodeでは計算の姿が違う: each layer keeps a Conv1D state and an SSM state): the token's
 * raw input is convolved with conv_state (the last W−1 inputs, fp32 [b][d][W−1], shifted in place; may be
 * NULL when W = 1), SiLU, Δ as in ssm_scan_fwd_conv, then the step of ssm_scan_step on state.
 *   state [b][d][N] fp32 in/out; xin, delta, z, y, x_out (nullable) [b][d] dtype; conv_w [d][W];
 *   conv_bias, delta_bias [d] or NULL; A, B, C, D as for ssm_scan_step.
 * The two states and the outputs may not overlap each other or any input. Errors as for ssm_scan_step.
 */
SSM_API ssm_status_t ssm_scan_step_conv(float *state, float *conv_state, const void *xin, const float *conv_w,
                                        const float *conv_bias, int64_t W, const void *delta,
                                        const float *delta_bias, int32_t delta_softplus, const float *A,
                                        const void *B, const void *C, const float *D, const void *z, void *y,
                                        void *x_out, int64_t b, int64_t d, int64_t N, ssm_dtype_t dtype,
                                        hipStream_t stream);

/*
 * The time-invariant (LTI) case evaluated as a convolution (page "State Space Models（SSM）とMamba" §2.3;
 * page "Mambaとは？Transformer以外の系列モデル", section 固定SSMには「再帰」と「畳み込み」の二つの顔がある):
 * when Ā, B̄ and C are the same at every step, the zero-state recurrence is y = x ∗ K̄ with
 * K̄ = (CB̄, CĀB̄, CĀ²B̄, …), which the FFT evaluates in O(L log L). Every channel is its own system.
 *
 * ssm_lti_kernel: K[d][k] = Σ_n C[d][n] · Ā^k · B̄ for k < L, with the ZOH of ssm_scan_fwd
 * (Ā = exp(delta[d]·A[d][n]), B̄ = (Ā − 1)/A · B[d][n], Δ·B at A = 0).
 *   delta [d], A, B, C [d][N], K [d][L] (output); all fp32. d, N >= 1, N <= SSM_MAX_N, 0 <= L < 2^24.
 *
 * ssm_lti_conv: y[b][d][t] = Σ_{s<=t} K[d][t−s] · x[b][d][s] + D[d] · x[b][d][t], times silu(z) when z
 * is given, by FFT (two batch rows of a channel per complex transform of 2^⌈log2 2L⌉ >= 1024 points).
 *   x, z, y [b][d][L] dtype (z may be NULL); K [d][L] fp32 (any kernel, e.g. from ssm_lti_kernel);
 *   D [d] fp32 or NULL. y may not overlap the inputs. b >= 1, 1 <= d <= 2^22,
 *   1 <= L <= SSM_LTI_MAX_L (SSM_ERR_UNSUPPORTED above it).
 *
 * ssm_lti_fwd: both: K̄ into scratch taken stream-ordered from `stream`, then the convolution; any L >= 1
 * (below 2^40). Up to SSM_LTI_MAX_L steps: K̄ over L taps (d·L·4 bytes of scratch) and one transform per
 * row pair. Longer: chunks of SSM_LTI_CHUNK steps, each convolved with K̄ over SSM_LTI_CHUNK taps, joined
 * through the state, the other face of the same system (same page and section): each chunk's end state
 * from zero, E_n = B̄_n·Σ_s Ā_n^{chunk−1−s}·x_s, is chained by h ← Ā^chunk·h + E into the state entering every
 * later chunk, whose response Σ_n C_n·Ā_n^{τ+1}·h_n that chunk adds to its output τ steps in (scratch:
 * d·SSM_LTI_CHUNK + b·d·(n_chunks − 1)·N floats). No final state is produced (the convolution form has none;
 * ssm_scan_fwd with the parameters repeated over t gives it). Errors as for ssm_scan_fwd.
 */
#define SSM_LTI_MAX_L 8192
#define SSM_LTI_CHUNK 4096
SSM_API ssm_status_t ssm_lti_kernel(const float *delta, const float *A, const float *B, const float *C, float *K,
                                    int64_t d, int64_t L, int64_t N, hipStream_t stream);
SSM_API ssm_status_t ssm_lti_conv(const void *x, const float *K, const float *D, const void *z, void *y, int64_t b,
                                  int64_t d, int64_t L, ssm_dtype_t dtype, hipStream_t stream);
SSM_API ssm_status_t ssm_lti_fwd(const void *x, const float *delta, const float *A, const float *B, const float *C,
                                 const float *D, const void *z, void *y, int64_t b, int64_t d, int64_t L, int64_t N,
                                 ssm_dtype_t dtype, hipStream_t stream);

/*
 * The scalar-decay selective SSM of Mamba-2's state space duality (page "State Space Models（SSM）とMamba"
 * §4.6 relates SSMs and linear attention; the pages give no formulas, so this is the selective scan of
 * ssm_scan_fwd with A restricted to one scalar per head). Channels come in H heads of P; head h has the
 * decay a_h (A[d][n] = a_h for its channels and all states) and one step delta[b][h][t] shared by its P
 * channels. Unrolled, y = (causal mask ∘ e^{a(c_t − c_s)} ∘ C Bᵀ)(β ∘ x) + D x per head, a masked linear
 * attention; it is evaluated chunk by chunk (64 steps) with matrix products on the MFMA units (fp32
 * products for fp32 storage; bf16 products, fp32 operands entering as bf16 hi + lo, for bf16 storage).
 *   x, z, y           [b][H·P][L] dtype (z may be NULL)
 *   delta             [b][H][L] dtype
 *   A                 [H] fp32 (the per-head decay a_h)
 *   B, C              [b][L][N] dtype (shared by all heads)
 *   D                 [H·P] fp32 or NULL
 *   initial_state     [b][H·P][N] fp32 or NULL (zeros); final_state [b][H·P][N] fp32 or NULL
 * Supported: P = 64, N in {32, 64, 128} (SSM_ERR_UNSUPPORTED otherwise); b, H >= 1, L >= 0. Scratch of
 * b·H·⌈L/64⌉·(P·N + 1) floats is taken stream-ordered from `stream`, except for bf16 storage with N of 64
 * or 128 and b·H at least twice the device's compute units, which needs none (the whole form then runs
 * as one ordered walk per (b, head)). Errors as for ssm_scan_fwd.
 */
SSM_API ssm_status_t ssm_ssd_fwd(const void *x, const void *delta, const float *A, const void *B, const void *C,
                                 const float *D, const void *z, const float *initial_state, void *y,
                                 float *final_state, int64_t b, int64_t H, int64_t P, int64_t L, int64_t N,
                                 ssm_dtype_t dtype, hipStream_t stream);

/*
 * Linear attention with a decay for each head: the scalar-decay recurrence of ssm_ssd_fwd on queries, keys and
 * values of any head width, token by token in memory as projections write them (page "State Space Models（SSM）と
 * Mamba" §4.6 relates the two; in the notation of ssm_ssd_fwd the queries are C, the keys B, the values β·x and
 * e^g the decay e^{a·Δ}). Per batch row and head h, with the queries and keys of group h·G/H (integer division):
 *     S_t = e^{g_t} · S_{t−1} + v_t k_tᵀ          [P][N], fp32, S_{−1} = initial_state or 0
 *     o_t = scale · S_t q_t
 * ssm_linattn_fwd evaluates it in chunks of 64 steps as matrix products (prompts), ssm_linattn_step advances a
 * stored state by one token, ssm_linattn_bwd gives the gradients of ssm_linattn_fwd.
 *   q, k              [b][L][G][N] dtype (step: [b][G][N])
 *   v, o              [b][L][H][P] dtype (step: [b][H][P])
 *   g                 log-decay, fp32: [b][L][H] (step: [b][H]) when g_per_step is 1, [H] (the same at every
 *                     step) when it is 0. Any value; −inf, and everything below −1e4, is a decay of exactly 0
 *                     (the state restarts at that step). Positive values let the state grow; where the growth over
 *                     a chunk, or a run of chunks, passes fp32's range (e^88), results may be Inf or NaN.
 *   states            [b][H][P][N] fp32, as ssm_ssd_fwd's
 *   lengths           [b] int32 on the device or NULL (every row has L steps): row i has lengths[i] steps (taken
 *                     as 0 below 0 and as L above L). Nothing past them is read; outputs past them (o, dq, dk, dv,
 *                     dg) are 0. The final state is the one after the row's last step.
 *   strides           NULL: q, k, v, do_ dense as above. Otherwise the distance in elements between batch rows
 *                     (b), steps (t) and heads or groups (h) of q, k, v and do_, each >= 0, t at most 2^24;
 *                     the last axis is dense. Inputs may so be slices of one packed projection, or broadcast (distance 0).
 *                     Outputs are always dense.
 *   workspace         device memory of at least the bytes ssm_linattn_workspace gives, 16-byte aligned, or NULL:
 *                     scratch is then taken stream-ordered as by the other entry points, which a capturing stream
 *                     may refuse. A call writes what it reads there, and keeps nothing in it; calls that
 *                     may overlap (other streams, captured graphs replayed at once) need one each.
 * Products are exact bf16 products summed in fp32 (bf16; fp32 operands, that is states and decayed scores, enter
 * as two bf16 parts, 2^-16 of the operand, where the result is bf16, as three where it is fp32) or fp32 products (f32). All sums,
 * decays and states are fp32, the running sums of g and the sums whose difference makes dg fp64. Results are
 * deterministic; the forward call's fp32 sums are cut by its segments, which depend on b, H, P and L. A NaN or Inf at one
 * step reaches outputs and gradients as the formulas say, for all later steps however strong the decay, except that an
 * Inf may come out as NaN, and that gradients (dq, dk, dv, dg) may become NaN at every step of the 64-step chunk it is in.
 * b, H, G, N, P >= 1; G divides H; H times the larger of 128 and P (rounded up to 64) is at most 2^24;
 * N <= SSM_LINATTN_MAX_N, P <= SSM_LINATTN_MAX_P (SSM_ERR_UNSUPPORTED above); L >= 0. A launch takes fewer than 2^32
 * threads: SSM_ERR_SHAPE where b·H·⌈P/64⌉ (forward: times the segments the steps are cut into, one where b·H is large)
 * reaches 2^23, in the step 2^24; and in the gradient where 2·b·H·⌈L/64⌉ reaches 2^24 (times ⌈P/128⌉, 2^23 where P > 64)
 * or b·H·P·N, P padded to 64s and N to 32, 64 or 128, reaches 2^33. With L = 0 the
 * forward call copies the initial state (or zeros) to final_state, the gradient call d_final_state (or zeros) to
 * d_initial_state and zeros to a g_per_step = 0 dg. No output may overlap an input,
 * the workspace or another output. Errors as for ssm_scan_fwd; SSM_ERR_SCRATCH: workspace_bytes is too small.
 */
#define SSM_LINATTN_MAX_N 128
#define SSM_LINATTN_MAX_P 1024
typedef struct {
    int64_t q_b, q_t, q_h, k_b, k_t, k_h, v_b, v_t, v_h, do_b, do_t, do_h;
} ssm_linattn_strides_t;

/* Workspace bytes of ssm_linattn_fwd (gradient = 0) or ssm_linattn_bwd (gradient = 1) for this shape (host
 * only, may be 0). Returns SSM_OK or the validation error. */
SSM_API ssm_status_t ssm_linattn_workspace(int32_t gradient, int64_t b, int64_t L, int64_t H, int64_t G, int64_t N,
                                           int64_t P, ssm_dtype_t dtype, int32_t g_per_step, int64_t *bytes);

/* o required (unless L = 0); initial_state, final_state, lengths, strides, workspace may be NULL. */
SSM_API ssm_status_t ssm_linattn_fwd(const void *q, const void *k, const void *v, const float *g, int32_t g_per_step,
                                     float scale, const float *initial_state, const int32_t *lengths, void *o,
                                     float *final_state, int64_t b, int64_t L, int64_t H, int64_t G, int64_t N,
                                     int64_t P, ssm_dtype_t dtype, const ssm_linattn_strides_t *strides,
                                     void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* One token: state is read and written in place (it may not overlap any other argument). The strides' t members
 * and do_ are not used. */
SSM_API ssm_status_t ssm_linattn_step(float *state, const void *q, const void *k, const void *v, const float *g,
                                      int32_t g_per_step, float scale, void *o, int64_t b, int64_t H, int64_t G,
                                      int64_t N, int64_t P, ssm_dtype_t dtype, const ssm_linattn_strides_t *strides,
                                      hipStream_t stream);

/* Gradients for an upstream gradient do_ [b][L][H][P] dtype on o and, optionally, d_final_state [b][H][P][N] fp32.
 *   dq, dk            [b][L][G][N] dtype, required (summed over the heads of the group in fp32)
 *   dv                [b][L][H][P] dtype, required
 *   dg                fp32, required: [b][L][H], or [H] (summed over rows and steps) when g_per_step is 0
 *   d_initial_state   [b][H][P][N] fp32 or NULL */
SSM_API ssm_status_t ssm_linattn_bwd(const void *q, const void *k, const void *v, const float *g, int32_t g_per_step,
                                     float scale, const float *initial_state, const int32_t *lengths,
                                     const void *do_, const float *d_final_state, void *dq, void *dk, void *dv,
                                     float *dg, float *d_initial_state, int64_t b, int64_t L, int64_t H, int64_t G,
                                     int64_t N, int64_t P, ssm_dtype_t dtype, const ssm_linattn_strides_t *strides,
                                     void *workspace, int64_t workspace_bytes, hipStream_t stream);

/*
 * Layer norm: the norm the Mamba block starts with (page "Mambaとは？Transformer以外の系列モデル", section Mamba
 * blockのarchitecture), or, with a weight row per head, the norm on each head's output of ssm_linattn_fwd. Per row
 * of d values, with mean μ and biased variance σ² over the row and r = 1/sqrt(σ² + eps):
 *     y = w ⊙ (x − μ)·r + bias
 *   x, y              [rows][d] dtype; x rows x_stride elements apart (>= d, or 0 for dense)
 *   w, bias           [w_rows][d] fp32 or NULL (1 and 0): row i uses row i mod w_rows; w_rows divides rows
 *   mean, rstd        [rows] fp32 outputs μ and r, or NULL
 *   eps               >= 0 and finite (SSM_ERR_UNSUPPORTED otherwise)
 * ssm_layernorm_bwd: with x̂ = (x − μ)·r, from the forward call's mean and rstd,
 *     dx = r·(w ⊙ dy − avg(w ⊙ dy) − x̂·avg(w ⊙ dy ⊙ x̂)),  dw = Σ_rows dy ⊙ x̂,  dbias = Σ_rows dy
 *   dy                [rows][d] dtype, rows dy_stride elements apart (>= d, or 0 for dense)
 *   dx                [rows][d] dtype, required; dw, dbias [w_rows][d] fp32 or NULL, summed in a fixed order
 *   workspace         as for ssm_linattn_fwd, of the bytes ssm_layernorm_bwd_workspace gives (0 without dw and dbias)
 * All sums are fp32 or wider. rows >= 0 (0: only dw and dbias are written, with zeros), d, w_rows >= 1,
 * d <= SSM_LAYERNORM_MAX_D (SSM_ERR_UNSUPPORTED above), rows times the distance of rows <= 2^40,
 * w_rows below 2^24 (2^22 where d > 4096: a launch takes fewer than 2^32 threads). y may be x itself (x dense), dx may
 * be dy or x itself (dense); other overlaps are refused. Errors as for ssm_scan_fwd and ssm_linattn_fwd.
 */
#define SSM_LAYERNORM_MAX_D 16384
SSM_API ssm_status_t ssm_layernorm_fwd(const void *x, const float *w, const float *bias, void *y, float *mean,
                                       float *rstd, int64_t rows, int64_t d, int64_t w_rows, int64_t x_stride,
                                       float eps, ssm_dtype_t dtype, hipStream_t stream);
SSM_API ssm_status_t ssm_layernorm_bwd_workspace(int64_t rows, int64_t d, int64_t w_rows, int64_t *bytes);
SSM_API ssm_status_t ssm_layernorm_bwd(const void *x, const float *w, const void *dy, const float *mean,
                                       const float *rstd, void *dx, float *dw, float *dbias, int64_t rows, int64_t d,
                                       int64_t w_rows, int64_t x_stride, int64_t dy_stride, ssm_dtype_t dtype,
                                       void *workspace, int64_t workspace_bytes, hipStream_t stream);

/*
 * Softmax attention, for the attention layers that hybrid stacks set between recurrent ones (page
 * "State Space Models（SSM）とMamba" §6). Per sequence of nq queries and nk keys, query head h reading key head h·G/H:
 *     s_ij = scale · q_i·k_j   over the keys j that query i sees: j <= i + nk − nq (causal) or all j < nk
 *     o_i  = Σ_j p_ij v_j,  p_ij = e^(s_ij − lse_i),  lse_i = log Σ_j e^s_ij
 * A query that sees no key has o = 0 and lse = −inf.
 *   q, o, do_         [tokens][H][D] dtype        k, v              [tokens][G][D] dtype
 *   lse               [tokens][H] fp32, or NULL where it is an output
 *   rows              where the sequences lie:
 *                     cu_q, cu_k both given: packed. b + 1 rising offsets each on the device into tokens_q and tokens_k
 *                       tokens; sequence i has those from cu[i] to cu[i+1]. They may be the same pointer. Lq and Lk are the
 *                       longest sequences' lengths, or more: a longer one counts as Lq (Lk) long. Outputs of tokens of
 *                       no sequence are left as they were. Offsets outside of the tokens are taken as the nearest one inside.
 *                     otherwise b rows of Lq queries and Lk keys, tokens_q and tokens_k unused; len_q and len_k (or NULL: all
 *                       count), [b] on the device, say how many of each row count. Nothing past them is read; outputs past
 *                       them (o, dq, dk, dv) are 0, lse −inf.
 *   strides           NULL: dense. Otherwise as ssm_linattn_strides_t's for q, k, v, do_ (b unused where packed). Outputs, and
 *                     o and lse as inputs, are always dense.
 *   workspace         as for ssm_linattn_fwd, of the bytes the call's _workspace function gives (may be 0)
 * Products are exact bf16 products summed in fp32 (bf16) or fp32 products (f32); the softmax' statistics and all sums are
 * fp32. With bf16, weights enter the product with v in two bf16 parts, 2^-16 of each, so that o is its own rounding off; in
 * gradients weights and ds, those of the scores, enter theirs so as well. Results are deterministic. A NaN or Inf reaches the
 * queries that see its key and no others (an Inf in v may come out as NaN); in gradients it may also reach queries and keys of
 * the same sequence less than 160 from it, a query standing at its last key. A query all of whose scores are −Inf counts as one
 * that sees no key.
 * b, H, G, D >= 1; G divides H; D <= SSM_ATTN_MAX_D and scale finite (SSM_ERR_UNSUPPORTED otherwise); Lq, Lk <= 2^30; H·D and
 * strides between tokens at most 2^24; a launch takes fewer than 2^32 threads: SSM_ERR_SHAPE where b·H·⌈Lq/128⌉ or
 * b·G·⌈Lk/128⌉ (b·G rounded up to a multiple of 8, and ⌈./128⌉ to one of ⌈8/G⌉) reaches 2^23. Packed sequences count as
 * ⌊tokens/128⌋ + b blocks in place of b·⌈L/128⌉ (rounded up to a multiple of 8) where that is less and b·⌈L/128⌉ times the heads
 * passes 2^16. No output may overlap an input, the workspace or another output. Where few blocks of 128 queries (keys, in the
 * gradient for k and v) leave the device idle, the keys (queries) are summed in up to 16 pieces: then fp32 sums, and so the last
 * bits, depend on b, H, G, the lengths' bounds and tokens.
 */
#define SSM_ATTN_MAX_D 128
typedef ssm_linattn_strides_t ssm_attn_strides_t;
typedef struct {
    const int32_t *cu_q, *cu_k, *len_q, *len_k;
    int64_t b, Lq, Lk, tokens_q, tokens_k;
} ssm_attn_rows_t;

SSM_API ssm_status_t ssm_attn_fwd_workspace(const ssm_attn_rows_t *rows, int64_t H, int64_t G, int64_t D, ssm_dtype_t dtype,
                                            int64_t *bytes);
SSM_API ssm_status_t ssm_attn_fwd(const void *q, const void *k, const void *v, float scale, int32_t causal,
                                  const ssm_attn_rows_t *rows, void *o, float *lse, int64_t H, int64_t G, int64_t D,
                                  ssm_dtype_t dtype, const ssm_attn_strides_t *strides, void *workspace,
                                  int64_t workspace_bytes, hipStream_t stream);

/* Gradients for an upstream gradient do_ on o, from the forward call's o and lse. dq [tokens][H][D], dk and dv
 * [tokens][G][D] (summed over the heads that share a key head, in fp32) dtype, all required. workspace as for
 * ssm_linattn_bwd, of the bytes ssm_attn_bwd_workspace gives. delta_i = do_i·o_i; with bf16, where o is rounded, it is
 * Σ_j p_ij do_i·v_j wherever that is within twice that rounding (2^-7 Σ_d |do_id o_id|) of do_i·o_i. So results are their own
 * rounding off, and o and lse may also be those of more keys than the call is given: with keys in shards, each call's dk and dv are
 * its keys', and dq is the sum of the calls' (with bf16 as exact as do_i·o_i of the rounded o). */
SSM_API ssm_status_t ssm_attn_bwd_workspace(const ssm_attn_rows_t *rows, int64_t H, int64_t G, int64_t D, int64_t *bytes);
SSM_API ssm_status_t ssm_attn_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                                  const void *do_, float scale, int32_t causal, const ssm_attn_rows_t *rows, void *dq,
                                  void *dk, void *dv, int64_t H, int64_t G, int64_t D, ssm_dtype_t dtype,
                                  const ssm_attn_strides_t *strides, void *workspace, int64_t workspace_bytes,
                                  hipStream_t stream);

/*
 * A paged cache of keys and values: token t of row i is in slot t mod page_size of page
 * page_table[i·max_pages + t / page_size].
 *   k_cache, v_cache  [pages][page_size][G][D] dtype; pages k_page and v_page elements apart (0: dense), so that both may
 *                     lie in one pool
 *   page_table        [b][max_pages] int32 on the device. An entry outside 0 .. pages − 1 is a page that is not there: its
 *                     tokens are not attended to, and not stored
 * pages, page_size, max_pages >= 1, page_size <= 2^20, max_pages·page_size <= 2^30, G·D <= 2^24.
 */
typedef struct {
    const int32_t *page_table;
    int64_t pages, page_size, max_pages, k_page, v_page;
} ssm_pages_t;

/* Attention of one new token a row, over the row's tokens in the cache (its own among them, ssm_kv_append stores it):
 *   q                 [b][H][D] dtype, rows q_b and heads q_h elements apart (0, 0: dense)
 *   lengths           [b] int32 on the device: tokens of each row in the cache, taken as 0 below 0 and as max_pages·page_size
 *                     above that. Rows of length 0 have o = 0 and lse = −inf. Nothing past them is read.
 *   o, lse            [b][H][D] dtype, required; [b][H] fp32 or NULL
 *   max_len           the longest length the call is planned for (0: max_pages·page_size); rows may be longer
 *   workspace         as for ssm_linattn_fwd, of the bytes ssm_attn_step_workspace gives (0 where no row is split)
 * Arithmetic, limits and errors as for ssm_attn_fwd; b·G·⌈H/G/16⌉ times the pieces (up to ⌈max_len/256⌉) and b·H below 2^24. */
SSM_API ssm_status_t ssm_attn_step_workspace(int64_t b, int64_t H, int64_t G, int64_t D, const ssm_pages_t *pages,
                                             int64_t max_len, int64_t *bytes);
SSM_API ssm_status_t ssm_attn_step(const void *q, const void *k_cache, const void *v_cache, const ssm_pages_t *pages,
                                   const int32_t *lengths, float scale, void *o, float *lse, int64_t b, int64_t H, int64_t G,
                                   int64_t D, int64_t q_b, int64_t q_h, int64_t max_len, ssm_dtype_t dtype, void *workspace,
                                   int64_t workspace_bytes, hipStream_t stream);

/*
 * New tokens into the cache, with the position rotation on the way. Coordinates of a head are turned in pairs: pair
 * m < rotary/2 of a token at position t by the angle t·freq[m] (coordinates m and m + rotary/2, or 2m and 2m + 1 where
 * interleaved), the others stay:  (x, y) -> (x cos − y sin, y cos + x sin). Angles are formed and reduced in fp64.
 *   tokens            which rows the T new tokens belong to: cu NULL: b rows of L tokens, T = b·L, of which new_lengths[i] (or
 *                     NULL: all) count; cu given: b + 1 rising offsets on the device, row i has those from cu[i] to cu[i+1]
 *   lengths           [b] int32 on the device: tokens of each row with the new ones; the new ones are the row's last.
 *                     NULL (ssm_rope only): they are all there are
 *   q, q_out          [T][H][D] dtype: rotated; both NULL, or q_out may be q (dense)
 *   k, k_out          [T][G][D] dtype: rotated into the cache and, where k_out is not NULL, into it; k_out may be k (dense)
 *   v                 [T][G][D] dtype: into the cache
 *   freq              [rotary/2] fp64 on the device, radians a position, or NULL: no rotation. rotary even, 2 .. D
 *   strides           as for ssm_attn_fwd (do_'s are not used)
 * Tokens whose position the row's pages do not reach are not stored. Two new tokens on the same slot (rows that share a page)
 * leave either's values there. Outputs q_out and k_out of tokens that belong to no row are 0 (left as they are in place). T below
 * 2^24, H, G, D and strides as for ssm_attn_fwd, errors too.
 */
typedef struct {
    const int32_t *cu, *new_lengths;
    int64_t b, L, T;
} ssm_tokens_t;
SSM_API ssm_status_t ssm_kv_append(const void *q, const void *k, const void *v, void *q_out, void *k_out, void *k_cache,
                                   void *v_cache, const ssm_pages_t *pages, const int32_t *lengths, const ssm_tokens_t *tokens,
                                   const double *freq, int64_t rotary, int32_t interleaved, int64_t H, int64_t G, int64_t D,
                                   ssm_dtype_t dtype, const ssm_attn_strides_t *strides, hipStream_t stream);

/* The rotation alone: x [T][H][D] dtype, x_b, x_t, x_h elements apart (all 0: dense), to out (dense; may be x where that is
 * dense). inverse: by the opposite angles, which is the gradient. */
SSM_API ssm_status_t ssm_rope(const void *x, void *out, const int32_t *lengths, const ssm_tokens_t *tokens, const double *freq,
                              int64_t rotary, int32_t interleaved, int32_t inverse, int64_t H, int64_t D, int64_t x_b,
                              int64_t x_t, int64_t x_h, ssm_dtype_t dtype, hipStream_t stream);

/*
 * Options of ssm_scan_fwd_ex. Zero-initialise, then set what you need; zero means "choose".
 *   seg_len            time-segment length (multiple of 32) carried across by the chunk-carry
 *                      pass; 0 = chosen from the shape, >= L = one segment
 *   lanes_per_channel  1, 2 or 4 lanes of a wavefront share one channel's N states (a wavefront
 *                      then covers 64 / this channels; each lane holds at most 16 states);
 *                      0 = chosen from the shape
 *   initial_state    [b][d][N] fp32 device pointer, h_{−1} (NULL = zeros); lets a caller
 *                    continue a sequence that an earlier call ended (pass its final_state)
 *   ev_begin, ev_end hipEvent_t values (may be NULL); when set, the dispatch of the output-pass
 *                    kernel of the fast (scaled-state) path sets them at its start and end, for
 *                    timing that kernel alone (hipExtLaunchKernel's start/stop events)
 */
typedef struct {
    int32_t seg_len;
    int32_t lanes_per_channel;
    const float *initial_state;
    void *ev_begin;
    void *ev_end;
    int64_t reserved[4];
} ssm_fwd_opts_t;

/* ssm_scan_fwd with explicit options (opts may be NULL = all defaults). */
SSM_API ssm_status_t ssm_scan_fwd_ex(const void *x, const void *delta, const float *A, const void *B,
                             const void *C, const float *D, const void *z, void *y,
                             float *final_state, int64_t b, int64_t d, int64_t L, int64_t N,
                             ssm_dtype_t dtype, hipStream_t stream, const ssm_fwd_opts_t *opts);

/* The launch plan ssm_scan_fwd_ex would use for this shape and these options (host only, no
 * device work), planned for a 256-CU device (MI355X): the resolved segment length, lanes per
 * channel and states per lane, the number of segments, the one-wavefront workgroups of each
 * segment and of each pass, and the scratch bytes. Returns SSM_OK or the validation error. */
typedef struct {
    int32_t seg_len;
    int32_t lanes_per_channel;
    int32_t states_per_lane;
    int32_t n_segments;
    int64_t waves_per_segment;
    int64_t groups_output_pass;
    int64_t groups_aggregate_pass;
    int64_t scratch_bytes;
} ssm_fwd_plan_t;

SSM_API ssm_status_t ssm_scan_fwd_plan(int64_t b, int64_t d, int64_t L, int64_t N, ssm_dtype_t dtype,
                               const ssm_fwd_opts_t *opts, ssm_fwd_plan_t *plan);

/*
 * ssm_scan_fwd_ex that allocates nothing, for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, and harnesses that forbid allocation. Same arguments, plan,
 * kernels and results as ssm_scan_fwd_ex. The scratch of a time-split plan (the segment aggregates,
 * and the carries past 16 segments: ssm_fwd_plan_t.scratch_bytes) lives in a fixed device array of
 * SSM_NOALLOC_SCRATCH_BYTES that each GPU the library runs on holds from its first use until the
 * process ends; no hipMalloc, hipFree or allocating library routine is called. A plan needing more
 * returns SSM_ERR_SCRATCH and launches nothing (a longer seg_len in opts shrinks it). Every call on a
 * GPU shares that GPU's array, which keeps the last call's contents: calls that overlap on one GPU
 * (different streams, or host threads) race and must be serialised by the caller. Nothing in the
 * array needs clearing: a call writes every scratch word before reading it. Other errors as for
 * ssm_scan_fwd.
 */
#define SSM_NOALLOC_SCRATCH_BYTES (32ll << 20)
SSM_API ssm_status_t ssm_scan_fwd_noalloc(const void *x, const void *delta, const float *A, const void *B,
                                          const void *C, const float *D, const void *z, void *y,
                                          float *final_state, int64_t b, int64_t d, int64_t L, int64_t N,
                                          ssm_dtype_t dtype, hipStream_t stream, const ssm_fwd_opts_t *opts);

/* Human-readable name of a status code (static string, never NULL). */
SSM_API const char *ssm_status_string(ssm_status_t s);

/* SSM_ABI_VERSION of the loaded library. */
SSM_API int ssm_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* SSM_SCAN_H */
