/* ps.h - C ABI of the MI355X (gfx950) fused low-precision optimizer step.
 *
 * One shared library, libps.so, built from precision_state_amd/csrc. Every
 * entry point is extern "C", takes plain pointers and sizes, and returns a
 * ps_status. Device pointers are HIP device memory (any allocator); calls are
 * asynchronous and ordered on the HIP stream passed in (NULL = the default
 * stream); nothing here synchronises unless stated.
 *
 * Pages this library implements (cited by title and section):
 *  [KAHAN]   kohya-ss/sd-scripts PR #2159, "Kahan summation for
 *            Adafactor-optimized Flux FFT": keep the 16 low bits that the bf16
 *            weight drops, restore the exact fp32 value before each update.
 *  [NADAM]   kohya-ss/sd-scripts PR #2187, "(N)AdamW / Adan with fused
 *            backwards pass & CPU offloading": opening post (AdamW / NAdamW
 *            with Kahan residuals, moments offloaded to host memory) and second
 *            post (moments stored as scaled, biased, pow()-companded uint16).
 *  [ADAF]    kohya-ss/sd-scripts commit 7983d3d, "Fused backward pass",
 *            library/adafactor_fused.py (factored second moment, update
 *            clipping, tensors without a gradient skipped).
 *  [PRODIGY] konstmish/prodigy PR #25, "no first moment and factored second
 *            moment" (beta1 = 0, factored v, update clipping, eps on g^2).
 *
 * Arithmetic contract (all kernels): IEEE binary32, round to nearest even,
 * fused multiply-add only where the formula below says fma, correctly
 * rounded division and square root, denormals preserved. Inputs are assumed
 * finite; results for non-finite inputs are unspecified.
 *
 * Error behaviour: every argument is validated on the host before any HIP
 * call, so a rejected call touches no device state and needs no GPU. A HIP
 * failure at launch returns PS_ERR_HIP. ps_last_error() gives a message for
 * the calling thread's most recent failure.
 */
#ifndef PS_H
#define PS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as hipStream_t. */
typedef struct ihipStream_t* ps_stream_t;

typedef int32_t ps_status;
enum {
  PS_OK = 0,
  PS_ERR_INVALID_ARG = 1, /* NULL where a pointer is required, bad enum, bad hyperparameter */
  PS_ERR_ALIGNMENT = 2,   /* a 16-bit or fp32 array not 16-byte aligned (scales: 4 bytes) */
  PS_ERR_SHAPE = 3,       /* numel < 0, rows * cols != numel, sizes out of range */
  PS_ERR_UNSUPPORTED = 4, /* valid but not implemented combination */
  PS_ERR_HIP = 5,         /* the HIP runtime reported an error */
  PS_ERR_NO_MEMORY = 6,   /* host or device allocation failed */
  PS_ERR_WORKSPACE = 7    /* caller workspace smaller than required */
};

enum { PS_ALGO_ADAM = 0, PS_ALGO_NADAM = 1 };
enum { PS_SPLIT_TRUNC = 0, PS_SPLIT_NEAREST_AWAY = 1, PS_SPLIT_STOCHASTIC = 2 };
enum { PS_MOMENT_SIGNED = 0, PS_MOMENT_UNSIGNED = 1 };

/* Elements per moment-scale block. */
#define PS_BLOCK 256

/* Per-tensor storage flags (ps_tensor.flags) [NADAM, second post: tensors of
 * at most 4096 elements keep fp32 moments; third post: the final layer trains
 * in fp32]. The update arithmetic is unchanged; only the storage differs.
 *   PS_TENSOR_FP32_MOMENTS  m_code and v_code point to float[numel] moments
 *                           (no codec); m_scale and v_scale are not used
 *   PS_TENSOR_FP32_PARAM    w_hi points to the float[numel] parameter and grad
 *                           to a float[numel] gradient (no residual); w_lo is
 *                           not used
 *   PS_TENSOR_F24_MOMENTS   [NADAM, third post: moments in the upper three
 *                           bytes of fp32] m_code and v_code point to
 *                           uint8[3 * numel]: value i is bytes 3i..3i+2, the
 *                           fp32 word's bits 8..31 little-endian (low byte
 *                           implied zero), rounded to nearest, ties to even;
 *                           m_scale and v_scale are not used. Excludes
 *                           PS_TENSOR_FP32_MOMENTS.
 * Supported by ps_opt_step_multi only (the factored step and the offload
 * pipeline reject non-zero flags with PS_ERR_UNSUPPORTED). */
enum { PS_TENSOR_FP32_MOMENTS = 1u << 0, PS_TENSOR_FP32_PARAM = 1u << 1, PS_TENSOR_F24_MOMENTS = 1u << 2 };

/* One parameter tensor's state. All arrays are device memory owned by the
 * caller, contiguous, `numel` elements unless noted; 16-bit and fp32 element
 * arrays must be 16-byte aligned, scale arrays 4-byte aligned.
 *   w_hi    bf16 weight bits (the model's parameter), read and written
 *   w_lo    uint16 residual: the fp32 master weight's low half [KAHAN]
 *   grad    bf16 gradient bits, read only; NULL skips the tensor [ADAF]
 *   m_code  exp_avg codes, signed kind (32768 +- k); unused by the factored step
 *   m_scale exp_avg block scales, ceil(numel / 256) floats
 *   v_code  exp_avg_sq codes, unsigned kind (k)
 *   v_scale exp_avg_sq block scales, ceil(numel / 256) floats
 *   row_ema, col_ema  factored step only: fp32[rows], fp32[cols]
 *   rows, cols        factored step only: rows * cols == numel for a 2-D
 *                     tensor (factored), both 0 for a 1-D tensor (v kept in
 *                     v_code / v_scale)
 * flags       PS_TENSOR_* storage flags (0: the formats above); reserved = 0
 * A tensor with numel == 0 is skipped and its pointers are not read. */
typedef struct ps_tensor {
  uint16_t* w_hi;
  uint16_t* w_lo;
  const uint16_t* grad;
  uint16_t* m_code;
  float* m_scale;
  uint16_t* v_code;
  float* v_scale;
  float* row_ema;
  float* col_ema;
  int64_t numel;
  int64_t rows;
  int64_t cols;
  uint32_t flags;
  uint32_t reserved;
} ps_tensor;

/* (N)AdamW hyperparameters [NADAM]. Constraints: algo in {ADAM, NADAM};
 * split_mode in {TRUNC, NEAREST_AWAY, STOCHASTIC}; lr >= 0; 0 <= beta1 < 1;
 * 0 <= beta2 < 1; eps > 0 and nonzero once rounded to fp32;
 * weight_decay >= 0; momentum_decay >= 0 (NAdam's psi, 0.004 by default);
 * all finite.
 *
 * split_mode STOCHASTIC [KAHAN, PR #2159 body: the stochastic rounding the
 * residual replaces; NADAM opening post]: no residual. w_lo is neither read
 * nor written (may be NULL); the master weight is the bf16 value itself, and
 * the updated fp32 weight w' is rounded to one of its two neighbouring bf16
 * values, away from zero with probability (low 16 bits of w') / 2^16:
 *   hi = (bits(w') + r) >> 16
 * with r the element's random 16 bits. They come from a SplitMix64 stream
 * (Steele, Lea, Flood, OOPSLA 2014; mix(z) = its output finaliser, G =
 * 0x9E3779B97F4A7C15): for the tensor at index i of the list and update
 * `step`, the stream starts at s = mix(seed ^ mix((step mod 2^32) << 32 | i));
 * element e takes bits 16*(e % 4) .. 16*(e % 4) + 15 of mix(s + (e/4 + 1) * G).
 * The same (seed, step, list position) always gives the same bits, so a
 * caller that steps one tensor per call (position 0 every time, as from a
 * gradient hook) should give each tensor a seed of its own, or all of them
 * draw the same stream. Supported by ps_opt_step_multi, the factored step
 * (ps_factored_hparams.seed) and the offload pipeline (which then moves no
 * residual); ps_split and ps_join return PS_ERR_UNSUPPORTED for it. `seed`
 * is not read in the other modes. */
typedef struct ps_hparams {
  int32_t algo;
  int32_t split_mode;
  double lr;
  double beta1;
  double beta2;
  double eps;
  double weight_decay;
  double momentum_decay;
  uint64_t seed;
} ps_hparams;

/* Factored-second-moment hyperparameters [ADAF; PRODIGY]: eps1 added to g^2,
 * update clipped to RMS clip_threshold.
 *   decay_rate  0: constant beta2. < 0: Adafactor's schedule [ADAF]: beta2 of
 *               update t is 1 - t^decay_rate (beta2 is then ignored); B2 and
 *               C2 = 1 - beta2_t are each rounded once from double
 *   beta1       0: no first moment [PRODIGY]. In (0, 1): the clipped,
 *               lr-scaled update x is replaced by its EMA m = fma(B1, m0, C1*x)
 *               (B1 = fp32(beta1), C1 = fp32(1 - beta1)) before weight decay
 *               [ADAF], m kept in m_code / m_scale (signed codec, per-256
 *               blocks of the flattened tensor); 2-D tensors then need
 *               numel < 2^31 (else PS_ERR_UNSUPPORTED)
 *   split_mode  TRUNC, NEAREST_AWAY, or STOCHASTIC (no residual; the random
 *               bits exactly as for ps_hparams, from `seed`, the update
 *               number and the tensor's index in the list)
 * Constraints: lr >= 0; 0 <= beta2 < 1; eps1 > 0 and nonzero once rounded to fp32;
 * clip_threshold > 0; weight_decay >= 0; decay_rate <= 0;
 * 0 <= beta1 < 1; all finite. */
typedef struct ps_factored_hparams {
  int32_t split_mode;
  int32_t reserved; /* must be 0 */
  double lr;
  double beta2;
  double eps1;
  double clip_threshold;
  double weight_decay;
  double decay_rate;
  double beta1;
  uint64_t seed;
} ps_factored_hparams;

/* ps_opt_step_multi - one fused (N)AdamW step over a list of tensors, in ONE
 * kernel launch [NADAM; KAHAN].
 * Per element, for update number `step` (>= 1, the first update is 1 [ADAF]):
 *   w   = join(w_hi, w_lo)                      exact fp32 master weight
 *   g   = fp32(grad)
 *   m0  = decode(m_code, m_scale), v0 = decode(v_code, v_scale)
 *   m   = fma(B1, m0, C1*g);  v = fma(B2, v0, C2*(g*g))
 *   d   = fma(sqrt(v), RS2, EPS)
 *   ADAM:  u = A*(m/d)             NADAM: u = fma(AG, g, AM*m)/d
 *   if weight_decay != 0: u = fma(CWD, w, u)    (decoupled, additive form)
 *   w'  = w - u;  (w_hi, w_lo) = split(w')
 *   new block scales = max|m|, max v over each 256-element block of this
 *   step's fp32 moments; codes re-encoded with them.
 * Scalars (ps_step_scalars) are computed on the host in double and rounded
 * once. `tensors` is a host array of n_tensors records (n_tensors == 0 is a
 * no-op); it is copied during the call. Lists of up to 16 records travel in
 * the kernel arguments; for longer lists, and for the records with storage
 * flags, the library keeps a device copy of each distinct list it has seen,
 * so repeated calls with the same list upload nothing. That cache holds up
 * to 16384 lists or 64 MiB per device; when it is full, the call waits
 * until no other call is between taking a cached list and enqueueing the
 * launch that reads it, then synchronizes the device once and empties it. Tensors with storage flags go
 * to a second launch with a generic-format kernel. Calls from several host
 * threads, on their own streams and over distinct tensors, are safe.
 * Errors: PS_ERR_INVALID_ARG, PS_ERR_ALIGNMENT, PS_ERR_SHAPE (host checks,
 * before any device work); PS_ERR_HIP; PS_ERR_NO_MEMORY. */
ps_status ps_opt_step_multi(const ps_tensor* tensors, int32_t n_tensors, const ps_hparams* hp, int64_t step,
                            ps_stream_t stream);

/* ps_step_scalars - the fp32 scalars of update number `step`, as used by
 * ps_opt_step_multi: out[0..9] = B1, C1, B2, C2, EPS, A, RS2, AG, AM, CWD.
 * Host only (no GPU needed). */
ps_status ps_step_scalars(const ps_hparams* hp, int64_t step, float out[10]);

/* ps_split / ps_join - fp32 master weight <-> (bf16 weight, uint16 residual)
 * [KAHAN, copy_kahan_ docstring]. Elementwise over n >= 0 elements.
 *   TRUNC:        hi = bits >> 16, lo = bits & 0xFFFF (bf16 truncated toward 0)
 *   NEAREST_AWAY: hi = ((bits + 0x8000) >> 16) & 0xFFFF (bf16 rounded to
 *                 nearest, ties away from zero), lo = bits & 0xFFFF
 * join inverts split exactly for every 32-bit pattern in both modes. */
ps_status ps_split(const float* w32, uint16_t* hi, uint16_t* lo, int64_t n, int32_t mode, ps_stream_t stream);
ps_status ps_join(const uint16_t* hi, const uint16_t* lo, float* w32, int64_t n, int32_t mode,
                  ps_stream_t stream);

/* ps_encode_moments / ps_decode_moments - the uint16 moment codec [NADAM,
 * second post], 1/4-power companding, one fp32 scale per 256-element block
 * (the last block of the array covers n mod 256 elements).
 * Encode, per block: s = max |x|; if s < 2^-126 then scale = 0 and every
 * code is the zero code (SIGNED 32768, UNSIGNED 0); else inv = 1/s and for
 * each element x' = |x|*inv and k = the largest k in 0..Q with k == 0 or
 * x' >= D(k - 1/2), where D(h) = ((h*K)^2)^2, K = fp32(1/Q), Q = 32767
 * (SIGNED) or 65535 (UNSIGNED). SIGNED code = 32768 - k for x < 0 else 32768 + k;
 * UNSIGNED code = k (the sign of x is ignored).
 * Decode: SIGNED x = sign(c - 32768) * D(|c - 32768|) * s; UNSIGNED x = D(c) * s.
 * scale has ceil(n / 256) entries. */
ps_status ps_encode_moments(const float* x, uint16_t* code, float* scale, int64_t n, int32_t kind,
                            ps_stream_t stream);
ps_status ps_decode_moments(const uint16_t* code, const float* scale, float* x, int64_t n, int32_t kind,
                            ps_stream_t stream);

/* ps_factored_workspace_size - device workspace bytes ps_factored_step needs
 * for this tensor list (partial row/column sums and per-tensor reductions).
 * Host only. */
ps_status ps_factored_workspace_size(const ps_tensor* tensors, int32_t n_tensors, size_t* bytes);
/* (The workspace does not depend on the hyperparameters: a first moment lives
 * in the tensors' m_code / m_scale.) */

/* ps_factored_step - Adafactor-style step [ADAF; PRODIGY]. For a 2-D tensor
 * [rows, cols] (row-major):
 *   q_ij = g_ij*g_ij + EPS1
 *   r_i = fma(B2, r_i, C2*fp32(mean_j q_ij)),  c_j = fma(B2, c_j, C2*fp32(mean_i q_ij))
 *   rbar = fp32(mean_i r_i); rho_i = 1/sqrt(r_i/rbar); kap_j = 1/sqrt(c_j)
 *   U_ij = (g_ij*rho_i)*kap_j; f = fp32(lr / max(1, RMS/clip_threshold)),
 *     RMS = sqrt(mean_ij g_ij^2 * mean_i(r_i) / (r_i c_j)) in double: the RMS
 *     of the exact U for the new EMAs
 *   x = U*f; with beta1: m = fma(B1, decode(m), C1*x), x = m, m re-encoded
 *   w' = w - x after x = fma(CWD, w, x) if weight_decay != 0
 * Means and RMS are accumulated in double. A 1-D tensor keeps v in the
 * uint16 codec: v = fma(B2, decode(v), C2*q); U = g*(1/sqrt(v)); the clip's
 * RMS = sqrt(mean g^2 / v) in double.
 * workspace: device memory of at least ps_factored_workspace_size bytes,
 * 256-byte aligned, owned by the caller; its contents on entry are ignored;
 * calls that may run at the same time need distinct workspaces. The step's
 * device plan goes through the same cache as ps_opt_step_multi's lists.
 * Errors as ps_opt_step_multi, plus PS_ERR_WORKSPACE. */
ps_status ps_factored_step(const ps_tensor* tensors, int32_t n_tensors, const ps_factored_hparams* hp,
                           int64_t step, void* workspace, size_t workspace_bytes, ps_stream_t stream);

/* ps_factored_step_noalloc - for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): ps_factored_step with no workspace argument and no device
 * allocation. The plan and the workspace go to a scratch array that the
 * library keeps in each GPU's memory for the life of the process,
 * PS_NOALLOC_SCRATCH_BYTES per GPU (its address is looked up on the first
 * call on each device). The plan, rounded up to 256 bytes, plus
 * ps_factored_workspace_size must fit in it, else the call returns
 * PS_ERR_WORKSPACE before any device work; one FLUX double block (24 tensors,
 * 22.0 MiB of workspace) fits. The plan reaches the scratch through kernel
 * arguments, so the call makes no copy from host memory either. Same kernels
 * and results as ps_factored_step; the scratch's contents on entry are
 * ignored. Every call on one GPU uses that GPU's single scratch array: calls
 * ordered on one stream are safe, calls that may overlap on one GPU (other
 * streams or host threads without ordering between them) race and must not
 * be made. Errors as ps_factored_step. */
#define PS_NOALLOC_SCRATCH_BYTES (32u << 20)
ps_status ps_factored_step_noalloc(const ps_tensor* tensors, int32_t n_tensors, const ps_factored_hparams* hp,
                                   int64_t step, ps_stream_t stream);

/* ---------------------------------------------------------------------------
 * AdamW over many tensors with 32-bit or 8-bit moments, and the global
 * gradient norm that clips it: the step of mixed-precision training, where a
 * model runs on 16-bit copies of fp32 master weights (or on bf16 weights, with
 * a residual or stochastic rounding), its parameters fall into groups with
 * hyperparameters of their own and its gradients are clipped by their norm.
 *
 * A PLAN is made once from the tensor list and then run every step. It reads
 * and writes a workspace that the caller owns (device memory), so a run
 * allocates nothing, copies nothing from the host and can be captured into a
 * HIP graph.
 * ------------------------------------------------------------------------- */

/* Element types of parameters, gradients and copies. */
enum { PS_TYPE_F32 = 0, PS_TYPE_BF16 = 1, PS_TYPE_F16 = 2 };
/* Moment storage of a tensor.
 *   PS_STATE_F32   m, v: float[numel]
 *   PS_STATE_E4M3  m, v: one byte per element (OCP e4m3fn), one scale per 256
 *                  elements; v holds sqrt(v). See ps_encode_fp8. */
enum { PS_STATE_F32 = 0, PS_STATE_E4M3 = 1 };
/* Rounding of the second moment's e4m3 codes. With beta2 = 0.999 a second
 * moment whose gradient has become small shrinks by 0.05% of sqrt(v) a step,
 * far less than half a code, so rounding to the nearest leaves it where it is
 * until its block's scale changes; STOCHASTIC moves it by the right amount on
 * average. */
enum { PS_ROUND_NEAREST = 0, PS_ROUND_STOCHASTIC = 1 };

#define PS_ADAMW_MAX_GROUPS 16

/* One parameter tensor. Contiguous device arrays of numel elements, 16-byte
 * aligned (scales: 4 bytes).
 *   param     float (PS_TYPE_F32) or bf16 (PS_TYPE_BF16), read and written.
 *             NULL: only the gradient counts (ps_adamw_grad_norm), the step
 *             passes the tensor by
 *   residual  PS_TYPE_BF16: the low halves of the fp32 master weights, as
 *             ps_tensor.w_lo; may be NULL if the steps' split_mode is
 *             STOCHASTIC. PS_TYPE_F32: NULL
 *   copy      PS_TYPE_F32: array of copy_type (BF16 or F16) that each step
 *             writes the new weights to, rounded to nearest even; NULL: none.
 *             PS_TYPE_BF16: NULL
 *   grad      array of grad_type, read only; NULL: the tensor is passed by
 *             (a later ps_adamw_set_grads may give it one)
 *   m, v      moments (state_type); m_scale, v_scale: PS_STATE_E4M3 only,
 *             ceil(numel / 256) floats. A moment is what ps_decode_fp8 makes of
 *             its code and scale; a step writes scales as ps_encode_fp8 does.
 *             All bytes zero is a fresh state
 *   group     index of the tensor's hyperparameters in ps_adamw_step's groups
 * A tensor with numel == 0 is passed by and its pointers are not read. */
typedef struct ps_adamw_tensor {
  void* param;
  uint16_t* residual;
  void* copy;
  const void* grad;
  void* m;
  float* m_scale;
  void* v;
  float* v_scale;
  int64_t numel;
  int32_t param_type;
  int32_t grad_type;
  int32_t copy_type;
  int32_t state_type;
  int32_t group;
  int32_t reserved; /* must be 0 */
} ps_adamw_tensor;

/* The first bytes of a plan's workspace, in device memory. ps_adamw_plan_create
 * sets grad_mul = 1, lr_mul = 1 and the rest to 0; a caller may read and write
 * them in stream order.
 *   norm      last ps_adamw_grad_norm: grad_scale * (2-norm of all gradients)
 *   grad_mul  last ps_adamw_grad_norm: what a clipped step multiplies the
 *             gradients by
 *   skip      last ps_adamw_grad_norm: 1 if a gradient was infinite or NaN; a
 *             clipped step then changes nothing
 *   skipped   number of ps_adamw_grad_norm calls that set skip
 *   step      updates made so far by steps that count on the device
 *   lr_mul    factor of the learning rate in steps that count on the device
 *             (a schedule for captured graphs) */
typedef struct ps_adamw_control {
  float norm;
  float grad_mul;
  uint32_t skip;
  uint32_t skipped;
  int64_t step;
  float lr_mul;
  uint32_t reserved[9];
} ps_adamw_control;

typedef struct ps_adamw_plan ps_adamw_plan;

/* ps_adamw_workspace_size - device workspace bytes of a plan over this list.
 * Host only. Errors: PS_ERR_INVALID_ARG, PS_ERR_ALIGNMENT, PS_ERR_SHAPE. */
ps_status ps_adamw_workspace_size(const ps_adamw_tensor* tensors, int32_t n_tensors, size_t* bytes);

/* ps_adamw_plan_create - checks the list and lays it out in the workspace
 * (256-byte aligned, at least ps_adamw_workspace_size bytes, on the current
 * device; its contents on entry are ignored, and it belongs to the plan until
 * the plan is destroyed and its last run has ended). Ordered on `stream`,
 * which it synchronizes; PS_ERR_UNSUPPORTED while `stream` is being captured.
 * The list itself is not kept. Arrays that are written (param, residual, copy,
 * moments, scales) must not overlap each other, a gradient or the workspace,
 * nor a gradient the workspace (PS_ERR_INVALID_ARG); gradients may overlap. */
ps_status ps_adamw_plan_create(const ps_adamw_tensor* tensors, int32_t n_tensors, void* workspace,
                               size_t workspace_bytes, ps_stream_t stream, ps_adamw_plan** plan);

/* ps_adamw_set_grads - new gradient arrays (types and sizes as before) for the
 * plan's tensors, in list order, n_grads == n_tensors; NULL: the tensor is
 * passed by from now on. Asynchronous, ordered on `stream`; the pointers are
 * copied during the call and travel in kernel arguments. */
ps_status ps_adamw_set_grads(ps_adamw_plan* plan, const void* const* grads, int32_t n_grads, ps_stream_t stream);

/* ps_adamw_grad_norm - the 2-norm of all the plan's gradients and the factor
 * that clips it, into the control block:
 *   norm = fp32(n), n = grad_scale * sqrt(sum g^2)
 *   grad_mul = fp32(grad_scale * min(1, max_norm / (n + 1e-6)))
 *   skip = 1 if n is infinite or NaN (grad_mul is then 0), else 0
 * Squares, sums and the formulas are in double, the sums in an order that
 * depends on the list's sizes and types only. grad_scale: finite, > 0 (the inverse of a loss
 * scale); max_norm: > 0, infinity for no clipping. */
ps_status ps_adamw_grad_norm(ps_adamw_plan* plan, double max_norm, double grad_scale, ps_stream_t stream);

/* ps_adamw_step - one (N)AdamW step over the plan's tensors.
 * groups[0 .. n_groups-1]: the hyperparameters of each group, n_groups at most
 * PS_ADAMW_MAX_GROUPS and above every tensor's group; algo and split_mode are
 * the same in all groups. Per element:
 *   g  = fp32(grad), times grad_mul if `clipped`
 *   m  = B1*m0 + C1*g;  v = B2*v0 + C2*(g*g);  r = sqrt(v);  d = r*RS2 + EPS
 *   ADAM: u = A*(m/d)             NADAM: u = (AG*g + AM*m)/d
 *   u  = u + CWD*w;  w' = w - u
 * Every operation is rounded to fp32 by itself (no fma; the sign of a zero
 * quotient is not specified); the scalars are those of ps_step_scalars. w is the fp32 parameter, the joined (bf16, residual)
 * pair, or with split_mode STOCHASTIC the bf16 value alone; w' is stored as
 * it is (and rounded to copy_type for the copy), split, or rounded
 * stochastically, with the random bits of ps_hparams for the tensor's index in
 * the plan's list. Moments are stored as fp32 or as ps_encode_fp8 would code m
 * and v; the update uses this step's fp32 values.
 *   step      >= 1: the update's number. 0: the number is counted in the
 *             control block: each call that is not skipped adds 1 and uses the
 *             sum, and the learning rate is lr * lr_mul (PS_ALGO_ADAM only;
 *             the scalars are then computed in double on the device)
 *   clipped   0 or 1: use the control block's grad_mul and skip
 *   rounding  PS_ROUND_*: the second moment's e4m3 codes. STOCHASTIC: the 16
 *             random bits of element e come from the stream of list index
 *             i + 2^31 (ps_hparams), fill the places below the last kept one
 *             and are cut off with them:
 *             code = floor(r/s in units of its last e4m3 place + bits / 2^16)
 * A captured call replays with the same step, groups and rounding: capture
 * calls with step = 0.
 * Calls on one plan must be ordered by the caller, as two calls on one stream
 * are; the current device must be the plan's (PS_ERR_INVALID_ARG).
 * What infinite or NaN gradients or state become is not specified, but a clipped
 * step after a norm that found such a gradient changes nothing.
 * Errors: PS_ERR_INVALID_ARG, PS_ERR_UNSUPPORTED, PS_ERR_HIP. */
ps_status ps_adamw_step(ps_adamw_plan* plan, const ps_hparams* groups, int32_t n_groups, int64_t step,
                        int32_t clipped, int32_t rounding, ps_stream_t stream);

/* Frees the host side of the plan. Waits for nothing: the workspace stays in
 * use until the plan's last run has ended. */
ps_status ps_adamw_plan_destroy(ps_adamw_plan* plan);

/* ps_encode_fp8 / ps_decode_fp8 - the 8-bit moment codec: OCP e4m3fn codes with
 * one fp32 scale per 256 elements (the last block covers n mod 256), a power of
 * two.
 * Encode, per block: y = x (SIGNED: a first moment) or sqrt(x) (UNSIGNED: a
 * second moment, x >= 0); s = the smallest power of two >= 2^-126 with
 * max|y| <= 448 s; code = y / s rounded to the nearest e4m3 value, ties to even;
 * UNSIGNED codes of x > 0 are at least 2^-9, the smallest e4m3 value, so that
 * no second moment above zero becomes zero.
 * Decode: SIGNED x = code * s; UNSIGNED x = (code * s)^2. Since s is a power of
 * two, SIGNED decode is exact and a block that is decoded and encoded again
 * keeps its values. A block with an infinite or NaN x has unspecified codes.
 * Arrays 16-byte aligned, scale 4-byte. */
ps_status ps_encode_fp8(const float* x, uint8_t* code, float* scale, int64_t n, int32_t kind, ps_stream_t stream);
ps_status ps_decode_fp8(const uint8_t* code, const float* scale, float* x, int64_t n, int32_t kind,
                        ps_stream_t stream);

/* ---------------------------------------------------------------------------
 * Activation checkpoints in 8 bits, and their use in the backward pass.
 *
 * What a forward pass saves for the backward one is held as e4m3 codes: the
 * inputs of linear layers and of feed-forward activations with a power-of-two
 * scale for each 128 columns of a row, normalised values with none. The
 * backward entries read the codes; no wider copy is made.
 *
 * Matrices are row-major; `ld` is the distance between rows in elements
 * (ld >= cols), codes are contiguous [rows, cols], scales contiguous
 * [rows, ceil(cols / 128)] floats. Arrays need the alignment of their element
 * only. `type` is the PS_TYPE_* of activations and their gradients; arithmetic
 * is fp32, each result rounded to `type` once, to nearest even. rows or cols of
 * 0: nothing is read, and only sums over no rows are written. rows < 2^31,
 * cols <= 2^24, rows * ceil(cols / 128) < 2^31.
 * What is written must not overlap anything else of the call unless it says so
 * (PS_ERR_INVALID_ARG). Calls allocate nothing and can be captured. An infinite
 * or NaN value is an ordinary input: where it goes through a code it becomes
 * NaN, so that it reaches the gradients that ps_adamw_grad_norm looks at.
 * ------------------------------------------------------------------------- */

/* Columns of a row that share a scale. */
#define PS_ACT_BLOCK 128

/* ps_encode_act / ps_decode_act - codes of a matrix and back. Per block:
 * s = the smallest power of two >= 2^-126 with max|x| <= 448 s over the finite
 * x; code = x / s rounded to the nearest e4m3 value, ties to even, NaN for an
 * infinite or NaN x. Decode: x = code * s (exact in fp32 and bf16, rounded to
 * fp16), whatever the finite scale. Decoded to its own type a finite x is
 * finite: 2^16 for fp16 and 2^128 for the other types, which codes of the largest
 * values stand for, become the type's largest value. */
ps_status ps_encode_act(const void* x, int32_t type, int64_t rows, int64_t cols, int64_t ld, uint8_t* code,
                        float* scale, ps_stream_t stream);
ps_status ps_decode_act(const uint8_t* code, const float* scale, void* x, int32_t type, int64_t rows, int64_t cols,
                        int64_t ld, ps_stream_t stream);

/* ps_glu_forward / ps_glu_backward - the activation of a feed-forward layer,
 * gated: out = f(a) * b, or not (b NULL): out = f(a).
 *   SILU       f(a) = a / (1 + exp(-a))
 *   GELU       f(a) = a * Phi(a), Phi the normal distribution function
 *   GELU_TANH  f(a) = a / 2 * (1 + tanh(sqrt(2 / pi) * (a + 0.044715 a^3)))
 * Forward: a_code, a_scale and, if gated, b_code, b_scale are what
 * ps_encode_act makes of a and b; all NULL: nothing is saved.
 * Backward, with a and b decoded: da = dout * b * f'(a), db = dout * f(a), and
 * out once more (NULL: not wanted). da or db may be dout itself (the same
 * pointer and ld), a and b may be halves of one matrix. b_code and b_scale NULL:
 * not gated, and db is NULL too. */
enum { PS_ACT_SILU = 0, PS_ACT_GELU = 1, PS_ACT_GELU_TANH = 2 };
ps_status ps_glu_forward(int64_t rows, int64_t cols, int32_t type, int32_t act, const void* a, int64_t lda,
                         const void* b, int64_t ldb, void* out, int64_t ldo, uint8_t* a_code, float* a_scale,
                         uint8_t* b_code, float* b_scale, ps_stream_t stream);
ps_status ps_glu_backward(int64_t rows, int64_t cols, int32_t type, int32_t act, const void* dout, int64_t ldd,
                          const uint8_t* a_code, const float* a_scale, const uint8_t* b_code, const float* b_scale,
                          void* da, int64_t lda, void* db, int64_t ldb, void* out, int64_t ldo, ps_stream_t stream);

/* The norms around a block's place in the residual stream: after the block
 * (post) and before the next one (pre), with the gate and scale between them.
 *   v = N1(y) * post_weight       N1: post_norm, NONE is v = y
 *   h = residual_scale * x + branch_scale * (gate * v)
 *   n = N2(h) * m + add           N2: pre_norm; m = mul, or 1 + mul (MUL_PLUS_ONE)
 * N(z) = z * r, r = 1 / sqrt(mean(z^2) + eps) (RMS) or (z - mean z) * r, with
 * the variance in place of the mean square (LAYER); means over a row's cols.
 * With no branch (y NULL) h is x. NULL vectors are left out (1, 0 for add).
 *   post_weight  [cols]; only with a post_norm
 *   gate         [cols], or [n_segs, cols] with GATE_BY_SEG
 *   mul, add     [cols], or [n_segs, cols] with MOD_BY_SEG
 *   seg_start    int32[n_segs + 1] in device memory, ascending: segment b is
 *                rows seg_start[b] .. seg_start[b + 1] - 1 (it may be empty).
 *                Rows of no segment are left as they are in every output and
 *                in no sum. NULL (n_segs 0): all rows are one segment
 * eps >= 0, scales finite; rows <= 2^30, cols <= PS_NORM_MAX_COLS. vec_type: PS_TYPE_* of the
 * four vectors. */
enum { PS_NORM_NONE = 0, PS_NORM_RMS = 1, PS_NORM_LAYER = 2 };
enum { PS_NORM_GATE_BY_SEG = 1u << 0, PS_NORM_MOD_BY_SEG = 1u << 1, PS_NORM_MUL_PLUS_ONE = 1u << 2 };
#define PS_NORM_MAX_COLS 16384
typedef struct ps_block_norm {
  int64_t rows;
  int64_t cols;
  const int32_t* seg_start;
  const void* post_weight;
  const void* gate;
  const void* mul;
  const void* add;
  double post_eps;
  double pre_eps;
  double residual_scale;
  double branch_scale;
  int32_t type;
  int32_t vec_type;
  int32_t post_norm;
  int32_t pre_norm;
  int32_t n_segs;
  uint32_t flags; /* PS_NORM_* bits */
} ps_block_norm;

/* Forward arrays. x, and y unless there is no branch, are read; n is written,
 * and h if there is a branch (h may be x itself, the same pointer and ld; NULL
 * without one). Saved for the backward pass, each NULL if not wanted (the
 * backward needs all that the call has):
 *   h_code, h_rstd  N2(h) as e4m3 (|N2(h)| <= sqrt(cols), no scale), r of N2
 *   y_code, y_rstd  with a post_norm: N1(y) as e4m3, r of N1
 *   y_code, y_scale with a gate and no post_norm: y as ps_encode_act codes it
 *                   (code * scale in fp32 is what the backward pass reads)
 * rstd arrays are float[rows]. */
typedef struct ps_block_norm_fwd {
  const void* x;
  int64_t ldx;
  const void* y;
  int64_t ldy;
  void* h;
  int64_t ldh;
  void* n;
  int64_t ldn;
  uint8_t* h_code;
  float* h_rstd;
  uint8_t* y_code;
  float* y_scale;
  float* y_rstd;
} ps_block_norm_fwd;

/* Backward arrays: the gradients dn of n and dh of h from elsewhere (NULL: 0)
 * are read with what the forward pass saved; dx and, with a branch, dy are
 * written (dy NULL: there is none, and the branch's gradients are not made).
 * dx or dy may be dh or dn itself. With xh, yh the decoded values and G the
 * whole gradient of h:
 *   G  = dh + back(dn * m, xh, h_rstd);  dx = residual_scale * G
 *   p  = branch_scale * G;  dy = back(p * gate * post_weight, yh, y_rstd), or
 *   p * gate with no post_norm
 *   back(g, z, r) = r * (g - z * mean(g z))          RMS
 *                   r * (g - mean g - z * mean(g z)) LAYER
 * Gradients of the vectors, float, shaped as they are, each NULL if not wanted:
 *   d_mul = sum dn * xh; d_add = sum dn; d_gate = sum p * yh * post_weight;
 *   d_post_weight = sum p * gate * yh
 * summed over the segment's rows, or over all segments', in an order that
 * depends on sizes and segments only. accumulate 1: they are added to what the
 * arrays hold. workspace: 16-byte aligned, ps_block_norm_workspace_size bytes;
 * its contents on entry are ignored and it belongs to one call at a time. */
typedef struct ps_block_norm_bwd {
  const void* dn;
  int64_t lddn;
  const void* dh;
  int64_t lddh;
  const uint8_t* h_code;
  const float* h_rstd;
  const uint8_t* y_code;
  const float* y_scale;
  const float* y_rstd;
  void* dx;
  int64_t lddx;
  void* dy;
  int64_t lddy;
  float* d_post_weight;
  float* d_gate;
  float* d_mul;
  float* d_add;
  void* workspace;
  size_t workspace_bytes;
  int32_t accumulate;
  int32_t reserved; /* must be 0 */
} ps_block_norm_bwd;

ps_status ps_block_norm_forward(const ps_block_norm* norm, const ps_block_norm_fwd* io, ps_stream_t stream);
/* Workspace bytes of a backward call with this rows, cols and n_segs. Host only. */
ps_status ps_block_norm_workspace_size(const ps_block_norm* norm, size_t* bytes);
ps_status ps_block_norm_backward(const ps_block_norm* norm, const ps_block_norm_bwd* io, ps_stream_t stream);

/* ps_linear_wgrad - the weight gradient of y = x W^T, W [out, in], from dy
 * [tokens, out] and the codes of x [tokens, in]:
 *   db[n]    = sum_t dy[t, n]
 *   dw[n, k] = mul[k] * (sum_t dy[t, n] * z[t, k]) + add[k] * db[n]
 * z is code * scale, or the code's value itself (scale NULL): with the h_code
 * of a block norm and its vectors as mul and add (NULL: 1 and 0; a mul that
 * means 1 + mul has to be given so), x is the norm's output n.
 * dy_type is PS_TYPE_BF16 or PS_TYPE_F16; z is multiplied in that type: bf16
 * holds it whole if scales are powers of two (2^128, which codes of 3.3e38 and
 * more stand for, is infinite), fp16 from 2^-21 on (below, it is rounded to a
 * multiple of 2^-24, which the codes of an fp16 x are already) up to 65504,
 * beyond which it is infinite. 2^16, which codes of an fp16 x from 63488 on stand
 * for, is 65504 as ps_decode_act has it; to that end a power of two in a block
 * whose scale is 2^8 or more is taken one step of fp16 lower. Products
 * and sums are fp32, in an order that depends on the sizes only. dw of dw_type
 * (PS_TYPE_*) with distance lddw between rows; db float[out], NULL: not wanted;
 * mul, add float[in]. accumulate 1: dw and db are added to what the arrays
 * hold, in fp32, and rounded once. tokens <= 2^30, lddy <= 2^24,
 * out_features * in_features <= 2^36. workspace as for a block norm's backward
 * call, ps_linear_wgrad_workspace_size bytes (0 of them: NULL). */
typedef struct ps_linear_wgrad_args {
  int64_t tokens;
  int64_t out_features;
  int64_t in_features;
  const void* dy;
  int64_t lddy;
  const uint8_t* code;
  const float* scale;
  const float* mul;
  const float* add;
  void* dw;
  int64_t lddw;
  float* db;
  void* workspace;
  size_t workspace_bytes;
  int32_t dy_type;
  int32_t dw_type;
  int32_t accumulate;
  int32_t reserved; /* must be 0 */
} ps_linear_wgrad_args;
ps_status ps_linear_wgrad_workspace_size(int64_t tokens, int64_t out_features, int64_t in_features, size_t* bytes);
ps_status ps_linear_wgrad(const ps_linear_wgrad_args* args, ps_stream_t stream);

/* Host-offload pipeline [NADAM, opening post: moments (and here the
 * residuals) live in host memory and cross PCIe every step].
 * A group is one set of tensors stepped together (e.g. one transformer
 * block). For every tensor, w_hi and grad are device pointers; w_lo, m_code,
 * m_scale, v_code and v_scale are PINNED HOST pointers (hipHostMalloc).
 * ps_offload_run steps the groups in order. In the STAGED mode group k's
 * host state is copied to a device staging slot on an upload stream, stepped,
 * and copied back on a download stream, with two slots so that uploads of
 * k+1 and downloads of k-1 overlap the step of k; in the DIRECT mode the step
 * kernel of group k works on the host arrays in place. The results are bit-identical
 * to ps_opt_step_multi on device-resident state (for stochastic rounding:
 * on the concatenation of the groups' tensor lists, whose positions key the
 * random streams).
 * Streams: STAGED makes an upload and a download stream, each created with a
 * CU mask (all CUs) so that each gets a hardware queue of its own and the two
 * directions overlap whatever other streams the process holds, and a
 * non-blocking stream for the step kernels; DIRECT makes one stream with a
 * CU mask of n_cus CUs for its kernels. Streams made with a CU mask are
 * blocking: they order themselves with the null stream of the device.
 * Stochastic rounding [NADAM, opening post: the stochastic updates used when
 * the residual does not fit in host memory]: runs with split_mode STOCHASTIC
 * move no residuals; w_lo may then be NULL, and a plan with any NULL w_lo
 * accepts only such runs (PS_ERR_INVALID_ARG otherwise). */
typedef struct ps_offload_group {
  const ps_tensor* tensors;
  int32_t n_tensors;
} ps_offload_group;

typedef struct ps_offload_plan ps_offload_plan;

/* Plan modes.
 *   PS_OFFLOAD_DIRECT  the step kernel reads and writes the host-resident
 *                      arrays in place over PCIe (through the device addresses
 *                      of the pinned allocations, hipHostGetDevicePointer), one
 *                      launch per group on a stream of the plan's own that is
 *                      restricted to n_cus compute units: no staging memory and
 *                      no copy engines; the rest of the GPU stays free for
 *                      other work
 *   PS_OFFLOAD_STAGED  two device staging slots, an upload and a download
 *                      stream (each with a hardware queue of its own) and the
 *                      step kernel on a third stream, as described above
 * Both move the same bytes over PCIe and give the same results. */
enum { PS_OFFLOAD_DIRECT = 0, PS_OFFLOAD_STAGED = 1 };
#define PS_OFFLOAD_DEFAULT_CUS 8
typedef struct ps_offload_options {
  int32_t mode;      /* PS_OFFLOAD_DIRECT or PS_OFFLOAD_STAGED */
  int32_t n_cus;     /* DIRECT: compute units the step kernels may use (0: all) */
  int32_t reserved0; /* must be 0 */
  int32_t reserved1; /* must be 0 */
} ps_offload_options;

/* Creates the plan: copies the group descriptions and builds the device
 * tables, streams and events. DIRECT also checks that every host array has a
 * device address; STAGED allocates two staging slots sized for the largest
 * group. Synchronous. options NULL: DIRECT on PS_OFFLOAD_DEFAULT_CUS compute
 * units. ps_offload_plan_create(g, n, p) is ps_offload_plan_create_ex(g, n,
 * NULL, p). */
ps_status ps_offload_plan_create(const ps_offload_group* groups, int32_t n_groups, ps_offload_plan** plan);
ps_status ps_offload_plan_create_ex(const ps_offload_group* groups, int32_t n_groups,
                                    const ps_offload_options* options, ps_offload_plan** plan);
/* Runs one optimizer step over all groups; asynchronous on `stream` (the
 * call returns once all work is queued; host state is final when `stream`
 * completes). Successive runs of one plan are ordered among themselves even
 * when given different streams; one plan must not be run from two host
 * threads at once. */
ps_status ps_offload_run(ps_offload_plan* plan, const ps_hparams* hp, int64_t step, ps_stream_t stream);
/* Bytes the most recent run moved host->device and device->host (before
 * any run: the bytes of a run with residuals). */
ps_status ps_offload_bytes(const ps_offload_plan* plan, uint64_t* h2d_bytes, uint64_t* d2h_bytes);
/* Waits for outstanding work and frees everything the plan owns. */
ps_status ps_offload_plan_destroy(ps_offload_plan* plan);

/* Static description of a status code. */
const char* ps_status_string(ps_status status);
/* Message of the calling thread's most recent failed call ("" if none). */
const char* ps_last_error(void);
/* Library version string. */
const char* ps_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PS_H */
