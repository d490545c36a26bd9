/*
 * libmuon -- the Muon optimizer step for AMD Instinct MI355X (gfx950).
 *
 * C ABI.  Plain pointers and sizes only; no C++ or framework types cross it.
 * All device memory (parameters, gradients, momentum buffers, outputs and the
 * workspace) is owned by the caller.  The library launches work on the
 * caller's HIP stream and never waits for it, except where a function below
 * says so.  A step whose matrices fall both into the fused class and into a
 * tiled class (muon_step) also uses one stream of the library's own per
 * device (a plan: its own), forked from the caller's stream with an event
 * after the normalisation pass and joined back before the update pass: work
 * queued on the caller's stream before the call still runs first, work queued
 * after it still sees the finished step.
 *
 * What one step computes, for every 2-D matrix in the list (pages cited by
 * title and section):
 *   1. momentum, EMA form:        M <- mu*M + (1-mu)*G
 *        ("Muon optimizer: matrix-aware LLM", airosetta.com, Muon.step loop;
 *         "Muon meets Mamba", wmrh.cn, section 4.2 _step_muon)
 *   2. Frobenius normalisation:   X0 = bf16(M / (||M||_F + eps))
 *        (airosetta.com, newtonschulz5; "AdamW vs Muon", adg.csdn.net,
 *         section "1. Preprocessing")
 *   3. short side: when rows > cols the iteration works on the transpose
 *        (airosetta.com, newtonschulz5).  Done by logical layout, never by a
 *        copy.
 *   4. ns_steps Newton-Schulz iterations, step k with (a_k, b_k, c_k):
 *        A = X X^T ; B = b_k A + c_k A A ; X <- a_k X + B X
 *        (airosetta.com newtonschulz5 loop; adg.csdn.net section
 *         "2. Newton-Schulz iteration"; the hybrid schedule of section
 *         "3. DeepSeek-V4 hybrid schedule" is a per-step coefficient list)
 *      X and A are held in bf16 (the pages cast to bf16); every product is
 *      accumulated in fp32 and rounded to bf16 once, to nearest-even.  The
 *      a_k X term is folded into the stored matrix, C = a_k I + b_k A +
 *      c_k A A, so X <- C X; C is rounded to bf16 once, and for matrices
 *      whose short side is <= 128 it is kept as a bf16 pair (C_hi + C_lo,
 *      two MFMA passes) to stay well inside the bf16 error budget.
 *   5. decayed, scaled update:    p <- p*(1 - lr*wd) - lr*s*O
 *        (wmrh.cn section 4.2; adg.csdn.net section "3. Scaling and update")
 *      s = 1, or sqrt(max(1, rows/cols)) under MUON_SCALE_SQRT_MAX1 (the
 *      csdn page asks for an RMS rescale by matrix size without a formula;
 *      this is the reading taken), or the per-matrix `scale` when > 0.
 *
 * Error behaviour: every function returns MUON_OK (0) or a negative status.
 * Argument errors are found on the host before anything is launched; nothing
 * is modified then.  Kernel faults are asynchronous and surface at the
 * caller's next synchronisation.  muon_status_string() describes a status;
 * after MUON_EHIP it includes the HIP error text of the calling thread's last
 * failure, after MUON_ENONFINITE the matrix that failed the check.
 *
 * Device: a call works on the calling thread's current HIP device.  Its
 * stream must belong to that device (else MUON_EINVAL, before anything is
 * launched), and so must every buffer it is given (not checkable here: a
 * pointer into another device's memory is the caller's error).
 *
 * Thread safety: calls may come from several host threads; two calls that
 * run concurrently must use different workspaces.
 *
 * Debugging: with MUON_DEBUG set in the environment (any value but "0"),
 * every call keeps all its launches on the caller's stream, synchronises and
 * checks for an error after each launch (MUON_EHIP names the phase), and
 * fills the workspace's iteration buffers with bf16 NaN before a step, so a
 * kernel that read a value no kernel of the step wrote would leave NaN in the
 * result.  The variable is read at every call.  Not for production: it
 * serialises the host with the device.
 *
 * Non-finite check: with MUON_CHECK_FINITE set in the environment (any value
 * but "0"), muon_step, muon_step_ex and an eager muon_plan_step wait for the
 * stream at the end of the step and read back the squared Frobenius norms of
 * the new momenta that the momentum pass already computed (one double per
 * matrix, in the workspace; the gradient's own under MUON_OPT_NS_FIRST).
 * When one is NaN or infinite (a NaN or infinite gradient or momentum entry,
 * or a sum of squares beyond the fp32 range) the call returns MUON_ENONFINITE
 * and muon_status_string() names the first such matrix (its index in the
 * call's list).  Detection only: the step has run, and that matrix's
 * parameter and momentum hold the non-finite values the arithmetic gave
 * ("Muon meets Mamba", section 6.1, lists NaN among the troubles to watch
 * for).  Ignored by muon_step_noalloc, and by a muon_plan_step on a
 * capturing stream (neither may wait or read back).
 *
 * Graph capture: every call stages its descriptor table through a small ring
 * of pinned host buffers that later calls reuse, so a captured copy would
 * replay stale tables.  A call on a stream that is capturing returns
 * MUON_ECAPTURE before anything is launched; muon_plan_step (below) is the
 * capturable form of a step.
 */
#ifndef LIBMUON_MUON_H
#define LIBMUON_MUON_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define MUON_OK          0
#define MUON_EINVAL     -1   /* bad argument (shape, pointer, count, value)   */
#define MUON_EWORKSPACE -2   /* workspace missing, too small or misaligned    */
#define MUON_EHIP       -3   /* a HIP runtime call or kernel launch failed    */
#define MUON_EALIAS     -4   /* param / grad / momentum ranges overlap        */
#define MUON_ECAPTURE   -5   /* the stream is capturing a graph (see below)    */
#define MUON_ENONFINITE -6   /* MUON_CHECK_FINITE: a momentum norm is NaN/inf  */

/* ---- element types ----------------------------------------------------- */
#define MUON_F32  0
#define MUON_BF16 1

/* ---- RMS scale modes (call level) -------------------------------------- */
#define MUON_SCALE_NONE        0   /* s = 1                                  */
#define MUON_SCALE_SQRT_MAX1   1   /* s = sqrt(max(1, rows / cols))          */

/* One matrix of a muon_step call.
 *   param     fp32, rows x cols, row-major, contiguous; updated in place.
 *   grad      rows x cols, row-major, contiguous, element type grad_dtype
 *             (MUON_F32 or MUON_BF16).  NULL: the matrix is skipped entirely
 *             (no momentum update, no decay), as the pages' optimizer skips
 *             parameters without a gradient.
 *   momentum  fp32, rows x cols, row-major, contiguous; updated in place.
 *             The caller zero-initialises it before the first step.
 *   rows, cols  >= 1 and <= MUON_MAX_DIM.  Only 2-D matrices are accepted;
 *             routing 1-D parameters, embeddings and heads elsewhere is the
 *             caller's job.
 *   scale     per-matrix update scale s when > 0; otherwise the call's
 *             rms_scale_mode decides.
 * param, grad and momentum must be 4-byte aligned (16-byte alignment and
 * cols % 8 == 0 select the vectorised path) and must not overlap each other
 * or any other matrix's param / momentum. */
typedef struct {
  float*       param;
  const void*  grad;
  float*       momentum;
  int64_t      rows;
  int64_t      cols;
  int32_t      grad_dtype;
  float        scale;
} muon_matrix_t;

/* Coefficients of one Newton-Schulz iteration X <- a X + (b A + c A^2) X. */
typedef struct { float a, b, c; } muon_ns_coeff_t;

#define MUON_MAX_DIM      (1 << 20)
#define MUON_MAX_NS_STEPS 64

/* Bytes of device workspace a muon_step (or muon_orthogonalize) call over
 * these shapes needs.  Depends only on the shapes (grad == NULL entries are
 * counted too, so one workspace serves every call over the same list).
 * Returns 0 when the list is invalid or empty. */
size_t muon_workspace_bytes(const muon_matrix_t* mats, int64_t n_mats);

/* One Muon step over a list of matrices, as grouped launches: one launch per
 * phase covers every matrix, whatever their number and shapes.  Matrices
 * whose whole iteration fits one workgroup's LDS (short side <= 128 and, with
 * both sides padded to 32, m x n + 2 m x m bf16 within 160 KB) run every
 * Newton-Schulz step in one fused launch; the others take three launches per
 * step (Gram, C, X update) by tile class.  In all at most 4 + 3 * ns_steps
 * launches (one more with zero-centering).
 *   lr, mu, wd   learning rate, momentum, decoupled weight decay (finite).
 *   ns_steps     0 .. MUON_MAX_NS_STEPS Newton-Schulz iterations.
 *   coeffs       n_coeffs triples: 1 (used for every step) or ns_steps (one
 *                per step).  May be NULL only when ns_steps == 0.
 *   rms_scale_mode  MUON_SCALE_NONE or MUON_SCALE_SQRT_MAX1.
 *   eps          >= 0, added to ||M||_F before dividing.
 *   workspace    device memory of at least muon_workspace_bytes(mats,
 *                n_mats) bytes, 256-byte aligned.  Its contents on entry do
 *                not matter; on return (once the stream reaches that point)
 *                it holds every intermediate, see muon_workspace_view().
 *   stream       HIP stream all work is queued on (0: the null stream).
 * The matrix list itself is read during the call only. */
int muon_step(const muon_matrix_t* mats, int64_t n_mats,
              float lr, float mu, float wd, int ns_steps,
              const muon_ns_coeff_t* coeffs, int n_coeffs,
              int rms_scale_mode, float eps,
              void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Step variants, as flags of muon_options_t (any combination except
 * NESTEROV | NS_FIRST).
 *   MUON_OPT_ZERO_CENTER  G <- G minus its column means (the mean over rows of
 *       each column of the stored rows x cols gradient), before anything else
 *       uses G ("Muon meets Mamba", wmrh.cn, section 2.1 zerocenter, applied by
 *       _step_muon in section 4.2).  Costs one extra read of G (a column-sum
 *       pass with fp64 accumulation) and sizeof(double) * cols of workspace,
 *       which muon_workspace_bytes() always reserves.
 *   MUON_OPT_NESTEROV     the iteration runs on mu*M_new + (1-mu)*G instead
 *       of M_new.  The pages carry a nesterov switch but never say what it
 *       computes (airosetta.com, Muon constructor; wmrh.cn section 4.1); this
 *       look-ahead form is the reading taken.  M itself is still the EMA.
 *   MUON_OPT_NS_FIRST     the other order that wmrh.cn section 4.2 discusses:
 *       O = NS(G / (||G||_F + eps)), then M <- mu*M + (1-mu)*O and
 *       p <- p*(1 - lr*wd) - lr*s*M.  The norm slot of the workspace then
 *       holds ||G||_F^2. */
#define MUON_OPT_ZERO_CENTER 1u
#define MUON_OPT_NESTEROV    2u
#define MUON_OPT_NS_FIRST    4u
typedef struct {
  uint32_t flags;     /* MUON_OPT_* */
  uint32_t reserved;  /* must be 0 */
} muon_options_t;

/* muon_step with step variants.  options == NULL (or flags == 0) is exactly
 * muon_step.  Unknown flags, reserved != 0 or NESTEROV together with
 * NS_FIRST give MUON_EINVAL before anything is launched; everything else is
 * as muon_step. */
int muon_step_ex(const muon_matrix_t* mats, int64_t n_mats,
                 float lr, float mu, float wd, int ns_steps,
                 const muon_ns_coeff_t* coeffs, int n_coeffs,
                 int rms_scale_mode, float eps, const muon_options_t* options,
                 void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ---- a step that allocates nothing ---------------------------------------
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): the same
 * step as muon_step, with the workspace replaced by a fixed scratch array of
 * MUON_NOALLOC_SCRATCH_BYTES that the library holds on each device it runs
 * on, for the life of the process.  The caller still passes every parameter,
 * gradient and momentum buffer.  The call allocates no device or pinned host
 * memory and creates no stream or event: the descriptor table reaches the
 * device in kernel arguments, and every launch stays on `stream` (no side
 * stream; phase timing and MUON_DEBUG do not apply).
 *   Arguments and errors as muon_step, plus MUON_EWORKSPACE when
 *   muon_workspace_bytes(mats, n_mats) exceeds MUON_NOALLOC_SCRATCH_BYTES
 *   (found before anything is launched; nothing is modified then).
 * Every call on one device shares that device's array, which keeps the last
 * call's contents (each call rewrites what it reads before reading it): two
 * calls whose work overlaps on one device race, so order them on one stream
 * or with events.  The intermediates of the last call are readable through
 * muon_noalloc_scratch() at the offsets muon_workspace_view() gives. */
#define MUON_NOALLOC_SCRATCH_BYTES (64u << 20)
int muon_step_noalloc(const muon_matrix_t* mats, int64_t n_mats, float lr, float mu, float wd,
                      int ns_steps, const muon_ns_coeff_t* coeffs, int n_coeffs,
                      int rms_scale_mode, float eps, hipStream_t stream);
/* Device address of the current device's scratch array (for reading the last
 * muon_step_noalloc call's intermediates); NULL if it cannot be resolved. */
void* muon_noalloc_scratch(void);

/* ---- a step prepared once over fixed buffers ----------------------------
 * The pages' optimizer steps the same parameters every iteration (the
 * Muon.step loop of airosetta.com; _step_muon of wmrh.cn section 4.2).  A plan
 * fixes that list once: validation, the workspace plan and the descriptor
 * table (with the coefficients) happen in muon_plan_create, which uploads the
 * table into the workspace and waits for that copy.  muon_plan_step then only
 * launches kernels: no host staging, no allocation, no synchronisation, so it
 * may be captured into a HIP graph and replayed.
 *   muon_plan_create  arguments as muon_step_ex (same errors, found before
 *       anything is launched; MUON_EHIP also when the host object cannot be
 *       allocated); *plan receives a host object the caller frees
 *       with muon_plan_destroy.  The param, grad and momentum pointers and the
 *       workspace are recorded: they must stay valid, and the workspace must
 *       not be used by other calls, while the plan lives.  New gradients are
 *       written into the same grad buffers.
 *   muon_plan_step    one step of the plan on `stream`, on the device the plan
 *       was created on (else MUON_EINVAL).  `hyper` points to three floats in
 *       device memory, {lr, mu, wd}, read by the kernels when they run, so a
 *       schedule updates them between replays.
 * Each step clears the workspace's norm slots with a fill kernel (no
 * memset), so replays do not depend on the previous step's workspace.  Phase
 * timing (muon_timing_enable) is skipped while the stream is capturing.  A
 * plan over both fused and tiled matrices owns a stream and two events
 * (created here, released by muon_plan_destroy, which first waits for the
 * work its steps queued there); a captured step forks onto that stream and
 * joins back, so the graph holds two parallel branches. */
typedef struct muon_plan muon_plan_t;
int muon_plan_create(const muon_matrix_t* mats, int64_t n_mats, int ns_steps,
                     const muon_ns_coeff_t* coeffs, int n_coeffs, int rms_scale_mode, float eps,
                     const muon_options_t* options, void* workspace, size_t workspace_bytes,
                     hipStream_t stream, muon_plan_t** plan);
int muon_plan_step(const muon_plan_t* plan, const float* hyper, hipStream_t stream);
void muon_plan_destroy(muon_plan_t* plan);

/* Orthogonalisation alone: out = NS(in) with the same normalisation,
 * short-side rule and bf16 iteration as muon_step, for a list of matrices.
 * The Newton-Schulz routine of the airosetta.com article (newtonschulz5) as a
 * standalone call.
 *   in       rows x cols, row-major, contiguous, type in_dtype (MUON_F32 or
 *            MUON_BF16); read only.
 *   out      bf16 (raw 16-bit patterns), rows x cols, row-major, contiguous;
 *            written.  Must not overlap `in`.
 * The workspace is sized by muon_workspace_bytes() over the same shapes
 * (build the muon_matrix_t list with any grad pointer). */
typedef struct {
  const void*  in;
  void*        out;
  int64_t      rows;
  int64_t      cols;
  int32_t      in_dtype;
} muon_ortho_t;

int muon_orthogonalize(const muon_ortho_t* mats, int64_t n_mats, int ns_steps,
                       const muon_ns_coeff_t* coeffs, int n_coeffs, float eps,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Where matrix `index`'s intermediates live in the workspace after a call
 * over the same shapes (byte offsets from the workspace base).  Each bf16
 * buffer is zero-padded: X buffers are rows_pad x cols_pad in the stored
 * (rows x cols) orientation, A and C are m_pad x m_pad with m the short side.
 *   x_off[0]  X0 and every even iterate; x_off[1] the odd iterates.
 *   a_off     A = X X^T of the last iteration.
 *   c_off     C = a I + b A + c A A of the last iteration (bf16 high part).
 *   c_lo_off  its low part C - bf16(C) (short side <= 128), else 0.
 *   o_off     the final iterate O for `ns_steps` iterations.
 *   nrm2_off  one double: sum of squares of M (of `in` for orthogonalize).
 * Host-only; launches nothing.  For tests and diagnostics. */
typedef struct {
  size_t  x_off[2];
  size_t  a_off;
  size_t  c_off;
  size_t  c_lo_off;
  size_t  o_off;
  size_t  nrm2_off;
  int64_t rows_pad;
  int64_t cols_pad;
  int64_t m_pad;
  int32_t transposed;   /* 1 when rows > cols: the iteration runs on X^T */
  int32_t tile;         /* padding granule: 256 or 128 (tiled kernels) or
                           32 (the fused small-matrix iteration)           */
} muon_workspace_view_t;

int muon_workspace_view(const muon_matrix_t* mats, int64_t n_mats, int64_t index,
                        int ns_steps, muon_workspace_view_t* view);

/* ------------------------------------------------------------------------
 * AdamW branch: the update the pages pair with Muon for the parameters Muon
 * does not take (1-D biases and norm weights, embeddings, output heads).
 * "Muon meets Mamba" (wmrh.cn), section 4.2, method _step_adamw; defaults in
 * section 4.1 (lr 1e-3, betas (0.9, 0.95), eps 1e-8, weight decay 0.01 shared
 * with the Muon group).  Per tensor with a gradient, elementwise in fp32:
 *
 *   p <- p (1 - lr wd)
 *   m <- beta1 m + (1 - beta1) g,        v <- beta2 v + (1 - beta2) g^2
 *   p <- p - (lr / (1 - beta1^t)) m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 *
 * with t the tensor's own step count (the page keeps one per parameter).
 * ------------------------------------------------------------------------ */
typedef struct {
  float*      param;       /* fp32 [numel], updated in place                        */
  const void* grad;        /* [numel] of grad_dtype; NULL: the tensor is skipped     */
                           /* (no decay, no moment update)                           */
  float*      exp_avg;     /* fp32 [numel] first moment m, in place; caller zero-inits */
  float*      exp_avg_sq;  /* fp32 [numel] second moment v, in place; caller zero-inits */
  int64_t     numel;       /* >= 1 elements (any tensor shape, flattened)            */
  int64_t     step;        /* t of this update, >= 1: the caller keeps the per-tensor */
                           /* count and increments it before the call                */
  int32_t     grad_dtype;  /* MUON_F32 or MUON_BF16                                  */
  int32_t     reserved;    /* must be 0                                              */
} muon_adamw_tensor_t;

/* Workspace for n_tensors tensors (descriptor table); 0 if n_tensors <= 0. */
size_t muon_adamw_workspace_bytes(int64_t n_tensors);

/* One AdamW update of every tensor with a gradient, one grouped launch on
 * `stream`.  Arguments: 0 <= beta1, beta2 < 1, eps >= 0, lr and wd finite.
 * Same ownership, aliasing and error rules as muon_step: MUON_EINVAL for a
 * bad argument (numel < 1, step < 1, unknown dtype, missing buffer, reserved
 * != 0), MUON_EALIAS when any two buffers of the call overlap,
 * MUON_EWORKSPACE for a missing, small or unaligned workspace, all found
 * before anything is launched; MUON_EHIP when a launch fails. */
int muon_adamw_step(const muon_adamw_tensor_t* tensors, int64_t n_tensors, float lr, float beta1,
                    float beta2, float eps, float wd, void* workspace, size_t workspace_bytes,
                    hipStream_t stream);

/* ------------------------------------------------------------------------
 * Training operators beside the optimizer step: what makes the gradients
 * that muon_step and muon_adamw_step take, from activations kept in 8 bits.
 *
 *   muon_rmsnorm_act8 / _grad   RMS norm with the residual's addition; keeps
 *                               the normalised rows in 8 bits
 *   muon_swiglu_act8 / _grad    gated unit silu(gate) * up; keeps both in 8 bits
 *   muon_act8_pack / _unpack    the 8-bit form of any matrix, and back
 *   muon_act8_wgrad             weight gradient dY^T X from an 8-bit X
 *   muon_embed / _grad          embedding lookup and its gradient
 *   muon_attention / _grad      attention over sequences of any lengths
 *   muon_distill, muon_policy   losses with the gradient of the logits
 *
 * Matrices are row-major with unit column stride; each has its own row
 * stride ("ld", in elements, >= the row's length; not read where there is one
 * row).  Rows may start anywhere (aligned to their element).  rows and tokens
 * are 0 .. 2^31 - 1 (0: nothing is written, except that gradients summed over
 * rows are zero then), cols 1 .. MUON_MAX_DIM.
 *
 * These calls stage nothing through host memory: their arguments travel with
 * the launches.  They may be captured into a graph, and the structs are read
 * during the call only.  Outputs must not overlap each other or an input
 * (MUON_EALIAS; column slices of one buffer with one row stride do not).
 * Sums run in fp32 in an order fixed by the sizes, the strides and alignments
 * (which decide how the weight gradient is cut) and, in the embedding's
 * gradient, the ids: the same call on the same values gives the same bits.  Errors, the stream's device
 * and MUON_DEBUG are as for muon_step (under MUON_DEBUG a workspace is filled
 * with NaN first; on a capturing stream the variable is ignored).  Phase
 * timing does not record them.
 * ------------------------------------------------------------------------ */

/* A matrix in 8 bits.  Each group of 32 consecutive columns of a row (the
 * last one may be shorter) shares a power of two s = 2^e, the smallest with
 * max |v| <= 448 s and -117 <= e <= 119; each value is v / s rounded to the
 * nearest 8-bit float of 4 exponent and 3 mantissa bits (finite, largest 448;
 * ties to even; 0x7F and 0xFF are NaN).  |v - value| <= max(2^-4 |v|, 2^-10 s),
 * and the value is exact in bf16.  Infinities and NaN become NaN and do not
 * count in the maximum, so they leave the rest of their group as it is;
 * finite values beyond 448 * 2^119 saturate.
 *   codes   rows x ld_codes bytes
 *   scales  rows x ld_scales bytes, e + 127 of each group (10 .. 246; the
 *           calls that read them take any byte, b as 2^(b - 127), but their
 *           results are defined for 10 .. 246 only) */
#define MUON_ACT8_GROUP 32
typedef struct {
  uint8_t* codes;
  uint8_t* scales;
  int64_t  ld_codes;    /* >= cols */
  int64_t  ld_scales;   /* >= (cols + 31) / 32 */
} muon_act8_t;

/* x (fp32 or bf16) -> its 8-bit form; and the values it stands for. */
int muon_act8_pack(const void* x, int64_t ld_x, int32_t dtype, int64_t rows, int64_t cols,
                   const muon_act8_t* out, hipStream_t stream);
int muon_act8_unpack(const muon_act8_t* in, int64_t rows, int64_t cols, void* out, int64_t ld_out,
                     int32_t dtype, hipStream_t stream);

/* RMS norm of h = x + residual, row by row, in fp32 from the unrounded sum:
 *   rstd = 1 / sqrt(mean(h^2) + eps),  n = h rstd,  y = n gain.
 * cols <= MUON_NORM_MAX_COLS (a row stays in one workgroup's registers).
 *   x, residual  dtype; residual may be NULL (h = x)
 *   gain         fp32 [cols], NULL: 1
 *   h, y         dtype, each rounded once; either may be NULL
 *   n            8-bit form of n (before the gain); codes NULL: not kept
 *   rstd         fp32 [rows]; may be NULL
 * n and rstd are all that the backward pass needs: x, residual and h may go. */
#define MUON_NORM_MAX_COLS 16384
typedef struct {
  const void*  x;
  const void*  residual;
  const float* gain;
  void*        h;
  void*        y;
  muon_act8_t  n;
  float*       rstd;
  int64_t      rows, cols;
  int64_t      ld_x, ld_residual, ld_h, ld_y;
  float        eps;       /* >= 0 */
  int32_t      dtype;     /* MUON_F32 or MUON_BF16: x, residual, h, y */
} muon_rmsnorm_t;
int muon_rmsnorm_act8(const muon_rmsnorm_t* op, hipStream_t stream);

/* Backward pass of the norm, with n read from its 8-bit form:
 *   dx    = rstd (gain dy - n mean(gain dy n)) + dres
 *   dgain = sum over rows of dy n
 * dx is the gradient of x and of residual alike (h is their sum).
 *   dy, dres  dtype; dres (the gradient that reaches h on its own path, the
 *             residual stream's) may be NULL
 *   dx        dtype;  dgain  fp32 [cols], may be NULL
 *   workspace muon_rmsnorm_act8_grad_workspace_bytes(rows, cols), 256-byte
 *             aligned; not needed where dgain is NULL */
typedef struct {
  const void*  dy;
  const void*  dres;
  const float* gain;
  const float* rstd;
  muon_act8_t  n;
  void*        dx;
  float*       dgain;
  int64_t      rows, cols;
  int64_t      ld_dy, ld_dres, ld_dx;
  int32_t      dtype;
  int32_t      reserved;  /* must be 0 */
} muon_rmsnorm_grad_t;
size_t muon_rmsnorm_act8_grad_workspace_bytes(int64_t rows, int64_t cols);
int muon_rmsnorm_act8_grad(const muon_rmsnorm_grad_t* op, void* workspace, size_t workspace_bytes,
                           hipStream_t stream);

/* Gated unit: a = silu(gate) up = gate / (1 + exp(-gate)) up, in fp32.
 *   gate, up       dtype
 *   a              dtype; may be NULL
 *   gate8, up8     8-bit forms of gate and up, for the backward pass; codes
 *                  NULL (both): not kept */
typedef struct {
  const void* gate;
  const void* up;
  void*       a;
  muon_act8_t gate8, up8;
  int64_t     rows, cols;
  int64_t     ld_gate, ld_up, ld_a;
  int32_t     dtype;
  int32_t     reserved;   /* must be 0 */
} muon_swiglu_t;
int muon_swiglu_act8(const muon_swiglu_t* op, hipStream_t stream);

/* Its backward pass from the 8-bit gate and up, with s = 1 / (1 + exp(-gate)):
 *   dgate = da up s (1 + gate (1 - s)),   dup = da gate s
 *   a8    8-bit form of a = gate s up, recomputed: the activation that the next
 *         product's weight gradient needs (codes NULL: not made)
 * da, dgate, dup: dtype. */
typedef struct {
  const void* da;
  muon_act8_t gate8, up8;
  void*       dgate;
  void*       dup;
  muon_act8_t a8;
  int64_t     rows, cols;
  int64_t     ld_da, ld_dgate, ld_dup;
  int32_t     dtype;
  int32_t     reserved;   /* must be 0 */
} muon_swiglu_grad_t;
int muon_swiglu_act8_grad(const muon_swiglu_grad_t* op, hipStream_t stream);

/* Weight gradient of y = x W^T (W: n x k, as muon_step holds it) from the
 * 8-bit form of x:
 *   dw[i][j] (+)= col_gain[j] sum_t dy[t][i] x[t][j]
 * Products of bf16 with the exact values of x8, summed in fp32; the total is
 * rounded once to dw's type.
 *   dy        bf16, tokens x n
 *   x8        tokens x k
 *   col_gain  fp32 [k], NULL: 1.  With x8 the norm's n this folds the norm's
 *             gain in: x = n gain
 *   dw        n x k, dw_dtype (MUON_F32 or MUON_BF16), 1 <= n, k; accumulate
 *             != 0 adds to what it holds, else it is overwritten
 *   workspace muon_act8_wgrad_workspace_bytes(op) bytes, 256-byte aligned
 *             (may be 0, and NULL then).  Depends on the sizes, strides and
 *             alignments. */
typedef struct {
  const void*  dy;
  muon_act8_t  x8;
  const float* col_gain;
  void*        dw;
  int64_t      tokens, n, k;
  int64_t      ld_dy, ld_dw;
  int32_t      dw_dtype;
  int32_t      accumulate;
} muon_act8_wgrad_t;
size_t muon_act8_wgrad_workspace_bytes(const muon_act8_wgrad_t* op);
int muon_act8_wgrad(const muon_act8_wgrad_t* op, void* workspace, size_t workspace_bytes,
                    hipStream_t stream);

/* Embedding lookup: out[t] = scale * table[ids[t]], the product in fp32,
 * rounded to out_dtype.  A token whose id is outside 0 .. vocab - 1 (-1 for padding, say)
 * gets a row of zeros, and no gradient below.
 *   table  vocab x cols, table_dtype;  ids  int32 or int64 (id_bytes 4 or 8)
 *   out    tokens x cols, out_dtype */
typedef struct {
  const void* table;
  const void* ids;
  void*       out;
  int64_t     tokens, vocab, cols;   /* vocab 1 .. 2^31 - 2 */
  int64_t     ld_table, ld_out;
  float       scale;                 /* finite */
  int32_t     table_dtype, out_dtype;
  int32_t     id_bytes;
} muon_embed_t;
int muon_embed(const muon_embed_t* op, hipStream_t stream);

/* Its gradient, from the tokens sorted by id:
 *   dtable[v] (+)= scale * sum over t with ids[t] == v of dy[t]
 * every row is written (zeros where no token has its id), except that with
 * accumulate only the rows that have tokens are read and written.
 *   dy        tokens x cols, dy_dtype;  dtable  vocab x cols, table_dtype
 *   workspace muon_embed_grad_workspace_bytes(tokens, vocab, cols) bytes,
 *             256-byte aligned */
typedef struct {
  const void* dy;
  const void* ids;
  void*       dtable;
  int64_t     tokens, vocab, cols;
  int64_t     ld_dy, ld_dtable;
  float       scale;
  int32_t     dy_dtype, table_dtype;
  int32_t     id_bytes;
  int32_t     accumulate;
  int32_t     reserved;              /* must be 0 */
} muon_embed_grad_t;
size_t muon_embed_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t cols);
int muon_embed_grad(const muon_embed_grad_t* op, void* workspace, size_t workspace_bytes,
                    hipStream_t stream);

/* A bf16 tensor of tokens x heads x dim: element (t, h, d) at
 * data[t ld_token + h ld_head + d], strides in elements.  Heads and tokens must not
 * overlap; the stride of an axis of length one is not read.  Slices of a fused
 * projection and heads-first tensors are such. */
typedef struct {
  void*   data;
  int64_t ld_token, ld_head;
} muon_heads_t;

/* Attention.  Query head h goes with key and value head h / (heads / kv_heads);
 * query i of a sequence of nq queries and nk keys sees all its keys, or, if
 * `causal`, keys j <= i + nk - nq:
 *   S = scale q k^T,   lse = log sum_j exp S_ij,   o = sum_j exp(S_ij - lse) v_j.
 * A query that sees no key gets zeros, lse -infinity, and no gradient.
 *   starts    int32 [sequences + 1] in device memory: sequence s has the tokens
 *             starts[s] .. starts[s+1] - 1 of q and o.  NULL: one sequence of all
 *             tokens (sequences is then not read).  Not decreasing, from 0 to at
 *             most `tokens`; what they hold is not checked, other values give
 *             undefined results, but no access outside the tensors.
 *   k_starts  the same of k and v; NULL: as starts (k_tokens == tokens then), not
 *             NULL without starts
 *   lse       fp32, heads x ld_lse >= tokens; may be NULL
 *   zero_rest what to do with tokens behind the last sequence: 0 leaves them as they
 *             are; MUON_ATTN_ZERO_O, _LSE write zeros (-infinity to lse)
 * dim is a multiple of 8 up to 128; tokens, k_tokens 0 .. 2^30; with t the larger
 * of them (t / 128 + sequences + 2) heads <= 2^22.  Products of bf16 summed in fp32,
 * softmax in fp32; the probabilities are rounded to bf16 for the second product,
 * outputs once.  Few, long rows are cut into parts that a second launch joins.
 *   workspace muon_attention_workspace_bytes(op) bytes, 256-byte aligned (may be 0, and
 *             NULL then); depends on the sizes
 * A value that is not finite may reach every row of its sequence and
 * head, masked or not, but no other sequence. */
#define MUON_ATTN_MAX_DIM 128
#define MUON_ATTN_ZERO_O 1
#define MUON_ATTN_ZERO_LSE 2
typedef struct {
  muon_heads_t   q, k, v, o;
  float*         lse;
  const int32_t* starts;
  const int32_t* k_starts;
  int64_t        tokens, k_tokens, sequences;
  int64_t        heads, kv_heads, dim;
  int64_t        ld_lse;
  float          scale;      /* > 0, at most 1e30 */
  int32_t        causal;     /* 0 or 1 */
  int32_t        zero_rest;
  int32_t        reserved;   /* must be 0 */
} muon_attention_t;
size_t muon_attention_workspace_bytes(const muon_attention_t* op);
int muon_attention(const muon_attention_t* op, void* workspace, size_t workspace_bytes,
                   hipStream_t stream);

/* Its backward pass; P is recomputed from lse:
 *   P = exp(S - lse),  dS = P (dout v^T - rowsum(dout o)),
 *   dq = scale dS k,   dk = scale dS^T q,   dv = P^T dout,
 * dk and dv summed over the heads that share them.  P and dS are rounded to bf16 for
 * the products.  No atomics: the same bits every time.
 *   o, lse     as the forward pass left them
 *   zero_rest  MUON_ATTN_ZERO_DQ, _DK, _DV: as above
 *   workspace  muon_attention_grad_workspace_bytes(op) bytes, 256-byte aligned */
#define MUON_ATTN_ZERO_DQ 1
#define MUON_ATTN_ZERO_DK 2
#define MUON_ATTN_ZERO_DV 4
typedef struct {
  muon_heads_t   dout, q, k, v, o;
  muon_heads_t   dq, dk, dv;
  const float*   lse;
  const int32_t* starts;
  const int32_t* k_starts;
  int64_t        tokens, k_tokens, sequences;
  int64_t        heads, kv_heads, dim;
  int64_t        ld_lse;
  float          scale;
  int32_t        causal;
  int32_t        zero_rest;
  int32_t        reserved;   /* must be 0 */
} muon_attention_grad_t;
size_t muon_attention_grad_workspace_bytes(const muon_attention_grad_t* op);
int muon_attention_grad(const muon_attention_grad_t* op, void* workspace, size_t workspace_bytes,
                        hipStream_t stream);

/* Distillation from a teacher's top logits, row by row, x = logits / temperature:
 *   p    = softmax over the row's entries of teacher / temperature
 *   loss = weight temperature^2 sum_k p_k (log p_k - log softmax(x)[ids_k])
 *   dlogits = d loss / d logits = weight temperature (softmax(x) - sum of p at the ids)
 * An entry whose id is outside 0 .. vocab - 1, or whose teacher logit is -infinity, is
 * not there; entries of the same id add up.  A row of weight 0 or without entries
 * has loss 0 and a gradient of zeros, whatever its logits hold.
 *   logits   dtype, tokens x vocab (vocab <= MUON_MAX_DIM)
 *   ids      int32 or int64 (id_bytes 4 or 8), tokens x top
 *   teacher  teacher_dtype, tokens x top
 *   weights  fp32 [tokens], NULL: 1
 *   loss     fp32 [tokens];  dlogits  dtype, tokens x vocab, NULL: not wanted */
#define MUON_DISTILL_MAX_TOP 1024
typedef struct {
  const void*  logits;
  const void*  ids;
  const void*  teacher;
  const float* weights;
  float*       loss;
  void*        dlogits;
  int64_t      tokens, vocab, top;   /* top 1 .. MUON_DISTILL_MAX_TOP */
  int64_t      ld_logits, ld_ids, ld_teacher, ld_dlogits;
  float        temperature;          /* 1e-6 .. 1e6 */
  int32_t      dtype, teacher_dtype, id_bytes;
} muon_distill_t;
int muon_distill(const muon_distill_t* op, hipStream_t stream);

/* Clipped policy loss with a KL term, token by token, x = logits / temperature:
 *   logp = log softmax(x)[action],   r = exp(logp - old_logp),   d = ref_logp - logp
 *   loss = weight (-min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A) + kl_coef (exp(d) - d - 1))
 *   g    = d loss / d logp = weight (-A r [r A <= clamp(r) A] + kl_coef (1 - exp(d)))
 *   dlogits = g / temperature (onehot(action) - softmax(x))
 * with A the advantage.  A token of weight 0, or whose action is outside 0 .. vocab - 1,
 * has loss and logp 0 and a gradient of zeros, whatever its logits hold.
 *   logits      dtype, tokens x vocab;  actions  int32 or int64 [tokens]
 *   old_logp, advantages, ref_logp, weights  fp32 [tokens]; no KL term where ref_logp
 *               is NULL or kl_coef 0; weights NULL: 1
 *   loss, logp  fp32 [tokens]; logp may be NULL
 *   dlogits     dtype, NULL: not wanted */
typedef struct {
  const void*  logits;
  const void*  actions;
  const float* old_logp;
  const float* advantages;
  const float* ref_logp;
  const float* weights;
  float*       loss;
  float*       logp;
  void*        dlogits;
  int64_t      tokens, vocab;
  int64_t      ld_logits, ld_dlogits;
  float        clip_low, clip_high;  /* 0 <= clip_low <= 1, clip_high >= 0 */
  float        kl_coef;              /* finite */
  float        temperature;          /* 1e-6 .. 1e6 */
  int32_t      dtype, id_bytes;
} muon_policy_t;
int muon_policy(const muon_policy_t* op, hipStream_t stream);

/* Phase timing with HIP events, for benchmarks.  When enabled, every launch
 * is bracketed by a pair of events on the call's stream, and a step keeps
 * all its launches on that stream (no side-stream overlap, so that each
 * phase's events bracket its own kernels only).  muon_timing_read()
 * waits for the recorded events, returns the summed milliseconds and launch
 * counts per phase (MUON_PHASES entries each; either pointer may be NULL) and
 * clears the record.  Phases: momentum+norm, normalise+cast, Gram X X^T,
 * Gram A A with the b A + c A^2 epilogue, X update, apply (or export),
 * AdamW, and the fused iteration of small matrices (every Newton-Schulz
 * step of each matrix whose whole iteration fits one workgroup's LDS). */
#define MUON_PHASES 8
int muon_timing_enable(int on);
int muon_timing_read(double* ms, int64_t* launches);

/* Static text for a status code (with HIP detail after MUON_EHIP). */
const char* muon_status_string(int status);

/* Library version, e.g. "libmuon 0.1 gfx950". */
const char* muon_version(void);

#ifdef __cplusplus
}
#endif
#endif /* LIBMUON_MUON_H */
