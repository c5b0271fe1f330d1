/*
 * muonh.h -- C ABI of the MI355X (gfx950) MuonH optimizer-step library.
 *
 * What the library computes, per wrapped 2-D fp32 matrix W (r x c), on the
 * caller's HIP stream:
 *
 *   1. momentum         M <- beta*M + G                (heavy-ball, in place)
 *   2. Muon update      u  = NS_5(Y), Y = M (or G + beta*M with Nesterov):
 *                       X_0 = Y / (||Y||_F + eps), then ns_steps times
 *                       A = X X^T, B = b A + c A A, X <- a X + B X
 *   3. Hyperball step   u^ = u/||u||_F, W~ = W - eta R u^, W <- R W~/||W~||_F
 *
 * Step 3 is Eq. (1) of "Puro-2B: Poor Lab's Qwen2-1.5B Trained on RTX 5090
 * within $5090" (arXiv HTML, §3.3), with the fixed radius R = ||W_0||_F of
 * the same section and the effective LR eta^H = m * eta_base of §3.3.1.
 * The pages name but do not define steps 1-2; the defaults below (beta 0.95,
 * five quintic iterations with (3.4445, -4.7750, 2.0315), eps 1e-7) are the
 * published Muon method's.  Two further modes reuse steps 1-2 with the other
 * updates of §3.3.1: ordinary Muon with decoupled weight decay (Eq. (3)) and
 * effective-LR-aligned Muon (Eq. (5)).
 *
 * Conventions for every entry point:
 *   - Return value: MUONH_OK (0) or a negative MUONH_E* code.  Nothing is
 *     thrown or aborted across the ABI.  muonh_last_error() gives the text of
 *     the last failure on the calling thread.
 *   - Device pointers are HIP device addresses; "stream" is a hipStream_t
 *     passed as void* (NULL = the default stream).
 *   - All matrices are row-major and contiguous (leading dimension = cols).
 *   - Work is enqueued asynchronously; errors from kernels surface at the
 *     next synchronising call (muonh_get_radii / muonh_get_stats).
 *   - A handle is not thread-safe; distinct handles are independent.
 *   - Environment, read at init: MUONH_DEBUG_SYNC=1 synchronises the stream
 *     after every kernel launch so a device fault is reported (MUONH_EHIP) by
 *     the step that caused it, naming the launch (slow; for debugging);
 *     MUONH_LOG=1 prints the plan (buckets, tile and chunk counts, workspace,
 *     FLOP per step) on stderr; MUONH_GEMM_TILE=64 or 256 forces the GEMM
 *     path (by default plans whose B'X product has fewer than 64 tiles of
 *     256 x 256 use 64 x 64 tiles over the unpadded dims; results agree to
 *     rounding, not bitwise).  Also read by muonh_workspace_size and
 *     muonh_plan_query.
 */
#ifndef MUONH_H_
#define MUONH_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define MUONH_OK         0
#define MUONH_EINVAL    -1   /* bad argument: null pointer, dims <= 0, dtype, alignment */
#define MUONH_EMISMATCH -2   /* step matrix list differs from the one given at init */
#define MUONH_ENOMEM    -3   /* workspace too small or device allocation failed */
#define MUONH_EHIP      -4   /* a HIP runtime call failed (see muonh_last_error) */
#define MUONH_ESTATE    -5   /* call out of order (e.g. copy_update before a step) */
#define MUONH_ENODEV    -6   /* no usable gfx950 device */

/* ---- enumerations ------------------------------------------------------ */
#define MUONH_F32   0        /* IEEE binary32 */
#define MUONH_BF16  1        /* bfloat16 (round-to-nearest-even when produced) */

#define MUONH_MODE_HYPERBALL   0  /* Eq. (1): normalised update + projection to radius R */
#define MUONH_MODE_MUON_WD     1  /* Eq. (3): W <- (1 - wd*eta) W - eta u */
#define MUONH_MODE_ELR_ALIGNED 2  /* Eq. (5): W <- W - eta_t u, eta_t = eta ||W|| / ||u|| */

/* One wrapped matrix.  The same list order, shapes and dtypes are used at
 * init and at every step; the pointers may change between steps.           */
typedef struct muonh_matrix_desc {
  void*       w;         /* fp32 [rows x cols], device, updated in place              */
  const void* g;         /* gradient [rows x cols], device, dtype g_dtype (read only) */
  void*       m;         /* fp32 momentum [rows x cols], device, updated in place     */
  int64_t     rows;      /* r >= 1                                                     */
  int64_t     cols;      /* c >= 1                                                     */
  int32_t     g_dtype;   /* MUONH_F32 or MUONH_BF16                                    */
  float       radius;    /* R; <= 0 means R = ||W||_F measured at init (resume: pass R) */
} muonh_matrix_desc;

typedef struct muonh_options {
  float   beta;          /* momentum coefficient, default 0.95                    */
  int32_t ns_steps;      /* Newton-Schulz iterations, 1..16, default 5             */
  float   ns_a, ns_b, ns_c; /* quintic coefficients, default 3.4445, -4.775, 2.0315 */
  float   ns_eps;        /* X_0 = Y / (||Y|| + eps), default 1e-7                  */
  int32_t ns_dtype;      /* operand type of the NS products: MUONH_BF16 (default) or MUONH_F32;
                            accumulation is always fp32                              */
  int32_t nesterov;      /* 0 (default): Y = M; 1: Y = G + beta*M                   */
  int32_t mode;          /* MUONH_MODE_*, default MUONH_MODE_HYPERBALL              */
  float   weight_decay;  /* lambda of MUONH_MODE_MUON_WD, default 0                  */
  int32_t symmetric;     /* 1 (default): X X^T and A A computed on upper tiles only */
  int32_t deterministic; /* 1 (default): every reduction runs in a fixed order (no
                            floating-point atomics), so repeated steps on the same
                            inputs are bitwise equal; 0 is accepted and behaves the
                            same (there is no faster non-deterministic path)        */
  void*   workspace;     /* optional caller-owned device memory; NULL: library allocates */
  size_t  workspace_bytes;
} muonh_options;

typedef struct muonh_step_args {
  float        elr;        /* eta: effective LR of this step (Hyperball: eta^H = m eta_base) */
  const float* elr_scale;  /* optional host array [n]: per-matrix factor on elr, or NULL     */
  int64_t      step;       /* caller's step counter (recorded, not used in the arithmetic)   */
  int32_t      want_stats; /* reserved: statistics are always produced on the device         */
} muonh_step_args;

/* Per-matrix diagnostics of the last step (cf. the per-group effective LR,
 * weight-norm and update-norm traces of App. D, Fig. 15).                  */
typedef struct muonh_stats {
  double y_norm;    /* ||Y||_F, the Newton-Schulz input                      */
  double u_norm;    /* ||u||_F, raw Newton-Schulz output                     */
  double w_norm;    /* ||W_t||_F before the step                             */
  double inner;     /* <W_t, u^>                                             */
  double c;         /* <W_t, u^> / R                                         */
  double wt_norm;   /* ||W~||_F (Hyperball) / ||W_{t+1}||_F (other modes)    */
  double elr;       /* effective LR: ||W_{t+1}^pre - W_t|| / ||W_t||          */
  double angle;     /* Hyperball: atan2(eta sqrt(1-c^2), 1 - eta c)          */
  int32_t nonfinite;/* 1 if any of the norms above is NaN or Inf             */
  int32_t reserved;
} muonh_stats;

/* Host-side plan summary (pure host computation, no device needed). */
typedef struct muonh_plan_info {
  int32_t n_matrices;
  int32_t n_buckets;        /* distinct padded NS shapes (m_pad x n_pad)            */
  int64_t gemm_tiles[3];    /* 256x256 output tiles per launch: XX^T, AA, BX          */
  int64_t mom_tiles;        /* blocks of the momentum / pack kernel: 64x64 tiles, or
                               1024-column row segments where X_0 is not transposed */
  int64_t flat_chunks;      /* chunks of the reduction and update kernels            */
  double  ns_dense_flops;   /* sum over matrices of steps*(4 m^2 n + 2 m^3)          */
  double  ns_exec_flops;    /* MFMA FLOP issued per step (padding + symmetric tiles) */
  double  elem_bytes;       /* algorithmic HBM bytes of the elementwise kernels/step */
  size_t  workspace_bytes;  /* bytes muonh_workspace_size would return              */
} muonh_plan_info;

typedef struct muonh_handle muonh_handle;

/* Fill *opt with the defaults listed above. */
void muonh_default_options(muonh_options* opt);

/* Bytes of device workspace a plan for these matrices needs (host only). */
int muonh_workspace_size(const muonh_matrix_desc* mats, int32_t n,
                         const muonh_options* opt, size_t* bytes);

/* Host-only plan summary for these matrices (no device work). */
int muonh_plan_query(const muonh_matrix_desc* mats, int32_t n,
                     const muonh_options* opt, muonh_plan_info* info);

/* Build the plan (shape buckets, tile tables, workspace layout) on the
 * current device and, for every matrix with radius <= 0, enqueue
 * R = ||W_0||_F on `stream`.  Keeps shapes and dtypes, not pointers.
 * The library owns only the plan and, when opt->workspace is NULL, its
 * workspace.  On failure *h is NULL.                                        */
int muonh_init(muonh_handle** h, const muonh_matrix_desc* mats, int32_t n,
               const muonh_options* opt, void* stream);

/* One optimizer step over all n matrices (same order / shapes / dtypes as
 * at init), enqueued on `stream`.  W and M are updated in place; G is read.
 * Buffers must stay valid until the stream has passed the step.            */
int muonh_step(muonh_handle* h, const muonh_matrix_desc* mats, int32_t n,
               const muonh_step_args* args, void* stream);

/* The same step as muonh_step (same arguments, same arithmetic: results are
 * bitwise equal), for callers whose steps are bound by launch overhead.  The
 * first call records the step's kernel launches into a HIP graph, on a
 * stream the handle owns; every call then enqueues on `stream` one small
 * kernel that stores this call's per-matrix step sizes
 * elr * elr_scale[i] (fp64) in the workspace, and one launch of the recorded
 * graph.  Pointer changes and elr / elr_scale are taken from each call as in
 * muonh_step; nothing needs recording again.  Returns MUONH_ESTATE when
 * per-phase timing is on or MUONH_DEBUG_SYNC is set (use muonh_step then).
 * Not for use while the caller is itself capturing `stream`.  The graph is
 * released by muonh_destroy.                                                */
int muonh_step_graph(muonh_handle* h, const muonh_matrix_desc* mats, int32_t n,
                     const muonh_step_args* args, void* stream);

/* Allocation-free variant of muonh_step, for callers that cannot allocate
 * device memory: code that must not call hipMalloc or hipFree (tight serving
 * or training loops, harnesses that forbid allocation).  One self-contained
 * step over n matrices with no handle: the plan is built on the host each
 * call, and every buffer the step needs beyond the caller's W, G and M
 * (tables, Newton-Schulz iterates, partial sums) lives in one static device
 * array of the library, MUONH_NOALLOC_MAX_WORKSPACE bytes per GPU, which
 * each GPU the library runs on holds until the process ends.  No device
 * memory is allocated or freed and no pinned host memory is used (the
 * tables are uploaded from a host buffer the library reuses; the host-side
 * plan uses the C++ heap).  The first call on a device looks up that
 * device's address of the array.
 *   mats, n, args, stream: as for muonh_step (pointers, shapes, dtypes);
 *     every desc.radius must be > 0: the caller holds R (||W_0||_F, or the
 *     value muonh_get_radii returns), since nothing persists between calls.
 *   opt: as for muonh_init; opt->workspace must be NULL.
 * Same plan, kernels and launch order as muonh_init + muonh_step with the
 * same options and radii: W and M come out bitwise equal.  Statistics and u
 * are not kept for the caller.
 * Errors: MUONH_EINVAL (as muonh_step, or a radius <= 0, or a workspace
 * given); MUONH_ENOMEM when the list's plan (muonh_workspace_size) exceeds
 * MUONH_NOALLOC_MAX_WORKSPACE, before anything is enqueued; MUONH_ENODEV;
 * MUONH_EHIP.  Every call on a GPU shares that GPU's array, which keeps the
 * last call's contents (each call uploads its own tables and clears the
 * Newton-Schulz buffers): calls that overlap in time on one GPU, on other
 * streams or from other threads, race; calls in order on one stream do
 * not.                                                                     */
#define MUONH_NOALLOC_MAX_WORKSPACE ((size_t)64 << 20)
int muonh_step_noalloc(const muonh_matrix_desc* mats, int32_t n, const muonh_options* opt,
                       const muonh_step_args* args, void* stream);

/* Synchronise the handle's last stream, then copy the n radii to host.  A
 * radius measured at init is rounded to float when measured, so these are
 * exactly the R the steps use: a new handle given them as the descriptors'
 * radius, with the saved W and M, continues bit for bit.                  */
int muonh_get_radii(muonh_handle* h, float* out, int32_t n);

/* Synchronise, then copy the n per-matrix statistics of the last step. */
int muonh_get_stats(muonh_handle* h, muonh_stats* out, int32_t n);

/* Test/debug: enqueue a copy of the Newton-Schulz output u of matrix idx
 * from the last step, in the matrix's own orientation (rows x cols, fp32,
 * row-major), to dst_device.                                              */
int muonh_copy_update(muonh_handle* h, int32_t idx, void* dst_device, void* stream);

/* Per-kernel timing with HIP events recorded on each step's stream.
 * muonh_set_timing(h, 1) starts recording (and clears the totals); every
 * later step records one event after each launch.  muonh_get_timing
 * synchronises, writes the totals in milliseconds over the *n_steps timed
 * steps since the last read into phases_ms[0..6] = momentum+pack (and its
 * finalise), NS X X^T, NS A A (each summed over the ns_steps launches), NS
 * B X (summed over the first ns_steps-1 launches), the last NS B X launch
 * (it writes u and reduces <W,u>, ||u||^2, ||W||^2 per tile), the finalise
 * of those sums, update; then clears the totals.
 * n_phases must be >= 7.                                                    */
int muonh_set_timing(muonh_handle* h, int32_t enable);
int muonh_get_timing(muonh_handle* h, float* phases_ms, int32_t n_phases, int32_t* n_steps);

/* Release the plan and any library-owned device memory.  NULL is a no-op. */
int muonh_destroy(muonh_handle* h);

const char* muonh_status_str(int status);
const char* muonh_last_error(void);

/* ---- host-only learning-rate helpers ------------------------------------
 * Eq. (11) of App. C: eta0 + (eta_min - eta0) s / S, s clamped to [0, S].   */
double muonh_lr_linear(double eta0, double eta_min, double s, double S);
/* Eq. (10) of App. C: linear warmup to `peak`, then
 * floor + (peak - floor) (1 + (k - warmup)/tau)^(-p).                         */
double muonh_lr_power(double k, double peak, double floor_, double warmup,
                      double tau, double p);
/* Warmup-stable-decay with linear decay over the last decay_ratio*total
 * steps (the §3.3.2 sweeps; plain reading of the pages).                     */
double muonh_lr_wsd(double k, double peak, double total, double decay_ratio,
                    double warmup, double eta_min);
/* Eq. (11) frozen from s_hold on: the constant-LR continuation that feeds
 * checkpoint averaging (§3.4: held from step 218,000 at base LR 4.08e-5).
 * Returns muonh_lr_linear(eta0, eta_min, min(s, s_hold), S).                */
double muonh_lr_linear_hold(double eta0, double eta_min, double s, double S, double s_hold);
/* Cosine decay from eta_max to eta_min over `total` steps after a linear
 * warmup of `warmup` steps (the post-training schedule, App. E); k is
 * clamped to [warmup, total] for the decay part.                            */
double muonh_lr_cosine(double k, double total, double eta_max, double eta_min, double warmup);
/* Effective LR of a Hyperball-wrapped matrix from the base schedule:
 * eta^H = multiplier * eta_base (§3.3.1; multiplier 10 in App. C, Tab. 8).
 * This is the value muonh_step_args.elr takes.                              */
double muonh_elr_from_base(double eta_base, double multiplier);

/* ---- AdamW for the parameters MuonH does not wrap -----------------------
 * The pages train embeddings, normalisation layers, the LM head and every
 * other non-wrapped parameter with AdamW at weight decay 0.1 on the base LR
 * schedule (§3.3; App. C, Tab. 8), and use Adam betas (0.9, 0.95) and
 * epsilon 1e-12 (App. E).  The update rule is the standard decoupled-decay
 * AdamW with bias correction, for step count t = 1, 2, ... and LR lr:
 *     W <- W (1 - lr wd);  m <- b1 m + (1-b1) g;  v <- b2 v + (1-b2) g^2
 *     W <- W - lr (m / (1-b1^t)) / (sqrt(v / (1-b2^t)) + eps)
 * computed in fp32 per element, one multi-tensor launch per step.
 * Conventions are those listed at the top of this file.                     */
typedef struct muonh_adamw_handle muonh_adamw_handle;

typedef struct muonh_adamw_tensor {
  void* w;          /* fp32 parameter, device, contiguous, updated in place    */
  const void* g;    /* gradient, device, g_dtype                                */
  void* m;          /* fp32 first moment, device, in place (zeros before t = 1) */
  void* v;          /* fp32 second moment, device, in place (zeros before t = 1)*/
  int64_t numel;    /* elements, >= 1                                           */
  int32_t g_dtype;  /* MUONH_F32 or MUONH_BF16                                  */
  int32_t reserved; /* must be 0                                                */
} muonh_adamw_tensor;

typedef struct muonh_adamw_options {
  float beta1;         /* 0.9  */
  float beta2;         /* 0.95 */
  float eps;           /* 1e-12 */
  float weight_decay;  /* 0.1  */
} muonh_adamw_options;

/* Fill *opt with the defaults listed above. */
void muonh_adamw_default_options(muonh_adamw_options* opt);

/* Plan the chunk table for these tensors (sizes and gradient dtypes are kept,
 * pointers are not) and allocate its small device tables on the current
 * device.  Errors: MUONH_EINVAL for n < 1, numel < 1, an unknown dtype, a
 * nonzero reserved field or options outside 0 <= beta < 1, eps > 0,
 * weight_decay >= 0; MUONH_EHIP for a HIP failure.  On failure *h is NULL. */
int muonh_adamw_init(muonh_adamw_handle** h, const muonh_adamw_tensor* t, int32_t n,
                     const muonh_adamw_options* opt);

/* One AdamW step at step count `step` (>= 1) with learning rate `lr` over the
 * same list (order, sizes, dtypes) as init; pointers may change between
 * steps.  w, m, v and an fp32 g must be 16-byte aligned, a bf16 g 8-byte
 * aligned.  Asynchronous on `stream`.  Errors: MUONH_EINVAL (null or
 * misaligned pointer, step < 1, non-finite lr), MUONH_EMISMATCH (list
 * differs from init), MUONH_EHIP.                                            */
int muonh_adamw_step(muonh_adamw_handle* h, const muonh_adamw_tensor* t, int32_t n,
                     float lr, int64_t step, void* stream);

/* Release the handle (waits for its last upload).  NULL is a no-op. */
int muonh_adamw_destroy(muonh_adamw_handle* h);

/* ---- block-scaled FP8 operands and products ------------------------------
 * The matrices MuonH steps are trained in block-scaled FP8 on the pages
 * (arXiv HTML §3.2; App. C): E4M3 values whose scales are powers of two, one
 * per group of 1 x 128 along the contraction for activations and gradients,
 * one per block of 128 x 128 for weights.  These entry points quantise and
 * multiply such operands; a layer's three products are
 *   forward          Y  = X W^T    rows of X   by rows of W
 *   data gradient    dX = dY W     rows of dY  by columns of W
 *   weight gradient  dW = dY^T X   columns of dY by columns of X
 * where "columns" is the column form below, so every product contracts two
 * operands along their contiguous axis.  dW (fp32 or bf16) is the gradient
 * muonh_step takes.  Conventions are those listed at the top of this file;
 * these entry points keep nothing between calls, allocate nothing, and may be
 * captured into a HIP graph.                                                */
typedef struct muonh_fp8_matrix {
  void*   data;        /* E4M3 (OCP, no infinities) [rows x ld], device, 16-byte aligned   */
  void*   scale;       /* E8M0 bytes [ceil(rows / block_rows) x ld_scale], device, 4-byte
                          aligned: value = data * 2^(byte - 127); byte 255 is NaN          */
  int64_t rows, cols;  /* cols: the contraction; either may be 0                           */
  int64_t ld;          /* bytes per row of data, a multiple of 128, >= cols; a product
                          reads columns cols .. up to the next multiple of 128, which
                          must be zero (the quantiser writes them)                         */
  int64_t ld_scale;    /* bytes per row of scale, a multiple of 4, >= ceil(cols / 128);
                          the quantiser zeroes the bytes up to the next multiple of 4      */
  int32_t block_rows;  /* 1 or 128                                                         */
  int32_t reserved;    /* must be 0                                                        */
} muonh_fp8_matrix;

/* Quantise x [rows x cols] (MUONH_F32 or MUONH_BF16, ldx elements between
 * rows) into its row form q (rows x cols) and / or its column form qt, that of
 * x transposed (cols x rows); either may be NULL.  Both take the same
 * block_rows.  For a block with largest finite magnitude amax the scale is the
 * least power of two 2^e with amax <= 448 2^e, e >= -127, and 1 for a block of
 * zeros; elements round to nearest even, NaN and Inf become NaN.
 * x needs element alignment only.  Errors: MUONH_EINVAL, MUONH_EHIP.        */
int muonh_block_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx,
                         const muonh_fp8_matrix* q, const muonh_fp8_matrix* qt, void* stream);

/* c [a.rows x b.rows] = a b^T, contracted over a.cols == b.cols in fp32 and
 * rounded once to c_dtype (MUONH_F32 or MUONH_BF16, ldc elements between
 * rows); accumulate = 1 adds the product to what c holds.  With a.cols = 0 the
 * product is zero.  Results are the same in every call on the same operands.
 * c_dtype chooses the arithmetic, too:
 *   bf16  the FP8 matrix unit, which of every 8 products drops what lies 2^-13
 *         below the largest.  With S the sum of |a_k b_k|, a sum is off by at most
 *         7 2^-13 S; 3e-7 S on normal operands, 4e-6 S on values over all of E4M3
 *         (measured, norms).  Where signs are random that is 2e-5 of the result,
 *         which bf16 hides (it rounds by 1.7e-3); where products cancel, not.
 *   fp32  the bf16 matrix unit on widened operands, with fp32 sums (at most
 *         K 2^-23 S; 1e-9 and 2e-8 S measured as above), at half that rate.  For a
 *         bf16 result with such sums, round this one.  Here an operand's value of
 *         2^128 or more (scale byte 247 and data of 256 or more) is infinite, and
 *         one below 2^-126 may lose bits.
 * workspace: device memory of muonh_block_matmul_workspace bytes, 256-byte
 * aligned, or NULL where that is 0; calls that may overlap in time need one
 * each.  Errors: MUONH_EINVAL, MUONH_ENOMEM (workspace too small), MUONH_EHIP. */
int muonh_block_matmul_workspace(const muonh_fp8_matrix* a, const muonh_fp8_matrix* b, int32_t c_dtype,
                                 size_t* bytes);
int muonh_block_matmul(const muonh_fp8_matrix* a, const muonh_fp8_matrix* b, void* c, int32_t c_dtype,
                       int64_t ldc, int32_t accumulate, void* workspace, size_t workspace_bytes,
                       void* stream);

/* muonh_step (same arguments, same arithmetic: W, M and the statistics come out
 * bitwise equal) whose update also writes the forms of the updated weights that
 * the next forward and backward passes multiply by: q[i], the row form of matrix
 * i, and qt[i], its column form, both with block_rows 128 and the bytes that
 * muonh_block_quantize gives for the updated W, without reading it again.  q or
 * qt may be NULL, and an entry whose data is NULL is not written (its other
 * members are not read).  The outputs must stay valid until the stream has
 * passed the step, and may change between steps.  The first call on a handle
 * allocates its tables on the device (12 bytes per 128 x 128 block), which
 * muonh_destroy releases; MUONH_ESTATE while `stream` is being captured.
 * Errors: as muonh_step; MUONH_EINVAL for an output whose shape, block_rows or
 * layout does not fit, that is named twice or that overlaps another (side by
 * side in rows of one pitch is allowed), a W, M or G of the step or the handle's
 * workspace (also the caller's, muonh_options.workspace); MUONH_ENOMEM.      */
int muonh_step_quantized(muonh_handle* h, const muonh_matrix_desc* mats, int32_t n,
                         const muonh_fp8_matrix* q, const muonh_fp8_matrix* qt,
                         const muonh_step_args* args, void* stream);

/* ---- layer norm and RMS norm ----------------------------------------------
 * The norms whose weights muonh_adamw_step trains, over the last axis of
 * x [rows x cols]:
 *   layer: mu = mean(x), r = 1/sqrt(mean((x - mu)^2) + eps), h = (x - mu) r
 *   rms:   r = 1/sqrt(mean(x^2) + eps),                      h = x r
 *   y = h weight (+ bias);  mean and rstd keep mu and r for the gradient
 *   dx = r (g - [mean(g)] - h mean(g h)),  g = dy weight     ([]: layer only)
 *   dweight = sum over rows of dy h,  dbias = sum over rows of dy
 * Statistics and sums are fp32, sums in a fixed order (those of squares too: a
 * row whose sum is beyond 3.4e38 gets rstd 0, and with eps 0 one whose squares are
 * below fp32's range an infinite one).  x, y, dy and dx share one dtype
 * (MUONH_F32 or MUONH_BF16) and need element alignment only; the vectors are
 * fp32.  y may be x, and dx may be x or dy (same address and pitch); an output or
 * workspace that overlaps anything else is refused.                          */
#define MUONH_NORM_LAYER 0
#define MUONH_NORM_RMS   1

typedef struct muonh_norm_args {
  const void*  x;
  const float* weight;   /* [cols]                                            */
  const float* bias;     /* [cols] or NULL                                    */
  void*        y;
  float*       mean;     /* [rows]; NULL for MUONH_NORM_RMS                   */
  float*       rstd;     /* [rows]                                            */
  int64_t      rows;     /* >= 0                                              */
  int64_t      cols;     /* 1 .. 2^26                                         */
  int64_t      ldx, ldy; /* elements between rows                             */
  int32_t      dtype;
  int32_t      kind;     /* MUONH_NORM_*                                      */
  float        eps;      /* >= 0                                              */
  int32_t      reserved; /* must be 0                                         */
} muonh_norm_args;

/* Errors: MUONH_EINVAL, MUONH_EHIP. */
int muonh_norm_forward(const muonh_norm_args* args, void* stream);

typedef struct muonh_norm_grad_args {
  const void*  dy;
  const void*  x;
  const float* weight;    /* [cols]                                           */
  const float* mean;      /* [rows]; NULL for MUONH_NORM_RMS                  */
  const float* rstd;      /* [rows]                                           */
  void*        dx;
  float*       dweight;   /* [cols]                                           */
  float*       dbias;     /* [cols] or NULL                                   */
  int64_t      rows;      /* >= 0; with 0 rows dweight and dbias are zero     */
  int64_t      cols;      /* 1 .. 2^26                                        */
  int64_t      ld_dy, ldx, ld_dx;
  int32_t      dtype;
  int32_t      kind;
  int32_t      accumulate; /* 1: add to dweight and dbias                     */
  int32_t      reserved;   /* must be 0                                       */
  void*        workspace;  /* muonh_norm_backward_workspace bytes, device,
                              256-byte aligned; calls that may overlap in time
                              need one each                                   */
  size_t       workspace_bytes;
} muonh_norm_grad_args;

/* Errors: MUONH_EINVAL, MUONH_ENOMEM (workspace too small), MUONH_EHIP. */
int muonh_norm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes);
int muonh_norm_backward(const muonh_norm_grad_args* args, void* stream);

/* ---- causal attention over packed sequences ---------------------------------
 * The attention between a layer's qkv and output products, and its gradients.
 * Sequence b of `sequences` is rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of the
 * tokens (an empty one is allowed); row i of it sees rows j <= i of the same
 * sequence.  Head h of q reads head h / (heads / kv_heads) of k and v:
 *   S_ij = scale q_i.k_j,  lse_i = log sum_j exp S_ij,  P_ij = exp(S_ij - lse_i)
 *   out_i = sum_j P_ij v_j
 *   dS_ij = scale P_ij (dout_i.v_j - dout_i.out_i)
 *   dq_i = sum_j dS_ij k_j,  dk_j = sum dS_ij q_i,  dv_j = sum P_ij dout_i
 * dk and dv over the rows i >= j and the heads that read them.
 *
 * q, out, dout, dq are bf16 [tokens x heads x dim], k, v, dk, dv [tokens x kv_heads x
 * dim], with contiguous heads and ld elements between tokens (slices of one fused
 * matrix are allowed), 16-byte aligned; ld a multiple of 8 below 2^23.  Scores,
 * softmax statistics and all sums are fp32; P and dS are rounded to bf16 where they
 * are multiplied, results once.  Sums run in a fixed order.
 *
 * The device reads cu_seqlens.  Its ends are taken into [0, tokens] and must not
 * decrease (repeat the last one to pad it to a fixed length): ends that do give undefined
 * results, but no access outside the tensors.  Rows that no sequence holds, before the
 * first and behind the last, are not read; in the results that zero_rest names they
 * become zeros, in others they stay as they were.
 *
 * A row all of whose scores are -inf has lse -inf and out NaN, one with a score of +inf NaN in
 * both.  A row whose lse is infinite or beyond 2^24 log 2 in magnitude, where fp32 does not
 * hold it to a unit, adds nothing to the gradients, and its dq is 0.  An infinity or a NaN in
 * a token of k or v reaches out and lse of later rows of its sequence (and its own), of no
 * earlier one; one in any operand of the backward pass but those rows' out and lse may
 * reach every gradient of its sequence.  Other sequences' results do not change.
 * An output or workspace that overlaps an input or another output is refused, unless
 * they lie side by side in rows of one pitch.                                */
#define MUONH_ZERO_OUT 1
#define MUONH_ZERO_LSE 2
#define MUONH_ZERO_DQ 4
#define MUONH_ZERO_DK 8
#define MUONH_ZERO_DV 16

typedef struct muonh_attention_args {
  const void*    q;
  const void*    k;
  const void*    v;
  void*          out;         /* read by muonh_attention_backward                 */
  float*         lse;         /* [heads x tokens]; read by the backward pass      */
  const int32_t* cu_seqlens;  /* [sequences + 1], device, not decreasing          */
  int64_t        tokens;      /* 0 .. 2^30                                        */
  int64_t        sequences;   /* >= 0                                             */
  int64_t        ld_q, ld_k, ld_v, ld_out;
  int32_t        heads;       /* a multiple of kv_heads                           */
  int32_t        kv_heads;    /* >= 1                                             */
  int32_t        dim;         /* 8, 16, .. 128                                    */
  float          scale;       /* > 0, usually dim^-1/2                            */
  int32_t        zero_rest;   /* a sum of MUONH_ZERO_*                            */
  int32_t        reserved;    /* must be 0                                        */
} muonh_attention_args;

typedef struct muonh_attention_grad_args {
  muonh_attention_args a;     /* the forward pass's arguments and results         */
  const void*    dout;
  void*          dq;
  void*          dk;
  void*          dv;
  int64_t        ld_dout, ld_dq, ld_dk, ld_dv;
  void*          workspace;   /* muonh_attention_backward_workspace bytes, device,
                                 256-byte aligned; calls that may overlap in time
                                 need one each                                    */
  size_t         workspace_bytes;
} muonh_attention_grad_args;

/* Errors: MUONH_EINVAL, MUONH_ENOMEM (workspace too small), MUONH_EHIP. */
int muonh_attention_forward(const muonh_attention_args* args, void* stream);
int muonh_attention_backward_workspace(const muonh_attention_args* args, size_t* bytes);
int muonh_attention_backward(const muonh_attention_grad_args* args, void* stream);

/* ---- residual addition, RMS norm and FP8 output ------------------------------
 * What stands between two linear layers of a block:
 *   h = x + residual, rounded to x's type        (residual NULL: h is x)
 *   rstd = 1/sqrt(mean(h^2) + eps),  y = h rstd weight   (rstd as muonh_norm_forward has it)
 * and y in block-scaled FP8 (blocks of 1 x 128, as muonh_block_quantize gives them): q,
 * its row form, and / or qt, its column form; either may be NULL.  y itself is
 * not stored: it is formed in fp32 from the h that is kept and rounded once, to
 * E4M3.  x, residual and h share one dtype and need element alignment only.  h may
 * be x or residual (same address and pitch); any other output that overlaps an
 * input or another output is refused.                                         */
typedef struct muonh_add_norm_args {
  const void*  x;
  const void*  residual;  /* or NULL                                          */
  const float* weight;    /* [cols]                                           */
  void*        h;         /* NULL if residual is                              */
  float*       rstd;      /* [rows]                                           */
  int64_t      rows;      /* >= 0                                             */
  int64_t      cols;      /* 1 .. 2^26                                        */
  int64_t      ldx, ld_residual, ldh;
  int32_t      dtype;     /* MUONH_F32 or MUONH_BF16                          */
  float        eps;       /* >= 0                                             */
} muonh_add_norm_args;

/* Errors: MUONH_EINVAL, MUONH_EHIP. */
int muonh_add_norm_quantize(const muonh_add_norm_args* args, const muonh_fp8_matrix* q, const muonh_fp8_matrix* qt,
                            void* stream);

/* The gradient of x (and of residual, which is the same) and of weight:
 *   dx = dh + rstd (g - n mean(g n)),  n = h rstd, g = dy weight;  dweight = sum dy n
 * dh, the gradient that reaches h by the residual stream, shares dy's dtype; dx may be dh, dy
 * or h.  args.x is h, args.kind MUONH_NORM_RMS, args.mean and args.dbias NULL; the
 * workspace is muonh_norm_backward_workspace's.                               */
typedef struct muonh_add_norm_grad_args {
  muonh_norm_grad_args g;
  const void*  dh;
  int64_t      ld_dh;
} muonh_add_norm_grad_args;

/* Errors: MUONH_EINVAL, MUONH_ENOMEM (workspace too small), MUONH_EHIP. */
int muonh_add_norm_backward(const muonh_add_norm_grad_args* args, void* stream);

/* ---- embedding ---------------------------------------------------------------
 * The table that muonh_adamw_step trains, [rows x cols]:
 *   out[t] = scale table[tokens[t]],  dtable[v] = scale sum over tokens[t] = v of dout[t]
 * A token outside 0 .. rows - 1 (padding) gives a row of zeros and adds nothing.
 * Each result is rounded once; sums are fp32, in a fixed order.  Matrices need element
 * alignment only; an output or workspace that overlaps anything else is refused.   */
typedef struct muonh_embedding_args {
  const void* tokens;       /* [count] int32 or int64, device                  */
  const void* table;        /* table_dtype                                     */
  void*       out;          /* [count x cols], out_dtype                       */
  int64_t     count;        /* 0 .. 2^24 - 1                                   */
  int64_t     rows;         /* 0 .. 2^30                                       */
  int64_t     cols;         /* 1 .. 2^20                                       */
  int64_t     ld_table, ld_out;
  int32_t     token_bytes;  /* 4 or 8                                          */
  int32_t     table_dtype;  /* MUONH_F32 or MUONH_BF16                         */
  int32_t     out_dtype;    /* MUONH_F32 or MUONH_BF16                         */
  float       scale;        /* finite                                          */
} muonh_embedding_args;

typedef struct muonh_embedding_grad_args {
  const void* tokens;
  const void* dout;         /* [count x cols], dout_dtype                      */
  void*       dtable;       /* [rows x cols], table_dtype; all of it is written */
  int64_t     count, rows, cols;   /* as above                                 */
  int64_t     ld_dout, ld_table;
  int32_t     token_bytes;
  int32_t     dout_dtype;
  int32_t     table_dtype;
  int32_t     accumulate;   /* 1: add to what dtable holds; rows that no token names
                               are then not touched                            */
  float       scale;
  int32_t     reserved;     /* must be 0                                       */
  void*       workspace;    /* muonh_embedding_backward_workspace bytes, device,
                               256-byte aligned; calls that may overlap in time
                               need one each                                   */
  size_t      workspace_bytes;
} muonh_embedding_grad_args;

/* Errors: MUONH_EINVAL, MUONH_ENOMEM (workspace too small), MUONH_EHIP. */
int muonh_embedding_forward(const muonh_embedding_args* args, void* stream);
int muonh_embedding_backward_workspace(int64_t count, int64_t rows, int64_t cols, size_t* bytes);
int muonh_embedding_backward(const muonh_embedding_grad_args* args, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MUONH_H_ */
