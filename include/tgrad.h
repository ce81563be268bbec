/*
 * tgrad.h - C ABI of the TensorGRaD optimizer step on AMD MI355X (gfx950).
 *
 * One handle optimises one weight tensor W of shape (I_1, ..., I_d) with the
 * TensorGRaD step. The gradient G splits into a sparse part S, held on an index set
 * Omega (the k = floor(rho * N) entries of largest |G|, taken out first), and a Tucker
 * low-rank part of what remains, R = G - scatter(S). Adam keeps its moments on the
 * small Tucker core and on the k sparse values. The full-size update comes back
 * through one factor product per mode; the sparse update is added into that same
 * buffer, and W is then updated in place. Omega and the factors are recomputed every
 * T steps: a top-k by magnitude, and an HOSVD from each mode's Gram matrix.
 *
 * Sources (no code exists on them): the nullthought.net summary of "TensorGRaD:
 * Tensor Gradient Robust Decomposition for Memory-Efficient Neural Operator
 * Training", sections 2-3 (G = L + S, sparse part extracted first, Tucker on the
 * residual, separate Adam updates, scatter-add after reconstruction, half-precision
 * weights with fp32 optimizer state, re-selection every T steps); the pith.science
 * review of arXiv 2501.02379, "What carries the argument" (factors reused for T
 * steps, projection to a core, Adam moments on the core, mode-wise reconstruction,
 * COO sparse set by top-k magnitude) and its appendix M excerpt of Theorem 2
 * (project, update optimizer states, project back).
 *
 * Conventions for every call:
 *   - Tensors are dense, contiguous, row-major (last index fastest). complex64 is
 *     interleaved (re, im) fp32 pairs. Element (linear) indices count complex
 *     elements, not floats.
 *   - Device pointers are HIP device addresses on the device that was current at
 *     tgrad_init; `stream` is a hipStream_t (NULL = the default stream). Every call
 *     that takes a stream only enqueues work on it and returns without waiting;
 *     device faults surface at the caller's next synchronisation.
 *   - Host pointers (marked host) are ordinary CPU memory; calls taking them
 *     synchronise the device before returning.
 *   - Return value: TGRAD_OK or an error code below; no call throws. After
 *     TGRAD_EHIP, tgrad_last_error() gives the HIP error string.
 *   - One handle is used by one host thread and one stream at a time. Separate
 *     handles are independent.
 */
#ifndef TGRAD_H
#define TGRAD_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct tgrad_handle tgrad_t;

/* Storage dtype of the weight and the gradient. A tgrad_t's state is always fp32. */
enum tgrad_dtype { TGRAD_F32 = 0, TGRAD_F16 = 1, TGRAD_BF16 = 2, TGRAD_C64 = 3 };

enum tgrad_status {
  TGRAD_OK = 0,
  TGRAD_EINVAL = 1,   /* invalid argument (null pointer, size or range) */
  TGRAD_ENOMEM = 2,   /* device allocation failed */
  TGRAD_EHIP = 3,     /* a HIP call or kernel launch failed */
  TGRAD_ESTATE = 4    /* call not valid in the handle's current state */
};

#define TGRAD_MAX_NDIM 8
#define TGRAD_MAX_FACTOR_DIM 128  /* largest I_n of a mode with r_n < I_n */

/*
 * Create a handle on the current HIP device and allocate all optimizer state.
 *   ndim            number of modes d, 1..8
 *   shape[d]        I_n >= 1; N = prod I_n must be < 2^32
 *   tucker_ranks[d] r_n in [1, I_n]. r_n == I_n keeps mode n uncompressed (identity
 *                   factor, no mode product); r_n < I_n needs I_n <= 128 and
 *                   r_n <= N / I_n (the rank of the mode-n unfolding).
 *   dtype           enum tgrad_dtype of W and G
 *   sparse_ratio    rho in [0, 1]; k = floor(rho * N) computed in IEEE double
 *   T               refresh period >= 1: a refresh runs before every step t with
 *                   (t - 1) mod T == 0, t = 1, 2, ... (pith.science: factors and
 *                   Omega reused for T steps; nullthought section 3)
 *   lr, beta1, beta2, eps   Adam: lr >= 0, beta in [0, 1), eps >= 0
 * Moments start at zero, t = 0. The handle owns every device buffer it allocates.
 * Errors: TGRAD_EINVAL, TGRAD_ENOMEM, TGRAD_EHIP. *out is NULL on error.
 */
int tgrad_init(tgrad_t **out, int ndim, const int64_t *shape, const int64_t *tucker_ranks,
               int dtype, double sparse_ratio, int64_t T, double lr, double beta1,
               double beta2, double eps);

/*
 * One optimizer step on device buffers `weight` (W, updated in place) and `grad`
 * (G, caller-owned, N elements of dtype, 16-byte aligned, only read).
 *   t <- t + 1; if a refresh is due for t and tgrad_refresh was not already called
 *   for it, refresh from `grad` first. Then: S = G[Omega] (fp32) and R = G with
 *   Omega zeroed; core C = R x_1 U1^H ... x_d Ud^H; Adam on C and on S (fp32
 *   moments); Delta = N_C x_1 U1 ... x_d Ud with lambda N_S added at Omega;
 *   W <- round(W * decay - lr * Delta), one rounding per element (lambda = 1 and
 *   decay = 1 unless tgrad_set_options says otherwise; nullthought section 3 step
 *   order; pith.science Theorem 2).
 * Both buffers must stay valid until the work on `stream` completes.
 * Errors: TGRAD_EINVAL (null handle/pointer, grad not 16-byte aligned), TGRAD_EHIP.
 * On an error t is not advanced (a refresh that completed for this t stays valid).
 */
int tgrad_step(tgrad_t *h, void *weight, const void *grad, void *stream);

/*
 * Several tensors' steps as one call (many small FNO layers per optimizer step):
 * tgrad_step(hs[i], weights[i], grads[i], .) for i < n, issued on up to four internal
 * streams (per device, created on first use, default priority) that start after the
 * work already queued on `stream`; `stream` then waits for all of them, so later work
 * on it sees every update. The tensors' kernels overlap on the device, filling the
 * tail of each launch with another tensor's work; each handle's results are bit for
 * bit those of tgrad_step. The handles must be distinct and on one device; calls are
 * serialised by an internal mutex. Errors: TGRAD_EINVAL (n < 0, a NULL array or entry,
 * a grad not 16-byte aligned, a repeated handle, handles on different devices), or the
 * first failing step's status (the steps before it are issued and joined).
 */
int tgrad_step_many(tgrad_t *const *hs, void *const *weights, const void *const *grads, int n,
                    void *stream);

/*
 * Refresh Omega and the Tucker factors from `grad` (device, N elements of dtype,
 * 16-byte aligned):
 * Omega = the k largest magnitudes (ties to the lowest linear index), stored
 * ascending; each U(n) (r_n < I_n) = the r_n leading eigenvectors of the mode-n Gram
 * matrix of the residual, descending eigenvalue order, each column scaled so its
 * largest-magnitude entry (lowest row on ties) is real positive. `grad` is only
 * read. Moments and t are untouched; the refresh serves step t + 1.
 * (nullthought section 3: re-select sparse indices and low-rank subspace every T
 * steps; pith.science: top-k magnitude, Tucker/HOSVD factors.)
 * Errors: TGRAD_EINVAL (null handle/pointer, grad not 16-byte aligned), TGRAD_EHIP.
 */
int tgrad_refresh(tgrad_t *h, const void *grad, void *stream);

/* Free every buffer of the handle. The caller synchronises first. NULL is a no-op. */
int tgrad_destroy(tgrad_t *h);

/* Static description of an error code; never NULL. */
const char *tgrad_status_string(int status);
/* Last HIP error message recorded on the handle (empty string if none). */
const char *tgrad_last_error(const tgrad_t *h);

/* ---------------------------------------------------------------- introspection.
 * Not on the hot path. Host buffers; each call synchronises the device. */

typedef struct tgrad_info {
  int64_t ndim, dtype, numel, k, core_numel, T, t;
  int64_t shape[TGRAD_MAX_NDIM];
  int64_t ranks[TGRAD_MAX_NDIM];
  int64_t state_bytes;      /* moments, core, factors, Omega (optimizer state) */
  int64_t workspace_bytes;  /* transient buffers owned by the handle */
  /* The eigensolver at the last refresh (0 before any): the most Jacobi sweeps any mode
   * took to reach its off-diagonal bound (0 for a mode that the tridiagonal route for
   * real modes up to 64 served), and the number of modes that reached the sweep cap
   * first (their factors are then less accurate than the bound promises). */
  int64_t eig_sweeps_max;
  int64_t eig_unconverged;
} tgrad_info;

/* Synchronises the device once the handle has refreshed (to read the eigensolver
 * report). Errors: TGRAD_EINVAL, TGRAD_EHIP. */
int tgrad_get_info(const tgrad_t *h, tgrad_info *out);

/* Omega, k uint32 linear indices ascending. cap = capacity of out (elements). */
int tgrad_get_omega(tgrad_t *h, uint32_t *out, int64_t cap);

/* U(n) as I_n x r_n row-major fp32 (complex: interleaved pairs, 2 I_n r_n floats).
 * TGRAD_EINVAL for an identity mode (r_n == I_n) or too small cap (floats). */
int tgrad_get_factor(tgrad_t *h, int mode, float *out, int64_t cap);

/* Gram-matrix eigenvalues of mode n from the last refresh, I_n doubles, descending. */
int tgrad_get_eigvals(tgrad_t *h, int mode, double *out, int64_t cap);

/* Adam moments (fp32; complex = pairs): core m, v (core_numel*P each) and sparse m,
 * v (k*P each). Any pointer may be NULL to skip it. */
int tgrad_get_moments(tgrad_t *h, float *m_core, float *v_core, float *m_sparse,
                      float *v_sparse);

/* Test hooks: replace Omega (k ascending unique indices < N) or U(n) (layout as
 * tgrad_get_factor) from host memory, and mark the handle refreshed for step t + 1
 * so the next step uses them. */
int tgrad_set_omega(tgrad_t *h, const uint32_t *omega, int64_t k);
int tgrad_set_factor(tgrad_t *h, int mode, const float *U, int64_t n_floats);
int tgrad_mark_refreshed(tgrad_t *h);

/* Test hook: while `delta` is set, every step also writes its fp32 update before the
 * weight rounding, Delta = Delta_L + lambda N_S at Omega (the value W * decay - lr * Delta
 * is rounded from), into `delta`: a caller-owned device buffer of N * P floats (P = 2
 * for complex64, interleaved), 16-byte aligned, valid until the stream's work is done.
 * The kernels that write it are separate instantiations of the weight-update launches,
 * with the same arithmetic; W is updated as usual. NULL turns the capture off.
 * Errors: TGRAD_EINVAL (NULL handle, misaligned buffer). */
int tgrad_debug_capture_delta(tgrad_t *h, float *delta);

/* Test / benchmark hook: when the last two modes are both compressed and a slab of
 * them fits in LDS, the projection's first two mode products and the reconstruction's
 * last two run as one launch each (the default). For bf16/fp16 tensors with small
 * enough slabs those launches use one wave per slab on bf16 MFMAs (exact bf16 splits of
 * the fp32 operands), otherwise workgroup-wide fp32 MFMA tiles; where mode d-3 is also
 * compressed (I(d-3) a multiple of 16 up to 64, rank <= 32), the projection's first
 * launch takes mode d-3 as well (one workgroup per index of the leading modes), and,
 * where I(d-3) is a multiple of 12 up to 64 (16-bit weights, 16-byte aligned), so does
 * the reconstruction's last launch, with the merge and the weight update (the mode d-2
 * tensor stays on chip). enable = 0 selects one launch per mode; 1 the fused form
 * (default choice of kernels); 2 the fused two-mode form with the workgroup-tile kernel
 * only; 3 the fused two-mode form with the slab kernels, without the three-mode
 * launches; 4 as 1 but with the two-mode reconstruction. enable = 1 to 4 returns
 * TGRAD_EINVAL where the fused form does not apply. The unfused plan projects a residual copy of grad, so enable = 0 allocates an
 * N-element workspace the first time (TGRAD_ENOMEM if that fails). Results agree to
 * fp32 rounding; takes effect at the next step. */
int tgrad_set_fusion(tgrad_t *h, int enable);

/* Test / benchmark hook: in a bf16/fp16 tensor whose last three modes are all
 * compressed, a refresh forms their three Grams in one launch that reads the residual
 * once (pith.science "What carries the argument": every factor comes from the Gram of
 * its mode's unfolding, and each Gram is a sum over slabs of the last three modes, so
 * one staged slab serves all three). It applies when the two modes before the last are
 * at most 64, the last at most 32, and one slab of the three modes is a multiple of 8
 * elements and at most 128 KiB; the input must be 16-byte aligned (otherwise one launch
 * per mode is used). Bit 0 of enable = 1 selects it (the default; TGRAD_EINVAL where it
 * does not apply), 0 one Gram launch per mode. Bit 1 (enable = 2 or 3) makes every Gram
 * launch read the gradient itself and clear Omega's entries in its staged tiles through
 * the membership bitmask, instead of reading the residual copy the top-k pass writes
 * (the default, enable 0 or 1). Results agree to fp32 rounding of the partial sums;
 * takes effect at the next refresh. */
int tgrad_set_gram_fusion(tgrad_t *h, int enable);

/* Test / benchmark hook: work that runs on a second stream the handle owns (created by
 * tgrad_init, default priority), forked from the caller's stream and joined back before
 * the call's later work, so every call stays ordered on the caller's stream.
 *  adam: when the COO gather is folded into the first projection launch and further
 *        launches follow it, the Adam update of the k sparse values (the nullthought
 *        summary, section 3: S and the low-rank core keep separate Adam states) waits
 *        for that first launch and overlaps the projection's later launches and the
 *        core's Adam update; the reconstruction waits for it. The update is element-wise:
 *        results are bit-identical either way. The fork and the join cost about 10 us a
 *        step, so adam = 1 (the default) selects it only when the sparse part holds at
 *        least 2^22 values (k, times 2 for complex data); 2 whenever it applies; 0 runs
 *        both updates in one launch on the caller's stream. Its launch is named
 *        adam_sparse (tgrad_kernel_name).
 *  eig:  at a refresh whose last three modes' Grams come from one launch (see
 *        tgrad_set_gram_fusion), the eigensolver of the compressed modes before them
 *        (pith.science "What carries the argument": each factor from its own mode's
 *        Gram) runs beside that launch, which then leaves one CU per such matrix free.
 *        1 (default) or 0. With fewer workgroups the three-mode launch sums its partial
 *        Grams in another grouping, so factors agree to fp64 rounding of the Grams.
 * Takes effect at the next step or refresh. */
int tgrad_set_stream_overlap(tgrad_t *h, int adam, int eig);

/* Test / benchmark hook: with the fused launch plan, two neighbouring compressed modes
 * ahead of the trailing ones (the projection's last two products, the reconstruction's
 * first two) run as one launch. The tensor between the two products is never written
 * (pith.science "What carries the argument": the projection and reconstruction are
 * chains of mode-wise products, so any two neighbours may be contracted together).
 * It applies to real tensors when the product of the sizes after the two modes is a
 * multiple of 16 and both modes' sizes on each side are multiples of 4 up to 64.
 * enable = 1 selects it (the default; TGRAD_EINVAL where it does not apply), 0 one
 * launch per mode. Results agree to fp32 rounding; takes effect at the next step. */
int tgrad_set_pair_fusion(tgrad_t *h, int enable);

/* Test / benchmark hook: a single mode product on fp32 data (the projection's later
 * modes, the reconstruction's leading ones) runs on a streaming kernel where it applies:
 * every wave owns all output rows of 64 consecutive trailing columns and loads the next
 * such tile while it multiplies the current one, without LDS staging or workgroup
 * barriers (pith.science "What carries the argument": projection and reconstruction are
 * chains of mode-wise products). It applies when the mode has at most 64 values on
 * either side (complex data: Re and Im of the factor in two accumulator sets) and the
 * trailing part is at least 32 values (complex: 16) and a multiple of 4 (complex: 2).
 * Products over the last mode (no trailing part: the one-mode plan's first projection
 * and its weight-updating last reconstruction) run on a kernel that streams rows of the
 * tensor with the factor in registers, where the factor fits. enable = 1 selects both
 * (the default), 0 the tiled kernel for every single mode product; enable = n >= 2
 * selects them with at most n - 1 workgroups of 4 waves for the first (so that small
 * tensors exercise a wave's walk over several tiles). Negative enable: TGRAD_EINVAL.
 * Results agree to fp32 rounding; takes effect at the next step. */
int tgrad_set_stream_products(tgrad_t *h, int enable);

/* ---------------------------------------------------------------- variants.
 * Choices the method leaves open, as options of a handle (defaults: the plain method,
 * bit for bit):
 *   weight_decay   decoupled decay as in AdamW (the nullthought summary trains L and S
 *                  with AdamW; the pith.science page's experiment settings use weight
 *                  decay 1e-4 and 2e-6): W <- round(fp32(W) * decay - lr * Delta) with
 *                  decay = fp32(1 - lr * weight_decay) formed in fp64. >= 0; default 0.
 *   sparse_scale   lambda, the sparse scale factor the pith.science page lists among the
 *                  method's hyper-parameters (its value is not reported): Delta at Omega
 *                  gets fp32(lambda) * N_S instead of N_S. Finite; default 1.
 *   selection      how a refresh picks Omega (pith.science "What carries the argument":
 *                  top-k magnitude or random sampling): TGRAD_SELECT_TOPK, or
 *                  TGRAD_SELECT_RANDK = a uniformly random k-subset: element e gets the top
 *                  31 bits of SplitMix64's output for the state
 *                  seed + 0x9E3779B97F4A7C15 * (t * 2^32 + e + 1), t the step the refresh
 *                  serves, and the k largest keys (ties to the lowest index) are taken.
 *   remap_moments  0 (default): the sparse Adam moments stay with their position in
 *                  Omega across a refresh; 1: they follow their element, and an element
 *                  new to Omega starts from zero moments. Enabling it allocates two more
 *                  k*P fp32 buffers and a second bitmask (synchronises the device).
 *   seed           rand-k base seed.
 *   order          the decomposition order (pith.science lists "sparse then low-rank" as
 *                  the tuned choice; the nullthought summary reports the reverse as
 *                  worse): TGRAD_ORDER_SPARSE_FIRST (default), or
 *                  TGRAD_ORDER_LOWRANK_FIRST: a refresh takes the Tucker factors from the
 *                  HOSVD of G itself and Omega as the top-k of the fp32 residual G - L,
 *                  L = (G x_n Un^H ...) x_n Un ... with the core in fp32; a step projects
 *                  the whole G to the core, reconstructs L and takes S = (G - L)[Omega].
 *                  Enabling it allocates an N-element fp32 workspace (complex: 2N).
 * Options take effect at the next step or refresh. Errors: TGRAD_EINVAL (NULL, a
 * negative or non-finite weight_decay, a non-finite sparse_scale, an unknown selection,
 * remap or order value), TGRAD_ENOMEM, TGRAD_EHIP. */
enum tgrad_selection { TGRAD_SELECT_TOPK = 0, TGRAD_SELECT_RANDK = 1 };
enum tgrad_order { TGRAD_ORDER_SPARSE_FIRST = 0, TGRAD_ORDER_LOWRANK_FIRST = 1 };
typedef struct tgrad_options {
  double weight_decay;
  double sparse_scale;
  int32_t selection;
  int32_t remap_moments;
  uint64_t seed;
  int32_t order;
  int32_t reserved;   /* 0 */
} tgrad_options;
void tgrad_default_options(tgrad_options *out);
int tgrad_set_options(tgrad_t *h, const tgrad_options *opt);
int tgrad_get_options(const tgrad_t *h, tgrad_options *out);

/* ---------------------------------------------------------------- checkpoint.
 * The optimizer state as one host byte string, to stop and resume training: the step
 * count and refresh mark, Omega, every U(n) with its Gram eigenvalues, and the core and
 * sparse Adam moments. tgrad_state_size gives its length (-1 for a NULL handle).
 * tgrad_save_state writes it into `buf` (cap >= that size, host memory).
 * The header also records T, lr, betas, eps and every tgrad_options field.
 * tgrad_load_state restores it into a handle created with the same shape, Tucker ranks,
 * dtype, sparse_ratio, T, betas and eps, and set to the same options; only the learning
 * rate may differ (the loading handle's lr is used, as a schedule would change it).
 * Steps then continue exactly as they would have in the saved handle.
 * Both synchronise the device. Errors: TGRAD_EINVAL (NULL, too small a buffer, a size,
 * header, shape, hyper-parameter, option or Omega that does not match), TGRAD_EHIP. */
int64_t tgrad_state_size(tgrad_t *h);
int tgrad_save_state(tgrad_t *h, void *buf, int64_t cap);
int tgrad_load_state(tgrad_t *h, const void *buf, int64_t size);

/* ---------------------------------------------------------------- without allocation.
 * For callers that cannot allocate device memory while they run: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.
 * tgrad_refresh_noalloc is tgrad_refresh (same kernels and results: Omega bit for bit,
 * factors to fp32 rounding of the Gram partial sums) with every scratch buffer its
 * kernels use -- the top-k workspace, the Gram partial sums and the Gram matrices -- in
 * one file-scope device array of the library, TGRAD_NOALLOC_SCRATCH_BYTES per GPU, held
 * until the process ends, instead of the handle's workspace. Its Gram launches read
 * `grad` with Omega's entries cleared through the membership bitmask, so no residual
 * copy is written, and where the partial sums would not fit they use fewer workgroups.
 * It calls no hipMalloc or hipFree (the array's address is looked up once per GPU).
 * Every call on one GPU uses that GPU's array, which keeps the last call's contents (the
 * kernels clear what must start at zero): calls that overlap on one GPU, from several
 * threads or streams, race. Per-launch timing is not recorded during the call.
 * Errors: as tgrad_refresh; TGRAD_EINVAL also when the refresh needs more than the array
 * holds (the top-k workspace grows as 16 N / 1024 bytes, so N up to about 2.9e9 fits; a
 * Gram partial sum needs 8 (I_n P)^2 bytes per workgroup) or the handle uses the
 * low-rank-first order (which needs full-size intermediates); TGRAD_EHIP when the
 * array's address cannot be obtained. */
#define TGRAD_NOALLOC_SCRATCH_BYTES (48ull << 20)
int tgrad_refresh_noalloc(tgrad_t *h, const void *grad, void *stream);

/* ---------------------------------------------------------------- launch record.
 * The kernel launches of the last tgrad_step, tgrad_refresh or tgrad_refresh_noalloc call
 * on the handle, in issue order (a step that refreshed lists the refresh's first), with
 * the algorithmic work of each: bytes_read and bytes_written count once every gradient,
 * weight, intermediate, index, moment and sparse value the launch's part of the method
 * needs (the membership bitmask and word ranks are counted only where a top-k pass
 * produces them or a masked Gram reads them); flops are 2 K M per column of each mode
 * product and Gram (K, M the real sizes of the contracted and produced mode). modes: bit
 * n set when the launch contracts mode n. Host memory; no device work.
 * Returns the number of launches (the first min(cap, number) are written to out), or
 * -1 for a NULL handle, cap < 0 or out NULL with cap > 0. */
typedef struct tgrad_launch {
  int32_t kernel;   /* kernel id, see tgrad_kernel_name */
  int32_t modes;
  int64_t bytes_read, bytes_written, flops;
} tgrad_launch;
int tgrad_last_launches(const tgrad_t *h, tgrad_launch *out, int cap);

/* ---------------------------------------------------------------- timing.
 * When enabled, every kernel launch of step/refresh is bracketed by HIP events on
 * the launch stream (at most max_records launches are kept). tgrad_timing_read
 * synchronises, then returns per-kernel-id totals: launches[id] and ms[id] for
 * id < n_ids (n_ids <= TGRAD_MAX_KERNEL_IDS) and resets the records. */
#define TGRAD_MAX_KERNEL_IDS 48
int tgrad_timing_enable(tgrad_t *h, int enable, int max_records);
int tgrad_timing_read(tgrad_t *h, int64_t *launches, double *ms, int n_ids);
/* Restricts the timing above to the launches of kernel id (0 <= id <
 * TGRAD_MAX_KERNEL_IDS, see tgrad_kernel_name), so that a timed run carries one event
 * pair per launch of that kernel and none around the others; id = -1 times every launch
 * again (the default). Errors: TGRAD_EINVAL (NULL handle, id out of range). */
int tgrad_timing_only(tgrad_t *h, int id);
const char *tgrad_kernel_name(int id);

/* ---------------------------------------------------------------- the other tensors.
 * AdamW over many tensors at once: the biases, norm weights and small products of a model
 * whose large tensors the calls above optimise. One handle steps n tensors in one launch
 * for every 240 of them (and every 2^32 values); weights and gradients are the caller's and
 * are passed to every call. Per value, each operation rounded to fp32 (the division is a product with a
 * reciprocal that is within one unit of the last place):
 *   g' = g * coefficient (see tgrad_adamw_grad_norm; g' = g without a clip)
 *   m = b1 m + (1 - b1) g';   v = b2 v + (1 - b2) g'^2
 *   w <- round(w * decay - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps))
 * with decay = fp32(1 - lr * weight_decay) and t the step's number, 1 for the first.
 * complex64 tensors are taken as twice as many real values.
 *
 * The state is one flat device buffer of the caller's (tgrad_adamw_state_bytes, 16-byte
 * aligned), zeroed for a new run or filled with a saved state before the first step. With
 * S = tgrad_adamw_state_values, in which every tensor's values start at a multiple of 128:
 *   state_bits 32:  m[S] and v[S], fp32.
 *   state_bits 8:   m[S] and q[S] codes, one byte each, then ms[S/128] and qs[S/128], one
 *     byte for every 128 of them. q is sqrt(v). A scale byte is the exponent field f of the
 *     largest magnitude of its 128 values as fp32 (zero: 0); a code's value is 2^(f - 14)
 *     times the fp32 number whose bits are code << 20 (m: sign in bit 7, the other 7 bits
 *     shifted) or code << 19 (q). f = 255 stands for NaN in all 128 values; a q that is
 *     not finite turns its group and m's into that. Rounding is random and unbiased: to the bits of
 *     the scaled value, h >> 12 (m) or h & 0x7FFFF (q) is added before the rest is cut off,
 *     h = mix(place ^ key): h *= 0xBF58476D, h ^= h >> 16, h *= 0x94D049BB, h ^= h >> 13 in
 *     32 bits, place the value's index in the flat state, key the low half of SplitMix64's
 *     output for the state seed + t * 0x9E3779B97F4A7C15. A q above zero keeps code 1 at
 *     least. The step itself uses m and v before they are rounded.
 *
 * The step number t is kept on the device and counts on under graph replay; tgrad_adamw_
 * get_steps and set_steps read and write the steps made (both synchronise the device).
 * As the other calls, one handle is used by one host thread and one stream at a time.
 */
typedef struct tgrad_adamw tgrad_adamw_t;

/* Values of the flat state and its bytes; -1 for invalid sizes (n < 1, a negative numel or
 * an unknown dtype or state_bits). Host only. */
int64_t tgrad_adamw_state_values(int n, const int64_t *numel, const int *dtype);
int64_t tgrad_adamw_state_bytes(int n, const int64_t *numel, const int *dtype, int state_bits);

/*
 * Create a handle on the current HIP device for n >= 1 tensors (synchronises the device).
 *   numel[n]         elements of each, >= 0; at most 2^27 pieces of 2048 values in all
 *   dtype[n]         enum tgrad_dtype of the weights
 *   grad_dtype[n]    of the gradients: the weight's, or TGRAD_F32 for a 16-bit weight
 *   weight_decay[n]  of each tensor, >= 0
 *   state_bits       32 or 8
 *   lr, beta1, beta2, eps   lr >= 0, beta in [0, 1), eps >= 0; lr and eps finite
 *                    (a positive eps below 2^-126 counts as that)
 *   seed             of the 8-bit state's rounding
 *   state            the buffer above; it must outlive the handle. Its contents are neither
 *                    read nor written by this call.
 * Errors: TGRAD_EINVAL, TGRAD_ENOMEM, TGRAD_EHIP. *out is NULL on error.
 */
int tgrad_adamw_init(tgrad_adamw_t **out, int n, const int64_t *numel, const int *dtype,
                     const int *grad_dtype, const double *weight_decay, int state_bits, double lr,
                     double beta1, double beta2, double eps, uint64_t seed, void *state);

/* Free the handle's own device memory (the state stays the caller's). The caller
 * synchronises first. NULL is a no-op. */
int tgrad_adamw_destroy(tgrad_adamw_t *h);
const char *tgrad_adamw_last_error(const tgrad_adamw_t *h);

/* The learning rate from the next step on (>= 0, finite); a captured step keeps its own. */
int tgrad_adamw_set_lr(tgrad_adamw_t *h, double lr);
int tgrad_adamw_get_steps(tgrad_adamw_t *h, int64_t *steps);
int tgrad_adamw_set_steps(tgrad_adamw_t *h, int64_t steps);

/*
 * One step of every tensor: weights[i] (updated in place) and grads[i] (only read) are
 * device buffers of numel[i] contiguous elements aligned to their element's real part (both
 * may be NULL where numel[i] is 0).
 *   clip          NULL, or two device floats from tgrad_adamw_grad_norm: the gradients are
 *                 multiplied by clip[1], and where the norm clip[0] is not finite the whole
 *                 step is left out on the device: weights, state and t stay as they are.
 *   m_out, v_out  both NULL, or (8-bit state) device buffers of S bf16 values, 16-byte
 *                 aligned, distinct: the new m and sqrt(v) as the values that the stored
 *                 codes stand for (at most 5 significant bits, so exact in bf16 above its
 *                 subnormal range). Left alone where the step is left out.
 * Errors: TGRAD_EINVAL (a NULL or misaligned argument), TGRAD_EHIP.
 */
int tgrad_adamw_step(tgrad_adamw_t *h, void *const *weights, const void *const *grads,
                     const float *clip, void *m_out, void *v_out, void *stream);

/*
 * The norm of all gradients together, for clipping and loss scaling, without a host
 * synchronisation: out[0] = norm = grad_scale * sqrt(sum g^2), out[1] = the coefficient
 * grad_scale * min(1, max_norm / norm) that turns the gradients as they are into scaled and
 * clipped ones. The sum is in fp64 and in a fixed order. max_norm > 0 (INFINITY: no
 * clipping), grad_scale > 0 and finite (1 over the loss scale). out: two device floats.
 * Errors: TGRAD_EINVAL, TGRAD_EHIP.
 */
int tgrad_adamw_grad_norm(tgrad_adamw_t *h, const void *const *grads, double max_norm,
                          double grad_scale, float *out, void *stream);

/*
 * Layer norm over the last axis of `rows` rows of `cols` elements, and its gradients; the
 * weight's and the bias's are among the tensors of a tgrad_adamw_t. Statistics and sums are
 * fp32, each result is rounded once:
 *   mean = sum x / cols;  rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps);  n = (x - mean) rstd
 *   y = n weight + bias
 *   dx = rstd (h - mean(h) - n mean(h n)),  h = dy weight
 *   dweight = sum over rows of dy n,  dbias = sum over rows of dy
 * The sums over rows are formed in a fixed order.
 *   x, dy           device, rows x_stride (dy_stride) >= cols elements apart
 *   y, dx           device, contiguous; no result overlaps an input
 *   mean, rstd      device, rows floats: written by forward, read by backward
 *   weight, bias    device, cols elements of weight_dtype; NULL: 1 and 0
 *   dweight, dbias  device, cols elements of weight_dtype, each may be NULL
 *   dtype           TGRAD_F32, TGRAD_F16 or TGRAD_BF16 of x, y, dy and dx
 *   weight_dtype    the same, or TGRAD_F32
 *   workspace       device, tgrad_layer_norm_workspace bytes, 16-byte aligned; only needed
 *                   for dweight or dbias. It may be reused once the stream's work is done.
 * rows = 0 is valid (dweight and dbias become 0). cols >= 1. Every pointer is aligned to its
 * element. Errors: TGRAD_EINVAL, TGRAD_EHIP.
 */
int tgrad_layer_norm_forward(const void *x, int64_t x_stride, const void *weight, const void *bias,
                             void *y, float *mean, float *rstd, int64_t rows, int64_t cols,
                             int dtype, int weight_dtype, double eps, void *stream);
/* Bytes of the workspace; -1 for invalid sizes. Host only. */
int64_t tgrad_layer_norm_workspace(int64_t rows, int64_t cols);
int tgrad_layer_norm_backward(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride,
                              const void *weight, const float *mean, const float *rstd, void *dx,
                              void *dweight, void *dbias, int64_t rows, int64_t cols, int dtype,
                              int weight_dtype, void *workspace, void *stream);

/* ---------------------------------------------------------------- matrices.
 * The products of a model's blocks, beside the tensors above: an optimizer for matrices and
 * the gated layer whose two weights are such matrices.
 *
 * Newton-Schulz orthogonalisation: with coefficients (a, b, c),
 *   X = U / (|U| + eps), |U| the root of the sum of squares; `steps` times:
 *   A = X X^T,  X = a X + (b A + c A A) X      (rows > cols: the same of the transpose)
 * which brings X's singular values near 1. (3.4445, -4.7750, 2.0315) and 5 steps are usual.
 * The products take fp16 parts of X, A and B = b A + c A A with fp32 sums, held under 2^12
 * (X) and 2^8: matrices whose X or B leave +-16 or +-256 in some step overflow, which with the
 * usual coefficients none do. X is carried in 22 bits between the steps. bf16 results come from
 * products of the upper parts (11 bits), 3e-4 to 2e-3 of the result's norm off before they are
 * rounded; fp32 and fp16 results, and those of matrices of up to 1024 values, from products of both
 * parts, 3e-7 to 1e-5. A matrix of zeros
 * stays one (where eps > 0); one with a value that is not finite becomes NaN.
 *
 * tgrad_orthogonalize: `count` matrices of rows x cols values.
 *   x          device, matrices matrix_stride and their rows row_stride >= cols elements apart
 *   out        device, contiguous, of x's type; may be x where that is contiguous
 *   dtype      TGRAD_F32, TGRAD_F16 or TGRAD_BF16
 *   steps      1 to 100;  coefficients: host, three finite values;  eps >= 0, finite
 *   workspace  device, tgrad_orthogonalize_workspace bytes, 16-byte aligned (NULL for 0). It may
 *              be reused once the stream's work is done.
 * count = 0 is valid. 1 <= rows, cols <= 2^19, and at most 2^21 workgroups' parts in a launch.
 * Errors: TGRAD_EINVAL, TGRAD_EHIP. The workspace's size is -1 for invalid sizes (host only). */
int64_t tgrad_orthogonalize_workspace(int64_t count, int64_t rows, int64_t cols, int dtype);
int tgrad_orthogonalize(const void *x, int64_t matrix_stride, int64_t row_stride, void *out,
                        int64_t count, int64_t rows, int64_t cols, int dtype, int steps,
                        const double *coefficients, double eps, void *workspace, void *stream);

/* Muon over many matrices at once. Per tensor (count matrices of rows x cols values, one after
 * the other), with g' = g * coefficient (see tgrad_adamw_grad_norm; g' = g without a clip):
 *   m = mu m + (1 - mu) g';   u = (1 - mu) g' + mu m  (nesterov)  or  m
 *   w <- round(w * decay - lr * scale * orthogonalised(u))
 * with decay = fp32(1 - lr * weight_decay), and products as for a result of w's type. The
 * momentum is one flat fp32 buffer of the caller's (tgrad_muon_state_values floats, 16-byte
 * aligned) in which every tensor's values start at a multiple of 128, zeroed for a new run.
 * A step is captured and replayed as it is; one handle is used by one host thread and one
 * stream at a time (its workspace, about 8 bytes a value, 4 or 8 min(rows, cols)^2 bytes a
 * matrix and up to 34 MB of shared sums, is its own). */
typedef struct tgrad_muon tgrad_muon_t;

/* Floats of the momentum; -1 for invalid sizes. Host only. */
int64_t tgrad_muon_state_values(int n, const int64_t *count, const int64_t *rows, const int64_t *cols);

/*
 * Create a handle on the current HIP device for n >= 1 tensors (synchronises the device).
 *   count, rows, cols [n]   count >= 0, 1 <= rows, cols <= 2^19
 *   dtype[n]         TGRAD_F32, TGRAD_F16 or TGRAD_BF16 of the weights
 *   grad_dtype[n]    of the gradients: the weight's, or TGRAD_F32
 *   weight_decay[n], scale[n]   of each tensor, >= 0 and finite
 *   lr >= 0, finite;  momentum in [0, 1);  nesterov: 0 or 1
 *   steps, coefficients, eps    as above
 *   state            the buffer above; it must outlive the handle. Neither read nor written by
 *                    this call.
 * Errors: TGRAD_EINVAL (also more than some 2^21 parts of 8192 values or matrices),
 * TGRAD_ENOMEM, TGRAD_EHIP. *out is NULL on error.
 */
int tgrad_muon_init(tgrad_muon_t **out, int n, const int64_t *count, const int64_t *rows,
                    const int64_t *cols, const int *dtype, const int *grad_dtype,
                    const double *weight_decay, const double *scale, double lr, double momentum,
                    int nesterov, int steps, const double *coefficients, double eps, float *state);
/* Free the handle's own device memory (the momentum stays the caller's). The caller
 * synchronises first. NULL is a no-op. */
int tgrad_muon_destroy(tgrad_muon_t *h);
const char *tgrad_muon_last_error(const tgrad_muon_t *h);
/* The learning rate from the next step on (>= 0, finite); a captured step keeps its own. */
int tgrad_muon_set_lr(tgrad_muon_t *h, double lr);
/* One step: weights[i] (updated in place) and grads[i] (only read) are contiguous device
 * buffers, aligned to their elements (both may be NULL where count[i] is 0). No weight overlaps
 * another (TGRAD_EINVAL) or a gradient. clip: NULL, or two
 * device floats from tgrad_adamw_grad_norm; where the norm clip[0] is not finite the step is
 * left out on the device. Errors: TGRAD_EINVAL, TGRAD_EHIP. */
int tgrad_muon_step(tgrad_muon_t *h, void *const *weights, const void *const *grads,
                    const float *clip, void *stream);

/*
 * Gated linear layer over `rows` rows of `in` values, to `hidden` values, and its gradients:
 *   g = x w_gate^T + b_gate,  u = x w_up^T + b_up,  y = act(g) u
 *   dg = dy u act'(g),  du = dy act(g),  dx = dg w_gate + du w_up
 *   dw_gate = dg^T x,  dw_up = du^T x,  db = sums over rows of dg and du
 * act: silu (g / (1 + e^-g)), gelu (g times the normal distribution's probability up to g),
 * sigmoid or relu (with slope 0 at 0). Sums are fp32, y is rounded once. The gradients form g
 * and u again from x; 16-bit dg and du are rounded to that type between the products, and few of
 * them (up to 2^14 of each, or 2^19 for results of up to 2^10) carried in two such parts (db comes
 * from the values before). In fp16 that is its range too: a dg or du over 65504 is infinite in the
 * products, also where dx or dw would not be. fp32 products are made of six products of bf16 parts, as exact as
 * fp32 sums; a value that is not finite makes what it enters NaN there. Results do not depend
 * on the order in which workgroups run.
 *   x, dy           device, rows x_stride >= in (dy_stride >= hidden, <= 2^20) elements apart
 *   w_gate, w_up    device, contiguous, hidden rows of in values;  dw_gate, dw_up alike
 *   b_gate, b_up, db_gate, db_up   device, hidden values;  b: NULL: 0
 *   y, dx           device, contiguous; no result overlaps an input
 *   dx, the dw and the db may be NULL, the latter in pairs
 *   dtype           TGRAD_F32, TGRAD_F16 or TGRAD_BF16, of all of them
 *   workspace       device, tgrad_gated_linear_workspace bytes, 16-byte aligned (NULL for 0).
 *                   It may be reused once the stream's work is done.
 * The workspace's size is that of a call with the same x, strides and weights, whose alignment
 * matters (rows that are not 16-byte aligned or no multiple of 8 values are copied); backward: 0
 * or 1; -1 for invalid sizes. Host only.
 * rows = 0 is valid (the weights' gradients become 0). rows <= 2^31 - 65537, 1 <= in, hidden <=
 * 2^19, and the copies of a call hold at most 2^35 values (else TGRAD_EHIP). Every pointer is
 * aligned to its element. Errors: TGRAD_EINVAL, TGRAD_EHIP.
 */
enum tgrad_activation { TGRAD_SILU = 0, TGRAD_GELU = 1, TGRAD_SIGMOID = 2, TGRAD_RELU = 3 };
int64_t tgrad_gated_linear_workspace(const void *x, int64_t x_stride, const void *w_gate,
                                     const void *w_up, int64_t rows, int64_t in, int64_t hidden,
                                     int dtype, int backward);
int tgrad_gated_linear_forward(const void *x, int64_t x_stride, const void *w_gate,
                               const void *w_up, const void *b_gate, const void *b_up, void *y,
                               int64_t rows, int64_t in, int64_t hidden, int dtype,
                               int activation, void *workspace, void *stream);
int tgrad_gated_linear_backward(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride,
                                const void *w_gate, const void *w_up, const void *b_gate,
                                const void *b_up, void *dx, void *dw_gate, void *dw_up,
                                void *db_gate, void *db_up, int64_t rows, int64_t in,
                                int64_t hidden, int dtype, int activation, void *workspace,
                                void *stream);

#ifdef __cplusplus
}
#endif
#endif /* TGRAD_H */
