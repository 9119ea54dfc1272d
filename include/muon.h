/*
 * libmuon — the Muon optimizer step on one NVIDIA GB300 GPU (sm_103a), and
 * operators that bring a block's activations to the gradients it reads (last
 * section).
 *
 * One call, muon_step(), updates every registered 2-D weight matrix:
 *
 *   1. momentum      M <- beta*M + G ; U = G + beta*M (Nesterov) or U = M
 *   2. normalise     X0 = U / (||U||_F + 1e-7), oriented short side first
 *                    (a matrix with rows > cols is processed as U^T)
 *   3. orthogonalise ns_steps quintic Newton-Schulz iterations, three
 *                    products each: A = X X^T, B = b A + c A A, X <- a X + B X
 *   4. update        W <- W - lr * max(1, rows/cols)^0.5 * O, O = X (or X^T)
 *
 * Sources: "Advancing Emerging Optimizers for Accelerated LLM Training"
 * (NVIDIA developer blog, 22 Apr 2026, and its summaries).  Section
 * "Distributed Newton-Schulz": the optimizer needs each layer's whole
 * momentum-buffer matrix; section "Duplicated mode": the iteration runs
 * "usually five" times per update and the weights are then updated with the
 * orthogonalised momentum; section "Distributed mode": three matrix products
 * per iteration; section "SYRK and fused all-reduce": the first two products
 * are symmetric rank-k updates that compute only the upper-triangle tiles
 * (diagonal tiles in full) and write the full, mirrored matrix; section
 * "Blockwise mode": each locally held block is orthogonalised and updated on
 * its own, with no communication; section "Load balancing": matrices differ
 * in cost, so work is balanced by estimated cost rather than round-robin.
 * The momentum form, the normalisation, the orientation rule and the shape
 * scale are not written out on the pages; the library takes the plain
 * readings listed above.
 *
 * Conventions for every entry point
 *   - Return value: MUON_OK (0) or a negative MUON_ERR_* code.  The text of
 *     the last error of a handle is available from muon_last_error().
 *   - All argument checks run before any GPU work is queued, so a call that
 *     returns an error has changed no memory.
 *   - Pointers named "device" are CUDA device addresses on the handle's
 *     device; nothing is copied from or to the host unless stated.
 *   - GPU work is queued on the handle's stream and runs asynchronously;
 *     errors raised on the GPU surface at muon_sync().
 *   - Results are deterministic: the same inputs give bit-identical outputs
 *     from run to run, and a matrix gives the same bits whether it is stepped
 *     alone or together with others.
 *   - A handle is not thread-safe; use one handle per host thread.
 */
#ifndef LIBMUON_MUON_H
#define LIBMUON_MUON_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define MUON_API __attribute__((visibility("default")))
#else
#define MUON_API
#endif

/* error codes */
#define MUON_OK                    0
#define MUON_ERR_INVALID_ARG      -1  /* null pointer, bad size, bad enum   */
#define MUON_ERR_UNSUPPORTED      -2  /* shape or dtype the library rejects */
#define MUON_ERR_NO_WORKSPACE     -3  /* no workspace, or too small         */
#define MUON_ERR_CUDA             -4  /* a CUDA runtime/driver call failed  */
#define MUON_ERR_TIMEOUT          -5  /* a bounded wait on the GPU ran out  */
#define MUON_ERR_STATE            -6  /* call out of order (e.g. no params) */

/* element types */
#define MUON_F32   0
#define MUON_BF16  1

/* orthogonalisation modes */
#define MUON_FULL       0   /* each registered matrix as a whole            */
#define MUON_BLOCKWISE  1   /* nb equal column blocks, each on its own      */
/* Distributed mode ("Advancing Emerging Optimizers for Accelerated LLM
 * Training", section "Distributed mode"): the iteration as a tensor-parallel
 * group of nb ranks runs it, each rank holding an equal contiguous slice of
 * the iterate's long side n.  The first product of every iteration is the
 * sum of the slices' partial products (the all-reduce), added in fp32 in
 * slice order 0, 1, ..., nb-1; the other two products are as in full mode.
 * One GPU computes all slices.  nb must divide every n with n / nb a
 * multiple of 64 (MUON_ERR_UNSUPPORTED otherwise); nb = 1 is full mode. */
#define MUON_DISTRIBUTED 2

typedef struct muon_ctx* muon_handle;

/* One 2-D parameter.  w, g and m are device pointers to row-major matrices
 * of rows x cols elements with leading dimensions ld_w, ld_g, ld_m (in
 * elements, >= cols).  w is updated in place (w_dtype: MUON_BF16 or
 * MUON_F32), g is read only (g_dtype: MUON_BF16 or MUON_F32), m is the fp32
 * momentum buffer, updated in place.  The caller owns all three and keeps
 * them valid while they are registered.  1 <= rows, cols <= 1048576 and
 * min(rows, cols) <= 32768 (the m x m intermediates stay addressable). */
typedef struct {
    void*       w;
    const void* g;
    float*      m;
    int64_t     rows, cols;
    int64_t     ld_w, ld_g, ld_m;
    int32_t     w_dtype, g_dtype;
} muon_param;

/* Creates a handle bound to CUDA device `device` and stream `cuda_stream`
 * (a cudaStream_t; NULL = the legacy default stream).  Allocates no device
 * memory.  *out receives the handle.  device = MUON_HOST_ONLY gives a handle
 * that makes no CUDA call at all: it registers parameters (pointers are not
 * dereferenced) and answers muon_workspace_size / muon_get_plan_info, while
 * muon_step and muon_sync return MUON_ERR_STATE. */
#define MUON_HOST_ONLY (-1)
MUON_API int muon_create(muon_handle* out, int device, void* cuda_stream);

/* Replaces the stream that later calls queue their work on. */
MUON_API int muon_set_stream(muon_handle h, void* cuda_stream);

/* Registers n >= 1 parameters (copied; the array may be freed afterwards),
 * replacing any previous set.  Invalidates the current plan. */
MUON_API int muon_register_params(muon_handle h, int n, const muon_param* params);

/* Workspace the step needs for `mode` / `nb` with the registered set.
 * *min_bytes: enough to run the step one group of matrices at a time
 * (the largest single matrix or block plus the plan's tables);
 * *full_bytes: enough to run every matrix in a single group.  Any size in
 * between works; larger sizes give fewer, larger groups.  In blockwise mode
 * nb must divide every registered cols, in distributed mode every long side
 * (see MUON_DISTRIBUTED); MUON_ERR_UNSUPPORTED otherwise. */
MUON_API int muon_workspace_size(muon_handle h, int mode, int nb, size_t* min_bytes,
                        size_t* full_bytes);

/* Hands the library a caller-owned device buffer of `bytes` bytes (start
 * aligned to 1024 bytes) to hold the plan's tables and all intermediate
 * matrices.  The library never allocates device memory itself.  The buffer
 * must stay valid until replaced or the handle is destroyed. */
MUON_API int muon_set_workspace(muon_handle h, void* dptr, size_t bytes);

/* One Muon step over all registered parameters.
 *   lr, beta, nesterov   learning rate, momentum factor, Nesterov on/off
 *   ns_steps             Newton-Schulz iterations (1..64; 5 is usual)
 *   a, b, c              coefficients of a X + (b A + c A A) X
 *   mode, nb             MUON_FULL (nb ignored), MUON_BLOCKWISE with nb
 *                        column blocks (nb >= 1 dividing every cols), or
 *                        MUON_DISTRIBUTED with nb tensor-parallel slices
 * The first step after registering params, changing the workspace, the mode
 * or nb builds the plan and uploads its tables (host work plus one copy);
 * later steps only queue kernels.  Returns once the work is queued.
 * A step carries no device state from earlier steps beyond W and M, so a
 * step queued while the handle's stream is being captured into a CUDA graph
 * replays correctly; the plan must exist before the capture (run one step
 * outside it first: MUON_ERR_STATE otherwise), and stage profiling must be
 * off during the capture. */
MUON_API int muon_step(muon_handle h, float lr, float beta, int nesterov, int ns_steps,
              float a, float b, float c, int mode, int nb);

/* The same step with the gradients taken from, and the updated weights
 * returned to, host memory.  n must equal the number of registered
 * parameters.  g_host[i] holds parameter i's gradient (rows x cols, row-major,
 * leading dimension cols, element type g_dtype); it is copied into the
 * registered device g before the step.  After the step the updated weight
 * (element type w_dtype) is copied to w_host[i] (rows x cols, leading
 * dimension cols); a NULL w_host[i] skips that copy.  Everything is queued on
 * the handle's stream and the call returns once it is queued: host buffers
 * must stay valid, and unchanged, until muon_sync returns, and should be
 * pinned (page-locked) for the copies to run asynchronously.  The caller
 * owns them.  Errors as muon_step; a failed copy is MUON_ERR_CUDA.
 * The copies overlap the compute: the step runs in groups of whole matrices
 * (about 1/16 of the registered elements each, at least 32 M elements), a
 * group's gradients are copied in on a second stream while earlier groups
 * compute, and its weights go out on a third stream once its update is
 * done; the handle's stream waits for all of them.  The first call builds
 * that grouping (later muon_step calls reuse it; results are the same bits
 * with any grouping). */
MUON_API int muon_step_host(muon_handle h, int n, const void* const* g_host,
                            void* const* w_host, float lr, float beta, int nesterov,
                            int ns_steps, float a, float b, float c, int mode, int nb);

/* Waits for the handle's stream and reports any error raised on the GPU
 * (MUON_ERR_TIMEOUT when a bounded wait ran out, MUON_ERR_CUDA otherwise). */
MUON_API int muon_sync(muon_handle h);

/* Releases the handle (no device memory is owned, none is freed). */
MUON_API int muon_destroy(muon_handle h);

/* Text of the handle's last error ("" if none).  Valid until the next call
 * on the handle.  h may be NULL (returns the last create error). */
MUON_API const char* muon_last_error(muon_handle h);

/* ---- measurement and validation helpers ------------------------------- */

/* Stage timing.  When on, muon_step records CUDA events around each kind of
 * launch on the handle's stream; muon_stage_times() (after muon_sync) fills
 * up to `n` totals in milliseconds for the last step, in the order
 * momentum, norm, normalise, syrk1, syrk2, gemm, update, chain (one launch
 * with every product of the step but the last X update), and the number
 * of launches of each kind into `launches` (may be NULL).  Returns the
 * number of stages written. */
#define MUON_N_STAGES 8
MUON_API int muon_set_profiling(muon_handle h, int on);
MUON_API int muon_stage_times(muon_handle h, float* ms, int* launches, int n);

/* Number of kernel launches the last muon_step queued. */
MUON_API int muon_last_launch_count(muon_handle h);

/* Optional exports written by the update stage of every later step, for
 * parameter i (0 <= i < n): w_f32[i] receives the updated weight in fp32
 * before it is stored in the weight's dtype, o_bf16[i] the orthogonalised
 * update O in bf16; both rows x cols row-major with leading dimension cols,
 * in the weight's orientation.  Entries (or whole arrays) may be NULL.
 * n = 0 turns exports off.  Changing exports rebuilds the plan. */
MUON_API int muon_debug_set_exports(muon_handle h, int n, float* const* w_f32,
                           void* const* o_bf16);

/* Failure-path check of the kernels' bounded waits: launches one block that
 * waits on a barrier nothing arrives at, with a limit of `limit_ms`
 * (1..10000) milliseconds, and reads the device error word `err_word` (a
 * caller-owned device int).  Returns MUON_ERR_TIMEOUT when the wait ran out
 * and reported it as the tensor-core kernels do (the expected outcome); the
 * CUDA context stays usable.  Makes no other change. */
MUON_API int muon_debug_wait_timeout(muon_handle h, int* err_word, int limit_ms);

/* Validation of the chained launch (see muon_get_plan_info: groups of few
 * large matrices run every product of a step in one launch whose tiles wait
 * on per-tile counters; the launch's last CTA zeroes them as it leaves).
 * skew_rounds > 0 makes the second products of later chained launches wait
 * for that many counter rounds more than will ever be completed, so their
 * bounded waits run out and muon_sync reports MUON_ERR_TIMEOUT (a timeout
 * test without a fault; 0 = off).  Applies to later steps of this handle;
 * MUON_ERR_INVALID_ARG for values out of range. */
MUON_API int muon_debug_set_chain_test(muon_handle h, int skew_rounds);

/* Host-only check of the chained launch's schedule for `mode`/`nb`: for every
 * group of the registered matrices (ignoring the size bounds that decide
 * whether a group chains), builds the per-pair tile lists and checks that
 * every tile appears once, that each pair's list is in stage order (first
 * products, second products, X updates: the order that keeps every wait on
 * tiles of earlier stages) and that the pair offsets and last-iteration ends
 * are consistent.  No CUDA call; works on MUON_HOST_ONLY handles.  Returns
 * MUON_OK, or MUON_ERR_STATE with the violated property in
 * muon_last_error. */
MUON_API int muon_debug_check_chain_schedule(muon_handle h, int mode, int nb);

/* Plan statistics for `mode`/`nb`: number of units (matrices or blocks),
 * groups, and tiles of the symmetric-product and GEMM stages. */
typedef struct {
    int64_t units, groups, syrk_tiles, gemm_tiles, ew_tiles;
    /* per Newton-Schulz iteration, all units: useful = upper-triangle
     * symmetric products + the GEMM; executed = what the tiles compute */
    int64_t useful_flops, executed_flops;
    /* groups whose products run as one chained launch per step (every
     * product but the last X update; groups of few large matrices) */
    int64_t chained_groups;
} muon_plan_info;
MUON_API int muon_get_plan_info(muon_handle h, int mode, int nb, muon_plan_info* out);

/* ---- distributed mode across ranks ------------------------------------- */

/* "Advancing Emerging Optimizers for Accelerated LLM Training", section
 * "Distributed mode": the iterate X (m x n, short side first) of one matrix
 * is split along n over the P ranks of a tensor-parallel group, one GPU
 * each.  A rank holds its slice of W, G and M and runs the step in phases;
 * between the phases the caller sums across the group (an all-reduce, e.g.
 * torch.distributed over NCCL).  Per iteration the only exchange is the sum
 * of the partial products X_r X_r^T (the all-reduce after the first matrix
 * product), plus one sum of squares for the norm before the first:
 *
 *   muon_dist_momentum(h, ...)        momentum on the slice; the slice's
 *                                     sum of squares of U -> sumsq
 *   [sum sumsq over the group]
 *   for s = 0 .. ns_steps - 1:
 *     muon_dist_gram(h, ...)          the partial X_r X_r^T -> A (fp32)
 *     [sum A over the group]
 *     muon_dist_update(h, ...)        B' = b A + c A A + a I from the sum,
 *                                     X_r <- B' X_r; on the last iteration
 *                                     W_r <- W_r - lr * scale * O_r
 *
 * The handle must hold exactly one registered parameter, the rank's slice,
 * and must have been configured with muon_dist_configure first; the phases
 * use its workspace (muon_workspace_size with MUON_FULL).  Phases are queued
 * on the handle's stream in the order above; errors as for muon_step, and
 * MUON_ERR_STATE for a phase out of order.  The weight update of the last
 * iteration is folded into the X update as in muon_step. */

/* The slice's place in the whole matrix: transposed = 1 if the whole weight
 * is tall (rows > cols; its iterate is W^T, and the slice is a block of W's
 * rows), 0 otherwise (the slice is a block of W's columns); shape_scale =
 * the whole matrix's max(1, rows / cols) ** 0.5.  The slice's short side must
 * then be the whole matrix's short side: its iterate is m x n_r with
 * m = cols (transposed) or rows.  Invalidates the plan. */
MUON_API int muon_dist_configure(muon_handle h, int transposed, float shape_scale);

/* M <- beta M + G and U on the slice; the iterate slice X_r = bf16(U), not
 * yet normalised.  *sumsq (device memory, one double) receives the slice's
 * sum of U^2, taken per 64 x 64 tile and then over the tiles in a fixed
 * order, so that the sum of all slices' values is ||U||_F^2. */
MUON_API int muon_dist_momentum(muon_handle h, float beta, int nesterov, double* sumsq);

/* Iteration s's partial product A_r = X_r X_r^T of the slice, unscaled fp32,
 * into the m x m row-major device buffer a (leading dimension lda >= m),
 * for the 256 x 256 tiles (ti, tj) with ti <= tj and band_begin <= ti <
 * band_end (256-row blocks; band_end = -1: to the last).  Nothing else of a
 * is written: the caller zeroes it once, so that the tiles below the
 * diagonal stay zero, and may sum the bands as each is queued (the
 * "SYRK and fused all-reduce" exchange of finished upper tiles). */
MUON_API int muon_dist_gram(muon_handle h, float* a, int64_t lda, int band_begin,
                            int band_end);

/* The rest of iteration s from the group's sum of the partial products in
 * a (fp32, upper tiles as written by muon_dist_gram): A = bf16(sum * scale)
 * with scale = 1 / (||U||_F + eps)^2 when first (sumsq_total: device double,
 * the group's sum of the momentum phase's values; ignored otherwise), then
 * B' = b A + c A A + a I and X_r <- B' X_r (times 1 / (||U||_F + eps) when
 * first).  When last, the update O_r = X_r (transposed back) is applied:
 * W_r <- W_r - lr * shape_scale * O_r. */
MUON_API int muon_dist_update(muon_handle h, const float* a, int64_t lda, int first, int last,
                              const double* sumsq_total, float lr, float ca, float cb, float cc);

/* ---- step without a workspace ------------------------------------------ */

/* One Muon step (full mode) on ONE matrix without any workspace: the plan
 * tables and every intermediate (partial sums, the two iterates X, and A, B)
 * live in a fixed 32 MiB array inside the library.  This is for callers who
 * cannot call cudaMalloc or hand over a buffer: a plugin whose host owns all
 * device memory through a pool it does not expose, a process whose caching
 * allocator has already reserved the GPU, or a hot loop that cannot afford
 * cudaMalloc's implicit device synchronisation.  The paper has no
 * counterpart of this entry point; it is a convenience of this library.
 *
 *   param          one matrix as for muon_register_params (device pointers;
 *                  W and M updated in place, G read only)
 *   lr ... c       as for muon_step
 *   cuda_stream    stream for the work (NULL = legacy default stream); the
 *                  CUDA device is the caller's current device
 *   err, err_len   optional buffer that receives a message on error
 *
 * Limits and behaviour:
 *   - The matrix must fit the fixed array: roughly 4 bytes per element of
 *     the matrix plus 4 bytes per element of its m x m square (m = short
 *     side), plus small tables, at most 33554432 bytes in total (a 1024 x
 *     4096 matrix fits, a 2048 x 2048 does not).  Larger matrices are
 *     rejected with MUON_ERR_UNSUPPORTED and a message before any GPU work.
 *   - The array exists once per device that loads this code and is held
 *     until the process exits.  The first call on a device is its set-up:
 *     it resolves the array's address (cudaGetSymbolAddress) with that
 *     device current, so make that first call before any stream capture.
 *     The address is resolved again only if the device's context has been
 *     replaced since (for example after cudaDeviceReset).
 *   - Every call reuses the same array and overwrites what the previous
 *     call left there; calls whose GPU work overlaps (different streams or
 *     threads) race and give wrong results.  Queue them on one stream.
 *   - No cudaMalloc, cudaFree or other allocating call is made.  The work is
 *     queued asynchronously; a bounded GPU wait that runs out makes the
 *     kernels return early, which this entry point cannot report (use the
 *     handle-based muon_step and muon_sync where that report matters). */
MUON_API int muon_step_noalloc(const muon_param* param, float lr, float beta,
                               int nesterov, int ns_steps, float a, float b,
                               float c, void* cuda_stream, char* err,
                               size_t err_len);

/* ---- operators of a block's training step ------------------------------ */

/* What a block of a model runs between its activations and the gradients
 * that muon_step reads: layer norm, activation checkpoints in 8 bits, the
 * weight gradient taken from a checkpoint, the router of a
 * mixture-of-experts block with its balance loss, the gated feed-forward block
 * (dense or per expert), rotary positions and dropout.  These entry points
 * need no handle.  Conventions, beside those at the top of this file:
 *   - The work is queued on cuda_stream (NULL = the legacy default stream)
 *     of the caller's current device.  Every device pointer, the workspace's
 *     included, must stay valid until that work is done.
 *   - err, err_len: optional buffer that receives a message on error.
 *   - Argument checks run before any CUDA call.
 *   - A workspace is device memory, 256-byte aligned, of the size that the
 *     operator's _workspace call gives for the same arguments (that call
 *     makes no CUDA call and looks behind no pointer).  Its contents before
 *     and after the call mean nothing.
 *   - Leading dimensions are in elements.  One of a tensor that is only read
 *     may be 0 (one row for all); every other is at least the row's length
 *     (rows <= 1: anything).  No alignment is asked for beyond the element's
 *     own unless stated; rows that start on 16 bytes are faster.
 *   - Sums are held in fp32 and in a fixed order: the same call gives the
 *     same bits again. */

/* An activation checkpoint: rows x cols values in 8 bits, in blocks of 32
 * consecutive values of a row that share a power of two.  A value stands for
 *     q[r * ld_q + c] * 2^(e[r * ld_e + c / 32] - 133),
 * q in -127 .. 127; e = 127 + floor(log2(largest magnitude of the block)),
 * 0 for a block whose magnitudes are all below 2^-126, 255 for a block that
 * held an infinity or a NaN (all of its values read as NaN).  Values are
 * rounded to nearest, ties to even, and limited to 127; each is exact in
 * bf16.  Device pointers: q 16-byte aligned with ld_q a multiple of 32 and
 * at least cols rounded up to 32 (the values past cols are written as zero),
 * ld_e at least ceil(cols / 32).  q = NULL where a checkpoint is optional
 * means none. */
typedef struct {
    int8_t*  q;
    uint8_t* e;
    int64_t  ld_q, ld_e;
} muon_ckpt8;

/* Writes the checkpoint of x (rows x cols, x_dtype), and the values of a
 * checkpoint to x.  0 <= rows < 2^31, 1 <= cols <= 1048576. */
MUON_API int muon_ckpt8_pack(const void* x, int x_dtype, int64_t rows, int64_t cols,
                             int64_t ld_x, const muon_ckpt8* saved, void* cuda_stream,
                             char* err, size_t err_len);
MUON_API int muon_ckpt8_unpack(const muon_ckpt8* saved, int64_t rows, int64_t cols, void* x,
                               int x_dtype, int64_t ld_x, void* cuda_stream, char* err,
                               size_t err_len);

/* Layer norm over the rows of x:
 *     h = (x - mean) * rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps),
 *     y = h * weight + bias.
 * x and y: rows x cols of x_dtype (y may be x); weight, bias: cols values of
 * w_dtype, NULL for ones and zeros; mean, rstd: rows fp32 values, either may
 * be NULL.  saved (optional): receives the checkpoint of h.
 * 0 <= rows < 2^31, 1 <= cols <= 1048576, eps >= 0. */
typedef struct {
    const void* x;
    const void* weight;
    const void* bias;
    void*       y;
    float*      mean;
    float*      rstd;
    muon_ckpt8  saved;
    int64_t     rows, cols;
    int64_t     ld_x, ld_y;
    int32_t     x_dtype, w_dtype;
    float       eps;
} muon_layer_norm_args;
MUON_API int muon_layer_norm(const muon_layer_norm_args* args, void* cuda_stream, char* err,
                             size_t err_len);

/* Its gradient.  With g = dy * weight:
 *     dx = rstd * (g - mean(g) - h * mean(g * h)),
 *     dweight = sum over rows of dy * h,  dbias = sum over rows of dy.
 * h comes from saved (the checkpoint the forward pass wrote; x and mean are
 * then NULL), or from x and mean.  dy, x and dx: rows x cols of x_dtype (dx
 * may be dy); weight: w_dtype or NULL; dweight, dbias: cols values of
 * w_dtype, either may be NULL.  rows = 0 gives zero dweight and dbias. */
typedef struct {
    const void*  dy;
    const void*  x;
    const float* mean;
    const float* rstd;
    const void*  weight;
    void*        dx;
    void*        dweight;
    void*        dbias;
    muon_ckpt8   saved;
    int64_t      rows, cols;
    int64_t      ld_dy, ld_x, ld_dx;
    int32_t      x_dtype, w_dtype;
} muon_layer_norm_grad_args;
MUON_API int muon_layer_norm_grad_workspace(const muon_layer_norm_grad_args* args,
                                            size_t* bytes);
MUON_API int muon_layer_norm_grad(const muon_layer_norm_grad_args* args, void* workspace,
                                  size_t bytes, void* cuda_stream, char* err, size_t err_len);

/* The gradient of a matrix W (n x k) of a product Y = X W^T, from the
 * checkpoint of X (or of the h that a norm made X from):
 *     G[i][j] = sum over t of dy[t][i] * (h[t][j] * weight[j] + bias[j])  (+ C[i][j])
 * dy: rows x n, bf16; saved: rows x k; weight, bias: k values of w_dtype, NULL
 * for ones and zeros; g: n x k of g_dtype; c (optional): n x k of g_dtype, may
 * be g itself (gradient accumulation).  The products run on the tensor cores
 * from exact bf16 operands with fp32 sums; weight and bias are applied to
 * the sums.  The tensor cores cut their running sums off at the last place
 * (sums of one sign lose 9e-7 in 1024 tokens and 4e-5 in 16384): fp32 results
 * add them up to nearest every 1024 tokens, bf16 ones every 16384.
 * offsets (optional): experts + 1 int32 values in device memory, rising from
 * 0 to at most rows: matrix e takes rows offsets[e] .. offsets[e + 1] of dy
 * and saved (none: G = 0, or C), and g and c are `experts` matrices, stride_g
 * and stride_c elements apart.  Values outside that rule are limited to it.
 * offsets = NULL: experts = 1, all rows.  0 <= rows < 2^31, 1 <= n, k <=
 * 1048576, 1 <= experts <= 65536. */
typedef struct {
    const void*    dy;
    const void*    weight;
    const void*    bias;
    const void*    c;
    void*          g;
    const int32_t* offsets;
    muon_ckpt8     saved;
    int64_t        rows, n, k, experts;
    int64_t        ld_dy, ld_c, ld_g, stride_c, stride_g;
    int32_t        g_dtype, w_dtype;
} muon_weight_grad_args;
MUON_API int muon_weight_grad_workspace(const muon_weight_grad_args* args, size_t* bytes);
MUON_API int muon_weight_grad(const muon_weight_grad_args* args, void* workspace, size_t bytes,
                              void* cuda_stream, char* err, size_t err_len);

/* The router of a mixture-of-experts block.  p = softmax(logits) over the
 * experts of every token; the k experts with the largest logits are taken
 * (equal ones: the lower index first; one at -infinity never):
 *     weights = p of those taken, divided by their sum if renormalise,
 *     counts[e] = tokens that took expert e, offsets = their running sum,
 *     loss = coef * experts / (k * kept^2) * sum over e of counts[e] * sum over t of p[t][e],
 * where kept is the number of tokens that take part: those with mask != 0
 * (mask NULL: all) and a logit above -infinity.  The others get indices -1
 * and weights 0 and count nowhere; so do a token's places past its last
 * logit above -infinity.  No token left: loss 0.  A NaN counts as the largest
 * logit and makes its token's weights, and the loss, NaN.
 * logits: tokens x experts of z_dtype; mask: one byte a token; indices,
 * weights: tokens x k, dense; counts: experts; offsets: experts + 1; loss,
 * kept: one value.  0 <= tokens, tokens * k < 2^31, 1 <= experts <= 1024,
 * 1 <= k <= min(experts, 32). */
typedef struct {
    const void*    logits;
    const uint8_t* mask;
    int32_t*       indices;
    float*         weights;
    int32_t*       counts;
    int32_t*       offsets;
    float*         loss;
    int32_t*       kept;
    int64_t        tokens, experts, k;
    int64_t        ld_z;
    int32_t        z_dtype, renormalise;
    float          coef;
} muon_route_args;
MUON_API int muon_route_workspace(const muon_route_args* args, size_t* bytes);
MUON_API int muon_route(const muon_route_args* args, void* workspace, size_t bytes,
                        void* cuda_stream, char* err, size_t err_len);

/* Its gradient with respect to the logits, from the indices, weights, counts
 * and kept that muon_route wrote (counts are constants of the loss), dloss
 * (one fp32 value, NULL for 0) and dweights (tokens x k fp32, NULL for 0).
 * dlogits: tokens x experts of z_dtype (may be logits); zero where a token
 * takes no part. */
typedef struct {
    const void*    logits;
    const int32_t* indices;
    const float*   weights;
    const int32_t* counts;
    const int32_t* kept;
    const float*   dloss;
    const float*   dweights;
    void*          dlogits;
    int64_t        tokens, experts, k;
    int64_t        ld_z, ld_dw, ld_dz;
    int32_t        z_dtype, renormalise;
    float          coef;
} muon_route_grad_args;
MUON_API int muon_route_grad(const muon_route_grad_args* args, void* cuda_stream, char* err,
                             size_t err_len);

/* A gated feed-forward block, dense or one per expert:
 *     g = x w_gate^T,  u = x w_up^T,  h = act(g) * u,  y = h w_down^T.
 * Both first products, act and their product are one kernel.  bf16 tensors:
 * x, y: rows x hidden; w_gate, w_up: inner x hidden; w_down: hidden x inner;
 * gate, up (both or neither, rows x inner, leading dimension ld_kept): receive
 * g and u for the backward pass.  Sums are fp32 in the tensor cores; g, u, h
 * and y are each rounded once, from fp32.
 * act: MUON_ACT_SILU g / (1 + e^-g), MUON_ACT_GELU g Phi(g),
 * MUON_ACT_GELU_TANH its approximation by tanh(sqrt(2/pi) (g + 0.044715 g^3)).
 * offsets (optional): experts + 1 int32 values in device memory, rising from
 * 0 to at most rows: expert e has rows offsets[e] .. offsets[e + 1] and the
 * matrices e, stride_gate, stride_up and stride_down elements apart.  Values
 * outside that rule are limited to it (one below another before it counts as
 * that one); rows of no expert are not written.
 * offsets = NULL: experts = 1, all rows.  y may be x or share memory with it; else no
 * output may share memory with another or with what is read (MUON_ERR_INVALID_ARG;
 * views that interleave, such as columns of one matrix, may).  The tensor cores cut
 * their running sums off at the last place (16384 terms of one sign lose 9e-5 of their
 * sum at most, and others in proportion); long sums of few rows are added up in parts,
 * so that a row's last bits may depend on the number of rows.
 * A stride of matrices may be 0 (one for all).  Operands whose rows do not all
 * start on 16 bytes are copied to the workspace first.  0 <= rows < 2^31 - 256,
 * 1 <= hidden, inner <= 262144, 1 <= experts <= 1024. */
#define MUON_ACT_SILU 0
#define MUON_ACT_GELU 1
#define MUON_ACT_GELU_TANH 2
typedef struct {
    const void*    x;
    const void*    w_gate;
    const void*    w_up;
    const void*    w_down;
    void*          y;
    void*          gate;
    void*          up;
    const int32_t* offsets;
    int64_t        rows, hidden, inner, experts;
    int64_t        ld_x, ld_gate, ld_up, ld_down, ld_y, ld_kept;
    int64_t        stride_gate, stride_up, stride_down;
    int32_t        activation;
} muon_gated_ffn_args;
MUON_API int muon_gated_ffn_workspace(const muon_gated_ffn_args* args, size_t* bytes);
MUON_API int muon_gated_ffn(const muon_gated_ffn_args* args, void* workspace, size_t bytes,
                            void* cuda_stream, char* err, size_t err_len);

/* Its gradient.  From gate and up as the forward pass kept them:
 *     dh = dy w_down,  dgate = dh * u * act'(g),  dup = dh * act(g),  h = act(g) * u
 * (one kernel; rounded to bf16, as the next products read them),
 *     dx = dgate w_gate + dup w_up   (one sum),
 *     dw_gate = dgate^T x,  dw_up = dup^T x,  dw_down = dy^T h.
 * dy, x, dx: rows x hidden; gate, up: rows x inner.  Every output may be NULL:
 * dx; dw_gate and dw_up (then x may be, too); dw_down; dgate, dup and h (bf16,
 * rows x inner, leading dimension ld_d), which muon_weight_grad takes with a
 * checkpoint of x.  The weight gradients are g_dtype, dense matrices laid out
 * as their weights (leading dimensions ld_dgate ..., strides stride_dgate ...);
 * with accumulate they are added to what is there, in fp32, and rounded once.
 * Their sums over tokens are added up to nearest every 8192 tokens (bf16) or
 * 4096 (fp32) at most; dh's over hidden and dx's over 2 * inner terms are cut off as
 * the forward pass's are (dx of the widest inner, 262144: 2.9e-3 of a sum of one
 * sign at most).  An expert without rows has zero gradients.  No output
 * may share memory with another or with what is read while or after it is
 * written: dx with dy only without dw_down, and with x only without dw_gate and
 * dw_up; dgate, dup and h may be gate or up, with their leading dimension.
 * offsets as above. */
typedef struct {
    const void*    dy;
    const void*    x;
    const void*    gate;
    const void*    up;
    const void*    w_gate;
    const void*    w_up;
    const void*    w_down;
    void*          dx;
    void*          dw_gate;
    void*          dw_up;
    void*          dw_down;
    void*          dgate;
    void*          dup;
    void*          h;
    const int32_t* offsets;
    int64_t        rows, hidden, inner, experts;
    int64_t        ld_dy, ld_x, ld_kept, ld_gate, ld_up, ld_down, ld_dx, ld_d;
    int64_t        ld_dw_gate, ld_dw_up, ld_dw_down;
    int64_t        stride_gate, stride_up, stride_down;
    int64_t        stride_dw_gate, stride_dw_up, stride_dw_down;
    int32_t        activation, g_dtype, accumulate;
} muon_gated_ffn_grad_args;
MUON_API int muon_gated_ffn_grad_workspace(const muon_gated_ffn_grad_args* args, size_t* bytes);
MUON_API int muon_gated_ffn_grad(const muon_gated_ffn_grad_args* args, void* workspace, size_t bytes,
                                 void* cuda_stream, char* err, size_t err_len);

/* Rotary positions of queries and keys.  Pair i of a head (values i and
 * pairs + i with MUON_ROTARY_HALF, 2 i and 2 i + 1 with
 * MUON_ROTARY_INTERLEAVED) turns by a = position * frequency[i]:
 *     y1 = scale (x1 cos a - x2 sin a),  y2 = scale (x2 cos a + x1 sin a);
 * with inverse by -a, which makes the gradient of x from that of y.  The
 * values of a head past 2 * pairs are copied (they stay where y is x).
 * q, k: tensors of batch x seq x heads x head values of x_dtype, each value
 * 1 element and batches, positions and heads the given strides apart; a
 * tensor of 0 heads is left out.  y may be x, with its strides; else no result may
 * share memory with another, with an input or with itself.
 * positions: batch rows (stride_positions apart, 0 for one row) of seq values, 32-
 * or 64-bit (positions_64), in device memory; NULL: 0, 1, ... seq - 1.  offset
 * is added to each, modulo 2^64.  turns: host memory, read during the call: every pair's
 * frequency in turns per position times 2^64 (muon_rotary_frequencies), so
 * that position * turns modulo 2^64 is the angle without whole turns, good to
 * what turns is: 2^-50 of the whole angle and 2^-64 turns a position.
 * 0 <= batch * seq < 2^31, 1 <= pairs <= 256, 2 * pairs <= head <= 65536, 0 <=
 * heads <= 65536 each, a position's values of both at most 2^28. */
#define MUON_ROTARY_HALF 0
#define MUON_ROTARY_INTERLEAVED 1
typedef struct {
    const void* x;
    void*       y;
    int64_t     heads;
    int64_t     x_batch, x_seq, x_head;
    int64_t     y_batch, y_seq, y_head;
} muon_rotary_tensor;
typedef struct {
    muon_rotary_tensor q, k;
    const void*     positions;
    const uint64_t* turns;
    int64_t         batch, seq, head, pairs;
    int64_t         stride_positions, offset;
    int32_t         x_dtype, layout, positions_64, inverse;
    float           scale;
} muon_rotary_args;
MUON_API int muon_rotary(const muon_rotary_args* args, void* cuda_stream, char* err, size_t err_len);

/* The frequencies of `pairs` pairs and the scale, for muon_rotary (host only).
 * frequency[i] = base^(-i / pairs) radians a position, and
 *   MUON_ROTARY_LINEAR: divided by factor;
 *   MUON_ROTARY_NTK: base times factor^(pairs / (pairs - 1)) (pairs > 1);
 *   MUON_ROTARY_YARN ("YaRN: Efficient Context Window Extension of Large
 *     Language Models", Peng, Quesnelle, Fan and Shippole, 2023): divided by
 *     factor for pairs that turn less than slow times in the `original`
 *     positions, unchanged above fast times, a linear ramp over the pairs
 *     between; scale = 0.1 ln(factor) + 1.
 * base > 1, factor >= 1; for yarn original >= 1 and 0 < slow < fast. */
#define MUON_ROTARY_PLAIN 0
#define MUON_ROTARY_LINEAR 1
#define MUON_ROTARY_NTK 2
#define MUON_ROTARY_YARN 3
MUON_API int muon_rotary_frequencies(int64_t pairs, double base, int scaling, double factor,
                                     double original, double fast, double slow, uint64_t* turns,
                                     float* scale, char* err, size_t err_len);

/* Dropout:  y = keep * x / (1 - p)  (+ residual),  keep made again wherever it
 * is needed: the backward pass is the same call on dy without the residual.
 * Element i = row * cols + col is dropped where number i % 8 of block i / 8 is
 * below round(65536 p), so that p is taken to the nearest 2^-16 and 1 / (1 - p)
 * is that of this p.  Block b: Philox4x32-10 ("Parallel random numbers: as easy
 * as 1, 2, 3", Salmon, Moraes, Dror and Shaw, 2011) of the counter words b, b >>
 * 32, o, o >> 32 under the key words seed, seed >> 32, o = offset + *counter
 * modulo 2^64; its four words are eight 16-bit numbers, low halves first.
 * counter (optional): one value in device memory, read when the kernel runs,
 * so that a captured graph drops others in every replay.  A dropped element
 * is 0 whatever x holds.  x, residual, y: rows x cols of x_dtype; y may be x or
 * the residual, with its leading dimension, and else shares no memory with them.  0 <= rows < 2^31, 1 <= cols <= 1048576, 0 <= p <= 1. */
typedef struct {
    const void*    x;
    const void*    residual;
    void*          y;
    const int64_t* counter;
    int64_t        rows, cols;
    int64_t        ld_x, ld_r, ld_y;
    uint64_t       seed, offset;
    double         p;
    int32_t        x_dtype;
} muon_dropout_args;
MUON_API int muon_dropout(const muon_dropout_args* args, void* cuda_stream, char* err, size_t err_len);

/* Waits for the stream and reports what the operators above met on the GPU
 * of the caller's current device: MUON_ERR_TIMEOUT if a bounded wait of
 * one of their kernels ran out since the last call (its output is then not
 * whole), MUON_ERR_CUDA for a CUDA error, else MUON_OK. */
MUON_API int muon_ops_sync(void* cuda_stream, char* err, size_t err_len);

/* Failure test only: queues a wait of the operators' kind that nothing
 * satisfies.  It runs out after limit_ms (1 .. 10000) and raises what
 * muon_ops_sync then reports as MUON_ERR_TIMEOUT. */
MUON_API int muon_debug_ops_wait_timeout(int limit_ms, void* cuda_stream, char* err,
                                         size_t err_len);
/* The same for the gated feed-forward kernels, which have an error word of
 * their own. */
MUON_API int muon_debug_ffn_wait_timeout(int limit_ms, void* cuda_stream, char* err,
                                         size_t err_len);

#ifdef __cplusplus
}
#endif
#endif /* LIBMUON_MUON_H */
