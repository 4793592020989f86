/*
 * mhc.h -- C ABI of the GB300 (sm_103a) mHC layer library (libmhc_gb300.so).
 *
 * The layer is the manifold-constrained hyper-connection of the "openPangu 2.0
 * -- architecture, training and Ascend systems" analysis notes, section 5.3:
 * for each token t with n residual streams x[t] in R^{n x D}, K = n*D,
 *
 *   x_bar  = RMSNorm(x[t])                 (flattened n*D row, unit weight)
 *   proj   = x_bar . phi                   (phi in R^{K x G}, G = 2n + n^2)
 *   logits = alpha_group * proj + b        (groups pre | post | res)
 *   H_pre  = sigmoid(logits[0:n])          in (0, 1)
 *   H_post = 2 sigmoid(logits[n:2n])       in (0, 2)
 *   H_res  = Sinkhorn(exp(reshape(logits[2n:], n, n)))   doubly stochastic
 *   x_in   = sum_i H_pre[i] x[t, i]                          (mhc_pre)
 *   x_next[i] = sum_j H_res[i, j] x[t, j] + H_post[i] y[t]   (mhc_post)
 *
 * The ranges of the gates and the doubly stochastic H_res (non-negative, rows
 * and columns summing to 1) are those of the Ascend mHC Triton operator
 * article (paragraph defining H^res / H^pre / H^post).  One Sinkhorn round
 * normalises the rows, then the columns; H_res[i][j] is logit 2n + i*n + j.
 *
 * Conventions shared by every entry point:
 *   - All pointers are device pointers owned by the caller.  The library
 *     allocates no memory; scratch space is passed in (mhc_pre_bwd).
 *   - Tensors are dense, row-major, with the shapes given per argument.
 *     Activations (x, y, x_in, x_next, g_in, g_next, dx, dy) have type `dt`;
 *     gates, phi, b, alpha, saved state and parameter gradients are float32.
 *   - Every pointer must be 16-byte aligned.  n must be 4.  D must be a
 *     multiple of 8 (bf16) or 4 (float32).  T = 0 launches no kernel; the
 *     backward entry points then write zero parameter gradients (below).
 *   - Calls are asynchronous on `stream` (0 = legacy default stream) and
 *     never synchronise the host.  A bad argument returns an error before
 *     anything is launched; a failed launch returns MHC_ERR_CUDA.  Errors that
 *     only the device can see (a bounded wait that ran out) are latched in a
 *     device word and reported by mhc_get_last_device_error().
 *   - Results are deterministic: no floating-point atomics.
 */
#ifndef MHC_GB300_H
#define MHC_GB300_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MHC_OK = 0,
    MHC_ERR_INVALID_ARG = 1,  /* null pointer, negative size, bad iters/eps, short workspace */
    MHC_ERR_UNSUPPORTED = 2,  /* n != 4, D not a multiple of the vector width, iters > MHC_MAX_ITERS */
    MHC_ERR_MISALIGNED = 3,   /* a pointer is not 16-byte aligned */
    MHC_ERR_CUDA = 4,         /* a CUDA runtime call or kernel launch failed */
    MHC_ERR_TIMEOUT = 5,      /* a bounded device-side wait gave up (see mhc_get_last_device_error) */
    MHC_ERR_RANGE = 6         /* a position, slot, length or page number in device memory is outside its tensor */
} mhc_status;

typedef enum { MHC_F32 = 0, MHC_BF16 = 1 } mhc_dtype;

/* Largest Sinkhorn round count the kernels accept (the backward keeps the
 * per-round normalisers of one token in registers / local memory). */
#define MHC_MAX_ITERS 64

/* Human-readable name of a status code (static string, never NULL). */
const char* mhc_status_string(mhc_status s);

/* Library version string, e.g. "mhc_gb300 0.1.0 sm_103a". */
const char* mhc_version(void);

/* Synchronises `stream`, then reads and clears the library's device error
 * word on the current device.  Returns MHC_OK if no kernel latched an error,
 * MHC_ERR_TIMEOUT if a bounded wait ran out, MHC_ERR_RANGE if a kernel of the
 * attention sublayer met a number in device memory that points outside its
 * tensor (and none ran out), MHC_ERR_CUDA if the synchronisation itself failed. */
mhc_status mhc_get_last_device_error(cudaStream_t stream);

/*
 * mhc_pre -- forward of the read side (steps RMSNorm, projection, gates,
 * Sinkhorn and the H_pre mix of section 5.3 of the openPangu 2.0 notes).
 *
 *   x       [T, n, D]  dt      the n-stream residual state
 *   phi     [n*D, G]   float   projection W_mHC (row k = i*D + d)
 *   b       [G]        float   logit bias
 *   alpha   [3]        float   logit scales of the pre, post and res groups
 *   iters              int     Sinkhorn rounds, 1 .. MHC_MAX_ITERS
 *   eps                float   RMSNorm epsilon (>= 0, inside the sqrt)
 * outputs (written):
 *   x_in    [T, D]     dt      sum_i H_pre[i] x[i]  (fp32 sum, one rounding)
 *   H_pre   [T, n]     float
 *   H_post  [T, n]     float
 *   H_res   [T, n, n]  float
 *   proj    [T, G]     float   x_bar . phi (saved for mhc_pre_bwd)
 *   inv_rms [T]        float   1/sqrt(mean(x^2) + eps) (saved for mhc_pre_bwd)
 */
mhc_status mhc_pre(mhc_dtype dt, const void* x, const float* phi,
                   const float* b, const float* alpha, int64_t T, int n,
                   int64_t D, int iters, float eps, void* x_in, float* H_pre,
                   float* H_post, float* H_res, float* proj, float* inv_rms,
                   cudaStream_t stream);

/*
 * mhc_post -- forward of the write side (residual update of section 5.3):
 *   x_next[t, i] = sum_j H_res[t, i, j] x[t, j] + H_post[t, i] y[t]
 *
 *   x [T, n, D] dt; y [T, D] dt; H_post [T, n] float; H_res [T, n, n] float
 *   x_next [T, n, D] dt (written; must not alias x or y)
 */
mhc_status mhc_post(mhc_dtype dt, const void* x, const void* y,
                    const float* H_post, const float* H_res, int64_t T, int n,
                    int64_t D, void* x_next, cudaStream_t stream);

/*
 * mhc_post_norm -- the residual update with openPangu's stability changes
 * (section 5.4 of the openPangu 2.0 notes), each selected by a bit of `flags`:
 *   MHC_POST_SANDWICH_NORM  y' = y r_y, r_y = 1/sqrt(mean_D(y^2) + eps): the
 *                           sublayer output normalised before the H_post
 *                           write-back ("sandwich normalisation");
 *   MHC_POST_BLOCK_NORM     x_next = z s, z = H_res x + H_post y',
 *                           s = 1/sqrt(mean_{n*D}(z^2) + eps): the updated
 *                           multi-stream state normalised ("block-level
 *                           post-normalisation"; the pages apply it after
 *                           the first layer and every fifth one).
 * Unit weights; eps inside the square root.  flags = 0 is mhc_post.
 *
 *   x [T, n, D] dt; y [T, D] dt; H_post [T, n], H_res [T, n, n] float
 * outputs (written): x_next [T, n, D] dt; inv_rms_y [T], inv_rms_out [T]
 *   float (r_y and s, 1 where the step is off; saved for the backward).
 * MHC_ERR_INVALID_ARG for flags outside 0..3; MHC_ERR_UNSUPPORTED when D is
 * above 8192 (bf16) or 4096 (float32).
 */
#define MHC_POST_SANDWICH_NORM 1
#define MHC_POST_BLOCK_NORM 2
mhc_status mhc_post_norm(mhc_dtype dt, const void* x, const void* y,
                         const float* H_post, const float* H_res, int flags,
                         float eps, int64_t T, int n, int64_t D, void* x_next,
                         float* inv_rms_y, float* inv_rms_out, cudaStream_t stream);

/*
 * mhc_post_norm_bwd -- gradients of <g_next, x_next> for mhc_post_norm with
 * the same flags, eps and the saved inv_rms_y, inv_rms_out:
 *   dx, dy written (not added); dH_post [T, n], dH_res [T, n, n] written.
 */
mhc_status mhc_post_norm_bwd(mhc_dtype dt, const void* g_next, const void* x,
                             const void* y, const float* H_post,
                             const float* H_res, int flags, float eps,
                             const float* inv_rms_y, const float* inv_rms_out,
                             int64_t T, int n, int64_t D, void* dx, void* dy,
                             float* dH_post, float* dH_res, cudaStream_t stream);

/*
 * mhc_post_pre -- mhc_post of layer l followed by mhc_pre of layer l + 1 on
 * the x_next it stores, in one pass over x and y where the shape allows (the
 * cross-layer fusion of the inference critical path, section 11.3 of the
 * openPangu 2.0 notes; each step as in section 5.3):
 *   x_next = mhc_post(x, y, H_post_l, H_res_l)                (stored in dt)
 *   (x_in, H_pre, H_post, H_res, proj, inv_rms) = mhc_pre(x_next, phi, b, alpha)
 *
 *   x [T, n, D] dt; y [T, D] dt; H_post_l [T, n], H_res_l [T, n, n] float
 *     (layer l's gates); phi, b, alpha, iters, eps: layer l + 1, as mhc_pre
 * outputs (written; none may alias an input):
 *   x_next [T, n, D] dt   bit-identical to mhc_post's
 *   x_in, H_pre, H_post, H_res, proj, inv_rms   as mhc_pre on the stored x_next
 *   workspace  device scratch of at least mhc_post_pre_workspace_bytes() bytes,
 *              16-byte aligned (NULL when that is 0); ws_bytes its size
 * bf16 shapes the fused kernel covers take two kernels that run at once: the
 * fused pass, and the x_in mix on the SMs the fused pass leaves free (it
 * reads each token tile once the fused pass has counted it done in the
 * workspace).  Every other shape runs mhc_post, then mhc_pre.  Errors as
 * mhc_pre; MHC_ERR_INVALID_ARG for a missing or short workspace.
 */
mhc_status mhc_post_pre(mhc_dtype dt, const void* x, const void* y,
                        const float* H_post_l, const float* H_res_l,
                        const float* phi, const float* b, const float* alpha,
                        int64_t T, int n, int64_t D, int iters, float eps,
                        void* x_next, void* x_in, float* H_pre, float* H_post,
                        float* H_res, float* proj, float* inv_rms,
                        void* workspace, size_t ws_bytes, cudaStream_t stream);

/* Bytes of scratch mhc_post_pre needs for these sizes (0: none). */
size_t mhc_post_pre_workspace_bytes(mhc_dtype dt, int64_t T, int n, int64_t D);

/*
 * mhc_post_bwd -- gradients of <g_next, x_next> for mhc_post:
 *   dx[t, j]      = sum_i H_res[t, i, j] g_next[t, i]     (written, not added)
 *   dy[t]         = sum_i H_post[t, i] g_next[t, i]
 *   dH_post[t, i] = <g_next[t, i], y[t]>
 *   dH_res[t,i,j] = <g_next[t, i], x[t, j]>
 *
 *   g_next, x, dx [T, n, D] dt; y, dy [T, D] dt;
 *   H_post, dH_post [T, n] float; H_res, dH_res [T, n, n] float
 */
mhc_status mhc_post_bwd(mhc_dtype dt, const void* g_next, const void* x,
                        const void* y, const float* H_post, const float* H_res,
                        int64_t T, int n, int64_t D, void* dx, void* dy,
                        float* dH_post, float* dH_res, cudaStream_t stream);

/*
 * mhc_test_force_timeout -- test hook of the failure path, off by default.
 * While on (nonzero), every launch of the bf16 forward kernels (the
 * tensor-core kernel and the small-batch cluster kernel of mhc_pre,
 * mhc_pre_gates and mhc_pre_critical), of mhc_paged_attn's tensor-core kernel
 * and of the pre backward's one-pass cluster kernel (mhc_pre_bwd) makes
 * thread 0 of each CTA wait on an mbarrier that nothing arrives on; the wait
 * gives up after about 100 us, the kernel
 * latches its device error word and returns before starting any copy or
 * tensor-memory allocation, leaving its outputs unwritten.  The next
 * mhc_get_last_device_error() then reports MHC_ERR_TIMEOUT, and the context
 * stays usable.  Synchronous for the backward (it writes a device flag); the
 * forward kernels take the setting as a launch parameter.  Applies to the
 * current device.  Not for production use.
 */
mhc_status mhc_test_force_timeout(int on);

/* Number of kernels the entry point `op` ("mhc_pre", "mhc_pre_gates",
 * "mhc_pre_critical", "mhc_post_res_gates",
 * "mhc_post", "mhc_post_norm", "mhc_post_norm_bwd", "mhc_post_pre",
 * "mhc_post_bwd", "mhc_pre_bwd" or "mhc_layer_bwd_recompute") launches for these sizes; -1 for an
 * unknown op or sizes the entry point would reject.  Useful when sizing CUDA
 * graphs or counting launches. */
int mhc_kernel_launches(const char* op, mhc_dtype dt, int64_t T, int n, int64_t D);

/* Bytes of scratch mhc_pre_bwd needs for these sizes (0 for T = 0). */
size_t mhc_pre_bwd_workspace_bytes(mhc_dtype dt, int64_t T, int n, int64_t D);

/*
 * mhc_pre_bwd -- backward of mhc_pre given the gradient of x_in and the
 * gradients of H_post and H_res (as produced by mhc_post_bwd).  The
 * Sinkhorn forward is recomputed from `proj`; its derivative is the exact
 * reverse mode of the unrolled `iters`-round map.
 *
 *   g_in    [T, D]     dt      dL/dx_in
 *   dH_post [T, n]     float   dL/dH_post
 *   dH_res  [T, n, n]  float   dL/dH_res
 *   x, phi, b, alpha, iters        as passed to mhc_pre
 *   proj, inv_rms      float   as written by mhc_pre
 * outputs:
 *   dx      [T, n, D]  dt      ACCUMULATED: dx += pre-side gradient (the
 *                              H_pre mix plus the projection / RMSNorm path),
 *                              so that after mhc_post_bwd it holds dL/dx
 *   dphi    [n*D, G]   float   written
 *   db      [G]        float   written
 *   dalpha  [3]        float   written
 *   workspace, ws_bytes        device scratch of at least
 *                              mhc_pre_bwd_workspace_bytes() bytes
 *
 * Data parallelism: dphi, db and dalpha are sums over this call's tokens, so
 * ranks that each hold a slice of the batch add them (one all-reduce) to get
 * the full-batch gradient; every other output is per token.  For T = 0 the
 * call writes zero parameter gradients (dphi, db and dalpha, the sums over no
 * tokens, with memsets on `stream`), so a rank with no tokens contributes
 * zero to that sum; the per-token pointers may then be null, dphi, db and
 * dalpha may not.
 */
mhc_status mhc_pre_bwd(mhc_dtype dt, const void* g_in, const float* dH_post,
                       const float* dH_res, const void* x, const float* phi,
                       const float* b, const float* alpha, const float* proj,
                       const float* inv_rms, int64_t T, int n, int64_t D,
                       int iters, void* dx, float* dphi, float* db,
                       float* dalpha, void* workspace, size_t ws_bytes,
                       cudaStream_t stream);

/* Size of the fixed device scratch array behind mhc_pre_bwd_noalloc. */
#define MHC_PRE_BWD_NOALLOC_SCRATCH_BYTES (16u << 20)

/*
 * mhc_pre_bwd_noalloc -- mhc_pre_bwd for callers that cannot allocate device
 * memory.  (The pages have no counterpart: this is a packaging variant.)
 *
 * mhc_pre_bwd needs caller-provided scratch.  Some callers cannot provide
 * it: a custom-op or plugin interface that hands an op its tensors but no
 * workspace, a runtime that plans every device allocation up front and
 * forbids allocating once it runs, or a latency-bound loop that cannot afford
 * cudaMalloc's implicit device synchronisation.  This entry point takes its
 * scratch from a fixed array inside the library's device memory instead and
 * calls no allocating routine.
 *
 * Arguments and results are those of mhc_pre_bwd without the workspace.
 * Limits and behaviour:
 *   - The array holds MHC_PRE_BWD_NOALLOC_SCRATCH_BYTES (16 MiB) on every GPU
 *     that loads the library, until the process exits.  The call returns
 *     MHC_ERR_UNSUPPORTED when T * 256 bytes of per-token records, one
 *     4*D x 24 float32 partial of dphi and D * 256 bytes of bf16 phi blocks
 *     exceed it (for D = 5120: T <= 52,736).
 *   - The first call in each CUDA context looks up the array's device address
 *     in that context (cudaGetSymbolAddress) and keeps it for that context;
 *     a context created later (for example after cudaDeviceReset) gets a
 *     lookup of its own.  That first call must not come while `stream` is
 *     being captured: it then returns MHC_ERR_UNSUPPORTED and does nothing.
 *   - All calls share the array; calls that overlap on the GPU race on it.
 *     Every element is written before it is read, so no state carries over
 *     from one call to the next.
 *   - T = 0 writes zero parameter gradients, as mhc_pre_bwd.
 */
mhc_status mhc_pre_bwd_noalloc(mhc_dtype dt, const void* g_in, const float* dH_post,
                               const float* dH_res, const void* x, const float* phi,
                               const float* b, const float* alpha, const float* proj,
                               const float* inv_rms, int64_t T, int n, int64_t D, int iters,
                               void* dx, float* dphi, float* db, float* dalpha,
                               cudaStream_t stream);

/*
 * The inference critical-path split.  The openPangu 2.0 notes (section 11.3,
 * the inference system) put the previous layer's merge, the RMSNorm and H^pre
 * on the critical path that feeds the sublayer, and move H^post and H^res
 * (with Sinkhorn) to a low-priority side stream that overlaps the sublayer.
 * The two calls below are that split: mhc_pre_critical writes what the
 * sublayer needs (x_in) and the saved state; mhc_post_res_gates computes
 * H^post and H^res from the saved projection and may run on another stream,
 * ordered after mhc_pre_critical by an event.  Together they write the same
 * values as mhc_pre, bit for bit.
 */

/*
 * mhc_pre_critical -- mhc_pre without H_post, H_res and Sinkhorn: x_in,
 * H_pre, proj and inv_rms exactly as mhc_pre writes them (same kernels and
 * arithmetic).  Arguments, layouts, ownership and errors as mhc_pre; there is
 * no iters (no Sinkhorn runs).
 */
mhc_status mhc_pre_critical(mhc_dtype dt, const void* x, const float* phi, const float* b,
                            const float* alpha, int64_t T, int n, int64_t D, float eps, void* x_in,
                            float* H_pre, float* proj, float* inv_rms, cudaStream_t stream);

/*
 * mhc_post_res_gates -- H_post = 2 sigmoid(logits[n:2n]) and H_res =
 * Sinkhorn(exp(reshape(logits[2n:], n, n))), `iters` rounds, from the
 * projection proj [T, 2n+n^2] (float32, as mhc_pre / mhc_pre_critical wrote
 * it), with logits = alpha_group * proj + b as in mhc_pre.  Writes H_post
 * [T, n] and H_res [T, n, n] (float32), bit for bit the values mhc_pre
 * writes.  proj must be complete on `stream` (an event if it was written on
 * another one).  n must be 4; iters in [1, MHC_MAX_ITERS]; every pointer
 * 16-byte aligned; T = 0 is a no-op.
 */
mhc_status mhc_post_res_gates(const float* proj, const float* b, const float* alpha, int64_t T, int n,
                              int iters, float* H_post, float* H_res, cudaStream_t stream);

/*
 * Recompute-oriented backward.  The Ascend mHC Triton operator article
 * (paragraphs on the activation memory of mHC and on recompute inside a
 * layer and across layers) keeps, for each mHC layer, only the input of
 * hc_pre (the multi-stream state x) and the sublayer's output y, and
 * recomputes everything else during the backward.  The two calls below do
 * that: mhc_pre_gates recomputes the gates and the saved state from x, and
 * mhc_layer_bwd_recompute is the whole layer's backward from (x, y) and the
 * incoming gradients.  Across layers, x of layer l + 1 is restored from
 * layer l's (x, y) with mhc_post_pre (or mhc_pre_gates, then mhc_post).
 */

/*
 * mhc_pre_gates -- mhc_pre without the H_pre mix: the same kernel and the
 * same arithmetic, so H_pre, H_post, H_res, proj and inv_rms are bit for bit
 * those mhc_pre writes for the same inputs.  x_in is neither computed nor
 * written.  Arguments, layouts, ownership and errors as mhc_pre.
 */
mhc_status mhc_pre_gates(mhc_dtype dt, const void* x, const float* phi,
                         const float* b, const float* alpha, int64_t T, int n,
                         int64_t D, int iters, float eps, float* H_pre,
                         float* H_post, float* H_res, float* proj,
                         float* inv_rms, cudaStream_t stream);

/* Bytes of scratch mhc_layer_bwd_recompute needs (0 for T = 0): the
 * recomputed gates and saved state (196 B per token), dH_post and dH_res
 * (80 B per token), each region rounded up to 256 B, then
 * mhc_pre_bwd_workspace_bytes(). */
size_t mhc_layer_bwd_recompute_workspace_bytes(mhc_dtype dt, int64_t T, int n,
                                               int64_t D);

/*
 * mhc_layer_bwd_recompute -- the backward of one mHC layer (mhc_pre, the
 * sublayer's output y, mhc_post) from its inputs alone:
 *   mhc_pre_gates(x)   -> H_pre, H_post, H_res, proj, inv_rms   (scratch)
 *   mhc_post_bwd       -> dx (written), dy, dH_post, dH_res     (dH: scratch)
 *   mhc_pre_bwd        -> dx (accumulated), dphi, db, dalpha
 * on `stream`, in that order.  The results are bit for bit those of
 * mhc_post_bwd then mhc_pre_bwd given the state a mhc_pre call on the same x
 * saved.
 *
 *   g_in    [T, D]     dt      dL/dx_in
 *   g_next  [T, n, D]  dt      dL/dx_next
 *   x, phi, b, alpha, iters, eps   as passed to mhc_pre
 *   y       [T, D]     dt      the sublayer output, as passed to mhc_post
 * outputs (written):
 *   dx      [T, n, D]  dt      dL/dx (both paths)
 *   dy      [T, D]     dt      dL/dy
 *   dphi    [n*D, G]   float
 *   db      [G]        float
 *   dalpha  [3]        float
 *   workspace, ws_bytes        device scratch of at least
 *                              mhc_layer_bwd_recompute_workspace_bytes() bytes
 * Errors as mhc_pre_bwd; MHC_ERR_INVALID_ARG for a missing or short
 * workspace.  Data parallelism and T = 0 (zero dphi, db, dalpha) as
 * mhc_pre_bwd.
 */
mhc_status mhc_layer_bwd_recompute(mhc_dtype dt, const void* g_in, const void* g_next,
                                   const void* x, const void* y, const float* phi,
                                   const float* b, const float* alpha, int64_t T, int n,
                                   int64_t D, int iters, float eps, void* dx, void* dy,
                                   float* dphi, float* db, float* dalpha, void* workspace,
                                   size_t ws_bytes, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * The attention sublayer, between mhc_pre (which writes its input x_in) and
 * mhc_post (which takes its output y): per-head normalisation of queries and
 * keys with the position rotation, in training and in serving, and attention
 * of new tokens over a paged key/value cache.
 *
 * Heads: Hq query heads and Hk key/value heads of Dh values, Hq a multiple of
 * Hk; query head h belongs to key head h / (Hq/Hk).  Dh is a multiple of 8, at
 * most 256.  A tensor of heads [T, H, Dh] is given with the distance between
 * its tokens in elements (>= H*Dh), so that q, k and v may be parts of one
 * packed projection; the heads of a token lie one after the other.  Pointers
 * and distances of activations, caches, weights, angles and workspaces are
 * multiples of 16 bytes, those of integers and of lse of their own size.
 *
 * Numbers that only the device sees (positions, slots, lengths, page numbers)
 * are checked by the kernels.  One that points outside its tensor is latched
 * (MHC_ERR_RANGE from mhc_get_last_device_error) and nothing outside the
 * tensors is read or written.
 * ------------------------------------------------------------------------- */

/* flags of the rotation: pairs (j, j + rot/2) by default, or (2j, 2j + 1) */
#define MHC_ROPE_ADJACENT 1

/*
 * mhc_qk_norm_rope -- for every head x of q (weight w = w_q) and k (w_k):
 *   z = x w / sqrt(mean_Dh(x^2) + eps)                 (RMSNorm of the head)
 *   y = z with its first `rot` values turned by the token's position p: each
 *       pair (a, b) with angle index j becomes
 *       (a cos[p, j] - b sin[p, j], b cos[p, j] + a sin[p, j])
 *   Sums in float32; y is rounded to dt once.
 *
 *   q [T, Hq, Dh], k [T, Hk, Dh]  dt       q_stride, k_stride between tokens
 *   w_q, w_k [Dh]        float
 *   positions [T]        int32            rows of cos_sin (0 <= p < max_pos)
 *   cos_sin [max_pos, rot] float          rot/2 cosines, then rot/2 sines
 *   rot                  int              multiple of 16, 0 <= rot <= Dh; with
 *                                         rot = 0 positions and cos_sin may be null
 *   flags                int              0 or MHC_ROPE_ADJACENT
 * outputs: q_out, k_out  dt               as q and k (may be the same memory
 *                                         with the same stride)
 * A token whose position is out of range gets zeros.  T = 0 is a no-op.
 */
mhc_status mhc_qk_norm_rope(mhc_dtype dt, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                            const float* w_q, const float* w_k, const int32_t* positions,
                            const float* cos_sin, int64_t max_pos, int64_t T, int Hq, int Hk, int Dh,
                            int rot, int flags, float eps, void* q_out, int64_t q_out_stride, void* k_out,
                            int64_t k_out_stride, cudaStream_t stream);

/*
 * mhc_qk_norm_rope_bwd -- gradients of <g_q, q_out> + <g_k, k_out>:
 * with h = the gradient turned back, r = 1/sqrt(mean(x^2) + eps), u = h w,
 *   dx = r u - x r^3 <u, x> / Dh,      dw = sum over tokens and heads of h x r
 * Nothing is saved by the forward: r is computed again from x.
 *
 *   g_q, g_k             dt               as q_out and k_out of the forward
 *   the rest as passed to mhc_qk_norm_rope
 * outputs (written): dq, dk dt as q and k; dw_q, dw_k [Dh] float (sums in a
 *   fixed order, so results repeat bit for bit; zeros for T = 0)
 *   workspace  device scratch of mhc_qk_norm_rope_bwd_workspace_bytes() bytes
 * A token whose position is out of range gets zero gradients.
 */
mhc_status mhc_qk_norm_rope_bwd(mhc_dtype dt, const void* g_q, int64_t gq_stride, const void* g_k,
                                int64_t gk_stride, const void* q, int64_t q_stride, const void* k,
                                int64_t k_stride, const float* w_q, const float* w_k,
                                const int32_t* positions, const float* cos_sin, int64_t max_pos, int64_t T,
                                int Hq, int Hk, int Dh, int rot, int flags, float eps, void* dq,
                                int64_t dq_stride, void* dk, int64_t dk_stride, float* dw_q, float* dw_k,
                                void* workspace, size_t ws_bytes, cudaStream_t stream);
size_t mhc_qk_norm_rope_bwd_workspace_bytes(int64_t T, int Dh);

/*
 * mhc_qk_norm_rope_append -- the serving form of mhc_qk_norm_rope: q_out as
 * there; the normalised, turned keys and the values as they are go to the
 * paged cache.  Token t goes to slot slots[t] = page * page_size + place in
 * the page; -1 writes no key and no value (a padding token).  Two tokens of a
 * call must not share a slot.
 *
 *   v [T, Hk, Dh]        dt               v_stride between tokens
 *   slots [T]            int64
 *   k_cache, v_cache     dt               element (page, place, head, d) at
 *     page*page_stride + place*slot_stride + head*head_stride + d: both
 *     [pages, page_size, Hk, Dh] and [pages, Hk, page_size, Dh] are covered
 */
mhc_status mhc_qk_norm_rope_append(mhc_dtype dt, const void* q, int64_t q_stride, const void* k,
                                   int64_t k_stride, const void* v, int64_t v_stride, const float* w_q,
                                   const float* w_k, const int32_t* positions, const float* cos_sin,
                                   int64_t max_pos, const int64_t* slots, int64_t T, int Hq, int Hk, int Dh,
                                   int rot, int flags, float eps, void* q_out, int64_t q_out_stride,
                                   void* k_cache, int64_t k_page_stride, int64_t k_slot_stride,
                                   int64_t k_head_stride, void* v_cache, int64_t v_page_stride,
                                   int64_t v_slot_stride, int64_t v_head_stride, int64_t num_pages,
                                   int page_size, cudaStream_t stream);

/*
 * mhc_rope_table -- the angles that the rotations take, for positions
 * 0 .. n - 1: row p holds amplitude cos(p f_j), then amplitude sin(p f_j), for
 * the rot/2 frequencies
 *   f_j = e_j (g_j + (1 - g_j) / factor),     e_j = base^(-2j / rot),
 *   g_j = (original e_j / 2 pi - low) / (high - low), held to [0, 1].
 * With factor = 1 that is the plain rotation.  For contexts `factor` times as
 * long as the trained one, original = 0 slows every pair down alike (positions
 * are interpolated linearly); with the trained length as `original`, pairs that
 * make more than `high` turns over it keep their frequency, those that make
 * fewer than `low` are slowed down, and the ones between are blended.  Scaling
 * the base is the caller's: base factor^(rot / (rot - 2)).
 * The blend is linear in a pair's turns.  Models whose blend is linear in the pair's
 * number instead, or that have a factor of their own for each pair, have other
 * frequencies (by up to 65 % for base 10000, factor 16, 1 to 32 turns over 8192):
 * their tables are not made here; the rotations take a table from anywhere.
 * Frequencies are computed in double and multiplied by positions in 64-bit integers,
 * so the angle of position p is off by at most
 *   p max(1, 1 / factor) (2^-49 + 2^-50 high / (high - low))
 * radians (the second term only where high > 0 and original > 0) for every pair: a
 * slow pair's angle has fewer right digits than a fast one's.  Values are right to
 * 3 2^-24 times the amplitude beside that.
 *
 *   base >= 1, factor > 0, original >= 0, low < high, all finite
 *   rot  int             multiple of 16, 16 <= rot <= 256
 * output: cos_sin [n, rot] float, 16-byte aligned.  n = 0 is a no-op.
 */
mhc_status mhc_rope_table(int64_t n, int rot, double base, double factor, double original, double low, double high,
                          float amplitude, float* cos_sin, cudaStream_t stream);

/*
 * mhc_rope -- mhc_qk_norm_rope without the normalisation: every head of q and k
 * has its first `rot` values turned by the token's position, the others are
 * copied.  Each value is rounded to dt once.  A table with an amplitude scales
 * the turned values.
 * mhc_rope_bwd -- gradients of <g_q, q_out> + <g_k, k_out>: the turned values
 * turned back (times the amplitude).  It needs neither q nor k.
 * mhc_rope_append -- the serving form, as mhc_qk_norm_rope_append.
 * Arguments as there; rot > 0.  Outputs may be the same memory as q and k with
 * the same strides.  A token whose position is out of range gets zeros
 * (gradients too) and is not appended.  T = 0 is a no-op.
 */
mhc_status mhc_rope(mhc_dtype dt, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                    const int32_t* positions, const float* cos_sin, int64_t max_pos, int64_t T, int Hq, int Hk,
                    int Dh, int rot, int flags, void* q_out, int64_t q_out_stride, void* k_out,
                    int64_t k_out_stride, cudaStream_t stream);
mhc_status mhc_rope_bwd(mhc_dtype dt, const void* g_q, int64_t gq_stride, const void* g_k, int64_t gk_stride,
                        const int32_t* positions, const float* cos_sin, int64_t max_pos, int64_t T, int Hq, int Hk,
                        int Dh, int rot, int flags, void* dq, int64_t dq_stride, void* dk, int64_t dk_stride,
                        cudaStream_t stream);
mhc_status mhc_rope_append(mhc_dtype dt, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const void* v, int64_t v_stride, const int32_t* positions, const float* cos_sin,
                           int64_t max_pos, const int64_t* slots, int64_t T, int Hq, int Hk, int Dh, int rot,
                           int flags, void* q_out, int64_t q_out_stride, void* k_cache, int64_t k_page_stride,
                           int64_t k_slot_stride, int64_t k_head_stride, void* v_cache, int64_t v_page_stride,
                           int64_t v_slot_stride, int64_t v_head_stride, int64_t num_pages, int page_size,
                           cudaStream_t stream);

/*
 * mhc_paged_attn -- causal attention of new tokens over a paged cache that
 * holds their keys and values already.  Sequence b of B has the rows
 * cu_q[b] .. cu_q[b+1] of q (its newest tokens, n of them; one in decoding, a
 * chunk of a prompt otherwise) and kv_lens[b] = m cached tokens, the n new ones
 * last.  Token j of the sequence is at place j % page_size of page
 * page_table[b, j / page_size].  For query i of the n, with scores
 *   z_ij = scale <q_i, k_j>,   z <- softcap tanh(z / softcap) if softcap > 0,
 * over the keys 0 <= j <= m - n + i, and, if window > 0, j > m - n + i - window:
 *   o_i = sum_j exp(z_ij) v_j / sum_j exp(z_ij),   lse_i = log sum_j exp(z_ij).
 * A row that sees no key (m < n) gets o = 0 and lse = -inf.  Sums and softmax
 * statistics are float32; on the tensor cores the exponentials of a block are
 * rounded to bf16 for their product with the values (by at most 2^-8 of each).
 * There a capped score is right to 2^-20 of a softcap of up to 256, and to a
 * relative 2^-18 of the score with a larger one.
 *
 *   q [T, Hq, Dh]        dt               q_stride between tokens
 *   k_cache, v_cache     dt               as in mhc_qk_norm_rope_append
 *   page_table [B, *]    int32            table_stride between rows, at least
 *                                         ceil(max_kv / page_size); entries of
 *                                         pages that no query of the sequence
 *                                         sees are not used
 *   cu_q [B+1], kv_lens [B] int32         or both null: the workspace holds
 *                                         the plan of mhc_paged_attn_plan
 *   max_q, max_kv                         no sequence has more new or cached tokens
 *   scale > 0, softcap >= 0 (0: off), window >= 0 (0: unlimited)
 * outputs: o [T, Hq, Dh] dt; lse [T, Hq] float (null: not wanted).  Rows of q
 *   that belong to no sequence are left as they are, and so are the rows of a
 *   sequence whose numbers do not fit the call (MHC_ERR_RANGE).
 *   workspace  device scratch of mhc_paged_attn_workspace_bytes() bytes; calls
 *              that may overlap need one each
 * The tokens of a page number outside the cache count as zeros, keys and values
 * (MHC_ERR_RANGE): their sequence's rows are computed with them, the other
 * sequences' as ever.
 * What the pages hold beyond the cached tokens, or outside what a tile of rows
 * can see, is never used (it may be NaN).  Values that some row of a call sees
 * must be finite for every row's result to be, and with a softcap between 31 and
 * 52 below 2^30: no running maximum is kept there on the tensor cores.
 *
 * mhc_paged_attn_plan -- splits the batch over the GPU (one small kernel) into
 * `workspace`, for any number of mhc_paged_attn calls with the same sizes: the
 * layers of one step.  It depends on cu_q, kv_lens, window and the sizes only.
 * A call whose sizes (max_q and max_kv among them) are not its plan's computes
 * nothing and sets MHC_ERR_RANGE, and so does every later call with the plan of a
 * call that ended with MHC_ERR_TIMEOUT: the batch has to be planned again.
 */
mhc_status mhc_paged_attn_plan(mhc_dtype dt, const int32_t* cu_q, const int32_t* kv_lens, int64_t T, int B,
                               int Hq, int Hk, int Dh, int page_size, int64_t max_q, int64_t max_kv,
                               int window, void* workspace, size_t ws_bytes, cudaStream_t stream);
mhc_status mhc_paged_attn(mhc_dtype dt, const void* q, int64_t q_stride, const void* k_cache,
                          int64_t k_page_stride, int64_t k_slot_stride, int64_t k_head_stride,
                          const void* v_cache, int64_t v_page_stride, int64_t v_slot_stride,
                          int64_t v_head_stride, int64_t num_pages, int page_size,
                          const int32_t* page_table, int64_t table_stride, const int32_t* cu_q,
                          const int32_t* kv_lens, int64_t T, int B, int Hq, int Hk, int Dh, int64_t max_q,
                          int64_t max_kv, int window, float scale, float softcap, void* o, float* lse,
                          void* workspace, size_t ws_bytes, cudaStream_t stream);
size_t mhc_paged_attn_workspace_bytes(mhc_dtype dt, int64_t T, int B, int Hq, int Hk, int Dh, int page_size,
                                      int64_t max_q);

/*
 * mhc_tree_attn -- attention of trees of drafted tokens over a paged cache that
 * holds their keys and values already: the verification of speculative decoding.
 * As mhc_paged_attn, but the n new tokens of a sequence (the rows cu_q[b] ..
 * cu_q[b+1] of q, and the last n of its m cached tokens) are the nodes of a tree
 * in any order.  Row t of `tree` says which of the sequence's new tokens node t
 * sees: bit i % 32 of word i / 32 for the i-th one (itself and its ancestors,
 * usually; any mask is taken).  Node t sees the m - n cached tokens before the
 * new ones (its context) and those.  With a window, it sees its nodes and the
 * last window - max(1, how many these are) tokens of the context: the window of
 * mhc_paged_attn where a node has at most `window` bits.  A node's bits count
 * whatever the window is: of a path that is longer, the mask has to leave out the
 * ancestors that lie `window` or more back (those of mhc_paged_step have all of them).
 * A row that sees no key gets o = 0 and lse = -inf; so does every row of a
 * sequence with m < n, whose drafted tokens are not all cached.
 * In bf16 on the tensor cores the exponentials are rounded as there: o is off by at
 * most 2^-8 (sum_j p_j |v_j| + |o|) beside float32 sums, with p_j the probabilities;
 * lse, and all of float32, is not touched by it.
 *
 *   tree [T, *]          int32            tree_stride words between rows, at
 *                                         least ceil(max_q / 32); bits past a
 *                                         sequence's new tokens are ignored
 *   max_q                                 at most 1024
 *   cu_q, kv_lens                         there is no plan: every call splits the
 *                                         batch by itself, from these
 * The rest, the workspace (mhc_paged_attn_workspace_bytes) and the errors are as
 * for mhc_paged_attn.  What the pages hold for a drafted token that no row of a
 * tile sees (padding, say) is never used; with a window the last window - 1
 * tokens of the context count as seen.
 */
mhc_status mhc_tree_attn(mhc_dtype dt, const void* q, int64_t q_stride, const void* k_cache,
                         int64_t k_page_stride, int64_t k_slot_stride, int64_t k_head_stride,
                         const void* v_cache, int64_t v_page_stride, int64_t v_slot_stride,
                         int64_t v_head_stride, int64_t num_pages, int page_size, const int32_t* page_table,
                         int64_t table_stride, const int32_t* tree, int64_t tree_stride, const int32_t* cu_q,
                         const int32_t* kv_lens, int64_t T, int B, int Hq, int Hk, int Dh, int64_t max_q,
                         int64_t max_kv, int window, float scale, float softcap, void* o, float* lse,
                         void* workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * mhc_paged_step -- the integer tensors of a step's new tokens, made on the GPU
 * from the lengths of its sequences (no host copy, so a captured step serves any
 * lengths): row starts, slots, positions, pages of the free list for those that
 * run out of room, and what each node of a drafted tree sees.
 *
 * Sequence b has lens[b] cached tokens and gets new_lens[b] new ones (0: none
 * this step), or ends (-1).  It holds held[b] pages, the first entries of its row
 * of page_table, which cover its cached tokens; tokens that were drafted and
 * dropped may have left it with more.  In order:
 *   1. the pages of sequences that end go back on the free list, sequence after
 *      sequence, each row's last page on top;
 *   2. each sequence needs max(0, ceil((lens + new) / page_size) - held) pages; in
 *      the order of the sequences they come from the top of the list, the page
 *      on top first.  A sequence gets all of them or none: from the first one
 *      for which too few are left on, only sequences that need none get room;
 *   3. new token i of sequence b is row cu_q[b] + i, and its place in the sequence
 *      lens[b] + i; slots holds page * page_size + place in the page, -1 where the
 *      sequence got no room.
 * kv_lens[b] is lens[b] + new_lens[b], lens[b] for a sequence without room (what
 * attention gives its rows means nothing; it can be given its tokens again once
 * others have ended), 0 for one that ends.
 * Positions are the places in the sequence, or with trees lens[b] + the number of
 * the node's ancestors.  Parent parents[t] of row t is a number among its
 * sequence's new tokens, below its own, or -1 (it follows the context); row t of
 * `tree` gets the bits of the node and all its ancestors, as mhc_tree_attn takes them
 * (layers with a window shorter than a path need their early ones taken out).
 *
 *   new_lens, lens [B]   int32
 *   page_table [B, *]    int32   in/out   table_width entries a row, table_stride apart
 *   held [B]             int32   in/out
 *   free_pages           int32   in/out   a stack of free_capacity entries, free_count
 *   free_count [1]       int32   in/out   of them in use, the last one on top
 *   T                                     rows of the outputs; those past the new
 *                                         tokens get slot -1, position 0, no bits
 *   parents [T]          int32            or null: no trees
 *   tree_words                            words of a row of `tree`, 1 to 32
 * outputs: cu_q [B+1], kv_lens [B], positions [T] int32, slots [T] int64,
 *   tree [T, tree_words] int32 (null without parents).  Nothing that is written may
 *   lie in the memory of another argument (kv_lens is not lens, say): such a call is
 *   refused with MHC_ERR_INVALID_ARG.  new_lens, lens and parents may be the same.
 * MHC_ERR_RANGE: sequences whose rows would pass T (they and all later ones get
 * none: cu_q stays), whose numbers do not fit (lengths below 0, or past held pages
 * or the table; they get slots -1, positions 0 and kv_lens 0), parents that are not
 * below their node (as -1), nodes past tree_words * 32 (without a bit; of their
 * paths the last 1024 nodes count), a list's
 * length outside its tensor, more pages coming back than it has room for (those
 * are lost).  At most 8192 sequences, 2^30 entries of the table.
 */
mhc_status mhc_paged_step(const int32_t* new_lens, const int32_t* lens, int B, int32_t* page_table,
                          int64_t table_stride, int64_t table_width, int32_t* held, int32_t* free_pages,
                          int64_t free_capacity, int32_t* free_count, int page_size, int64_t T,
                          const int32_t* parents, int tree_words, int32_t* cu_q, int32_t* kv_lens,
                          int32_t* positions, int64_t* slots, int32_t* tree, cudaStream_t stream);

/*
 * mhc_cache_keep -- after a drafted tree has been verified: the keys and values
 * of the accepted path move to the places behind the context, in the caches of
 * `layers` layers.  Sequence b has n = cu_q[b+1] - cu_q[b] drafted tokens, the
 * last of its m = kv_lens[b] cached ones, and keeps keep[b] of them: nodes
 * path[b, 0] < path[b, 1] < ... of 0 .. n - 1 go to the places m - n, m - n + 1,
 * ...; then lens[b] = m - n + keep[b].  keep[b] = 0 moves nothing and leaves
 * lens[b] as it is (as it must be for a sequence that mhc_paged_step gave no room:
 * its drafted tokens are not in the cache).  Places behind the kept tokens hold what
 * is left there.
 *
 *   k_caches, v_caches   host arrays of `layers` device pointers, each a cache as
 *                        in mhc_qk_norm_rope_append, all keys (and all values)
 *                        with the same strides; no two overlap
 *   page_table [B, *]    int32            table_stride between rows, at least
 *                                         ceil(max_kv / page_size)
 *   cu_q [B+1], kv_lens [B], keep [B] int32
 *   path [B, *]          int32            path_stride between rows, >= max_keep
 *   lens [B]             int32   out      or null; none of the inputs' memory
 * No sequences, no layers or max_keep = 0: a no-op, lens stays as it is too.
 * MHC_ERR_RANGE: a sequence whose numbers do not fit (a path that does not rise
 * or leaves the drafted tokens, keep past max_keep or n, m outside n .. max_kv) is
 * left as it is; a row on a page outside the cache is not moved.
 */
mhc_status mhc_cache_keep(mhc_dtype dt, void* const* k_caches, int64_t k_page_stride, int64_t k_slot_stride,
                          int64_t k_head_stride, void* const* v_caches, int64_t v_page_stride,
                          int64_t v_slot_stride, int64_t v_head_stride, int layers, int64_t num_pages,
                          int page_size, const int32_t* page_table, int64_t table_stride, const int32_t* cu_q,
                          const int32_t* kv_lens, int64_t max_kv, int B, int Hk, int Dh, const int32_t* path,
                          int64_t path_stride, int max_keep, const int32_t* keep, int32_t* lens,
                          cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MHC_GB300_H */
