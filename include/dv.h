/*
 * dv.h -- C ABI of the contextually sparse (DejaVu) decode step of one
 * transformer layer, for NVIDIA GB300 (sm_103a).
 *
 * The method (DejaVu, "Deja Vu: Contextual Sparsity for Efficient LLMs at
 * Inference Time", abstract; "DejaVu Guide: Contextual Sparsity for LLM
 * Inference", "Core Innovation 1: Asynchronous Lookahead Predictors" and
 * "Core Innovation 2: Hardware-Efficient Dynamic Sparse Matrix Execution"):
 * a cheap predictor scores the layer's attention heads and MLP neurons from
 * an input vector and keeps the top-k of each; the layer then reads from HBM
 * only the selected heads' QKV rows, out-projection rows and KV cache, and
 * the selected neurons' fc1 rows and fc2 rows.  Dense weights stay intact.
 *
 * Conventions for every entry point
 *  - All tensor pointers are DEVICE pointers owned by the caller, unless an
 *    entry point says "host".  The library allocates no memory and keeps no
 *    state between calls other than what lives in the caller's workspace.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = the legacy default
 *    stream) and returns without synchronising, except where stated.
 *    Index counts stay on the device; no call reads device memory on the
 *    host, so a call can be captured in a CUDA graph.
 *  - Arguments are checked on the host before anything is launched; a bad
 *    argument returns DV_ERR_INVALID_ARG (or DV_ERR_UNSUPPORTED for a shape
 *    the kernels do not handle) and launches nothing.  A launch failure
 *    returns DV_ERR_CUDA.  A kernel that meets a bad value at run time (an
 *    index outside its range) skips it and records the first such event in
 *    the workspace status word, which dv_check() reads.
 *  - The workspace (`ws`, `ws_bytes` >= dv_workspace_size()) must be zeroed
 *    once with dv_workspace_init() before its first use; every call leaves
 *    it ready for the next one.  Calls that share a workspace must not run
 *    concurrently.
 *  - Layouts are row-major.  Weight matrices, biases, norm parameters and the
 *    KV cache are stored in `desc.dtype` (binary32 or binary16); activations
 *    are binary32; accumulation is binary32.  Every weight and activation
 *    pointer must be 16-byte aligned.
 *
 * Shapes (d = d_model, H = n_heads, dh = head_dim, N = d_ffn, r = pred_rank,
 * B = batch, kv_cap = KV positions allocated per batch row and head):
 *   ln1_g, ln1_b, ln2_g, ln2_b, b_o, b2   [d]
 *   w_qkv  [3, H, dh, d]   (q, k, v rows of every head)
 *   b_qkv  [3, H, dh]
 *   w_oT   [H, dh, d]      (out-projection transposed: head h's input columns
 *                           are the contiguous rows w_oT[h])
 *   w1     [N, d]          (fc1: neuron j's row is contiguous)
 *   b1     [N]
 *   w2T    [N, d]          (fc2 transposed: neuron j's output column is the
 *                           contiguous row w2T[j])
 *   pred_h [H, d]          (head predictor)
 *   pred_a [r, d], pred_b [N, r]   (low-rank neuron predictor)
 *   k_cache, v_cache [B, H, kv_cap, dh]
 */
#ifndef DV_H
#define DV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DV_ABI_VERSION 2
#define DV_MAX_BATCH 32

typedef enum {
    DV_OK = 0,
    DV_ERR_INVALID_ARG = 1,  /* bad pointer, size, count or alignment */
    DV_ERR_UNSUPPORTED = 2,  /* valid but not handled (e.g. head_dim not a power of two) */
    DV_ERR_CUDA = 3,         /* a CUDA runtime call failed */
    DV_ERR_TIMEOUT = 4,      /* a bounded device-side wait gave up */
    DV_ERR_WORKSPACE = 5,    /* workspace missing, misaligned or too small */
    DV_ERR_DEVICE_INDEX = 6, /* a kernel met an index outside its range (skipped) */
    DV_ERR_SCRATCH_LIMIT = 7, /* dv_predict_topk_noalloc: shape needs more than its scratch */
    DV_ERR_PAGES = 8         /* dv_page_take: the pool has too few free pages */
} dv_status;

/* DV_I8 is a storage type of the KV-cache operators (dv_kv_desc) alone. */
typedef enum { DV_F32 = 0, DV_F16 = 1, DV_I8 = 2 } dv_dtype;
typedef enum { DV_LAYERNORM = 0, DV_RMSNORM = 1 } dv_norm;
/* MLP of the layer: OPT's fc1, ReLU, fc2 (w1 [N, d], w2T [N, d]) or the
 * LLaMA-style SwiGLU (gate and up rows of neuron j interleaved in w1
 * [N, 2, d], b1 [N, 2]; down-projection columns in w2T [N, d]). */
typedef enum { DV_MLP_RELU = 0, DV_MLP_SWIGLU = 1 } dv_mlp;

/* Shape and storage of one layer. */
typedef struct {
    int32_t d_model;
    int32_t n_heads;
    int32_t head_dim;   /* power of two; head_dim * sizeof(dtype) in [16, 512] */
    int32_t d_ffn;
    int32_t pred_rank;
    int32_t dtype;      /* dv_dtype of weights, biases, norms and KV cache */
    int32_t norm;       /* dv_norm used before attention and before the MLP */
    float ln_eps;
    int32_t kv_cap;     /* KV positions per (batch row, head) */
    /* 0 or 1: neurons are selected one by one.  32, 64 or 128 (dividing
     * d_ffn, at most 2048 blocks): neurons are selected in blocks
     * of that many contiguous channels ("DejaVu Guide ...", "Core Innovation
     * 2", "1. Blocked Channel Sparsity"): a block's score is the largest
     * score of its members, each row keeps its k_neurons / neuron_block best
     * blocks (ties to the lower block), and k_neurons must be a multiple of
     * neuron_block. */
    int32_t neuron_block;
    int32_t mlp;        /* dv_mlp */
} dv_layer_desc;

/* Device pointers to one layer's weights (shapes in the header comment). */
typedef struct {
    const void *ln1_g, *ln1_b;
    const void *w_qkv, *b_qkv;
    const void *w_oT, *b_o;
    const void *ln2_g, *ln2_b;
    const void *w1, *b1;
    const void *w2T, *b2;
    const void *pred_h, *pred_a, *pred_b;
} dv_layer_weights;

/* Device buffers receiving a selection.
 *   idx_h [B, k_heads], idx_n [B, k_neurons]: each row's top-k, ascending;
 *   u_h [min(H, B*k_heads)], u_n [min(N, B*k_neurons)]: union of the rows,
 *   ascending; its length is written to n_u_h[0] / n_u_n[0]. */
typedef struct {
    int32_t *idx_h, *idx_n;
    int32_t *u_h, *n_u_h;
    int32_t *u_n, *n_u_n;
} dv_selection;

/* Static description of a status code (never NULL). */
const char *dv_status_string(int status);

/* The CUDA runtime's error code behind the last DV_ERR_CUDA returned on
 * this host thread (reading it clears it; 0 if none).  Diagnostic. */
int dv_cuda_error(void);

/* DV_ABI_VERSION of the built library. */
int dv_abi_version(void);

/* Row-kernel variant of the fc1 rows on the tensor cores ("DejaVu Guide:
 * Contextual Sparsity for LLM Inference", the pipeline's "Sparse Gather GEMV
 * on Tensor Cores"), process-wide, for calls issued after it returns:
 *   0  mma.sync m16n8k16 kernel (the default);
 *   1  tcgen05.mma kernel (M = 128 gathered rows, accumulator in tensor
 *      memory) for binary16 ReLU layers from 9 batch rows with d_model a
 *      multiple of 64; every other case keeps variant 0.
 * Results agree within the binary32 accumulation error; the ring, segment
 * and partial order differ, so the bits may not.  DV_ERR_INVALID_ARG for
 * another value.  Not thread-safe against calls in flight on other
 * threads. */
dv_status dv_set_row_kernel(int variant);

/* Bytes of workspace the calls below need for this layer shape and batch
 * (sized for the largest possible unions).  0 if desc or batch is invalid. */
size_t dv_workspace_size(const dv_layer_desc *desc, int batch);

/* Zero a workspace on `stream` (one cudaMemsetAsync).  Needed once before a
 * workspace is first used. */
int dv_workspace_init(void *ws, size_t ws_bytes, void *stream);

/* Synchronise `stream`, then read the workspace status word (device faults
 * recorded by kernels, see DV_ERR_DEVICE_INDEX / DV_ERR_TIMEOUT) and clear
 * it.  Returns DV_OK if nothing was recorded. */
int dv_check(void *ws, size_t ws_bytes, void *stream);

/* Kernel launches one dv_layer_decode call enqueues (the events
 * dv_layer_decode_traced records sit around them).  0 if desc or batch is
 * invalid. */
int dv_layer_decode_launches(const dv_layer_desc *desc, int batch);

/* 1 if dv_sparse_mlp (and the MLP half of dv_layer_decode) with a neuron
 * union of at most max_u_n runs as one pass over the selected fc1 rows and
 * fc2 columns plus a kernel that adds the per-CTA partials of y, on the
 * current device; 0 if it runs as the fc1 and fc2 kernels, or for invalid
 * arguments. */
int dv_mlp_one_pass(const dv_layer_desc *desc, int batch, int max_u_n);



/* 1 if dv_layer_decode_persistent (the streaming kernel) serves this shape
 * and batch on the current device for every k_heads, k_neurons and kv_len,
 * else 0. */
int dv_layer_decode_persistent_ok(const dv_layer_desc *desc, int batch);

/*
 * dv_predict_topk -- the lookahead predictors and top-k selection.
 * ("DejaVu Guide ...", "1. Mathematical Formulation of Lookahead Predictors":
 * head mask = Top-k_head(x . W_pred_attn), neuron mask = Top-k_mlp(x .
 * W_pred_mlp); the guide's listing, DejaVuLookaheadPredictor.forward, returns
 * the kept indices sorted.)
 *   head scores   s_h[b][h] = x_pred[b] . pred_h[h]
 *   neuron scores s_n[b][j] = (x_pred[b] . pred_a^T) . pred_b[j]   (rank r)
 * For every row b: the k_heads / k_neurons largest binary32 scores, ties to
 * the lower index, written ascending to sel->idx_h[b] / sel->idx_n[b]; then
 * the union over rows to sel->u_h / sel->u_n with device counts.
 *   x_pred   [B, d] binary32 device input.
 *   scores_h [B, H], scores_n [B, N]: optional device outputs of the scores
 *            (NULL to skip).
 * Errors: DV_ERR_INVALID_ARG for k outside [1, H] / [1, N], batch outside
 * [1, DV_MAX_BATCH], NULL or misaligned pointers.
 */
int dv_predict_topk(const dv_layer_desc *desc, const dv_layer_weights *w, const float *x_pred,
                    int batch, int k_heads, int k_neurons, const dv_selection *sel,
                    float *scores_h, float *scores_n, void *ws, size_t ws_bytes, void *stream);

/*
 * dv_sparse_attn -- head-pruned attention block with its residual.
 * ("DejaVu Guide ...", "2. Head-Pruned Attention Dispatch": an inactive head's
 * projection weights, output-projection weights and historical KV cache are
 * not read.)  For every row b, with xn = norm(x[b]; ln1_g, ln1_b) and every
 * head h in u_h[0 .. *n_u_h):
 *   q, k, v = xn . w_qkv[{0,1,2}, h]^T + b_qkv[{0,1,2}, h];  q *= 1/sqrt(dh)
 *   k_cache[b, h, kv_len] = k, v_cache[b, h, kv_len] = v  (rounded to dtype)
 *   o_h = softmax(q . K[b, h, 0..kv_len]^T) . V[b, h, 0..kv_len]
 *   h1[b] = x[b] + b_o + sum_h o_h . w_oT[h]
 * Unselected heads' caches (slot kv_len included) are not touched.
 *   x [B, d], h1 [B, d] binary32 device; u_h / n_u_h device, max_u_h = the
 *   length of u_h (upper bound of *n_u_h, <= H); 0 <= kv_len < kv_cap.
 */
int dv_sparse_attn(const dv_layer_desc *desc, const dv_layer_weights *w, const float *x, int batch,
                   const int32_t *u_h, const int32_t *n_u_h, int max_u_h, void *k_cache,
                   void *v_cache, int kv_len, float *h1, void *ws, size_t ws_bytes, void *stream);

/*
 * dv_sparse_mlp -- contextually sparse MLP block with its residual.
 * ("DejaVu Guide ...", listing DejaVuSparseMLP.forward_sparse: gather the
 * selected fc1 rows, activation, gather the matching fc2 columns, project
 * down; DejaVuTransformerLayer.forward: pre-norm and residual add.)  For every
 * row b, with hn = norm(h1[b]; ln2_g, ln2_b) and i < *n_u_n, j = u_n[i]:
 *   a_i = max(0, hn . w1[j] + b1[j])
 *   y[b] = h1[b] + b2 + sum_i a_i * w2T[j]
 *   h1, y [B, d] binary32 device (may not alias); max_u_n = length of u_n.
 */
int dv_sparse_mlp(const dv_layer_desc *desc, const dv_layer_weights *w, const float *h1, int batch,
                  const int32_t *u_n, const int32_t *n_u_n, int max_u_n, float *y, void *ws,
                  size_t ws_bytes, void *stream);

/*
 * dv_layer_decode -- one sparse decode step of one layer: dv_predict_topk on
 * x_pred (x if NULL), then dv_sparse_attn and dv_sparse_mlp over the unions.
 * ("DejaVu Guide ...", listing DejaVuTransformerLayer.forward(x, x_prev,
 * k_heads, k_neurons).)
 *   h1: optional device output [B, d] of the attention block's result
 *       (NULL keeps it in the workspace).
 * Seven kernels (the predictors, QKV, attention, out-projection, fc1, fc2;
 * at batches 1-2 fc1 and fc2 are one pass plus a sum of partials) chained
 * by programmatic dependent launch.  Binary16 layers run QKV, fc1,
 * out-projection and fc2 on tensor cores from 3 batch rows and both
 * predictor stages from 5; there the stage-2 predictor -> QKV boundary is
 * in stream order, and from 8 rows every boundary is.  Serves every shape
 * and batch.
 */
int dv_layer_decode(const dv_layer_desc *desc, const dv_layer_weights *w, const float *x,
                    const float *x_pred, int batch, int k_heads, int k_neurons, void *k_cache,
                    void *v_cache, int kv_len, const dv_selection *sel, float *h1, float *y,
                    void *ws, size_t ws_bytes, void *stream);

/*
 * dv_layer_decode_chained -- the same call as dv_layer_decode (the name
 * states the launch structure for callers that compare the two paths).
 */
int dv_layer_decode_chained(const dv_layer_desc *desc, const dv_layer_weights *w, const float *x,
                            const float *x_pred, int batch, int k_heads, int k_neurons,
                            void *k_cache, void *v_cache, int kv_len, const dv_selection *sel,
                            float *h1, float *y, void *ws, size_t ws_bytes, void *stream);

/*
 * dv_layer_decode_persistent -- dv_layer_decode as ONE persistent streaming
 * kernel (binary16 layers with 128-wide heads, batches 1 and 2, shapes that
 * fit its tiling: see dv_layer_decode_persistent_ok; DV_ERR_UNSUPPORTED,
 * launching nothing, elsewhere).  A producer warp per SM streams every
 * selected weight row into a shared-memory ring with bulk copies while the
 * other warps compute; the steps hand over through counters in the
 * workspace (bounded waits; DV_ERR_TIMEOUT in the status word if one ran
 * out).  Same selections as the chain; sums in a different order, so the
 * outputs agree to rounding.  Measured slower than the chain at the
 * OPT-175B shape (about 250 against 128 us at batch 1), so not the default.
 * Arguments as dv_layer_decode.
 */
int dv_layer_decode_persistent(const dv_layer_desc *desc, const dv_layer_weights *w,
                               const float *x, const float *x_pred, int batch, int k_heads,
                               int k_neurons, void *k_cache, void *v_cache, int kv_len,
                               const dv_selection *sel, float *h1, float *y, void *ws,
                               size_t ws_bytes, void *stream);

/*
 * dv_layer_decode_stamped -- dv_layer_decode (persistent == 0) or
 * dv_layer_decode_persistent (persistent != 0) that also records a timeline
 * in stamps (device, 8-byte aligned): %globaltimer nanoseconds, G = the
 * device's SM count.  Points a CTA does not reach are left as they were.
 *   persistent == 0: n_stamps >= 7 * G * 8; kernel k of the chain (0 the
 *     first predictor, 1 the second, 2 QKV, 3 attention, 4 out-projection,
 *     5 fc1 or the one-pass MLP, 6 fc2 or the sum of the MLP's partials)
 *     writes for each of its CTAs c (first batch tile)
 *     stamps[(k * G + c) * 8 + i]: i = 0 the CTA starts, 1 its inputs are
 *     ready, 2 it ends, 3 the SM it ran on (%smid); 4 .. 7 points inside a
 *     kernel (attention: 4 warp 0's first batch of keys consumed, 5 warp
 *     0's keys done, 6 the chunk record written; the one-pass MLP: 4 its
 *     activations summed; row kernels: 4 activations staged, 5 rows done,
 *     6 a side CTA's selection done; column kernels: 4 the first
 *     coefficients staged, 5 the last piece consumed, 6 a block's combine
 *     starts; the sum of partials: 4 summed).  Slots a CTA never reaches
 *     keep what an earlier call wrote.
 *   persistent != 0: n_stamps >= 32 G; stamps[c * 32 + i] for CTA c at
 *     fixed points: its consumer warps: 0 start, 1 first predictor stage
 *     done, 2 predictor results complete, 3 neuron scoring starts, 4 done, 5
 *     selection pass done, 6/7 QKV start/done (last CTA: neuron selection
 *     start/done), 8/9 attention start/done, 10/11 out-projection
 *     coefficients start/done, 12 out-projection done, 13/14 h1 slice
 *     start/done, 15 norm statistics complete, 16 fc1 starts, 17 fc1 done,
 *     18 fc2 starts, 19 fc2 done, 20/21 y slice start/done; its producer
 *     warp: 24 + p when it starts issuing the copies of phase p (p = 0
 *     predictor, 1 neuron scorer, 2 QKV, 3 out-projection, 4 fc1, 5 fc2),
 *     30 when it has issued its last copy.  DV_ERR_UNSUPPORTED where the
 *     streaming kernel does not serve.
 * For profiling.
 */
int dv_layer_decode_stamped(const dv_layer_desc *desc, const dv_layer_weights *w, const float *x,
                            const float *x_pred, int batch, int k_heads, int k_neurons,
                            void *k_cache, void *v_cache, int kv_len, const dv_selection *sel,
                            float *h1, float *y, void *ws, size_t ws_bytes, int persistent,
                            unsigned long long *stamps, int n_stamps, void *stream);

/*
 * dv_layer_decode_presel -- the layer decode on a selection computed earlier:
 * dv_sparse_attn then dv_sparse_mlp in one call (five kernels, chained).
 * ("DejaVu Guide ...", "2. Pipelined Overlap Execution": the lookahead
 * predictor for layer l+1 runs while layer l computes, so by the time layer
 * l+1 starts its head and neuron sets are ready.)
 *   u_h / n_u_h (max_u_h), u_n / n_u_n (max_u_n): device unions, ascending,
 *   as dv_predict_topk writes them; x, y [B, d] binary32 device, distinct;
 *   h1 [B, d] optional output of the attention block (NULL: workspace).
 */
int dv_layer_decode_presel(const dv_layer_desc *desc, const dv_layer_weights *w, const float *x,
                           int batch, const int32_t *u_h, const int32_t *n_u_h, int max_u_h,
                           const int32_t *u_n, const int32_t *n_u_n, int max_u_n, void *k_cache,
                           void *v_cache, int kv_len, float *h1, float *y, void *ws,
                           size_t ws_bytes, void *stream);

/*
 * dv_layer_decode_traced -- dv_layer_decode that also records
 * events[0 .. dv_layer_decode_launches()] (cudaEvent_t handles created by the
 * caller): events[i] just before kernel i, the last one after the last
 * kernel.  For per-kernel timing; the events serialise the kernels.
 */
int dv_layer_decode_traced(const dv_layer_desc *desc, const dv_layer_weights *w, const float *x,
                           const float *x_pred, int batch, int k_heads, int k_neurons,
                           void *k_cache, void *v_cache, int kv_len, const dv_selection *sel,
                           float *h1, float *y, void *ws, size_t ws_bytes, void *const *events,
                           int n_events, void *stream);

/*
 * dv_layer_decode_host -- dv_layer_decode with HOST activations: copies
 * x_host [B, d] (and x_pred_host, may be NULL) from host memory into the
 * workspace, runs the step, copies y back to y_host [B, d] and synchronises
 * `stream` before returning.  Weights, KV cache and selection stay on the
 * device; `sel` may be NULL to keep the selection in the workspace.  Pinned
 * host memory gives asynchronous copies.
 */
int dv_layer_decode_host(const dv_layer_desc *desc, const dv_layer_weights *w, const float *x_host,
                         const float *x_pred_host, int batch, int k_heads, int k_neurons,
                         void *k_cache, void *v_cache, int kv_len, const dv_selection *sel,
                         float *y_host, void *ws, size_t ws_bytes, void *stream);

/*
 * dv_test_hold_wait -- TEST SUPPORT for the bounded waits of the streaming
 * kernel.  Arms the workspace so that the next streaming decode on it
 * (dv_layer_decode_persistent) gives every device-side wait a budget of `budget_us`
 * microseconds (> 0) and makes its wait number `wait_id` never complete:
 *   1 first predictor stage done      4 QKV done (attention starts)
 *   2 neuron scores done              5 attention done (out-projection)
 *   3 neuron selection pass done      6 out-projection partials of a group
 *   7 h1 and its norm statistics      8 fc1 done    9 fc2 partials of a group
 * That wait runs out: the kernel records DV_ERR_TIMEOUT in the status word
 * (dv_check), skips the rest of its work (outputs undefined), still returns,
 * and disarms the workspace and leaves it ready for the next call.
 * wait_id 0 disarms.  Enqueued on `stream` (a host-to-device copy of two
 * words into the workspace's control block).
 */
int dv_test_hold_wait(void *ws, size_t ws_bytes, int wait_id, int budget_us, void *stream);

/*
 * dv_hbm_copy -- copy `bytes` (a multiple of 16; both pointers 16-byte
 * aligned) from src to dst with a 16-byte-vector streaming kernel.  Used to
 * measure the copy bandwidth that serves as the roofline denominator.
 */
int dv_hbm_copy(void *dst, const void *src, size_t bytes, void *stream);

/*
 * dv_predict_topk_noalloc -- dv_predict_topk without a caller workspace.
 * This entry point is an addition of this library; the DejaVu pages have no
 * counterpart.  It is for callers that cannot provide device memory at the
 * point of prediction: a serving loop whose pool has already given all free
 * HBM to its KV cache, or code that must not call an allocator there because
 * cudaMalloc / cudaFree synchronise the device.  It allocates nothing.
 *
 * Computes exactly what dv_predict_topk computes (same kernels, same
 * arguments apart from the workspace).
 *
 * Scratch: a static device array of DV_NOALLOC_SCRATCH_BYTES inside this
 * library, one per device per process -- the exception to the "no state
 * outside the caller's workspace" convention above.  A shape and batch whose
 * scratch (status word, histograms, row counters, scores, partial sums,
 * bitmaps, candidates) does not fit is rejected with DV_ERR_SCRATCH_LIMIT and
 * nothing is launched; at the OPT-175B shape (N = 49152, r = 1000) the limit
 * is reached above batch 16.
 * Set-up: the first call on a device, with that device current, looks up the
 * scratch's device address (which may load the library's device code); the
 * address is kept per device and looked up again only when the device's CUDA
 * context has changed (for instance after cudaDeviceReset).  Make the first
 * call on a device before any stream capture begins.
 * Zeroing: every call first zeroes, on `stream`, the part of the scratch
 * that the kernels require to start at zero (status word, first-digit
 * histograms, candidate counters, row counters); everything else is written
 * before it is read.
 * Concurrency: calls whose execution overlaps on one device (different
 * streams, or different host threads) share the scratch and race; the
 * results are then wrong.  Serialise them.
 * Device-side status: none of the kernels this entry point runs records a
 * fault -- the predictor kernels read only whole weight rows inside their
 * matrices and the selection kernels take no caller indices -- so there is no
 * status word to read back (the workspace entries' dv_check has nothing to
 * report for this path either).
 */
#define DV_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)

int dv_predict_topk_noalloc(const dv_layer_desc *desc, const dv_layer_weights *w,
                            const float *x_pred, int batch, int k_heads, int k_neurons,
                            const dv_selection *sel, float *scores_h, float *scores_n,
                            void *stream);

/*
 * KV-cache operators: a cache that is written quantised and read back,
 * attention for a tree of drafted tokens over it, and attention over the
 * blocks of positions that a cheap score selects -- contextual sparsity along
 * the cached positions, beside the heads and neurons above.  They are an
 * addition of this library; the DejaVu pages have no counterpart.
 *
 * They serve caches of their own: every batch row has its own length (device
 * memory), query heads may share KV heads in groups of n_heads / n_kv_heads
 * (query head h reads KV head h / group), and rows may be held in 8 bits.
 * The conventions at the top of this file hold; the workspace is one of
 * dv_kv_workspace_size() bytes (not one of the layer calls'), zeroed once
 * with dv_workspace_init() and read by dv_check().  It may be shared by calls
 * of any shapes that fit it, one after another; calls, or graphs that hold
 * them, that may run at the same time need a workspace each (dv_tree_attn and
 * dv_block_attn keep pieces and counters in it).
 *
 * Device-side checks: a batch row whose length, token count, path or list of
 * blocks is out of range is skipped, its outputs and cache rows are left as
 * they were (a bad entry of a list of heads or blocks alone is skipped), and
 * DV_ERR_DEVICE_INDEX is recorded in the status word.
 *
 * Cache: k, v [B, Hkv, kv_cap, D] in desc.dtype.  DV_I8 holds a row of D
 * values as codes c in [-127, 127] (int8) and one scale s (k_scale, v_scale
 * [B, Hkv, kv_cap], binary32): value = c s, with s = max(amax |x| / 127,
 * 2^-126) and c = x / s rounded to the nearest whole number, ties to even
 * (both quotients in binary32).  A row that holds a NaN or an infinity is
 * stored with s = NaN and codes 0.
 * Block means (desc.block = n > 0): k_mean [B, Hkv, kv_cap / n, D] (int8) and
 * k_mean_scale [B, Hkv, kv_cap / n] hold the mean of the n keys of every
 * complete aligned block of positions, quantised like a row.  dv_kv_append
 * and dv_kv_keep write a block's mean when they write its last position (the
 * other n - 1 must be in the cache by then).  The mean's sum is taken over
 * the keys as stored, each rounded to a multiple of n 2^(e - 24) with 2^e the
 * power of two above the block's largest magnitude (e >= -100), so that it is
 * exact in any order.  A block with a NaN or an infinity, or whose mean rounds
 * to one, has codes 0 and scale +infinity.
 */
#define DV_KV_MAX_BATCH 256
#define DV_TREE_MAX_TOKENS 64

typedef struct {
    int32_t n_heads;    /* query heads: a multiple of n_kv_heads, at most 256 */
    int32_t n_kv_heads;
    int32_t head_dim;   /* power of two, at most 256; head_dim * sizeof(dtype) in [16, 512] */
    int32_t kv_cap;     /* positions per (batch row, KV head), at most 2^28 */
    int32_t dtype;      /* DV_F32, DV_F16 or DV_I8 */
    int32_t block;      /* 0 (no block means), or 16, 32, 64 or 128 <= kv_cap (head_dim >= 16,
                         * fewer than 16384 blocks) */
} dv_kv_desc;

typedef struct {
    void *k, *v;
    float *k_scale, *v_scale; /* DV_I8 only */
    int8_t *k_mean;           /* block > 0 only */
    float *k_mean_scale;
} dv_kv_cache;

/* Rows of head_dim contiguous values (DV_F32 or DV_F16): row (b, t, h) at
 * p + b stride_b + t stride_t + h stride_h, strides in elements, each a
 * non-negative multiple of 16 bytes (p 16-byte aligned); any slice of a
 * projection's output. */
typedef struct {
    const void *p;
    int32_t dtype;
    int64_t stride_b, stride_t, stride_h;
} dv_kv_rows;

/* Bytes of workspace the calls below need for this cache with up to `tokens`
 * query tokens a row (dv_tree_attn; 1 serves the others).  0 if invalid. */
size_t dv_kv_workspace_size(const dv_kv_desc *desc, int batch, int tokens);

/*
 * dv_kv_append -- write new keys and values, quantised for a DV_I8 cache.
 *   k, v: rows (b, t, h) of one type, t < tokens, h < n_kv_heads; token t of row b goes
 *   to position lens[b] + t, for t < n_tok[b] (n_tok [B], NULL: tokens).
 *   lens [B] device, lens[b] + n_tok[b] <= kv_cap; it is not advanced.  k and
 *   v must not overlap the cache.
 * Rounding to binary16 is to nearest (a value above 65504 becomes infinite).
 */
int dv_kv_append(const dv_kv_desc *desc, const dv_kv_cache *cache, const dv_kv_rows *k,
                 const dv_kv_rows *v, int batch, int tokens, const int32_t *lens,
                 const int32_t *n_tok, void *ws, size_t ws_bytes, void *stream);

/*
 * dv_kv_read -- read cached rows back as numbers: positions start[b] ..
 * start[b] + tokens - 1 of every head into k_out, v_out [B, Hkv, tokens, D]
 * in out_dtype (DV_F32, or DV_F16 rounded to nearest: the layout of a layer's
 * KV cache with kv_cap = tokens).  start[b] + tokens <= kv_cap.
 */
int dv_kv_read(const dv_kv_desc *desc, const dv_kv_cache *cache, int batch, int tokens,
               const int32_t *start, int out_dtype, void *k_out, void *v_out, void *ws,
               size_t ws_bytes, void *stream);

/*
 * dv_kv_keep -- after a draft has been verified: the cached rows of the
 * accepted path move together.  For i < n_keep[b], position lens[b] +
 * path[b][i] moves to lens[b] + i (codes and scales as they are).
 *   path [B, tokens] device, strictly ascending over its first n_keep[b]
 *   entries, each in [0, tokens); tokens <= DV_TREE_MAX_TOKENS.
 * Positions from lens[b] + n_keep[b] on keep what they held.
 */
int dv_kv_keep(const dv_kv_desc *desc, const dv_kv_cache *cache, int batch, int tokens,
               const int32_t *lens, const int32_t *path, const int32_t *n_keep, void *ws,
               size_t ws_bytes, void *stream);

/*
 * dv_tree_attn -- attention of the drafted tokens of every row over its
 * cached prefix and over each other.
 *   q: rows (b, t, h), t < tokens <= DV_TREE_MAX_TOKENS, h < n_heads.  The
 *   drafted tokens' own keys and values are in the cache at positions lens[b]
 *   + t (dv_kv_append), t < n_tok[b] (NULL: tokens).
 *   mask [B, tokens] device: bit j of mask[b][t]: token t sees drafted token
 *   j (itself included only if bit t is set; bits from n_tok[b] on are
 *   ignored).  NULL: token t sees drafted tokens 0 .. t.
 *   out [B, tokens, n_heads, D] binary32:
 *     out[b, t, h] = sum_p softmax_p(scale q . k_p) v_p
 *   over positions p < lens[b] and the drafted ones it sees; zeros where it
 *   sees none (scale log2(e) must be finite).  Tokens t >= n_tok[b] and heads
 *   that are not listed are left as they were.  A position that a token does
 *   not see cannot change its result, whatever it holds, nor can another token's
 *   query; a value row that it sees and that holds a NaN or an infinity, or a
 *   key row with a NaN, makes the result non-finite.  A key row with an infinity
 *   does so too, or counts as unseen (a score of -infinity).
 *   u_h, n_u_h, max_u_h: device list of distinct KV heads to compute, as
 *   dv_sparse_attn's (NULL, NULL, 0: every head; max_u_h <= n_kv_heads).
 * tokens = 1 is decode attention with one length a row.  Scores, weights and
 * sums are held in binary32 for every cache type.  The tensor-core kernels
 * (binary16 and 8-bit rows of 64 or 128 values) come near a binary32
 * evaluation, not to its last bit: a query element is two binary16 parts
 * (exact to 2^-22 of itself, or 2^-38 of its row's largest), a weight (with its
 * value row's scale) two parts (2^-22 of itself, or 2^-30 of the row's largest),
 * 2^x has a relative error of up to 2^-22, and up to 128 steps come between binary32
 * additions, of which each cuts 16 terms and their sum off (by up to 5.25 x 2^-23 of
 * the sum of the terms' sizes: 8e-5 in all at most, 6e-5 seen where one term
 * outweighs all others).  This holds for
 * 8-bit value rows with scales from 2^-60 to 2^100, and rows of zeros among
 * them, and key rows with scales up to 2^98; smaller values lose bits, larger
 * numbers overflow.  One launch; the order of every sum is fixed by the shapes,
 * the lengths and the device.
 */
int dv_tree_attn(const dv_kv_desc *desc, const dv_kv_cache *cache, const dv_kv_rows *q, int batch,
                 int tokens, const int32_t *lens, const int32_t *n_tok, const uint64_t *mask,
                 float scale, const int32_t *u_h, const int32_t *n_u_h, int max_u_h, float *out,
                 void *ws, size_t ws_bytes, void *stream);

/* Kernel of dv_tree_attn for more than 8 query rows per KV head (tokens x
 * group) over binary16 and 8-bit rows of 64 or 128 values, process-wide, for
 * calls issued after it returns:
 *   0  the faster one by the sizes known on the host (the default);
 *   1  mma.sync, 8 query rows at a time (the cache is read once for every 8);
 *   2  tcgen05, 64 query rows at a time.
 * Results agree within the binary32 error; the bits may not.
 * DV_ERR_INVALID_ARG for another value.  Not thread-safe against calls in
 * flight on other threads. */
dv_status dv_set_tree_kernel(int variant);

/*
 * dv_block_topk -- the blocks of cached positions each query attends to.
 * desc.block = n > 0; row b has nb = ceil(lens[b] / n) blocks.
 *   q: rows (b, 0, h) (stride_t is not used), one query per row and head.
 *   Score of block j: the query is quantised like a cached row to codes qc;
 *   score = float(sum_d qc_d k_mean[j]_d) k_mean_scale[j] (the sum is a whole
 *   number below 2^24), +infinity where the scale is.
 *   The first n_first and the last n_last >= 1 blocks are taken, and of the
 *   others the k_blocks - n_first - n_last with the largest scores (ties to
 *   the lower block).
 *   idx [B, n_heads, k_blocks]: ascending; -1 behind the last of nb blocks.
 * The workspace holds its status word only.
 */
int dv_block_topk(const dv_kv_desc *desc, const dv_kv_cache *cache, const dv_kv_rows *q, int batch,
                  const int32_t *lens, int k_blocks, int n_first, int n_last, int32_t *idx,
                  void *ws, size_t ws_bytes, void *stream);

/*
 * dv_block_attn -- attention of one query per row and head over its listed
 * blocks (positions p < lens[b] of them).
 *   idx [B, n_heads, k_blocks]: distinct blocks in any order, -1 for none;
 *   only the first min(k_blocks, ceil(lens[b] / n)) entries are read.
 *   out [B, n_heads, D] binary32; zeros where no position is left.
 * Arithmetic as dv_tree_attn's.
 */
int dv_block_attn(const dv_kv_desc *desc, const dv_kv_cache *cache, const dv_kv_rows *q, int batch,
                  const int32_t *lens, const int32_t *idx, int k_blocks, float scale, float *out,
                  void *ws, size_t ws_bytes, void *stream);

/*
 * Packed sequences and paged caches: what a serving step does with prompts and
 * with requests that share one pool of pages.  The new tokens of B requests lie
 * one behind the other, request b's at rows cu[b] .. cu[b + 1] - 1 (cu [B + 1],
 * device), any number of them from none to a whole prompt; request b has
 * lens[b] cached positions before them.  They are an addition of this library;
 * the DejaVu pages have no counterpart.
 *
 * The conventions at the top of this file hold; the workspace is one of
 * dv_seq_workspace_size() bytes, zeroed once with dv_workspace_init() and read
 * by dv_check().  It serves calls of any batch and length, one after another;
 * calls, or graphs that hold them, that may run at the same time need one each.
 * Query heads share KV heads in groups of n_heads / n_kv_heads.
 *
 * Device-side checks: a request whose offsets, length or token count are out of
 * range is skipped, what it would write is left as it was, and
 * DV_ERR_DEVICE_INDEX is recorded in the status word.  A page number out of
 * range in a block table is recorded too: dv_page_take gives its tokens slot
 * -1, dv_paged_attn reads its positions as zeros.
 *
 * Pool: k, v [n_pages, Hkv, page, D] in desc.dtype: position p of request b and
 * head h is row p % page of (tables[b][p / page], h).  Block tables: tables [B,
 * max_pages] page numbers, of which the first ceil(length / page) of a row
 * count; max_pages x page <= 2^30.  Slot of a token: page number x page + row.
 */
#define DV_SEQ_MAX_BATCH 1024

typedef struct {
    int32_t n_heads;    /* query heads: a multiple of n_kv_heads, at most 256 */
    int32_t n_kv_heads;
    int32_t head_dim;   /* power of two, 8 to 256, at most 512 bytes */
    int32_t dtype;      /* DV_F32 or DV_F16 */
    int32_t page;       /* positions a page: 16, 32, 64 or 128; 0: no pool (dv_qk_rope to rows,
                         * dv_prompt_attn) */
    int32_t n_pages;    /* pages of the pool, n_pages x page <= 2^30 (0 without a pool) */
} dv_seq_desc;

typedef struct {
    void *k, *v;
} dv_page_pool;

/* Bytes of workspace of the calls below.  0 if invalid. */
size_t dv_seq_workspace_size(const dv_seq_desc *desc);

/*
 * dv_page_release -- give back the pages of requests that have finished.
 *   free_pages [n_pages] device: a stack of page numbers, n_free[0] of them.
 *   done [B]: of requests with done[b] != 0 the pages of their first lens[b]
 *   positions are pushed, in the order of the requests and positions;
 *   n_free_out[0] (may be n_free) gets the new count.  tables and lens stay as
 *   they are.  A request with a page number out of range, or whose pages would
 *   not fit the stack, is skipped and recorded (DV_ERR_DEVICE_INDEX).
 */
int dv_page_release(const dv_seq_desc *desc, int batch, const int32_t *lens, const int32_t *done,
                    int max_pages, const int32_t *tables, int32_t *free_pages,
                    const int32_t *n_free, int32_t *n_free_out, void *ws, size_t ws_bytes,
                    void *stream);

/*
 * dv_page_take -- block tables and slots for n_tok[b] new tokens a request.
 *   Request b needs ceil((lens[b] + n_tok[b]) / page) - ceil(lens[b] / page) new
 *   pages; they are popped from the stack (free_pages, n_free as above) in the
 *   order of the requests and written behind the first ceil(lens[b] / page)
 *   entries of its table; n_free_out[0] (may be n_free) gets the new count.
 *   lens is not advanced.
 *   cu [B + 1]: offsets of the packed tokens; pos [max_tokens], slots
 *   [max_tokens]: each token's position and slot, -1 behind the last one.
 *   A request that the stack has too few pages for, those before it served,
 *   takes none: its tokens keep their places with slot -1 (nothing stores them, and
 *   attention over its pages has no meaning in this step), and DV_ERR_PAGES is
 *   recorded.  A request out of range (lens[b] + n_tok[b] > max_pages x page)
 *   counts as one of no tokens.  Offsets stop at max_tokens (recorded).
 */
int dv_page_take(const dv_seq_desc *desc, int batch, const int32_t *lens, const int32_t *n_tok,
                 int max_pages, int32_t *tables, const int32_t *free_pages, const int32_t *n_free,
                 int32_t *n_free_out, int32_t *cu, int32_t *pos, int32_t *slots, int max_tokens,
                 void *ws, size_t ws_bytes, void *stream);

/* How positions are scaled for contexts longer than the trained one.  With f_i
 * = theta^(-2 i / rot_dim) the angle of pair i per position:
 *   DV_ROPE_NONE    f_i
 *   DV_ROPE_LINEAR  f_i / factor
 *   DV_ROPE_BASE    f_i of theta factor^(rot_dim / (rot_dim - 2))
 *   DV_ROPE_RAMP    f_i (w + (1 - w) / factor), w rising from 0 to 1 as the
 *                   turns over the trained length, orig_len f_i / 2 pi, rise
 *                   from low to high
 *   DV_ROPE_RAMP_INDEX  the same with w = 1 - (i - a) / (b - a) held within 0 .. 1:
 *                   falling over the pairs a = max(floor(dim(high)), 0) to b =
 *                   min(ceil(dim(low)), rot_dim - 1) (b + 0.001 where they are
 *                   equal), dim(r) = rot_dim ln(orig_len / 2 pi r) / (2 ln theta):
 *                   the pair that makes r turns */
typedef enum {
    DV_ROPE_NONE = 0,
    DV_ROPE_LINEAR = 1,
    DV_ROPE_BASE = 2,
    DV_ROPE_RAMP = 3,
    DV_ROPE_RAMP_INDEX = 4
} dv_rope_scaling;

/* The angles as the kernel takes them, turns per position in units of 2^-64:
 * steps (HOST) [rot_dim / 2], to be copied to the device once.  A step is the exact
 * angle of these parameters rounded to the nearest unit, and a kernel's angle its
 * product with the position modulo 2^64: off by at most half a unit a position,
 * 2^-35 of a turn at position 2^30.  theta > 1, 1 <= factor, orig_len, low < high
 * where used. */
int dv_rope_steps(int rot_dim, double theta, int scaling, double factor, double orig_len,
                  double low, double high, uint64_t *steps);

typedef struct {
    const uint64_t *steps;  /* [rot_dim / 2] device (any angles of at most half a turn a position) */
    int32_t rot_dim;        /* even, 0 (no rotation) to head_dim: the first rot_dim values turn */
    int32_t interleaved;    /* 0: pairs (i, i + rot_dim / 2); 1: pairs (2 i, 2 i + 1) */
    float mscale;           /* factor of sines and cosines (1 unless the scaling has one) */
    int32_t norm;           /* dv_norm, over a head's D values, where there are gains */
    float eps;              /* > 0 */
    const float *q_gain, *k_gain;  /* [head_dim] device; NULL: queries (keys) as they are */
} dv_rope;

/*
 * dv_qk_rope -- normalise and rotate the queries and keys of packed tokens, and
 * store keys and values in the pool, in one pass.
 *   q, k, v: rows (t, h) (stride_b is not used), t < tokens; v NULL: no values.
 *   pos [tokens] device: positions; a token with a negative one is skipped.
 *   x' = x / sqrt(mean(x^2) + eps) gain (DV_LAYERNORM: of x less its mean), then
 *   each pair turns by its angle: (a, b) -> (a cos - b sin, b cos + a sin).  Values
 *   behind the first rot_dim do not turn: they are kept, infinities and NaN too.
 *   q_out: rows of the queries; may be q itself (same place, type, strides).
 *   k_out: rows of the keys, or NULL; may be k.  pool, slots [tokens]: where keys
 *   and values go (NULL: nowhere); a negative slot takes nothing, one out of
 *   range neither (recorded).  v goes to the pool alone, as it is.
 * Outputs otherwise overlap nothing.  Arithmetic is binary32; an angle is that of
 * its step to 2^-33 of a turn at any position, a sine or cosine within 2^-22 of the
 * angle's; a row is rounded once, when it is stored.
 */
int dv_qk_rope(const dv_seq_desc *desc, const dv_rope *rope, int tokens, const int32_t *pos,
               const dv_kv_rows *q, const dv_kv_rows *k, const dv_kv_rows *v,
               const dv_kv_rows *q_out, const dv_kv_rows *k_out, const dv_page_pool *pool,
               const int32_t *slots, void *ws, size_t ws_bytes, void *stream);

/*
 * dv_prompt_attn -- causal attention of packed prompts over themselves.
 *   q, k, v: rows (t, h) of desc.dtype, t < tokens (strides of rows that differ
 *   are at least D).  cu [batch + 1]: request b has rows cu[b] .. cu[b + 1] - 1,
 *   0 <= cu[b] <= cu[b + 1] <= tokens, at most max_tok of them.
 *   out [tokens, n_heads, D] of desc.dtype:
 *     out[cu[b] + i, h] = sum_{j <= i} softmax_j(scale q_i . k_j) v_j
 *   Rows of no request are left as they were.  scale log2(e): a positive normal
 *   number.
 * A row's result depends on the rows it sees alone, whatever others hold; a
 * value row that it sees and that holds a NaN or an infinity, or a key row with
 * a NaN, makes the result non-finite (every value of it, or that dimension's).
 * Scores, sums and outputs are held in binary32.  Binary16 rows of 64 or 128
 * values run on tensor cores (tcgen05): a weight is rounded to binary16 (2^-11
 * of itself, or 2^-31 of the row's largest) for its value and for the sum; all
 * other arithmetic is binary32, of which tensor cores cut sums off instead of rounding
 * them: outputs lose at most 5.25 x 2^-15 (1.6e-4) of the sum of their terms' sizes, a
 * score 2^-17 of its products'.  A row whose seen scores are all -infinity (infinite
 * keys) gives 0.  The order of every sum is fixed by the shapes, max_tok, the lengths
 * and the device.
 * max_tok is what the host knows of the requests: it decides the kernel and how many
 * query heads share a unit of work.  A loose bound gives the same results to rounding,
 * but may cost time: one token of each of 20 requests, 40 heads on 8, 4096 positions
 * takes 73 us with max_tok = 1 and 279 with 20.
 */
int dv_prompt_attn(const dv_seq_desc *desc, int batch, int tokens, int max_tok,
                   const dv_kv_rows *q, const dv_kv_rows *k, const dv_kv_rows *v,
                   const int32_t *cu, float scale, void *out, void *ws, size_t ws_bytes,
                   void *stream);

/*
 * dv_paged_attn -- causal attention of every request's new tokens over its
 * pages.  Their own keys and values are in the pool already, at positions
 * lens[b] + i (dv_qk_rope); one token a request is decode attention.
 *   q: rows (t, h) of desc.dtype; cu, max_tok, scale, out as dv_prompt_attn's;
 *   lens [batch], tables [batch, max_pages]; lens[b] + count <= max_pages x page.
 *     out[cu[b] + i, h] = sum_{p <= lens[b] + i} softmax_p(scale q_i . k_p) v_p
 * Arithmetic and what cannot change a result as dv_prompt_attn's.
 */
int dv_paged_attn(const dv_seq_desc *desc, const dv_page_pool *pool, int batch, int tokens,
                  int max_tok, const dv_kv_rows *q, const int32_t *cu, const int32_t *lens,
                  const int32_t *tables, int max_pages, float scale, void *out, void *ws,
                  size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DV_H */
