/*
 * effort.h -- C ABI of the B200 (sm_100a) library for the "Effort"
 * approximate matrix-vector multiply.
 *
 * The method (Hacker News item 40067677, "Show HN: Speeding up LLM inference
 * 2x times (possibly)", the pseudo-code quoted in a commenter's question and
 * the author's replies): every row of the weight matrix is stored sorted by
 * |w| descending; per call, an input vector v and an effort in (0, 1] pick a
 * cutoff c from per-row probes (cutoff_chart = v * probes, cutoff =
 * topK(chart, effort)), and only the products with |v_i| * |w_ij| >= c are
 * multiplied and added.  The author's complexity reply (Hacker News item
 * 40095016) gives O(effort * inDim * outDim) multiplications, O(inDim) for the
 * dispatch and about O(inDim log inDim) for the cutoff.
 *
 * Conventions (all entry points):
 *  - W is [in_dim x out_dim] binary16 (or, for effort_prepare_q8, int8 with one
 *    binary16 scale per row), row-major: row i holds the weights that
 *    multiply v[i], and out[j] = sum_i v[i] * W[i][j] (the matrix is already
 *    "flipped" in the sense of the pages).
 *  - Pointers named W, v, V, out, OUT, *_out are DEVICE pointers unless stated.
 *    The caller owns them; the library never frees them.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *  - Every call returns an effort_status_t.  Argument errors are detected on
 *    the host before anything is launched.  No exception or abort crosses the
 *    ABI.  Device faults are never used to signal errors.
 *  - Selection rule: a kept pair (i, j) is used iff the single-precision
 *    product fl32(|v_i| * |w_ij|) (round to nearest even, no FMA, no flush to
 *    zero) is >= c.  Ties at c are used.  Outputs are accumulated in fp32.
 */
#ifndef EFFORT_H
#define EFFORT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct effort_handle_s* effort_handle_t;        /* prepared matrix, library-owned */
typedef struct effort_workspace_s* effort_workspace_t;  /* per-call scratch, library-owned */

typedef enum {
  EFFORT_OK = 0,
  EFFORT_ERR_ARG = 1,          /* bad pointer, size, effort, keep fraction or dtype */
  EFFORT_ERR_CUDA = 2,         /* a CUDA runtime call or kernel launch failed */
  EFFORT_ERR_NOMEM = 3,        /* device or host allocation failed */
  EFFORT_ERR_NONFINITE = 4,    /* W (prepare) or v (reported by effort_check) held inf/NaN */
  EFFORT_ERR_DEVICE = 5,       /* a kernel reported an internal inconsistency or a wait timed out */
  EFFORT_ERR_UNSUPPORTED = 6   /* sizes outside the limits stated below */
} effort_status_t;

/* EFFORT_BF16 is taken by the feed-forward operators below; the Effort matvec
 * entry points take EFFORT_F32 and EFFORT_F16 and refuse it. */
typedef enum { EFFORT_F32 = 0, EFFORT_F16 = 1, EFFORT_BF16 = 2 } effort_dtype_t;

/* Size limits of this build. */
#define EFFORT_MAX_OUT_DIM 32768      /* a row is sorted inside one thread block */
#define EFFORT_MAX_IN_DIM 40960       /* a block's share of the chart lives in its shared memory */
#define EFFORT_STATIC_SCRATCH_BYTES (8u << 20) /* per-device scratch of effort_gemv_static */

/*
 * effort_prepare -- the offline pass: `precompute(W)` of the pages.
 *   Sorts every row of W by |w| descending (ties: lower column first), keeps
 *   the first n = floor(keep_fraction * out_dim + 1/2) entries of each row
 *   (the post text: the format lets the loader skip the least important
 *   weights), takes 16 midpoint-rank probes per row, and stores, for every row
 *   and every panel of 2048 output columns, the leading 3/8 of the row's kept
 *   entries in that panel in rank order, cut into chunks of 64 slots (each
 *   chunk sorted by column: fp16 value + 8-bit column gap); plus a dense copy
 *   of the kept weights for rows a call uses beyond that share.
 *   W: device, binary16 [in_dim x out_dim], 2-byte aligned; read only during
 *      the call (the stream is synchronised before returning; the caller may
 *      free W afterwards).
 *   keep_fraction: (0, 1].  Must keep at least one weight per row.
 *   Limits: 1 <= out_dim <= EFFORT_MAX_OUT_DIM, 1 <= in_dim <= EFFORT_MAX_IN_DIM,
 *           in_dim * out_dim < 2^32.
 *   Returns EFFORT_ERR_NONFINITE (and no handle) if W holds inf or NaN, and
 *   EFFORT_ERR_NOMEM if a device allocation fails or would take the library's
 *   device memory past the cap set by the environment variable
 *   EFFORT_ALLOC_CAP_BYTES (read at each allocation; unset = no cap).
 *   On success *out_handle owns all device storage; free it with effort_destroy.
 */
effort_status_t effort_prepare(const void* W, int64_t in_dim, int64_t out_dim, float keep_fraction,
                               void* stream, effort_handle_t* out_handle);

/*
 * effort_prepare_q8 -- effort_prepare for Q8 weights: int8 values q and one
 *   binary16 scale per row, the weight being w_ij = s_i * q_ij, taken exactly
 *   (the post says Q8 is in the works and the author that the algorithm
 *   should work on top of Q8: Hacker News item 40067677, "Show HN: Speeding
 *   up LLM inference 2x times (possibly)", the post text and the author's
 *   replies).  Everything the matvec computes follows from those weights as
 *   for effort_prepare: row order |w| descending with ties to the lower
 *   column, keep, probes, the cutoff c, the used set fl32(|v_i| |w_ij|) >= c
 *   and out.  The stored matrix holds q as int8: 2 bytes per chunk slot
 *   (value and gap) and 1 byte per column of the dense copy.
 *   q: device int8 [in_dim x out_dim], row-major (row i multiplies v[i]);
 *   scales: device binary16 bits [in_dim], 2-byte aligned, finite (zero and
 *   negative scales are allowed); both are read during the call only (the
 *   handle keeps its own copy of the scales).
 *   keep_fraction, stream, out_handle and the limits: as for effort_prepare.
 *   Returns EFFORT_ERR_NONFINITE if a scale is inf or NaN, EFFORT_ERR_ARG for
 *   a null or misaligned pointer or a bad keep_fraction.  Every matvec entry
 *   point accepts the handle (the dense baseline is for binary16 only).
 */
effort_status_t effort_prepare_q8(const int8_t* q, const uint16_t* scales, int64_t in_dim, int64_t out_dim,
                                  float keep_fraction, void* stream, effort_handle_t* out_handle);

/*
 * effort_gemv -- one approximate matvec: `approxMul(v, ...)` of the pages.
 *   v: device fp32 [in_dim]; out: device fp32 [out_dim], fully overwritten.
 *   effort in (0, 1]: K = llround(effort * in_dim * out_dim) products are
 *   targeted; the cutoff c is the weighted K-th largest entry of the chart
 *   fl32(|v_i| * probe_ik) (c = 0 if K >= the kept count, c = +inf if K = 0).
 *   Asynchronous and stream-ordered: no host synchronisation and no
 *   allocation; one kernel whose blocks (one per SM) compute the cutoff,
 *   the dispatch and the multiply-accumulate, meeting at grid-wide barriers.
 *   out is accumulated in fp32 with reductions whose order varies from call
 *   to call: c, |S| and the L_i are reproducible bit for bit, out to rounding.
 *   Each barrier wait has a time limit (0.2 s); a wait that runs out sets a
 *   status bit that effort_check reports as EFFORT_ERR_DEVICE.
 *   A handle holds one call's scratch: calls on the same handle must be
 *   ordered (same stream, or synchronised); concurrent calls on one handle race.
 */
effort_status_t effort_gemv(effort_handle_t h, const float* v, float effort, float* out, void* stream);

/*
 * effort_gemv_ex -- effort_gemv with a v dtype and optional device outputs.
 *   v: device, EFFORT_F32 or EFFORT_F16, [in_dim].
 *   cutoff_out: nullable device float, receives c.
 *   count_out: nullable device uint64, receives |S|, the number of used products.
 *   rowlen_out: nullable device uint32 [in_dim], receives L_i, the number of
 *     used products of row i (always a leading part of row i's sorted order).
 */
effort_status_t effort_gemv_ex(effort_handle_t h, const void* v, effort_dtype_t v_dtype, float effort,
                               float* out, float* cutoff_out, uint64_t* count_out, uint32_t* rowlen_out,
                               void* stream);

/*
 * effort_gemv_host -- effort_gemv_ex on HOST buffers, for callers that hold v
 *   and want out in host memory.  The pages have no counterpart: this is a
 *   library service around the same matvec.  On `stream`, in order, the same
 *   kernel as effort_gemv_ex, with v (in_dim elements of v_dtype) and out
 *   (out_dim fp32) moved across the host link as follows:
 *   - v is copied into the handle's device staging buffer with one
 *     cudaMemcpyAsync before the kernel (every block of the kernel reads v,
 *     so reading it in place across the host link would cost a host-link
 *     round trip per block);
 *   - out is accumulated in the staging buffer (the kernel adds partial sums
 *     into it with device-memory reductions).  When out_host is page-locked
 *     memory mapped into the device's address space (cudaHostAlloc,
 *     cudaMallocHost, cudaHostRegister with mapping; cudaPointerGetAttributes
 *     decides), the kernel's last block writes the finished out into it;
 *     otherwise it is copied back with one cudaMemcpyAsync after the kernel
 *     (CUDA stages copies to pageable memory, which may block the host).
 *   v_host, out_host: host memory, non-NULL.
 *   The call does not synchronise: out_host holds the result once the stream
 *   has passed this call (cudaStreamSynchronize, an event).  The caller must
 *   not modify v_host or read out_host before then.
 *   The staging buffer (in_dim x 4 + out_dim x 4 bytes) is allocated by
 *   effort_prepare and belongs to the handle: calls on one handle must be
 *   ordered (one stream), like the handle's workspace.
 */
effort_status_t effort_gemv_host(effort_handle_t h, const void* v_host, effort_dtype_t v_dtype, float effort,
                                 float* out_host, void* stream);

/*
 * effort_gemv_timed -- effort_gemv_ex (no optional outputs) that also stores
 *   the GPU global timer (ns) at fixed points of the call, for per-phase
 *   timing: marks is a device uint64 array [blocks][16] (blocks from
 *   effort_grid_blocks); entry k of block b is written by that block when it
 *   reaches point k: 0 start, 1 after waiting for the preceding grid, 2 chart
 *   histogram, entries and bin descriptors written, 3 after the first grid
 *   barrier, 4 crossing bin found, 5 the crossing bin's entries gathered
 *   (not reached with more than 4096 of them), 6 cutoff resolved, 7 work
 *   lists built,
 *   8 dense units streamed, 9 sparse chunks streamed, 10 registers added into
 *   the panel accumulator, 11 the block's sums added into out, 13 the block is
 *   done (12, 14 and 15 are not used); 8 and 9 are written by lane 0 of every
 *   warp (the last write stays).  Points a call does not reach (effort 1
 *   skips 2..5, a tiny effort returns after 1) keep their old
 *   contents.  The pages have no counterpart: a measurement service.
 */
effort_status_t effort_gemv_timed(effort_handle_t h, const void* v, effort_dtype_t v_dtype, float effort,
                                  float* out, uint64_t* marks, void* stream);

/* Blocks of the grid a matvec on this handle launches (one per SM). */
effort_status_t effort_grid_blocks(effort_handle_t h, int32_t* blocks);

/*
 * effort_gemv_static -- effort_gemv_ex (without rowlen_out) whose per-call
 *   scratch is a fixed array of EFFORT_STATIC_SCRATCH_BYTES (8 MiB) per device,
 *   compiled into the library, instead of the handle's workspace.  The pages
 *   have no counterpart: this is a library service, not part of the method.
 *   It is for callers that must not allocate device memory on the call path,
 *   e.g. code running under another component's allocator (a caching
 *   allocator that must account for every byte, a memory pool sized up
 *   front), or that needs its device footprint fixed before the first call.
 *   The call allocates nothing: no cudaMalloc, no cudaFree, no allocating
 *   library routine.  It issues one cudaMemsetAsync that clears the scratch
 *   words that must start at zero, the same kernel as effort_gemv_ex, and,
 *   if status_out is given, one 4-byte device-to-device copy.
 *   v, v_dtype, effort, out, cutoff_out, count_out: as for effort_gemv_ex.
 *   status_out: nullable device uint32; receives 0 if the call saw only
 *     finite entries of v and no internal inconsistency, nonzero otherwise
 *     (the output is then unspecified).  effort_check does not see this call.
 *   Set-up: the first call on a device looks up that device's copy of the
 *     array (cudaGetSymbolAddress, with the handle's device made current);
 *     make that first call before any stream capture on the device.
 *   Every call on one device shares the array: calls that may overlap on the
 *     GPU (unordered streams, concurrent host threads) race and give wrong
 *     results; order them on one stream.
 *   Returns EFFORT_ERR_UNSUPPORTED when the handle's geometry needs more than
 *     EFFORT_STATIC_SCRATCH_BYTES of scratch (a geometry needs about 2.4 MiB
 *     of histograms and bin descriptors on a 148-SM device plus 128 bytes per
 *     input row for the chart entries: 3.0 MiB at in_dim 4096, 7.7 MiB at
 *     EFFORT_MAX_IN_DIM), and when the device ordinal is 64 or above.
 *   The array's address is looked up again whenever the device's primary
 *     context has changed (after cudaDeviceReset), never kept across it.
 */
effort_status_t effort_gemv_static(effort_handle_t h, const void* v, effort_dtype_t v_dtype, float effort,
                                   float* out, float* cutoff_out, uint64_t* count_out, uint32_t* status_out,
                                   void* stream);

/*
 * effort_check -- synchronises the handle's last stream and reports whether a
 *   call since the previous check saw a non-finite entry of v
 *   (EFFORT_ERR_NONFINITE; those calls' outputs are unspecified) or a device
 *   inconsistency: a grid-wide wait that ran out of time, or, in a library
 *   built with -DEFFORT_DEBUG, an index a kernel found out of range
 *   (EFFORT_ERR_DEVICE; outputs of the calls since the previous check are
 *   unspecified).  Clears the flags; after an error it also resets the
 *   handle's scratch, so that later calls start clean.
 */
effort_status_t effort_check(effort_handle_t h);

/*
 * Workspaces: scratch for effort_gemv_batched and effort_dense_gemv.
 *   Sized for matrices of in_dim x out_dim and up to max_pairs concurrent pairs
 *   per call (max_pairs >= 1).  Allocates device memory (not stream-ordered).
 */
effort_status_t effort_workspace_create(int64_t in_dim, int64_t out_dim, int32_t max_pairs,
                                        effort_workspace_t* out_ws);
effort_status_t effort_workspace_destroy(effort_workspace_t ws);

/*
 * effort_gemv_batched -- n_pairs independent matvecs (MoE-style routing: each
 *   vector meets the experts it was routed to; the author's complexity reply
 *   likens the per-multiplication choice of buckets to expert routing).
 *   Pair p uses handles[hidx[p]], vector V + vidx[p] * in_dim (dtype v_dtype),
 *   efforts[p], and writes OUT + p * out_dim (fp32).  hidx, vidx, efforts:
 *   HOST arrays of n_pairs entries.  All handles must share in_dim/out_dim
 *   with the workspace.  cutoffs_out [n_pairs] float and counts_out
 *   [n_pairs] uint64 are nullable device arrays.  One cutoff per pair.
 *   Two pairs on the same handle whose cutoffs both select (0 < K < the kept
 *   count) run as one kernel that reads the union of their prefixes once:
 *   each (row, panel) of the matrix is read as far as the lower of the two
 *   thresholds needs, and each vector's own threshold is applied to it, so
 *   each pair's cutoff, count and output are those of its own call (outputs
 *   to rounding).  Every other pair runs as one kernel of its own.  All
 *   kernels run in order on `stream` and share the workspace's scratch (two
 *   slots, the second allocated when max_pairs >= 2).  n_pairs <= the
 *   workspace's max_pairs.
 */
effort_status_t effort_gemv_batched(effort_workspace_t ws, const effort_handle_t* handles, const int32_t* hidx,
                                    const int32_t* vidx, int32_t n_pairs, const void* V, effort_dtype_t v_dtype,
                                    const float* efforts, float* OUT, float* cutoffs_out, uint64_t* counts_out,
                                    void* stream);

/*
 * effort_dense_gemv -- the dense baseline out = W^T v (every weight, fp32
 *   accumulation), hand-written streaming kernel.  W: device binary16
 *   [in_dim x out_dim], out_dim a multiple of 8, 16-byte aligned.  v: fp32 or
 *   fp16 [in_dim].  Uses the workspace's first pair slot.
 */
effort_status_t effort_dense_gemv(effort_workspace_t ws, const void* W, int64_t in_dim, int64_t out_dim,
                                  const void* v, effort_dtype_t v_dtype, float* out, void* stream);

/* Sizes and footprint of a prepared matrix (device_bytes: its stored format,
 * not counting the per-call scratch and staging buffer). */
effort_status_t effort_get_info(effort_handle_t h, int64_t* in_dim, int64_t* out_dim, float* keep_fraction,
                                size_t* device_bytes);

/*
 * effort_layout_t -- read-only view of a handle's device storage, for format
 * checks.  Panel p covers columns [panel_width p, panel_width (p + 1)).
 * lists: [in_dim][n_panels] of {first chunk, stored chunks, tail, kept}: list
 *   (i, p) holds the kept entries of row i in panel p in row i's order (|w|
 *   descending, ties: lower column); its leading ceil(kept * store_num /
 *   store_den) entries are stored in chunks [first, first + stored chunks);
 *   tail is the |w| binary16 bits of the first entry not stored (0 if none).
 * vals / gaps: chunk c occupies slots [chunk_slots c, chunk_slots (c + 1)):
 *   binary16 value bits and 8-bit column gaps.  The slots of a chunk are in
 *   column order; the column of a slot is -1 + the sum of the gaps up to and
 *   including it (panel-local).  Filler slots (value +0, gap 255) bridge gaps
 *   above 255; pad slots (value +0, gap 0) fill the chunk.
 * head: [total_chunks] |w| bits of each chunk's first (largest) rank.
 * wdense: [in_dim][dense_stride] binary16: kept weights at their columns, +0
 *   elsewhere.  probes: [in_dim][16] |w| bits at the probe ranks (0 for empty
 *   segments).  scratch_bytes: the handle's per-call scratch.
 * weight_kind: 0 for a matrix from effort_prepare, 1 for one from
 *   effort_prepare_q8.  For Q8, vals and wdense hold int8 q (1 byte per slot
 *   or column), tail, head and probes hold the binary16 bits of |q| (0 on a
 *   row whose scale is 0), and scales is the handle's copy of the row
 *   scales [in_dim] (binary16); null for fp16.
 */
typedef struct {
  int64_t in_dim, out_dim;
  int32_t n_kept, n_panels, panel_width, chunk_slots, store_num, store_den, n_probes, dense_stride;
  uint32_t total_chunks;
  const void* vals;
  const void* gaps;
  const void* head;
  const void* lists;
  const void* wdense;
  const void* probes;
  size_t scratch_bytes;
  int32_t weight_kind;
  const void* scales;
} effort_layout_t;

effort_status_t effort_get_layout(effort_handle_t h, effort_layout_t* layout);

/* Frees the handle's device storage after synchronising its last stream. */
effort_status_t effort_destroy(effort_handle_t h);

/*
 * effort_last_call_bytes -- the bytes of the prepared matrix that the handle's
 *   last finished call (effort_gemv, _ex, _host) planned to read: dense_bytes
 *   for the (row, panel) units it read from the dense copy (512 bytes per
 *   256-column stripe; 256 for Q8), sparse_bytes for the chunks (3 bytes per
 *   slot, 2 for Q8; 64 slots per chunk).  Synchronises the handle's last stream.  The pages have
 *   no counterpart: a measurement service.  dense_bytes, sparse_bytes: host
 *   pointers, non-NULL.
 */
effort_status_t effort_last_call_bytes(effort_handle_t h, uint64_t* dense_bytes, uint64_t* sparse_bytes);

/*
 * effort_workspace_check -- effort_check for the workspace's calls
 *   (effort_gemv_batched, effort_dense_gemv): synchronises its last stream,
 *   reports EFFORT_ERR_NONFINITE if a pair's v held inf or NaN and
 *   EFFORT_ERR_DEVICE after a timed-out wait or an out-of-range index (debug
 *   build), clears the flags and, after an error, the workspace's scratch.
 */
effort_status_t effort_workspace_check(effort_workspace_t ws);

/*
 * effort_workspace_last_call_bytes -- the same for the workspace's last
 *   effort_gemv_batched call: the bytes its grids planned to read, summed
 *   over the grids (a grid serving two pairs on one matrix reads the union of
 *   their prefixes once, and counts it once).  Synchronises the workspace's
 *   last stream.  A measurement service.
 */
effort_status_t effort_workspace_last_call_bytes(effort_workspace_t ws, uint64_t* dense_bytes,
                                                 uint64_t* sparse_bytes);

/* Device memory the library holds at this moment, over all handles and
 * workspaces of the process (the figure EFFORT_ALLOC_CAP_BYTES is checked
 * against).  bytes: host pointer, non-NULL. */
effort_status_t effort_device_bytes_held(uint64_t* bytes);

/* ------------------------------------------------------------------------
 * Operators of the feed-forward block around the matvecs: the step between
 * two blocks (norms, gate, residual, quantisation), the product with e4m3
 * operands, and the mixture-of-experts layer for a few tokens.  The pages have
 * no counterpart; they name the norm-joined matvec chain and the mixture of
 * experts that these serve.  They are exact operators: no effort, no cutoff.
 *
 * They hold to the conventions above (device pointers owned by the caller,
 * stream as void*, argument errors found on the host before any launch), and
 * beyond them:
 *  - Strides are in elements, between rows; elements of a row are adjacent.
 *  - Sums, statistics and scales are held in fp32; each output is rounded once
 *    (what else is rounded is said below).
 *  - No call allocates, synchronises or keeps anything between calls: any of
 *    them may run on several streams at once, on one handle too, and may be
 *    captured into a graph.
 *  - Waits inside the kernels are bounded.  None runs out on a working device;
 *    where one does, the outputs that hang on it are NaN and the call's status is
 *    EFFORT_OK all the same.
 *  - rows (n_tokens) may be 0: nothing is launched.  Rows of an output beyond
 *    the call's rows, and elements between dim and the stride, are not touched.
 *  - inf and NaN follow IEEE arithmetic within their own row (token) and reach
 *    no other row.
 * ---------------------------------------------------------------------- */
#define EFFORT_BLOCK 128        /* elements that share one scale of an e4m3 operand */
#define EFFORT_MAX_FP8_DIM 262144   /* in_dim and out_dim of an e4m3 matrix */
#define EFFORT_MAX_ROWS (1 << 24)   /* rows of one call */

typedef enum { EFFORT_NORM_NONE = 0, EFFORT_NORM_RMS = 1, EFFORT_NORM_LAYER = 2 } effort_norm_kind_t;

/*
 * effort_block_norm -- the step between one block of a decoder layer and the
 * next, row by row, in one kernel:
 *
 *   u  = post(y)                                      (post_kind; NONE: y)
 *   x' = residual_scale * x + branch_scale * gate * u (y NULL: residual_scale * x)
 *   h  = pre(x')                                      (pre_kind; NONE: x')
 *
 *   RMS:   n(v) = v / sqrt(mean(v^2) + eps) * (weight_offset + weight) + bias
 *   LAYER: n(v) = (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) * (weight_offset + weight) + bias
 *
 * (a null weight multiplies by 1, whatever weight_offset is; a null bias adds
 * nothing).  Outputs, each nullable, one at least given:
 *   x_out  x' rounded to dtype.
 *   h_out  h rounded to h_dtype.
 *   q_out, q_scales  h in e4m3 with a scale per row and EFFORT_BLOCK columns:
 *     scale = max |h| over the block / 448 (fp32), q = h / scale rounded to
 *     nearest even (within +-448, which a subnormal scale's own rounding could
 *     pass); a block of zeros (or one whose scale underflows to zero) has scale 0
 *     and q 0.  A block that holds inf or NaN has scale inf or NaN.
 *     This is the form effort_fp8_matmul takes.
 * h is computed from x' before x' is rounded.  Squares and their sum are fp32: a row
 * whose sum of squares exceeds fp32 (values of 3e17 throughout 4096 columns) gives
 * h = bias (0 without one), and squares below fp32's normal numbers (values under
 * 1e-19) lose bits, which shows where eps is as small.
 *   dtype: of x, y, gate and x_out.  weight_dtype: of all weights and biases [dim].
 *   gate: nullable; gate_stride 0 uses one row for all rows.
 *   1 <= dim <= EFFORT_MAX_IN_DIM, 0 <= rows <= EFFORT_MAX_ROWS; every stride
 *   (but gate's 0) is at least dim (q_scales_stride: at least its blocks).
 *   Pointers are aligned to their element type.
 *   x_out and h_out may be the same array as x or y (same address, element
 *   size and stride).  Outputs that overlap inputs otherwise, or one another, are
 *   refused.
 *   Runs on the current device, where all pointers have to live.
 */
typedef struct {
  int64_t rows, dim;
  effort_dtype_t dtype, weight_dtype, h_dtype;
  effort_norm_kind_t post_kind, pre_kind;
  float eps, weight_offset, residual_scale, branch_scale;
  const void* x;
  int64_t x_stride;
  const void* y;
  int64_t y_stride;
  const void* gate;
  int64_t gate_stride;
  const void *post_weight, *post_bias, *pre_weight, *pre_bias;
  void* x_out;
  int64_t x_out_stride;
  void* h_out;
  int64_t h_stride;
  void* q_out;
  int64_t q_stride;
  float* q_scales;
  int64_t q_scales_stride;
} effort_block_norm_t;

effort_status_t effort_block_norm(const effort_block_norm_t* args, void* stream);

/*
 * effort_fp8_prepare -- an e4m3 weight matrix with one fp32 scale per 128 x 128
 *   block, laid out for effort_fp8_matmul: w_ij = scales[i / 128][j / 128] * q_ij.
 *   q: device e4m3 bytes [in_dim x out_dim], row-major (row i multiplies
 *   x[i]); scales: device fp32 [ceil(in_dim / 128) x ceil(out_dim / 128)],
 *   4-byte aligned.  Both are read during the call only (the stream is
 *   synchronised before returning).
 *   1 <= in_dim, out_dim <= EFFORT_MAX_FP8_DIM, in_dim * out_dim < 2^36.
 *   Returns EFFORT_ERR_NONFINITE if q holds a NaN or a scale is inf or NaN,
 *   EFFORT_ERR_NOMEM as effort_prepare does.
 *   The handle holds one byte per weight (both dims rounded up to 128) and the scales.
 */
typedef struct effort_fp8_s* effort_fp8_t;
effort_status_t effort_fp8_prepare(const void* q, const float* scales, int64_t in_dim, int64_t out_dim, void* stream,
                                   effort_fp8_t* out_matrix);

/*
 * effort_fp8_matmul -- out[r][n] = sum over blocks b of 128 of
 *     x_scales[r][b] * scales[b][n / 128] * sum over k in b of x[r][k] q[k][n].
 *   x: device e4m3 bytes [rows x in_dim], 16-byte aligned, x_stride a multiple
 *   of 16 (what effort_block_norm writes for such a q_out), of which a row's
 *   bytes are read up to the next multiple of 16 (any value); x_scales: device
 *   fp32 [rows x ceil(in_dim / 128)].  out: [rows x out_dim] of out_dtype.
 *   A block's sum meets its two scales one after the other, or (on the tensor cores)
 *   their product, in fp32: where that leaves fp32's range, so does the result.
 *   0 <= rows <= EFFORT_MAX_ROWS.  An out that overlaps x or x_scales is refused.
 *   One kernel (two for 9 to 16 rows where in_dim > 196608); results do not vary
 *   from call to call.
 */
effort_status_t effort_fp8_matmul(effort_fp8_t m, const void* x, int64_t x_stride, const float* x_scales,
                                  int64_t x_scales_stride, int64_t rows, effort_dtype_t out_dtype, void* out,
                                  int64_t out_stride, void* stream);

effort_status_t effort_fp8_get_info(effort_fp8_t m, int64_t* in_dim, int64_t* out_dim, size_t* device_bytes);

/* Frees the matrix's device storage.  The caller has synchronised the streams
 * that use it. */
effort_status_t effort_fp8_destroy(effort_fp8_t m);

/*
 * effort_moe_prepare -- the weights of a mixture-of-experts layer, laid out
 *   for effort_moe_forward.  Expert e computes
 *     y = W2_e^T (silu(W1_e^T x) * (W3_e^T x)),  silu(a) = a / (1 + exp(-a)).
 *   w1, w3: device [n_experts x in_dim x hidden_dim], w2: device [n_experts x
 *   hidden_dim x in_dim], row-major, aligned to their element; weight_kind
 *   gives their type.  EFFORT_W_E4M3: e4m3 bytes with s1, s3 [n_experts x
 *   ceil(in_dim / 128) x ceil(hidden_dim / 128)] and s2 [n_experts x
 *   ceil(hidden_dim / 128) x ceil(in_dim / 128)] fp32; else s1, s3, s2 are NULL.
 *   router: device [n_experts x in_dim] of router_dtype, row-major; nullable
 *   (every call then brings its routing).
 *   All are read during the call only (the stream is synchronised before
 *   returning); the handle keeps its own copies.
 *   1 <= n_experts <= EFFORT_MAX_EXPERTS, 1 <= in_dim, hidden_dim <= EFFORT_MAX_IN_DIM.
 *   Returns EFFORT_ERR_NONFINITE if an expert's weight or scale is inf or NaN (the
 *   router's values are not checked).
 */
#define EFFORT_MAX_EXPERTS 256
#define EFFORT_MAX_TOKENS 256   /* n_tokens of one call */
#define EFFORT_MAX_TOP_K 16
typedef enum { EFFORT_W_F16 = 0, EFFORT_W_BF16 = 1, EFFORT_W_E4M3 = 2 } effort_weight_kind_t;
typedef struct effort_moe_s* effort_moe_t;
typedef struct {
  int32_t n_experts;
  int64_t in_dim, hidden_dim;
  effort_weight_kind_t weight_kind;
  const void *w1, *w3, *w2;
  const float *s1, *s3, *s2;
  const void* router;
  effort_dtype_t router_dtype;
} effort_moe_weights_t;
effort_status_t effort_moe_prepare(const effort_moe_weights_t* weights, void* stream, effort_moe_t* out_layer);

/*
 * effort_moe_forward -- the layer on a few tokens (kernels: the router, the
 *   first products, the second product, the weighted sum):
 *     out[t] = sum over j < top_k of gates[t][j] * expert_{ids[t][j]}(x[t]).
 *   gate_mode
 *     EFFORT_GATE_SOFTMAX_OF_TOP: logits l = router x[t]; ids = the top_k
 *       largest, in falling order, ties to the lower expert; gates = softmax
 *       over the chosen logits.  ids and gates are written.
 *     EFFORT_GATE_TOP_OF_SOFTMAX: the same ids; gates = the chosen entries of
 *       the softmax over all experts (not renormalised).
 *     EFFORT_GATE_GIVEN: ids and gates are read.  An id below 0 or at or above
 *       n_experts adds nothing (padding); a token may name one expert twice.
 *   x: device [n_tokens x in_dim] of x_dtype; out: device [n_tokens x in_dim] of
 *   out_dtype, fully written (0 where every id is out of range); ids: device
 *   int32 [n_tokens x top_k], gates: device fp32 [n_tokens x top_k], packed.
 *   0 <= n_tokens <= EFFORT_MAX_TOKENS, 1 <= top_k <= EFFORT_MAX_TOP_K, and top_k <=
 *   n_experts unless the routing is given.
 *   scratch: device memory of effort_moe_scratch_bytes(layer, n_tokens, top_k)
 *   bytes, 256-byte aligned, whose contents mean nothing before and after the
 *   call; calls that may overlap on the GPU bring scratch of their own.
 *   out may lie over x, which has been read by then.  Any other overlap with what
 *   the call writes is refused.
 *   A token whose logits hold NaN counts them as lowest; its gates are NaN.
 *   Precision: products of 16-bit and e4m3 values are exact, and sums are fp32
 *   (the matrix instructions' own over 64 or 128 terms).  With bfloat16 weights
 *   x enters the first products in 24 bits or exactly, and the hidden activations
 *   silu(a) b enter the second in 16 bits (24 where out is fp32).  With binary16
 *   and e4m3 weights values enter in parts of 11 bits that are scaled together
 *   over a K block, 64 (e4m3: 128) inputs or hidden units of a token.  One part
 *   holds what is up to 2^28 below the block's bound in full and what is smaller
 *   to 2^-39 of the bound; two hold 22 bits, and to 2^-50 of the bound:
 *     x: binary16 exactly, bfloat16 in one part, fp32 in two; the bound is the
 *       block's largest |x| (or 2^-97);
 *     hidden activations: two parts; one where out is bfloat16, unless column
 *       norms of w1 or w3 differ by more than 32 times within a K block; the bound
 *       is |x|^2 times the largest column norms of w1 and w3 over the block (or 2^-96).
 *   The router's logits are fp32 sums: experts whose logits differ by less than
 *   their rounding may change places.
 *   Results do not vary from call to call.
 *   An expert's weights are read from memory once for up to 8 or 16 of its
 *   tokens and again, mostly from L2, for each 8 or 16 more.
 */
typedef enum {
  EFFORT_GATE_SOFTMAX_OF_TOP = 0,
  EFFORT_GATE_TOP_OF_SOFTMAX = 1,
  EFFORT_GATE_GIVEN = 2
} effort_gate_mode_t;
effort_status_t effort_moe_scratch_bytes(effort_moe_t layer, int64_t n_tokens, int32_t top_k, size_t* bytes);
effort_status_t effort_moe_forward(effort_moe_t layer, const void* x, effort_dtype_t x_dtype, int64_t x_stride,
                                   int64_t n_tokens, int32_t top_k, effort_gate_mode_t gate_mode, int32_t* ids,
                                   float* gates, void* out, effort_dtype_t out_dtype, int64_t out_stride, void* scratch,
                                   size_t scratch_bytes, void* stream);
effort_status_t effort_moe_get_info(effort_moe_t layer, int32_t* n_experts, int64_t* in_dim, int64_t* hidden_dim,
                                    size_t* device_bytes);

/* Frees the layer's device storage.  The caller has synchronised the streams
 * that use it. */
effort_status_t effort_moe_destroy(effort_moe_t layer);

/* Static string naming a status code. */
const char* effort_status_string(effort_status_t s);

#ifdef __cplusplus
}
#endif

#endif /* EFFORT_H */
