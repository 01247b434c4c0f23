/*
 * libqkvfront: the decode-batch attention front on one GB300 (sm_103a).
 *
 * Defined by the API pages of vllm.models.muse_spark.nvidia.specialized_decode:
 *   "cutedsl.attention.qkv_front" (module docstring; functions qkv_front,
 *   launch, unsupported, prepare, variant, hidden_rows_ok,
 *   kv_cache_layout_ok, supports_shape) and "runtime.cute_ops" (split_qkv,
 *   supports_call, unsupported_projection, attn2 paragraph for the cache).
 *
 * For 1 <= M <= 16 tokens one launch computes
 *     out[M, N] = bf16( x[M, 8192] @ W[N, 8192]^T )       (FP32 accumulation)
 * over packed rows [q | k | v | gate] (8 q heads, 1 k head, 1 v head and 8
 * gate heads of 64 columns per KV head, so N = 1152 * num_kv_heads), then for
 * each 64-wide q and k head the weightless RMS norm (eps 1e-6) and the
 * interleaved RoPE (pairs 2i, 2i+1; cos in table column i, sin in 32 + i) of
 * the token's position, stores the row in `out`, and writes each token's
 * k head g into the K half (elements 0..63) and v head g into the V half
 * (64..127) of cache slot `slots[t]` (page slot / 16, offset slot % 16) of KV
 * head g.  v and gate columns of `out` hold the rounded projection.
 *
 * Conventions of every entry point below:
 *   - bf16 arrays are passed as uint16_t bit patterns; all arrays are
 *     row-major and contiguous; all pointers are DEVICE pointers owned by the
 *     caller and must be 16-byte aligned;
 *   - the library allocates no device memory per call and keeps no state
 *     across calls except a device status word (qkv_front_status);
 *   - per device it caches, on first use, the kernels' attributes and the
 *     device address of its no-allocation array (attn2_split_kv_noalloc);
 *     after cudaDeviceReset on a device, do not call the library on that
 *     device again in the same process;
 *   - `stream` is a cudaStream_t (NULL: the legacy default stream); calls are
 *     asynchronous on it.  The kernel is launched with programmatic stream
 *     serialization (PDL): it may start while the previous kernel on the
 *     stream runs, reads only W before it waits for that kernel, and reads
 *     x / positions / slots / cos_sin and writes out / kv_cache after;
 *     so W must not be written by a kernel that may still be running when
 *     the call is launched (weights are written at load time only);
 *   - return value 0 (QKVF_OK) or a QKVF_ERR_* code; nothing is launched
 *     when a code is returned.  qkv_front_strerror gives its text.
 */
#ifndef QKVFRONT_H
#define QKVFRONT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- return codes -------------------------------------------------------- */
#define QKVF_OK 0
#define QKVF_ERR_TOKENS 1        /* M outside 0..16 */
#define QKVF_ERR_SHAPE 2         /* num_kv_heads < 1 or N != 1152 * num_kv_heads */
#define QKVF_ERR_NULL 3          /* a required pointer is NULL */
#define QKVF_ERR_ALIGN 4         /* a pointer is not 16-byte aligned */
#define QKVF_ERR_DEVICE 5        /* the current device is not compute capability 10.3 */
#define QKVF_ERR_CUDA 6          /* a CUDA runtime/driver call failed */
#define QKVF_ERR_SIZES 7         /* cos_sin_rows < 1, num_pages < 1, or too large */
#define QKVF_ERR_VARIANT 8       /* an explicit variant that this shape cannot use */
#define QKVF_ERR_ARG 9           /* any other bad argument */
#define QKVF_ERR_LAYOUT 10       /* head counts, head_dim, rotary width, dtype or strides (rope*, norm_rope*, prefix_attn, chunk_attn, key_weights, kv_evict) */

/* ---- device status bits (qkv_front_status) ------------------------------- */
#define QKVF_STATUS_BAD_SLOT 1u      /* a slot >= num_pages * 16: that token's insert skipped */
#define QKVF_STATUS_BAD_POSITION 2u  /* a position outside [0, cos_sin_rows): its q/k heads and insert skipped */
#define QKVF_STATUS_WAIT_TIMEOUT 4u  /* a bounded wait in the kernel gave up: outputs of that call are invalid */
#define QKVF_STATUS_BAD_REQUEST 8u   /* attn2: a request with L < 8, L beyond its table, or a page outside the cache: its rows skipped;
                                        prefix_attn: a length beyond its table or a page outside the cache: rows skipped */

/*
 * qkv_front: check the call, then launch the fused front.
 *   x          [M, 8192] bf16 bits.  The attention input.
 *   W          [N, 8192] bf16 bits.  Unquantized, bias-free QKV + o-gate weight.
 *   positions  [M] int64.  Token positions; each must be in [0, cos_sin_rows).
 *   slots      [M] int64.  Cache slot of each token (page * 16 + offset);
 *              a negative slot means "no insert" (padding token); a slot
 *              >= num_pages * 16 is skipped and flagged QKVF_STATUS_BAD_SLOT.
 *   cos_sin    [cos_sin_rows, 64] fp32.  Row p: cos(p f_i) in column i,
 *              sin(p f_i) in column 32 + i (interleaved, not neox style).
 *   out        [M, N] bf16 bits, written.
 *   kv_cache   [num_pages, num_kv_heads, 16, 128] bf16 bits; only the named
 *              slots change.
 *   M          0..16 tokens (M == 0 launches nothing and returns QKVF_OK).
 *   N          1152 * num_kv_heads.
 * Tokens must name distinct slots (two tokens writing one slot race).
 * x, W and cos_sin must not overlap out or kv_cache.
 */
int qkv_front(const uint16_t *x, const uint16_t *W, const int64_t *positions,
              const int64_t *slots, const float *cos_sin, int64_t cos_sin_rows,
              uint16_t *out, uint16_t *kv_cache, int64_t num_pages, int M, int N,
              int num_kv_heads, void *stream);

/*
 * qkv_front_unsupported: why qkv_front would refuse this call, or NULL when
 * it takes it (page qkv_front, function unsupported).  Host-only checks, no
 * CUDA call except the device query.  Returns a static string.
 */
const char *qkv_front_unsupported(const uint16_t *x, const uint16_t *W, const int64_t *positions,
                                  const int64_t *slots, const float *cos_sin,
                                  int64_t cos_sin_rows, uint16_t *out, uint16_t *kv_cache,
                                  int64_t num_pages, int M, int N, int num_kv_heads);

/*
 * qkv_front_launch: qkv_front without its argument checks, for a call that
 * qkv_front_unsupported already accepted (page qkv_front, function launch).
 * Out-of-contract arguments here are undefined behaviour.
 */
int qkv_front_launch(const uint16_t *x, const uint16_t *W, const int64_t *positions,
                     const int64_t *slots, const float *cos_sin, int64_t cos_sin_rows,
                     uint16_t *out, uint16_t *kv_cache, int64_t num_pages, int M, int N,
                     int num_kv_heads, void *stream);

/* ---- contraction engines (qkv_front_variant, qkv_front_launch_variant) --- */
#define QKVF_CONSUMER_DEFAULT 0   /* the library's choice */
#define QKVF_CONSUMER_MMA_SYNC 1  /* mma.sync m16n8k16 in four consumer warps */
#define QKVF_CONSUMER_TCGEN05 2   /* tcgen05.mma M=64 into tensor memory, one issuing thread */
#define QKVF_CONSUMER_RESIDENT 3  /* mma.sync with the CTA's whole W share on chip (shared memory and
                                     registers) before the PDL wait, partials pushed to the owner
                                     rank with st.async: splits 8, kb 4, stages 4 only */

/*
 * qkv_front_variant: the launch shape qkv_front uses for N columns and M
 * tokens on the current device (page qkv_front, function variant):
 *   *tiles    8-token column tiles (1 or 2),
 *   *stages   depth of the shared-memory weight ring,
 *   *splits   CTAs per head (the cluster size; K is split cyclically among them),
 *   *kb       64-wide K boxes per ring stage (1, 2 or 4),
 *   *consumer QKVF_CONSUMER_MMA_SYNC, QKVF_CONSUMER_TCGEN05 or
 *             QKVF_CONSUMER_RESIDENT (chosen when splits is 8: N = 1152).
 * Any output pointer may be NULL.  The result depends on the launch shape:
 * `splits` and `kb` fix how K is divided among CTAs, and the consumer fixes
 * the order inside one CTA; `stages` never changes it.
 */
int qkv_front_variant(int N, int M, int *tiles, int *stages, int *splits, int *kb, int *consumer);

/*
 * qkv_front_launch_variant: qkv_front (with its checks) at an explicit
 * variant, for tests and tuning.  splits in {1, 2, 4, 8, 16}; kb in {1, 2, 4}
 * (0: the default) with splits * kb <= 128; stages >= 2 within the
 * shared-memory limit; consumer one of QKVF_CONSUMER_* (the resident engine
 * takes splits 8, kb 4 or 0, stages 4).  Otherwise QKVF_ERR_VARIANT.
 */
int qkv_front_launch_variant(const uint16_t *x, const uint16_t *W, const int64_t *positions,
                             const int64_t *slots, const float *cos_sin,
                             int64_t cos_sin_rows, uint16_t *out, uint16_t *kv_cache,
                             int64_t num_pages, int M, int N, int num_kv_heads, int splits,
                             int stages, int kb, int consumer, void *stream);

/*
 * qkv_front_prepare: set the kernel attributes (dynamic shared memory,
 * non-portable cluster size) of the variants that N columns take, so that
 * later calls can be captured in a CUDA graph (page qkv_front, function
 * prepare).  Calls made without it prepare themselves on first use.
 */
int qkv_front_prepare(int N, int num_kv_heads);

/*
 * qkv_front_status: copy the device status word (an OR of QKVF_STATUS_* bits
 * raised by calls since the last read) into *bits and clear it.
 * Synchronizes the current device.
 */
int qkv_front_status(unsigned int *bits);

/*
 * qkv_front_from_host: the whole call for a caller whose tokens live in host
 * memory.  On `stream`, asynchronously: x [M, 8192], positions [M] and slots
 * [M] go from host memory into the caller's device `staging` buffer, qkv_front
 * runs on them, and out [M, N] goes back to `out_host`.  Pinned (page-locked,
 * device-mapped) host buffers are read by a staging kernel over the host link,
 * PDL-linked to the front so that its weight stream starts while x arrives,
 * and a pinned out_host is written by the front directly; pageable buffers go
 * through copies on the stream instead.  Host buffers must stay valid and
 * unchanged until the stream passes the call.  W, cos_sin and kv_cache are
 * device pointers as for qkv_front.
 *   staging        device buffer, 256-byte aligned, at least
 *                  qkv_front_staging_bytes(M, N) bytes; owned by the caller;
 *                  the call overwrites it (two calls in flight on different
 *                  streams need two buffers).
 * Same checks and codes as qkv_front, plus QKVF_ERR_SIZES when staging is too
 * small and QKVF_ERR_ALIGN when it is not 256-byte aligned.  The library
 * allocates nothing.
 */
int qkv_front_from_host(const uint16_t *x_host, const int64_t *positions_host,
                        const int64_t *slots_host, uint16_t *out_host, const uint16_t *W,
                        const float *cos_sin, int64_t cos_sin_rows, uint16_t *kv_cache,
                        int64_t num_pages, void *staging, uint64_t staging_bytes, int M, int N,
                        int num_kv_heads, void *stream);

/* Device staging bytes qkv_front_from_host needs for M tokens and N columns. */
uint64_t qkv_front_staging_bytes(int M, int N);

/*
 * qknorm_rope_kv_insert: the unfused epilogue on its own, for any number of
 * tokens (fused_muse_spark_qknorm_rope_kv_insert, the kernel the fused front
 * replaces: page qkv_front, module docstring; page cute_ops, qkv_front
 * paragraph).  In place on a BF16 projection output:
 *   qkv        [T, N] bf16 bits, rows [q | k | v | gate]; every q and k head
 *              is normed and rotated (same arithmetic as qkv_front), v and
 *              gate heads are not touched.
 *   positions, slots, cos_sin, cos_sin_rows, kv_cache, num_pages, N,
 *   num_kv_heads: as for qkv_front, with T entries in positions and slots.
 *   T          0 .. 2^24 tokens (0: no launch).
 * Each token's k head g goes to the K half and v head g to the V half of its
 * slot.  Out-of-range positions and slots follow qkv_front's rules and raise
 * the same status bits.  Launched with PDL like qkv_front (it waits for the
 * previous kernel before reading anything).  Allocates nothing.
 */
int qknorm_rope_kv_insert(uint16_t *qkv, const int64_t *positions, const int64_t *slots,
                          const float *cos_sin, int64_t cos_sin_rows, uint16_t *kv_cache,
                          int64_t num_pages, int T, int N, int num_kv_heads, void *stream);

/* Why qknorm_rope_kv_insert would refuse this call, or NULL (host checks only). */
const char *qknorm_rope_kv_insert_unsupported(uint16_t *qkv, const int64_t *positions,
                                              const int64_t *slots, const float *cos_sin,
                                              int64_t cos_sin_rows, uint16_t *kv_cache,
                                              int64_t num_pages, int T, int N, int num_kv_heads);

/*
 * layer_front: the kernel before the QKV front in the first decoder layer
 * (page layer_front, class LayerFront, run): for each of `rows` rows of
 * 8192 values,
 *   stream = x as FP32 (the residual stream), aux = stream (if aux is not
 *   NULL), out = bf16((stream * r) * w), r = 1 / sqrt(mean(stream^2) + eps),
 *   w the BF16 weight widened to FP32 (out = bf16(stream * r) when weight is
 *   NULL) — the attention input the QKV front reads as x.
 *   x          [rows, 8192], bf16 bits (x_is_f32 = 0) or fp32 (x_is_f32 = 1).
 *   weight     [8192] bf16 bits, or NULL.
 *   stream, aux [rows, 8192] fp32 (aux may be NULL); out [rows, 8192] bf16 bits.
 *   rows       0 .. 2^20 (0: no launch); eps in (0, 1].
 * All arrays are device pointers, 16-byte aligned; outputs must not overlap
 * each other or the inputs.  Launched with PDL: it waits for the previous
 * kernel, then at once lets the next kernel on the stream start, so a
 * qkv_front call issued after it streams its weights while this runs.
 */
int layer_front(const void *x, int x_is_f32, const uint16_t *weight, float *stream, float *aux,
                uint16_t *out, int rows, float eps, void *cuda_stream);

/*
 * attn2: paged decode attention of the 8-token verify step fused with the
 * output's weightless RMS norm and sigmoid gate — the o_proj input (page
 * cute_ops, attn2 paragraph).  For each request r (query rows 8r .. 8r+7 of
 * qkv, row i the token at position L_r - 8 + i):
 *   out[8r+i, head h] = bf16( o / sqrt(mean(o^2) + eps) * sigmoid(gate) ),
 *   o = softmax(scale * q K^T) V over keys j <= L_r - 8 + i (and, with a
 *   window W > 0, j > L_r - 8 + i - W); q = q head h of the row, gate = gate
 *   head h of the row, K and V from KV head h / 8 of the cache.
 *   qkv          [8 R, N] bf16 bits, rows [q | k | v | gate] (the front's out).
 *   kv_cache     [num_pages, num_kv_heads, 16, 128] bf16 bits (K | V per slot).
 *   block_table  [R, max_blocks] int32: key j of request r is slot j % 16 of
 *                page block_table[r][j / 16].
 *   context_lens [R] int32, each >= 8.
 *   out          [8 R, 512 num_kv_heads] bf16 bits.
 *   window       0 (none) or W >= 1; scale > 0 (1/8 for head_dim 64);
 *   eps in (0, 1].  num_reqs 0 .. 65535.
 * A request whose length is < 8 or needs more than max_blocks pages, or
 * whose table names a page outside the cache, is skipped (its rows left as
 * they were) and raises QKVF_STATUS_BAD_REQUEST.  Long contexts are split
 * over up to 8 CTAs of a cluster (attn2_launch_splits reaches 16), chosen
 * from num_reqs, num_kv_heads, max_blocks and window (not from the lengths,
 * which stay on the device): doubled while num_reqs * num_kv_heads * splits
 * stays within the SM count and each split keeps two or more of the pages a
 * row can see; the split partials are merged through distributed shared
 * memory in a fixed order.
 * Allocates nothing; launched with PDL like qkv_front.
 */
int attn2(const uint16_t *qkv, const uint16_t *kv_cache, int64_t num_pages,
          const int32_t *block_table, int max_blocks, const int32_t *context_lens, int num_reqs,
          int N, int num_kv_heads, int window, float scale, float eps, uint16_t *out,
          void *stream);

/*
 * attn2_unsupported: why attn2 (and attn2_split_kv / _noalloc, given a valid
 * workspace and split) would refuse this call, or NULL when it takes it
 * (page cute_ops, unsupported_attn2).  Host-only checks, no CUDA call except
 * the device query; returns a static string.  Of the page's refusals, the
 * layout ones are fixed by this ABI: head_dim 64 and 8 q heads per KV head
 * are implied by N = 1152 * num_kv_heads, and a layer without the o-norm and
 * sigmoid gate has nothing to call here (the Python binding's
 * unsupported_attn2 refuses such a layer).  The page's kernel is built for
 * one softmax scale and one o-norm eps, whose values the page does not
 * print; this kernel takes both per call and refuses only scale <= 0 and eps
 * outside (0, 1].
 */
const char *attn2_unsupported(const uint16_t *qkv, const uint16_t *kv_cache, int64_t num_pages,
                              const int32_t *block_table, int max_blocks, const int32_t *context_lens,
                              int num_reqs, int N, int num_kv_heads, int window, float scale, float eps,
                              uint16_t *out);

/* attn2 at an explicit split (1, 2, 4, 8 or 16 CTAs per request and KV head;
 * otherwise QKVF_ERR_VARIANT), for tests and tuning. */
int attn2_launch_splits(const uint16_t *qkv, const uint16_t *kv_cache, int64_t num_pages,
                        const int32_t *block_table, int max_blocks, const int32_t *context_lens,
                        int num_reqs, int N, int num_kv_heads, int window, float scale, float eps,
                        uint16_t *out, int splits, void *stream);

/* The split attn2 uses for this shape (window 0: none) on the current device
 * (0 on bad input). */
int attn2_splits(int num_reqs, int num_kv_heads, int max_blocks, int window);

/*
 * attn2, split-KV engine: the same result as attn2 (same arguments, readings
 * and bad-request rule) with the pages a row sees split over `splits` CTAs
 * per (request, KV head) without clusters, so that few requests can still
 * cover every SM.  Two grids on the stream (the second PDL-linked when the
 * first leaves SMs idle): the first writes each CTA's partial (row maxima,
 * sums and unnormalised O, FP32) to its slot of the caller's workspace; the
 * second merges a row's slots in split order (a fixed `splits` gives the
 * same bits every time) and finishes the rows.
 *   splits          1 .. 256, or 0 for attn2_split_kv_splits' choice;
 *                   otherwise QKVF_ERR_VARIANT.
 *   workspace       device memory, 256-byte aligned, at least
 *                   attn2_split_kv_workspace_bytes(num_reqs, num_kv_heads,
 *                   splits) bytes, owned by the caller, overlapping no other
 *                   argument, no initial contents needed; one workspace serves
 *                   one stream at a time.
 * With splits == 1 the call runs one grid (each CTA finishes its own rows)
 * and leaves the workspace untouched.
 * Returns QKVF_ERR_NULL / _ALIGN / _SIZES / _ARG for a missing, misaligned,
 * short or overlapping workspace, else as attn2.
 */
int attn2_split_kv(const uint16_t *qkv, const uint16_t *kv_cache, int64_t num_pages,
                   const int32_t *block_table, int max_blocks, const int32_t *context_lens, int num_reqs,
                   int N, int num_kv_heads, int window, float scale, float eps, uint16_t *out, int splits,
                   void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes attn2_split_kv needs (0 on bad input): num_reqs *
 * num_kv_heads * splits slots of 17152 bytes. */
size_t attn2_split_kv_workspace_bytes(int num_reqs, int num_kv_heads, int splits);

/* The split attn2_split_kv picks for splits == 0 on the current device: the
 * grid covers the SMs once (num_reqs * num_kv_heads * splits <= SM count) and
 * each split keeps two or more of the pages a row can see; 0 on bad input. */
int attn2_split_kv_splits(int num_reqs, int num_kv_heads, int max_blocks, int window);

/*
 * attn2_split_kv for callers that cannot allocate device memory: a plugin
 * whose host process owns every device allocation through its own pool, or
 * a decode step that must not risk cudaMalloc's implicit synchronisation or
 * a failed allocation mid-step.  The pages have no counterpart of this entry
 * point.  Same arguments and result as attn2_split_kv without the workspace:
 * the partials go to a file-scope device array of the library, 256 slots of
 * 17152 bytes (4,390,912 bytes), which every GPU that loads the library holds
 * until the process exits.  The call allocates nothing.
 *   When splits (after splits == 0 is resolved as attn2_split_kv_splits
 *   does) is above 1, num_reqs * num_kv_heads * splits must be <= 256, else
 *   QKVF_ERR_SIZES.  At one split the call runs the direct path (each CTA
 *   finishes its own rows), touches no array slot and takes any num_reqs.
 * The first call on a device looks up the array's device address (once per
 * device, with that device current); make that first call before any stream
 * capture.  The array needs no clearing: a call reads only slots it wrote.
 * Every call shares it, so calls that overlap on the GPU (other streams,
 * other host threads) race; run them one after another.
 */
int attn2_split_kv_noalloc(const uint16_t *qkv, const uint16_t *kv_cache, int64_t num_pages,
                           const int32_t *block_table, int max_blocks, const int32_t *context_lens,
                           int num_reqs, int N, int num_kv_heads, int window, float scale, float eps,
                           uint16_t *out, int splits, void *stream);

/*
 * The operators below serve any head layout around a paged cache
 * [num_pages, num_kv_heads, 16, 2 head_dim] (K | V per slot, as the front's
 * cache has at head_dim 64).  A [tokens, heads, head_dim] array is given by
 * its pointer and its token and head strides in elements (the last dimension
 * is contiguous), so the q, k and v columns of packed projection rows are
 * passed as they lie; strides are 0..2^36, and an output's heads must not
 * overlap one another.  A pointer is aligned to its elements; cos_sin and
 * kv_cache to 16 bytes.  Rows that are 16-byte aligned throughout move in
 * 16-byte accesses.  Every refusal has its reason in the *_unsupported
 * function beside it.
 */

/* ---- element types, rotary layouts, rotary scalings ---------------------- */
#define QKVF_DTYPE_BF16 0
#define QKVF_DTYPE_FP16 1
#define QKVF_DTYPE_FP32 2        /* rope only */
#define QKVF_DTYPE_ZERO_SKIPPED 16  /* or'ed onto a dtype: the rows of out (q_out) that a call would leave as they
                                       were become 0, for an output without earlier contents */

#define QKVF_ROPE_INTERLEAVED 0  /* pair i: columns 2i, 2i + 1 */
#define QKVF_ROPE_HALF 1         /* pair i: columns i, i + rot_dim / 2 */

#define QKVF_ROPE_NONE 0         /* f_i = base^(-2i / rot_dim) */
#define QKVF_ROPE_LINEAR 1       /* f_i / factor: every position compressed */
#define QKVF_ROPE_BASE 2         /* base * factor^(rot_dim / (rot_dim - 2)): the slowest pair stretched by factor */
#define QKVF_ROPE_RAMP 3         /* by parts: with n_i = original_len f_i / 2 pi turns over the original length and
                                    g = clamp((n_i - slow) / (fast - slow), 0, 1): (1 - g) f_i / factor + g f_i */

/*
 * rope_table: the cos | sin rows of positions first .. first + rows - 1, as
 * qkv_front, rope and rope_kv_append read them:
 *   table[r][i] = magnitude cos(p f_i), table[r][rot_dim / 2 + i] = magnitude sin(p f_i), p = first + r,
 * with the pairs' frequencies f_i scaled for long contexts as named above
 * (factor >= 1; original_len, slow and fast are read by QKVF_ROPE_RAMP only).
 * Angles are kept modulo one turn in 64-bit fixed point: what grows with the
 * position is the error of the frequency as a double (about position f 2^-51
 * radians), not that of a 32-bit product; cos and sin add 2^-22 or so.
 *   table    [rows, rot_dim] fp32, device memory, 16-byte aligned
 *   rows 0..2^32 (0: no launch), first 0..2^40, rot_dim even 2..512,
 *   base in (1, 1e30], magnitude in (0, 1e6].
 * Asynchronous on `stream`, PDL-launched; allocates nothing.
 */
int rope_table(float *table, int64_t first, int64_t rows, int rot_dim, double base, int scaling, double factor,
               int64_t original_len, double slow, double fast, double magnitude, void *stream);

const char *rope_table_unsupported(const float *table, int64_t first, int64_t rows, int rot_dim, double base,
                                   int scaling, double factor, int64_t original_len, double slow, double fast,
                                   double magnitude);

/*
 * rope: rotate the first rot_dim columns of every head by its token's
 * position; the columns behind them are copied.
 *   (a, b) -> (a c - b s, b c + a s), c | s = row positions[t] of cos_sin;
 *   inverse = 1: s negated, the gradient of the rotation with respect to x.
 *   x, out   [T, heads, head_dim] of dtype (bf16, fp16 or fp32), strided;
 *            out may be x itself (same pointer and strides), otherwise it
 *            must not overlap x.
 *   positions [T] int64; a position outside [0, cos_sin_rows) leaves its
 *            token's heads of out as they were and raises
 *            QKVF_STATUS_BAD_POSITION.
 *   cos_sin  [cos_sin_rows, rot_dim] fp32: cos in columns 0 .. rot_dim/2 - 1,
 *            sin behind them.
 *   T 0..2^24, heads 1..4096, head_dim 2..512, rot_dim even 2..head_dim.
 * Products and sums in FP32, one rounding to dtype.  PDL-launched; allocates
 * nothing.
 */
int rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, const int64_t *positions,
         const float *cos_sin, int64_t cos_sin_rows, void *out, int64_t out_token_stride,
         int64_t out_head_stride, int T, int heads, int head_dim, int rot_dim, int layout, int inverse,
         int dtype, void *stream);

const char *rope_unsupported(const void *x, int64_t x_token_stride, int64_t x_head_stride,
                             const int64_t *positions, const float *cos_sin, int64_t cos_sin_rows, void *out,
                             int64_t out_token_stride, int64_t out_head_stride, int T, int heads, int head_dim,
                             int rot_dim, int layout, int inverse, int dtype);

/*
 * rope_kv_append: rotate q into q_out, rotate k and write it with v into each
 * token's cache slot: the step between a projection and prefix_attn.
 *   q, q_out [T, q_heads, head_dim], k, v [T, num_kv_heads, head_dim] of dtype
 *            (bf16 or fp16), strided; q_out may be q itself, otherwise it must
 *            not overlap q, k or v.  q_heads 0 (q and q_out NULL): append only.
 *   positions, cos_sin as for rope; slots [T] int64 as for qkv_front: a
 *            negative slot inserts nothing, a slot >= 16 num_pages is skipped
 *            and raises QKVF_STATUS_BAD_SLOT; a bad position leaves the
 *            token's q_out heads and slot as they were and raises
 *            QKVF_STATUS_BAD_POSITION.  Tokens must name distinct slots.
 *   kv_cache [num_pages, num_kv_heads, 16, 2 head_dim] of dtype; only the
 *            named slots change.
 *   T 0..2^24, head_dim a multiple of 8 up to 512, num_kv_heads 1..1024.
 * PDL-launched; allocates nothing.
 */
int rope_kv_append(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
                   int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
                   int64_t v_head_stride, const int64_t *positions, const int64_t *slots, const float *cos_sin,
                   int64_t cos_sin_rows, void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                   void *kv_cache, int64_t num_pages, int T, int q_heads, int num_kv_heads, int head_dim,
                   int rot_dim, int layout, int dtype, void *stream);

const char *rope_kv_append_unsupported(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                       const void *k, int64_t k_token_stride, int64_t k_head_stride,
                                       const void *v, int64_t v_token_stride, int64_t v_head_stride,
                                       const int64_t *positions, const int64_t *slots, const float *cos_sin,
                                       int64_t cos_sin_rows, void *q_out, int64_t q_out_token_stride,
                                       int64_t q_out_head_stride, void *kv_cache, int64_t num_pages, int T,
                                       int q_heads, int num_kv_heads, int head_dim, int rot_dim, int layout,
                                       int dtype);

/*
 * prefix_attn: paged decode attention of num_reqs requests that share a
 * prefix; the prefix's keys are read once for all of them.  Row (request r,
 * its token i of q_len, q head h) attends to the prefix's prefix_len keys and
 * to its request's own keys j <= L_r - q_len + i under one softmax:
 *   out = sum_j exp(s_j) v_j / sum_j exp(s_j),  lse = ln sum_j exp(s_j),  s_j = scale q . k_j.
 * A row that sees no key gives out = 0 and lse = -infinity.
 *   q            [num_reqs q_len, q_heads, head_dim] of dtype (bf16 or fp16),
 *                16-byte aligned, strides multiples of 8; head h reads KV head
 *                h / (q_heads / num_kv_heads).
 *   kv_cache     [num_pages, num_kv_heads, 16, 2 head_dim] of dtype.
 *   prefix_pages [prefix_blocks] int32: prefix key j is slot j % 16 of page
 *                prefix_pages[j / 16]; prefix_len one int32 on the device,
 *                0 .. 16 prefix_blocks.  Both may be NULL when prefix_blocks is 0.
 *   block_table  [num_reqs, max_blocks] int32: the same for each request's own
 *                keys (NULL when max_blocks is 0); entries past a length are
 *                not used, whatever they hold.
 *   context_lens [num_reqs] int32: L_r, the request's own keys, the step's
 *                q_len tokens among them (0 .. 16 max_blocks; shorter than
 *                q_len leaves the first rows with the prefix alone).  Negative:
 *                a padding request, its rows of out and lse left as they were.
 *   out          [num_reqs q_len, q_heads, head_dim] of dtype, contiguous;
 *   lse          [num_reqs q_len, q_heads] fp32, or NULL.
 *   workspace    device memory, 256-byte aligned, prefix_attn_workspace_bytes
 *                bytes, overlapping no other argument, no initial contents
 *                needed; one workspace serves one stream at a time.
 * A request whose length is beyond its table is skipped (its rows left as they
 * were), and so are the rows that see a page outside the cache (with them other
 * rows of that request, but of no other): QKVF_STATUS_BAD_REQUEST is raised.  A
 * bad prefix does so for every request.  Cache
 * slots past a length are never used, whatever they hold, and a key reaches only
 * the rows that see it: an infinity or NaN in K or V of a request's later token
 * does not change its earlier tokens' rows.
 *   head_dim 64 or 128, q_heads 1..64 times num_kv_heads (1..64), q_len
 *   1..1024, num_reqs 0..65535, num_reqs q_len q_heads <= 2^24.
 * Scores, softmax statistics and sums in FP32; the weights exp(s - m) are
 * rounded to dtype for the product with V (fp16: by no more than 2^-33 of the
 * row's largest where that is more than half a step).  The lengths stay on the device,
 * so a captured call serves every step up to its tables' widths.
 * PDL-launched; allocates nothing.
 */
int prefix_attn(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *kv_cache,
                int64_t num_pages, const int32_t *prefix_pages, int prefix_blocks, const int32_t *prefix_len,
                const int32_t *block_table, int max_blocks, const int32_t *context_lens, int num_reqs, int q_len,
                int q_heads, int num_kv_heads, int head_dim, float scale, int dtype, void *out, float *lse,
                void *workspace, size_t workspace_bytes, void *stream);

const char *prefix_attn_unsupported(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                    const void *kv_cache, int64_t num_pages, const int32_t *prefix_pages,
                                    int prefix_blocks, const int32_t *prefix_len, const int32_t *block_table,
                                    int max_blocks, const int32_t *context_lens, int num_reqs, int q_len,
                                    int q_heads, int num_kv_heads, int head_dim, float scale, int dtype,
                                    const void *out, const float *lse, const void *workspace,
                                    size_t workspace_bytes);

/* Workspace bytes prefix_attn needs on the current device (0 on bad input).
 * A workspace for some prefix_blocks and max_blocks serves smaller ones too. */
size_t prefix_attn_workspace_bytes(int num_reqs, int q_len, int q_heads, int num_kv_heads, int head_dim,
                                   int prefix_blocks, int max_blocks);

/*
 * norm_rope: the RMS norm of every head, times a weight, then its rotation,
 * in one pass over x:
 *   y = R(position) (w * x r),  r = (mean of the head's head_dim squares + eps)^(-1/2),
 * R as in rope: the first rot_dim columns turned, the others (normed and
 * weighted like them) not.
 *   x, out, positions, cos_sin, T, heads, head_dim, rot_dim, layout, dtype as
 *            for rope (out may be x itself); a bad position leaves its token's
 *            heads of out as they were and raises QKVF_STATUS_BAD_POSITION.
 *   weight   [head_dim] of weight_dtype (dtype's type or fp32), or NULL for 1.
 *   eps in [0, 1].
 * Squares, products and sums in FP32, one rounding to dtype.  PDL-launched;
 * allocates nothing.
 */
int norm_rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, const void *weight, int weight_dtype,
              const int64_t *positions, const float *cos_sin, int64_t cos_sin_rows, void *out,
              int64_t out_token_stride, int64_t out_head_stride, int T, int heads, int head_dim, int rot_dim,
              int layout, float eps, int dtype, void *stream);

const char *norm_rope_unsupported(const void *x, int64_t x_token_stride, int64_t x_head_stride, const void *weight,
                                  int weight_dtype, const int64_t *positions, const float *cos_sin,
                                  int64_t cos_sin_rows, void *out, int64_t out_token_stride, int64_t out_head_stride,
                                  int T, int heads, int head_dim, int rot_dim, int layout, float eps, int dtype);

/*
 * norm_rope_backward: the gradients of norm_rope, from the gradient of its
 * output and its input x.  With g' = R(-position) grad and u = w * g':
 *   grad_x = r u - x r^3 mean(u * x),   grad_weight = sum over tokens and heads of g' * x r.
 *   grad_out, x, grad_x  [T, heads, head_dim] of dtype, strided; grad_x may be
 *            grad_out itself (same pointer and strides), otherwise it overlaps
 *            neither.  A head stride of 0 broadcasts.
 *   grad_weight [head_dim] of grad_weight_dtype (dtype's type or fp32), written,
 *            not added to; NULL: not formed.  NULL where weight is NULL.
 *   workspace device memory, 256-byte aligned, norm_rope_backward_workspace_bytes
 *            bytes, overlapping no other argument, no initial contents needed;
 *            one workspace serves one stream at a time.  Unused (may be NULL)
 *            without grad_weight.
 * A token of a bad position has its grad_x left as it was and adds nothing to
 * grad_weight; QKVF_STATUS_BAD_POSITION is raised.  All sums in FP32 and in a
 * fixed order.  PDL-launched; allocates nothing.
 */
int norm_rope_backward(const void *grad_out, int64_t grad_token_stride, int64_t grad_head_stride, const void *x,
                       int64_t x_token_stride, int64_t x_head_stride, const void *weight, int weight_dtype,
                       const int64_t *positions, const float *cos_sin, int64_t cos_sin_rows, void *grad_x,
                       int64_t grad_x_token_stride, int64_t grad_x_head_stride, void *grad_weight,
                       int grad_weight_dtype, int T, int heads, int head_dim, int rot_dim, int layout, float eps,
                       int dtype, void *workspace, size_t workspace_bytes, void *stream);

const char *norm_rope_backward_unsupported(const void *grad_out, int64_t grad_token_stride, int64_t grad_head_stride,
                                           const void *x, int64_t x_token_stride, int64_t x_head_stride,
                                           const void *weight, int weight_dtype, const int64_t *positions,
                                           const float *cos_sin, int64_t cos_sin_rows, void *grad_x,
                                           int64_t grad_x_token_stride, int64_t grad_x_head_stride, void *grad_weight,
                                           int grad_weight_dtype, int T, int heads, int head_dim, int rot_dim,
                                           int layout, float eps, int dtype, const void *workspace,
                                           size_t workspace_bytes);

/* Workspace bytes norm_rope_backward needs on the current device (0 on bad
 * input, or without tokens). */
size_t norm_rope_backward_workspace_bytes(int T, int heads, int head_dim);

/*
 * norm_rope_kv_append: rope_kv_append with the heads of q and k normed and
 * weighted before they are turned (norm_rope), v as it is.
 *   q_weight, k_weight [head_dim] of weight_dtype (dtype's type or fp32), each
 *            may be NULL for 1; eps in [0, 1]; the rest as for rope_kv_append.
 */
int norm_rope_kv_append(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
                        int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
                        int64_t v_head_stride, const void *q_weight, const void *k_weight, int weight_dtype,
                        const int64_t *positions, const int64_t *slots, const float *cos_sin, int64_t cos_sin_rows,
                        void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, void *kv_cache,
                        int64_t num_pages, int T, int q_heads, int num_kv_heads, int head_dim, int rot_dim,
                        int layout, float eps, int dtype, void *stream);

const char *norm_rope_kv_append_unsupported(
    const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k, int64_t k_token_stride,
    int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride, const void *q_weight,
    const void *k_weight, int weight_dtype, const int64_t *positions, const int64_t *slots, const float *cos_sin,
    int64_t cos_sin_rows, void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, void *kv_cache,
    int64_t num_pages, int T, int q_heads, int num_kv_heads, int head_dim, int rot_dim, int layout, float eps,
    int dtype);

/*
 * chunk_attn: attention of each request's new tokens, any number of them a
 * request, over its paged keys: prefill chunks and decode steps in one call.
 * Request r brings the n = starts[r + 1] - starts[r] rows from starts[r] on and
 * has L = context_lens[r] keys, its new tokens' (the last n) among them.  Its
 * token i sees keys j <= L - n + i (none where that is negative):
 *   out = sum_j exp(s_j) v_j / sum_j exp(s_j),  lse = ln sum_j exp(s_j),  s_j = scale q . k_j.
 * A row that sees no key gives out = 0 and lse = -infinity.
 *   q            [T, q_heads, head_dim] of dtype (bf16 or fp16), 16-byte
 *                aligned, strides multiples of 8; head h reads KV head
 *                h / (q_heads / num_kv_heads).
 *   kv_cache     [num_pages, num_kv_heads, 16, 2 head_dim] of dtype.
 *   starts       [num_reqs + 1] int32, not decreasing, 0 .. T.  Rows of no
 *                request (before starts[0], from starts[num_reqs] on) are left
 *                as they were.
 *   block_table  [num_reqs, max_blocks] int32: key j of a request is slot j % 16
 *                of page block_table[r][j / 16]; entries past a length are not
 *                used, whatever they hold.
 *   context_lens [num_reqs] int32, 0 .. 16 max_blocks.  Negative: a padding
 *                request, its rows of out and lse left as they were.
 *   out          [T, q_heads, head_dim] of dtype, contiguous; lse [T, q_heads]
 *                fp32, or NULL.
 *   workspace    device memory, 256-byte aligned, chunk_attn_workspace_bytes
 *                bytes, overlapping no other argument, no initial contents
 *                needed; one workspace serves one stream at a time.
 * A request whose length is beyond its table, whose starts decrease or leave
 * 0 .. T, or that sees a page outside the cache is skipped (its rows left as
 * they were; where only some of its rows see that page, others may be
 * computed): QKVF_STATUS_BAD_REQUEST is raised.  Cache slots past a length are
 * never used, whatever they hold, and a key reaches only the rows that see it.
 *   head_dim 64 or 128, q_heads 1..64 times num_kv_heads (1..64), num_reqs
 *   0..65535, T 0..2^24, T q_heads <= 2^30, max_blocks 1..2^20.
 * Scores, softmax statistics and sums in FP32; the weights exp(s - m) are
 * rounded to dtype for the product with V.  Starts and lengths stay on the
 * device, so a captured call serves every step of its sizes.
 * PDL-launched; allocates nothing.
 */
int chunk_attn(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *kv_cache, int64_t num_pages,
               const int32_t *starts, const int32_t *block_table, int max_blocks, const int32_t *context_lens, int T,
               int num_reqs, int q_heads, int num_kv_heads, int head_dim, float scale, int dtype, void *out,
               float *lse, void *workspace, size_t workspace_bytes, void *stream);

const char *chunk_attn_unsupported(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *kv_cache,
                                   int64_t num_pages, const int32_t *starts, const int32_t *block_table,
                                   int max_blocks, const int32_t *context_lens, int T, int num_reqs, int q_heads,
                                   int num_kv_heads, int head_dim, float scale, int dtype, void *out, float *lse,
                                   const void *workspace, size_t workspace_bytes);

/* Workspace bytes chunk_attn needs on the current device (0 on bad input). */
size_t chunk_attn_workspace_bytes(int T, int num_reqs, int q_heads, int num_kv_heads, int head_dim, int max_blocks);

/*
 * key_weights: the attention weight that each cached key received from the
 * step's rows, kept from step to step:
 *   out[r][g][j] = decay weights[r][g][j] + sum of exp(scale q . k_j - lse)
 * over the request's tokens that see key j (its last `window` tokens only, 0:
 * all) and the q heads of KV head g.  q (its strides above 0), starts,
 * block_table, context_lens, the cache and the limits as for chunk_attn; lse [T, q_heads] as it gave it (a row
 * of lse -infinity adds nothing, whatever its q holds).
 *   weights, out [num_reqs, num_kv_heads, 16 max_blocks] fp32; out may be
 *            weights itself, otherwise it must not overlap it.  Keys below a
 *            length are written, others left as they were.  decay in [0, 1];
 *            0: weights is not read (may be NULL).
 *   workspace as for chunk_attn, key_weights_workspace_bytes bytes.
 * A request that chunk_attn would skip has its weights left as they were (of
 * a page outside the cache, at least those keys'), QKVF_STATUS_BAD_REQUEST as
 * there.  Sums in FP32 and in a fixed order.  PDL-launched; allocates nothing.
 */
int key_weights(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *kv_cache, int64_t num_pages,
                const float *lse, const int32_t *starts, const int32_t *block_table, int max_blocks,
                const int32_t *context_lens, int T, int num_reqs, int q_heads, int num_kv_heads, int head_dim,
                int window, float decay, float scale, int dtype, const float *weights, float *out, void *workspace,
                size_t workspace_bytes, void *stream);

const char *key_weights_unsupported(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *kv_cache,
                                    int64_t num_pages, const float *lse, const int32_t *starts,
                                    const int32_t *block_table, int max_blocks, const int32_t *context_lens, int T,
                                    int num_reqs, int q_heads, int num_kv_heads, int head_dim, int window, float decay,
                                    float scale, int dtype, const float *weights, float *out, const void *workspace,
                                    size_t workspace_bytes);

/* Workspace bytes key_weights needs on the current device (0 on bad input). */
size_t key_weights_workspace_bytes(int T, int num_reqs, int q_heads, int num_kv_heads, int head_dim, int max_blocks);

/*
 * kv_evict: drop the keys of least weight.  Of each request's L keys, for each
 * KV head on its own, the last `recent` are kept and of the others the
 * keep - recent of largest weight (the lower index among equals; a NaN above
 * every number); with L <= keep all of them.  The kept keys, in their order,
 * become keys 0 .. min(L, keep) - 1:
 *   kept[r][g][i]  the index that key i had (-1 from min(L, keep) on);
 *   K and V of key kept[r][g][i] go to key i of out_table's pages;
 *   out_weights[r][g][i] = weights[r][g][kept[r][g][i]], and 0 behind them (as
 *            far as weights had keys, in place; otherwise to the row's end);
 *   out_lens[r] = min(L, keep).
 *   kv_cache     [num_pages, num_kv_heads, 16, 2 head_dim] of a 16-bit type.
 *   weights      [num_reqs, num_kv_heads, 16 max_blocks] fp32.
 *   block_table  [num_reqs, max_blocks], context_lens [num_reqs] as for
 *                chunk_attn (negative: a padding request, left alone).
 *   out_table    [num_reqs, out_blocks], out_weights [num_reqs, num_kv_heads, 16
 *                out_blocks], out_lens [num_reqs]: all three the inputs
 *                themselves (in place), or none of them; then 16 out_blocks >=
 *                keep, and no page that out_table names for a kept key may be a
 *                page of another key of this call.  A page that several
 *                requests share is not evicted in place.
 *   kept         [num_reqs, num_kv_heads, keep] int32.
 * A request whose length is beyond its table, or that needs a page outside the
 * cache, is left alone (its row of kept becomes -1): QKVF_STATUS_BAD_REQUEST.
 *   head_dim a multiple of 8 up to 512, num_kv_heads 1..1024, num_reqs 0..65535,
 *   max_blocks and out_blocks 1..2^20, keep 1..2^24, recent 0..keep.
 * PDL-launched; allocates nothing.
 */
int kv_evict(void *kv_cache, int64_t num_pages, const float *weights, const int32_t *block_table, int max_blocks,
             const int32_t *context_lens, int num_reqs, int num_kv_heads, int head_dim, int keep, int recent,
             const int32_t *out_table, int out_blocks, float *out_weights, int32_t *out_lens, int32_t *kept,
             void *stream);

const char *kv_evict_unsupported(void *kv_cache, int64_t num_pages, const float *weights, const int32_t *block_table,
                                 int max_blocks, const int32_t *context_lens, int num_reqs, int num_kv_heads,
                                 int head_dim, int keep, int recent, const int32_t *out_table, int out_blocks,
                                 float *out_weights, int32_t *out_lens, int32_t *kept);

/*
 * Packed calls: the same calls with their arguments up to the stream as an
 * array of 64-bit words, in order (pointers and integers as they are, floats
 * and doubles as a double's bits), for bindings that pay per argument.  An
 * integer that does not fit its parameter is refused with QKVF_ERR_SIZES.
 */
int rope_table_packed(const int64_t *args, void *stream);       /* 11 words */
int rope_packed(const int64_t *args, void *stream);             /* 16 words */
int rope_kv_append_packed(const int64_t *args, void *stream);   /* 25 words */
int prefix_attn_packed(const int64_t *args, void *stream);      /* 22 words */
int norm_rope_packed(const int64_t *args, void *stream);            /* 18 words */
int norm_rope_backward_packed(const int64_t *args, void *stream);   /* 25 words */
int norm_rope_kv_append_packed(const int64_t *args, void *stream);  /* 29 words */
int chunk_attn_packed(const int64_t *args, void *stream);           /* 20 words */
int key_weights_packed(const int64_t *args, void *stream);          /* 23 words */
int kv_evict_packed(const int64_t *args, void *stream);             /* 16 words */


/* Static text of a QKVF_* return code. */
const char *qkv_front_strerror(int code);

/*
 * qkv_front_selftest_wait: launch a one-CTA kernel that waits, through the
 * same bounded shared-memory barrier wait the front uses, on a barrier that
 * nothing completes, for at most timeout_ns nanoseconds (1..10^9); it then
 * raises QKVF_STATUS_WAIT_TIMEOUT and returns.  Tests that the kernel's waits
 * end without hanging the GPU.
 */
int qkv_front_selftest_wait(int64_t timeout_ns, void *stream);

/*
 * qkv_front_set_pdl: launch this library's kernels with programmatic stream
 * serialization (enable = 1, the default) or as plain stream-ordered launches
 * (0).  With PDL a kernel may start while the previous kernel on its stream
 * still runs and streams its weights before waiting for it; turn it off when
 * a kernel that may still be running writes W (or, for measurement, to see
 * what the overlap gains).  Other values: QKVF_ERR_ARG.  Applies to launches
 * made after the call, on every device.
 */
int qkv_front_set_pdl(int enable);

/* Bounded-wait limit of the front's barrier waits in nanoseconds
 * (default 2e9); values outside 1e3..1e10 are refused with QKVF_ERR_ARG. */
int qkv_front_set_wait_limit(int64_t ns);

#ifdef __cplusplus
}
#endif

#endif /* QKVFRONT_H */
