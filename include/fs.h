/*
 * fs.h — C ABI of the continuous-batched decode step (decode_step_batch).
 *
 * One handle holds one dense Llama-style model on one GPU, a paged KV arena
 * shared by up to max_lanes lanes, and the scratch panels of one step. One
 * call advances up to max_lanes lanes by one token each: every weight byte is
 * read once for the whole batch, while attention stays per lane over that
 * lane's own pages.
 *
 * Sources of the operations (page title, section):
 *   - "Fat-station continuous batching — the live-path integration",
 *     "The capture": decode_step_batch(kv caches, positions, tokens) advances
 *     K lanes by one token with one weight read for the wave; "Components",
 *     item 3: fill (reset a free lane, position 0), gather, fold (sample with
 *     the lane's temperature/seed, retire, free the lane).
 *   - "MODEL-BATCHING-RESULTS — multi-user batched decode, measured",
 *     "The lever": the seven projection matmuls and the LM head run as one
 *     GEMM over a [B, *] panel; attention is per user over its own KV cache;
 *     "API": StepBatch(ids) is the per-step primitive a continuous-batching
 *     scheduler calls after admitting/evicting users between steps.
 *   - mlx-bun "Parallel slots — configurable batched serving", "KV memory",
 *     rung 3: fixed-size KV blocks in a shared pool with a block manager.
 *
 * Conventions
 *   - Every call returns FS_OK (0) or a negative FS_ERR_* code; the message
 *     of the last failure is available from fs_last_error(handle) (or
 *     fs_last_error(NULL) for a failed fs_create). No C++ exception crosses
 *     this boundary.
 *   - A handle is used by one host thread at a time.
 *   - Calls that change lane state are atomic: on any error no lane length,
 *     position or page changes.
 *   - Unless stated otherwise, pointers are HOST pointers owned by the caller
 *     and only read during the call.
 *   - All kernels run on the handle's stream (fs_set_stream). Calls that
 *     return host results synchronise that stream; fs_decode_step_batch does
 *     not (its logits are ready once the stream reaches that point).
 */
#ifndef FS_H_
#define FS_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define FS_OK 0
#define FS_ERR_ARG (-1)       /* bad argument, size or descriptor field      */
#define FS_ERR_LANE (-2)      /* lane index outside [0, max_lanes)            */
#define FS_ERR_DUP_LANE (-3)  /* a lane appears twice in one step            */
#define FS_ERR_POSITION (-4)  /* positions[i] differs from the lane length   */
#define FS_ERR_TOKEN (-5)     /* token outside [0, vocab)                     */
#define FS_ERR_KV_FULL (-6)   /* page pool exhausted, or lane at max_pos      */
#define FS_ERR_OOM (-7)       /* device allocation failed                     */
#define FS_ERR_CUDA (-8)      /* a CUDA call failed (message has the detail)  */
#define FS_ERR_STATE (-9)     /* call out of order (e.g. sample before step)  */
#define FS_ERR_DEVICE (-10)   /* a kernel reported a device-side error flag   */
#define FS_ERR_SCRATCH (-11)  /* request exceeds fs_gemm_bf16_noalloc's static
                                 scratch                                      */

/* ---- element types ----------------------------------------------------- */
#define FS_DTYPE_F32 0   /* IEEE binary32                                     */
#define FS_DTYPE_BF16 1  /* bfloat16 bit patterns (uint16)                    */
#define FS_DTYPE_Q8_0 2  /* blocks of 32 inputs: fp16 scale d (little endian)
                            then 32 int8 codes q; value = q * d; 34 bytes.
                            A [rows, cols] matrix is rows*cols/32 blocks in
                            row-major order (cols must be a multiple of 32).  */

#define FS_DTYPE_Q8_ROW 3 /* KV only: 8-bit rows, see fs_kv_q8                   */

/* Model and arena description. */
typedef struct fs_model_desc {
  int32_t n_layers;        /* L                                              */
  int32_t d_model;         /* d                                              */
  int32_t n_heads;         /* H query heads                                  */
  int32_t n_kv_heads;      /* Hkv; H must be a multiple of Hkv (GQA)         */
  int32_t head_dim;        /* hd, even; RoPE pairs (i, i + hd/2)             */
  int32_t d_ffn;           /* F (SwiGLU width)                               */
  int32_t vocab;           /* V                                              */
  float rms_eps;           /* RMSNorm epsilon                                */
  double rope_theta;       /* RoPE base                                      */
  int32_t tied_embeddings; /* 1: LM head is the embedding matrix             */
  int32_t weight_dtype;    /* FS_DTYPE_F32 / _BF16 / _Q8_0 for all matrices  */
  int32_t kv_dtype;        /* FS_DTYPE_F32, _BF16, or _Q8_ROW (keys and values
                              quantised as they are appended, see fs_kv_q8;
                              head_dim 64, 128 or 256)                       */
  int32_t max_lanes;       /* lanes addressable by fs_decode_step_batch      */
  int32_t page_size;       /* tokens per KV page (e.g. 16)                   */
  int32_t n_pages;         /* pages in the shared arena                      */
  int32_t max_pos;         /* tokens a lane may hold                         */
  int32_t act_split;       /* 0: the bf16 activation panels (normed x,
                              attention output, SwiGLU product) feed the
                              tensor-core GEMMs as they are; 1: each panel
                              also carries its rounding remainder
                              lo = bf16(v - hi), and every tcgen05 GEMM
                              multiplies W by hi and by lo into one f32
                              accumulator (two MMAs per k-step), which keeps
                              the products near f32 accuracy at depth (bf16
                              and Q8_0 weights only)                         */
} fs_model_desc;

/* Per-layer weights in Hugging Face layout W[out, in], row-major, in
 * weight_dtype; norm gains are always f32. Pointers may be host or device
 * memory (the library copies them during fs_create; the caller keeps
 * ownership). */
typedef struct fs_layer_weights {
  const void* wq;        /* [H*hd, d]   */
  const void* wk;        /* [Hkv*hd, d] */
  const void* wv;        /* [Hkv*hd, d] */
  const void* wo;        /* [d, H*hd]   */
  const void* w_gate;    /* [F, d]      */
  const void* w_up;      /* [F, d]      */
  const void* w_down;    /* [d, F]      */
  const float* attn_norm; /* [d]        */
  const float* ffn_norm;  /* [d]        */
} fs_layer_weights;

typedef struct fs_weights {
  const void* embed;              /* [V, d]                               */
  const void* lm_head;            /* [V, d]; NULL when tied_embeddings    */
  const float* final_norm;        /* [d]                                  */
  const fs_layer_weights* layers; /* n_layers entries                     */
} fs_weights;

typedef struct fs_handle fs_handle;

/* Creates a handle on the current CUDA device: validates the descriptor,
 * uploads and re-lays out the weights, allocates the KV arena and scratch.
 * Errors: FS_ERR_ARG (descriptor), FS_ERR_OOM, FS_ERR_CUDA. */
int fs_create(const fs_model_desc* desc, const fs_weights* weights,
              fs_handle** out);

/* Frees every device buffer of the handle. NULL is accepted. */
int fs_destroy(fs_handle* h);

/* Message of the last failed call on h (or, when h is NULL, of this thread's
 * last failed fs_create or operator on the caller's buffers). Valid until the
 * next call on the same handle. */
const char* fs_last_error(const fs_handle* h);

/* Kernels of h run on `stream` (a cudaStream_t) from now on. NULL selects
 * the handle's own stream. */
int fs_set_stream(fs_handle* h, void* stream);

/* Fill step of the scheduler ("Components", item 3): lane k lets go of its
 * pages (a page returns to the pool once no lane holds it) and its length
 * becomes 0. Errors: FS_ERR_LANE. */
int fs_lane_reset(fs_handle* h, int32_t lane);

/* Clone, per-user prefix reuse kept under batching ("MODEL-BATCHING-RESULTS",
 * "Why in-kernel batching, not vLLM"): empty lane dst takes lane src's
 * history. dst shares src's full pages (a page holds a count of the lanes
 * that hold it; a full page is never written again), and src's partial last
 * page, which both lanes go on writing, is copied to a new page (lowest free
 * index) in every layer. Both lanes then have src's length, and a token fed
 * to either gives the logits the other gives for the same token. Enqueued
 * on the handle's stream; no synchronisation.
 * Errors: FS_ERR_LANE, FS_ERR_ARG (src == dst), FS_ERR_STATE (dst not
 * empty), FS_ERR_KV_FULL (a partial page and no free page); nothing changes
 * on error. */
int fs_lane_clone(fs_handle* h, int32_t src, int32_t dst);

/* Evict, quarantine of a span of one user's history (same passage as
 * fs_lane_clone): positions [start, end) leave the lane's cache. Entries at
 * positions p >= end move down to p - (end - start) and their keys are
 * rotated back by end - start positions, so the lane holds length - (end -
 * start) consecutive positions and the next token goes at that length.
 * K/V of the kept entries are not recomputed (they were computed while the
 * span was present). end == length drops a suffix and moves nothing. Pages
 * the lane writes (from the one holding `start` on) that another lane still
 * holds are first replaced by private copies (lowest free index); pages
 * past the new end are let go. An 8-bit key that is rotated back is quantised
 * anew, one more rounding of half a code; this quotient is f32, so within 1e-4
 * of the border of two codes it may take either. Enqueued on the handle's stream.
 * Errors: FS_ERR_LANE, FS_ERR_ARG (not 0 <= start <= end <= length),
 * FS_ERR_KV_FULL (too few free pages for the copies); nothing changes on
 * error. */
int fs_lane_evict(fs_handle* h, int32_t lane, int32_t start, int32_t end);

/* decode_step_batch. For each i < n, lane lanes[i], whose length must equal
 * positions[i], consumes tokens[i]: its K/V at that position are appended to
 * its pages (a new page, lowest free index first, when the length is a
 * multiple of page_size) and its next-token logits are produced. On success
 * positions[i] is incremented. lanes, positions and tokens are host arrays.
 * logits_out: DEVICE pointer to f32 [n, vocab] in input order, or NULL to
 * keep the logits inside the handle for fs_sample. n == 0 is a no-op.
 * With logits_out == NULL the step's kernels run as one CUDA graph, captured
 * on the first call with that n and replayed afterwards; the first call
 * for an n therefore must not happen inside another stream capture.
 * Errors (nothing changes): FS_ERR_ARG (n outside [0, max_lanes]),
 * FS_ERR_LANE, FS_ERR_DUP_LANE, FS_ERR_POSITION, FS_ERR_TOKEN,
 * FS_ERR_KV_FULL; FS_ERR_CUDA if a launch fails (lane state is then
 * undefined). */
int fs_decode_step_batch(fs_handle* h, const int32_t* lanes,
                         int32_t* positions, const int32_t* tokens, int32_t n,
                         float* logits_out);

/* decode_step_batch followed by greedy sampling, without materialising the
 * logits: the LM head's GEMM epilogue keeps, per lane and 128-row vocab
 * tile, the largest logit and its lowest index, and a small kernel takes each
 * lane's argmax over its tiles (lowest index on ties), the token fs_sample
 * returns with temperature 0 for the same step. Lanes, positions, tokens and
 * errors as fs_decode_step_batch. tokens_out: int32 [n] in DEVICE memory
 * (ready once the stream reaches this point; the call does not synchronise)
 * or host memory (written before the call returns). When the handle's LM head
 * is split across blocks the logits are written and argmaxed by the sampler
 * kernel instead (same tokens). After this call fs_sample refuses
 * (FS_ERR_STATE): the step left no logits. The pages have this as "fused
 * sampling" in their cost notes (the LM head's [B, V] output dominates the
 * small model at large B). */
int fs_decode_step_greedy(fs_handle* h, const int32_t* lanes,
                          int32_t* positions, const int32_t* tokens, int32_t n,
                          int32_t* tokens_out);

/* decode_step_batch with chunked prefill: the prompt of a lane is consumed in
 * chunks ("Fat-station continuous batching", "What /generate does today":
 * the prompt is prefilled in chunks) within one batched step, next to the
 * decoding lanes ("DGR-012", "Prefill does not starve decode": prefill per
 * tick is capped in tokens). Rows i < n: lane lanes[i] consumes tokens[i] at
 * positions[i]; a lane may appear on several rows, and its rows' positions
 * must be exactly its length, length + 1, ..., length + rows - 1, in any
 * order. Every row's K/V are appended before attention, so a row attends to
 * its lane's keys 0..positions[i], including the other rows of this step
 * at earlier positions; a row's logits equal, bit for bit, those of feeding
 * the same tokens one per call through fs_decode_step_batch. Pages are taken
 * per lane in position order, lanes in order of first appearance. n counts
 * rows (at most max_lanes). On success every positions[i] is incremented
 * and each lane's length grows by its row count. logits_out, graphs and
 * errors as fs_decode_step_batch, except that FS_ERR_POSITION also reports
 * positions that are not the lane's next consecutive ones (repeated lanes
 * are not FS_ERR_DUP_LANE here). */
int fs_step_batch_chunked(fs_handle* h, const int32_t* lanes,
                          int32_t* positions, const int32_t* tokens, int32_t n,
                          float* logits_out);

/* Samples one token per row of the last step's logits ("Components", item 3,
 * fold: the lane's temperature and seed). Row i: temps[i] == 0 selects the
 * argmax (lowest index on ties); otherwise z = logit / temps[i] in double,
 * u = (Philox4x32-10(key = seeds[i], counter = counters[i]) >> 11) * 2^-53,
 * and the first index whose running sum of exp(z - max z) reaches u times
 * the total. temps/seeds/counters are host arrays of n entries, n must equal
 * the last step's n; tokens_out is a host array. Synchronises the stream.
 * Errors: FS_ERR_STATE (no step yet, or n differs), FS_ERR_ARG. */
int fs_sample(fs_handle* h, int32_t n, const float* temps,
              const uint64_t* seeds, const uint64_t* counters,
              int32_t* tokens_out);

/* fs_sample on device buffers, without synchronising: temps (f32), seeds and
 * counters (uint64) and tokens_out (int32) are DEVICE arrays of n entries.
 * The tokens are ready once the stream reaches this point. Same rule and
 * errors as fs_sample. */
int fs_sample_device(fs_handle* h, int32_t n, const float* temps,
                     const uint64_t* seeds, const uint64_t* counters,
                     int32_t* tokens_out);

/* ---- inspection and test hooks ---------------------------------------- */

/* Copies the last step's logits (f32 [n, vocab], input order) to `dst`
 * (host or device memory). Synchronises the stream. Errors: FS_ERR_STATE
 * (no step yet). */
int fs_copy_logits(fs_handle* h, float* dst);

/* Kernel classes of the profiler. */
#define FS_PROF_GEMM 0      /* weight-streaming GEMM (all matrices)          */
#define FS_PROF_ATTN 1      /* attention partial + combine                  */
#define FS_PROF_OTHER 2     /* embed, norms, RoPE/append, sampler           */
#define FS_PROF_CLASSES 3

/* Enables (1) or disables (0) CUDA-event timing of every kernel launch of
 * the handle, on the handle's stream. */
int fs_profile_enable(fs_handle* h, int32_t enable);

/* Synchronises the stream and returns, for kernel class `cls`, the summed
 * device time in ms, the number of launches and the algorithmic bytes those
 * launches move (weights, activations, KV and outputs, each counted once)
 * since the last read; then clears that class. */
int fs_profile_read(fs_handle* h, int32_t cls, double* ms_out,
                    int64_t* launches_out, double* bytes_out);

/* Tokens one lane can hold (the descriptor's max_pos). */
int fs_lane_capacity(const fs_handle* h, int32_t* tokens_out);

/* Kernel timeline tracing (a diagnostic; no counterpart on the pages).
 * With capacity > 0, thread 0 of every block of the library's step kernels
 * appends one record of four uint64 to a device buffer of `capacity`
 * records: word 0 = tag << 40 | waited << 39 | SM id << 24 | linear block
 * index (waited: the block passed its wait for the preceding kernel; tag: 1
 * embed, 2 RMSNorm, 3 sampler, 4 tile argmax, 5 attention (cp.async), 6
 * attention (TMA), 7 attention (tiled), 8 attention (fused), 9 RoPE +
 * KV append, 10 GEMV, 11 / 12 split attention partials / combine (the
 * three-kernel path), 13 GEMV with the SwiGLU epilogue, 14 quantised KV
 * append, 15 / 20 attention over an 8-bit cache / its join, 16 + epilogue
 * kind for the tensor-core GEMM: 16
 * store, 17 residual, 18 SwiGLU, 19 argmax); words 1-3 = %globaltimer ns
 * at the block's entry, after its wait for the preceding kernel, and at its
 * end. Records past the capacity are counted, not stored. The buffer is
 * process-wide: one handle at a time may trace (FS_ERR_STATE otherwise);
 * capacity 0 turns tracing off and frees the buffer (also done by
 * fs_destroy). Synchronises the stream. */
int fs_trace_enable(fs_handle* h, int64_t capacity);

/* Copies min(appended, capacity, cap) records (4 uint64 each, in the order
 * they were appended) to host memory and the count appended so far to
 * *appended_out; reset != 0 then empties the buffer. Synchronises the
 * stream. Errors: FS_ERR_STATE (h is not tracing), FS_ERR_ARG. */
int fs_trace_read(fs_handle* h, uint64_t* records_out, int64_t cap, int64_t* appended_out,
                  int reset);

/* Current length (tokens held) of a lane. */
int fs_lane_length(const fs_handle* h, int32_t lane, int32_t* length_out);

/* Page table of a lane: writes min(cap, n_pages_of_lane) page indices and
 * the lane's page count to *n_out. */
int fs_lane_pages(const fs_handle* h, int32_t lane, int32_t* pages_out,
                  int32_t cap, int32_t* n_out);

/* Copies a lane's K (after RoPE) and V of one layer to host f32 arrays of
 * [length, Hkv, hd]. Synchronises the stream. */
int fs_lane_export_kv(fs_handle* h, int32_t lane, int32_t layer, float* k_out,
                      float* v_out);

/* Seeds lane `lane` (which must be empty) with n tokens of given K (already
 * rotated) and V for every layer: k and v are host f32 arrays
 * [n_layers, n, Hkv, hd]. Pages are allocated as by n decode steps.
 * Errors: FS_ERR_STATE (lane not empty), FS_ERR_KV_FULL, FS_ERR_ARG. */
int fs_lane_import_kv(fs_handle* h, int32_t lane, const float* k,
                      const float* v, int32_t n);

/* Seeds an empty lane with n tokens of pseudo-random K/V (values of unit
 * scale drawn on the device from `seed`) for timing long contexts, where
 * the content does not matter. Errors as fs_lane_import_kv. */
int fs_lane_fill_random_kv(fs_handle* h, int32_t lane, int32_t n,
                           uint64_t seed);

/* Q8_0 quantiser on the device: src is n f32 values (DEVICE pointer, n a
 * multiple of 32), blocks_out receives n/32 blocks of 34 bytes (DEVICE
 * pointer). Per block: d = max|x| / 127, q = round-half-away(x * (1/d))
 * clamped to [-127, 127], d stored as fp16 (round to nearest even); an
 * all-zero block stores d = 0 and q = 0. Runs on `stream` (a cudaStream_t,
 * NULL = default stream) and synchronises it. */
int fs_quantize_q8_0(const float* src, int64_t n, uint8_t* blocks_out,
                     void* stream);

/* Number of kernels the library launched on the handle since creation. */
int fs_kernel_launches(const fs_handle* h, int64_t* count_out);

/* Name of the GEMM path serving the handle's weight matrices: "tcgen05"
 * (bf16 weights on the tensor cores), "tcgen05-q8_0" (Q8_0 weights,
 * dequantised to bf16 in shared memory inside the GEMM), "tcgen05-q8_0+bf16"
 * or "warp-gemv" (f32 weights, d_ffn not a multiple of 64, or a device
 * without tcgen05). A Q8_0 handle whose lane capacity cuts a matrix's GEMM
 * into two or more lane groups (each of which would dequantise every weight
 * tile) also keeps that matrix as bf16(q * d), converted once by fs_create
 * (2 bytes per weight on top of the Q8_0 tiles); calls of that many groups
 * multiply the copy, the same operand bits ("tcgen05-q8_0+bf16"). The
 * environment variable FS_Q8_BF16_GROUPS, read by fs_create, sets that group
 * count (default 2; 0 keeps no copies). */
const char* fs_gemm_path(const fs_handle* h);

/* Work split of the tcgen05 GEMM for one weight matrix, as fs_create and the
 * decode step choose it (host arithmetic only: no device, handle or CUDA call;
 * a test and tuning hook). n_rows x k_inputs is the matrix (k_inputs a
 * multiple of 32), max_lanes the handle's lane capacity, n the call's lanes
 * (1 <= n <= max_lanes), sms the device's SM count, weight_dtype
 * FS_DTYPE_BF16 or FS_DTYPE_Q8_0. Writes out[8] (host):
 *   out[0] P, the stream-K width: blocks per lane group, a whole number of
 *          K splits of every 128-row tile; fixed per handle, never dependent
 *          on n (a lane's bits do not depend on its batch)
 *   out[1] lanes per group (the MMA's N), out[2] lane groups,
 *   out[3] TMEM columns a block allocates,
 *   out[4] 1 when a Q8_0 handle keeps a bf16 copy of the matrix,
 *   out[5] 1 when this call multiplies that copy,
 *   out[6] 128-row tiles, out[7] 64-wide k-blocks.
 * Reads the environment knobs fs_create reads for these choices.
 * Errors: FS_ERR_ARG (sizes, dtype, or a matrix too large for the GEMM). */
int fs_gemm_plan(int64_t n_rows, int64_t k_inputs, int max_lanes, int n, int sms,
                 int weight_dtype, int32_t* out);

/* Name of the decode-attention kernel serving the handle: "tma-mma" (KV
 * tiles by TMA, warp MMAs; bf16 KV, page_size a multiple of 8 that divides
 * or is a multiple of 64), "cp.async-mma" (KV tiles by cp.async, warp MMAs;
 * bf16 KV), "q8-mma" (8-bit KV), "tiled", "fused" or "three-kernel" (the
 * f32-KV and odd-shape paths). The environment variable FS_ATTN=mma|tiled|fused, read by
 * fs_create, selects a slower kernel (a comparison point). */
const char* fs_attention_path(const fs_handle* h);

/* Synchronises the stream, returns the handle's device error code (0: none;
 * non-zero: a kernel gave up on a bounded wait) and clears it. fs_sample
 * reports a set code as FS_ERR_DEVICE. */
int fs_device_error(fs_handle* h, int32_t* code_out);

/* Failure-detection check (no counterpart on the pages): launches on the
 * handle's stream a kernel that waits, bounded by timeout_us microseconds
 * (1 .. 1e6), on a barrier nothing arrives on, the way every wait of the
 * step kernels is bounded; on giving up it sets the handle's device error
 * code to 99 and returns. Then as fs_device_error: synchronises, writes the
 * code (99 when the check worked) and clears it. The handle stays usable.
 * Errors: FS_ERR_ARG, FS_ERR_CUDA. */
int fs_selftest_bounded_wait(fs_handle* h, int32_t timeout_us, int32_t* code_out);

/* Test hook: Y[b, n] = sum_k X[b, k] * W[n, k] for bf16 W [N, K] and
 * X [B, K] (K a multiple of 64), f32 Y [B, N]; all DEVICE pointers owned by
 * the caller. path 1 = tcgen05 kernel with `splits` equal K splits per
 * 128-row tile (1 <= splits <= min(8, K/64)); the splits of a tile sum
 * through a thread-block cluster where the partial tile fits in shared
 * memory, else through the workspace; path 2 = the same with the workspace
 * reduction always; path 0 = warp-GEMV kernel. Paths 1 and 2 give the same
 * bits. Allocates its own workspace; runs on
 * `stream` (NULL = default) and synchronises it. Errors: FS_ERR_ARG,
 * FS_ERR_OOM, FS_ERR_CUDA, FS_ERR_DEVICE (a bounded wait timed out). */
int fs_gemm_bf16(const uint16_t* W, int32_t N, int32_t K, const uint16_t* X,
                 int32_t B, float* Y, int32_t splits, int32_t path,
                 void* stream);

/* Test hook: the tcgen05 path of fs_gemm_bf16 with the stream-K width given
 * directly: the ceil(N/128) * K/64 k-blocks (row tile after row tile) are
 * cut into `width` equal ranges, one block per range and lane group, so a
 * range may end inside a row tile and cover parts of several
 * (1 <= width <= ceil(N/128) * K/64). Same operands, ownership, stream and
 * errors as fs_gemm_bf16. The pages have no counterpart; it exists to test
 * the work split that the decode step uses. */
int fs_gemm_bf16_width(const uint16_t* W, int32_t N, int32_t K, const uint16_t* X,
                       int32_t B, float* Y, int32_t width, void* stream);

/* Tuning hook: fs_gemm_bf16_width launched once and then `reps` times, each
 * launch between two CUDA events and after a 256 MiB memset that evicts the
 * operands from L2; *ms_out receives the mean device time of one launch in
 * ms. Same operands, ownership and errors as fs_gemm_bf16. The pages have
 * no counterpart. */
int fs_gemm_bf16_time(const uint16_t* W, int32_t N, int32_t K, const uint16_t* X,
                      int32_t B, float* Y, int32_t width, int32_t reps,
                      double* ms_out, void* stream);

/* fs_gemm_bf16 without any device allocation. The pages have no counterpart
 * of this entry point; it exists for callers that cannot call cudaMalloc or
 * cudaFree: for example a process whose device memory belongs to another
 * framework's caching allocator, a latency-critical loop in which cudaFree's
 * device-wide synchronisation or an unbounded allocation time is not
 * acceptable, or an embedder with a fixed device-memory budget.
 *
 * Computes Y[b, n] = sum_k X[b, k] * W[n, k] on the tcgen05 path with
 * `splits` K splits (1 <= splits <= min(8, K/64)), exactly as
 * fs_gemm_bf16(..., splits, path = 1, ...): bf16 W [N, K], bf16 X [B, K],
 * f32 Y [B, N], K a multiple of 64, all DEVICE pointers owned by the caller.
 * Runs on `stream` (NULL = default) and synchronises it.
 *
 * Scratch: a static device array of 8 MiB in this library (every GPU that
 * loads the library holds it until exit). It holds up to 16384 arrival
 * counters (ceil(N/128) * lane groups + 1 <= 16384) and, when splits > 1,
 * splits * B * ceil(N/128) * 128 f32 partials within 8 MiB - 64 KiB (for
 * example N = 4096, splits = 4, B <= 127). Larger requests return
 * FS_ERR_SCRATCH and run nothing. Every call looks up the array's device
 * address on the current device (cudaGetSymbolAddress), synchronises
 * `stream` after the launch and copies the kernel's error flag to the host
 * before returning. Every call shares the array and clears its counters and
 * error flag first; calls that overlap on the GPU race and must be
 * serialised by the caller.
 * Errors: FS_ERR_ARG, FS_ERR_SCRATCH, FS_ERR_CUDA, FS_ERR_DEVICE. */
int fs_gemm_bf16_noalloc(const uint16_t* W, int32_t N, int32_t K,
                         const uint16_t* X, int32_t B, float* Y,
                         int32_t splits, void* stream);

/* ---- 8-bit paged KV cache: operators on the caller's device buffers -------
 *
 * The paged cache of the handle (pages of page_size tokens, a page table per
 * lane) with keys and values held in 8 bits: half the bytes of a bf16 cache,
 * which is what bounds decode attention over long contexts. A row (one token's
 * key or value of one KV head) is head_dim codes and one f32 scale:
 *   scale = amax / 127, code = round(x * 127 / amax), ties to even,
 *   amax = max |x| of the row (0: scale 0 and codes 0),
 * stored as the byte code + 128 (1 .. 255). A value stands for code * scale,
 * off by at most scale / 2 and its share of the scale's own rounding (2^-24, more
 * in rows below 2^-119). A NaN is stored as 0, an infinity as the largest finite f32. Token t of a lane is in slot t % page_size of its page
 * t / page_size. A lane outside [0, n_lanes), a token outside
 * [0, max_pages * page_size) and a page-table entry outside [0, n_pages) hold
 * nothing: they are never written, read as zeros, and get no weight.
 *
 * Every pointer is a DEVICE pointer on the current device, owned by the caller
 * and used until the stream has passed the call; the struct itself is host
 * memory, read during the call. The calls enqueue on `stream` (a cudaStream_t,
 * NULL = default stream), allocate nothing, do not synchronise, and can be
 * captured into a graph. Code arrays are 16-byte aligned, the others aligned
 * to their element type.
 * Errors of these calls, with nothing enqueued: FS_ERR_ARG (a NULL pointer, a
 * size, a type, an alignment, memory of another device or of the host),
 * FS_ERR_SCRATCH (workspace too small); FS_ERR_CUDA (a launch failed: of an
 * attention over splits the first of two may have run, on its workspace). */
typedef struct fs_kv_q8 {
  uint8_t* k;       /* codes [n_pages][n_kv_heads][page_size][head_dim]       */
  uint8_t* v;
  float* k_scale;   /* [n_pages][n_kv_heads][page_size]                       */
  float* v_scale;
  const int32_t* page_table; /* [n_lanes][max_pages]                          */
  int32_t n_pages;
  int32_t n_kv_heads;
  int32_t page_size;  /* any positive number                                  */
  int32_t head_dim;   /* 64, 128 or 256                                       */
  int32_t n_lanes;
  int32_t max_pages;
} fs_kv_q8;

/* Quantises n tokens' keys and values as they are written: row i (k + i *
 * k_stride and v + i * v_stride elements, [n_kv_heads][head_dim] of dtype
 * FS_DTYPE_F32 or _BF16) goes to token positions[i] of lane lanes[i]. With
 * rope_cos / rope_sin (f32 [rope_len][head_dim / 2]) the key is first rotated
 * by its position, pairs (j, j + head_dim / 2); NULL for both stores keys as
 * they are. A row whose position is outside [0, rope_len) or outside the cache
 * is skipped, so -1 pads a batch. Two rows of one call must not name the same
 * token: which of them the slot then holds is not specified (it may mix the
 * two). A code is exact: the rounding of the real quotient, also next to a
 * border. The scale is one rounding of amax / 127; a rotated key's amax is that
 * of its f32 values, three roundings each. */
int fs_kv_q8_append(const fs_kv_q8* cache, const void* k, const void* v, int64_t k_stride,
                    int64_t v_stride, int32_t dtype, const int32_t* lanes,
                    const int32_t* positions, int32_t n, const float* rope_cos,
                    const float* rope_sin, int32_t rope_len, void* stream);

/* Reads n tokens back: the values of token positions[i] of lane lanes[i] into
 * row i of k_out and v_out (either may be NULL; strides and dtype as for
 * fs_kv_q8_append, one rounding of code * scale to f32 and one more to the
 * nearest finite bf16: a stored infinity reads as the type's largest value).
 * A token that the cache cannot hold reads as zeros. */
int fs_kv_q8_read(const fs_kv_q8* cache, const int32_t* lanes, const int32_t* positions,
                  int32_t n, void* k_out, void* v_out, int64_t k_stride, int64_t v_stride,
                  int32_t dtype, void* stream);

/* Bytes of workspace fs_kv_q8_attention needs for the same n, n_heads,
 * max_len and split_len on the current device (0 when no row is split), or a
 * negative FS_ERR_* code. Only n_kv_heads, page_size, head_dim and max_pages
 * of the cache are looked at. */
int64_t fs_kv_q8_attention_workspace(const fs_kv_q8* cache, int32_t n, int32_t n_heads,
                                     int32_t max_len, int32_t split_len);

/* Attention of one new token a row: row i attends to tokens 0 .. lengths[i] - 1
 * of lane lanes[i]. q and out are n rows of [n_heads][head_dim] of dtype
 * (FS_DTYPE_F32 or _BF16), q_stride and out_stride elements apart; head h reads
 * KV head h / (n_heads / n_kv_heads), at most 8 heads per KV head. scale
 * multiplies the scores (usually 1 / sqrt(head_dim)). With rope_cos / rope_sin
 * q is rotated by position lengths[i] - 1 (the token it belongs to). max_len is
 * an upper bound of the lengths, which sizes the launch (0: max_pages *
 * page_size; at most rope_len when q is rotated): a longer row is taken as one of
 * max_len tokens, in what it attends to and in the rotation of its q. A row of
 * length 0 (or less), or whose tokens the cache does not hold, gives zeros.
 * Several rows may name one lane (the rows of a drafted continuation, each with
 * its own length).
 *
 * Long rows are cut into splits of split_len tokens (a multiple of 64; at most
 * 8192 splits), joined in a fixed order; 0 chooses from n, n_kv_heads, head_dim,
 * max_len and the device. A row's bits depend on its own inputs and split_len
 * alone: give split_len for results that do not depend on the batch. Scores,
 * softmax sums, partial results and outputs are held in f32; q and the weights
 * enter the products as two f16 parts each, 22 bits (weights to fewer where the
 * scales of all values are below 2^-97); the result is rounded once. A head
 * whose q is not finite gives NaN and leaves the others alone. workspace (16-byte aligned) may be NULL
 * when fs_kv_q8_attention_workspace says 0, is needed only during the call's
 * own kernels and starts with any content; calls that may run at the same time
 * (other streams, other captured graphs) need one each. */
int fs_kv_q8_attention(const fs_kv_q8* cache, const void* q, int64_t q_stride,
                       const int32_t* lanes, const int32_t* lengths, int32_t n,
                       int32_t n_heads, int32_t max_len, float scale, const float* rope_cos,
                       const float* rope_sin, int32_t rope_len, void* out, int64_t out_stride,
                       int32_t dtype, int32_t split_len, void* workspace,
                       int64_t workspace_bytes, void* stream);

/* Verifies drafted tokens against the target's logits (the step after
 * fs_step_batch_chunked on a drafted continuation; the rejected suffix then
 * leaves the cache with fs_lane_evict). Sequence s owns rows row_start[s] ..
 * row_start[s + 1] - 1 of logits (f32 [n_rows][vocab], rows logits_stride
 * elements apart): one row per drafted token, in order, and one more for the
 * token after them all. Row r's draft is draft[r], drawn by the draft model
 * with the probabilities draft_probs row r (f32 [n_rows][vocab], rows
 * probs_stride apart) or, when draft_probs is NULL, given without any (a lookup
 * in the prompt: probability 1); the last row of a sequence has no draft, its
 * entries are not read. With z the row's logits and p = softmax(z / T),
 * T = temps[s], in order:
 *   accept draft x while u_accept[r] * q(x) < p(x);
 *   at the first that is not accepted the next token is drawn from
 *   max(p - q, 0) (without probabilities: p with x taken out; p itself if
 *   nothing is left); if all are, from the last row's p.
 * The draw takes the first token whose running sum of weights reaches
 * u_sample[s] times their total and whose weight is not zero. T = 0 (or
 * not positive) is greedy: x is accepted when it is the row's argmax, and the
 * next token is the argmax (lowest index on ties). Logits of -inf or NaN have
 * no probability; equal +inf logits share all of it; a row with no token at all
 * accepts nothing and gives token 0. A draft outside [0, vocab) is never
 * accepted. Random numbers are in [0, 1); T is held in [1e-30, 1e30]. What is
 * decided in f32 is clear of its border by more than f32 may be off; the rest is
 * decided from weights held to a relative 2^-36 and summed in pairs of f32
 * numbers. A weight below 2^-126 of the largest is 0, one below 2^-125 may be.
 * Writes n_accepted[s] and next_token[s]; a sequence without rows gets 0
 * and -1. row_start has n_seqs + 1 ascending entries in [0, n_rows] (others are
 * clamped). Pointers, stream and errors as for fs_kv_q8_append. */
int fs_verify_draft(const float* logits, int64_t logits_stride, int32_t n_rows, int32_t vocab,
                    const int32_t* row_start, int32_t n_seqs, const int32_t* draft,
                    const float* draft_probs, int64_t probs_stride, const float* temps,
                    const float* u_accept, const float* u_sample, int32_t* n_accepted,
                    int32_t* next_token, void* stream);

/* ---- what differs from request to request in a step: operators on the
 * caller's device buffers -----------------------------------------------------
 *
 * Pages and slots of the new tokens (fs_pages_update), their rotary positions
 * (fs_rope), each request's low-rank adapter beside a shared projection
 * (fs_lora_add) and its sampling settings (fs_sample_filtered). Pointers are
 * DEVICE pointers on the current device, owned by the caller and used until the
 * stream has passed the call, unless they are said to be HOST pointers. The calls
 * enqueue on `stream` (a cudaStream_t, NULL = default stream), allocate nothing,
 * need no workspace, do not synchronise, and can be captured into a graph. Arrays
 * are aligned to their element type.
 * Errors, with nothing enqueued: FS_ERR_ARG (a NULL pointer, a size, a type, an
 * alignment, overlapping buffers, memory of another device or of the host);
 * FS_ERR_CUDA (a launch failed: of fs_pages_update's two, for many rows, the first may
 * have run). */

/* Page tables and slot maps, kept on the GPU: one call lets lanes give up tokens
 * and take new ones. The pool is holders[n_pages] (how many lanes hold a page, 0:
 * free), a lane's pages are page_table[lane][0 .. ceil(length / page_size)) of
 * [n_lanes][max_pages], lengths[lane] its tokens: the page table of fs_kv_q8.
 *   1. lane l keeps its first min(lengths[l], keep[l]) tokens (keep NULL: all).
 *      Pages past their end lose a holder and their table entries become -1: a
 *      rejected draft's suffix, or (keep 0) a finished request.
 *   2. lane l takes grow[l] more tokens. The pages that needs are the lowest free
 *      ones, ascending, lanes in order, and get one holder; pages let go by 1. are
 *      free already. All lanes grow or none does.
 *   3. each new token is a row, lanes in order and tokens ascending: lane l's rows
 *      are row_start[l] .. row_start[l + 1] - 1 (n_lanes + 1 entries), and a row's
 *      row_lane, row_position (the token's place in its lane), row_length (that
 *      plus 1) and row_slot (page * page_size + place in the page) are what
 *      fs_kv_q8_append, fs_rope and fs_kv_q8_attention take. Rows up to max_rows
 *      behind the last get lane, position and slot -1 and length 0, which pad a
 *      batch there. row_lane, row_position, row_length and row_slot may each be NULL
 *      (max_rows limits the rows all the same); row_start is always written.
 * status (int32 [4]): FS_OK or why no lane grew, rows wanted, pages wanted, pages
 * that were free for them (counts past 2^31 - 1 as that). FS_ERR_KV_FULL: too few
 * free pages, or a lane past max_pages * page_size tokens; FS_ERR_SCRATCH: more than
 * max_rows rows; FS_ERR_STATE: a lane would grow into a partial last page that it does not
 * hold alone (one that another lane shares must be copied first; an entry outside the pool,
 * or of a page without holders, is none). 1. has happened then too, row_start is all 0 and
 * every row padding.
 * Lengths are taken as in [0, max_pages * page_size], negative keep and grow as 0. A
 * let go entry outside [0, n_pages) is only cleared, and a page that nobody holds
 * stays free. A page that several lanes hold is one that no lane writes: a lane that
 * shares its last, partial page must be given a copy before it grows. At most 8192
 * lanes; max_pages * page_size at most 2^30. One call at a time on one pool. */
int fs_pages_update(int32_t* holders, int32_t n_pages, int32_t* page_table, int32_t* lengths,
                    int32_t n_lanes, int32_t max_pages, int32_t page_size, const int32_t* keep,
                    const int32_t* grow, int32_t* row_start, int32_t* row_lane,
                    int32_t* row_position, int32_t* row_length, int64_t* row_slot,
                    int32_t max_rows, int32_t* status, void* stream);

/* How a model's frequencies are scaled for contexts longer than it was trained on. */
#define FS_ROPE_SCALING_NONE 0
#define FS_ROPE_SCALING_LINEAR 1 /* f / factor (position interpolation)           */
#define FS_ROPE_SCALING_BASE 2   /* theta * factor^(r / (r - 2)), r = rotary_dim (a
                                    factor of factor * len / original - (factor - 1)
                                    is its dynamic form)                         */
#define FS_ROPE_SCALING_RAMP 3   /* pairs below `lo` keep f, above `hi` take f /
                                    factor, between a linear mix; lo and hi are where
                                    a pair turns `high` and `low` times over
                                    `original` tokens, rounded outwards to [0, r - 1]
                                    ("YaRN", Peng et al. 2023); turned values are
                                    multiplied by 0.1 ln(factor) + 1 (factor > 1) */
#define FS_ROPE_SCALING_BANDS 4  /* pairs that turn at least `high` times over
                                    `original` tokens keep f, at most `low` times
                                    take f / factor, between a mix linear in turns */
typedef struct fs_rope_scaling {
  int32_t kind;
  int32_t original; /* tokens of the trained context (RAMP, BANDS)                */
  double factor;    /* > 0                                                        */
  double low;       /* RAMP: usually 1; BANDS: usually 1. 0 < low < high          */
  double high;      /* RAMP: usually 32; BANDS: usually 4                         */
} fs_rope_scaling;

/* Frequencies for fs_rope: inv_freq[j] (HOST, rotary_dim / 2 entries) = the angle a
 * position turns pair j by, theta^(-2 j / rotary_dim) scaled, and *factor_out (HOST)
 * the factor of the turned values (1 but for RAMP). Host arithmetic in 64 bits, no
 * device needed; scaling NULL is NONE. Errors: FS_ERR_ARG. */
int fs_rope_frequencies(int32_t rotary_dim, double theta, const fs_rope_scaling* scaling,
                        double* inv_freq, double* factor_out);

#define FS_ROPE_INTERLEAVED 1 /* pairs (2 j, 2 j + 1); else (j, j + rotary_dim / 2) */
#define FS_ROPE_INVERSE 2     /* turns by minus the angle                          */

/* Rotary positions of n rows of queries [n_heads][head_dim] and keys
 * [n_kv_heads][head_dim] (k NULL: queries alone), rows *_stride elements apart, of
 * dtype FS_DTYPE_F32 or _BF16: with a = positions[i] * inv_freq[j], pair j (x, y) of the
 * first rotary_dim values of each head becomes factor * (x cos a - y sin a, y cos a + x
 * sin a); the other values are copied. q_out may be q (in place, same stride), and k_out
 * k; buffers must not overlap otherwise. A negative position skips its row, which is
 * neither read nor written: -1 pads a batch. inv_freq is a HOST array of rotary_dim / 2
 * numbers within 2^20, read during the call. Angles are reduced as 64-bit fractions of a turn,
 * the first 48 bits of which are used (off by at most position * 2^-65 + 2^-48 turns), sines
 * and cosines are f32, and a result is rounded once to dtype. head_dim at most 1024,
 * rotary_dim even, at most 512, n_heads and n_kv_heads at most 65535. */
int fs_rope(const void* q, int64_t q_stride, int32_t n_heads, const void* k, int64_t k_stride,
            int32_t n_kv_heads, int32_t n, int32_t head_dim, int32_t dtype,
            const int32_t* positions, const double* inv_freq, int32_t rotary_dim, double factor,
            int32_t flags, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
            void* stream);

/* Low-rank adapters of many requests beside a shared projection: for rows i < n with
 * a = adapter[i] in [0, n_adapters),
 *   out[i] = base[i] + scale[a] * B[a] (A[a] x[i]),
 * other rows give out[i] = base[i]. x is n rows of K (x_dtype), base and out n rows of N
 * (y_dtype; FS_DTYPE_F32 or _BF16 each), strides in elements. base is what the projection
 * gave; it may be out (in place, same stride: rows without an adapter are then not
 * touched), or NULL for 0; buffers must not overlap otherwise. A [n_adapters][rank][K] and
 * B [n_adapters][N][rank] are bf16, 16-byte aligned; rank is a multiple of 8, at most 128
 * (smaller ones padded with zeros), K a multiple of 8; K and N at most 2^24. scale is f32
 * [n_adapters]. Rows may come in any order and mix; rows of one adapter within a block of
 * rows share its reads.
 * Products are exact, sums f32; A x is kept to 24 bits for f32 out and 16 for bf16; the
 * result is rounded once. scale multiplies A x; with infinities and NaN in x, A and B a
 * result is what that gives, and other rows and columns are as without them. A row's bits
 * depend on its own inputs alone, not on the batch. */
int fs_lora_add(const void* x, int64_t x_stride, int32_t x_dtype, const int32_t* adapter,
                int32_t n, int32_t K, int32_t N, const uint16_t* A, const uint16_t* B,
                const float* scale, int32_t n_adapters, int32_t rank, const void* base,
                int64_t base_stride, void* out, int64_t out_stride, int32_t y_dtype,
                void* stream);

/* One token a row from given random numbers, with each row's own settings. logits are
 * n rows of f32 [vocab], logits_stride apart (what fs_decode_step_batch writes). Tokens
 * rank by their logits, the larger first, and of equal ones the lower index. With w =
 * exp((z - max z) / temps[i]):
 *   top-k: the first top_k[i] tokens stay (0 or less: all);
 *   top-p: of those, the tokens ahead of which less than top_p[i] of their sum lies
 *          (1 or more: all; the first always stays);
 *   min-p: of those, the tokens with w >= min_p[i], and the first (0 or less: all).
 * The token is the first by index whose running sum of the kept weights reaches u[i]
 * (in [0, 1)) times their total and whose weight is not 0. temps[i] = 0 (or not
 * positive) takes the first in rank. kept[i] (kept may be NULL) is how many stay: 1 for
 * temps[i] = 0. top_k, top_p and min_p may each be NULL: all stay. Logits of -inf or NaN never stay; equal +inf
 * logits share all of the weight; a row without a token gives token 0 and kept 0. temps is
 * held in [1e-30, 1e30]; a NaN in top_p or min_p turns it off. Weights are good to a
 * relative 2^-37 and summed as whole numbers and as pairs of f32 numbers, so that a cut or a
 * draw is that of the real numbers but next to a border. A weight below 2^-125 of the
 * largest is 0; in the sums over runs of tokens one below 2^-54 of it may count as that
 * much. vocab is at most 2^20, n below 2^28. */
int fs_sample_filtered(const float* logits, int64_t logits_stride, int32_t n, int32_t vocab,
                       const float* temps, const int32_t* top_k, const float* top_p,
                       const float* min_p, const float* u, int32_t* tokens, int32_t* kept,
                       void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FS_H_ */
