/*
 * qg.h -- C ABI of libqg: dequantize-fused low-bit weight matrix-vector
 * product (batch-1 LLM decode), its small-batch and prefill matrix-matrix
 * form, a fused greedy (argmax) output head, and the embedding-row gather
 * from the same 4-bit matrix, for AMD MI355X (gfx950); and the serving-step
 * operators between those products: a paged key/value cache held in 4 bits
 * with its page plan, append, read-back and attention, and the log
 * probabilities of given tokens (second part of this file); and microscaled
 * (MX) numbers with their products and the router, sort and products of an
 * experts' layer (third part).
 *
 * Notation. W is M x K (M outputs, K inputs). Activations x are float32
 * [rows][K], outputs y are float32 [rows][M]; every array is row-major and
 * contiguous. For every output,
 *
 *     y[n][m] = sum over k of w[m][k] * x[n][k]
 *
 * where w[m][k] is the real weight decoded from the packed format below,
 * and the sum is carried in float32 (any order; the result is within
 * 1e-5 * sum_k |w[m][k] * x[n][k]| of the exact value).
 *
 * Weight formats
 *
 *   QG_I8_ROW   codes  int8  [M][K]      two's complement, any value
 *               scales fp32  [M]         w = scales[m] * q
 *               biases must be NULL.  K must be a multiple of 16.
 *     (MiniCPM-V-4.6 on a Tesla C2075, academ.us 2607.14568, section 2.3
 *     "Quantization and residency" and section 3.3 "Decode, and why 4-bit
 *     is slower": symmetric 8-bit weights with an FP32 scale, read without
 *     unpacking; here the scale is per row.)
 *
 *   QG_I8_G64   codes  int8  [M][K]      two's complement, any value
 *               scales fp32  [M][K/64]   w = scales[m][k/64] * q
 *               biases must be NULL.  K must be a multiple of 64.
 *     (MiniCPM-V-4.6 on a Tesla C2075, section 2.3: symmetric 8-bit codes,
 *     each run of 64 sharing an FP32 factor, as that backbone ships them.)
 *
 *   QG_U4_G64   codes  uint8 [M][K/2]    byte j of a row: k=2j in bits 0..3,
 *                                        k=2j+1 in bits 4..7, q in 0..15
 *               scales bf16  [M][K/64]   (uint16 bit patterns)
 *               biases bf16  [M][K/64]
 *               w = scales[m][k/64] * q + biases[m][k/64].  K multiple of 64.
 *     (Pushing the limits of legacy hardware, "Start with the machine that
 *     actually exists": group-64 affine 4-bit codes with bf16 scale and bias;
 *     I Built an LLM Inference Engine on a 15 year old GPU..., "Quantization:
 *     The Model Doesn't Run on INT4": code times scale plus the minimum.)
 *
 *   QG_B1_G128  codes  uint8 [M][K/8]    bit (k mod 8) of byte k/8, least
 *                                        significant bit first
 *               scales fp16  [M][K/128]  (uint16 bit patterns)
 *               w = +scales[m][k/128] if the bit is 1, -scales[..] if 0.
 *               biases must be NULL.  K multiple of 128.
 *     (A 27B model on two 4GB Maxwell GPUs: inference tuning, "Why this
 *     machine is awkward": binary weights with FP16 scales.)
 *
 * Conventions shared by every entry point
 *
 *   Ownership   The caller owns every buffer. All data pointers are device
 *               pointers (hipMalloc'd or equivalent) and stay resident; the
 *               library never allocates, frees, copies to or from the host,
 *               or synchronizes. (I Built an LLM Inference Engine..., "The
 *               memory movement problem" and "Cost 2": weights live on the
 *               device, and nothing is allocated on the hot path.)
 *   Streams     Work is enqueued on `stream` (0 = the null stream) and the
 *               call returns without waiting for it.
 *   Alignment   codes, scales, biases, x, y / logits / out and ws must be
 *               16-byte aligned; idx and ids 4-byte aligned.
 *   Aliasing    The written buffers (y or logits, idx, out, ws) must not overlap
 *               each other or any input.
 *   Errors      Every argument error is detected on the host before
 *               anything is enqueued; the outputs are then left untouched
 *               and a negative QG_ERR_* code is returned. QG_ERR_LAUNCH
 *               reports a failed kernel launch (hipGetLastError).
 *               (Pushing the limits of legacy hardware, "Build the execution
 *               path, then share the weights": a request that cannot be
 *               served fails before changing live state.)
 *   Threads     The library keeps no mutable state; calls are reentrant.
 *               Calls that share a workspace must not overlap in time; two
 *               that do (on different streams) may both return wrong
 *               results, but the calls after them are not affected.
 *   Workspace   `ws` is device memory of at least qg_workspace_bytes(...)
 *               bytes for the same (op, fmt, M, K, rows); it may be NULL
 *               when that size is 0. Its contents on entry do not matter,
 *               so freshly allocated memory serves. Its first
 *               QG_WS_CONTROL_BYTES bytes are completion words (counters of
 *               finished workgroups, for the greedy head and for combining
 *               partial sums of K chunks), each tagged by the kernel launch
 *               that counts on it and claimed afresh by every launch, so a
 *               call that was cut short, or stale or uninitialised words,
 *               cannot disturb a later call. The rest is scratch (partial
 *               sums, parked argmax keys). The workspace is caller-owned
 *               device memory because the library allocates nothing on the
 *               hot path (I Built an LLM Inference Engine on a 15 year old
 *               GPU..., "Cost 2").
 */
#ifndef QG_H
#define QG_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QG_ABI_VERSION 2

typedef enum {
    QG_I8_ROW = 1,
    QG_U4_G64 = 2,
    QG_B1_G128 = 3,
    QG_I8_G64 = 4
} qg_format;

typedef enum {
    QG_OP_GEMV = 1,
    QG_OP_GEMM = 2,
    QG_OP_GEMV_ARGMAX = 3
} qg_op;

enum {
    QG_OK = 0,
    QG_ERR_NULL = -1,        /* a required pointer is NULL, or biases given where none belong */
    QG_ERR_FORMAT = -2,      /* unknown format or element type */
    QG_ERR_SHAPE = -3,       /* a size, stride or count out of range or not a multiple of its unit */
    QG_ERR_ALIGN = -4,       /* a pointer is not aligned as required */
    QG_ERR_WORKSPACE = -5,   /* ws_bytes smaller than qg_workspace_bytes(...) (or the entry
                                point's own ..._workspace_bytes) */
    QG_ERR_ALIAS = -6,       /* a written buffer overlaps another buffer */
    QG_ERR_LAUNCH = -7,      /* the kernel launch failed */
    QG_ERR_UNSUPPORTED = -8, /* a known format this entry point does not implement
                                (only qembed returns it: 4-bit rows only) */
    QG_ERR_SCRATCH = -9      /* the call needs more than QG_STATIC_SCRATCH_BYTES of
                                the library's own scratch (qgemv_argmax_noalloc) */
};

/* Control words at the start of every workspace (see Workspace above). */
#define QG_WS_CONTROL_BYTES 8192

/* Largest batch of qgemv / qgemv_argmax. */
#define QG_MAX_GEMV_BATCH 16
/* Largest batch of the greedy head (qgemv_argmax); above QG_MAX_GEMV_BATCH
 * it runs as the prefill product with per-tile argmax keys. */
#define QG_MAX_ARGMAX_BATCH 256

/*
 * qgemv -- batch-1 (up to QG_MAX_GEMV_BATCH) quantized matrix-vector product.
 *   y[n][m] = sum_k w[m][k] * x[n][k],  0 <= n < batch, 0 <= m < M.
 * Every packed weight is read once per call (4-bit, 9 to 16 rows on the
 * small-batch matrix-core kernel: once per launch of up to 8 rows),
 * dequantized in registers and never written out. Batches of 2 to 16 rows
 * may run on the prefill kernel (see qgemm) where that is expected to be
 * faster; the result contract is the same. (MiniCPM-V-4.6 on a Tesla
 * C2075, section 3.3: decode reads each weight once and is bandwidth-bound;
 * I Built an LLM Inference Engine..., "Optimization 4: Quantized Kernels":
 * dequantization is fused into the product.)
 *   x  float32 [batch][K];  y  float32 [batch][M] (overwritten).
 *   1 <= M <= 2^31-1, 1 <= K <= 2^30, 1 <= batch <= QG_MAX_GEMV_BATCH.
 */
int qgemv(int fmt, const void *codes, const void *scales, const void *biases,
          const float *x, float *y, int64_t M, int64_t K, int batch,
          void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * qgemm -- prefill form: the same product over N token rows.
 *   Y[n][m] = sum_k w[m][k] * X[n][k],  0 <= n < N.
 * (MiniCPM-V-4.6 on a Tesla C2075, section 3.1 "Prefill projections": the
 * prompt's projections contract whole matrices, not vectors; A 27B model on two
 * 4GB Maxwell GPUs, "A packed Q1 prefill kernel with a narrow dispatch
 * window": the weights may be consumed packed.)
 *   X  float32 [N][K];  Y  float32 [N][M] (overwritten).  1 <= N <= 2^31-1;
 *   above QG_MAX_GEMV_BATCH rows (the matrix-core kernel) K <= 2^21.
 *   All four formats; for QG_U4_G64 the bias term sum_g b[m][g] * (sum of
 *   X[n][k] over group g) is added per group beside the scaled code sums.
 *   Needs a workspace when qg_workspace_bytes(QG_OP_GEMM, ...) is nonzero:
 *   up to QG_MAX_GEMV_BATCH rows as qgemv, and above that whenever the
 *   output has too few tiles to fill the chip (fewer than one per compute
 *   unit; two for the 8-bit formats, four for the 1-bit format) or a short
 *   last round of tiles, since K is then cut into pieces whose float32
 *   partial products are added in a fixed order by a second launch (the
 *   result does not depend on the stream or the schedule). 17..48 rows of the 4-bit format at K = 1024 or 2048 may
 *   run as launches of up to QG_MAX_GEMV_BATCH rows of the matrix-vector
 *   product where that reads the weights for less than the prefill kernel's
 *   padded work costs.
 */
int qgemm(int fmt, const void *codes, const void *scales, const void *biases,
          const float *x, float *y, int64_t M, int64_t K, int64_t N,
          void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * qgemv_argmax -- qgemv followed by greedy selection, fused.
 *   logits[n][m] = y[n][m] as qgemv computes it (float32, written),
 *   idx[n]       = the lowest m whose logits[n][m] is the maximum of row n
 *                  (ties go to the lowest index; -0 equals +0).
 * (Pushing the limits of legacy hardware, "Build the execution path, then
 * share the weights": for greedy decoding the head only has to report, per
 * tile of logits, the largest value and where it sits, and the choice of
 * token is made on the device.)
 *   logits  float32 [batch][M], or NULL: then no logits are written (the
 *           greedy-only head; the maxima still come from the same float32
 *           values a non-NULL call writes).
 *   idx     int32 [batch].
 *   1 <= batch <= QG_MAX_ARGMAX_BATCH; other limits as qgemv, and K <= 2^21
 *   above QG_MAX_GEMV_BATCH rows. Up to
 *   QG_MAX_GEMV_BATCH rows use the matrix-vector kernels; more rows use the
 *   prefill kernels, which keep one (value, index) key per tile (or part of
 *   one) and token row in the workspace and reduce them in a second launch
 *   (the per-tile reduction of the page above), except 17..48 rows of the
 *   4-bit format at K = 1024 or 2048, which may run as launches of up to
 *   QG_MAX_GEMV_BATCH rows on the matrix-vector kernels. Needs a workspace.
 */
int qgemv_argmax(int fmt, const void *codes, const void *scales,
                 const void *biases, const float *x, float *logits,
                 int32_t *idx, int64_t M, int64_t K, int batch,
                 void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * qgemv_argmax_noalloc -- qgemv_argmax without a caller workspace, for
 * callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation). Same arguments,
 * results and limits as qgemv_argmax; the workspace it would need comes from
 * a static array of QG_STATIC_SCRATCH_BYTES bytes that the library keeps on
 * each GPU it runs on until the process ends. The call allocates nothing
 * (no hipMalloc, hipFree or allocating library routine); its first call on
 * a device looks up that device's array (the device must be current, as
 * for every call). Calls that need more scratch than the array holds return
 * QG_ERR_SCRATCH before anything is enqueued. Every call on a GPU shares
 * that GPU's array: calls that overlap in time on one GPU (different
 * streams or host threads) race and may return wrong results, though calls
 * after them are not affected. Nothing in the array has to be cleared
 * between calls (its completion words are claimed by each launch).
 */
#define QG_STATIC_SCRATCH_BYTES (8u << 20)
int qgemv_argmax_noalloc(int fmt, const void *codes, const void *scales,
                         const void *biases, const float *x, float *logits,
                         int32_t *idx, int64_t M, int64_t K, int batch,
                         hipStream_t stream);

/*
 * qembed -- embedding rows gathered from the (tied) 4-bit weight matrix.
 *   out[t][k] = e(ids[t], k),  0 <= t < n, 0 <= k < K, where for a row m
 *   inside the table e(m, k) is decoded as three rounded steps:
 *     p = scales[m][k/64] * q        (float32; exact, 8 x 4 significant bits)
 *     a = p + biases[m][k/64]        (float32, round to nearest even; the
 *                                     product and the sum are not fused)
 *     e = a rounded to IEEE binary16 (nearest even, subnormals kept,
 *         overflow to infinity) and widened back to float32.
 *   A zero sum is -0 only when both terms are -0 (IEEE 754 sums under
 *   nearest-even), and a negative sum too small for binary16 becomes -0,
 *   not +0. A row id outside [0, M) gives a row of quiet NaNs.
 * (Pushing the limits of legacy hardware, "Half a billion values, and one
 * negative zero": that row decoder multiplies and adds in two steps and
 * passes each value through FP16 on its way to FP32, and the lookup on the
 * GPU had to reproduce denormals, the sign of zero and round-to-nearest-even
 * exactly; I Built an LLM Inference Engine..., "Cost 1: the embedding lookup
 * still runs on the CPU": the quantized rows are decoded on the device from
 * token ids instead of crossing PCIe.)
 *   fmt     QG_U4_G64 only; the other known formats give QG_ERR_UNSUPPORTED.
 *   ids     int32 [n], device memory (4-byte aligned); any values.
 *   out     float32 [n][K] (overwritten).
 *   1 <= n <= 2^31-1; M and K as qgemv. No workspace.
 */
int qembed(int fmt, const void *codes, const void *scales, const void *biases,
           const int32_t *ids, float *out, int64_t M, int64_t K, int64_t n,
           hipStream_t stream);

/* Bytes of device workspace the call (op, fmt, M, K, rows) needs; rows is
 * the batch for QG_OP_GEMV / QG_OP_GEMV_ARGMAX and N for QG_OP_GEMM.
 * Returns 0 when no workspace is needed, and also for arguments the entry
 * point would reject (the entry point then reports the error). The caller
 * allocates it once, off the hot path, and may reuse it for every call of
 * the same or a smaller size (I Built an LLM Inference Engine..., "Cost 2":
 * nothing is allocated per call; Pushing the limits of legacy hardware,
 * "Build the execution path, then share the weights": the greedy head
 * keeps per-tile (value, index) pairs instead of whole logits, which is
 * what the argmax part of the workspace holds). */
size_t qg_workspace_bytes(int op, int fmt, int64_t M, int64_t K, int64_t rows);

/* ------------------------------------------------------------------------
 * Serving-step operators
 *
 * One decode or prefill step of a batch of requests runs, between the
 * products above, qkv_plan (pages and slots of the new tokens), qkv_append
 * (their keys and values into the cache), qkv_attn (attention over the
 * cache) and, after the output head, qlogprobs. The conventions of the top
 * of this file hold (ownership, streams, aliasing, errors, threads);
 * contents of device memory, such as lengths, page and slot numbers, cannot
 * be checked on the host, so each entry point states what it makes of
 * contents out of range. None of them reads or writes out of its buffers
 * for any contents.
 *
 * The cache. Keys and values are held as the products' 4-bit weights are:
 * groups of 64 consecutive channels of one token's head share a bf16 scale
 * and a bf16 bias, value = scale * code + bias, code 0..15 (I Built an LLM
 * Inference Engine on a 15 year old GPU..., "Quantization: The Model
 * Doesn't Run on INT4": code times scale plus the minimum; Pushing the
 * limits of legacy hardware, "Start with the machine that actually exists":
 * group-64 codes with bf16 scale and bias). The cache is num_pages pages of
 * page_size tokens; one page of one head is one contiguous block of
 *
 *     page_size * (head_dim + head_dim / 8) bytes:
 *       K codes  uint8 [page_size][head_dim/2]   channel 2j in bits 0..3 of
 *                                                byte j, 2j+1 in bits 4..7
 *       K coefs  bf16  [page_size][head_dim/64][2]   (scale, bias)
 *       V codes, V coefs   the same
 *
 * ordered [num_pages][kv_heads]. A slot is page * page_size + (place within
 * the page). A whole step's cache is thus one allocation, kept resident (I
 * Built an LLM Inference Engine..., "Optimization 3": keys and values live
 * in preallocated memory).
 * ------------------------------------------------------------------------ */

typedef enum {
    QG_F32 = 1,   /* float32 activations */
    QG_BF16 = 2   /* bfloat16 activations */
} qg_dtype;

typedef struct {
    void *data;          /* device memory, 16-byte aligned, the size above times num_pages * kv_heads */
    int64_t num_pages;   /* >= 1; num_pages * page_size <= 2^31 - 1 */
    int32_t page_size;   /* 16, 32, 64, 128 or 256 tokens */
    int32_t kv_heads;    /* 1..1024 */
    int32_t head_dim;    /* 64, 128 or 256 */
} qg_kv_cache;

/* Bytes of a cache of this geometry (data is not looked at); 0 if it is invalid. */
size_t qkv_cache_bytes(const qg_kv_cache *cache);

/*
 * qkv_plan -- pages, lengths, row starts and slots of a step, from lengths.
 * Request b holds len_old[b] tokens in ceil(len_old/page_size) pages, whose
 * numbers start its row of block_table. It keeps its first keep[b] tokens
 * (fewer after rejected speculation, 0 when it has ended) and gets n_new[b]
 * new ones. Pages are taken from and given back to a ring of free pages:
 * state_in = {head, tail} are running counts, entry i is
 * ring[i mod ring_size], the free pages are entries head..tail-1.
 *   have = ceil(len_old/page), want = ceil((keep + n_new)/page).
 *   A request with want > have takes want - have pages from the front of the
 *   ring, requests being served in order; it is denied if they and those of
 *   the requests before it exceed the pages that were free before the call,
 *   or want > table_stride. A request denied gets no page or slot and falls
 *   back to keep[b] tokens. Pages given back (of shrinking requests, in
 *   request order) go to the ring's end and are not taken in the same call.
 *   block_table  int32 [batch][table_stride], entries have..want-1 of a
 *                growing request written, all others left as they are
 *   ring         int32 [ring_size], written at the tail; ring_size is at
 *                least the number of pages
 *   state_out    int64 [2], the new {head, tail}
 *   kv_len       int32 [batch]    keep + n_new (denied: keep)
 *   cu_q         int32 [batch+1]  running sums of n_new (denied requests
 *                included: their rows exist and are void)
 *   slots, pos   int32 [total]    slot and position of each new token, in
 *                request order; slot -1 for the tokens of a denied request
 *                and where the slot (page * page_size + place) is no int32;
 *                both -1 behind the last token (total may be larger, as
 *                under graph capture; tokens behind total are dropped)
 *   denied       int32 [1]        how many requests were denied
 * state_in and state_out are distinct, so that a step can be planned again.
 * Contents out of range: len_old, keep and n_new are taken into
 * [0, 2^30], keep into [0, len_old], sums past 2^31 - 1 are 2^31 - 1; a negative ring count is no free page;
 * pages of a request behind table_stride are neither read nor given back;
 * page numbers pass through as they are.
 *   1 <= batch <= QG_MAX_PLAN_BATCH, 0 <= total, table_stride >= 1,
 *   ring_size >= 1, page_size a power of two in 1..2^20.
 */
#define QG_MAX_PLAN_BATCH 8192
int qkv_plan(const int32_t *len_old, const int32_t *keep, const int32_t *n_new, int batch,
             int page_size, int32_t *block_table, int64_t table_stride, int32_t *ring,
             int64_t ring_size, const int64_t *state_in, int64_t *state_out, int32_t *kv_len,
             int32_t *cu_q, int32_t *slots, int32_t *pos, int64_t total, int32_t *denied,
             hipStream_t stream);

/*
 * qkv_append -- keys and values of n tokens quantized into their slots.
 *   k, v   [n] rows of kv_heads * head_dim elements of `dtype`, k_stride and
 *          v_stride elements apart (parts of a fused projection's rows)
 *   slots  int32 [n]; a token whose slot is outside the cache is skipped.
 *          Two tokens with one slot leave either token's bytes, mixed.
 * Each group x[0..63] is stored as
 *   scale = bf16((max x - min x) * f), bias = bf16(min x)   (nearest even),
 *   f the float32 nearest 1/15,
 *   code  = round_half_even((x - bias) / scale), into 0..15,
 * in float32 arithmetic. A scale below 2^-126 is stored as 0 with codes 0
 * (the group is its minimum); where scale or bias is not finite (a group
 * with a NaN, an infinity, or a range past bf16) both are stored as NaN
 * with codes 0, so that the group reads as NaN throughout.
 *   0 <= n; strides at least kv_heads * head_dim and multiples of 16 bytes.
 */
int qkv_append(int dtype, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
               const int32_t *slots, int64_t n, const qg_kv_cache *cache, hipStream_t stream);

/*
 * qkv_read -- the values that n slots of the cache stand for.
 *   k, v   [n] rows as in qkv_append, of `dtype` (written): scale * code +
 *          bias in float32 (fused), rounded to nearest even for bfloat16.
 *          Either may be NULL; both may be parts of the same wider rows
 *          (one stride, no shared elements).
 *   slots  a slot outside the cache gives a row of quiet NaNs.
 */
int qkv_read(int dtype, const qg_kv_cache *cache, const int32_t *slots, int64_t n, void *k,
             int64_t k_stride, void *v, int64_t v_stride, hipStream_t stream);

/*
 * qkv_attn -- causal attention of new tokens over the cache.
 * Request b has the query rows cu_q[b]..cu_q[b+1]-1; they are the last of
 * its kv_len[b] tokens, whose keys and values are in the cache already (the
 * new ones too). Row i of request b is token p = kv_len - n_q + i; head h
 * reads key/value head h / (q_heads / kv_heads), and
 *   out = sum_j w_j v_j / sum_j w_j,   w_j = exp(scale * q . k_j),
 *   lse = log sum_j w_j                (natural logarithm)
 * over the tokens j <= p, with window > 0 only those with j > p - window.
 * Codes enter the matrix cores exactly; float32 queries and weights as two
 * binary16 pieces (22 bits), bfloat16 queries exactly and their weights as
 * one; scales, softmax statistics and sums are float32. Every group of 64
 * channels keeps these bits whatever the sizes of the others' values, where
 * its weighted values are not 2^60 times smaller than another's of the head.
 * Queries, and scales and biases of keys, are below 2^100 in size. One token a request
 * is a decode step, a few a speculation's check, many a prompt chunk: one
 * entry point, kernels chosen by the sizes. Results repeat from call to call,
 * on any stream; a row's rounding depends on the kernel, the splits and the
 * rows it shares a tile with, hence on the sizes and on the batch around it.
 *   q, out   rows of q_heads * head_dim elements of `dtype`, q_stride and
 *            out_stride elements apart; both may be parts of the same wider
 *            rows (one stride, no shared elements)
 *   lse      float32 [total_q][q_heads], or NULL
 *   block_table  int32 [batch][table_stride]
 *   max_q    at least the longest request's rows (chooses the kernel; a
 *            smaller value costs time, not correctness)
 *   max_kv   at least the longest kv_len; max_kv <= table_stride * page_size
 * A row that sees no token (kv_len 0, or fewer tokens than rows) gives out 0
 * and lse -infinity. Contents out of range: a request with kv_len > max_kv,
 * and rows that see a page number outside the cache, give NaN; kv_len < 0 is
 * 0; rows outside [0, total_q) do not exist (the others of their request keep
 * their tokens: a call may have fewer rows than the plan that made cu_q), and
 * rows of no request are not
 * written; where the starts in cu_q are not in order, the rows from the
 * least to the largest of them may hold anything. What masked places hold (codes or coefficients of tokens a row
 * does not see, NaN and infinities among them) does not matter.
 *   1 <= batch <= 65535, 1 <= total_q <= 2^31 - 1, 1 <= max_q, 1 <= max_kv
 *   <= 2^30, q_heads a multiple of kv_heads, q_heads <= 1024, total_q *
 *   q_heads <= 2^31 - 1, batch * kv_heads + total_q * q_heads / 16 < 2^24
 *   (a launch's workgroups), scale finite and > 0, window >= 0, strides as in
 *   qkv_append.
 * Workspace: qkv_attn_workspace_bytes(...) for the same arguments (partial
 * sums where the keys of a request are split over workgroups).
 */
int qkv_attn(int dtype, const void *q, int64_t q_stride, const qg_kv_cache *cache,
             const int32_t *block_table, int64_t table_stride, const int32_t *cu_q,
             const int32_t *kv_len, int batch, int64_t total_q, int64_t max_q, int64_t max_kv,
             int q_heads, float scale, int64_t window, void *out, int64_t out_stride, float *lse,
             void *ws, size_t ws_bytes, hipStream_t stream);
size_t qkv_attn_workspace_bytes(const qg_kv_cache *cache, int batch, int64_t total_q, int64_t max_q,
                                int64_t max_kv, int q_heads);

/*
 * qlogprobs -- log probabilities of given tokens, entropy and the best
 * alternatives, from logits such as qgemv_argmax or qgemm writes (Pushing
 * the limits of legacy hardware, "Build the execution path, then share the
 * weights": greedy selection needs only the maxima; sampling, scoring and
 * returned alternatives need the normalised distribution).
 * With x a row and L = log sum_m exp(x[m]):
 *   logprob[n] = x[ids[n]] - L
 *   entropy[n] = -sum_m p[m] log p[m],  p = exp(x - L), 0 log 0 = 0
 *   rank[n]    = 1 + how many tokens come before ids[n] in the order of
 *                larger logits first, ties by lower index
 *   top_ids, top_logprobs [rows][top]: the first `top` tokens of that order
 * -0 equals +0. An id outside [0, vocab) gives logprob NaN and rank 0. A row
 * with a NaN or +infinity, or with nothing but -infinity, has no
 * distribution: logprob, entropy and top_logprobs are NaN; rank and top_ids
 * are then within range but otherwise unspecified.
 *   logits  float32, rows `ld` elements apart (ld >= vocab, 4-byte aligned)
 *   ids     int32 [rows], or NULL (then logprob and rank must be NULL)
 *   logprob, entropy float32 [rows], rank int32 [rows]: each may be NULL
 *   top_ids int32, top_logprobs float32 [rows][top]; both NULL if top is 0
 *   1 <= rows <= 2^31 - 1, 1 <= vocab <= 2^30, 0 <= top <= min(vocab,
 *   QG_MAX_TOP). Workspace: qlogprobs_workspace_bytes(rows, vocab, top).
 */
#define QG_MAX_TOP 64
int qlogprobs(const float *logits, int64_t ld, int64_t rows, int64_t vocab, const int32_t *ids, int top,
              float *logprob, float *entropy, int32_t *rank, int32_t *top_ids, float *top_logprobs,
              void *ws, size_t ws_bytes, hipStream_t stream);
size_t qlogprobs_workspace_bytes(int64_t rows, int64_t vocab, int top);

/* ------------------------------------------------------------------------
 * Microscaled (MX) numbers and experts' layers
 *
 * MX rows hold blocks of 32 consecutive elements that share one scale byte s,
 * which stands for 2^(s - 127); 255 makes the block NaN (OCP Microscaling
 * Formats specification, version 1.0). The matrix cores take both as they lie
 * in memory, so nothing is dequantized on the way.
 *
 *   QMX_E2M1  4 bits: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; byte j
 *             of a row holds k = 2j in bits 0..3 and k = 2j+1 in bits 4..7
 *   QMX_E4M3  8 bits: largest 448, no infinities
 *
 *   codes   uint8 [rows][K/2] or [rows][K], 16-byte aligned
 *   scales  uint8 [rows][qmx_scale_pitch(K)], 4-byte aligned: K/32 bytes and
 *           up to 3 of padding, whose contents do not matter
 *   K is a multiple of 32, 32 <= K <= QMX_MAX_K.
 *
 * Weights are QMX_E2M1 (quantized once with qmx_quant, or brought along),
 * activations either. An experts' layer of a decoder runs qmoe_route (or
 * qmoe_plan, behind a router of one's own), qmx_quant, qmoe_gemm with
 * QMX_SILU_MUL over the gate and up matrices, qmx_quant, qmoe_gemm over the
 * down matrices without `order`, and qmoe_combine. The conventions of the top
 * of this file hold; a call with 0 rows is valid (and writes offsets only).
 * No entry point reads or writes out of its buffers for any contents of
 * offsets, order, slots or ids.
 * ------------------------------------------------------------------------ */

typedef enum {
    QMX_E2M1 = 1,
    QMX_E4M3 = 2
} qmx_format;

typedef enum {
    QMX_NONE = 0,
    QMX_SILU_MUL = 1   /* gate / (1 + exp(-gate)) * up */
} qmx_act;

#define QMX_MAX_K (1 << 21)
#define QMX_MAX_M (1 << 23)
#define QMOE_MAX_EXPERTS 1024
#define QMOE_MAX_TOP 32

/* Bytes from a row of scales to the next: K/32 rounded up to a multiple of 4
 * (0 for a K out of range). */
int64_t qmx_scale_pitch(int64_t K);

/*
 * qmx_quant -- rows of activations (or weights) quantized into MX blocks.
 * With E the exponent field of the block's largest magnitude (as float32),
 *   s = max(E - emax, 0),  emax = 2 (QMX_E2M1) or 8 (QMX_E4M3),
 * and each element is x * 2^(127 - s) rounded to the nearest element, ties to
 * the even code, beyond the largest element to that one; the sign of a zero
 * is kept. A block with a NaN or an infinity gets s = 255 and codes 0.
 * Padding bytes of scales are written as 0.
 *   x  rows of K elements of `dtype` (qg_dtype), x_stride elements apart
 *      (x_stride >= K, a multiple of 16 bytes)
 *   0 <= rows <= 2^31 - 1.
 */
int qmx_quant(int dtype, const void *x, int64_t x_stride, int64_t rows, int64_t K, int fmt,
              void *codes, void *scales, hipStream_t stream);

/*
 * qmx_dequant -- the values that MX rows stand for: element * 2^(s - 127),
 * exact in float32 (past its range infinity; from 2^-149 on down rounded), rounded to
 * nearest even for QG_BF16. Blocks with s = 255 are quiet NaNs.
 */
int qmx_dequant(int fmt, const void *codes, const void *scales, int64_t rows, int64_t K,
                int dtype, void *x, int64_t x_stride, hipStream_t stream);

/*
 * qmx_gemm -- product of MX rows with MX weights, from one row to long prompts.
 *   y[n][m] = sum over k of x[n][k] * w[m][k],  0 <= n < N, 0 <= m < M,
 * with QMX_SILU_MUL W has 2 M rows, and of g from rows 0..M-1 and u from rows
 * M..2M-1, both float32 sums,  y = g / (1 + exp(-g)) * u  (of these sums within
 * 8 roundings to float32 for QG_F32; for QG_BF16 within 2^-15 |y| + 2^-246 |u|
 * and the rounding to it; NaN where g is -infinity).
 * Products of elements and scales are exact; sums are float32, to which blocks of
 * 32 inputs are added one by one (of e4m3 rows twice): a product that is 2^-27 of
 * the sum so far or less may be dropped, and each such addition rounds. Every
 * output is within (K / 8 + 4) * 2^-23 * sum_k |x w| + K * 2^-148 of the exact sum
 * (where sum_k |x w| is out of float32's range, infinity or NaN) before the activation
 * and the rounding to `dtype`. A block with s = 255, or an e4m3 NaN, makes the
 * outputs of its row (of x) or column (of W) NaN. Results repeat from call
 * to call; the rounding of a row depends on how many rows there are.
 *   xfmt   QMX_E2M1 or QMX_E4M3;  W is QMX_E2M1
 *   y      `dtype` [N][M], 16-byte aligned
 *   1 <= M <= QMX_MAX_M, 0 <= N <= 2^31 - 1, the workgroups and tiles of a
 *   launch below 2^24 (QG_ERR_SHAPE).
 * Workspace: qmx_gemm_workspace_bytes(...) for the same arguments (both
 * operands' scales in the order in which tiles of many rows take them).
 */
int qmx_gemm(int xfmt, const void *x_codes, const void *x_scales, const void *w_codes,
             const void *w_scales, int act, int dtype, void *y, int64_t M, int64_t K, int64_t N,
             void *ws, size_t ws_bytes, hipStream_t stream);
size_t qmx_gemm_workspace_bytes(int xfmt, int act, int64_t M, int64_t K, int64_t N);

/*
 * qmoe_plan -- the pairs (token n, choice j), p = n * top + j, of tokens and
 * their experts, sorted by expert.
 *   ids      int32 [rows][top]; a pair whose id is outside [0, experts) has no
 *            expert (none was to be had, or another GPU has it)
 *   offsets  int32 [experts + 1]  places of expert e's pairs: offsets[e] ..
 *            offsets[e + 1] - 1; within an expert pairs keep their order
 *   order    int32 [rows * top]   the pair at each place; -1 behind the last
 *   slots    int32 [rows][top]    the place of each pair; -1 for those of no
 *            expert
 *   0 <= rows, rows * top <= 2^31 - 1, 1 <= top <= min(experts, QMOE_MAX_TOP),
 *   experts <= QMOE_MAX_EXPERTS.
 * Workspace: qmoe_plan_workspace_bytes(...).
 */
int qmoe_plan(const int32_t *ids, int64_t rows, int experts, int top, int32_t *offsets,
              int32_t *order, int32_t *slots, void *ws, size_t ws_bytes, hipStream_t stream);
size_t qmoe_plan_workspace_bytes(int64_t rows, int experts, int top);

/*
 * qmoe_route -- the best `top` experts of each row of a router's logits, with
 * their softmax weights, and the plan of their pairs (as qmoe_plan).
 *   ids[n][j]      the j-th expert of row n in the order of larger logits
 *                  first, ties by lower index (-0 equals +0), among logits
 *                  above -infinity; -1 where there are fewer than top
 *   weights[n][j]  exp(x - L), L = log sum exp over all experts, or with
 *                  renorm = 1 over the chosen ones; 0 where ids is -1
 * A row with a NaN or +infinity has ids -1 and weights NaN.
 *   logits  `dtype` rows, ld >= experts elements apart, aligned to an element
 */
int qmoe_route(int dtype, const void *logits, int64_t ld, int64_t rows, int experts, int top,
               int renorm, int32_t *ids, float *weights, int32_t *offsets, int32_t *order,
               int32_t *slots, void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * qmoe_gemm -- qmx_gemm of each expert over its rows of a plan.
 *   y[s][m] = sum over k of x[r(s)][k] * w[e(s)][m][k]   (or with QMX_SILU_MUL
 *   as there), for places s < offsets[experts]; rows of y behind are left as
 *   they were.
 *   order  r(s) = order[s] / top: x has `rows` rows, gathered on the way; or
 *          NULL, r(s) = s: x has rows * top rows in the plan's order. An entry
 *          outside [0, rows * top) stands for a row of zeros. With order, x_codes
 *          is at most 2^31 - 1 bytes (QG_ERR_SHAPE).
 *   W      QMX_E2M1, the experts' matrices one behind the other: M (or 2 M)
 *          rows each
 *   y      `dtype` [rows * top][M]
 *   offsets that are no plan's (not rising, outside [0, rows * top]): any rows
 *   of y may hold anything.
 * Sizes as qmx_gemm and qmoe_plan. Workspace: qmoe_gemm_workspace_bytes(...).
 */
int qmoe_gemm(int xfmt, const void *x_codes, const void *x_scales, const void *w_codes,
              const void *w_scales, const int32_t *offsets, const int32_t *order, int64_t rows,
              int experts, int top, int act, int dtype, void *y, int64_t M, int64_t K, void *ws,
              size_t ws_bytes, hipStream_t stream);
size_t qmoe_gemm_workspace_bytes(int xfmt, int act, int64_t rows, int experts, int top, int64_t M,
                                 int64_t K);

/*
 * qmoe_combine -- the experts' rows back to their tokens, weighted.
 *   out[n][m] = sum over j of weights[n][j] * y[slots[n][j]][m], in float32 and
 *   in the order of j; a slot outside [0, rows * top) adds weights[n][j] * 0 (so
 *   that a row the router could not read is NaN, and not silently 0).
 *   y  `dtype` [rows * top][M];  out  `out_dtype` [rows][M];  1 <= M <= QMX_MAX_M.
 */
int qmoe_combine(int dtype, const void *y, const int32_t *slots, const float *weights, int64_t rows,
                 int top, int64_t M, int out_dtype, void *out, hipStream_t stream);

/* Static text for a status code. */
const char *qg_status_str(int status);

/* QG_ABI_VERSION of the built library. */
int qg_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QG_H */
