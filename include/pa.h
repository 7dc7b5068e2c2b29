/*
 * pa.h -- C ABI of libpa_gb300: batched attention over a paged key/value pool
 * for a continuous-batching engine, on one NVIDIA GB300 (sm_103a).
 *
 * What it computes ("GPU inference engine engineering", section "Batching
 * without running out of cache"; "Building an LLM runtime from scratch on
 * NVIDIA H100", section "Bug #1"; "llm-rs: LLM Inference in Rust ...",
 * section "4. Going down a level: SIMT kernels"):
 *   - K/V live in a pool of fixed-size pages; each sequence owns a block table
 *     mapping its logical page j (tokens j*P .. j*P+P-1) to a physical page.
 *   - A step is a set of rows; each row carries its own query, sequence id and
 *     position.  pa_append_kv scatters the rows' new keys and values into their
 *     page slots; pa_attention then computes, for every row r and query head g,
 *         out[r][g] = softmax_t( scale * q[r][g] . K_s[t] ) . V_s[t],  t = 0..position
 *     over the row's own sequence s, with kv head g / (Hq / Hkv) (grouped-query
 *     heads), an FP32 online softmax, and a split-KV path for long contexts whose
 *     partial (max, sum, acc) triples are merged in a fixed order.
 *   - Rows listed in a prefill chunk (consecutive rows of one sequence at
 *     consecutive positions) run on a tensor-core tile path in the same launch.
 *
 * Conventions for every entry point:
 *   - All device memory (pools, q, k/v, out, tables, workspace, status) is
 *     allocated and owned by the caller.  The library owns only the small host
 *     pa_pool and pa_rope objects.  No call allocates device memory or synchronises.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default).
 *   - Any host thread may call, several at once on one pool where their workspaces
 *     and outputs are their own (pa_pool_set_head_scales comes before).
 *   - Host-side argument errors return a status at once, launch nothing, and
 *     set a thread-local message readable with pa_last_error().  No C++
 *     exception crosses the ABI.
 *   - Device-side errors (a sequence id, position or page id out of range, a
 *     bounded wait that ran out) are recorded in *status_dev (int32 in device
 *     memory, may be NULL): the first error code wins (compare-and-swap from
 *     PA_OK).  The caller zeroes it and reads it back when it wants to know.
 *     Rows hit by such an error get unspecified output (zeros for rows whose
 *     sequence id or position is invalid); the kernels never trap.
 *
 * Layouts (row-major, innermost last):
 *   k_pool, v_pool   [num_pages][Hkv][P][D]     kv_dtype, 16-byte aligned
 *   q, out           [n_rows][Hq][D]            q_dtype (out has q's dtype), 16-byte aligned
 *   k_new, v_new     [n_rows][Hkv][D]           in_dtype
 *   seq_ids, positions [n_rows]                 int32
 *   block_tables     [num_seqs][max_blocks_per_seq] int32, unused entries -1
 */
#ifndef PA_GB300_H
#define PA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = 1, /* host-side: a bad pointer, size, dtype or alignment */
    PA_ERR_UNSUPPORTED = 2, /* host-side: a valid but unimplemented shape (e.g. head_dim 96) */
    PA_ERR_OUT_OF_RANGE = 3, /* device-side: sequence id, position or page id out of range */
    PA_ERR_TIMEOUT = 4,     /* device-side: a bounded wait on a copy gave up */
    PA_ERR_CUDA = 5,        /* a CUDA runtime call failed (launch, attribute, driver entry point), or a kernel found its launch configuration inconsistent */
    PA_ERR_NO_PAGES = 6     /* an admission (host-side) or a pa_tables_grow (device-side) needs more free pages or rows than there are */
} pa_status;

typedef enum { PA_F32 = 0, PA_BF16 = 1, PA_FP8_E4M3 = 2, PA_INT4 = 3 } pa_dtype;

/* Pool geometry.  page_size in {16, 32, 64, 128, 256}; head_dim in {64, 128};
 * kv_dtype PA_F32, PA_BF16 or PA_FP8_E4M3 (PA_INT4: pa_pool_create_int4).  k_scale / v_scale are the fp8
 * per-tensor scales ("Engines for the card you have", section "One checkpoint,
 * many engines": an FP8 key/value cache, calibrated): a stored code c means
 * value(c) * scale, and appending x stores e4m3_satfinite_rne(x / scale).
 * They are ignored (taken as 1) for f32 and bf16 pools. */
typedef struct {
    int32_t num_pages;
    int32_t page_size;
    int32_t num_kv_heads;
    int32_t head_dim;
    pa_dtype kv_dtype;
    float k_scale;
    float v_scale;
} pa_pool_desc;

typedef struct pa_pool pa_pool; /* opaque host object */

/* Rows row_begin .. row_begin + n_rows - 1 of a step form one causal prefill
 * chunk: they must share one sequence id and have consecutive increasing
 * positions.  Host memory. */
typedef struct {
    int32_t row_begin;
    int32_t n_rows;
} pa_chunk;

/* Bytes of ONE of the two pool buffers (K or V) for this geometry: the memory
 * need, computed without allocating ("GPU inference engine engineering",
 * "Batching without running out of cache": the engine computes its memory need
 * without allocating).  Returns 0 for an invalid descriptor. */
size_t pa_pool_bytes(const pa_pool_desc *desc);

/* Wrap caller-owned device buffers k_pool and v_pool (each pa_pool_bytes(desc)
 * bytes, 16-byte aligned) in a host object.  Contents are not touched.
 * Errors: PA_ERR_INVALID_ARG (NULL pointer, misaligned buffer, non-positive
 * sizes, fp8 scale not finite and > 0), PA_ERR_UNSUPPORTED (page_size or
 * head_dim outside the supported sets). */
pa_status pa_pool_create(const pa_pool_desc *desc, void *k_pool, void *v_pool, pa_pool **out);

/* A pool of 4-bit codes.  Every token of a kv head has its own range, for K and for V:
 *     value(c) = step * c + low,  c = 0..15,  one binary32 multiply-add
 * and storing the head_dim elements x of one token and kv head takes, with x clamped to
 * +-65504 and every step one rounding to nearest even,
 *     low  = f16(min x)
 *     step = f16(max((max x - low) / 15, 0))      (binary32 subtraction and division)
 *     c    = clamp(rint((x - low) / step), 0, 15) (the same; 0 where step is 0)
 * A row that holds a NaN gets low = step = NaN and reads as NaN.
 *   desc      kv_dtype PA_INT4; k_scale and v_scale are ignored
 *   k_codes, v_codes    [num_pages][Hkv][P][D / 2] bytes, pa_pool_bytes(desc) each, 16-byte
 *                       aligned: element 2i in the low, 2i + 1 in the high four bits of byte i
 *   k_ranges, v_ranges  [num_pages][Hkv][P][2] f16 (step, low), pa_pool_range_bytes(desc) each,
 *                       16-byte aligned
 * Such a pool is taken by pa_append_kv, pa_rope_append, pa_read_kv, pa_attention, pa_step and
 * pa_attention_noalloc; pa_attention_mass, pa_evict_compact and pa_beam_reorder
 * refuse it with PA_ERR_UNSUPPORTED.  Errors as for pa_pool_create. */
size_t pa_pool_range_bytes(const pa_pool_desc *desc);
pa_status pa_pool_create_int4(const pa_pool_desc *desc, void *k_codes, void *v_codes, void *k_ranges, void *v_ranges,
                              pa_pool **out);

/* Free the host object (not the device buffers).  NULL is allowed. */
void pa_pool_destroy(pa_pool *pool);

/* One fp8 scale per kv head instead of the descriptor's per-tensor scales
 * ("Engines for the card you have", section "One checkpoint, many engines":
 * a calibrated FP8 key/value cache; the calibration's granularity is the
 * caller's).  k_scales, v_scales: HOST arrays of num_kv_heads floats, copied;
 * kv head h stores e4m3_satfinite_rne(x / k_scales[h]) and decodes
 * value(c) * k_scales[h] (likewise V).  Both NULL: back to the per-tensor
 * scales.  Errors: PA_ERR_INVALID_ARG (one array NULL, a pool that is not
 * fp8, a scale not finite and positive), PA_ERR_UNSUPPORTED (more than 64 kv
 * heads).  Takes effect for calls made after it. */
pa_status pa_pool_set_head_scales(pa_pool *pool, const float *k_scales, const float *v_scales);

/* K/V append ("GPU inference engine engineering", "Batching without running
 * out of cache"): for each row r, kv head h and element d,
 *     pool[block_tables[s][p / P]][h][p % P][d] = enc(new[r][h][d]),  s = seq_ids[r], p = positions[r]
 * for K and V.  enc is a copy (f32->f32, bf16->bf16, bf16->f32 widening),
 * fp32->bf16 round-to-nearest-even, or for fp8 pools e4m3 satfinite
 * round-to-nearest-even of (x / scale) with one IEEE binary32 division.
 * in_dtype is PA_F32 or PA_BF16.  One launch on `stream`.
 * Precondition: no two rows of one call write the same (page, slot); shared
 * prefix pages are never append targets.  n_rows == 0 is a no-op.
 * Device-side: a row with s outside [0, num_seqs), p outside
 * [0, max_blocks_per_seq * P) or a page id outside [0, num_pages) is skipped
 * and records PA_ERR_OUT_OF_RANGE. */
pa_status pa_append_kv(const pa_pool *pool, int32_t n_rows, const void *k_new, const void *v_new,
                       pa_dtype in_dtype, const int32_t *seq_ids, const int32_t *positions,
                       const int32_t *block_tables, int32_t num_seqs, int32_t max_blocks_per_seq,
                       int32_t *status_dev, void *stream);

/* The cached K and V of tokens, as dense rows: the counterpart of pa_append_kv, for every
 * pool type.  Row r, kv head h and element d:
 *     out[r][h][d] = value(pool[block_tables[s][p / P]][h][p % P][d]),  s = seq_ids[r], p = positions[r]
 * the value that the stored element stands for (fp8 and 4-bit pools: scaled), computed in
 * binary32 and rounded once to out_dtype, PA_F32 or PA_BF16.
 *   k_out, v_out  [n_rows][Hkv][D], 16-byte aligned; either may be NULL
 * A row may be listed more than once.  n_rows == 0 is a no-op.  One launch; graph-capturable.
 * Device-side: a row that pa_append_kv would skip gets zeros and records PA_ERR_OUT_OF_RANGE. */
pa_status pa_read_kv(const pa_pool *pool, int32_t n_rows, const int32_t *seq_ids, const int32_t *positions,
                     const int32_t *block_tables, int32_t num_seqs, int32_t max_blocks_per_seq, void *k_out,
                     void *v_out, pa_dtype out_dtype, int32_t *status_dev, void *stream);

/* Workspace bytes pa_attention needs for these rows, this block-table width
 * and these prefill chunks (the split-KV partial triples of decode rows and of
 * chunk tiles, their counters, and the decode rows' launch order when
 * pa_set_unit_order asks for one).  0 when nothing can be split or ordered.
 * Computed on the host from sizes only; for a bf16 pool it assumes the chunks
 * take the tensor-core tile path (bf16 queries), which never needs less. */
size_t pa_attention_workspace_bytes(const pa_pool *pool, int32_t n_rows, int32_t num_q_heads,
                                    int32_t max_blocks_per_seq, const pa_chunk *chunks, int32_t n_chunks);

/* Paged attention over a step's rows (see the top of this file).
 *   q_dtype      PA_F32 or PA_BF16; out has the same dtype, rounded to nearest even
 *   num_q_heads  a multiple of the pool's num_kv_heads, with Hq / Hkv in 1..8
 *   chunks       host array of n_chunks prefill chunks (may be NULL when n_chunks == 0);
 *                at most 16 chunks.  Rows not in a chunk are decode rows.
 *   softmax_scale <= 0 selects 1 / sqrt(head_dim)
 *   workspace    device memory of at least pa_attention_workspace_bytes(...), 256-byte
 *                aligned, ZERO-FILLED BEFORE ITS FIRST USE; every call leaves the split
 *                counters in it at zero again, so it is reused without clearing (except
 *                after a call that reported PA_ERR_TIMEOUT: clear it again); the other
 *                bytes are scratch that each call writes before it reads them.  Calls that
 *                share a workspace must not overlap on the GPU.  May be NULL when 0 bytes
 *                are needed.
 * Each row attends keys 0..positions[r] of its own sequence (its own token
 * included, so append the step's rows first).  A row's output bits depend only
 * on that row's inputs and on the rows of its own chunk, never on the other
 * rows of the call or the physical placement of its pages.
 * One launch on `stream` (split partials are merged inside it), preceded by
 * the one-CTA launch that orders the decode rows when pa_set_unit_order says
 * so; no allocation; graph-capturable.  Errors: PA_ERR_INVALID_ARG (NULL or misaligned pointer,
 * bad sizes, overlapping chunks, workspace too small), PA_ERR_UNSUPPORTED (a
 * group size or head_dim without a kernel), PA_ERR_CUDA (a failed launch). */
pa_status pa_attention(const pa_pool *pool, int32_t n_rows, const void *q, pa_dtype q_dtype,
                       int32_t num_q_heads, const int32_t *seq_ids, const int32_t *positions,
                       const int32_t *block_tables, int32_t num_seqs, int32_t max_blocks_per_seq,
                       const pa_chunk *chunks, int32_t n_chunks, float softmax_scale, void *out,
                       void *workspace, size_t workspace_bytes, int32_t *status_dev, void *stream);

/* One decode/prefill step: pa_append_kv of the step's rows, then pa_attention
 * over the same rows ("GPU inference engine engineering", section "Speed that
 * counts end to end": fewer launches per step; "Building an LLM runtime from
 * scratch on NVIDIA H100", section "Bug #2: Eager Decode and the CUDA Graph
 * Necessity": the launch gaps of eager decoding).
 *   - Rows outside every chunk (decode rows) append their own new K/V inside
 *     the attention launch: for each kv head, the attention unit that holds
 *     the row's position stores the row's converted key and value in the pool
 *     before it copies that page, so a step without chunks is ONE attention
 *     launch (behind the one-CTA order launch when pa_set_unit_order orders
 *     its rows; a step with chunks has its append launch write the order).
 *   - Chunk rows read one another's keys, so they are appended first by an
 *     append launch over the chunks' rows only; the attention kernel is its
 *     programmatic dependent (its CTAs start their lookups while the append
 *     runs; chunk tiles and chunk rows wait for it before reading the pools,
 *     decode rows do not wait).
 * Precondition (beyond those of pa_append_kv and pa_attention): a row outside
 * every chunk is the only row of its sequence in the step; a sequence that
 * contributes several rows to one step lists them as a chunk.
 *   k_new, v_new, kv_in_dtype: as pa_append_kv's k_new, v_new, in_dtype
 *   the other arguments: as pa_attention
 * Results (pool bytes and outputs) are bit-identical to pa_append_kv followed
 * by pa_attention on the same stream.  Every argument of both is checked
 * before anything is launched; errors as for those two calls.  Capturable in
 * a CUDA graph. */
pa_status pa_step(const pa_pool *pool, int32_t n_rows, const void *q, pa_dtype q_dtype, int32_t num_q_heads,
                  const void *k_new, const void *v_new, pa_dtype kv_in_dtype, const int32_t *seq_ids,
                  const int32_t *positions, const int32_t *block_tables, int32_t num_seqs, int32_t max_blocks_per_seq,
                  const pa_chunk *chunks, int32_t n_chunks, float softmax_scale, void *out, void *workspace,
                  size_t workspace_bytes, int32_t *status_dev, void *stream);

/* Rotary positions.  The first rotary_dim elements of a head are pairs; pair i of a row at
 * position p turns by the angle p * f_i and is scaled by `magnitude`:
 *     (a, b) -> magnitude * (a cos - b sin, a sin + b cos)
 * The elements behind rotary_dim stay.  PA_ROPE_HALF pairs elements i and i + rotary_dim / 2,
 * PA_ROPE_INTERLEAVED elements 2i and 2i + 1.  f_i = base^(-2i / rotary_dim), changed for
 * contexts longer than the `original_positions` that the weights know:
 *   PA_ROPE_LINEAR  f_i / factor
 *   PA_ROPE_BASE    with base * factor^(rotary_dim / (rotary_dim - 2)) in place of base
 *   PA_ROPE_RAMP    f_i / factor for pairs that turn fewer than `low` times over the original
 *                   positions, f_i for those that turn more than `high` times, and a linear ramp
 *                   over the pair index between (the indices at which a pair turns t times,
 *                   rotary_dim ln(original_positions / (2 pi t)) / (2 ln base), rounded outwards
 *                   and kept within 0 .. rotary_dim - 1); magnitude 0 stands for 0.1 ln(factor) + 1,
 *                   and for 1 where factor is 1 or less
 *   PA_ROPE_BANDS   the same ends, with t_i = original_positions f_i / (2 pi) turns and the weight
 *                   (t_i - low) / (high - low), clamped to 0..1, on f_i
 * f_i is a binary64 number, f_i / 2 pi is held as a 64-bit fraction of a turn (off by 2^-64 of a turn
 * for f_i up to 10^12), and p * f_i is taken modulo whole turns in integers: at any int32 position the
 * angle is off by 2^-33 of a turn at most before it is rounded.  Sines, cosines and products are FP32. */
typedef enum { PA_ROPE_HALF = 0, PA_ROPE_INTERLEAVED = 1 } pa_rope_layout;
typedef enum { PA_ROPE_NONE = 0, PA_ROPE_LINEAR = 1, PA_ROPE_BASE = 2, PA_ROPE_RAMP = 3, PA_ROPE_BANDS = 4 } pa_rope_scaling;
typedef struct {
    int32_t rotary_dim;          /* even, 2..128 */
    pa_rope_layout layout;
    double base;                 /* > 1 */
    pa_rope_scaling scaling;
    double factor;               /* > 0 (ignored by PA_ROPE_NONE) */
    int32_t original_positions;  /* > 0 (PA_ROPE_RAMP and PA_ROPE_BANDS) */
    double low, high;            /* 0 < low < high (the same two) */
    double magnitude;            /* 0: 1, or PA_ROPE_RAMP's; otherwise > 0 in binary32 */
} pa_rope_desc;
typedef struct pa_rope pa_rope; /* opaque host object, unchanged after its creation */

/* Errors: PA_ERR_INVALID_ARG (a number outside the ranges above, PA_ROPE_BASE with
 * rotary_dim 2, a base and factor whose frequencies are not finite).  pa_rope_frequencies copies f_i (rotary_dim / 2 numbers, radians per
 * position) and the magnitude, either of which may be NULL. */
pa_status pa_rope_create(const pa_rope_desc *desc, pa_rope **out);
void pa_rope_destroy(pa_rope *rope);
pa_status pa_rope_frequencies(const pa_rope *rope, double *frequencies, double *magnitude);

/* Rotate rows: out[r][h] = rotated x[r][h] at positions[r].
 *   x, out       [n_rows][n_heads][head_dim] of dtype (PA_F32 or PA_BF16), 16-byte aligned; a
 *                row's heads are contiguous, rows x_stride / out_stride elements apart (a
 *                multiple of 16 bytes, at least n_heads * head_dim).  out may be x (with its
 *                stride); otherwise they do not overlap
 *   head_dim     64 or 128, at least rotary_dim
 *   positions    any int32: a negative one turns back
 *   inverse      non-zero: the transposed map, magnitude * (a cos + b sin, b cos - a sin): the
 *                gradient of x from the gradient of out
 * One launch; graph-capturable. */
pa_status pa_rope_rows(const pa_rope *rope, int32_t n_rows, const void *x, int64_t x_stride, void *out,
                       int64_t out_stride, pa_dtype dtype, int32_t n_heads, int32_t head_dim, const int32_t *positions,
                       int32_t inverse, void *stream);

/* A step's projections taken in: queries rotated into q_out, keys rotated and stored in
 * their page slots, values stored, in one launch (in place of pa_rope_rows for q and k and
 * pa_append_kv).  Keys are stored from the FP32 result: an f32 or bf16 pool gets it rounded once, an
 * fp8 or 4-bit pool its code.  Values are stored as pa_append_kv stores them.
 *   q            [n_rows][num_q_heads][D], k, v [n_rows][Hkv][D] of dtype (PA_F32 or PA_BF16); rows
 *                q_stride, k_stride, v_stride elements apart as for pa_rope_rows (the three may be
 *                parts of one packed projection)
 *   q_out        [n_rows][num_q_heads][D], contiguous; may be q where q_stride is num_q_heads * D
 *   num_q_heads  any number >= 0 (0: q and q_out are not read)
 *   rope         its rotary_dim at most the pool's head_dim; NULL: nothing is rotated
 *   the other arguments and preconditions: as pa_append_kv
 * Device-side: a row with an invalid sequence, position or page stores nothing, leaves its
 * q_out as it was and records PA_ERR_OUT_OF_RANGE. */
pa_status pa_rope_append(const pa_pool *pool, const pa_rope *rope, int32_t n_rows, const void *q, int64_t q_stride,
                         int32_t num_q_heads, void *q_out, const void *k, int64_t k_stride, const void *v,
                         int64_t v_stride, pa_dtype dtype, const int32_t *seq_ids, const int32_t *positions,
                         const int32_t *block_tables, int32_t num_seqs, int32_t max_blocks_per_seq, int32_t *status_dev,
                         void *stream);

/* Causal attention over whole prompts, packed one behind the other, before or beside their
 * append: no cache is read.  For token i of sequence s (rows row_starts[s] .. row_starts[s + 1] - 1)
 * and query head g,
 *     out[i][g] = softmax_j(scale * q[i][g] . k[j][g / (Hq / Hkv)]) . v[j][g / (Hq / Hkv)],  j <= i of the same sequence
 *   q            [n_rows][Hq][D], k, v [n_rows][Hkv][D], PA_BF16, rows q_stride, k_stride, v_stride
 *                elements apart (multiples of 8, at least a row), heads contiguous, 16-byte aligned
 *   out          [n_rows][Hq][D] contiguous, PA_BF16; rows behind the last sequence (and any
 *                before the first) are left as they were.  It overlaps no input
 *   lse          f32 [n_rows][Hq] or NULL: the natural logarithm of the sum of a row's exponentials
 *                (to join the result with that over a cached prefix)
 *   row_starts   int32 [n_seqs + 1] in device memory, ascending, within 0..n_rows; a sequence may
 *                be empty
 *   num_q_heads  a multiple of num_kv_heads, any group size; head_dim 64 or 128
 *   softmax_scale <= 0 selects 1 / sqrt(head_dim)
 *   workspace    pa_prompt_workspace_bytes(...) bytes, 256-byte aligned; scratch that each call
 *                writes before it reads it.  Calls that share one must not overlap on the GPU
 * Scores, sums and accumulators are FP32; a softmax weight enters its product with V as bf16, off by
 * 2^-8 of itself at most.  (The chunk tiles of pa_attention and pa_step take a weight in two parts, 2^-16:
 * the same causal attention of a prompt is the more exact one there.  Against 64 bits the results of this
 * call are off by 2.0e-3 of their norm, of which the output's rounding alone makes 1.6e-3.)
 * What masked keys and values hold (infinities and NaN too, other sequences' rows too) has no
 * influence.  An infinite value that a row attends to gives that element +-infinity, or NaN.
 * A row's bits depend on its own sequence alone.  One launch for few units of work (tiles of 128
 * rows and two heads, or of 256 rows: at most one for each SM, of at most 32 sequences), else two, the
 * second a programmatic dependent of the first; graph-capturable.
 * Errors: PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED (dtype PA_F32, head_dim), PA_ERR_CUDA.
 * Device-side: row_starts that descend or leave 0..n_rows compute nothing and record
 * PA_ERR_OUT_OF_RANGE; a wait that ran out records PA_ERR_TIMEOUT and leaves out unspecified. */
size_t pa_prompt_workspace_bytes(int32_t n_rows, int32_t n_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                 int32_t head_dim);
pa_status pa_prompt_attention(int32_t n_rows, int32_t n_seqs, const void *q, int64_t q_stride, const void *k,
                              int64_t k_stride, const void *v, int64_t v_stride, pa_dtype dtype, int32_t num_q_heads,
                              int32_t num_kv_heads, int32_t head_dim, const int32_t *row_starts, float softmax_scale,
                              void *out, float *lse, void *workspace, size_t workspace_bytes, int32_t *status_dev,
                              void *stream);

/* Block tables and the rows of a step, made on the GPU (no host copy of the tables, so a
 * captured loop can run it).  The free pages of the pool are a stack in device memory:
 * free_pages[0 .. *free_count - 1], taken from its end.  Request i has lengths[i] tokens
 * cached in slot seq_ids[i] and takes new_tokens[i] more:
 *   - its table row gets pages for columns ceil(lengths / P) .. ceil((lengths + new) / P) - 1, in
 *     request order and then column order the next ones of the stack;
 *   - its rows are row_starts[i] .. row_starts[i + 1] - 1, at positions lengths[i] .. + new - 1:
 *     row_seqs, row_positions (the seq_ids and positions of the other calls) and row_slots, the
 *     token's place page * P + position % P in a pool's [num_pages * P] tokens of a kv head
 *     (-1: its page is not one of the pool).
 * Requests are served in order as long as pages and rows suffice: the first that does not fit and
 * every one behind it get nothing (row_starts stays where it is) and PA_ERR_NO_PAGES is recorded.
 * A request with an invalid slot, count, length or new length (together more than
 * max_blocks_per_seq * P), or a slot that is listed twice, takes nothing and PA_ERR_OUT_OF_RANGE is recorded.
 *   free_pages    int32 [num_pages]; an entry outside [0, num_pages) enters the table as -1
 *                 and records PA_ERR_OUT_OF_RANGE
 *   free_count    int32 [1], within 0..num_pages;  free_left  int32 [1], receives what remains (may
 *                 be free_count)
 *   row_starts, page_starts  int32 [n + 1], receive the exclusive sums of rows and of pages taken
 *   row_seqs, row_positions  int32 [max_rows], row_slots int64 [max_rows] (may be NULL); entries behind
 *                 row_starts[n] are left as they were.  All three may be NULL where max_rows is 0
 * The calls that take the rows take all of them as real: a step of a fixed n_rows (a captured
 * one) fills row_seqs with -1 before this call, in the step itself.  A row without a sequence stores
 * nothing, gets zeros (pa_rope_append: its q_out stays) and records PA_ERR_OUT_OF_RANGE in that call's
 * status word.  A request's tokens number row_starts[i + 1] - row_starts[i] from here on, not new_tokens[i].
 * Outputs overlap no input (but free_left).  The pages of a pool are handed out here or by
 * pa_pages_*, not by both; pages are not shared between slots.
 * num_seqs <= 2^19.  One launch for at most 2048 rows, else two, the second a programmatic
 * dependent of the first; no workspace; graph-capturable. */
pa_status pa_tables_grow(int32_t n, const int32_t *seq_ids, const int32_t *lengths, const int32_t *new_tokens,
                         const int32_t *free_pages, const int32_t *free_count, int32_t *free_left, int32_t num_pages,
                         int32_t page_size, int32_t *block_tables, int32_t num_seqs, int32_t max_blocks_per_seq,
                         int32_t *row_starts, int32_t *page_starts, int32_t max_rows, int32_t *row_seqs,
                         int32_t *row_positions, int64_t *row_slots, int32_t *status_dev, void *stream);

/* Give pages back to the stack: slot seq_ids[i] holds lengths[i] tokens and keeps the first
 * keep_tokens[i] (NULL: none).  The pages of columns ceil(keep / P) .. ceil(lengths / P) - 1 go on
 * the stack, the last request's last column first, so that a pa_tables_grow that asks for the
 * same again gets the same pages, and their table entries become -1.  A request with an invalid
 * slot or length, a slot that is listed twice, or an invalid page in those columns gives nothing back and
 * records PA_ERR_OUT_OF_RANGE; so does the whole call where the stack would hold more than
 * num_pages.  keep_tokens beyond lengths keeps everything.
 *   free_count    int32 [1], the stack's height, changed in place
 * num_seqs <= 2^19.  One launch of one CTA; no workspace; graph-capturable. */
pa_status pa_tables_release(int32_t n, const int32_t *seq_ids, const int32_t *lengths, const int32_t *keep_tokens,
                            int32_t *free_pages, int32_t *free_count, int32_t num_pages, int32_t page_size,
                            int32_t *block_tables, int32_t num_seqs, int32_t max_blocks_per_seq, int32_t *status_dev,
                            void *stream);

/* Attention weight per cached key: what eviction by accumulated attention
 * looks at.  For row r with sequence s and position p, kv head h and the G
 * query heads that read it,
 *     mass[s][h][t] += sum over those heads of softmax_t(scale * q[r][g] . K_s[t]),  t = 0..p
 * so one row adds G to the sum of its (sequence, kv head).  V is not read;
 * append the step's rows first.
 *   mass      f32 [num_seqs][Hkv][max_blocks_per_seq * page_size] in device memory,
 *             16-byte aligned; the caller zeroes a sequence's rows when it admits it.
 *             Entries past a row's position are not touched.
 *   chunks    as for pa_attention: the rows of one prompt (its last rows as an
 *             observation window, or all of them) are listed as a chunk.  Chunks
 *             with bf16 queries over a bf16 pool run on the tensor-core tile path.
 *   workspace device memory of at least pa_attention_mass_workspace_bytes(...) bytes,
 *             256-byte aligned (may be NULL when 0 are needed); scratch that each call
 *             writes before it reads it.  Calls that share one must not overlap on the GPU.
 *   the other arguments: as pa_attention
 * Precondition: a sequence has one row outside the chunks, or the rows of one
 * chunk, in a call (a step's rows satisfy it): its sums then have one writer
 * and the same bits in any batch.
 * Scores, sums and weights are FP32.  The products behind a score take bf16 and
 * e4m3 values as they are, f32 ones as three bf16 parts (24 bits, fewer below
 * 2^-110), an f32 query over an e4m3 pool as two f16 parts (22 bits).  A score of
 * -infinity (an infinite key) is a weight of zero; one of +infinity or NaN makes
 * its row's weights NaN for that kv head.
 * max_blocks_per_seq * page_size <= 2^30.  Errors as for pa_attention; a row with an
 * invalid sequence, position or page, or a chunk with such a row or whose rows
 * are not consecutive positions of one sequence, adds nothing and records
 * PA_ERR_OUT_OF_RANGE.  After PA_ERR_TIMEOUT (pa_set_wait_limit) the sums of the
 * call's chunks are unspecified.  Graph-capturable. */
size_t pa_attention_mass_workspace_bytes(const pa_pool *pool, int32_t n_rows, int32_t num_q_heads,
                                         int32_t max_blocks_per_seq, const pa_chunk *chunks, int32_t n_chunks);
pa_status pa_attention_mass(const pa_pool *pool, int32_t n_rows, const void *q, pa_dtype q_dtype,
                            int32_t num_q_heads, const int32_t *seq_ids, const int32_t *positions,
                            const int32_t *block_tables, int32_t num_seqs, int32_t max_blocks_per_seq,
                            const pa_chunk *chunks, int32_t n_chunks, float softmax_scale, float *mass,
                            void *workspace, size_t workspace_bytes, int32_t *status_dev, void *stream);

/* Which tokens of a cache stay.  For each listed sequence i (slot seq_ids[i],
 * lengths[i] tokens cached) and kv head h, keep[i][h][0..count) receives the
 * tokens to keep in ascending order, count = min(lengths[i], budget), and -1
 * behind them: the first keep_first and the last keep_last tokens, and of the
 * others those with the most mass, ties to the lowest token.  NaN counts as
 * less than any number.  A sequence no longer than the budget keeps
 * everything.  Each kv head keeps its own tokens (a page holds each head's
 * slots apart).
 *   seq_ids, lengths  int32 [n] in device memory
 *   mass              f32 [num_seqs][num_kv_heads][max_tokens], as pa_attention_mass
 *                     fills it with max_tokens = max_blocks_per_seq * page_size; weights that
 *                     another stream changes during the call leave a row's choice unspecified
 *   keep              int32 [n][num_kv_heads][budget], written whole
 *   kept_lengths      int32 [n], receives count (may be NULL; may be neither `lengths` nor `seq_ids`)
 * keep_first + keep_last <= budget; max_tokens <= 2^30.  One launch, no workspace; graph-capturable.
 * A row whose sequence is outside [0, num_seqs) or whose length is outside
 * [0, max_tokens] keeps nothing (all -1, count 0) and records
 * PA_ERR_OUT_OF_RANGE. */
pa_status pa_evict_select(int32_t n, const int32_t *seq_ids, const int32_t *lengths, const float *mass,
                          int32_t num_seqs, int32_t num_kv_heads, int32_t max_tokens, int32_t budget,
                          int32_t keep_first, int32_t keep_last, int32_t *keep, int32_t *kept_lengths,
                          int32_t *status_dev, void *stream);

/* Close the gaps: token keep[i][h][j] of slot seq_ids[i] becomes token j, for
 * K, V and (mass not NULL) the weights, j < count = min(lengths[i], budget).
 *   keep          int32 [n][Hkv][budget] in device memory, from pa_evict_select or a
 *                 policy of the caller's: strictly ascending tokens below lengths[i]
 *   dst_seq_ids   int32 [n]: slot dst_seq_ids[i] receives the tokens, through its own
 *                 row of the same block tables (a cache whose pages other sequences
 *                 share is compacted into a slot of its own).  NULL: in place.
 *   mass          f32 [num_seqs][Hkv][max_blocks_per_seq * page_size]; the destination's
 *                 entries count .. lengths[i] - 1 become zero.  NULL: left alone.
 * The caller's next token goes to position count; pages behind the last token
 * still to come can be given back (pa_pages_trim).  Slots behind count keep their
 * bytes.  A sequence compacted in place no longer holds its prompt (every kv head
 * keeps tokens of its own): it is no prefix parent for pa_pages_admit.
 * Precondition: no slot is listed twice, as a source of one row and a
 * destination of another either, and a page that receives tokens belongs to
 * that one sequence (in place: pages shared with another sequence would change
 * under it).  max_blocks_per_seq * page_size <= 2^30.  One launch, no workspace;
 * graph-capturable.
 * Device-side, with PA_ERR_OUT_OF_RANGE: a row with an invalid slot or length
 * moves nothing; a kept token out of range or out of order (not above the one
 * before it, or below its own place j, which no ascending list has) is not moved
 * and leaves a weight of zero, one whose page id is invalid is not moved; the
 * others move as listed. */
pa_status pa_evict_compact(const pa_pool *pool, int32_t n, const int32_t *seq_ids, const int32_t *dst_seq_ids,
                           const int32_t *lengths, const int32_t *keep, int32_t budget, const int32_t *block_tables,
                           int32_t num_seqs, int32_t max_blocks_per_seq, float *mass, int32_t *status_dev,
                           void *stream);

/* Beam search's choice.  For each group of `beams` hypotheses, the n_out best
 * continuations over beams x vocabulary by
 *     score[b][v] = scores[b] + logits[b][v] - log(sum_u exp(logits[b][u]))
 * best first; equal scores go to the lower beam, then the lower token.  A
 * finished beam has one continuation: itself, with its score unchanged and
 * token end_token.
 *   logits      f32 or bf16 [n_groups * beams] rows of `vocab`, row_stride elements
 *               apart (>= vocab), aligned to their element
 *   scores      f32 [n_groups * beams], the hypotheses' log-probabilities so far
 *   finished    int32 [n_groups * beams], non-zero: finished (may be NULL: none)
 *   parents, tokens   int32 [n_groups][n_out]: the beam (0..beams-1) a continuation
 *               extends, and its token;  out_scores  f32 [n_groups][n_out] (may be
 *               `scores` where n_out = beams; otherwise outputs overlap no input)
 * beams <= 32, n_out <= 64, vocab <= 2^20.  A logit of -infinity is no continuation; a beam
 * whose log-sum-exp is not finite (NaN or +infinity among its logits, or
 * nothing but -infinity) or whose score is not finite has none.  Where fewer
 * than n_out exist the rest is parent -1, token -1, score -infinity.
 * Sums of exponentials are FP32 within 128 KB of a row and FP64 across them;
 * scores are compared in FP64 and rounded once.  A group's results do not depend on the
 * other groups, nor on the alignment of its rows.
 *   workspace   device memory of at least pa_beam_workspace_bytes(...), 256-byte
 *               aligned; scratch that each call writes before it reads it.  Calls
 *               that share one must not overlap on the GPU.
 * Two launches, the second a programmatic dependent of the first; graph-capturable. */
size_t pa_beam_workspace_bytes(int32_t n_groups, int32_t beams, int32_t vocab, int32_t n_out);
pa_status pa_beam_select(int32_t n_groups, int32_t beams, int32_t vocab, const void *logits, pa_dtype logits_dtype,
                         int64_t row_stride, const float *scores, const int32_t *finished, int32_t end_token,
                         int32_t n_out, int32_t *parents, int32_t *tokens, float *out_scores, void *workspace,
                         size_t workspace_bytes, void *stream);

/* Give every beam its parent's cache.  Beam b of group i sits in slot
 * seq_ids[i][b] and becomes a copy of beam parents[i][b] (-1: of itself), all
 * beams at once.  The beams of a group hold lengths[i] tokens each:
 *   - whole pages (columns 0 .. lengths[i] / page_size - 1 of the block tables)
 *     are shared: the beam's table row takes the parent's page ids;
 *   - the unfinished page (column lengths[i] / page_size, when lengths[i] is not a
 *     multiple of page_size) stays each beam's own, and its slots in use are copied
 *     from the parent's;
 *   - later columns stay: they are the beam's own pages for the tokens to come.
 * A parent of 0 for every beam fans a prompt out, its unfinished page included.
 * Pages of beams that died stay referenced by the survivors' tables: the slots
 * of a group are released together, and none of them is trimmed (pa_pages_trim)
 * or compacted in place (pa_evict_compact) before.  The tables are changed on the
 * device alone: an allocator's host rows of these slots keep naming the pages that
 * each slot holds, and are not copied to the device again while the group lives.
 *   state      per-slot rows of the caller's (e.g. the attention weights), permuted the
 *              same way: state_row_bytes (a multiple of 4) for each of num_seqs slots,
 *              4-byte aligned.  NULL: none.
 * Precondition: a slot is listed once in a call, and an unfinished page belongs
 * to one beam.  beams <= 32, n_groups <= 65535.  One launch, no workspace;
 * graph-capturable.  A group with an invalid slot, parent, length or unfinished
 * page, a slot listed twice or an unfinished page shared by two of its beams is
 * left as it was and records PA_ERR_OUT_OF_RANGE. */
pa_status pa_beam_reorder(const pa_pool *pool, int32_t n_groups, int32_t beams, const int32_t *seq_ids,
                          const int32_t *parents, const int32_t *lengths, int32_t *block_tables, int32_t num_seqs,
                          int32_t max_blocks_per_seq, void *state, size_t state_row_bytes, int32_t *status_dev,
                          void *stream);

/* pa_attention without a workspace argument, for callers that cannot allocate
 * device memory: code handed only its input and output buffers by a host
 * runtime that owns and budgets all device memory (a plugin interface), or a
 * serving loop that forbids cudaMalloc after start-up because an allocation on
 * the hot path can synchronise the device or fail under memory pressure.  The
 * pages have no counterpart to this entry point; it exists for such callers.
 * The split-KV partials go to a scratch array of 32 MiB compiled into the
 * library's device image: every GPU that loads the library holds it until the
 * process exits, and this call allocates nothing (no cudaMalloc, no cudaFree,
 * no allocating library routine).  Arguments and results are those of
 * pa_attention, checked the same way first.  A call whose split-KV plan (the
 * bytes pa_attention would need for these rows, chunks, dtypes and split
 * length) exceeds 32 MiB is rejected with PA_ERR_UNSUPPORTED and a message in
 * pa_last_error(); the split length is read once per call.
 * The first call on a device that needs the array looks up its device
 * address (with that device current), and looks it up again when the
 * device's CUDA context has changed since (after cudaDeviceReset, for
 * instance); make that first call before any stream capture.  Every call
 * shares the one array and finds the previous call's contents in it; each
 * call clears its plan's split counters on `stream` first (every other byte
 * it reads, it has written).  Calls that can run at the same time on the GPU
 * (unordered streams) race on the array. */
pa_status pa_attention_noalloc(const pa_pool *pool, int32_t n_rows, const void *q, pa_dtype q_dtype,
                               int32_t num_q_heads, const int32_t *seq_ids, const int32_t *positions,
                               const int32_t *block_tables, int32_t num_seqs, int32_t max_blocks_per_seq,
                               const pa_chunk *chunks, int32_t n_chunks, float softmax_scale, void *out,
                               int32_t *status_dev, void *stream);

/* Split-KV chunk length in tokens: a row at position p is cut into
 * ceil((p + 1) / split) pieces merged in ascending order.  A process-wide
 * constant (default 4096), a multiple of 64 up to 4096, never derived from the batch.
 * These settings (split length, row groups, wait limit, injected stall) may be changed from
 * any thread; a call reads each of them once, when it starts, so one call never
 * mixes two values.  A workspace sized by pa_attention_workspace_bytes before a
 * change may be too small after it: the call then returns PA_ERR_INVALID_ARG.
 * Changing it changes output bits (within tolerance) for rows longer than it.
 * Returns PA_ERR_INVALID_ARG for a value that is not a positive multiple of 64. */
pa_status pa_set_split_tokens(int32_t tokens);
int32_t pa_get_split_tokens(void);

/* Row groups for the FP8 (E4M3) tensor-core decode units (head_dim 128, bf16
 * queries): with rows = 2, 4 or 8, one CTA takes that many consecutive decode
 * rows of the call for one kv head and split, and the leading pages that all
 * of its rows share (the same physical page ids, full 32-token stages, none a
 * row's last) are copied into shared memory once and read by every row
 * ("GPU inference engine engineering", section "The same bits in any batch":
 * a shared prompt prefix staged once for eight rows).  Rows share pages only
 * when the caller lists the rows of one prefix next to one another (a
 * scheduler that groups its batches by prefix, section "Caching measured on
 * the real prompt structure").  1 (the default) runs one row per CTA.  Output
 * bits never depend on it: each row's arithmetic is the same in both forms.
 * Other pools and query dtypes ignore it.  A process-wide setting, read once
 * per call like the split length.  Returns PA_ERR_INVALID_ARG for a value
 * other than 1, 2, 4 or 8. */
pa_status pa_set_row_groups(int32_t rows);
int32_t pa_get_row_groups(void);

/* Launch order of the decode rows.  A decode launch runs one CTA per (row,
 * split, kv head) and the GPU starts CTAs roughly in index order, so a long
 * row listed late starts in the last wave and runs on after the rest of the
 * launch has finished, reading HBM at a fraction of its rate (the pages
 * measure a kernel by its fraction of the bandwidth ceiling: "llm-rs ...",
 * section "2. Why decode is a memory problem"; they describe no launch
 * order).  PA_ORDER_LONGEST_FIRST runs the units of the rows with the most
 * keys per unit first: one CTA, of a launch of its own or of pa_step's append
 * launch, sorts the rows by the key
 * count of their longest unit into the workspace, and the attention launch
 * reads the order (its programmatic dependent).  PA_ORDER_CALL keeps the
 * call's order, one launch fewer.  PA_ORDER_AUTO (the default) orders a call
 * of at least 128 decode rows whose units can hold 1024 keys or more
 * (max_blocks_per_seq * page_size and the split length both at least 1024),
 * and keeps the order of other calls.  Output bits never depend on it: a
 * row's arithmetic is the same wherever it runs.  Row groups (rows > 1 above)
 * keep the call's order.  A process-wide setting, read once per call like the
 * split length; the workspace size depends on it.  Returns PA_ERR_INVALID_ARG
 * for another value. */
enum { PA_ORDER_AUTO = 0, PA_ORDER_CALL = 1, PA_ORDER_LONGEST_FIRST = 2 };
pa_status pa_set_unit_order(int32_t mode);
int32_t pa_get_unit_order(void);

/* Longest time, in microseconds, one device-side wait (for a copy or an MMA
 * to complete) may take before it gives up with PA_ERR_TIMEOUT; 0 restores
 * the default of one second.  A debugging knob for failure-path tests. */
void pa_set_wait_limit(uint32_t microseconds);

/* Failure-path testing without a GPU fault: with enable != 0, every attention
 * CTA additionally waits on a barrier that nothing ever completes, so that
 * wait runs out after the current wait limit; the call then reports
 * PA_ERR_TIMEOUT in *status_dev, its outputs are unspecified, and the kernel
 * still returns normally.  Set a small wait limit first (e.g. 1000 us).
 * Off by default; affects calls made while it is on. */
void pa_debug_stall_waits(int32_t enable);

const char *pa_status_string(pa_status status);

/* Detail text of the last host-side error on this thread ("" if none). */
const char *pa_last_error(void);

/* Number of CUDA kernels this library has launched in this process (all
 * entry points, all devices): lets a caller count the launches of a region. */
uint64_t pa_kernel_launches(void);

/* Library version string. */
const char *pa_version(void);

/* ---- Page allocator with admission (host side) ----------------------------
 * "GPU inference engine engineering", section "Batching without running out of
 * cache": a request is admitted only if the pages for its whole prompt AND its
 * whole answer can be reserved up front; a refusal gives a typed reason and
 * the numbers; the need is computable without allocating; a refused admission
 * takes nothing.  The allocator owns page ids of one pool (0 .. num_pages-1)
 * and the block-table rows of num_seqs sequence slots; it fills rows of a
 * caller-owned HOST array int32 [num_seqs][max_blocks_per_seq] (unused
 * entries -1), which the caller copies to the device for pa_append_kv /
 * pa_attention.  Prefix sharing: a sequence may share the whole pages of an
 * admitted parent's prompt prefix (reference counted; the page holding the
 * prefix's last partial tokens is the sequence's own).  Page ids are handed
 * out in a deterministic order (lowest first from a fresh allocator; a
 * release followed by the same admission returns the same pages).  Not
 * thread-safe: one scheduler thread owns an allocator. */
typedef struct pa_pages pa_pages; /* opaque host object */

typedef enum {
    PA_ADMIT_OK = 0,
    PA_ADMIT_NO_PAGES = 1,   /* fewer free pages than the admission needs (status PA_ERR_NO_PAGES) */
    PA_ADMIT_TOO_LONG = 2,   /* prompt + answer exceed max_blocks_per_seq * page_size tokens */
    PA_ADMIT_SEQ_IN_USE = 3, /* the sequence slot already holds pages */
    PA_ADMIT_BAD_ARG = 4     /* slot out of range, negative counts, prefix parent not admitted */
} pa_admit_reason;

typedef struct {
    pa_admit_reason reason;
    int32_t pages_needed;  /* new pages the admission takes (shared prefix pages excluded) */
    int32_t pages_free;    /* free pages when the admission was asked */
    int32_t pages_shared;  /* whole prefix pages shared with the parent */
    int32_t tokens;        /* prompt + answer tokens asked for */
    int32_t max_tokens;    /* tokens one block-table row can hold */
} pa_admit_info;

/* Pages a sequence of prompt_tokens + max_new_tokens tokens needs:
 * ceil((prompt + answer) / page_size).  No state; -1 on bad arguments.
 * Times pa_pool_bytes(desc) / desc.num_pages it is the device memory. */
int32_t pa_pages_needed(int32_t page_size, int32_t prompt_tokens, int32_t max_new_tokens);

/* An allocator over num_pages pages of page_size tokens for num_seqs sequence
 * slots of max_blocks_per_seq pages.  Errors: PA_ERR_INVALID_ARG. */
pa_status pa_pages_create(int32_t num_pages, int32_t page_size, int32_t num_seqs, int32_t max_blocks_per_seq,
                          pa_pages **out);
void pa_pages_destroy(pa_pages *pages);

/* Admit sequence slot seq for prompt_tokens + max_new_tokens tokens: reserve
 * every page up front and write the slot's row of block_tables (host, may be
 * NULL).  prefix_parent >= 0 shares the parent's first prefix_tokens / page_size
 * pages (prefix_tokens <= prompt_tokens), whose contents the caller vouches for
 * (not after pa_evict_compact in place on the parent); -1 for none.  *info (may be NULL)
 * receives the reason and the numbers.  Returns PA_OK; PA_ERR_NO_PAGES when
 * too few pages are free; PA_ERR_INVALID_ARG for the other reasons.  A refused
 * admission changes nothing. */
pa_status pa_pages_admit(pa_pages *pages, int32_t seq, int32_t prompt_tokens, int32_t max_new_tokens,
                         int32_t prefix_parent, int32_t prefix_tokens, int32_t *block_tables, pa_admit_info *info);

/* Release slot seq: drop its hold on each page (a page returns to the free
 * list when no sequence holds it) and reset its block_tables row to -1
 * (block_tables may be NULL).  PA_ERR_INVALID_ARG if the slot holds nothing. */
pa_status pa_pages_release(pa_pages *pages, int32_t seq, int32_t *block_tables);

/* Give back the pages of slot seq behind its first `tokens` tokens (after an
 * eviction): the slot keeps ceil(tokens / page_size) pages, the rest lose its
 * hold, and their block_tables entries become -1 (block_tables may be NULL).
 * A slot cannot be given pages again: `tokens` counts those that it will still
 * receive beside those that it holds.  Copy the slot's row to the device's block
 * tables before the next call that writes through them: the old row names pages that the next
 * admission may hand to another sequence, whose first append belongs behind the
 * eviction on the GPU.
 * A slot that holds no more pages than that is left as it is.
 * PA_ERR_INVALID_ARG if the slot holds nothing or tokens < 0. */
pa_status pa_pages_trim(pa_pages *pages, int32_t seq, int32_t tokens, int32_t *block_tables);

int32_t pa_pages_free_count(const pa_pages *pages);            /* -1 if pages is NULL */
int32_t pa_pages_refcount(const pa_pages *pages, int32_t page); /* sequences holding page; -1 if out of range */

#ifdef __cplusplus
}
#endif

#endif /* PA_GB300_H */
