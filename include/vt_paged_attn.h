/*
 * vt_paged_attn -- single-token decode attention over a paged KV cache,
 * hand-written for NVIDIA GB300 (sm_103a), and what a serving step runs around
 * it: rotary positions (vt_rope), the append of new keys and values to their
 * pages (vt_paged_kv_append), the attention of ragged batches of prompts and
 * chunks (vt_paged_attn_prefill).
 *
 * The operation (issue "ROCm gfx1200: PagedAttnOnline is 8.1x slower per call
 * than vLLM's paged-attention kernel", section "Where to look"; PR
 * "perf(cuda): head_dim-128 arm for the warp-split-KV decode kernel", commit
 * message): every sequence b has one query row per query head; query head i
 * attends, with a numerically stable softmax, over the keys and values of kv
 * head h = i / (num_q_heads / num_kv_heads) for the tokens of its context,
 * which live in 32-token pages named by the sequence's block-table row:
 *
 *   L = context_lens[b]; t0 = window > 0 ? max(0, L - window) : 0
 *   s_t = scale * <q[b][i], k_cache[bt[b][t/32]][t%32][h]>      t0 <= t < L
 *   out[b][i] = sum_t softmax(s)_t * v_cache[bt[b][t/32]][t%32][h]
 *
 * Storage is bf16 (or fp32); all arithmetic accumulates in fp32.  A context
 * of 0 tokens produces a zero row.
 *
 * Threading / ordering: every call only enqueues work on `stream` and
 * returns; it never synchronises the device.  The library keeps one
 * split-KV workspace per device (its own, or one the caller hands it with
 * vt_paged_attn_set_workspace); calls that share a device must be ordered on
 * the GPU (same stream, or streams ordered by events), otherwise they race on
 * that workspace.
 */
#ifndef VT_PAGED_ATTN_H
#define VT_PAGED_ATTN_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define VT_API __attribute__((visibility("default")))
#else
#define VT_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as CUDA's cudaStream_t / CUstream (NULL = legacy default stream). */
typedef struct CUstream_st* vt_stream_t;

typedef enum {
  VT_OK = 0,
  VT_ERR_INVALID_ARG = 1,   /* an argument is out of range, NULL or misaligned */
  VT_ERR_UNSUPPORTED = 2,   /* well-formed but not implemented (head_dim, block_size, group) */
  VT_ERR_CUDA = 3,          /* a CUDA runtime/driver call failed; see vt_last_cuda_error() */
  VT_ERR_OOM = 4,           /* the split workspace could not be allocated */
  VT_ERR_DEVICE_TIMEOUT = 5, /* a kernel gave up a bounded wait (see vt_paged_attn_device_status) */
  VT_ERR_SCRATCH_LIMIT = 6   /* the call needs more scratch than a fixed buffer holds (the static array
                                of vt_paged_attn_decode_noalloc, or the caller's vt_paged_attn_set_workspace) */
} vt_status;

/* Storage types.  VT_E4M3 is an FP8 K/V cache (with bf16 q and out) and is
 * taken only by the entry points whose names end in _fp8. */
typedef enum { VT_BF16 = 0, VT_F32 = 1, VT_E4M3 = 2 } vt_dtype;

/*
 * vt_paged_attn_decode -- the decode step.
 *
 * Device pointers (all caller-owned; nothing is retained after the call):
 *   out          [num_seqs][num_q_heads][head_dim] dtype, written.  16-byte aligned.
 *   q            [num_seqs][num_q_heads][head_dim] dtype.  16-byte aligned.
 *   k_cache      [num_blocks][block_size][num_kv_heads][head_dim] dtype ("NHD"
 *                pages, head_dim contiguous).  16-byte aligned.
 *   v_cache      same layout as k_cache.  16-byte aligned.
 *   block_tables [num_seqs][max_blocks_per_seq] int32 physical page ids; only
 *                the first ceil(L_b / block_size) entries of row b are read,
 *                and of those only pages that overlap the window.
 *   context_lens [num_seqs] int32, 0 <= L_b <= max_blocks_per_seq * block_size.
 * Sizes:
 *   num_seqs >= 0 (0 is a no-op), num_q_heads % num_kv_heads == 0,
 *   head_dim in {64, 128, 256} (and 512 for bf16 storage; the pages' widest
 *   arm), block_size == 32, scale finite (1/sqrt(head_dim)
 *   is usual), window <= 0 for full context else the number of most recent
 *   tokens attended (query token included).
 * Forced additions to the classic signature:
 *   max_blocks_per_seq  block-table row stride (entries) and per-row bound;
 *   num_blocks          pool size in pages: extent of the cache tensors, and
 *                       the bound every page id read is checked against;
 *   dtype               storage type of q, k_cache, v_cache and out.
 *
 * Invalid data found on the device never faults: a context length outside
 * [0, max_blocks_per_seq*block_size] or a page id outside [0, num_blocks)
 * turns that sequence's (or that kv head's) output rows into NaN.
 *
 * Returns VT_OK once the work is enqueued; argument errors return before any
 * launch; VT_ERR_CUDA reports a launch or runtime failure.
 */
VT_API vt_status vt_paged_attn_decode(void* out, const void* q, const void* k_cache,
                               const void* v_cache, const int32_t* block_tables,
                               const int32_t* context_lens, int num_seqs,
                               int num_q_heads, int num_kv_heads, int head_dim,
                               int block_size, float scale, int window,
                               vt_stream_t stream, int max_blocks_per_seq,
                               int num_blocks, vt_dtype dtype);

/*
 * vt_paged_attn_decode_noalloc -- the same decode, for callers that cannot
 * allocate device memory.  The pages this library follows have no
 * counterpart to it; it exists for the caller's sake.
 *
 * vt_paged_attn_decode allocates its split scratch (partial results and
 * arrival counters) itself, on first use and whenever a call needs more,
 * with cudaMallocAsync.  Some callers cannot let a library do that: serving
 * engines that hand nearly all device memory to their KV-cache pool up front,
 * programs whose device memory belongs to one external allocator or arena
 * that no library may bypass, and latency-critical decode loops where a
 * library may not enter the CUDA allocator after start-up.  This entry point
 * never allocates: it takes its scratch from one file-scope device array of
 * VT_NOALLOC_SCRATCH_BYTES (8 MiB), which every GPU that loads the library
 * holds until the process exits.  The caller still passes q, the caches, the
 * tables and out, exactly as for vt_paged_attn_decode; arguments, layouts,
 * results and error codes are the same.
 *
 * - The first call on each device looks up the array's device address with
 *   that device current (a one-time set-up); make that first call before
 *   any stream capture.
 * - A call whose scratch would exceed the array (very large batches, or a
 *   very large forced grid) returns VT_ERR_SCRATCH_LIMIT before launching
 *   anything; vt_last_cuda_error() names the sizes.
 * - All calls share the one array and it keeps the previous call's contents;
 *   each call clears the parts that must start at zero (status word and
 *   arrival counters) on its stream first.  Calls that overlap on the GPU
 *   (concurrent streams, or several host threads) race on the array and
 *   produce wrong results: order them.
 * - The status words of bounded waits live in the array; the next call
 *   clears them.  vt_paged_attn_device_status and
 *   vt_paged_attn_device_status_detail read them (with the other scratch
 *   areas of the device), so a give-up on this path is reported like any
 *   other.
 * - Nothing here calls cudaMalloc, cudaFree or any allocating routine.
 */
#define VT_NOALLOC_SCRATCH_BYTES (8u << 20)
VT_API vt_status vt_paged_attn_decode_noalloc(void* out, const void* q, const void* k_cache,
                                              const void* v_cache, const int32_t* block_tables,
                                              const int32_t* context_lens, int num_seqs,
                                              int num_q_heads, int num_kv_heads, int head_dim,
                                              int block_size, float scale, int window,
                                              vt_stream_t stream, int max_blocks_per_seq,
                                              int num_blocks, vt_dtype dtype);

/*
 * vt_paged_attn_decode_fp8 -- the decode step over an FP8 (E4M3) KV cache
 * with one dequantisation scale per kv head, for keys and for values.
 *
 * A storage extension beyond the pages, whose kernels keep the cache in
 * bf16: the path reads K/V bytes from HBM, so one-byte codes halve the bytes
 * of every step.  The operation is the decode of vt_paged_attn_decode with
 *   k_cache[page][slot][h][d] standing for  e4m3(code) * k_scale[h]
 *   v_cache[page][slot][h][d] standing for  e4m3(code) * v_scale[h]
 * where e4m3() is the OCP 8-bit floating-point value of the code (4 exponent
 * bits with bias 7, 3 mantissa bits, no infinities, S.1111.111 is NaN).
 *
 * Arguments as for vt_paged_attn_decode, except:
 *   q, out            bf16 [num_seqs][num_q_heads][head_dim].
 *   k_cache, v_cache  uint8 E4M3 codes, [num_blocks][block_size][num_kv_heads]
 *                     [head_dim] (NHD), 16-byte aligned.
 *   k_scale, v_scale  device float32 [num_kv_heads], 4-byte aligned; NULL is
 *                     VT_ERR_INVALID_ARG.
 *   head_dim          64, 128 or 256 (512 is VT_ERR_UNSUPPORTED).
 * Arithmetic: the K and V codes are widened exactly to f16 and enter f16
 * tensor-core MMAs with fp32 accumulation.  Each query row is scaled by a
 * power of two that puts its largest magnitude in [2^14, 2^15) and rounded
 * to f16, which holds the bf16 values exactly down to 2^-28 of that largest
 * (rows below 2^-100 in magnitude count as zero); the softmax weights enter
 * PV as f16 (11 significant bits).  k_scale folds into the score scale and
 * v_scale into the final normalisation.
 * Workspace, plan, status and errors are those of vt_paged_attn_decode.
 */
VT_API vt_status vt_paged_attn_decode_fp8(void* out, const void* q, const void* k_cache,
                                          const void* v_cache, const float* k_scale,
                                          const float* v_scale, const int32_t* block_tables,
                                          const int32_t* context_lens, int num_seqs,
                                          int num_q_heads, int num_kv_heads, int head_dim,
                                          int block_size, float scale, int window,
                                          vt_stream_t stream, int max_blocks_per_seq,
                                          int num_blocks);

/*
 * vt_paged_attn_decode_multi -- several new tokens per sequence over the same
 * paged cache: a chunk of a prefill, or draft tokens to verify.
 *
 * The pages list a head_dim-128 prefill as owed (PR "perf(rocm): head_dim=128
 * decode arm", section "Not claimed"); the reading taken: every sequence b
 * carries q_len new tokens whose keys and values are already in its pages as
 * the last q_len of its L = context_lens[b] tokens.  New token j
 * (0 <= j < q_len), at position L - q_len + j, attends with the decode's
 * arithmetic to the tokens t with
 *   t0_j <= t <= L - q_len + j,   t0_j = window > 0 ? max(0, L - q_len + 1 + j - window) : 0
 * (causal within the chunk), i.e. it is the single-token decode over a
 * context of L - q_len + 1 + j tokens.
 *
 * Arguments as for vt_paged_attn_decode, except:
 *   q, out   [num_seqs][q_len][num_q_heads][head_dim] (bf16 or fp32).
 *   q_len    >= 1 (1 is vt_paged_attn_decode); q_len * group <= 4096.
 * The query rows of one kv head (q_len tokens x its group of query heads)
 * share every page the head's kv tile is read for, so the cache is read once
 * per kv head for the whole chunk.  A sequence with L < q_len gets NaN rows
 * for all its new tokens.  dtype VT_E4M3 is VT_ERR_INVALID_ARG (an FP8 cache
 * takes vt_paged_attn_decode_multi_fp8).
 */
VT_API vt_status vt_paged_attn_decode_multi(void* out, const void* q, const void* k_cache,
                                            const void* v_cache, const int32_t* block_tables,
                                            const int32_t* context_lens, int num_seqs, int q_len,
                                            int num_q_heads, int num_kv_heads, int head_dim,
                                            int block_size, float scale, int window,
                                            vt_stream_t stream, int max_blocks_per_seq,
                                            int num_blocks, vt_dtype dtype);

/*
 * vt_paged_attn_decode_multi_fp8 -- several new tokens per sequence over an
 * FP8 (E4M3) cache: the operation of vt_paged_attn_decode_multi on the cache
 * that vt_paged_attn_decode_fp8 reads (codes times per-kv-head scales).
 *
 * Arguments as for vt_paged_attn_decode_fp8, plus q_len after num_seqs:
 *   q, out   bf16 [num_seqs][q_len][num_q_heads][head_dim].
 *   q_len    >= 1 (1 is vt_paged_attn_decode_fp8); q_len * group <= 4096.
 * Arithmetic as for vt_paged_attn_decode_fp8; causal limits, windows and the
 * NaN rows of L < q_len as for vt_paged_attn_decode_multi.  NULL scales are
 * VT_ERR_INVALID_ARG.
 */
VT_API vt_status vt_paged_attn_decode_multi_fp8(void* out, const void* q, const void* k_cache,
                                                const void* v_cache, const float* k_scale,
                                                const float* v_scale, const int32_t* block_tables,
                                                const int32_t* context_lens, int num_seqs, int q_len,
                                                int num_q_heads, int num_kv_heads, int head_dim,
                                                int block_size, float scale, int window,
                                                vt_stream_t stream, int max_blocks_per_seq,
                                                int num_blocks);

/*
 * Rotary positions.  Each rotated pair j (0 <= j < rot_dim / 2) of a head's
 * row is turned by the angle position * inv_freq[j] and scaled by amplitude:
 *   a' = amplitude * (a cos - b sin)      b' = amplitude * (b cos + a sin)
 * with (a, b) = (x[j], x[j + rot_dim / 2]) in the half layout
 * (interleaved = 0) and (x[2j], x[2j + 1]) in the interleaved one; elements
 * at and past rot_dim are copied.  The angle is reduced exactly (the turn per
 * token is held as a 64-bit fraction of a full turn), so far positions are as
 * accurate as near ones; sin, cos and the products are fp32, rounded once to
 * the storage type.  Any int32 position is taken; a negative one turns back,
 * so the call with -position is the gradient of the call with position.
 */

/* How vt_rope_frequencies stretches the frequencies for contexts longer than
 * the one a model was trained on.  Frequencies are f_j = base^(-2j / rot_dim)
 * radians per token before that. */
typedef enum {
  VT_ROPE_PLAIN = 0,  /* f_j as they are; amplitude 1 */
  VT_ROPE_LINEAR = 1, /* f_j / factor (position interpolation) */
  VT_ROPE_NTK = 2,    /* base * factor^(rot_dim / (rot_dim - 2)) instead of base: the slowest pair is stretched
                         by factor, the fastest not at all (rot_dim >= 4) */
  VT_ROPE_YARN = 3,   /* f_j / factor where a pair makes fewer than beta_slow turns in original_context tokens,
                         f_j where it makes more than beta_fast, a linear ramp over j between; amplitude
                         0.1 ln(factor) + 1 for factor > 1 */
  VT_ROPE_BANDED = 4  /* the same bounds, the ramp linear in the number of turns; amplitude 1 */
} vt_rope_kind;

typedef struct {
  vt_rope_kind kind;
  double factor;           /* > 0 (all kinds but plain) */
  double original_context; /* tokens, > 0 (YaRN, banded) */
  double beta_fast;        /* turns, > beta_slow (YaRN: 32 is usual; banded: 4) */
  double beta_slow;        /* turns, > 0 (usually 1) */
} vt_rope_stretch;

/*
 * vt_rope_frequencies -- fills host arrays for the calls below: inv_freq
 * [rot_dim / 2] (radians per token, fp64) and *amplitude.  rot_dim even and
 * positive, base finite and > 1; stretch NULL is VT_ROPE_PLAIN.  Host
 * arithmetic only; copy inv_freq to the device once.
 */
VT_API vt_status vt_rope_frequencies(double* inv_freq, float* amplitude, int rot_dim, double base,
                                     const vt_rope_stretch* stretch);

/*
 * vt_rope -- rotary positions on packed rows.
 *
 *   out, x      [num_tokens] rows of [num_heads][head_dim], consecutive rows out_stride and x_stride elements
 *               apart (>= num_heads * head_dim; e.g. the queries inside the rows of a fused projection).  Row
 *               starts 16-byte aligned.  out == x with equal strides rotates in place; other overlaps are not
 *               allowed.
 *   positions   [num_tokens] int32.
 *   inv_freq    [rot_dim / 2] device fp64, finite, 8-byte aligned.
 *   num_tokens >= 0 (0 is a no-op) and below 2^31 - 2^20, head_dim a multiple of 8 and at most 1024 (else
 *   VT_ERR_UNSUPPORTED), rot_dim
 *   even, 0 < rot_dim <= head_dim; interleaved 0 or 1; amplitude finite; dtype VT_BF16 or VT_F32.
 * Needs no workspace.
 */
VT_API vt_status vt_rope(void* out, const void* x, const int32_t* positions, const double* inv_freq, int num_tokens,
                         int num_heads, int head_dim, int rot_dim, int interleaved, float amplitude,
                         long long x_stride, long long out_stride, vt_stream_t stream, vt_dtype dtype);

/*
 * vt_paged_kv_append -- writes the keys and values of new tokens into the
 * paged cache and rotates keys and queries on the way.
 *
 * A ragged batch: the rows of all sequences are packed, sequence b owns rows
 * [q_starts[b], q_starts[b + 1]), which are the last
 * n_b = q_starts[b + 1] - q_starts[b] (0 or more) of its context_lens[b]
 * tokens.  Row j of sequence b goes to token t = context_lens[b] - n_b + j:
 *   k_cache[bt[b][t/32]][t%32][h] = rotated k row,   v_cache[...] = v row,
 *   q_out row = rotated q row,
 * at position t, or positions[row] where positions is not NULL.
 *
 *   k_cache, v_cache  as for vt_paged_attn_decode, written; no other slot is touched.
 *   q_out, q    [num_tokens][num_q_heads][head_dim], q_out contiguous, q rows q_stride elements apart; both NULL
 *               to append alone (num_q_heads is then not looked at).  q_out == q with q_stride == num_q_heads * head_dim rotates in place.
 *   k, v        [num_tokens] rows of [num_kv_heads][head_dim], k_stride and v_stride elements apart.
 *   q_starts    [num_seqs + 1] int32, q_starts[0] = 0, not decreasing, last entry <= num_tokens.  Rows behind the
 *               last sequence (a padded batch) are left as they were.
 *   inv_freq, rot_dim, interleaved, amplitude  as for vt_rope; rot_dim 0 (inv_freq NULL) rotates nothing.
 *   num_tokens  rows that q, k, v and q_out hold; num_seqs or num_tokens 0 is a no-op, 2^31 - 2^20 of either
 *               VT_ERR_UNSUPPORTED.
 *   head_dim    64, 128, 256 or 512 (fp32: up to 256).
 * All pointers 16-byte aligned (int32 arrays 4, inv_freq 8), strides multiples of 16 bytes.
 *
 * Invalid device data never faults: a sequence with a context outside [n_b, max_blocks_per_seq * 32] writes nothing
 * to the cache and gets NaN q_out rows; a token whose page id is outside [0, num_blocks) is not written; a sequence
 * whose q_starts are below 0, decrease or pass num_tokens has no rows (where they decrease, rows of the sequences
 * around them may be left as they were).  Two rows of one call that name the same slot leave one of the two there.  Needs no workspace.
 */
VT_API vt_status vt_paged_kv_append(void* k_cache, void* v_cache, void* q_out, const void* k, const void* v,
                                    const void* q, const int32_t* q_starts, const int32_t* block_tables,
                                    const int32_t* context_lens, const int32_t* positions, const double* inv_freq,
                                    int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                    int block_size, int rot_dim, int interleaved, float amplitude,
                                    long long q_stride, long long k_stride, long long v_stride, vt_stream_t stream,
                                    int max_blocks_per_seq, int num_blocks, vt_dtype dtype);

/*
 * vt_paged_kv_append_fp8 -- the append into an FP8 (E4M3) cache: q, k, v and
 * q_out bf16, a cached code is the E4M3 value nearest to row / k_scale[h]
 * (v_scale[h]; the quotient as fp32, two roundings at most), ties to even,
 * magnitudes past 448 held at 448, NaN kept.
 * head_dim 64, 128 or 256; k_scale, v_scale device float32 [num_kv_heads].
 */
VT_API vt_status vt_paged_kv_append_fp8(void* k_cache, void* v_cache, void* q_out, const void* k, const void* v,
                                        const void* q, const float* k_scale, const float* v_scale,
                                        const int32_t* q_starts, const int32_t* block_tables,
                                        const int32_t* context_lens, const int32_t* positions,
                                        const double* inv_freq, int num_seqs, int num_tokens, int num_q_heads,
                                        int num_kv_heads, int head_dim, int block_size, int rot_dim,
                                        int interleaved, float amplitude, long long q_stride, long long k_stride,
                                        long long v_stride, vt_stream_t stream, int max_blocks_per_seq,
                                        int num_blocks);

/*
 * vt_paged_attn_prefill -- attention of a ragged batch of chunks of new
 * tokens (whole prompts, chunks of prompts, draft tokens, single tokens
 * beside them) over the paged cache that already holds their keys and values.
 *
 * Rows are packed as for vt_paged_kv_append; row j of sequence b stands at
 * p = context_lens[b] - n_b + j and attends to the tokens
 *   t0 <= t <= p,   t0 = window > 0 ? max(0, p + 1 - window) : 0
 * which is the operation of vt_paged_attn_decode_multi with a chunk length of
 * its own for each sequence and no bound on it.
 *
 *   out, q      [num_tokens][num_q_heads][head_dim], not overlapping; out rows behind the last sequence are left as
 *               they were.
 *   q_starts, num_seqs, num_tokens  as for vt_paged_kv_append.
 *   num_q_heads / num_kv_heads at most 128, fp32 64 (else VT_ERR_UNSUPPORTED); the other arguments, layouts and
 *   limits as for vt_paged_attn_decode.
 * bf16 runs on the tensor cores: scores and sums in fp32, softmax weights rounded to bf16 before the product with
 * V (8 bits of each; vt_paged_attn_decode and vt_paged_attn_decode_multi keep 16, so the same rows are closer to the
 * exact value there).  fp32 runs on CUDA cores.
 *
 * The values of slots outside [0, context_lens[b]) of a sequence's pages are never used, whatever they hold.  A value
 * that is not finite reaches every row that sees its key, whatever its weight, and no other row: that column is then
 * the infinity, NaN where infinities of both signs or a NaN are seen (or where the infinity's weight is 0 in 32 bits).
 * The same call on the same data gives the same bits.
 * Invalid device data never faults: rows of a sequence with a context outside [n_b, max_blocks_per_seq * 32] are
 * NaN, and so are rows that attend to a page whose id is outside [0, num_blocks) (other rows of that sequence may be
 * too).  q_starts below 0, that decrease or pass num_tokens are read as sequences without rows.
 *
 * Workspace: as for vt_paged_attn_decode, but the library's own prefill scratch is apart from the decode's; it is
 * sized by the head_dim and the device, not by the batch, and a call that would have to allocate it inside a stream
 * capture returns VT_ERR_SCRATCH_LIMIT (make one call before capturing).  With vt_paged_attn_set_workspace the
 * caller's area is used instead, from its end, and must hold vt_paged_attn_prefill_workspace_bytes() beyond the
 * decodes' counters; once a prefill on it has been captured, a decode whose counters would reach what that prefill
 * uses returns VT_ERR_SCRATCH_LIMIT.
 * vt_paged_attn_set_override (min_units_per_cta in blocks of 128 keys) and vt_paged_attn_set_test_wait (withhold_tile
 * the key block of the CTA, fp32 has no waits) apply; vt_paged_attn_device_status reports.
 */
VT_API vt_status vt_paged_attn_prefill(void* out, const void* q, const void* k_cache, const void* v_cache,
                                       const int32_t* q_starts, const int32_t* block_tables,
                                       const int32_t* context_lens, int num_seqs, int num_tokens, int num_q_heads,
                                       int num_kv_heads, int head_dim, int block_size, float scale, int window,
                                       vt_stream_t stream, int max_blocks_per_seq, int num_blocks, vt_dtype dtype);

/*
 * vt_paged_attn_prefill_fp8 -- the same over an FP8 (E4M3) cache (bf16 q and
 * out; codes times per-kv-head scales, as for vt_paged_attn_decode_fp8);
 * head_dim 64, 128 or 256.
 * Arithmetic: each query row is scaled by a power of two that puts its largest
 * magnitude in [2^7, 2^8) and split into two E4M3 terms, which hold a bf16
 * value exactly down to 2^-9 of that largest and to 2^-17 of it absolutely
 * below (vt_paged_attn_decode_fp8's queries keep 2^-28); key codes enter the
 * products as they are.  Value codes are widened exactly to f16 and the weights
 * rounded to f16, as there.  Sums are fp32.
 */
VT_API vt_status vt_paged_attn_prefill_fp8(void* out, const void* q, const void* k_cache, const void* v_cache,
                                           const float* k_scale, const float* v_scale, const int32_t* q_starts,
                                           const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                                           int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                           int block_size, float scale, int window, vt_stream_t stream,
                                           int max_blocks_per_seq, int num_blocks);

/* Bytes of workspace a prefill call with this head_dim and cache type, causal or of trees, uses at most on the current
 * device (0: not taken). */
VT_API size_t vt_paged_attn_prefill_workspace_bytes(int head_dim, vt_dtype dtype);

/*
 * The operators below serve a step of speculative decoding on the paged cache:
 * page tables, the masks of trees of drafted tokens, the norm of query and key
 * heads in the append's pass, the trees' attention, and the accepted branch
 * moved to consecutive slots.
 */

/*
 * vt_paged_step_tables -- block tables, row starts, positions and slots of the
 * next step, on the device, from request lengths and a stack of free pages.
 *
 * A sequence of L = context_lens[b] tokens keeps k = keep_lens[b] of them (all
 * where keep_lens is NULL) and gets n = new_lens[b] new ones.  With
 * pg(x) = ceil(x / 32), in this order:
 *   pages pg(k) .. pg(L) - 1 of its block-table row go to the stack of free pages (of all sequences, before any
 *   page is taken);
 *   pages pg(k) .. pg(k + n) - 1 of its row are taken from it;
 *   context_lens[b] = k + n, and its n rows of the packed batch, from q_starts[b] on, get the positions k + j and the
 *   slots page * 32 + position % 32 (-1 where a page's id is outside [0, num_blocks)).
 * Pages are given back and taken in the order of the sequences and of their rows, and the first given back lies on
 * top: sequences that take as many pages as they give back keep theirs.  A finished sequence keeps 0 and gets 0.
 *
 * A sequence does not grow where k + n > max_blocks_per_seq * 32, and from the first other one on whose pages the
 * stack or whose rows num_tokens does not hold, none does: such sequences are left with k tokens and no rows.  One
 * whose lengths are none (L or k negative, k > L, L > max_blocks_per_seq * 32, n < 0) is left as it is, without rows.
 *
 * Rows lie as they were granted: behind a sequence that got fewer than it asked for, those of later ones begin
 * earlier than the lengths asked for say.  Tokens, parents or projections that the caller packed by those lengths
 * would then belong to other sequences, which no operator behind can notice: a caller that packs ahead asks only for
 * what fits, or looks at counters[1] or q_starts first.
 *
 *   block_tables  [num_seqs][max_blocks_per_seq] int32, in and out; entries behind a context are left as they were.
 *   context_lens  [num_seqs] int32, in and out.
 *   free_pages    [num_blocks] int32, in and out: a stack with room for every page of the pool, entry 0 at the bottom.
 *   counters      [2] int32: pages on the stack, in and out; sequences that asked for something they did not get, out.
 *   q_starts      [num_seqs + 1] int32, out.
 *   positions, slots  [num_tokens] int32, out, either may be NULL; entries behind the last row are left as they were.
 *   keep_lens, new_lens  [num_seqs] int32.
 *   num_seqs      0 to 16384 (else VT_ERR_UNSUPPORTED); num_tokens, num_blocks, max_blocks_per_seq as for
 *                 vt_paged_kv_append.
 * keep_lens may be context_lens; no other arrays may overlap.  All are 4-byte aligned.  One launch, no workspace.
 */
VT_API vt_status vt_paged_step_tables(int32_t* block_tables, int32_t* context_lens, int32_t* free_pages,
                                      int32_t* counters, int32_t* q_starts, int32_t* positions, int32_t* slots,
                                      const int32_t* keep_lens, const int32_t* new_lens, int num_seqs, int num_tokens,
                                      int block_size, vt_stream_t stream, int max_blocks_per_seq, int num_blocks);

/*
 * vt_tree_masks -- masks and positions of trees of drafted tokens.
 *
 * The rows of a sequence (packed as for vt_paged_kv_append, already counted in
 * context_lens) are a tree: parents[row] is the place within the sequence's
 * rows of the token that a row follows, less than its own, or -1 where it
 * follows the context (any other value is read as -1).  Bit i % 32 of word
 * i / 32 of a row's mask says that the row sees its sequence's i-th new token:
 * itself and those it follows.
 *
 *   masks      [num_tokens][mask_words] int32, out.
 *   positions  [num_tokens] int32, out, may be NULL: context_lens[b] - n_b + the number of tokens the row follows.
 *   parents    [num_tokens] int32.  The outputs overlap neither the inputs nor each other.
 *   mask_words 1 to 32 (else VT_ERR_UNSUPPORTED).
 * Rows of a sequence with more than 32 * mask_words rows, or with fewer context tokens than rows, and those behind
 * the last sequence are left as they were.  num_seqs or num_tokens 0 is a no-op.  Needs no workspace.
 */
VT_API vt_status vt_tree_masks(int32_t* masks, int32_t* positions, const int32_t* parents, const int32_t* q_starts,
                               const int32_t* context_lens, int num_seqs, int num_tokens, int mask_words,
                               vt_stream_t stream);

/*
 * vt_norm_rope -- the RMS norm of each head's row, then vt_rope's rotation:
 *   y = x / sqrt(mean(x^2) + eps) * weight,   out = y turned,
 * in fp32, rounded once.
 *
 *   weight      device fp32, 16-byte aligned: [head_dim], shared by the heads (weight_stride 0), or a row for each
 *               head, weight_stride elements apart (>= head_dim, a multiple of 4).
 *   rot_dim     0 (inv_freq NULL, positions not looked at) rotates nothing.
 *   eps         finite, >= 0.
 * The other arguments and limits as for vt_rope.
 */
VT_API vt_status vt_norm_rope(void* out, const void* x, const float* weight, const int32_t* positions,
                              const double* inv_freq, int num_tokens, int num_heads, int head_dim, int rot_dim,
                              int interleaved, float amplitude, float eps, long long x_stride, long long out_stride,
                              long long weight_stride, vt_stream_t stream, vt_dtype dtype);

/*
 * vt_paged_kv_norm_append, vt_paged_kv_norm_append_fp8 -- vt_paged_kv_append
 * and vt_paged_kv_append_fp8 of queries and keys that are normed first, as
 * vt_norm_rope norms them (values are not).  k_weight for the kv heads,
 * q_weight for the query heads (not looked at without q).
 */
VT_API vt_status vt_paged_kv_norm_append(void* k_cache, void* v_cache, void* q_out, const void* k, const void* v,
                                         const void* q, const float* k_weight, const float* q_weight,
                                         const int32_t* q_starts, const int32_t* block_tables,
                                         const int32_t* context_lens, const int32_t* positions,
                                         const double* inv_freq, int num_seqs, int num_tokens, int num_q_heads,
                                         int num_kv_heads, int head_dim, int block_size, int rot_dim,
                                         int interleaved, float amplitude, float eps, long long q_stride,
                                         long long k_stride, long long v_stride, long long q_weight_stride,
                                         long long k_weight_stride, vt_stream_t stream, int max_blocks_per_seq,
                                         int num_blocks, vt_dtype dtype);
VT_API vt_status vt_paged_kv_norm_append_fp8(void* k_cache, void* v_cache, void* q_out, const void* k,
                                             const void* v, const void* q, const float* k_weight,
                                             const float* q_weight, const float* k_scale, const float* v_scale,
                                             const int32_t* q_starts, const int32_t* block_tables,
                                             const int32_t* context_lens, const int32_t* positions,
                                             const double* inv_freq, int num_seqs, int num_tokens, int num_q_heads,
                                             int num_kv_heads, int head_dim, int block_size, int rot_dim,
                                             int interleaved, float amplitude, float eps, long long q_stride,
                                             long long k_stride, long long v_stride, long long q_weight_stride,
                                             long long k_weight_stride, vt_stream_t stream, int max_blocks_per_seq,
                                             int num_blocks);

/*
 * vt_paged_attn_prefill_tree, vt_paged_attn_prefill_tree_fp8 -- attention of
 * trees of drafted tokens over the paged cache, which already holds their keys
 * and values (vt_paged_attn_prefill's rows with masks of their own).
 *
 * A row of sequence b sees every token t < context_lens[b] - n_b, and new
 * token i where bit i % 32 of word i / 32 of its mask is set (bits from n_b on
 * are not looked at); with window > 0 the last `window` of those, in the
 * order of their slots.  So a chain of tokens with vt_tree_masks' masks is
 * vt_paged_attn_prefill.  Any masks are taken, not only trees'; a row that
 * sees nothing is 0.
 *
 *   masks       [num_tokens][mask_words] int32, 1 <= mask_words <= 32 (else VT_ERR_UNSUPPORTED).
 * Rows of a sequence with more than 32 * mask_words rows are NaN.  For given lengths a row depends, to the bit, on its
 * own sequence alone.  The other arguments, limits, arithmetic, invalid
 * device data and workspace (vt_paged_attn_prefill_workspace_bytes) as for vt_paged_attn_prefill and
 * vt_paged_attn_prefill_fp8.
 */
VT_API vt_status vt_paged_attn_prefill_tree(void* out, const void* q, const void* k_cache, const void* v_cache,
                                            const int32_t* masks, const int32_t* q_starts,
                                            const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                                            int num_tokens, int mask_words, int num_q_heads, int num_kv_heads,
                                            int head_dim, int block_size, float scale, int window,
                                            vt_stream_t stream, int max_blocks_per_seq, int num_blocks,
                                            vt_dtype dtype);
VT_API vt_status vt_paged_attn_prefill_tree_fp8(void* out, const void* q, const void* k_cache, const void* v_cache,
                                                const float* k_scale, const float* v_scale, const int32_t* masks,
                                                const int32_t* q_starts, const int32_t* block_tables,
                                                const int32_t* context_lens, int num_seqs, int num_tokens,
                                                int mask_words, int num_q_heads, int num_kv_heads, int head_dim,
                                                int block_size, float scale, int window, vt_stream_t stream,
                                                int max_blocks_per_seq, int num_blocks);

/*
 * vt_paged_kv_keep_path -- the accepted branch of each sequence's tree moved to
 * consecutive slots, in all layers.
 *
 * accepted[b] is the place within sequence b's rows of its last accepted token,
 * -1 for none (so is any other value outside its rows).  With i_0 < i_1 < ... the tokens that this row's mask names
 * (itself and those it follows), the keys and values of token
 * context_lens[b] - n_b + i_r go to the slot of token context_lens[b] - n_b + r, and
 *   kept_lens[b] = context_lens[b] - n_b + the number of those tokens.
 * No other slot is touched.  Positions are a matter of the rows: a branch's tokens have the positions of their new
 * places already.
 *
 *   k_cache, v_cache  [num_layers] pools as for vt_paged_attn_decode, k_layer_stride and v_layer_stride elements
 *               apart (>= a pool, multiples of 16 bytes; not looked at for one layer); 16-byte aligned, a slot's row
 *               a multiple of 16 bytes.
 *   kept_lens   [num_seqs] int32, out, none of the inputs.
 *   masks       [num_tokens][mask_words] int32, 1 <= mask_words <= 32.
 * A sequence with no rows, more than 32 * mask_words rows, or a context outside [n_b, max_blocks_per_seq * 32] keeps
 * its context_lens[b], and nothing of it moves; nor does a token from or to a page whose id is outside
 * [0, num_blocks).  num_seqs 0 is a no-op.  Needs no workspace.
 */
VT_API vt_status vt_paged_kv_keep_path(void* k_cache, void* v_cache, int32_t* kept_lens, const int32_t* accepted,
                                       const int32_t* masks, const int32_t* q_starts, const int32_t* block_tables,
                                       const int32_t* context_lens, int num_seqs, int num_tokens, int mask_words,
                                       int num_layers, int num_kv_heads, int head_dim, int block_size,
                                       long long k_layer_stride, long long v_layer_stride, vt_stream_t stream,
                                       int max_blocks_per_seq, int num_blocks, vt_dtype dtype);

/*
 * vt_call -- any of the speculative step's operators above, its arguments in
 * 8-byte slots: for callers whose foreign-function interface costs by the
 * argument.
 *
 *   args  args[0].i a vt_op, args[1].i the number of arguments that follow, then the operator's arguments in their
 *         order: pointers, integers and vt_dtype as i, float as f.
 * Returns what the operator returns; VT_ERR_INVALID_ARG where the operator is none, the number is not its number of
 * arguments, or an int's value is outside an int's range.
 */
typedef enum vt_op {
  VT_OP_STEP_TABLES = 1,
  VT_OP_TREE_MASKS = 2,
  VT_OP_NORM_ROPE = 3,
  VT_OP_NORM_APPEND = 4,
  VT_OP_NORM_APPEND_FP8 = 5,
  VT_OP_PREFILL_TREE = 6,
  VT_OP_PREFILL_TREE_FP8 = 7,
  VT_OP_KEEP_PATH = 8,
} vt_op;
typedef union vt_arg {
  long long i;
  double f;
} vt_arg;
VT_API vt_status vt_call(const vt_arg* args);

/* What the last successful decode or prefill call on this host thread
 * launched (a prefill: group_tile is the query rows of a work item, subgroups
 * 1, min_units_per_cta in 128-key blocks, q_len 0). */
typedef struct {
  int grid_ctas;          /* CTAs launched (persistent, balanced split of the work) */
  int ctas_per_sm;        /* resident CTAs per SM for this kernel variant */
  int num_sms;            /* SMs of the device */
  int consumer_warps;     /* compute warps per CTA (plus one TMA producer warp) */
  int tensor_cores;       /* 1: QK^T and PV on tensor cores (bf16, fp8), 0: CUDA cores (fp32) */
  int stages;             /* K/V page tiles in flight per CTA */
  int group_tile;         /* query heads computed per kv head and CTA (padded) */
  int subgroups;          /* ceil(group / group_tile) */
  int min_units_per_cta;  /* lower bound on work units per CTA (page tiles plus item weights) */
  int head_dim;
  int dtype;              /* vt_dtype of the K/V cache */
  size_t smem_bytes;      /* dynamic shared memory per CTA */
  size_t workspace_bytes; /* split-KV workspace used (partials + arrival counters) */
  int launch_overlap;     /* 1: launched as a programmatic dependent (vt_paged_attn_set_overlap) */
  int segment_cost;       /* partition weight of a segment boundary, in tiles (vt_paged_attn_set_segment_cost) */
  int scratch_source;     /* split scratch used: 0 library-owned, 1 the caller's (vt_paged_attn_set_workspace),
                             2 the static array (vt_paged_attn_decode_noalloc) */
  int q_len;              /* new tokens per sequence (1 except for vt_paged_attn_decode_multi) */
} vt_plan;

VT_API vt_status vt_paged_attn_last_plan(vt_plan* plan);

/*
 * Test / benchmark override of the launch plan for this host thread, read on
 * every call.  grid_ctas > 0 forces the number of CTAs (so tests can force
 * every sequence to be split, or never split); min_units_per_cta > 0 replaces
 * the default lower bound on work per CTA.  0 restores the automatic choice.
 */
VT_API vt_status vt_paged_attn_set_override(int grid_ctas, int min_units_per_cta);

/*
 * Launch overlap for this host thread, read on every call (default 0).  Not
 * an operation of the pages: a launch choice of this library.
 *
 * enabled = 1 launches each decode as a programmatic dependent of the kernel
 * before it on the same stream (CUDA programmatic dependent launch; it also
 * applies inside stream capture).  The decode's CTAs may then start while
 * that kernel finishes: they read context_lens and block_tables and plan the
 * split at once, and wait for it to complete before they read q, k_cache or
 * v_cache, or touch out and the workspace.  The decode itself lets the next
 * kernel start the same way.  Back-to-back decode steps (CUDA graphs of
 * layers or steps) overlap one call's start-up with the previous call's
 * tail.
 *
 * Contract: with enabled = 1, the kernel launched immediately before the
 * decode on its stream must not write context_lens or block_tables (step
 * metadata usually comes from host copies, which do not overlap).  Results
 * are identical either way.  Returns VT_ERR_INVALID_ARG unless enabled is 0
 * or 1.
 */
VT_API vt_status vt_paged_attn_set_overlap(int enabled);

/*
 * Partition weight of a segment boundary for this host thread, read on every
 * call.  Not an operation of the pages: a scheduling choice of this library.
 *
 * The kernel splits the (sequence, kv head, page) tiles evenly over its CTAs.
 * Every (sequence, kv head) a CTA starts costs it time beyond its pages (an
 * epilogue, a new query tile, a block-table row), so each one also weighs
 * `tiles` tiles in the split: CTAs whose share crosses many short sequences
 * get fewer pages.  The weight applies when the batch gives every CTA at
 * least 4 pages (below that the split is latency-bound and weights only add
 * partial results).  tiles < 0 restores the default: 2 for bf16 and fp32
 * K/V, 6 for an FP8 cache or several new tokens per sequence (their tiles
 * take less time per segment boundary); 0 balances pages alone.  Results are the same within rounding (split points move, and with
 * them the order of the log-sum-exp merge).  Returns VT_ERR_INVALID_ARG for
 * tiles > 64.
 */
VT_API vt_status vt_paged_attn_set_segment_cost(int tiles);

/*
 * Reads and clears the device status word that kernels set when a bounded
 * wait gives up (bit 0: page tile never arrived, bit 1: stage never released,
 * bit 2: consumer-warp rendezvous, bit 3: drain of copies in flight, bit 5:
 * partials staged for a split-KV combine) or a
 * self-check fails (bit 4: a CTA's tile walk did not match its share).
 * Synchronises `stream` first.  *status is 0 when all is well; the call
 * returns VT_ERR_DEVICE_TIMEOUT if it was not.  Clearing also resets the
 * split workspace's arrival counters.
 */
VT_API vt_status vt_paged_attn_device_status(vt_stream_t stream, unsigned* status);

/*
 * Copies the first n_words (<= 8) words of the device status area without
 * clearing them: [0] status bits as above; [1] 1 + index of the CTA whose
 * wait gave up first (0: none); [2] its status bit | (thread index << 8);
 * [3] shared-memory address of the barrier it waited on; [4] the phase
 * parity it waited for.  Synchronises `stream` first.
 */
VT_API vt_status vt_paged_attn_device_status_detail(vt_stream_t stream, unsigned* words, int n_words);

/*
 * vt_paged_attn_set_workspace -- hand the library a caller-owned split-KV
 * workspace for the current device (the boundary's optional workspace; the
 * operation itself is unchanged).
 *
 * vt_paged_attn_decode needs device scratch for split-KV partial results and
 * arrival counters.  By default the library allocates it lazily with
 * cudaMallocAsync on the call's stream and grows it when a call needs more.
 * After this call, decodes on the current device use [dev_ptr, dev_ptr +
 * bytes) instead and never allocate:
 *   dev_ptr  device memory, 256-byte aligned, owned by the caller; it must
 *            stay allocated and be touched by nothing else while it is set.
 *            NULL returns the device to the library-owned workspace.
 *   bytes    >= VT_MIN_WORKSPACE_BYTES.  The arrival counters must stay
 *            zeroed between calls, so their region only grows: a call needs
 *            256 bytes, plus the largest counter region any call on this
 *            workspace used, plus its own partial records.  For one model
 *            shape (heads, head_dim, dtype) the partials do not depend on the
 *            batch, so vt_paged_attn_workspace_bytes() of the largest
 *            num_seqs in use is enough for every call; for several shapes,
 *            the sum of their largest needs is.
 *   stream   the first 256 bytes (status words) are zeroed on it; later
 *            calls zero newly used counter space on their own streams.
 * The call begins anew, with the same area too: graphs captured on it before
 * are not replayed after it.
 * A decode that needs more than `bytes` returns VT_ERR_SCRATCH_LIMIT before
 * launching anything, and so does one whose counters would reach what a
 * captured vt_paged_attn_prefill uses at the area's end.  Calls that share the workspace must be ordered on
 * the GPU.  vt_paged_attn_device_status reads its status words.
 * Returns VT_ERR_INVALID_ARG for a misaligned pointer or a too-small size.
 */
#define VT_MIN_WORKSPACE_BYTES 4096u
VT_API vt_status vt_paged_attn_set_workspace(void* dev_ptr, size_t bytes, vt_stream_t stream);

/*
 * Test hook for the failure path of bounded waits (this host thread, read on
 * every call; not an operation of the pages).  Every wait on an mbarrier in
 * the kernel gives up after a limit of about one second of SM clock cycles,
 * sets a status bit and lets the CTA exit; this hook shortens the limit to
 * wait_limit_cycles (<= 0: the default) and, when withhold_tile >= 0, makes
 * CTA withhold_cta stop feeding its consumers before its withhold_tile-th
 * ring stage (counting from 0; stages that only close a segment count too).
 * The consumers' wait for that stage then runs out, the kernel returns
 * without faulting, and vt_paged_attn_device_status reports
 * VT_ERR_DEVICE_TIMEOUT (bit 0); the output of that call is incomplete.
 * vt_paged_attn_set_test_wait(0, -1, -1) restores normal operation.
 * Returns VT_ERR_INVALID_ARG when withhold_tile >= 0 and withhold_cta < 0.
 */
VT_API vt_status vt_paged_attn_set_test_wait(long long wait_limit_cycles, int withhold_cta, int withhold_tile);

/* Bytes of split-KV workspace a call with these sizes uses on the current device. */
VT_API size_t vt_paged_attn_workspace_bytes(int num_seqs, int num_q_heads,
                                     int num_kv_heads, int head_dim,
                                     vt_dtype dtype);

/* Frees the library's per-device workspaces.  No call may be in flight. */
VT_API void vt_paged_attn_release(void);

VT_API const char* vt_status_string(vt_status status);

/* Text of the last CUDA error seen by this host thread ("" if none). */
VT_API const char* vt_last_cuda_error(void);

/* Library version, major * 10000 + minor * 100 + patch. */
VT_API int vt_paged_attn_version(void);

#ifdef __cplusplus
} /* extern "C" */
#endif

#endif /* VT_PAGED_ATTN_H */
