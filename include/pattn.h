/*
 * pattn.h -- C ABI of the GB300 (sm_103a) paged variable-length attention
 * library, libpattn.so.
 *
 * One call computes exact softmax attention for a batch of requests that
 * mixes prefills, chunked prefills and single-token decodes, over a paged KV
 * cache.  The operation is defined on these pages:
 *   - "[vLLM] FlashAttention", FlashAttentionBackend.get_kv_cache_shape:
 *     the cache is (2, num_blocks, block_size, num_kv_heads, head_size), index
 *     0 of the first dimension is K and 1 is V, and block_size must be a
 *     multiple of 16;
 *   - same page, FlashAttentionImpl.__init__: num_queries_per_kv =
 *     num_heads / num_kv_heads query heads share one KV head (GQA);
 *   - same page, FlashAttentionMetadata: query_start_loc, seq_lens,
 *     block_table, max_query_len, max_seq_len let one call serve requests of
 *     different lengths;
 *   - "[vLLM] other attention backends", TritonAttentionMetadata:
 *     seq_len = context_len + query_len, so query row i of a request sits at
 *     position context_len + i;
 *   - "RBLN Attention modes", overview / Full Attention / SWA: scores over the
 *     valid tokens, softmax, product with V; causal masking; a sliding window;
 *     per-partition results merged with online softmax;
 *   - "[vLLM] FlashAttention", "why this design" item 4: tiled online softmax
 *     is exact attention, not an approximation.
 *
 * For request r: q_len = query_start_loc[r+1] - query_start_loc[r],
 * s = seq_lens[r], ctx = s - q_len.  Row i (position p = ctx + i) of head h
 * reads KV head g = h / (num_heads / num_kv_heads).  Key k < s lives in
 * physical block block_table[r * max_blocks_per_seq + k / block_size], slot
 * k % block_size.  Key k is visible iff (causal == 0 or k <= p) and
 * (window <= 0 or p - k < window).  out = softmax(scale * q . K^T over the
 * visible keys) . V.  A request with q_len == 1 is a decode (the page
 * "[vLLM] Lightning & Linear Attention", prefill/decode split with
 * threshold 1); any other q_len > 0 is a prefill; q_len == 0 produces nothing.
 *
 * Conventions for every entry point
 *   - Device pointers are marked [device]; everything else is host memory.
 *   - The caller owns every buffer.  The library allocates no memory, keeps
 *     no state between calls and may be called from several host threads.
 *   - Work is enqueued on ext->stream and the call returns without waiting.
 *   - Errors are returned, never thrown, and no call aborts the process.
 */
#ifndef PATTN_H
#define PATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PATTN_OK = 0,
  PATTN_ERR_INVALID_ARGUMENT = 1,   /* NULL pointer, bad size, bad scale     */
  PATTN_ERR_UNSUPPORTED = 2,        /* valid but not built (head_size, ...)  */
  PATTN_ERR_WORKSPACE_TOO_SMALL = 3,
  PATTN_ERR_CUDA = 4,               /* a CUDA runtime call failed            */
  PATTN_ERR_BAD_METADATA = 5,       /* device-detected: see read_device_status */
  PATTN_ERR_DEVICE_TIMEOUT = 6      /* device-detected: a bounded wait expired */
} pattn_status_t;

typedef enum {
  PATTN_KV_BF16 = 0,      /* K and V stored as bf16                          */
  PATTN_KV_FP8_E4M3 = 1,  /* K and V stored as e4m3 bytes, one fp32 scale each */
  PATTN_KV_F16 = 2,       /* K and V stored as f16; q and out are f16 too (the
                             FlashAttention backend supports float16 and
                             bfloat16 models)                                 */
  PATTN_KV_FP8_E4M3_ROW = 3 /* K and V stored as e4m3 bytes with one fp32 scale
                             per (token, KV head) row of K and of V, in a
                             buffer of their own (see PATTN_ROW_SCALE_MIN)    */
} pattn_kv_dtype_t;

/*
 * The scales of a PATTN_KV_FP8_E4M3_ROW cache: fp32 [num_blocks][block_size / 16]
 * [num_kv_heads][2][16], on the device, 16-B aligned.  Slot i of block b stands
 * for code * scale with scale = row_scales[b][i / 16][head][0 for K, 1 for V]
 * [i % 16].  (So the scales that go with 16 slots of one head are one 128-byte
 * line, and those of neighbouring heads follow it.)  Scales are within
 * [PATTN_ROW_SCALE_MIN, PATTN_ROW_SCALE_MAX] = [2^-60, 2^60]; the writers below
 * keep to it.
 */
#define PATTN_ROW_SCALE_MIN 8.673617379884035e-19f
#define PATTN_ROW_SCALE_MAX 1.152921504606847e+18f

/*
 * Host-side sizes and resources of one call.  Everything a device-pointer API
 * cannot learn without a device-to-host copy is passed here, so no call ever
 * synchronises.  The FlashAttentionMetadata fields (num_actual_tokens,
 * max_query_len, max_seq_len) have the same meaning.
 */
typedef struct {
  size_t struct_size;     /* sizeof(pattn_ext_t)                              */
  int num_seqs;           /* B: requests in the batch                         */
  int num_tokens;         /* T: rows of q and out (>= query_start_loc[B])     */
  int max_blocks_per_seq; /* row stride of block_table                        */
  int num_blocks;         /* physical blocks in kv_cache                      */
  int max_query_len;      /* >= every q_len in the batch                      */
  int max_seq_len;        /* >= every seq_len in the batch                    */
  int num_splits;         /* decode KV partitions: 0 = library chooses,
                             1..PATTN_MAX_SPLITS forces the count             */
  void* workspace;        /* [device] scratch of >= workspace_bytes, 256-B aligned */
  size_t workspace_bytes;
  void* stream;           /* cudaStream_t; NULL = the legacy default stream   */
  void* const* timing_events; /* optional host array of 8 cudaEvent_t, or NULL.
                             If set, events [2k] and [2k+1] are recorded on
                             stream right before and after phase k: 0 plan,
                             1 prefill, 2 decode, 3 combine (a phase that does
                             not run records both back to back).  For
                             profiling; the caller owns the events.          */
  const float* sinks;     /* [device] fp32 [num_heads] attention-sink logits, or
                             NULL for none.  Head h's sink joins the softmax
                             normaliser as a term with no value:
                               out = sum_k e^{s_k} V_k / (e^{sinks[h]} + sum_k e^{s_k}),
                             s_k = scale * q . k (the sink is not scaled).  A
                             sink of -inf is no sink; values must be finite or
                             -inf.  The pages ("RBLN Attention modes", Full
                             Attention: flash attention serves layers with
                             attention sinks) give no formula; this is the
                             reading taken.  A caller built against the
                             header without this field passes the smaller
                             struct_size and gets no sinks.                  */
  int head_size_v;        /* 0: K and V share head_size and the cache is
                             [2, num_blocks, block_size, num_kv_heads, head_size].
                             > 0: the DiffKV layout ("[vLLM] other attention
                             backends", FlashAttention DiffKV: V has its own
                             head size and the cache is asymmetric; the page
                             gives no shape, this is the reading taken): the
                             cache is [num_blocks, block_size, num_kv_heads,
                             head_size + head_size_v], each row the token's K
                             then its V, and out is [num_tokens, num_heads,
                             head_size_v].  head_size and head_size_v are then
                             multiples of 32 up to 256, the cache is bf16 or
                             f16 (PATTN_KV_F16), and a generic (not tensor-core)
                             kernel serves every row.  A caller built against
                             the header without this field gets 0.           */
} pattn_ext_t;

#define PATTN_MAX_SPLITS 64

/*
 * pattn_varlen_fwd -- the forward pass.
 *
 *   q               [device] bf16 [num_tokens, num_heads, head_size], contiguous
 *                   (f16 when kv_dtype is PATTN_KV_F16)
 *   kv_cache        [device] [2, num_blocks, block_size, num_kv_heads, head_size],
 *                   contiguous, bf16 or e4m3 bytes per kv_dtype; 16-B aligned
 *   block_table     [device] int32 [num_seqs, max_blocks_per_seq]; entries past
 *                   ceil(seq_len / block_size) are never read
 *   seq_lens        [device] int32 [num_seqs]
 *   query_start_loc [device] int32 [num_seqs + 1], non-decreasing prefix sum
 *   out             [device] bf16 (f16 with PATTN_KV_F16) [num_tokens, num_heads,
 *                   head_size]; rows of
 *                   tokens outside [query_start_loc[0], query_start_loc[B]) are
 *                   left untouched
 *   scale           multiplies q . k; finite and >= 0
 *   num_heads, num_kv_heads   num_heads % num_kv_heads == 0 and
 *                   num_heads / num_kv_heads <= 16
 *   head_size       64 or 128 (with ext->head_size_v > 0: the K head size, a
 *                   multiple of 32 up to 256; see pattn_ext_t.head_size_v)
 *   block_size      a multiple of 16 (the ValueError of get_kv_cache_shape)
 *   window          <= 0: no window; > 0: keys with p - k < window are visible
 *   causal          1: k <= p; 0: every key < seq_len (then window must be <= 0)
 *   kv_dtype        a pattn_kv_dtype_t.  With e4m3, decode rows run on the
 *                   bandwidth-bound decode kernel and prefill rows on the
 *                   tensor-core prefill kernel.  At head_size 128 its score
 *                   MMAs take the K codes as they are, against each q row
 *                   split exactly into two e4m3 codes per value after a
 *                   power-of-two scaling, and V tiles are widened to f16
 *                   (exactly) for f16 P V MMAs; at 64 K and V are widened and
 *                   q is scaled per row into f16 (the decode kernel likewise
 *                   per head).  With row scales a prefill V element is the f16
 *                   product of its code and the row's scale rounded to f16 (2^-11
 *                   each); the decode kernel puts the scales into the weights
 *   kv_scale        host float[2] {k_scale, v_scale}; required for e4m3, ignored
 *                   for bf16 (may be NULL).  For PATTN_KV_FP8_E4M3_ROW: the
 *                   [device] row scales (layout at PATTN_ROW_SCALE_MIN), 16-B
 *                   aligned; the scales of keys at or past seq_len are not used
 *   ext             host sizes, workspace and stream (see pattn_ext_t)
 *
 * Returns PATTN_OK once the work is enqueued.  Host-side checks return
 * INVALID_ARGUMENT / UNSUPPORTED / WORKSPACE_TOO_SMALL before any CUDA call;
 * a failed launch returns PATTN_ERR_CUDA.  Metadata the host cannot see
 * (q_len > seq_len, a block id outside [0, num_blocks), seq_len above
 * max_blocks_per_seq * block_size or max_seq_len) is detected on the device:
 * the offending ids are clamped so no access leaves the buffers, the rows of
 * that request are unspecified but finite, and a status word in the
 * workspace records it for pattn_read_device_status.
 */
pattn_status_t pattn_varlen_fwd(const void* q, const void* kv_cache,
                                const int32_t* block_table, const int32_t* seq_lens,
                                const int32_t* query_start_loc, void* out, float scale,
                                int num_heads, int num_kv_heads, int head_size,
                                int block_size, int window, int causal, int kv_dtype,
                                const float* kv_scale, const pattn_ext_t* ext);

/*
 * Workspace bytes pattn_varlen_fwd needs for these sizes (reads num_seqs,
 * num_tokens, max_query_len, max_seq_len and num_splits from ext; ignores its
 * workspace and stream).  Returns 0 if the arguments are invalid.
 */
size_t pattn_workspace_bytes(const pattn_ext_t* ext, int num_heads, int num_kv_heads,
                             int head_size, int block_size);

/*
 * The decode KV partition count pattn_varlen_fwd will use for these sizes
 * (ext->num_splits if set, else the library's choice).  Over a
 * PATTN_KV_FP8_E4M3_ROW cache the library's own choice is bounded further, by
 * max(1, sqrt(visible keys / 16) - 1) (in pattn_decode_fwd_static and in each
 * pass of pattn_cascade_fwd as well).  Partitions are runs of
 * ceil(n / splits) whole KV blocks over the n blocks a decode row can see,
 * merged by log-sum-exp ("RBLN Attention modes", flash attention; the Triton
 * backend's 16 parallel softmax segments).
 */
int pattn_decode_splits(const pattn_ext_t* ext, int num_heads, int num_kv_heads,
                        int block_size, int window);

/*
 * Reads and clears the device status word of ext->workspace (workspace_bytes as
 * for the call: calls of few CTAs leave more words behind it).  Synchronises
 * ext->stream.  Returns PATTN_OK, PATTN_ERR_BAD_METADATA or
 * PATTN_ERR_DEVICE_TIMEOUT for the calls since the last read (each
 * pattn_varlen_fwd call first clears the word on its stream), or
 * PATTN_ERR_CUDA if the copy fails.
 */
pattn_status_t pattn_read_device_status(const pattn_ext_t* ext);

/*
 * pattn_decode_fwd_static -- the decode rows of a batch, with no workspace.
 *
 * The pages have no counterpart to this entry point.  It exists for callers
 * that cannot allocate device memory or hand over a workspace: a plugin inside
 * an application whose allocator owns all device memory, or code on a
 * latency-critical path where cudaMalloc / cudaFree would synchronise the
 * device.  It computes exactly what pattn_varlen_fwd computes for the requests
 * with query_len == 1 (same kernels, same partition count for the same sizes),
 * leaves the rows of every other request untouched, and allocates nothing: no
 * cudaMalloc, no cudaFree, no allocating library routine.
 *
 * Arguments are those of pattn_varlen_fwd; the sizes of pattn_ext_t are passed
 * directly and `stream` is a cudaStream_t (NULL = legacy default stream).
 * Scratch comes from a fixed device array of PATTN_STATIC_SCRATCH_BYTES
 * inside the library, held by every GPU that loads the library until the
 * process exits.  A batch whose partials need more
 * (num_seqs * num_heads * splits * (head_size + 1) * 4 bytes, roughly) returns
 * PATTN_ERR_WORKSPACE_TOO_SMALL before any GPU work; pass a smaller
 * num_splits or use pattn_varlen_fwd.  Every call looks up the array's device
 * address in the current context (cudaGetSymbolAddress, which allocates
 * nothing), so the device that owns `stream` must be current; the first call
 * in a context may load the library's device code, so make it before any
 * stream capture.  Any context the runtime API can make current is served
 * (the primary one, or one a host application created and made current).
 * All calls share the array and it keeps the last call's contents: the
 * status word and the partition counters are cleared on `stream` at the start
 * of each call; calls whose work may overlap on the GPU (different streams or
 * host threads) race and must be serialised by the caller.  Requests with
 * query_len != 1 are skipped: their output rows are neither read nor written
 * and they are not reported.  Device-detected metadata errors of the decode
 * rows (a block id outside the pool, seq_len beyond the block table) are
 * clamped as in pattn_varlen_fwd, those rows are zeroed, and nothing is
 * reported (there is no workspace to read a status from).
 */
#define PATTN_STATIC_SCRATCH_BYTES (32u << 20)
pattn_status_t pattn_decode_fwd_static(const void* q, const void* kv_cache,
                                       const int32_t* block_table, const int32_t* seq_lens,
                                       const int32_t* query_start_loc, void* out, float scale,
                                       int num_heads, int num_kv_heads, int head_size,
                                       int block_size, int window, int causal, int kv_dtype,
                                       const float* kv_scale, int num_seqs, int num_tokens,
                                       int max_blocks_per_seq, int num_blocks, int max_seq_len,
                                       int num_splits, void* stream);

/*
 * pattn_cascade_fwd -- pattn_varlen_fwd for a batch whose requests all start
 * with the same cached prefix ("[vLLM] FlashAttention", Cascade Attention;
 * FlashAttentionMetadata.use_cascade / common_prefix_len).
 *
 * The prefix's attention is computed once for every query token of the batch
 * (one request of num_tokens queries over common_prefix_len keys, not causal:
 * every query sits after the prefix), each request's suffix (its keys past
 * the prefix) separately and causally, and the two are merged by
 * log-sum-exp.  The result is pattn_varlen_fwd's up to rounding; the prefix's
 * K/V pages are read once for the batch instead of once per request.
 *
 * Arguments are pattn_varlen_fwd's, plus common_prefix_len: a positive
 * multiple of block_size, at most max_seq_len.  The first
 * common_prefix_len / block_size block-table entries of every request must
 * name the same blocks (the pass reads row 0's), and every request's cached
 * context (seq_len - query_len) must cover the prefix; a request whose
 * context does not is reported as bad metadata (its rows are finite but
 * unspecified).  causal must be 1 and window <= 0 (else
 * PATTN_ERR_UNSUPPORTED); bf16, f16 and e4m3 caches are served as by
 * pattn_varlen_fwd.  The workspace comes from
 * pattn_cascade_workspace_bytes: besides the two passes' own scratch it holds
 * their fp32 partial results, 2 * num_tokens * num_heads * (head_size + 1)
 * floats.  The status word is read with pattn_read_device_status as usual.
 */
pattn_status_t pattn_cascade_fwd(const void* q, const void* kv_cache,
                                 const int32_t* block_table, const int32_t* seq_lens,
                                 const int32_t* query_start_loc, void* out, float scale,
                                 int num_heads, int num_kv_heads, int head_size,
                                 int block_size, int window, int causal, int kv_dtype,
                                 const float* kv_scale, int common_prefix_len,
                                 const pattn_ext_t* ext);

/* Workspace bytes pattn_cascade_fwd needs (0 if the arguments are invalid). */
size_t pattn_cascade_workspace_bytes(const pattn_ext_t* ext, int num_heads, int num_kv_heads,
                                     int head_size, int block_size, int common_prefix_len);

/*
 * pattn_reshape_and_cache -- write new key and value rows into the paged cache.
 *
 * The step that fills the cache pattn_varlen_fwd reads ("[vLLM]
 * FlashAttention", FlashAttentionMetadata.slot_mapping; the cache-write
 * kernel of the DiffKV backend in "[vLLM] other attention backends").
 *
 *   key, value      [device] bf16 [num_tokens, num_kv_heads, head_size],
 *                   contiguous, 16-B aligned
 *   kv_cache        [device] the cache of pattn_varlen_fwd, 16-B aligned,
 *                   updated in place
 *   slot_mapping    [device] int64 [num_tokens]: token t goes to block
 *                   slot / block_size, offset slot % block_size; a negative
 *                   slot writes nothing (padding).  Slots of one call must be
 *                   distinct (two tokens on one slot leave either's row).
 *   head_size       a multiple of 8; block_size a multiple of 16
 *   kv_dtype        bf16: the bits are copied; e4m3: each element x is stored
 *                   as e4m3(x / scale) (fp32 division, round to nearest even,
 *                   saturated at +-448, NaN stays NaN), scale = kv_scale[0]
 *                   for K and kv_scale[1] for V (host floats, > 0, finite)
 *   device_status   [device] optional (may be NULL): a slot at or beyond
 *                   num_blocks * block_size writes nothing and ORs
 *                   PATTN_ERR_BAD_METADATA's device bit (1) into this word
 *   stream          a cudaStream_t (NULL = legacy default stream)
 *
 * Returns PATTN_OK once enqueued; argument errors before any CUDA call;
 * PATTN_ERR_CUDA if the launch fails.  Allocates nothing, never synchronises.
 */
pattn_status_t pattn_reshape_and_cache(const void* key, const void* value, void* kv_cache,
                                       const int64_t* slot_mapping, int num_tokens,
                                       int num_kv_heads, int head_size, int block_size,
                                       int num_blocks, int kv_dtype, const float* kv_scale,
                                       unsigned* device_status, void* stream);

/*
 * pattn_reshape_and_cache_diffkv -- pattn_reshape_and_cache for the DiffKV
 * layout (pattn_ext_t.head_size_v; the DiffKV backend of "[vLLM] other
 * attention backends" has its own cache-write kernel for its asymmetric
 * cache).
 *
 *   key             [device] 16-bit [num_tokens, num_kv_heads, head_size]
 *   value           [device] 16-bit [num_tokens, num_kv_heads, head_size_v]
 *   kv_cache        [device] [num_blocks, block_size, num_kv_heads,
 *                   head_size + head_size_v], updated in place: token t's key
 *                   row then its value row go to row [s / block_size]
 *                   [s % block_size][h], s = slot_mapping[t]
 *   head_size, head_size_v   multiples of 8; block_size a multiple of 16
 *   kv_dtype        PATTN_KV_BF16 or PATTN_KV_F16 (the bits are copied)
 *   slot_mapping, device_status, stream   as for pattn_reshape_and_cache
 *
 * All buffers 16-B aligned.  Returns PATTN_OK once enqueued; argument errors
 * before any CUDA call.  Allocates nothing, never synchronises.
 */
pattn_status_t pattn_reshape_and_cache_diffkv(const void* key, const void* value,
                                              void* kv_cache, const int64_t* slot_mapping,
                                              int num_tokens, int num_kv_heads, int head_size,
                                              int head_size_v, int block_size, int num_blocks,
                                              int kv_dtype, unsigned* device_status,
                                              void* stream);

/*
 * pattn_reshape_and_cache_rows -- pattn_reshape_and_cache for a
 * PATTN_KV_FP8_E4M3_ROW cache: each (token, KV head) row of K and of V is
 * stored with a scale of its own,
 *   scale = max|x| / 448 clamped to [2^-60, 2^60] (NaN elements do not count),
 *   code  = e4m3(x / scale), fp32 division, round to nearest even, saturated
 *           at +-448, NaN stays NaN.
 * An infinity (and a magnitude above 448 * 2^60) is stored as the largest code.
 * Two tokens on one slot of a row-scaled cache can leave the codes of one with
 * the scale of the other, here and in pattn_rope_and_cache: slots must be distinct.
 *
 *   key, value      [device] bf16 [num_tokens, num_kv_heads, head_size]
 *   kv_cache        [device] e4m3 bytes, the cache of pattn_varlen_fwd
 *   row_scales      [device] the cache's scales, updated in place
 *   head_size       a multiple of 16, at most 256
 *   the rest        as for pattn_reshape_and_cache
 */
pattn_status_t pattn_reshape_and_cache_rows(const void* key, const void* value, void* kv_cache,
                                            float* row_scales, const int64_t* slot_mapping,
                                            int num_tokens, int num_kv_heads, int head_size,
                                            int block_size, int num_blocks,
                                            unsigned* device_status, void* stream);

/*
 * pattn_rope_and_cache -- rotary embedding of q and k and the cache write of k
 * and v, in one kernel: what a layer does between its q/k/v projection and
 * pattn_varlen_fwd.
 *
 * For token t: each q head and each k head is first normed if its weight is
 * given, x <- x * w / sqrt(mean(x^2) + norm_eps); then its first rot_dim
 * elements are rotated pair by pair,
 *   (a, b) -> (a c - b s, b c + a s),  c = cos_sin[P][i],
 *   s = cos_sin[P][rot_dim / 2 + i] for rotary pair i,
 *   P = positions[axis of pair i][t].
 * q goes to q_out, k and v to the cache slot slot_mapping[t], stored as kv_dtype
 * says: PATTN_KV_BF16 / PATTN_KV_F16 rounded to that type (q, key and value are
 * then of it too; they are bf16 with the e4m3 caches), PATTN_KV_FP8_E4M3 and
 * PATTN_KV_FP8_E4M3_ROW quantised as pattn_reshape_and_cache and
 * pattn_reshape_and_cache_rows do.  The norm, the rotation and the quantisation
 * are fp32 with one rounding at the end.
 *
 * Either q (with q_out) or key (with value) may be NULL, and is then left out.
 */
typedef struct {
  size_t struct_size;     /* sizeof(pattn_rope_t)                             */
  const void* q;          /* [device] [num_tokens] rows of num_heads * head_size;
                             token t's at q + t * q_stride elements           */
  void* q_out;            /* [device] likewise with q_out_stride; may be q itself
                             with the same stride, else must not overlap it   */
  const void* key;        /* [device] rows of num_kv_heads * head_size        */
  const void* value;      /* [device] likewise                                */
  long long q_stride, q_out_stride, key_stride, value_stride;
                          /* elements between tokens, multiples of 8 and at least
                             a token's row (so q, key and value may be parts of
                             one packed projection); all buffers 16-B aligned */
  const float* cos_sin;   /* [device] fp32 [max_position][rot_dim]: the cosines of
                             the rot_dim / 2 pairs, then their sines; 16-B aligned */
  const int64_t* positions; /* [device] [num_axes] rows of num_tokens         */
  long long positions_stride; /* elements between the axes' rows              */
  const unsigned char* pair_axis; /* host [rot_dim / 2]: the axis whose position
                             turns pair i; NULL with one axis                 */
  const void* q_norm;     /* [device] [head_size] weight of the norm of q heads, of
                             q's type, or NULL for no norm                    */
  const void* k_norm;     /* [device] likewise for k heads                    */
  void* kv_cache;         /* [device] the cache of pattn_varlen_fwd, updated  */
  float* row_scales;      /* [device] PATTN_KV_FP8_E4M3_ROW: the row scales, updated */
  const float* kv_scale;  /* PATTN_KV_FP8_E4M3: host float[2] {k_scale, v_scale} */
  const int64_t* slot_mapping; /* [device] [num_tokens], as for
                             pattn_reshape_and_cache: negative writes no key and
                             value (q is still rotated)                       */
  unsigned* device_status; /* [device] optional (may be NULL): a slot past the
                             pool (its key and value are not written) and a
                             position outside the table (nothing of the token is
                             written) OR bit 1 into it                        */
  void* stream;           /* cudaStream_t; NULL = the legacy default stream   */
  float norm_eps;         /* finite, >= 0                                     */
  int num_tokens;
  int num_heads;
  int num_kv_heads;
  int head_size;          /* a multiple of 16, at most 256                    */
  int rot_dim;            /* a multiple of 16, at most head_size              */
  int interleaved;        /* 0: pair i is elements (i, i + rot_dim / 2);
                             1: elements (2 i, 2 i + 1)                       */
  int num_axes;           /* 0: no rotation; 1: one position per token; 2..4  */
  int max_position;       /* rows of cos_sin.  A token whose first axis' position
                             is negative is padding: nothing of it is written */
  int kv_dtype;
  int block_size;         /* a multiple of 16                                 */
  int num_blocks;
} pattn_rope_t;

/* Returns PATTN_OK once enqueued; argument errors before any CUDA call;
 * PATTN_ERR_CUDA if the launch fails.  Allocates nothing, never synchronises. */
pattn_status_t pattn_rope_and_cache(const pattn_rope_t* args);

/*
 * pattn_gather_cache -- read ranges of the cache back into contiguous rows (to
 * hand a prefix to another instance, or to a kernel that wants dense K and V).
 *
 * Request r's output rows are [out_start_loc[r], out_start_loc[r + 1]); row
 * out_start_loc[r] + i holds its key key_starts[r] + i.  A code of an e4m3
 * cache becomes code * scale (fp32), rounded once to bf16; 16-bit caches are
 * copied.
 *
 *   kv_cache, block_table, kv_dtype, kv_scale   as for pattn_varlen_fwd
 *   key_starts      [device] int32 [num_seqs], or NULL for 0
 *   out_start_loc   [device] int32 [num_seqs + 1], non-decreasing
 *   key_out, value_out   [device] [num_rows, num_kv_heads, head_size], bf16 (f16
 *                   for PATTN_KV_F16), 16-B aligned; rows outside
 *                   [out_start_loc[0], out_start_loc[num_seqs]) are left as they
 *                   are, and no row at or past num_rows is written
 *   head_size       a multiple of 8
 *   device_status   [device] optional (may be NULL): a key outside its block-table
 *                   row or a block id outside the pool zeroes the output row and
 *                   ORs bit 1 into this word
 *
 * Returns PATTN_OK once enqueued; argument errors before any CUDA call;
 * PATTN_ERR_CUDA if the launch fails.  Allocates nothing, never synchronises.
 */
pattn_status_t pattn_gather_cache(const void* kv_cache, const int32_t* block_table,
                                  const int32_t* key_starts, const int32_t* out_start_loc,
                                  void* key_out, void* value_out, int num_seqs, int num_rows,
                                  int max_blocks_per_seq, int num_blocks, int num_kv_heads,
                                  int head_size, int block_size, int kv_dtype,
                                  const float* kv_scale, unsigned* device_status, void* stream);

/*
 * Attention with keys and values from one shared latent vector a token.
 *
 * A model of this kind caches, per token, one row that all heads share: a latent
 * vector c (latent_size elements) and a rotary key k (rope_size elements).  The
 * cache is [num_blocks, block_size, latent_size + rope_size], 16-bit
 * (PATTN_KV_BF16 or PATTN_KV_F16; q, out and the other tensors are of its type),
 * addressed by block table and slot mapping like the caches above.  The
 * attention has two forms.  Absorbed: the up-projection of the keys is folded
 * into q and that of the values into what follows, so every head attends the
 * cached rows themselves (pattn_latent_fwd; single tokens and short chunks).
 * Expanded: keys and values are projected up to a pair per head and attended
 * densely (pattn_latent_expanded_fwd; prompts).  ("[vLLM] other attention
 * backends" and "RBLN Attention modes" name this attention and its latent cache;
 * they give no layout, this is the reading taken.)
 *
 * Sizes of every entry point below: latent_size a multiple of 128 up to 512,
 * rope_size a multiple of 16 up to 64, block_size a multiple of 16.
 *
 * Both attentions hold scores, maxima, sums and outputs in fp32 and round twice: a
 * weight to the cache's type, half a step of it (2^-8 or 2^-11 relative; an f16
 * weight below 2^-14 of the largest by 2^-25 of that one), as the tensor cores take
 * their operands, and the result.  The normaliser sums the weights unrounded.
 *
 * As the product p . V defines it, a weight of 0 times an infinity or a NaN is NaN: a
 * non-finite value of a key that the causal mask hides can reach rows of its
 * request.  Keys at or past seq_len and other requests' keys never do.
 */

/*
 * pattn_latent_rope_and_cache -- the cache write of a step's tokens, in one
 * kernel: for token t the latent is normed if a weight is given,
 *   c <- c * w / sqrt(mean(c^2) + norm_eps),
 * the rotary key and the rotary part of every q head are turned pair by pair,
 *   (a, b) -> (a cos - b sin, b cos + a sin),  cos = cos_sin[positions[t]][i],
 *   sin = cos_sin[positions[t]][rope_size / 2 + i] for pair i,
 * and c and the key become the cache row of slot_mapping[t].  fp32 with one
 * rounding at the end.
 */
typedef struct {
  size_t struct_size;     /* sizeof(pattn_latent_rope_t)                      */
  const void* q;          /* [device] rotary parts of q: head h of token t at
                             q + t * q_stride + h * q_head_stride, rope_size
                             elements; NULL: the cache row only               */
  void* q_out;            /* [device] likewise; may be q with the same strides,
                             else must not overlap it                         */
  const void* latent;     /* [device] token t's at latent + t * latent_stride */
  const void* k_rope;     /* [device] token t's at k_rope + t * k_rope_stride */
  void* row_out;          /* [device] optional: the written row densely as well,
                             token t's at row_out + t * row_out_stride (latent,
                             then key); may be the rows that latent and k_rope
                             are the parts of                                 */
  long long q_stride, q_head_stride, q_out_stride, q_out_head_stride, latent_stride,
      k_rope_stride, row_out_stride; /* elements, multiples of 8; all buffers 16-B
                             aligned                                          */
  const void* latent_norm; /* [device] [latent_size] weight, or NULL          */
  const float* cos_sin;   /* [device] fp32 [max_position][rope_size], 16-B aligned */
  const int64_t* positions; /* [device] [num_tokens], or NULL for no rotation.  A
                             negative one marks padding: nothing of the token
                             is written                                       */
  void* kv_cache;         /* [device] the cache, updated                      */
  const int64_t* slot_mapping; /* [device] [num_tokens]; negative: no cache row.
                             Slots must be distinct                           */
  unsigned* device_status; /* [device] optional: a slot past the pool (no row is
                             written) and a position outside the table (nothing
                             of the token is) OR bit 1 into it                */
  void* stream;           /* cudaStream_t; NULL = the legacy default stream   */
  float norm_eps;         /* finite, >= 0                                     */
  int num_tokens;
  int num_heads;
  int latent_size;
  int rope_size;
  int interleaved;        /* 0: pair i is elements (i, i + rope_size / 2);
                             1: elements (2 i, 2 i + 1)                       */
  int max_position;       /* rows of cos_sin                                  */
  int kv_dtype;
  int block_size;
  int num_blocks;
} pattn_latent_rope_t;

/* Returns PATTN_OK once enqueued; argument errors before any CUDA call;
 * PATTN_ERR_CUDA if the launch fails.  Allocates nothing, never synchronises. */
pattn_status_t pattn_latent_rope_and_cache(const pattn_latent_rope_t* args);

/*
 * pattn_gather_latent -- pattn_gather_cache for a cache of latent rows: request
 * r's keys key_starts[r] (NULL: 0), ... into rows [out_start_loc[r],
 * out_start_loc[r + 1]) of latent_out [num_rows, latent_size] and rope_out
 * [num_rows, rope_size] (what an up-projection and the expanded form take).  Rows
 * outside are left as they are; a key outside its block-table row or a block id
 * outside the pool zeroes the row and ORs bit 1 into device_status (may be NULL).
 */
pattn_status_t pattn_gather_latent(const void* kv_cache, const int32_t* block_table,
                                   const int32_t* key_starts, const int32_t* out_start_loc,
                                   void* latent_out, void* rope_out, int num_seqs, int num_rows,
                                   int max_blocks_per_seq, int num_blocks, int latent_size,
                                   int rope_size, int block_size, int kv_dtype,
                                   unsigned* device_status, void* stream);

/*
 * pattn_latent_fwd -- the absorbed form over the paged cache.
 *
 *   out[t][h] = softmax over visible keys k of (scale * q[t][h] . [c_k | key_k]) . c
 *
 * with the requests, block table, lengths, causal mask, metadata checks and
 * status word of pattn_varlen_fwd (row i of request r at position seq_len -
 * q_len + i); a seq_len above 2^31 - 256 is bad metadata too, however wide the
 * block table.  A request's cached rows are read once for all its rows' heads up
 * to 64 (row, head) pairs; the keys are cut into equal shares over the GPU, and
 * requests that several shares touch are merged by log-sum-exp in a fixed order.
 */
typedef struct {
  size_t struct_size;     /* sizeof(pattn_latent_t)                           */
  const void* q;          /* [device] [num_tokens][num_heads][latent_size +
                             rope_size], contiguous, 16-B aligned             */
  const void* kv_cache;   /* [device] 16-B aligned                            */
  void* out;              /* [device] [num_tokens][num_heads][latent_size], rows
                             outside the requests are left untouched          */
  const int32_t* block_table;     /* [device] [num_seqs][max_blocks_per_seq]  */
  const int32_t* seq_lens;        /* [device] [num_seqs]                      */
  const int32_t* query_start_loc; /* [device] [num_seqs + 1]                  */
  void* workspace;        /* [device] 256-B aligned; its status word is read with
                             pattn_read_device_status                         */
  size_t workspace_bytes; /* >= pattn_latent_workspace_bytes                  */
  void* stream;
  float scale;            /* finite, >= 0                                     */
  int causal;             /* 1: k <= position; 0: every key < seq_len         */
  int kv_dtype;
  int num_seqs, num_tokens, num_heads, latent_size, rope_size, block_size;
  int max_blocks_per_seq, num_blocks;
  int max_query_len;      /* >= every q_len                                   */
} pattn_latent_t;

pattn_status_t pattn_latent_fwd(const pattn_latent_t* args);

/* Workspace bytes pattn_latent_fwd needs on the current device (0 if the arguments are
 * invalid).  They follow from latent_size; num_seqs and num_heads are only checked. */
size_t pattn_latent_workspace_bytes(int num_seqs, int num_heads, int latent_size);

/*
 * pattn_latent_expanded_fwd -- the expanded form over contiguous ragged rows.
 *
 *   out[t][h] = softmax over visible keys k of
 *               scale * (q[t][h][:nope] . k_nope[k][h] + q[t][h][nope:] . k_rope[k])
 *               . value[k][h]
 *
 * Request r has q rows [query_start_loc[r], query_start_loc[r + 1]) and keys
 * [key_start_loc[r], key_start_loc[r + 1]); with causal its i-th row sees its
 * first keys - queries + i + 1 keys.  A request with causal and more rows than
 * keys, or rows or keys outside the tensors, is reported as bad metadata and its
 * rows are zeroed; a request without keys has rows of zeros.
 */
typedef struct {
  size_t struct_size;     /* sizeof(pattn_latent_expanded_t)                  */
  const void* q;          /* [device] head h of token t at q + t * q_stride +
                             h * q_head_stride: nope_size + rope_size elements */
  const void* k_nope;     /* [device] likewise, nope_size elements            */
  const void* k_rope;     /* [device] key k's at k_rope + k * k_rope_stride   */
  const void* value;      /* [device] as k_nope, value_size elements          */
  void* out;              /* [device] [num_tokens][num_heads][value_size]     */
  long long q_stride, q_head_stride, k_stride, k_head_stride, k_rope_stride, v_stride,
      v_head_stride;      /* elements, positive multiples of 8; buffers 16-B aligned */
  const int32_t* query_start_loc; /* [device] [num_seqs + 1], non-decreasing  */
  const int32_t* key_start_loc;   /* [device] [num_seqs + 1], non-decreasing  */
  void* workspace;        /* as in pattn_latent_t                             */
  size_t workspace_bytes; /* >= pattn_latent_expanded_workspace_bytes         */
  void* stream;
  float scale;
  int causal;
  int kv_dtype;
  int num_seqs, num_tokens, num_keys, num_heads;
  int nope_size, rope_size, value_size; /* 64 or 128, the same for value; rope_size
                             a multiple of 16 up to 64                        */
} pattn_latent_expanded_t;

pattn_status_t pattn_latent_expanded_fwd(const pattn_latent_expanded_t* args);

/* Workspace bytes pattn_latent_expanded_fwd needs (0 if the arguments are invalid). */
size_t pattn_latent_expanded_workspace_bytes(int num_seqs, int num_tokens);

/* A static, human-readable name for a status code. */
const char* pattn_status_string(int status);

/* Library ABI version: major * 10000 + minor * 100 + patch. */
int pattn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PATTN_H */
