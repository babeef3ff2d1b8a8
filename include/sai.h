/*
 * sai.h -- C ABI of libsai, the GB300 (sm_103a) sparse-attention indexer
 * top-k library.
 *
 * Conventions for every entry point
 * ---------------------------------
 * - All array pointers are DEVICE pointers on the calling thread's current
 *   CUDA device, owned by the caller. The library allocates nothing; where
 *   scratch memory helps, the caller passes a workspace sized by the matching
 *   *_workspace query (same arguments, same device).
 * - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL = the
 *   legacy default stream). No entry point synchronizes, except
 *   sai_device_status.
 * - Host-visible argument errors are reported before anything is launched.
 *   Row metadata that lives on the device (seq_lens, row_starts,
 *   row_to_batch, page/block ids) is checked by the kernels: an out-of-range
 *   row is treated as empty (all -1 outputs) and a bit is set in the
 *   library's device status word, read with sai_device_status. No kernel
 *   ever reads outside the extents the caller declares.
 * - Row-local index order of the k outputs: higher score first, equal scores
 *   to the lower row-local index (-0.0 == +0.0; +-inf are ordinary values;
 *   NaN scores are not admissible). Positions [min(seq_len, k), k) are -1.
 * - No C++ exception crosses this boundary.
 */
#ifndef SAI_H_
#define SAI_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t; declared here so users need no CUDA headers. */
typedef struct CUstream_st* sai_stream_t;

typedef enum {
  SAI_OK = 0,
  SAI_ERR_NULL = -1,        /* a required pointer is NULL */
  SAI_ERR_SHAPE = -2,       /* a size or count is out of range */
  SAI_ERR_UNSUPPORTED = -3, /* valid but not implemented (e.g. k != 512) */
  SAI_ERR_WORKSPACE = -4,   /* workspace too small or misaligned */
  SAI_ERR_CUDA = -5,        /* a CUDA runtime call or launch failed */
  SAI_ERR_DEVICE_CHECK = -6,/* a kernel flagged bad device-side metadata */
  SAI_ERR_ALIGN = -7        /* a pointer lacks the alignment its type needs */
} sai_status;

/* Fixed top-k of this library (the "512" of topk_transform_512_v2). */
#define SAI_TOPK 512

/* Human-readable name of a status code (static storage). */
const char* sai_status_string(int status);

/*
 * Text of the CUDA error behind the calling thread's most recent
 * SAI_ERR_CUDA ("" if none); valid until that thread's next call.
 */
const char* sai_last_error(void);

/*
 * Read (and optionally clear) the device status word of the current device
 * after synchronizing `stream`. *out_bits receives the OR of the bits set by
 * kernels since the last clear: 1 = bad row metadata, 2 = an internal
 * pipeline wait gave up, 4 = a block id out of range, 8 = a request got no
 * pages (sai_resize_pages). Returns SAI_ERR_DEVICE_CHECK if any bit was set, else SAI_OK.
 */
int sai_device_status(int* out_bits, int clear, sai_stream_t stream);

/*
 * Test hook for the bounded waits (not part of the computation; the paper
 * has no counterpart). Every pipeline wait inside the kernels gives up after
 * about two seconds, sets status bit 2 and lets the launch finish, so a lost
 * arrival can never hang the GPU. To exercise that exit, the next
 * sai_index_score_topk / sai_index_score_topk_bf16 call made by this host
 * thread streams no key tiles for its work unit `unit` (a unit is a group of
 * query rows and a chunk of their KV blocks; unit 0 holds the first rows'
 * first chunk): that unit's waits run out, the call completes with status
 * bit 2 set, and the rows of that unit are undefined. -1 clears the hook;
 * the call consumes it either way.
 */
void sai_test_stall_next_fused(int32_t unit);

/*
 * Workspace bytes that sai_topk_transform wants for these sizes on the
 * current device: a 256-byte header (a work counter that lets CTAs take
 * rows as they finish, zeroed by the call on its stream), plus, when long
 * rows on few rows are split over several CTAs, their partial top-k lists.
 */
size_t sai_topk_transform_workspace(int64_t rows, int64_t score_stride, int32_t k);

/*
 * sai_topk_transform -- per-row window top-k and page-table transform.
 *
 * Follows sglang PR #37889 "[AMD] Enable GLM DSA prefill top-k to the v2
 * kernel" (Modifications: the two optional (rows,) int32 indirections of
 * topk_transform_512_v2) and ROCm/ATOM PR #1282 "merge build sparse block
 * into topk" (the physical addressing is produced by the top-k kernel).
 *
 * For each row i in [0, rows):
 *   n      = seq_lens[i]
 *   start  = row_starts ? row_starts[i] : 0
 *   window = scores[i*score_stride + start + t], t in [0, n)
 *   b      = row_to_batch ? row_to_batch[i] : i
 *   idx[j] = row-local position of the j-th best score (j < min(n, k))
 *   slot[j]= page_tables[b*pt_stride + idx[j]/page_size]*page_size
 *            + idx[j]%page_size
 *
 * scores       fp32 [rows, score_stride], 4-byte aligned; any stride and any
 *              row start work (the 16-byte-aligned interior of each window
 *              is streamed with bulk TMA copies, the ragged ends with scalar
 *              loads).
 * row_starts   int32 [rows] or NULL. The caller guarantees
 *              start + n <= score_stride (checked on device).
 * seq_lens     int32 [rows], >= 0.
 * page_tables  int32 [pt_rows, pt_stride]; required when out_slots or
 *              out_blocks is given.
 *              Without row_to_batch, pt_rows >= rows is checked here; with
 *              it, 0 <= row_to_batch[i] < pt_rows is checked on device.
 * page_size    >= 1 (1 = one slot per token, the "wide" table).
 * k            must be 512 (SAI_ERR_UNSUPPORTED otherwise).
 * out_slots    int32 [rows, 512] or NULL; out_indices int32 [rows, 512] or
 *              NULL (row-local positions).
 * out_blocks   int32 [rows, 512] or NULL: the row's selected slots as the
 *              ascending distinct blocks slot / block_size, -1 padded, built
 *              by the same call from the slots it picks (ROCm/ATOM PR #1282
 *              "merge build sparse block into topk": the block list comes out
 *              of the top-k, not out of a second pass over the slots); needs
 *              page_tables. block_size >= 1 when out_blocks is given (128:
 *              a 128-token KV block; ignored otherwise). out_counts int32
 *              [rows] or NULL: each row's number of blocks (only with
 *              out_blocks). At least one of out_slots, out_indices and
 *              out_blocks must be given.
 * workspace    device memory of workspace_bytes (16-byte aligned) or NULL.
 *              If it is smaller than sai_topk_transform_workspace asks for,
 *              every row is processed by a single CTA (correct, slower for
 *              few long rows); below 256 bytes (or NULL) the CTAs also take
 *              rows in a fixed order instead of from the work counter.
 *              Calls that share a workspace must not overlap on the GPU.
 */
int sai_topk_transform(const float* scores, int64_t rows, int64_t score_stride, const int32_t* row_starts,
                       const int32_t* seq_lens, const int32_t* page_tables, int64_t pt_rows, int64_t pt_stride,
                       const int32_t* row_to_batch, int32_t page_size, int32_t k, int32_t* out_slots,
                       int32_t* out_indices, int32_t block_size, int32_t* out_blocks, int32_t* out_counts,
                       void* workspace, size_t workspace_bytes, sai_stream_t stream);

/*
 * Workspace bytes that sai_index_score_topk needs for these sizes on the
 * current device (the per-(row, KV chunk) candidate lists).
 */
size_t sai_index_score_topk_workspace(int64_t rows, int32_t max_seq_len, int32_t group_rows, int32_t k);

/*
 * sai_index_score_topk -- FP8 index scores and top-k in one pass.
 *
 * Follows ROCm/ATOM PR #1473 "enable minimax m3 fp8 index cache and fuse
 * index_score_kernel with partial_topk kernel" (pull request overview: FP8
 * index cache, the score computed in FP8, index score and partial top-k fused
 * so that no score tensor is written; the fused decode kernel walks the
 * request's block table and masks keys at or beyond the causal length).
 * For each query row i, with b = row_to_batch ? row_to_batch[i] : i and
 * n = seq_lens[i]:
 *   score(t) = kscale[p*128 + o] * sum_h w[i*64 + h] * relu(sum_d q[i,h,d] k[p,o,d])
 *   for t < n, p = block_table[b*bt_stride + t/128], o = t % 128;
 * then the top-k keys by (score desc, index asc):
 *   out_indices[i*512 + j] = t_j, out_slots[...] = p_j*128 + o_j,
 *   out_scores[...] = score(t_j) (fp32), padded with -1 / NaN;
 *   optionally out_blocks[i*512 + j] = the row's ascending distinct
 *   out_slots / list_block_size (-1 padded) and out_counts[i] their number,
 *   as for sai_topk_transform (list_block_size 128 gives the block ids p_j).
 *
 * q_fp8       e4m3fn [rows, heads, dim], 16-byte aligned.
 * w           fp32 [rows, heads].
 * kcache_fp8  e4m3fn [num_blocks, block_size, dim], 16-byte aligned.
 * kscale      fp32 [num_blocks, block_size].
 * block_table int32 [bt_rows, bt_stride]; block ids outside [0, num_blocks)
 *             mask their keys and set status bit 4.
 * seq_lens    int32 [rows], 0 <= n <= max_seq_len and ceil(n/128) <= bt_stride
 *             (checked on device; a bad row is emptied and sets bit 1).
 * heads = 64, dim = 128, block_size = 128, k = 512 (else SAI_ERR_UNSUPPORTED).
 * group_rows  1, or 4 when every 4 consecutive rows share one row_to_batch
 *             value (packed prefill): the kernel then scores the rows in
 *             pairs, each key block once per pair. A pair whose rows differ
 *             is emptied and sets bit 1.
 * out_*       any of out_slots, out_indices, out_scores, out_blocks may be
 *             NULL, not all; out_counts only with out_blocks, which needs
 *             list_block_size >= 1.
 * workspace   at least sai_index_score_topk_workspace(...) bytes, 16-byte aligned.
 */
int sai_index_score_topk(const uint8_t* q_fp8, const float* w, const uint8_t* kcache_fp8, const float* kscale,
                         int64_t num_blocks, const int32_t* block_table, int64_t bt_rows, int64_t bt_stride,
                         const int32_t* row_to_batch, const int32_t* seq_lens, int64_t rows, int32_t heads,
                         int32_t dim, int32_t block_size, int32_t max_seq_len, int32_t group_rows, int32_t k,
                         int32_t* out_slots, int32_t* out_indices, float* out_scores, int32_t list_block_size,
                         int32_t* out_blocks, int32_t* out_counts, void* workspace, size_t workspace_bytes,
                         sai_stream_t stream);

/*
 * sai_index_score -- the same FP8 index scores written densely (for tests):
 * out_scores[i*out_stride + t] = score(i, t) for t < seq_lens[i]; other
 * cells are not written. out_stride >= max_seq_len. Same argument rules.
 */
int sai_index_score(const uint8_t* q_fp8, const float* w, const uint8_t* kcache_fp8, const float* kscale,
                    int64_t num_blocks, const int32_t* block_table, int64_t bt_rows, int64_t bt_stride,
                    const int32_t* row_to_batch, const int32_t* seq_lens, int64_t rows, int32_t heads, int32_t dim,
                    int32_t block_size, int32_t max_seq_len, int32_t group_rows, float* out_scores,
                    int64_t out_stride, sai_stream_t stream);

/*
 * sai_index_score_topk_bf16 / sai_index_score_bf16 -- the same two calls for
 * a bf16 index cache.
 *
 * The index cache may be kept at the model dtype instead of FP8 (ROCm/ATOM PR
 * #1473: the index-cache type option whose default "auto" is the model dtype,
 * and its commit "convert auto for bf16 type"; FP8 only when the KV cache
 * dtype is an fp8 one). Then q and the keys are bfloat16 bit patterns and the
 * dot products run in bf16 with fp32 accumulation; the score, selection,
 * outputs, workspace (sai_index_score_topk_workspace) and status bits are those
 * of the FP8 calls.
 *
 * q_bf16       bf16 [rows, heads, dim], 16-byte aligned.
 * kcache_bf16  bf16 [num_blocks, block_size, dim], 16-byte aligned.
 * kscale       fp32 [num_blocks, block_size], or NULL: the pages give a bf16
 *              cache no per-key scale, and NULL means scale 1.
 * Other arguments as for sai_index_score_topk / sai_index_score.
 */
int sai_index_score_topk_bf16(const uint16_t* q_bf16, const float* w, const uint16_t* kcache_bf16,
                              const float* kscale, int64_t num_blocks, const int32_t* block_table, int64_t bt_rows,
                              int64_t bt_stride, const int32_t* row_to_batch, const int32_t* seq_lens, int64_t rows,
                              int32_t heads, int32_t dim, int32_t block_size, int32_t max_seq_len, int32_t group_rows,
                              int32_t k, int32_t* out_slots, int32_t* out_indices, float* out_scores,
                              int32_t list_block_size, int32_t* out_blocks, int32_t* out_counts, void* workspace,
                              size_t workspace_bytes, sai_stream_t stream);
int sai_index_score_bf16(const uint16_t* q_bf16, const float* w, const uint16_t* kcache_bf16, const float* kscale,
                         int64_t num_blocks, const int32_t* block_table, int64_t bt_rows, int64_t bt_stride,
                         const int32_t* row_to_batch, const int32_t* seq_lens, int64_t rows, int32_t heads,
                         int32_t dim, int32_t block_size, int32_t max_seq_len, int32_t group_rows, float* out_scores,
                         int64_t out_stride, sai_stream_t stream);

/*
 * Per-index-head top-k: one selection per (query row, index head).
 *
 * The fused decode kernel of ROCm/ATOM PR #1473 is launched over (query,
 * index head, key chunk) (review diff of index_topk.py), which admits a
 * selection per index head. Head h's score is its summand of the
 * head-summed score:
 *   score_h(t) = kscale[p*128 + o] * w[i*64 + h] * relu(sum_d q[i,h,d] k[p,o,d])
 * (p, o, n, b as for sai_index_score_topk), and each (i, h) takes its top-k
 * keys by (score desc, index asc).
 *
 * sai_index_score_per_head[_bf16] writes the scores densely:
 *   out_scores[(i*64 + h)*out_stride + t] = score_h(t) for t < seq_lens[i]
 * (other cells untouched; a key on a block id outside [0, num_blocks) gets
 * -inf and sets status bit 4). out_stride >= max_seq_len.
 *
 * sai_index_score_topk_per_head[_bf16] computes those scores into its
 * workspace and selects with the top-k kernel:
 *   out_indices[(i*64 + h)*512 + j] = t_j, out_slots[...] = p_j*128 + o_j
 * (-1 padded; either output may be NULL, not both). The workspace holds
 * rows*64 score rows of max_seq_len floats (rounded up to 4) plus metadata:
 * sai_index_score_topk_per_head_workspace(...) bytes, 256-byte aligned
 * (about 17 MB per decode row of 32768 keys).
 *
 * Arguments as for sai_index_score_topk (FP8) / sai_index_score_topk_bf16
 * (bf16, kscale may be NULL), without group_rows (rows are scored one per
 * unit). Same host errors; bad rows are emptied and flagged as there.
 */
size_t sai_index_score_topk_per_head_workspace(int64_t rows, int32_t max_seq_len, int32_t k);
int sai_index_score_per_head(const uint8_t* q_fp8, const float* w, const uint8_t* kcache_fp8, const float* kscale,
                             int64_t num_blocks, const int32_t* block_table, int64_t bt_rows, int64_t bt_stride,
                             const int32_t* row_to_batch, const int32_t* seq_lens, int64_t rows, int32_t heads,
                             int32_t dim, int32_t block_size, int32_t max_seq_len, float* out_scores,
                             int64_t out_stride, sai_stream_t stream);
int sai_index_score_per_head_bf16(const uint16_t* q_bf16, const float* w, const uint16_t* kcache_bf16,
                                  const float* kscale, int64_t num_blocks, const int32_t* block_table,
                                  int64_t bt_rows, int64_t bt_stride, const int32_t* row_to_batch,
                                  const int32_t* seq_lens, int64_t rows, int32_t heads, int32_t dim,
                                  int32_t block_size, int32_t max_seq_len, float* out_scores, int64_t out_stride,
                                  sai_stream_t stream);
int sai_index_score_topk_per_head(const uint8_t* q_fp8, const float* w, const uint8_t* kcache_fp8,
                                  const float* kscale, int64_t num_blocks, const int32_t* block_table,
                                  int64_t bt_rows, int64_t bt_stride, const int32_t* row_to_batch,
                                  const int32_t* seq_lens, int64_t rows, int32_t heads, int32_t dim,
                                  int32_t block_size, int32_t max_seq_len, int32_t k, int32_t* out_slots,
                                  int32_t* out_indices, void* workspace, size_t workspace_bytes,
                                  sai_stream_t stream);
int sai_index_score_topk_per_head_bf16(const uint16_t* q_bf16, const float* w, const uint16_t* kcache_bf16,
                                       const float* kscale, int64_t num_blocks, const int32_t* block_table,
                                       int64_t bt_rows, int64_t bt_stride, const int32_t* row_to_batch,
                                       const int32_t* seq_lens, int64_t rows, int32_t heads, int32_t dim,
                                       int32_t block_size, int32_t max_seq_len, int32_t k, int32_t* out_slots,
                                       int32_t* out_indices, void* workspace, size_t workspace_bytes,
                                       sai_stream_t stream);

/*
 * sai_sparse_blocks -- per-row distinct KV blocks of top-k slots.
 *
 * For callers that already hold slots; the top-k entry points above build
 * the same lists in their last stage when given out_blocks.
 * Follows ROCm/ATOM PR #1282 "merge build sparse block into topk" (title and
 * Motivation): the sparse attention after the indexer reads KV blocks, so
 * each row's selected physical slots (the out_slots of sai_topk_transform
 * or sai_index_score_topk) become the list of distinct blocks they fall in.
 * For each row i:
 *   B_i = ascending distinct values of slots[i*k + j] / block_size over the
 *         j in [0, k) with slots[i*k + j] >= 0 (negative slots are padding)
 *   out_blocks[i*k + t] = B_i[t] for t < |B_i|, -1 for |B_i| <= t < k
 *   out_counts[i] = |B_i|
 *
 * slots       int32 [rows, k], 4-byte aligned; k in [1, 512].
 * block_size  >= 1 (128: the KV block of the fused path; a slot of the
 *             page_size=1 top-k is a token slot, so its block is slot / 128).
 * out_blocks  int32 [rows, k]; out_counts int32 [rows] or NULL.
 * Errors: NULL pointers, k outside [1, 512] or block_size < 1 are reported
 * before anything is launched.
 */
int sai_sparse_blocks(const int32_t* slots, int64_t rows, int32_t k, int32_t block_size, int32_t* out_blocks,
                      int32_t* out_counts, sai_stream_t stream);

/*
 * Size of the library-owned device scratch used by
 * sai_topk_transform_noalloc: 8 MiB, held on every GPU that loads the
 * library until the process exits.
 */
#define SAI_NOALLOC_SCRATCH_BYTES (8u << 20)

/*
 * sai_topk_transform_noalloc -- sai_topk_transform without a workspace
 * argument, for callers that cannot allocate device memory where they need
 * the top-k (inside an allocator callback or a region that forbids
 * allocation, a pool owner whose memory is all handed out, or code with no
 * allocator beyond its fixed input and output buffers). The paper has no
 * counterpart: this entry point exists only for such callers.
 *
 * Arguments, outputs, ordering and errors are those of sai_topk_transform
 * without the block-list outputs. Instead of a caller workspace, every call
 * uses a fixed library-owned
 * device array of SAI_NOALLOC_SCRATCH_BYTES: its first 256 bytes hold the
 * work counter from which the CTAs take rows (reset to zero by each call on
 * its stream), and the split path for few long rows also keeps its partial
 * top-k lists there. Calls whose sizes need more scratch than that (as
 * reported by sai_topk_transform_workspace) are rejected with
 * SAI_ERR_WORKSPACE before anything is launched. Nothing is allocated: no
 * cudaMalloc, no cudaFree.
 *
 * The first call on a device looks up the array's device address with that
 * device current; make that first call before any stream capture. All calls
 * on a device share the one array and it keeps the previous call's contents
 * (the counter is the only part that must start at zero, and each call
 * clears it). Any two calls that can overlap on the GPU (different streams
 * without ordering between them), short rows or long, race on the work
 * counter and, when split, on the partial lists: rows can be skipped and
 * outputs left unwritten. The caller must serialize them.
 */
int sai_topk_transform_noalloc(const float* scores, int64_t rows, int64_t score_stride, const int32_t* row_starts,
                               const int32_t* seq_lens, const int32_t* page_tables, int64_t pt_rows,
                               int64_t pt_stride, const int32_t* row_to_batch, int32_t page_size, int32_t k,
                               int32_t* out_slots, int32_t* out_indices, sai_stream_t stream);

/*
 * Paged key/value caches and the attention over them.
 *
 * What the indexer's caller does next to the calls above: the step's keys and
 * values go into a paged cache (sai_append_kv), the attention reads the slots
 * that the top-k picked (sai_sparse_attention), and layers without the
 * indexer attend over all keys or a sliding window of them
 * (sai_paged_attention). Rows, seq_lens, row_to_batch and block_table mean
 * what they mean for sai_index_score_topk: row i belongs to request
 * b = row_to_batch ? row_to_batch[i] : i and sits at position seq_lens[i] - 1
 * of it, token t of request b is cell t % block_size of block
 * block_table[b*bt_stride + t/block_size], and its slot is
 * block * block_size + cell. A row with seq_lens[i] = 0 is padding.
 *
 * sai_kv_cache describes one layer's cache; the arrays belong to the caller.
 *
 * k, v        [num_blocks, heads, block_size, dim], bf16 or e4m3 codes; the
 *             last axis has unit stride, the strides of the others (in
 *             elements) are given, so that heads and tokens may be in either
 *             order and k and v may share one array. 16-byte aligned, every
 *             stride a multiple of 16 bytes.
 * k_scale,    fp32 [num_blocks, heads], contiguous: value = code * scale, one
 * v_scale     scale for each block of tokens and kv head, 0 included. e4m3
 *             only. The attention sums are exact to their rounding while the
 *             value scales that a row sees are within 2^100 of each other
 *             (those below 2^-64 count as 2^-64); beyond that, weights of keys
 *             with small scales may be lost from the sums.
 * block_size  16, 32, 64 or 128; dim 64 or 128.
 */
#define SAI_CACHE_BF16 0
#define SAI_CACHE_E4M3 1
#define SAI_PACKED_TILES 2

typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t num_blocks;
  int64_t k_stride[3]; /* between blocks, heads, tokens */
  int64_t v_stride[3];
  int32_t heads;
  int32_t block_size;
  int32_t dim;
  int32_t dtype; /* SAI_CACHE_BF16 or SAI_CACHE_E4M3 */
} sai_kv_cache;

/*
 * sai_append_kv -- rotate the rows' keys (and queries) by their positions and
 * write keys and values into the cache.
 *
 * With p = seq_lens[i] - 1 and c_j, s_j = cos_sin[p*rot_dim + j],
 * cos_sin[p*rot_dim + rot_dim/2 + j], each head of k (and of q) becomes, for
 * the pairs (x1, x2) = (x[j], x[j + rot_dim/2]), or (x[2j], x[2j+1]) when
 * interleaved, j < rot_dim/2:
 *   (x1*c_j - x2*s_j, x2*c_j + x1*s_j)
 * and the dims at rot_dim and above stay. Products and sums are single fp32
 * operations. A bf16 cache takes the result rounded to nearest.
 *
 * An e4m3 cache takes round(x / s) with the block's scale s, a power of two:
 * need = the least 2^e, e >= -64, with |x| <= 448 * 2^e for every finite x
 * that the call puts into this block and head; s = need when the call writes
 * the block's first cell, else max(old scale, need), and then the codes of the
 * cells before the call's first one are rounded to the new scale (exact
 * but for values that become subnormal). An old scale that is no power of two
 * and stays is applied as x * (1 / s) in fp32. Infinities saturate, NaN stays NaN.
 *
 * k, v        bf16 [rows, heads, dim]; heads and dims contiguous, the stride
 *             between rows given in elements (a slice of a fused projection).
 *             16-byte aligned, strides multiples of 8 elements.
 * q, out_q    bf16 [rows, q_heads, dim] like k, and the rotated queries
 *             (contiguous; zeros for padding rows), or both NULL.
 * cos_sin     fp32 [max_pos, rot_dim], 16-byte aligned, or NULL with
 *             rot_dim = 0: no rotation, and max_pos is a bound of the positions
 *             alone (0: none). rot_dim is a multiple of 16 up to dim.
 * The rows of one request that meet in one block are neighbours in the order
 * of their positions, without gaps (a decode row by itself, or a packed
 * chunk). A row with a length below 0 or above bt_stride*block_size or
 * max_pos, or with a request outside [0, bt_rows), sets status
 * bit 1 and is skipped; a block id outside [0, num_blocks) sets bit 4 and its
 * rows are skipped.
 */
int sai_append_kv(const sai_kv_cache* cache, const uint16_t* k, int64_t k_row_stride, const uint16_t* v,
                  int64_t v_row_stride, const uint16_t* q, int64_t q_row_stride, int32_t q_heads, uint16_t* out_q,
                  const float* cos_sin, int64_t max_pos, int32_t rot_dim, int32_t interleaved,
                  const int32_t* block_table, int64_t bt_rows, int64_t bt_stride, const int32_t* row_to_batch,
                  const int32_t* seq_lens, int64_t rows, sai_stream_t stream);

/*
 * sai_paged_attention -- softmax attention of each row over its request's keys.
 *
 * Row i with n = seq_lens[i] sees key t when t < n and (window = 0, or
 * t >= n - window, or t < sinks). For query head a, which reads kv head
 * a / (q_heads / heads):
 *   out[i, a] = sum_t e_t v_t / sum_t e_t,  e_t = exp(sm_scale * q[i, a].k_t)
 *   out_lse[i, a] = log sum_t e_t
 * with fp32 sums. A row that sees no key (or only keys of score -inf), and a
 * bad row (status bit 1), gets zeros and -inf. What an unseen cell holds, NaN included, does not matter.
 * Keys on a block id outside [0, num_blocks) are not seen and set bit 4.
 *
 * q           bf16 [rows, q_heads, dim], row stride in elements as above.
 * max_seq_len host-side bound of seq_lens (longer rows are bad rows, and rows
 *             above 2^31 - 8192 keys).
 * packed      0: each row by itself (decode; its keys are split over CTAs).
 *             1: neighbouring rows mostly share a request and have
 *             neighbouring lengths (prefill): they are taken as tiles where
 *             the sizes make that faster, which needs row_to_batch.
 *             SAI_PACKED_TILES: as tiles whatever the sizes (not with more
 *             than 128 query heads to a kv head or sm_scale <= 0).
 *             Any rows give right results in every case.
 * out         bf16 [rows, q_heads, dim], not overlapping q; out_lse fp32
 *             [rows, q_heads] or NULL.
 * workspace   sai_paged_attention_workspace(...) bytes (same arguments, same
 *             device), 16-byte aligned; NULL when that is 0. Calls that share
 *             a workspace must not overlap on the GPU.
 */
size_t sai_paged_attention_workspace(int64_t rows, int32_t q_heads, int32_t heads, int32_t dim, int32_t dtype,
                                     int32_t max_seq_len, int32_t window, int32_t sinks, int32_t packed);
int sai_paged_attention(const uint16_t* q, int64_t q_row_stride, int32_t q_heads, const sai_kv_cache* cache,
                        const int32_t* block_table, int64_t bt_rows, int64_t bt_stride, const int32_t* row_to_batch,
                        const int32_t* seq_lens, int64_t rows, int32_t max_seq_len, int32_t window, int32_t sinks,
                        float sm_scale, int32_t packed, uint16_t* out, float* out_lse, void* workspace,
                        size_t workspace_bytes, sai_stream_t stream);

/*
 * sai_sparse_attention -- the same attention over chosen slots: row i sees
 * the slots[i*slots_stride + j], j < k, that are >= 0 (the out_slots of
 * sai_topk_transform or sai_index_score_topk with block_size pages; a slot
 * named twice counts twice). Slots at or above num_blocks*block_size are not
 * seen and set bit 4. 1 <= k <= 65536.
 */
size_t sai_sparse_attention_workspace(int64_t rows, int32_t q_heads, int32_t heads, int32_t dim, int32_t dtype,
                                      int32_t k);
int sai_sparse_attention(const uint16_t* q, int64_t q_row_stride, int32_t q_heads, const sai_kv_cache* cache,
                         const int32_t* slots, int64_t slots_stride, int32_t k, int64_t rows, float sm_scale,
                         uint16_t* out, float* out_lse, void* workspace, size_t workspace_bytes,
                         sai_stream_t stream);

/*
 * sai_paged_attention_mod, sai_sparse_attention_mod -- the same attentions with
 * scores changed before the softmax, and masks by document and by prefix.
 *
 * With x = sm_scale * q[i, a].k_t, n = seq_lens[i]:
 *   softcap > 0:   x becomes softcap * tanh(x / softcap)
 *   slopes:        then x becomes x - slopes[a] * |n - 1 - t|
 *   row_starts:    row i sees no key t < row_starts[i] (its document's first
 *                  token); its `sinks` are the first tokens from there on
 *   prefix_lens:   row i also sees the keys t < prefix_lens[i] at and behind its
 *                  own position (not before its start or its window)
 * so that row i, n > 0, with b = row_starts[i] and e = max(n, prefix_lens[i]),
 * sees b <= t < e with (window = 0, or t >= n - window, or t < b + sinks); a
 * start at or past e leaves it none. The changed scores are fp32; a capped one is
 * off by at most 2^-20 of itself (2^-22 of the cap beyond it). Slopes are finite,
 * and so are their products with distances.
 *
 * softcap      0: none; else in [1e-30, 1e30].
 * slopes       fp32 [q_heads] or NULL; row_starts, prefix_lens int32 [rows] or
 *              NULL. A start or prefix outside [0, max_seq_len] makes a bad row,
 *              as does a prefix past the table's columns.
 * sai_sparse_attention_mod takes softcap alone (SAI_ERR_UNSUPPORTED otherwise:
 * slots have no positions). mod = NULL or all unset: the plain call. Workspaces
 * are those of the plain calls; with prefix_lens that of window = 0, so that long
 * prefixes are split over CTAs (that of the window itself is taken too, for rows
 * split as the window alone would be).
 */
typedef struct {
  float softcap;
  const float* slopes;
  const int32_t* row_starts;
  const int32_t* prefix_lens;
} sai_score_mod;

int sai_paged_attention_mod(const uint16_t* q, int64_t q_row_stride, int32_t q_heads, const sai_kv_cache* cache,
                            const int32_t* block_table, int64_t bt_rows, int64_t bt_stride, const int32_t* row_to_batch,
                            const int32_t* seq_lens, int64_t rows, int32_t max_seq_len, int32_t window, int32_t sinks,
                            float sm_scale, int32_t packed, const sai_score_mod* mod, uint16_t* out, float* out_lse,
                            void* workspace, size_t workspace_bytes, sai_stream_t stream);
int sai_sparse_attention_mod(const uint16_t* q, int64_t q_row_stride, int32_t q_heads, const sai_kv_cache* cache,
                             const int32_t* slots, int64_t slots_stride, int32_t k, int64_t rows, float sm_scale,
                             const sai_score_mod* mod, uint16_t* out, float* out_lse, void* workspace,
                             size_t workspace_bytes, sai_stream_t stream);

/*
 * Pages of the caches: copying, forking, growing and ending requests, compacting.
 *
 * A pool of num_blocks pages (the blocks of the caches) is shared by all layers:
 * page p is block p of every array of the pool. refs[p] (int32) counts the
 * requests whose table names page p, and whoever else holds it (a prompt store);
 * 0 or below: free. Request r holds the first ceil(seq_lens[r] / block_size)
 * entries of row r of block_table ([requests, width], rows bt_stride elements
 * apart), here one row and one length for each request, not for each query row.
 * The calls below read tables, lengths and counts on the device, decide there
 * and write new ones; nothing comes back to the host. Which page is taken
 * depends on the counts alone (the lowest free pages, in the order of requests),
 * so equal states give equal tables.
 *
 * sai_page_array describes one array of the pool: page p is count[0] x count[1]
 * rows of row_bytes contiguous bytes, stride[] apart, at base + p * page_stride
 * (all in bytes, multiples of 4). cells names the axis (0 or 1) that counts the
 * page's tokens, so that a partly filled page may be copied in part; -1: it is
 * copied whole. A page has at most 2^24 - 1024 units of 16 bytes (of 4 where
 * an address, stride or row is no multiple of 16). sai_cache_page_arrays writes
 * the arrays of a cache (k, v, and for e4m3 k_scale, v_scale) to out[4] and
 * returns how many they are, or an error below 0. Pages of one array must not overlap.
 */
typedef struct {
  void* base;
  int64_t page_stride;
  int64_t stride[2];
  int32_t count[2];
  int32_t row_bytes;
  int32_t cells;
} sai_page_array;

int sai_cache_page_arrays(const sai_kv_cache* cache, sai_page_array* out);

/*
 * sai_copy_pages -- page dst[i] becomes a copy of page src[i] in every array,
 * i < pairs. A pair with an id below 0 or with src[i] = dst[i] is left out, one
 * with an id at or above num_blocks too, and sets status bit 4. A page may be a
 * source more than once; a page that is the target of two pairs, or a source and
 * a target, ends up with a mixture. arrays is a HOST array of descriptors.
 */
int sai_copy_pages(const sai_page_array* arrays, int32_t num_arrays, int64_t num_blocks, const int32_t* src,
                   const int32_t* dst, int64_t pairs, sai_stream_t stream);

/*
 * sai_fork_pages -- request i of the new batch, i < children, continues request
 * parents[i] of the old one (-1: none), sharing all its pages:
 *   out_table[i, :] = block_table[parents[i], :] (-1: every entry -1)
 *   out_lens[i] = seq_lens[parents[i]] (-1: 0)
 *   out_refs[p] = refs[p] + sum over the old requests that hold p of
 *                 (number of their children - 1)
 * so that old requests without a child are freed. No page is copied: a shared
 * last page is, by sai_resize_pages, when one of its requests grows.
 * A parent outside [-1, requests) sets status bit 1 and counts as -1; an old
 * request with a length outside [0, width * block_size] sets bit 1 and counts as
 * one of length 0 without children. A held id outside [0, num_blocks) sets bit 4
 * and is not counted. out_refs may be refs; out_table and out_lens are memory of
 * their own.
 */
int sai_fork_pages(const int32_t* block_table, int64_t requests, int64_t width, int64_t bt_stride,
                   const int32_t* seq_lens, int32_t block_size, const int32_t* refs, int64_t num_blocks,
                   const int32_t* parents, int64_t children, int32_t* out_table, int64_t out_stride, int32_t* out_lens,
                   int32_t* out_refs, sai_stream_t stream);

/*
 * sai_resize_pages -- every request r gets the pages that new_lens[r] tokens
 * need (to be called before sai_append_kv), or gives back those that it does
 * not need any more (0: all of them).
 *
 * Growing: with a last page that is partly filled and has refs above 1, the
 * request first gets a page of its own with a copy of the filled cells (arrays
 * without a cells axis: of the whole page), unless it is the last of as
 * many growing requests as refs counts, all with this last page: that one keeps
 * it. Then come the pages for the new tokens. New pages are free ones, lowest id
 * first, request by request, the copy before the others; their refs become 1.
 * Shrinking: entries from ceil(new_lens / block_size) on become -1 and their refs
 * one less. Pages that the call frees are not given out by it.
 *
 * A request is served when the pages wanted by it and by all before it are
 * there (and always when it wants none); one that is not keeps table, length
 * and pages, and sets status bit 8. out_lens[r] is new_lens[r] where served,
 * else seq_lens[r]. A length outside [0, width * block_size] sets bit 1, a last
 * page outside [0, num_blocks) bit 4: the request is left as it is. out_table,
 * out_lens and out_refs may be the inputs themselves (not partly overlap them).
 * workspace: sai_resize_pages_workspace(...) bytes, 16-byte aligned; calls that
 * share it must not overlap on the GPU.
 */
size_t sai_resize_pages_workspace(int64_t num_blocks, int64_t requests);
int sai_resize_pages(const sai_page_array* arrays, int32_t num_arrays, int64_t num_blocks, int32_t block_size,
                     const int32_t* block_table, int64_t requests, int64_t width, int64_t bt_stride,
                     const int32_t* seq_lens, const int32_t* new_lens, const int32_t* refs, int32_t* out_table,
                     int64_t out_stride, int32_t* out_lens, int32_t* out_refs, void* workspace, size_t workspace_bytes,
                     sai_stream_t stream);

/*
 * sai_compact_pages -- brings the H pages with refs above 0 to the ids [0, H):
 * those at H and above move, in ascending order, to the free ids below H, in
 * ascending order; the others stay. out_moves[p] is page p's new id (-1: free),
 * for whatever else names pages; out_refs moves along; the entries that requests
 * hold are renamed in out_table (the others stay as they are). A length outside
 * [0, width * block_size] sets status bit 1 and its row stays; a held id outside
 * [0, num_blocks) sets bit 4 and stays; one of a free page sets bit 4 and becomes
 * -1. out_table and out_refs may be the inputs. workspace as above.
 */
size_t sai_compact_pages_workspace(int64_t num_blocks);
int sai_compact_pages(const sai_page_array* arrays, int32_t num_arrays, int64_t num_blocks, int32_t block_size,
                      const int32_t* block_table, int64_t requests, int64_t width, int64_t bt_stride,
                      const int32_t* seq_lens, const int32_t* refs, int32_t* out_table, int64_t out_stride,
                      int32_t* out_refs, int32_t* out_moves, void* workspace, size_t workspace_bytes,
                      sai_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SAI_H_ */
