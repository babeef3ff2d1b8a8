// Internal launch interface between the C-ABI layer (sai_api.cu) and the
// kernel translation units. Not part of the public header.
#pragma once
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace sai {

// Device status bits (OR-ed into the library's device status word).
enum DevStatusBits : int {
  kDevBadRowMeta = 1,      // a row's seq_len / row_start / row_to_batch was out of range
  kDevWaitTimeout = 2,     // a pipeline wait gave up (the affected rows are undefined)
  kDevBadPage = 4,         // a block-table entry was out of range (fused path)
  kDevNoPages = 8,         // a request got no pages (resize_pages)
};

struct TopkLaunch {
  const float* scores;
  long long stride;
  int rows;
  const int* row_starts;
  const int* seq_lens;
  const int* page_tables;
  long long pt_rows, pt_stride;
  const int* row_to_batch;
  int page_size;
  int* out_slots;
  int* out_idx;
  int chunks;      // work units per row (1 = one unit per row)
  int chunk_len;   // window elements per unit when chunks > 1
  uint32_t* part_key;  // [rows*chunks, 512] when chunks > 1
  int32_t* part_idx;
  int* part_cnt;       // [rows*chunks]
  int* work;           // unit counter, zero at launch (null: fixed unit order)
  int* status;
  int block_size;      // out_blocks: per-row ascending distinct blocks of the slots
  int* out_blocks;     // [rows, 512] or null
  int* out_counts;     // [rows] or null
};

// Bytes at the start of a topk_transform workspace: the unit counter.
constexpr size_t kTopkWorkHeader = 256;

// How a topk_transform call is split; shared by the workspace query and the
// launcher so both always agree.
struct TopkPlan {
  int chunks;
  int chunk_len;
  size_t workspace_bytes;
};

TopkPlan topk_plan(long long rows, long long max_window, int num_sms);
cudaError_t launch_topk_transform(const TopkLaunch& p, int num_sms, cudaStream_t stream);

// Final merge of per-unit candidate lists (also used by the fused path).
struct MergeLaunch {
  int rows;
  int units_per_row;
  const uint32_t* part_key;
  const int32_t* part_idx;
  const int* part_cnt;
  const int* seq_lens;         // for the padding count (may be null: use candidates)
  const int* page_tables;
  long long pt_rows, pt_stride;
  const int* row_to_batch;
  int page_size;
  int* out_slots;
  int* out_idx;
  float* out_scores;           // optional: scores of the selected (fused path)
  int* status;
  int block_size;              // out_blocks: per-row ascending distinct blocks of the slots
  int* out_blocks;             // [rows, 512] or null
  int* out_counts;             // [rows] or null
};
cudaError_t launch_merge(const MergeLaunch& p, cudaStream_t stream);

// Per-row distinct blocks of top-k slots (sparse_blocks.cu).
cudaError_t launch_sparse_blocks(const int32_t* slots, int rows, int k, int block_size, int32_t* out_blocks,
                                 int32_t* out_counts, cudaStream_t stream);

struct FusedLaunch {
  const void* q;           // [rows, 64, 128] e4m3 codes or bf16
  const float* w;          // [rows, 64]
  const float* kscale;     // [num_blocks, 128], or null (scale 1; bf16 cache only)
  long long num_blocks;
  const int* block_table;  // [bt_rows, bt_stride]
  long long bt_rows, bt_stride;
  const int* row_to_batch;
  const int* seq_lens;
  int rows;
  int max_len;       // caller's bound on seq_lens (checked per row)
  int chunks;        // work units per row group
  int chunk_blocks;  // KV blocks per unit
  uint32_t* part_key;
  int32_t* part_idx;
  int* part_cnt;     // [rows * chunks]
  float* dense;      // dense modes: [rows, dense_stride] or [rows, 64, dense_stride]
  int sign_w;        // per-head mode: use sign(w_h) for w_h (same order per (row, head), comparable scales)
  long long dense_stride;
  int* status;
  int stall_unit;    // test hook: this work unit streams no key tiles (-1: none)
};
struct FusedPlan {
  int group;         // query rows per CTA (1 or 4)
  int chunks;        // KV chunks per row group
  int chunk_blocks;  // KV blocks per chunk
  size_t workspace_bytes;
};
FusedPlan fused_plan(long long rows, int max_seq_len, int group_rows, int num_sms);
// What a fused launch writes: per-(row, chunk) partial top-k lists, dense
// head-summed scores [rows, dense_stride], or dense per-head scores
// [rows, 64, dense_stride].
enum class FusedOut { kTopk, kDense, kPerHead };
cudaError_t launch_fused(const FusedLaunch& p, int group, FusedOut out, bool bf16, const void* kcache,
                         cudaStream_t stream);
// Per-(row, head) lengths and block-table rows of the per-head top-k:
// n = seq_lens[row] (0 for a row the fused kernel would reject), batch =
// row_to_batch ? row_to_batch[row] : row.
cudaError_t launch_per_head_expand(const int* seq_lens, const int* row_to_batch, int rows, int max_len,
                                   long long bt_rows, long long bt_stride, int* out_lens, int* out_batch,
                                   cudaStream_t stream);

// Per-device set-up shared by the C-ABI files (sai_api.cu): the current
// device, its status word and SM count; false when CUDA refuses.
bool device_setup(int* dev_out, int** status, int* sms);
// Map a CUDA error to a sai_status, remembering its text for sai_last_error.
int cuda_status(cudaError_t e);

// ------------------------------------------------- caches and attention
struct CacheView {
  char* k;
  char* v;
  float* ks;  // [num_blocks, heads] or null (bf16)
  float* vs;
  long long num_blocks;
  long long kst[3], vst[3];  // bytes between blocks, heads, tokens
  int heads, bs_log2, dim;
  bool f8;
};

struct AppendLaunch {
  CacheView c;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* q;  // or null
  uint16_t* out_q;
  long long k_row, v_row, q_row;  // elements between rows
  int q_heads;
  const float* cos_sin;  // [max_pos, rot] or null
  long long max_pos;
  int rot, interleaved;
  const int* block_table;
  long long bt_rows, bt_stride;
  const int* row_to_batch;
  const int* seq_lens;
  int rows;
  int* status;
};
cudaError_t launch_append_kv(const AppendLaunch& p, cudaStream_t stream);

// One attention call; the keys of a row are its request's (block_table) or
// its slots.
struct AttnLaunch {
  CacheView c;
  const uint16_t* q;
  long long q_row;
  int q_heads, group;  // group = q_heads / kv heads
  const int* block_table;
  long long bt_rows, bt_stride;
  const int* row_to_batch;
  const int* seq_lens;
  int max_len, window, sinks;
  const int* slots;  // or null
  long long slots_stride;
  int slots_k;
  int rows;
  float scale_log2;  // sm_scale * log2(e)
  uint16_t* out;
  float* lse;
  int chunks;      // row kernel: key chunks per row; > 1: partial results
  bool own, clustered;  // row kernel: see AttnPlan
  float* part_o;   // row kernel: [rows, q_heads, chunks, dim]; tile kernel: [slots, rows and heads of a unit, dim]
  float2* part_ml; // without dim: running maximum (log2 units) and sum
  int* status;
  // changed scores and masks (`modified`: any of them)
  bool modified;
  float cap_log2;          // softcap * log2(e), 0: none
  const float* slopes;     // [q_heads] or null
  const int* row_starts;   // [rows] or null
  const int* prefix_lens;  // [rows] or null
  // prefix_lens under a window: rows of up to so many keys (the window's) are split as without prefixes (-1: none)
  int short_keys = -1, short_chunks = 1;
};
// Chunks per row of the row kernel, and its partial results' bytes.
struct AttnPlan {
  int chunks;
  size_t workspace_bytes;
  bool own;        // a unit for each team of warps instead of each CTA
  bool clustered;  // a unit's chunks are a cluster and need no workspace
  bool idle;       // half of the GPU is
};
// `even_out`: long rows are cut past a full wave too, else within one.
AttnPlan attn_rows_plan(long long rows, int q_heads, int heads, int dim, bool f8, long long max_keys, int num_sms,
                        bool even_out = true);
cudaError_t launch_attn_rows(const AttnLaunch& p, cudaStream_t stream);
cudaError_t launch_attn_rows_mod(const AttnLaunch& p, cudaStream_t stream);
// The tile kernel of packed rows: whether it takes a call, whether it beats the
// row kernel on these sizes, its workspace, its launch.
bool attn_tiles_apply(int group, float scale_log2);
bool attn_tiles_pay(long long rows, int q_heads, int heads, int dim, bool f8, long long max_keys, int num_sms);
bool attn_tiles_fill(long long rows, int q_heads, int heads, int dim, int num_sms);  // a unit for every CTA (pair)
size_t attn_tiles_workspace(long long rows, int q_heads, int heads, int dim, long long max_keys, int num_sms);
cudaError_t launch_attn_tiles(const AttnLaunch& p, long long max_keys, void* workspace, int num_sms,
                              cudaStream_t stream);
cudaError_t launch_attn_tiles_mod(const AttnLaunch& p, long long max_keys, void* workspace, int num_sms,
                                  cudaStream_t stream);
cudaError_t launch_attn_tiles_cap(const AttnLaunch& p, long long max_keys, void* workspace, int num_sms,
                                  cudaStream_t stream);

// ------------------------------------------------- pages of a pool
// One array of the pool, axes joined where they are contiguous: a page is rows
// of `row_units` units (16 or 4 bytes) in an outer and an inner (`inner`) axis.
struct PageArray {
  char* base;
  long long page_stride, s0, s1;  // bytes between pages, outer rows, inner rows
  uint32_t units;                 // of a page
  uint32_t row_units, inner;
  uint32_t m_row, m_inner;        // division by them: (u * m) >> (24 + sh), for u < 2^24
  uint8_t sh_row, sh_inner;
  uint8_t wide;                   // unit of 16 bytes (else 4)
  int8_t cells;                   // the page's tokens are 0: outer, 1: inner rows, 2: cell_units of the row, -1: copied whole
  uint32_t cell_units;
};
constexpr int kPageArrays = 32;       // of one launch
constexpr uint32_t kPagePiece = 1024;  // units that a CTA copies at a time
struct PageCopy {
  PageArray a[kPageArrays];
  uint32_t first[kPageArrays + 1];  // pieces of a page before array i
  int arrays;
  const int* src;
  const int* dst;
  const int* count;     // number of pairs on the device, or null: `pairs`
  long long pairs;
  long long num_blocks;
  int* status;
};
struct PageTable {
  const int* table;
  long long requests, width, stride;
  const int* lens;
  int* out;
  long long out_stride;
  int block_size;
};
// Free pages of the pool, chunk by chunk of `chunk` pages.
struct PoolScan {
  const int* refs;
  int* out_refs;
  long long num_blocks, chunk;
  int chunks;
  int* counts;       // [chunks] free pages of each
  int* free_list;    // [num_blocks]: chunk c's from c * chunk on
  uint32_t* held;    // a bit a page: refs above 0 (compact)
};
struct ForkLaunch {
  PageTable t;
  const int* refs;
  int* out_refs;
  long long num_blocks;
  const int* parents;
  long long children;
  int* out_lens;
  int* status;
};
constexpr int kPlanShared = 128;
struct ResizeLaunch {
  PageTable t;
  PoolScan s;
  const int* new_lens;
  int* out_lens;
  int4* plan;        // [requests]: first of its free pages, their number, state, last page
  int2* sharers;     // [num_blocks], above kPlanShared requests: growing requests whose shared last page it is, last of them
  int4* copies;      // [requests + 1]: page, first of its request's free pages, their number, filled cells; last: number
  int* status;
};
struct CompactLaunch {
  PageTable t;
  PoolScan s;
  int* moves;
  int* src;  // [num_blocks / 2]
  int* dst;
  int* count;
  int* status;
};
void pool_chunks(long long num_blocks, PoolScan* s);  // fills num_blocks, chunk, chunks
cudaError_t launch_page_copy(const PageCopy& c, int num_sms, cudaStream_t stream);
cudaError_t launch_fork(const ForkLaunch& p, int num_sms, cudaStream_t stream);
// What is decided; then the table's rows (`rows`) and the copies in c's arrays.
cudaError_t launch_resize(const ResizeLaunch& p, cudaStream_t stream);
cudaError_t launch_resize_apply(const PageCopy& c, const ResizeLaunch& p, bool rows, int num_sms, cudaStream_t stream);
cudaError_t launch_compact(const CompactLaunch& p, cudaStream_t stream);
cudaError_t launch_compact_apply(const PageCopy& c, const CompactLaunch& p, bool rows, int num_sms, cudaStream_t stream);

}  // namespace sai
