// C-ABI layer of the caches and the attention over them: argument checks,
// plans, launches on the caller's stream. See include/sai.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/sai.h"
#include "sai_internal.h"

namespace {

using sai::cuda_status;
using sai::device_setup;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Checks a cache descriptor; fills the kernels' view of it.
int check_cache(const sai_kv_cache* c, sai::CacheView* out) {
  if (!c) return SAI_ERR_NULL;
  if (c->dtype != SAI_CACHE_BF16 && c->dtype != SAI_CACHE_E4M3) return SAI_ERR_UNSUPPORTED;
  if (c->dim != 64 && c->dim != 128) return SAI_ERR_UNSUPPORTED;
  int log2 = 4;
  while (log2 < 7 && (1 << log2) != c->block_size) ++log2;
  if ((1 << log2) != c->block_size) return SAI_ERR_UNSUPPORTED;
  if (c->heads < 1 || c->num_blocks < 1 || c->num_blocks > INT_MAX / c->block_size) return SAI_ERR_SHAPE;
  const bool f8 = c->dtype == SAI_CACHE_E4M3;
  if (!c->k || !c->v || (f8 && (!c->k_scale || !c->v_scale))) return SAI_ERR_NULL;
  const int elem = f8 ? 1 : 2;
  for (int i = 0; i < 3; ++i) {
    // the stride of an axis of one means nothing; the tensor maps want a valid one
    const bool one = i == 0 ? c->num_blocks == 1 : i == 1 && c->heads == 1;
    if (c->k_stride[i] < 0 || c->v_stride[i] < 0) return SAI_ERR_SHAPE;
    out->kst[i] = one ? 16 : c->k_stride[i] * elem;
    out->vst[i] = one ? 16 : c->v_stride[i] * elem;
    if (out->kst[i] % 16 || out->vst[i] % 16) return SAI_ERR_ALIGN;
  }
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || (f8 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))))
    return SAI_ERR_ALIGN;
  out->k = static_cast<char*>(c->k);
  out->v = static_cast<char*>(c->v);
  out->ks = f8 ? c->k_scale : nullptr;
  out->vs = f8 ? c->v_scale : nullptr;
  out->num_blocks = c->num_blocks;
  out->heads = c->heads;
  out->bs_log2 = log2;
  out->dim = c->dim;
  out->f8 = f8;
  return SAI_OK;
}

// The changes of scores and masks; NULL or nothing set: none.
int check_mod(const sai_score_mod* mod, bool slots, sai::AttnLaunch* p) {
  if (!mod) return SAI_OK;
  if (!std::isfinite(mod->softcap) || mod->softcap < 0.f) return SAI_ERR_SHAPE;
  // 1 / cap and what is capped stay normal numbers
  if (mod->softcap != 0.f && (mod->softcap < 1e-30f || mod->softcap > 1e30f)) return SAI_ERR_SHAPE;
  if (slots && (mod->slopes || mod->row_starts || mod->prefix_lens)) return SAI_ERR_UNSUPPORTED;
  if (!aligned(mod->slopes, 4) || !aligned(mod->row_starts, 4) || !aligned(mod->prefix_lens, 4)) return SAI_ERR_ALIGN;
  p->cap_log2 = mod->softcap * 1.44269504088896340736f;
  p->slopes = mod->slopes;
  p->row_starts = mod->row_starts;
  p->prefix_lens = mod->prefix_lens;
  p->modified = mod->softcap > 0.f || mod->slopes || mod->row_starts || mod->prefix_lens;
  return SAI_OK;
}

int check_table(const int32_t* block_table, int64_t bt_rows, int64_t bt_stride, const int32_t* row_to_batch,
                const int32_t* seq_lens, int64_t rows) {
  if (!block_table || !seq_lens) return SAI_ERR_NULL;
  if (bt_rows < 1 || bt_stride < 1) return SAI_ERR_SHAPE;
  if (!row_to_batch && bt_rows < rows) return SAI_ERR_SHAPE;
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || (row_to_batch && !aligned(row_to_batch, 4)))
    return SAI_ERR_ALIGN;
  return SAI_OK;
}

// Rows of `heads` heads of `dim` bf16 values, `stride` elements apart.
int check_rows(const void* x, int64_t stride, int64_t heads, int64_t dim) {
  if (!x) return SAI_ERR_NULL;
  if (stride < heads * dim) return SAI_ERR_SHAPE;
  if (!aligned(x, 16) || stride % 8) return SAI_ERR_ALIGN;
  return SAI_OK;
}

int check_attention(const uint16_t* q, int64_t q_row_stride, int32_t q_heads, const sai::CacheView& c, int64_t rows,
                    float sm_scale, uint16_t* out, float* out_lse) {
  if (q_heads < 1 || q_heads % c.heads || q_heads > 65536) return SAI_ERR_SHAPE;
  if (!std::isfinite(sm_scale)) return SAI_ERR_SHAPE;
  if (rows == 0) return SAI_OK;
  int e = check_rows(q, q_row_stride, q_heads, c.dim);
  if (e != SAI_OK) return e;
  if (!out) return SAI_ERR_NULL;
  if (!aligned(out, 16) || (out_lse && !aligned(out_lse, 4))) return SAI_ERR_ALIGN;
  return SAI_OK;
}

// Longest row of paged_attention: the kernels step past a row's end by up to 64
// chunks of 64 keys in 32 bits.
constexpr int kMostLen = INT_MAX - 8191;

long long most_keys(int32_t max_seq_len, int32_t window, int32_t sinks) {
  if (window <= 0) return max_seq_len;
  return std::min<long long>(max_seq_len, static_cast<long long>(window) + sinks);
}

bool space(const void* workspace, size_t bytes, size_t need) {
  return need == 0 || (workspace && bytes >= need && aligned(workspace, 16));
}

// Whether a call's rows are taken as tiles: packed 1 by sizes, 2 wherever they can be.
bool as_tiles(int32_t packed, int64_t rows, int32_t q_heads, int32_t heads, int32_t dim, bool f8, long long keys, int sms,
              float scale_log2) {
  if (!packed || !sai::attn_tiles_apply(q_heads / heads, scale_log2)) return false;
  return packed == SAI_PACKED_TILES || sai::attn_tiles_pay(rows, q_heads, heads, dim, f8, keys, sms);
}

// Enough for either kernel: the tile kernel leaves calls with sm_scale <= 0 to the row kernel.
size_t paged_workspace(int64_t rows, int32_t q_heads, int32_t heads, int32_t dim, bool f8, long long keys, int32_t packed,
                       int sms) {
  size_t bytes = sai::attn_rows_plan(rows, q_heads, heads, dim, f8, keys, sms).workspace_bytes;
  if (as_tiles(packed, rows, q_heads, heads, dim, f8, keys, sms, 1.f))
    bytes = std::max(bytes, sai::attn_tiles_workspace(rows, q_heads, heads, dim, keys, sms));
  return bytes;
}

// Splits rows over key chunks and launches the row kernel.
int run_rows(sai::AttnLaunch& p, long long max_keys, void* workspace, size_t workspace_bytes, int sms,
             sai_stream_t stream, bool even_out = true) {
  const sai::AttnPlan plan = sai::attn_rows_plan(p.rows, p.q_heads, p.c.heads, p.c.dim, p.c.f8, max_keys, sms, even_out);
  if (!space(workspace, workspace_bytes, plan.workspace_bytes)) return SAI_ERR_WORKSPACE;
  p.chunks = plan.chunks;
  p.own = plan.own;
  p.clustered = plan.clustered;
  if (plan.workspace_bytes) {
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<size_t>(p.rows) * p.q_heads * plan.chunks * p.c.dim);
  }
  const long long units = static_cast<long long>(p.rows) * p.c.heads * ((p.group + 15) / 16) * plan.chunks;
  if (units > INT_MAX || static_cast<long long>(p.rows) * p.q_heads > INT_MAX) return SAI_ERR_SHAPE;
  return cuda_status(sai::launch_attn_rows(p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int sai_append_kv(const sai_kv_cache* cache, const uint16_t* k, int64_t k_row_stride, const uint16_t* v,
                  int64_t v_row_stride, const uint16_t* q, int64_t q_row_stride, int32_t q_heads, uint16_t* out_q,
                  const float* cos_sin, int64_t max_pos, int32_t rot_dim, int32_t interleaved,
                  const int32_t* block_table, int64_t bt_rows, int64_t bt_stride, const int32_t* row_to_batch,
                  const int32_t* seq_lens, int64_t rows, sai_stream_t stream) {
  sai::AppendLaunch p{};
  int e = check_cache(cache, &p.c);
  if (e != SAI_OK) return e;
  if (rows < 0 || rows > INT_MAX / 16) return SAI_ERR_SHAPE;
  if (rot_dim < 0 || rot_dim > p.c.dim || rot_dim % 16) return SAI_ERR_UNSUPPORTED;
  if ((rot_dim > 0) != (cos_sin != nullptr)) return SAI_ERR_NULL;
  if (cos_sin && max_pos < 1) return SAI_ERR_SHAPE;
  if ((q != nullptr) != (out_q != nullptr)) return SAI_ERR_NULL;
  if (q && q_heads < 1) return SAI_ERR_SHAPE;
  if (rows == 0) return SAI_OK;
  if ((e = check_rows(k, k_row_stride, p.c.heads, p.c.dim)) != SAI_OK) return e;
  if ((e = check_rows(v, v_row_stride, p.c.heads, p.c.dim)) != SAI_OK) return e;
  if (q && (e = check_rows(q, q_row_stride, q_heads, p.c.dim)) != SAI_OK) return e;
  if ((e = check_table(block_table, bt_rows, bt_stride, row_to_batch, seq_lens, rows)) != SAI_OK) return e;
  if ((cos_sin && !aligned(cos_sin, 16)) || (out_q && !aligned(out_q, 16))) return SAI_ERR_ALIGN;
  int dev, sms;
  if (!device_setup(&dev, &p.status, &sms)) return SAI_ERR_CUDA;
  p.k = k;
  p.v = v;
  p.q = q;
  p.out_q = out_q;
  p.k_row = k_row_stride;
  p.v_row = v_row_stride;
  p.q_row = q_row_stride;
  p.q_heads = q ? q_heads : 0;
  p.cos_sin = cos_sin;
  p.max_pos = cos_sin || max_pos > 0 ? max_pos : INT64_MAX;
  p.rot = rot_dim;
  p.interleaved = interleaved != 0;
  p.block_table = block_table;
  p.bt_rows = bt_rows;
  p.bt_stride = bt_stride;
  p.row_to_batch = row_to_batch;
  p.seq_lens = seq_lens;
  p.rows = static_cast<int>(rows);
  return cuda_status(sai::launch_append_kv(p, reinterpret_cast<cudaStream_t>(stream)));
}

size_t sai_paged_attention_workspace(int64_t rows, int32_t q_heads, int32_t heads, int32_t dim, int32_t dtype,
                                     int32_t max_seq_len, int32_t window, int32_t sinks, int32_t packed) {
  if (rows <= 0 || heads < 1 || q_heads < heads || dim < 1 || max_seq_len < 0 || window < 0 || sinks < 0) return 0;
  int dev, sms;
  int* st;
  if (!device_setup(&dev, &st, &sms)) return 0;
  return paged_workspace(rows, q_heads, heads, dim, dtype == SAI_CACHE_E4M3, most_keys(max_seq_len, window, sinks), packed, sms);
}

int sai_paged_attention(const uint16_t* q, int64_t q_row_stride, int32_t q_heads, const sai_kv_cache* cache,
                        const int32_t* block_table, int64_t bt_rows, int64_t bt_stride, const int32_t* row_to_batch,
                        const int32_t* seq_lens, int64_t rows, int32_t max_seq_len, int32_t window, int32_t sinks,
                        float sm_scale, int32_t packed, uint16_t* out, float* out_lse, void* workspace,
                        size_t workspace_bytes, sai_stream_t stream) {
  return sai_paged_attention_mod(q, q_row_stride, q_heads, cache, block_table, bt_rows, bt_stride, row_to_batch, seq_lens,
                                 rows, max_seq_len, window, sinks, sm_scale, packed, nullptr, out, out_lse, workspace,
                                 workspace_bytes, stream);
}

int sai_paged_attention_mod(const uint16_t* q, int64_t q_row_stride, int32_t q_heads, const sai_kv_cache* cache,
                            const int32_t* block_table, int64_t bt_rows, int64_t bt_stride, const int32_t* row_to_batch,
                            const int32_t* seq_lens, int64_t rows, int32_t max_seq_len, int32_t window, int32_t sinks,
                            float sm_scale, int32_t packed, const sai_score_mod* mod, uint16_t* out, float* out_lse,
                            void* workspace, size_t workspace_bytes, sai_stream_t stream) {
  sai::AttnLaunch p{};
  int e = check_cache(cache, &p.c);
  if (e != SAI_OK) return e;
  if ((e = check_mod(mod, false, &p)) != SAI_OK) return e;
  if (rows < 0 || rows > INT_MAX / 16 || max_seq_len < 0 || window < 0 || sinks < 0) return SAI_ERR_SHAPE;
  if ((e = check_attention(q, q_row_stride, q_heads, p.c, rows, sm_scale, out, out_lse)) != SAI_OK) return e;
  if (rows == 0) return SAI_OK;
  if ((e = check_table(block_table, bt_rows, bt_stride, row_to_batch, seq_lens, rows)) != SAI_OK) return e;
  if (packed < 0 || packed > SAI_PACKED_TILES) return SAI_ERR_UNSUPPORTED;
  if (packed && !row_to_batch) return SAI_ERR_NULL;
  int dev, sms;
  if (!device_setup(&dev, &p.status, &sms)) return SAI_ERR_CUDA;
  p.q = q;
  p.q_row = q_row_stride;
  p.q_heads = q_heads;
  p.group = q_heads / p.c.heads;
  p.block_table = block_table;
  p.bt_rows = bt_rows;
  p.bt_stride = bt_stride;
  p.row_to_batch = row_to_batch;
  p.seq_lens = seq_lens;
  p.max_len = std::min(max_seq_len, kMostLen);
  p.window = window;
  p.sinks = sinks;
  p.rows = static_cast<int>(rows);
  p.scale_log2 = sm_scale * 1.44269504088896340736f;
  p.out = out;
  p.lse = out_lse;
  // A row sees its prefix from the window's first key on, however short the window.
  // Whether rows do is not known here, so their keys are taken for long ones where they
  // leave half the GPU idle otherwise and the workspace allows it: one row of a window of 512
  // and a prefix of 30000 113 us on four chunks, 27 on 57 (a short one 8.4 and 10.3); 8 rows
  // 159 on four chunks and 163 on 57. Rows that are short after all are split as without
  // prefixes.
  const long long keys = most_keys(max_seq_len, window, sinks);
  const bool maybe_long = p.prefix_lens && keys < max_seq_len &&
                          space(workspace, workspace_bytes,
                                paged_workspace(rows, q_heads, p.c.heads, p.c.dim, p.c.f8, max_seq_len, packed, sms));
  const long long most = maybe_long ? max_seq_len : keys;
  if (as_tiles(packed, rows, q_heads, p.c.heads, p.c.dim, p.c.f8, most, sms, p.scale_log2)) {
    const long long tiled = sai::attn_tiles_fill(rows, q_heads, p.c.heads, p.c.dim, sms) ? keys : most;
    const size_t need = sai::attn_tiles_workspace(rows, q_heads, p.c.heads, p.c.dim, tiled, sms);
    if (!space(workspace, workspace_bytes, need)) return SAI_ERR_WORKSPACE;
    return cuda_status(sai::launch_attn_tiles(p, tiled, workspace, sms, reinterpret_cast<cudaStream_t>(stream)));
  }
  const sai::AttnPlan plan = sai::attn_rows_plan(rows, q_heads, p.c.heads, p.c.dim, p.c.f8, keys, sms);
  if (!maybe_long || !plan.idle) return run_rows(p, keys, workspace, workspace_bytes, sms, stream);
  p.short_keys = static_cast<int>(keys);
  p.short_chunks = plan.chunks;
  return run_rows(p, most, workspace, workspace_bytes, sms, stream, false);
}

size_t sai_sparse_attention_workspace(int64_t rows, int32_t q_heads, int32_t heads, int32_t dim, int32_t dtype,
                                      int32_t k) {
  if (rows <= 0 || heads < 1 || q_heads < heads || dim < 1 || k < 1) return 0;
  int dev, sms;
  int* st;
  if (!device_setup(&dev, &st, &sms)) return 0;
  return sai::attn_rows_plan(rows, q_heads, heads, dim, dtype == SAI_CACHE_E4M3, k, sms).workspace_bytes;
}

int sai_sparse_attention(const uint16_t* q, int64_t q_row_stride, int32_t q_heads, const sai_kv_cache* cache,
                         const int32_t* slots, int64_t slots_stride, int32_t k, int64_t rows, float sm_scale,
                         uint16_t* out, float* out_lse, void* workspace, size_t workspace_bytes,
                         sai_stream_t stream) {
  return sai_sparse_attention_mod(q, q_row_stride, q_heads, cache, slots, slots_stride, k, rows, sm_scale, nullptr, out,
                                  out_lse, workspace, workspace_bytes, stream);
}

int sai_sparse_attention_mod(const uint16_t* q, int64_t q_row_stride, int32_t q_heads, const sai_kv_cache* cache,
                             const int32_t* slots, int64_t slots_stride, int32_t k, int64_t rows, float sm_scale,
                             const sai_score_mod* mod, uint16_t* out, float* out_lse, void* workspace,
                             size_t workspace_bytes, sai_stream_t stream) {
  sai::AttnLaunch p{};
  int e = check_cache(cache, &p.c);
  if (e != SAI_OK) return e;
  if ((e = check_mod(mod, true, &p)) != SAI_OK) return e;
  if (rows < 0 || rows > INT_MAX / 16 || k < 1 || k > 65536) return SAI_ERR_SHAPE;
  if ((e = check_attention(q, q_row_stride, q_heads, p.c, rows, sm_scale, out, out_lse)) != SAI_OK) return e;
  if (rows == 0) return SAI_OK;
  if (!slots) return SAI_ERR_NULL;
  if (slots_stride < k) return SAI_ERR_SHAPE;
  if (!aligned(slots, 4)) return SAI_ERR_ALIGN;
  int dev, sms;
  if (!device_setup(&dev, &p.status, &sms)) return SAI_ERR_CUDA;
  p.q = q;
  p.q_row = q_row_stride;
  p.q_heads = q_heads;
  p.group = q_heads / p.c.heads;
  p.slots = slots;
  p.slots_stride = slots_stride;
  p.slots_k = k;
  p.rows = static_cast<int>(rows);
  p.scale_log2 = sm_scale * 1.44269504088896340736f;
  p.out = out;
  p.lse = out_lse;
  return run_rows(p, k, workspace, workspace_bytes, sms, stream);
}

}  // extern "C"
