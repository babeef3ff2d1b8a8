// C-ABI layer of the pages of a pool: argument checks, descriptors, workspace
// layouts, launches on the caller's stream. See include/sai.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "../../include/sai.h"
#include "sai_internal.h"

namespace {

using sai::cuda_status;
using sai::device_setup;

constexpr int64_t kMostPages = 1 << 28;
constexpr int32_t kMostArrays = 1 << 16;
constexpr uint32_t kMostUnits = (1u << 24) - sai::kPagePiece;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

void divisor(uint32_t d, uint32_t* m, uint8_t* sh) {
  const int s = d > 1 ? 32 - __builtin_clz(d - 1) : 0;
  *sh = static_cast<uint8_t>(s);
  *m = static_cast<uint32_t>(((1ull << (24 + s)) + d - 1) / d);
}

// Checks a descriptor and joins its axes where they are contiguous. block_size
// above 0: pages may be copied in part.
int describe(const sai_page_array& in, int32_t block_size, sai::PageArray* out) {
  if (!in.base) return SAI_ERR_NULL;
  if (in.cells < -1 || in.cells > 1 || in.row_bytes < 1 || in.page_stride < 0) return SAI_ERR_SHAPE;
  int64_t count[2], stride[2], row = in.row_bytes;
  bool wide = aligned(in.base, 16) && in.page_stride % 16 == 0 && row % 16 == 0;
  if (!aligned(in.base, 4) || in.page_stride % 4 || row % 4) return SAI_ERR_ALIGN;
  for (int i = 0; i < 2; ++i) {
    count[i] = in.count[i];
    if (count[i] < 1) return SAI_ERR_SHAPE;
    stride[i] = count[i] == 1 ? 0 : in.stride[i];
    if (count[i] > 1 && stride[i] < row) return SAI_ERR_SHAPE;
    if (stride[i] % 4) return SAI_ERR_ALIGN;
    wide = wide && stride[i] % 16 == 0;
  }
  if (block_size && in.cells >= 0 && count[in.cells] != block_size) return SAI_ERR_SHAPE;
  const int64_t unit = wide ? 16 : 4;
  if (count[0] * count[1] > kMostUnits || count[0] * count[1] * (row / unit) > kMostUnits) return SAI_ERR_SHAPE;
  int cells = block_size ? in.cells : -1;
  if (count[0] == 1 || (count[1] > 1 && stride[0] < stride[1])) {  // the wider stride outside
    std::swap(count[0], count[1]);
    std::swap(stride[0], stride[1]);
    if (cells >= 0) cells ^= 1;
  }
  int64_t cell = 0;
  if (count[1] == 1 || stride[1] == row) {
    if (cells == 1) {
      cells = 2;
      cell = row;
    }
    row *= count[1];
    count[1] = 1;
    if (count[0] == 1 || (stride[0] == row && cells != 2)) {
      if (cells == 0) {
        cells = 2;
        cell = row;
      }
      row *= count[0];
      count[0] = 1;
    }
  }
  out->base = static_cast<char*>(in.base);
  out->page_stride = in.page_stride;
  out->s0 = stride[0];
  out->s1 = stride[1];
  out->row_units = static_cast<uint32_t>(row / unit);
  out->inner = static_cast<uint32_t>(count[1]);
  out->units = static_cast<uint32_t>(count[0] * count[1]) * out->row_units;
  divisor(out->row_units, &out->m_row, &out->sh_row);
  divisor(out->inner, &out->m_inner, &out->sh_inner);
  out->wide = wide;
  out->cells = static_cast<int8_t>(cells);
  out->cell_units = static_cast<uint32_t>(cell / unit);
  return SAI_OK;
}

// block_size 0: pages are copied whole.
// Leaves the first launch's arrays in c.
int check_arrays(const sai_page_array* arrays, int32_t n, int64_t num_blocks, int32_t block_size, sai::PageCopy* c) {
  if (n < 0 || n > kMostArrays || num_blocks < 1 || num_blocks > kMostPages) return SAI_ERR_SHAPE;
  if (n && !arrays) return SAI_ERR_NULL;
  c->arrays = std::min(n, sai::kPageArrays);
  c->first[0] = 0;
  for (int32_t i = 0; i < n; ++i) {
    sai::PageArray beyond, *a = i < sai::kPageArrays ? &c->a[i] : &beyond;
    const int e = describe(arrays[i], block_size, a);
    if (e != SAI_OK) return e;
    if (i < sai::kPageArrays) c->first[i + 1] = c->first[i] + (a->units + sai::kPagePiece - 1) / sai::kPagePiece;
  }
  return SAI_OK;
}

// One launch for as many arrays as it takes: launch(first). c has the first of
// them; one launch at least.
template <typename F>
int each_arrays(sai::PageCopy& c, const sai_page_array* arrays, int32_t n, int32_t block_size, F launch) {
  int32_t i0 = 0;
  do {
    if (i0) check_arrays(arrays + i0, n - i0, 1, block_size, &c);
    const cudaError_t e = launch(i0 == 0);
    if (e != cudaSuccess) return cuda_status(e);
    i0 += sai::kPageArrays;
  } while (i0 < n);
  return SAI_OK;
}

int check_table(const int32_t* table, int64_t requests, int64_t width, int64_t stride, const int32_t* lens,
                int32_t block_size, int32_t* out, int64_t out_stride, int64_t out_rows, sai::PageTable* t) {
  if (requests < 0 || requests > INT_MAX / 16 || width < 1 || width > INT_MAX / 16 || stride < width || out_stride < width ||
      block_size < 1 || block_size > 65536)
    return SAI_ERR_SHAPE;
  if ((requests && (!table || !lens)) || (out_rows && !out)) return SAI_ERR_NULL;
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(out, 4)) return SAI_ERR_ALIGN;
  if (out == table && out_stride != stride) return SAI_ERR_SHAPE;
  *t = sai::PageTable{table, requests, width, stride, lens, out, out_stride, block_size};
  return SAI_OK;
}

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return a_bytes > 0 && b_bytes > 0 && x < y + b_bytes && y < x + a_bytes;
}
int64_t span(int64_t rows, int64_t stride, int64_t width) { return rows ? 4 * ((rows - 1) * stride + width) : 0; }
// An output that is the input, or apart from it.
bool in_place_or_apart(const void* a, const void* b, int64_t bytes) { return a == b || !overlap(a, bytes, b, bytes); }

size_t round16(size_t x) { return (x + 15) & ~static_cast<size_t>(15); }

struct Space {
  char* base;  // or null, to know the size
  size_t used = 0;
  template <typename T>
  T* take(int64_t n) {
    T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
    used += round16(static_cast<size_t>(n) * sizeof(T));
    return p;
  }
};

// Workspaces laid out at `base`; their size.
size_t lay_out(sai::ResizeLaunch* p, int64_t num_blocks, int64_t requests, char* base) {
  Space w{base};
  sai::pool_chunks(num_blocks, &p->s);
  p->s.counts = w.take<int>(p->s.chunks);
  p->s.free_list = w.take<int>(num_blocks);
  p->plan = w.take<int4>(requests);
  p->copies = w.take<int4>(requests + 1);
  p->sharers = w.take<int2>(requests > sai::kPlanShared ? num_blocks : 0);
  return w.used;
}
size_t lay_out(sai::CompactLaunch* p, int64_t num_blocks, char* base) {
  Space w{base};
  sai::pool_chunks(num_blocks, &p->s);
  p->count = w.take<int>(4);
  p->s.counts = w.take<int>(p->s.chunks);
  p->s.free_list = w.take<int>(num_blocks);
  p->s.held = w.take<uint32_t>((num_blocks + 31) / 32);
  p->src = w.take<int>(num_blocks / 2 + 1);
  p->dst = w.take<int>(num_blocks / 2 + 1);
  return w.used;
}

}  // namespace

extern "C" {

int sai_cache_page_arrays(const sai_kv_cache* c, sai_page_array* out) {
  if (!c || !out || !c->k || !c->v) return SAI_ERR_NULL;
  if (c->dtype != SAI_CACHE_BF16 && c->dtype != SAI_CACHE_E4M3) return SAI_ERR_UNSUPPORTED;
  if (c->heads < 1 || c->block_size < 1 || c->dim < 1 || c->dim > 65536) return SAI_ERR_SHAPE;
  const int elem = c->dtype == SAI_CACHE_E4M3 ? 1 : 2;
  for (int kv = 0; kv < 2; ++kv) {
    const int64_t* st = kv ? c->v_stride : c->k_stride;
    out[kv] = sai_page_array{kv ? c->v : c->k, st[0] * elem, {st[1] * elem, st[2] * elem}, {c->heads, c->block_size},
                             c->dim * elem, 1};
  }
  if (elem == 2) return 2;
  if (!c->k_scale || !c->v_scale) return SAI_ERR_NULL;
  for (int kv = 0; kv < 2; ++kv)
    out[2 + kv] = sai_page_array{kv ? c->v_scale : c->k_scale, 4LL * c->heads, {0, 0}, {1, 1}, 4 * c->heads, -1};
  return 4;
}

int sai_copy_pages(const sai_page_array* arrays, int32_t num_arrays, int64_t num_blocks, const int32_t* src,
                   const int32_t* dst, int64_t pairs, sai_stream_t stream) {
  sai::PageCopy c;
  const int e = check_arrays(arrays, num_arrays, num_blocks, 0, &c);
  if (e != SAI_OK) return e;
  if (pairs < 0 || pairs > INT_MAX) return SAI_ERR_SHAPE;
  if (pairs == 0 || num_arrays == 0) return SAI_OK;
  if (!src || !dst) return SAI_ERR_NULL;
  if (!aligned(src, 4) || !aligned(dst, 4)) return SAI_ERR_ALIGN;
  int dev, sms;
  if (!device_setup(&dev, &c.status, &sms)) return SAI_ERR_CUDA;
  c.src = src;
  c.dst = dst;
  c.count = nullptr;
  c.pairs = pairs;
  c.num_blocks = num_blocks;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return each_arrays(c, arrays, num_arrays, 0, [&](bool) { return sai::launch_page_copy(c, sms, s); });
}

int sai_fork_pages(const int32_t* block_table, int64_t requests, int64_t width, int64_t bt_stride,
                   const int32_t* seq_lens, int32_t block_size, const int32_t* refs, int64_t num_blocks,
                   const int32_t* parents, int64_t children, int32_t* out_table, int64_t out_stride, int32_t* out_lens,
                   int32_t* out_refs, sai_stream_t stream) {
  sai::ForkLaunch p{};
  int e = check_table(block_table, requests, width, bt_stride, seq_lens, block_size, out_table, out_stride, children, &p.t);
  if (e != SAI_OK) return e;
  if (children < 0 || children > INT_MAX / 16 || num_blocks < 1 || num_blocks > kMostPages) return SAI_ERR_SHAPE;
  if (!refs || !out_refs || (children && (!parents || !out_lens))) return SAI_ERR_NULL;
  if (!aligned(refs, 4) || !aligned(out_refs, 4) || !aligned(parents, 4) || !aligned(out_lens, 4)) return SAI_ERR_ALIGN;
  // rows are gathered: no output may lie over an input that is still to be read
  const int64_t tb = span(requests, bt_stride, width), ob = span(children, out_stride, width);
  if (overlap(block_table, tb, out_table, ob) || overlap(seq_lens, 4 * requests, out_lens, 4 * children) ||
      overlap(parents, 4 * children, out_lens, 4 * children) || !in_place_or_apart(refs, out_refs, 4 * num_blocks))
    return SAI_ERR_SHAPE;
  int dev, sms;
  if (!device_setup(&dev, &p.status, &sms)) return SAI_ERR_CUDA;
  p.refs = refs;
  p.out_refs = out_refs;
  p.num_blocks = num_blocks;
  p.parents = parents;
  p.children = children;
  p.out_lens = out_lens;
  return cuda_status(sai::launch_fork(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t sai_resize_pages_workspace(int64_t num_blocks, int64_t requests) {
  if (num_blocks < 1 || num_blocks > kMostPages || requests < 0 || requests > INT_MAX / 16) return 0;
  sai::ResizeLaunch p{};
  return lay_out(&p, num_blocks, requests, nullptr);
}

int sai_resize_pages(const sai_page_array* arrays, int32_t num_arrays, int64_t num_blocks, int32_t block_size,
                     const int32_t* block_table, int64_t requests, int64_t width, int64_t bt_stride,
                     const int32_t* seq_lens, const int32_t* new_lens, const int32_t* refs, int32_t* out_table,
                     int64_t out_stride, int32_t* out_lens, int32_t* out_refs, void* workspace, size_t workspace_bytes,
                     sai_stream_t stream) {
  sai::ResizeLaunch p{};
  int e = check_table(block_table, requests, width, bt_stride, seq_lens, block_size, out_table, out_stride, requests, &p.t);
  if (e != SAI_OK) return e;
  sai::PageCopy c;
  if ((e = check_arrays(arrays, num_arrays, num_blocks, block_size, &c)) != SAI_OK) return e;
  if (!refs || !out_refs || (requests && (!new_lens || !out_lens))) return SAI_ERR_NULL;
  if (!aligned(refs, 4) || !aligned(out_refs, 4) || !aligned(new_lens, 4) || !aligned(out_lens, 4)) return SAI_ERR_ALIGN;
  if ((out_table != block_table &&
       overlap(block_table, span(requests, bt_stride, width), out_table, span(requests, out_stride, width))) ||
      !in_place_or_apart(seq_lens, out_lens, 4 * requests) || !in_place_or_apart(new_lens, out_lens, 4 * requests) ||
      !in_place_or_apart(refs, out_refs, 4 * num_blocks))
    return SAI_ERR_SHAPE;
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < sai_resize_pages_workspace(num_blocks, requests))
    return SAI_ERR_WORKSPACE;
  int dev, sms;
  if (!device_setup(&dev, &p.status, &sms)) return SAI_ERR_CUDA;
  lay_out(&p, num_blocks, requests, static_cast<char*>(workspace));
  p.s.refs = refs;
  p.s.out_refs = out_refs;
  p.new_lens = new_lens;
  p.out_lens = out_lens;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if ((e = cuda_status(sai::launch_resize(p, s))) != SAI_OK || requests == 0) return e;
  c.pairs = requests;
  return each_arrays(c, arrays, num_arrays, block_size,
                     [&](bool first) { return sai::launch_resize_apply(c, p, first, sms, s); });
}

size_t sai_compact_pages_workspace(int64_t num_blocks) {
  if (num_blocks < 1 || num_blocks > kMostPages) return 0;
  sai::CompactLaunch p{};
  return lay_out(&p, num_blocks, nullptr);
}

int sai_compact_pages(const sai_page_array* arrays, int32_t num_arrays, int64_t num_blocks, int32_t block_size,
                      const int32_t* block_table, int64_t requests, int64_t width, int64_t bt_stride,
                      const int32_t* seq_lens, const int32_t* refs, int32_t* out_table, int64_t out_stride,
                      int32_t* out_refs, int32_t* out_moves, void* workspace, size_t workspace_bytes,
                      sai_stream_t stream) {
  sai::CompactLaunch p{};
  int e = check_table(block_table, requests, width, bt_stride, seq_lens, block_size, out_table, out_stride, requests, &p.t);
  if (e != SAI_OK) return e;
  sai::PageCopy c;
  if ((e = check_arrays(arrays, num_arrays, num_blocks, 0, &c)) != SAI_OK) return e;
  if (!refs || !out_refs || !out_moves) return SAI_ERR_NULL;
  if (!aligned(refs, 4) || !aligned(out_refs, 4) || !aligned(out_moves, 4)) return SAI_ERR_ALIGN;
  if ((out_table != block_table &&
       overlap(block_table, span(requests, bt_stride, width), out_table, span(requests, out_stride, width))) ||
      !in_place_or_apart(refs, out_refs, 4 * num_blocks) || overlap(refs, 4 * num_blocks, out_moves, 4 * num_blocks) ||
      overlap(out_refs, 4 * num_blocks, out_moves, 4 * num_blocks))
    return SAI_ERR_SHAPE;
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < sai_compact_pages_workspace(num_blocks))
    return SAI_ERR_WORKSPACE;
  int dev, sms;
  if (!device_setup(&dev, &p.status, &sms)) return SAI_ERR_CUDA;
  lay_out(&p, num_blocks, static_cast<char*>(workspace));
  p.s.refs = refs;
  p.s.out_refs = out_refs;
  p.moves = out_moves;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if ((e = cuda_status(sai::launch_compact(p, s))) != SAI_OK) return e;
  c.src = p.src;
  c.dst = p.dst;
  c.count = p.count;
  c.pairs = num_blocks / 2 + 1;
  c.num_blocks = num_blocks;
  c.status = p.status;
  return each_arrays(c, arrays, num_arrays, 0, [&](bool first) { return sai::launch_compact_apply(c, p, first, sms, s); });
}

}  // extern "C"
