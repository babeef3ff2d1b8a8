// Pages of a pool: copies, forks, growing and ending requests, compacting.
//
// All of it is moving bytes: a copied page is read and written once, tables and
// counts likewise, and what is decided in between is small. So the copies are
// one kernel over 16-byte units, spread over all SMs whatever the number of
// pages, and the decisions are prefix sums over the pool's counts (which pages
// are free) and over the requests (how many each wants), which make the answer
// independent of the order in which CTAs run.
//
// The decisions are phases, each of which needs the whole of the one before. What
// a small call costs is its launches, about 2 us each on the host and as much on
// the GPU, and a trip to L2 for each step of a phase. So tables are written by the
// same launch as the copies, beside them, and the phases before are one kernel
// for small calls, a cluster of eight CTAs with a barrier of the cluster between
// them; for large ones each is a kernel as wide as the GPU. Every kernel is
// launched while the one before ends, and waits for it.
//
// On the GPU, us: copy of 3 pages 2.3, of 500 pages of 24 arrays 167 (6.68 TB/s, a
// plain copy's rate); fork of 8 requests 3.3, of 512 to 600 with a pool of 131072
// pages 5.7; resize of 16 beams with their copies 8.8, of 160 requests 6.5; compact of
// 512 pages 6.2, of 4096 pages of 16 arrays 83 (72 are its bytes).
#include "sai_internal.h"
#include "sai_ptx.cuh"

#include <algorithm>
#include <climits>

namespace sai {
namespace {

// ------------------------------------------------------------------ copies
constexpr int kCopyThreads = 256;
constexpr int kCopyUnits = kPagePiece / kCopyThreads;  // of a thread, in flight at once
// CTAs of a launch for each SM: four times what fits. 500 pages of 24 arrays
// (0.56 GB) take 175 us with 32, 188 with 8 and 174 with 64; with pieces of 512 or
// 2048 units 179 to 191, with streaming loads and stores 194.
constexpr int kCopyCtas = 32;

__device__ __forceinline__ uint32_t divided(uint32_t u, uint32_t m, uint32_t sh) {
  return static_cast<uint32_t>((static_cast<unsigned long long>(u) * m) >> (24 + sh));
}

template <typename V>
__device__ __forceinline__ void copy_piece(const PageArray& a, long long src, long long dst, uint32_t u0, uint32_t cells) {
  V x[kCopyUnits];
  long long at[kCopyUnits];
#pragma unroll
  for (int i = 0; i < kCopyUnits; ++i) {
    const uint32_t u = u0 + i * kCopyThreads + threadIdx.x;
    const uint32_t row = divided(u, a.m_row, a.sh_row), o = u - row * a.row_units;
    const uint32_t outer = divided(row, a.m_inner, a.sh_inner), inner = row - outer * a.inner;
    const bool in = a.cells < 0 || (a.cells == 0 ? outer < cells : a.cells == 1 ? inner < cells : o < cells * a.cell_units);
    at[i] = u < a.units && in ? outer * a.s0 + inner * a.s1 + static_cast<long long>(o) * sizeof(V) : -1;
    if (at[i] >= 0) x[i] = *reinterpret_cast<const V*>(a.base + src * a.page_stride + at[i]);
  }
#pragma unroll
  for (int i = 0; i < kCopyUnits; ++i)
    if (at[i] >= 0) *reinterpret_cast<V*>(a.base + dst * a.page_stride + at[i]) = x[i];
}

// What a CTA copies at a time: pair, and piece of the pair's pages.
struct CopyWalk {
  long long pair;
  uint32_t piece, pieces, step_pair, step_piece;
  __device__ __forceinline__ CopyWalk(const PageCopy& c, uint32_t cta, uint32_t ctas) {
    pieces = c.first[c.arrays];
    step_pair = ctas / pieces;
    step_piece = ctas % pieces;
    pair = cta / pieces;
    piece = cta % pieces;
  }
  __device__ __forceinline__ void next() {
    pair += step_pair;
    piece += step_piece;
    if (piece >= pieces) {
      piece -= pieces;
      ++pair;
    }
  }
};

__device__ __forceinline__ void copy_page(const PageCopy& c, uint32_t piece, int src, int dst, uint32_t cells) {
  int lo = 0, hi = c.arrays - 1;  // the array with first[i] <= piece < first[i + 1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (c.first[mid] <= piece)
      lo = mid;
    else
      hi = mid - 1;
  }
  const uint32_t u0 = (piece - c.first[lo]) * kPagePiece;
  if (c.a[lo].wide)
    copy_piece<uint4>(c.a[lo], src, dst, u0, cells);
  else
    copy_piece<uint32_t>(c.a[lo], src, dst, u0, cells);
}

// The pairs of c.src and c.dst, by `ctas` CTAs of which this is number `cta`.
__device__ __forceinline__ void copy_pairs(const PageCopy& c, uint32_t cta, uint32_t ctas) {
  CopyWalk w(c, cta, ctas);
  const long long pairs = c.count ? *c.count : c.pairs;
  // there is room for c.pairs: the first pair is read along with their number
  for (bool go = w.pair < c.pairs; go; w.next(), go = w.pair < pairs) {
    const int src = c.src[w.pair], dst = c.dst[w.pair];
    if (w.pair >= pairs) return;
    if (src < 0 || dst < 0 || src == dst) continue;
    if (src < c.num_blocks && dst < c.num_blocks)
      copy_page(c, w.piece, src, dst, 0);
    else if (w.piece == 0 && threadIdx.x == 0)
      atomicOr(c.status, kDevBadPage);
  }
}

__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const __grid_constant__ PageCopy c) {
  pdl_wait();
  copy_pairs(c, blockIdx.x, gridDim.x);
}

// ------------------------------------------------------- sums over a CTA
// Exclusive prefix sum of x over the CTA and the total; every thread calls it.
template <int THREADS, typename T>
__device__ __forceinline__ T block_scan(T x, T* total) {
  __shared__ T sums[THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  if (lane == 31) sums[warp] = y;
  __syncthreads();
  T before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    before += w < warp ? sums[w] : 0;
    all += sums[w];
  }
  __syncthreads();  // sums may be written again
  *total = all;
  return before + y - x;
}

__device__ __forceinline__ long long pages_of(int len, int bs) { return (static_cast<long long>(len) + bs - 1) / bs; }
__device__ __forceinline__ bool good_len(int len, const PageTable& t) {
  return len >= 0 && len <= t.width * t.block_size;
}

// ------------------------------------------------------------ free pages
constexpr int kScanThreads = 512;
constexpr int kScanPages = 16;  // of a thread
constexpr long long kChunk = kScanThreads * kScanPages;
constexpr int kMostChunks = 512;

// One chunk: the free pages' list and number, the held pages' bits, a copy of
// the counts.
__device__ __forceinline__ void scan_chunk(const PoolScan& s, int chunk) {
  const long long c0 = chunk * s.chunk;
  int found = 0;
  for (long long base = c0; base < min(c0 + s.chunk, s.num_blocks); base += kChunk) {
    const long long p0 = base + threadIdx.x * kScanPages;
    int r[kScanPages];
    uint32_t free = 0;
    const bool whole = p0 + kScanPages <= s.num_blocks;
    if (whole && (reinterpret_cast<uintptr_t>(s.refs) & 15) == 0) {
#pragma unroll
      for (int i = 0; i < kScanPages / 4; ++i)
        *reinterpret_cast<int4*>(r + 4 * i) = *reinterpret_cast<const int4*>(s.refs + p0 + 4 * i);
    } else {
#pragma unroll
      for (int i = 0; i < kScanPages; ++i) r[i] = p0 + i < s.num_blocks ? s.refs[p0 + i] : 1;
    }
#pragma unroll
    for (int i = 0; i < kScanPages; ++i) free |= (r[i] <= 0 ? 1u : 0u) << i;
    if (s.out_refs != s.refs) {
      if (whole && (reinterpret_cast<uintptr_t>(s.out_refs) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < kScanPages / 4; ++i)
          *reinterpret_cast<int4*>(s.out_refs + p0 + 4 * i) = *reinterpret_cast<const int4*>(r + 4 * i);
      } else {
#pragma unroll
        for (int i = 0; i < kScanPages; ++i)
          if (p0 + i < s.num_blocks) s.out_refs[p0 + i] = r[i];
      }
    }
    if (s.held) {
      // pages past the end count as held in `free`, but have no bit
      const long long left = s.num_blocks - p0;
      const uint32_t here = left >= kScanPages ? 0xffffu : left <= 0 ? 0u : (1u << left) - 1u;
      const uint32_t mine = ~free & here, other = __shfl_down_sync(0xffffffffu, mine, 1);
      if ((threadIdx.x & 1) == 0 && left > 0) s.held[p0 / 32] = mine | other << 16;
    }
    int total;
    int at = found + block_scan<kScanThreads>(__popc(free), &total);
    while (free) {
      s.free_list[c0 + at++] = static_cast<int>(p0) + __ffs(free) - 1;
      free &= free - 1;
    }
    found += total;
  }
  if (threadIdx.x == 0) s.counts[chunk] = found;
}

// Free pages before each chunk, in shared memory, and their number.
template <int THREADS>
__device__ __forceinline__ int free_before(const PoolScan& s, int (&before)[kMostChunks]) {
  int sum = 0;
  if (s.chunks == 1) {
    if (threadIdx.x == 0) before[0] = 0;
    sum = s.counts[0];
    __syncthreads();
    return sum;
  }
  for (int c0 = 0; c0 < s.chunks; c0 += THREADS) {
    const int c = c0 + threadIdx.x;
    int total;
    const int x = block_scan<THREADS>(c < s.chunks ? s.counts[c] : 0, &total);
    if (c < s.chunks) before[c] = sum + x;
    sum += total;
  }
  __syncthreads();
  return sum;
}
// The k-th free page.
__device__ __forceinline__ int free_page(const PoolScan& s, const int (&before)[kMostChunks], int k) {
  int lo = 0, hi = s.chunks - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (before[mid] <= k)
      lo = mid;
    else
      hi = mid - 1;
  }
  return s.free_list[lo * s.chunk + k - before[lo]];
}

// Rows are dealt out to teams of TEAM threads: warps in a cluster, whole CTAs in
// a launch as wide as the GPU. This thread's team, how many there are in `ctas`
// CTAs, and its place in the team.
struct Team {
  int me, all, lane;
};
template <int TEAM>
__device__ __forceinline__ Team team_here(int ctas) {
  const int per = blockDim.x / TEAM;
  return Team{static_cast<int>(blockIdx.x) * per + static_cast<int>(threadIdx.x) / TEAM, ctas * per,
              static_cast<int>(threadIdx.x) % TEAM};
}
template <int TEAM>
__device__ __forceinline__ int team_sum(int x) {
  if (TEAM == 32) return __reduce_add_sync(0xffffffffu, x);
  int total;
  block_scan<TEAM>(x, &total);
  return total;
}
// End of a phase in a cluster: what its CTAs wrote is there for all of them.
__device__ __forceinline__ void phase_end() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
constexpr int kCluster = 8;

// ------------------------------------------------------------------ forks
constexpr int kForkThreads = 128;
// Entries of tables and counts, and columns, that one cluster takes: there the host
// saves 1 us by one launch less. On the GPU (called one after another), us, as a
// cluster: 1536 entries of 32 columns 3.6 (5.5), 6144 of 32 4.0 (5.9), 12288 of 64
// 4.6 (6.4), 8192 of 256 6.1 (8.3), 32768 of 512 9.4 (10.6); in two launches 3.6
// (6.9), 4.0 (7.0), 4.0 (7.0), 4.3 (7.1), 5.2 (6.8).
constexpr long long kForkSmall = 1 << 13, kForkNarrow = 64;

// The counts before the change.
__device__ __forceinline__ void fork_counts(const ForkLaunch& p) {
  if (p.out_refs != p.refs)
    for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < p.num_blocks;
         i += static_cast<long long>(gridDim.x) * blockDim.x)
      p.out_refs[i] = p.refs[i];
}

// Children's rows and lengths.
template <int TEAM>
__device__ __forceinline__ void fork_rows(const ForkLaunch& p) {
  const Team w = team_here<TEAM>(gridDim.x);
  for (long long i = w.me; i < p.children; i += w.all) {
    long long r = p.parents[i];
    const bool bad = r < -1 || r >= p.t.requests;
    const int len = bad || r < 0 ? 0 : p.t.lens[r];
    if (bad && w.lane == 0) atomicOr(p.status, kDevBadRowMeta);
    if (bad || !good_len(len, p.t)) r = -1;
#pragma unroll 4
    for (long long c = w.lane; c < p.t.width; c += TEAM)
      p.t.out[i * p.t.out_stride + c] = r < 0 ? -1 : p.t.table[r * p.t.stride + c];
    if (w.lane == 0) p.out_lens[i] = r < 0 ? 0 : len;
  }
}

// Up to so many children for each column of the table an old request's team counts
// its own by reading all parents; above, each old request gives its pages back and
// each child holds its parent's, so that the time grows with the table and not with
// the square of the requests, for two atomics a page where one child takes none. As
// many children as requests, on the GPU, us, by counting (giving back): 4096 of 48
// pages in 64 columns 11.7 (8.3), 32768 310 (42); of 700 in 1024 columns 17.5 (35)
// and 424 (553).
constexpr long long kForkCounted = 64;

// `add` to the counts of the pages of request r, of a length that is good.
__device__ __forceinline__ void hold_pages(const ForkLaunch& p, long long r, int len, int add, int lane, int team) {
  const int pages = static_cast<int>(pages_of(len, p.t.block_size));
  bool bad = false;
#pragma unroll 4
  for (int c = lane; c < pages; c += team) {
    const int page = p.t.table[r * p.t.stride + c];
    if (page < 0 || page >= p.num_blocks)
      bad = true;
    else if (add)
      atomicAdd(p.out_refs + page, add);
  }
  if (bad) atomicOr(p.status, kDevBadPage);
}

// Each old request's pages are held once for each child. WAIT: the counts are
// there after pdl_wait, which every thread calls.
template <int TEAM, bool WAIT>
__device__ __forceinline__ void fork_refs(const ForkLaunch& p) {
  const Team w = team_here<TEAM>(gridDim.x);
  if (p.children <= kForkCounted * p.t.width) {
    bool waited = !WAIT;
    for (long long r = w.me; r < p.t.requests; r += w.all) {
      const int len = p.t.lens[r];
      if (!good_len(len, p.t)) {
        if (w.lane == 0) atomicOr(p.status, kDevBadRowMeta);
        continue;
      }
      int children = 0;
#pragma unroll 4
      for (long long i = w.lane; i < p.children; i += TEAM) children += p.parents[i] == r;
      children = team_sum<TEAM>(children);
      if (!waited) pdl_wait();
      waited = true;
      hold_pages(p, r, len, children - 1, w.lane, TEAM);
    }
    if (!waited) pdl_wait();
    return;
  }
  if (WAIT) pdl_wait();
  for (long long i = w.me; i < p.t.requests + p.children; i += w.all) {
    const bool old = i < p.t.requests;
    const long long r = old ? i : p.parents[i - p.t.requests];
    if (r < 0 || r >= p.t.requests) continue;
    const int len = p.t.lens[r];
    if (good_len(len, p.t))
      hold_pages(p, r, len, old ? -1 : 1, w.lane, TEAM);
    else if (w.lane == 0)
      atomicOr(p.status, kDevBadRowMeta);
  }
}

__global__ void __launch_bounds__(kForkThreads) fork_counts_kernel(const ForkLaunch p) {
  pdl_trigger();
  fork_counts(p);
}
// The rows, and the numbers of children, do not wait for the counts. 16 CTAs an SM,
// of 32 registers a thread: with 37 the CTAs of 2048 requests take 7.0 us for
// 6.3.
__global__ void __launch_bounds__(kForkThreads, 16) fork_rows_kernel(const ForkLaunch p) {
  fork_rows<kForkThreads>(p);
  fork_refs<kForkThreads, true>(p);
}
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kScanThreads) fork_kernel(const ForkLaunch p) {
  fork_counts(p);
  fork_rows<32>(p);
  phase_end();
  fork_refs<32, false>(p);
}

// ------------------------------------------------- growing and shrinking
enum : int { kGood = 1, kCopies = 2, kKeeps = 4 };

// What each request wants, and which free pages (by number) are for it. One CTA,
// a request to a thread, in turns where there are more; those of the first turn stay
// in registers. How many share a last page, and which is the last of them: up to
// kPlanShared requests keep their pages in shared memory, and each looks at all of
// them; more are counted page by page in memory, so that the time grows with the
// requests and not with their square. Pairs on one page, all growing, a call in us,
// looking at all (counting): 128 requests 13.8 (14.4), 256 15.8 (14.4), 512 29
// (14), 2048 314 (28), 131072 1 s (1.35 ms).
__device__ __forceinline__ void plan_requests(const ResizeLaunch& p) {
  const PageTable& t = p.t;
  __shared__ int others[kPlanShared];
  struct Wish {
    int need, state, last, shared, refs;  // shared: the last page, if others hold it too, else -1
  };
  auto wish = [&](long long r) -> Wish {
    Wish w{0, 0, -1, -1, 0};
    if (r >= t.requests) return w;
    const int len = t.lens[r], want = p.new_lens[r];
    if (!good_len(len, t) || !good_len(want, t)) {
      atomicOr(p.status, kDevBadRowMeta);
      return w;
    }
    if (want > len && len % t.block_size) {
      w.last = t.table[r * t.stride + len / t.block_size];
      if (w.last < 0 || w.last >= p.s.num_blocks) {
        atomicOr(p.status, kDevBadPage);
        return w;
      }
      w.refs = p.s.refs[w.last];
      if (w.refs > 1) w.shared = w.last;
    }
    w.state = kGood | (w.shared >= 0 ? kCopies : 0);
    w.need = static_cast<int>(max(0LL, pages_of(want, t.block_size) - pages_of(len, t.block_size)));
    return w;
  };
  const bool few = t.requests <= kPlanShared;
  const Wish first = wish(threadIdx.x);
  int any = 0;
  for (long long r0 = 0; r0 < t.requests; r0 += kScanThreads) {
    const long long r = r0 + threadIdx.x;
    const Wish w = r0 == 0 ? first : wish(r);
    if (few && r < t.requests) others[r] = w.shared;
    if (!few && w.shared >= 0) p.sharers[w.shared] = make_int2(0, -1);
    any |= __syncthreads_or(w.shared >= 0);
  }
  if (!few && any) {
    for (long long r = threadIdx.x; r < t.requests; r += kScanThreads) {
      const Wish w = r < kScanThreads ? first : wish(r);
      if (w.shared < 0) continue;
      atomicAdd(&p.sharers[w.shared].x, 1);
      atomicMax(&p.sharers[w.shared].y, static_cast<int>(r));
    }
    __syncthreads();
  }
  long long upto = 0;
  int copied = 0;
  for (long long r0 = 0; r0 < t.requests; r0 += kScanThreads) {
    const long long r = r0 + threadIdx.x;
    Wish w = r0 == 0 ? first : wish(r);
    if (any) {
      int same = 0;
      bool later = false;
      if (w.shared >= 0 && few) {
#pragma unroll 8
        for (int k = 0; k < static_cast<int>(t.requests); ++k)
          if (others[k] == w.shared) {
            ++same;
            later = later || k > r;
          }
      } else if (w.shared >= 0) {
        const int2 x = __ldcg(p.sharers + w.shared);
        same = x.x;
        later = x.y > r;
      }
      if (w.shared >= 0) {
        // the last of all its holders keeps the page: those before it leave it, or it is not served either
        if (!later && same == w.refs)
          w.state = (w.state & ~kCopies) | kKeeps;
        else
          ++w.need;
      }
    }
    long long total;
    const long long before = block_scan<kScanThreads>(static_cast<long long>(w.need), &total);
    const int at = static_cast<int>(min(upto + before, 1LL << 30));  // past every pool's end
    if (r < t.requests) p.plan[r] = make_int4(at, w.need, w.state, w.last);
    upto += total;
    if (any) {
      int more;
      const bool copies = w.state & kCopies;
      const int k = copied + block_scan<kScanThreads>(copies ? 1 : 0, &more);
      if (copies) p.copies[k] = make_int4(w.last, at, w.need, t.lens[r] % t.block_size);
      copied += more;
    }
  }
  if (threadIdx.x == 0) p.copies[t.requests] = make_int4(copied, 0, 0, 0);
}

// The rows of the table, by the first `ctas` CTAs. `free` pages in all.
__device__ __forceinline__ void apply_plan(const ResizeLaunch& p, const int (&before)[kMostChunks], int free, int ctas) {
  const PageTable& t = p.t;
  for (long long r = blockIdx.x; r < t.requests; r += ctas) {
    const int4 x = p.plan[r];
    const int len = t.lens[r], want = p.new_lens[r], bs = t.block_size;
    const bool wants = x.y > 0 || (x.z & kKeeps);
    const bool served = (x.z & kGood) && (!wants || static_cast<long long>(x.x) + x.y <= free);
    const int have = static_cast<int>(pages_of(len, bs)), to = static_cast<int>(pages_of(want, bs));
    const int copies = (x.z & kCopies) ? 1 : 0;
    bool bad = false;
#pragma unroll 4
    for (long long c = threadIdx.x; c < t.width; c += kCopyThreads) {
      const int old = t.table[r * t.stride + c];
      int page = old;
      if (served) {
        if (copies && c == have - 1) {
          page = free_page(p.s, before, x.x);
          atomicAdd(p.s.out_refs + old, -1);
        } else if (c >= have && c < to) {
          page = free_page(p.s, before, x.x + copies + static_cast<int>(c) - have);
        } else if (c >= to && c < have) {
          page = -1;
          if (old < 0 || old >= p.s.num_blocks)
            bad = true;
          else
            atomicAdd(p.s.out_refs + old, -1);
        }
        if (page != old && page >= 0) p.s.out_refs[page] = 1;
      }
      if (page != old || t.out != t.table) t.out[r * t.out_stride + c] = page;
    }
    if (bad) atomicOr(p.status, kDevBadPage);
    __syncthreads();  // out_lens may be the lengths that the others read
    if (threadIdx.x == 0) {
      p.out_lens[r] = served ? want : len;
      if ((x.z & kGood) && !served) atomicOr(p.status, kDevNoPages);
    }
  }
}

__global__ void __launch_bounds__(kScanThreads) resize_plan_kernel(const ResizeLaunch p) {
  pdl_trigger();
  if (blockIdx.x == 0)
    plan_requests(p);
  else
    scan_chunk(p.s, blockIdx.x - 1);
}

// The table's rows by the first `rows_ctas` CTAs, the copies by the others.
__global__ void __launch_bounds__(kCopyThreads)
    resize_apply_kernel(const __grid_constant__ PageCopy c, const __grid_constant__ ResizeLaunch p, const int rows_ctas) {
  __shared__ int before[kMostChunks];
  pdl_wait();
  if (blockIdx.x < rows_ctas) {
    const int free = free_before<kCopyThreads>(p.s, before);
    apply_plan(p, before, free, rows_ctas);
    return;
  }
  CopyWalk w(c, blockIdx.x - rows_ctas, gridDim.x - rows_ctas);
  // the number of copies and the first one are read together (there is room for one a request)
  const int copies = p.copies[p.t.requests].x;
  int4 x = w.pair < p.t.requests ? p.copies[w.pair] : make_int4(0, 0, 0, 0);
  const int free = free_before<kCopyThreads>(p.s, before);
  while (w.pair < copies) {
    // x: page, first of the request's free pages, their number, filled cells
    if (static_cast<long long>(x.y) + x.z <= free) copy_page(c, w.piece, x.x, free_page(p.s, before, x.y), x.w);
    w.next();
    if (w.pair < copies) x = p.copies[w.pair];
  }
}

// ------------------------------------------------------------- compacting
// New ids of one chunk's held pages; the counts move, and the copies are written
// down. `held` pages in all, of which `moving` move.
__device__ __forceinline__ void move_chunk(const CompactLaunch& p, const int (&before)[kMostChunks], int held, int moving,
                                           int chunk) {
  __shared__ uint32_t word[kChunk / 32];
  __shared__ int first[kChunk / 32];  // held pages before the word's
  const PoolScan& s = p.s;
  const long long c0 = chunk * s.chunk;
  int rank = static_cast<int>(c0) - before[chunk];  // held pages before the chunk
  for (long long base = c0; base < min(c0 + s.chunk, s.num_blocks); base += kChunk) {
    const int n = static_cast<int>(min(kChunk, s.num_blocks - base));
    const uint32_t bits = threadIdx.x * 32 < n ? s.held[base / 32 + threadIdx.x] : 0u;
    int total;
    const int x = rank + block_scan<kScanThreads>(__popc(bits), &total);
    if (threadIdx.x * 32 < n) {
      word[threadIdx.x] = bits;
      first[threadIdx.x] = x;
    }
    __syncthreads();
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kScanThreads) {
      const int page = static_cast<int>(base) + i;
      const uint32_t w = word[i / 32], bit = 1u << (i & 31);
      int to = -1;
      if (w & bit) {
        to = page;
        if (page >= held) {
          const int j = first[i / 32] + __popc(w & (bit - 1)) - (held - moving);  // number among the pages that move
          to = free_page(s, before, j);
          p.src[j] = page;
          p.dst[j] = to;
          s.out_refs[to] = s.refs[page];
          s.out_refs[page] = 0;
        }
      }
      p.moves[page] = to;
    }
    rank += total;
    __syncthreads();  // the words are written again
  }
}

// How many pages are held, and how many of them move: as many as there are free
// pages below that number.
__device__ __forceinline__ int2 count_moves(const PoolScan& s, int (&before)[kMostChunks]) {
  __shared__ int below;
  const int held = static_cast<int>(s.num_blocks) - free_before<kScanThreads>(s, before);
  if (threadIdx.x == 0) below = 0;
  __syncthreads();
  const int last = held == s.num_blocks ? -1 : static_cast<int>(held / s.chunk);
  if (last >= 0) {
    int n = 0;
    for (long long w = last * s.chunk / 32 + threadIdx.x; w * 32 < held; w += kScanThreads) {
      const long long here = held - w * 32;
      n += __popc(~s.held[w] & (here >= 32 ? ~0u : (1u << here) - 1u));
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if ((threadIdx.x & 31) == 0 && n) atomicAdd(&below, n);
  }
  __syncthreads();
  return make_int2(held, last < 0 ? 0 : before[last] + below);
}

// The rows of the table, by the first `ctas` CTAs.
__device__ __forceinline__ void rename_rows(const CompactLaunch& p, int ctas) {
  const PageTable& t = p.t;
  for (long long r = blockIdx.x; r < t.requests; r += ctas) {
    const int len = t.lens[r];
    const bool good = good_len(len, t);
    if (!good && threadIdx.x == 0) atomicOr(p.status, kDevBadRowMeta);
    const long long pages = good ? pages_of(len, t.block_size) : 0;
    bool bad = false;
#pragma unroll 4
    for (long long c = threadIdx.x; c < t.width; c += kCopyThreads) {
      const int old = t.table[r * t.stride + c];
      int page = old;
      if (c < pages) {
        if (old >= 0 && old < p.s.num_blocks)
          page = p.moves[old];
        else
          bad = true;
        bad = bad || page < 0;
      }
      if (page != old || t.out != t.table) t.out[r * t.out_stride + c] = page;
    }
    if (bad) atomicOr(p.status, kDevBadPage);
  }
}

__global__ void __launch_bounds__(kScanThreads) compact_scan_kernel(const PoolScan s) {
  pdl_trigger();
  scan_chunk(s, blockIdx.x);
}
__global__ void __launch_bounds__(kScanThreads) compact_moves_kernel(const CompactLaunch p) {
  __shared__ int before[kMostChunks];
  pdl_wait();
  pdl_trigger();
  const int2 n = count_moves(p.s, before);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.count = n.y;
  move_chunk(p, before, n.x, n.y, blockIdx.x);
}
// A pool of one chunk: one CTA, whose phases end by its own barrier (64 pages 6.0
// us, 512 6.2, 2048 7.9, 8192 15.3; as a cluster 6.8, 7.4, 8.8, 17.3).
__global__ void __launch_bounds__(kScanThreads) compact_chunk_kernel(const CompactLaunch p) {
  __shared__ int before[kMostChunks];
  pdl_trigger();
  scan_chunk(p.s, 0);
  __syncthreads();
  const int2 n = count_moves(p.s, before);
  if (threadIdx.x == 0) *p.count = n.y;
  move_chunk(p, before, n.x, n.y, 0);
}
// A pool of a few chunks, as a cluster: as long on the GPU as two launches (16384
// pages 23.6 us, 65536 43.5 and 43.1), and 2 us less of the host at 16384 pages.
constexpr long long kCompactSmall = 1 << 16;
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kScanThreads) compact_kernel(const CompactLaunch p) {
  __shared__ int before[kMostChunks];
  pdl_trigger();
  for (int c = blockIdx.x; c < p.s.chunks; c += kCluster) scan_chunk(p.s, c);
  phase_end();
  const int2 n = count_moves(p.s, before);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.count = n.y;
  for (int c = blockIdx.x; c < p.s.chunks; c += kCluster) move_chunk(p, before, n.x, n.y, c);
}

// The table's rows by the first `rows_ctas` CTAs, the copies by the others.
__global__ void __launch_bounds__(kCopyThreads)
    compact_apply_kernel(const __grid_constant__ PageCopy c, const __grid_constant__ CompactLaunch p, const int rows_ctas) {
  pdl_wait();
  if (blockIdx.x < rows_ctas)
    rename_rows(p, rows_ctas);
  else
    copy_pairs(c, blockIdx.x - rows_ctas, gridDim.x - rows_ctas);
}

template <typename... P>
cudaError_t launch(void (*kernel)(P...), long long grid, int threads, bool dependent, cudaStream_t stream, const P&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// CTAs of a launch that copy; c.pairs is at least the number of pairs.
long long copy_ctas(const PageCopy& c, int num_sms) {
  return c.arrays ? std::min<long long>(static_cast<long long>(kCopyCtas) * num_sms, c.pairs * c.first[c.arrays]) : 0;
}

}  // namespace

void pool_chunks(long long num_blocks, PoolScan* s) {
  s->num_blocks = num_blocks;
  s->chunk = kChunk;
  while ((num_blocks + s->chunk - 1) / s->chunk > kMostChunks) s->chunk *= 2;
  s->chunks = static_cast<int>((num_blocks + s->chunk - 1) / s->chunk);
}

cudaError_t launch_page_copy(const PageCopy& c, int num_sms, cudaStream_t stream) {
  return launch(page_copy_kernel, copy_ctas(c, num_sms), kCopyThreads, false, stream, c);
}

cudaError_t launch_fork(const ForkLaunch& p, int num_sms, cudaStream_t stream) {
  if (p.children == 0 && p.t.requests == 0 && p.out_refs == p.refs) return cudaSuccess;
  if (p.t.width <= kForkNarrow && (p.t.requests + p.children) * p.t.width + p.num_blocks <= kForkSmall)
    return launch(fork_kernel, kCluster, kScanThreads, false, stream, p);
  const long long most = 16LL * num_sms;
  const long long copies = p.out_refs == p.refs ? 0 : std::min(most, (p.num_blocks + 4 * kForkThreads - 1) / (4 * kForkThreads));
  const long long rows = std::min(most, std::max(p.children, p.t.requests));
  const cudaError_t e = copies ? launch(fork_counts_kernel, copies, kForkThreads, false, stream, p) : cudaSuccess;
  return e == cudaSuccess && rows ? launch(fork_rows_kernel, rows, kForkThreads, copies > 0, stream, p) : e;
}

cudaError_t launch_resize(const ResizeLaunch& p, cudaStream_t stream) {
  return launch(resize_plan_kernel, 1 + p.s.chunks, kScanThreads, false, stream, p);
}
cudaError_t launch_resize_apply(const PageCopy& c, const ResizeLaunch& p, bool rows, int num_sms, cudaStream_t stream) {
  const int rows_ctas = rows ? static_cast<int>(std::min<long long>(p.t.requests, 16LL * num_sms)) : 0;
  const long long ctas = rows_ctas + copy_ctas(c, num_sms);
  return ctas ? launch(resize_apply_kernel, ctas, kCopyThreads, rows, stream, c, p, rows_ctas) : cudaSuccess;
}

cudaError_t launch_compact(const CompactLaunch& p, cudaStream_t stream) {
  if (p.s.chunks == 1) return launch(compact_chunk_kernel, 1, kScanThreads, false, stream, p);
  if (p.s.num_blocks <= kCompactSmall) return launch(compact_kernel, kCluster, kScanThreads, false, stream, p);
  const cudaError_t e = launch(compact_scan_kernel, p.s.chunks, kScanThreads, false, stream, p.s);
  return e == cudaSuccess ? launch(compact_moves_kernel, p.s.chunks, kScanThreads, true, stream, p) : e;
}
cudaError_t launch_compact_apply(const PageCopy& c, const CompactLaunch& p, bool rows, int num_sms, cudaStream_t stream) {
  const int rows_ctas = rows ? static_cast<int>(std::min<long long>(p.t.requests, 16LL * num_sms)) : 0;
  const long long ctas = rows_ctas + copy_ctas(c, num_sms);
  return ctas ? launch(compact_apply_kernel, ctas, kCopyThreads, rows, stream, c, p, rows_ctas) : cudaSuccess;
}

}  // namespace sai
