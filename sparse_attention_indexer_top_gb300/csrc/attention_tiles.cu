// Tile kernel of the attention over a paged cache: packed rows (prefill).
//
// A CTA takes the query heads that share one kv head for two tiles of
// floor(128 / group) neighbouring rows, so an MMA tile is 128 (row, head)
// pairs, and walks the 128-key tiles that any of its rows sees:
//   S = Q K^T (tcgen05, fp32 in TMEM), P = 2^(scale S - m), O += P V
// with the running maximum m and sum l of each (row, head) in the registers of
// the thread that owns its TMEM lane, and P written back over S as the next
// MMA's left operand. Rows of several requests in one CTA are walked request
// by request, with the other rows masked; any lengths are right, neighbouring
// ones are fast.
//
// Bound: the tensor core (4 * dim flops per query head, row and key) together
// with the softmax's instruction issue, about equal at dim 128; the keys are
// read from HBM once per CTA and mostly hit in L2. So the two tiles take
// turns: while the softmax warps of one tile work, the tensor core runs
// the other tile's P V and its next Q K^T. In steady state the
// tensor core order is PV_A(j) QK_A(j+1) PV_B(j) QK_B(j+1); products of one
// CTA complete in order, so a tile's S(j+1) being there means its PV(j) is
// too, and O may be rescaled without another wait.
//
// Roles (12 warps): 0-3 softmax of tile A, 4-7 softmax of tile B, 8 TMA, 9
// MMA, 10-11 make the value tile safe to multiply: a weight of 0 times a
// NaN or infinity that a row must not see would still be NaN, so in tiles that
// some row sees only in part, rows of V past the request's end become 0, and
// rows with a non-finite value too; if such a row of V is seen by some query
// row, its share is added at the end from global memory.
#include <cuda.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "sai_internal.h"
#include "sai_ptx.cuh"
#include "sai_tmap.h"

namespace sai {
namespace {

constexpr int kTile = 128;       // keys of a tile, and (row, head) pairs of an MMA tile
constexpr int kMaxRows = 256;    // query rows of a CTA (group 1)
constexpr int kSoftmaxWarps = 8;
constexpr int kTmaWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kPrepWarp = 10;
constexpr int kPrepWarps = 2;
constexpr int kThreads = (kPrepWarp + kPrepWarps) * 32;
constexpr int kStages = 2;       // K and V tiles in flight each
constexpr float kLn2 = 0.69314718055994530942f;

// TMEM columns: S (and P over it) of tiles A and B, then their O.
constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;

struct TilesLaunch {
  AttnLaunch a;
  int rows_per_tile;  // floor(128 / group)
  int row_tiles;      // CTAs along the rows
};

template <int D>
struct Shared {
  static constexpr int kSlabs = D / 64;
  static constexpr int kTileBytes = kSlabs * kTile * 128;
  unsigned char q[2][kTileBytes];
  unsigned char k[kStages][kTileBytes];
  unsigned char v[kStages][kTileBytes];
  uint64_t q_full, k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], v_safe[kStages];
  uint64_t s_ready[2], p_ready[2], o_done[2];
  uint32_t tmem;
  int nonfinite;  // number of the last pass (from 1) that met a non-finite value row
  int segs;
  int warp_starts[8];
  int row_n[kMaxRows], row_b[kMaxRows];
  int seg_start[kMaxRows + 1], seg_most[kMaxRows], seg_least[kMaxRows], seg_low[kMaxRows];
};

// One request's rows of the CTA and the tiles that this CTA's chunk walks.
struct Pass {
  int s, e;        // rows [s, e) of the CTA
  int batch;
  int most, least; // longest and shortest (above 0) row
  int low;         // least first key of a row's window (0: no window)
  int first_tiles; // tiles that hold the first `sinks` tokens before the window's tiles
  int low_tile;
  int i0, i1;      // tile indices of this chunk
  bool act[2];     // MMA tile has rows of the pass
  __device__ __forceinline__ int tile0(int i) const {
    return (i < first_tiles ? i : i - first_tiles + low_tile) * kTile;
  }
  // does every row of the pass see all of the tile?
  __device__ __forceinline__ bool partial(int t0, const AttnLaunch& p) const {
    if (t0 + kTile > least) return true;
    if (p.window == 0 || t0 >= most - p.window) return false;
    return !(t0 + kTile <= p.sinks && t0 + kTile <= low);
  }
};

template <int D>
__device__ __forceinline__ Pass get_pass(const Shared<D>& S, const TilesLaunch& L, int seg, int chunk) {
  const AttnLaunch& p = L.a;
  Pass r;
  r.s = S.seg_start[seg];
  r.e = S.seg_start[seg + 1];
  r.batch = S.row_b[r.s];
  r.most = S.seg_most[seg];
  r.least = S.seg_least[seg];
  r.low = S.seg_low[seg];
  r.act[0] = r.s < L.rows_per_tile;
  r.act[1] = r.e > L.rows_per_tile;
  int tiles = 0;
  r.first_tiles = r.low_tile = 0;
  if (r.most > 0) {
    r.low_tile = r.low / kTile;
    if (r.low > 0) r.first_tiles = min((min(p.sinks, r.low) + kTile - 1) / kTile, r.low_tile);
    tiles = r.first_tiles + (r.most + kTile - 1) / kTile - r.low_tile;
  }
  r.i0 = static_cast<int>(static_cast<long long>(tiles) * chunk / p.chunks);
  r.i1 = static_cast<int>(static_cast<long long>(tiles) * (chunk + 1) / p.chunks);
  return r;
}

__device__ __forceinline__ void tma_4d(void* dst, const void* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_3d(void* dst, const void* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}
// D[tmem] (+)= A[tmem] x B[smem], 16-bit A packed two to a column.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a));
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Wait for TMEM loads whose registers pass through, so that no use of them
// is moved before the wait.
__device__ __forceinline__ void tmem_ld_wait32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}
// Shared-memory descriptor of a [keys x dim] tile used with dim as its outer
// (N) axis: rows of 64 dims in 128-byte swizzled atoms of 8 keys, atoms 1024
// bytes apart along the keys, 64-dim slabs `slab` bytes apart.
__device__ __forceinline__ uint64_t umma_desc_sw128_mnmajor(uint32_t smem_addr, uint32_t slab) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(slab >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
constexpr uint32_t kTransposeB = 1u << 16;  // instruction descriptor: B is N-major

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// Any infinity or NaN among two bf16 values?
__device__ __forceinline__ bool nonfinite2(uint32_t x) {
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}

// ------------------------------------------------------------------ softmax
// Thread of one (row, head) pair.
struct Lane {
  int row;         // row of the call
  int n, first, sinks;  // sees t < n with t >= first or t < sinks
  long long head;  // row * q_heads + head
  bool live;       // belongs to the pass
};

// Adds to o[] the values that were kept out of the product for being
// non-finite: every such key of the tiles that were checked.
template <int D>
__device__ __noinline__ void add_nonfinite(const AttnLaunch& p, const Pass& ps, int kvh, const Lane& ln, float m,
                                           float (&o)[D]) {
  const int lane = threadIdx.x & 31;
  const uint16_t* q = p.q + static_cast<long long>(ln.row) * p.q_row +
                      (ln.head - static_cast<long long>(ln.row) * p.q_heads) * D;
  for (int i = ps.i0; i < ps.i1; ++i) {
    const int t0 = ps.tile0(i);
    if (!ps.partial(t0, p)) continue;
    for (int t = t0; t < min(t0 + kTile, ps.most); ++t) {
      const int blk = p.block_table[ps.batch * p.bt_stride + (t >> p.c.bs_log2)];
      if (blk < 0 || blk >= p.c.num_blocks) continue;
      const long long off = t & ((1 << p.c.bs_log2) - 1);
      const uint32_t* v = reinterpret_cast<const uint32_t*>(p.c.v + blk * p.c.vst[0] + kvh * p.c.vst[1] + off * p.c.vst[2]);
      const uint32_t* k = reinterpret_cast<const uint32_t*>(p.c.k + blk * p.c.kst[0] + kvh * p.c.kst[1] + off * p.c.kst[2]);
      bool bad = false;
      for (int d = lane; d < D / 2; d += 32) bad = bad || nonfinite2(v[d]);
      if (!__any_sync(0xffffffffu, bad)) continue;
      if (!ln.live || t >= ln.n || (t < ln.first && t >= ln.sinks)) continue;
      float s = 0.f;
      for (int d = 0; d < D / 2; ++d) {
        const uint32_t a = reinterpret_cast<const uint32_t*>(q)[d], b = k[d];
        s = fmaf(bf16_lo(a), bf16_lo(b), fmaf(bf16_hi(a), bf16_hi(b), s));
      }
      const float w = ex2(s * p.scale_log2 - (m == -INFINITY ? 0.f : m));
#pragma unroll
      for (int d = 0; d < D / 2; ++d) {
        const uint32_t x = v[d];
        o[2 * d] = fmaf(w, bf16_lo(x), o[2 * d]);
        o[2 * d + 1] = fmaf(w, bf16_hi(x), o[2 * d + 1]);
      }
    }
  }
}

template <int D>
__device__ __forceinline__ void write_rows(const AttnLaunch& p, const Lane& ln, int chunk, float m, float l,
                                           float (&o)[D]) {
  if (!ln.live) return;
  if (p.chunks > 1) {
    float4* dst = reinterpret_cast<float4*>(p.part_o + (ln.head * p.chunks + chunk) * D);
#pragma unroll
    for (int d = 0; d < D / 4; ++d)
      dst[d] = l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                        : make_float4(o[4 * d], o[4 * d + 1], o[4 * d + 2], o[4 * d + 3]);
    p.part_ml[ln.head * p.chunks + chunk] = make_float2(m, l);
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint4* dst = reinterpret_cast<uint4*>(p.out + ln.head * D);
#pragma unroll
  for (int d = 0; d < D / 8; ++d) {
    uint4 x;
    x.x = pack_bf16(o[8 * d] * inv, o[8 * d + 1] * inv);
    x.y = pack_bf16(o[8 * d + 2] * inv, o[8 * d + 3] * inv);
    x.z = pack_bf16(o[8 * d + 4] * inv, o[8 * d + 5] * inv);
    x.w = pack_bf16(o[8 * d + 6] * inv, o[8 * d + 7] * inv);
    dst[d] = l == 0.f ? make_uint4(0, 0, 0, 0) : x;  // an unseen row's O may hold anything
  }
  if (p.lse) p.lse[ln.head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D>
__device__ __forceinline__ bool softmax_role(Shared<D>& S, const TilesLaunch& L, int x, int kvh, int chunk, int row0) {
  const AttnLaunch& p = L.a;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;
  const int r = quad * 32 + lane;  // the thread's TMEM lane
  const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t ts = S.tmem + lanes + kColS + 128 * x;
  const uint32_t to = S.tmem + lanes + kColO + 128 * x;
  const int local = x * L.rows_per_tile + r / p.group;
  const bool in_tile = r < L.rows_per_tile * p.group;
  int tiles_done = 0, passes_done = 0;
  const uint64_t scale2 = pair(p.scale_log2, p.scale_log2);

  for (int seg = 0; seg < S.segs; ++seg) {
    const Pass ps = get_pass(S, L, seg, chunk);
    if (!ps.act[x]) continue;
    Lane ln;
    ln.row = row0 + local;
    ln.live = in_tile && local >= ps.s && local < ps.e && ln.row < p.rows;
    ln.n = ln.live ? S.row_n[local] : 0;
    ln.first = p.window > 0 ? max(0, ln.n - p.window) : 0;
    ln.sinks = min(p.sinks, ln.first);
    ln.head = static_cast<long long>(ln.row) * p.q_heads + kvh * p.group + r % p.group;
    float m = -INFINITY, l = 0.f;
    if (ps.i0 == ps.i1) {
      float o[D];
#pragma unroll
      for (int d = 0; d < D; ++d) o[d] = 0.f;
      write_rows<D>(p, ln, chunk, m, l, o);
      continue;
    }
    // block ids of the tile's eight 16-key groups, read one tile ahead
    auto blocks_bad = [&](int i) -> bool {
      if (i >= ps.i1 || lane >= 8) return false;
      const int t = ps.tile0(i) + 16 * lane;
      if (t >= ps.most) return false;
      const int blk = p.block_table[ps.batch * p.bt_stride + (t >> p.c.bs_log2)];
      return blk < 0 || blk >= p.c.num_blocks;
    };
    bool bad_next = blocks_bad(ps.i0);
    for (int i = ps.i0; i < ps.i1; ++i) {
      const uint32_t bad = __ballot_sync(0xffffffffu, bad_next);
      bad_next = blocks_bad(i + 1);
      const bool ok = mbar_wait(&S.s_ready[x], tiles_done & 1);
      if (!__all_sync(0xffffffffu, ok)) return false;
      ++tiles_done;
      tc_fence_after();
      uint32_t s[kTile];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, s + 32 * c);
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld_wait32(s + 32 * c);
      const int t0 = ps.tile0(i);
      const bool whole = t0 + kTile <= ln.n && (t0 >= ln.first || t0 + kTile <= ln.sinks);
      if (!__all_sync(0xffffffffu, whole) || bad) {
        const int hi = ln.n - t0, lo = ln.first - t0, sk = ln.sinks - t0;
#pragma unroll
        for (int c = 0; c < kTile; ++c) {
          const bool see = c < hi && (c >= lo || c < sk) && !((bad >> (c / 16)) & 1);
          if (!see) s[c] = 0xff800000u;
        }
        if (bad && lane == 0) atomicOr(p.status, kDevBadPage);
      }
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) mx[c] = __uint_as_float(s[c]);
#pragma unroll
      for (int c = 4; c < kTile; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mx[e] = fmaxf(mx[e], c + 4 + e < kTile ? fmaxf(__uint_as_float(s[c + e]), __uint_as_float(s[c + 4 + e]))
                                                 : __uint_as_float(s[c + e]));
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
      // the maximum moves only when it is passed by more than 2^8: weights up
      // to 256 are as exact in bf16 as weights up to 1, and O is rarely rescaled
      const bool up = top > m + 8.f;
      if (__any_sync(0xffffffffu, up)) {
        const float f = up ? (m == -INFINITY ? 0.f : ex2(m - top)) : 1.f;
        if (up) m = top;
        l *= f;
        if (i > ps.i0) {
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(to + c, o);
            tmem_ld_wait32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(to + c, o);
          }
        }
      }
      const float base = m == -INFINITY ? 0.f : m;
      const uint64_t base2 = pair(-base, -base);
      uint64_t sum[2] = {pair(l, 0.f), pair(0.f, 0.f)};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          float a, b;
          unpair(fma2(pair(__uint_as_float(s[64 * h + c]), __uint_as_float(s[64 * h + c + 1])), scale2, base2), a, b);
          a = ex2(a);
          b = ex2(b);
          sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pair(a, b));
          // weights in bf16 (relative error 2^-9, under the output's own)
          s[32 * h + c / 2] = pack_bf16(a, b);
        }
        tmem_st32(ts + 32 * h, s + 32 * h);
      }
      float a, b;
      unpair(add2(sum[0], sum[1]), a, b);
      l = a + b;
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&S.p_ready[x]);
    }
    const bool ok = mbar_wait(&S.o_done[x], passes_done & 1);
    if (!__all_sync(0xffffffffu, ok)) return false;
    ++passes_done;
    tc_fence_after();
    float o[D];
#pragma unroll
    for (int c = 0; c < D; c += 32) tmem_ld32(to + c, reinterpret_cast<uint32_t*>(o) + c);
#pragma unroll
    for (int c = 0; c < D; c += 32) tmem_ld_wait32(reinterpret_cast<uint32_t*>(o) + c);
    tc_fence_before();
    if (*reinterpret_cast<volatile int*>(&S.nonfinite) == seg + 1) add_nonfinite<D>(p, ps, kvh, ln, m, o);
    write_rows<D>(p, ln, chunk, m, l, o);
  }
  return true;
}

// ---------------------------------------------------------------------- TMA
template <int D>
__device__ __forceinline__ bool tma_role(Shared<D>& S, const TilesLaunch& L, const CUtensorMap* qmap,
                                         const CUtensorMap* kmap, const CUtensorMap* vmap, int kvh, int chunk,
                                         int row0) {
  const AttnLaunch& p = L.a;
  const int lane = threadIdx.x & 31;
  constexpr int kSlabs = D / 64;
  if (lane == 0) {
    mbar_arrive_expect_tx(&S.q_full, 2 * kSlabs * L.rows_per_tile * p.group * 128);
    for (int x = 0; x < 2; ++x)
      for (int c = 0; c < kSlabs; ++c)
        tma_3d(S.q[x] + c * kTile * 128, qmap, 64 * c, kvh * p.group, row0 + x * L.rows_per_tile, &S.q_full);
  }
  const int bs = 1 << p.c.bs_log2;
  const int blocks = kTile >> p.c.bs_log2;  // blocks of a tile
  int done = 0;
  for (int seg = 0; seg < S.segs; ++seg) {
    const Pass ps = get_pass(S, L, seg, chunk);
    auto block_of = [&](int i) -> int {
      if (i >= ps.i1 || lane >= blocks) return -1;
      const int t = ps.tile0(i) + lane * bs;
      if (t >= ps.most) return -1;
      const int blk = p.block_table[ps.batch * p.bt_stride + (t >> p.c.bs_log2)];
      return blk >= p.c.num_blocks ? -1 : blk;
    };
    int next = block_of(ps.i0);
    for (int i = ps.i0; i < ps.i1; ++i, ++done) {
      const int blk = next;
      next = block_of(i + 1);
      const int st = done % kStages;
      const uint32_t ph = ((done / kStages) & 1) ^ 1;
      const int bytes = __popc(__ballot_sync(0xffffffffu, blk >= 0)) * bs * 128 * kSlabs;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const bool ok = mbar_wait(kv ? &S.v_empty[st] : &S.k_empty[st], ph);
        if (!__all_sync(0xffffffffu, ok)) return false;
        uint64_t* full = kv ? &S.v_full[st] : &S.k_full[st];
        if (lane == 0) mbar_arrive_expect_tx(full, bytes);
        __syncwarp();
        if (blk >= 0) {
          unsigned char* dst = (kv ? S.v[st] : S.k[st]) + lane * bs * 128;
#pragma unroll
          for (int c = 0; c < kSlabs; ++c) tma_4d(dst + c * kTile * 128, kv ? vmap : kmap, 64 * c, 0, kvh, blk, full);
        }
      }
    }
  }
  return true;
}

// ---------------------------------------------------------------------- MMA
template <int D>
__device__ __forceinline__ bool mma_role(Shared<D>& S, const TilesLaunch& L, int chunk) {
  constexpr uint32_t kIdescQk = umma_idesc_bf16(kTile, kTile);
  constexpr uint32_t kIdescPv = umma_idesc_bf16(kTile, D) | kTransposeB;
  constexpr uint32_t kSlab = kTile * 128;
  const uint32_t tmem = S.tmem;
  auto qk = [&](int x, int st) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const uint32_t off = (s / 4) * kSlab + (s % 4) * 32;
      umma_bf16(tmem + kColS + 128 * x, umma_desc_sw128_kmajor(smem_u32(S.q[x]) + off),
                umma_desc_sw128_kmajor(smem_u32(S.k[st]) + off), kIdescQk, s > 0);
    }
    umma_commit(&S.s_ready[x]);
  };
  auto pv = [&](int x, int st, bool first) {
#pragma unroll
    for (int s = 0; s < kTile / 16; ++s)
      umma_ts(tmem + kColO + 128 * x, tmem + kColS + 128 * x + 8 * s,
              umma_desc_sw128_mnmajor(smem_u32(S.v[st]) + s * 2048, kSlab), kIdescPv, !(first && s == 0));
  };
  if (!mbar_wait(&S.q_full, 0)) return false;
  int done = 0, p_done[2] = {0, 0};
  for (int seg = 0; seg < S.segs; ++seg) {
    const Pass ps = get_pass(S, L, seg, chunk);
    const int n = ps.i1 - ps.i0;
    if (n == 0) continue;
    if (!mbar_wait(&S.k_full[done % kStages], (done / kStages) & 1)) return false;
    tc_fence_after();
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (ps.act[x]) qk(x, done % kStages);
    umma_commit(&S.k_empty[done % kStages]);
    for (int i = 0; i < n; ++i, ++done) {
      const int st = done % kStages, nst = (done + 1) % kStages;
      const bool more = i + 1 < n;
      if (more && !mbar_wait(&S.k_full[nst], ((done + 1) / kStages) & 1)) return false;
      if (!mbar_wait(&S.v_safe[st], (done / kStages) & 1)) return false;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!ps.act[x]) continue;
        if (!mbar_wait(&S.p_ready[x], p_done[x] & 1)) return false;
        ++p_done[x];
        tc_fence_after();
        pv(x, st, i == 0);
        if (more)
          qk(x, nst);
        else
          umma_commit(&S.o_done[x]);
      }
      umma_commit(&S.v_empty[st]);
      if (more) umma_commit(&S.k_empty[nst]);
    }
  }
  return true;
}

// --------------------------------------------------------------------- prep
template <int D>
__device__ __forceinline__ bool prep_role(Shared<D>& S, const TilesLaunch& L, int chunk) {
  const AttnLaunch& p = L.a;
  const int tid = threadIdx.x - kPrepWarp * 32;
  int done = 0;
  for (int seg = 0; seg < S.segs; ++seg) {
    const Pass ps = get_pass(S, L, seg, chunk);
    for (int i = ps.i0; i < ps.i1; ++i, ++done) {
      const int st = done % kStages;
      const bool ok = mbar_wait(&S.v_full[st], (done / kStages) & 1);
      if (!__all_sync(0xffffffffu, ok)) return false;
      const int t0 = ps.tile0(i);
      if (ps.partial(t0, p)) {
        // 16 keys at a time, four lanes to a key row (swizzling keeps a row's
        // bytes in its row)
        const int part = tid & 3;
        for (int k0 = 0; k0 < kTile; k0 += kPrepWarps * 8) {
          const int key = k0 + (tid >> 2);
          unsigned char* at = S.v[st] + key * 128 + part * 32;
          bool zero = t0 + key >= ps.most;
          bool bad = false;
          if (!zero) {
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint4 x = *reinterpret_cast<const uint4*>(at + c * kTile * 128 + e * 16);
                bad = bad || nonfinite2(x.x) || nonfinite2(x.y) || nonfinite2(x.z) || nonfinite2(x.w);
              }
          }
          const uint32_t b = __ballot_sync(0xffffffffu, bad);
          if ((b >> (threadIdx.x & 28)) & 0xfu) {
            zero = true;
            *reinterpret_cast<volatile int*>(&S.nonfinite) = seg + 1;
          }
          if (zero) {
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                *reinterpret_cast<uint4*>(at + c * kTile * 128 + e * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();  // the MMA reads these stores through the async proxy
      }
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&S.v_safe[st]);
    }
  }
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tiles_kernel(const __grid_constant__ TilesLaunch L, const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ unsigned char raw[];
  Shared<D>& S = *reinterpret_cast<Shared<D>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const AttnLaunch& p = L.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int u = blockIdx.x;
  const int chunk = u % p.chunks;
  u /= p.chunks;
  const int kvh = u % p.c.heads;
  // the last rows first: with causal lengths they have the most keys
  const int rows_here = 2 * L.rows_per_tile;
  const int row0 = (L.row_tiles - 1 - u / p.c.heads) * rows_here;

  // ---- set-up: barriers, TMEM, the rows' lengths and the runs of one request
  if (tid == 0) {
    mbar_init(&S.q_full, 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&S.k_full[i], 1);
      mbar_init(&S.k_empty[i], 1);
      mbar_init(&S.v_full[i], 1);
      mbar_init(&S.v_empty[i], 1);
      mbar_init(&S.v_safe[i], kPrepWarps);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&S.s_ready[x], 1);
      mbar_init(&S.p_ready[x], 128);
      mbar_init(&S.o_done[x], 1);
    }
    S.nonfinite = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&S.tmem, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  int n = 0, b = -1;
  if (tid < kMaxRows) {
    const int row = row0 + tid;
    if (tid < rows_here && row < p.rows) {
      n = p.seq_lens[row];
      b = p.row_to_batch[row];
      if (n < 0 || n > p.max_len || b < 0 || b >= p.bt_rows ||
          ((static_cast<long long>(n) - 1) >> p.c.bs_log2) >= p.bt_stride) {
        atomicOr(p.status, kDevBadRowMeta);
        n = 0;
        b = -1;
      }
    }
    S.row_n[tid] = n;
    S.row_b[tid] = b;
    S.seg_most[tid] = 0;
    S.seg_least[tid] = S.seg_low[tid] = INT_MAX;
  }
  __syncthreads();
  bool start = false;
  uint32_t starts = 0;
  if (tid < kMaxRows) {
    start = tid < rows_here && (tid == 0 || S.row_b[tid - 1] != b);
    starts = __ballot_sync(0xffffffffu, start);
    if (lane == 0) S.warp_starts[warp] = __popc(starts);
  }
  __syncthreads();
  if (tid < kMaxRows) {
    int id = -1;
    for (int w = 0; w < warp; ++w) id += S.warp_starts[w];
    id += __popc(starts & ((2u << lane) - 1u));
    if (start) S.seg_start[id] = tid;
    if (tid == rows_here - 1) {
      S.segs = id + 1;
      S.seg_start[id + 1] = rows_here;
    }
    if (tid < rows_here && n > 0) {
      atomicMax(&S.seg_most[id], n);
      atomicMin(&S.seg_least[id], n);
      atomicMin(&S.seg_low[id], p.window > 0 ? max(0, n - p.window) : 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  bool ok = true;
  // registers: 168 a thread at launch; the softmax warps hold a row of S (128)
  // and take 216, the others give up the difference (2 * 216 + 72 = 3 * 168)
  if (warp < kSoftmaxWarps)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp < kSoftmaxWarps) {
    ok = softmax_role<D>(S, L, warp >> 2, kvh, chunk, row0);
  } else if (warp == kTmaWarp) {
    ok = tma_role<D>(S, L, &qmap, &kmap, &vmap, kvh, chunk, row0);
  } else if (warp == kMmaWarp) {
    if (lane == 0) ok = mma_role<D>(S, L, chunk);
  } else {
    ok = prep_role<D>(S, L, chunk);
  }
  if (!ok) atomicOr(p.status, kDevWaitTimeout);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(S.tmem, kTmemCols);
  }
  if (p.chunks > 1) pdl_trigger();
}

// 4-D map of a cache: (dim, token, head, block), boxes of 64 dims of one
// block's tokens, 128-byte swizzle.
bool cache_map(CUtensorMap* map, const void* base, const CacheView& c, const long long* st) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t bs = 1u << c.bs_log2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dim), bs, static_cast<cuuint64_t>(c.heads),
                              static_cast<cuuint64_t>(c.num_blocks)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(st[2]), static_cast<cuuint64_t>(st[1]),
                                 static_cast<cuuint64_t>(st[0])};
  const cuuint32_t box[4] = {64, bs, 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D map of the queries: (dim, head, row), boxes of 64 dims of the heads of
// one kv head and the rows of one tile.
bool query_map(CUtensorMap* map, const AttnLaunch& p, int rows_per_tile) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.c.dim), static_cast<cuuint64_t>(p.q_heads),
                              static_cast<cuuint64_t>(p.rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.c.dim) * 2, static_cast<cuuint64_t>(p.q_row) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(rows_per_tile)};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p.q), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_tiles_t(const AttnLaunch& p, cudaStream_t stream) {
  TilesLaunch L{p, kTile / p.group, 0};
  L.row_tiles = (p.rows + 2 * L.rows_per_tile - 1) / (2 * L.rows_per_tile);
  CUtensorMap qmap, kmap, vmap;
  if (!query_map(&qmap, p, L.rows_per_tile) || !cache_map(&kmap, p.c.k, p.c, p.c.kst) ||
      !cache_map(&vmap, p.c.v, p.c, p.c.vst))
    return cudaErrorInvalidValue;
  constexpr size_t smem = sizeof(Shared<D>) + 1024;
  static bool attr_done[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_done[dev]) {
    cudaError_t e = cudaFuncSetAttribute(attn_tiles_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done[dev] = true;
  }
  const long long grid = static_cast<long long>(L.row_tiles) * p.c.heads * p.chunks;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  attn_tiles_kernel<D><<<static_cast<unsigned>(grid), kThreads, smem, stream>>>(L, qmap, kmap, vmap);
  return cudaGetLastError();
}

}  // namespace

bool attn_tiles_apply(int group, bool f8, float scale_log2) { return group <= kTile && !f8 && scale_log2 > 0.f; }

AttnPlan attn_tiles_plan(long long rows, int q_heads, int heads, int dim, long long max_keys, int num_sms) {
  const int per = kTile / (q_heads / heads);
  const long long units = (rows + 2 * per - 1) / (2 * per) * heads;
  const long long tiles = std::max<long long>(1, (max_keys + kTile - 1) / kTile);
  // cost in tile steps: waves of CTAs, each its share of the tiles and about
  // four steps of start and end, and the partial results' traffic
  AttnPlan pl{1, 0};
  double best = 1e300;
  for (long long c = 1; c <= std::min<long long>(tiles, 32); ++c) {
    const double waves = static_cast<double>((units * c + num_sms - 1) / num_sms);
    double cost = waves * (static_cast<double>(tiles) / c + 4);
    if (c > 1) cost += 6 + static_cast<double>(rows) * q_heads * c * dim * 8 / 3e6;
    if (cost < best * 0.98) {
      best = cost;
      pl.chunks = static_cast<int>(c);
    }
  }
  if (pl.chunks > 1)
    pl.workspace_bytes = static_cast<size_t>(rows) * q_heads * pl.chunks * (static_cast<size_t>(dim) * 4 + 8);
  return pl;
}

cudaError_t launch_attn_tiles(const AttnLaunch& p, cudaStream_t stream) {
  const cudaError_t e = p.c.dim == 128 ? launch_tiles_t<128>(p, stream) : launch_tiles_t<64>(p, stream);
  if (e != cudaSuccess || p.chunks == 1) return e;
  return launch_attn_join(p, true, stream);
}

}  // namespace sai
