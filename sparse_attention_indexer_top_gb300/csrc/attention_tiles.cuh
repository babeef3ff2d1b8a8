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
// At dim 128 two CTAs of a cluster pair up (cta_group::2): an MMA tile is 256
// pairs, 128 in each CTA's TMEM, and each CTA holds half of every K tile (64
// keys) and of every V tile (64 dims). One CTA alone reads 128 bytes of shared
// memory per clock for Q K^T, all there is, besides what the copies write; the
// pair needs 96 and half the copies. The first CTA's MMA thread issues for
// both; the second CTA's softmax and prep warps report to its barriers.
//
// Work: a unit is a kv head and the rows of one CTA (pair). With many units
// each CTA (pair) takes one; with few, the CTAs stay and the units' key tiles,
// end to end, are dealt out in equal shares, so that the last wave is full and
// a few long units fill the GPU: a unit cut by a share's border leaves two or
// more partial results (maximum, sum, O) that a second kernel joins.
//
// Roles (12 warps): 0-3 softmax of tile A, 4-7 softmax of tile B, 8 TMA, 9
// MMA, 10-11 "prep", which makes the value tile safe to multiply: a weight of 0
// times a NaN or infinity that a row must not see would still be NaN, so in
// tiles that some row sees only in part, rows of V past the request's end become
// 0, and rows with a non-finite value too; if such a row of V is seen by some
// query row, its share is added at the end from global memory.
//
// e4m3 cache: the products run in f16, which holds e4m3 codes exactly. The prep
// warps turn the codes of each K and V tile into halves in the MMA's layout, one
// conversion for all the tiles of rows; with 2^E the power of two of the
// tile's largest block scale, a block of scale 2^e f, 1 <= f < 2, is multiplied
// by 2^(e - E) (exact down to e - E = -12), and the softmax applies 2^E: a key
// tile's in its multiplier, a value tile's in the exponent, w_t = 2^(s_t + Ev -
// m) with m up to 2^14 below the maximum of s + Ev, so that weights fit f16 whatever
// the scales; l adds w_t / 2^Ev. What is left of a scale, f or a power below 2^-12,
// goes to the softmax too, 16 keys at a time: nothing when scales are
// powers of two, as append_kv makes them. The queries are brought to [2^14,
// 2^15) by a power of two for each (row, head) and stored as halves.
//
// MOD: rows see a document or a prefix of their request (kMasks), and scores are
// capped (kCap) and biased by distance (kBias) before the softmax
// (attention_mod.cuh). These instances are apart, in attention_tiles_mod.cu and
// attention_tiles_cap.cu. Bound: the softmax warps, whose two-element operations a
// pair of scores go from 2 to 4 (bias), 5 (cap, scores below a quarter of it; e4m3 6), 6
// (below half; 7) or, with both, 2 more; scores above go the longer way (rough_tile). 2048
// rows on 32768 keys, 32 / 4 heads, bf16 (e4m3), us: plain 623 (783), masks 647 (813),
// bias 672 (818), cap 760 (884), 862 (946), 1541 (1801) with scores below a quarter, below
// half, above half of it, both 820 (1042).
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "attention_mod.cuh"
#include "sai_internal.h"
#include "sai_ptx.cuh"
#include "sai_tmap.h"

namespace sai {
namespace {

constexpr int kTile = 128;       // keys of a tile, and (row, head) pairs of an MMA tile
template <int D>
constexpr int kPair = D == 128 ? 2 : 1;               // CTAs of a pair
template <int D>
constexpr int kMaxRows = 2 * kTile * kPair<D>;        // query rows of a pair (group 1)
constexpr int kSoftmaxWarps = 8;
constexpr int kTmaWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kPrepWarp = 10;
constexpr int kPrepWarps = 2;
constexpr int kThreads = (kPrepWarp + kPrepWarps) * 32;
constexpr int kMasks = 1, kCap = 2, kBias = 4;  // MOD
constexpr uint32_t kSetUpBar = 1;  // named barrier of all threads between pieces
constexpr float kLn2 = 0.69314718055994530942f;

// The running maximum m of a row moves only when it is passed by more than
// 2^8, so that O is rarely rescaled. Weights in bf16 are as exact up to 2^8 as
// up to 1. Weights in f16 (e4m3) use its range: m is set 2^6 below the maximum,
// weights reach 2^14 (below 2^15 with what is left of a scale), and one below
// 2^-14 is off by 2^-25 at most, 2^-31 of the largest.
template <bool F8>
constexpr float kLift = F8 ? 6.f : 0.f;
template <bool F8>
constexpr float kPassed = kLift<F8> + 8.f;

// TMEM columns: S (and P over it) of tiles A and B, then their O.
constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;

struct TilesLaunch {
  AttnLaunch a;
  int rows_per_tile;  // floor(128 / group): rows of one CTA's part of an MMA tile
  int row_tiles;      // CTAs (pairs) along the rows
  int dealt;          // units' tiles dealt out over the grid (else one unit per CTA or pair)
  int4* borders;      // dealt: the first step of each share after the first: kv head, row tile, step of the unit, unit's
                      // steps; entry 0: number of shares, steps of a kv head
};

constexpr int kMaxDealt = 1024;  // most row tiles when dealt out
constexpr int kUnitWeight = 3;   // a unit's start and end, in tile steps
constexpr int kLeastShare = 8;   // tile steps that are worth a CTA (pair) of their own

// Shares: share i holds the steps [i * total / n, (i + 1) * total / n).
__device__ __forceinline__ long long share_start(long long i, long long total, int n) { return i * total / n; }
__device__ __forceinline__ int share_of(long long step, long long total, int n) {
  return static_cast<int>(((step + 1) * n - 1) / total);
}

// What a CTA (pair) does at a time: a unit's tiles from `from` to `to` of `of`.
struct Piece {
  int kvh, row0;
  int from, to, of;
  int slot;  // place of its partial results, -1: the piece is the whole unit
};

template <int D, bool F8>
struct Shared {
  static constexpr int kPairN = kPair<D>;
  static constexpr int kKeys = kTile / kPairN;  // keys of a K tile in this CTA
  static constexpr int kDims = D / kPairN;      // dims of a V tile in this CTA (64)
  static_assert(kDims == 64, "V is one slab of 64 dims");
  static constexpr int kSlabs = D / 64;
  static constexpr int kQBytes = kSlabs * kTile * 128;
  static constexpr int kKBytes = kSlabs * kKeys * 128, kVBytes = kTile * 128;
  // K and V tiles of the MMA; of e4m3 fewer, fed from a ring of code tiles
  // that K and V take in turn
  static constexpr int kStages = F8 ? 2 : 3;
  static constexpr int kRaw = F8 ? 8 : 0;
  unsigned char q[2][kQBytes];
  unsigned char k[kStages][kKBytes];
  unsigned char v[kStages][kVBytes];
  unsigned char raw[kRaw ? kRaw : 1][kRaw ? kKeys * D : 16];
  unsigned char stage[kSoftmaxWarps][32 * 64];  // rows on their way out
  // In the first CTA of a pair, for both (the MMA waits there): q_full (bf16),
  // q_ready, k_full, v_safe, p_ready. In each CTA for itself: the others.
  uint64_t q_full, q_ready, k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], v_safe[kStages];
  uint64_t raw_full[kRaw ? kRaw : 1], raw_empty[kRaw ? kRaw : 1];
  uint64_t s_ready[2], p_ready[2][2], o_done[2];  // p_ready: first and second half of the keys
  uint32_t tmem;
  // A pass of the piece met a non-finite value row. One mark for all passes: prep runs ahead of the softmax, over a
  // pass's end too, and add_nonfinite looks for its own pass's rows.
  int nonfinite;
  int stop;       // a wait gave up: no further piece
  int segs;
  int gap;  // with the piece at a multiple of 16 bytes plain e4m3 tiles take 803 us for 782
  Piece piece;             // at work on
  long long step, begin, end;  // dealt: next step, and the share
  int more;                // a piece follows
  int deal[kMaxDealt + 2];  // dealt: the row tiles' weights, summed up, and the number of shares
  int warp_starts[16];
  int row_n[kMaxRows<D>], row_b[kMaxRows<D>];
  // of each run of rows of one request. MOD has more to keep in them, in tiles (pack_segment).
  int seg_start[kMaxRows<D> + 1], seg_most[kMaxRows<D>], seg_least[kMaxRows<D>], seg_low[kMaxRows<D>];
  float2 factors[F8 ? kSoftmaxWarps : 1][8];  // per softmax warp: what the tiles leave of the k and v scales of 16 keys
};

// MOD: what a segment's three words hold: tiles of 128 keys, and counts of them in 8
// bits each, 255 meaning as many as there are (shared memory has no room for whole
// words; a tile more than needed is masked).
struct Segment {
  int low_tile;     // of the least first key
  int high_tiles;   // tiles from there on that some row does not see the start of
  int base_tile;    // of the first tokens that lie before low_tile, and of how many tiles
  int first_tiles;
  int least_tiles;  // last tiles that some row does not see the end of
};
__device__ __forceinline__ int count8(int n) { return max(0, min(n, 255)); }
__device__ __forceinline__ void pack_segment(const Segment& g, int& start, int& least, int& low) {
  low = g.low_tile << 8 | count8(g.high_tiles);
  least = g.base_tile << 8 | count8(g.first_tiles);
  start |= count8(g.least_tiles) << 16;
}
__device__ __forceinline__ Segment unpack_segment(int start, int least, int low) {
  return Segment{static_cast<int>(static_cast<uint32_t>(low) >> 8), low & 255,
                 static_cast<int>(static_cast<uint32_t>(least) >> 8), least & 255, start >> 16};
}

// One request's rows of the CTA (pair) and the tiles that the piece walks.
template <int MOD>
struct PassMore {
  int base_tile;  // of the first tokens
  int high;       // up to there, some row does not see a tile's start
  int last;       // index of the last tile
};
template <>
struct PassMore<0> {
  static constexpr int base_tile = 0, high = 0, last = 0;
};
template <int MOD>
struct Pass : PassMore<MOD> {
  int s, e;        // rows [s, e) of the pair
  int batch;
  int most, least; // longest and shortest (above 0) row (MOD: in whole tiles)
  int low;         // least first key of a row's window (0: no window)
  int first_tiles; // tiles that hold the first `sinks` tokens before the window's tiles
  int low_tile;
  int i0, i1;      // tile indices of this piece
  bool act[2];     // MMA tile has rows of the pass
  // With a bias the nearest tiles come first: from the first tile on, every
  // nearer one would pass the running maximum by its 128 steps of the slope.
  __device__ __forceinline__ int tile0(int i) const {
    if (MOD & kBias) i = this->last - i;
    return (i < first_tiles ? i + this->base_tile : i - first_tiles + low_tile) * kTile;
  }
  // does every row of the pass see all of the tile?
  __device__ __forceinline__ bool partial(int t0, const AttnLaunch& p) const {
    if (t0 + kTile > least) return true;
    if (MOD) return t0 < this->high;
    if (p.window == 0 || t0 >= most - p.window) return false;
    return !(t0 + kTile <= p.sinks && t0 + kTile <= low);
  }
};

template <int MOD, int D, bool F8>
__device__ __forceinline__ Pass<MOD> get_pass(const Shared<D, F8>& S, const TilesLaunch& L, int seg) {
  const AttnLaunch& p = L.a;
  const Piece& pc = S.piece;
  Pass<MOD> r;
  constexpr int kStart = MOD ? 0xffff : -1;
  r.s = S.seg_start[seg] & kStart;
  r.e = S.seg_start[seg + 1] & kStart;
  r.batch = S.row_b[r.s];
  r.most = S.seg_most[seg];
  r.least = S.seg_least[seg];
  r.low = S.seg_low[seg];
  const int per = kPair<D> * L.rows_per_tile;
  r.act[0] = r.s < per;
  r.act[1] = r.e > per;
  int tiles = 0;
  r.first_tiles = r.low_tile = 0;
  if constexpr (MOD != 0) {
    const Segment g = unpack_segment(S.seg_start[seg], r.least, r.low);
    const int end = (r.most + kTile - 1) / kTile;
    r.base_tile = g.base_tile;
    r.low_tile = g.low_tile;
    r.first_tiles = g.first_tiles < 255 ? g.first_tiles : g.low_tile - g.base_tile;
    r.high = g.high_tiles < 255 ? (g.low_tile + g.high_tiles) * kTile : INT_MAX;
    r.least = g.least_tiles < 255 ? (end - g.least_tiles) * kTile : 0;
    tiles = r.first_tiles + end - r.low_tile;
  } else if (r.most > 0) {
    r.low_tile = r.low / kTile;
    if (r.low > 0) r.first_tiles = min((min(p.sinks, r.low) + kTile - 1) / kTile, r.low_tile);
    tiles = r.first_tiles + (r.most + kTile - 1) / kTile - r.low_tile;
  }
  if constexpr (MOD != 0) r.last = tiles - 1;
  r.i0 = static_cast<int>(static_cast<long long>(tiles) * pc.from / pc.of);
  r.i1 = static_cast<int>(static_cast<long long>(tiles) * pc.to / pc.of);
  return r;
}

// TMA loads into this CTA; `bar` is a shared::cluster address, in a pair
// possibly the first CTA's barrier.
template <int PAIR>
__device__ __forceinline__ void tma_4d(void* dst, const void* map, int c0, int c1, int c2, int c3, uint32_t bar) {
  if (PAIR == 2)
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}
template <int PAIR>
__device__ __forceinline__ void tma_3d(void* dst, const void* map, int c0, int c1, int c2, uint32_t bar) {
  if (PAIR == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// shared::cluster address of the same variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
// Barrier address in the first CTA of the pair (this CTA without a pair).
template <int PAIR>
__device__ __forceinline__ uint32_t first_cta(const uint64_t* bar) {
  return PAIR == 2 ? peer_addr(bar, 0) : smem_u32(bar);
}
template <int PAIR>
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
  if (PAIR == 2)
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(peer_addr(bar, 0)) : "memory");
  else
    mbar_arrive(bar);
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrive, in every CTA of the pair, when the products issued so far are done.
template <int PAIR>
__device__ __forceinline__ void commit_all(uint64_t* bar) {
  if (PAIR == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    umma_commit(bar);
}
// True in one thread of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
template <int PAIR>
__device__ __forceinline__ void tmem_take(uint32_t* result) {
  if (PAIR == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(result)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(result, kTmemCols);
    tmem_relinquish();
  }
}
template <int PAIR>
__device__ __forceinline__ void tmem_give(uint32_t addr) {
  if (PAIR == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(kTmemCols) : "memory");
  else
    tmem_dealloc(addr, kTmemCols);
}
// Shared-memory matrix descriptors of 128-byte swizzled tiles (rows of 128
// bytes in atoms of 8 rows, 1024 bytes apart). Low word: start address and
// leading offset (not used: a tile's outer extent is one 128-byte row); the high
// word is the same for all: stride offset 1024, version 1, 128-byte swizzle.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t smem_addr) { return ((smem_addr & 0x3FFFFu) >> 4) | (1u << 16); }
// D[tmem] (+)= A[smem] x B[smem], 16-bit types.
template <int PAIR>
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
#define SAI_UMMA_SS(N)                                                                                    \
  asm volatile(                                                                                           \
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"            \
      "setp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::" #N ".kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),  \
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)                                      \
      : "memory")
  if (PAIR == 2)
    SAI_UMMA_SS(2);
  else
    SAI_UMMA_SS(1);
#undef SAI_UMMA_SS
}
// D[tmem] (+)= A[tmem] x B[smem], 16-bit A packed two to a column.
template <int PAIR>
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
#define SAI_UMMA_TS(N)                                                                                    \
  asm volatile(                                                                                           \
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"            \
      "tcgen05.mma.cta_group::" #N ".kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),                        \
      "r"(a), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)                                         \
      : "memory")
  if (PAIR == 2)
    SAI_UMMA_TS(2);
  else
    SAI_UMMA_TS(1);
#undef SAI_UMMA_TS
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
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
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
constexpr uint32_t kTransposeB = 1u << 16;  // instruction descriptor: B is N-major

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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

// Exponent of a block scale (scales outside 2^-64 .. 2^120, 0 among them, leave
// the rest to their factor; l holds weights over the value scale's power, which
// fits fp32 down to 2^-64 for any number of keys; 2^120 is the scale of the
// largest bf16 values), and 2^e.
constexpr int kLeastExp = -64;
__device__ __forceinline__ int exponent_of(float scale) {
  return max(kLeastExp, min(120, static_cast<int>((__float_as_uint(scale) >> 23) & 255u) - 127));
}
__device__ __forceinline__ float power_of(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
constexpr int kNoScale = -1000;   // exponent of a group without a block
constexpr int kLeastShift = -12;  // e - E that is still exact in f16

// Four e4m3 codes to halves, exactly.
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t c, uint32_t& a, uint32_t& b) {
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(c));
}
__device__ __forceinline__ void mul_f16x2(uint32_t& a, uint32_t power) {
  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(a) : "r"(power));
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// ------------------------------------------------------------------ softmax
// Thread of one (row, head) pair.
template <int MOD>
struct LaneMore {
  int start, pos;  // sees t >= start; its position
  float slope;     // in log2 units
};
template <>
struct LaneMore<0> {
  static constexpr int start = 0, pos = 0;
  static constexpr float slope = 0.f;
};
template <int MOD>
struct Lane : LaneMore<MOD> {
  int row;         // row of the call
  int n, first, sinks;  // sees t < n with t >= first or t < sinks
  long long head;  // row * q_heads + head
  bool live;       // belongs to the pass
};

// Two values of a cache row: bf16 pair d, or e4m3 codes 2d and 2d + 1.
template <bool F8>
__device__ __forceinline__ float2 values2(const char* row, int d) {
  if (F8) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(reinterpret_cast<const uint16_t*>(row)[d]));
    return __half22float2(*reinterpret_cast<__half2*>(&r));
  }
  const uint32_t x = reinterpret_cast<const uint32_t*>(row)[d];
  return make_float2(bf16_lo(x), bf16_hi(x));
}

// Adds to o[], 32 columns of O from column c0, the values that were kept out
// of the product for being non-finite: every such key of the tiles that were
// checked.
template <int D, bool F8, int MOD>
__device__ __noinline__ void add_nonfinite(const AttnLaunch& p, const Pass<MOD>& ps, int kvh, const Lane<MOD>& ln, float m,
                                           int c0, float (&o)[32]) {
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
      const char* v = p.c.v + blk * p.c.vst[0] + kvh * p.c.vst[1] + off * p.c.vst[2];
      const char* k = p.c.k + blk * p.c.kst[0] + kvh * p.c.kst[1] + off * p.c.kst[2];
      bool bad = false;
      // what was kept out goes by the 64 dims of one V tile
      for (int d = c0 / 64 * 32 + lane; d < c0 / 64 * 32 + 32; d += 32) {
        const float2 x = values2<F8>(v, d);
        bad = bad || !(fabsf(x.x) <= 3.402823466e38f) || !(fabsf(x.y) <= 3.402823466e38f);
      }
      if (!__any_sync(0xffffffffu, bad)) continue;
      if (!ln.live || t >= ln.n || (t < ln.first && t >= ln.sinks) || (MOD && t < ln.start)) continue;
      float s = 0.f;
      for (int d = 0; d < D / 2; ++d) {
        const uint32_t a = reinterpret_cast<const uint32_t*>(q)[d];
        const float2 b = values2<F8>(k, d);
        s = fmaf(bf16_lo(a), b.x, fmaf(bf16_hi(a), b.y, s));
      }
      float e = s * p.scale_log2, vscale = 1.f;
      if (F8) {
        const long long at = static_cast<long long>(blk) * p.c.heads + kvh;
        e *= p.c.ks[at];
        vscale = p.c.vs[at];
      }
      if (MOD & kCap) e = capped(e, p.cap_log2, 1.f / p.cap_log2);
      if (MOD & kBias) e = fmaf(-ln.slope, static_cast<float>(abs(ln.pos - t)), e);
      const float w = ex2(e - (m == -INFINITY ? 0.f : m)) * vscale;
#pragma unroll
      for (int d = 0; d < 16; ++d) {
        const float2 x = values2<F8>(v, c0 / 2 + d);
        o[2 * d] = fmaf(w, x.x, o[2 * d]);
        o[2 * d + 1] = fmaf(w, x.y, o[2 * d + 1]);
      }
    }
  }
}

// Writes 64 bytes of each of the warp's 32 rows (`mine` of the lane's own, to
// `dst`, null: not written). A lane's row is a line of its own in memory, so
// the rows go through 2 KB of shared memory and four lanes write one
// row's 64 bytes: a quarter of the store's passes (an epilogue of 10,400 cycles
// without).
__device__ __forceinline__ void write_rows64(unsigned char* stage, const uint4 (&mine)[4], char* dst) {
  const int lane = threadIdx.x & 31;
  __syncwarp();  // the last 64 bytes have been read
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = mine[c];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 8 * i + lane / 4, c = lane % 4;
    const uint4 x = *reinterpret_cast<const uint4*>(stage + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
    char* to = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), row));
    if (to) *reinterpret_cast<uint4*>(to + 16 * c) = x;
  }
}

// 32 columns of the thread's row, from column c0; an unseen row's O may hold
// anything. `part`: place of the row's partial results, -1: they are final.
template <int D, int MOD>
__device__ __forceinline__ void write_columns(const AttnLaunch& p, const Lane<MOD>& ln, long long part, float l, int c0,
                                              const float (&o)[32], unsigned char* stage) {
  const bool none = l == 0.f;
  uint4 x[4];
  if (part >= 0) {
    char* dst = ln.live ? reinterpret_cast<char*>(p.part_o + part * D + c0) : nullptr;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const float* v = o + 16 * h + 4 * d;
        x[d] = none ? make_uint4(0, 0, 0, 0)
                    : make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      }
      write_rows64(stage, x, dst ? dst + 64 * h : nullptr);
    }
    return;
  }
  const float inv = none ? 0.f : 1.f / l;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const float* v = o + 8 * d;
    x[d] = none ? make_uint4(0, 0, 0, 0)
                : make_uint4(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv),
                             pack_bf16(v[4] * inv, v[5] * inv), pack_bf16(v[6] * inv, v[7] * inv));
  }
  write_rows64(stage, x, ln.live ? reinterpret_cast<char*>(p.out + ln.head * D + c0) : nullptr);
}
template <int MOD>
__device__ __forceinline__ void write_sums(const AttnLaunch& p, const Lane<MOD>& ln, long long part, float m, float l) {
  if (!ln.live) return;
  if (part >= 0)
    p.part_ml[part] = make_float2(m, l);
  else if (p.lse)
    p.lse[ln.head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Brings this thread's row of the query tile from bf16 to halves, times a
// power of two that puts its largest magnitude into [2^14, 2^15); returns the
// factor's inverse. Values down to 2^-28 of the largest are exact, the rest
// off by at most 2^-39 of it.
template <int D>
__device__ __forceinline__ float query_to_f16(unsigned char* tile, int r) {
  float amax = 0.f;
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    const uint4 x = *reinterpret_cast<const uint4*>(tile + (c / 8) * kTile * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
  }
  const int e = static_cast<int>(__float_as_uint(amax) >> 23);
  const int up = (e == 0 || e == 255) ? 0 : min(126, 14 - (e - 127));  // 2^up and 2^-up are normal numbers
  const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    uint4* at = reinterpret_cast<uint4*>(tile + (c / 8) * kTile * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    const uint4 x = *at;
    *at = make_uint4(pack_f16(bf16_lo(x.x) * f, bf16_hi(x.x) * f), pack_f16(bf16_lo(x.y) * f, bf16_hi(x.y) * f),
                     pack_f16(bf16_lo(x.z) * f, bf16_hi(x.z) * f), pack_f16(bf16_lo(x.w) * f, bf16_hi(x.w) * f));
  }
  return __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
}

// Which of 32 columns the row sees, a bit each: those below n, except below
// `first` that are not below `sinks` (MOD: and those below `start`); bits 0 and 1
// of `bad` take out 16 each.
template <int MOD>
__device__ __forceinline__ uint32_t seen32(int n, int first, int sinks, int start, uint32_t bad) {
  auto below = [](int x) { return x <= 0 ? 0u : x >= 32 ? ~0u : (1u << x) - 1u; };
  uint32_t see = below(n) & (~below(first) | below(sinks));
  if (MOD) see &= ~below(start);
  if (bad & 1) see &= 0xffff0000u;
  if (bad & 2) see &= 0x0000ffffu;
  return see;
}
// Scores of 32 columns that the row does not see become -inf. One bit a column,
// so that an element costs a test and a select.
template <int MOD>
__device__ __forceinline__ void mask32(uint32_t* s, int n, int first, int sinks, int start, uint32_t bad) {
  const uint32_t see = seen32<MOD>(n, first, sinks, start, bad);
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (!(see & (1u << c))) s[c] = 0xff800000u;
}

// Multiplies the thread's row of O by f.
template <int D>
__device__ __forceinline__ void rescale_o(uint32_t to, float f) {
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t u[32];
    tmem_ld32(to + c, u);
    tmem_ld_wait32(u);
#pragma unroll
    for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * f);
    tmem_st16(to + c, u);
    tmem_st16(to + c + 16, u + 16);
  }
}

// What a thread's row does to its scores, in log2 units, besides the multiplier.
struct Change {
  float cap, inv_cap;
  float slope;
  int ahead;  // the row's position less the tile's first token
};

// Changes 32 columns of scores s, from column c0 of the tile: times `mul`,
// capped, biased. Two elements to an instruction. FAR 0: no score is above half
// the cap; 1: none above the cap (three coefficients more, but no exponentials and
// reciprocals, of which a pair would take as long as two dozen FMAs); 2: those above
// half of it are cap (1 - 2 / (1 + e^(2x / cap))), off by 2^-22 of the cap.
template <int MOD, int FAR>
__device__ __forceinline__ void change32(uint32_t* s, int c0, float mul, const Change& ch) {
  const float xm = fminf(mul * ch.inv_cap, 1e38f), em = xm * 2.885390081777927f;  // finite: a score of 0 stays 0
  const uint64_t mul_2 = pair(mul, mul), x_2 = pair(xm, xm), e_2 = pair(em, em), slope_2 = pair(-ch.slope, -ch.slope);
  const uint64_t cap_2 = pair(ch.cap, ch.cap), less_2 = pair(-2.f * ch.cap, -2.f * ch.cap), one_2 = pair(1.f, 1.f);
  // distances of the two columns, whole numbers, less 2 at each step
  uint64_t d = pair(static_cast<float>(ch.ahead - c0), static_cast<float>(ch.ahead - c0 - 1));
  const uint64_t step = pair(-2.f, -2.f);
  constexpr int Q = FAR == 1 ? 7 : 4;
  uint64_t q_2[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const float f = ch.cap * (FAR == 1 ? tanh_q(i) : tanh_near(i < 4 ? i : 0));
    q_2[i] = pair(f, f);
  }
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    uint64_t v = pair(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
    if (MOD & kCap) {
      const uint64_t x = mul2(v, x_2), y = mul2(x, x);
      uint64_t q = q_2[Q - 1];
#pragma unroll
      for (int i = Q - 2; i >= 0; --i) q = fma2(q, y, q_2[i]);
      q = mul2(x, q);
      if (FAR == 2) {
        float a, b, xa, xb, na, nb;
        unpair(mul2(v, e_2), a, b);
        unpair(add2(pair(ex2(a), ex2(b)), one_2), a, b);
        unpair(fma2(pair(rcp(a), rcp(b)), less_2, cap_2), a, b);
        unpair(x, xa, xb);
        unpair(q, na, nb);
        q = pair(fabsf(xa) <= kNear ? na : a, fabsf(xb) <= kNear ? nb : b);
      }
      v = q;
    } else {
      v = mul2(v, mul_2);
    }
    if (MOD & kBias) {
      v = fma2(slope_2, d & 0x7fffffff7fffffffull, v);
      d = add2(d, step);
    }
    float lo, hi;
    unpair(v, lo, hi);
    s[c] = __float_as_uint(lo);
    s[c + 1] = __float_as_uint(hi);
  }
}

// Weights 2^(changed score + off) of 32 columns from column c0, two to a word in
// s[0..16), and what they add up to: change and exponent in one go. One 16-bit term
// each, off by 2^-8 (f16 2^-11) as in the plain kernel, which leaves bf16 results off by
// 0.0023 for 0.0017 with exact weights (2048 rows on 32768 keys): the second term that
// the row kernel takes would be half as many products again here. The bias is
// linear in the column, slope * column and part of `off`; MASKED: columns without
// their bit in `see` get 0.
template <bool F8, int MOD, int Q, bool MASKED>
__device__ __forceinline__ uint64_t changed_weights32(uint32_t* s, int c0, uint64_t mul_2, const uint64_t (&q_2)[Q],
                                                      uint64_t off_2, uint64_t slope_2, uint32_t see) {
  uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
  uint64_t col = pair(static_cast<float>(c0), static_cast<float>(c0 + 1));
  const uint64_t two = pair(2.f, 2.f);
#pragma unroll
  for (int c = 0; c < 32; c += 8) {
    uint64_t x[4], w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = off_2;
      if (MOD & kBias) {
        w[j] = fma2(col, slope_2, off_2);
        col = add2(col, two);
      }
      x[j] = pair(__uint_as_float(s[c + 2 * j]), __uint_as_float(s[c + 2 * j + 1]));
    }
    if (MOD & kCap) {
      uint64_t y[4], q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (F8) x[j] = mul2(x[j], mul_2);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = mul2(x[j], x[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = q_2[Q - 1];
#pragma unroll
      for (int k = Q - 2; k >= 0; --k)
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = fma2(q[j], y[j], q_2[k]);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = fma2(x[j], q[j], w[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = fma2(x[j], mul_2, w[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a, b;
      unpair(w[j], a, b);
      a = ex2(a);
      b = ex2(b);
      if (MASKED) {
        a = see & (1u << (c + 2 * j)) ? a : 0.f;
        b = see & (2u << (c + 2 * j)) ? b : 0.f;
      }
      sum[j & 1] = add2(sum[j & 1], pair(a, b));
      s[c / 2 + j] = F8 ? pack_f16(a, b) : pack_bf16(a, b);
    }
  }
  return add2(sum[0], sum[1]);
}

// The largest magnitude of 32 columns and `top`.
__device__ __forceinline__ float largest32(const uint32_t* s, float top) {
  float a[4] = {top, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 32; c += 2)
    a[c / 2 & 3] = max3(a[c / 2 & 3], fabsf(__uint_as_float(s[c])), fabsf(__uint_as_float(s[c + 1])));
  return fmaxf(max3(a[0], a[1], a[2]), a[3]);
}

// Any tile, by the longer way: an e4m3 cache's whose scales are not all in the
// tile's powers (factors[g] are left over of 16 keys' scales; null: nothing is),
// and with changed scores one that may move the maximum, has scores near its
// cap, or keys on both sides of a row's position (`keep`: the maximum is known to
// stay, and one reading does). Out of line, and S is read twice 32 columns at a
// time: beside the plain code it slowed that by half.
template <int D, bool F8, int MOD>
__device__ __noinline__ float2 rough_tile(uint32_t ts, uint32_t to, float2 ml, float mul, float ev, float un_ev,
                                          const float2* factors, int4 sees, uint32_t bad, bool masked, bool have_o,
                                          bool keep, Change ch) {
  constexpr bool kChanged = (MOD & (kCap | kBias)) != 0;
  uint32_t s[32];
  // masked after the scaling: a scale may be 0, and 0 * -inf is NaN
  auto scaled = [&](int c0) {
    if (!kChanged || factors) {
#pragma unroll
      for (int c = 0; c < 32; ++c) s[c] = __float_as_uint(__uint_as_float(s[c]) * factors[(c0 + c) / 16].x);
    }
    if (kChanged) {
      const float far = MOD & kCap ? largest32(s, 0.f) * (mul * ch.inv_cap) : 0.f;
      if (!(MOD & kCap) || __all_sync(0xffffffffu, far <= kNear))
        change32<MOD, 0>(s, c0, mul, ch);
      else if (__all_sync(0xffffffffu, far <= 1.f))
        change32<MOD, 1>(s, c0, mul, ch);
      else
        change32<MOD, 2>(s, c0, mul, ch);
    }
    if (!kChanged || masked) mask32<MOD>(s, sees.x - c0, sees.y - c0, sees.z - c0, sees.w - c0, bad >> (c0 / 16));
  };
  const float mul1 = kChanged ? 1.f : mul;
  float top = -INFINITY;
#pragma unroll 1
  for (int c0 = 0; c0 < kTile && !(kChanged && keep); c0 += 32) {
    tmem_ld32(ts + c0, s);
    tmem_ld_wait32(s);
    scaled(c0);
    if (kChanged) {  // the second time they are read as they are
      tmem_st16(ts + c0, s);
      tmem_st16(ts + c0 + 16, s + 16);
    }
    float t[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int c = 0; c < 32; c += 2) t[c / 2 & 3] = max3(t[c / 2 & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
    top = fmaxf(max3(t[0], t[1], t[2]), t[3]);
  }
  if (kChanged) tmem_st_wait();
  top = fmaf(top, mul1, ev);
  const bool up = top > ml.x + kPassed<F8>;
  if (__any_sync(0xffffffffu, up)) {
    const float to_m = top - kLift<F8>;
    const float f = up ? (ml.x == -INFINITY ? 0.f : ex2(ml.x - to_m)) : 1.f;
    if (up) ml.x = to_m;
    ml.y *= f;
    if (have_o) rescale_o<D>(to, f);
  }
  const float off = ev - (ml.x == -INFINITY ? 0.f : ml.x);
  float sum = 0.f;
#pragma unroll 1
  for (int c0 = 0; c0 < kTile; c0 += 32) {  // weights of chunk c go over scores of chunk c / 2
    tmem_ld32(ts + c0, s);
    tmem_ld_wait32(s);
    if (!kChanged || keep) scaled(c0);
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      const float f = !kChanged || factors ? factors[(c0 + c) / 16].y : 1.f;
      const float a = ex2(fmaf(__uint_as_float(s[c]), mul1, off));
      const float b = ex2(fmaf(__uint_as_float(s[c + 1]), mul1, off));
      sum += a + b;
      s[c / 2] = F8 ? pack_f16(a * f, b * f) : pack_bf16(a, b);
    }
    tmem_st16(ts + c0 / 2, s);
  }
  tmem_st_wait();
  ml.y = fmaf(sum, un_ev, ml.y);
  return ml;
}

// What a role has behind it, over the pieces: the phases of its barriers.
struct Progress {
  int pieces = 0, tiles = 0, passes = 0;
  int weights[2] = {0, 0};  // MMA: tiles' weights taken
};

template <int D, bool F8, int MOD>
__device__ __forceinline__ bool softmax_role(Shared<D, F8>& S, const TilesLaunch& L, int x, int rank, Progress& at) {
  const Piece& pc = S.piece;
  constexpr int PAIR = kPair<D>;
  const AttnLaunch& p = L.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = warp & 3;
  const int r = quad * 32 + lane;  // the thread's TMEM lane
  const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t ts = S.tmem + lanes + kColS + 128 * x;
  const uint32_t to = S.tmem + lanes + kColO + 128 * x;
  const int local = (x * PAIR + rank) * L.rows_per_tile + r / p.group;
  const bool in_tile = r < L.rows_per_tile * p.group;
  float scale = p.scale_log2;
  bool lost = false;  // as in the MMA role: no way out of the loop
  const float cap = MOD & kCap ? p.cap_log2 : 0.f, inv_cap = MOD & kCap ? 1.f / cap : 0.f;
  // bf16: may the polynomial be one in the products themselves? Its last coefficient
  // has the 7th power of the scale over the cap, times the cap: normal numbers are
  // needed, and a cap below 2^17 times the scale (11,585 at dim 128; above it every
  // tile goes the longer way).
  const float over = MOD & kCap ? scale * inv_cap : 1.f, over3 = over * over * over;
  const bool in_products = F8 || (over > 0x1p-17f && over < 0x1p17f && scale * over3 * over3 < 0x1p126f);
  if (F8) {
    lost = !mbar_wait(&S.q_full, at.pieces & 1);
    scale *= query_to_f16<D>(S.q[x], r);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) arrive_first<PAIR>(&S.q_ready);
  }

  for (int seg = 0; seg < S.segs; ++seg) {
    const Pass<MOD> ps = get_pass<MOD>(S, L, seg);
    if (!ps.act[x]) continue;
    Lane<MOD> ln;
    float m = -INFINITY, l = 0.f;
    ln.row = pc.row0 + local;
    ln.live = in_tile && local >= ps.s && local < ps.e && ln.row < p.rows;
    ln.n = ln.live ? S.row_n[local] : 0;
    ln.first = p.window > 0 ? max(0, ln.n - p.window) : 0;
    ln.sinks = min(p.sinks, ln.first);
    // the row's head, and its place among the partial results (-1: final). MOD: known
    // at the end alone, the loop has no registers to keep them in. Until then a row that
    // sees nothing, padding say, is not live: it would have no maximum to keep, and send
    // all its unit's tiles the longer way (2048 rows on 32768 keys, every 50th of
    // them padding, softcap 50: 1535 us for 761).
    long long part = -1;
    auto place = [&]() {
      if (MOD) {
        ln.live = in_tile && local >= ps.s && local < ps.e && ln.row < p.rows;
        if (ln.n == 0) {
          m = -INFINITY;
          l = 0.f;
        }
      }
      ln.head = static_cast<long long>(ln.row) * p.q_heads + pc.kvh * p.group + r % p.group;
      part = pc.slot < 0 ? -1 : (static_cast<long long>(pc.slot) * 2 * PAIR * L.rows_per_tile + local) * p.group + r % p.group;
    };
    if (!MOD) place();
    if constexpr (MOD != 0) {
      ln.live = ln.n > 0;
      ln.start = ln.pos = 0;
      ln.slope = 0.f;
      if (ln.n > 0) {
        const int len = p.seq_lens[ln.row];
        const RowSpan span = row_span(p, ln.row, len);
        ln.first = span.first;
        ln.sinks = span.sinks_end;
        ln.start = span.start;
        ln.pos = len - 1;
        if (MOD & kBias) ln.slope = p.slopes[pc.kvh * p.group + r % p.group] * 1.44269504088896340736f;
      }
    }
    if (ps.i0 == ps.i1) {
      if (MOD) place();
      const float o[32] = {};
#pragma unroll 1
      for (int c = 0; c < D; c += 32) write_columns<D, MOD>(p, ln, part, l, c, o, S.stage[warp]);
      write_sums(p, ln, part, m, l);
      continue;
    }
    // lanes 0-7: block of the tile's 16-key group (-1: none, -2: bad), read
    // two tiles ahead, and its scales, read one ahead
    auto block_of = [&](int i) -> int {
      if (i >= ps.i1 || lane >= 8) return -1;
      const int t = ps.tile0(i) + 16 * lane;
      if (t >= ps.most) return -1;
      const int blk = p.block_table[ps.batch * p.bt_stride + (t >> p.c.bs_log2)];
      return blk < 0 || blk >= p.c.num_blocks ? -2 : blk;
    };
    auto scales_of = [&](int blk) -> float2 {
      if (!F8 || blk < 0) return make_float2(1.f, 1.f);
      const long long at = static_cast<long long>(blk) * p.c.heads + pc.kvh;
      return make_float2(p.c.ks[at], p.c.vs[at]);
    };
    int blk1 = block_of(ps.i0), blk2 = block_of(ps.i0 + 1);
    float2 sc1 = scales_of(blk1);
    for (int i = ps.i0; i < ps.i1; ++i) {
      const uint32_t bad = __ballot_sync(0xffffffffu, blk1 == -2);
      // the tile's multiplier and exponent; rough: scales are not all of it
      float mul = scale, ev = 0.f, un_ev = 1.f;
      bool rough = false;
      const float2* factors = S.factors[F8 ? warp : 0];
      if (F8) {
        const int ek = blk1 >= 0 ? exponent_of(sc1.x) : kNoScale, e2 = blk1 >= 0 ? exponent_of(sc1.y) : kNoScale;
        const int tk = max(kLeastExp, __reduce_max_sync(0xffffffffu, ek)), tv = max(kLeastExp, __reduce_max_sync(0xffffffffu, e2));
        mul = fmaxf(scale * power_of(tk), 1.17549435e-38f);  // not 0: masked scores are -inf
        ev = static_cast<float>(tv);
        un_ev = power_of(-tv);
        const float2 f = blk1 >= 0 ? make_float2(sc1.x * power_of(-max(ek, tk + kLeastShift)),
                                                 sc1.y * power_of(-max(e2, tv + kLeastShift)))
                                   : make_float2(1.f, 1.f);
        rough = __any_sync(0xffffffffu, f.x != 1.f || f.y != 1.f);
        if (rough) {
          if (lane < 8) S.factors[warp][lane] = f;
          __syncwarp();
        }
        sc1 = scales_of(blk2);
      }
      blk1 = blk2;
      blk2 = block_of(i + 2);
      lost = lost || !mbar_wait(&S.s_ready[x], at.tiles & 1);
      __syncwarp();
      ++at.tiles;
      tc_fence_after();
      const int t0 = ps.tile0(i);
      // (MOD: whatever a lane without a row of the pass computes, nobody reads)
      const bool whole = (MOD && !ln.live) ||
                         (t0 + kTile <= ln.n && (t0 >= ln.first || t0 + kTile <= ln.sinks) && (!MOD || t0 >= ln.start));
      const bool masked = !__all_sync(0xffffffffu, whole) || bad;
      if (bad && lane == 0) atomicOr(p.status, kDevBadPage);
      auto mask = [&](uint32_t* s, int c0) {
        mask32<MOD>(s, ln.n - t0 - c0, ln.first - t0 - c0, ln.sinks - t0 - c0, ln.start - t0 - c0, bad >> (c0 / 16));
      };
      // largest exponent of 32 columns
      auto largest = [&](const uint32_t* s, int c0, float top) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          auto at = [&](int e) { return __uint_as_float(s[16 * g + e]); };
          float a = max3(at(0), at(1), at(2)), b = max3(at(3), at(4), at(5));
          a = max3(a, at(6), at(7));
          b = max3(b, at(8), at(9));
          a = max3(a, at(10), at(11));
          b = max3(b, at(12), at(13));
          a = max3(a, at(14), at(15));
          top = max3(top, a, b);
        }
        return top;
      };
      const Change ch{cap, inv_cap, ln.slope, ln.pos - t0};
      auto rough_path = [&](const float2* factors, bool keep) {
        const float2 ml = rough_tile<D, F8, MOD>(ts, to, make_float2(m, l), mul, ev, un_ev, factors,
                                                 make_int4(ln.n - t0, ln.first - t0, ln.sinks - t0, ln.start - t0), bad,
                                                 masked, i > ps.i0, keep, ch);
        m = ml.x;
        l = ml.y;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive_first<PAIR>(&S.p_ready[x][0]);
          arrive_first<PAIR>(&S.p_ready[x][1]);
        }
      };
      if (F8 && rough) {
        rough_path(factors, false);
        continue;
      }
      auto hand_over = [&](int half) {
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first<PAIR>(&S.p_ready[x][half]);
      };
      if constexpr ((MOD & (kCap | kBias)) != 0) {
        // A bound of the row's changed scores, cheaper than their maximum: while
        // it does not pass the running maximum, that stays, and change and
        // exponent go together. It is that of the largest magnitude (with a cap)
        // or product, columns that are not seen among them, and of the bias at
        // the tile's nearest (slope below 0: farthest) column. (Reading S twice, 32
        // columns ahead of their use, leaves more registers and is slower: 1001
        // against 873 us.)
        float bound = MOD & kCap ? 0.f : -INFINITY;
        uint32_t u[2][32];
        tmem_ld32(ts, u[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_ld_wait32(u[c & 1]);
          tmem_ld32(ts + 32 * (c + 1) % kTile, u[(c + 1) & 1]);  // at last the first again
          bound = MOD & kCap ? largest32(u[c & 1], bound) : largest(u[c & 1], 0, bound);
        }
        bool quick = true, nearest = false;
        float far = 0.f, most = 0.f;  // largest magnitude over the cap; the most that the bias adds
        if (MOD & kCap) {
          const float t = bound * (mul * inv_cap), y = t * t;
          far = t;
          nearest = __all_sync(0xffffffffu, !ln.live || t <= kNearest);
          quick = t <= kNear && in_products;
          bound = cap * (t * fmaf(fmaf(fmaf(tanh_near(3), y, tanh_near(2)), y, tanh_near(1)), y, tanh_near(0)));
        } else {
          bound *= mul;
        }
        float off = ev, slope = 0.f;
        if (MOD & kBias) {
          const float d0 = static_cast<float>(ch.ahead), d1 = d0 - (kTile - 1);
          const float lo = d1 > 0.f ? d1 : d0 < 0.f ? -d0 : 0.f, hi = fmaxf(d0, -d1);
          most = -ln.slope * (ln.slope >= 0.f ? lo : hi);
          bound += most;
          slope = d0 < 0.f ? -ln.slope : ln.slope;
          off = fmaf(-slope, d0, ev);
          quick = quick && !(d0 >= 0.f && d1 < 0.f && ln.n > ln.pos + 1);  // no keys on both sides of the position
        }
        tmem_ld_wait32(u[0]);
        if (!__all_sync(0xffffffffu, !ln.live || (quick && bound + ev <= m + kPassed<F8>))) {
          if (MOD & kCap && far > kNear) bound = fmaf(cap, tanh_far(far), most);
          rough_path(nullptr, __all_sync(0xffffffffu, !ln.live || bound + ev <= m + kPassed<F8>));
          continue;
        }
        off -= m == -INFINITY ? 0.f : m;
        const float x1 = MOD & kCap ? mul * inv_cap : mul;
        const uint64_t off_2 = pair(off, off), x_2 = pair(x1, x1), slope_2 = pair(slope, slope);
        uint64_t sum = pair(0.f, 0.f);
        // the polynomial in the scores themselves, or (e4m3, whose products are of any
        // size) in the scores over the cap
        auto coefficients = [&](auto& q_2, auto value) {
          constexpr int Q = sizeof(q_2) / sizeof(q_2[0]);
          float f = F8 ? cap : cap * x1;
#pragma unroll
          for (int j = 0; j < Q; ++j) {
            q_2[j] = pair(f * value(j), f * value(j));
            if (!F8) f *= x1 * x1;
          }
        };
        // Half by half. e4m3: one copy of the code for both, since the prep warps'
        // conversions take their share of the instruction cache (928 us with it, 974
        // without, softcap 50; bf16 770 and 754).
        auto go = [&](const auto& q_2, auto masks) {
          constexpr int Q = sizeof(q_2) / sizeof(q_2[0]);
          constexpr bool MASKED = decltype(masks)::value;
#pragma unroll(F8 ? 1 : 2)
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int c0 = 64 * half + 32 * c, at = t0 + c0;
              if (half || c) tmem_ld_wait32(u[c]);
              if (!half || !c) tmem_ld32(ts + c0 + 32, u[c ^ 1]);
              const uint32_t see =
                  MASKED ? seen32<MOD>(ln.n - at, ln.first - at, ln.sinks - at, ln.start - at, bad >> (c0 / 16)) : ~0u;
              sum = add2(sum, changed_weights32<F8, MOD, Q, MASKED>(u[c], c0, x_2, q_2, off_2, slope_2, see));
              tmem_st16(ts + c0 / 2, u[c]);
            }
            hand_over(half);
          }
        };
        if (MOD & kCap && !masked && nearest) {
          uint64_t q_2[3];
          coefficients(q_2, [](int j) { return tanh_nearest(j); });
          go(q_2, std::false_type());
        } else {
          uint64_t q_2[4];
          coefficients(q_2, [](int j) { return tanh_near(j); });
          if (masked)
            go(q_2, std::true_type());
          else
            go(q_2, std::false_type());
        }
        float a, b;
        unpair(sum, a, b);
        l = fmaf(a + b, un_ev, l);
        continue;
      }
      uint32_t s[kTile];
#pragma unroll
      for (int c = 0; c < kTile; c += 32) tmem_ld32(ts + c, s + c);
#pragma unroll
      for (int c = 0; c < kTile; c += 32) tmem_ld_wait32(s + c);
      if (masked) {
#pragma unroll
        for (int c = 0; c < kTile; c += 32) mask(s + c, c);
      }
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < kTile; c += 32) top = largest(s + c, c, top);
      top = fmaf(top, mul, ev);
      const bool up = top > m + kPassed<F8>;
      if (__any_sync(0xffffffffu, up)) {
        top -= kLift<F8>;
        const float f = up ? (m == -INFINITY ? 0.f : ex2(m - top)) : 1.f;
        if (up) m = top;
        l *= f;
        if (i > ps.i0) rescale_o<D>(to, f);
      }
      const float base = m == -INFINITY ? 0.f : m;
      // weights of 32 columns in 16 bits (relative error 2^-8, as the output's own
      // rounding; f16 2^-11 and the absolute term of kLift), over the scores' TMEM
      // columns
      float tile_l = 0.f;
      auto weights = [&](uint32_t* s, int c0) {
        uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
        const float off = ev - base;
        float a, b;
        const uint64_t mul2 = pair(mul, mul), off2 = pair(off, off);
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          unpair(fma2(pair(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), mul2, off2), a, b);
          a = ex2(a);
          b = ex2(b);
          sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pair(a, b));
          s[c / 2] = F8 ? pack_f16(a, b) : pack_bf16(a, b);
        }
        unpair(add2(sum[0], sum[1]), a, b);
        tile_l += a + b;
        tmem_st16(ts + c0 / 2, s);
      };
      weights(s, 0);
      weights(s + 32, 32);
      hand_over(0);
      weights(s + 64, 64);
      weights(s + 96, 96);
      hand_over(1);
      l = fmaf(tile_l, un_ev, l);
    }
    lost = lost || !mbar_wait(&S.o_done[x], at.passes & 1);
    __syncwarp();
    ++at.passes;
    tc_fence_after();
    if (MOD) place();
    bool extra = *reinterpret_cast<volatile int*>(&S.nonfinite) != 0;
    if (PAIR == 2) {
      int other;
      asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(other) : "r"(peer_addr(&S.nonfinite, rank ^ 1)) : "memory");
      extra = extra || other != 0;
    }
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t u[32];
      tmem_ld32(to + c, u);
      tmem_ld_wait32(u);
      float o[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(u[e]);
      if (extra) {
        float t[32];  // o itself stays in registers: only what is passed by address lives in memory
#pragma unroll
        for (int e = 0; e < 32; ++e) t[e] = o[e];
        add_nonfinite<D, F8, MOD>(p, get_pass<MOD>(S, L, seg), pc.kvh, ln, m, c, t);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = t[e];
      }
      write_columns<D, MOD>(p, ln, part, l, c, o, S.stage[warp]);
    }
    tc_fence_before();
    write_sums(p, ln, part, m, l);
  }
  return !lost;
}

// ---------------------------------------------------------------------- TMA
template <int MOD, int D, bool F8>
__device__ __forceinline__ bool tma_role(Shared<D, F8>& S, const TilesLaunch& L, const CUtensorMap* qmap,
                                         const CUtensorMap* kmap, const CUtensorMap* vmap, int rank, Progress& progress) {
  const Piece& pc = S.piece;
  using Sh = Shared<D, F8>;
  constexpr int PAIR = kPair<D>, kStages = Sh::kStages, kRaw = F8 ? Sh::kRaw : 1;
  const AttnLaunch& p = L.a;
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
    // bf16: the MMA waits for both CTAs' queries; e4m3: each CTA converts its own first
    const uint32_t bar = F8 ? smem_u32(&S.q_full) : first_cta<PAIR>(&S.q_full);
    const int bytes = 2 * Sh::kSlabs * L.rows_per_tile * p.group * 128;
    if (F8)
      mbar_arrive_expect_tx(&S.q_full, bytes);
    else if (rank == 0)
      mbar_arrive_expect_tx(&S.q_full, PAIR * bytes);
    for (int x = 0; x < 2; ++x)
      for (int c = 0; c < Sh::kSlabs; ++c)
        tma_3d<PAIR>(S.q[x] + c * kTile * 128, qmap, 64 * c, pc.kvh * p.group,
                     pc.row0 + (x * PAIR + rank) * L.rows_per_tile, bar);
  }
  const int bs = 1 << p.c.bs_log2;
  const int k_box = min(bs, Sh::kKeys);  // keys of one K copy; a V copy takes a block
  int& done = progress.tiles;
  for (int seg = 0; seg < S.segs; ++seg) {
    const Pass<MOD> ps = get_pass<MOD>(S, L, seg);
    // block of the lane's copy, copies being `box` keys each; -1: none. A bad
    // block is read as the one past the end, which the copy fills with zeros.
    auto block_of = [&](int i, int box) -> int {
      if (i >= ps.i1 || lane >= kTile / box) return -1;
      const int t = ps.tile0(i) + lane * box;
      if (t >= ps.most) return -1;
      const int blk = p.block_table[ps.batch * p.bt_stride + (t >> p.c.bs_log2)];
      return blk < 0 || blk >= p.c.num_blocks ? static_cast<int>(p.c.num_blocks) : blk;
    };
    int next_k = block_of(ps.i0, k_box), next_v = block_of(ps.i0, bs);
    for (int i = ps.i0; i < ps.i1; ++i, ++done) {
      const int blk[2] = {next_k, next_v};
      next_k = block_of(i + 1, k_box);
      next_v = block_of(i + 1, bs);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int box = kv ? bs : k_box;
        const bool mine = blk[kv] >= 0 && (kv || PAIR == 1 || lane * box / Sh::kKeys == rank);
        // bf16 keys report to the first CTA, which expects both CTAs' bytes
        const bool shared = !F8 && !kv;
        const int copies = __popc(__ballot_sync(0xffffffffu, shared ? blk[kv] >= 0 : mine));
        const int bytes = copies * box * (kv ? Sh::kDims : D) * (F8 ? 1 : 2);
        uint64_t *empty, *full;
        unsigned char* dst;
        uint32_t ph;
        const int at = kv ? lane * box : lane * box % Sh::kKeys;  // row of the copy in the tile
        if (F8) {
          const int idx = 2 * done + kv, st = idx % kRaw;
          empty = &S.raw_empty[st];
          full = &S.raw_full[st];
          dst = S.raw[st] + at * (kv ? Sh::kDims : D);
          ph = (idx / kRaw) & 1;
        } else {
          const int st = done % kStages;
          empty = kv ? &S.v_empty[st] : &S.k_empty[st];
          full = kv ? &S.v_full[st] : &S.k_full[st];
          dst = (kv ? S.v[st] : S.k[st]) + at * 128;
          ph = (done / kStages) & 1;
        }
        const bool ok = mbar_wait(empty, ph ^ 1);
        if (!__all_sync(0xffffffffu, ok)) return false;
        if (lane == 0 && (!shared || rank == 0)) mbar_arrive_expect_tx(full, bytes);
        __syncwarp();
        if (mine) {
          const uint32_t bar = shared ? first_cta<PAIR>(full) : smem_u32(full);
          const int tok = lane * box & (bs - 1);
          if (kv)
            tma_4d<PAIR>(dst, vmap, Sh::kDims * rank, 0, pc.kvh, blk[kv], bar);
          else if (F8)
            tma_4d<PAIR>(dst, kmap, 0, tok, pc.kvh, blk[kv], bar);
          else
#pragma unroll
            for (int c = 0; c < Sh::kSlabs; ++c)
              tma_4d<PAIR>(dst + c * Sh::kKeys * 128, kmap, 64 * c, tok, pc.kvh, blk[kv], bar);
        }
      }
    }
  }
  return true;
}

// ---------------------------------------------------------------------- MMA
template <int MOD, int D, bool F8>
__device__ __forceinline__ bool mma_role(Shared<D, F8>& S, const TilesLaunch& L, Progress& progress) {
  using Sh = Shared<D, F8>;
  constexpr int PAIR = kPair<D>, kStages = Sh::kStages;
  constexpr uint32_t kF16 = F8 ? (1u << 7) | (1u << 10) : 0u;  // format fields: 1 bf16, 0 f16
  constexpr uint32_t kIdescQk = umma_idesc_bf16(kTile * PAIR, kTile) ^ kF16;
  constexpr uint32_t kIdescPv = (umma_idesc_bf16(kTile * PAIR, D) ^ kF16) | kTransposeB;
  const uint32_t tmem = S.tmem;
  // The whole warp walks the loop, so that descriptors stay in uniform
  // registers, and one thread issues.
  const uint32_t q_lo = desc_lo(smem_u32(S.q[0])), k_lo = desc_lo(smem_u32(S.k[0])), v_lo = desc_lo(smem_u32(S.v[0]));
  const bool lead = elect_one();
  // A wait that gives up does not leave the loop, which would split the warp:
  // the rest runs through without waiting, on whatever is in the buffers, and the
  // piece is reported.
  bool lost = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) { lost = lost || !mbar_wait(bar, parity); };
  auto qk = [&](int x, int st) {
    if (!lead) return;
    const uint32_t a = q_lo + x * (Sh::kQBytes >> 4), b = k_lo + st * (Sh::kKBytes >> 4);
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      umma_ss<PAIR>(tmem + kColS + 128 * x, a + (((s / 4) * kTile * 128 + (s % 4) * 32) >> 4),
                    b + (((s / 4) * Sh::kKeys * 128 + (s % 4) * 32) >> 4), kIdescQk, s > 0);
    commit_all<PAIR>(&S.s_ready[x]);
  };
  auto pv = [&](int x, int st, int half, bool first) {
    if (!lead) return;
    const uint32_t b = v_lo + st * (Sh::kVBytes >> 4);
#pragma unroll
    for (int s = 4 * half; s < 4 * half + 4; ++s)
      umma_ts<PAIR>(tmem + kColO + 128 * x, tmem + kColS + 128 * x + 8 * s, b + ((s * 2048) >> 4), kIdescPv,
                    !(first && s == 0));
  };
  wait(F8 ? &S.q_ready : &S.q_full, progress.pieces & 1);
  int& done = progress.tiles;
  int(&p_done)[2] = progress.weights;
  for (int seg = 0; seg < S.segs; ++seg) {
    const Pass<MOD> ps = get_pass<MOD>(S, L, seg);
    const int n = ps.i1 - ps.i0;
    if (n == 0) continue;
    wait(&S.k_full[done % kStages], (done / kStages) & 1);
    tc_fence_after();
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (ps.act[x]) qk(x, done % kStages);
    if (lead) commit_all<PAIR>(&S.k_empty[done % kStages]);
    for (int i = 0; i < n; ++i, ++done) {
      const int st = done % kStages, nst = (done + 1) % kStages;
      const bool more = i + 1 < n;
      bool k_there = false;
      wait(&S.v_safe[st], (done / kStages) & 1);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!ps.act[x]) continue;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          wait(&S.p_ready[x][half], p_done[x] & 1);
          tc_fence_after();
          pv(x, st, half, i == 0);
        }
        ++p_done[x];
        if (lead && (x == 1 || !ps.act[1])) commit_all<PAIR>(&S.v_empty[st]);
        if (more) {
          if (!k_there) wait(&S.k_full[nst], ((done + 1) / kStages) & 1);
          k_there = true;
          tc_fence_after();
          qk(x, nst);
        } else if (lead) {
          commit_all<PAIR>(&S.o_done[x]);
        }
      }
      if (lead && more) commit_all<PAIR>(&S.k_empty[nst]);
    }
  }
  if (lost) {  // let the products in flight end before their memory goes
    const unsigned long long t = global_timer_ns();
    while (global_timer_ns() - t < 200000ull) {
    }
  }
  return !lost;
}

// --------------------------------------------------------------------- prep
template <int MOD, int D>
__device__ __forceinline__ bool prep_role(Shared<D, false>& S, const TilesLaunch& L, int, Progress& progress) {
  const AttnLaunch& p = L.a;
  constexpr int PAIR = kPair<D>, kStages = Shared<D, false>::kStages;
  const int tid = threadIdx.x - kPrepWarp * 32;
  int& done = progress.tiles;
  bool lost = false;
  for (int seg = 0; seg < S.segs; ++seg) {
    const Pass<MOD> ps = get_pass<MOD>(S, L, seg);
    for (int i = ps.i0; i < ps.i1; ++i, ++done) {
      const int st = done % kStages;
      lost = lost || !mbar_wait(&S.v_full[st], (done / kStages) & 1);
      __syncwarp();
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
            for (int e = 0; e < 2; ++e) {
              const uint4 x = *reinterpret_cast<const uint4*>(at + e * 16);
              bad = bad || nonfinite2(x.x) || nonfinite2(x.y) || nonfinite2(x.z) || nonfinite2(x.w);
            }
          }
          const uint32_t b = __ballot_sync(0xffffffffu, bad);
          if ((b >> (threadIdx.x & 28)) & 0xfu) {
            zero = true;
            *reinterpret_cast<volatile int*>(&S.nonfinite) = 1;
          }
          if (zero) {
#pragma unroll
            for (int e = 0; e < 2; ++e) *reinterpret_cast<uint4*>(at + e * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();  // the MMA reads these stores through the async proxy
      }
      __syncwarp();
      if ((threadIdx.x & 31) == 0) arrive_first<PAIR>(&S.v_safe[st]);
    }
  }
  return !lost;
}

// e4m3: 16-code pieces of a raw tile (ROWS rows of ROW codes) to halves in the
// MMA's layout: 128-byte swizzled rows of 64 dims, slabs of ROWS rows. The
// lanes of one row read its pieces; a piece becomes two 16-byte chunks, written
// in an order that keeps the eight lanes of a store on different banks. Lane
// `lane0` + g of the warp has the power of two of the rows 16g to 16g + 15
// (SHIFT; without, all of them are 1). `check`: rows from `dead` on and rows with
// a NaN become 0; returns whether there was a NaN.
template <int ROWS, int ROW, bool SHIFT>
__device__ __forceinline__ bool codes_to_halves(const uint4* raw, unsigned char* out, uint32_t tid, uint32_t power,
                                                int lane0, bool check, int dead) {
  constexpr uint32_t kPieces = ROW / 16, kStep = kPrepWarps * 32, kRowStep = kStep / kPieces;
  static_assert(ROWS * kPieces == 8 * kStep && kRowStep % 8 == 0, "eight pieces per thread, alike in swizzle");
  const uint32_t piece = tid % kPieces, row0 = tid / kPieces;
  const uint32_t odd = kPieces == 8 ? piece >> 2 : 0;  // dims above 64 write their second chunk first
  const uint32_t c0 = 2 * (piece & 3) + odd;
  unsigned char* first = out + (piece / 4) * ROWS * 128 + row0 * 128 + ((c0 ^ (row0 & 7)) << 4);
  unsigned char* second = out + (piece / 4) * ROWS * 128 + row0 * 128 + (((c0 ^ 1) ^ (row0 & 7)) << 4);
  bool met = false;
#pragma unroll 1
  for (uint32_t j0 = 0; j0 < 8; j0 += 4) {
    uint4 x[4];
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) x[j] = raw[j * kStep + tid];
    raw += 4 * kStep;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
      uint4 c = x[j];
      if (check) {
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        bool nan = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t y = (w[e] & 0x7f7f7f7fu) ^ 0x7f7f7f7fu;  // a zero byte: NaN
          nan = nan || (((y - 0x01010101u) & ~y & 0x80808080u) != 0u);
        }
        bool zero = static_cast<int>((j0 + j) * kRowStep + row0) >= dead;
        const uint32_t b = __ballot_sync(0xffffffffu, nan && !zero);
        if ((b >> ((tid & 31) / kPieces * kPieces)) & ((1u << kPieces) - 1u)) zero = met = true;
        if (zero) c = make_uint4(0, 0, 0, 0);
      }
      uint4 a, b;
      e4m3x4_f16x4(c.x, a.x, a.y);
      e4m3x4_f16x4(c.y, a.z, a.w);
      e4m3x4_f16x4(c.z, b.x, b.y);
      e4m3x4_f16x4(c.w, b.z, b.w);
      if (SHIFT) {
        const uint32_t f = __shfl_sync(0xffffffffu, power, lane0 + (j0 + j) * kRowStep / 16);
        mul_f16x2(a.x, f);
        mul_f16x2(a.y, f);
        mul_f16x2(a.z, f);
        mul_f16x2(a.w, f);
        mul_f16x2(b.x, f);
        mul_f16x2(b.y, f);
        mul_f16x2(b.z, f);
        mul_f16x2(b.w, f);
      }
      *reinterpret_cast<uint4*>(first + j * kRowStep * 128) = odd ? b : a;
      *reinterpret_cast<uint4*>(second + j * kRowStep * 128) = odd ? a : b;
    }
    first += 4 * kRowStep * 128;
    second += 4 * kRowStep * 128;
  }
  return met;
}

template <int MOD, int D>
__device__ __forceinline__ bool prep_role(Shared<D, true>& S, const TilesLaunch& L, int rank, Progress& progress) {
  using Sh = Shared<D, true>;
  constexpr int PAIR = kPair<D>, kRaw = Sh::kRaw, kStages = Sh::kStages;
  const AttnLaunch& p = L.a;
  const int tid = threadIdx.x - kPrepWarp * 32, lane = threadIdx.x & 31;
  const int kvh = S.piece.kvh;
  int& done = progress.tiles;
  bool lost = false;
  for (int seg = 0; seg < S.segs; ++seg) {
    const Pass<MOD> ps = get_pass<MOD>(S, L, seg);
    // lanes 0-7: block of the tile's 16-key group, read two tiles ahead, and its
    // scales, read one ahead
    auto block_of = [&](int i) -> int {
      if (i >= ps.i1 || lane >= 8) return -1;
      const int t = ps.tile0(i) + 16 * lane;
      if (t >= ps.most) return -1;
      return p.block_table[ps.batch * p.bt_stride + (t >> p.c.bs_log2)];
    };
    auto exponents_of = [&](int blk) -> int2 {
      if (blk < 0 || blk >= p.c.num_blocks) return make_int2(kNoScale, kNoScale);
      const long long at = static_cast<long long>(blk) * p.c.heads + kvh;
      return make_int2(exponent_of(p.c.ks[at]), exponent_of(p.c.vs[at]));
    };
    int blk1 = block_of(ps.i0 + 1);
    int2 ex = exponents_of(block_of(ps.i0));
    // 2^(e - E) as two halves, of this lane's 16 keys (a group without a block: 1)
    auto shift_of = [&](int e) -> uint32_t {
      const int top = max(kLeastExp, __reduce_max_sync(0xffffffffu, e));
      const int d = e == kNoScale ? 0 : max(kLeastShift, e - top);
      return static_cast<uint32_t>(15 + d) << 10 | static_cast<uint32_t>(15 + d) << 26;
    };
    for (int i = ps.i0; i < ps.i1; ++i, ++done) {
      const uint32_t k_power = shift_of(ex.x), v_power = shift_of(ex.y);
      ex = exponents_of(blk1);
      blk1 = block_of(i + 2);
      const int t0 = ps.tile0(i), st = done % kStages;
      const bool check = ps.partial(t0, p);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int idx = 2 * done + kv, rs = idx % kRaw;
        lost = lost || !mbar_wait(&S.raw_full[rs], (idx / kRaw) & 1);
        lost = lost || !mbar_wait(kv ? &S.v_empty[st] : &S.k_empty[st], ((done / kStages) & 1) ^ 1);
        __syncwarp();
        const uint4* raw = reinterpret_cast<const uint4*>(S.raw[rs]);
        constexpr uint32_t kOne = 0x3c003c00u;
        if (kv) {
          const bool met = __any_sync(0xffffffffu, v_power != kOne)
                               ? codes_to_halves<kTile, Sh::kDims, true>(raw, S.v[st], tid, v_power, 0, check, ps.most - t0)
                               : codes_to_halves<kTile, Sh::kDims, false>(raw, S.v[st], tid, 0, 0, check, ps.most - t0);
          if (met) *reinterpret_cast<volatile int*>(&S.nonfinite) = 1;
        } else if (__any_sync(0xffffffffu, k_power != kOne)) {
          codes_to_halves<Sh::kKeys, D, true>(raw, S.k[st], tid, k_power, rank * (Sh::kKeys / 16), false, 0);
        } else {
          codes_to_halves<Sh::kKeys, D, false>(raw, S.k[st], tid, 0, 0, false, 0);
        }
        fence_proxy_async_smem();  // the MMA reads these stores through the async proxy
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&S.raw_empty[rs]);
          arrive_first<PAIR>(kv ? &S.v_safe[st] : &S.k_full[st]);
        }
      }
    }
  }
  return !lost;
}

// The row tiles' weights, summed up, in S.deal (every CTA computes the same);
// the number of shares behind them.
template <int MOD, int D, bool F8>
__device__ __forceinline__ void deal_units(Shared<D, F8>& S, const TilesLaunch& L, int most_shares) {
  const AttnLaunch& p = L.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows_here = 2 * kPair<D> * L.rows_per_tile;
  for (int t = warp; t < L.row_tiles; t += kThreads / 32) {
    int most = 0, low = INT_MAX;
    for (int i = lane; i < rows_here && t * rows_here + i < p.rows; i += 32) {
      const int n = p.seq_lens[t * rows_here + i];
      if (MOD) {
        const RowSpan span = row_span(p, t * rows_here + i, n);
        if (span.good && n > 0) {
          most = max(most, span.end);
          low = min(low, span.first);
        }
      } else if (n > 0 && n <= p.max_len) {
        most = max(most, n);
        low = min(low, p.window > 0 ? max(0, n - p.window) : 0);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
      low = min(low, __shfl_xor_sync(0xffffffffu, low, o));
    }
    // at most 2^20, so that kMaxDealt of them fit 32 bits (a step is then several tiles)
    if (lane == 0) S.deal[t + 1] = kUnitWeight + (most > 0 ? min((most + kTile - 1) / kTile - low / kTile, 1 << 20) : 0);
  }
  __syncthreads();
  if (warp == 0) {
    int sum = 0;
    for (int t0 = 0; t0 < L.row_tiles; t0 += 32) {
      const int t = t0 + lane;
      int x = t < L.row_tiles ? S.deal[t + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (t < L.row_tiles) S.deal[t + 1] = sum + x;
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
      S.deal[0] = 0;
      const long long total = static_cast<long long>(sum) * p.c.heads;
      const int shares = static_cast<int>(max(1LL, min(static_cast<long long>(most_shares), total / kLeastShare)));
      S.deal[L.row_tiles + 1] = shares;
      if (blockIdx.x == 0) L.borders[0] = make_int4(shares, sum, 0, 0);
    }
  }
  __syncthreads();
}

// The piece that holds this CTA's (pair's) step `step` of its share [.., end);
// moves `step` to the next piece.
template <int D, bool F8>
__device__ __forceinline__ Piece next_piece(const Shared<D, F8>& S, const TilesLaunch& L, int share, long long& step,
                                            long long begin, long long end) {
  const int sum = S.deal[L.row_tiles];
  Piece pc;
  pc.kvh = static_cast<int>(step / sum);
  const int in_head = static_cast<int>(step - static_cast<long long>(pc.kvh) * sum);
  int lo = 0, hi = L.row_tiles - 1;  // the row tile with deal[t] <= in_head < deal[t + 1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (S.deal[mid] <= in_head)
      lo = mid;
    else
      hi = mid - 1;
  }
  const long long a = static_cast<long long>(pc.kvh) * sum + S.deal[lo];
  pc.of = S.deal[lo + 1] - S.deal[lo];
  pc.row0 = lo * 2 * kPair<D> * L.rows_per_tile;
  pc.from = static_cast<int>(step - a);
  pc.to = static_cast<int>(min(static_cast<long long>(pc.of), end - a));
  pc.slot = pc.from == 0 && pc.to == pc.of ? -1 : 2 * share + (a <= begin ? 0 : 1);
  step = a + pc.to;
  return pc;
}

// The rows of the piece: lengths, and the runs of one request. Both CTAs of a
// pair look at all its rows. Every thread calls it; ends with a barrier.
template <int D, bool F8>
__device__ __forceinline__ void set_up_rows(Shared<D, F8>& S, const TilesLaunch& L) {
  const Piece& pc = S.piece;
  constexpr int kRows = kMaxRows<D>, kGroups = kRows / 32;
  const AttnLaunch& p = L.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows_here = 2 * kPair<D> * L.rows_per_tile;
  if (tid == 0) S.nonfinite = 0;
  for (int i = tid; i < kRows; i += kThreads) {
    int n = 0, b = -1;
    const int row = pc.row0 + i;
    if (i < rows_here && row < p.rows) {
      n = p.seq_lens[row];
      b = p.row_to_batch[row];
      if (n < 0 || n > p.max_len || b < 0 || b >= p.bt_rows ||
          ((static_cast<long long>(n) - 1) >> p.c.bs_log2) >= p.bt_stride) {
        atomicOr(p.status, kDevBadRowMeta);
        n = 0;
        b = -1;
      }
    }
    S.row_n[i] = n;
    S.row_b[i] = b;
    S.seg_most[i] = 0;
    S.seg_least[i] = S.seg_low[i] = INT_MAX;
  }
  named_bar(kSetUpBar, kThreads);
  for (int w = warp; w < kGroups; w += kThreads / 32) {
    const int i = 32 * w + lane;
    const uint32_t starts = __ballot_sync(0xffffffffu, i < rows_here && (i == 0 || S.row_b[i - 1] != S.row_b[i]));
    if (lane == 0) S.warp_starts[w] = __popc(starts);
  }
  named_bar(kSetUpBar, kThreads);
  for (int w = warp; w < kGroups; w += kThreads / 32) {
    const int i = 32 * w + lane;
    const bool start = i < rows_here && (i == 0 || S.row_b[i - 1] != S.row_b[i]);
    const uint32_t starts = __ballot_sync(0xffffffffu, start);
    int id = -1;
    for (int v = 0; v < w; ++v) id += S.warp_starts[v];
    id += __popc(starts & ((2u << lane) - 1u));
    if (start) S.seg_start[id] = i;
    if (i == rows_here - 1) {
      S.segs = id + 1;
      S.seg_start[id + 1] = rows_here;
    }
    const int n = S.row_n[i];
    if (i < rows_here && n > 0) {
      atomicMax(&S.seg_most[id], n);
      atomicMin(&S.seg_least[id], n);
      atomicMin(&S.seg_low[id], p.window > 0 ? max(0, n - p.window) : 0);
    }
  }
  named_bar(kSetUpBar, kThreads);
}

// The same with documents and prefixes; a thread's rows' spans stay in registers
// over the steps.
template <int D, bool F8>
__device__ __forceinline__ void set_up_spans(Shared<D, F8>& S, const TilesLaunch& L) {
  const Piece& pc = S.piece;
  constexpr int kRows = kMaxRows<D>, kGroups = kRows / 32;
  const AttnLaunch& p = L.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows_here = 2 * kPair<D> * L.rows_per_tile;
  // bounds of the segments' keys, where rows leave later: least length, least and
  // highest first key, least and highest first token before the former's tile
  int(*bounds)[kRows] = reinterpret_cast<int(*)[kRows]>(S.stage);
  static_assert(5 * kRows * sizeof(int) <= sizeof(S.stage), "bounds fit");
  int *least = bounds[0], *low = bounds[1], *high = bounds[2], *first = bounds[3], *behind = bounds[4];
  if (tid == 0) S.nonfinite = 0;
  constexpr int kTurns = (kRows + kThreads - 1) / kThreads;
  RowSpan spans[kTurns];  // of the rows tid + t * kThreads
#pragma unroll
  for (int t = 0; t < kTurns; ++t) {
    const int i = tid + t * kThreads;
    if (i >= kRows) break;
    int n = 0, b = -1;
    const int row = pc.row0 + i;
    if (i < rows_here && row < p.rows) {
      n = p.seq_lens[row];
      b = p.row_to_batch[row];
      spans[t] = row_span(p, row, n);
      n = spans[t].good ? spans[t].end : -1;
      if (n < 0 || b < 0 || b >= p.bt_rows ||
          ((static_cast<long long>(n) - 1) >> p.c.bs_log2) >= p.bt_stride) {
        atomicOr(p.status, kDevBadRowMeta);
        n = 0;
        b = -1;
      }
      if (spans[t].start == spans[t].end) n = 0;  // sees nothing
    }
    S.row_n[i] = n;
    S.row_b[i] = b;
    S.seg_most[i] = 0;
    least[i] = low[i] = first[i] = INT_MAX;
    high[i] = behind[i] = 0;
  }
  named_bar(kSetUpBar, kThreads);
  for (int w = warp; w < kGroups; w += kThreads / 32) {
    const int i = 32 * w + lane;
    const uint32_t starts = __ballot_sync(0xffffffffu, i < rows_here && (i == 0 || S.row_b[i - 1] != S.row_b[i]));
    if (lane == 0) S.warp_starts[w] = __popc(starts);
  }
  named_bar(kSetUpBar, kThreads);
  int ids[kTurns];  // segments of this thread's rows
#pragma unroll
  for (int t = 0; t < kTurns; ++t) {
    const int w = warp + t * (kThreads / 32);
    if (w >= kGroups) break;
    const int i = 32 * w + lane;
    const bool start = i < rows_here && (i == 0 || S.row_b[i - 1] != S.row_b[i]);
    const uint32_t starts = __ballot_sync(0xffffffffu, start);
    int id = -1;
    for (int v = 0; v < w; ++v) id += S.warp_starts[v];
    id += __popc(starts & ((2u << lane) - 1u));
    ids[t] = id;
    if (start) S.seg_start[id] = i;
    if (i == rows_here - 1) {
      S.segs = id + 1;
      S.seg_start[id + 1] = rows_here;
    }
    const int n = S.row_n[i];
    if (i < rows_here && n > 0) {
      atomicMax(&S.seg_most[id], n);
      atomicMin(&least[id], n);
      atomicMin(&low[id], spans[t].first);
      atomicMax(&high[id], spans[t].first);
    }
  }
  named_bar(kSetUpBar, kThreads);
  if (p.window > 0 && p.sinks > 0) {
    // First tokens in the window's tiles, a later document's say, are walked anyway.
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
      const int i = tid + t * kThreads;
      if (i >= rows_here || S.row_n[i] <= 0) continue;
      const RowSpan& span = spans[t];
      if (span.sinks_end > span.start && span.start / kTile < low[ids[t]] / kTile) {
        atomicMin(&first[ids[t]], span.start);
        atomicMax(&behind[ids[t]], span.sinks_end);
      }
    }
    named_bar(kSetUpBar, kThreads);
  }
  for (int g = tid; g < S.segs; g += kThreads) {
    Segment sg{0, 0, 0, 0, 0};
    const int most = S.seg_most[g];
    if (most > 0) {
      sg.low_tile = low[g] / kTile;
      sg.high_tiles = (high[g] + kTile - 1) / kTile - sg.low_tile;
      sg.base_tile = min(first[g] / kTile, sg.low_tile);
      sg.first_tiles = min((behind[g] + kTile - 1) / kTile, sg.low_tile) - sg.base_tile;
      sg.least_tiles = (most + kTile - 1) / kTile - least[g] / kTile;
    }
    pack_segment(sg, S.seg_start[g], S.seg_least[g], S.seg_low[g]);
  }
  named_bar(kSetUpBar, kThreads);
}

template <int D, bool F8, int MOD>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tiles_kernel(const __grid_constant__ TilesLaunch L, const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ unsigned char raw[];
  using Sh = Shared<D, F8>;
  constexpr int PAIR = kPair<D>;
  Sh& S = *reinterpret_cast<Sh*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const AttnLaunch& p = L.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = PAIR == 2 ? static_cast<int>(cta_rank()) : 0;

  if (tid == 0) {
    mbar_init(&S.q_full, 1);
    mbar_init(&S.q_ready, kSoftmaxWarps * PAIR);
    for (int i = 0; i < Sh::kStages; ++i) {
      mbar_init(&S.k_full[i], F8 ? kPrepWarps * PAIR : 1);
      mbar_init(&S.k_empty[i], 1);
      mbar_init(&S.v_full[i], 1);
      mbar_init(&S.v_empty[i], 1);
      mbar_init(&S.v_safe[i], kPrepWarps * PAIR);
    }
    for (int i = 0; i < Sh::kRaw; ++i) {
      mbar_init(&S.raw_full[i], 1);
      mbar_init(&S.raw_empty[i], kPrepWarps);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&S.s_ready[x], 1);
      mbar_init(&S.p_ready[x][0], 4 * PAIR);
      mbar_init(&S.p_ready[x][1], 4 * PAIR);
      mbar_init(&S.o_done[x], 1);
    }
    S.stop = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_take<PAIR>(&S.tmem);
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  const int group = blockIdx.x / PAIR;  // CTA, or pair
  if (L.dealt) deal_units<MOD>(S, L, gridDim.x / PAIR);
  if (tid == 0) {
    S.more = 1;
    if (!L.dealt) {
      // the last rows first: with causal lengths they have the most keys
      S.piece = Piece{group % p.c.heads, (L.row_tiles - 1 - group / p.c.heads) * 2 * PAIR * L.rows_per_tile, 0, 1, 1, -1};
    } else {
      const int shares = S.deal[L.row_tiles + 1];
      const long long total = static_cast<long long>(S.deal[L.row_tiles]) * p.c.heads;
      S.more = group < shares;
      S.step = S.begin = share_start(group, total, shares);
      S.end = share_start(group + 1, total, shares);
      if (group < shares) {
        S.piece = next_piece(S, L, group, S.step, S.begin, S.end);
        const Piece& pc = S.piece;
        if (rank == 0 && group > 0)
          L.borders[group] = make_int4(pc.kvh, pc.row0 / (2 * PAIR * L.rows_per_tile), pc.from, pc.of);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR == 2) cluster_sync();  // the other CTA's barriers are set up
  tc_fence_after();

  // Piece by piece; `role` is one role's work on one.
  auto pieces = [&](auto role) {
    Progress at;
    while (S.more) {
      if constexpr (MOD != 0)
        set_up_spans(S, L);
      else
        set_up_rows(S, L);
      const bool ok = role(at);
      ++at.pieces;
      if (!ok) {
        // both CTAs of a pair stop after this piece
        atomicOr(p.status, kDevWaitTimeout);
        S.stop = 1;
        if (PAIR == 2)
          asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(peer_addr(&S.stop, rank ^ 1)), "r"(1) : "memory");
      }
      __syncwarp();
      tc_fence_before();
      named_bar(kSetUpBar, kThreads);
      // neither CTA goes on, or ends, while the other may still read or signal it
      if (PAIR == 2) cluster_sync();
      tc_fence_after();
      if (!L.dealt) break;
      if (tid == 0) {
        S.more = S.step < S.end && !S.stop;
        if (S.more) S.piece = next_piece(S, L, group, S.step, S.begin, S.end);
      }
      named_bar(kSetUpBar, kThreads);
    }
  };
  // the softmax warps hold a row of S (128 registers); the others give up what
  // they take beyond the launch's share: 2 * 200 + 104 = 3 * 168
  if (warp < kSoftmaxWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    pieces([&](Progress& at) { return softmax_role<D, F8, MOD>(S, L, warp >> 2, rank, at); });
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    pieces([&](Progress& at) {
      if (warp == kTmaWarp) return tma_role<MOD>(S, L, &qmap, &kmap, &vmap, rank, at);
      if (warp == kMmaWarp) return rank != 0 || mma_role<MOD>(S, L, at);
      return prep_role<MOD>(S, L, rank, at);
    });
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_give<PAIR>(S.tmem);
  }
  if (L.dealt) pdl_trigger();
}

// Joins the units that were cut: block (j, i) does rows and heads 4j to 4j + 3,
// one warp each, of the unit that share i + 1 begins inside of, if that is
// the unit's first cut.
template <int D>
__global__ void __launch_bounds__(128) attn_tiles_join_kernel(const __grid_constant__ TilesLaunch L) {
  const AttnLaunch& p = L.a;
  const int rows_here = 2 * kPair<D> * L.rows_per_tile, lane = threadIdx.x & 31;
  const int first = blockIdx.y;
  const int item = blockIdx.x * 4 + (threadIdx.x >> 5);
  pdl_wait();
  const int4 head4 = L.borders[0], cut = L.borders[first + 1];
  const int shares = head4.x, sum = head4.y, kvh = cut.x;
  if (first + 1 >= shares || cut.z == 0 || item >= rows_here * p.group) return;
  const long long total = static_cast<long long>(sum) * p.c.heads;
  const long long a = share_start(first + 1, total, shares) - cut.z, b = a + cut.w;  // the unit's steps
  if (a < share_start(first, total, shares)) return;  // an earlier share cut it first
  const int last = share_of(b - 1, total, shares);
  const int row = cut.y * rows_here + item / p.group;
  if (row >= p.rows) return;
  auto slot = [&](int share) { return 2 * share + (a <= share_start(share, total, shares) ? 0 : 1); };
  constexpr int V = D / 32;
  float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
  for (int j = 0; j < V; ++j) o[j] = 0.f;
  const long long items = static_cast<long long>(rows_here) * p.group;
  for (int i = first; i <= last; ++i) m = fmaxf(m, p.part_ml[slot(i) * items + item].x);
  const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 2
  for (int i = first; i <= last; ++i) {
    const long long at = slot(i) * items + item;
    const float2 x = p.part_ml[at];
    const float f = x.y != x.y ? x.y : (x.x == -INFINITY ? 0.f : ex2(x.x - base));
    l += f * x.y;
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] += f * p.part_o[at * D + lane * V + j];
  }
  const long long head = static_cast<long long>(row) * p.q_heads + kvh * p.group + item % p.group;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + head * D + lane * V);
#pragma unroll
  for (int j = 0; j < V; j += 2) dst[j / 2] = pack_bf16(o[j] * inv, o[j + 1] * inv);
  if (lane == 0 && p.lse) p.lse[head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// 4-D map of a cache: (dim, token, head, block), boxes of `dims` dims of up to
// `keys` tokens of a block. bf16: in the MMA's 128-byte swizzled layout; codes:
// plain rows for the prep warps.
bool cache_map(CUtensorMap* map, const void* base, const CacheView& c, const long long* st, int dims, int keys) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t bs = 1u << c.bs_log2;
  const cuuint64_t size[4] = {static_cast<cuuint64_t>(c.dim), bs, static_cast<cuuint64_t>(c.heads),
                              static_cast<cuuint64_t>(c.num_blocks)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(st[2]), static_cast<cuuint64_t>(st[1]),
                                 static_cast<cuuint64_t>(st[0])};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(dims), std::min(bs, static_cast<cuuint32_t>(keys)), 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(map, c.f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
            size, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            c.f8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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

// Row tiles of a call, CTAs (pairs) of the GPU, and whether the units' tiles
// are dealt out. In tile steps, whole units take (waves of units) x (most tiles
// + 4 for a unit's start and end); dealt out they take their even share, a
// second start and end, and about 14 steps for the deal, the partial
// results and the join. 2048 rows on 32768 keys, 32 / 4 heads (128 units, 76
// pairs, 256 tiles): 0.63 ms dealt out, 0.68 whole; 512 rows on 4512 keys,
// 64 / 8 heads (64 units, 36 tiles): 87 us and 62; 512 rows on 16512 keys,
// 8 / 1 heads (8 units): 60 us and 182. From three waves on, units of unlike
// lengths fill the gaps by themselves: 1849 rows of four requests (232 units)
// 0.45 ms dealt out, 0.40 whole.
struct Work {
  int rows_here, row_tiles, shares;
  bool dealt;
};
Work work_of(long long rows, int group, int heads, int dim, long long max_keys, int num_sms) {
  const int pair = dim == 128 ? kPair<128> : kPair<64>;
  Work w;
  w.rows_here = 2 * pair * (kTile / group);
  w.row_tiles = static_cast<int>((rows + w.rows_here - 1) / w.rows_here);
  w.shares = num_sms / pair;
  const long long units = static_cast<long long>(w.row_tiles) * heads;
  const long long tiles = (max_keys + kTile - 1) / kTile, waves = (units + w.shares - 1) / w.shares;
  w.dealt = w.row_tiles <= kMaxDealt && waves <= 3 &&
            units * (tiles + kUnitWeight) / w.shares + 18 < waves * (tiles + 4) * 92 / 100;
  return w;
}
size_t border_bytes(const Work& w) { return (static_cast<size_t>(w.shares) * sizeof(int4) + 255) & ~static_cast<size_t>(255); }

template <int D, bool F8, int MOD>
cudaError_t launch_tiles_t(const AttnLaunch& p, const Work& w, void* workspace, cudaStream_t stream) {
  using Sh = Shared<D, F8>;
  constexpr int PAIR = kPair<D>;
  TilesLaunch L{p, kTile / p.group, w.row_tiles, w.dealt ? 1 : 0, nullptr};
  if (w.dealt) {
    char* at = static_cast<char*>(workspace);
    const size_t items = static_cast<size_t>(2) * w.shares * w.rows_here * p.group;
    L.borders = reinterpret_cast<int4*>(at);
    L.a.part_o = reinterpret_cast<float*>(at + border_bytes(w));
    L.a.part_ml = reinterpret_cast<float2*>(L.a.part_o + items * D);
  }
  CUtensorMap qmap, kmap, vmap;
  if (!query_map(&qmap, p, L.rows_per_tile) || !cache_map(&kmap, p.c.k, p.c, p.c.kst, F8 ? D : 64, Sh::kKeys) ||
      !cache_map(&vmap, p.c.v, p.c, p.c.vst, Sh::kDims, kTile))
    return cudaErrorInvalidValue;
  constexpr size_t smem = sizeof(Sh) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  static bool attr_done[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_done[dev]) {
    cudaError_t e = cudaFuncSetAttribute(attn_tiles_kernel<D, F8, MOD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done[dev] = true;
  }
  const long long grid = (w.dealt ? w.shares : static_cast<long long>(L.row_tiles) * p.c.heads) * PAIR;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {PAIR, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, attn_tiles_kernel<D, F8, MOD>, L, qmap, kmap, vmap);
  if (e != cudaSuccess || !w.dealt || w.shares < 2) return e;
  cudaLaunchConfig_t join{};
  join.gridDim = dim3((w.rows_here * p.group + 3) / 4, w.shares - 1);
  join.blockDim = dim3(128);
  join.stream = stream;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  join.attrs = at;
  join.numAttrs = 1;
  return cudaLaunchKernelEx(&join, attn_tiles_join_kernel<D>, L);
}

template <int MOD>
cudaError_t launch_tiles(const AttnLaunch& p, long long max_keys, void* workspace, int num_sms, cudaStream_t stream) {
  const Work w = work_of(p.rows, p.group, p.c.heads, p.c.dim, max_keys, num_sms);
  if (p.c.dim == 128)
    return p.c.f8 ? launch_tiles_t<128, true, MOD>(p, w, workspace, stream)
                  : launch_tiles_t<128, false, MOD>(p, w, workspace, stream);
  return p.c.f8 ? launch_tiles_t<64, true, MOD>(p, w, workspace, stream)
                : launch_tiles_t<64, false, MOD>(p, w, workspace, stream);
}

}  // namespace
}  // namespace sai
