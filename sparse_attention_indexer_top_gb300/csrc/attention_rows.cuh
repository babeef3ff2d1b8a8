// Row kernel of the attention over a paged cache: single-token rows (decode)
// and rows on chosen slots (sparse).
//
// For one row and one kv head, with up to 16 * MT query heads that share it,
//   m = max_t s_t, l = sum_t 2^(s_t - m), O = sum_t 2^(s_t - m) v_t,
//   s_t = scale * log2(e) * q.k_t,  out = O / l,  lse = (m + log2 l) ln 2
// in one pass over the keys, with m running: when it grows, l and O are
// multiplied by 2^(m_old - m_new). Two partial results over different keys
// join the same way, which is what splits a row's keys over warps and CTAs.
//
// Bound: reading the keys and values once, 2 * dim * (1 or 2) bytes per token
// and kv head against 4 * dim flops per query head, so with at most 64 heads
// per kv head the legacy warp-level MMA (16 x 8 x 16) keeps ahead of HBM and
// needs no tile of queries. Each warp of a CTA streams its own 16-key groups
// through a private ring of 16-byte asynchronous copies (a lane computes its
// key's address from the block table or the slot list, so pages of any size
// and gathered slots are the same loop), and no CTA-wide barrier runs in the
// loop.
//
// Up to 8 heads per kv head (FEW): the products are S^T = K Q^T and O^T =
// V^T P^T, with the heads as the MMA's 8-wide side, so that no half of a tile is
// padding; P goes from the accumulator layout to the operand's by one 8 x 8
// transpose for 8 keys. Up to 16 heads: S = Q K^T, O = P V with the heads as the
// 16-wide side. More: MT warps form a team that loads each key once and
// shares it, one 16-head tile per warp.
//
// MOD: scores are capped and biased on the way (attention_mod.cuh), and a row
// sees a document or a prefix of its request. These instances are apart, in
// attention_rows_mod.cu, so that the plain ones hold none of it; what is done is
// chosen at run time, since reading the keys takes longer: 64 rows of 4096-32768
// keys, 64 / 8 heads, e4m3, 399 us plain, 411 capped, 404 biased, 412 both; bf16 723
// for all of them.
#pragma once
#include "attention_mod.cuh"
#include "sai_internal.h"
#include "sai_ptx.cuh"

#include <algorithm>
#include <cmath>

namespace sai {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kMinExp = -64;  // scales below 2^-64 count as 2^-64 in the running maximum

// The running maximum m moves only when it is passed by more than 2^8, so that
// O is rarely rescaled. Weights in bf16 are as exact up to 2^8 as up to 1.
// Weights times value scales in f16 (e4m3) use its range: m is set 2^6 below the
// maximum, they reach 2^15, and one below 2^-14 is off by 2^-25 at most, 2^-31
// of the largest.
template <bool F8>
constexpr float kLift = F8 ? 6.f : 0.f;
template <bool F8>
constexpr float kPassed = kLift<F8> + 8.f;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit values, row lane/4, columns 2(lane%4) + {0, 1} per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes (low 16 bits) to two halves, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(codes));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(codes));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// Two weights w >= 0 as two bf16 terms each, off by 2^-15 of w at most together: the
// upper half of w's bits (2^-7), and the rest, rounded (2^-8 of it). The rest of a weight above 0 is above 0 too
// (2^-126 at least): both terms multiply the same values, and 0, or anything
// below it, times an infinite one would turn the sum into NaN.
__device__ __forceinline__ uint32_t upper_bf16(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ uint32_t rest_bf16(float a, float b, uint32_t upper) {
  return pack_bf16(fmaxf(a - bf16_lo(upper), fminf(a, 0x1p-126f)), fmaxf(b - bf16_hi(upper), fminf(b, 0x1p-126f)));
}

// Ring depth of each warp's (team's) 16-key (16 * MT keys) stages. A group's
// work is a chain of dependent steps, so more warps beat deeper rings: at dim
// 128, 4096 rows on 512 slots take 427 us with two bf16 stages (three CTAs per
// SM), 527 with three (two CTAs), 863 with four; e4m3 324 us with three stages,
// 366 with four, 489 with six; 64 decode rows of 4096-32768 keys 712, 697, 842
// and 411, 405, 519 us.
template <int D, bool F8>
constexpr int kDepth = F8 ? (D == 128 ? 3 : 4) : (D == 128 ? 2 : 3);

// What a row sees: keys j in [0, count), key j being token j (MOD: start + j)
// for j < low, or shift + j of the request, or slot j.
struct RowKeys {
  int count, low, shift;
  int start;
  long long batch;
};

template <bool MOD>
__device__ __forceinline__ RowKeys row_keys(const AttnLaunch& p, int row) {
  RowKeys k{0, 0, 0, 0, 0};
  if (p.slots) {
    k.count = p.slots_k;
    return k;
  }
  k.batch = p.row_to_batch ? p.row_to_batch[row] : row;
  const int n = p.seq_lens[row];
  if (MOD) {
    const RowSpan r = row_span(p, row, n);
    if (!r.good || k.batch < 0 || k.batch >= p.bt_rows ||
        ((static_cast<long long>(r.end) - 1) >> p.c.bs_log2) >= p.bt_stride) {
      k.count = -1;
      return k;
    }
    k.start = r.start;
    k.low = r.sinks_end - r.start;
    k.shift = r.first - k.low;
    k.count = k.low + r.end - r.first;
    return k;
  }
  if (n < 0 || n > p.max_len || k.batch < 0 || k.batch >= p.bt_rows ||
      ((static_cast<long long>(n) - 1) >> p.c.bs_log2) >= p.bt_stride) {
    k.count = -1;
    return k;
  }
  k.count = k.low = n;
  if (p.window > 0 && n > p.window) {
    const int first = n - p.window;
    k.low = min(p.sinks, first);
    k.shift = first - k.low;
    k.count = k.low + p.window;
  }
  return k;
}

// Keys of each chunk when a row's keys are split: even shares in 64-key steps.
template <bool MOD>
__device__ __forceinline__ int chunk_keys(const AttnLaunch& p, int count) {
  const int chunks = MOD && count <= p.short_keys ? p.short_chunks : p.chunks;
  return ((count + chunks - 1) / chunks + 63) & ~63;
}

// Four dims of a finished row; a sum of 0 gives zeros whatever the values are
// (0 times a NaN or infinite value has made the accumulator NaN).
template <int D>
__device__ __forceinline__ void write_row4(const AttnLaunch& p, long long head, int d, float m, float l, float4 a) {
  const bool none = l == 0.f;
  const float inv = 1.f / l;
  *reinterpret_cast<uint2*>(p.out + head * D + d) =
      none ? make_uint2(0u, 0u) : make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
  if (d == 0 && p.lse) p.lse[head] = none ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Weight of a partial result (maximum, sum) when joined under the maximum
// `base`; NaN sums stay NaN.
__device__ __forceinline__ float join_factor(float2 ml, float base) {
  return ml.y != ml.y ? ml.y : (ml.x == -INFINITY ? 0.f : ex2(ml.x - base));
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A variable of another CTA of the cluster, by its address in this one.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 peer_load4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 peer_load2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

// OWN: each team has a unit (row, kv head, head group) of its own; else the
// teams of a CTA share one unit's keys and join at the end. A unit's chunks,
// if it has several, are the CTAs of a cluster and join through each other's
// shared memory (up to 8), or leave partial results for a second kernel.
template <int D, bool F8, int MT, bool OWN, bool FEW, bool MOD>
__global__ void __launch_bounds__(kThreads) attn_rows_kernel(const AttnLaunch p) {
  constexpr int E = F8 ? 1 : 2;
  constexpr int RB = D * E;         // bytes of a key row
  constexpr int CPR = RB / 16;      // 16-byte chunks of a key row
  constexpr int SK = 16 * MT;       // keys per stage
  constexpr int TEAMS = kWarps / MT;
  constexpr int DEPTH = kDepth<D, F8>;
  constexpr int KB = SK * RB;       // bytes of a stage's keys (and of its values)
  constexpr int STAGE = 2 * KB + SK * 8 + MT * 4 + (16 - MT * 4 % 16) % 16;
  constexpr int NS = D / 16;        // k16 steps of q.k, and 16-dim column groups of O
  constexpr int HT = FEW ? 8 : 16;  // heads of a tile
  // Changed scores, bf16: the weights go to the MMA as two bf16 terms, 2^-15
  // together, so that the result is off by its own rounding alone; the time is that
  // of the keys. (Masks alone change nothing, the last bit included.)
  const bool split = MOD && !F8 && (p.cap_log2 > 0.f || p.slopes);
  static_assert(!FEW || MT == 1, "one tile of few heads");

  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = warp / MT, mt = warp % MT;
  const int g = lane >> 2, t = lane & 3;

  const int hg_count = (p.group + HT * MT - 1) / (HT * MT);
  int chunk = 0, hg, kvh, row;
  if (OWN) {
    // kv head by kv head, so that the rows at work share one head's keys in L2
    const long long u = static_cast<long long>(blockIdx.x) * TEAMS + team;
    if (u >= static_cast<long long>(p.rows) * p.c.heads * hg_count) return;
    hg = static_cast<int>(u % hg_count);
    row = static_cast<int>(u / hg_count % p.rows);
    kvh = static_cast<int>(u / hg_count / p.rows);
  } else {
    long long u = blockIdx.x;
    chunk = static_cast<int>(u % p.chunks);
    u /= p.chunks;
    hg = static_cast<int>(u % hg_count);
    u /= hg_count;
    kvh = static_cast<int>(u % p.c.heads);
    row = static_cast<int>(u / p.c.heads);
  }

  RowKeys rk = row_keys<MOD>(p, row);
  if (rk.count < 0) {
    rk.count = 0;
    if (lane == 0) atomicOr(p.status, kDevBadRowMeta);
  }
  int k_begin = 0, k_end = rk.count;
  if (p.chunks > 1) {
    const int per = chunk_keys<MOD>(p, rk.count);
    k_begin = min(rk.count, chunk * per);
    k_end = min(rk.count, k_begin + per);
    if (!p.clustered && k_begin >= k_end) return;  // the joining kernel knows which chunks there are
  }

  // ---- the 16 heads of this warp as A fragments; rows g and g + 8 per lane
  const int head_in_group = hg * HT * MT + mt * HT;
  const int head0 = kvh * p.group + head_in_group;
  const bool v0 = head_in_group + g < p.group, v1 = !FEW && head_in_group + g + 8 < p.group;
  const uint16_t* q0 = p.q + static_cast<long long>(row) * p.q_row + static_cast<long long>(head0 + g) * D;
  const uint16_t* q1 = q0 + 8 * D;
  uint32_t qa[NS][4];
  float sc0 = p.scale_log2, sc1 = p.scale_log2;
  if (!F8) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int d = 16 * s + 2 * t;
      qa[s][0] = v0 ? *reinterpret_cast<const uint32_t*>(q0 + d) : 0u;
      qa[s][1] = v1 ? *reinterpret_cast<const uint32_t*>(q1 + d) : 0u;
      qa[s][2] = v0 ? *reinterpret_cast<const uint32_t*>(q0 + d + 8) : 0u;
      qa[s][3] = v1 ? *reinterpret_cast<const uint32_t*>(q1 + d + 8) : 0u;
    }
  } else {
    // e4m3 keys are exact as halves, so the product runs in f16. A head's
    // query is brought to [2^14, 2^15) by a power of two first: its bf16
    // values are then exact as halves down to 2^-28 of the largest one, and
    // below that off by at most 2^-39 of it. The lane's four bytes of a
    // 16-byte chunk are dims 4t..4t+3, which sets the order of the k axis.
    float a0 = 0.f, a1 = 0.f;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const uint2 x0 = v0 ? *reinterpret_cast<const uint2*>(q0 + 16 * s + 4 * t) : make_uint2(0u, 0u);
      const uint2 x1 = v1 ? *reinterpret_cast<const uint2*>(q1 + 16 * s + 4 * t) : make_uint2(0u, 0u);
      qa[s][0] = x0.x;
      qa[s][1] = x1.x;
      qa[s][2] = x0.y;
      qa[s][3] = x1.y;
      a0 = fmaxf(a0, fmaxf(fmaxf(fabsf(bf16_lo(x0.x)), fabsf(bf16_hi(x0.x))),
                           fmaxf(fabsf(bf16_lo(x0.y)), fabsf(bf16_hi(x0.y)))));
      a1 = fmaxf(a1, fmaxf(fmaxf(fabsf(bf16_lo(x1.x)), fabsf(bf16_hi(x1.x))),
                           fmaxf(fabsf(bf16_lo(x1.y)), fabsf(bf16_hi(x1.y)))));
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, o));
      a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, o));
    }
    // 2^(14 - exponent), from the exponent field (0 and infinity: as they are)
    auto factor = [](float a, float* inv) {
      const int e = static_cast<int>(__float_as_uint(a) >> 23);
      const int up = (e == 0 || e == 255) ? 0 : min(126, 14 - (e - 127));  // 2^up and 2^-up are normal numbers
      *inv = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
      return __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
    };
    float i0, i1;
    const float f0 = factor(a0, &i0), f1 = factor(a1, &i1);
    sc0 *= i0;
    sc1 *= i1;
    if (FEW) {  // the lane's scores are of heads 2t and 2t + 1
      sc1 = __shfl_sync(0xffffffffu, sc0, 8 * t + 4);
      sc0 = __shfl_sync(0xffffffffu, sc0, 8 * t);
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      qa[s][0] = pack_f16(bf16_lo(qa[s][0]) * f0, bf16_hi(qa[s][0]) * f0);
      qa[s][1] = pack_f16(bf16_lo(qa[s][1]) * f1, bf16_hi(qa[s][1]) * f1);
      qa[s][2] = pack_f16(bf16_lo(qa[s][2]) * f0, bf16_hi(qa[s][2]) * f0);
      qa[s][3] = pack_f16(bf16_lo(qa[s][3]) * f1, bf16_hi(qa[s][3]) * f1);
    }
  }

  // ---- the ring
  unsigned char* ring = smem + team * (DEPTH * STAGE);
  const uint32_t ring_u = smem_u32(ring);
  const char* kbase = p.c.k + kvh * p.c.kst[1];
  const char* vbase = p.c.v + kvh * p.c.vst[1];
  const long long slot_limit = p.c.num_blocks << p.c.bs_log2;
  const int bs_mask = (1 << p.c.bs_log2) - 1;
  constexpr int STEP = OWN ? 1 : TEAMS;  // a team's stages are STEP apart
  const int first = OWN ? 0 : team;
  const int stages = (k_end - k_begin + SK - 1) / SK;
  const int my_stages = stages > first ? (stages - first + STEP - 1) / STEP : 0;
  bool bad_slot = false;

  // With a bias the nearest keys come first: from the first group on, every
  // nearer one would pass the running maximum by its 16 steps of the slope.
  const bool biased = MOD && p.slopes;
  auto place_of = [&](int s) { return biased ? stages - 1 - first - s * STEP : first + s * STEP; };
  // slot of this lane's key (lane & 15) in the team's stage s, -1: none
  auto slot_of = [&](int s) -> int {
    const int j = k_begin + place_of(s) * SK + mt * 16 + (lane & 15);
    if (s >= my_stages || j >= k_end) return -1;
    long long slot;
    if (p.slots) {
      slot = p.slots[row * p.slots_stride + j];
      if (slot < 0) return -1;
    } else {
      const int tok = j < rk.low ? j + (MOD ? rk.start : 0) : j + rk.shift;
      const int blk = p.block_table[rk.batch * p.bt_stride + (tok >> p.c.bs_log2)];
      slot = blk < 0 ? slot_limit : (static_cast<long long>(blk) << p.c.bs_log2) + (tok & bs_mask);
    }
    if (slot >= slot_limit) {
      bad_slot = true;
      return -1;
    }
    return static_cast<int>(slot);
  };
  // copy the warp's 16 keys and values of stage s into its ring place
  auto issue = [&](int s, int slot) {
    if (s < my_stages) {
      const uint32_t st = ring_u + (s % DEPTH) * STAGE;
      const int c = lane % CPR;
#pragma unroll
      for (int i = 0; i < 16 * CPR / 32; ++i) {
        const int key = i * (32 / CPR) + lane / CPR;
        const int sl = __shfl_sync(0xffffffffu, slot, key);
        const int bytes = sl < 0 ? 0 : 16;
        const long long blk = sl < 0 ? 0 : sl >> p.c.bs_log2;
        const long long off = sl < 0 ? 0 : sl & bs_mask;
        const int row_in_stage = mt * 16 + key;
        uint32_t at;
        if (CPR >= 8)
          at = row_in_stage * RB + ((c ^ (key & 7)) << 4);
        else  // two 64-byte rows to a 128-byte line
          at = row_in_stage * RB + ((c ^ ((key >> 1) & 3)) << 4);
        cp_async16(st + at, kbase + blk * p.c.kst[0] + off * p.c.kst[2] + c * 16, bytes);
        cp_async16(st + KB + at, vbase + blk * p.c.vst[0] + off * p.c.vst[2] + c * 16, bytes);
      }
      if (F8 && lane < 16) {
        const long long sidx = slot < 0 ? 0 : static_cast<long long>(slot >> p.c.bs_log2) * p.c.heads + kvh;
        const uint32_t at = st + 2 * KB + (mt * 16 + lane) * 4;
        cp_async4(at, p.c.ks + sidx, slot < 0 ? 0 : 4);
        cp_async4(at + SK * 4, p.c.vs + sidx, slot < 0 ? 0 : 4);
      }
      const uint32_t live = __ballot_sync(0xffffffffu, slot >= 0) & 0xffffu;
      if (lane == 0) *reinterpret_cast<uint32_t*>(ring + (s % DEPTH) * STAGE + 2 * KB + SK * 8 + mt * 4) = live;
    }
    cp_commit();
  };
  auto team_sync = [&]() {
    if (MT == 1)
      __syncwarp();
    else
      named_bar(1 + team, 32 * MT);
  };

  // MOD: the cap, and the slopes of the lane's two heads
  const float cap = MOD ? p.cap_log2 : 0.f, inv_cap = MOD && cap > 0.f ? 1.f / cap : 0.f;
  float slope0 = 0.f, slope1 = 0.f;
  if (biased) {
    const int h0 = FEW ? 2 * t : g, h1 = FEW ? 2 * t + 1 : g + 8;
    if (head_in_group + h0 < p.group) slope0 = p.slopes[head0 + h0] * 1.44269504088896340736f;
    if (head_in_group + h1 < p.group) slope1 = p.slopes[head0 + h1] * 1.44269504088896340736f;
  }
  // distance of key 0 of the group at work, were all keys behind the row's first tokens
  const int behind = biased ? p.seq_lens[row] - 1 - rk.shift : 0;
  int ahead = behind - k_begin - place_of(0) * SK;
  // distances of the lane's key `key` of the group, and of key + step
  auto distances = [&](int key, int step, float& d0, float& d1) {
    const int a = ahead - key;
    d0 = fabsf(static_cast<float>(a));
    d1 = fabsf(static_cast<float>(a - step));
    if (rk.low > 0) {  // first tokens before the window
      const int at = behind - a, back = rk.shift - rk.start;
      if (at < rk.low) d0 = fabsf(static_cast<float>(a + back));
      if (at + step < rk.low) d1 = fabsf(static_cast<float>(a - step + back));
    }
  };
  // The lane's four scores, two keys of two heads: x[head][key]
  auto change = [&](float (&x)[2][2], float d0, float d1) {
    if (cap > 0.f) {
      float t[4], most = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t[i] = x[i / 2][i % 2] * inv_cap;
        most = fmaxf(most, fabsf(t[i]));
      }
      if (__all_sync(0xffffffffu, most <= kNear)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = t[i] * t[i];
          x[i / 2][i % 2] *= fmaf(fmaf(fmaf(tanh_near(3), y, tanh_near(2)), y, tanh_near(1)), y, tanh_near(0));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i / 2][i % 2] = capped(x[i / 2][i % 2], cap, inv_cap);
      }
    }
    if (biased) {
      x[0][0] = fmaf(-slope0, d0, x[0][0]);
      x[0][1] = fmaf(-slope0, d1, x[0][1]);
      x[1][0] = fmaf(-slope1, d0, x[1][0]);
      x[1][1] = fmaf(-slope1, d1, x[1][1]);
    }
  };

  constexpr int NO = FEW ? 1 : 2;  // accumulator tiles per 16 dims
  float o[NS][NO][4];
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int e = 0; e < NO; ++e) o[s][e][0] = o[s][e][1] = o[s][e][2] = o[s][e][3] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

  {
    int sl[DEPTH];
#pragma unroll
    for (int s = 0; s < DEPTH; ++s) sl[s] = slot_of(s);
#pragma unroll
    for (int s = 0; s < DEPTH - 1; ++s) issue(s, sl[s]);
    int next = sl[DEPTH - 1];

    for (int s = 0; s < my_stages; ++s, ahead += MOD ? (STEP + 1) * SK : 0) {
      cp_wait<DEPTH - 2>();
      team_sync();  // the stage is whole for every lane, and the place refilled below is free
      const int after = slot_of(s + DEPTH);
      issue(s + DEPTH - 1, next);
      next = after;
      const uint32_t st = ring_u + (s % DEPTH) * STAGE;
      const unsigned char* stp = ring + (s % DEPTH) * STAGE;
#pragma unroll 1
      for (int kg = 0; kg < MT; ++kg, ahead -= MOD ? 16 : 0) {
        const uint32_t live = *reinterpret_cast<const uint32_t*>(stp + 2 * KB + SK * 8 + kg * 4);
        if (live == 0) continue;
        const uint32_t kb = st + kg * 16 * RB, vb = kb + KB;
        if constexpr (FEW) {
          // scores of 16 keys x 8 heads: the lane has keys g and g + 8 of
          // heads 2t and 2t + 1
          float c[4] = {0.f, 0.f, 0.f, 0.f}, c2[4] = {0.f, 0.f, 0.f, 0.f};  // two chains of products
          const int krow = (lane & 7) + ((lane >> 3) & 1) * 8, khalf = lane >> 4;
          if (!F8) {
#pragma unroll
            for (int s2 = 0; s2 < NS; ++s2) {
              uint32_t r[4];
              ldsm4(kb + krow * RB + (((2 * s2 + khalf) ^ (krow & 7)) << 4), r);
              mma16816<false>(s2 & 1 ? c2 : c, r, qa[s2][0], qa[s2][2]);
            }
          } else {
#pragma unroll
            for (int s2 = 0; s2 < NS; s2 += 2) {
              uint32_t r[4];
              const int ch = s2 + khalf;
              ldsm4(kb + krow * RB + ((CPR >= 8 ? (ch ^ (krow & 7)) : (ch ^ ((krow >> 1) & 3))) << 4), r);
              const uint32_t a0[4] = {e4m3x2_f16x2(r[0]), e4m3x2_f16x2(r[1]), e4m3x2_f16x2_hi(r[0]),
                                      e4m3x2_f16x2_hi(r[1])};
              const uint32_t a1[4] = {e4m3x2_f16x2(r[2]), e4m3x2_f16x2(r[3]), e4m3x2_f16x2_hi(r[2]),
                                      e4m3x2_f16x2_hi(r[3])};
              mma16816<true>(c, a0, qa[s2][0], qa[s2][2]);
              mma16816<true>(c2, a1, qa[s2 + 1][0], qa[s2 + 1][2]);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) c[e] += c2[e];
          float vs[2], ev[2];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int key = g + 8 * n;
            const bool on = (live >> key) & 1;
            float k0 = sc0, k1 = sc1;
            vs[n] = 1.f;
            ev[n] = 0.f;
            if (F8) {
              const float* sp = reinterpret_cast<const float*>(stp + 2 * KB) + kg * 16 + key;
              k0 *= sp[0];
              k1 *= sp[0];
              vs[n] = sp[SK];
              ev[n] = static_cast<float>(max(kMinExp, static_cast<int>((__float_as_uint(vs[n]) >> 23) & 255) - 127));
            }
            c[2 * n] *= k0;
            c[2 * n + 1] *= k1;
            if (!MOD) {
              c[2 * n] = on ? c[2 * n] : -INFINITY;
              c[2 * n + 1] = on ? c[2 * n + 1] : -INFINITY;
            }
          }
          if (MOD) {
            float x[2][2] = {{c[0], c[2]}, {c[1], c[3]}}, d0 = 0.f, d1 = 0.f;
            if (biased) distances(g, 8, d0, d1);
            change(x, d0, d1);
            const bool on0 = (live >> g) & 1, on1 = (live >> (g + 8)) & 1;
            c[0] = on0 ? x[0][0] : -INFINITY;
            c[1] = on0 ? x[1][0] : -INFINITY;
            c[2] = on1 ? x[0][1] : -INFINITY;
            c[3] = on1 ? x[1][1] : -INFINITY;
          }
          float x0 = fmaxf(c[0] + ev[0], c[2] + ev[1]), x1 = fmaxf(c[1] + ev[0], c[3] + ev[1]);
          if (__any_sync(0xffffffffu, x0 > m0 + kPassed<F8> || x1 > m1 + kPassed<F8>)) {
#pragma unroll
            for (int f = 4; f < 32; f <<= 1) {
              x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, f));
              x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, f));
            }
            const bool up0 = x0 > m0 + kPassed<F8>, up1 = x1 > m1 + kPassed<F8>;
            x0 -= kLift<F8>;
            x1 -= kLift<F8>;
            const float f0 = up0 ? (m0 == -INFINITY ? 0.f : ex2(m0 - x0)) : 1.f;
            const float f1 = up1 ? (m1 == -INFINITY ? 0.f : ex2(m1 - x1)) : 1.f;
            if (up0) m0 = x0;
            if (up1) m1 = x1;
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int s2 = 0; s2 < NS; ++s2) {
              o[s2][0][0] *= f0;
              o[s2][0][1] *= f1;
              o[s2][0][2] *= f0;
              o[s2][0][3] *= f1;
            }
          }
          const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
          uint32_t pb[2], rest[2] = {0u, 0u};
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            float w0 = ex2(c[2 * n] - b0), w1 = ex2(c[2 * n + 1] - b1);
            l0 += w0;
            l1 += w1;
            if (F8) {
              w0 *= vs[n];
              w1 *= vs[n];
            }
            pb[n] = F8 ? pack_f16(w0, w1) : split ? upper_bf16(w0, w1) : pack_bf16(w0, w1);
            if (split) rest[n] = transpose8x8(rest_bf16(w0, w1, pb[n]));
            pb[n] = transpose8x8(pb[n]);
          }
          if (!F8) {
            const int vrow = (lane & 7) + (lane >> 4) * 8, vhalf = (lane >> 3) & 1;
#pragma unroll
            for (int s2 = 0; s2 < NS; ++s2) {
              uint32_t r[4];
              ldsm4_t(vb + vrow * RB + (((2 * s2 + vhalf) ^ (vrow & 7)) << 4), r);
              mma16816<false>(o[s2][0], r, pb[0], pb[1]);
              if (split) mma16816<false>(o[s2][0], r, rest[0], rest[1]);
            }
          } else {
            // transposed 16-bit pairs hold two dims of keys 2t and 2t + 1; a
            // byte permute makes them two keys of one dim each: even dims of
            // the 16-byte chunk are the tile's rows 0-7, odd dims rows 8-15
            const int vrow = lane & 15, vhalf = lane >> 4;
#pragma unroll
            for (int s2 = 0; s2 < NS; s2 += 2) {
              uint32_t r[4];
              const int ch = s2 + vhalf;
              ldsm4_t(vb + vrow * RB + ((CPR >= 8 ? (ch ^ (vrow & 7)) : (ch ^ ((vrow >> 1) & 3))) << 4), r);
#pragma unroll
              for (int i = 0; i < 4; ++i) r[i] = __byte_perm(r[i], 0u, 0x3120);
              const uint32_t a0[4] = {e4m3x2_f16x2(r[0]), e4m3x2_f16x2_hi(r[0]), e4m3x2_f16x2(r[1]),
                                      e4m3x2_f16x2_hi(r[1])};
              const uint32_t a1[4] = {e4m3x2_f16x2(r[2]), e4m3x2_f16x2_hi(r[2]), e4m3x2_f16x2(r[3]),
                                      e4m3x2_f16x2_hi(r[3])};
              mma16816<true>(o[s2][0], a0, pb[0], pb[1]);
              mma16816<true>(o[s2 + 1][0], a1, pb[0], pb[1]);
            }
          }
        } else {
        // scores of 16 heads x 16 keys
        float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const int krow = (lane & 7) + ((lane >> 4) & 1) * 8, khalf = (lane >> 3) & 1;
        if (!F8) {
#pragma unroll
          for (int s2 = 0; s2 < NS; ++s2) {
            uint32_t r[4];
            ldsm4(kb + krow * RB + (((2 * s2 + khalf) ^ (krow & 7)) << 4), r);
            mma16816<false>(c[0], qa[s2], r[0], r[1]);
            mma16816<false>(c[1], qa[s2], r[2], r[3]);
          }
        } else {
#pragma unroll
          for (int s2 = 0; s2 < NS; s2 += 2) {
            uint32_t r[4];
            const int ch = s2 + khalf;
            ldsm4(kb + krow * RB + ((CPR >= 8 ? (ch ^ (krow & 7)) : (ch ^ ((krow >> 1) & 3))) << 4), r);
            mma16816<true>(c[0], qa[s2], e4m3x2_f16x2(r[0]), e4m3x2_f16x2_hi(r[0]));
            mma16816<true>(c[0], qa[s2 + 1], e4m3x2_f16x2(r[1]), e4m3x2_f16x2_hi(r[1]));
            mma16816<true>(c[1], qa[s2], e4m3x2_f16x2(r[2]), e4m3x2_f16x2_hi(r[2]));
            mma16816<true>(c[1], qa[s2 + 1], e4m3x2_f16x2(r[3]), e4m3x2_f16x2_hi(r[3]));
          }
        }
        // the lane's keys are 2t, 2t + 1, 8 + 2t, 9 + 2t. With block scales,
        // the running maximum is that of s_t + exponent(v scale): the weights
        // that multiply v codes then fit f16 whatever the scales; l adds the
        // same weights without the scale.
        float x0 = -INFINITY, x1 = -INFINITY;
        float vs[2][2], evs[2][2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = 8 * n + 2 * t + e;
            float ks = 1.f, ev = 0.f;
            if (F8) {
              const float* sp = reinterpret_cast<const float*>(stp + 2 * KB) + kg * 16 + key;
              ks = sp[0];
              vs[n][e] = sp[SK];
              ev = static_cast<float>(max(kMinExp, static_cast<int>((__float_as_uint(vs[n][e]) >> 23) & 255) - 127));
            }
            const bool on = (live >> key) & 1;
            c[n][e] *= sc0 * ks;
            c[n][e + 2] *= sc1 * ks;
            evs[n][e] = ev;
            if (!MOD) {
              c[n][e] = on ? c[n][e] : -INFINITY;
              c[n][e + 2] = on ? c[n][e + 2] : -INFINITY;
            }
          }
          if (MOD) {
            float x[2][2] = {{c[n][0], c[n][1]}, {c[n][2], c[n][3]}}, d0 = 0.f, d1 = 0.f;
            if (biased) distances(8 * n + 2 * t, 1, d0, d1);
            change(x, d0, d1);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const bool on = (live >> (8 * n + 2 * t + e)) & 1;
              c[n][e] = on ? x[0][e] : -INFINITY;
              c[n][e + 2] = on ? x[1][e] : -INFINITY;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x0 = fmaxf(x0, c[n][e] + evs[n][e]);
            x1 = fmaxf(x1, c[n][e + 2] + evs[n][e]);
          }
        }
        if (__any_sync(0xffffffffu, x0 > m0 + kPassed<F8> || x1 > m1 + kPassed<F8>)) {
#pragma unroll
          for (int f = 1; f < 4; f <<= 1) {
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, f));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, f));
          }
          const bool up0 = x0 > m0 + kPassed<F8>, up1 = x1 > m1 + kPassed<F8>;
          x0 -= kLift<F8>;
          x1 -= kLift<F8>;
          const float f0 = up0 ? (m0 == -INFINITY ? 0.f : ex2(m0 - x0)) : 1.f;
          const float f1 = up1 ? (m1 == -INFINITY ? 0.f : ex2(m1 - x1)) : 1.f;
          if (up0) m0 = x0;
          if (up1) m1 = x1;
          l0 *= f0;
          l1 *= f1;
#pragma unroll
          for (int s2 = 0; s2 < NS; ++s2)
#pragma unroll
            for (int e = 0; e < NO; ++e) {
              o[s2][e][0] *= f0;
              o[s2][e][1] *= f0;
              o[s2][e][2] *= f1;
              o[s2][e][3] *= f1;
            }
        }
        const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            c[n][e] = ex2(c[n][e] - b0);
            c[n][e + 2] = ex2(c[n][e + 2] - b1);
            l0 += c[n][e];
            l1 += c[n][e + 2];
            if (F8) {
              c[n][e] *= vs[n][e];
              c[n][e + 2] *= vs[n][e];
            }
          }
        // the weights as bf16 (f16 with e4m3 values): the MMA's other operand
        // is the cache's type; relative error 2^-8, as the output's own rounding
        // (split: 2^-15; f16 2^-11 and the absolute term of kLift)
        uint32_t pa[4], rest[4] = {0u, 0u, 0u, 0u};
        if (F8) {
          pa[0] = pack_f16(c[0][0], c[0][1]);
          pa[1] = pack_f16(c[0][2], c[0][3]);
          pa[2] = pack_f16(c[1][0], c[1][1]);
          pa[3] = pack_f16(c[1][2], c[1][3]);
        } else if (split) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = c[i / 2][i % 2 * 2], b = c[i / 2][i % 2 * 2 + 1];
            pa[i] = upper_bf16(a, b);
            rest[i] = rest_bf16(a, b, pa[i]);
          }
        } else {
          pa[0] = pack_bf16(c[0][0], c[0][1]);
          pa[1] = pack_bf16(c[0][2], c[0][3]);
          pa[2] = pack_bf16(c[1][0], c[1][1]);
          pa[3] = pack_bf16(c[1][2], c[1][3]);
        }
        const int vrow = lane & 15, vhalf = lane >> 4;
        if (!F8) {
#pragma unroll
          for (int s2 = 0; s2 < NS; ++s2) {
            uint32_t r[4];
            ldsm4_t(vb + vrow * RB + (((2 * s2 + vhalf) ^ (vrow & 7)) << 4), r);
            mma16816<false>(o[s2][0], pa, r[0], r[1]);
            mma16816<false>(o[s2][NO - 1], pa, r[2], r[3]);
            if (split) {
              mma16816<false>(o[s2][0], rest, r[0], r[1]);
              mma16816<false>(o[s2][NO - 1], rest, r[2], r[3]);
            }
          }
        } else {
          // transposed 16-bit pairs hold two dims of keys 2t and 2t + 1; a
          // byte permute makes them two keys of one dim each: even dims of
          // the 16-byte chunk go to one column tile, odd dims to the other
#pragma unroll
          for (int s2 = 0; s2 < NS; s2 += 2) {
            uint32_t r[4];
            const int ch = s2 + vhalf;
            ldsm4_t(vb + vrow * RB + ((CPR >= 8 ? (ch ^ (vrow & 7)) : (ch ^ ((vrow >> 1) & 3))) << 4), r);
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = __byte_perm(r[i], 0u, 0x3120);
            mma16816<true>(o[s2][0], pa, e4m3x2_f16x2(r[0]), e4m3x2_f16x2(r[1]));
            mma16816<true>(o[s2][NO - 1], pa, e4m3x2_f16x2_hi(r[0]), e4m3x2_f16x2_hi(r[1]));
            mma16816<true>(o[s2 + 1][0], pa, e4m3x2_f16x2(r[2]), e4m3x2_f16x2(r[3]));
            mma16816<true>(o[s2 + 1][NO - 1], pa, e4m3x2_f16x2_hi(r[2]), e4m3x2_f16x2_hi(r[3]));
          }
        }
        }
      }
    }
  }
  cp_wait<0>();
  if (bad_slot) atomicOr(p.status, kDevBadPage);
#pragma unroll
  for (int f = FEW ? 4 : 1; f < (FEW ? 32 : 4); f <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, f);
    l1 += __shfl_xor_sync(0xffffffffu, l1, f);
  }

  // ---- join the teams' results (same head tile mt, different keys); with
  // OWN the same way through the team's own ring, for whole-line stores
  constexpr int JOIN = OWN ? 1 : TEAMS;
  auto part_sync = [&]() {
    if (OWN)
      team_sync();
    else
      __syncthreads();
  };
  part_sync();  // the ring is done with; its memory holds the partial results
  constexpr int OS = D + 4;  // floats between rows
  float* po = reinterpret_cast<float*>(OWN ? ring : smem);            // [JOIN * MT][HT][OS]
  float2* pml = reinterpret_cast<float2*>(po + JOIN * MT * HT * OS);  // [JOIN * MT][HT]
  {
    const int slot = OWN ? mt : warp;
    float* w = po + slot * HT * OS;
    if constexpr (FEW) {
      float *w0 = w + 2 * t * OS, *w1 = w0 + OS;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int d = 16 * s + (F8 ? 2 * g : g), d2 = d + (F8 ? 1 : 8);
        w0[d] = o[s][0][0];
        w1[d] = o[s][0][1];
        w0[d2] = o[s][0][2];
        w1[d2] = o[s][0][3];
      }
      if (g == 0) {
        pml[slot * HT + 2 * t] = make_float2(m0, l0);
        pml[slot * HT + 2 * t + 1] = make_float2(m1, l1);
      }
    } else {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        if (!F8) {
#pragma unroll
          for (int e = 0; e < NO; ++e) {
            const int d = 16 * s + 8 * e + 2 * t;
            *reinterpret_cast<float2*>(w + g * OS + d) = make_float2(o[s][e][0], o[s][e][1]);
            *reinterpret_cast<float2*>(w + (g + 8) * OS + d) = make_float2(o[s][e][2], o[s][e][3]);
          }
        } else {
          const int d = 16 * s + 4 * t;
          *reinterpret_cast<float4*>(w + g * OS + d) =
              make_float4(o[s][0][0], o[s][NO - 1][0], o[s][0][1], o[s][NO - 1][1]);
          *reinterpret_cast<float4*>(w + (g + 8) * OS + d) =
              make_float4(o[s][0][2], o[s][NO - 1][2], o[s][0][3], o[s][NO - 1][3]);
        }
      }
      if (t == 0) {
        pml[slot * HT + g] = make_float2(m0, l0);
        pml[slot * HT + g + 8] = make_float2(m1, l1);
      }
    }
  }
  part_sync();
  constexpr int LPR = D / 4;  // lanes of four dims to a head row
  const int heads_here = min(HT * MT, p.group - hg * HT * MT);
  float* joined = reinterpret_cast<float*>(pml + JOIN * MT * HT);         // clustered: [HT * MT][D]
  float2* joined_ml = reinterpret_cast<float2*>(joined + HT * MT * D);  // [HT * MT]
  for (int i = OWN ? mt * 32 + lane : threadIdx.x; i < heads_here * LPR; i += OWN ? 32 * MT : kThreads) {
    const int hr = i / LPR, d = (i % LPR) * 4;
    const int tile = hr / HT, r = hr % HT;
    const int hin = hg * HT * MT + hr;
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < JOIN; ++k) m = fmaxf(m, pml[(k * MT + tile) * HT + r].x);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < JOIN; ++k) {
      const float2 ml = pml[(k * MT + tile) * HT + r];
      const float f = join_factor(ml, base);
      const float4 x = *reinterpret_cast<const float4*>(po + ((k * MT + tile) * HT + r) * OS + d);
      l += f * ml.y;
      a.x += f * x.x;
      a.y += f * x.y;
      a.z += f * x.z;
      a.w += f * x.w;
    }
    const long long head = static_cast<long long>(row) * p.q_heads + kvh * p.group + hin;
    if (!OWN && p.clustered) {
      *reinterpret_cast<float4*>(joined + hr * D + d) = a;
      if (d == 0) joined_ml[hr] = make_float2(m, l);
    } else if (!OWN && p.chunks > 1) {
      *reinterpret_cast<float4*>(p.part_o + (head * p.chunks + chunk) * D + d) = a;
      if (d == 0) p.part_ml[head * p.chunks + chunk] = make_float2(m, l);
    } else {
      write_row4<D>(p, head, d, m, l, a);
    }
  }
  if (OWN || p.chunks == 1) return;
  if (!p.clustered) {
    pdl_trigger();
    return;
  }
  cluster_sync();
  for (int i = chunk * kThreads + threadIdx.x; i < heads_here * LPR; i += p.chunks * kThreads) {
    const int hr = i / LPR, d = (i % LPR) * 4;
    float2 ml[8];
    float m = -INFINITY;
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < p.chunks) {
        ml[c] = peer_load2(peer_addr(joined_ml + hr, c));
        m = fmaxf(m, ml[c].x);
      }
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < p.chunks) {
        const float f = join_factor(ml[c], base);
        const float4 x = peer_load4(peer_addr(joined + hr * D + d, c));
        l += f * ml[c].y;
        a.x += f * x.x;
        a.y += f * x.y;
        a.z += f * x.z;
        a.w += f * x.w;
      }
    write_row4<D>(p, static_cast<long long>(row) * p.q_heads + kvh * p.group + hg * HT * MT + hr, d, m, l, a);
  }
  cluster_sync();  // no CTA ends while another may read its memory
}

// Joins the chunks (at most 64) of one (row, head): four dims to a thread, the
// chunks dealt over the groups of D / 4 threads so that few loads follow one
// another (one warp walking 64 chunks took 11 us).
template <int D, bool MOD>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnLaunch p) {
  constexpr int LPR = D / 4, GROUPS = 128 / LPR;
  __shared__ float4 part[GROUPS][LPR];
  const long long head = blockIdx.x;
  const int lane = threadIdx.x & 31, grp = threadIdx.x / LPR, d = (threadIdx.x % LPR) * 4;
  const RowKeys rk = row_keys<MOD>(p, static_cast<int>(head / p.q_heads));
  int used = 0;
  if (rk.count > 0) {
    const int per = chunk_keys<MOD>(p, rk.count);
    used = (rk.count + per - 1) / per;
  }
  pdl_wait();
  // every warp: the weights of chunks lane and lane + 32
  const float2* ml = p.part_ml + head * p.chunks;
  const float2 none = make_float2(-INFINITY, 0.f);
  const float2 x0 = lane < used ? ml[lane] : none, x1 = lane + 32 < used ? ml[lane + 32] : none;
  float m = fmaxf(x0.x, x1.x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float base = m == -INFINITY ? 0.f : m;
  const float f0 = join_factor(x0, base), f1 = join_factor(x1, base);
  float l = f0 * x0.y + f1 * x1.y;
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c0 = 0; c0 < used; c0 += GROUPS) {
    const int c = c0 + grp;
    const float g0 = __shfl_sync(0xffffffffu, f0, c & 31), g1 = __shfl_sync(0xffffffffu, f1, c & 31);
    if (c < used) {
      const float f = c < 32 ? g0 : g1;
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + (head * p.chunks + c) * D + d);
      a.x += f * v.x;
      a.y += f * v.y;
      a.z += f * v.z;
      a.w += f * v.w;
    }
  }
  part[grp][threadIdx.x % LPR] = a;
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int g = 1; g < GROUPS; ++g) {
    const float4 v = part[g][threadIdx.x];
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
  write_row4<D>(p, head, d, m, l, a);
}

template <int D, bool F8, int MT, bool FEW>
constexpr size_t rows_smem() {
  constexpr int SK = 16 * MT;
  constexpr size_t stage = 2 * SK * D * (F8 ? 1 : 2) + SK * 8 + MT * 4 + (16 - MT * 4 % 16) % 16;
  constexpr size_t ring = stage * kDepth<D, F8> * (kWarps / MT);
  constexpr int heads = FEW ? 8 : 16;
  constexpr size_t join = kWarps * heads * ((D + 4) * 4 + 8) + heads * MT * (D * 4 + 8);
  return ring > join ? ring : join;
}

template <int D, bool F8, int MT, bool OWN, bool FEW, bool MOD>
cudaError_t launch_rows_t(const AttnLaunch& p, cudaStream_t stream) {
  constexpr size_t smem = rows_smem<D, F8, MT, FEW>();
  static bool attr_done[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_done[dev]) {
    cudaError_t e = cudaFuncSetAttribute(attn_rows_kernel<D, F8, MT, OWN, FEW, MOD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done[dev] = true;
  }
  constexpr int heads = (FEW ? 8 : 16) * MT;
  const long long groups = (p.group + heads - 1) / heads;
  long long grid = static_cast<long long>(p.rows) * p.c.heads * groups * p.chunks;
  if (OWN) grid = (grid * MT + kWarps - 1) / kWarps;
  if (!p.clustered) {
    attn_rows_kernel<D, F8, MT, OWN, FEW, MOD><<<static_cast<unsigned>(grid), kThreads, smem, stream>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {static_cast<unsigned>(p.chunks), 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_rows_kernel<D, F8, MT, OWN, FEW, MOD>, p);
}

template <int D, bool F8, int MT, bool FEW, bool MOD>
cudaError_t launch_rows_m(const AttnLaunch& p, cudaStream_t stream) {
  return p.own ? launch_rows_t<D, F8, MT, true, FEW, MOD>(p, stream) : launch_rows_t<D, F8, MT, false, FEW, MOD>(p, stream);
}

template <int D, bool F8, bool MOD>
cudaError_t launch_rows_d(const AttnLaunch& p, cudaStream_t stream) {
  if (p.group <= 8) return launch_rows_m<D, F8, 1, true, MOD>(p, stream);
  if (p.group <= 16) return launch_rows_m<D, F8, 1, false, MOD>(p, stream);
  if (p.group <= 32) return launch_rows_m<D, F8, 2, false, MOD>(p, stream);
  return launch_rows_m<D, F8, 4, false, MOD>(p, stream);
}

template <bool MOD>
cudaError_t launch_rows(const AttnLaunch& p, cudaStream_t stream) {
  cudaError_t e;
  if (p.c.dim == 128)
    e = p.c.f8 ? launch_rows_d<128, true, MOD>(p, stream) : launch_rows_d<128, false, MOD>(p, stream);
  else
    e = p.c.f8 ? launch_rows_d<64, true, MOD>(p, stream) : launch_rows_d<64, false, MOD>(p, stream);
  if (e != cudaSuccess || p.chunks == 1 || p.clustered) return e;
  // the joining kernel starts while the last chunks run, and waits for them
  // before it reads their results
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(p.rows) * p.q_heads));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return p.c.dim == 128 ? cudaLaunchKernelEx(&cfg, attn_join_kernel<128, MOD>, p)
                        : cudaLaunchKernelEx(&cfg, attn_join_kernel<64, MOD>, p);
}

}  // namespace
}  // namespace sai
