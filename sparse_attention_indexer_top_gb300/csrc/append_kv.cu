// Rotate the step's keys and queries by their positions and write keys and
// values into the paged cache (bf16, or e4m3 with a scale for each block of
// tokens and kv head).
//
// Every row is read once and written once; a lane holds 16 dims of a head as
// two 8-dim chunks that are rotation partners (or two halves of the part that
// is not rotated), so a pair's two members meet in registers.
//
// Bound: bytes (a few operations per element). One launch of two kinds of
// CTA: "row" CTAs rotate heads of one row each, keeping the row's cosines in
// registers over its heads; "block" CTAs (e4m3 cache) own everything the call
// appends to one (block of tokens, kv head), whose scale needs the largest of
// all those values before the first code can be written: the values wait in
// registers for it, so they are read once.
#include "sai_internal.h"
#include "sai_ptx.cuh"

#include <algorithm>

namespace sai {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSmallUnit = 4;  // units of up to 4 tokens take one warp, longer ones the CTA
constexpr int kMinExp = -64;

struct RowPlace {
  int pos;        // position, -1: nothing to append
  int batch;
  int blk;        // physical block, -1: none
};

__device__ __forceinline__ RowPlace row_place(const AppendLaunch& p, int row, bool flag) {
  RowPlace r{-1, 0, -1};
  const int n = p.seq_lens[row];
  const int b = p.row_to_batch ? p.row_to_batch[row] : row;
  if (n == 0) return r;
  const int pos = n - 1;
  if (n < 0 || b < 0 || b >= p.bt_rows || (pos >> p.c.bs_log2) >= p.bt_stride || pos >= p.max_pos) {
    if (flag) atomicOr(p.status, kDevBadRowMeta);
    return r;
  }
  const int blk = p.block_table[b * p.bt_stride + (pos >> p.c.bs_log2)];
  if (blk < 0 || blk >= p.c.num_blocks) {
    if (flag) atomicOr(p.status, kDevBadPage);
    return r;
  }
  r.pos = pos;
  r.batch = b;
  r.blk = blk;
  return r;
}

__device__ __forceinline__ float lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ void unpack8(uint4 x, float (&f)[8]) {
  f[0] = lo(x.x); f[1] = hi(x.x); f[2] = lo(x.y); f[3] = hi(x.y);
  f[4] = lo(x.z); f[5] = hi(x.z); f[6] = lo(x.w); f[7] = hi(x.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
// Four fp32 to four e4m3 codes (nearest, saturating; NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\t"
      "mov.b32 %0, {x, y};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t c, float (&f)[4]) {
  uint32_t a, b;
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(c));
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\t}"
      : "=f"(f[0]), "=f"(f[1])
      : "r"(a));
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\t}"
      : "=f"(f[2]), "=f"(f[3])
      : "r"(b));
}

// The two 8-dim chunks of lane `l` (of dim / 16): partners l and l + rot/16
// inside the rotated part, the same halves of what lies above it.
struct Chunks {
  int a, b;    // chunk indices
  bool rotated;
};
__device__ __forceinline__ Chunks chunks_of(int l, int rot, int dim) {
  const int rc = rot / 16;
  if (l < rc) return Chunks{l, l + rc, true};
  return Chunks{rc + l, dim / 16 + l, false};
}

// The lane's cosines and sines at a position: angles 8a..8a+7 when the pairs
// are (d, d + rot/2), else angles 4a..4a+3 and 4b..4b+3 (pairs inside a chunk).
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void load_angles(const AppendLaunch& p, int pos, const Chunks& ch, Angles& g) {
  const float* cs = p.cos_sin + static_cast<long long>(pos) * p.rot;
  const int half = p.rot / 2;
  const int i0 = p.interleaved ? 4 * ch.a : 8 * ch.a;
  const int i1 = p.interleaved ? 4 * ch.b : 8 * ch.a + 4;
  *reinterpret_cast<float4*>(g.c) = __ldg(reinterpret_cast<const float4*>(cs + i0));
  *reinterpret_cast<float4*>(g.c + 4) = __ldg(reinterpret_cast<const float4*>(cs + i1));
  *reinterpret_cast<float4*>(g.s) = __ldg(reinterpret_cast<const float4*>(cs + half + i0));
  *reinterpret_cast<float4*>(g.s + 4) = __ldg(reinterpret_cast<const float4*>(cs + half + i1));
}
__device__ __forceinline__ void rot2(float& x1, float& x2, float c, float s) {
  // single operations, so that a plain fp32 computation gives the same bits
  const float y1 = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
  const float y2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
  x1 = y1;
  x2 = y2;
}
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const Angles& g, int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rot2(a[2 * i], a[2 * i + 1], g.c[i], g.s[i]);
      rot2(b[2 * i], b[2 * i + 1], g.c[4 + i], g.s[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) rot2(a[i], b[i], g.c[i], g.s[i]);
  }
}

// ------------------------------------------------------------- row CTAs
// n heads of one row, `src_step` values and `dst_step` bytes apart, four of
// them in flight.
__device__ __forceinline__ void move_heads(const uint16_t* src, int src_step, char* dst, long long dst_step, int n,
                                           const Chunks& ch, bool live, bool turn, const Angles& ang, int interleaved) {
  constexpr int kAhead = 4;
  for (; n > 0; n -= kAhead) {
    uint4 xa[kAhead], xb[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      xa[j] = xb[j] = make_uint4(0, 0, 0, 0);
      if (j < n && live) {
        xa[j] = __ldg(reinterpret_cast<const uint4*>(src + j * src_step) + ch.a);
        xb[j] = __ldg(reinterpret_cast<const uint4*>(src + j * src_step) + ch.b);
      }
    }
    src += kAhead * src_step;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (j >= n) break;
      if (turn) {
        float a[8], b[8];
        unpack8(xa[j], a);
        unpack8(xb[j], b);
        rotate(a, b, ang, interleaved);
        xa[j] = pack8(a);
        xb[j] = pack8(b);
      }
      reinterpret_cast<uint4*>(dst)[ch.a] = xa[j];
      reinterpret_cast<uint4*>(dst)[ch.b] = xb[j];
      dst += dst_step;
    }
  }
}

// `rows` neighbouring rows: their query heads, and with a bf16 cache their
// keys and values. A thread stays with one row and one place in the heads, so
// it loads its angles once.
__device__ __forceinline__ void row_cta(const AppendLaunch& p, int row0, int rows) {
  const int dim = p.c.dim, lph = dim / 16;  // lanes to a head
  const int slots = kThreads / lph / rows;  // heads of a row at once
  const int l = threadIdx.x % lph, slot = threadIdx.x / lph;
  const int row = row0 + slot / slots, first = slot % slots;
  if (row >= p.rows || slot >= slots * rows) return;
  const RowPlace r = row_place(p, row, l == 0 && first == 0);
  const Chunks ch = chunks_of(l, p.rot, dim);
  const bool live = r.pos >= 0, turn = ch.rotated && live;
  Angles ang;
  if (turn) load_angles(p, r.pos, ch, ang);
  const int step = slots * dim;
  if (p.q) {
    char* dst = reinterpret_cast<char*>(p.out_q + (static_cast<long long>(row) * p.q_heads + first) * dim);
    move_heads(p.q + row * p.q_row + first * dim, step, dst, 2 * step, (p.q_heads - first + slots - 1) / slots, ch, live,
               turn, ang, p.interleaved);
  }
  if (p.c.f8 || !live) return;
  const int n = (p.c.heads - first + slots - 1) / slots;
  const long long off = r.pos & ((1 << p.c.bs_log2) - 1);
  move_heads(p.k + row * p.k_row + first * dim, step, p.c.k + r.blk * p.c.kst[0] + first * p.c.kst[1] + off * p.c.kst[2],
             slots * p.c.kst[1], n, ch, true, turn, ang, p.interleaved);
  move_heads(p.v + row * p.v_row + first * dim, step, p.c.v + r.blk * p.c.vst[0] + first * p.c.vst[1] + off * p.c.vst[2],
             slots * p.c.vst[1], n, ch, true, false, ang, p.interleaved);
}

// ------------------------------------------------------------- block CTAs
// Largest finite magnitude of 16 values.
__device__ __forceinline__ float amax16(const float (&a)[8], const float (&b)[8], float m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = fabsf(a[i]), y = fabsf(b[i]);
    m = fmaxf(m, x <= 3.402823466e38f ? x : 0.f);
    m = fmaxf(m, y <= 3.402823466e38f ? y : 0.f);
  }
  return m;
}
// Least 2^e, e >= kMinExp, with amax <= 448 * 2^e: 448 = 1.75 * 2^8.
__device__ __forceinline__ float needed_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  if (amax == 0.f) e = kMinExp;
  e = max(e, kMinExp);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The lane's 16 dims of token `row`, head h, as they came.
struct Raw {
  uint4 a, b;
};
template <bool KEYS>
__device__ __forceinline__ Raw load_raw(const AppendLaunch& p, int row, int h, const Chunks& ch) {
  const uint4* src = reinterpret_cast<const uint4*>((KEYS ? p.k + row * p.k_row : p.v + row * p.v_row) +
                                                    static_cast<long long>(h) * p.c.dim);
  return Raw{__ldg(src + ch.a), __ldg(src + ch.b)};
}
// ... and as they are stored: keys rotated. Done once for the scale and once
// for the codes: the raw values are half the registers of the rotated ones.
template <bool KEYS>
__device__ __forceinline__ void values_of(const AppendLaunch& p, const Raw& x, int pos, const Chunks& ch, float (&a)[8],
                                          float (&b)[8]) {
  unpack8(x.a, a);
  unpack8(x.b, b);
  if (KEYS && ch.rotated) {
    Angles g;
    load_angles(p, pos, ch, g);
    rotate(a, b, g, p.interleaved);
  }
}
__device__ __forceinline__ void store_codes(char* dst, const Chunks& ch, const float (&a)[8], const float (&b)[8],
                                            float inv) {
  reinterpret_cast<uint2*>(dst)[ch.a] = make_uint2(e4m3x4(a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv),
                                                   e4m3x4(a[4] * inv, a[5] * inv, a[6] * inv, a[7] * inv));
  reinterpret_cast<uint2*>(dst)[ch.b] = make_uint2(e4m3x4(b[0] * inv, b[1] * inv, b[2] * inv, b[3] * inv),
                                                   e4m3x4(b[4] * inv, b[5] * inv, b[6] * inv, b[7] * inv));
}
// Bring the codes of cells [0, n) to a scale that is 1 / f times the old one.
__device__ __forceinline__ void rescale_cells(char* base, long long tok_stride, int n, int dim, float f, int tid,
                                              int nthreads) {
  const int per = dim / 16;
  for (int i = tid; i < n * per; i += nthreads) {
    uint4* at = reinterpret_cast<uint4*>(base + (i / per) * tok_stride) + i % per;
    uint4 x = *at;
    uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[4];
      e4m3x4_to_f32(w[j], v);
      w[j] = e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
    }
    *at = x;
  }
}

// Rows [r0, r0 + window): the units that begin there. A unit is a run of
// neighbouring rows that are successive tokens of one request in one block.
// TPT: tokens of a whole block per thread.
template <bool KEYS, int TPT>
__device__ void block_cta(const AppendLaunch& p, int r0, int window, int h) {
  __shared__ uint32_t s_more[kWarps];  // bit j: row r0 + j goes on with the unit of the row before it
  __shared__ uint32_t s_live[kWarps];  // bit j: row r0 + j is appended
  __shared__ float s_amax[kWarps];
  __shared__ int s_pos[kThreads], s_blk[kThreads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int dim = p.c.dim, lph = dim / 16;
  const int bs = 1 << p.c.bs_log2;
  const long long* st = KEYS ? p.c.kst : p.c.vst;
  float* scales = KEYS ? p.c.ks : p.c.vs;
  char* cache = (KEYS ? p.c.k : p.c.v) + h * st[1];
  {
    const int row = r0 + tid;
    RowPlace r{-1, 0, -1};
    // each row is reported once: by the window it lies in
    if (row < p.rows && tid < window + bs) r = row_place(p, row, KEYS && h == 0 && tid < window);
    bool more = false;
    if (r.pos >= 0 && (r.pos & (bs - 1)) != 0 && row > 0) {
      const int n = p.seq_lens[row - 1];
      const int b = p.row_to_batch ? p.row_to_batch[row - 1] : row - 1;
      more = n == r.pos && b == r.batch;  // the row before is the token before (a live row: same block)
    }
    s_pos[tid] = r.pos;
    s_blk[tid] = r.blk;
    const uint32_t live = __ballot_sync(0xffffffffu, r.pos >= 0);
    const uint32_t go = __ballot_sync(0xffffffffu, more);
    if (lane == 0) {
      s_live[warp] = live;
      s_more[warp] = go;
    }
  }
  __syncthreads();
  // length of the unit that begins at row r0 + j
  auto unit_len = [&](int j) {
    int e = j + 1;
    while (e < kThreads) {
      const uint32_t w = ~s_more[e >> 5] >> (e & 31);
      if (w) {
        e += __ffs(w) - 1;
        break;
      }
      e = (e | 31) + 1;
    }
    return min(e, kThreads) - j;
  };
  const int l = lane % lph;
  const Chunks ch = chunks_of(l, KEYS ? p.rot : 0, dim);
  int small = 0;
  // the unit that begins at row r0 + j
  auto unit = [&](int j) {
    const int len = unit_len(j);
    const bool by_warp = len <= kSmallUnit;
    if (by_warp && (small++ % kWarps) != warp) return;
    const int row = r0 + j;
    const int pos = s_pos[j], blk = s_blk[j];
    const int off = pos & (bs - 1);
    char* base = cache + blk * st[0];
    float* scale = scales + static_cast<long long>(blk) * p.c.heads + h;
    const float old = off ? *scale : 0.f;
    if (by_warp) {
      const int tpw = 32 / lph;  // tokens at once: 4 (dim 128) or 8
      const int tok = lane / lph;
      const bool on = tok < len && tok < tpw;
      float a[8], bb[8], m = 0.f;
      if (on) {
        values_of<KEYS>(p, load_raw<KEYS>(p, row + tok, h, ch), pos + tok, ch, a, bb);
        m = amax16(a, bb, 0.f);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float s = fmaxf(old, needed_scale(m));
      if (on) store_codes(base + (off + tok) * st[2], ch, a, bb, 1.f / s);
      if (off && s != old) rescale_cells(base, st[2], off, dim, old / s, lane, 32);
      __syncwarp();  // every lane has read the old scale
      if (lane == 0) *scale = s;
    } else {
      const int tok0 = tid / lph, tstep = kThreads / lph;
      Raw x[TPT];
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < TPT; ++i)
        if (tok0 + i * tstep < len) x[i] = load_raw<KEYS>(p, row + tok0 + i * tstep, h, ch);
#pragma unroll
      for (int i = 0; i < TPT; ++i) {
        const int tok = tok0 + i * tstep;
        if (tok < len) {
          float a[8], bb[8];
          values_of<KEYS>(p, x[i], pos + tok, ch, a, bb);
          m = amax16(a, bb, m);
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (lane == 0) s_amax[warp] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_amax[w]);
      const float s = fmaxf(old, needed_scale(m));
      const float inv = 1.f / s;
#pragma unroll
      for (int i = 0; i < TPT; ++i) {
        const int tok = tok0 + i * tstep;
        if (tok < len) {
          float a[8], bb[8];
          // opaque, or the compiler keeps the rotated values of the first time
          asm volatile("" : "+r"(x[i].a.x), "+r"(x[i].a.y), "+r"(x[i].a.z), "+r"(x[i].a.w), "+r"(x[i].b.x),
                       "+r"(x[i].b.y), "+r"(x[i].b.z), "+r"(x[i].b.w));
          values_of<KEYS>(p, x[i], pos + tok, ch, a, bb);
          store_codes(base + (off + tok) * st[2], ch, a, bb, inv);
        }
      }
      if (off && s != old) rescale_cells(base, st[2], off, dim, old / s, tid, kThreads);
      __syncthreads();  // s_amax and the old scale have been read
      if (tid == 0) *scale = s;
    }
  };
  for (int w = 0; w < window; w += 32) {
    uint32_t begins = s_live[w >> 5] & ~s_more[w >> 5];
    if (window - w < 32) begins &= (1u << (window - w)) - 1u;
    for (; begins; begins &= begins - 1) unit(w + __ffs(begins) - 1);
  }
}

template <int TPT>
__global__ void __launch_bounds__(kThreads, 3) append_kv_kernel(const AppendLaunch p, int rows_per_cta,
                                                              int block_ctas, int window) {
  // the block CTAs first: they are the longer ones
  if (static_cast<int>(blockIdx.x) >= block_ctas) {
    row_cta(p, (blockIdx.x - block_ctas) * rows_per_cta, rows_per_cta);
    return;
  }
  const int u = blockIdx.x;
  const int h = u % p.c.heads;
  const int w = (u / p.c.heads) >> 1;
  if ((u / p.c.heads) & 1)
    block_cta<false, TPT>(p, w * window, window, h);
  else
    block_cta<true, TPT>(p, w * window, window, h);
}

}  // namespace

cudaError_t launch_append_kv(const AppendLaunch& p, cudaStream_t stream) {
  // one row per CTA while that gives every SM at most a few, else four: fewer
  // CTAs, whose threads have more heads each to keep in flight
  const int rows_per_cta = p.rows <= 512 ? 1 : 4;
  const int row_ctas = (p.q || !p.c.f8) ? (p.rows + rows_per_cta - 1) / rows_per_cta : 0;
  // decode rows are units of their own, one per warp; packed rows make units
  // of up to a block, so a window of a block leaves few CTAs without a unit
  const int window = p.row_to_batch ? std::max(32, 1 << p.c.bs_log2) : kWarps;
  const long long block_ctas = p.c.f8 ? (static_cast<long long>(p.rows) + window - 1) / window * p.c.heads * 2 : 0;
  const long long grid = row_ctas + block_ctas;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  // tokens of a block per thread: block_size / (256 threads / (dim / 16) lanes)
  const int tpt = std::max(1, (1 << p.c.bs_log2) * (p.c.dim / 16) / kThreads);
  const unsigned g = static_cast<unsigned>(grid);
  if (tpt == 1)
    append_kv_kernel<1><<<g, kThreads, 0, stream>>>(p, rows_per_cta, static_cast<int>(block_ctas), window);
  else if (tpt == 2)
    append_kv_kernel<2><<<g, kThreads, 0, stream>>>(p, rows_per_cta, static_cast<int>(block_ctas), window);
  else
    append_kv_kernel<4><<<g, kThreads, 0, stream>>>(p, rows_per_cta, static_cast<int>(block_ctas), window);
  return cudaGetLastError();
}

}  // namespace sai
