// What the three forms of the paged attention and their join share.
#pragma once

#include "common.cuh"
#include "paged.h"

namespace csa2 {

// A row's weight of a token, as it multiplies the token's codes of V, is the softmax's times the V scale of the
// token's page.  All forms hold it as 2^(u - M + 11) in fp16, u = z + log2(v scale) with the score z in log2 units
// and M the running maximum of u over the tokens that the row has seen, which may be 2^4 too small: it stays 11 bits
// down to 2^-25 of the row's largest, whatever the scales of pages that the row does not see or gives no weight.  The
// softmax's sum takes each weight's fp32 value over its V scale, times 2^-20, which keeps the sum within
// fp32 for V scales from 2^-100 (what lies below counts as that) to 2^100.
constexpr float kPagedLift = 11.f;
constexpr float kPagedSlack = 4.f;
constexpr float kPagedBias = 20.f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// log2 of a page's V scale.  The exponent is taken out: near 1 the approximation's error is absolute, 2^-22.
__device__ __forceinline__ float paged_v_log(float scale) {
  const uint32_t u = __float_as_uint(fmaxf(scale, 7.888609e-31f));  // 2^-100; a NaN counts as that
  float m;
  asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(m) : "f"(__uint_as_float((u & 0x7fffffu) | 0x3f800000u)));
  return (float)((int)(u >> 23) - 127) + m;
}
// What a weight is multiplied by in the softmax's sum.
__device__ __forceinline__ float paged_v_back(float v_log) { return ex2(-v_log - kPagedBias); }

// Bounded wait of a whole warp for an mbarrier's phase that lets the hardware suspend it for about a microsecond
// at a time: the default suspension is a few tens of cycles, and the parts of these kernels that wait then take
// issue slots from those that work.  Gives up after so many tries; its lanes agree on the answer (the chunk of
// paged_wide.cu 1,965 us, 1,941 where each lane goes by its own: what follows may be for the whole warp).
__device__ __forceinline__ bool paged_wait(uint64_t* bar, uint32_t parity, uint32_t tries) {
  const uint32_t a = smem_u32(bar);
#pragma unroll 1
  for (uint32_t i = 0; i < tries; ++i) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred P1;\n mbarrier.try_wait.parity.shared::cta.b64 P1, [%1], %2, %3;\n selp.b32 %0, 1, 0, P1;\n}\n"
        : "=r"(done)
        : "r"(a), "r"(parity), "r"(1000u)
        : "memory");
    if (__all_sync(0xffffffffu, done)) return true;
  }
  return false;
}
// A block whose waits ran out leaves nothing in flight: the copies' warp waits for the last of the `sent` copies
// (the n-th on barrier n % STAGES, one phase each) before the block ends.
template <int STAGES>
__device__ __forceinline__ void paged_drain(uint64_t (&full)[STAGES], uint32_t sent) {
  for (uint32_t i = sent > STAGES ? sent - STAGES : 0; i < sent; ++i) paged_wait(&full[i % STAGES], i / STAGES & 1, kPagedTries);
}

// Two fp32 at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;\n"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;\n"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}

// Four values as a register of codes.
__device__ __forceinline__ uint32_t e4m3_word(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 x, y;\n cvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n"
      " mov.b32 %0, {x, y};\n}\n"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// The four codes of a register (low byte first) as two pairs of f16.
__device__ __forceinline__ void f16_pairs(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}

// What a row's sums of weighted codes, relative to its maximum M (log2 units), are to be multiplied by: one over
// its denominator.  A row that saw no key is 0.
__device__ __forceinline__ float paged_factor(const PagedAttnParams& p, int head, float M, float L) {
  float den = L;
  if (p.sink != nullptr && M > -INFINITY) den += ex2(p.sink[head] * 1.4426950408889634f - M + (kPagedLift - kPagedBias));
  return L == 0.f ? 0.f : __fdividef(9.5367432e-7f, den);  // 2^-kPagedBias
}
// Four values of an output row.
template <int D>
__device__ __forceinline__ void paged_put(const PagedAttnParams& p, int row, int head, int d, float4 o, float factor) {
  const long long at = ((long long)row * (p.kv_heads * p.group) + head) * D + d;
  o.x *= factor, o.y *= factor, o.z *= factor, o.w *= factor;
  if (p.out_dtype == CSA2_T_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = o;
  } else {
    const bool h = p.out_dtype == CSA2_T_F16;
    const uint2 u = h ? make_uint2(pack_f16x2(o.x, o.y), pack_f16x2(o.z, o.w)) : make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = u;
  }
}

// What the warp that finds the pages tells the others about 128 tokens.
struct __align__(16) PagedInfo {
  float k_scale[8];   // of each 16 tokens
  float v_log[8];     // paged_v_log of their V scale
  float v_back[8];    // paged_v_back of that
  uint32_t flags;     // bits 0-7: 16 tokens have a page; 8-15: their scales say NaN
};
// Filled in by a whole warp, lane l (as l & 7) with the page id (-1: no token, -2: a bad entry) and scales of
// tokens 16 l ...
__device__ __forceinline__ void paged_tell(PagedInfo& info, int lane, int id, float sk, float sv) {
  const uint32_t pages = __ballot_sync(0xffffffffu, id != -2) & 0xffu;
  const uint32_t nans = __ballot_sync(0xffffffffu, sk != sk || sv != sv) & 0xffu;
  if (lane < 8) {
    const float v_log = paged_v_log(sv);
    info.k_scale[lane] = sk == sk ? sk : 0.f;
    info.v_log[lane] = v_log;
    info.v_back[lane] = paged_v_back(v_log);
    if (lane == 0) info.flags = pages | nans << 8;
  }
}

// n / group of a row index.  (The inverse is too large by less than one 2^64th, n below 2^31: exact.)
__device__ __forceinline__ int by_group(const PagedAttnParams& p, int n) {
  return p.group == 1 ? n : (int)__umul64hi((uint64_t)n, p.group_inv);
}
// The first token that a row at a position sees.
__device__ __forceinline__ int first_seen(const PagedAttnParams& p, int pos) {
  return p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
}
// Division of numbers that rarely need 64 bits.
__device__ __forceinline__ long long div_rarely_long(long long a, int b) {
  return (unsigned long long)a >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}

// The query rows and tokens of one sequence.
struct PagedSeq {
  int index;
  int first, rows;     // its first query row; query rows x heads of a group
  int ctx, kv;         // position of its first query row; cached tokens
  int tiles;           // tiles of a kv head
};
template <int NR>
__device__ __forceinline__ PagedSeq paged_seq(const PagedAttnParams& p, int b) {
  PagedSeq s;
  const int r0 = p.row_start[b], r1 = p.row_start[b + 1];
  s.index = b;
  s.first = min(max(r0, 0), p.n_rows);
  const int n = max(min(r1, p.n_rows) - s.first, 0);
  const int kv = min(max(p.kv_len[b], 0), kPagedMostTokens);
  s.ctx = n > 0 ? kv - (r1 - s.first) : 0;
  s.kv = min(kv, p.table_cols << p.page_shift);
  s.rows = n * p.group;
  s.tiles = (s.rows + NR - 1) / NR;
  return s;
}

}  // namespace csa2
