// Page plan (block tables and slot maps from request lengths) and rotary positions with several
// axes.
#include "common.cuh"
#include "paged.h"

namespace csa2 {

int device_sm_count();

namespace {

// ----------------------------------------------------------------------------- page plan
// Two exclusive sums over the sequences, of the new rows and of the pages these need, then one
// lookup per row: its sequence (the last whose first row is at or before it), position and slot.
//
// Every block forms both sums for itself in shared memory (a few KB of lengths, read from L2) and
// then takes its share of the rows and pages, so that one launch does it all: a scan in a kernel of
// its own would add a launch to a call that takes a few microseconds at the sizes of a decode step.
// Bound by that latency below some 10^5 rows and by the 20 bytes written per row above: 256 decoding sequences
// 4.7 us (a launch and three dependent loads), 260,000 rows of 48 prompts 5.4 us.
constexpr int kPlanThreads = 512;
constexpr int kPlanRows = 4;  // consecutive rows of a thread: one search, 16-byte stores

constexpr int kMostTokens = 1 << 30;  // of a sequence, cached and new: their sum and a row's position fit an int
constexpr unsigned kMostSum = 0x7fffffffu;

// A sum that stays at the largest int: lengths that have it are reported, and the table and rows below stay in
// their bounds.
__device__ __forceinline__ unsigned sum_of(unsigned a, unsigned b) { return min(a + b, kMostSum); }
__device__ __forceinline__ int cached(const PagePlanParams& p, int b) { return min(max(p.ctx_len[b], 0), kMostTokens); }
__device__ __forceinline__ int pages_of(int tokens, int page) { return (int)(((unsigned)tokens + page - 1) / (unsigned)page); }

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PagePlanParams p) {
  extern __shared__ int sums[];  // [n_seq + 1] first rows, [n_seq + 1] first new pages
  int* row0 = sums;
  int* page0 = sums + p.n_seq + 1;
  __shared__ uint2 warp_sum_s[kPlanThreads / 32];
  const int tid = threadIdx.x;
  prior_done();
  // a thread sums a run of sequences, the block scans the threads' sums
  const int run = (p.n_seq + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * run, p.n_seq), b1 = min(b0 + run, p.n_seq);
  bool bad = false;
  unsigned rows = 0, need = 0;
  for (int b = b0; b < b1; ++b) {
    const int c = cached(p, b), n = min(max(p.new_len[b], 0), kMostTokens - 1);
    bad |= p.ctx_len[b] > kMostTokens || p.new_len[b] >= kMostTokens;
    row0[b] = (int)rows;
    page0[b] = (int)need;
    rows = sum_of(rows, n);
    need = sum_of(need, pages_of(c + n, p.page_size) - pages_of(c, p.page_size));
  }
  const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, rows, o), z = __shfl_up_sync(0xffffffffu, need, o);
    if (lane >= o) rows = sum_of(rows, y), need = sum_of(need, z);
  }
  if (lane == 31) warp_sum_s[warp] = make_uint2(rows, need);
  rows = __shfl_up_sync(0xffffffffu, rows, 1), need = __shfl_up_sync(0xffffffffu, need, 1);
  if (lane == 0) rows = need = 0;
  __syncthreads();
  uint2 before = make_uint2(0, 0), total = make_uint2(0, 0);
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const uint2 of = warp_sum_s[w];
    if (w < warp) before = make_uint2(sum_of(before.x, of.x), sum_of(before.y, of.y));
    total = make_uint2(sum_of(total.x, of.x), sum_of(total.y, of.y));
  }
  const int total_rows = (int)total.x, total_need = (int)total.y;
  const unsigned first_row = sum_of(before.x, rows), first_need = sum_of(before.y, need);
  for (int b = b0; b < b1; ++b) {
    row0[b] = (int)sum_of(row0[b], first_row);
    page0[b] = (int)sum_of(page0[b], first_need);
  }
  if (tid == 0) row0[p.n_seq] = total_rows, page0[p.n_seq] = total_need;
  __syncthreads();

  const int at = blockIdx.x * kPlanThreads + tid, all = gridDim.x * kPlanThreads;
  for (int b = at; b <= p.n_seq; b += all) {
    p.row_start[b] = row0[b];
    if (b < p.n_seq) {
      const int c = cached(p, b), kv = c + row0[b + 1] - row0[b];
      p.kv_len[b] = kv;
      bad |= pages_of(kv, p.page_size) > p.table_cols;
    }
  }
  if (at == 0) {
    p.n_taken[0] = total_need;
    bad |= total_need > p.n_free || total_rows > p.max_rows;
  }
  // the new pages' table entries
  for (unsigned u = at; u < (unsigned)total_need; u += all) {
    const int f = (int)u;
    int lo = 0, hi = p.n_seq;  // page0[lo] <= f < page0[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (page0[mid] <= f) lo = mid; else hi = mid;
    }
    const int col = pages_of(cached(p, lo), p.page_size) + f - page0[lo];
    if (col < p.table_cols) p.table[(long long)lo * p.table_cols + col] = f < p.n_free ? p.free_pages[f] : -1;
  }
  // rows
  for (int r = at * kPlanRows; r < p.max_rows; r += all * kPlanRows) {
    int lo = 0, hi = p.n_seq;
    if (r < total_rows)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (row0[mid] <= r) lo = mid; else hi = mid;
      }
    int seq[kPlanRows];
    int64_t pos[kPlanRows], slot[kPlanRows];
    int b = lo, known = -1, c = 0, held = 0;
#pragma unroll
    for (int k = 0; k < kPlanRows; ++k) {
      seq[k] = -1, pos[k] = -1, slot[k] = -1;
      if (r + k >= total_rows) continue;
      while (row0[b + 1] <= r + k) ++b;  // empty sequences too
      if (b != known) {
        c = cached(p, b);
        held = pages_of(c, p.page_size);
        known = b;
      }
      const int at_pos = c + r + k - row0[b];
      const int col = at_pos / p.page_size;
      int page = -1;
      if (col < p.table_cols) {
        const int f = page0[b] + col - held;
        page = col < held ? p.table[(long long)b * p.table_cols + col] : f < p.n_free ? p.free_pages[f] : -1;
      }
      seq[k] = b;
      pos[k] = at_pos;
      slot[k] = page < 0 ? -1 : (int64_t)page * p.page_size + at_pos % p.page_size;
      bad |= page < 0;
    }
    if (r + kPlanRows <= p.max_rows) {
      *reinterpret_cast<int4*>(p.seq_of_row + r) = make_int4(seq[0], seq[1], seq[2], seq[3]);
      longlong2* pp = reinterpret_cast<longlong2*>(p.pos + r);
      longlong2* ps = reinterpret_cast<longlong2*>(p.slot + r);
      pp[0] = make_longlong2(pos[0], pos[1]), pp[1] = make_longlong2(pos[2], pos[3]);
      ps[0] = make_longlong2(slot[0], slot[1]), ps[1] = make_longlong2(slot[2], slot[3]);
    } else {
#pragma unroll
      for (int k = 0; k < kPlanRows; ++k)
        if (r + k < p.max_rows) p.seq_of_row[r + k] = seq[k], p.pos[r + k] = pos[k], p.slot[r + k] = slot[k];
    }
  }
  if (bad && p.dev_status) atomicExch(p.dev_status, (int)CSA2_EDEVICE_INDEX);
}

// ----------------------------------------------------------------------------- rotary axes
// y = R(angle) x for each pair of a head's rotary dims, angle = pos[axis] * theta^(-2i/R).  The
// inverse turns by -angle, which is also the gradient: R is orthogonal.
//
// The angle is formed in turns as a 64-bit fixed-point product, position times frequency modulo one
// turn: exact but for the frequency's own rounding to 2^-64, so that one integer multiplication
// without a reduction keeps fp32's accuracy up to positions of some 2^38 (beyond, off by a 2^-64th of
// the position in turns).
//
// A thread owns one 16-byte piece of a token's head (for half-split pairs: the two pieces of
// partners) and walks the heads with it, so that its angles' sines are formed once and stay in
// registers.  Bound by memory: every element read and written once.  Half pairs of bf16, 336 MB in and out:
// 58.2 us, 5.8 TB/s (85% of a copy's rate); adjacent pairs of fp32, 64 of 192 dims turned, 208 MB: 35.3 us, 87%;
// a decode step's 1.2 MB: 3.0 us, a launch.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(uint4 u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) f[2 * k] = bf16_lo(w[k]), f[2 * k + 1] = bf16_hi(w[k]);
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(uint4 u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
      f[2 * k] = v.x, f[2 * k + 1] = v.y;
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    return make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]), pack_f16x2(f[6], f[7]));
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(uint4 u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// Sine and cosine of pair i's angle at a position.
__device__ __forceinline__ void turn(const RopeAxesParams& p, int i, int token, float& c, float& s) {
  const int64_t at = p.pos[(long long)p.axis[i] * p.n_tokens + token];
  const int32_t frac = (int32_t)(((uint64_t)at * p.turns[i] + 0x80000000ull) >> 32);  // of a turn, nearest 2^-32
  sincospif((float)frac * 4.656612873077393e-10f, &s, &c);                            // 2^-31: half turns
}

template <typename T, bool HALF, bool INV>
__global__ void __launch_bounds__(256) rope_axes_kernel(const __grid_constant__ RopeAxesParams p, int pieces,
                                                        int turned, int heads_per) {
  constexpr int N = Vec<T>::N;
  constexpr int NP = HALF ? N : N / 2;  // pairs of a piece
  const long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const int token = (int)(u / pieces), piece = (int)(u - (long long)token * pieces);
  if (token >= p.n_tokens) return;
  prior_done();
  const int h0 = blockIdx.y * heads_per, h1 = min(h0 + heads_per, p.n_heads);
  const T* src = static_cast<const T*>(p.x) + token * p.x_row + h0 * p.x_head;
  T* dst = static_cast<T*>(p.out) + token * p.out_row + h0 * p.out_head;
  const bool turns = piece < turned;
  int d0 = p.rot_first + piece * N;
  if (!turns) {  // dims outside the rotary range
    d0 = (piece - turned) * N;
    if (d0 >= p.rot_first) d0 += p.rot_dim;
  }
  if (HALF && !turns) {
#pragma unroll 4
    for (int h = h0; h < h1; ++h, src += p.x_head, dst += p.out_head)
      __stcs(reinterpret_cast<uint4*>(dst + d0), __ldcs(reinterpret_cast<const uint4*>(src + d0)));
    return;
  }
  float c[NP] = {}, s[NP] = {};
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    if (turns) turn(p, piece * NP + k, token, c[k], s[k]);
    if (INV) s[k] = -s[k];
  }
  const int d1 = d0 + p.rot_dim / 2;
#pragma unroll 4
  for (int h = h0; h < h1; ++h, src += p.x_head, dst += p.out_head) {
    float a[N];
    const uint4 ua = __ldcs(reinterpret_cast<const uint4*>(src + d0));
    if constexpr (HALF) {
      const uint4 ub = __ldcs(reinterpret_cast<const uint4*>(src + d1));
      float b[N], x[N], y[N];
      Vec<T>::get(ua, a);
      Vec<T>::get(ub, b);
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = a[k] * c[k] - b[k] * s[k], y[k] = a[k] * s[k] + b[k] * c[k];
      __stcs(reinterpret_cast<uint4*>(dst + d0), Vec<T>::put(x));
      __stcs(reinterpret_cast<uint4*>(dst + d1), Vec<T>::put(y));
    } else {
      float x[N];
      Vec<T>::get(ua, a);
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        x[2 * k] = a[2 * k] * c[k] - a[2 * k + 1] * s[k];
        x[2 * k + 1] = a[2 * k] * s[k] + a[2 * k + 1] * c[k];
      }
      __stcs(reinterpret_cast<uint4*>(dst + d0), turns ? Vec<T>::put(x) : ua);  // one way for both: a warp has both
    }
  }
}

template <typename T>
cudaError_t rope_launch(const RopeAxesParams& p, bool half, bool inv, cudaStream_t stream) {
  constexpr int N = Vec<T>::N;
  const int turned = half ? p.rot_dim / 2 / N : p.rot_dim / N;
  const int pieces = turned + (p.copy_rest ? (p.head_dim - p.rot_dim) / N : 0);
  const long long threads = (long long)p.n_tokens * pieces;
  const int blocks = (int)((threads + 255) / 256);
  // heads split over blocks until some sixteen blocks per SM are there, so that their ends even out; below
  // four heads a thread only for the sake of four blocks per SM, since each forms its sines anew
  int per = p.n_heads;
  const int sms = device_sm_count();
  while (per > 4 && (long long)blocks * ((p.n_heads + per - 1) / per) < 16LL * sms) per = (per + 1) / 2;
  while (per > 1 && (long long)blocks * ((p.n_heads + per - 1) / per) < 4LL * sms) per = (per + 1) / 2;
  const dim3 grid(blocks, (p.n_heads + per - 1) / per);
  auto go = [&](auto kernel) { return launch_behind(kernel, grid, 256, 0, stream, p, pieces, turned, per); };
  if (half) return inv ? go(rope_axes_kernel<T, true, true>) : go(rope_axes_kernel<T, true, false>);
  return inv ? go(rope_axes_kernel<T, false, true>) : go(rope_axes_kernel<T, false, false>);
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanParams& p, cudaStream_t stream) {
  const int smem = 2 * (p.n_seq + 1) * (int)sizeof(int);
  if (smem > 40 * 1024) {
    const cudaError_t e = allow_smem<page_plan_kernel>(2 * (8192 + 1) * (int)sizeof(int));
    if (e != cudaSuccess) return e;
  }
  const long long per = (long long)kPlanThreads * kPlanRows;
  long long blocks = (p.max_rows + per - 1) / per;
  if (blocks > device_sm_count()) blocks = device_sm_count();
  if (blocks < 1) blocks = 1;
  return launch_behind(page_plan_kernel, dim3((unsigned)blocks), kPlanThreads, smem, stream, p);
}

cudaError_t launch_rope_axes(const RopeAxesParams& p, int dtype, bool half_pairs, bool inverse, cudaStream_t stream) {
  if (dtype == CSA2_T_BF16) return rope_launch<__nv_bfloat16>(p, half_pairs, inverse, stream);
  if (dtype == CSA2_T_F16) return rope_launch<__half>(p, half_pairs, inverse, stream);
  return rope_launch<float>(p, half_pairs, inverse, stream);
}

}  // namespace csa2
