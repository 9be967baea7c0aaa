// Page writer: key and value rows into a cache of E4M3 codes with one power-of-two scale per (page,
// head).
//
//   need  = the smallest 2^e with max |x| <= 448 * 2^e over the page's new rows of the head
//   scale = need, or max(the page's scale, need) where the page holds older tokens of the sequence
//   code  = E4M3(x / scale), nearest even
//
// E4M3 is a floating-point format, so a power of two loses nothing against max / 448: the scale only
// moves the range.  It makes x / scale exact, and older tokens whose page's scale grows are moved by
// an exact factor: only codes that reach the subnormals lose bits.
//
// A task is one page and head of K or of V.  A block looks at `chunk` rows for those that open a page
// or a sequence, and spreads these tasks over its eight warps: eight tasks of a warp in a decode step
// (a row each), two of four warps for a whole page.  The rows are read once into registers (up to 8
// pieces a thread; what a long page has beyond is read again from L2), reduced to the largest
// magnitude, and written as codes.  Bound by memory: 2 (or 4) bytes read and one written per value.
#include "common.cuh"
#include "paged.h"

namespace csa2 {
namespace {

constexpr int kThreads = 256;
constexpr int kHeldPieces = 8;
constexpr int kExpMin = -100, kExpMax = 119;
constexpr uint32_t kNaN = 0x7fc00000u;

template <typename T>
struct In;  // a piece of 16 bytes as floats
template <>
struct In<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(uint4 u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) f[2 * k] = bf16_lo(w[k]), f[2 * k + 1] = bf16_hi(w[k]);
  }
};
template <>
struct In<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(uint4 u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
      f[2 * k] = v.x, f[2 * k + 1] = v.y;
    }
  }
};
template <>
struct In<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(uint4 u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  }
};

// Two codes, `lo` in the low byte; a NaN becomes code 0 (the page's scale says NaN instead, so that
// every code is finite and a masked token cannot spoil a sum).
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t r;
  lo = lo != lo ? 0.f : lo;
  hi = hi != hi ? 0.f : hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 values2(uint32_t codes) {
  const uint32_t h = e4m3x2_to_f16x2((uint16_t)codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The smallest 2^e >= amax / 448, e in [kExpMin, kExpMax]: 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, kExpMin), kExpMax);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
__device__ __forceinline__ bool power_of_two(float s) {
  const uint32_t u = __float_as_uint(s);
  return (u & 0x7fffffu) == 0 && (u >> 23) > 0 && (u >> 23) < 254;  // and 1 / s a normal number
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) page_write_kernel(const PageWriteParams p) {
  constexpr int N = In<T>::N;
  constexpr int PR = D / N;  // pieces of a row
  __shared__ int list[128];  // rows that open a task
  __shared__ int count;
  __shared__ float warp_max_s[kThreads / 32];
  __shared__ int warp_nan_s[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = blockIdx.y;
  const int page = 1 << p.page_shift;
  if (tid == 0) count = 0;
  __syncthreads();
  const int r0 = blockIdx.x * p.chunk;
  if (tid < p.chunk && r0 + tid < p.n_rows) {
    const int r = r0 + tid, b = p.seq_of_row[r];
    if ((unsigned)b < (unsigned)p.n_seq) {
      const int first = p.row_start[b], end = p.row_start[b + 1];
      const int pos = p.kv_len[b] - end + r;
      if (r >= first && r < end && pos >= 0 && (r == first || pos == 0 || (pos & (page - 1)) == 0)) list[atomicAdd(&count, 1)] = r;
    }
  }
  __syncthreads();
  const int tasks = 2 * count;
  if (tasks == 0) return;
  const int wpt = tasks <= 2 ? 4 : tasks <= 4 ? 2 : 1;  // warps of a task
  const int group = warp / wpt, groups = kThreads / 32 / wpt;
  const int gt = tid - group * wpt * 32, gn = wpt * 32;  // thread of the group, its threads
  for (int task = group; task < tasks; task += groups) {
    const int r = list[task >> 1], kv = task & 1;
    const int b = p.seq_of_row[r];
    const int end = min(p.row_start[b + 1], p.n_rows);
    const int pos = p.kv_len[b] - p.row_start[b + 1] + r;
    const int off = pos & (page - 1), col = pos >> p.page_shift;
    const int n = min(page - off, end - r);
    const int id = col < p.table_cols ? p.table[(long long)b * p.table_cols + col] : -1;
    if ((unsigned)id >= (unsigned)p.n_pages) {
      if (gt == 0 && p.dev_status) atomicExch(p.dev_status, (int)CSA2_EDEVICE_INDEX);
      continue;  // the whole group
    }
    const T* src = static_cast<const T*>(p.x[kv]) + (long long)r * p.x_row[kv] + (long long)head * p.x_head[kv];
    const long long slab = ((long long)id * p.kv_heads + head);
    uint8_t* dst = p.codes[kv] + (slab << p.page_shift) * D;
    float* sp = p.scale[kv] + slab;
    const float old = off ? *sp : 0.f;

    uint4 held[kHeldPieces];
    float amax = 0.f;
    bool nan = false;
    const int all = n * PR;
    auto take = [&](uint4 u) {
      float f[N];
      In<T>::get(u, f);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float a = fabsf(f[k]);
        nan |= a != a;
        amax = fmaxf(amax, a == INFINITY ? 0.f : a);  // infinities saturate and do not move the scale
      }
    };
#pragma unroll
    for (int k = 0; k < kHeldPieces; ++k) {
      const int i = gt + k * gn;
      if (i < all) held[k] = *reinterpret_cast<const uint4*>(src + (long long)(i / PR) * p.x_row[kv] + (i % PR) * N);
    }
#pragma unroll
    for (int k = 0; k < kHeldPieces; ++k)
      if (gt + k * gn < all) take(held[k]);
    for (int i = gt + kHeldPieces * gn; i < all; i += gn)
      take(*reinterpret_cast<const uint4*>(src + (long long)(i / PR) * p.x_row[kv] + (i % PR) * N));
    amax = warp_max(amax);
    nan = __any_sync(0xffffffffu, nan);
    if (wpt > 1) {
      if (lane == 0) warp_max_s[warp] = amax, warp_nan_s[warp] = nan;
      asm volatile("bar.sync %0, %1;\n" ::"r"(1 + group), "r"(gn) : "memory");
      for (int w = 0; w < wpt; ++w) {
        amax = fmaxf(amax, warp_max_s[group * wpt + w]);
        nan |= warp_nan_s[group * wpt + w] != 0;
      }
    }
    float s = amax > 0.f ? scale_for(amax) : __uint_as_float((uint32_t)(kExpMin + 127) << 23);
    nan |= old != old;
    if (off && old > s) s = old;
    if (off && !nan && old < s) {  // older tokens move to the larger scale
      const float f = __fdiv_rn(old, s);
      for (int i = gt; i < off * (D / 8); i += gn) {
        uint2* w = reinterpret_cast<uint2*>(dst) + i;
        uint2 u = *w;
        const float2 a = values2(u.x & 0xffffu), c = values2(u.x >> 16), d = values2(u.y & 0xffffu), e = values2(u.y >> 16);
        u.x = codes2(a.x * f, a.y * f) | codes2(c.x * f, c.y * f) << 16;
        u.y = codes2(d.x * f, d.y * f) | codes2(e.x * f, e.y * f) << 16;
        *w = u;
      }
    }
    const bool exact = power_of_two(s);
    const float inv = exact ? __fdiv_rn(1.f, s) : 0.f;
    auto write = [&](uint4 u, int i) {
      float f[N];
      In<T>::get(u, f);
#pragma unroll
      for (int k = 0; k < N; ++k) f[k] = exact ? f[k] * inv : __fdiv_rn(f[k], s);
      uint8_t* to = dst + (long long)(off + i / PR) * D + (i % PR) * N;
      const uint32_t w0 = codes2(f[0], f[1]) | codes2(f[2], f[3]) << 16;
      if constexpr (N == 8)
        *reinterpret_cast<uint2*>(to) = make_uint2(w0, codes2(f[4], f[5]) | codes2(f[6], f[7]) << 16);
      else
        *reinterpret_cast<uint32_t*>(to) = w0;
    };
#pragma unroll
    for (int k = 0; k < kHeldPieces; ++k)
      if (gt + k * gn < all) write(held[k], gt + k * gn);
    for (int i = gt + kHeldPieces * gn; i < all; i += gn)
      write(*reinterpret_cast<const uint4*>(src + (long long)(i / PR) * p.x_row[kv] + (i % PR) * N), i);
    if (wpt > 1) asm volatile("bar.sync %0, %1;\n" ::"r"(1 + group), "r"(gn) : "memory");  // all have read `old`
    else __syncwarp();
    if (gt == 0) *sp = nan ? __uint_as_float(kNaN) : s;
  }
}

template <typename T>
cudaError_t write_launch(const PageWriteParams& p, int head_dim, cudaStream_t stream) {
  const dim3 grid((p.n_rows + p.chunk - 1) / p.chunk, p.kv_heads);
  if (head_dim == 128) page_write_kernel<T, 128><<<grid, kThreads, 0, stream>>>(p);
  else page_write_kernel<T, 64><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_page_write(const PageWriteParams& p, int dtype, int head_dim, cudaStream_t stream) {
  if (dtype == CSA2_T_BF16) return write_launch<__nv_bfloat16>(p, head_dim, stream);
  if (dtype == CSA2_T_F16) return write_launch<__half>(p, head_dim, stream);
  return write_launch<float>(p, head_dim, stream);
}

}  // namespace csa2
