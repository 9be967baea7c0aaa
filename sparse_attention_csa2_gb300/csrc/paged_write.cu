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
// (a row each), two of four warps for a page of 64.  The rows are read once into registers (up to 8
// pieces a thread; what a long page has beyond is read again from L2), reduced to the largest
// magnitude, and written as codes; four blocks per SM (six where a thread holds one piece) keep the
// loads of some in flight while others reduce and write.  Bound by memory: 2 (or 4) bytes read and one
// written per value.  32,768 rows of 8 heads of 128, bf16 (202 MB): 34.5 us, 5.8 TB/s (86% of a copy's
// rate), fp32 (336 MB) 56.3 us, 6.0 TB/s; 512 rows that append to their pages: 6.4 to 8.3 us in either, the chain of
// lookups, rows, scale and older codes.
#include "common.cuh"
#include "paged.h"

namespace csa2 {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksWanted = 2048;
constexpr int kExpMin = -100, kExpMax = 119;
constexpr uint32_t kNaN = 0x7fc00000u;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <typename T>
struct In;  // a piece of 16 bytes: as floats, and the largest magnitude of its words
template <>
struct In<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kOdd = 0x7f80u;  // magnitudes from here on are infinities and NaN
  static __device__ __forceinline__ uint32_t most(uint32_t m, uint32_t w) { return max_u16x2(m, w & 0x7fff7fffu); }
  static __device__ __forceinline__ uint32_t magnitude(uint32_t m) { return max(m & 0xffffu, m >> 16); }
  static __device__ __forceinline__ float value(uint32_t m) { return __uint_as_float(m << 16); }
  static __device__ __forceinline__ void get(uint4 u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) f[2 * k] = bf16_lo(w[k]), f[2 * k + 1] = bf16_hi(w[k]);
  }
};
template <>
struct In<__half> {
  static constexpr int N = 8;
  static constexpr uint32_t kOdd = 0x7c00u;
  static __device__ __forceinline__ uint32_t most(uint32_t m, uint32_t w) { return max_u16x2(m, w & 0x7fff7fffu); }
  static __device__ __forceinline__ uint32_t magnitude(uint32_t m) { return max(m & 0xffffu, m >> 16); }
  static __device__ __forceinline__ float value(uint32_t m) { return __half2float(__ushort_as_half((unsigned short)m)); }
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
  static constexpr uint32_t kOdd = 0x7f800000u;
  static __device__ __forceinline__ uint32_t most(uint32_t m, uint32_t w) { return max(m, w & 0x7fffffffu); }
  static __device__ __forceinline__ uint32_t magnitude(uint32_t m) { return m; }
  static __device__ __forceinline__ float value(uint32_t m) { return __uint_as_float(m); }
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
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {  // of finite values
  uint32_t r;
  asm("{\n .reg .b16 x, y;\n cvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n"
      " mov.b32 %0, {x, y};\n}\n"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
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

// HELD: pieces of a thread that stay in registers.
template <typename T, int D, int HELD>
__global__ void __launch_bounds__(kThreads, HELD == 1 ? 6 : 4) page_write_kernel(const PageWriteParams p) {
  constexpr int N = In<T>::N;
  constexpr int PR = D / N;  // pieces of a row
  __shared__ int4 list[128];  // rows that open a task: row, rows of the task, place in the page, page
  __shared__ int count;
  __shared__ uint32_t warp_most[kThreads / 32];
  __shared__ float warp_max_s[kThreads / 32];
  __shared__ int warp_nan_s[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int page = 1 << p.page_shift;
  if (tid == 0) count = 0;
  prior_done();
  __syncthreads();
  const int r0 = blockIdx.x * p.chunk;
  if (HELD == 1) {  // the rows' way from memory overlaps the lookups that say where they go
    constexpr int LINES = D * (int)sizeof(T) / 128;
    const int i = tid / LINES, line = tid % LINES, kv = i & 1, r = r0 + (i >> 1);
    if (i < 2 * p.chunk && r < p.n_rows) {
      const char* at = reinterpret_cast<const char*>(static_cast<const T*>(p.x[kv]) + (long long)r * p.x_row[kv] +
                                                     (long long)blockIdx.y * p.x_head[kv]) + 128 * line;
      asm volatile("prefetch.global.L2 [%0];\n" ::"l"(at));
    }
  }
  if (tid < p.chunk && r0 + tid < p.n_rows) {
    const int r = r0 + tid, b = p.seq_of_row[r];
    if ((unsigned)b < (unsigned)p.n_seq) {
      const int first = p.row_start[b], end = p.row_start[b + 1];
      const int pos = p.kv_len[b] - end + r, off = pos & (page - 1);
      if (r >= first && r < end && pos >= 0 && (r == first || pos == 0 || off == 0)) {
        const int col = pos >> p.page_shift;
        const int at = atomicAdd(&count, 1);
        list[at] = make_int4(r, min(page - off, min(end, p.n_rows) - r), off,
                             col < p.table_cols ? p.table[(long long)b * p.table_cols + col] : -1);
      }
    }
  }
  __syncthreads();
  const int tasks = 2 * count;  // of a head
  if (tasks == 0) return;
  // warps of a task: those that hold a page's pieces in registers, or more where the tasks are few
  const int fit = HELD == 1 ? 1 : max(1, min(8, (PR << p.page_shift) / (32 * HELD)));
  const int wpt = max(fit, tasks <= 2 ? 4 : tasks <= 4 ? 2 : 1);
  const int group = warp / wpt, groups = kThreads / 32 / wpt;
  const int gt = tid - group * wpt * 32, gn = wpt * 32;  // thread of the group, its threads
  for (int head = blockIdx.y; head < p.kv_heads; head += gridDim.y)
  for (int task = group; task < tasks; task += groups) {
    const int4 what = list[task >> 1];
    const int r = what.x, n = what.y, off = what.z, id = what.w, kv = task & 1;
    if ((unsigned)id >= (unsigned)p.n_pages) {
      if (gt == 0 && p.dev_status) atomicExch(p.dev_status, (int)CSA2_EDEVICE_INDEX);
      continue;  // the whole group
    }
    const T* src = static_cast<const T*>(p.x[kv]) + (long long)r * p.x_row[kv] + (long long)head * p.x_head[kv];
    const long long slab = ((long long)id * p.kv_heads + head);
    uint8_t* dst = p.codes[kv] + (slab << p.page_shift) * D;
    float* sp = p.scale[kv] + slab;
    const float old = off ? *sp : 0.f;

    uint4 held[HELD];
    // this thread's pieces: column gt % PR of rows gt / PR, + rows_at_once, ..
    const int row0 = gt / PR, rows_at_once = gn / PR;
    const T* from = src + row0 * p.x_row[kv] + gt % PR * N;
    const long long step = rows_at_once * p.x_row[kv];
    auto piece = [&](const T* at) { return *reinterpret_cast<const uint4*>(at); };
    auto group_sync = [&]() {
      if (wpt > 1) asm volatile("bar.sync %0, %1;\n" ::"r"(1 + group), "r"(gn) : "memory");
      else __syncwarp();
    };
#pragma unroll
    for (int k = 0; k < HELD; ++k) held[k] = row0 + k * rows_at_once < n ? piece(from + k * step) : make_uint4(0, 0, 0, 0);
    uint32_t most = 0;
    auto take = [&](uint4 u) { most = In<T>::most(In<T>::most(In<T>::most(In<T>::most(most, u.x), u.y), u.z), u.w); };
#pragma unroll
    for (int k = 0; k < HELD; ++k) take(held[k]);
    for (int r1 = row0 + HELD * rows_at_once; r1 < n; r1 += rows_at_once) take(piece(from + (r1 - row0) * p.x_row[kv]));
    most = __reduce_max_sync(0xffffffffu, In<T>::magnitude(most));
    if (wpt > 1) {
      if (lane == 0) warp_most[warp] = most;
      group_sync();
      for (int w = 0; w < wpt; ++w) most = max(most, warp_most[group * wpt + w]);
    }
    float amax = In<T>::value(most);
    bool nan = false;
    const bool odd = most >= In<T>::kOdd;
    if (odd) {  // infinities do not move the scale, a NaN is told by it: once more, value by value
      amax = 0.f;
      for (int r1 = row0; r1 < n; r1 += rows_at_once) {
        float f[N];
        In<T>::get(piece(from + (r1 - row0) * p.x_row[kv]), f);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const float a = fabsf(f[k]);
          nan |= a != a;
          amax = fmaxf(amax, a == INFINITY ? 0.f : a);
        }
      }
      amax = warp_max(amax);
      nan = __any_sync(0xffffffffu, nan);
      if (wpt > 1) {
        if (lane == 0) warp_max_s[warp] = amax, warp_nan_s[warp] = nan;
        group_sync();
        for (int w = 0; w < wpt; ++w) {
          amax = fmaxf(amax, warp_max_s[group * wpt + w]);
          nan |= warp_nan_s[group * wpt + w] != 0;
        }
      }
    }
    float s = amax > 0.f ? scale_for(amax) : __uint_as_float((uint32_t)(kExpMin + 127) << 23);
    nan |= old != old;
    if (off && !nan && old > s) s = old;  // codes of a page that says NaN go by its new rows alone: the same again
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
    const float inv = __uint_as_float(0x7f000000u - __float_as_uint(s));  // of a power of two
    const bool plain = exact && !odd;  // the usual case: no division, no NaN
    uint8_t* into = dst + (off + row0) * D + gt % PR * N;
    auto put = [&](uint8_t* to, const uint32_t (&w)[N / 4]) {
      if constexpr (N == 8) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(to) = w[0];
    };
    if (plain) {
      auto write = [&](uint4 u, uint8_t* to) {
        float f[N];
        In<T>::get(u, f);
        uint32_t w[N / 4];
#pragma unroll
        for (int k = 0; k < N / 4; ++k) w[k] = codes4(f[4 * k] * inv, f[4 * k + 1] * inv, f[4 * k + 2] * inv, f[4 * k + 3] * inv);
        put(to, w);
      };
#pragma unroll
      for (int k = 0; k < HELD; ++k)
        if (row0 + k * rows_at_once < n) write(held[k], into + k * rows_at_once * D);
      for (int r1 = row0 + HELD * rows_at_once; r1 < n; r1 += rows_at_once)
        write(piece(from + (r1 - row0) * p.x_row[kv]), into + (r1 - row0) * D);
    } else {
#pragma unroll 1
      for (int r1 = row0; r1 < n; r1 += rows_at_once) {
        float f[N];
        In<T>::get(piece(from + (r1 - row0) * p.x_row[kv]), f);
        uint32_t w[N / 4];
#pragma unroll
        for (int k = 0; k < N; ++k) f[k] = __fdiv_rn(f[k], s);
#pragma unroll
        for (int k = 0; k < N / 4; ++k) w[k] = codes2(f[4 * k], f[4 * k + 1]) | codes2(f[4 * k + 2], f[4 * k + 3]) << 16;
        put(into + (r1 - row0) * D, w);
      }
    }
    group_sync();  // all have read `old` and the warps' maxima
    if (gt == 0) *sp = nan ? __uint_as_float(kNaN) : s;
  }
}

template <typename T>
cudaError_t write_launch(const PageWriteParams& p, int head_dim, cudaStream_t stream) {
  // heads split over blocks until each SM has some blocks one after the other
  const int chunks = (p.n_rows + p.chunk - 1) / p.chunk;
  int y = 1;
  while (y < p.kv_heads && (long long)chunks * y < kBlocksWanted) y = y * 2 < p.kv_heads ? y * 2 : p.kv_heads;
  const dim3 grid(chunks, y);
  auto go = [&](auto kernel) { return launch_behind(kernel, grid, kThreads, 0, stream, p); };
  if (p.chunk > 4) return head_dim == 128 ? go(page_write_kernel<T, 128, 8>) : go(page_write_kernel<T, 64, 8>);
  return head_dim == 128 ? go(page_write_kernel<T, 128, 1>) : go(page_write_kernel<T, 64, 1>);  // a row or two to a task
}

}  // namespace

cudaError_t launch_page_write(const PageWriteParams& p, int dtype, int head_dim, cudaStream_t stream) {
  if (dtype == CSA2_T_BF16) return write_launch<__nv_bfloat16>(p, head_dim, stream);
  if (dtype == CSA2_T_F16) return write_launch<__half>(p, head_dim, stream);
  return write_launch<float>(p, head_dim, stream);
}

}  // namespace csa2
