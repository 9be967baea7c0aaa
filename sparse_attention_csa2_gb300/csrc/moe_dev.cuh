// What the two forms of the experts share: waits, copies and maps of weights, and a job's way from the router's ids.
#pragma once

#include "common.cuh"
#include "paged_dev.cuh"
#include "paged_tma.cuh"
#include "step.h"

namespace csa2 {

__device__ __forceinline__ bool try_phase(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n .reg .pred P1;\n mbarrier.try_wait.parity.shared::cta.b64 P1, [%1], %2;\n selp.b32 %0, 1, 0, P1;\n}\n"
               : "=r"(done)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return done != 0;
}
// Waits of a whole warp, for one barrier or for two at once, that end early once another part of the block has given up.
__device__ __forceinline__ bool moe_wait(uint64_t* bar, uint32_t parity, uint32_t tries, volatile int* dead) {
#pragma unroll 1
  for (uint32_t i = 0; i < tries; ++i) {
    if (__all_sync(0xffffffffu, try_phase(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *dead != 0)) return false;
  }
  *dead = 1;
  return false;
}
__device__ __forceinline__ bool moe_wait(uint64_t* bar, uint32_t parity, uint64_t* bar2, uint32_t parity2, uint32_t tries, volatile int* dead) {
#pragma unroll 1
  for (uint32_t i = 0; i < tries; ++i) {
    const bool one = try_phase(bar, parity), two = try_phase(bar2, parity2);
    if (__all_sync(0xffffffffu, one && two)) return true;
    if (__any_sync(0xffffffffu, *dead != 0)) return false;
  }
  *dead = 1;
  return false;
}
// Waits for the last of n copies.
__device__ __forceinline__ void drain(uint64_t* full, int stages, uint32_t n) {
  for (uint32_t i = n > (uint32_t)stages ? n - stages : 0; i < n; ++i) paged_wait(&full[i % stages], i / stages & 1, kPagedTries);
}

// A barrier of some warps of a block (N threads), and whether any of their threads says so.
template <int ID, int N>
__device__ __forceinline__ void part_sync() {
  asm volatile("bar.sync %0, %1;\n" ::"n"(ID), "n"(N) : "memory");
}
template <int ID, int N>
__device__ __forceinline__ bool part_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(ID), "n"(N)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ int load_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];\n" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void copy_row(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* tm, int col, int row, int expert, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(col), "r"(row), "r"(expert), "r"(smem_u32(bar))
      : "memory");
}

// Moves a counter on behind what the block has written and this thread knows of (a release is enough: with a
// fence before it 5 tokens' layer of 60 experts took 2 us more), also for copies by others; and with the old value,
// behind what others have told.
__device__ __forceinline__ void tell(int* counter) {
  asm volatile("fence.proxy.async.global;\nred.release.gpu.global.add.s32 [%0], 1;\n" ::"l"(counter) : "memory");
}
__device__ __forceinline__ int count_on(int* counter) {
  int v;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;\n" : "=r"(v) : "l"(counter) : "memory");
  return v;
}
// A counter that other blocks move on; false where it does not get there.
__device__ __forceinline__ bool wait_count(const int* counter, int most, uint32_t tries, volatile int* dead) {
  bool ok = true;
  for (uint32_t i = 0; load_acquire(counter) < most; ++i) {
    if (i >= tries || *dead) {
      ok = false;
      break;
    }
    __nanosleep(100);
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) *dead = 1;
  return ok;
}

// The expert of entry i of the tokens' ids, or -1: none, or out of range (reported); and whether the entries of its token
// before it name the same one (its weight then counts there).
__device__ __forceinline__ int expert_of(const MoeParams& p, int i) {
  const int e = p.ids[i];
  if (e >= 0 && e < p.experts) return e;
  if (e != -1 && blockIdx.x == 0 && p.dev_status != nullptr) atomicExch(p.dev_status, (int)CSA2_EDEVICE_INDEX);
  return -1;
}
__device__ __forceinline__ bool named_before(const int16_t* ids, int k, int i) {
  const int e = ids[i];
  bool before = false;
  if (e >= 0)
    for (int j = i / k * k; j < i; ++j) before |= ids[j] == e;
  return before;
}
// The weight of an expert that entry (t, s) names first: with those of the entries that name it again.
__device__ __forceinline__ float weight_of(const MoeParams& p, int t, int s, bool dup) {
  float w = p.weights[t * p.k + s];
  if (dup) {
    const int e = p.ids[t * p.k + s];
    for (int j = s + 1; j < p.k; ++j)
      if (p.ids[t * p.k + j] == e) w += p.weights[t * p.k + j];
  }
  return w;
}
// h of its two products.
__device__ __forceinline__ float gated(float gate, float up, float limit) {
  gate = gate > limit ? limit : gate;  // a NaN stays
  up = up > limit ? limit : up < -limit ? -limit : up;
  return gate / (1.f + expf(-gate)) * up;
}
__device__ __forceinline__ void put_out(const MoeParams& p, long long row, int d, float v) {
  const long long at = row * p.out_row + d;
  if (p.out_dtype == CSA2_T_F32) static_cast<float*>(p.out)[at] = v;
  else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
}

// `rows` rows of y from `row` on, of tokens t0 .. t0 + nt: the sums of what their experts gave, in the order of their slots;
// row_of(t, s) is the place of a token's slot among the parts, or -1.  By N threads, AT_ONCE sums to a thread and some of their
// parts at a time, since the last ones are what a call ends with.
template <int N, int AT_ONCE, typename F>
__device__ __forceinline__ void add_parts_of(const MoeParams& p, int thread, int row, int rows, int t0, int nt, int slots, F row_of) {
  constexpr int PARTS = 8 / AT_ONCE;
  const int per = rows / 4, all = nt * per;
  for (int o0 = thread; o0 < all; o0 += AT_ONCE * N) {
    float4 v[AT_ONCE] = {};
    int t[AT_ONCE], d[AT_ONCE];
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const int o = o0 + u * N;
      t[u] = t0 + o / per, d[u] = row + o % per * 4;
      if (o >= all || d[u] >= p.dim) t[u] = -1;
    }
    for (int s0 = 0; s0 < slots; s0 += PARTS) {
      float4 x[AT_ONCE][PARTS];
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u)
#pragma unroll
        for (int s = 0; s < PARTS; ++s) {
          const int at = t[u] >= 0 && s0 + s < slots ? row_of(t[u], s0 + s) : -1;
          x[u][s] = at >= 0 ? __ldcg(reinterpret_cast<const float4*>(p.part + (long long)at * p.dim + d[u])) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u)
#pragma unroll
        for (int s = 0; s < PARTS; ++s) v[u].x += x[u][s].x, v[u].y += x[u][s].y, v[u].z += x[u][s].z, v[u].w += x[u][s].w;
    }
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u)
      if (t[u] >= 0) {
        put_out(p, t[u], d[u], v[u].x), put_out(p, t[u], d[u] + 1, v[u].y);
        put_out(p, t[u], d[u] + 2, v[u].z), put_out(p, t[u], d[u] + 3, v[u].w);
      }
  }
}
template <int N, typename F>
__device__ __forceinline__ void add_parts(const MoeParams& p, int thread, int row, int rows, int t0, int nt, int slots, F row_of) {
  if (nt * (rows / 4) <= N) add_parts_of<N, 1>(p, thread, row, rows, t0, nt, slots, row_of);
  else add_parts_of<N, 4>(p, thread, row, rows, t0, nt, slots, row_of);
}

// The end of a block, by one thread: 0 while others are still at it; of the last one 1, or 2 where a wait ran out in one of them.
__device__ __forceinline__ int leave(const MoeParams& p, bool dead) {
  __threadfence();
  if (dead && p.dev_status != nullptr) atomicExch(p.dev_status, (int)CSA2_ETIMEOUT);
  const int left = atomicAdd(p.left, dead ? 1 << 16 | 1 : 1) + (dead ? 1 << 16 | 1 : 1);
  return (left & 0xffff) != (int)gridDim.x ? 0 : left >> 16 ? 2 : 1;
}
// Rows of y from `first` on, every `step`-th, by N threads.
template <int N>
__device__ __forceinline__ void fill_out(const MoeParams& p, int thread, int first, int step, float v) {
#pragma unroll 1
  for (int t = first; t < p.tokens; t += step)
#pragma unroll 1
    for (int d = thread; d < p.dim; d += N) put_out(p, t, d, v);
}

struct MoeMaps {
  CUtensorMap up, down;
};
// Boxes of 128 bytes x box_rows rows of matrices [n, rows, cols].
inline bool make_expert_map(CUtensorMap* map, const void* base, bool codes, uint64_t cols, uint64_t rows, uint64_t n, uint32_t box_rows) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  if (fn == nullptr) return false;
  const uint64_t size = codes ? 1 : 2;
  const cuuint64_t dims[3] = {cols, rows, n};
  const cuuint64_t strides[2] = {cols * size, cols * rows * size};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / size), box_rows, 1}, one[3] = {1, 1, 1};
  return fn(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
            box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}


}  // namespace csa2
