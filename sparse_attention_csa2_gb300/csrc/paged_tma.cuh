// Copies of a cache's codes by TMA, and shared-memory operands in the swizzles that TMA and tcgen05 share.
#pragma once

#include <cudaTypedefs.h>

#include "common.cuh"
#include "paged.h"
#include "tc05.cuh"

namespace csa2 {

struct CopyMaps {
  CUtensorMap k, v;
};

// A box of the map at (dim 0, token of the page, slab = page * heads + head).
__device__ __forceinline__ void tma_load_codes(void* dst, const CUtensorMap* tm, int token, int slab, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(0), "r"(token), "r"(slab), "r"(smem_u32(bar))
      : "memory");
}

// Byte offset of a 16-byte chunk in rows of B bytes in the swizzle of that width.
template <int B>
__device__ __forceinline__ int swizzled(int row, int chunk) {
  return row * B + ((B == 128 ? chunk ^ (row & 7) : B == 64 ? chunk ^ (row >> 1 & 3) : chunk ^ (row >> 2 & 1)) << 4);
}
// Shared-memory descriptors of such rows, groups of 8 rows one after the other, in two halves: the lower holds
// address >> 4 and the distance of the next panel along the dense dimension, the upper goes by the row's width.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr & 0x3ffffu) >> 4 | (lbo >> 4) << 16; }
__host__ __device__ constexpr uint32_t desc_hi(int row_bytes) {
  return (uint32_t)(8 * row_bytes >> 4) | 1u << 14 | (row_bytes == 128 ? 2u : row_bytes == 64 ? 4u : 6u) << 29;
}
// One lane of a converged warp.  The warp that issues products runs their loops as a whole, on values that are
// the same in all lanes, and only the instructions themselves in one: the descriptors then stay in uniform
// registers.  (One lane running the loops by itself issued a product every 70 to 85 cycles, slower than the
// tensor cores take them.)
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// D[tmem] (+)= A[smem] * B[smem], kind::f16 and kind::f8f6f4, and D (+)= A[tmem] * B[smem], kind::f16.
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %6};\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(a_hi), "r"(b_hi)
      : "memory");
}
__device__ __forceinline__ void mma_f8_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(hi)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 db;\n mov.b64 db, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(b_hi)
      : "memory");
}

// The map of the codes [pages x heads, page, dim] for boxes of `box` tokens.
inline bool make_codes_map(CUtensorMap* map, const uint8_t* codes, const PagedAttnParams& p, int dim, int box, CUtensorMapSwizzle swizzle) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  if (p.n_pages == 0 || p.table_cols == 0) return true;  // no page is ever read
  if (fn == nullptr) return false;
  const cuuint64_t page = 1ull << p.page_shift;
  const cuuint64_t dims[3] = {(cuuint64_t)dim, page, (cuuint64_t)p.n_pages * p.kv_heads};
  const cuuint64_t strides[2] = {(cuuint64_t)dim, dim * page};
  const cuuint32_t sizes[3] = {(cuuint32_t)dim, (cuuint32_t)box, 1}, one[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(codes), dims, strides, sizes, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace csa2
