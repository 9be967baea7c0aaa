// Parameters and launchers of the paged 8-bit cache's kernels (page plan, rotary positions with
// several axes, page writer, paged attention); the host side is paged_api.cu.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/csa2.h"

namespace csa2 {

// Raises a kernel's dynamic shared memory limit, once per kernel (Kernel: its address) and device.
template <auto Kernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launches a kernel behind the stream's work that may start before that is done: it calls prior_done() before
// it reads or writes memory, and reads nothing by the non-coherent path, whose loads may move ahead of it.  Decode steps
// are made of kernels of a few microseconds, of which a launch takes two.  They give no early leave themselves (what follows
// them may read what they write; from the attention to its join, at its start or at a tile's end, it measured no gain), but
// for the router, once the work before it is done: what follows that waits for what it writes.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}
#ifdef __CUDACC__
__device__ __forceinline__ void prior_done() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
#endif

// Places of a sequence's tokens that the attention computes with stay below the largest int: a table has no more
// columns, and what a length says beyond is cut.
constexpr int kPagedMostTokens = 0x7fffffff - 8192;

struct PagePlanParams {
  const int32_t* ctx_len;
  const int32_t* new_len;
  int n_seq;
  int page_size;
  int32_t* table;
  int table_cols;
  const int32_t* free_pages;
  int n_free;
  int max_rows;
  int32_t* row_start;
  int32_t* kv_len;
  int32_t* seq_of_row;
  int64_t* pos;
  int64_t* slot;
  int32_t* n_taken;
  int32_t* dev_status;
};
cudaError_t launch_page_plan(const PagePlanParams& p, cudaStream_t stream);

struct RopeAxesParams {
  const void* x;
  void* out;
  long long x_row, x_head, out_row, out_head;  // strides in elements
  int n_tokens, n_heads, head_dim;
  int rot_first, rot_dim;
  int copy_rest;                               // the dims outside the rotary range are copied to out
  const int64_t* pos;                          // [n_axes, n_tokens]
  uint64_t turns[CSA2_ROPE_AXES_MAX_PAIRS];    // frequency of a pair in turns per position, times 2^64
  uint8_t axis[CSA2_ROPE_AXES_MAX_PAIRS];
};
cudaError_t launch_rope_axes(const RopeAxesParams& p, int dtype, bool half_pairs, bool inverse, cudaStream_t stream);

struct PageWriteParams {
  const void* x[2];                 // k, v
  long long x_row[2], x_head[2];    // strides in elements
  uint8_t* codes[2];                // [n_pages, kv_heads, page, dim]
  float* scale[2];                  // [n_pages, kv_heads]
  int n_rows, n_seq, kv_heads, page_shift;
  int n_pages, table_cols;
  const int32_t* row_start;
  const int32_t* kv_len;
  const int32_t* seq_of_row;
  const int32_t* table;
  int chunk;                        // rows a block looks at
  int32_t* dev_status;
};
cudaError_t launch_page_write(const PageWriteParams& p, int dtype, int head_dim, cudaStream_t stream);

// What a block of the split attention leaves open: a tile whose last unit lies beyond its range, in so
// many pieces (its own and one of each block after it); 0: nothing is open.
struct PagedOpen {
  int pieces;
  int row0;                         // first row of the tile within the sequence's rows x heads
  int n;                            // its rows
  int first_row;                    // the sequence's first query row
  int kv_head;
};

constexpr uint32_t kPagedTries = 1u << 22;  // of a wait: each may suspend for about a microsecond, some 0.1 to 4 seconds

struct PagedAttnParams {
  const void* q;
  long long q_row, q_head;          // strides in elements
  int n_rows, n_seq, kv_heads, group;
  uint64_t group_inv;               // floor(2^64 / group) + 1 (0 for group 1): n / group is the product's upper half
  const int32_t* row_start;
  const int32_t* kv_len;
  const int32_t* table;
  int table_cols, n_pages, page_shift;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  float scale_log2;                 // softmax_scale * log2(e)
  int window;                       // 0: none
  const float* sink;
  void* out;                        // [n_rows, kv_heads * group, dim]
  int out_dtype;
  float* part_o;                    // [2 * blocks, rows of a tile, dim]: a block's first tile where it began before
  float* part_ml;                   // [.., 2] the block, its last where it goes on behind it
  PagedOpen* open;                  // [blocks]
  int few_pieces;                   // a tile lies in a few blocks in the mean, not in many
  uint32_t wait_tries;              // of a wait for a barrier (kPagedTries, or fewer in a self-test)
  int32_t* dev_status;
};
// Few query rows per (sequence, kv head): tiles of 8, or (dim 64) of 16.
cudaError_t launch_paged_attn(const PagedAttnParams& p, int q_dtype, int head_dim, int rows, int blocks, cudaStream_t stream);
// Some: tiles of 16 or 32, dim 128.
cudaError_t launch_paged_rows(const PagedAttnParams& p, int q_dtype, int rows, int blocks, cudaStream_t stream);
// Many: tiles of 256.
cudaError_t launch_paged_wide(const PagedAttnParams& p, int q_dtype, int head_dim, int blocks, cudaStream_t stream);
// The open tiles' pieces; both launch it.
cudaError_t launch_paged_join(const PagedAttnParams& p, int head_dim, int rows, int blocks, cudaStream_t stream);

}  // namespace csa2
