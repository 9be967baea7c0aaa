// Parameters and launchers of the kernels that follow attention in a decode step (norm with residual, router,
// experts, token sampling); the host side is step_api.cu.
#pragma once

#include <cuda_bf16.h>

#include "paged.h"

namespace csa2 {

struct AddNormParams {
  const void* x;
  const void* residual;
  void* sum;
  const void* gain;
  void* out;
  uint8_t* codes;
  float* scales;
  long long x_row, residual_row, sum_row, out_row;  // strides in elements
  int n_rows, dim;
  int gain_dtype, out_dtype;
  int group;                                        // 0: the row
  float eps, gain_offset;
};
// sum_dtype: a csa2_type, or -1 without a residual.
cudaError_t launch_add_norm(const AddNormParams& p, int x_dtype, int sum_dtype, bool vectors, cudaStream_t stream);

#ifdef __CUDACC__
// Leave for a kernel launched behind (launch_behind) to take the SMs' room and wait there for this one's end.
// Behind prior_done(): what starts next need only wait for this kernel, not for those before it.
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
#endif

struct RouteParams {
  const void* x;
  long long x_row;
  const void* w;                // [experts, dim]
  const float* bias;            // [experts] or NULL
  int tokens, dim, experts, k;
  int score;                    // csa2_score
  int normalize;
  float scale;
  int32_t* ids;                 // [tokens, k]
  float* weights;
  float4* z;                    // [tokens, experts] product, how far off what is chosen by may be, what is chosen by
  int* done;                    // [pieces of the tokens] blocks that have ended
};
cudaError_t launch_route(const RouteParams& p, int x_dtype, int w_dtype, cudaStream_t stream);
constexpr int kRouteMostExperts = 1024, kRouteMostK = 32, kRouteMostTokens = 16384;
constexpr int kRouteTokens = 8;  // of a block, at most

struct MoeParams {
  const void* x;                // bf16 or E4M3 codes
  long long x_row;              // in elements
  const float* x_scale;         // [tokens], of codes
  const int32_t* ids;           // [tokens, k]
  const float* weights;
  const void* up;               // [experts + shared, 2 inner, dim]
  const void* down;             // [experts + shared, dim, inner]
  const float* up_scale;
  const float* down_scale;
  int tokens, k, experts, shared, dim, inner;
  float limit;
  void* out;
  long long out_row;
  int out_dtype;
  // workspace; a slot is one of a token's k + shared experts
  uint8_t* h;                   // [tokens, slots, inner] fp32, or (the wide form) [2, tokens x slots, inner] bf16
  float* part;                  // [tokens, slots, dim]
  void* x_rows;                 // [tokens, slots, dim] bf16: x's rows by experts (the wide form, whose h and part go by those too)
  int* ticket;
  int* left;                    // blocks that have ended
  int* gathered;                // pieces of x_rows (the wide form)
  int* up_done;                 // [most_jobs] tiles
  int* down_done;               // [tiles of dim] jobs
  uint32_t* h_top;              // [tokens, slots] largest |h| as bits (codes as weights)
  int most_jobs;                // a job: some tokens of an expert
  uint32_t wait_tries;
  int32_t* dev_status;
};
struct MoeTiles {
  int rows, tokens;
};
// Few tokens per expert, and some: weight rows of a tile, tokens of a job; launches.
MoeTiles moe_tiles();
MoeTiles moe_wide_tiles();
cudaError_t launch_moe(const MoeParams& p, bool w8, bool x8, cudaStream_t stream);
cudaError_t launch_moe_wide(const MoeParams& p, bool w8, bool x8, cudaStream_t stream);

constexpr int kSampleMostVocab = 524288;
struct SampleParams {
  const void* logits;
  long long row;                // stride in elements
  int rows, vocab;
  const float* u;               // [rows]; the other settings may be NULL
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int64_t* token;
  float* logprob;               // or NULL
  uint2 pow2[256];              // 2^(j/256): in units of 2^-30, and the bits of the fp32 value
};
cudaError_t launch_sample(const SampleParams& p, int dtype, cudaStream_t stream);

}  // namespace csa2
