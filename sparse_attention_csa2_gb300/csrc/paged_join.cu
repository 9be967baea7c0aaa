// Joins what the blocks of the paged attention left open.
#include "common.cuh"
#include "paged.h"
#include "paged_dev.cuh"

namespace csa2 {
namespace {

// Joins the pieces of the tile that block x of the attention left open: its own sums and those of the
// blocks after it up to the tile's end.  WPR warps take a row: they take its pieces in turn (every load
// independent of the others), then are summed in order.  Four warps where there are few tiles, each in many
// blocks, one where the tiles are many or of 256 rows and their pieces few (96 sequences x 8 heads of 15 rows,
// 456 blocks: 3 us less than with four).  Bound by the latency of its loads: the first maxima set out with the word
// whether a tile is open, the first sums before their weights are known (one request of 2,048 tokens, both kernels:
// 9.0 -> 8.5 us).
constexpr int kJoinWarps = 4;
template <int D, int ROWS, int WPR>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const PagedAttnParams p) {
  __shared__ float weight[kJoinWarps][32];
  __shared__ float4 sum[kJoinWarps][D / 4];
  __shared__ float2 stat[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, of_row = warp % WPR;
  constexpr int L4 = D / 4, SUB = 32 / L4;  // lanes of a piece, pieces of a warp's load
  constexpr int AT_ONCE = kJoinWarps / WPR;
  constexpr int AHEAD = 8;                  // loads of a round that set out before its weights are known
  auto at = [](int i) { return i == 0 ? ROWS : 2 * ROWS * i; };  // row of piece i: the first block's second slot, then first slots
  auto stats = [&](int r, int i) {
    return *reinterpret_cast<const float2*>(p.part_ml + (2LL * blockIdx.x * ROWS + r + at(i)) * 2);
  };
  prior_done();
  // the first round's maxima and sums come together with the word whether there is anything
  const int r_first = blockIdx.y * AT_ONCE + warp / WPR, i_first = lane * WPR + of_row;
  const float2 ml_first = blockIdx.x + i_first < gridDim.x && r_first < ROWS ? stats(r_first, i_first) : make_float2(0.f, 0.f);
  const PagedOpen o = p.open[blockIdx.x];
  if (o.pieces == 0) return;
  for (int r0 = blockIdx.y * AT_ONCE; r0 < o.n; r0 += gridDim.y * AT_ONCE) {
    const int r = r0 + warp / WPR;
    if (WPR == 1 && r >= o.n) return;
    const float* part = p.part_o + (2LL * blockIdx.x * ROWS + r) * D + lane % L4 * 4;
    float M = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < o.pieces; i0 += 32 * WPR) {  // a round: pieces i0 + of_row, + WPR, ..
      const int n = min(32, (o.pieces - i0 - of_row + WPR - 1) / WPR);
      auto sums = [&](int i) { return *reinterpret_cast<const float4*>(part + (long long)at(i0 + i * WPR + of_row) * D); };
      float4 v[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) v[k] = lane / L4 + k * SUB < n ? sums(lane / L4 + k * SUB) : make_float4(0.f, 0.f, 0.f, 0.f);
      const int mine = i0 + lane * WPR + of_row;
      const float2 ml = mine >= o.pieces ? make_float2(-INFINITY, 0.f) : r == r_first && i0 == 0 ? ml_first : stats(r, mine);
      const float m = fmaxf(M, warp_max(ml.x));
      const float old = M == -INFINITY ? 1.f : ex2(M - m);
      const float w = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2(ml.x - m);
      weight[warp][lane] = w;
      __syncwarp();
      L = L * old + warp_sum(ml.y * w);
      a.x *= old, a.y *= old, a.z *= old, a.w *= old;
      M = m;
      auto take = [&](int i, float4 x) {
        const float f = weight[warp][i];
        a.x += x.x * f, a.y += x.y * f, a.z += x.z * f, a.w += x.w * f;
      };
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (lane / L4 + k * SUB < n) take(lane / L4 + k * SUB, v[k]);
#pragma unroll 8
      for (int i = lane / L4 + AHEAD * SUB; i < n; i += SUB) take(i, sums(i));
      __syncwarp();
    }
    if (SUB == 2) {
      a.x += __shfl_xor_sync(0xffffffffu, a.x, 16), a.y += __shfl_xor_sync(0xffffffffu, a.y, 16);
      a.z += __shfl_xor_sync(0xffffffffu, a.z, 16), a.w += __shfl_xor_sync(0xffffffffu, a.w, 16);
    }
    const int rr = o.row0 + r, tokn = by_group(p, rr), hq = o.kv_head * p.group + rr - tokn * p.group;
    if (WPR == 1) {
      if (lane < L4) paged_put<D>(p, o.first_row + tokn, hq, lane * 4, a, paged_factor(p, hq, M, L));
      continue;
    }
    if (lane < L4) sum[warp][lane] = a;
    if (lane == 0) stat[warp] = make_float2(M, L);
    __syncthreads();
    if (threadIdx.x < L4) {
      float T = -INFINITY, N = 0.f;
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) T = fmaxf(T, stat[w].x);
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) {
        const float2 ml = stat[w];
        if (ml.x == -INFINITY && ml.y == 0.f) continue;
        const float f = ml.x == -INFINITY ? 1.f : ex2(ml.x - T);
        const float4 v = sum[w][threadIdx.x];
        N += ml.y * f;
        t.x += v.x * f, t.y += v.y * f, t.z += v.z * f, t.w += v.w * f;
      }
      paged_put<D>(p, o.first_row + tokn, hq, threadIdx.x * 4, t, paged_factor(p, hq, T, N));
    }
    __syncthreads();
  }
}

template <int D, int ROWS>
cudaError_t join(const PagedAttnParams& p, int blocks, cudaStream_t stream) {
  if (ROWS == 256) return launch_behind(paged_join_kernel<D, ROWS, 1>, dim3(blocks, 32), kJoinWarps * 32, 0, stream, p);
  if (p.few_pieces) return launch_behind(paged_join_kernel<D, ROWS, 1>, dim3(blocks, ROWS / kJoinWarps), kJoinWarps * 32, 0, stream, p);
  return launch_behind(paged_join_kernel<D, ROWS, kJoinWarps>, dim3(blocks, ROWS), kJoinWarps * 32, 0, stream, p);
}

}  // namespace

cudaError_t launch_paged_join(const PagedAttnParams& p, int head_dim, int rows, int blocks, cudaStream_t stream) {
  if (head_dim == 128)
    return rows == 8    ? join<128, 8>(p, blocks, stream)
           : rows == 16 ? join<128, 16>(p, blocks, stream)
           : rows == 32 ? join<128, 32>(p, blocks, stream)
                        : join<128, 256>(p, blocks, stream);
  return rows == 8    ? join<64, 8>(p, blocks, stream)
         : rows == 16 ? join<64, 16>(p, blocks, stream)
                      : join<64, 256>(p, blocks, stream);
}

}  // namespace csa2
