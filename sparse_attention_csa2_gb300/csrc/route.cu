// Router of a mixture-of-experts layer:
//
//   z = W x,  score = softmax(z) | 1 / (1 + e^-z) | sqrt(log(1 + e^z)),  ids = the k experts with the largest
//   score + bias (ties to the lower id),  w = score of those, over their sum, times a factor
//
// One launch: blocks compute the products of some experts with some tokens, and the block that ends last of those of a
// group of tokens chooses their experts, a warp per token.  Bound by latency for the few tokens of a decode step: W (some
// MB) and x are read once, all loads set out early, the choice is k rounds of two warp reductions.  At 4,096
// values and 384 experts, W 3 MB: one token 8 us, 32 tokens 11 to 14, 512 tokens 43 to 47.
//
// Which expert comes next can hang on the last bits of near scores.  Every product comes with a bound of its error (sums
// of the sizes of what was rounded on the way, so that it holds for large values that cancel, too).  Where two scores of
// which one is chosen are nearer than their bounds together, the warp computes the products in question again to some
// 2^-45 and chooses by those: the result is that of exact arithmetic but for scores that are equal to that (with softmax
// and a bias the sum under the scores is that of the first products).  By sums in two fp32 values (D. Knuth, "The Art of
// Computer Programming", volume 2, 4.2.2): in 64 bits, of which an SM has some two operations a cycle, 32 tokens
// of 384 experts, of which one or two ask for it, took 53 us instead of 26.
#include "common.cuh"
#include "step.h"

namespace csa2 {

int device_sm_count();

namespace {

constexpr int kWarps = 8;
constexpr int kTileWarps = 16;  // 4,096 values, 384 experts: 32 tokens 13 us, 512 45; with 8 warps 17 and 51, with 32 12 and 63

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
      } else {
        v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
      }
    }
  }
}
__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// The score of a product; softmax's before the division by its sum.
__device__ __forceinline__ float score_of(int kind, float z, float top) {
  if (kind == CSA2_SCORE_SOFTMAX) return expf(z - top);
  if (kind == CSA2_SCORE_SIGMOID) return 1.f / (1.f + expf(-z));
  return sqrtf(log1pf(expf(-fabsf(z))) + fmaxf(z, 0.f));
}
// How far score + bias may be off where z is off by `off`: its slope, softmax's sum moving by as much, and the functions'
// own roundings.  `score` with softmax's sum divided out.
__device__ __forceinline__ float slack_of(int kind, float z, float off, float score, float bias) {
  const float slope = kind == CSA2_SCORE_SOFTMAX   ? 2.f * score
                      : kind == CSA2_SCORE_SIGMOID ? score * (1.f - score)
                                                   : 0.5f / ((1.f + expf(-z)) * fmaxf(score, 1e-30f));
  return off * fmaxf(slope, 1e-3f) + 9.5367e-7f * (fabsf(score) + fabsf(bias));  // 2^-20
}
__device__ __forceinline__ double score_of64(int kind, double z, double top) {
  if (kind == CSA2_SCORE_SOFTMAX) return exp(z - top);
  if (kind == CSA2_SCORE_SIGMOID) return 1. / (1. + exp(-z));
  return sqrt(log1p(exp(-fabs(z))) + fmax(z, 0.));
}

// A sum in two fp32 values.
struct Sum2 {
  float sum = 0.f, rest = 0.f;
  template <bool EXACT>  // the product of a and b is an fp32 value, as those of two 16-bit values are
  __device__ __forceinline__ void add(float a, float b) {
    const float v = __fmul_rn(a, b), s = __fadd_rn(sum, v), of = __fsub_rn(s, sum);
    rest += __fadd_rn(__fsub_rn(sum, __fsub_rn(s, of)), __fsub_rn(v, of));
    if constexpr (!EXACT) rest += fmaf(a, b, -v);
    sum = s;
  }
};
// The products of x with two rows, to some 2^-45 of the sizes of what is added, by a warp.
template <typename TX, typename TW>
__device__ __forceinline__ double2 exact_products(const TW* w0, const TW* w1, const TX* x, int dim, int lane) {
  constexpr bool EXACT = sizeof(TW) == 2;
  Sum2 s0, s1;
#pragma unroll 4
  for (int j = lane * 8; j < dim; j += 256) {
    float a[8], b[8], c[8];
    load8(x + j, a);
    load8(w0 + j, b);
    load8(w1 + j, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) s0.template add<EXACT>(b[i], a[i]), s1.template add<EXACT>(c[i], a[i]);
  }
  return make_double2(warp_sum64((double)s0.sum + (double)s0.rest), warp_sum64((double)s1.sum + (double)s1.rest));
}

// Shared memory of the choice, per warp of it: the products, exact ones where they are needed, and keys.
__host__ __device__ constexpr int choice_bytes(int experts) { return (experts * 20 + 15) / 16 * 16; }

// What an expert is chosen by, and how far that may be off: without a bias the product itself, as scores grow with it.
// (Not softmax's score, which needs all.)  An infinite product is what it is.
__device__ __forceinline__ float4 told(const RouteParams& p, int e, float z, float off) {
  const bool infinite = fabsf(z) == INFINITY;
  if (infinite) off = 0.f;
  if (p.bias == nullptr || p.score == CSA2_SCORE_SOFTMAX) return make_float4(z, off, z, 0.f);
  const float score = score_of(p.score, z, 0.f);
  return make_float4(z, infinite ? 0.f : slack_of(p.score, z, off, score, p.bias[e]), score + p.bias[e], 0.f);
}

// The experts of token t, by a warp.
template <typename TX, typename TW>
__device__ void choose(const RouteParams& p, uint8_t* smem, int lane, int t) {
  double* exact = reinterpret_cast<double*>(smem);
  float2* product = reinterpret_cast<float2*>(exact + p.experts);  // and the slack of what it is chosen by
  uint32_t* key = reinterpret_cast<uint32_t*>(product + p.experts);
  const TX* x = static_cast<const TX*>(p.x) + (long long)t * p.x_row;
  const TW* w = static_cast<const TW*>(p.w);
  uint32_t mine = 0;  // the lane's best key, and its expert
  int at = 0;
  auto enter = [&](int e, float by) {
    const uint32_t k = by == by ? score_key(by) : 1u;  // a NaN comes last; 0: taken
    key[e] = k;
    if (k > mine) mine = k, at = e;
  };
  auto by_of = [](uint32_t k) { return k > 1u ? key_score(k) : __int_as_float(0x7fc00000); };
  const bool by_share = p.score == CSA2_SCORE_SOFTMAX && p.bias != nullptr;
#pragma unroll 4
  for (int e = lane; e < p.experts; e += 32) {
    const float4 z = __ldcg(p.z + (long long)t * p.experts + e);
    product[e] = make_float2(z.x, z.y);
    if (!by_share) enter(e, z.z);
  }
  // what softmax needs of all experts
  float top = 0.f, sum = 1.f;
  if (p.score == CSA2_SCORE_SOFTMAX) {
    top = -INFINITY;
    for (int e = lane; e < p.experts; e += 32) top = fmaxf(top, product[e].x);
    top = warp_max(top);
    sum = 0.f;
#pragma unroll 4
    for (int e = lane; e < p.experts; e += 32) sum += expf(product[e].x - top);
    sum = warp_sum(sum);
  }
  if (by_share)
    for (int e = lane; e < p.experts; e += 32) {
      const float score = score_of(p.score, product[e].x, top) / sum;
      product[e].y = slack_of(p.score, product[e].x, product[e].y, score, p.bias[e]);
      enter(e, score + p.bias[e]);
    }
  int id = 0;               // lane i: the i-th choice, and what it was chosen by
  float by = __int_as_float(0x7fc00000);
  for (int i = 0; i < p.k; ++i) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, mine);
    const int e = (int)__reduce_min_sync(0xffffffffu, mine == m ? (unsigned)at : 0x7fffffffu);
    if (mine == m && at == e) {
      key[e] = 0, mine = 0;
      for (int j = lane; j < p.experts; j += 32)
        if (key[j] > mine) mine = key[j], at = j;
    }
    if (lane == i) id = e, by = by_of(m);
  }
  // Choices in question: those that another one, or one that is left out, may lie before or behind.  (NaN: none.)
  const float slack = lane < p.k ? product[id].y : 0.f;
  float left_out = -INFINITY;  // the most that one of those may have
#pragma unroll 4
  for (int e = lane; e < p.experts; e += 32)
    if (key[e] > 1u) left_out = fmaxf(left_out, by_of(key[e]) + product[e].y);
  left_out = warp_max(left_out);
  bool in_question = by - slack < left_out;
  for (int i = 0; i < p.k; ++i) {
    const float other = __shfl_sync(0xffffffffu, by, i), its = __shfl_sync(0xffffffffu, slack, i);
    in_question |= i != lane && fabsf(by - other) < slack + its;
  }
  const long long to = (long long)t * p.k;
  if (__any_sync(0xffffffffu, in_question)) {
    // Again, by their exact products and those of whatever may lie before one of them; the list of these takes the keys'
    // place, behind it the other choices with what they were chosen by.
    const float least = -warp_max(in_question ? slack - by : -INFINITY);
    bool zero = true;  // a row of zeros, as padding has them
    int n = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
      const int e = e0 + lane;
      const uint32_t k = e < p.experts ? key[e] : 0u;
      if (e < p.experts) zero &= product[e].x == 0.f;
      const bool close = k > 1u && by_of(k) + product[e].y > least;
      const uint32_t m = __ballot_sync(0xffffffffu, close);
      if (close) key[n + __popc(m & lanemask_lt())] = e;
      n += __popc(m);
      __syncwarp();
    }
    uint32_t m = __ballot_sync(0xffffffffu, in_question);
    if (in_question) key[n + __popc(m & lanemask_lt())] = id;
    n += __popc(m);
    m = __ballot_sync(0xffffffffu, lane < p.k && !in_question);
    if (lane < p.k && !in_question) {
      const int i = n + __popc(m & lanemask_lt());
      key[i] = id, exact[i] = by == by ? by : -INFINITY;
    }
    const int listed = n + __popc(m);
    __syncwarp();
    if (__all_sync(0xffffffffu, zero)) {  // are they all because x is?
      for (int j = lane * 8; j < p.dim; j += 256) {
        float a[8];
        load8(x + j, a);
#pragma unroll
        for (int i = 0; i < 8; ++i) zero &= a[i] == 0.f;
      }
    }
    zero = __all_sync(0xffffffffu, zero);
    for (int i = 0; i < n; i += 2) {
      const int j = min(i + 1, n - 1);
      const double2 d = zero ? make_double2(0., 0.) : exact_products(w + (long long)key[i] * p.dim, w + (long long)key[j] * p.dim, x, p.dim, lane);
      // a product beyond fp32 has no remainders to add up
      const float first_i = product[key[i]].x, first_j = product[key[j]].x;
      if (lane == 0) exact[i] = d.x == d.x ? d.x : first_i, exact[j] = j == i ? exact[i] : d.y == d.y ? d.y : first_j;
    }
    __syncwarp();
    double sum64 = 1.;
    if (by_share) {
      sum64 = 0.;
      for (int e = lane; e < p.experts; e += 32) sum64 += exp((double)product[e].x - top);
      sum64 = warp_sum64(sum64);
    }
    for (int i = lane; i < n; i += 32) {
      const double s = p.bias == nullptr ? exact[i] : score_of64(p.score, exact[i], top) / sum64 + (double)p.bias[key[i]];
      exact[i] = s == s ? s : -INFINITY;
    }
    __syncwarp();
    float all = 0.f;  // the scores of the first k
    for (int turn = 0; turn < 2; ++turn) {
      for (int i = lane; i < listed; i += 32) {
        const double mine = exact[i];
        const int e = (int)key[i];
        int before = 0;
        for (int j = 0; j < listed; ++j) before += exact[j] > mine || (exact[j] == mine && (int)key[j] < e);
        if (before >= p.k) continue;
        const float s = score_of(p.score, product[e].x, top) / sum;
        if (turn == 0) all += s;
        else p.ids[to + before] = e, p.weights[to + before] = (p.normalize ? s / all : s) * p.scale;
      }
      if (turn == 0) all = warp_sum(all);
    }
    return;
  }
  const float z = lane < p.k ? product[id].x : 0.f;
  float s = lane < p.k ? score_of(p.score, z, top) / sum : 0.f;
  if (p.normalize) s /= warp_sum(s);
  if (lane < p.k) {
    p.ids[to + lane] = id;
    p.weights[to + lane] = s * p.scale;
  }
}

// Whether the block ends last of those of its tokens; what the others wrote is then there.
__device__ __forceinline__ bool ends_last(const RouteParams& p, int blocks, int of) {
  __shared__ int last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();  // the block's, of which the barrier has told this thread
    last = atomicAdd(p.done + of, 1) == blocks - 1;
    if (last) p.done[of] = 0;
    __threadfence();
  }
  __syncthreads();
  return last;
}

// A row of W per warp, with up to TB tokens.
template <typename TX, typename TW, int TB>
__global__ void __launch_bounds__(kWarps * 32) route_rows_kernel(const RouteParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * kWarps + warp, t0 = blockIdx.y * TB, nt = min(TB, p.tokens - t0);
  prior_done();
  next_may_start();  // not before: what starts then may read at once what came before this kernel
  if (e < p.experts) {
    const TX* x = static_cast<const TX*>(p.x) + (long long)t0 * p.x_row;
    const TW* w = static_cast<const TW*>(p.w) + (long long)e * p.dim;
    float acc[TB] = {}, off[TB] = {};  // each sum is rounded by up to 2^-24 of itself
#pragma unroll(TB == 1 ? 8 : 2)
    for (int d = lane * 8; d < p.dim; d += 256) {
      float a[8], b[8];
      load8(w + d, a);
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        load8(x + min(t, nt - 1) * p.x_row + d, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[t] = fmaf(a[j], b[j], acc[t]), off[t] += fabsf(acc[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      const float z = warp_sum(acc[t]), sizes = warp_sum(off[t] + 5.f * fabsf(acc[t]));  // five more additions of those
      if (lane == 0 && t < nt) p.z[(long long)(t0 + t) * p.experts + e] = told(p, e, z, 6.0e-8f * sizes);  // 2^-24 and some
    }
  }
  static_assert(TB <= kWarps, "a warp per token");
  if (ends_last(p, gridDim.x, blockIdx.y) && warp < nt) choose<TX, TW>(p, smem + warp * choice_bytes(p.experts), lane, t0 + warp);
}

__device__ __forceinline__ uint4 unsigned_pairs(const uint4& v) {
  return make_uint4(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu);
}

// Eight tokens with 16 experts on the tensor cores, the block's warps sharing the columns.  A lane's 16 bytes of a row
// are what two instructions take of it: their columns are in another order, in that of both operands.  Each instruction
// begins at zero (its sum is added as fp32), so that it cuts off its 16 products to a whole step of the largest, 16 times
// 2^-23 of the sum of their sizes at most, which the same products with signs taken off give.  (Two that share an
// accumulator cut off 33, and twice as many scores are near: 32 tokens of 4,096 values and
// 384 experts 26 us instead of 19.)
template <typename T>
__global__ void __launch_bounds__(kTileWarps * 32) route_tiles_kernel(const RouteParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 part[kTileWarps][16][9];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * kRouteTokens, nt = min(kRouteTokens, p.tokens - t0);
  prior_done();
  next_may_start();  // not before: what starts then may read at once what came before this kernel
  auto row = [&](const void* base, long long r, long long stride) { return static_cast<const T*>(base) + r * stride + t * 8; };
  const T* a_lo = row(p.w, min(e0 + g, p.experts - 1), p.dim);
  const T* a_hi = row(p.w, min(e0 + g + 8, p.experts - 1), p.dim);
  const T* b_at = row(p.x, t0 + min(g, nt - 1), p.x_row);
  float acc[4] = {}, sums[4] = {}, sizes[2][4] = {};
#pragma unroll 4
  for (int d = warp * 64; d < p.dim; d += kTileWarps * 64) {
#pragma unroll
    for (int h = 0; h < 64; h += 32) {
      const bool in = d + h + t * 8 < p.dim;
      const uint4 none = make_uint4(0, 0, 0, 0);
      const uint4 a = in ? *reinterpret_cast<const uint4*>(a_lo + d + h) : none;
      const uint4 b = in ? *reinterpret_cast<const uint4*>(a_hi + d + h) : none;
      const uint4 x = in ? *reinterpret_cast<const uint4*>(b_at + d + h) : none;
      auto products = [&](float (&to)[2][4], const uint4& a, const uint4& b, const uint4& x) {
        if constexpr (std::is_same<T, __half>::value) {
          mma_f16(to[0], a.x, b.x, a.y, b.y, x.x, x.y);
          mma_f16(to[1], a.z, b.z, a.w, b.w, x.z, x.w);
        } else {
          mma_bf16(to[0], a.x, b.x, a.y, b.y, x.x, x.y);
          mma_bf16(to[1], a.z, b.z, a.w, b.w, x.z, x.w);
        }
      };
      float c[2][4] = {};
      products(c, a, b, x);
      products(sizes, unsigned_pairs(a), unsigned_pairs(b), unsigned_pairs(x));
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += c[j][i], sums[i] += fabsf(acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)  // additions of the warps' sums; 1.2e-7: 2^-23 and some
    part[warp][g + (i >> 1) * 8][2 * t + (i & 1)] =
        make_float2(acc[i], 1.2e-7f * (16.f * (sizes[0][i] + sizes[1][i]) + 0.5f * sums[i] + 0.5f * kTileWarps * fabsf(acc[i])));
  __syncthreads();
  if (threadIdx.x < 16 * kRouteTokens) {
    const int e = threadIdx.x % 16, k = threadIdx.x / 16;
    float z = 0.f, off = 0.f;
#pragma unroll
    for (int w = 0; w < kTileWarps; ++w) z += part[w][e][k].x, off += part[w][e][k].y;
    if (k < nt && e0 + e < p.experts) p.z[(long long)(t0 + k) * p.experts + e0 + e] = told(p, e0 + e, z, off);
  }
  static_assert(kRouteTokens <= kTileWarps, "a warp per token");
  if (ends_last(p, gridDim.x, blockIdx.y) && warp < nt) choose<T, T>(p, smem + warp * choice_bytes(p.experts), lane, t0 + warp);
}

// Up to four tokens: a row of W per warp and token (they end together, and W comes from L2 for the second token on), for
// tensor cores' types while that is no more than two thirds of a block per SM (4,096 values: 4 tokens of 64 experts 6.1 us,
// as tiles 7.0; 3 of 384 10.9 and 9.2 to 10.4, 2 of 384 8.3 to 9.4 both).  More: tiles of 16 experts and 8 tokens, or with fp32 weights, which
// tensor cores would round, rows with 8 tokens.
template <typename TX, typename TW>
cudaError_t launch(const RouteParams& p, cudaStream_t stream) {
  const int groups = (p.tokens + kRouteTokens - 1) / kRouteTokens, rows = (p.experts + kWarps - 1) / kWarps;
  constexpr bool kTiles = std::is_same<TX, TW>::value && sizeof(TX) == 2;
  if (p.tokens == 1 || (p.tokens <= 4 && (!kTiles || p.tokens * rows * 3 <= device_sm_count() * 2)))
    return launch_behind(route_rows_kernel<TX, TW, 1>, dim3(rows, p.tokens), kWarps * 32, choice_bytes(p.experts), stream, p);
  const int smem = (p.tokens < kRouteTokens ? p.tokens : kRouteTokens) * choice_bytes(p.experts);
  constexpr int kMostSmem = kRouteTokens * choice_bytes(kRouteMostExperts);
  if constexpr (kTiles) {
    const cudaError_t e = allow_smem<route_tiles_kernel<TX>>(kMostSmem);
    if (e != cudaSuccess) return e;
    return launch_behind(route_tiles_kernel<TX>, dim3((p.experts + 15) / 16, groups), kTileWarps * 32, smem, stream, p);
  } else {
    const cudaError_t e = allow_smem<route_rows_kernel<TX, TW, kRouteTokens>>(kMostSmem);
    if (e != cudaSuccess) return e;
    return launch_behind(route_rows_kernel<TX, TW, kRouteTokens>, dim3(rows, groups), kWarps * 32, smem, stream, p);
  }
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, int x_dtype, int w_dtype, cudaStream_t stream) {
  if (x_dtype == CSA2_T_BF16)
    return w_dtype == CSA2_T_F32 ? launch<__nv_bfloat16, float>(p, stream) : launch<__nv_bfloat16, __nv_bfloat16>(p, stream);
  if (x_dtype == CSA2_T_F16) return w_dtype == CSA2_T_F32 ? launch<__half, float>(p, stream) : launch<__half, __half>(p, stream);
  return launch<float, float>(p, stream);
}

}  // namespace csa2
