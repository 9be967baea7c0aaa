// Root-mean-square norm of rows with the residual's addition before it and an 8-bit output after it.
//
//   s = x + r;  y = s (mean s^2 + eps)^(-1/2) (g + offset);  codes = E4M3(y / (max|y| / 448))
//
// Bound by the bytes: x and r in, s and y (or its codes) out, each once.  A block takes a row and holds it in
// registers between the sum of squares, the maximum and the outputs, so that nothing is read twice; one block
// reduction stands between: y = (s (g + offset)) (..)^(-1/2), whose largest is the largest s (g + offset) times that root.
// All loads of a row set out before the first is used, and where rows are many a block's next row's set out before the
// present one is summed: 16,384 rows of 5,120 in bf16 with residual and codes, 587 MB, 92 us or 6.4 TB/s (a row per block
// and no more: 106 us).  32 rows of 4,096 take 2.8 us, a launch and a memory latency.
#include "common.cuh"
#include "paged_dev.cuh"
#include "step.h"

namespace csa2 {

int device_sm_count();

namespace {

enum { kNoSum = 0, kSameSum = 1, kF32Sum = 2 };

// VEC values of a row: 16-byte pieces of it, or one value.
template <typename T, int VEC>
struct Piece {
  static constexpr int kWords = VEC * (int)sizeof(T) / 16;
  uint4 w[kWords > 0 ? kWords : 1];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC > 1) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    } else if constexpr (sizeof(T) == 4) {
      w[0].x = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0].x = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    if constexpr (sizeof(T) == 4) return __uint_as_float(u[i]);
    const uint32_t v = i & 1 ? u[i / 2] >> 16 : u[i / 2] & 0xffffu;
    if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half((unsigned short)v));
    return __uint_as_float(v << 16);
  }
};
template <typename T>
__device__ __forceinline__ uint32_t bits16(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) return pack_f16x2(a, b);
  return pack_bf16x2(a, b);
}
template <typename T>
__device__ __forceinline__ float rounded(float v) {
  if constexpr (sizeof(T) == 4) return v;
  if constexpr (std::is_same<T, __half>::value) return __half2float(__float2half_rn(v));
  return __bfloat162float(__float2bfloat16_rn(v));
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T* p, const float* v) {
  if constexpr (VEC == 1) {
    if constexpr (sizeof(T) == 4) *reinterpret_cast<float*>(p) = v[0];
    else *reinterpret_cast<uint16_t*>(p) = (uint16_t)bits16<T>(v[0], 0.f);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 8)
      *reinterpret_cast<uint4*>(p + i) = make_uint4(bits16<T>(v[i], v[i + 1]), bits16<T>(v[i + 2], v[i + 3]),
                                                    bits16<T>(v[i + 4], v[i + 5]), bits16<T>(v[i + 6], v[i + 7]));
  }
}

// Two sums of 16-bit values, each rounded once.  (As fp32 and back they are the same: a sum that 24 bits do not hold is of
// values so far apart that the smaller one is no half step of the larger.)
template <typename T>
__device__ __forceinline__ uint32_t add_pairs(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (std::is_same<T, __half>::value) asm("add.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  else asm("add.rn.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The largest size of three values, NaN where one is.
__device__ __forceinline__ float largest(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int VEC>
__device__ __forceinline__ void load_gain(const AddNormParams& p, int at, float* g) {
  if (p.gain == nullptr) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) g[i] = 1.f;
  } else if (p.gain_dtype == CSA2_T_F32) {
    Piece<float, VEC> v;
    v.load(static_cast<const float*>(p.gain) + at);
#pragma unroll
    for (int i = 0; i < VEC; ++i) g[i] = v.get(i);
  } else if (p.gain_dtype == CSA2_T_F16) {
    Piece<__half, VEC> v;
    v.load(static_cast<const __half*>(p.gain) + at);
#pragma unroll
    for (int i = 0; i < VEC; ++i) g[i] = v.get(i);
  } else {
    Piece<__nv_bfloat16, VEC> v;
    v.load(static_cast<const __nv_bfloat16*>(p.gain) + at);
#pragma unroll
    for (int i = 0; i < VEC; ++i) g[i] = v.get(i);
  }
}

// v / scale as the division rounds it, for a scale whose reciprocal is an fp32 number: the quotient by the reciprocal, put
// right by what it leaves (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000", 1990).
__device__ __forceinline__ float over(float v, float scale, float inverse) {
  const float q = v * inverse;
  return fmaf(fmaf(-q, scale, v), inverse, q);
}

// The scale of values up to max |y| (a product's rounding keeps the order, so that this is the root times the largest
// s (g + offset)).
struct Scale {
  float scale, inverse;
  bool none;   // codes are 0: the peak is not finite, or so small that its 448th part is no fp32 value any more
  bool small;  // it may have no reciprocal
};
__device__ __forceinline__ Scale scale_of(float peak) {
  Scale f;
  const bool finite = peak < INFINITY;
  const float part = peak > 1e-30f ? over(peak, 448.f, 1.f / 448.f) : peak / 448.f;
  f.scale = finite ? peak > 0.f ? part : 1.f : __uint_as_float(0x7fc00000u);
  f.none = !finite || f.scale == 0.f, f.small = f.scale < 1e-36f;
  f.inverse = __frcp_rn(f.scale);
  return f;
}

// Rows blockIdx.x, + gridDim.x ..; thread t has pieces t, t + threads, ... of VEC values each.
template <typename T, int SUM, int VEC, int PER>
__global__ void __launch_bounds__(1024) add_norm_kernel(const AddNormParams p) {
  using R = typename std::conditional<SUM == kF32Sum, float, T>::type;
  extern __shared__ uint32_t peaks[];  // single values with groups: the largest |y| of each as bits
  __shared__ float part[2][32];        // by turns, so that a row's sums are read before they are written again
  __shared__ uint32_t part_top[2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, warps = nt >> 5;
  const int pieces = p.dim / VEC;
  Piece<T, VEC> in[PER];
  Piece<R, VEC> res[SUM ? PER : 1];
  auto load = [&](long long row) {
    const T* x = static_cast<const T*>(p.x) + row * p.x_row;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int c = tid + j * nt;
      if (c < pieces) in[j].load(x + (long long)c * VEC);
    }
    if constexpr (SUM != kNoSum) {
      const R* r = static_cast<const R*>(p.residual) + row * p.residual_row;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int c = tid + j * nt;
        if (c < pieces) res[j].load(r + (long long)c * VEC);
      }
    }
  };
  prior_done();
  load(blockIdx.x);
  int turn = 0;
  for (long long row = blockIdx.x; row < p.n_rows; row += gridDim.x, turn ^= 1) {
    if (VEC == 1 && p.group > 0) {
      for (int i = tid; i < p.dim / p.group; i += nt) peaks[i] = 0;
      __syncthreads();
    }
    // s, stored by the threads that have read what it may lie on; s (g + offset) with its squares' sum and largest values
    float v[PER][VEC], sq = 0.f;
    uint32_t top[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int c = tid + j * nt;
      top[j] = 0;
      if (c < pieces) {
        float g[VEC];
        load_gain<VEC>(p, c * VEC, g);
        R* sum_at = SUM != kNoSum ? static_cast<R*>(p.sum) + row * p.sum_row + (long long)c * VEC : nullptr;
        if constexpr (SUM == kSameSum && VEC > 1 && sizeof(T) == 2) {
          Piece<T, VEC> both;
          both.w[0] = make_uint4(add_pairs<T>(in[j].w[0].x, res[j].w[0].x), add_pairs<T>(in[j].w[0].y, res[j].w[0].y),
                                 add_pairs<T>(in[j].w[0].z, res[j].w[0].z), add_pairs<T>(in[j].w[0].w, res[j].w[0].w));
          *reinterpret_cast<uint4*>(sum_at) = both.w[0];
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[j][i] = both.get(i);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            v[j][i] = in[j].get(i);
            if constexpr (SUM != kNoSum) v[j][i] = rounded<R>(v[j][i] + res[j].get(i));
          }
          if constexpr (SUM != kNoSum) store<R, VEC>(sum_at, v[j]);
        }
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) sq += v[j][i] * v[j][i], v[j][i] *= g[i] + p.gain_offset;
        if constexpr (VEC == 1) m = largest(m, v[j][0], v[j][0]);
        else {
#pragma unroll
          for (int i = 0; i < VEC; i += 2) m = largest(m, v[j][i], v[j][i + 1]);
        }
        top[j] = __float_as_uint(m) & 0x7fffffffu;
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j][i] = 0.f;
      }
    }
    if (row + gridDim.x < p.n_rows) load(row + gridDim.x);
    // the largest of what shares a scale, as bits: a NaN's are above an infinity's, and those above the rest
    sq = warp_sum(sq);
    if (lane == 0) part[turn][warp] = sq;
    if (p.codes != nullptr) {
      if (p.group == 0) {
        uint32_t m = top[0];
#pragma unroll
        for (int j = 1; j < PER; ++j) m = max(m, top[j]);
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) part_top[turn][warp] = m;
      } else if constexpr (VEC > 1) {  // a group is some neighbouring lanes' pieces
#pragma unroll
        for (int j = 0; j < PER; ++j)
          for (int o = 1; o < p.group / VEC; o <<= 1) top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
      } else {
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (tid + j * nt < pieces) atomicMax(&peaks[(tid + j * nt) / p.group], top[j]);
      }
    }
    __syncthreads();
    const float total = warp_sum(lane < warps ? part[turn][lane] : 0.f);
    const float inv = 1.f / sqrtf(total / (float)p.dim + p.eps);
#pragma unroll
    for (int j = 0; j < PER; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j][i] *= inv;
    if (p.out != nullptr) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (tid + j * nt >= pieces) continue;
        const long long at = row * p.out_row + (long long)(tid + j * nt) * VEC;
        if (p.out_dtype == CSA2_T_F32) store<float, VEC>(static_cast<float*>(p.out) + at, v[j]);
        else if (p.out_dtype == CSA2_T_F16) store<__half, VEC>(static_cast<__half*>(p.out) + at, v[j]);
        else store<__nv_bfloat16, VEC>(static_cast<__nv_bfloat16*>(p.out) + at, v[j]);
      }
    }
    if (p.codes == nullptr) continue;
    Scale of_row{};
    if (p.group == 0) {
      of_row = scale_of(__uint_as_float(__reduce_max_sync(0xffffffffu, lane < warps ? part_top[turn][lane] : 0)) * inv);
      if (tid == 0) p.scales[row] = of_row.scale;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int c = tid + j * nt;
      if (c >= pieces) continue;
      Scale f = of_row;
      if (p.group > 0) {
        f = scale_of(__uint_as_float(VEC > 1 ? top[j] : peaks[c * VEC / p.group]) * inv);
        if (c * VEC % p.group == 0) p.scales[row * (p.dim / p.group) + c * VEC / p.group] = f.scale;
      }
      uint8_t* at = p.codes + row * p.dim + (long long)c * VEC;
      float q[VEC];
      if (!f.small) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) q[i] = over(v[j][i], f.scale, f.inverse);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) q[i] = v[j][i] / f.scale;
      }
      if constexpr (VEC == 1) {
        *at = f.none ? 0 : (uint8_t)e4m3_word(q[0], 0.f, 0.f, 0.f);
      } else {
        uint2 w = make_uint2(e4m3_word(q[0], q[1], q[2], q[3]), e4m3_word(q[4], q[5], q[6], q[7]));
        if (f.none) w = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(at) = w;
      }
    }
    if (VEC == 1 && p.group > 0) __syncthreads();  // the peaks have been read
  }
}

template <typename T, int SUM>
cudaError_t launch(const AddNormParams& p, bool vectors, cudaStream_t stream) {
  // Threads for one piece each where rows are few (their latency is all there is), two where they are many: the fewer
  // warps a barrier joins, the less of a row's time it is (16,384 rows of 5,120, bf16 to codes: 164 us with one piece, 92
  // with two, 147 with four, which leave room for fewer warps).
  const int pieces = vectors ? p.dim / 8 : p.dim;
  const int want = p.n_rows <= 2 * device_sm_count() ? 1 : 2;
  int nt = ((pieces + want - 1) / want + 31) / 32 * 32;
  if (nt > 1024) nt = 1024;
  const int per = (pieces + nt - 1) / nt;
  // a row each, or as many blocks as an SM has threads for.  (Some half of those are there at once: 61 to 64 registers, to
  // which a block of 1,024 threads binds all, leave room for 1,024 threads.)
  const int most = device_sm_count() * (2048 / nt);
  const dim3 grid((unsigned)(p.n_rows < most ? p.n_rows : most));
  if (vectors) {
    if (per <= 2) return launch_behind(add_norm_kernel<T, SUM, 8, 2>, grid, nt, 0, stream, p);
    return launch_behind(add_norm_kernel<T, SUM, 8, 4>, grid, nt, 0, stream, p);
  }
  const size_t smem = p.codes != nullptr && p.group > 0 ? p.dim / p.group * sizeof(uint32_t) : 0;
  if (per <= 2) return launch_behind(add_norm_kernel<T, SUM, 1, 2>, grid, nt, smem, stream, p);
  return launch_behind(add_norm_kernel<T, SUM, 1, 8>, grid, nt, smem, stream, p);
}
template <typename T>
cudaError_t launch_sum(const AddNormParams& p, bool f32_sum, bool none, bool vectors, cudaStream_t stream) {
  if (none) return launch<T, kNoSum>(p, vectors, stream);
  if constexpr (sizeof(T) == 2)
    if (f32_sum) return launch<T, kF32Sum>(p, vectors, stream);
  return launch<T, kSameSum>(p, vectors, stream);
}

}  // namespace

cudaError_t launch_add_norm(const AddNormParams& p, int x_dtype, int sum_dtype, bool vectors, cudaStream_t stream) {
  const bool none = sum_dtype < 0, f32 = sum_dtype == CSA2_T_F32;
  if (x_dtype == CSA2_T_BF16) return launch_sum<__nv_bfloat16>(p, f32, none, vectors, stream);
  if (x_dtype == CSA2_T_F16) return launch_sum<__half>(p, f32, none, vectors, stream);
  return launch_sum<float>(p, f32, none, vectors, stream);
}

}  // namespace csa2
