// Attention over a paged cache of E4M3 codes with one scale per (page, head), few query rows per
// key-value head: split over the cached tokens and joined.
//
//   z_ij = softmax_scale * q_i . k_j,  k_j = code * k_scale[page, head];  j <= pos_i, j > pos_i - window
//   o_i  = sum_j exp(z_ij) v_j / (sum_j exp(z_ij) + exp(sink))
//
// Bound by the codes' way from memory: 2 * dim bytes per cached token and head, each read once.
//
// Split.  A tile is up to 8 or 16 query rows (tokens x heads of the group) of one sequence and kv head;
// its unit of work is 128 cached tokens.  The units of all tiles of the call form one line, of which
// every block takes an equal piece, so that ragged lengths, one long sequence or many short ones load
// the SMs alike and the host needs no lengths.  A block finds its place by summing the sequences'
// units itself.  A tile that ends inside a block is written out by it; an open one leaves partial
// sums, and a second kernel joins the pieces in order.
//
// Within a block each of the four warps streams its own 32 tokens of a unit through a ring in shared
// memory (cp.async, two stages of K and of V; no block barrier until the tile's end) and keeps its own
// running maximum, sum and output.
//
// Arithmetic.  K stays in its 8 bits: a query row, scaled by a power of two, is split into E4M3 pieces
// (two hold a bf16's 8 bits, three an fp16's 11, below 2^-9 of a row maximum in [224, 448]), and the
// scores are the sum of the pieces' E4M3 products in fp32: mma.m16n8k32 runs at twice the rate per
// instruction of the fp16 form with twice its depth, and no conversion is needed.  V is converted to
// fp16 (exact), weights are fp16 of exp2(z - max + 15), at most 2^15, so that weights down to 2^-29
// of the largest keep 11 bits.  A page's V scale enters the weight relative to the largest seen.
// Maxima, sums and outputs are fp32.
#include "common.cuh"
#include "paged.h"

namespace csa2 {
namespace {

constexpr int kWarps = 4;
constexpr int kTok = 32;                // tokens of a warp's step
constexpr int kUnit = kWarps * kTok;    // tokens of a unit
constexpr float kLift = 15.f;           // weights are held times 2^15
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_e4m3(float* c, const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four values of an output row: sums o relative to maximum M (log2 units) over the row's denominator.
// A row that saw no key is 0.
template <int D>
__device__ __forceinline__ void store_row(const PagedAttnParams& p, int row, int head, int d, float4 o, float M, float L) {
  float den = L;
  if (p.sink != nullptr && M > -INFINITY) den += ex2(p.sink[head] * kLog2e - M + kLift);
  const float inv = L == 0.f ? 0.f : __fdividef(1.f, den);
  const long long at = ((long long)row * (p.kv_heads * p.group) + head) * D + d;
  o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
  if (p.out_dtype == CSA2_T_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = o;
  } else {
    const bool h = p.out_dtype == CSA2_T_F16;
    const uint2 u = h ? make_uint2(pack_f16x2(o.x, o.y), pack_f16x2(o.z, o.w)) : make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = u;
  }
}

// The rows and units of one sequence.
struct Seq {
  int first, rows;     // its first query row; query rows x heads of a group
  int ctx, kv;         // position of its first query row; cached tokens
  int lo, blocks;      // first token any row sees (down to a multiple of 16); units of a tile
  int tiles;           // tiles of a kv head
  long long units;
};
template <int NR>
__device__ __forceinline__ Seq seq_of(const PagedAttnParams& p, int b) {
  Seq s;
  const int r0 = p.row_start[b], r1 = p.row_start[b + 1];
  s.first = min(max(r0, 0), p.n_rows);
  const int n = max(min(r1, p.n_rows) - s.first, 0);
  const long long cap = (long long)p.table_cols << p.page_shift;
  const int kv = max(p.kv_len[b], 0);
  s.ctx = kv - (r1 - r0);
  s.kv = (int)min((long long)kv, cap);
  s.rows = n * p.group;
  s.lo = p.window > 0 ? max(s.ctx - p.window + 1, 0) & ~15 : 0;
  s.blocks = max((max(s.kv - s.lo, 0) + kUnit - 1) / kUnit, 1);
  s.tiles = (s.rows + NR - 1) / NR;
  s.units = (long long)s.tiles * p.kv_heads * s.blocks;
  return s;
}

template <int D>
__device__ __forceinline__ int phys(int row, int chunk) {  // byte offset of a 16-byte chunk in a stage
  // D = 128: chunk ^ row, so that the 8 lanes of a phase (two rows of K, four of V) meet 8 banks groups
  return D == 128 ? row * 128 + ((chunk ^ (row & 7)) << 4) : row * 64 + (chunk << 4);
}

template <int D, int NR, int PIECES, bool F16>
__global__ void __launch_bounds__(kWarps * 32, 3) paged_attn_kernel(const PagedAttnParams p) {
  constexpr int KS = D / 32;            // MMA steps of a score
  constexpr int NT = D / 8;             // MMA columns of an output
  constexpr int kStage = kTok * D;      // bytes of K (or V) of a step
  constexpr bool FULL = NR == 16;       // rows 8 .. 15 in use
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float scales[kWarps][2][4];
  __shared__ float ml[kWarps][16][3];
  __shared__ long long scan_warp[kWarps];
  __shared__ long long place[2];        // sequence, its first unit
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;

  // ---- this block's piece of the line of units
  long long u, u_end;
  int b;
  long long b_first;
  {
    const int run = (p.n_seq + kWarps * 32 - 1) / (kWarps * 32);
    const int q0 = min(tid * run, p.n_seq), q1 = min(q0 + run, p.n_seq);
    long long mine = 0;
    for (int i = q0; i < q1; ++i) mine += seq_of<NR>(p, i).units;
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scan_warp[warp] = x;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += scan_warp[w];
      total += scan_warp[w];
    }
    before += x - mine;
    u = total * blockIdx.x / gridDim.x;
    u_end = total * (blockIdx.x + 1) / gridDim.x;
    if (blockIdx.x == 0 && tid == 0) p.units[0] = total;
    if (u < u_end && before <= u && u < before + mine) {
      long long at = before;
      int i = q0;
      for (;; ++i) {
        const long long n = seq_of<NR>(p, i).units;
        if (u < at + n) break;
        at += n;
      }
      place[0] = i;
      place[1] = at;
    }
    __syncthreads();
    if (u >= u_end) {
      if (tid == 0) p.open[blockIdx.x].end = -1;
      return;
    }
    b = (int)place[0];
    b_first = place[1];
  }
  uint8_t* ring = smem + warp * 4 * kStage;  // K0 K1 V0 V1
  long long open_end = -1;
  bool bad = false;

  while (u < u_end) {
    const Seq s = seq_of<NR>(p, b);
    if (s.units == 0) {
      ++b;
      continue;
    }
    const long long in_seq = u - b_first;
    const long long item = in_seq / s.blocks;
    const int blk0 = (int)(in_seq - item * s.blocks);
    const int head = (int)(item / s.tiles), tile = (int)(item - (long long)head * s.tiles);
    const int seg = (int)min((long long)(s.blocks - blk0), u_end - u);
    const int row0 = tile * NR, n = min(NR, s.rows - row0);
    const int pos_last = s.ctx + (row0 + n - 1) / p.group;
    const int t_begin = s.lo + blk0 * kUnit;
    const int t_end = min(min(t_begin + seg * kUnit, s.kv), pos_last + 1);
    // the two rows of this thread: their positions and their first token
    const int ra = min(g, n - 1), rb = min(g + 8, n - 1);
    const int pos_a = s.ctx + (row0 + ra) / p.group, pos_b = s.ctx + (row0 + rb) / p.group;
    const int pos_first = s.ctx + row0 / p.group;
    const int lo_a = p.window > 0 ? pos_a - p.window + 1 : 0, lo_b = p.window > 0 ? pos_b - p.window + 1 : 0;
    const int lo_last = p.window > 0 ? pos_last - p.window + 1 : 0;

    // ---- loads: page ids one step ahead of the copies, copies one step ahead of their use
    const int32_t* trow = p.table + (long long)b * p.table_cols;
    auto page_id = [&](int tok) -> int {  // -1: no such token, -2: a bad entry
      if (tok >= t_end) return -1;
      const int id = __ldg(trow + (tok >> p.page_shift));
      return (unsigned)id < (unsigned)p.n_pages ? id : -2;
    };
    const int page_mask = (1 << p.page_shift) - 1;
    auto copy = [&](const uint8_t* codes, uint8_t* to, int tok, int id0, int id1) {
      const long long o0 = id0 < 0 ? 0 : ((((long long)id0 * p.kv_heads + head) << p.page_shift) + (tok & page_mask)) * D;
      const long long o1 = id1 < 0 ? 0 : ((((long long)id1 * p.kv_heads + head) << p.page_shift) + ((tok + 16) & page_mask)) * D;
#pragma unroll
      for (int i = 0; i < kStage / 512; ++i) {
        const int chunk = i * 32 + lane, row = chunk / (D / 16), ch = chunk % (D / 16);
        const bool second = i >= kStage / 1024;
        const bool ok = (second ? id1 : id0) >= 0 && tok + row < t_end;
        cp_async16(to + phys<D>(row, ch), codes + (second ? o1 : o0) + (ok ? (row & 15) * D + ch * 16 : 0), ok);
      }
    };
    auto copy_k = [&](int slot, int tok, int id0, int id1) {
      if (tok < t_end) {
        copy(p.k, ring + slot * kStage, tok, id0, id1);
        if (lane < 4) {
          const int id = lane & 1 ? id1 : id0;
          const float* sc = lane < 2 ? p.k_scale : p.v_scale;
          cp_async4(&scales[warp][slot][lane], sc + (id < 0 ? 0 : (long long)id * p.kv_heads + head), id >= 0);
        }
      }
      cp_async_commit();
    };
    auto copy_v = [&](int slot, int tok, int id0, int id1) {
      if (tok < t_end) copy(p.v, ring + (2 + slot) * kStage, tok, id0, id1);
      cp_async_commit();
    };
    int tok = t_begin + warp * kTok;
    int ida0 = page_id(tok), ida1 = page_id(tok + 16);
    int idb0 = page_id(tok + kUnit), idb1 = page_id(tok + kUnit + 16);
    copy_k(0, tok, ida0, ida1);
    copy_v(0, tok, ida0, ida1);
    copy_k(1, tok + kUnit, idb0, idb1);
    copy_v(1, tok + kUnit, idb0, idb1);

    // ---- the query rows as E4M3 pieces: this thread's dims are D/4 * c .. of rows g and g + 8
    uint32_t qa[PIECES][KS][4];
    float f_a, f_b;  // score in log2 units = f * sum of products * k_scale
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float x[D / 4];
      const int r = g + 8 * half;
      const bool has = r < n && (FULL || half == 0);
      float amax = 0.f;
      bool odd = false;
      if (has) {
        const int rr = row0 + r, i = rr / p.group;
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + (long long)(s.first + i) * p.q_row +
                              (long long)(head * p.group + rr - i * p.group) * p.q_head + D / 4 * c;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const uint4 w4 = *reinterpret_cast<const uint4*>(src + 8 * k);
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float2 v;
            if (F16) v = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            else v = make_float2(bf16_lo(w[j]), bf16_hi(w[j]));
            x[8 * k + 2 * j] = v.x, x[8 * k + 2 * j + 1] = v.y;
            odd |= !(fabsf(v.x) < INFINITY) || !(fabsf(v.y) < INFINITY);
            amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < D / 4; ++k) x[k] = 0.f;
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      odd = odd || __shfl_xor_sync(0xffffffffu, (int)odd, 1);
      odd = odd || __shfl_xor_sync(0xffffffffu, (int)odd, 2);
      // 2^e with amax / 2^e in [224, 448): e = exponent of amax - 8 (1.75 * 2^8 = 448), or one more
      const uint32_t ua = __float_as_uint(amax);
      int e = (int)(ua >> 23) - 127 - 8 + ((ua & 0x7fffffu) >= 0x600000u ? 1 : 0);
      e = min(max(e, -110), 119);
      const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
      (half ? f_b : f_a) = odd ? __uint_as_float(0x7fc00000u) : p.scale_log2 * up;  // a NaN or infinity: the row is NaN
#pragma unroll
      for (int k = 0; k < D / 4; ++k) x[k] = odd ? 0.f : x[k] * down;
#pragma unroll
      for (int m = 0; m < PIECES; ++m)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int j = 0; j < 2; ++j) {  // words of 4 dims: j = 0 the MMA's k 4c .. , j = 1 its k 16 + 4c ..
            float* y = x + 8 * ks + 4 * j;
            const uint32_t w0 = e4m3_pair(y[0], y[1]), w1 = e4m3_pair(y[2], y[3]);
            qa[m][ks][2 * j + half] = w0 | w1 << 16;
            if (m + 1 < PIECES) {
              const uint32_t h0 = e4m3x2_to_f16x2((uint16_t)w0), h1 = e4m3x2_to_f16x2((uint16_t)w1);
              const float2 v0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
              const float2 v1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
              y[0] -= v0.x, y[1] -= v0.y, y[2] -= v1.x, y[3] -= v1.y;  // exact
            }
          }
    }

    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f, vref = 0.f, vinv = 0.f;

    for (int slot = 0; tok < t_end; tok += kUnit, slot ^= 1) {
      const int idc0 = page_id(tok + 2 * kUnit), idc1 = page_id(tok + 2 * kUnit + 16);
      bad |= ida0 == -2 || ida1 == -2;
      cp_async_wait<3>();
      __syncwarp();
      // ---- scores of 32 tokens: S[4][4], token 8t + (column)
      float S[4][4];
      const uint8_t* kt = ring + slot * kStage;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        uint32_t w[2 * KS];
        const int row = 8 * t + g;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          const uint4 v = *reinterpret_cast<const uint4*>(kt + phys<D>(row, D / 64 * c + h));
          w[4 * h] = v.x, w[4 * h + 1] = v.y, w[4 * h + 2] = v.z, w[4 * h + 3] = v.w;
        }
        S[t][0] = S[t][1] = S[t][2] = S[t][3] = 0.f;
#pragma unroll
        for (int m = 0; m < PIECES; ++m)
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) mma_e4m3(S[t], qa[m][ks], w[2 * ks], w[2 * ks + 1]);
      }
      const float4 sc = *reinterpret_cast<const float4*>(scales[warp][slot]);  // k scales, v scales
      __syncwarp();
      copy_k(slot, tok + 2 * kUnit, idc0, idc1);

      // a NaN in either scale marks the page: its visible tokens give NaN
      const float k0 = sc.x + 0.f * sc.z, k1 = sc.y + 0.f * sc.w;
      const bool whole = tok + kTok - 1 <= min(pos_first, t_end - 1) && tok >= lo_last && ida0 >= 0 && ida1 >= 0;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float ks = t < 2 ? k0 : k1;
        S[t][0] *= f_a * ks, S[t][1] *= f_a * ks;
        if (FULL) S[t][2] *= f_b * ks, S[t][3] *= f_b * ks;
      }
      if (!whole) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int at = tok + 8 * t + 2 * c + j;
            const bool there = (t < 2 ? ida0 : ida1) >= 0 && at < t_end;
            if (!(there && at <= pos_a && at >= lo_a)) S[t][j] = -INFINITY;
            if (FULL && !(there && at <= pos_b && at >= lo_b)) S[t][2 + j] = -INFINITY;
          }
      }
      float x_a = m_a, x_b = m_b;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        x_a = fmaxf(x_a, fmaxf(S[t][0], S[t][1]));
        if (FULL) x_b = fmaxf(x_b, fmaxf(S[t][2], S[t][3]));
      }
      x_a = fmaxf(x_a, __shfl_xor_sync(0xffffffffu, x_a, 1));
      x_a = fmaxf(x_a, __shfl_xor_sync(0xffffffffu, x_a, 2));
      if (FULL) {
        x_b = fmaxf(x_b, __shfl_xor_sync(0xffffffffu, x_b, 1));
        x_b = fmaxf(x_b, __shfl_xor_sync(0xffffffffu, x_b, 2));
      }
      float v0 = sc.z, v1 = sc.w;
      if (!(v0 > 0.f)) v0 = 0.f;
      if (!(v1 > 0.f)) v1 = 0.f;
      const float vnew = fmaxf(vref, fmaxf(v0, v1));
      if (__any_sync(0xffffffffu, x_a > m_a || (FULL && x_b > m_b) || vnew > vref)) {
        if (vnew > vref) vinv = __fdiv_rn(1.f, vnew);
        const float vf = vref * vinv;
        const float e_a = m_a == -INFINITY ? 0.f : ex2(m_a - x_a), e_b = FULL && m_b > -INFINITY ? ex2(m_b - x_b) : 0.f;
        l_a *= e_a, l_b *= e_b;
        const float o_a = e_a * vf, o_b = e_b * vf;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          acc[i][0] *= o_a, acc[i][1] *= o_a;
          if (FULL) acc[i][2] *= o_b, acc[i][3] *= o_b;
        }
        m_a = x_a, m_b = x_b, vref = vnew;
      }
      const float c0 = v0 * vinv, c1 = v1 * vinv;
      const float s_a = m_a == -INFINITY ? 0.f : kLift - m_a, s_b = m_b == -INFINITY ? 0.f : kLift - m_b;
      uint32_t pw[4][2];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float cv = t < 2 ? c0 : c1;
        const float p0 = ex2(S[t][0] + s_a), p1 = ex2(S[t][1] + s_a);
        l_a += p0 + p1;
        pw[t][0] = pack_f16x2(p0 * cv, p1 * cv);
        if (FULL) {
          const float p2 = ex2(S[t][2] + s_b), p3 = ex2(S[t][3] + s_b);
          l_b += p2 + p3;
          pw[t][1] = pack_f16x2(p2 * cv, p3 * cv);
        } else {
          pw[t][1] = 0u;
        }
      }
      // ---- outputs: two steps of 16 tokens; this thread's tokens 2c, 2c + 1, 2c + 8, 2c + 9, dims D/8 * g ..
      cp_async_wait<3>();
      __syncwarp();
      const uint8_t* vt = ring + (2 + slot) * kStage;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        constexpr int W = D / 32;  // words of D/8 dims
        uint32_t w[4][W];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = 16 * h + 2 * c + (j & 1) + 8 * (j >> 1);
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(vt + phys<D>(row, g));
            w[j][0] = v.x, w[j][1] = v.y, w[j][2] = v.z, w[j][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(vt + row * 64 + 8 * g);
            w[j][0] = v.x, w[j][1] = v.y;
          }
        }
#pragma unroll
        for (int k = 0; k < W; ++k) {
          const uint32_t lo0 = __byte_perm(w[0][k], w[1][k], 0x5140), hi0 = __byte_perm(w[0][k], w[1][k], 0x7362);
          const uint32_t lo1 = __byte_perm(w[2][k], w[3][k], 0x5140), hi1 = __byte_perm(w[2][k], w[3][k], 0x7362);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t b0 = j < 2 ? lo0 : hi0, b1 = j < 2 ? lo1 : hi1;
            mma_f16(acc[4 * k + j], pw[2 * h][0], pw[2 * h][1], pw[2 * h + 1][0], pw[2 * h + 1][1],
                    e4m3x2_to_f16x2((uint16_t)(j & 1 ? b0 >> 16 : b0 & 0xffffu)),
                    e4m3x2_to_f16x2((uint16_t)(j & 1 ? b1 >> 16 : b1 & 0xffffu)));
          }
        }
      }
      __syncwarp();
      copy_v(slot, tok + 2 * kUnit, idc0, idc1);
      ida0 = idb0, ida1 = idb1, idb0 = idc0, idb1 = idc1;
    }
    cp_async_wait<0>();

    // ---- the four warps' sums joined
    l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
    l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
    if (FULL) {
      l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
      l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
    }
    __syncthreads();  // every warp has left its ring
    float* part = reinterpret_cast<float*>(smem);  // [warp][NR][D]
    {
      float* to = part + (warp * NR + g) * D + D / 4 * c;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < NT; i += 4) {
          *reinterpret_cast<float4*>(to + k * NT + i) = make_float4(acc[i][k], acc[i + 1][k], acc[i + 2][k], acc[i + 3][k]);
          if (FULL)
            *reinterpret_cast<float4*>(to + 8 * D + k * NT + i) =
                make_float4(acc[i][2 + k], acc[i + 1][2 + k], acc[i + 2][2 + k], acc[i + 3][2 + k]);
        }
      if (c == 0) {
        ml[warp][g][0] = m_a, ml[warp][g][1] = l_a, ml[warp][g][2] = vref;
        if (FULL) ml[warp][g + 8][0] = m_b, ml[warp][g + 8][1] = l_b, ml[warp][g + 8][2] = vref;
      }
    }
    __syncthreads();
    const bool starts = blk0 == 0, ends = blk0 + seg == s.blocks;
    const int slot_of = 2 * blockIdx.x + (starts ? 1 : 0);
    for (int i = tid; i < n * (D / 4); i += kWarps * 32) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w][r][0]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = ml[w][r][0];
        if (mw == -INFINITY && ml[w][r][1] == 0.f) continue;  // a warp that saw nothing (not one whose sum is NaN)
        const float e = mw == -INFINITY ? 1.f : ex2(mw - M), f = e * ml[w][r][2];
        const float4 a = *reinterpret_cast<const float4*>(part + (w * NR + r) * D + d);
        L += ml[w][r][1] * e;
        o.x += a.x * f, o.y += a.y * f, o.z += a.z * f, o.w += a.w * f;
      }
      if (starts && ends) {
        const int rr = row0 + r, tokn = rr / p.group, hq = head * p.group + rr - tokn * p.group;
        store_row<D>(p, s.first + tokn, hq, d, o, M, L);
      } else {
        *reinterpret_cast<float4*>(p.part_o + ((long long)slot_of * 16 + r) * D + d) = o;
        if (d == 0) *reinterpret_cast<float2*>(p.part_ml + ((long long)slot_of * 16 + r) * 2) = make_float2(M, L);
      }
    }
    if (starts && !ends && tid == 0) {
      PagedOpen& o = p.open[blockIdx.x];
      o.row0 = row0, o.n = n, o.first_row = s.first, o.kv_head = head;
    }
    open_end = starts && !ends ? u - blk0 + s.blocks : -1;
    __syncthreads();  // the sums are read before the ring is filled again
    u += seg;
    if (u == b_first + s.units) {
      b_first = u;
      ++b;
    }
  }
  if (tid == 0) p.open[blockIdx.x].end = open_end;
  if (bad && p.dev_status && lane == 0) atomicExch(p.dev_status, (int)CSA2_EDEVICE_INDEX);
}

// Joins the pieces of the tile that block x of the attention left open: its own sums and those of the
// blocks after it up to the tile's end, in that order.  blockIdx.y takes every gridDim.y-th row.
template <int D>
__global__ void __launch_bounds__(128) paged_join_kernel(const PagedAttnParams p) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const PagedOpen o = p.open[blockIdx.x];
  if (o.end < 0) return;
  const long long total = p.units[0];
  int last = blockIdx.x + 1;  // blocks blockIdx.x + 1 .. last - 1 computed the rest
  while (last < (int)gridDim.x && total * last / gridDim.x < o.end) ++last;
  constexpr int L4 = D / 4, ROWS = 128 / L4;
  const int d = threadIdx.x % L4 * 4;
  for (int r = threadIdx.x / L4 + ROWS * blockIdx.y; r < o.n; r += ROWS * gridDim.y) {
    float M = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = blockIdx.x; x < last; ++x) {
      const int slot = 2 * x + (x == (int)blockIdx.x ? 1 : 0);
      const long long at = (long long)slot * 16 + r;
      if (total * x / gridDim.x == total * (x + 1) / gridDim.x) continue;  // a block without units wrote nothing
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + at * D + d);
      if (ml.x == -INFINITY && ml.y == 0.f) continue;
      const float m = fmaxf(M, ml.x);
      const float e0 = M == -INFINITY ? 1.f : ex2(M - m), e1 = ml.x == -INFINITY ? 1.f : ex2(ml.x - m);
      a.x = a.x * e0 + v.x * e1, a.y = a.y * e0 + v.y * e1, a.z = a.z * e0 + v.z * e1, a.w = a.w * e0 + v.w * e1;
      L = L * e0 + ml.y * e1;
      M = m;
    }
    const int rr = o.row0 + r, tokn = rr / p.group, hq = o.kv_head * p.group + rr - tokn * p.group;
    store_row<D>(p, o.first_row + tokn, hq, d, a, M, L);
  }
}

template <int D, int NR, int PIECES, bool F16>
cudaError_t launch(const PagedAttnParams& p, int blocks, cudaStream_t stream) {
  constexpr int smem = kWarps * 4 * kTok * D;
  static_assert(smem >= kWarps * NR * D * 4, "the joined sums fit the ring");
  cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<D, NR, PIECES, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  paged_attn_kernel<D, NR, PIECES, F16><<<blocks, kWarps * 32, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks, 4);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D>, p);
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttnParams& p, int q_dtype, int head_dim, bool rows8, int blocks,
                              cudaStream_t stream) {
  const bool f16 = q_dtype == CSA2_T_F16;
  if (head_dim == 128) {
    if (f16) return rows8 ? launch<128, 8, 3, true>(p, blocks, stream) : launch<128, 16, 3, true>(p, blocks, stream);
    return rows8 ? launch<128, 8, 2, false>(p, blocks, stream) : launch<128, 16, 2, false>(p, blocks, stream);
  }
  if (f16) return rows8 ? launch<64, 8, 3, true>(p, blocks, stream) : launch<64, 16, 3, true>(p, blocks, stream);
  return rows8 ? launch<64, 8, 2, false>(p, blocks, stream) : launch<64, 16, 2, false>(p, blocks, stream);
}

}  // namespace csa2
