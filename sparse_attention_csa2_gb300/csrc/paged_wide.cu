// Attention over a paged cache of E4M3 codes, many query rows per key-value head (prompts, chunks,
// long drafts): tiles of 256 query rows on the tensor cores' 5th generation form.
//
// The same sums as the split attention (paged_attn.cu).  Bound by the tensor cores: 4 * dim
// operations per row, head and token, half of them scores (Q K^T) and half outputs (P V).  4,096 rows of 32 heads
// over 8 of 128 dims, behind 32,768 tokens (2.34 TFLOP): 1.97 ms, 1.19 PFLOP/s, 63% of a bf16 product's rate.  A
// score product (128 x 64 x 32 codes) takes 66 cycles, since both its operands come from shared memory (tensor memory
// is full: two row tiles' scores and outputs); the products' cycles add up to three quarters of the time, the rest is
// the chain from scores to weights.
//
// A block holds a tile of 256 rows (tokens x heads of a group) as two of 128 and walks its cached
// tokens 128 at a time:
//   1 warp    copies of whole pages into rings of K and of V (TMA), page ids and scales ahead of them
//   4 warps   V's codes to fp16 (exact), once for both row tiles
//   1 thread  tcgen05.mma: S_t = Q_t K^T into tensor memory (kind::f8f6f4: K's codes as they come, the query
//             rows as E4M3 pieces added up in the accumulator), O_t += P_t V with P_t read from tensor
//             memory (kind::f16).  Scores come in halves of 64 tokens, so that the next half's are there when
//             the softmax of one is done
//   2 x 4 warps  softmax, a row per thread: maximum, weights as fp16 over the scores' own columns,
//             sum; the output is rescaled only where a score exceeds the running maximum by 2^4
//
// K's page scale multiplies the fp32 scores, V's is an addition to the weight's exponent, taken back from each 16
// tokens' sum.  Weights as in the split attention: at most 2^15, 11 bits down to 2^-25 of the largest.
//
// Work is split as there: the units (128 tokens of a tile) of the call form one line, of which each
// block (one per SM) takes an equal piece; open tiles leave partial sums that a second kernel joins.
#include "common.cuh"
#include "paged.h"
#include "paged_dev.cuh"
#include "paged_tma.cuh"

namespace csa2 {
namespace {

constexpr int kRows = 256;
constexpr int kTile = 128;              // tokens of a unit
constexpr int kThreads = 16 * 32;       // warps: softmax 0 .. 7, conversion 8 .. 11, products 12, copies 13 (14, 15 idle)
constexpr int kInfos = 8;
// Registers of a thread of each part, from 128 at launch: 2 * 152 + 104 + 104 = 4 * 128.
constexpr int kSoftmaxRegs = 152, kConvertRegs = 104, kProductRegs = 104;
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }

struct Tile {
  int row0, n, pos_first, pos_last, lo, hi, blocks;
};
__device__ __forceinline__ Tile tile_of(const PagedAttnParams& p, const PagedSeq& s, int t) {
  Tile g;
  g.row0 = t * kRows;
  g.n = min(kRows, s.rows - g.row0);
  g.pos_first = s.ctx + by_group(p, g.row0);
  g.pos_last = s.ctx + by_group(p, g.row0 + g.n - 1);
  g.hi = min(s.kv, g.pos_last + 1);
  g.lo = first_seen(p, g.pos_first) >> p.page_shift << p.page_shift;  // a page's first token
  g.blocks = max((max(g.hi - g.lo, 0) + kTile - 1) / kTile, 1);
  return g;
}

// A place on the line of units: sequence, tile, head, block of the tile.
struct Place {
  int b, t, h, blk;
};
struct Segment {
  PagedSeq s;
  Tile g;
  int h, blk, n;      // its blocks blk .. blk + n - 1
};
// The block's segments one after the other; every role walks them for itself.
struct Walk {
  const PagedAttnParams& p;
  Place at;
  long long u, u_end;
  __device__ __forceinline__ bool next(Segment& x) {
    if (u >= u_end) return false;
    for (;;) {
      x.s = paged_seq<kRows>(p, at.b);
      if (at.t < x.s.tiles) break;
      ++at.b, at.t = at.h = at.blk = 0;
    }
    x.g = tile_of(p, x.s, at.t);
    x.h = at.h, x.blk = at.blk;
    x.n = (int)min((long long)(x.g.blocks - at.blk), u_end - u);
    u += x.n;
    at.blk += x.n;
    if (at.blk == x.g.blocks) {
      at.blk = 0;
      if (++at.h == p.kv_heads) at.h = 0, ++at.t;
    }
    return true;
  }
};

template <int KS, int VS>
struct Shared {
  uint64_t k_full[KS], k_free[KS], r_full[VS], r_free[VS], v_full[2], v_free[2], q_full[2];
  uint64_t s_full[2][2], p_ready[2][2], o_done[2][2];  // [row tile][half]
  uint64_t info_full[kInfos], drained;
  PagedInfo info[kInfos];
  float factor[8][32];  // of the rows of the softmax warps: score in log2 units = factor * k_scale * product
  uint32_t tmem;
  Place place;
  long long scan[kThreads / 32];
};

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1) paged_wide_kernel(const PagedAttnParams p, const __grid_constant__ CopyMaps maps) {
  constexpr int PIECES = F16 ? 3 : 2;          // of a query row: they hold an fp16's 11 bits, a bf16's 8
  constexpr int KS = F16 && D == 128 ? 2 : 3;  // stages of the rings
  constexpr int VS = F16 && D == 128 ? 1 : 2;
  constexpr int kCodes = kTile * D;            // bytes of 128 tokens' (or rows') codes
  constexpr int kPanel = kTile * 128;          // 64 dims of V in fp16
  constexpr int kV = D / 64 * kPanel;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared<KS, VS> sh;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* q_tiles = smem;                     // [row tile][piece]
  uint8_t* k_ring = q_tiles + 2 * PIECES * kCodes;
  uint8_t* v_ring = k_ring + KS * kCodes;
  uint8_t* v_tiles = v_ring + VS * kCodes;     // fp16, two
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < KS; ++i) tc05::mbar_init(&sh.k_full[i], 1), tc05::mbar_init(&sh.k_free[i], 1);
    for (int i = 0; i < VS; ++i) tc05::mbar_init(&sh.r_full[i], 1), tc05::mbar_init(&sh.r_free[i], 128);
    for (int i = 0; i < 2; ++i) {
      tc05::mbar_init(&sh.v_full[i], 128), tc05::mbar_init(&sh.v_free[i], 1);
      tc05::mbar_init(&sh.q_full[i], 128);
      for (int h = 0; h < 2; ++h)
        tc05::mbar_init(&sh.s_full[i][h], 1), tc05::mbar_init(&sh.p_ready[i][h], 128), tc05::mbar_init(&sh.o_done[i][h], 1);
    }
    for (int i = 0; i < kInfos; ++i) tc05::mbar_init(&sh.info_full[i], 1);
    tc05::mbar_init(&sh.drained, 1);
    tc05::fence_barrier_init();
  }

  prior_done();
  if (warp == 12) tc05::tmem_alloc(&sh.tmem, 512);  // not before: the work before may still want tensor memory

  // ---- this block's piece of the line: tiles of the sequences before each (in the space of the tiles),
  // then units of the tiles before each thread's run of tiles
  long long all, u, u_end;
  int used;
  {
    int* tiles_before = reinterpret_cast<int*>(smem);  // [n_seq + 1]
    auto scan = [&](long long v, long long& total) {       // exclusive sum over the block's threads
      long long x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) sh.scan[warp] = x;
      __syncthreads();
      long long before = 0;
      total = 0;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sh.scan[w];
        total += sh.scan[w];
      }
      __syncthreads();
      return before + x - v;
    };
    const int run = (p.n_seq + kThreads - 1) / kThreads;
    const int q0 = min(tid * run, p.n_seq), q1 = min(q0 + run, p.n_seq);
    int mine = 0;
    for (int b = q0; b < q1; ++b) mine += paged_seq<kRows>(p, b).tiles;
    long long n_tiles;
    int before = (int)scan(mine, n_tiles);
    for (int b = q0; b < q1; ++b) tiles_before[b] = before, before += paged_seq<kRows>(p, b).tiles;
    if (tid == 0) tiles_before[p.n_seq] = (int)n_tiles;
    __syncthreads();
    const int trun = (int)((n_tiles + kThreads - 1) / kThreads);
    const int t0 = min(tid * trun, (int)n_tiles), t1 = min(t0 + trun, (int)n_tiles);
    int lo = 0, hi = p.n_seq;  // the sequence of tile t0: the last with tiles_before <= t0 that has tiles
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tiles_before[mid] <= t0) lo = mid; else hi = mid;
    }
    auto walk = [&](auto&& visit) {
      int b = lo;
      PagedSeq s = paged_seq<kRows>(p, b);
      for (int t = t0; t < t1; ++t) {
        while (t >= tiles_before[b + 1]) s = paged_seq<kRows>(p, ++b);
        visit(b, t - tiles_before[b], (long long)tile_of(p, s, t - tiles_before[b]).blocks * p.kv_heads);
      }
    };
    long long units = 0;
    walk([&](int, int, long long n) { units += n; });
    long long first = scan(units, all);
    used = (int)min((long long)gridDim.x, all);
    u = (int)blockIdx.x < used ? div_rarely_long(all * blockIdx.x, used) : 0;
    u_end = (int)blockIdx.x < used ? div_rarely_long(all * (blockIdx.x + 1), used) : 0;
    if (u < u_end && first <= u && u < first + units) {
      walk([&](int b, int t, long long n) {
        if (first <= u && u < first + n) {
          const int blocks = (int)(n / p.kv_heads), in = (int)(u - first);
          sh.place = {b, t, in / blocks, in % blocks};
        }
        first += n;
      });
    }
    // with many sequences the list of tiles reaches into the ring that copies fill next
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    tc05::fence_before();
    __syncthreads();
    tc05::fence_after();
  }
  const uint32_t tmem = sh.tmem;  // all 512 columns: they begin at 0, as the products below know
  Walk walk{p, sh.place, u, u_end};
  Segment x;
  int pieces = 0;
  bool dead = false, bad = false;
  uint32_t k_sent = 0, v_sent = 0;  // copies
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!dead && !paged_wait(bar, parity, p.wait_tries)) dead = true;
  };

  if (warp < 8) {
    more_registers<kSoftmaxRegs>();
    // ------------------------------------------------------------------ softmax: a row per thread
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;  // row of the tile of 128
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_cols = lanes + 256 + D * t;
    uint32_t turn = 0;            // units of this row tile
    uint32_t count = 0;           // units of the block
    while (walk.next(x) && !dead) {
      const int r = 128 * t + row;
      if (128 * t >= x.g.n) {  // no rows in this half: its products are not computed
        count += x.n;
        continue;
      }
      const bool has = r < x.g.n;
      const int rr = x.g.row0 + min(r, x.g.n - 1), i = by_group(p, rr);
      const int pos = x.s.ctx + i;
      // the warp's query rows, scaled to a maximum in [224, 448), as E4M3 pieces: a row at a time by PL lanes, 8
      // values each.  A negative softmax scale turns the sign.
      {
        constexpr int PL = D / 8, AT_ONCE = 32 / PL;
        const int c = lane % PL;
#pragma unroll 4
        for (int k = 0; k < PL; ++k) {
          const int in_warp = k * AT_ONCE + lane / PL, in_tile = (warp & 3) * 32 + in_warp, q_r = 128 * t + in_tile;
          const int q_rr = x.g.row0 + min(q_r, x.g.n - 1), q_i = by_group(p, q_rr);
          const uint16_t* src = static_cast<const uint16_t*>(p.q) + (long long)(x.s.first + q_i) * p.q_row +
                                (long long)(x.h * p.group + q_rr - q_i * p.group) * p.q_head + 8 * c;
          const uint4 v4 = q_r < x.g.n ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {v4.x, v4.y, v4.z, v4.w};
          float2 v[4];
          float amax = 0.f;
          bool odd = false;
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            v[n] = F16 ? __half22float2(*reinterpret_cast<const __half2*>(&w[n])) : make_float2(bf16_lo(w[n]), bf16_hi(w[n]));
            odd |= !(fabsf(v[n].x) < INFINITY) || !(fabsf(v[n].y) < INFINITY);
            amax = fmaxf(amax, fmaxf(fabsf(v[n].x), fabsf(v[n].y)));
          }
#pragma unroll
          for (int o = 1; o < PL; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          odd = (__ballot_sync(0xffffffffu, odd) >> (lane / PL * PL) & (PL == 16 ? 0xffffu : 0xffu)) != 0;
          const uint32_t ua = __float_as_uint(amax);
          int e = (int)(ua >> 23) - 127 - 8 + ((ua & 0x7fffffu) >= 0x600000u ? 1 : 0);
          e = min(max(e, -110), 119);
          float down = odd ? 0.f : __uint_as_float((uint32_t)(127 - e) << 23);
          const float up = __uint_as_float((uint32_t)(127 + e) << 23);
          if (p.scale_log2 < 0.f) down = -down;
#pragma unroll
          for (int n = 0; n < 4; ++n) v[n] = odd ? make_float2(0.f, 0.f) : make_float2(v[n].x * down, v[n].y * down);
          uint8_t* to = q_tiles + t * PIECES * kCodes + swizzled<D>(in_tile, c >> 1) + 8 * (c & 1);
#pragma unroll
          for (int m = 0; m < PIECES; ++m) {
            uint32_t o[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              o[n] = e4m3_word(v[2 * n].x, v[2 * n].y, v[2 * n + 1].x, v[2 * n + 1].y);
              if (m + 1 < PIECES) {
                uint32_t h0, h1;
                f16_pairs(o[n], h0, h1);
                const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
                const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
                v[2 * n].x -= a.x, v[2 * n].y -= a.y, v[2 * n + 1].x -= b.x, v[2 * n + 1].y -= b.y;  // exact
              }
            }
            *reinterpret_cast<uint2*>(to + m * kCodes) = make_uint2(o[0], o[1]);
          }
          if (c == 0) sh.factor[warp][in_warp] = odd ? __uint_as_float(0x7fc00000u) : fabsf(p.scale_log2) * up;
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        tc05::mbar_arrive(&sh.q_full[t]);
        __syncwarp();
      }
      const float f = sh.factor[warp][lane];
      float m = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      const int see_hi = min(pos + 1, x.g.hi), see_lo = first_seen(p, pos);
      for (int j = 0; j < x.n && !dead; ++j, ++count, ++turn) {
        const int tok = x.g.lo + (x.blk + j) * kTile;
        const PagedInfo& info = sh.info[count % kInfos];
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {  // 64 tokens
          wait(&sh.s_full[t][half], turn & 1);
          if (dead) break;
          tc05::fence_after();
          const uint32_t s_cols = lanes + 128 * t + 64 * half;
          const float4 k4 = *reinterpret_cast<const float4*>(info.k_scale + 4 * half);
          const float4 l4 = *reinterpret_cast<const float4*>(info.v_log + 4 * half);
          const float4 b4 = *reinterpret_cast<const float4*>(info.v_back + 4 * half);
          const float k_scale[4] = {f * k4.x, f * k4.y, f * k4.z, f * k4.w};  // of 16 tokens each
          const float v_log[4] = {l4.x, l4.y, l4.z, l4.w}, v_back[4] = {b4.x, b4.y, b4.z, b4.w};
          const int hi = see_hi - tok - 64 * half, lo = see_lo - tok - 64 * half;  // the row sees columns lo .. hi - 1
          const uint32_t flags = info.flags >> 4 * half & 0xf0fu;                   // bits 0-3 and 8-11
          const bool whole = __all_sync(0xffffffffu, hi >= 64 && lo <= 0) && flags == 0xfu;
          // the weights' maximum: of columns that all rows of the warp see from registers, where the scores then
          // stay; otherwise 32 at a time from tensor memory, hidden ones left out
          float top = -INFINITY;
          uint32_t v[2][32];
          const uint32_t from = (uint32_t)max(lo, 0), span = (uint32_t)max(min(hi, 64) - max(lo, 0), 0);
          if (whole) {
#pragma unroll
            for (int c = 0; c < 2; ++c) tc05::tmem_ld32(s_cols + 32 * c, v[c]);
            tc05::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float a = __uint_as_float(v[c][0]), b = __uint_as_float(v[c][16]);
#pragma unroll
              for (int k = 1; k < 16; ++k) a = fmaxf(a, __uint_as_float(v[c][k])), b = fmaxf(b, __uint_as_float(v[c][16 + k]));
              top = fmaxf(top, fmaxf(fmaf(a, k_scale[2 * c], v_log[2 * c]), fmaf(b, k_scale[2 * c + 1], v_log[2 * c + 1])));
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              uint32_t y[32];
              tc05::tmem_ld32(s_cols + 32 * c, y);
              tc05::tmem_ld_wait();
              const uint32_t col = 32u * c - from;
              float a = -INFINITY, b = -INFINITY;
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                if (col + k < span) a = fmaxf(a, __uint_as_float(y[k]));
                if (col + 16 + k < span) b = fmaxf(b, __uint_as_float(y[16 + k]));
              }
              const float *ks = info.k_scale + 4 * half + 2 * c, *vl = info.v_log + 4 * half + 2 * c;
              if ((flags >> (2 * c) & 1) && a > -INFINITY) top = fmaxf(top, fmaf(a, f * ks[0], vl[0]));
              if ((flags >> (2 * c + 1) & 1) && b > -INFINITY) top = fmaxf(top, fmaf(b, f * ks[1], vl[1]));
            }
          }
          const bool grows = top > m + kPagedSlack;
          if (__any_sync(0xffffffffu, grows)) {
            const float to = grows ? top : m;
            const float e = m == -INFINITY ? 0.f : to == m ? 1.f : ex2(m - to);
            l2.x *= e, l2.y *= e;
            m = to;
            if (j + half > 0) {
              wait(&sh.o_done[t][half ^ 1], (turn - (half ^ 1)) & 1);  // the products before: this unit's, or the last one's
              if (dead) break;
              tc05::fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t y[16];
                tc05::tmem_ld16(o_cols + 16 * c, y);
                tc05::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * e);
                tc05::tmem_st16(o_cols + 16 * c, y);
              }
            }
          }
          // weights, over the score columns that have been read
          const float off = m == -INFINITY ? 0.f : kPagedLift - m;
          if (whole) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t w[16];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float ks = k_scale[2 * c + h], o = off + v_log[2 * c + h], back = v_back[2 * c + h];
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 8 * h; k < 8 * h + 8; ++k) {
                  const float2 z = fma2(make_float2(__uint_as_float(v[c][2 * k]), __uint_as_float(v[c][2 * k + 1])), make_float2(ks, ks), make_float2(o, o));
                  const float2 e = make_float2(ex2(z.x), ex2(z.y));
                  sum = add2(sum, e);
                  w[k] = pack_f16x2(e.x, e.y);
                }
                l2 = fma2(sum, make_float2(back, back), l2);
              }
              tc05::tmem_st16(s_cols + 16 * c, w);
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              uint32_t y[32], w[16];
              tc05::tmem_ld32(s_cols + 32 * c, y);
              tc05::tmem_ld_wait();
              const uint32_t col = 32u * c - from;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int g = 2 * c + h;
                const float ks = flags >> (8 + g) & 1 ? __uint_as_float(0x7fc00000u) : f * info.k_scale[4 * half + g];
                const float o = off + info.v_log[4 * half + g];
                const uint32_t here = flags >> g & 1 ? span : 0;  // a page that is not there hides its columns
                float sum = 0.f;
#pragma unroll
                for (int k = 16 * h; k < 16 * h + 16; ++k) {
                  y[k] = __float_as_uint(col + k < here ? ex2(fmaf(__uint_as_float(y[k]), ks, o)) : 0.f);
                  sum += __uint_as_float(y[k]);
                }
                l2.x = fmaf(sum, info.v_back[4 * half + g], l2.x);
              }
#pragma unroll
              for (int k = 0; k < 16; ++k) w[k] = pack_f16x2(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1]));
              tc05::tmem_st16(s_cols + 16 * c, w);
            }
          }
          tc05::tmem_st_wait();
          tc05::fence_before();
          tc05::mbar_arrive(&sh.p_ready[t][half]);
        }
      }
      // ---- the row's output, or its partial sums
      wait(&sh.o_done[t][1], (turn - 1) & 1);
      if (dead) break;
      tc05::fence_after();
      const bool starts = x.blk == 0, ends = x.blk + x.n == x.g.blocks;
      const float L = l2.x + l2.y;
      const long long slot = (2LL * blockIdx.x + (starts ? 1 : 0)) * kRows + r;
      const int head = x.h * p.group + rr - i * p.group;
      const float factor = starts && ends ? paged_factor(p, head, m, L) : 1.f;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        tc05::tmem_ld32(o_cols + 32 * c, v);
        tc05::tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          if (!has) break;
          const float4 o = make_float4(__uint_as_float(v[k]), __uint_as_float(v[k + 1]), __uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
          if (starts && ends) paged_put<D>(p, x.s.first + i, head, 32 * c + k, o, factor);
          else *reinterpret_cast<float4*>(p.part_o + slot * D + 32 * c + k) = o;
        }
      }
      if (has && !(starts && ends)) *reinterpret_cast<float2*>(p.part_ml + slot * 2) = make_float2(m, L);
      tc05::fence_before();
    }
  } else if (warp < 12) {
    fewer_registers<kConvertRegs>();
    // ------------------------------------------------------------------ V's codes to fp16
    const int gt = tid - 256;                  // thread of the group
    constexpr int PR = D / 16;                 // 16-byte pieces of a token's codes
    constexpr int RPL = 128 / PR;              // tokens that the threads' pieces cover at once
    const int row_in = gt / PR, c16 = gt % PR;
    // fp16 pieces 2 c16 and 2 c16 + 1 of the row's panel; the second panel's lanes store them in the other
    // order, so that a phase's eight lanes meet all banks.  (RPL is a multiple of 8: one swizzle for all.)
    const int sw = c16 >> 2, at0 = 2 * (c16 & 3);
    const int to = sw * kPanel + row_in * 128;
    const int to0 = to + (((at0 + sw) ^ (row_in & 7)) << 4), to1 = to + (((at0 + 1 - sw) ^ (row_in & 7)) << 4);
    uint32_t count = 0;
    while (walk.next(x) && !dead) {
      for (int j = 0; j < x.n && !dead; ++j, ++count) {
        const int stage = count % VS;
        wait(&sh.r_full[stage], count / VS & 1);
        wait(&sh.info_full[count % kInfos], count / kInfos & 1);
        wait(&sh.v_free[count & 1], (count >> 1 & 1) ^ 1);
        if (dead) break;
        const uint8_t* raw = v_ring + stage * kCodes + row_in * D + 16 * c16;
        uint8_t* tile = v_tiles + (count & 1) * kV;
        auto piece = [&](int q, uint4 w) {
          uint4 h0, h1;
          f16_pairs(sw ? w.z : w.x, h0.x, h0.y);
          f16_pairs(sw ? w.w : w.y, h0.z, h0.w);
          f16_pairs(sw ? w.x : w.z, h1.x, h1.y);
          f16_pairs(sw ? w.y : w.w, h1.z, h1.w);
          *reinterpret_cast<uint4*>(tile + to0 + q * RPL * 128) = h0;
          *reinterpret_cast<uint4*>(tile + to1 + q * RPL * 128) = h1;
        };
        const uint32_t flags = sh.info[count % kInfos].flags;
        const int left = x.g.hi - x.g.lo - (x.blk + j) * kTile;  // tokens that are there: what lies behind may be anything
        if (left >= kTile && (flags & 0xffu) == 0xffu) {
#pragma unroll
          for (int q = 0; q < kTile / RPL; ++q) piece(q, *reinterpret_cast<const uint4*>(raw + q * RPL * D));
        } else {
#pragma unroll 1
          for (int q = 0; q < kTile / RPL; ++q) {
            const int row = q * RPL + row_in;
            piece(q, row < left && (flags >> (row >> 4) & 1) ? *reinterpret_cast<const uint4*>(raw + q * RPL * D) : make_uint4(0, 0, 0, 0));
          }
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        tc05::mbar_arrive(&sh.v_full[count & 1]);
        tc05::mbar_arrive(&sh.r_free[stage]);
      }
    }
  } else {
    fewer_registers<kProductRegs>();
    if (warp == 13) {
      // ---------------------------------------------------------------- copies
      const int mask = (1 << p.page_shift) - 1, rows = min(1 << p.page_shift, kTile);
      uint32_t count = 0;
      while (walk.next(x) && !dead) {
        const int32_t* trow = p.table + (long long)x.s.index * p.table_cols;
        // lane l (as l & 7) knows the page of tokens 16 l .. of a unit
        auto ids = [&](int j) {
          const int tok = x.g.lo + (x.blk + j) * kTile + 16 * (lane & 7);
          if (j >= x.n || tok >= x.g.hi) return -1;
          const int id = trow[tok >> p.page_shift];
          return (unsigned)id < (unsigned)p.n_pages ? id : -2;
        };
        int id = ids(0);
        for (int j = 0; j < x.n && !dead; ++j, ++count) {
          const int id_next = ids(j + 1);
          const long long slab = id >= 0 ? (long long)id * p.kv_heads + x.h : 0;
          const float sk = id >= 0 ? p.k_scale[slab] : 0.f, sv = id >= 0 ? p.v_scale[slab] : 0.f;
          bad |= id == -2;
          // a lane whose 16 tokens begin a page (or, in pages of 128, the unit) copies it
          const bool copies = lane < 8 && id >= 0 && (16 * lane & mask & (kTile - 1)) == 0;
          const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, copies)) * rows * D;
          const int tok = x.g.lo + (x.blk + j) * kTile + 16 * lane;
          const int ks = count % KS, vs = count % VS;
          wait(&sh.k_free[ks], (count / KS & 1) ^ 1);
          if (dead) break;
          if (lane == 0) tc05::mbar_expect_tx(&sh.k_full[ks], bytes);
          __syncwarp();
          if (copies) tma_load_codes(k_ring + ks * kCodes + 16 * lane * D, &maps.k, tok & mask, (int)slab, &sh.k_full[ks]);
          k_sent = count + 1;
          paged_tell(sh.info[count % kInfos], lane, id, sk, sv);
          __syncwarp();
          if (lane == 0) tc05::mbar_arrive(&sh.info_full[count % kInfos]);
          wait(&sh.r_free[vs], (count / VS & 1) ^ 1);
          if (dead) break;
          if (lane == 0) tc05::mbar_expect_tx(&sh.r_full[vs], bytes);
          __syncwarp();
          if (copies) tma_load_codes(v_ring + vs * kCodes + 16 * lane * D, &maps.v, tok & mask, (int)slab, &sh.r_full[vs]);
          v_sent = count + 1;
          id = id_next;
        }
      }
    } else if (warp == 12) {
      // ---------------------------------------------------------------- products
      constexpr uint32_t id_s = tc05::idesc_e4m3(128, 64);
      constexpr uint32_t id_o = (1u << 4) | 1u << 16 | (uint32_t)(D >> 3) << 17 | (uint32_t)(128 >> 4) << 24;  // fp16, B's dims dense
      const uint32_t q_d = desc_lo(smem_u32(q_tiles), 16), k_d = desc_lo(smem_u32(k_ring), 16), v_d = desc_lo(smem_u32(v_tiles), kPanel);
      uint32_t count = 0, segs = 0, turns = 0;  // bits 0, 1: parity of the row tiles' next use
      // unit n's scores of one half (64 tokens) into the columns that its weights will take
      auto scores = [&](int t, int half, uint32_t n) {
        const uint32_t a = q_d + t * (PIECES * kCodes >> 4), b = k_d + (n % KS) * (kCodes >> 4) + half * (64 * D >> 4);
#pragma unroll
        for (int m = 0; m < PIECES; ++m)
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            mma_f8_ss(128 * t + 64 * half, a + (m * kCodes + 32 * k >> 4), b + (32 * k >> 4), desc_hi(D), id_s, m + k > 0);
        tc05::mma_commit(&sh.s_full[t][half]);
      };
      auto outputs = [&](int t, int half, uint32_t n, bool acc) {
        const uint32_t b = v_d + (n & 1) * (kV >> 4) + half * (64 * 128 >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16_ts(256 + D * t, 128 * t + 64 * half + 8 * k, b + (2048 * k >> 4), desc_hi(128), id_o, acc || k > 0);
        tc05::mma_commit(&sh.o_done[t][half]);
      };
      auto keys = [&](uint32_t n) {  // unit n's codes, and what the softmax, that waits for the scores alone, needs of it
        wait(&sh.info_full[n % kInfos], n / kInfos & 1);
        wait(&sh.k_full[n % KS], n / KS & 1);
      };
      while (walk.next(x) && !dead) {
        const int tiles = uniform(x.g.n) > 128 ? 2 : 1, n = uniform(x.n);
        for (int t = 0; t < tiles; ++t) wait(&sh.q_full[t], segs >> t & 1);
        segs ^= tiles == 2 ? 3u : 1u;
        keys(count);
        if (dead) break;
        tc05::fence_after();
        if (elected()) {
          for (int half = 0; half < 2; ++half)
            for (int t = 0; t < tiles; ++t) scores(t, half, count);
          tc05::mma_commit(&sh.k_free[count % KS]);
        }
        __syncwarp();
        for (int j = 0; j < n && !dead; ++j, ++count) {
          const bool more = j + 1 < n;
          wait(&sh.v_full[count & 1], count >> 1 & 1);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (t == tiles || dead) break;
              wait(&sh.p_ready[t][half], turns >> t & 1);
              if (half + t == 0 && more) keys(count + 1);
              if (dead) break;
              tc05::fence_after();
              if (elected()) {
                outputs(t, half, count, j + half > 0);
                if (more) scores(t, half, count + 1);
                if (half == 1 && t == tiles - 1) {
                  tc05::mma_commit(&sh.v_free[count & 1]);
                  if (more) tc05::mma_commit(&sh.k_free[(count + 1) % KS]);
                }
              }
              __syncwarp();
            }
          }
          turns ^= tiles == 2 ? 3u : 1u;
        }
      }
    }
  }
  if (dead && p.dev_status) atomicExch(p.dev_status, (int)CSA2_ETIMEOUT);
  if (bad && p.dev_status) atomicExch(p.dev_status, (int)CSA2_EDEVICE_INDEX);
  // the tile that stays open at the end
  if (tid == 0 && u < u_end) {
    Walk last{p, sh.place, u, u_end};
    while (last.next(x)) {
    }
    if (x.blk == 0 && x.n < x.g.blocks) {
      pieces = (int)(((u_end - x.n + x.g.blocks) * used - 1) / all) - (int)blockIdx.x + 1;
      PagedOpen& o = p.open[blockIdx.x];
      o.row0 = x.g.row0, o.n = x.g.n, o.first_row = x.s.first, o.kv_head = x.h;
    }
  }
  __syncwarp();
  const int any_dead = __syncthreads_or(dead);
  if (tid == 0) p.open[blockIdx.x].pieces = any_dead ? 0 : pieces;
  if (any_dead) {  // copies and products that are under way come to their end before the block does
    if (warp == 13) {
      paged_drain(sh.k_full, k_sent);
      paged_drain(sh.r_full, v_sent);
    } else if (warp == 12) {
      if (elected()) tc05::mma_commit(&sh.drained);
      __syncwarp();
      paged_wait(&sh.drained, 0, kPagedTries);
    }
    __syncthreads();
  }
  if (warp == 12) tc05::tmem_dealloc(tmem, 512);
}

template <int D, bool F16>
cudaError_t launch(const PagedAttnParams& p, int blocks, cudaStream_t stream) {
  constexpr bool LARGE = F16 && D == 128;
  constexpr int smem = (2 * (F16 ? 3 : 2) + (LARGE ? 3 : 5)) * kTile * D + 2 * kTile * D * 2 + 1024;
  CopyMaps maps{};
  const int page = min(1 << p.page_shift, kTile);
  if (!make_codes_map(&maps.k, p.k, p, D, page, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) ||
      !make_codes_map(&maps.v, p.v, p, D, page, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorNotSupported;
  const cudaError_t e = allow_smem<paged_wide_kernel<D, F16>>(smem);
  if (e != cudaSuccess) return e;
  return launch_behind(paged_wide_kernel<D, F16>, dim3(blocks), kThreads, smem, stream, p, maps);
}

}  // namespace

cudaError_t launch_paged_wide(const PagedAttnParams& p, int q_dtype, int head_dim, int blocks, cudaStream_t stream) {
  const bool f16 = q_dtype == CSA2_T_F16;
  const cudaError_t e = head_dim == 128 ? (f16 ? launch<128, true>(p, blocks, stream) : launch<128, false>(p, blocks, stream))
                                        : (f16 ? launch<64, true>(p, blocks, stream) : launch<64, false>(p, blocks, stream));
  return e != cudaSuccess ? e : launch_paged_join(p, head_dim, kRows, blocks, stream);
}

}  // namespace csa2
