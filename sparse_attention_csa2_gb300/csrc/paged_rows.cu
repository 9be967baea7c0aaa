// Attention over a paged cache of E4M3 codes, some query rows per key-value head (shared heads, drafted
// tokens), dim 128: tiles of 16 or 32 rows on the tensor cores' 5th generation form, tokens as its rows.
//
// The same sums as the split attention (paged_attn.cu), which serves up to 8 rows at this dim: with 16 its
// outputs and query rows leave registers for two blocks per SM only, which wait for memory more than they
// read (4 sequences of 1M tokens, when both were there: 209 us against 182; in fp16 232 against 183).  Here, per 128
// tokens,
//
//   S^T [128 tokens x rows] = K Q^T      kind::f8f6f4, K's codes as they come from memory (no conversion),
//                                        the query rows as E4M3 pieces added up in the accumulator
//   P^T = fp16 weights, a token per thread
//   O^T [128 dims x rows] += V^T P^T     kind::f16, V's codes converted to fp16 (exact)
//
// with accumulators in tensor memory, so that a thread holds one token's few scores and no outputs.  Bound by
// the codes' way from memory: 256 bytes per cached token and head.  4 sequences of 1M tokens, one head of 16
// rows (1.08 GB): 178 us, 6.0 TB/s, 89% of a copy's rate (pages of 16 tokens; of 64 172 us, 92%; fp16 180 us).
//
//   4 warps  weights (a token per thread), and at a tile's end its output (a dim per thread)
//   4 warps  V to fp16, and the next tile's query pieces
//   1 warp   copies of whole pages into rings of K and of V (TMA), page ids and scales ahead of them
//   1 thread products; the next scores are computed while the present weights are formed
//
// The parts run through the block's tiles without a common barrier, so that one tile's end overlaps the next
// one's copies; work is split over the blocks as in the split attention.  Two blocks per SM with 16 rows.
#include "common.cuh"
#include "paged.h"
#include "paged_dev.cuh"
#include "paged_tma.cuh"

namespace csa2 {
namespace {

constexpr int kTile = 128;              // tokens of a unit
constexpr int kLead = 4;                // units that a tile's beginning and end take (as in paged_attn.cu; not swept here)
constexpr int kThreads = 10 * 32;       // warps: weights 0 .. 3, conversion 4 .. 7, copies 8, products 9
constexpr int kInfos = 8;

// A tile, as its end needs it.
struct TileEnd {
  int first_row, row0, rows, head, blk;
  long long end;  // behind its last unit
};

template <int R, int STAGES>
struct Shared {
  uint64_t k_full[STAGES], k_free[STAGES], v_full[STAGES], v_free[STAGES], s_full[2], s_free[2], info_full[kInfos];
  uint64_t w_full, p_full, pv_done, q_full, q_free, o_full, drained;
  PagedInfo info[kInfos];
  float factor[2][R];  // of a query row: score in log2 units = factor * k_scale * sum of products
  int pos[2][R];       // its position
  float top[R];        // running maxima
  float alpha[R], sum[R];
  float part[4][R];    // of the four warps
  TileEnd tile;
  uint32_t tmem;
  int place_seq;
  long long place_first;
  long long scan[kThreads / 32];
};

// A tile's part in a block: tokens lo + 128 blk .. of n units, none behind hi.
struct Segment {
  PagedSeq s;
  int head, row0, rows, blk, n, blocks, lo, hi, pos_first, pos_last;
};
template <int R>
struct Walk {
  const PagedAttnParams& p;
  long long u, u_end, first;  // first: the sequence's first unit
  int b, known;               // known: the sequence that the segment holds
  __device__ __forceinline__ static int lo_of(const PagedAttnParams& p, const PagedSeq& s) {  // a page's first token
    return first_seen(p, s.ctx) >> p.page_shift << p.page_shift;
  }
  __device__ __forceinline__ static int blocks_of(const PagedAttnParams& p, const PagedSeq& s) {
    return max((max(s.kv - lo_of(p, s), 0) + kTile - 1) / kTile, 1);
  }
  __device__ __forceinline__ static long long units_of(const PagedAttnParams& p, const PagedSeq& s) {
    return (long long)s.tiles * p.kv_heads * (blocks_of(p, s) + kLead);
  }
  __device__ __forceinline__ bool next(Segment& x) {
    while (u < u_end) {
      if (known != b) x.s = paged_seq<R>(p, b);
      known = b;
      const long long units = units_of(p, x.s);
      if (u >= first + units) {
        first += units;
        ++b;
        continue;
      }
      x.blocks = blocks_of(p, x.s);
      const long long item = div_rarely_long(u - first, x.blocks + kLead);
      const int from = (int)(u - first - item * (x.blocks + kLead)) - kLead;
      const int run = (int)min((long long)(x.blocks - from), u_end - u);
      u += run;
      x.blk = max(from, 0), x.n = from + run - x.blk;
      if (x.n <= 0) continue;
      x.head = (int)div_rarely_long(item, x.s.tiles);
      x.row0 = (int)(item - (long long)x.head * x.s.tiles) * R;
      x.rows = min(R, x.s.rows - x.row0);
      x.pos_first = x.s.ctx + by_group(p, x.row0);
      x.pos_last = x.s.ctx + by_group(p, x.row0 + x.rows - 1);
      x.lo = lo_of(p, x.s);
      x.hi = min(x.s.kv, x.pos_last + 1);
      // units behind the last token that a row sees add nothing; one stays, so that every piece has its sums
      x.n = min(x.n, max((max(x.hi - x.lo, 0) + kTile - 1) / kTile - x.blk, 1));
      return true;
    }
    return false;
  }
  // The place on the line of the segment that next() gave last: its tile's first unit.
  __device__ __forceinline__ long long tile_first(const Segment& x) const {
    const long long tile = (long long)x.head * x.s.tiles + x.row0 / R;
    return first + tile * (x.blocks + kLead) + kLead;
  }
};

// R values of each of the warp's lanes (v[r], 0 <= r < R; rows of a tile) to one value per row: halves are
// exchanged and joined until a lane holds row_of_lane<R>'s, in R shuffles or so instead of 5 R.
template <int R>
__device__ __forceinline__ int row_of_lane(int lane) { return R == 32 ? lane : lane >> 1; }
template <int R, typename Op>
__device__ __forceinline__ float over_rows(float (&v)[R], int lane, Op op) {
#pragma unroll
  for (int n = R / 2, o = 16; n > 0; n /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float keep = up ? v[k + n] : v[k], give = up ? v[k] : v[k + n];
      v[k] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  if (R == 16) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
  return v[0];
}
// Barrier of the four weight warps.
__device__ __forceinline__ void weights_sync() { asm volatile("bar.sync 1, 128;\n" ::: "memory"); }
__device__ __forceinline__ bool weights_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

template <int R, int PIECES, bool F16, int STAGES>
__global__ void __launch_bounds__(kThreads, R == 16 ? 2 : 1)
    paged_rows_kernel(const PagedAttnParams p, const __grid_constant__ CopyMaps maps) {
  constexpr int D = 128;
  constexpr int kCodes = kTile * D;            // bytes of a tile's codes
  constexpr int kPanel = kTile * 128;          // 64 dims of V in fp16
  constexpr int kW = D / 64 * kPanel;
  constexpr int kQ = R * D;                    // bytes of a query piece
  constexpr int kCols = R == 16 ? 64 : 128;    // of tensor memory: S0, S1, O
  using Sh = Shared<R, STAGES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* k_ring = smem;
  uint8_t* v_ring = k_ring + STAGES * kCodes;
  uint8_t* w_tile = v_ring + STAGES * kCodes;
  uint8_t* q_tile = w_tile + kW;
  uint8_t* p_tile = q_tile + PIECES * kQ;
  __shared__ Sh sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      tc05::mbar_init(&sh.k_full[i], 1), tc05::mbar_init(&sh.k_free[i], 1);
      tc05::mbar_init(&sh.v_full[i], 1), tc05::mbar_init(&sh.v_free[i], 128);
    }
    for (int i = 0; i < 2; ++i) tc05::mbar_init(&sh.s_full[i], 1), tc05::mbar_init(&sh.s_free[i], 128);
    for (int i = 0; i < kInfos; ++i) tc05::mbar_init(&sh.info_full[i], 1);
    tc05::mbar_init(&sh.w_full, 128), tc05::mbar_init(&sh.p_full, 128), tc05::mbar_init(&sh.pv_done, 1);
    tc05::mbar_init(&sh.q_full, 128), tc05::mbar_init(&sh.q_free, 1), tc05::mbar_init(&sh.o_full, 1);
    tc05::mbar_init(&sh.drained, 1);
    tc05::fence_barrier_init();
  }

  prior_done();
  if (warp == 9) tc05::tmem_alloc(&sh.tmem, kCols);  // not before: the work before may still want tensor memory

  // ---- this block's piece of the line of units
  long long all, u, u_end;
  int used;
  {
    const int run = (p.n_seq + kThreads - 1) / kThreads;
    const int q0 = min(tid * run, p.n_seq), q1 = min(q0 + run, p.n_seq);
    long long mine = 0;
    for (int i = q0; i < q1; ++i) mine += Walk<R>::units_of(p, paged_seq<R>(p, i));
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sh.scan[warp] = x;
    __syncthreads();
    long long before = 0;
    all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sh.scan[w];
      all += sh.scan[w];
    }
    before += x - mine;
    used = (int)min((long long)gridDim.x, all);
    u = (int)blockIdx.x < used ? div_rarely_long(all * blockIdx.x, used) : 0;
    u_end = (int)blockIdx.x < used ? div_rarely_long(all * (blockIdx.x + 1), used) : 0;
    if (u < u_end && before <= u && u < before + mine) {
      int i = q0;
      for (;; ++i) {
        const long long n = Walk<R>::units_of(p, paged_seq<R>(p, i));
        if (u < before + n) break;
        before += n;
      }
      sh.place_seq = i;
      sh.place_first = before;
    }
    tc05::fence_before();
    __syncthreads();
    tc05::fence_after();
  }
  const uint32_t tmem = sh.tmem;
  Walk<R> walk{p, u, u_end, sh.place_first, sh.place_seq, -1};
  Segment x;
  bool dead = false, bad = false;
  int pieces = 0;                // of the tile that this block leaves open
  uint32_t count = 0, segs = 0;  // units, tiles of the block so far
  uint32_t k_sent = 0;           // K's copies (V's: count)
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!dead && !paged_wait(bar, parity, p.wait_tries)) dead = true;
  };

  if (warp < 4) {
    // ------------------------------------------------------------------ weights: a token per thread
    // These warps meet at barriers of their own.  One whose wait ran out while another's was just in time must not
    // leave it there: it goes on through all units and barriers, without waiting, to the block's end.
    const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
    const uint32_t o_cols = lanes + 2 * R;
    while (walk.next(x)) {
      const int par = segs & 1;
      // what the units need of the tile, the rest waits in shared memory
      const int units = x.n, hi = x.hi;
      int tok0 = x.lo + x.blk * kTile;
      // every row sees all 128 tokens of a unit that begins in [seen_lo, seen_hi]
      const int seen_lo = first_seen(p, x.pos_last), seen_hi = min(x.pos_first, x.hi - 1) - kTile + 1;
      const int window = p.window == 0 ? 0x7fffffff : p.window;
      const long long tile_first = walk.tile_first(x);
      if (tid == 0) sh.tile = {x.s.first, x.row0, x.rows, x.head, x.blk, tile_first + x.blocks};
      float2 l[R / 2], low[R / 2];  // sums and minus the maxima of the rows
#pragma unroll
      for (int r = 0; r < R / 2; ++r) l[r] = make_float2(0.f, 0.f), low[r] = make_float2(INFINITY, INFINITY);
      for (int j = 0; j < units; ++j, ++count, tok0 += kTile) {
        const int buf = count & 1;
        wait(&sh.s_full[buf], count >> 1 & 1);
        tc05::fence_after();
        uint32_t s[R];
        tc05::tmem_ld<R>(lanes + R * buf, s);
        const PagedInfo& info = sh.info[count % kInfos];
        const int tok = tok0 + tid, g = tid >> 4;
        const uint32_t flags = info.flags;
        const float ks = flags >> (8 + g) & 1 ? __uint_as_float(0x7fc00000u) : info.k_scale[g];
        const float v_log = info.v_log[g], v_back = info.v_back[g], lift = kPagedLift + v_log;
        const bool whole = flags == 0xffu && tok0 <= seen_hi && tok0 >= seen_lo;
        uint32_t sees = 0xffffffffu;  // bit r: row r sees the token
        if (!whole) {
          sees = 0;
          if (tok < hi && (flags >> g & 1)) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const int ps = sh.pos[par][r];
              if (tok <= ps && ps - tok < window) sees |= 1u << r;
            }
          }
        }
        tc05::tmem_ld_wait();
        tc05::fence_before();
        tc05::mbar_arrive(&sh.s_free[buf]);
        float2 t[R / 2];  // scores
        const float2 ks2 = make_float2(ks, ks);
        float over = -INFINITY;
#pragma unroll
        for (int r = 0; r < R / 2; ++r)
          t[r] = mul2(make_float2(__uint_as_float(s[2 * r]), __uint_as_float(s[2 * r + 1])),
                      mul2(*reinterpret_cast<const float2*>(&sh.factor[par][2 * r]), ks2));
        if (whole) {
#pragma unroll
          for (int r = 0; r < R / 2; ++r) {
            const float2 y = add2(t[r], low[r]);
            over = fmaxf(over, fmaxf(y.x, y.y));
          }
        } else {
#pragma unroll
          for (int r = 0; r < R / 2; ++r) {
            const float2 y = add2(t[r], low[r]);
            if (sees >> (2 * r) & 1) over = fmaxf(over, y.x);
            if (sees >> (2 * r + 1) & 1) over = fmaxf(over, y.y);
          }
        }
        // a first unit, or a weight 2^4 above its row's maximum: everything moves there
        if (j == 0 || weights_any(over + v_log > kPagedSlack)) {
          float top[R];
#pragma unroll
          for (int r = 0; r < R; ++r) top[r] = sees >> r & 1 ? (r & 1 ? t[r / 2].y : t[r / 2].x) + v_log : -INFINITY;
          sh.part[warp][row_of_lane<R>(lane)] = over_rows<R>(top, lane, [](float a, float b) { return fmaxf(a, b); });
          weights_sync();
          if (tid < R) {
            const float old = j == 0 ? -INFINITY : sh.top[tid];
            const float now = fmaxf(old, fmaxf(fmaxf(sh.part[0][tid], sh.part[1][tid]), fmaxf(sh.part[2][tid], sh.part[3][tid])));
            sh.top[tid] = now;
            sh.alpha[tid] = old == -INFINITY ? 0.f : ex2(old - now);
          }
          weights_sync();
#pragma unroll
          for (int r = 0; r < R / 2; ++r) {
            const float2 m = *reinterpret_cast<const float2*>(&sh.top[2 * r]);
            low[r] = make_float2(-m.x, -m.y);
          }
          if (j > 0) {
            wait(&sh.pv_done, (count - 1) & 1);
            tc05::fence_after();
            uint32_t o[R];
            tc05::tmem_ld<R>(o_cols, o);
            tc05::tmem_ld_wait();
#pragma unroll
            for (int r = 0; r < R / 2; ++r) {
              const float2 a = *reinterpret_cast<const float2*>(&sh.alpha[2 * r]);
              l[r] = mul2(l[r], a);
              o[2 * r] = __float_as_uint(__uint_as_float(o[2 * r]) * a.x);
              o[2 * r + 1] = __float_as_uint(__uint_as_float(o[2 * r + 1]) * a.y);
            }
            if constexpr (R == 16) tc05::tmem_st16(o_cols, o);
            else tc05::tmem_st32(o_cols, o);
            tc05::tmem_st_wait();
          }
        }
        // weights
        uint32_t w[R / 2];
        const float2 lift2 = make_float2(lift, lift), back2 = make_float2(v_back, v_back);
        if (whole) {
#pragma unroll
          for (int r = 0; r < R / 2; ++r) {
            const float2 z = add2(add2(t[r], low[r]), lift2);
            const float2 e = make_float2(ex2(z.x), ex2(z.y));
            l[r] = fma2(e, back2, l[r]);
            w[r] = pack_f16x2(e.x, e.y);
          }
        } else {
#pragma unroll
          for (int r = 0; r < R / 2; ++r) {
            const float2 z = add2(add2(t[r], low[r]), lift2);
            const float2 e = make_float2(sees >> (2 * r) & 1 ? ex2(z.x) : 0.f, sees >> (2 * r + 1) & 1 ? ex2(z.y) : 0.f);
            l[r] = fma2(e, back2, l[r]);
            w[r] = pack_f16x2(e.x, e.y);
          }
        }
        if (count > 0) wait(&sh.pv_done, (count - 1) & 1);  // the weights before have been read
#pragma unroll
        for (int k = 0; k < R / 8; ++k)
          *reinterpret_cast<uint4*>(p_tile + swizzled<2 * R>(tid, k)) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        tc05::fence_before();
        tc05::mbar_arrive(&sh.p_full);
      }
      // ---- the tile's outputs, or its partial sums
      {
        float sum[R];
#pragma unroll
        for (int r = 0; r < R; ++r) sum[r] = r & 1 ? l[r / 2].y : l[r / 2].x;
        sh.part[warp][row_of_lane<R>(lane)] = over_rows<R>(sum, lane, [](float a, float b) { return a + b; });
      }
      weights_sync();
      if (tid < R) {  // a row's sum, and what its outputs are to be multiplied by
        const float L = sh.part[0][tid] + sh.part[1][tid] + sh.part[2][tid] + sh.part[3][tid], M = sh.top[tid];
        float den = L;
        if (p.sink != nullptr && M > -INFINITY && tid < sh.tile.rows) {
          const int rr = sh.tile.row0 + tid;
          den += ex2(p.sink[sh.tile.head * p.group + rr - by_group(p, rr) * p.group] * 1.4426950408889634f - M + (kPagedLift - kPagedBias));
        }
        sh.sum[tid] = L;
        sh.alpha[tid] = L == 0.f ? 0.f : __fdividef(9.5367432e-7f, den);
      }
      weights_sync();
      wait(&sh.o_full, segs & 1);
      ++segs;
      tc05::fence_after();
      const auto tile = sh.tile;
      const bool starts = tile.blk == 0, ends = tile.end <= u_end;
      const long long slot = (2LL * blockIdx.x + (starts ? 1 : 0)) * R;
      uint32_t o[R];
      tc05::tmem_ld<R>(o_cols, o);
      tc05::tmem_ld_wait();
      tc05::fence_before();
      const int d = tid;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= tile.rows || dead) break;
        if (starts && ends) {
          const int rr = tile.row0 + r, i = by_group(p, rr);
          const long long at = ((long long)(tile.first_row + i) * (p.kv_heads * p.group) + tile.head * p.group + rr - i * p.group) * D + d;
          const float val = __uint_as_float(o[r]) * sh.alpha[r];
          if (p.out_dtype == CSA2_T_F32) static_cast<float*>(p.out)[at] = val;
          else if (p.out_dtype == CSA2_T_F16) static_cast<__half*>(p.out)[at] = __float2half_rn(val);
          else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(val);
        } else {
          p.part_o[(slot + r) * D + d] = __uint_as_float(o[r]);
          if (d == 0) *reinterpret_cast<float2*>(p.part_ml + (slot + r) * 2) = make_float2(sh.top[r], sh.sum[r]);
        }
      }
      weights_sync();  // maxima and sums are read before the next tile's
      if (starts && !ends) {
        pieces = (int)((tile.end * used - 1) / all) - (int)blockIdx.x + 1;
        if (tid == 0) {
          PagedOpen& open = p.open[blockIdx.x];
          open.row0 = tile.row0, open.n = tile.rows, open.first_row = tile.first_row, open.kv_head = tile.head;
        }
      } else {
        pieces = 0;
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------ query pieces; V to fp16
    const int gt = tid - 128;
    constexpr int TR = 128 / R;                // threads of a query row
    constexpr int QD = D / TR;                 // dims of a thread
    const int qr = gt / TR, qc = gt % TR;
    constexpr int PR = D / 16;                 // 16-byte pieces of a token's codes
    constexpr int RPL = 128 / PR;              // tokens that the threads' pieces cover at once
    const int row_in = gt / PR, c16 = gt % PR;
    while (walk.next(x) && !dead) {
      const int par = segs & 1;
      // the tile's query rows: scaled by a power of two to a maximum in [224, 448), as E4M3 pieces
      const int rr = x.row0 + min(qr, x.rows - 1), i = by_group(p, rr);
      float y[QD];
      float amax = 0.f;
      bool odd = false;
      {
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + (long long)(x.s.first + i) * p.q_row +
                              (long long)(x.head * p.group + rr - i * p.group) * p.q_head + QD * qc;
#pragma unroll
        for (int k = 0; k < QD / 8; ++k) {
          const uint4 v4 = qr < x.rows ? *reinterpret_cast<const uint4*>(src + 8 * k) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const float2 v = F16 ? __half22float2(*reinterpret_cast<const __half2*>(&w[n])) : make_float2(bf16_lo(w[n]), bf16_hi(w[n]));
            y[8 * k + 2 * n] = v.x, y[8 * k + 2 * n + 1] = v.y;
            odd |= !(fabsf(v.x) < INFINITY) || !(fabsf(v.y) < INFINITY);
            amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
        }
      }
#pragma unroll
      for (int o = 1; o < TR; o <<= 1) {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        odd = __shfl_xor_sync(0xffffffffu, (int)odd, o) | odd;
      }
      const uint32_t ua = __float_as_uint(amax);
      int e = (int)(ua >> 23) - 127 - 8 + ((ua & 0x7fffffu) >= 0x600000u ? 1 : 0);
      e = min(max(e, -110), 119);
      const float down = odd ? 0.f : __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int k = 0; k < QD; ++k) y[k] = odd ? 0.f : y[k] * down;
      // the weights of the tile before the last have been formed: its factors may go
      if (segs > 0) wait(&sh.q_free, (segs - 1) & 1);
      if (dead) break;
      if (qc == 0) {
        sh.factor[par][qr] = odd ? __uint_as_float(0x7fc00000u) : p.scale_log2 * up;
        sh.pos[par][qr] = x.s.ctx + i;
      }
#pragma unroll
      for (int m = 0; m < PIECES; ++m)
#pragma unroll
        for (int k = 0; k < QD / 4; ++k) {
          float* z = y + 4 * k;
          const uint32_t w = e4m3_word(z[0], z[1], z[2], z[3]);
          if (m + 1 < PIECES) {
            uint32_t h0, h1;
            f16_pairs(w, h0, h1);
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
            const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
            z[0] -= a.x, z[1] -= a.y, z[2] -= b.x, z[3] -= b.y;  // exact
          }
          const int at = QD * qc + 4 * k;  // byte of the row
          *reinterpret_cast<uint32_t*>(q_tile + m * kQ + swizzled<D>(qr, at >> 4) + (at & 15)) = w;
        }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      tc05::mbar_arrive(&sh.q_full);
      ++segs;
      for (int j = 0; j < x.n && !dead; ++j, ++count) {
        const int stage = count % STAGES;
        wait(&sh.v_full[stage], count / STAGES & 1);
        wait(&sh.info_full[count % kInfos], count / kInfos & 1);
        if (count > 0) wait(&sh.pv_done, (count - 1) & 1);
        if (dead) break;
        const uint8_t* raw = v_ring + stage * kCodes + row_in * D + 16 * c16;
        // fp16 pieces 2 c16 and 2 c16 + 1 of the row's panel; the second panel's lanes store them in the other
        // order, so that a phase's eight lanes meet all banks.  (RPL is a multiple of 8: one swizzle for all.)
        const int sw = c16 >> 2, a = 2 * (c16 & 3);
        uint8_t* to = w_tile + sw * kPanel + row_in * 128;
        uint8_t* to0 = to + (((a + sw) ^ (row_in & 7)) << 4);
        uint8_t* to1 = to + (((a + 1 - sw) ^ (row_in & 7)) << 4);
        auto piece = [&](int q, uint4 w) {
          uint4 h0, h1;
          f16_pairs(sw ? w.z : w.x, h0.x, h0.y);
          f16_pairs(sw ? w.w : w.y, h0.z, h0.w);
          f16_pairs(sw ? w.x : w.z, h1.x, h1.y);
          f16_pairs(sw ? w.y : w.w, h1.z, h1.w);
          *reinterpret_cast<uint4*>(to0 + q * RPL * 128) = h0;
          *reinterpret_cast<uint4*>(to1 + q * RPL * 128) = h1;
        };
        const uint32_t flags = sh.info[count % kInfos].flags;
        const int left = x.hi - x.lo - (x.blk + j) * kTile;  // tokens that are there: what lies behind may be anything
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
        tc05::mbar_arrive(&sh.w_full);
        tc05::mbar_arrive(&sh.v_free[stage]);
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------------ copies
    const int page = 1 << p.page_shift, mask = page - 1;
    while (walk.next(x) && !dead) {
      const int32_t* trow = p.table + (long long)x.s.index * p.table_cols;
      // lane l (as l & 7) knows the page of tokens 16 l .. of a unit
      auto ids = [&](int j) {
        const int tok = x.lo + (x.blk + j) * kTile + 16 * (lane & 7);
        if (j >= x.n || tok >= x.hi) return -1;
        const int id = trow[tok >> p.page_shift];
        return (unsigned)id < (unsigned)p.n_pages ? id : -2;
      };
      int id = ids(0);
      for (int j = 0; j < x.n && !dead; ++j, ++count) {
        const int id_next = ids(j + 1);
        const int stage = count % STAGES;
        const uint32_t parity = (count / STAGES & 1) ^ 1;
        const long long slab = id >= 0 ? (long long)id * p.kv_heads + x.head : 0;
        const float sk = id >= 0 ? p.k_scale[slab] : 0.f, sv = id >= 0 ? p.v_scale[slab] : 0.f;
        bad |= id == -2;
        // a lane whose 16 tokens begin a page (or, in pages of 128, the unit) copies it
        const bool copies = lane < 8 && id >= 0 && (16 * lane & mask & (kTile - 1)) == 0;
        const int rows = min(page, kTile);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, copies)) * rows * D;
        const int tok = x.lo + (x.blk + j) * kTile + 16 * lane;
        wait(&sh.k_free[stage], parity);
        if (dead) break;
        if (lane == 0) tc05::mbar_expect_tx(&sh.k_full[stage], bytes);
        __syncwarp();
        if (copies) tma_load_codes(k_ring + stage * kCodes + 16 * lane * D, &maps.k, tok & mask, (int)slab, &sh.k_full[stage]);
        k_sent = count + 1;
        wait(&sh.v_free[stage], parity);
        if (dead) break;
        if (lane == 0) tc05::mbar_expect_tx(&sh.v_full[stage], bytes);
        __syncwarp();
        if (copies) tma_load_codes(v_ring + stage * kCodes + 16 * lane * D, &maps.v, tok & mask, (int)slab, &sh.v_full[stage]);
        paged_tell(sh.info[count % kInfos], lane, id, sk, sv);
        __syncwarp();
        if (lane == 0) tc05::mbar_arrive(&sh.info_full[count % kInfos]);
        id = id_next;
      }
    }
  } else {
    // ------------------------------------------------------------------ products
    const uint32_t base = uniform(tmem);
    constexpr uint32_t id_s = tc05::idesc_e4m3(128, R);
    // fp32 D, fp16 A and B, both with their other dimension dense
    constexpr uint32_t id_o = (1u << 4) | (1u << 15) | (1u << 16) | ((uint32_t)(R >> 3) << 17) | ((uint32_t)(D >> 4) << 24);
    const uint32_t k_d = desc_lo(smem_u32(k_ring), 16), q_d = desc_lo(smem_u32(q_tile), 16);
    const uint32_t w_d = desc_lo(smem_u32(w_tile), kPanel), p_d = desc_lo(smem_u32(p_tile), 16);
    auto scores = [&](uint32_t n, bool last) {
      const int stage = n % STAGES, buf = n & 1;
      wait(&sh.k_full[stage], n / STAGES & 1);
      wait(&sh.info_full[n % kInfos], n / kInfos & 1);  // for the weights, that wait for the scores alone
      wait(&sh.s_free[buf], (n >> 1 & 1) ^ 1);
      if (dead) return;
      tc05::fence_after();
      const uint32_t a = k_d + (stage * kCodes >> 4);
      if (elected()) {
#pragma unroll
      for (int m = 0; m < PIECES; ++m)
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          mma_f8_ss(base + R * buf, a + (32 * k >> 4), q_d + (m * kQ + 32 * k >> 4), desc_hi(D), id_s, m + k > 0);
        tc05::mma_commit(&sh.s_full[buf]);
        tc05::mma_commit(&sh.k_free[stage]);
        if (last) tc05::mma_commit(&sh.q_free);
      }
      __syncwarp();
    };
    while (walk.next(x) && !dead) {
      const int n = uniform(x.n);
      wait(&sh.q_full, segs & 1);
      ++segs;
      scores(count, n == 1);
      for (int j = 0; j < n && !dead; ++j, ++count) {
        if (j + 1 < n) scores(count + 1, j + 2 == n);
        wait(&sh.w_full, count & 1);
        wait(&sh.p_full, count & 1);
        if (dead) break;
        tc05::fence_after();
        if (elected()) {
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_f16_ss(base + 2 * R, w_d + (2048 * k >> 4), desc_hi(128), p_d + (16 * 2 * R * k >> 4), desc_hi(2 * R), id_o, j > 0 || k > 0);
          tc05::mma_commit(&sh.pv_done);
          if (j + 1 == n) tc05::mma_commit(&sh.o_full);
        }
        __syncwarp();
      }
    }
  }
  if (dead && p.dev_status) atomicExch(p.dev_status, (int)CSA2_ETIMEOUT);
  if (bad && p.dev_status) atomicExch(p.dev_status, (int)CSA2_EDEVICE_INDEX);
  __syncwarp();
  const int any_dead = __syncthreads_or(dead);
  if (tid == 0) p.open[blockIdx.x].pieces = any_dead ? 0 : pieces;
  if (any_dead) {  // copies and products that are under way come to their end before the block does
    if (warp == 8) {
      paged_drain(sh.k_full, k_sent);
      paged_drain(sh.v_full, count);
    } else if (warp == 9) {
      if (elected()) tc05::mma_commit(&sh.drained);
      __syncwarp();
      paged_wait(&sh.drained, 0, kPagedTries);
    }
    __syncthreads();
  }
  if (warp == 9) tc05::tmem_dealloc(tmem, kCols);
}

template <int R, int PIECES, bool F16, int STAGES>
cudaError_t launch(const PagedAttnParams& p, int blocks, cudaStream_t stream) {
  constexpr int D = 128;
  constexpr int smem = 2 * STAGES * kTile * D + kTile * D * 2 + PIECES * R * D + kTile * 2 * R + 1024;
  CopyMaps maps{};
  const int page = min(1 << p.page_shift, kTile);
  if (!make_codes_map(&maps.k, p.k, p, D, page, CU_TENSOR_MAP_SWIZZLE_128B) || !make_codes_map(&maps.v, p.v, p, D, page, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorNotSupported;
  const cudaError_t e = allow_smem<paged_rows_kernel<R, PIECES, F16, STAGES>>(smem);
  if (e != cudaSuccess) return e;
  return launch_behind(paged_rows_kernel<R, PIECES, F16, STAGES>, dim3(blocks), kThreads, smem, stream, p, maps);
}

}  // namespace

cudaError_t launch_paged_rows(const PagedAttnParams& p, int q_dtype, int rows, int blocks, cudaStream_t stream) {
  const bool f16 = q_dtype == CSA2_T_F16;
  const cudaError_t e = rows == 16 ? (f16 ? launch<16, 3, true, 2>(p, blocks, stream) : launch<16, 2, false, 2>(p, blocks, stream))
                                   : (f16 ? launch<32, 3, true, 4>(p, blocks, stream) : launch<32, 2, false, 4>(p, blocks, stream));
  return e != cudaSuccess ? e : launch_paged_join(p, 128, rows, blocks, stream);
}

}  // namespace csa2
