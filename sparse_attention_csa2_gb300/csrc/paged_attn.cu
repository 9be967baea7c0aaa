// Attention over a paged cache of E4M3 codes with one scale per (page, head), few query rows per
// key-value head: split over the cached tokens and joined.
//
//   z_ij = softmax_scale * q_i . k_j,  k_j = code * k_scale[page, head];  j <= pos_i, j > pos_i - window
//   o_i  = sum_j exp(z_ij) v_j / (sum_j exp(z_ij) + exp(sink))
//
// Bound by the codes' way from memory: 2 * dim bytes per cached token and head, each read once.  32 sequences of
// 65,536 tokens, 8 heads of 8 rows (4.3 GB at dim 128): 637 to 650 us, 6.7 TB/s, 98% of a copy's rate; at dim 64
// 355 us, 89%.  Many short tiles are bound by instructions instead and by their beginnings and ends: 96 sequences of
// 5 tokens, 8 heads, window 1,024 (101 MB, 23.0 M warp instructions) 51 us, of which some 23 are steps; one sequence
// of 2,048 tokens 8.1 us, the chain of two launches, lengths, pages, codes.
// (Sending a tile's first copies out before the one before is joined gained nothing: the SM's other blocks work then.)
//
// Split.  A tile is up to 8 or 16 query rows (tokens x heads of the group) of one sequence and kv head;
// its unit of work is 128 cached tokens.  The units of all tiles of the call form one line, of which
// every block takes an equal piece, so that ragged lengths, one long sequence or many short ones load
// the SMs alike and the host needs no lengths.  A block finds its place by summing the sequences'
// units itself.  A tile that ends inside a block is written out by it; an open one leaves partial
// sums, and a second kernel joins the pieces in order.
//
// Within a block each of the four warps streams its own 32 tokens of a unit through a ring in shared
// memory (TMA copies of 32 tokens of a page, or of two pages of 16; two stages, at dim 64 three or four; a step's keys
// and values arrive on one barrier, which 96 sequences of 5 tokens take 52.0 us with and 55.4 without; no block
// barrier until the tile's end) and keeps its own running maximum, sum and output.
//
// Arithmetic.  Tokens are the MMAs' rows and query rows their columns, eight to a column block, so that
// the few query rows of a decode step fill the tensor cores' shape.  Codes are converted to fp16 (exact).
// A query row is scaled by a power of two to a maximum in [2^14, 2^15): as fp16 its values keep all their
// bits down to 2^-29 of that, and products are summed in fp32.  (K left in its 8 bits against rows as two or
// three E4M3 pieces took more instructions, not fewer: an E4M3 mma.sync counts as two fp16 ones with the
// conversions of both operands and four additions.  Per 32 tokens of 16 rows at dim 64, fp16: 808 against 614
// at that time; 96 sequences of 5 drafted tokens each, window 1,024: 74 against 60 us.)  Weights are fp16 of
// exp2(u - max + 11), u = z + log2(the page's V scale), where the row's maximum of u follows a larger one only when
// that exceeds it by 2^4: weights are at most 2^15, those down to 2^-25 of the largest keep 11 bits, and the output is
// rarely rescaled (paged_dev.cuh).  Maxima, sums and outputs are fp32.  For fp16 rows, whose outputs round as finely
// as the weights (2^-11), what the weights' rounding leaves is multiplied too: the error against 64 bits falls from
// 2.7e-4 to the output's own 2.1e-4, at 5% of the time.
#include "common.cuh"
#include "paged.h"
#include "paged_dev.cuh"
#include "paged_tma.cuh"

namespace csa2 {
namespace {

constexpr int kWarps = 4;
constexpr int kTok = 32;                // tokens of a warp's step
constexpr int kUnit = kWarps * kTok;    // tokens of a unit
constexpr int kLead = 4;                // units that a tile's beginning and end take: each tile lies on the line
                                        // behind so many empty ones (96 sequences of 5 tokens: 3 and 4 take
                                        // 50.1 us, 5 and 6 51.2)

// A sequence with its units.
struct Seq : PagedSeq {
  int lo, blocks;      // first token any row sees, down to a step within its page; units of a tile
  long long units;
};
template <int NR>
__device__ __forceinline__ Seq seq_of(const PagedAttnParams& p, int b) {
  Seq s;
  static_cast<PagedSeq&>(s) = paged_seq<NR>(p, b);
  s.lo = first_seen(p, s.ctx) & (p.page_shift == 4 ? ~15 : ~31);
  s.blocks = max((max(s.kv - s.lo, 0) + kUnit - 1) / kUnit, 1);
  s.units = (long long)s.tiles * p.kv_heads * (s.blocks + kLead);
  return s;
}

// 8x8 matrix of 16-bit values over a warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
  return r;
}
// Stages of the ring: 64 KB a block, 48 KB where four blocks share an SM (dim 64 and 8 rows: 32 sequences of
// 65,536 tokens with 8 heads, when it was tried, 380 us with the fourth block, 414 without; with 16 rows its registers
// spill).
template <int D, int NB>
constexpr int kStages = D == 128 ? 2 : NB == 1 ? 3 : 4;

template <int D, int NB, bool F16>
__global__ void __launch_bounds__(kWarps * 32, D == 64 && NB == 1 ? 4 : 3)
    paged_attn_kernel(const PagedAttnParams p, const __grid_constant__ CopyMaps maps) {
  constexpr int NR = 8 * NB;            // query rows of a tile
  constexpr int KS = D / 16;            // MMA steps of a score
  constexpr int MT = D / 16;            // MMA rows of an output, in sixteens
  constexpr int kStage = kTok * D;      // bytes of K (or V) of a step
  constexpr int kHalf = kStage / 2;     // of 16 tokens: a copy
  constexpr int ST = kStages<D, NB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(16) float scales[kWarps][ST][4];
  __shared__ __align__(8) uint64_t full[kWarps][ST];
  __shared__ float ml[kWarps][NR][2];
  __shared__ long long scan_warp[kWarps];
  __shared__ long long place[2];        // sequence, its first unit
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  if (lane == 0) {  // a warp's barriers are its own
    for (int i = 0; i < ST; ++i) tc05::mbar_init(&full[warp][i], 1);
    tc05::fence_barrier_init();
  }
  __syncwarp();

  prior_done();

  // ---- this block's piece of the line of units
  long long u, u_end, all;
  int b, used;
  long long b_first;
  auto share = [&](long long total) {
    all = total;
    used = (int)min((long long)gridDim.x, total);  // blocks with work: every one of them has some
    u = (int)blockIdx.x < used ? div_rarely_long(total * blockIdx.x, used) : 0;
    u_end = (int)blockIdx.x < used ? div_rarely_long(total * (blockIdx.x + 1), used) : 0;
  };
  auto warp_scan = [&](long long x) {  // inclusive sum over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  if (p.n_seq <= 32) {  // every warp for itself: a sequence a lane
    const long long mine = lane < p.n_seq ? seq_of<NR>(p, lane).units : 0, x = warp_scan(mine);
    share(__shfl_sync(0xffffffffu, x, 31));
    const uint32_t here = __ballot_sync(0xffffffffu, x - mine <= u && u < x);
    b = here ? __ffs(here) - 1 : 0;
    b_first = __shfl_sync(0xffffffffu, x - mine, b);
  } else {
    const int run = (p.n_seq + kWarps * 32 - 1) / (kWarps * 32);
    const int q0 = min(tid * run, p.n_seq), q1 = min(q0 + run, p.n_seq);
    long long mine = 0;
    for (int i = q0; i < q1; ++i) mine += seq_of<NR>(p, i).units;
    const long long x = warp_scan(mine);
    if (lane == 31) scan_warp[warp] = x;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += scan_warp[w];
      total += scan_warp[w];
    }
    before += x - mine;
    share(total);
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
    b = (int)place[0];
    b_first = place[1];
  }
  if (u >= u_end) {
    if (tid == 0) p.open[blockIdx.x].pieces = 0;
    return;
  }
  uint8_t* ring = smem + warp * 2 * ST * kStage;  // stages of K and V
  uint32_t phases = 0;                       // bit of each barrier of `full`: parity of its next completion
  int pieces = 0;                            // of the tile that this block leaves open
  bool bad = false, dead = false;

  while (u < u_end) {
    const Seq s = seq_of<NR>(p, b);
    if (s.units == 0) {
      ++b;
      continue;
    }
    const long long in_seq = u - b_first;
    const long long item = div_rarely_long(in_seq, s.blocks + kLead);
    const int from = (int)(in_seq - item * (s.blocks + kLead)) - kLead;  // place in the tile; below 0 the empty units
    const int run = (int)min((long long)(s.blocks - from), u_end - u);
    const int blk0 = max(from, 0), seg = from + run - blk0;
    if (seg <= 0) {
      u += run;
      continue;
    }
    const int head = s.tiles == 1 ? (int)item : (int)div_rarely_long(item, s.tiles), tile = (int)(item - (long long)head * s.tiles);
    const int row0 = tile * NR, n = min(NR, s.rows - row0);
    const int pos_first = s.ctx + by_group(p, row0), pos_last = s.ctx + by_group(p, row0 + n - 1);
    const int t_begin = s.lo + blk0 * kUnit;
    const int t_end = min(min(t_begin + seg * kUnit, s.kv), pos_last + 1);
    const int lo_last = first_seen(p, pos_last);

    // ---- loads: page ids one step ahead of the copies, copies up to two steps ahead of their use
    const int32_t* trow = p.table + (long long)b * p.table_cols;
    const int page_mask = (1 << p.page_shift) - 1;
    auto page_id = [&](int tok) -> int {  // -1: no such token, -2: a bad entry
      if (tok >= t_end) return -1;
      const int id = trow[tok >> p.page_shift];
      return (unsigned)id < (unsigned)p.n_pages ? id : -2;
    };
    auto second_id = [&](int tok, int id0) -> int {  // pages of 32 tokens and more hold a whole step
      return p.page_shift == 4 ? page_id(tok + 16) : id0;
    };
    auto copy = [&](int slot, int tok, int id0, int id1) {
      if (tok < t_end) {
        uint8_t* to = ring + 2 * slot * kStage;
        if (id0 < 0 || id1 < 0) {  // a half without a page reads as zeros
#pragma unroll
          for (int i = 0; i < 2 * kStage / 512; ++i)
            if ((i % (kStage / 512) < kHalf / 512 ? id0 : id1) < 0) reinterpret_cast<uint4*>(to + 512 * i)[lane] = make_uint4(0, 0, 0, 0);
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          __syncwarp();
        }
        if (lane == 0) {
          uint64_t* bar = &full[warp][slot];
          if (p.page_shift > 4) {  // the maps' boxes are whole steps
            tc05::mbar_expect_tx(bar, id0 >= 0 ? 2 * kStage : 0);
            if (id0 >= 0) {
              tma_load_codes(to, &maps.k, tok & page_mask, id0 * p.kv_heads + head, bar);
              tma_load_codes(to + kStage, &maps.v, tok & page_mask, id0 * p.kv_heads + head, bar);
            }
          } else {
            tc05::mbar_expect_tx(bar, (id0 >= 0 ? kStage : 0) + (id1 >= 0 ? kStage : 0));
            if (id0 >= 0) {
              tma_load_codes(to, &maps.k, 0, id0 * p.kv_heads + head, bar);
              tma_load_codes(to + kStage, &maps.v, 0, id0 * p.kv_heads + head, bar);
            }
            if (id1 >= 0) {
              tma_load_codes(to + kHalf, &maps.k, 0, id1 * p.kv_heads + head, bar);
              tma_load_codes(to + kStage + kHalf, &maps.v, 0, id1 * p.kv_heads + head, bar);
            }
          }
        }
        if (lane < 4) {
          const int id = lane & 1 ? id1 : id0;
          const float* sc = lane < 2 ? p.k_scale : p.v_scale;
          cp_async4(&scales[warp][slot][lane], sc + (id < 0 ? 0 : (long long)id * p.kv_heads + head), id >= 0);
        }
      }
      cp_async_commit();
    };
    auto arrived = [&](int slot) {
      if (!paged_wait(&full[warp][slot], phases >> slot & 1, p.wait_tries)) return false;
      phases ^= 1u << slot;
      return true;
    };
    int tok = t_begin + warp * kTok;
    // the query rows set out first: they and the page ids come together
    uint4 raw[NB][D / 32];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = 8 * nb + g;
      if (r < n) {
        const int rr = row0 + r, i = by_group(p, rr);
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + (long long)(s.first + i) * p.q_row +
                              (long long)(head * p.group + rr - i * p.group) * p.q_head + D / 4 * c;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) raw[nb][k] = *reinterpret_cast<const uint4*>(src + 8 * k);
      } else {
#pragma unroll
        for (int k = 0; k < D / 32; ++k) raw[nb][k] = make_uint4(0, 0, 0, 0);
      }
    }
    uint32_t okay = 0;  // two bits a stage: its halves have pages
    auto note = [&](int slot, int id0, int id1) {
      okay = (okay & ~(3u << 2 * slot)) | (uint32_t)((id0 >= 0) | (id1 >= 0) << 1) << 2 * slot;
      bad |= id0 == -2 || id1 == -2;
    };
    {
      int id0[ST], id1[ST];
#pragma unroll
      for (int i = 0; i < ST; ++i) id0[i] = page_id(tok + i * kUnit), id1[i] = second_id(tok + i * kUnit, id0[i]);
#pragma unroll
      for (int i = 0; i < ST; ++i) {
        note(i, id0[i], id1[i]);
        copy(i, tok + i * kUnit, id0[i], id1[i]);
      }
    }

    // ---- the query rows as fp16: this thread's dims are D/4 * c .. of rows 8 nb + g
    uint32_t qb[NB][KS][2];
    float f[NB][2];   // rows 8 nb + 2c, + 1: score in log2 units = f * sum of products * k_scale
    int pos[NB][2];   // their positions
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      auto pair = [&](int i) -> float2 {  // dims 2i, 2i + 1 of this thread's
        const uint4 u = raw[nb][i >> 2];
        const uint32_t w = (i & 3) == 0 ? u.x : (i & 3) == 1 ? u.y : (i & 3) == 2 ? u.z : u.w;
        return F16 ? __half22float2(*reinterpret_cast<const __half2*>(&w)) : make_float2(bf16_lo(w), bf16_hi(w));
      };
      float amax = 0.f;
      bool odd = false;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float2 v = pair(i);
        odd |= !(fabsf(v.x) < INFINITY) || !(fabsf(v.y) < INFINITY);
        amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      odd = (__ballot_sync(0xffffffffu, odd) >> (4 * g) & 15u) != 0;
      // 2^e with amax / 2^e in [2^14, 2^15)
      const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127 - 14, -110), 119);
      const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
      const float factor = odd ? __uint_as_float(0x7fc00000u) : p.scale_log2 * up;  // a NaN or infinity: the row is NaN
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float2 v = pair(i);
        qb[nb][i >> 1][i & 1] = odd ? 0u : pack_f16x2(v.x * down, v.y * down);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        f[nb][j] = __shfl_sync(0xffffffffu, factor, 4 * (2 * c + j));
        pos[nb][j] = s.ctx + by_group(p, row0 + min(8 * nb + 2 * c + j, n - 1));
      }
    }

    float acc[MT][NB][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) acc[i][nb][0] = acc[i][nb][1] = acc[i][nb][2] = acc[i][nb][3] = 0.f;
    float m[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) m[nb][0] = m[nb][1] = -INFINITY, l[nb][0] = l[nb][1] = 0.f;

    int slot = 0;
    for (; tok < t_end; tok += kUnit, slot = slot + 1 == ST ? 0 : slot + 1) {
      const int next = tok + ST * kUnit;
      const int idc0 = page_id(next), idc1 = second_id(next, idc0);
      const bool ok0 = okay >> 2 * slot & 1, ok1 = okay >> 2 * slot & 2;
      cp_async_wait<ST - 1>();
      dead = !arrived(slot);
      if (dead) break;
      // ---- scores of 32 tokens: S[half][rows of 8][..], tokens 16 half + g (0, 1) and + 8 (2, 3), rows 2c, 2c + 1
      float S[2][NB][4];
      const uint8_t* kt = ring + 2 * slot * kStage;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t wa[KS], wb[KS];
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          const uint4 v = *reinterpret_cast<const uint4*>(kt + swizzled<D>(16 * h + g, D / 64 * c + k));
          const uint4 x = *reinterpret_cast<const uint4*>(kt + swizzled<D>(16 * h + 8 + g, D / 64 * c + k));
          wa[4 * k] = v.x, wa[4 * k + 1] = v.y, wa[4 * k + 2] = v.z, wa[4 * k + 3] = v.w;
          wb[4 * k] = x.x, wb[4 * k + 1] = x.y, wb[4 * k + 2] = x.z, wb[4 * k + 3] = x.w;
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) S[h][nb][0] = S[h][nb][1] = S[h][nb][2] = S[h][nb][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t a0, a1, a2, a3;
          f16_pairs(wa[ks], a0, a2);
          f16_pairs(wb[ks], a1, a3);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma_f16(S[h][nb], a0, a1, a2, a3, qb[nb][ks][0], qb[nb][ks][1]);
        }
      }
      const float4 sc = *reinterpret_cast<const float4*>(scales[warp][slot]);  // k scales, v scales

      // a NaN in either scale marks the page: its visible tokens give NaN
      const float k0 = sc.x + 0.f * sc.z, k1 = sc.y + 0.f * sc.w;
      const float v_log[2] = {paged_v_log(sc.z), paged_v_log(sc.w)};
      const bool whole = tok + kTok - 1 <= min(pos_first, t_end - 1) && tok >= lo_last && ok0 && ok1;
      bool grows = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float2 f2 = make_float2(f[nb][0], f[nb][1]);
        const float2 by[2] = {mul2(f2, make_float2(k0, k0)), mul2(f2, make_float2(k1, k1))};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const float2 z = fma2(make_float2(S[h][nb][j], S[h][nb][j + 1]), by[h], make_float2(v_log[h], v_log[h]));
            S[h][nb][j] = z.x, S[h][nb][j + 1] = z.y;
          }
      }
      if (!whole) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = tok + 16 * h + 8 * (j >> 1) + g;
            const bool there = (h ? ok1 : ok0) && at < t_end;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              const int ps = pos[nb][j & 1];
              if (!(there && at <= ps && (p.window == 0 || at > ps - p.window))) S[h][nb][j] = -INFINITY;
            }
          }
      }
      float top[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          top[nb][j] = fmaxf(fmaxf(S[0][nb][j], S[0][nb][2 + j]), fmaxf(S[1][nb][j], S[1][nb][2 + j]));
          grows |= top[nb][j] > m[nb][j] + kPagedSlack;
        }
      if (__any_sync(0xffffffffu, grows)) {  // a new maximum: what is there moves to it
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float o[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = fmaxf(top[nb][j], m[nb][j]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const float e = m[nb][j] == -INFINITY ? 0.f : ex2(m[nb][j] - x);
            l[nb][j] *= e;
            o[j] = e;
            m[nb][j] = x;
          }
#pragma unroll
          for (int i = 0; i < MT; ++i)
            acc[i][nb][0] *= o[0], acc[i][nb][1] *= o[1], acc[i][nb][2] *= o[0], acc[i][nb][3] *= o[1];
        }
      }
      uint32_t pw[2][NB][2], pr[2][NB][F16 ? 2 : 1];  // weights, and (fp16) what their rounding left
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float2 over = make_float2(m[nb][0] == -INFINITY ? 0.f : kPagedLift - m[nb][0], m[nb][1] == -INFINITY ? 0.f : kPagedLift - m[nb][1]);
        float2 sum = make_float2(l[nb][0], l[nb][1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float back = paged_v_back(v_log[h]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 z = add2(make_float2(S[h][nb][2 * j], S[h][nb][2 * j + 1]), over);
            const float2 e = make_float2(ex2(z.x), ex2(z.y));
            sum = fma2(e, make_float2(back, back), sum);
            const uint32_t w = pack_f16x2(e.x, e.y);
            pw[h][nb][j] = transpose8(w);
            if constexpr (F16) {
              const float2 r = fma2(__half22float2(*reinterpret_cast<const __half2*>(&w)), make_float2(-1.f, -1.f), e);
              pr[h][nb][j] = transpose8(pack_f16x2(r.x, r.y));
            }
          }
        }
        l[nb][0] = sum.x, l[nb][1] = sum.y;
      }
      // ---- outputs: this thread's tokens 2c, 2c + 1, 2c + 8, 2c + 9 of each half, dims D/8 * g ..
      uint8_t* vt = ring + (2 * slot + 1) * kStage;
      if (tok + kTok > t_end) {  // slots behind the last token may hold anything: 0 * NaN is not 0
        if (tok + lane >= t_end) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) *reinterpret_cast<uint4*>(vt + lane * D + 16 * k) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        constexpr int W = D / 32;  // words of D/8 dims
        uint32_t w[4][W];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = 16 * h + 2 * c + (j & 1) + 8 * (j >> 1);
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(vt + swizzled<D>(row, g));
            w[j][0] = v.x, w[j][1] = v.y, w[j][2] = v.z, w[j][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(vt + swizzled<D>(row, g >> 1) + 8 * (g & 1));
            w[j][0] = v.x, w[j][1] = v.y;
          }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {  // dims D/8 * g + 2i, + 1
          const int k = i >> 1, sel = i & 1 ? 0x7362 : 0x5140;
          uint32_t a0, a1, a2, a3;
          f16_pairs(__byte_perm(w[0][k], w[1][k], sel), a0, a1);
          f16_pairs(__byte_perm(w[2][k], w[3][k], sel), a2, a3);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma_f16(acc[i][nb], a0, a1, a2, a3, pw[h][nb][0], pw[h][nb][1]);
            if constexpr (F16) mma_f16(acc[i][nb], a0, a1, a2, a3, pr[h][nb][0], pr[h][nb][1]);
          }
        }
      }
      __syncwarp();
      note(slot, idc0, idc1);
      copy(slot, next, idc0, idc1);
    }
    cp_async_wait<0>();
    if (dead)  // the copies of this step and of those behind it are still under way
      for (int k = 0; k < ST && tok + k * kUnit < t_end; ++k) {
        const int i = (slot + k) % ST;
        paged_wait(&full[warp][i], phases >> i & 1, kPagedTries);
      }

    // ---- the four warps' sums joined
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], 4);
        l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], 8);
        l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], 16);
      }
    if (__syncthreads_or(dead)) {  // a copy never came
      if (tid == 0) {
        if (p.dev_status) atomicExch(p.dev_status, (int)CSA2_ETIMEOUT);
        p.open[blockIdx.x].pieces = 0;
      }
      return;
    }
    float* part = reinterpret_cast<float*>(smem);  // [warp][NR][D]
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float* to = part + (warp * NR + 8 * nb + 2 * c + j) * D + D / 8 * g;
#pragma unroll
        for (int i = 0; i < MT; i += 2)
          *reinterpret_cast<float4*>(to + 2 * i) = make_float4(acc[i][nb][j], acc[i][nb][2 + j], acc[i + 1][nb][j], acc[i + 1][nb][2 + j]);
        if (g == 0) {
          float* to_ml = ml[warp][8 * nb + 2 * c + j];
          to_ml[0] = m[nb][j], to_ml[1] = l[nb][j];
        }
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
        const float e = mw == -INFINITY ? 1.f : ex2(mw - M);
        const float4 a = *reinterpret_cast<const float4*>(part + (w * NR + r) * D + d);
        L += ml[w][r][1] * e;
        o.x += a.x * e, o.y += a.y * e, o.z += a.z * e, o.w += a.w * e;
      }
      if (starts && ends) {
        const int rr = row0 + r, tokn = by_group(p, rr), hq = head * p.group + rr - tokn * p.group;
        paged_put<D>(p, s.first + tokn, hq, d, o, paged_factor(p, hq, M, L));
      } else {
        *reinterpret_cast<float4*>(p.part_o + ((long long)slot_of * NR + r) * D + d) = o;
        if (d == 0) *reinterpret_cast<float2*>(p.part_ml + ((long long)slot_of * NR + r) * 2) = make_float2(M, L);
      }
    }
    if (starts && !ends && tid == 0) {
      PagedOpen& o = p.open[blockIdx.x];
      o.row0 = row0, o.n = n, o.first_row = s.first, o.kv_head = head;
    }
    // the block of the tile's last unit w: the largest x with all * x / used <= w
    pieces = starts && !ends ? (int)(((u - from + s.blocks) * used - 1) / all) - (int)blockIdx.x + 1 : 0;
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    __syncthreads();  // the sums are read before the ring is filled again
    u += run;
    if (u == b_first + s.units) {
      b_first = u;
      ++b;
    }
  }
  if (tid == 0) p.open[blockIdx.x].pieces = pieces;
  if (bad && p.dev_status && lane == 0) atomicExch(p.dev_status, (int)CSA2_EDEVICE_INDEX);
}

template <int D, int NB, bool F16>
cudaError_t launch(const PagedAttnParams& p, int blocks, cudaStream_t stream) {
  constexpr int smem = kWarps * 2 * kStages<D, NB> * kTok * D + 1024;
  static_assert(smem - 1024 >= kWarps * 8 * NB * D * 4, "the joined sums fit the ring");
  CopyMaps maps{};
  constexpr CUtensorMapSwizzle swizzle = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  const int box = p.page_shift == 4 ? 16 : kTok;
  if (!make_codes_map(&maps.k, p.k, p, D, box, swizzle) || !make_codes_map(&maps.v, p.v, p, D, box, swizzle)) return cudaErrorNotSupported;
  cudaError_t e = allow_smem<paged_attn_kernel<D, NB, F16>>(smem);
  if (e != cudaSuccess) return e;
  e = launch_behind(paged_attn_kernel<D, NB, F16>, dim3(blocks), kWarps * 32, smem, stream, p, maps);
  return e != cudaSuccess ? e : launch_paged_join(p, D, 8 * NB, blocks, stream);
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttnParams& p, int q_dtype, int head_dim, int rows, int blocks, cudaStream_t stream) {
  const bool f16 = q_dtype == CSA2_T_F16;
  if (head_dim == 128) return f16 ? launch<128, 1, true>(p, blocks, stream) : launch<128, 1, false>(p, blocks, stream);
  if (f16) return rows == 8 ? launch<64, 1, true>(p, blocks, stream) : launch<64, 2, true>(p, blocks, stream);
  return rows == 8 ? launch<64, 1, false>(p, blocks, stream) : launch<64, 2, false>(p, blocks, stream);
}

}  // namespace csa2
