// The experts of a mixture-of-experts layer where an expert meets some tokens (moe.cu has the formulas, the order of the
// work and what bounds it, and serves the others): tiles of 128 weight rows and 64 tokens on the 5th generation's tensor
// cores, weights as A and tokens as B.
//
// The rows of the tokens, an expert's one after the other, are first brought together (16-bit x, so that they are boxes
// of a tensor map like the weights); h is written in that order, as two bf16 that add up to it to 2^-17, of which both
// are multiplied (a third would be read from memory and multiplied like them; what the tensor cores cut off of the sums is as
// much: h's rest 2.5e-6 of fp32 outputs in the mean, all 4.8e-6 at 4,096 x 4,096).  In a block
//
//   warp 0        copies weights (TMA, 128-byte swizzle)          warp 1       copies rows of x or h beside them
//   warp 2        issues the products into two accumulators in tensor memory, by turns
//   warp 3        takes tickets some tiles ahead, and waits for what a tile needs of others
//   warps 4-7     take a tile out of tensor memory; gather rows of x before that, and add up the parts of y behind it
//   warp 8        makes results known to other blocks
//   warps 9-16    with 8-bit weights: codes to bf16 in shared memory, by shifts: the code's exponent as bf16's, 2^-120 too
//                 small, met halfway by rows of x and h times 2^60
//
// Bound by the weights' bytes where an expert meets up to some 100 tokens: 128 tokens of two of 8 experts of 4,096 x 4,096
// in bf16, 805 MB, in 155 us (5.2 TB/s; on the few tokens' kernel 445); in 8 bits, 403 MB, in 183, as the codes' way through
// shared memory (16 KB converted, 16 KB read by the products for 8 KB of codes) is longer than theirs from memory.
#include "moe_dev.cuh"
#include "tc05.cuh"

namespace csa2 {

int device_sm_count();

namespace {

constexpr int kRows = 128, kTokens = 64;
constexpr int kTiles = 4;
constexpr int kEpi = 4, kConv = 8;
constexpr int kFirstEpi = 4, kEnds = 8, kFirstConv = 9;
constexpr int kAtEpi = 1;                     // a barrier
constexpr int kStep = 64;                     // columns of a step of the products
constexpr int kABytes = kRows * 128, kXBytes = 2 * kTokens * 128;
// Tensor memory of a tile: four sums of an up tile, two of a down tile (whose products with both parts of h lie side by side),
// which take the products of 16 columns by turns and are added as fp32: the tensor cores cut a sum off each time that they add
// to it, always towards 0, by more the larger it has grown.  One sum of 8,192 positive products was 3.0e-5 too small, four
// are 3e-6 and two 9e-6.  (128 tokens of 8 experts as a layer: 162.2 us, with one sum 162.0; in 8 bits 196 to 198 and 194.)
constexpr int kAccCols = 4 * kTokens;
constexpr int kGather = 4;                    // rows that a ticket gathers
constexpr int kMost = 8;                      // stages of a ring
constexpr int kSumTokens = 16;                // of a piece of y
constexpr int kUp = 0, kDown = 1, kEnd = 2, kRowsTogether = 3, kSum = 4;
constexpr float kBack = 1152921504606846976.f;  // 2^60

struct WideTile {
  float scale[kRows];      // of the weight rows, where they are codes
  float weight[kTokens];   // of an up tile, the scales of x; of a down tile, the expert's
  int kind, job, expert, row;
  int first, n;            // rows of x or h
  int cols;
  int pad[1];
};
struct WideControl {
  WideTile tile[kTiles];
  uint64_t w_full[kMost], w_free[kMost], x_full[kMost], x_free[kMost], a_full[kMost], a_free[kMost];
  uint64_t tile_full[kTiles], scales_full[kTiles], tile_ready[kTiles], tile_done[kTiles], tile_free[kTiles];
  uint64_t acc_full[2], acc_free[2], drained;
  float exchange[2][64][33];
  int warp_tmp[32];
  uint32_t tmem;
  int dup, dead, last;
};
struct WideMaps {
  MoeMaps w;
  CUtensorMap x, h;
};
struct WideRings {
  int w, x, a;  // stages
};

// A place in a ring.
struct Place {
  int st = 0;
  uint32_t ph = 0, n = 0;
  __device__ __forceinline__ void next(int stages) {
    ++n;
    if (++st == stages) st = 0, ph ^= 1;
  }
  // The stage is free again; true without a wait in the first round.
  __device__ __forceinline__ bool wait_free(uint64_t* bar, int stages, uint32_t tries, volatile int* dead) const {
    return n < (uint32_t)stages || moe_wait(&bar[st], ph ^ 1, tries, dead);
  }
};
__device__ __forceinline__ uint32_t times_2_60(uint32_t v) {  // two bf16
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(v), "r"(0x5d805d80u));
  return r;
}
// Four codes as bf16 times 2^-120.
__device__ __forceinline__ void bf16_tiny(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t even = ((w << 4) & 0x07f007f0u) | ((w << 8) & 0x80008000u), odd = ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
  lo = __byte_perm(even, odd, 0x5410), hi = __byte_perm(even, odd, 0x7632);
}

__host__ __device__ constexpr int threads_of(bool w8) { return (w8 ? kFirstConv + kConv : kFirstConv) * 32; }

template <bool W8, bool X8>
__global__ void __launch_bounds__(threads_of(W8), 1)
    moe_wide_kernel(const __grid_constant__ WideMaps maps, const MoeParams p, const WideRings rings) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int NT = threads_of(W8);
  constexpr int kReaders = kEpi + 4 + (W8 ? kConv : 0);  // warps that look at a tile's description
  uint8_t* w_ring = smem;                                  // weights, or codes of 128 columns
  uint8_t* x_ring = w_ring + rings.w * kABytes;
  uint8_t* a_ring = x_ring + rings.x * kXBytes;            // converted
  WideControl& c = *reinterpret_cast<WideControl*>(a_ring + rings.a * kABytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int every = p.experts + p.shared, slots = p.k + p.shared, pairs = p.tokens * p.k;
  int* jobs = reinterpret_cast<int*>(&c + 1);              // [most_jobs] expert | part << 16
  int* count = jobs + p.most_jobs;                         // [every] rows of an expert
  int* base = count + every;                               // its first
  uint16_t* owner = reinterpret_cast<uint16_t*>(base + every);        // [tokens x slots] of a row: token * slots + slot
  uint16_t* row_of = owner + p.tokens * slots;                        // [tokens x k] the row of an entry
  int16_t* table = reinterpret_cast<int16_t*>(row_of + pairs);        // [tokens x k] expert, or -1
  volatile int* dead = &c.dead;

  if (tid == 0) {
    for (int i = 0; i < kMost; ++i) {
      tc05::mbar_init(&c.w_full[i], 1);
      tc05::mbar_init(&c.w_free[i], W8 ? kConv : 1);
      tc05::mbar_init(&c.x_full[i], 1);
      tc05::mbar_init(&c.x_free[i], 1);
      tc05::mbar_init(&c.a_full[i], kConv);
      tc05::mbar_init(&c.a_free[i], 1);
    }
    for (int i = 0; i < kTiles; ++i) {
      tc05::mbar_init(&c.tile_full[i], 1);
      tc05::mbar_init(&c.scales_full[i], 1);
      tc05::mbar_init(&c.tile_ready[i], 1);
      tc05::mbar_init(&c.tile_done[i], kEpi);
      tc05::mbar_init(&c.tile_free[i], kReaders);
    }
    for (int i = 0; i < 2; ++i) {
      tc05::mbar_init(&c.acc_full[i], 1);
      tc05::mbar_init(&c.acc_free[i], kEpi);
    }
    tc05::mbar_init(&c.drained, 1);
    c.dup = c.dead = 0;
    tc05::fence_barrier_init();
  }
  for (int i = tid; i < every; i += NT) count[i] = i < p.experts ? 0 : p.tokens;
  __syncthreads();
  prior_done();
  if (warp == 0) tc05::tmem_alloc(&c.tmem, 2 * kAccCols);
  int next = 0;  // the first ticket comes while the tokens are looked at
  if (tid == 3 * 32) next = atomicAdd(p.ticket, 1);
  int16_t* ids = reinterpret_cast<int16_t*>(row_of);  // what a token names twice still in it
  for (int i = tid; i < pairs; i += NT) ids[i] = (int16_t)expert_of(p, i);
  __syncthreads();
  for (int i = tid; i < pairs; i += NT) {
    const bool again = named_before(ids, p.k, i);
    if (again) c.dup = 1;
    table[i] = again ? (int16_t)-1 : ids[i];
  }
  __syncthreads();
  if (warp == 1) {  // an entry's place among those of its expert
    for (int q = 0; q < pairs; q += 32) {
      const int i = q + lane, e = i < pairs ? table[i] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      if (e >= 0) row_of[i] = (uint16_t)(count[e] + __popc(same & lanemask_lt()));
      __syncwarp();
      if (e >= 0 && (same & lanemask_lt()) == 0) count[e] += __popc(same);
      __syncwarp();
    }
  }
  tc05::fence_before();
  __syncthreads();
  tc05::fence_after();
  int n_jobs = 0, n_rows = 0;
  for (int o = 0; o < every; o += NT) {  // shared experts first
    const int at = o + tid, e = at < p.shared ? p.experts + at : at - p.shared;
    const int n = at < every ? count[e] : 0, parts = (n + kTokens - 1) / kTokens;
    int all_parts, all_n;
    const int first = n_jobs + block_excl_scan<NT>(parts, c.warp_tmp, &all_parts), row = n_rows + block_excl_scan<NT>(n, c.warp_tmp, &all_n);
    if (at < every) base[e] = row;
    for (int i = 0; i < parts; ++i) jobs[first + i] = e | i << 16;
    n_jobs += all_parts, n_rows += all_n;
  }
  __syncthreads();
  for (int i = tid; i < pairs; i += NT)
    if (table[i] >= 0) {
      const int row = base[table[i]] + row_of[i];
      row_of[i] = (uint16_t)row;
      owner[row] = (uint16_t)(i / p.k * slots + i % p.k);
    }
  for (int i = tid; i < p.shared * p.tokens; i += NT) {
    const int s = i / p.tokens, t = i % p.tokens;
    owner[base[p.experts + s] + t] = (uint16_t)(t * slots + p.k + s);
  }
  __syncthreads();
  const uint32_t tmem = c.tmem;
  const int up_tiles = (p.inner + kRows / 2 - 1) / (kRows / 2), down_tiles = (p.dim + kRows - 1) / kRows;
  const int gathers = (n_rows + kGather - 1) / kGather, first_down = gathers + n_jobs * up_tiles, first_sum = first_down + n_jobs * down_tiles;
  const int sum_parts = (p.tokens + kSumTokens - 1) / kSumTokens, all = first_sum + down_tiles * sum_parts;
  const uint32_t tries = p.wait_tries;
  uint16_t* xg = reinterpret_cast<uint16_t*>(p.x_rows);
  __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(p.h);
  const long long h_plane = (long long)p.tokens * slots * p.inner;
  auto release = [&](int ti) {
    __syncwarp();
    if (lane == 0) tc05::mbar_arrive(&c.tile_free[ti]);
  };
  // The next tile's description; false at the list's end or where a wait ran out.
  auto next_tile = [&](uint32_t i, uint64_t* bar) { return moe_wait(&bar[i % kTiles], i / kTiles & 1, tries, dead) && c.tile[i % kTiles].kind != kEnd; };

  if (n_jobs == 0) {  // no expert is asked for
    fill_out<NT>(p, tid, blockIdx.x, gridDim.x, 0.f);
  } else if (warp == 0) {
    // ---- weights
    constexpr int COLS = W8 ? 128 : kStep;
    Place at;
    bool ok = true;
    for (uint32_t i = 0; ok && next_tile(i, c.tile_full); ++i) {
      const int kind = c.tile[i % kTiles].kind, e = c.tile[i % kTiles].expert, row = c.tile[i % kTiles].row;
      const int cols = c.tile[i % kTiles].cols;
      release(i % kTiles);
      for (int k = 0; k < cols; k += COLS) {
        if (!(ok = at.wait_free(c.w_free, rings.w, tries, dead))) break;
        if (lane == 0) {
          uint8_t* to = w_ring + at.st * kABytes;
          uint64_t* bar = &c.w_full[at.st];
          tc05::mbar_expect_tx(bar, kABytes);
          if (kind == kUp) {
            load_box(to, &maps.w.up, k, row, e, bar);
            load_box(to + kABytes / 2, &maps.w.up, k, p.inner + row, e, bar);
          } else {
            load_box(to, &maps.w.down, k, row, e, bar);
          }
        }
        __syncwarp();
        at.next(rings.w);
      }
    }
    drain(c.w_full, rings.w, at.n);  // nothing is left in flight where a wait ran out
  } else if (warp == 1) {
    // ---- rows of x and h
    Place at;
    bool ok = true;
    for (uint32_t i = 0; ok && next_tile(i, c.tile_ready); ++i) {
      const int kind = c.tile[i % kTiles].kind, first = c.tile[i % kTiles].first;
      const int cols = c.tile[i % kTiles].cols;
      release(i % kTiles);
      asm volatile("fence.proxy.async;\n" ::: "memory");  // they were written by plain stores
      for (int k = 0; k < cols; k += kStep) {
        if (!(ok = at.wait_free(c.x_free, rings.x, tries, dead))) break;
        if (lane == 0) {
          uint8_t* to = x_ring + at.st * kXBytes;
          uint64_t* bar = &c.x_full[at.st];
          tc05::mbar_expect_tx(bar, kind == kUp ? kXBytes / 2 : kXBytes);
          if (kind == kUp) {
            load_box(to, &maps.x, k, first, 0, bar);
          } else {
            load_box(to, &maps.h, k, first, 0, bar);
            load_box(to + kXBytes / 2, &maps.h, k, p.tokens * slots + first, 0, bar);
          }
        }
        __syncwarp();
        at.next(rings.x);
      }
    }
    drain(c.x_full, rings.x, at.n);
  } else if (warp == 2) {
    // ---- products
    uint64_t* a_full = W8 ? c.a_full : c.w_full;
    uint64_t* a_free = W8 ? c.a_free : c.w_free;
    const uint32_t a_base = smem_u32(W8 ? a_ring : w_ring), x_base = smem_u32(x_ring);
    const int a_stages = W8 ? rings.a : rings.w;
    Place a, x;
    uint32_t done = 0;
    bool ok = true;
    for (uint32_t i = 0; ok && next_tile(i, c.tile_full); ++i) {
      const int kind = uniform(c.tile[i % kTiles].kind), cols = uniform(c.tile[i % kTiles].cols);
      const int buf = done & 1;
      // both parts of h side by side: the weights are read from shared memory once
      const uint32_t idesc = kind == kUp ? tc05::idesc_bf16(kRows, kTokens) : tc05::idesc_bf16(kRows, 2 * kTokens);
      release(i % kTiles);
      if (kind == kRowsTogether || kind == kSum) continue;
      if (done >= 2 && !(ok = moe_wait(&c.acc_free[buf], (done / 2 - 1) & 1, tries, dead))) break;
      tc05::fence_after();
      for (int k = 0; k < cols; k += kStep) {
        if (!(ok = moe_wait(&a_full[a.st], a.ph, &c.x_full[x.st], x.ph, tries, dead))) break;
        tc05::fence_after();
        const uint32_t ad = desc_lo(a_base + a.st * kABytes, 16), bd = desc_lo(x_base + x.st * kXBytes, 16);
        if (elected()) {
#pragma unroll
          for (int s = 0; s < 4; ++s)
            mma_f16_ss(tmem + buf * kAccCols + (kind == kUp ? s : s % 2 * 2) * kTokens, ad + 2 * s, desc_hi(128), bd + 2 * s, desc_hi(128),
                       idesc, k > 0 || (kind != kUp && s > 1));
          tc05::mma_commit(&a_free[a.st]);
          tc05::mma_commit(&c.x_free[x.st]);
        }
        __syncwarp();
        a.next(a_stages), x.next(rings.x);
      }
      if (!ok) break;
      if (elected()) tc05::mma_commit(&c.acc_full[buf]);
      __syncwarp();
      ++done;
    }
    if (elected()) tc05::mma_commit(&c.drained);
    __syncwarp();
    paged_wait(&c.drained, 0, kPagedTries);
  } else if (warp == 3) {
    // ---- tickets and what belongs to them, up to kTiles tiles ahead
    uint32_t told = 0;
    bool together = false;  // the rows of x are
    for (uint32_t i = 0;; ++i) {
      const int ti = i % kTiles;
      if (i >= kTiles && !moe_wait(&c.tile_free[ti], (i / kTiles - 1) & 1, tries, dead)) break;
      const int ticket = __shfl_sync(0xffffffffu, next, 0);
      WideTile& tile = c.tile[ti];
      if (ticket >= all) {
        if (lane == 0) {
          tile.kind = kEnd;
          tc05::mbar_arrive(&c.tile_full[ti]);
          tc05::mbar_arrive(&c.tile_ready[ti]);
        }
        break;
      }
      if (lane == 0) next = atomicAdd(p.ticket, 1);  // on its way while this one is looked up
      const int kind = ticket < gathers ? kRowsTogether : ticket < first_down ? kUp : ticket < first_sum ? kDown : kSum;
      if (kind == kRowsTogether) {
        if (lane == 0) {
          tile.kind = kind, tile.first = ticket * kGather, tile.n = min(kGather, n_rows - ticket * kGather);
          tile.cols = 0;
          tc05::mbar_arrive(&c.scales_full[ti]);
          tc05::mbar_arrive(&c.tile_full[ti]);
          tc05::mbar_arrive(&c.tile_ready[ti]);
        }
        __syncwarp();
        if constexpr (W8) ++told;
        continue;
      }
      if (kind == kSum) {
        const int left = ticket - first_sum, row = left / sum_parts, t0 = left % sum_parts * kSumTokens;
        if (lane == 0) {
          tile.kind = kind, tile.row = row * kRows, tile.first = t0, tile.n = min(kSumTokens, p.tokens - t0);
          tile.cols = 0;
          tc05::mbar_arrive(&c.scales_full[ti]);
          tc05::mbar_arrive(&c.tile_full[ti]);
        }
        __syncwarp();
        if constexpr (W8) ++told;
        if (!wait_count(&p.down_done[row], n_jobs, tries, dead)) break;
        if (lane == 0) tc05::mbar_arrive(&c.tile_ready[ti]);
        continue;
      }
      const bool up = kind == kUp;
      const int left = ticket - (up ? gathers : first_down), tiles = up ? up_tiles : down_tiles;
      const int job = left / tiles, e = jobs[job] & 0xffff, part = (jobs[job] >> 16) * kTokens;
      const int row = left % tiles * (up ? kRows / 2 : kRows);
      const int first = base[e] + part, n = min(kTokens, count[e] - part);
      for (int j = lane; j < n; j += 32) {
        const int of = owner[first + j], t = of / slots, s = of - t * slots;
        tile.weight[j] = up ? (X8 ? p.x_scale[t] : 1.f) : s < p.k ? weight_of(p, t, s, c.dup) : 1.f;
      }
      __syncwarp();
      if (lane == 0) {
        tile.kind = kind, tile.job = job, tile.expert = e, tile.row = row, tile.first = first, tile.n = n;
        tile.cols = up ? p.dim : p.inner;
        if constexpr (W8) {  // the rows' scales, both halves' of an up tile
          const int per = up ? kRows / 2 : kRows, rows = min(per, (up ? p.inner : p.dim) - row);
          const float* from = up ? p.up_scale + (long long)e * 2 * p.inner + row : p.down_scale + (long long)e * p.dim + row;
          tc05::mbar_expect_tx(&c.scales_full[ti], rows * (up ? 8 : 4));
          copy_row(tile.scale, from, rows * 4, &c.scales_full[ti]);
          if (up) copy_row(tile.scale + per, from + p.inner, rows * 4, &c.scales_full[ti]);
        }
        tc05::mbar_arrive(&c.tile_full[ti]);
      }
      __syncwarp();
      if constexpr (W8) ++told;
      if (!(up ? together || wait_count(p.gathered, gathers, tries, dead) : wait_count(&p.up_done[job], up_tiles, tries, dead))) break;
      together = true;
      if (lane == 0) tc05::mbar_arrive(&c.tile_ready[ti]);
    }
    drain(c.scales_full, kTiles, told);
  } else if (warp < kEnds) {
    // ---- results
    const int quarter = warp - kFirstEpi, half = quarter >> 1, r = quarter % 2 * 32 + lane;  // r: a row of each half of an up tile
    uint32_t done = 0;
    for (uint32_t i = 0;; ++i) {
      const int ti = i % kTiles;
      bool ok = moe_wait(&c.tile_full[ti], i / kTiles & 1, tries, dead);
      if (part_any<kAtEpi, kEpi * 32>(!ok || *dead)) break;  // all warps go into a tile, or none
      const WideTile& tile = c.tile[ti];
      const int kind = tile.kind, n = tile.n, first = tile.first;
      if (kind == kEnd) break;
      if (kind == kRowsTogether) {
        for (int j = quarter; j < n; j += kEpi) {
          const long long t = owner[first + j] / slots;
          uint4* to = reinterpret_cast<uint4*>(xg + (long long)(first + j) * p.dim);
          if constexpr (X8) {
            const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.x) + t * p.x_row);
            for (int q = lane; q < p.dim / 16; q += 32) {
              const uint4 v = from[q];
              uint32_t b[8];
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                b[2 * m] = e4m3x2_to_bf16x2((uint16_t)w[m]), b[2 * m + 1] = e4m3x2_to_bf16x2((uint16_t)(w[m] >> 16));
                if constexpr (W8) b[2 * m] = times_2_60(b[2 * m]), b[2 * m + 1] = times_2_60(b[2 * m + 1]);
              }
              to[2 * q] = make_uint4(b[0], b[1], b[2], b[3]), to[2 * q + 1] = make_uint4(b[4], b[5], b[6], b[7]);
            }
          } else {
            const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + t * p.x_row);
#pragma unroll 4
            for (int q = lane; q < p.dim / 8; q += 32) {
              uint4 v = from[q];
              if constexpr (W8) v = make_uint4(times_2_60(v.x), times_2_60(v.y), times_2_60(v.z), times_2_60(v.w));
              to[q] = v;
            }
          }
        }
      } else if (kind == kSum) {
        if (moe_wait(&c.tile_ready[ti], i / kTiles & 1, tries, dead))
          add_parts<kEpi * 32>(p, tid - kFirstEpi * 32, tile.row, kRows, first, n, slots, [&](int t, int s) {
            return s >= p.k ? base[p.experts + s - p.k] + t : table[t * p.k + s] >= 0 ? (int)row_of[t * p.k + s] : -1;
          });
      } else {
        const int buf = done & 1;
        ok = moe_wait(&c.acc_full[buf], done / 2 & 1, tries, dead) && (!W8 || moe_wait(&c.scales_full[ti], i / kTiles & 1, tries, dead));
        ++done;
        tc05::fence_after();
        const uint32_t acc = tmem + buf * kAccCols + ((uint32_t)(quarter * 32) << 16);
        auto taken = [&] {
          tc05::fence_before();
          __syncwarp();
          if (lane == 0) tc05::mbar_arrive(&c.acc_free[buf]);
        };
        if (kind == kUp) {
          // warps 0, 1 hold gates, 2, 3 the up projection; each pair gives half of its tokens for half of the others'
          float v[32];
          auto add_up = [&](uint32_t at) {
#pragma unroll
            for (int j0 = 0; j0 < 32; j0 += 8) {
              uint32_t u[4][8];
#pragma unroll
              for (int q = 0; q < 4; ++q) tc05::tmem_ld8(at + q * kTokens + j0, u[q]);
              tc05::tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 8; ++j)
                v[j0 + j] = (__uint_as_float(u[0][j]) + __uint_as_float(u[1][j])) + (__uint_as_float(u[2][j]) + __uint_as_float(u[3][j]));
            }
          };
          add_up(acc + (half == 0 ? 32 : 0));
#pragma unroll
          for (int j = 0; j < 32; ++j) c.exchange[half][r][j] = v[j];
          add_up(acc + (half == 0 ? 0 : 32));
          taken();
          part_sync<kAtEpi, kEpi * 32>();
          const int f = tile.row + r;
          if (ok && f < p.inner) {
            float gate_scale = 1.f, up_scale = 1.f;
            if constexpr (W8) gate_scale = tile.scale[r] * kBack, up_scale = tile.scale[r + kRows / 2] * kBack;
            __nv_bfloat16* at = h + (long long)(first + half * 32) * p.inner + f;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (half * 32 + j >= n) continue;
              const float mine = v[j], others = c.exchange[half ^ 1][r][j], xs = tile.weight[half * 32 + j];
              const float hv = gated((half == 0 ? mine : others) * xs * gate_scale, (half == 0 ? others : mine) * xs * up_scale, p.limit) *
                               (W8 ? kBack : 1.f);
              const __nv_bfloat16 up = __float2bfloat16_rn(hv);
              const float rest = hv - __bfloat162float(up);
              at[(long long)j * p.inner] = up;
              at[h_plane + (long long)j * p.inner] = __float2bfloat16_rn(rest == rest ? rest : 0.f);  // an infinity's is none
            }
          }
          part_sync<kAtEpi, kEpi * 32>();
        } else {
          const int d = tile.row + quarter * 32 + lane;
          float scale = 1.f;
          if constexpr (W8) scale = tile.scale[quarter * 32 + lane] * kBack;
          float* at = p.part + (long long)first * p.dim + d;
#pragma unroll
          for (int j0 = 0; j0 < kTokens; j0 += 8) {
            uint32_t u[4][8];
#pragma unroll
            for (int q = 0; q < 4; ++q) tc05::tmem_ld8(acc + q * kTokens + j0, u[q]);  // h's first parts, second, first, second
            tc05::tmem_ld_wait();
            if (j0 + 8 == kTokens) taken();
            if (ok && d < p.dim) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float v = (__uint_as_float(u[1][j]) + __uint_as_float(u[3][j])) + (__uint_as_float(u[0][j]) + __uint_as_float(u[2][j]));
                if (j0 + j < n) at[(long long)(j0 + j) * p.dim] = v * scale * tile.weight[j0 + j];
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0 && !*dead) tc05::mbar_arrive(&c.tile_done[ti]);
      release(ti);
    }
  } else if (warp == kEnds) {
    // ---- tiles' ends: results are made known while the next ones are computed
    for (uint32_t i = 0; next_tile(i, c.tile_full); ++i) {
      const int ti = i % kTiles, kind = c.tile[ti].kind, row = c.tile[ti].row, job = c.tile[ti].job;
      if (!moe_wait(&c.tile_done[ti], i / kTiles & 1, tries, dead)) break;
      if (lane == 0 && kind != kSum) {
        tell(kind == kUp ? p.up_done + job : kind == kDown ? p.down_done + row / kRows : p.gathered);  // rows of x and h are read by copies
      }
      release(ti);
    }
  } else if constexpr (W8) {
    // ---- codes to bf16
    const int t = tid - kFirstConv * 32;
    Place w, a;
    bool ok = true;
    for (uint32_t i = 0; ok && next_tile(i, c.tile_full); ++i) {
      const int cols = c.tile[i % kTiles].cols;
      release(i % kTiles);
      for (int k = 0; k < cols; k += 128) {
        if (!(ok = moe_wait(&c.w_full[w.st], w.ph, tries, dead))) break;
        const uint8_t* codes = w_ring + w.st * kABytes;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          if (k + part * kStep >= cols) break;
          if (!(ok = a.wait_free(c.a_free, rings.a, tries, dead))) break;
          uint8_t* to = a_ring + a.st * kABytes;
#pragma unroll
          for (int q = t; q < kRows * 4; q += kConv * 32) {  // 16 codes of a row
            const int r = q >> 2, chunk = q & 3;
            const uint4 v = *reinterpret_cast<const uint4*>(codes + swizzled<128>(r, part * 4 + chunk));
            uint4 lo, hi;
            bf16_tiny(v.x, lo.x, lo.y), bf16_tiny(v.y, lo.z, lo.w), bf16_tiny(v.z, hi.x, hi.y), bf16_tiny(v.w, hi.z, hi.w);
            *reinterpret_cast<uint4*>(to + swizzled<128>(r, 2 * chunk)) = lo;
            *reinterpret_cast<uint4*>(to + swizzled<128>(r, 2 * chunk + 1)) = hi;
          }
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          __syncwarp();
          if (lane == 0) tc05::mbar_arrive(&c.a_full[a.st]);
          a.next(rings.a);
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) tc05::mbar_arrive(&c.w_free[w.st]);
        w.next(rings.w);
      }
    }
  }
  tc05::fence_before();
  __syncthreads();
  tc05::fence_after();
  if (warp == 0) tc05::tmem_dealloc(tmem, 2 * kAccCols);
  // the block that leaves last leaves the counters as it found them, and no output that could pass for one after a time-out
  if (tid == 0) c.last = leave(p, c.dead);
  __syncthreads();
  if (c.last) {
    if (c.last == 2) fill_out<NT>(p, tid, 0, 1, __int_as_float(0x7fc00000));
    for (int i = tid; i < n_jobs; i += NT) p.up_done[i] = 0;
    for (int i = tid; i < down_tiles; i += NT) p.down_done[i] = 0;
    if (tid == 0) *p.ticket = 0, *p.left = 0, *p.gathered = 0;
  }
}

// Boxes of 64 columns x 64 rows of 16-bit rows.
bool make_rows_map(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows) {
  return make_expert_map(map, base, false, cols, rows, 1, kTokens);
}

template <bool W8, bool X8>
cudaError_t launch(const MoeParams& p, cudaStream_t stream) {
  WideMaps maps;
  const uint64_t every = p.experts + p.shared, rows = (uint64_t)p.tokens * (p.k + p.shared);
  if (!make_expert_map(&maps.w.up, p.up, W8, p.dim, 2ull * p.inner, every, kRows / 2) ||
      !make_expert_map(&maps.w.down, p.down, W8, p.inner, p.dim, every, kRows) || !make_rows_map(&maps.x, p.x_rows, p.dim, rows) ||
      !make_rows_map(&maps.h, p.h, p.inner, 2 * rows))
    return cudaErrorNotSupported;
  constexpr int kMostSmem = 227 * 1024;
  const int fixed = (int)sizeof(WideControl) + 4 * p.most_jobs + 8 * (int)every + 2 * (int)rows + 4 * p.tokens * p.k + 16;
  // bf16: as many stages of both rings as there is room for; 8 bits: two converted steps, and a stage of codes is two steps
  WideRings rings{};
  if (W8) {
    const int room = (kMostSmem - fixed) / kABytes;  // all stages are of one size
    rings.a = room >= 10 ? 3 : 2;
    rings.w = (room - rings.a) / 2, rings.x = room - rings.a - rings.w;
  } else {
    rings.w = rings.x = (kMostSmem - fixed) / (kABytes + kXBytes);
  }
  static_assert(kABytes == kXBytes, "");
  if (rings.w > kMost) rings.w = kMost;
  if (rings.x > kMost) rings.x = kMost;
  if (rings.w < 2 || rings.x < 2) return cudaErrorInvalidConfiguration;
  const cudaError_t e = allow_smem<moe_wide_kernel<W8, X8>>(kMostSmem);
  if (e != cudaSuccess) return e;
  return launch_behind(moe_wide_kernel<W8, X8>, dim3(device_sm_count()), threads_of(W8),
                       (size_t)(rings.w + rings.x + rings.a) * kABytes + fixed, stream, maps, p, rings);
}

}  // namespace

MoeTiles moe_wide_tiles() { return {kRows, kTokens}; }

cudaError_t launch_moe_wide(const MoeParams& p, bool w8, bool x8, cudaStream_t stream) {
  if (w8) return x8 ? launch<true, true>(p, stream) : launch<true, false>(p, stream);
  return x8 ? launch<false, true>(p, stream) : launch<false, false>(p, stream);
}

}  // namespace csa2
