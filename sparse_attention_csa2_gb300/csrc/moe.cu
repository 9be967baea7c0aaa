// The experts of a mixture-of-experts layer for a few tokens, as one kernel:
//
//   [g; u] = W_up[e] x_t,  h = silu(min(g, L)) clamp(u, -L, L),  y_t = sum_e w_te W_down[e] h
//
// over the routed experts of each token and the shared ones.  Bound by the weights of the experts that are met, which
// are read once (per 8 tokens of an expert): of 4,096 x 2,048 in 8 bits, a token's 6 experts and the shared one, 176 MB, in
// 41 us, of which some 12 are the launch's beginning, the first copies' way and the end; 32 tokens' 154 experts, 3.9 GB, in
// 604 us or 6.5 TB/s (582 with h in one part).  The work is a list of tiles of weight rows: all tiles of gate and
// up rows, expert after expert, then all of down rows.  Blocks, one per SM, take tiles from a counter.  In a block
//
//   warp 16      copies weights (TMA, 128-byte swizzle) into a ring of stages
//   warp 17      copies the tokens' rows of x, or of h, beside them
//   warp 18      takes tickets some tiles ahead, finds the tiles' tokens, and waits for the up tiles that a down tile needs
//   warps 0-15   products (mma.sync: weights as A, 8 tokens as B), sums over the warps' parts of the columns, results
//   warps 19-22  make a tile's results known to other blocks, and add up the parts of y where they are the last
//
// so that the weights' way from memory is never broken: the copies of a down tile are under way while its h is not yet
// there.  A tile waits only for tiles with earlier tickets, and those are held by blocks that run and do not wait
// themselves (up tiles wait for nothing), so the list ends whatever blocks are resident.  The block that finishes the
// last tile of some rows of y adds up their parts in the order of the token's experts: results do not depend on timing.
//
// tcgen05 is not used here: at a few tokens per expert the tensor cores have little to win, and 8-bit weights have to be
// converted in registers in front of them, from where mma.sync takes them as they are.
//
// bf16 weights multiply bf16: x as it is, fp32 h as three bf16 that add up to it (two leave 2^-17 of it, six times what the
// sums of 512 columns are off by; 5 tokens' layer of 60 experts 51.8 us, with three 53).  E4M3 codes become fp16 (exact, an
// instruction for two; as bf16 they take seven for four) and multiply fp16: codes of x exactly, bf16 x and fp32 h times a
// power of two that brings the row's largest to 2^14 .. 2^15, so that nothing is lost of x, and h in two parts keeps 22 bits
// whatever the output's type (one part, 11 bits, moves a tenth of the bf16 outputs to their neighbour; 32 tokens' layer of 384
// experts 494 us with one part, 509 with two).
#include "moe_dev.cuh"

namespace csa2 {

int device_sm_count();

namespace {

constexpr int kWarps = 16;                  // of products
constexpr int kEnds = 4;                    // of the tiles' ends
constexpr int kThreads = (kWarps + 3 + kEnds) * 32;
constexpr int kTiles = 4;                   // of the ring of tile descriptions
constexpr int kRedRow = 10;                 // floats of a row of 8 tokens among the parts to be summed

constexpr int kR = 64;                      // weight rows of a tile
constexpr int kTok = 8;                     // tokens
constexpr int kKW = 8;                      // parts of a stage's columns: a warp has one of them, of 32 rows
constexpr int kMT = 2;                      // 16-row pieces of a warp
static_assert(kKW * (kR / (16 * kMT)) == kWarps, "");
static_assert(kR / 2 == 32 && kR * kTok == kWarps * 32, "a result of a tile per thread");
constexpr int kRed = kKW * kR * kRedRow * 4;

// 512 columns a stage of codes: with 256 (16 KB) what a stage costs the products' warps besides (two waits, operands'
// latencies) is twice as much in all (a batch of 32 tokens 692 us; 34 experts 163, with 256 columns 200).
template <bool W8_, bool X8_>
struct Shape {
  static constexpr bool W8 = W8_, X8 = X8_;
  static constexpr int KST = W8 ? 512 : 256;      // columns of a stage
  static constexpr int KWARP = KST / kKW;         // of a warp
  static constexpr int BOXES = KST * (W8 ? 1 : 2) / 128;
  static constexpr int BOXCOLS = W8 ? 128 : 64;
  // Rows of x and h beside the weights, apart so that a load meets no bank twice.
  static constexpr int PITCH = KST * 2 + (W8 ? 32 : 16);  // 16-bit values
  __host__ __device__ static constexpr int value_bytes(int kind) { return kind == 0 ? (X8 ? 1 : 2) : 4; }
  __host__ __device__ static constexpr int row_bytes(int kind) { return kind == 0 ? (X8 ? KST + 16 : PITCH) : KST * 4 + (W8 ? 64 : 32); }
  static constexpr int W_BYTES = kR * 128 * BOXES;
  __host__ __device__ static constexpr int parts(int kind) { return kind == 0 ? 1 : W8 ? 2 : 3; }  // of the tokens' values
  static constexpr int X_BYTES = kTok * row_bytes(1);
  static constexpr int STAGE = W_BYTES + (X_BYTES + 1023) / 1024 * 1024;
};
constexpr int kMaxStages = 8;

struct Tile {
  float scale[kR];     // of the weight rows, where they are codes
  int slot[kTok];     // token * slots + slot
  float lift[kTok];   // what rows that become fp16 are multiplied by
  float weight[kTok]; // what the products are multiplied by: x's scale or the expert's weight, over the lift
  int kind;           // 0: up, 1: down, 2: the list is at its end
  int job, expert, row;  // row: the tile's first
  int n;              // tokens
  int pad[3];
};
struct Control {
  Tile tile[kTiles];
  uint64_t w_full[kMaxStages], x_full[kMaxStages], free_[kMaxStages];
  uint64_t tile_full[kTiles], scales_full[kTiles], tile_ready[kTiles], tile_done[kTiles], tile_free[kTiles];
  int warp_tmp[kThreads / 32];
  int dup, dead, last;
};

constexpr int kProducts = 1, kAtEnds = 2;  // barriers of the products' warps and of the tiles' ends
// The power of two that brings a largest value (as bits) to 2^14 .. 2^15, and its inverse.  Beside an infinity nothing else
// becomes one.
__device__ __forceinline__ int lift_of(uint32_t top) { return top == 0 ? 0 : min(14 - ((int)(top >> 23) - 127), 100); }
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }

// Two fp16 of which a NaN becomes the lowest finite value: beside an infinity that what is left of it.
__device__ __forceinline__ uint32_t above_lowest(uint32_t v) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(v), "r"(0xfbfffbffu));
  return r;
}

// The B operand of 8 tokens x 16 columns, row g of them at `at`, in the order in which the weights' operand has its
// columns: their own for bf16, for codes four neighbours to a lane.  b[1], b[2]: what h's roundings leave.
template <class S, int KIND>
__device__ __forceinline__ void load_b(const uint8_t* at, int t, float lift, uint32_t (&b)[3][2]) {
  if constexpr (S::W8 && KIND == 1) {
    const float4 v = *reinterpret_cast<const float4*>(at + 16 * t);
    const float2 lifts = make_float2(lift, lift), less = make_float2(-1.f, -1.f);
    const float2 f[2] = {mul2(make_float2(v.x, v.y), lifts), mul2(make_float2(v.z, v.w), lifts)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      b[0][i] = pack_f16x2(f[i].x, f[i].y);
      const float2 rest = fma2(__half22float2(*reinterpret_cast<const __half2*>(&b[0][i])), less, f[i]);
      b[1][i] = above_lowest(pack_f16x2(rest.x, rest.y));
    }
  } else if constexpr (S::W8 && S::X8) {
    f16_pairs(*reinterpret_cast<const uint32_t*>(at + 4 * t), b[0][0], b[0][1]);
  } else if constexpr (S::W8) {
    const uint2 v = *reinterpret_cast<const uint2*>(at + 8 * t);
    b[0][0] = pack_f16x2(bf16_lo(v.x) * lift, bf16_hi(v.x) * lift);
    b[0][1] = pack_f16x2(bf16_lo(v.y) * lift, bf16_hi(v.y) * lift);
  } else if constexpr (S::X8 && KIND == 0) {
    b[0][0] = e4m3x2_to_bf16x2(*reinterpret_cast<const uint16_t*>(at + 2 * t));
    b[0][1] = e4m3x2_to_bf16x2(*reinterpret_cast<const uint16_t*>(at + 2 * t + 8));
  } else if constexpr (KIND == 0) {
    b[0][0] = *reinterpret_cast<const uint32_t*>(at + 4 * t);
    b[0][1] = *reinterpret_cast<const uint32_t*>(at + 4 * t + 16);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float2 v = *reinterpret_cast<const float2*>(at + 8 * t + 32 * i);
#pragma unroll
      for (int part = 0; part < 3; ++part) {  // 8 bits of 24 are cut off each
        b[part][i] = __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632);
        v.x -= bf16_lo(b[part][i]), v.y -= bf16_hi(b[part][i]);
        if (part == 0) v.x = v.x == v.x ? v.x : 0.f, v.y = v.y == v.y ? v.y : 0.f;  // an infinity leaves nothing
      }
    }
  }
}

// The products of a stage: KIND 0 with rows of x, 1 with rows of h.
template <class S, int KIND>
__device__ __forceinline__ void stage_products(const uint8_t* w, const uint8_t* x, int cols, const Tile& tile, int warp, int lane,
                                               float (&acc)[kMT][4]) {
  const int g = lane >> 2, t = lane & 3;
  const int k_first = warp % kKW * S::KWARP, row_first = warp / kKW * (kMT * 16);
  const int arow = row_first + (lane & 15), achunk = lane >> 4;
  constexpr int PER = S::W8 ? 2 : 1;  // 16-column steps of one load of A
  constexpr int ROW = S::row_bytes(KIND), SIZE = S::value_bytes(KIND);
  const float lift = S::W8 && !(S::X8 && KIND == 0) ? tile.lift[g] : 1.f;
#pragma unroll
  for (int k = 0; k < S::KWARP; k += 16 * PER) {
    const int at = k_first + k;  // column within the stage
    if (at >= cols) break;
    uint32_t a[kMT][4];
    const int byte = at * (S::W8 ? 1 : 2);
    const uint8_t* box = w + byte / 128 * (kR * 128);
#pragma unroll
    for (int m = 0; m < kMT; ++m)
      ldsm_x4(a[m][0], a[m][1], a[m][2], a[m][3], smem_u32(box + swizzled<128>(arow + m * 16, byte % 128 / 16 + achunk)));
#pragma unroll
    for (int s = 0; s < PER; ++s) {
      if (s && at + 16 >= cols) break;
      uint32_t f[kMT][4];
#pragma unroll
      for (int m = 0; m < kMT; ++m) {
        if constexpr (S::W8) {
          f16_pairs(a[m][2 * s], f[m][0], f[m][2]);
          f16_pairs(a[m][2 * s + 1], f[m][1], f[m][3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) f[m][i] = a[m][i];
        }
      }
      uint32_t b[3][2];
      load_b<S, KIND>(x + g * ROW + (at + 16 * s) * SIZE, t, lift, b);
#pragma unroll
      for (int i = 0; i < S::parts(KIND); ++i) {
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
          if constexpr (S::W8) mma_f16(acc[m], f[m][0], f[m][1], f[m][2], f[m][3], b[i][0], b[i][1]);
          else mma_bf16(acc[m], f[m][0], f[m][1], f[m][2], f[m][3], b[i][0], b[i][1]);
        }
      }
    }
  }
}

template <class S>
__global__ void __launch_bounds__(kThreads, 1) moe_kernel(const __grid_constant__ MoeMaps maps, const MoeParams p, const int stages) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;
  float* red = reinterpret_cast<float*>(smem + stages * S::STAGE);
  Control& c = *reinterpret_cast<Control*>(reinterpret_cast<uint8_t*>(red) + kRed);
  const int every = p.experts + p.shared, slots = p.k + p.shared, pairs = p.tokens * p.k;
  int* jobs = reinterpret_cast<int*>(&c + 1);            // [p.most_jobs] expert | part of its tokens << 16
  int* count = jobs + p.most_jobs;                       // [experts] tokens
  uint32_t* x_top = reinterpret_cast<uint32_t*>(count + p.experts + p.shared);  // [tokens] largest |x|, where it becomes fp16
  int16_t* table = reinterpret_cast<int16_t*>((reinterpret_cast<uintptr_t>(x_top + p.tokens) + 15) / 16 * 16);  // [tokens x k, up to a multiple of 8] expert, or -1
  int16_t* ids = table + (pairs + 7) / 8 * 8;                                                // the same with what a token names twice
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < stages; ++i) {
      tc05::mbar_init(&c.w_full[i], 1);
      tc05::mbar_init(&c.x_full[i], 1);
      tc05::mbar_init(&c.free_[i], kWarps);
    }
    for (int i = 0; i < kTiles; ++i) {
      tc05::mbar_init(&c.tile_full[i], 1);
      tc05::mbar_init(&c.scales_full[i], 1);
      tc05::mbar_init(&c.tile_ready[i], 1);
      tc05::mbar_init(&c.tile_done[i], kWarps);
      tc05::mbar_init(&c.tile_free[i], kWarps + kEnds + 2);
    }
    c.dup = c.dead = 0;
    tc05::fence_barrier_init();
  }
  for (int i = tid; i < every; i += kThreads) count[i] = i < p.experts ? 0 : p.tokens;
  for (int i = tid; i < p.tokens; i += kThreads) x_top[i] = 0;
  __syncthreads();
  prior_done();

  // the tokens of each expert, and the list of jobs: a job is up to TOK tokens of an expert; shared experts first
  int next = 0;  // the first ticket comes while the tokens are looked at
  if (tid == (kWarps + 2) * 32) next = atomicAdd(p.ticket, 1);
  for (int i = tid; i < pairs; i += kThreads) ids[i] = (int16_t)expert_of(p, i);
  if constexpr (S::W8 && !S::X8) {  // pieces of 512 columns to a warp, from the last warp down: the first ones have entries
    const int per = (p.dim + 511) / 512;
    for (int u = kThreads / 32 - 1 - warp; u < p.tokens * per; u += kThreads / 32) {
      const int t = u / per, at = u % per * 512;
      const uint8_t* row = static_cast<const uint8_t*>(p.x) + (long long)t * p.x_row * 2;
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = at + i * 256 + lane * 8;
        if (col >= p.dim) break;
        const uint4 v = *reinterpret_cast<const uint4*>(row + col * 2);
#pragma unroll
        for (uint32_t q : {v.x, v.y, v.z, v.w}) top = max(top, max(q & 0x7fff0000u, q << 16 & 0x7fff0000u));
      }
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) atomicMax(&x_top[t], top);
    }
  }
  __syncthreads();
  for (int i = tid; i < pairs; i += kThreads) {
    const bool again = named_before(ids, p.k, i);
    const int mine = again ? -1 : ids[i];
    if (again) c.dup = 1;
    if (mine >= 0) atomicAdd(&count[mine], 1);
    table[i] = (int16_t)mine;
  }
  if (tid < 8 && pairs + tid < (pairs + 7) / 8 * 8) table[pairs + tid] = -1;
  __syncthreads();
  int base = 0;
  for (int o = 0; o < every; o += kThreads) {
    const int at = o + tid, e = at < p.shared ? p.experts + at : at - p.shared;
    const int parts = at < every ? (count[e] + kTok - 1) / kTok : 0;
    int total;
    const int first = base + block_excl_scan<kThreads>(parts, c.warp_tmp, &total);
    for (int i = 0; i < parts; ++i) jobs[first + i] = e | i << 16;
    base += total;
  }
  __syncthreads();
  const int n_jobs = base;
  const int up_tiles = (p.inner + kR / 2 - 1) / (kR / 2), down_tiles = (p.dim + kR - 1) / kR;
  const int all_up = n_jobs * up_tiles, all = n_jobs * (up_tiles + down_tiles);
  volatile int* dead = &c.dead;

  if (n_jobs == 0) {  // no expert is asked for
    fill_out<kThreads>(p, tid, blockIdx.x, gridDim.x, 0.f);
  } else if (warp == kWarps) {
    // ---- weights
    uint32_t sent = 0;
    int st = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (uint32_t i = 0; ok; ++i) {
      const int ti = i % kTiles;
      if (!moe_wait(&c.tile_full[ti], i / kTiles & 1, p.wait_tries, dead) || c.tile[ti].kind == 2) break;
      const bool up = c.tile[ti].kind == 0;
      const int e = c.tile[ti].expert, row = c.tile[ti].row, cols = up ? p.dim : p.inner;
      __syncwarp();
      if (lane == 0) tc05::mbar_arrive(&c.tile_free[ti]);
      for (int k = 0; k < cols; k += S::KST) {
        if (sent >= (uint32_t)stages && !(ok = moe_wait(&c.free_[st], ph ^ 1, p.wait_tries, dead))) break;
        const int boxes = min(S::BOXES, (cols - k + S::BOXCOLS - 1) / S::BOXCOLS);
        if (lane == 0) {
          uint8_t* to = ring + st * S::STAGE;
          tc05::mbar_expect_tx(&c.w_full[st], boxes * kR * 128);
          for (int b = 0; b < boxes; ++b, to += kR * 128) {
            if (up) {
              load_box(to, &maps.up, k + b * S::BOXCOLS, row, e, &c.w_full[st]);
              load_box(to + kR / 2 * 128, &maps.up, k + b * S::BOXCOLS, p.inner + row, e, &c.w_full[st]);
            } else {
              load_box(to, &maps.down, k + b * S::BOXCOLS, row, e, &c.w_full[st]);
            }
          }
        }
        __syncwarp();
        ++sent;
        if (++st == stages) st = 0, ph ^= 1;
      }
    }
    // nothing is left in flight where a wait ran out
    drain(c.w_full, stages, sent);
  } else if (warp == kWarps + 1) {
    // ---- rows of x and h
    uint32_t sent = 0;
    int st = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (uint32_t i = 0; ok; ++i) {
      const int ti = i % kTiles;
      if (!moe_wait(&c.tile_ready[ti], i / kTiles & 1, p.wait_tries, dead) || c.tile[ti].kind == 2) break;
      const Tile& tile = c.tile[ti];
      const bool up = tile.kind == 0;
      const int n = tile.n, cols = up ? p.dim : p.inner;
      if (!up) asm volatile("fence.proxy.async;\n" ::: "memory");  // h was written by plain stores
      for (int k = 0; k < cols; k += S::KST) {
        if (sent >= (uint32_t)stages && !(ok = moe_wait(&c.free_[st], ph ^ 1, p.wait_tries, dead))) break;
        const uint32_t bytes = min(S::KST, cols - k) * (up ? S::value_bytes(0) : S::value_bytes(1));
        if (lane == 0) tc05::mbar_expect_tx(&c.x_full[st], n * bytes);
        __syncwarp();
        uint8_t* to = ring + st * S::STAGE + S::W_BYTES;
        for (int j = lane; j < n; j += 32) {
          if (up) {
            const uint8_t* from = static_cast<const uint8_t*>(p.x) + ((long long)(tile.slot[j] / slots) * p.x_row + k) * S::value_bytes(0);
            copy_row(to + j * S::row_bytes(0), from, bytes, &c.x_full[st]);
          } else {
            const uint8_t* from = p.h + ((long long)tile.slot[j] * p.inner + k) * S::value_bytes(1);
            copy_row(to + j * S::row_bytes(1), from, bytes, &c.x_full[st]);
          }
        }
        __syncwarp();
        ++sent;
        if (++st == stages) st = 0, ph ^= 1;
      }
      if (lane == 0) tc05::mbar_arrive(&c.tile_free[ti]);
    }
    drain(c.x_full, stages, sent);
  } else if (warp == kWarps + 2) {
    // ---- tickets and what belongs to them, up to kTiles tiles ahead of the products
    // One warp's chain of instructions for every tile, some of which are of one stage: 158 tokens' 5 of 227 experts of
    // 128 x 1,280, 214 MB, take 150 us with the router (with 32 entries looked at in turn 247, with
    // sums over the lanes and whole divisions 161).
    uint32_t told = 0, done = 0;
    int done_from = 0;
    const float per_up = 1.f / up_tiles, per_down = 1.f / down_tiles, per_k = 1.f / p.k, per_slots = 1.f / slots;
    auto token_of = [&](int i) { return __float2int_rz((i + 0.5f) * per_k); };  // of an entry: up to 8,192 over up to 32
    for (uint32_t i = 0;; ++i) {
      const int ti = i % kTiles;
      if (i >= kTiles && !moe_wait(&c.tile_free[ti], (i / kTiles - 1) & 1, p.wait_tries, dead)) break;
      const int ticket = __shfl_sync(0xffffffffu, next, 0);
      Tile& tile = c.tile[ti];
      if (ticket >= all) {
        if (lane == 0) {
          tile.kind = 2;
          tc05::mbar_arrive(&c.tile_full[ti]);
          tc05::mbar_arrive(&c.tile_ready[ti]);
        }
        break;
      }
      if (lane == 0) next = atomicAdd(p.ticket, 1);  // on its way while this one is looked up
      const bool up = ticket < all_up;
      const int left = up ? ticket : ticket - all_up, tiles = up ? up_tiles : down_tiles;
      int job = __float2int_rz((float)left * (up ? per_up : per_down)), of = left - job * tiles;
      if (of < 0) --job, of += tiles;
      if (of >= tiles) ++job, of -= tiles;
      const int listed = jobs[job], e = listed & 0xffff, first = (listed >> 16) * kTok;
      const int row = of * (up ? kR / 2 : kR);
      int n = 0;
      if (e >= p.experts) {
        n = min(kTok, p.tokens - first);
        if (lane < n) tile.slot[lane] = (first + lane) * slots + p.k + e - p.experts;
      } else {
        // the entries of the expert in their order: eight to a lane, then those of the lanes that have some
        int seen = 0;
        for (int q = 0; q < pairs && seen < first + kTok; q += 256) {
          const int i0 = q + lane * 8;
          uint32_t hits = 0;
          if (i0 < pairs) {
            const uint4 v = *reinterpret_cast<const uint4*>(table + i0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) hits |= (uint32_t)((int16_t)w[j] == e) << 2 * j | (uint32_t)((int16_t)(w[j] >> 16) == e) << (2 * j + 1);
          }
          for (uint32_t m = __ballot_sync(0xffffffffu, hits != 0); m && seen < first + kTok; m &= m - 1) {
            const int from = __ffs(m) - 1;
            const uint32_t h = __shfl_sync(0xffffffffu, hits, from);
            const int at = seen - first + __popc(h & lanemask_lt()), i = q + from * 8 + lane;
            if (h >> lane & 1 && at >= 0 && at < kTok) tile.slot[at] = i + token_of(i) * p.shared;
            seen += __popc(h);
          }
        }
        n = min(kTok, seen - first);
      }
      __syncwarp();
      // lane j: token j's weight, or the scale of its x; on its way until the tile is ready
      const int slot = lane < n ? tile.slot[lane] : 0, t = __float2int_rz((slot + 0.5f) * per_slots);
      float weight = 1.f;
      int lift = 0;
      if (lane < n) {
        if (!up) {
          if (slot - t * slots < p.k) weight = weight_of(p, t, slot - t * slots, c.dup);
        } else if constexpr (S::X8) {
          weight = p.x_scale[t];
        } else if constexpr (S::W8) {
          lift = lift_of(x_top[t]);
        }
      }
      if (lane == 0) {
        tile.kind = up ? 0 : 1;
        tile.job = job, tile.expert = e, tile.n = n, tile.row = row;
        if constexpr (S::W8) {  // the rows' scales, both halves' of an up tile
          const int per = up ? kR / 2 : kR, rows = min(per, (up ? p.inner : p.dim) - row);
          const float* from = up ? p.up_scale + (long long)e * 2 * p.inner + row : p.down_scale + (long long)e * p.dim + row;
          tc05::mbar_expect_tx(&c.scales_full[ti], rows * (up ? 8 : 4));
          copy_row(tile.scale, from, rows * 4, &c.scales_full[ti]);
          if (up) copy_row(tile.scale + per, from + p.inner, rows * 4, &c.scales_full[ti]);
        }
        tc05::mbar_arrive(&c.tile_full[ti]);
      }
      if constexpr (S::W8) ++told;
      if (!up) {  // h is there when the job's up tiles are done; 32 jobs are looked at at once, and not again
        const int ahead = job - done_from;
        if (ahead < 0 || ahead >= 32 || !(done >> ahead & 1)) {
          bool ok = true;
          done_from = job;
          for (uint32_t j = 0;; ++j) {
            done = __ballot_sync(0xffffffffu, job + lane < n_jobs && load_acquire(p.up_done + job + lane) >= up_tiles);
            ok = done & 1;
            if (ok || j >= p.wait_tries || __any_sync(0xffffffffu, *dead != 0)) break;
            __nanosleep(100);
          }
          if (!ok) {
            *dead = 1;
            break;
          }
          __syncwarp();
        }
        if constexpr (S::W8)
          if (lane < n) lift = lift_of(__ldcg(p.h_top + slot));
      }
      if (lane < n) {
        tile.weight[lane] = S::W8 ? weight * pow2(-lift) : weight;
        if constexpr (S::W8) tile.lift[lane] = pow2(lift);
      }
      __syncwarp();
      if (lane == 0) tc05::mbar_arrive(&c.tile_ready[ti]);
    }
    drain(c.scales_full, kTiles, told);
  } else if (warp > kWarps + 2) {
    // ---- tiles' ends: the products go on meanwhile, a fence and an atomic take longer than a stage
    for (uint32_t i = 0;; ++i) {
      const int ti = i % kTiles;
      bool ok = moe_wait(&c.tile_full[ti], i / kTiles & 1, p.wait_tries, dead);
      if (part_any<kAtEnds, kEnds * 32>(!ok || *dead) || c.tile[ti].kind == 2) break;
      const int kind = c.tile[ti].kind, row = c.tile[ti].row, job = c.tile[ti].job;
      ok = moe_wait(&c.tile_done[ti], i / kTiles & 1, p.wait_tries, dead);
      if (ok && kind == 0 && tid == (kWarps + 3) * 32) {
        tell(p.up_done + job);  // h is read by copies
      }
      if (kind == 1) {
        if (tid == (kWarps + 3) * 32) {
          c.last = ok && count_on(p.down_done + row / kR) == n_jobs - 1;
        }
        part_sync<kAtEnds, kEnds * 32>();
        if (c.last) {  // all experts' parts of these rows are there
          add_parts<kEnds * 32>(p, tid - (kWarps + 3) * 32, row, kR, 0, p.tokens, slots,
                                [&](int t, int s) { return s >= p.k || table[t * p.k + s] >= 0 ? t * slots + s : -1; });
        }
        part_sync<kAtEnds, kEnds * 32>();
      }
      __syncwarp();
      if (lane == 0) tc05::mbar_arrive(&c.tile_free[ti]);
    }
  } else {
    // ---- products
    int st = 0;
    uint32_t ph = 0;
    const int g = lane >> 2, t = lane & 3;
    for (uint32_t i = 0;; ++i) {
      const int ti = i % kTiles;
      bool ok = moe_wait(&c.tile_full[ti], i / kTiles & 1, p.wait_tries, dead);
      if (part_any<kProducts, kWarps * 32>(!ok || *dead)) break;  // all warps go into a tile, or none: they meet at its barriers
      const Tile& tile = c.tile[ti];
      const int kind = tile.kind;
      if (kind == 2) break;
      const int n = tile.n, cols = kind == 0 ? p.dim : p.inner;
      float acc[kMT][4] = {};
      for (int k = 0; k < cols; k += S::KST) {
        ok = moe_wait(&c.w_full[st], ph, &c.x_full[st], ph, p.wait_tries, dead);
        if (!ok) break;
        const uint8_t* w = ring + st * S::STAGE;
        if (kind == 0) stage_products<S, 0>(w, w + S::W_BYTES, min(S::KST, cols - k), tile, warp, lane, acc);
        else stage_products<S, 1>(w, w + S::W_BYTES, min(S::KST, cols - k), tile, warp, lane, acc);
        __syncwarp();
        if (lane == 0) tc05::mbar_arrive(&c.free_[st]);
        if (++st == stages) st = 0, ph ^= 1;
      }
      if (S::W8 && ok) ok = moe_wait(&c.scales_full[ti], i / kTiles & 1, p.wait_tries, dead);
      // a warp that gave up goes on through the tile's barriers with the others; what it adds is not written
      // (all warps have read what was there: they have met at this tile's beginning)
      float* mine = red + (warp % kKW * kR + warp / kKW * (kMT * 16) + g) * kRedRow + 2 * t;
#pragma unroll
      for (int m = 0; m < kMT; ++m) {
        *reinterpret_cast<float2*>(mine + m * 16 * kRedRow) = make_float2(acc[m][0], acc[m][1]);
        *reinterpret_cast<float2*>(mine + (m * 16 + 8) * kRedRow) = make_float2(acc[m][2], acc[m][3]);
      }
      part_sync<kProducts, kWarps * 32>();
      auto sum = [&](int r, int col) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kKW; ++w) v += red[(w * kR + r) * kRedRow + col];
        return v;
      };
      if (!*dead) {
        if (kind == 0) {  // a warp's 32 values are of one token
          const int r = lane, col = warp, f = tile.row + r;
          if (col < n) {
            const int slot = tile.slot[col];
            float gate = sum(r, col), up = sum(r + kR / 2, col);
            if constexpr (S::W8 || S::X8) gate *= tile.weight[col], up *= tile.weight[col];
            if constexpr (S::W8) gate *= tile.scale[r], up *= tile.scale[r + kR / 2];
            const float h = gated(gate, up, p.limit);
            const bool in = f < p.inner;
            if (in) reinterpret_cast<float*>(p.h)[(long long)slot * p.inner + f] = h;
            if constexpr (S::W8) {
              const uint32_t top = __reduce_max_sync(0xffffffffu, in ? __float_as_uint(h) & 0x7fffffffu : 0u);
              if (lane == 0) atomicMax(p.h_top + slot, top);
            }
          }
        } else {
          const int r = tid % kR, col = tid / kR, d = tile.row + r;
          if (col < n && d < p.dim) {
            float v = sum(r, col) * tile.weight[col];
            if constexpr (S::W8) v *= tile.scale[r];
            p.part[(long long)tile.slot[col] * p.dim + d] = v;
          }
        }
      }
      __syncwarp();
      if (lane == 0 && !*dead) {
        tc05::mbar_arrive(&c.tile_done[ti]);
        tc05::mbar_arrive(&c.tile_free[ti]);
      }
    }
  }
  __syncthreads();
  // the block that leaves last leaves the counters as it found them, and no output that could pass for one after a time-out
  if (tid == 0) c.last = leave(p, c.dead);
  __syncthreads();
  if (c.last) {
    if (c.last == 2) fill_out<kThreads>(p, tid, 0, 1, __int_as_float(0x7fc00000));
    for (int i = tid; i < n_jobs; i += kThreads) p.up_done[i] = 0;
    for (int i = tid; i < down_tiles; i += kThreads) p.down_done[i] = 0;
    if constexpr (S::W8)
      for (int i = tid; i < p.tokens * slots; i += kThreads) p.h_top[i] = 0;
    if (tid == 0) *p.ticket = 0, *p.left = 0;
  }
}

template <class S>
cudaError_t launch(const MoeParams& p, cudaStream_t stream) {
  MoeMaps maps;
  const uint64_t every = p.experts + p.shared;
  if (!make_expert_map(&maps.up, p.up, S::W8, p.dim, 2ull * p.inner, every, kR / 2) ||
      !make_expert_map(&maps.down, p.down, S::W8, p.inner, p.dim, every, kR))
    return cudaErrorNotSupported;
  constexpr int kMostSmem = 227 * 1024;
  const int fixed = kRed + (int)sizeof(Control) + 4 * p.most_jobs + 4 * (int)every + 4 * p.tokens + 4 * p.tokens * p.k + 64;
  int stages = (kMostSmem - fixed) / S::STAGE;
  if (stages > kMaxStages) stages = kMaxStages;
  if (stages < 2) return cudaErrorInvalidConfiguration;
  const cudaError_t e = allow_smem<moe_kernel<S>>(kMostSmem);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)p.most_jobs * ((p.inner + kR / 2 - 1) / (kR / 2) + (p.dim + kR - 1) / kR);
  int blocks = device_sm_count();
  if (tiles < blocks) blocks = (int)tiles;
  if (blocks < 1) blocks = 1;
  return launch_behind(moe_kernel<S>, dim3(blocks), kThreads, (size_t)stages * S::STAGE + fixed, stream, maps, p, stages);
}

}  // namespace

MoeTiles moe_tiles() { return {kR, kTok}; }

cudaError_t launch_moe(const MoeParams& p, bool w8, bool x8, cudaStream_t stream) {
  if (w8) return x8 ? launch<Shape<true, true>>(p, stream) : launch<Shape<true, false>>(p, stream);
  return x8 ? launch<Shape<false, true>>(p, stream) : launch<Shape<false, false>>(p, stream);
}

}  // namespace csa2
