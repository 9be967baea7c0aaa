// C ABI of the paged 8-bit cache (include/csa2.h): validation and launches of the page plan, the
// rotary axes, the page writer and the paged attention.
#include <cmath>
#include <cstring>

#include "kernels.h"
#include "paged.h"

namespace csa2 {

int device_sm_count();

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align_up(size_t v) { return (v + 255) / 256 * 256; }
csa2_status cuda_status(cudaError_t e) { return e == cudaSuccess ? CSA2_OK : CSA2_ECUDA; }
bool type_ok(int32_t t) { return t >= CSA2_T_BF16 && t <= CSA2_T_F32; }
int type_size(int32_t t) { return t == CSA2_T_F32 ? 4 : 2; }
bool stride_ok(int64_t row, int64_t head, int32_t t) { return row % (16 / type_size(t)) == 0 && head % (16 / type_size(t)) == 0; }
int page_shift(int32_t page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : 0; }

// Turns per position of each pair, times 2^64, whole turns left out: theta^(-2i/R) / (2 pi).  A double's 53 bits
// would be off by 2^-56 of a turn per position; long double (113 bits on Arm, 64 on x86) keeps 2^-64, as powers of one
// root, whose errors of i roundings the powers' decay outruns.  A model calls with one theta and R, or some by turns,
// so the thread's last tables are kept (a table takes longer than a launch).
const uint64_t* rope_turns(float theta, int rot_dim) {
  struct Table {
    float theta;
    int rot_dim;
    uint64_t turns[CSA2_ROPE_AXES_MAX_PAIRS];
  };
  thread_local Table kept[4] = {};
  thread_local int next = 0;
  for (const Table& k : kept)
    if (k.theta == theta && k.rot_dim == rot_dim) return k.turns;
  Table& k = kept[next];
  next = (next + 1) % 4;
  const long double root = std::pow((long double)theta, -2.0L / rot_dim);
  long double t = 1.0L / 6.283185307179586476925286766559005768L;
  for (int i = 0; i < rot_dim / 2; ++i, t *= root) {
    const long double units = std::rint(std::ldexp(t - std::floor(t), 64));
    k.turns[i] = units < 18446744073709551616.0L ? (uint64_t)units : 0;
  }
  k.theta = theta, k.rot_dim = rot_dim;
  return k.turns;
}

// Which kernel, and its workspace, by the query rows per sequence and kv head in the mean (the host knows no more).
//   up to 8      of single tokens (no more rows than sequences): paged_attn.cu's tiles of 8, three blocks per SM
//                (four at dim 64).  Drafts, which may be ragged, take the tiles below from 2 tokens on: 64 sequences
//                of 4,096 tokens, 8 heads of groups of 4, dim 128 / 64: 2 tokens each 97 / 60 us against 91 / 53
//                by tiles of 8, but 3 and 1 by turns 98 / 61 against 130 / 69, 4 and 0 59 / 37 against 64 / 50
//   up to 32     at dim 64 its tiles of 16 (64 sequences x 4 heads x 1,000 tokens, 16 / 32 rows: 18 / 26 us against
//                30 / 48 by paged_rows.cu's form; 32 sequences x 16,000 tokens and 32 rows 102 against 139);
//                at dim 128 paged_rows.cu's tiles of 16 (two blocks per SM) or 32 (one): 8 heads of 16 rows x 16
//                sequences x 65,535 tokens 326 us against 354 by tiles of 16 of paged_attn.cu (two blocks per SM
//                there), one head x 4 sequences x 1M tokens in fp16 180 against 232; short contexts lose by it
//                (64 sequences of 1,000 tokens 47 against 43) and stay here, as one form less.  (The other sides
//                are from when both were there.)
//   more         paged_wide.cu's tiles of 256, one block per SM (dim 64, 64 rows, the second case: 154 us)
// A batch that mixes a prompt chunk with decodes takes one form for all, which the mean makes wrong for some: 255
// sequences of 4,096 tokens and a chunk of 512 behind 32,768, 8 heads of groups of 8, dim 128: 2,100 us together,
// 330 and 497 in two calls.  Sequences without rows lower the mean too (the chunk with 200 of them: 1,650 us).
// No more blocks than there can be units of 128 tokens (a tile has at most the table's, a sequence one tile
// more than its rows fill).
struct AttnPlan {
  int rows;  // of a tile
  int blocks;
  bool few_pieces;
  size_t part_o, part_ml, open, bytes;
};
AttnPlan attn_plan(const csa2_paged_attn_args* a) {
  AttnPlan pl{};
  const long long group = a->heads / a->kv_heads, rows = a->n_rows * group;
  pl.rows = rows <= 8LL * a->n_seq && a->n_rows <= a->n_seq                ? 8
            : rows <= (a->head_dim == 64 ? 32LL : 16LL) * a->n_seq         ? 16
            : rows <= 32LL * a->n_seq                                      ? 32
                                                                           : 256;
  if (pl.rows == 256 && a->n_seq > 16384) pl.rows = a->head_dim == 64 ? 16 : 32;  // its sequences' tiles fit shared memory
  const long long tiles = (rows + pl.rows - 1) / pl.rows + a->n_seq;
  const long long units = ((long long)a->table_cols * a->page_size + 127) / 128 + 1;
  const long long most = (pl.rows == 256 ? 1 : pl.rows == 8 ? (a->head_dim == 64 ? 4 : 3) : a->head_dim == 64 ? 3 : pl.rows == 16 ? 2 : 1) * device_sm_count();
  const double all = (double)tiles * a->kv_heads * units;
  pl.blocks = all < (double)most ? (int)all : (int)most;
  pl.few_pieces = tiles * a->kv_heads * 4 >= pl.blocks;
  size_t at = 0;
  const size_t slots = 2 * (size_t)pl.blocks * pl.rows;
  pl.part_o = at, at += align_up(slots * a->head_dim * 4);
  pl.part_ml = at, at += align_up(slots * 8);
  pl.open = at, at += align_up((size_t)pl.blocks * sizeof(PagedOpen));
  pl.bytes = at;
  return pl;
}

csa2_status check_attn_sizes(const csa2_paged_attn_args* a) {
  if (!a || a->n_rows < 0 || a->n_seq < 0 || a->heads < 1 || a->kv_heads < 1 || a->heads % a->kv_heads ||
      a->n_pages < 0 || a->table_cols < 0)
    return CSA2_EINVAL;
  if ((a->head_dim != 64 && a->head_dim != 128) || !page_shift(a->page_size)) return CSA2_EUNSUPPORTED;
  if ((long long)a->n_rows * (a->heads / a->kv_heads) > 0x7fffffffLL - 1024 ||
      (long long)a->table_cols * a->page_size > kPagedMostTokens ||
      (long long)a->n_pages * a->kv_heads > 0x7fffffffLL)
    return CSA2_EUNSUPPORTED;
  return CSA2_OK;
}

}  // namespace
}  // namespace csa2

using namespace csa2;

extern "C" {

csa2_status csa2_page_plan(const csa2_page_plan_args* a, void* stream) {
  if (!a || a->n_seq < 0 || a->max_rows < 0 || a->n_free < 0 || a->page_size < 1 || a->page_size > 65536 ||
      a->table_cols < 1)
    return CSA2_EINVAL;
  if (a->n_seq > 8192 || a->max_rows > 0x7fffffff - (1 << 20)) return CSA2_EUNSUPPORTED;
  if (!a->row_start || !a->n_taken || (a->n_seq > 0 && (!a->ctx_len || !a->new_len || !a->table || !a->kv_len)) ||
      (a->n_free > 0 && !a->free_pages) || (a->max_rows > 0 && (!a->seq_of_row || !a->pos || !a->slot)))
    return CSA2_EINVAL;
  if (!aligned(a->seq_of_row, 16) || !aligned(a->pos, 16) || !aligned(a->slot, 16)) return CSA2_EINVAL;
  PagePlanParams p{};
  p.ctx_len = a->ctx_len;
  p.new_len = a->new_len;
  p.n_seq = a->n_seq;
  p.page_size = a->page_size;
  p.table = a->table;
  p.table_cols = a->table_cols;
  p.free_pages = a->free_pages;
  p.n_free = a->n_free;
  p.max_rows = a->max_rows;
  p.row_start = a->row_start;
  p.kv_len = a->kv_len;
  p.seq_of_row = a->seq_of_row;
  p.pos = a->pos;
  p.slot = a->slot;
  p.n_taken = a->n_taken;
  p.dev_status = a->dev_status;
  return cuda_status(launch_page_plan(p, static_cast<cudaStream_t>(stream)));
}

csa2_status csa2_rope_axes(const csa2_rope_axes_args* a, void* stream) {
  if (!a || a->n_tokens < 0 || a->n_heads < 1 || a->head_dim < 8 || a->head_dim % 8 || !type_ok(a->dtype) ||
      a->n_axes < 1 || a->n_axes > 16 || a->rot_first < 0 || a->rot_first % 8 || a->rot_dim < 16 || a->rot_dim % 16 ||
      a->rot_first + (long long)a->rot_dim > a->head_dim || !(a->theta > 0.f) || !std::isfinite(a->theta))
    return CSA2_EINVAL;
  if (a->head_dim > 4096 || a->rot_dim > 2 * CSA2_ROPE_AXES_MAX_PAIRS) return CSA2_EUNSUPPORTED;
  for (int i = 0; i < a->rot_dim / 2; ++i)
    if (a->axis_of_pair[i] >= a->n_axes) return CSA2_EINVAL;
  if (a->n_tokens == 0) return CSA2_OK;
  if (!a->x || !a->out || !a->pos || !aligned(a->x, 16) || !aligned(a->out, 16) || !aligned(a->pos, 8) ||
      !stride_ok(a->x_row, a->x_head, a->dtype) || !stride_ok(a->out_row, a->out_head, a->dtype))
    return CSA2_EINVAL;
  if (a->x == a->out && (a->x_row != a->out_row || a->x_head != a->out_head)) return CSA2_EINVAL;
  if ((long long)a->n_tokens * (a->head_dim / 4) > (1LL << 38)) return CSA2_EUNSUPPORTED;
  RopeAxesParams p{};
  p.x = a->x;
  p.out = a->out;
  p.x_row = a->x_row, p.x_head = a->x_head, p.out_row = a->out_row, p.out_head = a->out_head;
  p.n_tokens = a->n_tokens, p.n_heads = a->n_heads, p.head_dim = a->head_dim;
  p.rot_first = a->rot_first, p.rot_dim = a->rot_dim;
  p.copy_rest = a->x != a->out;
  p.pos = a->pos;
  std::memcpy(p.turns, rope_turns(a->theta, a->rot_dim), a->rot_dim / 2 * sizeof(uint64_t));
  std::memcpy(p.axis, a->axis_of_pair, a->rot_dim / 2);
  return cuda_status(launch_rope_axes(p, a->dtype, a->half_pairs != 0, a->inverse != 0, static_cast<cudaStream_t>(stream)));
}

csa2_status csa2_write_pages(const csa2_write_pages_args* a, void* stream) {
  if (!a || a->n_rows < 0 || a->n_seq < 0 || a->kv_heads < 1 || !type_ok(a->dtype) || a->n_pages < 0 ||
      a->table_cols < 0)
    return CSA2_EINVAL;
  if ((a->head_dim != 64 && a->head_dim != 128) || !page_shift(a->page_size) || a->kv_heads > 65535)
    return CSA2_EUNSUPPORTED;
  if (a->n_rows == 0 || a->n_seq == 0) return CSA2_OK;
  if (!a->k || !a->v || !a->row_start || !a->kv_len || !a->seq_of_row || (a->table_cols > 0 && !a->table) ||
      (a->n_pages > 0 && (!a->k_codes || !a->v_codes || !a->k_scale || !a->v_scale)))
    return CSA2_EINVAL;
  if (!aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->k_codes, 16) || !aligned(a->v_codes, 16) ||
      !stride_ok(a->k_row, a->k_head, a->dtype) || !stride_ok(a->v_row, a->v_head, a->dtype))
    return CSA2_EINVAL;
  PageWriteParams p{};
  p.x[0] = a->k, p.x[1] = a->v;
  p.x_row[0] = a->k_row, p.x_row[1] = a->v_row;
  p.x_head[0] = a->k_head, p.x_head[1] = a->v_head;
  p.codes[0] = a->k_codes, p.codes[1] = a->v_codes;
  p.scale[0] = a->k_scale, p.scale[1] = a->v_scale;
  p.n_rows = a->n_rows, p.n_seq = a->n_seq, p.kv_heads = a->kv_heads;
  p.page_shift = page_shift(a->page_size);
  p.n_pages = a->n_pages, p.table_cols = a->table_cols;
  p.row_start = a->row_start, p.kv_len = a->kv_len, p.seq_of_row = a->seq_of_row, p.table = a->table;
  // 64 rows (or a page of 128) per block where sequences bring pages: eight tasks of 16 rows, or two of 64,
  // for its eight warps; four rows where they bring a token or two
  p.chunk = a->n_rows >= 4LL * a->n_seq ? (a->page_size > 64 ? a->page_size : 64) : 4;
  p.dev_status = a->dev_status;
  return cuda_status(launch_page_write(p, a->dtype, a->head_dim, static_cast<cudaStream_t>(stream)));
}

size_t csa2_paged_attn_workspace_size(const csa2_paged_attn_args* a) {
  if (check_attn_sizes(a) != CSA2_OK || a->n_rows == 0 || a->n_seq == 0) return 0;
  return attn_plan(a).bytes;
}

static csa2_status paged_attn(const csa2_paged_attn_args* a, uint32_t wait_tries, void* stream) {
  const csa2_status st = check_attn_sizes(a);
  if (st != CSA2_OK) return st;
  if (!type_ok(a->q_dtype) || a->q_dtype == CSA2_T_F32 || !type_ok(a->out_dtype) || a->window < 0 ||
      !std::isfinite(a->softmax_scale))
    return CSA2_EINVAL;
  if (a->n_rows == 0 || a->n_seq == 0) return CSA2_OK;
  if (!a->q || !a->out || !a->row_start || !a->kv_len || (a->table_cols > 0 && !a->table) ||
      (a->table_cols > 0 && a->n_pages > 0 && (!a->k_codes || !a->v_codes || !a->k_scale || !a->v_scale)))
    return CSA2_EINVAL;
  if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->k_codes, 16) || !aligned(a->v_codes, 16) ||
      !stride_ok(a->q_row, a->q_head, a->q_dtype))
    return CSA2_EINVAL;
  const AttnPlan pl = attn_plan(a);
  if (!a->workspace || a->workspace_bytes < pl.bytes || !aligned(a->workspace, 16)) return CSA2_EWORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  PagedAttnParams p{};
  p.q = a->q, p.q_row = a->q_row, p.q_head = a->q_head;
  p.n_rows = a->n_rows, p.n_seq = a->n_seq, p.kv_heads = a->kv_heads, p.group = a->heads / a->kv_heads;
  p.group_inv = p.group == 1 ? 0 : ~0ull / p.group + 1;
  p.row_start = a->row_start, p.kv_len = a->kv_len, p.table = a->table;
  p.table_cols = a->table_cols, p.n_pages = a->n_pages, p.page_shift = page_shift(a->page_size);
  p.k = a->k_codes, p.v = a->v_codes, p.k_scale = a->k_scale, p.v_scale = a->v_scale;
  // without pages, copies of no bytes still name an address
  if (!p.k_scale || !p.v_scale) p.k_scale = p.v_scale = reinterpret_cast<const float*>(ws);
  p.scale_log2 = a->softmax_scale * 1.4426950408889634f;
  p.window = a->window, p.sink = a->sink;
  p.out = a->out, p.out_dtype = a->out_dtype;
  p.part_o = reinterpret_cast<float*>(ws + pl.part_o);
  p.part_ml = reinterpret_cast<float*>(ws + pl.part_ml);
  p.open = reinterpret_cast<PagedOpen*>(ws + pl.open);
  p.few_pieces = pl.few_pieces;
  p.wait_tries = wait_tries;
  p.dev_status = a->dev_status;
  cudaStream_t on = static_cast<cudaStream_t>(stream);
  return cuda_status(pl.rows == 256                        ? launch_paged_wide(p, a->q_dtype, a->head_dim, pl.blocks, on)
                     : a->head_dim == 128 && pl.rows > 8 ? launch_paged_rows(p, a->q_dtype, pl.rows, pl.blocks, on)
                                                         : launch_paged_attn(p, a->q_dtype, a->head_dim, pl.rows, pl.blocks, on));
}

csa2_status csa2_paged_attn(const csa2_paged_attn_args* a, void* stream) { return paged_attn(a, kPagedTries, stream); }

csa2_status csa2_selftest_paged_waits(const csa2_paged_attn_args* a, int32_t tries, void* stream) {
  if (!a || !a->dev_status || tries < 0 || tries > (1 << 20)) return CSA2_EINVAL;
  return paged_attn(a, (uint32_t)tries, stream);
}

}  // extern "C"
