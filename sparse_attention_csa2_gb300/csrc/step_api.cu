// C ABI of the kernels that follow attention in a decode step (include/csa2.h): validation and launches of the norm
// with residual, the router, the experts and the token sampling.
#include <array>
#include <cmath>
#include <cstring>

#include "kernels.h"
#include "step.h"

namespace csa2 {

int device_sm_count();

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
csa2_status cuda_status(cudaError_t e) { return e == cudaSuccess ? CSA2_OK : CSA2_ECUDA; }
bool type_ok(int32_t t) { return t >= CSA2_T_BF16 && t <= CSA2_T_F32; }
int type_size(int32_t t) { return t == CSA2_T_F32 ? 4 : 2; }

size_t align_up(size_t v) { return (v + 255) / 256 * 256; }

csa2_status check_route_sizes(const csa2_route_args* a) {
  if (!a || a->tokens < 0 || a->dim < 8 || a->dim % 8 || a->experts < 1 || a->k < 1 || a->k > a->experts) return CSA2_EINVAL;
  if (a->tokens > kRouteMostTokens || a->experts > kRouteMostExperts || a->k > kRouteMostK) return CSA2_EUNSUPPORTED;
  return CSA2_OK;
}

// Which form, and its workspace.
struct MoePlan {
  bool many;
  int most_jobs, down_tiles;
  size_t h, part, x_rows, bytes;
};
MoePlan moe_plan(const csa2_moe_args* a) {
  MoePlan pl{};
  const long long pairs = (long long)a->tokens * a->k;
  // The few tokens' form reads (from L2) and converts the weights again for every 8 tokens of an expert, in tiles of 64 rows, the
  // other begins some 6 us later and has less room for 8-bit ones.  In us, that form and the other,
  // at t tokens per expert in the mean:
  //   8 experts of 4,096 x 4,096, bf16:  t = 4  124  142,  8  155  149,  12  202  151,  24  342  154
  //   the same in 8 bits:                t = 8   96  183,  16  160  184,  24  215  184
  //   64 of 4,096 x 2,048, 8 bits:       t = 12  514  609,  18  721  620
  // and at n tiles per SM of the few tokens' form, where t is large (two experts of 1,024 x 512 in bf16, from 3.6 on):
  //   n = 1.1  15  21,  2.7  21  26,  3.6  21  26,  4.0  23  27,  4.4  25  27,  5.3  27  27,  6.9  36  27,  21  159  37
  const long long met = pairs < a->experts ? pairs : a->experts;
  const double tiles = ((pairs + 4 * met) / 8.0 + a->n_shared * ((a->tokens + 7) / 8)) * ((a->inner + 31) / 32 + (a->dim + 63) / 64);
  pl.many = a->form != CSA2_MOE_AUTO ? a->form == CSA2_MOE_MANY : pairs > (a->w_codes ? 16LL : 6LL) * a->experts && tiles > 4.0 * device_sm_count();
  const MoeTiles t = pl.many ? moe_wide_tiles() : moe_tiles();
  pl.most_jobs = (int)(met + pairs / t.tokens + (long long)a->n_shared * ((a->tokens + t.tokens - 1) / t.tokens));
  pl.down_tiles = (a->dim + t.rows - 1) / t.rows;
  const size_t slots = (size_t)a->tokens * (a->k + a->n_shared);
  size_t at = CSA2_COUNTER_BYTES;
  pl.h = at, at += align_up(slots * 4 * a->inner);
  pl.part = at, at += align_up(slots * a->dim * 4);
  if (pl.many) pl.x_rows = at, at += align_up(slots * a->dim * 2);
  pl.bytes = at;
  return pl;
}
csa2_status check_moe_sizes(const csa2_moe_args* a) {
  if (!a || a->form < CSA2_MOE_AUTO || a->form > CSA2_MOE_MANY) return CSA2_EINVAL;
  if (a->tokens < 0 || a->k < 1 || a->experts < 1 || a->n_shared < 0 || a->dim < 16 || a->dim % 16 || a->inner < 16 || a->inner % 16)
    return CSA2_EINVAL;
  if (a->tokens > 512 || a->k > 32 || (long long)a->tokens * a->k > 8192 || a->experts > 1024 || a->n_shared > 8 || a->dim > 32768 ||
      a->inner > 32768)
    return CSA2_EUNSUPPORTED;
  return CSA2_OK;
}

csa2_status moe(const csa2_moe_args* a, uint32_t wait_tries, void* stream) {
  const csa2_status st = check_moe_sizes(a);
  if (st != CSA2_OK) return st;
  if ((a->out_dtype != CSA2_T_BF16 && a->out_dtype != CSA2_T_F32) || !(a->limit > 0.f)) return CSA2_EINVAL;
  if (a->tokens == 0) return CSA2_OK;
  if (!a->x || !a->ids || !a->weights || !a->up || !a->down || !a->out || (a->x_codes && !a->x_scale) ||
      (a->w_codes && (!a->up_scale || !a->down_scale)))
    return CSA2_EINVAL;
  if (!aligned(a->x, 16) || !aligned(a->up, 16) || !aligned(a->down, 16) || !aligned(a->up_scale, 16) ||
      !aligned(a->down_scale, 16) || !aligned(a->out, type_size(a->out_dtype)) ||
      (a->tokens > 1 && (a->x_row % (a->x_codes ? 16 : 8) || a->out_row < a->dim)))
    return CSA2_EINVAL;
  const MoePlan pl = moe_plan(a);
  if (!a->workspace || a->workspace_bytes < pl.bytes || !aligned(a->workspace, 256)) return CSA2_EWORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  MoeParams p{};
  p.x = a->x, p.x_row = a->x_row, p.x_scale = a->x_scale;
  p.ids = a->ids, p.weights = a->weights;
  p.up = a->up, p.down = a->down, p.up_scale = a->up_scale, p.down_scale = a->down_scale;
  p.tokens = a->tokens, p.k = a->k, p.experts = a->experts, p.shared = a->n_shared, p.dim = a->dim, p.inner = a->inner;
  p.limit = a->limit;
  p.out = a->out, p.out_row = a->out_row, p.out_dtype = a->out_dtype;
  p.h = ws + pl.h;
  p.part = reinterpret_cast<float*>(ws + pl.part);
  int* counters = reinterpret_cast<int*>(ws);
  p.ticket = counters, p.left = counters + 1, p.gathered = counters + 2;
  p.down_done = counters + 3;
  p.up_done = p.down_done + pl.down_tiles;
  p.h_top = reinterpret_cast<uint32_t*>(p.up_done + pl.most_jobs);
  p.most_jobs = pl.most_jobs;
  p.x_rows = pl.many ? ws + pl.x_rows : nullptr;
  p.wait_tries = wait_tries;
  p.dev_status = a->dev_status;
  cudaStream_t on = static_cast<cudaStream_t>(stream);
  return cuda_status(pl.many ? launch_moe_wide(p, a->w_codes != 0, a->x_codes != 0, on) : launch_moe(p, a->w_codes != 0, a->x_codes != 0, on));
}

}  // namespace
}  // namespace csa2

using namespace csa2;

extern "C" {

csa2_status csa2_add_norm(const csa2_add_norm_args* a, void* stream) {
  if (!a || a->n_rows < 0 || a->dim < 1 || !type_ok(a->x_dtype) || !type_ok(a->out_dtype) || !type_ok(a->gain_dtype) ||
      !(a->eps >= 0.f) || !std::isfinite(a->eps) || !std::isfinite(a->gain_offset))
    return CSA2_EINVAL;
  const bool sum = a->residual != nullptr;
  if (sum != (a->sum != nullptr) || (sum && a->sum_dtype != a->x_dtype && a->sum_dtype != CSA2_T_F32)) return CSA2_EINVAL;
  const int g = a->group;
  if (g != 0 && ((g != 16 && g != 32 && g != 64 && g != 128 && g != 256) || a->dim % g)) return CSA2_EINVAL;
  if ((a->codes != nullptr) != (a->scales != nullptr)) return CSA2_EINVAL;
  if (a->n_rows == 0) return CSA2_OK;
  if (!a->x || (!a->out && !a->codes && !a->sum)) return CSA2_EINVAL;
  if (!aligned(a->scales, 4)) return CSA2_EINVAL;
  // an array's rows: in place, apart from one another where they are written
  bool vectors = a->dim % 8 == 0 && aligned(a->codes, 8);
  auto rows = [&](const void* p, int64_t row, int32_t type, bool written) {
    if (p == nullptr) return true;
    if (!aligned(p, type_size(type)) || (written && a->n_rows > 1 && row < a->dim)) return false;
    if (!aligned(p, 16) || (a->n_rows > 1 && row % 8)) vectors = false;
    return true;
  };
  if (!rows(a->x, a->x_row, a->x_dtype, false) || !rows(a->residual, a->residual_row, a->sum_dtype, false) ||
      !rows(a->sum, a->sum_row, a->sum_dtype, true) || !rows(a->out, a->out_row, a->out_dtype, true) ||
      !rows(a->gain, 0, a->gain_dtype, false))
    return CSA2_EINVAL;
  // in place means the same place: a block writes its row when it has read it, not the others'
  auto same = [&](const void* p, int64_t prow, int32_t ptype, const void* q, int64_t qrow, int32_t qtype) {
    return p == nullptr || p != q || (type_size(ptype) == type_size(qtype) && (a->n_rows == 1 || prow == qrow));
  };
  if (!same(a->sum, a->sum_row, a->sum_dtype, a->residual, a->residual_row, a->sum_dtype) ||
      !same(a->sum, a->sum_row, a->sum_dtype, a->x, a->x_row, a->x_dtype) ||
      !same(a->out, a->out_row, a->out_dtype, a->x, a->x_row, a->x_dtype) ||
      !same(a->out, a->out_row, a->out_dtype, a->residual, a->residual_row, a->sum_dtype) || (a->out && a->out == a->sum))
    return CSA2_EINVAL;
  if (a->dim > (vectors ? 32768 : 8192)) return CSA2_EUNSUPPORTED;
  AddNormParams p{};
  p.x = a->x, p.residual = a->residual, p.sum = a->sum, p.gain = a->gain, p.out = a->out;
  p.codes = a->codes, p.scales = a->scales;
  p.x_row = a->x_row, p.residual_row = a->residual_row, p.sum_row = a->sum_row, p.out_row = a->out_row;
  p.n_rows = a->n_rows, p.dim = a->dim;
  p.gain_dtype = a->gain_dtype, p.out_dtype = a->out_dtype;
  p.group = g;
  p.eps = a->eps, p.gain_offset = a->gain_offset;
  return cuda_status(launch_add_norm(p, a->x_dtype, sum ? a->sum_dtype : -1, vectors, static_cast<cudaStream_t>(stream)));
}

size_t csa2_route_workspace_size(const csa2_route_args* a) {
  if (check_route_sizes(a) != CSA2_OK || a->tokens == 0) return 0;
  return CSA2_COUNTER_BYTES + (size_t)a->tokens * a->experts * sizeof(float4);
}

csa2_status csa2_route(const csa2_route_args* a, void* stream) {
  const csa2_status st = check_route_sizes(a);
  if (st != CSA2_OK) return st;
  if (!type_ok(a->x_dtype) || (a->w_dtype != a->x_dtype && a->w_dtype != CSA2_T_F32) || a->score < CSA2_SCORE_SOFTMAX ||
      a->score > CSA2_SCORE_SQRTSOFTPLUS || !std::isfinite(a->scale))
    return CSA2_EINVAL;
  if (a->tokens == 0) return CSA2_OK;
  if (!a->x || !a->w || !a->ids || !a->weights || !aligned(a->x, 16) || !aligned(a->w, 16) ||
      (a->tokens > 1 && a->x_row % (16 / type_size(a->x_dtype))))
    return CSA2_EINVAL;
  if (!a->workspace || a->workspace_bytes < csa2_route_workspace_size(a) || !aligned(a->workspace, 16)) return CSA2_EWORKSPACE;
  RouteParams p{};
  p.x = a->x, p.x_row = a->x_row, p.w = a->w, p.bias = a->bias;
  p.tokens = a->tokens, p.dim = a->dim, p.experts = a->experts, p.k = a->k;
  p.score = a->score, p.normalize = a->normalize != 0, p.scale = a->scale;
  p.ids = a->ids, p.weights = a->weights;
  p.done = static_cast<int*>(a->workspace);
  p.z = reinterpret_cast<float4*>(static_cast<uint8_t*>(a->workspace) + CSA2_COUNTER_BYTES);
  return cuda_status(launch_route(p, a->x_dtype, a->w_dtype, static_cast<cudaStream_t>(stream)));
}

size_t csa2_moe_workspace_size(const csa2_moe_args* a) {
  if (check_moe_sizes(a) != CSA2_OK || a->tokens == 0) return 0;
  return moe_plan(a).bytes;
}

csa2_status csa2_moe(const csa2_moe_args* a, void* stream) { return moe(a, kPagedTries, stream); }

csa2_status csa2_selftest_moe_waits(const csa2_moe_args* a, int32_t tries, void* stream) {
  if (!a || !a->dev_status || tries < 0 || tries > (1 << 20)) return CSA2_EINVAL;
  return moe(a, (uint32_t)tries, stream);
}

csa2_status csa2_capture_id(void* stream, uint64_t* id) {
  if (!id) return CSA2_EINVAL;
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  unsigned long long of = 0;
  const cudaError_t e = cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &status, &of);
  *id = e == cudaSuccess && status != cudaStreamCaptureStatusNone ? of : 0;
  return cuda_status(e);
}

csa2_status csa2_event_done(void* event, int32_t wait, int32_t* done) {
  if (!event || !done) return CSA2_EINVAL;
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // other work's event is no matter of a capture, which stays valid
  cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
  if (e != cudaSuccess) return cuda_status(e);
  e = wait ? cudaEventSynchronize(static_cast<cudaEvent_t>(event)) : cudaEventQuery(static_cast<cudaEvent_t>(event));
  const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
  *done = e == cudaSuccess;
  return cuda_status(e != cudaSuccess && e != cudaErrorNotReady ? e : back);
}

csa2_status csa2_sample(const csa2_sample_args* a, void* stream) {
  if (!a || a->n_rows < 0 || a->vocab < 1 || !type_ok(a->dtype)) return CSA2_EINVAL;
  if (a->vocab > kSampleMostVocab || a->n_rows > (1 << 26)) return CSA2_EUNSUPPORTED;
  if (a->n_rows == 0) return CSA2_OK;
  if (!a->logits || !aligned(a->logits, type_size(a->dtype)) || !a->u || !a->token || !aligned(a->token, 8)) return CSA2_EINVAL;
  for (const void* q : {(const void*)a->u, (const void*)a->temperature, (const void*)a->top_k, (const void*)a->top_p,
                        (const void*)a->min_p, (const void*)a->logprob})
    if (!aligned(q, 4)) return CSA2_EINVAL;
  SampleParams p{};
  p.logits = a->logits, p.row = a->row;
  p.rows = a->n_rows, p.vocab = a->vocab;
  p.u = a->u, p.temperature = a->temperature, p.top_k = a->top_k, p.top_p = a->top_p, p.min_p = a->min_p;
  p.token = a->token, p.logprob = a->logprob;
  static const std::array<uint2, 256> pow2 = [] {
    std::array<uint2, 256> t;
    for (int j = 0; j < 256; ++j) {
      const double v = std::exp2(j / 256.0);
      const float f = (float)v;
      t[j].x = (uint32_t)std::llrint(std::ldexp(v, 30));
      std::memcpy(&t[j].y, &f, 4);
    }
    return t;
  }();
  std::memcpy(p.pow2, pow2.data(), sizeof(p.pow2));
  return cuda_status(launch_sample(p, a->dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
