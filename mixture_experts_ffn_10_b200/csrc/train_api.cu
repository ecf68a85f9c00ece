// train_api.cu -- the entry points of moe_train.h: argument checks and launches.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "fp8.cuh"
#include "moe_train.h"
#include "train.cuh"

namespace moe {
namespace {

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return set_error(code, buf);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

int check(const moe_shape* s, const moe_options* o, int64_t B) {
  const int rc = check_layer(s, o);
  if (rc) return rc;
  if (B < 1 || B > (1 << 24)) return fail(MOE_ERR_SHAPE, "need 1 <= B <= 2^24 sequences (B=%lld)", (long long)B);
  return MOE_OK;
}

struct BalanceLayout {
  int chunk, nchunks;
  size_t ticket, psum, pcnt, part, total;
};

BalanceLayout balance_layout(const moe_shape* s, int64_t B) {
  BalanceLayout l;
  const int64_t chunk = (s->T + kBalanceMaxChunks - 1) / kBalanceMaxChunks;
  l.chunk = (int)(chunk < 16 ? 16 : chunk);
  l.nchunks = (int)((s->T + l.chunk - 1) / l.chunk);
  if (l.nchunks < 1) l.nchunks = 1;
  const size_t rows = ((size_t)l.nchunks + B) * s->E * 4;
  l.ticket = 0;
  l.psum = 256;
  l.pcnt = align256(l.psum + rows);
  l.part = align256(l.pcnt + rows);
  l.total = align256(l.part + (size_t)B * ((s->E + 31) / 32) * 8);
  return l;
}

RouterTrainArgs common_args(const moe_shape* s, const moe_options* o, const void* logits, const void* router_bias,
                            const int32_t* idx, const int32_t* seq, int64_t B, float coef) {
  RouterTrainArgs a{};
  a.logits = logits;
  a.router_bias = router_bias;
  a.idx = idx;
  a.seq = seq;
  a.T = (int)s->T;
  a.E = (int)s->E;
  a.k = (int)s->k;
  a.B = (int)B;
  a.bf16 = s->logit_dtype == MOE_BF16;
  a.score = o->score;
  a.coef = coef;
  a.renorm = o->renormalize;
  a.scale = o->routed_scale;
  a.vec = s->E % (a.bf16 ? 8 : 4) == 0 && aligned(logits, 16);
  return a;
}

int check_inputs(const moe_shape* s, const void* logits, const void* router_bias, const int32_t* idx, const int32_t* seq,
                 int64_t B, float coef) {
  const int elt = s->logit_dtype == MOE_BF16 ? 2 : 4;
  if (s->T > 0 && (!logits || !idx)) return fail(MOE_ERR_NULL, "logits and idx are required");
  if (!aligned(logits, elt) || !aligned(router_bias, elt) || !aligned(idx, 4) || !aligned(seq, 4))
    return fail(MOE_ERR_ALIGN, "logits, router_bias, idx and seq_offsets must be aligned to their elements");
  if (!seq && B != 1) return fail(MOE_ERR_NULL, "seq_offsets is required for more than one sequence");
  if (!std::isfinite(coef)) return fail(MOE_ERR_ARG, "coef must be finite");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_balance_workspace_size(const moe_shape* s, const moe_options* o, int64_t B) {
  if (moe::check(s, o, B) != MOE_OK) return 0;
  return moe::balance_layout(s, B).total;
}

int moe_balance_loss(const moe_shape* s, const moe_options* o, const void* logits, const void* router_bias,
                     const int32_t* idx, const int32_t* seq_offsets, int64_t B, float coef, int32_t* counts, float* loss,
                     void* ws, size_t ws_bytes, void* stream) {
  using namespace moe;
  int rc = check(s, o, B);
  if (rc) return rc;
  if ((rc = check_inputs(s, logits, router_bias, idx, seq_offsets, B, coef))) return rc;
  if (!counts || !loss) return fail(MOE_ERR_NULL, "counts and loss are required");
  if (!aligned(counts, 4) || !aligned(loss, 4)) return fail(MOE_ERR_ALIGN, "counts and loss must be 4-byte aligned");
  const BalanceLayout l = balance_layout(s, B);
  if (!ws || ws_bytes < l.total)
    return fail(MOE_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", l.total, ws ? ws_bytes : 0);
  if (!aligned(ws, 256)) return fail(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  uint8_t* base = static_cast<uint8_t*>(ws);
  RouterTrainArgs a = common_args(s, o, logits, router_bias, idx, seq_offsets, B, coef);
  a.chunk = l.chunk;
  a.nchunks = l.nchunks;
  a.ticket = reinterpret_cast<int32_t*>(base + l.ticket);
  a.psum = reinterpret_cast<float*>(base + l.psum);
  a.pcnt = reinterpret_cast<int32_t*>(base + l.pcnt);
  a.part = reinterpret_cast<double*>(base + l.part);
  a.counts = counts;
  a.loss = loss;
  const cudaError_t e = launch_balance_loss(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "balance loss: %s", cudaGetErrorString(e));
}

int moe_router_backward(const moe_shape* s, const moe_options* o, const void* logits, const void* router_bias,
                        const int32_t* idx, const float* dw, const int32_t* counts, const int32_t* seq_offsets, int64_t B,
                        float coef, const float* dloss, void* dlogits, void* stream) {
  using namespace moe;
  if (!counts) {  // no balance part
    seq_offsets = nullptr;
    B = 1;
    coef = 0.f;
    dloss = nullptr;
  }
  int rc = check(s, o, B);
  if (rc) return rc;
  if (!dw && !counts) return fail(MOE_ERR_NULL, "dw or counts is required");
  if ((rc = check_inputs(s, logits, router_bias, idx, seq_offsets, B, coef))) return rc;
  if (s->T == 0) return MOE_OK;
  if (!dlogits) return fail(MOE_ERR_NULL, "dlogits is required");
  if (!aligned(dlogits, s->logit_dtype == MOE_BF16 ? 2 : 4) || !aligned(dw, 4) || !aligned(counts, 4) || !aligned(dloss, 4))
    return fail(MOE_ERR_ALIGN, "dlogits, dw, counts and dloss must be aligned to their elements");
  if (dlogits == logits) return fail(MOE_ERR_ARG, "dlogits must not alias logits");
  RouterTrainArgs a = common_args(s, o, logits, router_bias, idx, seq_offsets, B, coef);
  a.vec = a.vec && aligned(dlogits, 16);
  a.dw = dw;
  a.counts = const_cast<int32_t*>(counts);
  a.dloss = dloss;
  a.dlogits = dlogits;
  const cudaError_t e = launch_router_backward(a, device_sms(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "router backward: %s", cudaGetErrorString(e));
}

}  // extern "C"
