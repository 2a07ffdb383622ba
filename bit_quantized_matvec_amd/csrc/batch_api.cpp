// batch_api.cpp -- C ABI of what differs from row to row in a batch (experts,
// adapters, sampling): argument validation on the host, then the launchers of
// batch.h.  Nothing here allocates, frees or synchronizes.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/tq.h"
#include "api_status.h"
#include "batch.h"

// The Python binding packs these field by field (batch.py).
static_assert(sizeof(tq_route_args) == 88 && sizeof(tq_gemm_experts_args) == 96 && sizeof(tq_adapter_add_args) == 160 && sizeof(tq_sample_args) == 112,
              "argument structs");

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 20;
constexpr int64_t kMaxPairs = int64_t(1) << 25;
constexpr int64_t kMaxVocab = int64_t(1) << 20;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxRows = int64_t(1) << 26;
constexpr int64_t kMaxCols = int64_t(1) << 20;
constexpr int64_t kMaxValues = int64_t(1) << 40;
constexpr int kMaxExperts = 1 << 16;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool type_ok(int t) { return t == TQ_F32 || t == TQ_BF16 || t == TQ_F16; }
bool half_ok(int t) { return t == TQ_BF16 || t == TQ_F16; }
int bytes_of(int t) { return t == TQ_F32 ? 4 : 2; }
bool stride_ok(int64_t s) { return s >= -kMaxStride && s <= kMaxStride; }

int route_status(const tq_route_args& a) {
  if (!type_ok(a.in_type) || (a.score != TQ_SOFTMAX && a.score != TQ_SIGMOID)) return TQ_ERR_FORMAT;
  if (a.tokens < 0 || a.tokens > kMaxTokens || a.experts < 1 || a.experts > 1024 || a.k < 1 || a.k > 32 || !stride_ok(a.logit_stride)) return TQ_ERR_SHAPE;
  if (a.groups < 1 || a.groups > 64 || a.experts % a.groups || a.top_groups < 1 || a.top_groups > a.groups || a.group_best < 1 || a.group_best > 2 ||
      a.k > a.experts / a.groups * a.top_groups || !std::isfinite(a.scale))
    return TQ_ERR_SHAPE;
  if (a.groups > 1 && a.group_best > a.experts / a.groups) return TQ_ERR_SHAPE;
  if (a.tokens == 0) return TQ_OK;
  if (!a.logits || !a.weights || !a.ids) return TQ_ERR_NULL;
  if (!aligned(a.logits, bytes_of(a.in_type)) || !aligned(a.bias, 4) || !aligned(a.weights, 4) || !aligned(a.ids, 4)) return TQ_ERR_ALIGN;
  return TQ_OK;
}

int experts_status(const tq_gemm_experts_args& a) {
  if (a.fmt != TQ_FMT_PQ2_0 && a.fmt != TQ_FMT_PTQ1_0) return TQ_ERR_FORMAT;
  if (a.pairs < 0 || a.pairs > kMaxPairs || a.inputs < 0 || a.experts < 1 || a.experts > kMaxExperts) return TQ_ERR_SHAPE;
  const int st = tq_check_shape(a.fmt, a.rows, a.cols, 1);
  if (st != TQ_OK) return st;
  if (a.pairs > 0 && (a.inputs < 1 || a.pairs % a.inputs || a.inputs > kMaxValues / a.cols || a.pairs > kMaxValues / a.rows)) return TQ_ERR_SHAPE;
  if (a.fmt != TQ_FMT_PQ2_0) return TQ_ERR_UNSUPPORTED;
  if (a.pairs == 0) return TQ_OK;
  if (!a.w || !a.q || !a.d || !a.order || !a.offsets || !a.y) return TQ_ERR_NULL;
  if (!aligned(a.w, 16) || !aligned(a.q, 16) || !aligned(a.d, 4) || !aligned(a.order, 4) || !aligned(a.offsets, 4) || !aligned(a.y, 4) ||
      !aligned(a.bad_flag, 4))
    return TQ_ERR_ALIGN;
  return TQ_OK;
}

int adapter_sizes(int64_t tokens, int adapters, int rank, int64_t cols) {
  if (tokens < 0 || tokens > kMaxTokens || adapters < 1 || adapters > kMaxExperts || rank < 8 || rank > 256 || rank % 8 || cols < 8 || cols > kMaxCols ||
      cols % 8)
    return TQ_ERR_SHAPE;
  return TQ_OK;
}

int adapter_status(const tq_adapter_add_args& a) {
  if (!half_ok(a.w_type) || (a.x_type != TQ_F32 && a.x_type != a.w_type) || !type_ok(a.y_type)) return TQ_ERR_FORMAT;
  const int st = adapter_sizes(a.tokens, a.adapters, a.rank, a.cols);
  if (st != TQ_OK) return st;
  if (a.rows < 1 || a.rows > kMaxRows || !stride_ok(a.x_stride) || !stride_ok(a.y_stride) || !stride_ok(a.out_stride)) return TQ_ERR_SHAPE;
  if (a.out == a.y && a.out_stride != a.y_stride) return TQ_ERR_SHAPE;
  if (a.tokens > 1 && a.out_stride < a.rows && a.out_stride > -a.rows) return TQ_ERR_SHAPE;  // rows that overlap
  if (a.tokens == 0) return TQ_OK;
  if (!a.x || !a.y || !a.a || !a.b || !a.out || !a.index || !a.workspace) return TQ_ERR_NULL;
  const int ye = bytes_of(a.y_type);
  if (!aligned(a.x, 16) || !aligned(a.a, 16) || !aligned(a.b, 16) || !aligned(a.y, ye) || !aligned(a.out, ye) || !aligned(a.index, 4) ||
      !aligned(a.ranks, 4) || !aligned(a.scale, 4) || !aligned(a.workspace, 16) || !aligned(a.bad_flag, 4) || a.x_stride * bytes_of(a.x_type) % 16)
    return TQ_ERR_ALIGN;
  if (a.workspace_bytes < tq::adapter_workspace_bytes(a.tokens, a.adapters, a.rank, a.cols)) return TQ_ERR_SHAPE;
  return TQ_OK;
}

int sample_sizes(int64_t rows, int64_t vocab) {
  return rows < 0 || rows > (int64_t(1) << 16) || vocab < 1 || vocab > kMaxVocab ? TQ_ERR_SHAPE : TQ_OK;
}

int sample_status(const tq_sample_args& a) {
  if (!type_ok(a.in_type)) return TQ_ERR_FORMAT;
  const int st = sample_sizes(a.rows, a.vocab);
  if (st != TQ_OK || !stride_ok(a.logit_stride)) return TQ_ERR_SHAPE;
  if (a.rows == 0) return TQ_OK;
  if (!a.logits || !a.u || !a.tokens || !a.workspace) return TQ_ERR_NULL;
  if (!aligned(a.logits, bytes_of(a.in_type)) || !aligned(a.u, 4) || !aligned(a.temperature, 4) || !aligned(a.top_k, 4) || !aligned(a.top_p, 4) ||
      !aligned(a.min_p, 4) || !aligned(a.tokens, 4) || !aligned(a.logprob, 4) || !aligned(a.workspace, 16))
    return TQ_ERR_ALIGN;
  if (a.workspace_bytes < tq::sample_workspace_bytes(a.rows, a.vocab)) return TQ_ERR_SHAPE;
  return TQ_OK;
}

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

int tq_route(const tq_route_args* a, void* stream) {
  if (!a) return TQ_ERR_NULL;
  const int st = route_status(*a);
  if (st != TQ_OK || a->tokens == 0) return st;
  return tq::hip_status(tq::launch_route(*a, as_stream(stream)));
}

int tq_expert_lists(const int32_t* ids, int64_t pairs, int32_t experts, int32_t* order, int32_t* offsets, void* stream) {
  if (pairs < 0 || pairs > kMaxPairs || experts < 1 || experts > kMaxExperts) return TQ_ERR_SHAPE;
  if (!offsets || (pairs > 0 && (!ids || !order))) return TQ_ERR_NULL;
  if (!aligned(ids, 4) || !aligned(order, 4) || !aligned(offsets, 4)) return TQ_ERR_ALIGN;
  return tq::hip_status(tq::launch_expert_lists(ids, pairs, experts, order, offsets, as_stream(stream)));
}

int tq_gemm_experts(const tq_gemm_experts_args* a, void* stream) {
  if (!a) return TQ_ERR_NULL;
  const int st = experts_status(*a);
  if (st != TQ_OK || a->pairs == 0) return st;
  return tq::hip_status(tq::launch_gemm_experts_pq2(*a, as_stream(stream)));
}

int64_t tq_adapter_workspace_bytes(int64_t tokens, int32_t adapters, int32_t rank, int64_t cols) {
  if (adapter_sizes(tokens, adapters, rank, cols) != TQ_OK) return 0;
  return tq::adapter_workspace_bytes(tokens, adapters, rank, cols);
}

int tq_adapter_add(const tq_adapter_add_args* a, void* stream) {
  if (!a) return TQ_ERR_NULL;
  const int st = adapter_status(*a);
  if (st != TQ_OK || a->tokens == 0) return st;
  return tq::hip_status(tq::launch_adapter_add(*a, as_stream(stream)));
}

int64_t tq_sample_workspace_bytes(int64_t rows, int64_t vocab) {
  if (sample_sizes(rows, vocab) != TQ_OK) return 0;
  return tq::sample_workspace_bytes(rows, vocab);
}

int tq_sample(const tq_sample_args* a, void* stream) {
  if (!a) return TQ_ERR_NULL;
  const int st = sample_status(*a);
  if (st != TQ_OK || a->rows == 0) return st;
  return tq::hip_status(tq::launch_sample(*a, as_stream(stream)));
}

}  // extern "C"
