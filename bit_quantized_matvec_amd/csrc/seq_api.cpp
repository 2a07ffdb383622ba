// seq_api.cpp -- C ABI of the operators between a block's projections (rotary
// append, paged attention, gated delta rule): argument validation on the host,
// then the launchers of seq.h.  Nothing here allocates, frees or synchronizes.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/tq.h"
#include "api_status.h"
#include "seq.h"

// The Python binding packs these field by field (seq.py).
static_assert(sizeof(tq_rope_append_args) == 200 && sizeof(tq_paged_attn_args) == 184 && sizeof(tq_gdn_args) == 224, "argument structs");

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 20;
constexpr int64_t kMaxSeqs = int64_t(1) << 16;
constexpr int64_t kMaxPages = int64_t(1) << 30;
constexpr int64_t kMaxTable = int64_t(1) << 24;
constexpr int kMaxHeads = 1024;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool type_ok(int t) { return t == TQ_F32 || t == TQ_BF16 || t == TQ_F16; }
bool cache_type_ok(int t) { return t == TQ_BF16 || t == TQ_F16; }
bool attn_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }
bool page_ok(int p) { return p >= 16 && p <= 256 && (p & (p - 1)) == 0; }
bool heads_ok(int q, int kv) { return kv >= 1 && q >= kv && q <= kMaxHeads && q % kv == 0; }

// A tensor read with strides: aligned to 16 bytes at every row.  Strides are
// bounded so that no offset passes 63 bits.
int strided(const void* p, int64_t token, int64_t head, int esz) {
  const int64_t limit = int64_t(1) << 40;
  if (token < -limit || token > limit || head < -limit || head > limit) return TQ_ERR_SHAPE;
  if (!aligned(p, 16) || token * esz % 16 || head * esz % 16) return TQ_ERR_ALIGN;
  return TQ_OK;
}

int first_error(std::initializer_list<int> v) {
  for (int s : v)
    if (s != TQ_OK) return s;
  return TQ_OK;
}

int rope_status(const tq_rope_append_args& a) {
  if (!type_ok(a.in_type) || !cache_type_ok(a.cache_type) || (a.layout != TQ_ROPE_HALF && a.layout != TQ_ROPE_INTERLEAVED))
    return TQ_ERR_FORMAT;
  if (a.tokens < 0 || a.tokens > kMaxTokens || a.pages < 1 || a.pages > kMaxPages || !heads_ok(a.heads, a.kv_heads)) return TQ_ERR_SHAPE;
  if (!attn_dim_ok(a.dim) || !page_ok(a.page) || a.rot < 0 || a.rot > a.dim || a.rot % 16) return TQ_ERR_SHAPE;
  if (!(a.eps >= 0.f) || !std::isfinite(a.eps) || !std::isfinite(a.rope_scale)) return TQ_ERR_SHAPE;
  if (a.tokens == 0) return TQ_OK;
  if (!a.q || !a.k || !a.v || !a.slots || !a.q_out || !a.k_cache || !a.v_cache) return TQ_ERR_NULL;
  if (a.rot > 0 && (!a.positions || !a.inv_freq)) return TQ_ERR_NULL;
  if (!aligned(a.positions, 4) || !aligned(a.slots, 8) || !aligned(a.inv_freq, 8) || !aligned(a.q_norm, 16) || !aligned(a.k_norm, 16) ||
      !aligned(a.q_out, 16) || !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) || !aligned(a.bad_flag, 4))
    return TQ_ERR_ALIGN;
  const int e = tq::type_bytes(a.in_type);
  return first_error({strided(a.q, a.q_token, a.q_head, e), strided(a.k, a.k_token, a.k_head, e), strided(a.v, a.v_token, a.v_head, e)});
}

int attn_sizes(int64_t tokens, int64_t seqs, int heads, int kv_heads, int dim) {
  if (tokens < 0 || tokens > kMaxTokens || seqs < 0 || seqs > kMaxSeqs || !heads_ok(heads, kv_heads) || !attn_dim_ok(dim)) return TQ_ERR_SHAPE;
  return TQ_OK;
}

int attn_status(const tq_paged_attn_args& a) {
  if (!cache_type_ok(a.cache_type) || (a.out_type != a.cache_type && a.out_type != TQ_F32)) return TQ_ERR_FORMAT;
  const int st = attn_sizes(a.tokens, a.seqs, a.heads, a.kv_heads, a.dim);
  if (st != TQ_OK) return st;
  if (a.pages < 1 || a.pages > kMaxPages || !page_ok(a.page) || a.table_width < 0 || a.table_width > kMaxTable || a.table_stride < a.table_width ||
      a.table_stride > kMaxTable || a.table_width * a.page > (int64_t(1) << 31) - 2 * kMaxTokens || a.max_len < 0 || a.window < 0 || !std::isfinite(a.scale))
    return TQ_ERR_SHAPE;
  if (!a.cu && a.tokens != a.seqs) return TQ_ERR_SHAPE;
  if (a.tokens > 0 && a.seqs == 0) return TQ_ERR_SHAPE;
  if (a.tokens == 0) return TQ_OK;
  if (!a.q || !a.k_cache || !a.v_cache || !a.kv_len || !a.out || (a.table_width > 0 && !a.block_table)) return TQ_ERR_NULL;
  if (!aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) || !aligned(a.block_table, 4) || !aligned(a.kv_len, 4) || !aligned(a.cu, 4) ||
      !aligned(a.out, 16) || !aligned(a.lse, 4) || !aligned(a.workspace, 16) || !aligned(a.bad_flag, 4))
    return TQ_ERR_ALIGN;
  if (a.workspace && a.workspace_bytes < tq::paged_attn_workspace_bytes(a.tokens, a.seqs, a.heads, a.kv_heads, a.dim)) return TQ_ERR_SHAPE;
  return strided(a.q, a.q_token, a.q_head, 2);
}

int gdn_sizes(int64_t tokens, int64_t seqs, int64_t max_len, int v_heads, int dk, int dv) {
  if (tokens < 0 || tokens > kMaxTokens || seqs < 0 || seqs > kMaxSeqs || max_len < 0 || v_heads < 1 || v_heads > kMaxHeads) return TQ_ERR_SHAPE;
  if ((dk != 64 && dk != 128) || dv < 32 || dv > 256 || dv % 32) return TQ_ERR_SHAPE;
  return TQ_OK;
}

int gdn_status(const tq_gdn_args& a) {
  if (!type_ok(a.in_type) || (a.out_type != a.in_type && a.out_type != TQ_F32)) return TQ_ERR_FORMAT;
  const int st = gdn_sizes(a.tokens, a.seqs, a.max_len, a.v_heads, a.dk, a.dv);
  if (st != TQ_OK) return st;
  if (!heads_ok(a.v_heads, a.k_heads) || a.states < 1 || a.states > (int64_t(1) << 32) || !std::isfinite(a.scale) || !(a.eps >= 0.f) ||
      !std::isfinite(a.eps))
    return TQ_ERR_SHAPE;
  if (!a.cu && a.tokens != a.seqs) return TQ_ERR_SHAPE;
  if (a.tokens > 0 && a.seqs == 0) return TQ_ERR_SHAPE;
  if (!a.slots && a.seqs > a.states) return TQ_ERR_SHAPE;
  if (a.seqs == 0) return TQ_OK;
  if (!a.state || !a.state_out) return TQ_ERR_NULL;
  if (a.tokens > 0 && (!a.q || !a.k || !a.v || !a.g || !a.beta || !a.out)) return TQ_ERR_NULL;
  if (!aligned(a.g, 4) || !aligned(a.beta, 4) || !aligned(a.state, 16) || !aligned(a.state_out, 16) || !aligned(a.slots, 4) ||
      !aligned(a.cu, 4) || !aligned(a.out, 16) || !aligned(a.workspace, 16) || !aligned(a.bad_flag, 4))
    return TQ_ERR_ALIGN;
  if (a.workspace && a.workspace_bytes < tq::gdn_workspace_bytes(a.tokens, a.seqs, a.max_len, a.v_heads, a.dk, a.dv)) return TQ_ERR_SHAPE;
  const int e = tq::type_bytes(a.in_type);
  return first_error({strided(a.q, a.q_token, a.q_head, e), strided(a.k, a.k_token, a.k_head, e), strided(a.v, a.v_token, a.v_head, e)});
}

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

int tq_rope_append(const tq_rope_append_args* a, void* stream) {
  if (!a) return TQ_ERR_NULL;
  const int st = rope_status(*a);
  if (st != TQ_OK || a->tokens == 0) return st;
  return tq::hip_status(tq::launch_rope_append(*a, as_stream(stream)));
}

int64_t tq_paged_attn_workspace_bytes(int64_t tokens, int64_t seqs, int32_t heads, int32_t kv_heads, int32_t dim) {
  if (attn_sizes(tokens, seqs, heads, kv_heads, dim) != TQ_OK) return 0;
  return tq::paged_attn_workspace_bytes(tokens, seqs, heads, kv_heads, dim);
}

int tq_paged_attn_tile_rows(int64_t tokens, int64_t seqs, int64_t max_len, int32_t heads, int32_t kv_heads, int32_t dim) {
  if (attn_sizes(tokens, seqs, heads, kv_heads, dim) != TQ_OK || max_len < 0 || (tokens > 0 && seqs == 0)) return 0;
  return tq::paged_attn_tile_rows(tokens, seqs, max_len, heads, kv_heads, dim);
}

int tq_paged_attn(const tq_paged_attn_args* a, void* stream) {
  if (!a) return TQ_ERR_NULL;
  const int st = attn_status(*a);
  if (st != TQ_OK || a->tokens == 0) return st;
  return tq::hip_status(tq::launch_paged_attn(*a, as_stream(stream)));
}

int64_t tq_gdn_workspace_bytes(int64_t tokens, int64_t seqs, int64_t max_len, int32_t v_heads, int32_t dk, int32_t dv) {
  if (gdn_sizes(tokens, seqs, max_len, v_heads, dk, dv) != TQ_OK) return 0;
  return tq::gdn_workspace_bytes(tokens, seqs, max_len, v_heads, dk, dv);
}

int tq_gdn(const tq_gdn_args* a, void* stream) {
  if (!a) return TQ_ERR_NULL;
  const int st = gdn_status(*a);
  if (st != TQ_OK || a->seqs == 0) return st;
  return tq::hip_status(tq::launch_gdn(*a, as_stream(stream)));
}

}  // extern "C"
