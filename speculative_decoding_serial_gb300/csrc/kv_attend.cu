// kv_attend.cu — the call of the attention over the 4-bit paged cache, and its kernels for few rows without first keys that stay visible.
#include "kv_attend_rows.cuh"

namespace whead_kv_impl {
template int launch_few<false>(const HostCache& h, const AttendArgs& a, int max_q, int tile);
extern template int launch_few<true>(const HostCache& h, const AttendArgs& a, int max_q, int tile);  // kv_attend_sinks.cu
}

using namespace whead_kv_impl;

extern "C" int whead_kv_attend(const whead_kv* kv, const whead_kv_attend_args* x) {
  if (!kv || !x) return WHEAD_ERR_INVALID_ARG;
  if (x->n < 0 || x->n > kv->max_seqs || x->total < 0 || x->total >= INT_MAX || x->max_q < 0 || x->heads < 1) return WHEAD_ERR_INVALID_ARG;
  if (kv->kv_heads < 1 || x->heads % kv->kv_heads) return WHEAD_ERR_INVALID_ARG;
  if (x->dtype != WHEAD_KV_BF16 && x->dtype != WHEAD_KV_F16) return WHEAD_ERR_UNSUPPORTED;
  if (x->window < 0 || (x->window > 0 && x->sinks < 0) || ((x->window || x->tree) && !x->causal) || !std::isfinite(x->scale)) return WHEAD_ERR_INVALID_ARG;
  if (x->tree && (x->tree_words < 1 || (int64_t)x->tree_words * 64 < x->max_q || !aligned(x->tree, 8))) return WHEAD_ERR_INVALID_ARG;
  HostCache h;
  if (x->n == 0 || x->total == 0) return x->total > 0 ? WHEAD_ERR_INVALID_ARG : host_cache(kv, &h);
  if (!x->q || !x->out || !aligned(x->q, 2) || !aligned(x->out, 16) || !aligned(x->lse, 4) || !aligned(x->indptr, 4) || !aligned(x->slots, 4) || x->max_q < 1) return WHEAD_ERR_INVALID_ARG;
  if (!x->indptr && (x->total % x->n || x->total / x->n > x->max_q)) return WHEAD_ERR_INVALID_ARG;
  const int group = x->heads / kv->kv_heads;
  const int max_q = (int)std::min<int64_t>(x->max_q, x->total);
  const int64_t rows = (int64_t)max_q * group;
  const int tile = tile_rows(kv->head_dim, rows);
  if (rows >= INT_MAX / 2 || (rows + tile - 1) / tile * x->n > kMaxItems) return WHEAD_ERR_UNSUPPORTED;
  const int rc = host_cache(kv, &h);
  if (rc != WHEAD_OK) return rc;
  AttendArgs a{};
  a.q = x->q;
  a.out = x->out;
  a.lse = x->lse;
  a.indptr = x->indptr;
  a.slots = x->slots;
  a.tree = reinterpret_cast<const unsigned long long*>(x->tree);
  a.total = x->total;
  a.q_token_stride = x->q_token_stride;
  a.q_head_stride = x->q_head_stride;
  a.n = x->n;
  a.each = (int)(x->total / x->n);
  a.max_q = max_q;
  a.heads = x->heads;
  set_group(&a, group);
  a.row_tiles = 1;
  a.dtype = x->dtype;
  a.causal = x->causal;
  a.window = x->window;
  a.sinks = x->window ? x->sinks : 0;
  a.tree_words = x->tree_words;
  a.scale = x->scale;
  a.wide_q16 = aligned(x->q, 16) && x->q_token_stride % 8 == 0 && x->q_head_stride % 8 == 0;
  a.wide_q = aligned(x->q, 8) && x->q_token_stride % 4 == 0 && x->q_head_stride % 4 == 0;
  if (tile > 32) return a.sinks ? launch_tiles<true>(h, a, max_q) : launch_tiles<false>(h, a, max_q);
  return a.sinks ? launch_few<true>(h, a, max_q, tile) : launch_few<false>(h, a, max_q, tile);
}
