// C ABI of the attention-side operators (declared and documented in include/orbq.h): argument
// checks on the host, then asynchronous launches.
#include <hip/hip_runtime.h>

#include "attention_checks.h"

#define ORBQ_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace orbq::checks;
using orbq::set_error;
using orbq::set_ok;

int kv_move(bool read, const orbq_kv_cache* cache, const orbq_page_table* table, const int32_t* first, const int32_t* cu,
            int64_t total, int32_t max_rows, void* k, int64_t kt, int64_t kh, void* v, int64_t vt, int64_t vh,
            orbq_dtype type, void* stream, const char* what) {
  orbq::KvCache c;
  int s;
  if ((s = check_cache(cache, table, &c, what))) return s;
  if ((s = check_type(type, true, what))) return s;
  if ((s = check_packed(total, max_rows, c.batch, cu, what))) return s;
  if (total == 0 || max_rows == 0) return set_ok();
  if ((s = check_cache_buffers(c, what))) return s;
  if (!first) return set_error(ORBQ_ERR_INVALID_ARG, "%s: NULL positions", what);
  if (!aligned(first, 4)) return set_error(ORBQ_ERR_ALIGNMENT, "%s: positions misaligned", what);
  const int size = orbq::dtype_size(type);
  if ((s = check_strided(k, kt, kh, size, 16, what))) return s;
  if ((s = check_strided(v, vt, vh, size, 16, what))) return s;
  if (read) {
    if ((s = check_written(kt, kh, total, c.heads, c.d, what))) return s;
    if ((s = check_written(vt, vh, total, c.heads, c.d, what))) return s;
  }
  if (!read && c.max_pages == 0) return set_ok();  // nowhere to write
  const orbq::KvTokens x{cu, first, total, bound_rows(max_rows, total), k, v, kt, kh, vt, vh};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return hip_status(read ? orbq::launch_kv_read(c, x, type, st) : orbq::launch_kv_append(c, x, type, st), what);
}

// workspace: tiles in f16 and their factors, then the parts of split rows
size_t turned_bytes(const orbq::AttnPlan& p, int32_t batch, int32_t kv_heads, int32_t d) {
  return static_cast<size_t>(batch) * kv_heads * p.turned * 256 * d;
}
size_t factor_bytes(const orbq::AttnPlan& p, int32_t batch, int32_t kv_heads) {
  return static_cast<size_t>(batch) * kv_heads * p.turned * 64;
}
size_t part_bytes(const orbq::AttnPlan& p, int32_t d) {
  return p.splits > 1 ? static_cast<size_t>(p.part_rows) * p.splits * (d + 2) * sizeof(float) : 0;
}

}  // namespace

ORBQ_API int orbq_rope_apply(const orbq_rope* rope, const float* positions, int64_t n_positions, int64_t n,
                             int32_t head_dim, const orbq_heads* tensors, int32_t count, orbq_dtype type, int32_t inverse,
                             void* stream) {
  const char* what = "orbq_rope_apply";
  int s;
  orbq::RopeArgs a{};
  if ((s = check_rope(rope, head_dim, type, &a, what))) return s;
  if (n < 0 || count < 1 || count > 2) return set_error(ORBQ_ERR_INVALID_ARG, "%s: n %lld, %d tensors (1 or 2)", what, static_cast<long long>(n), count);
  if (!tensors) return set_error(ORBQ_ERR_INVALID_ARG, "%s: tensors are NULL", what);
  if (n == 0) return set_ok();
  if ((s = check_positions(rope, positions, n_positions, n, &a, what))) return s;
  const int size = orbq::dtype_size(type);
  int64_t all = 0;
  for (int i = 0; i < count; ++i) {
    const orbq_heads& t = tensors[i];
    if (t.heads < 0) return set_error(ORBQ_ERR_INVALID_ARG, "%s: negative heads", what);
    if (t.heads == 0) continue;
    if (t.heads > 16384) return set_error(ORBQ_ERR_UNSUPPORTED, "%s: heads above 16384", what);
    if ((s = check_strided(t.x, t.x_token, t.x_head, size, size, what))) return s;
    if ((s = check_strided(t.y, t.y_token, t.y_head, size, size, what))) return s;
    if ((s = check_written(t.y_token, t.y_head, n, t.heads, head_dim, what))) return s;
    a.t[i] = orbq::RopeTensor{t.x, t.y, t.heads, t.x_token, t.x_head, t.y_token, t.y_head};
    all += t.heads;
  }
  if (all == 0) return set_ok();
  a.n = n;
  a.d = head_dim;
  a.inverse = inverse != 0;
  return hip_status(orbq::launch_rope(a, type, static_cast<hipStream_t>(stream)), what);
}

ORBQ_API int orbq_kv_append(const orbq_kv_cache* cache, const orbq_page_table* table, const int32_t* start,
                            const int32_t* cu, int64_t total, int32_t max_new, const void* k, int64_t k_token,
                            int64_t k_head, const void* v, int64_t v_token, int64_t v_head, orbq_dtype type, void* stream) {
  return kv_move(false, cache, table, start, cu, total, max_new, const_cast<void*>(k), k_token, k_head,
                 const_cast<void*>(v), v_token, v_head, type, stream, "orbq_kv_append");
}

ORBQ_API int orbq_kv_read(const orbq_kv_cache* cache, const orbq_page_table* table, const int32_t* first,
                          const int32_t* cu, int64_t total, int32_t max_tokens, void* k, int64_t k_token, int64_t k_head,
                          void* v, int64_t v_token, int64_t v_head, orbq_dtype type, void* stream) {
  return kv_move(true, cache, table, first, cu, total, max_tokens, k, k_token, k_head, v, v_token, v_head, type, stream,
                 "orbq_kv_read");
}

ORBQ_API size_t orbq_kv_attention_workspace_bytes(const orbq_kv_cache* cache, int32_t batch, int64_t total,
                                                  int32_t max_new, int32_t heads, int64_t max_len, int32_t causal_block,
                                                  int32_t window) {
  if (!cache || batch < 1 || total < 1 || max_new < 1 || heads < 1 || cache->kv_heads < 1 || heads % cache->kv_heads ||
      max_len < 0 || max_len > kMaxTokens || causal_block < 0 || window < 0 ||
      static_cast<int64_t>(max_new) * (heads / cache->kv_heads) > kMaxRows)
    return 0;
  const orbq::AttnPlan p = orbq::plan_attention(batch, total, bound_rows(max_new, total), heads, cache->kv_heads, cache->head_dim,
                                                max_len, causal_block, window, true, orbq::device_cus());
  return turned_bytes(p, batch, cache->kv_heads, cache->head_dim) + factor_bytes(p, batch, cache->kv_heads) +
         part_bytes(p, cache->head_dim);
}

ORBQ_API int orbq_kv_attention(const orbq_kv_cache* cache, const orbq_page_table* table, const int32_t* lens,
                               const int32_t* cu, int64_t total, int32_t max_new, int64_t max_len, const void* q,
                               int64_t q_token, int64_t q_head, int32_t heads, void* o, int64_t o_token, int64_t o_head,
                               float* lse, orbq_dtype type, float scale, int32_t causal_block, int32_t window,
                               void* workspace, size_t ws_bytes, void* stream) {
  const char* what = "orbq_kv_attention";
  orbq::AttnArgs a{};
  int s;
  if ((s = check_cache(cache, table, &a.c, what))) return s;
  if ((s = check_type(type, false, what))) return s;
  if ((s = check_packed(total, max_new, a.c.batch, cu, what))) return s;
  if (heads < 1 || heads % a.c.heads)
    return set_error(ORBQ_ERR_INVALID_ARG, "%s: %d query heads for %d cache heads", what, heads, a.c.heads);
  if (heads > 16384) return set_error(ORBQ_ERR_UNSUPPORTED, "%s: heads above 16384", what);
  if (static_cast<int64_t>(max_new) * (heads / a.c.heads) > kMaxRows)
    return set_error(ORBQ_ERR_UNSUPPORTED, "%s: more than 2^36 rows a cache head", what);
  if (max_len < 0) return set_error(ORBQ_ERR_INVALID_ARG, "%s: max_len negative", what);
  if (causal_block < 0 || window < 0) return set_error(ORBQ_ERR_INVALID_ARG, "%s: causal_block or window negative", what);
  if (!std::isfinite(scale)) return set_error(ORBQ_ERR_INVALID_ARG, "%s: scale is not finite", what);
  if (total == 0 || max_new == 0) return set_ok();
  if ((s = check_cache_buffers(a.c, what))) return s;
  if (!lens) return set_error(ORBQ_ERR_INVALID_ARG, "%s: NULL lens", what);
  if (!aligned(lens, 4) || !aligned(lse, 4)) return set_error(ORBQ_ERR_ALIGNMENT, "%s: lens or lse misaligned", what);
  if ((s = check_strided(q, q_token, q_head, 2, 16, what))) return s;
  if ((s = check_strided(o, o_token, o_head, 2, 8, what))) return s;
  if ((s = check_written(o_token, o_head, total, heads, a.c.d, what))) return s;
  max_new = bound_rows(max_new, total);
  const int64_t most = static_cast<int64_t>(a.c.max_pages) * a.c.page;
  const int64_t len = max_len && max_len < most ? max_len : most;
  // tiles are turned into the workspace only where it is known how many there can be
  const orbq::AttnPlan p = orbq::plan_attention(a.c.batch, total, max_new, heads, a.c.heads, a.c.d, len, causal_block, window,
                                                len == most, orbq::device_cus());
  if (p.many && static_cast<int64_t>(a.c.batch) * a.c.heads * p.row_tiles > orbq::kMostTiles)
    return set_error(ORBQ_ERR_UNSUPPORTED, "%s: more than 2^31 row tiles (batch, heads and max_new too large)", what);
  const size_t turned = turned_bytes(p, a.c.batch, a.c.heads, a.c.d), factors = factor_bytes(p, a.c.batch, a.c.heads);
  const size_t need = turned + factors + part_bytes(p, a.c.d);
  if (need) {
    if (!workspace || ws_bytes < need)
      return set_error(ORBQ_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", what, workspace ? ws_bytes : 0, need);
    if (!aligned(workspace, 256)) return set_error(ORBQ_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", what);
    if (p.splits > 1 && (p.part_rows > 0x7fffffff || static_cast<int64_t>(a.c.batch) * max_new * heads > 0x7fffffff))
      return set_error(ORBQ_ERR_UNSUPPORTED, "%s: more than 2^31 rows over split keys", what);
    a.turned = workspace;
    a.factors = static_cast<char*>(workspace) + turned;
    a.turned_tiles = p.turned;
    a.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + turned + factors);
    a.part_ml = a.part_o + p.part_rows * p.splits * a.c.d;
  }
  a.page_shift = __builtin_ctz(a.c.page);
  a.lens = lens;
  a.cu = cu;
  a.total = total;
  a.max_new = max_new;
  a.heads = heads;
  a.group = heads / a.c.heads;
  a.q = q;
  a.o = o;
  a.qt = q_token;
  a.qh = q_head;
  a.ot = o_token;
  a.oh = o_head;
  a.lse = lse;
  a.scale_log2e = static_cast<float>(std::fabs(static_cast<double>(scale)) * 1.4426950408889634);
  a.negative = scale < 0.0f;
  a.f16 = type == ORBQ_F16;
  a.causal_block = causal_block;
  a.window = window;
  return hip_status(orbq::launch_kv_attention(a, p, static_cast<hipStream_t>(stream)), what);
}
