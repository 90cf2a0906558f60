// Argument checks that the attention-side entry points share (attention_api.cpp, block_api.cpp).
#pragma once

#include <cmath>

#include "../../include/orbq.h"
#include "attention.h"
#include "internal.h"

namespace orbq {
namespace checks {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int hip_status(int e, const char* what) {
  if (e != hipSuccess) return set_error(ORBQ_ERR_HIP, "%s: %s", what, hipGetErrorString(static_cast<hipError_t>(e)));
  return set_ok();
}

inline int check_type(orbq_dtype t, bool f32, const char* what) {
  if (t == ORBQ_BF16 || t == ORBQ_F16 || (t == ORBQ_F32 && f32)) return ORBQ_OK;
  return set_error(t == ORBQ_F32 ? ORBQ_ERR_UNSUPPORTED : ORBQ_ERR_INVALID_ARG, "%s: type %d", what, static_cast<int>(t));
}

constexpr int64_t kMaxTokens = int64_t{1} << 30;  // of a sequence: positions are 32-bit in the kernels

constexpr int64_t kMaxRows = int64_t{1} << 36;    // queries times query heads of one cache head: row tiles are 32-bit

inline int check_cache(const orbq_kv_cache* c, const orbq_page_table* t, KvCache* out, const char* what) {
  if (!c || !t) return set_error(ORBQ_ERR_INVALID_ARG, "%s: cache or page table is NULL", what);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return set_error(ORBQ_ERR_UNSUPPORTED, "%s: head_dim %d not in {64, 128, 256}", what, c->head_dim);
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
    return set_error(ORBQ_ERR_UNSUPPORTED, "%s: page_tokens %d not in {16, 32, 64, 128}", what, c->page_tokens);
  if (c->num_pages < 1 || c->kv_heads < 1) return set_error(ORBQ_ERR_INVALID_ARG, "%s: num_pages or kv_heads below 1", what);
  if (c->kv_heads > 16384) return set_error(ORBQ_ERR_UNSUPPORTED, "%s: kv_heads above 16384", what);
  if (t->batch < 0 || t->max_pages < 0 || t->ld < t->max_pages)
    return set_error(ORBQ_ERR_INVALID_ARG, "%s: page table batch %d, max_pages %d, ld %lld", what, t->batch, t->max_pages,
                     static_cast<long long>(t->ld));
  if (t->batch > 65535) return set_error(ORBQ_ERR_UNSUPPORTED, "%s: batch above 65535", what);
  if (static_cast<int64_t>(t->max_pages) * c->page_tokens > kMaxTokens)
    return set_error(ORBQ_ERR_UNSUPPORTED, "%s: more than 2^30 tokens a sequence", what);
  *out = KvCache{c->k_codes, c->v_codes, c->k_scales, c->v_scales, c->num_pages, c->kv_heads, c->page_tokens,
                       c->head_dim, t->table, t->ld, t->max_pages, t->batch};
  return ORBQ_OK;
}

// pointers that a call with work to do dereferences
inline int check_cache_buffers(const KvCache& c, const char* what) {
  if (!c.k || !c.v || !c.ks || !c.vs || (!c.table && c.max_pages)) return set_error(ORBQ_ERR_INVALID_ARG, "%s: NULL cache buffer or page table", what);
  if (!aligned(c.k, 16) || !aligned(c.v, 16)) return set_error(ORBQ_ERR_ALIGNMENT, "%s: codes must be 16-byte aligned", what);
  if (!aligned(c.ks, 4) || !aligned(c.vs, 4) || !aligned(c.table, 4))
    return set_error(ORBQ_ERR_ALIGNMENT, "%s: scales and page table must be 4-byte aligned", what);
  return ORBQ_OK;
}

inline int check_packed(int64_t total, int32_t max_rows, int32_t batch, const int32_t* cu, const char* what) {
  if (total < 0 || max_rows < 0) return set_error(ORBQ_ERR_INVALID_ARG, "%s: negative count", what);
  if (total > kMaxTokens || max_rows > (1 << 30)) return set_error(ORBQ_ERR_UNSUPPORTED, "%s: more than 2^30 rows", what);
  if (total && !batch) return set_error(ORBQ_ERR_INVALID_ARG, "%s: rows but no sequence", what);
  if (total && !cu && total % batch) return set_error(ORBQ_ERR_INVALID_ARG, "%s: without cu every sequence has total / batch rows", what);
  if (!aligned(cu, 4)) return set_error(ORBQ_ERR_ALIGNMENT, "%s: cu misaligned", what);
  return ORBQ_OK;
}

// A caller's bound may be far above the work (one for all the calls of a captured graph): grids and plans go by what
// there can be.
inline int32_t bound_rows(int32_t max_rows, int64_t total) { return total < max_rows ? static_cast<int32_t>(total) : max_rows; }

// [rows][heads][...] with strides in elements of `size` bytes, which divide `align`
inline int check_strided(const void* p, int64_t token, int64_t head, int size, int align, const char* what) {
  if (!p) return set_error(ORBQ_ERR_INVALID_ARG, "%s: NULL buffer", what);
  if (token < 0 || head < 0) return set_error(ORBQ_ERR_INVALID_ARG, "%s: negative stride", what);
  if (!aligned(p, align) || token % (align / size) || head % (align / size))
    return set_error(ORBQ_ERR_ALIGNMENT, "%s: base and strides must be multiples of %d bytes", what, align);
  return ORBQ_OK;
}

// Whether any two rows of `width` elements, tokens `token` apart and heads `head` apart, share an element.
inline bool rows_overlap(int64_t token, int64_t head, int64_t tokens, int32_t heads, int32_t width) {
  if ((heads > 1 && head < width) || (tokens > 1 && token < width)) return true;
  if (heads <= 1 || tokens <= 1) return false;
  // [token][head] and [head][token], the usual orders: one dimension's rows lie between two steps of the other
  if ((token - width) / (heads - 1) >= head || (head - width) / (tokens - 1) >= token) return false;
  // else no number of heads may come within a row of a number of tokens
  for (int64_t j = 1; j < heads; ++j) {
    const unsigned __int128 at = static_cast<unsigned __int128>(j) * static_cast<uint64_t>(head);
    const unsigned __int128 i = at / static_cast<uint64_t>(token);
    const uint64_t rest = static_cast<uint64_t>(at % static_cast<uint64_t>(token));
    if (i < static_cast<uint64_t>(tokens) && rest < static_cast<uint64_t>(width)) return true;
    if (i + 1 < static_cast<uint64_t>(tokens) && static_cast<uint64_t>(token) - rest < static_cast<uint64_t>(width)) return true;
  }
  return false;
}

// an output whose rows must not overlap
inline int check_written(int64_t token, int64_t head, int64_t tokens, int32_t heads, int32_t width, const char* what) {
  if (rows_overlap(token, head, tokens, heads, width)) return set_error(ORBQ_ERR_INVALID_ARG, "%s: rows of the output overlap", what);
  return ORBQ_OK;
}

// A rope's axes, layout and the head that it turns part of; and what the kernels need of them.
template <class A> int check_rope(const orbq_rope* rope, int32_t head_dim, orbq_dtype type, A* a, const char* what) {
  int s;
  if (!rope) return set_error(ORBQ_ERR_INVALID_ARG, "%s: rope is NULL", what);
  if (rope->axes < 1 || rope->axes > 4) return set_error(ORBQ_ERR_UNSUPPORTED, "%s: %d axes (1..4 supported)", what, rope->axes);
  if (head_dim < 2 || head_dim > 512 || head_dim % 2)
    return set_error(ORBQ_ERR_UNSUPPORTED, "%s: head_dim %d not an even number in [2, 512]", what, head_dim);
  if (rope->layout != ORBQ_ROPE_PAIRS && rope->layout != ORBQ_ROPE_HALVES)
    return set_error(ORBQ_ERR_INVALID_ARG, "%s: layout %d", what, static_cast<int>(rope->layout));
  if ((s = check_type(type, true, what))) return s;
  int64_t pairs = 0;
  for (int i = 0; i < rope->axes; ++i) {
    if (rope->dims[i] < 0 || rope->dims[i] % 2 || rope->dims[i] > head_dim)
      return set_error(ORBQ_ERR_INVALID_ARG, "%s: axis %d has %d entries", what, i, rope->dims[i]);
    pairs += rope->dims[i] / 2;
    a->ends[i] = static_cast<int32_t>(pairs);
  }
  if (pairs < 1 || 2 * pairs > head_dim)
    return set_error(ORBQ_ERR_INVALID_ARG, "%s: axes take %lld of %d entries", what, static_cast<long long>(2 * pairs), head_dim);
  a->freqs = rope->freqs;
  a->axes = rope->axes;
  a->pairs = static_cast<int32_t>(pairs);
  a->halves = rope->layout == ORBQ_ROPE_HALVES;
  return ORBQ_OK;
}

// positions of n tokens (n > 0), shared by n / n_positions equal parts of them
template <class A> int check_positions(const orbq_rope* rope, const float* positions, int64_t n_positions, int64_t n, A* a, const char* what) {
  if (n > (int64_t{1} << 30)) return set_error(ORBQ_ERR_UNSUPPORTED, "%s: more than 2^30 tokens", what);
  if (n_positions < 1 || n % n_positions)
    return set_error(ORBQ_ERR_INVALID_ARG, "%s: %lld positions for %lld tokens", what, static_cast<long long>(n_positions), static_cast<long long>(n));
  if (!positions || !rope->freqs) return set_error(ORBQ_ERR_INVALID_ARG, "%s: NULL positions or freqs", what);
  if (!aligned(positions, 4) || !aligned(rope->freqs, 4)) return set_error(ORBQ_ERR_ALIGNMENT, "%s: positions or freqs misaligned", what);
  a->pos = positions;
  a->n_pos = n_positions;
  return ORBQ_OK;
}

}  // namespace checks
}  // namespace orbq
