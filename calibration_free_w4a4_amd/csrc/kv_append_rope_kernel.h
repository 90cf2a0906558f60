// kv_append_rope: keys are normalised (where the model says so), turned by their positions, quantised and written behind
// what the cache holds; values are quantised and written; queries are normalised, turned and written out.  One launch.
//
//   q' = turn(q f_q w_q), k' = turn(k f_k w_k),  f = 1 / sqrt(mean of the head's squares + eps) or 1
//
// then k' and v go through kv_append's rule (kv_cache.hip).  k' is quantised from its fp32 value: it is rounded once, to
// its code.  Every element is read once and written once.
//
// Keys and values: a workgroup for each (touched page, head, keys or values), as in kv_append.  A thread's column of 8 entries
// holds whole pairs, or in the split-half order has its partners in a second column, which it reads too (from L1: a
// row's lanes are in one wave).  A head's sum of squares is taken over the D / 8 lanes that hold the row.
// Queries: a thread holds one column of one token for `per` heads, so that sines and cosines are shared; where a sequence
// has few new tokens a workgroup's rows are heads instead.
#pragma once

#include <algorithm>

#include "kv_cache_device.h"
#include "rope_device.h"

namespace orbq {
int device_cus();
namespace {

// sum over the N lanes (8, 16 or 32, aligned) that hold a row
template <int N> __device__ __forceinline__ float lanes_sum(float x) {
  const auto moved = [](float v, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  x += moved(x, std::integral_constant<int, 0xB1>{});   // quad_perm [1,0,3,2]
  x += moved(x, std::integral_constant<int, 0x4E>{});   // quad_perm [2,3,0,1]
  x += moved(x, std::integral_constant<int, 0x141>{});  // row_half_mirror
  if constexpr (N >= 16) x += moved(x, std::integral_constant<int, 0x140>{});  // row_mirror
  if constexpr (N >= 32) x += __shfl_xor(x, 16);
  return x;
}

// A thread's column of a head: entries e .. e + 7, and what turns them.
template <int DT, int D, bool HALVES> struct Column {
  using T = typename Elem<DT>::T;
  static constexpr int P = HALVES ? 8 : 4;  // pairs that touch the column
  int e;
  const float* weight;  // of the norm, or NULL
  float w[8], pw[8];    // weights of the entries and (HALVES) of their partners

  // the partner of entry j (split halves): i + pairs or i - pairs; the entry itself where it passes through
  static __device__ __forceinline__ int partner(const TurnArgs& r, int i) {
    return i < r.pairs ? i + r.pairs : (i < 2 * r.pairs ? i - r.pairs : i);
  }

  __device__ __forceinline__ void init(const TurnArgs& r, int entry, const float* norm_weight) {
    e = entry;
    weight = norm_weight;
    if (!weight) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = weight[e + j];
      if constexpr (HALVES) pw[j] = weight[partner(r, e + j)];
    }
  }

  __device__ __forceinline__ void sincos(const TurnArgs& r, int64_t row, float* s, float* c) const {
    const float* pos = r.pos + (row < r.n_pos ? row : row % r.n_pos) * r.axes;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int i = HALVES ? e + k : e / 2 + k;
      const int pair = HALVES && i >= r.pairs ? i - r.pairs : i;
      s[k] = 0.0f;
      c[k] = 1.0f;
      if (pair < r.pairs) pair_sincos(r, pos, pair, &s[k], &c[k]);
    }
  }

  // the partners' entries of the row at `head`, as they lie there
  __device__ __forceinline__ void partners(const TurnArgs& r, const T* head, float* b) const {
    if constexpr (HALVES) {
      if (r.pairs % 8 == 0) {
        const int at = partner(r, e);
        Vec<DT, DT == kF32 ? 4 : 8>::load(head, at, b);
        if constexpr (DT == kF32) Vec<DT, 4>::load(head, at + 4, b + 4);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = static_cast<float>(head[partner(r, e + j)]);
      }
    }
  }

  // f: the entries, b: their partners' (HALVES)
  __device__ __forceinline__ void apply(const TurnArgs& r, float* f, float* b, const float* s, const float* c) const {
    if (weight) {
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(f[j], f[j], sum);
      const float unit = 1.0f / __builtin_sqrtf(lanes_sum<D / 8>(sum) * (1.0f / D) + r.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[j] = f[j] * unit * w[j];
        if constexpr (HALVES) b[j] = b[j] * unit * pw[j];
      }
    }
    if constexpr (HALVES) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float u, v;
        if (e + j < r.pairs) {
          turn(f[j], b[j], s[j], c[j], &u, &v);
          f[j] = u;
        } else if (e + j < 2 * r.pairs) {
          turn(b[j], f[j], s[j], c[j], &u, &v);
          f[j] = v;
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (e / 2 + k < r.pairs) {
          const float p = f[2 * k], q = f[2 * k + 1];
          turn(p, q, s[k], c[k], &f[2 * k], &f[2 * k + 1]);
        }
      }
    }
  }
};

// append_page's change of a page's keys
template <int DT, int D, int PAGE, bool HALVES> struct Turned {
  static constexpr bool kChanges = true;
  using S = Share<D, PAGE>;
  using T = typename Elem<DT>::T;
  const TurnArgs& r;
  __device__ __forceinline__ void operator()(float (&f)[S::PER][8], const void* src, int64_t sh, int64_t st, int64_t row, int had, int end) const {
    const int tid = threadIdx.x;
    Column<DT, D, HALVES> col;
    col.init(r, S::entry(tid), r.k_weight);
#pragma unroll
    for (int i = 0; i < S::PER; ++i) {
      const int t = S::token(tid, i);
      if (t >= had && t < end) {
        float s[Column<DT, D, HALVES>::P], c[Column<DT, D, HALVES>::P], b[8];
        col.partners(r, static_cast<const T*>(src) + (row + t) * st + sh, b);
        col.sincos(r, row + t, s, c);
        col.apply(r, f[i], b, s, c);
      } else {  // a neighbour's row was read: it is not written, and must not count
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = 0.0f;
      }
    }
  }
};

struct AppendGrid {
  int64_t kv_items;          // workgroups of keys and values, for each sequence
  int64_t first;             // the launch's first workgroup
  int32_t tokens_log, per;   // queries: tokens of a workgroup; heads of a thread
  int32_t q_groups;          // workgroups that share a sequence's tokens
};

template <int DT, int D, int PAGE, bool HALVES>
__global__ __launch_bounds__(threads_for(D* PAGE)) void k_append_rope(const KvCache c, const KvTokens x, const TurnArgs r, const AppendGrid g) {
  using S = Share<D, PAGE>;
  using T = typename Elem<DT>::T;
  __shared__ PageSpace<D, PAGE> space;
  const int b = blockIdx.y;
  const int64_t all_items = g.first + blockIdx.x;
  if (all_items < g.kv_items) {
    const int64_t page = all_items / (2 * c.heads);
    const int what = static_cast<int>(all_items - page * (2 * c.heads)), head = what >> 1;
    if (what & 1) append_page<DT, D, PAGE>(c, x, b, head, true, page, space, Unchanged{});
    else append_page<DT, D, PAGE>(c, x, b, head, false, page, space, Turned<DT, D, PAGE, HALVES>{r});
    return;
  }
  const int64_t item = all_items - g.kv_items, tile = item / g.q_groups;
  constexpr int COLS = D / 8;
  const int slot = threadIdx.x / COLS, tokens = 1 << g.tokens_log, slots = S::NT / COLS >> g.tokens_log;
  const int64_t token = tile * tokens + (slot & (tokens - 1));
  const int h0 = (static_cast<int>(item - tile * g.q_groups) * slots + (slot >> g.tokens_log)) * g.per;
  const int h1 = min(h0 + g.per, r.q.heads);
  int64_t row0;
  int32_t rows, all;
  rows_of(x.cu, x.total, c.batch, x.max_rows, b, &row0, &rows, &all);
  if (token >= rows || h0 >= h1) return;
  const int64_t row = row0 + token;
  Column<DT, D, HALVES> col;
  col.init(r, threadIdx.x % COLS * 8, r.q_weight);
  float s[Column<DT, D, HALVES>::P], cs[Column<DT, D, HALVES>::P];
  col.sincos(r, row, s, cs);
#pragma unroll 2
  for (int h = h0; h < h1; ++h) {
    const T* from = static_cast<const T*>(r.q.x) + row * r.q.xt + h * r.q.xh;
    T* to = static_cast<T*>(r.q.y) + row * r.q.yt + h * r.q.yh;
    float f[8], p[8];
    Vec<DT, DT == kF32 ? 4 : 8>::load(from, col.e, f);
    if constexpr (DT == kF32) Vec<DT, 4>::load(from, col.e + 4, f + 4);
    col.partners(r, from, p);
    col.apply(r, f, p, s, cs);
    Vec<DT, DT == kF32 ? 4 : 8>::store(to, col.e, f);
    if constexpr (DT == kF32) Vec<DT, 4>::store(to, col.e + 4, f + 4);
  }
}

template <int DT, int D, int PAGE, bool HALVES> int launch(const KvCache& c, const KvTokens& x, const TurnArgs& r, hipStream_t stream) {
  constexpr int NT = threads_for(D * PAGE), SLOTS = NT / (D / 8);
  AppendGrid g{};
  // pages that max_rows tokens in a row can touch; nothing is written behind the table
  g.kv_items = std::min<int64_t>((static_cast<int64_t>(x.max_rows) + PAGE - 2) / PAGE + 1, c.max_pages) * 2 * c.heads;
  int64_t q_items = 0;
  if (r.q.heads) {
    while ((1 << g.tokens_log) < SLOTS && (1 << g.tokens_log) < x.max_rows) ++g.tokens_log;
    const int slots = SLOTS >> g.tokens_log;
    const int64_t tiles = (static_cast<int64_t>(x.max_rows) + (1 << g.tokens_log) - 1) >> g.tokens_log;
    // heads that share a thread's sines: as many as leave the card full
    const int64_t fill = static_cast<int64_t>(device_cus()) * 2048 / NT;
    g.per = static_cast<int32_t>(std::min<int64_t>(8, std::max<int64_t>(1, tiles * c.batch * r.q.heads / slots / fill)));
    g.q_groups = (r.q.heads + slots * g.per - 1) / (slots * g.per);
    q_items = tiles * g.q_groups;
  }
  constexpr int64_t kMost = (int64_t{1} << 31) / NT;  // workgroups of a launch: 2^31 threads
  for (; g.first < g.kv_items + q_items; g.first += kMost) {
    const dim3 grid(static_cast<uint32_t>(std::min(kMost, g.kv_items + q_items - g.first)), c.batch);
    hipLaunchKernelGGL((k_append_rope<DT, D, PAGE, HALVES>), grid, dim3(NT), 0, stream, c, x, r, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return static_cast<int>(e);
  }
  return static_cast<int>(hipSuccess);
}

template <int DT, int D> int by_page(const KvCache& c, const KvTokens& x, const TurnArgs& r, hipStream_t stream) {
  switch (c.page) {
    case 16: return r.halves ? launch<DT, D, 16, true>(c, x, r, stream) : launch<DT, D, 16, false>(c, x, r, stream);
    case 32: return r.halves ? launch<DT, D, 32, true>(c, x, r, stream) : launch<DT, D, 32, false>(c, x, r, stream);
    case 64: return r.halves ? launch<DT, D, 64, true>(c, x, r, stream) : launch<DT, D, 64, false>(c, x, r, stream);
    default: return r.halves ? launch<DT, D, 128, true>(c, x, r, stream) : launch<DT, D, 128, false>(c, x, r, stream);
  }
}

template <int DT> int by_d(const KvCache& c, const KvTokens& x, const TurnArgs& r, hipStream_t stream) {
  switch (c.d) {
    case 64: return by_page<DT, 64>(c, x, r, stream);
    case 128: return by_page<DT, 128>(c, x, r, stream);
    default: return by_page<DT, 256>(c, x, r, stream);
  }
}

}  // namespace
}  // namespace orbq
