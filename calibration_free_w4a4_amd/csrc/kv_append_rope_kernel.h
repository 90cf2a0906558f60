// kv_append_rope: keys are normalised (where the model says so), turned by their positions, quantised and written behind
// what the cache holds; values are quantised and written; queries are normalised, turned and written out.  One launch.
//
//   q' = turn(q f_q w_q), k' = turn(k f_k w_k),  f = 1 / sqrt(mean of the head's squares + eps) or 1
//
// then k' and v go through kv_append's rule (kv_cache.hip).  k' is quantised from its fp32 value: it is rounded once, to
// its code.  Every element is read once and written once.
//
// A workgroup has a touched page: keys of some heads, and queries of some, which share the sines and cosines of its tokens; or
// values of some heads.  A thread's column of 8 entries holds whole pairs, or in the split-half order has its partners in
// a second column, which it reads too (from L1: a row's lanes are in one wave).  A head's sum of squares is taken over the
// D / 8 lanes that hold the row, and its pairs' sines are dealt out to them, at most four each, and exchanged through LDS.
// Where a sequence has few new tokens every head has workgroups of its own, and queries others whose rows are heads: a
// page of them would be nearly empty.
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

template <int DT> __device__ __forceinline__ void load8(const void* p, int at, float* f) {
  Vec<DT, DT == kF32 ? 4 : 8>::load(p, at, f);
  if constexpr (DT == kF32) Vec<DT, 4>::load(p, at + 4, f + 4);
}
template <int DT> __device__ __forceinline__ void store8(void* p, int at, const float* f) {
  Vec<DT, DT == kF32 ? 4 : 8>::store(p, at, f);
  if constexpr (DT == kF32) Vec<DT, 4>::store(p, at + 4, f + 4);
}

// 1 / sqrt(v) to an ulp, also of a denormal number, which the instruction takes for zero
__device__ __forceinline__ float inverse_root(float v) {
  const bool small = v < 0x1p-126f;
  return __builtin_amdgcn_rsqf(small ? v * 0x1p64f : v) * (small ? 0x1p32f : 1.0f);
}

// LDS of a wave: sines and cosines of the tokens of its rows (512 / D rows of D / 2 pairs at most, SETS times), and their entries.
template <int SETS> struct WaveSpace {
  float2 sines[SETS][256];
  float entries[512];
};

// A thread's column of a head: entries e .. e + 7, and what normalises and turns them.  In pairs' order it has both entries of
// each pair.  In split halves the partner of entry i < pairs is i + pairs: the lanes that hold the row exchange their
// normalised entries through LDS, and of the turn (lo cos - hi sin, lo sin + hi cos) each computes its own side.
template <int DT, int D, bool HALVES> struct Column {
  using T = typename Elem<DT>::T;
  static constexpr int L = D / 8;  // lanes of a row
  static constexpr int F = HALVES ? 8 : 4;
  int e;
  bool normed;
  float w[8];  // weights of the norm

  struct Factors {  // pairs: cosine and sine of pair j.  HALVES: entry j is x a + y b, see apply
    float a[F], b[F];
  };

  __device__ __forceinline__ void weigh(const float* weight) {
    normed = weight != nullptr;
    if (normed) __builtin_memcpy(w, weight + e, sizeof(w));
  }

  // The sines and cosines of a row's token, dealt out to the lanes that hold the row: at most four pairs each.  Rows of a wave
  // that have none are not here; the others' lanes all are.
  static __device__ __forceinline__ void deal(const TurnArgs& r, int64_t row, float2* space) {
    const float* pos = r.pos + (row < r.n_pos ? row : row % r.n_pos) * r.axes;
    const int lane = threadIdx.x & 63, share = (r.pairs + L - 1) / L;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int pair = lane % L * share + k;
      if (k < share && pair < r.pairs) {
        float2 v;
        pair_sincos(r, pos, pair, &v.x, &v.y);
        space[lane / L * r.pairs + pair] = v;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  // the column's factors, from there
  __device__ __forceinline__ void take(const TurnArgs& r, const float2* space, Factors* f) const {
    space += (threadIdx.x & 63) / L * r.pairs;
#pragma unroll
    for (int j = 0; j < F; ++j) {
      if constexpr (HALVES) {
        const int i = e + j, pair = i < r.pairs ? i : i - r.pairs;
        const float2 v = space[min(pair, r.pairs - 1)];
        f->a[j] = i < r.pairs ? v.y : v.x;
        f->b[j] = i < r.pairs ? -v.x : v.y;
      } else {
        const float2 v = space[min(e / 2 + j, r.pairs - 1)];
        f->a[j] = v.y;
        f->b[j] = v.x;
      }
    }
  }
  __device__ __forceinline__ void factors(const TurnArgs& r, int64_t row, float2* space, Factors* f) const {
    if (!HALVES && r.pairs == D / 2) {  // a lane's pairs are its own
      const float* pos = r.pos + (row < r.n_pos ? row : row % r.n_pos) * r.axes;
#pragma unroll
      for (int k = 0; k < F; ++k) pair_sincos(r, pos, e / 2 + k, &f->b[k], &f->a[k]);
      return;
    }
    deal(r, row, space);
    take(r, space, f);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // read before the next are written
  }

  // x: the column's entries, normalised and turned in place
  __device__ __forceinline__ void apply(const TurnArgs& r, const Factors& f, float* space, float* x) const {
    if (normed) {
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(x[j], x[j], sum);
      const float unit = inverse_root(lanes_sum<L>(sum) * (1.0f / D) + r.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] * w[j] * unit;
    }
    if constexpr (HALVES) {
      float* mine = space + (threadIdx.x & 63) / L * D;
      *reinterpret_cast<f32x4_t*>(mine + e) = f32x4_t{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4_t*>(mine + e + 4) = f32x4_t{x[4], x[5], x[6], x[7]};
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      float other[8];
      if (r.pairs % 8 == 0) {  // the partners are a column
        const float* p = mine + (e < r.pairs ? e + r.pairs : (e < 2 * r.pairs ? e - r.pairs : e));
        const f32x4_t u = *reinterpret_cast<const f32x4_t*>(p), v = *reinterpret_cast<const f32x4_t*>(p + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          other[j] = u[j];
          other[4 + j] = v[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = e + j;
          other[j] = mine[i < r.pairs ? i + r.pairs : (i < 2 * r.pairs ? i - r.pairs : i)];
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // read before the next are written
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = e + j;
        const bool first = i < r.pairs;
        const float lo = first ? x[j] : other[j], hi = first ? other[j] : x[j];
        float b = hi * f.b[j];
        asm("" : "+v"(b));  // rounded by itself, the other product with the sum: as rope does
        float y = __builtin_fmaf(lo, f.a[j], b);
        asm("" : "+v"(y));  // an fp32 value, then the output type: not one rounding of both
        x[j] = i < 2 * r.pairs ? y : x[j];
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float u, v;
        turn(x[2 * k], x[2 * k + 1], f.b[k], f.a[k], &u, &v);
        const bool in = e / 2 + k < r.pairs;
        x[2 * k] = in ? u : x[2 * k];
        x[2 * k + 1] = in ? v : x[2 * k + 1];
      }
    }
  }
};

// What turns the tokens of a page that a thread holds.  Their sines are found once for all the heads: in pairs' order they stay in
// registers, in split halves, of which a thread would hold twice as many, in LDS; pages of which a thread has more than
// four columns find them again for each head.
template <int DT, int D, int PAGE, bool HALVES> struct Turned {
  static constexpr bool kChanges = true;
  using S = Share<D, PAGE>;
  using C = Column<DT, D, HALVES>;
  using T = typename Elem<DT>::T;
  static constexpr bool kKeep = S::PER <= 4;
  using Space = WaveSpace<HALVES && kKeep ? S::PER : 1>;

  const TurnArgs& r;
  const PageSpot& spot;
  Space& space;
  C col;
  typename C::Factors held[!HALVES && kKeep ? S::PER : 1];

  __device__ __forceinline__ bool fresh(int i) const {
    const int t = S::token(threadIdx.x, i);
    return t >= spot.had && t < spot.end;
  }
  __device__ __forceinline__ int64_t row(int i) const {  // of a token that is not new: a neighbour's
    const int t = S::token(threadIdx.x, i);
    return spot.base + (t < spot.had ? spot.had : (t >= spot.end ? spot.end - 1 : t));
  }
  __device__ __forceinline__ void prepare() {
    if constexpr (kKeep) {
#pragma unroll
      for (int i = 0; i < S::PER; ++i) {
        if (!fresh(i)) continue;
        if constexpr (HALVES) C::deal(r, row(i), space.sines[i]);
        else col.factors(r, row(i), space.sines[0], &held[i]);
      }
    }
  }
  __device__ __forceinline__ void turn_token(int i, float* x) const {
    if constexpr (!HALVES && kKeep) {
      col.apply(r, held[i], space.entries, x);
    } else {
      typename C::Factors f;
      if constexpr (HALVES && kKeep) col.take(r, space.sines[i], &f);
      else col.factors(r, row(i), space.sines[0], &f);
      col.apply(r, f, space.entries, x);
    }
  }
  // append_page's change: the keys of a head
  __device__ __forceinline__ void operator()(float (&f)[S::PER][8]) const {
#pragma unroll
    for (int i = 0; i < S::PER; ++i) {
      if (fresh(i)) {
        turn_token(i, f[i]);
      } else {  // it is not written, and must not count
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = 0.0f;
      }
    }
  }
  // the queries of heads h, h + step, ...: a few at a time where a thread has few tokens
  __device__ __forceinline__ void queries(int h, int step) const {
    constexpr int G = S::PER < 4 ? S::PER : 4, H = 4 / G;
    for (; h < r.q.heads; h += H * step) {
#pragma unroll
      for (int i0 = 0; i0 < S::PER; i0 += G) {
        float x[H][G][8];
#pragma unroll
        for (int k = 0; k < H; ++k)
#pragma unroll
          for (int i = 0; i < G; ++i)  // a head that is not there: one that is
            load8<DT>(static_cast<const T*>(r.q.x) + min(h + k * step, r.q.heads - 1) * r.q.xh + row(i0 + i) * r.q.xt, col.e, x[k][i]);
#pragma unroll
        for (int i = 0; i < G; ++i) {
          if (!fresh(i0 + i)) continue;
#pragma unroll
          for (int k = 0; k < H; ++k) {
            if (h + k * step >= r.q.heads) continue;
            turn_token(i0 + i, x[k][i]);
            store8<DT>(static_cast<T*>(r.q.y) + (h + k * step) * r.q.yh + row(i0 + i) * r.q.yt, col.e, x[k][i]);
          }
        }
      }
    }
  }
};

// The registers of four waves a SIMD for pages of which a thread has up to four columns (4680 tokens, 12 + 12 heads of 128: 20.4 us,
// with what the compiler takes by itself, three waves, 23.4; five 31.5), what they need for larger ones.
constexpr int waves_for(int bytes) { return bytes <= 8192 ? 4 : 1; }
// Queries go with the pages where a sequence may fill one.
constexpr int kPageQueries = 1;
// Waves for each compute unit that the pages' heads are dealt to: fewer share the sines of more heads and the way to the page
// (same call: 12 19.2 us, 8 20.8, 6 26.0, 16 20.4, 24 22.7).
constexpr int kWavesPerCu = 12;

struct AppendGrid {
  int64_t kv_items;          // workgroups of pages, for each sequence
  int64_t first;             // the launch's first workgroup
  int32_t k_groups, v_groups;  // workgroups of a page: keys and queries, values
  int32_t queries;           // the pages' workgroups have the queries too
  // else: tokens of a query workgroup, heads of a thread, workgroups that share a sequence's tokens
  int32_t tokens_log, per, q_groups;
};

template <int DT, int D, int PAGE, bool HALVES>
__global__ __launch_bounds__(threads_for(D* PAGE), waves_for(D* PAGE)) void k_append_rope(const KvCache c, const KvTokens x, const TurnArgs r, const AppendGrid g) {
  using S = Share<D, PAGE>;
  using C = Column<DT, D, HALVES>;
  using T = typename Elem<DT>::T;
  __shared__ PageSpace<D, PAGE> space;
  using Turn = Turned<DT, D, PAGE, HALVES>;
  __shared__ typename Turn::Space spaces[S::NT / 64];
  const int b = blockIdx.y;
  typename Turn::Space& mine = spaces[threadIdx.x >> 6];
  const int64_t all_items = g.first + blockIdx.x;
  if (all_items < g.kv_items) {
    const int groups = g.k_groups + g.v_groups;
    const int64_t page = all_items / groups;
    const int group = static_cast<int>(all_items - page * groups);
    PageSpot spot;
    if (group >= g.k_groups) {
      if (!locate_page<PAGE>(c, x, b, page, &spot)) return;
      for (int h = group - g.k_groups; h < c.heads; h += g.v_groups) {
        append_page<DT, D, PAGE>(c, x, spot, h, true, space, Unchanged{});
        __syncthreads();  // before the next head takes the space
      }
      return;
    }
    Turn turned{r, spot, mine, C{S::entry(threadIdx.x)}, {}};
    turned.col.weigh(r.k_weight);
    if (!locate_page<PAGE, true>(c, x, b, page, &spot)) return;
    turned.prepare();
    for (int h = group; h < c.heads; h += g.k_groups) {
      append_page<DT, D, PAGE>(c, x, spot, h, false, space, turned);
      __syncthreads();
    }
    if (g.queries) {
      turned.col.weigh(r.q_weight);
      turned.queries(group, g.k_groups);
    }
    return;
  }
  const int64_t item = all_items - g.kv_items, tile = item / g.q_groups;
  constexpr int COLS = D / 8;
  const int slot = threadIdx.x / COLS, tokens = 1 << g.tokens_log, slots = S::NT / COLS >> g.tokens_log;
  const int64_t token = tile * tokens + (slot & (tokens - 1));
  const int h0 = (static_cast<int>(item - tile * g.q_groups) * slots + (slot >> g.tokens_log)) * g.per;
  const int h1 = min(h0 + g.per, r.q.heads);
  C col{static_cast<int>(threadIdx.x % COLS * 8)};
  col.weigh(r.q_weight);
  int64_t row0;
  int32_t rows, all;
  rows_of(x.cu, x.total, c.batch, x.max_rows, b, &row0, &rows, &all);
  if (token >= rows || h0 >= h1) return;
  const int64_t row = row0 + token;
  float entries[8], next[8];
  typename C::Factors factors;
  const T* from = static_cast<const T*>(r.q.x) + row * r.q.xt;
  load8<DT>(from + h0 * r.q.xh, col.e, entries);  // under way while the sines are found
  col.factors(r, row, mine.sines[0], &factors);
  for (int h = h0; h < h1; ++h) {
    load8<DT>(from + min(h + 1, h1 - 1) * r.q.xh, col.e, next);
    col.apply(r, factors, mine.entries, entries);
    store8<DT>(static_cast<T*>(r.q.y) + row * r.q.yt + h * r.q.yh, col.e, entries);
#pragma unroll
    for (int j = 0; j < 8; ++j) entries[j] = next[j];
  }
}

template <int DT, int D, int PAGE, bool HALVES> int launch(const KvCache& c, const KvTokens& x, const TurnArgs& r, hipStream_t stream) {
  constexpr int NT = threads_for(D * PAGE), SLOTS = NT / (D / 8);
  AppendGrid g{};
  // pages that max_rows tokens in a row can touch; nothing is written behind the table
  const int64_t touched = (static_cast<int64_t>(x.max_rows) + PAGE - 2) / PAGE + 1, pages = std::min<int64_t>(touched, c.max_pages);
  g.queries = r.q.heads && x.max_rows >= kPageQueries * PAGE && pages == touched;
  g.k_groups = g.v_groups = c.heads;
  int64_t q_items = 0;
  if (g.queries) {
    // as many workgroups as keep the card busy, dealt to keys and queries, and values, by their shares of the bytes
    const int64_t waves = static_cast<int64_t>(device_cus()) * kWavesPerCu;
    const int64_t groups = std::max<int64_t>(2, waves * 64 / NT / std::max<int64_t>(1, pages * c.batch));
    const int most = std::max(c.heads, r.q.heads);
    g.v_groups = static_cast<int32_t>(std::min<int64_t>(c.heads, std::max<int64_t>(1, groups * c.heads / (2 * c.heads + r.q.heads))));
    g.k_groups = static_cast<int32_t>(std::min<int64_t>(most, std::max<int64_t>(1, groups - g.v_groups)));
  } else if (r.q.heads) {
    while ((1 << g.tokens_log) < SLOTS && (1 << g.tokens_log) < x.max_rows) ++g.tokens_log;
    const int slots = SLOTS >> g.tokens_log;
    const int64_t tiles = (static_cast<int64_t>(x.max_rows) + (1 << g.tokens_log) - 1) >> g.tokens_log;
    // heads that share a thread's sines: as many as leave the card full
    const int64_t fill = static_cast<int64_t>(device_cus()) * 2048 / NT;
    g.per = static_cast<int32_t>(std::min<int64_t>(8, std::max<int64_t>(1, tiles * c.batch * r.q.heads / slots / fill)));
    g.q_groups = (r.q.heads + slots * g.per - 1) / (slots * g.per);
    q_items = tiles * g.q_groups;
  }
  g.kv_items = pages * (g.k_groups + g.v_groups);
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
