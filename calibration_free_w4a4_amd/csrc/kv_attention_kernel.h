// Attention over the 8-bit paged cache.  For query row r (one token, one head; the `group` query
// heads of one cache head are rows of the same tile, so that keys and values are read once for
// all of them):
//   S_j = scale q . k_j,  O = sum_j softmax(S)_j v_j  over the visible keys lo <= j < hi,
//   k_j = kc_j ks[block of j],  v_j = vc_j vs[block of j].
//
// Both products run on the matrix cores in f16 with fp32 accumulation, on the codes themselves: a
// code is exact in f16, q enters as q 2^-e with 2^e its row's magnitude (exact but for entries below
// 2^-14 of the row's largest, which are rounded by 2^-25 of it at most), and the key scale joins the softmax's
// own factor.  The value scale goes into the exponent:
//   w_j = exp2(S_j log2(e) + log2(vs_j) - m),  m the running maximum of S_j log2(e) + log2(vs_j),
//   O = sum_j w_j vc_j / l,  l = sum over blocks (1/vs) sum_j w_j,
// so no element is multiplied by a scale and the rounding of w to f16 is relative to the row's largest
// weight whatever the scales are.  m, l and O are fp32.  m may lag behind the true maximum, which saves most of the
// rescaling of O: it is set 2^kRise below the largest weight and set again when a weight passes 2^kSlack.  What f16
// holds above that is used for the small ones: a weight is rounded by half a unit of its 11 bits or, below 2^-14, by
// 2^-25, which is 2^-28 of the row's largest or less (with m at the maximum itself it would be 2^-25: 60000 keys at
// 2^-25.4 of one large one were lost altogether, and now lose 1 % of their share).
// The exponent is one fused operation on the raw score and log2(vs_j) - m, both rounded apart: a relative error of
// 2^-24 of the score each, which the row's sum shares.  With scores to 2^25 it adds 4 to the 11 of kSlack at most, and
// w stays within f16 (2^16); subtracting rounded scores instead would need no such limit and one more
// instruction for each weight.
//
// The products are taken transposed: S^T = K Q^T has one query row a lane and its keys down the
// accumulator registers, which is, up to an order of the keys that the values follow, the layout in
// which O^T = V^T w^T takes its second operand.  The weights never leave their registers, and m, l and
// the rescaling factors are one value a lane.
//
// Two forms:
//   few   up to 64 rows, 16 or 32 a workgroup (token-by-token serving): bound by the cache's bytes.  Four waves, or
//         eight for a short cache, take 64-key tiles in turn straight from memory into registers, and are
//         joined at the end.
//   many  128 or 256 rows a workgroup: bound by the matrix cores, the softmax's vector work and the LDS reads
//         between them.  Codes are turned into f16 once a workgroup on their way into LDS, double
//         buffered, or once a call by k_turn, and then fetched into LDS as they are.
// Either splits the keys over workgroups, few where there are few rows, many where the last round of workgroups
// would leave CUs idle; k_join joins the parts.
//
// Measured: few, one token of 48 sequences to 16384 long, 32 / 8 heads of 128: 169 us and 6 of joining, 5.1 TB/s of
// cache; 4 tokens over 262157, 64 / 8 heads of 64: 60 us, 6 of them joining, 4.5 TB/s.  many, 4680 queries over 32760
// tokens, 12 heads of 128: 0.94 ms, 0.95 PFLOP/s (a library f16 product of 8192^3 on such a card: 1.20); heads of 256,
// 2 x 4605 queries that all see all: 444 us, 0.78 PFLOP/s; heads of 64, ragged prompts with a window of 1024: 83 us,
// 0.43 PFLOP/s.
#pragma once

#include <algorithm>

#include "attention_device.h"

namespace orbq {
namespace attn {

constexpr float kSlack = 11.0f;      // log2 of what a weight may reach before O is rescaled
constexpr float kRise = 3.0f;        // log2 of the largest weight then
constexpr float kNone = -1.0e30f;    // running maximum before the first visible key
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// the larger one, or a NaN where either is: one instruction takes two of them, and unlike fmax it needs none that
// quiet its operands first
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// x of this lane and of the lane 32 (16) away, combined: one vector instruction, where a shuffle would go through LDS
__device__ __forceinline__ float max_over32(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return larger(__builtin_bit_cast(float, static_cast<uint32_t>(r[0])), __builtin_bit_cast(float, static_cast<uint32_t>(r[1])));
}
__device__ __forceinline__ float max_over16(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return larger(__builtin_bit_cast(float, static_cast<uint32_t>(r[0])), __builtin_bit_cast(float, static_cast<uint32_t>(r[1])));
}

// four signed codes -> f16: byte u = code + 128 behind 0x64 is 1024 + u, less 1152 is the code
__device__ __forceinline__ void codes_to_f16(uint32_t q, half2_t* lo, half2_t* hi) {
  const uint32_t u = q ^ 0x80808080u;
  const half2_t bias = {static_cast<_Float16>(-1152.0f), static_cast<_Float16>(-1152.0f)};
  *lo = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) + bias;
  *hi = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) + bias;
}

__device__ __forceinline__ half8_t codes_to_half8(uint32_t a, uint32_t b) {
  half2_t h[4];
  codes_to_f16(a, &h[0], &h[1]);
  codes_to_f16(b, &h[2], &h[3]);
  return half8_t{h[0][0], h[0][1], h[1][0], h[1][1], h[2][0], h[2][1], h[3][0], h[3][1]};
}

__device__ __forceinline__ half8_t load_q8(const AttnArgs& a, int64_t at) {
  const u32x4_t w = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a.q) + at);
  return __builtin_bit_cast(half8_t, w);  // raw bits; q_scaled reads them by type
}

// eight q entries of either type, times `by`, in f16
__device__ __forceinline__ half8_t q_scaled(half8_t raw, bool f16, float by) {
  half8_t r;
  const u32x4_t w = __builtin_bit_cast(u32x4_t, raw);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = f16 ? static_cast<float>(raw[i])
                        : __builtin_bit_cast(float, (i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
    r[i] = static_cast<_Float16>(x * by);
  }
  return r;
}

__device__ __forceinline__ float q_most(half8_t raw, bool f16) {
  const u32x4_t w = __builtin_bit_cast(u32x4_t, raw);
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = f16 ? static_cast<float>(raw[i])
                        : __builtin_bit_cast(float, (i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
    m = __builtin_fmaxf(m, __builtin_fabsf(x));
  }
  return m;
}

// 2^e with 2^e <= most < 2^(e+1), within [2^-100, 2^126]; 1 for an infinite row
__device__ __forceinline__ float row_power(float most) {
  const int e = static_cast<int>(__builtin_bit_cast(uint32_t, most) >> 23) - 127;
  const int k = e > 127 ? 0 : (e < -100 ? -100 : (e > 126 ? 126 : e));
  return __builtin_bit_cast(float, static_cast<uint32_t>(k + 127) << 23);
}

// first and one past the last visible key of the query at `pos`
__device__ __forceinline__ void visible(const AttnArgs& a, int64_t pos, int32_t len, int32_t* lo, int32_t* hi) {
  int64_t h = len;
  if (a.causal_block) {
    const int64_t end = pos < 0 ? 0 : (static_cast<int64_t>(static_cast<uint32_t>(pos) / static_cast<uint32_t>(a.causal_block)) + 1) *
                                          a.causal_block;
    h = end < h ? end : h;
  }
  *hi = static_cast<int32_t>(h);
  *lo = a.window && h > a.window ? static_cast<int32_t>(h - a.window) : 0;
}

struct Seq {
  int64_t row0;   // first packed query
  int32_t rows;   // queries that are processed
  int32_t all;    // queries, max_new or not: the first stands at len - all
  int32_t len;    // cached tokens, within the table
};

__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
  Seq s;
  rows_of(a.cu, a.total, a.c.batch, a.max_new, b, &s.row0, &s.rows, &s.all);
  const int64_t most = static_cast<int64_t>(a.c.max_pages) << a.page_shift;
  const int32_t n = a.lens[b];
  s.len = n < 0 ? 0 : (n > most ? static_cast<int32_t>(most) : n);
  return s;
}

// one value a lane that covers a block's keys: c = ks |scale| log2(e), log2(vs), 1/vs; a block that is absent
// has no weight.  The value scale is kept finite: a block before the window may hold anything, and an infinite
// logarithm would turn the -infinity of its masked scores into a NaN.
__device__ __forceinline__ void block_scales(const AttnArgs& a, float ks, float vs, bool have, float* c, float* lv, float* iv) {
  const float v = __builtin_fminf(__builtin_fmaxf(vs, kScaleFloor), kScaleMost);
  *c = have ? ks * a.scale_log2e : 0.0f;
  *lv = have ? __builtin_amdgcn_logf(v) : -__builtin_inff();  // log2, exact to a unit of its last place for a normal number
  *iv = have ? __builtin_amdgcn_rcpf(v) : 0.0f;
}

__device__ __forceinline__ void store4(const AttnArgs& a, int64_t at, f32x4_t v) {
  uint16_t* o = static_cast<uint16_t*>(a.o);
  if (a.f16) Vec<kF16, 4>::store(o, at, reinterpret_cast<const float*>(&v));
  else Vec<kBF16, 4>::store(o, at, reinterpret_cast<const float*>(&v));
}

// ------------------------------------------------------------------------------------------ few
template <int D, int RT, int NW> __global__ __launch_bounds__(64 * NW) void k_few(const AttnArgs a) {
  constexpr int NC = D / 64, ND = D / 16;
  __shared__ __attribute__((aligned(16))) f32x4_t join_o[NW][RT][ND][64];
  __shared__ float join_m[NW][RT][16], join_l[NW][RT][16];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, l15 = lane & 15, g = lane >> 4;
  const int split = blockIdx.x, kvh = blockIdx.y / a.row_tiles, tile = blockIdx.y - kvh * a.row_tiles, b = blockIdx.z;
  const Seq s = seq_of(a, b);
  const int all = s.rows * a.group, r0 = tile * 16 * RT;
  if (r0 >= all) return;
  const int r1 = r0 + 16 * RT < all ? r0 + 16 * RT : all;

  // the rows' keys
  int32_t lo[RT], hi[RT], lo_most, hi_least, first, last;
  visible(a, static_cast<int64_t>(s.len) - s.all + r0 / a.group, s.len, &first, &hi_least);
  visible(a, static_cast<int64_t>(s.len) - s.all + (r1 - 1) / a.group, s.len, &lo_most, &last);
  const int t_first = first / 64, t_end = (last + 63) / 64;
  const int t0 = t_first + split * a.chunk;
  const int t1 = split + 1 < a.splits && t0 + a.chunk < t_end ? t0 + a.chunk : t_end;
  if (a.splits > 1 && t0 >= t1) {  // nothing here: an empty part
    for (int i = tid; i < r1 - r0; i += 64 * NW) {
      const int r = r0 + i;
      const int64_t row = (s.row0 + r / a.group) * a.heads + kvh * a.group + r % a.group;
      float* ml = a.part_ml + (row * a.splits + split) * 2;
      ml[0] = kNone;
      ml[1] = 0.0f;
    }
    return;
  }

  f32x4_t o[RT][ND];
  float m[RT], l[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = kNone;
    l[rt] = 0.0f;
#pragma unroll
    for (int i = 0; i < ND; ++i) o[rt][i] = f32x4_t{0, 0, 0, 0};
  }

  // This lane's loads of a tile: keys 16 (l15 / 4) + 4 t + l15 % 4, t = 0..3, entries 64 c + 16 g ..
  // + 15; and for values entries 16 i + l15, keys 16 g .. + 15.  Nothing branches: keys past the
  // sequence's end are read and masked, and for a block that is absent the first of the cache is read
  // and has no weight.  The table's entries are loaded a tile earlier and judged when they are used, so that no
  // load is waited for where it is issued.
  const int page_mask = a.c.page - 1;
  const int64_t block_bytes = static_cast<int64_t>(D) * a.c.page;
  const int32_t* table = a.c.table + b * a.c.ldt;
  u32x4_t kr[4][NC], vr[ND];
  const auto entry = [&](int key) {
    const int p = key >> a.page_shift;
    return table[p < a.c.max_pages ? p : a.c.max_pages - 1];
  };
  const auto present = [&](int pg, int key) { return key < s.len && static_cast<uint32_t>(pg) < static_cast<uint32_t>(a.c.pages); };
  const auto slot_of = [&](int pg, int key) {  // pg heads + kvh, an absent block as page 0
    return static_cast<uint64_t>(present(pg, key) ? static_cast<uint32_t>(pg) : 0u) * static_cast<uint32_t>(a.c.heads) + kvh;
  };
  const auto key_of = [&](int t) { return 64 * t + 16 * (l15 >> 2); };
  const auto val_of = [&](int t) { return 64 * t + 16 * g; };
  const int k_off = (l15 & 3) * D + 16 * g, v_off = l15 * a.c.page;
  const auto load_k = [&](int t, int pg) {
    const int key = key_of(t);
    const int8_t* p = a.c.k + slot_of(pg, key) * block_bytes + (key & page_mask) * D + k_off;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c) kr[i][c] = *reinterpret_cast<const u32x4_t*>(p + 4 * i * D + 64 * c);
  };
  const auto load_v = [&](int t, uint64_t slot) {
    const int8_t* p = a.c.v + slot * block_bytes + (val_of(t) & page_mask) + v_off;
#pragma unroll
    for (int i = 0; i < ND; ++i) vr[i] = *reinterpret_cast<const u32x4_t*>(p + 16 * i * a.c.page);
  };

  // The first table entries, q and the first keys are on their way together.
  // q: lane l15 holds row l15, entries 64 c + 16 g + 0..15 as two operands
  int t = t0 + wave;
  int kpg = 0, vpg = 0;  // table entries of the tile to load next
  if (t < t1) {
    kpg = entry(key_of(t));
    vpg = entry(val_of(t));
  }
  half8_t q[RT][NC][2];
  float qs[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = r0 + 16 * rt + l15;
    const bool live = r < r1;
    const int rr = live ? r : r0, tok = rr / a.group, h = kvh * a.group + rr - tok * a.group;
    const int64_t at = (s.row0 + tok) * a.qt + h * a.qh;
    visible(a, static_cast<int64_t>(s.len) - s.all + tok, s.len, &lo[rt], &hi[rt]);
    if (!live) hi[rt] = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) q[rt][c][k] = load_q8(a, at + 64 * c + 16 * g + 8 * k);
  }
  if (t < t1) {
    load_k(t, kpg);
    kpg = entry(key_of(t + NW));
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    float most = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) most = __builtin_fmaxf(most, q_most(q[rt][c][k], a.f16));
    most = max_over32(max_over16(most));
    qs[rt] = row_power(most);
    const float by = (a.negative ? -1.0f : 1.0f) / qs[rt];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) q[rt][c][k] = q_scaled(q[rt][c][k], a.f16, by);
  }
  for (; t < t1; t += NW) {
    const bool have = present(vpg, val_of(t));
    const uint64_t slot = slot_of(vpg, val_of(t));
    load_v(t, slot);
    const float ks = a.c.ks[slot], vs = a.c.vs[slot];
    vpg = entry(val_of(t + NW));
    // S^T: accumulator register 4 i + j of this lane is key 16 g + 4 i + j of row l15
    f32x4_t st[RT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) st[rt][i] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const half8_t k0 = codes_to_half8(kr[i][c][0], kr[i][c][1]), k1 = codes_to_half8(kr[i][c][2], kr[i][c][3]);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          st[rt][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, q[rt][c][0], st[rt][i], 0, 0, 0);
          st[rt][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, q[rt][c][1], st[rt][i], 0, 0, 0);
        }
      }
    }
    load_k(t + NW, kpg);
    kpg = entry(key_of(t + 2 * NW));
    float sc, lv, iv;
    block_scales(a, ks, vs, have, &sc, &lv, &iv);
    const bool whole = 64 * t >= lo_most && 64 * t + 64 <= hi_least;
    half8_t p[RT][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      // positive (zero is taken as the least normal number, so that a masked score stays at -infinity), so
      // that the largest score is the largest weight's
      const float c = __builtin_fmaxf(sc * qs[rt], 0x1p-126f);
      if (!whole) {
        asm volatile("; masked tile");  // keeps this a branch: few tiles take it
        const int k0 = 64 * t + 16 * g;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (k0 + i < lo[rt] || k0 + i >= hi[rt]) st[rt][i >> 2][i & 3] = -__builtin_inff();
      }
      float top = st[rt][0][0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = __builtin_fmaxf(top, st[rt][i >> 2][i & 3]);
      top = __builtin_fmaf(top, c, lv);
      top = max_over32(max_over16(top));
      if (__any(top > m[rt] + kSlack)) {
        const float mn = __builtin_fmaxf(m[rt], top - kRise), by = exp2_fast(m[rt] - mn);
        m[rt] = mn;
        l[rt] *= by;
#pragma unroll
        for (int i = 0; i < ND; ++i) o[rt][i] *= by;
      }
      const float y = lv - m[rt];
      float total = 0.0f;  // of the weights before their rounding: the logarithm of l is an output in 32 bits
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float w = exp2_fast(__builtin_fmaf(st[rt][i >> 2][i & 3], c, y));
        total += w;
        p[rt][i >> 3][i & 7] = static_cast<_Float16>(w);
      }
      l[rt] = __builtin_fmaf(total, iv, l[rt]);
    }
#pragma unroll
    for (int i = 0; i < ND; ++i) {
      const half8_t v0 = codes_to_half8(vr[i][0], vr[i][1]), v1 = codes_to_half8(vr[i][2], vr[i][3]);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        o[rt][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p[rt][0], o[rt][i], 0, 0, 0);
        o[rt][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p[rt][1], o[rt][i], 0, 0, 0);
      }
    }
  }

  // join the waves
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    l[rt] += __shfl_xor(l[rt], 16);
    l[rt] += __shfl_xor(l[rt], 32);
    if (g == 0) {
      join_m[wave][rt][l15] = m[rt];
      join_l[wave][rt][l15] = l[rt];
    }
  }
  __syncthreads();
  float mt[RT], lt[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    mt[rt] = kNone;
    lt[rt] = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) mt[rt] = __builtin_fmaxf(mt[rt], join_m[w][rt][l15]);
#pragma unroll
    for (int w = 0; w < NW; ++w) lt[rt] += join_l[w][rt][l15] * exp2_fast(join_m[w][rt][l15] - mt[rt]);
    const float by = exp2_fast(m[rt] - mt[rt]);
#pragma unroll
    for (int i = 0; i < ND; ++i) o[rt][i] *= by;
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int i = 0; i < ND; ++i) join_o[wave][rt][i][lane] = o[rt][i];
  __syncthreads();
  // each wave sums and writes its share of the entries
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = r0 + 16 * rt + l15;
    const bool live = r < r1;
    const int rr = live ? r : r0, tok = rr / a.group, h = kvh * a.group + rr - tok * a.group;
    const int64_t row = (s.row0 + tok) * a.heads + h, at = (s.row0 + tok) * a.ot + h * a.oh;
    float* po = a.part_o + (row * a.splits + split) * D;
    const float by = lt[rt] == 0.0f ? 0.0f : 1.0f / lt[rt];
    for (int i = wave; i < ND; i += NW) {
      f32x4_t x = join_o[0][rt][i][lane];
#pragma unroll
      for (int w = 1; w < NW; ++w) x += join_o[w][rt][i][lane];
      if (!live) continue;
      if (a.splits > 1) *reinterpret_cast<f32x4_t*>(po + 16 * i + 4 * g) = x;
      else store4(a, at + 16 * i + 4 * g, x * by);
    }
    if (wave || g || !live) continue;
    if (a.splits > 1) {
      float* ml = a.part_ml + (row * a.splits + split) * 2;
      ml[0] = mt[rt];
      ml[1] = lt[rt];
    } else if (a.lse) {
      a.lse[row] = lt[rt] == 0.0f ? -__builtin_inff() : (mt[rt] + __builtin_log2f(lt[rt])) * kLn2;
    }
  }
}

// ----------------------------------------------------------------------------------------- many
// TURNED: k_turn has laid the tiles out in f16 before, and they come into LDS as they are.
template <int D, bool TURNED = false> struct Many {
  static constexpr int kRows = many_rows(D), kWaves = kRows / 32, kThreads = 64 * kWaves;
  // LDS of one tile in 16-byte pieces: keys [d / 8][64], values [8][d] (pieces of 8 keys).  A wave's
  // operand reads are 32 consecutive pieces; where threads turn codes themselves, a pitch of 1 and 2 more
  // pieces spreads them over banks.
  static constexpr int kKPitch = TURNED ? 64 : 65, kVPitch = TURNED ? D : D + 2;
  static constexpr int kKPieces = D / 8 * kKPitch, kVPieces = 8 * kVPitch;
  static constexpr int kFactors = TURNED ? 16 : 4;  // 16 bytes each; four are used, the rest is a wave's fetch
  static constexpr int kLoads = 4 * D / kThreads;  // 16-byte loads a thread for a tile's keys, and for its values
};

struct Factors {  // of each 16 keys of a tile: on raw scores, log2 of the value scale, 1 / value scale
  float c[4], lv[4], iv[4];
};

// the first 64-key tile that a sequence's rows see
__device__ __forceinline__ int first_of(const AttnArgs& a, const Seq& s) {
  int32_t lo, hi;
  visible(a, static_cast<int64_t>(s.len) - s.all, s.len, &lo, &hi);
  return lo / 64;
}

// the n-th row tile in the order of the launch
__device__ __forceinline__ int tile_of(const AttnArgs& a, int n, int* b, int* kvh) {
  const int streams = a.c.batch * a.c.heads, turn = n / streams, stream = n - turn * streams;
  *b = stream / a.c.heads;
  *kvh = stream - *b * a.c.heads;
  return a.row_tiles - 1 - turn;
}

// One workgroup's rows, its part of the keys, and one wave's 32 rows of them: lane l31 of either half
// holds row l31.  Everything here is inlined; the members live in registers.
template <int D, bool TURNED = false> struct ManyRows {
  using M = Many<D, TURNED>;
  static constexpr int NS = D / 16, ND = D / 32, NL = M::kLoads;
  const AttnArgs& a;
  half8_t (*lk)[M::kKPieces];   // [2]: tile t in t & 1
  half8_t (*lv)[M::kVPieces];   // [2]
  f32x4_t (*lsc)[M::kFactors];  // [4]: tile t in t & 3; for each 16 keys ks |scale| log2(e), log2(vs), 1 / vs
  int tid, wave, lane, l31, hi32;
  int b, kvh, parts, split, h;  // parts that this row tile's keys are split into
  Seq s;
  bool live;
  int64_t tok, row, part_row;
  int t0, t1;                   // 64-key tiles of this workgroup
  int32_t lo, hi;               // this lane's visible keys
  int32_t all_lo, all_hi;       // keys from all_lo to all_hi are visible to all rows of this wave
  half8_t q[NS];
  float qs, m, l;
  f32x16_t o[ND];
  // staging
  const int32_t* table;
  int64_t block_bytes;
  int page_mask;
  uint32_t k_off[NL], v_off[NL];
  u32x4_t kr[NL], vr[NL];
  int kpg[NL], vpg, spg;        // table entries of the next tiles' keys, values and scales
  float ks, vs;                 // scales of the keys to stage next, of 16 keys a lane (tid < 4)
  bool have;
  // TURNED: this stream's tiles and their factors
  const half8_t* turned;
  const f32x4_t* factors;

  __device__ __forceinline__ ManyRows(const AttnArgs& args, half8_t (*k)[M::kKPieces], half8_t (*v)[M::kVPieces], f32x4_t (*sc4)[M::kFactors])
      : a(args), lk(k), lv(v), lsc(sc4) {}

  // false: this workgroup has no rows
  __device__ __forceinline__ bool begin() {
    tid = threadIdx.x;
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    lane = tid & 63;
    l31 = tid & 31;
    hi32 = (tid >> 5) & 1;
    // Row tiles of all streams (sequence, head) in turn, the last rows, which see most under a causal mask, first;
    // from a.whole on each in a.splits parts.  Keeping a stream on one die instead leaves the dies unevenly loaded
    // where sequences differ (the ragged prompts: 142 us, 82 in this order) and gains nothing where they do not.
    int n = a.first + static_cast<int>(blockIdx.x);
    parts = 1;
    split = 0;
    if (n >= a.whole) {
      parts = a.splits;
      split = (n - a.whole) % parts;
      n = a.whole + (n - a.whole) / parts;
    }
    part_row = static_cast<int64_t>(n - a.whole) * M::kRows;
    const int tile = tile_of(a, n, &b, &kvh);
    s = seq_of(a, b);
    const int64_t all = static_cast<int64_t>(s.rows) * a.group, r0 = static_cast<int64_t>(tile) * M::kRows;
    if (r0 >= all) return false;
    const int64_t r1 = r0 + M::kRows < all ? r0 + M::kRows : all;
    const int64_t base = static_cast<int64_t>(s.len) - s.all;
    int32_t first, last, x;
    visible(a, base + r0 / a.group, s.len, &first, &x);
    visible(a, base + (r1 - 1) / a.group, s.len, &x, &last);
    const int t_end = (last + 63) / 64;
    t0 = first / 64 + split * a.chunk;
    t1 = split + 1 < parts && t0 + a.chunk < t_end ? t0 + a.chunk : t_end;
    const int64_t mine = r0 + 32 * wave + l31;
    part_row += 32 * wave + l31;
    live = mine < r1;
    const int64_t rr = live ? mine : r0;
    tok = rr / a.group;
    h = kvh * a.group + static_cast<int>(rr - tok * a.group);
    row = (s.row0 + tok) * a.heads + h;
    visible(a, base + tok, s.len, &lo, &hi);
    if (!live) hi = 0;
    const int64_t w0 = r0 + 32 * wave < r1 ? r0 + 32 * wave : r1 - 1, w1 = r0 + 32 * wave + 31 < r1 ? r0 + 32 * wave + 31 : r1 - 1;
    visible(a, base + w0 / a.group, s.len, &x, &all_hi);
    visible(a, base + w1 / a.group, s.len, &all_lo, &x);

    const int64_t at = (s.row0 + tok) * a.qt + h * a.qh;
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      q[i] = load_q8(a, at + 16 * i + 8 * hi32);
      most = __builtin_fmaxf(most, q_most(q[i], a.f16));
    }
    most = max_over32(most);
    qs = row_power(most);
    const float by = (a.negative ? -1.0f : 1.0f) / qs;
#pragma unroll
    for (int i = 0; i < NS; ++i) q[i] = q_scaled(q[i], a.f16, by);
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    m = kNone;
    l = 0.0f;
    if constexpr (TURNED) {
      // tile t of the stream is its (t - first_of)th
      const int64_t first_tile = (static_cast<int64_t>(b) * a.c.heads + kvh) * a.turned_tiles - first_of(a, s);
      turned = static_cast<const half8_t*>(a.turned) + first_tile * (16 * D);
      factors = static_cast<const f32x4_t*>(a.factors) + first_tile * 4;
      return true;
    }
    table = a.c.table + b * a.c.ldt;
    block_bytes = static_cast<int64_t>(D) * a.c.page;
    page_mask = a.c.page - 1;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int at = i * M::kThreads + tid;
      k_off[i] = (at / (D / 16) & 15) * D + at % (D / 16) * 16;
      v_off[i] = entry_of(i) * a.c.page;
    }
    return true;
  }

  // Loads of a tile: 16 codes each; keys (key, 16 entries), values (entry, 16 keys).  A wave's load stays
  // within 16 keys, so its page is one scalar and its address one scalar and an offset that never
  // changes.  Nothing branches: where a block is absent the first of the cache is read, and its weight is
  // zero.  The table's entries are loaded a tile earlier and judged when they are used, so that no load is
  // waited for where it is issued.
  __device__ __forceinline__ int entry(int key) const {
    const int p = key >> a.page_shift;
    return table[p < a.c.max_pages ? p : a.c.max_pages - 1];
  }
  __device__ __forceinline__ bool present(int pg, int key) const {
    return key < s.len && static_cast<uint32_t>(pg) < static_cast<uint32_t>(a.c.pages);
  }
  __device__ __forceinline__ uint64_t slot_of(int pg, int key) const {  // pg heads + kvh, an absent block as page 0
    return static_cast<uint64_t>(present(pg, key) ? static_cast<uint32_t>(pg) : 0u) * static_cast<uint32_t>(a.c.heads) + kvh;
  }
  // first of the 16 keys that hold this wave's load i of keys, and of its loads of values
  __device__ __forceinline__ int key_of(int t, int i) const { return 64 * t + ((i * M::kWaves + wave) * (1024 / D) & ~15); }
  __device__ __forceinline__ int val_of(int t) const { return 64 * t + 16 * (wave & 3); }
  // entry of this thread's load i of values
  __device__ __forceinline__ int entry_of(int i) const { return 64 * (i * (M::kWaves / 4) + (wave >> 2)) + lane; }
  __device__ __forceinline__ void pages_k(int t) {
#pragma unroll
    for (int i = 0; i < NL; ++i) kpg[i] = entry(key_of(t, i));
    if (wave == 0) spg = entry(64 * t + 16 * (lane & 3));
  }
  __device__ __forceinline__ void pages_v(int t) { vpg = entry(val_of(t)); }
  __device__ __forceinline__ void load_k(int t) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int key = key_of(t, i);
      const int8_t* p = a.c.k + slot_of(kpg[i], key) * block_bytes + (key & page_mask) * D;
      kr[i] = *reinterpret_cast<const u32x4_t*>(p + k_off[i]);
    }
    if (wave == 0) {
      const int key = 64 * t + 16 * (lane & 3);
      const uint64_t slot = slot_of(spg, key);
      ks = a.c.ks[slot];
      vs = a.c.vs[slot];
      have = present(spg, key);
    }
  }
  __device__ __forceinline__ void load_v(int t) {
    const int key = val_of(t);
    const int8_t* p = a.c.v + slot_of(vpg, key) * block_bytes + (key & page_mask);
#pragma unroll
    for (int i = 0; i < NL; ++i) vr[i] = *reinterpret_cast<const u32x4_t*>(p + v_off[i]);
  }
  __device__ __forceinline__ void stage_k(int t) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int at = i * M::kThreads + tid, key = at / (D / 16), u = at % (D / 16);
      lk[t & 1][(2 * u) * M::kKPitch + key] = codes_to_half8(kr[i][0], kr[i][1]);
      lk[t & 1][(2 * u + 1) * M::kKPitch + key] = codes_to_half8(kr[i][2], kr[i][3]);
    }
    if (tid < 4) {
      float c, x, y;
      block_scales(a, ks, vs, have, &c, &x, &y);
      lsc[t & 3][tid] = f32x4_t{c, x, y, 0.0f};
    }
  }
  __device__ __forceinline__ void stage_v(int t) {
    const int g = wave & 3;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      // keys 0-3 and 8-11 of the sixteen, then 4-7 and 12-15: as the weights lie in their registers
      lv[t & 1][(2 * g) * M::kVPitch + entry_of(i)] = codes_to_half8(vr[i][0], vr[i][2]);
      lv[t & 1][(2 * g + 1) * M::kVPitch + entry_of(i)] = codes_to_half8(vr[i][1], vr[i][3]);
    }
  }

  // TURNED: half a tile, 8 D pieces, straight into LDS by every wave's share of 64 pieces at a time.  The loads
  // are written out because the compiler would wait for all of them before the next LDS read of any kind; they
  // have no register results, and arrived() ends them.
  __device__ __forceinline__ void fetch(const half8_t* from, half8_t* to) const {
#pragma unroll
    for (int i = 0; i < D / 8 / M::kWaves; ++i) {
      const int j = 64 * (i * M::kWaves + wave);
      const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) half8_t*)(to + j)));
      asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from + j + lane),
                   "s"(__builtin_amdgcn_readfirstlane(at))
                   : "memory", "m0");
    }
  }
  // keys, and the tile's factors: 16 words (the other lanes fetch them again, into the room behind).  Loaded where they
  // are used instead, each step would wait for them and for its fetches (frames of 12 heads of 128: 972 us, 958 so).
  __device__ __forceinline__ void fetch_k(int t) const {
    fetch(turned + static_cast<int64_t>(t) * (16 * D), lk[t & 1]);
    if (wave == 0) {
      const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) f32x4_t*)(lsc[t & 3])));
      asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(
                       reinterpret_cast<const float*>(factors + 4 * t) + (lane & 15)),
                   "s"(__builtin_amdgcn_readfirstlane(at))
                   : "memory", "m0");
    }
  }
  __device__ __forceinline__ void fetch_v(int t) const { fetch(turned + static_cast<int64_t>(t) * (16 * D) + 8 * D, lv[t & 1]); }
  __device__ __forceinline__ void arrived() const { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

  // S^T of tile t: register 8 (g & 1) + 4 k + j of st[g / 2] is key 16 g + 8 k + 4 hi32 + j
  __device__ __forceinline__ void scores(int t, f32x16_t* st) const {
#pragma unroll
    for (int j = 0; j < 16; ++j) st[0][j] = st[1][j] = 0.0f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const half8_t k0 = lk[t & 1][(2 * i + hi32) * M::kKPitch + l31], k1 = lk[t & 1][(2 * i + hi32) * M::kKPitch + 32 + l31];
      st[0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k0, q[i], st[0], 0, 0, 0);
      st[1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k1, q[i], st[1], 0, 0, 0);
    }
  }
  // O^T += V^T w^T of tile t
  __device__ __forceinline__ void values(int t, const half8_t* p) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int i = 0; i < ND; ++i)
        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(lv[t & 1][(2 * g + hi32) * M::kVPitch + 32 * i + l31], p[g], o[i], 0, 0, 0);
  }
  // a block's factor on raw scores; positive (zero is taken as the least normal number, so that a masked
  // score stays at -infinity), so that a block's largest weight is its largest score's
  __device__ __forceinline__ float factor(float f) const { return __builtin_fmaxf(f * qs, 0x1p-126f); }
  // masks tile t and finds the exponent of each row's largest weight in it
  __device__ __forceinline__ float largest(int t, f32x16_t* st, Factors* f) const {
    if (64 * t < all_lo || 64 * t + 64 > all_hi) {
      asm volatile("; masked tile");  // keeps this a branch: few tiles take it
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int key = 64 * t + 16 * g + 8 * (j >> 2) + 4 * hi32 + (j & 3);
          if (key < lo || key >= hi) st[g >> 1][8 * (g & 1) + j] = -__builtin_inff();
        }
    }
    float top = -__builtin_inff();
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const f32x4_t x4 = lsc[t & 3][g];
      f->c[g] = factor(x4[0]);
      f->lv[g] = x4[1];
      f->iv[g] = x4[2];
      float x = st[g >> 1][8 * (g & 1)];
#pragma unroll
      for (int j = 1; j < 8; ++j) x = larger(x, st[g >> 1][8 * (g & 1) + j]);
      top = larger(top, __builtin_fmaf(x, f->c[g], f->lv[g]));
    }
    return max_over32(top);
  }
  __device__ __forceinline__ void raise(float top) {
    if (__any(top > m + kSlack)) {
      const float mn = __builtin_fmaxf(m, top - kRise), by = exp2_fast(m - mn);
      m = mn;
      l *= by;
#pragma unroll
      for (int i = 0; i < ND; ++i) o[i] *= by;
    }
  }
  __device__ __forceinline__ void weights(const f32x16_t* st, const Factors& f, half8_t* p) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float y = f.lv[g] - m;
      float total = 0.0f;  // of the weights before their rounding: the logarithm of l is an output in 32 bits
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float w = exp2_fast(__builtin_fmaf(st[g >> 1][8 * (g & 1) + j], f.c[g], y));
        total += w;
        p[g][j] = static_cast<_Float16>(w);
      }
      l = __builtin_fmaf(total, f.iv[g], l);
    }
  }

  __device__ __forceinline__ void finish() {
    l += __shfl_xor(l, 32);
    if (!live) return;
    // register 4 k + j of o[i]: entry 32 i + 8 k + 4 hi32 + j
    if (parts > 1) {
      float* po = a.part_o + (part_row * parts + split) * D;
      if (l != 0.0f) {
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<f32x4_t*>(po + 32 * i + 8 * k + 4 * hi32) =
                f32x4_t{o[i][4 * k], o[i][4 * k + 1], o[i][4 * k + 2], o[i][4 * k + 3]};
      }
      if (hi32 == 0) {
        float* ml = a.part_ml + (part_row * parts + split) * 2;
        ml[0] = m;
        ml[1] = l;
      }
      return;
    }
    const float by = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t at = (s.row0 + tok) * a.ot + h * a.oh;
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        store4(a, at + 32 * i + 8 * k + 4 * hi32,
               f32x4_t{o[i][4 * k] * by, o[i][4 * k + 1] * by, o[i][4 * k + 2] * by, o[i][4 * k + 3] * by});
    if (a.lse && hi32 == 0) a.lse[row] = l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
  }
};

template <int D> __global__ __launch_bounds__(Many<D>::kThreads, 2) void k_many(const AttnArgs a) {
  using M = Many<D>;
  __shared__ __attribute__((aligned(16))) half8_t lk[2][M::kKPieces], lv[2][M::kVPieces];
  __shared__ __attribute__((aligned(16))) f32x4_t lsc[4][4];
  ManyRows<D> r(a, lk, lv, lsc);
  if (!r.begin()) return;
  if (r.t0 < r.t1) {
    r.pages_k(r.t0);
    r.pages_v(r.t0);
    r.load_k(r.t0);
    r.load_v(r.t0);
    r.pages_k(r.t0 + 1);
    r.pages_v(r.t0 + 1);
    r.stage_k(r.t0);
    r.stage_v(r.t0);
    r.load_k(r.t0 + 1);
    r.load_v(r.t0 + 1);
    r.pages_k(r.t0 + 2);
    r.pages_v(r.t0 + 2);
    __syncthreads();
    for (int t = r.t0; t < r.t1; ++t) {
      f32x16_t st[2];
      half8_t p[4];
      r.scores(t, st);
      Factors f;
      r.raise(r.largest(t, st, &f));
      r.weights(st, f, p);
      r.values(t, p);
      r.stage_k(t + 1);
      r.stage_v(t + 1);
      r.load_k(t + 2);
      r.load_v(t + 2);
      r.pages_k(t + 3);
      r.pages_v(t + 3);
      __syncthreads();
    }
  }
  r.finish();
}

// Lays out the tiles that a call's rows will read, in f16 and in the order of LDS: for tile t of a stream (sequence,
// cache head) 8 d pieces of keys [d / 8][64] and 8 d of values [8][d], and the factors of its four blocks of
// 16 keys.  One workgroup a tile; lanes follow the pieces, so that writes are whole lines.
template <int D> __global__ __launch_bounds__(256) void k_turn(const AttnArgs a) {
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, kvh = blockIdx.y, b = blockIdx.z;
  const Seq s = seq_of(a, b);
  if (s.rows == 0) return;
  int32_t last, x;
  visible(a, static_cast<int64_t>(s.len) - s.all + s.rows - 1, s.len, &x, &last);
  const int t = first_of(a, s) + blockIdx.x;  // as many workgroups as a stream has room for tiles
  if (t >= (last + 63) / 64) return;
  const int64_t tile = (static_cast<int64_t>(b) * a.c.heads + kvh) * a.turned_tiles + blockIdx.x;
  half8_t* out = static_cast<half8_t*>(a.turned) + tile * (16 * D);
  const int page_mask = a.c.page - 1;
  const auto page = [&](int key) { return key < s.len ? page_of(a.c, b, key >> a.page_shift) : -1; };
  {
    const int key = 64 * t + lane, pg = page(key & ~15);
    const int8_t* p = a.c.k + ((static_cast<int64_t>(pg < 0 ? 0 : pg) * a.c.heads + kvh) * a.c.page + (key & page_mask)) * D;
    u32x4_t q[D / 64];
#pragma unroll
    for (int i = 0; i < D / 64; ++i) q[i] = *reinterpret_cast<const u32x4_t*>(p + 16 * (4 * i + wave));
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const int u = 4 * i + wave;
      out[2 * u * 64 + lane] = codes_to_half8(q[i][0], q[i][1]);
      out[(2 * u + 1) * 64 + lane] = codes_to_half8(q[i][2], q[i][3]);
    }
  }
  {
    const int key = 64 * t + 16 * wave, pg = page(key);
    const int8_t* p = a.c.v + ((static_cast<int64_t>(pg < 0 ? 0 : pg) * a.c.heads + kvh) * D + lane) * a.c.page + (key & page_mask);
    u32x4_t q[D / 64];
#pragma unroll
    for (int i = 0; i < D / 64; ++i) q[i] = *reinterpret_cast<const u32x4_t*>(p + 64 * i * a.c.page);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      // keys 0-3 and 8-11 of the sixteen, then 4-7 and 12-15: as the weights lie in their registers
      out[8 * D + 2 * wave * D + 64 * i + lane] = codes_to_half8(q[i][0], q[i][2]);
      out[8 * D + (2 * wave + 1) * D + 64 * i + lane] = codes_to_half8(q[i][1], q[i][3]);
    }
    if (lane == 0) {
      const int64_t slot = static_cast<int64_t>(pg < 0 ? 0 : pg) * a.c.heads + kvh;
      float c, y, z;
      block_scales(a, a.c.ks[slot], a.c.vs[slot], pg >= 0, &c, &y, &z);
      static_cast<f32x4_t*>(a.factors)[4 * tile + wave] = f32x4_t{c, y, z, 0.0f};
    }
  }
}

// Heads of 256: a wave's rows fill the registers of a SIMD, so the overlap is made within the wave (2 x 4605
// queries: 925 us without, 800 with; heads of 128, two waves a SIMD: 1157 us without, 1188 with).  Step t takes
// the weights of tile t beside the scores of tile t + 1 on the matrix cores, and finds the maximum of tile t + 1
// and stages what comes next beside the values of tile t.
template <int D> __global__ __launch_bounds__(Many<D>::kThreads, 1) void k_wide(const AttnArgs a) {
  using M = Many<D>;
  __shared__ __attribute__((aligned(16))) half8_t lk[2][M::kKPieces], lv[2][M::kVPieces];
  __shared__ __attribute__((aligned(16))) f32x4_t lsc[4][4];
  ManyRows<D> r(a, lk, lv, lsc);
  if (!r.begin()) return;
  f32x16_t st[2][2];
  Factors fa[2];
  if (r.t0 < r.t1) {
    r.pages_k(r.t0);
    r.pages_v(r.t0);
    r.load_k(r.t0);
    r.load_v(r.t0);
    r.pages_k(r.t0 + 1);
    r.pages_v(r.t0 + 1);
    r.stage_k(r.t0);
    r.stage_v(r.t0);
    r.load_k(r.t0 + 1);
    r.load_v(r.t0 + 1);
    r.pages_k(r.t0 + 2);
    r.pages_v(r.t0 + 2);
    r.stage_k(r.t0 + 1);
    r.load_k(r.t0 + 2);
    r.pages_k(r.t0 + 3);
  }
  __syncthreads();
  if (r.t0 < r.t1) {
    r.scores(r.t0, st[0]);
    r.raise(r.largest(r.t0, st[0], &fa[0]));
  }
  __syncthreads();  // keys t0 are read before keys t0 + 2 are staged
  const auto step = [&](int t, f32x16_t* now, f32x16_t* next, const Factors& f, Factors* fnext) {
    r.stage_k(t + 2);
    r.stage_v(t + 1);
    r.load_k(t + 3);
    r.load_v(t + 2);
    r.pages_k(t + 4);
    r.pages_v(t + 3);
    r.scores(t + 1, next);
    half8_t p[4];
    r.weights(now, f, p);
    r.values(t, p);
    const float top = r.largest(t + 1, next, fnext);
    if (t + 1 < r.t1) r.raise(top);
    __syncthreads();
  };
  int t = r.t0;
  for (; t + 1 < r.t1; t += 2) {
    step(t, st[0], st[1], fa[0], &fa[1]);
    step(t + 1, st[1], st[0], fa[1], &fa[0]);
  }
  if (t < r.t1) step(t, st[0], st[1], fa[0], &fa[1]);
  r.finish();
}

template <int D> __global__ __launch_bounds__(Many<D>::kThreads, D <= 128 ? 2 : 1) void k_turned(const AttnArgs a) {
  using M = Many<D, true>;
  __shared__ __attribute__((aligned(16))) half8_t lk[2][M::kKPieces], lv[2][M::kVPieces];
  __shared__ __attribute__((aligned(16))) f32x4_t lsc[4][M::kFactors];
  ManyRows<D, true> r(a, lk, lv, lsc);
  if (!r.begin()) return;
  f32x16_t st[2][2];
  Factors fa[2];
  if (r.t0 < r.t1) {
    r.fetch_k(r.t0);
    r.fetch_v(r.t0);
    if (r.t0 + 1 < r.t1) r.fetch_k(r.t0 + 1);
    r.arrived();
  }
  __syncthreads();
  if (r.t0 < r.t1) {
    r.scores(r.t0, st[0]);
    r.raise(r.largest(r.t0, st[0], &fa[0]));
  }
  __syncthreads();  // keys t0 are read before keys t0 + 2 come
  // the last step's scores are of a tile that was never fetched: finite or not, they are not used
  const auto step = [&](int t, f32x16_t* now, f32x16_t* next, const Factors& f, Factors* fnext) {
    const bool more = t + 1 < r.t1;
    if (t + 2 < r.t1) r.fetch_k(t + 2);
    if (more) r.fetch_v(t + 1);
    r.scores(t + 1, next);
    half8_t p[4];
    r.weights(now, f, p);
    r.values(t, p);
    if (more) r.raise(r.largest(t + 1, next, fnext));
    r.arrived();
    __syncthreads();
  };
  int t = r.t0;
  for (; t + 1 < r.t1; t += 2) {
    step(t, st[0], st[1], fa[0], &fa[1]);
    step(t + 1, st[1], st[0], fa[1], &fa[0]);
  }
  if (t < r.t1) step(t, st[0], st[1], fa[0], &fa[1]);
  r.finish();
}

// ----------------------------------------------------------------------------------------- join
// D / 4 threads a part.  Many parts of a row are dealt to the 1024 / D teams of a workgroup; with few, each
// team takes a row (FEW).  `rows` rows: of the few-row form [batch][max_new][heads], of the many-row form those
// of the split row tiles in turn.
template <int D, bool FEW> __global__ __launch_bounds__(256) void k_join(const AttnArgs a, int64_t rows, int many) {
  constexpr int TEAM = D / 4, TEAMS = 256 / TEAM;
  __shared__ __attribute__((aligned(16))) f32x4_t lo[FEW ? 1 : TEAMS][TEAM];
  __shared__ float red[256];
  const int tid = threadIdx.x, team = tid / TEAM, e = tid % TEAM;
  const int64_t at = FEW ? static_cast<int64_t>(blockIdx.x) * TEAMS + team : blockIdx.x;
  if (at >= rows) return;
  int64_t tok, part_row;
  int h;
  if (many) {
    int b, kvh;
    const int n = static_cast<int>(at / many_rows(D));
    const int64_t r = static_cast<int64_t>(tile_of(a, a.whole + n, &b, &kvh)) * many_rows(D) + at % many_rows(D);
    const Seq s = seq_of(a, b);
    if (r >= static_cast<int64_t>(s.rows) * a.group) return;
    tok = s.row0 + r / a.group;
    h = kvh * a.group + static_cast<int>(r % a.group);
    part_row = at;
  } else {
    const int64_t query = at / a.heads;
    h = static_cast<int>(at - query * a.heads);
    const int b = static_cast<int>(query / a.max_new), i = static_cast<int>(query - static_cast<int64_t>(b) * a.max_new);
    const Seq s = seq_of(a, b);
    if (i >= s.rows) return;
    tok = s.row0 + i;
    part_row = tok * a.heads + h;
  }
  const float* ml = a.part_ml + part_row * a.splits * 2;
  float m = kNone;
  if constexpr (FEW) {
    for (int i = 0; i < a.splits; ++i) m = ml[2 * i + 1] != 0.0f ? __builtin_fmaxf(m, ml[2 * i]) : m;
  } else {
    for (int i = tid; i < a.splits; i += 256) m = ml[2 * i + 1] != 0.0f ? __builtin_fmaxf(m, ml[2 * i]) : m;
    red[tid] = m;
    __syncthreads();
#pragma unroll
    for (int off = 128; off >= 1; off >>= 1) {
      if (tid < off) red[tid] = __builtin_fmaxf(red[tid], red[tid + off]);
      __syncthreads();
    }
    m = red[0];
  }
  f32x4_t o = {0, 0, 0, 0};
  float l = 0.0f;
  for (int i = FEW ? 0 : team; i < a.splits; i += FEW ? 1 : TEAMS) {
    const float li = ml[2 * i + 1];
    if (li == 0.0f) continue;  // nothing visible in that part: its values were not written
    const float by = exp2_fast(ml[2 * i] - m);
    l = __builtin_fmaf(li, by, l);
    o += *reinterpret_cast<const f32x4_t*>(a.part_o + (part_row * a.splits + i) * D + 4 * e) * by;
  }
  if constexpr (!FEW) {
    __syncthreads();
    lo[team][e] = o;
    red[tid] = l;
    __syncthreads();
    if (team) return;
    for (int i = 1; i < TEAMS; ++i) {
      o += lo[i][e];
      l += red[i * TEAM];
    }
  }
  const float by = l == 0.0f ? 0.0f : 1.0f / l;
  store4(a, tok * a.ot + h * a.oh + 4 * e, o * by);
  if (a.lse && e == 0) a.lse[tok * a.heads + h] = l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
}

}  // namespace attn

template <int D> int launch_attn(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  if (p.many) {
    const int64_t tiles = static_cast<int64_t>(a.c.batch) * a.c.heads * a.row_tiles, grid = a.whole + (tiles - a.whole) * a.splits;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    if constexpr (D > 64) {
      if (p.turned) hipLaunchKernelGGL((attn::k_turn<D>), dim3(p.turned, a.c.heads, a.c.batch), dim3(256), 0, stream, a);
    }
    // a launch takes fewer than 2^32 threads; row tiles come near where a caller bounds ragged sequences loosely
    constexpr int64_t most = 0xffffffffu / attn::Many<D>::kThreads;
    for (int64_t first = 0; first < grid; first += most) {
      AttnArgs s = a;
      s.first = static_cast<int32_t>(first);
      const dim3 g(static_cast<uint32_t>(std::min(most, grid - first))), t(attn::Many<D>::kThreads);
      if constexpr (D > 64) {
        if (p.turned) hipLaunchKernelGGL((attn::k_turned<D>), g, t, 0, stream, s);
      }
      if (!p.turned) {
        if constexpr (D <= 128) hipLaunchKernelGGL((attn::k_many<D>), g, t, 0, stream, s);
        else hipLaunchKernelGGL((attn::k_wide<D>), g, t, 0, stream, s);
      }
    }
  } else {
    const dim3 grid(a.splits, a.c.heads * a.row_tiles, a.c.batch);
    if constexpr (D <= 128) {
      if (p.rt == 2) hipLaunchKernelGGL((attn::k_few<D, 2, 4>), grid, dim3(256), 0, stream, a);
      else if (p.waves == 8) hipLaunchKernelGGL((attn::k_few<D, 1, 8>), grid, dim3(512), 0, stream, a);
    }
    if (p.rt == 1 && p.waves == 4) hipLaunchKernelGGL((attn::k_few<D, 1, 4>), grid, dim3(256), 0, stream, a);
  }
  if (a.splits > 1) {
    const int64_t rows = p.many ? p.part_rows : static_cast<int64_t>(a.c.batch) * a.max_new * a.heads;
    if (a.splits <= 8)
      hipLaunchKernelGGL((attn::k_join<D, true>), dim3(static_cast<uint32_t>((rows + 1024 / D - 1) / (1024 / D))), dim3(256), 0, stream, a,
                         rows, p.many);
    else hipLaunchKernelGGL((attn::k_join<D, false>), dim3(static_cast<uint32_t>(rows)), dim3(256), 0, stream, a, rows, p.many);
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace orbq
