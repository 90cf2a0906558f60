// Attention over the 8-bit paged cache.  For query row r (one token, one head; the `group` query
// heads of one cache head are rows of the same tile, so that keys and values are read once for
// all of them):
//   S_j = scale q . k_j,  O = sum_j softmax(S)_j v_j  over the visible keys lo <= j < hi,
//   k_j = kc_j ks[block of j],  v_j = vc_j vs[block of j].
//
// Both products run on the matrix cores in f16 with fp32 accumulation, on the codes themselves: a
// code is exact in f16, q enters as q 2^-e with 2^e its row's magnitude (exact for f16 input and, but
// for entries below 2^-14 of the row's largest, for bf16), and the key scale joins the softmax's
// own factor.  The value scale goes into the exponent:
//   w_j = exp2(S_j log2(e) + log2(vs_j) - m),  m the running maximum of S_j log2(e) + log2(vs_j),
//   O = sum_j w_j vc_j / l,  l = sum over blocks (1/vs) sum_j w_j,
// so no element is multiplied by a scale and the rounding of w to f16 is relative to the row's largest
// weight whatever the scales are.  m, l and O are fp32.  m may lag behind the true maximum by up
// to 2^kSlack (w stays below the f16 limit), which saves most of the rescaling of O.
//
// The products are taken transposed: S^T = K Q^T has one query row a lane and its keys down the
// accumulator registers, which is, up to an order of the keys that the values follow, the layout in
// which O^T = V^T w^T takes its second operand.  The weights never leave their registers, and m, l and
// the rescaling factors are one value a lane.
//
// Two forms:
//   few   16 or 32 rows a workgroup (token-by-token serving): bound by the cache's bytes.  Four waves
//         take 64-key tiles in turn straight from memory into registers, and are joined at the end.
//   many  128 rows a workgroup: bound by the matrix cores and the softmax's vector work.  Codes
//         are turned into f16 once a workgroup on their way into LDS, double buffered.
// Either splits the keys over workgroups where there are few rows; k_join joins the parts.
#pragma once

#include <algorithm>

#include "attention_device.h"

namespace orbq {
namespace attn {

constexpr float kSlack = 8.0f;       // log2 by which a weight may pass 1 before O is rescaled
constexpr float kNone = -1.0e30f;    // running maximum before the first visible key
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

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
  int32_t rows;   // queries
  int32_t len;    // cached tokens, within the table
};

__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
  Seq s;
  rows_of(a.cu, a.total, a.c.batch, a.max_new, b, &s.row0, &s.rows);
  const int64_t most = static_cast<int64_t>(a.c.max_pages) << a.page_shift;
  const int32_t n = a.lens[b];
  s.len = n < 0 ? 0 : (n > most ? static_cast<int32_t>(most) : n);
  return s;
}

// one value a lane that covers a block's keys: c = ks |scale| log2(e), log2(vs), 1/vs
__device__ __forceinline__ void block_scales(const AttnArgs& a, int64_t slot, float* c, float* lv, float* iv) {
  *c = a.c.ks[slot] * a.scale_log2e;
  const float v = __builtin_fmaxf(a.c.vs[slot], kScaleFloor);
  *lv = __builtin_amdgcn_logf(v);  // log2, exact to a unit of its last place for a normal number
  *iv = __builtin_amdgcn_rcpf(v);
}

__device__ __forceinline__ void store4(const AttnArgs& a, int64_t at, f32x4_t v) {
  uint16_t* o = static_cast<uint16_t*>(a.o);
  if (a.f16) Vec<kF16, 4>::store(o, at, reinterpret_cast<const float*>(&v));
  else Vec<kBF16, 4>::store(o, at, reinterpret_cast<const float*>(&v));
}

// ------------------------------------------------------------------------------------------ few
constexpr int kFewWaves = 4;

template <int D, int RT> __global__ __launch_bounds__(64 * kFewWaves) void k_few(const AttnArgs a) {
  constexpr int NC = D / 64, ND = D / 16;
  __shared__ __attribute__((aligned(16))) f32x4_t join_o[kFewWaves / 2][RT][ND][64];
  __shared__ float join_m[kFewWaves][RT][16], join_l[kFewWaves][RT][16];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, l15 = lane & 15, g = lane >> 4;
  const int split = blockIdx.x, kvh = blockIdx.y / a.row_tiles, tile = blockIdx.y - kvh * a.row_tiles, b = blockIdx.z;
  const Seq s = seq_of(a, b);
  const int all = s.rows * a.group, r0 = tile * 16 * RT;
  if (r0 >= all) return;
  const int r1 = r0 + 16 * RT < all ? r0 + 16 * RT : all;

  // the rows' keys
  int32_t lo[RT], hi[RT], lo_most, hi_least, first, last;
  visible(a, static_cast<int64_t>(s.len) - s.rows + r0 / a.group, s.len, &first, &hi_least);
  visible(a, static_cast<int64_t>(s.len) - s.rows + (r1 - 1) / a.group, s.len, &lo_most, &last);
  const int t_first = first / 64, t_end = (last + 63) / 64;
  const int t0 = t_first + split * a.chunk;
  const int t1 = split + 1 < a.splits && t0 + a.chunk < t_end ? t0 + a.chunk : t_end;
  if (a.splits > 1 && t0 >= t1) {  // nothing here: an empty part
    for (int i = tid; i < r1 - r0; i += 64 * kFewWaves) {
      const int r = r0 + i;
      const int64_t row = (s.row0 + r / a.group) * a.heads + kvh * a.group + r % a.group;
      float* ml = a.part_ml + (row * a.splits + split) * 2;
      ml[0] = kNone;
      ml[1] = 0.0f;
    }
    return;
  }

  // q: lane l15 holds row l15, entries 64 c + 16 g + 0..15 as two operands
  half8_t q[RT][NC][2];
  float qs[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = r0 + 16 * rt + l15;
    const bool live = r < r1;
    const int rr = live ? r : r0, tok = rr / a.group, h = kvh * a.group + rr - tok * a.group;
    const int64_t at = (s.row0 + tok) * a.qt + h * a.qh;
    visible(a, static_cast<int64_t>(s.len) - s.rows + tok, s.len, &lo[rt], &hi[rt]);
    if (!live) hi[rt] = 0;
    float most = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        q[rt][c][k] = load_q8(a, at + 64 * c + 16 * g + 8 * k);
        most = __builtin_fmaxf(most, q_most(q[rt][c][k], a.f16));
      }
    most = __builtin_fmaxf(most, __shfl_xor(most, 16));
    most = __builtin_fmaxf(most, __shfl_xor(most, 32));
    qs[rt] = row_power(most);
    const float by = (a.negative ? -1.0f : 1.0f) / qs[rt];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) q[rt][c][k] = q_scaled(q[rt][c][k], a.f16, by);
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
  // + 15; and for values entries 16 i + l15, keys 16 g .. + 15.  Keys past the sequence's end in a
  // block that it holds are read and masked; blocks that it does not hold are not read.
  const int page_mask = a.c.page - 1;
  u32x4_t kr[4][NC], vr[ND];
  int kpg, vpg;                      // pages of the tile to load next
  const auto pages = [&](int t, int* kp, int* vp) {
    const int kk = 64 * t + 16 * (l15 >> 2), vk = 64 * t + 16 * g;
    *kp = t < t1 && kk < s.len ? page_of(a.c, b, kk >> a.page_shift) : -1;
    *vp = t < t1 && vk < s.len ? page_of(a.c, b, vk >> a.page_shift) : -1;
  };
  const auto load_k = [&](int t, int pg) {
    const int at = (64 * t + 16 * (l15 >> 2) + (l15 & 3)) & page_mask;
    const int8_t* p = a.c.k + ((static_cast<int64_t>(pg) * a.c.heads + kvh) * a.c.page + at) * D + 16 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c)
        kr[i][c] = pg >= 0 ? *reinterpret_cast<const u32x4_t*>(p + 4 * i * D + 64 * c) : u32x4_t{0, 0, 0, 0};
  };
  const auto load_v = [&](int t, int pg) {
    const int8_t* p = a.c.v + ((static_cast<int64_t>(pg) * a.c.heads + kvh) * D + l15) * a.c.page + ((64 * t + 16 * g) & page_mask);
#pragma unroll
    for (int i = 0; i < ND; ++i)
      vr[i] = pg >= 0 ? *reinterpret_cast<const u32x4_t*>(p + static_cast<int64_t>(16 * i) * a.c.page) : u32x4_t{0, 0, 0, 0};
  };
  const auto load_s = [&](int pg, float* c, float* lv, float* iv) {
    *c = *iv = 0.0f;
    *lv = -__builtin_inff();  // a block that is absent has no weight
    if (pg >= 0) block_scales(a, static_cast<int64_t>(pg) * a.c.heads + kvh, c, lv, iv);
  };

  int t = t0 + wave;
  pages(t, &kpg, &vpg);
  load_k(t, kpg);
  for (; t < t1; t += kFewWaves) {
    load_v(t, vpg);
    float sc, lv, iv;
    load_s(vpg, &sc, &lv, &iv);
    pages(t + kFewWaves, &kpg, &vpg);
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
    load_k(t + kFewWaves, kpg);
    const bool whole = 64 * t >= lo_most && 64 * t + 64 <= hi_least;
    half8_t p[RT][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float c = sc * qs[rt];
      float x[16];
      float top = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __builtin_fmaf(st[rt][i >> 2][i & 3], c, lv);
      if (!whole) {
        const int k0 = 64 * t + 16 * g;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = k0 + i >= lo[rt] && k0 + i < hi[rt] ? x[i] : -__builtin_inff();
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, x[i]);
      top = __builtin_fmaxf(top, __shfl_xor(top, 16));
      top = __builtin_fmaxf(top, __shfl_xor(top, 32));
      if (__any(top > m[rt] + kSlack)) {
        const float mn = __builtin_fmaxf(m[rt], top), by = exp2_fast(m[rt] - mn);
        m[rt] = mn;
        l[rt] *= by;
#pragma unroll
        for (int i = 0; i < ND; ++i) o[rt][i] *= by;
      }
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float w = exp2_fast(x[i] - m[rt]);
        sum += w;
        p[rt][i >> 3][i & 7] = static_cast<_Float16>(w);
      }
      l[rt] = __builtin_fmaf(sum, iv, l[rt]);
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

  // join the four waves
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
    for (int w = 0; w < kFewWaves; ++w) mt[rt] = __builtin_fmaxf(mt[rt], join_m[w][rt][l15]);
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) lt[rt] += join_l[w][rt][l15] * exp2_fast(join_m[w][rt][l15] - mt[rt]);
    const float by = exp2_fast(m[rt] - mt[rt]);
#pragma unroll
    for (int i = 0; i < ND; ++i) o[rt][i] *= by;
  }
#pragma unroll
  for (int half = kFewWaves / 2; half >= 1; half >>= 1) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = 0; i < ND; ++i) join_o[wave - half][rt][i][lane] = o[rt][i];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = 0; i < ND; ++i) o[rt][i] += join_o[wave][rt][i][lane];
    }
    __syncthreads();
  }
  if (wave) return;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = r0 + 16 * rt + l15;
    if (r >= r1) continue;
    const int tok = r / a.group, h = kvh * a.group + r - tok * a.group;
    const int64_t row = (s.row0 + tok) * a.heads + h;
    if (a.splits > 1) {
      float* po = a.part_o + (row * a.splits + split) * D;
#pragma unroll
      for (int i = 0; i < ND; ++i) *reinterpret_cast<f32x4_t*>(po + 16 * i + 4 * g) = o[rt][i];
      if (g == 0) {
        float* ml = a.part_ml + (row * a.splits + split) * 2;
        ml[0] = mt[rt];
        ml[1] = lt[rt];
      }
    } else {
      const float by = lt[rt] == 0.0f ? 0.0f : 1.0f / lt[rt];
      const int64_t at = (s.row0 + tok) * a.ot + h * a.oh;
#pragma unroll
      for (int i = 0; i < ND; ++i) store4(a, at + 16 * i + 4 * g, o[rt][i] * by);
      if (a.lse && g == 0)
        a.lse[row] = lt[rt] == 0.0f ? -__builtin_inff() : (mt[rt] + __builtin_log2f(lt[rt])) * kLn2;
    }
  }
}

// ----------------------------------------------------------------------------------------- many
template <int D> struct Many {
  static constexpr int kWaves = D == 128 ? 8 : 4, kRows = 32 * kWaves, kThreads = 64 * kWaves;
  // LDS of one tile in 16-byte pieces: keys [d / 8][64 + 1], values [8][d + 2] (pieces of 8 keys).
  // A wave's operand reads are 32 consecutive pieces; the pitches spread the writers over banks.
  static constexpr int kKPitch = 65, kVPitch = D + 2;
  static constexpr int kKPieces = D / 8 * kKPitch, kVPieces = 8 * kVPitch;
  static constexpr int kLoads = D / (16 * kWaves);  // 16-byte loads a thread, keys; values the same
};

template <int D> __global__ __launch_bounds__(Many<D>::kThreads, D <= 128 ? 2 : 1) void k_many(const AttnArgs a, int streams) {
  using M = Many<D>;
  constexpr int NL = M::kLoads, NT = M::kThreads, NS = D / 16, ND = D / 32;
  __shared__ __attribute__((aligned(16))) half8_t lk[2][M::kKPieces], lv[2][M::kVPieces];
  __shared__ float lsc[2][4][3];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, l31 = lane & 31, hi32 = lane >> 5;

  // Workgroups are given out to the eight dies in turn: the row tiles of one stream (sequence, head,
  // split) go to one die, whose L2 then reads their keys and values once; a launch of few streams is
  // spread tile by tile.  Long rows of a causal mask come first.
  int stream, tile;
  if (streams >= 16) {
    const int total = streams * a.row_tiles, per = (total + 7) >> 3;
    const int lin = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (lin >= total || static_cast<int>(blockIdx.x >> 3) >= per) return;
    stream = lin / a.row_tiles;
    tile = lin - stream * a.row_tiles;
  } else {
    if (static_cast<int>(blockIdx.x) >= streams * a.row_tiles) return;
    tile = blockIdx.x / streams;
    stream = blockIdx.x - tile * streams;
  }
  tile = a.row_tiles - 1 - tile;
  const int split = stream % a.splits, kvh = stream / a.splits % a.c.heads, b = stream / a.splits / a.c.heads;
  const Seq s = seq_of(a, b);
  const int64_t all = static_cast<int64_t>(s.rows) * a.group;
  const int64_t r0 = static_cast<int64_t>(tile) * M::kRows;
  if (r0 >= all) return;
  const int64_t r1 = r0 + M::kRows < all ? r0 + M::kRows : all;
  const int64_t base = static_cast<int64_t>(s.len) - s.rows;

  int32_t first, last, x0, x1;
  visible(a, base + r0 / a.group, s.len, &first, &x0);
  visible(a, base + (r1 - 1) / a.group, s.len, &x1, &last);
  const int t_first = first / 64, t_end = (last + 63) / 64;
  const int t0 = t_first + split * a.chunk;
  const int t1 = split + 1 < a.splits && t0 + a.chunk < t_end ? t0 + a.chunk : t_end;

  // this lane's row
  const int64_t row_local = r0 + 32 * wave + l31;
  const bool live = row_local < r1;
  const int64_t rr = live ? row_local : r0;
  const int64_t tok = rr / a.group;
  const int h = kvh * a.group + static_cast<int>(rr - tok * a.group);
  const int64_t row = (s.row0 + tok) * a.heads + h;
  int32_t lo, hi;
  visible(a, base + tok, s.len, &lo, &hi);
  if (!live) hi = 0;
  // the wave's: keys from any_lo to any_hi are visible to some row, from all_lo to all_hi to all
  int32_t any_lo, any_hi, all_lo, all_hi;
  {
    const int64_t w0 = r0 + 32 * wave < r1 ? r0 + 32 * wave : r1 - 1, w1 = r0 + 32 * wave + 31 < r1 ? r0 + 32 * wave + 31 : r1 - 1;
    visible(a, base + w0 / a.group, s.len, &any_lo, &all_hi);
    visible(a, base + w1 / a.group, s.len, &all_lo, &any_hi);
    if (r0 + 32 * wave >= r1) any_hi = 0;
  }

  half8_t q[NS];
  float qs;
  {
    const int64_t at = (s.row0 + tok) * a.qt + h * a.qh;
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      q[i] = load_q8(a, at + 16 * i + 8 * hi32);
      most = __builtin_fmaxf(most, q_most(q[i], a.f16));
    }
    most = __builtin_fmaxf(most, __shfl_xor(most, 32));
    qs = row_power(most);
    const float by = (a.negative ? -1.0f : 1.0f) / qs;
#pragma unroll
    for (int i = 0; i < NS; ++i) q[i] = q_scaled(q[i], a.f16, by);
  }

  f32x16_t o[ND];
#pragma unroll
  for (int i = 0; i < ND; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
  float m = kNone, l = 0.0f;

  // staging: 16 codes a load; keys (key, 16 entries), values (entry, 16 keys)
  const int page_mask = a.c.page - 1;
  const int32_t* table = a.c.table + b * a.c.ldt;
  u32x4_t kr[NL], vr[NL];
  int kpg[NL], vpg;
  float sc[3];
  // Loads never branch: where a block is absent the first of the cache is read, and its weight is zero.
  const int64_t block_bytes = static_cast<int64_t>(D) * a.c.page;
  const auto page_at = [&](int key) {  // the table's entry for a key of this sequence, -1: absent
    const int p = key >> a.page_shift;
    const int32_t pg = table[p < a.c.max_pages ? p : a.c.max_pages - 1];
    return key < s.len && static_cast<uint32_t>(pg) < static_cast<uint32_t>(a.c.pages) ? pg : -1;
  };
  const auto pages = [&](int t) {
#pragma unroll
    for (int i = 0; i < NL; ++i) kpg[i] = page_at(64 * t + (i * NT + tid) / (D / 16));
    vpg = page_at(64 * t + 16 * (tid & 3));
  };
  const auto block_of = [&](int pg) {  // (pg heads + kvh) blocks, pg < 0 as 0
    return (static_cast<uint64_t>(static_cast<uint32_t>(pg < 0 ? 0 : pg)) * static_cast<uint32_t>(a.c.heads) + kvh) * block_bytes;
  };
  const auto load = [&](int t) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int at = i * NT + tid, key = 64 * t + at / (D / 16), u = at % (D / 16);
      kr[i] = *reinterpret_cast<const u32x4_t*>(a.c.k + block_of(kpg[i]) + (key & page_mask) * D + 16 * u);
    }
    const int8_t* v = a.c.v + block_of(vpg) + ((64 * t + 16 * (tid & 3)) & page_mask) + (tid >> 2) * a.c.page;
#pragma unroll
    for (int i = 0; i < NL; ++i) vr[i] = *reinterpret_cast<const u32x4_t*>(v + (i * NT / 4) * a.c.page);
    if (tid < 4) {
      block_scales(a, static_cast<int64_t>(vpg < 0 ? 0 : vpg) * a.c.heads + kvh, &sc[0], &sc[1], &sc[2]);
      if (vpg < 0) {  // a block that is absent has no weight
        sc[0] = sc[2] = 0.0f;
        sc[1] = -__builtin_inff();
      }
    }
  };
  const auto stage = [&](int buf) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int at = i * NT + tid, key = at / (D / 16), u = at % (D / 16);
      lk[buf][(2 * u) * M::kKPitch + key] = codes_to_half8(kr[i][0], kr[i][1]);
      lk[buf][(2 * u + 1) * M::kKPitch + key] = codes_to_half8(kr[i][2], kr[i][3]);
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int at = i * NT + tid, d = at >> 2, g = at & 3;
      // keys 0-3 and 8-11 of the sixteen, then 4-7 and 12-15: as the weights lie in their registers
      lv[buf][(2 * g) * M::kVPitch + d] = codes_to_half8(vr[i][0], vr[i][2]);
      lv[buf][(2 * g + 1) * M::kVPitch + d] = codes_to_half8(vr[i][1], vr[i][3]);
    }
    if (tid < 4) {
#pragma unroll
      for (int i = 0; i < 3; ++i) lsc[buf][tid][i] = sc[i];
    }
  };

  if (t0 < t1) {
    pages(t0);
    load(t0);
    pages(t0 + 1);
    stage(0);
  }
  __syncthreads();
  int buf = 0;
  for (int t = t0; t < t1; ++t, buf ^= 1) {
    if (t + 1 < t1) {
      load(t + 1);
      pages(t + 2);
    }
    if (64 * t < any_hi && 64 * t + 64 > any_lo) {
      f32x16_t st[2];
#pragma unroll
      for (int j = 0; j < 16; ++j) st[0][j] = st[1][j] = 0.0f;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const half8_t k0 = lk[buf][(2 * i + hi32) * M::kKPitch + l31], k1 = lk[buf][(2 * i + hi32) * M::kKPitch + 32 + l31];
        st[0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k0, q[i], st[0], 0, 0, 0);
        st[1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k1, q[i], st[1], 0, 0, 0);
      }
      // register 8 (g & 1) + 4 k + j of st[g / 2]: key 16 g + 8 k + 4 hi32 + j
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
      // c is positive (a factor of zero is taken as the least normal number, so that a masked score stays
      // at -infinity): a block's largest weight is its largest score's
      float c[4], v[4], top = -__builtin_inff();
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        c[g] = __builtin_fmaxf(lsc[buf][g][0] * qs, 0x1p-126f);
        v[g] = lsc[buf][g][1];
        float x = st[g >> 1][8 * (g & 1)];
#pragma unroll
        for (int j = 1; j < 8; ++j) x = __builtin_fmaxf(x, st[g >> 1][8 * (g & 1) + j]);
        top = __builtin_fmaxf(top, __builtin_fmaf(x, c[g], v[g]));
      }
      top = __builtin_fmaxf(top, __shfl_xor(top, 32));
      if (__any(top > m + kSlack)) {
        const float mn = __builtin_fmaxf(m, top), by = exp2_fast(m - mn);
        m = mn;
        l *= by;
#pragma unroll
        for (int i = 0; i < ND; ++i) o[i] *= by;
      }
      half8_t p[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float y = v[g] - m;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float w = exp2_fast(__builtin_fmaf(st[g >> 1][8 * (g & 1) + j], c[g], y));
          sum += w;
          p[g][j] = static_cast<_Float16>(w);
        }
        l = __builtin_fmaf(sum, lsc[buf][g][2], l);
      }
#pragma unroll
      for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(lv[buf][(2 * g + hi32) * M::kVPitch + 32 * i + l31], p[g], o[i], 0, 0, 0);
    }
    if (t + 1 < t1) stage(buf ^ 1);
    __syncthreads();
  }

  l += __shfl_xor(l, 32);
  if (!live) return;
  // register 4 k + j of o[i]: entry 32 i + 8 k + 4 hi32 + j
  if (a.splits > 1) {
    float* po = a.part_o + (row * a.splits + split) * D;
    if (l != 0.0f) {
#pragma unroll
      for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<f32x4_t*>(po + 32 * i + 8 * k + 4 * hi32) =
              f32x4_t{o[i][4 * k], o[i][4 * k + 1], o[i][4 * k + 2], o[i][4 * k + 3]};
    }
    if (hi32 == 0) {
      float* ml = a.part_ml + (row * a.splits + split) * 2;
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

// ----------------------------------------------------------------------------------------- join
// One workgroup a row: D / 4 threads a part, the parts dealt to 1024 / D teams.
template <int D> __global__ __launch_bounds__(256) void k_join(const AttnArgs a) {
  constexpr int TEAM = D / 4, TEAMS = 256 / TEAM;
  __shared__ __attribute__((aligned(16))) f32x4_t lo[TEAMS][TEAM];
  __shared__ float red[256];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, team = tid / TEAM, e = tid % TEAM;
  const float* ml = a.part_ml + row * a.splits * 2;
  float m = kNone;
  for (int i = tid; i < a.splits; i += 256) m = ml[2 * i + 1] != 0.0f ? __builtin_fmaxf(m, ml[2 * i]) : m;
  red[tid] = m;
  __syncthreads();
#pragma unroll
  for (int off = 128; off >= 1; off >>= 1) {
    if (tid < off) red[tid] = __builtin_fmaxf(red[tid], red[tid + off]);
    __syncthreads();
  }
  m = red[0];
  f32x4_t o = {0, 0, 0, 0};
  float l = 0.0f;
  for (int i = team; i < a.splits; i += TEAMS) {
    const float li = ml[2 * i + 1];
    if (li == 0.0f) continue;  // nothing visible in that part: its values were not written
    const float by = exp2_fast(ml[2 * i] - m);
    l = __builtin_fmaf(li, by, l);
    o += *reinterpret_cast<const f32x4_t*>(a.part_o + (row * a.splits + i) * D + 4 * e) * by;
  }
  __syncthreads();
  lo[team][e] = o;
  red[tid] = l;
  __syncthreads();
  if (team) return;
  for (int i = 1; i < TEAMS; ++i) {
    o += lo[i][e];
    l += red[i * TEAM];
  }
  const int64_t tok = row / a.heads;
  const int h = static_cast<int>(row - tok * a.heads);
  const float by = l == 0.0f ? 0.0f : 1.0f / l;
  store4(a, tok * a.ot + h * a.oh + 4 * e, o * by);
  if (a.lse && e == 0) a.lse[row] = l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
}

}  // namespace attn

template <int D> int launch_attn(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  if (p.many) {
    const int streams = a.c.batch * a.c.heads * a.splits;
    const int64_t total = static_cast<int64_t>(streams) * a.row_tiles, grid = (total + 7) / 8 * 8;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL((attn::k_many<D>), dim3(static_cast<uint32_t>(grid)), dim3(attn::Many<D>::kThreads), 0, stream, a, streams);
  } else {
    const dim3 grid(a.splits, a.c.heads * a.row_tiles, a.c.batch);
    if (p.rt == 1) hipLaunchKernelGGL((attn::k_few<D, 1>), grid, dim3(64 * attn::kFewWaves), 0, stream, a);
    else hipLaunchKernelGGL((attn::k_few<D, 2>), grid, dim3(64 * attn::kFewWaves), 0, stream, a);
  }
  if (a.splits > 1)
    hipLaunchKernelGGL((attn::k_join<D>), dim3(static_cast<uint32_t>(a.total * a.heads)), dim3(256), 0, stream, a);
  return static_cast<int>(hipGetLastError());
}

}  // namespace orbq
