// Device helpers of the 8-bit paged cache: codes, and the append of one page's keys or values of one head.
#pragma once

#include <type_traits>

#include "attention_device.h"

namespace orbq {

constexpr float kInv127 = 1.0f / 127.0f;

// bytes of a page's [page][d] block / 32, within one to four waves
constexpr int threads_for(int bytes) { return bytes / 32 < 64 ? 64 : (bytes / 32 > 256 ? 256 : bytes / 32); }

__device__ __forceinline__ uint32_t code_of(float x, float inv) {
  float c = __builtin_rintf(x * inv);
  c = __builtin_fminf(__builtin_fmaxf(c, -127.0f), 127.0f);
  c = x == x ? c : 0.0f;
  return static_cast<uint32_t>(static_cast<int>(c)) & 0xffu;
}

// the codes of four finite values within 127.5 / inv: adding 1.5 2^23 rounds to the integer (ties to even) that
// is then the low byte
__device__ __forceinline__ uint32_t codes_of_finite(const float* x, float inv) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y = x[i] * inv;
    asm("" : "+v"(y));  // rounded by itself, as rint(x inv) asks: not one fused operation with the sum
    c[i] = __builtin_bit_cast(uint32_t, y + 12582912.0f);
  }
  return __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400u) | __builtin_amdgcn_perm(c[3], c[2], 0x04000c0cu);
}

template <bool FINITE> __device__ __forceinline__ uint32_t codes_of(const float* x, float inv) {
  if constexpr (FINITE) return codes_of_finite(x, inv);
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) r |= code_of(x[i], inv) << (8 * i);
  return r;
}

// four codes of a scale that grew
__device__ __forceinline__ uint32_t rescale4(uint32_t q, float ratio) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r |= code_of(static_cast<float>(static_cast<int8_t>(q >> (8 * i))), ratio) << (8 * i);
  return r;
}

// the bytes of a dword at positions at .. at + 3 that lie below `end`
__device__ __forceinline__ uint32_t below(int at, int end) {
  const int n = end - at;
  return n <= 0 ? 0u : (n >= 4 ? 0xffffffffu : (1u << (8 * n)) - 1u);
}

// The largest of N 16-byte words' magnitudes as an unsigned integer, two entries an instruction where they have 16
// bits; above the largest number's it is an infinity's or a NaN's.
template <int DT, int N> __device__ __forceinline__ uint32_t largest_bits(const u32x4_t* w) {
  typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
  if constexpr (DT == kF32) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max(m, w[i][j] & 0x7fffffffu);
    return m;
  } else {
    u16x2_t m = {0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w[i][j] & 0x7fff7fffu));
    return max(static_cast<uint32_t>(m[0]), static_cast<uint32_t>(m[1]));
  }
}

// maximum over the workgroup
template <int NT> __device__ __forceinline__ uint32_t wide_max(uint32_t m, uint32_t* top) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), off)));
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) m = max(m, top[w]);
  }
  return m;
}

// A thread's share of a page: PER columns of 8 entries, TP consecutive tokens each time, so that the codes of
// TP tokens cross LDS as one word where values are turned.
template <int D, int PAGE> struct Share {
  static constexpr int NT = threads_for(D * PAGE), PER = D * PAGE / (8 * NT), TP = PER < 4 ? PER : 4;
  static constexpr int LD = PAGE + 4;  // LDS pitch of a value row
  static_assert(TP == 2 || TP == 4, "");
  static __device__ __forceinline__ int token(int tid, int i) { return (i / TP * (NT / (D / 8)) + tid / (D / 8)) * TP + i % TP; }
  static __device__ __forceinline__ int entry(int tid) { return tid % (D / 8) * 8; }
};

struct Unchanged {
  static constexpr bool kChanges = false;
};

// LDS of append_page
template <int D, int PAGE> struct PageSpace {
  using S = Share<D, PAGE>;
  __attribute__((aligned(16))) uint8_t turned[D * S::LD];
  uint32_t top[S::NT / 64];
};

// A page that a sequence's new tokens touch.
struct PageSpot {
  int64_t base;    // packed row of the page's token t: base + t
  int had, end;    // tokens held before, and after
  int32_t entry;   // of the page table, not yet judged
  bool inside;     // the table has one
};

// The `page_of_call`th page that sequence b's new tokens touch, if there is one.  UNPLACED: also of tokens at negative
// positions, which have none: counted from token 0.
template <int PAGE, bool UNPLACED = false>
__device__ __forceinline__ bool locate_page(const KvCache& c, const KvTokens& x, int b, int64_t page_of_call, PageSpot* spot) {
  int64_t row0;
  int32_t rows, all;
  rows_of(x.cu, x.total, c.batch, x.max_rows, b, &row0, &rows, &all);
  const int64_t first = x.first[b];
  if ((first < 0 && !UNPLACED) || rows == 0) return false;
  const int64_t start = first < 0 ? 0 : first;
  const int64_t p = start / PAGE + page_of_call;
  const int64_t t0 = p * PAGE;                       // the page's first token
  if (t0 >= start + rows) return false;
  spot->had = static_cast<int>(start > t0 ? start - t0 : 0);
  spot->end = static_cast<int>(start + rows - t0 < PAGE ? start + rows - t0 : PAGE);
  spot->base = row0 + t0 - start;
  spot->inside = first >= 0 && p < c.max_pages;
  // the page, and with it the old scale, are looked up while the new values are on their way
  spot->entry = c.table[b * c.ldt + (spot->inside ? p : 0)];
  return true;
}

// The new keys (or values) of one head that fall into a page: their scale, the page's earlier codes where it grows, their
// codes.  Called by a whole workgroup.  `change` may replace the entries, as floats, before that.
template <int DT, int D, int PAGE, class Change>
__device__ __forceinline__ void append_page(const KvCache& c, const KvTokens& x, const PageSpot& spot, int head, bool values,
                                            PageSpace<D, PAGE>& space, const Change& change) {
  using S = Share<D, PAGE>;
  constexpr int NT = S::NT, PER = S::PER, TP = S::TP, LD = S::LD;
  auto& turned = space.turned;
  auto& top = space.top;
  const int tid = threadIdx.x, had = spot.had, end = spot.end;
  const void* src = values ? x.v : x.k;
  const int64_t st = values ? x.vt : x.kt, sh = (values ? x.vh : x.kh) * head;
  // no load depends on a branch (a token that is not new reads a neighbour's row), so that all are under way at once
  typedef typename Elem<DT>::T T;
  constexpr int W = sizeof(T) / 2;  // 16-byte words of 8 entries
  u32x4_t raw[PER][W];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    int t = S::token(tid, i);
    t = t < had ? had : (t >= end ? end - 1 : t);
    const T* from = static_cast<const T*>(src) + (spot.base + t) * st + sh + S::entry(tid);
#pragma unroll
    for (int w = 0; w < W; ++w) raw[i][w] = reinterpret_cast<const u32x4_t*>(from)[w];
  }
  const int32_t pg = spot.inside && spot.entry >= 0 && spot.entry < c.pages ? spot.entry : -1;
  if (pg < 0) return;
  const int64_t slot = static_cast<int64_t>(pg) * c.heads + head;
  float* scales = (values ? c.vs : c.ks) + slot;
  const float old = had ? *scales : 0.0f;
  // values: old codes that share a 16-byte piece with new ones are fetched meanwhile
  constexpr int PIECES = D * PAGE / 16 / NT;
  uint8_t* const block = reinterpret_cast<uint8_t*>(values ? c.v : c.k) + slot * (D * PAGE);
  u32x4_t kept[PIECES];
  if (values && had % 16) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int at = i * NT + tid, t = at % (PAGE / 16) * 16;
      if (t < had && t + 16 > had) kept[i] = *reinterpret_cast<const u32x4_t*>(block + 16 * at);
    }
  }
  float f[PER][8];
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i][j] = static_cast<float>(reinterpret_cast<const T*>(&raw[i][0])[j]);
  constexpr int BITS = Change::kChanges ? static_cast<int>(kF32) : DT;  // changed entries are floats
  if constexpr (Change::kChanges) change(f);
  // the largest magnitude, as the integer that its bits are
  uint32_t big;
  if constexpr (Change::kChanges) {
    big = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) big = max(big, __builtin_bit_cast(uint32_t, f[i][j]) & 0x7fffffffu);
  } else {
    big = largest_bits<DT, PER * W>(&raw[0][0]);
  }
  uint32_t bits = wide_max<NT>(big, top);
  constexpr uint32_t kInf = BITS == kF32 ? 0x7f800000u : (BITS == kBF16 ? 0x7f80u : 0x7c00u);
  const bool odd = bits >= kInf;  // an infinity or a NaN: the largest finite one is looked for value by value
  if (odd) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = __builtin_fabsf(f[i][j]);
        m = v < __builtin_inff() ? __builtin_fmaxf(m, v) : m;
      }
    __syncthreads();
    bits = wide_max<NT>(__builtin_bit_cast(uint32_t, m), top);
  }
  float most;
  if constexpr (BITS == kF32) most = __builtin_bit_cast(float, bits);
  else most = odd ? __builtin_bit_cast(float, bits) : static_cast<float>(__builtin_bit_cast(T, static_cast<uint16_t>(bits)));
  const float need = __builtin_fmaxf(most * kInv127, kScaleFloor);
  const bool grow = !(need <= old);
  const float scale = grow ? __builtin_fmaxf(need, kScaleGrow * old) : old;
  const float inv = 1.0f / scale, ratio = old / scale;
  if (tid == 0 && grow) *scales = scale;

  const auto write = [&](auto finite) {
    constexpr bool F = decltype(finite)::value;
    if (!values) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int t = S::token(tid, i);
        u32x2_t* to = reinterpret_cast<u32x2_t*>(block + t * D + S::entry(tid));
        if (t >= had && t < end) {
          *to = u32x2_t{codes_of<F>(&f[i][0], inv), codes_of<F>(&f[i][4], inv)};
        } else if (t < had && grow) {
          const u32x2_t q = *to;
          *to = u32x2_t{rescale4(q[0], ratio), rescale4(q[1], ratio)};
        }
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < PER; i += TP) {
      uint8_t* to = &turned[S::entry(tid) * LD + S::token(tid, i)];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < TP; ++k) x[k] = f[i + k][j];
        const uint32_t q = codes_of<F>(x, inv);
        if constexpr (TP == 4) *reinterpret_cast<uint32_t*>(to + j * LD) = q;
        else *reinterpret_cast<uint16_t*>(to + j * LD) = static_cast<uint16_t>(q);
      }
    }
  };
  if (odd) write(std::false_type{});
  else write(std::true_type{});
  if (!values) return;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int at = i * NT + tid, e = at / (PAGE / 16), t = at % (PAGE / 16) * 16;
    if (t >= end || (t + 16 <= had && !grow)) continue;  // nothing to write here
    u32x4_t* to = reinterpret_cast<u32x4_t*>(block + 16 * at);
    u32x4_t q;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = *reinterpret_cast<const uint32_t*>(&turned[e * LD + t + 4 * j]);
    if (t < had) {
      u32x4_t o = t + 16 > had ? kept[i] : *to;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t mask = below(t + 4 * j, had);
        if (grow) o[j] = rescale4(o[j], ratio);
        q[j] = (o[j] & mask) | (q[j] & ~mask);
      }
    }
    *to = q;
  }
}

}  // namespace orbq
