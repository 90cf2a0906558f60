// The 8-bit paged cache: quantised as it is written (kv_append), and read back (kv_read).
//
// A page holds `page` tokens of one sequence; each (page, head) has one fp32 scale for its keys and
// one for its values.  Keys lie [page][d], values [d][page]: attention's second product takes its
// operand with the tokens of one entry side by side, and here the turn costs one pass through LDS
// for each value written instead of one for each value attended to.
//
// append, for each (page, head) that the new tokens touch:
//   A = max |x| over the new finite values, need = max(A (1/127), 2^-64);
//   scale = need on a page without earlier tokens; else the old one if it suffices, else
//   max(need, 1.25 old), and the page's earlier codes become rint(code (old / scale));
//   code = rint(x (1/scale)) within +-127; a NaN is written as 0, an infinity as +-127, so that one
//   bad value does not take its block along.
// The factor 1.25 bounds what growing again and again can cost: the roundings of earlier steps shrink
// by it, 0.5 (1 + 1/1.25 + ...) = 2.5 steps of the last scale at most.
//
// One workgroup for each (touched page, head, keys or values): it holds the page's new values in
// registers between the maximum and the quantisation, so every byte crosses HBM once, and no two
// workgroups write the same page (no atomics; the result does not depend on any order).  4680 tokens of 12 heads
// of 128 in bf16: append 10.7 us (29 MB in, 14 out), read 9.5 us; the quantisation's vector work and the chain of
// dependent reads (counts, table, scale) keep it from the memory's rate.  One token for 48 sequences of 8
// heads: 7 us each, latency alone.
#include <type_traits>

#include "attention_device.h"

namespace orbq {
namespace {

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

template <int DT> __device__ __forceinline__ auto half_bits() {
  if constexpr (DT == kF32) return uint32_t{};
  else return uint16_t{};
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

template <int DT, int D, int PAGE>
__global__ __launch_bounds__(threads_for(D* PAGE)) void k_append(const KvCache c, const KvTokens x) {
  using S = Share<D, PAGE>;
  constexpr int NT = S::NT, PER = S::PER, TP = S::TP, LD = S::LD;
  __shared__ __attribute__((aligned(16))) uint8_t turned[D * LD];
  __shared__ uint32_t top[NT / 64];
  const int tid = threadIdx.x, head = blockIdx.y >> 1, b = blockIdx.z;
  const bool values = blockIdx.y & 1;
  int64_t row0;
  int32_t rows, all;
  rows_of(x.cu, x.total, c.batch, x.max_rows, b, &row0, &rows, &all);
  const int64_t start = x.first[b];
  if (start < 0 || rows == 0) return;
  const int64_t p = start / PAGE + blockIdx.x;
  const int64_t t0 = p * PAGE;                       // the page's first token
  if (t0 >= start + rows) return;
  const int had = static_cast<int>(start > t0 ? start - t0 : 0);                        // tokens held before
  const int end = static_cast<int>(start + rows - t0 < PAGE ? start + rows - t0 : PAGE);  // and after
  // the page, and with it the old scale, are looked up while the new values are on their way
  const int32_t entry = c.table[b * c.ldt + (p < c.max_pages ? p : 0)];

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
    const T* from = static_cast<const T*>(src) + (row0 + t0 + t - start) * st + sh + S::entry(tid);
#pragma unroll
    for (int w = 0; w < W; ++w) raw[i][w] = reinterpret_cast<const u32x4_t*>(from)[w];
  }
  const int32_t pg = p < c.max_pages && entry >= 0 && entry < c.pages ? entry : -1;
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
  // the largest magnitude, as the integer that its bits are
  const uint32_t big = largest_bits<DT, PER * W>(&raw[0][0]);
  uint32_t bits = wide_max<NT>(big, top);
  constexpr uint32_t kInf = DT == kF32 ? 0x7f800000u : (DT == kBF16 ? 0x7f80u : 0x7c00u);
  const bool odd = bits >= kInf;  // an infinity or a NaN: the largest finite one is looked for value by value
  float f[PER][8];
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i][j] = static_cast<float>(reinterpret_cast<const T*>(&raw[i][0])[j]);
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
  const float most = odd || DT == kF32 ? __builtin_bit_cast(float, bits)
                                       : static_cast<float>(__builtin_bit_cast(T, static_cast<decltype(half_bits<DT>())>(bits)));
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

template <int DT, int D, int PAGE>
__global__ __launch_bounds__(threads_for(D* PAGE)) void k_read(const KvCache c, const KvTokens x) {
  using S = Share<D, PAGE>;
  constexpr int NT = S::NT, PER = S::PER, TP = S::TP, LD = S::LD;
  __shared__ __attribute__((aligned(16))) uint8_t turned[D * LD];
  const int tid = threadIdx.x, head = blockIdx.y >> 1, b = blockIdx.z;
  const bool values = blockIdx.y & 1;
  int64_t row0;
  int32_t rows, all;
  rows_of(x.cu, x.total, c.batch, x.max_rows, b, &row0, &rows, &all);
  const int64_t first = x.first[b];
  if (rows == 0) return;
  const int64_t p = (first - (first & (PAGE - 1))) / PAGE + blockIdx.x;  // rounded down: pages before token 0 are absent
  const int64_t t0 = p * PAGE;
  if (t0 >= first + rows) return;
  const int32_t pg = page_of(c, b, p);
  const int from = static_cast<int>(first > t0 ? first - t0 : 0);
  const int end = static_cast<int>(first + rows - t0 < PAGE ? first + rows - t0 : PAGE);
  const int64_t slot = static_cast<int64_t>(pg < 0 ? 0 : pg) * c.heads + head;  // an absent page: page 0, times zero
  const float scale = pg < 0 ? 0.0f : (values ? c.vs : c.ks)[slot];
  const uint8_t* src = reinterpret_cast<const uint8_t*>(values ? c.v : c.k) + slot * (D * PAGE);
  if (values) {
#pragma unroll
    for (int i = 0; i < D * PAGE / 16 / NT; ++i) {
      const int at = i * NT + tid, e = at / (PAGE / 16), t = at % (PAGE / 16) * 16;
      const u32x4_t q = *reinterpret_cast<const u32x4_t*>(src + 16 * at);
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t*>(&turned[e * LD + t + 4 * j]) = q[j];
    }
    __syncthreads();
  }
  void* dst = values ? x.v : x.k;
  const int64_t st = values ? x.vt : x.kt, sh = (values ? x.vh : x.kh) * head;
  const int e = S::entry(tid);
#pragma unroll
  for (int i = 0; i < PER; i += TP) {
    float f[TP][8];
    if (values) {
      const uint8_t* at = &turned[e * LD + S::token(tid, i)];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t w;
        if constexpr (TP == 4) w = *reinterpret_cast<const uint32_t*>(at + j * LD);
        else w = *reinterpret_cast<const uint16_t*>(at + j * LD);
#pragma unroll
        for (int k = 0; k < TP; ++k) f[k][j] = static_cast<float>(static_cast<int8_t>(w >> (8 * k)));
      }
    } else {
      u32x2_t q[TP];
#pragma unroll
      for (int k = 0; k < TP; ++k) q[k] = *reinterpret_cast<const u32x2_t*>(src + S::token(tid, i + k) * D + e);
#pragma unroll
      for (int k = 0; k < TP; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[k][j] = static_cast<float>(static_cast<int8_t>(q[k][j >> 2] >> (8 * (j & 3))));
    }
#pragma unroll
    for (int k = 0; k < TP; ++k) {
      const int t = S::token(tid, i + k);
      if (t < from || t >= end) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[k][j] = pg < 0 ? 0.0f : f[k][j] * scale;
        asm("" : "+v"(f[k][j]));  // an fp32 product, then the output type: not one rounding of both here and two there
      }
      const int64_t to = (row0 + t0 + t - first) * st + sh + e;
      if constexpr (DT == kF32) {
        Vec<DT, 4>::store(dst, to, f[k]);
        Vec<DT, 4>::store(dst, to + 4, f[k] + 4);
      } else {
        Vec<DT, 8>::store(dst, to, f[k]);
      }
    }
  }
}

template <bool READ, int DT, int D, int PAGE> int launch(const KvCache& c, const KvTokens& x, hipStream_t stream) {
  // pages that max_rows tokens in a row can touch
  int64_t pages = (static_cast<int64_t>(x.max_rows) + PAGE - 2) / PAGE + 1;
  if (!READ && pages > c.max_pages) pages = c.max_pages;  // nothing is written behind the table (which has pages)
  const dim3 grid(static_cast<uint32_t>(pages), 2 * c.heads, c.batch), block(threads_for(D * PAGE));
  if constexpr (READ) hipLaunchKernelGGL((k_read<DT, D, PAGE>), grid, block, 0, stream, c, x);
  else hipLaunchKernelGGL((k_append<DT, D, PAGE>), grid, block, 0, stream, c, x);
  return static_cast<int>(hipGetLastError());
}

template <bool READ, int DT, int D> int by_page(const KvCache& c, const KvTokens& x, hipStream_t stream) {
  switch (c.page) {
    case 16: return launch<READ, DT, D, 16>(c, x, stream);
    case 32: return launch<READ, DT, D, 32>(c, x, stream);
    case 64: return launch<READ, DT, D, 64>(c, x, stream);
    default: return launch<READ, DT, D, 128>(c, x, stream);
  }
}

template <bool READ, int DT> int by_d(const KvCache& c, const KvTokens& x, hipStream_t stream) {
  switch (c.d) {
    case 64: return by_page<READ, DT, 64>(c, x, stream);
    case 128: return by_page<READ, DT, 128>(c, x, stream);
    default: return by_page<READ, DT, 256>(c, x, stream);
  }
}

template <bool READ> int by_type(const KvCache& c, const KvTokens& x, int dtype, hipStream_t stream) {
  switch (dtype) {
    case kF32: return by_d<READ, kF32>(c, x, stream);
    case kBF16: return by_d<READ, kBF16>(c, x, stream);
    default: return by_d<READ, kF16>(c, x, stream);
  }
}

}  // namespace

int launch_kv_append(const KvCache& c, const KvTokens& x, int dtype, hipStream_t stream) {
  return by_type<false>(c, x, dtype, stream);
}
int launch_kv_read(const KvCache& c, const KvTokens& x, int dtype, hipStream_t stream) {
  return by_type<true>(c, x, dtype, stream);
}

}  // namespace orbq
