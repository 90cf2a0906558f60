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
// workgroups write the same page (no atomics; the result does not depend on any order).
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

template <int DT, int D, int PAGE>
__global__ __launch_bounds__(threads_for(D* PAGE)) void k_append(const KvCache c, const KvTokens x) {
  constexpr int NT = threads_for(D * PAGE), PER = D * PAGE / (8 * NT);  // groups of 8 values a thread
  constexpr int LD = PAGE + 4;                                          // LDS pitch of a value row
  __shared__ __attribute__((aligned(16))) uint8_t turned[D * LD];
  __shared__ float top[NT / 64];
  const int tid = threadIdx.x, head = blockIdx.y >> 1, b = blockIdx.z;
  const bool values = blockIdx.y & 1;
  int64_t row0;
  int32_t rows;
  rows_of(x.cu, x.total, c.batch, x.max_rows, b, &row0, &rows);
  const int64_t start = x.first[b];
  if (start < 0 || rows == 0) return;
  const int64_t p = start / PAGE + blockIdx.x;
  const int64_t t0 = p * PAGE;                       // the page's first token
  if (t0 >= start + rows) return;
  const int32_t pg = page_of(c, b, p);
  if (pg < 0) return;
  const int had = static_cast<int>(start > t0 ? start - t0 : 0);                        // tokens held before
  const int end = static_cast<int>(start + rows - t0 < PAGE ? start + rows - t0 : PAGE);  // and after
  const int64_t slot = static_cast<int64_t>(pg) * c.heads + head;
  float* scales = (values ? c.vs : c.ks) + slot;
  const float old = had ? *scales : 0.0f;

  const void* src = values ? x.v : x.k;
  const int64_t st = values ? x.vt : x.kt, sh = (values ? x.vh : x.kh) * head;
  float f[PER][8];
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = i * NT + tid, t = at / (D / 8), e = at % (D / 8) * 8;
    if (t >= had && t < end) {
      const int64_t from = (row0 + t0 + t - start) * st + sh + e;
      if constexpr (DT == kF32) {
        Vec<DT, 4>::load(src, from, f[i]);
        Vec<DT, 4>::load(src, from + 4, f[i] + 4);
      } else {
        Vec<DT, 8>::load(src, from, f[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = __builtin_fabsf(f[i][j]);
        most = a < __builtin_inff() ? __builtin_fmaxf(most, a) : most;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] = 0.0f;
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) most = __builtin_fmaxf(most, __shfl_xor(most, off));
  if constexpr (NT > 64) {
    if ((tid & 63) == 0) top[tid >> 6] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) most = __builtin_fmaxf(most, top[w]);
  }
  const float need = __builtin_fmaxf(most * kInv127, kScaleFloor);
  const bool grow = !(need <= old);
  const float scale = grow ? __builtin_fmaxf(need, kScaleGrow * old) : old;
  const float inv = 1.0f / scale, ratio = old / scale;
  if (tid == 0 && grow) *scales = scale;

  if (!values) {
    uint8_t* dst = reinterpret_cast<uint8_t*>(c.k) + slot * (D * PAGE);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = i * NT + tid, t = at / (D / 8);
      u32x2_t* to = reinterpret_cast<u32x2_t*>(dst + 8 * at);
      if (t >= had && t < end) {
        u32x2_t q = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j >> 2] |= code_of(f[i][j], inv) << (8 * (j & 3));
        *to = q;
      } else if (t < had && grow) {
        const u32x2_t q = *to;
        *to = u32x2_t{rescale4(q[0], ratio), rescale4(q[1], ratio)};
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = i * NT + tid, t = at / (D / 8), e = at % (D / 8) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) turned[(e + j) * LD + t] = static_cast<uint8_t>(code_of(f[i][j], inv));
  }
  __syncthreads();
  uint8_t* dst = reinterpret_cast<uint8_t*>(c.v) + slot * (D * PAGE);
  for (int at = tid; at < D * PAGE / 16; at += NT) {
    const int e = at / (PAGE / 16), t = at % (PAGE / 16) * 16;
    if (t >= end || (t + 16 <= had && !grow)) continue;  // nothing to write here
    u32x4_t* to = reinterpret_cast<u32x4_t*>(dst + 16 * at);
    u32x4_t q;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = *reinterpret_cast<const uint32_t*>(&turned[e * LD + t + 4 * j]);
    if (t < had) {
      u32x4_t o = *to;
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
  constexpr int NT = threads_for(D * PAGE), PER = D * PAGE / (8 * NT);
  constexpr int LD = PAGE + 4;
  __shared__ __attribute__((aligned(16))) uint8_t turned[D * LD];
  const int tid = threadIdx.x, head = blockIdx.y >> 1, b = blockIdx.z;
  const bool values = blockIdx.y & 1;
  int64_t row0;
  int32_t rows;
  rows_of(x.cu, x.total, c.batch, x.max_rows, b, &row0, &rows);
  const int64_t first = x.first[b];
  if (first < 0 || rows == 0) return;
  const int64_t p = first / PAGE + blockIdx.x;
  const int64_t t0 = p * PAGE;
  if (t0 >= first + rows) return;
  const int32_t pg = page_of(c, b, p);
  const int from = static_cast<int>(first > t0 ? first - t0 : 0);
  const int end = static_cast<int>(first + rows - t0 < PAGE ? first + rows - t0 : PAGE);
  const int64_t slot = static_cast<int64_t>(pg < 0 ? 0 : pg) * c.heads + head;
  const float scale = pg < 0 ? 0.0f : (values ? c.vs : c.ks)[slot];
  const uint8_t* src = reinterpret_cast<const uint8_t*>(values ? c.v : c.k) + slot * (D * PAGE);
  if (values) {
    if (pg >= 0) {
      for (int at = tid; at < D * PAGE / 16; at += NT) {
        const int e = at / (PAGE / 16), t = at % (PAGE / 16) * 16;
        const u32x4_t q = *reinterpret_cast<const u32x4_t*>(src + 16 * at);
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t*>(&turned[e * LD + t + 4 * j]) = q[j];
      }
    }
    __syncthreads();
  }
  void* dst = values ? x.v : x.k;
  const int64_t st = values ? x.vt : x.kt, sh = (values ? x.vh : x.kh) * head;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = i * NT + tid, t = at / (D / 8), e = at % (D / 8) * 8;
    if (t < from || t >= end) continue;
    float f[8];
    if (pg < 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    } else if (values) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = static_cast<float>(static_cast<int8_t>(turned[(e + j) * LD + t])) * scale;
    } else {
      const u32x2_t q = *reinterpret_cast<const u32x2_t*>(src + 8 * at);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = static_cast<float>(static_cast<int8_t>(q[j >> 2] >> (8 * (j & 3)))) * scale;
    }
    const int64_t to = (row0 + t0 + t - first) * st + sh + e;
    if constexpr (DT == kF32) {
      Vec<DT, 4>::store(dst, to, f);
      Vec<DT, 4>::store(dst, to + 4, f + 4);
    } else {
      Vec<DT, 8>::store(dst, to, f);
    }
  }
}

template <bool READ, int DT, int D, int PAGE> int launch(const KvCache& c, const KvTokens& x, hipStream_t stream) {
  // pages that max_rows tokens in a row can touch
  const int64_t pages = (static_cast<int64_t>(x.max_rows) + PAGE - 2) / PAGE + 1;
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
