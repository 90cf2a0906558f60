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
#include "kv_cache_device.h"

namespace orbq {
namespace {

template <int DT, int D, int PAGE>
__global__ __launch_bounds__(threads_for(D* PAGE)) void k_append(const KvCache c, const KvTokens x) {
  __shared__ PageSpace<D, PAGE> space;
  PageSpot spot;
  if (!locate_page<PAGE>(c, x, blockIdx.z, blockIdx.x, &spot)) return;
  append_page<DT, D, PAGE>(c, x, spot, blockIdx.y >> 1, blockIdx.y & 1, space, Unchanged{});
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
