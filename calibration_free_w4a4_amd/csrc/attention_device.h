// Device helpers of the attention-side kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "attention.h"

namespace orbq {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

template <int DT> struct Elem;
template <> struct Elem<kF32> { using T = float; };
template <> struct Elem<kBF16> { using T = __bf16; };
template <> struct Elem<kF16> { using T = _Float16; };

// E consecutive elements as floats, by one load or store where E elements are 16 or 8 bytes
template <int DT, int E> struct Vec {
  using T = typename Elem<DT>::T;
  typedef T V __attribute__((ext_vector_type(E)));
  static __device__ __forceinline__ void load(const void* base, int64_t at, float* f) {
    if constexpr (E == 1) {
      f[0] = static_cast<float>(static_cast<const T*>(base)[at]);
    } else {
      const V v = *reinterpret_cast<const V*>(static_cast<const T*>(base) + at);
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = static_cast<float>(v[i]);
    }
  }
  static __device__ __forceinline__ void store(void* base, int64_t at, const float* f) {
    if constexpr (E == 1) {
      static_cast<T*>(base)[at] = static_cast<T>(f[0]);
    } else {
      V v;
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = static_cast<T>(f[i]);
      *reinterpret_cast<V*>(static_cast<T*>(base) + at) = v;
    }
  }
};

// The rows of sequence b in the packed arrays, kept inside [0, total) whatever cu holds: the first of them, how many a
// call processes, and how many there are (total is at most 2^30).
__device__ __forceinline__ void rows_of(const int32_t* cu, int64_t total, int32_t batch, int32_t max_rows, int32_t b,
                                        int64_t* row0, int32_t* rows, int32_t* all) {
  int64_t r0, r1;
  if (cu) {
    r0 = cu[b];
    r1 = cu[b + 1];
    r0 = r0 < 0 ? 0 : (r0 > total ? total : r0);
    r1 = r1 < r0 ? r0 : (r1 > total ? total : r1);
  } else {
    const int64_t each = total / batch;
    r0 = each * b;
    r1 = r0 + each;
  }
  *row0 = r0;
  *all = static_cast<int32_t>(r1 - r0);
  *rows = *all < max_rows ? *all : max_rows;
}

// Page of block p of sequence b, or -1 where the table has none (entries outside the cache are
// treated as absent, so that a wrong table cannot make a kernel leave its buffers).
__device__ __forceinline__ int32_t page_of(const KvCache& c, int32_t b, int64_t p) {
  if (p < 0 || p >= c.max_pages) return -1;
  const int32_t pg = c.table[b * c.ldt + p];
  return pg >= 0 && pg < c.pages ? pg : -1;
}

}  // namespace orbq
