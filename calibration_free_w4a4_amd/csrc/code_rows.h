// Device helpers of the few-row products (a16_gemm.hip, lut_gemm_few_kernel.h): the 32 codes of a lane's slot in a row, by bit width.
#pragma once

#include "lut_gemm_kernel.h"

namespace orbq {
namespace lg {

// A buffer resource from wave-uniform values, forced into scalar registers: the compiler keeps
// values derived from 64-bit compares and selects in VGPRs, which would wrap every load that
// uses the resource in a waterfall loop.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo), 0,
                                           __builtin_amdgcn_readfirstlane(bytes), kBufWord3);
}

template <int BW>
struct CodesA16;  // the 32 codes of one (row, super-step) lane slot and their decode

template <>
struct CodesA16<4> {
  uint4 w;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
    w = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
  }
  __device__ __forceinline__ uint4 get(int s, const Tab4& t, const void*) const {
    const uint32_t x = s == 0 ? w.x : s == 1 ? w.y : s == 2 ? w.z : w.w;
    return decode4_b(x, decode4_a(x, t));
  }
};

template <>
struct CodesA16<2> {
  v2u_t w;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
    w = __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0);
  }
  __device__ __forceinline__ uint4 get(int s, const Tab4& t, const void*) const {
    const uint32_t x = ((s < 2 ? w.x : w.y) >> (16 * (s & 1))) & 0xFFFFu;
    return decode2_b(decode2_a(x, t), t);
  }
};

template <>
struct CodesA16<3> {
  v2u_t a;
  uint32_t b;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
    a = __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0);
    b = __builtin_amdgcn_raw_buffer_load_b32(rs, off + 8, 0, 0);
  }
  __device__ __forceinline__ uint4 get(int s, const Tab4& t, const void*) const {
    // 24 bits per 8 codes: s = 0 -> a.x [0, 24), 1 -> (a.x, a.y) [24, 48), 2 -> (a.y, b) [48, 72), 3 -> b [72, 96)
    const uint32_t x = s == 0 ? a.x : s == 1 ? __builtin_amdgcn_alignbit(a.y, a.x, 24)
                     : s == 2 ? __builtin_amdgcn_alignbit(b, a.y, 16) : (b >> 8);
    return decode3_b(decode3_a(x, t), t);
  }
};

template <>
struct CodesA16<6> {
  uint4 a;
  v2u_t b;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
    a = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
    b = __builtin_amdgcn_raw_buffer_load_b64(rs, off + 16, 0, 0);
  }
  __device__ __forceinline__ uint4 get(int s, const Tab4&, const void* lut) const {
    // 48 bits per 8 codes: s = 0 -> (a.x, a.y lo), 1 -> (a.y hi, a.z), 2 -> (a.w, b.x lo), 3 -> (b.x hi, b.y)
    uint32_t lo, hi;
    if (s == 0) { lo = a.x; hi = a.y & 0xFFFFu; }
    else if (s == 1) { lo = __builtin_amdgcn_alignbit(a.z, a.y, 16); hi = a.z >> 16; }
    else if (s == 2) { lo = a.w; hi = b.x & 0xFFFFu; }
    else { lo = __builtin_amdgcn_alignbit(b.y, b.x, 16); hi = b.y >> 16; }
    return decode6(lo, hi, static_cast<const uint32_t*>(lut));
  }
};

}  // namespace lg
}  // namespace orbq
