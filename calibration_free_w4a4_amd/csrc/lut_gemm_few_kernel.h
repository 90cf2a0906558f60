// The codes x codes product with the fused epilogue for few token rows (to 64): the weights' codes are read once and decoded
// once for all tokens, so that the call is bound by their bytes and by latency.  lut_gemm's tiles hold 256 or 384 tokens, of
// which nearly all would be padding, on m / 192 or m / 256 compute units.
//
// As in the weight-only product (a16_gemm.hip) a workgroup owns 16 CB weight rows and its waves take one split of the K
// range each; a super-step covers 128 codes, of which lane (m = l % 16, g = l / 16) holds codes 32 g .. 32 g + 31 of one
// row, tokens and weights alike, decodes them 8 at a time and gives them to v_mfma_f32_16x16x32_bf16.  The splits' sums
// meet in LDS and are added in split order.  The next super-step's codes are under way while one is multiplied.
#pragma once

#include "code_rows.h"

namespace orbq {
namespace lg {

constexpr int kFewSS = 128;        // codes of a super-step
constexpr int kFewSplits = 16;     // waves of a workgroup

struct FewArgs {
  const uint8_t* xc;
  const float* xs;
  const uint8_t* wc;
  const uint16_t* wn;
  void* Y;
  int64_t ldy, m;
  int32_t n, xrb, wrb;             // tokens (at most 16 TB); code bytes of a row
  int32_t nss, per, splits;        // super-steps, of a split, splits
  int32_t act, y_bf16;
  Tab4 ta, tw;
  uint16_t mag_a[32], mag_w[32];
  EpilogueArgs e;
};

// TB, CB: 16-row blocks of tokens and of weights
template <int BA, int BW, int TB, int CB>
__global__ __launch_bounds__(64 * kFewSplits) void k_few(const FewArgs a) {
  constexpr int kRows = 16 * CB;
  __shared__ __align__(16) unsigned char lut_a[BA == 6 ? 4096 * 4 : 16];
  __shared__ __align__(16) unsigned char lut_w[BW == 6 ? 4096 * 4 : 16];
  __shared__ uint16_t mags[64];
  extern __shared__ float red[];  // [splits][n][16 CB]
  const int tid = threadIdx.x, lane = tid & 63, split = tid >> 6, nthreads = blockDim.x;
  if constexpr (needs_lut(BA) || needs_lut(BW)) {
    if (tid < 32) mags[tid] = a.mag_a[tid];
    else if (tid < 64) mags[tid] = a.mag_w[tid - 32];
    __syncthreads();
    build_lut<BA>(mags, lut_a, tid, nthreads);
    build_lut<BW>(mags + 32, lut_w, tid, nthreads);
    __syncthreads();
  }
  const int ss0 = split * a.per, ss1 = min(a.nss, ss0 + a.per);
  const int m16 = lane & 15, g = lane >> 4;
  const int64_t row_base = static_cast<int64_t>(blockIdx.x) * kRows;
  // rows behind the last token and the last weight row read as zeros and are not stored
  const __amdgpu_buffer_rsrc_t xs = uniform_rsrc(a.xc, static_cast<uint32_t>(a.n * a.xrb));
  const __amdgpu_buffer_rsrc_t ws = uniform_rsrc(a.wc + row_base * a.wrb, static_cast<uint32_t>(min<int64_t>(a.m - row_base, kRows) * a.wrb));
  f32x4_t acc[TB][CB];
#pragma unroll
  for (int t = 0; t < TB; ++t)
#pragma unroll
    for (int c = 0; c < CB; ++c) acc[t][c] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  struct Set {
    CodesA16<BA> x[TB];
    CodesA16<BW> w[CB];
  };
  const auto load = [&](Set& s, int ss) {
    const int k0 = ss * kFewSS + 32 * g;
#pragma unroll
    for (int c = 0; c < CB; ++c) s.w[c].load(ws, static_cast<uint32_t>((16 * c + m16) * a.wrb + k0 * BW / 8));
#pragma unroll
    for (int t = 0; t < TB; ++t) s.x[t].load(xs, static_cast<uint32_t>((16 * t + m16) * a.xrb + k0 * BA / 8));
  };
  Set now, next;
  if (ss0 < ss1) load(now, ss0);
  for (int ss = ss0; ss < ss1; ++ss) {
    if (ss + 1 < ss1) load(next, ss + 1);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      bf16x8_t x[TB];
#pragma unroll
      for (int t = 0; t < TB; ++t) x[t] = __builtin_bit_cast(bf16x8_t, now.x[t].get(s, a.ta, lut_a));
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        const bf16x8_t w = __builtin_bit_cast(bf16x8_t, now.w[c].get(s, a.tw, lut_w));
#pragma unroll
        for (int t = 0; t < TB; ++t) acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[t], w, acc[t][c], 0, 0, 0);
      }
    }
    now = next;
  }
  // D[t][n]: t = 4 (lane / 16) + i, n = lane % 16
#pragma unroll
  for (int t = 0; t < TB; ++t)
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int token = 16 * t + 4 * g + i;
        if (token < a.n) red[(split * a.n + token) * kRows + 16 * c + m16] = acc[t][c][i];
      }
  __syncthreads();
  for (int e = tid; e < a.n * kRows; e += nthreads) {
    const int t = e / kRows, c = e - t * kRows;
    const int64_t j = row_base + c;
    if (j >= a.m) continue;
    float sum = 0.0f;
    for (int s = 0; s < a.splits; ++s) sum += red[(s * a.n + t) * kRows + c];
    finish_element(a.e, a.act, sum * a.xs[t] * as_float(a.wn[j]), a.Y, a.ldy, a.y_bf16 != 0, t, j);
  }
}

template <int BA, int BW, int TB> hipError_t launch_few_cb(int cb, const FewArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>((a.m + 16 * cb - 1) / (16 * cb))), block(64 * a.splits);
  const size_t lds = static_cast<size_t>(a.splits) * a.n * 16 * cb * sizeof(float);
  switch (cb) {
    case 1: hipLaunchKernelGGL((k_few<BA, BW, TB, 1>), grid, block, lds, st, a); break;
    case 2: hipLaunchKernelGGL((k_few<BA, BW, TB, 2>), grid, block, lds, st, a); break;
    default: hipLaunchKernelGGL((k_few<BA, BW, TB, 4>), grid, block, lds, st, a); break;
  }
  return hipGetLastError();
}

template <int BA, int BW> hipError_t launch_few_bits(int cb, const FewArgs& a, hipStream_t st) {
  if (a.n <= 16) return launch_few_cb<BA, BW, 1>(cb, a, st);
  if (a.n <= 32) return launch_few_cb<BA, BW, 2>(cb, a, st);
  return launch_few_cb<BA, BW, 4>(cb, a, st);
}

template <int BA> hipError_t launch_few_ba(int bw, int cb, const FewArgs& a, hipStream_t st) {
  if constexpr (BA == 3) {
    return launch_few_bits<3, 3>(cb, a, st);
  } else {
    switch (bw) {
      case 2: return launch_few_bits<BA, 2>(cb, a, st);
      case 4: return launch_few_bits<BA, 4>(cb, a, st);
      default: return launch_few_bits<BA, 6>(cb, a, st);
    }
  }
}

// one translation unit for each activation bit width
hipError_t launch_few_a2(int bw, int cb, const FewArgs& a, hipStream_t st);
hipError_t launch_few_a3(int bw, int cb, const FewArgs& a, hipStream_t st);
hipError_t launch_few_a4(int bw, int cb, const FewArgs& a, hipStream_t st);
hipError_t launch_few_a6(int bw, int cb, const FewArgs& a, hipStream_t st);

}  // namespace lg
}  // namespace orbq
