// The codes x codes product with the fused epilogue for few token rows: lut_gemm's tiles hold 256 or 384 tokens, of which
// nearly all would be padding, and one workgroup walks the whole K range of a tile while compute units without a tile idle.
// Here the K range is split over a workgroup's waves and a workgroup has 16 to 64 tokens, so that a few rows are spread over
// the chip.  Up to 64 tokens the weights' codes are read and decoded once: bound by latency, and with 64 tokens by the
// decoding (A4 x W4, 5 tokens x 1536 -> 8960: 5.9 us, the 6.9 MB of codes at 1.2 TB/s; 64 tokens 16 us; the tiles 39 and 41).
//
// As in the weight-only product (a16_gemm.hip) a workgroup owns 16 CB weight rows and its waves take one split of the K
// range each; a super-step covers 128 codes, of which lane (m = l % 16, g = l / 16) holds codes 32 g .. 32 g + 31 of one
// row, tokens and weights alike, decodes them 8 at a time and gives them to v_mfma_f32_16x16x32_bf16.  The splits' sums
// meet in LDS and are added in split order.  The next super-step's codes are under way while one is multiplied.  Of a last half
// super-step the tokens' other half is made zeros, whatever the codes there are.
#pragma once

#include <algorithm>

#include "code_rows.h"

namespace orbq {
namespace lg {

constexpr int kFewSS = 128;        // codes of a super-step

// How a product is cut: tokens and 16-row blocks of weights of a workgroup, its waves
struct FewPlan {
  int tokens, cb, splits;
};

struct FewArgs {
  const uint8_t* xc;
  const float* xs;
  const uint8_t* wc;
  const uint16_t* wn;
  void* Y;
  int64_t ldy, m;
  int32_t n, xrb, wrb;             // tokens; code bytes of a row
  int32_t nss, per, splits;        // super-steps, of a split, splits
  int32_t half;                    // the last super-step is half one
  int32_t act, y_bf16;
  Tab4 ta, tw;
  uint16_t mag_a[32], mag_w[32];
  EpilogueArgs e;
};

// TB, CB: 16-row blocks of tokens and of weights; blockIdx.y counts the 16 TB tokens.  HALF: d ends with half a super-step
// (looked for in one kernel for both, it took 15 % of 64 tokens' time)
template <int BA, int BW, int TB, int CB, int SPLITS, bool HALF>
__global__ __launch_bounds__(64 * SPLITS) void k_few(const FewArgs a) {
  constexpr int kRows = 16 * CB;
  __shared__ __align__(16) unsigned char lut_a[BA == 6 ? 4096 * 4 : 16];
  __shared__ __align__(16) unsigned char lut_w[BW == 6 ? 4096 * 4 : 16];
  __shared__ uint16_t mags[64];
  extern __shared__ float red[];  // [splits][tokens here][16 CB]
  const int tid = threadIdx.x, lane = tid & 63, split = __builtin_amdgcn_readfirstlane(tid >> 6), nthreads = blockDim.x;
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
  const int token_base = 16 * TB * blockIdx.y, tokens = min(a.n - token_base, 16 * TB);
  // rows behind the last token and the last weight row read as zeros and are not stored
  const __amdgpu_buffer_rsrc_t xs = uniform_rsrc(a.xc + static_cast<int64_t>(token_base) * a.xrb, static_cast<uint32_t>(tokens * a.xrb));
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
    const bool tail = HALF && ss + 1 == a.nss;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      bf16x8_t x[TB];
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        uint4 v = now.x[t].get(s, a.ta, lut_a);
        if (HALF && tail) v = g < 2 ? v : uint4{0, 0, 0, 0};
        x[t] = __builtin_bit_cast(bf16x8_t, v);
      }
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
        if (token < tokens) red[(split * tokens + token) * kRows + 16 * c + m16] = acc[t][c][i];
      }
  __syncthreads();
  for (int e = tid; e < tokens * kRows; e += nthreads) {
    const int t = e / kRows, c = e - t * kRows;
    const int64_t j = row_base + c;
    if (j >= a.m) continue;
    float sum = 0.0f;
    for (int s = 0; s < a.splits; ++s) sum += red[(s * tokens + t) * kRows + c];
    finish_element(a.e, a.act, sum * a.xs[token_base + t] * as_float(a.wn[j]), a.Y, a.ldy, a.y_bf16 != 0, token_base + t, j);
  }
}

template <int BA, int BW, int TB, int CB, int SPLITS> hipError_t launch_few_form(const FewArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>((a.m + 16 * CB - 1) / (16 * CB)), (a.n + 16 * TB - 1) / (16 * TB)), block(64 * a.splits);
  const size_t lds = static_cast<size_t>(a.splits) * std::min(a.n, 16 * TB) * 16 * CB * sizeof(float);
  if (a.half) hipLaunchKernelGGL((k_few<BA, BW, TB, CB, SPLITS, true>), grid, block, lds, st, a);
  else hipLaunchKernelGGL((k_few<BA, BW, TB, CB, SPLITS, false>), grid, block, lds, st, a);
  return hipGetLastError();
}

template <int BA, int BW> hipError_t launch_few_bits(const FewPlan& p, const FewArgs& a, hipStream_t st) {
  if (p.splits == 4) return launch_few_form<BA, BW, 4, 2, 4>(a, st);
  if (p.tokens == 16) return p.cb == 1 ? launch_few_form<BA, BW, 1, 1, 16>(a, st) : launch_few_form<BA, BW, 1, 2, 16>(a, st);
  if (p.tokens == 32) return launch_few_form<BA, BW, 2, 1, 16>(a, st);
  return p.cb == 1 ? launch_few_form<BA, BW, 4, 1, 16>(a, st) : launch_few_form<BA, BW, 4, 2, 16>(a, st);
}

template <int BA> hipError_t launch_few_ba(int bw, const FewPlan& p, const FewArgs& a, hipStream_t st) {
  if constexpr (BA == 3) {
    return launch_few_bits<3, 3>(p, a, st);
  } else {
    switch (bw) {
      case 2: return launch_few_bits<BA, 2>(p, a, st);
      case 4: return launch_few_bits<BA, 4>(p, a, st);
      default: return launch_few_bits<BA, 6>(p, a, st);
    }
  }
}

// one translation unit for each activation bit width
hipError_t launch_few_a2(int bw, const FewPlan& p, const FewArgs& a, hipStream_t st);
hipError_t launch_few_a3(int bw, const FewPlan& p, const FewArgs& a, hipStream_t st);
hipError_t launch_few_a4(int bw, const FewPlan& p, const FewArgs& a, hipStream_t st);
hipError_t launch_few_a6(int bw, const FewPlan& p, const FewArgs& a, hipStream_t st);

}  // namespace lg
}  // namespace orbq
