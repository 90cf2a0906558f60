// Host side of the few-row products with the fused epilogue (lut_gemm_few_kernel.h): when they are taken, and how they are
// cut into workgroups.
#include "lut_gemm_few_kernel.h"

namespace orbq {

using namespace lg;

// Token rows up to which the few-row form is taken (d in whole super-steps).
constexpr int64_t kFewRows = 64;

bool takes_few_rows(int64_t n, int64_t d) { return n <= kFewRows && d % kFewSS == 0; }

int launch_lut_gemm_few(const uint8_t* x_codes, const float* x_norms, const DecodeParams& da, const uint8_t* w_codes,
                        const uint16_t* w_norms, const DecodeParams& dw, int64_t n, int64_t m, int64_t d, void* Y,
                        int y_bf16, int64_t ldy, const ProductEpilogue& ep, hipStream_t stream) {
  FewArgs a{};
  a.xc = x_codes;
  a.xs = x_norms;
  a.wc = w_codes;
  a.wn = w_norms;
  a.Y = Y;
  a.ldy = ldy;
  a.m = m;
  a.n = static_cast<int32_t>(n);
  a.xrb = static_cast<int32_t>(d * da.bits / 8);
  a.wrb = static_cast<int32_t>(d * dw.bits / 8);
  a.nss = static_cast<int32_t>(d / kFewSS);
  a.per = (a.nss + kFewSplits - 1) / kFewSplits;
  a.splits = (a.nss + a.per - 1) / a.per;
  a.act = ep.act;
  a.y_bf16 = y_bf16;
  tab4(da, &a.ta.lt_lo, &a.ta.lt_hi, &a.ta.ht_lo, &a.ta.ht_hi);
  tab4(dw, &a.tw.lt_lo, &a.tw.lt_hi, &a.tw.ht_lo, &a.tw.ht_hi);
  for (int i = 0; i < 32; ++i) {
    a.mag_a[i] = da.mag[i];
    a.mag_w[i] = dw.mag[i];
  }
  a.e = epilogue_args(ep, n, 0, 0, y_bf16 ? 2 : 4);
  // weight rows of a workgroup: the fewest whose workgroups fit one for each compute unit, as far as the sums of the
  // splits fit in LDS
  const int64_t cus = device_cus();
  int cb = 1;
  while (cb < 4 && (m + 16 * cb - 1) / (16 * cb) > cus && static_cast<int64_t>(a.splits) * n * 32 * cb * 4 <= 98304) cb *= 2;
  hipError_t e;
  switch (da.bits) {
    case 2: e = launch_few_a2(dw.bits, cb, a, stream); break;
    case 3: e = launch_few_a3(dw.bits, cb, a, stream); break;
    case 4: e = launch_few_a4(dw.bits, cb, a, stream); break;
    default: e = launch_few_a6(dw.bits, cb, a, stream); break;
  }
  return static_cast<int>(e);
}

}  // namespace orbq
