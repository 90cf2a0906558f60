// Host side of the few-row products with the fused epilogue (lut_gemm_few_kernel.h): when they are taken, and how they are
// cut into workgroups.
#include "lut_gemm_few_kernel.h"

namespace orbq {

using namespace lg;

namespace {

// 64 tokens (or the 16 or 32 that there are) x 16 weight rows on 16 waves as long as a round of the compute units takes them
// all, then 32 weight rows, and when these come in rounds 4 waves, of which a unit has several workgroups.  Microseconds,
// A4 x W4, 16 waves x 16 rows / 16 or 8 x 32 / 4 x 32:
//   1536 -> 1536, 128, 256 and 1024 tokens    7.1 / 8.7 / 12.6     11.8 / 8.9 / 12.7     31 / 24 / 20
//   8960 -> 1536, 128, 256 and 2048 tokens   19.6 / 23 / 28         36 / 24 / 28        213 / 110 / 106
//   1536 -> 8960, 5 and 128 tokens            6.4 / 5.9 / -         25 / 23 / 20
// 32 tokens x 32 rows never came out ahead of x 16 (1536 -> 8960: 8.5 against 8.3).
FewPlan plan_few(int64_t n, int64_t m, int64_t d) {
  const int64_t cus = device_cus(), nss = (d + kFewSS - 1) / kFewSS;
  FewPlan p;
  p.tokens = n <= 16 ? 16 : n <= 32 ? 32 : 64;
  const auto blocks = [&](int cb) { return (n + p.tokens - 1) / p.tokens * ((m + 16 * cb - 1) / (16 * cb)); };
  p.cb = p.tokens == 32 || blocks(1) <= cus ? 1 : 2;
  p.splits = 16;
  if (p.tokens == 64 && blocks(2) > cus) p.splits = 4;
  // the splits' sums have 96 KiB of LDS, beside the tables of 6-bit codes
  else if (std::min<int64_t>(p.splits, nss) * std::min<int64_t>(n, p.tokens) * 16 * p.cb * 4 > 98304) p.splits = 8;
  return p;
}

}  // namespace

// To 64 tokens always (8960 -> 1536: 20 against 168 us); beyond as long as the time expected is less than that of the
// tiles, both as measured for A4 x W4: a block of 64 x 32 takes a compute unit 0.2 us for each super-step and 3.6 besides, a
// round of tiles 2.4 for each super-step and 10 besides.  Either side of it, few rows against tiles: 1536 -> 8960, 256 and
// 512 tokens 29 / 42 and 53 / 43 us; 4096 -> 4096, 1024 and 2048 tokens 78 / 88 and 136 / 90; other bit widths are within a
// third of that, and on the same side but for A6 x W4 (512 tokens of the former 78 / 100).
bool takes_few_rows(int64_t n, int64_t m, int64_t d) {
  if (n > 4096) return false;
  if (n <= 64) return true;
  const int64_t cus = device_cus(), nss = (d + kFewSS - 1) / kFewSS;
  const int64_t tiles = (n + 255) / 256 * ((m + 255) / 256), blocks = (n + 63) / 64 * ((m + 31) / 32);
  return blocks * (nss + 18) < 12 * ((tiles + cus - 1) / cus) * cus * (nss + 4);
}

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
  a.nss = static_cast<int32_t>((d + kFewSS - 1) / kFewSS);
  a.half = d % kFewSS != 0;
  const FewPlan p = plan_few(n, m, d);
  a.per = (a.nss + p.splits - 1) / p.splits;
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
  hipError_t e;
  switch (da.bits) {
    case 2: e = launch_few_a2(dw.bits, p, a, stream); break;
    case 3: e = launch_few_a3(dw.bits, p, a, stream); break;
    case 4: e = launch_few_a4(dw.bits, p, a, stream); break;
    default: e = launch_few_a6(dw.bits, p, a, stream); break;
  }
  return static_cast<int>(e);
}

}  // namespace orbq
