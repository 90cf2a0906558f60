// lut_gemm host side: tile choice, launch chunking and the dispatch over bit widths.  The
// kernel and its design notes are in lut_gemm_kernel.h.
#include "lut_gemm_kernel.h"

namespace orbq {
namespace lg {
namespace {

size_t lut_bytes(int bits) { return bits == 6 ? 4096 * 4 : 0; }

}  // namespace

GemmPlan plan_gemm(const DecodeParams& da, const DecodeParams& dw, int64_t n, int64_t m, int64_t d, GemmArgs* a) {
  a->xrow_bytes = static_cast<int32_t>(d * da.bits / 8);
  a->wrow_bytes = static_cast<int32_t>(d * dw.bits / 8);
  a->nk = static_cast<int32_t>(d / KT);
  tab4(da, &a->lt_lo_a, &a->lt_hi_a, &a->ht_lo_a, &a->ht_hi_a);
  tab4(dw, &a->lt_lo_w, &a->lt_hi_w, &a->ht_lo_w, &a->ht_hi_w);
  for (int i = 0; i < 32; ++i) {
    a->mag_a[i] = da.mag[i];
    a->mag_w[i] = dw.mag[i];
  }
  // tile shape: the one that leaves the least idle work when the tiles are dealt to the
  // compute units in rounds (384 x 192 needs its LDS stages plus the tables to fit in 160 KB)
  const int cus = device_cus();
  const size_t luts = lut_bytes(da.bits) + lut_bytes(dw.bits);
  int cfg = 1;
  double best = 1e300;
  for (int k = 0; k < 2; ++k) {
    const int64_t bm = k == 0 ? 384 : 256, bn = k == 0 ? 192 : 256;
    const size_t lds = (k == 0 ? Cfg<384, 192>::LDS : Cfg<256, 256>::LDS) + luts;
    if (lds > 160 * 1024) continue;
    const int64_t tiles = ((n + bm - 1) / bm) * ((m + bn - 1) / bn);
    const int64_t rounds = (tiles + cus - 1) / cus;
    const double cost = static_cast<double>(rounds) * bm * bn * (k == 0 ? 1.0 : 1.0001);
    if (cost < best) {
      best = cost;
      cfg = k;
    }
  }
  return GemmPlan{cfg, cfg == 0 ? 384 : 256, cfg == 0 ? 192 : 256,
                  (cfg == 0 ? Cfg<384, 192>::LDS : Cfg<256, 256>::LDS) + luts};
}

int part_of(const GemmPlan& p, const GemmArgs& a, int64_t r0, int64_t rows, int64_t c0, int64_t cols, int64_t esz, GemmArgs* b) {
  b->n = rows;
  b->m = cols;
  b->xc = a.xc + r0 * a.xrow_bytes;
  b->xs = a.xs + r0;
  b->wc = a.wc + c0 * a.wrow_bytes;
  b->wn = a.wn + c0;
  b->Y = static_cast<unsigned char*>(a.Y) + (r0 * a.ldy + c0) * esz;
  b->tiles_n = static_cast<int32_t>((rows + p.bm - 1) / p.bm);
  b->tiles_m = static_cast<int32_t>((cols + p.bn - 1) / p.bn);
  // grouped XCD order when the column tiles split evenly over the 8 XCDs: groups of token
  // tiles x the XCD's cw column tiles, sized to about one round of its compute units.
  // Measured at 4608 x 3072 -> 12288: fetched bytes 195 -> 109 MB per launch (9216 tokens:
  // 709 -> 212 MB), the time unchanged (285.3 against 285.8 us); outputs identical.
  b->group_n = 0;
  if (b->tiles_m % 8 == 0) {
    const int cw = b->tiles_m / 8;
    b->group_n = std::max(1, (device_cus() / 8) / cw);
  }
  return b->tiles_n * b->tiles_m;
}

}  // namespace lg

using namespace lg;

int device_cus() {
  static thread_local int cached_dev = -1, cached_cus = 0;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 256;
  if (dev != cached_dev) {
    int cus = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) cus = 256;
    cached_dev = dev;
    cached_cus = cus;
  }
  return cached_cus;
}

int launch_lut_gemm(const uint8_t* x_codes, const float* x_norms, const DecodeParams& da, const uint8_t* w_codes,
                    const uint16_t* w_norms, const DecodeParams& dw, int64_t n, int64_t m, int64_t d, void* Y,
                    int y_bf16, int64_t ldy, int act, hipStream_t stream) {
  GemmArgs a{};
  const GemmPlan p = plan_gemm(da, dw, n, m, d, &a);
  a.act = act;
  a.xc = x_codes;
  a.xs = x_norms;
  a.wc = w_codes;
  a.wn = w_norms;
  a.Y = Y;
  a.ldy = ldy;
  // launches over row / column blocks keep every code extent addressable with 32-bit offsets
  const int64_t max_rows_x = std::max<int64_t>(p.bm, (int64_t(1) << 31) / a.xrow_bytes / p.bm * p.bm);
  const int64_t max_rows_w = std::max<int64_t>(p.bn, (int64_t(1) << 31) / a.wrow_bytes / p.bn * p.bn);
  hipError_t e = hipSuccess;
  for (int64_t r0 = 0; r0 < n && e == hipSuccess; r0 += max_rows_x) {
    for (int64_t c0 = 0; c0 < m && e == hipSuccess; c0 += max_rows_w) {
      GemmArgs b = a;
      const int grid = part_of(p, a, r0, std::min(max_rows_x, n - r0), c0, std::min(max_rows_w, m - c0), y_bf16 ? 2 : 4, &b);
      switch (da.bits) {
        case 2: e = launch_gemm_a2(dw.bits, p.cfg, y_bf16 != 0, b, grid, p.lds, stream); break;
        case 3: e = launch_gemm_a3(dw.bits, p.cfg, y_bf16 != 0, b, grid, p.lds, stream); break;
        case 4: e = launch_gemm_a4(dw.bits, p.cfg, y_bf16 != 0, b, grid, p.lds, stream); break;
        case 16: e = launch_gemm_abf(dw.bits, p.cfg, y_bf16 != 0, b, grid, p.lds, stream); break;
        default: e = launch_gemm_a6(dw.bits, p.cfg, y_bf16 != 0, b, grid, p.lds, stream); break;
      }
    }
  }
  return static_cast<int>(e);
}

int launch_lut_gemm_fused(const uint8_t* x_codes, const float* x_norms, const DecodeParams& da, const uint8_t* w_codes,
                          const uint16_t* w_norms, const DecodeParams& dw, int64_t n, int64_t m, int64_t d, void* Y,
                          int y_bf16, int64_t ldy, const ProductEpilogue& ep, hipStream_t stream) {
  FusedArgs a{};
  const GemmPlan p = plan_gemm(da, dw, n, m, d, &a);
  a.act = ep.act;
  a.xc = x_codes;
  a.xs = x_norms;
  a.wc = w_codes;
  a.wn = w_norms;
  a.Y = Y;
  a.ldy = ldy;
  const int64_t max_rows_x = std::max<int64_t>(p.bm, (int64_t(1) << 31) / a.xrow_bytes / p.bm * p.bm);
  const int64_t max_rows_w = std::max<int64_t>(p.bn, (int64_t(1) << 31) / a.wrow_bytes / p.bn * p.bn);
  const int64_t esz = y_bf16 ? 2 : 4;
  const size_t lds = std::max<size_t>(p.lds, p.cfg == 0 ? FusedLds<384, 192>::kBytes : FusedLds<256, 256>::kBytes);
  hipError_t e = hipSuccess;
  for (int64_t r0 = 0; r0 < n && e == hipSuccess; r0 += max_rows_x) {
    for (int64_t c0 = 0; c0 < m && e == hipSuccess; c0 += max_rows_w) {
      FusedArgs b = a;
      const int grid = part_of(p, a, r0, std::min(max_rows_x, n - r0), c0, std::min(max_rows_w, m - c0), esz, &b);
      b.e = epilogue_args(ep, n, r0, c0, esz);
      switch (da.bits) {
        case 2: e = launch_fused_a2(dw.bits, p.cfg, y_bf16 != 0, b, grid, lds, stream); break;
        case 3: e = launch_fused_a3(dw.bits, p.cfg, y_bf16 != 0, b, grid, lds, stream); break;
        case 4: e = launch_fused_a4(dw.bits, p.cfg, y_bf16 != 0, b, grid, lds, stream); break;
        case 16: e = launch_fused_abf(dw.bits, p.cfg, y_bf16 != 0, b, grid, lds, stream); break;
        default: e = launch_fused_a6(dw.bits, p.cfg, y_bf16 != 0, b, grid, lds, stream); break;
      }
    }
  }
  return static_cast<int>(e);
}
}  // namespace orbq
