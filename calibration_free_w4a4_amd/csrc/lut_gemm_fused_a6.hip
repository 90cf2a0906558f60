// lut_gemm kernels with the fused epilogue for 6-bit activation codes.
#include "lut_gemm_kernel.h"

namespace orbq {
namespace lg {

hipError_t launch_fused_a6(int bw, int cfg, bool out_bf16, const FusedArgs& a, int grid, size_t lds, hipStream_t st) {
  return launch_ba<6>(bw, cfg, out_bf16, a, grid, lds, st);
}

}  // namespace lg
}  // namespace orbq
