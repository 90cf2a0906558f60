// The few-row products of 6-bit activation codes.
#include "lut_gemm_few_kernel.h"

namespace orbq {
namespace lg {

hipError_t launch_few_a6(int bw, int cb, const FewArgs& a, hipStream_t st) { return launch_few_ba<6>(bw, cb, a, st); }

}  // namespace lg
}  // namespace orbq
