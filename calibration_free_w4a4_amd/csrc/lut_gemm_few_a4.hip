// The few-row products of 4-bit activation codes.
#include "lut_gemm_few_kernel.h"

namespace orbq {
namespace lg {

hipError_t launch_few_a4(int bw, const FewPlan& p, const FewArgs& a, hipStream_t st) { return launch_few_ba<4>(bw, p, a, st); }

}  // namespace lg
}  // namespace orbq
