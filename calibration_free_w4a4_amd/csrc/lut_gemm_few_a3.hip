// The few-row products of 3-bit activation codes.
#include "lut_gemm_few_kernel.h"

namespace orbq {
namespace lg {

hipError_t launch_few_a3(int bw, const FewPlan& p, const FewArgs& a, hipStream_t st) { return launch_few_ba<3>(bw, p, a, st); }

}  // namespace lg
}  // namespace orbq
