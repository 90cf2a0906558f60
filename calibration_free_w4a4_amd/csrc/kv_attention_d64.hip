// kv_attention for heads of 64 entries.
#include "kv_attention_kernel.h"

namespace orbq {
template int launch_attn<64>(const AttnArgs&, const AttnPlan&, hipStream_t);
}
