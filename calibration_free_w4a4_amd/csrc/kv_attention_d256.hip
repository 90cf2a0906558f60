// kv_attention for heads of 256 entries.
#include "kv_attention_kernel.h"

namespace orbq {
template int launch_attn<256>(const AttnArgs&, const AttnPlan&, hipStream_t);
}
