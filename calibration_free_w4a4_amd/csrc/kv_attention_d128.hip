// kv_attention for heads of 128 entries.
#include "kv_attention_kernel.h"

namespace orbq {
template int launch_attn<128>(const AttnArgs&, const AttnPlan&, hipStream_t);
}
