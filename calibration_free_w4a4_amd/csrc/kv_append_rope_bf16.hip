// kv_append_rope for inputs of one type (a translation unit each, so that they compile in parallel).
#include "kv_append_rope_kernel.h"

namespace orbq {

int launch_kv_append_rope_bf16(const KvCache& c, const KvTokens& x, const TurnArgs& r, hipStream_t stream) { return by_d<kBF16>(c, x, r, stream); }

}  // namespace orbq
