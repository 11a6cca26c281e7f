// Attention over the 8-bit paged cache with rules: capped scores, biases by
// distance, a prefix in view of all rows, trees of drafts (kernels: q8_attn.h).
#include "q8_attn.h"

namespace avae {

hipError_t launch_attn_rules_q8(int dtype, const AttnQ8& a, const AttnRules& x, const CacheQ8& c,
                                const Ragged& r, void* ws, hipStream_t stream) {
    if (dtype != AVAE_F32 && x.cap > kQuickCap)
        return launch_attn_caps_q8(dtype, a, x, c, r, ws, stream);
    return launch_attn(dtype, a, x, c, r, ws, "attn_rules_q8_kernel", stream);
}

}  // namespace avae
