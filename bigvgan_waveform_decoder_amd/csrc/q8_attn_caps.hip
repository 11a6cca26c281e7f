// Attention over the 8-bit paged cache with rules, 16-bit types under caps that
// their scores may lie far below (kernels: q8_attn.h).
#include "q8_attn.h"

namespace avae {

hipError_t launch_attn_caps_q8(int dtype, const AttnQ8& a, const AttnRules& x, const CacheQ8& c,
                               const Ragged& r, void* ws, hipStream_t stream) {
    return launch_attn(dtype, a, FineRules(x), c, r, ws, "attn_caps_q8_kernel", stream);
}

}  // namespace avae
