// The attention of several new tokens per stream on the matrix cores, for
// bf16 queries over e4m3 caches.
#include "kextend_mfma.h"

namespace convt {

hipError_t launch_extend_bf16_q8(const ExtendArgs &a, const ExtendTiles &t, hipStream_t stream) {
    return run_dims<__bf16, true>(a, t, stream);
}

}  // namespace convt
