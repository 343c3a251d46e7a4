// The attention of several new tokens per stream on the matrix cores, for
// bf16 queries over caches of that type.
#include "kextend_mfma.h"

namespace convt {

hipError_t launch_extend_bf16(const ExtendArgs &a, const ExtendTiles &t, hipStream_t stream) {
    return run_dims<__bf16, false>(a, t, stream);
}

}  // namespace convt
