// packed_fwd_f16.cu -- packed_fwd.cuh for binary16.
#include "packed_fwd.cuh"

namespace fa {
cudaError_t launch_packed_fwd_f16(const PackedFwdArgs &a, int hd, bool cap, int blocks, cudaStream_t stream) {
    return launch_fwd_type<false>(a, hd, cap, blocks, stream);
}
}  // namespace fa
