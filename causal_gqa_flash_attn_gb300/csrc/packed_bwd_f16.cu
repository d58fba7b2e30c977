// packed_bwd_f16.cu -- packed_bwd.cuh for binary16.
#include "packed_bwd.cuh"

namespace fa {
cudaError_t launch_packed_grad_f16(const PackedGradArgs &a, int mode, int hd, bool cap, int blocks, cudaStream_t stream) {
    return launch_grad_type<false>(a, mode, hd, cap, blocks, stream);
}
}  // namespace fa
