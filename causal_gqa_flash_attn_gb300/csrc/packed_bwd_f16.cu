// packed_bwd_f16.cu -- packed_bwd.cuh for binary16.
#include "packed_bwd.cuh"

namespace fa {
cudaError_t launch_packed_grad_f16(const PackedGradPair &p, const PackedGradArgs *v, int hd, bool cap, cudaStream_t stream) {
    return launch_grad_type<false>(p, v, hd, cap, stream);
}
}  // namespace fa
