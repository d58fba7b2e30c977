// packed_bwd_bf16.cu -- packed_bwd.cuh for bfloat16.
#include "packed_bwd.cuh"

namespace fa {
cudaError_t launch_packed_grad_bf16(const PackedGradPair &p, const PackedGradArgs *v, int hd, bool cap, cudaStream_t stream) {
    return launch_grad_type<true>(p, v, hd, cap, stream);
}
}  // namespace fa
