// packed_bwd_bf16.cu -- packed_bwd.cuh for bfloat16.
#include "packed_bwd.cuh"

namespace fa {
cudaError_t launch_packed_grad_bf16(const PackedGradArgs &a, int mode, int hd, bool cap, int blocks, cudaStream_t stream) {
    return launch_grad_type<true>(a, mode, hd, cap, blocks, stream);
}
}  // namespace fa
