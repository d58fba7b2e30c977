// paged_attn.cu -- paged_attn.cuh as fa_paged_attn has it.
#include "paged_attn.cuh"

namespace fa {

size_t paged_attn_ws_bytes(int hd) {
    const size_t warps = static_cast<size_t>(device_sm_count()) * kMostWarps;
    const size_t rows = hd < 256 ? 16 : 8;  // of a unit
    return ws_head(device_sm_count(), 4) + ws_head(device_sm_count(), sizeof(Task)) +
           warps * 2 * rows * (2 + hd) * 4;
}

cudaError_t launch_paged_attn(const PagedAttnArgs &a, int dtype, int hd, cudaStream_t stream) {
    return launch_paged<false>(a, dtype, hd, stream);
}

}  // namespace fa
