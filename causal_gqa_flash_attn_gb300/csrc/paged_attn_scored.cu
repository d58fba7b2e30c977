// paged_attn_scored.cu -- paged_attn.cuh with capped scores and a bias by distance.
#include "paged_attn.cuh"

namespace fa {

cudaError_t launch_paged_attn_scored(const PagedAttnArgs &a, int dtype, int hd, cudaStream_t stream) {
    return launch_paged<true>(a, dtype, hd, stream);
}

}  // namespace fa
