// q4mm_attn_bf16.cu -- the warp-MMA attention kernels of one kind of operands.
#include <algorithm>

#include "q4mm_attn_warp.cuh"

namespace q4 {

cudaError_t launch_attn_bf16(const AttnArgs &a, int sm_count, cudaStream_t s, int *ctas)
{
    return launch_kind<kBF16, 1>(a, sm_count, s, ctas);
}

} // namespace q4
