// q4mm_attn_i8x2.cu -- the warp-MMA attention kernels of one kind of operands.
#include <algorithm>

#include "q4mm_attn_warp.cuh"

namespace q4 {

cudaError_t launch_attn_i8x2(const AttnArgs &a, int sm_count, cudaStream_t s, int *ctas)
{
    return launch_kind<kI8, 2>(a, sm_count, s, ctas);
}

} // namespace q4
