// q4mm_norm_stream_any.cu -- the streaming norms (q4mm_norm_stream.cuh) over rows
// that start anywhere: a unit of its own because it takes as long to compile as the
// aligned ones.
#include <cuda_runtime.h>

#include "q4mm_norm_stream.cuh"

namespace q4 {

cudaError_t launch_norm_after_stream_any(const NormStreamPlan &p, const NormAfterArgs &a, int type, cudaStream_t s)
{
    return launch_stream<AfterStream, true>(p, a, type, s);
}
cudaError_t launch_norm_before_bwd_stream_any(const NormStreamPlan &p, const NormBeforeBwdArgs &a, int type, cudaStream_t s)
{
    return launch_stream<BeforeBwdStream, true>(p, a, type, s);
}
cudaError_t launch_norm_after_bwd_stream_any(const NormStreamPlan &p, const NormAfterBwdArgs &a, int type, cudaStream_t s)
{
    return launch_stream<AfterBwdStream, true>(p, a, type, s);
}

} // namespace q4
