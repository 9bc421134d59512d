// q4mm_norm_stream.cu -- the streaming norms (q4mm_norm_stream.cuh) over rows that
// start on 16 bytes, and the choice between them and the general kernels.
#include <algorithm>
#include <cuda_runtime.h>

#include "q4mm_norm_stream.cuh"

namespace q4 {

bool plan_norm_stream(int64_t m, int64_t d, int type, bool any, int matrices, int sm_count, NormStreamPlan *plan)
{
    const int size = type_size(type);
    any = any || d * size % 16 != 0;
    // of a row's place in shared memory; its vectors at most
    const int64_t bytes = any ? (d * size + 30 - size) / 16 * 16 : d * size, vecs = d * size / 16;
    // shorter rows go faster several to an SM in the general kernels (16384 x 1000
    // bf16: 39 us there, 46 here); with fewer rows than CTAs nothing is read ahead
    if (d * size < 2048 || vecs > 2048 || m <= 2 * sm_count) return false;
    NormStreamPlan p;
    const int most = size == 2 ? 2 : 4;   // vectors whose weights stay in registers
    p.NV = vecs <= 256 ? 1 : vecs <= 512 ? 2 : vecs <= 1024 ? most : 4;
    p.G = static_cast<int>(round_up(ceil_div(vecs, p.NV), 32));
    const size_t stage = static_cast<size_t>(matrices) * bytes + 16;
    // as many CTAs as the registers of their bound (224 threads' worth at 256, and
    // so on) leave room for, and three rows ahead
    int per_sm = p.G > 256 ? 1 : 576 / (p.G + 32);
    for (; per_sm > 0; --per_sm) {
        p.stages = static_cast<int>(std::min<size_t>(6, (kSmemPerSM / per_sm - 3 * 1024) / stage));
        if (p.stages >= 3) break;
    }
    if (per_sm == 0) return false;
    p.smem = stage * p.stages;
    if (p.smem > kSmemOptIn - 1024) return false;
    p.ctas = std::min<int64_t>(m, round_row_step(std::min<int64_t>(kNormPartials, static_cast<int64_t>(sm_count) * per_sm)));
    p.any = any;
    *plan = p;
    return true;
}

cudaError_t launch_norm_after_stream(const NormStreamPlan &p, const NormAfterArgs &a, int type, cudaStream_t s)
{
    return p.any ? launch_norm_after_stream_any(p, a, type, s) : launch_stream<AfterStream, false>(p, a, type, s);
}
cudaError_t launch_norm_before_bwd_stream(const NormStreamPlan &p, const NormBeforeBwdArgs &a, int type, cudaStream_t s)
{
    return p.any ? launch_norm_before_bwd_stream_any(p, a, type, s) : launch_stream<BeforeBwdStream, false>(p, a, type, s);
}
cudaError_t launch_norm_after_bwd_stream(const NormStreamPlan &p, const NormAfterBwdArgs &a, int type, cudaStream_t s)
{
    return p.any ? launch_norm_after_bwd_stream_any(p, a, type, s) : launch_stream<AfterBwdStream, false>(p, a, type, s);
}

} // namespace q4
