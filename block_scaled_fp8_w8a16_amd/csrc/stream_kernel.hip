// The stream kernels of one GEMM and of the batched grid.

#include "stream_kernel.h"

namespace w8a16 {

hipError_t launch_stream(const GemmArgs &g, const w8a16_plan_t &p, hipStream_t stream)
{
    return stream::launch_stream_any(g, p, stream);
}

hipError_t launch_stream_batched(const BatchArgs &b, const w8a16_plan_t &p, hipStream_t stream)
{
    return stream::launch_stream_any(b, p, stream);
}

}  // namespace w8a16
