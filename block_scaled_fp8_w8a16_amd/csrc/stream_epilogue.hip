// The stream kernels with an epilogue.

#include "stream_kernel.h"

namespace w8a16 {

hipError_t launch_stream(const EpilogueArgs &g, const w8a16_plan_t &p, hipStream_t stream)
{
    return stream::launch_stream_any(g, p, stream);
}

}  // namespace w8a16
