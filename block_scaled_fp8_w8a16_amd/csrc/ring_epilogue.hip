// The ring kernels with an epilogue (as in stream_epilogue.hip).

#include "ring_kernel.h"

namespace w8a16 {

hipError_t launch_ring(const EpilogueArgs &g, const w8a16_plan_t &p, hipStream_t stream)
{
    return ring::launch_any(g, p, stream);
}

}  // namespace w8a16
