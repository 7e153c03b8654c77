// The stream kernels with an epilogue: a sum meets its bias, gate and
// residual in the registers it is stored from, so that no output is rounded
// or moved in between.  They are loaded before the waves' partial sums are
// joined, under the last of the weight's reads.
// Bound like the plain ones by reading the weight: 8 x 4096 x 4096 with a
// residual 5.6 us (17.0 MB, 3.0 TB/s; the plain product and an addition in
// torch 79 with its casts), 16 x 12288 x 5120 with SiLU and a gate 13.9 us (63.9
// MB, 4.6 TB/s).

#include "stream_kernel.h"

namespace w8a16 {

hipError_t launch_stream(const EpilogueArgs &g, const w8a16_plan_t &p, hipStream_t stream)
{
    return stream::launch_stream_any(g, p, stream);
}

}  // namespace w8a16
