// The append kernels of tokens with positions of several axes.

#include "kv_append_kernel.h"

namespace w8a16 {

hipError_t launch_kv_append_axes(const AppendAxesArgs &a, uint32_t dtype, hipStream_t stream)
{
    return append::launch_any(a, dtype, stream);
}

}  // namespace w8a16
