// The append kernels of tokens with positions of several axes.  They differ
// from the others by where a pair's cosine and sine come from: as many table
// rows as there are axes, and their positions loaded first, one more step in
// a chain of dependent loads.
// Bound like the others by HBM where they are large (6 prompts of up to 4099
// tokens, 32 query and 8 KV heads of 128 channels, 462 MB, 91.7 us, 5.0 TB/s),
// else by the call (64 sequences of one token 6.8 us, 5.0 on the GPU).

#include "kv_append_kernel.h"

namespace w8a16 {

hipError_t launch_kv_append_axes(const AppendAxesArgs &a, uint32_t dtype, hipStream_t stream)
{
    return append::launch_any(a, dtype, stream);
}

}  // namespace w8a16
