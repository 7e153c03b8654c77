// The tile kernels of windows with sinks (figures in kv_tile_kernel.h).

#include "kv_tile_kernel.h"

namespace w8a16 {

template hipError_t launch_kv_tile(const SinkArgs &, uint32_t, hipStream_t);

}  // namespace w8a16
