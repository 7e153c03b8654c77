// The tile kernels of the two passes over a shared prefix.

#include "kv_tile_kernel.h"

namespace w8a16 {

template hipError_t launch_kv_tile(const PrefixArgs &, uint32_t, hipStream_t);
template hipError_t launch_kv_tile(const SuffixArgs &, uint32_t, hipStream_t);

}  // namespace w8a16
