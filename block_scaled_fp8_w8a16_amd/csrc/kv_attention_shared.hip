// The row kernels of the two passes over a shared prefix.

#include "kv_rows_kernel.h"

namespace w8a16 {

template hipError_t launch_kv_rows(const PrefixArgs &, const w8a16_kv_plan_t &, uint32_t, hipStream_t);
template hipError_t launch_kv_rows(const SuffixArgs &, const w8a16_kv_plan_t &, uint32_t, hipStream_t);
template hipError_t launch_kv_join(const SuffixArgs &, const w8a16_kv_plan_t &, uint32_t, uint32_t, hipStream_t);

}  // namespace w8a16
