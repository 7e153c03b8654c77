// The row kernels of plain attention.

#include "kv_rows_kernel.h"

namespace w8a16 {

template hipError_t launch_kv_rows(const AttnArgs &, const w8a16_kv_plan_t &, uint32_t, hipStream_t);
template hipError_t launch_kv_join(const AttnArgs &, const w8a16_kv_plan_t &, uint32_t, uint32_t, hipStream_t);

}  // namespace w8a16
