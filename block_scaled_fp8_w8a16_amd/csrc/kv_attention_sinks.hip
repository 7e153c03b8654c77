// The row kernels of windows with sinks: the tiles of the first tokens, as
// far as they lie before the window's, come in front of them in the same
// loop, so both parts have one maximum and one sum and there is nothing to
// join.  Kernels of their own, since the second condition on every masked key
// cost the others registers.
// Bound like the others: 32 decode steps of 32 query and 8 KV heads of 128
// channels, a window of 1024 keys and 4 sinks, 16.4 us, 4.15 TB/s of the 68 MB
// they cannot do without (75 are read); 12 drafts of 5 tokens, windows of 509
// keys and 67 sinks of 64 channels 7.4, the chain of first loads and the join
// of 8 waves.

#include "kv_rows_kernel.h"

namespace w8a16 {

template hipError_t launch_kv_rows(const SinkArgs &, const w8a16_kv_plan_t &, uint32_t, hipStream_t);
template hipError_t launch_kv_join(const SinkArgs &, const w8a16_kv_plan_t &, uint32_t, uint32_t, hipStream_t);

}  // namespace w8a16
