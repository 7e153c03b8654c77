// The tile kernels with an epilogue: the variants that a default plan names.
// Without K splits the kernel loads what a column block's outputs need and
// stores them; with splits the reduction does (split_reduce.hip), a thread
// for four adjacent outputs.
// 123 x 8190 x 8192 with a bias, GELU and an FP32 residual and output: 33.5 to
// 35 us (30 for the product, 5.6 to 6 for the reduction of four splits, whose
// partial sums are 17 MB each way); 16.5 GFLOP are 13.6 us at a library's
// rate, its 77 MB 15.1.
#include "tile_kernel.h"

namespace w8a16 {

hipError_t launch_tile(const EpilogueArgs &g, const w8a16_plan_t &p, hipStream_t stream)
{
    const uint32_t key = tile_variant_key(p.m_blocks, p.n_blocks, p.depth, p.a_depth);
    if (key == tile_variant_key(4, 8, 4, 4) && p.waves == 10)
        return launch_tile_t<64, 128, 4, 4, 2, true>(g, p, stream);
    if (p.waves != 8)
        return hipErrorInvalidValue;
    switch (key) {
    case tile_variant_key(4, 4, 4, 6): return launch_tile_t<64, 64, 4, 6, 2, false>(g, p, stream);
    case tile_variant_key(8, 8, 3, 2): return launch_tile_t<128, 128, 3, 2, 2, false>(g, p, stream);
    case tile_variant_key(8, 4, 4, 2): return launch_tile_t<128, 64, 4, 2, 2, false>(g, p, stream);
    case tile_variant_key(8, 8, 3, 3): return launch_tile_t<128, 128, 3, 3, 2, false>(g, p, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace w8a16
