// Rotary positions: the table of cosines and sines, and the rotation.
//
// The rotation reads and writes each element once and is bound by HBM.  A
// thread owns P pairs of one or of four heads: P = 8 (two 16-byte loads and
// stores of 16-bit elements) where rows and halves are aligned to it, else 4
// or 1 (16384 tokens of 32 heads of 128 BF16 channels: 51, 57 and 64 us).
// Four heads share the cosines and sines (4 bytes per rotated element, more
// than the element itself, if each head reads them from the caches) and have
// their loads in flight together: 16381 tokens of 32 heads out of wider rows
// 75 -> 47 us, 2048 tokens 12.9 -> 8.8, 512 tokens 4.6 -> 3.7.  With fewer
// than 512 such threads per CU one head each keeps the chip busier: 64 tokens
// are one launch's latency, 2.6 us, either way.
// Measured: 277 MB in 47 to 54 us, 5.1 to 5.9 TB/s with part of the rows in
// the last-level cache, where a large copy moves 4.9.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention.h"
#include "rope_device.h"

namespace w8a16 {

namespace {

using namespace dev;

// One thread per (position, pair), in FP64: position * f_i reaches 10^5 to
// 10^6 radians, where an FP32 angle would be off by up to 0.06.
__global__ __launch_bounds__(256) void w8a16_rope_table_kernel(w8a16_rope_config_t c, float *table,
                                                               uint64_t total, uint32_t pairs)
{
    const uint64_t idx = (uint64_t)blockIdx.x * 256u + threadIdx.x;
    if (idx >= total)
        return;
    const uint32_t i = (uint32_t)(idx % pairs);
    const double p = (double)(idx / pairs), r = 2.0 * pairs;
    double base = c.base;
    if (c.scaling == W8A16_ROPE_BASE)
        base *= pow(c.factor, r / (r - 2.0));
    double f = pow(base, -2.0 * i / r);
    if (c.scaling == W8A16_ROPE_LINEAR) {
        f /= c.factor;
    } else if (c.scaling == W8A16_ROPE_BANDS) {
        const double turns = c.original * f / 6.283185307179586476925287;
        double w = (turns - c.low_turns) / (c.high_turns - c.low_turns);
        w = w < 0.0 ? 0.0 : (w > 1.0 ? 1.0 : w);
        f *= w + (1.0 - w) / c.factor;
    }
    double sn, cs;
    sincos(p * f, &sn, &cs);
    float2 v;
    v.x = (float)(c.magnitude * cs);
    v.y = (float)(c.magnitude * sn);
    reinterpret_cast<float2 *>(table)[idx] = v;
}

template <class T, int P, int N, bool HALF>
__global__ __launch_bounds__(256) void w8a16_rope_kernel(RopeArgs a)
{
    const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
    if (idx >= a.total)
        return;
    const uint32_t t = a.by_row.div(idx), rest = idx - t * a.by_row.d;
    const uint32_t hg = a.r.by_items.div(rest), item = rest - hg * a.r.items;
    const uint32_t pos = (uint32_t)a.positions[t];
    const float *cs = pos < a.r.table_positions ? a.r.table + (size_t)pos * a.r.rot : nullptr;
    rope_heads<T, P, N, HALF>(a.r, reinterpret_cast<const T *>(a.r.x) + (int64_t)t * a.r.x_token,
                        reinterpret_cast<T *>(a.r.y) + (int64_t)t * a.r.y_token, hg * N, item, cs,
                        a.inverse != 0);
}

template <class T, int N, bool HALF>
hipError_t launch_heads(const RopeArgs &a, hipStream_t stream)
{
    const dim3 grid((a.total + 255u) / 256u), block(256);
    switch (a.r.pairs) {
    case 8: hipLaunchKernelGGL((w8a16_rope_kernel<T, 8, N, HALF>), grid, block, 0, stream, a); break;
    case 4: hipLaunchKernelGGL((w8a16_rope_kernel<T, 4, N, HALF>), grid, block, 0, stream, a); break;
    default: hipLaunchKernelGGL((w8a16_rope_kernel<T, 1, N, HALF>), grid, block, 0, stream, a); break;
    }
    return hipGetLastError();
}

template <class T>
hipError_t launch_type(const RopeArgs &a, hipStream_t stream)
{
    if (a.heads_per_thread == 1)
        return a.r.half ? launch_heads<T, 1, true>(a, stream) : launch_heads<T, 1, false>(a, stream);
    return a.r.half ? launch_heads<T, kRopeHeads, true>(a, stream)
                    : launch_heads<T, kRopeHeads, false>(a, stream);
}

}  // namespace

hipError_t launch_rope_table(const w8a16_rope_config_t &c, float *table, uint32_t positions,
                             uint32_t rot_dim, hipStream_t stream)
{
    const uint64_t total = (uint64_t)positions * (rot_dim / 2);
    hipLaunchKernelGGL(w8a16_rope_table_kernel, dim3((uint32_t)((total + 255u) / 256u)), dim3(256),
                       0, stream, c, table, total, rot_dim / 2);
    return hipGetLastError();
}

hipError_t launch_rope(const RopeArgs &a, uint32_t dtype, hipStream_t stream)
{
    switch (dtype) {
    case W8A16_BF16: return launch_type<__bf16>(a, stream);
    case W8A16_FP16: return launch_type<_Float16>(a, stream);
    default: return launch_type<float>(a, stream);
    }
}

}  // namespace w8a16
