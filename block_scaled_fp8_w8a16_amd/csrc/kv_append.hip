// Appending keys and values to the paged FP8 cache, with the rotation of
// keys (and queries) on the way.
//
// One wave owns one block of 16 slots of one KV head, keys or values, so
// that the block's scale needs no atomics: its lanes hold the new tokens'
// elements in registers (8 consecutive elements of a token each), rotate
// them, reduce the largest magnitude over the wave, and quantise.  Scales
// are powers of two (E8M0), so quantising is one exact multiplication and
// one rounding, and a block whose scale grows keeps its older codes exactly
// unless they fall into E4M3's subnormals.
//
// Values are stored with a block's 16 tokens adjacent for each channel: the
// attention's P V product then takes 16 keys of a channel in one 16-byte
// load.  A wave transposes through LDS and merges the new bytes into the
// 16-byte rows that hold them.
//
// The queries' rotation runs in further workgroups of the same launch: for
// a decode step all of it is launch latency, and one launch does.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention.h"
#include "device_common.h"
#include "rope_device.h"

namespace w8a16 {

namespace {

using namespace dev;

constexpr uint32_t kBlock = W8A16_KV_BLOCK;

__device__ __forceinline__ float power_of_two(int32_t field)   // 2^(field - 127), field 1..254
{
    return __builtin_bit_cast(float, (uint32_t)field << 23);
}

// Smallest byte b >= 1 with amax <= 448 * 2^(b - 127).  448 = 1.75 * 2^8, so
// b is the exponent field less 8, plus one if the mantissa exceeds 0.75.
__device__ __forceinline__ int32_t scale_byte(float amax)
{
    const int32_t b = (int32_t)((__builtin_bit_cast(uint32_t, amax) + 0x1fffffu) >> 23) - 8;
    return b < 1 ? 1 : b;
}

// Saturates to +-448 (infinities too) and keeps NaN, which the hardware
// conversion stores as NaN.
__device__ __forceinline__ float saturate(float x)
{
    x = x > 448.0f ? 448.0f : x;
    return x < -448.0f ? -448.0f : x;
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d)
{
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(saturate(a), saturate(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(saturate(c), saturate(d), v, true);
}

// Four codes of an older scale stored for one 2^-n times as fine.
__device__ __forceinline__ uint32_t rescale4(uint32_t raw, float f)
{
    auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)raw, false);
    auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)raw, true);
    return codes4(lo[0] * f, lo[1] * f, hi[0] * f, hi[1] * f);
}

// Elements 8c .. 8c+7 of a key row, rotated by cs (null: not rotated), in
// loads of W elements that lie whole on one side of rot and of rot / 2.
template <class T, int W>
__device__ __forceinline__ void load_pieces(const AppendArgs &a, const T *x, uint32_t c, const float *cs,
                                            float *out)
{
    typedef typename Vec<T, W>::type V;
    const uint32_t rot = cs ? a.q.rot : 0u, h = rot / 2;
#pragma unroll
    for (int p = 0; p < 8; p += W) {
        const uint32_t e = 8 * c + p;
        const V v = *reinterpret_cast<const V *>(x + e);
#pragma unroll
        for (int i = 0; i < W; ++i)
            out[p + i] = to_f32(v[i]);
        if (e >= rot)
            continue;
        if (a.q.half) {
            const bool upper = e >= h;
            const uint32_t i0 = upper ? e - h : e;
            const V w = *reinterpret_cast<const V *>(x + (upper ? i0 : e + h));
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float own = out[p + i], other = to_f32(w[i]);
                float y0, y1;
                rotate(upper ? other : own, upper ? own : other, cs[2 * (i0 + i)], cs[2 * (i0 + i) + 1], y0, y1);
                out[p + i] = upper ? y1 : y0;
            }
        } else if (W > 1) {
#pragma unroll
            for (int i = 0; i + 1 < W; i += 2)
                rotate(out[p + i], out[p + i + 1], cs[e + i], cs[e + i + 1], out[p + i], out[p + i + 1]);
        } else {
            const bool second = (e & 1u) != 0;
            const float own = out[p], other = to_f32(x[e ^ 1u]);
            float y0, y1;
            rotate(second ? other : own, second ? own : other, cs[e & ~1u], cs[e | 1u], y0, y1);
            out[p] = second ? y1 : y0;
        }
    }
}

template <class T>
__device__ __forceinline__ void load_chunk(const AppendArgs &a, const T *x, uint32_t c, const float *cs,
                                           float *out)
{
    if (a.vec == 8)
        load_pieces<T, 8>(a, x, c, cs, out);
    else if (a.vec == 4)
        load_pieces<T, 4>(a, x, c, cs, out);
    else
        load_pieces<T, 1>(a, x, c, cs, out);
}

// NV: 8-element chunks of a block per lane (16 * dim / 8 / 64, rounded up).
template <class T, int NV>
__device__ __forceinline__ void append_block(const AppendArgs &a, uint32_t unit, uint8_t *lds)
{
    const uint32_t lane = threadIdx.x & 63u;
    const KvPool &pool = a.pool;
    const KvSeqs &sq = a.seqs;
    const uint32_t b = a.by_seq_units.div(unit);
    uint32_t rest = unit - b * a.by_seq_units.d;
    const uint32_t nth = a.by_units.div(rest);
    rest -= nth * a.by_units.d;
    const uint32_t head = rest >> 1;
    const bool is_v = (rest & 1u) != 0;
    if (b >= sq.seqs)
        return;
    // the sequence's new tokens: first .. first + n - 1, at start ..
    uint32_t first = b * sq.uniform, end = first + sq.uniform;
    if (sq.cu) {
        first = (uint32_t)sq.cu[b];
        end = (uint32_t)sq.cu[b + 1];
        if (first > sq.tokens || end > sq.tokens || end < first)
            return;
    }
    const int32_t len = sq.kv_lens[b];
    int32_t start = len - (int32_t)(end - first);
    if (start < 0) {
        first += (uint32_t)(-start);
        start = 0;
    }
    const int32_t blk = (int32_t)(start / (int32_t)kBlock + (int32_t)nth);
    const int32_t p0 = blk * (int32_t)kBlock;
    if (p0 >= len || first >= end)
        return;
    const uint32_t col = pool.by_blocks.div((uint32_t)blk);
    const uint32_t within = (uint32_t)blk - col * pool.blocks;
    if (col >= sq.bt_width)
        return;
    const uint32_t page = (uint32_t)sq.block_table[(size_t)b * sq.bt_stride + col];
    if (page >= pool.pages)
        return;
    // slots lo .. hi-1 are new, slots below lo hold older tokens
    const uint32_t lo = start > p0 ? (uint32_t)(start - p0) : 0u;
    const uint32_t hi = len - p0 < (int32_t)kBlock ? (uint32_t)(len - p0) : kBlock;
    const uint32_t dim = pool.dim, chunks = dim / 8;
    const uint32_t slot0 = head * pool.blocks + within;   // block inside the page

    float x[NV][8];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const uint32_t id = lane + 64u * i, t = id / chunks, c = id - t * chunks;
        if (t < lo || t >= hi) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[i][j] = 0.f;
            continue;
        }
        const uint32_t tok = first + (uint32_t)(p0 + (int32_t)t - start);
        if (is_v) {
            load_chunk<T>(a, reinterpret_cast<const T *>(a.v) + (int64_t)tok * a.v_token +
                          (int64_t)head * a.v_head, c, nullptr, x[i]);
        } else {
            const uint32_t pos = (uint32_t)p0 + t;
            const float *cs = a.q.table ? a.q.table + (size_t)pos * a.q.rot : nullptr;
            if (cs && pos >= a.q.table_positions) {
                // no angle for this position: NaN, as the rotation gives
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[i][j] = __builtin_nanf("");
                if (8 * c >= a.q.rot)
                    cs = nullptr;
            }
            if (!cs || pos < a.q.table_positions)
                load_chunk<T>(a, reinterpret_cast<const T *>(a.k) + (int64_t)tok * a.k_token +
                              (int64_t)head * a.k_head, c, cs, x[i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float m = fabsf(x[i][j]);
            amax = m < __builtin_inff() ? fmaxf(amax, m) : amax;
        }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        amax = fmaxf(amax, __shfl_xor(amax, off, 64));
    uint8_t *scale = is_v ? pool.v_scale + page * pool.vs_page + slot0
                          : pool.k_scale + page * pool.ks_page + slot0;
    int32_t byte = scale_byte(amax), old = byte;
    if (lo > 0) {
        old = *scale;
        byte = byte > old ? byte : old;
    }
    // 2^(127 - byte); byte <= 247 for amax below 2^128, and 254 at the most
    // from an older block
    const float inv = power_of_two(254 - byte < 1 ? 1 : 254 - byte);
    const int32_t drop = byte - old;
    const float shrink = drop > 126 ? 0.f : power_of_two(127 - drop);

    if (!is_v) {
        uint8_t *row0 = pool.k + page * pool.k_page + (size_t)slot0 * kBlock * dim;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t id = lane + 64u * i, t = id / chunks, c = id - t * chunks;
            u32x2_t *dst = reinterpret_cast<u32x2_t *>(row0 + t * dim + 8 * c);
            u32x2_t v;
            if (t >= lo && t < hi) {
                v.x = codes4(x[i][0] * inv, x[i][1] * inv, x[i][2] * inv, x[i][3] * inv);
                v.y = codes4(x[i][4] * inv, x[i][5] * inv, x[i][6] * inv, x[i][7] * inv);
                *dst = v;
            } else if (t < lo && drop > 0) {
                v = *dst;
                v.x = rescale4(v.x, shrink);
                v.y = rescale4(v.y, shrink);
                *dst = v;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t id = lane + 64u * i, t = id / chunks, c = id - t * chunks;
            if (t < lo || t >= hi)
                continue;
            const uint32_t w0 = codes4(x[i][0] * inv, x[i][1] * inv, x[i][2] * inv, x[i][3] * inv);
            const uint32_t w1 = codes4(x[i][4] * inv, x[i][5] * inv, x[i][6] * inv, x[i][7] * inv);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                lds[(8 * c + j) * kBlock + t] = (uint8_t)((j < 4 ? w0 : w1) >> (8 * (j & 3)));
        }
        // the wave's own LDS bytes: complete before they are read back
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_wave_barrier();
        uint8_t *blk0 = pool.v + page * pool.v_page + (size_t)slot0 * kBlock * dim;
        const bool whole = lo == 0 && hi == kBlock;
        for (uint32_t d = lane; d < dim; d += 64u) {
            u32x4_t *dst = reinterpret_cast<u32x4_t *>(blk0 + d * kBlock);
            u32x4_t v = *reinterpret_cast<const u32x4_t *>(lds + d * kBlock);
            if (!whole) {
                const u32x4_t have = *dst;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t is_new = 0, is_old = 0;
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) {
                        const uint32_t t = 4u * w + j;
                        is_new |= t >= lo && t < hi ? 0xffu << (8 * j) : 0u;
                        is_old |= t < lo ? 0xffu << (8 * j) : 0u;
                    }
                    const uint32_t kept = drop > 0 ? rescale4(have[w], shrink) : have[w];
                    v[w] = (v[w] & is_new) | (kept & is_old) | (have[w] & ~(is_new | is_old));
                }
            }
            *dst = v;
        }
    }
    if (lane == 0)
        *scale = (uint8_t)byte;
}

template <class T, int P, int N>
__device__ __forceinline__ void rotate_queries(const AppendArgs &a, uint32_t t, uint32_t part)
{
    const uint32_t idx = part * 256u + threadIdx.x;
    const uint32_t hg = a.q.by_items.div(idx), h = hg * N, item = idx - hg * a.q.items;
    if (h >= a.q.heads)
        return;
    uint32_t b;
    int32_t pos = 0;
    const bool owned = token_place(a.seqs, t, b, pos);
    const T *x = reinterpret_cast<const T *>(a.q.x) + (int64_t)t * a.q.x_token;
    T *y = reinterpret_cast<T *>(a.q.y) + (int64_t)t * a.q.y_token;
    if (owned) {
        const float *cs = (uint32_t)pos < a.q.table_positions ? a.q.table + (size_t)pos * a.q.rot : nullptr;
        if (a.q.half)
            rope_heads<T, P, N, true>(a.q, x, y, h, item, cs, false);
        else
            rope_heads<T, P, N, false>(a.q, x, y, h, item, cs, false);
        return;
    }
    const bool pair = item < a.q.pair_items;
    const uint32_t e0 = pair ? (a.q.half ? item * P : 2 * item * P)
                             : a.q.rot + (item - a.q.pair_items) * 2 * P;
    const uint32_t e1 = pair && a.q.half ? e0 + a.q.rot / 2 : e0 + P;
    for (uint32_t n = 0; n < N && h + n < a.q.heads; ++n)
        for (uint32_t i = 0; i < P; ++i) {
            T *row = y + (int64_t)(h + n) * a.q.y_head;
            row[e0 + i] = static_cast<T>(0.f);
            if (e1 + i < a.q.dim)
                row[e1 + i] = static_cast<T>(0.f);
        }
}

template <class T, int N>
__device__ __forceinline__ void rotate_queries_by(const AppendArgs &a, uint32_t t, uint32_t part)
{
    switch (a.q.pairs) {
    case 8: rotate_queries<T, 8, N>(a, t, part); break;
    case 4: rotate_queries<T, 4, N>(a, t, part); break;
    default: rotate_queries<T, 1, N>(a, t, part); break;
    }
}

template <class T, int NV>
__global__ __launch_bounds__(256) void w8a16_kv_append_kernel(AppendArgs a)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[4][NV * 32 * kBlock];
    if (blockIdx.x < a.kv_groups) {
        const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        append_block<T, NV>(a, blockIdx.x * 4u + wave, lds[wave]);
        return;
    }
    const uint32_t g = blockIdx.x - a.kv_groups;
    const uint32_t t = a.by_q_groups.div(g), part = g - t * a.q_groups;
    if (a.q_heads_per_thread == 1)
        rotate_queries_by<T, 1>(a, t, part);
    else
        rotate_queries_by<T, kRopeHeads>(a, t, part);
}

template <class T>
hipError_t launch_type(const AppendArgs &a, hipStream_t stream)
{
    const uint32_t tokens = a.q.x ? a.seqs.tokens : 0u;
    const dim3 grid(a.kv_groups + tokens * a.q_groups), block(256);
    switch ((a.pool.dim + 63u) / 64u) {
    case 1: hipLaunchKernelGGL((w8a16_kv_append_kernel<T, 2>), grid, block, 0, stream, a); break;
    case 2: hipLaunchKernelGGL((w8a16_kv_append_kernel<T, 4>), grid, block, 0, stream, a); break;
    case 3: hipLaunchKernelGGL((w8a16_kv_append_kernel<T, 6>), grid, block, 0, stream, a); break;
    default: hipLaunchKernelGGL((w8a16_kv_append_kernel<T, 8>), grid, block, 0, stream, a); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, uint32_t dtype, hipStream_t stream)
{
    switch (dtype) {
    case W8A16_BF16: return launch_type<__bf16>(a, stream);
    case W8A16_FP16: return launch_type<_Float16>(a, stream);
    default: return launch_type<float>(a, stream);
    }
}

}  // namespace w8a16
