// Appending keys and values to the paged FP8 cache, with the rotation of
// keys (and queries) on the way.
//
// One wave owns one block of 16 slots of one KV head, keys or values, so
// that the block's scale needs no atomics: its lanes hold the new tokens'
// elements in registers (all loads in flight at once), rotate them, reduce
// the largest magnitude over the wave, and quantise.  Scales are powers of
// two (E8M0), so quantising is one exact multiplication and one rounding,
// and a block whose scale grows keeps its older codes exactly unless they
// fall into E4M3's subnormals.  Keys lie in lanes as pairs, as in the
// rotation.
//
// Values are stored with a block's 16 tokens adjacent for each channel: the
// attention's P V product then takes 16 keys of a channel in one 16-byte
// load.  A wave transposes through LDS, where a lane's four tokens of a
// channel make one word, and merges the new bytes into the 16-byte rows that
// hold them.
//
// The queries' rotation runs in further workgroups of the same launch: for
// a decode step all of it is launch latency, and one launch does.
//
// HBM bounds long appends: 6 prompts of up to 4099 tokens with 32 query and
// 8 KV heads of 128 channels, about 460 MB, take 89 us, 5.2 TB/s (a large
// copy moves 4.9).  A decode step of 256 sequences takes 7.5 us of the GPU,
// of 4 sequences 4.4: the chain of loads from the lengths through the page
// to the tokens and the block.  The block's byte and rows are asked for with
// the tokens, not after the largest magnitude is known (from cold caches 4
// sequences 8.5 -> 7.7 us, 48 sequences of up to 7 tokens 10.6 -> 9.8).

#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attention.h"
#include "device_common.h"
#include "rope_device.h"

namespace w8a16 {

namespace append {

using namespace dev;

// Whether a call brings positions of several axes (AppendAxesArgs) rather
// than the sequences' own (AppendArgs).
template <class Args> constexpr bool has_axes = std::is_same<Args, AppendAxesArgs>::value;

constexpr uint32_t kBlock = W8A16_KV_BLOCK;
// LDS bytes of 8 channels x 16 tokens, padded so that lanes writing the same
// token's byte of different chunks use different banks.
constexpr uint32_t kChunkPitch = 8 * kBlock + 16;

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

// Codes of four values within +-448, or NaN.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d)
{
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

// Four codes of an older scale stored for one 2^-n times as fine.
__device__ __forceinline__ uint32_t rescale4(uint32_t raw, float f)
{
    auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)raw, false);
    auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)raw, true);
    return codes4(lo[0] * f, lo[1] * f, hi[0] * f, hi[1] * f);
}

// The block a wave works on: slots lo .. hi-1 are new, slots below lo hold
// older tokens; the token of slot lo is `first` of the token axis, at
// position pos0 + lo.
struct BlockAt {
    uint32_t lo, hi, first, pos0, head, slot, page;
};

// The wave's largest finite |x| of N values per lane.
template <int N> __device__ __forceinline__ float wave_amax(const float (&x)[N])
{
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        amax = fmaxf(amax, fabsf(x[i]));
    if (__ballot(!(amax < __builtin_inff()))) {
        // infinities (and NaN that the maximum has not skipped) leave the
        // scale to the finite elements
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float m = fabsf(x[i]);
            amax = m < __builtin_inff() ? fmaxf(amax, m) : amax;
        }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        amax = fmaxf(amax, __shfl_xor(amax, off, 64));
    return amax;
}

// A block's new scale byte, what its new elements are multiplied by, and
// how far the byte grew.
struct BlockScale {
    int32_t byte, drop;
    float inv, shrink;
    __device__ __forceinline__ BlockScale(float amax, uint32_t lo, int32_t held)
    {
        byte = scale_byte(amax);
        int32_t old = byte;
        if (lo > 0) {
            old = held;
            byte = byte > old ? byte : old;
        }
        // byte <= 247 for amax below 2^128, and 255 at the most if held
        inv = power_of_two(254 - byte < 1 ? 1 : 254 - byte);
        drop = byte - old;
        shrink = drop > 126 ? 0.f : power_of_two(127 - drop);
    }
    // |x| * inv <= 448 unless x is infinite
    __device__ __forceinline__ float operator()(float x) const
    {
        return fabsf(x) == __builtin_inff() ? __builtin_copysignf(448.0f, x) : x * inv;
    }
};

// N codes (1, 4 or 8) at dst, which is aligned to them.
template <int N> __device__ __forceinline__ void store_codes(uint8_t *dst, const float *y)
{
    if constexpr (N == 1) {
        *dst = (uint8_t)codes4(y[0], 0.f, 0.f, 0.f);
    } else if constexpr (N == 4) {
        *reinterpret_cast<uint32_t *>(dst) = codes4(y[0], y[1], y[2], y[3]);
    } else {
        *reinterpret_cast<u32x2_t *>(dst) =
            u32x2_t{codes4(y[0], y[1], y[2], y[3]), codes4(y[4], y[5], y[6], y[7])};
    }
}

// Keys.  A lane's items are P pairs of one token (two pieces of P elements,
// as in the rotation), or 2P elements past rot; NI items per lane.
template <class T, int P, int NI, bool HALF, class Args>
__device__ __forceinline__ void append_keys(const Args &a, const BlockAt &at)
{
    typedef typename Vec<T, P>::type V;
    const uint32_t lane = threadIdx.x & 63u, rot = a.q.table ? a.q.rot : 0u, dim = a.pool.dim;
    const uint32_t pair_items = rot / 2 / P;
    V va[NI], vb[NI];
    float2 cs[NI][P];
    uint32_t tok[NI], e0[NI], e1[NI];
    bool on[NI], pair[NI];
#pragma unroll
    for (int n = 0; n < NI; ++n) {
        const uint32_t id = lane + 64u * n, t = a.by_k_items.div(id), item = id - t * a.by_k_items.d;
        tok[n] = t;
        on[n] = t >= at.lo && t < at.hi;
        pair[n] = item < pair_items;
        const uint32_t q = item - pair_items;
        e0[n] = pair[n] ? (HALF ? item * P : item * 2 * P) : rot + q * 2 * P;
        e1[n] = pair[n] && HALF ? e0[n] + rot / 2 : e0[n] + P;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            va[n][i] = static_cast<T>(0.f);
            vb[n][i] = static_cast<T>(0.f);
            cs[n][i] = float2{1.f, 0.f};
        }
        if (on[n]) {
            const T *x = reinterpret_cast<const T *>(a.k) + (int64_t)(at.first + t - at.lo) * a.k_token +
                         (int64_t)at.head * a.k_head;
            va[n] = *reinterpret_cast<const V *>(x + e0[n]);
            vb[n] = *reinterpret_cast<const V *>(x + e1[n]);
            const uint32_t pos = at.pos0 + t;
            if constexpr (has_axes<Args>) {
                if (pair[n]) {
                    float c[P], s[P];
                    AxesAngles(a.axes, a.q.table, a.q.table_positions, at.first + t - at.lo).load(item * P, c, s);
#pragma unroll
                    for (int i = 0; i < P; ++i)
                        cs[n][i] = float2{c[i], s[i]};
                }
            } else if (pair[n] && pos < a.q.table_positions) {
                const float2 *row = reinterpret_cast<const float2 *>(a.q.table) +
                                    (size_t)pos * (rot / 2) + item * P;
#pragma unroll
                for (int i = 0; i < P; ++i)
                    cs[n][i] = row[i];
            }
        }
    }
    // (under way with the tokens; a page that does not exist is page 0 here)
    const bool there = at.page < a.pool.pages;
    uint8_t *scale = a.pool.k_scale + (there ? at.page : 0u) * a.pool.ks_page + at.slot;
    const int32_t held = at.lo > 0 ? (int32_t)*scale : 0;
    float x[NI * 2 * P];
#pragma unroll
    for (int n = 0; n < NI; ++n) {
        float u[2 * P], *y = x + n * 2 * P;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            u[i] = to_f32(va[n][i]);
            u[P + i] = to_f32(vb[n][i]);
        }
        // no angle for the position: NaN, as the rotation gives
        const bool lost = !has_axes<Args> && on[n] && pair[n] && at.pos0 + tok[n] >= a.q.table_positions;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            constexpr bool apart = HALF || P == 1;
            const int i0 = apart ? i : 2 * i, i1 = apart ? P + i : 2 * i + 1;
            float y0, y1;
            rotate(u[i0], u[i1], cs[n][i].x, cs[n][i].y, y0, y1);
            y[i0] = lost ? __builtin_nanf("") : (pair[n] ? y0 : u[i0]);
            y[i1] = lost ? __builtin_nanf("") : (pair[n] ? y1 : u[i1]);
        }
    }
    const float amax = wave_amax(x);
    if (!there)
        return;
    const BlockScale sc(amax, at.lo, held);
    uint8_t *row0 = a.pool.k + at.page * a.pool.k_page + (size_t)at.slot * kBlock * dim;
#pragma unroll
    for (int n = 0; n < NI; ++n) {
        if (!on[n])
            continue;
        float y[2 * P];
#pragma unroll
        for (int i = 0; i < 2 * P; ++i)
            y[i] = sc(x[n * 2 * P + i]);
        store_codes<P>(row0 + tok[n] * dim + e0[n], y);
        store_codes<P>(row0 + tok[n] * dim + e1[n], y + P);
    }
    if (sc.drop > 0)     // the older rows, of the new scale
        for (uint32_t i = lane; i < at.lo * dim / 4; i += 64u) {
            uint32_t *w = reinterpret_cast<uint32_t *>(row0) + i;
            *w = rescale4(*w, sc.shrink);
        }
    if (lane == 0)
        *scale = (uint8_t)sc.byte;
}

// Values.  A lane's items are four consecutive tokens of one 8-element
// chunk, so that four tokens' codes of a channel make one LDS word of the
// transposition.  NP: items per lane; loads of W elements.
template <class T, int W, int NP>
__device__ __forceinline__ void append_values(const AppendArgs &a, const BlockAt &at, uint8_t *lds)
{
    typedef typename Vec<T, W>::type V;
    const uint32_t lane = threadIdx.x & 63u, dim = a.pool.dim;
    V raw[NP][4][8 / W];
    uint32_t tg[NP], c[NP];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const uint32_t id = lane + 64u * n;
        tg[n] = a.by_chunks.div(id);
        c[n] = id - tg[n] * a.by_chunks.d;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t t = 4u * tg[n] + i;
#pragma unroll
            for (int p = 0; p < 8 / W; ++p)
#pragma unroll
                for (int k = 0; k < W; ++k)
                    raw[n][i][p][k] = static_cast<T>(0.f);
            if (t >= at.lo && t < at.hi) {
                const T *x = reinterpret_cast<const T *>(a.v) + (int64_t)(at.first + t - at.lo) * a.v_token +
                             (int64_t)at.head * a.v_head + 8 * c[n];
#pragma unroll
                for (int p = 0; p < 8 / W; ++p)
                    raw[n][i][p] = *reinterpret_cast<const V *>(x + p * W);
            }
        }
    }
    // The block's byte and rows, under way with the tokens (a page that does
    // not exist is page 0 here).
    const bool whole = at.lo == 0 && at.hi == kBlock, there = at.page < a.pool.pages;
    const uint32_t page = there ? at.page : 0u;
    uint8_t *scale = a.pool.v_scale + page * a.pool.vs_page + at.slot;
    uint8_t *blk0 = a.pool.v + page * a.pool.v_page + (size_t)at.slot * kBlock * dim;
    const int32_t held = at.lo > 0 ? (int32_t)*scale : 0;
    u32x4_t have[2 * NP];
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) {
        have[i] = u32x4_t{0u, 0u, 0u, 0u};
        if (!whole && lane + 64u * i < dim)
            have[i] = *reinterpret_cast<const u32x4_t *>(blk0 + (lane + 64u * i) * kBlock);
    }
    float x[NP * 32];       // [item][token][element]
#pragma unroll
    for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[n * 32 + i * 8 + j] = to_f32(raw[n][i][j / W][j % W]);
    const float amax = wave_amax(x);
    if (!there)
        return;
    const BlockScale sc(amax, at.lo, held);
#pragma unroll
    for (int n = 0; n < NP; ++n)
        if (tg[n] < 4u) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint32_t *>(lds + c[n] * kChunkPitch + j * kBlock + 4u * tg[n]) =
                    codes4(sc(x[n * 32 + j]), sc(x[n * 32 + 8 + j]), sc(x[n * 32 + 16 + j]),
                           sc(x[n * 32 + 24 + j]));
        }
    // the wave's own LDS words: complete before they are read back
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) {
        const uint32_t d = lane + 64u * i;
        if (d >= dim)
            continue;
        u32x4_t *dst = reinterpret_cast<u32x4_t *>(blk0 + d * kBlock);
        u32x4_t v = *reinterpret_cast<const u32x4_t *>(lds + (d >> 3) * kChunkPitch + (d & 7u) * kBlock);
        if (!whole) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t is_new = 0, is_old = 0;
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) {
                    const uint32_t t = 4u * w + j;
                    is_new |= t >= at.lo && t < at.hi ? 0xffu << (8 * j) : 0u;
                    is_old |= t < at.lo ? 0xffu << (8 * j) : 0u;
                }
                const uint32_t kept = sc.drop > 0 ? rescale4(have[i][w], sc.shrink) : have[i][w];
                v[w] = (v[w] & is_new) | (kept & is_old) | (have[i][w] & ~(is_new | is_old));
            }
        }
        *dst = v;
    }
    if (lane == 0)
        *scale = (uint8_t)sc.byte;
}

// DP: the head's channels rounded up to 128.
template <class T, int DP, int W, class Args>
__device__ __forceinline__ void append_block(const Args &a, uint32_t unit, uint8_t *lds)
{
    const KvPool &pool = a.pool;
    const KvSeqs &sq = a.seqs;
    const uint32_t b = a.by_seq_units.div(unit);
    uint32_t rest = unit - b * a.by_seq_units.d;
    const uint32_t nth = a.by_units.div(rest);
    rest -= nth * a.by_units.d;
    if (b >= sq.seqs)
        return;
    // the sequence's new tokens: first .. end - 1, at start ..
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
    if (col >= sq.bt_width)
        return;
    BlockAt at;
    at.head = rest >> 1;
    at.slot = at.head * pool.blocks + (uint32_t)blk - col * pool.blocks;
    // (checked once the tokens' loads are under way)
    at.page = (uint32_t)sq.block_table[(size_t)b * sq.bt_stride + col];
    at.pos0 = (uint32_t)p0;
    at.lo = start > p0 ? (uint32_t)(start - p0) : 0u;
    at.hi = len - p0 < (int32_t)kBlock ? (uint32_t)(len - p0) : kBlock;
    at.first = first + (uint32_t)(p0 + (int32_t)at.lo - start);
    if (rest & 1u)
        append_values<T, W, DP / 128>(a, at, lds);
    else if (a.q.half)
        append_keys<T, W, DP / 8 / W, true>(a, at);
    else
        append_keys<T, W, DP / 8 / W, false>(a, at);
}

template <class T, int P, int N, class Args>
__device__ __forceinline__ void rotate_queries(const Args &a, uint32_t t, uint32_t part)
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
        auto turn = [&](const auto &angles) {
            if (a.q.half)
                rope_heads<T, P, N, true>(a.q, x, y, h, item, angles, false);
            else
                rope_heads<T, P, N, false>(a.q, x, y, h, item, angles, false);
        };
        if constexpr (has_axes<Args>)
            turn(AxesAngles(a.axes, a.q.table, a.q.table_positions, t));
        else
            turn(RowAngles{(uint32_t)pos < a.q.table_positions ? a.q.table + (size_t)pos * a.q.rot : nullptr});
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

template <class T, int N, class Args>
__device__ __forceinline__ void rotate_queries_by(const Args &a, uint32_t t, uint32_t part)
{
    switch (a.q.pairs) {
    case 8: rotate_queries<T, 8, N>(a, t, part); break;
    case 4: rotate_queries<T, 4, N>(a, t, part); break;
    default: rotate_queries<T, 1, N>(a, t, part); break;
    }
}

template <class T, int DP, int W, class Args>
__global__ __launch_bounds__(256) void w8a16_kv_append_kernel(Args a)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[4][DP / 8 * kChunkPitch];
    if (blockIdx.x < a.kv_groups) {
        const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        append_block<T, DP, W>(a, blockIdx.x * 4u + wave, lds[wave]);
        return;
    }
    const uint32_t g = blockIdx.x - a.kv_groups;
    const uint32_t t = a.by_q_groups.div(g), part = g - t * a.q_groups;
    if (a.q_heads_per_thread == 1)
        rotate_queries_by<T, 1>(a, t, part);
    else
        rotate_queries_by<T, kRopeHeads>(a, t, part);
}

template <class T, int DP, class Args>
hipError_t launch_width(const Args &a, hipStream_t stream)
{
    const uint32_t tokens = a.q.x ? a.seqs.tokens : 0u;
    const dim3 grid(a.kv_groups + tokens * a.q_groups), block(256);
    switch (a.vec) {
    case 8: hipLaunchKernelGGL((w8a16_kv_append_kernel<T, DP, 8, Args>), grid, block, 0, stream, a); break;
    case 4: hipLaunchKernelGGL((w8a16_kv_append_kernel<T, DP, 4, Args>), grid, block, 0, stream, a); break;
    default: hipLaunchKernelGGL((w8a16_kv_append_kernel<T, DP, 1, Args>), grid, block, 0, stream, a); break;
    }
    return hipGetLastError();
}

template <class T, class Args>
hipError_t launch_type(const Args &a, hipStream_t stream)
{
    return a.pool.dim <= 128 ? launch_width<T, 128>(a, stream) : launch_width<T, 256>(a, stream);
}

template <class Args>
hipError_t launch_any(const Args &a, uint32_t dtype, hipStream_t stream)
{
    switch (dtype) {
    case W8A16_BF16: return launch_type<__bf16>(a, stream);
    case W8A16_FP16: return launch_type<_Float16>(a, stream);
    default: return launch_type<float>(a, stream);
    }
}

}  // namespace append

}  // namespace w8a16
