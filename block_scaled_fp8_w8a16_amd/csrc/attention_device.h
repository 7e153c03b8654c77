// Device pieces shared by the attention kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attention.h"
#include "device_common.h"
#include "rope_device.h"

namespace w8a16 {
namespace dev {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

constexpr float kNegInf = -__builtin_inff();

// A row's running references.  With x the base-2 logarithm of a key's weight
// before the softmax's division, and e the exponent of its block's V scale,
//     l sums 2^(x - sum),   the outputs sum 2^(x + e - out) times V's codes:
// the V scales ride on the weights, so a block enters only the rows that see
// it, and V's codes are exact in FP16.  Both references are whole numbers
// (moving them rounds nothing) and left alone until a maximum passes them by
// too much: the operand, rounded to FP16, is at most 2^15, and a row's
// largest at least 2^(kTop - 1).
constexpr float kTop = 11.0f;
constexpr float kLazy = 4.0f;
constexpr float kUnset = -3.0e38f;     // of a row that has seen no key: below any, and
                                       // finite, so that references can be subtracted
constexpr float kFar = 60.0f;
struct RowRef {
    float sum = kUnset, out = kUnset;
    // Whether `top`, the largest x of a block of exponent e, is too far above.
    __device__ __forceinline__ bool passed(float top, float e) const
    {
        return top > sum + kLazy || top + e > out + (kTop + kLazy);
    }
    __device__ __forceinline__ void move(float top, float top_out)
    {
        sum = top > sum + kLazy ? ceilf(top) : sum;
        out = top_out > out + (kTop + kLazy) ? ceilf(top_out) - kTop : out;
    }
    // What turns the operands of a block into the weights that l sums, as an
    // exponent: one multiplication per block in place of an exponential per
    // key.  Past kFar (a V scale far from the row's others) the operands may
    // have left FP32's range where the weights have not: those blocks'
    // weights are computed by themselves and the operands' sum is dropped.
    __device__ __forceinline__ float shift(float e) const { return out - sum - e; }
};

// Query types: K codes are widened to the query's type with scale 1, which
// is exact for both (E4M3 spans 2^-9 .. 448), so the products see the query
// unrounded; the block's scale multiplies the FP32 sums.
template <bool HI>
__device__ __forceinline__ uint32_t f16_pair_from_fp8(uint32_t raw, float scale)
{
    auto v = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw, scale, HI);
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ u32x4_t f16_from_fp8x8(uint32_t a, uint32_t b, float scale)
{
    u32x4_t r;
    r.x = f16_pair_from_fp8<false>(a, scale);
    r.y = f16_pair_from_fp8<true>(a, scale);
    r.z = f16_pair_from_fp8<false>(b, scale);
    r.w = f16_pair_from_fp8<true>(b, scale);
    return r;
}

struct QueryBf16 {
    typedef __bf16 elem;
    static __device__ __forceinline__ u32x4_t widen(uint32_t a, uint32_t b)
    {
        u32x4_t r;
        r.x = bf16_pair_from_fp8<false>(a);
        r.y = bf16_pair_from_fp8<true>(a);
        r.z = bf16_pair_from_fp8<false>(b);
        r.w = bf16_pair_from_fp8<true>(b);
        return r;
    }
    static __device__ __forceinline__ f32x4_t mfma16(u32x4_t k, u32x4_t q, f32x4_t c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, k),
                                                       __builtin_bit_cast(bf16x8_t, q), c, 0, 0, 0);
    }
};

struct QueryF16 {
    typedef _Float16 elem;
    static __device__ __forceinline__ u32x4_t widen(uint32_t a, uint32_t b)
    {
        return f16_from_fp8x8(a, b, 1.0f);
    }
    static __device__ __forceinline__ f32x4_t mfma16(u32x4_t k, u32x4_t q, f32x4_t c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, k),
                                                      __builtin_bit_cast(f16x8_t, q), c, 0, 0, 0);
    }
};

__device__ __forceinline__ f32x4_t mfma16_f16(u32x4_t a, u32x4_t b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t f16_pair(float a, float b)
{
    f16x2_t v = {static_cast<_Float16>(a), static_cast<_Float16>(b)};
    return __builtin_bit_cast(uint32_t, v);
}

// 2^x of the hardware (within 1 ulp); 2^-inf is 0.
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// x * 2^n of a whole number n, subnormal results included.
__device__ __forceinline__ float scale2(float x, float n)
{
    return ldexpf(x, (int)fminf(fmaxf(n, -400.0f), 400.0f));
}

__device__ __forceinline__ float pow2_byte(uint32_t byte)     // 2^(byte - 127), bytes 1..254
{
    return __builtin_bit_cast(float, byte << 23);
}

// 0x80 in each byte of w whose code is NaN (0x7f or 0xff).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w)
{
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// What one workgroup knows about its sequence and rows.
struct RowTile {
    uint32_t first, count;       // the sequence's new tokens
    int32_t kv_len, base;        // tokens held; position of new token 0
    uint32_t rows, row0;         // rows (token * group + head) of the sequence; first of the tile
    int32_t lo, hi;              // keys some row of the tile may see: [lo, hi)
    int32_t all_lo, all_hi;      // keys every row of the tile sees: [all_lo, all_hi)
};

// Sequence b's extent; false if its offsets do not lie in the token axis.
__device__ __forceinline__ bool seq_extent(const KvSeqs &s, uint32_t b, RowTile &t)
{
    t.first = b * s.uniform;
    uint32_t end = t.first + s.uniform;
    if (s.cu) {
        t.first = (uint32_t)s.cu[b];
        end = (uint32_t)s.cu[b + 1];
    }
    t.count = end - t.first;
    t.kv_len = s.kv_lens[b];
    t.base = t.kv_len - (int32_t)t.count;
    return t.first <= s.tokens && end <= s.tokens && end >= t.first;
}

// The workgroup's sequence; the first pass over a shared prefix takes all of
// the call's tokens for one.
__device__ __forceinline__ bool extent(const AttnArgs &a, uint32_t b, RowTile &t)
{
    return seq_extent(a.seqs, b, t);
}

__device__ __forceinline__ bool extent(const PrefixArgs &a, uint32_t, RowTile &t)
{
    t.first = 0;
    t.count = a.seqs.tokens;
    t.kv_len = (int32_t)a.shared;
    t.base = 0;
    return true;
}

__device__ __forceinline__ uint32_t sequences(const AttnArgs &a) { return a.seqs.seqs; }
__device__ __forceinline__ uint32_t sequences(const PrefixArgs &) { return 1; }

// The row of the block table that leads to the keys: for a shared prefix
// that of a sequence which holds all of it, else (every row then sees less
// of it) of the longest.  A slot that brings no tokens leads nowhere: its
// length and row may be anything.
__device__ __forceinline__ uint32_t table_row(const AttnArgs &, uint32_t b) { return b; }

__device__ __forceinline__ uint32_t table_row(const PrefixArgs &a, uint32_t)
{
    const KvSeqs &s = a.seqs;
    const uint32_t lane = threadIdx.x & 63u;
    int32_t most = -1;
    uint32_t longest = 0;
    for (uint32_t b0 = 0; b0 < s.seqs; b0 += 64u) {
        const uint32_t b = b0 + lane, in = b < s.seqs ? b : s.seqs - 1u;
        int32_t len = s.kv_lens[in];
        if (s.cu) {
            const uint32_t first = (uint32_t)s.cu[in], end = (uint32_t)s.cu[in + 1];
            len = first < end && end <= s.tokens ? len : -1;
        }
        len = b < s.seqs ? len : -1;
        const uint64_t whole = __ballot(len >= (int32_t)a.shared);
        if (whole)
            return __builtin_amdgcn_readfirstlane(b0 + (uint32_t)__builtin_ctzll(whole));
        if (len > most) {
            most = len;
            longest = b;
        }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const int32_t len = __shfl_xor(most, off, 64);
        const uint32_t b = __shfl_xor(longest, off, 64);
        longest = len > most || (len == most && b < longest) ? b : longest;
        most = len > most ? len : most;
    }
    return __builtin_amdgcn_readfirstlane(longest);
}

__device__ __forceinline__ void tile_range(const AttnArgs &a, uint32_t tile_rows, RowTile &t)
{
    const uint32_t last = t.row0 + tile_rows < t.rows ? t.row0 + tile_rows : t.rows;
    const int32_t p0 = t.base + (int32_t)a.by_group.div(t.row0);
    const int32_t p1 = t.base + (int32_t)a.by_group.div(last - 1);
    t.hi = a.causal ? (p1 + 1 < t.kv_len ? p1 + 1 : t.kv_len) : t.kv_len;
    if (p1 < 0)
        t.hi = 0;      // rows of no sequence see nothing
    t.lo = 0;
    if (a.window && p0 >= (int32_t)a.window)
        t.lo = p0 - (int32_t)a.window + 1;
    t.hi = t.hi > t.lo ? t.hi : t.lo;
    t.all_lo = a.window && p1 >= (int32_t)a.window ? p1 - (int32_t)a.window + 1 : 0;
    t.all_hi = p0 < 0 ? 0 : (a.causal && p0 + 1 < t.kv_len ? p0 + 1 : t.kv_len);
}

// Keys row `row` sees: [lo, hi).
__device__ __forceinline__ void row_range(const AttnArgs &a, const RowTile &t, uint32_t row,
                                          int32_t &lo, int32_t &hi)
{
    const int32_t p = t.base + (int32_t)a.by_group.div(row);
    hi = row < t.rows && p >= 0 ? (a.causal && p + 1 < t.kv_len ? p + 1 : t.kv_len) : 0;
    lo = a.window && p >= (int32_t)a.window ? p - (int32_t)a.window + 1 : 0;
}

__device__ __forceinline__ void row_range(const PrefixArgs &a, const RowTile &t, uint32_t row, int32_t &lo,
                                          int32_t &hi)
{
    lo = hi = 0;
    if (row >= t.rows)
        return;
    uint32_t b;
    int32_t p;
    if (!token_place(a.seqs, a.by_group.div(row), b, p))
        return;
    const int32_t len = a.causal ? p + 1 : a.seqs.kv_lens[b];
    hi = len < (int32_t)a.shared ? len : (int32_t)a.shared;
}

// (all lanes of the wave together)
__device__ __forceinline__ void tile_range(const PrefixArgs &a, uint32_t tile_rows, RowTile &t)
{
    int32_t most = 0, least = (int32_t)a.shared;
    for (uint32_t r = threadIdx.x & 63u; r < tile_rows && t.row0 + r < t.rows; r += 64u) {
        int32_t lo, hi;
        row_range(a, t, t.row0 + r, lo, hi);
        most = hi > most ? hi : most;
        least = hi < least ? hi : least;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const int32_t x = __shfl_xor(most, off, 64), y = __shfl_xor(least, off, 64);
        most = x > most ? x : most;
        least = y < least ? y : least;
    }
    t.lo = t.all_lo = 0;
    t.hi = __builtin_amdgcn_readfirstlane(most);
    t.all_hi = __builtin_amdgcn_readfirstlane(least);
}

__device__ __forceinline__ void row_range(const SuffixArgs &a, const RowTile &t, uint32_t row, int32_t &lo,
                                          int32_t &hi)
{
    row_range(static_cast<const AttnArgs &>(a), t, row, lo, hi);
    lo = (int32_t)a.shared;
}

__device__ __forceinline__ void tile_range(const SuffixArgs &a, uint32_t tile_rows, RowTile &t)
{
    tile_range(static_cast<const AttnArgs &>(a), tile_rows, t);
    t.lo = t.all_lo = (int32_t)a.shared;
    t.hi = t.hi > t.lo ? t.hi : t.lo;
}

// First tokens that rows see besides their range (no further than it ends),
// and their tiles in front of a row tile's range.
__device__ __forceinline__ int32_t sinks_of(const AttnArgs &) { return 0; }
__device__ __forceinline__ int32_t sinks_of(const SinkArgs &a) { return (int32_t)a.sinks; }

template <class Args> constexpr bool has_sinks = std::is_same<Args, SinkArgs>::value;
template <class Args> constexpr bool is_prefix = std::is_same<Args, PrefixArgs>::value;
template <class Args> constexpr bool is_suffix = std::is_same<Args, SuffixArgs>::value;

// The tiles a row tile goes over, numbered from 0: those of its sinks, as far
// as they lie before its range, then its range's.  apart: all of the sinks',
// then those of its range behind the sinks (so one tile can be in both parts).
struct TileList {
    uint32_t front, tile0, tiles;
    template <class Args> __device__ __forceinline__ TileList(const Args &a, const RowTile &t, bool apart = false)
    {
        uint32_t lo = (uint32_t)t.lo;
        front = 0;
        if constexpr (has_sinks<Args>) {
            const uint32_t hi = (uint32_t)t.hi, sinks = a.sinks < hi ? a.sinks : hi;
            const uint32_t n = apart ? (sinks + kKvTile - 1) / kKvTile : (a.sinks - 1u) / kKvTile + 1u;
            if (apart)
                lo = lo > sinks ? lo : sinks;
            front = apart || n < lo / kKvTile ? n : lo / kKvTile;
            if (apart && lo >= hi)
                lo = n * kKvTile;      // (all of the range is sinks)
        }
        tile0 = lo / kKvTile;
        const uint32_t end = ((uint32_t)t.hi + kKvTile - 1) / kKvTile;
        tiles = (end > tile0 ? end - tile0 : 0u) + front;
    }
    __device__ __forceinline__ uint32_t at(uint32_t n) const { return n < front ? n : n - front + tile0; }
};

// Where the first pass has left the partial row of row `row` of the call
// (token * group + head of the group) and chunk c of the prefix.
template <class Args>
__device__ __forceinline__ size_t prefix_partial(const Args &a, uint32_t head, uint32_t row, uint32_t c)
{
    if constexpr (is_suffix<Args>) {
        const uint32_t tile = row >> a.prefix_shift;
        return ((((size_t)head * a.prefix_tiles + tile) * a.prefix_chunks + c) << a.prefix_shift) +
               (row - (tile << a.prefix_shift));
    }
    return 0;
}

// (Such a row gives zeros.  One whose visible scores are all -inf sums to
// zero too, and has no softmax: its 0 / 0 stays.)
// (Over a shared prefix: whatever part of the keys a pass takes.)
__device__ __forceinline__ bool sees_nothing(const AttnArgs &a, const RowTile &t, uint32_t row)
{
    int32_t lo, hi;
    row_range(a, t, row, lo, hi);
    return hi <= lo;
}

// Four outputs of a row, v * 2^n, rounded to its type.
template <class E> __device__ __forceinline__ void store_row4(E *dst, f32x4_t v, float n)
{
    const E e[4] = {static_cast<E>(scale2(v.x, n)), static_cast<E>(scale2(v.y, n)),
                    static_cast<E>(scale2(v.z, n)), static_cast<E>(scale2(v.w, n))};
    if ((reinterpret_cast<uintptr_t>(dst) & 7u) == 0) {
        u32x2_t p;
        p.x = (uint32_t)__builtin_bit_cast(uint16_t, e[0]) | ((uint32_t)__builtin_bit_cast(uint16_t, e[1]) << 16);
        p.y = (uint32_t)__builtin_bit_cast(uint16_t, e[2]) | ((uint32_t)__builtin_bit_cast(uint16_t, e[3]) << 16);
        *reinterpret_cast<u32x2_t *>(dst) = p;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            dst[i] = e[i];
    }
}

// Zeros, and log-sums of -inf, for the rows of tokens that no sequence
// brings, among those of this wave: each of workgroup `part`'s `waves` waves
// takes fill_tokens of the token axis and lays its lanes over the sequences.
// Beside the attention's own workgroups it costs little: 64 sequences of 300
// tokens 9.2 us with no token left out, 10.7 with 192.
template <class E>
__device__ __forceinline__ void fill_unowned(const AttnArgs &a, uint32_t part, uint32_t waves)
{
    const KvSeqs &s = a.seqs;
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t t0 = (part * waves + wave) * a.fill_tokens;
    if (t0 >= s.tokens)
        return;
    const uint32_t n = s.tokens - t0 < a.fill_tokens ? s.tokens - t0 : a.fill_tokens;
    uint64_t left = n < 64u ? (1ull << n) - 1u : ~0ull;      // a bit per token
    for (uint32_t b0 = 0; b0 < s.seqs; b0 += 64u) {
        uint32_t first = ~0u, end = 0;
        if (b0 + lane < s.seqs) {
            first = (uint32_t)s.cu[b0 + lane];
            end = (uint32_t)s.cu[b0 + lane + 1];
        }
        if (end > s.tokens)
            end = 0;
        for (uint32_t i = 0; i < n; ++i)
            if (__ballot(t0 + i >= first && t0 + i < end))
                left &= ~(1ull << i);
    }
    const uint32_t pieces = a.pool.dim / 4, all = a.q_heads * pieces;
    for (; left; left &= left - 1) {
        const size_t t = t0 + (uint32_t)__builtin_ctzll(left);
        for (uint32_t i = lane; i < all; i += 64u) {
            const uint32_t h = i / pieces;
            store_row4(reinterpret_cast<E *>(a.out) + (int64_t)t * a.out_token + (int64_t)h * a.out_head +
                           4 * (i - h * pieces), f32x4_t{0.f, 0.f, 0.f, 0.f}, 0.f);
        }
        for (uint32_t h = lane; a.lse && h < a.q_heads; h += 64u)
            a.lse[t * a.q_heads + h] = kNegInf;
    }
}

}  // namespace dev
}  // namespace w8a16
