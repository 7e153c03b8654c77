// Attention of many rows (prompts, prompt chunks) over the paged FP8 cache.
//
// The mathematics is that of the row kernel (kv_rows_kernel.h): S^T = K Q^T,
// l += 2^(x - m), O^T += V^T p^T, p = 2^(x + e - M + 11) in FP16, V as its
// codes.
// A wave needs about 320 vector instructions (128 conversions of codes, 34
// exponentials, the rest sums, maxima and conversions of p) beside the 32
// matrix instructions of 64 keys and 128 channels.  So a workgroup takes 128
// rows, its four waves 32 each with 32x32x16 matrix instructions, two
// workgroups share a CU where registers allow (up to 128 channels), and:
//   * 64 keys at a time, K and V as codes (half of what 16-bit operands
//     would read from LDS), brought to LDS by DMA into the third buffer of
//     four from the one in use, one barrier per tile.  Each wave brings one
//     block of 16 keys; page lookups are scalar.
//   * Row 8a + 4h + b of the K operand holds key 16h + 4a + b, so a lane
//     ends up with the 16 scores of one block in order, and its p are the
//     second product's operand as they stand, whose other side is one
//     16-byte read of V (16 keys of one channel), widened in registers.
//   * K rows lie in LDS with their 16-byte chunks permuted (xor) so that the
//     8 lanes served together hit different banks; V needs no permutation.
//   * Tiles that every row sees take a loop without masks.  In it the first
//     products run at a raised wave priority, so that the waves of a SIMD
//     fall out of step and one's exponentials run under another's matrix
//     instructions; the second product follows each half's exponentials at
//     once.
// What bounds it: where two workgroups fill every CU, the rate that the card
// sustains its matrix instructions at beside the widening of codes (without
// the widening 434 us in place of 532, a library's rate for plain products;
// without the exponentials, maxima or sums 520 to 530).  One workgroup alone on
// a CU takes 1.24 us per tile, two between them 2.2.
// Measured, 2 x 2048 tokens of 32 query and 8 KV heads over 8192 keys of 128
// channels: 490 to 520 us by run and card, 925 to 982 TFLOP/s (a plain FP16
// matrix product of 8192^3 reaches 1151 here).  Operands read from LDS ahead of
// their use and scale bytes by DMA took 128 channels from 520 to 514 us, 64
// from 372 to 340, 192 (2 x 1024 tokens over 4024) from 133 to 119, 256 from
// 184 to 155, windows of 1024 keys from 86 to 82.  Windows of 1024 keys with 4
// sinks, 2 x 1501 tokens: 82 to 88, without the sinks 74 to 77 (a tile more,
// seen in part).  While the loop of whole tiles asked for each tile whether
// it was the sinks' or the window's that took 97: 14 moves of spilled scalar
// registers a tile.  Tried on forms of this kernel
// that took 488 to 508: two buffers and one loop for all tiles 530, no
// priority 512, widening once per workgroup into LDS as 16-bit operands 584,
// the next tile's scores under this one's exponentials 602, the raised
// priority for the second product as well 503 or for the exponentials 516.
// FP8 products of queries split in two E4M3 numbers took 508 and summed too
// coarsely (errors of 2e-3 in a row's log-sum).

#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attention.h"
#include "attention_device.h"
#include "device_common.h"
#include "kernels.h"

namespace w8a16 {

namespace tile {

using namespace dev;

typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr uint32_t kRows = 128;      // rows per workgroup
constexpr uint32_t kBuffers = 4;     // tiles in LDS: one in use, three on their way

__device__ const uint8_t no_scale[4] = {0, 0, 0, 0};

template <class Q> __device__ __forceinline__ f32x16_t mfma32(u32x4_t a, u32x4_t b, f32x16_t c);
template <> __device__ __forceinline__ f32x16_t mfma32<QueryBf16>(u32x4_t a, u32x4_t b, f32x16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
template <> __device__ __forceinline__ f32x16_t mfma32<QueryF16>(u32x4_t a, u32x4_t b, f32x16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// max of x over lanes l and l ^ 32
__device__ __forceinline__ float max_halves(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}

// Workgroup `group_id` of a launch of a.grid; AT: where `a` stands among the
// kernel's arguments, in bytes.  Either pass over a shared prefix leaves
// partial rows and no outputs.
template <class Q, int DP, size_t AT, class Args>
__device__ __forceinline__ void kv_tile(const Args &a, uint32_t group_id, uint8_t *lds)
{
    constexpr int QC = DP / 32;             // 32-channel groups of the first product
    constexpr int VT = DP / 32;             // 32-channel tiles of the second
    constexpr uint32_t BLK = 16 * DP;       // LDS bytes of one block of K, and of V
    constexpr uint32_t BUF = 8 * BLK;       // of one buffer
    constexpr uint32_t SWZ = DP == 128 || DP == 256 ? 7 : 3;
    struct Scale { uint32_t ks, vs; };
    struct ScaleRow { Scale s, unused[31]; };     // a wave's DMA writes a word per lane
    // kBuffers buffers of K and V codes, then the blocks' scale bytes
    ScaleRow (*const scl)[4] = reinterpret_cast<ScaleRow (*)[4]>(lds + kBuffers * BUF);
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t col = lane & 31u, h = lane >> 5;
    const KvPool &pool = a.pool;

    // KV heads fastest: with 8 or more of them a head's row tiles share an
    // XCD's L2; the row tiles with the longest rows start first.
    const uint32_t groups = sequences(a) * pool.heads;
    uint32_t id = group_id;
    const uint32_t grp = id % groups;
    id /= groups;
    const uint32_t chunk = id % a.chunks, rtile = a.row_tiles - 1u - id / a.chunks;
    const uint32_t head = grp % pool.heads, b = grp / pool.heads;

    RowTile t;
    if (!extent(a, b, t) || group_id >= a.grid) {
        if (group_id >= a.grid)
            fill_unowned<typename Q::elem>(a, group_id - a.grid, 4);
        return;
    }
    t.rows = t.count * a.group;
    t.row0 = rtile * kRows;
    if (t.row0 >= t.rows)
        return;
    tile_range(a, kRows, t);
    const TileList list(a, t, true);
    const uint32_t tiles = list.tiles;
    const uint32_t begin = chunk * a.chunk_tiles;
    if (begin >= tiles && chunk > 0 && !is_prefix<Args>)
        return;
    const uint32_t end = chunk + 1 == a.chunks || begin + a.chunk_tiles > tiles
                             ? tiles : begin + a.chunk_tiles;
    const bool alone = !is_prefix<Args> && !is_suffix<Args> && (a.chunks == 1 || tiles <= a.chunk_tiles);

    // this wave's rows, and the keys they see
    RowTile w = t;
    w.row0 = t.row0 + 32u * wave;
    if (w.row0 < t.rows)
        tile_range(a, 32u, w);
    else
        w.lo = w.hi = w.all_lo = w.all_hi = 0;
    const uint32_t row = w.row0 + col;
    int32_t rlo, rhi;
    row_range(a, t, row, rlo, rhi);
    const bool none = rhi <= rlo;
    if constexpr (has_sinks<Args>) {      // what is seen behind the sinks
        const int32_t sinks = (int32_t)a.sinks;
        rlo = rlo > sinks ? rlo : sinks;
        w.lo = w.lo > sinks ? w.lo : sinks;
        t.all_lo = t.all_lo > sinks ? t.all_lo : sinks;
    }
    const uint32_t tok = a.by_group.div(row), hq = head * a.group + row - tok * a.group;
    u32x4_t q[QC][2];
    {
        const typename Q::elem *src = reinterpret_cast<const typename Q::elem *>(a.q) +
                                      (int64_t)(t.first + tok) * a.q_token + (int64_t)hq * a.q_head;
        const bool wide = (reinterpret_cast<uintptr_t>(src) & 15u) == 0;
        auto eight = [&](uint32_t d) {
            u32x4_t v = {0u, 0u, 0u, 0u};
            if (row < t.rows && d < pool.dim) {
                if (wide) {
                    v = *reinterpret_cast<const u32x4_t *>(src + d);
                } else {
                    const uint16_t *s16 = reinterpret_cast<const uint16_t *>(src + d);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        v[x] = (uint32_t)s16[2 * x] | ((uint32_t)s16[2 * x + 1] << 16);
                }
            }
            return v;
        };
#pragma unroll
        for (int i = 0; i < QC; ++i) {
            q[i][0] = eight(32u * i + 16u * h);
            q[i][1] = eight(32u * i + 16u * h + 8u);
        }
    }

    // staging: wave x brings block x of a tile
    const uint32_t last_block = t.kv_len > 0 ? (uint32_t)(t.kv_len - 1) / 16u : 0u;
    // (read through the scalar cache: a vector load would have to be waited
    // for together with the DMA in flight)
    typedef const __attribute__((address_space(4))) int32_t *scalar_ptr;
    const scalar_ptr bt = (scalar_ptr)(uintptr_t)(a.seqs.block_table + (size_t)table_row(a, b) * a.seqs.bt_stride);
    struct Where { uint32_t page, slot, ok; };
    auto locate = [&](uint32_t tile) {
        uint32_t blk = 4u * tile + wave;
        blk = blk < last_block ? blk : last_block;
        const uint32_t c = pool.by_blocks.div(blk);
        Where p;
        p.slot = head * pool.blocks + blk - c * pool.blocks;
        const bool in = c < a.seqs.bt_width;
        p.page = (uint32_t)bt[in ? c : 0u];
        p.ok = in && p.page < pool.pages ? 1u : 0u;
        p.page = p.ok ? p.page : 0u;
        return p;
    };
    // lane's place in each 1 KiB piece of a block
    uint32_t koff[DP / 64], voff[DP / 64];
#pragma unroll
    for (int j = 0; j < DP / 64; ++j) {
        const uint32_t byte = 1024u * j + 16u * lane, r = byte / DP, slot = byte % DP / 16u;
        const uint32_t f = SWZ == 7 ? (r & 3u) | ((wave & 1u) << 2) : ((r >> 1) & 1u) | ((wave & 1u) << 1);
        uint32_t c = slot ^ f;
        c = 16u * c < pool.dim ? c : 0u;      // channels past the head meet queries of zero
        koff[j] = r * pool.dim + 16u * c;
        const uint32_t d = 64u * j + lane;
        voff[j] = 16u * (d < pool.dim ? d : 0u);
    }
    auto stage = [&](const Where &p, uint32_t buf) {
        const size_t base = (size_t)p.slot * 16u * pool.dim;
        const uint8_t *kp = pool.k + p.page * pool.k_page + base;
        const uint8_t *vp = pool.v + p.page * pool.v_page + base;
#pragma unroll
        for (int j = 0; j < DP / 64; ++j) {
            __builtin_amdgcn_global_load_lds(kp + koff[j], (lds_void_t *)(lds + buf * BUF + wave * BLK + 1024u * j),
                                             16, 0, 0);
            __builtin_amdgcn_global_load_lds(vp + voff[j], (lds_void_t *)(lds + buf * BUF + (4 + wave) * BLK + 1024u * j),
                                             16, 0, 0);
        }
        // The block's scale bytes, of a page that does not exist 0 (no
        // scale).  By DMA like the codes: as vector loads the compiler waited
        // for them, hence for every load in flight, a tile later, and as
        // scalar loads every wait for LDS waited for them.
        const uint8_t *const kb = p.ok ? pool.k_scale + p.page * pool.ks_page + p.slot : no_scale;
        const uint8_t *const vb = p.ok ? pool.v_scale + p.page * pool.vs_page + p.slot : no_scale;
        __builtin_amdgcn_global_load_lds(lane & 1u ? vb : kb, (lds_void_t *)&scl[buf][wave], 1, 0, 0);
    };
    f32x16_t o[VT];
#pragma unroll
    for (int x = 0; x < VT; ++x)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[x][i] = 0.f;
    RowRef m;
    float l = 0.f;

    // LDS offsets of the lane's K row for each chunk pair, and of its V row
    const uint32_t krow = 16u * ((col >> 2) & 1u) + 4u * (col >> 3) + (col & 3u);
    const uint32_t kf = SWZ == 7 ? (krow & 3u) | ((krow >> 4) << 2) : ((krow >> 1) & 1u) | ((krow >> 4) << 1);
    const uint32_t kbase = krow * DP;

    auto k_frag = [&](uint32_t buf, int x, int i) {
        return *reinterpret_cast<const u32x4_t *>(lds + buf * BUF + x * 2 * BLK + kbase + 16u * ((2u * i + h) ^ kf));
    };
    // Scores of 32 keys (half x of the tile), as the codes have them.
    auto products = [&](uint32_t buf, int x) {
        f32x16_t s;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s[i] = 0.f;
#pragma unroll
        for (int i = 0; i < QC; ++i) {
            const u32x4_t raw = k_frag(buf, x, i);
            s = mfma32<Q>(Q::widen(raw.x, raw.y), q[i][0], s);
            s = mfma32<Q>(Q::widen(raw.z, raw.w), q[i][1], s);
        }
        return s;
    };
    auto v_frag = [&](uint32_t buf, int x, int d) {
        return *reinterpret_cast<const u32x4_t *>(lds + buf * BUF + (4u + 2u * x + h) * BLK +
                                                  (32u * d + col) * 16u);
    };
    // Moves a row's references if the tile's largest score passes them by too
    // much; mx: the largest of each half in this lane, e its V exponent.
    auto refer = [&](const float (&mx)[2], const float (&e)[2]) {
        if (__ballot(m.passed(mx[0], e[0]) || m.passed(mx[1], e[1]))) {
            const RowRef was = m;
            m.move(max_halves(fmaxf(mx[0], mx[1])), max_halves(fmaxf(mx[0] + e[0], mx[1] + e[1])));
            l *= exp2_fast(was.sum - m.sum);
            const float f = exp2_fast(was.out - m.out);
#pragma unroll
            for (int x = 0; x < VT; ++x)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[x][i] *= f;
        }
    };
    // A block far from the row's others: its weights by themselves to l, its
    // operands' sum to nothing.  (Some lanes of a wave may take this branch.
    // In one form of the masked tiles below the compiler moved the 16
    // accumulators of a channel tile to other registers right behind it, before
    // it had put the other lanes back in EXEC, and those lost them: the wrong
    // copies stand in that build's assembly, in no kernel's here, and not
    // without -amdgpu-mfma-vgpr-form.)
    auto far = [&](const f32x16_t &s, float c, float &shift) {
        shift = kNegInf;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            l += s[i] == kNegInf ? 0.f : exp2_fast(fmaf(s[i], c, -m.sum));
    };
    // Scores of one block to operands of the second product, and to l, where
    // their sum counts 2^shift; hidden: some may be -inf under a scale of NaN
    // or 0.
    auto weigh = [&](f32x16_t &s, float c, float e, float shift, auto hidden) {
        const float mu = m.out - e;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float v = exp2_fast(fmaf(s[i], c, -mu));
            s[i] = decltype(hidden)::value && s[i] == kNegInf ? 0.f : v;
            sum += s[i];
        }
        l = fmaf(sum, exp2_fast(shift), l);
    };
    auto largest = [&](const f32x16_t &s) {
        float mx = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i)
            mx = fmaxf(mx, s[i]);
        return mx;
    };
    auto pack = [&](const f32x16_t &s, u32x4_t (&p)[2]) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            p[i >> 2][i & 3] = f16_pair(s[2 * i], s[2 * i + 1]);
    };

    // What is seldom needed of the arguments is read where it is: loaded with
    // the others it would stay in scalar registers, or be moved out of them
    // and back, all through the loop (the outputs' strides, windows of 1000
    // keys of 64 channels: 71.3 us, so 67.8).
    typedef const __attribute__((address_space(4))) Args *args_ptr;
    auto late_args = [&]() {
        args_ptr late = (args_ptr)((const __attribute__((address_space(4))) uint8_t *)
                                       __builtin_amdgcn_kernarg_segment_ptr() + AT);
        asm volatile("" : "+s"(late));
        return late;
    };

    // A tile that every row of the workgroup sees, its blocks all with scales.
    auto whole = [&](uint32_t buf) {
        f32x16_t s[2];
        float c[2], e[2], mx[2];
        // K of the whole tile is under way before its first product, V of a
        // half before its exponentials or the other half's products.  (Left to
        // the compiler each pair of reads was waited for.)
        u32x4_t k[2][QC], v[VT];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < QC; ++i)
                k[x][i] = k_frag(buf, x, i);
        const Scale sc[2] = {scl[buf][h].s, scl[buf][2 + h].s};
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[x][i] = 0.f;
#pragma unroll
            for (int i = 0; i < QC; ++i) {
                s[x] = mfma32<Q>(Q::widen(k[x][i].x, k[x][i].y), q[i][0], s[x]);
                s[x] = mfma32<Q>(Q::widen(k[x][i].z, k[x][i].w), q[i][1], s[x]);
            }
        }
        __builtin_amdgcn_s_setprio(0);
#pragma unroll
        for (int d = 0; d < VT; ++d)
            v[d] = v_frag(buf, 0, d);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            c[x] = pow2_byte(sc[x].ks) * a.scale_log2;
            e[x] = (float)sc[x].vs - 127.0f;
            mx[x] = largest(s[x]) * c[x];
        }
        refer(mx, e);
        // (one branch for the tile: the masked form's one for each half cost
        // 2 to 4 % here, 64 channels 345 us and 337, and both forms' one for
        // the tile spilled at 128 channels)
        float shift[2] = {m.shift(e[0]), m.shift(e[1])};
        if (__ballot(fabsf(shift[0]) > kFar || fabsf(shift[1]) > kFar)) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (fabsf(shift[x]) > kFar)
                    far(s[x], c[x], shift[x]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            u32x4_t p[2];
            weigh(s[x], c[x], e[x], shift[x], std::false_type{});
            pack(s[x], p);
#pragma unroll
            for (int d = 0; d < VT; ++d) {
                const u32x4_t raw = v[d];
                if (x == 0)
                    v[d] = v_frag(buf, 1, d);
                o[d] = mfma32<QueryF16>(f16_from_fp8x8(raw.x, raw.y, 1.0f), p[0], o[d]);
                o[d] = mfma32<QueryF16>(f16_from_fp8x8(raw.z, raw.w, 1.0f), p[1], o[d]);
            }
        }
    };

    // Any tile: some rows may not see all of it, blocks may have no scale.
    // first: one of the sinks', of which no other keys are seen.
    auto partly = [&](uint32_t tile, uint32_t buf, bool first) {
        int32_t lo = rlo, hi = rhi, wlo = w.lo, whi = w.hi;
        if constexpr (has_sinks<Args>)
            if (first) {
                const int32_t sinks = (int32_t)late_args()->sinks;
                lo = wlo = 0;
                hi = hi < sinks ? hi : sinks;
                whi = whi < sinks ? whi : sinks;
            }
        const int32_t tk = (int32_t)(tile * kKvTile), key0 = tk + 16 * (int32_t)h;   // of half x: + 32 x
        f32x16_t s[2];
        float c[2], e[2], mx[2];
        uint32_t poison[2];      // a block without a V scale reads as NaN codes
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const Scale sc = scl[buf][2 * x + h].s;
            c[x] = sc.ks - 1u >= 254u ? __builtin_nanf("") : pow2_byte(sc.ks) * a.scale_log2;
            e[x] = (float)sc.vs - 127.0f;
            poison[x] = sc.vs - 1u >= 254u ? 0x7f7f7f7fu : 0u;
            s[x] = products(buf, x);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[x][i] = key0 + 32 * x + i >= lo && key0 + 32 * x + i < hi ? s[x][i] : kNegInf;
            mx[x] = largest(s[x]) * c[x];
        }
        refer(mx, e);
        u32x4_t p[2][2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float shift = m.shift(e[x]);
            if (fabsf(shift) > kFar)
                far(s[x], c[x], shift);
            weigh(s[x], c[x], e[x], shift, std::true_type{});
            pack(s[x], p[x]);
        }
        // Codes of half x that some row of the wave may see.
        auto kept = [&](int x, int d) {
            u32x4_t v = v_frag(buf, x, d) | (x ? poison[1] : poison[0]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t keep = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int32_t key = key0 + 32 * x + 4 * i + j;
                    keep |= key >= wlo && key < whi ? 0xffu << (8 * j) : 0u;
                }
                v[i] &= keep;
            }
            return v;
        };
        uint32_t any = 0;
#pragma unroll
        for (int d = 0; d < VT; ++d)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                // 0 * NaN must not reach rows that do not see the key
                u32x4_t raw = kept(x, d);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t nan = nan_bytes(raw[i]);
                    any |= nan;
                    raw[i] &= ~((nan >> 7) * 0xffu);
                }
                o[d] = mfma32<QueryF16>(f16_from_fp8x8(raw.x, raw.y, 1.0f), p[x][0], o[d]);
                o[d] = mfma32<QueryF16>(f16_from_fp8x8(raw.z, raw.w, 1.0f), p[x][1], o[d]);
            }
        if (__ballot(any != 0)) {
            // NaN for the rows that do see one: a product that counts them
#pragma unroll
            for (int d = 0; d < VT; ++d) {
                f32x16_t n;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    n[i] = 0.f;
#pragma unroll 1
                for (int x = 0; x < 2; ++x) {
                    const u32x4_t raw = kept(x, d);
                    u32x4_t bad[2], seen[2];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t nb = nan_bytes(raw[i]) >> 7;
                        bad[i >> 1][2 * (i & 1)] = ((nb & 1u) | ((nb & 0x100u) << 8)) * 0x3c00u;
                        bad[i >> 1][2 * (i & 1) + 1] = (((nb >> 16) & 1u) | ((nb >> 8) & 0x10000u)) * 0x3c00u;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int32_t key = key0 + 32 * x + 2 * i;
                        seen[i >> 2][i & 3] =
                            (key >= lo && key < hi ? 0x3c00u : 0u) |
                            (key + 1 >= lo && key + 1 < hi ? 0x3c000000u : 0u);
                    }
                    n = mfma32<QueryF16>(bad[0], seen[0], n);
                    n = mfma32<QueryF16>(bad[1], seen[1], n);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[d][i] = n[i] > 0.f ? __builtin_nanf("") : o[d][i];
            }
        }
    };

    if (begin < end) {
        // Tiles every row of the workgroup sees run in a loop of their own; it
        // ends early at a block without a scale.
        const int32_t past = (int32_t)list.tile0 - (int32_t)list.front;   // a tile of the range is this much less in the list
        const int32_t w0 = (t.all_lo + (int32_t)kKvTile - 1) / (int32_t)kKvTile - past;
        const int32_t w1 = t.all_hi / (int32_t)kKvTile - past;
        const uint32_t whole0 = w0 > (int32_t)begin ? (uint32_t)w0 : begin;
        const uint32_t whole1 = w1 > (int32_t)end ? end : w1 > 0 ? (uint32_t)w1 : 0u;
        // (all of the first tiles' loads before the first wait for one)
        Where at[kBuffers - 1];
#pragma unroll
        for (uint32_t k = 0; k + 1 < kBuffers; ++k)
            at[k] = locate(list.at(begin + k));
#pragma unroll
        for (uint32_t k = 0; k + 1 < kBuffers; ++k)
            stage(at[k], k);
        Where next = locate(list.at(begin + kBuffers - 1));
        wait_vm<0>();
        __syncthreads();
        uint32_t tile = begin, buf = 0;
        // (behind the sinks' tiles: whether the tile at hand is)
        auto place = [&](uint32_t n, auto behind) {
            return decltype(behind)::value ? n + (uint32_t)past : list.at(n);
        };
        auto ahead = [&](auto behind) {
            stage(next, (buf + 3u) & 3u);
            next = locate(place(tile + kBuffers, behind));
        };
        // The next tile has arrived when no more loads are open than the two
        // tiles after it take: K and V pieces and the scale bytes each.
        auto turn = [&]() {
            wait_vm<2 * (2 * (DP / 64) + 1)>();
            barrier_lds();
            ++tile;
            buf = (buf + 1u) & 3u;
        };
        auto scaled = [&](uint32_t in) {
            const Scale s = scl[in][lane & 3u].s;
            return !__ballot(s.ks - 1u >= 254u || s.vs - 1u >= 254u);
        };
        auto general = [&](uint32_t stop, auto behind) {
            while (tile < stop) {
                ahead(behind);
                const uint32_t at_tile = place(tile, behind);
                const int32_t tk = (int32_t)(at_tile * kKvTile);
                const bool first = has_sinks<Args> && !decltype(behind)::value && tile < list.front;
                if (tk < w.hi && (tk + (int32_t)kKvTile > w.lo || first))      // some key of it is for this wave
                    partly(at_tile, buf, first);
                turn();
            }
        };
        general(whole0 < end ? whole0 : end, std::false_type{});
        while (tile < whole1 && scaled(buf)) {
            ahead(std::true_type{});
            whole(buf);
            turn();
        }
        general(end, std::true_type{});
        wait_vm<0>();
    }

    // a row's sum is in two lanes; its output in both, 4 channels at a time
    l += __shfl_xor(l, 32, 64);
    if (row >= t.rows)
        return;
    const args_ptr late = late_args();
    if (alone) {
        const float inv = none ? 0.f : 1.0f / l;
        const float unit = m.out - m.sum;
        typename Q::elem *dst = reinterpret_cast<typename Q::elem *>(late->out) +
                                (int64_t)(t.first + tok) * late->out_token + (int64_t)hq * late->out_head;
        const bool wide = (reinterpret_cast<uintptr_t>(dst) & 7u) == 0;
#pragma unroll
        for (int d = 0; d < VT; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t c = 32u * d + 8u * g + 4u * h;
                if (c >= pool.dim)
                    continue;
                typename Q::elem v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = static_cast<typename Q::elem>(scale2(o[d][4 * g + i] * inv, unit));
                if (wide) {
                    u32x2_t pk;
                    pk.x = (uint32_t)__builtin_bit_cast(uint16_t, v[0]) |
                           ((uint32_t)__builtin_bit_cast(uint16_t, v[1]) << 16);
                    pk.y = (uint32_t)__builtin_bit_cast(uint16_t, v[2]) |
                           ((uint32_t)__builtin_bit_cast(uint16_t, v[3]) << 16);
                    *reinterpret_cast<u32x2_t *>(dst + c) = pk;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        dst[c + i] = v[i];
                }
            }
        if (late->lse && h == 0)
            late->lse[(size_t)(t.first + tok) * late->q_heads + hq] =
                none ? kNegInf : (m.sum + log2f(l)) * 0.69314718055994531f;
        return;
    }
    // partial rows in the join kernel's order: ((b, head), rtile, chunk)
    const size_t part = (((size_t)grp * a.row_tiles + rtile) * a.chunks + chunk) * kRows + 32u * wave + col;
    float *wo = late->ws + part * pool.dim;
    float *wst = late->ws + (size_t)late->grid * kRows * pool.dim + part * 4u;
#pragma unroll
    for (int d = 0; d < VT; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const uint32_t c = 32u * d + 8u * g + 4u * h;
            if (c < pool.dim)
                *reinterpret_cast<f32x4_t *>(wo + c) =
                    f32x4_t{o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]};
        }
    if (h == 0) {
        wst[0] = m.sum;
        wst[1] = l;
        wst[2] = m.out;
    }
}

template <class Q, int DP, class Args>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void w8a16_kv_tile_kernel(Args a)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    kv_tile<Q, DP, 0>(a, blockIdx.x, lds);
}

// Dynamic LDS: codes and scale bytes.
template <int DP> constexpr uint32_t tile_lds = kBuffers * (8 * 16 * DP + 4 * 64 * 4);

template <class Q, int DP, class Args>
hipError_t launch_dim(const Args &a, hipStream_t stream)
{
    const uint32_t bytes = tile_lds<DP>;
    static std::atomic<uint64_t> lds_set{0};
    auto kern = w8a16_kv_tile_kernel<Q, DP, Args>;
    hipError_t e = allow_lds(reinterpret_cast<const void *>(kern), bytes, bytes, lds_set);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(kern, dim3((uint32_t)kv_launch_groups(a, 4)), dim3(256), bytes, stream, a);
    return hipGetLastError();
}

template <class Q, class Args>
hipError_t launch_type(const Args &a, hipStream_t stream)
{
    switch ((a.pool.dim + 63u) / 64u) {
    case 1: return launch_dim<Q, 64>(a, stream);
    case 2: return launch_dim<Q, 128>(a, stream);
    case 3: return launch_dim<Q, 192>(a, stream);
    default: return launch_dim<Q, 256>(a, stream);
    }
}

}  // namespace tile

template <class Args> hipError_t launch_kv_tile(const Args &a, uint32_t dtype, hipStream_t stream)
{
    return dtype == W8A16_BF16 ? tile::launch_type<dev::QueryBf16>(a, stream)
                               : tile::launch_type<dev::QueryF16>(a, stream);
}

}  // namespace w8a16
