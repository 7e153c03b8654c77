// Attention of a few rows (decode, drafts) over the paged FP8 cache.
//
// Mathematics.  For one KV head, the rows r = (new token, query head of the
// group) are the columns of S^T = K Q^T, computed 64 keys at a time with
// 16x16x32 matrix instructions.  With m the row's running reference,
//     x = S k_scale scale log2(e),  l += 2^(x - m),  O^T += V^T p^T,  p = 2^(x + e - M + 11)
// and out = O 2^(M - 11 - m) / l, where e is the exponent of the key's V
// scale: V enters as its codes, exact in FP16, and its scales ride on p, so
// that a block's scale is nothing to the rows that do not see the block.  m
// and M move only when a row's maximum (of x and of x + e) passes them by
// more than 4, so the accumulators are rarely multiplied.  l and O are FP32;
// p is rounded to FP16 for the second product, and l sums FP32 weights.  The
// largest p of a row is between 2^10 (M is a maximum rounded up to a whole
// number) and 2^15; FP16 holds 11 bits of those down to 2^-24 of the largest
// (an order finer than a BF16 output) and fewer down to 2^-35 of it.
//
// Layout.  S^T keeps a row's statistics in one column: 16 of a row's 64
// scores in one lane, the others in the lanes 16, 32 and 48 further.  The
// rows of the K operand are a permutation of the keys (row 4x + i of matrix
// t holds key 16x + 4t + i) chosen so that a lane ends up with 16
// consecutive keys, one block of the cache: one K scale and one V scale for
// all its scores, and its p are in place as the second product's operand,
// whose other side is one 16-byte load of V (16 keys of one channel).
// Nothing passes through LDS before the waves' results are joined.
//
// What bounds it: reading the cache.  64 sequences of up to 8192 tokens (8 KV
// heads of 128 channels, 673 MB) take 136 us, 4.9 TB/s; one of 131072 tokens, cut
// into 32 chunks per head, 58 us, 4.6 TB/s, where a large copy moves 4.9.
// Each wave has one 64-key tile of loads in flight (16 KB) while it computes
// another, 4 waves to a workgroup and two workgroups to a CU up to 128
// channels; 8 waves where there are few row tiles (figures in kv_plan.cpp).
// (Refilling two sets of tile registers as they are consumed, so that loads
// stay in flight longer, gained nothing at 64 channels and spilled at 128.)
// Short caches are bound by the chain of loads (length, page, block): 300
// tokens take 7.9 us, 24 windows of about 1000 keys with 25 rows each 12.7,
// twice what their bytes and about what their widening and exponentials
// take on a half-filled chip.
//
// Hidden keys: their scores are -inf, so their p are zero.  0 * NaN would
// still reach the sums, so where a partly hidden tile has NaN among its V
// codes, those that no row sees are replaced by zero, and a second product
// counts the others for the rows that see them.

#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention.h"
#include "attention_device.h"
#include "device_common.h"

namespace w8a16 {

namespace rows {

using namespace dev;

constexpr uint32_t kInFlight = 16;  // partial loads of a thread at a time in the join: each is a
                                    // round trip past the L2

// What a wave needs to know to load a tile.
struct TileAt {
    const uint8_t *k, *v;     // this lane's rows of the tile's K and V
    uint32_t ks, vs;          // scale bytes of the lane's block (0: no such page)
    bool ok;
};

// LDS of a workgroup.
template <int DP, int WAVES> struct RowsLds {
    static constexpr int SEG = DP % 128 || WAVES > 4 ? 64 : 128;    // channels joined at a time
    static constexpr int PART = 16 * (SEG + 4);
    float part[WAVES * PART];           // [wave][16][SEG + 4]
    f32x4_t stat[WAVES][16];            // sum reference, l, output reference
    float red[2 * 64 * WAVES];
    uint32_t last;
};

// Workgroup `group_id` of a launch of a.grid.  Either pass over a shared prefix
// leaves partial rows and no outputs.
template <class Q, int DP, int WAVES, class Args>
__device__ __forceinline__ void kv_rows(const Args &a, uint32_t group_id, RowsLds<DP, WAVES> &lds)
{
    auto &part = lds.part;
    auto &stat = lds.stat;
    auto &red = lds.red;
    auto &last = lds.last;
    constexpr bool PARTS = is_prefix<Args> || is_suffix<Args>;
    constexpr int QC = DP / 64;       // 64-channel groups of the first product
    constexpr int VT = DP / 16;       // 16-channel tiles of the second
    constexpr uint32_t THREADS = 64 * WAVES;
    constexpr int SEG = RowsLds<DP, WAVES>::SEG;
    static_assert(DP % SEG == 0, "the join's passes take whole output tiles");
    constexpr int NR = 16;            // rows
    constexpr int PART = RowsLds<DP, WAVES>::PART;
    static_assert(WAVES * PART >= (int)kKvMaxChunks * NR && WAVES * PART >= 4 * (int)THREADS, "LDS of the join");
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t col = lane & 15u, g = lane >> 4;
    const KvPool &pool = a.pool;

    // (sequence, KV head) pairs fastest and chunks slowest: were chunks
    // fastest, a power of two of them would put each chunk on its own XCD,
    // and ragged lengths leave the later chunks empty
    const uint32_t groups = sequences(a) * pool.heads;
    const uint32_t grp = group_id % groups, rest = group_id / groups;
    const uint32_t rtile = rest % a.row_tiles, chunk = rest / a.row_tiles;
    const uint32_t head = grp % pool.heads, b = grp / pool.heads;

    const uint32_t kx = col >> 2, kr = col & 3u;   // the lane's block and row of the K operand
    // The tile's four page numbers are read through the scalar cache (a
    // vector load would have to be waited for together with the tiles in
    // flight) and picked by lane.
    typedef const __attribute__((address_space(4))) int32_t *scalar_ptr;
    const scalar_ptr bt = (scalar_ptr)(uintptr_t)(a.seqs.block_table + (size_t)table_row(a, b) * a.seqs.bt_stride);
    // Blocks past `last_block` are read as that one; none of their keys is
    // visible.
    auto place = [&](uint32_t tile, uint32_t last_block) {
        uint32_t page[4];
        const uint32_t last_col = a.seqs.bt_width - 1u;
#pragma unroll
        for (uint32_t x = 0; x < 4; ++x) {
            const uint32_t c = pool.by_blocks.div(4u * tile + x < last_block ? 4u * tile + x : last_block);
            page[x] = (uint32_t)bt[c < last_col ? c : last_col];
        }
        auto pick = [&](uint32_t x, uint32_t &pg, uint32_t &slot) {
            const uint32_t lo = x & 1u ? page[1] : page[0], hi = x & 1u ? page[3] : page[2];
            const uint32_t blk = 4u * tile + x < last_block ? 4u * tile + x : last_block;
            const uint32_t c = pool.by_blocks.div(blk);
            pg = x & 2u ? hi : lo;
            slot = head * pool.blocks + blk - c * pool.blocks;
            const bool ok = pg < pool.pages && c <= last_col;
            pg = ok ? pg : 0u;
            return ok;
        };
        TileAt at;
        uint32_t pk, sk, pv, sv;
        pick(kx, pk, sk);
        at.ok = pick(g, pv, sv);
        at.k = pool.k + pk * pool.k_page + ((size_t)sk * 16u + kr) * pool.dim;
        at.v = pool.v + pv * pool.v_page + ((size_t)sv * pool.dim + col) * 16u;
        at.ks = pool.k_scale[pv * pool.ks_page + sv];
        at.vs = pool.v_scale[pv * pool.vs_page + sv];
        return at;
    };
    auto load = [&](const TileAt &at, u32x4_t (&k)[QC][4], u32x4_t (&v)[VT]) {
#pragma unroll
        for (int i = 0; i < QC; ++i) {
            // channels past the head meet queries of zero: read any of the row
            const uint32_t d = 64u * i + 16u * g;
            const uint8_t *p = at.k + (d < pool.dim ? d : 0u);
#pragma unroll
            for (int x = 0; x < 4; ++x)
                k[i][x] = *reinterpret_cast<const u32x4_t *>(p + (size_t)(4 * x) * pool.dim);
        }
#pragma unroll
        for (int x = 0; x < VT; ++x)
            v[x] = *reinterpret_cast<const u32x4_t *>(at.v + (16u * x < pool.dim ? 256u * x : 0u));
    };

    // Without a window the first chunk starts with key 0 whatever the
    // sequence's length: its first tiles are under way before the length is
    // known.  (Past the sequence's end the block table may hold anything:
    // what no page of the cache is reads as page 0.)
    // With sinks key 0 is the first wave's; behind a shared prefix the first
    // tile is its end's; the prefix's tiles are all known.
    u32x4_t k[QC][4], v[VT];
    TileAt at;
    bool early = chunk == 0 && !a.window;
    uint32_t early_tile = wave, early_last = ~0u;
    if constexpr (has_sinks<Args>)
        early = chunk == 0 && wave == 0;
    if constexpr (is_suffix<Args>)
        early_tile += a.shared / kKvTile;
    if constexpr (is_prefix<Args>) {
        early = true;
        early_tile += chunk * a.chunk_tiles;
        early_last = a.shared / 16u - 1u;
    }
    if (early) {
        at = place(early_tile, early_last);
        load(at, k, v);
    }

    RowTile t;
    const bool extra = chunk >= a.chunks;      // past the plan's workgroups
    if (!extent(a, b, t) && !extra)
        return;
    t.rows = t.count * a.group;
    t.row0 = rtile * NR;
    if (t.row0 >= t.rows || extra) {
        if (extra)
            fill_unowned<typename Q::elem>(a, group_id - a.grid, WAVES);
        return;
    }
    tile_range(a, NR, t);
    const TileList list(a, t);
    const uint32_t tiles = list.tiles;
    const uint32_t begin = chunk * a.chunk_tiles;
    if (begin >= tiles && chunk > 0 && !is_prefix<Args>)
        return;
    // the last chunk takes all that is left, should the caller's bound on
    // the lengths have been too small
    const uint32_t end = chunk + 1 == a.chunks || begin + a.chunk_tiles > tiles
                             ? tiles : begin + a.chunk_tiles;
    const bool alone = !PARTS && (a.chunks == 1 || tiles <= a.chunk_tiles);

    // queries: column col is row row0 + col; the lane's
    // channels of group i are 64 i + 16 g .. + 15 (8 for each of two products)
    u32x4_t q[QC][2];
    int32_t rlo, rhi;
    {
        const uint32_t row = t.row0 + col;
        row_range(a, t, row, rlo, rhi);
        const uint32_t tok = a.by_group.div(row), hq = head * a.group + row - tok * a.group;
        const typename Q::elem *src = reinterpret_cast<const typename Q::elem *>(a.q) +
                                      (int64_t)(t.first + tok) * a.q_token + (int64_t)hq * a.q_head;
#pragma unroll
        for (int i = 0; i < QC; ++i) {
            const uint32_t d = 64u * i + 16u * g;
            q[i][0] = q[i][1] = u32x4_t{0u, 0u, 0u, 0u};
            if (row < t.rows && d < pool.dim) {
                if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
                    q[i][0] = *reinterpret_cast<const u32x4_t *>(src + d);
                    q[i][1] = *reinterpret_cast<const u32x4_t *>(src + d + 8);
                } else {
                    const uint16_t *s16 = reinterpret_cast<const uint16_t *>(src + d);
#pragma unroll
                    for (int w = 0; w < 8; ++w)
                        q[i][w >> 2][w & 3] = (uint32_t)s16[2 * w] | ((uint32_t)s16[2 * w + 1] << 16);
                }
            }
        }
    }

    f32x4_t o[VT];
    RowRef m;
    float l = 0.f;
#pragma unroll
    for (int v = 0; v < VT; ++v)
        o[v] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    const int32_t sinks = sinks_of(a);
    auto before_sinks = [&](int32_t key) { return has_sinks<Args> && key < sinks; };
    auto compute = [&](uint32_t tile) {
        const int32_t key0 = (int32_t)(tile * kKvTile + 16u * g);   // the lane's first key
        const bool seen = key0 < t.hi && (key0 + 16 > t.lo || before_sinks(key0));   // some key of the block, by some row
        const float ksc = !seen ? 1.0f : (at.ok && at.ks - 1u < 254u ? pow2_byte(at.ks) * a.scale_log2
                                                                      : __builtin_nanf(""));
        const float e = (float)at.vs - 127.0f;     // (255 and 0, no scale: the codes become NaN)

        const bool masked = ((int32_t)(tile * kKvTile) < t.all_lo && !before_sinks((int32_t)(tile * kKvTile + kKvTile - 1))) ||
                            (int32_t)(tile * kKvTile + kKvTile) > t.all_hi;
        f32x4_t s[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            s[x] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < QC; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                s[x] = Q::mfma16(Q::widen(k[i][x].x, k[i][x].y), q[i][0], s[x]);
                s[x] = Q::mfma16(Q::widen(k[i][x].z, k[i][x].w), q[i][1], s[x]);
            }

        const bool bad = seen && (!at.ok || at.vs - 1u >= 254u);
        if (__ballot(bad)) {
            // a block without a V scale reads as NaN codes
            const uint32_t poison = bad ? 0x7f7f7f7fu : 0u;
#pragma unroll
            for (int x = 0; x < VT; ++x)
                v[x] |= poison;
        }
        uint32_t hit = 0;
        if (masked) {
            // (hidden numbers meet p of 0; only NaN would not vanish)
            uint32_t odd = 0;
#pragma unroll
            for (int x = 0; x < VT; ++x)
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    odd |= (v[x][w] & 0x7f7f7f7fu) + 0x01010101u;
            hit = __ballot((odd & 0x80808080u) != 0) != 0 ? 1u : 0u;
        }
        if (hit) {
            // codes of keys no row of the tile sees
            uint32_t any = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t keep = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int32_t key = key0 + 4 * w + j;
                    keep |= (key >= t.lo || before_sinks(key)) && key < t.hi ? 0xffu << (8 * j) : 0u;
                }
#pragma unroll
                for (int x = 0; x < VT; ++x) {
                    v[x][w] &= keep;
                    any |= nan_bytes(v[x][w]);
                }
            }
            hit = __ballot(any != 0) != 0 ? 1u : 0u;
        }

        if (masked) {
            const int32_t up = rhi - key0, low = rlo - key0;
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[x][i] = 4 * x + i < up ? s[x][i] : kNegInf;
            if (a.window || is_suffix<Args>)
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[x][i] = 4 * x + i >= low || (has_sinks<Args> && 4 * x + i < sinks - key0) ? s[x][i] : kNegInf;
        }
        float mx = kNegInf;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mx = fmaxf(mx, s[x][i]);
        mx *= ksc;
        if (__ballot(m.passed(mx, e))) {
            const RowRef was = m;
            float top = mx, top_out = mx + e;
#pragma unroll
            for (int off = 16; off <= 32; off <<= 1) {
                top = fmaxf(top, __shfl_xor(top, off, 64));
                top_out = fmaxf(top_out, __shfl_xor(top_out, off, 64));
            }
            m.move(top, top_out);
            l *= exp2_fast(was.sum - m.sum);
            const float f = exp2_fast(was.out - m.out);
#pragma unroll
            for (int x = 0; x < VT; ++x)
                o[x] *= f;
        }
        float shift = m.shift(e);
        if (fabsf(shift) > kFar) {
            shift = kNegInf;
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    l += s[x][i] == kNegInf ? 0.f : exp2_fast(fmaf(s[x][i], ksc, -m.sum));
        }
        const float mu = m.out - e;
        u32x4_t p[2];
        if (masked && __ballot(!(ksc > 0.f))) {
            // a NaN scale must not reach hidden keys, nor a factor of 0 their -inf
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[x][i] = s[x][i] == kNegInf ? 0.f : exp2_fast(fmaf(s[x][i], ksc, -mu));
        } else {
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[x][i] = exp2_fast(fmaf(s[x][i], ksc, -mu));
        }
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sum += s[x][i];
        l = fmaf(sum, exp2_fast(shift), l);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            p[u].x = f16_pair(s[2 * u][0], s[2 * u][1]);
            p[u].y = f16_pair(s[2 * u][2], s[2 * u][3]);
            p[u].z = f16_pair(s[2 * u + 1][0], s[2 * u + 1][1]);
            p[u].w = f16_pair(s[2 * u + 1][2], s[2 * u + 1][3]);
        }
        if (hit) {
            // NaN codes: counted for the rows that see them, then zeroed
#pragma unroll
            for (int x = 0; x < VT; ++x) {
                u32x4_t bad[2], seen[2];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t nb = nan_bytes(v[x][w]) >> 7;
                    v[x][w] &= ~(nb * 0xffu);
                    bad[w >> 1][2 * (w & 1)] = ((nb & 1u) | ((nb & 0x100u) << 8)) * 0x3c00u;
                    bad[w >> 1][2 * (w & 1) + 1] = (((nb >> 16) & 1u) | ((nb >> 8) & 0x10000u)) * 0x3c00u;
                }
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    const int32_t key = key0 + 2 * w;
                    seen[w >> 2][w & 3] =
                        ((key >= rlo || before_sinks(key)) && key < rhi ? 0x3c00u : 0u) |
                        ((key + 1 >= rlo || before_sinks(key + 1)) && key + 1 < rhi ? 0x3c000000u : 0u);
                }
                f32x4_t n = {0.f, 0.f, 0.f, 0.f};
                n = mfma16_f16(bad[0], seen[0], n);
                n = mfma16_f16(bad[1], seen[1], n);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[x][i] = n[i] > 0.f ? __builtin_nanf("") : o[x][i];
            }
        }
#pragma unroll
        for (int x = 0; x < VT; ++x) {
            o[x] = mfma16_f16(f16_from_fp8x8(v[x].x, v[x].y, 1.0f), p[0], o[x]);
            o[x] = mfma16_f16(f16_from_fp8x8(v[x].z, v[x].w, 1.0f), p[1], o[x]);
        }
    };

    // the wave's tiles: begin + wave, begin + wave + 4, ... below end; the
    // next tile's loads are in flight while one is computed
    uint32_t tile = begin + wave;
    if (tile < end) {
        const uint32_t last_block = t.kv_len > 0 ? (uint32_t)(t.kv_len - 1) / 16u : 0u;
        if (!early) {
            at = place(list.at(tile), last_block);
            load(at, k, v);
        }
        while (tile + WAVES < end) {
            u32x4_t kn[QC][4], vn[VT];
            const TileAt next = place(list.at(tile + WAVES), last_block);
            load(next, kn, vn);
            compute(list.at(tile));
            at = next;
#pragma unroll
            for (int i = 0; i < QC; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    k[i][x] = kn[i][x];
#pragma unroll
            for (int x = 0; x < VT; ++x)
                v[x] = vn[x];
            tile += WAVES;
        }
        compute(list.at(tile));
    }

    // join the waves: common references per row
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (g == 0)
        stat[wave][col] = f32x4_t{m.sum, l, m.out, 0.f};
    __syncthreads();
    const uint32_t n_rows = t.rows - t.row0 < (uint32_t)NR ? t.rows - t.row0 : (uint32_t)NR;
    const uint32_t dim4 = pool.dim / 4;
    // partial rows: [(b, head, rtile)][chunk][row][dim], then as many (sum
    // reference, l, output reference) quadruples
    const size_t tile_id = (size_t)grp * a.row_tiles + rtile;
    f32x4_t *const wo = reinterpret_cast<f32x4_t *>(a.ws) + tile_id * a.chunks * NR * dim4;
    f32x4_t *const wst = reinterpret_cast<f32x4_t *>(a.ws) + (size_t)a.grid * NR * dim4 +
                         tile_id * a.chunks * NR;
    float out_all = kUnset;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
        out_all = fmaxf(out_all, stat[w][col].z);
    const float wave_fac = exp2_fast(m.out - out_all);
    constexpr uint32_t TPR = THREADS / NR;       // threads per row
    const uint32_t tr = threadIdx.x / TPR, row = t.row0 + tr;
    RowRef mr;
    float lr = 0.f;
    f32x4_t st_row[WAVES];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        st_row[w] = stat[w][tr];
        mr.sum = fmaxf(mr.sum, st_row[w].x);
        mr.out = fmaxf(mr.out, st_row[w].z);
    }
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
        lr += st_row[w].y * exp2_fast(st_row[w].x - mr.sum);
    const uint32_t tok = a.by_group.div(row), hq = head * a.group + row - tok * a.group;
    const bool none = sees_nothing(a, t, row);
    const float inv = none ? 0.f : 1.0f / lr, unit = mr.out - mr.sum;
    typename Q::elem *const dst = reinterpret_cast<typename Q::elem *>(a.out) +
                                  (int64_t)(t.first + tok) * a.out_token + (int64_t)hq * a.out_head;
#pragma unroll
    for (int s0 = 0; s0 < DP; s0 += SEG) {
        if (s0)
            __syncthreads();
#pragma unroll
        for (int x = 0; x < SEG / 16; ++x)
            *reinterpret_cast<f32x4_t *>(&part[wave * PART + col * (SEG + 4) + 16 * x + 4 * g]) =
                o[s0 / 16 + x] * wave_fac;
        __syncthreads();
        if (tr >= n_rows)
            continue;
#pragma unroll
        for (uint32_t i = 0; i < SEG; i += 4 * TPR) {
            const uint32_t c = 4u * (threadIdx.x % TPR) + i;
            if (c >= (uint32_t)SEG || s0 + c >= pool.dim)
                continue;
            f32x4_t acc = *reinterpret_cast<const f32x4_t *>(&part[tr * (SEG + 4) + c]);
#pragma unroll
            for (int w = 1; w < WAVES; ++w)
                acc += *reinterpret_cast<const f32x4_t *>(&part[w * PART + tr * (SEG + 4) + c]);
            if (alone)
                store_row4(dst + s0 + c, acc * inv, unit);
            else if (PARTS)
                wo[((size_t)chunk * NR + tr) * dim4 + (s0 + c) / 4] = acc;
            else
                store_agent(wo + ((size_t)chunk * NR + tr) * dim4 + (s0 + c) / 4, acc);
        }
    }
    if (tr < n_rows && threadIdx.x % TPR == 0) {
        if (PARTS)
            wst[(size_t)chunk * NR + tr] = f32x4_t{mr.sum, lr, mr.out, 0.f};
        else if (!alone)
            store_agent(wst + (size_t)chunk * NR + tr, f32x4_t{mr.sum, lr, mr.out, 0.f});
        else if (a.lse)
            a.lse[(size_t)(t.first + tok) * a.q_heads + hq] =
                none ? kNegInf : (mr.sum + log2f(lr)) * 0.69314718055994531f;
    }
    if (alone || PARTS)
        return;

    // The last of the row tile's chunks to arrive joins them, in chunk
    // order.  The partial rows were written through to where any XCD's loads
    // past the L1 see them, and are complete before the arrival counts.
    uint32_t n = (tiles + a.chunk_tiles - 1) / a.chunk_tiles;
    n = n < a.chunks ? n : a.chunks;
    wait_vm<0>();
    __syncthreads();
    uint32_t *const counter = a.counters + tile_id * kKvCounterStride;
    const uint32_t tid = threadIdx.x;
    if (tid == 0)
        last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u == n;
    __syncthreads();
    if (!last)
        return;
    if (tid == 0)      // ready for the next call that uses this workspace
        __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // statistics: thread (row sr, every SG-th chunk from sg on)
    constexpr uint32_t SG = THREADS / NR, PER = kKvMaxChunks / SG;
    const uint32_t sr = tid % NR, sg = tid / NR;
    f32x4_t st[PER];
    float mj = kUnset, ex = kUnset;
#pragma unroll
    for (uint32_t i = 0; i < PER; ++i) {
        st[i] = f32x4_t{kUnset, 0.f, kUnset, 0.f};
        if (sr < n_rows && sg + i * SG < n)
            st[i] = load_agent(wst + (size_t)(sg + i * SG) * NR + sr);
    }
#pragma unroll
    for (uint32_t i = 0; i < PER; ++i) {
        mj = fmaxf(mj, st[i].x);
        ex = fmaxf(ex, st[i].z);
    }
    red[tid] = mj;
    red[THREADS + tid] = ex;
    __syncthreads();
    for (uint32_t k = 0; k < SG; ++k) {
        mj = fmaxf(mj, red[k * NR + sr]);
        ex = fmaxf(ex, red[THREADS + k * NR + sr]);
    }
    float lj = 0.f;
    float *const fac = part;      // [chunk][row]
#pragma unroll
    for (uint32_t i = 0; i < PER; ++i)
        if (sg + i * SG < n) {
            lj += exp2_fast(st[i].x - mj) * st[i].y;
            fac[(sg + i * SG) * NR + sr] = exp2_fast(st[i].z - ex);
        }
    __syncthreads();
    red[tid] = lj;
    if (sg == 0) {
        red[THREADS + sr] = mj;
        red[THREADS + NR + sr] = ex;
    }
    __syncthreads();
    if (tid < (uint32_t)NR) {
        lj = 0.f;
        for (uint32_t k = 0; k < SG; ++k)
            lj += red[k * NR + tid];
        red[THREADS + 2 * NR + tid] = lj;
    }
    __syncthreads();
    // outputs: four channels of one row per thread; where that leaves half
    // of the threads or more without any, they share the chunks
    const uint32_t items = n_rows * dim4;
    const uint32_t teams = items <= THREADS / 2 ? THREADS / items : 1u;
    for (uint32_t base = 0; base < items; base += THREADS) {
        const uint32_t team = teams > 1 ? tid / items : 0u, it = base + (teams > 1 ? tid - team * items : tid);
        const bool on = it < items && team < teams;
        const uint32_t jr = on ? it / dim4 : 0u, c4 = on ? it - jr * dim4 : 0u;
        f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
        if (on)
            for (uint32_t c = team; c < n; c += kInFlight * teams) {
                f32x4_t v[kInFlight];
#pragma unroll
                for (uint32_t u = 0; u < kInFlight; ++u)
                    if (c + u * teams < n)
                        v[u] = load_agent(wo + ((size_t)(c + u * teams) * NR + jr) * dim4 + c4);
#pragma unroll
                for (uint32_t u = 0; u < kInFlight; ++u)
                    if (c + u * teams < n)
                        acc += fac[(c + u * teams) * NR + jr] * v[u];
            }
        if (teams > 1) {
            __syncthreads();       // fac has been read
            f32x4_t *const sums = reinterpret_cast<f32x4_t *>(part);
            sums[tid] = acc;
            __syncthreads();
            for (uint32_t k = 1; on && team == 0 && k < teams; ++k)
                acc += sums[k * items + it];
        }
        if (!on || team)
            continue;
        const float mg = red[THREADS + jr], eg = red[THREADS + NR + jr], lg = red[THREADS + 2 * NR + jr];
        const uint32_t jtok = a.by_group.div(t.row0 + jr), jh = head * a.group + t.row0 + jr - jtok * a.group;
        const bool empty = sees_nothing(a, t, t.row0 + jr);
        const float inv_all = empty ? 0.f : 1.0f / lg;
        store_row4(reinterpret_cast<typename Q::elem *>(a.out) + (int64_t)(t.first + jtok) * a.out_token +
                       (int64_t)jh * a.out_head + 4 * c4, acc * inv_all, eg - mg);
        if (c4 == 0 && a.lse)
            a.lse[(size_t)(t.first + jtok) * a.q_heads + jh] =
                empty ? kNegInf : (mg + log2f(lg)) * 0.69314718055994531f;
    }
}

template <class Q, int DP, int WAVES, class Args>
__global__ __launch_bounds__(64 * WAVES, DP <= 128 && WAVES == 4 ? 2 : 1) void w8a16_kv_rows_kernel(Args a)
{
    __shared__ __attribute__((aligned(16))) RowsLds<DP, WAVES> lds;
    kv_rows<Q, DP, WAVES>(a, blockIdx.x, lds);
}

// Adds the chunks' partial results of the tile kernel, or of the two passes
// over a shared prefix: one wave per (row, KV head).  Its lanes are groups of
// dim / 4, four channels each, that take the chunks in turn; the groups' sums
// are added in group order.
constexpr uint32_t kJoinAhead = 4;

template <class E, class Args>
__global__ __launch_bounds__(256) void w8a16_kv_join_kernel(Args a, uint32_t tile_rows,
                                                            uint32_t rows_used, uint32_t rows_all,
                                                            uint32_t grid_rows)
{
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t idx = 4u * blockIdx.x + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (idx >= rows_all)
        return;
    const uint32_t r = idx % rows_used, id = idx / rows_used;   // id: ((b, head), rtile)
    const uint32_t rtile = id % a.row_tiles;
    const uint32_t head = id / a.row_tiles % a.pool.heads, b = id / a.row_tiles / a.pool.heads;
    RowTile t;
    if (!extent(a, b, t))
        return;
    t.rows = t.count * a.group;
    t.row0 = rtile * tile_rows;
    const uint32_t row = t.row0 + r;
    if (row >= t.rows)
        return;
    uint32_t n = 1;
    if (!is_suffix<Args> || a.chunks > 1) {     // (else known before the sequence's length)
        tile_range(a, tile_rows, t);
        const uint32_t tiles = TileList(a, t, true).tiles;
        if (tiles <= a.chunk_tiles && !is_suffix<Args>)
            return;      // one chunk: its workgroup has stored the row
        n = (tiles + a.chunk_tiles - 1) / a.chunk_tiles;
        n = n < a.chunks ? n : a.chunks;
    }
    const uint32_t own_chunks = n ? n : 1u;
    if constexpr (is_suffix<Args>)      // the prefix's after the row's own
        n = own_chunks + a.prefix_chunks;
    const uint32_t dim = a.pool.dim, per = dim / 4, groups = 64u / per;
    const size_t first = (size_t)id * a.chunks * tile_rows + r;
    const float *wo = a.ws + first * dim;
    const float *wst = a.ws + (size_t)grid_rows * dim + first * 4u;
    auto prefix_row = [&](uint32_t c) { return prefix_partial(a, head, t.first * a.group + row, c - own_chunks); };
    auto stat_of = [&](uint32_t c) {
        if constexpr (is_suffix<Args>)
            if (c >= own_chunks)
                return reinterpret_cast<const f32x4_t *>(a.prefix + a.prefix_rows * dim)[prefix_row(c)];
        return *reinterpret_cast<const f32x4_t *>(wst + (size_t)c * tile_rows * 4u);
    };
    auto part_of = [&](uint32_t c, uint32_t d) {
        if constexpr (is_suffix<Args>)
            if (c >= own_chunks)
                return *reinterpret_cast<const f32x4_t *>(a.prefix + prefix_row(c) * dim + d);
        return *reinterpret_cast<const f32x4_t *>(wo + (size_t)c * tile_rows * dim + d);
    };

    // The lanes' pieces of the first chunks are under way before the
    // statistics have come.
    const uint32_t grp = lane / per, d = lane % per * 4u;
    f32x4_t v[kJoinAhead];
    auto fetch = [&](uint32_t base, uint32_t stop) {
#pragma unroll
        for (uint32_t u = 0; u < kJoinAhead; ++u) {
            const uint32_t c = base + u * groups + grp;
            v[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            if (c < stop && grp < groups)
                v[u] = part_of(c, d);
        }
    };
    fetch(0, n < 64u ? n : 64u);
    // the row's largest references over all chunks
    float m = kUnset, ex = kUnset;
    f32x4_t st = {kUnset, 0.f, kUnset, 0.f};
    for (uint32_t c = lane; c < n; c += 64u) {
        const f32x4_t x = stat_of(c);
        st = c < 64u ? x : st;
        m = fmaxf(m, x.x);
        ex = fmaxf(ex, x.z);
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        m = fmaxf(m, __shfl_xor(m, off, 64));
        ex = fmaxf(ex, __shfl_xor(ex, off, 64));
    }
    f32x4_t own = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;       // this lane's chunks c = lane, lane + 64, ...
    for (uint32_t c0 = 0; c0 < n; c0 += 64u) {
        float fac = 0.f;
        if (c0 + lane < n) {
            if (c0)
                st = stat_of(c0 + lane);
            l += exp2_fast(st.x - m) * st.y;
            fac = exp2_fast(st.z - ex);
        }
        // all lanes: each lends its factor
        const uint32_t stop = n - c0 < 64u ? n - c0 : 64u;
        for (uint32_t base = 0; base < stop; base += kJoinAhead * groups) {
            if (c0 + base)
                fetch(c0 + base, c0 + stop);
#pragma unroll
            for (uint32_t u = 0; u < kJoinAhead; ++u) {
                const uint32_t c = base + u * groups + grp;
                const float f = __shfl(fac, (int)(c & 63u), 64);
                own += (c < stop ? f : 0.f) * v[u];
            }
        }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        l += __shfl_xor(l, off, 64);
    f32x4_t acc = own;
    for (uint32_t k = 1; k < groups; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[i] += __shfl(own[i], (int)((lane + k * per) & 63u), 64);
    if (lane >= per)
        return;
    const uint32_t tok = a.by_group.div(row), hq = head * a.group + row - tok * a.group;
    const bool none = sees_nothing(a, t, row);
    const float inv = none ? 0.f : 1.0f / l;
    store_row4(reinterpret_cast<E *>(a.out) + (int64_t)(t.first + tok) * a.out_token +
                   (int64_t)hq * a.out_head + d, acc * inv, ex - m);
    if (lane == 0 && a.lse)
        a.lse[(size_t)(t.first + tok) * a.q_heads + hq] =
            none ? kNegInf : (m + log2f(l)) * 0.69314718055994531f;
}

template <class Q, int DP, class Args>
hipError_t launch_dim(const Args &a, const w8a16_kv_plan_t &p, hipStream_t stream)
{
    const dim3 grid((uint32_t)kv_launch_groups(a, p.waves));
    if constexpr (DP <= 128) {
        if (p.waves == 8) {
            hipLaunchKernelGGL((w8a16_kv_rows_kernel<Q, DP, 8, Args>), grid, dim3(512), 0, stream, a);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((w8a16_kv_rows_kernel<Q, DP, 4, Args>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <class Q, class Args>
hipError_t launch_type(const Args &a, const w8a16_kv_plan_t &p, hipStream_t stream)
{
    switch ((a.pool.dim + 63u) / 64u) {
    case 1: return launch_dim<Q, 64>(a, p, stream);
    case 2: return launch_dim<Q, 128>(a, p, stream);
    case 3: return launch_dim<Q, 192>(a, p, stream);
    default: return launch_dim<Q, 256>(a, p, stream);
    }
}

}  // namespace rows

template <class Args>
hipError_t launch_kv_rows(const Args &a, const w8a16_kv_plan_t &p, uint32_t dtype, hipStream_t stream)
{
    return dtype == W8A16_BF16 ? rows::launch_type<dev::QueryBf16>(a, p, stream)
                               : rows::launch_type<dev::QueryF16>(a, p, stream);
}

template <class Args>
hipError_t launch_kv_join(const Args &a, const w8a16_kv_plan_t &p, uint32_t max_rows, uint32_t dtype,
                          hipStream_t stream)
{
    const uint32_t rows = 16u * p.row_blocks;
    const uint32_t used = max_rows < rows ? max_rows : rows;     // rows of a tile that exist
    const uint32_t all = p.grid / p.chunks * used;
    const dim3 grid((all + 3u) / 4u), block(256);
    if (dtype == W8A16_BF16)
        hipLaunchKernelGGL((rows::w8a16_kv_join_kernel<__bf16, Args>), grid, block, 0, stream, a, rows, used, all,
                           p.grid * rows);
    else
        hipLaunchKernelGGL((rows::w8a16_kv_join_kernel<_Float16, Args>), grid, block, 0, stream, a, rows, used,
                           all, p.grid * rows);
    return hipGetLastError();
}

}  // namespace w8a16
