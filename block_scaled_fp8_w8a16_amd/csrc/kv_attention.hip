// Attention of a few rows (decode, drafts) over the paged FP8 cache.
//
// Mathematics.  For one KV head, the rows r = (new token, query head of the
// group) are the columns of S^T = K Q^T, computed 64 keys at a time with
// 16x16x32 matrix instructions.  With m the row's running reference,
//     p = 2^(S k_scale scale log2(e) - m),  l += p,  O^T += V^T p^T,
// and out = O / l.  m moves only when a row's maximum passes it by more than
// 2^8 (p stays below 256, in range of FP16), so the accumulators are
// rarely multiplied.  l and O are FP32; p is rounded to FP16 (11 bits, an
// order finer than a BF16 output) for the second product, and l sums the
// unrounded p.
//
// Layout.  S^T keeps a row's statistics in one column: 16 of a row's 64
// scores in one lane, the others in the lanes 16, 32 and 48 further.  The
// rows of the K operand are a permutation of the keys (row 4x + i of matrix
// t holds key 16x + 4t + i) chosen so that a lane ends up with 16
// consecutive keys, one block of the cache: one K scale and one V scale for
// all its scores, and its p are in place as the second product's operand,
// whose other side is one 16-byte load of V (16 keys of one channel).
// Nothing passes through LDS before the four waves' results are joined.
//
// V codes are widened to FP16 by 2^(e - E), e the block's scale exponent
// and E the largest seen by the wave, at most 2^7 above it: exact for blocks
// within 2^22 of the largest; O counts in units of 2^E.
//
// Hidden keys: their p is set to zero, and V codes that no row sees are
// replaced by zero, since 0 * NaN would reach the sums.  Where a NaN code is
// seen by some rows and hidden from others, a second product counts it for
// the rows that see it.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention.h"
#include "attention_device.h"
#include "device_common.h"

namespace w8a16 {

namespace {

using namespace dev;

constexpr int kWaves = 4;
constexpr float kLazy = 8.0f;       // log2 growth of a row's maximum that is left alone
constexpr int32_t kHeadroom = 7;    // V operands reach 448 * 2^7 < 65504
constexpr int32_t kNoExp = -100000;

// What a wave needs to know to load a tile.
struct TileAt {
    const uint8_t *k, *v;     // this lane's rows of the tile's K and V
    uint32_t ks, vs;          // scale bytes of the lane's block (0: no such page)
    bool ok;
};

template <class Q, int DP, int RB>
__global__ __launch_bounds__(256, 2) void w8a16_kv_rows_kernel(AttnArgs a)
{
    constexpr int QC = DP / 64;       // 64-channel groups of the first product
    constexpr int VT = DP / 16;       // 16-channel tiles of the second
    constexpr int SEG = DP < 128 ? DP : 128;
    __shared__ float part[kWaves][16][SEG + 4];
    __shared__ float stat[kWaves][RB * 16][2];
    __shared__ int32_t exps[kWaves];
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t col = lane & 15u, g = lane >> 4;
    const KvPool &pool = a.pool;

    uint32_t id = blockIdx.x;
    const uint32_t chunk = id % a.chunks;
    id /= a.chunks;
    const uint32_t rtile = id % a.row_tiles;
    id /= a.row_tiles;
    const uint32_t head = id % pool.heads, b = id / pool.heads;

    RowTile t;
    if (!seq_extent(a.seqs, b, t))
        return;
    t.rows = t.count * a.group;
    t.row0 = rtile * (16u * RB);
    if (t.row0 >= t.rows)
        return;
    tile_range(a, 16u * RB, t);
    const uint32_t tile0 = (uint32_t)t.lo / kKvTile;
    const uint32_t tiles = ((uint32_t)t.hi + kKvTile - 1) / kKvTile - tile0;
    const uint32_t begin = chunk * a.chunk_tiles;
    if (begin >= tiles && chunk > 0)
        return;
    // the last chunk takes all that is left, should the caller's bound on
    // the lengths have been too small
    const uint32_t end = chunk + 1 == a.chunks || begin + a.chunk_tiles > tiles
                             ? tiles : begin + a.chunk_tiles;
    const bool alone = a.chunks == 1 || tiles <= a.chunk_tiles;

    // queries: column col of matrix rb is row row0 + 16 rb + col; the lane's
    // channels of group i are 64 i + 16 g .. + 15 (8 for each of two products)
    u32x4_t q[RB][QC][2];
    int32_t rlo[RB], rhi[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const uint32_t row = t.row0 + 16u * rb + col;
        row_range(a, t, row, rlo[rb], rhi[rb]);
        const uint32_t tok = a.by_group.div(row), hq = head * a.group + row - tok * a.group;
        const typename Q::elem *src = reinterpret_cast<const typename Q::elem *>(a.q) +
                                      (int64_t)(t.first + tok) * a.q_token + (int64_t)hq * a.q_head;
#pragma unroll
        for (int i = 0; i < QC; ++i) {
            const uint32_t d = 64u * i + 16u * g;
            q[rb][i][0] = q[rb][i][1] = u32x4_t{0u, 0u, 0u, 0u};
            if (row < t.rows && d < pool.dim) {
                if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
                    q[rb][i][0] = *reinterpret_cast<const u32x4_t *>(src + d);
                    q[rb][i][1] = *reinterpret_cast<const u32x4_t *>(src + d + 8);
                } else {
                    const uint16_t *s16 = reinterpret_cast<const uint16_t *>(src + d);
#pragma unroll
                    for (int w = 0; w < 8; ++w)
                        q[rb][i][w >> 2][w & 3] = (uint32_t)s16[2 * w] | ((uint32_t)s16[2 * w + 1] << 16);
                }
            }
        }
    }

    f32x4_t o[RB][VT];
    float m[RB], l[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        m[rb] = kNegInf;
        l[rb] = 0.f;
#pragma unroll
        for (int v = 0; v < VT; ++v)
            o[rb][v] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    int32_t exp_ref = kNoExp;

    const uint32_t last_block = t.kv_len > 0 ? (uint32_t)(t.kv_len - 1) / 16u : 0u;
    const int32_t *bt = a.seqs.block_table + (size_t)b * a.seqs.bt_stride;
    const uint32_t kx = col >> 2, kr = col & 3u;   // the lane's block and row of the K operand

    // Page and place of block 4 * tile + x.  Blocks past the sequence are
    // read as its last one; none of their keys is visible.
    auto locate = [&](uint32_t tile, uint32_t x, uint32_t &page, uint32_t &slot) {
        uint32_t blk = 4u * tile + x;
        blk = blk < last_block ? blk : last_block;
        const uint32_t c = pool.by_blocks.div(blk);
        slot = head * pool.blocks + blk - c * pool.blocks;
        const bool in = c < a.seqs.bt_width;
        page = (uint32_t)bt[in ? c : 0u];
        page = in ? page : pool.pages;
    };
    auto place = [&](uint32_t tile) {
        TileAt at;
        uint32_t pk, sk, pv, sv;
        locate(tile, kx, pk, sk);
        locate(tile, g, pv, sv);
        at.ok = pv < pool.pages;
        pk = pk < pool.pages ? pk : 0u;
        pv = at.ok ? pv : 0u;
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

    auto compute = [&](uint32_t tile, const TileAt &at, const u32x4_t (&k)[QC][4], u32x4_t (&v)[VT]) {
        const int32_t key0 = (int32_t)(tile * kKvTile + 16u * g);   // the lane's first key
        const float ksc = at.ok && at.ks - 1u < 254u ? pow2_byte(at.ks) * a.scale_log2
                                                     : __builtin_nanf("");
        int32_t e = at.vs - 1u < 254u ? (int32_t)at.vs - 127 : kNoExp;
        if (key0 >= t.hi)
            e = kNoExp;     // no visible key in the block
        int32_t emax = e;
#pragma unroll
        for (int off = 16; off <= 32; off <<= 1) {
            const int32_t other = __shfl_xor(emax, off, 64);
            emax = emax > other ? emax : other;
        }
        emax = __builtin_amdgcn_readfirstlane(emax);
        float vrescale = 1.0f;
        if (emax > exp_ref + kHeadroom) {
            vrescale = exp_ref == kNoExp ? 0.0f : exp2_fast((float)(exp_ref - emax));
            exp_ref = emax;
        }
        const float vsc = e == kNoExp || e - exp_ref < -120 ? pow2_byte(7) : pow2_byte((uint32_t)(e - exp_ref + 127));

        const bool masked = (int32_t)(tile * kKvTile) < t.all_lo ||
                            (int32_t)(tile * kKvTile + kKvTile) > t.all_hi;
        f32x4_t s[RB][4];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                s[rb][x] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < QC; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const u32x4_t k0 = Q::widen(k[i][x].x, k[i][x].y), k1 = Q::widen(k[i][x].z, k[i][x].w);
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) {
                    s[rb][x] = Q::mfma16(k0, q[rb][i][0], s[rb][x]);
                    s[rb][x] = Q::mfma16(k1, q[rb][i][1], s[rb][x]);
                }
            }

        if (__ballot(!at.ok || at.vs - 1u >= 254u)) {
            // a block without a V scale reads as NaN codes
            const uint32_t poison = !at.ok || at.vs - 1u >= 254u ? 0x7f7f7f7fu : 0u;
#pragma unroll
            for (int x = 0; x < VT; ++x)
                v[x] |= poison;
        }
        uint32_t hit = 0;
        if (masked) {
            // codes of keys no row of the tile sees
            uint32_t any = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t keep = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int32_t key = key0 + 4 * w + j;
                    keep |= key >= t.lo && key < t.hi ? 0xffu << (8 * j) : 0u;
                }
#pragma unroll
                for (int x = 0; x < VT; ++x) {
                    v[x][w] &= keep;
                    any |= nan_bytes(v[x][w]);
                }
            }
            hit = __ballot(any != 0) != 0 ? 1u : 0u;
        }

        u32x4_t p[RB][2], seen[RB][2];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            if (masked) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int32_t key = key0 + 4 * x + i;
                        s[rb][x][i] = key >= rlo[rb] && key < rhi[rb] ? s[rb][x][i] : kNegInf;
                    }
            }
            float mx = kNegInf;
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mx = fmaxf(mx, s[rb][x][i]);
            mx *= ksc;
            mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
            mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
            float alpha = vrescale;
            if (__ballot(mx > m[rb] + kLazy || vrescale != 1.0f)) {
                const float mn = mx > m[rb] + kLazy ? mx : m[rb];
                const float grow = m[rb] == kNegInf ? 0.0f : exp2_fast(m[rb] - mn);
                l[rb] *= grow;
                alpha *= grow;
                m[rb] = mn;
#pragma unroll
                for (int x = 0; x < VT; ++x)
                    o[rb][x] *= alpha;
            }
            const float mu = m[rb] == kNegInf ? 0.0f : m[rb];
            float sum = 0.f;
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float e2 = exp2_fast(fmaf(s[rb][x][i], ksc, -mu));
                    if (masked)   // a NaN scale must not reach hidden keys
                        e2 = s[rb][x][i] == kNegInf ? 0.f : e2;
                    s[rb][x][i] = e2;
                    sum += e2;
                }
            l[rb] += sum;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                p[rb][u].x = f16_pair(s[rb][2 * u][0], s[rb][2 * u][1]);
                p[rb][u].y = f16_pair(s[rb][2 * u][2], s[rb][2 * u][3]);
                p[rb][u].z = f16_pair(s[rb][2 * u + 1][0], s[rb][2 * u + 1][1]);
                p[rb][u].w = f16_pair(s[rb][2 * u + 1][2], s[rb][2 * u + 1][3]);
            }
            if (hit) {
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    const int32_t key = key0 + 2 * w;
                    seen[rb][w >> 2][w & 3] = (key >= rlo[rb] && key < rhi[rb] ? 0x3c00u : 0u) |
                                              (key + 1 >= rlo[rb] && key + 1 < rhi[rb] ? 0x3c000000u : 0u);
                }
            }
        }
#pragma unroll
        for (int x = 0; x < VT; ++x) {
            if (hit) {
                // NaN codes: counted for the rows that see them, then zeroed
                u32x4_t bad[2];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t nb = nan_bytes(v[x][w]) >> 7;
                    v[x][w] &= ~(nb * 0xffu);
                    bad[w >> 1][2 * (w & 1)] = ((nb & 1u) | ((nb & 0x100u) << 8)) * 0x3c00u;
                    bad[w >> 1][2 * (w & 1) + 1] = (((nb >> 16) & 1u) | ((nb >> 8) & 0x10000u)) * 0x3c00u;
                }
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) {
                    f32x4_t n = {0.f, 0.f, 0.f, 0.f};
                    n = mfma16_f16(bad[0], seen[rb][0], n);
                    n = mfma16_f16(bad[1], seen[rb][1], n);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[rb][x][i] = n[i] > 0.f ? __builtin_nanf("") : o[rb][x][i];
                }
            }
            const u32x4_t v0 = f16_from_fp8x8(v[x].x, v[x].y, vsc), v1 = f16_from_fp8x8(v[x].z, v[x].w, vsc);
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                o[rb][x] = mfma16_f16(v0, p[rb][0], o[rb][x]);
                o[rb][x] = mfma16_f16(v1, p[rb][1], o[rb][x]);
            }
        }
    };

    // the wave's tiles: begin + wave, begin + wave + 4, ... below end; the
    // next tile's loads are in flight while one is computed
    uint32_t tile = begin + wave;
    if (tile < end) {
        u32x4_t k[QC][4], v[VT];
        TileAt at = place(tile0 + tile);
        load(at, k, v);
        while (tile + kWaves < end) {
            u32x4_t kn[QC][4], vn[VT];
            const TileAt next = place(tile0 + tile + kWaves);
            load(next, kn, vn);
            compute(tile0 + tile, at, k, v);
            at = next;
#pragma unroll
            for (int i = 0; i < QC; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    k[i][x] = kn[i][x];
#pragma unroll
            for (int x = 0; x < VT; ++x)
                v[x] = vn[x];
            tile += kWaves;
        }
        compute(tile0 + tile, at, k, v);
    }

    // join the waves: a common reference per row and a common exponent
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        l[rb] += __shfl_xor(l[rb], 16, 64);
        l[rb] += __shfl_xor(l[rb], 32, 64);
        if (g == 0) {
            stat[wave][rb * 16 + col][0] = m[rb];
            stat[wave][rb * 16 + col][1] = l[rb];
        }
    }
    if (lane == 0)
        exps[wave] = exp_ref;
    __syncthreads();
    int32_t exp_all = exps[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
        exp_all = exp_all > exps[w] ? exp_all : exps[w];
    const float efac = exp_ref == kNoExp ? 0.f : exp2_fast((float)(exp_ref - exp_all));
    const size_t slot = ((size_t)blockIdx.x) * (16u * RB);    // partial rows of this workgroup
    float *wo = a.ws + slot * pool.dim;
    float *wst = a.ws + (size_t)gridDim.x * (16u * RB) * pool.dim + slot * 4u;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        float mall = kNegInf;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            mall = fmaxf(mall, stat[w][rb * 16 + col][0]);
        const float fac = m[rb] == kNegInf ? 0.f : efac * exp2_fast(m[rb] - mall);
#pragma unroll
        for (int s0 = 0; s0 < DP; s0 += SEG) {
            __syncthreads();
            // a wave that saw no key of the row (m = -inf) adds zeros
#pragma unroll
            for (int x = 0; x < SEG / 16; ++x)
                *reinterpret_cast<f32x4_t *>(&part[wave][col][16 * x + 4 * g]) =
                    o[rb][s0 / 16 + x] * fac;
            __syncthreads();
            const uint32_t r = threadIdx.x >> 4, row = t.row0 + 16u * rb + r;
            float mr = kNegInf, lr = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                mr = fmaxf(mr, stat[w][rb * 16 + r][0]);
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                lr += stat[w][rb * 16 + r][1] *     // m = -inf: l is 0, or NaN
                      (stat[w][rb * 16 + r][0] == kNegInf ? 1.f : exp2_fast(stat[w][rb * 16 + r][0] - mr));
            if (row >= t.rows)
                continue;
            const uint32_t tok = a.by_group.div(row), hq = head * a.group + row - tok * a.group;
            const uint32_t c0 = (threadIdx.x & 15u) * (SEG / 16);
            if (s0 + c0 < pool.dim) {
                float acc[SEG / 16];
#pragma unroll
                for (int i = 0; i < SEG / 16; ++i) {
                    acc[i] = part[0][r][c0 + i];
#pragma unroll
                    for (int w = 1; w < kWaves; ++w)
                        acc[i] += part[w][r][c0 + i];
                }
                if (alone) {
                    // O counts in 2^exp_all; a row that sees nothing is zero
                    const float unit = exp_all == kNoExp ? 0.f : ldexpf(1.0f, exp_all);
                    const float inv = mr == kNegInf && lr == 0.f ? 0.f : 1.0f / lr;
                    typename Q::elem *dst = reinterpret_cast<typename Q::elem *>(a.out) +
                        (int64_t)(t.first + tok) * a.out_token + (int64_t)hq * a.out_head + s0 + c0;
#pragma unroll
                    for (int i = 0; i < SEG / 16; ++i)
                        dst[i] = static_cast<typename Q::elem>(acc[i] * inv * unit);
                } else {
                    float *dst = wo + (size_t)(16 * rb + r) * pool.dim + s0 + c0;
#pragma unroll
                    for (int i = 0; i < SEG / 16; ++i)
                        dst[i] = acc[i];
                }
            }
            if (s0 == 0 && (threadIdx.x & 15u) == 0) {
                if (!alone) {
                    wst[(16 * rb + r) * 4 + 0] = mr;
                    wst[(16 * rb + r) * 4 + 1] = lr;
                    wst[(16 * rb + r) * 4 + 2] = (float)exp_all;
                } else if (a.lse) {
                    a.lse[(size_t)(t.first + tok) * a.q_heads + hq] =
                        mr == kNegInf && lr == 0.f ? kNegInf : (mr + log2f(lr)) * 0.69314718055994531f;
                }
            }
        }
    }
}

// Adds the chunks' partial results of one row, in chunk order: one wave per
// (row, KV head).
template <class E>
__global__ __launch_bounds__(256) void w8a16_kv_join_kernel(AttnArgs a, uint32_t tile_rows,
                                                            uint32_t grid_rows, uint32_t total)
{
    const uint32_t unit = blockIdx.x * 4u + (threadIdx.x >> 6), lane = threadIdx.x & 63u;
    if (unit >= total)
        return;
    const uint32_t r = unit % tile_rows;
    uint32_t id = unit / tile_rows;       // ((b * heads) + head) * row_tiles + rtile
    const uint32_t rtile = id % a.row_tiles;
    const uint32_t head = id / a.row_tiles % a.pool.heads, b = id / a.row_tiles / a.pool.heads;
    RowTile t;
    if (!seq_extent(a.seqs, b, t))
        return;
    t.rows = t.count * a.group;
    t.row0 = rtile * tile_rows;
    const uint32_t row = t.row0 + r;
    if (row >= t.rows)
        return;
    tile_range(a, tile_rows, t);
    const uint32_t tiles = ((uint32_t)t.hi + kKvTile - 1) / kKvTile - (uint32_t)t.lo / kKvTile;
    if (tiles <= a.chunk_tiles)
        return;      // one chunk: its workgroup has stored the row
    uint32_t n = (tiles + a.chunk_tiles - 1) / a.chunk_tiles;
    n = n < a.chunks ? n : a.chunks;
    const uint32_t dim = a.pool.dim;
    const float *wo = a.ws + ((size_t)id * a.chunks * tile_rows + r) * dim;
    const float *wst = a.ws + (size_t)grid_rows * dim + ((size_t)id * a.chunks * tile_rows + r) * 4u;
    float m = kNegInf, ex = (float)kNoExp;
    for (uint32_t c = 0; c < n; ++c) {
        m = fmaxf(m, wst[(size_t)c * tile_rows * 4u]);
        ex = fmaxf(ex, wst[(size_t)c * tile_rows * 4u + 2]);
    }
    float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (uint32_t c = 0; c < n; ++c) {
        const float *st = wst + (size_t)c * tile_rows * 4u;
        const float f = st[0] == kNegInf ? 1.f : exp2_fast(st[0] - m);   // -inf: l is 0, or NaN
        l += f * st[1];
        const float fe = f * exp2_fast(st[2] - ex);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t d = lane + 64u * i;
            if (d < dim)
                acc[i] += fe * wo[(size_t)c * tile_rows * dim + d];
        }
    }
    const uint32_t tok = a.by_group.div(row), hq = head * a.group + row - tok * a.group;
    const bool none = m == kNegInf && l == 0.f;
    const float inv = none ? 0.f : 1.0f / l, unit_e = none ? 0.f : ldexpf(1.0f, (int)ex);
    E *dst = reinterpret_cast<E *>(a.out) + (int64_t)(t.first + tok) * a.out_token + (int64_t)hq * a.out_head;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t d = lane + 64u * i;
        if (d < dim)
            dst[d] = static_cast<E>(acc[i] * inv * unit_e);
    }
    if (lane == 0 && a.lse)
        a.lse[(size_t)(t.first + tok) * a.q_heads + hq] =
            none ? kNegInf : (m + log2f(l)) * 0.69314718055994531f;
}

template <class Q, int DP>
hipError_t launch_dim(const AttnArgs &a, const w8a16_kv_plan_t &p, hipStream_t stream)
{
    const dim3 grid(p.grid), block(256);
    if (p.row_blocks == 1)
        hipLaunchKernelGGL((w8a16_kv_rows_kernel<Q, DP, 1>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((w8a16_kv_rows_kernel<Q, DP, 2>), grid, block, 0, stream, a);
    return hipGetLastError();
}

template <class Q>
hipError_t launch_type(const AttnArgs &a, const w8a16_kv_plan_t &p, hipStream_t stream)
{
    switch ((a.pool.dim + 63u) / 64u) {
    case 1: return launch_dim<Q, 64>(a, p, stream);
    case 2: return launch_dim<Q, 128>(a, p, stream);
    case 3: return launch_dim<Q, 192>(a, p, stream);
    default: return launch_dim<Q, 256>(a, p, stream);
    }
}

}  // namespace

hipError_t launch_kv_rows(const AttnArgs &a, const w8a16_kv_plan_t &p, uint32_t dtype,
                          hipStream_t stream)
{
    return dtype == W8A16_BF16 ? launch_type<QueryBf16>(a, p, stream)
                               : launch_type<QueryF16>(a, p, stream);
}

hipError_t launch_kv_join(const AttnArgs &a, const w8a16_kv_plan_t &p, uint32_t dtype,
                          hipStream_t stream)
{
    const uint32_t rows = 16u * p.row_blocks, total = p.grid / p.chunks * rows;
    const dim3 grid((total + 3u) / 4u), block(256);
    if (dtype == W8A16_BF16)
        hipLaunchKernelGGL(w8a16_kv_join_kernel<__bf16>, grid, block, 0, stream, a, rows, p.grid * rows, total);
    else
        hipLaunchKernelGGL(w8a16_kv_join_kernel<_Float16>, grid, block, 0, stream, a, rows, p.grid * rows, total);
    return hipGetLastError();
}

}  // namespace w8a16
