// Launch plans of the cache attention.  Pure host code with no HIP
// dependency, like the GEMM planner.

#include <cstdio>
#include <cstring>

#include "plan.h"

namespace w8a16 {

namespace {

constexpr uint64_t kKeysPerTile = 64;
constexpr uint64_t kMinTiles = 4;      // of a chunk; 8 where a CU has one already
constexpr uint64_t kCutTiles = 10;     // that a cut has to spare, and one more

uint64_t div_up(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

}  // namespace

// Fills the derived fields of a plan whose kernel, row_blocks and
// chunk_tiles are set, or refuses it.
int kv_plan_finalize(uint32_t seqs, uint32_t max_new, uint32_t max_kv, uint32_t q_heads,
                     uint32_t kv_heads, uint32_t head_dim, uint32_t window, w8a16_kv_plan_t *p)
{
    const bool rows_ok = p->kernel == W8A16_KV_ROWS && p->row_blocks == 1 &&
                         (p->waves == 4 || (p->waves == 8 && head_dim <= 128));
    const bool tile_ok = p->kernel == W8A16_KV_TILE && p->row_blocks == 8 && p->waves == 4;
    if ((!rows_ok && !tile_ok) || p->chunk_tiles < 1)
        return fail(W8A16_ERR_BAD_PLAN, "w8a16_kv_attention: plan needs kernel W8A16_KV_ROWS with "
                                        "row_blocks 1 and 4 waves (or 8, of heads up to 128), or "
                                        "W8A16_KV_TILE with row_blocks 8 and 4 waves, and "
                                        "chunk_tiles of at least 1");
    // the tiles a row tile can see: all of the cache, or the window's and
    // those its rows' positions add
    const uint64_t tile_rows = 16ull * p->row_blocks, rows = (uint64_t)max_new * (q_heads / kv_heads);
    uint64_t keys = max_kv;
    if (window && (uint64_t)window + max_new < keys)
        keys = (uint64_t)window + max_new;
    uint64_t tiles = div_up(keys, kKeysPerTile) + (window ? 1 : 0);
    if (tiles < 1)
        tiles = 1;
    const uint64_t row_tiles = div_up(rows, tile_rows), chunks = div_up(tiles, p->chunk_tiles);
    const uint64_t grid = (uint64_t)seqs * kv_heads * row_tiles * chunks;
    if (grid * 64ull * p->waves > kMaxThreads)
        return fail(W8A16_ERR_SHAPE, "w8a16_kv_attention: too many workgroups (2^32 threads) for one call");
    p->row_tiles = (uint32_t)row_tiles;
    p->chunks = (uint32_t)chunks;
    p->grid = (uint32_t)grid;
    if (p->kernel == W8A16_KV_ROWS && chunks > kKvMaxChunks) {
        char buf[128];
        snprintf(buf, sizeof buf, "w8a16_kv_attention: %llu chunks, the row kernel joins at most %u",
                 (unsigned long long)chunks, kKvMaxChunks);
        return fail(W8A16_ERR_BAD_PLAN, buf);
    }
    p->workspace_bytes = chunks > 1 ? grid * tile_rows * (head_dim + 4) * 4 : 0;
    return W8A16_OK;
}

int make_kv_plan(uint32_t seqs, uint32_t max_new, uint32_t max_kv, uint32_t q_heads,
                 uint32_t kv_heads, uint32_t head_dim, uint32_t window, uint32_t cu_count,
                 w8a16_kv_plan_t *out)
{
    if (!out)
        return fail(W8A16_ERR_NULL_PTR, "w8a16_plan_kv_attention: null plan");
    if (!seqs || !max_new || !q_heads || !kv_heads || q_heads % kv_heads || head_dim < 16 ||
        head_dim > W8A16_KV_MAX_HEAD_DIM || head_dim % 16 || max_kv > (1u << 30)) {
        char buf[224];
        snprintf(buf, sizeof buf,
                 "w8a16_plan_kv_attention: seqs=%u max_new=%u max_kv=%u q_heads=%u kv_heads=%u "
                 "head_dim=%u is not a shape the attention takes",
                 seqs, max_new, max_kv, q_heads, kv_heads, head_dim);
        return fail(W8A16_ERR_SHAPE, buf);
    }
    const uint64_t cus = cu_count ? cu_count : kDefaultCUs;
    w8a16_kv_plan_t p;
    std::memset(&p, 0, sizeof p);
    const uint64_t rows = (uint64_t)max_new * (q_heads / kv_heads);
    // Up to 32 rows the row kernel, whose work grows with the rows; beyond,
    // the tile kernel takes as long for 33 rows as for 128, which pays where
    // the row tiles would wait for CUs.  8 KV heads of 128 channels, row
    // kernel and tile kernel, us:
    //   32 rows  64 sequences of 1000 tokens (1024 row tiles)  46  55
    //   48 rows  64 of 1000 (1536) 65  54;  32 of 2000 (768)  62  59
    //   64 rows  64 of 1000 (2048) 85  52;  32 of 2000 (1024) 81  58
    //            16 of 1000 (512)  19  32;  1 of 500 (32)      9  19
    //  128 rows  16 of 1000 (1024) 32  34;  8 of 4000 (512)   49  42
    // so up to 128 rows where there are at most 4 row tiles per CU (at that
    // end short caches gain by it and long ones lose).  Of 256 channels a CU
    // holds one workgroup: 32 rows of one sequence of 16000 34 and 39, 48
    // rows 40 and 40, 64 rows 44 and 41.
    const bool narrow = head_dim <= 128;
    const uint64_t row_grid = (uint64_t)seqs * kv_heads * div_up(rows, 16);
    p.kernel = rows <= 32 || (narrow && rows <= 128 && row_grid <= 4 * cus) ? W8A16_KV_ROWS : W8A16_KV_TILE;
    p.row_blocks = p.kernel == W8A16_KV_ROWS ? 1 : 8;
    p.waves = 4;
    p.chunk_tiles = 1u << 30;
    int st = kv_plan_finalize(seqs, max_new, max_kv, q_heads, kv_heads, head_dim, window, &p);
    if (st != W8A16_OK)
        return st;
    uint64_t tiles = div_up(window && (uint64_t)window + max_new < max_kv
                                ? (uint64_t)window + max_new : max_kv, kKeysPerTile) + (window ? 1 : 0);
    if (tiles < 1)
        tiles = 1;
    // Cut the keys while that leaves no more workgroups than run at once: two
    // per CU, one of 8 waves or of heads above 128 channels.  Eight waves
    // where the row tiles alone do not give every CU a workgroup: half as
    // many chunks to join (4 new tokens over 16000 20 us against 22 with four
    // waves, 32 sequences of 2000 29 either way), but slower where more
    // workgroups wait (48 sequences 49 against 43, 256 of 500 79 against 55).
    //
    // A cut has to spare more tiles of a workgroup's time than the join
    // costs.  Row kernel, us: 4 sequences of 768 tokens 9.7 uncut, 11.0 cut;
    // one of 900 11.2 and 10.9, of 1500 14.1 and 10.9; 16 sequences, which
    // can be cut in two, of 1200 14.1 and 15.8, of 2000 19.8 and 19.5.  Tile
    // kernel, whose partial rows grow with the workgroups: 128 new tokens
    // over 1500 45 and 27 (96 workgroups); 2 x 256 over 1024 32 and 39, over
    // 2048 56 and 42, 4 x 256 over 2048 of 64 channels 42 and 56, 2 x 512
    // over 4096 102 and 100 (512 workgroups).
    // A chunk has at least 4 tiles (2000 tokens: 8 tiles 11.9 us, 4 10.8; of
    // 256 channels 16.1 and 12.7; 64 new tokens 27 and 24), or 8 where it
    // would be a CU's second (128 new tokens over 4096: 34 and 36).
    if (p.kernel == W8A16_KV_ROWS && narrow && p.grid <= cus)
        p.waves = 8;
    const uint64_t slots = narrow && p.waves == 4 ? 2 * cus : cus;
    const uint64_t cuts = slots > p.grid ? slots / p.grid : 1;
    uint64_t per = div_up(tiles, cuts);
    const uint64_t once = cus > p.grid ? div_up(tiles, cus / p.grid) : tiles;    // a workgroup per CU
    const uint64_t least = once < 2 * kMinTiles ? once : 2 * kMinTiles;
    if (per < least)
        per = least;
    if (per < kMinTiles)
        per = kMinTiles;
    if (p.kernel == W8A16_KV_ROWS && per < div_up(tiles, kKvMaxChunks))
        per = div_up(tiles, kKvMaxChunks);
    const uint64_t join = p.kernel == W8A16_KV_ROWS ? kCutTiles : 4 + 12 * p.grid * div_up(tiles, per) / slots;
    if (per + join >= tiles)
        per = tiles;
    p.chunk_tiles = (uint32_t)per;
    st = kv_plan_finalize(seqs, max_new, max_kv, q_heads, kv_heads, head_dim, window, &p);
    if (st != W8A16_OK)
        return st;
    *out = p;
    return W8A16_OK;
}

}  // namespace w8a16

extern "C" int w8a16_plan_kv_attention(uint32_t seqs, uint32_t max_new, uint32_t max_kv,
                                       uint32_t q_heads, uint32_t kv_heads, uint32_t head_dim,
                                       uint32_t window, uint32_t cu_count, w8a16_kv_plan_t *out)
{
    return w8a16::make_kv_plan(seqs, max_new, max_kv, q_heads, kv_heads, head_dim, window, cu_count,
                               out);
}
