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

// The tiles a row tile can see: all of the cache, or the window's, those its
// rows' positions add, and the sinks'; at least one.  (Without sinks the
// positions of all rows count, which is more than enough.)
uint64_t tiles_of(uint32_t max_new, uint32_t max_kv, uint32_t window, uint32_t sinks, uint64_t tile_tokens)
{
    uint64_t keys = max_kv;
    const uint64_t span = window + (sinks && tile_tokens < max_new ? tile_tokens : (uint64_t)max_new);
    if (window && span < keys)
        keys = span;
    uint64_t tiles = div_up(keys, kKeysPerTile) + (window ? 1 : 0);
    if (window && sinks) {
        tiles += div_up(sinks, kKeysPerTile);
        const uint64_t all = div_up(max_kv, kKeysPerTile);
        tiles = tiles < all ? tiles : all;
    }
    return tiles < 1 ? 1 : tiles;
}

const char *const kTooMany = "w8a16_kv_attention: too many workgroups (2^32 threads) for one call";

// Whether the launch that joins a plan's partial rows fits, a wave per row
// that exists (of at most `rows` of a sequence) and KV head.
bool join_fits(const w8a16_kv_plan_t &p, uint64_t rows)
{
    const uint64_t tile = 16ull * p.row_blocks, all = (uint64_t)(p.grid / p.chunks) * (rows < tile ? rows : tile);
    return div_up(all, 4) * 256 <= kMaxThreads;
}

}  // namespace

// Fills the derived fields of a plan whose kernel, row_blocks and
// chunk_tiles are set, or refuses it.
int kv_plan_finalize(uint32_t seqs, uint32_t max_new, uint32_t max_kv, uint32_t q_heads,
                     uint32_t kv_heads, uint32_t head_dim, uint32_t window, w8a16_kv_plan_t *p,
                     uint32_t sinks)
{
    const bool rows_ok = p->kernel == W8A16_KV_ROWS && p->row_blocks == 1 &&
                         (p->waves == 4 || (p->waves == 8 && head_dim <= 128));
    const bool tile_ok = p->kernel == W8A16_KV_TILE && p->row_blocks == 8 && p->waves == 4;
    if ((!rows_ok && !tile_ok) || p->chunk_tiles < 1)
        return fail(W8A16_ERR_BAD_PLAN, "w8a16_kv_attention: plan needs kernel W8A16_KV_ROWS with "
                                        "row_blocks 1 and 4 waves (or 8, of heads up to 128), or "
                                        "W8A16_KV_TILE with row_blocks 8 and 4 waves, and "
                                        "chunk_tiles of at least 1");
    const uint64_t tile_rows = 16ull * p->row_blocks, rows = (uint64_t)max_new * (q_heads / kv_heads);
    const uint64_t tiles = tiles_of(max_new, max_kv, window, sinks, tile_rows / (q_heads / kv_heads) + 2);
    const uint64_t row_tiles = div_up(rows, tile_rows), chunks = div_up(tiles, p->chunk_tiles);
    const uint64_t grid = (uint64_t)seqs * kv_heads * row_tiles * chunks;
    if (grid * 64ull * p->waves > kMaxThreads)
        return fail(W8A16_ERR_SHAPE, kTooMany);
    p->row_tiles = (uint32_t)row_tiles;
    p->chunks = (uint32_t)chunks;
    p->grid = (uint32_t)grid;
    if (p->kernel == W8A16_KV_ROWS && chunks > kKvMaxChunks) {
        char buf[128];
        snprintf(buf, sizeof buf, "w8a16_kv_attention: %llu chunks, the row kernel joins at most %u",
                 (unsigned long long)chunks, kKvMaxChunks);
        return fail(W8A16_ERR_BAD_PLAN, buf);
    }
    if (p->kernel == W8A16_KV_TILE && chunks > 1 && !join_fits(*p, rows))
        return fail(W8A16_ERR_SHAPE, kTooMany);
    p->workspace_bytes = chunks > 1 ? grid * tile_rows * (head_dim + 4) * 4 : 0;
    return W8A16_OK;
}

int make_kv_plan(uint32_t seqs, uint32_t max_new, uint32_t max_kv, uint32_t q_heads,
                 uint32_t kv_heads, uint32_t head_dim, uint32_t window, uint32_t cu_count,
                 w8a16_kv_plan_t *out, uint32_t sinks)
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
    int st = kv_plan_finalize(seqs, max_new, max_kv, q_heads, kv_heads, head_dim, window, &p, sinks);
    if (st != W8A16_OK)
        return st;
    const uint64_t tiles = tiles_of(max_new, max_kv, window, sinks, 16ull * p.row_blocks / (q_heads / kv_heads) + 2);
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
    st = kv_plan_finalize(seqs, max_new, max_kv, q_heads, kv_heads, head_dim, window, &p, sinks);
    if (st != W8A16_OK)
        return st;
    *out = p;
    return W8A16_OK;
}

namespace {

// A join takes both passes' chunks of a row tile.
constexpr uint64_t kMaxPassChunks = kKvMaxChunks / 2;

// A pass's plan over `keys` keys, with room for its partial rows: the given
// kernel and chunks.  joined: the join goes by its rows (the own keys' pass).
int pass_plan(uint32_t seqs, uint32_t max_new, uint32_t keys, uint32_t q_heads, uint32_t kv_heads,
              uint32_t head_dim, bool joined, w8a16_kv_plan_t *p)
{
    const int st = kv_plan_finalize(seqs, max_new, keys, q_heads, kv_heads, head_dim, 0, p);
    if (st != W8A16_OK)
        return st;
    if (p->chunks > kMaxPassChunks || p->waves != 4)
        return fail(W8A16_ERR_BAD_PLAN, "w8a16_kv_attention: behind a shared part a plan has 4 waves and at "
                                        "most 64 chunks");
    if (joined && !join_fits(*p, (uint64_t)max_new * (q_heads / kv_heads)))
        return fail(W8A16_ERR_SHAPE, kTooMany);
    p->workspace_bytes = (uint64_t)p->grid * 16 * p->row_blocks * (head_dim + 4) * 4;
    return W8A16_OK;
}

w8a16_kv_plan_t chunked(uint32_t kernel, uint64_t chunk_tiles)
{
    w8a16_kv_plan_t p;
    std::memset(&p, 0, sizeof p);
    p.kernel = kernel;
    p.row_blocks = kernel == W8A16_KV_ROWS ? 1 : 8;
    p.waves = 4;
    p.chunk_tiles = (uint32_t)chunk_tiles;
    return p;
}

// Times of the attention over caches with a shared part, in us, to choose
// between one pass and two and between their chunks.  Fitted to some 300
// times of 8 KV heads of 128 channels, 2 to 128 sequences of 1 to 250 new
// tokens behind 512 to 30016 shared ones; most agree within 10 %.  One pass
// and two, and what is chosen, 32 query heads, one new token:
//     2 sequences of  100 own tokens behind   512    8.8  10.1  one
//     2 of  100 behind  8192   13.1  13.6  two;     64 channels   9.8  10.5  two
//     6 of  333 behind  1984   12.0  11.8  two;     64 channels   9.7  10.2  two
//    16 of  400 behind  1984   16.5  12.3  two;     64 channels  11.4  10.2  two
//    64 of  700 behind   512   22.0  25.7  one;    behind 8192   89.5  38.3  two
//   128 of 2000 behind   512   96    115   one;    behind 30016  606   158   two
// and 24 of 4 new tokens and 101 own behind 1984 17.5 and 22.8 (one), behind
// 8192 46.0 and 36.0 (two; 64 channels 26.8 and 28.6, two, the farthest off).
struct Cost {
    double cus, slots, size;       // size: of a tile against 128 channels' (above them a CU holds one
                                   // workgroup, and its loads wait more)
    Cost(uint32_t cu_count, uint32_t head_dim)
        : cus(cu_count), slots(head_dim <= 128 ? 2.0 * cu_count : cu_count),
          size(head_dim / 128.0 * (head_dim <= 128 ? 1.0 : 1.15))
    {
    }
    // A CU's time for a tile of keys and a row tile: as many as it runs at
    // once share it.
    double tile(uint32_t kernel) const { return (kernel == W8A16_KV_ROWS ? 0.3 : 1.15) * size; }
    // A workgroup's time for one where it has the CU for itself.
    double alone(uint32_t kernel) const { return (kernel == W8A16_KV_ROWS ? 0.3 : 1.25) * size; }
    // The CU with the most workgroups of n.
    double most(double n) const { return n <= cus ? 1.0 : (double)div_up((uint64_t)n, (uint64_t)cus); }
    // Reading n tiles of keys from HBM.
    double read(double n) const { return 0.85 * size * n / cus; }
    // Partial rows written and read.
    double partial(double rows, uint32_t dim) const { return 2.0 * rows * (dim + 4) * 4 / 4.0e6; }
};

// Shared tiles come from the caches, own ones from HBM.
double one_pass(const Cost &c, const w8a16_kv_plan_t &p, uint64_t shared_tiles, uint64_t own_tiles, uint32_t dim)
{
    const double tile = c.tile(p.kernel), fetch = 0.85 * c.size / p.row_tiles;
    const double all = (double)(shared_tiles + own_tiles);
    const double mean = (shared_tiles * tile + own_tiles * (tile > fetch ? tile : fetch)) / all;
    const double rows = p.chunks > 1 ? (double)p.grid * 16 * p.row_blocks : 0;
    return 8.0 + (p.chunks > 1 ? 4.0 : 0.0) + c.most(p.grid) * (p.chunks > 1 ? p.chunk_tiles : all) * mean +
           (p.kernel == W8A16_KV_TILE ? 2.0 + c.partial(rows, dim) : 0.0);
}

// The prefix's products run while the own keys are read.
double two_passes(const Cost &c, const w8a16_kv_plan_t &p, const w8a16_kv_plan_t &o, uint64_t own_tiles,
                  uint64_t rows, uint32_t kv_heads, uint32_t dim)
{
    const double own_tile = c.tile(o.kernel) * o.grid / o.chunks * own_tiles / c.cus;
    const double read = c.read((double)o.grid / o.chunks / o.row_tiles * own_tiles);
    const double chunk = c.alone(p.kernel) * p.chunk_tiles;
    double busy = c.most(p.grid) * p.chunk_tiles * c.tile(p.kernel) + own_tile;
    busy = busy > read ? busy : read;
    busy = busy > chunk ? busy : chunk;
    const double rounds = (double)div_up((uint64_t)p.grid + o.grid, (uint64_t)c.slots);
    return 11.5 + (dim <= 128 ? 3.0 : 8.0) * (rounds - 1.0) + busy +
           c.partial((double)rows * kv_heads * (p.chunks + o.chunks), dim);
}

}  // namespace

int make_kv_shared_plans(uint32_t seqs, uint32_t tokens, uint32_t max_new, uint32_t max_kv,
                         uint32_t shared, uint32_t q_heads, uint32_t kv_heads, uint32_t head_dim,
                         uint32_t cu_count, const w8a16_kv_plan_t *given, w8a16_kv_plan_t *prefix,
                         w8a16_kv_plan_t *suffix)
{
    std::memset(prefix, 0, sizeof *prefix);
    w8a16_kv_plan_t whole;
    int st = make_kv_plan(seqs, max_new, max_kv, q_heads, kv_heads, head_dim, 0, cu_count, &whole);
    if (st != W8A16_OK)
        return st;
    *suffix = whole;
    if (!shared || (seqs < 2 && !given))
        return W8A16_OK;
    // the own keys' pass: they start in the tile that the shared ones end in
    const uint32_t before = shared / (uint32_t)kKeysPerTile * (uint32_t)kKeysPerTile;
    const uint32_t own = max_kv > before ? max_kv - before : 1u;
    const uint64_t own_tiles = div_up(own, kKeysPerTile), shared_tiles = div_up(shared, kKeysPerTile);
    w8a16_kv_plan_t o;
    if (given) {
        o = *given;
    } else {
        st = make_kv_plan(seqs, max_new, own, q_heads, kv_heads, head_dim, 0, cu_count, &o);
        if (st != W8A16_OK)
            return st;
        const uint64_t least = div_up(own_tiles, kMaxPassChunks);
        o = chunked(o.kernel, o.chunk_tiles < least ? least : o.chunk_tiles);
    }
    st = pass_plan(seqs, max_new, own, q_heads, kv_heads, head_dim, true, &o);
    if (st != W8A16_OK) {
        if (given)
            return st;
        return W8A16_OK;      // (too many workgroups: one pass)
    }
    // The shared keys' pass: either kernel (the tile kernel where the own
    // keys' takes it: the launch holds no other pair), in chunks of twice as
    // many tiles each time, or as many as give each CU one workgroup or two.
    // One pass is kept unless two promise 5 % (what the estimates are off by
    // where they are close).
    const Cost c(cu_count ? cu_count : kDefaultCUs, head_dim);
    const uint64_t rows = (uint64_t)tokens * (q_heads / kv_heads);
    double best = given ? 1e30 : 0.95 * one_pass(c, whole, shared_tiles, own_tiles, head_dim);
    auto consider = [&](uint32_t kernel, uint64_t per) {
        per = per > kMinTiles ? per : kMinTiles;
        w8a16_kv_plan_t p = chunked(kernel, per < shared_tiles ? per : shared_tiles);
        if (div_up(shared_tiles, p.chunk_tiles) > kMaxPassChunks ||
            pass_plan(1, tokens, shared, q_heads, kv_heads, head_dim, false, &p) != W8A16_OK)
            return;
        // (one launch, with the workgroups that fill tokens of no sequence:
        // kv_launch_groups)
        if (((uint64_t)p.grid + o.grid + 513 + tokens / 256) * 256 > kMaxThreads)
            return;
        const double t = two_passes(c, p, o, own_tiles, rows, kv_heads, head_dim);
        if (t < best) {
            best = t;
            *prefix = p;
            *suffix = o;
        }
    };
    for (uint32_t kernel = o.kernel == W8A16_KV_TILE ? W8A16_KV_TILE : W8A16_KV_ROWS; kernel <= W8A16_KV_TILE;
         ++kernel) {
        const uint64_t row_tiles = kv_heads * div_up(rows, kernel == W8A16_KV_ROWS ? 16 : 128);
        for (uint64_t per = kMinTiles; per / 2 < shared_tiles; per *= 2)
            consider(kernel, per);
        for (uint64_t n = 1; n <= 2; ++n)
            if (n * (uint64_t)c.cus > row_tiles)
                consider(kernel, div_up(shared_tiles, n * (uint64_t)c.cus / row_tiles));
    }
    if (given && !prefix->grid)
        return fail(W8A16_ERR_SHAPE, kTooMany);
    return W8A16_OK;
}

}  // namespace w8a16

extern "C" int w8a16_plan_kv_shared(uint32_t seqs, uint32_t tokens, uint32_t max_new, uint32_t max_kv,
                                    uint32_t shared, uint32_t q_heads, uint32_t kv_heads,
                                    uint32_t head_dim, uint32_t cu_count, w8a16_kv_plan_t *prefix,
                                    w8a16_kv_plan_t *own)
{
    using namespace w8a16;
    if (!prefix || !own)
        return fail(W8A16_ERR_NULL_PTR, "w8a16_plan_kv_shared: null plan");
    w8a16_kv_plan_t p;
    int st = make_kv_plan(seqs, max_new, max_kv, q_heads, kv_heads, head_dim, 0, cu_count, &p);
    if (st == W8A16_OK && (tokens < max_new || shared > max_kv))
        st = fail(W8A16_ERR_SHAPE, "w8a16_plan_kv_shared: tokens must be at least max_new, and shared at "
                                   "most max_kv");
    if (st != W8A16_OK)
        return st;
    return make_kv_shared_plans(seqs, tokens, max_new, max_kv, shared, q_heads, kv_heads, head_dim, cu_count,
                                nullptr, prefix, own);
}

extern "C" int w8a16_plan_kv_attention(uint32_t seqs, uint32_t max_new, uint32_t max_kv,
                                       uint32_t q_heads, uint32_t kv_heads, uint32_t head_dim,
                                       uint32_t window, uint32_t cu_count, w8a16_kv_plan_t *out)
{
    return w8a16_plan_kv_sinks(seqs, max_new, max_kv, q_heads, kv_heads, head_dim, window, 0, cu_count, out);
}

extern "C" int w8a16_plan_kv_sinks(uint32_t seqs, uint32_t max_new, uint32_t max_kv, uint32_t q_heads,
                                   uint32_t kv_heads, uint32_t head_dim, uint32_t window, uint32_t sinks,
                                   uint32_t cu_count, w8a16_kv_plan_t *out)
{
    window = w8a16::kv_window(window);
    return w8a16::make_kv_plan(seqs, max_new, max_kv, q_heads, kv_heads, head_dim, window, cu_count, out,
                               w8a16::kv_sinks(window, sinks));
}
