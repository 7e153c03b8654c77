// Host-only driver for the attention's planner (kv_plan.cpp), built with
// AddressSanitizer and UndefinedBehaviorSanitizer by the CPU test suite: a
// sweep of w8a16_plan_kv_attention over shapes, wild ones among them, and
// of caller-edited plans through kv_plan_finalize.  A sanitizer report
// aborts the run; an accepted plan that does not cover its rows and keys, or
// whose launch does not fit, exits with status 1.
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "plan.h"
#include "w8a16.h"

namespace {

uint64_t g_state = 0x243f6a8885a308d3ull;

// xorshift64 (Marsaglia, "Xorshift RNGs", 2003)
uint32_t next_u32()
{
    g_state ^= g_state << 13;
    g_state ^= g_state >> 7;
    g_state ^= g_state << 17;
    return (uint32_t)(g_state >> 32);
}

// Usually in 1..small, sometimes zero or anything.
uint32_t wild(uint32_t small)
{
    const uint32_t r = next_u32();
    return r % 16 == 0 ? next_u32() : (r % 16 == 1 ? 0u : next_u32() % small + 1u);
}

int g_fail = 0;
unsigned long g_accepted = 0, g_rejected = 0;

void check(int st, uint32_t seqs, uint32_t max_new, uint32_t max_kv, uint32_t hq, uint32_t hkv,
           uint32_t dim, uint32_t window, const w8a16_kv_plan_t &p)
{
    if (st != W8A16_OK) {
        ++g_rejected;
        return;
    }
    ++g_accepted;
    const uint64_t tile_rows = 16ull * p.row_blocks, rows = (uint64_t)max_new * (hq / hkv);
    uint64_t keys = max_kv;     // what a row tile sees at the most
    if (window && (uint64_t)window + max_new < keys)
        keys = (uint64_t)window + max_new;
    const bool ok = (p.kernel == W8A16_KV_ROWS || p.kernel == W8A16_KV_TILE) &&
                    (p.waves == 4 || p.waves == 8) && p.row_tiles * tile_rows >= rows &&
                    (uint64_t)p.chunks * p.chunk_tiles * 64 >= keys && p.chunks >= 1 &&
                    p.grid == (uint64_t)seqs * hkv * p.row_tiles * p.chunks && p.grid < (1u << 31) &&
                    (p.kernel == W8A16_KV_TILE || p.chunks <= w8a16::kKvMaxChunks) &&
                    p.workspace_bytes == (p.chunks > 1 ? p.grid * tile_rows * (dim + 4) * 4 : 0);
    if (!ok) {
        std::fprintf(stderr, "seqs=%u max_new=%u max_kv=%u heads=%u/%u dim=%u window=%u: kernel=%u "
                     "row_blocks=%u waves=%u row_tiles=%u chunk_tiles=%u chunks=%u grid=%u ws=%llu\n",
                     seqs, max_new, max_kv, hq, hkv, dim, window, p.kernel, p.row_blocks, p.waves,
                     p.row_tiles, p.chunk_tiles, p.chunks, p.grid, (unsigned long long)p.workspace_bytes);
        g_fail = 1;
    }
}

}  // namespace

int main()
{
    w8a16_kv_plan_t p;
    if (w8a16_plan_kv_attention(1, 1, 1, 1, 1, 64, 0, 0, nullptr) != W8A16_ERR_NULL_PTR)
        g_fail = 1;
    for (int i = 0; i < 200000; ++i) {
        const uint32_t seqs = wild(300), max_new = wild(1u << (next_u32() % 15)),
                       max_kv = next_u32() % 4 ? wild(1u << (next_u32() % 21)) : 0u,
                       hkv = wild(16), hq = next_u32() % 8 ? hkv * (next_u32() % 16 + 1) : wild(64),
                       dim = next_u32() % 8 ? 16 * (next_u32() % 16 + 1) : wild(300),
                       window = next_u32() % 2 ? 0u : wild(9000), cus = next_u32() % 3 ? 0u : wild(400);
        std::memset(&p, 0, sizeof p);
        int st = w8a16_plan_kv_attention(seqs, max_new, max_kv, hq, hkv, dim, window, cus, &p);
        check(st, seqs, max_new, max_kv, hq, hkv, dim, window, p);
        if (st != W8A16_OK)
            continue;
        p.kernel = wild(2);
        p.row_blocks = next_u32() % 2 ? 8 : (next_u32() % 4 ? 1 : wild(8));
        p.waves = next_u32() % 4 ? 4 : wild(8);
        p.chunk_tiles = wild(64);
        st = w8a16::kv_plan_finalize(seqs, max_new, max_kv, hq, hkv, dim, window, &p);
        check(st, seqs, max_new, max_kv, hq, hkv, dim, window, p);
    }
    std::printf("attention planner sweep done (%lu accepted, %lu refused): %s\n", g_accepted, g_rejected,
                g_fail ? "FAILED" : "ok");
    return g_fail;
}
