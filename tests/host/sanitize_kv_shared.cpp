// Host-only driver for the planner of attention with sinks and over a shared
// prefix (kv_plan.cpp), built with AddressSanitizer and
// UndefinedBehaviorSanitizer by the CPU test suite: a sweep over shapes, wild
// ones among them.  A sanitizer report aborts the run; accepted plans that do
// not cover their rows and keys, or whose launch or join does not fit, exit
// with status 1.
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "plan.h"
#include "w8a16.h"

namespace {

uint64_t g_state = 0x13198a2e03707344ull;

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
unsigned long g_one = 0, g_two = 0, g_refused = 0;

bool covers(const w8a16_kv_plan_t &p, uint64_t seqs, uint64_t rows, uint64_t keys, uint32_t hkv)
{
    return (p.kernel == W8A16_KV_ROWS || p.kernel == W8A16_KV_TILE) && p.chunks >= 1 &&
           (uint64_t)p.row_tiles * 16 * p.row_blocks >= rows && (uint64_t)p.chunks * p.chunk_tiles * 64 >= keys &&
           p.grid == seqs * hkv * p.row_tiles * p.chunks;
}

}  // namespace

int main()
{
    w8a16_kv_plan_t a, b;
    if (w8a16_plan_kv_shared(2, 2, 1, 64, 16, 1, 1, 64, 0, nullptr, &b) != W8A16_ERR_NULL_PTR ||
        w8a16_plan_kv_shared(2, 2, 1, 64, 16, 1, 1, 64, 0, &a, nullptr) != W8A16_ERR_NULL_PTR)
        g_fail = 1;
    for (int i = 0; i < 100000; ++i) {
        const uint32_t seqs = wild(300), max_new = wild(1u << (next_u32() % 12)),
                       max_kv = wild(1u << (next_u32() % 21)), hkv = wild(16),
                       hq = next_u32() % 8 ? hkv * (next_u32() % 16 + 1) : wild(64),
                       dim = next_u32() % 8 ? 16 * (next_u32() % 16 + 1) : wild(300),
                       cus = next_u32() % 3 ? 0u : wild(400);
        const uint32_t tokens = next_u32() % 8 ? seqs * max_new : wild(5000);
        const uint32_t shared = max_kv && next_u32() % 8 ? next_u32() % max_kv : wild(70000);
        const int st = w8a16_plan_kv_shared(seqs, tokens, max_new, max_kv, shared, hq, hkv, dim, cus, &a, &b);
        bool ok = true;
        if (st != W8A16_OK) {
            ++g_refused;
        } else if (!a.grid) {
            ++g_one;
            ok = covers(b, seqs, (uint64_t)max_new * (hq / hkv), max_kv, hkv);
        } else {
            ++g_two;
            const uint64_t before = shared / 64 * 64, group = hq / hkv;
            ok = covers(a, 1, tokens * group, shared, hkv) &&
                 covers(b, seqs, max_new * group, max_kv > before ? max_kv - before : 1, hkv) && a.waves == 4 &&
                 b.waves == 4 && a.chunks + b.chunks <= w8a16::kKvMaxChunks &&
                 (a.kernel == W8A16_KV_TILE || b.kernel == W8A16_KV_ROWS) &&
                 a.workspace_bytes == (uint64_t)a.grid * 16 * a.row_blocks * (dim + 4) * 4 &&
                 b.workspace_bytes == (uint64_t)b.grid * 16 * b.row_blocks * (dim + 4) * 4;
        }
        // a window with sinks: chunks for all tiles of a row tile
        const uint32_t window = wild(9000), sinks = wild(3000);
        w8a16_kv_plan_t s;
        if (w8a16::make_kv_plan(seqs, max_new, max_kv, hq, hkv, dim, window, cus, &s, sinks) == W8A16_OK && ok) {
            const uint64_t span = 16 * s.row_blocks / (hq / hkv) + 1, some = span < max_new ? span : max_new;
            uint64_t keys = (uint64_t)window + some;
            keys = window && keys < max_kv ? keys : max_kv;
            ok = covers(s, seqs, (uint64_t)max_new * (hq / hkv), keys, hkv);
        }
        if (!ok) {
            std::fprintf(stderr, "seqs=%u tokens=%u max_new=%u max_kv=%u shared=%u heads=%u/%u dim=%u window=%u "
                         "sinks=%u: prefix %u x %u tiles of %u workgroups, own %u x %u of %u\n", seqs, tokens,
                         max_new, max_kv, shared, hq, hkv, dim, window, sinks, a.chunks, a.chunk_tiles, a.grid,
                         b.chunks, b.chunk_tiles, b.grid);
            g_fail = 1;
        }
    }
    std::printf("shared planner sweep done (%lu two passes, %lu one, %lu refused): %s\n", g_two, g_one, g_refused,
                g_fail ? "FAILED" : "ok");
    return g_fail;
}
