// Kernel arguments and launch interface of the attention operators (rotary
// positions, paged FP8 cache, attention over it).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "plan.h"
#include "w8a16.h"

namespace w8a16 {

// Division of n < 2^31 by a constant d >= 1 by a multiplication and a shift
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994): with s = ceil(log2 d) and mul = ceil(2^(31 + s) / d),
// n * mul >> (31 + s) is floor(n / d).
struct FastDiv {
    uint32_t d = 1, mul = 1u << 31, shift = 31;
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div)
    {
        uint32_t s = 0;
        while (s < 31 && (1u << s) < div)
            ++s;
        shift = 31 + s;
        mul = (uint32_t)((((uint64_t)1 << shift) + div - 1) / div);
    }
    __host__ __device__ uint32_t div(uint32_t n) const
    {
        return (uint32_t)(((uint64_t)n * mul) >> shift);
    }
};

// One token row of a rotation: `pair_items` items of P pairs, then
// `pass_items` items of 2P unrotated elements.
struct RopeRows {
    const uint8_t *x;
    uint8_t *y;
    int64_t x_token, x_head, y_token, y_head;   // strides in elements
    const float *table;
    uint32_t table_positions, rot, dim, half;   // half: pairs are i and i + rot/2
    uint32_t heads, pair_items, items;          // items per head
    FastDiv by_items;                           // items per head
    uint32_t pairs;                             // P: pairs per item (1, 4 or 8)
};

// Heads a thread rotates where there are enough of them to fill the chip.
constexpr uint32_t kRopeHeads = 4;

struct RopeArgs {
    RopeRows r;
    const int32_t *positions;
    uint32_t total;                             // threads: tokens * head groups * items
    FastDiv by_row;                             // head groups * items
    uint32_t inverse, heads_per_thread;         // 1 or kRopeHeads
};

struct KvPool {
    uint8_t *k, *v, *k_scale, *v_scale;
    uint64_t k_page, v_page, ks_page, vs_page;  // page strides in bytes
    uint32_t pages, heads, dim, blocks;         // blocks of 16 tokens per page
    FastDiv by_blocks;
};

struct KvSeqs {
    const int32_t *block_table, *kv_lens, *cu;
    uint32_t bt_stride, bt_width, seqs, tokens, uniform;   // uniform: tokens per sequence without cu
    FastDiv by_uniform;
};

struct AppendArgs {
    KvPool pool;
    KvSeqs seqs;
    const uint8_t *k, *v;
    int64_t k_token, k_head, v_token, v_head;
    uint32_t vec;              // elements of a load (8, 4 or 1): aligned, and whole in the rotated halves
    uint32_t seq_blocks;       // blocks a sequence's new tokens may touch
    uint32_t kv_groups;        // workgroups of the append; the rest rotate queries
    FastDiv by_units, by_seq_units;
    FastDiv by_chunks, by_k_items;   // 8-element chunks, and 2 * vec-element items, of a head
    RopeRows q;                // q.x null: no queries
    uint32_t q_groups;         // workgroups per token of the queries
    uint32_t q_heads_per_thread;
    FastDiv by_q_groups;
};

struct AttnArgs {
    KvPool pool;
    KvSeqs seqs;
    const uint8_t *q;
    uint8_t *out;
    float *lse, *ws;
    uint32_t *counters;        // arrival counters of the row kernel, zero between calls
    int64_t q_token, q_head, out_token, out_head;
    float scale_log2;          // scale * log2(e)
    uint32_t group;            // query heads per KV head
    FastDiv by_group;
    uint32_t q_heads, causal, window;
    uint32_t row_tiles, chunks, chunk_tiles;
    uint32_t grid;             // workgroups of the plan; the launch's others look at the token axis
                               // for tokens that no sequence brings
    uint32_t fill_tokens;      // that one of their waves takes (at most 64)
};

constexpr uint32_t kKvTile = 64;                // keys per tile

hipError_t launch_rope_table(const w8a16_rope_config_t &c, float *table, uint32_t positions,
                             uint32_t rot_dim, hipStream_t stream);
hipError_t launch_rope(const RopeArgs &a, uint32_t dtype, hipStream_t stream);
hipError_t launch_kv_append(const AppendArgs &a, uint32_t dtype, hipStream_t stream);
// Workgroups of the attention's launch: the plan's and, where offsets are
// given, those of the tokens outside them.
inline uint64_t kv_launch_groups(const AttnArgs &a, uint32_t waves)
{
    const uint32_t tokens = a.fill_tokens * waves;
    return (uint64_t)a.grid + (a.seqs.cu ? (a.seqs.tokens + tokens - 1) / tokens : 0u);
}
hipError_t launch_kv_rows(const AttnArgs &a, const w8a16_kv_plan_t &p, uint32_t dtype,
                          hipStream_t stream);
hipError_t launch_kv_tile(const AttnArgs &a, uint32_t dtype, hipStream_t stream);
// Adds the chunks' partial results of the tile kernel; max_rows: rows of the
// longest sequence.
hipError_t launch_kv_join(const AttnArgs &a, const w8a16_kv_plan_t &p, uint32_t max_rows,
                          uint32_t dtype, hipStream_t stream);

}  // namespace w8a16
