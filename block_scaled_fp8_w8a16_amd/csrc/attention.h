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

// Rotation by several positions of a token (frame, row, column, ...): which
// of them turns a pair, and by which column of the table.
struct RopeAxes {
    const int32_t *positions;                   // axis a of token t at a * stride + t
    int64_t stride;
    uint32_t count, columns;                    // axes; the table's pairs per position
    uint32_t first[W8A16_ROPE_MAX_AXES];        // axis a's first pair (axes past count: past every pair)
    uint32_t stop[W8A16_ROPE_MAX_AXES];         // in turns: axis a > 0 has the pairs a, a + count, ... below it
    uint32_t turns, own;                        // the order (neither: split)
    uint32_t by_count;                          // 65536 / count + 1: i * by_count >> 16 is i / count for i < 512
    uint32_t whole;                             // every item's pairs are of one axis
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

struct RopeAxesArgs : RopeArgs {
    RopeAxes axes;
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

struct AppendAxesArgs : AppendArgs {
    RopeAxes axes;             // positions of the token axis; the items of a.q and of the keys are whole or not together
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

// A window beside which the first tokens stay visible.
struct SinkArgs : AttnArgs {
    uint32_t sinks;            // at least 1
};

// The two passes over a cache whose sequences share their first `shared`
// tokens (a multiple of the block): all rows of the call over those, as if
// of one sequence, then each sequence over its own.  The first leaves its
// chunks' partial rows for the second's join.
struct PrefixArgs : AttnArgs {
    uint32_t shared;
};
struct SuffixArgs : AttnArgs {
    uint32_t shared;
    const float *prefix;       // partial rows [(head, row tile)][chunk][row][dim], then their statistics
    uint32_t prefix_tiles, prefix_chunks, prefix_shift;    // row tiles, of 2^shift rows
    uint64_t prefix_rows;      // partial rows in all
};

constexpr uint32_t kKvTile = 64;                // keys per tile

hipError_t launch_rope_table(const w8a16_rope_config_t &c, float *table, uint32_t positions,
                             uint32_t rot_dim, hipStream_t stream);
hipError_t launch_rope(const RopeArgs &a, uint32_t dtype, hipStream_t stream);
hipError_t launch_rope_axes(const RopeAxesArgs &a, uint32_t dtype, hipStream_t stream);
hipError_t launch_kv_append(const AppendArgs &a, uint32_t dtype, hipStream_t stream);
hipError_t launch_kv_append_axes(const AppendAxesArgs &a, uint32_t dtype, hipStream_t stream);
// Workgroups of the attention's launch: the plan's and, where offsets are
// given, those of the tokens outside them.
inline uint64_t kv_launch_groups(const AttnArgs &a, uint32_t waves)
{
    const uint32_t tokens = a.fill_tokens * waves;
    return (uint64_t)a.grid + (a.seqs.cu ? (a.seqs.tokens + tokens - 1) / tokens : 0u);
}
// Args: AttnArgs or SinkArgs (defined in kv_attention.hip and
// kv_attention_sinks.hip; the tile kernel's in kv_tile*.hip).
template <class Args>
hipError_t launch_kv_rows(const Args &a, const w8a16_kv_plan_t &p, uint32_t dtype, hipStream_t stream);
template <class Args> hipError_t launch_kv_tile(const Args &a, uint32_t dtype, hipStream_t stream);
// Adds the chunks' partial results of the tile kernel; max_rows: rows of the
// longest sequence.
template <class Args>
hipError_t launch_kv_join(const Args &a, const w8a16_kv_plan_t &p, uint32_t max_rows, uint32_t dtype,
                          hipStream_t stream);
// Both passes over a shared prefix, and their join.
hipError_t launch_kv_shared(const PrefixArgs &a, const w8a16_kv_plan_t &pa, const SuffixArgs &b,
                            const w8a16_kv_plan_t &pb, uint32_t max_rows, uint32_t dtype, hipStream_t stream);

}  // namespace w8a16
