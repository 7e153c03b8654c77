// C ABI of the attention operators: argument checks, plans, launches.

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <exception>

#include "attention.h"
#include "host.h"
#include "plan.h"

namespace w8a16 {

namespace {

int refuse(int status, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int refuse(int status, const char *fmt, ...)
{
    char buf[288];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return fail(status, buf);
}

// The shared helpers name w8a16_gemm in their HIP errors.
int named(int status, const char *entry)
{
    return status == W8A16_OK ? status : fail_with_name(status, entry);
}

uint32_t elem_size(uint32_t dtype) { return dtype == W8A16_FP32 ? 4 : 2; }

bool aligned(const void *p, uint32_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Largest P of 8, 4 and 1 for which every group of P elements that an item
// loads or stores is whole and aligned to its size (16 bytes at the most).
uint32_t rope_pairs(const void *x, const void *y, const int64_t strides[4], uint32_t rot,
                    uint32_t dim, uint32_t size)
{
    for (uint32_t p = 8; p >= 4; p /= 2) {
        const uint32_t bytes = p * size < 16 ? p * size : 16;
        bool ok = rot % (2 * p) == 0 && (dim - rot) % (2 * p) == 0 && aligned(x, bytes) && aligned(y, bytes);
        for (int i = 0; i < 4; ++i)
            ok = ok && strides[i] * (int64_t)size % bytes == 0;
        if (ok)
            return p;
    }
    return 1;
}

void fill_rope(RopeRows &r, const void *x, void *y, const int64_t strides[4], const float *table,
               uint32_t table_positions, uint32_t rot, uint32_t dim, uint32_t layout,
               uint32_t heads, uint32_t dtype)
{
    r.x = static_cast<const uint8_t *>(x);
    r.y = static_cast<uint8_t *>(y);
    r.x_token = strides[0];
    r.x_head = strides[1];
    r.y_token = strides[2];
    r.y_head = strides[3];
    r.table = table;
    r.table_positions = table_positions;
    r.rot = rot;
    r.dim = dim;
    r.half = layout == W8A16_ROPE_HALF;
    r.heads = heads;
    r.pairs = rope_pairs(x, y, strides, rot, dim, elem_size(dtype));
    r.pair_items = rot / 2 / r.pairs;
    r.items = r.pair_items + (dim - rot + 2 * r.pairs - 1) / (2 * r.pairs);
    r.by_items = FastDiv(r.items);
}

// Several heads per thread where that still leaves every CU 512 threads
// (figures in rope_kernel.hip).
uint32_t rope_heads_per_thread(uint64_t items)
{
    return items >= 512ull * kDefaultCUs * kRopeHeads ? kRopeHeads : 1;
}

// Whether rows of dim elements that a call writes, `token` and `head` apart,
// lie on top of each other.
int check_apart(const char *entry, const char *name, int64_t token, int64_t head, uint32_t tokens,
                uint32_t heads, uint32_t dim)
{
    const uint64_t t = token < 0 ? 0 - (uint64_t)token : (uint64_t)token;
    const uint64_t h = head < 0 ? 0 - (uint64_t)head : (uint64_t)head;
    if ((tokens > 1 && t < dim) || (heads > 1 && h < dim) || (tokens > 1 && heads > 1 && t == h))
        return refuse(W8A16_ERR_SHAPE, "%s: %s rows of %u elements overlap (strides %lld by token, %lld by "
                      "head)", entry, name, dim, (long long)token, (long long)head);
    return W8A16_OK;
}

// A rotation's shape: dtype, layout, an even part of the head.
int check_rope(const char *entry, uint32_t dtype, uint32_t head_dim, uint32_t rot, uint32_t layout)
{
    if (dtype < W8A16_BF16 || dtype > W8A16_FP32)
        return refuse(W8A16_ERR_SHAPE, "%s: dtype=%u is not a w8a16_dtype", entry, dtype);
    if (layout > W8A16_ROPE_INTERLEAVED)
        return refuse(W8A16_ERR_SHAPE, "%s: layout=%u is not a w8a16_rope_layout", entry, layout);
    if (rot < 2 || rot % 2 || rot > head_dim)
        return refuse(W8A16_ERR_SHAPE, "%s: rot_dim=%u must be even, in 2..head_dim=%u", entry, rot, head_dim);
    return W8A16_OK;
}

int check_cache(const char *entry, const w8a16_kv_cache_t *c)
{
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale)
        return refuse(W8A16_ERR_NULL_PTR, "%s: null cache", entry);
    if (c->head_dim < 16 || c->head_dim > W8A16_KV_MAX_HEAD_DIM || c->head_dim % 16)
        return refuse(W8A16_ERR_SHAPE, "%s: head_dim=%u must be a multiple of 16 in 16..%u", entry,
                      c->head_dim, (unsigned)W8A16_KV_MAX_HEAD_DIM);
    if (c->page_size < W8A16_KV_BLOCK || c->page_size > 1024 || c->page_size % W8A16_KV_BLOCK)
        return refuse(W8A16_ERR_SHAPE, "%s: page_size=%u must be a multiple of 16 in 16..1024", entry,
                      c->page_size);
    if (!c->pages || c->pages > 0x7fffffffu || !c->kv_heads || c->kv_heads > 65535)
        return refuse(W8A16_ERR_SHAPE, "%s: pages=%u and kv_heads=%u must be in 1..2^31-1 and 1..65535",
                      entry, c->pages, c->kv_heads);
    const uint64_t page = (uint64_t)c->kv_heads * c->page_size * c->head_dim;
    const uint64_t blocks = (uint64_t)c->kv_heads * (c->page_size / W8A16_KV_BLOCK);
    if (page > (1ull << 31) || c->k_page_stride < page || c->v_page_stride < page ||
        c->k_scale_page_stride < blocks || c->v_scale_page_stride < blocks)
        return refuse(W8A16_ERR_SHAPE, "%s: page strides must cover a page (%llu code bytes, at most "
                      "2^31, and %llu scale bytes)", entry, (unsigned long long)page,
                      (unsigned long long)blocks);
    if (c->k_page_stride % 16 || c->v_page_stride % 16 || !aligned(c->k, 16) || !aligned(c->v, 16))
        return refuse(W8A16_ERR_SHAPE, "%s: k and v and their page strides must be 16-byte aligned", entry);
    return W8A16_OK;
}

int check_seqs(const char *entry, const w8a16_kv_seqs_t *s)
{
    if (!s)
        return refuse(W8A16_ERR_NULL_PTR, "%s: null sequences", entry);
    if (s->tokens == 0)
        return W8A16_OK;
    if (!s->block_table || !s->kv_lens)
        return refuse(W8A16_ERR_NULL_PTR, "%s: block_table and kv_lens must be non-null", entry);
    if (!s->seqs || s->seqs > 0x7fffffffu || s->tokens > 0x7fffffffu)
        return refuse(W8A16_ERR_SHAPE, "%s: %u tokens of %u sequences", entry, s->tokens, s->seqs);
    if (!s->cu_seqlens && s->tokens % s->seqs)
        return refuse(W8A16_ERR_SHAPE, "%s: without cu_seqlens, tokens=%u must be a multiple of seqs=%u",
                      entry, s->tokens, s->seqs);
    if (!s->block_table_width || s->block_table_stride < s->block_table_width)
        return refuse(W8A16_ERR_SHAPE, "%s: block_table_stride=%u must cover block_table_width=%u >= 1",
                      entry, s->block_table_stride, s->block_table_width);
    if (s->max_new == 0 || s->max_new > s->tokens)
        return refuse(W8A16_ERR_SHAPE, "%s: max_new=%u must be in 1..tokens=%u", entry, s->max_new,
                      s->tokens);
    if (!s->cu_seqlens && s->max_new != s->tokens / s->seqs)
        return refuse(W8A16_ERR_SHAPE, "%s: without cu_seqlens, max_new=%u must be tokens / seqs = %u",
                      entry, s->max_new, s->tokens / s->seqs);
    return W8A16_OK;
}

KvPool pool_of(const w8a16_kv_cache_t &c)
{
    KvPool p;
    p.k = static_cast<uint8_t *>(c.k);
    p.v = static_cast<uint8_t *>(c.v);
    p.k_scale = c.k_scale;
    p.v_scale = c.v_scale;
    p.k_page = c.k_page_stride;
    p.v_page = c.v_page_stride;
    p.ks_page = c.k_scale_page_stride;
    p.vs_page = c.v_scale_page_stride;
    p.pages = c.pages;
    p.heads = c.kv_heads;
    p.dim = c.head_dim;
    p.blocks = c.page_size / W8A16_KV_BLOCK;
    p.by_blocks = FastDiv(p.blocks);
    return p;
}

KvSeqs seqs_of(const w8a16_kv_seqs_t &s)
{
    KvSeqs q;
    q.block_table = s.block_table;
    q.kv_lens = s.kv_lens;
    q.cu = s.cu_seqlens;
    q.bt_stride = s.block_table_stride;
    q.bt_width = s.block_table_width;
    q.seqs = s.seqs;
    q.tokens = s.tokens;
    q.uniform = s.cu_seqlens ? 0u : s.tokens / s.seqs;
    q.by_uniform = FastDiv(q.uniform ? q.uniform : 1u);
    return q;
}

int rope_table(const w8a16_rope_config_t *c, float *table, uint32_t positions, uint32_t rot,
               hipStream_t stream)
{
    const char *entry = "w8a16_rope_table";
    int st = check_levers(entry);
    if (st != W8A16_OK)
        return st;
    if (!c || !table)
        return refuse(W8A16_ERR_NULL_PTR, "%s: config and table must be non-null", entry);
    if (c->scaling > W8A16_ROPE_BANDS)
        return refuse(W8A16_ERR_SHAPE, "%s: scaling=%u is not a w8a16_rope_scaling", entry, c->scaling);
    if (rot < (c->scaling == W8A16_ROPE_BASE ? 4u : 2u) || rot % 2 || rot > 1024)
        return refuse(W8A16_ERR_SHAPE, "%s: rot_dim=%u must be even and at most 1024", entry, rot);
    if (!(c->base > 1.0) || !(c->magnitude == c->magnitude) || (c->scaling && !(c->factor >= 1.0)))
        return refuse(W8A16_ERR_SHAPE, "%s: base=%g must exceed 1, factor=%g must be at least 1", entry,
                      c->base, c->factor);
    if (c->scaling == W8A16_ROPE_BANDS &&
        !(c->original > 0.0 && c->low_turns >= 0.0 && c->high_turns > c->low_turns))
        return refuse(W8A16_ERR_SHAPE, "%s: bands need original=%g > 0 and 0 <= low_turns=%g < high_turns=%g",
                      entry, c->original, c->low_turns, c->high_turns);
    if (positions > 0x7fffffffu)
        return refuse(W8A16_ERR_SHAPE, "%s: positions=%u must be below 2^31", entry, positions);
    if ((uint64_t)positions * (rot / 2) > kMaxThreads - 255)
        return refuse(W8A16_ERR_SHAPE, "%s: %u positions of %u pairs are too many for one call", entry,
                      positions, rot / 2);
    if (positions == 0)
        return W8A16_OK;
    hipError_t e = launch_rope_table(*c, table, positions, rot, stream);
    if (e != hipSuccess)
        return named(hip_fail(e, "kernel launch"), entry);
    if (log_enabled()) {
        char line[160];
        snprintf(line, sizeof line, "w8a16: %s positions=%u rot_dim=%u scaling=%u\n", entry, positions,
                 rot, c->scaling);
        log_line(line);
    }
    return named(launched(stream), entry);
}

int rope(const void *x, const int64_t strides[4], void *y, uint32_t dtype, uint32_t tokens,
         uint32_t heads, uint32_t head_dim, const float *table, uint32_t table_positions,
         uint32_t rot, const int32_t *positions, uint32_t layout, uint32_t inverse, hipStream_t stream)
{
    const char *entry = "w8a16_rope";
    int st = check_levers(entry);
    if (st != W8A16_OK)
        return st;
    if (tokens && (!x || !y || !table || !positions))
        return refuse(W8A16_ERR_NULL_PTR, "%s: x, y, table and positions must be non-null", entry);
    st = check_rope(entry, dtype, head_dim, rot, layout);
    if (st != W8A16_OK)
        return st;
    if (!heads)
        return refuse(W8A16_ERR_SHAPE, "%s: heads must be at least 1", entry);
    if (tokens == 0)
        return W8A16_OK;
    st = check_apart(entry, "y", strides[2], strides[3], tokens, heads, head_dim);
    if (st != W8A16_OK)
        return st;
    RopeArgs a;
    std::memset(static_cast<void *>(&a), 0, sizeof a);
    fill_rope(a.r, x, y, strides, table, table_positions, rot, head_dim, layout, heads, dtype);
    a.heads_per_thread = rope_heads_per_thread((uint64_t)heads * a.r.items * tokens);
    const uint64_t row = (uint64_t)((heads + a.heads_per_thread - 1) / a.heads_per_thread) * a.r.items;
    const uint64_t total = row * tokens;
    if (total >= (1ull << 31))
        return refuse(W8A16_ERR_SHAPE, "%s: %u tokens of %u heads are too many for one call", entry,
                      tokens, heads);
    a.positions = positions;
    a.total = (uint32_t)total;
    a.by_row = FastDiv((uint32_t)row);
    a.inverse = inverse != 0;
    hipError_t e = launch_rope(a, dtype, stream);
    if (e != hipSuccess)
        return named(hip_fail(e, "kernel launch"), entry);
    if (log_enabled()) {
        char line[200];
        snprintf(line, sizeof line,
                 "w8a16: %s tokens=%u heads=%u head_dim=%u rot_dim=%u: %u pairs of %u heads per thread\n",
                 entry, tokens, heads, head_dim, rot, a.r.pairs, a.heads_per_thread);
        log_line(line);
    }
    return named(launched(stream), entry);
}

int kv_append(const w8a16_kv_cache_t *cache, const w8a16_kv_seqs_t *seqs,
              const w8a16_kv_append_args_t *g, hipStream_t stream)
{
    const char *entry = "w8a16_kv_append";
    int st = check_levers(entry);
    if (st != W8A16_OK)
        return st;
    st = check_cache(entry, cache);
    if (st != W8A16_OK)
        return st;
    st = check_seqs(entry, seqs);
    if (st != W8A16_OK)
        return st;
    if (!g || (seqs->tokens && (!g->k || !g->v)) || (g->q && !g->q_out))
        return refuse(W8A16_ERR_NULL_PTR, "%s: k, v and, with q, q_out must be non-null", entry);
    if (g->dtype < W8A16_BF16 || g->dtype > W8A16_FP32)
        return refuse(W8A16_ERR_SHAPE, "%s: dtype=%u is not a w8a16_dtype", entry, g->dtype);
    if (g->table) {
        st = check_rope(entry, g->dtype, cache->head_dim, g->rot_dim, g->layout);
        if (st != W8A16_OK)
            return st;
    }
    if (g->q && (!g->table || !g->q_heads))
        return refuse(W8A16_ERR_SHAPE, "%s: queries need a table and q_heads >= 1", entry);
    if (seqs->tokens == 0)
        return W8A16_OK;
    AppendArgs a;
    std::memset(static_cast<void *>(&a), 0, sizeof a);
    a.pool = pool_of(*cache);
    a.seqs = seqs_of(*seqs);
    a.k = static_cast<const uint8_t *>(g->k);
    a.v = static_cast<const uint8_t *>(g->v);
    a.k_token = g->k_token_stride;
    a.k_head = g->k_head_stride;
    a.v_token = g->v_token_stride;
    a.v_head = g->v_head_stride;
    const uint32_t size = elem_size(g->dtype), dim = cache->head_dim, rot = g->table ? g->rot_dim : 0;
    const int64_t ks[4] = {a.k_token, a.k_head, a.v_token, a.v_head};
    // widest whole pieces: of the rows' alignment, and of the rotated halves
    // (4 x 2048 tokens of 8 KV heads: pieces of 8 elements 13.7 us, of 4 15.1,
    // of 1 30.1)
    a.vec = 1;
    for (uint32_t n = 8; n >= 4 && a.vec == 1; n /= 2) {
        const uint32_t bytes = n * size < 16 ? n * size : 16;
        bool ok = aligned(g->k, bytes) && aligned(g->v, bytes) && rot % (2 * n) == 0;
        for (int i = 0; i < 4; ++i)
            ok = ok && ks[i] * (int64_t)size % bytes == 0;
        a.vec = ok ? n : 1;
    }
    // n tokens touch at most ceil((n + 15) / 16) blocks of 16 slots
    a.seq_blocks = (seqs->max_new - 1 + 2 * W8A16_KV_BLOCK - 1) / W8A16_KV_BLOCK;
    const uint64_t units = (uint64_t)seqs->seqs * a.seq_blocks * cache->kv_heads * 2;
    uint64_t groups = (units + 3) / 4;
    a.by_units = FastDiv(cache->kv_heads * 2);
    a.by_chunks = FastDiv(dim / 8);
    a.by_k_items = FastDiv(dim / (2 * a.vec));
    const uint64_t seq_units = (uint64_t)a.seq_blocks * cache->kv_heads * 2;
    a.by_seq_units = FastDiv((uint32_t)(seq_units < 0x7fffffffu ? seq_units : 0x7fffffffu));
    a.kv_groups = (uint32_t)groups;
    const int64_t qs[4] = {g->q_token_stride, g->q_head_stride, g->q_out_token_stride,
                           g->q_out_head_stride};
    fill_rope(a.q, g->q, g->q_out, qs, g->table, g->table_positions, rot, dim, g->layout,
              g->q ? g->q_heads : 0, g->dtype);
    if (g->q) {
        a.q_heads_per_thread = rope_heads_per_thread((uint64_t)g->q_heads * a.q.items * seqs->tokens);
        const uint64_t head_groups = (g->q_heads + a.q_heads_per_thread - 1) / a.q_heads_per_thread;
        const uint64_t per = (head_groups * a.q.items + 255) / 256;
        a.q_groups = (uint32_t)per;
        a.by_q_groups = FastDiv(a.q_groups);
        groups += per * seqs->tokens;
    }
    if (units >= (1ull << 31) || groups * 256ull > kMaxThreads)
        return refuse(W8A16_ERR_SHAPE, "%s: %u tokens of %u sequences (max_new=%u) are too many for one "
                      "call", entry, seqs->tokens, seqs->seqs, seqs->max_new);
    if (g->q) {
        st = check_apart(entry, "q_out", g->q_out_token_stride, g->q_out_head_stride, seqs->tokens,
                         g->q_heads, cache->head_dim);
        if (st != W8A16_OK)
            return st;
    }
    hipError_t e = launch_kv_append(a, g->dtype, stream);
    if (e != hipSuccess)
        return named(hip_fail(e, "kernel launch"), entry);
    if (log_enabled()) {
        char line[256];
        snprintf(line, sizeof line,
                 "w8a16: %s tokens=%u seqs=%u kv_heads=%u head_dim=%u page_size=%u rot_dim=%u q_heads=%u: "
                 "%u blocks per sequence, grid=%llu\n", entry, seqs->tokens, seqs->seqs, cache->kv_heads,
                 dim, cache->page_size, rot, g->q ? g->q_heads : 0, a.seq_blocks,
                 (unsigned long long)groups);
        log_line(line);
    }
    return named(launched(stream), entry);
}

int kv_attention(const w8a16_kv_cache_t *cache, const w8a16_kv_seqs_t *seqs,
                 const w8a16_kv_attention_args_t *g, hipStream_t stream)
{
    const char *entry = "w8a16_kv_attention";
    int st = check_levers(entry);
    if (st != W8A16_OK)
        return st;
    st = check_cache(entry, cache);
    if (st != W8A16_OK)
        return st;
    st = check_seqs(entry, seqs);
    if (st != W8A16_OK)
        return st;
    if (!g || (seqs->tokens && (!g->q || !g->out)))
        return refuse(W8A16_ERR_NULL_PTR, "%s: q and out must be non-null", entry);
    if (g->dtype != W8A16_BF16 && g->dtype != W8A16_FP16)
        return refuse(W8A16_ERR_SHAPE, "%s: dtype=%u must be W8A16_BF16 or W8A16_FP16", entry, g->dtype);
    if (!g->q_heads || g->q_heads % cache->kv_heads)
        return refuse(W8A16_ERR_SHAPE, "%s: q_heads=%u must be a positive multiple of kv_heads=%u", entry,
                      g->q_heads, cache->kv_heads);
    if (!(g->scale >= 0.f && g->scale < 3.0e38f))
        return refuse(W8A16_ERR_SHAPE, "%s: scale=%g must be finite and not negative", entry,
                      (double)g->scale);
    if (seqs->tokens == 0)
        return W8A16_OK;
    st = check_apart(entry, "out", g->out_token_stride, g->out_head_stride, seqs->tokens, g->q_heads,
                     cache->head_dim);
    if (st != W8A16_OK)
        return st;
    const uint32_t group = g->q_heads / cache->kv_heads;
    if ((uint64_t)seqs->max_new * group >= (1ull << 31))
        return refuse(W8A16_ERR_SHAPE, "%s: max_new=%u rows of %u query heads per KV head are too many",
                      entry, seqs->max_new, group);
    const uint64_t held = (uint64_t)seqs->block_table_width * cache->page_size;
    uint32_t max_kv = held < (1u << 30) ? (uint32_t)held : 1u << 30;
    if (g->max_kv && g->max_kv < max_kv)
        max_kv = g->max_kv;
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return named(hip_fail(e, "hipGetDevice"), entry);
    uint32_t cus = 0;
    st = device_cu_count(dev, &cus);
    if (st != W8A16_OK)
        return named(st, entry);
    const uint32_t window = g->window < 0x7fffffffu ? g->window : 0;
    w8a16_kv_plan_t p;
    if (g->plan) {
        p = *g->plan;
        st = kv_plan_finalize(seqs->seqs, seqs->max_new, max_kv, g->q_heads, cache->kv_heads,
                              cache->head_dim, window, &p);
    } else {
        st = make_kv_plan(seqs->seqs, seqs->max_new, max_kv, g->q_heads, cache->kv_heads,
                          cache->head_dim, window, cus, &p);
    }
    if (st != W8A16_OK)
        return st;
    AttnArgs a;
    std::memset(static_cast<void *>(&a), 0, sizeof a);
    a.seqs = seqs_of(*seqs);
    a.grid = p.grid;
    // (a long token axis by some 512 workgroups)
    const uint32_t fill = seqs->tokens / (512u * p.waves) + 1;
    a.fill_tokens = fill < 64u ? fill : 64u;
    if (kv_launch_groups(a, p.waves) * 64ull * p.waves > kMaxThreads)
        return refuse(W8A16_ERR_SHAPE, "%s: %u tokens of %u sequences are too many for one call", entry,
                      seqs->tokens, seqs->seqs);
    if (p.workspace_bytes) {
        w8a16_plan_t need;
        std::memset(&need, 0, sizeof need);
        need.workspace_bytes = p.workspace_bytes;
        if (p.kernel == W8A16_KV_ROWS)
            need.counter_count = p.grid / p.chunks * kKvCounterStride;
        Workspace ws;
        st = get_workspace(dev, stream, need, &ws);
        if (st != W8A16_OK)
            return named(st, entry);
        a.ws = ws.ws;
        a.counters = ws.counters;
    }
    a.pool = pool_of(*cache);
    a.q = static_cast<const uint8_t *>(g->q);
    a.out = static_cast<uint8_t *>(g->out);
    a.lse = g->lse;
    a.q_token = g->q_token_stride;
    a.q_head = g->q_head_stride;
    a.out_token = g->out_token_stride;
    a.out_head = g->out_head_stride;
    a.scale_log2 = g->scale * 1.4426950408889634f;
    a.group = group;
    a.by_group = FastDiv(group);
    a.q_heads = g->q_heads;
    a.causal = g->causal != 0;
    a.window = window;
    a.row_tiles = p.row_tiles;
    a.chunks = p.chunks;
    a.chunk_tiles = p.chunk_tiles;
    e = p.kernel == W8A16_KV_ROWS ? launch_kv_rows(a, p, g->dtype, stream)
                                  : launch_kv_tile(a, g->dtype, stream);
    if (e == hipSuccess && p.kernel == W8A16_KV_TILE && p.chunks > 1)
        e = launch_kv_join(a, p, seqs->max_new * group, g->dtype, stream);
    if (e != hipSuccess)
        return named(hip_fail(e, "kernel launch"), entry);
    if (log_enabled()) {
        char line[320];
        snprintf(line, sizeof line,
                 "w8a16: %s tokens=%u seqs=%u q_heads=%u kv_heads=%u head_dim=%u max_new=%u max_kv=%u "
                 "window=%u: kernel=%s row_blocks=%u row_tiles=%u chunks=%u (%u tiles each) grid=%u "
                 "workspace=%llu%s\n", entry, seqs->tokens, seqs->seqs, g->q_heads, cache->kv_heads,
                 cache->head_dim, seqs->max_new, max_kv, window,
                 p.kernel == W8A16_KV_ROWS ? "kv-rows" : "kv-tile", p.row_blocks, p.row_tiles, p.chunks,
                 p.chunk_tiles, p.grid, (unsigned long long)p.workspace_bytes,
                 g->plan ? ": caller's plan" : "");
        log_line(line);
    }
    return named(launched(stream), entry);
}

// No C++ exception (an allocation in the maps and strings behind the
// helpers) leaves a C entry.
template <class F> int guarded(const char *entry, F f)
{
    try {
        return f();
    } catch (const std::exception &e) {
        try {
            return refuse(W8A16_ERR_HIP, "%s: %s", entry, e.what());
        } catch (...) {
        }
    } catch (...) {
    }
    return W8A16_ERR_HIP;
}

}  // namespace

}  // namespace w8a16

extern "C" {

int w8a16_rope_table(const w8a16_rope_config_t *config, float *table, uint32_t positions,
                     uint32_t rot_dim, void *stream)
{
    return w8a16::guarded("w8a16_rope_table", [&] {
        return w8a16::rope_table(config, table, positions, rot_dim, static_cast<hipStream_t>(stream));
    });
}

int w8a16_rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, void *y,
               int64_t y_token_stride, int64_t y_head_stride, uint32_t dtype, uint32_t tokens,
               uint32_t heads, uint32_t head_dim, const float *table, uint32_t table_positions,
               uint32_t rot_dim, const int32_t *positions, uint32_t layout, uint32_t inverse,
               void *stream)
{
    const int64_t strides[4] = {x_token_stride, x_head_stride, y_token_stride, y_head_stride};
    return w8a16::guarded("w8a16_rope", [&] {
        return w8a16::rope(x, strides, y, dtype, tokens, heads, head_dim, table, table_positions, rot_dim,
                           positions, layout, inverse, static_cast<hipStream_t>(stream));
    });
}

int w8a16_kv_append(const w8a16_kv_cache_t *cache, const w8a16_kv_seqs_t *seqs,
                    const w8a16_kv_append_args_t *args, void *stream)
{
    return w8a16::guarded("w8a16_kv_append", [&] {
        return w8a16::kv_append(cache, seqs, args, static_cast<hipStream_t>(stream));
    });
}

int w8a16_kv_attention(const w8a16_kv_cache_t *cache, const w8a16_kv_seqs_t *seqs,
                       const w8a16_kv_attention_args_t *args, void *stream)
{
    return w8a16::guarded("w8a16_kv_attention", [&] {
        return w8a16::kv_attention(cache, seqs, args, static_cast<hipStream_t>(stream));
    });
}

}  // extern "C"
