/*
 * w8a16.h -- C ABI of the block-scaled FP8 W8A16 small-M GEMM for MI355X
 * (gfx950).
 *
 * The operation (page "w8a16_gemm_pipelined_m32.rs", doc comment of
 * `w8a16_gemm_pipelined_m32_strided`; one FP8 scale block per 128-wide K
 * step, doc comment of `W8A16_M32_K_BLOCK`):
 *
 *   C[i][j] = bf16( sum_{b < K/128} S[j/128][b] * sum_{t < 128} A[i][128b+t] * W[j][128b+t] )
 *
 *   A  BF16 (bits, 2 bytes)   [m, a_row_stride]   first k elements of each row are read
 *   W  FP8 E4M3 (OCP E4M3FN)  [n, k]              row-major, contiguous, 1 byte per weight
 *   S  FP32                   [ceil(n/128), k/128] row-major: scale of W block (j/128, k/128)
 *   C  BF16                   [m, c_row_stride]   first n elements of each row are written
 *
 * Strides are in elements.  Products are taken in BF16 x BF16 with FP32
 * accumulation; each 128-wide K step's partial sum is multiplied by its
 * block scale once and added in FP32; the result is rounded to BF16 with
 * round-to-nearest-even.  The association of the K reduction inside a step,
 * across the waves of a workgroup and across K splits is fixed by the plan,
 * so a given plan gives the same bits on every run.
 *
 * Ownership: every pointer passed to w8a16_gemm* is a DEVICE pointer owned
 * by the caller, who keeps the buffers alive until the stream has passed
 * the call.  The library keeps no pointer to them.  It owns one split-K
 * workspace and counter array per (device, stream), allocated with
 * hipMalloc on first use and grown when a larger plan needs it.  Growing
 * allocates new buffers and keeps the old ones until the process ends, so
 * calls in flight and HIP graphs captured earlier on that stream stay
 * valid; it needs no synchronisation.  Growth cannot happen while the
 * stream is being captured: such a call returns W8A16_ERR_WORKSPACE and
 * enqueues nothing, so make one call with the largest plan on a stream
 * before capturing it.  A graph keeps using the workspace of the stream it
 * was captured on: two replays of graphs captured on one stream must not
 * overlap in time.
 *
 * Threads: calls may come from several threads, on one stream too; the
 * launches of a call that use a workspace are enqueued with none of another
 * call's that uses it between them.  hipStreamPerThread is a stream of each
 * thread's but has one workspace: calls on it that use one must not overlap.
 *
 * Alignment and aliasing: A, W, S and C must be 16-byte aligned (torch
 * allocations are).  C must not overlap A, W or S.  c_row_stride may be any
 * value >= n.
 *
 * Errors: every entry point returns a w8a16_status.  Argument errors are
 * detected before anything is enqueued, in the order of the enum below
 * (codes 1..4 in the order the page checks them; 5..7 and 9 are checks the
 * page does not make; 10, a bad diagnostic setting, is checked first).
 * w8a16_last_error() then holds a message for the calling thread.  Launches are asynchronous: the call returns once the kernel is
 * enqueued on `stream`; a failed enqueue returns W8A16_ERR_HIP.
 */
#ifndef W8A16_H
#define W8A16_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum w8a16_status {
    W8A16_OK = 0,
    W8A16_ERR_M_ZERO = 1,            /* m == 0: no rows to compute */
    W8A16_ERR_K_NOT_MULT_128 = 2,    /* k == 0 or k % 128 != 0 */
    W8A16_ERR_PITCH_TOO_SHORT = 3,   /* a_row_stride < k or c_row_stride < n */
    W8A16_ERR_A_STRIDE_ALIGN = 4,    /* a_row_stride % 8 != 0 (16-byte rows) */
    W8A16_ERR_N_ZERO = 5,            /* n == 0: empty launch */
    W8A16_ERR_NULL_PTR = 6,          /* a, w_fp8, block_scale or c is null */
    W8A16_ERR_BAD_PLAN = 7,          /* a plan that does not fit the problem */
    W8A16_ERR_HIP = 8,               /* allocation or launch failed in HIP */
    W8A16_ERR_WORKSPACE = 9,         /* the plan's workspace cannot be provided:
                                        it would have to grow during stream capture,
                                        or it exceeds w8a16_gemm_noalloc's scratch */
    W8A16_ERR_ENV = 10,              /* a diagnostic environment variable holds a value
                                        other than 0 or 1 (see Diagnostics below) */
    W8A16_ERR_SHAPE = 11             /* attention operators: a size, type, stride or
                                        alignment the operator does not take */
} w8a16_status;

/* Diagnostics.  Two environment variables, read once per process at the
 * first call of an entry point that enqueues work (w8a16_gemm,
 * _gemm_planned, _gemm_noalloc, _gemm_batched, _act_quant_fp8,
 * _gemm_epilogue, _gemm_w8a8[_planned], _gemm_w4a4[_planned], _rope_table, _rope,
 * _rope_axes, _kv_append[_axes], _kv_attention[_span]); unset, empty or "0" is off,
 * "1" is on, and any other value makes each of those calls return
 * W8A16_ERR_ENV, before any other check, with the variable named in
 * w8a16_last_error().  The pure planning calls ignore them.
 *   W8A16_LOG=1: each distinct launch (entry point, m, n, k and plan) is
 *     printed once to stderr: kernel, tile, K splits, waves, grid, LDS,
 *     workspace, and for a default plan the planner rule that chose it.
 *   W8A16_DEBUG_SYNC=1: after enqueuing, the call waits for the stream and
 *     returns W8A16_ERR_HIP if the kernel failed.  On a stream being
 *     captured into a graph it does not wait (nothing runs until replay).
 *     It serialises the caller with the GPU: for debugging only. */

/* Kernel families a plan can name. */
typedef enum w8a16_kernel {
    /* Weight-streaming kernel: a workgroup owns n_blocks 16-column blocks
     * of C and m_blocks 16-row blocks, its waves take interleaved 128-wide
     * K steps, and K may be split across workgroups with a fixed-order
     * FP32 fix-up. */
    W8A16_KERNEL_STREAM = 1,
    /* Tiled kernel for m above 32: a workgroup owns a 16*m_blocks-row
     * (64 or 128) x 16*n_blocks-column (64 or 128) tile of C, stages A and
     * the FP8 weight of each K step in LDS rings (a_depth and depth
     * buffers), and its waves split the tile (8 waves: also each K step). */
    W8A16_KERNEL_TILE = 2,
    /* Ring kernel for small m: a workgroup owns n_blocks 16-column blocks
     * and m_blocks 16-row blocks of C over all of K, streams K in stages of
     * stage_steps steps with a ring of `depth` stages in flight (1 KiB
     * row-contiguous LDS-DMA loads), and its waves, grouped per column
     * block, take the stages' steps round-robin.  No K split. */
    W8A16_KERNEL_RING = 3,
    /* W8A8 kernel (w8a16_gemm_w8a8 only): A given as FP8 codes with one
     * scale per (row, K step); the stream kernel's organisation with A
     * staged like the weight and one FP8 MFMA per K step.  No K split. */
    W8A16_KERNEL_W8A8 = 4,
    /* W4A4 MX kernel (w8a16_gemm_w4a4 only): a workgroup owns n_blocks
     * 16-column blocks and m_blocks 16-row blocks of C over all of K, its
     * waves take interleaved groups of four 128-wide K steps with one scaled
     * FP4 MFMA per block and step, each activation fragment feeding the
     * n_blocks weight blocks.  No K split. */
    W8A16_KERNEL_W4A4 = 5,
    /* Persistent W4A4 MX kernel: one workgroup per CU owns an equal
     * contiguous range of 16-row weight tiles and stages all of A in LDS;
     * its waves split the range's (tile, 4-step K group) items evenly and
     * add the partials of tiles split between them in wave order. */
    W8A16_KERNEL_W4A4_PS = 6
} w8a16_kernel;

/* Launch plan.  w8a16_plan() fills every field; callers may change
 * kernel, m_blocks, n_blocks, splits, depth, flags, waves, stage_steps and
 * a_depth and pass the result to
 * w8a16_gemm_planned(), which recomputes the derived fields and rejects a
 * plan the kernels do not support (W8A16_ERR_BAD_PLAN). */
typedef struct w8a16_plan {
    uint32_t kernel;          /* w8a16_kernel */
    uint32_t m_blocks;        /* 16-row blocks of C per workgroup tile */
    uint32_t n_blocks;        /* 16-column blocks of C per workgroup tile */
    uint32_t splits;          /* K splits across workgroups (>= 1) */
    uint32_t steps_per_split; /* 128-wide K steps per split (derived) */
    uint32_t m_tiles;         /* ceil(m / (16 * m_blocks)) (derived) */
    uint32_t n_tiles;         /* ceil(n / (16 * n_blocks)) (derived) */
    uint32_t grid;            /* workgroups launched (derived) */
    uint32_t block;           /* threads per workgroup (derived) */
    uint32_t lds_bytes;       /* LDS per workgroup (derived) */
    uint64_t workspace_bytes; /* split-K FP32 partials (derived; 0 if splits == 1) */
    uint32_t counter_count;   /* 32-bit words of split-K arrival counters, one counter
                                 per tile every 64 words (derived) */
    uint32_t cu_count;        /* compute units the plan was sized for */
    uint32_t depth;           /* stream: K steps each wave keeps in flight (1, 2, 4);
                                 tile: weight ring buffers; ring: stages in flight (2..4) */
    uint32_t flags;           /* W8A16_FLAG_* bits */
    uint32_t waves;           /* waves per workgroup (stream 4/8/16, ring 8/16,
                                 tile 4/6/8/10) */
    uint32_t stage_steps;     /* ring: K steps per stage (4 or 8); 0 for the others */
    uint32_t a_depth;         /* tile: A ring buffers (2..6; 0 means 2); 0 for the others */
} w8a16_plan_t;

/* Plan flags. */
enum {
    /* Stream kernel: load A fragments straight into the MFMA register
     * layout instead of staging coalesced loads through LDS (the weight is
     * always staged). */
    W8A16_FLAG_DIRECT = 1u,
    /* Ring kernel, m <= 8 with m_blocks == 1: stage 8 A rows instead of 16
     * (derived by w8a16_plan_finalize from m; callers need not set it). */
    W8A16_FLAG_A8 = 2u,
    /* Stream kernel with splits > 1: the K splits of every tile run on one
     * XCD (consecutive logical workgroups inside one XCD's contiguous range
     * of the grid), so the partials they exchange stay in that XCD's L2.
     * w8a16_plan() sets it on every plan that splits K.
     * w8a16_plan_finalize() rejects it (W8A16_ERR_BAD_PLAN) unless
     * splits >= 2, the grid is a multiple of 8 and each eighth of the grid
     * holds whole tiles.  The publication itself is the same with or
     * without the flag: each split stores its partial with agent-scope
     * (write-through) stores, waits for them, then counts its arrival; the
     * last one acquires at agent scope and reads the partials with
     * agent-scope loads.  It is correct on whichever XCDs the splits run. */
    W8A16_FLAG_XCD_LOCAL = 4u
};

/* Validate the scalar arguments alone, in the documented order.  Pure: no
 * GPU call.  Returns W8A16_OK or the first failing check's code. */
int w8a16_check_args(uint32_t m, uint32_t n, uint32_t k,
                     uint32_t a_row_stride, uint32_t c_row_stride);

/* Default plan for (m, n, k) on a device with `cu_count` compute units
 * (0 means 256, MI355X).  Pure: no GPU call.  Checks m, n and k as
 * w8a16_check_args does (pitches are not part of a plan). */
int w8a16_plan(uint32_t m, uint32_t n, uint32_t k, uint32_t cu_count,
               w8a16_plan_t *out);

/* Recompute the derived fields of a caller-edited plan and check it.
 * Pure: no GPU call. */
int w8a16_plan_finalize(uint32_t m, uint32_t n, uint32_t k, w8a16_plan_t *plan);

/* The GEMM.  a: BF16 [m, a_row_stride]; w_fp8: E4M3 [n, k]; block_scale:
 * FP32 [ceil(n/128), k/128]; c: BF16 [m, c_row_stride].  All device
 * pointers.  stream: a hipStream_t (NULL for the null stream).  Picks the
 * plan with w8a16_plan() for the current device's CU count. */
int w8a16_gemm(const void *a, uint32_t a_row_stride,
               const void *w_fp8, const float *block_scale,
               void *c, uint32_t c_row_stride,
               uint32_t m, uint32_t n, uint32_t k, void *stream);

/* The GEMM with an explicit plan (kernel, m_blocks, n_blocks, splits taken
 * from *plan; derived fields recomputed).  For tests and tuning: every
 * valid plan computes the same operation; plans differ only in the order of
 * the FP32 additions. */
int w8a16_gemm_planned(const void *a, uint32_t a_row_stride,
                       const void *w_fp8, const float *block_scale,
                       void *c, uint32_t c_row_stride,
                       uint32_t m, uint32_t n, uint32_t k,
                       const w8a16_plan_t *plan, void *stream);

/* ---- No-allocation entry point --------------------------------------------
 * For callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.
 *
 * w8a16_gemm_noalloc() computes exactly what w8a16_gemm() computes, with
 * the same default plan, arguments, checks (codes 1..6) and asynchronous
 * launch, but the split-K partials and arrival counters of a plan that
 * splits K come from a static device array the library holds on each GPU
 * it runs on until the process ends (W8A16_NOALLOC_WORKSPACE_BYTES of
 * partials plus W8A16_NOALLOC_COUNTERS 32-bit counter words, 17 MiB).  It
 * calls no hipMalloc, hipFree or other allocating routine.  A plan needing
 * more than that returns W8A16_ERR_WORKSPACE and enqueues nothing.  The
 * first call on a device looks the array up and clears its counters with a
 * small kernel on `stream`; every later call leaves them at zero.
 *
 * All calls on one GPU share its array: calls that overlap in time on that
 * GPU (other streams, concurrent graph replays) race and give wrong
 * results.  Order them (one stream, or events). */
#define W8A16_NOALLOC_WORKSPACE_BYTES (16u << 20)
#define W8A16_NOALLOC_COUNTERS (1u << 18)

int w8a16_gemm_noalloc(const void *a, uint32_t a_row_stride,
                       const void *w_fp8, const float *block_scale,
                       void *c, uint32_t c_row_stride,
                       uint32_t m, uint32_t n, uint32_t k, void *stream);

/* ---- Batched tier ------------------------------------------------------
 * The pages' strided launch exists so that a multi-sequence Q/K/V tier can
 * hold it as one arm among several with their own pitches (page
 * "w8a16_gemm_pipelined_m32.rs", module doc and the doc comment of
 * `w8a16_gemm_pipelined_m32_strided`).  Here the arms run in one launch. */

/* Most GEMMs one batched call takes. */
#define W8A16_MAX_BATCH 8

/* One GEMM of a batch: the arguments of w8a16_gemm(), same meaning, layout
 * and ownership (device pointers owned by the caller). */
typedef struct w8a16_gemm_desc {
    const void *a;            /* BF16 [m, a_row_stride] */
    const void *w_fp8;        /* E4M3 [n, k] */
    const float *block_scale; /* FP32 [ceil(n/128), k/128] */
    void *c;                  /* BF16 [m, c_row_stride] */
    uint32_t a_row_stride;
    uint32_t c_row_stride;
    uint32_t m, n, k;
} w8a16_gemm_desc_t;

/* Plan of a batched call from the descriptors' m, n and k (pointers and
 * pitches are not read).  Pure: no GPU call.  One stream-kernel variant
 * serves every problem, without K splits; grid is the total workgroup
 * count, m_tiles the largest per problem and n_tiles the sum.  Errors:
 * W8A16_ERR_NULL_PTR (descs or out null), W8A16_ERR_BAD_PLAN (count not in
 * 1..W8A16_MAX_BATCH, or some m above 64), or the first failing problem's
 * w8a16_check_args() code, with its index in w8a16_last_error(). */
int w8a16_plan_batched(const w8a16_gemm_desc_t *descs, uint32_t count, uint32_t cu_count,
                       w8a16_plan_t *out);

/* `count` independent GEMMs (descs is a host array) in one launch of the
 * stream kernel on `stream`; problem i computes exactly what w8a16_gemm()
 * would with descs[i].  Each descriptor is checked as w8a16_gemm() checks
 * its arguments, in order; on the first failure nothing is launched and
 * that code is returned (index in w8a16_last_error()).  Asynchronous.  The
 * problems' outputs must not overlap each other or any input. */
int w8a16_gemm_batched(const w8a16_gemm_desc_t *descs, uint32_t count, void *stream);

/* ---- FP8 activations and the W8A8 GEMM ----------------------------------
 * The per-token FP8 activation quantizer of page "fp8_act_quant.rs" (one
 * group = 128 consecutive K elements of one token; tokens on grid X, groups
 * on grid Y) and the block-scaled GEMM that consumes its output.  The page
 * gives the grouping, not the arithmetic; the reading used: per (token,
 * group) s = amax / 448 and code = E4M3 round-to-nearest-even of x / s, both
 * divisions in binary32, saturated to +-448; an all-zero group gets s = 0
 * and zero codes. */

/* Quantize a: BF16 [m, a_row_stride] (first k of each row) into q: E4M3
 * [m, q_row_stride] (first k of each row written) and scales: FP32
 * [m, k/128] row-major.  Device pointers owned by the caller.  Errors, in
 * order: m == 0; k not a positive multiple of 128; a_row_stride or
 * q_row_stride below k (W8A16_ERR_PITCH_TOO_SHORT); a_row_stride not a
 * multiple of 8 or q_row_stride not a multiple of 16 (16-byte rows,
 * W8A16_ERR_A_STRIDE_ALIGN); a null pointer.  Nothing is launched on an
 * error.  Asynchronous on `stream`. */
int w8a16_act_quant_fp8(const void *a, uint32_t a_row_stride, void *q, uint32_t q_row_stride,
                        float *scales, uint32_t m, uint32_t k, void *stream);

/* Default plan of the W8A8 GEMM (kernel W8A16_KERNEL_W8A8).  Pure. */
int w8a16_plan_w8a8(uint32_t m, uint32_t n, uint32_t k, uint32_t cu_count,
                    w8a16_plan_t *out);

/*   C[i, j] = bf16( sum_b a_scales[i, b] * block_scale[j/128, b] *
 *                   sum_t qa[i, 128b + t] * w_fp8[j, 128b + t] )
 * qa: E4M3 [m, qa_row_stride]; a_scales: FP32 [m, k/128]; w_fp8 and
 * block_scale as for w8a16_gemm; c: BF16 [m, c_row_stride].  The two scales
 * are multiplied in FP32 and folded once per K step.  Checks as w8a16_gemm
 * with qa_row_stride in place of a_row_stride, which must be a multiple of
 * 16 (16-byte rows).  Asynchronous. */
int w8a16_gemm_w8a8(const void *qa, uint32_t qa_row_stride, const float *a_scales,
                    const void *w_fp8, const float *block_scale, void *c,
                    uint32_t c_row_stride, uint32_t m, uint32_t n, uint32_t k, void *stream);

/* w8a16_gemm_w8a8 with an explicit plan (kernel must be W8A16_KERNEL_W8A8;
 * m_blocks, n_blocks and waves taken from it).  For tests and tuning. */
int w8a16_gemm_w8a8_planned(const void *qa, uint32_t qa_row_stride, const float *a_scales,
                            const void *w_fp8, const float *block_scale, void *c,
                            uint32_t c_row_stride, uint32_t m, uint32_t n, uint32_t k,
                            const w8a16_plan_t *plan, void *stream);

/* ---- W4A4 MX projection GEMV ---------------------------------------------
 * The m-row W4A4 projection of page "w4a4_proj/mx_plan.rs" (up to 64 rows;
 * weight rows in 16-row tiles; tiers by m; activation reuse across weight
 * tiles; a persistent entry for wide weights).  The page states no number
 * format; the reading is OCP MXFP4 for both operands: FP4 E2M1 elements
 * (values 0, 0.5, 1, 1.5, 2, 3, 4, 6 and negatives), two per byte with the
 * even element in the low nibble, and one E8M0 scale byte (2^(e - 127)) per
 * 32 consecutive K elements of a row:
 *
 *   C[i][j] = bf16( sum_b 2^(ea[i][b]-127) * 2^(ew[j][b]-127) * sum_{t<32} a[i][32b+t] * w[j][32b+t] )
 *
 *   a        FP4   [m, a_row_stride]  elements; a row is a_row_stride / 2 bytes
 *   a_scale  E8M0  [m, k/32]          row-major, contiguous
 *   w_fp4    FP4   [n, k]             row-major, contiguous (k/2 bytes per row)
 *   w_scale  E8M0  [n, k/32]          row-major, contiguous
 *   c        BF16  [m, c_row_stride]  first n elements of each row written
 *
 * Products are exact, sums FP32 (the matrix cores apply the two block scales
 * to each 32-element partial), one round-to-nearest-even to BF16.  Device
 * pointers owned by the caller, 16-byte aligned.  Errors, in order: m == 0;
 * k not a positive multiple of 128; a_row_stride < k or c_row_stride < n;
 * a_row_stride not a multiple of 32 (16-byte rows); n == 0; k or
 * a_row_stride above 2^24 elements (W8A16_ERR_BAD_PLAN: the kernels address
 * a tile's rows through 32-bit buffer ranges); a null pointer; m above 64
 * (W8A16_ERR_BAD_PLAN).  No workspace.  Asynchronous. */
int w8a16_gemm_w4a4(const void *a, uint32_t a_row_stride, const uint8_t *a_scale,
                    const void *w_fp4, const uint8_t *w_scale, void *c, uint32_t c_row_stride,
                    uint32_t m, uint32_t n, uint32_t k, void *stream);

/* Default plan of the W4A4 GEMV (kernel W8A16_KERNEL_W4A4 or _W4A4_PS).
 * Pure: no GPU call. */
int w8a16_plan_w4a4(uint32_t m, uint32_t n, uint32_t k, uint32_t cu_count,
                    w8a16_plan_t *out);

/* w8a16_gemm_w4a4 with an explicit plan (kernel W8A16_KERNEL_W4A4:
 * m_blocks 1, 2 or 4 and n_blocks 1, 2 or 4, not both 4, with 4 waves, 8
 * waves up to m_blocks + n_blocks = 4, 16 waves for 1 x 1; kernel
 * W8A16_KERNEL_W4A4_PS: m_blocks 1, 2 or 4 covering m, 4, 8 or 16 waves,
 * and the staged activations plus two partial tiles per wave within the
 * LDS, else W8A16_ERR_BAD_PLAN).  For tests and tuning. */
int w8a16_gemm_w4a4_planned(const void *a, uint32_t a_row_stride, const uint8_t *a_scale,
                            const void *w_fp4, const uint8_t *w_scale, void *c,
                            uint32_t c_row_stride, uint32_t m, uint32_t n, uint32_t k,
                            const w8a16_plan_t *plan, void *stream);

/* ---- Attention between the projections -----------------------------------
 * What a decoder layer does between its Q/K/V and output projections:
 * rotary positions, a paged cache of keys and values held in FP8, and
 * attention over that cache.  Device pointers owned by the caller; calls are
 * asynchronous on `stream`.  Errors, in order: W8A16_ERR_ENV, then
 * W8A16_ERR_NULL_PTR, then W8A16_ERR_SHAPE; nothing is enqueued on an error.
 * A call with no tokens enqueues nothing and succeeds.  Strides of
 * activations are in elements, the last axis is contiguous, and rows need
 * only the alignment of their type (16-byte rows run fastest).  Rows of an
 * output must not overlap; strides shorter than a row are refused. */

typedef enum w8a16_dtype { W8A16_BF16 = 1, W8A16_FP16 = 2, W8A16_FP32 = 3 } w8a16_dtype;

/* Which elements of a head form a pair: i and i + rot_dim/2, or 2i and
 * 2i + 1 (i < rot_dim/2).  Elements from rot_dim on are not rotated. */
typedef enum w8a16_rope_layout {
    W8A16_ROPE_HALF = 0,
    W8A16_ROPE_INTERLEAVED = 1
} w8a16_rope_layout;

/* Frequencies of the rotation, f_i = base^(-2i / rot_dim), and how they are
 * stretched for contexts longer than the `original` positions a model was
 * trained on:
 *   LINEAR  f_i / factor
 *   BASE    base replaced by base * factor^(rot_dim / (rot_dim - 2))
 *   BANDS   with turns = original * f_i / (2 pi): f_i from high_turns up,
 *           f_i / factor up to low_turns, and between them
 *           f_i * (w + (1 - w) / factor), w = (turns - low_turns) / (high_turns - low_turns)
 * Cosines and sines are multiplied by `magnitude`. */
typedef enum w8a16_rope_scaling {
    W8A16_ROPE_PLAIN = 0,
    W8A16_ROPE_LINEAR = 1,
    W8A16_ROPE_BASE = 2,
    W8A16_ROPE_BANDS = 3
} w8a16_rope_scaling;

typedef struct w8a16_rope_config {
    double base, factor, original, low_turns, high_turns, magnitude;
    uint32_t scaling;         /* w8a16_rope_scaling */
} w8a16_rope_config_t;

/* table: FP32 [positions, rot_dim/2, 2], (cos, sin) of position * f_i,
 * computed in FP64 and rounded once.  rot_dim even, 2..1024 (4 and up for
 * BASE); base > 1; factor >= 1; for BANDS original > 0 and
 * 0 <= low_turns < high_turns. */
int w8a16_rope_table(const w8a16_rope_config_t *config, float *table, uint32_t positions,
                     uint32_t rot_dim, void *stream);

/* y = x rotated: for pair i of a head of the token at position p, with
 * (c, s) = table[p][i]:  y0 = x0 c - x1 s,  y1 = x1 c + x0 s, each product
 * and sum rounded to FP32, then once to the type.  inverse != 0 rotates by
 * -p, which is also the gradient of the forward rotation: dx from dy.
 * x, y: [tokens, heads, head_dim] of `dtype`; y may be x with the same
 * strides, and must not overlap it otherwise.  positions: int32 [tokens]; a
 * position outside the table gives NaN in that token's rotated elements. */
int w8a16_rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, void *y,
               int64_t y_token_stride, int64_t y_head_stride, uint32_t dtype, uint32_t tokens,
               uint32_t heads, uint32_t head_dim, const float *table, uint32_t table_positions,
               uint32_t rot_dim, const int32_t *positions, uint32_t layout, uint32_t inverse,
               void *stream);

/* Rotary positions of several axes: a token has a position on each of 1 to
 * W8A16_ROPE_MAX_AXES axes (a picture's or video's frame, row and column),
 * and each pair of a head turns by one of them.  Axis a has pairs[a] pairs
 * (0 is allowed); rot_dim is twice their sum, at most 1024.
 *   SPLIT  the first pairs[0] pairs are axis 0's, the next pairs[1] axis 1's, ...
 *   TURNS  pair i is axis a = i mod count's while i < count * pairs[a], else
 *          (and where a = 0) axis 0's.  Each axis a > 0 must find its pairs:
 *          a + count * (pairs[a] - 1) below the sum
 *   OWN    as SPLIT, and each axis counts its pairs from 0: the pair takes
 *          column i of the table for the i-th pair of its axis
 * In SPLIT and TURNS pair i takes column i. */
#define W8A16_ROPE_MAX_AXES 4
typedef enum w8a16_rope_order {
    W8A16_ROPE_SPLIT = 0,
    W8A16_ROPE_TURNS = 1,
    W8A16_ROPE_OWN = 2
} w8a16_rope_order;
typedef struct w8a16_axes {
    const int32_t *positions; /* token t on axis a: positions[a * axis_stride + t] */
    int64_t axis_stride;
    uint32_t count;           /* axes */
    uint32_t order;           /* w8a16_rope_order */
    uint32_t pairs[W8A16_ROPE_MAX_AXES];
    uint32_t table_pairs;     /* columns of the table: the sum of pairs; OWN: at least the largest */
} w8a16_axes_t;

/* w8a16_rope with a position per axis: with (c, s) =
 * table[positions[axis of i][t]][column of i] for pair i, the same formula,
 * roundings, gradient and errors.  table: FP32 [table_positions, table_pairs,
 * 2], at least one position; a position outside it gives NaN in its axis's
 * elements alone. */
int w8a16_rope_axes(const void *x, int64_t x_token_stride, int64_t x_head_stride, void *y,
                    int64_t y_token_stride, int64_t y_head_stride, uint32_t dtype, uint32_t tokens,
                    uint32_t heads, uint32_t head_dim, const float *table, uint32_t table_positions,
                    const w8a16_axes_t *axes, uint32_t layout, uint32_t inverse, void *stream);

/* The cache.  A page holds page_size tokens (a multiple of W8A16_KV_BLOCK up
 * to 1024) of every KV head; inside a page, blocks of 16 tokens of one head
 * share a scale.
 *   k        E4M3 [pages, kv_heads, page_size, head_dim]
 *   v        E4M3 [pages, kv_heads, page_size / 16, head_dim, 16]: the 16
 *            tokens of a block are adjacent for each channel
 *   k_scale, v_scale  E8M0 [pages, kv_heads, page_size / 16]: a code stands
 *            for code * 2^(byte - 127).  Bytes 1..254; a visible block whose
 *            byte is 0 or 255 (never written) gives NaN.
 * Page strides are in bytes, so that a cache may be a slice of a larger
 * one; everything inside a page is contiguous.  k and v 16-byte aligned,
 * their page strides multiples of 16; head_dim a multiple of 16 up to 256.
 * Slots past a sequence's length may hold anything. */
#define W8A16_KV_BLOCK 16
#define W8A16_KV_MAX_HEAD_DIM 256
typedef struct w8a16_kv_cache {
    void *k, *v;
    uint8_t *k_scale, *v_scale;
    uint64_t k_page_stride, v_page_stride, k_scale_page_stride, v_scale_page_stride;
    uint32_t pages, page_size, kv_heads, head_dim;
} w8a16_kv_cache_t;

/* The sequences of a call.  Sequence b brings new tokens
 * cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of the flat token axis (cu_seqlens
 * null: tokens / seqs each), n_b of them, and holds kv_lens[b] tokens in all,
 * the new ones among them: its new token j has position kv_lens[b] - n_b + j.
 * A token whose position is negative belongs to no sequence (an empty slot
 * of a padded batch), nor does one outside all of these ranges, or in a range
 * that decreases or ends past the token axis.  Its tokens i * page_size onwards are on page
 * block_table[b * block_table_stride + i], i < block_table_width.
 * max_new: at least the largest n_b.  All arrays int32. */
typedef struct w8a16_kv_seqs {
    const int32_t *block_table, *kv_lens, *cu_seqlens;
    uint32_t block_table_stride, block_table_width;
    uint32_t seqs, tokens, max_new;
} w8a16_kv_seqs_t;

/* New keys and values, and optionally queries to rotate by the same
 * positions.  k, v: [tokens, kv_heads, head_dim]; q, q_out: [tokens,
 * q_heads, head_dim] (q null: none; q_out may be q).  table null: no
 * rotation (then q must be null). */
typedef struct w8a16_kv_append_args {
    const void *k, *v, *q;
    void *q_out;
    int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride;
    int64_t q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride;
    const float *table;
    uint32_t table_positions, rot_dim, layout, dtype, q_heads;
} w8a16_kv_append_args_t;

/* Append: rotate each new key as w8a16_rope does (in FP32, not rounded to
 * the type), and store keys and values as codes.  For a block of 16 slots
 * that new tokens fall into, with A the largest finite magnitude among them:
 *   byte = max(smallest b >= 1 with A <= 448 * 2^(b - 127),
 *              the block's byte if it holds older tokens of the sequence)
 *   code = E4M3, nearest even, of x * 2^(127 - byte), saturated to +-448
 * NaN is stored as NaN.  If the byte grew, the older tokens' codes are
 * stored again for it, rounded once more only where they become subnormal.
 * Rotated queries are rounded once to the type; a query without a position
 * comes back as zeros.  Tokens past the block table, or whose page number is
 * outside the cache, are not stored.  Two sequences of a call must not
 * append to the same page. */
int w8a16_kv_append(const w8a16_kv_cache_t *cache, const w8a16_kv_seqs_t *seqs,
                    const w8a16_kv_append_args_t *args, void *stream);

/* w8a16_kv_append whose keys and queries turn by positions of several axes,
 * as in w8a16_rope_axes, in place of their place in the sequence (which still
 * says where they are stored).  args->table must be given, and args->rot_dim
 * be twice the axes' pairs. */
int w8a16_kv_append_axes(const w8a16_kv_cache_t *cache, const w8a16_kv_seqs_t *seqs,
                         const w8a16_kv_append_args_t *args, const w8a16_axes_t *axes, void *stream);

/* Launch plan of the attention. */
typedef enum w8a16_kv_kernel {
    /* Row kernel: a workgroup takes 16 (query, head) rows of one KV head
     * (row_blocks 1) and a chunk of the keys; its waves take interleaved
     * 64-key tiles straight from the cache into matrix operands.  The last
     * chunk of a row tile to finish joins them (at most 128). */
    W8A16_KV_ROWS = 1,
    /* Tile kernel: 128 rows (row_blocks 8), 32 per wave; K and V tiles of 64
     * keys are staged in LDS for the four waves. */
    W8A16_KV_TILE = 2
} w8a16_kv_kernel;
typedef struct w8a16_kv_plan {
    uint32_t kernel;          /* w8a16_kv_kernel */
    uint32_t row_blocks;      /* 16-row blocks per workgroup: rows 1, tile 8 */
    uint32_t waves;           /* waves per workgroup: 4; rows also 8, of heads up to 128 */
    uint32_t row_tiles;       /* row tiles of the longest sequence (derived) */
    uint32_t chunk_tiles;     /* 64-key tiles per chunk */
    uint32_t chunks;          /* chunks the longest sequence is cut into (derived) */
    uint32_t grid;            /* workgroups launched (derived) */
    uint64_t workspace_bytes; /* partial results (derived; 0 if chunks == 1, but for the two
                                 passes over a shared part, which always leave some) */
} w8a16_kv_plan_t;

/* For query row i of sequence b at position p = kv_lens[b] - n_b + i and
 * query head h, KV head h / (q_heads / kv_heads):
 *   out = sum_j softmax_j(scale * q . k_j) v_j,  lse = ln sum_j exp(scale * q . k_j)
 * over the visible keys j < kv_lens[b]; causal: j <= p; window > 0:
 * j > p - window.  A row that sees nothing gives zeros and lse = -inf, and so
 * does a token of no sequence.  What hidden places hold, NaN included,
 * changes nothing.  q, out: [tokens,
 * q_heads, head_dim] of `dtype` (BF16 or FP16); lse: FP32 [tokens, q_heads]
 * contiguous, or null.  max_kv: at least the largest kv_lens (0: the block
 * table's width); it shapes the launch only, longer sequences stay right.
 * scale: finite, not negative.  plan: null for the default. */
typedef struct w8a16_kv_attention_args {
    const void *q;
    void *out;
    float *lse;
    int64_t q_token_stride, q_head_stride, out_token_stride, out_head_stride;
    const w8a16_kv_plan_t *plan;
    float scale;
    uint32_t q_heads, dtype, causal, window, max_kv;
} w8a16_kv_attention_args_t;

/* Sums and softmax statistics are FP32.  In the sum of the values a weight,
 * times its block's V scale, is rounded to 11 bits, fewer below 2^-24 of the
 * row's largest such product and none from 2^-35 on.  Every order of addition
 * is fixed by the plan, so a plan gives the same bits on every run.  A plan
 * with chunks uses the (device, stream) workspace under the rules at the top
 * of this file (growth is refused during capture). */
int w8a16_kv_attention(const w8a16_kv_cache_t *cache, const w8a16_kv_seqs_t *seqs,
                       const w8a16_kv_attention_args_t *args, void *stream);

/* What more of the cache is seen, and what of it is read once.
 * sinks: the first tokens of a sequence that stay visible behind a window: a
 *   row sees key j < kv_lens[b] (causal: j <= p) if j > p - window or
 *   j < sinks.  Without a window it says nothing.
 * shared: at least two sequences hold the same first `shared` tokens, on the
 *   same pages: for every two of them, their rows of the block table agree on
 *   the pages of the first min(shared, the shorter one's kv_lens) tokens.
 *   The whole pages among them are read once for all rows where that pays.
 *   Results are those without it, up to the order of additions.  With a
 *   window it is not used.  A given plan is that of the second pass, over the
 *   keys from the shared part's last 64-key tile on, and asks for two passes;
 *   it has 4 waves and may have 64 chunks. */
typedef struct w8a16_kv_span {
    uint32_t sinks, shared;
} w8a16_kv_span_t;

/* w8a16_kv_attention() with a span (null: none).  A call that reads a shared
 * part once uses the workspace whatever its plan. */
int w8a16_kv_attention_span(const w8a16_kv_cache_t *cache, const w8a16_kv_seqs_t *seqs,
                            const w8a16_kv_attention_args_t *args, const w8a16_kv_span_t *span,
                            void *stream);

/* Default plans of the attention over a shared part (whole pages): of the
 * pass of all `tokens` rows over it, and of the pass over the sequences' own
 * keys; prefix->grid 0 where one pass over everything, with the plan in *own,
 * is as fast.  Pure: no GPU call. */
int w8a16_plan_kv_shared(uint32_t seqs, uint32_t tokens, uint32_t max_new, uint32_t max_kv,
                         uint32_t shared, uint32_t q_heads, uint32_t kv_heads, uint32_t head_dim,
                         uint32_t cu_count, w8a16_kv_plan_t *prefix, w8a16_kv_plan_t *own);

/* Default plan of the attention.  Pure: no GPU call. */
int w8a16_plan_kv_attention(uint32_t seqs, uint32_t max_new, uint32_t max_kv, uint32_t q_heads,
                            uint32_t kv_heads, uint32_t head_dim, uint32_t window,
                            uint32_t cu_count, w8a16_kv_plan_t *out);

/* The same of a window with sinks, whose tiles a plan's chunks have to cover as
 * well.  Pure: no GPU call. */
int w8a16_plan_kv_sinks(uint32_t seqs, uint32_t max_new, uint32_t max_kv, uint32_t q_heads,
                        uint32_t kv_heads, uint32_t head_dim, uint32_t window, uint32_t sinks,
                        uint32_t cu_count, w8a16_kv_plan_t *out);

/* ---- Product with an epilogue ---------------------------------------------
 *   c[i][j] = residual[i][j] + act(s + bias[j]) * gate[i][j]
 * with s the FP32 sum that w8a16_gemm() rounds, everything after it in FP32,
 * and one rounding to c's type; parts that are null are left out. */
typedef enum w8a16_activation {
    W8A16_ACT_NONE = 0,
    W8A16_ACT_RELU = 1,
    W8A16_ACT_SILU = 2,       /* x / (1 + exp(-x)) */
    W8A16_ACT_GELU = 3,       /* x (1 + erf(x / sqrt 2)) / 2 */
    W8A16_ACT_GELU_TANH = 4   /* x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) / 2 */
} w8a16_activation;

typedef struct w8a16_epilogue {
    const void *bias;         /* [n], contiguous */
    const void *gate;         /* BF16 [m, gate_row_stride] */
    const void *residual;     /* [m, residual_row_stride]; may be c, with c's type and stride */
    uint32_t gate_row_stride, residual_row_stride;   /* in elements, at least n */
    uint32_t activation;      /* w8a16_activation */
    uint32_t bias_dtype, residual_dtype, out_dtype;  /* w8a16_dtype: W8A16_BF16 or W8A16_FP32 */
} w8a16_epilogue_t;

/* w8a16_gemm() with an epilogue: same operands, plan, workspace and checks,
 * then W8A16_ERR_NULL_PTR (null epilogue), W8A16_ERR_SHAPE (an unknown
 * activation or type) and W8A16_ERR_PITCH_TOO_SHORT (a stride below n).  c:
 * [m, c_row_stride] of out_dtype, aligned to it like bias, gate and residual
 * to theirs.  c must not overlap another operand, but for residual as above. */
int w8a16_gemm_epilogue(const void *a, uint32_t a_row_stride, const void *w_fp8,
                        const float *block_scale, void *c, uint32_t c_row_stride, uint32_t m,
                        uint32_t n, uint32_t k, const w8a16_epilogue_t *epilogue, void *stream);

/* Static text for a status code (never null). */
const char *w8a16_status_string(int status);

/* Message of the calling thread's last failing call ("" if none). */
const char *w8a16_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* W8A16_H */
