// Attention of a batch whose sequences share their first tokens.
//
// A softmax over the shared keys and each sequence's own is the two parts'
// softmaxes joined by their running references: with (m, l, O) of each chunk
// of keys, l = sum 2^(m_c - m) l_c and O likewise, so the shared keys can be
// gone over once for all rows of the batch, as if they were one sequence's,
// and each sequence's own keys apart.  Every chunk of either pass leaves its
// partial rows and a second launch adds them, a wave per row: the prefix's
// row tiles hold rows of many sequences, so no workgroup of the first launch
// could do that for its own rows alone.
//
// Both passes are one launch, the prefix's workgroups in front: where its
// rows fill tiles (32 and more of a head) that pass is bound by its
// instructions and the other by reading the cache, so a CU that holds one of
// each has both its parts at work.
//
// What bounds it: few sequences, the chain of a workgroup's first loads
// (lengths, table, tiles), a few tiles, and the second launch; many rows, the
// prefix's products, whose matrix instructions and widening of codes run at
// the tile kernel's rate; in between both, and reading the own keys.
// Measured, 32 query and 8 KV heads of 128 channels, one new token: 6
// sequences of up to 333 own tokens behind 1984 shared ones 11.8 us (8.0 and
// 3.8 for the join; as two launches and a join 20.5), in one pass over
// everything 12.0; 64 of up to 512 behind 8192 31.5 (26 and 6.5; 41.0),
// reading 67 MB of HBM where 60 are the least, in one pass 85.5.  24 sequences
// of 4 new tokens, 64 query heads, 101 own tokens behind 30016: 123 to 128
// (130; the products alone 78 at a library's rate), in one pass 284.  In the middle case a prefix workgroup takes 6 us to its first
// products, 15 for 8 tiles beside the own keys' workgroups and 2 for its
// partial rows.  Tried there: the first tiles' loads before the rows' ranges
// 31.2, partial rows through LDS, by whole rows, 31.4; in the last, eight
// pieces ahead in the join in place of four 126.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv_rows_kernel.h"
#include "kv_tile_kernel.h"

namespace w8a16 {

namespace {

using namespace dev;

struct SharedArgs {
    SuffixArgs own;
    PrefixArgs prefix;
};
constexpr size_t kPrefixAt = sizeof(SuffixArgs);     // bytes into SharedArgs
static_assert(kPrefixAt % alignof(PrefixArgs) == 0 && sizeof(SharedArgs) == kPrefixAt + sizeof(PrefixArgs),
              "the members of SharedArgs");

// PT, ST: the prefix's and the own keys' pass take the tile kernel (else the
// row kernel, four waves).
template <class Q, int DP, bool PT, bool ST>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void w8a16_kv_shared_kernel(SharedArgs s)
{
#ifdef __HIP_DEVICE_COMPILE__     // (the host's pass knows no DMA builtin, and instantiates what it is shown)
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    auto &r = *reinterpret_cast<rows::RowsLds<DP, 4> *>(lds);
    if (blockIdx.x < s.prefix.grid) {
        if constexpr (PT)
            tile::kv_tile<Q, DP, kPrefixAt>(s.prefix, blockIdx.x, lds);
        else
            rows::kv_rows<Q, DP, 4>(s.prefix, blockIdx.x, r);
    } else {
        if constexpr (ST)
            tile::kv_tile<Q, DP, 0>(s.own, blockIdx.x - s.prefix.grid, lds);
        else
            rows::kv_rows<Q, DP, 4>(s.own, blockIdx.x - s.prefix.grid, r);
    }
#endif
}

template <class Q, int DP, bool PT, bool ST>
hipError_t launch_parts(const SharedArgs &s, hipStream_t stream)
{
    constexpr uint32_t rows_bytes = sizeof(rows::RowsLds<DP, 4>);
    constexpr uint32_t bytes = (PT || ST) && tile::tile_lds<DP> > rows_bytes ? tile::tile_lds<DP> : rows_bytes;
    static std::atomic<uint64_t> lds_set{0};
    auto kern = w8a16_kv_shared_kernel<Q, DP, PT, ST>;
    hipError_t e = allow_lds(reinterpret_cast<const void *>(kern), bytes, bytes, lds_set);
    if (e != hipSuccess)
        return e;
    const uint32_t grid = s.prefix.grid + (uint32_t)kv_launch_groups(s.own, 4);
    hipLaunchKernelGGL(kern, dim3(grid), dim3(256), bytes, stream, s);
    return hipGetLastError();
}

template <class Q, int DP>
hipError_t launch_dim(const SharedArgs &s, bool pt, bool st, hipStream_t stream)
{
    if (st)
        return pt ? launch_parts<Q, DP, true, true>(s, stream) : hipErrorInvalidValue;
    return pt ? launch_parts<Q, DP, true, false>(s, stream) : launch_parts<Q, DP, false, false>(s, stream);
}

template <class Q>
hipError_t launch_type(const SharedArgs &s, bool pt, bool st, hipStream_t stream)
{
    switch ((s.own.pool.dim + 63u) / 64u) {
    case 1: return launch_dim<Q, 64>(s, pt, st, stream);
    case 2: return launch_dim<Q, 128>(s, pt, st, stream);
    case 3: return launch_dim<Q, 192>(s, pt, st, stream);
    default: return launch_dim<Q, 256>(s, pt, st, stream);
    }
}

}  // namespace

hipError_t launch_kv_shared(const PrefixArgs &a, const w8a16_kv_plan_t &pa, const SuffixArgs &b,
                            const w8a16_kv_plan_t &pb, uint32_t max_rows, uint32_t dtype, hipStream_t stream)
{
    SharedArgs s;
    s.prefix = a;
    s.own = b;
    const bool pt = pa.kernel == W8A16_KV_TILE, st = pb.kernel == W8A16_KV_TILE;
    hipError_t e = dtype == W8A16_BF16 ? launch_type<QueryBf16>(s, pt, st, stream)
                                       : launch_type<QueryF16>(s, pt, st, stream);
    return e == hipSuccess ? launch_kv_join(b, pb, max_rows, dtype, stream) : e;
}

}  // namespace w8a16
