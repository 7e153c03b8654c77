// Rotation of one row's items, shared by the rotation kernel and the append
// kernel's queries.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention.h"

namespace w8a16 {
namespace dev {

template <class T> __device__ __forceinline__ float to_f32(T x) { return static_cast<float>(x); }

template <class T, int N> struct Vec {
    typedef T type __attribute__((ext_vector_type(N)));
};

// y0 = x0 c - x1 s, y1 = x1 c + x0 s with every product and sum rounded by
// itself: a contracted multiply-add would round differently from the same
// formula written in separate operations, and codes quantised from the
// result would then differ in rare ties.
__device__ __forceinline__ void rotate(float x0, float x1, float c, float s, float &y0, float &y1)
{
#pragma clang fp contract(off)
    const float a = x0 * c, b = x1 * s, d = x1 * c, e = x0 * s;
    y0 = a - b;
    y1 = d + e;
}

// The sequence of token t and its position; false if no sequence owns t.
__device__ __forceinline__ bool token_place(const KvSeqs &s, uint32_t t, uint32_t &b, int32_t &pos)
{
    uint32_t first, end;
    if (s.cu) {
        // last b with cu[b] <= t
        uint32_t lo = 0, hi = s.seqs;
        while (hi - lo > 1) {
            const uint32_t mid = (lo + hi) / 2;
            if ((uint32_t)s.cu[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        b = lo;
        first = (uint32_t)s.cu[b];
        end = (uint32_t)s.cu[b + 1];
        if (t < first || t >= end || end > s.tokens)
            return false;
    } else {
        b = s.by_uniform.div(t);
        first = b * s.uniform;
        end = first + s.uniform;
    }
    pos = s.kv_lens[b] - (int32_t)(end - t);
    return pos >= 0;
}

// Item `item` of N heads from head `h` on (those below r.heads): P pairs, or
// 2P elements past rot.  T: element type; x, y: the token's rows; cs: the
// position's table row, null for a position outside the table.  The heads'
// loads are issued together and share the cosines and sines.
template <class T, int P, int N, bool HALF>
__device__ __forceinline__ void rope_heads(const RopeRows &r, const T *x, T *y, uint32_t h, uint32_t item,
                                           const float *cs, bool inverse)
{
    typedef typename Vec<T, P>::type V;
    x += (int64_t)h * r.x_head;
    y += (int64_t)h * r.y_head;
    const bool pair = item < r.pair_items;
    const uint32_t p0 = item * P;
    uint32_t e0, e1;
    if (pair) {
        e0 = HALF ? p0 : 2 * p0;
        e1 = HALF ? p0 + r.rot / 2 : 2 * p0 + P;
    } else {
        e0 = r.rot + (item - r.pair_items) * (2 * P);
        e1 = e0 + P;
        if (x == y)
            return;
        if (P == 1) {   // the last item may hold one element
            for (int n = 0; n < N && h + n < r.heads; ++n)
                for (uint32_t i = e0; i < e0 + 2 && i < r.dim; ++i)
                    y[(int64_t)n * r.y_head + i] = x[(int64_t)n * r.x_head + i];
            return;
        }
    }
    V a[N], b[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const T *row = x + (h + n < r.heads ? (int64_t)n * r.x_head : 0);
        a[n] = *reinterpret_cast<const V *>(row + e0);
        b[n] = *reinterpret_cast<const V *>(row + e1);
    }
    if (pair) {
        float c[P], s[P];
        const float nan = __builtin_nanf("");
#pragma unroll
        for (int i = 0; i < P; ++i) {
            c[i] = cs ? cs[2 * (p0 + i)] : nan;
            s[i] = cs ? cs[2 * (p0 + i) + 1] : nan;
            s[i] = inverse ? -s[i] : s[i];
        }
        constexpr bool apart = HALF || P == 1;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            // adjacent pairs: the first P/2 of them are in a, the others in b
            float u[2 * P], v[2 * P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                u[i] = to_f32(a[n][i]);
                u[P + i] = to_f32(b[n][i]);
            }
#pragma unroll
            for (int i = 0; i < P; ++i)
                rotate(apart ? u[i] : u[2 * i], apart ? u[P + i] : u[2 * i + 1], c[i], s[i], v[2 * i],
                       v[2 * i + 1]);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                a[n][i] = static_cast<T>(apart ? v[2 * i] : v[i]);
                b[n][i] = static_cast<T>(apart ? v[2 * i + 1] : v[P + i]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
        if (h + n < r.heads) {
            *reinterpret_cast<V *>(y + (int64_t)n * r.y_head + e0) = a[n];
            *reinterpret_cast<V *>(y + (int64_t)n * r.y_head + e1) = b[n];
        }
}

}  // namespace dev
}  // namespace w8a16
