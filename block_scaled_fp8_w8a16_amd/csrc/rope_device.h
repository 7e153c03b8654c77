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
        if (t < first || t >= end)
            return false;
    } else {
        b = s.by_uniform.div(t);
        first = b * s.uniform;
        end = first + s.uniform;
    }
    pos = s.kv_lens[b] - (int32_t)(end - t);
    return pos >= 0;
}

// Item `item` of one head row: P pairs, or 2P elements past rot.  T: element
// type.  cs: the position's table row, null for a position outside the table.
template <class T, int P>
__device__ __forceinline__ void rope_item(const RopeRows &r, const T *x, T *y, uint32_t item,
                                          const float *cs, bool inverse)
{
    typedef typename Vec<T, P>::type V;
    if (item >= r.pair_items) {
        const uint32_t e = r.rot + (item - r.pair_items) * (2 * P);
        if (P == 1) {   // an odd tail is possible: one element at a time
            if (x != y)
                for (uint32_t i = e; i < e + 2 && i < r.dim; ++i)
                    y[i] = x[i];
            return;
        }
        if (x != y) {
            const V a = *reinterpret_cast<const V *>(x + e), b = *reinterpret_cast<const V *>(x + e + P);
            *reinterpret_cast<V *>(y + e) = a;
            *reinterpret_cast<V *>(y + e + P) = b;
        }
        return;
    }
    const uint32_t p0 = item * P;
    const uint32_t e0 = r.half ? p0 : 2 * p0, e1 = r.half ? p0 + r.rot / 2 : 2 * p0 + P;
    const V a = *reinterpret_cast<const V *>(x + e0), b = *reinterpret_cast<const V *>(x + e1);
    float c[P], s[P];
    const float nan = __builtin_nanf("");
#pragma unroll
    for (int i = 0; i < P; ++i) {
        c[i] = cs ? cs[2 * (p0 + i)] : nan;
        s[i] = cs ? cs[2 * (p0 + i) + 1] : nan;
        if (inverse)
            s[i] = -s[i];
    }
    float u[P], v[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        u[i] = to_f32(a[i]);
        v[i] = to_f32(b[i]);
    }
    V ya, yb;
    if (r.half || P == 1) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float y0, y1;
            rotate(u[i], v[i], c[i], s[i], y0, y1);
            ya[i] = static_cast<T>(y0);
            yb[i] = static_cast<T>(y1);
        }
    } else {
        // pairs are adjacent: the first P/2 in a, the others in b
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int j = 2 * i;
            float y0, y1;
            if (j < P) {
                rotate(u[j], u[j + 1 < P ? j + 1 : 0], c[i], s[i], y0, y1);
                ya[j] = static_cast<T>(y0);
                ya[j + 1 < P ? j + 1 : 0] = static_cast<T>(y1);
            } else {
                rotate(v[j - P], v[j + 1 - P], c[i], s[i], y0, y1);
                yb[j - P] = static_cast<T>(y0);
                yb[j + 1 - P] = static_cast<T>(y1);
            }
        }
    }
    *reinterpret_cast<V *>(y + e0) = ya;
    *reinterpret_cast<V *>(y + e1) = yb;
}

}  // namespace dev
}  // namespace w8a16
