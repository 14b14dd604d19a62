// cache_rows.cuh -- the columns of a call's caches: one vector (16 bytes, or 8) of a row
// of one head and layer, at every page and slot.  Moving rows moves each column for itself,
// so threads never wait for one another.
#pragma once

#include <cstdint>

#include "fdec_internal.h"

namespace fdec {

// The cache whose columns block `blk` holds.
template <int N>
__device__ __forceinline__ const CacheRows& cache_of(const CacheList<N>& list, int blk) {
    int lo = 0, hi = list.n - 1;  // the last cache that begins at or before blk
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (list.c[mid].first_block <= blk)
            lo = mid;
        else
            hi = mid - 1;
    }
    return list.c[lo];
}

// Move rows of the block's columns: row i in [begin, end) from (page, slot) `from(i)` to
// `to(i)`, in this order but for the loads of V rows, which come before their stores: a
// row may be stored where a later one was read, not the other way round.
template <typename V, typename From, typename To>
__device__ __forceinline__ void move_columns(const CacheRows& c, int blk, int begin, int end, From from, To to) {
    constexpr int U = kRowsAhead;
    const int64_t columns = static_cast<int64_t>(c.layers) * c.heads * c.row_vecs;
    const int64_t x = static_cast<int64_t>(blk - c.first_block) * kColumnThreads + threadIdx.x;
    if (x >= columns) return;
    const int64_t lh = x / c.row_vecs;
    const int64_t layer = lh / c.heads;
    uint8_t* col = c.base + layer * c.s_layer + (lh - layer * c.heads) * c.s_head + (x - lh * c.row_vecs) * sizeof(V);
    for (int i0 = begin; i0 < end; i0 += U) {
        V val[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u >= end) break;
            const int2 f = from(i0 + u);  // (page, slot), page < 0: not moved
            if (f.x >= 0) val[u] = *reinterpret_cast<const V*>(col + f.x * c.s_page + f.y * c.s_token);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u >= end) break;
            const int2 f = from(i0 + u), t = to(i0 + u);
            if (f.x >= 0) *reinterpret_cast<V*>(col + t.x * c.s_page + t.y * c.s_token) = val[u];
        }
    }
}

// The first N caches of a list (kernel arguments are copied with every launch).
template <int N>
inline CacheList<N> shorter(const CacheList<kMaxCaches>& list) {
    CacheList<N> out = {};
    out.n = list.n;
    for (int i = 0; i < list.n; ++i) out.c[i] = list.c[i];
    return out;
}

// Blocks of columns of a list.
inline int64_t column_blocks(const CacheList<kMaxCaches>& list) {
    if (list.n == 0) return 0;
    const CacheRows& c = list.c[list.n - 1];
    const int64_t columns = static_cast<int64_t>(c.layers) * c.heads * c.row_vecs;
    return c.first_block + (columns + kColumnThreads - 1) / kColumnThreads;
}

}  // namespace fdec
