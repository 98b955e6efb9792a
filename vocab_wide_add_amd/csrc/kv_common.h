// kv_common.h -- host checks shared by the operators over the paged cache.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "host_common.h"
#include "xpress_argmax.h"

namespace xpress {

inline int64_t element_bytes(int64_t dtype) { return dtype == XPRESS_E4M3 ? 1 : 2; }

inline bool is_aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// One dimension of a strided array: n places, `stride` elements apart.
struct Dim {
    int64_t n, stride;
};

// Elements from the first to the last of the array, both included, or -1
// when that passes 2^60; strides are not negative.
template <int K>
inline int64_t span_of(const Dim (&d)[K], int64_t inner)
{
    unsigned __int128 last = (unsigned __int128)inner;
    for (const Dim& x : d) {
        last += (unsigned __int128)(x.n - 1) * (unsigned __int128)x.stride;
    }
    return last > ((unsigned __int128)1 << 60) ? -1 : (int64_t)last;
}

// Whether no two elements share an address: with the dimensions ordered by
// stride, each stride passes everything below it.
template <int K>
inline bool is_disjoint(Dim (&d)[K], int64_t inner)
{
    for (int i = 1; i < K; ++i) {
        for (int j = i; j > 0 && d[j].stride < d[j - 1].stride; --j) {
            const Dim t = d[j];
            d[j] = d[j - 1];
            d[j - 1] = t;
        }
    }
    unsigned __int128 below = (unsigned __int128)inner;
    for (const Dim& x : d) {
        if (x.n <= 1) continue;
        if ((unsigned __int128)x.stride < below) return false;
        below += (unsigned __int128)(x.n - 1) * (unsigned __int128)x.stride;
    }
    return true;
}

// The layout and pointers of a cache's two arrays; *bytes receives the span of
// each.
inline bool pool_ok(const xpress_kv_cache& c, size_t* bytes)
{
    const int64_t most = 0x7FFFFFFFll;
    if (c.pages < 1 || c.pages > most || c.page_size < 1 || c.page_size > most || c.heads < 1 ||
        c.heads > 65536 || c.dim < 1 || c.dim > 65536) {
        return false;
    }
    if (c.dtype != XPRESS_BF16 && c.dtype != XPRESS_FP16 && c.dtype != XPRESS_E4M3) return false;
    if (c.stride_page < 1 || c.stride_head < 1 || c.stride_token < 1) return false;
    if (!c.k || !c.v || c.k == c.v) return false;
    const int64_t e = element_bytes(c.dtype);
    if (!is_aligned(c.k, (size_t)e) || !is_aligned(c.v, (size_t)e)) return false;
    if (c.dtype != XPRESS_E4M3 && (c.k_scale || c.v_scale)) return false;
    if (!is_aligned(c.k_scale, 4) || !is_aligned(c.v_scale, 4)) return false;
    Dim d[3] = {{c.pages, c.stride_page}, {c.heads, c.stride_head}, {c.page_size, c.stride_token}};
    const int64_t span = span_of(d, c.dim);
    if (span < 0 || !is_disjoint(d, c.dim)) return false;
    *bytes = (size_t)(span * e);
    return true;
}

// A table [seqs, width] of pages of page_size tokens: positions in 32 bits.
inline bool table_ok(const int32_t* table, int64_t seqs, int64_t width, int64_t stride, int64_t page_size)
{
    const int64_t most = 0x7FFFFFFFll;
    return seqs >= 0 && seqs <= most && page_size >= 1 && page_size <= most && width >= 1 &&
           width <= most / page_size && stride >= 0 && (seqs <= 1 || stride >= width) &&
           stride <= ((int64_t)1 << 58) / (seqs > 0 ? seqs : 1) && table && is_aligned(table, 4);
}

// The layout and pointers of a cache with its table; *bytes as above.
inline bool cache_ok(const xpress_kv_cache& c, size_t* bytes)
{
    const int64_t most = 0x7FFFFFFFll;
    if (c.page_size < 1 || c.seqs < 0 || c.seqs > most || c.table_width < 1 ||
        c.table_width > most / c.page_size) {
        return false;
    }
    if (c.stride_table < 0 || (c.seqs > 1 && c.stride_table < c.table_width)) return false;
    if (!c.page_table || !is_aligned(c.page_table, 4)) return false;
    return pool_ok(c, bytes);
}

// Bytes from a table's first entry to its last.
inline size_t table_bytes(int64_t seqs, int64_t width, int64_t stride)
{
    return seqs > 0 ? (size_t)((seqs - 1) * stride + width) * 4u : 0;
}

// Whether [p, p + n) lies apart from both arrays of the cache (a null p does).
inline bool apart_from_cache(const xpress_kv_cache& c, size_t cache_bytes, const void* p, size_t n)
{
    return !p || !(ranges_overlap(c.k, cache_bytes, p, n) || ranges_overlap(c.v, cache_bytes, p, n));
}

}  // namespace xpress
