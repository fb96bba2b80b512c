// tdg_paged.cuh -- what the operators on the paged key-value cache share: the
// cache as kernels see it, the address of a page's rows, and the host checks.
#pragma once

#include <cuda_fp8.h>
#include <math.h>
#include <string.h>

#include "tdg_internal.h"

namespace tdg {

struct PagedView {
    uint8_t *regions;
    uint64_t region_bytes, k_off, v_off;
    const float *k_scale, *v_scale;
    int64_t pages;     // per rank
    int64_t all_pages; // world * pages
    int Hkv, D;
    int ps_log2;       // log2(page_size)
};

// Byte offset, inside its region's pool, of slot `slot` of head `h` in page
// `local`; esz bytes per element.
__device__ __forceinline__ uint64_t paged_row(const PagedView &c, int64_t local, int h, int slot, int esz)
{
    return ((((uint64_t)local * c.Hkv + h) << c.ps_log2) + slot) * (uint64_t)(c.D * esz);
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

} // namespace tdg

namespace tdg_host {

inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline bool page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256; }

inline bool overlap(uint64_t a, uint64_t an, uint64_t b, uint64_t bn) { return a < b + bn && b < a + an; }

// Checks a cache description against the heap and fills the kernels' view.
inline int paged_view(const tdg_symm *h, const tdg_paged_cache &c, tdg::PagedView &v)
{
    if (c.pages <= 0 || c.pages > INT32_MAX || (int64_t)h->world * c.pages > INT32_MAX ||
        c.Hkv <= 0 || c.pages > INT32_MAX / c.Hkv || c.k_off % 1024 ||
        c.v_off % 1024)
        return TDG_ERR_INVALID;
    const uint64_t pool = tdg_paged_pool_bytes(c.pages, c.page_size, c.Hkv, c.D, c.kv_type);
    if (!pool)
        return TDG_ERR_INVALID;
    const bool e4m3 = c.kv_type == TDG_KV_E4M3;
    if ((c.k_scale != nullptr) != e4m3 || (c.v_scale != nullptr) != e4m3 || !aligned4(c.k_scale) || !aligned4(c.v_scale))
        return TDG_ERR_INVALID;
    const uint64_t R = h->region_bytes;
    if (pool > R || c.k_off > R - pool || c.v_off > R - pool)
        return TDG_ERR_NOMEM;
    if (overlap(c.k_off, pool, c.v_off, pool))
        return TDG_ERR_INVALID;
    v.regions = h->base;
    v.region_bytes = R;
    v.k_off = c.k_off;
    v.v_off = c.v_off;
    v.k_scale = c.k_scale;
    v.v_scale = c.v_scale;
    v.pages = c.pages;
    v.all_pages = (int64_t)h->world * c.pages;
    v.Hkv = (int)c.Hkv;
    v.D = (int)c.D;
    v.ps_log2 = __builtin_ctz((unsigned)c.page_size);
    return TDG_OK;
}

inline bool table_ok(const int32_t *table, int64_t entries, int64_t stride, int page_size)
{
    return table && aligned4(table) && entries >= 0 && stride >= entries && entries <= INT32_MAX / page_size &&
           stride <= INT32_MAX;
}

// `rows` rows of `width` elements, `stride` elements apart: strides and pointer alignment
inline bool rows_ok(const void *p, int64_t stride, int64_t width)
{
    return p && aligned16(p) && stride % 8 == 0 && stride >= width;
}

// bytes from the first to past the last element of `rows` bf16 rows
inline uint64_t rows_extent(int64_t rows, int64_t stride, int64_t width)
{
    return rows <= 0 ? 0 : ((uint64_t)(rows - 1) * stride + width) * 2;
}

inline bool rows_overlap(const void *a, uint64_t an, const void *b, uint64_t bn)
{
    return a && b && an && bn && overlap(reinterpret_cast<uintptr_t>(a), an, reinterpret_cast<uintptr_t>(b), bn);
}

// Whether two sets of rows (an and bn of them; bf16, widths and strides in
// elements) share an element; columns of one buffer (equal strides) are told apart.
inline bool rows_clash(int64_t an, const void *a, int64_t as, int64_t aw, int64_t bn, const void *b, int64_t bs, int64_t bw)
{
    if (!a || !b || aw <= 0 || bw <= 0 || !rows_overlap(a, rows_extent(an, as, aw), b, rows_extent(bn, bs, bw)))
        return false;
    if (as != bs || as <= 0)
        return true;
    int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)) / 2 % as;
    if (d < 0)
        d += as;
    return d < aw || d + bw > as;
}

// Bytes that a call writes or reads.
struct Range {
    const void *at;
    uint64_t bytes;
};

template <int A, int B> bool ranges_overlap(const Range (&a)[A], const Range (&b)[B])
{
    for (const Range &x : a)
        for (const Range &y : b)
            if (rows_overlap(x.at, x.bytes, y.at, y.bytes))
                return true;
    return false;
}

// whether a range reaches into a pool of any rank
template <int A> bool pools_overlap(const tdg_symm *h, const tdg_paged_cache &c, const Range (&a)[A])
{
    const uint64_t pool = tdg_paged_pool_bytes(c.pages, c.page_size, c.Hkv, c.D, c.kv_type);
    for (const Range &x : a) {
        if (!rows_overlap(x.at, x.bytes, h->base, h->world * h->region_bytes)) // outside the heap, as most are
            continue;
        for (int r = 0; r < h->world; ++r) {
            const uint8_t *region = h->base + (uint64_t)r * h->region_bytes;
            if (rows_overlap(x.at, x.bytes, region + c.k_off, pool) || rows_overlap(x.at, x.bytes, region + c.v_off, pool))
                return true;
        }
    }
    return false;
}

inline Range table_range(const int32_t *table, int64_t rows, int64_t entries, int64_t stride)
{
    return {table, rows <= 0 ? 0 : ((uint64_t)(rows - 1) * stride + entries) * 4};
}

// the scales of an 8-bit cache (none otherwise)
inline uint64_t scale_bytes(const tdg_paged_cache &c) { return c.kv_type == TDG_KV_E4M3 ? (uint64_t)c.Hkv * 4 : 0; }

} // namespace tdg_host
