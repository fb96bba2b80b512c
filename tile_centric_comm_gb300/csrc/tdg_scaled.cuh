// tdg_scaled.cuh -- what the 8-bit operators and the MoE gradients share: the
// rows that a token's choices stand for, and host checks of strides and ranges.
#pragma once

#include "tdg_paged.cuh"

namespace tdg {

// The tokens of every rank and the receive rows of their choices.
struct MoeRows {
    DevStatus *status;
    uint32_t epoch;
    int k;
    int64_t T, H, tokens, rows; // tokens: world * T; rows: world * T * k
    uint8_t *regions;
    uint64_t region_bytes;
    const int64_t *slot;
};

// The receive row of choice kk of token tok (src * T + t), or -1.  `tells`:
// the one thread that reports a row outside the buffer.
__device__ __forceinline__ int64_t moe_row(const MoeRows &m, int64_t tok, int kk, bool tells)
{
    const int64_t row = m.slot[tok * m.k + kk];
    if (row >= 0 && row < m.rows)
        return row;
    if (row != -1 && tells)
        report_fault(m.status, TDG_ERR_DEVICE, TDG_WHERE_SLOT, (uint32_t)(tok * m.k + kk), m.epoch);
    return -1;
}

} // namespace tdg

namespace tdg_host {

inline bool aligned8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// a row stride in elements: a multiple of `unit`, at least the row's extent
inline bool stride_ok(int64_t stride, int64_t width, int64_t unit)
{
    return stride >= width && stride % unit == 0 && stride <= INT32_MAX;
}

// bytes from the first to past the last element of `rows` rows
inline uint64_t extent(int64_t rows, int64_t stride, int64_t width, int esz)
{
    return rows <= 0 ? 0 : ((uint64_t)(rows - 1) * stride + width) * esz;
}

// `n` rows of a matrix, stride and width in bytes
struct ByteRows {
    const void *at;
    int64_t stride, width;
};
// Whether two matrices of n rows share a byte; columns of one buffer (equal
// strides) are told apart.  All sizes here are even, for rows_clash's units of 2.
inline bool rows_share(int64_t n, const ByteRows &a, const ByteRows &b)
{
    return rows_clash(n, a.at, a.stride / 2, a.width / 2, n, b.at, b.stride / 2, b.width / 2);
}

inline bool in_region(const tdg_symm *h, uint64_t off, uint64_t bytes)
{
    return bytes <= h->region_bytes && off <= h->region_bytes - bytes;
}

// whether a range reaches into [off, off + bytes) of any rank's region
template <int A> bool shards_overlap(const tdg_symm *h, uint64_t off, uint64_t bytes, const Range (&a)[A])
{
    for (const Range &x : a) {
        if (!rows_overlap(x.at, x.bytes, h->base, h->world * h->region_bytes)) // outside the heap
            continue;
        for (int r = 0; r < h->world; ++r)
            if (rows_overlap(x.at, x.bytes, h->base + (uint64_t)r * h->region_bytes + off, bytes))
                return true;
    }
    return false;
}

// The checks that the calls over a token's choices share; fills all but the epoch.
inline int moe_rows(const tdg_symm *h, int world, int k, int64_t T, int64_t H, const int64_t *slot, int unit, tdg::MoeRows &m)
{
    if (world != h->world || T < 0 || T > INT32_MAX || k < 1 || k > 32 || H < unit || H % unit || H >= (1 << 30) ||
        (int64_t)world * T * k >= INT32_MAX || !aligned8(slot))
        return TDG_ERR_INVALID;
    m.status = h->status;
    m.epoch = 0;
    m.k = k;
    m.T = T;
    m.H = H;
    m.tokens = (int64_t)world * T;
    m.rows = m.tokens * k;
    m.regions = h->base;
    m.region_bytes = h->region_bytes;
    m.slot = slot;
    return TDG_OK;
}

} // namespace tdg_host
