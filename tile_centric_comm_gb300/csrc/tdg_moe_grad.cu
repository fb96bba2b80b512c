// tdg_moe_grad.cu -- the gradients of the MoE dispatch and combine.
//
//   combine:  dy[slot(t,kk)] = gate[t][kk] dout[t],  dgate[t][kk] = <dout[t], y[slot(t,kk)]>
//   dispatch: dx[t] = sum_kk drecv[slot(t,kk)]
//
// Bound by memory: every row of dout, y and drecv is read once, every row of
// dy and dx written once.  A token's threads, a warp to a CTA, hold 8 elements of
// dout each while they walk over the token's rows, so that dy and the partial
// sums of dgate come from one pass.  No atomics: the sums' order is fixed by
// the call's sizes.
// 8192 tokens of 7168 with 8 rows each, both gradients: 464 us, 6.6 TB/s.  Few
// long tokens are bound by latency, since a token has one CTA at most: 1 of them
// 11.5 us, 128 17.3.
#include <type_traits>

#include "tdg_scaled.cuh"

namespace tdg {

namespace mg {
constexpr int THREADS = 256;
constexpr int GROUP = 8; // rows whose loads are in flight together

// The threads of a token.  Many tokens: few threads, so that short rows leave none
// idle and the ends of all rows are short (both gradients by 32, 64, 128 and 256 in
// us; 32768 tokens of 256, 2 rows each 38, 63, 107 and 192; 8192 of 1032, 8 rows each
// 99, 97, 103 and 112; 8192 of 7168 513, 481, 468 and 478).  Few tokens: more, up to
// what holds a row at once (128 tokens of 7168 84, 45, 25 and 17; 514 of 520, 2 rows
// each 7.4, 6.4, 5.5 and 6.0).
inline int threads_of(const MoeRows &m, int sms)
{
    int threads = m.H < 1024 ? 32 : m.H < 2048 ? 64 : 128;
    while (threads < THREADS && threads * 8 < m.H && m.tokens * threads < (int64_t)4 * sms * THREADS)
        threads *= 2;
    return threads;
}
} // namespace mg

__device__ __forceinline__ void widen8(const uint4 &u, float (&f)[8])
{
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __bfloat1622float2(h[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}

__device__ __forceinline__ uint4 narrow8(const float (&f)[8])
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// A row of this call's own: read once, past L1.  dy may be y: not through the read-only
// path, and with "memory", since the stores to dy do not depend on the values read from
// y and nothing else keeps them behind these loads.
__device__ __forceinline__ uint4 ld_row(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// G threads a token
template <int G>
__global__ void __launch_bounds__(mg::THREADS) moe_combine_grad_kernel(const __grid_constant__ MoeRows m, uint64_t gate_off, uint64_t dout_off,
                                                                      uint64_t dgate_off, const uint8_t *y, uint8_t *dy)
{
    constexpr int TOKENS = mg::THREADS / G;
    __shared__ int64_t rows[TOKENS][32];
    __shared__ float gates[TOKENS][32], part[mg::THREADS / 32][32];
    griddep_launch_dependents();
    griddep_wait();
    const int own = threadIdx.x / G, at = threadIdx.x % G, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t *row = rows[own];
    float *gate = gates[own];
    const uint32_t tok32 = blockIdx.x * TOKENS + own, src = tok32 / (uint32_t)m.T;
    const bool in = tok32 < (uint64_t)m.tokens;
    const int64_t tok = tok32, t = tok32 - src * (uint32_t)m.T;
    uint8_t *region = m.regions + (uint64_t)src * m.region_bytes;
    if (in && at < m.k) {
        row[at] = moe_row(m, tok, at, true);
        gate[at] = reinterpret_cast<const float *>(region + gate_off)[t * m.k + at];
    }
    __syncthreads();
    const uint64_t row_bytes = (uint64_t)m.H * 2;
    const uint8_t *dout = region + dout_off + (uint64_t)t * row_bytes;
    const int64_t vecs = in ? m.H / 8 : 0;
    for (int k0 = 0; k0 < m.k; k0 += mg::GROUP) {
        float dot[mg::GROUP] = {};
        for (int64_t v = at; v < vecs; v += G) {
            uint4 yv[mg::GROUP];
            const uint4 dv = *reinterpret_cast<const uint4 *>(dout + v * 16);
#pragma unroll
            for (int j = 0; j < mg::GROUP; ++j)
                if (k0 + j < m.k && row[k0 + j] >= 0)
                    yv[j] = ld_row(y + (uint64_t)row[k0 + j] * row_bytes + v * 16);
            float d[8];
            widen8(dv, d);
#pragma unroll
            for (int j = 0; j < mg::GROUP; ++j) {
                if (k0 + j < m.k && row[k0 + j] >= 0) {
                    float f[8], o[8];
                    widen8(yv[j], f);
                    const float g = gate[k0 + j];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dot[j] = fmaf(d[i], f[i], dot[j]);
                        o[i] = g * d[i];
                    }
                    *reinterpret_cast<uint4 *>(dy + (uint64_t)row[k0 + j] * row_bytes + v * 16) = narrow8(o);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < mg::GROUP; ++j) {
#pragma unroll
            for (int s = 16; s > 0; s >>= 1)
                dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], s);
            if (lane == 0 && k0 + j < m.k)
                part[warp][k0 + j] = dot[j];
        }
    }
    __syncthreads();
    if (in && at < m.k) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < G / 32; ++w)
            sum += part[own * (G / 32) + w][at];
        reinterpret_cast<float *>(region + dgate_off)[t * m.k + at] = sum;
    }
}

template <int G>
__global__ void __launch_bounds__(mg::THREADS) moe_dispatch_grad_kernel(const __grid_constant__ MoeRows m, uint64_t dx_off, const uint8_t *drecv)
{
    constexpr int TOKENS = mg::THREADS / G;
    __shared__ int64_t rows[TOKENS][32];
    griddep_launch_dependents();
    griddep_wait();
    const int own = threadIdx.x / G, at = threadIdx.x % G;
    int64_t *row = rows[own];
    const uint32_t tok32 = blockIdx.x * TOKENS + own, src = tok32 / (uint32_t)m.T;
    const bool in = tok32 < (uint64_t)m.tokens;
    const int64_t tok = tok32, t = tok32 - src * (uint32_t)m.T;
    if (in && at < m.k)
        row[at] = moe_row(m, tok, at, true);
    __syncthreads();
    if (!in)
        return;
    const uint64_t row_bytes = (uint64_t)m.H * 2;
    uint8_t *dx = m.regions + (uint64_t)src * m.region_bytes + dx_off + (uint64_t)t * row_bytes;
    const int64_t vecs = m.H / 8;
    for (int64_t v = at; v < vecs; v += G) {
        float sum[8] = {};
        for (int k0 = 0; k0 < m.k; k0 += mg::GROUP) {
            uint4 r[mg::GROUP];
#pragma unroll
            for (int j = 0; j < mg::GROUP; ++j)
                if (k0 + j < m.k && row[k0 + j] >= 0)
                    r[j] = ld_row(drecv + (uint64_t)row[k0 + j] * row_bytes + v * 16);
#pragma unroll
            for (int j = 0; j < mg::GROUP; ++j)
                if (k0 + j < m.k && row[k0 + j] >= 0) {
                    float f[8];
                    widen8(r[j], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sum[i] += f[i];
                }
        }
        *reinterpret_cast<uint4 *>(dx + v * 16) = narrow8(sum);
    }
}

} // namespace tdg

using namespace tdg;
using namespace tdg_host;

namespace {

// the kernel with G threads a token
template <class F> int launch_for(const tdg_symm *h, const MoeRows &m, cudaStream_t s, void **args, const char *what, F kernel)
{
    const int threads = mg::threads_of(m, h->sm_count);
    const int64_t grid = (m.tokens + mg::THREADS / threads - 1) / (mg::THREADS / threads);
    const void *fn = threads == 32    ? kernel(std::integral_constant<int, 32>{})
                     : threads == 64  ? kernel(std::integral_constant<int, 64>{})
                     : threads == 128 ? kernel(std::integral_constant<int, 128>{})
                                      : kernel(std::integral_constant<int, 256>{});
    return cuda_err(launch(fn, dim3((unsigned)grid), dim3(mg::THREADS), 0, s, args, false, 1, true), what);
}

} // namespace

extern "C" int tdg_moe_combine_grad(tdg_symm *h, const tdg_moe_combine_grad_args *a, void *stream)
{
    if (!h || !a)
        return TDG_ERR_INVALID;
    if (const int drc = check_device(h))
        return drc;
    MoeRows m;
    if (const int rc = moe_rows(h, a->world, a->k, a->T, a->H, a->slot, 8, m))
        return rc;
    if (a->T == 0)
        return TDG_OK;
    const uint64_t shard = (uint64_t)a->T * a->H * 2, gates = (uint64_t)a->T * a->k * 4, rows = (uint64_t)m.rows * a->H * 2;
    if (!a->slot || !a->y || !aligned16(a->y) || !a->dy || !aligned16(a->dy) || !aligned16(a->dout_off) || (a->gate_off & 3) ||
        (a->dgate_off & 3))
        return TDG_ERR_INVALID;
    if (!in_region(h, a->gate_off, gates) || !in_region(h, a->dgate_off, gates) || !in_region(h, a->dout_off, shard))
        return TDG_ERR_NOMEM;
    const Range slot{a->slot, (uint64_t)m.rows * 8}, y{a->y, rows}, dy{a->dy, rows};
    if (ranges_overlap({dy}, {slot}) || (a->dy != a->y && ranges_overlap({dy}, {y})) || shards_overlap(h, a->dgate_off, gates, {slot, y, dy}) ||
        shards_overlap(h, a->gate_off, gates, {dy}) || shards_overlap(h, a->dout_off, shard, {dy}) ||
        overlap(a->dgate_off, gates, a->gate_off, gates) || overlap(a->dgate_off, gates, a->dout_off, shard))
        return TDG_ERR_INVALID;
    m.epoch = next_epoch(h);
    uint64_t gate_off = a->gate_off, dout_off = a->dout_off, dgate_off = a->dgate_off;
    const uint8_t *yp = static_cast<const uint8_t *>(a->y);
    uint8_t *dyp = static_cast<uint8_t *>(a->dy);
    void *args[] = {&m, &gate_off, &dout_off, &dgate_off, &yp, &dyp};
    return launch_for(h, m, static_cast<cudaStream_t>(stream), args, "moe combine grad launch",
                      [](auto g) { return reinterpret_cast<const void *>(&moe_combine_grad_kernel<decltype(g)::value>); });
}

extern "C" int tdg_moe_dispatch_grad(tdg_symm *h, const tdg_moe_dispatch_grad_args *a, void *stream)
{
    if (!h || !a)
        return TDG_ERR_INVALID;
    if (const int drc = check_device(h))
        return drc;
    MoeRows m;
    if (const int rc = moe_rows(h, a->world, a->k, a->T, a->H, a->slot, 8, m))
        return rc;
    if (a->T == 0)
        return TDG_OK;
    const uint64_t shard = (uint64_t)a->T * a->H * 2;
    if (!a->slot || !a->drecv || !aligned16(a->drecv) || !aligned16(a->dx_off))
        return TDG_ERR_INVALID;
    if (!in_region(h, a->dx_off, shard))
        return TDG_ERR_NOMEM;
    const Range slot{a->slot, (uint64_t)m.rows * 8}, drecv{a->drecv, (uint64_t)m.rows * a->H * 2};
    if (shards_overlap(h, a->dx_off, shard, {slot, drecv}))
        return TDG_ERR_INVALID;
    m.epoch = next_epoch(h);
    uint64_t dx_off = a->dx_off;
    const uint8_t *rp = static_cast<const uint8_t *>(a->drecv);
    void *args[] = {&m, &dx_off, &rp};
    return launch_for(h, m, static_cast<cudaStream_t>(stream), args, "moe dispatch grad launch",
                      [](auto g) { return reinterpret_cast<const void *>(&moe_dispatch_grad_kernel<decltype(g)::value>); });
}
