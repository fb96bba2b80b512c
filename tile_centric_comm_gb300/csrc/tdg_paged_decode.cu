// tdg_paged_decode.cu -- attention of one new token per sequence over the
// paged cache: softmax(scale q K^T) V over lens[b] cached tokens.
//
// One CTA per (sequence, query head); its 4 warps take every fourth token, a
// lane holds D/32 of the head's elements, and each warp keeps a running
// maximum, sum and output (online softmax, float32), merged at the end.
#include "tdg_paged.cuh"

namespace tdg {

namespace pd {
constexpr int WARPS = 4;
constexpr int MAX_CTAS = 512; // CTAs whose partial results the caller provides room for
constexpr int ROWS = 16;      // query heads of a partial result
} // namespace pd

struct PagedDecodeParams {
    DevStatus *status;
    uint32_t epoch;
    PagedView c;
    int64_t B, table_entries, table_stride, qs, os;
    int Hq, G;
    float scale;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    float *lse;
    const int32_t *table, *lens;
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(pd::WARPS * 32) paged_decode_kernel(const __grid_constant__ PagedDecodeParams p)
{
    constexpr int N = D / 32;
    __shared__ float sm[pd::WARPS], sl[pd::WARPS], so[pd::WARPS][D];
    const int h = blockIdx.x, b = blockIdx.y, g = h / p.G;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t len = p.lens[b];
    if (len < 0 || len > p.table_entries << p.c.ps_log2) {
        if (threadIdx.x == 0)
            report_fault(p.status, TDG_ERR_DEVICE, TDG_WHERE_PAGE, (uint32_t)b, p.epoch);
        len = 0;
    }
    float q[N], o[N], m = -INFINITY, l = 0.f;
    const float ks = E4M3 ? p.c.k_scale[g] : 1.f, vs = E4M3 ? p.c.v_scale[g] : 1.f;
    for (int i = 0; i < N; ++i) {
        q[i] = __bfloat162float(p.q[b * p.qs + (int64_t)h * D + lane * N + i]) * p.scale * ks;
        o[i] = 0.f;
    }
    for (int64_t t = warp; t < len; t += pd::WARPS) {
        int32_t page = p.table[b * p.table_stride + (t >> p.c.ps_log2)];
        if (page < 0 || page >= p.c.all_pages) {
            if (lane == 0)
                report_fault(p.status, TDG_ERR_DEVICE, TDG_WHERE_PAGE, (uint32_t)b, p.epoch);
            continue;
        }
        const uint8_t *at = p.c.regions + (uint64_t)(page / p.c.pages) * p.c.region_bytes +
                            paged_row(p.c, page % p.c.pages, g, (int)(t & ((1 << p.c.ps_log2) - 1)), E4M3 ? 1 : 2);
        auto load = [&](const uint8_t *row, int i) -> float {
            if (E4M3)
                return (float)reinterpret_cast<const __nv_fp8_e4m3 *>(row)[lane * N + i];
            return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(row)[lane * N + i]);
        };
        float s = 0.f;
        for (int i = 0; i < N; ++i)
            s += q[i] * load(at + p.c.k_off, i);
        for (int x = 16; x; x >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, x);
        const float mn = fmaxf(m, s), ms = mn == -INFINITY ? 0.f : mn;
        const float al = expf(m - ms), w = expf(s - ms);
        m = mn;
        l = l * al + w;
        for (int i = 0; i < N; ++i)
            o[i] = o[i] * al + w * load(at + p.c.v_off, i);
    }
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    for (int i = 0; i < N; ++i)
        so[warp][lane * N + i] = o[i];
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < pd::WARPS; ++w)
        M = fmaxf(M, sm[w]);
    const float Ms = M == -INFINITY ? 0.f : M;
    for (int w = 0; w < pd::WARPS; ++w)
        L += sl[w] * expf(sm[w] - Ms);
    for (int d = threadIdx.x; d < D; d += blockDim.x) {
        float a = 0.f;
        for (int w = 0; w < pd::WARPS; ++w)
            a += so[w][d] * expf(sm[w] - Ms);
        p.out[b * p.os + (int64_t)h * D + d] = __float2bfloat16_rn(len > 0 ? a / L * vs : 0.f);
    }
    if (p.lse && threadIdx.x == 0)
        p.lse[(int64_t)b * p.Hq + h] = len > 0 ? M + logf(L) : -INFINITY;
}

} // namespace tdg

using namespace tdg;
using namespace tdg_host;

extern "C" size_t tdg_paged_decode_part_bytes(int64_t Hq, int64_t Hkv, int64_t D)
{
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv || Hq / Hkv > 128 || (D != 64 && D != 128))
        return 0;
    // per CTA two partial results (rows x (D + maximum and sum) float32) and one description of 16 bytes
    return (size_t)pd::MAX_CTAS * (2 * pd::ROWS * (D + 2) * sizeof(float) + 16);
}

extern "C" int tdg_paged_decode(tdg_symm *h, const tdg_paged_decode_args *a, void *stream)
{
    if (!h || !a)
        return TDG_ERR_INVALID;
    if (const int drc = check_device(h))
        return drc;
    const int64_t D = a->cache.D, Hkv = a->cache.Hkv, Hq = a->Hq;
    if (a->world != h->world || a->root < 0 || a->root >= h->world || a->B < 0 || a->B > 65535 || Hq <= 0 || Hkv <= 0 ||
        Hq > 65536 || Hq % Hkv || Hq / Hkv > 128 || !(a->scale >= 0.f) || isinf(a->scale))
        return TDG_ERR_INVALID;
    PagedDecodeParams p;
    memset(&p, 0, sizeof p);
    if (const int rc = paged_view(h, a->cache, p.c))
        return rc;
    if (a->part_off % 16)
        return TDG_ERR_INVALID;
    const size_t part = tdg_paged_decode_part_bytes(Hq, Hkv, D);
    const uint64_t pool = tdg_paged_pool_bytes(a->cache.pages, a->cache.page_size, Hkv, D, a->cache.kv_type);
    if (part > h->region_bytes || a->part_off > h->region_bytes - part)
        return TDG_ERR_NOMEM;
    if (overlap(a->part_off, part, a->cache.k_off, pool) || overlap(a->part_off, part, a->cache.v_off, pool))
        return TDG_ERR_INVALID;
    if (a->B == 0)
        return TDG_OK;
    if (!rows_ok(a->q, a->q_stride, Hq * D) || !rows_ok(a->out, a->out_stride, Hq * D) || !a->lens ||
        !aligned4(a->lens) || !aligned4(a->lse) ||
        !table_ok(a->table, a->table_entries, a->table_stride, a->cache.page_size))
        return TDG_ERR_INVALID;
    if (rows_clash(a->B, a->out, a->out_stride, Hq * D, a->B, a->q, a->q_stride, Hq * D))
        return TDG_ERR_INVALID;
    p.status = h->status;
    p.epoch = next_epoch(h);
    p.B = a->B;
    p.table_entries = a->table_entries;
    p.table_stride = a->table_stride;
    p.qs = a->q_stride;
    p.os = a->out_stride;
    p.Hq = (int)Hq;
    p.G = (int)(Hq / Hkv);
    p.scale = a->scale > 0.f ? a->scale : 1.0f / sqrtf((float)D);
    p.q = static_cast<const __nv_bfloat16 *>(a->q);
    p.out = static_cast<__nv_bfloat16 *>(a->out);
    p.lse = a->lse;
    p.table = a->table;
    p.lens = a->lens;
    const bool e4m3 = a->cache.kv_type == TDG_KV_E4M3;
    const void *fn = D == 128 ? (e4m3 ? reinterpret_cast<const void *>(&paged_decode_kernel<128, true>)
                                      : reinterpret_cast<const void *>(&paged_decode_kernel<128, false>))
                              : (e4m3 ? reinterpret_cast<const void *>(&paged_decode_kernel<64, true>)
                                      : reinterpret_cast<const void *>(&paged_decode_kernel<64, false>));
    void *args[] = {&p};
    return cuda_err(launch(fn, dim3((unsigned)Hq, (unsigned)a->B), dim3(pd::WARPS * 32), 0,
                           static_cast<cudaStream_t>(stream), args, false),
                    "paged decode launch");
}
