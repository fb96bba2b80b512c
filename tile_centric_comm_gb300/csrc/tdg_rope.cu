// tdg_rope.cu -- rotary positions on one to three axes, and the write of the
// new tokens' keys and values into the pages of the symmetric heap's cache.
//
// Per head and pair i: (x, y) -> (c x - s y, c y + s x) with (c, s) from a
// table row chosen by the position on the pair's axis.  One CTA handles one
// row (token); a thread keeps the cosines and sines of 8 pairs and walks over
// the row's heads with them.
#include "tdg_paged.cuh"

namespace tdg {

namespace rp {
constexpr int THREADS = 256;
} // namespace rp

struct RopeParams {
    DevStatus *status;
    uint32_t epoch;
    PagedView c;
    int64_t B, max_pos, pos_stride, table_entries, table_stride;
    int64_t qs, ks, vs, qos, kos;
    int Hq, rot, axes, sec0, sec01;
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *q_out, *k_out;
    const float *cos_sin;
    const int32_t *pos, *cu, *table, *lens;
};

__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8])
{
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __bfloat1622float2(h[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// 8 values divided by the head's scale, in e4m3 (clamped to +-448, NaN kept)
__device__ __forceinline__ uint2 pack8_e4m3(const float (&f)[8], float scale)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i] / scale, f[2 * i + 1] / scale), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

template <bool INTER, bool E4M3>
__global__ void __launch_bounds__(rp::THREADS) rope_append_kernel(const __grid_constant__ RopeParams p)
{
    const int t = blockIdx.x;
    const int D = p.c.D, units = D / 16; // 16-element units of a head
    // the sequence of this row: the first b with cu[b + 1] > t
    bool store = p.table != nullptr;
    int b = t;
    int64_t newer = 1; // rows of the sequence from this one on
    if (store && p.cu) {
        b = 0;
        for (int64_t i = threadIdx.x; i - threadIdx.x < p.B; i += rp::THREADS)
            b += __syncthreads_count(i < p.B && p.cu[i + 1] <= t);
        store = b < p.B && p.cu[b] <= t && p.cu[b + 1] > t; // offsets out of order cover no row
        if (store)
            newer = (int64_t)p.cu[b + 1] - t;
    }
    // the axes' positions
    int32_t pos[3] = {0, 0, 0};
    if (p.rot) {
        bool ok = true;
        for (int a = 0; a < 3; ++a)
            if (a < p.axes) {
                pos[a] = p.pos[(int64_t)a * p.pos_stride + t];
                ok = ok && pos[a] >= 0 && pos[a] < p.max_pos;
            }
        if (!ok) {
            if (threadIdx.x == 0)
                report_fault(p.status, TDG_ERR_DEVICE, TDG_WHERE_POS, (uint32_t)t, p.epoch);
            return;
        }
    }
    uint8_t *kc = nullptr, *vc = nullptr; // head 0's slot in the cache
    constexpr int ESZ = E4M3 ? 1 : 2;
    if (store) {
        const int64_t len = p.lens[b], at = len - newer;
        const int64_t first = p.cu ? len - ((int64_t)p.cu[b + 1] - p.cu[b]) : at;
        int32_t page = -1;
        if (first >= 0 && at >= 0 && len <= p.table_entries << p.c.ps_log2)
            page = p.table[b * p.table_stride + (at >> p.c.ps_log2)];
        if (page < 0 || page >= p.c.all_pages) {
            if (threadIdx.x == 0)
                report_fault(p.status, TDG_ERR_DEVICE, TDG_WHERE_PAGE, (uint32_t)t, p.epoch);
            store = false;
        } else {
            const int slot = (int)(at & ((1 << p.c.ps_log2) - 1));
            uint8_t *base = p.c.regions + (uint64_t)(page / p.c.pages) * p.c.region_bytes +
                            paged_row(p.c, page % p.c.pages, 0, slot, ESZ);
            kc = base + p.c.k_off;
            vc = base + p.c.v_off;
        }
    }
    const uint64_t head_bytes = (uint64_t)(D * ESZ) << p.c.ps_log2; // from one head's slot to the next one's

    const int u = threadIdx.x % units;       // this thread's unit in every head
    const bool turned = u * 16 < p.rot;
    int lo, hi;                               // its two runs of 8 elements
    if (INTER || !turned) {
        lo = u * 16;
        hi = lo + 8;
    } else {
        lo = u * 8;
        hi = p.rot / 2 + u * 8;
    }
    float cs[8], sn[8];
    if (turned) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = u * 8 + j;
            const int a = (i >= p.sec0 ? 1 : 0) + (i >= p.sec01 ? 1 : 0);
            const float *row = p.cos_sin + (int64_t)(a == 0 ? pos[0] : a == 1 ? pos[1] : pos[2]) * p.rot;
            cs[j] = row[i];
            sn[j] = row[p.rot / 2 + i];
        }
    }
    const int heads = p.Hq + 2 * p.c.Hkv;
    for (int hh = threadIdx.x / units; hh < heads; hh += rp::THREADS / units) {
        const bool is_q = hh < p.Hq;
        const bool is_v = hh >= p.Hq + p.c.Hkv;
        const int h = is_q ? hh : is_v ? hh - p.Hq - p.c.Hkv : hh - p.Hq;
        if (is_v && !store)
            break;
        const __nv_bfloat16 *src = (is_q ? p.q + (int64_t)t * p.qs : is_v ? p.v + (int64_t)t * p.vs : p.k + (int64_t)t * p.ks) + (int64_t)h * D;
        float x[8], y[8];
        unpack8(*reinterpret_cast<const uint4 *>(src + lo), x);
        unpack8(*reinterpret_cast<const uint4 *>(src + hi), y);
        if (turned && !is_v) {
            if (INTER) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a0 = x[2 * j], a1 = x[2 * j + 1], b0 = y[2 * j], b1 = y[2 * j + 1];
                    x[2 * j] = cs[j] * a0 - sn[j] * a1;
                    x[2 * j + 1] = cs[j] * a1 + sn[j] * a0;
                    y[2 * j] = cs[j + 4] * b0 - sn[j + 4] * b1;
                    y[2 * j + 1] = cs[j + 4] * b1 + sn[j + 4] * b0;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float a = x[j], c = y[j];
                    x[j] = cs[j] * a - sn[j] * c;
                    y[j] = cs[j] * c + sn[j] * a;
                }
            }
        }
        if (!is_v) {
            __nv_bfloat16 *dst = is_q ? p.q_out + (int64_t)t * p.qos : p.k_out ? p.k_out + (int64_t)t * p.kos : nullptr;
            if (dst) {
                *reinterpret_cast<uint4 *>(dst + (int64_t)h * D + lo) = pack8(x);
                *reinterpret_cast<uint4 *>(dst + (int64_t)h * D + hi) = pack8(y);
            }
        }
        if (!is_q && store) {
            uint8_t *dst = (is_v ? vc : kc) + (uint64_t)h * head_bytes;
            if (E4M3) {
                const float scale = (is_v ? p.c.v_scale : p.c.k_scale)[h];
                *reinterpret_cast<uint2 *>(dst + lo) = pack8_e4m3(x, scale);
                *reinterpret_cast<uint2 *>(dst + hi) = pack8_e4m3(y, scale);
            } else {
                *reinterpret_cast<uint4 *>(dst + lo * 2) = pack8(x);
                *reinterpret_cast<uint4 *>(dst + hi * 2) = pack8(y);
            }
        }
    }
}

} // namespace tdg

using namespace tdg;
using namespace tdg_host;

extern "C" size_t tdg_paged_pool_bytes(int64_t pages, int page_size, int64_t Hkv, int64_t D, int kv_type)
{
    if (pages <= 0 || pages > INT32_MAX || !page_size_ok(page_size) || Hkv <= 0 || Hkv > 65536 || (D != 64 && D != 128) ||
        (kv_type != TDG_KV_BF16 && kv_type != TDG_KV_E4M3))
        return 0;
    // at most 2^31 * 2^8 * 2^16 * 2^8: below 2^63
    return (size_t)pages * page_size * Hkv * D * (kv_type == TDG_KV_E4M3 ? 1 : 2);
}

extern "C" int tdg_rope_append(tdg_symm *h, const tdg_rope_append_args *a, void *stream)
{
    if (!h || !a)
        return TDG_ERR_INVALID;
    if (const int drc = check_device(h))
        return drc;
    const int64_t D = a->cache.D, Hkv = a->cache.Hkv, Hq = a->Hq, T = a->T;
    if (a->world != h->world || T < 0 || T > INT32_MAX || a->B < 0 || a->B > INT32_MAX || Hq < 0 || Hq > 65536 ||
        Hkv <= 0 || Hkv > 65536 || (D != 64 && D != 128) || (a->interleaved & ~1))
        return TDG_ERR_INVALID;
    if (a->rot_dim < 0 || a->rot_dim % 16 || a->rot_dim > D)
        return TDG_ERR_INVALID;
    if (a->rot_dim) {
        if (a->axes < 1 || a->axes > 3 || a->max_pos <= 0 || !a->cos_sin || !aligned16(a->cos_sin) || !a->pos || !aligned4(a->pos) ||
            (a->axes > 1 && a->pos_stride < T))
            return TDG_ERR_INVALID;
        int64_t sum = 0;
        for (int i = 0; a->axes > 1 && i < a->axes; ++i) {
            if (a->sections[i] < 0)
                return TDG_ERR_INVALID;
            sum += a->sections[i];
        }
        if (a->axes > 1 && sum != a->rot_dim / 2)
            return TDG_ERR_INVALID;
    }
    if (T == 0)
        return TDG_OK;
    if ((a->q != nullptr) != (Hq > 0) || (a->q_out != nullptr) != (Hq > 0))
        return TDG_ERR_INVALID;
    if (Hq && (!rows_ok(a->q, a->q_stride, Hq * D) || !rows_ok(a->q_out, a->q_out_stride, Hq * D)))
        return TDG_ERR_INVALID;
    // an output is exactly its own input, or apart from every input and output
    const struct { const void *at; int64_t stride, width; } in[] = {{a->q, a->q_stride, Hq * D}, {a->k, a->k_stride, Hkv * D}, {a->table ? a->v : nullptr, a->v_stride, Hkv * D}};
    const struct { const void *at; int64_t stride, width; } out[] = {{a->q_out, a->q_out_stride, Hq * D}, {a->k_out, a->k_out_stride, Hkv * D}};
    for (int o = 0; o < 2; ++o)
        for (int i = 0; i < 3; ++i)
            if (!(o == i && out[o].at == in[i].at && out[o].stride == in[i].stride) &&
                rows_clash(T, out[o].at, out[o].stride, out[o].width, T, in[i].at, in[i].stride, in[i].width))
                return TDG_ERR_INVALID;
    if (rows_clash(T, out[0].at, out[0].stride, out[0].width, T, out[1].at, out[1].stride, out[1].width))
        return TDG_ERR_INVALID;
    if (!rows_ok(a->k, a->k_stride, Hkv * D) || (a->k_out && !rows_ok(a->k_out, a->k_out_stride, Hkv * D)))
        return TDG_ERR_INVALID;
    RopeParams p;
    memset(&p, 0, sizeof p);
    const uint64_t qx = rows_extent(T, a->q_stride, Hq * D), qox = rows_extent(T, a->q_out_stride, Hq * D);
    const uint64_t kx = rows_extent(T, a->k_stride, Hkv * D), kox = rows_extent(T, a->k_out_stride, Hkv * D);
    if (a->table) {
        if (const int rc = paged_view(h, a->cache, p.c))
            return rc;
        if (!rows_ok(a->v, a->v_stride, Hkv * D) || !a->lens || !aligned4(a->lens) || !aligned4(a->cu) ||
            !table_ok(a->table, a->table_entries, a->table_stride, a->cache.page_size) || (!a->cu && a->B != T))
            return TDG_ERR_INVALID;
        // the pools (written) hold none of the rows
        const uint64_t vx = rows_extent(T, a->v_stride, Hkv * D);
        const uint64_t pool = tdg_paged_pool_bytes(a->cache.pages, a->cache.page_size, Hkv, D, a->cache.kv_type);
        const struct { const void *at; uint64_t n; } rows[] = {{a->q, qx}, {a->k, kx}, {a->v, vx}, {a->q_out, qox}, {a->k_out, kox}};
        for (int r = 0; r < h->world; ++r)
            for (const auto &x : rows)
                if (rows_overlap(x.at, x.n, h->base + (uint64_t)r * h->region_bytes + a->cache.k_off, pool) ||
                    rows_overlap(x.at, x.n, h->base + (uint64_t)r * h->region_bytes + a->cache.v_off, pool))
                    return TDG_ERR_INVALID;
    } else {
        p.c.Hkv = (int)Hkv;
        p.c.D = (int)D;
    }
    p.status = h->status;
    p.epoch = next_epoch(h);
    p.B = a->B;
    p.max_pos = a->max_pos;
    p.pos_stride = a->pos_stride;
    p.table_entries = a->table_entries;
    p.table_stride = a->table_stride;
    p.qs = a->q_stride;
    p.ks = a->k_stride;
    p.vs = a->v_stride;
    p.qos = a->q_out_stride;
    p.kos = a->k_out_stride;
    p.Hq = (int)Hq;
    p.rot = a->rot_dim;
    p.axes = a->axes;
    p.sec0 = a->axes > 1 ? a->sections[0] : a->rot_dim;
    p.sec01 = a->axes > 2 ? a->sections[0] + a->sections[1] : a->rot_dim;
    p.q = static_cast<const __nv_bfloat16 *>(a->q);
    p.k = static_cast<const __nv_bfloat16 *>(a->k);
    p.v = static_cast<const __nv_bfloat16 *>(a->v);
    p.q_out = static_cast<__nv_bfloat16 *>(a->q_out);
    p.k_out = static_cast<__nv_bfloat16 *>(a->k_out);
    p.cos_sin = a->cos_sin;
    p.pos = a->pos;
    p.cu = a->cu;
    p.table = a->table;
    p.lens = a->lens;
    const bool e4m3 = a->table && a->cache.kv_type == TDG_KV_E4M3;
    const void *fn = a->interleaved ? (e4m3 ? reinterpret_cast<const void *>(&rope_append_kernel<true, true>)
                                            : reinterpret_cast<const void *>(&rope_append_kernel<true, false>))
                                    : (e4m3 ? reinterpret_cast<const void *>(&rope_append_kernel<false, true>)
                                            : reinterpret_cast<const void *>(&rope_append_kernel<false, false>));
    void *args[] = {&p};
    return cuda_err(launch(fn, dim3((unsigned)T), dim3(rp::THREADS), 0, static_cast<cudaStream_t>(stream), args, false),
                    "rope append launch");
}
