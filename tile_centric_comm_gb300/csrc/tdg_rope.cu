// tdg_rope.cu -- rotary positions on one to three axes, and the write of the
// new tokens' keys and values into the pages of the symmetric heap's cache.
//
// Per head and pair i: (x, y) -> (c x - s y, c y + s x) with (c, s) from a
// table row chosen by the position on the pair's axis.
//
// Bound by memory: every row is read once and written once (keys twice: to
// k_out and to the cache).  One CTA handles a group of up to 8 rows.  First
// its threads look the rows up (sequence, page, slot, positions: chains of
// dependent loads, paid once per group) and put the rows' cosines and sines
// into shared memory; then they walk over all (row, head) pairs of the group,
// 16 elements a thread, four pairs' loads in flight at a time.
//
// Measured on one GB300 (copy rate 6.79 TB/s), 64 / 8 heads of 128: 9 prompts of
// 301..4093 tokens (927 MB) 160 us, 5.8 TB/s; 8 prompts of 2500 153 us, 5.7 TB/s,
// and 157 us, 5.3 TB/s, into an 8-bit cache (the divisions by the scale; 152 with
// a reciprocal, whose codes differ); heads of 64 80 and 88 us.  256 tokens into an
// 8-bit cache 5.6 us and one token 4.1 us: the launch, and lookups that this code
// does one after the other, of which only the page id waits for the length and
// the cosines for the position (a call of either takes the host 6 us).
#include "tdg_paged.cuh"

namespace tdg {

namespace rp {
constexpr int THREADS = 256;
constexpr int MAX_ROWS = 8; // rows of a group
constexpr int DEPTH = 4;    // units whose loads a thread has in flight
} // namespace rp

struct RopeParams {
    DevStatus *status;
    uint32_t epoch;
    PagedView c;
    int64_t T, B, max_pos, pos_stride, table_entries, table_stride;
    int64_t qs, ks, vs, qos, kos;
    int Hq, rot, axes, sec0, sec01, rows; // rows: of a group
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

// 8 quotients by the scale, in e4m3 (clamped to +-448, NaN kept).  The division
// itself: the product with a rounded reciprocal falls off a tie (27 of 1820
// values at a scale of 7/256), and the reciprocal of a scale below 2^-128 is
// infinite.
__device__ __forceinline__ uint2 pack8_e4m3(const float (&f)[8], float scale)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i] / scale, f[2 * i + 1] / scale), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// rows are read once: past L1 (and not through the read-only path, since an
// output may be its own input)
__device__ __forceinline__ uint4 ld_once(const __nv_bfloat16 *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// (four CTAs per SM rather than three are worth 5 % of a long bf16 write, with 4 to
// 12 bytes a thread spilled; the 8-bit kernel does not fit the registers that this
// leaves)
template <int D, bool INTER, bool E4M3>
__global__ void __launch_bounds__(rp::THREADS, E4M3 ? 3 : 4) rope_append_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int UNITS = D / 16; // 16-element units of a head
    constexpr int ESZ = E4M3 ? 1 : 2;
    constexpr int LANES = rp::THREADS / UNITS;
    __shared__ __align__(16) float turn[rp::MAX_ROWS][D]; // cosines, then sines, of a row's pairs
    __shared__ uint8_t *slot_k[rp::MAX_ROWS], *slot_v[rp::MAX_ROWS]; // head 0's slot in the cache, or NULL
    __shared__ int skip[rp::MAX_ROWS]; // a row with a position outside the table
    __shared__ int seq[rp::MAX_ROWS];
    griddep_launch_dependents();
    griddep_wait();
    const int64_t first = (int64_t)blockIdx.x * p.rows;
    const int rows = (int)min((int64_t)p.rows, p.T - first);
    // the sequence of each row: the first b with cu[b + 1] > t.  All threads
    // scan cu at once; with offsets in order the rows' counts ascend.
    if (p.table && p.cu) {
        if (threadIdx.x < rp::MAX_ROWS)
            seq[threadIdx.x] = 0;
        __syncthreads();
        int count[rp::MAX_ROWS] = {};
        for (int64_t i = threadIdx.x; i < p.B; i += rp::THREADS) {
            const int64_t end = p.cu[i + 1];
#pragma unroll
            for (int r = 0; r < rp::MAX_ROWS; ++r)
                count[r] += end <= first + r ? 1 : 0;
        }
#pragma unroll
        for (int r = 0; r < rp::MAX_ROWS; ++r) {
            const int n = __reduce_add_sync(0xffffffffu, count[r]);
            if (n && (threadIdx.x & 31) == 0)
                atomicAdd(&seq[r], n);
        }
        __syncthreads();
    }
    if ((int)threadIdx.x < rows) {
        const int r = threadIdx.x;
        const int64_t t = first + r;
        int bad = 0;
        for (int a = 0; p.rot && a < p.axes; ++a) {
            const int32_t pos = p.pos[(int64_t)a * p.pos_stride + t];
            bad |= pos < 0 || pos >= p.max_pos ? 1 : 0;
        }
        if (bad)
            report_fault(p.status, TDG_ERR_DEVICE, TDG_WHERE_POS, (uint32_t)t, p.epoch);
        skip[r] = bad;
        uint8_t *at_slot = nullptr;
        if (p.table && !bad) {
            const int64_t b = p.cu ? seq[r] : t;
            int64_t lo = t, hi = t + 1; // the sequence's new rows
            if (p.cu) {
                lo = b < p.B ? p.cu[b] : t + 1;
                hi = b < p.B ? p.cu[b + 1] : t + 1;
            }
            if (lo <= t && t < hi) { // else the row belongs to no sequence (or the offsets are out of order)
                const int64_t len = p.lens[b], at = len - (hi - t);
                int32_t page = -1;
                if (len >= hi - lo && len <= p.table_entries << p.c.ps_log2)
                    page = p.table[b * p.table_stride + (at >> p.c.ps_log2)];
                if (page < 0 || page >= p.c.all_pages)
                    report_fault(p.status, TDG_ERR_DEVICE, TDG_WHERE_PAGE, (uint32_t)t, p.epoch);
                else
                    at_slot = p.c.regions + (uint64_t)(page / p.c.pages) * p.c.region_bytes +
                              paged_row(p.c, page % p.c.pages, 0, (int)(at & ((1 << p.c.ps_log2) - 1)), ESZ);
            }
        }
        slot_k[r] = at_slot ? at_slot + p.c.k_off : nullptr;
        slot_v[r] = at_slot ? at_slot + p.c.v_off : nullptr;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * p.rot; i += rp::THREADS) {
        const int r = i / p.rot, c = i % p.rot, pair = c < p.rot / 2 ? c : c - p.rot / 2;
        if (!skip[r]) {
            const int a = (pair >= p.sec0 ? 1 : 0) + (pair >= p.sec01 ? 1 : 0);
            turn[r][c] = p.cos_sin[(int64_t)p.pos[(int64_t)a * p.pos_stride + first + r] * p.rot + c];
        }
    }
    __syncthreads();

    const int u = threadIdx.x % UNITS; // this thread's unit in every head
    const bool turned = u * 16 < p.rot;
    // its two runs of 8 elements
    const int lo = INTER || !turned ? u * 16 : u * 8;
    const int hi = INTER || !turned ? lo + 8 : p.rot / 2 + u * 8;
    const uint64_t head_bytes = (uint64_t)(D * ESZ) << p.c.ps_log2; // from one head's slot to the next one's
    const int heads = p.Hq + 2 * p.c.Hkv, kv_end = p.Hq + p.c.Hkv;
    const int pairs = rows * heads;
    int r = 0, hh = threadIdx.x / UNITS;
    while (hh >= heads) {
        hh -= heads;
        ++r;
    }
    for (int i = threadIdx.x / UNITS; i < pairs; i += rp::DEPTH * LANES) {
        uint4 x4[rp::DEPTH], y4[rp::DEPTH];
        int rr[rp::DEPTH], hd[rp::DEPTH];
#pragma unroll
        for (int d = 0; d < rp::DEPTH; ++d) {
            rr[d] = -1;
            hd[d] = hh;
            if (i + d * LANES < pairs && !skip[r] && (hh < kv_end || slot_v[r])) {
                rr[d] = r;
                const int64_t t = first + r;
                const __nv_bfloat16 *src = hh < p.Hq ? p.q + t * p.qs + (int64_t)hh * D
                                           : hh < kv_end ? p.k + t * p.ks + (int64_t)(hh - p.Hq) * D
                                                         : p.v + t * p.vs + (int64_t)(hh - kv_end) * D;
                x4[d] = ld_once(src + lo);
                y4[d] = ld_once(src + hi);
            }
            hh += LANES;
            while (hh >= heads) {
                hh -= heads;
                ++r;
            }
        }
#pragma unroll
        for (int d = 0; d < rp::DEPTH; ++d) {
            if (rr[d] < 0)
                continue;
            const int row = rr[d], head = hd[d];
            const bool is_v = head >= kv_end;
            if (is_v && !E4M3) { // a copy
                uint8_t *dst = slot_v[row] + (uint64_t)(head - kv_end) * head_bytes;
                *reinterpret_cast<uint4 *>(dst + lo * 2) = x4[d];
                *reinterpret_cast<uint4 *>(dst + hi * 2) = y4[d];
                continue;
            }
            float x[8], y[8];
            unpack8(x4[d], x);
            unpack8(y4[d], y);
            if (turned && !is_v) {
                const float *cs = &turn[row][u * 8], *sn = &turn[row][p.rot / 2 + u * 8];
                float c[8], s[8];
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    *reinterpret_cast<float4 *>(&c[j]) = *reinterpret_cast<const float4 *>(cs + j);
                    *reinterpret_cast<float4 *>(&s[j]) = *reinterpret_cast<const float4 *>(sn + j);
                }
                if (INTER) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float a0 = x[2 * j], a1 = x[2 * j + 1], b0 = y[2 * j], b1 = y[2 * j + 1];
                        x[2 * j] = c[j] * a0 - s[j] * a1;
                        x[2 * j + 1] = c[j] * a1 + s[j] * a0;
                        y[2 * j] = c[j + 4] * b0 - s[j + 4] * b1;
                        y[2 * j + 1] = c[j + 4] * b1 + s[j + 4] * b0;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float a = x[j], b = y[j];
                        x[j] = c[j] * a - s[j] * b;
                        y[j] = c[j] * b + s[j] * a;
                    }
                }
                x4[d] = pack8(x);
                y4[d] = pack8(y);
            }
            const int64_t t = first + row;
            if (!is_v) {
                __nv_bfloat16 *dst = head < p.Hq ? p.q_out + t * p.qos + (int64_t)head * D
                                     : p.k_out   ? p.k_out + t * p.kos + (int64_t)(head - p.Hq) * D
                                                 : nullptr;
                if (dst) {
                    *reinterpret_cast<uint4 *>(dst + lo) = x4[d];
                    *reinterpret_cast<uint4 *>(dst + hi) = y4[d];
                }
            }
            uint8_t *slot = is_v ? slot_v[row] : slot_k[row];
            if (head >= p.Hq && slot) {
                const int h = head - (is_v ? kv_end : p.Hq);
                uint8_t *dst = slot + (uint64_t)h * head_bytes;
                if (E4M3) {
                    const float scale = (is_v ? p.c.v_scale : p.c.k_scale)[h];
                    *reinterpret_cast<uint2 *>(dst + lo) = pack8_e4m3(x, scale);
                    *reinterpret_cast<uint2 *>(dst + hi) = pack8_e4m3(y, scale);
                } else {
                    *reinterpret_cast<uint4 *>(dst + lo * 2) = x4[d];
                    *reinterpret_cast<uint4 *>(dst + hi * 2) = y4[d];
                }
            }
        }
    }
}

} // namespace tdg

using namespace tdg;
using namespace tdg_host;

namespace {
template <int D> const void *pick(bool inter, bool e4m3)
{
    return inter ? (e4m3 ? reinterpret_cast<const void *>(&rope_append_kernel<D, true, true>)
                         : reinterpret_cast<const void *>(&rope_append_kernel<D, true, false>))
                 : (e4m3 ? reinterpret_cast<const void *>(&rope_append_kernel<D, false, true>)
                         : reinterpret_cast<const void *>(&rope_append_kernel<D, false, false>));
}
} // namespace

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
    const Range q_out{a->q_out, rows_extent(T, a->q_out_stride, Hq * D)}, k_out{a->k_out, rows_extent(T, a->k_out_stride, Hkv * D)};
    const uint64_t turn = a->rot_dim ? (uint64_t)a->max_pos * a->rot_dim * 4 : 0;
    const Range cos_sin{a->cos_sin, turn}, pos{a->pos, turn ? ((uint64_t)(a->axes - 1) * a->pos_stride + T) * 4 : 0};
    if (ranges_overlap({q_out, k_out}, {cos_sin, pos}))
        return TDG_ERR_INVALID;
    if (a->table) {
        if (const int rc = paged_view(h, a->cache, p.c))
            return rc;
        if (!rows_ok(a->v, a->v_stride, Hkv * D) || !a->lens || !aligned4(a->lens) || !aligned4(a->cu) ||
            !table_ok(a->table, a->table_entries, a->table_stride, a->cache.page_size) || (!a->cu && a->B != T))
            return TDG_ERR_INVALID;
        // the pools (written) hold nothing else of the call, and the rows written
        // none of the indices
        const Range q{a->q, rows_extent(T, a->q_stride, Hq * D)}, k{a->k, rows_extent(T, a->k_stride, Hkv * D)};
        const Range v{a->v, rows_extent(T, a->v_stride, Hkv * D)};
        const Range k_scale{a->cache.k_scale, scale_bytes(a->cache)}, v_scale{a->cache.v_scale, scale_bytes(a->cache)};
        const Range cu{a->cu, (uint64_t)(a->B + 1) * 4}, lens{a->lens, (uint64_t)a->B * 4};
        const Range table = table_range(a->table, a->B, a->table_entries, a->table_stride);
        if (ranges_overlap({q_out, k_out}, {k_scale, v_scale, cu, lens, table}) ||
            pools_overlap(h, a->cache, {q, k, v, q_out, k_out, cos_sin, pos, k_scale, v_scale, cu, lens, table}))
            return TDG_ERR_INVALID;
    } else {
        p.c.Hkv = (int)Hkv;
        p.c.D = (int)D;
    }
    p.status = h->status;
    p.epoch = next_epoch(h);
    p.T = T;
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
    // rows of a group: up to 8, as long as that leaves every SM four CTAs
    const int64_t rows = T / ((int64_t)h->sm_count * 4);
    p.rows = (int)(rows < 1 ? 1 : rows > rp::MAX_ROWS ? rp::MAX_ROWS : rows);
    const bool e4m3 = a->table && a->cache.kv_type == TDG_KV_E4M3;
    const void *fn = D == 128 ? pick<128>(a->interleaved, e4m3) : pick<64>(a->interleaved, e4m3);
    void *args[] = {&p};
    return cuda_err(launch(fn, dim3((unsigned)((T + p.rows - 1) / p.rows)), dim3(rp::THREADS), 0,
                           static_cast<cudaStream_t>(stream), args, false, 1, true),
                    "rope append launch");
}
