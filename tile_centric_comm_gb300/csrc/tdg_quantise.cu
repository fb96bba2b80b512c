// tdg_quantise.cu -- bf16 values into e4m3 codes with a float32 scale for each
// block: rows (1 x 128 blocks), rows of a gated projection, weights (128 x 128
// blocks), and the MoE dispatch whose rows are quantised on the way.
//
// Per block: scale = max(largest |x| / 448, 2^-100), code = x / scale rounded
// to e4m3.  Bound by memory: 2 bytes read (4 gated) and 1 written an element,
// for the dispatch 1 written for each of a token's k rows.  8 lanes hold one
// 1 x 128 block, 16 elements each (two 16-byte loads, one 16-byte store), so a
// block's maximum takes three shuffles and a value is read once.  32768 gated rows
// of 2048: 53 us, 6.3 TB/s; 8 weights of 4096 x 7168: 109 us, 6.5 TB/s; dispatch of
// 8192 tokens of 7168 to 8 experts each: 92 us, 6.6 TB/s.
#include "tdg_scaled.cuh"

namespace tdg {

namespace qn {
constexpr int THREADS = 256;
constexpr int LANES = 8;               // of a 1 x 128 block
constexpr int UNITS = THREADS / LANES; // blocks that a CTA holds at a time
constexpr float LEAST = 7.888609052210118e-31f; // 2^-100
} // namespace qn

struct QuantParams {
    DevStatus *status;
    uint32_t epoch;
    int64_t rows, K, xs, cs, ss;
    int64_t blocks;      // 1 x 128 blocks of a row
    const __nv_bfloat16 *x;
    uint8_t *codes;
    float *scale;
    const int64_t *count;
};

// |x| of 16 bf16 values: the largest, NaN left out
__device__ __forceinline__ float largest16(const uint4 &a, const uint4 &b)
{
    const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&a), *q = reinterpret_cast<const __nv_bfloat162 *>(&b);
    __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = __hmax2(m, __hmax2(__habs2(p[i]), __habs2(q[i])));
    return fmaxf(__low2float(m), __high2float(m));
}

__device__ __forceinline__ void widen16(const uint4 &a, const uint4 &b, float (&v)[16])
{
    const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&a), *q = reinterpret_cast<const __nv_bfloat162 *>(&b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(p[i]), g = __bfloat1622float2(q[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
        v[8 + 2 * i] = g.x;
        v[9 + 2 * i] = g.y;
    }
}

__device__ __forceinline__ float scale_for(float largest) { return fmaxf(largest / 448.f, qn::LEAST); }

// What the quotients by a block's scale need.  x / s is the product q = x (1/s)
// with one correction, q + (x - q s) (1/s) (Markstein's: with 1/s rounded
// correctly and the remainder exact, it is the rounded quotient).  It holds
// where neither the quotient nor the remainder leaves float32's range: s >= 2^-100
// keeps remainders of quotients that are not 0 in e4m3 above 2^-134, whose
// missing bits lie 2^16 below the rounding's, and 1/s is normal.  An infinite s
// has the reciprocal 0 and the remainder's s set to 0: 0 for finite x, NaN for
// an infinite one.  With divisions weights of 8 x 4096 x 7168 take 140 us instead
// of 109, rows of 32768 x 7168 150 instead of 113.
struct Divisor {
    float reciprocal, scale;
};
__device__ __forceinline__ Divisor divisor(float scale) { return {__frcp_rn(scale), isinf(scale) ? 0.f : scale}; }
__device__ __forceinline__ float quotient(float x, const Divisor &d)
{
    const float q = x * d.reciprocal;
    return fmaf(-fmaf(q, d.scale, -x), d.reciprocal, q); // (signs so that -0 stays -0)
}

// 16 codes: the quotients by the scale, clamped to +-448, to nearest even
__device__ __forceinline__ uint4 codes16(const float (&v)[16], float scale)
{
    const Divisor d = divisor(scale);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(quotient(v[4 * i], d), quotient(v[4 * i + 1], d)), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(quotient(v[4 * i + 2], d), quotient(v[4 * i + 3], d)), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// the largest of the 8 lanes that hold a block
__device__ __forceinline__ float largest_of_lanes(float v)
{
#pragma unroll
    for (int d = 1; d < qn::LANES; d <<= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

// rows are read once: past L1
__device__ __forceinline__ uint4 ld_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// silu(g) * u = g / (1 + 2^(-g log2 e)) * u by the approximate 2^x and reciprocal
// (2 ulp and 1).  The product -g log2 e is rounded, and log2 e is, to 2^-24 of
// it each: a negative gate's value is off by |g| 2^-23 relative, next to 2^-20 of
// all else, a positive one's by less than the latter.  A gate below -87 gives 0
// (1 + e leaves the reciprocal's range).  With expf and a division by 1 to 2 the
// kernel is bound by its instructions: 32768 rows of 2048 in 79 us instead of 53.
__device__ __forceinline__ float gated(float g, float u)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp2_approx(g * -1.44269504f)));
    return g * r * u;
}

// DEPTH blocks a thread, their loads in flight together; gated always one, by which
// 32768 x 2048 take 53 us and by two 67.  (Six CTAs an SM are asked for there, 40
// registers a thread: without that 59 us.)
template <bool GATED, int DEPTH>
__global__ void __launch_bounds__(qn::THREADS, GATED ? 6 : 1) quantise_rows_kernel(const __grid_constant__ QuantParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    int64_t rows = p.rows;
    if (p.count) {
        const int64_t n = *p.count;
        if ((n < 0 || n > rows) && blockIdx.x == 0 && threadIdx.x == 0)
            report_fault(p.status, TDG_ERR_DEVICE, TDG_WHERE_CU, 0, p.epoch);
        rows = n < 0 ? 0 : n < rows ? n : rows;
    }
    const int piece = threadIdx.x % qn::LANES;
    uint4 a[DEPTH], b[DEPTH], c[DEPTH], d[DEPTH];
    int64_t row[DEPTH], blk[DEPTH];
    bool in[DEPTH];
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
        const uint32_t u = (blockIdx.x * DEPTH + i) * qn::UNITS + threadIdx.x / qn::LANES; // (32 bits: with 64-bit divisions rows of 32768 x 7168 take 143 us instead of 113)
        const uint32_t r = u / (uint32_t)p.blocks;
        row[i] = r;
        blk[i] = u - r * (uint32_t)p.blocks;
        const int64_t col = blk[i] * 128 + piece * 16;
        in[i] = row[i] < rows && col < p.K;
        a[i] = b[i] = c[i] = d[i] = make_uint4(0, 0, 0, 0);
        if (in[i]) {
            const __nv_bfloat16 *src = p.x + row[i] * p.xs + col;
            a[i] = ld_stream(src);
            b[i] = ld_stream(src + 8);
            if (GATED) {
                c[i] = ld_stream(src + p.K);
                d[i] = ld_stream(src + p.K + 8);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
        float v[16], most;
        widen16(a[i], b[i], v);
        if (GATED) {
            float u[16];
            widen16(c[i], d[i], u);
            most = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                v[j] = gated(v[j], u[j]);
                most = fmaxf(most, fabsf(v[j]));
            }
        } else {
            most = largest16(a[i], b[i]);
        }
        const float s = scale_for(largest_of_lanes(most));
        if (in[i]) {
            *reinterpret_cast<uint4 *>(p.codes + row[i] * p.cs + blk[i] * 128 + piece * 16) = codes16(v, s);
            if (piece == 0)
                p.scale[row[i] * p.ss + blk[i]] = s;
        }
    }
}

// One CTA a 128 x 128 block of a matrix: 64 elements a thread, in registers
// between the maximum and the codes.
__global__ void __launch_bounds__(qn::THREADS) quantise_blocks_kernel(const __grid_constant__ QuantParams p, int64_t row_blocks)
{
    __shared__ float part[qn::THREADS / 32];
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t nb = (uint32_t)p.blocks, rbs = (uint32_t)row_blocks;
    const uint32_t band32 = blockIdx.x / nb, e32 = band32 / rbs; // band: of 128 rows, over all matrices
    const int64_t band = band32, blk = blockIdx.x - band32 * nb, e = e32, rb = band32 - e32 * rbs;
    const int piece = threadIdx.x % qn::LANES, first = threadIdx.x / qn::LANES;
    const int64_t col = blk * 128 + piece * 16;
    const int left = (int)min((int64_t)128, p.rows - rb * 128); // rows of this block
    const int64_t row0 = e * p.rows + rb * 128;
    uint4 a[4], b[4];
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = first + i * qn::UNITS;
        a[i] = b[i] = make_uint4(0, 0, 0, 0);
        if (r < left && col < p.K) {
            const __nv_bfloat16 *src = p.x + (row0 + r) * p.xs + col;
            a[i] = ld_stream(src);
            b[i] = ld_stream(src + 8);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        most = fmaxf(most, largest16(a[i], b[i]));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < qn::THREADS / 32; ++i)
        most = fmaxf(most, part[i]);
    const float s = scale_for(most);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = first + i * qn::UNITS;
        if (r < left && col < p.K) {
            float v[16];
            widen16(a[i], b[i], v);
            *reinterpret_cast<uint4 *>(p.codes + (row0 + r) * p.cs + col) = codes16(v, s);
        }
    }
    if (threadIdx.x == 0)
        p.scale[band * p.blocks + blk] = s;
}

// Dispatch: a token's block is read and quantised once and written to its k rows.
__global__ void __launch_bounds__(qn::THREADS) moe_dispatch_e4m3_kernel(const __grid_constant__ MoeRows m, uint64_t x_off,
                                                                       uint8_t *codes, float *scale, int64_t blocks)
{
    griddep_launch_dependents();
    griddep_wait();
    const int piece = threadIdx.x % qn::LANES;
    const uint32_t u = blockIdx.x * qn::UNITS + threadIdx.x / qn::LANES, tok32 = u / (uint32_t)blocks;
    const int64_t tok = tok32, blk = u - tok32 * (uint32_t)blocks; // tok: src * T + t
    const int64_t col = blk * 128 + piece * 16;
    const bool token = tok < m.tokens, in = token && col < m.H;
    // The rows of 8 choices, one a lane: read together and before x, not each behind the
    // store before (128 tokens of 7168, 8 choices, on several GPUs: 3.5 to 6.7 us, and 3.4
    // to 3.5 like this; 8192 tokens 90.7 and 91.7).
    auto rows_from = [&](int k0) { return token && k0 + piece < m.k ? (int)moe_row(m, tok, k0 + piece, blk == 0) : -1; };
    int mine = rows_from(0);
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (in) {
        const uint32_t src = tok32 / (uint32_t)m.T, t = tok32 - src * (uint32_t)m.T;
        const uint8_t *at = m.regions + (uint64_t)src * m.region_bytes + x_off + ((uint64_t)t * m.H + col) * 2;
        a = ld_stream(at);
        b = ld_stream(at + 16);
    }
    const float s = scale_for(largest_of_lanes(largest16(a, b)));
    float v[16];
    widen16(a, b, v);
    const uint4 c = codes16(v, s);
    for (int k0 = 0; k0 < m.k; k0 += qn::LANES) {
        if (k0)
            mine = rows_from(k0);
#pragma unroll
        for (int j = 0; j < qn::LANES; ++j) {
            const int64_t row = __shfl_sync(0xffffffffu, mine, j, qn::LANES);
            if (!in || row < 0)
                continue;
            *reinterpret_cast<uint4 *>(codes + row * m.H + col) = c;
            if (piece == 0)
                scale[row * blocks + blk] = s;
        }
    }
}

} // namespace tdg

using namespace tdg;
using namespace tdg_host;

extern "C" int tdg_quantise(tdg_symm *h, const tdg_quantise_args *a, void *stream)
{
    if (!h || !a)
        return TDG_ERR_INVALID;
    if (const int drc = check_device(h))
        return drc;
    const bool gate = a->kind == TDG_QUANT_GATED, blocks = a->kind == TDG_QUANT_BLOCKS;
    if (a->kind < TDG_QUANT_ROWS || a->kind > TDG_QUANT_BLOCKS || a->rows < 0 || a->rows > INT32_MAX || a->E < 0 || a->E > INT32_MAX ||
        (!blocks && a->E != 1) || a->K < 16 || a->K % 16 || a->K >= (1 << 30))
        return TDG_ERR_INVALID;
    if (a->E && a->rows > INT32_MAX / a->E)
        return TDG_ERR_INVALID;
    const int64_t rows = a->rows * a->E, kb = (a->K + 127) / 128, width = gate ? 2 * a->K : a->K;
    if (rows == 0)
        return TDG_OK;
    if (!a->x || !aligned16(a->x) || !a->codes || !aligned16(a->codes) || !a->scale || !aligned4(a->scale) || (blocks && a->count) ||
        !aligned8(a->count) || !stride_ok(a->x_stride, width, 8) || !stride_ok(a->codes_stride, a->K, 16) ||
        !stride_ok(a->scale_stride, kb, 1) || (blocks && a->scale_stride != kb))
        return TDG_ERR_INVALID;
    const int64_t bands = (a->rows + 127) / 128; // of one matrix
    const Range x{a->x, extent(rows, a->x_stride, width, 2)}, codes{a->codes, extent(rows, a->codes_stride, a->K, 1)};
    const Range scale{a->scale, extent(blocks ? bands * a->E : a->rows, a->scale_stride, kb, 4)}, count{a->count, 8};
    const ByteRows xr{a->x, 2 * a->x_stride, 2 * width}, cr{a->codes, a->codes_stride, a->K}, sr{a->scale, 4 * a->scale_stride, 4 * kb};
    if (ranges_overlap({codes, scale}, {count}) || rows_share(rows, cr, xr) ||
        (blocks ? ranges_overlap({scale}, {x, codes}) : rows_share(rows, sr, xr) || rows_share(rows, sr, cr)))
        return TDG_ERR_INVALID;
    QuantParams p;
    memset(&p, 0, sizeof p);
    p.status = h->status;
    p.epoch = next_epoch(h);
    p.rows = a->rows;
    p.K = a->K;
    p.xs = a->x_stride;
    p.cs = a->codes_stride;
    p.ss = a->scale_stride;
    p.blocks = kb;
    p.x = static_cast<const __nv_bfloat16 *>(a->x);
    p.codes = static_cast<uint8_t *>(a->codes);
    p.scale = a->scale;
    p.count = a->count;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (blocks) {
        int64_t row_blocks = bands;
        const int64_t grid = bands * a->E * kb;
        if (grid > INT32_MAX)
            return TDG_ERR_INVALID;
        void *args[] = {&p, &row_blocks};
        return cuda_err(launch(reinterpret_cast<const void *>(&quantise_blocks_kernel), dim3((unsigned)grid), dim3(qn::THREADS), 0, s, args,
                               false, 1, true),
                        "quantise blocks launch");
    }
    const int64_t units = rows * kb;
    const int depth = !gate && units > (int64_t)h->sm_count * 8 * qn::UNITS ? 2 : 1;
    const int64_t grid = (units + depth * qn::UNITS - 1) / (depth * qn::UNITS);
    if (units > UINT32_MAX - 4 * qn::UNITS)
        return TDG_ERR_INVALID;
    const void *fn = gate         ? reinterpret_cast<const void *>(&quantise_rows_kernel<true, 1>)
                     : depth == 2 ? reinterpret_cast<const void *>(&quantise_rows_kernel<false, 2>)
                                  : reinterpret_cast<const void *>(&quantise_rows_kernel<false, 1>);
    void *args[] = {&p};
    return cuda_err(launch(fn, dim3((unsigned)grid), dim3(qn::THREADS), 0, s, args, false, 1, true), "quantise rows launch");
}

extern "C" int tdg_moe_dispatch_e4m3(tdg_symm *h, const tdg_moe_dispatch_e4m3_args *a, void *stream)
{
    if (!h || !a)
        return TDG_ERR_INVALID;
    if (const int drc = check_device(h))
        return drc;
    MoeRows m;
    if (const int rc = moe_rows(h, a->world, a->k, a->T, a->H, a->slot, 16, m))
        return rc;
    if (a->T == 0)
        return TDG_OK;
    const int64_t blocks = (a->H + 127) / 128, rows = m.rows;
    const uint64_t shard = (uint64_t)a->T * a->H * 2;
    if (!a->slot || !a->codes || !aligned16(a->codes) || !a->scale || !aligned4(a->scale) || !aligned16(a->x_off))
        return TDG_ERR_INVALID;
    if (!in_region(h, a->x_off, shard))
        return TDG_ERR_NOMEM;
    const Range codes{a->codes, (uint64_t)rows * a->H}, scale{a->scale, (uint64_t)rows * blocks * 4}, slot{a->slot, (uint64_t)rows * 8};
    if (ranges_overlap({codes, scale}, {slot}) || ranges_overlap({codes}, {scale}) || shards_overlap(h, a->x_off, shard, {codes, scale}))
        return TDG_ERR_INVALID;
    const int64_t grid = (m.tokens * blocks + qn::UNITS - 1) / qn::UNITS;
    if (m.tokens * blocks > UINT32_MAX - 4 * qn::UNITS)
        return TDG_ERR_INVALID;
    m.epoch = next_epoch(h);
    uint64_t x_off = a->x_off;
    uint8_t *c = static_cast<uint8_t *>(a->codes);
    float *sc = a->scale;
    int64_t kb = blocks;
    void *args[] = {&m, &x_off, &c, &sc, &kb};
    return cuda_err(launch(reinterpret_cast<const void *>(&moe_dispatch_e4m3_kernel), dim3((unsigned)grid), dim3(qn::THREADS), 0,
                           static_cast<cudaStream_t>(stream), args, false, 1, true),
                    "moe dispatch e4m3 launch");
}
