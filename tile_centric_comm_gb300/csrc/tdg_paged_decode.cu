// tdg_paged_decode.cu -- attention of one new token per sequence over the
// paged cache: softmax(scale q K^T) V over lens[b] cached tokens.
//
// Mathematics: with scores in base 2, a running maximum m and sum l per query
// head, each group of 16 tokens updates  m' = max(m, s),  l' = l 2^(m - m') +
// sum 2^(s - m'),  o' = o 2^(m - m') + P V;  partial results (m, l, o) join the
// same way.  All of m, l, o are float32; P is rounded to bf16 for the
// product, the only rounding besides the output's (keys and queries of an
// 8-bit cache meet in f16, exactly but for elements below 2^-17 of a query's
// largest).
//
// Bound by HBM: K and V are read once, about 2 G flops per byte, for up to 16
// query heads a key head (G = Hq/Hkv): they are the 16 rows of mma.sync
// (m16n8k16).  More heads are taken in groups of 16, each of which fetches the
// pages for itself: 64 sequences of 1..16384 on one key head 52 us with 16 query
// heads, 77 with 20 or 32, 230 with 128 (8-bit 191).
//
// Split: the (sequence, key head) pairs' tiles (64 tokens; 128 of an 8-bit
// cache) form one long line, in which a pair also counts for the tiles that its
// beginning and end cost, and each of the two CTAs per SM takes an equal run of
// it, wherever it begins and ends: ragged lengths leave no SM idle, and the
// partial results are at most two per CTA whatever the lengths.  A second launch
// joins the split pairs.  When the pairs are few and short, a cluster takes each
// one and joins through distributed shared memory, in one launch.
//
// In a CTA, warp 4 looks up page ids and issues one TMA copy per page (or
// tile) for K and for V into a ring of stages; warps 0-3 each take 16 tokens
// of every tile (32 of an 8-bit cache: two chains of work to interleave).  The
// 5-D tensor map (one box is a tile's tokens of the page, both 128-byte halves
// of a 256-byte row in one copy) writes the 128-byte-swizzled layout that
// ldmatrix reads without bank conflicts.
//
// Measured on one GB300 (copy rate 6.79 TB/s), 64 / 8 heads of 128, both launches:
//   2 sequences of 200,000..262,144          288 us, 7.0 TB/s
//   64 of 1..8192, pages of 16               174 us, 6.6 TB/s
//   128 of 2048..4096, 8-bit                 145 us, 5.5 TB/s: the conversions
//                                            e4m3 -> f16 -> bf16 and what waits
//                                            for them (44 bytes a thread spilled, 68
//                                            with clusters; three CTAs an SM spill more)
//   64 of 1..512                             19 us, 4.3 TB/s: pairs of a few tiles
//   one sequence of 1000                     7.3 to 7.7 us in a table as wide as it
//                                            (a cluster a pair: launch, lookups, two
//                                            tiles), 9.0 in one of 131,072 tokens
//   64 of 1..8192, 64 / 8 heads of 64        94 us, 5.9 TB/s; 8-bit 63 us, 4.4 TB/s
#include <cuda_fp16.h>

#include "tdg_paged.cuh"

namespace tdg {

namespace pd {
constexpr int WARPS = 4;                      // consumer warps
constexpr int THREADS = WARPS * 32 + 32;
constexpr int MAX_CTAS = 512;                 // CTAs whose partial results the caller provides room for
constexpr int ROWS = 16;                      // query heads of a partial result
constexpr int JOIN_ROWS = 2;                  // rows of a join CTA
constexpr int JOIN_THREADS = 256;
constexpr int BAR_BYTES = 384;
constexpr int MAX_SPLIT = 8;                  // CTAs of a cluster (PAIRS)
// What a pair costs beside its tiles, in tiles: its queries and the join of the
// four warps.  With runs equal in tiles alone the CTAs of the short sequences were
// the last: 64 sequences of 1..512 27.5 us, 19 with 2 (20.9 with 1, 18.7 with 3),
// 128 of 2048..4096 in 8 bits 144.5 (146.1 with 3).
constexpr int PAIR_UNITS = 2;

template <int D, bool E4M3> struct Shape {
    static constexpr int ESZ = E4M3 ? 1 : 2;
    static constexpr int NG = E4M3 ? 2 : 1;                   // groups of 16 tokens that a warp takes at once
    static constexpr int TILE = WARPS * NG * 16;              // tokens of a tile
    static constexpr int RB = D * ESZ < 128 ? D * ESZ : 128; // bytes of a block's row
    static constexpr int NB = D * ESZ / RB;                   // blocks of a token's row
    static constexpr int KV = TILE * D * ESZ;                 // bytes of a tile of K or of V
    static constexpr int STAGES = KV >= 16384 ? 3 : 6;
    static constexpr int Q_BYTES = ROWS * D * 2;
    static constexpr int OFF_Q = STAGES * 2 * KV;
    static constexpr int ML_FLOATS = WARPS * ROWS * 2;        // the warps' maxima and sums of a pair
    static constexpr int OFF_ML = OFF_Q + 2 * Q_BYTES;
    static constexpr int OFF_BAR = OFF_ML + 2 * ML_FLOATS * 4;
    // A warp's own keys and values of a tile are as many bytes as its 16 rows
    // of output, in pieces of 16 rows: a piece takes COLS columns.
    static constexpr int PIECES = 2 * NG * NB, COLS = D / PIECES;
    static_assert(COLS * 4 == RB, "a piece's rows are a block's");
    static constexpr int SMEM = OFF_BAR + BAR_BYTES;
};
static_assert(2 * (Shape<128, false>::SMEM + 1024) <= 228 * 1024 && 2 * (Shape<128, true>::SMEM + 1024) <= 228 * 1024,
              "two CTAs per SM");
} // namespace pd

struct PagedDecodeParams {
    DevStatus *status;
    uint32_t epoch;
    PagedView c;
    int64_t B, table_entries, table_stride, qs, os;
    int Hq, G, groups; // groups of 16 query heads per key head
    int box;           // tokens of one TMA copy
    int split;         // CTAs that share a pair (PAIRS)
    float scale_log2;
    uint64_t timeout_ns;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    float *lse;
    const int32_t *table, *lens;
    int4 *desc;     // [MAX_CTAS]: the split pair that ends in a CTA (sequence or -1, line, first CTA, pd_tag)
    float *part_ml; // [MAX_CTAS][2][ROWS][2]
    float *part_o;  // [MAX_CTAS][2][ROWS][D]
};

// A position on the line of tiles: tile `tile` of the pair (b, hg).
struct PdWalk {
    int64_t b;
    int hg, tile, tiles;
};

struct PdBars {
    uint64_t kfull[8], vfull[8], empty[8], qfull[2], qempty[2];
    int64_t sums[pd::THREADS / 32];
    PdWalk begin;
};
static_assert(sizeof(PdBars) <= pd::BAR_BYTES, "barrier block");

__device__ __forceinline__ void pd_ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void pd_ldsm4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// c += a b, one m16n8k16 tile with bf16 or f16 inputs
template <bool F16>
__device__ __forceinline__ void pd_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// two 8-bit floats (the low or the high half of r) as two f16, exactly
__device__ __forceinline__ uint32_t e4m3x2_lo(uint32_t r)
{
    uint32_t d;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(r));
    return d;
}
__device__ __forceinline__ uint32_t e4m3x2_hi(uint32_t r)
{
    uint32_t d;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(d) : "r"(r));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// two f16 that hold 8-bit floats, as bf16 (exact: 4 significant bits)
__device__ __forceinline__ uint32_t f16x2_bf16x2(uint32_t r)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r));
    return pack_bf16x2(f.x, f.y);
}

// e for a row whose largest magnitude is `top`, so that the row times 2^-e lies
// within +-2 (+-4 from 2^127 on): f16 (whose smallest step is 2^-24) then holds every bf16 value, of
// 8 significant bits, down to 2^-17 of the largest exactly and the smaller ones
// to 2^-25 of it.
__device__ __forceinline__ int pd_exponent(float top)
{
    const int e = (int)(__float_as_uint(top) >> 23) - 127;
    return top > 0.f && top < INFINITY ? min(max(e, -126), 126) : 0;
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// tiles of sequence b; a length that does not fit the table counts as none
template <int TILE> __device__ __forceinline__ int pd_tiles(const PagedDecodeParams &p, int64_t b)
{
    const int64_t len = p.lens[b];
    return len <= 0 || len > p.table_entries << p.c.ps_log2 ? 0 : (int)((len + TILE - 1) / TILE);
}

// what one pair of sequence b is on the line: its tiles, behind what a pair costs
// beside them (its queries, and the join of the four warps)
template <int TILE> __device__ __forceinline__ int64_t pd_units(const PagedDecodeParams &p, int64_t b)
{
    const int tiles = pd_tiles<TILE>(p, b);
    return tiles ? tiles + pd::PAIR_UNITS : 0;
}

// What a description ends with: in which of its first CTA's two places the pair
// lies, behind the call's epoch (below 2^31).  The join takes only its own call's
// descriptions: another call that has the same room at the same time may be of
// other sizes, and what it describes may lie outside this one's output.
__device__ __forceinline__ int pd_tag(const PagedDecodeParams &p, int place) { return (int)(p.epoch << 1 | (uint32_t)place); }

// the first CTA whose run holds unit u, given total = base * ctas + rem
__device__ __forceinline__ int pd_owner(int64_t u, int64_t base, int64_t rem)
{
    return (int)(u < rem * (base + 1) ? u / (base + 1) : rem + (u - rem * (base + 1)) / base);
}

// Scores, softmax update and output update of this warp's NG groups of 16
// tokens of a tile.  valid: tokens of them that exist (all unless TAIL); at:
// shared addresses of the groups' key rows, the value rows S::KV behind; blk:
// bytes between a row's 128-byte blocks.
template <int D, bool E4M3, bool TAIL, class WaitV>
__device__ __forceinline__ void pd_group(const uint32_t (&qa)[D / 16][4], const float (&mul)[2],
                                         const uint32_t (&at)[pd::Shape<D, E4M3>::NG], uint32_t blk, int valid, int lane,
                                         float (&m)[2], float (&l)[2], float (&o)[D / 8][4], WaitV &&wait_v)
{
    using S = pd::Shape<D, E4M3>;
    constexpr int NG = S::NG;
    const int tig = lane & 3, mi = lane >> 3, ri = lane & 7;
    float s[NG][2][4];
    auto swz = [](int row) -> uint32_t { return S::RB == 128 ? (uint32_t)(row & 7) << 4 : (uint32_t)((row >> 1) & 3) << 4; };
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s[g][i / 4][i % 4] = 0.f;
    if constexpr (!E4M3) {
        const int tok = (mi >> 1) * 8 + ri;
        const uint32_t row = tok * S::RB, x = swz(tok) ^ ((mi & 1) * 16);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint32_t b[4];
                pd_ldsm4(at[g] + row + (ks / 4) * blk + (x ^ ((ks % 4) * 32)), b);
                pd_mma<false>(s[g][0], qa[ks], b[0], b[1]);
                pd_mma<false>(s[g][1], qa[ks], b[2], b[3]);
            }
    } else {
        // a lane's four bytes are four neighbouring dimensions of one token;
        // the query's fragments are laid out in the same order
        const int tok = (mi & 1) * 8 + ri;
        const uint32_t row = tok * S::RB, x = swz(tok) ^ ((mi >> 1) * 16);
#pragma unroll
        for (int ks = 0; ks < D / 16; ks += 2)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint32_t b[4];
                pd_ldsm4(at[g] + row + (x ^ (ks * 16)), b);
                pd_mma<true>(s[g][0], qa[ks], e4m3x2_lo(b[0]), e4m3x2_hi(b[0]));
                pd_mma<true>(s[g][1], qa[ks], e4m3x2_lo(b[1]), e4m3x2_hi(b[1]));
                pd_mma<true>(s[g][0], qa[ks + 1], e4m3x2_lo(b[2]), e4m3x2_hi(b[2]));
                pd_mma<true>(s[g][1], qa[ks + 1], e4m3x2_lo(b[3]), e4m3x2_hi(b[3]));
            }
    }
    // base-2 scores; tokens behind the length weigh nothing, whatever their key holds
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[g][nt][c] *= mul[c / 2];
                if (TAIL && g * 16 + nt * 8 + tig * 2 + (c & 1) >= valid)
                    s[g][nt][c] = -INFINITY;
            }
    // m follows the row's true maximum only when that has grown by more than 8
    // (a factor of 256), so the output is rarely rescaled; weights stay below
    // 2^8, and any m serves the sums as well as another
    bool grown = false;
    float al[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float mx = -INFINITY;
#pragma unroll
        for (int g = 0; g < NG; ++g)
            mx = fmaxf(mx, fmaxf(fmaxf(s[g][0][2 * r], s[g][0][2 * r + 1]), fmaxf(s[g][1][2 * r], s[g][1][2 * r + 1])));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const bool up = mx - m[r] > 8.f; // also from -inf
        al[r] = up ? exp2_approx(m[r] - mx) : 1.f;
        m[r] = up ? mx : m[r];
        grown = grown || up;
        const float ms = m[r] == -INFINITY ? 0.f : m[r];
        float sum = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    s[g][nt][2 * r + c] = exp2_approx(s[g][nt][2 * r + c] - ms);
                    sum += s[g][nt][2 * r + c];
                }
        l[r] = l[r] * al[r] + sum; // this lane's share; the four lanes of a row are added at the end
    }
    if (__any_sync(0xffffffffu, grown))
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            o[n][0] *= al[0];
            o[n][1] *= al[0];
            o[n][2] *= al[1];
            o[n][3] *= al[1];
        }
    wait_v();
    const int vtok = (mi & 1) * 8 + ri;
    const uint32_t vrow = S::KV + vtok * S::RB, vx = swz(vtok) ^ ((mi >> 1) * 16);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        // bf16 for an 8-bit cache too: f16 is finer, but it loses weights below
        // 2^-24 of the largest, which carry an output whose heavy tokens hold 0
        const uint32_t pa[4] = {pack_bf16x2(s[g][0][0], s[g][0][1]), pack_bf16x2(s[g][0][2], s[g][0][3]),
                                pack_bf16x2(s[g][1][0], s[g][1][1]), pack_bf16x2(s[g][1][2], s[g][1][3])};
        // a register of V holds tokens 2 tig, 2 tig + 1 (+ 8); those behind the
        // length are cleared, since 0 times infinity or NaN is not 0
        uint32_t keep[2] = {~0u, ~0u};
        if (TAIL)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = g * 16 + i * 8 + tig * 2;
                keep[i] = (t < valid ? 0x0000FFFFu : 0u) | (t + 1 < valid ? 0xFFFF0000u : 0u);
            }
        if constexpr (!E4M3) {
#pragma unroll
            for (int nd = 0; nd < D / 8; nd += 2) {
                uint32_t b[4];
                pd_ldsm4_t(at[g] + vrow + (nd / 8) * blk + (vx ^ ((nd % 8) * 16)), b);
                if (TAIL) {
                    b[0] &= keep[0];
                    b[1] &= keep[1];
                    b[2] &= keep[0];
                    b[3] &= keep[1];
                }
                pd_mma<false>(o[nd], pa, b[0], b[1]);
                pd_mma<false>(o[nd + 1], pa, b[2], b[3]);
            }
        } else {
            // 16 dimensions per matrix; a register holds two neighbouring
            // dimensions of two tokens, sorted into one product of the even
            // dimensions and one of the odd
#pragma unroll
            for (int j = 0; j < D / 16; j += 2) {
                uint32_t b[4];
                pd_ldsm4_t(at[g] + vrow + (vx ^ (j * 16)), b);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    b[i] = __byte_perm(TAIL ? b[i] & keep[i & 1] : b[i], 0u, 0x3120);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    pd_mma<false>(o[2 * (j + i)], pa, f16x2_bf16x2(e4m3x2_lo(b[2 * i])), f16x2_bf16x2(e4m3x2_lo(b[2 * i + 1])));
                    pd_mma<false>(o[2 * (j + i) + 1], pa, f16x2_bf16x2(e4m3x2_hi(b[2 * i])), f16x2_bf16x2(e4m3x2_hi(b[2 * i + 1])));
                }
            }
        }
    }
}

// Joins the shares of a cluster's pair: each CTA takes some of its rows, four
// columns a thread, and reads all shares' maxima, sums and outputs in one round
// of loads.
template <int D, bool E4M3> __device__ void pd_join_pair(const PagedDecodeParams &p, uint8_t *smem, const PdWalk &w)
{
    if (p.split == 1 || w.tiles <= 1) // one CTA had it all (the same for all of the cluster)
        return;
    __syncwarp();
    cluster_sync();
    const int g = w.hg / p.groups, mg = w.hg % p.groups, rows = min(pd::ROWS, p.G - mg * pd::ROWS);
    const int per = pd::ROWS / p.split, row0 = (int)cluster_ctarank() * per;
    using S = pd::Shape<D, E4M3>;
    const uint32_t out_at = smem_u32(smem + S::OFF_Q), ml_at = smem_u32(smem + S::OFF_ML); // (pair is 1 when they are left)
    for (int u = threadIdx.x; u < per * (D / 4); u += pd::THREADS) {
        const int row = row0 + u / (D / 4), c4 = u % (D / 4) * 4;
        if (row >= rows)
            break;
        float2 ml[pd::MAX_SPLIT];
        float4 x[pd::MAX_SPLIT];
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int c = 0; c < pd::MAX_SPLIT; ++c) {
            ml[c] = make_float2(-INFINITY, 0.f);
            x[c] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < p.split && w.tiles * (c + 1) / p.split > w.tiles * c / p.split) { // a share that has tiles
                ml[c] = ld_cluster_f2(mapa_shared(ml_at + row * 8, (uint32_t)c));
                x[c] = ld_cluster_f4(mapa_shared(out_at + (row * D + c4) * 4, (uint32_t)c));
            }
        }
#pragma unroll
        for (int c = 0; c < pd::MAX_SPLIT; ++c)
            M = fmaxf(M, ml[c].x);
        const float Ms = M == -INFINITY ? 0.f : M;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < pd::MAX_SPLIT; ++c) {
            const float wt = exp2_approx(ml[c].x - Ms);
            L += ml[c].y * wt;
            a.x += x[c].x * wt;
            a.y += x[c].y * wt;
            a.z += x[c].z * wt;
            a.w += x[c].w * wt;
        }
        const int h = g * p.G + mg * pd::ROWS + row;
        const float f = (E4M3 ? p.c.v_scale[g] : 1.f) / L;
        *reinterpret_cast<uint2 *>(p.out + w.b * p.os + (int64_t)h * D + c4) =
            make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
        if (p.lse && c4 == 0)
            p.lse[w.b * p.Hq + h] = (M + log2f(L)) * 0.6931471805599453f;
    }
    __syncwarp();
    cluster_sync(); // no CTA leaves while another reads its shared memory
}

// PAIRS: a cluster of p.split CTAs takes one pair and joins through distributed
// shared memory; otherwise a CTA takes its run of the line.
template <int D, bool E4M3, bool PAIRS> __global__ void __launch_bounds__(pd::THREADS, 2)
    paged_decode_kernel(const __grid_constant__ PagedDecodeParams p, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap)
{
    using S = pd::Shape<D, E4M3>;
    extern __shared__ __align__(1024) uint8_t smem[];
    PdBars *bar = reinterpret_cast<PdBars *>(smem + S::OFF_BAR);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pairs = p.c.Hkv * p.groups; // lines of tiles per sequence

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(&bar->kfull[i], 1);
            mbar_init(&bar->vfull[i], 1);
            mbar_init(&bar->empty[i], pd::WARPS);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar->qfull[i], 1);
            mbar_init(&bar->qempty[i], pd::WARPS);
        }
        fence_mbar_init();
        fence_proxy_async_smem();
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    // launched while the kernel before may still run: nothing above touches memory
    griddep_launch_dependents();
    griddep_wait();
    int64_t u0, u1, base = 0, rem = 0;
    PdWalk w;
    if constexpr (PAIRS) {
        // this CTA's share of its pair; u counts the pair's own tiles
        const int pair = (int)(blockIdx.x / (unsigned)p.split), rank = (int)(blockIdx.x % (unsigned)p.split);
        w.b = pair / pairs;
        w.hg = pair % pairs;
        w.tiles = pd_tiles<S::TILE>(p, w.b);
        u0 = w.tiles * rank / p.split;
        u1 = w.tiles * (rank + 1) / p.split;
        w.tile = (int)u0;
        if (w.tiles == 0 && rank == 0) { // no tokens, or a bad length
            if (w.hg == 0 && threadIdx.x == 0 && p.lens[w.b] != 0)
                report_fault(p.status, TDG_ERR_DEVICE, TDG_WHERE_PAGE, (uint32_t)w.b, p.epoch);
            const int h0 = w.hg / p.groups * p.G + w.hg % p.groups * pd::ROWS, rows = min(pd::ROWS, p.G - w.hg % p.groups * pd::ROWS);
            for (int i = threadIdx.x; i < rows * D / 8; i += pd::THREADS)
                *reinterpret_cast<uint4 *>(p.out + w.b * p.os + (int64_t)h0 * D + (int64_t)i * 8) = make_uint4(0, 0, 0, 0);
            if (p.lse && (int)threadIdx.x < rows)
                p.lse[w.b * p.Hq + h0 + threadIdx.x] = -INFINITY;
        }
        __syncthreads(); // the barriers are ready
    } else {
        // this CTA's run of the line: the warps' sums of tiles, then the sequence
        // in which the run begins
        const int64_t per = (p.B + pd::THREADS - 1) / pd::THREADS; // sequences of a thread
        const int64_t b_lo = min((int64_t)threadIdx.x * per, p.B), b_hi = min(b_lo + per, p.B);
        int64_t mine = 0;
        for (int64_t b = b_lo; b < b_hi; ++b)
            mine += pd_units<S::TILE>(p, b);
        int64_t upto = mine;
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d)
                upto += x;
        }
        if (lane == 31)
            bar->sums[warp] = upto;
        // sequences without tokens (and those of a bad length) are nobody's run
        for (int64_t b = blockIdx.x; b < p.B; b += gridDim.x)
            if (pd_tiles<S::TILE>(p, b) == 0) {
                if (p.lens[b] != 0 && threadIdx.x == 0)
                    report_fault(p.status, TDG_ERR_DEVICE, TDG_WHERE_PAGE, (uint32_t)b, p.epoch);
                for (int i = threadIdx.x; i < p.Hq * D / 8; i += pd::THREADS)
                    *reinterpret_cast<uint4 *>(p.out + b * p.os + (int64_t)i * 8) = make_uint4(0, 0, 0, 0);
                if (p.lse)
                    for (int i = threadIdx.x; i < p.Hq; i += pd::THREADS)
                        p.lse[b * p.Hq + i] = -INFINITY;
            }
        __syncthreads();
        int64_t total = 0, before = 0;
        for (int i = 0; i < pd::THREADS / 32; ++i) {
            if (i < warp)
                before += bar->sums[i];
            total += bar->sums[i];
        }
        upto += before;
        base = total * pairs / gridDim.x;
        rem = total * pairs % gridDim.x;
        u0 = blockIdx.x * base + min((int64_t)blockIdx.x, rem);
        u1 = u0 + base + (blockIdx.x < rem ? 1 : 0);
        if ((upto - mine) * pairs <= u0 && u0 < upto * pairs && u0 < u1) {
            int64_t at = u0 - (upto - mine) * pairs;
            for (w.b = b_lo;; ++w.b) {
                const int64_t units = pd_units<S::TILE>(p, w.b);
                if (at < units * pairs) {
                    w.tiles = (int)(units - pd::PAIR_UNITS);
                    w.hg = (int)(at / units);
                    w.tile = (int)(at % units) - pd::PAIR_UNITS; // below 0: the pair's tiles begin so far on
                    break;
                }
                at -= units * pairs;
            }
            bar->begin = w;
        }
        __syncthreads();
        if (u0 >= u1) {
            if (threadIdx.x == 0)
                p.desc[blockIdx.x] = make_int4(-1, 0, 0, pd_tag(p, 0));
            return;
        }
        w = bar->begin;
    }
    int64_t u = u0;
    if (w.tile < 0) {
        u -= w.tile;
        w.tile = 0;
    }
    // the next pair, of the next sequence that has tiles (there is one while u < u1)
    auto next_pair = [&](PdWalk &x) {
        x.tile = 0;
        if (++x.hg == pairs) {
            x.hg = 0;
            do {
                x.tiles = pd_tiles<S::TILE>(p, ++x.b);
            } while (x.tiles == 0);
        }
    };

    if (warp == pd::WARPS) {
        // ---- loads: a chunk is up to 32 copies of one pair, their page ids one per lane ----
        const int per_tile = S::TILE / p.box;               // copies of a tile
        const int shift = p.c.ps_log2;
        const int box_log2 = 31 - __clz(p.box);
        const uint32_t copy_bytes = (uint32_t)p.box * D * S::ESZ;
        auto chunk_ids = [&](const PdWalk &x, int tiles) -> int32_t {
            const int64_t tok = (int64_t)x.tile * S::TILE + ((int64_t)lane << box_log2);
            if (lane >= tiles * per_tile || tok >= p.lens[x.b])
                return 0;
            const int32_t id = p.table[x.b * p.table_stride + (tok >> shift)];
            if (id >= 0 && id < p.c.all_pages)
                return id;
            report_fault(p.status, TDG_ERR_DEVICE, TDG_WHERE_PAGE, (uint32_t)x.b, p.epoch);
            return 0; // any page: the result is undefined, the access is not
        };
        auto chunk_tiles = [&](const PdWalk &x, int64_t at) -> int {
            return (int)min(min((int64_t)(32 / per_tile), (int64_t)(x.tiles - x.tile)), u1 - at);
        };
        int n = u < u1 ? chunk_tiles(w, u) : 0, stage = 0, pair = 0;
        uint32_t phase = 0;
        bool fresh = true, dead = false;
        int32_t ids = n ? chunk_ids(w, n) : 0;
        int64_t issued = 0;
        int queries = 0; // query copies issued
        while (n && !dead) {
            // look the next chunk up while this one's copies are issued
            PdWalk y = w;
            y.tile += n;
            u += n;
            if (y.tile == y.tiles && u < u1) {
                next_pair(y);
                u += pd::PAIR_UNITS;
            }
            const int n2 = u < u1 ? chunk_tiles(y, u) : 0;
            const int32_t ids2 = n2 ? chunk_ids(y, n2) : 0;
            const int64_t len = p.lens[w.b];
            const int g = w.hg / p.groups;
            if (fresh && lane == 0) { // a new pair: its queries
                const int h0 = g * p.G + (w.hg % p.groups) * pd::ROWS;
                const uint32_t bytes = (uint32_t)min(pd::ROWS, p.G - (w.hg % p.groups) * pd::ROWS) * D * 2;
                const int qb = pair & 1;
                if (!mbar_wait(&bar->qempty[qb], ((pair >> 1) & 1) ^ 1u, p.timeout_ns)) {
                    report_fault(p.status, TDG_ERR_TIMEOUT, TDG_WHERE_PIPE, 0, p.epoch);
                    dead = true;
                } else {
                    mbar_arrive_expect_tx(&bar->qfull[qb], bytes);
                    bulk_load(smem + S::OFF_Q + qb * S::Q_BYTES, p.q + w.b * p.qs + (int64_t)h0 * D, bytes, &bar->qfull[qb]);
                    queries = pair + 1;
                }
            }
            dead = __shfl_sync(0xffffffffu, dead ? 1 : 0, 0) != 0;
            for (int i = 0; i < n && !dead; ++i) {
                const int64_t t0 = (int64_t)(w.tile + i) * S::TILE;
                const int copies = (int)min((int64_t)per_tile, (len - t0 + p.box - 1) >> box_log2);
                if (lane == 0) {
                    if (!mbar_wait(&bar->empty[stage], phase ^ 1u, p.timeout_ns)) {
                        report_fault(p.status, TDG_ERR_TIMEOUT, TDG_WHERE_PIPE, 1, p.epoch);
                        dead = true;
                    } else {
                        mbar_arrive_expect_tx(&bar->kfull[stage], copies * copy_bytes);
                        mbar_arrive_expect_tx(&bar->vfull[stage], copies * copy_bytes);
                    }
                }
                dead = __shfl_sync(0xffffffffu, dead ? 1 : 0, 0) != 0;
                if (dead)
                    break;
                const int32_t id = __shfl_sync(0xffffffffu, ids, (i * per_tile + lane) & 31);
                if (lane < copies) {
                    const int row = (int)((t0 + ((int64_t)lane << box_log2)) & ((1 << shift) - 1)); // inside the page
                    const int rank = id / (int)p.c.pages, local = id % (int)p.c.pages;
                    uint8_t *dst = smem + stage * 2 * S::KV + lane * copy_bytes;
                    tma_load_5d(dst, &kmap, &bar->kfull[stage], 0, row, 0, local * p.c.Hkv + g, rank);
                    tma_load_5d(dst + S::KV, &vmap, &bar->vfull[stage], 0, row, 0, local * p.c.Hkv + g, rank);
                }
                ++issued;
                if (++stage == S::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            fresh = y.tile == 0;
            pair += fresh ? 1 : 0;
            w = y;
            n = n2;
            ids = ids2;
        }
        // after a timeout: leave only when the copies in flight have landed
        if (dead && lane == 0) {
            for (int f = max(0, queries - 2); f < queries; ++f)
                (void)mbar_wait(&bar->qfull[f & 1], (uint32_t)(f >> 1) & 1u, p.timeout_ns);
            for (int64_t f = max((int64_t)0, issued - S::STAGES); f < issued; ++f) {
                (void)mbar_wait(&bar->kfull[f % S::STAGES], (uint32_t)(f / S::STAGES) & 1u, p.timeout_ns);
                (void)mbar_wait(&bar->vfull[f % S::STAGES], (uint32_t)(f / S::STAGES) & 1u, p.timeout_ns);
            }
        }
    } else {
        // ---- consumers ----
        const int gid = lane >> 2, tig = lane & 3;
        const uint32_t ring = smem_u32(smem);
        const uint32_t blk = (uint32_t)p.box * S::RB;
        // this warp's rows of a tile: which copy, and where in it
        const int first = warp * S::NG * 16;
        const int box_log2 = 31 - __clz(p.box);
        auto group_at = [&](int token) -> uint32_t { // where a group's rows begin, in a tile's keys or values
            return (uint32_t)((token >> box_log2 << box_log2) * (D * S::ESZ) + (token & (p.box - 1)) * S::RB);
        };
        uint32_t group_off[S::NG];
#pragma unroll
        for (int i = 0; i < S::NG; ++i)
            group_off[i] = group_at(first + i * 16);
        int stage = 0, pair = 0;
        uint32_t phase = 0;
        bool dead = false; // a wait ran out: wait no more, run on to the end (the call has reported it)
        auto wait = [&](uint64_t *b, uint32_t ph, uint32_t what) {
            if (!dead && !mbar_wait(b, ph, p.timeout_ns)) {
                if (lane == 0)
                    report_fault(p.status, TDG_ERR_TIMEOUT, TDG_WHERE_PIPE, what, p.epoch);
                dead = true;
            }
            __syncwarp(); // what follows (ldmatrix, mma, named barriers) wants the whole warp
        };
        int4 desc = make_int4(-1, 0, 0, pd_tag(p, 0));
        while (u < u1) {
            const int64_t len = p.lens[w.b];
            const int g = w.hg / p.groups, mg = w.hg % p.groups;
            const int rows = min(pd::ROWS, p.G - mg * pd::ROWS);
            const int64_t pair_u0 = u - w.tile; // the pair's first unit
            const int end = (int)min((int64_t)w.tiles, w.tile + (u1 - u));
            // the queries as the A operand
            const int qb = pair & 1;
            wait(&bar->qfull[qb], (pair >> 1) & 1, 2);
            uint32_t qa[D / 16][4];
            float mul[2] = {p.scale_log2, p.scale_log2};
            const uint8_t *qs = smem + S::OFF_Q + qb * S::Q_BYTES;
            if constexpr (!E4M3) {
    #pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    pd_ldsm4(smem_u32(qs) + ((lane & 7) + ((lane >> 3) & 1) * 8) * D * 2 + ks * 32 + (lane >> 4) * 16, qa[ks]);
            } else {
                // f16, in the order in which the 8-bit keys arrive: four neighbours per lane
                float x[2][D / 16][4], top[2] = {0.f, 0.f};
    #pragma unroll
                for (int r = 0; r < 2; ++r)
    #pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint2 y = *reinterpret_cast<const uint2 *>(qs + (gid + r * 8) * D * 2 + ks * 32 + tig * 8);
                        x[r][ks][0] = __uint_as_float(y.x << 16);
                        x[r][ks][1] = __uint_as_float(y.x & 0xFFFF0000u);
                        x[r][ks][2] = __uint_as_float(y.y << 16);
                        x[r][ks][3] = __uint_as_float(y.y & 0xFFFF0000u);
    #pragma unroll
                        for (int i = 0; i < 4; ++i)
                            top[r] = fmaxf(top[r], fabsf(x[r][ks][i]));
                    }
                int e[2];
    #pragma unroll
                for (int r = 0; r < 2; ++r) {
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
                    e[r] = pd_exponent(top[r]);
                }
    #pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
    #pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float f = pow2i(-e[r]);
                        qa[ks][r] = pack_f16x2(x[r][ks][0] * f, x[r][ks][1] * f);
                        qa[ks][2 + r] = pack_f16x2(x[r][ks][2] * f, x[r][ks][3] * f);
                    }
                const float ks = p.c.k_scale[g];
                mul[0] *= ks * pow2i(e[0]);
                mul[1] *= ks * pow2i(e[1]);
            }
            ++pair;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[D / 8][4];
    #pragma unroll
            for (int n = 0; n < D / 8; ++n)
                o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
            for (int t = w.tile; t < end; ++t) {
                const int64_t left = len - (int64_t)t * S::TILE - first;
                uint32_t at[S::NG];
    #pragma unroll
                for (int i = 0; i < S::NG; ++i)
                    at[i] = ring + stage * 2 * S::KV + group_off[i];
                wait(&bar->kfull[stage], phase, 3);
                auto wait_v = [&] { wait(&bar->vfull[stage], phase, 4); };
                if (left >= S::NG * 16)
                    pd_group<D, E4M3, false>(qa, mul, at, blk, S::NG * 16, lane, m, l, o, wait_v);
                else if (left > 0)
                    pd_group<D, E4M3, true>(qa, mul, at, blk, (int)left, lane, m, l, o, wait_v);
                else
                    wait_v();
                if (t + 1 == end)
                    break; // the last tile's slot is kept for the join
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bar->empty[stage]);
                if (++stage == S::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            // The queries' buffer is free.  Lane 0's arrival orders only what the
            // warp barrier has put before it: without one, the other lanes' reads of
            // the queries may still be under way when the next pair's land.
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bar->qempty[qb]);
            // Join the four warps.  Each leaves its output where its own keys and
            // values of the last tile were, which nobody else reads; the slot is
            // released when all that has been read.
            float *mls = reinterpret_cast<float *>(smem + S::OFF_ML) + (pair & 1) * S::ML_FLOATS; // [WARPS][ROWS][2]
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
                if (tig == 0) {
                    mls[(warp * pd::ROWS + gid + r * 8) * 2] = m[r];
                    mls[(warp * pd::ROWS + gid + r * 8) * 2 + 1] = l[r];
                }
            }
            uint8_t *slot_at = smem + stage * 2 * S::KV;
            auto piece = [&](uint32_t group, int i) -> float * { // piece i: values or keys, group, block
                return reinterpret_cast<float *>(slot_at + i / (S::NG * S::NB) * S::KV + i % S::NB * blk + group);
            };
            constexpr int SWIZZLE = S::COLS / 4 - 1; // columns xored by the row: no bank conflicts either way
#pragma unroll
            for (int i = 0; i < S::PIECES; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float *dst = piece(group_off[i / S::NB % S::NG], i) + (gid + r * 8) * S::COLS;
                    const int c8 = i * S::COLS / 8;
                    if constexpr (!E4M3) {
#pragma unroll
                        for (int n = 0; n < S::COLS / 8; ++n)
                            *reinterpret_cast<float2 *>(dst + ((n * 8 + tig * 2) ^ ((gid & SWIZZLE) * 4))) =
                                make_float2(o[c8 + n][2 * r], o[c8 + n][2 * r + 1]);
                    } else {
#pragma unroll
                        for (int n = 0; n < S::COLS / 8; n += 2)
                            *reinterpret_cast<float4 *>(dst + ((n * 8 + tig * 4) ^ ((gid & SWIZZLE) * 4))) = make_float4(
                                o[c8 + n][2 * r], o[c8 + n + 1][2 * r], o[c8 + n][2 * r + 1], o[c8 + n + 1][2 * r + 1]);
                    }
                }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            const bool whole = pair_u0 >= u0 && end == w.tiles;
            const int slot = w.tile == 0 && pair_u0 > u0 ? 1 : 0; // 0: the pair that holds this CTA's first unit
            // 16 rows of COLS / 4 chunks a piece; the threads take AT_ONCE pieces at a time
            constexpr int CHUNKS = S::COLS / 4, AT_ONCE = 128 / (pd::ROWS * CHUNKS);
            const int row = threadIdx.x / CHUNKS % pd::ROWS, col4 = threadIdx.x % CHUNKS * 4, p0 = threadIdx.x / (pd::ROWS * CHUNKS);
            const int h = g * p.G + mg * pd::ROWS + row;
            float M = -INFINITY, L = 0.f, wt[pd::WARPS];
#pragma unroll
            for (int i = 0; i < pd::WARPS; ++i)
                M = fmaxf(M, mls[(i * pd::ROWS + row) * 2]);
            const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int i = 0; i < pd::WARPS; ++i) {
                wt[i] = exp2_approx(mls[(i * pd::ROWS + row) * 2] - Ms);
                L += mls[(i * pd::ROWS + row) * 2 + 1] * wt[i];
            }
            const float f = whole ? (E4M3 ? p.c.v_scale[g] : 1.f) / L : 1.f;
            // (rolled for bf16, whose code is short enough to fetch: 17 against 19.5 us
            // for 64 sequences of 1..512; unrolled for 8 bits: 145 against 148.5 us for
            // 128 of 2048..4096)
            constexpr int STEPS = E4M3 ? S::PIECES / AT_ONCE : 1;
            if (row < rows) {
#pragma unroll STEPS
                for (int q = 0; q < S::PIECES / AT_ONCE; ++q) {
                    const int pc = q * AT_ONCE + p0, c = pc * S::COLS + col4;
                    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < pd::WARPS; ++i) {
                        const float4 x = *reinterpret_cast<const float4 *>(
                            piece(group_at((i * S::NG + pc / S::NB % S::NG) * 16), pc) + row * S::COLS + (col4 ^ ((row & SWIZZLE) * 4)));
                        a.x += x.x * wt[i];
                        a.y += x.y * wt[i];
                        a.z += x.z * wt[i];
                        a.w += x.w * wt[i];
                    }
                    if (whole)
                        *reinterpret_cast<uint2 *>(p.out + w.b * p.os + (int64_t)h * D + c) =
                            make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
                    else if constexpr (PAIRS) // over the queries, which all warps have read
                        *reinterpret_cast<float4 *>(smem + S::OFF_Q + (row * D + c) * 4) = a;
                    else
                        __stcg(reinterpret_cast<float4 *>(p.part_o + ((size_t)(blockIdx.x * 2 + slot) * pd::ROWS + row) * D + c), a);
                }
                if (col4 == 0 && p0 == 0) {
                    if (PAIRS && !whole) // (the other pair's place: there is none)
                        *reinterpret_cast<float2 *>(smem + S::OFF_ML + (((pair & 1) ^ 1) * S::ML_FLOATS + row * 2) * 4) = make_float2(M, L);
                    else if (!whole)
                        __stcg(reinterpret_cast<float2 *>(p.part_ml + ((size_t)(blockIdx.x * 2 + slot) * pd::ROWS + row) * 2),
                               make_float2(M, L));
                    else if (p.lse)
                        p.lse[w.b * p.Hq + h] = (M + log2f(L)) * 0.6931471805599453f;
                }
            }
            fence_proxy_async_smem(); // the slot's next tile comes by TMA
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bar->empty[stage]);
            if (++stage == S::STAGES) {
                stage = 0;
                phase ^= 1u;
            }
            if (!PAIRS && pair_u0 < u0 && end == w.tiles) { // a pair from earlier CTAs ends here
                const int c0 = pd_owner(pair_u0, base, rem);
                const int64_t c0_u0 = c0 * base + min((int64_t)c0, rem);
                desc = make_int4((int)w.b, w.hg, c0, pd_tag(p, pair_u0 > c0_u0 ? 1 : 0));
            }
            u += end - w.tile;
            w.tile = end;
            if (end == w.tiles && u < u1) {
                next_pair(w);
                u += pd::PAIR_UNITS;
            }
        }
        if (!PAIRS && threadIdx.x == 0)
            p.desc[blockIdx.x] = desc;
    }
    if constexpr (PAIRS)
        pd_join_pair<D, E4M3>(p, smem, w);
}

// Joins the partial results of the pair that ends in CTA blockIdx.x (if one
// does): rows blockIdx.y * JOIN_ROWS on.  A pair may be split over every CTA,
// so groups of D/4 threads (four columns each) share the partial results of a
// row, each group four at a time, maxima, sums and outputs in one round of
// loads; the first group of a row then joins the groups.  The order is fixed by
// the split alone.
template <int D> __global__ void __launch_bounds__(pd::JOIN_THREADS) paged_join_kernel(const __grid_constant__ PagedDecodeParams p)
{
    constexpr int LANES = D / 4, GROUPS = pd::JOIN_THREADS / LANES, U = 4;
    __shared__ float2 gml[GROUPS];
    __shared__ float4 go[GROUPS][LANES];
    griddep_launch_dependents();
    griddep_wait();
    const int4 desc = p.desc[blockIdx.x];
    const int place = desc.w & 1;
    if (desc.w - place != pd_tag(p, 0)) {
        if (threadIdx.x == 0)
            report_fault(p.status, TDG_ERR_DEVICE, TDG_WHERE_PART, blockIdx.x, p.epoch);
        return;
    }
    if (desc.x < 0)
        return;
    const int g = desc.y / p.groups, mg = desc.y % p.groups;
    const int all = min(pd::ROWS, p.G - mg * pd::ROWS);
    const int c0 = desc.z, c1 = blockIdx.x;
    if (c1 - c0 < U) { // few partial results: one CTA takes all rows, a group of threads a row
        for (int row = threadIdx.x / LANES; blockIdx.y == 0 && row < all; row += GROUPS) {
            const int col = threadIdx.x % LANES * 4;
            float2 ml[U];
            float4 x[U];
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                ml[i] = make_float2(-INFINITY, 0.f);
                x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c0 + i <= c1) {
                    const size_t at = (size_t)((c0 + i) * 2 + (i == 0 ? place : 0)) * pd::ROWS + row;
                    ml[i] = __ldcg(reinterpret_cast<const float2 *>(p.part_ml + at * 2));
                    x[i] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + at * D + col));
                }
                M = fmaxf(M, ml[i].x);
            }
            const float Ms = M == -INFINITY ? 0.f : M;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const float w = exp2_approx(ml[i].x - Ms);
                L += ml[i].y * w;
                a.x += x[i].x * w;
                a.y += x[i].y * w;
                a.z += x[i].z * w;
                a.w += x[i].w * w;
            }
            const int h = g * p.G + mg * pd::ROWS + row;
            const float f = (p.c.v_scale ? p.c.v_scale[g] : 1.f) / L;
            *reinterpret_cast<uint2 *>(p.out + desc.x * p.os + (int64_t)h * D + col) =
                make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
            if (p.lse && col == 0)
                p.lse[(int64_t)desc.x * p.Hq + h] = (M + log2f(L)) * 0.6931471805599453f;
        }
        return;
    }
    const int rows = min(pd::JOIN_ROWS, all - (int)blockIdx.y * pd::JOIN_ROWS);
    if (rows <= 0)
        return;
    const int per = GROUPS / (rows == 1 ? 1 : 2); // groups of a row
    const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    const int row = blockIdx.y * pd::JOIN_ROWS + group / per, part = group % per;
    const bool used = group / per < rows;
    // slot of CTA c: the first one's may be its second
    auto at = [&](int c) -> size_t { return (size_t)(c * 2 + (c == c0 ? place : 0)) * pd::ROWS + row; };
    float M = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float2 &ml, const float4 &x, float ms) {
        const float w = exp2_approx(ml.x - ms);
        L += ml.y * w;
        a.x += x.x * w;
        a.y += x.y * w;
        a.z += x.z * w;
        a.w += x.w * w;
    };
    auto raise = [&](float top) -> float { // brings M, L and a to a new maximum
        const float ms = top == -INFINITY ? 0.f : top, al = exp2_approx(M - ms);
        M = top;
        L *= al;
        a.x *= al;
        a.y *= al;
        a.z *= al;
        a.w *= al;
        return ms;
    };
    for (int c = c0 + part; used && c <= c1; c += per * U) {
        float2 ml[U];
        float4 x[U];
        float top = M;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            ml[i] = make_float2(-INFINITY, 0.f);
            x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c + i * per <= c1) {
                ml[i] = __ldcg(reinterpret_cast<const float2 *>(p.part_ml + at(c + i * per) * 2));
                x[i] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + at(c + i * per) * D + lane * 4));
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
            top = fmaxf(top, ml[i].x);
        const float ms = raise(top);
#pragma unroll
        for (int i = 0; i < U; ++i)
            add(ml[i], x[i], ms);
    }
    if (lane == 0)
        gml[group] = make_float2(M, L);
    go[group][lane] = a;
    __syncthreads();
    if (!used || part != 0)
        return;
    float top = M;
    for (int i = 1; i < per; ++i)
        top = fmaxf(top, gml[group + i].x);
    const float ms = raise(top);
    for (int i = 1; i < per; ++i)
        add(gml[group + i], go[group + i][lane], ms);
    const int h = g * p.G + mg * pd::ROWS + row;
    const float f = (p.c.v_scale ? p.c.v_scale[g] : 1.f) / L;
    *reinterpret_cast<uint2 *>(p.out + desc.x * p.os + (int64_t)h * D + lane * 4) =
        make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
    if (p.lse && lane == 0)
        p.lse[(int64_t)desc.x * p.Hq + h] = (M + log2f(L)) * 0.6931471805599453f;
}

} // namespace tdg

using namespace tdg;
using namespace tdg_host;

namespace {

// The pool as a 5-D tensor: {bytes of a 128-byte block, slot in the page, block
// of the row, page and head, rank}; one box is `box` slots of every block.
template <int D, bool E4M3> bool pool_map(CUtensorMap *m, const tdg_symm *h, const tdg_paged_cache &c, size_t off, int box)
{
    using S = pd::Shape<D, E4M3>;
    const uint64_t row = (uint64_t)D * S::ESZ;
    const uint64_t dims[5] = {S::RB / S::ESZ, (uint64_t)c.page_size, S::NB, (uint64_t)c.pages * c.Hkv, (uint64_t)h->world};
    const uint64_t str[4] = {row, S::RB, row * c.page_size, h->region_bytes};
    const uint32_t bx[5] = {S::RB / S::ESZ, (uint32_t)box, S::NB, 1, 1};
    return encode_tiled(m, E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, h->base + off, dims,
                        str, bx, S::RB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

template <int D, bool E4M3> int launch_decode(const tdg_symm *h, const tdg_paged_decode_args *a, PagedDecodeParams &p, cudaStream_t st)
{
    using S = pd::Shape<D, E4M3>;
    p.box = a->cache.page_size < S::TILE ? a->cache.page_size : S::TILE;
    CUtensorMap km, vm;
    if (!pool_map<D, E4M3>(&km, h, a->cache, a->cache.k_off, p.box) || !pool_map<D, E4M3>(&vm, h, a->cache, a->cache.v_off, p.box))
        return TDG_ERR_CUDA;
    // Few short sequences: a cluster of up to 8 CTAs for each pair, and no second
    // launch, when its longest share is at most CAP tiles and at most SAVED (what
    // the launch costs, in tiles) longer than an equal run of the line.
    // By the line and so: one of 1000, 64 / 8 heads, 8.6 -> 7.3 us, 30 of 100
    // 9.1 -> 6.1, 8-bit 32 of 200 11.3 -> 8.0; but one of 4000 on one key head 8.9 ->
    // 9.9, 8-bit one of 4000 10.4 -> 11.4.
    const int64_t pairs = a->B * a->cache.Hkv * p.groups, most = (a->table_entries * a->cache.page_size + S::TILE - 1) / S::TILE;
    constexpr int64_t CAP = E4M3 ? 4 : 8, SAVED_HALVES = E4M3 ? 5 : 11;
    const int64_t ctas = h->sm_count * 2 < pd::MAX_CTAS ? h->sm_count * 2 : pd::MAX_CTAS;
    p.split = pairs > ctas ? 0 : pd::MAX_SPLIT;
    while (p.split > 1 && (pairs * p.split > ctas || p.split / 2 >= most))
        p.split /= 2;
    if (most > CAP * p.split || 2 * most * ctas > p.split * (SAVED_HALVES * ctas + 2 * pairs * most))
        p.split = 0;
    const void *fn = p.split ? reinterpret_cast<const void *>(&paged_decode_kernel<D, E4M3, true>)
                             : reinterpret_cast<const void *>(&paged_decode_kernel<D, E4M3, false>);
    if (const cudaError_t e = set_smem(fn, S::SMEM); e != cudaSuccess)
        return cuda_err(e, "paged decode smem");
    if (p.split) {
        void *args[] = {&p, &km, &vm};
        return cuda_err(launch(fn, dim3((unsigned)(pairs * p.split)), dim3(pd::THREADS), S::SMEM, st, args, false, p.split, true),
                        "paged decode launch");
    }
    void *args[] = {&p, &km, &vm};
    if (const cudaError_t e = launch(fn, dim3((unsigned)ctas), dim3(pd::THREADS), S::SMEM, st, args, false, 1, true); e != cudaSuccess)
        return cuda_err(e, "paged decode launch");
    void *jargs[] = {&p};
    const int join_rows = p.G < pd::ROWS ? p.G : pd::ROWS;
    return cuda_err(launch(reinterpret_cast<const void *>(&paged_join_kernel<D>),
                           dim3((unsigned)ctas, (unsigned)((join_rows + pd::JOIN_ROWS - 1) / pd::JOIN_ROWS)), dim3(pd::JOIN_THREADS), 0, st,
                           jargs, false, 1, true),
                    "paged join launch");
}

} // namespace

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
    // nothing that is written lies over anything else
    uint8_t *part_at = h->base + (uint64_t)a->root * h->region_bytes + a->part_off;
    const Range q{a->q, rows_extent(a->B, a->q_stride, Hq * D)}, out{a->out, rows_extent(a->B, a->out_stride, Hq * D)};
    const Range lse{a->lse, (uint64_t)a->B * Hq * 4}, partials{part_at, part};
    const Range k_scale{a->cache.k_scale, scale_bytes(a->cache)}, v_scale{a->cache.v_scale, scale_bytes(a->cache)};
    const Range lens{a->lens, (uint64_t)a->B * 4}, table = table_range(a->table, a->B, a->table_entries, a->table_stride);
    if (ranges_overlap({out, lse, partials}, {k_scale, v_scale, lens, table}) || ranges_overlap({lse, partials}, {q, out}) ||
        ranges_overlap({lse}, {partials}) || pools_overlap(h, a->cache, {out, lse}))
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
    p.groups = (p.G + pd::ROWS - 1) / pd::ROWS;
    p.scale_log2 = (a->scale > 0.f ? a->scale : 1.0f / sqrtf((float)D)) * 1.4426950408889634f; // scores live in base 2
    p.timeout_ns = timeout_or_default(0);
    p.q = static_cast<const __nv_bfloat16 *>(a->q);
    p.out = static_cast<__nv_bfloat16 *>(a->out);
    p.lse = a->lse;
    p.table = a->table;
    p.lens = a->lens;
    p.desc = reinterpret_cast<int4 *>(part_at);
    p.part_ml = reinterpret_cast<float *>(p.desc + pd::MAX_CTAS);
    p.part_o = p.part_ml + (size_t)pd::MAX_CTAS * 2 * pd::ROWS * 2;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool e4m3 = a->cache.kv_type == TDG_KV_E4M3;
    if (D == 128)
        return e4m3 ? launch_decode<128, true>(h, a, p, st) : launch_decode<128, false>(h, a, p, st);
    return e4m3 ? launch_decode<64, true>(h, a, p, st) : launch_decode<64, false>(h, a, p, st);
}
