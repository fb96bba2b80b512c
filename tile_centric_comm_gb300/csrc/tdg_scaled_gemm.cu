// tdg_scaled_gemm.cu -- products of e4m3 matrices with a float32 scale for each
// block of 128 along the contraction, of one matrix of weights or of many
// experts' (rows sorted by expert, offsets on the device).
//
//   out[m][n] = sum_j sa[m][j] sw[n/128][j] (sum_{k in block j} a[m][k] w[n][k])
//
// A block's product of codes is one accumulator in TMEM.  The epilogue warps
// take it from there and add it, times its two scales, to sums in registers
// while the next block is multiplied; at the end of the tile the sums are
// rounded and stored.  Two kernels, by the number of rows:
//
//   wide    256 rows of a x 256 weight rows by a pair of CTAs.  Rows of a are
//           TMEM's lanes, so a thread of the epilogue needs one scale a block.
//           Bound by the accumulator's way (products, epilogue, release; TMEM holds two
//           of 256 columns): 0.42 us a block against 0.27 of tensor work, 1.9 us a
//           tile for start and store.  8192 rows by 7168 x 8192: 369 us
//           among other calls, 2610 TFLOP/s, and 332 repeated back to back, 2900.
//           For few tiles two pairs, a cluster of four, halve K and exchange halves
//           of their sums (192 rows by 7168 x 8192: 32 us by one pair a tile, 21 by two).
//   narrow  128 weight rows x up to 64 or 128 rows of a.  The weights are the lanes
//           and the rows of a the columns, which an instruction takes in steps of 16:
//           an expert with few rows costs what it has, and streaming the weights
//           is what bounds the call.  With few tiles the blocks of K are divided
//           over the CTAs of a cluster, whose sums are added in rank order.  64 experts
//           of 4096 x 7168 with 16 rows each: 280 us, 6.7 TB/s, with 128 rows 329; one
//           row by 3200 x 5120 7.3 us, which is latency.
//
// Warps of a CTA (either kernel):
//   warp 0      TMA loader: the codes of a block into a ring of shared memory
//   warp 1      MMA issuer: four tcgen05.mma.kind::f8f6f4 (K = 32) a block
//   warps 2, 3  scales: sa * sw of the tile's rows, some blocks at a time
//   warps 4..   epilogue
#include <atomic>
#include <cmath>
#include <type_traits>

#include "tdg_scaled.cuh"

namespace tdg {

namespace sg {
constexpr int BK = 128;                 // codes of a block: one scale, one swizzled row
constexpr int ROWS = 128;               // lanes of TMEM: rows of a CTA's first operand
constexpr int A_BYTES = ROWS * BK;
constexpr int NGROUP = 8;               // weight tiles that are visited together
constexpr int MAX_E = 4096;
constexpr int BAR_BYTES = 512;
} // namespace sg

struct WideShape {
    static constexpr int BOX = sg::ROWS;             // rows of a TMA box
    static constexpr bool PAIR = true;
    static constexpr int BT = 256;                   // rows of a in a tile, over the pair
    static constexpr int WTILE = 256;                // weight rows of a tile
    static constexpr int BPS = 1;                    // blocks of a ring stage
    static constexpr int BLOCK_BYTES = 2 * sg::A_BYTES, STAGES = 4, STAGE_BYTES = BLOCK_BYTES;
    static constexpr int TBUF = 2, TCOLS = 256;      // accumulators in TMEM
    static constexpr int EPIW = 8, THREADS = 128 + 32 * EPIW;
    static constexpr int REGS_OTHER = 72, REGS_EPI = 216; // registers of a thread
    static_assert(128 * REGS_OTHER + 32 * EPIW * REGS_EPI <= THREADS * (65536 / THREADS / 8 * 8), "registers of the launch");
    static constexpr int SK = 4, SCH = 3;            // blocks whose scales are loaded together, such chunks in the ring
    static constexpr int SROW = 2 * sg::ROWS + 8;    // floats of a block's scales: for each half of the columns, and a pad
    static constexpr int STG = 32 * 128;             // staged rows of an epilogue warp: 128 bytes of each, twice
    static constexpr int OFF_STG = STAGES * STAGE_BYTES; // (swizzled by address: 1024-byte aligned)
    static constexpr int OFF_SCALE = OFF_STG + 2 * EPIW * STG;
    static constexpr int OFF_BAR = OFF_SCALE + SCH * SK * SROW * 4;
    static constexpr int OFF_PRE = OFF_BAR + sg::BAR_BYTES; // tiles before each expert
    static constexpr int SMEM = OFF_PRE + 1024;      // + 4 (E + 1); + alignment slack
};

template <int ROWS> struct NarrowShape {
    static constexpr bool PAIR = false;
    static constexpr int BT = ROWS;                  // rows of a in a tile, at most
    static constexpr int WTILE = sg::ROWS;
    static constexpr int STEP = 16, BOX = 64;        // of an instruction's columns; rows of a TMA box, for up to STEP rows and for more
    static constexpr int BPS = 2;                    // two blocks a wait, which costs every role 100 cycles
    static constexpr int BLOCK_BYTES = sg::A_BYTES + BT * sg::BK, STAGES = BT == 64 ? 4 : 3, STAGE_BYTES = BPS * BLOCK_BYTES;
    static constexpr int TCOLS = BT, TBUF = 512 / (BPS * TCOLS);
    static constexpr int GROUPS = BT / 64, EPIW = 4 * GROUPS, THREADS = 128 + 32 * EPIW; // groups of epilogue warps: 64 sums a thread
    static constexpr bool REGS = GROUPS > 1;         // registers are moved to the epilogue
    static constexpr int REGS_OTHER = 72, REGS_EPI = 216;
    static constexpr int SK = 4, SCH = 3;
    static constexpr int SROW = BT + 8;
    static constexpr int STG_ROW = 80;               // bytes of a staged row: 32 bf16 and a pad
    static constexpr int STG = 8 * STG_ROW;          // of an epilogue warp
    static constexpr int RED = 132;                  // floats of a row of partial sums: 128 and a pad
    static constexpr int OFF_SCALE = STAGES * STAGE_BYTES;
    static constexpr int OFF_STG = OFF_SCALE + SCH * SK * SROW * 4;
    static constexpr int OFF_BAR = OFF_STG + EPIW * STG;
    static constexpr int OFF_PRE = OFF_BAR + sg::BAR_BYTES;
    static constexpr int SMEM = OFF_PRE + 1024;
    static_assert(BT * RED * 4 <= OFF_SCALE, "partial sums fit the ring");
};
static_assert(WideShape::SMEM + 4 * (sg::MAX_E + 1) <= 232448 && NarrowShape<64>::SMEM + 4 * (sg::MAX_E + 1) <= 232448 &&
                  NarrowShape<128>::SMEM + 4 * (sg::MAX_E + 1) <= 232448, "shared memory");

struct ScaledParams {
    DevStatus *status;
    uint32_t epoch;
    uint64_t timeout_ns;
    int64_t M, a_scale_stride, out_stride;
    int N, E, k_blocks, n_tiles, n_blocks, out_f32;
    int split;                   // CTAs (wide: pairs) of a cluster that share K (1: none)
    uint32_t item0, item1;       // the tiles of this launch, [item0, item1): at most those that offsets in order give
    const float *a_scale, *b_scale;
    void *out;
    const int64_t *base;
};

// tile: wide, the tiles whose scales the ring holds.  The scale warps are at most
// SCH chunks ahead of the epilogue, so a tile's entry is written again only when
// the epilogue has stored that tile.
struct ScaledSmem {
    uint64_t full[8], empty[8], tfull[8], tempty[8];
    uint64_t sfull[4], sempty[4], drain;
    uint32_t tmem_base;
    volatile int abort;
    uint32_t issued, consumed; // ring fills issued by the loader, consumed by the issuer
    uint32_t scan[16];
    struct {
        int64_t row, end; // of this CTA's first row, and of the tile
        int n0;
    } tile[4];
};
static_assert(sizeof(ScaledSmem) <= sg::BAR_BYTES, "barrier block");

// e4m3 A and B (K-major), float32 D
__device__ __forceinline__ constexpr uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

template <bool PAIR> __device__ __forceinline__ void umma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if (PAIR)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                     : "memory");
}

// 16 lanes x 32 columns: r[4i], r[4i+1] are columns 8i + 2(t%4) and the next of
// lane t/4, r[4i+2], r[4i+3] those of lane t/4 + 8
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
                   "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}

// acc += (lo, hi) * scale.  volatile: it stays behind the wait for its values.
__device__ __forceinline__ void fma_pair(uint64_t &acc, uint32_t lo, uint32_t hi, uint64_t scale)
{
    asm volatile("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}" : "+l"(acc) : "r"(lo), "r"(hi), "l"(scale));
}

// acc += v * scale, one at a time: a packed multiply-add takes two cycles for two
// and wants its values in pairs of registers (8192 x 7168 x 8192 took 448 us by
// packed ones when it took 420 like this)
__device__ __forceinline__ void fma_one(float &acc, uint32_t v, float scale)
{
    asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(acc) : "f"(__uint_as_float(v)), "f"(scale));
}

__device__ __forceinline__ float2 halves(uint64_t v)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}

__device__ __forceinline__ uint32_t narrowed(uint64_t v)
{
    const float2 f = halves(v);
    return pack_bf16x2(f.x, f.y);
}

__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// A wait whose thread is suspended until the phase completes, for up to 10 us at
// a time: 12 warps that poll without a time hint take issue slots and barrier
// accesses from the ones at work (481 us instead of 437 at 8192 x 7168 x 8192).
// One piece of PTX, since the epilogue waits once a block and a phase that is
// complete must cost it one instruction and one branch.  Sets `failed` when the
// time is up (the clock is read only between the suspensions); a thread that has
// failed before waits no more than two suspensions.
__device__ __forceinline__ void mbar_wait_suspended(uint32_t bar, uint32_t parity, uint64_t timeout_ns, uint32_t &failed)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .u64 t, end;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %4;\n\t"
                 "@p bra DONE_%=;\n\t"
                 "mov.u64 end, %%globaltimer;\n\t"
                 "setp.eq.u32 p, %0, 0;\n\t"
                 "@p add.u64 end, end, %3;\n\t"
                 "AGAIN_%=:\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %4;\n\t"
                 "@p bra DONE_%=;\n\t"
                 "mov.u64 t, %%globaltimer;\n\t"
                 "setp.lt.u64 p, t, end;\n\t"
                 "@p bra AGAIN_%=;\n\t"
                 "mov.u32 %0, 1;\n\t"
                 "DONE_%=:\n\t}"
                 : "+r"(failed)
                 : "r"(bar), "r"(parity), "l"(timeout_ns), "r"(10000u)
                 : "memory");
}
__device__ __forceinline__ bool mbar_wait_suspended(uint64_t *bar, uint32_t parity, uint64_t timeout_ns)
{
    uint32_t failed = 0;
    mbar_wait_suspended(smem_u32(bar), parity, timeout_ns, failed);
    return !failed;
}

// Arrivals that tell of loads which are in registers (tcgen05.wait::ld, or
// values already used), so that no memory is released: with .release an arrival
// waits for all of the thread's memory operations (1300 cycles a block on the
// pair leader's barrier, twice the block's tensor work; 350 on an own one that
// follows an arrival there).  By the lanes with `by`, without a branch.
__device__ __forceinline__ void mbar_arrive_remote_relaxed(uint32_t cluster_addr, bool by)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                 "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(cluster_addr), "r"(by ? 1u : 0u)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive_relaxed(uint64_t *bar, bool by)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                 "@p mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(by ? 1u : 0u)
                 : "memory");
}

struct ScaledTile {
    int e;             // expert
    int n0;            // first weight row
    int width;         // narrow: columns of the instruction
    int64_t tok0, end; // rows of a: [tok0, end)
};

// The item's tile.  pre: the tiles before each expert.  The tiles of an expert
// are visited in groups of NGROUP weight tiles, so that those in flight
// together share both operands in L2.  Narrow: an expert's rows are divided
// evenly over as few tiles as hold them.
template <class S> __device__ __forceinline__ ScaledTile scaled_tile(const ScaledParams &p, const uint32_t *pre, uint32_t item)
{
    ScaledTile t;
    int lo = 0, hi = p.E; // pre[lo] <= item < pre[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= item)
            lo = mid;
        else
            hi = mid;
    }
    t.e = lo;
    const int64_t first = p.base ? p.base[lo] : 0, rows = (p.base ? p.base[lo + 1] : p.M) - first;
    const uint32_t tiles = (uint32_t)((rows + S::BT - 1) / S::BT);
    if constexpr (S::PAIR)
        t.width = S::BT;
    else
        t.width = (int)(((uint32_t)((rows + tiles - 1) / tiles) + S::STEP - 1) / S::STEP * S::STEP);
    const uint32_t local = item - pre[lo], per = sg::NGROUP * tiles, g = local / per, r = local - g * per;
    const uint32_t in_group = min((uint32_t)sg::NGROUP, (uint32_t)p.n_tiles - g * sg::NGROUP);
    const uint32_t row = r / in_group;
    t.n0 = (int)(g * sg::NGROUP + (r - row * in_group)) * S::WTILE;
    t.tok0 = first + (int64_t)row * t.width;
    t.end = min(first + rows, t.tok0 + t.width);
    return t;
}

// Barriers and TMEM, then (behind the launch before) the tiles before each
// expert: a segment of experts a thread, then a scan.  Sums are cut at 2^31 - 1:
// offsets that are in order never reach that.
template <class S> __device__ __forceinline__ void scaled_begin(const ScaledParams &p, ScaledSmem *ps, uint32_t *pre)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(&ps->full[i], 1);
            mbar_init(&ps->empty[i], 1);
        }
        for (int i = 0; i < S::TBUF; ++i) {
            mbar_init(&ps->tfull[i], 1);
            mbar_init(&ps->tempty[i], S::EPIW * (S::PAIR ? 2 : 1));
        }
        for (int i = 0; i < S::SCH; ++i) {
            mbar_init(&ps->sfull[i], 2);
            mbar_init(&ps->sempty[i], S::EPIW);
        }
        mbar_init(&ps->drain, 1);
        ps->abort = 0;
        ps->issued = 0;
        ps->consumed = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        if (S::PAIR) {
            tmem_alloc_pair(&ps->tmem_base, 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&ps->tmem_base, 512);
            tmem_relinquish();
        }
        tc_fence_before();
    }
    griddep_launch_dependents();
    griddep_wait();
    if (!p.base) {
        if (threadIdx.x == 0) {
            pre[0] = 0;
            pre[1] = (uint32_t)((p.M + S::BT - 1) / S::BT) * p.n_tiles;
        }
        __syncthreads();
        if (S::PAIR)
            cluster_sync(); // the peer's barriers are initialised before any remote use
        tc_fence_after();
        return;
    }
    const int per = (p.E + S::THREADS - 1) / S::THREADS;
    const int lo = min(p.E, (int)threadIdx.x * per), hi = min(p.E, lo + per);
    const uint64_t most = 0x7fffffffu;
    auto tiles_of = [&](int e) -> uint64_t {
        const int64_t b0 = p.base[e], b1 = p.base[e + 1];
        if (b0 < 0 || b1 < b0 || b1 > p.M) {
            if (blockIdx.x == 0)
                report_fault(p.status, TDG_ERR_DEVICE, TDG_WHERE_CU, (uint32_t)e, p.epoch);
            return 0;
        }
        return (uint64_t)((b1 - b0 + S::BT - 1) / S::BT) * p.n_tiles;
    };
    uint64_t upto = 0; // of the warp's lanes up to this one
    for (int e = lo; e < hi; ++e)
        upto = min(most, upto + tiles_of(e));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint64_t v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d)
            upto = min(most, upto + v);
    }
    if (lane == 31)
        ps->scan[warp] = (uint32_t)upto;
    __syncthreads();
    uint64_t run = 0;
    for (int w = 0; w < warp; ++w)
        run = min(most, run + ps->scan[w]);
    const uint64_t before = __shfl_up_sync(0xffffffffu, upto, 1);
    run = lane ? min(most, run + before) : run;
    for (int e = lo; e < hi; ++e) {
        pre[e] = (uint32_t)run;
        run = min(most, run + tiles_of(e));
        if (e == p.E - 1)
            pre[p.E] = (uint32_t)run;
    }
    __syncthreads();
    if (S::PAIR)
        cluster_sync();
    tc_fence_after();
}

// one lane of a converged warp
__device__ __forceinline__ bool elected()
{
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
    return is != 0;
}

// The MMA issuer's loop, of one warp (of the pair's leader).  The whole warp
// walks it and one elected lane issues, so that what the loop computes is the
// same in all lanes (walked by one lane, four MMAs and two commits took 440 cycles
// to issue, of the 512 that the tensor cores need for them).
// columns(tile): those of the instruction; pair: its CTAs in the cluster, as a mask.
template <class S, class F>
__device__ __forceinline__ void scaled_issue(const ScaledParams &p, ScaledSmem *ps, uint32_t sbase, uint32_t tmem, const uint32_t *pre, uint32_t items,
                                             uint32_t unit, uint32_t units, int kb0, int kb1, uint16_t pair, F columns)
{
    const uint64_t tmo = p.timeout_ns;
    // a ring slot's offset never carries out of the descriptor's address field
    const uint64_t ad0 = sdesc_sw128(sbase, 16, 1024);
    int stage = 0, buf = 0;
    uint32_t phase = 0, bphase = 0, consumed = 0;
    bool ok = true;
    for (uint32_t it = unit; it < items && ok; it += units) {
        const uint32_t idesc = idesc_e4m3(S::PAIR ? 2 * sg::ROWS : sg::ROWS, columns(scaled_tile<S>(p, pre, it)));
        for (int kb = kb0; kb < kb1; kb += S::BPS) {
            const uint64_t ad = ad0 + (uint64_t)(stage * (S::STAGE_BYTES >> 4));
            const uint32_t d = tmem + (uint32_t)(buf * S::BPS * S::TCOLS);
            // the accumulator last: it is what is waited for
            ok = mbar_wait_suspended(&ps->full[stage], phase, tmo) && mbar_wait_suspended(&ps->tempty[buf], bphase ^ 1u, tmo);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                break;
            tc_fence_after();
            if (elected()) {
#pragma unroll
                for (int j = 0; j < S::BPS; ++j)
                    if (j == 0 || kb + j < kb1) {
                        const uint64_t aj = ad + (uint64_t)(j * (S::BLOCK_BYTES >> 4)), bj = aj + (sg::A_BYTES >> 4);
#pragma unroll
                        for (int k = 0; k < sg::BK / 32; ++k)
                            umma_e4m3<S::PAIR>(d + j * S::TCOLS, aj + 2 * k, bj + 2 * k, idesc, k ? 1u : 0u);
                    }
                if (S::PAIR) {
                    umma_commit_pair_mask(&ps->empty[stage], pair);
                    umma_commit_pair_mask(&ps->tfull[buf], pair);
                } else {
                    umma_commit(&ps->empty[stage]);
                    umma_commit(&ps->tfull[buf]); // the last arrival of a CTA is one that is waited for
                }
            }
            __syncwarp();
            ++consumed;
            if (++stage == S::STAGES) {
                stage = 0;
                phase ^= 1u;
            }
            if (++buf == S::TBUF) {
                buf = 0;
                bphase ^= 1u;
            }
        }
    }
    if (elected()) {
        ps->consumed = consumed;
        if (!ok) {
            report_fault(p.status, TDG_ERR_TIMEOUT, TDG_WHERE_PIPE, 1, p.epoch);
            ps->abort = 1;
        }
    }
    __syncwarp();
}

// After the roles: where any wait of this CTA ran out, wait (bounded) until no
// MMA that it issued and no TMA write of its own is still in flight.  (Where none
// did, its epilogue has waited for all of them; a pair's are the leader's.)
template <class S> __device__ __forceinline__ void scaled_drain(const ScaledParams &p, ScaledSmem *ps)
{
    __syncthreads();
    const uint32_t rank = S::PAIR ? cluster_ctarank() : 0; // (read again: kept, it costs the wide epilogue a register)
    const bool leader = (rank & 1) == 0;
    // (commits tell of the executing thread's own: the lane elected here is the issuing one)
    if (ps->abort && leader && threadIdx.x >> 5 == 1 && elected()) {
        if (S::PAIR)
            umma_commit_pair_mask(&ps->drain, (uint16_t)(3u << rank));
        else
            umma_commit(&ps->drain);
        (void)mbar_wait(&ps->drain, 0, p.timeout_ns);
    }
    if (ps->abort && threadIdx.x == 0) {
        if (leader) {
            for (uint32_t f = ps->consumed; f < ps->issued; ++f)
                (void)mbar_wait(&ps->full[f % S::STAGES], (f / S::STAGES) & 1u, p.timeout_ns);
        } else { // a peer's fill is known done once the leader has freed its slot
            for (uint32_t f = ps->issued > (uint32_t)S::STAGES ? ps->issued - S::STAGES : 0u; f < ps->issued; ++f)
                (void)mbar_wait(&ps->empty[f % S::STAGES], (f / S::STAGES) & 1u, p.timeout_ns);
        }
    }
    __syncthreads();
}

__global__ void __launch_bounds__(WideShape::THREADS, 1)
    scaled_wide_kernel(const __grid_constant__ ScaledParams p, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_out)
{
    using S = WideShape;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    ScaledSmem *ps = reinterpret_cast<ScaledSmem *>(smem + S::OFF_BAR);
    uint32_t *pre = reinterpret_cast<uint32_t *>(smem + S::OFF_PRE);
    float *scales = reinterpret_cast<float *>(smem + S::OFF_SCALE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the pair's place in the cluster is its part of K, the CTA's place in the pair its half of the tile
    const int rank = (int)cluster_ctarank(), half = rank & 1, part = rank >> 1, leader = rank & ~1;
    const uint32_t unit = p.item0 + blockIdx.x / 2 / p.split, units = gridDim.x / 2 / p.split;
    const int kb0 = part * p.k_blocks / p.split, kb1 = (part + 1) * p.k_blocks / p.split;
    const uint64_t tmo = p.timeout_ns;
    scaled_begin<S>(p, ps, pre);
    const uint32_t tmem = ps->tmem_base;
    const uint32_t items = min(pre[p.E], p.split > 1 ? p.item0 + units : p.item1); // with K divided a cluster has one tile
    // an instruction's columns: the weight rows of the tile in steps of 32, each CTA holding half of them
    auto columns = [&](const ScaledTile &t) { return min(S::WTILE, (p.N - t.n0 + 31) / 32 * 32); };

    if (warp == 0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::REGS_OTHER));
        if (lane == 0) {
            const uint32_t full0 = mapa_shared(smem_u32(&ps->full[0]), leader);
            int stage = 0;
            uint32_t phase = 0, issued = 0;
            for (uint32_t it = unit; it < items && !ps->abort; it += units) {
                const ScaledTile t = scaled_tile<S>(p, pre, it);
                const int row = (int)((uint32_t)t.tok0 + half * sg::ROWS), wrow = t.n0 + half * (columns(t) / 2);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait_suspended(&ps->empty[stage], phase ^ 1u, tmo)) {
                        report_fault(p.status, TDG_ERR_TIMEOUT, TDG_WHERE_PIPE, 0, p.epoch);
                        ps->abort = 1;
                        break;
                    }
                    uint8_t *dst = smem + stage * S::STAGE_BYTES;
                    if (half == 0) // for both CTAs' bytes
                        mbar_arrive_expect_tx(&ps->full[stage], 2 * S::STAGE_BYTES);
                    tma_load_2d_pair(dst, &map_a, full0 + stage * 8, kb * sg::BK, row);
                    tma_load_3d_pair(dst + sg::A_BYTES, &map_w, full0 + stage * 8, kb * sg::BK, wrow, t.e);
                    ++issued;
                    if (++stage == S::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            ps->issued = issued;
        }
        __syncwarp();
    } else if (warp == 1) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::REGS_OTHER));
        if (half == 0)
            scaled_issue<S>(p, ps, smem_u32(smem), tmem, pre, items, unit, units, kb0, kb1, (uint16_t)(3 << leader), columns);
    } else if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::REGS_OTHER));
        // scales: each warp half of the CTA's rows, 32 / SK rows x SK blocks a step, for both column halves
        constexpr int RS = 32 / S::SK;
        const int j = lane % S::SK, r0 = lane / S::SK + (warp - 2) * 64;
        int chunk = 0;
        uint32_t phase = 0;
        bool ok = true;
        uint32_t nth = 0;
        for (uint32_t it = unit; it < items && ok; it += units, ++nth) {
            const ScaledTile t = scaled_tile<S>(p, pre, it);
            const float *sw = p.b_scale + ((int64_t)t.e * p.n_blocks + t.n0 / 128) * p.k_blocks;
            const int64_t next = t.n0 / 128 + 1 < p.n_blocks ? p.k_blocks : 0;
            const int64_t first = t.tok0 + half * sg::ROWS;
            const int rows = (int)max((int64_t)0, min((int64_t)sg::ROWS, t.end - first));
            const float *sa = p.a_scale + first * p.a_scale_stride;
            for (int kb = kb0; kb < kb1; kb += S::SK) {
                const bool in = kb + j < kb1;
                const float w0 = in ? sw[kb + j] : 0.f, w1 = in ? sw[next + kb + j] : 0.f;
                float v[64 / RS];
#pragma unroll
                for (int i = 0; i < 64 / RS; ++i)
                    v[i] = in && r0 + RS * i < rows ? sa[(int64_t)(r0 + RS * i) * p.a_scale_stride + kb + j] : 0.f;
                ok = mbar_wait_suspended(&ps->sempty[chunk], phase ^ 1u, tmo);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) {
                    if (lane == 0)
                        report_fault(p.status, TDG_ERR_TIMEOUT, TDG_WHERE_PIPE, 2, p.epoch);
                    ps->abort = 1;
                    break;
                }
                if (kb == kb0 && warp == 2 && lane == 0) {
                    ps->tile[nth & 3].row = first;
                    ps->tile[nth & 3].end = t.end;
                    ps->tile[nth & 3].n0 = t.n0;
                }
                float *dst = scales + (chunk * S::SK + j) * S::SROW + r0;
#pragma unroll
                for (int i = 0; i < 64 / RS; ++i) {
                    dst[RS * i] = v[i] * w0;
                    dst[RS * i + sg::ROWS] = v[i] * w1;
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&ps->sfull[chunk]);
                if (++chunk == S::SCH) {
                    chunk = 0;
                    phase ^= 1u;
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::REGS_EPI));
        const int q = warp & 3, cg = (warp - 4) >> 2; // lanes of TMEM, half of the columns
        const uint32_t tempty0 = mapa_shared(smem_u32(&ps->tempty[0]), leader);
        const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(cg * 128);
        const uint32_t tfull0 = smem_u32(&ps->tfull[0]), sfull0 = smem_u32(&ps->sfull[0]);
        const float *scale_at = scales + cg * sg::ROWS + q * 32 + lane;
        int chunk = 0;
        uint32_t buf = 0, bphase = 0, sphase = 0, failed = 0;
        bool ok = true;
        uint8_t *const stg0 = smem + S::OFF_STG + 2 * (warp - 4) * S::STG;
        int side = 0; // of the two staging buffers
        uint32_t nth = 0;
        for (uint32_t it = unit; it < items && ok; it += units, ++nth) {
            float acc[8][16];
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[c][i] = 0.f;
            // Half of the warp's columns at a time, as many as the registers take: what the
            // tensor cores wait for is the accumulator's release, so its loads come first
            // and what can wait stands behind the release (chunks of 16 columns, each on
            // its way while the one before is added, released it 160 cycles later: 374 us
            // for 8192 x 7168 x 8192 when this took 348).
            uint32_t r[2][32];
            auto load = [&](int col) {
                tmem_ld_32x32b_x32(at + buf * S::TCOLS + col, r[0]);
                tmem_ld_32x32b_x32(at + buf * S::TCOLS + col + 32, r[1]);
            };
            mbar_wait_suspended(tfull0 + buf * 8, bphase, tmo, failed);
            mbar_wait_suspended(sfull0 + chunk * 8, sphase, tmo, failed);
            tc_fence_after();
            load(0);
            float s = scale_at[chunk * S::SK * S::SROW];
            // Walked to its end also after a wait that has run out: lanes may differ in that,
            // and the loads of TMEM take the whole warp.  (Unrolled, registers spill; ended by
            // a vote of the lanes, 8192 x 7168 x 8192 takes 1 % longer.)
#pragma unroll 1
            for (int kb = kb0, in_chunk = 0; kb < kb1; ++kb) {
                const bool more = kb + 1 < kb1;
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    fma_one(acc[i >> 4][i & 15], r[i >> 5][i & 31], s);
                load(64);
                tmem_ld_wait();
                tc_fence_before();
                mbar_arrive_remote_relaxed(tempty0 + buf * 8, lane == 0);
                buf ^= 1;
                bphase ^= buf ^ 1;
                // the next block's scale
                if (++in_chunk == S::SK || !more) {
                    in_chunk = 0;
                    __syncwarp();
                    mbar_arrive_relaxed(&ps->sempty[chunk], lane == 0);
                    if (++chunk == S::SCH) {
                        chunk = 0;
                        sphase ^= 1u;
                    }
                    if (more)
                        mbar_wait_suspended(sfull0 + chunk * 8, sphase, tmo, failed);
                }
                float next = 0.f;
                if (more)
                    next = scale_at[(chunk * S::SK + in_chunk) * S::SROW];
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    fma_one(acc[4 + (i >> 4)][i & 15], r[i >> 5][i & 31], s);
                if (more) {
                    mbar_wait_suspended(tfull0 + buf * 8, bphase, tmo, failed);
                    tc_fence_after();
                    load(0);
                }
                s = next;
            }
            tmem_ld_wait();
            ok = __all_sync(0xffffffffu, !failed);
            if (!ok) {
                if (lane == 0)
                    report_fault(p.status, TDG_ERR_TIMEOUT, TDG_WHERE_PIPE, 3, p.epoch);
                ps->abort = 1;
                if (p.split > 1)
                    cluster_sync();
                break;
            }
            // Where two pairs share the tile's K: each leaves the half of its columns that
            // the other stores in its ring, whose loads the last products have used up.
            // (a + b is b + a: the sums do not depend on who adds.)
            if (p.split > 1) {
                float4 *give = reinterpret_cast<float4 *>(smem) + (threadIdx.x - 128);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float *lo = &acc[i >> 2][(i & 3) * 4], *hi = &acc[4 + (i >> 2)][(i & 3) * 4];
                    give[i * 32 * S::EPIW] = part ? make_float4(lo[0], lo[1], lo[2], lo[3]) : make_float4(hi[0], hi[1], hi[2], hi[3]);
                }
                cluster_sync();
                const uint32_t take = mapa_shared(smem_u32(give), (uint32_t)(rank ^ 2));
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float4 v = ld_cluster_f4(take + i * 32 * S::EPIW * 16);
                    float *lo = &acc[i >> 2][(i & 3) * 4], *hi = &acc[4 + (i >> 2)][(i & 3) * 4];
                    lo[0] = (part ? hi[0] : lo[0]) + v.x;
                    lo[1] = (part ? hi[1] : lo[1]) + v.y;
                    lo[2] = (part ? hi[2] : lo[2]) + v.z;
                    lo[3] = (part ? hi[3] : lo[3]) + v.w;
                }
            }
            // 128 bytes of each of the warp's 32 rows at a time through shared memory, from
            // where one TMA store takes them while the next tile is multiplied (an SM writes
            // about 22 bytes a cycle, 3000 cycles for a tile).  Rows that end inside the
            // tile are stored by the lanes.
            const int64_t row = ps->tile[nth & 3].row + q * 32, end = ps->tile[nth & 3].end;
            const int n = ps->tile[nth & 3].n0 + cg * 128 + part * 64, piece = lane & 7;
            const bool whole = row + 32 <= end || end == p.M; // (the map ends at row M)
            auto pass = [&](int col, int per16, auto words) { // columns from col on, per16 of them in 16 bytes
                uint8_t *stg = stg0 + side * S::STG;
                side ^= 1;
                if (lane == 0)
                    bulk_wait_read<1>(); // the copy from this buffer, two passes ago
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4 *>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) = words(j);
                if (whole)
                    fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (whole && row < end && n + col < p.N)
                        tma_store_2d(&map_out, stg, n + col, (int)row);
                    bulk_commit(); // one group a pass, if an empty one: the wait above counts them
                }
                if (whole)
                    return;
                const int left = p.N - n - col - piece * per16;
                uint8_t *out = static_cast<uint8_t *>(p.out) + ((row + (lane >> 3)) * p.out_stride + n + col) * (16 / per16) + piece * 16;
                const int64_t step = 4 * p.out_stride * (16 / per16);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = 4 * i + (lane >> 3);
                    const uint4 v = *reinterpret_cast<const uint4 *>(stg + r * 128 + ((piece ^ (r & 7)) << 4));
                    if (row + r < end && left > 0)
                        *reinterpret_cast<uint4 *>(out + i * step) = v;
                }
            };
            if (p.out_f32) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c == 2 && p.split > 1)
                        break;
                    pass(c * 32, 4, [&](int j) {
                        const float *a = &acc[2 * c + (j >> 2)][(j & 3) * 4];
                        return make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]), __float_as_uint(a[3]));
                    });
                }
            } else {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (c == 1 && p.split > 1)
                        break;
                    pass(c * 64, 8, [&](int j) {
                        const float *a = &acc[4 * c + (j >> 1)][(j & 1) * 8];
                        return make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7]));
                    });
                }
            }
        }
        if (lane == 0)
            bulk_wait<0>();
    }
    if (p.split > 1 && (warp < 4 || unit >= items))
        cluster_sync(); // the one of the epilogue's exchange
    scaled_drain<S>(p, ps);
    cluster_sync(); // no CTA leaves while the other may still touch it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// A thread of the epilogue holds, of each 8 x 8 square, two neighbouring rows
// of a (their scales are a float pair, so the multiply-adds are packed) for one
// row of the weights; for the store a transposing stmatrix turns the squares.
template <class S>
__global__ void __launch_bounds__(S::THREADS, 1)
    scaled_narrow_kernel(const __grid_constant__ ScaledParams p, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                         const __grid_constant__ CUtensorMap map_a16)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    ScaledSmem *ps = reinterpret_cast<ScaledSmem *>(smem + S::OFF_BAR);
    uint32_t *pre = reinterpret_cast<uint32_t *>(smem + S::OFF_PRE);
    float *scales = reinterpret_cast<float *>(smem + S::OFF_SCALE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = p.split > 1 ? (int)cluster_ctarank() : 0;
    const uint32_t unit = blockIdx.x / p.split, units = gridDim.x / p.split;
    const uint64_t tmo = p.timeout_ns;
    if (threadIdx.x == 64) {
        prefetch_tensormap(&map_w);
        prefetch_tensormap(&map_a);
        prefetch_tensormap(&map_a16);
    }
    scaled_begin<S>(p, ps, pre);
    const uint32_t tmem = ps->tmem_base;
    const uint32_t items = min(pre[p.E], p.split > 1 ? units : p.item1); // with K divided a cluster has one tile
    // this CTA's blocks of K
    const int kb0 = (int)((int64_t)p.k_blocks * crank / p.split), kb1 = (int)((int64_t)p.k_blocks * (crank + 1) / p.split);

    if (warp == 0) {
        if constexpr (S::REGS)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::REGS_OTHER));
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, issued = 0;
            for (uint32_t it = unit; it < items && !ps->abort; it += units) {
                const ScaledTile t = scaled_tile<S>(p, pre, it);
                // (boxes of 16 rows alone: 64 experts of 4096 x 7168 with 128 rows each 420 us, 331 like this)
                const int box = t.width <= S::STEP ? S::STEP : S::BOX, boxes = (t.width + box - 1) / box;
                const CUtensorMap *map = t.width <= S::STEP ? &map_a16 : &map_a;
                for (int kb = kb0; kb < kb1; kb += S::BPS) {
                    if (!mbar_wait_suspended(&ps->empty[stage], phase ^ 1u, tmo)) {
                        report_fault(p.status, TDG_ERR_TIMEOUT, TDG_WHERE_PIPE, 0, p.epoch);
                        ps->abort = 1;
                        break;
                    }
                    const int blocks = min(S::BPS, kb1 - kb);
                    const uint32_t bar = smem_u32(&ps->full[stage]);
                    mbar_arrive_expect_tx(&ps->full[stage], (uint32_t)(blocks * (sg::A_BYTES + boxes * box * sg::BK)));
                    for (int j = 0; j < blocks; ++j) {
                        uint8_t *dst = smem + stage * S::STAGE_BYTES + j * S::BLOCK_BYTES;
                        tma_load_3d_addr(dst, &map_w, bar, (kb + j) * sg::BK, t.n0, t.e);
                        for (int i = 0; i < boxes; ++i)
                            tma_load_2d_addr(dst + sg::A_BYTES + i * box * sg::BK, map, bar, (kb + j) * sg::BK, (int)((uint32_t)t.tok0 + i * box));
                    }
                    ++issued;
                    if (++stage == S::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            ps->issued = issued;
        }
        __syncwarp();
    } else if (warp == 1) {
        if constexpr (S::REGS)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::REGS_OTHER));
        scaled_issue<S>(p, ps, smem_u32(smem), tmem, pre, items, unit, units, kb0, kb1, 0, [](const ScaledTile &t) { return t.width; });
    } else if (warp < 4) {
        if constexpr (S::REGS)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::REGS_OTHER));
        // scales: 8 rows of a x SK blocks a step, each warp every other step
        const int j = lane % S::SK, r0 = lane / S::SK + (warp - 2) * 8;
        int chunk = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (uint32_t it = unit; it < items && ok; it += units) {
            const ScaledTile t = scaled_tile<S>(p, pre, it);
            const float *sw = p.b_scale + ((int64_t)t.e * p.n_blocks + t.n0 / 128) * p.k_blocks;
            const int rows = (int)(t.end - t.tok0);
            const float *sa = p.a_scale + t.tok0 * p.a_scale_stride;
            for (int kb = kb0; kb < kb1; kb += S::SK) {
                const bool in = kb + j < kb1;
                const float w = in ? sw[kb + j] : 0.f;
                float v[S::BT / 16];
#pragma unroll
                for (int i = 0; i < S::BT / 16; ++i) {
                    const int r = r0 + 16 * i;
                    v[i] = in && r < rows ? sa[(int64_t)r * p.a_scale_stride + kb + j] : 0.f;
                }
                ok = mbar_wait_suspended(&ps->sempty[chunk], phase ^ 1u, tmo);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) {
                    if (lane == 0)
                        report_fault(p.status, TDG_ERR_TIMEOUT, TDG_WHERE_PIPE, 2, p.epoch);
                    ps->abort = 1;
                    break;
                }
                float *dst = scales + (chunk * S::SK + j) * S::SROW + r0;
#pragma unroll
                for (int i = 0; i < S::BT / 16; ++i)
                    dst[16 * i] = v[i] * w;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&ps->sfull[chunk]);
                if (++chunk == S::SCH) {
                    chunk = 0;
                    phase ^= 1u;
                }
            }
        }
    } else {
        if constexpr (S::REGS)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::REGS_EPI));
        // lanes of TMEM; the group's chunks of 32 columns are g, g + GROUPS, ...
        const int q = warp & 3, g = (warp - 4) >> 2;
        uint8_t *stg = smem + S::OFF_STG + (warp - 4) * S::STG;
        constexpr int CH = S::BT / 32 / S::GROUPS, CW = 32 * S::GROUPS; // chunks of a warp, columns from one to the next
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + g * 32;
        const uint32_t tfull0 = smem_u32(&ps->tfull[0]), sfull0 = smem_u32(&ps->sfull[0]);
        int buf = 0, chunk = 0;
        uint32_t bphase = 0, sphase = 0, failed = 0;
        bool ok = true;
        for (uint32_t it = unit; it < items && ok; it += units) {
            const ScaledTile t = scaled_tile<S>(p, pre, it);
            uint64_t acc[CH][2][8];
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[c][0][i] = acc[c][1][i] = 0;
            // The blocks of a tile whose rows fill N chunks: code without a branch for each
            // chunk (with one, a block of 16 rows took 750 cycles).  One block's
            // accumulator is on its way while the one before is added.
            auto add_blocks = [&](auto chunks) {
                constexpr int N = decltype(chunks)::value;
#pragma unroll 1
                for (int kb = kb0, in_chunk = 0; kb < kb1; kb += S::BPS) { // (to the end, as in the wide kernel)
                    const bool two = kb + 1 < kb1;
                    if (in_chunk == 0)
                        mbar_wait_suspended(sfull0 + chunk * 8, sphase, tmo, failed);
                    uint64_t s[S::BPS][N][4];
                    const float *sc = scales + (chunk * S::SK + in_chunk) * S::SROW + g * 32 + 2 * (lane & 3);
#pragma unroll
                    for (int j = 0; j < S::BPS; ++j) // (a chunk holds whole pairs; zeros behind the last block)
#pragma unroll
                        for (int c = 0; c < N; ++c)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                s[j][c][i] = *reinterpret_cast<const uint64_t *>(sc + j * S::SROW + c * CW + 8 * i);
                    uint32_t lo[S::BPS][N][16], hi[S::BPS][N][16];
                    auto load = [&](int j) {
                        const uint32_t at = lanes + (uint32_t)((buf * S::BPS + j) * S::TCOLS);
#pragma unroll
                        for (int c = 0; c < N; ++c) {
                            tmem_ld_16x256b_x4(at + c * CW, lo[j][c]);
                            tmem_ld_16x256b_x4(at + (16u << 16) + c * CW, hi[j][c]);
                        }
                    };
                    auto add = [&](int j) {
#pragma unroll
                        for (int c = 0; c < N; ++c)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                fma_pair(acc[c][0][2 * i], lo[j][c][4 * i], lo[j][c][4 * i + 1], s[j][c][i]);
                                fma_pair(acc[c][0][2 * i + 1], lo[j][c][4 * i + 2], lo[j][c][4 * i + 3], s[j][c][i]);
                                fma_pair(acc[c][1][2 * i], hi[j][c][4 * i], hi[j][c][4 * i + 1], s[j][c][i]);
                                fma_pair(acc[c][1][2 * i + 1], hi[j][c][4 * i + 2], hi[j][c][4 * i + 3], s[j][c][i]);
                            }
                    };
                    mbar_wait_suspended(tfull0 + buf * 8, bphase, tmo, failed);
                    tc_fence_after();
                    load(0);
                    tmem_ld_wait();
                    if (two) {
                        load(1);
                        add(0);
                        tmem_ld_wait();
                        tc_fence_before();
                        mbar_arrive_relaxed(&ps->tempty[buf], lane == 0);
                        add(1);
                    } else {
                        tc_fence_before();
                        mbar_arrive_relaxed(&ps->tempty[buf], lane == 0);
                        add(0);
                    }
                    if (++buf == S::TBUF) {
                        buf = 0;
                        bphase ^= 1u;
                    }
                    in_chunk += S::BPS;
                    if (in_chunk == S::SK || kb + S::BPS >= kb1) {
                        in_chunk = 0;
                        __syncwarp();
                        mbar_arrive_relaxed(&ps->sempty[chunk], lane == 0);
                        if (++chunk == S::SCH) {
                            chunk = 0;
                            sphase ^= 1u;
                        }
                    }
                }
            };
            if (t.width <= CW)
                add_blocks(std::integral_constant<int, 1>{});
            else
                add_blocks(std::integral_constant<int, 2>{});
            ok = __all_sync(0xffffffffu, !failed);
            if (!ok) {
                if (lane == 0)
                    report_fault(p.status, TDG_ERR_TIMEOUT, TDG_WHERE_PIPE, 3, p.epoch);
                ps->abort = 1;
            }
            if (!ok)
                break;
            if (p.split > 1) { // partial sums, for the cluster to add
                float *red = reinterpret_cast<float *>(smem);
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    if (c * CW + g * 32 < t.width)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                const float2 f = halves(acc[c][m >> 1][2 * i + (m & 1)]);
                                float *d = red + (c * CW + g * 32 + 8 * i + 2 * (lane & 3)) * S::RED + q * 32 + 8 * m + (lane >> 2);
                                d[0] = f.x;
                                d[S::RED] = f.y;
                            }
                continue;
            }
            const int n = t.n0 + q * 32;
            if (p.out_f32) {
                float *out = static_cast<float *>(p.out);
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const float2 f = halves(acc[c][m >> 1][2 * i + (m & 1)]);
                            const int64_t row = t.tok0 + c * CW + g * 32 + 8 * i + 2 * (lane & 3);
                            const int col = n + 8 * m + (lane >> 2);
                            if (col < p.N && row < t.end)
                                out[row * p.out_stride + col] = f.x;
                            if (col < p.N && row + 1 < t.end)
                                out[(row + 1) * p.out_stride + col] = f.y;
                        }
            } else {
                const uint32_t put = smem_u32(stg) + (lane & 7) * S::STG_ROW + (lane >> 3) * 16;
                const uint8_t *get = stg + (lane >> 2) * S::STG_ROW + (lane & 3) * 16;
                const int col = n + (lane & 3) * 8;
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    if (c * CW + g * 32 < t.width)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            __syncwarp();
                            stmatrix_x4_trans(put, narrowed(acc[c][0][2 * i]), narrowed(acc[c][0][2 * i + 1]), narrowed(acc[c][1][2 * i]),
                                              narrowed(acc[c][1][2 * i + 1]));
                            __syncwarp();
                            const uint4 v = *reinterpret_cast<const uint4 *>(get);
                            const int64_t row = t.tok0 + c * CW + g * 32 + 8 * i + (lane >> 2);
                            if (col < p.N && row < t.end)
                                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + row * p.out_stride + col) = v;
                        }
            }
        }
    }
    scaled_drain<S>(p, ps);
    if (p.split > 1) {
        cluster_sync(); // the partial sums are there
        if (unit < items && !ps->abort) {
            // this CTA's share of the rows, summed over the cluster in rank order
            const ScaledTile t = scaled_tile<S>(p, pre, unit);
            const int rows = (int)(t.end - t.tok0), mine = (rows - crank + p.split - 1) / p.split;
            const uint32_t red = smem_u32(smem);
            for (int i = threadIdx.x; i < mine * 32; i += S::THREADS) {
                const int r = crank + (i >> 5) * p.split, c = (i & 31) * 4;
                if (t.n0 + c >= p.N)
                    continue;
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < p.split; ++k) {
                    const float4 v = ld_cluster_f4(mapa_shared(red + (uint32_t)(r * S::RED + c) * 4, (uint32_t)k));
                    sum.x += v.x;
                    sum.y += v.y;
                    sum.z += v.z;
                    sum.w += v.w;
                }
                const int64_t at = (t.tok0 + r) * p.out_stride + t.n0 + c;
                if (p.out_f32)
                    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = sum;
                else
                    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) =
                        make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
            }
        }
        cluster_sync(); // no CTA leaves while another may still read its sums
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

} // namespace tdg

using namespace tdg;
using namespace tdg_host;

namespace {

bool map_codes(CUtensorMap *m, const void *base, int64_t inner, int64_t rows, int64_t row_bytes, int64_t matrices, int box_rows, bool flat)
{
    const uint64_t dims[3] = {(uint64_t)inner, (uint64_t)rows, (uint64_t)matrices};
    const uint64_t strides[2] = {(uint64_t)row_bytes, (uint64_t)(rows * row_bytes)};
    const uint32_t box[3] = {sg::BK, (uint32_t)box_rows, 1};
    return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, flat ? 2 : 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <class S> const void *kernel_of()
{
    if constexpr (S::PAIR)
        return reinterpret_cast<const void *>(&scaled_wide_kernel);
    else
        return reinterpret_cast<const void *>(&scaled_narrow_kernel<S>);
}

// The clusters of cl CTAs of a kernel that run at once; a property of the device,
// asked once for each (the query takes microseconds).
template <class S> int clusters_at_once(int device, int cl)
{
    static std::atomic<int> known[64][5];
    const bool keep = device >= 0 && device < 64;
    int n = keep ? known[device][cl].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        const int smem = S::SMEM + 4 * (sg::MAX_E + 1);
        if (set_smem(kernel_of<S>(), smem) == cudaSuccess)
            n = max_clusters(kernel_of<S>(), S::THREADS, smem, cl);
        if (keep)
            known[device][cl].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <class S> int run(tdg_symm *h, const tdg_scaled_gemm_args *a, ScaledParams &p, int split, int64_t units, cudaStream_t s)
{
    CUtensorMap map_w, map_a, third; // of the output; narrow: of a, in smaller boxes
    if (!map_codes(&map_w, a->b, a->K, a->N, a->K, a->E, sg::ROWS, false) || !map_codes(&map_a, a->a, a->K, a->M, a->a_stride, 1, S::BOX, true))
        return TDG_ERR_CUDA;
    if constexpr (!S::PAIR) {
        if (!map_codes(&third, a->a, a->K, a->M, a->a_stride, 1, S::STEP, true))
            return TDG_ERR_CUDA;
    } else if (!(a->out_f32 ? map_f32_2d(&third, a->out, a->N, a->M, a->out_stride * 4, 32, 32)
                            : map_bf16_2d(&third, a->out, a->N, a->M, a->out_stride * 2, 64, 32)))
        return TDG_ERR_CUDA;
    const void *fn = kernel_of<S>();
    const int smem = S::SMEM + 4 * (sg::MAX_E + 1);
    cudaError_t e = set_smem(fn, smem);
    if (e != cudaSuccess)
        return cuda_err(e, "scaled gemm smem");
    p.split = split;
    p.n_tiles = (int)((a->N + S::WTILE - 1) / S::WTILE);
    const int cl = S::PAIR ? 2 * split : split;
    void *args[] = {&p, &map_w, &map_a, &third};
    return cuda_err(launch(fn, dim3((unsigned)(units * cl)), dim3(S::THREADS), S::SMEM + 4 * ((size_t)a->E + 1), s, args, false, cl, true),
                    "scaled gemm launch");
}

} // namespace

extern "C" int tdg_scaled_gemm(tdg_symm *h, const tdg_scaled_gemm_args *a, void *stream)
{
    if (!h || !a)
        return TDG_ERR_INVALID;
    if (const int drc = check_device(h))
        return drc;
    if (a->M < 0 || a->M > INT32_MAX || a->N < 8 || a->N % 8 || a->N >= (1 << 24) || a->K < 16 || a->K % 16 || a->K >= (1 << 24) || a->E < 1 ||
        a->E > sg::MAX_E || a->E * a->N > INT32_MAX || (!a->base && a->E != 1) || (a->out_f32 & ~1))
        return TDG_ERR_INVALID;
    const int64_t kb = (a->K + 127) / 128, nb = (a->N + 127) / 128;
    if (a->M == 0)
        return TDG_OK;
    const int esz = a->out_f32 ? 4 : 2;
    if (!a->a || !aligned16(a->a) || !a->b || !aligned16(a->b) || !a->out || !aligned16(a->out) || !a->a_scale || !aligned4(a->a_scale) ||
        !a->b_scale || !aligned4(a->b_scale) || !aligned8(a->base) || !stride_ok(a->a_stride, a->K, 16) ||
        !stride_ok(a->a_scale_stride, kb, 1) || !stride_ok(a->out_stride, a->N, 16 / esz))
        return TDG_ERR_INVALID;
    const Range out{a->out, extent(a->M, a->out_stride, a->N, esz)}, rb{a->b, (uint64_t)a->E * a->N * a->K};
    const Range rbs{a->b_scale, (uint64_t)a->E * nb * kb * 4}, base{a->base, (uint64_t)(a->E + 1) * 8};
    const ByteRows outr{a->out, esz * a->out_stride, esz * a->N};
    if (ranges_overlap({out}, {rb, rbs, base}) || rows_share(a->M, outr, {a->a, a->a_stride, a->K}) ||
        rows_share(a->M, outr, {a->a_scale, 4 * a->a_scale_stride, 4 * kb}))
        return TDG_ERR_INVALID;
    // the tiles, at most, of each kernel's shape: with experts, one more for each than its rows fill
    auto most_tiles = [&](int64_t bt, int64_t wtile) {
        const int64_t rows = a->base ? (a->E < a->M ? a->E : a->M) + a->M / bt : (a->M + bt - 1) / bt;
        return rows * ((a->N + wtile - 1) / wtile);
    };
    if (most_tiles(NarrowShape<64>::BT, NarrowShape<64>::WTILE) > INT32_MAX)
        return TDG_ERR_INVALID;
    const int64_t wide = most_tiles(WideShape::BT, WideShape::WTILE);
    ScaledParams p;
    memset(&p, 0, sizeof p);
    p.status = h->status;
    p.epoch = next_epoch(h);
    p.timeout_ns = pipe_timeout(timeout_or_default(0));
    p.M = a->M;
    p.a_scale_stride = a->a_scale_stride;
    p.out_stride = a->out_stride;
    p.N = (int)a->N;
    p.E = (int)a->E;
    p.k_blocks = (int)kb;
    p.n_blocks = (int)nb;
    p.out_f32 = a->out_f32;
    p.a_scale = a->a_scale;
    p.b_scale = a->b_scale;
    p.out = a->out;
    p.base = a->base;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // The kernel whose tiles take less time (us): rounds of the grid, each of a time for
    // the tile and one for every block of K.  Experts' shares are counted as what tokens
    // sent at random exceed the average by, its square root (64 experts of 4096 x 7168
    // with 64 rows each on average: 320 us by tiles of 64, 309 by tiles of 128; with 128:
    // 431 by tiles of 128, 392 wide).
    const int64_t used = a->E < a->M ? a->E : a->M, even = (a->M + used - 1) / used, share = a->E > 1 ? even + (int64_t)std::sqrt((double)even) : even, pairs = h->sm_count / 2;
    auto time_of = [&](int64_t bt, int64_t wtile, int64_t at_once, double tile, double block) {
        const int64_t tiles = used * ((share + bt - 1) / bt) * ((a->N + wtile - 1) / wtile);
        return (double)((tiles + at_once - 1) / at_once) * (tile + block * (double)kb);
    };
    // Narrow, few tiles: K divided over the CTAs of a cluster, two blocks of it each at
    // least, as long as all clusters run at once.  How many do is less than the SMs hold
    // (46 of 3, 36 of 4), since a cluster stays in its part of the chip: 38 weight tiles
    // of 2048, one row, 6.1 us by clusters of 3 and 10.4 by clusters of 4.  (Clusters of
    // 6 and 8 start 5 us later: 2048 x 2048, one row, 5.4 by 4 CTAs and 11.8 by 8.)
    struct Plan {
        int split;
        int64_t units, tiles;
        double time;
    };
    auto narrow = [&](auto shape, double tile, double block, double join) {
        using S = decltype(shape);
        const int64_t tiles = most_tiles(S::BT, S::WTILE);
        int split = 4, at_once = h->sm_count;
        for (; split > 1; --split)
            if (kb / 2 >= split && tiles <= clusters_at_once<S>(h->device, split)) {
                at_once = clusters_at_once<S>(h->device, split);
                break;
            }
        return Plan{split, tiles < at_once ? tiles : at_once, tiles, time_of(S::BT, S::WTILE, at_once, tile + (split > 1 ? join : 0.), block / split)};
    };
    // us measured with tiles of 64 rows, of 128, wide, and wide by two pairs a tile:
    //   64 experts of 4096 x 7168, 64 rows each   291  299
    //                              80 rows        383  315  385
    //                              128 rows            329  396
    //   7168 x 8192, 128 rows                      25   19   32   21
    //   5120 x 3200, 96 rows                      9.3 10.3 15.5 12.7
    //                333 rows                      20 13.1 15.6
    // (4 us: partial sums of 128 x 128 are joined)
    const Plan n64 = narrow(NarrowShape<64>{}, 0.5, 0.30, 0.), n128 = narrow(NarrowShape<128>{}, 1., 0.36, 4.);
    const double by_narrow = n64.time <= n128.time ? n64.time : n128.time;
    const double by_wide = time_of(WideShape::BT, WideShape::WTILE, pairs, 1.6, 0.415);
    // By two pairs a tile, as many tiles as run at once: all, or, where their number is
    // known, those behind whole rounds, by a launch of their own, 4.5 us (1024 rows by
    // 7168 x 8192, 112 tiles: 59 us in two whole rounds, 54 like this; 5120 x 3200, 80
    // tiles: 26.6 and 27.8).  Halves of K always have a block: two pairs take less time
    // from 10 blocks on.
    const int64_t rest = wide % pairs, whole = wide - rest;
    p.item1 = (uint32_t)wide;
    if (rest && (!whole || !a->base) && rest <= clusters_at_once<WideShape>(h->device, 4)) {
        const double by_two = 3.6 + 0.415 / 2 * (double)kb + (whole ? (double)(whole / pairs) * (1.6 + 0.415 * (double)kb) + 4.5 : 0.);
        if (by_two < by_wide && by_two < by_narrow) {
            if (whole) {
                p.item1 = (uint32_t)whole;
                if (const int rc = run<WideShape>(h, a, p, 1, pairs, s))
                    return rc;
                p.item0 = (uint32_t)whole;
                p.item1 = (uint32_t)wide;
            }
            return run<WideShape>(h, a, p, 2, rest, s);
        }
    }
    if (by_wide < by_narrow)
        return run<WideShape>(h, a, p, 1, wide < pairs ? wide : pairs, s);
    p.item1 = (uint32_t)(n64.time <= n128.time ? n64 : n128).tiles;
    if (n64.time <= n128.time)
        return run<NarrowShape<64>>(h, a, p, n64.split, n64.units, s);
    return run<NarrowShape<128>>(h, a, p, n128.split, n128.units, s);
}
