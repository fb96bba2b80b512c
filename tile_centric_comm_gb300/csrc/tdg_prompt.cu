// tdg_prompt.cu -- attention over whole prompts packed one after another:
// softmax(scale Q K^T) V per sequence, causal from the last key back.
//
// Mathematics: per query row a running maximum m and sum l over blocks of
// keys, in base 2:  P = 2^(c s - m),  l += sum P,  O += P V,  c = scale log2 e.
// m follows the row's true maximum only when that has grown by more than 8
// (a factor of 256): until then P stays below 2^8 and the old m serves as
// well, so the output, which lives in TMEM, is rarely rescaled.  S, m, l and O
// are float32; P is rounded to bf16 for its product.
//
// Work: an item is 256 rows of one key head -- two tiles of 128, each 128/G
// tokens times the G = Hq/Hkv query heads that share the key head, so a block
// of keys and values is fetched once for all of them and a tile's causal edge
// is only 128/G tokens wide.  The grid has a CTA per item, and a CTA that is
// done takes over one that has not been launched (cluster launch control): no
// counter in memory, and SMs are busy until the items run out.  Roles:
//   warps 0-3, 4-7  softmax of tile 0 and 1: a thread owns a row
//   warp 8          issues tcgen05.mma: S_t = Q_t K^T from shared memory,
//                   O_t += P_t V with P_t read from TMEM, where the softmax
//                   left it in S_t's own columns
//   warp 9          finds items, loads Q, K and V by TMA into a ring of 4 slots
//   warps 10, 11    (one CTA an SM) idle: they complete the warpgroup that
//                   gives registers up
// While the softmax works on one tile, the tensor cores work on the other.
// Blocks are 128 keys with one CTA on an SM.  Heads of 64 with many items take
// 64 keys and two CTAs an SM instead: their products are half as long, and one
// CTA's two tiles leave the tensor cores waiting.  Few items of many keys:
// a cluster of up to 8 CTAs shares an item's keys and joins through
// distributed shared memory.
//
// Bound: 4 D flops per query, key and head on the tensor cores.  Measured on
// one GB300 (dense peak measured there: 1876 TFLOP/s):
// (a call alone; back to back the power cap lowers the clock: 8192 tokens 670 to 690)
//   8192 tokens, 64 / 8 heads of 128           632 us, 1740 TFLOP/s, 93 %; not
//                                              causal 1236 us, 1780 TFLOP/s
//   1000 behind 7000, 2 x, same heads          333 us, 1505 TFLOP/s; 3.4 items
//                                              an SM: 85 % of what 4 would take
//   12 of 17..2311, 40 / 8 heads of 128        214 us, 1200 TFLOP/s: short items; at
//                                              each one's end the softmax's warps also
//                                              divide and store, and its next scores wait
//   4 of 2048..4096, 32 heads of 64            230 us, 870 TFLOP/s (60 bytes a thread
//                                              spilled): with weights left as they are
//                                              167 us, that is what products of 64
//                                              columns reach here
//   119 tokens, 64 / 8 heads of 128            8.8 us: launch, table, one block
#include <type_traits>

#include "tdg_paged.cuh"

namespace tdg {

namespace pa {
// registers a thread, one CTA an SM: 168 at launch; 2 x 208 + 88 = 3 x 168, so
// the split asks for no more than the launch holds (two CTAs: 96 for all)
constexpr int REGS_SOFTMAX = 208, REGS_OTHER = 88;
constexpr int MMA_WARP = 8, LOAD_WARP = 9;
constexpr int CHUNKS = 256;   // entries of the item table
constexpr int SLOTS = 2;      // items in hand
// Items go by their length, the longest of all sequences first, when there are
// several sequences, more items than SMs, and K and V take less than this; else
// by sequences, the longest first, which share what they read.  By sequence and
// by length: 8 of 1700 tokens, 8 heads of 64 (28 MB) 57 -> 45 us, 24 of 790, 14 / 2
// heads of 128 (19 MB) 72 -> 66; but 12 of 17..2311, 8 key heads of 128 (54 MB)
// 214 -> 219, 16 of 4096 (268 MB) 2880 -> 3460.
constexpr int64_t BY_LENGTH_BYTES = (int64_t)32 << 20;
// Heads of 64: two CTAs an SM from this many items for each SM.  One and two:
// 46 of 350 tokens, 32 / 4 heads (13 items) 84 -> 72 us, 32 of 300..3000, 32 / 8 heads
// (43 items) 700 -> 555; but 8 of 1700, 8 heads (3 items) 45 -> 58.
constexpr int TWO_CTAS_ITEMS = 6;
constexpr int MAX_SPLIT = 8;  // CTAs that share an item's keys

// BLOCK: keys of a block, 128, or 64 where two CTAs share an SM
template <int D, int BLOCK> struct Shape {
    static constexpr int BN = BLOCK;
    static constexpr int CTAS = BN == 64 ? 2 : 1; // of an SM
    static constexpr int THREADS = BN == 64 ? 320 : 384;
    static constexpr int O_COL = 2 * BN; // columns of TMEM: S_t begins at t BN, O_t at O_COL + t D
    static constexpr uint32_t TMEM_COLS = BN == 64 ? 256 : 512;
    static constexpr int HALVES = D / 64;
    static constexpr int Q_BYTES = 128 * D * 2;
    static constexpr int KV_BYTES = BN * D * 2;
    static constexpr int STAGES = 4; // an item takes 2 slots a block: it begins in slot 0 or 2
    static constexpr int OFF_KV = 2 * Q_BYTES;
    static constexpr int OFF_CTL = OFF_KV + STAGES * KV_BYTES;
};
} // namespace pa

struct PromptParams {
    DevStatus *status;
    uint32_t epoch;
    uint64_t timeout_ns;
    int64_t Tq, Tk, B, os;
    int Hq, Hkv, G, NT; // NT: tokens of a tile, 128 / G
    int causal;
    int split; // CTAs of a cluster that share an item's keys (SPLIT)
    int out32; // rows of out are 32-byte aligned
    int by_length; // items in the order of their lengths
    float scale_log2;
    __nv_bfloat16 *out;
    float *lse;
    const int32_t *cu_q, *cu_k;
};

// Tokens [t0, t0 + 2 NT) of a sequence and key head g.
struct PromptItem {
    int q0, Lq, k0, Lk, g, t0, valid, pad;
};

// The key blocks [lo, hi) of a SPLIT item that are this CTA's.
struct PromptShare {
    int lo, hi;
};

struct PromptCtl {
    uint64_t kvfull[8], kvempty[8], qfull[2], qempty[2], sfull[2], pfull[2], ofull[2];
    uint64_t ifull[pa::SLOTS], iempty[pa::SLOTS], tail, drain, steal;
    PromptItem item[pa::SLOTS];
    uint4 stolen;                      // answer to the request for a further item
    float2 stat[2][128];               // SPLIT: maximum and sum of this CTA's rows
    PromptShare share;
    uint32_t tmem_base;
    volatile int abort;
    uint32_t first[pa::CHUNKS + 1];    // first item of every table entry
    uint16_t order[pa::CHUNKS];        // the sequence of an entry, longest first
    uint32_t top[pa::CHUNKS];          // length of an entry's longest item, in spans of an item
};
template <int D, int BN> constexpr int prompt_smem() { return pa::Shape<D, BN>::OFF_CTL + (int)sizeof(PromptCtl); }
static_assert(prompt_smem<128, 128>() <= 227 * 1024 && prompt_smem<64, 64>() <= 113 * 1024, "shared memory");

// Rows of sequence b; false when the offsets are out of order or range (the
// sequence then counts as empty).
__device__ __forceinline__ bool prompt_sequence(const PromptParams &p, int64_t b, PromptItem &it)
{
    const int64_t qa = p.cu_q[b], qb = p.cu_q[b + 1], ka = p.cu_k[b], kb = p.cu_k[b + 1];
    const bool ok = qa >= 0 && qb >= qa && qb <= p.Tq && ka >= 0 && kb >= ka && kb <= p.Tk;
    it.q0 = (int)qa;
    it.k0 = (int)ka;
    it.Lq = ok ? (int)(qb - qa) : 0;
    it.Lk = ok ? (int)(kb - ka) : 0;
    return ok;
}

// Keys that token `tok` of the item's sequence sees.
__device__ __forceinline__ int prompt_limit(const PromptParams &p, const PromptItem &it, int tok)
{
    return p.causal ? min(it.Lk, max(0, tok + it.Lk - it.Lq + 1)) : it.Lk;
}

// Keys that the last token of tile t (0 or 1) sees: the tile's key blocks end there.
__device__ __forceinline__ int prompt_most(const PromptParams &p, const PromptItem &it, int t)
{
    const int lo = it.t0 + t * p.NT, hi = min(lo + p.NT, it.Lq);
    return hi > lo ? prompt_limit(p, it, hi - 1) : 0;
}
// The tile's key blocks (SPLIT: those that are this CTA's).
template <int BN, bool SPLIT>
__device__ __forceinline__ int prompt_blocks(const PromptParams &p, const PromptItem &it, int t, const PromptShare &share)
{
    const int all = (prompt_most(p, it, t) + BN - 1) / BN;
    return SPLIT ? max(0, min(all, share.hi) - share.lo) : all;
}

// The MMA warp runs its whole loop converged and the instructions themselves
// are predicated on one elected lane: their operands then stay in uniform
// registers.  (Issued from a branch that only one lane takes, each instruction
// of 64 cycles' tensor work costs more than 64 cycles to issue.)
// Shared-memory matrix descriptors (128-byte swizzle, 8 rows 1 KB apart) come
// by halves: the low word holds the address and the leading offset, the high
// word is the same for all.
constexpr uint32_t SDESC_HI = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t sdesc_lo(uint32_t saddr, uint32_t lbo) { return (saddr & 0x3FFFFu) >> 4 | (lbo >> 4) << 16; }

// Items are CTAs of the grid: a running CTA takes over one that has not been
// launched yet (cluster launch control), so every SM is busy until the items
// run out, whatever they cost, and no counter in memory is needed.
__device__ __forceinline__ void steal_request(uint4 *answer, uint64_t *bar)
{
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(answer)),
                 "r"(smem_u32(bar))
                 : "memory");
}
// the index of the CTA taken over, or -1 when none is left
__device__ __forceinline__ int64_t steal_answer(const uint4 *answer)
{
    uint32_t ok, x;
    asm volatile("{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
                 "ld.shared.b128 r, [%2];\n\t"
                 "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
                 "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
                 : "=r"(ok), "=r"(x)
                 : "r"(smem_u32(answer))
                 : "memory");
    return ok ? (int64_t)x : -1;
}

__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}

// D[tmem] (+)= A[smem] B[smem], by the lane with `leader`
__device__ __forceinline__ void umma_ss(uint32_t leader, uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc,
                                        uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 e, %0, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 da, {%2, %6};\n\tmov.b64 db, {%3, %6};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%1], da, db, %4, p;\n\t}" ::"r"(leader),
        "r"(d_tmem), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(SDESC_HI)
        : "memory");
}

// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void umma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t idesc,
                                        uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\t"
        "setp.ne.b32 e, %0, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 db, {%3, %6};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], db, %4, p;\n\t}" ::"r"(leader),
        "r"(d_tmem), "r"(a_tmem), "r"(b), "r"(idesc), "r"(accumulate), "r"(SDESC_HI)
        : "memory");
}

__device__ __forceinline__ void umma_commit_if(uint32_t leader, uint64_t *bar)
{
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %0, 0;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(leader),
                 "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 bytes in one store (32-byte aligned)
__device__ __forceinline__ void st_global_32(void *p, const uint32_t *w)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// (a.x, a.y) * (b.x, b.y) + (c.x, c.y) in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

template <int D, int BN, bool SPLIT>
__global__ void __launch_bounds__(pa::Shape<D, BN>::THREADS, pa::Shape<D, BN>::CTAS)
    prompt_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using S = pa::Shape<D, BN>;
    static_assert(!SPLIT || S::STAGES * S::KV_BYTES >= 256 * D * 4, "the join's rows lie over the ring");
    extern __shared__ __align__(1024) uint8_t smem[];
    PromptCtl *ctl = reinterpret_cast<PromptCtl *>(smem + S::OFF_CTL);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(&ctl->kvfull[i], 1);
            mbar_init(&ctl->kvempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->qfull[i], 1);
            mbar_init(&ctl->qempty[i], 1);
            mbar_init(&ctl->sfull[i], 1);
            mbar_init(&ctl->pfull[i], 4);
            mbar_init(&ctl->ofull[i], 1);
        }
        for (int i = 0; i < pa::SLOTS; ++i) {
            mbar_init(&ctl->ifull[i], 1);
            mbar_init(&ctl->iempty[i], 9); // the issuer and eight softmax warps
        }
        mbar_init(&ctl->tail, 1);
        mbar_init(&ctl->drain, 1);
        mbar_init(&ctl->steal, 1);
        ctl->abort = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
        prefetch_tensormap(&qmap);
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    if (warp == pa::MMA_WARP) {
        tmem_alloc(&ctl->tmem_base, S::TMEM_COLS);
        tmem_relinquish();
        tc_fence_before();
    }
    // launched while the kernel before may still run: nothing above touches memory
    griddep_launch_dependents();
    griddep_wait();
    // The item table.  Up to CHUNKS sequences: one entry each, the longest
    // first, so that what is left at the end is short; more: runs of
    // sequences in their own order (each is then a small part of the whole).
    // An entry's items are numbered from its last tokens, and each is one span
    // shorter than the one before.
    const int64_t per = (p.B + pa::CHUNKS - 1) / pa::CHUNKS;
    const int span = 2 * p.NT; // tokens of an item
    {
        const int i = threadIdx.x;
        const int64_t lo = min(i * per, p.B), hi = i < pa::CHUNKS ? min(lo + per, p.B) : lo;
        int64_t n = 0, past = 0;
        for (int64_t b = lo; b < hi; ++b) {
            PromptItem it;
            if (!prompt_sequence(p, b, it) && blockIdx.x == 0)
                report_fault(p.status, TDG_ERR_DEVICE, TDG_WHERE_CU, (uint32_t)b, p.epoch);
            n += (it.Lq + span - 1) / span;
            if (p.by_length)
                past = max(0, it.Lk - it.Lq) / span;
        }
        if (i < pa::CHUNKS)
            ctl->first[i] = (uint32_t)n;
        __syncthreads();
        if (i < pa::CHUNKS) {
            int rank = 0;
            if (per == 1) {
                for (int j = 0; j < (int)p.B; ++j) {
                    const uint32_t x = ctl->first[j];
                    rank += x > (uint32_t)n || (x == (uint32_t)n && j < i) ? 1 : 0;
                }
                if (i >= p.B)
                    rank = i;
            } else {
                rank = i;
            }
            ctl->order[rank] = (uint16_t)i;
            ctl->top[rank] = (uint32_t)(n + past);
        }
        __syncthreads();
        if (warp == 0) { // exclusive sums in that order, 8 entries a lane
            uint32_t x[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = sum;
                sum += ctl->first[ctl->order[lane * 8 + j]];
            }
            uint32_t upto = sum;
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d)
                    upto += y;
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                ctl->first[lane * 8 + j] = upto - sum + x[j];
            if (lane == 31)
                ctl->first[pa::CHUNKS] = upto;
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    const uint32_t items = ctl->first[pa::CHUNKS] * (uint32_t)p.Hkv;
    const uint64_t tmo = p.timeout_ns;
    auto wait = [&](uint64_t *b, uint32_t phase, uint32_t what) -> bool {
        if (mbar_wait(b, phase, tmo))
            return true;
        report_fault(p.status, TDG_ERR_TIMEOUT, TDG_WHERE_PIPE, what, p.epoch);
        ctl->abort = 1;
        return false;
    };

    if (warp < pa::MMA_WARP) {
        if constexpr (S::CTAS == 1)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(pa::REGS_SOFTMAX));
        const int t = warp >> 2; // tile
        const int r = (warp & 3) * 32 + lane;
        const int row_tok = r / p.G;
        const bool row_used = r < p.NT * p.G;
        const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16;
        const uint32_t s_addr = tmem + lanes + t * BN, o_addr = tmem + lanes + S::O_COL + t * D;
        int slot = 0;
        uint32_t slot_phase = 0, s_phase = 0, o_phase = 0;
        while (true) {
            bool ok = wait(&ctl->ifull[slot], slot_phase, 30);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                break;
            const PromptItem &it = ctl->item[slot]; // held to its end: registers are short
            if (!it.valid)
                break;
            const PromptShare share = SPLIT ? ctl->share : PromptShare{0, 0};
            const int nb = prompt_blocks<BN, SPLIT>(p, it, t, share);
            const int open = prompt_limit(p, it, it.t0 + t * p.NT); // keys every row of the tile sees
            float m = -INFINITY, l = 0.f;                        // m: in units of s
            for (int j = 0; j < nb; ++j) {
                ok = __all_sync(0xffffffffu, wait(&ctl->sfull[t], s_phase, 31));
                if (!ok)
                    break;
                s_phase ^= 1u;
                tc_fence_after();
                uint32_t s[BN / 32][32];
#pragma unroll
                for (int c = 0; c < BN / 32; ++c)
                    tmem_ld_32x32b_x32(s_addr + c * 32, s[c]);
                tmem_ld_wait();
                const int key0 = ((SPLIT ? share.lo : 0) + j) * BN; // the block's first key
                if (key0 + BN > open) { // the causal edge or the sequence's end runs through this block
                    const int lim = prompt_limit(p, it, it.t0 + t * p.NT + row_tok) - key0;
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) {
                        const int n = lim - c * 32; // of this chunk's 32
                        const uint32_t sees = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            s[c][i] = sees >> i & 1 ? s[c][i] : 0xFF800000u; // -inf
                    }
                }
                float mx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mx[i] = __uint_as_float(s[i * BN / 128][i * BN / 4 % 32]);
#pragma unroll
                for (int c = 1; c < BN / 4; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mx[i] = fmaxf(mx[i], __uint_as_float(s[i * BN / 128][i * BN / 4 % 32 + c]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const bool grown = j > 0 && (top - m) * p.scale_log2 > 8.f; // also from -inf
                const float al = grown ? exp2_approx((m - top) * p.scale_log2) : 1.f;
                m = j == 0 || grown ? top : m;
                const float ms = m == -INFINITY ? 0.f : m * p.scale_log2;
                const float2 c2 = make_float2(p.scale_log2, p.scale_log2), m2 = make_float2(-ms, -ms);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < BN / 16; ++c) {
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t *sc = s[c / 2] + c % 2 * 16 + 2 * i;
                        const float2 x = fma2(make_float2(__uint_as_float(sc[0]), __uint_as_float(sc[1])), c2, m2);
                        const float2 e = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                        sum[i & 1] = add2(sum[i & 1], e);
                        w[i] = pack_bf16x2(e.x, e.y);
                    }
                    tmem_st_32x32b_x8(s_addr + c * 8, w);
                }
                // O follows a new m only now, off the weights' path.  The block
                // before has left the tensor cores: its product was issued ahead
                // of this block's scores.
                if (__any_sync(0xffffffffu, grown)) {
                    l *= al;
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tmem_ld_32x32b_x16(o_addr + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
                        tmem_st_32x32b_x16(o_addr + c, o);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&ctl->pfull[t]);
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
            }
            if (!ok)
                break;
            if (nb) {
                ok = __all_sync(0xffffffffu, wait(&ctl->ofull[t], o_phase, 32));
                if (!ok)
                    break;
                o_phase ^= 1u;
                tc_fence_after();
            }
            if constexpr (SPLIT) {
                // This CTA's maximum, sum and output of the row go to shared
                // memory, the output over the ring, once nothing reads the ring.
                if (prompt_blocks<BN, SPLIT>(p, it, t ^ 1, share))
                    ok = __all_sync(0xffffffffu, wait(&ctl->ofull[t ^ 1], 0, 32));
                tc_fence_after();
                ctl->stat[t][r] = make_float2(nb ? m * p.scale_log2 : -INFINITY, l);
                float *dst = reinterpret_cast<float *>(smem + S::OFF_KV) + (t * 128 + r) * D;
                const bool wanted = row_used && it.t0 + t * p.NT + row_tok < it.Lq;
#pragma unroll 1
                for (int c = 0; nb && c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(o_addr + c, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; wanted && i < 8; ++i) // chunks of 16 bytes xored by the row: no bank conflicts
                        *reinterpret_cast<uint4 *>(dst + (((c / 4 + i) ^ (r & (D / 4 - 1))) * 4)) =
                            make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&ctl->iempty[slot]);
                slot = 1;
                continue; // the next item is the end
            }
            const int tok = it.t0 + t * p.NT + row_tok;
            const bool mine = row_used && tok < it.Lq;
            const bool sees = prompt_limit(p, it, tok) > 0;
            const float f = sees ? 1.f / l : 0.f;
            const int64_t row = (int64_t)it.q0 + tok;
            const int h = it.g * p.G + r - row_tok * p.G;
            __nv_bfloat16 *dst = p.out + row * p.os + (int64_t)h * D;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                if (nb) {
                    tmem_ld_32x32b_x16(o_addr + c, o);
                    tmem_ld_wait();
                }
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i] = sees ? pack_bf16x2(__uint_as_float(o[2 * i]) * f, __uint_as_float(o[2 * i + 1]) * f) : 0u;
                if (mine && p.out32) { // whole 32-byte sectors
                    st_global_32(dst + c, w);
                } else if (mine) {
#pragma unroll
                    for (int i = 0; i < 8; i += 4)
                        *reinterpret_cast<uint4 *>(dst + c + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
                }
            }
            tc_fence_before(); // the next item's first product writes O after this tile's next pfull
            if (p.lse && mine)
                p.lse[row * p.Hq + h] = sees ? (m * p.scale_log2 + log2f(l)) * 0.6931471805599453f : -INFINITY;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&ctl->iempty[slot]);
            if (++slot == pa::SLOTS) {
                slot = 0;
                slot_phase ^= 1u;
            }
        }
    } else {
        if constexpr (S::CTAS == 1)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(pa::REGS_OTHER));
        if (warp == pa::LOAD_WARP) {
            int slot = 0, stage = 0;
            uint32_t slot_phase = 0, phase = 0, q_phase[2] = {0, 0}, tail_phase = 0;
            int issued = 0;
            bool ok = true;
            uint32_t steal_phase = 0;
            int64_t idx = SPLIT ? blockIdx.x / p.split : blockIdx.x;
            int longest = 0;
            for (int j = lane; p.by_length && j < (int)p.B; j += 32)
                longest = max(longest, (int)ctl->top[j]);
            longest = __reduce_max_sync(0xffffffffu, longest);
            PromptShare share = {0, 0};
            while (true) {
                PromptItem it;
                it.valid = idx >= 0 && idx < items ? 1 : 0;
                if (idx >= items) {
                    it.Lq = it.Lk = it.t0 = 0; // the grid is an upper bound of the items: skip
                } else if (it.valid) {
                    const uint32_t unit = (uint32_t)idx / (uint32_t)p.Hkv;
                    int e = 0, left;
                    if (p.by_length) {
                        // items of at least x spans, in all entries
                        auto count = [&](int x) -> uint32_t {
                            int n = 0;
                            for (int j = lane; j < (int)p.B; j += 32)
                                n += max(0, min((int)ctl->top[j] - x + 1, (int)(ctl->first[j + 1] - ctl->first[j])));
                            return __reduce_add_sync(0xffffffffu, (uint32_t)n);
                        };
                        // the item's length: the largest x with more than `unit` items
                        int x = 1, hi = longest;
                        uint32_t longer = 0;
                        while (x < hi) {
                            const int mid = (x + hi + 1) / 2;
                            const uint32_t c = count(mid);
                            if (c > unit) {
                                x = mid;
                            } else {
                                hi = mid - 1;
                                longer = c;
                            }
                        }
                        // the entry: one of those that have an item of this length
                        int skip = (int)(unit - longer);
                        for (int j = 0; j < (int)p.B; j += 32) {
                            const int top = (int)ctl->top[j + lane], n = (int)(ctl->first[j + lane + 1] - ctl->first[j + lane]);
                            const bool has = top - n < x && x <= top;
                            const uint32_t own = __ballot_sync(0xffffffffu, has);
                            const bool it_is = has && __popc(own & ((1u << lane) - 1)) == skip;
                            const uint32_t found = __ballot_sync(0xffffffffu, it_is);
                            if (found) {
                                e = j + __ffs(found) - 1;
                                break;
                            }
                            skip -= __popc(own);
                        }
                        left = (int)ctl->top[e] - x;
                    } else {
                        // the table entry: the last one whose first item is not behind
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            e += __popc(__ballot_sync(0xffffffffu, ctl->first[j * 32 + lane] <= unit));
                        --e;
                        left = (int)(unit - ctl->first[e]);
                    }
                    int64_t b = (int64_t)ctl->order[e] * per;
                    const int64_t end = min(b + per, p.B);
                    int n = 0;
                    for (; b < end; ++b) {
                        prompt_sequence(p, b, it);
                        n = (it.Lq + span - 1) / span;
                        if (left < n)
                            break;
                        left -= n;
                    }
                    if (b == end) // only with offsets that cover rows again and again: nothing to do
                        it.Lq = it.Lk = n = left = 0;
                    it.g = (int)((uint32_t)idx % (uint32_t)p.Hkv);
                    it.t0 = max(0, n - 1 - left) * span; // the last tokens, which see the most, first
                    if (SPLIT) { // this CTA's share of the key blocks
                        const int all = max(prompt_blocks<BN, false>(p, it, 0, share), prompt_blocks<BN, false>(p, it, 1, share));
                        const int rank = (int)cluster_ctarank();
                        share.lo = all * rank / p.split;
                        share.hi = all * (rank + 1) / p.split;
                    }
                }
                if (idx < items) { // the item, or the end
                    if (lane == 0) {
                        ok = wait(&ctl->iempty[slot], slot_phase ^ 1u, 10);
                        if (ok) {
                            ctl->item[slot] = it;
                            if (SPLIT && it.valid)
                                ctl->share = share;
                            mbar_arrive(&ctl->ifull[slot]);
                        }
                    }
                    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                    if (++slot == pa::SLOTS) {
                        slot = 0;
                        slot_phase ^= 1u;
                    }
                    if (!it.valid || !ok)
                        break;
                }
                // ask for the next item now, take the answer once this one's loads are under way
                if (!SPLIT && lane == 0) {
                    fence_proxy_async_smem(); // the last answer has been read
                    mbar_arrive_expect_tx(&ctl->steal, sizeof(uint4));
                    steal_request(&ctl->stolen, &ctl->steal);
                }
                const int nb0 = prompt_blocks<BN, SPLIT>(p, it, 0, share), nb1 = prompt_blocks<BN, SPLIT>(p, it, 1, share);
                const int nb = max(nb0, nb1);
                if (lane == 0) {
                    for (int t = 0; t < 2 && ok; ++t)
                        if (t == 0 ? nb0 : nb1) {
                            ok = wait(&ctl->qempty[t], q_phase[t] ^ 1u, 11);
                            if (!ok)
                                break;
                            q_phase[t] ^= 1u;
                            mbar_arrive_expect_tx(&ctl->qfull[t], (uint32_t)(p.NT * p.G * D * 2));
#pragma unroll
                            for (int hf = 0; hf < S::HALVES; ++hf)
                                tma_load_3d_addr(smem + t * S::Q_BYTES + hf * 16384, &qmap, smem_u32(&ctl->qfull[t]), hf * 64,
                                                 it.g * p.G, it.q0 + it.t0 + t * p.NT);
                        }
                }
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                for (int j = 0; j < nb && ok; ++j)
                    for (int kv = 0; kv < 2 && ok; ++kv) {
                        uint8_t *dst = smem + S::OFF_KV + stage * S::KV_BYTES;
                        const int key0 = ((SPLIT ? share.lo : 0) + j) * BN;
                        const int rows = it.Lk - key0; // keys of this block that are the sequence's own
                        // values behind the sequence's end are cleared: weight 0 times
                        // whatever the neighbour holds must be 0
                        const bool clear = kv == 1 && rows < BN;
                        if (lane == 0) {
                            ok = wait(&ctl->kvempty[stage], phase ^ 1u, 12);
                            if (ok) {
                                uint64_t *bar = clear ? &ctl->tail : &ctl->kvfull[stage];
                                mbar_arrive_expect_tx(bar, S::KV_BYTES);
#pragma unroll
                                for (int hf = 0; hf < S::HALVES; ++hf)
                                    tma_load_3d_addr(dst + hf * 16384, kv ? &vmap : &kmap, smem_u32(bar), hf * 64, it.g,
                                                     it.k0 + key0);
                            }
                        }
                        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                        if (!ok)
                            break;
                        if (clear) {
                            const bool landed = wait(&ctl->tail, tail_phase, 13);
                            tail_phase ^= 1u;
                            __syncwarp();
                            for (int i = rows * 8 + lane; i < BN * 8; i += 32)
#pragma unroll
                                for (int hf = 0; hf < S::HALVES; ++hf)
                                    *reinterpret_cast<uint4 *>(dst + hf * 16384 + i * 16) = make_uint4(0, 0, 0, 0);
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0)
                                mbar_arrive(&ctl->kvfull[stage]);
                            ok = __all_sync(0xffffffffu, landed);
                        }
                        ++issued;
                        if (++stage == S::STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                if (SPLIT) { // one item a cluster
                    idx = -1;
                    if (!ok)
                        break;
                    continue;
                }
                // (also after a timeout: the answer must have landed before the CTA leaves)
                const bool answered = wait(&ctl->steal, steal_phase, 14);
                steal_phase ^= 1u;
                ok = __all_sync(0xffffffffu, ok && answered);
                if (!ok)
                    break;
                idx = steal_answer(&ctl->stolen);
                __syncwarp();
            }
            if (ctl->abort && lane == 0) {
                // leave only when the copies in flight have landed
                for (int t = 0; t < 2; ++t)
                    if (q_phase[t] || issued)
                        (void)mbar_wait(&ctl->qfull[t], q_phase[t] ^ 1u, tmo);
                for (int f = max(0, issued - S::STAGES); f < issued; ++f)
                    (void)mbar_wait(&ctl->kvfull[f % S::STAGES], (uint32_t)(f / S::STAGES) & 1u, tmo);
            }
            __syncwarp();
        } else if (warp == pa::MMA_WARP) {
            constexpr uint32_t idesc_s = idesc_bf16(128, BN, 0), idesc_o = idesc_bf16(128, D, 1);
            const uint32_t base = smem_u32(smem), leader = elect_one();
            int slot = 0, stage = 0;
            uint32_t slot_phase = 0, phase = 0, q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
            // (a CTA that has all 512 columns of TMEM has them from column 0)
            const uint32_t s_col = S::CTAS == 1 ? 0u : __reduce_max_sync(0xffffffffu, tmem), o_col = s_col + S::O_COL;
            // S_t = Q_t K^T: both K-major, 16 elements are 32 bytes, 64 are a half
            auto qk = [&](int t, int st) {
                const uint32_t a = sdesc_lo(base + t * S::Q_BYTES, 16), b = sdesc_lo(base + S::OFF_KV + st * S::KV_BYTES, 16);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k / 4) * 1024 + (k % 4) * 2;
                    umma_ss(leader, s_col + t * BN, a + off, b + off, idesc_s, k != 0 ? 1u : 0u);
                }
                umma_commit_if(leader, &ctl->sfull[t]);
            };
            // O_t += P_t V: P_t is bf16 pairs over S_t; V is
            // MN-major: halves of 64 dimensions 16 KB apart, 16 keys are 2 KB
            auto pv = [&](int t, int st, uint32_t first) {
                const uint32_t b = sdesc_lo(base + S::OFF_KV + st * S::KV_BYTES, 16384);
#pragma unroll
                for (int k = 0; k < BN / 16; ++k)
                    umma_ts(leader, o_col + t * D, s_col + t * BN + k * 8, b + k * 128, idesc_o, k != 0 ? 1u : first ^ 1u);
            };
            // the same for the first `cols` keys of a block (a multiple of 16)
            auto qk_part = [&](int t, int st, int cols) {
                const uint32_t a = sdesc_lo(base + t * S::Q_BYTES, 16), b = sdesc_lo(base + S::OFF_KV + st * S::KV_BYTES, 16);
                const uint32_t idesc = (idesc_s & ~(0x3Fu << 17)) | (uint32_t)(cols >> 3) << 17;
#pragma unroll 1
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k / 4) * 1024 + (k % 4) * 2;
                    umma_ss(leader, s_col + t * BN, a + off, b + off, idesc, k != 0 ? 1u : 0u);
                }
                umma_commit_if(leader, &ctl->sfull[t]);
            };
            auto pv_part = [&](int t, int st, uint32_t first, int cols) {
                const uint32_t b = sdesc_lo(base + S::OFF_KV + st * S::KV_BYTES, 16384);
#pragma unroll 1
                for (int k = 0; k < cols / 16; ++k)
                    umma_ts(leader, o_col + t * D, s_col + t * BN + k * 8, b + k * 128, idesc_o, k != 0 ? 1u : first ^ 1u);
            };
            auto next = [&](int &st, uint32_t &ph) {
                if (++st == S::STAGES) {
                    st = 0;
                    ph ^= 1u;
                }
            };
            auto all_wait = [&](uint64_t *b, uint32_t ph, uint32_t what) -> bool {
                const bool ok = __all_sync(0xffffffffu, wait(b, ph, what));
                tc_fence_after();
                return ok;
            };
            bool ok = true;
            while (ok) {
                ok = all_wait(&ctl->ifull[slot], slot_phase, 20);
                if (!ok)
                    break;
                const PromptItem it = ctl->item[slot];
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&ctl->iempty[slot]);
                if (++slot == pa::SLOTS) {
                    slot = 0;
                    slot_phase ^= 1u;
                }
                if (!__any_sync(0xffffffffu, it.valid))
                    break;
                const int keys[2] = {__reduce_max_sync(0xffffffffu, prompt_most(p, it, 0)),
                                     __reduce_max_sync(0xffffffffu, prompt_most(p, it, 1))};
                int lo = 0, nb[2] = {(keys[0] + BN - 1) / BN, (keys[1] + BN - 1) / BN};
                if constexpr (SPLIT) {
                    lo = __reduce_max_sync(0xffffffffu, ctl->share.lo);
                    const int hi = __reduce_max_sync(0xffffffffu, ctl->share.hi);
                    nb[0] = max(0, min(nb[0], hi) - lo);
                    nb[1] = max(0, min(nb[1], hi) - lo);
                }
                auto cols = [&](int t, int j) -> int { return min(BN, (keys[t] - (lo + j) * BN + 15) & ~15); };
                const int most = max(nb[0], nb[1]);
                if (!most)
                    continue;
                ok = all_wait(&ctl->kvfull[stage], phase, 21);
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (ok && nb[t]) {
                        ok = all_wait(&ctl->qfull[t], q_phase[t], 22);
                        if (!ok)
                            break;
                        q_phase[t] ^= 1u;
                        qk_part(t, stage, cols(t, 0));
                        if (nb[t] == 1)
                            umma_commit_if(leader, &ctl->qempty[t]);
                    }
                if (!ok)
                    break;
                umma_commit_if(leader, &ctl->kvempty[stage]);
                next(stage, phase);
                // any block: what the tiles need of it
                auto any_block = [&](int j) {
                    const int vst = stage;
                    const uint32_t vph = phase;
                    next(stage, phase);
                    const bool more = j + 1 < most; // there is a next block of keys: it is in `stage`
                    ok = all_wait(&ctl->kvfull[vst], vph, 23);
                    if (ok && more)
                        ok = all_wait(&ctl->kvfull[stage], phase, 25);
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        if (ok && j < nb[t]) {
                            ok = all_wait(&ctl->pfull[t], p_phase[t], 24);
                            if (!ok)
                                break;
                            p_phase[t] ^= 1u;
                            pv_part(t, vst, j == 0 ? 1u : 0u, cols(t, j));
                            if (j + 1 < nb[t]) {
                                qk_part(t, stage, cols(t, j + 1));
                                if (j + 2 == nb[t])
                                    umma_commit_if(leader, &ctl->qempty[t]);
                            } else {
                                umma_commit_if(leader, &ctl->ofull[t]);
                            }
                        }
                    if (!ok)
                        return;
                    umma_commit_if(leader, &ctl->kvempty[vst]);
                    if (more) {
                        umma_commit_if(leader, &ctl->kvempty[stage]);
                        next(stage, phase);
                    }
                };
                // a block followed by two more of both tiles, its values in slot V
                // and the next keys in the slot behind: no conditions between the
                // instructions, and every descriptor and barrier a constant
                auto whole_block = [&](auto vslot, int j) {
                    static_assert(S::STAGES == 4, "values lie in slots 1 and 3, and the ring wraps at K only");
                    constexpr int V = decltype(vslot)::value, K = (V + 1) % S::STAGES;
                    const uint32_t vph = phase, kph = phase ^ (K == 0 ? 1u : 0u);
                    ok = all_wait(&ctl->kvfull[V], vph, 23) && all_wait(&ctl->kvfull[K], kph, 25) &&
                         all_wait(&ctl->pfull[0], p_phase[0], 24);
                    if (!ok)
                        return;
                    pv(0, V, j == 0 ? 1u : 0u);
                    qk(0, K);
                    ok = all_wait(&ctl->pfull[1], p_phase[1], 24);
                    if (!ok)
                        return;
                    pv(1, V, j == 0 ? 1u : 0u);
                    qk(1, K);
                    umma_commit_if(leader, &ctl->kvempty[V]);
                    umma_commit_if(leader, &ctl->kvempty[K]);
                    p_phase[0] ^= 1u;
                    p_phase[1] ^= 1u;
                    stage = (V + 2) % S::STAGES;
                    phase = kph;
                };
                int j = 0;
                const int both = min(nb[0], nb[1]) - 2;
                for (; ok && j < both; ++j)
                    if (stage == 1)
                        whole_block(std::integral_constant<int, 1>{}, j);
                    else
                        whole_block(std::integral_constant<int, 3>{}, j);
                for (; ok && j < most; ++j)
                    any_block(j);
            }
            if (__any_sync(0xffffffffu, ctl->abort)) { // every MMA issued finishes before TMEM is freed
                umma_commit_if(leader, &ctl->drain);
                (void)mbar_wait(&ctl->drain, 0, tmo);
            }
            __syncwarp();
        }
    }
    __syncthreads();
    if (warp == pa::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, S::TMEM_COLS);
    }
    if constexpr (SPLIT) {
        // join the cluster's shares: every CTA takes 256 / split rows, four
        // dimensions a thread, and reads the others' shared memory
        cluster_sync();
        const PromptItem it = ctl->item[0];
        if (it.valid && threadIdx.x < 256) {
            const int per = 256 / p.split, row0 = (int)cluster_ctarank() * per;
            const uint32_t stat0 = smem_u32(&ctl->stat[0][0]), out0 = smem_u32(smem + S::OFF_KV);
            for (int u = threadIdx.x; u < per * (D / 4); u += 256) {
                const int row = row0 + u / (D / 4), ch = u % (D / 4), t = row >> 7, r = row & 127;
                const int tok = it.t0 + t * p.NT + r / p.G;
                if (r >= p.NT * p.G || tok >= it.Lq)
                    continue;
                float2 st[pa::MAX_SPLIT];
                float M = -INFINITY;
#pragma unroll
                for (int c = 0; c < pa::MAX_SPLIT; ++c) {
                    st[c] = make_float2(-INFINITY, 0.f);
                    if (c < p.split)
                        st[c] = ld_cluster_f2(mapa_shared(stat0 + row * 8, c));
                    M = fmaxf(M, st[c].x);
                }
                float L = 0.f;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int c = 0; c < pa::MAX_SPLIT; ++c)
                    if (st[c].x != -INFINITY) { // a share that the row sees something of
                        const float w = exp2_approx(st[c].x - M);
                        const float4 x = ld_cluster_f4(mapa_shared(out0 + (row * D + (ch ^ (r & (D / 4 - 1))) * 4) * 4, c));
                        L += st[c].y * w;
                        a.x += x.x * w;
                        a.y += x.y * w;
                        a.z += x.z * w;
                        a.w += x.w * w;
                    }
                const float f = prompt_limit(p, it, tok) > 0 ? 1.f / L : 0.f;
                const int64_t at = (int64_t)it.q0 + tok;
                const int h = it.g * p.G + r % p.G;
                *reinterpret_cast<uint2 *>(p.out + at * p.os + (int64_t)h * D + ch * 4) =
                    make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
                if (p.lse && ch == 0)
                    p.lse[at * p.Hq + h] = f != 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
            }
        }
        cluster_sync(); // no CTA leaves while another reads its shared memory
    }
}

} // namespace tdg

using namespace tdg;
using namespace tdg_host;

extern "C" int tdg_prompt_attention(tdg_symm *h, const tdg_prompt_attention_args *a, void *stream)
{
    if (!h || !a)
        return TDG_ERR_INVALID;
    if (const int drc = check_device(h))
        return drc;
    const int64_t D = a->D, Hq = a->Hq, Hkv = a->Hkv;
    if (a->Tq < 0 || a->Tq > INT32_MAX || a->Tk < 0 || a->Tk > INT32_MAX || a->B < 0 || a->B > 65535 || Hq <= 0 ||
        Hkv <= 0 || Hq > 65535 || Hq % Hkv || Hq / Hkv > 128 || (D != 64 && D != 128) || (a->causal & ~1) ||
        !(a->scale >= 0.f) || isinf(a->scale))
        return TDG_ERR_INVALID;
    if (a->Tq == 0 || a->B == 0)
        return TDG_OK;
    if (!rows_ok(a->q, a->q_stride, Hq * D) || !rows_ok(a->out, a->out_stride, Hq * D) || !a->cu_q || !a->cu_k || !aligned4(a->cu_q) ||
        !aligned4(a->cu_k) || !aligned4(a->lse))
        return TDG_ERR_INVALID;
    if (a->Tk && (!rows_ok(a->k, a->k_stride, Hkv * D) || !rows_ok(a->v, a->v_stride, Hkv * D)))
        return TDG_ERR_INVALID;
    if (rows_clash(a->Tq, a->out, a->out_stride, Hq * D, a->Tq, a->q, a->q_stride, Hq * D) ||
        rows_clash(a->Tq, a->out, a->out_stride, Hq * D, a->Tk, a->k, a->k_stride, Hkv * D) ||
        rows_clash(a->Tq, a->out, a->out_stride, Hq * D, a->Tk, a->v, a->v_stride, Hkv * D))
        return TDG_ERR_INVALID;
    const Range q{a->q, rows_extent(a->Tq, a->q_stride, Hq * D)}, out{a->out, rows_extent(a->Tq, a->out_stride, Hq * D)};
    const Range k{a->k, rows_extent(a->Tk, a->k_stride, Hkv * D)}, v{a->v, rows_extent(a->Tk, a->v_stride, Hkv * D)};
    const Range lse{a->lse, (uint64_t)a->Tq * Hq * 4}, cu_q{a->cu_q, (uint64_t)(a->B + 1) * 4}, cu_k{a->cu_k, (uint64_t)(a->B + 1) * 4};
    if (ranges_overlap({lse}, {q, k, v, out}) || ranges_overlap({out, lse}, {cu_q, cu_k}))
        return TDG_ERR_INVALID;
    PromptParams p;
    memset(&p, 0, sizeof p);
    p.status = h->status;
    p.G = (int)(Hq / Hkv);
    p.NT = 128 / p.G;
    // items: at most one per 2 NT tokens and one more per sequence, of every key head
    const int64_t items = (a->Tq / (2 * p.NT) + a->B) * Hkv;
    if (items > INT32_MAX)
        return TDG_ERR_INVALID;
    p.epoch = next_epoch(h);
    p.timeout_ns = timeout_or_default(0);
    p.Tq = a->Tq;
    p.Tk = a->Tk;
    p.B = a->B;
    p.os = a->out_stride;
    p.Hq = (int)Hq;
    p.Hkv = (int)Hkv;
    p.causal = a->causal;
    p.scale_log2 = (a->scale > 0.f ? a->scale : 1.0f / sqrtf((float)D)) * 1.4426950408889634f;
    p.out = static_cast<__nv_bfloat16 *>(a->out);
    p.out32 = (reinterpret_cast<uintptr_t>(a->out) & 31u) == 0 && a->out_stride % 16 == 0;
    p.lse = a->lse;
    p.cu_q = a->cu_q;
    p.cu_k = a->cu_k;
    const bool two = D == 64 && items >= (int64_t)pa::TWO_CTAS_ITEMS * h->sm_count;
    const uint32_t bn = two ? 64 : 128;
    p.by_length = a->B > 1 && a->B <= pa::CHUNKS && items > h->sm_count && a->Tk * Hkv * D * 4 < pa::BY_LENGTH_BYTES;
    CUtensorMap qm, km, vm;
    // rows of heads: {D, heads, rows}; a box is 64 dimensions of a tile's heads and tokens
    if (!map_bf16_3d(&qm, a->q, D, Hq, a->Tq, D * 2, a->q_stride * 2, 64, (uint32_t)p.G, (uint32_t)p.NT))
        return TDG_ERR_CUDA;
    km = vm = qm; // no keys: nothing is loaded through them
    if (a->Tk && (!map_bf16_3d(&km, a->k, D, Hkv, a->Tk, D * 2, a->k_stride * 2, 64, 1, bn) ||
                  !map_bf16_3d(&vm, a->v, D, Hkv, a->Tk, D * 2, a->v_stride * 2, 64, 1, bn)))
        return TDG_ERR_CUDA;
    // Few items of many keys: up to 8 CTAs share an item's keys, as many as the
    // SMs allow, if an average sequence's item is spared 8 blocks by it (a block
    // is 1.2 us of an item, the cluster and its join cost 5 to 6 us).
    const int64_t room = h->sm_count / items, blocks = a->Tk / a->B / 128;
    p.split = room >= 8 ? 8 : room >= 4 ? 4 : room >= 2 ? 2 : 1;
    if (blocks - blocks / p.split < 8)
        p.split = 1;
    const bool split = p.split > 1;
    const void *fn = D == 128 ? (split ? reinterpret_cast<const void *>(&prompt_kernel<128, 128, true>)
                                       : reinterpret_cast<const void *>(&prompt_kernel<128, 128, false>))
                     : two    ? reinterpret_cast<const void *>(&prompt_kernel<64, 64, false>)
                     : split  ? reinterpret_cast<const void *>(&prompt_kernel<64, 128, true>)
                              : reinterpret_cast<const void *>(&prompt_kernel<64, 128, false>);
    const int smem = D == 128 ? prompt_smem<128, 128>() : two ? prompt_smem<64, 64>() : prompt_smem<64, 128>();
    if (const cudaError_t e = set_smem(fn, smem); e != cudaSuccess)
        return cuda_err(e, "prompt attention smem");
    void *args[] = {&p, &qm, &km, &vm};
    const int threads = two ? pa::Shape<64, 64>::THREADS : pa::Shape<64, 128>::THREADS;
    return cuda_err(launch(fn, dim3((unsigned)(items * p.split)), dim3(threads), smem, static_cast<cudaStream_t>(stream), args, false,
                           p.split, true),
                    "prompt attention launch");
}
