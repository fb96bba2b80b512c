// tdg_prompt.cu -- attention over whole prompts packed one after another:
// softmax(scale Q K^T) V per sequence, causal from the last key back.
//
// One warp per (query row, head): a lane holds D/32 of the head's elements and
// the warp keeps a running maximum, sum and output in float32.
#include "tdg_paged.cuh"

namespace tdg {

struct PromptParams {
    DevStatus *status;
    uint32_t epoch;
    int64_t Tq, Tk, B, qs, ks, vs, os;
    int Hq, Hkv, G, causal;
    float scale;
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *out;
    float *lse;
    const int32_t *cu_q, *cu_k;
};

// Rows of sequence b; false (and a report by one thread) when the offsets are
// out of order or range.
__device__ __forceinline__ bool prompt_sequence(const PromptParams &p, int64_t b, bool report, int64_t &q0, int &Lq,
                                                int64_t &k0, int &Lk)
{
    const int64_t qa = p.cu_q[b], qb = p.cu_q[b + 1], ka = p.cu_k[b], kb = p.cu_k[b + 1];
    const bool ok = qa >= 0 && qb >= qa && qb <= p.Tq && ka >= 0 && kb >= ka && kb <= p.Tk;
    if (!ok && report)
        report_fault(p.status, TDG_ERR_DEVICE, TDG_WHERE_CU, (uint32_t)b, p.epoch);
    q0 = qa;
    k0 = ka;
    Lq = ok ? (int)(qb - qa) : 0;
    Lk = ok ? (int)(kb - ka) : 0;
    return ok;
}

template <int D>
__global__ void __launch_bounds__(128) prompt_kernel(const __grid_constant__ PromptParams p)
{
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.x, g = h / p.G;
    int64_t q0, k0;
    int Lq, Lk;
    prompt_sequence(p, blockIdx.y, threadIdx.x == 0, q0, Lq, k0, Lk);
    for (int i = blockIdx.z * 4 + (threadIdx.x >> 5); i < Lq; i += gridDim.z * 4) {
        const int n = p.causal ? min(Lk, i + Lk - Lq + 1) : Lk;
        float q[N], o[N], m = -INFINITY, l = 0.f;
        for (int x = 0; x < N; ++x) {
            q[x] = __bfloat162float(p.q[(q0 + i) * p.qs + (int64_t)h * D + lane * N + x]) * p.scale;
            o[x] = 0.f;
        }
        for (int j = 0; j < n; ++j) {
            float s = 0.f;
            for (int x = 0; x < N; ++x)
                s += q[x] * __bfloat162float(p.k[(k0 + j) * p.ks + (int64_t)g * D + lane * N + x]);
            for (int x = 16; x; x >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, x);
            const float mn = fmaxf(m, s), ms = mn == -INFINITY ? 0.f : mn;
            const float al = expf(m - ms), w = expf(s - ms);
            m = mn;
            l = l * al + w;
            for (int x = 0; x < N; ++x)
                o[x] = o[x] * al + w * __bfloat162float(p.v[(k0 + j) * p.vs + (int64_t)g * D + lane * N + x]);
        }
        for (int x = 0; x < N; ++x)
            p.out[(q0 + i) * p.os + (int64_t)h * D + lane * N + x] = __float2bfloat16_rn(n > 0 ? o[x] / l : 0.f);
        if (p.lse && lane == 0)
            p.lse[(q0 + i) * p.Hq + h] = n > 0 ? m + logf(l) : -INFINITY;
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
    PromptParams p;
    memset(&p, 0, sizeof p);
    p.status = h->status;
    p.epoch = next_epoch(h);
    p.Tq = a->Tq;
    p.Tk = a->Tk;
    p.B = a->B;
    p.qs = a->q_stride;
    p.ks = a->k_stride;
    p.vs = a->v_stride;
    p.os = a->out_stride;
    p.Hq = (int)Hq;
    p.Hkv = (int)Hkv;
    p.G = (int)(Hq / Hkv);
    p.causal = a->causal;
    p.scale = a->scale > 0.f ? a->scale : 1.0f / sqrtf((float)D);
    p.q = static_cast<const __nv_bfloat16 *>(a->q);
    p.k = static_cast<const __nv_bfloat16 *>(a->k);
    p.v = static_cast<const __nv_bfloat16 *>(a->v);
    p.out = static_cast<__nv_bfloat16 *>(a->out);
    p.lse = a->lse;
    p.cu_q = a->cu_q;
    p.cu_k = a->cu_k;
    const void *fn = D == 128 ? reinterpret_cast<const void *>(&prompt_kernel<128>) : reinterpret_cast<const void *>(&prompt_kernel<64>);
    void *args[] = {&p};
    const unsigned z = (unsigned)(a->Tq < 1024 ? (a->Tq + 3) / 4 : 256);
    return cuda_err(launch(fn, dim3((unsigned)Hq, (unsigned)a->B, z), dim3(128), 0, static_cast<cudaStream_t>(stream), args, false),
                    "prompt attention launch");
}
