// Attention over whole prompts: mla_prolog_attend_prompt.
#include <cmath>
#include <cstdint>

#include "attend.cuh"
#include "ptx.cuh"

namespace mlap {
namespace {

struct PromptParams {
    const void* q;
    const float* q_scale;
    const uint16_t* k;
    const uint16_t* v;
    const int32_t* cu_q;
    const int32_t* cu_k;
    uint16_t* out;
    float* lse;
    int32_t* status;
    int Tq, Tk, B, H, Hk, Dqk, Dv;
    float scale;
    int causal, q_int8, q_per_head;
};

__device__ __forceinline__ float bf16f(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// One warp per (row, head): each lane scores a key of 32, then the lanes share
// the columns of v.
__global__ void __launch_bounds__(128) mla_attend_prompt_kernel(PromptParams p) {
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5), h = blockIdx.y, hk = h / (p.H / p.Hk);
    if (row >= p.Tq) return;
    int bits = 0, found = -1, q0 = 0, q1 = 0;
    for (int s = 0; s < p.B; ++s) {
        const int a = p.cu_q[s], b = p.cu_q[s + 1];
        const int ka = p.cu_k[s], kb = p.cu_k[s + 1];
        if (a < 0 || b < a || b > p.Tq || ka < 0 || kb < ka || kb > p.Tk) bits = kStatusSeqRange;
        const int lo = max(a, 0), hi = min(b, p.Tq);
        if (found < 0 && row >= lo && row < hi) found = s, q0 = lo, q1 = hi;
    }
    if (lane == 0 && row == 0 && h == 0) raise_status(p.status, bits);
    if (found < 0) return;
    const int k0 = max(p.cu_k[found], 0), k1 = max(k0, min(p.cu_k[found + 1], p.Tk));
    int n = k1 - k0;
    if (p.causal) n = min(n, row - q0 + 1 + (k1 - k0) - (q1 - q0));
    float c = p.scale;
    if (p.q_int8) c *= p.q_scale[p.q_per_head ? static_cast<int64_t>(row) * p.H + h : row];
    const int64_t qat = (static_cast<int64_t>(row) * p.H + h) * p.Dqk;
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < n; j0 += 32) {
        const int j = j0 + lane;
        float s = 0.f;
        if (j < n) {
            const uint16_t* k = p.k + (static_cast<int64_t>(k0 + j) * p.Hk + hk) * p.Dqk;
            for (int d = 0; d < p.Dqk; ++d) {
                const float qd = p.q_int8 ? static_cast<float>(static_cast<const int8_t*>(p.q)[qat + d])
                                          : bf16f(static_cast<const uint16_t*>(p.q)[qat + d]);
                s = fmaf(qd, bf16f(k[d]), s);
            }
        }
        s = j < n ? s * c : -INFINITY;
        float mx = s;
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
        const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.f : mn;
        const float keep = expf(m - ref), e = j < n ? expf(s - ref) : 0.f;
        float sum = e;
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        l = l * keep + sum;
        m = mn;
        for (int x = 0; x < 4; ++x) acc[x] *= keep;
        for (int i = 0; i < 32 && j0 + i < n; ++i) {
            const float w = __shfl_sync(~0u, e, i);
            const uint16_t* v = p.v + (static_cast<int64_t>(k0 + j0 + i) * p.Hk + hk) * p.Dv;
            for (int x = 0; x < 4; ++x)
                if (x * 32 + lane < p.Dv) acc[x] = fmaf(w, bf16f(v[x * 32 + lane]), acc[x]);
        }
    }
    const int64_t at = static_cast<int64_t>(row) * p.H + h;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int x = 0; x < 4; ++x)
        if (x * 32 + lane < p.Dv)
            p.out[at * p.Dv + x * 32 + lane] = static_cast<uint16_t>(pack_bf16x2(acc[x] * inv, 0.f) & 0xFFFFu);
    if (lane == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace
}  // namespace mlap

using namespace mlap;

extern "C" int mla_prolog_attend_prompt(const mla_prolog_prompt_dims* d, const void* q, const float* q_scale,
                                        const void* k, const void* v, const int32_t* cu_q, const int32_t* cu_k,
                                        void* out, float* lse, int32_t* status, void* stream) {
    if (!d) return MLA_ERR_INVALID_ARG;
    const uint32_t known = MLA_PROMPT_CAUSAL | MLA_PROMPT_Q_INT8 | MLA_PROMPT_Q_SCALE_PER_HEAD;
    const bool int8 = d->flags & MLA_PROMPT_Q_INT8, per_head = d->flags & MLA_PROMPT_Q_SCALE_PER_HEAD;
    if ((d->flags & ~known) || (per_head && !int8)) return MLA_ERR_INVALID_ARG;
    if (d->Tq < 0 || d->Tk < 0 || d->sequences < 0 || d->kv_heads < 1 || d->num_heads < 1 ||
        d->num_heads % d->kv_heads || d->num_heads > 65535 || d->qk_dim < 16 || d->qk_dim > 256 || d->qk_dim % 16 ||
        d->v_dim < 16 || d->v_dim > 128 || d->v_dim % 16 || !(d->scale > 0.f) || !std::isfinite(d->scale))
        return MLA_ERR_UNSUPPORTED_DIMS;
    if (int8 ? !ptr_ok(q_scale, 4) : q_scale != nullptr) return MLA_ERR_INVALID_ARG;
    if (d->Tq == 0 || d->sequences == 0) return MLA_OK;
    if (!ptr_ok(q, 16) || !ptr_ok(out, 16) || !ptr_ok(cu_q, 4) || !ptr_ok(cu_k, 4)) return MLA_ERR_INVALID_ARG;
    if (d->Tk && (!ptr_ok(k, 16) || !ptr_ok(v, 16))) return MLA_ERR_INVALID_ARG;
    if ((lse && !ptr_ok(lse, 4)) || (status && !ptr_ok(status, 4))) return MLA_ERR_INVALID_ARG;
    int sms;
    const int rc = current_sm103(&sms);
    if (rc != MLA_OK) return rc;
    PromptParams p{q, q_scale, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), cu_q, cu_k,
                   static_cast<uint16_t*>(out), lse, status, d->Tq, d->Tk, d->sequences, d->num_heads, d->kv_heads,
                   d->qk_dim, d->v_dim, d->scale, (d->flags & MLA_PROMPT_CAUSAL) != 0, int8, per_head};
    mla_attend_prompt_kernel<<<dim3((d->Tq + 3) / 4, d->num_heads), 128, 0, static_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MLA_OK : report_cuda(e, "launch mla_attend_prompt_kernel");
}
