// One decoding step over the latent KV cache: mla_prolog_attend_cache.
#include <cmath>
#include <cstdint>

#include "attend.cuh"
#include "ptx.cuh"

namespace mlap {
namespace {

struct CacheParams {
    const uint16_t* q;
    const uint16_t* cache;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* seqs;
    const int32_t* shared;
    uint16_t* out;
    float* lse;
    int32_t* status;
    int B, H, Lkv, C, page_size, table_rows, max_pages;
    int64_t num_pages;
    float scale;
};

__device__ __forceinline__ float bf16f(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// One warp per (sequence, head): each lane scores a key of 32, then the lanes
// share the columns of c_kv.
__global__ void __launch_bounds__(128) mla_attend_cache_kernel(CacheParams p) {
    const int lane = threadIdx.x & 31;
    const int r = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (r >= p.B * p.H) return;
    const int b = r / p.H;
    int bits = 0, n = 0;
    const int s = p.seqs ? p.seqs[b] : b;
    const int cap = p.max_pages * p.page_size;
    if (s < 0 || s >= p.table_rows) {
        bits = kStatusSeqRange;
    } else {
        n = p.lens[s];
        if (n < 0 || n > cap) bits = kStatusSeqRange, n = n < 0 ? 0 : cap;
    }
    const uint16_t* q = p.q + static_cast<int64_t>(r) * p.C;
    float m = -INFINITY, l = 0.f, acc[16] = {};
    for (int j0 = 0; j0 < n; j0 += 32) {
        const int j = j0 + lane;
        float x = 0.f;
        const uint16_t* row = nullptr;
        if (j < n) {
            const int page = p.table[static_cast<int64_t>(s) * p.max_pages + j / p.page_size];
            if (page < 0 || page >= p.num_pages) bits |= kStatusPageRange;
            else row = p.cache + (static_cast<int64_t>(page) * p.page_size + j % p.page_size) * p.C;
            if (row)
                for (int d = 0; d < p.C; ++d) x = fmaf(bf16f(q[d]), bf16f(row[d]), x);
        }
        x = j < n ? x * p.scale : -INFINITY;
        float mx = x;
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
        const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.f : mn;
        const float keep = expf(m - ref), e = j < n ? expf(x - ref) : 0.f;
        float sum = e;
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        l = l * keep + sum;
        m = mn;
        for (int i = 0; i < 16; ++i) acc[i] *= keep;
        for (int i = 0; i < 32 && j0 + i < n; ++i) {
            const float w = __shfl_sync(~0u, e, i);
            const uint16_t* v = reinterpret_cast<const uint16_t*>(
                __shfl_sync(~0u, reinterpret_cast<unsigned long long>(row), i));
            if (!v) continue;
            for (int c = 0; c < 16; ++c)
                if (c * 32 + lane < p.Lkv) acc[c] = fmaf(w, bf16f(v[c * 32 + lane]), acc[c]);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int c = 0; c < 16; ++c)
        if (c * 32 + lane < p.Lkv)
            p.out[static_cast<int64_t>(r) * p.Lkv + c * 32 + lane] = static_cast<uint16_t>(pack_bf16x2(acc[c] * inv, 0.f) & 0xFFFFu);
    if (lane == 0 && p.lse) p.lse[r] = l == 0.f ? -INFINITY : m + logf(l);
    raise_status(p.status, bits);
}

int check_cache_dims(const mla_prolog_cache_dims& d) {
    const int64_t most = INT32_MAX;
    if (d.batch < 0 || d.num_heads < 1 || static_cast<int64_t>(d.batch) * d.num_heads > (1 << 24) ||
        d.kv_lora_rank < 16 || d.kv_lora_rank > 512 || d.kv_lora_rank % 16 || d.rope_dim < 0 || d.rope_dim > 128 ||
        d.rope_dim % 16 || d.kv_lora_rank + d.rope_dim > 576)
        return MLA_ERR_UNSUPPORTED_DIMS;
    if (d.page_size < 16 || d.page_size % 16 || d.table_rows < 0 || d.max_pages < 1 || d.num_pages < 0 ||
        d.num_pages > most / d.page_size || static_cast<int64_t>(d.max_pages) * d.page_size > (1 << 30) ||
        !(d.scale > 0.f) || !std::isfinite(d.scale))
        return MLA_ERR_UNSUPPORTED_DIMS;
    return MLA_OK;
}

}  // namespace
}  // namespace mlap

using namespace mlap;

extern "C" {

int mla_prolog_attend_cache_workspace(const mla_prolog_cache_dims* d, size_t* bytes) {
    if (!d || !bytes) return MLA_ERR_INVALID_ARG;
    *bytes = 0;
    const int rc = check_cache_dims(*d);
    if (rc != MLA_OK) return rc;
    *bytes = 16;
    return MLA_OK;
}

int mla_prolog_attend_cache(const mla_prolog_cache_dims* d, const void* q, const void* kv_cache,
                            const int32_t* page_table, const int32_t* seq_lens, const int32_t* seqs,
                            const int32_t* shared_len, void* out, float* lse, void* workspace,
                            size_t workspace_bytes, int32_t* status, void* stream) {
    if (!d) return MLA_ERR_INVALID_ARG;
    int rc = check_cache_dims(*d);
    if (rc != MLA_OK) return rc;
    if (!seqs && d->table_rows < d->batch) return MLA_ERR_INVALID_ARG;
    if (d->batch == 0) return MLA_OK;
    if (!ptr_ok(q, 16) || !ptr_ok(out, 16) || (d->num_pages && !ptr_ok(kv_cache, 16))) return MLA_ERR_INVALID_ARG;
    if (d->table_rows && (!ptr_ok(page_table, 4) || !ptr_ok(seq_lens, 4))) return MLA_ERR_INVALID_ARG;
    if ((seqs && !ptr_ok(seqs, 4)) || (shared_len && !ptr_ok(shared_len, 4)) || (lse && !ptr_ok(lse, 4)) ||
        (status && !ptr_ok(status, 4)))
        return MLA_ERR_INVALID_ARG;
    int sms;
    if ((rc = current_sm103(&sms)) != MLA_OK) return rc;
    size_t need = 0;
    if ((rc = mla_prolog_attend_cache_workspace(d, &need)) != MLA_OK) return rc;
    if (!ptr_ok(workspace, 16) || workspace_bytes < need) return MLA_ERR_INVALID_ARG;
    CacheParams p{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(kv_cache), page_table, seq_lens, seqs,
                  shared_len, static_cast<uint16_t*>(out), lse, status, d->batch, d->num_heads, d->kv_lora_rank,
                  d->kv_lora_rank + d->rope_dim, d->page_size, d->table_rows, d->max_pages, d->num_pages, d->scale};
    mla_attend_cache_kernel<<<(d->batch * d->num_heads + 3) / 4, 128, 0, static_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MLA_OK : report_cuda(e, "launch mla_attend_cache_kernel");
}

}  // extern "C"
