// Writing the latent cache in 8 bits and reading it back: mla_prolog_cache8_write
// and mla_prolog_cache8_read (the page format: cache8.cuh).
//
// Write.  The rows of a call that lie in one block of a page are a run:
// consecutive entries with consecutive slots.  A run's scale is the least power
// of two 2^k with |x| <= 448 * 2^k for all its finite values; a run that does
// not begin with the block's first row keeps at least the stored scale, and
// where it needs a larger one, the rows before it are moved to that: a change
// of exponent, exact but for subnormal codes.
//
// Read.  Codes times 2^k, which BF16 holds exactly (4 significant bits).
#include <algorithm>
#include <cstdint>

#include "cache8.cuh"
#include "ptx.cuh"

namespace mlap {
namespace {

constexpr int kMaxBlock = 128;
constexpr int kMaxWindow = 64;
constexpr int kMaxEntries = kMaxWindow + 2 * kMaxBlock;
constexpr int kRowChunks = 72;                // 8 columns each
constexpr int kLaneChunks = (kRowChunks + 31) / 32;
constexpr int kReadWarps = 8, kReadRows = 4;

// 8 codes of 8 BF16 values (four pairs), times 2^-k.
__device__ __forceinline__ uint2 quantised8(const uint4& v, uint64_t down) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        upk2(mul2(pk2(bf16_lo(w[i]), bf16_hi(w[i])), down), a, b);
        c[i] = e4m3x2(a, b);
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Four codes times `by` (a power of two), rounded anew.
__device__ __forceinline__ uint32_t rescaled4(uint32_t codes, float by) {
    float a, b, c, d;
    f32_of_f16x2(f16x2_of_e4m3x2(codes), a, b);
    f32_of_f16x2(f16x2_of_e4m3x2(codes >> 16), c, d);
    return e4m3x2(a * by, b * by) | e4m3x2(c * by, d * by) << 16;
}

struct WriteShared {
    // the window's tokens, a block before them and a block behind: entry i is token first - block + i
    int32_t slot[kMaxEntries];                  // -1: nothing is written
    uint32_t linked[(kMaxEntries + 31) / 32];   // bit i: entry i + 1 goes on with the run of entry i
    uint16_t start[kMaxEntries];                // first entry of the run (as far as the entries go)
    int32_t need[kMaxEntries];                  // of a run, at its first entry
    int32_t back, ahead;                        // entries before and behind the window that belong to its first and last run
    int32_t jobs;
    int32_t job_slot[kMaxWindow], job_rows[kMaxWindow], job_by[kMaxWindow];
};

// Entries before i, and from i on, that a row of set bits joins to it: at most `most`.
__device__ __forceinline__ int linked_before(const uint32_t* bits, int i, int most) {
    int n = 0;
    while (n < most && i > 0) {  // the bits below i in its word
        const int in = (i - 1) & 31;
        const uint32_t gaps = ~bits[(i - 1) >> 5] << (31 - in);
        const int run = gaps ? __clz(gaps) : in + 1;
        n += run;
        i -= run;
        if (run < in + 1) break;
    }
    return n < most ? n : most;
}
__device__ __forceinline__ int linked_behind(const uint32_t* bits, int i, int most) {
    int n = 0;
    while (n < most) {
        const int in = i & 31;
        const uint32_t gaps = ~bits[i >> 5] >> in;
        const int run = gaps ? __ffs(gaps) - 1 : 32 - in;
        n += run;
        i += run;
        if (run < 32 - in) break;
    }
    return n < most ? n : most;
}

// A CTA writes a window of tokens, a warp kRows of them, which stay in registers between the maximum and the rounding:
// each row is read once.  (Rows of a run that another window holds are read for their maximum alone, one after another.
// Windows are 8 to 64 rows, by the dispatch below, so that in blocks of 128 every window reads rows of others: 4096 tokens
// in blocks of 16, 64 and 128 take 2.9, 4.8 and 7.1 us, 16384 take 6.9, 6.5 and 11.)  It moves 3 bytes per element: 262144
// rows of 576 in 77 us, 5.9 TB/s (87% of a copy's rate); 16384 in 6.5; few tokens by the launch and three dependent reads
// (slot, scale, row): 2.0 us for one.
template <int kWriteWarps, int kRows>
__global__ void __launch_bounds__(kWriteWarps * 32, kWriteWarps == 8 && kRows < 8 ? 3 : 2)
    mla_cache8_write_kernel(const Cache8 c, const Divide by_page, const Divide by_block, const uint16_t* rows, const int32_t* slots,
                            int T, int32_t* status) {
    constexpr int kWindow = kWriteWarps * kRows;
    __shared__ WriteShared sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chunks = c.C / 8;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kWindow;
    const int num_slots = c.num_pages * c.page_size, block = c.block, entries = kWindow + 2 * block;
    pdl_launch_dependents();
    pdl_wait();
    uint4 v[kRows][kLaneChunks];
    auto load = [&](int64_t t, uint4 (&x)[kLaneChunks]) {
        const uint4* row = reinterpret_cast<const uint4*>(rows + t * c.C);
#pragma unroll
        for (int k = 0; k < kLaneChunks; ++k) {
            x[k] = make_uint4(0, 0, 0, 0);
            if (k * 32 + lane < chunks) x[k] = row[k * 32 + lane];
        }
    };
    auto need = [&](const uint4 (&x)[kLaneChunks]) {
        uint32_t most = 0;
#pragma unroll
        for (int k = 0; k < kLaneChunks; ++k) most = max2(max2(max2(max2(most, x[k].x), x[k].y), x[k].z), x[k].w);
        uint32_t top = __reduce_max_sync(~0u, max(most & 0xffffu, most >> 16));
        if (top >= 0x7f80u) {  // (rare) infinities and NaN are left out: six instructions more per word
            most = 0;
#pragma unroll 1
            for (int k = 0; k < kLaneChunks; ++k) {
                const uint4 w = k == 0 ? x[0] : k == 1 ? x[1] : x[2];
                most = max_finite2(max_finite2(max_finite2(max_finite2(most, w.x), w.y), w.z), w.w);
            }
            top = __reduce_max_sync(~0u, max(most & 0xffffu, most >> 16));
        }
        return need_exp(top);
    };
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int64_t t = first + warp * kRows + r;
        if (t < T) load(t, v[r]);
    }
    // slots, and which of them go on with the run of the one before
    int bits = 0;
    for (int i = threadIdx.x; i - lane < entries; i += kWriteWarps * 32) {
        const int64_t t = first - block + i;
        int s = i < entries && t >= 0 && t < T ? slots[t] : -1, next = i + 1 < entries && t + 1 >= 0 && t + 1 < T ? slots[t + 1] : -1;
        if (s >= num_slots) {
            if (i >= block && i < block + kWindow) bits |= MLA_STATUS_SLOT_RANGE;
            s = -1;
        }
        if (i < entries) sh.slot[i] = s < 0 ? -1 : s, sh.need[i] = kLowExp;
        const bool link = s >= 0 && next == s + 1 && next < num_slots && next != by_block(next) * block;
        const uint32_t word = __ballot_sync(~0u, link);
        if (lane == 0 && i < kMaxEntries) sh.linked[i >> 5] = word;
    }
    if (threadIdx.x == 0) sh.jobs = 0;
    __syncthreads();
    if (threadIdx.x == kWriteWarps * 32 - 1) sh.back = linked_before(sh.linked, block, block - 1);
    if (threadIdx.x == kWriteWarps * 32 - 33) sh.ahead = linked_behind(sh.linked, block + kWindow - 1, block - 1);
    for (int i = threadIdx.x; i < entries; i += kWriteWarps * 32) sh.start[i] = i - linked_before(sh.linked, i, i < block - 1 ? i : block - 1);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int i = block + warp * kRows + r;
        if (first - block + i >= T) break;
        const int k = need(v[r]);
        if (lane == 0 && sh.slot[i] >= 0) atomicMax(&sh.need[sh.start[i]], k);
    }
    const int back = sh.back, both = back + sh.ahead;
    for (int e = warp; e < both; e += kWriteWarps) {
        const int i = e < back ? block - 1 - e : block + kWindow + e - back;
        uint4 x[kLaneChunks];
        load(first - block + i, x);
        const int k = need(x);
        if (lane == 0) atomicMax(&sh.need[sh.start[i]], k);
    }
    __syncthreads();
    // each lane finds the place and scale of one of the rows
    int64_t place = -1;
    int k = 0;
    const int mine = block + warp * kRows + lane % kRows;
    if (first - block + mine < T && sh.slot[mine] >= 0) {
        const int slot = sh.slot[mine], start = sh.start[mine], before = mine - start;
        const int page = by_page(slot), row = slot - page * c.page_size, unit = by_block(row), in = row - unit * block;
        place = page * c.page_bytes + static_cast<int64_t>(row) * c.C;
        uint8_t* const exp_at = c.pages + page * c.page_bytes + static_cast<int64_t>(c.page_size) * c.C + unit;
        k = sh.need[start];
        if (in > before) {  // rows before the run: their scale holds
            // (Another window of this run may have stored the new one by now: the larger of the two is the same.)
            const int old = scale_exp(*const_cast<volatile uint8_t*>(exp_at));
            if (before == 0 && k > old && lane < kRows) {
                const int j = atomicAdd(&sh.jobs, 1);
                sh.job_slot[j] = slot - in;
                sh.job_rows[j] = in;
                sh.job_by[j] = old - k;
            }
            k = max(k, old);
        }
        if (before == 0 && lane < kRows) *exp_at = static_cast<uint8_t>(k + kExpBias);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int64_t at = kRows == 1 ? place : __shfl_sync(~0u, place, r);
        const float by = pow2(-(kRows == 1 ? k : __shfl_sync(~0u, k, r)));
        if (at < 0) continue;  // (the same in the whole warp)
        const uint64_t down = pk2(by, by);
        uint2* const to = reinterpret_cast<uint2*>(c.pages + at);
#pragma unroll
        for (int n = 0; n < kLaneChunks; ++n)
            if (n * 32 + lane < chunks) to[n * 32 + lane] = quantised8(v[r][n], down);
    }
    __syncthreads();
    for (int j = 0; j < sh.jobs; ++j) {
        const int slot = sh.job_slot[j], page = by_page(slot);
        uint4* const at = reinterpret_cast<uint4*>(c.pages + page * c.page_bytes + static_cast<int64_t>(slot - page * c.page_size) * c.C);
        // (2^-120 at the least; below 2^-18 every code becomes 0)
        const float by = pow2(sh.job_by[j]);
        for (int u = threadIdx.x; u < sh.job_rows[j] * (c.C / 16); u += kWriteWarps * 32) {
            uint4 x = at[u];
            x.x = rescaled4(x.x, by), x.y = rescaled4(x.y, by), x.z = rescaled4(x.z, by), x.w = rescaled4(x.w, by);
            at[u] = x;
        }
    }
    raise_status(status, bits);
}

struct ReadParams {
    Cache8 c;
    Divide by_page, by_block;
    const int32_t *table, *seqs, *starts, *cu;
    int table_rows, max_pages, n, T;
    uint16_t* out;
    int32_t* status;
};

// A warp has kReadRows rows: a lane finds each one's place, then all lanes take eight columns at a time of the rows
// together, every load on its way before the first store.  It moves 3 bytes per element: 159k rows of 576 in 44 us, 6.3
// TB/s (93% of a copy's rate; a row at a time 72 us); 10k in 5.4 us, of which the floor is 3.2 and the rest the launch and
// four dependent reads (cu, table, scale, row).
__global__ void __launch_bounds__(kReadWarps * 32) mla_cache8_read_kernel(const __grid_constant__ ReadParams p) {
    const int lane = threadIdx.x & 31, chunks = p.c.C / 8;
    const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * kReadWarps + (threadIdx.x >> 5)) * kReadRows;
    pdl_launch_dependents();
    pdl_wait();
    int bits = 0;
    int64_t from = -1;   // offset of the row in the cache; -1: zeros, -2: nobody's row
    int exponent = 0;
    const int64_t mine = r0 + lane;
    if (lane < kReadRows) {
        from = -2;
        if (mine < p.T) {
            // the last sequence that starts at or before the row
            int a = 0, b = p.n;
            while (b - a > 1) {
                const int m = (a + b) >> 1;
                if (p.cu[m] <= mine) a = m;
                else b = m;
            }
            const int64_t at = mine - p.cu[a];
            if (at >= 0 && mine < p.cu[a + 1]) {
                const int64_t token = at + (p.starts ? p.starts[a] : 0);
                const int seq = p.seqs ? p.seqs[a] : a;
                from = -1;
                if (seq < 0 || seq >= p.table_rows || token < 0 || token >= static_cast<int64_t>(p.max_pages) * p.c.page_size) {
                    bits = kStatusSeqRange;
                } else {
                    const int nth = p.by_page(static_cast<int>(token)), row = static_cast<int>(token) - nth * p.c.page_size;
                    const int page = p.table[static_cast<int64_t>(seq) * p.max_pages + nth];
                    if (page < 0 || page >= p.c.num_pages) {
                        bits = kStatusPageRange;
                    } else {
                        from = page * p.c.page_bytes + static_cast<int64_t>(row) * p.c.C;
                        exponent = p.c.pages[page * p.c.page_bytes + static_cast<int64_t>(p.c.page_size) * p.c.C + p.by_block(row)];
                    }
                }
            }
        }
    }
    uint2 x[kLaneChunks * kReadRows];
    uint32_t has = 0;    // bit n: the lane's n-th eight columns are a sequence's
#pragma unroll
    for (int n = 0; n < kLaneChunks * kReadRows; ++n) {
        const int i = n * 32 + lane, row = (i >= chunks) + (i >= 2 * chunks) + (i >= 3 * chunks);
        const int64_t at = __shfl_sync(~0u, from, row);
        x[n] = make_uint2(0, 0);
        if (i < kReadRows * chunks && at > -2) {
            has |= 1u << n;
            if (at >= 0) x[n] = __ldcs(reinterpret_cast<const uint2*>(p.c.pages + at) + (i - row * chunks));
        }
    }
    const float by_mine = pow2(scale_exp(exponent));
    uint4* const to = reinterpret_cast<uint4*>(p.out + r0 * p.c.C);
#pragma unroll
    for (int n = 0; n < kLaneChunks * kReadRows; ++n) {
        const int i = n * 32 + lane, row = (i >= chunks) + (i >= 2 * chunks) + (i >= 3 * chunks);
        const float by = __shfl_sync(~0u, by_mine, row);
        if (!(has >> n & 1)) continue;
        float f[8];
        f32_of_f16x2(f16x2_of_e4m3x2(x[n].x), f[0], f[1]);
        f32_of_f16x2(f16x2_of_e4m3x2(x[n].x >> 16), f[2], f[3]);
        f32_of_f16x2(f16x2_of_e4m3x2(x[n].y), f[4], f[5]);
        f32_of_f16x2(f16x2_of_e4m3x2(x[n].y >> 16), f[6], f[7]);
        __stcs(to + i, make_uint4(pack_bf16x2(f[0] * by, f[1] * by), pack_bf16x2(f[2] * by, f[3] * by),
                                  pack_bf16x2(f[4] * by, f[5] * by), pack_bf16x2(f[6] * by, f[7] * by)));
    }
    raise_status(p.status, bits);
}

}  // namespace
}  // namespace mlap

using namespace mlap;

extern "C" {

int mla_prolog_cache8_page_bytes(const mla_prolog_cache8* cache, int64_t* bytes) {
    if (!bytes) return MLA_ERR_INVALID_ARG;
    *bytes = 0;
    Cache8 c;
    const int rc = check_cache8(cache, &c);
    if (rc == MLA_OK) *bytes = c.page_bytes;
    return rc;
}

int mla_prolog_cache8_write(const mla_prolog_cache8* cache, const void* rows, const int32_t* slot_mapping, int32_t T,
                            int32_t* status, void* stream) {
    Cache8 c;
    int rc = check_cache8(cache, &c), sms;
    if (rc != MLA_OK) return rc;
    if (T < 0 || T > (1 << 30)) return MLA_ERR_UNSUPPORTED_DIMS;
    if (status && !ptr_ok(status, 4)) return MLA_ERR_INVALID_ARG;
    if (T == 0) return MLA_OK;
    if (!ptr_ok(rows, 16) || !ptr_ok(slot_mapping, 4) || (c.num_pages && !ptr_ok(c.pages, 16))) return MLA_ERR_INVALID_ARG;
    if ((rc = current_sm103(&sms)) != MLA_OK) return rc;
    // Windows of 8, 16 and 32 tokens while the SMs hold all windows at once (128 sequences' tokens: 8 2.29 us, 16 2.50; 8192
    // in one chunk, blocks of 16: 16 5.0, 32 4.0), then of 32 by CTAs of 8 warps, which an SM has three of (262144: 77 us, by
    // those of 16 warps 91).  Rows of a block that another window has are read twice: long blocks take longer windows (16384
    // in blocks of 64: windows of 32 10.2 us, of 64 6.5), but not at the price of few CTAs (1024: of 16 4.0, of 64 5.2).
    const int kind = T > 32 * sms ? (c.block > 32 ? 4 : T > 64 * sms ? 3 : 2) : c.block > 16 || T > 8 * sms ? 1 : 0;
    const decltype(&mla_cache8_write_kernel<8, 1>) kernels[] = {&mla_cache8_write_kernel<8, 1>, &mla_cache8_write_kernel<16, 1>,
        &mla_cache8_write_kernel<16, 2>, &mla_cache8_write_kernel<8, 4>, &mla_cache8_write_kernel<8, 8>};
    const auto kernel = kernels[kind];
    const int window = kind == 0 ? 8 : kind == 1 ? 16 : kind == 4 ? 64 : 32, threads = kind == 1 || kind == 2 ? 512 : 256;
    const cudaError_t e = launch_kernel(kernel, dim3((T + window - 1) / window), dim3(threads), 0,
                                        static_cast<cudaStream_t>(stream), true, c, divide_by(c.page_size), divide_by(c.block),
                                        static_cast<const uint16_t*>(rows),
                                        slot_mapping, T, status);
    return e == cudaSuccess ? MLA_OK : report_cuda(e, "launch mla_cache8_write_kernel");
}

int mla_prolog_cache8_read(const mla_prolog_cache8* cache, const int32_t* page_table, int32_t table_rows, int32_t max_pages,
                           const int32_t* seqs, const int32_t* starts, const int32_t* cu, int32_t sequences, void* out,
                           int32_t T, int32_t* status, void* stream) {
    Cache8 c;
    int rc = check_cache8(cache, &c), sms;
    if (rc != MLA_OK) return rc;
    if (T < 0 || T > (1 << 30) || sequences < 0 || table_rows < 0 || max_pages < 1 ||
        static_cast<int64_t>(max_pages) * c.page_size > (1 << 30))
        return MLA_ERR_UNSUPPORTED_DIMS;
    if (!seqs && table_rows < sequences) return MLA_ERR_INVALID_ARG;
    if ((seqs && !ptr_ok(seqs, 4)) || (starts && !ptr_ok(starts, 4)) || (status && !ptr_ok(status, 4))) return MLA_ERR_INVALID_ARG;
    if (T == 0 || sequences == 0) return MLA_OK;
    if (!ptr_ok(cu, 4) || !ptr_ok(out, 16) || (table_rows && !ptr_ok(page_table, 4)) || (c.num_pages && !ptr_ok(c.pages, 16)))
        return MLA_ERR_INVALID_ARG;
    if ((rc = current_sm103(&sms)) != MLA_OK) return rc;
    const ReadParams p{c, divide_by(c.page_size), divide_by(c.block), page_table, seqs, starts, cu, table_rows, max_pages, sequences, T, static_cast<uint16_t*>(out), status};
    const cudaError_t e = launch_kernel(mla_cache8_read_kernel, dim3((T + kReadWarps * kReadRows - 1) / (kReadWarps * kReadRows)), dim3(kReadWarps * 32), 0,
                                        static_cast<cudaStream_t>(stream), true, p);
    return e == cudaSuccess ? MLA_OK : report_cuda(e, "launch mla_cache8_read_kernel");
}

}  // extern "C"
