// The page pool of the latent cache: extend, fork, release and compact move
// whole numbers (page table, lengths, reference counts); copy_pages moves the
// cache's contents.
//
// The bookkeeping calls run as one CTA of 1024 threads.  They touch a few
// hundred KB at most and are bound by latency (launch, then two or three
// dependent passes over refs), so one CTA that needs no grid-wide hand-over
// beats a spread of the same work over SMs that would have to meet twice.
#include <cstdint>

#include "attend.cuh"
#include "ptx.cuh"

namespace mlap {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxList = 1024;
constexpr int kPer = kMaxList / kThreads;  // list entries per thread
constexpr int kMost = 1 << 30;             // tokens of a sequence, slots or copies of a call: 32-bit sums hold twice that

struct Pool {
    int32_t sequences, max_pages, page_size, num_pages;
    int32_t* table;
    int32_t* lens;
    int32_t* refs;
    int32_t* status;
};

// First thing in every kernel here: the next one of the stream may be brought
// to the SMs meanwhile, and what the one before wrote is awaited.
__device__ __forceinline__ void pdl_begin() {
    pdl_launch_dependents();
    pdl_wait();
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Length of sequence s, cut to what its table row can hold.
__device__ __forceinline__ int seq_len(const Pool& p, int s) {
    const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
    const int n = p.lens[s];
    return n < 0 ? 0 : (n > cap ? static_cast<int>(cap) : n);
}

// Exclusive prefix sum of v over the block; *total receives the block's sum.
// All threads call it.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* total) {
    __shared__ int64_t warp_sum[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // a scan before this one has read warp_sum
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int64_t w = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(~0u, w, 31);
    const int64_t before = __shfl_sync(~0u, w, (warp + 31) & 31);
    return x - v + (warp ? before : 0);
}

// One pass over refs covers kWarps x words x 32 pages: warp w the words * 32
// pages from base + w * words * 32 on, whose bits lane k < words keeps for the
// k-th 32 of them.  Few pages are spread over all warps, many go in several
// passes of the largest size.
struct Span {
    int words;
    int64_t pages;
};
__device__ __forceinline__ Span span_of(const Pool& p) {
    const int w = (p.num_pages - 1) / kThreads + 1;
    const int words = w < 1 ? 1 : w > 32 ? 32 : w;
    return Span{words, static_cast<int64_t>(words) * kThreads};
}
__device__ __forceinline__ int64_t warp_base(const Span& sp, int64_t base) {
    return base + static_cast<int64_t>(threadIdx.x >> 5) * sp.words * 32;
}

__device__ __forceinline__ uint32_t free_mask(const Pool& p, const Span& sp, int64_t base) {
    const int lane = threadIdx.x & 31;
    const int64_t at = warp_base(sp, base);
    uint32_t mine = 0;
#pragma unroll 8
    for (int k = 0; k < sp.words; ++k) {
        const int64_t q = at + k * 32 + lane;
        const uint32_t m = __ballot_sync(~0u, q < p.num_pages && p.refs[q] == 0);
        if (lane == k) mine = m;
    }
    return mine;
}

// Bits of this lane's 32 pages that lie in [from, to).
__device__ __forceinline__ uint32_t range_mask(const Span& sp, int64_t base, int64_t from, int64_t to) {
    const int lane = threadIdx.x & 31;
    if (lane >= sp.words) return 0;
    const int64_t first = warp_base(sp, base) + lane * 32, a = from - first, b = to - first;
    const uint32_t below = b >= 32 ? ~0u : b <= 0 ? 0u : (1u << b) - 1u;
    return a >= 32 ? 0u : a <= 0 ? below : below & ~((1u << a) - 1u);
}

// Runs f(page, whether its bit is set, its rank) with a lane per page; `rank`
// is the rank of the lane's first bit.
template <class F>
__device__ __forceinline__ void for_pages(const Pool& p, const Span& sp, int64_t base, uint32_t bits, int64_t rank, F f) {
    const int lane = threadIdx.x & 31;
    const int64_t at = warp_base(sp, base);
    for (int k = 0; k < sp.words && at + k * 32 < p.num_pages; ++k) {
        const uint32_t m = __shfl_sync(~0u, bits, k);
        const int64_t r = __shfl_sync(~0u, rank, k) + __popc(m & ((1u << lane) - 1u));
        const int64_t page = at + k * 32 + lane;
        if (page < p.num_pages) f(static_cast<int32_t>(page), (m >> lane & 1u) != 0, r);
    }
}

// Sets again[i] for entries that repeat one before them.  A warp per entry.
__device__ __forceinline__ void find_repeats(const int32_t* list, int n, uint8_t* again) {
    for (int e = threadIdx.x >> 5; e < n; e += kWarps) {
        bool hit = false;
        const int v = list[e];
        for (int j = threadIdx.x & 31; j < e; j += 32) hit |= list[j] == v;
        if (__any_sync(~0u, hit)) hit = true;
        if ((threadIdx.x & 31) == 0) again[e] = hit;
    }
}

// The last entry e of the ascending first[0 .. n) with first[e] <= r.
__device__ __forceinline__ int find_entry(const int64_t* first, int n, int64_t r) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= r) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Deals out the lowest free pages: entry e of the list takes need[e] of them,
// in order, and `place(e, k, page)` stores its k-th.  An entry whose needs
// and those before it exceed the free pages gets none and `fits(e, false)`.
// first[] holds the exclusive sums of need[] and `want` their total.
template <class Fits, class Place>
__device__ __forceinline__ void deal_pages(const Pool& p, const int64_t* first, const int32_t* need, int n,
                                           int64_t want, Fits fits, Place place) {
    const Span sp = span_of(p);
    int64_t have = 0, rank = 0, sum, at = -1;
    uint32_t mask = 0;
    for (int64_t base = 0; base < p.num_pages && have < want; base += sp.pages) {
        mask = free_mask(p, sp, base);
        at = base;
        rank = block_scan(__popc(mask), &sum);
        have += sum;
    }
    for (int e = threadIdx.x; e < n; e += kThreads) fits(e, first[e] + need[e] <= have);
    int64_t before = 0;
    for (int64_t base = 0; base < p.num_pages && before < want; base += sp.pages) {
        if (base != at) {
            mask = free_mask(p, sp, base);
            at = base;
            rank = block_scan(__popc(mask), &sum);
        }
        for_pages(p, sp, base, mask, before + rank, [&](int32_t page, bool set, int64_t r) {
            if (!set || r >= want) return;
            const int e = find_entry(first, n, r);  // (an entry that needs nothing is never the last at or below r)
            if (first[e] + need[e] <= have) place(e, static_cast<int>(r - first[e]), page);
        });
        before += sum;
    }
}

__global__ void __launch_bounds__(kThreads) mla_pages_extend_kernel(Pool p, const int32_t* __restrict__ seqs,
                                                                    const int32_t* __restrict__ counts, int n,
                                                                    int32_t* __restrict__ slots,
                                                                    int32_t* __restrict__ positions, int total) {
    __shared__ int32_t seq[kMaxList], need[kMaxList], old[kMaxList];
    __shared__ int64_t first[kMaxList], tok[kMaxList];
    __shared__ uint8_t ok[kMaxList], again[kMaxList];
    pdl_begin();
    const int t = threadIdx.x;
    const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
    for (int i = t; i < n; i += kThreads) seq[i] = seqs[i];
    __syncthreads();
    find_repeats(seq, n, again);
    __syncthreads();
    int64_t sum_need = 0, sum_tok = 0;
    int64_t cnt[kPer];
    int bits = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = t * kPer + k;
        cnt[k] = 0;
        if (i >= n) continue;
        const int s = seq[i];
        const int c = counts[i];
        cnt[k] = c > 0 ? c : 0;
        int nd = 0, len = 0;
        uint8_t good = 0;
        if (s < 0 || s >= p.sequences || c < 0 || again[i]) {
            bits |= kStatusSeqRange;
        } else {
            len = seq_len(p, s);
            if (len + static_cast<int64_t>(c) > cap) {
                bits |= kStatusPoolFull;
            } else {
                good = 1;
                nd = ceil_div(len + c, p.page_size) - ceil_div(len, p.page_size);
            }
        }
        old[i] = len;
        need[i] = nd;
        ok[i] = good;
        sum_need += nd;
        sum_tok += cnt[k];
    }
    int64_t want, tokens;
    int64_t f = block_scan(sum_need, &want);
    int64_t g = block_scan(sum_tok, &tokens);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = t * kPer + k;
        if (i >= n) break;
        first[i] = f;
        tok[i] = g;
        f += need[i];
        g += cnt[k];
    }
    __syncthreads();
    deal_pages(
        p, first, need, n, want,
        [&](int e, bool fit) {
            if (ok[e] && need[e] && !fit) {
                ok[e] = 0;
                bits |= kStatusPoolFull;
            }
        },
        [&](int e, int k, int32_t page) {
            p.table[static_cast<int64_t>(seq[e]) * p.max_pages + ceil_div(old[e], p.page_size) + k] = page;
            p.refs[page] = 1;
        });
    __syncthreads();
    if (slots || positions) {
        if (tokens > total) bits |= kStatusSlotRange;
        for (int j = t; j < total; j += kThreads) {
            int slot = -1, pos = 0;
            if (j < tokens) {
                const int e = find_entry(tok, n, j);
                if (ok[e]) {
                    pos = old[e] + static_cast<int>(j - tok[e]);
                    slot = p.table[static_cast<int64_t>(seq[e]) * p.max_pages + pos / p.page_size] * p.page_size +
                           pos % p.page_size;
                }
            }
            if (slots) slots[j] = slot;
            if (positions) positions[j] = pos;
        }
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = t * kPer + k;
        if (i < n && ok[i]) p.lens[seq[i]] = old[i] + static_cast<int>(cnt[k]);
    }
    raise_status(p.status, bits);
}

__global__ void __launch_bounds__(kThreads) mla_pages_fork_kernel(Pool p, const int32_t* __restrict__ parents,
                                                                  const int32_t* __restrict__ children, int n,
                                                                  int32_t* __restrict__ src,
                                                                  int32_t* __restrict__ dst) {
    __shared__ int32_t par[kMaxList], child[kMaxList], need[kMaxList], len[kMaxList];
    __shared__ int64_t first[kMaxList];
    __shared__ uint8_t ok[kMaxList], again[kMaxList];
    pdl_begin();
    const int t = threadIdx.x;
    for (int i = t; i < n; i += kThreads) par[i] = parents[i], child[i] = children[i];
    __syncthreads();
    find_repeats(child, n, again);
    __syncthreads();
    int64_t sum_need = 0;
    int bits = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = t * kPer + k;
        if (i >= n) continue;
        const int a = par[i], c = child[i];
        const bool good = a >= 0 && a < p.sequences && c >= 0 && c < p.sequences && p.lens[c] == 0 && !again[i];
        if (!good) bits |= kStatusSeqRange;
        len[i] = good ? seq_len(p, a) : 0;
        need[i] = len[i] % p.page_size != 0;
        ok[i] = good;
        sum_need += need[i];
        src[i] = dst[i] = -1;
    }
    int64_t want;
    int64_t f = block_scan(sum_need, &want);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = t * kPer + k;
        if (i >= n) break;
        first[i] = f;
        f += need[i];
    }
    __syncthreads();
    deal_pages(
        p, first, need, n, want,
        [&](int e, bool fit) {
            if (ok[e] && need[e] && !fit) {
                ok[e] = 0;
                bits |= kStatusPoolFull;
            }
        },
        [&](int e, int, int32_t page) {
            const int full = len[e] / p.page_size;
            p.table[static_cast<int64_t>(child[e]) * p.max_pages + full] = page;
            p.refs[page] = 1;
            src[e] = p.table[static_cast<int64_t>(par[e]) * p.max_pages + full];
            dst[e] = page;
        });
    __syncthreads();
    // the shared pages: a warp per child
    for (int e = t >> 5; e < n; e += kWarps) {
        if (!ok[e]) continue;
        const int full = len[e] / p.page_size;
        const int32_t* from = p.table + static_cast<int64_t>(par[e]) * p.max_pages;
        int32_t* to = p.table + static_cast<int64_t>(child[e]) * p.max_pages;
        for (int j = t & 31; j < full; j += 32) {
            const int32_t page = from[j];
            to[j] = page;
            if (page >= 0 && page < p.num_pages) atomicAdd(p.refs + page, 1);
            else bits |= kStatusPageRange;
        }
        if ((t & 31) == 0) p.lens[child[e]] = len[e];
    }
    raise_status(p.status, bits);
}

__global__ void __launch_bounds__(kThreads) mla_pages_release_kernel(Pool p, const int32_t* __restrict__ seqs, int n) {
    __shared__ int32_t seq[kMaxList];
    pdl_begin();
    const int t = threadIdx.x;
    for (int i = t; i < n; i += kThreads) seq[i] = seqs[i];
    __syncthreads();
    int bits = 0;
    for (int e = t >> 5; e < n; e += kWarps) {
        const int s = seq[e];
        if (s < 0 || s >= p.sequences) {
            bits |= kStatusSeqRange;
            continue;
        }
        // the first listing ends the sequence
        bool again = false;
        for (int j = t & 31; j < e; j += 32) again |= seq[j] == s;
        if (__any_sync(~0u, again)) continue;
        const int held = ceil_div(seq_len(p, s), p.page_size);
        int32_t* row = p.table + static_cast<int64_t>(s) * p.max_pages;
        for (int j = t & 31; j < p.max_pages; j += 32) {
            const int32_t page = row[j];
            row[j] = -1;
            if (j >= held) continue;
            if (page >= 0 && page < p.num_pages) atomicSub(p.refs + page, 1);
            else bits |= kStatusPageRange;
        }
        __syncwarp();
        if ((t & 31) == 0) p.lens[s] = 0;
    }
    raise_status(p.status, bits);
}

// Where each live page goes.  The holes (free pages below L) are listed in
// moved_to[0 ..) first: a mover's rank is below L and its own place at or
// above, so reading the list and writing the movers' places do not meet; the
// places below L are written last.
__global__ void __launch_bounds__(kThreads) mla_pages_compact_kernel(Pool p, int32_t* __restrict__ moved_to,
                                                                     int32_t* __restrict__ live_out) {
    pdl_begin();
    const int t = threadIdx.x;
    const Span sp = span_of(p);
    int64_t live = 0, sum, at = -1;
    uint32_t mask = 0;
    auto load = [&](int64_t base) {
        if (base != at) mask = free_mask(p, sp, base), at = base;
    };
    for (int64_t base = 0; base < p.num_pages; base += sp.pages) {
        load(base);
        block_scan(__popc(range_mask(sp, base, 0, p.num_pages) & ~mask), &sum);
        live += sum;
    }
    if (t == 0 && live_out) *live_out = static_cast<int32_t>(live);
    int64_t before = 0;
    for (int64_t base = 0; base < live; base += sp.pages) {
        load(base);
        const uint32_t holes = mask & range_mask(sp, base, 0, live);
        const int64_t rank = before + block_scan(__popc(holes), &sum);
        for_pages(p, sp, base, holes, rank, [&](int32_t page, bool set, int64_t r) {
            if (set) moved_to[r] = page;
        });
        before += sum;
    }
    __syncthreads();
    before = 0;
    for (int64_t base = live / sp.pages * sp.pages; base < p.num_pages; base += sp.pages) {
        load(base);
        const uint32_t go = range_mask(sp, base, live, p.num_pages) & ~mask;
        const int64_t rank = before + block_scan(__popc(go), &sum);
        for_pages(p, sp, base, go, rank, [&](int32_t page, bool set, int64_t r) {
            if (page >= live) moved_to[page] = set ? moved_to[r] : -1;
        });
        before += sum;
    }
    __syncthreads();
    for (int64_t base = 0; base < live; base += sp.pages) {
        load(base);
        for_pages(p, sp, base, mask, 0, [&](int32_t page, bool free, int64_t) {
            if (page < live) moved_to[page] = free ? -1 : page;
        });
    }
    __syncthreads();
    for (int64_t page = live + t; page < p.num_pages; page += kThreads) {
        const int32_t place = moved_to[page];
        if (place < 0) continue;
        p.refs[place] = p.refs[page];
        p.refs[page] = 0;
    }
}

__global__ void __launch_bounds__(256) mla_pages_retable_kernel(Pool p, const int32_t* __restrict__ moved_to) {
    pdl_begin();
    const int64_t n = static_cast<int64_t>(p.sequences) * p.max_pages;
    int bits = 0;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const int32_t page = p.table[i];
        if (page < 0) continue;
        if (page >= p.num_pages) {
            bits |= kStatusPageRange;
            continue;
        }
        const int32_t to = moved_to[page];
        if (to >= 0 && to != page) p.table[i] = to;
    }
    raise_status(p.status, bits);
}

// A CTA copies `per` entries' pages of one layer, or one of `pieces` pieces of
// one entry's page; each thread keeps 8 loads of 16 bytes in flight.
constexpr int kCopyThreads = 256, kCopyLoads = 8, kCopyStep = kCopyThreads * kCopyLoads;

__global__ void __launch_bounds__(kCopyThreads) mla_copy_pages_kernel(uint8_t* __restrict__ cache, int64_t layer_stride,
                                                                     int64_t num_pages, int64_t page_bytes,
                                                                     const int32_t* __restrict__ src,
                                                                     const int32_t* __restrict__ dst, int n, int per,
                                                                     int pieces, int32_t* status) {
    pdl_begin();
    uint8_t* layer = cache + blockIdx.y * layer_stride;
    const int64_t words = page_bytes / 16;
    const int64_t piece = (words + pieces - 1) / pieces, from_word = blockIdx.z * piece;
    const int64_t to_word = from_word + piece < words ? from_word + piece : words;
    // the entries' pages in one look (the first `per` lanes' answers)
    const int lane = threadIdx.x & 31, i0 = blockIdx.x * per;
    int a = -1, b = -1;
    if (lane < per && i0 + lane < n) {
        b = dst[i0 + lane];
        a = src ? src[i0 + lane] : i0 + lane;
    }
    bool go = a >= 0 && b >= 0 && a != b;
    if (go && (a >= num_pages || b >= num_pages)) {
        go = false;
        if (threadIdx.x < 32) raise_status(status, kStatusPageRange);
    }
    for (uint32_t todo = __ballot_sync(~0u, go); todo; todo &= todo - 1) {
        const int e = __ffs(todo) - 1;
        const uint4* from = reinterpret_cast<const uint4*>(layer + __shfl_sync(~0u, a, e) * page_bytes);
        uint4* to = reinterpret_cast<uint4*>(layer + __shfl_sync(~0u, b, e) * page_bytes);
        for (int64_t j = from_word + threadIdx.x; j < to_word; j += kCopyStep) {
            uint4 v[kCopyLoads];
#pragma unroll
            for (int k = 0; k < kCopyLoads; ++k)
                if (j + k * kCopyThreads < to_word) v[k] = __ldcs(from + j + k * kCopyThreads);
#pragma unroll
            for (int k = 0; k < kCopyLoads; ++k)
                if (j + k * kCopyThreads < to_word) __stcs(to + j + k * kCopyThreads, v[k]);
        }
    }
}

int check_pool(const mla_prolog_pool* h, Pool* p) {
    if (!h) return MLA_ERR_INVALID_ARG;
    if (h->sequences < 0 || h->num_pages < 0 || h->max_pages < 1 || h->page_size < 1) return MLA_ERR_UNSUPPORTED_DIMS;
    if (static_cast<int64_t>(h->max_pages) * h->page_size > kMost ||
        static_cast<int64_t>(h->num_pages) * h->page_size > INT32_MAX)
        return MLA_ERR_UNSUPPORTED_DIMS;
    if (h->sequences && (!ptr_ok(h->page_table, 4) || !ptr_ok(h->seq_lens, 4))) return MLA_ERR_INVALID_ARG;
    if (h->num_pages && !ptr_ok(h->refs, 4)) return MLA_ERR_INVALID_ARG;
    if (h->status && !ptr_ok(h->status, 4)) return MLA_ERR_INVALID_ARG;
    *p = Pool{h->sequences, h->max_pages, h->page_size, h->num_pages, h->page_table, h->seq_lens, h->refs, h->status};
    return MLA_OK;
}

int check_list(int32_t n, const void* a, const void* b) {
    if (n < 0) return MLA_ERR_INVALID_ARG;
    if (n > kMaxList) return MLA_ERR_UNSUPPORTED_DIMS;
    return n == 0 || (ptr_ok(a, 4) && ptr_ok(b, 4)) ? MLA_OK : MLA_ERR_INVALID_ARG;
}

template <class... KArgs, class... Args>
int start(const char* what, void (*kernel)(KArgs...), dim3 grid, int threads, void* stream, Args... args) {
    const cudaError_t e = launch_kernel(kernel, grid, dim3(threads), 0, static_cast<cudaStream_t>(stream), true, args...);
    return e == cudaSuccess ? MLA_OK : report_cuda(e, what);
}

}  // namespace
}  // namespace mlap

using namespace mlap;

extern "C" {

int mla_prolog_pages_extend(const mla_prolog_pool* pool, const int32_t* seqs, const int32_t* counts, int32_t n,
                            int32_t* slot_mapping, int32_t* positions, int32_t total, void* stream) {
    Pool p;
    int rc = check_pool(pool, &p);
    if (rc == MLA_OK) rc = check_list(n, seqs, counts);
    if (rc != MLA_OK) return rc;
    if (total > kMost) return MLA_ERR_UNSUPPORTED_DIMS;
    if (total < 0 || (slot_mapping && !ptr_ok(slot_mapping, 4)) || (positions && !ptr_ok(positions, 4)))
        return MLA_ERR_INVALID_ARG;
    if (n == 0 && total == 0) return MLA_OK;
    int sms;
    if ((rc = current_sm103(&sms)) != MLA_OK) return rc;
    return start("launch mla_pages_extend_kernel", mla_pages_extend_kernel, 1, kThreads, stream, p, seqs, counts, n,
                 slot_mapping, positions, total);
}

int mla_prolog_pages_fork(const mla_prolog_pool* pool, const int32_t* parents, const int32_t* children, int32_t n,
                          int32_t* copy_src, int32_t* copy_dst, void* stream) {
    Pool p;
    int rc = check_pool(pool, &p);
    if (rc == MLA_OK) rc = check_list(n, parents, children);
    if (rc == MLA_OK) rc = check_list(n, copy_src, copy_dst);
    if (rc != MLA_OK || n == 0) return rc;
    int sms;
    if ((rc = current_sm103(&sms)) != MLA_OK) return rc;
    return start("launch mla_pages_fork_kernel", mla_pages_fork_kernel, 1, kThreads, stream, p, parents, children, n,
                 copy_src, copy_dst);
}

int mla_prolog_pages_release(const mla_prolog_pool* pool, const int32_t* seqs, int32_t n, void* stream) {
    Pool p;
    int rc = check_pool(pool, &p);
    if (rc == MLA_OK) rc = check_list(n, seqs, seqs);
    if (rc != MLA_OK || n == 0) return rc;
    int sms;
    if ((rc = current_sm103(&sms)) != MLA_OK) return rc;
    return start("launch mla_pages_release_kernel", mla_pages_release_kernel, 1, kThreads, stream, p, seqs, n);
}

int mla_prolog_pages_compact(const mla_prolog_pool* pool, int32_t* moved_to, int32_t* live, void* stream) {
    Pool p;
    int rc = check_pool(pool, &p);
    if (rc != MLA_OK) return rc;
    if ((p.num_pages && !ptr_ok(moved_to, 4)) || (live && !ptr_ok(live, 4))) return MLA_ERR_INVALID_ARG;
    int sms;
    if ((rc = current_sm103(&sms)) != MLA_OK) return rc;
    rc = start("launch mla_pages_compact_kernel", mla_pages_compact_kernel, 1, kThreads, stream, p, moved_to, live);
    const int64_t entries = static_cast<int64_t>(p.sequences) * p.max_pages;
    if (rc != MLA_OK || entries == 0) return rc;
    const int64_t blocks = (entries + 255) / 256;
    return start("launch mla_pages_retable_kernel", mla_pages_retable_kernel,
                 static_cast<unsigned>(blocks < 8 * sms ? blocks : 8 * sms), 256, stream, p, moved_to);
}

int mla_prolog_copy_pages(void* cache, int32_t layers, int64_t layer_stride, int64_t num_pages, int64_t page_bytes,
                          const int32_t* src, const int32_t* dst, int32_t n, int32_t* status, void* stream) {
    if (layers < 0 || num_pages < 0 || n < 0 || page_bytes <= 0 || page_bytes % 16 || layers > 65535)
        return MLA_ERR_INVALID_ARG;
    if (n > kMost) return MLA_ERR_UNSUPPORTED_DIMS;
    if (num_pages > INT64_MAX / page_bytes) return MLA_ERR_INVALID_ARG;
    if (layers > 1 && (layer_stride % 16 || layer_stride < num_pages * page_bytes)) return MLA_ERR_INVALID_ARG;
    if (status && !ptr_ok(status, 4)) return MLA_ERR_INVALID_ARG;
    if (layers == 0 || n == 0) return MLA_OK;
    if ((num_pages && !ptr_ok(cache, 16)) || (src && !ptr_ok(src, 4)) || !ptr_ok(dst, 4)) return MLA_ERR_INVALID_ARG;
    int sms;
    const int rc = current_sm103(&sms);
    if (rc != MLA_OK) return rc;
    // Most entries of a long list are skipped (a compaction's): eight to a CTA then, so that the empty CTAs do not
    // take longer than the copies; a short list is cut into pieces, so that few pages still fill the SMs.
    const bool many = static_cast<int64_t>(n) * layers > 16 * sms;
    const int per = many ? 8 : 1;
    const int64_t step_bytes = kCopyStep * 16;
    const int pieces = many ? 1 : static_cast<int>(std::min<int64_t>((page_bytes + step_bytes - 1) / step_bytes, 16));
    return start("launch mla_copy_pages_kernel", mla_copy_pages_kernel, dim3((n + per - 1) / per, layers, pieces), kCopyThreads,
                 stream, static_cast<uint8_t*>(cache), layer_stride, num_pages, page_bytes, src, dst, n, per, pieces, status);
}

}  // extern "C"
