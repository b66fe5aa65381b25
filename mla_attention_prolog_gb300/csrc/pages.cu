// The page pool of the latent cache: extend, fork, release and compact move
// whole numbers (page table, lengths, reference counts); copy_pages moves the
// cache's contents.
//
// The bookkeeping calls run as one CTA of 1024 threads.  They touch a few
// hundred KB at most and are bound by latency (lists, lengths, a pass over
// refs, the dealing out), so one CTA that needs no grid-wide hand-over beats a
// spread of the same work over SMs that would have to meet twice.  All calls
// are dependent launches, which hide each other's launch latency.
#include <cstdint>

#include "attend.cuh"
#include "ptx.cuh"

namespace mlap {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxList = 1024;
static_assert(kMaxList <= kThreads, "a thread per list entry");
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

// A sequence's length, cut to what its table row can hold.
__device__ __forceinline__ int cut_len(const Pool& p, int n) {
    const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
    return n < 0 ? 0 : (n > cap ? static_cast<int>(cap) : n);
}
__device__ __forceinline__ int len_bits(const Pool& p, int n) { return cut_len(p, n) != n ? kStatusSeqRange : 0; }
__device__ __forceinline__ bool in_pool(const Pool& p, int32_t page) { return page >= 0 && page < p.num_pages; }

// Exclusive prefix sums over the block, in place; total[k]: the block's sums.
// All threads call it.
template <int N>
__device__ __forceinline__ void block_scan(int64_t (&v)[N], int64_t (&total)[N]) {
    __shared__ int64_t warp_sum[N][kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x[N], w[N];
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int64_t y = __shfl_up_sync(~0u, x[k], o);
            if (lane >= o) x[k] += y;
        }
    }
    __syncthreads();  // a scan before this one has read warp_sum
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (lane == 31) warp_sum[k][warp] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = warp_sum[k][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int64_t y = __shfl_up_sync(~0u, w[k], o);
            if (lane >= o) w[k] += y;
        }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        total[k] = __shfl_sync(~0u, w[k], 31);
        const int64_t before = __shfl_sync(~0u, w[k], (warp + 31) & 31);
        v[k] = x[k] - v[k] + (warp ? before : 0);
    }
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

// The first place of each value of a list: a hash table with linear probing,
// half full at most (values >= 0).
struct Firsts {
    int32_t value[2 * kMaxList], place[2 * kMaxList];

    __device__ __forceinline__ void clear() {
        for (int i = threadIdx.x; i < 2 * kMaxList; i += kThreads) value[i] = -1, place[i] = kMaxList;
    }
    // The value's bucket, whose place is final after the next barrier.
    __device__ __forceinline__ int add(int v, int i) {
        static_assert(kMaxList == 1024, "the hash below has 11 bits");
        int b = static_cast<int>(static_cast<uint32_t>(v) * 0x9E3779B1u >> 21);
        for (;;) {
            const int was = atomicCAS(value + b, -1, v);
            if (was == -1 || was == v) break;
            b = (b + 1) % (2 * kMaxList);
        }
        atomicMin(place + b, i);
        return b;
    }
};

// Lists of pages on their way to their entries take the table's place.
constexpr int kWindow = 4 * kMaxList;
union Scratch {
    Firsts firsts;
    int32_t pages[kWindow];
};

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
// first[] holds the exclusive sums of need[] and `want` their total.  The free
// pages are listed by rank first (a bit scan), so that the search for a
// page's entry runs once per page dealt and not once per page of the pool.
template <class Fits, class Place>
__device__ __forceinline__ void deal_pages(const Pool& p, const int64_t* first, const int32_t* need, int n,
                                           int64_t want, int32_t* window, Fits fits, Place place) {
    const Span sp = span_of(p);
    int64_t have = 0, rank[1], sum[1], at = -1;
    uint32_t mask = 0;
    auto look = [&](int64_t base) {
        if (base == at) return;
        mask = free_mask(p, sp, base);
        rank[0] = __popc(mask);
        block_scan(rank, sum);
        at = base;
    };
    for (int64_t base = 0; base < p.num_pages && have < want; base += sp.pages) {
        look(base);
        have += sum[0];
    }
    if (threadIdx.x < n) fits(threadIdx.x, first[threadIdx.x] + need[threadIdx.x] <= have);
    const int64_t give = want < have ? want : have;
    int64_t before = 0;
    for (int64_t base = 0; before < give; base += sp.pages) {
        look(base);
        const int64_t upto = before + sum[0] < give ? before + sum[0] : give;
        for (int64_t from = before; from < upto; from += kWindow) {
            const int count = static_cast<int>(upto - from < kWindow ? upto - from : kWindow);
            __syncthreads();  // the window has been read
            for_pages(p, sp, base, mask, before + rank[0], [&](int32_t page, bool set, int64_t r) {
                if (set && r >= from && r < from + count) window[r - from] = page;
            });
            __syncthreads();
            for (int i = threadIdx.x; i < count; i += kThreads) {
                const int e = find_entry(first, n, from + i);  // (one that needs nothing is never the last at or below)
                if (first[e] + need[e] <= have) place(e, static_cast<int>(from + i - first[e]), window[i]);
            }
        }
        before += sum[0];
    }
    __syncthreads();
}

// Figures of the kernels below: 256 sequences, 4096 pages of 64, GB300, in a
// stream of calls.
// A thread per entry; the lists, then the lengths, are on their way while
// repeats are looked for.  240 entries of 17 tokens: 9.7 us (14.9 with a search per token and per free
// page).
__global__ void __launch_bounds__(kThreads) mla_pages_extend_kernel(Pool p, const int32_t* __restrict__ seqs,
                                                                    const int32_t* __restrict__ counts, int n,
                                                                    int32_t* __restrict__ slots,
                                                                    int32_t* __restrict__ positions, int total) {
    __shared__ Scratch scratch;
    __shared__ int32_t seq[kMaxList], need[kMaxList], old[kMaxList];
    __shared__ int64_t first[kMaxList], tok[kMaxList];
    __shared__ uint8_t ok[kMaxList];
    pdl_begin();
    const int t = threadIdx.x;
    const bool mine = t < n;
    const int s = mine ? seqs[t] : -1, c = mine ? counts[t] : 0;
    const bool inside = s >= 0 && s < p.sequences;
    const int held = inside ? p.lens[s] : 0;
    scratch.firsts.clear();
    __syncthreads();
    const int bucket = inside ? scratch.firsts.add(s, t) : 0;
    __syncthreads();
    const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
    int bits = 0;
    if (mine) {
        int nd = 0, len = 0;
        bool good = false;
        if (!inside || c < 0 || scratch.firsts.place[bucket] != t) {
            bits |= kStatusSeqRange;
        } else {
            len = cut_len(p, held);
            bits |= len_bits(p, held);
            if (len + static_cast<int64_t>(c) > cap) {
                bits |= kStatusPoolFull;
            } else {
                good = true;
                nd = ceil_div(len + c, p.page_size) - ceil_div(len, p.page_size);
            }
        }
        seq[t] = s;
        old[t] = len;
        need[t] = nd;
        ok[t] = good;
    }
    int64_t sums[2] = {mine ? need[t] : 0, c > 0 ? c : 0}, totals[2];
    block_scan(sums, totals);
    if (mine) first[t] = sums[0], tok[t] = sums[1];
    const int64_t tokens = totals[1];
    __syncthreads();
    deal_pages(
        p, first, need, n, totals[0], scratch.pages,
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
    if (slots || positions) {
        if (tokens > total) bits |= kStatusSlotRange;
        // With more tokens than threads a thread takes four in a row, which share the search for their entry and,
        // mostly, the look at their page.
        const int run = total > kThreads ? 4 : 1;
        for (int j0 = t * run; j0 < total; j0 += kThreads * run) {
            int e = j0 < tokens ? find_entry(tok, n, j0) : n, pos = 0, slot = 0, room = 0;
            bool good = false, fresh = true, paged = false;
            for (int j = j0; j < j0 + run && j < total; ++j) {
                while (e < n && j >= (e + 1 < n ? tok[e + 1] : tokens)) ++e, fresh = true;
                if (fresh) {
                    good = e < n && ok[e];
                    if (good) pos = old[e] + static_cast<int>(j - tok[e]);
                    room = 0;
                    fresh = false;
                }
                if (good && room == 0) {
                    const int in = pos % p.page_size;
                    const int32_t page = p.table[static_cast<int64_t>(seq[e]) * p.max_pages + pos / p.page_size];
                    paged = in_pool(p, page);  // (the page that the sequence ended in need not be)
                    slot = paged ? page * p.page_size + in : 0;
                    room = p.page_size - in;
                    if (!paged) bits |= kStatusPageRange;
                }
                if (slots) slots[j] = good && paged ? slot : -1;
                if (positions) positions[j] = good ? pos : 0;
                ++slot, ++pos, --room;
            }
        }
    }
    if (mine && ok[t]) p.lens[s] = old[t] + c;
    raise_status(p.status, bits);
}

// 48 children: 7.2 us.
__global__ void __launch_bounds__(kThreads) mla_pages_fork_kernel(Pool p, const int32_t* __restrict__ parents,
                                                                  const int32_t* __restrict__ children, int n,
                                                                  int32_t* __restrict__ src,
                                                                  int32_t* __restrict__ dst) {
    __shared__ Scratch scratch;
    __shared__ int32_t par[kMaxList], child[kMaxList], need[kMaxList], len[kMaxList];
    __shared__ int64_t first[kMaxList];
    __shared__ uint8_t ok[kMaxList];
    pdl_begin();
    const int t = threadIdx.x;
    const bool mine = t < n;
    const int a = mine ? parents[t] : -1, c = mine ? children[t] : -1;
    const bool from = a >= 0 && a < p.sequences, to = c >= 0 && c < p.sequences;
    const int held = from ? p.lens[a] : 0, empty = to ? p.lens[c] : 1;
    scratch.firsts.clear();
    __syncthreads();
    const int bucket = to ? scratch.firsts.add(c, t) : 0;
    __syncthreads();
    int bits = 0;
    if (mine) {
        const bool good = from && to && empty == 0 && scratch.firsts.place[bucket] == t;
        if (!good) bits |= kStatusSeqRange;
        if (good) bits |= len_bits(p, held);
        par[t] = a;
        child[t] = c;
        len[t] = good ? cut_len(p, held) : 0;
        need[t] = len[t] % p.page_size != 0;
        ok[t] = good;
        src[t] = dst[t] = -1;
    }
    int64_t sums[1] = {mine ? need[t] : 0}, want[1];
    block_scan(sums, want);
    if (mine) first[t] = sums[0];
    __syncthreads();
    deal_pages(
        p, first, need, n, want[0], scratch.pages,
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
            const int32_t old = p.table[static_cast<int64_t>(par[e]) * p.max_pages + full];
            if (in_pool(p, old)) src[e] = old, dst[e] = page;
            else bits |= kStatusPageRange;
        });
    // the shared pages: a warp per child
    for (int e = t >> 5; e < n; e += kWarps) {
        if (!ok[e]) continue;
        const int full = len[e] / p.page_size;
        const int32_t* old = p.table + static_cast<int64_t>(par[e]) * p.max_pages;
        int32_t* row = p.table + static_cast<int64_t>(child[e]) * p.max_pages;
        for (int j = t & 31; j < full; j += 32) {
            const int32_t page = old[j];
            row[j] = page;
            if (in_pool(p, page)) atomicAdd(p.refs + page, 1);
            else bits |= kStatusPageRange;
        }
        if ((t & 31) == 0) p.lens[child[e]] = len[e];
    }
    raise_status(p.status, bits);
}

// 64 sequences: 2.8 us.
__global__ void __launch_bounds__(kThreads) mla_pages_release_kernel(Pool p, const int32_t* __restrict__ seqs, int n) {
    __shared__ Firsts firsts;
    __shared__ int32_t seq[kMaxList], held[kMaxList];
    pdl_begin();
    const int t = threadIdx.x;
    const int s = t < n ? seqs[t] : 0;
    const bool inside = t < n && s >= 0 && s < p.sequences;
    const int len = inside ? p.lens[s] : 0;
    firsts.clear();
    __syncthreads();
    const int bucket = inside ? firsts.add(s, t) : 0;
    __syncthreads();
    int bits = t < n && !inside ? kStatusSeqRange : 0;
    if (t < n) {
        seq[t] = inside && firsts.place[bucket] == t ? s : -1;  // the first listing ends the sequence
        if (seq[t] >= 0) bits |= len_bits(p, len);
        held[t] = ceil_div(cut_len(p, len), p.page_size);
    }
    __syncthreads();
    for (int e = t >> 5; e < n; e += kWarps) {
        if (seq[e] < 0) continue;
        int32_t* row = p.table + static_cast<int64_t>(seq[e]) * p.max_pages;
        for (int j = t & 31; j < p.max_pages; j += 32) {
            const int32_t page = row[j];
            row[j] = -1;
            if (j >= held[e]) continue;
            if (in_pool(p, page)) atomicSub(p.refs + page, 1);
            else bits |= kStatusPageRange;
        }
        if ((t & 31) == 0) p.lens[seq[e]] = 0;
    }
    raise_status(p.status, bits);
}

// Where each live page goes.  The holes (free pages below L) are listed in
// moved_to[0 ..) first: a mover's rank is below L and its own place at or
// above, so reading the list and writing the movers' places do not meet; the
// places below L are written last.  One prefix sum of the free pages ranks
// both: a hole by the free pages before it, a mover by the live pages between
// L and it.  5.6 us, and 1.9 for the table.
__global__ void __launch_bounds__(kThreads) mla_pages_compact_kernel(Pool p, int32_t* __restrict__ moved_to,
                                                                     int32_t* __restrict__ live_out) {
    __shared__ int32_t holes_below;
    pdl_begin();
    const int t = threadIdx.x;
    const Span sp = span_of(p);
    int64_t rank[1] = {0}, sum[1], at = -1, live = p.num_pages;
    uint32_t mask = 0;
    auto look = [&](int64_t base) {
        if (base == at) return;
        mask = free_mask(p, sp, base);
        rank[0] = __popc(mask);
        block_scan(rank, sum);
        at = base;
    };
    if (t == 0) holes_below = 0;
    for (int64_t base = 0; base < p.num_pages; base += sp.pages) {
        look(base);
        live -= sum[0];
    }
    if (t == 0 && live_out) *live_out = static_cast<int32_t>(live);
    // free pages before the first pass that holds a page at or above L
    int64_t before = 0;
    for (int64_t base = 0; base < live; base += sp.pages) {
        look(base);
        const uint32_t holes = mask & range_mask(sp, base, 0, live);
        for_pages(p, sp, base, holes, before + rank[0], [&](int32_t page, bool set, int64_t r) {
            if (set) moved_to[r] = page;
        });
        const int count = __reduce_add_sync(~0u, __popc(holes));
        if ((t & 31) == 0 && count) atomicAdd(&holes_below, count);
        if (base + sp.pages <= live) before += sum[0];
    }
    __syncthreads();
    const int64_t stay = live - holes_below;  // live pages below L
    for (int64_t base = live / sp.pages * sp.pages; base < p.num_pages; base += sp.pages) {
        look(base);
        const uint32_t go = range_mask(sp, base, live, p.num_pages) & ~mask;
        const int64_t first = warp_base(sp, base) + (t & 31) * 32, r0 = first - before - rank[0] - stay;
        for_pages(p, sp, base, go, r0 > 0 ? r0 : 0, [&](int32_t page, bool set, int64_t r) {
            if (page >= live) moved_to[page] = set ? moved_to[r] : -1;
        });
        before += sum[0];
    }
    __syncthreads();
    for (int64_t base = 0; base < live; base += sp.pages) {
        look(base);
        for_pages(p, sp, base, mask, 0, [&](int32_t page, bool free, int64_t) {
            if (page < live) moved_to[page] = free ? -1 : page;
        });
    }
    __syncthreads();
    for (int64_t page0 = live + t; page0 < p.num_pages; page0 += 4 * kThreads) {
        int32_t place[4], n[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t page = page0 + k * kThreads;
            place[k] = page < p.num_pages ? moved_to[page] : -1;
            n[k] = page < p.num_pages ? p.refs[page] : 0;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (place[k] >= 0) p.refs[place[k]] = n[k], p.refs[page0 + k * kThreads] = 0;
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
// one entry's page; each thread keeps 8 loads of 16 bytes in flight.  Bound by
// HBM: 1.09 GB in 174 us, 6.3 TB/s (94 % of the measured copy rate).
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
    // take longer than the copies; a short list is cut into pieces, so that few pages still fill the SMs.  (A step of
    // both, 256 sequences and 8 layers: 221 us; all as short lists 243, all as long ones 235.)
    const bool many = static_cast<int64_t>(n) * layers > 16 * sms;
    const int per = many ? 8 : 1;
    const int64_t step_bytes = kCopyStep * 16;
    const int pieces = many ? 1 : static_cast<int>(std::min<int64_t>((page_bytes + step_bytes - 1) / step_bytes, 16));
    return start("launch mla_copy_pages_kernel", mla_copy_pages_kernel, dim3((n + per - 1) / per, layers, pieces), kCopyThreads,
                 stream, static_cast<uint8_t*>(cache), layer_stride, num_pages, page_bytes, src, dst, n, per, pieces, status);
}

}  // extern "C"
