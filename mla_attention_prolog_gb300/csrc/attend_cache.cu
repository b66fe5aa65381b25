// One decoding step over the latent KV cache: mla_prolog_attend_cache.
//
// A tile is 128 query rows (sequence, head) that see the same keys: the rows
// of one sequence on its own pages, or 128 rows of any sequences on the
// shared prefix, whose rows are thus read and multiplied once per 128 rows
// instead of once per sequence.  Every key is one cache row of Lkv + R
// columns, of which the first Lkv are the value too.
//
//   S = Q K^T   128 x 64 keys, 576 deep     O += P V   128 x Lkv, 64 deep
//
// O of 128 rows x 512 columns in FP32 would fill TMEM alone, so two CTAs share
// a tile: each makes all of S and half of the columns of O (256 TMEM columns).
// Doing S twice costs 1.5 times the products of a perfect split; halving the
// rows instead would cost twice the key traffic into each SM for the same
// products, and exchanging S or P between the CTAs a round trip per key tile.
// Two thirds of Q stay in TMEM as well (192 columns, read as the A operand),
// S takes the last 64; the rest of Q, two key tiles and P fill shared memory.
//
// The work is cut into as many equal runs of key tiles as there are CTA pairs
// (a tile costs its key tiles plus kOverhead for its start and end); a run
// takes whole or partial tiles.  Partial results go to the workspace in FP32,
// and a second kernel joins them.
#include <cmath>
#include <cstdint>

#include "attend.cuh"
#include "ptx.cuh"

namespace mlap {
namespace {

constexpr int kRows = 128;                // query rows per tile
constexpr int kKeys = 64;                 // keys per step
constexpr int kSlotBytes = kKeys * 128;   // 64 keys x 64 BF16 columns
constexpr int kQBytes = kRows * 128;      // 128 rows x 64 BF16 columns
constexpr int kMaxChunks = 9;             // 64-column chunks of a cache row
constexpr int kGroup = 4;                 // value chunks of a CTA (its columns of O)
constexpr int kOthers = kMaxChunks - kGroup;  // the chunks that only S needs, two steps of them in the ring
constexpr int kPairs = 5;                 // pairs of value chunks in the ring: two and a half steps
constexpr int kTmemChunks = 6;            // chunks of Q kept in TMEM
constexpr int kHalf = 256;                // columns of O per CTA
constexpr int kThreads = 192;
constexpr int kMmaWarp = 4, kLoadWarp = 5;
constexpr int kMiscBytes = 1024;
constexpr int kSmemQ = (kMaxChunks - kTmemChunks) * kQBytes, kSmemX = 2 * kOthers * kSlotBytes;
constexpr int kSmemY = 2 * kPairs * kSlotBytes;
constexpr int kSmem = 1024 + kMiscBytes + kSmemQ + kQBytes + kSmemX + kSmemY;
static_assert(kSmem <= 232448, "227 KB");
constexpr uint32_t kColO = 0, kColQ = 256, kColS = 448;
constexpr uint64_t kTimeoutNs = 1000000000ull;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;             // log2 of the largest P
// Own pages are asked of L2 this many steps before their copies: the ring holds two steps, which cover the
// latency of L2 but not that of HBM.
constexpr int kFetch = 2;
constexpr int kOverhead = 7;              // a tile's start and end, in key steps
constexpr int kMinRun = 8;                // shortest run worth a CTA pair, in key steps

// What the join kernel needs to know of the cut (start of the workspace).
struct Cut {
    int64_t prefix_cost;  // cost of the prefix tiles
    int64_t run;          // cost per unit
    int32_t shared;       // keys of the shared prefix (a multiple of kKeys; 0: none)
    int32_t source;       // batch row whose pages hold it
};

struct CacheParams {
    const uint16_t* q;
    const uint16_t* cache;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* seqs;
    const int32_t* shared_len;
    uint16_t* out;
    float* lse;
    int32_t* status;
    Cut* cut;           // workspace: the cut,
    int64_t* bases;     //   cost of the sequences before each [B],
    float* part_o;      //   partial results [part rows][Lkv]
    float* part_lse;    //   and their log2-sum-exp [part rows]
    int B, H, Lkv, C, page_size, table_rows, max_pages, num_rows, num_pages, box;
    int row_tiles, head_tiles, halves, units;
    float scale;
};

// Table row (-1: none) and length of batch row b.
__device__ __forceinline__ int batch_len(const CacheParams& p, int b, int* row, int* bits) {
    const int s = p.seqs ? p.seqs[b] : b;
    if (s < 0 || s >= p.table_rows) {
        *row = -1;
        *bits |= kStatusSeqRange;
        return 0;
    }
    *row = s;
    const int n = p.lens[s], cap = p.max_pages * p.page_size;
    if (n < 0 || n > cap) *bits |= kStatusSeqRange;
    return n < 0 ? 0 : n > cap ? cap : n;
}

// Keys of batch row b before its own ones, and steps over its own.
__device__ __forceinline__ int own_start(int len, int shared) { return len >= shared ? shared : 0; }
__device__ __forceinline__ int own_steps(int len, int shared) {
    return (len - own_start(len, shared) + kKeys - 1) / kKeys;
}
__device__ __forceinline__ int64_t seq_cost(const CacheParams& p, int steps) {
    return steps ? static_cast<int64_t>(p.head_tiles) * (steps + kOverhead) : 0;
}

// The steps [*j0, *j1) of a tile of `steps` at cost `base` that the costs
// [from, to) cover.
__device__ __forceinline__ void covered(int64_t base, int steps, int64_t from, int64_t to, int* j0, int* j1) {
    const int64_t a = from - base - kOverhead, e = to - base - kOverhead;
    *j0 = a < 0 ? 0 : a > steps ? steps : static_cast<int>(a);
    *j1 = e < 0 ? 0 : e > steps ? steps : static_cast<int>(e);
}

// First row of the partial results of (tile, unit): the tile's rows in a list
// of all tiles' rows, moved on by a tile per unit, so that no two overlap.
__device__ __forceinline__ int64_t part_row(const CacheParams& p, int64_t tile_row, int unit) {
    return tile_row + static_cast<int64_t>(unit) * kRows;
}

struct Piece {
    int64_t part;    // first row of its partial result
    int row0, rows;  // rows of q
    int page_row;    // row of the page table
    int key0, end;   // first key of the first step, end of the keys
    int n;           // steps
    bool prefix, whole;  // whole: covers the tile's keys
};

// A unit's walk over its pieces; every role walks on its own.
struct Walk {
    int64_t at, end, prefix_cost, base;  // base: cost before batch row b
    int shared, source_row, b, len, row, unit;

    __device__ __forceinline__ void enter(const CacheParams& p) {
        int bits = 0;
        if (b < p.B) len = batch_len(p, b, &row, &bits);
    }

    // (Out of line: one copy for the three roles keeps their loops in the instruction cache.)
    __device__ __noinline__ bool next(const CacheParams& p, Piece* x) {
        while (at < end) {
            int64_t tile_base, tile_row;
            int steps;
            if (at < prefix_cost) {
                steps = shared / kKeys;
                const int t = static_cast<int>(at / (steps + kOverhead));
                tile_base = static_cast<int64_t>(t) * (steps + kOverhead);
                x->row0 = t * kRows;
                x->rows = min(kRows, p.B * p.H - x->row0);
                tile_row = x->row0;
                x->page_row = source_row;
                x->key0 = 0;
                x->end = shared;
                x->prefix = true;
            } else {
                steps = own_steps(len, shared);
                while (b < p.B && at >= base + seq_cost(p, steps)) {
                    base += seq_cost(p, steps);
                    ++b;
                    enter(p);
                    steps = own_steps(len, shared);
                }
                if (b >= p.B) return false;
                const int ht = static_cast<int>((at - base) / (steps + kOverhead));
                tile_base = base + static_cast<int64_t>(ht) * (steps + kOverhead);
                x->row0 = b * p.H + ht * kRows;
                x->rows = min(kRows, p.H - ht * kRows);
                tile_row = static_cast<int64_t>(p.row_tiles) * kRows + x->row0;
                x->page_row = row;
                x->key0 = own_start(len, shared);
                x->end = len;
                x->prefix = false;
            }
            int j0, j1;
            covered(tile_base, steps, at, end, &j0, &j1);
            const int64_t tile_end = tile_base + steps + kOverhead;
            at = tile_end < end ? tile_end : end;
            if (j1 <= j0) continue;
            x->part = part_row(p, tile_row, unit);
            x->key0 += j0 * kKeys;
            x->n = j1 - j0;
            x->whole = x->n == steps;
            return true;
        }
        return false;
    }
};

struct Shared {
    uint64_t x_full[2], x_empty[2], y_full[kPairs], y_empty[kPairs];  // other chunks by step, value chunks by pair
    uint64_t q_full, s_full, s_free, p_full, pv_done, drain;
    uint32_t tmem;
    int abort_flag;
    int64_t scan[kThreads / 32];
    int64_t total, first_base;
    int first_b, sharers, source, shared;
};
static_assert(sizeof(Shared) <= kMiscBytes, "");

// Exclusive prefix sum over the block; *total: the block's sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* scratch, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    int64_t before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += scratch[w];
        sum += scratch[w];
    }
    *total = sum;
    return before + x - v;
}

// The cut, and where this unit's run starts.  Every CTA computes it from the
// lengths (a few hundred loads at most batch sizes); CTA 0 leaves it in the
// workspace for the join.  False: the unit has no run.
__device__ __forceinline__ bool make_cut(const CacheParams& p, int unit, Shared* sh, Walk* w) {
    const bool writer = blockIdx.x == 0;
    int bits = 0, row, first_row = -1;
    // this thread's row of the first kThreads: read once, beside the shared length
    const int first_len = threadIdx.x < p.B ? batch_len(p, threadIdx.x, &first_row, &bits) : 0;
    auto len_of = [&](int b) {
        if (b == static_cast<int>(threadIdx.x)) return first_len;
        return b < p.B ? batch_len(p, b, &row, &bits) : 0;
    };
    // who shares the prefix
    int shared = p.shared_len ? *p.shared_len : 0;
    const int cap = p.max_pages * p.page_size;
    shared = shared < 0 ? 0 : (shared > cap ? cap : shared) / kKeys * kKeys;
    if (threadIdx.x == 0) sh->sharers = 0, sh->source = p.B;
    __syncthreads();
    if (shared > 0) {
        int count = 0, first = p.B;
        for (int b = threadIdx.x; b < p.B; b += kThreads)
            if (len_of(b) >= shared) ++count, first = min(first, b);
        if (count) {
            atomicAdd(&sh->sharers, count);
            atomicMin(&sh->source, first);
        }
        __syncthreads();
        if (sh->sharers < 2) shared = 0;
    }
    const int source = sh->source;
    const int64_t prefix = shared ? static_cast<int64_t>(p.row_tiles) * (shared / kKeys + kOverhead) : 0;
    int64_t total = prefix, sum;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        const int len = len_of(b);
        const int64_t mine = b < p.B ? seq_cost(p, own_steps(len, shared)) : 0;
        const int64_t before = total + block_scan(mine, sh->scan, &sum);
        if (writer && b < p.B) p.bases[b] = before;
        total += sum;
    }
    int64_t run = (total + p.units - 1) / p.units;
    if (run < kMinRun) run = kMinRun;
    if (writer) {
        if (threadIdx.x == 0) *p.cut = Cut{prefix, run, shared, source};
        raise_status(p.status, bits);
    }
    w->unit = unit;
    w->at = run * unit;
    w->end = w->at + run < total ? w->at + run : total;
    w->prefix_cost = prefix;
    w->shared = shared;
    w->b = 0;
    w->base = prefix;
    w->len = w->row = 0;
    w->source_row = -1;
    if (w->at >= total) return false;
    if (shared) batch_len(p, source, &w->source_row, &bits);
    if (w->at >= prefix) {  // the batch row that holds `at`
        if (p.B <= kThreads) {
            const int b = threadIdx.x;
            const int len = len_of(b);
            const int64_t mine = b < p.B ? seq_cost(p, own_steps(len, shared)) : 0;
            const int64_t before = prefix + block_scan(mine, sh->scan, &sum);
            if (mine && w->at >= before && w->at < before + mine) sh->first_b = b, sh->first_base = before;
        } else {
            int64_t base = prefix;
            for (int b0 = 0; b0 < p.B; b0 += kThreads) {
                const int b = b0 + threadIdx.x;
                const int len = len_of(b);
                const int64_t mine = b < p.B ? seq_cost(p, own_steps(len, shared)) : 0;
                const int64_t before = base + block_scan(mine, sh->scan, &sum);
                if (mine && w->at >= before && w->at < before + mine) sh->first_b = b, sh->first_base = before;
                base += sum;
                if (base > w->at) break;
            }
        }
        __syncthreads();
        w->b = sh->first_b;
        w->base = sh->first_base;
    }
    w->enter(p);
    return true;
}

__global__ void __launch_bounds__(kThreads, 1)
    mla_attend_cache_kernel(const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_4,
                            const __grid_constant__ CUtensorMap tm_2, const CacheParams p) {
    extern __shared__ uint8_t raw[];
    const uint32_t raw_at = smem_u32(raw);
    const uint32_t pad = (1024u - (raw_at & 1023u)) & 1023u;
    const int chunks = (p.C + 63) / 64;
    const uint32_t sm_q = raw_at + pad, sm_p = sm_q + kSmemQ, sm_x = sm_p + kQBytes, sm_y = sm_x + kSmemX;
    Shared* sh = reinterpret_cast<Shared*>(raw + pad + kSmemQ + kQBytes + kSmemX + kSmemY);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x / p.halves, half = blockIdx.x % p.halves;
    // This CTA's columns of O lie in value chunks 4 half .. + 3 of a cache row; the others only go into S.
    const int dv0 = half * kHalf, dv = min(kHalf, p.Lkv - dv0);
    const int v0 = half * kGroup, nvc = min(kGroup, chunks - v0), nx = chunks - nvc, pairs = (nvc + 1) / 2;
    auto other = [&](int i) { return i < v0 ? i : i + nvc; };  // chunk of ring place i
    // Place of a chunk of Q: 0-5 in TMEM, the value chunks first, 6-8 in shared memory.
    auto q_place = [&](int ck) { return ck >= 2 * kGroup ? ck : (ck ^ v0); };

    Walk walk;
    if (!make_cut(p, unit, sh, &walk)) return;
    if (warp == kLoadWarp && lane == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh->x_full[i]), 1);
            mbar_init(smem_u32(&sh->x_empty[i]), 1);
        }
        for (int i = 0; i < kPairs; ++i) {
            mbar_init(smem_u32(&sh->y_full[i]), 1);
            mbar_init(smem_u32(&sh->y_empty[i]), 1);
        }
        mbar_init(smem_u32(&sh->q_full), kRows);
        mbar_init(smem_u32(&sh->s_full), 1);
        mbar_init(smem_u32(&sh->s_free), kRows);
        mbar_init(smem_u32(&sh->p_full), kRows);
        mbar_init(smem_u32(&sh->pv_done), 1);
        mbar_init(smem_u32(&sh->drain), 1);
        sh->abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(&sh->tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    const volatile int* abort_flag = &sh->abort_flag;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_wait_lean(smem_u32(bar), parity & 1u, kTimeoutNs, abort_flag);
    };
    bool ok = true;
    int step = 0;  // key steps so far, over all pieces: the phase of every barrier
    Piece x;

    if (warp < 4) {
        // ------------------------------------------------------------ softmax
        const int r = threadIdx.x;
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        const float c = p.scale * kLog2e;
        auto load_q = [&](const Piece& y) {
            // Q: places 0-5 to TMEM, by way of the warp's rows of the shared-memory places 6-8, and those then to
            // shared memory in the swizzled layout of a TMA box.  A warp reads four rows of 128 bytes at a time.
            const uint4* q = reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(y.row0) + warp * 32) * p.C);
            const int pitch = p.C / 8, wrows = y.rows - warp * 32;
#pragma unroll 1
            for (int place0 = 0; place0 < kMaxChunks; place0 += 3) {
                uint4 w[24];
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    const int ck = q_place(place0 + e);  // its own inverse
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int row = i * 4 + (lane >> 3), col = ck * 8 + (lane & 7);
                        w[8 * e + i] = row < wrows && col < pitch ? q[row * pitch + col] : make_uint4(0, 0, 0, 0);
                    }
                }
                const uint32_t base = sm_q + warp * 32 * 128;
                __syncwarp();  // the round before has been read
#pragma unroll
                for (int e = 0; e < 3; ++e)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int row = i * 4 + (lane >> 3);
                        st_shared_v4(base + e * kQBytes + row * 128 + (((lane & 7) ^ (row & 7)) << 4), w[8 * e + i].x,
                                     w[8 * e + i].y, w[8 * e + i].z, w[8 * e + i].w);
                    }
                if (place0 < kTmemChunks) {
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 3; ++e) {
                        uint32_t t[32];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            ld_shared_v4(base + e * kQBytes + lane * 128 + ((i ^ (lane & 7)) << 4), t[4 * i], t[4 * i + 1],
                                         t[4 * i + 2], t[4 * i + 3]);
                        tmem_st32_raw(tmem + lanes + kColQ + (place0 + e) * 32, t);
                    }
                }
            }
            tmem_wait_st();
            fence_proxy_async_shared();
            tc_fence_before();
            mbar_arrive(smem_u32(&sh->q_full));
        };
        bool more = walk.next(p, &x);
        if (more) load_q(x);
        while (more && ok) {
            const Piece now = x;
            const bool mine = r < now.rows;
            float m = -INFINITY, ms = 0.f, l = 0.f;
            for (int j = 0; j < now.n; ++j, ++step) {
                ok = __all_sync(~0u, wait(&sh->s_full, step));
                if (!ok) break;
                tc_fence_after();
                uint32_t s[kKeys];
                float mt = tmem_ld64_max(tmem + lanes + kColS, s);  // of the row
                tc_fence_before();
                mbar_arrive(smem_u32(&sh->s_free));
                const int left = now.end - now.key0 - j * kKeys;
                if (left < kKeys) {
#pragma unroll
                    for (int i = 0; i < kKeys; ++i)
                        if (i >= left) s[i] = 0xFF800000u;
                    mt = -INFINITY;
#pragma unroll
                    for (int i = 0; i < kKeys; ++i) mt = fmaxf(mt, __uint_as_float(s[i]));
                }
                const bool grow = mt > m && (m == -INFINITY || mt * c > ms + kSlack);
                float alpha = 1.f;
                if (__any_sync(~0u, grow)) {
                    if (mt > m) {
                        const float next = mt * c;
                        if (m != -INFINITY) alpha = ex2(ms - next);
                        m = mt;
                        ms = next;
                    }
                    l *= alpha;
                }
                const uint64_t cc = pk2(c, c), mm = pk2(-ms, -ms);
                uint64_t sum0 = 0, sum1 = 0;
                uint32_t w[kKeys / 2];
#pragma unroll
                for (int i = 0; i < kKeys; i += 4) {
                    float e0, e1, e2, e3;
                    upk2(fma2(pk2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), cc, mm), e0, e1);
                    upk2(fma2(pk2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), cc, mm), e2, e3);
                    e0 = ex2(e0), e1 = ex2(e1), e2 = ex2(e2), e3 = ex2(e3);
                    sum0 = add2(sum0, pk2(e0, e1));
                    sum1 = add2(sum1, pk2(e2, e3));
                    w[i >> 1] = pack_bf16x2(e0, e1);
                    w[(i >> 1) + 1] = pack_bf16x2(e2, e3);
                }
                float a0, a1;
                upk2(add2(sum0, sum1), a0, a1);
                l += a0 + a1;
                // the step before has read P, and O is at rest
                if (step > 0) {
                    ok = __all_sync(~0u, wait(&sh->pv_done, step - 1));
                    if (!ok) break;
                    tc_fence_after();
                }
                if (j > 0 && __any_sync(~0u, alpha != 1.f)) {
#pragma unroll 1
                    for (int d = 0; d < dv; d += 16) {
                        float o[16];
                        tmem_ld16(tmem + lanes + kColO + d, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= alpha;
                        tmem_st16(tmem + lanes + kColO + d, o);
                    }
                }
                const uint32_t dst = sm_p + r * 128;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    st_shared_v4(dst + ((i ^ (r & 7)) << 4), w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                if (left < kKeys) {
                    // rows behind the end may hold anything: as values they have to be zero
                    for (int k = r; k < (kKeys - left) * nvc * 8; k += kRows) {
                        const int row = left + k / (nvc * 8), in = k % (nvc * 8), c2 = in / 8;
                        const int slot = (step * pairs + c2 / 2) % kPairs * 2 + (c2 & 1);
                        st_shared_v4(sm_y + slot * kSlotBytes + row * 128 + (in & 7) * 16, 0, 0, 0, 0);
                    }
                }
                fence_proxy_async_shared();
                tc_fence_before();
                mbar_arrive(smem_u32(&sh->p_full));
            }
            if (!ok) break;
            // every score of this piece is done: the next piece's Q can take Q's place while P V finishes
            more = walk.next(p, &x);
            if (more) load_q(x);
            ok = __all_sync(~0u, wait(&sh->pv_done, step - 1));
            if (!ok) break;
            tc_fence_after();
            // A row whose keys this piece covers alone is finished; the others leave a partial result.
            bool direct = now.whole;
            const int b = (now.row0 + r) / p.H;
            if (walk.shared && direct && mine) {
                int trow, bits = 0;
                const int len = batch_len(p, b, &trow, &bits);
                direct = now.prefix ? len == walk.shared : len < walk.shared;
            }
            // A warp's rows pass through its part of P's buffer, 128 bytes of each at a time, so that it stores
            // four rows' whole lines at once: 64 columns of finished rows, 32 of partial ones.
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int64_t at = static_cast<int64_t>(now.row0) + r;
            const uint32_t direct_rows = __ballot_sync(~0u, direct && mine), part_rows = __ballot_sync(~0u, !direct && mine);
            const uint32_t stage = sm_p + warp * 32 * 128;
            auto put = [&](int i, uint32_t a, uint32_t b, uint32_t c2, uint32_t d2) {
                st_shared_v4(stage + lane * 128 + ((i ^ (lane & 7)) << 4), a, b, c2, d2);
            };
            auto flush = [&](uint8_t* rows, int64_t row_bytes, uint32_t which, int bytes) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = i * 4 + (lane >> 3), col = (lane & 7) * 16;
                    uint4 v;
                    ld_shared_v4(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4), v.x, v.y, v.z, v.w);
                    if ((which >> row & 1u) && col < bytes) *reinterpret_cast<uint4*>(rows + row * row_bytes + col) = v;
                }
                __syncwarp();
            };
            uint8_t* out = reinterpret_cast<uint8_t*>(p.out + (static_cast<int64_t>(now.row0) + warp * 32) * p.Lkv + dv0);
            uint8_t* part = reinterpret_cast<uint8_t*>(p.part_o + (now.part + warp * 32) * p.Lkv + dv0);
#pragma unroll 1
            for (int d = 0; d < dv; d += 64) {
                uint32_t o[64];  // (what lies behind dv is not stored)
                tmem_ld64_raw(tmem + lanes + kColO + d, o);
#pragma unroll
                for (int i = 0; i < 64; ++i) o[i] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(o[i]) * inv);
                const int left = dv - d;
                if (part_rows) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (k * 32 >= left) break;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            put(i, o[k * 32 + 4 * i], o[k * 32 + 4 * i + 1], o[k * 32 + 4 * i + 2], o[k * 32 + 4 * i + 3]);
                        flush(part + (d + k * 32) * 4, p.Lkv * 4, part_rows, (left - k * 32) * 4);
                    }
                }
                if (direct_rows) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * e]), __uint_as_float(o[8 * i + 2 * e + 1]));
                        put(i, w[0], w[1], w[2], w[3]);
                    }
                    flush(out + d * 2, p.Lkv * 2, direct_rows, left * 2);
                }
            }
            if (mine && half == 0) {
                const float lg = l == 0.f ? -INFINITY : ms + log2f(l);
                if (!direct) p.part_lse[now.part + r] = lg;
                else if (p.lse) p.lse[at] = lg * kLn2;
            }
            tc_fence_before();
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- MMA
        if (elect_one()) {
            const uint32_t idesc_s = idesc_bf16_f32(kRows, kKeys);
            const uint32_t x_full = smem_u32(&sh->x_full[0]), x_empty = smem_u32(&sh->x_empty[0]);
            const uint32_t y_full = smem_u32(&sh->y_full[0]), y_empty = smem_u32(&sh->y_empty[0]);
            constexpr uint32_t kSlotStep = kSlotBytes >> 4, kQStep = kQBytes >> 4;
            const uint64_t dq = smem_desc_sw128(sm_q), dp = smem_desc_sw128(sm_p);
            const uint64_t dx = smem_desc_sw128(sm_x), dy = smem_desc_sw128(sm_y);
            const uint64_t dvals = smem_desc_sw128_mn(sm_y, kSlotBytes);
            const uint32_t tq = tmem + kColQ, ts = tmem + kColS, to = tmem + kColO;
            const bool widest = p.C == 64 * kMaxChunks;
            auto look = [&](uint32_t bar, uint32_t parity) {
                ok = ok && mbar_wait_lean(bar, parity, kTimeoutNs, abort_flag);
                tc_fence_after();
                return ok;
            };
            // S (+)= Q K^T over one chunk of any width
            auto chunk_mma = [&](int ck, uint64_t b, bool first) {
                const int place = q_place(ck), ks = min(4, p.C / 16 - ck * 4);
#pragma unroll 1
                for (int e = 0; e < ks; ++e) {
                    const uint32_t acc = !(first && e == 0);
                    if (place < kTmemChunks) mma_bf16_ts(ts, tq + place * 32 + e * 8, b + 2 * e, idesc_s, acc);
                    else mma_bf16(ts, dq + (place - kTmemChunks) * kQStep + 2 * e, b + 2 * e, idesc_s, acc);
                }
            };
            int y = 0;  // ring place and parity of the next pair of value chunks
            uint32_t yp = 0;
            int at[2] = {0, 0}, was[2] = {0, 0};  // places of this step's and the step before's pairs
            const uint32_t id[2] = {idesc_bf16_f32(kRows, min(dv, 128)) | kIdescBMnMajor,
                                    idesc_bf16_f32(kRows, dv > 128 ? dv - 128 : 16) | kIdescBMnMajor};
            for (int piece = 0; walk.next(p, &x); ++piece) {
                const int n = x.n;
                look(smem_u32(&sh->q_full), piece & 1);
                // Per round: the scores of step t, then P V of step t - 1, whose softmax ran meanwhile.
#pragma unroll 1
                for (int t = 0; t <= n && ok; ++t) {
                    const int st = step + t;
                    was[0] = at[0], was[1] = at[1];
                    if (t < n) {
                        if (st > 0 && !look(smem_u32(&sh->s_free), (st - 1) & 1)) break;
                        if (nx && !look(x_full + 8 * (st & 1), (st >> 1) & 1)) break;
                        const uint64_t b = dx + (st & 1) * (kOthers * kSlotStep);
                        if (widest) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                mma_bf16_ts(ts, tq + 128 + k * 8, b + (k >> 2) * kSlotStep + 2 * (k & 3), idesc_s, k > 0);
#pragma unroll
                            for (int k = 8; k < 20; ++k)
                                mma_bf16(ts, dq + ((k >> 2) - 2) * kQStep + 2 * (k & 3),
                                         b + (k >> 2) * kSlotStep + 2 * (k & 3), idesc_s, 1);
                        } else {
                            for (int i = 0; i < nx; ++i) chunk_mma(other(i), b + i * kSlotStep, i == 0);
                        }
                        if (nx) mma_commit(x_empty + 8 * (st & 1));
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (e >= pairs) break;
                            if (!look(y_full + 8 * y, yp)) break;
                            const uint64_t v = dy + y * (2 * kSlotStep);
                            if (widest) {
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    mma_bf16_ts(ts, tq + e * 64 + k * 8, v + (k >> 2) * kSlotStep + 2 * (k & 3), idesc_s, 1);
                            } else {
                                for (int i = 0; i < 2 && 2 * e + i < nvc; ++i)
                                    chunk_mma(v0 + 2 * e + i, v + i * kSlotStep, nx == 0 && e == 0 && i == 0);
                            }
                            at[e] = y;
                            if (++y == kPairs) y = 0, yp ^= 1u;
                        }
                        if (!ok) break;
                        mma_commit(smem_u32(&sh->s_full));
                    }
                    if (t > 0) {
                        if (!look(smem_u32(&sh->p_full), (st - 1) & 1)) break;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (e >= pairs) break;
                            if (e * 128 < dv) {  // (a pair may hold no value column)
                                const uint64_t v = dvals + was[e] * (2 * kSlotStep);
#pragma unroll
                                for (int k = 0; k < kKeys / 16; ++k)
                                    mma_bf16(to + e * 128, dp + 2 * k, v + k * (2048 >> 4), id[e], t > 1 || k > 0);
                            }
                            mma_commit(y_empty + 8 * was[e]);
                        }
                        mma_commit(smem_u32(&sh->pv_done));
                    }
                }
                if (!ok) break;
                step += n;
            }
            if (!ok) {  // no MMA may still run when the CTA leaves
                mma_commit(smem_u32(&sh->drain));
                mbar_wait(smem_u32(&sh->drain), 0, kTimeoutNs, nullptr);
            }
        }
    } else {
        // --------------------------------------------------------------- TMA
        // The lanes look up the rows of 32 boxes at a time; one thread issues the copies.
        const int per = kKeys / p.box, batch = 32 / per;  // boxes per step, steps per lookup
        const bool lead = elect_one();
        const uint32_t x_full = smem_u32(&sh->x_full[0]), x_empty = smem_u32(&sh->x_empty[0]);
        const uint32_t y_full = smem_u32(&sh->y_full[0]), y_empty = smem_u32(&sh->y_empty[0]);
        const uint32_t box_bytes = p.box * 128;
        const bool whole = per == 1 && p.C == 64 * kMaxChunks;
        int bits = 0, y = 0, xs = 0, ys = 0;  // xs, ys: barriers armed
        uint32_t yp = 1;
        // `count` chunks from chunk `ck` on to `dst`, box by box
        auto copy = [&](uint32_t dst, uint32_t bar, int ck, int count, int rows, int box0) {
#pragma unroll 1
            for (int e = 0; e < per; ++e) {
                const int row = __shfl_sync(~0u, rows, box0 + e);
                if (lead)
                    for (int c = 0; c < count; ++c)
                        tma_load_3d(dst + e * box_bytes + c * kSlotBytes, &tm_c, bar, (ck + c) * 64, 0, row);
            }
        };
        while (ok && walk.next(p, &x)) {
            const int n = x.n, key0 = x.key0, end = x.end;
            const int32_t* row_table = p.table + static_cast<int64_t>(x.page_row) * p.max_pages;
            // first row of box `lane` of the batch that starts at step j; a row outside the cache reads as zeros
            auto look_up = [&](int j) {
                const int key = key0 + (j * per + lane) * p.box;
                if (j * per + lane >= n * per || key >= end) return p.num_rows;
                const int page = row_table[key / p.page_size];
                if (page >= 0 && page < p.num_pages) return page * p.page_size + key % p.page_size;
                bits |= kStatusPageRange;
                return p.num_rows;
            };
            // Asks L2 for this lane's box of cache rows, which lie in one piece of memory.
            auto fetch = [&](int row) {
                if (row < p.num_rows) bulk_prefetch_l2(p.cache + static_cast<int64_t>(row) * p.C, p.box * p.C * 2);
            };
            int rows = look_up(0), ahead = batch < n ? look_up(batch) : p.num_rows;
            const bool far = !x.prefix && lane / per < batch;
            if (far && lane / per < kFetch && (lane / per & (p.halves - 1)) == half) fetch(rows);
#pragma unroll 1
            for (int j0 = 0; j0 < n && ok; j0 += batch) {
                if (j0) {
                    rows = ahead;
                    ahead = j0 + batch < n ? look_up(j0 + batch) : p.num_rows;
                }
                const int steps = min(batch, n - j0);
#pragma unroll 1
                for (int j = 0; j < steps && ok; ++j, ++step) {
                    const int st = step & 1;
                    const int row0 = __shfl_sync(~0u, rows, j * per);
                    // step j + kFetch of the run, alternately by the two CTAs
                    if (far && lane / per == (j + kFetch) % batch && (j & (p.halves - 1)) == half)
                        fetch(j + kFetch < batch ? rows : ahead);
                    if (nx) {
                        const uint32_t bar = x_full + 8 * st, dst = sm_x + st * kOthers * kSlotBytes;
                        if (lead) {
                            ok = mbar_wait_lean(x_empty + 8 * st, ((step >> 1) & 1) ^ 1, kTimeoutNs, abort_flag);
                            if (ok) {
                                mbar_arrive_expect_tx(bar, nx * kSlotBytes);
                                ++xs;
                                if (whole) {
                                    tma_load_3d(dst, &tm_4, bar, 0, row0, v0 ^ kGroup);
                                    tma_load_3d(dst + kGroup * kSlotBytes, &tm_c, bar, 2 * kGroup * 64, 0, row0);
                                }
                            }
                        }
                        ok = __all_sync(~0u, ok);
                        if (!ok) break;
                        if (!whole) {
                            copy(dst, bar, other(0), min(nx, v0 ? v0 : nx), rows, j * per);
                            if (v0 && nx > v0) copy(dst + v0 * kSlotBytes, bar, other(v0), nx - v0, rows, j * per);
                        }
                    }
#pragma unroll 1
                    for (int e = 0; e < pairs; ++e) {
                        const uint32_t bar = y_full + 8 * y, dst = sm_y + y * 2 * kSlotBytes;
                        const int count = min(2, nvc - 2 * e);
                        if (lead) {
                            ok = mbar_wait_lean(y_empty + 8 * y, yp, kTimeoutNs, abort_flag);
                            if (ok) {
                                mbar_arrive_expect_tx(bar, count * kSlotBytes);
                                ++ys;
                                if (whole) tma_load_3d(dst, &tm_2, bar, 0, row0, v0 + 2 * e);
                            }
                        }
                        ok = __all_sync(~0u, ok);
                        if (!ok) break;
                        if (!whole) copy(dst, bar, v0 + 2 * e, count, rows, j * per);
                        if (++y == kPairs) y = 0, yp ^= 1u;
                    }
                }
            }
        }
        // no copy may still be landing when the CTA leaves
        if (lead) {
            for (int u = max(xs - 2, 0); u < xs; ++u) mbar_wait(x_full + 8 * (u & 1), (u >> 1) & 1, kTimeoutNs, nullptr);
            for (int u = max(ys - kPairs, 0); u < ys; ++u)
                mbar_wait(y_full + 8 * (u % kPairs), (u / kPairs) & 1, kTimeoutNs, nullptr);
        }
        if (bits) raise_status(p.status, bits);
    }
    if (!ok) {
        sh->abort_flag = 1;
        raise_status(p.status, kStatusWaitTimeout);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the partial results of each row, in the order of the cut; a row with
// one piece was finished by that piece.  One warp per row.
__global__ void __launch_bounds__(128) mla_attend_join_kernel(const CacheParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= static_cast<int64_t>(p.B) * p.H) return;
    pdl_wait();
    const Cut cut = *p.cut;
    const int b = static_cast<int>(row / p.H), h = static_cast<int>(row % p.H);
    int trow, bits = 0;
    const int len = batch_len(p, b, &trow, &bits);
    // the tile of the prefix, the tile of the own keys: cost, steps, units that hold steps of it, partial row
    int64_t base[2], part[2];
    int steps[2], u0[2], u1[2], count = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (k == 0) {
            steps[0] = len >= cut.shared ? cut.shared / kKeys : 0;
            base[0] = row / kRows * (cut.shared / kKeys + kOverhead);
            part[0] = row;
        } else {
            steps[1] = own_steps(len, cut.shared);
            base[1] = p.bases[b] + static_cast<int64_t>(h / kRows) * (steps[1] + kOverhead);
            part[1] = static_cast<int64_t>(p.row_tiles) * kRows + row;
        }
        u0[k] = static_cast<int>((base[k] + kOverhead) / cut.run);
        u1[k] = steps[k] ? static_cast<int>((base[k] + kOverhead + steps[k] - 1) / cut.run) : u0[k] - 1;
        count += u1[k] - u0[k] + 1;
    }
    if (count == 1) return;
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        for (int u = u0[k]; u <= u1[k]; ++u) {
            const float v = p.part_lse[part_row(p, part[k], u)];
            top = v != v ? v : fmaxf(top, v);
        }
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    float4 acc[4] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k)
        for (int u = u0[k]; u <= u1[k]; ++u) {
            const int64_t at = part_row(p, part[k], u);
            const float w = exp2f(p.part_lse[at] - ref);
            sum += w;
            const float4* o = reinterpret_cast<const float4*>(p.part_o + at * p.Lkv);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if ((i * 32 + lane) * 4 < p.Lkv) {
                    const float4 v = o[i * 32 + lane];
                    acc[i].x = fmaf(w, v.x, acc[i].x), acc[i].y = fmaf(w, v.y, acc[i].y);
                    acc[i].z = fmaf(w, v.z, acc[i].z), acc[i].w = fmaf(w, v.w, acc[i].w);
                }
        }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if ((i * 32 + lane) * 4 < p.Lkv)
            reinterpret_cast<uint2*>(p.out + row * p.Lkv)[i * 32 + lane] =
                make_uint2(pack_bf16x2(acc[i].x * inv, acc[i].y * inv), pack_bf16x2(acc[i].z * inv, acc[i].w * inv));
    if (lane == 0 && p.lse) p.lse[row] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * kLn2;
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

// Workspace: the cut, the costs before each sequence, the partial results.
struct Layout {
    int row_tiles, head_tiles, halves, units;
    size_t bases, part_lse, part_o, bytes;
};

Layout layout(const mla_prolog_cache_dims& d, int sms) {
    Layout y;
    const int64_t rows = static_cast<int64_t>(d.batch) * d.num_heads;
    y.row_tiles = static_cast<int>((rows + kRows - 1) / kRows);
    y.head_tiles = (d.num_heads + kRows - 1) / kRows;
    y.halves = d.kv_lora_rank > kHalf ? 2 : 1;
    y.units = sms / y.halves > 0 ? sms / y.halves : 1;
    auto round = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t parts = static_cast<size_t>(y.row_tiles) * kRows + rows + static_cast<size_t>(y.units) * kRows;
    y.bases = round(sizeof(Cut));
    y.part_lse = y.bases + round(sizeof(int64_t) * d.batch);
    y.part_o = y.part_lse + round(sizeof(float) * parts);
    y.bytes = y.part_o + sizeof(float) * parts * d.kv_lora_rank;
    return y;
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

}  // namespace
}  // namespace mlap

using namespace mlap;

extern "C" {

int mla_prolog_attend_cache_workspace(const mla_prolog_cache_dims* d, size_t* bytes) {
    if (!d || !bytes) return MLA_ERR_INVALID_ARG;
    *bytes = 0;
    int rc = check_cache_dims(*d), sms;
    if (rc != MLA_OK || (rc = current_sm103(&sms)) != MLA_OK) return rc;
    *bytes = layout(*d, sms).bytes;
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
        (status && !ptr_ok(status, 4)) || !ptr_ok(workspace, 16))
        return MLA_ERR_INVALID_ARG;
    int sms;
    if ((rc = current_sm103(&sms)) != MLA_OK) return rc;
    const Layout y = layout(*d, sms);
    if (workspace_bytes < y.bytes) return MLA_ERR_INVALID_ARG;
    const int C = d->kv_lora_rank + d->rope_dim, box = gcd(d->page_size, kKeys);
    const int64_t rows = d->num_pages * d->page_size;
    CUtensorMap tm, tm4, tm2;
    // an empty cache has no valid page: every read is outside the map, which then only needs a valid address
    const void* base = rows ? kv_cache : q;
    bool good = encode_bf16_3d(&tm, base, C, 1, rows ? rows : 1, 1, box);
    // the same rows by whole chunks, [chunk][row][64], four or two of them in one copy
    const bool widest = C == 64 * kMaxChunks;
    tm4 = tm2 = tm;
    if (widest)
        good = good && encode_bf16_chunks(&tm4, base, C, rows ? rows : 1, box, 4) &&
               encode_bf16_chunks(&tm2, base, C, rows ? rows : 1, box, 2);
    if (!good) return report_cuda(cudaErrorInvalidValue, "tensor maps of attend_cache");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    CacheParams p{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(kv_cache), page_table, seq_lens, seqs, shared_len, static_cast<uint16_t*>(out),
                  lse, status, reinterpret_cast<Cut*>(ws), reinterpret_cast<int64_t*>(ws + y.bases),
                  reinterpret_cast<float*>(ws + y.part_o), reinterpret_cast<float*>(ws + y.part_lse), d->batch,
                  d->num_heads, d->kv_lora_rank, C, d->page_size, d->table_rows, d->max_pages,
                  static_cast<int>(rows ? rows : 1), static_cast<int>(d->num_pages), box, y.row_tiles, y.head_tiles,
                  y.halves, y.units, d->scale};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = allow_smem(&mla_attend_cache_kernel, kSmem, &ready);
    if (e != cudaSuccess) return report_cuda(e, "mla_attend_cache_kernel attributes");
    mla_attend_cache_kernel<<<y.units * y.halves, kThreads, kSmem, st>>>(tm, tm4, tm2, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return report_cuda(e, "launch mla_attend_cache_kernel");
    const int64_t blocks = (static_cast<int64_t>(d->batch) * d->num_heads + 3) / 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, mla_attend_join_kernel, p);
    return e == cudaSuccess ? MLA_OK : report_cuda(e, "launch mla_attend_join_kernel");
}

}  // extern "C"
