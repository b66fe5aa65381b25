// One decoding step over the latent KV cache: mla_prolog_attend_cache.
//
// A tile is 128 query rows (sequence, head) that see the same keys: the rows
// of one sequence on its own pages, or, where that takes fewer steps, 128 rows
// of any sequences on the shared prefix, whose rows are then read and
// multiplied once per 128 rows instead of once per sequence.  Every key is one
// cache row of Lkv + R columns, of which the first Lkv are the value too.
//
//   S = Q K^T   128 x 64 keys, 576 deep     O += P V   128 x Lkv, 64 deep
//
// O of 128 rows x 512 columns in FP32 would fill the TMEM of an SM alone, so
// a pair of CTAs works on a tile (cta_group::2, M = 128): each holds 64 of its
// rows, and the tensor core spreads their columns over both halves of the
// lanes, so that O takes 256 columns and S 32.  Each CTA brings half of the
// operands that both multiply: for S half of the keys (all columns), for P V
// half of the value columns (all keys).  A lane's row is shared by two
// threads, 64 lanes apart, one for each half of the keys and of the value
// columns.
//
// The work is cut into as many equal runs of key steps as there are CTA pairs
// (a tile costs its steps and some more for its start and end); a run takes
// whole or partial tiles.  Partial results go to the workspace in FP32, and a
// second kernel joins them in the order of the cut.
//
// Roundings: P to BF16 for the product with V, out to BF16 once; scores,
// maxima, sums, partial results and lse are FP32.
//
// What bounds it: a step's products take the pair 1.42k cycles, a step in all
// 1.6 to 1.7k (0.78 us, in which 76 pairs read 5.6 MB: 7.2 TB/s, so that own
// pages of few heads run at the rate of memory); a tile's start and end ~3.5
// us, of which the copies of the next tile overlap all but the last products
// and the results' way out; a call's start 6 us and its join 3 to 13 us (see
// there).  V2-Lite (16 heads), 64 sequences of 1 to 4096: 48 us, 3.8 TB/s; V3
// (128 heads), 32 of 2000 to 32768: 147 us, 4.6 TB/s and 1100 TFLOP/s; 128 of 1
// to 1024 behind a prefix of 8192: 231 us, 1340 TFLOP/s; one sequence of 100:
// 12 us.
#include <cstdint>

#include "attend.cuh"
#include "attend_ptx.cuh"

namespace mlap {
namespace {

constexpr int kRows = 128;                // query rows per tile (64 per CTA)
constexpr int kKeys = 64;                 // keys per step
constexpr int kMaxChunks = 9;             // 64-column chunks of a cache row
constexpr int kMaxValues = 4;             // 64-column chunks of a CTA's value columns
constexpr int kQBytes = 64 * 128;         // a chunk of this CTA's rows of Q,
constexpr int kKBytes = 32 * 128;         //   of its half of a step's keys,
constexpr int kVBytes = kKeys * 128;      //   of its value columns of a step
constexpr int kPBytes = 64 * 128;
constexpr int kStageBytes = 4 * 32 * 128;  // where results pass through on their way out, and P of two steps
static_assert(2 * kPBytes <= kStageBytes, "");
constexpr int kThreads = 192;
constexpr int kMmaWarp = 4, kLoadWarp = 5;
constexpr int kMiscBytes = 2048;
constexpr int kSmemQ = kMaxChunks * kQBytes, kSmemK = 2 * kMaxChunks * kKBytes, kSmemV = 2 * kMaxValues * kVBytes;
constexpr int kSmem = 1024 + kMiscBytes + kSmemQ + kSmemK + kSmemV + kStageBytes;
static_assert(kSmem <= 232448, "227 KB");
constexpr int kAhead = 4;                 // S of so many steps in TMEM
constexpr uint32_t kColO = 0, kColS = 256;
constexpr uint64_t kTimeoutNs = 1000000000ull;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;             // log2 of the largest P
// Own pages are asked of L2 this many steps before their copies: the ring holds two steps, which cover the
// latency of L2 but not that of HBM.  (V2-Lite 64 sequences 48.1 us, two steps 48.7, three 51.)
constexpr int kFetch = 1;
// A tile's start and end, in key steps: so many, and one per so many rows.  (One call after a flush of L2, 128 sequences
// behind a shared 8192 of 64 heads and of 16 heads: 144 and 68 us; 4 alone 171 and 70; 3 and one per 32 rows 167 and 74;
// 3 and one per 16 rows 151 and 71; 2 and one per 16 rows 155 and 74.  V2-Lite 64 sequences 58 to 61 with any.)
constexpr int kOverhead = 4, kRowsPerStep = 16;
// A shared prefix in tiles of its own makes a partial result of every row and leaves the rows that share it to the join:
// as many key steps of each CTA pair (see prefix_pays()).
constexpr int kJoinSteps = 4;
constexpr int kMinRun = 4;                // shortest run worth a CTA pair, in key steps after its tile's start (1 to 16 measure alike)

// A walk passes over empty sequences one by one, in a role that others wait for: so many take 74 ms (0.56 us each), far
// below the waits' limit.
constexpr int kMaxBatch = 1 << 17;

// What the join kernel needs to know of the cut (start of the workspace).
struct Cut {
    int64_t prefix_cost;  // cost of the prefix tiles
    int64_t run;          // cost per unit
    int32_t shared;       // keys of the shared prefix (a multiple of kKeys; 0: none)
    int32_t least;        // sequences of at least so many tokens share it
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
    int row_tiles, head_tiles, units;
    int dv_half;   // value columns of a CTA
    int overhead;  // cost of a tile beside its steps
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

// Keys of a sequence before its own ones, and steps over its own.
__device__ __forceinline__ int own_start(int len, int shared, int least) { return len >= least ? shared : 0; }
__device__ __forceinline__ int own_steps(int len, int shared, int least) {
    return (len - own_start(len, shared, least) + kKeys - 1) / kKeys;
}
__device__ __forceinline__ int64_t seq_cost(const CacheParams& p, int steps) {
    return steps ? static_cast<int64_t>(p.head_tiles) * (steps + p.overhead) : 0;
}

// Whether a prefix that `sharers` sequences share is multiplied in tiles of its own, which hold the rows of the whole
// batch (of sequences that do not share it, too), rather than by each of them with its own keys: the fewer key steps
// win.  128 rows of more than one sequence have to share a tile for that, so few of 128 heads or more do, nor do a few
// sequences of a large batch.  In us, tiles of their own / with the own keys, 128 sequences of 1 to 1024 behind 8192:
// 128 heads 231 / 220, 96 heads 191 / 215, 64 heads 143 / 213, 16 heads 69 / 206; 128 heads of which 2 share 199 / 38;
// 64 heads of which 32 / 64 / 80 share 121 / 72, 130 / 119, 134 / 144; 16 heads of which 16 / 20 / 32 share 48 / 46, 50 / 52,
// 52 / 68.  64 sequences of 16 heads behind 64 / 256 / 1024: 33 / 31, 35 / 35, 36 / 43; 8 behind 128: 25 / 21.
__device__ __forceinline__ bool prefix_pays(const CacheParams& p, int shared, int sharers) {
    const int64_t steps = shared / kKeys;
    return p.row_tiles * (steps + p.overhead) + static_cast<int64_t>(p.units) * kJoinSteps < sharers * steps * p.head_tiles;
}

// Most quotients here fit 32 bits, whose division takes a third of the time.
__device__ __forceinline__ int quotient(int64_t a, int b) {
    return static_cast<int>(a <= INT32_MAX ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b);
}

// The steps [*j0, *j1) of a tile of `steps` at cost `base` that the costs
// [from, to) cover.
__device__ __forceinline__ void covered(const CacheParams& p, int64_t base, int steps, int64_t from, int64_t to, int* j0,
                                        int* j1) {
    const int64_t a = from - base - p.overhead, e = to - base - p.overhead;
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

// A unit's walk over its pieces; every warp walks on its own, one lane of it,
// with its state in shared memory (on the stack it fell out of what L1 the
// tiles leave: 1.2 to 3 us a piece against 0.4).
struct Walk {
    int64_t at, end, prefix_cost, base;  // base: cost before batch row b
    int shared, least, source_row, b, len, row, unit;

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
                const int t = quotient(at, steps + p.overhead);
                tile_base = static_cast<int64_t>(t) * (steps + p.overhead);
                x->row0 = t * kRows;
                x->rows = min(kRows, p.B * p.H - x->row0);
                tile_row = x->row0;
                x->page_row = source_row;
                x->key0 = 0;
                x->end = shared;
                x->prefix = true;
            } else {
                steps = own_steps(len, shared, least);
                while (b < p.B && at >= base + seq_cost(p, steps)) {
                    base += seq_cost(p, steps);
                    ++b;
                    enter(p);
                    steps = own_steps(len, shared, least);
                }
                if (b >= p.B) return false;
                const int ht = p.head_tiles == 1 ? 0 : quotient(at - base, steps + p.overhead);
                tile_base = base + static_cast<int64_t>(ht) * (steps + p.overhead);
                x->row0 = b * p.H + ht * kRows;
                x->rows = min(kRows, p.H - ht * kRows);
                tile_row = static_cast<int64_t>(p.row_tiles) * kRows + x->row0;
                x->page_row = row;
                x->key0 = own_start(len, shared, least);
                x->end = len;
                x->prefix = false;
            }
            int j0, j1;
            covered(p, tile_base, steps, at, end, &j0, &j1);
            const int64_t tile_end = tile_base + steps + p.overhead;
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
    // full: K and V of step i at i % 2, Q of a piece; the even CTA's count for both.  s_full and pv_done also tell the
    // loaders that K and V have been read, and p_full (of the step before last) that an S has: the thread that issues the
    // products waits and commits as rarely as it can.
    uint64_t k_full[2], v_full[2], q_full;
    uint64_t s_full[kAhead], p_full[2], pv_done[2], v_seen, drain;
    uint32_t tmem;
    int abort_flag;
    float row_max[kRows], row_sum[kRows];  // what the two threads of a row tell each other
    int64_t scan[kThreads / 32];
    int64_t total, first_base;
    int first_b, sharers, source, shared;
    Walk walk[kThreads / 32];
    Piece piece[kThreads / 32];  // the next one of each
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
    // (the callers' word holds for sequences of `least` tokens or more; the prefix is handled in whole steps)
    const int least = p.shared_len ? *p.shared_len : 0, cap = p.max_pages * p.page_size;
    int shared = least;
    shared = shared < 0 ? 0 : (shared > cap ? cap : shared) / kKeys * kKeys;
    if (threadIdx.x == 0) sh->sharers = 0, sh->source = p.B;
    __syncthreads();
    if (shared > 0) {
        int count = 0, first = p.B;
        for (int b = threadIdx.x; b < p.B; b += kThreads)
            if (len_of(b) >= least) ++count, first = min(first, b);
        if (count) {
            atomicAdd(&sh->sharers, count);
            atomicMin(&sh->source, first);
        }
        __syncthreads();
        if (!prefix_pays(p, shared, sh->sharers)) shared = 0;
    }
    const int source = sh->source;
    const int64_t prefix = shared ? static_cast<int64_t>(p.row_tiles) * (shared / kKeys + p.overhead) : 0;
    int64_t total = prefix, sum, first_base = 0, first_cost = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        const int len = len_of(b);
        const int64_t mine = b < p.B ? seq_cost(p, own_steps(len, shared, least)) : 0;
        const int64_t before = total + block_scan(mine, sh->scan, &sum);
        if (writer && b < p.B) p.bases[b] = before;
        if (b0 == 0) first_base = before, first_cost = mine;
        total += sum;
    }
    int64_t run = (total + p.units - 1) / p.units;
    if (run < kMinRun + p.overhead) run = kMinRun + p.overhead;
    if (writer) {
        if (threadIdx.x == 0) *p.cut = Cut{prefix, run, shared, least, source};
        raise_status(p.status, bits);
    }
    w->unit = unit;
    w->at = run * unit;
    w->end = w->at + run < total ? w->at + run : total;
    w->prefix_cost = prefix;
    w->shared = shared;
    w->least = least;
    w->b = 0;
    w->base = prefix;
    w->len = w->row = 0;
    w->source_row = -1;
    if (w->at >= total) return false;
    if (shared) batch_len(p, source, &w->source_row, &bits);
    if (w->at >= prefix) {  // the batch row that holds `at`
        if (p.B <= kThreads) {
            if (first_cost && w->at >= first_base && w->at < first_base + first_cost)
                sh->first_b = threadIdx.x, sh->first_base = first_base;
        } else {
            int64_t base = prefix;
            for (int b0 = 0; b0 < p.B; b0 += kThreads) {
                const int b = b0 + threadIdx.x;
                const int len = len_of(b);
                const int64_t mine = b < p.B ? seq_cost(p, own_steps(len, shared, least)) : 0;
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
    mla_attend_cache_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CacheParams p) {
    extern __shared__ uint8_t raw[];
    const uint32_t raw_at = smem_u32(raw);
    const uint32_t pad = (1024u - (raw_at & 1023u)) & 1023u;  // the same in both CTAs of a pair
    const int chunks = (p.C + 63) / 64;
    const uint32_t sm_q = raw_at + pad, sm_k = sm_q + kSmemQ, sm_v = sm_k + kSmemK, sm_p = sm_v + kSmemV;
    Shared* sh = reinterpret_cast<Shared*>(raw + pad + kSmemQ + kSmemK + kSmemV + kStageBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x / 2, rank = blockIdx.x % 2;
    const int v0 = rank * p.dv_half, nvc = (p.dv_half + 63) / 64;  // value columns that this CTA brings

    if (warp == kLoadWarp && lane == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh->k_full[i]), 1);
            mbar_init(smem_u32(&sh->v_full[i]), 1);
            mbar_init(smem_u32(&sh->p_full[i]), 8);  // the softmax warps of both CTAs
            mbar_init(smem_u32(&sh->pv_done[i]), 1);
        }
        for (int i = 0; i < kAhead; ++i) mbar_init(smem_u32(&sh->s_full[i]), 1);
        mbar_init(smem_u32(&sh->q_full), 1);
        mbar_init(smem_u32(&sh->v_seen), 1);
        mbar_init(smem_u32(&sh->drain), 1);
        sh->abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    if (warp == kMmaWarp) {
        tmem_alloc_pair(smem_u32(&sh->tmem), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    pdl_wait();  // what the kernel before in the stream wrote
    __syncwarp();
    cluster_arrive();  // the peer's barriers are ready once both have come here; the cut is made meanwhile
    Walk start;
    const bool any = make_cut(p, unit, sh, &start);
    if (lane == 0) sh->walk[warp] = start;
    cluster_wait();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    if (!any) {  // (the same in both CTAs)
        if (warp == kMmaWarp) tmem_dealloc_pair(tmem, 512);
        return;
    }
    const volatile int* abort_flag = &sh->abort_flag;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_wait_lean(smem_u32(bar), parity & 1u, kTimeoutNs, abort_flag);
    };
    bool ok = true;
    int step = 0;  // key steps so far, over all pieces: the phase of every barrier
    Piece x;
    Walk& walk = sh->walk[warp];
    Piece& next = sh->piece[warp];
    // The warp's next piece, which one lane has found (`got`) or finds now.
    auto take = [&](bool got) {
        __syncwarp();
        x = next;
        return __shfl_sync(~0u, static_cast<int>(got), 0) != 0;
    };

    if (warp < 4) {
        // ------------------------------------------------------------ softmax
        const int r = (warp & 1) * 32 + lane, side = warp >> 1;  // row of this CTA; half of the keys, of the columns
        const int tile_row = rank * 64 + r;
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        const uint32_t to = tmem + lanes + kColO, ts = tmem + lanes + kColS;
        const uint32_t p_full = map_shared_rank(smem_u32(&sh->p_full[0]), 0);
        auto arrive = [&](uint32_t bar) {  // one arrival per warp, at the even CTA
            __syncwarp();
            if (lane == 0) mbar_arrive_peer(bar);
        };
        const float c = p.scale * kLog2e;
        int tails = 0;  // steps so far that ended inside
        const int dv0 = side * p.dv_half, dv = min(p.dv_half, p.Lkv - dv0);  // value columns of this thread
        bool got = lane == 0 && walk.next(p, &next);
        while (ok && take(got)) {
            const bool mine = tile_row < x.rows;
            const int n = x.n, keys = x.end - x.key0;
            float m = -INFINITY, ms = 0.f, l = 0.f;  // row maximum of S, ms = m c, sum of this thread's half of P
            for (int j = 0; j < n; ++j, ++step) {
                // A failed wait stays failed, and the step makes and hands over nothing after it; a barrier of the
                // whole group follows in every step, where all four warps learn of it and leave together.
                ok = __all_sync(~0u, ok && wait(&sh->s_full[step % kAhead], step / kAhead));
                uint32_t s[32];
                tc_fence_after();
                float mt = tmem_ld32_max(ts + step % kAhead * 32, s);
                const int left = keys - j * kKeys - side * 32;
                if (left < 32) {
                    mt = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (i >= left) s[i] = 0xFF800000u;
                        mt = fmaxf(mt, __uint_as_float(s[i]));
                    }
                }
                bool grow = mt > m && (m == -INFINITY || mt * c > ms + kSlack);
                float alpha = 1.f;
                // rare after the first step: the row's two threads agree on a new scale
                if (named_bar_or(1, 128, grow || !ok)) {
                    sh->row_max[threadIdx.x] = mt;
                    if (named_bar_or(1, 128, !ok)) {
                        ok = false;
                        break;
                    }
                    const float other = *const_cast<volatile float*>(&sh->row_max[threadIdx.x ^ 64]);
                    mt = fmaxf(mt, other);
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
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
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
                // P of two steps before has been read; O is at rest where it has to be scaled
                if (step > 1) ok = __all_sync(~0u, ok && wait(&sh->pv_done[step & 1], (step >> 1) - 1));
                if (j > 0 && __any_sync(~0u, alpha != 1.f)) {
                    ok = __all_sync(~0u, ok && wait(&sh->pv_done[(step - 1) & 1], (step - 1) >> 1));
                    if (!ok) continue;
                    tc_fence_after();
#pragma unroll 1
                    for (int d = 0; d < p.dv_half; d += 16) {
                        float o[16];
                        tmem_ld16(to + d, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= alpha;
                        tmem_st16(to + d, o);
                    }
                }
                if (!ok) continue;
                const uint32_t dst = sm_p + (step & 1) * kPBytes + r * 128;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    st_shared_v4(dst + (((side * 4 + i) ^ (r & 7)) << 4), w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                const int rest = keys - j * kKeys;
                if (rest < kKeys) {
                    // rows behind the end may hold anything: as values they have to be zero
                    ok = __all_sync(~0u, ok && wait(&sh->v_seen, tails));
                    if (!ok) continue;
                    ++tails;
                    for (int k = threadIdx.x; k < (kKeys - rest) * nvc * 8; k += 128) {
                        const int row = rest + k / (nvc * 8), in = k % (nvc * 8);
                        st_shared_v4(sm_v + ((step & 1) * kMaxValues + in / 8) * kVBytes + row * 128 + (in & 7) * 16, 0, 0, 0, 0);
                    }
                }
                fence_proxy_async_shared();
                tc_fence_before();
                arrive(p_full + 8 * (step & 1));
            }
            got = lane == 0 && walk.next(p, &next);  // while the last products run
            sh->row_sum[threadIdx.x] = l;
            ok = __all_sync(~0u, ok && wait(&sh->pv_done[(step - 1) & 1], (step - 1) >> 1));
            if (named_bar_or(1, 128, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            l = sh->row_sum[threadIdx.x & 63] + sh->row_sum[(threadIdx.x & 63) + 64];
            // A row whose keys this piece covers alone is finished; the others leave a partial result.
            bool direct = x.whole;
            const int b = (x.row0 + tile_row) / p.H;
            if (start.shared && direct && mine) {
                int trow, bits = 0;
                const int len = batch_len(p, b, &trow, &bits);
                direct = x.prefix ? len >= start.least && len == start.shared : len < start.least;
            }
            // A warp's rows pass through shared memory, 128 bytes of each at a time, so that it stores four rows'
            // whole lines at once: 64 columns of finished rows, 32 of partial ones.
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int64_t at = static_cast<int64_t>(x.row0) + tile_row;
            const uint32_t direct_rows = __ballot_sync(~0u, direct && mine), part_rows = __ballot_sync(~0u, !direct && mine);
            const uint32_t stage = sm_p + warp * 32 * 128;
            auto put = [&](int i, uint32_t a, uint32_t b2, uint32_t c2, uint32_t d2) {
                st_shared_v4(stage + lane * 128 + ((i ^ (lane & 7)) << 4), a, b2, c2, d2);
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
            const int64_t row32 = rank * 64 + (warp & 1) * 32;  // the warp's first row of the tile
            uint8_t* out = reinterpret_cast<uint8_t*>(p.out + (x.row0 + row32) * p.Lkv + dv0);
            uint8_t* part = reinterpret_cast<uint8_t*>(p.part_o + (x.part + row32) * p.Lkv + dv0);
#pragma unroll 1
            for (int d0 = 0; d0 < dv; d0 += 128) {
                uint32_t o[128];  // (what lies behind dv is not stored)
                tmem_ld128_max(to + d0, o);
#pragma unroll
                for (int i = 0; i < 128; ++i) o[i] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(o[i]) * inv);
                if (part_rows) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (d0 + k * 32 >= dv) break;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            put(i, o[k * 32 + 4 * i], o[k * 32 + 4 * i + 1], o[k * 32 + 4 * i + 2], o[k * 32 + 4 * i + 3]);
                        flush(part + (d0 + k * 32) * 4, p.Lkv * 4, part_rows, (dv - d0 - k * 32) * 4);
                    }
                }
                if (direct_rows) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (d0 + k * 64 >= dv) break;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = pack_bf16x2(__uint_as_float(o[k * 64 + 8 * i + 2 * e]), __uint_as_float(o[k * 64 + 8 * i + 2 * e + 1]));
                            put(i, w[0], w[1], w[2], w[3]);
                        }
                        flush(out + (d0 + k * 64) * 2, p.Lkv * 2, direct_rows, (dv - d0 - k * 64) * 2);
                    }
                }
            }
            if (mine && side == 0) {
                const float lg = l == 0.f ? -INFINITY : ms + log2f(l);
                if (!direct) p.part_lse[x.part + tile_row] = lg;
                else if (p.lse) p.lse[at] = lg * kLn2;
            }
            tc_fence_before();
            named_bar_sync(1, 128);  // the next piece's P takes the place that results pass through
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------ MMA (the even CTA's, for both)
        if (rank == 0 && elect_one()) {
            const uint32_t idesc_s = idesc_bf16_f32(kRows, kKeys);
            const uint64_t dq = smem_desc_sw128(sm_q), dk = smem_desc_sw128(sm_k), dp = smem_desc_sw128(sm_p);
            const uint64_t dvals = smem_desc_sw128_mn(sm_v, kVBytes);
            const uint32_t to = tmem + kColO;
            const bool widest = p.C == 64 * kMaxChunks;
            // value columns in products of up to 128 per CTA
            const int first = min(p.dv_half, 128), second = p.dv_half - first;
            const uint32_t id0 = idesc_bf16_f32(kRows, 2 * first) | kIdescBMnMajor;
            const uint32_t id1 = idesc_bf16_f32(kRows, second ? 2 * second : 32) | kIdescBMnMajor;
            auto look = [&](uint64_t* bar, uint32_t parity) {
                ok = ok && wait(bar, parity);
                tc_fence_after();
                return ok;
            };
            auto commit = [&](uint64_t* bar) { mma_commit_pair(smem_u32(bar), 0x3); };
            bool got = walk.next(p, &next);
            for (int piece = 0; got; ++piece) {
                x = next;
                const int n = x.n;
                if (!look(&sh->q_full, piece)) break;
                // Per round: the scores of step t, then P V of step t - 2, whose softmax ran meanwhile.
#pragma unroll 1
                for (int t = 0; t < n + 2 && ok; ++t) {
                    const int st = step + t, e = st & 1, f4 = st % kAhead;
                    if (t < n) {
                        // (S of step t - 4 has been read: P of step t - 3 was waited for in the round before)
                        if (!look(&sh->k_full[e], st >> 1)) break;
                        const uint32_t d = tmem + kColS + f4 * 32;
                        const uint64_t b = dk + e * (kMaxChunks * kKBytes >> 4);
                        if (widest) {
#pragma unroll
                            for (int k = 0; k < 4 * kMaxChunks; ++k)
                                mma_bf16_pair(d, dq + (k >> 2) * (kQBytes >> 4) + 2 * (k & 3),
                                              b + (k >> 2) * (kKBytes >> 4) + 2 * (k & 3), idesc_s, k > 0);
                        } else {
#pragma unroll 1
                            for (int k = 0; k < p.C / 16; ++k)
                                mma_bf16_pair(d, dq + (k >> 2) * (kQBytes >> 4) + 2 * (k & 3),
                                              b + (k >> 2) * (kKBytes >> 4) + 2 * (k & 3), idesc_s, k > 0);
                        }
                        commit(&sh->s_full[f4]);
                        if (t + 1 == n) got = walk.next(p, &next);
                    }
                    if (t > 1) {
                        const int pv = st - 2, f = pv & 1;
                        if (!look(&sh->v_full[f], pv >> 1)) break;
                        if (t == n + 1 && x.end - x.key0 < n * kKeys) {  // both CTAs clear the rows behind the end first
                            mbar_arrive(smem_u32(&sh->v_seen));
                            mbar_arrive_peer(map_shared_rank(smem_u32(&sh->v_seen), 1));
                        }
                        if (!look(&sh->p_full[f], pv >> 1)) break;
                        const uint64_t b = dvals + f * (kMaxValues * kVBytes >> 4);
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k) {
                            mma_bf16_pair(to, dp + f * (kPBytes >> 4) + 2 * k, b + k * (2048 >> 4), id0, t > 2 || k > 0);
                            if (second) mma_bf16_pair(to + 128, dp + f * (kPBytes >> 4) + 2 * k, b + (2 * kVBytes >> 4) + k * (2048 >> 4), id1, t > 2 || k > 0);
                        }
                        commit(&sh->pv_done[f]);
                    }
                }
                if (!ok) break;
                step += n;
            }
            if (!ok) {  // no MMA may still run when the CTAs leave
                commit(&sh->drain);
                mbar_wait(smem_u32(&sh->drain), 0, kTimeoutNs, nullptr);
            }
        }
    } else {
        // --------------------------------------------------------------- TMA
        // The lanes look up the rows of 32 boxes at a time; one thread issues the copies, each CTA its halves, which
        // complete on the even CTA's barriers; the even CTA tells them how many bytes both bring.
        const int per = kKeys / p.box, batch = 32 / per;  // boxes per step, steps per lookup
        const bool lead = elect_one();
        const uint32_t box_bytes = p.box * 128;
        const bool whole = p.box >= 32 && p.C == 64 * kMaxChunks && p.dv_half == 256;
        auto s_made = [&](int u) { return wait(&sh->s_full[u % kAhead], u / kAhead); };  // the scores of step u,
        auto pv_made = [&](int u) { return wait(&sh->pv_done[u & 1], u >> 1); };           // its P V
        auto at_even = [&](uint64_t* bar) { return map_shared_rank(smem_u32(bar), 0); };
        int bits = 0, pieces = 0, ks = 0, vs = 0;  // Q, K and V places filled
        // first row of box `lane` of the batch that starts at a piece's step j; a row outside the cache reads as zeros
        auto look_up = [&](const Piece& y, int j) {
            const int key = y.key0 + (j * per + lane) * p.box;
            if (j * per + lane >= y.n * per || key >= y.end) return p.num_rows;
            const int page = p.table[static_cast<int64_t>(y.page_row) * p.max_pages + key / p.page_size];
            if (page >= 0 && page < p.num_pages) return page * p.page_size + key % p.page_size;
            bits |= kStatusPageRange;
            return p.num_rows;
        };
        // Asks L2 for this lane's box of cache rows, which lie in one piece of memory.
        auto fetch = [&](int row) {
            if (row < p.num_rows) bulk_prefetch_l2(p.cache + static_cast<int64_t>(row) * p.C, p.box * p.C * 2);
        };
        // The first steps of a piece, which is found and asked of L2 while the one before still runs.
        auto begin = [&](const Piece& y) {
            const int rows = look_up(y, 0);
            if (!y.prefix && lane / per < batch && lane / per < kFetch && (lane / per & 1) == rank) fetch(rows);
            const int mine = min(64, y.rows - rank * 64);  // this CTA's rows of Q
            if (lane == 31 && mine > 0)
                bulk_prefetch_l2(p.q + (static_cast<int64_t>(y.row0) + rank * 64) * p.C, mine * p.C * 2);
            return rows;
        };
        bool have = take(lane == 0 && walk.next(p, &next));
        int rows = have ? begin(x) : 0, rows_next = 0;
        while (ok && have) {
            const int n = x.n;
            if (lead) {  // Q, once the scores of the piece before are made
                if (step) ok = s_made(step - 1);
                if (ok) {
                    if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sh->q_full), 2 * chunks * kQBytes);
                    const int row = x.row0 + rank * 64;
                    if (p.C == 64 * kMaxChunks) {
                        for (int k = 0; k < kMaxChunks; k += 3)
                            tma_load_3d_pair(sm_q + k * kQBytes, &tm_q, at_even(&sh->q_full), 0, row, k);
                    } else {
                        for (int k = 0; k < chunks; ++k)
                            tma_load_3d_pair(sm_q + k * kQBytes, &tm_q, at_even(&sh->q_full), k * 64, 0, row);
                    }
                    ++pieces;
                }
            }
            ok = __all_sync(~0u, ok);
            int ahead = batch < n ? look_up(x, batch) : p.num_rows;
            const bool far = !x.prefix && lane / per < batch;
            // K of step j, then V of step j - 2, as they are used: so K never waits behind a V whose place is not free.
            int row[kKeys / 16], row1[kKeys / 16], row2[kKeys / 16];  // the boxes of steps j, j - 1, j - 2
#pragma unroll
            for (int e = 0; e < kKeys / 16; ++e) row[e] = row1[e] = row2[e] = p.num_rows;
#pragma unroll 1
            for (int j = 0; j < n + 2 && ok; ++j) {
                const int i = j & (batch - 1);
                if (i == 0 && j > 0 && j < n) {
                    rows = ahead;
                    ahead = j + batch < n ? look_up(x, j + batch) : p.num_rows;
                }
#pragma unroll
                for (int e = 0; e < kKeys / 16; ++e) {
                    row2[e] = row1[e];
                    row1[e] = row[e];
                    row[e] = __shfl_sync(~0u, rows, min(i * per + e, 31));
                }
                // step j + kFetch of the run, alternately by the two CTAs
                if (far && j < n && lane / per == ((i + kFetch) & (batch - 1)) && (j & 1) == rank)
                    fetch(i + kFetch < batch ? rows : ahead);
                if (lead && j < n) {
                    const int st = (step + j) & 1;
                    ok = step + j < 2 || s_made(step + j - 2);
                    if (ok) {
                        ++ks;
                        const uint32_t bar = at_even(&sh->k_full[st]), dst = sm_k + st * kMaxChunks * kKBytes;
                        if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sh->k_full[st]), 2 * chunks * kKBytes);
                        // this CTA's 32 keys: half of a box of 64 (or outside, like it), a box of 32, two of 16
                        const int k0 = per == 1 ? (rank && row[0] < p.num_rows ? row[0] + 32 : row[0])
                                                : rank == 0 ? row[0] : per == 2 ? row[1] : row[2];
                        if (whole) {
#pragma unroll
                            for (int k = 0; k < kMaxChunks; k += 3)
                                tma_load_3d_pair(dst + k * kKBytes, &tm_k, bar, 0, k0, k);
                        } else {
                            for (int k = 0; k < chunks; ++k) {
                                tma_load_3d_pair(dst + k * kKBytes, &tm_k, bar, k * 64, 0, k0);
                                if (per == 4)
                                    tma_load_3d_pair(dst + k * kKBytes + box_bytes, &tm_k, bar, k * 64, 0, rank ? row[3] : row[1]);
                            }
                        }
                    }
                }
                if (lead && j > 1 && ok) {
                    const int st = (step + j) & 1;
                    ok = step + j < 4 || pv_made(step + j - 4);
                    if (ok) {
                        ++vs;
                        const uint32_t bar = at_even(&sh->v_full[st]), dst = sm_v + st * kMaxValues * kVBytes;
                        if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sh->v_full[st]), 2 * nvc * kVBytes);
                        if (whole && per == 1) {
                            tma_load_3d_pair(dst, &tm_v, bar, 0, row2[0], rank * 4);
                        } else {
                            const int boxes = per == 1 ? 2 : per;  // a box of 64 in two of 32
                            const uint32_t bytes = per == 1 ? 32 * 128 : box_bytes;
#pragma unroll
                            for (int e = 0; e < kKeys / 16; ++e) {
                                if (e >= boxes) break;
                                const int vr = per == 1 ? (e && row2[0] < p.num_rows ? row2[0] + 32 : row2[0]) : row2[e];
                                for (int k = 0; k < nvc; ++k)
                                    tma_load_3d_pair(dst + k * kVBytes + e * bytes, &tm_v, bar, v0 + k * 64, 0, vr);
                            }
                        }
                    }
                }
                if (j == n - 1) {
                    __syncwarp();
                    have = __shfl_sync(~0u, static_cast<int>(lane == 0 && walk.next(p, &next)), 0);
                    __syncwarp();
                    if (have) rows_next = begin(next);
                }
                ok = __all_sync(~0u, ok);
            }
            step += n;
            x = next;
            rows = rows_next;
        }
        // no copy of either CTA may still be landing when they leave
        if (lead && rank == 0) {
            if (pieces) mbar_wait(smem_u32(&sh->q_full), (pieces - 1) & 1, kTimeoutNs, nullptr);
            for (int u = max(ks - 2, 0); u < ks; ++u) mbar_wait(smem_u32(&sh->k_full[u & 1]), (u >> 1) & 1, kTimeoutNs, nullptr);
            for (int u = max(vs - 2, 0); u < vs; ++u) mbar_wait(smem_u32(&sh->v_full[u & 1]), (u >> 1) & 1, kTimeoutNs, nullptr);
        }
        // and what the tensor core frees has arrived (a piece's last products have ended before its results go out)
        if (lead) {
            for (int u = max(ks - kAhead, 0); u < ks; ++u) ok = ok && s_made(u);
            for (int u = max(vs - 2, 0); u < vs; ++u) ok = ok && pv_made(u);
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
    cluster_sync_all();  // neither CTA leaves or frees TMEM while the other's copies and products may touch it
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// Joins the partial results of each row, in the order of the cut; a row with
// one piece was finished by that piece.  One warp per row; bound by the latency
// of its few dependent reads (cut, length, sums, rows): 3.3 us where nothing is
// to join, 5.7 for 64 sequences of 16 heads, 9.2 for 32 and 13 for 128 of 128.
__global__ void __launch_bounds__(128) mla_attend_join_kernel(const __grid_constant__ CacheParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    pdl_launch_dependents();
    pdl_wait();
    if (row >= static_cast<int64_t>(p.B) * p.H) return;
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
            steps[0] = len >= cut.least ? cut.shared / kKeys : 0;
            base[0] = row / kRows * (cut.shared / kKeys + p.overhead);
            part[0] = row;
        } else {
            steps[1] = own_steps(len, cut.shared, cut.least);
            base[1] = p.bases[b] + static_cast<int64_t>(h / kRows) * (steps[1] + p.overhead);
            part[1] = static_cast<int64_t>(p.row_tiles) * kRows + row;
        }
        u0[k] = static_cast<int>((base[k] + p.overhead) / cut.run);
        u1[k] = steps[k] ? static_cast<int>((base[k] + p.overhead + steps[k] - 1) / cut.run) : u0[k] - 1;
        count += u1[k] - u0[k] + 1;
    }
    if (count == 1) return;
    // Two pieces are on their way at once; the running maximum, sum and row go on from one two to the next.
    constexpr int kAtOnce = 2;
    float ref = 0.f, sum = 0.f, top = -INFINITY;
    float4 acc[4] = {};
    const int count0 = u1[0] - u0[0] + 1;
    for (int first = 0; first < count; first += kAtOnce) {
        float lse[kAtOnce];
        float4 o[kAtOnce][4];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int i = first + k;
            const bool own = i >= count0;
            const int64_t at = i < count ? part_row(p, own ? part[1] : part[0], own ? u0[1] + i - count0 : u0[0] + i) : 0;
            lse[k] = i < count ? p.part_lse[at] : -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (i < count && (c * 32 + lane) * 4 < p.Lkv)
                    o[k][c] = reinterpret_cast<const float4*>(p.part_o + at * p.Lkv)[c * 32 + lane];
        }
        float next = top;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) next = fmaxf(next, lse[k]);
        const float keep = top == -INFINITY ? 0.f : exp2f(top - next);
        top = next;
        ref = top == -INFINITY ? 0.f : top;
        sum *= keep;
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c].x *= keep, acc[c].y *= keep, acc[c].z *= keep, acc[c].w *= keep;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (first + k >= count) break;
            const float w = exp2f(lse[k] - ref);
            sum += w;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if ((c * 32 + lane) * 4 < p.Lkv) {
                    acc[c].x = fmaf(w, o[k][c].x, acc[c].x), acc[c].y = fmaf(w, o[k][c].y, acc[c].y);
                    acc[c].z = fmaf(w, o[k][c].z, acc[c].z), acc[c].w = fmaf(w, o[k][c].w, acc[c].w);
                }
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
    if (d.batch < 0 || d.batch > kMaxBatch || d.num_heads < 1 || static_cast<int64_t>(d.batch) * d.num_heads > (1 << 24) ||
        d.kv_lora_rank < 16 || d.kv_lora_rank > 512 || d.kv_lora_rank % 16 || d.rope_dim < 0 || d.rope_dim > 128 ||
        d.rope_dim % 16 || d.kv_lora_rank + d.rope_dim > 576)
        return MLA_ERR_UNSUPPORTED_DIMS;
    if (d.page_size < 16 || d.page_size % 16 || d.table_rows < 0 || d.max_pages < 1 || d.num_pages < 0 ||
        d.num_pages > most / d.page_size || static_cast<int64_t>(d.max_pages) * d.page_size > (1 << 30) ||
        !scale_ok(d.scale))
        return MLA_ERR_UNSUPPORTED_DIMS;
    return MLA_OK;
}

// Workspace: the cut, the costs before each sequence, the partial results.
struct Layout {
    int row_tiles, head_tiles, units;
    size_t bases, part_lse, part_o, bytes;
};

Layout layout(const mla_prolog_cache_dims& d, int sms) {
    Layout y;
    const int64_t rows = static_cast<int64_t>(d.batch) * d.num_heads;
    y.row_tiles = static_cast<int>((rows + kRows - 1) / kRows);
    y.head_tiles = (d.num_heads + kRows - 1) / kRows;
    y.units = sms / 2 > 0 ? sms / 2 : 1;
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
    const int dv_half = (d->kv_lora_rank / 2 + 15) / 16 * 16;
    CUtensorMap tq, tk, tv;
    // an empty cache has no valid page: every read is outside the map, which then only needs a valid address
    const void* base = rows ? kv_cache : q;
    const uint64_t map_rows = rows ? rows : 1;
    // The widest rows by whole chunks, [chunk][row][64], several in one copy: Q and the 32 keys for the scores by three,
    // the 64 keys of values by four.  (whole, per: as in the kernel.)
    const uint64_t q_rows = static_cast<uint64_t>(d->batch) * d->num_heads;
    const bool wide = C == 64 * kMaxChunks, whole = wide && box >= 32 && dv_half == 256;
    const uint32_t box_rows = box < 32 ? box : 32;
    bool good = wide ? encode_bf16_chunks(&tq, q, C, q_rows, 64, 3) : encode_bf16_3d(&tq, q, C, 1, q_rows, 1, 64);
    good = good && (whole ? encode_bf16_chunks(&tk, base, C, map_rows, 32, 3) : encode_bf16_3d(&tk, base, C, 1, map_rows, 1, box_rows));
    if (!whole) tv = tk;
    else good = good && (box == kKeys ? encode_bf16_chunks(&tv, base, C, map_rows, kKeys, 4) : encode_bf16_3d(&tv, base, C, 1, map_rows, 1, box_rows));
    if (!good) return report_cuda(cudaErrorInvalidValue, "tensor maps of attend_cache");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    CacheParams p{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(kv_cache), page_table, seq_lens, seqs, shared_len, static_cast<uint16_t*>(out),
                  lse, status, reinterpret_cast<Cut*>(ws), reinterpret_cast<int64_t*>(ws + y.bases),
                  reinterpret_cast<float*>(ws + y.part_o), reinterpret_cast<float*>(ws + y.part_lse), d->batch,
                  d->num_heads, d->kv_lora_rank, C, d->page_size, d->table_rows, d->max_pages,
                  static_cast<int>(rows ? rows : 1), static_cast<int>(d->num_pages), box, y.row_tiles, y.head_tiles,
                  y.units, dv_half, kOverhead + (d->num_heads < kRows ? d->num_heads : kRows) / kRowsPerStep, d->scale};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = allow_smem(&mla_attend_cache_kernel, kSmem, &ready);
    if (e != cudaSuccess) return report_cuda(e, "mla_attend_cache_kernel attributes");
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(y.units * 2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    e = cudaLaunchKernelEx(&cfg, mla_attend_cache_kernel, tq, tk, tv, p);
    if (e != cudaSuccess) return report_cuda(e, "launch mla_attend_cache_kernel");
    const int64_t blocks = (static_cast<int64_t>(d->batch) * d->num_heads + 3) / 4;
    e = launch_kernel(mla_attend_join_kernel, dim3(static_cast<unsigned>(blocks)), dim3(128), 0, st, true, p);
    return e == cudaSuccess ? MLA_OK : report_cuda(e, "launch mla_attend_join_kernel");
}

}  // extern "C"
