// Attention over whole prompts: mla_prolog_attend_prompt.
//
// One CTA takes 256 query rows of one sequence and head, as two tiles of 128
// rows, and walks the keys in tiles of 128 with the running maximum and sum
// of a softmax (one pass over K and V).  Per key tile and query tile:
//
//   S = Q K^T         tcgen05.mma, Q and K tiles in shared memory (TMA), S in TMEM
//   P = exp2(S c - m) the tile's softmax warpgroup: one row per thread, S read
//                     from TMEM once, P written back over S as BF16
//   O += P V          tcgen05.mma, P from TMEM, V in shared memory read along
//                     its columns, O in TMEM in FP32
//
// Two query tiles, because the tensor core then works on one tile's products
// while the other tile's warpgroup is at its exponentials; S, P and O of two
// tiles fill the 512 columns of TMEM exactly (v_dim <= 128).  Warp roles: 0-3
// and 4-7 softmax of tile 0 and 1, 8 issues the MMAs, 9 the TMA loads.
//
// With few tile pairs a cluster of 2, 4 or 8 CTAs takes each: every CTA the
// key tiles of its rank, with its own maximum and sum, and the rows are joined
// through the cluster's shared memory.
//
// The maximum that P is scaled by moves only when a row's maximum has grown
// by more than 2^8: until then P <= 2^8, which neither BF16 nor the FP32 sums
// mind, and O need not be rescaled.
//
// Roundings: P to BF16 for the product with V (the tensor core takes 16-bit
// operands; the row sum is of the FP32 values), out to BF16 once.  S, maximum,
// sum, O and lse are FP32.  INT8 codes become BF16 exactly.
//
// What bounds it: the chain of one query tile per key tile, softmax (1.6k
// cycles), then P V and the next Q K^T (1.3k), with hand-overs 3.1 to 3.6k
// cycles for the two tiles, which the tensor core alone would do in 2.56k
// (qk_dim 192, v_dim 128); and 11k to 17k cycles of a CTA's start and end.  A
// CTA that keeps 64 keys per step, P in halves, exponentials on the last
// tile's maximum, a persistent CTA or a CTA pair per 256 rows each measured
// slower.  128 heads x 16384 tokens, INT8 q: 6.83 ms, 1610 TFLOP/s (84 % of the
// measured cuBLAS rate); four prompts of 700 to 4099: 932 us, 1023 TFLOP/s;
// 16 heads x 4096: 70.5 us, 1220; eight ragged prompts: 43.4 us, 647.
#include <cstdint>

#include "attend.cuh"
#include "attend_ptx.cuh"

namespace mlap {
namespace {

constexpr int kTile = 128;                 // query rows per tile, keys per tile
constexpr int kSlotBytes = kTile * 128;    // 128 rows x 64 BF16 columns: one TMA box
constexpr int kMaxSlots = 8;               // K and V of a tile and a half at qk_dim 192 (more does not fit beside Q)
constexpr int kAhead = 4;                  // K (V) tiles whose barriers are in use at once
constexpr int kThreads = 320;
constexpr int kMaxShift = 3;               // at most 8 CTAs share a tile pair's keys,
constexpr int kSplitTiles = 6;             //   of sequences of this many key tiles on average
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kMiscBytes = 512;
constexpr int kSmemMax = 232448;           // 227 KB
constexpr uint64_t kTimeoutNs = 1000000000ull;
constexpr uint32_t kColS = 0, kColO = 256;  // TMEM: S/P of tile t at 128 t, O of tile t at 256 + 128 t
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;              // log2 of the largest P

struct PromptParams {
    const int8_t* q8;  // null: BF16 q
    const float* q_scale;
    const uint16_t* v;
    const int32_t* cu_q;
    const int32_t* cu_k;
    uint16_t* out;
    float* lse;
    int32_t* status;
    int Tq, Tk, B, H, Hk, Dqk, Dv;
    float scale;
    int causal, q_per_head;
    int slots;        // ring slots
    int shift;        // log2 of the CTAs that share a tile pair's keys
    int tile_bound;   // >= 256-row tiles of all sequences
    int head_group;   // query heads whose K and V stay in L2 together
};

// Everything the roles share.  (Shared memory, after the tiles.)
struct Shared {
    uint64_t q_full[2], s_full[2], p_full[2], o_done[2], drain;
    uint64_t k_full[kAhead], v_full[kAhead], k_free[kAhead], v_free[kAhead];  // of key tile j at j % kAhead
    uint32_t tmem;
    int abort_flag;
    int job[5];        // q0, nq, k0, nk, first row of the tile pair; job[1] = 0: nothing to do
    uint32_t bad[12];  // keys of the masked tiles whose v holds a NaN or an infinity
};
static_assert(sizeof(Shared) <= kMiscBytes, "");

template <int N>
struct Steps {
    static constexpr int value = N;
};

struct Job {
    int q0, nq, k0, nk, r0;
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

// Rows [*a, *a + *n) of sequence s in a buffer of `rows`, cut to the buffer.
__device__ __forceinline__ bool seq_rows(const int32_t* cu, int s, int rows, int* a, int* n) {
    const int x = cu[s], y = cu[s + 1];
    const int lo = clampi(x, 0, rows), hi = clampi(y, 0, rows);
    *a = lo;
    *n = hi > lo ? hi - lo : 0;
    return x >= 0 && y >= x && y <= rows;
}

// The t-th tile pair in the order of their keys, most first (so that no long
// one starts when the others end), for at most 32 sequences: a lane per
// sequence, whose pairs of a cost or more are a formula, and a search for the
// cost at which the t-th lies.  One warp; job[1] = 0: there are fewer.  Chunks
// of 512, 300 and 1 rows on 7680, 4097 and 1023 earlier keys: 106 us by place,
// 100 by cost; four prompts of 128 heads 1026, 1014; where nothing is uneven
// the search costs 0.4 us.
__device__ __forceinline__ void find_job_by_cost(const PromptParams& p, int t, bool report, Shared* sh) {
    const int lane = threadIdx.x & 31;
    int a = 0, n = 0, ka = 0, kn = 0;
    bool good = true;
    if (lane < p.B) {
        good = seq_rows(p.cu_q, lane, p.Tq, &a, &n);
        good &= seq_rows(p.cu_k, lane, p.Tk, &ka, &kn);
    }
    if (report && !__all_sync(~0u, good) && lane == 0) raise_status(p.status, kStatusSeqRange);
    const int pairs = (n + 2 * kTile - 1) / (2 * kTile);
    // this sequence's pairs of at least c key tiles: its last ones
    auto at_least = [&](int c) {
        const int x = (c - 1) * kTile;
        if (c == 0) return pairs;
        if (x >= kn) return 0;
        return p.causal ? pairs - clampi((x - (kn - n)) >> 8, 0, pairs) : pairs;
    };
    static_assert(2 * kTile == 1 << 8, "");
    const int total = __reduce_add_sync(~0u, pairs);
    if (t >= total) {
        if (lane == 0) sh->job[1] = 0;
        return;
    }
    int lo = 0, hi = __reduce_max_sync(~0u, kn + kTile - 1) / kTile + 1;  // more than t pairs at lo, not so at hi
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (static_cast<int>(__reduce_add_sync(~0u, at_least(mid))) > t) lo = mid;
        else hi = mid;
    }
    const int above = at_least(lo + 1), mine = at_least(lo) - above;
    int end = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, end, o);
        if (lane >= o) end += y;
    }
    const int rank = t - static_cast<int>(__reduce_add_sync(~0u, above));
    if (rank >= end - mine && rank < end) {
        sh->job[0] = a;
        sh->job[1] = n;
        sh->job[2] = ka;
        sh->job[3] = kn;
        sh->job[4] = (pairs - above - 1 - (rank - (end - mine))) * 2 * kTile;
    }
}

// The t-th tile pair, counted from the last pair of the last sequence (the
// last pairs of a causal sequence see the most keys: they start first).  One
// warp; job[1] = 0: there are fewer.  `all`: look at every sequence.
__device__ __forceinline__ void find_job(const PromptParams& p, int t, bool all, Shared* sh) {
    if (p.B > 1 && p.B <= 32) return find_job_by_cost(p, t, all, sh);
    const int lane = threadIdx.x & 31;
    int before = 0;
    bool good = true, found = false;
    for (int s0 = p.B - 1; s0 >= 0; s0 -= 32) {
        const int s = s0 - lane;
        int a = 0, n = 0, ka = 0, kn = 0;
        if (s >= 0) {
            good &= seq_rows(p.cu_q, s, p.Tq, &a, &n);
            good &= seq_rows(p.cu_k, s, p.Tk, &ka, &kn);
        }
        const int tiles = (n + 2 * kTile - 1) / (2 * kTile);
        int end = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(~0u, end, o);
            if (lane >= o) end += y;
        }
        end += before;
        if (t >= end - tiles && t < end) {
            sh->job[0] = a;
            sh->job[1] = n;
            sh->job[2] = ka;
            sh->job[3] = kn;
            sh->job[4] = (end - 1 - t) * 2 * kTile;
            found = true;
        }
        before = __shfl_sync(~0u, end, 31);
        if (!all && before > t) break;
    }
    if (!__any_sync(~0u, found) && lane == 0) sh->job[1] = 0;
    if (all && !__all_sync(~0u, good) && lane == 0) raise_status(p.status, kStatusSeqRange);
}

// Two INT8 codes (bytes of `four`, named by the byte selector 0x4b4a) as BF16:
// with the low seven bits of a code as the fraction of 128 and its sign bit
// turning 128 into 256, code = (128 + low) - (128 or 256) exactly.
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t four, uint32_t selector) {
    const uint32_t two = __byte_perm(four, 0, selector);
    const uint32_t a = (two & 0x007F007Fu) | 0x43004300u, b = (two & 0x00800080u) | 0x43004300u;
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// True if the 64 values of a v row's chunk are finite: x * 0 added up stays 0
// unless an x is infinite or NaN.
__device__ __forceinline__ bool finite_row(uint32_t smem, int row) {
    const int lane = threadIdx.x & 31;
    uint32_t w[8][4], acc[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) ld_shared_v4(smem + row * 128 + (((i + lane) & 7) << 4), w[i][0], w[i][1], w[i][2], w[i][3]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[k]) : "r"(w[i][k]), "r"(0));
    return ((acc[0] | acc[1] | acc[2] | acc[3]) & 0x7FFF7FFFu) == 0;
}

// Zeroes what no row may multiply, in one slot of v: rows behind the sequence's
// end, and NaN or infinite elements (in tiles where the mask hides keys from
// some rows); their keys are noted, and the rows that do see them add them in
// the epilogue.  One key row per thread of the warpgroup.
__device__ __forceinline__ void clean_v(uint32_t smem, int row, bool inside, uint32_t* bad) {
    const int lane = threadIdx.x & 31;
    if (!inside) {
#pragma unroll
        for (int i = 0; i < 8; ++i) st_shared_v4(smem + row * 128 + (((i + lane) & 7) << 4), 0, 0, 0, 0);
    } else if (!finite_row(smem, row)) {
        atomicOr(bad + (row >> 5), 1u << (row & 31));  // noted before it is gone
        __threadfence_block();
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            const uint32_t at = smem + row * 128 + (((i + lane) & 7) << 4);
            uint32_t w[4];
            ld_shared_v4(at, w[0], w[1], w[2], w[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if ((w[k] & 0x7F80u) == 0x7F80u) w[k] &= 0xFFFF0000u;
                if ((w[k] & 0x7F800000u) == 0x7F800000u) w[k] &= 0xFFFFu;
            }
            st_shared_v4(at, w[0], w[1], w[2], w[3]);
        }
    }
}

// Joins what the S CTAs of a cluster made of a tile pair's rows, each from its
// share of the keys: O (not divided by the row sum) and, behind it, (ms, sum) of
// every row lie in each one's shared memory at `sm`, with rows of `pitch`
// bytes whose 16-byte pieces are turned by the row.  Each CTA takes 256 / S of
// the rows, a warp 32 / S, eight loads of O in flight.
template <int S, class RowsOf, class Limit>
__device__ __forceinline__ void join_rows(const PromptParams& p, const Job& jb, int h, int hk, uint32_t sm, int pitch,
                                          uint32_t bad, int first_masked, int rank, RowsOf rows_of, Limit limit) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t sm_of[S], words = 0;  // lane w: word w of the keys whose v holds a NaN or an infinity, of any CTA
#pragma unroll
    for (int k = 0; k < S; ++k) {
        sm_of[k] = map_shared_rank(sm, k);
        if (lane < 12) words |= ld_cluster_u32(map_shared_rank(bad, k) + lane * 4);
    }
    const uint32_t any_bad = __ballot_sync(~0u, words != 0);
    const bool in = lane * 4 < p.Dv;
    constexpr int kAtOnce = 8 / S;
#pragma unroll 1
    for (int k0 = 0; k0 < 32 / S; k0 += kAtOnce) {
        const int row0 = rank * (2 * kTile / S) + warp * (32 / S) + k0;
        float4 o[kAtOnce][S];
        float2 st[kAtOnce][S];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
            for (int k = 0; k < S; ++k) {
                const int r = row0 + i;
                st[i][k] = ld_cluster_f2(sm_of[k] + 2 * kTile * pitch + r * 8);
                o[i][k] = in ? ld_cluster_f4(sm_of[k] + r * pitch + ((lane ^ (r & 7)) << 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int t = (row0 + i) / kTile, r = (row0 + i) % kTile;
            if (r >= rows_of(t)) continue;
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int k = 0; k < S; ++k)
                if (st[i][k].y != 0.f) top = fmaxf(top, st[i][k].x);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < S; ++k) {
                if (st[i][k].y == 0.f) continue;  // no key of this share: its O was not written
                const float w = ex2(st[i][k].x - top);
                sum = fmaf(w, st[i][k].y, sum);
                acc.x = fmaf(w, o[i][k].x, acc.x), acc.y = fmaf(w, o[i][k].y, acc.y);
                acc.z = fmaf(w, o[i][k].z, acc.z), acc.w = fmaf(w, o[i][k].w, acc.w);
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            float v[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
            const int row = jb.r0 + t * kTile + r, lim = limit(row);
            if (any_bad)
                for (int w = 0; w < 12; ++w)
                    for (uint32_t bits = __shfl_sync(~0u, words, w); bits; bits &= bits - 1) {
                        const int key = (first_masked + w / 4) * kTile + (w & 3) * 32 + __ffs(bits) - 1;
                        if (key >= lim || !in) continue;
                        const uint16_t* x = p.v + ((static_cast<int64_t>(jb.k0) + key) * p.Hk + hk) * p.Dv + lane * 4;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if ((x[e] & 0x7F80) == 0x7F80) v[e] += __uint_as_float(static_cast<uint32_t>(x[e]) << 16);
                    }
            const int64_t at = (static_cast<int64_t>(jb.q0) + row) * p.H + h;
            if (in)
                *reinterpret_cast<uint2*>(p.out + at * p.Dv + lane * 4) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
            if (lane == 0 && p.lse) p.lse[at] = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum);
        }
    }
}

template <bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    mla_attend_prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                             const __grid_constant__ CUtensorMap tm_v, const PromptParams p) {
    extern __shared__ uint8_t raw[];
    const uint32_t raw_at = smem_u32(raw);
    const uint32_t pad = (1024u - (raw_at & 1023u)) & 1023u;
    const int nqk = (p.Dqk + 63) / 64, nv = (p.Dv + 63) / 64;
    const uint32_t sm_q = raw_at + pad, sm_ring = sm_q + 2 * nqk * kSlotBytes;
    Shared* sh = reinterpret_cast<Shared*>(raw + pad + (2 * nqk + p.slots) * kSlotBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // blockIdx -> (group of heads, tile pair, head of the group, share of the keys)
    const int shift = kSplit ? p.shift : 0, split = 1 << shift, rank = blockIdx.x & (split - 1);
    const int per_group = p.head_group * p.tile_bound;
    const int g = (blockIdx.x >> shift) / per_group, in_group = (blockIdx.x >> shift) % per_group;
    const int width = min(p.head_group, p.H - g * p.head_group);
    const int tile = in_group / width, h = g * p.head_group + in_group % width;
    const int hk = h / (p.H / p.Hk);
    if (warp == 0) {
        pdl_wait();
        find_job(p, tile, blockIdx.x == 0, sh);
    }
    if (warp == kLoadWarp && lane == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&sh->q_full[t]), p.q8 ? kTile : 1);
            mbar_init(smem_u32(&sh->s_full[t]), 1);
            mbar_init(smem_u32(&sh->p_full[t]), kTile);
            mbar_init(smem_u32(&sh->o_done[t]), 1);
        }
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(smem_u32(&sh->k_full[i]), 1);
            mbar_init(smem_u32(&sh->v_full[i]), 1);
            mbar_init(smem_u32(&sh->k_free[i]), 1);
            mbar_init(smem_u32(&sh->v_free[i]), 1);
        }
        mbar_init(smem_u32(&sh->drain), 1);
        sh->abort_flag = 0;
        for (int i = 0; i < 12; ++i) sh->bad[i] = 0;
        fence_barrier_init();
        if (!p.q8) prefetch_tensormap(&tm_q);
        if (p.Tk) prefetch_tensormap(&tm_k), prefetch_tensormap(&tm_v);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(&sh->tmem), 512);
        tmem_relinquish();
    }
    pdl_wait();  // what the kernel before in the stream wrote
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // The next kernel of the stream may be brought to the SMs, now that this CTA has its TMEM: one that took
    // TMEM first and then waited for this grid would never get to run.
    pdl_launch_dependents();
    const uint32_t tmem = sh->tmem;
    const Job jb{sh->job[0], sh->job[1], sh->job[2], sh->job[3], sh->job[4]};
    if (jb.nq == 0) {
        if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
        return;
    }

    // Keys that row r of the sequence sees: [0, limit(r)).
    const int off = jb.nk - jb.nq;
    auto limit = [&](int r) { return p.causal ? clampi(off + r + 1, 0, jb.nk) : jb.nk; };
    auto rows_of = [&](int t) { return clampi(jb.nq - jb.r0 - t * kTile, 0, kTile); };
    auto tiles_of = [&](int t) {
        const int rows = rows_of(t);
        return rows ? (limit(jb.r0 + t * kTile + rows - 1) + kTile - 1) / kTile : 0;
    };
    // this CTA's key tiles: the rank-th of every `split` (the tiles at a causal row's end hold less work)
    auto share = [&](int n) { return (max(n - rank, 0) + split - 1) >> shift; };
    const int n0 = share(tiles_of(0)), n1 = share(tiles_of(1)), nmax = max(n0, n1);
    const int first_masked = limit(jb.r0) / kTile;
    const int span = nqk + nv;  // ring slots per key tile: K's, then V's
    auto phase_of = [&](int j) { return static_cast<uint32_t>(j / kAhead) & 1u; };  // of key tile j's barriers
    const int pitch = (p.Dv + 31) / 32 * 128;  // bytes of a row of O in shared memory
    const volatile int* abort_flag = &sh->abort_flag;
    bool ok = true;

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        const int t = warp >> 2, r = threadIdx.x & 127;  // r: TMEM lane, row of the tile
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + kColS + t * kTile, to = tmem + lanes + kColO + t * kTile;
        const int row = jb.r0 + t * kTile + r;                    // of the sequence
        const int64_t at = (static_cast<int64_t>(jb.q0) + row) * p.H + h;  // of out and lse
        const int rows = rows_of(t), n = t ? n1 : n0;
        const bool mine = r < rows;
        float c = p.scale * kLog2e;
        if (p.q8 && n) {
            const float qs = mine ? p.q_scale[p.q_per_head ? at : jb.q0 + row] : 0.f;
            c *= fabsf(qs);  // a negative scale turns the codes' sign, so that c > 0 keeps the order of the scores
            if (c < 1e-30f) c = 1e-30f;  // a zero row: its scores are 0 (hidden ones stay -inf)
            // The warp's 32 rows of codes in pieces of 16, a lane's pieces 32 apart: neighbouring lanes read
            // neighbouring pieces of a row.  Up to 12 loads (Dqk = 192) are in flight.
            const int8_t* rows8 = p.q8 + (at - static_cast<int64_t>(r & 31) * p.H) * p.Dqk;
            const int64_t row_pitch = static_cast<int64_t>(p.H) * p.Dqk;
            const int pieces = p.Dqk / 16, wrow = (warp & 3) * 32, wrows = clampi(rows - wrow, 0, 32);
            const int row_step = 32 / pieces, piece_step = 32 % pieces;
            const uint32_t negative = __ballot_sync(~0u, qs < 0.f);
            int row0 = lane / pieces, piece0 = lane % pieces;  // of this lane's next load
            int row1 = row0, piece1 = piece0;                  // of its next store
            auto advance = [&](int& row, int& piece) {
                row += row_step;
                piece += piece_step;
                if (piece >= pieces) piece -= pieces, ++row;
            };
#pragma unroll 1
            for (int k0 = 0; k0 < pieces; k0 += 12) {
                uint4 w[12];
#pragma unroll
                for (int k = 0; k < 12; ++k) {
                    w[k] = k0 + k < pieces && row0 < wrows
                               ? *reinterpret_cast<const uint4*>(rows8 + row0 * row_pitch + piece0 * 16)
                               : make_uint4(0, 0, 0, 0);
                    advance(row0, piece0);
                }
#pragma unroll
                for (int k = 0; k < 12; ++k) {
                    if (k0 + k >= pieces) break;
                    const uint32_t turn = (negative >> row1 & 1u) ? 0x80008000u : 0u;
                    const uint32_t dst = sm_q + (t * nqk + (piece1 >> 2)) * kSlotBytes + (wrow + row1) * 128;
                    const uint32_t c16 = (piece1 & 3) * 2;
                    st_shared_v4(dst + ((c16 ^ (row1 & 7)) << 4), codes_bf16x2(w[k].x, 0x4140) ^ turn,
                                 codes_bf16x2(w[k].x, 0x4342) ^ turn, codes_bf16x2(w[k].y, 0x4140) ^ turn,
                                 codes_bf16x2(w[k].y, 0x4342) ^ turn);
                    st_shared_v4(dst + (((c16 + 1) ^ (row1 & 7)) << 4), codes_bf16x2(w[k].z, 0x4140) ^ turn,
                                 codes_bf16x2(w[k].z, 0x4342) ^ turn, codes_bf16x2(w[k].w, 0x4140) ^ turn,
                                 codes_bf16x2(w[k].w, 0x4342) ^ turn);
                    advance(row1, piece1);
                }
            }
            fence_proxy_async_shared();
            mbar_arrive(smem_u32(&sh->q_full[t]));
        }
        const int lim = mine ? limit(row) : jb.nk;
        const int lim0 = limit(jb.r0 + t * kTile);  // of the tile's first row, which sees the fewest
        float m = -INFINITY, ms = 0.f, l = 0.f;     // row maximum of S, ms = m c, row sum of P
        for (int j = 0; j < n; ++j) {
            const int key0 = ((j << shift) + rank) * kTile;
            ok = mbar_wait(smem_u32(&sh->s_full[t]), j & 1, kTimeoutNs, abort_flag);
            if (!__all_sync(~0u, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t s[kTile];
            float mt = tmem_ld128_max(ts, s);  // of the row
            const bool masked = key0 + kTile > lim0;
            if (masked) {
                const int left = lim - key0;
#pragma unroll
                for (int i = 0; i < kTile; ++i)
                    if (i >= left) s[i] = 0xFF800000u;
                mt = -INFINITY;
#pragma unroll
                for (int i = 0; i < kTile; ++i) mt = fmaxf(mt, __uint_as_float(s[i]));
            }
            // rows that have no maximum yet take this tile's; the others only one that has grown by the slack
            const bool grow = mt > m && (m == -INFINITY || mt * c > ms + kSlack);
            if (__any_sync(~0u, grow)) {
                float alpha = 1.f;
                if (mt > m) {
                    const float next = mt * c;
                    if (m != -INFINITY) alpha = ex2(ms - next);
                    m = mt;
                    ms = next;
                }
                l *= alpha;
                if (j > 0 && __any_sync(~0u, alpha != 1.f)) {
                    ok = mbar_wait(smem_u32(&sh->o_done[t]), (j - 1) & 1, kTimeoutNs, abort_flag);
                    if (!__all_sync(~0u, ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int d = 0; d < p.Dv; d += 16) {
                        float o[16];
                        tmem_ld16(to + d, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= alpha;
                        tmem_st16(to + d, o);
                    }
                }
            }
            const uint64_t cc = pk2(c, c), mm = pk2(-ms, -ms);
            uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
            for (int b = 0; b < kTile; b += 32) {
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    float e0, e1, e2, e3;
                    upk2(fma2(pk2(__uint_as_float(s[b + i]), __uint_as_float(s[b + i + 1])), cc, mm), e0, e1);
                    upk2(fma2(pk2(__uint_as_float(s[b + i + 2]), __uint_as_float(s[b + i + 3])), cc, mm), e2, e3);
                    e0 = ex2(e0), e1 = ex2(e1), e2 = ex2(e2), e3 = ex2(e3);
                    sum0 = add2(sum0, pk2(e0, e1));
                    sum1 = add2(sum1, pk2(e2, e3));
                    w[i >> 1] = pack_bf16x2(e0, e1);
                    w[(i >> 1) + 1] = pack_bf16x2(e2, e3);
                }
                tmem_st16_raw(ts + b / 2, w);
            }
            float a0, a1;
            upk2(add2(sum0, sum1), a0, a1);
            l += a0 + a1;
            if (masked) {
                const int use = j * span + nqk;
                ok = mbar_wait(smem_u32(&sh->v_full[j % kAhead]), phase_of(j), kTimeoutNs, abort_flag);
                if (!__all_sync(~0u, ok)) {
                    ok = false;
                    break;
                }
                for (int cidx = 0; cidx < nv; ++cidx)
                    clean_v(sm_ring + (use + cidx) % p.slots * kSlotBytes, r, key0 + r < jb.nk,
                            sh->bad + (key0 / kTile - first_masked) * 4);
                fence_proxy_async_shared();
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(smem_u32(&sh->p_full[t]));
        }
        if (lim == 0) l = 0.f;  // a row without a key, whatever its scale: NaN would have come through the hidden scores
        if (ok && n) {
            ok = mbar_wait(smem_u32(&sh->o_done[t]), (n - 1) & 1, kTimeoutNs, abort_flag);
            ok = __all_sync(~0u, ok);
            tc_fence_after();
        }
        if (kSplit) {
            // The tiles have been read when both warpgroups' products are made: O and the sums take their place.
            const bool all = named_bar_and(1, 2 * kTile, ok);
            if (all) {
                const uint32_t sm_o = sm_q + (t * kTile + r) * pitch;
                if (n)
#pragma unroll 1
                    for (int d = 0; d < p.Dv; d += 32) {  // (what lies behind v_dim is not read)
                        float o[32];
                        tmem_ld32(to + d, o);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            st_shared_v4(sm_o + (((d / 4 + i) ^ (r & 7)) << 4), __float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]),
                                         __float_as_uint(o[4 * i + 2]), __float_as_uint(o[4 * i + 3]));
                    }
                st_shared_v2(sm_q + 2 * kTile * pitch + (t * kTile + r) * 8, __float_as_uint(ms), __float_as_uint(l));
            }
        } else if (ok && rows) {
            uint32_t any_bad = 0;
#pragma unroll
            for (int i = 0; i < 12; ++i) any_bad |= *const_cast<volatile uint32_t*>(sh->bad + i);
            const float inv = l == 0.f ? 0.f : 1.f / l;
            // A warp's rows pass through its part of the tile's Q (no score is left to make), 64 columns at a
            // time, so that it stores four rows' whole lines at once.
            const uint32_t stage = sm_q + t * nqk * kSlotBytes + (warp & 3) * 32 * 128;
            const int64_t row_bytes = static_cast<int64_t>(p.H) * p.Dv * 2;
            uint8_t* rows_out = reinterpret_cast<uint8_t*>(p.out + (at - static_cast<int64_t>(lane) * p.H) * p.Dv);
            const int wrows = clampi(rows - (warp & 3) * 32, 0, 32);
#pragma unroll 1
            for (int d = 0; d < p.Dv; d += 64) {
                float o[64];  // (what lies behind v_dim is not stored)
                if (n) {
                    uint32_t raw_o[64];
                    tmem_ld64_raw(to + d, raw_o);
#pragma unroll
                    for (int i = 0; i < 64; ++i) o[i] = l == 0.f ? 0.f : __uint_as_float(raw_o[i]) * inv;
                } else {
#pragma unroll
                    for (int i = 0; i < 64; ++i) o[i] = 0.f;
                }
                if (any_bad) {
                    for (int w = 0; w < 12; ++w)
                        for (uint32_t bits = *const_cast<volatile uint32_t*>(sh->bad + w); bits; bits &= bits - 1) {
                            const int key = (first_masked + w / 4) * kTile + (w & 3) * 32 + __ffs(bits) - 1;
                            if (key >= lim) continue;
                            const uint16_t* v = p.v + ((static_cast<int64_t>(jb.k0) + key) * p.Hk + hk) * p.Dv + d;
#pragma unroll
                            for (int i = 0; i < 64; ++i)
                                if (d + i < p.Dv && (v[i] & 0x7F80) == 0x7F80)
                                    o[i] += __uint_as_float(static_cast<uint32_t>(v[i]) << 16);
                        }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    st_shared_v4(stage + lane * 128 + ((i ^ (lane & 7)) << 4), pack_bf16x2(o[8 * i], o[8 * i + 1]),
                                 pack_bf16x2(o[8 * i + 2], o[8 * i + 3]), pack_bf16x2(o[8 * i + 4], o[8 * i + 5]),
                                 pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row2 = i * 4 + (lane >> 3), col = d + (lane & 7) * 8;
                    uint4 v;
                    ld_shared_v4(stage + row2 * 128 + (((lane & 7) ^ (row2 & 7)) << 4), v.x, v.y, v.z, v.w);
                    if (row2 < wrows && col < p.Dv) *reinterpret_cast<uint4*>(rows_out + row2 * row_bytes + col * 2) = v;
                }
                __syncwarp();
            }
            if (mine && p.lse) p.lse[at] = l == 0.f ? -INFINITY : ms * kLn2 + logf(l);
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- MMA
        if (elect_one()) {
            const uint32_t idesc_s = idesc_bf16_f32(kTile, kTile);
            const uint32_t idesc_o = idesc_bf16_f32(kTile, p.Dv) | kIdescBMnMajor;
            constexpr uint32_t kSlotStep = kSlotBytes >> 4;
            const uint64_t dq = smem_desc_sw128(sm_q), dk = smem_desc_sw128(sm_ring);
            const uint64_t dv = smem_desc_sw128_mn(sm_ring, kSlotBytes);
            const int ksteps = p.Dqk / 16;
            // slots of the key tile at hand: the descriptors of K's chunks, and V's first slot
            int at = 0;
            uint64_t kd[4];
            auto take = [&](int count) {
                const int x = at;
                at += count;
                if (at >= p.slots) at -= p.slots;
                return x;
            };
            auto take_k = [&]() {
                int x = take(nqk);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    kd[c] = dk + x * kSlotStep;
                    if (++x == p.slots) x = 0;
                }
            };
            auto scores = [&](int t, int j, bool last) {
                const uint64_t a = dq + t * nqk * kSlotStep;
                const uint32_t d = tmem + kColS + t * kTile;
                auto run = [&](auto steps) {
#pragma unroll
                    for (int k = 0; k < decltype(steps)::value; ++k)
                        mma_bf16(d, a + (k >> 2) * kSlotStep + 2 * (k & 3), kd[k >> 2] + 2 * (k & 3), idesc_s, k > 0);
                };
                if (ksteps == 12) run(Steps<12>());
                else if (ksteps == 8) run(Steps<8>());
                else if (ksteps == 4) run(Steps<4>());
                else
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        for (int k = 0; k < 4 && c * 4 + k < ksteps; ++k)
                            mma_bf16(d, a + c * kSlotStep + 2 * k, kd[c] + 2 * k, idesc_s, c > 0 || k > 0);
                mma_commit(smem_u32(&sh->s_full[t]));
                if (last) mma_commit(smem_u32(&sh->k_free[j % kAhead]));
            };
            auto values = [&](int t, int j, int slot, bool last) {
                const uint32_t o = tmem + kColO + t * kTile, pr = tmem + kColS + t * kTile;
                const uint64_t b = dv + slot * kSlotStep;
                // one product over V's two slots where they are neighbours, two of 64 columns where the ring wraps
                if (nv == 1 || slot + 1 < p.slots) {
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        mma_bf16_ts(o, pr + k * 8, b + k * (2048 >> 4), idesc_o, j > 0 || k > 0);
                } else {
                    const uint32_t id0 = (idesc_o & ~(0x3Fu << 17)) | 8u << 17;
                    const uint32_t id1 = (idesc_o & ~(0x3Fu << 17)) | static_cast<uint32_t>((p.Dv - 64) >> 3) << 17;
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k) {
                        mma_bf16_ts(o, pr + k * 8, b + k * (2048 >> 4), id0, j > 0 || k > 0);
                        mma_bf16_ts(o + 64, pr + k * 8, dv + k * (2048 >> 4), id1, j > 0 || k > 0);
                    }
                }
                mma_commit(smem_u32(&sh->o_done[t]));
                if (last) mma_commit(smem_u32(&sh->v_free[j % kAhead]));
            };
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                ok = ok && mbar_wait(smem_u32(bar), parity, kTimeoutNs, abort_flag);
                tc_fence_after();
                return ok;
            };
            take_k();
            if (n0 && wait(&sh->q_full[0], 0) && wait(&sh->k_full[0], 0)) scores(0, 0, n1 == 0);
            if (n1 && wait(&sh->q_full[1], 0) && wait(&sh->k_full[0], 0)) scores(1, 0, true);
            for (int j = 0; j < nmax && ok; ++j) {
                const int v = take(nv);
                take_k();
                if (!wait(&sh->v_full[j % kAhead], phase_of(j))) break;
                if (j < n0) {
                    if (!wait(&sh->p_full[0], j & 1)) break;
                    values(0, j, v, j >= n1);
                    if (j + 1 < n0) {
                        if (!wait(&sh->k_full[(j + 1) % kAhead], phase_of(j + 1))) break;
                        scores(0, j + 1, j + 1 >= n1);
                    }
                }
                if (j < n1) {
                    if (!wait(&sh->p_full[1], j & 1)) break;
                    values(1, j, v, true);
                    if (j + 1 < n1) {
                        if (!wait(&sh->k_full[(j + 1) % kAhead], phase_of(j + 1))) break;
                        scores(1, j + 1, true);
                    }
                }
            }
            if (!ok) {  // no MMA may still run when the CTA leaves
                mma_commit(smem_u32(&sh->drain));
                mbar_wait(smem_u32(&sh->drain), 0, kTimeoutNs, nullptr);
            }
        }
    } else if (lane == 0) {
        // --------------------------------------------------------------- TMA
        // Tiles go out in the order of their use (K 0, V 0, K 1, ...), each as soon as the ring has room for it.
        int slot = 0, room = p.slots, q_loaded = 0, sent = 0, freed = 0;  // sent, freed: tiles 2 j (K) and 2 j + 1 (V)
        auto load_q = [&](int t) {
            if (p.q8 || !(t ? n1 : n0)) return;
            mbar_arrive_expect_tx(smem_u32(&sh->q_full[t]), nqk * kSlotBytes);
            for (int c = 0; c < nqk; ++c)
                tma_load_3d(sm_q + (t * nqk + c) * kSlotBytes, &tm_q, smem_u32(&sh->q_full[t]), c * 64, h,
                            jb.q0 + jb.r0 + t * kTile);
            q_loaded |= 1 << t;
        };
        auto load = [&](const CUtensorMap* map, uint64_t* full, int chunks, int j) {
            while (ok && (room < chunks || freed < sent - 2 * kAhead + 1)) {
                const int f = freed >> 1;
                ok = mbar_wait(smem_u32(freed & 1 ? &sh->v_free[f % kAhead] : &sh->k_free[f % kAhead]), phase_of(f),
                               kTimeoutNs, abort_flag);
                room += freed & 1 ? nv : nqk;
                ++freed;
            }
            if (!ok) return;
            room -= chunks;
            ++sent;
            mbar_arrive_expect_tx(smem_u32(&full[j % kAhead]), chunks * kSlotBytes);
            for (int c = 0; c < chunks; ++c) {
                tma_load_3d(sm_ring + slot * kSlotBytes, map, smem_u32(&full[j % kAhead]), c * 64, hk,
                            jb.k0 + ((j << shift) + rank) * kTile);
                if (++slot == p.slots) slot = 0;
            }
        };
        load_q(0);
        for (int j = 0; j < nmax && ok; ++j) {
            load(&tm_k, sh->k_full, nqk, j);
            if (j == 0) load_q(1);
            load(&tm_v, sh->v_full, nv, j);
        }
        // no copy may still be landing when the CTA leaves
        for (int u = max(sent - 2 * kAhead, 0); u < sent; ++u)
            mbar_wait(smem_u32(u & 1 ? &sh->v_full[(u >> 1) % kAhead] : &sh->k_full[(u >> 1) % kAhead]), phase_of(u >> 1),
                      kTimeoutNs, nullptr);
        for (int t = 0; t < 2; ++t)
            if (q_loaded >> t & 1) mbar_wait(smem_u32(&sh->q_full[t]), 0, kTimeoutNs, nullptr);
        // and what the tensor core frees has arrived (it ends before the epilogue does)
        for (int u = max(sent - 2 * kAhead, 0); u < sent; ++u)
            ok = ok && mbar_wait(smem_u32(u & 1 ? &sh->v_free[(u >> 1) % kAhead] : &sh->k_free[(u >> 1) % kAhead]),
                                 phase_of(u >> 1), kTimeoutNs, abort_flag);
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
    if (kSplit) {
        __syncwarp();
        cluster_sync_all();
        if (warp < 8) {
            auto join = [&](auto s) {
                join_rows<decltype(s)::value>(p, jb, h, hk, sm_q, pitch, smem_u32(sh->bad), first_masked, rank, rows_of, limit);
            };
            if (split == 2) join(Steps<2>());
            else if (split == 4) join(Steps<4>());
            else join(Steps<8>());
        }
        __syncwarp();
        cluster_sync_all();  // no CTA leaves while another reads its shared memory
    }
}

// Clusters of 1 << shift CTAs of the current device that run at the same time
// (asked of the driver once per device).
cudaError_t clusters_at_once(int shift, int* most) {
    static std::atomic<int> known[64][kMaxShift + 1];  // 0: not asked yet, else the answer + 1
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64) {
        const int k = known[dev][shift].load(std::memory_order_acquire);
        if (k) return *most = k - 1, cudaSuccess;
    }
    static std::atomic<uint64_t> ready{0};
    e = allow_smem(&mla_attend_prompt_kernel<true>, kSmemMax, &ready);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(1u << shift);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemMax;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << shift;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    e = cudaOccupancyMaxActiveClusters(most, &mla_attend_prompt_kernel<true>, &cfg);
    if (e == cudaSuccess && dev < 64) known[dev][shift].store(*most + 1, std::memory_order_release);
    return e;
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
        d->v_dim < 16 || d->v_dim > 128 || d->v_dim % 16 || d->Tq > (1 << 30) || d->Tk > (1 << 30) || !scale_ok(d->scale))
        return MLA_ERR_UNSUPPORTED_DIMS;
    if (int8 ? !ptr_ok(q_scale, 4) : q_scale != nullptr) return MLA_ERR_INVALID_ARG;
    if (d->Tq == 0 || d->sequences == 0) return MLA_OK;
    if (!ptr_ok(q, 16) || !ptr_ok(out, 16) || !ptr_ok(cu_q, 4) || !ptr_ok(cu_k, 4)) return MLA_ERR_INVALID_ARG;
    if (d->Tk && (!ptr_ok(k, 16) || !ptr_ok(v, 16))) return MLA_ERR_INVALID_ARG;
    if ((lse && !ptr_ok(lse, 4)) || (status && !ptr_ok(status, 4))) return MLA_ERR_INVALID_ARG;
    // 256-row tiles of sequences that hold a row: each wastes 255 rows at most
    const int64_t ragged = d->sequences < d->Tq ? d->sequences : d->Tq;
    const int64_t tiles = (d->Tq + (2 * kTile - 1) * ragged) / (2 * kTile);
    const int64_t jobs = tiles * d->num_heads;
    if (jobs > INT32_MAX) return MLA_ERR_UNSUPPORTED_DIMS;
    int sms;
    const int rc = current_sm103(&sms);
    if (rc != MLA_OK) return rc;
    CUtensorMap tq, tk, tv;
    bool good = true;
    if (!int8) good &= encode_bf16_3d(&tq, q, d->qk_dim, d->num_heads, d->Tq, 1, kTile);
    if (d->Tk) {
        good &= encode_bf16_3d(&tk, k, d->qk_dim, d->kv_heads, d->Tk, 1, kTile);
        good &= encode_bf16_3d(&tv, v, d->v_dim, d->kv_heads, d->Tk, 1, kTile);
    }
    if (!good) return report_cuda(cudaErrorInvalidValue, "tensor maps of attend_prompt");
    if (int8) tq = d->Tk ? tk : CUtensorMap{};  // not read
    if (!d->Tk) tk = tv = tq;                   // not read
    const int nqk = (d->qk_dim + 63) / 64;
    int slots = (kSmemMax - 1024 - kMiscBytes) / kSlotBytes - 2 * nqk;
    if (slots > kMaxSlots) slots = kMaxSlots;
    const int smem = 1024 + kMiscBytes + (2 * nqk + slots) * kSlotBytes;
    // Heads go in groups whose K and V fit L2 together, and within a group the
    // tile pairs with the most keys first: few heads at a time keep K and V on
    // chip when they are large, many spread uneven tiles over the SMs when
    // they are small.  In us, groups of 12 / 24 / 48 / 96 MB / all heads: eight
    // ragged prompts 63 / 57 / 43 / 43 / 43; four V3 prompts 979 / 949 / 961 / 933
    // / 1073; V3 16384 6850 / 6877 / 6843 / 7052 / 8085.  Groups are made alike,
    // so that a small last one does not leave SMs idle (961: 14 of 9 heads and one
    // of 2; 12 of 10 and one of 8: 931).
    const int64_t kv_bytes = static_cast<int64_t>(d->Tk) * (d->qk_dim + d->v_dim) * 2;
    const int per_kv = d->num_heads / d->kv_heads;
    int64_t group = kv_bytes > 0 ? (int64_t(48) << 20) / kv_bytes : d->kv_heads;
    group = group < 1 ? 1 : group > d->kv_heads ? d->kv_heads : group;
    const int64_t groups = d->kv_heads / group;
    group = (d->kv_heads + groups - 1) / groups * per_kv;
    // Few tile pairs with many keys: a cluster shares a tile pair's keys, as large a one as leaves room for all of
    // them at once.  In us, on 1 / 2 / 4 / 8 CTAs, D 192: 4 pairs of 156 key tiles 218 / 115 / 63 / 37; 16 pairs
    // 220 / 116 / 65 / 78 (their clusters of 8 do not fit at once); 32 pairs of 64 tiles 125 / 72 / 44 / 77; 64 pairs
    // of 8 tiles 21.8 / 19.8 / 30 / 67; 128 pairs of 32 tiles 60 / 77.  Short ones have nothing to share: 16 pairs of
    // 2 tiles 12.1 / 14.2 / 13.9 / 26.
    int shift = 0;
    if (d->Tk >= kSplitTiles * kTile * static_cast<int64_t>(d->sequences)) {
        for (shift = kMaxShift; shift > 0; --shift) {
            int most = 0;
            const cudaError_t e = clusters_at_once(shift, &most);
            if (e != cudaSuccess) return report_cuda(e, "clusters of mla_attend_prompt_kernel");
            if (jobs <= most) break;
        }
    }
    PromptParams p{int8 ? static_cast<const int8_t*>(q) : nullptr, q_scale, static_cast<const uint16_t*>(v), cu_q, cu_k,
                   static_cast<uint16_t*>(out), lse, status, d->Tq, d->Tk, d->sequences, d->num_heads, d->kv_heads,
                   d->qk_dim, d->v_dim, d->scale, (d->flags & MLA_PROMPT_CAUSAL) != 0, per_head, slots, shift,
                   static_cast<int>(tiles), static_cast<int>(group)};
    static std::atomic<uint64_t> ready[2];
    auto kernel = shift ? &mla_attend_prompt_kernel<true> : &mla_attend_prompt_kernel<false>;
    cudaError_t e = allow_smem(kernel, kSmemMax, &ready[shift ? 1 : 0]);
    if (e != cudaSuccess) return report_cuda(e, "mla_attend_prompt_kernel attributes");
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(jobs << shift));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = shift ? 2 : 1;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1u << shift;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, tq, tk, tv, p);
    return e == cudaSuccess ? MLA_OK : report_cuda(e, "launch mla_attend_prompt_kernel");
}
