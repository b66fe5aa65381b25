// One decoding step over the latent cache in 8 bits for more than 64 heads:
// mla_prolog_attend_cache8 (the mathematics and precision: attend_cache8.cu).
//
// A tile is 128 heads of one sequence on 128 keys a step, worked on by a pair of
// CTAs (cta_group::2, M = 128): each has 64 of the heads, and both multiply them
// by keys and values that each brings half of.  Heads run along the lanes:
//
//   S [heads][keys] = (Qh + Ql) K^T          N = 128, C deep, twice
//   O [heads][value columns] += (P4 + P5) V   N = 256, 128 keys deep, twice
//
// In each CTA the products' operands are 331 KB of shared memory a step, where
// with keys along the lanes they would be 433 KB for the same heads and keys, and
// a key's place is free once its scores are made.  The tensor core spreads the
// columns of a CTA's 64 rows over both halves of the lanes: a row belongs to four
// threads, one for each 32 keys of a step and a quarter of the value columns.
//
// What bounds it: the products.  Two terms of 64 heads on 128 keys of 576 and 512
// columns are 17.8 M multiply-adds a step and CTA, 2176 cycles at the tensor
// core's 8192 a cycle (2213 measured alone); a step takes 2.5k (1.25 us) on a few
// pairs, 1.35 us on all of them from L2 and 1.48 from memory.  V3, 32 sequences of
// 2000 to 32768 keys: 132 to 134 us, of which the partial results and their join
// take 12; 128 of up to 1024, dealt whole: 41; one of 131072, 14 steps a pair: 41.
#include <cstdint>

#include "attend_cache8.cuh"

namespace mlap {
namespace {

constexpr int kRows = 64;                             // heads of a CTA
constexpr int kQTerm = kRows * (4 * 128 + 64);        // a term of its query rows,
constexpr int kKeyBytes = 64 * (4 * 128 + 64);        //   its half of a step's keys,
constexpr int kValueChunk = 64 * 256;                 //   its value columns of 64 keys, by 128 columns,
constexpr int kValueBytes = 2 * kValueChunk;
constexpr int kPTerm = kRows * kKeys;                 //   a term of its weights
constexpr int kSmemK = 2 * kQTerm, kSmemV = kSmemK + 2 * kKeyBytes, kSmemP = kSmemV + 2 * kValueBytes, kMisc = kSmemP + 2 * kPTerm;
constexpr int kSmem = kMisc + kMiscBytes;
static_assert(kSmem <= 232448, "227 KB");
static_assert(2 * kQTerm == kPairQBytes, "");
constexpr uint32_t kColO = 0, kColS = 256, kStages = 4;  // TMEM: O, S of so many steps (64 columns each)
constexpr int kScales = 3;                            // steps whose scales are found ahead
constexpr float kFar = 65536.f;                       // a bound whose last bit is 2^-7 of a binade

struct Shared {
    // (of the even CTA for both: k_full, v_full, p_full, q_full, o_free)
    uint64_t k_full[2], v_full[2], s_full[kStages], pv_done[2], p_full, q_full, q_here, q_free, o_free, v_seen, drain;
    uint64_t piece_full[kAhead], piece_free[kAhead], scale_full[kScales], scale_free[kScales];
    uint32_t tmem;
    int abort_flag;
    Piece piece[kAhead];
    alignas(16) float f[3][kRows];           // factors of the heads' scores: of a piece, while its weights are made, and two behind it
    alignas(16) float up[kScales][kKeys];    // scales of a step's keys
};
static_assert(sizeof(Shared) <= kMiscBytes, "");
// What the four threads of a row tell each other, in the place of P while no product reads that.
struct Scratch {
    float top[4][kRows], all[4][kRows], squares[4][kRows], sum[4][kRows];
    alignas(16) uint32_t failed[kSoftWarps];
};
static_assert(sizeof(Scratch) <= 2 * kPTerm, "");

// 4-D tma_load_3d_pair().
__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1, int32_t c2,
                                                 int32_t c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// D[tmem] (+)= A B^T over the pair, 8-bit floats.
__device__ __forceinline__ void mma_pair8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The turns of keys i and i + 1 of 32 that a thread has (attend_cache8.cuh), less half a step, before they are crossed with
// the 32 keys': their numbers' bits backwards, in the upper five.
__host__ __device__ constexpr uint32_t turn_at(int i) {
    return static_cast<uint32_t>((i & 1) << 7 | (i & 2) << 5 | (i & 4) << 3 | (i & 8) << 1 | i >> 1 & 8 | 4) ^ 0x80u;
}
__host__ __device__ constexpr uint32_t turns_at(int i) { return turn_at(i) | turn_at(i + 1) << 16; }

// The score of a row's largest weight and log2 of its key's scale, the same in all four threads of the row: `up` the scales of
// this one's 32 keys, `left` its step's keys.  (A call: the hot loop is not to be longer by it.)
static __device__ __noinline__ float2 far_bound(uint32_t s_at, const float* up, int key_at, int left, Scratch* scratch, int r, int mine,
                                                float f, float from) {
    float top = -INFINITY, score = 0.f, scale = 0.f;
#pragma unroll 1
    for (int c = 0; c < 32; c += 8) {
        float w[8];
        __syncwarp();
        tmem_ld8(s_at + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = w[i] * up[c + i], k = static_cast<float>((__float_as_int(up[c + i]) >> 23) - 127), t = fmaf(y - from, f, k);
            if (key_at + c + i < left && t > top) top = t, score = y, scale = k;  // (NaN is left out)
        }
    }
    scratch->top[mine][r] = top;
    scratch->all[mine][r] = score;
    scratch->squares[mine][r] = scale;
    named_bar_sync(1, kSoft);
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (scratch->top[i][r] > top) top = scratch->top[i][r], score = scratch->all[i][r], scale = scratch->squares[i][r];
    named_bar_sync(1, kSoft);
    return make_float2(score, scale);
}

__global__ void __launch_bounds__(kThreads, 1)
    mla_attend_cache8_pair_kernel(const __grid_constant__ CUtensorMap tm_rows, const __grid_constant__ CUtensorMap tm_rest,
                                  const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                                  const __grid_constant__ Attend8 p) {
    extern __shared__ __align__(1024) uint8_t raw[];
    const uint32_t sm_q = smem_u32(raw), sm_k = sm_q + kSmemK, sm_v = sm_q + kSmemV, sm_p = sm_q + kSmemP;
    Shared* const sh = reinterpret_cast<Shared*>(raw + kMisc);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x / 2, rank = blockIdx.x % 2;
    const int C = p.c.C, chunks = C > 512 ? 4 : (C + 127) / 128, rest = C > 512 ? C - 512 : 0;
    const int half = ((p.Lkv + 127) / 128 + 1) / 2;   // 128-column chunks of values of each CTA

    Walk walk;
    if (warp == kScaleWarp && lane == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh->k_full[i]), 1);
            mbar_init(smem_u32(&sh->v_full[i]), 1);
            mbar_init(smem_u32(&sh->pv_done[i]), 1);
        }
        for (int i = 0; i < static_cast<int>(kStages); ++i) mbar_init(smem_u32(&sh->s_full[i]), 1);
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(smem_u32(&sh->piece_full[i]), 1);
            mbar_init(smem_u32(&sh->piece_free[i]), kSoftWarps + 2 + (rank == 0));  // (values, scales, the MMA thread)
        }
        for (int i = 0; i < kScales; ++i) {
            mbar_init(smem_u32(&sh->scale_full[i]), 1);
            mbar_init(smem_u32(&sh->scale_free[i]), kSoftWarps);
        }
        mbar_init(smem_u32(&sh->p_full), 2 * kSoftWarps);
        mbar_init(smem_u32(&sh->q_full), 2);
        mbar_init(smem_u32(&sh->q_here), 1);
        mbar_init(smem_u32(&sh->q_free), 1);
        mbar_init(smem_u32(&sh->o_free), 2 * kSoftWarps);
        mbar_init(smem_u32(&sh->v_seen), 1);
        mbar_init(smem_u32(&sh->drain), 1);
        sh->abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tm_rows);
        prefetch_tensormap(&tm_rest);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    if (warp == kMmaWarp) {
        tmem_alloc_pair(smem_u32(&sh->tmem), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    pdl_launch_dependents();
    __syncwarp();
    cluster_arrive();  // the peer's barriers are ready once both have come here; the cut is made meanwhile
    uint32_t* const scratch = reinterpret_cast<uint32_t*>(raw + kSmemK);  // (that is empty yet)
    if (p.rounds > 1) deal_tiles(p, unit, scratch);
    if (warp == kLoadWarp) walk.start(p, unit, rank, scratch);
    cluster_wait();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    const volatile int* abort_flag = &sh->abort_flag;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_wait_lean(smem_u32(bar), parity & 1u, kTimeoutNs, abort_flag);
    };
    bool ok = true;
    int step = 0;    // key steps so far, over all pieces: the phase of every barrier of a step
    int pieces = 0;  // pieces so far
    Piece x = {};
    // The next piece, whole warp: false where there is none (or a wait failed).
    auto next_piece = [&]() {
        ok = __all_sync(~0u, ok && wait(&sh->piece_full[pieces % kAhead], pieces / kAhead));
        if (!ok) return false;
        x = sh->piece[pieces % kAhead];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh->piece_free[pieces % kAhead]));
        ++pieces;
        return x.n > 0;
    };
    // One arrival per warp, at the even CTA.
    auto arrive_even = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive_peer(map_shared_rank(smem_u32(bar), 0));
    };

    // Whether a lane has a box of a piece's step j, that begins `mine` keys into it; its page, looked at when it is used;
    // the page that is read then (what lies outside the cache reads as zeros), and the place there.  Whole boxes' keys.
    auto has_box = [&](const Piece& y, int j, int mine, int boxes) { return lane < boxes && j < y.n && y.key0 + j * kKeys + mine < y.len; };
    auto look_up = [&](const Piece& y, int j, int mine, int boxes) {
        return has_box(y, j, mine, boxes) ? p.table[static_cast<int64_t>(y.row) * p.max_pages + p.by_page(y.key0 + j * kKeys + mine)] : -1;
    };
    auto page_at = [&](int found) { return found < 0 || found >= p.c.num_pages ? max(p.c.num_pages, 1) : found; };
    auto in_page = [&](const Piece& y, int j, int mine) {
        const int key = y.key0 + j * kKeys + mine;
        return key - p.by_page(key) * p.c.page_size;
    };
    auto up_to = [&](int keys) { return (keys + p.box - 1) / p.box * p.box; };

    if (warp < kSoftWarps) {
        // ------------------------------------------------------------ softmax
        const int r = (warp & 1) * 32 + lane, side = warp >> 1 & 1, part = warp >> 2;  // row; half of the lanes; of its columns
        const int key_at = side * 64 + part * 32, mine = side * 2 + part;              // its keys of a step
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + kColS + part * 32, to_ = tmem + lanes + kColO + part * half * 64;
        Scratch* const scratch = reinterpret_cast<Scratch*>(raw + kSmemP);
        int turn = 0;  // pieces so far modulo 3
        int tails = 0;  // steps so far that ended inside
        while (true) {
            const bool more = next_piece();
            if (named_bar_or(1, kSoft, !more)) break;
            const float* const f_at = sh->f[turn] + r;
            turn = turn == 2 ? 0 : turn + 1;
            // The row's bound: its factor times `from`, and m (weights are 2^(factor (score - from) - m)); sum of its weights
            // over this thread's keys.
            float from = 0.f, m = 0.f, l = 0.f;
            uint64_t ff = 0;
            for (int j = 0; j < x.n; ++j, ++step) {
                const int left = x.len - x.key0 - j * kKeys;  // keys from this step on
                const int z = step % kScales;
                ok = __all_sync(~0u, ok && wait(&sh->scale_full[z], step / kScales));
                ok = __all_sync(~0u, ok && wait(&sh->s_full[step % kStages], step / kStages));
                tc_fence_after();
                if (j == 0) ff = pk2(*f_at, *f_at);
                const uint32_t s_at = ts + step % kStages * 64;
                const float* const up = sh->up[z] + key_at;
                // The weights, and what the tensor core takes of them times their key's scale; where one passes kMostP, the
                // bound moves and the scores are read again.
                uint32_t four[8], five[8];
                uint64_t sum = 0;
                bool set = j > 0, moved = false, failed = false;
                while (true) {
                    float w[32];
                    tmem_ld32(s_at, w);
                    if (set) {
                        if (left < kKeys) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) w[i] = key_at + i < left ? w[i] : -INFINITY;
                        }
                        const uint32_t turns = turn_of((x.key0 + j * kKeys + key_at) >> 5) * 0x00010001u;
                        const uint64_t mm = pk2(-m, -m), ss = pk2(-from, -from);
                        uint32_t big = 0;
                        sum = 0;
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            uint64_t u[2];
                            uint32_t c4[2], c5[2];
                            ld_shared_2x2(up + i, u[0], u[1]);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float a, b;
                                uint32_t pp;
                                upk2(fma2(fma2(pk2(w[i + 2 * h], w[i + 2 * h + 1]), u[h], ss), ff, mm), a, b);
                                const uint64_t e = pk2(ex2(a), ex2(b));
                                sum = add2(sum, e);
                                upk2(mul2(e, u[h]), a, b);
                                split_weights(a, b, turns ^ turns_at(i + 2 * h), pp, c4[h], c5[h]);
                                asm("max.f16x2 %0, %0, %1;" : "+r"(big) : "r"(pp));
                            }
                            four[i / 4] = c4[0] | c4[1] << 16;
                            five[i / 4] = __byte_perm(c5[0], c5[1], 0x7531);
                        }
                        uint32_t over;
                        asm("set.gt.u32.f16x2 %0, %1, %2;" : "=r"(over) : "r"(big), "r"(0x6aba6abau));  // kMostP
                        if (!named_bar_or(1, kSoft, (over && !moved) || !ok)) break;
                        ok = __all_sync(~0u, ok && wait(&sh->pv_done[(step - 1) & 1], (step - 1) >> 1));  // O is at rest
                        tc_fence_after();
                        tmem_ld32(s_at, w);
                    }
                    // the row's largest weight (times its scale); of all keys of a first step their sum and squares too
                    float top = -INFINITY;
                    const bool last = x.n - j == 1;
                    {
                        uint64_t all = 0, squares = 0;
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const uint64_t u = *reinterpret_cast<const uint64_t*>(up + i);
                            float a, b;
                            upk2(u, a, b);
                            // the exponents of the scales, as FP32 by way of 2^23 + their bits
                            const uint64_t k = add2(pk2(__uint_as_float(__float_as_uint(a) >> 23 | 0x4b000000u), __uint_as_float(__float_as_uint(b) >> 23 | 0x4b000000u)),
                                                    pk2(-8388735.f, -8388735.f));
                            const uint64_t t = add2(fma2(fma2(pk2(w[i], w[i + 1]), u, pk2(-from, -from)), ff, k), pk2(-m, -m));
                            all = add2(all, t);
                            squares = fma2(t, t, squares);
                            upk2(t, a, b);
                            if (key_at + i < left) top = fmaxf(top, a);   // (NaN is left out)
                            if (key_at + i + 1 < left) top = fmaxf(top, b);
                        }
                        float a, b, c, d;
                        upk2(all, a, b);
                        upk2(squares, c, d);
                        scratch->top[mine][r] = top;
                        scratch->all[mine][r] = a + b;
                        scratch->squares[mine][r] = c + d;
                    }
                    if (lane == 0) scratch->failed[warp] = !ok;
                    named_bar_sync(1, kSoft);
                    float all = 0.f, squares = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        top = fmaxf(top, scratch->top[i][r]);
                        all += scratch->all[i][r];
                        squares += scratch->squares[i][r];
                    }
                    // (A failed wait stays failed: all the warps learn of it here and leave together.)
                    const uint4 fail0 = *reinterpret_cast<const uint4*>(scratch->failed), fail1 = *reinterpret_cast<const uint4*>(scratch->failed + 4);
                    failed = (fail0.x | fail0.y | fail0.z | fail0.w | fail1.x | fail1.y | fail1.z | fail1.w) != 0;
                    const float place = last ? kTopAlone : set ? fminf(first_top(top, all, squares), kTopLater) : first_top(top, all, squares);
                    const bool moves = set ? top > place : top > -INFINITY;   // (up, after the first; not a row that has NaN alone)
                    const float by_log = moves ? top - place : 0.f;
                    m += by_log;
                    // Bounds that FP32 holds to a fraction of a binade only, or not at all: the score of the largest weight
                    // becomes part of them, whose differences to others it does hold.
                    const bool far = named_bar_or(1, kSoft, fabsf(m) > kFar);
                    if (failed) break;
                    if (far) {
                        float f, f2;
                        upk2(ff, f, f2);
                        const float2 bound = far_bound(s_at, up, key_at, left, scratch, r, mine, f, from);
                        if (moves) from = bound.x, m = bound.y - place;
                    }
                    if (set && __any_sync(~0u, moves)) {
                        const float by = ex2(-by_log);
                        l *= by;
#pragma unroll 1
                        for (int d = 0; d < half * 64; d += 16) {
                            float o[16];
                            tmem_ld16(to_ + d, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] *= by;
                            tmem_st16(to_ + d, o);
                        }
                    }
                    set = moved = true;
                }
                if (failed) {
                    ok = false;
                    break;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh->scale_free[z]));
                float s0, s1;
                upk2(sum, s0, s1);
                l += s0 + s1;
                // P of the step before has been read
                if (step > 0) ok = __all_sync(~0u, ok && wait(&sh->pv_done[(step - 1) & 1], (step - 1) >> 1));
                if (!ok) continue;
                const uint32_t row = sm_p + r * 128;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t at = ((key_at / 16 + i) ^ (r & 7)) << 4;
                    st_shared_v4(row + at, four[4 * i], four[4 * i + 1], four[4 * i + 2], four[4 * i + 3]);
                    st_shared_v4(row + kPTerm + at, five[4 * i], five[4 * i + 1], five[4 * i + 2], five[4 * i + 3]);
                }
                if (left < kKeys) {
                    // rows behind the end may hold anything: as values they have to be zero
                    ok = __all_sync(~0u, ok && wait(&sh->v_seen, tails));
                    if (!ok) continue;
                    mbar_acquire_cluster(smem_u32(&sh->v_seen), tails & 1);
                    ++tails;
                    const int rows = (left + 31) / 32 * 32 - left;
                    for (int i = threadIdx.x; i < rows * half * 8; i += kSoft)
                        {
                        const int row_v = left + i % (rows * 8) / 8;
                        st_shared_v4(sm_v + (step & 1) * kValueBytes + (row_v >> 6) * kValueChunk + i / (rows * 8) * 8192 + (row_v & 63) * 128 + (i & 7) * 16, 0, 0, 0, 0);
                    }
                }
                fence_proxy_async_shared();
                tc_fence_before();
                arrive_even(&sh->p_full);
            }
            // the sum over the keys, and the results
            ok = __all_sync(~0u, ok && wait(&sh->pv_done[(step - 1) & 1], (step - 1) >> 1));
            if (ok) scratch->sum[mine][r] = l;
            if (named_bar_or(1, kSoft, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            l = scratch->sum[0][r] + scratch->sum[1][r] + scratch->sum[2][r] + scratch->sum[3][r];
            named_bar_sync(1, kSoft);  // (the results pass through the same place)
            const int head0 = x.tile * kRows, nh = min(kRows, p.H - head0);
            const int64_t part_row = ((static_cast<int64_t>(unit) * 2 + x.place) * 2 + rank) * kRows;
            const int64_t out_row = static_cast<int64_t>(x.b) * p.H + head0;
            if (mine == 0 && r < nh) {
                float f, f2;
                upk2(ff, f, f2);  // (its place may have the factors of a later piece by now)
                const float lg = log2f(l) + fmaf(from, f, m);
                if (x.place >= 0) p.part_lse[part_row + r] = lg;
                else if (p.lse) p.lse[out_row + r] = lg * kLn2;
            }
            // A warp's rows pass through shared memory, 64 bytes of each at a time, so that it stores whole sectors.
            const float inv = 1.f / l;
            const uint32_t stage = sm_p + warp * 2048;
            const int row32 = (warp & 1) * 32;
            const int col0 = side * half * 128 + part * half * 64;
            const int piece = lane & 3, rows = nh - row32 - (lane >> 2);
            const int64_t first_row = (x.place >= 0 ? part_row : out_row) + row32 + (lane >> 2);
            uint8_t* to_row = (x.place >= 0 ? reinterpret_cast<uint8_t*>(p.part_o + first_row * p.Lkv + col0)
                                            : reinterpret_cast<uint8_t*>(p.out + first_row * p.Lkv + col0)) + piece * 16;
            const int64_t rows8 = static_cast<int64_t>(p.Lkv) * (x.place >= 0 ? 32 : 16);
#pragma unroll 1
            for (int d = 0; d < half * 64; d += 32) {
                if (col0 + d >= p.Lkv || row32 >= nh) break;
                float o[32];
                __syncwarp();  // (tensor memory is read by converged warps)
                tmem_ld32(to_ + d, o);
                // 32 columns: 64 bytes of finished rows, twice 64 of partial ones
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (x.place < 0 && t > 0) break;
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t at = stage + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4);
                        if (x.place >= 0) {
                            const float* v = o + t * 16 + i * 4;
                            st_shared_v4(at, __float_as_uint(v[0] * inv), __float_as_uint(v[1] * inv), __float_as_uint(v[2] * inv), __float_as_uint(v[3] * inv));
                        } else {
                            const float* v = o + i * 8;
                            st_shared_v4(at, pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv),
                                         pack_bf16x2(v[4] * inv, v[5] * inv), pack_bf16x2(v[6] * inv, v[7] * inv));
                        }
                    }
                    __syncwarp();
                    const int col = col0 + d + (x.place >= 0 ? t * 16 + piece * 4 : piece * 8);
                    uint8_t* at = to_row + (x.place >= 0 ? d * 4 + t * 64 : d * 2);
#pragma unroll
                    for (int i = 0; i < 4; ++i, at += rows8) {
                        const int rr = i * 8 + (lane >> 2);
                        uint4 q;
                        ld_shared_v4(stage + rr * 64 + ((piece ^ (rr >> 1 & 3)) << 4), q.x, q.y, q.z, q.w);
                        if (i * 8 < rows && col < p.Lkv) *reinterpret_cast<uint4*>(at) = q;
                    }
                }
            }
            tc_fence_before();
            arrive_even(&sh->o_free);
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------ MMA (the even CTA's, for both)
        if (rank == 0 && elect_one()) {
            const uint32_t id_s = idesc_e4m3(kKeys, false);
            const uint32_t id_4 = (idesc_e4m3(256, false) | 1u << 16), id_5 = id_4 | 1u << 7;   // B MN-major; A E4M3, E5M2
            const uint64_t dq = desc_128(sm_q), dq_rest = desc_64(sm_q + 32768), dk = desc_128(sm_k), dk_rest = desc_64(sm_k + 32768);
            const uint64_t dp = desc_128(sm_p), dv = desc_128(sm_v);
            auto look = [&](uint64_t* bar, uint32_t parity) {
                ok = ok && wait(bar, parity);
                tc_fence_after();
                return ok;
            };
            auto commit = [&](uint64_t* bar) { mma_commit_pair(smem_u32(bar), 0x3); };
            int opened = 0;  // pieces whose first values have been multiplied
            auto scores = [&]() {
                const int e = step & 1;
                if (!look(&sh->k_full[e], step >> 1)) return;
                const uint32_t d = tmem + kColS + step % kStages * 64;
                const uint64_t b = dk + e * (kKeyBytes >> 4), b_rest = dk_rest + e * (kKeyBytes >> 4);
                // (the most columns there are, and the usual ones, without a loop: long contexts 134 us, by the loop 145)
                if (C == 576) {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            mma_pair8(d, dq + t * (kQTerm >> 4) + (k >> 2) * 512 + 2 * (k & 3), b + (k >> 2) * 512 + 2 * (k & 3), id_s, t > 0 || k > 0);
#pragma unroll
                        for (int k = 0; k < 2; ++k) mma_pair8(d, dq_rest + t * (kQTerm >> 4) + 2 * k, b_rest + 2 * k, id_s, 1);
                    }
                } else {
#pragma unroll 1
                    for (int t = 0; t < 2; ++t) {
#pragma unroll 1
                        for (int k = 0; k < (min(C, 512) + 31) / 32; ++k)
                            mma_pair8(d, dq + t * (kQTerm >> 4) + (k >> 2) * 512 + 2 * (k & 3), b + (k >> 2) * 512 + 2 * (k & 3), id_s, t > 0 || k > 0);
#pragma unroll 1
                        for (int k = 0; k < (rest + 31) / 32; ++k) mma_pair8(d, dq_rest + t * (kQTerm >> 4) + 2 * k, b_rest + 2 * k, id_s, 1);
                    }
                }
                commit(&sh->s_full[step % kStages]);
            };
            auto values = [&](int u, bool first, int keys) {
                const int e = u & 1;
                if (!look(&sh->v_full[e], u >> 1)) return;
                if (keys < kKeys)  // both CTAs clear the rows behind the end first
                    copies_seen(smem_u32(&sh->v_full[e]), u >> 1 & 1, smem_u32(&sh->v_seen));
                if (!look(&sh->p_full, u)) return;
                // (a piece's first values overwrite O, from which the results of the piece before have been read)
                if (first && opened++ > 0 && !look(&sh->o_free, opened - 2)) return;
                const uint64_t b = dv + e * (kValueBytes >> 4);
#pragma unroll
                for (int k = 0; k < kKeys / 32; ++k) {
                    if (k * 32 >= keys) break;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (i >= half) break;
                        const uint64_t bi = b + (k >> 1) * (kValueChunk >> 4) + i * 512 + (k & 1) * 256;
                        mma_pair8(tmem + kColO + i * 128, dp + 2 * k, bi, id_4, !first || k > 0);
                        mma_pair8(tmem + kColO + i * 128, dp + (kPTerm >> 4) + 2 * k, bi, id_5, 1);
                    }
                }
                commit(&sh->pv_done[e]);
            };
            // Per round: the scores of a step, then P V of the step before, whose softmax runs meanwhile.
            bool due = false, first = false;
            int keys_due = 0;  // of the step before
            while (look(&sh->piece_full[pieces % kAhead], pieces / kAhead)) {
                const int n = sh->piece[pieces % kAhead].n, keys = sh->piece[pieces % kAhead].len - sh->piece[pieces % kAhead].key0;
                mbar_arrive(smem_u32(&sh->piece_free[pieces % kAhead]));
                if (n == 0) break;
                if (due && !mbar_test(smem_u32(&sh->q_full), pieces & 1)) {  // the next query is not there yet
                    values(step - 1, first, keys_due);
                    due = false;
                }
                if (!look(&sh->q_full, pieces)) break;
                for (int t = 0; t < n && ok; ++t) {
                    scores();
                    if (!ok) break;
                    if (t + 1 == n) commit(&sh->q_free);
                    ++step;
                    if (due) values(step - 2, first, keys_due);
                    first = t == 0;
                    due = true;
                    keys_due = min(kKeys, keys - t * kKeys);
                }
                if (!ok) break;
                ++pieces;
            }
            if (ok && due) values(step - 1, first, keys_due);
            if (!ok) {  // no MMA may still run when the CTAs leave
                commit(&sh->drain);
                mbar_wait(smem_u32(&sh->drain), 0, kTimeoutNs, nullptr);
            }
        }
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------- pieces, keys by TMA
        // Each CTA brings its halves of the keys and (the next warp) of the values, which complete on the even CTA's
        // barriers; the even CTA tells them how many bytes both bring.  A lane has a box of the cache's rows.  (A copy
        // takes its issuer as long as its bytes: with keys and values in one warp a step took 3.0k cycles instead of 2.5k.)
        const int boxes = 64 / p.box, mine = rank * 64 + lane * p.box;  // of this CTA's keys; the lane's first key of a step
        const bool whole = p.box == 64 && C >= 512;
        while (ok) {
            x = walk.next(p);
            ok = put_piece(sh, wait, pieces++, x);
            if (!ok || x.n == 0) break;
            int found = look_up(x, 0, mine, boxes);
            for (int j = 0; j < x.n; ++j, ++step) {
                const int page = page_at(found), in = in_page(x, j, mine);
                const bool has = has_box(x, j, mine, boxes);
                found = look_up(x, j + 1, mine, boxes);
                const int keys = min(kKeys, x.len - x.key0 - j * kKeys), e = step & 1;
                if (step >= 2) ok = __all_sync(~0u, ok && wait(&sh->s_full[(step - 2) % kStages], (step - 2) / kStages));
                if (!ok) break;
                const uint32_t dst = sm_k + e * kKeyBytes, bar = map_shared_rank(smem_u32(&sh->k_full[e]), 0);
                const int rows = up_to(min(keys, 64)) + (keys > 64 ? up_to(keys - 64) : 0);
                if (rank == 0 && lane == 0) mbar_arrive_expect_tx(smem_u32(&sh->k_full[e]), rows * (chunks * 128 + (rest ? 64 : 0)));
                if (has) {
                    if (whole) tma_load_4d_pair(dst, &tm_k, bar, 0, in, page, 0);
                    else
                        for (int c = 0; c < chunks; ++c) tma_load_3d_pair(dst + c * 8192 + lane * p.box * 128, &tm_rows, bar, c * 128, in, page);
                    if (rest) tma_load_3d_pair(dst + 32768 + lane * p.box * 64, &tm_rest, bar, 512, in, page);
                }
                __syncwarp();
            }
        }
        if (!ok && rank == 0)  // no copy of either CTA may still be landing when they leave
            for (int u = max(step - 1, 0); u <= step; ++u) mbar_wait(smem_u32(&sh->k_full[u & 1]), (u >> 1) & 1, kTimeoutNs, nullptr);
    } else if (warp == kLoadWarp + 1) {
        // ------------------------------------------------------ values by TMA
        const int boxes = kKeys / p.box, mine = lane * p.box;
        const bool whole = p.box == 64 && C >= 512 && p.Lkv > 384;
        while (next_piece()) {
            int found = look_up(x, 0, mine, boxes);
            for (int j = 0; j < x.n; ++j, ++step) {
                const int page = page_at(found), in = in_page(x, j, mine);
                const bool has = has_box(x, j, mine, boxes);
                found = look_up(x, j + 1, mine, boxes);
                const int keys = min(kKeys, x.len - x.key0 - j * kKeys), e = step & 1;
                if (step >= 2) ok = __all_sync(~0u, ok && wait(&sh->pv_done[e], (step - 2) >> 1));
                if (!ok) break;
                const uint32_t bar = map_shared_rank(smem_u32(&sh->v_full[e]), 0);
                const uint32_t dst = sm_v + e * kValueBytes + (mine >> 6) * kValueChunk + (mine & 63) * 128;
                if (rank == 0 && lane == 0) mbar_arrive_expect_tx(smem_u32(&sh->v_full[e]), 2 * half * up_to(keys) * 128);
                if (has) {
                    if (whole) tma_load_4d_pair(dst, &tm_v, bar, 0, in, page, rank * 2);
                    else
                        for (int i = 0; i < half; ++i) tma_load_3d_pair(dst + i * 8192, &tm_rows, bar, (rank * half + i) * 128, in, page);
                }
                __syncwarp();
            }
            if (!ok) break;
        }
        if (!ok && rank == 0)
            for (int u = max(step - 2, 0); u < step; ++u) mbar_wait(smem_u32(&sh->v_full[u & 1]), (u >> 1) & 1, kTimeoutNs, nullptr);
    } else if (warp == kScaleWarp) {
        // ------------------------------------------------- queries and scales
        pdl_wait();  // the kernel that split the queries
        int turn = 0;
        auto begin = [&]() {
            if (pieces > 1) ok = __all_sync(~0u, ok && wait(&sh->q_free, pieces - 2));
            if (ok && lane == 0) {
                const int64_t tile = static_cast<int64_t>(x.b) * p.tiles + x.tile;
                mbar_arrive_expect_tx(smem_u32(&sh->q_here), kPairQBytes + sizeof(sh->f[0]));
                bulk_load(sm_q, p.terms + tile * kPairQBytes, kPairQBytes, smem_u32(&sh->q_here));
                bulk_load(smem_u32(sh->f[turn]), p.factors + tile * kRows, sizeof(sh->f[0]), smem_u32(&sh->q_here));
            }
            turn = turn == 2 ? 0 : turn + 1;
            __syncwarp();
            return ok;
        };
        find_scales(p, x, next_piece, begin, [&](int j, uint32_t four) {
            const int z = step % kScales;
            if (step >= kScales) ok = __all_sync(~0u, ok && wait(&sh->scale_free[z], step / kScales - 1));
            if (ok) {
                *reinterpret_cast<float4*>(sh->up[z] + lane * 4) =
                    make_float4(pow2(scale_exp(four & 255)), pow2(scale_exp(four >> 8 & 255)), pow2(scale_exp(four >> 16 & 255)), pow2(scale_exp(four >> 24)));
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh->scale_full[z]));
                ++step;
            }
            if (j == 0) {
                const bool here = __all_sync(~0u, mbar_wait(smem_u32(&sh->q_here), (pieces - 1) & 1, kTimeoutNs, nullptr));
                ok = ok && here;
                if (ok) arrive_even(&sh->q_full);
            }
            return ok;
        });
        // (the tensor core's last arrival has come)
        if (ok && pieces > 1) ok = __all_sync(~0u, wait(&sh->q_free, pieces - 2));
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

}  // namespace

cudaError_t launch_attend8_pair(const CUtensorMap& rows, const CUtensorMap& rest, const CUtensorMap& k, const CUtensorMap& v, const Attend8& p,
                                cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(&mla_attend_cache8_pair_kernel, kSmem, &ready);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(p.units * 2);
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
    return cudaLaunchKernelEx(&cfg, mla_attend_cache8_pair_kernel, rows, rest, k, v, p);
}

}  // namespace mlap
