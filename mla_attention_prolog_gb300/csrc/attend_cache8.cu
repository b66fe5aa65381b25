// One decoding step over the latent cache in 8 bits: mla_prolog_attend_cache8.
//
// A cache row is code_j * 2^(x_j) (E4M3 codes, a power of two for each block of
// tokens), key and, in its first Lkv columns, value of every head.  With f the
// softmax scale times log2 e, and in log2 of the weights:
//
//   t_j = f 2^(x_j) <q, code_j>          P_j = 2^(t_j + x_j - m)
//   out = sum_j P_j code_j / l           l = sum_j 2^(-x_j) P_j
//
// so that the codes are multiplied as they lie in memory: m is a running bound
// of t_j + x_j, the weight with its block's scale.
//
// The tensor core multiplies 8-bit floats at twice the BF16 rate, so q and P go
// in as sums of such values, with FP32 sums.  q: an E4M3 value and what its
// rounding left in E4M3 (4 + 4 significant bits: exactly; elements below 2^-10 of
// a row's largest to 2^-18 of that).  P, up to 32 heads: three E5M2 values, to
// 2^-9 of itself or 2^-18 of the largest weight; of 64 heads an E4M3 and an E5M2
// value, whose smaller steps below 1 keep weights that lie far under the largest
// (a first token's, say): to 2^-7 of itself, as near on average as a rounding to
// BF16, or to 2^-15 of the largest (2^-24 where that one stands alone).  Weights
// so small that the second bound holds are rounded up or down by turns along the
// keys, so that many of them that are alike keep their sum (attend_cache8.cuh).
//
// A tile is kHeads heads of one sequence on 128 keys a step, keys along the
// lanes, so that one copy of the cache rows in shared memory serves both
// products:
//
//   S [128 keys][h | l terms of the heads] = K [128][C] (Qh | Ql)^T
//   O^T [128 value columns][terms of the heads] += V^T [128][128 keys] P,  Lkv / 128 times
//
// A thread has a key: its block's scale is a factor of its own.  The heads'
// maxima run across the lanes, so m only bounds them: it moves (and O with it)
// when a weight would pass 2^11.75.
//
// The work is cut into equal runs of key steps (a tile costs its steps and some
// more for its start and end), one per unit: a CTA, or for more than 64 heads a
// pair (attend_cache8_pair.cu).  Partial results go to the workspace in FP32,
// and another kernel joins them in the order of the cut.  Where it takes no
// longer, whole tiles are dealt to the units instead.
//
// What bounds it.  Many keys of 16 and 32 heads: the reading of the cache, 5.6 and
// 5.5 TB/s (83 and 81% of a copy's rate; 152 sequences of 8192, C = 576: 129 and
// 132 us), of 64 heads shared memory and the ring, that holds two steps (4.4 TB/s;
// 167 us).  A step from L2 takes 1.4, 1.7 and 2.2 us for 16, 32 and 64 heads; the
// products alone would take 0.7, 0.9 and 1.3.  Few keys: the launches and a cold
// start (each instruction comes from L2 the first time): 9.5 us for 100 keys of one
// sequence.  V2-Lite, 64 sequences of 1 to 4096: 30 us, of which the join takes 5.
#include <cstdint>

#include "attend_cache8.cuh"

namespace mlap {
namespace {

constexpr int kChunkBytes = kKeys * 128;        // 128 columns of a step's rows
constexpr int kRestBytes = kKeys * 64;          // columns 512 .. 575
constexpr int kMaxSlots = 11, kMaxRests = 3;
constexpr int kMaxBatch = 1 << 17;

// P of 64 heads is an E4M3 and an E5M2 term, of fewer three E5M2 terms: those go side by side into one product, and a
// product of less than 64 columns takes as long as one of 64 does.
__host__ __device__ constexpr bool three_terms(int heads) { return heads < 64; }
__host__ __device__ constexpr int p_row(int heads) { return heads == 32 ? 128 : 64; }  // bytes of a key's weights
// Shared memory: a ring of chunks and one of the columns behind 512, P, both terms of Q.  With 64 heads P's first term takes
// the place of a step's columns behind 512, whose scores are made by then; with fewer those make room at once for others.
__host__ __device__ constexpr int slots_of(int heads) { return heads == 64 ? 8 : heads == 32 ? 9 : 11; }
__host__ __device__ constexpr int rests_of(int heads) { return heads == 32 ? 3 : 2; }
__host__ __device__ constexpr int q_bytes(int heads) { return 2 * heads * (4 * 128 + 64); }
__host__ __device__ constexpr int p_at(int heads) { return slots_of(heads) * kChunkBytes + rests_of(heads) * kRestBytes; }  // (64: second term)
__host__ __device__ constexpr int q_at(int heads) { return p_at(heads) + kKeys * p_row(heads); }
__host__ __device__ constexpr int misc_at(int heads) { return q_at(heads) + q_bytes(heads); }
__host__ __device__ constexpr int smem_bytes(int heads) { return misc_at(heads) + kMiscBytes; }
static_assert(q_bytes(64) == kPairQBytes, "");
static_assert(smem_bytes(64) <= 232448 && smem_bytes(32) <= 232448 && smem_bytes(16) <= 232448, "227 KB");

struct Shared {
    uint64_t kv_full[kMaxSlots], kv_free[kMaxSlots], rest_full[kMaxRests], rest_free[kMaxRests];
    uint64_t s_full[2], pv_done[2], p_full, q_full, q_free, o_free, piece_full[kAhead], piece_free[kAhead];
    uint64_t scale_full[kAhead], scale_free[kAhead], drain;
    uint32_t tmem;
    int abort_flag;
    Piece piece[kAhead];
    alignas(16) float f[3][64];  // factors of the heads' scores: of a piece, while its weights are made, and two behind it
    alignas(16) float m[64];     // minus the bound of a head's weights
    alignas(16) float by[64];    // factor of what that moves; behind the last step 1 / sum of the head's weights
    alignas(16) uint8_t scale[kAhead][kKeys];  // exponent bytes of a step's keys
};
static_assert(sizeof(Shared) <= kMiscBytes, "");
// What the softmax warps tell each other, in the place of P (its second term) while no product reads that.
struct Scratch {
    float of_warp[4][64], all[4][64], squares[4][64];  // of a warp's keys: each head's largest weight (or their sum); sums
    alignas(16) uint32_t failed[kSoftWarps];
};
static_assert(sizeof(Scratch) <= kRestBytes, "");

// Where a row's eight columns from `col` on lie in shared memory, of query rows in chunks of kRows (both terms', or one's).
template <int kRows>
__device__ __forceinline__ uint32_t query_at(int row, int col) {
    return col < 512 ? (col >> 7) * (kRows * 128) + row * 128 + ((col & 127) ^ ((row & 7) << 4))
                     : 4 * (kRows * 128) + row * 64 + ((col - 512) ^ ((row >> 1 & 3) << 4));
}

// kSplit: the softmax warps split the query rows themselves, with the same results (else a kernel before this one has).
template <int kHeads, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    mla_attend_cache8_kernel(const __grid_constant__ CUtensorMap tm_rows, const __grid_constant__ CUtensorMap tm_rest,
                             const __grid_constant__ Attend8 p) {
    constexpr int kQChunk = 2 * kHeads * 128;                  // 128 columns of Q's two terms
    constexpr uint32_t kColS = 0, kStageS = 2 * kHeads;        // TMEM: S of two steps,
    constexpr uint32_t kColO = 2 * kStageS;                    //   O^T by 128 value columns, term by term
    constexpr bool kThree = three_terms(kHeads);
    constexpr int kTerms = kThree ? 3 : 1, kWidth = kTerms * kHeads;
    constexpr uint32_t kTmem = kHeads == 16 ? 256 : 512;
    constexpr int kSlots = slots_of(kHeads), kRests = rests_of(kHeads);
    constexpr int kMine = kHeads / 2;                          // heads of a softmax thread
    extern __shared__ __align__(1024) uint8_t raw[];
    const uint32_t sm_kv = smem_u32(raw), sm_rest = sm_kv + kSlots * kChunkBytes, sm_p = sm_kv + p_at(kHeads), sm_q = sm_kv + q_at(kHeads);
    Shared* const sh = reinterpret_cast<Shared*>(raw + misc_at(kHeads));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x / p.group, rank = blockIdx.x % p.group;
    // 128-column chunks of a row, all of its columns but those behind 512; the chunks that hold values
    const int C = p.c.C, chunks = C > 512 ? 4 : (C + 127) / 128, rest = C > 512 ? C - 512 : 0;
    const int blocks = (p.Lkv + 127) / 128;

    Walk walk;
    uint32_t* const scratch = reinterpret_cast<uint32_t*>(raw);  // (of the ring, that is empty yet)
    if constexpr (!kSplit) {  // (else there are no more tiles than CTAs)
        if (p.rounds > 1) deal_tiles(p, unit, scratch);
    }
    if (warp == kLoadWarp) {
        if (kSplit) pdl_wait();
        walk.start(p, unit, rank, scratch);  // (the lengths are on their way first)
    } else if (warp == kScaleWarp && lane == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(smem_u32(&sh->kv_full[i]), 1), mbar_init(smem_u32(&sh->kv_free[i]), 1);
        for (int i = 0; i < kRests; ++i) mbar_init(smem_u32(&sh->rest_full[i]), 1), mbar_init(smem_u32(&sh->rest_free[i]), 1);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sh->s_full[i]), 1), mbar_init(smem_u32(&sh->pv_done[i]), 1);
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(smem_u32(&sh->piece_full[i]), 1);
            mbar_init(smem_u32(&sh->piece_free[i]), kSoftWarps + 3);  // (the other copying warp, scales, the MMA thread)
            mbar_init(smem_u32(&sh->scale_full[i]), 1);
            mbar_init(smem_u32(&sh->scale_free[i]), kSoftWarps);
        }
        mbar_init(smem_u32(&sh->p_full), kSoftWarps);
        mbar_init(smem_u32(&sh->q_full), kSplit ? kSoftWarps : 1);
        mbar_init(smem_u32(&sh->q_free), 1);
        mbar_init(smem_u32(&sh->o_free), kSoftWarps);
        mbar_init(smem_u32(&sh->drain), 1);
        sh->abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tm_rows);
        prefetch_tensormap(&tm_rest);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(&sh->tmem), kTmem);
        tmem_relinquish();
    }
    if (threadIdx.x < 64) sh->m[threadIdx.x] = 0.f;
    tc_fence_before();
    // (The next kernel may come before this CTA has its TMEM: none that takes some fits beside its shared memory.)
    pdl_launch_dependents();
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

    if (warp < kSoftWarps) {
        // ------------------------------------------------------------ softmax
        // A thread has a key (its TMEM lane) and half of the heads.
        const int tid = threadIdx.x & 127, h0 = threadIdx.x / 128 * kMine;
        const uint32_t lanes = static_cast<uint32_t>(tid / 32 * 32) << 16;
        const uint32_t ts = tmem + lanes + kColS + h0, to_ = tmem + lanes + kColO + h0;
        // eight heads of O in a block of 128 columns, and the same times `by`
        auto get_o = [&](int d, int h, float (&o)[8]) {
            tmem_ld8(to_ + d * kWidth + h, o);
            if constexpr (kThree) {
                float y[8], z[8];
                tmem_ld8x2(to_ + d * kWidth + kHeads + h, to_ + d * kWidth + 2 * kHeads + h, y, z);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] += y[i] + z[i];
            }
        };
        Scratch* const scratch = reinterpret_cast<Scratch*>(raw + p_at(kHeads));
        int turn = 0;  // pieces so far modulo 3
        if (kSplit) pdl_wait();
        while (true) {
            const bool more = next_piece();
            if (named_bar_or(1, kSoft, !more)) break;
            float* const f = sh->f[turn];
            turn = turn == 2 ? 0 : turn + 1;
            if constexpr (kSplit) {
                const int nh = min(kHeads, p.H - x.tile * kHeads), padded = C > 512 ? 576 : chunks * 128;
                const uint16_t* const rows = p.q + (static_cast<int64_t>(x.b) * p.H + x.tile * kHeads) * C;
                if (pieces > 1) ok = __all_sync(~0u, ok && wait(&sh->q_free, pieces - 2));
                uint4 v[3], next[3];
                auto load = [&](int r, uint4 (&to)[3]) {
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        to[k] = make_uint4(0, 0, 0, 0);
                        if (r < nh && (k * 32 + lane) * 8 < C) to[k] = reinterpret_cast<const uint4*>(rows + r * C)[k * 32 + lane];
                    }
                };
                load(warp, v);
#pragma unroll 1
                for (int r = warp; r < kHeads && ok; r += kSoftWarps) {
                    load(r + kSoftWarps, next);
                    const float factor = split_row(p, v, [&](int k, uint2 hi, uint2 lo) {
                        const int col = (k * 32 + lane) * 8;
                        if (col >= padded) return;
                        st_shared_v2(sm_q + query_at<2 * kHeads>(r, col), hi.x, hi.y);
                        st_shared_v2(sm_q + query_at<2 * kHeads>(r + kHeads, col), lo.x, lo.y);
                    });
                    if (lane == 0) f[r] = factor;
#pragma unroll
                    for (int k = 0; k < 3; ++k) v[k] = next[k];
                }
                fence_proxy_async_shared();
                named_bar_sync(1, kSoft);
                if (ok && lane == 0) mbar_arrive(smem_u32(&sh->q_full));
            }
            uint64_t l[kMine / 2];
#pragma unroll
            for (int i = 0; i < kMine / 2; ++i) l[i] = 0;
            for (int j = 0; j < x.n; ++j, ++step) {
                const int left = x.len - x.key0 - j * kKeys;  // keys from this step on
                const bool mine = tid < left;
                ok = __all_sync(~0u, ok && wait(&sh->scale_full[step % kAhead], step / kAhead));
                const int k = scale_exp(sh->scale[step % kAhead][tid]);
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(smem_u32(&sh->scale_free[step % kAhead]));
                const uint64_t up = pk2(pow2(k), pow2(k)), kf = pk2(static_cast<float>(k), static_cast<float>(k));
                const uint64_t back = pk2(pow2(-k), pow2(-k));
                ok = __all_sync(~0u, ok && wait(&sh->s_full[step & 1], step >> 1));
                tc_fence_after();
                const uint32_t s_at = ts + (step & 1) * kStageS;
                // log2 of the weights, times the block's scale, over the bound; where one passes that, the bound moves and
                // the scores are read again.  (What runs once in a while is kept short: it comes from L2 each time.)
                float t[kMine];
                bool set = j > 0, moved = false, failed = false;
                while (true) {
                    if (set) {
                        float big = -INFINITY;
                        constexpr int kWide = kMine < 16 ? kMine : 16;
#pragma unroll
                        for (int h = 0; h < kMine; h += kWide) {
                            uint32_t a[kWide], b[kWide];
                            if constexpr (kWide == 16) {
                                tmem_ld16x2(s_at + h, s_at + kHeads + h, a, b);
                            } else {
                                float fa[8], fb[8];
                                tmem_ld8x2(s_at + h, s_at + kHeads + h, fa, fb);
#pragma unroll
                                for (int i = 0; i < 8; ++i) a[i] = __float_as_uint(fa[i]), b[i] = __float_as_uint(fb[i]);
                            }
#pragma unroll
                            for (int i = 0; i < kWide; i += 4) {
                                uint64_t f0, f1, m0, m1;
                                ld_shared_2x2(f + h0 + h + i, f0, f1);
                                ld_shared_2x2(sh->m + h0 + h + i, m0, m1);
                                auto two = [&](int e, uint64_t ff, uint64_t mm) {
                                    const uint64_t s = add2(pk2(__uint_as_float(a[e]), __uint_as_float(a[e + 1])),
                                                            pk2(__uint_as_float(b[e]), __uint_as_float(b[e + 1])));
                                    upk2(add2(fma2(mul2(s, up), ff, kf), mm), t[h + e], t[h + e + 1]);
                                    big = fmaxf(big, fmaxf(t[h + e], t[h + e + 1]));
                                };
                                two(i, f0, m0);
                                two(i + 2, f1, m1);
                            }
                        }
                        if (!mine) {
                            big = -INFINITY;
#pragma unroll
                            for (int h = 0; h < kMine; ++h) t[h] = -INFINITY;
                        }
                        if (!named_bar_or(1, kSoft, (big > kMost && !moved) || !ok)) break;
                        ok = __all_sync(~0u, ok && wait(&sh->pv_done[(step - 1) & 1], (step - 1) >> 1));  // O is at rest
                        tc_fence_after();
                    }
                    // each head's largest weight; of all keys of a first step their sum and squares too
                    const bool last = x.n - j == 1;
#pragma unroll 1
                    for (int h = 0; h < kMine; h += 8) {
                        float a[8], b[8];
                        __syncwarp();  // (tensor memory is read by converged warps)
                        tmem_ld8x2(s_at + h, s_at + kHeads + h, a, b);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            a[i] = fmaf((a[i] + b[i]) * pow2(k), f[h0 + h + i], static_cast<float>(k)) + sh->m[h0 + h + i];
                            const int most = __reduce_max_sync(~0u, ordered(mine && a[i] == a[i] ? a[i] : -INFINITY));
                            if (lane == i) scratch->of_warp[warp & 3][h0 + h + i] = unordered(most);
                        }
                        if (!last) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) b[i] = a[i] * a[i];
                            sum_across(a, lane);
                            sum_across(b, lane);
                            if (lane % 4 == 0) scratch->all[warp & 3][h0 + h + lane / 4] = a[0], scratch->squares[warp & 3][h0 + h + lane / 4] = b[0];
                        }
                    }
                    if (lane == 0) scratch->failed[warp] = !ok;
                    named_bar_sync(1, kSoft);
                    if (tid < kMine) {
                        const int h = h0 + tid;
                        float top = -INFINITY, all = 0.f, squares = 0.f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            top = fmaxf(top, scratch->of_warp[i][h]);
                            all += scratch->all[i][h];
                            squares += scratch->squares[i][h];
                        }
                        // (not by a head that has NaN alone)
                        const float place = last ? kTopAlone : set ? fminf(first_top(top, all, squares), kTopLater) : first_top(top, all, squares);
                        const bool moves = set ? top > place : top > -INFINITY;  // (up, after the first)
                        // (By what it moves: of a bound beyond 2^17 FP32 does not hold each fraction of a binade, and beyond
                        // 2^27 that may be too little by five.)
                        const float was = sh->m[h];
                        float now = was - (top - place);
                        if (top + (now - was) > kMost) now = was - top;
                        sh->by[h] = moves ? ex2(now - was) : 1.f;
                        if (moves) sh->m[h] = now;
                    }
                    // (A failed wait stays failed: all the warps learn of it here and leave together.)
                    const uint4 fail0 = *reinterpret_cast<const uint4*>(scratch->failed), fail1 = *reinterpret_cast<const uint4*>(scratch->failed + 4);
                    failed = (fail0.x | fail0.y | fail0.z | fail0.w | fail1.x | fail1.y | fail1.z | fail1.w) != 0;
                    named_bar_sync(1, kSoft);
                    if (failed) break;
                    if (set) {
#pragma unroll
                        for (int h = 0; h < kMine; h += 4) {
                            uint64_t b0, b1;
                            ld_shared_2x2(sh->by + h0 + h, b0, b1);
                            l[h / 2] = mul2(l[h / 2], b0);
                            l[h / 2 + 1] = mul2(l[h / 2 + 1], b1);
                        }
#pragma unroll 1
                        for (int h = 0; h < kMine; h += 8) {
                            float by[8];
                            bool still = true;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                by[i] = sh->by[h0 + h + i];
                                still = still && by[i] == 1.f;
                            }
                            if (still) continue;
#pragma unroll 1
                            for (int d = 0; d < blocks * kTerms; ++d) {
                                float o[8];
                                tmem_ld8(to_ + d * kHeads + h, o);
#pragma unroll
                                for (int i = 0; i < 8; ++i) o[i] *= by[i];
                                tmem_st8(to_ + d * kHeads + h, o);
                            }
                        }
                    }
                    set = moved = true;
                }
                if (failed) {
                    ok = false;
                    break;
                }
                const uint32_t turns = (turn_of(x.key0 + j * kKeys + tid) ^ 0x80u) * 0x00010001u;
                uint32_t term[kThree ? 3 : 2][kMine / 4];
#pragma unroll
                for (int h = 0; h < kMine; h += 4) {
                    const float a = ex2(t[h]), b = ex2(t[h + 1]), c = ex2(t[h + 2]), d = ex2(t[h + 3]);
                    l[h / 2] = fma2(pk2(a, b), back, l[h / 2]);
                    l[h / 2 + 1] = fma2(pk2(c, d), back, l[h / 2 + 1]);
                    uint32_t x0, x1, y0, y1, z0, z1;
                    if constexpr (kThree) {
                        split_weights3(a, b, turns, x0, y0, z0);
                        split_weights3(c, d, turns, x1, y1, z1);
                        term[0][h / 4] = __byte_perm(x0, x1, 0x7531);
                        term[2][h / 4] = __byte_perm(z0, z1, 0x7531);
                    } else {
                        split_weights(a, b, turns, z0, x0, y0);
                        split_weights(c, d, turns, z1, x1, y1);
                        term[0][h / 4] = x0 | x1 << 16;
                    }
                    term[1][h / 4] = __byte_perm(y0, y1, 0x7531);
                }
                // P of the step before has been read
                if (step > 0) ok = __all_sync(~0u, ok && wait(&sh->pv_done[(step - 1) & 1], (step - 1) >> 1));
                if (!ok) continue;
                const uint32_t row = sm_p + tid * p_row(kHeads);
                if constexpr (kHeads == 16) {
#pragma unroll
                    for (int i = 0; i < 3; ++i) st_shared_v2(row + ((i ^ (tid >> 1 & 3)) << 4) + h0, term[i][0], term[i][1]);
                } else if constexpr (kHeads == 32) {
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        st_shared_v4(row + (((2 * i + h0 / 16) ^ (tid & 7)) << 4), term[i][0], term[i][1], term[i][2], term[i][3]);
                } else {
                    const uint32_t first = sm_rest + step % kRests * kRestBytes + tid * 64;
#pragma unroll
                    for (int i = 0; i < kMine / 16; ++i) {
                        const uint32_t at = ((h0 / 16 + i) ^ (tid >> 1 & 3)) << 4;
                        st_shared_v4(first + at, term[0][4 * i], term[0][4 * i + 1], term[0][4 * i + 2], term[0][4 * i + 3]);
                        st_shared_v4(row + at, term[1][4 * i], term[1][4 * i + 1], term[1][4 * i + 2], term[1][4 * i + 3]);
                    }
                }
                // rows behind the end may hold anything: as values they have to be zero
                if (left < kKeys) {
                    const int rows = (left + 31) / 32 * 32 - left;
                    for (int i = threadIdx.x; i < rows * blocks * 8; i += kSoft)
                        st_shared_v4(sm_kv + (step * chunks + i / (rows * 8)) % kSlots * kChunkBytes + (left + i % (rows * 8) / 8) * 128 + (i & 7) * 16, 0, 0, 0, 0);
                }
                fence_proxy_async_shared();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh->p_full));
            }
            // the sums over the keys, and the results
            ok = __all_sync(~0u, ok && wait(&sh->pv_done[(step - 1) & 1], (step - 1) >> 1));
            {
                float sums[kMine];
#pragma unroll
                for (int i = 0; i < kMine / 2; ++i) upk2(l[i], sums[2 * i], sums[2 * i + 1]);
                sum_across(sums, lane);
                constexpr int kLanes = 32 / kMine;
                if (ok && lane % kLanes == 0) scratch->of_warp[warp & 3][h0 + lane / kLanes] = sums[0];
            }
            if (named_bar_or(1, kSoft, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int head0 = x.tile * kHeads, nh = min(kHeads, p.H - head0);
            const int64_t part = ((static_cast<int64_t>(unit) * 2 + x.place) * p.group + rank) * kHeads;
            const int64_t row = static_cast<int64_t>(x.b) * p.H + head0;
            if (threadIdx.x < kHeads) {
                const int h = threadIdx.x;
                const float sum = scratch->of_warp[0][h] + scratch->of_warp[1][h] + scratch->of_warp[2][h] + scratch->of_warp[3][h];
                sh->by[h] = 1.f / sum;
                if (h < nh) {
                    const float z = log2f(sum) - sh->m[h];
                    if (x.place >= 0) p.part_lse[part + h] = z;
                    else if (p.lse) p.lse[row + h] = z * kLn2;
                }
                sh->m[h] = 0.f;
            }
            named_bar_sync(1, kSoft);
            // A thread has a value column of each block and its half of the heads.
            float* to_part = p.part_o + (part + h0) * p.Lkv + tid;
            uint16_t* to_out = p.out + (row + h0) * p.Lkv + tid;
            const int64_t next8 = static_cast<int64_t>(p.Lkv) * 8;
#pragma unroll 1
            for (int h = 0; h < kMine && h0 + h < nh; h += 8, to_part += next8, to_out += next8) {
                const float4 a = *reinterpret_cast<const float4*>(sh->by + h0 + h), b = *reinterpret_cast<const float4*>(sh->by + h0 + h + 4);
                const float inv[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                const int some = nh - h0 - h;  // heads left
#pragma unroll 1
                for (int d = 0; d < blocks; ++d) {
                    float o[8];
                    __syncwarp();
                    get_o(d, h, o);
                    const bool column = d * 128 + tid < p.Lkv;
                    if (x.place >= 0) {
                        float* at = to_part + d * 128;
#pragma unroll
                        for (int i = 0; i < 8; ++i, at += p.Lkv)
                            if (column && i < some) *at = o[i] * inv[i];
                    } else {
                        uint16_t* at = to_out + d * 128;
#pragma unroll
                        for (int i = 0; i < 8; ++i, at += p.Lkv)
                            if (column && i < some) *at = static_cast<uint16_t>(pack_bf16x2(o[i] * inv[i], 0.f));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh->o_free));
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- MMA
        if (elect_one()) {
            const uint32_t id_s = idesc_e4m3(2 * kHeads, false), id_4 = idesc_e4m3(kWidth, true), id_5 = id_4 | kIdescBE5m2;
            const uint64_t dkv = desc_128(sm_kv), drest = desc_64(sm_rest), dq = desc_128(sm_q), dq_rest = desc_64(sm_q + 4 * kQChunk);
            const uint64_t dp = p_row(kHeads) == 128 ? desc_128(sm_p) : desc_64(sm_p);
            constexpr int kNext = 32 * p_row(kHeads) >> 4;  // the next 32 keys of P
            auto look = [&](uint64_t* bar, uint32_t parity) {
                ok = ok && wait(bar, parity);
                tc_fence_after();
                return ok;
            };
            int slot = 0, round = 0, slot_v = 0;  // of the ring: the next chunk of K, of V
            int opened = 0;                       // pieces whose first values have been multiplied
            // S of step `step`, chunk by chunk as they arrive
            auto scores = [&]() {
                const uint32_t d = tmem + kColS + (step & 1) * kStageS;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c >= chunks) break;
                    if (!look(&sh->kv_full[slot], round)) return;
                    const uint64_t a = dkv + slot * (kChunkBytes >> 4), b = dq + c * (kQChunk >> 4);
                    if (C >= (c + 1) * 128) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_e4m3(d, a + 2 * k, b + 2 * k, id_s, c > 0 || k > 0);
                    } else {
                        for (int k = 0; k < (C - c * 128 + 31) / 32; ++k) mma_e4m3(d, a + 2 * k, b + 2 * k, id_s, c > 0 || k > 0);
                    }
                    if (++slot == kSlots) slot = 0, ++round;
                }
                if (rest) {
                    const int r = step % kRests;
                    if (!look(&sh->rest_full[r], step / kRests)) return;
                    const uint64_t a = drest + r * (kRestBytes >> 4);
                    for (int k = 0; k < (rest + 31) / 32; ++k) mma_e4m3(d, a + 2 * k, dq_rest + 2 * k, id_s, 1);
                }
                mma_commit(smem_u32(&sh->s_full[step & 1]));
                if (kThree && rest) mma_commit(smem_u32(&sh->rest_free[step % kRests]));
            };
            // O^T of step u
            auto values = [&](int u, bool first, int keys32) {
                // (a piece's first values overwrite O, from which the results of the piece before have been read)
                if (first && opened++ > 0 && !look(&sh->o_free, opened - 2)) return;
                const uint64_t b = kThree ? dp : drest + u % kRests * (kRestBytes >> 4);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    if (m >= chunks) break;
                    if (m < blocks) {
                        const uint64_t a = dkv + slot_v * (kChunkBytes >> 4);
#pragma unroll
                        for (int k = 0; k < kKeys / 32; ++k) {
                            if (k >= keys32) break;
                            mma_e4m3(tmem + kColO + m * kWidth, a + k * (32 * 128 >> 4), b + k * kNext, kThree ? id_5 : id_4, !first || k > 0);
                            if (!kThree) mma_e4m3(tmem + kColO + m * kWidth, a + k * (32 * 128 >> 4), dp + k * kNext, id_5, 1);
                        }
                    }
                    // (Chunks without values too, though their scores are all that reads them: places become free in the
                    // order of the chunks.  The copying warps, which do not come to every turn of a place, tell its
                    // phases apart by that.)
                    mma_commit(smem_u32(&sh->kv_free[slot_v]));
                    if (++slot_v == kSlots) slot_v = 0;
                }
                if (!kThree && rest) mma_commit(smem_u32(&sh->rest_free[u % kRests]));
                mma_commit(smem_u32(&sh->pv_done[u & 1]));
            };
            // What is ready: the scores of the next steps, at most two ahead (whose S and weights have places), so that the
            // softmax has some, else the values of a step whose weights are there.  (Values first: 33.9 us
            // instead of 32.7 for V2-Lite 64 sequences; scores chunk by chunk between them: 33.5 instead of 31.0.)
            // Scores begin with the first chunk of 16 heads, with two of more: those would keep the values waiting that free
            // the ring (152 sequences of 8192: of 32 heads 157 us with the first, 136 with the second, 138 with the third,
            // of 64 170, 167, 166; of 16 heads 131, 130, 128, but V2-Lite 64 sequences 29.2, 29.4, 29.8).
            const int begin = kHeads == 16 || chunks == 1 ? 0 : 1;
            auto chunk_there = [&](int c) {
                const bool over = slot + c >= kSlots;
                return mbar_test(smem_u32(&sh->kv_full[over ? slot + c - kSlots : slot + c]), (over ? round + 1 : round) & 1);
            };
            int n = 0, t = 0, keys = 0;             // steps of the piece, those scored; its keys from the next step on
            int values_done = 0, started = 0;       // steps whose values are multiplied; pieces whose first scores are
            uint32_t firsts = 0, tails = 0;         // of two steps, by parity: a piece's first; 32 keys (up to 4), a byte each
            bool end = false;
            uint64_t idle_since = 0;
            uint32_t spins = 0;
            while (true) {
                if (!end && t == n && mbar_test(smem_u32(&sh->piece_full[pieces % kAhead]), pieces / kAhead & 1)) {
                    const Piece y = sh->piece[pieces % kAhead];
                    mbar_arrive(smem_u32(&sh->piece_free[pieces % kAhead]));
                    ++pieces;
                    n = y.n, t = 0, keys = y.len - y.key0;
                    end = n == 0;
                }
                bool idle = true;
                if (t < n && step - values_done <= 1 && (t > 0 || mbar_test(smem_u32(&sh->q_full), started & 1)) && chunk_there(begin)) {
                    scores();
                    if (!ok) break;
                    const int e = step & 1;
                    firsts = (firsts & ~(1u << e)) | static_cast<uint32_t>(t == 0) << e;
                    tails = (tails & ~(255u << 8 * e)) | static_cast<uint32_t>(keys >= kKeys ? kKeys / 32 : (keys + 31) / 32) << 8 * e;
                    if (t == 0) ++started;
                    keys -= kKeys;
                    ++step;
                    if (++t == n) mma_commit(smem_u32(&sh->q_free));
                    idle = false;
                }
                if (values_done < step && mbar_test(smem_u32(&sh->p_full), values_done & 1)) {
                    tc_fence_after();
                    values(values_done, firsts >> (values_done & 1) & 1, tails >> 8 * (values_done & 1) & 255);
                    if (!ok) break;
                    ++values_done;
                    idle = false;
                }
                if (idle) {
                    if (end && values_done == step) break;
                    if (++spins & 63) continue;
                    if (*abort_flag) ok = false;
                    const uint64_t now = global_timer_ns();
                    if (idle_since == 0) idle_since = now;
                    if (now - idle_since > kTimeoutNs) ok = false;
                    if (!ok) break;
                    continue;
                }
                idle_since = 0;
            }
            if (!ok) {  // no MMA may still run when the CTA leaves
                mma_commit(smem_u32(&sh->drain));
                mbar_wait(smem_u32(&sh->drain), 0, kTimeoutNs, nullptr);
            }
        }
    } else if (warp == kLoadWarp || warp == kLoadWarp + 1) {
        // ------------------------------------------------------- pieces, TMA
        // The first warp finds the pieces and copies the first two chunks of each step, the second the others (one warp for
        // all: pages of 16 or 48, boxes of 16 rows, 2.15 us a step of 16 heads instead of 1.93; of 64 alike).  Lane i has box
        // i of a step.
        const bool lead = warp == kLoadWarp;
        const int c0 = lead ? 0 : 2, c1 = lead ? min(chunks, 2) : chunks;
        const int per = kKeys / p.box;
        const int outside = p.c.num_pages > 0 ? p.c.num_pages : 1;  // reads as zeros
        int copied = 0, rests = 0;  // chunks, and columns behind 512, that this warp has copied
        int slot = c0, round = 0;
        auto look_up = [&](int j) {  // the page, looked at when it is used
            const int key = x.key0 + j * kKeys + lane * p.box;
            return lane < per && j < x.n && key < x.len ? p.table[static_cast<int64_t>(x.row) * p.max_pages + p.by_page(key)] : -1;
        };
        auto next_lot = [&]() {
            if (!lead) return next_piece();
            x = walk.next(p);
            ok = put_piece(sh, wait, pieces++, x);
            return ok && x.n > 0;
        };
        while (ok && next_lot()) {
            int found = look_up(0);
            for (int j = 0; j < x.n && ok; ++j, ++step) {
                const int page = found < 0 || found >= p.c.num_pages ? outside : found, key = x.key0 + j * kKeys + lane * p.box;
                const int boxes = min(per, (x.len - x.key0 - j * kKeys + p.box - 1) / p.box), in = key - p.by_page(key) * p.c.page_size;
                found = look_up(j + 1);
                for (int c = c0; c < c1; ++c) {
                    if (round > 0) ok = __all_sync(~0u, ok && wait(&sh->kv_free[slot], round - 1));
                    if (!ok) break;
                    const uint32_t bar = smem_u32(&sh->kv_full[slot]);
                    if (lane == 0) mbar_arrive_expect_tx(bar, boxes * p.box * 128);
                    __syncwarp();
                    if (lane < boxes) tma_load_3d(sm_kv + slot * kChunkBytes + lane * p.box * 128, &tm_rows, bar, c * 128, in, page);
                    ++copied;
                    if (++slot == kSlots) slot = 0, ++round;
                }
                slot += chunks - (c1 > c0 ? c1 - c0 : 0);  // (the other warp's)
                if (slot >= kSlots) slot -= kSlots, ++round;
                if (!lead && rest && ok) {
                    const int r = step % kRests;
                    if (step >= kRests) ok = __all_sync(~0u, ok && wait(&sh->rest_free[r], step / kRests - 1));
                    if (!ok) break;
                    const uint32_t bar = smem_u32(&sh->rest_full[r]);
                    if (lane == 0) mbar_arrive_expect_tx(bar, boxes * p.box * 64);
                    __syncwarp();
                    if (lane < boxes) tma_load_3d(sm_rest + r * kRestBytes + lane * p.box * 64, &tm_rest, bar, 512, in, page);
                    ++rests;
                }
                __syncwarp();
            }
        }
        if (!ok) {  // no copy may still be landing when the CTA leaves: of the last steps
            for (int i = max(copied - kSlots, 0); i < copied; ++i) {
                const int at = i / (c1 - c0) * chunks + c0 + i % (c1 - c0);
                mbar_wait(smem_u32(&sh->kv_full[at % kSlots]), at / kSlots & 1, kTimeoutNs, nullptr);
            }
            for (int u = max(rests - kRests, 0); u < rests; ++u) mbar_wait(smem_u32(&sh->rest_full[u % kRests]), u / kRests & 1, kTimeoutNs, nullptr);
        }
    } else if (warp == kScaleWarp) {
        // ------------------------------------------------- queries and scales
        pdl_wait();  // the kernel that split the queries, or what came before
        int turn = 0, copies = 0;
        auto begin = [&]() {
            if (kSplit) return ok;
            if (pieces > 1) ok = __all_sync(~0u, ok && wait(&sh->q_free, pieces - 2));
            if (ok && lane == 0) {
                const int64_t tile = static_cast<int64_t>(x.b) * p.tiles + x.tile;
                constexpr int kFactors = kHeads * sizeof(float);
                mbar_arrive_expect_tx(smem_u32(&sh->q_full), q_bytes(kHeads) + kFactors);
                bulk_load(sm_q, p.terms + tile * q_bytes(kHeads), q_bytes(kHeads), smem_u32(&sh->q_full));
                bulk_load(smem_u32(sh->f[turn]), p.factors + tile * kHeads, kFactors, smem_u32(&sh->q_full));
                ++copies;
            }
            turn = turn == 2 ? 0 : turn + 1;
            __syncwarp();
            return ok;
        };
        find_scales(p, x, next_piece, begin, [&](int, uint32_t four) {
            if (step >= kAhead) ok = __all_sync(~0u, ok && wait(&sh->scale_free[step % kAhead], step / kAhead - 1));
            if (!ok) return false;
            *reinterpret_cast<uint32_t*>(&sh->scale[step % kAhead][lane * 4]) = four;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh->scale_full[step % kAhead]));
            ++step;
            return true;
        });
        // (the tensor core's last arrival has come)
        if (ok && pieces > 1) ok = __all_sync(~0u, wait(&sh->q_free, pieces - 2));
        // no copy may still be landing when the CTA leaves
        if (!ok && copies) mbar_wait(smem_u32(&sh->q_full), (copies - 1) & 1, kTimeoutNs, nullptr);
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
        tmem_dealloc(tmem, kTmem);
    }
}

// The query rows as two E4M3 terms each, tile after tile as the attention kernels have them in shared memory (zeros behind
// a row's columns and a sequence's heads), and the factors of their scores.  A warp per row.  kPair: as the kernel of CTA
// pairs has them, term after term.  The attention kernel may start as soon as all CTAs are here: what came before has ended.
constexpr int kQueryWarps = 8;
template <int kHeads, bool kPair>
__global__ void __launch_bounds__(kQueryWarps * 32) mla_attend8_query_kernel(const __grid_constant__ Attend8 p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, C = p.c.C, padded = C > 512 ? 576 : (C + 127) / 128 * 128;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kQueryWarps + (threadIdx.x >> 5), tile = at / kHeads;
    const int r = static_cast<int>(at % kHeads), h = static_cast<int>(tile % p.tiles) * kHeads + r;
    if (tile >= static_cast<int64_t>(p.B) * p.tiles) return;
    const uint4* const row = reinterpret_cast<const uint4*>(p.q + (tile / p.tiles * p.H + h) * C);
    uint4 v[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        v[k] = make_uint4(0, 0, 0, 0);
        if (h < p.H && (k * 32 + lane) * 8 < C) v[k] = row[k * 32 + lane];
    }
    uint8_t* const dst = p.terms + tile * q_bytes(kHeads);
    constexpr int kRows = kPair ? kHeads : 2 * kHeads;  // of a chunk: of one term or both
    const float factor = split_row(p, v, [&](int k, uint2 hi, uint2 lo) {
        const int col = (k * 32 + lane) * 8;
        if (col >= padded) return;
        *reinterpret_cast<uint2*>(dst + query_at<kRows>(r, col)) = hi;
        *reinterpret_cast<uint2*>(dst + (kPair ? q_bytes(kHeads) / 2 + query_at<kRows>(r, col) : query_at<kRows>(r + kHeads, col))) = lo;
    });
    if (lane == 0) p.factors[at] = factor;
}

// Joins the partial results of the tiles that several units shared, in the order of the cut (a tile of one piece was
// finished by that piece), and sets the rows without keys.  A warp per 128 columns of a row, or, where there are many
// pieces, the warps of a CTA; with four pieces on their way.  It has to move the partial results (V3 128 sequences: 8 us of
// 50) and to start: each instruction comes from L2 the first time.  So the code is short (with eight pieces on their way,
// or four rows at once, V2-Lite 64 sequences took 0.3 and 2.5 us more, one V3 sequence of 131072 3.0 and 5.3 more).
constexpr int kJoinCtas = 4, kJoinWarps = 8, kJoinThreads = kJoinWarps * 32, kJoinMost = 512, kJoinFew = 8;

__global__ void __launch_bounds__(kJoinThreads, kJoinCtas) mla_attend8_join_kernel(const __grid_constant__ Attend8 p) {
    __shared__ Joint8 joints[kJoinMost];
    __shared__ int units[kJoinMost], turns[kJoinMost + 1];  // of each: its first unit, turns before it
    __shared__ int found_all;
    __shared__ float tops[kJoinWarps], sums[kJoinWarps];
    __shared__ float4 others[kJoinWarps][32];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = p.group * p.heads;
    const int parts = (p.Lkv + 127) / 128;   // of a row
    if (warp == 0) {  // the tiles to join, and their turns
        int before = 0, found = 0;
#pragma unroll 1
        for (int u0 = 0; u0 < p.units; u0 += 160) {
            Joint8 j[5];
#pragma unroll
            for (int k = 0; k < 5; ++k) {
                const int u = u0 + k * 32 + lane;
                j[k].count = 0;
                if (u < p.units) j[k] = p.joints[u];
            }
#pragma unroll
            for (int k = 0; k < 5; ++k) {
                const int u = u0 + k * 32 + lane;
                const Joint8& x = j[k];
                // (an attention that gave up may have left some unwritten)
                const bool some = x.count > 0 && x.count <= p.units - u && static_cast<unsigned>(x.b) < static_cast<unsigned>(p.B) &&
                                  static_cast<unsigned>(x.pass) < static_cast<unsigned>(p.passes) && static_cast<unsigned>(x.place) < 2;
                const uint32_t all = __ballot_sync(~0u, some), few = __ballot_sync(~0u, some && x.count <= kJoinFew);
                const uint32_t below = (1u << lane) - 1;
                const int each = rows * parts, each_few = each / kJoinWarps;
                if (some) {
                    const int i = found + __popc(all & below);
                    joints[i] = x;
                    units[i] = u;
                    turns[i] = before + __popc(few & below) * each_few + __popc(all & ~few & below) * each;
                }
                found += __popc(all);
                before += __popc(few) * each_few + __popc(all & ~few) * each;
            }
        }
        if (lane == 0) turns[found] = before, found_all = found;
    }
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        int row, bits = 0;
        if (batch_len(p, b, &row, &bits)) continue;
        uint4* const out = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(b) * p.H * p.Lkv);
        for (int64_t i = threadIdx.x; i < static_cast<int64_t>(p.H) * p.Lkv / 8; i += kJoinThreads) out[i] = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int h = threadIdx.x; h < p.H; h += kJoinThreads) p.lse[static_cast<int64_t>(b) * p.H + h] = -INFINITY;
    }
    __syncthreads();
    const int end = turns[found_all];
    int at = 0;
#pragma unroll 1
    for (int turn = blockIdx.x; turn < end; turn += gridDim.x) {
        while (turn >= turns[at + 1]) ++at;
        const Joint8 j = joints[at];
        const bool few = j.count <= kJoinFew;
        const int task = few ? (turn - turns[at]) * kJoinWarps + warp : turn - turns[at];
        const int r = task / parts, quad = (task - r * parts) * 32 + lane, step = few ? 1 : kJoinWarps;
        const int h = j.pass * rows + r;
        const bool mine = h < p.H && quad * 4 < p.Lkv;
        float top = -INFINITY, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (mine) {
#pragma unroll 1
            for (int i0 = few ? 0 : warp; i0 < j.count; i0 += 4 * step) {
                float z[4];
                float4 o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = i0 + k * step;
                    z[k] = -INFINITY;
                    o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i < j.count) {
                        const int64_t part = static_cast<int64_t>((units[at] + i) * 2 + (i == 0 ? j.place : 0)) * rows + r;
                        z[k] = p.part_lse[part];
                        o[k] = reinterpret_cast<const float4*>(p.part_o + part * p.Lkv)[quad];
                    }
                }
                const float next = fmaxf(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])), top);
                const float keep = ex2(top - next);  // (NaN where every z is: the sum then is too)
                top = next;
                sum *= keep, acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float w = ex2(z[k] - next);
                    sum += w;
                    acc.x = fmaf(w, o[k].x, acc.x), acc.y = fmaf(w, o[k].y, acc.y), acc.z = fmaf(w, o[k].z, acc.z), acc.w = fmaf(w, o[k].w, acc.w);
                }
            }
        }
        if (!few) {  // (the same in all warps)
            if (lane == 0) tops[warp] = top, sums[warp] = sum;
            others[warp][lane] = acc;
            __syncthreads();
            if (warp == 0) {
                for (int g = 1; g < kJoinWarps; ++g) top = fmaxf(top, tops[g]);
                sum = 0.f;
                acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                for (int g = 0; g < kJoinWarps; ++g) {
                    const float w = ex2(tops[g] - top);
                    const float4 o = others[g][lane];
                    sum = fmaf(w, sums[g], sum);
                    acc.x = fmaf(w, o.x, acc.x), acc.y = fmaf(w, o.y, acc.y), acc.z = fmaf(w, o.z, acc.z), acc.w = fmaf(w, o.w, acc.w);
                }
            }
            __syncthreads();
        }
        if (mine && (few || warp == 0)) {
            const int64_t row = static_cast<int64_t>(j.b) * p.H + h;
            const float inv = 1.f / sum;
            reinterpret_cast<uint2*>(p.out + row * p.Lkv)[quad] = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            if (quad == 0 && p.lse) p.lse[row] = (top + log2f(sum)) * kLn2;
        }
    }
}

int check_attend8(const Cache8& c, const mla_prolog_attend8_dims* d) {
    if (!d) return MLA_ERR_INVALID_ARG;
    if (d->batch < 0 || d->batch > kMaxBatch || d->num_heads < 1 || static_cast<int64_t>(d->batch) * d->num_heads > (1 << 24) ||
        d->kv_lora_rank < 16 || d->kv_lora_rank > 512 || d->kv_lora_rank % 16 || d->kv_lora_rank > c.C ||
        d->table_rows < 0 || d->max_pages < 1 || static_cast<int64_t>(d->max_pages) * c.page_size > (1 << 30) || !scale_ok(d->scale))
        return MLA_ERR_UNSUPPORTED_DIMS;
    return MLA_OK;
}

// Workspace: what is to join, the partial results, the queries' terms.
struct Layout8 {
    int heads, group, passes, units;
    size_t part_lse, part_o, terms, factors, bytes;
};

Layout8 layout8(const mla_prolog_attend8_dims& d, int sms) {
    Layout8 y;
    y.heads = d.num_heads <= 16 ? 16 : d.num_heads <= 32 ? 32 : 64;
    const int tiles = (d.num_heads + y.heads - 1) / y.heads;
    y.group = tiles > 1 ? 2 : 1;
    y.passes = (tiles + y.group - 1) / y.group;
    y.units = sms < kJoinMost ? sms / y.group : kJoinMost / y.group;
    if (y.units < 1) y.units = 1;
    auto round = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t parts = static_cast<size_t>(y.units) * 2 * y.group * y.heads;
    y.part_lse = round(sizeof(Joint8) * y.units);
    y.part_o = y.part_lse + round(sizeof(float) * parts);
    y.terms = y.part_o + round(sizeof(float) * parts * d.kv_lora_rank);
    const size_t q_tiles = static_cast<size_t>(d.batch) * y.passes * y.group;
    y.factors = y.terms + q_tiles * q_bytes(y.heads);
    y.bytes = y.factors + q_tiles * y.heads * sizeof(float);
    return y;
}

// The codes [pages][page_size][C] in boxes of 1 x `rows` x `width` columns under the swizzle of that width; what lies
// outside reads as 0.  chunks > 0: the whole 128-column chunks, [chunk][page][row][128], so many in a box.
bool encode_rows(CUtensorMap* m, const void* base, const Cache8& c, uint32_t width, uint32_t rows, uint32_t chunks = 0) {
    auto fn = reinterpret_cast<CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                            CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                            CUtensorMapFloatOOBfill)>(tensor_map_encoder());
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(chunks ? 128 : c.C), static_cast<cuuint64_t>(c.page_size),
                                static_cast<cuuint64_t>(c.num_pages > 0 ? c.num_pages : 1), static_cast<cuuint64_t>(c.C / 128)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.C), static_cast<cuuint64_t>(c.page_bytes), 128};
    const cuuint32_t box[4] = {width, rows, 1, chunks}, each[4] = {1, 1, 1, 1};
    return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, chunks ? 4 : 3, const_cast<void*>(base), dims, strides, box, each,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

template <int kHeads, bool kSplit>
cudaError_t launch8(const CUtensorMap& rows, const CUtensorMap& rest, const Attend8& p, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(&mla_attend_cache8_kernel<kHeads, kSplit>, smem_bytes(kHeads), &ready);
    if (e != cudaSuccess) return e;
    return launch_kernel(mla_attend_cache8_kernel<kHeads, kSplit>, dim3(p.units * p.group), dim3(kThreads), smem_bytes(kHeads), st,
                         true, rows, rest, p);
}

}  // namespace
}  // namespace mlap

using namespace mlap;

extern "C" {

int mla_prolog_attend_cache8_workspace(const mla_prolog_cache8* cache, const mla_prolog_attend8_dims* d, size_t* bytes) {
    if (!bytes) return MLA_ERR_INVALID_ARG;
    *bytes = 0;
    Cache8 c;
    int rc = check_cache8(cache, &c), sms;
    if (rc != MLA_OK || (rc = check_attend8(c, d)) != MLA_OK || (rc = current_sm103(&sms)) != MLA_OK) return rc;
    *bytes = layout8(*d, sms).bytes;
    return MLA_OK;
}

int mla_prolog_attend_cache8(const mla_prolog_cache8* cache, const mla_prolog_attend8_dims* d, const void* q,
                             const int32_t* page_table, const int32_t* seq_lens, const int32_t* seqs, void* out, float* lse,
                             void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
    Cache8 c;
    int rc = check_cache8(cache, &c), sms;
    if (rc != MLA_OK || (rc = check_attend8(c, d)) != MLA_OK) return rc;
    if (!seqs && d->table_rows < d->batch) return MLA_ERR_INVALID_ARG;
    if (d->batch == 0) return MLA_OK;
    if (!ptr_ok(q, 16) || !ptr_ok(out, 16) || (c.num_pages && !ptr_ok(c.pages, 16))) return MLA_ERR_INVALID_ARG;
    if (d->table_rows && (!ptr_ok(page_table, 4) || !ptr_ok(seq_lens, 4))) return MLA_ERR_INVALID_ARG;
    if ((seqs && !ptr_ok(seqs, 4)) || (lse && !ptr_ok(lse, 4)) || (status && !ptr_ok(status, 4)) || !ptr_ok(workspace, 16))
        return MLA_ERR_INVALID_ARG;
    if ((rc = current_sm103(&sms)) != MLA_OK) return rc;
    const Layout8 y = layout8(*d, sms);
    if (workspace_bytes < y.bytes) return MLA_ERR_INVALID_ARG;
    const int box = gcd(c.page_size, kKeys);
    // an empty cache has no valid page: every read is outside the map, which then only needs a valid address
    const void* base = c.num_pages ? c.pages : q;
    const bool pair = y.group == 2;
    // (a pair's CTAs have 64 keys each: boxes of up to 64 rows, several chunks at once where those are whole)
    const int rows_box = pair && box > 64 ? 64 : box;
    CUtensorMap rows, rest, k, v;
    bool good = encode_rows(&rows, base, c, 128, rows_box);
    if (c.C > 512) good = good && encode_rows(&rest, base, c, 64, rows_box);
    else rest = rows;
    k = v = rows;
    if (pair && c.C >= 512 && rows_box == 64) {
        good = good && encode_rows(&k, base, c, 128, 64, 4);
        if (d->kv_lora_rank > 384) good = good && encode_rows(&v, base, c, 128, 64, 2);
    }
    if (!good) return report_cuda(cudaErrorInvalidValue, "tensor maps of attend_cache8");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    // whole tiles are looked at while each has a thread and each unit's a lane
    const int64_t whole = static_cast<int64_t>(d->batch) * y.passes;
    const int rounds = whole <= kThreads && y.units <= kThreads && whole <= 32 * y.units ? static_cast<int>((whole + y.units - 1) / y.units) : 0;
    const int most_cost = pair ? kJoinCostPair : join_cost(y.heads);
    const int join = kJoinCostLeast + (most_cost - kJoinCostLeast) * static_cast<int>(whole < y.units ? whole : y.units) / y.units;
    const Attend8 p{c, divide_by(c.page_size), divide_by(c.block), static_cast<const uint16_t*>(q), page_table, seq_lens, seqs, static_cast<uint16_t*>(out), lse, status,
                    reinterpret_cast<Joint8*>(ws),
                    reinterpret_cast<float*>(ws + y.part_o), reinterpret_cast<float*>(ws + y.part_lse), ws + y.terms,
                    reinterpret_cast<float*>(ws + y.factors), d->batch,
                    d->num_heads, d->kv_lora_rank, d->table_rows, d->max_pages, rows_box, y.heads, y.group, y.passes, y.passes * y.group, y.units, pair ? kOverheadPair : kOverheadOne, join, rounds,
                    d->scale};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // 16 rows are split by the CTA that uses them, where most have one tile: a launch less (one sequence 10.3 -> 9.6 us, 152
    // of up to 500 17.8 -> 16.2; 64 of up to 3000, cut into two pieces a CTA, 26.2 -> 26.9; of 32 heads 32.3 -> 35.0)
    cudaError_t e;
    if (y.heads == 16 && whole <= y.units) {
        e = launch8<16, true>(rows, rest, p, st);
    } else {
        const int64_t rows_all = static_cast<int64_t>(d->batch) * p.tiles * p.heads;
        const auto query = pair ? &mla_attend8_query_kernel<64, true> : y.heads == 16 ? &mla_attend8_query_kernel<16, false>
                           : y.heads == 32 ? &mla_attend8_query_kernel<32, false> : &mla_attend8_query_kernel<64, false>;
        e = launch_kernel(query, dim3(static_cast<unsigned>((rows_all + kQueryWarps - 1) / kQueryWarps)), dim3(kQueryWarps * 32), 0, st, true, p);
        if (e != cudaSuccess) return report_cuda(e, "launch mla_attend8_query_kernel");
        e = pair ? launch_attend8_pair(rows, rest, k, v, p, st) : y.heads == 16 ? launch8<16, false>(rows, rest, p, st)
            : y.heads == 32 ? launch8<32, false>(rows, rest, p, st) : launch8<64, false>(rows, rest, p, st);
    }
    if (e != cudaSuccess) return report_cuda(e, "launch the attend_cache8 kernel");
    // as many CTAs as are resident at once, no more than there can be rows to join or to clear
    const int64_t most = static_cast<int64_t>(d->batch) + static_cast<int64_t>(y.units) * y.group * y.heads;
    e = launch_kernel(mla_attend8_join_kernel, dim3(static_cast<unsigned>(most < kJoinCtas * sms ? most : kJoinCtas * sms)), dim3(kJoinThreads), 0, st, true, p);
    return e == cudaSuccess ? MLA_OK : report_cuda(e, "launch mla_attend8_join_kernel");
}

}  // extern "C"
