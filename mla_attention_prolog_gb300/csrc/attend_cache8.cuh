// What the two attention kernels over the 8-bit latent cache share: the cut of
// the work, the pieces, the scales and the queries as E4M3 terms.
#pragma once

#include "attend_ptx.cuh"
#include "cache8.cuh"

namespace mlap {

constexpr int kKeys = 128;                      // keys per step
constexpr int kThreads = 384;                   // (three warps a scheduler: 168 registers)
constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp = 9, kScaleWarp = 11;  // (the last: queries too)
constexpr int kSoft = kSoftWarps * 32;
constexpr int kAhead = 4;                       // pieces found ahead
constexpr int kMiscBytes = 3 * 1024;
constexpr uint64_t kTimeoutNs = 1000000000ull;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// The bound of a row's (a head's) weights: log2 of the largest P before it has to move is kMost, and P of at most kMostP
// passes.  With a piece's first keys it is set so that a key kDeviations standard deviations above their mean stays below
// it, between 2^kLow and 2^kTopAlone for the largest of them: rows that vary little, or in which one key (a first token,
// say) outweighs the others, keep their small weights far above the smallest P.  Where a weight passes it later, the bounds
// of all rows for which that step's keys ask for a higher one move, to at most 2^kTopLater for the largest.  (One move
// takes as long as one to two steps.  Steps in which a bound moves, of 57 on scales that differ by 4 from block to block,
// 64 heads: 1.3, with 6 deviations 2.4; with 7 and the passed rows alone 8, without a look at the deviation 13 or more.)
constexpr float kMost = 11.75f, kMostP = 3444.f, kTopAlone = 11.f, kTopLater = 7.f, kLow = 2.f, kDeviations = 7.f;
__device__ __forceinline__ float first_top(float top, float sum, float squares) {  // of kKeys keys
    const float mean = sum * (1.f / kKeys), variance = fmaxf(squares * (1.f / kKeys) - mean * mean, 0.f);
    const float room = fmaxf(mean + kDeviations * sqrtf(variance) - top, 0.f);
    return fminf(fmaxf(kMost - room, kLow), kTopAlone);
}
// A tile's start and end, in key steps: on CTA pairs, alone.  (V3 128 sequences of 1 to 1024, cut: 4 51.2 us, 2 54.4, 6 54.3,
// long contexts 131 to 133 with 3 to 5.  37 sequences of 5 heads: 2 17.7, 3 19.0, 4 20.0; V2-Lite 64: 29.2, 29.2, 29.5.)
constexpr int kOverheadPair = 4, kOverheadOne = 2;
// What joining shared tiles costs, in key steps: from kJoinCostLeast of few tiles to these of as many as there are units.
// Whole tiles are dealt to the units where that takes no longer.  (128 heads, 128 sequences of 1 to 4096: dealt 66 us, cut
// 84; 76 of them, 10 steps longer dealt: 59, 62; 60, 16 longer: 55, 50.  64 heads, 200, 7 longer: 96, 100; 152, 13 longer:
// 93, 82.  16 heads, 200 of 1 to 4096, 7 longer: 77, 76; of up to 1024, 152, one longer: 25, 31; 40, 4 longer: 21, 19; 40
// of up to 256, 2 shorter: 13, 18.)
constexpr int kJoinCostLeast = 2, kJoinCostPair = 10;
constexpr int join_cost(int heads) { return heads == 64 ? 8 : heads == 32 ? 6 : 5; }
constexpr int kLargeBatch = kThreads;           // rows; more are never dealt
constexpr int kMinRun = 2;                      // shortest run worth a unit, in key steps after its tile's start (37
                                                // sequences of 5 heads: 17.6 us, with 1 17.7, with 3 19.9)

// A tile whose steps several units share, found by the unit with the first of them.
struct Joint8 {
    int32_t b, pass;  // batch row, round over its tiles
    int32_t count;    // units; 0: none
    int32_t place;    // of the first unit's partial result
};

struct Attend8 {
    Cache8 c;
    Divide by_page, by_block;
    const uint16_t* q;
    const int32_t *table, *lens, *seqs;
    uint16_t* out;
    float* lse;
    int32_t* status;
    Joint8* joints;   // workspace: what is to join [units],
    float* part_o;    //   partial results [units][2][group * heads][Lkv]
    float* part_lse;  //   and their log2-sum-exp,
    uint8_t* terms;   //   the query rows' terms as they lie in shared memory [B][tiles][q_bytes]
    float* factors;   //   and the factors of their scores [B][tiles][heads]
    int B, H, Lkv, table_rows, max_pages, box;
    int heads;        // of a tile
    int group;        // CTAs of a unit: that many tiles of a sequence at once
    int passes;       // rounds over a sequence's tiles
    int tiles;        // of a sequence: passes * group
    int units;
    int overhead;     // cost of a tile beside its steps
    int join_cost;    // and of joining the tiles that units share
    int rounds;       // of dealing whole tiles to the units (0: too many)
    float scale;
};

// Table row (-1: none) and length of batch row b.
__device__ __forceinline__ int batch_len(const Attend8& p, int b, int* row, int* bits) {
    const int s = p.seqs ? p.seqs[b] : b;
    if (s < 0 || s >= p.table_rows) {
        *row = -1;
        *bits |= kStatusSeqRange;
        return 0;
    }
    *row = s;
    const int n = p.lens[s], cap = p.max_pages * p.c.page_size;
    if (n < 0 || n > cap) *bits |= kStatusSeqRange;
    return n < 0 ? 0 : n > cap ? cap : n;
}

__device__ __forceinline__ int steps_of(int len) { return (len + kKeys - 1) / kKeys; }
__device__ __forceinline__ int64_t seq_cost(const Attend8& p, int len) {
    return len ? static_cast<int64_t>(p.passes) * (steps_of(len) + p.overhead) : 0;
}

struct Piece {
    int b, row;    // batch row, row of the page table
    int tile;      // of heads
    int key0, len; // first key, the sequence's length
    int n;         // steps; 0: the unit has no more pieces
    int place;     // of its partial result (0: begun before the unit, 1: in it), -1: covers the sequence
};

// a / b, both positive: most quotients fit 32 bits, whose division is far shorter.
static __device__ __noinline__ int64_t quotient64(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return (a | b) >> 32 ? quotient64(a, b) : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// D[tmem] (+)= A[smem] B[smem]^T, E4M3 operands, FP32 sums.
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Shared-memory descriptors: rows of 128 or 64 bytes under the swizzle of that width, in atoms of 8 rows; along K where
// the rows run along M or N, and the other way round.
__device__ __forceinline__ uint64_t desc_128(uint32_t addr) { return smem_desc_sw128(addr); }
__device__ __forceinline__ uint64_t desc_64(uint32_t addr) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(512u >> 4) << 32 |
           static_cast<uint64_t>(1u) << 46 | static_cast<uint64_t>(4u) << 61;
}

// Instruction descriptor of kind::f8f6f4: D FP32 (bits 4-5 = 1), A and B E4M3 (bits 7-9 = 10-12 = 0; 1: E5M2), A and B
// MN-major (bits 15, 16), N >> 3 at bits 17-22, M >> 4 at bits 24-28.
constexpr uint32_t kIdescBE5m2 = 1u << 10;
__device__ __forceinline__ constexpr uint32_t idesc_e4m3(int n, bool mn_major) {
    return (1u << 4) | (mn_major ? 3u << 15 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

// The sum over a warp's lanes of each of N values (N a power of two up to 32): lane i is left with that of value
// i / (32 / N) in v[0].
template <int N>
__device__ __forceinline__ void sum_across(float (&v)[N], int lane) {
#pragma unroll
    for (int o = 16, n = N; o > 0; o >>= 1) {
        if (n == 1) {
            v[0] += __shfl_xor_sync(~0u, v[0], o);
            continue;
        }
        n >>= 1;
        const bool upper = lane & o;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if (i >= n) break;
            const float keep = upper ? v[i + n] : v[i], give = upper ? v[i] : v[i + n];
            v[i] = keep + __shfl_xor_sync(~0u, give, o);
        }
    }
}

// FP32 as integers of the same order, and back.
__device__ __forceinline__ int ordered(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

__device__ __forceinline__ void ld_shared_2x2(const float* at, uint64_t& a, uint64_t& b) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(smem_u32(at)) : "memory");
}
// 16 columns at `ta` and at `tb`, and the wait for both.
__device__ __forceinline__ void tmem_ld16x2(uint32_t ta, uint32_t tb, uint32_t (&a)[16], uint32_t (&b)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(a[8]),
          "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]), "=r"(b[0]), "=r"(b[1]),
          "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]), "=r"(b[8]), "=r"(b[9]), "=r"(b[10]),
          "=r"(b[11]), "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15])
        : "r"(ta), "r"(tb)
        : "memory");
}

// Two values up to 448 as the sums of two E4M3 values each.
__device__ __forceinline__ void split_query(float a, float b, uint32_t& first, uint32_t& second) {
    uint32_t v, left;
    uint16_t c, d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(v));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(left) : "r"(v), "r"(f16x2_of_e4m3x2(c)));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(left));
    first = c, second = d;
}

// A contiguous copy global -> shared, completion counted on `bar` (16-byte aligned).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(bar), "r"(parity)
        : "memory");
    return r != 0;
}

// Weights far under the largest are rounded up or down by turns.  Where 8 bits leave a weight only a few steps, weights
// that are alike would all be rounded the same way: 16384 keys at 2^-18 of one other had 5 to 11% less or more than their
// share.  So the last term of a small weight is rounded up in as many keys as its remainder asks for: where the byte that
// is cut off and a key's turn pass 255.  Turns are the leading bits of the keys' numbers times the golden ratio (modulo
// 1), which lie evenly for any run of keys: the share is within 0.1% then.  The error of one such weight is a step where it
// was half of one.  (It takes 1 to 2% on CTA pairs, long contexts 128.5 -> 130.7 us, 1% with 64 heads, nothing with fewer.)
__device__ __forceinline__ uint32_t turn_of(int i) { return static_cast<uint32_t>(i) * 0x9E3779B1u >> 24; }  // 2^32 / 1.618...
// What is added to FP16 bits (two values, `p` of weights) before their lower bytes are cut off: half a step, or of weights
// below `small` (FP16, both halves) the turn.  `turn`: in both halves, less half a step (exclusive or 0x80).
__device__ __forceinline__ uint32_t round_up(uint32_t p, uint32_t small, uint32_t turn) {
    uint32_t is_small;
    asm("set.lt.u32.f16x2 %0, %1, %2;" : "=r"(is_small) : "r"(p), "r"(small));
    return (is_small & turn) ^ 0x00800080u;
}

// Two weights as the sum of an E4M3 and an E5M2 value each (bytes in the halves' order; `five` in the upper byte of each
// half), in FP16, of which E5M2 is the upper byte.  From 256 on E5M2 takes the value and E4M3 what is left of it, below
// the other way round: to 2^-7 of the weight up to 3584 and down to 2^-6, to 2^-13 below that, by turns.  NaN goes by E4M3.
// `p`: the weights in FP16.
__device__ __forceinline__ void split_weights(float a, float b, uint32_t turn, uint32_t& p, uint32_t& four, uint32_t& five) {
    uint32_t is_large, large, rest, again, left;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(p) : "f"(b), "f"(a));
    asm("set.ge.u32.f16x2 %0, %1, %2;" : "=r"(is_large) : "r"(p), "r"(0x5c005c00u));
    large = (p + 0x00800080u) & 0xff00ff00u & is_large;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(p), "r"(large));
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(rest));
    four = c;
    again = f16x2_of_e4m3x2(c);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(left) : "r"(rest), "r"(again));
    five = large | ((left + round_up(p, 0x24002400u, turn)) & 0xff00ff00u & ~is_large);  // 2^-6
}
// The same as the sum of three E5M2 values each, upper bytes of the halves: to 2^-9 of the weight (2^-11 for FP16) down to
// 2^-8, to 2^-16 below that, by turns.
__device__ __forceinline__ void split_weights3(float a, float b, uint32_t turn, uint32_t& x, uint32_t& y, uint32_t& z) {
    uint32_t p;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(p) : "f"(b), "f"(a));
    const uint32_t up = round_up(p, 0x1c001c00u, turn);  // 2^-8
    x = (p + 0x00800080u) & 0xff00ff00u;
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(p) : "r"(x));
    y = (p + 0x00800080u) & 0xff00ff00u;
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(p) : "r"(y));
    z = p + up;
}

// Sum of values below 2^45 over the warp.
__device__ __forceinline__ int64_t warp_sum(int64_t v) {
    const uint32_t low = __reduce_add_sync(~0u, static_cast<uint32_t>(v) & 0xfffffu);
    return (static_cast<int64_t>(__reduce_add_sync(~0u, static_cast<uint32_t>(v >> 20))) << 20) + low;
}

// Costs of a large batch: lane i gets the cost up to the end of its i-th part of `each` times 32 rows.  (A function of its own,
// that small batches do not read from L2.)
static __device__ __noinline__ int64_t part_costs(const int32_t* lens, const int32_t* seqs, int32_t* status, int B, int table_rows, int cap,
                                                  int passes, int overhead, int each) {
    const int lane = threadIdx.x & 31;
    int64_t upto = 0, mine = 0;
    int part = 0, in = 0, next[8];
    bool outside = false;
    // batch_len of a lane's rows, in two steps: eight rows' lengths are on their way while those before are summed
    auto load = [&](int b) {
        int s[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            s[k] = b + k * 32 + lane;
            if (seqs && s[k] < B) s[k] = seqs[s[k]];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const bool in_batch = b + k * 32 + lane < B, in_table = s[k] >= 0 && s[k] < table_rows;
            next[k] = 0;
            if (in_batch && in_table) next[k] = lens[s[k]];
            outside |= in_batch && !in_table;
        }
    };
    load(0);
#pragma unroll 1
    for (int b = 0; b < B; b += 256) {
        int len[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) len[k] = next[k];
        load(b + 256);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            outside |= len[k] < 0 || len[k] > cap;
            len[k] = max(0, min(len[k], cap));
            if (len[k]) mine += static_cast<int64_t>(passes) * (steps_of(len[k]) + overhead);
            if (++in == each) {
                const int64_t sum = warp_sum(mine);
                if (lane == part) upto = sum;
                mine = 0, in = 0, ++part;
            }
        }
    }
    const int64_t sum = warp_sum(mine);  // (of a last part that is not full)
    if (lane == part) upto = sum;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += v;
    }
    if (blockIdx.x == 0 && __any_sync(~0u, outside) && lane == 0) raise_status(status, kStatusSeqRange);
    return upto;
}

// Deals whole tiles to the units, the longest first, forth and back: scratch[kThreads + u]: the cost of unit u's,
// scratch[2 * kThreads + i]: 1 + the one that this unit gets in round i (0: none).  All threads, p.rounds > 1.
__device__ __forceinline__ void deal_tiles(const Attend8& p, int unit, uint32_t* scratch) {
    const int t = threadIdx.x, n = p.B * p.passes;
    int row, bits = 0;
    const int steps = t < n ? steps_of(batch_len(p, t / p.passes, &row, &bits)) : 0;
    const uint32_t key = t < n ? static_cast<uint32_t>(min(steps, (1 << 23) - 1)) * 512 + (511 - t) : 0;  // (no two alike)
    scratch[t] = key;
    scratch[kThreads + t] = 0;
    if (t < 32) scratch[2 * kThreads + t] = 0;
    __syncthreads();
    if (t < n) {
        int rank = 0;
#pragma unroll 4
        for (int i = 0; i < n; i += 4) {
            const uint4 k = *reinterpret_cast<const uint4*>(scratch + i);
            rank += (k.x > key) + (k.y > key) + (k.z > key) + (k.w > key);
        }
        const int i = rank / p.units, m = rank - i * p.units, u = i & 1 ? p.units - 1 - m : m;
        if (steps) atomicAdd(scratch + kThreads + u, static_cast<uint32_t>(steps + p.overhead));
        if (u == unit) scratch[2 * kThreads + i] = t + 1;
    }
    fence_proxy_async_shared();  // (copies will land here)
    __syncthreads();
}

// Cuts the work and finds the pieces of a unit, one after another; the lanes of a warp hold the lengths of 32 batch rows.
// (One warp does so in each CTA while the others get under way: what runs once is read from L2, 8 instructions at a time.)
struct Walk {
    int64_t run, from, to;  // cost per unit, and of this one
    int64_t base, at;       // cost before batch row b; where the walk is
    int unit, rank, b, len32, row32;
    Joint8 joint;
    int round, dealt;       // of whole tiles: the next one's round; lane i: the tile of round i
    bool whole;

    // Costs of the 32 batch rows from `first` on, a lane each.
    __device__ __forceinline__ int64_t costs(const Attend8& p, int first, int* bits) {
        const int i = first + (threadIdx.x & 31);
        row32 = -1;
        len32 = i < p.B ? batch_len(p, i, &row32, bits) : 0;
        return seq_cost(p, len32);
    }

    // Whole warp.  scratch: what deal_tiles left there.
    __device__ __forceinline__ void start(const Attend8& p, int unit_, int rank_, const uint32_t* scratch) {
        unit = unit_, rank = rank_, joint = Joint8{0, 0, 0, 0};
        const int lane = threadIdx.x & 31;
        int bits = 0, longest = 0;
        int64_t total = 0, upto = 0;
        // (4096 sequences of up to 200 keys 205 us, without the parts 257: the first row of a unit is found with a look at all
        // before it, one length at a time)
        const bool large = p.B > kLargeBatch;
        const int each = (p.B + 1023) / 1024;
        if (large) {
            upto = part_costs(p.lens, p.seqs, p.status, p.B, p.table_rows, p.max_pages * p.c.page_size, p.passes, p.overhead, each);
            total = __shfl_sync(~0u, upto, 31);
        } else {
#pragma unroll 4
            for (b = 0; b < p.B; b += 32) {
                total += costs(p, b, &bits);
                longest = max(longest, len32);
            }
            if (__any_sync(~0u, total >> 26)) {
#pragma unroll 1
                for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
            } else {
                total = __reduce_add_sync(~0u, static_cast<uint32_t>(total));
            }
        }
        if (blockIdx.x == 0 && __any_sync(~0u, bits) && lane == 0) raise_status(p.status, kStatusSeqRange);
        // Equal runs of whole steps.  (Runs on all units that differ by a step were no faster: V2-Lite 64 sequences 32.3 us
        // against 31.7, V3 128 sequences 52.0 against 51.7.)
        run = quotient(total + p.units - 1, p.units);
        if (run < kMinRun + p.overhead) run = kMinRun + p.overhead;
        whole = false;
        if (p.rounds) {
            uint32_t most = steps_of(longest) + p.overhead;
            round = 0;
            dealt = lane == 0 && unit < p.B * p.passes ? unit : -1;
            if (p.rounds > 1) {
                most = 0;
#pragma unroll 1
                for (int u = lane; u < p.units; u += 32) most = max(most, scratch[kThreads + u]);
                dealt = static_cast<int>(scratch[2 * kThreads + lane]) - 1;
            }
            whole = __reduce_max_sync(~0u, most) <= run + p.overhead + p.join_cost;
            if (whole) return;
        }
        b = 0;
        base = 0;
        from = to = at = run * unit;
        if (from >= total) return;  // (no pieces)
        to = from + run < total ? from + run : total;
        if (large) {
            const int part = __ffs(__ballot_sync(~0u, upto > at)) - 1;
            if (part) base = __shfl_sync(~0u, upto, part - 1);
            b = part * each * 32;
        }
        if (total >> 31) find<int64_t>(p);
        else find<uint32_t>(p);
    }

    // The batch row that holds `at`, and the cost before it.
    template <class T>
    __device__ __forceinline__ void find(const Attend8& p) {
        const int lane = threadIdx.x & 31;
        int bits = 0;
        const T target = static_cast<T>(at);
        T before = static_cast<T>(base);
#pragma unroll 1
        while (true) {
            const T mine = static_cast<T>(costs(p, b, &bits));
            T upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const T v = __shfl_up_sync(~0u, upto, o);
                if (lane >= o) upto += v;
            }
            const uint32_t ends = __ballot_sync(~0u, before + upto > target);  // (the first of them holds it)
            if (ends) {
                const int i = __ffs(ends) - 1;
                base = before + __shfl_sync(~0u, upto - mine, i);
                b += i;
                return;
            }
            before += __shfl_sync(~0u, upto, 31);
            b += 32;
        }
    }

    // The next piece (n = 0: none).  Whole warp.
    __device__ __forceinline__ Piece next(const Attend8& p) {
        const int lane = threadIdx.x & 31;
        int bits = 0;
        while (whole && round < p.rounds) {
            const int t = __shfl_sync(~0u, dealt, round++), i = t / p.passes;
            int row = -1;
            const int len = t < 0 ? 0 : batch_len(p, i, &row, &bits);
            if (len) return Piece{i, row, (t - i * p.passes) * p.group + rank, 0, len, steps_of(len), -1};
        }
        while (!whole && at < to && b < p.B) {
            const int len = __shfl_sync(~0u, len32, b & 31), row = __shfl_sync(~0u, row32, b & 31);
            const int64_t cost = seq_cost(p, len);
            if (at >= base + cost) {
                base += cost;
                if (!(++b & 31)) costs(p, b, &bits);
                continue;
            }
            const int steps = steps_of(len), each = steps + p.overhead;
            const int pass = p.passes == 1 ? 0 : static_cast<int>(quotient(at - base, each));
            const int64_t tile_base = base + static_cast<int64_t>(pass) * each;
            const int64_t a = at - tile_base - p.overhead, e = to - tile_base - p.overhead;
            const int j0 = a < 0 ? 0 : static_cast<int>(a), j1 = e < 0 ? 0 : e > steps ? steps : static_cast<int>(e);
            at = tile_base + each < to ? tile_base + each : to;
            if (j1 <= j0) continue;
            if (j0 == 0 && j1 < steps)
                joint = Joint8{b, pass, static_cast<int>(quotient(tile_base + p.overhead + steps - 1, run)) - unit + 1, tile_base < from ? 0 : 1};
            return Piece{b, row, pass * p.group + rank, j0 * kKeys, j1 * kKeys < len ? j1 * kKeys : len, j1 - j0,
                         j1 - j0 == steps ? -1 : tile_base < from ? 0 : 1};
        }
        // (that was all: what is to join)
        if (lane == 0 && rank == 0) p.joints[unit] = joint;
        return Piece{};
    }
};

// Hands the pieces to the other warps: piece `i` of the CTA.  Whole warp; false: a wait failed.
template <class Shared, class Wait>
__device__ __forceinline__ bool put_piece(Shared* sh, Wait& wait, int i, const Piece& y) {
    if (i >= kAhead && !__all_sync(~0u, wait(&sh->piece_free[i % kAhead], i / kAhead - 1))) return false;
    if ((threadIdx.x & 31) == 0) {
        sh->piece[i % kAhead] = y;
        mbar_arrive(smem_u32(&sh->piece_full[i % kAhead]));
    }
    __syncwarp();
    return true;
}

// Hands `store` (with the step's number in its piece) the exponent bytes of each step's keys, four consecutive keys (of
// one page) to a lane, step after step of the pieces that `next` brings; `begin` is called once per piece before them.
// Whole warp; both return false where a wait failed.
template <class Next, class Begin, class Store>
__device__ __forceinline__ void find_scales(const Attend8& p, const Piece& x, Next& next, Begin begin, Store store) {
    const int lane = threadIdx.x & 31;
    int bits = 0;
    auto look_up = [&](int j) {  // the page of a step's keys, looked at when it is used
        const int key = x.key0 + j * kKeys + lane * 4;
        return j < x.n && key < x.len ? p.table[static_cast<int64_t>(x.row) * p.max_pages + p.by_page(key)] : -1;
    };
    bool ok = true;
    while (ok && next()) {
        int found = look_up(0);
        ok = begin();
        for (int j = 0; j < x.n && ok; ++j) {
            const int page = found, key = x.key0 + j * kKeys + lane * 4;
            found = look_up(j + 1);
            uint32_t four = 0x01010101u * kExpBias;  // (a page outside the cache reads as zeros)
            if (page >= 0 && page < p.c.num_pages) {
                const int in = key - p.by_page(key) * p.c.page_size;
                const uint8_t* const at = p.c.pages + page * p.c.page_bytes + static_cast<int64_t>(p.c.page_size) * p.c.C;
                four = at[p.by_block(in)] | at[p.by_block(in + 1)] << 8 | at[p.by_block(in + 2)] << 16 |
                       static_cast<uint32_t>(at[p.by_block(in + 3)]) << 24;
            } else if (key < x.len) {
                bits = kStatusPageRange;
            }
            ok = store(j, four);
        }
    }
    bits = __reduce_or_sync(~0u, bits);
    if (lane == 0) raise_status(p.status, bits);
}

// A query row (8 columns in each of a lane's three words) as two E4M3 terms on a power of two of its own, by FP16, which
// holds a BF16 value of a row on that scale to 2^-25: put(k, first, second) gets the codes of word k.  Returns the factor
// of the row's scores.  Whole warp.
template <class Put>
__device__ __forceinline__ float split_row(const Attend8& p, const uint4 (&v)[3], Put put) {
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k)
        most = __vmaxu2(__vmaxu2(__vmaxu2(__vmaxu2(most, v[k].x & 0x7fff7fffu), v[k].y & 0x7fff7fffu), v[k].z & 0x7fff7fffu),
                        v[k].w & 0x7fff7fffu);
    const uint32_t top = __reduce_max_sync(~0u, max(most & 0xffffu, most >> 16));
    int e = static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7f) > 0x60);
    e = e < -120 ? -120 : e;
    const uint64_t down = pk2(pow2(-e), pow2(-e));
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float a, b;
            upk2(mul2(pk2(bf16_lo(u[n]), bf16_hi(u[n])), down), a, b);
            split_query(a, b, hi[n], lo[n]);
        }
        put(k, make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16), make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16));
    }
    // (a row with an infinity or a NaN has no weights: inf - inf)
    // (never 0: a masked key's -inf times it stays -inf)
    return top < 0x7f80u ? fmaxf(p.scale * kLog2e * pow2(e), 1.2e-38f) : NAN;
}

// Launches the kernel of CTA pairs (attend_cache8_pair.cu).
cudaError_t launch_attend8_pair(const CUtensorMap& rows, const CUtensorMap& rest, const CUtensorMap& k, const CUtensorMap& v, const Attend8& p,
                                cudaStream_t st);
constexpr int kPairQBytes = 2 * 64 * 576;

}  // namespace mlap
