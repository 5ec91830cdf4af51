// tree_kernel.cuh -- attention of trees of drafted tokens over the paged K/V cache, on the tcgen05
// tensor cores.
//
// A sequence holds ctx cached tokens and n drafted ones behind them.  Drafted token j sees the whole
// context and the drafted tokens k whose bit is set in its mask:
//     out[j, h] = sum_t softmax_t(scale * q[j, h] . K_t) V_t,  t < ctx, or t = ctx + k with bit k of mask[j],
// K_t and V_t of KV head h / G.  The tokens of a tree times the G heads of a KV head are the rows of one
// dense contraction over the same keys: each key is read once for all of them.
//
// GB300 design (times of 64 sequences of 8K tokens x 256 rows are of a build with weights rounded once, those between 437 and
// 470 us with loads shared by two CTAs as well; both sides of a choice are always of one build):
//  * A unit is up to NR query rows (32, 64 or 128) of one sequence and KV head over its keys, in tiles of BN keys (128;
//    64 at head_dim 256).  S = Q K^T is one M = 128 product whatever NR is: the tile holds 128 / NR copies of the rows, and
//    each copy takes its own share of the tile's keys.  So 128 threads (one a row of the tile, a TMEM lane each) share the
//    softmax of few rows without exchanging anything: a copy is a split of the keys with a maximum and a sum of its own,
//    and the copies are joined once, at the unit's end.  The weights go back to TMEM as the A operand of O += P V, with zeros
//    in the columns of the other copies' keys.  The least NR that holds the rows:
//    16 rows in the 32 / 64 / 128-row kernels, 256 sequences of 50..650 tokens 100 / 129 / 127 us, 64 of 100..4096 96 / 98 / 97, one of
//    1000 12.0 / 14.0 / 14.4, 64 at 64 columns 66 / 72 / 79.
//  * At 128 rows two threads share a row, half a tile's keys each (one thread a row, or four in 80 registers each, with weights
//    rounded once: 64 sequences of 8K tokens x 256 rows 553 / 521, two 456 us).  They keep one reference, by a vote of the
//    row's two warps a tile (a reference and an accumulator for each, in two buffers: 128 rows 104 -> 113 us; a vote that is cast
//    before the remainders' arithmetic and read behind it: 109).
//  * K and V arrive by TMA in boxes of 16 tokens (8 in blocks of 8) x 64 columns, 128-byte swizzled, in two rings of whole
//    tiles; K is released by its product, V by its own.  QK and PV have an issuer each.  (Boxes of 64 tokens: no faster.
//    A third V tile beside three of K takes the L1 that block tables and masks need; 2 K and 3 V tiles 1..2 % faster than 3
//    and 2, 256 rows 335..341 us to 341..346.  Tiles prefetched into L2: 328 -> 360 us.)
//  * The running maximum is lazy: weights are taken against the old one, and only where their sum over a thread's keys
//    exceeds 2^8 are the maximum raised (to a whole power of two) and O and l rescaled.  Weights up to 2^8 are exact in
//    fp32; in fp16, where they are scaled by 2^7, their sum of up to 2^15 is half of what the format holds.
//  * A weight enters the second product as its value rounded to the cache's type and the remainder rounded likewise (16 bits
//    in bf16, 22 in fp16), two instructions on the same V rows, as in the chunks' kernel; l sums the unrounded weights and
//    everything else is fp32.  In fp16 weights are scaled by 2^7, so that small ones are not subnormal.  Both sides
//    measured: root-mean-square error against 64 bits, relative to the output, 0.0016..0.0017 in bf16 and 0.00021 in fp16,
//    which are the output's own rounding (weights rounded once: 0.0023 and 0.00025..0.00029).  Time with remainders / without: 64
//    sequences of 100..4096 tokens at 32 / 64 / 128 rows 96 / 95.7, 100 / 99.4, 104 / 102 us, 256 of 50..650 100 / 102, 64 of
//    1K..8K at 256 rows 325 / 299 (without: before the code was shortened, below).
//  * Weights lie over the scores that they come from: the remainders double what is handed over, and scores and weights with
//    places of their own leave room for one buffer of weights (32 / 128 rows: 97.3 / 119, 256 short ones 116).
//  * All units laid end to end and measured in cost (a unit's start and output, then its tiles) are cut into equal ranges,
//    one a CTA; units that a range's end cuts leave fp32 partials which tree_merge_kernel joins in a fixed order.  No
//    host-side lengths, no atomics, two partials a CTA.  One thread of a CTA walks its range and tells the other warps the
//    segments through a ring (each warp walking on its own, 4 KB of code in each that runs once a unit: 256 sequences of
//    50..650 tokens 127 us instead of 99, 64 of 100..4096 104 instead of 95, x 256 rows 277 instead of 265).
//  * Trees of more than 128 rows are `group` blocks of tokens (further ones in further passes), worked by CTAs next to each
//    other that walk the same keys at the same time, each loading them for itself: all but the first find them in L2.  A
//    CTA passes over the sequences in which its block has no rows.  (One load for two blocks, sent to both CTAs of a
//    cluster, took 437 us where this takes 492, 64 sequences of 8K tokens x 256 rows.  It is not used: a cache may lie in
//    memory of another GPU, where such loads are not safe.)
//  * The cache rows of drafted tokens that some row does not see may hold anything (a padded token's row was never
//    written): scores are replaced before the softmax, and a warp of its own looks at the drafted V rows before their
//    product: one that is not finite is zeroed in shared memory, the rows that see it becoming NaN.
//  * A successful wait on a barrier costs ~200 cycles of a warp that does nothing else, so the softmax looks at the next
//    tile's barriers while this one's weights are under way (493 -> 463 us at 256 rows).  A thread reads all its scores of a
//    tile at once (64 in two parts: 494 instead of 450); tiles of context alone have a loop of their own without a test
//    (64 columns 66 us, 256 rows 324; with one loop 72 and 335).
//  * The kernels are 90..110 KB of code and sensitive to its size and place: 100 instructions that never run, in front of the
//    loaders' loop, cost 11 % at 128 rows and more (110 -> 123 us; 256 rows 365 -> 412).  So what stands at every wait and
//    every division is kept short, and loops that run once a unit are not unrolled (125 -> 111 KB: 128 rows 111 -> 104,
//    256 rows 366 -> 327, 256 sequences of 50..650 tokens 111 -> 100).
//  * Waits have a time limit; on expiry PA_DEVERR_TIMEOUT is set, the warps that load or issue products stop there, and the
//    others go on without waiting, so that every barrier of the block is still met.  Loads and products under way are
//    waited for (again with the limit); the results are not used.
//  * No wait can be overtaken: a barrier two phases on looks like one that is not complete.  So what a warp waits for goes
//    on only after that warp has arrived at something that it needs: every V tile passes the scanner on its way to the
//    product, the softmax looks at the scanner's barrier before it hands over the tile's weights, and a score buffer is written
//    again only when the product of its weights is complete.  (Tiles without
//    drafted tokens straight to the product, released by the scanner as well: 256 rows x 8K 551 us instead of 450.)
//
// What bounds it: memory up to 128 rows, 6.4..6.8 TB/s between the starts and ends of units (a tile of 64 KB in ~2800
// cycles; DRAM traffic 1.00 x the keys' bytes).  At 256 rows the products (three of 512 cycles at best a tile, the tensor pipe 64 %
// busy) and the softmax beside them: of 363 us for 64 x 1K..8K the remainders' product takes 49, their arithmetic 50, the
// vote of a row's warps 28 (each left out alone); in a row of calls the chip's power limit lowers the clock, 330 -> 360.  Fixed: ~4
// us to the first weights, 1.5..2.3 us a unit that the rings do not cover (the last product, the join, the first tile's
// maximum), ~3 us of merge.  Whole calls (GB300, in a graph): 64 sequences of 100..4096 tokens, 16 drafted, 16 q / 8 KV heads
// 94..96 us (83 us of bytes at the copy rate), 4 x 30K..32K 90..92 (76), 64 x 1K..8K, 64 drafted, 32 q heads 325..365 (190), 256 x
// 50..650 100 (61), one of 100 9.1.
#pragma once

#include <type_traits>

#include "pa_launch.h"
#include "tcgen05.cuh"

namespace pa {
namespace tree {

template <bool BF16>
constexpr float kShift = BF16 ? 0.f : 7.f;

constexpr int MERGE_THREADS = 256;
static_assert(PA_TREE_MAX_CTAS <= MERGE_THREADS, "the merge gives every partial of a unit a thread");

template <int D, int NR>
struct Cfg {
    static_assert(D == 64 || D == 128 || D == 256, "head_dim of the kernel");
    static_assert(NR == 32 || NR == 64 || NR == 128, "query rows of a unit");
    static constexpr int BN = D == 256 ? 64 : 128;      // keys per tile
    static constexpr int COPIES = 128 / NR;
    static constexpr int SPLIT = NR < 128 ? 1 : 2;  // threads a row of the tile
    static constexpr int KW = BN / COPIES / SPLIT;      // keys of a tile that one thread takes
    static constexpr int SOFTMAX = 4 * SPLIT;           // softmax warps; then the issuers, the Q loader, two K and two V loaders, the V scanner
    static constexpr int QK_WARP = SOFTMAX, PV_WARP = SOFTMAX + 1, Q_WARP = SOFTMAX + 2, K_WARP = SOFTMAX + 3,
                         V_WARP = SOFTMAX + 5, CHECK_WARP = SOFTMAX + 7, THREADS = (SOFTMAX + 8) * 32;
    // registers a thread: launched with as many as fit (a multiple of 8), then split
    static constexpr int REGS = 65536 / THREADS / 8 * 8, REGS_OTHERS = 96, REGS_SOFTMAX = SPLIT > 1 ? 160 : 232;
    static_assert(32 * SOFTMAX * REGS_SOFTMAX + (THREADS - 32 * SOFTMAX) * REGS_OTHERS <= THREADS * REGS, "the split exceeds the launch");
    static constexpr int NS = 3;                        // score buffers
    static constexpr int SLABS = D / 64;
    static constexpr int QSLAB = 128 * 128, KSLAB = BN * 128;
    static constexpr int TILE = SLABS * KSLAB;          // bytes of K (or V) of a tile
    // The output passes through a place of its own where there is one (the copies are joined there in fp32; at 128 rows it is
    // turned there, in 16 bits, so that rows are written whole), while the next unit's Q loads; at D 256 there is none: the
    // copies are joined in the Q tile's, 128 rows are written as they stand.  Tiles in the rings: what fits beside that
    static constexpr bool OWN_STAGE = D < 256;
    static constexpr int NK = D == 64 ? 6 : 2, NV = D == 64 ? 6 : 3;
    static constexpr int SEGS = D == 64 ? 6 : 8, READERS = SOFTMAX + 7;  // segments told ahead; warps that are told
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = SLABS * QSLAB, V_OFF = K_OFF + NK * TILE;
    static constexpr int STAGE_OFF = OWN_STAGE ? V_OFF + NV * TILE : Q_OFF;
    static constexpr int ML_OFF = V_OFF + NV * TILE + (OWN_STAGE ? NR * D * (COPIES > 1 ? 4 : 2) : 0);  // what a row's threads tell each other
    static constexpr int BAR_OFF = ML_OFF + (SPLIT > 2 ? SPLIT : 2) * 128 * 4;
    static constexpr int K_FULL = 0, K_EMPTY = NK, V_FULL = 2 * NK, V_EMPTY = V_FULL + NV, V_OK = V_EMPTY + NV, Q_FULL = V_OK + NV, Q_EMPTY = Q_FULL + 1,
                         S_FULL = Q_FULL + 2, P_FULL = S_FULL + NS, PV_DONE = P_FULL + NS,
                         O_FREE = PV_DONE + NS, DRAIN = O_FREE + 1, SEG_FULL = DRAIN + 2, SEG_EMPTY = SEG_FULL + SEGS, NUM_BARS = SEG_EMPTY + SEGS;
    static constexpr int MISC_OFF = (BAR_OFF + NUM_BARS * 8 + 15) & ~15;  // start record, TMEM address, scan scratch
    static constexpr int BAD_OFF = MISC_OFF + 192;                       // the V ring's rows that are not finite: a bit a row
    static constexpr int SEG_OFF = BAD_OFF + NV * 16;                    // the ring of segments
    static constexpr int SMEM_BYTES = SEG_OFF + SEGS * 48 + 1024;        // + alignment slack
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
    static_assert(COPIES == 1 || OWN_STAGE || NR * D * 4 <= SLABS * QSLAB, "the copies are joined in the Q tile's place");
    // TMEM: three S buffers and O.  A weight takes as many columns as a score, 16 bits and its remainder's 16: a thread writes
    // them over the scores that it has read
    static constexpr uint32_t S2_COL = D == 256 ? 128 : 384, O_COL = 256, TMEM_COLS = 512;
    static_assert(2 * BN <= (int)O_COL && (D == 256 ? S2_COL + BN <= O_COL : O_COL + D <= S2_COL && S2_COL + BN <= TMEM_COLS), "columns");
    static __device__ __forceinline__ uint32_t s_col(int b) { return b < 2 ? (uint32_t)(b * BN) : S2_COL; }
};

__device__ __forceinline__ void mma_ss(uint32_t el, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t el, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t el, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(el)
        : "memory");
}
__device__ __forceinline__ void tma_box(uint32_t el, uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                        uint32_t bar, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %8, 0;\n\t"
        "@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar), "l"(policy), "r"(el)
        : "memory");
}
__device__ __forceinline__ void tma_q(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ uint64_t l2_policy_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// barrier of N threads, plain and with an OR over them: 1: all softmax warps; 2 + q: the two warps of lanes 32 q .. 32 q + 31
template <int N>
__device__ __forceinline__ void bar_sync(int id) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ bool bar_or(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id), "n"(N)
        : "memory");
    return r != 0;
}

// Branches that few tiles take: their code is laid out of the others' way.
__device__ __forceinline__ bool rare(bool v) { return __builtin_expect(v, 0); }

// Waits, with the limit of all waits (few instructions: it stands at every wait).
__device__ __forceinline__ bool wait_limited(uint32_t bar, uint32_t parity, unsigned* err) {
    uint32_t t0, t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t0));
    bool done;
    do {
        done = mbar_try_wait(bar, parity);
        asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    } while (!done && t - t0 < (uint32_t)kWaitLimitNs);
    if (!done) flag_error(err, PA_DEVERR_TIMEOUT);
    return done;
}
// The warp waits; the polling loop stays out of line.  One result for the warp.
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, unsigned* err) {
    return __all_sync(0xffffffffu, wait_limited(bar, parity, err));
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, unsigned* err) {
    if (rare(__any_sync(0xffffffffu, !mbar_try_wait(bar, parity)))) return wait_slow(bar, parity, err);
    return true;
}

// whether a phase is complete, without waiting
__device__ __forceinline__ bool mbar_test(uint32_t bar, int phase) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"((uint32_t)(phase & 1))
        : "memory");
    return ok != 0;
}

// 0 * v + z for pairs of 16-bit values
template <bool BF16>
__device__ __forceinline__ uint32_t zero_times(uint32_t v, uint32_t z) {
    uint32_t d;
    if constexpr (BF16) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(0u), "r"(z));
    else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(0u), "r"(z));
    return d;
}

template <int N>
__device__ __forceinline__ void ldn(uint32_t taddr, uint32_t (&r)[N]) {
    if constexpr (N == 16) tc::ld16(taddr, r);
    else if constexpr (N == 32) tc::ld32(taddr, r);
    else tc::ld64(taddr, r);
}
template <int N>
__device__ __forceinline__ void stn(uint32_t taddr, const uint32_t (&r)[N]) {
    if constexpr (N == 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                     "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    else if constexpr (N == 16) tc::st16(taddr, r);
    else tc::st32(taddr, r);
}

// ---- the split of all units' tiles over the CTAs ---------------------------------------------

// A sequence: its first query row (token), drafted tokens and keys.  Lengths out of range: it is skipped.
struct Seq {
    int q0, n, kv_len;
    bool bad;
};
__device__ __forceinline__ Seq load_seq(const TreeParams& p, int s) {
    Seq k;
    k.kv_len = ld_global(p.kv_lens + s);
    k.q0 = ld_global(p.q_loc + s);
    const int q1 = ld_global(p.q_loc + s + 1);
    k.n = q1 - k.q0;
    k.bad = k.q0 < 0 || q1 < k.q0 || q1 > p.total_q || k.n > p.max_q_len || k.kv_len < k.n ||
            k.kv_len > p.max_blocks_per_seq * p.block_size;
    if (k.bad) k.n = 0;
    return k;
}

// A sequence's units: its KV heads times the passes over its blocks of tokens, `cost` each (its start and its
// output count unit_cost tiles).  A pass is p.group blocks, one for each CTA of a group.
__device__ __forceinline__ int tiles_of(const TreeParams& p, const Seq& k) { return (k.kv_len + (1 << p.tile_log2) - 1) >> p.tile_log2; }
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// ceil(n / d), n >= 0, d > 0 and a result of at most 21 bits: the estimate, right to 2^-22, is off by one at most
__device__ __forceinline__ int ceil_div(int n, int d) {
    const int q = (int)((float)n * rcp((float)d)), rest = n - q * d;
    return q + (rest > 0 ? 1 : 0) + (rest > d ? 1 : 0) - (rest <= -d ? 1 : 0);
}
// n / d and n mod d, n >= 0 and d > 0: of 22 bits from an estimate
__device__ __forceinline__ long long quotient(long long n, int d, int& rest) {
    const float r = rcp((float)d);
    if (n < 1 << 22) {
        const int m = (int)n, q = (int)((float)m * r);
        rest = m - q * d;
        const int off = rest < 0 ? -1 : rest >= d ? 1 : 0;
        rest -= off * d;
        return q + off;
    }
    const long long q = n / d;
    rest = (int)(n - q * d);
    return q;
}
__device__ __forceinline__ int passes_of(const TreeParams& p, const Seq& k) {
    const int per = p.tb * p.group;
    return k.n > per ? ceil_div(k.n, per) : k.n > 0;
}

// A range: where it starts (sequence, cost into its units) and its cost.
struct Start {
    long long at;
    int s, q0, n, kv_len, per;  // per 0: nothing
};
static_assert(sizeof(Start) <= 32, "record area");

__device__ __forceinline__ long long cost_of(const TreeParams& p, const Seq& k) {
    return (long long)p.n_kv_heads * passes_of(p, k) * (tiles_of(p, k) + p.unit_cost);
}
__device__ __forceinline__ long long prefix(long long v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}
__device__ __forceinline__ int cost_of_range(const TreeParams& p, long long total, int ranges) {
    int rest;
    return (int)max(quotient(total + ranges - 1, ranges, rest), (long long)p.min_tiles);
}

// Range `range` of `ranges` equal ones.  Up to kWarpSeqs sequences: by a warp, two a lane; the result is the first lane's.
// (By the block: one sequence of 100 tokens 10.5 us instead of 9.5, eight of 500 14.1 instead of 13.4.)
constexpr int kWarpSeqs = 64;
__device__ __forceinline__ Start find_start_warp(const TreeParams& p, int range, int ranges, int lane) {
    Seq k[2] = {{0, 0, 0, false}, {0, 0, 0, false}};
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (2 * lane + j < p.num_seqs) k[j] = load_seq(p, 2 * lane + j);
    if ((k[0].bad || k[1].bad) && blockIdx.x == 0) flag_error(p.err, PA_DEVERR_LENGTH);
    const long long c0 = cost_of(p, k[0]), c = c0 + cost_of(p, k[1]), incl = prefix(c, lane);
    Start r;
    r.per = cost_of_range(p, __shfl_sync(0xffffffffu, incl, 31), ranges);
    const long long lo = (long long)range * r.per, into = lo - (incl - c);
    const unsigned at = __ballot_sync(0xffffffffu, lo < incl);  // the first of these lanes holds it
    const bool second = into >= c0;
    const int from = __ffs(at) - 1;
    if (at == 0u) r.per = 0;
    r.at = __shfl_sync(0xffffffffu, second ? into - c0 : into, from & 31);
    r.s = __shfl_sync(0xffffffffu, 2 * lane + second, from & 31);
    r.q0 = __shfl_sync(0xffffffffu, second ? k[1].q0 : k[0].q0, from & 31);
    r.n = __shfl_sync(0xffffffffu, second ? k[1].n : k[0].n, from & 31);
    r.kv_len = __shfl_sync(0xffffffffu, second ? k[1].kv_len : k[0].kv_len, from & 31);
    return r;
}

// More: by all THREADS threads of the block.  (Then the CTA is synchronised.)
template <int THREADS>
__device__ __forceinline__ void find_start(const TreeParams& p, int range, int ranges, volatile long long* warp_sum, Start* rec) {
    constexpr int NW = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) rec->per = 0;
    Seq k{0, 0, 0, false};
    long long mine = 0;
#pragma unroll 1
    for (int s = tid; s < p.num_seqs; s += THREADS) {
        k = load_seq(p, s);
        if (k.bad && blockIdx.x == 0) flag_error(p.err, PA_DEVERR_LENGTH);
        mine += cost_of(p, k);
    }
    mine = prefix(mine, lane);
    if (lane == 31) warp_sum[warp] = mine;
    __syncthreads();
    long long total = 0;
#pragma unroll 1
    for (int w = 0; w < NW; ++w) total += warp_sum[w];
    const int per = cost_of_range(p, total, ranges);
    const long long lo = (long long)range * per;
    if (lo < total) {
        // the sequence that holds it: by prefix sums, THREADS sequences at a time
        long long base = 0;
#pragma unroll 1
        for (int s0 = 0; s0 < p.num_seqs && base <= lo; s0 += THREADS) {
            const int s = s0 + tid;
            long long cost = 0;
            if (s < p.num_seqs) {
                k = load_seq(p, s);
                cost = cost_of(p, k);
            }
            const long long incl = prefix(cost, lane);
            __syncthreads();
            if (lane == 31) warp_sum[warp] = incl;
            __syncthreads();
            long long before = base;
#pragma unroll 1
            for (int w = 0; w < NW; ++w) {
                const long long x = warp_sum[w];
                if (w < warp) before += x;
                base += x;
            }
            const long long from = before + incl - cost;
            if (cost > 0 && lo >= from && lo < from + cost) {
                rec->s = s;
                rec->at = lo - from;
                rec->q0 = k.q0;
                rec->n = k.n;
                rec->kv_len = k.kv_len;
                rec->per = per;
            }
        }
    }
    __syncthreads();
}

// One segment of a range: tiles [tile, tile + n) of one unit's.  n == 0: there are no more.
struct Segment {
    int s, head, tok0, toks;  // sequence, KV head, the unit's first token (of total_q) and tokens
    int q0;                   // the sequence's first token
    int tile, n;
    int ctx, keys, drafted;
    int parts, back;          // ranges the unit's tiles span (0: this one alone), and how many of them are before this one
};
static_assert(sizeof(Segment) == 48, "three 16-byte words");

// The segments of the CTA's range in which it has rows: a block of each pass, `blk` further on (of p.group) with every
// sequence and head, so that those of few drafted tokens, which have rows in the first block alone, are dealt out over the group's
// CTAs (64 sequences of 100..4096 tokens, every eighth with 200 drafted ones, the others with one: 365 us; 520 without).
struct Walk {
    const TreeParams& p;
    Seq k;
    int s, head, pass, passes, at, left, per, blk;  // `at`: cost into the unit
    __device__ __forceinline__ Walk(const TreeParams& p_, const Start& st, int blk_)
        : p(p_), k{st.q0, st.n, st.kv_len, false}, s(st.s), head(0), pass(0), passes(1), at(0), left(st.per), per(st.per), blk(blk_) {
        if (left <= 0) return;
        passes = passes_of(p, k);
        const int unit = (int)quotient(st.at, tiles_of(p, k) + p.unit_cost, at);
        head = unit;
        if (passes > 1) head = (int)quotient(unit, passes, pass);
    }
    // the next one
    __device__ __forceinline__ void next(Segment& g) {
        g.n = 0;
        while (left > 0) {
            const int tiles = tiles_of(p, k);
            const int cost = min(tiles + p.unit_cost - at, left);  // of the unit in this range
            left -= cost;
            g.tile = max(0, at - p.unit_cost);
            g.n = max(0, at + cost - p.unit_cost) - g.tile;
            const int rest = tiles - g.tile - g.n;
            g.back = g.tile > 0 ? ceil_div(g.tile, per) : 0;
            g.parts = (g.tile > 0 || rest > 0) ? g.back + 1 + (rest > 0 ? ceil_div(rest, per) : 0) : 0;
            g.s = s;
            g.head = head;
            int j = pass * p.group + blk;
            if (p.group > 1) j = pass * p.group + (int)(((uint32_t)s * (uint32_t)p.n_kv_heads + (uint32_t)(head + blk)) % (uint32_t)p.group);
            g.tok0 = k.q0 + j * p.tb;
            g.q0 = k.q0;
            g.toks = max(0, min(p.tb, k.n - j * p.tb));
            g.ctx = k.kv_len - k.n;
            g.keys = k.kv_len;
            g.drafted = k.n;
            at = 0;
            if (left > 0 && ++pass == passes) {
                pass = 0;
                if (++head == p.n_kv_heads) {
                    head = 0;
                    do {
                        if (++s >= p.num_seqs) left = 0;
                        else k = load_seq(p, s);
                    } while (left > 0 && k.n == 0);
                    passes = passes_of(p, k);
                }
            }
            if (g.n > 0 && g.toks > 0) return;
            g.n = 0;
        }
    }
};

// Bits k0 .. k0 + 31 (keys) that a row sees: the context, and the drafted tokens of its mask words (32-bit ones here).
__device__ __forceinline__ uint32_t sees32(const uint32_t* row, int words, int k0, int ctx, int drafted) {
    const int rel = k0 - ctx;
    if (rel <= -32) return 0xffffffffu;
    const int b = max(rel, 0), left = drafted - b;
    uint32_t w = 0;
    if (left > 0) {
        const int i = b >> 5;
        const uint32_t lo = i < words ? ld_global(row + i) : 0u, hi = (b & 31) && i + 1 < words ? ld_global(row + i + 1) : 0u;
        w = __funnelshift_r(lo, hi, b & 31);
        if (left < 32) w &= (1u << left) - 1u;
    }
    return rel < 0 ? (w << -rel) | ((1u << -rel) - 1u) : w;
}

}  // namespace tree

template <bool BF16, int D, int NR>
__global__ void __launch_bounds__(tree::Cfg<D, NR>::THREADS, 1)
tree_kernel(const TreeParams p, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
            const __grid_constant__ CUtensorMap tmQ) {
    using namespace tree;
    using C = Cfg<D, NR>;
    using F = F16x2<BF16>;
    constexpr int BN = C::BN, KW = C::KW, NS = C::NS, COPIES = C::COPIES, SPLIT = C::SPLIT, SOFTMAX = C::SOFTMAX;
    constexpr int QK_WARP = C::QK_WARP, PV_WARP = C::PV_WARP, Q_WARP = C::Q_WARP, K_WARP = C::K_WARP, V_WARP = C::V_WARP;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_addr(smem);
    const uint32_t sStage = sbase + C::STAGE_OFF, sQ = sbase + C::Q_OFF, sK = sbase + C::K_OFF, sV = sbase + C::V_OFF, bars = sbase + C::BAR_OFF;
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    Start* rec = reinterpret_cast<Start*>(smem + C::MISC_OFF);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::MISC_OFF + 32);
    volatile uint32_t* bad_keys = reinterpret_cast<volatile uint32_t*>(smem + C::BAD_OFF);  // [NV][4]
    long long* warp_sum = reinterpret_cast<long long*>(smem + C::MISC_OFF + 64);
    float* m_s = reinterpret_cast<float*>(smem + C::ML_OFF);
    float* l_s = m_s + 128;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int range = (int)blockIdx.x / p.group, blk = (int)blockIdx.x % p.group;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NK; ++i) {
            mbar_init(bar(C::K_FULL + i), 2);
            mbar_init(bar(C::K_EMPTY + i), 1);
        }
        for (int i = 0; i < C::NV; ++i) {
            mbar_init(bar(C::V_FULL + i), 2);
            mbar_init(bar(C::V_EMPTY + i), 1);
            mbar_init(bar(C::V_OK + i), 1);
        }
        mbar_init(bar(C::Q_FULL), 1);
        mbar_init(bar(C::Q_EMPTY), COPIES > 1 && !C::OWN_STAGE ? 1 + SOFTMAX : 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(bar(C::S_FULL + i), 1);
            mbar_init(bar(C::P_FULL + i), SOFTMAX);
            mbar_init(bar(C::PV_DONE + i), 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(bar(C::DRAIN + i), 1);
        mbar_init(bar(C::O_FREE), SOFTMAX);
        for (int i = 0; i < C::SEGS; ++i) {
            mbar_init(bar(C::SEG_FULL + i), 1);
            mbar_init(bar(C::SEG_EMPTY + i), C::READERS);
        }
        fence_barrier_init();
    }
    if (warp == QK_WARP) {
        tc::alloc(smem_addr(const_cast<uint32_t*>(tmem_slot)), C::TMEM_COLS);
        tc::relinquish();
    }
    // a programmatic dependent of the kernel before it: nothing is read before that one is complete; the merge may be
    // set up now (it waits for this grid before it reads)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc::fence_before();
    const bool by_warp = p.num_seqs <= kWarpSeqs;
    if (by_warp) __syncthreads();
    else find_start<C::THREADS>(p, range, (int)gridDim.x / p.group, warp_sum, rec);
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;  // none of this warp's waits has run out
    auto wait = [&](int b, int phase) {
        if (ok) ok = warp_wait(bar(b), (uint32_t)(phase & 1), p.err);
    };
    // segment number j, as the walking thread told it; false: there is none, or a wait has run out
    auto segment = [&](int j, Segment& g) {
        wait(C::SEG_FULL + j % C::SEGS, j / C::SEGS);
        if (!ok) return false;
        const uint32_t at = sbase + C::SEG_OFF + (uint32_t)(j % C::SEGS) * 48u;
        const uint4 a = lds128(at), b = lds128(at + 16), c = lds128(at + 32);
        g.s = (int)a.x, g.head = (int)a.y, g.tok0 = (int)a.z, g.toks = (int)a.w;
        g.q0 = (int)b.x, g.tile = (int)b.y, g.n = (int)b.z, g.ctx = (int)b.w;
        g.keys = (int)c.x, g.drafted = (int)c.y, g.parts = (int)c.z, g.back = (int)c.w;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::SEG_EMPTY + j % C::SEGS));
        return g.n > 0;
    };
    int slot = 0, use = 0;  // loader warps: the next tile's slot of the ring, and how often it has been filled
    // token of a unit's row, row / g_heads (exact for rows below 128 and up to 16 heads)
    auto row_token = [&](int row) { return (int)(((uint32_t)row * (uint32_t)p.g_magic) >> 16); };
    int4 begins = make_int4(0, 0, 0, 0), goes_on = begins;  // the units cut at the range's end and at its start

    // registers from the warps that move data to those that compute (a thread of 64 keys holds as many scores and as many
    // weights: without, 128 rows of 100..4096 tokens 119 us instead of 111)
    if (warp < SOFTMAX) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHERS));
    if (warp < SOFTMAX) {
        // ------------------------------------------------------------ softmax, rescale, epilogue
        // row of the tile; of the unit; which copy of it, or which of its two threads (its share of a tile's keys)
        const int quarter = warp & 3, R = 32 * quarter + lane, share = SPLIT > 1 ? warp >> 2 : COPIES == 1 ? 0 : (32 * warp) / NR;
        const int r = SPLIT > 1 ? R : R - share * NR;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_base + (uint32_t)(share * KW), tO = tmem + lane_base + C::O_COL;
        // the threads of a row share its reference: what one finds the others have to know
        auto row_or = [&](bool v) {
            if constexpr (SPLIT > 1) return bar_or<32 * SPLIT>(2 + quarter, v);
            else return __any_sync(0xffffffffu, v) != 0;
        };
        // (scale 0: all scores that are seen count the same, as with the smallest scale)
        const float sc = p.qk_scale_log2 != 0.f ? p.qk_scale_log2 : 0x1p-126f;
        const uint32_t unseen = sc > 0.f ? 0xFF800000u : 0x7F800000u;  // -inf, +inf
        constexpr float kMost = BF16 ? 0x1p8f : 0x1p15f;  // 2^(8 + kShift)
        const int tok_r = row_token(r);
        bool ready = false;  // the next tile's barriers were seen complete
        int i = 0;  // tile number over the CTA's range
        constexpr int MW = (KW + 31) / 32;
        Segment g;
        // (a wait that ran out ends all of these warps' loops at the same segment: they meet at barriers inside)
        for (int seg = 0; !bar_or<32 * SOFTMAX>(6, !segment(seg, g)); ++seg) {
            const int rows = g.toks * p.g_heads;
            const bool valid = r < rows;
            const uint32_t* mask = reinterpret_cast<const uint32_t*>(p.mask + (size_t)(valid ? g.tok0 + tok_r : g.q0) * p.mask_words);
            // which keys of tile `tile` the row sees (bits of this thread's); loaded a tile ahead
            auto row_sees = [&](int tile, uint32_t (&w)[MW]) {
#pragma unroll
                for (int x = 0; x < MW; ++x)
                    w[x] = sees32(mask, 2 * p.mask_words, tile * BN + share * KW + 32 * x, g.ctx, g.drafted);
            };
            uint32_t sees[MW], sees_next[MW];
            float m_ref = -INFINITY, l = 0.f;
            bool fresh = true;  // a row may be without a reference
            // tiles of context alone, then those that hold drafted tokens or keys past them
            const int plain = max(0, min(g.n, g.ctx / BN - g.tile));
            if (plain < g.n) row_sees(g.tile + plain, sees_next);
            int u = 0;
            auto step = [&](auto with_drafts) {
                constexpr bool DRAFTS = decltype(with_drafts)::value;
                const int b = i % NS, before = (i + NS - 1) % NS, next = (i + 1) % NS;
                if (rare(!__all_sync(0xffffffffu, ready))) wait(C::S_FULL + b, i / NS);
                tc::fence_after();
                const uint32_t tSb = tS + C::s_col(b);
                if constexpr (COPIES > 1) {  // no weights of the other copies' keys
                    constexpr int Z = KW < 32 ? KW : 32;
                    uint32_t z[Z];
#pragma unroll
                    for (int e = 0; e < Z; ++e) z[e] = 0u;
#pragma unroll
                    for (int c = Z; c < BN; c += Z)
                        if (KW <= Z || c >= KW) stn<Z>(tmem + lane_base + C::s_col(b) + (uint32_t)((share * KW + c) & (BN - 1)), z);
                }
                float add = 0.f;
                uint32_t w[KW / 2], rem[KW / 2];
                // this thread's scores; those of keys that the row does not see, where the tile holds such keys, become what the
                // scale turns into -inf
                auto scores = [&](uint32_t (&x)[KW]) {
                    ldn<KW>(tSb, x);
                    tc::wait_ld();
                    if constexpr (DRAFTS) {
#pragma unroll
                        for (int e = 0; e < KW; ++e)
                            if (!((sees[e / 32] >> (e & 31)) & 1u)) x[e] = unseen;
                    }
                };
                bool raise = fresh, raised = false;
#pragma unroll 1
                for (;;) {
                    if (rare(raise)) {
                        uint32_t x[KW];
                        scores(x);
                        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int e = 0; e < KW; ++e) m4[e & 3] = fmaxf(m4[e & 3], __uint_as_float(x[e]) * sc);
                        float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                        if constexpr (SPLIT > 1) {
                            m_s[128 * share + R] = mx;
                            bar_sync<32 * SPLIT>(2 + quarter);
#pragma unroll
                            for (int k = 0; k < SPLIT; ++k) mx = fmaxf(mx, m_s[128 * k + R]);
                        }
                        const float mt = ceilf(mx);
                        float alpha = 1.f;
                        if (valid && mt > m_ref) {
                            alpha = m_ref == -INFINITY ? 1.f : ex2(m_ref - mt);
                            m_ref = mt;
                            l *= alpha;
                        }
                        fresh = __any_sync(0xffffffffu, valid && m_ref == -INFINITY);
                        if (u > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                            wait(C::PV_DONE + before, (i - 1) / NS);  // O holds every tile before this one
                            tc::fence_after();
#pragma unroll 1
                            for (int q = 0; q < D / 16 / SPLIT; ++q) {  // (each thread of a row its part of the columns)
                                uint32_t o[16];
                                const uint32_t at = tO + (uint32_t)((SPLIT > 1 ? share * (D / SPLIT) : 0) + 16 * q);
                                tc::ld16(at, o);
                                tc::wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tc::st16(at, o);
                            }
                        }
                        raised = true;
                    }
                    const float mu = m_ref == -INFINITY ? 0.f : m_ref - kShift<BF16>;
                    const float2 sc2 = make_float2(sc, sc), nmu2 = make_float2(-mu, -mu);
                    float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    uint32_t x[KW];
                    scores(x);
#pragma unroll
                    for (int e = 0; e < KW / 2; ++e) {
                        float2 v = ffma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), sc2, nmu2);
                        v = make_float2(ex2(v.x), ex2(v.y));
                        ls[e & 1] = fadd2(ls[e & 1], v);
                        w[e] = F::pack_rn(v.x, v.y);
                        v = fsub2(v, F::unpack(w[e]));
                        rem[e] = F::pack_rn(v.x, v.y);
                    }
                    // the next tile's scores, without waiting
                    ready = mbar_test(bar(C::S_FULL + next), (i + 1) / NS);
                    ls[0] = fadd2(ls[0], ls[1]);
                    add = ls[0].x + ls[0].y;
                    // (no weight is above their sum; the vote also says that a row's other thread has read this one's maximum)
                    raise = row_or(valid && add > kMost);
                    if (!rare(raise) || raised) break;
                    // a row outgrew its reference by more than 2^8: once more
                }
                l += add;
                stn<KW / 2>(tSb, w);
                stn<KW / 2>(tSb + KW / 2, rem);
                if constexpr (DRAFTS) {
                    // a drafted V row that is not finite makes the row NaN if it sees it.  (Before the weights are given: the
                    // tile's product releases its slot, and a slot's barrier is not looked at two phases late)
                    wait(C::V_OK + i % C::NV, i / C::NV);
#pragma unroll
                    for (int w = 0; w < MW; ++w) {
                        const int at = share * KW + 32 * w;  // this thread's keys of the tile: KW from share * KW on
                        uint32_t k = bad_keys[4 * (i % C::NV) + (at >> 5)] >> (at & 31);
                        if constexpr (KW < 32) k &= (1u << KW) - 1u;
                        if (k & sees[w]) l = __uint_as_float(0x7FC00000u);
                    }
                }
                tc::wait_st();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::P_FULL + b));  // (the scores have been read, too)
                ++i;
            };
#pragma unroll 1
            for (; u < plain; ++u) step(std::false_type{});
#pragma unroll 1
            for (; u < g.n; ++u) {
#pragma unroll
                for (int w = 0; w < MW; ++w) sees[w] = sees_next[w];
                if (u + 1 < g.n) row_sees(g.tile + u + 1, sees_next);  // a tile ahead
                step(std::true_type{});
            }
            // the segment's end: O / l, or the partial
            const bool whole = g.parts == 0;
            const int slot = 2 * (int)blockIdx.x + (g.tile == 0 ? 1 : 0);
            const size_t row0 = (size_t)g.tok0 * p.n_q_heads + (size_t)g.head * p.g_heads;
            auto product = [&]() {  // the last one; what the row's threads have to tell each other is told before
                wait(C::PV_DONE + (i - 1) % NS, (i - 1) / NS);
                tc::fence_after();
            };
            if constexpr (COPIES == 1) {
                constexpr int W = D / SPLIT, CW = W < 32 ? W : 32;  // columns of this thread, at a time
                const int c0 = share * W;
                uint32_t o[CW];
                auto read_o = [&](int q) {
                    ldn<CW>(tO + (uint32_t)(c0 + CW * q), o);
                    tc::wait_ld();
                    if (q == W / CW - 1) {  // O read: the next segment's first PV may overwrite it
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(C::O_FREE));
                    }
                };
                // the row's sum, in a fixed order
                m_s[128 * share + R] = l;
                bar_sync<32 * SPLIT>(2 + quarter);
                l = 0.f;
#pragma unroll
                for (int k = 0; k < SPLIT; ++k) l += m_s[128 * k + R];
                bar_sync<32 * SPLIT>(2 + quarter);
                const float f = !whole ? 1.f : l != 0.f ? 1.f / l : 0.f;
                if (!whole && valid && share == 0) p.part_ml[(size_t)slot * NR + r] = make_float2(m_ref, l);
                uint16_t* dst = static_cast<uint16_t*>(p.out) + (row0 + (size_t)tok_r * p.n_q_heads + (r - tok_r * p.g_heads)) * p.hd + c0;
                float4* part = p.part_o + ((size_t)slot * (D / 4) + c0 / 4) * NR + r;
                product();
#pragma unroll
                for (int q = 0; q < W / CW; ++q) {
                    read_o(q);
                    if (!whole) {
                        if (valid && ok) {
#pragma unroll
                            for (int v = 0; v < CW / 4; ++v)
                                part[(CW / 4 * q + v) * NR] = make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                                                          __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
                        }
                        continue;
                    }
#pragma unroll
                    for (int v = 0; v < CW / 8; ++v) {
                        const uint4 w = make_uint4(F::pack_rn(__uint_as_float(o[8 * v]) * f, __uint_as_float(o[8 * v + 1]) * f),
                                                   F::pack_rn(__uint_as_float(o[8 * v + 2]) * f, __uint_as_float(o[8 * v + 3]) * f),
                                                   F::pack_rn(__uint_as_float(o[8 * v + 4]) * f, __uint_as_float(o[8 * v + 5]) * f),
                                                   F::pack_rn(__uint_as_float(o[8 * v + 6]) * f, __uint_as_float(o[8 * v + 7]) * f));
                        const int ch = (c0 + CW * q) / 8 + v;
                        if constexpr (C::OWN_STAGE) sts128(sStage + (uint32_t)(R * D * 2 + ((ch ^ (R & 7)) << 4)), w);
                        else if (valid && ok && 8 * ch < p.hd) *reinterpret_cast<uint4*>(dst + CW * q + 8 * v) = w;
                    }
                }
                if constexpr (C::OWN_STAGE) {
                    if (whole) {  // rows of this quarter, whole rows by neighbouring lanes
                        bar_sync<32 * SPLIT>(2 + quarter);
                        constexpr int CH = D / 8, RP = 32 * SPLIT / CH;  // chunks a row, rows at a time
                        const int ch = lane % CH;
#pragma unroll
                        for (int q = 0; q < 32 / RP; ++q) {
                            const int row = 32 * quarter + RP * q + (32 * share + lane) / CH, tok = row_token(row);
                            const uint4 w = lds128(sStage + (uint32_t)(row * D * 2 + ((ch ^ (row & 7)) << 4)));
                            if (row < rows && ok && 8 * ch < p.hd)
                                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) +
                                                          (row0 + (size_t)tok * p.n_q_heads + (row - tok * p.g_heads)) * p.hd + 8 * ch) = w;
                        }
                    }
                }
            } else {
                // join the copies: factors 2^(m - max m), then every copy adds its O, a share of the columns at a time; who adds
                // last has the sum
                m_s[R] = m_ref;
                l_s[R] = l;
                bar_sync<128>(1);
                float mc[COPIES], mx = m_ref, lt = 0.f;
#pragma unroll
                for (int c = 0; c < COPIES; ++c) mx = fmaxf(mx, mc[c] = m_s[c * NR + r]);
#pragma unroll
                for (int c = 0; c < COPIES; ++c) lt = fmaf(l_s[c * NR + r], mc[c] == -INFINITY ? 1.f : ex2(mc[c] - mx), lt);  // (l is 0 there, or NaN)
                float f = m_ref == -INFINITY ? 0.f : ex2(m_ref - mx);
                if (whole) f = lt != 0.f ? f / lt : 0.f;
                else if (valid && share == 0) p.part_ml[(size_t)slot * NR + r] = make_float2(mx, lt);
                constexpr int W = D / COPIES, CW = W < 32 ? W : 32;  // columns of a share, at a time
                const uint32_t srow = sStage + (uint32_t)(r * D * 4);
                uint16_t* dst = static_cast<uint16_t*>(p.out) + (row0 + (size_t)tok_r * p.n_q_heads + (r - tok_r * p.g_heads)) * p.hd;
                float4* part = p.part_o + (size_t)slot * (D / 4) * NR + r;
                product();
#pragma unroll 1
                for (int k = 0; k < COPIES; ++k) {
                    const int c0 = ((share + k) % COPIES) * W;
                    const bool last = k == COPIES - 1;
#pragma unroll 1
                    for (int c = c0; c < c0 + W; c += CW) {
                        uint32_t o[CW];
                        uint4 x[CW / 4];
                        ldn<CW>(tO + (uint32_t)c, o);
#pragma unroll
                        for (int v = 0; v < CW / 4; ++v)
                            x[v] = k > 0 ? lds128(srow + (uint32_t)(((c / 4 + v) ^ (r & 7)) << 4)) : make_uint4(0u, 0u, 0u, 0u);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < CW; ++e) {
                            const uint32_t before = e % 4 == 0 ? x[e / 4].x : e % 4 == 1 ? x[e / 4].y : e % 4 == 2 ? x[e / 4].z : x[e / 4].w;
                            o[e] = __float_as_uint(fmaf(__uint_as_float(o[e]), f, __uint_as_float(before)));
                        }
                        if (!last) {
#pragma unroll
                            for (int v = 0; v < CW / 4; ++v)
                                sts128(srow + (uint32_t)(((c / 4 + v) ^ (r & 7)) << 4), make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]));
                        } else if (!valid || !ok) {
                        } else if (whole) {
#pragma unroll
                            for (int v = 0; v < CW / 8; ++v)
                                if (c + 8 * v < p.hd)
                                    *reinterpret_cast<uint4*>(dst + c + 8 * v) =
                                        make_uint4(F::pack_rn(__uint_as_float(o[8 * v]), __uint_as_float(o[8 * v + 1])),
                                                   F::pack_rn(__uint_as_float(o[8 * v + 2]), __uint_as_float(o[8 * v + 3])),
                                                   F::pack_rn(__uint_as_float(o[8 * v + 4]), __uint_as_float(o[8 * v + 5])),
                                                   F::pack_rn(__uint_as_float(o[8 * v + 6]), __uint_as_float(o[8 * v + 7])));
                        } else {
#pragma unroll
                            for (int v = 0; v < CW / 4; ++v)
                                part[(c / 4 + v) * NR] = make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                                                     __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
                        }
                    }
                    if (last) {  // O read: the next segment's first PV may overwrite it
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(C::O_FREE));
                    } else {
                        bar_sync<128>(1);
                    }
                }
                if constexpr (!C::OWN_STAGE) {
                    tc::fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::Q_EMPTY));
                }
            }
            // what the merge needs to know of a cut unit, from each range that it spans: ranges, rows, first row of out,
            // the CTA it starts in
            if (!whole)
                (g.tile == 0 ? begins : goes_on) = make_int4(g.parts, rows, (int)row0, (int)blockIdx.x - g.back * p.group);
        }
    } else if (warp == C::CHECK_WARP) {
        // ------------------------------------------------------------ V rows of tiles with drafted tokens, before their product:
        // rows past the keys may hold anything (their weights are 0, but 0 * NaN is NaN) and are zeroed, up to the end of the
        // last box that was loaded (the others are zero already); so are drafted rows that are not finite, which are noted
        int i = 0;
        Segment g;
        for (int seg = 0; segment(seg, g); ++seg) {
            for (int u = 0; u < g.n; ++u, ++i) {
                const int kbase = (g.tile + u) * BN, st = i % C::NV;
                wait(C::V_FULL + st, i / C::NV);
                if (!ok) break;
                if (kbase + BN > g.ctx) {
                    volatile uint32_t* bits = bad_keys + 4 * st;
                    const uint32_t tile = sV + (uint32_t)(st * C::TILE);
                    if (lane < 4) bits[lane] = 0u;
                    __syncwarp();
                    // 16 rows at a time, two lanes each: half of its chunks, starting at different banks
                    const int half = lane & 1, d1 = min(BN, g.keys - kbase);
#pragma unroll 1
                    for (int t0 = max(0, g.ctx - kbase); t0 < d1; t0 += 16) {
                        const int t = t0 + (lane >> 1);
                        const uint32_t vrow = tile + (uint32_t)(t * 128);
                        uint32_t z[4] = {0u, 0u, 0u, 0u};  // 0 * v: NaN where v is not finite
                        if (t < d1) {
#pragma unroll 2
                            for (int c = 0; c < C::SLABS * 4; ++c) {
                                const uint4 v = lds128(vrow + (uint32_t)((c >> 2) * C::KSLAB + (((c & 3) + 4 * half + t) & 7) * 16));
                                z[0] = zero_times<BF16>(v.x, z[0]);
                                z[1] = zero_times<BF16>(v.y, z[1]);
                                z[2] = zero_times<BF16>(v.z, z[2]);
                                z[3] = zero_times<BF16>(v.w, z[3]);
                            }
                        }
                        bool bad = ((z[0] | z[1] | z[2] | z[3]) & 0x7FFF7FFFu) != 0u;
                        const uint32_t all = __ballot_sync(0xffffffffu, bad);
                        if (all) {
                            bad = (all >> (lane & ~1) & 3u) != 0u;  // either half
                            if (bad) {
                                if (half == 0) atomicOr(const_cast<uint32_t*>(bits) + (t >> 5), 1u << (t & 31));
                                for (int c = half; c < C::SLABS * 8; c += 2) sts128(vrow + (uint32_t)((c >> 3) * C::KSLAB + (c & 7) * 16), make_uint4(0u, 0u, 0u, 0u));
                            }
                        }
                    }
                    // the rows past the keys, up to the end of the last box
                    const int z1 = min(BN, ((g.keys + 15) & ~15) - kbase);
                    for (int e = lane; e < (z1 - d1) * C::SLABS * 8; e += 32) {
                        const int c = e % (C::SLABS * 8);
                        sts128(tile + (uint32_t)((d1 + e / (C::SLABS * 8)) * 128 + (c >> 3) * C::KSLAB + (c & 7) * 16), make_uint4(0u, 0u, 0u, 0u));
                    }
                    tc::fence_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::V_OK + st));
            }
        }
    } else if (warp >= K_WARP) {
        // ------------------------------------------------------------ cache rows into the rings, every second box of K or V
        const bool is_v = warp >= V_WARP;
        const int first = (warp - K_WARP) & 1;
        const CUtensorMap* map = is_v ? &tmV : &tmK;
        if (lane == 0) tma_prefetch_desc(map);
        const uint64_t pol = p.group == 1 ? l2_policy_evict_first() : l2_policy_normal();  // read once, or by the group's CTAs
        const int br = min(p.block_size, 16), nbox = BN / br;
        const int full0 = is_v ? C::V_FULL : C::K_FULL, empty0 = is_v ? C::V_EMPTY : C::K_EMPTY;
        const int slots = is_v ? C::NV : C::NK;
        const uint32_t ring = is_v ? sV : sK, el = elect_one();
        auto entry = [&](const Segment& g, int tile) {  // block id of box `lane` of the tile; past the keys or invalid: zero fill
            const int t = tile * BN + lane * br;
            if (lane >= nbox || t >= g.keys) return p.num_blocks;
            const int e = ld_global(p.block_tables + (size_t)g.s * p.max_blocks_per_seq + (t >> p.block_log2));
            if (e < 0 || e >= p.num_blocks) {
                flag_error(p.err, PA_DEVERR_BLOCK);
                return p.num_blocks;
            }
            return e;
        };
        Segment g, ahead;
        bool more = segment(0, g);
        int id = more ? entry(g, g.tile) : 0;
        for (int seg = 1; more && ok; ++seg, g = ahead) {
            for (int u = 0; u < g.n; ++u) {
                const int tile = g.tile + u;
                int nxt = 0;
                if (u + 1 == g.n) more = segment(seg, ahead);
                if (u + 1 < g.n || more) nxt = u + 1 < g.n ? entry(g, tile + 1) : entry(ahead, ahead.tile);
                const int st = (int)uniform((uint32_t)slot);
                if (use > 0) wait(empty0 + st, use - 1);
                if (!ok) break;
                const uint32_t full = bar(full0 + st), dst = ring + (uint32_t)(st * C::TILE);
                if (el) mbar_arrive_expect_tx(full, C::TILE / 2);
                __syncwarp();
#pragma unroll 1
                for (int x = first; x < nbox; x += 2) {
                    const int e = __shfl_sync(0xffffffffu, id, x);
                    const int row = (int)uniform((uint32_t)((tile * BN + x * br) & (p.block_size - 1)));
#pragma unroll
                    for (int sl = 0; sl < C::SLABS; ++sl)
                        tma_box(el, dst + (uint32_t)(sl * C::KSLAB + x * br * 128), map, sl * 64, g.head, row, e, full, pol);
                }
                id = nxt;
                if (++slot == slots) slot = 0, ++use;
            }
        }
        // the last releases too: none is on its way when the block leaves
        for (int s = 0; s < slots; ++s)
            if (use > 0 || s < slot) wait(empty0 + s, s < slot ? use : use - 1);
    } else if (warp == Q_WARP) {
        // ------------------------------------------------------------ tells the others the segments, and loads the units'
        // query rows, once for each copy.  Two segments are told ahead whatever it takes (the loaders look one ahead of the
        // products), more where the others have read what was there
        const Start start = by_warp ? find_start_warp(p, range, (int)gridDim.x / p.group, lane) : *rec;
        if (lane == 0) {
            tma_prefetch_desc(&tmQ);
            const uint32_t box = (uint32_t)(p.tb * p.g_heads * 128);
            uint4* ring = reinterpret_cast<uint4*>(smem + C::SEG_OFF);
            Walk walk(p, start, blk);
            int told = 0, seg = 0;  // segments told; query rows loaded
            bool more = true;
            for (;;) {
                bool tell = more && told < seg + C::SEGS && (told != 1 || seg > 0);
                if (tell && told >= C::SEGS) {
                    const int sl = told % C::SEGS, phase = told / C::SEGS - 1;
                    if (told < seg + 2) ok = wait_limited(bar(C::SEG_EMPTY + sl), (uint32_t)(phase & 1), p.err);
                    else tell = mbar_test(bar(C::SEG_EMPTY + sl), phase);
                    if (!ok) break;
                }
                if (tell) {
                    Segment g;
                    walk.next(g);
                    more = g.n > 0;
                    uint4* to = ring + 3 * (told % C::SEGS);
                    to[0] = make_uint4((uint32_t)g.s, (uint32_t)g.head, (uint32_t)g.tok0, (uint32_t)g.toks);
                    to[1] = make_uint4((uint32_t)g.q0, (uint32_t)g.tile, (uint32_t)g.n, (uint32_t)g.ctx);
                    to[2] = make_uint4((uint32_t)g.keys, (uint32_t)g.drafted, (uint32_t)g.parts, (uint32_t)g.back);
                    mbar_arrive(bar(C::SEG_FULL + told % C::SEGS));
                    ++told;
                    continue;
                }
                const uint4 a = ring[3 * (seg % C::SEGS)];
                if (ring[3 * (seg % C::SEGS) + 1].z == 0u) break;
                if (seg > 0) ok = wait_limited(bar(C::Q_EMPTY), (uint32_t)((seg - 1) & 1), p.err);
                if (!ok) break;
                mbar_arrive_expect_tx(bar(C::Q_FULL), box * C::SLABS * COPIES);
#pragma unroll 1
                for (int c = 0; c < COPIES; ++c)
#pragma unroll 1
                    for (int sl = 0; sl < C::SLABS; ++sl)
                        tma_q(sQ + (uint32_t)(sl * C::QSLAB + c * NR * 128), &tmQ, sl * 64, (int)a.y * p.g_heads, (int)a.z, bar(C::Q_FULL));
                ++seg;
            }
            if (seg > 0) (void)wait_limited(bar(C::Q_FULL), (uint32_t)((seg - 1) & 1), p.err);
        }
    } else if (warp == QK_WARP) {
        // ------------------------------------------------------------ QK issue: the whole warp walks the loop and one elected
        // lane issues, from descriptors that a shuffle makes warp-uniform
        constexpr uint32_t ID_QK = tc::idesc_f16(BF16, false, 128, BN);
        const uint64_t dq = tc::sdesc_sw128(sQ, 16, 1024), dk0 = tc::sdesc_sw128(sK, 16, 1024);
        const uint32_t el = elect_one(), tS = uniform(tmem);
        int i = 0, seg = 0;
        for (Segment g; segment(seg, g);) {
            wait(C::Q_FULL, seg);
            for (int u = 0; u < g.n; ++u, ++i) {
                const int b = (int)uniform((uint32_t)(i % NS)), st = (int)uniform((uint32_t)(i % C::NK));
                wait(C::K_FULL + st, i / C::NK);
                if (i >= NS) wait(C::PV_DONE + b, i / NS - 1);  // the weights in the buffer have been used
                if (!ok) break;
                tc::fence_after();
                const uint64_t dk = dk0 + (uint32_t)((st * C::TILE) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(el, tS + C::s_col(b), dq + (uint32_t)(((kk >> 2) * C::QSLAB + (kk & 3) * 32) >> 4),
                           dk + (uint32_t)(((kk >> 2) * C::KSLAB + (kk & 3) * 32) >> 4), ID_QK, kk > 0);
                commit(el, bar(C::S_FULL + b));
                commit(el, bar(C::K_EMPTY + st));
                if (u == g.n - 1) commit(el, bar(C::Q_EMPTY));
            }
            if (!ok) break;
            ++seg;
        }
        if (i > 0) {  // every MMA must be complete before TMEM is released
            commit(el, bar(C::DRAIN));
            (void)warp_wait(bar(C::DRAIN), 0, p.err);
        }
    } else if (warp == PV_WARP) {
        // ------------------------------------------------------------ PV issue: O += P V, P in tensor memory
        constexpr uint32_t ID_PV = tc::idesc_f16(BF16, true, 128, D);
        const uint64_t dv0 = tc::sdesc_sw128(sV, C::KSLAB, 1024);
        const uint32_t el = elect_one(), dO = uniform(tmem + C::O_COL), tP = uniform(tmem);
        int i = 0, seg = 0;
        for (Segment g; segment(seg, g);) {
            if (seg > 0) wait(C::O_FREE, seg - 1);  // O of the segment before has been read
            for (int u = 0; u < g.n; ++u, ++i) {
                const int b = (int)uniform((uint32_t)(i % NS)), st = (int)uniform((uint32_t)(i % C::NV));
                const uint32_t acc = uniform(u > 0);
                wait(C::V_OK + st, i / C::NV);
                wait(C::P_FULL + b, i / NS);
                if (!ok) break;
                tc::fence_after();
                const uint64_t dv = dv0 + (uint32_t)((st * C::TILE) >> 4);
                const int steps = (int)uniform((uint32_t)((g.keys - (g.tile + u) * BN + 15) / 16));  // those that hold keys
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk) {
                    // the columns of 16 keys' weights and of their remainders
                    const uint32_t at = tP + C::s_col(b) + (uint32_t)(kk / (KW / 16) * KW + 8 * (kk % (KW / 16)));
                    mma_ts(kk < steps ? el : 0u, dO, at, dv + (uint32_t)((kk * 2048) >> 4), ID_PV, kk > 0 ? 1u : acc);
                    mma_ts(kk < steps ? el : 0u, dO, at + (uint32_t)(KW / 2), dv + (uint32_t)((kk * 2048) >> 4), ID_PV, 1u);
                }
                commit(el, bar(C::V_EMPTY + st));
                commit(el, bar(C::PV_DONE + b));
            }
            if (!ok) break;
            ++seg;
        }
        if (i > 0) {
            commit(el, bar(C::DRAIN + 1));
            (void)warp_wait(bar(C::DRAIN + 1), 0, p.err);
        }
    }
    tc::fence_before();
    // Every load is behind a wait of the issuers.  If all went well nothing is in flight now; if some role's wait ran
    // out, no copy may be left behind: the last ones of each ring (the loaders stopped there; a phase that waits for another
    // loader's arrival as well runs out, long after the copies themselves are done)
    const bool failed = __syncthreads_or(!ok);
    if (failed && warp >= K_WARP) {
        const int full0 = warp >= V_WARP ? C::V_FULL : C::K_FULL, slots = warp >= V_WARP ? C::NV : C::NK;
        for (int s = 0; s < slots; ++s)
            if (use > 0 || s < slot) (void)warp_wait(bar(full0 + s), (uint32_t)((s < slot ? use : use - 1) & 1), p.err);
    }
    if (threadIdx.x == 0) {
        if (failed) begins = goes_on = make_int4(0, 0, 0, 0);
        p.desc[blockIdx.x] = begins;
        p.desc[gridDim.x + blockIdx.x] = goes_on;
    }
    if (warp == QK_WARP) {
        tc::fence_after();
        tc::dealloc(tmem, C::TMEM_COLS);
    }
}

// Joins the partials of the units that the ranges' ends cut: out = sum_k 2^(m_k - max m) o_k / sum_k 2^(m_k - max m) l_k,
// in a fixed order.  A partial holds columns 4 c .. 4 c + 3 of all its rows next to each other.  A unit of few partials by
// the blocks of the CTA it starts in (a block for 16 rows, their columns over its threads); one of many (few long contexts) by
// the blocks of all the CTAs it spans, a block a row, whose warps take every 8th partial each.
template <bool BF16, int D, int NR>
__global__ void __launch_bounds__(tree::MERGE_THREADS) tree_merge_kernel(const TreeParams p) {
    using F = F16x2<BF16>;
    constexpr int NW = tree::MERGE_THREADS / 32, V = D / 64, V4 = (D / 4 + 31) / 32;  // 16-byte columns a thread; a lane
    constexpr int kFew = 8;
    __shared__ float4 acc[NW][D / 4];
    __shared__ float wt[tree::MERGE_THREADS], red[2][NW];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = (int)blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the next kernel of the step may start its launch; it waits for this grid before reading anything
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int4 cut[2] = {ld_l2(p.desc + cta), ld_l2(p.desc + gridDim.x + cta)};
    auto store = [&](int row0, int row, int c4, float4 a, float inv) {
        const int tok = (int)(((uint32_t)row * (uint32_t)p.g_magic) >> 16);
        if (4 * c4 < p.hd)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) +
                                      ((size_t)row0 + (size_t)tok * p.n_q_heads + (row - tok * p.g_heads)) * p.hd + 4 * c4) =
                make_uint2(F::pack_rn(a.x * inv, a.y * inv), F::pack_rn(a.z * inv, a.w * inv));
    };
    auto add = [](float4& a, const float4& x, float f) {
        a.x = fmaf(x.x, f, a.x);
        a.y = fmaf(x.y, f, a.y);
        a.z = fmaf(x.z, f, a.z);
        a.w = fmaf(x.w, f, a.w);
    };
    const int row16 = (int)blockIdx.y * 16 + (tid & 15);
    if (cut[0].x > 0 && cut[0].x <= kFew && row16 < cut[0].y) {
        const int4 u = cut[0];
        const int c = (tid >> 4) * V;  // this thread's columns
        auto slot_at = [&](int k) { return (size_t)(2 * (cta + k * p.group) + (k == 0)); };
        float2 ml[kFew];
#pragma unroll
        for (int k = 0; k < kFew; ++k) ml[k] = k < u.x ? ld_l2(p.part_ml + slot_at(k) * NR + row16) : make_float2(-INFINITY, 0.f);
        float4 a[V] = {}, x[4][V];
        auto fetch = [&](int k0) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k0 + k < u.x)
#pragma unroll
                    for (int v = 0; v < V; ++v) x[k][v] = ld_l2(p.part_o + (slot_at(k0 + k) * (D / 4) + c + v) * NR + row16);
        };
        fetch(0);
        float mx = -INFINITY, l = 0.f;
#pragma unroll
        for (int k = 0; k < kFew; ++k) mx = fmaxf(mx, ml[k].x);
#pragma unroll
        for (int k = 0; k < kFew; ++k) {
            const float f = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - mx);
            l += ml[k].x == -INFINITY ? ml[k].y : ml[k].y * f;
            ml[k].x = f;
        }
#pragma unroll
        for (int k0 = 0; k0 < kFew; k0 += 4) {
            if (k0 > 0 && k0 < u.x) fetch(k0);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k0 + k < u.x)
#pragma unroll
                    for (int v = 0; v < V; ++v) add(a[v], x[k][v], ml[k0 + k].x);
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) store(u.z, row16, c + v, a[v], inv);
    }
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const int4 u = which == 0 ? cut[0] : cut[1];
        const int parts = u.x, b = u.w;
        if (parts <= kFew) continue;
        auto slot_at = [&](int k) { return (size_t)(2 * (b + k * p.group) + (k == 0)); };
        const int mine = (cta - b) / p.group;
        for (int row = mine * (int)gridDim.y + (int)blockIdx.y; row < u.y; row += parts * (int)gridDim.y) {
            const float2 ml = tid < parts ? ld_l2(p.part_ml + slot_at(tid) * NR + row) : make_float2(-INFINITY, 0.f);
            const float m = ml.x;
            float mx = m;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (lane == 0) red[0][warp] = mx;
            __syncthreads();
            mx = red[0][0];
            for (int w = 1; w < NW; ++w) mx = fmaxf(mx, red[0][w]);
            const float w = m == -INFINITY ? 0.f : ex2(m - mx);
            wt[tid] = w;
            float lw = m == -INFINITY ? ml.y : ml.y * w;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
            if (lane == 0) red[1][warp] = lw;
            __syncthreads();
            float4 a[V4] = {};
#pragma unroll 4
            for (int k = warp; k < parts; k += NW) {
                const float f = wt[k];
#pragma unroll
                for (int v = 0; v < V4; ++v)
                    if (lane + 32 * v < D / 4) add(a[v], ld_l2(p.part_o + (slot_at(k) * (D / 4) + lane + 32 * v) * NR + row), f);
            }
#pragma unroll
            for (int v = 0; v < V4; ++v)
                if (lane + 32 * v < D / 4) acc[warp][lane + 32 * v] = a[v];
            __syncthreads();
            if (tid < D / 4) {
                float lt = 0.f;
                for (int k = 0; k < NW; ++k) lt += red[1][k];
                float4 s = acc[0][tid];
                for (int k = 1; k < NW; ++k) add(s, acc[k][tid], 1.f);
                store(u.z, row, tid, s, lt != 0.f ? 1.f / lt : 0.f);
            }
            __syncthreads();
        }
    }
}

}  // namespace pa
