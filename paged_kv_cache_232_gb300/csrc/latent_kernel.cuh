// latent_kernel.cuh -- attention over a paged cache of latent vectors (absorbed form), on the
// tcgen05 tensor cores.
//
// A cache row of a token is [c (DL columns), kr (64 columns)]: its latent vector and the rotated
// key part all heads share.  Every head's key is the whole row, its value the latent part:
//     out[h] = sum_t softmax_t(scale * q[h] . row_t) c_t,
// so the H heads of a token are H rows of one dense contraction over the same keys: each cache
// row is read once for all of them.  Decode (one query token a sequence) and ragged chunks
// (bottom-right causal) are one kernel: a unit is up to NR query rows (tokens x heads, 64 heads
// at most) of one sequence over its keys (more rows: latent_pair_kernel.cuh).
//
// GB300 design:
//  * Keys come in tiles of 64 tokens, as DL / 128 "pair" slots (two 64-column slabs of 64 rows,
//    128-byte swizzled, 16 KB) and one rotary slot (8 KB).  Pair slots and rotary slots are two
//    rings: a pair slot is released as soon as the PV product of its 128 columns is done, the
//    rotary slot after the QK product, so loads stay in flight at a finer grain than whole tiles.
//  * S = Q K^T: M = 64 query rows, N = 64 tokens, both operands K-major.  At M = 64 row r sits in
//    TMEM lane (r mod 16) + 32 (r / 16), so one thread owns one row: the softmax needs no
//    exchange between threads.  With NR < 64 the A operand's rows past NR read the shared memory
//    behind the Q tile: rows of D are independent and those are never looked at.
//  * O^T = C^T P^T: M = 128 latent columns (A: the pair slot read MN-major), N = NR query rows
//    (B: the weights, K-major), so the accumulator takes DL / 128 x NR TMEM columns (256 at 64
//    rows x 512; rows on M would take all 512 columns and leave none for S).
//  * The running maximum is updated lazily: O and l are rescaled only when a row's maximum grows
//    by more than 2^8; weights up to 2^8 above the reference are exact in fp32 and far from the
//    16-bit formats' limits.
//  * A weight enters the PV product rounded once to the cache's 16-bit type (half a step is 2^-8 in
//    bf16, 2^-11 in fp16, relative), and l sums the rounded weights, so that they still sum to one.
//    The roundings of different keys are independent, so their sum stays below the rounding of the
//    output to that type.  Both sides measured: root-mean-square error against 64 bits, relative to
//    the output, 0.0019..0.0020 in bf16 (weights of 32 bits: 0.0016..0.0017) and 0.00022..0.00027 in
//    fp16 (0.00020..0.00021), the most for one short context.  The remainders as further columns of the
//    operand or (64 rows x 512) as a second product, as prefill_kernel.cuh has them: built and timed in
//    turn, 64 x 100..2048 tokens at 16 heads 25.6 -> 27.0 us, 4 x 32K at 64 heads 40.7 -> 44.0, 64 x 1K..8K
//    at 64 heads 81 -> 88.  For pairs their MMAs alone (the product issued twice): 128 x 1K..8K at 128 heads
//    134 -> 162 us, prefill 905 -> 1196, and shared memory has no place for them (16 KB, 0.2 are left).
//  * All units, laid end to end and measured in cost (a unit's start and output, then its tiles), are
//    cut into equal ranges, one a CTA (one CTA per SM): units that end inside a range are written
//    directly, the two that its ends cut leave fp32 partials that latent_merge_kernel joins in a fixed
//    order (no atomics).  The split needs no host-side lengths and no workspace beyond two partials a CTA.
//  * The softmax warps also write the output, transposed back by 2-byte stores (64 bytes a warp and row):
//    staging or shuffling it would go through shared memory, whose path the MMA operands keep busy.
//  * Waits have a time limit; on expiry PA_DEVERR_TIMEOUT is set, the roles leave their loops and
//    TMEM is released.
//
// What bounds it: memory, up to 64 rows a unit.  In steady state a 64-token tile (73.7 KB) takes ~3160
// cycles at 16 rows and ~3450 at 64 (GB300, 256 sequences of 1K..2K tokens): 6.9 and 6.3 TB/s over the
// 152 SMs, about the copy rate.  What is left is fixed: ~6 us to the first S (lengths, block table, first
// rows from DRAM, each waiting for the one before), 1..3 us for output or partials, ~4 us for the merge.
// Whole calls: 64 sequences of 100..2048 tokens at 16 heads 25.7 us (12 us of bytes at the copy rate), 4 of
// 32K at 64 heads 40.8 us (22).  Steps on the way: one MMA issuer for QK and PV 38 and 67 us (the PV that frees
// the ring queued behind the next tile's QK); descriptors formed in a divergent lane ~90 cycles an MMA.
#pragma once

#include "pa_launch.h"
#include "tcgen05.cuh"

namespace pa {
namespace lat {

constexpr int TK = 64;                  // tokens per tile
constexpr int ROPE = 64;                // rotary columns of a cache row
constexpr int SLAB = TK * 128;          // bytes of 64 tokens x 64 columns
constexpr int PAIR = 2 * SLAB;
// Weights are 2^(score - reference + kShift): in fp16 up to 2^15 (the reference may lag by 2^8), so that weights of
// 2^-21 of the largest are still normal numbers -- many equal small weights would all round the same way as subnormals
template <bool BF16>
constexpr float kShift = BF16 ? 0.f : 7.f;
// warps 0..3: softmax; then the two MMA issuers, the Q loader, and the cache row loaders (one a pair slot of a tile, one
// for the rotary slot)
constexpr int SOFTMAX_WARPS = 4, QK_WARP = 4, PV_WARP = 5, Q_WARP = 6, TMA_WARP = 7;
// threads of a merge block (16 rows): a warp a row where the blocks then still run at once
constexpr int merge_threads(int nr) { return nr <= 32 ? 512 : 256; }
constexpr int MAX_CTAS = 256;           // of the split: the merge gives every partial a thread
static_assert(MAX_CTAS <= merge_threads(128) && PA_LATENT_MAX_CTAS <= MAX_CTAS, "partials of a unit");

template <int DL, int NR>
struct Cfg {
    static_assert(DL == 256 || DL == 512, "latent columns");
    static_assert(NR == 16 || NR == 32 || NR == 64, "query rows per unit");
    static constexpr int NB = DL / 128;                 // pair slots per tile = M blocks of O^T
    static constexpr int THREADS = (TMA_WARP + NB + 1) * 32;
    static constexpr int QSLABS = DL / 64 + 1;
    static constexpr int QSLAB = NR * 128;
    // as many ring slots as fit next to the Q tile and the weights
    static constexpr int NPAIR = DL == 512 ? (NR == 64 ? 8 : NR == 32 ? 10 : 11) : (NR == 64 ? 8 : 10);
    static constexpr int NROPE = DL == 512 ? (NR == 64 ? 2 : 3) : (NR == 64 ? 4 : 5);
    static constexpr int Q_OFF = 0;
    static constexpr int P_OFF = QSLABS * QSLAB;
    static constexpr int PAIR_OFF = P_OFF + NR * 128;
    static constexpr int ROPE_OFF = PAIR_OFF + NPAIR * PAIR;
    static constexpr int BAR_OFF = ROPE_OFF + NROPE * SLAB;
    // barriers
    static constexpr int PAIR_FULL = 0, PAIR_EMPTY = NPAIR, ROPE_FULL = 2 * NPAIR, ROPE_EMPTY = 2 * NPAIR + NROPE;
    static constexpr int Q_FULL = 2 * (NPAIR + NROPE), Q_EMPTY = Q_FULL + 1, S_FULL = Q_FULL + 2, P_FULL = Q_FULL + 4,
                         PV_DONE = Q_FULL + 5, O_FREE = Q_FULL + 6, DRAIN = Q_FULL + 7, S_EMPTY = Q_FULL + 9,
                         NUM_BARS = Q_FULL + 11;
    static constexpr int MISC_OFF = (BAR_OFF + NUM_BARS * 8 + 15) & ~15;  // start record, TMEM address, scan scratch
    static constexpr int ROW_OFF = MISC_OFF + 192;               // alpha [NR] and 1 / l [NR]
    static constexpr int SMEM_BYTES = ROW_OFF + 2 * NR * 4 + 1024;  // + alignment slack
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
    static_assert(ROW_OFF % 16 == 0, "1 / l is read 16 bytes at a time");
    // the A operand of QK reads 64 rows of each Q slab, whatever NR is
    static_assert((QSLABS - 1) * QSLAB + 64 * 128 <= BAR_OFF, "QK operand stays inside the tile area");
    static constexpr uint32_t O_COL = 128;                       // two S buffers of 64 columns, then O^T
    static constexpr uint32_t TMEM_COLS = 128 + NB * NR <= 256 ? 256 : 512;
};

// kind::f16 instruction descriptor with the A operand's major-ness (bit 15), see tc::idesc_f16
__host__ __device__ constexpr uint32_t idesc(bool bf16, bool a_mn_major, int M, int N) {
    return tc::idesc_f16(bf16, false, M, N) | ((a_mn_major ? 1u : 0u) << 15);
}

__device__ __forceinline__ void tma_load_3d(uint32_t el, uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                            uint32_t bar, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %7, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy), "r"(el)
        : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// Issue, commits and loads are predicated on `el` (the warp's elected lane) rather than branched around: the
// issuing warp stays converged, so that descriptors are formed once for the warp.
__device__ __forceinline__ void mma(uint32_t el, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
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

// barrier of the four softmax warps that ORs a predicate over them
__device__ __forceinline__ bool softmax_or(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ float lds_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}

// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// The warp waits, all lanes polling (one request); the polling loop stays out of line, so that the waits'
// usual path is a few instructions (the roles' code competes for the instruction cache).  The result is the
// warp's, false as soon as one lane's wait ran out: the lanes keep their own clocks, and a role that went on in
// some of its lanes would meet its next warp-wide instruction without the others.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, unsigned* err) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, err));
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, unsigned* err) {
    if (__any_sync(0xffffffffu, !mbar_try_wait(bar, parity))) return wait_slow(bar, parity, err);
    return true;
}

// ---- the split of all units' tiles over the CTAs ---------------------------------------------

// One sequence's chunk: its first query row, query tokens and keys.  Decode: one token, the rows
// in sequence order.  Lengths out of range: decode takes the sequence as empty (its rows become
// zero), a chunk is skipped (q_len 0).
struct Chunk {
    int q0, q_len, kv_len;
    bool bad;
};

__device__ __forceinline__ Chunk load_chunk(const LatentParams& p, int c) {
    Chunk k;
    const int cap = p.max_blocks_per_seq * p.block_size;
    k.kv_len = __ldg(p.kv_lens + c);
    if (p.q_loc == nullptr) {
        k.q0 = c;
        k.q_len = 1;
        k.bad = k.kv_len < 0 || k.kv_len > cap;
        if (k.bad) k.kv_len = 0;
    } else {
        k.q0 = __ldg(p.q_loc + c);
        const int q1 = __ldg(p.q_loc + c + 1);
        k.q_len = q1 - k.q0;
        k.bad = k.q0 < 0 || q1 < k.q0 || q1 > p.total_q || k.q_len > p.max_q_len || k.kv_len < k.q_len ||
                k.kv_len > cap;
        if (k.bad) k.q_len = 0;
    }
    return k;
}

// keys that token block j of a chunk sees: up to its last token's limit
__device__ __forceinline__ int keys_of(const LatentParams& p, const Chunk& k, int j) {
    return k.kv_len - k.q_len + min((j + 1) * p.tb, k.q_len);
}
__device__ __forceinline__ int tiles_of(const LatentParams& p, int keys) {
    return max(1, (keys + (1 << p.tile_log2) - 1) >> p.tile_log2);
}

// sum over i < n of floor((a i + b) / m), by the Euclidean reduction of the lattice-point count
// (a, m at most 128: from the first reduction of b on, a n + b fits 32 bits for n below 2^24)
__device__ __forceinline__ long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
    unsigned long long s = 0;
    while (true) {
        if (a >= m) {
            s += (unsigned long long)n * (n - 1) / 2 * (a / m);
            a %= m;
        }
        if (b >= m) {
            s += (unsigned long long)n * (b / m);
            b %= m;
        }
        const uint32_t y = a * n + b;
        if (y < m) return (long long)s;
        n = y / m;
        b = y % m;
        const uint32_t t = m;
        m = a;
        a = t;
    }
}

// The ranges are cut in units of cost: a unit (a token block of a chunk) counts unit_cost for its start and
// its output, then one a tile.
// cost of token blocks 0 .. n - 1 of a chunk (n at most its number of blocks)
__device__ __forceinline__ long long tiles_before(const LatentParams& p, const Chunk& k, int n) {
    if (n == 0) return 0;
    const int last = (k.q_len + p.tb - 1) / p.tb - 1;  // the last block may be short
    const int full = min(n, last), ctx = k.kv_len - k.q_len, round = (1 << p.tile_log2) - 1;
    long long s = (long long)n * p.unit_cost;
    if (full > 0) {  // block i: ceil((ctx + (i + 1) tb) / tile) tiles
        const int lo = (ctx + p.tb + round) >> p.tile_log2, hi = (ctx + full * p.tb + round) >> p.tile_log2;
        if (hi - lo <= 8) {
            // few different counts: the blocks with more than t tiles are those from floor((t tile - ctx) / tb) on
            s += (long long)full * lo;
            for (int t = lo; t < hi; ++t) s += full - ((t << p.tile_log2) - ctx) / p.tb;
        } else {
            s += floor_sum((uint32_t)full, 1u << p.tile_log2, (uint32_t)p.tb, (uint32_t)(ctx + p.tb + round));
        }
    }
    if (n > last) s += tiles_of(p, k.kv_len);
    return s;
}

__device__ __forceinline__ long long tiles_in(const LatentParams& p, const Chunk& k) {
    if (k.q_len == 0) return 0;
    return p.q_loc == nullptr ? (long long)tiles_of(p, k.kv_len) + p.unit_cost
                              : tiles_before(p, k, (k.q_len + p.tb - 1) / p.tb);
}

// A range: where it starts (chunk, token block, cost into that block) and its cost.
struct Start {
    long long rem;  // (while it is looked for: the cost into the chunk)
    int c, j, at, count, per;
};
static_assert(sizeof(Start) <= 32, "record area");

// Range `range` of `ranges`.  Every thread of the CTA calls it; all return the same record.  One pass over the
// sequences' lengths where they are at most as many as threads, two otherwise.
template <int THREADS>
__device__ __forceinline__ Start find_start(const LatentParams& p, int range, int ranges, long long* warp_sum, Start* rec) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int NW = THREADS / 32;
    if (tid == 0) rec->count = 0;
    Chunk k{0, 0, 0, false};
    long long mine = 0, n = 0;  // cost of this thread's sequences, of the one in k
    for (int c = tid; c < p.num_chunks; c += THREADS) {
        k = load_chunk(p, c);
        if (k.bad && blockIdx.x == 0) flag_error(p.err, PA_DEVERR_LENGTH);
        n = tiles_in(p, k);
        mine += n;
    }
    const bool one = p.num_chunks <= THREADS;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    long long total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const long long x = warp_sum[w];
        if (w < warp) before += x;
        total += x;
    }
    const long long even = (total + ranges - 1) / ranges;
    const int per = (int)max(even, (long long)p.min_tiles);
    const long long lo = (long long)range * per;
    if (lo < total) {
        auto found = [&](int c, const Chunk& q, long long at, long long cost) {
            if (cost > 0 && lo >= at && lo < at + cost) {
                rec->c = c;
                rec->j = 0;
                rec->at = (int)(lo - at);
                rec->rem = p.q_loc != nullptr && q.q_len > p.tb ? lo - at : -1;  // -1: one token block, nothing to look for
                rec->count = (int)min((long long)per, total - lo);
            }
        };
        if (one) {
            found(tid, k, before + incl - n, n);
        } else {
            // prefix sums, THREADS sequences at a time
            long long base = 0;
            for (int c0 = 0; c0 < p.num_chunks && base <= lo; c0 += THREADS) {
                __syncthreads();
                const int c = c0 + tid;
                Chunk q{0, 0, 0, false};
                if (c < p.num_chunks) q = load_chunk(p, c);
                const long long m = c < p.num_chunks ? tiles_in(p, q) : 0;
                long long in = m;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, in, o);
                    if (lane >= o) in += y;
                }
                if (lane == 31) warp_sum[warp] = in;
                __syncthreads();
                long long all = base, bef = base;
                for (int w = 0; w < NW; ++w) {
                    if (w < warp) bef += warp_sum[w];
                    all += warp_sum[w];
                }
                found(c, q, bef + in - m, m);
                base = all;
            }
        }
        if (p.q_loc != nullptr) {
            // the last token block of the chunk whose cost starts at or before the range, THREADS candidates a round
            __syncthreads();
            const Start r = *rec;
            if (r.rem >= 0) {
                const Chunk q = load_chunk(p, r.c);
                int j0 = 0, m = (q.q_len + p.tb - 1) / p.tb;  // it is in [j0, j0 + m)
                do {
                    const int step = (m + THREADS - 1) / THREADS, j = j0 + tid * step;
                    const long long at = tid * step < m ? tiles_before(p, q, j) : 0;
                    const int hit = __syncthreads_count(tid * step < m && at <= r.rem);  // (j0 itself: always)
                    if (tid == hit - 1) {
                        rec->j = j;
                        rec->at = (int)(r.rem - at);
                    }
                    j0 += (hit - 1) * step;
                    m = min(step, m - (hit - 1) * step);
                } while (m > 1);
            }
        }
    }
    __syncthreads();
    Start s = *rec;
    s.per = per;
    return s;
}

// One segment of a range: tiles [tile, tile + n) of one unit's `tiles`.
struct Segment {
    int c, j;
    int tile, n, tiles;
    int ctx, keys;          // token jt of the block sees keys <= ctx + j tb + jt; the unit's tokens see [0, keys)
    int rows;               // query rows of the unit
    int row0;               // the first one's row of q and out, [total_q * n_heads]
    int parts, back;        // ranges the unit's tiles span (0: this one alone), and how many of them are before this one
};

// A cut unit's partials: the range it starts in writes slot 2 range + 1, those behind it slot 2 range.
__device__ __forceinline__ int slot_of(const Segment& g, int range) { return 2 * range + (g.tile == 0 ? 1 : 0); }

// What the merge needs to know of a cut unit, from each range it spans
__device__ __forceinline__ int4 cut_of(const Segment& g, int range) {
    return make_int4(g.parts, g.rows, g.row0, range - g.back);
}

template <typename F>
__device__ __forceinline__ void for_each_segment(const LatentParams& p, const Start& s, F&& f) {
    int c = s.c, j = s.j, at = s.at, left = s.count;
    if (left <= 0) return;
    Chunk k = load_chunk(p, c);
    while (left > 0) {
        Segment g;
        g.c = c;
        g.j = j;
        g.keys = keys_of(p, k, j);
        g.tiles = tiles_of(p, g.keys);
        const int n = min(g.tiles + p.unit_cost - at, left);  // cost of the unit in this range
        left -= n;
        g.tile = max(0, at - p.unit_cost);
        g.n = max(0, at + n - p.unit_cost) - g.tile;
        const int rest = g.tiles - g.tile - g.n;  // behind this range, and g.tile before it: whole ranges but for the ends
        g.back = (g.tile + s.per - 1) / s.per;
        g.parts = (g.tile > 0 || rest > 0) ? g.back + 1 + (rest + s.per - 1) / s.per : 0;
        g.ctx = k.kv_len - k.q_len;
        g.rows = min(p.tb, k.q_len - j * p.tb) * p.n_heads;
        g.row0 = (k.q0 + j * p.tb) * p.n_heads;
        if (g.n > 0 && !f(g)) return;
        if (left <= 0) return;
        at = 0;
        if ((++j) * p.tb < k.q_len) continue;
        j = 0;
        do {
            if (++c >= p.num_chunks) return;
            k = load_chunk(p, c);
        } while (k.q_len == 0);
    }
}

}  // namespace lat

template <bool BF16, int DL, int NR>
__global__ void __launch_bounds__(lat::Cfg<DL, NR>::THREADS, 1)
latent_kernel(const LatentParams p, const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmQ) {
    using namespace lat;
    using C = Cfg<DL, NR>;
    using F = F16x2<BF16>;
    constexpr int NB = C::NB;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_addr(smem);
    const uint32_t sQ = sbase + C::Q_OFF, sP = sbase + C::P_OFF, sPair = sbase + C::PAIR_OFF, sRope = sbase + C::ROPE_OFF;
    const uint32_t bars = sbase + C::BAR_OFF;
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    Start* rec = reinterpret_cast<Start*>(smem + C::MISC_OFF);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::MISC_OFF + 32);
    long long* warp_sum = reinterpret_cast<long long*>(smem + C::MISC_OFF + 64);
    float* alpha_s = reinterpret_cast<float*>(smem + C::ROW_OFF);
    float* inv_s = alpha_s + NR;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NPAIR; ++i) {
            mbar_init(bar(C::PAIR_FULL + i), 1);
            mbar_init(bar(C::PAIR_EMPTY + i), 1);
        }
        for (int i = 0; i < C::NROPE; ++i) {
            mbar_init(bar(C::ROPE_FULL + i), 1);
            mbar_init(bar(C::ROPE_EMPTY + i), 1);
        }
        mbar_init(bar(C::Q_FULL), 1);
        mbar_init(bar(C::Q_EMPTY), 1);
        mbar_init(bar(C::S_FULL), 1);
        mbar_init(bar(C::S_FULL + 1), 1);
        mbar_init(bar(C::P_FULL), SOFTMAX_WARPS);
        mbar_init(bar(C::PV_DONE), 1);
        mbar_init(bar(C::O_FREE), SOFTMAX_WARPS);
        mbar_init(bar(C::DRAIN), 1);
        mbar_init(bar(C::DRAIN + 1), 1);
        mbar_init(bar(C::S_EMPTY), NR / 16);
        mbar_init(bar(C::S_EMPTY + 1), NR / 16);
        fence_barrier_init();
    }
    if (warp == QK_WARP) {
        tc::alloc(smem_addr(const_cast<uint32_t*>(tmem_slot)), C::TMEM_COLS);
        tc::relinquish();
    }
    // a programmatic dependent of the kernel before it: nothing is read before that one is complete;
    // the merge may be set up now (it waits for this grid before it reads)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc::fence_before();
    const Start start = find_start<C::THREADS>(p, (int)blockIdx.x, (int)gridDim.x, warp_sum, rec);  // (synchronises the CTA)
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;    // none of this thread's waits has run out
    int done = 0;      // loader warps: tiles loaded

    if (warp < SOFTMAX_WARPS) {
        // ------------------------------------------------------------ softmax, rescale, epilogue
        const int r = lane < 16 ? 16 * warp + lane : -1;  // this thread's query row of the unit
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const uint32_t tS = tmem + lane_base, tO = tmem + lane_base + C::O_COL;
        const bool row_warp = 16 * warp < NR;             // the warp holds rows of S at all
        const float sc = p.qk_scale_log2;
        int i = 0;             // tile number over the CTA's range
        int pv_seen = 0;       // PV_DONE phases this warp has waited for
        int pair0 = 0;         // ring position of the tile's first pair slot
        int4 begins = make_int4(0, 0, 0, 0), goes_on = begins;  // the units cut at the range's end and at its start
        auto wait_pv = [&](int n) {  // PVs of tiles 0 .. n - 1 complete
            while (pv_seen < n) {
                ok = warp_wait(bar(C::PV_DONE), (uint32_t)(pv_seen & 1), p.err) && ok;
                ++pv_seen;
            }
        };
        for_each_segment(p, start, [&](const Segment& g) -> bool {
            const bool valid = r >= 0 && r < g.rows;
            const int tok = valid ? r / p.n_heads : 0;
            const int lim = valid ? g.ctx + g.j * p.tb + tok : -1;  // the row sees keys <= lim
            // the smallest limit of the unit's rows.  Lanes without one (and rows past them: other tokens' queries) are
            // not masked: rows are independent in both products, theirs are never written and never ask for a rescale
            const int lim_min = g.ctx + g.j * p.tb;
            float m_ref = -INFINITY, l = 0.f;
            for (int u = 0; u < g.n; ++u, ++i) {
                const int kbase = (g.tile + u) * TK;
                const uint32_t tSb = tS + (uint32_t)((i & 1) * 64);
                float x[64];
                float mx = -INFINITY;
                if (row_warp) {
                    ok = warp_wait(bar(C::S_FULL + (i & 1)), (uint32_t)((i >> 1) & 1), p.err) && ok;
                    tc::fence_after();
                    uint32_t s[64];
                    tc::ld64(tSb, s);
                    tc::wait_ld();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::S_EMPTY + (i & 1)));
#pragma unroll
                    for (int e = 0; e < 64; e += 2) {
                        const float2 v = __fmul2_rn(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), make_float2(sc, sc));
                        x[e] = v.x;
                        x[e + 1] = v.y;
                    }
                    if (kbase + TK - 1 > lim_min) {
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            if (kbase + e > lim) x[e] = -INFINITY;
                    }
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 64; ++e) m4[e & 3] = fmaxf(m4[e & 3], x[e]);
                    mx = valid ? fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) : -INFINITY;
                }
                const bool first = u == 0;
                if (first) m_ref = mx;  // no O yet: the first tile's own maximum is the reference
                if (softmax_or(!ok || mx > m_ref + 8.f)) {
                    if (softmax_or(!ok)) {  // some warp's wait ran out: all four leave together
                        ok = false;
                        return false;
                    }
                    const uint32_t alpha = smem_addr(alpha_s);
                    float a = 1.f;
                    if (mx > m_ref) {
                        a = m_ref == -INFINITY ? 1.f : ex2(m_ref - mx);
                        m_ref = mx;
                        l *= a;
                    }
                    if (r >= 0 && r < NR) alpha_s[r] = a;
                    wait_pv(i);  // O holds every tile before this one
                    softmax_sync();
                    tc::fence_after();
#pragma unroll 1
                    for (int q = 0; q < NB * NR / 16; ++q) {
                        uint32_t o[16];
                        tc::ld16(tO + 16 * q, o);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * lds_f32(alpha + (uint32_t)(((16 * q + e) & (NR - 1)) * 4)));
                        tc::st16(tO + 16 * q, o);
                    }
                    tc::wait_st();
                }
                if (row_warp) {
                    const float mu = m_ref == -INFINITY ? 0.f : m_ref - kShift<BF16>;
                    uint32_t w[32];
                    float2 ls = make_float2(0.f, 0.f);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float2 v = fadd2(make_float2(x[2 * e], x[2 * e + 1]), make_float2(-mu, -mu));
                        w[e] = F::pack_rn(ex2(v.x), ex2(v.y));
                        ls = fadd2(ls, F::unpack(w[e]));
                    }
                    l += ls.x + ls.y;
                    wait_pv(i);  // the weights' buffer is free
                    if (r >= 0) {
#pragma unroll
                        for (int ch = 0; ch < 8; ++ch)
                            sts128(sP + swz128(r, ch), make_uint4(w[4 * ch], w[4 * ch + 1], w[4 * ch + 2], w[4 * ch + 3]));
                    }
                } else {
                    wait_pv(i);  // in step with PV_DONE's phases, one a tile
                }
                if (kbase + TK > g.keys) {
                    // rows past the keys may hold anything (their weights are 0, but 0 * NaN is NaN): zero them
                    // (this tile's S, which also read them, is complete: the warps with rows have seen it
                    // before the vote above)
                    const int z = max(g.keys - kbase, 0), nz = (TK - z) * 8;
                    for (int b = 0; b < 2 * NB; ++b) {
                        const int slot = (pair0 + (b >> 1)) % C::NPAIR;
                        const uint32_t dst = sPair + slot * PAIR + (b & 1) * SLAB + z * 128;
                        for (int e = threadIdx.x; e < nz; e += 128) sts128(dst + e * 16, make_uint4(0u, 0u, 0u, 0u));
                    }
                }
                pair0 = (pair0 + NB) % C::NPAIR;
                tc::fence_async_smem();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::P_FULL));
            }
            // the segment's end: O^T / l, or the partial
            const bool whole = g.parts == 0;
            const int slot = slot_of(g, (int)blockIdx.x);
            if (r >= 0 && r < NR) {
                inv_s[r] = whole ? (l != 0.f ? 1.f / l : 0.f) : 1.f;
                if (!whole && valid) {
                    p.part_ml[((size_t)slot * NR + r) * 2] = m_ref;
                    p.part_ml[((size_t)slot * NR + r) * 2 + 1] = l;
                }
            }
            wait_pv(i);
            if (softmax_or(!ok)) {
                ok = false;
                return false;
            }
            tc::fence_after();
            const int col = warp * 32 + lane;  // this thread's latent column within a block of 128
            constexpr int W = NR < 32 ? NR : 32;
#pragma unroll 1
            for (int q = 0; q < NB * NR / W; ++q) {
                uint32_t o[W];
                if constexpr (W == 16) tc::ld16(tO + W * q, o);
                else tc::ld32(tO + W * q, o);
                tc::wait_ld();
                if (q == NB * NR / W - 1) {  // O^T read: the next segment's first PV may overwrite it
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::O_FREE));
                }
                const int blk = (W * q) / NR, h0 = (W * q) & (NR - 1);
                if (whole) {
                    // 2-byte stores, 64 bytes a warp and row: pairing lanes by shuffles to store 4 bytes was
                    // slower (shuffles share the path to shared memory with the MMA operands)
                    uint16_t* dst = static_cast<uint16_t*>(p.out) + (size_t)(g.row0 + h0) * DL + blk * 128 + col;
                    const uint32_t inv = smem_addr(inv_s) + (uint32_t)(h0 * 4);
                    uint4 iv[W / 4];
#pragma unroll
                    for (int e = 0; e < W / 4; ++e) iv[e] = lds128(inv + e * 16);
#pragma unroll
                    for (int e = 0; e < W; e += 2) {
                        const float a = __uint_as_float(e & 2 ? iv[e / 4].z : iv[e / 4].x);
                        const float b = __uint_as_float(e & 2 ? iv[e / 4].w : iv[e / 4].y);
                        const uint32_t v = F::pack_rn(__uint_as_float(o[e]) * a, __uint_as_float(o[e + 1]) * b);
                        if (h0 + e < g.rows) dst[(size_t)e * DL] = (uint16_t)v;
                        if (h0 + e + 1 < g.rows) dst[(size_t)(e + 1) * DL] = (uint16_t)(v >> 16);
                    }
                } else {
                    float* dst = p.part_o + ((size_t)slot * NR + h0) * DL + blk * 128 + col;
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (h0 + e < g.rows) dst[(size_t)e * DL] = __uint_as_float(o[e]);
                }
            }
            if (!whole) (g.tile == 0 ? begins : goes_on) = cut_of(g, (int)blockIdx.x);
            return true;
        });
        if (threadIdx.x == 0) {
            if (!ok) begins = goes_on = make_int4(0, 0, 0, 0);
            p.desc[blockIdx.x] = begins;
            p.desc[gridDim.x + blockIdx.x] = goes_on;
        }
    } else if (warp >= TMA_WARP) {
        // ------------------------------------------------------------ cache rows into the rings.  One warp a
        // pair slot of the tile and one for the rotary slot: a box of 16 rows moves 2 KB, so at small cache
        // blocks the issue of boxes, not the copies, would set the pace of a single warp (GB300: 36 boxes a
        // tile took one warp ~4000 cycles).  An elected lane issues from warp-uniform operands, as for the MMAs
        if (lane == 0) tma_prefetch_desc(&tmC);
        const uint64_t pol = l2_policy_evict_first();  // one unit a sequence: every row is read once
        const int b = warp - TMA_WARP;                          // pair of the tile; NB: the rotary slot
        const bool rope = b == NB;
        const int br = min(p.block_size, TK), nbox = TK / br;   // rows per box, boxes per slab
        const int slabs = rope ? 1 : 2, slots = rope ? C::NROPE : C::NPAIR;
        const int full0 = rope ? C::ROPE_FULL : C::PAIR_FULL, empty0 = rope ? C::ROPE_EMPTY : C::PAIR_EMPTY;
        const uint32_t el = elect_one();
        const uint32_t bytes = (uint32_t)(slabs * SLAB), ring = rope ? sRope : sPair;
        int n = rope ? 0 : b;    // slot number of this warp's next load, over the whole range
        const int step = rope ? 1 : NB;
        for_each_segment(p, start, [&](const Segment& g) -> bool {
            const int32_t* bt = p.block_tables + (size_t)g.c * p.max_blocks_per_seq;
            auto entry = [&](int tile) {  // block id of box `lane` of the tile; past the keys or invalid: zero fill
                const int t = tile * TK + lane * br;
                if (lane >= nbox || t >= g.keys) return p.num_blocks;
                const int e = __ldg(bt + (t >> p.block_log2));
                if (e < 0 || e >= p.num_blocks) {
                    flag_error(p.err, PA_DEVERR_BLOCK);
                    return p.num_blocks;
                }
                return e;
            };
            int blk = entry(g.tile);
            for (int u = 0; u < g.n; ++u, n += step, ++done) {
                const int tile = g.tile + u;
                const int nxt = u + 1 < g.n ? entry(tile + 1) : 0;
                const int slot = (int)uniform((uint32_t)(n % slots)), use = n / slots;
                if (use > 0 && !(ok = warp_wait(bar(empty0 + slot), (uint32_t)((use - 1) & 1), p.err))) return false;
                const uint32_t full = bar(full0 + slot), dst = ring + (uint32_t)slot * bytes;
                const int row = nbox == 1 ? (int)uniform((uint32_t)(tile * TK)) & (p.block_size - 1) : 0;  // a whole block, or 64 rows
                if (el) mbar_arrive_expect_tx(full, bytes);
                __syncwarp();
#pragma unroll 1
                for (int x = 0; x < nbox; ++x) {
                    const int e = __shfl_sync(0xffffffffu, blk, x);
                    tma_load_3d(el, dst + x * br * 128, &tmC, b * 128, row, e, full, pol);
                    if (!rope) tma_load_3d(el, dst + SLAB + x * br * 128, &tmC, b * 128 + 64, row, e, full, pol);
                }
                blk = nxt;
            }
            return true;
        });
    } else if (warp == Q_WARP && lane == 0) {
        // ------------------------------------------------------------ the units' query rows
        tma_prefetch_desc(&tmQ);
        int seg = 0;
        bool pending = false;
        for_each_segment(p, start, [&](const Segment& g) -> bool {
            if (seg > 0 && !(ok = mbar_wait(bar(C::Q_EMPTY), (uint32_t)((seg - 1) & 1), p.err))) return false;
            mbar_arrive_expect_tx(bar(C::Q_FULL), C::QSLABS * C::QSLAB);
#pragma unroll 1
            for (int s = 0; s < C::QSLABS; ++s) tma_load_2d(sQ + s * C::QSLAB, &tmQ, s * 64, g.row0, bar(C::Q_FULL));
            ++seg;
            pending = true;
            return true;
        });
        if (pending) (void)mbar_wait(bar(C::Q_FULL), (uint32_t)((seg - 1) & 1), p.err);
    } else if (warp == QK_WARP) {
        // ------------------------------------------------------------ QK issue.  QK and PV have an issuer
        // each: a tile's PV frees the ring for the tile after the next, so it must not queue behind the
        // next tile's QK, which waits for that tile's loads.  The whole warp walks the loop and one elected
        // lane issues, from descriptors that a shuffle makes warp-uniform: the instruction takes them from
        // uniform registers, and moving divergent ones there costs ~90 cycles an MMA
        constexpr uint32_t ID_QK = idesc(BF16, false, 64, TK);
        const uint64_t dq = tc::sdesc_sw128(sQ, 16, 1024), dkp = tc::sdesc_sw128(sPair, 16, 1024),
                       dkr = tc::sdesc_sw128(sRope, 16, 1024);
        const uint32_t el = elect_one(), tS = uniform(tmem);
        int i = 0, seg = 0, nk = 0, nr = 0;  // tiles, segments, pair and rotary slots read
        bool issued = false;
        for_each_segment(p, start, [&](const Segment& g) -> bool {
            if (!(ok = warp_wait(bar(C::Q_FULL), (uint32_t)(seg & 1), p.err))) return false;
            for (int u = 0; u < g.n; ++u, ++i) {
                const uint32_t dS = tS + uniform((uint32_t)(i & 1)) * 64;
                if (i >= 2 && !(ok = warp_wait(bar(C::S_EMPTY + (i & 1)), (uint32_t)(((i >> 1) - 1) & 1), p.err))) return false;
#pragma unroll
                for (int b = 0; b < NB; ++b, ++nk) {
                    const int slot = (int)uniform((uint32_t)(nk % C::NPAIR));
                    const uint64_t dk = dkp + (uint32_t)((slot * PAIR) >> 4);
                    if (!(ok = warp_wait(bar(C::PAIR_FULL + slot), (uint32_t)((nk / C::NPAIR) & 1), p.err))) return false;
                    tc::fence_after();
                    issued = true;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma(el, dS, dq + (uint32_t)(((2 * b + (kk >> 2)) * C::QSLAB + (kk & 3) * 32) >> 4),
                            dk + (uint32_t)(((kk >> 2) * SLAB + (kk & 3) * 32) >> 4), ID_QK, b > 0 || kk > 0);
                }
                const int rs = (int)uniform((uint32_t)(nr % C::NROPE));
                const uint64_t dk = dkr + (uint32_t)((rs * SLAB) >> 4);
                if (!(ok = warp_wait(bar(C::ROPE_FULL + rs), (uint32_t)((nr / C::NROPE) & 1), p.err))) return false;
                tc::fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma(el, dS, dq + (uint32_t)(((C::QSLABS - 1) * C::QSLAB + kk * 32) >> 4), dk + (uint32_t)((kk * 32) >> 4),
                        ID_QK, 1u);
                commit(el, bar(C::S_FULL + (i & 1)));
                commit(el, bar(C::ROPE_EMPTY + rs));
                if (u == g.n - 1) commit(el, bar(C::Q_EMPTY));
                ++nr;
            }
            ++seg;
            return true;
        });
        if (issued) {  // every MMA must be complete before TMEM is released
            commit(el, bar(C::DRAIN));
            (void)warp_wait(bar(C::DRAIN), 0, p.err);
        }
    } else if (warp == PV_WARP) {
        // ------------------------------------------------------------ PV issue: O^T += C^T P^T
        constexpr uint32_t ID_PV = idesc(BF16, true, 128, NR);
        const uint64_t dp = tc::sdesc_sw128(sP, 16, 1024), dv0 = tc::sdesc_sw128(sPair, SLAB, 1024);
        const uint32_t el = elect_one(), dO = uniform(tmem + C::O_COL);
        int i = 0, seg = 0, nv = 0;
        bool issued = false;
        for_each_segment(p, start, [&](const Segment& g) -> bool {
            // O^T of the segment before must have been read before the first product overwrites it
            if (seg > 0 && !(ok = warp_wait(bar(C::O_FREE), (uint32_t)((seg - 1) & 1), p.err))) return false;
            for (int u = 0; u < g.n; ++u, ++i) {
                const uint32_t acc = uniform(u > 0);
                const int slot0 = (int)uniform((uint32_t)(nv % C::NPAIR));
                if (!(ok = warp_wait(bar(C::P_FULL), (uint32_t)(i & 1), p.err))) return false;
                tc::fence_after();
                issued = true;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int slot = slot0 + b < C::NPAIR ? slot0 + b : slot0 + b - C::NPAIR;
                    const uint64_t dv = dv0 + (uint32_t)((slot * PAIR) >> 4);
#pragma unroll
                    for (int kk = 0; kk < TK / 16; ++kk)
                        mma(el, dO + b * NR, dv + (uint32_t)((kk * 2048) >> 4), dp + (uint32_t)((kk * 32) >> 4), ID_PV,
                            kk > 0 ? 1u : acc);
                    commit(el, bar(C::PAIR_EMPTY + slot));
                }
                commit(el, bar(C::PV_DONE));
                nv += NB;
            }
            ++seg;
            return true;
        });
        if (issued) {
            commit(el, bar(C::DRAIN + 1));
            (void)warp_wait(bar(C::DRAIN + 1), 0, p.err);
        }
    }
    tc::fence_before();
    // Every load is behind a wait of the QK issuer, every weight behind one of the PV issuer.  If all went well nothing is
    // in flight now; if some role's wait ran out, no copy may be left behind: the last ones of each ring
    if (__syncthreads_or(!ok) && warp >= TMA_WARP) {
        const bool rope = warp == TMA_WARP + NB;
        const int slots = rope ? C::NROPE : C::NPAIR, step = rope ? 1 : NB, full0 = rope ? C::ROPE_FULL : C::PAIR_FULL;
        for (int k = max(0, done - (slots + step - 1) / step); k < done; ++k) {
            const int m = (rope ? 0 : warp - TMA_WARP) + k * step;
            (void)warp_wait(bar(full0 + m % slots), (uint32_t)((m / slots) & 1), p.err);
        }
    }
    if (warp == QK_WARP) {
        tc::fence_after();
        tc::dealloc(tmem, C::TMEM_COLS);
    }
}

// Joins the partials of the units that the ranges' ends cut: out = sum_k 2^(m_k - max m) o_k / sum_k 2^(m_k - max m) l_k.
// A unit of few partials (the usual cut: two) is joined by the blocks of the range it starts in, a warp a row, DL / 32
// columns a lane.  One of many (few long contexts) by the blocks of all the ranges it spans, a block a row: its
// groups of DL / 4 threads every KG-th partial each, their sums added in order.  Fixed orders: the same inputs give
// the same bits.
template <bool BF16, int DL, int NR>
__global__ void __launch_bounds__(lat::merge_threads(NR)) latent_merge_kernel(const LatentParams p) {
    using F = F16x2<BF16>;
    constexpr int TH = lat::merge_threads(NR), NW = TH / 32, TG = DL / 4, KG = TH / TG, CV = DL / 128;
    constexpr int kFew = 8;
    __shared__ float4 acc[TH];
    __shared__ float wt[lat::MAX_CTAS];
    __shared__ float red[NW], l_s[1];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, range = (int)blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the next kernel of the step may start its launch; it waits for this grid before reading anything
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int4 cut[2] = {__ldcg(p.desc + range), __ldcg(p.desc + gridDim.x + range)};
    const int4 few = cut[0].x <= kFew ? cut[0] : make_int4(0, 0, 0, 0);
#pragma unroll 1
    for (int row = (int)blockIdx.y * 16 + warp; row < min(few.y, ((int)blockIdx.y + 1) * 16); row += NW) {
        const int4 u = few;
        float m = -INFINITY, l = 0.f;
        if (lane < u.x) {
            const int slot = 2 * (range + lane) + (lane == 0);
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + (size_t)slot * NR + row);
            m = ml.x;
            l = ml.y;
        }
        float4 a[CV] = {};
        float4 v[4][CV];
        auto fetch4 = [&](int k0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k0 + k >= u.x) break;
                const int slot = 2 * (range + k0 + k) + (k0 + k == 0);
#pragma unroll
                for (int c = 0; c < CV; ++c)
                    v[k][c] = __ldcg(reinterpret_cast<const float4*>(p.part_o + ((size_t)slot * NR + row) * DL) + lane + 32 * c);
            }
        };
        fetch4(0);  // in flight before their weights are known
        float mx = m;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mx = __shfl_sync(0xffffffffu, mx, 0);
        const float w = m == -INFINITY ? 0.f : ex2(m - mx);
        float lw = l != 0.f ? l * w : 0.f;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
        lw = __shfl_sync(0xffffffffu, lw, 0);
        for (int k0 = 0; k0 < u.x; k0 += 4) {
            if (k0 > 0) fetch4(k0);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k0 + k >= u.x) break;
                const float f = __shfl_sync(0xffffffffu, w, k0 + k);
                if (f == 0.f) continue;
#pragma unroll
                for (int c = 0; c < CV; ++c) {
                    a[c].x = fmaf(v[k][c].x, f, a[c].x);
                    a[c].y = fmaf(v[k][c].y, f, a[c].y);
                    a[c].z = fmaf(v[k][c].z, f, a[c].z);
                    a[c].w = fmaf(v[k][c].w, f, a[c].w);
                }
            }
        }
        const float inv = lw != 0.f ? 1.f / lw : 0.f;
        uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (size_t)(u.z + row) * DL);
#pragma unroll
        for (int c = 0; c < CV; ++c)
            dst[lane + 32 * c] = make_uint2(F::pack_rn(a[c].x * inv, a[c].y * inv), F::pack_rn(a[c].z * inv, a[c].w * inv));
    }
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const int4 u = which == 0 ? cut[0] : cut[1];
        const int parts = u.x, b = u.w;
        if (parts <= kFew) continue;
        auto slot_at = [&](int k) { return 2 * (b + k) + (k == 0); };
        for (int row = (range - b) * (int)gridDim.y + (int)blockIdx.y; row < u.y; row += parts * (int)gridDim.y) {
            float m = -INFINITY, l = 0.f;
            if (tid < parts) {
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + (size_t)slot_at(tid) * NR + row);
                m = ml.x;
                l = ml.y;
            }
            float mx = m;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (lane == 0) red[warp] = mx;
            __syncthreads();
            mx = red[0];
            for (int w = 1; w < NW; ++w) mx = fmaxf(mx, red[w]);
            const float w = m == -INFINITY ? 0.f : ex2(m - mx);
            if (tid < parts) wt[tid] = w;
            float lw = tid < parts && l != 0.f ? l * w : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
            __syncthreads();
            if (lane == 0) red[warp] = lw;
            __syncthreads();
            if (tid == 0) {
                float t = 0.f;
                for (int k = 0; k < NW; ++k) t += red[k];
                l_s[0] = t;
            }
            const int gidx = tid / TG, t = tid % TG;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int k = gidx; k < parts; k += KG) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part_o + ((size_t)slot_at(k) * NR + row) * DL) + t);
                const float f = wt[k];
                if (f != 0.f) {
                    a.x = fmaf(v.x, f, a.x);
                    a.y = fmaf(v.y, f, a.y);
                    a.z = fmaf(v.z, f, a.z);
                    a.w = fmaf(v.w, f, a.w);
                }
            }
            acc[tid] = a;
            __syncthreads();
            if (tid < TG) {
                for (int k = 1; k < KG; ++k) {
                    const float4 v = acc[k * TG + tid];
                    a.x += v.x;
                    a.y += v.y;
                    a.z += v.z;
                    a.w += v.w;
                }
                const float lt = l_s[0], inv = lt != 0.f ? 1.f / lt : 0.f;
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (size_t)(u.z + row) * DL + 4 * tid) =
                    make_uint2(F::pack_rn(a.x * inv, a.y * inv), F::pack_rn(a.z * inv, a.w * inv));
            }
            __syncthreads();
        }
    }
}

}  // namespace pa
