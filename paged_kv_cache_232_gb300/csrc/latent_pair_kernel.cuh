// latent_pair_kernel.cuh -- latent-cache attention (latent_kernel.cuh) for units of up to 128 query
// rows: a pair of CTAs (a cluster of two SMs) works one unit with cta_group::2 MMAs.
//
// One SM cannot hold it: 128 query rows x 576 columns are 147 KB of shared memory, and O takes all
// of TMEM.  Two SMs with 64 rows each would both read every cache row (twice the L2 traffic) at
// M = 64, half the tensor rate.  As a pair:
//  * Tiles of 128 tokens.  CTA r loads the whole rows of its 64 tokens (T_r) and holds 64 of the query
//    rows: S = Q K^T is one M = 128, N = 128 product of the pair.  CTA r gets its 64 rows of S, row h
//    in TMEM lanes h (tokens of T_0) and 64 + h (tokens of T_1), 64 columns.
//  * O^T = C^T P^T: CTA r accumulates the latent columns [r DL/2, (r + 1) DL/2) of all 128 rows
//    (M = 256, N = 128 over the pair, DL / 256 blocks of 128 columns), so it needs its half of the
//    columns for all 128 tokens.  The half for its own tokens is in place; of its rows the other half
//    is dead once S is done, and those slots are reloaded with its half of the peer's tokens.  A tile
//    buffer is DL / 128 pair slots A_0.. (columns below DL / 2), B_0.. (above): the product over T_0
//    reads A_b in both CTAs (CTA 0: own, CTA 1: reloaded), over T_1 B_b (CTA 0: reloaded, CTA 1: own),
//    at one offset in both as the paired instruction wants.  So two whole tile buffers fit beside the
//    64 query rows and the weights, and a cache row crosses L2 -> SM 1.4 times instead of twice.
//  * The leader (rank 0) issues every MMA; loads of both CTAs complete on its barriers, its commits
//    arrive on both.  Eight softmax warps: four threads a row, 32 tokens each; they agree on the row's
//    reference when some row outgrows it by 2^8 (a vote a tile, as in latent_kernel.cuh).  Each CTA
//    holds columns of O for all 128 rows, so rescale factors, and 1 / l at the end, go to both; four
//    more warps apply them and write the output, beside the next unit's softmax.
//
// What bounds it.  Prefill (rows from L2): shared-memory bandwidth.  A tile's products are 2176 cycles of
// tensor work an SM and ~2750 of operand reads and tile writes; measured ~3000 a tile, 890..945 us (by box) for 4
// chunks of 512 tokens at 128 heads over 0..4096 cached ones (1.31 PFLOP: 1.39..1.47 PFLOP/s, 0.71..0.75 of the
// measured burst rate, 0.81..0.85 of the sustained).  Decode at 128 heads is balanced between memory and tensor
// cores: ~3200 cycles a tile in steady state (the copy rate), 136..148 us for 128 sequences of 1K..8K tokens (0.70..0.76
// of the floor): ~104 us of tiles, ~12 of start and merge; the rest is not accounted for (units' ends, most likely: no
// load looks past one).  Steps on the way (prefill / decode, us, each of its own build): two independent CTAs of 64
// rows 3360 / 322; this pair with cluster-scope arrivals and waits, 10500 cycles a tile, 3750 / 397; without them, MMA
// issue predicated in a converged warp, two waits a role and tile, 1081 / 188; ranges cut by cost and rows kept in
// L2 for the second read 875 / 164; the tile after the next prefetched into L2 870 / 143.  Taken out of this build:
// the units' own cost in the cut, 905 -> 1413 / 136 -> 138.
#pragma once

#include "latent_kernel.cuh"

namespace pa {
namespace latp {

using lat::PAIR;
using lat::SLAB;
constexpr int TK = 128;                 // tokens per tile
constexpr int NR = 128;                 // query rows per unit
constexpr int SOFTMAX_WARPS = 8, CORR_WARP = 8, QK_WARP = 12, PV_WARP = 13, Q_WARP = 14, X_WARP = 15, ROPE_WARP = 16,
              TMA_WARP = 17, LOADERS = 2;
// To the rescale warps: a segment's last PV is issued; or (below it) bits 0, 1: whose rows to rescale, bit 2: the
// tile's parity, bit 3: its phase on T_FULL
constexpr uint32_t CMD_END = 16;

template <int DL>
struct Cfg {
    static_assert(DL == 256 || DL == 512, "latent columns");
    static constexpr int NP = DL / 128;                 // pair slots of a tile buffer
    static constexpr int NB = DL / 256;                 // blocks of 128 latent columns a CTA accumulates
    static constexpr int THREADS = (TMA_WARP + LOADERS) * 32;
    static constexpr int SLABS_EACH = 2 * NP / LOADERS;   // slabs of a tile a loader warp brings
    static constexpr int QSLABS = DL / 64 + 1;
    static constexpr int Q_OFF = 0;                     // 64 rows x 9 (5) slabs
    static constexpr int P_OFF = QSLABS * SLAB;         // two slabs: 64 rows x 64 tokens of T_0, of T_1
    static constexpr int BUF_OFF = P_OFF + 2 * SLAB;    // two tile buffers
    static constexpr int ROPE_OFF = BUF_OFF + 2 * NP * PAIR;  // one slot: it is free again after the first MMAs of S
    static constexpr int BAR_OFF = ROPE_OFF + SLAB;
    // barriers (buffer, tile or segment parity where there are two).  On the leader alone: FULL (a tile's own rows, both
    // CTAs'), ROPE_FULL, X_FULL (the reloaded ones), Q_FULL, S_EMPTY, P_FULL, CORR (a rescale is done), O_FREE, SEEN (the
    // peer's T_FULL is complete), DRAIN; on both: the others.  T_FULL: a tile's rescale flags and factors are there;
    // F_FULL: a segment's 1 / l; CMD: the next command to the rescale warps; X_TAIL: see the loaders
    static constexpr int FULL = 0, X_FULL = 2, EMPTY = 4, ROPE_FULL = 6, ROPE_EMPTY = 7, Q_FULL = 8, Q_EMPTY = 9,
                         S_FULL = 10, S_EMPTY = 12, P_FULL = 14, PV_DONE = 15, CORR = 16, O_FREE = 17, T_FULL = 18,
                         F_FULL = 20, CMD = 22, X_TAIL = 23, SEEN = 24, DRAIN = 26, NUM_BARS = 28;
    static constexpr int MISC_OFF = (BAR_OFF + NUM_BARS * 8 + 15) & ~15;  // start record, TMEM address, rescale flags, command
    static constexpr int EXCH_OFF = MISC_OFF + 80;                        // [4][64] row maxima or sums; scan scratch before
    static constexpr int ALPHA_OFF = EXCH_OFF + 4 * 64 * 4;               // [2][128] by tile parity
    static constexpr int INV_OFF = ALPHA_OFF + 2 * NR * 4;                // [128]
    static constexpr int USED_BYTES = INV_OFF + NR * 4;
    static_assert(USED_BYTES <= 227 * 1024, "shared memory per CTA");
    // + alignment slack, as far as it goes (512 latent columns: 208 bytes)
    static constexpr int SMEM_BYTES = USED_BYTES + 1024 <= 227 * 1024 ? USED_BYTES + 1024 : 227 * 1024;
    static_assert(EXCH_OFF % 16 == 0 && THREADS / 32 * 8 <= 1024, "scratch");
    static constexpr uint32_t O_COL = 128;              // two S buffers of 64 columns, then NB x 128 of O^T
    static constexpr uint32_t TMEM_COLS = 512;
};

template <int N>
struct Int {
    static constexpr int value = N;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// address in the cluster's shared window of CTA `rank`'s counterpart of a shared address
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrivals and waits keep the default CTA scope: cluster-scope release and acquire cost ~700 cycles each here,
// several a tile.  What crosses the pair does not need them: the weights are behind a proxy fence and read by
// the tensor cores, TMEM accesses are behind tcgen05 fences, and values the peer's threads read travel by
// st.async, whose completion on the barrier follows the data, for a reader that waits for that barrier.  So every
// reader waits for the barrier of its own CTA that counts what it reads:
//  * flags: the PV issuer, T_FULL of the tile.  alpha: the rescale warps, T_FULL of the tile that the command names.
//    1 / l: the rescale warps, F_FULL of the segment.  The command: CMD.
// and no barrier is used again before its phase is known to be complete in both CTAs, nor its data overwritten
// before they are read:
//  * T_FULL and alpha of a tile are next used two tiles on, by softmax warps that have seen this tile's PV.  The PV
//    was issued behind T_FULL of the leader, behind SEEN, which a warp of the peer gives once its own T_FULL is
//    complete (on tiles without a rescale nobody else there waits for it), and behind the rescale (CORR).
//  * 1 / l and F_FULL of a segment: the next segment's first PV is issued behind O_FREE, which the rescale warps give
//    once they have read; the softmax warps see a PV of the next segment before they send again.
//  * CMD: the next command follows CORR or O_FREE.
// Nothing is in flight when a CTA ends: its T_FULL, F_FULL and CMD have all been waited for there.
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
__device__ __forceinline__ void arrive_expect_at(uint32_t cluster_bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_bar), "r"(bytes) : "memory");
}
// a value into a CTA's shared memory, counted (4 bytes) on a barrier of that CTA
__device__ __forceinline__ void send_u32(uint32_t addr, uint32_t v, uint32_t cluster_bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(addr), "r"(v),
                 "r"(cluster_bar)
                 : "memory");
}
// loads into this CTA, counted on a barrier of the pair's leader
__device__ __forceinline__ void load_3d(uint32_t el, uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                        uint32_t bar, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %7, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy), "r"(el)
        : "memory");
}
// rows of the cache into L2 (16-byte aligned, a multiple of 16 bytes)
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
// Issue and commits are predicated on `el` (the warp's elected lane) rather than branched around: the issuing warp
// stays converged, so that descriptors are formed once for the warp.
__device__ __forceinline__ void mma(uint32_t el, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
        : "memory");
}
// arrive on the barrier at this offset in both CTAs (commit2) or in the leader (commit1) once the MMAs
// issued so far are complete
__device__ __forceinline__ void commit2(uint32_t el, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"((uint16_t)3), "r"(el)
        : "memory");
}
__device__ __forceinline__ void commit1(uint32_t el, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(el)
        : "memory");
}
__device__ __forceinline__ bool softmax_or(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 1, 256;" ::: "memory"); }

}  // namespace latp

template <bool BF16, int DL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(latp::Cfg<DL>::THREADS, 1)
latent_pair_kernel(const LatentParams p, const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmQ) {
    using namespace latp;
    using lat::elect_one;
    using lat::for_each_segment;
    using lat::Segment;
    using lat::Start;
    using lat::uniform;
    using lat::warp_wait;
    using C = Cfg<DL>;
    using F = F16x2<BF16>;
    constexpr int NB = C::NB, NP = C::NP;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    // The tiles' swizzle and the operand descriptors need a base of 1024 bytes' alignment.  The launch gives one (the kernel
    // has no static shared memory); should that change, the base moves up, or the kernel gives up where it cannot
    const uint32_t skip = (0u - smem_addr(smem_raw)) & 1023u;
    const bool aligned = skip + C::USED_BYTES <= C::SMEM_BYTES;
    unsigned char* smem = smem_raw + (aligned ? skip : 0u);
    const uint32_t sbase = smem_addr(smem);
    const uint32_t sQ = sbase + C::Q_OFF, sP = sbase + C::P_OFF, sBuf = sbase + C::BUF_OFF, sRope = sbase + C::ROPE_OFF;
    auto bar = [&](int i) { return sbase + C::BAR_OFF + 8u * (uint32_t)i; };
    Start* rec = reinterpret_cast<Start*>(smem + C::MISC_OFF);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::MISC_OFF + 32);
    volatile uint32_t* flag_s = reinterpret_cast<volatile uint32_t*>(smem + C::MISC_OFF + 48);  // [tile parity][rank]
    volatile uint32_t* cmd_s = flag_s + 4;
    float* exch = reinterpret_cast<float*>(smem + C::EXCH_OFF);
    const uint32_t alpha_a = sbase + C::ALPHA_OFF, inv_a = sbase + C::INV_OFF, flag_a = sbase + C::MISC_OFF + 48,
                   cmd_a = flag_a + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), peer = rank ^ 1u;
    const int range = (int)(blockIdx.x >> 1), ranges = (int)(gridDim.x >> 1);
    auto lead = [&](int i) { return map_to(bar(i), 0); };  // a barrier of the leader

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NUM_BARS; ++i) {
            const int n = i == C::S_EMPTY || i == C::S_EMPTY + 1 || i == C::P_FULL ? 2 * SOFTMAX_WARPS
                          : i == C::CORR || i == C::O_FREE                         ? 8
                          : i == C::FULL || i == C::FULL + 1                       ? LOADERS
                          : (i >= C::T_FULL && i < C::CMD) || i == C::X_FULL || i == C::X_FULL + 1 ? 2
                                                                                   : 1;
            mbar_init(bar(i), n);
        }
        fence_barrier_init();
        if (!aligned) flag_error(p.err, PA_DEVERR_SMEM);
    }
    if (warp == QK_WARP) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(const_cast<uint32_t*>(tmem_slot))),
                     "r"(C::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Start start = lat::find_start<C::THREADS>(p, range, ranges, reinterpret_cast<long long*>(exch), rec);
    if (!aligned) start.count = 0;
    tc::fence_before();
    cluster_sync();  // both CTAs' barriers and TMEM are ready
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;          // none of this thread's waits has run out
    int loaded = 0;          // loader warps: tiles loaded
    bool tail_out = false;   // X_WARP: copies counted on X_TAIL are in flight

    if (warp < SOFTMAX_WARPS) {
        // ------------------------------------------------------------ softmax: thread = (row, 32 tokens)
        const int quarter = warp & 3, ch = warp >> 2, th = quarter >> 1;
        const int hr = (quarter & 1) * 32 + lane;              // row of this CTA's 64
        const int R = 64 * (int)rank + hr;                     // row of the unit
        const int part = th * 2 + ch;
        const bool speaks = part == 0;                         // warps 0 and 1: one thread a row
        const uint32_t tS = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(ch * 32);
        const float sc = p.qk_scale_log2;
        const uint32_t p_full = lead(C::P_FULL);
        auto announce = [&](int b, uint32_t bytes) {  // `bytes` come to both CTAs on their barrier b
            arrive_expect_at(map_to(bar(b), rank), bytes);
            arrive_expect_at(map_to(bar(b), peer), bytes);
        };
        auto send = [&](uint32_t addr, uint32_t v, int b) {
            send_u32(map_to(addr, rank), v, map_to(bar(b), rank));
            send_u32(map_to(addr, peer), v, map_to(bar(b), peer));
        };
        int i = 0, pv_seen = 0, seg = 0;
        int4 begins = make_int4(0, 0, 0, 0), goes_on = begins;  // the units cut at the range's end and at its start
        auto wait_pv = [&](int n) {
            while (pv_seen < n) {
                ok = warp_wait(bar(C::PV_DONE), (uint32_t)(pv_seen & 1), p.err) && ok;
                ++pv_seen;
            }
        };
        for_each_segment(p, start, [&](const Segment& g) -> bool {
            const bool valid = R < g.rows;
            const int lim = valid ? g.ctx + g.j * p.tb + R / p.n_heads : -1;
            // the smallest limit of the unit's rows.  Rows past them (other tokens' queries) are not masked: rows are
            // independent in both products, theirs are never written and never ask for a rescale
            const int lim_min = g.ctx + g.j * p.tb;
            float m_ref = -INFINITY, l = 0.f;
            for (int u = 0; u < g.n; ++u, ++i) {
                const int kbase = (g.tile + u) * TK + 64 * th + 32 * ch;
                ok = warp_wait(bar(C::S_FULL + (i & 1)), (uint32_t)((i >> 1) & 1), p.err) && ok;
                tc::fence_after();
                float x[32];
                {
                    uint32_t s[32];
                    tc::ld32(tS + (uint32_t)((i & 1) * 64), s);
                    tc::wait_ld();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_at(lead(C::S_EMPTY + (i & 1)));
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 v = __fmul2_rn(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), make_float2(sc, sc));
                        x[e] = v.x;
                        x[e + 1] = v.y;
                    }
                }
                if (kbase + 31 > lim_min) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (kbase + e > lim) x[e] = -INFINITY;
                }
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 32; ++e) m4[e & 3] = fmaxf(m4[e & 3], x[e]);
                const float mx = valid ? fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) : -INFINITY;
                const bool first = u == 0;
                uint32_t rescale = 0;
                if (softmax_or(!ok || first || mx > m_ref + 8.f)) {
                    if (softmax_or(!ok)) {  // some warp's wait ran out: all leave together
                        ok = false;
                        return false;
                    }
                    exch[part * 64 + hr] = mx;
                    softmax_sync();
                    const float mr = fmaxf(fmaxf(exch[hr], exch[64 + hr]), fmaxf(exch[128 + hr], exch[192 + hr]));
                    float a = 1.f;
                    if (mr > m_ref) {
                        a = m_ref == -INFINITY ? 1.f : ex2(m_ref - mr);
                        m_ref = mr;
                        l *= a;
                    }
                    if (!first) {
                        rescale = 1;
                        if (speaks)  // to both CTAs: each holds columns of O of this row
                            send(alpha_a + (uint32_t)(((i & 1) * NR + R) * 4), __float_as_uint(a), C::T_FULL + (i & 1));
                    }
                }
                if (threadIdx.x == 0) {  // whether this tile rescales is settled for this CTA's rows
                    const int b = C::T_FULL + (i & 1);
                    announce(b, rescale ? 4 + 64 * 4 : 4);
                    send(flag_a + (uint32_t)(((i & 1) * 2 + (int)rank) * 4), rescale, b);
                }
                __syncwarp();
                const float mu = m_ref == -INFINITY ? 0.f : m_ref - lat::kShift<BF16>;
                uint32_t w[16];
                float2 ls = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 v = fadd2(make_float2(x[2 * e], x[2 * e + 1]), make_float2(-mu, -mu));
                    w[e] = F::pack_rn(ex2(v.x), ex2(v.y));
                    ls = fadd2(ls, F::unpack(w[e]));
                }
                l += ls.x + ls.y;
                wait_pv(i);  // the weights' buffer is free
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    sts128(sP + (uint32_t)(th * SLAB) + swz128(hr, 4 * ch + c),
                           make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]));
                const int own0 = (g.tile + u) * TK + 64 * (int)rank;
                if (own0 + 64 > g.keys) {
                    // this CTA's rows past the keys may hold anything (their weights are 0, but 0 * NaN is NaN): zero the
                    // columns that PV reads (S, which read the rows too, is complete)
                    const int z = max(g.keys - own0, 0), nz = (64 - z) * 8;
                    for (int b = 0; b < 2 * NB; ++b) {
                        const uint32_t dst = sBuf + (uint32_t)(((i & 1) * NP + (int)rank * NB) * PAIR + b * SLAB + z * 128);
                        for (int e = (int)threadIdx.x; e < nz; e += 256) sts128(dst + e * 16, make_uint4(0u, 0u, 0u, 0u));
                    }
                }
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) arrive_at(p_full);
            }
            // the segment's end: the rows' sums to the rescale warps of both CTAs, which write the output
            const bool whole = g.parts == 0;
            const int slot = lat::slot_of(g, range);
            softmax_sync();  // (exch: the last tile's maxima have been read)
            exch[part * 64 + hr] = l;
            softmax_sync();
            if (g.n == 1) wait_pv(i);  // 1 / l of the segment before has been read: this one's PV came after that
            if (speaks) {
                const float lr = (exch[hr] + exch[64 + hr]) + (exch[128 + hr] + exch[192 + hr]);
                const float inv = whole ? (lr != 0.f ? 1.f / lr : 0.f) : 1.f;
                const int b = C::F_FULL + (seg & 1);
                if (threadIdx.x == 0) announce(b, 64 * 4);
                __syncwarp();
                send(inv_a + (uint32_t)(R * 4), __float_as_uint(inv), b);
                if (!whole && valid) {
                    p.part_ml[((size_t)slot * NR + R) * 2] = m_ref;
                    p.part_ml[((size_t)slot * NR + R) * 2 + 1] = lr;
                }
            }
            if (!whole) (g.tile == 0 ? begins : goes_on) = lat::cut_of(g, range);
            ++seg;
            return true;
        });
        if (threadIdx.x == 0 && rank == 0) {
            if (!ok) begins = goes_on = make_int4(0, 0, 0, 0);
            p.desc[range] = begins;
            p.desc[ranges + range] = goes_on;
        }
    } else if (warp < CORR_WARP + 4) {
        // ------------------------------------------------------------ rescale of O^T and the output: lane = latent
        // column.  Commands come from the PV issuer: see CMD_END
        const int quarter = warp & 3;
        const uint32_t tO = tmem + ((uint32_t)(quarter * 32) << 16) + C::O_COL;
        const uint32_t corr = lead(C::CORR), o_free = lead(C::O_FREE);
        const int col = (int)rank * (DL / 2) + quarter * 32 + lane;  // of block 0
        int i = 0, cmds = 0, seg = 0;
        for_each_segment(p, start, [&](const Segment& g) -> bool {
            while (true) {
                if (!(ok = warp_wait(bar(C::CMD), (uint32_t)(cmds & 1), p.err))) return false;
                ++cmds;
                const uint32_t cmd = *cmd_s;
                if (cmd == CMD_END) break;
                const int par = (int)((cmd >> 2) & 1);
                // this CTA's copies of the factors: the leader's command says nothing about the peer's
                if (!(ok = warp_wait(bar(C::T_FULL + par), (cmd >> 3) & 1, p.err))) return false;
                tc::fence_after();
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    if (!((cmd >> c) & 1)) continue;
                    const uint32_t al = alpha_a + (uint32_t)((par * NR + 64 * c) * 4);
#pragma unroll 1
                    for (int q = 0; q < NB * 4; ++q) {  // 16 of CTA c's 64 rows in block q / 4
                        const uint32_t at = tO + (uint32_t)((q >> 2) * NR + 64 * c + (q & 3) * 16);
                        uint32_t o[16];
                        tc::ld16(at, o);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * lat::lds_f32(al + (uint32_t)(((q & 3) * 16 + e) * 4)));
                        tc::st16(at, o);
                    }
                    tc::wait_st();
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) arrive_at(corr);
            }
            const bool whole = g.parts == 0;
            const int slot = lat::slot_of(g, range);
            i += g.n;
            if (!(ok = warp_wait(bar(C::F_FULL + (seg & 1)), (uint32_t)((seg >> 1) & 1), p.err))) return false;
            if (!(ok = warp_wait(bar(C::PV_DONE), (uint32_t)((i - 1) & 1), p.err))) return false;
            tc::fence_after();
#pragma unroll 1
            for (int q = 0; q < NB * 4; ++q) {
                const int h0 = (q & 3) * 32, b = q >> 2;
                uint32_t o[32];
                tc::ld32(tO + (uint32_t)(b * NR + h0), o);
                uint4 iv[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) iv[e] = lds128(inv_a + (uint32_t)(h0 * 4 + e * 16));
                tc::wait_ld();
                if (q == NB * 4 - 1) {  // O^T and 1 / l read: the next segment may go on
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_at(o_free);
                }
                if (whole) {
                    uint16_t* dst = static_cast<uint16_t*>(p.out) + (size_t)(g.row0 + h0) * DL + b * 128 + col;
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float fa = __uint_as_float(e & 2 ? iv[e / 4].z : iv[e / 4].x);
                        const float fb = __uint_as_float(e & 2 ? iv[e / 4].w : iv[e / 4].y);
                        const uint32_t v = F::pack_rn(__uint_as_float(o[e]) * fa, __uint_as_float(o[e + 1]) * fb);
                        if (h0 + e < g.rows) dst[(size_t)e * DL] = (uint16_t)v;
                        if (h0 + e + 1 < g.rows) dst[(size_t)(e + 1) * DL] = (uint16_t)(v >> 16);
                    }
                } else {
                    float* dst = p.part_o + ((size_t)slot * NR + h0) * DL + b * 128 + col;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (h0 + e < g.rows) dst[(size_t)e * DL] = __uint_as_float(o[e]);
                }
            }
            ++seg;
            return true;
        });
    } else if (warp >= X_WARP) {
        // ------------------------------------------------------------ cache rows.  Warps TMA_WARP + k: the k-th half
        // of the slabs of this CTA's 64 tokens; ROPE_WARP: their rotary part; X_WARP: after a tile's S, this CTA's columns
        // of the peer's tokens
        if (lane == 0) tma_prefetch_desc(&tmC);
        // both CTAs read each row's values: evict-first would lose them in between (decode of 128 sequences at 128 heads
        // 174 us, 167 with this)
        const uint64_t pol = l2_policy_evict_last();
        const uint32_t el = elect_one();
        const int br = min(p.block_size, 64), nbox = 64 / br;
        const bool extra = warp == X_WARP, rope = warp == ROPE_WARP;
        const int slab0 = C::SLABS_EACH * (warp - TMA_WARP); // first slab of this warp
        const int half = extra ? (int)peer : (int)rank;      // whose tokens
        int i = 0, tails = 0;
        for_each_segment(p, start, [&](const Segment& g) -> bool {
            const int32_t* bt = p.block_tables + (size_t)g.c * p.max_blocks_per_seq;
            auto entry = [&](int tile) {
                const int t = tile * TK + half * 64 + lane * br;
                if (lane >= nbox || t >= g.keys) return p.num_blocks;
                const int e = ld_global(bt + (t >> p.block_log2));
                if (e < 0 || e >= p.num_blocks) {
                    flag_error(p.err, PA_DEVERR_BLOCK);
                    return p.num_blocks;
                }
                return e;
            };
            int blk = entry(g.tile), nxt = g.n > 1 ? entry(g.tile + 1) : p.num_blocks;
            for (int u = 0; u < g.n; ++u, ++i) {
                const int tile = g.tile + u;
                const int nxt2 = u + 2 < g.n ? entry(tile + 2) : p.num_blocks;
                const uint32_t buf = uniform((uint32_t)(i & 1)), dst = sBuf + buf * (NP * PAIR);
                const int first = (int)uniform((uint32_t)(tile * TK + half * 64));  // of the 64 tokens
                const int row = nbox == 1 ? first & (p.block_size - 1) : 0;  // a box is a whole block, or 64 rows of one
                // boxes of N slabs from column c0, `to` onwards, counted on barrier fb
                auto load = [&](auto slabs, uint32_t to, int c0, uint32_t fb) {
                    constexpr int N = decltype(slabs)::value;
#pragma unroll 1
                    for (int x = 0; x < nbox; ++x) {
                        const int e = __shfl_sync(0xffffffffu, blk, x);
                        const uint32_t at = to + (uint32_t)(x * br * 128);
#pragma unroll
                        for (int s = 0; s < N; ++s) load_3d(el, at + s * SLAB, &tmC, c0 + 64 * s, row, e, fb, pol);
                    }
                };
                if (extra) {
                    const uint32_t to = dst + (uint32_t)((rank == 0 ? NB : 0) * PAIR);
                    const bool tail = first + 64 > g.keys;
                    // with rows past the keys: wait for the copies here, zero those rows, then hand over
                    const uint32_t fb = tail ? map_to(bar(C::X_TAIL), rank) : lead(C::X_FULL + buf);
                    if (!(ok = warp_wait(bar(C::S_FULL + buf), (uint32_t)((i >> 1) & 1), p.err))) return false;
                    tail_out = tail;
                    if (el) arrive_expect_at(fb, NB * PAIR);
                    __syncwarp();
                    load(Int<2 * NB>{}, to, (int)rank * (DL / 2), fb);
                    if (tail) {
                        if (!(ok = warp_wait(bar(C::X_TAIL), (uint32_t)(tails & 1), p.err))) return false;
                        ++tails;
                        tail_out = false;
                        const int z = max(g.keys - first, 0), nz = (64 - z) * 8;
                        for (int b2 = 0; b2 < 2 * NB; ++b2)
                            for (int e = lane; e < nz; e += 32)
                                sts128(to + (uint32_t)(b2 * SLAB + z * 128 + e * 16), make_uint4(0u, 0u, 0u, 0u));
                        tc::fence_async_smem();
                        __syncwarp();
                        if (lane == 0) arrive_at(lead(C::X_FULL + buf));
                    }
                    // these tokens of the tile after the next into L2 (the two CTAs' loaders cover both halves): its loads
                    // start once this tile's PV is done, and their DRAM latency would be on the way from tile to tile
                    if (p.stream_once && nxt2 < p.num_blocks)
                        prefetch_l2(static_cast<const uint16_t*>(p.cache) +
                                        ((int64_t)nxt2 * p.block_size + row) * (DL + lat::ROPE),
                                    (uint32_t)(br * (DL + lat::ROPE) * 2));
                    __syncwarp();
                } else if (rope) {
                    if (i > 0 && !(ok = warp_wait(bar(C::ROPE_EMPTY), (uint32_t)((i - 1) & 1), p.err))) return false;
                    if (rank == 0 && el) mbar_arrive_expect_tx(bar(C::ROPE_FULL), 2 * SLAB);  // both CTAs'
                    __syncwarp();
                    load(Int<1>{}, sRope, DL, lead(C::ROPE_FULL));
                } else {
                    if (i > 1 && !(ok = warp_wait(bar(C::EMPTY + buf), (uint32_t)(((i >> 1) - 1) & 1), p.err))) return false;
                    if (rank == 0 && el) mbar_arrive_expect_tx(bar(C::FULL + buf), 2 * C::SLABS_EACH * SLAB);  // both CTAs'
                    __syncwarp();
                    load(Int<C::SLABS_EACH>{}, dst + (uint32_t)(slab0 * SLAB), 64 * slab0, lead(C::FULL + buf));
                }
                blk = nxt;
                nxt = nxt2;
            }
            return true;
        });
        if (tail_out) (void)warp_wait(bar(C::X_TAIL), (uint32_t)(tails & 1), p.err);  // ran out: once more
        loaded = i;
    } else if (warp == Q_WARP) {
        // ------------------------------------------------------------ this CTA's 64 query rows of the unit
        if (lane == 0) tma_prefetch_desc(&tmQ);
        int seg = 0;
        bool pending = false;
        for_each_segment(p, start, [&](const Segment& g) -> bool {
            if (seg > 0 && !(ok = warp_wait(bar(C::Q_EMPTY), (uint32_t)((seg - 1) & 1), p.err))) return false;
            const uint32_t full = lead(C::Q_FULL);
            if (rank == 0 && elect_one()) mbar_arrive_expect_tx(bar(C::Q_FULL), (uint32_t)(2 * C::QSLABS * SLAB));
            __syncwarp();
            const int row = (int)uniform((uint32_t)(g.row0 + 64 * (int)rank));
            if (elect_one()) {
#pragma unroll 1
                for (int s = 0; s < C::QSLABS; ++s) load_2d(sQ + s * SLAB, &tmQ, s * 64, row, full);
            }
            __syncwarp();
            ++seg;
            pending = true;
            return true;
        });
        if (pending && rank == 0) (void)warp_wait(bar(C::Q_FULL), (uint32_t)((seg - 1) & 1), p.err);
    } else if (warp == QK_WARP && rank == 0) {
        // ------------------------------------------------------------ S = Q K^T over the pair (rotary part first:
        // its slot is the only one)
        constexpr uint32_t ID_QK = lat::idesc(BF16, false, 128, TK);
        const uint64_t dq = tc::sdesc_sw128(sQ, 16, 1024), dk0 = tc::sdesc_sw128(sBuf, 16, 1024),
                       dkr = tc::sdesc_sw128(sRope, 16, 1024);
        const uint32_t el = elect_one(), tS = uniform(tmem);
        int i = 0, seg = 0;
        bool issued = false;
        for_each_segment(p, start, [&](const Segment& g) -> bool {
            if (!(ok = warp_wait(bar(C::Q_FULL), (uint32_t)(seg & 1), p.err))) return false;
            for (int u = 0; u < g.n; ++u, ++i) {
                const uint32_t buf = uniform((uint32_t)(i & 1)), dS = tS + buf * 64;
                const uint64_t dk = dk0 + ((buf * (NP * PAIR)) >> 4);
                if (i >= 2 && !(ok = warp_wait(bar(C::S_EMPTY + buf), (uint32_t)(((i >> 1) - 1) & 1), p.err))) return false;
                if (!(ok = warp_wait(bar(C::ROPE_FULL), (uint32_t)(i & 1), p.err))) return false;
                tc::fence_after();
                issued = true;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma(el, dS, dq + (uint32_t)(((C::QSLABS - 1) * SLAB + kk * 32) >> 4), dkr + (uint32_t)((kk * 32) >> 4), ID_QK,
                        kk > 0);
                commit2(el, bar(C::ROPE_EMPTY));
                if (!(ok = warp_wait(bar(C::FULL + buf), (uint32_t)((i >> 1) & 1), p.err))) return false;
                tc::fence_after();
#pragma unroll
                for (int kk = 0; kk < 4 * (C::QSLABS - 1); ++kk)
                    mma(el, dS, dq + (uint32_t)(((kk >> 2) * SLAB + (kk & 3) * 32) >> 4),
                        dk + (uint32_t)(((kk >> 2) * SLAB + (kk & 3) * 32) >> 4), ID_QK, 1u);
                commit2(el, bar(C::S_FULL + buf));
                if (u == g.n - 1) commit2(el, bar(C::Q_EMPTY));
            }
            ++seg;
            return true;
        });
        if (issued) {
            commit1(el, bar(C::DRAIN));
            (void)warp_wait(bar(C::DRAIN), 0, p.err);
        }
    } else if (warp == PV_WARP && rank == 0) {
        // ------------------------------------------------------------ O^T += C^T P^T over the pair
        constexpr uint32_t ID_PV = lat::idesc(BF16, true, 256, NR);
        const uint64_t dp = tc::sdesc_sw128(sP, 16, 1024), dv0 = tc::sdesc_sw128(sBuf, SLAB, 1024);
        const uint32_t el = elect_one(), dO = uniform(tmem + C::O_COL);
        int i = 0, seg = 0, corrs = 0;
        bool issued = false;
        auto command = [&](uint32_t c) {  // to the rescale warps of both CTAs
            if (lane < 2) {
                const uint32_t b = map_to(bar(C::CMD), (uint32_t)lane);
                arrive_expect_at(b, 4);
                send_u32(map_to(cmd_a, (uint32_t)lane), c, b);
            }
            __syncwarp();
        };
        for_each_segment(p, start, [&](const Segment& g) -> bool {
            if (seg > 0 && !(ok = warp_wait(bar(C::O_FREE), (uint32_t)((seg - 1) & 1), p.err))) return false;
            for (int u = 0; u < g.n; ++u, ++i) {
                const uint32_t acc = uniform(u > 0), buf = uniform((uint32_t)(i & 1));
                const uint64_t dv = dv0 + ((buf * (NP * PAIR)) >> 4);
                if (!(ok = warp_wait(bar(C::T_FULL + buf), (uint32_t)((i >> 1) & 1), p.err))) return false;
                const uint32_t flags = flag_s[2 * buf] | (flag_s[2 * buf + 1] << 1);
                if (flags) {  // O^T is rescaled once it holds every tile before this one
                    if (!(ok = warp_wait(bar(C::PV_DONE), (uint32_t)((i - 1) & 1), p.err))) return false;
                    command(flags | (buf << 2) | ((uint32_t)((i >> 1) & 1) << 3));
                    if (!(ok = warp_wait(bar(C::CORR), (uint32_t)(corrs & 1), p.err))) return false;
                    ++corrs;
                }
                if (!(ok = warp_wait(bar(C::X_FULL + buf), (uint32_t)((i >> 1) & 1), p.err))) return false;
                if (!(ok = warp_wait(bar(C::SEEN + buf), (uint32_t)((i >> 1) & 1), p.err))) return false;
                if (!(ok = warp_wait(bar(C::P_FULL), (uint32_t)(i & 1), p.err))) return false;
                tc::fence_after();
                issued = true;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)  // T_0: slots A, then T_1: slots B
                        mma(el, dO + b * NR, dv + (uint32_t)(((kk >> 2) * NB * PAIR + b * PAIR + (kk & 3) * 2048) >> 4),
                            dp + (uint32_t)(((kk >> 2) * SLAB + (kk & 3) * 32) >> 4), ID_PV, kk > 0 ? 1u : acc);
                commit2(el, bar(C::EMPTY + buf));
                commit2(el, bar(C::PV_DONE));
            }
            command(CMD_END);
            ++seg;
            return true;
        });
        if (issued) {
            commit1(el, bar(C::DRAIN + 1));
            (void)warp_wait(bar(C::DRAIN + 1), 0, p.err);
        }
    } else if (warp == PV_WARP) {
        // ------------------------------------------------------------ the peer's T_FULL, seen tile by tile for the leader
        int i = 0;
        for_each_segment(p, start, [&](const Segment& g) -> bool {
            for (int u = 0; u < g.n; ++u, ++i) {
                if (!(ok = warp_wait(bar(C::T_FULL + (i & 1)), (uint32_t)((i >> 1) & 1), p.err))) return false;
                if (lane == 0) arrive_at(lead(C::SEEN + (i & 1)));
                __syncwarp();
            }
            return true;
        });
    }
    __syncwarp();
    tc::fence_before();
    // Every load of both CTAs is behind a wait of the leader's issuers.  If those went well nothing is in flight now; if
    // a wait ran out (one in the peer makes one of the leader's run out, or had nothing left to load), no copy may be left
    // behind: the last ones of each buffer, both CTAs'
    if (__syncthreads_or(!ok) && rank == 0 && warp >= X_WARP) {
        const bool rope = warp == ROPE_WARP;
        for (int k = max(0, loaded - (rope ? 1 : 2)); k < loaded; ++k) {
            if (rope) (void)warp_wait(bar(C::ROPE_FULL), (uint32_t)(k & 1), p.err);
            else (void)warp_wait(bar((warp == X_WARP ? C::X_FULL : C::FULL) + (k & 1)), (uint32_t)((k >> 1) & 1), p.err);
        }
    }
    cluster_sync();  // every MMA and every access to the peer's shared memory is complete
    if (warp == QK_WARP) {
        tc::fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS) : "memory");
    }
}

}  // namespace pa
