// pages.cuh -- what moves, shares, takes and frees the pages of a cache between two forward passes:
// copies of pages, the accepted rows of a verified tree moved to the front of its drafted ones, forks of
// sequences, and sequences brought to new lengths (pages from and back to a free list, a shared last page
// copied before it is written).  The data are moved bit by bit, in all layers of a model by one call: a
// cache is `planes` arrays (layers, K and V) of [num_blocks, block_size, row].
//
// All of it is memory traffic and latency.  The copies keep eight 16-byte loads in flight a thread: 1.6 GB of pages at
// 6.7 TB/s (0.98 of the measured copy rate), the accepted rows of 64 sequences in 28 layers (66 MB) 11 us (0.88), of one
// layer 3.4 us, which are five dependent reads.  The ledger's calls are the same few reads (fork 3 us, a step's growth
// or trim 4 + 5 us) and, for many pages, atomics and the order in which freed pages are put back.
#pragma once

#include "pa_device.cuh"

namespace pa {

// K and V (or the latent rows alone) of all layers: plane l is layer l of k, plane layers + l layer l of v.
struct Planes {
    uint4 *k, *v;            // v: null where the cache is one array a layer
    int layers, planes;
    int row_vecs, block_size;
    int64_t plane_vecs;      // 16-byte chunks of a layer's array
    int num_blocks;
};

__device__ __forceinline__ uint4* plane_of(const Planes& c, int plane) {
    return plane < c.layers ? c.k + plane * c.plane_vecs : c.v + (plane - c.layers) * c.plane_vecs;
}

constexpr int kCopyThreads = 256, kCopyUnroll = 8;

// Pages pairs[i][0] -> pairs[i][1] of every plane.  An item is a segment of one page of one plane, worked by
// `lanes` threads (a power of two) with kCopyUnroll chunks each in flight.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const Planes c, const int32_t* pairs, unsigned items,
                                                                 unsigned segs, int seg_vecs, int page_vecs, int lanes_log2,
                                                                 unsigned* err) {
    constexpr int U = kCopyUnroll;
    const unsigned per_block = kCopyThreads >> lanes_log2;
    const int lanes = 1 << lanes_log2, lane = threadIdx.x & (lanes - 1);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (unsigned it = blockIdx.x * per_block + (threadIdx.x >> lanes_log2); it < items; it += gridDim.x * per_block) {
        const unsigned rest = it / segs, seg = it - rest * segs;
        const unsigned pair = rest / (unsigned)c.planes, plane = rest - pair * (unsigned)c.planes;
        const int src = ld_global(pairs + 2 * (size_t)pair), dst = ld_global(pairs + 2 * (size_t)pair + 1);
        if (src == -1 || dst == -1) continue;
        if (src < 0 || src >= c.num_blocks || dst < 0 || dst >= c.num_blocks) {
            if (lane == 0) flag_error(err, PA_DEVERR_BLOCK);
            continue;
        }
        uint4* const base = plane_of(c, (int)plane);
        const int v0 = (int)seg * seg_vecs, n = min(seg_vecs, page_vecs - v0);
        const uint4* s = base + (size_t)src * page_vecs + v0;
        uint4* d = base + (size_t)dst * page_vecs + v0;
        for (int e = lane; e < n; e += U * lanes) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (e + u * lanes < n) x[u] = ld_stream(s + e + u * lanes);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (e + u * lanes < n) d[e + u * lanes] = x[u];
        }
    }
}

// ---- the accepted path of a verified tree --------------------------------------------------------

struct CommitParams {
    Planes c;
    const int32_t *block_tables, *query_start_loc, *seq_lens, *path, *num_accepted;
    int32_t* new_lens;
    unsigned* err;
    int max_blocks_per_seq, max_path, num_seqs;
};

constexpr int kCommitThreads = 256, kCommitRows = 256;  // threads; rows of a path in shared memory at a time

// Row ctx + path[i] -> ctx + i for i < accepted, path rising: path[i] >= i, so a column of 16 bytes that one
// thread moves in this order (loads of a few rows, then their stores) reads every row before it is overwritten:
// row ctx + j is stored for i = j and read for the i with path[i] = j, which is at most j.
__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const CommitParams p) {
    constexpr int U = 8;
    __shared__ int64_t from[kCommitRows], to[kCommitRows];  // rows of a plane; -1: not moved
    const int s = blockIdx.x, tid = threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int n = ld_global(p.query_start_loc + s + 1) - ld_global(p.query_start_loc + s), kv_len = ld_global(p.seq_lens + s);
    const int acc = ld_global(p.num_accepted + s), ctx = kv_len - n;
    const int cap = p.max_blocks_per_seq * p.c.block_size;
    const bool bad_len = n < 0 || kv_len < n || kv_len > cap;
    const int32_t* path = p.path + (size_t)s * p.max_path;
    bool bad = !bad_len && (acc < 0 || acc > n || acc > p.max_path);
    if (!bad && !bad_len) {
        bool mine = false;
        for (int i = tid; i < acc; i += kCommitThreads) {
            const int t = ld_global(path + i), before = i > 0 ? ld_global(path + i - 1) : -1;
            mine = mine || t <= before || t >= n;
        }
        bad = __syncthreads_or(mine);
    }
    if (bad_len || bad) {
        if (blockIdx.y == 0 && tid == 0) {
            flag_error(p.err, bad_len ? PA_DEVERR_LENGTH : PA_DEVERR_PATH);
            p.new_lens[s] = bad_len ? kv_len : ctx;
        }
        return;
    }
    if (blockIdx.y == 0 && tid == 0) p.new_lens[s] = ctx + acc;
    const int32_t* bt = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    const int bs = p.c.block_size;
    const int64_t columns = (int64_t)p.c.planes * p.c.row_vecs;
    for (int i0 = 0; i0 < acc; i0 += kCommitRows) {
        const int rows = min(kCommitRows, acc - i0);
        __syncthreads();
        if (tid < rows) {
            const int a = ctx + ld_global(path + i0 + tid), b = ctx + i0 + tid;
            int64_t f = -1, t = -1;
            if (a != b) {
                const int pa_ = ld_global(bt + a / bs), pb = ld_global(bt + b / bs);
                if (pa_ < 0 || pa_ >= p.c.num_blocks || pb < 0 || pb >= p.c.num_blocks) {
                    flag_error(p.err, PA_DEVERR_BLOCK);
                } else {
                    f = ((int64_t)pa_ * bs + a % bs) * p.c.row_vecs;
                    t = ((int64_t)pb * bs + b % bs) * p.c.row_vecs;
                }
            }
            from[tid] = f;
            to[tid] = t;
        }
        __syncthreads();
        for (int64_t col = (int64_t)blockIdx.y * kCommitThreads + tid; col < columns; col += (int64_t)gridDim.y * kCommitThreads) {
            const int plane = (int)(col / p.c.row_vecs);
            uint4* const base = plane_of(p.c, plane) + (col - (int64_t)plane * p.c.row_vecs);
            for (int i = 0; i < rows; i += U) {
                uint4 x[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i + u < rows && from[i + u] >= 0) x[u] = ld_stream(base + from[i + u]);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i + u < rows && from[i + u] >= 0) base[to[i + u]] = x[u];
            }
        }
    }
}

// ---- forks ---------------------------------------------------------------------------------------

// Sequence s, which is empty, becomes a fork of parents[s]: the same pages, one reference more each.  A block for
// kForkSeqs sequences: those with the same parent are served by one pass over its row, with one addition to a page's
// count (496 forks of 16 sequences of 8K..32K tokens: 9.5 us with a block and an addition for each).  No block reads
// what another writes: a parent is nobody's child in the call.
constexpr int kForkThreads = 512, kForkSeqs = 8;

__global__ void __launch_bounds__(kForkThreads) fork_pages_kernel(int32_t* block_tables, int mb, int32_t* seq_lens,
                                                                 const int32_t* parents, int num_seqs,
                                                                 int32_t* ref_counts, int block_size, int num_blocks, unsigned* err) {
    constexpr int U = 4;
    __shared__ int parent_s[kForkSeqs], len_s[kForkSeqs];
    const int tid = threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid < kForkSeqs) {
        const int s = blockIdx.x * kForkSeqs + tid;
        int par = s < num_seqs ? ld_global(parents + s) : -1, len = 0;
        if (par != -1) {
            const bool known = par >= 0 && par < num_seqs;
            if (!known || ld_global(parents + par) != -1 || seq_lens[s] != 0) {
                flag_error(err, PA_DEVERR_FORK);
                par = -1;
            } else {
                len = seq_lens[par];
                if (len < 0 || len > mb * block_size) {
                    flag_error(err, PA_DEVERR_LENGTH);
                    par = -1;
                } else {
                    seq_lens[s] = len;  // (nobody else reads it: s is no parent)
                }
            }
        }
        parent_s[tid] = par;
        len_s[tid] = len;
    }
    __syncthreads();
    unsigned left = 0;
    for (int i = 0; i < kForkSeqs; ++i) left |= (parent_s[i] >= 0 ? 1u : 0u) << i;
    while (left) {
        const int first = __ffs(left) - 1, par = parent_s[first];
        unsigned mine = 0;
        for (int i = first; i < kForkSeqs; ++i) mine |= (parent_s[i] == par ? 1u : 0u) << i;
        left &= ~mine;
        const int pages = (len_s[first] + block_size - 1) / block_size, count = __popc(mine);
        const int32_t* from = block_tables + (size_t)par * mb;
        int32_t* to = block_tables + (size_t)blockIdx.x * kForkSeqs * mb;
        for (int c = tid; c < pages; c += U * kForkThreads) {
            int id[U];
#pragma unroll
            for (int u = 0; u < U; ++u) id[u] = c + u * kForkThreads < pages ? from[c + u * kForkThreads] : 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c + u * kForkThreads >= pages) break;
                for (unsigned m = mine; m; m &= m - 1) to[(size_t)(__ffs(m) - 1) * mb + c + u * kForkThreads] = id[u];
                if (id[u] >= 0 && id[u] < num_blocks) atomicAdd(ref_counts + id[u], count);
                else flag_error(err, PA_DEVERR_BLOCK);
            }
        }
    }
}

// ---- new lengths -----------------------------------------------------------------------------------

// What the plan leaves for a sequence: first of its pages among those taken from the free list (-1: nothing to
// do), the shared last page that it copies (-1: none), its pages before and after.
struct ResizePlan {
    int start, cow, have, want;
};
struct ResizeHead {
    int top, taken;          // entries of the free list before the call, those taken
    unsigned ticket, freed;  // blocks done, pages whose last reference went
};

struct ResizeParams {
    Planes c;
    int32_t *block_tables, *seq_lens, *ref_counts, *free_list, *free_count;
    const int32_t* new_lens;
    ResizeHead* head;
    ResizePlan* plan;        // [num_seqs]
    unsigned* bits;          // [ceil(num_blocks / 32)]: pages that got free
    unsigned* err;
    int max_blocks_per_seq, num_seqs;
    int push_blocks;         // blocks of resize_push_kernel, 0: none
};

constexpr int kPlanThreads = 1024, kApplyThreads = 512, kScanWords = 512;

// One block: which sequences get their pages (in their order, as long as the free list lasts), where these
// stand in the list, and which shared pages are copied -- all from the state before the call.
__global__ void __launch_bounds__(kPlanThreads) resize_plan_kernel(const ResizeParams p) {
    __shared__ long long warp_sum[32];
    __shared__ int popped;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int words = (p.c.num_blocks + 31) / 32;
    for (int w = tid; w < words; w += kPlanThreads) p.bits[w] = 0u;
    int top = *p.free_count;
    if (top < 0 || top > p.c.num_blocks) {
        if (tid == 0) flag_error(p.err, PA_DEVERR_COUNT);
        top = -1;  // the list cannot be used: nothing is taken from it or put back
    }
    if (tid == 0) popped = 0;
    const int bs = p.c.block_size, cap = p.max_blocks_per_seq * bs;
    long long base = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += kPlanThreads) {
        const int s = s0 + tid;
        ResizePlan r{-1, -1, 0, 0};
        int demand = 0;
        if (s < p.num_seqs && top >= 0) {
            const int want = ld_global(p.new_lens + s), have = p.seq_lens[s];
            if (want < -1 || want > cap || have < 0 || have > cap) {
                flag_error(p.err, PA_DEVERR_LENGTH);
            } else if (want != -1 && want != have) {
                r.start = 0;
                r.have = (have + bs - 1) / bs;
                r.want = (want + bs - 1) / bs;
                if (want > have) {
                    demand = r.want - r.have;
                    if (have % bs) {
                        const int last = p.block_tables[(size_t)s * p.max_blocks_per_seq + r.have - 1];
                        if (last < 0 || last >= p.c.num_blocks) {
                            flag_error(p.err, PA_DEVERR_BLOCK);
                        } else if (p.ref_counts[last] > 1) {
                            r.cow = last;
                            ++demand;
                        }
                    }
                }
            }
        }
        long long end = demand;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += y;
        }
        __syncthreads();
        if (lane == 31) warp_sum[warp] = end;
        __syncthreads();
        long long all = 0;
        end += base;
#pragma unroll 8
        for (int w = 0; w < 32; ++w) {
            const long long x = warp_sum[w];
            if (w < warp) end += x;
            all += x;
        }
        base += all;
        if (demand > 0) {
            if (end <= top) {
                r.start = (int)(end - demand);
                atomicMax(&popped, (int)end);
            } else {
                flag_error(p.err, PA_DEVERR_PAGES);
                r.start = -1;
            }
        }
        if (s < p.num_seqs) p.plan[s] = r;
    }
    __syncthreads();
    if (tid == 0) *p.head = ResizeHead{top, popped, 0u, 0u};
}

// A reference less; the page is marked, and 1 returned, when that was the last one.
__device__ __forceinline__ int release_page(const ResizeParams& p, int id) {
    if (id < 0 || id >= p.c.num_blocks) {
        flag_error(p.err, PA_DEVERR_BLOCK);
        return 0;
    }
    const int before = atomicSub(p.ref_counts + id, 1);
    if (before == 1) {
        atomicOr(p.bits + (id >> 5), 1u << (id & 31));
        return 1;
    }
    if (before <= 0) {  // nobody's page: its count stays
        atomicAdd(p.ref_counts + id, 1);
        flag_error(p.err, PA_DEVERR_COUNT);
    }
    return 0;
}

// Sequences to their lengths, by the threads of `blocks` blocks.
__device__ __forceinline__ void write_lengths(const ResizeParams& p, int block, int blocks) {
    for (int i = block * kApplyThreads + (int)threadIdx.x; i < p.num_seqs; i += blocks * kApplyThreads)
        if (p.plan[i].start >= 0) p.seq_lens[i] = ld_global(p.new_lens + i);
}

__device__ __forceinline__ void write_count(const ResizeParams& p, int count) {
    if (count > p.c.num_blocks) flag_error(p.err, PA_DEVERR_COUNT);  // (a page was on the list and in a table)
    *p.free_count = min(count, p.c.num_blocks);
}

// The marked pages of words [w0, w0 + kScanWords) into the list from entry `at` on, in the order of their numbers; a block.
// Loaded together; a warp's run of them is counted, then its pages put behind those of the warps before, a word by 32
// lanes.
__device__ __forceinline__ void push_pages(const ResizeParams& p, int w0, int at) {
    constexpr int NW = kApplyThreads / 32, RUN = kScanWords / NW;
    __shared__ unsigned words_s[kScanWords];
    __shared__ int warp_sum[NW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, words = (p.c.num_blocks + 31) / 32;
#pragma unroll
    for (int k = tid; k < kScanWords; k += kApplyThreads) words_s[k] = w0 + k < words ? ld_l2(p.bits + w0 + k) : 0u;
    __syncthreads();
    const unsigned* run = words_s + warp * RUN;
    int mine = 0;
#pragma unroll
    for (int k = 0; k < RUN / 32; ++k) mine += __popc(run[32 * k + lane]);
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) warp_sum[warp] = mine;
    __syncthreads();
    if (mine == 0) return;
    for (int w = 0; w < warp; ++w) at += warp_sum[w];
#pragma unroll 1
    for (int k = 0; k < RUN; k += 32) {
        const unsigned my = run[k + lane];
        int end = __popc(my);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += y;
        }
        const int before = at + end - __popc(my);
        at += __shfl_sync(0xffffffffu, end, 31);
#pragma unroll 4
        for (unsigned any = __ballot_sync(0xffffffffu, my != 0u); any; any &= any - 1) {
            const int j = __ffs(any) - 1;
            const unsigned b = run[k + j];
            const int to = __shfl_sync(0xffffffffu, before, j) + __popc(b & ((1u << lane) - 1u));
            if ((b >> lane & 1u) && to < p.c.num_blocks) p.free_list[to] = 32 * (w0 + warp * RUN + k + j) + lane;
        }
    }
}

// A sequence a block column; its first block changes the table and the counts, all of them copy a shared last
// page's rows.  The pages that got free go on the list in the order of their numbers, so that the same call leaves the
// same list whatever the order of the blocks: in pools of up to 32 kScanWords pages by the block that is done last, in
// larger ones by a kernel behind this one (one block takes 10 us for 262144 pages of which 500 got free and 60 for
// 131000; the launch 2).
__global__ void __launch_bounds__(kApplyThreads) resize_apply_kernel(const ResizeParams p) {
    constexpr int U = kCopyUnroll;
    __shared__ bool last_block;
    const int s = blockIdx.x, tid = threadIdx.x, bs = p.c.block_size;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const ResizePlan r = p.plan[s];
    const int top = p.head->top;
    if (r.start >= 0) {
        int32_t* bt = p.block_tables + (size_t)s * p.max_blocks_per_seq;
        const int first = r.have - (r.cow >= 0 ? 1 : 0);
        auto taken = [&](int i) {  // i-th page that the sequence gets, -1 where the list holds no page of the pool
            const int id = p.free_list[top - 1 - (r.start + i)];
            return id >= 0 && id < p.c.num_blocks ? id : -1;
        };
        if (r.cow >= 0) {
            // (the lengths are written last of all, below)
            const int dst = taken(0), n = p.seq_lens[s] % bs * p.c.row_vecs;
            if (dst >= 0) {
                const int64_t page = (int64_t)bs * p.c.row_vecs;
                for (int plane = blockIdx.y; plane < p.c.planes; plane += gridDim.y) {
                    uint4* const base = plane_of(p.c, plane);
                    const uint4* from = base + r.cow * page;
                    uint4* to = base + dst * page;
                    for (int e = tid; e < n; e += U * kApplyThreads) {
                        uint4 x[U];
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            if (e + u * kApplyThreads < n) x[u] = ld_stream(from + e + u * kApplyThreads);
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            if (e + u * kApplyThreads < n) to[e + u * kApplyThreads] = x[u];
                    }
                }
            }
        }
        if (blockIdx.y == 0) {
            for (int c = first + tid; c < r.want; c += kApplyThreads) {
                const int id = taken(c - first);
                bt[c] = id;
                if (id < 0 || atomicExch(p.ref_counts + id, 1) != 0) flag_error(p.err, PA_DEVERR_COUNT);
            }
            int freed = 0;  // (one addition a warp: 134000 on one address took 60 us)
            for (int c = r.want + tid; c < r.have; c += kApplyThreads) {
                freed += release_page(p, bt[c]);
                bt[c] = -1;
            }
            if (r.cow >= 0 && tid == 0) freed += release_page(p, r.cow);
            freed = __reduce_add_sync(0xffffffffu, freed);
            if (freed > 0 && (tid & 31) == 0) atomicAdd(&p.head->freed, (unsigned)freed);
        }
    }
    if (p.push_blocks > 0) return;
    __threadfence();
    __syncthreads();
    if (tid == 0) last_block = atomicAdd(&p.head->ticket, 1u) == gridDim.x * gridDim.y - 1;
    __syncthreads();
    if (!last_block) return;
    __threadfence();
    write_lengths(p, 0, 1);
    if (top < 0) return;
    const int left = top - p.head->taken, freed = (int)ld_l2(&p.head->freed);
    if (tid == 0) write_count(p, left + freed);
    if (freed > 0) push_pages(p, 0, left);
}

__global__ void __launch_bounds__(kApplyThreads) resize_push_kernel(const ResizeParams p) {
    __shared__ int sum;
    const int tid = threadIdx.x, b = (int)blockIdx.x;
    if (tid == 0) sum = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    write_lengths(p, b, (int)gridDim.x);
    const int top = p.head->top;
    if (top < 0) return;
    const int left = top - p.head->taken, freed = (int)p.head->freed;
    if (b == 0 && tid == 0) write_count(p, left + freed);
    if (freed == 0) return;
    // pages of the words before this block's
    int before = 0;
    const uint4* bits = reinterpret_cast<const uint4*>(p.bits);
#pragma unroll 4
    for (int w = tid; w < b * (kScanWords / 4); w += kApplyThreads) {
        const uint4 v = ld_l2(bits + w);
        before += __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w);
    }
    __syncthreads();
    before = __reduce_add_sync(0xffffffffu, before);
    if ((tid & 31) == 0 && before > 0) atomicAdd(&sum, before);
    __syncthreads();
    push_pages(p, b * kScanWords, left + sum);
}

}  // namespace pa
