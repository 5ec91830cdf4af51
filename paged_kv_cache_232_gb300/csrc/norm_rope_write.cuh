// norm_rope_write.cuh -- the KV-cache write with the per-head RMS norm of queries and keys and the
// rotary embedding applied on the way, and the latent-cache write.
//
// A head row x of D columns becomes y = x rsqrt(mean(x^2) + eps) w, then turns by its position as
// in rope_write.cuh; a cached latent row is its norm over the latent columns beside the rotated key
// part.  All in fp32 with one rounding to the 16-bit format at the end.
//
// Both are one pass over the rows, bound by memory traffic: what matters is bytes in flight, so a
// thread keeps one role (its head row and its weights, no divisions in the loop) and walks tokens with
// the next one's loads issued ahead.  GB300, 64K rows of 16 q / 8 KV heads x 128: a warp an item with a
// division each 246 us, four tokens unrolled 320 (registers cost occupancy), one 199, one ahead 180 (1.09 GB:
// 0.89 of the measured copy bandwidth); 42 or fewer registers spill (330 and more).  32K latent rows with 16
// heads: 59 -> 47.5 us (0.68; two tokens ahead, other grids and register limits no better).  Part of what is left
// there: the key part is the first of a token's rotary rows, so at a multiple of 8 heads the token's last warp
// holds one row in 4 of its 32 lanes (one warp in four at 16 heads) and keeps few bytes in flight.
#pragma once

#include "rope_write.cuh"

namespace pa {

template <bool BF16>
__device__ __forceinline__ float sum_sq(const uint4& v, float scale) {
    float f[8], s = 0.f;
    unpack8<BF16>(v, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(f[e] * scale, f[e] * scale, s);
    return s;
}

// The rare case of inv_rms, out of line: the row scaled by k, a power of two near 1 / its largest value m.  Returns
// r and the factor that the row's values take before they are multiplied by r:
//   1 / sqrt(mean(x^2) + eps) = k / sqrt(mean((k x)^2) + eps k^2).
// Large rows (k < 1): r = k / sqrt(..), at least 2^-128.  Tiny ones: k stays with the values, for k / sqrt(..) may be past
// fp32 (one value of 2^-126 in 256 columns: 2^130).  Where eps k^2 is past 1e30 the row is nothing beside eps (mean((k x)^2)
// is at most 4), so the unscaled r was right; m is then so small that eps k^2 itself may be past fp32.
template <bool BF16, int GL, int D, int N>
__device__ __noinline__ float2 inv_rms_scaled(uint4 v0, uint4 v1, float eps, float ss, float r, bool lost) {
    const uint4 v[2] = {v0, v1};
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float f[8];
        unpack8<BF16>(v[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
    }
#pragma unroll
    for (int o = GL / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float k = __int_as_float((127 - min(max(ilogbf(m), -126), 126)) << 23);
    float st = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) st += sum_sq<BF16>(v[i], k);
#pragma unroll
    for (int o = GL / 2; o > 0; o >>= 1) st += __shfl_xor_sync(0xffffffffu, st, o);
    if (ss != ss) return make_float2(ss, 1.f);
    // an infinite value leaves the finite ones 0 and itself NaN (0 * inf), as the formula does
    if (lost && m == INFINITY) return make_float2(0.f, 1.f);
    const float ek = eps * k * k;
    if (!lost || m == 0.f || !(ek <= 1e30f)) return make_float2(r, 1.f);
    const float t = rsqrtf(st * (1.f / D) + ek);
    return k < 1.f ? make_float2(k * t, 1.f) : make_float2(t, k);
}

// 1 / sqrt(mean(x^2) + eps) of a row of D values that GL neighbouring lanes hold (N 16-byte chunks
// each, zeros where a lane holds none).  The whole warp calls it.  bf16 reaches 2^128 and down to 2^-133: where a
// sum of squares overflows fp32 (or, next to a tiny eps, vanishes), the row is scaled by its largest value first.  In
// two factors (usually 1 / sqrt and 1), the second, a power of two, for the values before the first.
template <bool BF16, int GL, int D, int N>
__device__ __forceinline__ float2 inv_rms(const uint4 (&v)[N], float eps) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) ss += sum_sq<BF16>(v[i], 1.f);
#pragma unroll
    for (int o = GL / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    float2 r = make_float2(rsqrtf(ss * (1.f / D) + eps), 1.f);
    const bool lost = !(ss <= 1e37f) || (eps < 1e-30f && ss < 1e-25f);
    if (__any_sync(0xffffffffu, lost)) r = inv_rms_scaled<BF16, GL, D, N>(v[0], v[N - 1], eps, ss, r.x, lost);
    return r;
}

// eight values x * r * w (r of inv_rms), rounded by the caller's next step only: kept as floats
template <bool BF16>
__device__ __forceinline__ void norm8(const uint4& x, const uint4& w, float2 r, float* y) {
    float a[8], b[8];
    unpack8<BF16>(x, a);
    unpack8<BF16>(w, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = a[e] * r.y * r.x * b[e];
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float* f) {
    using F = F16x2<BF16>;
    return make_uint4(F::pack_rn(f[0], f[1]), F::pack_rn(f[2], f[3]), F::pack_rn(f[4], f[5]), F::pack_rn(f[6], f[7]));
}

// the pairs (a[e], b[e]) turned by cos c8 .. c8 + 7 and the sin beside them, in place
__device__ __forceinline__ void turn8(float* a, float* b, const float* cs_row, int c8, int half) {
    const float4 ca = ldg_f4(cs_row + c8), cb = ldg_f4(cs_row + c8 + 4);
    const float4 sa = ldg_f4(cs_row + half + c8), sb = ldg_f4(cs_row + half + c8 + 4);
    const float c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
    const float s[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = a[e], y = b[e];
        a[e] = fmaf(x, c[e], -(y * s[e]));
        b[e] = fmaf(y, c[e], x * s[e]);
    }
}

struct NormRopeParams {
    const uint16_t *q, *key, *value;  // rows of n_q_heads / n_kv_heads heads, strides in elements
    uint16_t* q_out;
    int64_t q_stride, key_stride, value_stride, q_out_stride;
    const uint16_t *q_weight, *k_weight;  // [D]
    uint16_t *k_cache, *v_cache;          // [slots, n_kv_heads, D]
    const int64_t *slot_mapping, *positions;
    const float* cos_sin;                 // [max_position, D]
    int64_t num_tokens, num_slots, max_position;
    int n_q_heads, n_kv_heads;
    float eps;
    unsigned* err;
};

// A head row takes GL lanes, each the 16-byte chunks c and c + D / 16 of it (both halves of eight
// rotations), so the sum of squares is a shuffle over GL lanes.  A thread keeps its head row and its
// weights and walks tokens, the next token's loads in flight while it works on one.
template <bool BF16, int D>
__global__ void __launch_bounds__(512, 2) norm_rope_write_kernel(const NormRopeParams p) {
    constexpr int PAIRS = D / 16;
    constexpr int GL = D == 64 ? 4 : D == 256 ? 16 : 8;  // 96 columns: 6 of 8 lanes
    // the next kernel of the step may start its launch; it waits for this grid before reading anything
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int c = threadIdx.x % GL;
    const int heads = p.n_q_heads + 2 * p.n_kv_heads;
    // (whole warps take part in the shuffles: the head loop runs to a multiple of the block's head rows)
    for (int h0 = 0; h0 < heads; h0 += (int)blockDim.x / GL) {
        const int h = h0 + (int)threadIdx.x / GL;
        const int kind = h < p.n_q_heads ? 0 : h < p.n_q_heads + p.n_kv_heads ? 1 : 2;
        const int hh = kind == 0 ? h : kind == 1 ? h - p.n_q_heads : h - p.n_q_heads - p.n_kv_heads;
        const bool mine = h < heads && c < PAIRS;
        const uint16_t* src = (kind == 0 ? p.q : kind == 1 ? p.key : p.value) + (int64_t)hh * D + 8 * c;
        uint16_t* dst = (kind == 0 ? p.q_out : kind == 1 ? p.k_cache : p.v_cache) + (int64_t)hh * D + 8 * c;
        const int64_t in_stride = kind == 0 ? p.q_stride : kind == 1 ? p.key_stride : p.value_stride;
        const int64_t out_stride = kind == 0 ? p.q_out_stride : (int64_t)p.n_kv_heads * D;
        const uint4* weight = reinterpret_cast<const uint4*>(kind == 0 ? p.q_weight : p.k_weight) + c;
        uint4 nxt[2];
        int64_t npos = 0, nslot = -1;
        auto fetch = [&](int64_t t) {
            nxt[0] = nxt[1] = make_uint4(0u, 0u, 0u, 0u);
            if (t >= p.num_tokens) return;
            npos = __ldg(p.positions + t);
            nslot = __ldg(p.slot_mapping + t);
            if (mine) {
                const uint4* row = reinterpret_cast<const uint4*>(src + t * in_stride);
                nxt[0] = row[0];
                nxt[1] = row[PAIRS];
            }
        };
        fetch(blockIdx.x);
        for (int64_t t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
            uint4 x[2] = {nxt[0], nxt[1]};
            const int64_t pos = npos;
            int64_t slot = nslot;
            // (the row in flight is another token's: also where q is rewritten in place)
            fetch(t + gridDim.x);
            const float2 r = inv_rms<BF16, GL, D>(x, p.eps);
            if (pos < 0 || pos >= p.max_position) {  // the row is left untouched
                if (threadIdx.x == 0 && h0 == 0) flag_error(p.err, PA_DEVERR_POSITION);
                continue;
            }
            if (slot < -1 || slot >= p.num_slots) {
                if (threadIdx.x == 0 && h0 == 0) flag_error(p.err, PA_DEVERR_SLOT);
                slot = -1;
            }
            if (!mine || (kind != 0 && slot < 0)) continue;
            uint4* out = reinterpret_cast<uint4*>(dst + (kind == 0 ? t : slot) * out_stride);
            if (kind < 2) {
                float a[8], b[8];
                norm8<BF16>(x[0], __ldg(weight), r, a);
                norm8<BF16>(x[1], __ldg(weight + PAIRS), r, b);
                turn8(a, b, p.cos_sin + pos * D, 8 * c, D / 2);
                x[0] = pack8<BF16>(a);
                x[1] = pack8<BF16>(b);
            }
            out[0] = x[0];
            out[PAIRS] = x[1];
        }
    }
}

struct LatentWriteParams {
    const uint16_t* kv;      // [num_tokens] rows of DL + 64 columns, kv_stride elements apart
    const uint16_t* weight;  // [DL] or null: no norm
    const uint16_t* q_pe;    // [num_tokens, n_heads, 64], strides in elements; null: none
    uint16_t* q;             // [num_tokens, n_heads, DL + 64]: the rotated q_pe goes to its last 64 columns
    uint16_t* cache;         // [slots, DL + 64]
    int64_t kv_stride, pe_token_stride, pe_head_stride;
    const int64_t *slot_mapping, *positions;
    const float* cos_sin;    // [max_position, 64]
    int64_t num_tokens, num_slots, max_position;
    int n_heads, interleaved;
    float eps;
    unsigned* err;
};

// A warp keeps one task of a token and walks tokens, the next token's loads in flight: task 0 its latent
// columns (DL / 32 a lane, the sum of squares over the warp), task 1 .. eight of its 64-column rotary rows
// (four lanes each: the shared key part, then the query heads').  A lane holds the 16-byte chunks c and
// c + 4 of its rotary row: the rotate-half pairs of eight angles, or (interleaved) the neighbours of four
// angles in each chunk.  A block's eight warps hold the tasks of `per_block` tokens (up to eight tasks a
// token), or eight of one token's tasks (blockIdx.y: which eight).
template <bool BF16, int DL>
__global__ void __launch_bounds__(256, 4) latent_write_kernel(const LatentWriteParams p, int tasks, int per_block) {
    constexpr int ROW = DL + 64, CH = DL / 256;  // 16-byte chunks of the latent columns per lane
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 3;
    const int task = tasks <= 8 ? warp % tasks : (int)blockIdx.y * 8 + warp;
    if (task >= tasks || warp >= tasks * per_block) return;
    const int rows = 1 + (p.q_pe ? p.n_heads : 0);
    const int rr = (task - 1) * 8 + (lane >> 2);  // rotary row: 0 the key part, 1 .. query head rr - 1
    const bool mine = task == 0 || rr < rows;
    const int hop = task == 0 ? (CH - 1) * 32 : 4;  // chunks between this lane's two (none: one chunk, read twice)
    const uint16_t* src = task == 0 ? p.kv + 8 * lane
                          : rr == 0 ? p.kv + DL + 8 * c
                                    : p.q_pe + (int64_t)(rr - 1) * p.pe_head_stride + 8 * c;
    const int64_t in_stride = rr <= 0 ? p.kv_stride : p.pe_token_stride;
    const int64_t step = (int64_t)gridDim.x * per_block;
    uint4 nxt[2];
    int64_t npos = 0, nslot = -1;
    auto fetch = [&](int64_t t) {
        nxt[0] = nxt[1] = make_uint4(0u, 0u, 0u, 0u);
        if (t >= p.num_tokens) return;
        npos = __ldg(p.positions + t);
        nslot = __ldg(p.slot_mapping + t);
        if (mine) {
            const uint4* row = reinterpret_cast<const uint4*>(src + t * in_stride);
            nxt[0] = row[0];
            nxt[1] = row[hop];
        }
    };
    int64_t t = (int64_t)blockIdx.x * per_block + (tasks <= 8 ? warp / tasks : 0);
    fetch(t);
    for (; t < p.num_tokens; t += step) {
        uint4 x[2] = {nxt[0], nxt[1]};
        const int64_t pos = npos;
        int64_t slot = nslot;
        fetch(t + step);
        if (pos < 0 || pos >= p.max_position) {  // the row is left untouched
            if (task == 0 && lane == 0) flag_error(p.err, PA_DEVERR_POSITION);
            continue;
        }
        if (slot < -1 || slot >= p.num_slots) {
            if (task == 0 && lane == 0) flag_error(p.err, PA_DEVERR_SLOT);
            slot = -1;
        }
        if (task == 0) {
            if (slot < 0) continue;  // (the same in the whole warp)
            if (p.weight) {
                const uint4* w = reinterpret_cast<const uint4*>(p.weight) + lane;
                uint4 v[CH];
#pragma unroll
                for (int e = 0; e < CH; ++e) v[e] = x[e];
                const float2 r = inv_rms<BF16, 32, DL>(v, p.eps);
#pragma unroll
                for (int e = 0; e < CH; ++e) {
                    float f[8];
                    norm8<BF16>(x[e], __ldg(w + 32 * e), r, f);
                    x[e] = pack8<BF16>(f);
                }
            }
            uint4* dst = reinterpret_cast<uint4*>(p.cache + slot * ROW) + lane;
#pragma unroll
            for (int e = 0; e < CH; ++e) dst[32 * e] = x[e];
            continue;
        }
        if (!mine || (rr == 0 && slot < 0)) continue;
        uint16_t* dst = rr == 0 ? p.cache + slot * ROW + DL : p.q + (t * p.n_heads + rr - 1) * ROW + DL;
        const float* cs = p.cos_sin + pos * 64;
        float a[8], b[8];
        unpack8<BF16>(x[0], a);
        unpack8<BF16>(x[1], b);
        if (!p.interleaved) {
            turn8(a, b, cs, 8 * c, 32);
        } else {
            const float4 c0 = ldg_f4(cs + 4 * c), s0 = ldg_f4(cs + 32 + 4 * c);
            const float4 c1 = ldg_f4(cs + 16 + 4 * c), s1 = ldg_f4(cs + 48 + 4 * c);
            const float ca[4] = {c0.x, c0.y, c0.z, c0.w}, sa[4] = {s0.x, s0.y, s0.z, s0.w};
            const float cb[4] = {c1.x, c1.y, c1.z, c1.w}, sb[4] = {s1.x, s1.y, s1.z, s1.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x0 = a[2 * e], y0 = a[2 * e + 1], x1 = b[2 * e], y1 = b[2 * e + 1];
                a[2 * e] = fmaf(x0, ca[e], -(y0 * sa[e]));
                a[2 * e + 1] = fmaf(y0, ca[e], x0 * sa[e]);
                b[2 * e] = fmaf(x1, cb[e], -(y1 * sb[e]));
                b[2 * e + 1] = fmaf(y1, cb[e], x1 * sb[e]);
            }
        }
        reinterpret_cast<uint4*>(dst)[c] = pack8<BF16>(a);
        reinterpret_cast<uint4*>(dst)[c + 4] = pack8<BF16>(b);
    }
}

}  // namespace pa
