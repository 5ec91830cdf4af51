// norm_rope_write.cuh -- the KV-cache write with the per-head RMS norm of queries and keys and the
// rotary embedding applied on the way, and the latent-cache write.
//
// A head row x of D columns becomes y = x rsqrt(mean(x^2) + eps) w, then turns by its position as
// in rope_write.cuh; a cached latent row is its norm over the latent columns beside the rotated key
// part.  All in fp32 with one rounding to the 16-bit format at the end.  Both are one pass over the
// rows, bound by memory traffic.
#pragma once

#include "rope_write.cuh"

namespace pa {

template <bool BF16, int N>
__device__ __forceinline__ float sum_sq(const uint4 (&v)[N], float scale) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float f[8];
        unpack8<BF16>(v[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(f[e] * scale, f[e] * scale, s);
    }
    return s;
}

// 1 / sqrt(mean(x^2) + eps) of a row of D values that GL neighbouring lanes hold (N 16-byte chunks
// each, zeros where a lane holds none).  The whole warp calls it.  bf16 reaches 2^128: where a sum of
// squares overflows fp32 (or, next to a tiny eps, vanishes), the row is scaled by its largest value first.
template <bool BF16, int GL, int D, int N>
__device__ __forceinline__ float inv_rms(const uint4 (&v)[N], float eps) {
    float ss = sum_sq<BF16>(v, 1.f);
#pragma unroll
    for (int o = GL / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    float r = rsqrtf(ss * (1.f / D) + eps);
    const bool lost = !(ss <= 1e37f) || (eps < 1e-30f && ss < 1e-25f);
    if (__any_sync(0xffffffffu, lost)) {
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
        // a power of two near 1 / m, so that scaling is exact
        const float k = exp2f(-(float)min(max(ilogbf(m), -126), 126));
        float st = sum_sq<BF16>(v, k);
#pragma unroll
        for (int o = GL / 2; o > 0; o >>= 1) st += __shfl_xor_sync(0xffffffffu, st, o);
        // an infinite value leaves the finite ones 0 and itself NaN (0 * inf), as the formula does
        if (lost && m > 0.f) r = m == INFINITY ? 0.f : k * rsqrtf(st * (1.f / D) + fminf(eps * k * k, 1e37f));
        if (ss != ss) r = ss;
    }
    return r;
}

// eight values x * r * w, rounded by the caller's next step only: kept as floats
template <bool BF16>
__device__ __forceinline__ void norm8(const uint4& x, const uint4& w, float r, float* y) {
    float a[8], b[8];
    unpack8<BF16>(x, a);
    unpack8<BF16>(w, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = a[e] * r * b[e];
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
// rotations), so the sum of squares is a shuffle over GL lanes.  A warp takes 32 / GL head rows of
// one token; the warps of the grid walk (token, group of head rows) items.
template <bool BF16, int D>
__global__ void __launch_bounds__(256) norm_rope_write_kernel(const NormRopeParams p) {
    constexpr int PAIRS = D / 16;
    constexpr int GL = D == 64 ? 4 : D == 256 ? 16 : 8;  // 96 columns: 6 of 8 lanes
    constexpr int RPW = 32 / GL;
    // the next kernel of the step may start its launch; it waits for this grid before reading anything
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, c = lane % GL;
    const int heads = p.n_q_heads + 2 * p.n_kv_heads;
    const int groups = (heads + RPW - 1) / RPW;
    const int64_t items = p.num_tokens * groups;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t it = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items; it += step) {
        const int64_t t = it / groups;
        const int gr = (int)(it - t * groups);
        const int h = gr * RPW + lane / GL;
        const int64_t pos = __ldg(p.positions + t);
        int64_t slot = __ldg(p.slot_mapping + t);
        if (pos < 0 || pos >= p.max_position) {  // the row is left untouched
            if (gr == 0 && lane == 0) flag_error(p.err, PA_DEVERR_POSITION);
            continue;
        }
        if (slot < -1 || slot >= p.num_slots) {
            if (gr == 0 && lane == 0) flag_error(p.err, PA_DEVERR_SLOT);
            slot = -1;
        }
        const int kind = h < p.n_q_heads ? 0 : h < p.n_q_heads + p.n_kv_heads ? 1 : 2;
        const int hh = kind == 0 ? h : kind == 1 ? h - p.n_q_heads : h - p.n_q_heads - p.n_kv_heads;
        const bool act = h < heads && c < PAIRS && (kind == 0 || slot >= 0);
        uint4 x[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        uint4 &lo = x[0], &hi = x[1];
        if (act) {
            const uint16_t* src = kind == 0 ? p.q + t * p.q_stride : kind == 1 ? p.key + t * p.key_stride
                                                                              : p.value + t * p.value_stride;
            const uint4* row = reinterpret_cast<const uint4*>(src + (int64_t)hh * D);
            lo = row[c];
            hi = row[c + PAIRS];
        }
        const float r = inv_rms<BF16, GL, D>(x, p.eps);
        if (!act) continue;
        uint4* dst;
        if (kind == 0) dst = reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride + (int64_t)hh * D);
        else dst = reinterpret_cast<uint4*>((kind == 1 ? p.k_cache : p.v_cache) + (slot * p.n_kv_heads + hh) * D);
        if (kind < 2) {
            const uint4* w = reinterpret_cast<const uint4*>(kind == 0 ? p.q_weight : p.k_weight);
            float a[8], b[8];
            norm8<BF16>(lo, __ldg(w + c), r, a);
            norm8<BF16>(hi, __ldg(w + c + PAIRS), r, b);
            turn8(a, b, p.cos_sin + pos * D, 8 * c, D / 2);
            lo = pack8<BF16>(a);
            hi = pack8<BF16>(b);
        }
        dst[c] = lo;
        dst[c + PAIRS] = hi;
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

// A warp takes one token's latent columns (item 0: DL / 32 columns a lane, the sum of squares over
// the warp) or eight of its 64-column rotary rows (four lanes each: the shared key part, then the
// query heads').  A lane holds the 16-byte chunks c and c + 4 of its rotary row: the rotate-half
// pairs of eight angles, or (interleaved) the neighbours of four angles in each chunk.
template <bool BF16, int DL>
__global__ void __launch_bounds__(256) latent_write_kernel(const LatentWriteParams p) {
    constexpr int ROW = DL + 64, CH = DL / 256;  // 16-byte chunks of the latent columns per lane
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, c = lane & 3;
    const int rows = 1 + (p.q_pe ? p.n_heads : 0);
    const int groups = 1 + (rows + 7) / 8;
    const int64_t items = p.num_tokens * groups;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t it = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items; it += step) {
        const int64_t t = it / groups;
        const int gr = (int)(it - t * groups);
        const int64_t pos = __ldg(p.positions + t);
        int64_t slot = __ldg(p.slot_mapping + t);
        if (pos < 0 || pos >= p.max_position) {  // the row is left untouched
            if (gr == 0 && lane == 0) flag_error(p.err, PA_DEVERR_POSITION);
            continue;
        }
        if (slot < -1 || slot >= p.num_slots) {
            if (gr == 0 && lane == 0) flag_error(p.err, PA_DEVERR_SLOT);
            slot = -1;
        }
        if (gr == 0) {
            if (slot < 0) continue;
            const uint4* src = reinterpret_cast<const uint4*>(p.kv + t * p.kv_stride);
            uint4* dst = reinterpret_cast<uint4*>(p.cache + slot * ROW);
            uint4 v[CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) v[i] = src[lane + 32 * i];
            if (p.weight) {
                const float r = inv_rms<BF16, 32, DL>(v, p.eps);
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    float y[8];
                    norm8<BF16>(v[i], __ldg(reinterpret_cast<const uint4*>(p.weight) + lane + 32 * i), r, y);
                    v[i] = pack8<BF16>(y);
                }
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) dst[lane + 32 * i] = v[i];
            continue;
        }
        const int rr = (gr - 1) * 8 + (lane >> 2);  // 0: the key part, 1 ..: query head rr - 1
        if (rr >= rows || (rr == 0 && slot < 0)) continue;
        const uint16_t* src = rr == 0 ? p.kv + t * p.kv_stride + DL
                                      : p.q_pe + t * p.pe_token_stride + (int64_t)(rr - 1) * p.pe_head_stride;
        uint16_t* dst = rr == 0 ? p.cache + slot * ROW + DL : p.q + (t * p.n_heads + rr - 1) * ROW + DL;
        const uint4 lo = reinterpret_cast<const uint4*>(src)[c], hi = reinterpret_cast<const uint4*>(src)[c + 4];
        const float* cs = p.cos_sin + pos * 64;
        float a[8], b[8];
        unpack8<BF16>(lo, a);
        unpack8<BF16>(hi, b);
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
