// gdn_attn_prep.cuh -- from a layer's q, k, v projections to its attention's
// inputs: per-head RMSNorm of q and k, rotation of their leading d_rot
// elements by the row's position, k and v into the paged cache.  One pass:
// each element is read once and written once.
//
// The angle of pair i at position p is p * inv_freq[i] radians.  Only its
// fraction of a full turn matters, and in 64-bit fixed point that fraction is
// exact: with t = frac(inv_freq / 2 pi) * 2^64 as an integer, off by 1 at
// most, p * t modulo 2^64 (one integer product) is the turn's fraction,
// 2^-64 * |p| off at most.  Its upper 32 bits go through sincospif, so a position of a million is
// as exact as position one, where an fp32 product would be off by 0.06 rad.
#pragma once

#include "gdn_attn_common.cuh"

namespace gdn {

struct PrepParams {
    const char *q, *k, *v;
    char *q_out;
    long long q_row, q_head, k_row, k_head, v_row, v_head;   // strides in elements
    const char *q_norm, *k_norm;   // [D] or nullptr
    const double *inv_freq;        // [d_rot / 2]
    char *ck, *cv;                 // [n_pages, Hkv, page_size, D]
    const float *k_scale, *v_scale;   // [Hkv] or nullptr
    const int *row_pos, *row_slot;
    int Hq, Hkv, d_rot, interleaved, n_pages, page_size, n_rows;
    float rot_gain, norm_offset, eps;
    int *err;
};

constexpr int kPrepThreads = 256, kPrepCtas = 3;

// 2^64 * frac(inv_freq / 2 pi): the product and, from 1 / 2 pi in two parts, what it was rounded by
__device__ __forceinline__ unsigned long long turn_of(double inv_freq) {
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57, kTurn = 18446744073709551616.0;
    const double x = fabs(inv_freq), f = x * kHi, rest = fma(x, kLo, fma(x, kHi, -f));
    const unsigned long long t = __double2ull_rn((f - floor(f)) * kTurn) + (unsigned long long)__double2ll_rn(rest * kTurn);
    return inv_freq < 0.0 ? 0ull - t : t;
}

// cos and sin of pos * (the turn), times gain
__device__ __forceinline__ float2 rotation(int pos, unsigned long long turn, float gain) {
    const unsigned long long at = (unsigned long long)(long long)pos * turn;
    float s, c;
    sincospif((float)(int)(at >> 32) * 4.656612873077393e-10f, &s, &c);
    return make_float2(c * gain, s * gain);
}

// CTAs take rows in turn, kPrepCtas an SM; a lane has 8 consecutive elements of
// a head, a warp 256 / D heads.  The next row (or the next four groups of heads of this one) is on its way
// while one is worked on, and a pair's turn is a thread's for all its rows.  4722 rows of 48 heads of 128 take 30.7 us
// (3.8 TB/s): a row a CTA took 33.4, a head a warp with one load at a time 41, and four CTAs an SM, for which the
// registers do not suffice, 40.9.  No one limit is reached: 183 instructions for the 256 elements of a warp fill 62 % of
// the issue slots, the copies have 56 % of their rate; a warp's loads, shuffles and stores wait for one another.
template <int D, int ACT, int KV>
__global__ void __launch_bounds__(kPrepThreads, kPrepCtas) gdn_attn_prep_kernel(const PrepParams p) {
    constexpr int kLanes = D / 8, kGroup = kPrepThreads / kLanes, kAhead = 4;
    static_assert(D / 2 <= kPrepThreads, "a pair a thread");
    __shared__ __align__(16) float2 cs_of[2][D / 2];
    __shared__ __align__(16) float gains[2][D];   // of q and k
    const int tid = threadIdx.x, lane = tid & 31, h0 = tid / kLanes, e0 = tid % kLanes * 8;
    const int w0 = tid / 32 * (32 / kLanes);   // the warp's first head of a group
    const int normed = p.Hq + p.Hkv, heads = normed + p.Hkv, half = p.d_rot / 2, hl = half / 8;
    const int shift = __ffs(p.page_size) - 1;
    const bool first = e0 < half, rotated = e0 < p.d_rot;
    // of half-rotation: the lane whose elements are d_rot / 2 away
    const int other = rotated ? (first ? lane + hl : lane - hl) : lane;
    // where this thread's elements of a row are, and how far it is to the next row's
    const char *from[kAhead];
    long long stride[kAhead];
    auto aim = [&](int base) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int hh = base + j * kGroup + h0;
            from[j] = hh < p.Hq ? p.q + 2 * (hh * p.q_head) : hh < normed ? p.k + 2 * ((hh - p.Hq) * p.k_head)
                                                                          : p.v + 2 * ((hh - normed) * p.v_head);
            from[j] += 2 * e0;
            stride[j] = 2 * (hh < p.Hq ? p.q_row : hh < normed ? p.k_row : p.v_row);
        }
    };
    auto load = [&](int row, int base, uint4(&raw)[kAhead]) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (base + j * kGroup + h0 < heads) raw[j] = *reinterpret_cast<const uint4 *>(from[j] + row * stride[j]);
    };
    // (before the first row's loads: behind them it cost 4722 rows of 128-element heads 7 us, for want of registers)
    const unsigned long long turn = tid < half ? turn_of(p.inv_freq[tid]) : 0;
    aim(0);
    uint4 next[kAhead];
    int row = blockIdx.x, base = 0, buffer = 0;
    bool kept = false;
    load(row, 0, next);
    int pos = p.row_pos[row], place = p.row_slot[row];
    if (tid < D / 8) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const char *w = k ? p.k_norm : p.q_norm;
            float g[8] = {};
            if (w) load_floats<ACT, 8>(w + 16 * tid, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) gains[k][8 * tid + i] = p.norm_offset + g[i];
        }
    }
    const float2 *cs = cs_of[0];
    long long cached = 0;   // the row's place in the pools, of head 0
    auto cache = [&](char *pool, const float *scale, int h, float(&x)[8]) {
        if constexpr (KV == GDN_E4M3) {
            if (scale) {
                const float s = scale[h];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], s);
            }
        }
        store_floats<KV, 8>(pool + (cached + ((long long)(h << shift) * D + e0)) * elem_bytes<KV>, x);   // (a page may pass 2^31)
    };
#pragma unroll 1
    while (row < p.n_rows) {
        uint4 raw[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) raw[j] = next[j];
        const int row_now = row, base_now = base;
        const int pos_now = pos, place_now = place;
        base += kAhead * kGroup;
        if (base < heads) {
            aim(base);
        } else {
            if (base_now > 0) aim(0);
            base = 0;
            row += gridDim.x;
            if (row < p.n_rows) {
                pos = p.row_pos[row];
                place = p.row_slot[row];
            }
        }
        if (row < p.n_rows) load(row, base, next);
        if (base_now == 0) {
            // (a buffer is written again two rows later, when all threads are past the row between)
            if (tid < half) cs_of[buffer][tid] = rotation(pos_now, turn, p.rot_gain);
            kept = false;
            if (place_now < -1 || place_now >= (long long)p.n_pages * p.page_size) {
                if (tid == 0) raise_error(p.err, GDN_DERR_PAGES);
            } else if (place_now >= 0) {
                kept = true;
                cached = (((long long)(place_now >> shift) * p.Hkv << shift) + (place_now & (p.page_size - 1))) * D;
            }
            __syncthreads();
            cs = cs_of[buffer];
            buffer ^= 1;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (base_now + j * kGroup + w0 >= heads) break;   // (all of the warp)
            const int hh = base_now + j * kGroup + h0;
            const bool is_q = hh < p.Hq, turns = rotated && hh < normed;
            float x[8];
            load_floats<ACT, 8>(&raw[j], x);
            if (base_now + j * kGroup + w0 >= normed) {   // values only
                if (kept && hh < heads) cache(p.cv, p.v_scale, hh - normed, x);
                continue;
            }
            const bool has = hh < normed && (is_q ? p.q_norm : p.k_norm);
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = __fmaf_rn(x[i], x[i], ss);
#pragma unroll
            for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
            if (has) {
                const float r = __frsqrt_rn(__fmaf_rn(ss, 1.0f / D, p.eps));
                const float4 *g = reinterpret_cast<const float4 *>(&gains[is_q ? 0 : 1][e0]);
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float4 w = g[i / 4];
                    x[i] = x[i] * r * w.x;
                    x[i + 1] = x[i + 1] * r * w.y;
                    x[i + 2] = x[i + 2] * r * w.z;
                    x[i + 3] = x[i + 3] * r * w.w;
                }
            }
            // (elements a, b of a pair: a c - b s, b c + a s)
            const float4 *t = reinterpret_cast<const float4 *>(cs + (p.interleaved ? e0 / 2 : first ? e0 : e0 - half));
            if (p.interleaved) {
                if (turns) {
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const float4 w = t[i / 4];
                        const float a = x[i], b = x[i + 1], c = x[i + 2], d = x[i + 3];
                        x[i] = a * w.x - b * w.y;
                        x[i + 1] = b * w.x + a * w.y;
                        x[i + 2] = c * w.z - d * w.w;
                        x[i + 3] = d * w.z + c * w.w;
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float y = __shfl_sync(kFull, x[i], other), z = __shfl_sync(kFull, x[i + 1], other);
                    if (turns) {
                        const float4 w = t[i / 2];
                        x[i] = first ? x[i] * w.x - y * w.y : x[i] * w.x + y * w.y;
                        x[i + 1] = first ? x[i + 1] * w.z - z * w.w : x[i + 1] * w.z + z * w.w;
                    }
                }
            }
            if (is_q) store_floats<ACT, 8>(p.q_out + 2 * ((size_t)row_now * (p.Hq * D) + (hh * D + e0)), x);
            else if (kept && hh < normed) cache(p.ck, p.k_scale, hh - p.Hq, x);
            else if (kept && hh < heads) cache(p.cv, p.v_scale, hh - normed, x);
        }
    }
}

}  // namespace gdn
