// gdn_attn_step.cuh -- attention of at most 16 rows a key head (a step's
// query heads, or a window row or two): the rows are the columns of the
// products, the keys their rows,
//     S^T [128 keys x 16] = K [128 x D] . Q^T,   O^T [D x 16] = V^T [D x 128] . P^T,
// so a tile costs an eighth of the tensor time that rows padded to 128
// would, and a step is bound by the copies.
//
// Five parts of a CTA run at their own pace, a tile or two apart: copies,
// products, weights (warpgroup 0), sums (warpgroup 1) and, an item ahead, the
// queries.  Scores, weights and products have two buffers each.
//
// Measured: 64 streams of 8192 tokens of 16 bits (32 heads on 8 of 128): 345 us, 6.2 TB/s,
// the copies bind.  4 streams of 65 to 131 k e4m3 tokens (24 heads on 4 of 256): 178 us, 5.2 TB/s, where a tile's copy
// and the issue of its products take about as long (187 us with fp16 rows, whose queries are three parts).
// One stream of 4722 bf16 tokens: 16.4 us, latency.
//
// The e4m3 parts of a query or a weight are columns side by side: a product
// of 48 columns takes the tensor cores no longer than one of 16 (46 clocks), so
// three parts cost what one does, and their results are added as they are read.  So are the two 16-bit parts of
// a weight for heads of up to 128 elements (64 uneven streams: 67 us fp16, 69 bf16; one after the other into one sum
// 80).  For 256 the window kernel has no room in TMEM for two sums, and its rows have a step's bits, so there they are
// one after the other.
#pragma once

#include "gdn_attn_join.cuh"

namespace gdn {

constexpr int kStepThreads = 384;   // weights, sums, then copies, products and two warps of queries

struct StepShared {
    float wmax[8][4][kStepCols], wsum[8][4][kStepCols];   // [tile & 7][warp][column]: sums run up to 4 tiles behind
    float2 fac[2][kStepCols], whole[2][kStepCols];        // factors of the fold onto a span, and of that onto an item
    float inv[2][kStepCols];                              // 1 / sum of an item
    AttnRows<kStepCols> rows;
};

// The weights of W columns of a tile, thread = key.
template <int W, int D, int ACT, int KV>
__device__ __forceinline__ void step_weights_of(AttnShared &sh, StepShared &st, const AttnFacts &f, int item, float c,
                                                uint32_t scores, uint8_t *to, int it, int *err) {
    using Parts = AttnParts<ACT, KV>;
    constexpr int N = kStepCols;
    const int key = threadIdx.x, lane = key & 31, warp = key >> 5;
    uint32_t hide = 0;   // columns that do not see this key
    if (key >= f.tail) {
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (!(key < f.last && (st.rows.sees[item & 3][j] >> (key - f.tail)) & 1)) hide |= 1u << j;
    }
    float t[W], r[W];
    tmem_ld(scores + ((uint32_t)(warp * 32) << 16), t);
#pragma unroll
    for (int q = 1; q < Parts::kQuery; ++q) {
        tmem_ld(scores + q * N + ((uint32_t)(warp * 32) << 16), r);
#pragma unroll
        for (int j = 0; j < W; ++j) t[j] = __fmaf_rn(r[j], q == 1 ? 1.0f / Parts::kNext : 1.0f / (Parts::kNext * Parts::kNext), t[j]);
    }
    // the tile's largest score of each column
#pragma unroll
    for (int j = 0; j < W; ++j) {
        if constexpr (KV == GDN_E4M3) t[j] = __fmul_rn(t[j], st.rows.unscale[item & 3][j]);
        r[j] = warp_max((hide >> j) & 1 ? -INFINITY : __fmul_rn(t[j], c));
    }
    if (lane == 0) {
#pragma unroll
        for (int j = 0; j < W; j += 4)
            *reinterpret_cast<float4 *>(&st.wmax[it & 7][warp][j]) = make_float4(r[j], r[j + 1], r[j + 2], r[j + 3]);
    }
    named_barrier<1, 128>();
#pragma unroll
    for (int j = 0; j < W; j += 4) {
        float4 m = *reinterpret_cast<const float4 *>(&st.wmax[it & 7][0][j]);
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            const float4 o = *reinterpret_cast<const float4 *>(&st.wmax[it & 7][w][j]);
            m = make_float4(fmaxf(m.x, o.x), fmaxf(m.y, o.y), fmaxf(m.z, o.z), fmaxf(m.w, o.w));
        }
        r[j] = ref_of<ACT, KV>(reference_of(m.x)), r[j + 1] = ref_of<ACT, KV>(reference_of(m.y));
        r[j + 2] = ref_of<ACT, KV>(reference_of(m.z)), r[j + 3] = ref_of<ACT, KV>(reference_of(m.w));
    }
#pragma unroll
    for (int j = 0; j < W; ++j) t[j] = (hide >> j) & 1 ? 0.0f : weight_of(t[j], c, r[j]);
    // the weights of the tile before last have been read
    if (it >= 2) attn_wait(sh, &sh.ofull[it & 1], ((it >> 1) - 1) & 1, err);
    // as the second operand: column j's keys in swizzled rows of 128 bytes
    if constexpr (KV == GDN_E4M3) {
#pragma unroll
        for (int j = 0; j < W; j += 2) {
            uint8_t *at0 = to + j * 128 + ((uint32_t)key ^ ((uint32_t)(j & 7) << 4));
            uint8_t *at1 = to + (j + 1) * 128 + ((uint32_t)key ^ ((uint32_t)((j + 1) & 7) << 4));
            float x = t[j], y = t[j + 1];
#pragma unroll
            for (int q = 0; q < Parts::kWeight; ++q) {
                const uint16_t two = Elem<GDN_E4M3>::pack2(x, y);
                at0[q * N * 128] = (uint8_t)two;
                at1[q * N * 128] = (uint8_t)(two >> 8);
                const float2 top = Elem<GDN_E4M3>::unpack2(two);
                x = __fmaf_rn(top.x, -Parts::kNext, x * Parts::kNext);   // (exact)
                y = __fmaf_rn(top.y, -Parts::kNext, y * Parts::kNext);
            }
        }
    } else {
        uint8_t *rows = to + (key >> 6) * Parts::kWeight * N * 128;
#pragma unroll
        for (int j = 0; j < W; j += 2) {
            float x = t[j], y = t[j + 1];
            const uint32_t top = first_parts<KV>(x, y), rest = Elem<KV>::pack2(x, y);
            uint8_t *at0 = rows + j * 128 + ((uint32_t)(key & 63) * 2 ^ ((uint32_t)(j & 7) << 4));
            uint8_t *at1 = rows + (j + 1) * 128 + ((uint32_t)(key & 63) * 2 ^ ((uint32_t)((j + 1) & 7) << 4));
            *reinterpret_cast<uint16_t *>(at0) = (uint16_t)top;
            *reinterpret_cast<uint16_t *>(at1) = (uint16_t)(top >> 16);
            *reinterpret_cast<uint16_t *>(at0 + N * 128) = (uint16_t)rest;
            *reinterpret_cast<uint16_t *>(at1 + N * 128) = (uint16_t)(rest >> 16);
        }
    }
    const float l = reduce_scatter<W>(t, lane);
    if (lane % (32 / W) == 0) st.wsum[it & 7][warp][lane / (32 / W)] = l;
}

template <int D, int ACT, int KV>
__global__ void __launch_bounds__(kStepThreads, 1) gdn_attn_step_kernel(const __grid_constant__ AttnTcParams p) {
    using T = AttnTile<D, KV>;
    using Parts = AttnParts<ACT, KV>;
    constexpr int N = kStepCols, kScores = N * Parts::kQuery, kSums = N * kAside<D, ACT, KV>;   // columns of the two products
    constexpr uint32_t kNeed = 2 * kScores + 2 * T::kHalves * kSums;                         // of TMEM: each twice
    constexpr uint32_t kTmemCols = kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
    constexpr uint32_t kQueries = attn_queries<D, ACT, KV>(N);
    static_assert(sizeof(AttnShared) + sizeof(StepShared) <= 227 * 1024 - kStepSmem, "shared memory");
    extern __shared__ uint8_t dyn[];
    __shared__ AttnShared sh;
    __shared__ StepShared st;
    const AttnParams &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t *stages = dyn + ((1024 - (tc::smem_u32(dyn) & 1023)) & 1023);
    uint8_t *sq = stages + p.n_stages * T::kBytes, *sp = sq + 2 * kQueries;
    int lo, hi;
    if (!attn_prologue<kStepThreads>(p, sh, kTmemCols, 4, false, lo, hi)) return;
    const int n = hi - lo;
    const uint32_t tmem = sh.tmem, tmem_o = tmem + 2 * kScores;

    if (warp == 8) {
        attn_copies<T>(p, sh, stages, lo, hi);
    } else if (warp == 9) {
        if (lane == 0) {
            constexpr uint32_t kDescS = kMmaDesc<ACT, KV> | ((uint32_t)(kScores >> 3) << 17);
            constexpr uint32_t kDescO = kMmaDesc<ACT, KV> | ((uint32_t)(kSums >> 3) << 17) | (1u << 15);
            const uint32_t saddr = tc::smem_u32(stages);
            const uint64_t dq = swizzled_desc<T::kBlock>(tc::smem_u32(sq), 16, T::kAtom);
            const uint64_t dp = swizzled_desc<128>(tc::smem_u32(sp), 16, 1024);
            int items = -1;
            AttnRing ring = {0, 0};
            // scores of tile it + 1, then the product of tile it
#pragma unroll 1
            for (int it = -1; it < n; ++it) {
                if (it + 1 < n) {
#pragma unroll 1
                    for (int half = 0; half < T::kPieces; ++half, ring.next(p.n_stages)) {
                        attn_wait(sh, &sh.full[ring.at], ring.parity, a.err);
                        if (half == 0 && (sh.facts[(it + 1) % kAttnTiles].flags & kOpens)) {
                            if (items >= 0) tc::mma_commit(&sh.qempty[items & 1]);
                            ++items;
                            attn_wait(sh, &sh.qfull[items & 1], (uint32_t)(items >> 1) & 1, a.err);
                        }
                        tc::fence_after_sync();
                        const uint64_t dk = swizzled_desc<T::kBlock>(saddr + ring.at * T::kBytes, 16, T::kGroup);
                        const uint64_t qi = dq + (items & 1) * (kQueries / 16);
#pragma unroll
                        for (int k = 0; k < T::kBlocks * T::kBlock / 32; ++k) {
                            const int b = k / (T::kBlock / 32), kk = k % (T::kBlock / 32);
                            mma_ss<KV>(tmem + ((it + 1) & 1) * kScores, dk + b * (T::kAtom / 16) + kk * 2,
                                       qi + (half * T::kBlocks + b) * (kScores * T::kBlock / 16) + kk * 2, kDescS, half + k > 0);
                        }
                        tc::mma_commit(&sh.empty[ring.at]);
                    }
                    tc::mma_commit(&sh.sfull[(it + 1) & 1]);
                }
                if (it < 0) continue;
                attn_wait(sh, &sh.pfull[it & 1], (it >> 1) & 1, a.err);
                if (it >= 2) attn_wait(sh, &sh.ofree[it & 1], ((it >> 1) - 1) & 1, a.err);
                const int steps = value_steps<T>(sh.facts[it % kAttnTiles].last);
#pragma unroll 1
                for (int half = 0; half < T::kHalves; ++half) {
                    if (half == 0 || T::kPiecesHalf) attn_wait(sh, &sh.full[ring.at], ring.parity, a.err);
                    tc::fence_after_sync();
                    const uint64_t dv = swizzled_desc<T::kBlock>(
                        saddr + ring.at * T::kBytes + half * T::kBlocksHalf * T::kAtom, T::kAtom, T::kGroup);
                    const uint64_t pi = dp + (it & 1) * (step_weights<ACT, KV> / 16);
                    const uint32_t to = tmem_o + ((it & 1) * T::kHalves + half) * kSums;
                    auto value_step = [&](int k) {
#pragma unroll
                        for (int q = 0; q < Parts::kWeight / kAside<D, ACT, KV>; ++q)
                            mma_ss<KV>(to, dv + k * ((T::kStepKeys / 8) * T::kGroup / 16),
                                       pi + (k / 4 * Parts::kWeight + q) * (N * 128 / 16) + k % 4 * 2, kDescO, k + q > 0);
                    };
                    if (steps == T::kSteps) {   // (a branch a step would double the products' issue)
#pragma unroll
                        for (int k = 0; k < T::kSteps; ++k) value_step(k);
                    } else {
#pragma unroll 1
                        for (int k = 0; k < steps; ++k) value_step(k);
                    }
                    if (half == T::kHalves - 1 || T::kPiecesHalf) {
                        tc::mma_commit(&sh.empty[ring.at]);
                        ring.next(p.n_stages);
                    }
                }
                tc::mma_commit(&sh.ofull[it & 1]);
            }
            tc::mma_commit(&sh.done);
            tc::mbar_wait(&sh.done, 0, kAttnWaitLimit);
        }
    } else if (warp >= 10) {
        attn_queries_ahead<D, ACT, KV, 2, 2>(p, sh, st.rows, sq, kQueries, N, kScores, N * T::kBlock, n, tid - 320);
    } else if (warp < 4) {
        // ---- weights: thread = key of the tile
        int item = -1;
        const float l2e = 1.4426950408889634f * a.scale;
#pragma unroll 1
        for (int it = 0; it < n; ++it) {
            attn_wait(sh, &sh.sfull[it & 1], (it >> 1) & 1, a.err);
            tc::fence_after_sync();
            const AttnFacts f = sh.facts[it % kAttnTiles];
            if (f.flags & kOpens) ++item;
            const float c = a.k_scale ? l2e * a.k_scale[f.head] : l2e;
            uint8_t *to = sp + (it & 1) * step_weights<ACT, KV>;
            // (4 columns for themselves: 64 uneven streams of 4 query heads a key head 67 us, 80 with 8; over an 8-bit
            // cache 70 and 85, but there the third copy of the code costs items of 6 columns 4 %: 177 to 184 us)
            if (KV != GDN_E4M3 && f.cols <= 4) step_weights_of<4, D, ACT, KV>(sh, st, f, item, c, tmem + (it & 1) * kScores, to, it, a.err);
            else if (f.cols <= 8) step_weights_of<8, D, ACT, KV>(sh, st, f, item, c, tmem + (it & 1) * kScores, to, it, a.err);
            else step_weights_of<16, D, ACT, KV>(sh, st, f, item, c, tmem + (it & 1) * kScores, to, it, a.err);
            if (f.tail < kTileKeys)
                clean_values<D, KV, 128>(p, sh, stages, it, n, f.tail, f.last, &sh.vbad[it & 7], tid);
            tc::fence_before_sync();
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.pfull[it & 1]);
        }
    } else {
        // ---- sums: thread = element of a half of the head
        const int wl = warp & 3, elem = wl * 32 + lane, col = elem;
        const uint32_t lane_base = (uint32_t)(wl * 32) << 16;
        const bool owns = D != 64 || elem < 64;
        float A[T::kHalves][N], Y[T::kHalves][N];         // of the span; of an item that lies whole in this run
        float run_m = 0.0f, run_l = 0.0f, item_m = 0.0f, item_l = 0.0f;   // of column `col`
        bool fresh = false;                               // no span of the item yet
        uint32_t vbad = 0;
        bool bad = false;
#pragma unroll 1
        for (int it = 0; it < n; ++it) {
            attn_wait(sh, &sh.ofull[it & 1], (it >> 1) & 1, a.err);
            tc::fence_after_sync();
            const AttnFacts f = sh.facts[it % kAttnTiles];
            const bool first = f.flags & kFirst, last = f.flags & kLast, whole = f.flags & kWhole;
            if (f.flags & kOpens) {
                bad = false;
                vbad = 0;
                fresh = true;
            }
            bad |= (f.flags & kRefused) != 0;
            if (f.tail < kTileKeys) vbad |= sh.vbad[it & 7];
            if (col < N) {
                const float(*m)[N] = st.wmax[it & 7], (*l)[N] = st.wsum[it & 7];
                const float tm = reference_of(fmaxf(fmaxf(m[0][col], m[1][col]), fmaxf(m[2][col], m[3][col])));
                const float tl = __fadd_rn(__fadd_rn(__fadd_rn(l[0][col], l[1][col]), l[2][col]), l[3][col]);
                Fold e = {0.0f, 1.0f};
                if (first) {
                    run_m = tm;
                    run_l = tl;
                } else {
                    e = fold_stats(run_m, run_l, tm, tl);
                }
                st.fac[it & 1][col] = make_float2(e.e1, e.e2);
                if (last && whole) {
                    Fold w = {0.0f, 1.0f};
                    if (fresh) {
                        item_m = run_m;
                        item_l = run_l;
                    } else {
                        w = fold_stats(item_m, item_l, run_m, run_l);
                    }
                    st.whole[it & 1][col] = make_float2(w.e1, w.e2);
                    st.inv[it & 1][col] = __fdiv_rn(1.0f, item_l);
                } else if (last) {
                    float2 *to = slot_stat(p, f.slot);
                    if (col < f.cols) to[col] = make_float2(run_m, bad || *(volatile int *)&sh.abort ? -1.0f : run_l);
                    if (col == 0) to[p.slot_cols] = make_float2(__uint_as_float(vbad), 0.0f);
                }
            }
            named_barrier<2, 128>();
            if (col == 0) sh.vbad[it & 7] = 0;
#pragma unroll
            for (int half = 0; half < T::kHalves; ++half) {
#pragma unroll
                for (int c8 = 0; c8 < N; c8 += 8) {
                    if (c8 >= f.cols) break;
                    float o[8];
                    const uint32_t from = tmem_o + ((it & 1) * T::kHalves + half) * kSums + c8 + lane_base;
                    tmem_ld(from, o);
#pragma unroll
                    for (int q = 1; q < kAside<D, ACT, KV>; ++q) {
                        float more[8];
                        tmem_ld(from + q * N, more);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            o[j] = __fmaf_rn(more[j], q == 1 ? 1.0f / Parts::kNext : 1.0f / (Parts::kNext * Parts::kNext), o[j]);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 e = st.fac[it & 1][c8 + j];
                        const float sum = fold_sum(A[half][c8 + j], o[j], Fold{e.x, e.y});
                        A[half][c8 + j] = first ? o[j] : sum;
                    }
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.ofree[it & 1]);
            if (!last || !owns) continue;
            if (!whole) {
#pragma unroll
                for (int half = 0; half < T::kHalves; ++half) {
                    const int e = half * 128 + elem;
                    float *dst = slot_sums(p, f.slot) + (e >> 2) * p.slot_cols * 4 + (e & 3);
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        if (j < f.cols) dst[j * 4] = A[half][j];
                }
                continue;
            }
#pragma unroll
            for (int half = 0; half < T::kHalves; ++half) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    if (j >= f.cols) break;
                    const float2 w = st.whole[it & 1][j];
                    const float sum = fold_sum(Y[half][j], A[half][j], Fold{w.x, w.y});
                    Y[half][j] = fresh ? A[half][j] : sum;
                }
            }
            fresh = false;
            if (!(f.flags & kEnds) || *(volatile int *)&sh.abort) continue;
            if (bad) {
                if (elem == 0) raise_error(a.err, GDN_DERR_PAGES);
                continue;
            }
            const float vs = a.v_scale ? a.v_scale[f.head] : 1.0f;
#pragma unroll
            for (int half = 0; half < T::kHalves; ++half) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    if (j >= f.cols) break;
                    const float y = Y[half][j] * st.inv[it & 1][j] * vs;
                    const int i = j * p.inv_G >> 16;
                    typename Elem<ACT>::type *to = reinterpret_cast<typename Elem<ACT>::type *>(
                                                       out_row(a, D, f.row, f.head, i, j - i * a.G)) + half * 128 + elem;
                    if constexpr (ACT == GDN_BF16) *to = __float2bfloat16_rn(y);
                    else *to = __float2half_rn(y);
                }
            }
            if (vbad) {
#pragma unroll 1
                for (int j = 0; j < f.cols; ++j) {
                    const int i = j * p.inv_G >> 16;
                    char *row = out_row(a, D, f.row, f.head, i, j - i * a.G);
#pragma unroll 1
                    for (int half = 0; half < T::kHalves; ++half)
                        give_back<D, ACT, KV>(p, f.stream, f.head, f.i0 + i, vbad, row, half * 128 + elem, 1);
                }
            }
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 9) tc::tmem_dealloc(tmem, kTmemCols);
    attn_finish<D, ACT, KV, kStepThreads, true>(p, sh, stages, p.n_stages * T::kBytes);
}

}  // namespace gdn
