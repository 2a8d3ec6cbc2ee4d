// gdn_attn_window.cuh -- attention of windows: up to 128 rows of a key head
// (window rows times the query heads that read it) against 128 keys at once,
//     S [128 rows x 128 keys] = Q . K^T,   O [128 x D] = P . V.
// A thread of the weights has one row: its maximum, weights and sum need no
// other thread.  The weights take the place of the scores in TMEM and are the
// second product's first operand.  Two warpgroups hold the sums, a row a
// thread and half of the head each.  The parts run as in the step kernel;
// scores have two buffers, the product one (TMEM is full).
//
// Measured: 16 streams x 16 rows over 512 to 8192 bf16 tokens (24 heads on 4 of 256): 87 us, 205 TFLOP/s,
// 2.2 TB/s of cache beside 57 MB of pieces out and in.  The chain within a tile binds, scores to weights to
// product to sums: with equal lengths each further tile of a CTA takes 4.6 us (96 rows, heads of 256), 2.7
// (64 rows of 128) or 3.1 (128 rows of 128), where its copies need 2.9 and 1.5.  At 128 registers a thread the kernels for
// 256 elements spill 100 to 250 bytes, those for 64 and 128 16 to 28.
#pragma once

#include "gdn_attn_join.cuh"

namespace gdn {

constexpr int kWindowThreads = 512;   // weights, sums of two halves, then copies, products, queries and cleaning

struct WindowShared {
    float2 stat[8][128];      // [tile & 7][row]: reference and sum of weights
    AttnRows<128> rows;
};

// Cleaning of values, by a warp of its own while the weights are worked out: by their warps it took 1 to 2.5 k clocks
// of a last tile's 6.  (The step kernel's do it themselves: there a fifth arrival a tile cost more, 72 -> 78 us for 64 streams.)
template <int D, int KV>
__device__ __forceinline__ void attn_clean(const AttnTcParams &p, AttnShared &sh, uint8_t *stages, int n) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int it = 0; it < n; ++it) {
        attn_wait(sh, &sh.sfull[it & 1], (it >> 1) & 1, p.a.err);   // (its facts are known)
        const int tail = sh.facts[it % kAttnTiles].tail, last = sh.facts[it % kAttnTiles].last;
        if (tail < kTileKeys) {
            // (the sums of the tile eight before have read theirs: their product's place was free for a later one)
            if (lane == 0) sh.vbad[it & 7] = 0;
            __syncwarp();
            clean_values<D, KV, 32>(p, sh, stages, it, n, tail, last, &sh.vbad[it & 7], lane);
            tc::fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.pfull[it & 1]);
    }
}

template <int D, int ACT, int KV>
__global__ void __launch_bounds__(kWindowThreads, 1) gdn_attn_window_kernel(const __grid_constant__ AttnTcParams p) {
    using T = AttnTile<D, KV>;
    using Parts = AttnParts<ACT, KV>;
    constexpr bool kApart = KV != GDN_E4M3 && kAside<D, ACT, KV> > 1;   // (the second part's product 128 columns on)
    constexpr int FN = D / 2;                             // sums a thread holds
    constexpr uint32_t kTmemCols = 512;                   // scores (then weights) twice, the product
    static_assert(sizeof(AttnShared) + sizeof(WindowShared) <= 227 * 1024 - kWindowSmem, "shared memory");
    extern __shared__ uint8_t dyn[];
    __shared__ AttnShared sh;
    __shared__ WindowShared st;
    const AttnParams &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nc = p.nc;
    // the queries first: a product reads 128 rows from there, of which the last may be pieces
    const uint32_t queries = (uint32_t)attn_queries<D, ACT, KV>(nc), query_part = queries / Parts::kQuery;
    uint8_t *sq = dyn + ((1024 - (tc::smem_u32(dyn) & 1023)) & 1023), *stages = sq + queries;
    int lo, hi;
    if (!attn_prologue<kWindowThreads>(p, sh, kTmemCols, 8, true, lo, hi)) return;
    const int n = hi - lo;
    const uint32_t tmem = sh.tmem, tmem_o = tmem + 256;

    // registers of the warpgroups: 104 + 2 x 176 + 56 = 4 x 128, what the block was launched with
    if (warp >= 12) {
        registers_down<56>();
        if (warp == 12) {
            attn_copies<T>(p, sh, stages, lo, hi);
        } else if (warp == 13) {
            if (lane == 0) {
                constexpr uint32_t kDescS = kMmaDesc<ACT, KV> | ((uint32_t)(kTileKeys >> 3) << 17);
                constexpr uint32_t kDescO = kMmaDesc<ACT, KV> | ((uint32_t)((D < 128 ? D : 128) >> 3) << 17) | (1u << 16);
                const uint32_t saddr = tc::smem_u32(stages);
                const uint64_t dq = swizzled_desc<T::kBlock>(tc::smem_u32(sq), 16, T::kAtom);
                int items = -1;
                AttnRing ring = {0, 0};
                // scores of tile it + 1, then the product of tile it
#pragma unroll 1
                for (int it = -1; it < n; ++it) {
                    if (it + 1 < n) {
                        const uint32_t d = tmem + ((it + 1) & 1) * kTileKeys;
#pragma unroll 1
                        for (int half = 0; half < T::kPieces; ++half, ring.next(p.n_stages)) {
                            attn_wait(sh, &sh.full[ring.at], ring.parity, a.err);
                            if (half == 0 && (sh.facts[(it + 1) % kAttnTiles].flags & kOpens)) {
                                ++items;
                                attn_wait(sh, &sh.qfull[0], (uint32_t)items & 1, a.err);
                            }
                            tc::fence_after_sync();
                            const uint64_t dk = swizzled_desc<T::kBlock>(saddr + ring.at * T::kBytes, 16, T::kGroup);
#pragma unroll
                            for (int t = 0; t < Parts::kQuery * T::kBlocks; ++t) {
                                const int b = t % T::kBlocks, part = t / T::kBlocks;
                                const uint64_t kb = dk + b * (T::kAtom / 16),
                                               qb = dq + (part * query_part + (half * T::kBlocks + b) * nc * T::kBlock) / 16;
#pragma unroll
                                for (int kk = 0; kk < T::kBlock / 32; ++kk)
                                    mma_ss<KV>(d, qb + kk * 2, kb + kk * 2,
                                               KV == GDN_E4M3 && part + 1 == Parts::kQuery ? kDescS | kDescE5m2 : kDescS, half + t + kk > 0);
                            }
                            tc::mma_commit(&sh.empty[ring.at]);
                        }
                        tc::mma_commit(&sh.sfull[(it + 1) & 1]);
                        if (sh.facts[(it + 1) % kAttnTiles].flags & kEnds) tc::mma_commit(&sh.qempty[0]);
                    }
                    if (it < 0) continue;
                    attn_wait(sh, &sh.pfull[it & 1], (it >> 1) & 1, a.err);
                    if (it >= 1) attn_wait(sh, &sh.ofree[0], (uint32_t)(it - 1) & 1, a.err);
                    const uint32_t w = tmem + (it & 1) * kTileKeys;
                    const int steps = value_steps<T>(sh.facts[it % kAttnTiles].last);
#pragma unroll 1
                    for (int half = 0; half < T::kHalves; ++half) {
                        if (half == 0 || T::kPiecesHalf) attn_wait(sh, &sh.full[ring.at], ring.parity, a.err);
                        tc::fence_after_sync();
                        const uint64_t dv = swizzled_desc<T::kBlock>(
                            saddr + ring.at * T::kBytes + half * T::kBlocksHalf * T::kAtom, T::kAtom, T::kGroup);
                        auto value_step = [&](int k) {
#pragma unroll
                            for (int part = 0; part < Parts::kWeight; ++part)
                                mma_ts<KV>(tmem_o + (half + (kApart ? part : 0)) * 128, w + k * T::kStepKeys + part * 8,
                                           dv + k * ((T::kStepKeys / 8) * T::kGroup / 16),
                                           KV == GDN_E4M3 && part + 1 == Parts::kWeight ? kDescO | kDescE5m2 : kDescO,
                                           k + (kApart ? 0 : part) > 0);
                        };
                        if (steps == T::kSteps) {
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
        } else if (warp == 14) {
            attn_queries_ahead<D, ACT, KV, 1, 1>(p, sh, st.rows, sq, queries, nc, nc, query_part, n, lane);
        } else {
            attn_clean<D, KV>(p, sh, stages, n);
        }
    } else if (warp < 4) {
        registers_down<104>();
        // ---- weights: thread = row
        const int row = tid;
        int item = -1;
        const float l2e = 1.4426950408889634f * a.scale;
#pragma unroll 1
        for (int it = 0; it < n; ++it) {
            attn_wait(sh, &sh.sfull[it & 1], (it >> 1) & 1, a.err);
            tc::fence_after_sync();
            const AttnFacts f = sh.facts[it % kAttnTiles];
            if (f.flags & kOpens) ++item;
            if (warp * 32 < f.cols) {
                const float c = a.k_scale ? l2e * a.k_scale[f.head] : l2e;
                const float unscale = KV == GDN_E4M3 && row < f.cols ? st.rows.unscale[item & 3][row] : 1.0f;
                const uint32_t scores = tmem + (it & 1) * kTileKeys + ((uint32_t)(warp * 32) << 16);
                // keys from `tail` on are seen as the row's mask says (its bits end with the window)
                uint32_t in = 0;
                if (f.tail < kTileKeys && row < f.cols) in = st.rows.sees[item & 3][row] & ((1u << (f.last - f.tail)) - 1);
                auto hidden = [&](int b) {   // of keys 32 b .. 32 b + 31
                    const int at = f.tail - b * 32;
                    return at >= 32 ? 0u : ~(at >= 0 ? ((1u << at) - 1) | (in << at) : at > -32 ? in >> -at : 0u);
                };
                // (loops that stay loops: a tile's code, unrolled, would not fit the instruction caches)
                float m = -INFINITY;
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    uint32_t s0[16], s1[16];
                    tc::tmem_ld16_nowait(scores + b * 32, s0);
                    tc::tmem_ld16_nowait(scores + b * 32 + 16, s1);
                    tc::tmem_wait_ld();
                    const uint32_t hide = hidden(b);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        float x = __uint_as_float(j < 16 ? s0[j & 15] : s1[j & 15]);
                        x = __fmul_rn(KV == GDN_E4M3 ? __fmul_rn(x, unscale) : x, c);
                        if (hide && (hide >> j) & 1) x = -INFINITY;
                        m = fmaxf(m, x);
                    }
                }
                m = reference_of(m);
                const float ref = ref_of<ACT, KV>(m);
                float sum = 0.0f;
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    float t[32];
                    uint32_t s0[16], s1[16];
                    tc::tmem_ld16_nowait(scores + b * 32, s0);
                    tc::tmem_ld16_nowait(scores + b * 32 + 16, s1);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float x = __uint_as_float(j < 16 ? s0[j & 15] : s1[j & 15]);
                        t[j] = weight_of(KV == GDN_E4M3 ? __fmul_rn(x, unscale) : x, c, ref);
                    }
                    if (const uint32_t hide = hidden(b)) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if ((hide >> j) & 1) t[j] = 0.0f;
                    }
                    float s[16];   // in the order of a warp's butterfly, as the step kernel adds them
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[j] = __fadd_rn(t[j], t[j + 16]);
#pragma unroll
                    for (int off = 8; off; off >>= 1)
#pragma unroll
                        for (int j = 0; j < off; ++j) s[j] = __fadd_rn(s[j], s[j + off]);
                    sum = __fadd_rn(sum, s[0]);
                    // over the scores that were read: a step's first parts in 8 columns, then its next
#pragma unroll
                    for (int q = 0; q < 32 / T::kStepKeys; ++q) {
#pragma unroll
                        for (int part = 0; part < Parts::kWeight; ++part) {
                            uint32_t w[8];
#pragma unroll
                            for (int j = 0; j < T::kStepKeys / 2; ++j) {
                                float &x = t[q * T::kStepKeys + 2 * j], &y = t[q * T::kStepKeys + 2 * j + 1];
                                uint32_t two;
                                if (KV != GDN_E4M3 && part == 0) {
                                    two = first_parts<KV>(x, y);
                                } else if (KV == GDN_E4M3 && part + 1 == Parts::kWeight) {
                                    two = pack2_e5m2(x, y);
                                } else {
                                    two = Elem<KV>::pack2(x, y);
                                    if (part + 1 < Parts::kWeight) {
                                        const float2 top = Elem<KV>::unpack2(two);
                                        x = __fsub_rn(x, top.x);
                                        y = __fsub_rn(y, top.y);
                                    }
                                }
                                if constexpr (KV == GDN_E4M3) w[j / 2] = j & 1 ? w[j / 2] | two << 16 : two;
                                else w[j] = two;
                            }
                            tc::tmem_st8_nowait(scores + b * 32 + q * T::kStepKeys + part * 8, w);
                        }
                    }
                }
                st.stat[it & 7][row] = make_float2(m, sum);
                tc::tmem_wait_st();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.pfull[it & 1]);
        }
    } else {
        registers_up<176>();
        // ---- sums: thread = row, warpgroup = half of the head
        const int half = (warp >> 2) - 1, wl = warp & 3, row = wl * 32 + lane;
        const uint32_t fold_t = tmem_o + half * FN + ((uint32_t)(wl * 32) << 16);
        float A[FN];
        float run_m = 0.0f, run_l = 0.0f;                 // of the span
        float item_m = 0.0f, item_l = 0.0f;               // of an item that lies whole in this run
        int item_slot = 0;                                // where its sums wait between spans
        bool fresh = false;                               // no span of the item yet
        uint32_t vbad = 0;
        bool bad = false;
#pragma unroll 1
        for (int it = 0; it < n; ++it) {
            attn_wait(sh, &sh.ofull[it & 1], (it >> 1) & 1, a.err);
            tc::fence_after_sync();
            const AttnFacts f = sh.facts[it % kAttnTiles];
            const bool first = f.flags & kFirst, last = f.flags & kLast, live = wl * 32 < f.cols;
            const bool ends = f.flags & kEnds, whole = f.flags & kWhole;
            if (f.flags & kOpens) {
                bad = false;
                vbad = 0;
                fresh = true;
            }
            bad |= (f.flags & kRefused) != 0;
            if (f.tail < kTileKeys) vbad |= sh.vbad[it & 7];
            Fold e = {0.0f, 1.0f};
            if (live) {
                const float2 tile = st.stat[it & 7][row];
                if (first) {
                    run_m = tile.x;
                    run_l = tile.y;
                } else {
                    e = fold_stats(run_m, run_l, tile.x, tile.y);
                }
#pragma unroll
                for (int b = 0; b < FN; b += 16) {
                    float t[16];
                    tc::tmem_ld16(fold_t + b, t);
                    if constexpr (kApart) {
                        float more[16];
                        tc::tmem_ld16(fold_t + 128 + b, more);
#pragma unroll
                        for (int j = 0; j < 16; ++j) t[j] = __fadd_rn(t[j], more[j]);
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float sum = fold_sum(A[b + j], t[j], e);
                        A[b + j] = first ? t[j] : sum;
                    }
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.ofree[0]);
            if (!last) continue;
            if (fresh) item_slot = f.slot;
            if (row < f.cols) {
                float4 *slot = reinterpret_cast<float4 *>(slot_sums(p, whole ? item_slot : f.slot)) +
                               half * (FN / 4) * p.slot_cols + row;
                if (!whole) {
                    if (half == 0) {
                        float2 *to = slot_stat(p, f.slot);
                        to[row] = make_float2(run_m, bad || *(volatile int *)&sh.abort ? -1.0f : run_l);
                        if (row == 0) to[p.slot_cols] = make_float2(__uint_as_float(vbad), 0.0f);
                    }
                } else if (fresh) {
                    item_m = run_m;
                    item_l = run_l;
                } else {
                    // a span joins the item: its sums so far are in the workspace, each thread's own
                    const Fold w = fold_stats(item_m, item_l, run_m, run_l);
                    const float4 *old = slot;
#pragma unroll
                    for (int b = 0; b < FN / 4; ++b, old += p.slot_cols) {
                        const float4 t = *old;
                        A[4 * b] = fold_sum(t.x, A[4 * b], w);
                        A[4 * b + 1] = fold_sum(t.y, A[4 * b + 1], w);
                        A[4 * b + 2] = fold_sum(t.z, A[4 * b + 2], w);
                        A[4 * b + 3] = fold_sum(t.w, A[4 * b + 3], w);
                    }
                }
                if (!whole || !ends) {
#pragma unroll
                    for (int b = 0; b < FN / 4; ++b, slot += p.slot_cols)
                        *slot = make_float4(A[4 * b], A[4 * b + 1], A[4 * b + 2], A[4 * b + 3]);
                } else if (bad) {
                    if (tid == 128) raise_error(a.err, GDN_DERR_PAGES);
                } else if (!*(volatile int *)&sh.abort) {
                    const float inv = __fdiv_rn(1.0f, item_l), vs = a.v_scale ? a.v_scale[f.head] : 1.0f;
                    const int i = row * p.inv_G >> 16;
                    char *to = out_row(a, D, f.row, f.head, i, row - i * a.G);
#pragma unroll
                    for (int b = 0; b < FN; b += 8) {
                        float y[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[j] = A[b + j] * inv;
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[j] *= vs;
                        store_floats<ACT, 8>(to + (half * FN + b) * 2, y);
                    }
                    if (vbad) give_back<D, ACT, KV>(p, f.stream, f.head, f.i0 + i, vbad, to, half * FN, FN);
                }
            }
            fresh = false;
        }
    }
    __syncwarp();
    if (warp < 4 || warp >= 12) registers_up<128>();
    else registers_down<128>();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 13) tc::tmem_dealloc(tmem, kTmemCols);
    attn_finish<D, ACT, KV, kWindowThreads, false>(p, sh, sq, (int)queries + p.n_stages * T::kBytes);
}

}  // namespace gdn
