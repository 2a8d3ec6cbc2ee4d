// gdn_attn_join.cuh -- items that several runs share: their pieces, weighted
// by powers of two relative to the largest reference, are summed in order
// within a span and the spans added in order, which rounds as the kernels' folds do.
//
// An SM takes in some 23 bytes a clock, and an item's pieces are up to a
// megabyte, so each of the CTAs that share an item joins its part: of the
// item's sums as much as it had of the tiles.  They wait for each other, which a cooperative
// launch allows (all CTAs are there at once).  The counters need no
// preparation: a CTA gives them this call's token before it counts.
#pragma once

#include "gdn_attn_tc.cuh"

namespace gdn {

constexpr int kJoinSpans = 256;                         // spans at a time, at most
constexpr int kJoinPieces = kJoinSpans * kSpanMost;

// True once all tiles of the item have been counted in.  A CTA that gives up, here or before, says so in the counter
// before it counts (its tiles are counted in and out all the same), and nobody takes the item for complete any more.
__device__ __forceinline__ bool count_full(unsigned long long *counter, int all, uint32_t limit, int *err) {
#pragma unroll 1
    for (uint32_t i = 0; i < limit; ++i) {
        unsigned long long v;
        asm volatile("ld.acquire.gpu.u64 %0, [%1];" : "=l"(v) : "l"(counter) : "memory");
        if (v & kGaveUp) break;
        if (count_of(v) >= all) return true;
    }
    atomicOr(counter, kGaveUp);
    raise_error(err, GDN_DERR_TIMEOUT);
    return false;
}

// A piece of weight w joins a span's sums.
__device__ __forceinline__ float4 weigh(float4 t, float w, float4 s) {
    return make_float4(__fmaf_rn(t.x, w, s.x), __fmaf_rn(t.y, w, s.y), __fmaf_rn(t.z, w, s.z), __fmaf_rn(t.w, w, s.w));
}
// An item's four sums and sum of weights.
struct JoinSums {
    float y[4], L;
    __device__ __forceinline__ void scale(float f) {
#pragma unroll
        for (int v = 0; v < 4; ++v) y[v] *= f;
        L *= f;
    }
    __device__ __forceinline__ void add_span(float4 s, float l) {
        y[0] = __fadd_rn(y[0], s.x), y[1] = __fadd_rn(y[1], s.y), y[2] = __fadd_rn(y[2], s.z), y[3] = __fadd_rn(y[3], s.w);
        L = __fadd_rn(L, l);
    }
};

// This CTA's part of an item, T threads with four sums each; `smem` of `bytes` is free.  The part is lines of 32 sums
// (four elements of a column, column by column).  STAGED (steps, whose parts are a few lines of many
// pieces): the lines of all pieces are copied to shared memory while the pieces'
// statistics become weights.  Else (windows: hundreds of lines) a thread loads eight pieces at a time, which took
// 24 k clocks of a window's 377 KB a CTA where the staged copies took 42 k.
// False if the part is empty and nothing was waited for.
template <int D, int ACT, int KV, int T, bool STAGED>
__device__ __forceinline__ bool attn_join(const AttnTcParams &p, AttnShared &sh, const AttnCut &cut, uint8_t *smem,
                                          int bytes) {
    static_assert(T >= kJoinSpans, "a thread a span");
    const AttnParams &a = p.a;
    const AttnRuns runs = sh.runs;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cols = cut.cols;
    uint32_t *slots = reinterpret_cast<uint32_t *>(smem);          // [kJoinPieces] 16-byte units from the first slot
    uint32_t *ends = slots + kJoinPieces;                          // bits: pieces that end their span
    int *upto = reinterpret_cast<int *>(ends + kJoinPieces / 32);  // [8] pieces of a warp's spans
    int *starts = upto + kJoinSpans / 32;                          // [kJoinSpans + 4] a span's first piece
    uint32_t *flags = reinterpret_cast<uint32_t *>(starts + kJoinSpans + 4);   // given up; refused; window rows not all finite
    float *tops = reinterpret_cast<float *>(flags + 4);            // [128] per column: the largest reference so far
    float2 *stat = reinterpret_cast<float2 *>(tops + kAttnMaxCols);   // [column][piece and one]: (reference, sum of weights),
                                                                      // then (weight of the piece, sum)
    const int room = bytes - (int)(reinterpret_cast<uint8_t *>(stat) - smem);
    const int spans = stream_spans(cut.tiles), most = cut_most(runs), unit = p.slot_bytes / 16;
    // spans at a time: half of the room is for the statistics, half for a line at least; spans are
    // a piece each and up to `most` more for every run that starts in them, and 8 pieces at the most
    const int extra = (run_of(runs, cut.g0 + cut.tiles - 1) - cut.run) * most;
    const int fit = min(kJoinPieces, room / 2 / max(cols * (int)sizeof(float2), 128) - 2);
    const int block = min(min(kJoinSpans, spans), max(fit / kSpanMost, fit - extra));
    const int lines = cols * (D / 32);
    const int far = max(0, 12 - __clz(cut.tiles));   // (the products stay below 2^31)
    const int l0 = (unsigned)(lines * (cut.before >> far)) / (unsigned)(cut.tiles >> far);
    const int l1 = cut.before + cut.mine == cut.tiles
                       ? lines : (unsigned)(lines * ((cut.before + cut.mine) >> far)) / (unsigned)(cut.tiles >> far);
    bool waited = false;
    int pieces = 0, pitch = 0, group = 1;
    uint4 *data = nullptr;   // [piece][line][8]
#pragma unroll 1
    for (int line = l0; line < l1; line += group) {
        JoinSums at = {};
#pragma unroll 1
        for (int b = 0; b < spans; b += block) {
            const int m = min(block, spans - b);
            const bool lists = line == l0 || spans > block;
            if (lists) {
                if (waited) __syncthreads();
                if (tid < kJoinSpans) {
                    if (!STAGED && tid < kJoinPieces / 32) ends[tid] = 0;
                    // a span's pieces: what the run of its first tile folded, then tile by tile
                    int n = 0, run = 0, sum;
                    if (tid < m) {
                        const int stop = cut.g0 + min(cut.tiles, span_begin(b + tid + 1));
                        run = run_of(runs, cut.g0 + span_begin(b + tid));
                        n = 1 + max(0, stop - run_start(runs, run + 1));
                    }
                    sum = n;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int v = __shfl_up_sync(kFull, sum, o);
                        if (lane >= o) sum += v;
                    }
                    if (lane == 31) upto[warp] = sum;
                    named_barrier<1, kJoinSpans>();
#pragma unroll
                    for (int v = 0; v < kJoinSpans / 32; ++v)
                        if (v < warp) sum += upto[v];
                    starts[tid] = sum - n;
                    if (tid == m - 1) starts[m] = sum;
                    if (n) {
                        uint32_t slot = (uint32_t)slot_of(cut.span0 + b + tid, run, most) * unit;
#pragma unroll 1
                        for (int k = sum - n; k < sum; ++k, slot += unit) slots[k] = slot;
                        if (!STAGED) atomicOr(&ends[(sum - 1) >> 5], 1u << ((sum - 1) & 31));
                    }
                } else if (!waited && tid == kJoinSpans) {
                    // meanwhile the item's other runs are waited for
                    flags[1] = flags[2] = 0;
                    flags[0] = !count_full(p.counters + cut.run, cut.tiles, p.wait_limit, a.err);
                }
                waited = true;
                __syncthreads();
                if (flags[0]) return true;
                pieces = 0;
#pragma unroll
                for (int v = 0; v < kJoinSpans / 32; ++v) pieces += upto[v];
                pitch = (pieces + 1) | 1;
                data = reinterpret_cast<uint4 *>(stat) + (cols * pitch + 1) / 2;
                // (as many lines as any of several blocks has room for)
                const int upper = spans > block ? min(block * kSpanMost, block + extra) : pieces;
                group = STAGED ? min(T / 8, (room - (cols * (upper + 2) + 2) * 8) / (upper * 128)) : T / 8;
            }
            const int wide = min(group, l1 - line) * 8, k0 = tid / wide, at_once = T / wide;
            const int u = tid - k0 * wide, q = line * 8 + u, e4 = q / cols;
            const char *mine = p.slots + p.stat_bytes + (size_t)(e4 * p.slot_cols + q - e4 * cols) * 16;
            if (STAGED && k0 < at_once) {
#pragma unroll 2
                for (int k = k0; k < pieces; k += at_once) cp_async16(data + k * wide + u, mine + (size_t)slots[k] * 16);
            }
            if (lists) {
                // a warp a piece, a lane a column
                uint32_t bits = 0;
                bool refused = false;
#pragma unroll 1
                for (int u = warp * 4; u < pieces; u += T / 8) {
                    const float2 *st[4];
                    float2 v[4];
                    float odd[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        st[k] = reinterpret_cast<const float2 *>(p.slots + (size_t)slots[min(u + k, pieces - 1)] * 16);
                        odd[k] = __ldcg(&st[k][p.slot_cols].x);
                    }
#pragma unroll 1
                    for (int c = lane; c < cols; c += 32) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = __ldcg(st[k] + c);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            refused |= v[k].y == -1.0f;
                            stat[c * pitch + min(u + k, pieces - 1)] = v[k];
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) bits |= __float_as_uint(odd[k]);
                }
                if (refused) flags[1] = 1;
                if (bits) atomicOr(&flags[2], bits);
                __syncthreads();
                // a warp a column: the largest reference so far, and the pieces' weights
#pragma unroll 1
                for (int c = warp; c < cols; c += T / 32) {
                    float2 *of = stat + c * pitch;
                    const float before = b ? tops[c] : -INFINITY;
                    float top = before;
                    for (int u = lane; u < pieces; u += 32) top = fmaxf(top, of[u].x);
                    top = warp_max(top);
                    const float ref = zero_if_none(top);
                    for (int u = lane; u < pieces; u += 32) of[u].x = whole_exp2(__fsub_rn(of[u].x, ref));
                    __syncwarp();
                    if (lane == 0) {
                        tops[c] = top;
                        of[pieces].x = whole_exp2(__fsub_rn(before, ref));
                    }
                }
            }
            if (STAGED) cp_async_wait_all();
            if (STAGED || lists) __syncthreads();
            if constexpr (STAGED) {
                // a thread four sums of a span, left in the place of its first piece; then the spans in their order
                float4 *staged = reinterpret_cast<float4 *>(data);
#pragma unroll 1
                for (int w = tid; w < wide * m; w += T) {
                    const int span = w / wide, v = w - span * wide, end = starts[span + 1];
                    const float2 *weight = stat + (line * 8 + v) % cols * pitch;
                    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
                    for (int k = starts[span]; k < end; ++k) sum = weigh(staged[k * wide + v], weight[k].x, sum);
                    staged[starts[span] * wide + v] = sum;
                }
#pragma unroll 1
                for (int w = lists ? tid : cols * m; w < cols * m; w += T) {   // (their sums of weights, for all lines)
                    const int c = w / m, span = w - c * m, end = starts[span + 1];
                    float2 *weight = stat + c * pitch;
                    float l = 0.0f;
#pragma unroll 1
                    for (int k = starts[span]; k < end; ++k) l = __fmaf_rn(weight[k].y, weight[k].x, l);
                    weight[starts[span]].y = l;
                }
                __syncthreads();
                if (tid < wide) {
                    const float2 *weight = stat + q % cols * pitch;
                    at.scale(weight[pieces].x);
#pragma unroll 4
                    for (int span = 0; span < m; ++span) {
                        const int k = starts[span];
                        at.add_span(staged[k * wide + tid], weight[k].y);
                    }
                }
            } else if (tid < wide) {
                const float2 *weight = stat + q % cols * pitch;
                at.scale(weight[pieces].x);
                float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                float l = 0.0f;
#pragma unroll 1
                for (int k = 0; k < pieces; k += 8) {
                    const int n = min(8, pieces - k);
                    const uint32_t end = ends[k >> 5] >> (k & 31);
                    float4 t[8];
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        if (v < n) t[v] = __ldcg(reinterpret_cast<const float4 *>(mine + (size_t)slots[k + v] * 16));
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        if (v >= n) break;
                        const float2 of = weight[k + v];
                        sum = weigh(t[v], of.x, sum);
                        l = __fmaf_rn(of.y, of.x, l);
                        if (!((end >> v) & 1)) continue;
                        at.add_span(sum, l);
                        sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        l = 0.0f;
                    }
                }
            }
            if (STAGED) __syncthreads();   // (the next lines take these ones' place)
        }
        const int q = line * 8 + tid, e4 = q / cols, c = q - e4 * cols;
        if (tid >= min(group, l1 - line) * 8 || flags[1]) continue;
        const float inv = __fdiv_rn(1.0f, at.L), vs = a.v_scale ? a.v_scale[cut.head] : 1.0f;
#pragma unroll
        for (int v = 0; v < 4; ++v) at.y[v] = at.y[v] * inv * vs;
        const int i = c * p.inv_G >> 16;
        char *row = out_row(a, D, cut.x.r0 + cut.i0, cut.head, i, c - i * a.G);
        store_floats<ACT, 4>(row + e4 * 8, at.y);
        if (flags[2]) give_back<D, ACT, KV>(p, cut.stream, cut.head, cut.i0 + i, flags[2], row, e4 * 4, 4);
    }
    if (waited && tid == 0 && flags[1]) raise_error(a.err, GDN_DERR_PAGES);
    return waited;
}

// The end of a run: the items that it shares are counted in and joined.
template <int D, int ACT, int KV, int T, bool STAGED>
__device__ __forceinline__ void attn_finish(const AttnTcParams &p, AttnShared &sh, uint8_t *smem, int bytes) {
    // (all parts of the CTA are through)
    const int n_cut = sh.n_cut, i = threadIdx.x - kJoinSpans;
    if (i >= 0 && i < n_cut && sh.abort) atomicOr(p.counters + sh.cut[i].run, kGaveUp);
    if (i >= 0 && i < n_cut)   // after the CTA's pieces
        asm volatile("red.release.gpu.global.add.u64 [%0], %1;" ::"l"(p.counters + sh.cut[i].run),
                     "l"((unsigned long long)sh.cut[i].mine)
                     : "memory");
    int waited = 0;
#pragma unroll 1
    for (int k = 0; k < n_cut; ++k) {
        if (k) __syncthreads();
        if (attn_join<D, ACT, KV, T, STAGED>(p, sh, sh.cut[k], smem, bytes)) waited |= 1 << k;
    }
    // and out again, but not before all are in (an empty part has not waited); the last leaves 0 behind
    if (i >= 0 && i < n_cut) {
        unsigned long long *counter = p.counters + sh.cut[i].run;
        if (!((waited >> i) & 1)) count_full(counter, sh.cut[i].tiles, p.wait_limit, p.a.err);
        const unsigned long long sum = atomicAdd(counter, (unsigned long long)sh.cut[i].mine) + sh.cut[i].mine;
        if (count_of(sum) == 2 * sh.cut[i].tiles) atomicExch(counter, 0ull);
    }
}

}  // namespace gdn
