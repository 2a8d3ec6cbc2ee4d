// gdn_attn_tc.cuh -- what the two attention kernels on the 5th-generation
// tensor cores share: tiles and spans, a CTA's run of them, the copies and the queries.
//
// Tiles and spans.  A tile is 128 keys at fixed tokens of its stream.  Each
// tile gets its own reference (a power of two), sum of weights and product
// O = P V from zero; tiles are folded in order into spans, A <- A e1 + O e2
// with powers of two, and spans are added in order.  A CTA takes an equal run of all tiles of the call
// (streams, key heads, tokens), so the load is even whatever the lengths
// are.  An item (a stream's pass of rows and a key head) that lies whole in
// a run is finished there.  Of one that runs share, each leaves pieces in the
// workspace: a whole span, the beginning of a span (its first tiles, folded:
// what follows folds onto it), or, where the run starts inside a span, each
// tile of the rest by itself.  The sharing CTAs add the pieces up with
// the same operations in the same order, each a part of the item.  So the bits of a row depend on its own
// stream alone, not on the batch or the grid.  Spans have 4 tiles for the
// first 64 of a stream and 8 from there on: short spans leave fewer single
// tiles, long ones fewer pieces in all (with 8 throughout 16 windows over up to 8192 tokens take 95 us, not 88;
// with 4 throughout 4 streams of some 100 k e4m3 tokens 203, not 177).
//
// Tiles in shared memory.  K and V come as they lie in the cache, in pieces of
// 128 keys x at most 256 bytes: groups of 8 keys, in each group the 128-byte
// blocks of a row (64 bytes where a row has no more), 8 rows each, swizzled.  A
// tensor map of five axes (block, 8 keys, blocks, groups, pages) makes one
// copy of each page, whatever the page size.  Both operands' descriptors
// reach that layout: K by rows (K-major, 8-row groups a group apart), V
// transposed (MN-major, blocks an atom apart, 8-key groups a group apart).
//
// Operands of few bits.  Weights are held in two 16-bit parts for the second
// product, as one would be off about as much as the output's own rounding
// (fp16 2^-11, bf16 2^-8): bf16 2^-16 relative, fp16, scaled by 2^15, 2^-20
// down to weights of 2^-19 and 2^-39 of the tile's largest at the least.  An 8-bit cache is multiplied as it is: the
// tensor cores' e4m3 products are exact and summed in 32 bits (measured:
// 2^-22 of the sum of magnitudes), so only q and the weights have to become sums of e4m3 parts of
// 4 bits each: a bf16 q is two parts (8 bits), an fp16 q and a weight three
// (2^-13 relative).  Where parts have sums of their own (steps) each is 2^5 times what it stands for relative to the
// one before, so that small numbers keep their bits: 2^-26 of the tile's largest weight at the least, 2^-21 of a
// query's largest element.  Where they share a sum (windows) the last part is e5m2, whose least number is 2^-16
// instead of 2^-9: 2^-22 of the power of two above the tile's largest weight, 2^-21 of a query's largest element.
// Sums are taken from the fp32 weights.
#pragma once

#include <cuda.h>

#include "gdn_attn.cuh"
#include "gdn_tc.cuh"

namespace gdn {

constexpr int kTileKeys = 128;
constexpr int kSpanMost = 8;            // tiles of a span
constexpr int kAttnMaxCols = 128;
constexpr int kTableStreams = 64;
constexpr uint32_t kAttnWaitLimit = 1u << 20;

// The runs: `total` tiles over the grid, the first `more` CTAs with one more.
struct AttnRuns {
    int each, more;
};

// An item that this run shares with others.
struct AttnCut {
    int g0, tiles, span0;   // its first tile of the call, its tiles, its first span
    int run;                // the run of its first tile
    int before, mine;       // its tiles before this run, and in it
    int head, i0, cols, stream;
    AttnStream x;
};

struct AttnTcParams {
    AttnParams a;
    CUtensorMap map_k, map_v, map_q;   // (map_q: 16-bit caches)
    int nc;          // columns (rows of a tile's products) that shared memory and TMEM have room for
    int slot_cols;   // and a slot
    int rows_pass;   // window rows in one pass: nc / G
    int page_shift;  // log2 of the page size
    int inv_G;       // ceil(2^16 / G): x / G = x * inv_G >> 16 for x < 256
    int n_stages;    // pieces in shared memory
    int grid;
    int n_slots;
    // workspace: a counter per run (of the shared item that starts in it), then the pieces' slots: (reference, sum of
    // weights) by column and the window rows whose values are not all finite, then the sums [D / 4][slot_cols][4]
    unsigned long long *counters;
    unsigned long long token;
    uint32_t wait_limit;   // polls after which a wait gives up (kAttnWaitLimit but in tests)
    char *slots;
    uint32_t slot_bytes, stat_bytes;
};

// The span of a tile, and a span's first tile.
__device__ __forceinline__ int span_of(int tile) { return tile < 64 ? tile / 4 : 8 + tile / 8; }
__device__ __forceinline__ int span_begin(int span) { return span < 16 ? span * 4 : (span - 8) * 8; }

// Tiles and spans of one item of a stream, an item being a pass of window
// rows and a key head (0 where it has no rows or is refused), and its items.
__device__ __forceinline__ int stream_tiles(const AttnStream &x) { return x.n ? (x.len + x.n - 1) / kTileKeys + 1 : 0; }
__device__ __forceinline__ int stream_spans(int tiles) { return tiles ? span_of(tiles - 1) + 1 : 0; }
__device__ __forceinline__ int stream_items(const AttnParams &a, int rows_pass, const AttnStream &x) {
    return (x.n + rows_pass - 1) / rows_pass * a.Hkv;
}

__device__ __forceinline__ int checked_stream(const AttnParams &a, int s, AttnStream &x) {
    int bits = attn_stream(a, s, x);
    unsigned long long packed;
    if (!bits && a.parent && !pack_parents(a.parent + x.r0, x.n, packed)) bits = GDN_DERR_PARENT;
    if (bits) x.n = 0;
    return bits;
}

__device__ __forceinline__ AttnRuns attn_runs(int total, int grid) {
    const int q = (unsigned)total / (unsigned)grid;
    return AttnRuns{q, total - q * grid};
}
__device__ __forceinline__ int run_start(AttnRuns r, int cta) { return cta * r.each + min(cta, r.more); }
__device__ __forceinline__ int run_of(AttnRuns r, int tile) {
    const int big = r.more * (r.each + 1);
    return tile < big ? (unsigned)tile / (unsigned)(r.each + 1) : r.more + (unsigned)(tile - big) / (unsigned)r.each;
}

// exp2 with a few ulp; -inf gives 0
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Tiles are kept relative to a whole power of two: the largest score (in
// halvings) rounded up.  Factors between two of them are powers of two, so
// scaling a sum is exact, and a fold rounds as the plain sum of the pieces does, whatever it is relative to.
__device__ __forceinline__ float reference_of(float m) { return ceilf(m); }
__device__ __forceinline__ float zero_if_none(float m) { return m == -INFINITY ? 0.0f : m; }
// 2^d for a whole d <= 0, 0 from 2^-127 on
__device__ __forceinline__ float whole_exp2(float d) { return __int_as_float((max(__float2int_rn(d), -127) + 127) << 23); }

// One step of a fold: the piece (m, l) joins the sum (M, L); what the sums are multiplied by.
struct Fold {
    float e1, e2;
};
__device__ __forceinline__ Fold fold_stats(float &M, float &L, float m, float l) {
    const float mn = fmaxf(M, m), ref = zero_if_none(mn);
    Fold f;
    f.e1 = whole_exp2(__fsub_rn(M, ref));
    f.e2 = whole_exp2(__fsub_rn(m, ref));
    L = __fmaf_rn(l, f.e2, __fmul_rn(L, f.e1));
    M = mn;
    return f;
}
__device__ __forceinline__ float fold_sum(float A, float O, Fold f) { return __fmaf_rn(O, f.e2, __fmul_rn(A, f.e1)); }

// Parts of q and of a weight as operands, and the power of two that weights are scaled by.
template <int ACT, int KV>
struct AttnParts {
    static constexpr int kQuery = KV != GDN_E4M3 ? 1 : ACT == GDN_BF16 ? 2 : 3;
    static constexpr int kWeight = KV == GDN_E4M3 ? 3 : 2;
    static constexpr float kNext = KV == GDN_E4M3 ? 32.0f : 1.0f;   // scale of a part against the one before, if their sums are apart
    static constexpr float kShift = KV == GDN_E4M3 ? 8.0f : ACT == GDN_BF16 ? 0.0f : 15.0f;
};

// Parts of a weight whose products are summed apart and added as they are read (16-bit ones of 256 elements in one sum:
// the window kernel's TMEM is full).  A window's rows have a step's bits, so the kernels go by the same rule.
template <int D, int ACT, int KV>
constexpr int kAside = KV == GDN_E4M3 || D <= 128 ? AttnParts<ACT, KV>::kWeight : 1;

// A weight of the second product is 2^(s c - ref).
template <int ACT, int KV>
__device__ __forceinline__ float ref_of(float m) {
    return __fsub_rn(zero_if_none(m), AttnParts<ACT, KV>::kShift);
}
__device__ __forceinline__ float weight_of(float s, float c, float ref) { return fast_exp2(__fmaf_rn(s, c, -ref)); }

// The first 16-bit parts of two weights; what is left becomes the second.  The first is rounded down and what is
// left is not 0 either (fp16: 2^-24 at least; bf16: 2^-22 of the weight more) unless the weight is, so that both parts
// of an infinite value's product are infinities of one sign.
template <int KV>
__device__ __forceinline__ uint32_t first_parts(float &x, float &y) {
    uint32_t two;
    if constexpr (KV == GDN_FP16) asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(two) : "f"(y), "f"(x));
    else two = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
    const float2 top = Elem<KV>::unpack2(two);
    if constexpr (KV == GDN_FP16) {
        x = fmaxf(__fsub_rn(x, top.x), fminf(x, 5.9604644775390625e-08f));
        y = fmaxf(__fsub_rn(y, top.y), fminf(y, 5.9604644775390625e-08f));
    } else {
        x = __fmaf_rn(x, 1.0000002384185791f, -top.x);
        y = __fmaf_rn(y, 1.0000002384185791f, -top.y);
    }
    return two;
}

// ---- PTX pieces

// Shared-memory matrix descriptor of swizzled blocks of BB bytes.  K-major:
// 8-row groups `group` bytes apart (lbo unused).  MN-major: a block of the
// long axis wide, the next block lbo bytes on, 8 steps of the other axis `group` bytes apart.
template <int BB>
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t saddr, uint32_t lbo, uint32_t group) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(group >> 4) << 32) |
           (1ull << 46) | ((BB == 128 ? 2ull : 4ull) << 61);
}
// Where the 16-byte piece c of row r lies in its block.
template <int BB>
__device__ __forceinline__ uint32_t swizzled_piece(int r, int c) {
    return (uint32_t)((r & 7) * BB + (BB == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) * 16);
}
constexpr uint32_t kDescE5m2 = 1u << 7;   // the first operand is e5m2
// Instruction descriptor: D in fp32, A and B of the operands' type, M = 128.
template <int ACT, int KV>
constexpr uint32_t kMmaDesc = (1u << 4) | (KV != GDN_E4M3 && ACT == GDN_BF16 ? (1u << 7) | (1u << 10) : 0u) | (8u << 24);
// One step of 32 bytes of the shared axis: 16 elements of 16 bits or 32 of 8.
template <int KV>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    if constexpr (KV == GDN_E4M3)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc));
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc));
}
// The same with the first operand in TMEM.
template <int KV>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    if constexpr (KV == GDN_E4M3)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc));
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc));
}
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ void mbar_arrive(uint64_t *mbar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(mbar)) : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[N]) {
    static_assert(N == 4 || N == 8 || N == 16, "columns");
    uint32_t r[N];
    if constexpr (N == 16) {
        tc::tmem_ld16_nowait(addr, r);
    } else if constexpr (N == 4) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
    } else {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(addr));
    }
    tc::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}
// Five-axis load: 64 elements and 8 keys from their start, blocks from x2, groups from x3, page x4.
__device__ __forceinline__ void tma_load_5d(void *smem_dst, const void *map, int x2, int x3, int x4, uint64_t *mbar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %2, %3, %4, %5}], [%6];" ::"r"(tc::smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(x2), "r"(x3), "r"(x4), "r"(tc::smem_u32(mbar))
        : "memory");
}
// Four-axis load: 64 elements from their start, heads from x1, rows from x2, block x3.
__device__ __forceinline__ void tma_load_4d(void *smem_dst, const void *map, int x1, int x2, int x3, uint64_t *mbar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4, %5}], [%6];" ::"r"(tc::smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(x1), "r"(x2), "r"(x3), "r"(tc::smem_u32(mbar))
        : "memory");
}
// A warpgroup gives registers back, or takes some of those.
template <int R>
__device__ __forceinline__ void registers_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void registers_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int ID, int THREADS>
__device__ __forceinline__ void named_barrier() {
    asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}

// Zeros in the place of the elements of `w` that are not finite; true if there were any.
template <int T>
__device__ __forceinline__ bool drop_not_finite(uint4 &w) {
    constexpr int kBits = T == GDN_E4M3 ? 8 : 16;
    constexpr uint32_t kSpecial = T == GDN_E4M3 ? 0x7fu : T == GDN_BF16 ? 0x7f80u : 0x7c00u;
    bool any = false;
    uint32_t *x = &w.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int b = 0; b < 32; b += kBits) {
            if ((x[i] & (kSpecial << b)) == (kSpecial << b)) {
                x[i] &= ~(((1u << kBits) - 1) << b);
                any = true;
            }
        }
    }
    return any;
}

// ---- a CTA's walk over its tiles

struct AttnWalk {
    int s;            // stream
    int head, i0;     // key head; the pass's first window row
    int tile;         // within the item (a pass and head)
    int tiles;        // of the item
    int span0;        // the item's first span
    int cols;         // the item's columns
    AttnStream x;
};

constexpr int kAttnStages = 16;
constexpr int kAttnTiles = 32;   // facts of tiles that are kept (a lane each at the start): more than the copies can be ahead of the sums

// What the other parts of a CTA have to know of a tile, written by its copies' warp.
struct AttnFacts {
    int tail, last;   // committed tokens, and tokens, from the tile's first key on
    int slot;         // of its piece
    int head;         // key head
    int stream, i0;   // and the pass's first window row
    int row;          // its packed row
    uint16_t cols;    // of its item
    uint16_t flags;   // kOpens ..
};
// A tile opens or ends an item in this run; begins or ends a piece; has a page out of range; its item lies whole in the run.
constexpr int kOpens = 1, kEnds = 2, kFirst = 4, kLast = 8, kRefused = 16, kWhole = 32;

struct AttnShared {
    uint64_t full[kAttnStages], empty[kAttnStages], sfull[2], pfull[2], ofull[2], ofree[2], qfull[2], qempty[2], done;
    AttnFacts facts[kAttnTiles];
    uint32_t vbad[8];          // by tile & 7: window rows whose values in the cache are not all finite
    uint32_t tmem, first_poll;   // (a wait counts its polls from there to kAttnWaitLimit)
    int abort;
    int first_stream, n_table, first_tile, span0;
    AttnRuns runs;
    AttnCut cut[2];
    int n_cut;
    long long sums[2][16];
    int4 table[kTableStreams];
};

// Wait for a phase; after one wait has given up every wait returns at once,
// and the kernel runs to its end on whatever is there (all trip counts are
// fixed beforehand), with the error raised and no result written.  What is
// there: a tile's facts may be those of the tile kAttnTiles before or zeros,
// and two warps may see different ones, so no barrier of several warps
// stands behind a condition on them.
__device__ __forceinline__ bool mbar_done(uint64_t *mbar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(tc::smem_u32(mbar)), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ void attn_wait_on(AttnShared &sh, uint64_t *mbar, uint32_t parity, int *err) {
#pragma unroll 1
    for (uint32_t i = sh.first_poll; i < kAttnWaitLimit; ++i) {
        if (*(volatile int *)&sh.abort || mbar_done(mbar, parity)) return;
    }
    *(volatile int *)&sh.abort = 1;
    raise_error(err, GDN_DERR_TIMEOUT);
}
__device__ __forceinline__ void attn_wait(AttnShared &sh, uint64_t *mbar, uint32_t parity, int *err) {
    if (!mbar_done(mbar, parity)) attn_wait_on(sh, mbar, parity, err);
}

// A place in the ring of pieces and the parity of its use.
struct AttnRing {
    int at;
    uint32_t parity;
    __device__ __forceinline__ void next(int n_stages) {
        if (++at == n_stages) {
            at = 0;
            parity ^= 1;
        }
    }
};

__device__ __forceinline__ void walk_stream(const AttnTcParams &p, const AttnShared &sh, AttnWalk &k) {
    const int at = k.s - sh.first_stream;
    if (at < sh.n_table) {
        const int4 t = sh.table[at];
        k.x = AttnStream{t.x, t.y, t.z, t.w};
    } else {
        checked_stream(p.a, k.s, k.x);
    }
    k.tiles = stream_tiles(k.x);
    k.head = k.i0 = 0;
    k.cols = min(p.rows_pass, k.x.n) * p.a.G;
}

__device__ __forceinline__ AttnWalk walk_begin(const AttnTcParams &p, const AttnShared &sh) {
    AttnWalk k;
    k.s = sh.first_stream;
    walk_stream(p, sh, k);
    const int item = (unsigned)sh.first_tile / (unsigned)k.tiles, pass = (unsigned)item / (unsigned)p.a.Hkv;
    k.tile = sh.first_tile - item * k.tiles;
    k.head = item - pass * p.a.Hkv;
    k.i0 = pass * p.rows_pass;
    k.cols = min(p.rows_pass, k.x.n - k.i0) * p.a.G;
    k.span0 = sh.span0 + item * stream_spans(k.tiles);
    return k;
}

// The next tile; true if it starts another item.  Only called while there is one.
__device__ __forceinline__ bool walk_next(const AttnTcParams &p, const AttnShared &sh, AttnWalk &k) {
    if (++k.tile < k.tiles) return false;
    k.tile = 0;
    k.span0 += stream_spans(k.tiles);
    if (++k.head < p.a.Hkv) return true;
    k.head = 0;
    k.i0 += p.rows_pass;
    k.cols = min(p.rows_pass, k.x.n - k.i0) * p.a.G;
    if (k.i0 < k.x.n) return true;
    do {
        ++k.s;
        walk_stream(p, sh, k);
    } while (!k.x.n && k.s + 1 < p.a.n_streams);
    return true;
}

// A tile's K or V.
template <int D, int KV>
struct AttnTile {
    static constexpr int kRow = D * elem_bytes<KV>;              // bytes of a key
    static constexpr int kBlock = kRow < 128 ? kRow : 128;       // bytes of a swizzled block's rows
    static constexpr int kAtom = 8 * kBlock;                     // 8 rows of a block
    static constexpr int kRowBlocks = kRow / kBlock;
    static constexpr int kPieces = kRow > 256 ? 2 : 1;
    static constexpr int kBlocks = kRowBlocks / kPieces;         // of a piece
    static constexpr int kGroup = kBlocks * kAtom;               // 8 keys of a piece
    static constexpr int kBytes = kTileKeys / 8 * kGroup;        // of a piece
    static constexpr int kStepKeys = 32 / elem_bytes<KV>;        // keys of a step of the second product
    static constexpr int kSteps = kTileKeys / kStepKeys;
    static constexpr int kHalves = D == 256 ? 2 : 1;             // 128 elements of the head each (64 for D = 64)
    static constexpr int kPiecesHalf = kPieces == 2 ? 1 : 0;     // pieces and blocks from one half to the next
    static constexpr int kBlocksHalf = kPieces == 2 ? 0 : 1;
};

// The pieces' order of use (keys run one tile ahead of values): K0 K1 V0 K2 V1 .. K(n-1) V(n-2) V(n-1).
__device__ __forceinline__ int v_block(int it, int n) { return it < n - 1 ? 2 * it + 2 : 2 * it + 1; }

// The slot of a span's first piece, `run` being that of its first tile.  The
// span's other pieces follow it: each is a tile at the start of a later run, of
// which a run has `most` at most.
__device__ __forceinline__ int cut_most(AttnRuns r) { return min(kSpanMost - 1, r.each + 1); }
__device__ __forceinline__ int slot_of(int span, int run, int most) { return span + run * most; }
__device__ __forceinline__ float2 *slot_stat(const AttnTcParams &p, int slot) {
    return reinterpret_cast<float2 *>(p.slots + (size_t)slot * p.slot_bytes);
}
__device__ __forceinline__ float *slot_sums(const AttnTcParams &p, int slot) {
    return reinterpret_cast<float *>(p.slots + (size_t)slot * p.slot_bytes + p.stat_bytes);
}

// Whether a tile begins or ends the piece it belongs to, and the piece's slot.
struct AttnPiece {
    bool first, last;
    int slot;
};

// Tile `g` of the call, tile `tile` of an item of `tiles` whose first span is `span0`, in a run [lo, hi).
__device__ __forceinline__ AttnPiece piece_of(int g, int tile, int tiles, int span0, int lo, int hi, int cta,
                                              AttnRuns runs) {
    const int span = span_of(tile), in_span = tile - span_begin(span), g0 = g - in_span, most = cut_most(runs);
    const int end = g0 + min(tiles, span_begin(span + 1)) - span_begin(span);
    AttnPiece q;
    if (g0 < lo) {
        const int run = run_of(runs, g0);
        q.first = q.last = true;
        q.slot = slot_of(span0 + span, run, most) + 1 + g - run_start(runs, run + 1);
    } else {
        q.first = in_span == 0;
        q.last = g + 1 == min(end, hi);
        q.slot = slot_of(span0 + span, cta, most);
    }
    return q;
}

// The streams' tiles counted, this CTA's run [lo, hi) of them found, barriers
// and TMEM made ready.  False where there is nothing to do (all threads).
// T threads; the copies' warp is the first of the last four.
template <int T>
__device__ __forceinline__ bool attn_prologue(const AttnTcParams &p, AttnShared &sh, uint32_t tmem_cols, int sum_warps,
                                              bool clean_warp, int &lo, int &hi) {
    const AttnParams &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
    constexpr int kCopies = T / 32 - 4, kProducts = kCopies + 1;
    if (warp == kCopies) {
        if (lane < kAttnStages) {
            tc::mbar_init(&sh.full[lane], 1);
            tc::mbar_init(&sh.empty[lane], 1);
        }
        if (lane < 2) {
            tc::mbar_init(&sh.sfull[lane], 1);
            tc::mbar_init(&sh.pfull[lane], clean_warp ? 5 : 4);
            tc::mbar_init(&sh.ofull[lane], 1);
            tc::mbar_init(&sh.ofree[lane], sum_warps);
            tc::mbar_init(&sh.qfull[lane], clean_warp ? 1 : 2);
            tc::mbar_init(&sh.qempty[lane], 1);
        }
        if (lane < 8) sh.vbad[lane] = 0;
        sh.facts[lane] = AttnFacts{};   // (for parts whose first wait gives up)
        if (lane == 0) {
            sh.abort = 0;
            sh.first_poll = kAttnWaitLimit - p.wait_limit;
            tc::mbar_init(&sh.done, 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kProducts) tc::tmem_alloc(&sh.tmem, tmem_cols);
    auto count = [&](int s, AttnStream &x, long long &tiles, long long &spans) {
        const int bits = checked_stream(a, s, x);
        const int each = stream_tiles(x), items = stream_items(a, p.rows_pass, x);
        tiles += (long long)each * items;
        spans += (long long)stream_spans(each) * items;
        return bits;
    };
    auto scan = [&](long long &ti, long long &si) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(kFull, ti, o), v = __shfl_up_sync(kFull, si, o);
            if (lane >= o) {
                ti += u;
                si += v;
            }
        }
        if (lane == 31) {
            sh.sums[0][warp] = ti;
            sh.sums[1][warp] = si;
        }
    };
    // all tiles; with no more streams than threads a thread's sums are its stream's
    AttnStream x = {};
    long long tv = 0, sv = 0;
#pragma unroll 1
    for (int s = tid; s < a.n_streams; s += T) {
        const int bits = count(s, x, tv, sv);
        if (bits && cta == 0) raise_error(a.err, bits);
    }
    long long ti = tv, si = sv;
    scan(ti, si);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    long long tall = 0, sall = 0;
    auto finish = [&]() {   // the warps before this one, and all
        tall = sall = 0;
#pragma unroll 1
        for (int v = 0; v < min(T / 32, (a.n_streams + 31) / 32); ++v) {   // (a stream a lane)
            if (v == warp) {
                ti += tall;
                si += sall;
            }
            tall += sh.sums[0][v];
            sall += sh.sums[1][v];
        }
    };
    finish();
    const bool fits = tall <= INT32_MAX && sall + (long long)p.grid * (kSpanMost - 1) <= p.n_slots;
    const int total = fits ? (int)tall : 0;
    const AttnRuns runs = attn_runs(total, p.grid);
    if (cta == 0 && tid == 0 && !fits) raise_error(a.err, GDN_DERR_SPACE);
    if (tid == 0) sh.runs = runs;
    lo = run_start(runs, cta);
    hi = run_start(runs, cta + 1);
    if (lo < hi) {
        // the stream of the run's first tile, and a table of it and those after it
        long long t0 = 0, s0 = 0;
#pragma unroll 1
        for (int b = 0; b < a.n_streams; b += T) {
            const int s = b + tid;
            if (a.n_streams > T) {
                x = AttnStream{};
                tv = sv = 0;
                if (s < a.n_streams) count(s, x, tv, sv);
                ti = tv;
                si = sv;
                __syncthreads();
                scan(ti, si);
                __syncthreads();
                finish();
                ti += t0;
                si += s0;
            }
            if (t0 + tall > lo) {   // (the first block of streams that does)
                if (tv && ti - tv <= lo && lo < ti) {
                    sh.first_stream = s;
                    sh.first_tile = lo - (int)(ti - tv);
                    sh.span0 = (int)(si - sv);
                    sh.n_table = min(kTableStreams, min(a.n_streams, b + T) - s);
                }
                __syncthreads();
                const int at = s - sh.first_stream;
                if (s < a.n_streams && at >= 0 && at < kTableStreams) sh.table[at] = make_int4(x.sl, x.r0, x.n, x.len);
            }
            t0 += tall;
            s0 += sall;
            if (t0 > lo) break;
        }
    }
    __syncthreads();
    if (lo == hi) {
        if (warp == kProducts) tc::tmem_dealloc(sh.tmem, tmem_cols);
        return false;
    }
    return true;
}

// A shared item's counter: its tiles, counted in and out (26 bits), whether a CTA gave up on it, and the token.
constexpr int kCountBits = 27;
constexpr unsigned long long kGaveUp = 1ull << (kCountBits - 1);
__device__ __forceinline__ int count_of(unsigned long long v) { return (int)(v & (kGaveUp - 1)); }

// An item's counter carries the token from here on; one that does not counts as 0.
__device__ __forceinline__ void count_from(unsigned long long *counter, unsigned long long token) {
    unsigned long long old = __ldcg(counter), seen;
    while (old >> kCountBits != token) {
        seen = old;
        old = atomicCAS(counter, seen, token << kCountBits);
        if (old == seen) break;
    }
}

// The copies' warp: pages to pieces, K one tile ahead of V.
template <class T>
__device__ __forceinline__ void attn_copies(const AttnTcParams &p, AttnShared &sh, uint8_t *stages, int lo, int hi) {
    const AttnRuns runs = sh.runs;
    const AttnParams &a = p.a;
    const int lane = threadIdx.x & 31;
    const int shift = p.page_shift, ps = 1 << shift, pages_tile = ps >= kTileKeys ? 1 : kTileKeys >> shift;
    const int box_keys = min(ps, kTileKeys), box_shift = min(shift, 7);
    const int n = hi - lo;
    AttnWalk k = walk_begin(p, sh);
    bool opens = true;
    // the items that the run's ends cut
    auto cut_of = [&](int it, int mine) {
        if (lane != 0) return;
        const int g0 = lo + it - k.tile, run = g0 >= lo ? (int)blockIdx.x : run_of(runs, g0);
        sh.cut[sh.n_cut++] = AttnCut{g0, k.tiles, k.span0, run, max(0, lo - g0), mine, k.head, k.i0, k.cols, k.s, k.x};
    };
    if (lane == 0) sh.n_cut = 0;
    if (k.tile > 0 || k.tiles > n) cut_of(0, min(k.tiles - k.tile, n));
    AttnRing ring = {0, 1};   // (a fresh barrier counts as the phase before done)
    int issued = 0;   // (none is issued after a wait has given up)
    struct Tile {
        int page, pages, group;   // this lane's page (a lane is a page), pages of the tile, first group of 8 keys in them
        AttnFacts facts;
    };
    // a page out of range is read as page 0, and the tile's results are refused
    auto tile_of = [&](int it) {
        const long long tok = (long long)k.tile * kTileKeys + lane * ps;
        Tile t;
        t.page = lane < pages_tile && tok < k.x.len + k.x.n ? a.block_table[(size_t)k.x.sl * a.max_pages + ((int)tok >> shift)] : 0;
        t.pages = (min(kTileKeys, k.x.len + k.x.n - k.tile * kTileKeys) + box_keys - 1) >> box_shift;
        t.group = ((k.head << shift) + (k.tile * kTileKeys & (ps - 1))) >> 3;
        const AttnPiece piece = piece_of(lo + it, k.tile, k.tiles, k.span0, lo, hi, blockIdx.x, runs);
        t.facts.tail = k.x.len - k.tile * kTileKeys;
        t.facts.last = t.facts.tail + k.x.n;
        t.facts.slot = piece.slot;
        t.facts.head = k.head;
        t.facts.stream = k.s;
        t.facts.i0 = k.i0;
        t.facts.row = k.x.r0 + k.i0;
        t.facts.cols = (uint16_t)k.cols;
        const bool whole = k.tile <= it && k.tiles - k.tile <= n - it;
        t.facts.flags = (uint16_t)((opens ? kOpens : 0) | (piece.first ? kFirst : 0) | (piece.last ? kLast : 0) |
                                   (k.tile + 1 == k.tiles ? kEnds : 0) | (whole ? kWhole : 0));
        if (it == n - 1 && k.tile + 1 < k.tiles && k.tile < it) cut_of(it, k.tile + 1);
        return t;
    };
    auto check = [&](Tile &t, int it) {
        bool bad = t.page < 0 || t.page >= a.n_pages;
        if (bad) t.page = 0;
        if (__any_sync(kFull, bad)) t.facts.flags |= kRefused;
        if (lane == 0) sh.facts[it % kAttnTiles] = t.facts;   // (the arrival below makes it known)
    };
    auto push = [&](const CUtensorMap *map, const Tile &t) {
#pragma unroll
        for (int half = 0; half < T::kPieces; ++half, ring.next(p.n_stages)) {
            const int at = ring.at;
            attn_wait(sh, &sh.empty[at], ring.parity, a.err);
            __syncwarp();
            if (__any_sync(kFull, *(volatile int *)&sh.abort)) continue;
            if (lane == 0) tc::mbar_expect_tx(&sh.full[at], (uint32_t)((t.pages << box_shift) / 8 * T::kGroup));
            __syncwarp();
            if (lane < t.pages)
                tma_load_5d(stages + at * T::kBytes + (lane << box_shift) / 8 * T::kGroup, map, half * T::kBlocks, t.group,
                            t.page, &sh.full[at]);
            ++issued;
        }
    };
    // keys of tile it + 1, then values of tile it; a tile's pages are looked up a tile before they are copied
    Tile t = {}, ahead = tile_of(0);
#pragma unroll 1
    for (int it = -1; it < n; ++it) {
        const Tile v = t;
        if (it + 1 < n) {
            t = ahead;
            check(t, it + 1);
            if (it + 2 < n) {
                opens = walk_next(p, sh, k);
                ahead = tile_of(it + 2);
            }
        }
#pragma unroll 1
        for (int what = it + 1 < n ? 0 : 1; what < (it < 0 ? 1 : 2); ++what) push(what ? &p.map_v : &p.map_k, what ? v : t);
    }
    __syncwarp();
    if (lane < sh.n_cut) count_from(p.counters + sh.cut[lane].run, p.token);
    // copies that nobody has waited for (after a wait gave up) land before the CTA goes on
    for (int u = max(0, issued - p.n_stages); u < issued; ++u)
        tc::mbar_wait(&sh.full[u % p.n_stages], (u / p.n_stages) & 1, kAttnWaitLimit);
}

// The item's query rows as the operand of an 8-bit cache, by THREADS threads:
// blocks of a row's 128 bytes, in each block the rows, swizzled (as the copies of 16-bit queries lie).
// A row is scaled by a power of two (its largest element to [128, 256)) and taken in e4m3 parts,
// `part` bytes apart in blocks of `rows` rows; unscale[row] undoes the scale.  Rows from `cols` to `pad` are zeros.
// APART: each part has sums of its own, else the last is e5m2.
template <int D, int ACT, bool APART, int THREADS>
__device__ __forceinline__ void load_queries(const AttnTcParams &p, const AttnWalk &w, int cols, int pad, uint8_t *sq,
                                             int rows, uint32_t part, float *unscale, int tid) {
    using T = AttnTile<D, GDN_E4M3>;
    using Parts = AttnParts<ACT, GDN_E4M3>;
    const AttnParams &a = p.a;
    const char *q = a.q + (((size_t)w.x.r0 + w.i0) * a.Hq + w.head * a.G) * D * 2;
    // 8 lanes a row, a lane D / 8 consecutive elements
    constexpr int kPer = D / 8;
    const int sub = tid & 7;
#pragma unroll 1
    for (int c = tid >> 3; c < pad; c += THREADS / 8) {
        float x[kPer];
        float most = 0.0f;
        if (c < cols) {
            const int i = c * p.inv_G >> 16;
            const char *src = q + (((size_t)i * (a.Hq - a.G) + c) * D + sub * kPer) * 2;
#pragma unroll
            for (int e = 0; e < kPer; e += 8) load_floats<ACT, 8>(src + e * 2, *reinterpret_cast<float(*)[8]>(x + e));
        } else {
#pragma unroll
            for (int e = 0; e < kPer; ++e) x[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) most = fmaxf(most, fabsf(x[e]));
#pragma unroll
        for (int o = 4; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, o, 8));
        // (an infinity makes its row's scores NaN, as the sums of infinities that they are)
        const bool fine = isfinite(most);
        const int ex = most > 0.0f && fine ? 7 - ilogbf(most) : 0;
        if (sub == 0) unscale[c] = fine ? ldexpf(1.0f, -ex) : __int_as_float(0x7fc00000);
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[e] = ldexpf(x[e], ex);
#pragma unroll
        for (int t = 0; t < Parts::kQuery; ++t) {
#pragma unroll
            for (int e = 0; e < kPer; e += 8) {
                uint16_t b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (!APART && t + 1 == Parts::kQuery) {
                        b[j] = pack2_e5m2(x[e + 2 * j], x[e + 2 * j + 1]);
                        continue;
                    }
                    b[j] = Elem<GDN_E4M3>::pack2(x[e + 2 * j], x[e + 2 * j + 1]);
                    const float2 top = Elem<GDN_E4M3>::unpack2(b[j]);
                    const float next = APART ? Parts::kNext : 1.0f;
                    x[e + 2 * j] = (x[e + 2 * j] - top.x) * next;
                    x[e + 2 * j + 1] = (x[e + 2 * j + 1] - top.y) * next;
                }
                const int at = sub * kPer + e, piece = at / 16;
                *reinterpret_cast<uint2 *>(sq + t * part + (piece / (T::kBlock / 16) * rows + (c & ~7)) * T::kBlock +
                                           swizzled_piece<T::kBlock>(c, piece % (T::kBlock / 16)) + at % 16) =
                    *reinterpret_cast<uint2 *>(b);
            }
        }
    }
}
// What window row i sees of its window, as bits.
__device__ __forceinline__ uint32_t row_sees(const AttnParams &a, const AttnStream &x, int i) {
    if (!a.parent) return (2u << i) - 1;
    unsigned long long packed;
    pack_parents(a.parent + x.r0, x.n, packed);
    return path_bits(packed, i);
}

// What a row's softmax has to know: what it sees of its window, and the
// scale of its scores (8-bit caches).  Kept for four items: an item's are
// written when the item two (or, with one buffer of queries, one) before it
// has had its last scores, and the weights are at most two tiles behind those.
template <int ROWS>
struct AttnRows {
    uint32_t sees[4][ROWS];
    float unscale[4][ROWS];
};

// The queries' WARPS: the rows of each item of the run, BUFFERS items
// ahead of the scores (two for steps, whose parts have sums of their own, one for windows).  Those of 16 bits are copied as they are (a copy a block; rows behind the
// pass come along, are multiplied and seen by nothing).
template <int D, int ACT, int KV, int BUFFERS, int WARPS, int ROWS>
__device__ __forceinline__ void attn_queries_ahead(const AttnTcParams &p, AttnShared &sh, AttnRows<ROWS> &rows, uint8_t *sq,
                                                   uint32_t buffer, int pad, int block_rows, uint32_t part, int n, int tid) {
    constexpr int kBlocks = D * 2 / 128;
    const int lane = tid & 31;
    AttnWalk k = walk_begin(p, sh);
    int item = 0;
#pragma unroll 1
    for (; n > 0; ++item) {
        const int b = item % BUFFERS;
        if (item >= BUFFERS) attn_wait(sh, &sh.qempty[b], (uint32_t)(item / BUFFERS - 1) & 1, p.a.err);
        const uint32_t seen = k.i0 + lane < k.x.n ? row_sees(p.a, k.x, k.i0 + lane) : 0u;
#pragma unroll 1
        for (int c0 = tid - lane; c0 < pad; c0 += 32 * WARPS) {
            const int c = c0 + lane;
            const uint32_t mine = __shfl_sync(kFull, seen, min(31, c * p.inv_G >> 16));
            if (c < pad) {
                rows.sees[item & 3][c] = c < k.cols ? mine : 0u;
                if constexpr (KV != GDN_E4M3) rows.unscale[item & 3][c] = 1.0f;
            }
        }
        if constexpr (KV == GDN_E4M3) {
            load_queries<D, ACT, BUFFERS == 2, 32 * WARPS>(p, k, k.cols, pad, sq + b * buffer, block_rows, part, rows.unscale[item & 3], tid);
            tc::fence_async_smem();
        }
        __syncwarp();
        if (KV == GDN_E4M3 || tid >= 32) {
            if (lane == 0) mbar_arrive(&sh.qfull[b]);
        } else {
            if (__any_sync(kFull, *(volatile int *)&sh.abort)) break;
            if (lane == 0) tc::mbar_expect_tx(&sh.qfull[b], (uint32_t)(p.rows_pass * p.a.G * D * 2));
            __syncwarp();
            if (lane < kBlocks)
                tma_load_4d(sq + b * buffer + lane * block_rows * 128, &p.map_q, k.head * p.a.G, k.x.r0 + k.i0, lane,
                            &sh.qfull[b]);
        }
        n -= k.tiles - k.tile;
        if (n > 0) {
            k.tile = k.tiles - 1;
            walk_next(p, sh, k);
        }
    }
    // copies that nobody has waited for (after a wait gave up) land before the CTA goes on
    if (KV != GDN_E4M3 && tid < 32) {
        for (int u = max(0, item - BUFFERS); u < item; ++u)
            tc::mbar_wait(&sh.qfull[u % BUFFERS], (u / BUFFERS) & 1, kAttnWaitLimit);
    }
}

// Weights of 0 do not keep a value that is not finite out of a product.
// Values behind the stream's last token (key >= last) become zeros, whatever
// is there, as far as the products go (value_steps()); so do elements of the window's own (key >= tail) that are not
// finite, which are given back to the rows that see them.
// (THREADS threads; vbad gets those rows' bits.)
// The values have landed when their places' barriers say so, but a barrier can only be asked for the phase after its
// last: with four or five places for pieces and two a tile, the use before may be the values of the tile before, not
// there yet.  So the product of the tile before is waited for first.
template <class T>
__device__ __forceinline__ int value_steps(int last) { return min(T::kSteps, (last + T::kStepKeys - 1) / T::kStepKeys); }

template <int D, int KV, int THREADS>
__device__ __forceinline__ void clean_values(const AttnTcParams &p, AttnShared &sh, uint8_t *stages, int it, int n,
                                             int tail, int last, uint32_t *vbad, int tid) {
    using T = AttnTile<D, KV>;
    const int first_stage = v_block(it, n) * T::kPieces;
    if (it) attn_wait(sh, &sh.ofull[(it - 1) & 1], (uint32_t)((it - 1) >> 1) & 1, p.a.err);
    constexpr int kRow = T::kBlocks * T::kBlock / 16;   // 16-byte pieces of a key's row
    const int end = value_steps<T>(last) * T::kStepKeys;
    const uint32_t round = (uint32_t)first_stage / (uint32_t)p.n_stages;
    AttnRing ring = {first_stage - (int)round * p.n_stages, round & 1};
#pragma unroll 1
    for (int half = 0; half < T::kPieces; ++half, ring.next(p.n_stages)) {
        const int at = ring.at;
        attn_wait(sh, &sh.full[at], ring.parity, p.a.err);
#pragma unroll 1
        for (int u = max(tail, 0) * kRow + tid; u < end * kRow; u += THREADS) {
            const int key = u / kRow, c = u % kRow;
            uint4 *q = reinterpret_cast<uint4 *>(stages + at * T::kBytes + (key >> 3) * T::kGroup +
                                                 c / (T::kBlock / 16) * T::kAtom + (key & 7) * T::kBlock +
                                                 c % (T::kBlock / 16) * 16);
            if (key >= last) {
                *q = make_uint4(0, 0, 0, 0);
            } else if (uint4 w = *q; drop_not_finite<KV>(w)) {
                *q = w;
                atomicOr(vbad, 1u << (key - tail));
            }
        }
    }
}

// 16-bit rows of results: the item's columns are (window row, query head).
__device__ __forceinline__ char *out_row(const AttnParams &a, int D, int row, int head, int i, int g) {
    return a.out + ((size_t)(row + i) * a.Hq + head * a.G + g) * D * 2;
}

// What clean_values() kept out of the products reaches the rows that see it:
// elements e .. e + n of window row i, whose results without it `row` holds (written by this thread).
template <int D, int ACT, int KV>
__device__ __forceinline__ void give_back(const AttnTcParams &p, int stream, int head, int i, uint32_t vbad, char *row, int e,
                                          int n) {
    const AttnParams &a = p.a;
    AttnStream x;
    if (attn_stream(a, stream, x)) return;
    const float vs = a.v_scale ? a.v_scale[head] : 1.0f;
#pragma unroll 1
    for (uint32_t left = row_sees(a, x, i) & vbad; left; left &= left - 1) {
        const int t = x.len + __ffs(left) - 1;
        const int page = a.block_table[(size_t)x.sl * a.max_pages + (t >> p.page_shift)];
        if (page < 0 || page >= a.n_pages) continue;
        const size_t at = (((size_t)page * a.Hkv + head) * a.page_size + (t & (a.page_size - 1))) * D;
#pragma unroll 1
        for (int k = e; k < e + n; ++k) {
            float v;
            if constexpr (KV == GDN_E4M3) v = Elem<KV>::unpack2(reinterpret_cast<const uint8_t *>(a.v)[at + k]).x;
            else v = (float)reinterpret_cast<const typename Elem<KV>::type *>(a.v)[at + k];
            if (isfinite(v)) continue;
            typename Elem<ACT>::type *to = reinterpret_cast<typename Elem<ACT>::type *>(row) + k;
            const float y = (float)*to + v * vs;
            if constexpr (ACT == GDN_BF16) *to = __float2bfloat16_rn(y);
            else *to = __float2half_rn(y);
        }
    }
}

// Launches, one file per head size.
cudaError_t launch_attn_tc_d64(int act, int kv, const AttnTcParams &p, cudaStream_t st);
cudaError_t launch_attn_tc_d128(int act, int kv, const AttnTcParams &p, cudaStream_t st);
cudaError_t launch_attn_tc_d256(int act, int kv, const AttnTcParams &p, cudaStream_t st);

// More columns than this go to the window kernel, whose products have 128 rows whatever is in them.  64 uneven streams
// on 8 key heads of 128, step kernel / window kernel: 4 columns 67 / 116 us, 8 84 / 117, 16 115 / 119;
// 64 windows of two rows with 8 query heads each 125 / 125, with 9 (18 columns) - / 128.
constexpr int kStepCols = 16;

// Shared memory of a block beside the static part of either kernel.
constexpr size_t kStepSmem = 227 * 1024 - 8 * 1024, kWindowSmem = 227 * 1024 - 16 * 1024;

// Bytes of the operands beside the pieces: the step kernel has two items'
// queries and two tiles' weights, the window kernel one item's queries (and reads 128 rows from there).
template <int D, int ACT, int KV>
__host__ __device__ constexpr size_t attn_queries(int nc) {
    return (size_t)nc * D * elem_bytes<KV> * AttnParts<ACT, KV>::kQuery;
}
template <int ACT, int KV>
constexpr size_t step_weights = (size_t)AttnParts<ACT, KV>::kWeight * elem_bytes<KV> * kStepCols * kTileKeys;
template <int D, int ACT, int KV>
__host__ __device__ constexpr size_t attn_smem_fixed(int nc) {
    return 1024 + (nc <= kStepCols ? 2 * (attn_queries<D, ACT, KV>(kStepCols) + step_weights<ACT, KV>)
                                   : attn_queries<D, ACT, KV>(nc));
}

}  // namespace gdn
