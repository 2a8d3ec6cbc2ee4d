// gdn_attn.cu -- launches of the attention over the paged cache.
#include <algorithm>
#include <atomic>
#include <chrono>
#include <cstdint>
#include <random>

#include "gdn_attn_tc.cuh"
#include "gdn_tensor_map.h"

namespace gdn {

// The device's SM count, looked up once per device.
int sm_count() {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> count[kMaxDevices];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    int n = count[dev].load(std::memory_order_relaxed);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        count[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Entropy where the system gives it (it throws where not, and the entries are C), else the clock and an address.
static unsigned long long random_start() noexcept {
    unsigned long long x;
    try {
        x = std::random_device{}();
    } catch (...) {
        x = (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count() ^ (uintptr_t)&x;
    }
    return x * 0x9E3779B97F4A7C15ull;
}

// A number that no earlier call of this process has, within 37 bits from a
// random start: what an old workspace holds is taken for this call's counts only by an accident of that size.
static unsigned long long call_token() {
    static std::atomic<unsigned long long> next{random_start()};
    return next.fetch_add(1, std::memory_order_relaxed) % ((1ull << (64 - kCountBits)) - 1) + 1;
}

// Polls after which a wait of later calls gives up (gdn_debug_attn_wait_limit).
static std::atomic<uint32_t> wait_limit{kAttnWaitLimit};
bool attn_wait_limit(uint32_t polls) {
    if (polls > kAttnWaitLimit) return false;
    wait_limit.store(polls, std::memory_order_relaxed);
    return true;
}

// Columns of a tile: the rows of a pass times G, 16 or a multiple of 32.
static int columns_for(int rows, int G) {
    const int c = std::min(kAttnMaxCols, rows * G);
    return c <= 16 ? 16 : (c + 31) / 32 * 32;
}

// The workspace: a counter per run, then slots.
struct AttnLayout {
    size_t base, stat_bytes, slot_bytes, bytes;
    int slot_cols;
    long long slots;
};
// `r` window rows a pass, of at most `max_rows`: a stream takes ceil(rows / r) passes.  A pass over t tokens has
// ceil(t / 512) spans, from 8192 tokens on 8 + ceil(t / 1024), so 1 + min(t / 512, 8 + t / 1024) at most: added up over
// the passes, whose tokens are at most those of the table's rows, and those of the pool as often as a stream has passes
// (pages that are in one row each; the kernels refuse lengths that need more).
static AttnLayout attn_layout(int r, int max_rows, const AttnParams &a, int D, int grid) {
    AttnLayout l;
    const long long streams = a.n_streams, each = (max_rows + r - 1) / r;
    const long long passes = std::min({(long long)a.n_rows, streams * each, streams + a.n_rows / r});
    const long long row = (long long)a.max_pages * a.page_size, pool = each * a.n_pages * a.page_size;
    const long long row_spans = row <= 8192 ? (row + 511) / 512 : 8 + (row + 1023) / 1024;
    const long long spans = std::min(passes * row_spans, passes + std::min(pool / 512, 8 * passes + pool / 1024));
    l.slots = spans * a.Hkv + (long long)grid * (kSpanMost - 1);
    l.base = ((size_t)grid * 8 + 255) / 256 * 256;
    l.slot_cols = r * a.G;
    l.stat_bytes = ((size_t)(l.slot_cols + 1) * 8 + 15) / 16 * 16;
    l.slot_bytes = l.stat_bytes + (size_t)l.slot_cols * D * 4;
    l.bytes = l.base + l.slot_bytes * (size_t)l.slots;
    return l;
}

constexpr int kSizingSms = 160;   // at least the SMs of a GB300: a size must not depend on a device being there

static int most_rows(const AttnParams &a) { return std::min(a.n_rows, (int)GDN_MAX_WINDOW); }

// Sized for windows in one pass (as many rows as fit 128 columns) where
// there are more rows than streams, and else for a row a pass, which any division of the rows fits.
size_t attn_workspace(const AttnParams &a, int D) {
    const int rows = a.n_rows > a.n_streams ? std::min(most_rows(a), kAttnMaxCols / a.G) : 1;
    return attn_layout(rows, most_rows(a), a, D, kSizingSms).bytes;
}

// The cache as (block of a row, 8 keys, blocks, groups of 8 keys of all heads, pages); one copy
// brings a page's (or 128 keys') share of a piece.
static bool kv_map(CUtensorMap *m, const AttnParams &p, int D, int kv, void *base) {
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const int bytes = kv == GDN_E4M3 ? 1 : 2;
    const cuuint64_t row = (cuuint64_t)D * bytes, block = std::min<cuuint64_t>(row, 128);
    const cuuint64_t groups = (cuuint64_t)p.Hkv * p.page_size / 8;
    const cuuint64_t dims[5] = {block / bytes, 8, row / block, groups, (cuuint64_t)p.n_pages};
    const cuuint64_t strides[4] = {row, block, row * 8, row * 8 * groups};
    const cuuint32_t box[5] = {(cuuint32_t)(block / bytes), 8, row > 128 ? 2u : 1u,
                               (cuuint32_t)std::min(p.page_size, kTileKeys) / 8, 1};
    const cuuint32_t step[5] = {1, 1, 1, 1, 1};
    const CUtensorMapDataType type = kv == GDN_E4M3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : kv == GDN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return fn(m, type, 5, base, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              block == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as (64 elements, query heads, rows, blocks of 64 elements); one copy brings a block of a key head's pass.
static bool q_map(CUtensorMap *m, const AttnParams &p, int D, int act, int rows_pass) {
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[4] = {64, (cuuint64_t)p.Hq, (cuuint64_t)p.n_rows, (cuuint64_t)D / 64};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)p.Hq * D * 2, 128};
    const cuuint32_t box[4] = {64, (cuuint32_t)p.G, (cuuint32_t)rows_pass, 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return fn(m, act == GDN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
              const_cast<char *>(p.q), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_attn(int D, int act, int kv, int max_rows, const AttnParams &a, cudaStream_t st) {
    AttnTcParams p = {};
    p.a = a;
    p.grid = std::min(sm_count(), kSizingSms);
    if (p.grid <= 0) return cudaErrorInvalidDevice;
    if (!kv_map(&p.map_k, a, D, kv, a.k) || !kv_map(&p.map_v, a, D, kv, a.v)) return cudaErrorInvalidValue;
    // as many rows a pass as 128 columns hold and the workspace was sized for; fewer take more passes over the cache
    int r = std::min(max_rows, kAttnMaxCols / a.G);
    AttnLayout l = attn_layout(r, max_rows, a, D, p.grid);
    while (l.bytes > a.ws_bytes && r > 1) l = attn_layout(--r, max_rows, a, D, p.grid);
    if (l.bytes > a.ws_bytes) return cudaErrorInvalidValue;
    p.rows_pass = r;
    if (kv != GDN_E4M3 && !q_map(&p.map_q, a, D, act, r)) return cudaErrorInvalidValue;
    p.nc = columns_for(r, a.G);
    // windows over an 8-bit cache always go to the window kernel: the step kernel adds up the parts of its operands
    // apart, so the few windows that would fit it would have other bits alone than among others
    if (kv == GDN_E4M3 && a.row_ptr) p.nc = std::max(p.nc, 2 * kStepCols);
    p.inv_G = (65536 + a.G - 1) / a.G;
    for (p.page_shift = 0; (1 << p.page_shift) < a.page_size; ++p.page_shift) {}
    p.slot_cols = l.slot_cols;
    p.stat_bytes = (uint32_t)l.stat_bytes;
    p.slot_bytes = (uint32_t)l.slot_bytes;
    // (a slot's place is counted in 16-byte units of 32 bits)
    p.n_slots = (int)std::min<size_t>((a.ws_bytes - l.base) / l.slot_bytes, UINT32_MAX / (l.slot_bytes / 16) - 1);
    p.counters = reinterpret_cast<unsigned long long *>(a.ws);
    p.token = call_token();
    p.wait_limit = wait_limit.load(std::memory_order_relaxed);
    p.slots = a.ws + l.base;
    switch (D) {
        case 64: return launch_attn_tc_d64(act, kv, p, st);
        case 128: return launch_attn_tc_d128(act, kv, p, st);
        default: return launch_attn_tc_d256(act, kv, p, st);
    }
}

}  // namespace gdn
