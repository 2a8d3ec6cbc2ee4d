// gdn_pages.cuh -- the bookkeeping of the paged keys and values, on the GPU:
// pages for a round's rows off a free stack, each row's position and place
// in the cache, kept rows counted as committed, pages given back.  No length
// passes through the host, so a round's launches can stand in a graph.
#pragma once

#include <climits>

#include "gdn_paths.cuh"

namespace gdn {

struct PagesParams {
    int *block_table;   // [n_slots, max_pages]
    int *kv_len;        // [n_slots]
    int *n_held;        // [n_slots]
    int *free_pages;    // [n_pages], a stack
    int *n_free;        // [1]
    int n_slots, max_pages, n_pages, page_size;
    const int *slot;    // [S]
    const int *row_ptr; // [S + 1]
    const int *parent;  // [R] or nullptr
    const int *keep_row;
    int n_streams, n_rows;
    int *row_pos, *row_slot;   // [R]
    int *err;
};

constexpr int kPagesThreads = 1024;

// Rows [r0, r0 + n) of stream s behind `len` tokens of slot `sl`; the error
// bits where any of it is out of range (0: fine).
struct StreamRows {
    int sl, r0, n, len, held;
};

__device__ __forceinline__ int stream_rows(const PagesParams &p, int s, StreamRows &x) {
    x.sl = p.slot[s];
    x.r0 = p.row_ptr[s];
    const int r1 = p.row_ptr[s + 1];
    if (x.sl < 0 || x.sl >= p.n_slots) return GDN_DERR_SLOT;
    if (x.r0 < 0 || r1 < x.r0 || r1 > p.n_rows) return GDN_DERR_ROWS;
    x.n = r1 - x.r0;
    if (p.parent && x.n > GDN_MAX_WINDOW) return GDN_DERR_ROWS;
    x.len = p.kv_len[x.sl];
    x.held = p.n_held[x.sl];
    if (x.len < 0 || (long long)x.len + x.n > (long long)p.max_pages * p.page_size) return GDN_DERR_PAGES;
    return 0;
}

// Pages 0 .. all - 1 of the CTA's `streams` streams, whose running sums `ends` has: each is copied from *src(its number, its
// stream's thread, its number there) to *dst(the same).  Warps take the streams in turn,
// four pages a lane on the way.  (Plan, place and release of 256 prompts with 38 pages each: 20.4 us in a graph; 26.8
// with a thread a page of all streams, which has to search for its stream; 46 with a lane a stream.)
template <class Src, class Dst>
__device__ __forceinline__ void copy_pages(int streams, int all, const int *ends, Src src, Dst dst) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int l = threadIdx.x >> 5; l < streams; l += blockDim.x >> 5) {
        const int first = l ? ends[l - 1] : 0, end = min(all, ends[l]);
#pragma unroll 1
        for (int at = first + lane; at < end; at += 128) {
            int page[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (at + u * 32 < end) page[u] = *src(at + u * 32, l, at + u * 32 - first);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (at + u * 32 < end) *dst(at + u * 32, l, at + u * 32 - first) = page[u];
        }
    }
}

// Inclusive sum over the CTA's threads; *total gets the sum of all.
__device__ __forceinline__ long long cta_scan(long long v, long long *warp_sums, long long *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long u = __shfl_up_sync(kFull, v, off);
        if (lane >= off) v += u;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        long long w = lane < warps ? warp_sums[lane] : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long u = __shfl_up_sync(kFull, w, off);
            if (lane >= off) w += u;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    const long long before = warp ? warp_sums[warp - 1] : 0;
    *total = warp_sums[warps - 1];
    __syncthreads();   // warp_sums may be written again
    return before + v;
}

// Position and place of packed row r: its stream is the last one that starts
// at or before it.
__device__ __forceinline__ void place_row(const PagesParams &p, int r) {
    int lo = 0, hi = p.n_streams;   // row_ptr[lo] <= r < row_ptr[hi], if r is anyone's
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.row_ptr[mid] <= r) lo = mid;
        else hi = mid;
    }
    if (p.row_ptr[lo] > r || r >= p.row_ptr[lo + 1]) return;   // no stream's row
    StreamRows x;
    int pos = -1, place = -1;
    if (stream_rows(p, lo, x) == 0) {
        const int i = r - x.r0;
        const int held = x.held;
        bool ok = held >= 0 && held <= p.max_pages && (long long)held * p.page_size >= (long long)x.len + x.n;
        int depth = i;
        if (p.parent) {
            unsigned long long packed;
            if (!pack_parents(p.parent + x.r0, x.n, packed)) {
                ok = false;
                raise_error(p.err, GDN_DERR_PARENT);
            } else {
                depth = __popc(path_bits(packed, i)) - 1;
            }
        }
        if (ok) {
            const int at = x.len + i, shift = __ffs(p.page_size) - 1;
            const int page = p.block_table[(size_t)x.sl * p.max_pages + (at >> shift)];
            if (page < 0 || page >= p.n_pages) {
                raise_error(p.err, GDN_DERR_PAGES);
            } else {
                pos = x.len + depth;
                place = page * p.page_size + (at & (p.page_size - 1));
            }
        }
    }
    p.row_pos[r] = pos;
    p.row_slot[r] = place;
}

// Pages for the streams' rows, one CTA: a running sum of what the streams
// need gives each its piece of the stack.  With PLACE the CTA also places the
// rows, else a second kernel does.
template <bool PLACE>
__global__ void __launch_bounds__(kPagesThreads) gdn_pages_plan_kernel(const PagesParams p) {
    __shared__ long long warp_sums[32];
    __shared__ int taken, ends[kPagesThreads];
    __shared__ int *entry[kPagesThreads];   // a stream's first new table entry
    const int tid = threadIdx.x;
    int n_free = *p.n_free;
    if (n_free < 0 || n_free > p.n_pages) {
        if (tid == 0) raise_error(p.err, GDN_DERR_PAGES);
        n_free = 0;
    }
    if (tid == 0) taken = 0;
    __syncthreads();
    long long before = 0;
    for (int base = 0; base < p.n_streams; base += blockDim.x) {
        const int s = base + tid;
        StreamRows x = {};
        int held = 0, bits = 0;
        long long need = 0;
        if (s < p.n_streams) {
            bits = stream_rows(p, s, x);
            if (!bits) {
                held = x.held;
                if (held < 0 || held > p.max_pages) bits = GDN_DERR_PAGES;
                else need = (((long long)x.len + x.n + p.page_size - 1) >> (__ffs(p.page_size) - 1)) - held;
            }
            if (bits || need < 0) need = 0;
        }
        long long total;
        const long long end = before + cta_scan(need, warp_sums, &total);
        const bool served = need > 0 && end <= n_free;
        if (need > 0 && !served) bits |= GDN_DERR_PAGES;
        if (bits) raise_error(p.err, bits);
        if (served) {
            p.n_held[x.sl] = held + (int)need;
            atomicMax(&taken, (int)end);
        }
        // pages come off the stack in the streams' order; those that are not served are behind the others
        ends[tid] = (int)min(end - before, (long long)INT_MAX);
        entry[tid] = p.block_table + (size_t)x.sl * p.max_pages + held;
        __syncthreads();
        const int *stack = p.free_pages + (n_free - 1 - min(before, (long long)n_free));
        copy_pages(min((int)blockDim.x, p.n_streams - base), (int)max(taken - before, 0ll), ends, [&](int at, int, int) { return stack - at; },
                   [&](int, int l, int j) { return entry[l] + j; });
        __syncthreads();
        before += total;
    }
    __syncthreads();
    if (tid == 0 && taken) *p.n_free = n_free - taken;
    if constexpr (PLACE) {
        for (int r = tid; r < p.n_rows; r += blockDim.x) place_row(p, r);
    }
}

// A thread a row (623,845 rows of 256 prompts: 9 us from cold caches, most of it the search and the chain slot,
// length, page).
__global__ void __launch_bounds__(256) gdn_pages_place_kernel(const PagesParams p) {
    const int r = blockIdx.x * 256 + threadIdx.x;
    if (r < p.n_rows) place_row(p, r);
}

__global__ void __launch_bounds__(256) gdn_pages_commit_kernel(const PagesParams p) {
    const int s = blockIdx.x * 256 + threadIdx.x;
    if (s >= p.n_streams) return;
    const int kr = p.keep_row[s];
    if (kr == -1) return;
    const int sl = p.slot[s], r0 = p.row_ptr[s], r1 = p.row_ptr[s + 1];
    if (sl < 0 || sl >= p.n_slots) {
        raise_error(p.err, GDN_DERR_SLOT);
        return;
    }
    if (r0 < 0 || r1 > p.n_rows || kr < r0 || kr >= r1) {
        raise_error(p.err, GDN_DERR_KEEP);
        return;
    }
    int more = kr - r0 + 1;
    if (p.parent) {
        unsigned long long packed;
        if (r1 - r0 > GDN_MAX_WINDOW) {
            raise_error(p.err, GDN_DERR_ROWS);
            return;
        }
        if (!pack_parents(p.parent + r0, r1 - r0, packed)) {
            raise_error(p.err, GDN_DERR_PARENT);
            return;
        }
        more = __popc(path_bits(packed, kr - r0));
    }
    const int len = p.kv_len[sl], held = p.n_held[sl];
    if (len < 0 || held < 0 || held > p.max_pages || (long long)len + more > (long long)held * p.page_size) {
        raise_error(p.err, GDN_DERR_PAGES);
        return;
    }
    p.kv_len[sl] = len + more;
}

__global__ void __launch_bounds__(kPagesThreads) gdn_pages_release_kernel(const PagesParams p) {
    __shared__ long long warp_sums[32];
    __shared__ int ends[kPagesThreads];
    __shared__ const int *entry[kPagesThreads];   // a stream's table entries
    const int tid = threadIdx.x;
    auto held_of = [&](int s, int &sl) {
        if (s >= p.n_streams) return 0;
        sl = p.slot[s];
        if (sl < 0 || sl >= p.n_slots) return -GDN_DERR_SLOT;
        const int h = p.n_held[sl];
        return h < 0 || h > p.max_pages ? -GDN_DERR_PAGES : h;
    };
    long long all = 0;
    for (int base = 0; base < p.n_streams; base += blockDim.x) {
        int sl;
        const int h = held_of(base + tid, sl);
        if (h < 0) raise_error(p.err, -h);
        long long total;
        cta_scan(h > 0 ? h : 0, warp_sums, &total);
        all += total;
    }
    const int n_free = *p.n_free;
    if (n_free < 0 || n_free + all > p.n_pages) {
        if (tid == 0) raise_error(p.err, GDN_DERR_PAGES);
        return;
    }
    const int top = n_free + (int)all - 1;
    long long before = 0;
    for (int base = 0; base < p.n_streams; base += blockDim.x) {
        int sl = 0;
        const int h = held_of(base + tid, sl);
        const int n = h > 0 ? h : 0;
        long long total;
        ends[tid] = (int)cta_scan(n, warp_sums, &total);
        entry[tid] = p.block_table + (size_t)sl * p.max_pages;
        __syncthreads();
        int *stack = p.free_pages + (top - (int)before);
        copy_pages(min((int)blockDim.x, p.n_streams - base), (int)total, ends, [&](int, int l, int j) { return entry[l] + j; }, [&](int at, int, int) { return stack - at; });
        __syncthreads();
        if (h >= 0 && base + tid < p.n_streams) {
            p.n_held[sl] = 0;
            p.kv_len[sl] = 0;
        }
        before += total;
    }
    if (tid == 0) *p.n_free = top + 1;
}

}  // namespace gdn
