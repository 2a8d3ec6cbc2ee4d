// gdn_attn.cuh -- what the attention over the paged cache and the move of a
// tree's kept path take, and the check of one stream's part of a round.
#pragma once

#include "gdn_attn_common.cuh"

namespace gdn {

struct AttnParams {
    const char *q;
    char *out;                        // [R, Hq, D]
    char *k, *v;                      // [n_pages, Hkv, page_size, D]
    const float *k_scale, *v_scale;   // [Hkv] or nullptr
    const int *block_table, *kv_len, *n_held;
    const int *slot, *row_ptr, *parent, *keep_row;   // row_ptr nullptr: one row a stream
    int n_slots, max_pages, n_pages, page_size, n_streams, n_rows;
    int Hq, Hkv, G;
    float scale;
    char *ws;
    size_t ws_bytes;
    int *err;
};

// A stream's part of a round.
struct AttnStream {
    int sl, r0, n, len;
};

__device__ __forceinline__ int attn_stream(const AttnParams &p, int s, AttnStream &x) {
    x.sl = p.slot[s];
    x.r0 = s;
    x.n = 1;
    if (x.sl < 0 || x.sl >= p.n_slots) return GDN_DERR_SLOT;
    if (p.row_ptr) {
        x.r0 = p.row_ptr[s];
        const int r1 = p.row_ptr[s + 1];
        x.n = r1 - x.r0;
        if (x.r0 < 0 || r1 < x.r0 || r1 > p.n_rows || x.n > GDN_MAX_WINDOW) return GDN_DERR_ROWS;
    }
    x.len = p.kv_len[x.sl];
    // (entries of the table behind the slot's own pages may name pages that others hold by now)
    const int held = p.n_held[x.sl];
    if (x.len < 0 || held < 0 || held > p.max_pages || (long long)x.len + x.n > (long long)held * p.page_size)
        return GDN_DERR_PAGES;
    return 0;
}

// SMs of the current device (0: none).
int sm_count();
// Bytes of workspace (include/gdn.h: gdn_attn_workspace_size).
size_t attn_workspace(const AttnParams &sizes, int D);
bool attn_wait_limit(uint32_t polls);
cudaError_t launch_attn(int d_head, int act, int kv, int max_rows, const AttnParams &p, cudaStream_t st);

}  // namespace gdn
