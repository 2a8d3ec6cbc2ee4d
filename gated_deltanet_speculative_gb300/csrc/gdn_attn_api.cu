// gdn_attn_api.cu -- the C ABI of the attention layers (include/gdn.h):
// host-side validation and launches of the page bookkeeping, the attention's
// preparation, the attention itself and the move of a tree's kept path.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gdn_attn.cuh"
#include "gdn_attn_commit.cuh"
#include "gdn_attn_prep.cuh"
#include "gdn_context.h"
#include "gdn_pages.cuh"

namespace {

bool aligned(const void *ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

#define GDN_TRY(expr)                 \
    do {                              \
        const int rc_ = (expr);       \
        if (rc_ != GDN_OK) return rc_; \
    } while (0)

int check_attn_dims(const gdn_attn_dims *d) {
    if (!d) return GDN_ENULL;
    if (d->n_kv_heads <= 0 || d->n_q_heads <= 0 || d->n_q_heads > 65535) return GDN_EINVAL;
    if (d->n_q_heads % d->n_kv_heads != 0 || d->n_q_heads / d->n_kv_heads > 16) return GDN_EINVAL;
    if (d->d_head != 64 && d->d_head != 128 && d->d_head != 256) return GDN_EINVAL;
    if (d->d_rot < 0 || d->d_rot > d->d_head || d->d_rot % 16 != 0) return GDN_EINVAL;
    if (d->rot_style != GDN_ROT_HALF && d->rot_style != GDN_ROT_INTERLEAVED) return GDN_EINVAL;
    if (d->act_type != GDN_BF16 && d->act_type != GDN_FP16) return GDN_EINVAL;
    if (d->kv_type != d->act_type && d->kv_type != GDN_E4M3) return GDN_EINVAL;
    if (!std::isfinite(d->scale) || !std::isfinite(d->rot_gain) || !std::isfinite(d->norm_offset)) return GDN_EINVAL;
    if (!(d->eps >= 0.0f) || !std::isfinite(d->eps)) return GDN_EINVAL;
    return GDN_OK;
}

// Sizes of the page state; places and tokens are counted in 31 bits.
int check_pages_sizes(const gdn_pages *g) {
    if (!g) return GDN_ENULL;
    if (g->n_slots <= 0 || g->max_pages <= 0 || g->n_pages <= 0) return GDN_EINVAL;
    if (g->page_size < 16 || g->page_size > 1024 || (g->page_size & (g->page_size - 1))) return GDN_EINVAL;
    if ((int64_t)g->n_pages * g->page_size > INT32_MAX || (int64_t)g->max_pages * g->page_size > INT32_MAX)
        return GDN_EINVAL;
    return GDN_OK;
}

// The table, lengths and held pages (what every call that looks tokens up needs), or with `stack` all of it.
int check_pages(const gdn_pages *g, bool stack) {
    GDN_TRY(check_pages_sizes(g));
    if (!g->block_table || !g->kv_len || !g->n_held) return GDN_ENULL;
    if (stack && (!g->free_pages || !g->n_free)) return GDN_ENULL;
    if (!aligned(g->block_table, 4) || !aligned(g->kv_len, 4) || !aligned(g->n_held, 4)) return GDN_EALIGN;
    if (stack && (!aligned(g->free_pages, 4) || !aligned(g->n_free, 4))) return GDN_EALIGN;
    return GDN_OK;
}

int check_attn_cache(const gdn_attn_cache *c, const gdn_attn_dims *d) {
    if (!c || !c->k || !c->v) return GDN_ENULL;
    if (d->kv_type != GDN_E4M3 && (c->k_scale || c->v_scale)) return GDN_EINVAL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return GDN_EALIGN;
    return GDN_OK;
}

int check_counts(int32_t n_streams, int32_t n_rows) {
    return n_streams <= 0 || n_streams > 65535 || n_rows <= 0 ? GDN_EINVAL : GDN_OK;
}

gdn::PagesParams pages_params(const gdn_pages *g, const int32_t *slot, int32_t n_streams, int *err) {
    gdn::PagesParams p = {};
    p.block_table = g->block_table;
    p.kv_len = g->kv_len;
    p.n_held = g->n_held;
    p.free_pages = g->free_pages;
    p.n_free = g->n_free;
    p.n_slots = g->n_slots;
    p.max_pages = g->max_pages;
    p.n_pages = g->n_pages;
    p.page_size = g->page_size;
    p.slot = slot;
    p.n_streams = n_streams;
    p.err = err;
    return p;
}

int launched() { return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ECUDA; }

void attn_sizes(gdn::AttnParams &p, const gdn_attn_dims *d, const gdn_pages *g, int32_t n_streams, int32_t n_rows) {
    p.n_slots = g->n_slots;
    p.max_pages = g->max_pages;
    p.n_pages = g->n_pages;
    p.page_size = g->page_size;
    p.n_streams = n_streams;
    p.n_rows = n_rows;
    p.Hq = d->n_q_heads;
    p.Hkv = d->n_kv_heads;
    p.G = d->n_q_heads / d->n_kv_heads;
}

int attn_params(gdn::AttnParams &p, const gdn_attn_dims *d, const gdn_attn_cache *c, const gdn_pages *g,
                const int32_t *slot, int32_t n_streams, int32_t n_rows) {
    GDN_TRY(check_attn_dims(d));
    GDN_TRY(check_pages(g, false));
    GDN_TRY(check_attn_cache(c, d));
    if (!slot) return GDN_ENULL;
    GDN_TRY(check_counts(n_streams, n_rows));
    if (!aligned(slot, 4)) return GDN_EALIGN;
    p.k = static_cast<char *>(c->k);
    p.v = static_cast<char *>(c->v);
    p.k_scale = c->k_scale;
    p.v_scale = c->v_scale;
    p.block_table = g->block_table;
    p.kv_len = g->kv_len;
    p.n_held = g->n_held;
    p.slot = slot;
    attn_sizes(p, d, g, n_streams, n_rows);
    p.scale = d->scale;
    return GDN_OK;
}

int attn_entry(const gdn_attn_dims *dims, const gdn_attn_cache *cache, const gdn_pages *pages, const int32_t *slot,
               const int32_t *row_ptr, const int32_t *parent, int32_t n_streams, int32_t n_rows, const void *q,
               void *out, void *workspace, size_t workspace_bytes, void *stream) {
    gdn::AttnParams p = {};
    GDN_TRY(attn_params(p, dims, cache, pages, slot, n_streams, n_rows));
    if (!q || !out) return GDN_ENULL;
    if (!workspace || workspace_bytes < gdn_attn_workspace_size(dims, pages, n_streams, n_rows)) return GDN_EWORKSPACE;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(row_ptr, 4) || !aligned(parent, 4))
        return GDN_EALIGN;
    p.q = static_cast<const char *>(q);
    p.out = static_cast<char *>(out);
    p.row_ptr = row_ptr;
    p.parent = parent;
    p.ws = static_cast<char *>(workspace);
    p.ws_bytes = workspace_bytes;
    if (!(p.err = gdn::device_error_word())) return GDN_ECUDA;
    const int max_rows = row_ptr ? std::min(n_rows, (int32_t)GDN_MAX_WINDOW) : 1;
    return gdn::launch_attn(dims->d_head, dims->act_type, dims->kv_type, max_rows, p,
                            static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GDN_OK
               : GDN_ECUDA;
}

// A thread a stream or row, in whole warps.
int pages_threads(int n) { return std::min((n + 31) / 32 * 32, gdn::kPagesThreads); }

template <int D>
void launch_prep(const gdn_attn_dims *d, const gdn::PrepParams &p, cudaStream_t st) {
    const dim3 grid(std::min(p.n_rows, std::max(1, gdn::sm_count()) * gdn::kPrepCtas)), block(gdn::kPrepThreads);
    if (d->act_type == GDN_BF16) {
        if (d->kv_type == GDN_E4M3) gdn::gdn_attn_prep_kernel<D, GDN_BF16, GDN_E4M3><<<grid, block, 0, st>>>(p);
        else gdn::gdn_attn_prep_kernel<D, GDN_BF16, GDN_BF16><<<grid, block, 0, st>>>(p);
    } else {
        if (d->kv_type == GDN_E4M3) gdn::gdn_attn_prep_kernel<D, GDN_FP16, GDN_E4M3><<<grid, block, 0, st>>>(p);
        else gdn::gdn_attn_prep_kernel<D, GDN_FP16, GDN_FP16><<<grid, block, 0, st>>>(p);
    }
}

}  // namespace

extern "C" {

int gdn_pages_plan(const gdn_pages *pages, const int32_t *slot, const int32_t *row_ptr, const int32_t *parent,
                   int32_t n_streams, int32_t n_rows, int32_t *row_pos, int32_t *row_slot, void *stream) {
    GDN_TRY(check_pages(pages, true));
    if (!slot || !row_ptr || !row_pos || !row_slot) return GDN_ENULL;
    GDN_TRY(check_counts(n_streams, n_rows));
    if (!aligned(slot, 4) || !aligned(row_ptr, 4) || !aligned(parent, 4) || !aligned(row_pos, 4) ||
        !aligned(row_slot, 4))
        return GDN_EALIGN;
    int *err = gdn::device_error_word();
    if (!err) return GDN_ECUDA;
    gdn::PagesParams p = pages_params(pages, slot, n_streams, err);
    p.row_ptr = row_ptr;
    p.parent = parent;
    p.n_rows = n_rows;
    p.row_pos = row_pos;
    p.row_slot = row_slot;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (n_rows <= 4 * gdn::kPagesThreads) {
        gdn::gdn_pages_plan_kernel<true><<<1, pages_threads(std::max(n_streams, n_rows)), 0, st>>>(p);
        return launched();
    }
    gdn::gdn_pages_plan_kernel<false><<<1, gdn::kPagesThreads, 0, st>>>(p);
    GDN_TRY(launched());
    gdn::gdn_pages_place_kernel<<<(n_rows - 1) / 256 + 1, 256, 0, st>>>(p);
    return launched();
}

int gdn_pages_commit(const gdn_pages *pages, const int32_t *slot, const int32_t *row_ptr, const int32_t *parent,
                     const int32_t *keep_row, int32_t n_streams, int32_t n_rows, void *stream) {
    GDN_TRY(check_pages(pages, false));
    if (!slot || !row_ptr || !keep_row) return GDN_ENULL;
    GDN_TRY(check_counts(n_streams, n_rows));
    if (!aligned(slot, 4) || !aligned(row_ptr, 4) || !aligned(parent, 4) || !aligned(keep_row, 4)) return GDN_EALIGN;
    int *err = gdn::device_error_word();
    if (!err) return GDN_ECUDA;
    gdn::PagesParams p = pages_params(pages, slot, n_streams, err);
    p.row_ptr = row_ptr;
    p.parent = parent;
    p.keep_row = keep_row;
    p.n_rows = n_rows;
    gdn::gdn_pages_commit_kernel<<<(n_streams - 1) / 256 + 1, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return launched();
}

int gdn_pages_release(const gdn_pages *pages, const int32_t *slot, int32_t n_streams, void *stream) {
    GDN_TRY(check_pages(pages, true));
    if (!slot) return GDN_ENULL;
    GDN_TRY(check_counts(n_streams, 1));
    if (!aligned(slot, 4)) return GDN_EALIGN;
    int *err = gdn::device_error_word();
    if (!err) return GDN_ECUDA;
    const gdn::PagesParams p = pages_params(pages, slot, n_streams, err);
    gdn::gdn_pages_release_kernel<<<1, gdn::kPagesThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return launched();
}

int gdn_attn_prep(const gdn_attn_dims *dims, const gdn_attn_weights *w, const gdn_attn_cache *cache,
                  const gdn_pages *pages, const gdn_attn_rows *rows, const int32_t *row_pos,
                  const int32_t *row_slot, int32_t n_rows, void *stream) {
    GDN_TRY(check_attn_dims(dims));
    GDN_TRY(check_pages_sizes(pages));
    GDN_TRY(check_attn_cache(cache, dims));
    if (!w || !rows || !rows->q || !rows->k || !rows->v || !rows->q_out || !row_pos || !row_slot) return GDN_ENULL;
    if (dims->d_rot > 0 && !w->inv_freq) return GDN_ENULL;
    if (n_rows <= 0) return GDN_EINVAL;
    for (int64_t s : {rows->q_row, rows->q_head, rows->k_row, rows->k_head, rows->v_row, rows->v_head})
        if (s < 0 || s % 8 != 0) return GDN_EINVAL;
    if (!aligned(rows->q, 16) || !aligned(rows->k, 16) || !aligned(rows->v, 16) || !aligned(rows->q_out, 16) ||
        !aligned(w->q_norm, 16) || !aligned(w->k_norm, 16) || !aligned(w->inv_freq, 8) || !aligned(row_pos, 4) ||
        !aligned(row_slot, 4))
        return GDN_EALIGN;
    gdn::PrepParams p = {};
    if (!(p.err = gdn::device_error_word())) return GDN_ECUDA;
    p.q = static_cast<const char *>(rows->q);
    p.k = static_cast<const char *>(rows->k);
    p.v = static_cast<const char *>(rows->v);
    p.q_out = static_cast<char *>(rows->q_out);
    p.q_row = rows->q_row;
    p.q_head = rows->q_head;
    p.k_row = rows->k_row;
    p.k_head = rows->k_head;
    p.v_row = rows->v_row;
    p.v_head = rows->v_head;
    p.q_norm = static_cast<const char *>(w->q_norm);
    p.k_norm = static_cast<const char *>(w->k_norm);
    p.inv_freq = w->inv_freq;
    p.ck = static_cast<char *>(cache->k);
    p.cv = static_cast<char *>(cache->v);
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.row_pos = row_pos;
    p.row_slot = row_slot;
    p.Hq = dims->n_q_heads;
    p.Hkv = dims->n_kv_heads;
    p.d_rot = dims->d_rot;
    p.interleaved = dims->rot_style == GDN_ROT_INTERLEAVED;
    p.n_pages = pages->n_pages;
    p.page_size = pages->page_size;
    p.n_rows = n_rows;
    p.rot_gain = dims->rot_gain;
    p.norm_offset = dims->norm_offset;
    p.eps = dims->eps;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dims->d_head) {
        case 64: launch_prep<64>(dims, p, st); break;
        case 128: launch_prep<128>(dims, p, st); break;
        default: launch_prep<256>(dims, p, st); break;
    }
    return launched();
}

size_t gdn_attn_workspace_size(const gdn_attn_dims *dims, const gdn_pages *pages, int32_t n_streams, int32_t n_rows) {
    if (check_attn_dims(dims) != GDN_OK || check_pages_sizes(pages) != GDN_OK ||
        check_counts(n_streams, n_rows) != GDN_OK)
        return 0;
    gdn::AttnParams p = {};
    attn_sizes(p, dims, pages, n_streams, n_rows);
    return gdn::attn_workspace(p, dims->d_head);
}

int gdn_attn_step(const gdn_attn_dims *dims, const gdn_attn_cache *cache, const gdn_pages *pages,
                  const int32_t *slot, int32_t n_streams, const void *q, void *out, void *workspace,
                  size_t workspace_bytes, void *stream) {
    return attn_entry(dims, cache, pages, slot, nullptr, nullptr, n_streams, n_streams, q, out, workspace,
                      workspace_bytes, stream);
}

int gdn_attn_window(const gdn_attn_dims *dims, const gdn_attn_cache *cache, const gdn_pages *pages,
                    const int32_t *slot, const int32_t *row_ptr, int32_t n_streams, int32_t n_rows, const void *q,
                    void *out, void *workspace, size_t workspace_bytes, void *stream) {
    if (!row_ptr) return GDN_ENULL;
    return attn_entry(dims, cache, pages, slot, row_ptr, nullptr, n_streams, n_rows, q, out, workspace,
                      workspace_bytes, stream);
}

int gdn_attn_tree(const gdn_attn_dims *dims, const gdn_attn_cache *cache, const gdn_pages *pages,
                  const int32_t *slot, const int32_t *row_ptr, const int32_t *parent, int32_t n_streams,
                  int32_t n_rows, const void *q, void *out, void *workspace, size_t workspace_bytes, void *stream) {
    if (!row_ptr || !parent) return GDN_ENULL;
    return attn_entry(dims, cache, pages, slot, row_ptr, parent, n_streams, n_rows, q, out, workspace,
                      workspace_bytes, stream);
}

int gdn_debug_attn_wait_limit(uint32_t polls) { return gdn::attn_wait_limit(polls) ? GDN_OK : GDN_EINVAL; }

int gdn_attn_commit(const gdn_attn_dims *dims, const gdn_attn_cache *cache, const gdn_pages *pages,
                    const int32_t *slot, const int32_t *row_ptr, const int32_t *parent, const int32_t *keep_row,
                    int32_t n_streams, int32_t n_rows, void *stream) {
    gdn::AttnParams p = {};
    GDN_TRY(attn_params(p, dims, cache, pages, slot, n_streams, n_rows));
    if (!row_ptr || !parent || !keep_row) return GDN_ENULL;
    if (!aligned(row_ptr, 4) || !aligned(parent, 4) || !aligned(keep_row, 4)) return GDN_EALIGN;
    p.row_ptr = row_ptr;
    p.parent = parent;
    p.keep_row = keep_row;
    if (!(p.err = gdn::device_error_word())) return GDN_ECUDA;
    const int row_bytes = dims->d_head * (dims->kv_type == GDN_E4M3 ? 1 : 2);
    gdn::gdn_attn_commit_kernel<<<dim3(p.Hkv, n_streams), gdn::kMoveThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        p, row_bytes);
    return launched();
}

}  // extern "C"
