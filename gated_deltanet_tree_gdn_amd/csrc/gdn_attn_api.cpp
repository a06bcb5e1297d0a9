// gdn_attn_api.cpp -- the C ABI declared in include/gdn_attn.h: O(1) host
// argument checks (made before any HIP call) and dispatch to the kernel
// launchers.  Nothing here allocates device memory or synchronises.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <string>

#include "gdn_attn.h"
#include "gdn_attn_internal.h"
#include "gdn_internal.h"

namespace {

// The detail message is composed in a fixed buffer and assigned under a
// catch-all, so that no exception crosses the C boundary.
gdn_status fail(gdn_status s, const char* fmt, const char* name = "") noexcept {
    char msg[192];
    std::snprintf(msg, sizeof msg, fmt, name);
    try {
        gdn::set_last_error(msg);
    } catch (...) {
    }
    return s;
}

gdn_status done(hipError_t e, const char* what) noexcept {
    if (e != hipSuccess) {
        char msg[192];
        std::snprintf(msg, sizeof msg, "%s launch: %s", what, hipGetErrorString(e));
        return fail(GDN_ERR_HIP, "%s", msg);
    }
    return fail(GDN_OK, "");
}

#define GDN_TRY(expr)                       \
    do {                                    \
        gdn_status _s = (expr);             \
        if (_s != GDN_OK) return _s;        \
    } while (0)

gdn_status check_ptr(const void* p, size_t align, const char* name, bool required = true) {
    if (!p) return required ? fail(GDN_ERR_NULL, "%s is NULL", name) : GDN_OK;
    if (reinterpret_cast<uintptr_t>(p) % align != 0) return fail(GDN_ERR_ALIGN, "%s is not aligned as required", name);
    return GDN_OK;
}

gdn_status check_stride(int64_t s, int64_t unit, const char* name) {
    if (s < 0 || s > (int64_t(1) << 40)) return fail(GDN_ERR_SHAPE, "%s must be in [0, 2^40]", name);
    if (s % unit) return fail(GDN_ERR_ALIGN, "%s must be a multiple of 16 bytes", name);
    return GDN_OK;
}

gdn_status check_cache(const gdn_kv_cache* c) {
    if (!c) return fail(GDN_ERR_NULL, "cache is NULL");
    if (c->dtype != GDN_BF16 && c->dtype != GDN_E4M3) return fail(GDN_ERR_DTYPE, "a cache is GDN_BF16 or GDN_E4M3");
    if (c->d != 64 && c->d != 128 && c->d != 256) return fail(GDN_ERR_SHAPE, "d must be 64, 128 or 256");
    if (c->n_pages < 1) return fail(GDN_ERR_SHAPE, "n_pages must be at least 1");
    if (c->page_size < 1 || c->page_size > 65536 || (c->page_size & (c->page_size - 1)))
        return fail(GDN_ERR_SHAPE, "page_size must be a power of two up to 65536");
    if (int64_t(c->n_pages) * c->page_size > INT32_MAX) return fail(GDN_ERR_SHAPE, "n_pages * page_size must be at most 2^31 - 1");
    if (c->H_kv < 1 || c->H_kv > 65535) return fail(GDN_ERR_SHAPE, "H_kv must be in [1, 65535]");
    if (c->reserved != 0) return fail(GDN_ERR_SHAPE, "reserved must be 0");
    const int64_t unit = c->dtype == GDN_BF16 ? 8 : 16;
    GDN_TRY(check_stride(c->k_page_stride, unit, "k_page_stride"));
    GDN_TRY(check_stride(c->k_row_stride, unit, "k_row_stride"));
    GDN_TRY(check_stride(c->k_head_stride, unit, "k_head_stride"));
    GDN_TRY(check_stride(c->v_page_stride, unit, "v_page_stride"));
    GDN_TRY(check_stride(c->v_row_stride, unit, "v_row_stride"));
    GDN_TRY(check_stride(c->v_head_stride, unit, "v_head_stride"));
    if (c->k_row_stride > GDN_MAX_SEQ_STRIDE || c->v_row_stride > GDN_MAX_SEQ_STRIDE)
        return fail(GDN_ERR_SHAPE, "row strides of a cache must be at most 2^24");
    GDN_TRY(check_ptr(c->k, 16, "k of the cache"));
    GDN_TRY(check_ptr(c->v, 16, "v of the cache"));
    GDN_TRY(check_ptr(c->k_scale, 4, "k_scale", false));
    return check_ptr(c->v_scale, 4, "v_scale", false);
}

gdn_status check_pages(int32_t max_pages, int32_t page_size, int64_t table_stride) {
    if (max_pages < 0 || int64_t(max_pages) * page_size > (int64_t(1) << 30))
        return fail(GDN_ERR_SHAPE, "max_pages * page_size must be in [0, 2^30]");
    return check_stride(table_stride, 1, "table_stride");
}

gdn_status check_attn(const gdn_attn_dims* d, const gdn_kv_cache* c, gdn::AttnKind kind) {
    if (!d) return fail(GDN_ERR_NULL, "dims is NULL");
    GDN_TRY(check_cache(c));
    if (d->B < 0 || d->B > 65535) return fail(GDN_ERR_SHAPE, "B must be in [0, 65535]");
    if (kind != gdn::kAttnDecode && d->T < 0) return fail(GDN_ERR_SHAPE, "T must be >= 0");
    if (kind == gdn::kAttnVerify && d->T > GDN_ATTN_MAX_N) return fail(GDN_ERR_SHAPE, "N must be at most 256");
    if (d->H_q < 1 || d->H_q % c->H_kv) return fail(GDN_ERR_SHAPE, "H_q must be a multiple of H_kv, at least 1");
    const int64_t rows = kind == gdn::kAttnDecode ? d->B : kind == gdn::kAttnVerify ? int64_t(d->B) * d->T : d->T;
    // (the last tile's rows are numbered in 32 bits as if it were whole)
    if (rows * d->H_q > INT32_MAX - 255 || d->H_q > (1 << 24))
        return fail(GDN_ERR_SHAPE, "rows of q times H_q must be at most 2^31 - 256");
    if (!(d->scale >= 0.0f) || !std::isfinite(d->scale)) return fail(GDN_ERR_SHAPE, "scale must be >= 0 and finite");
    if (d->reserved != 0) return fail(GDN_ERR_SHAPE, "reserved must be 0");
    GDN_TRY(check_stride(d->q_stride, 8, "q_stride"));
    GDN_TRY(check_stride(d->gate_stride, 1, "gate_stride"));
    GDN_TRY(check_stride(d->gate_head_stride, 1, "gate_head_stride"));
    return check_pages(d->max_pages, c->page_size, d->table_stride);
}

// Nothing to compute: no query.
bool is_empty(const gdn_attn_dims& d, gdn::AttnKind kind) { return d.B == 0 || (kind != gdn::kAttnDecode && d.T == 0); }

size_t workspace_bytes_of(const gdn_attn_dims* d, const gdn_kv_cache* c, gdn::AttnKind kind) {
    if (check_attn(d, c, kind) != GDN_OK || is_empty(*d, kind)) return 0;
    gdn::AttnArgs a{};
    a.d = *d;
    a.cache = *c;
    a.kind = kind;
    gdn::attn_shape(a);
    return gdn::attn_ws_bytes(a);
}

// Whether the parts have room in a workspace of `bytes`.  Teams are whole, so the
// parts of a tree may be a little fewer than those of one with fewer nodes; what a
// larger tree asks for, which is two thirds or more, serves a smaller one with
// fewer teams.
bool attn_fit(gdn::AttnArgs& a, size_t bytes) {
    const size_t need = gdn::attn_ws_bytes(a);
    if (bytes >= need) return true;
    if (a.kind != gdn::kAttnVerify) return false;
    size_t least = need;
    gdn::AttnArgs larger = a;
    while (++larger.d.T <= GDN_ATTN_MAX_N) {
        gdn::attn_shape(larger);
        if (const size_t n = gdn::attn_ws_bytes(larger)) least = std::min(least, n);
    }
    if (bytes < least) return false;
    a.teams = int(bytes / (need / a.teams));
    a.join = a.teams > 1;
    return true;
}

gdn_status run(gdn::AttnArgs& a, size_t workspace_bytes, hipStream_t stream, const char* what) {
    const bool prefill = a.kind == gdn::kAttnPrefill;
    if (a.d.B == 0) return fail(GDN_OK, "");
    GDN_TRY(check_ptr(a.cu, 4, "cu_seqlens", prefill));
    GDN_TRY(check_ptr(a.table, 4, "table", a.d.max_pages > 0));
    GDN_TRY(check_ptr(a.length, 4, "length"));
    GDN_TRY(check_ptr(a.seq_status, 4, "seq_status", false));
    const bool empty = is_empty(a.d, a.kind);
    if (!empty) {
        GDN_TRY(check_ptr(a.q, 16, "q"));
        GDN_TRY(check_ptr(a.anc, 4, "anc", a.kind == gdn::kAttnVerify));
        GDN_TRY(check_ptr(a.gate, 2, "gate", false));
        GDN_TRY(check_ptr(a.o, 16, "o"));
        if (a.o == a.q) return fail(GDN_ERR_SHAPE, "o may not be q");
    }
    gdn::attn_shape(a);
    if (!empty) {
        if (gdn::attn_ws_bytes(a) > 0) {
            if (!a.ws || !attn_fit(a, workspace_bytes)) return fail(GDN_ERR_WORKSPACE, "workspace missing or smaller than required");
            GDN_TRY(check_ptr(a.ws, 256, "workspace"));
        }
        hipError_t e = a.kind == gdn::kAttnDecode ? gdn::launch_attn_decode(a, stream) : gdn::launch_attn_tiles(a, stream);
        if (e == hipSuccess && a.join) e = gdn::launch_attn_join(a, stream);
        if (e != hipSuccess) return done(e, what);
    }
    return done(a.seq_status ? gdn::launch_attn_status(a, stream) : hipSuccess, what);
}

}  // namespace

extern "C" {

gdn_status gdn_kv_append(const gdn_kv_append_dims* dims, const gdn_kv_cache* cache, const void* q, const void* k,
                         const void* v, const float* q_weight, const float* k_weight, const float* inv_freq,
                         const int32_t* position, const int32_t* slot, void* q_out, hipStream_t stream) {
    if (!dims) return fail(GDN_ERR_NULL, "dims is NULL");
    GDN_TRY(check_cache(cache));
    const gdn_kv_append_dims& d = *dims;
    if (d.in_dtype != GDN_BF16 && d.in_dtype != GDN_F32) return fail(GDN_ERR_DTYPE, "in_dtype must be GDN_BF16 or GDN_F32");
    if (d.T < 0 || d.H_q < 0 || d.H_q > 65535) return fail(GDN_ERR_SHAPE, "T must be >= 0 and H_q in [0, 65535]");
    if (d.rot < 0 || d.rot > cache->d || (d.rot & 1)) return fail(GDN_ERR_SHAPE, "rot must be even and in [0, d]");
    if (d.interleaved != 0 && d.interleaved != 1) return fail(GDN_ERR_SHAPE, "interleaved must be 0 or 1");
    if (!(d.eps >= 0.0f)) return fail(GDN_ERR_SHAPE, "eps must be >= 0");
    if (d.reserved != 0) return fail(GDN_ERR_SHAPE, "reserved must be 0");
    const int64_t strides[] = {d.q_stride, d.q_head_stride, d.k_stride, d.k_head_stride, d.v_stride, d.v_head_stride};
    const char* names[] = {"q_stride", "q_head_stride", "k_stride", "k_head_stride", "v_stride", "v_head_stride"};
    for (int i = 0; i < 6; ++i) GDN_TRY(check_stride(strides[i], 1, names[i]));
    if (d.T == 0) return fail(GDN_OK, "");
    const size_t unit = d.in_dtype == GDN_BF16 ? 2 : 4;
    if (d.H_q > 0) {
        GDN_TRY(check_ptr(q, unit, "q"));
        GDN_TRY(check_ptr(q_out, 16, "q_out"));
        if (q == q_out && (d.in_dtype != GDN_BF16 || (d.q_head_stride != cache->d && d.H_q > 1) ||
                           (d.q_stride != int64_t(d.H_q) * cache->d && d.T > 1)))
            return fail(GDN_ERR_SHAPE, "q_out in place needs bf16 and dense q");
    }
    GDN_TRY(check_ptr(k, unit, "k"));
    GDN_TRY(check_ptr(v, unit, "v"));
    GDN_TRY(check_ptr(q_weight, 4, "q_weight", false));
    GDN_TRY(check_ptr(k_weight, 4, "k_weight", false));
    GDN_TRY(check_ptr(inv_freq, 4, "inv_freq", d.rot > 0));
    GDN_TRY(check_ptr(position, 4, "position", d.rot > 0));
    GDN_TRY(check_ptr(slot, 4, "slot"));
    return done(gdn::launch_kv_append({d, *cache, q, k, v, q_weight, k_weight, inv_freq, position, slot, q_out}, stream),
                "kv_append");
}

size_t gdn_attn_prefill_workspace_bytes(const gdn_attn_dims* dims, const gdn_kv_cache* cache) {
    return workspace_bytes_of(dims, cache, gdn::kAttnPrefill);
}
size_t gdn_attn_decode_workspace_bytes(const gdn_attn_dims* dims, const gdn_kv_cache* cache) {
    return workspace_bytes_of(dims, cache, gdn::kAttnDecode);
}
size_t gdn_attn_verify_workspace_bytes(const gdn_attn_dims* dims, const gdn_kv_cache* cache) {
    return workspace_bytes_of(dims, cache, gdn::kAttnVerify);
}

gdn_status gdn_attn_decode(const gdn_attn_dims* dims, const gdn_kv_cache* cache, const void* q, const int32_t* table,
                           const int32_t* length, const void* gate, void* o, int32_t* seq_status, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
    GDN_TRY(check_attn(dims, cache, gdn::kAttnDecode));
    gdn::AttnArgs a{};
    a.d = *dims;
    a.cache = *cache;
    a.q = static_cast<const uint16_t*>(q);
    a.table = table;
    a.length = length;
    a.gate = static_cast<const uint16_t*>(gate);
    a.o = static_cast<uint16_t*>(o);
    a.seq_status = seq_status;
    a.ws = workspace;
    a.kind = gdn::kAttnDecode;
    return run(a, workspace_bytes, stream, "attn_decode");
}

gdn_status gdn_attn_prefill(const gdn_attn_dims* dims, const gdn_kv_cache* cache, const void* q,
                            const int32_t* cu_seqlens, const int32_t* table, const int32_t* length, const void* gate,
                            void* o, int32_t* seq_status, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    GDN_TRY(check_attn(dims, cache, gdn::kAttnPrefill));
    gdn::AttnArgs a{};
    a.d = *dims;
    a.cache = *cache;
    a.q = static_cast<const uint16_t*>(q);
    a.cu = cu_seqlens;
    a.table = table;
    a.length = length;
    a.gate = static_cast<const uint16_t*>(gate);
    a.o = static_cast<uint16_t*>(o);
    a.seq_status = seq_status;
    a.ws = workspace;
    a.kind = gdn::kAttnPrefill;
    return run(a, workspace_bytes, stream, "attn_prefill");
}

gdn_status gdn_attn_verify(const gdn_attn_dims* dims, const gdn_kv_cache* cache, const void* q, const uint32_t* anc,
                           const int32_t* table, const int32_t* length, const void* gate, void* o, int32_t* seq_status,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
    GDN_TRY(check_attn(dims, cache, gdn::kAttnVerify));
    gdn::AttnArgs a{};
    a.d = *dims;
    a.cache = *cache;
    a.q = static_cast<const uint16_t*>(q);
    a.anc = anc;
    a.table = table;
    a.length = length;
    a.gate = static_cast<const uint16_t*>(gate);
    a.o = static_cast<uint16_t*>(o);
    a.seq_status = seq_status;
    a.ws = workspace;
    a.kind = gdn::kAttnVerify;
    return run(a, workspace_bytes, stream, "attn_verify");
}

gdn_status gdn_kv_commit(const gdn_kv_commit_dims* dims, const gdn_kv_cache* caches, int32_t n_caches,
                         const uint32_t* anc, const int32_t* accepted, const int32_t* table, const int32_t* length,
                         int32_t* new_length, int32_t* seq_status, hipStream_t stream) {
    if (!dims) return fail(GDN_ERR_NULL, "dims is NULL");
    if (!caches) return fail(GDN_ERR_NULL, "caches is NULL");
    const gdn_kv_commit_dims& d = *dims;
    if (d.B < 0 || d.B > 65535) return fail(GDN_ERR_SHAPE, "B must be in [0, 65535]");
    if (d.N < 0 || d.N > GDN_ATTN_MAX_N) return fail(GDN_ERR_SHAPE, "N must be in [0, 256]");
    if (d.reserved != 0) return fail(GDN_ERR_SHAPE, "reserved must be 0");
    if (n_caches < 1) return fail(GDN_ERR_SHAPE, "n_caches must be at least 1");
    for (int i = 0; i < n_caches; ++i) {
        GDN_TRY(check_cache(caches + i));
        const gdn_kv_cache &x = caches[0], &y = caches[i];
        if (x.n_pages != y.n_pages || x.page_size != y.page_size || x.H_kv != y.H_kv || x.d != y.d || x.dtype != y.dtype ||
            x.k_page_stride != y.k_page_stride || x.k_row_stride != y.k_row_stride || x.k_head_stride != y.k_head_stride ||
            x.v_page_stride != y.v_page_stride || x.v_row_stride != y.v_row_stride || x.v_head_stride != y.v_head_stride)
            return fail(GDN_ERR_SHAPE, "the caches of a commit must have the same sizes and strides");
    }
    GDN_TRY(check_pages(d.max_pages, caches->page_size, d.table_stride));
    if (d.B == 0) return fail(GDN_OK, "");
    GDN_TRY(check_ptr(anc, 4, "anc", d.N > 0));
    GDN_TRY(check_ptr(accepted, 4, "accepted"));
    GDN_TRY(check_ptr(table, 4, "table", d.max_pages > 0));
    GDN_TRY(check_ptr(length, 4, "length"));
    GDN_TRY(check_ptr(new_length, 4, "new_length"));
    GDN_TRY(check_ptr(seq_status, 4, "seq_status", false));
    if (new_length == length) return fail(GDN_ERR_SHAPE, "new_length may not be length");
    for (int first = 0; first < n_caches; first += gdn::kCommitCaches) {
        const int n = std::min(n_caches - first, gdn::kCommitCaches);
        gdn::KvCommitArgs a{d, *caches, {}, {}, 0, 0, anc, accepted, table, length, first ? nullptr : new_length, seq_status};
        for (int i = 0; i < n; ++i) {
            a.k[i] = caches[first + i].k;
            a.v[i] = caches[first + i].v;
            for (int j = 0; j < first + i; ++j) {
                if (caches[j].k == a.k[i]) a.k_moved |= 1u << i;
                if (caches[j].v == a.v[i]) a.v_moved |= 1u << i;
            }
        }
        const hipError_t e = gdn::launch_kv_commit(a, n, stream);
        if (e != hipSuccess) return done(e, "kv_commit");
    }
    return fail(GDN_OK, "");
}

}  // extern "C"
