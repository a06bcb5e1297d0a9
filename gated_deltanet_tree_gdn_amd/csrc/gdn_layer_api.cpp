// gdn_layer_api.cpp -- the C ABI declared in include/gdn_layer.h: O(1) host
// argument checks (made before any HIP call) and dispatch to the kernel
// launchers.  Nothing here allocates device memory or synchronises.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <string>

#include "gdn_internal.h"
#include "gdn_layer.h"
#include "gdn_layer_internal.h"

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

gdn_status check_ptr(const void* p, const char* name, bool required = true) {
    if (!p) return required ? fail(GDN_ERR_NULL, "%s is NULL", name) : GDN_OK;
    if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0) return fail(GDN_ERR_ALIGN, "%s is not 16-byte aligned", name);
    return GDN_OK;
}

// Rows that kernels read in pieces of any alignment.
gdn_status check_rows(const void* p, int32_t dtype, const char* name, bool required = true) {
    if (!p) return required ? fail(GDN_ERR_NULL, "%s is NULL", name) : GDN_OK;
    if (reinterpret_cast<uintptr_t>(p) % (dtype == GDN_BF16 ? 2 : 4) != 0)
        return fail(GDN_ERR_ALIGN, "%s is not aligned to its elements", name);
    return GDN_OK;
}

gdn_status check_dtype(int32_t t, const char* name) {
    if (t != GDN_BF16 && t != GDN_F32) return fail(GDN_ERR_DTYPE, "%s must be GDN_BF16 or GDN_F32", name);
    return GDN_OK;
}

gdn_status check_in_stride(int64_t s, const char* name) {
    if (s < 0) return fail(GDN_ERR_SHAPE, "%s must be >= 0", name);
    return GDN_OK;
}

gdn_status check_out_stride(int64_t s, int64_t row, int64_t rows, const char* name) {
    if (s < row && rows > 1) return fail(GDN_ERR_SHAPE, "%s is smaller than a row", name);
    if (s < 0) return fail(GDN_ERR_SHAPE, "%s must be >= 0", name);
    return GDN_OK;
}

#define GDN_TRY(expr)                       \
    do {                                    \
        gdn_status _s = (expr);             \
        if (_s != GDN_OK) return _s;        \
    } while (0)

// !(x >= 0) also refuses NaN.
gdn_status check_eps(float e, const char* name) {
    if (!(e >= 0.0f)) return fail(GDN_ERR_SHAPE, "%s must be >= 0", name);
    return GDN_OK;
}

gdn_status check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return GDN_OK;
    if (!ws || have < need) return fail(GDN_ERR_WORKSPACE, "workspace missing or smaller than required");
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return fail(GDN_ERR_ALIGN, "workspace is not 256-byte aligned");
    return GDN_OK;
}

gdn_status check_seq_dims(const gdn_seq_dims* d, bool prefill) {
    if (!d) return fail(GDN_ERR_NULL, "dims is NULL");
    GDN_TRY(check_dtype(d->qkv_dtype, "qkv_dtype"));
    GDN_TRY(check_dtype(d->o_dtype, "o_dtype"));
    if (d->B < 0 || (prefill && d->T < 0)) return fail(GDN_ERR_SHAPE, "B and T must be >= 0");
    if (d->B > 65535) return fail(GDN_ERR_SHAPE, "B must be at most 65535");
    if (d->H_k < 1 || d->H_v < 1 || d->H_v > 65535) return fail(GDN_ERR_SHAPE, "H_k and H_v must be in [1, 65535]");
    if (int64_t(d->B) * d->H_v > (1 << 24)) return fail(GDN_ERR_SHAPE, "B * H_v must be at most 2^24");
    if (d->H_v % d->H_k != 0) return fail(GDN_ERR_SHAPE, "H_v must be a multiple of H_k");
    if ((d->d_k != 64 && d->d_k != 128) || (d->d_v != 64 && d->d_v != 128))
        return fail(GDN_ERR_SHAPE, "d_k and d_v must be 64 or 128");
    if (d->n_slots < 0) return fail(GDN_ERR_SHAPE, "n_slots must be >= 0");
    GDN_TRY(check_eps(d->l2_eps, "l2_eps"));
    GDN_TRY(check_in_stride(d->q_stride, "q_stride"));
    GDN_TRY(check_in_stride(d->k_stride, "k_stride"));
    GDN_TRY(check_in_stride(d->v_stride, "v_stride"));
    if (d->q_stride > GDN_MAX_SEQ_STRIDE || d->k_stride > GDN_MAX_SEQ_STRIDE || d->v_stride > GDN_MAX_SEQ_STRIDE)
        return fail(GDN_ERR_SHAPE, "q, k and v strides must be at most 2^24");
    if (int64_t(d->H_v) * d->d_v > GDN_MAX_SEQ_STRIDE) return fail(GDN_ERR_SHAPE, "H_v * d_v must be at most 2^24");
    const int64_t unit = d->qkv_dtype == GDN_BF16 ? 8 : 4;
    if (d->q_stride % unit || d->k_stride % unit || d->v_stride % unit)
        return fail(GDN_ERR_ALIGN, "q, k and v strides must be multiples of 16 bytes");
    return GDN_OK;
}

}  // namespace

extern "C" {

size_t gdn_prefill_workspace_bytes(const gdn_seq_dims* dims) {
    if (!dims || dims->B <= 0 || dims->T <= 0 || dims->H_k < 1 || dims->H_v < 1) return 0;
    return gdn::prefill_ws_bytes(*dims);
}

gdn_status gdn_prefill(const gdn_seq_dims* dims, const void* q, const void* k, const void* v, const float* g,
                       const float* beta, const int32_t* cu_seqlens, const int32_t* slot, const int32_t* has_state,
                       float* S, void* o, int32_t* seq_status, void* workspace, size_t workspace_bytes,
                       hipStream_t stream) {
    GDN_TRY(check_seq_dims(dims, true));
    if (dims->B == 0) return fail(GDN_OK, "");
    GDN_TRY(check_ptr(cu_seqlens, "cu_seqlens"));
    if (dims->T > 0) {
        GDN_TRY(check_ptr(q, "q"));
        GDN_TRY(check_ptr(k, "k"));
        GDN_TRY(check_ptr(v, "v"));
        GDN_TRY(check_ptr(g, "g"));
        GDN_TRY(check_ptr(beta, "beta"));
        GDN_TRY(check_ptr(o, "o"));
    }
    GDN_TRY(check_ptr(S, "S", dims->n_slots > 0));
    GDN_TRY(check_ptr(slot, "slot", false));
    GDN_TRY(check_ptr(has_state, "has_state", false));
    GDN_TRY(check_ptr(seq_status, "seq_status", false));
    if (!slot && dims->n_slots > 0 && dims->n_slots < dims->B)
        return fail(GDN_ERR_SHAPE, "without slot, n_slots must be 0 or at least B");
    GDN_TRY(check_workspace(workspace, workspace_bytes, gdn_prefill_workspace_bytes(dims)));
    gdn::SeqArgs a{*dims, q, k, v, g, beta, cu_seqlens, slot, has_state, S, o, seq_status, workspace};
    return done(gdn::launch_prefill(a, stream), "prefill");
}

gdn_status gdn_decode(const gdn_seq_dims* dims, const void* q, const void* k, const void* v, const float* g,
                      const float* beta, const int32_t* slot, float* S, void* o, hipStream_t stream) {
    GDN_TRY(check_seq_dims(dims, false));
    if (dims->B == 0) return fail(GDN_OK, "");
    GDN_TRY(check_ptr(q, "q"));
    GDN_TRY(check_ptr(k, "k"));
    GDN_TRY(check_ptr(v, "v"));
    GDN_TRY(check_ptr(g, "g"));
    GDN_TRY(check_ptr(beta, "beta"));
    GDN_TRY(check_ptr(slot, "slot", false));
    GDN_TRY(check_ptr(S, "S", dims->n_slots > 0));
    GDN_TRY(check_ptr(o, "o"));
    if (!slot && dims->n_slots < dims->B) return fail(GDN_ERR_SHAPE, "without slot, n_slots must be at least B");
    gdn::SeqArgs a{*dims, q, k, v, g, beta, nullptr, slot, nullptr, S, o, nullptr, nullptr};
    return done(gdn::launch_decode(a, stream), "decode");
}

gdn_status gdn_add_norm(const gdn_add_norm_dims* dims, const void* x, const void* residual, const float* weight,
                        const float* post_weight, const float* chan_scale, void* h, void* y, hipStream_t stream) {
    if (!dims) return fail(GDN_ERR_NULL, "dims is NULL");
    const gdn_add_norm_dims& d = *dims;
    GDN_TRY(check_dtype(d.x_dtype, "x_dtype"));
    GDN_TRY(check_dtype(d.res_dtype, "res_dtype"));
    GDN_TRY(check_dtype(d.y_dtype, "y_dtype"));
    if (d.T < 0) return fail(GDN_ERR_SHAPE, "T must be >= 0");
    if (d.D < 1 || d.D > GDN_NORM_MAX_D) return fail(GDN_ERR_SHAPE, "D must be in [1, 16384]");
    GDN_TRY(check_eps(d.eps, "eps"));
    GDN_TRY(check_in_stride(d.x_stride, "x_stride"));
    if (residual) GDN_TRY(check_in_stride(d.res_stride, "res_stride"));
    if (h) GDN_TRY(check_out_stride(d.h_stride, d.D, d.T, "h_stride"));
    GDN_TRY(check_out_stride(d.y_stride, d.D, d.T, "y_stride"));
    if (d.T == 0) return fail(GDN_OK, "");
    GDN_TRY(check_rows(x, d.x_dtype, "x"));
    GDN_TRY(check_rows(residual, d.res_dtype, "residual", false));
    GDN_TRY(check_ptr(weight, "weight"));
    GDN_TRY(check_ptr(post_weight, "post_weight", false));
    GDN_TRY(check_ptr(chan_scale, "chan_scale", false));
    GDN_TRY(check_rows(h, d.res_dtype, "h", false));
    GDN_TRY(check_rows(y, d.y_dtype, "y"));
    if (h && h == residual && d.h_stride != d.res_stride && d.T > 1)
        return fail(GDN_ERR_SHAPE, "h in place of residual needs the same stride");
    return done(gdn::launch_add_norm({d, x, residual, weight, post_weight, chan_scale, h, y}, stream), "add_norm");
}

gdn_status gdn_gated_norm(const gdn_gated_norm_dims* dims, const void* o, const void* z, const float* weight,
                          void* y, hipStream_t stream) {
    if (!dims) return fail(GDN_ERR_NULL, "dims is NULL");
    const gdn_gated_norm_dims& d = *dims;
    GDN_TRY(check_dtype(d.o_dtype, "o_dtype"));
    GDN_TRY(check_dtype(d.z_dtype, "z_dtype"));
    GDN_TRY(check_dtype(d.y_dtype, "y_dtype"));
    if (d.T < 0 || d.H < 1) return fail(GDN_ERR_SHAPE, "T must be >= 0 and H >= 1");
    if (d.d < 1 || d.d > GDN_NORM_MAX_D) return fail(GDN_ERR_SHAPE, "d must be in [1, 16384]");
    if (d.gate != GDN_ACT_SILU && d.gate != GDN_ACT_SIGMOID)
        return fail(GDN_ERR_SHAPE, "gate must be GDN_ACT_SILU or GDN_ACT_SIGMOID");
    GDN_TRY(check_eps(d.eps, "eps"));
    GDN_TRY(check_in_stride(d.o_stride, "o_stride"));
    GDN_TRY(check_in_stride(d.z_stride, "z_stride"));
    GDN_TRY(check_out_stride(d.y_stride, int64_t(d.H) * d.d, d.T, "y_stride"));
    if (d.T == 0) return fail(GDN_OK, "");
    GDN_TRY(check_rows(o, d.o_dtype, "o"));
    GDN_TRY(check_rows(z, d.z_dtype, "z"));
    GDN_TRY(check_ptr(weight, "weight"));
    GDN_TRY(check_rows(y, d.y_dtype, "y"));
    if ((y == o && (d.y_dtype != d.o_dtype || (d.y_stride != d.o_stride && d.T > 1))) ||
        (y == z && (d.y_dtype != d.z_dtype || (d.y_stride != d.z_stride && d.T > 1))))
        return fail(GDN_ERR_SHAPE, "y in place needs the same dtype and stride");
    return done(gdn::launch_gated_norm({d, o, z, weight, y}, stream), "gated_norm");
}

static gdn_status check_linear_dims(const gdn_linear_dims* dims) {
    if (!dims) return fail(GDN_ERR_NULL, "dims is NULL");
    if (dims->M < 0 || dims->N < 0 || dims->K < 0) return fail(GDN_ERR_SHAPE, "M, N and K must be >= 0");
    GDN_TRY(check_dtype(dims->y_dtype, "y_dtype"));
    GDN_TRY(check_dtype(dims->res_dtype, "res_dtype"));
    if (dims->act < GDN_ACT_NONE || dims->act > GDN_ACT_SIGMOID) return fail(GDN_ERR_SHAPE, "unknown act");
    GDN_TRY(check_in_stride(dims->x_stride, "x_stride"));
    GDN_TRY(check_in_stride(dims->w_stride, "w_stride"));
    return check_out_stride(dims->y_stride, dims->N, dims->M, "y_stride");
}

size_t gdn_linear_workspace_bytes(const gdn_linear_dims* dims) {
    if (!dims || dims->M <= 0 || dims->N <= 0 || dims->K <= 0) return 0;
    return gdn::linear_ws_bytes(*dims);
}

gdn_status gdn_linear(const gdn_linear_dims* dims, const void* x, const void* w, const float* bias,
                      const void* residual, void* y, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    GDN_TRY(check_linear_dims(dims));
    if (dims->M == 0 || dims->N == 0) return fail(GDN_OK, "");
    if (dims->K > 0) {
        GDN_TRY(check_ptr(x, "x"));
        GDN_TRY(check_ptr(w, "w"));
    }
    GDN_TRY(check_ptr(bias, "bias", false));
    GDN_TRY(check_ptr(residual, "residual", false));
    GDN_TRY(check_ptr(y, "y"));
    if (residual) GDN_TRY(check_in_stride(dims->res_stride, "res_stride"));
    if (residual == y && (dims->res_dtype != dims->y_dtype || (dims->res_stride != dims->y_stride && dims->M > 1)))
        return fail(GDN_ERR_SHAPE, "y in place of residual needs the same dtype and stride");
    GDN_TRY(check_workspace(workspace, workspace_bytes, gdn_linear_workspace_bytes(dims)));
    return done(gdn::launch_linear({*dims, x, w, bias, residual, y, workspace}, stream), "linear");
}

}  // extern "C"
