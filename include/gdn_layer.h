/*
 * gdn_layer.h -- C ABI of the operators around the tree verification of
 * gdn_tree.h: what brings a Gated DeltaNet (GDN) layer from a prompt to the
 * prefix state S0 that gdn_tree_verify reads, and what sits before and after
 * the layer.
 *
 *   gdn_prefill     the delta rule over packed prompts, in chunks
 *   gdn_decode      the delta rule over one token per sequence
 *   gdn_add_norm    residual sum and RMS norm before a block, optionally with
 *                   the RMS norm after the previous block
 *   gdn_gated_norm  RMS norm of every head's output times its gate
 *   gdn_linear      matrix product with bias, activation, scale and residual
 *
 * Conventions of gdn_tree.h hold (device pointers, caller-owned buffers, no
 * allocation, no synchronisation, host argument checks before any HIP call,
 * status codes, gdn_last_error, stream order).  In addition:
 *  - Base pointers are 16-byte aligned (rows of the norms: aligned to their
 *    elements); workspaces 256-byte aligned.
 *  - A "stride" is the distance in ELEMENTS between two consecutive rows
 *    (tokens); what one row holds is dense.  An input's stride may be any
 *    value >= 0 (0: every row is the same); an output's is at least the row.
 *  - dtypes are gdn_dtype codes.
 *  - Outputs must not overlap inputs except where an argument says so.
 *  - Non-finite inputs propagate to the outputs that depend on them.
 *  - Every call is deterministic: no sum depends on the order in which
 *    workgroups run.
 */
#ifndef GDN_LAYER_H
#define GDN_LAYER_H

#include "gdn_tree.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * The delta rule over sequences.  For every token t of a sequence, in order,
 * and every value head (which reads key head h / (H_v / H_k)),
 *
 *     S <- exp(g_t) S (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,
 *     o_t = q_scale * S q_t                  (after token t's own update),
 *
 * the recurrence of gdn_tree_verify along a chain.  With qk_l2norm != 0,
 * q_t and k_t stand for q_t / sqrt(|q_t|^2 + l2_eps) and the same of k_t.
 * The range stated in gdn_tree.h (beta in [0, 1], |k|^2 <= 2 after the
 * norm) applies.
 *
 * States live in a pool S [n_slots][H_v][d_v][d_k] fp32 and are updated in
 * place: sequence b uses entry slot[b] (b itself if slot is NULL).  Two
 * sequences of one call must not share an entry.
 * ------------------------------------------------------------------------ */
typedef struct {
    int32_t B;         /* sequences, at most 65535; B H_v at most 2^24           */
    int32_t T;         /* tokens of all sequences together (gdn_decode: ignored) */
    int32_t H_k;       /* key/query heads                                        */
    int32_t H_v;       /* value heads (a multiple of H_k, at most 65535; H_v d_v
                          at most GDN_MAX_SEQ_STRIDE)                            */
    int32_t d_k;       /* key dimension, 64 or 128                               */
    int32_t d_v;       /* value dimension, 64 or 128                             */
    int32_t qkv_dtype; /* gdn_dtype of q, k, v                                   */
    int32_t o_dtype;   /* gdn_dtype of o                                         */
    int32_t n_slots;   /* entries of the state pool                              */
    int32_t qk_l2norm; /* 1: q and k are L2-normalised by the operator           */
    float q_scale;     /* factor on the output                                   */
    float l2_eps;      /* epsilon of the L2 norm, >= 0 (0: a zero vector is 0 / 0) */
    int64_t q_stride;  /* elements between tokens of q: a multiple of 16 bytes,
                          at most GDN_MAX_SEQ_STRIDE                             */
    int64_t k_stride;  /* the same of k                                          */
    int64_t v_stride;  /* the same of v                                          */
} gdn_seq_dims;
#define GDN_MAX_SEQ_STRIDE (1 << 24)

/* Bytes of device workspace gdn_prefill needs for `dims` (a multiple of 256;
 * 0 where none is needed or dims is NULL). */
size_t gdn_prefill_workspace_bytes(const gdn_seq_dims* dims);

/* Runs B packed sequences: sequence b owns tokens [cu_seqlens[b],
 * cu_seqlens[b + 1]), possibly none (its state is then only initialised).
 *   q, k       [T][H_k][d_k]  rows q_stride, k_stride apart
 *   v          [T][H_v][d_v]  rows v_stride apart
 *   g, beta    [T][H_v]       fp32 log-decay and write strength
 *   cu_seqlens [B + 1]        int32, device, non-decreasing, in [0, T]
 *   slot       [B]            int32, device, or NULL.  Outside [0, n_slots):
 *                             the sequence starts from a zero state and its
 *                             final state is not kept
 *   has_state  [B]            int32, device, or NULL (all 1).  0: the
 *                             sequence starts from a zero state; otherwise
 *                             from its pool entry
 *   S          the pool, in place; may be NULL if n_slots == 0
 *   o          [T][H_v][d_v]  o_dtype, dense
 *   seq_status [B]            int32, written, or NULL: 0, or GDN_ERR_SHAPE
 *                             for a sequence whose cu_seqlens entries are
 *                             not 0 <= start <= end <= T (it is run as empty;
 *                             the others are right all the same, if slower, and
 *                             a token of two of them holds the output of either)
 * Tokens that no sequence owns are not written. */
gdn_status gdn_prefill(const gdn_seq_dims* dims, const void* q, const void* k, const void* v, const float* g,
                       const float* beta, const int32_t* cu_seqlens, const int32_t* slot, const int32_t* has_state,
                       float* S, void* o, int32_t* seq_status, void* workspace, size_t workspace_bytes,
                       hipStream_t stream);

/* One token per sequence: q, k [B][H_k][d_k], v [B][H_v][d_v], g, beta
 * [B][H_v], o [B][H_v][d_v] dense.  A row whose slot[b] is outside
 * [0, n_slots) is idle: no state is touched and its o is zero. */
gdn_status gdn_decode(const gdn_seq_dims* dims, const void* q, const void* k, const void* v, const float* g,
                      const float* beta, const int32_t* slot, float* S, void* o, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Norms.  rms(a) = a / sqrt(mean(a^2) + eps) over the row; all in fp32.
 * ------------------------------------------------------------------------ */
typedef struct {
    int32_t T;          /* rows                                       */
    int32_t D;          /* elements of a row, 1 .. GDN_NORM_MAX_D     */
    int32_t x_dtype;    /* the block's output                         */
    int32_t res_dtype;  /* residual and h                             */
    int32_t y_dtype;    /* the normed output                          */
    float scale;        /* residual scale                             */
    float eps;          /* >= 0                                       */
    float weight_offset; /* added to weight and post_weight (1 for weights stored around zero) */
    int64_t x_stride, res_stride, h_stride, y_stride;
} gdn_add_norm_dims;
#define GDN_NORM_MAX_D 16384

/*     p = post_weight ? rms(x) * (post_weight + weight_offset) : x
 *     h = residual + scale * (chan_scale ? chan_scale * p : p)
 *     y = rms(h) * (weight + weight_offset)
 *   x           [T][D] x_dtype
 *   residual    [T][D] res_dtype, or NULL (zero)
 *   weight, post_weight, chan_scale [D] fp32; the last two may be NULL
 *   h           [T][D] res_dtype, written; may be exactly `residual` (same
 *               pointer and stride); may be NULL
 *   y           [T][D] y_dtype, written; formed from the unrounded h */
gdn_status gdn_add_norm(const gdn_add_norm_dims* dims, const void* x, const void* residual, const float* weight,
                        const float* post_weight, const float* chan_scale, void* h, void* y, hipStream_t stream);

typedef enum { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1, GDN_ACT_GELU = 2, GDN_ACT_SIGMOID = 3 } gdn_act;

typedef struct {
    int32_t T;       /* tokens                               */
    int32_t H;       /* heads                                */
    int32_t d;       /* elements of a head, 1 .. GDN_NORM_MAX_D */
    int32_t o_dtype; /* the layer's output                   */
    int32_t z_dtype; /* the gate                             */
    int32_t y_dtype;
    int32_t gate;    /* GDN_ACT_SILU or GDN_ACT_SIGMOID      */
    float eps;       /* >= 0                                 */
    int64_t o_stride, z_stride, y_stride; /* between tokens  */
} gdn_gated_norm_dims;

/* y[t][h] = rms(o[t][h]) * weight * gate(z[t][h]), rms over the d elements
 * of the head; o, z, y [T][H][d], weight [d] fp32.  y may be exactly o or z
 * (same pointer, stride and dtype). */
gdn_status gdn_gated_norm(const gdn_gated_norm_dims* dims, const void* o, const void* z, const float* weight,
                          void* y, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Projections: y = residual + scale * act(x w^T + bias), accumulated in fp32
 * and rounded once.  act: none, silu a/(1+e^-a), gelu a(1+erf(a/sqrt 2))/2,
 * sigmoid.
 * ------------------------------------------------------------------------ */
typedef struct {
    int32_t M, N, K;   /* rows, outputs, inputs; each >= 0 (K == 0: x w^T is zero) */
    int32_t res_dtype;
    int32_t y_dtype;
    int32_t act;       /* gdn_act */
    float scale;
    int64_t x_stride, w_stride, res_stride, y_stride;
} gdn_linear_dims;

/* Bytes of device workspace gdn_linear needs for `dims` (a multiple of 256;
 * 0 where none is needed or dims is NULL). */
size_t gdn_linear_workspace_bytes(const gdn_linear_dims* dims);

/*   x        [M][K] bf16
 *   w        [N][K] bf16
 *   bias     [N] fp32, or NULL
 *   residual [M][N] res_dtype, or NULL; may be exactly y (same pointer,
 *            stride and dtype)
 *   y        [M][N] y_dtype, written */
gdn_status gdn_linear(const gdn_linear_dims* dims, const void* x, const void* w, const float* bias,
                      const void* residual, void* y, void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LAYER_H */
