/*
 * gdn_attn.h -- C ABI of the softmax attention layers that stand between the
 * Gated DeltaNet layers of a model, over a paged cache of keys and values.
 * The steps are those of gdn_layer.h and gdn_tree.h: prompts, single tokens,
 * the verification of a whole proposal tree, and the commit of its accepted
 * path.
 *
 *   gdn_kv_append     norm and rotation of new queries and keys; keys and
 *                     values into the cache
 *   gdn_attn_prefill  packed prompts (or chunks of them) over the cache
 *   gdn_attn_decode   one token per sequence over the cache
 *   gdn_attn_verify   every node of a tree over the prefix and its ancestors
 *   gdn_kv_commit     the accepted path's keys and values move to the end of
 *                     the prefix, in all layers' caches
 *
 * Conventions of gdn_tree.h and gdn_layer.h hold (device pointers,
 * caller-owned buffers, no allocation, no synchronisation, host argument
 * checks before any HIP call, status codes, gdn_last_error, stream order,
 * strides in elements, deterministic results).  In addition:
 *  - A sequence's tokens 0, 1, ... lie in the pages of its row of `table`:
 *    token t in row t % page_size of page table[b][t / page_size].  Entries
 *    of pages that no token of the call lies in are not read.
 *  - Tokens on pages outside [0, n_pages) are left out, as if masked, and
 *    lengths are cut to [0, max_pages page_size]; seq_status reports both.
 *  - A query that no key is visible to gets an output of zero.
 *  - Keys and values that a query may not see (behind its sequence's end, on
 *    other branches of a tree, later in a prompt) have no influence on its
 *    output, whatever they hold, infinities and NaN included.
 *    Of those that it sees, a score of NaN or +infinity makes the query's
 *    output NaN, one of -infinity is a weight of zero (a query that sees no
 *    other gets zero, too), and a value that is not finite makes its element
 *    of the output infinite or NaN.
 *  - A workspace is one call's until that call has run: calls that may overlap
 *    (on two streams, or graphs replayed at once) need one each.
 *  - Scores, maxima and sums of the softmax and all accumulations are fp32.
 *    For the product with the values a weight is rounded: to two bf16 (16 bits
 *    together) by gdn_attn_decode, to one (off by 2^-8 of the weight at most)
 *    by gdn_attn_prefill and gdn_attn_verify, where the sum is that of the
 *    rounded weights.
 */
#ifndef GDN_ATTN_H
#define GDN_ATTN_H

#include "gdn_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of a cache beside GDN_BF16: 8-bit floats with 4 bits of
 * exponent and 3 of mantissa (OCP E4M3, no infinities, largest value 448). */
#define GDN_E4M3 2

/* One layer's cache: pools of pages of keys and of values.  Key j of head h
 * of row r of page p lies at k + p k_page_stride + r k_row_stride +
 * h k_head_stride + j, a value likewise; the d elements of a head are dense.
 * The strides are in elements, >= 0 and multiples of 16 bytes, those of rows
 * at most GDN_MAX_SEQ_STRIDE; any order of pages, rows and heads can be
 * described, also keys and values in one pool.
 * No two (page, row, head) may share memory in a call that writes. */
typedef struct {
    void* k;              /* 16-byte aligned                                     */
    void* v;
    const float* k_scale; /* [H_kv], device; what is stored stands for itself    */
    const float* v_scale; /*   times its head's scale (> 0, finite). NULL: 1     */
    int32_t n_pages;      /* pages of a pool, at least 1                         */
    int32_t page_size;    /* tokens of a page: a power of two up to 65536;
                             n_pages page_size at most 2^31 - 1                  */
    int32_t H_kv;         /* key and value heads, at most 65535                  */
    int32_t d;            /* elements of a head: 64, 128 or 256                  */
    int32_t dtype;        /* GDN_BF16 or GDN_E4M3                                */
    int32_t reserved;     /* 0                                                   */
    int64_t k_page_stride, k_row_stride, k_head_stride;
    int64_t v_page_stride, v_row_stride, v_head_stride;
} gdn_kv_cache;

typedef struct {
    int32_t T;             /* tokens                                              */
    int32_t H_q;           /* query heads; 0: keys and values only                */
    int32_t in_dtype;      /* q, k, v: GDN_BF16 or GDN_F32                        */
    int32_t rot;           /* elements of a head that are rotated: even, 0 .. d   */
    int32_t interleaved;   /* 1: pairs (x[2i], x[2i+1]); 0: (x[i], x[i + rot/2])  */
    float eps;             /* of the norms, >= 0                                  */
    float weight_offset;   /* added to q_weight and k_weight                      */
    int32_t reserved;      /* 0                                                   */
    int64_t q_stride, q_head_stride; /* between tokens, between heads             */
    int64_t k_stride, k_head_stride;
    int64_t v_stride, v_head_stride;
} gdn_kv_append_dims;

/* For every token t and head of q and k, in fp32:
 *     x <- x / sqrt(mean(x^2) + eps) * (weight + weight_offset)   with a weight
 *     pair i of the first rot elements turns by position[t] inv_freq[i]:
 *         (a, b) <- (a cos - b sin, b cos + a sin)
 * and q goes to q_out, k and v to row slot[t] % page_size of page
 * slot[t] / page_size, divided by their head's scale if there is one, rounded
 * once to nearest even (GDN_E4M3: clamped to +-448 first; infinities and NaN
 * become NaN).
 *   q, k, v   [T][heads][d] in_dtype, rows aligned to their elements
 *   q_weight, k_weight [d] fp32, or NULL (no norm)
 *   inv_freq  [rot / 2] fp32; the angle is formed in fp64
 *   position  [T] int32; may be NULL if rot == 0
 *   slot      [T] int32; outside [0, n_pages page_size): the token's k and v
 *             are not stored (its q_out is written).  No two tokens of a call
 *             may have the same slot inside
 *   q_out     [T][H_q][d] bf16, dense; may be exactly q where q is bf16 and
 *             dense.  q and q_out may be NULL if H_q == 0 */
gdn_status gdn_kv_append(const gdn_kv_append_dims* dims, const gdn_kv_cache* cache, const void* q, const void* k,
                         const void* v, const float* q_weight, const float* k_weight, const float* inv_freq,
                         const int32_t* position, const int32_t* slot, void* q_out, hipStream_t stream);

typedef struct {
    int32_t B;            /* sequences, at most 65535                                 */
    int32_t T;            /* prefill: rows of q; verify: tree nodes N of a sequence;
                             decode: ignored.  Rows of q times H_q at most 2^31 - 256 */
    int32_t H_q;          /* query heads, a multiple of H_kv: head h reads key head
                             h / (H_q / H_kv)                                         */
    int32_t max_pages;    /* entries of a row of table; max_pages page_size at most
                             2^30                                                     */
    float scale;          /* factor on the scores, >= 0 and finite                    */
    int32_t reserved;     /* 0                                                        */
    int64_t q_stride;     /* between tokens of q (a multiple of 8); heads are dense   */
    int64_t gate_stride;  /* between tokens of the gate                               */
    int64_t gate_head_stride; /* between its heads                                    */
    int64_t table_stride; /* between sequences of table                               */
} gdn_attn_dims;

/* Bytes of device workspace the calls below need (a multiple of 256; 0 where
 * none is needed or an argument is NULL or out of range).  The workspace
 * holds nothing between calls.  One of n > 0 bytes serves every call whose
 * sizes are not greater (B, max_pages; T) and otherwise the same; for a tree of
 * fewer nodes than it was asked for, the keys may then be divided into fewer
 * parts.  Where no workspace is needed for a large tree, one may be for a
 * smaller. */
size_t gdn_attn_prefill_workspace_bytes(const gdn_attn_dims* dims, const gdn_kv_cache* cache);
size_t gdn_attn_decode_workspace_bytes(const gdn_attn_dims* dims, const gdn_kv_cache* cache);
size_t gdn_attn_verify_workspace_bytes(const gdn_attn_dims* dims, const gdn_kv_cache* cache);

/* o = softmax(scale q k^T) v over the keys visible to the query, times
 * sigmoid(gate) if there is a gate, rounded once to bf16.  Common arguments:
 *   q      bf16, rows 16-byte aligned
 *   table  [B][max_pages] int32
 *   length [B] int32
 *   gate   bf16, in q's shape, aligned to its elements, or NULL
 *   o      bf16, in q's shape, dense; may not be q
 *   seq_status [B] int32, written, or NULL: 0, or GDN_ERR_SHAPE for a
 *          sequence whose length, page numbers or cu_seqlens are out of range
 */

/* One token per sequence: q, o [B][H_q][d]; the query sees tokens
 * 0 .. length[b] - 1 (its own, appended before, being the last). */
gdn_status gdn_attn_decode(const gdn_attn_dims* dims, const gdn_kv_cache* cache, const void* q, const int32_t* table,
                           const int32_t* length, const void* gate, void* o, int32_t* seq_status, void* workspace,
                           size_t workspace_bytes, hipStream_t stream);

/* Packed sequences: q, o [T][H_q][d].  Rows cu_seqlens[b] .. cu_seqlens[b+1] - 1
 * (n of them, possibly none) are the last n of the length[b] tokens of
 * sequence b, and see the tokens up to their own: row i sees tokens
 * 0 .. length[b] - n + i.  A sequence whose cu_seqlens entries are not
 * 0 <= start <= end <= T is run as empty.  Rows that no sequence owns are not
 * written.
 *   cu_seqlens [B + 1] int32, non-decreasing, in [0, T] */
gdn_status gdn_attn_prefill(const gdn_attn_dims* dims, const gdn_kv_cache* cache, const void* q,
                            const int32_t* cu_seqlens, const int32_t* table, const int32_t* length, const void* gate,
                            void* o, int32_t* seq_status, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Trees of N = dims->T <= GDN_ATTN_MAX_N nodes: q, o [B][N][H_q][d] (token
 * b N + i is node i).  The cache holds the prefix, tokens 0 .. length[b] - 1,
 * and node i as token length[b] + i.  Node i sees the prefix and the nodes
 * whose bits are set in anc[b][i].
 *   anc [B][N][ceil(N / 32)] uint32, as written by gdn_tree_ancestors (bits
 *       from N on are ignored) */
#define GDN_ATTN_MAX_N 256
gdn_status gdn_attn_verify(const gdn_attn_dims* dims, const gdn_kv_cache* cache, const void* q, const uint32_t* anc,
                           const int32_t* table, const int32_t* length, const void* gate, void* o, int32_t* seq_status,
                           void* workspace, size_t workspace_bytes, hipStream_t stream);

typedef struct {
    int32_t B;            /* sequences, at most 65535   */
    int32_t N;            /* tree nodes, 0 .. GDN_ATTN_MAX_N */
    int32_t max_pages;    /* as in gdn_attn_dims        */
    int32_t reserved;     /* 0                          */
    int64_t table_stride;
} gdn_kv_commit_dims;

/* After the verify of a tree: the keys and values of the accepted node's path
 * (the set bits of anc[b][accepted[b]], in order) move from tokens
 * length[b] + node to tokens length[b], length[b] + 1, ..., in each of
 * `n_caches` caches that differ in k and v only.
 * No two sequences of a call may share a page that rows move to.
 *   caches     host array; k or v of an earlier one in it moves once
 *   accepted   [B] int32, in [-1, N - 1]; -1 (or outside) moves nothing
 *   new_length [B] int32, written: length[b] + tokens of the path; not length
 *   seq_status [B] int32, written, or NULL: 0, GDN_ERR_ACCEPT for an accepted
 *              node out of range, GDN_ERR_SHAPE for a length or a page of the
 *              path out of range (rows on such pages are not moved) */
gdn_status gdn_kv_commit(const gdn_kv_commit_dims* dims, const gdn_kv_cache* caches, int32_t n_caches,
                         const uint32_t* anc, const int32_t* accepted, const int32_t* table, const int32_t* length,
                         int32_t* new_length, int32_t* seq_status, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ATTN_H */
