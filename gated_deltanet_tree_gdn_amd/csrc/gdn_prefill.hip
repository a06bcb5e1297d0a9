// gdn_prefill.hip -- the delta rule over packed prompts, in chunks of 64
// tokens (bf16 q/k/v).
//
// Inside a chunk that starts from the state S (d_v x d_k), with
// G_i = g_1 + .. + g_i, gamma_i = e^{G_i} and u_i = beta_i (v_i - alpha_i S_{i-1} k_i):
//
//     (I + A) U = diag(beta) (V - diag(gamma) K S^T),  A_ij = beta_i e^{G_i - G_j} k_i.k_j  (j < i)
//     O     = diag(gamma) Q S^T + M U,                 M_ij = e^{G_i - G_j} q_i.k_j         (j <= i)
//     S_new = gamma_64 S + sum_j e^{G_64 - G_j} u_j k_j^T.
//
// T = (I + A)^-1 diag(beta) and M do not depend on S, so two kernels run:
//  1. prep_kernel, parallel over (chunk, key head): T and M as MFMA operands,
//     and the chunk's scalars, into the workspace;
//  2. chain_kernel, one workgroup per (sequence, value head, slice of d_v):
//     the chunks in order with the state in registers.
// Rows of d_v are independent of each other, so slices need no exchange.
//
// Chunk slots: sequence b's chunks are numbered from cu[b] / 64 + b, which
// leaves every sequence room without a prefix sum over lengths (at most
// T / 64 + B slots) as long as the offsets do not decrease.  Where they do, slots
// may belong to two sequences or be taken for another's, so no sequence uses them:
// the first kernel's first workgroup looks at all offsets, and the second kernel then
// walks every sequence token by token.
//
// Precision: q, k and v are exact bf16 operands.  Every fp32 operand (S, R = V -
// gamma K S^T, the off-diagonal part of T, U, the decayed U, M) is split into three
// bf16 parts, 24 bits, and of a product of two such operands the six products of
// parts above 2^-24 of it are taken.  The diagonal of T acts in fp32.  Two parts for
// S, T, or M and U multiply the error by 5 to 200 where keys reach |k|^2 = 2 and
// nothing decays, and that of outputs of ordinary inputs by up to 20.
// Sums, states and the decay are fp32, G is fp64 (a difference G_i - G_j stays exact
// to fp32 however far the chunk has decayed), and so are the products that form T:
// near |k|^2 = 2 their terms are larger than T.  Relative error after 2000 tokens:
// states and fp32 outputs 2e-7 (3e-7 token by token in fp32); with |k|^2 = 2, beta
// = 1 and no decay up to 6e-6 (keys in a plane; 1e-6 token by token).
//
// Measured, H_k 16, H_v 32, d 128, bf16, half of the 13 states resumed: one of
// 16384 tokens 530 us (prep 97, chain 433), 13 of 7919 tokens in all 250 us.
// The inputs, outputs and states are 409 MB and 238 MB; at the rate of a copy
// (5.2 TB/s) that is 79 and 46 us.

#include <type_traits>

#include "gdn_layer_internal.h"
#include "gdn_layer_util.h"
#include "gdn_mfma.h"

namespace gdn {
namespace {

constexpr int kC = 64;  // tokens per chunk

// What prep_kernel hands to chain_kernel, all in the order in which a
// wavefront's lanes read it (16 bytes per lane, 1 KiB per fragment): T in parts, M
// in fp32 (the outputs have the time to split it, 20 us less of 560 for the long
// prompt; the chain has not, 30 us more).  Tokens
// of a 32-token step sit at k-slot j of lane group g as token
// 16 (j / 4) + 4 g + j % 4, the order in which accumulators hold rows, so that
// a product's result is the next product's operand without moving lanes.
struct PrepLayout {
    size_t t, m, sc, ordered, total;
};
constexpr int kScalars = 4 * kC + 4;  // floats per (slot, head), whole 16-byte pieces
// T and M: the (row tile, 32-token step) pairs that reach the lower triangle.
constexpr int kPairs = 6;
// bf16 parts of an fp32 operand.
constexpr int kParts = 3;
__host__ __device__ constexpr int pair_at(int tile, int step) { return tile < 2 ? tile : 2 * tile - 2 + step; }

__host__ inline PrepLayout prep_layout(const gdn_seq_dims& d) {
    // one slot more than can be used: the chain loads a chunk ahead
    const size_t slots = size_t(d.T) / kC + d.B + 1, heads = slots * d.H_v;
    PrepLayout l;
    l.t = 0;
    l.m = l.t + heads * kPairs * kParts * 1024;
    l.sc = l.m + heads * kPairs * 2 * 1024;
    l.ordered = l.sc + heads * kScalars * sizeof(float);
    l.total = (l.ordered + sizeof(int) + 255) & ~size_t(255);
    return l;
}

struct ChunkArgs {
    SeqArgs s;
    uint4* t;
    uint4* m;
    float* sc;     // 4 x 64: gamma |k|^-1, beta, e^{G_64 - G} |k|^-1 and scale gamma |q|^-1 of every token (norms
                   // 1 unless asked for), the first NaN where k, g or beta is not finite; then gamma_64
    int* ordered;  // whether cu is 0 <= cu[0] <= .. <= cu[B] <= T
    int slots;
};

struct Range {
    int64_t start;
    int len;
    bool ok;
};
__device__ __forceinline__ Range seq_range(const SeqArgs& a, int b) {
    const int64_t s = a.cu[b], e = a.cu[b + 1];
    const bool ok = 0 <= s && s <= e && e <= a.d.T;
    return {ok ? s : 0, ok ? int(e - s) : 0, ok};
}

__device__ __forceinline__ int slot_base(const SeqArgs& a, int b) {
    const int s = a.cu[b];
    return (s < 0 ? 0 : s > a.d.T ? a.d.T : s) / kC + b;
}

// The sequence that a chunk slot belongs to: the last b with base(b) <= slot,
// 64 candidates at a time.
__device__ __forceinline__ int find_seq(const SeqArgs& a, int slot) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = a.d.B;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int b = lo + lane * step;
        const bool le = lane * step < n && slot_base(a, b) <= slot;
        const int last = 63 - __builtin_clzll(__ballot(le) | 1ull);
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

// The sequence with the r-th most tokens of up to 64 (the lower index first
// among equals): workgroups start in order of their number, and a long
// sequence that starts late is what the others wait for.  More sequences than
// that are taken as they come.
__device__ __forceinline__ int longest_seq(const SeqArgs& a, int r) {
    const int B = a.d.B;
    if (B > 64) return r;
    const int lane = threadIdx.x & 63;
    const int len = lane < B ? seq_range(a, lane).len : -1;
    int rank = 0;
    for (int j = 0; j < B; ++j) {
        const int other = __builtin_amdgcn_readlane(len, j);
        rank += other > len || (other == len && j < lane);
    }
    return __builtin_ctzll(__ballot(lane < B && rank == r));
}

// Accumulator r of lane group g is row 4 r + g of the product; in the other MFMAs
// here it is row 4 g + r.  The operand whose rows those are takes them in the order
// of row_of (column by column of a 4 x 4 arrangement), so that both agree.
typedef double f64x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ f64x4 mfma_f64(double a, double b, const f64x4& c) {
    return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ int row_of(int i) { return 4 * (i & 3) + (i >> 2); }

// Four accumulators as packed bf16 parts, x = part[0] + part[1] + part[2], each
// rounded to nearest; in pairs, as the conversions come.
__device__ __forceinline__ uint2 take4(f32x4& x) {  // the leading part; x keeps the rest
    const uint2 part = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
    x -= f32x4{bf16_lo(part.x), bf16_hi(part.x), bf16_lo(part.y), bf16_hi(part.y)};
    return part;
}
__device__ __forceinline__ void split4(f32x4 x, uint2 (&part)[kParts]) {
    part[0] = take4(x);
    part[1] = take4(x);
    part[2] = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}
__device__ __forceinline__ uint4 join(const uint2& a, const uint2& b) { return make_uint4(a.x, a.y, b.x, b.y); }

// Adds a b of operands in three parts: the six products above 2^-24 of it, by
// size into three sums.
__device__ __forceinline__ void mfma_parts(const bf16x8 (&a)[kParts], const bf16x8 (&b)[kParts], f32x4 (&sum)[kParts]) {
    sum[2] = mfma(a[2], b[0], sum[2]);
    sum[1] = mfma(a[1], b[0], sum[1]);
    sum[0] = mfma(a[0], b[0], sum[0]);
    sum[2] = mfma(a[1], b[1], sum[2]);
    sum[1] = mfma(a[0], b[1], sum[1]);
    sum[2] = mfma(a[0], b[2], sum[2]);
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __builtin_inff(); }

// Orders LDS between the lanes of one wavefront.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// ----------------------------------------------------------------------------
// 1. per (chunk, key head)
// ----------------------------------------------------------------------------

constexpr int kGramLd = 68;  // row stride of the Gram matrix in LDS: rows 4 apart fall on different banks
constexpr int kTriLd = 20;   // row stride of a 16 x 16 block

// e^{x} for a difference of log-decays held times log2(e).
__device__ __forceinline__ float exp_diff(double hi, double lo) {
    return __builtin_amdgcn_exp2f(static_cast<float>(hi - lo));
}

// Four wavefronts: the Gram matrices on MFMA once per key head; then two value
// heads at a time, a wavefront each half of T's row blocks: 16 x 16 diagonal
// blocks by substitution (a column per lane), the blocks below them by fp64 MFMA
// (in fp32 their rounding is most of the error where |k|^2 is 2).  Bound by memory: it
// writes T and M, 480 bytes per (token, value head), and reads q and k; 16384
// tokens, H_v 32: 395 MB in 97 us, 4.1 TB/s.
template <int DK>
__global__ void __launch_bounds__(256, 3) prep_kernel(ChunkArgs c) {
    constexpr int KS = DK / 32;
    constexpr int kKl = 4 * KS * 64 * 16, kTri = 4 * 4 * 16 * kTriLd * 4;
    // K rows as fragments [token tile][step][lane]; then per wavefront the
    // diagonal blocks of A and of T
    __shared__ __align__(16) char buf[kKl > kTri ? kKl : kTri];
    __shared__ __align__(16) float gram[kC * kGramLd];  // |k_i|^-1 |k_j|^-1 k_i.k_j, j's tile <= i's
    __shared__ double gcum[2][kC];                      // G log2(e) of two value heads
    __shared__ __align__(16) float bet[2][kC];
    __shared__ __align__(16) float rks[kC], rqs[kC];
    __shared__ unsigned badk[2];  // tokens whose k is not finite, a bit each
    const SeqArgs& a = c.s;
    const gdn_seq_dims& d = a.d;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, g = lane >> 4;
    if (block_id() == 0) {
        bool ok = true;
        for (int i = threadIdx.x; i <= d.B; i += 256) ok &= 0 <= a.cu[i] && a.cu[i] <= (i < d.B ? a.cu[i + 1] : d.T);
        ok = __syncthreads_and(ok);
        if (threadIdx.x == 0) *c.ordered = ok;
        return;
    }
    // The key heads of a slot run on one XCD one after the other: rows of g and
    // beta hold all heads, so its L2 reads them once.
    const int id = int(block_id()) - 1, j8 = id >> 3, slot = j8 / d.H_k * 8 + (id & 7), hk = j8 % d.H_k;
    if (slot >= c.slots) return;
    const int b = find_seq(a, slot);
    const Range seq = seq_range(a, b);
    const int ch = slot - slot_base(a, b);
    if (ch < 0 || ch * kC >= seq.len) return;
    const int64_t t0 = seq.start + int64_t(ch) * kC;
    const int n = min(kC, seq.len - ch * kC);
    auto kl = [&](int tile, int step, int l) { return reinterpret_cast<uint4*>(buf) + (tile * KS + step) * 64 + l; };

    // K and Q rows of token tile w: lane (row col, elements 32 s + 8 g ..)
    const int row = 16 * w + col;
    const bool in = row < n;
    const int64_t tr = t0 + (in ? row : 0);
    const uint16_t* kp = static_cast<const uint16_t*>(a.k) + tr * d.k_stride + int64_t(hk) * DK + 8 * g;
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + tr * d.q_stride + int64_t(hk) * DK + 8 * g;
    uint4 kf[KS], qf[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        kf[s] = *reinterpret_cast<const uint4*>(kp + 32 * s);
        qf[s] = *reinterpret_cast<const uint4*>(qp + 32 * s);
    }
    // the gates of the first two value heads, a token per lane
    const int group = d.H_v / d.H_k;
    const int64_t gi = (t0 + min(lane, n - 1)) * d.H_v + hk * group;
    float gv = a.g[gi + min(w >> 1, group - 1)], bv = a.beta[gi + min(w >> 1, group - 1)];
    if (threadIdx.x < 2) badk[threadIdx.x] = 0;
    float kk = 0.0f, qq = 0.0f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const uint32_t ku[4] = {kf[s].x, kf[s].y, kf[s].z, kf[s].w}, qu[4] = {qf[s].x, qf[s].y, qf[s].z, qf[s].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float k0 = bf16_lo(ku[j]), k1 = bf16_hi(ku[j]), q0 = bf16_lo(qu[j]), q1 = bf16_hi(qu[j]);
            kk += k0 * k0 + k1 * k1;
            qq += q0 * q0 + q1 * q1;
        }
    }
    kk += __shfl_xor(kk, 16);
    kk += __shfl_xor(kk, 32);
    qq += __shfl_xor(qq, 16);
    qq += __shfl_xor(qq, 32);
    __syncthreads();
    // a k that is not finite, or whose inverse norm is not (k = 0 without an epsilon),
    // is taken out of the chunk here and its token marked
    const float rk = d.qk_l2norm ? 1.0f / sqrtf(kk + d.l2_eps) : 1.0f;
    const bool kbad = in && !(finite(kk) && finite(rk));
    if (kbad && g == 0) atomicOr(&badk[row >> 5], 1u << (row & 31));
    if (!in || kbad)
#pragma unroll
        for (int s = 0; s < KS; ++s) kf[s] = make_uint4(0, 0, 0, 0);
    if (!in)
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[s] = make_uint4(0, 0, 0, 0);
    const float rq = d.q_scale * (d.qk_l2norm ? 1.0f / sqrtf(qq + d.l2_eps) : 1.0f);
    if (g == 0) {
        rks[row] = in && !kbad ? rk : 0.0f;
        rqs[row] = in ? rq : 0.0f;
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) *kl(w, s, lane) = kf[s];
    __syncthreads();

    // Transposed products: accumulators hold column i = 16 w + col, rows
    // j = 16 jt + 4 g + r.
    f32x4 qk[4];
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
        f32x4 kkt = {0.0f, 0.0f, 0.0f, 0.0f};
        qk[jt] = kkt;
        if (jt <= w) {
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const bf16x8 kj = __builtin_bit_cast(bf16x8, *kl(jt, s, lane));
                kkt = mfma(kj, __builtin_bit_cast(bf16x8, kf[s]), kkt);
                qk[jt] = mfma(kj, __builtin_bit_cast(bf16x8, qf[s]), qk[jt]);
            }
            const float4 rj = *reinterpret_cast<const float4*>(&rks[16 * jt + 4 * g]);
            const float rr[4] = {rj.x, rj.y, rj.z, rj.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                kkt[r] *= rks[row] * rr[r];
                qk[jt][r] *= rqs[row] * rr[r];
            }
            *reinterpret_cast<f32x4*>(&gram[row * kGramLd + 16 * jt + 4 * g]) = kkt;
        }
    }

    // The value heads of this key head, two at a time, two wavefronts each:
    // both invert the diagonal blocks, the first then forms rows 0 .. 47 of T,
    // the second rows 48 .. 63.
    __syncthreads();
    float(*tri)[16][kTriLd] = reinterpret_cast<float(*)[16][kTriLd]>(buf + w * (kTri / 4));
    const int hw = w >> 1, part = w & 1;
    for (int h0 = 0; h0 < group; h0 += 2) {
        const int nh = min(2, group - h0);
        if (hw < nh) {
            const int h = hk * group + h0 + hw;
            const int64_t sh = int64_t(slot) * d.H_v + h;
            if (h0 > 0) {
                gv = a.g[gi + h0 + hw];
                bv = a.beta[gi + h0 + hw];
            }
            // G and the scalars: lane = token
            if (lane >= n) gv = bv = 0.0f;
            const bool gbad = !(gv < __builtin_inff()) || !finite(bv);
            const unsigned long long bad = (static_cast<unsigned long long>(badk[1]) << 32 | badk[0]) | __ballot(gbad);
            if (bad >> lane & 1) bv = 0.0f;
            // exp(g) is zero below -104, so larger decays would only cost precision
            gv = gbad ? 0.0f : fmaxf(gv, -104.0f);
            double G = gv * 1.4426950408889634;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const double y = __shfl_up(G, o);
                if (lane >= o) G += y;
            }
            const double G63 = __shfl(G, 63);
            if (part == 0) {
                gcum[hw][lane] = G;
                bet[hw][lane] = bv;
                const float gam = __builtin_amdgcn_exp2f(static_cast<float>(G));
                float* sc = c.sc + sh * kScalars + lane;
                sc[0] = bad >> lane & 1 ? __builtin_nanf("") : gam * rks[lane];
                sc[kC] = bv;
                sc[2 * kC] = exp_diff(G63, G) * rks[lane];
                sc[3 * kC] = gam * rqs[lane];
                if (lane == 0) sc[4 * kC] = __builtin_amdgcn_exp2f(static_cast<float>(G63));
            }
        }
        __syncthreads();
        if (hw < nh) {
            const int64_t sh = int64_t(slot) * d.H_v + hk * group + h0 + hw;
            const double* G = gcum[hw];
            const float* be = bet[hw];
            // diagonal blocks of A: lane group g = block, col = column
            const double Gc = G[16 * g + col];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = 16 * g + i;
                tri[g][i][col] = i > col ? be[r] * exp_diff(G[r], Gc) * gram[r * kGramLd + 16 * g + col] : 0.0f;
            }
            wave_lds_fence();
            // their inverses by forward substitution, one column per lane
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s0 = i == col ? 1.0f : 0.0f, s1 = 0.0f;
#pragma unroll
                for (int m = 0; m < i; m += 4) {
                    const float4 am = *reinterpret_cast<const float4*>(&tri[g][i][m]);
                    s0 -= am.x * x[m];
                    if (m + 1 < i) s1 -= am.y * x[m + 1];
                    if (m + 2 < i) s0 -= am.z * x[m + 2];
                    if (m + 3 < i) s1 -= am.w * x[m + 3];
                }
                x[i] = s0 + s1;
            }
            wave_lds_fence();
#pragma unroll
            for (int i = 0; i < 16; ++i) tri[g][i][col] = x[i];
            wave_lds_fence();
            // Row block i of T, transposed: X[j] = T_ij^T = -T_jj^T sum_m A_mj^T T_im^T
            // as accumulators (column = row of block i, rows = columns of block j);
            // then T diag(beta) without its diagonal as fragments of tile i's rows.
            uint4* tp = c.t + sh * kPairs * kParts * 64;
            auto row_block = [&](auto ii) {
                constexpr int i = ii.value;
                f64x4 X[i + 1];
#pragma unroll
                for (int r = 0; r < 4; ++r) X[i][r] = tri[i][col][4 * g + r];
                const int pc = row_of(col);
#pragma unroll
                for (int j = i - 1; j >= 0; --j) {
                    f64x4 acc = {0.0, 0.0, 0.0, 0.0}, out = acc;
                    const double Gj = G[16 * j + pc];
#pragma unroll
                    for (int m = j + 1; m <= i; ++m)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int tm = 16 * m + 4 * g + r;
                            acc = mfma_f64(be[tm] * exp_diff(G[tm], Gj) * gram[tm * kGramLd + 16 * j + pc], X[m][r], acc);
                        }
#pragma unroll
                    for (int r = 0; r < 4; ++r) out = mfma_f64(-tri[j][4 * g + r][pc], acc[r], out);
                    X[j] = out;
                }
#pragma unroll
                for (int s = 0; s <= i / 2; ++s) {
                    uint2 x[2][kParts];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int jt = 2 * s + half;
                        const f32x4 bj = *reinterpret_cast<const f32x4*>(&be[16 * jt + 4 * g]);
                        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
                        if (jt <= i)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                v[r] = jt < i || 4 * g + r < col ? static_cast<float>(X[jt < i ? jt : i][r]) * bj[r] : 0.0f;
                        split4(v, x[half]);
                    }
                    uint4* p = tp + pair_at(i, s) * kParts * 64 + lane;
#pragma unroll
                    for (int q = 0; q < kParts; ++q) p[64 * q] = join(x[0][q], x[1][q]);
                }
            };
            if (part == 0) {
                row_block(std::integral_constant<int, 0>());
                row_block(std::integral_constant<int, 1>());
                row_block(std::integral_constant<int, 2>());
            } else {
                row_block(std::integral_constant<int, 3>());
            }
        }
        // M of both heads: rows of token tile w
        for (int hh = 0; hh < nh; ++hh) {
            const int64_t sh = int64_t(slot) * d.H_v + hk * group + h0 + hh;
            const double Gi = gcum[hh][row];
            uint4* mp = c.m + sh * kPairs * 2 * 64;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (2 * s > w) continue;
                uint4* p = mp + pair_at(w, s) * 2 * 64 + lane;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int jt = 2 * s + half;
                    f32x4 v;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int tok = 16 * jt + 4 * g + r;
                        v[r] = tok <= row ? exp_diff(Gi, gcum[hh][tok]) * qk[jt][r] : 0.0f;
                    }
                    p[64 * half] = __builtin_bit_cast(uint4, v);
                }
            }
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------------------
// 2. per (sequence, value head, slice of d_v)
// ----------------------------------------------------------------------------

// A load from a uniform base and a lane's 32-bit byte offset.
template <typename T>
__device__ __forceinline__ T load_at(const void* base, uint32_t off) {
    return *reinterpret_cast<const T*>(static_cast<const char*>(base) + off);
}

// Four 16-bit elements of each lane, transposed over groups of 16 lanes.
__device__ __forceinline__ uint2 read_tr(const uint2* p) {
    typedef short s16x4v __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(
        uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4v*)(p)));
}

// Rows of K and Q go straight to LDS in the order of memory (a wavefront's load
// covers whole rows; loading the MFMA layout directly would touch 16 rows per
// 256 bytes) and are read from there as operands.  The 16-byte pieces of a row
// are permuted so that both reads below use all banks: a fragment (piece p of
// 16 rows) and a transposing read (4 adjacent pieces of 4 adjacent rows).
template <int DK>
__device__ __forceinline__ int piece_xor(int row) {
    return DK == 128 ? ((row >> 2) & 3) | (row & 3) << 2 : ((row >> 2) & 3) | (row >> 1 & 1) << 2;
}
template <int DK>
__device__ __forceinline__ int piece_at(int row, int p) {
    return row * (DK / 8) + (p ^ piece_xor<DK>(row));
}

// The 16 rows of one token tile: load number j brings slots 64 j .. 64 j + 63.
template <int DK>
struct TileRows {
    static constexpr int P = DK / 8, L = DK / 32;  // pieces per row, loads
    uint32_t off[L];                               // bytes
    // `left` > 0 rows exist from the chunk's first on; further ones repeat the last.
    __device__ __forceinline__ void rows(int64_t stride, int left, int tile, int lane) {
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int r = (64 * j + lane) / P;
            off[j] = (uint32_t(min(16 * tile + r, left - 1)) * uint32_t(stride) + 8 * (lane % P ^ piece_xor<DK>(r))) * 2;
        }
    }
    __device__ __forceinline__ void load(const uint16_t* base, uint4* tile_lds) const {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass rejects the 16-byte form
        // rows lie within 63 * 2^24 elements of the first
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base), 0, 0x7fffffff, 0x00027000);
#pragma unroll
        for (int j = 0; j < L; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)(tile_lds + 64 * j), 16,
                                                     off[j], 0, 0, 0);
#endif
    }
};

// LDS of one chain workgroup: operands of the products over the state and over
// tokens as [step][part][lane].
template <int DK>
struct ChainLds {
    uint4 K[2][4][16 * DK / 8];    // rows of this chunk's K and the next one's by token tile, pieces permuted
    uint4 Q[4][16 * DK / 8];       // rows of Q, each tile read by its own wavefront only
    uint4 S[DK / 32][kParts][64];  // state
    uint4 R[2][kParts][64];        // R
    uint4 D[2][kParts][64];        // decayed U
    f32x4 U[4][64];                // U in fp32, rows of token tile [i] as accumulated
    uint4 V[kC * 2];               // the chunk's rows of the slice's values
    float sc[kScalars];            // its scalars
    uint32_t marks[4];             // whether wavefront i's R has a value that is not finite
    uint8_t badrow[4][64];         // its rows, where marked
};

// The first row of the lane's column that is not finite; kC if none.
template <int DK>
__device__ __forceinline__ int first_bad(const ChainLds<DK>& l, int col) {
    for (int w = 0; w < 4; ++w)
        if (l.marks[w]) {
            int first = kC;
            for (int g = 0; g < 4; ++g) {
                const unsigned m = l.badrow[w][16 * g + col];
                if (m) first = min(first, 16 * w + 4 * g + __builtin_ctz(m));
            }
            if (first < kC) return first;
        }
    return kC;
}

// 16 state rows of one sequence token by token, 32 lanes to a row.
template <int DK>
__device__ __forceinline__ void walk_rows(const SeqArgs& a, int b, int hk, int h, int v0) {
    constexpr int E = DK / 32;
    const gdn_seq_dims& d = a.d;
    const int l = threadIdx.x & 31, row = v0 + (threadIdx.x >> 5);
    const Range seq = seq_range(a, b);
    if (a.seq_status && threadIdx.x == 0 && h == 0 && v0 == 0) a.seq_status[b] = seq.ok ? GDN_OK : GDN_ERR_SHAPE;
    const int pool = a.slot ? a.slot[b] : b;
    const bool keep = pool >= 0 && pool < d.n_slots;
    const bool resume = keep && (!a.has_state || a.has_state[b] != 0);
    float* Sp = keep ? a.S + ((int64_t(pool) * d.H_v + h) * d.d_v + row) * DK + E * l : nullptr;
    float s[E];
#pragma unroll
    for (int e = 0; e < E; ++e) s[e] = resume ? Sp[e] : 0.0f;
    for (int64_t t = seq.start; t < seq.start + seq.len; ++t) {
        float kk = 0.0f, qq = 0.0f, kq = 0.0f, sk = 0.0f, sq = 0.0f, k[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            k[e] = load1(a.k, GDN_BF16, t * d.k_stride + int64_t(hk) * DK + E * l + e);
            const float q = load1(a.q, GDN_BF16, t * d.q_stride + int64_t(hk) * DK + E * l + e);
            kk += k[e] * k[e];
            qq += q * q;
            kq += k[e] * q;
            sk += s[e] * k[e];
            sq += s[e] * q;
        }
        const float rk = d.qk_l2norm ? 1.0f / sqrtf(lane_sum<32>(kk) + d.l2_eps) : 1.0f;
        const float rq = d.q_scale * (d.qk_l2norm ? 1.0f / sqrtf(lane_sum<32>(qq) + d.l2_eps) : 1.0f);
        const float alpha = expf(a.g[t * d.H_v + h]), v = load1(a.v, GDN_BF16, t * d.v_stride + int64_t(h) * d.d_v + row);
        const float u = a.beta[t * d.H_v + h] * (v - alpha * (rk * lane_sum<32>(sk))) * rk;
        const float o = rq * (alpha * lane_sum<32>(sq) + u * lane_sum<32>(kq));
#pragma unroll
        for (int e = 0; e < E; ++e) s[e] = alpha * s[e] + u * k[e];
        if (l == 0) store1(a.o, d.o_dtype, (t * d.H_v + h) * d.d_v + row, o);
    }
    if (keep)
#pragma unroll
        for (int e = 0; e < E; ++e) Sp[e] = s[e];
}

// What bounds it: a chunk takes 1.7 us (3,600 clocks) of three dependent phases,
// each a chain of LDS reads (some 300 clocks), 12 MFMAs, the split of their
// sums and a barrier; LDS is busy for 2,000 of the clocks, a SIMD for 900 with
// MFMAs and 1,900 with the rest, most of it splits.  The outputs' M U, which splits
// M and U, outlasts the state update beside it by 700.  The chain cannot be cut
// along the sequence (S enters every chunk), so it is cut along d_v as finely as
// MFMA tiles allow.  With two parts per operand, one wavefront per 16 columns and no
// barriers took 840 us where this split took 353.
//
// Eight wavefronts: 0 .. 3 carry the state from chunk to chunk, 4 .. 7 form
// the outputs beside them.  Three barriers per chunk:
//   chain:  state operands | K S^T, R, K^T operands | U     | state update, next T, V
//   output:                | store, next K and Q    | Q S^T | M U, next M
// LDS bandwidth is what the phases compete for: the outputs read the state
// operands a phase after the chain does, and operands that do not depend on the
// chain are read outside its critical phases.
// Wavefront i of either kind owns token tile i (16 rows of the chunk); chain
// wavefront i also owns d_k / 4 elements of the state's rows.
//
// Vector memory instructions are dear too (16 clocks each for 1 KiB or less), so
// values and scalars go through LDS rather than to each lane from memory, and
// outputs are formed transposed: a lane then stores 4 adjacent values.
template <int DK>
__global__ void __launch_bounds__(512, 2) chain_kernel(ChunkArgs c) {
    constexpr int KS = DK / 32, TPW = DK / 64;
    __shared__ ChainLds<DK> l;
    const SeqArgs& a = c.s;
    const gdn_seq_dims& d = a.d;
    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave & 3;
    // Workgroups go to the 8 XCDs in turn: the slices and value heads of one
    // (sequence, key head) are numbered onto one XCD, whose L2 then serves
    // their common K, Q, K^T, T and M.
    const int group = d.H_v / d.H_k, slices = d.d_v / 16, per = group * slices;
    const int id = int(block_id()), j8 = id >> 3, item = (id & 7) + 8 * (j8 / per), part = j8 % per;
    if (item >= d.B * d.H_k) return;
    const int b = longest_seq(a, item / d.H_k), hk = item % d.H_k, h = hk * group + part / slices;
    const int v0 = part % slices * 16;
    if (!*c.ordered) return walk_rows<DK>(a, b, hk, h, v0);

    const Range seq = seq_range(a, b);
    const int base = slot_base(a, b), chunks = (seq.len + kC - 1) / kC;
    const int64_t sh0 = int64_t(base) * d.H_v + h;
    if (lane == 0 && wave < 4) l.marks[w] = 0;

    if (wave >= 4) {
        // ---- outputs ----
        if (chunks == 0) return;
        const uint16_t* qp = static_cast<const uint16_t*>(a.q) + seq.start * d.q_stride + int64_t(hk) * DK;
        const uint16_t* kp = static_cast<const uint16_t*>(a.k) + seq.start * d.k_stride + int64_t(hk) * DK;
        const uint4* mp = c.m + (sh0 * kPairs + pair_at(w, 0)) * 2 * 64;
        const int64_t q_step = kC * d.q_stride, k_step = kC * d.k_stride, m_step = int64_t(d.H_v) * kPairs * 2 * 64;
        const uint32_t ld = uint32_t(d.H_v) * d.d_v, o_off = (16 * w + col) * ld + 4 * g;
        int64_t o_at = (seq.start * d.H_v + h) * d.d_v + v0;
        auto run = [&](auto steps_of_tile) {
            constexpr int kSteps = steps_of_tile.value;  // 32-token steps up to token tile w
            uint4 mf[2 * kSteps], qf[KS];
            TileRows<DK> qr, kr;
            qr.rows(d.q_stride, seq.len, w, lane);
            kr.rows(d.k_stride, seq.len, w, lane);
            // The chunk that `left` tokens are left from on.  The loads are not behind
            // a branch (whose end would wait for them): past the sequence the last
            // chunk is loaded again.
            auto load_q = [&](int left) {
                if (left < kC && left > 0) qr.rows(d.q_stride, left, w, lane);
                qp += left > 0 ? q_step : 0;
                qr.load(qp - q_step, l.Q[w]);
            };
            auto load_k = [&](int left, int buffer) {
                if (left < kC && left > 0) kr.rows(d.k_stride, left, w, lane);
                kp += left > 0 ? k_step : 0;
                kr.load(kp - k_step, l.K[buffer][w]);
            };
            auto load_m = [&]() {
#pragma unroll
                for (int i = 0; i < 2 * kSteps; ++i) mf[i] = load_at<uint4>(mp + i * 64, lane * 16);
                mp += m_step;
            };
            load_k(seq.len, 0);
            load_q(seq.len);
            __builtin_amdgcn_sched_barrier(0);
            load_m();
            __builtin_amdgcn_sched_barrier(0);
            f32x4 O;  // transposed: column = token 16 w + col, rows = values 4 g + r
            int first = kC;
            bool poisoned = false;
            auto store = [&](int n) {
                if (poisoned)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (16 * w + col >= __shfl(first, 4 * g + r)) O[r] = __builtin_nanf("");
                if (16 * w + col < n) {
                    if (d.o_dtype == GDN_BF16)
                        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + o_at + o_off) =
                            make_uint2(pack_bf16(O[0], O[1]), pack_bf16(O[2], O[3]));
                    else
                        *reinterpret_cast<f32x4*>(static_cast<float*>(a.o) + o_at + o_off) = O;
                }
                o_at += int64_t(kC) * ld;
            };
            for (int ch = 0; ch < chunks; ++ch) {
                // state operands, values and scalars written; K and Q there, since only
                // the loads of M are younger
                loads_barrier<2 * kSteps>();
#pragma unroll
                for (int s = 0; s < KS; ++s) qf[s] = l.Q[w][piece_at<DK>(col, 4 * s + g)];
                load_k(seq.len - (ch + 1) * kC, ~ch & 1);
                wait_count<kAnyLoads>();  // Q read
                load_q(seq.len - (ch + 1) * kC);
                __builtin_amdgcn_sched_barrier(0);
                if (ch > 0) store(kC);
                loads_barrier<kAnyLoads>();  // R written
                const float cq = l.sc[3 * kC + 16 * w + col];
                f32x4 Q[kParts] = {};
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int p = 0; p < kParts; ++p)
                        Q[p] = mfma(__builtin_bit_cast(bf16x8, l.S[s][p][lane]), __builtin_bit_cast(bf16x8, qf[s]), Q[p]);
                O = cq * (Q[0] + (Q[1] + Q[2]));
                loads_barrier<kAnyLoads>();  // U written
                const uint32_t mark = l.marks[lane & 3];
                f32x4 u[2 * kSteps];
#pragma unroll
                for (int i = 0; i < 2 * kSteps; ++i) u[i] = l.U[i][lane];
                f32x4 sum[kParts] = {O};
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    uint2 x0[kParts], x1[kParts];
                    split4(u[2 * s], x0);
                    split4(u[2 * s + 1], x1);
                    uint2 m0[kParts], m1[kParts];
                    split4(__builtin_bit_cast(f32x4, mf[2 * s]), m0);
                    split4(__builtin_bit_cast(f32x4, mf[2 * s + 1]), m1);
                    bf16x8 uq[kParts], mq[kParts];
#pragma unroll
                    for (int p = 0; p < kParts; ++p) {
                        uq[p] = __builtin_bit_cast(bf16x8, join(x0[p], x1[p]));
                        mq[p] = __builtin_bit_cast(bf16x8, join(m0[p], m1[p]));
                    }
                    mfma_parts(uq, mq, sum);
                }
                O = sum[0] + (sum[1] + sum[2]);
                poisoned = __ballot(mark) != 0;
                if (poisoned) first = first_bad(l, col);
                __builtin_amdgcn_sched_barrier(0);
                load_m();
                __builtin_amdgcn_sched_barrier(0);
            }
            store(seq.len - (chunks - 1) * kC);
            wait_count<0>();  // nothing is on its way to LDS when the workgroup ends
        };
        if (w < 2)
            run(std::integral_constant<int, 1>());
        else
            run(std::integral_constant<int, 2>());
        return;
    }

    // ---- the state ----
    if (a.seq_status && threadIdx.x == 0 && h == 0 && v0 == 0) a.seq_status[b] = seq.ok ? GDN_OK : GDN_ERR_SHAPE;
    const int pool = a.slot ? a.slot[b] : b;
    const bool keep = pool >= 0 && pool < d.n_slots;
    const bool resume = keep && (!a.has_state || a.has_state[b] != 0);
    // state rows (elements of d_k) 32 (tau / 2) + 8 g + 4 (tau % 2) + r of tile tau
    float* Sp = keep ? a.S + ((int64_t(pool) * d.H_v + h) * d.d_v + v0 + col) * DK + 8 * g : nullptr;
    f32x4 S[TPW];
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
        const int tau = w * TPW + i;
        S[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (resume) S[i] = *reinterpret_cast<const f32x4*>(Sp + 32 * (tau >> 1) + 4 * (tau & 1));
    }
    auto run = [&](auto steps_of_tile) {
        constexpr int kSteps = steps_of_tile.value;  // 32-token steps up to token tile w
        const uint16_t* vp = static_cast<const uint16_t*>(a.v) + seq.start * d.v_stride + int64_t(h) * d.d_v + v0;
        const uint4* tp = c.t + (sh0 * kPairs + pair_at(w, 0)) * kParts * 64;
        const int64_t v_step = kC * d.v_stride, t_step = int64_t(d.H_v) * kPairs * kParts * 64;
        // wavefront 2 loads the scalars of every token, wavefront 3 gamma_64
        const float* xp = c.sc + sh0 * kScalars;
        const uint32_t x_off = (w == 3 ? kC : lane) * 16;
        const int64_t x_step = int64_t(d.H_v) * kScalars;
        // Each group of inputs is loaded for the next chunk (or the one after) as
        // soon as this chunk has used it, so one set of registers covers a chunk's
        // latency.  As for the outputs, no load is behind a branch.
        uint4 tf[kSteps][kParts], vr, xr;
        // V: a row of the slice is 2 pieces, wavefronts 0 and 1 hold all of them
        const int vi = w * 64 + lane;
        uint32_t v_off;
        auto v_rows = [&](int left) {
            v_off = (uint32_t(min(vi / 2, left - 1)) * uint32_t(d.v_stride) + 8 * (vi % 2)) * 2;
        };
        v_rows(seq.len);
        auto load_v = [&](int left) {
            if constexpr (kSteps == 1) {
                if (left < kC && left > 0) v_rows(left);
                vp += left > 0 ? v_step : 0;
                vr = load_at<uint4>(vp - v_step, v_off);
            } else {
                xp += left > 0 ? x_step : 0;
                xr = load_at<uint4>(xp - x_step, x_off);
            }
        };
        auto put_v = [&]() {
            if constexpr (kSteps == 1)
                l.V[vi] = vr;
            else if (w == 2 || lane == 0)
                *reinterpret_cast<uint4*>(&l.sc[x_off / 4]) = xr;
        };
        auto load_t = [&]() {
#pragma unroll
            for (int i = 0; i < kParts * kSteps; ++i) tf[i / kParts][i % kParts] = load_at<uint4>(tp + i * 64, lane * 16);
            tp += t_step;
        };
        // issued in the order of the loop: a wait for one group then lets the
        // groups behind it stay in flight
        load_v(seq.len);
        put_v();
        __builtin_amdgcn_sched_barrier(0);
        load_t();
        __builtin_amdgcn_sched_barrier(0);
        load_v(seq.len - kC);
        __builtin_amdgcn_sched_barrier(0);
        bool was_marked = false;
        for (int ch = 0; ch < chunks; ++ch) {
            const int n = seq.len - ch * kC;  // 64 or more but for the last

            // the state as operands
#pragma unroll
            for (int i = 0; i < TPW; ++i) {
                const int tau = w * TPW + i;
                uint2 x[kParts];
                split4(S[i], x);
#pragma unroll
                for (int p = 0; p < kParts; ++p) reinterpret_cast<uint2*>(&l.S[tau >> 1][p][lane])[tau & 1] = x[p];
            }
            loads_barrier<kAnyLoads>();

            // K S^T of token tile w, then R = V - gamma K S^T
            uint4 kf[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) kf[s] = l.K[ch & 1][w][piece_at<DK>(col, 4 * s + g)];
            const f32x4 cp = *reinterpret_cast<const f32x4*>(&l.sc[16 * w + 4 * g]);
            // the lane's column of rows 16 w + 4 g + r
            const uint2 v = read_tr(reinterpret_cast<const uint2*>(l.V) + (16 * w + 4 * g + (col >> 2)) * 4 + (col & 3));
            f32x4 P[kParts] = {};
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int p = 0; p < kParts; ++p)
                    P[p] = mfma(__builtin_bit_cast(bf16x8, kf[s]), __builtin_bit_cast(bf16x8, l.S[s][p][lane]), P[p]);
            // K^T of the wavefront's state rows: accumulator row rho of tile tau is
            // element 32 (tau / 2) + 8 (rho / 4) + 4 (tau % 2) + rho % 4.  In a
            // transposing read lane i of 16 names 4 elements of row i / 4 and gets
            // element i of the 4 rows.
            uint4 ktf[TPW][2];
#pragma unroll
            for (int i = 0; i < TPW; ++i)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int tau = w * TPW + i;
                    uint2 x[2];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint4* p =
                            &l.K[ch & 1][2 * s + half][piece_at<DK>(4 * g + (col >> 2), 4 * (tau >> 1) + (col & 3))];
                        x[half] = read_tr(reinterpret_cast<const uint2*>(p) + (tau & 1));
                    }
                    ktf[i][s] = make_uint4(x[0].x, x[0].y, x[1].x, x[1].y);
                }
            const f32x4 vv = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
            f32x4 R = vv - cp * (P[0] + (P[1] + P[2]));
            if (n < kC)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (16 * w + 4 * g + r >= n) R[r] = 0.0f;
            // A value that is not finite must not reach earlier tokens through a
            // product with a masked zero: it is taken out here, its row is marked,
            // and rows from the first marked one on come out as NaN.
            float check = 0.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r) check = fmaf(R[r], 0.0f, check);
            const bool marked = __ballot(!(check == 0.0f)) != 0;
            if (marked || was_marked) {
                if (lane == 0) l.marks[w] = marked;
                was_marked = marked;
                unsigned m = 0;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (!finite(R[r])) {
                        m |= 1u << r;
                        R[r] = 0.0f;
                    }
                l.badrow[w][lane] = m;
            }
            uint2 x[kParts];
            split4(R, x);
#pragma unroll
            for (int p = 0; p < kParts; ++p) reinterpret_cast<uint2*>(&l.R[w >> 1][p][lane])[w & 1] = x[p];
            loads_barrier<kAnyLoads>();

            // U = beta R + T R below the diagonal
            const f32x4 be = *reinterpret_cast<const f32x4*>(&l.sc[kC + 16 * w + 4 * g]);
            const f32x4 cu = *reinterpret_cast<const f32x4*>(&l.sc[2 * kC + 16 * w + 4 * g]);
            const float gam = l.sc[4 * kC];
            f32x4 sum[kParts] = {be * R};
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                bf16x8 tq[kParts], rq[kParts];
#pragma unroll
                for (int p = 0; p < kParts; ++p) {
                    tq[p] = __builtin_bit_cast(bf16x8, tf[s][p]);
                    rq[p] = __builtin_bit_cast(bf16x8, l.R[s][p][lane]);
                }
                mfma_parts(tq, rq, sum);
            }
            const uint32_t mark = l.marks[lane & 3];
            const f32x4 u = sum[0] + (sum[1] + sum[2]);
            f32x4 e = u * cu;
            if (__ballot(mark)) {
                const int first = first_bad(l, col);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (16 * w + 4 * g + r == first) e[r] = __builtin_nanf("");
            }
            split4(e, x);
#pragma unroll
            for (int p = 0; p < kParts; ++p) reinterpret_cast<uint2*>(&l.D[w >> 1][p][lane])[w & 1] = x[p];
            l.U[w][lane] = u;
            loads_barrier<kAnyLoads>();

            // S <- gamma_64 S + K^T diag(decay) U
            bf16x8 du[2][kParts];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int p = 0; p < kParts; ++p) du[s][p] = __builtin_bit_cast(bf16x8, l.D[s][p][lane]);
#pragma unroll
            for (int i = 0; i < TPW; ++i) S[i] *= gam;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int p = 0; p < kParts; ++p)
#pragma unroll
                    for (int i = 0; i < TPW; ++i)
                        S[i] = mfma(__builtin_bit_cast(bf16x8, ktf[i][s]), du[s][p], S[i]);
            __builtin_amdgcn_sched_barrier(0);
            load_t();
            __builtin_amdgcn_sched_barrier(0);
            put_v();
            load_v(n - 2 * kC);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if (chunks > 0) {
        if (w < 2)
            run(std::integral_constant<int, 1>());
        else
            run(std::integral_constant<int, 2>());
    }
    if (keep)
#pragma unroll
        for (int i = 0; i < TPW; ++i) {
            const int tau = w * TPW + i;
            *reinterpret_cast<f32x4*>(Sp + 32 * (tau >> 1) + 4 * (tau & 1)) = S[i];
        }
}

template <int DK>
hipError_t launch_chunks(const ChunkArgs& c, hipStream_t stream) {
    const gdn_seq_dims& d = c.s.d;
    prep_kernel<DK><<<grid_of(int64_t(c.slots + 7) / 8 * 8 * d.H_k + 1), 256, 0, stream>>>(c);
    const int items8 = (d.B * d.H_k + 7) / 8 * 8, per16 = d.H_v / d.H_k * (d.d_v / 16);
    chain_kernel<DK><<<grid_of(int64_t(items8) * per16), 512, 0, stream>>>(c);
    return hipGetLastError();
}

// fp32 q, k and v would need three parts each, so those are walked token by token,
// as are sequences of 8 tokens on average, which fill a small part of their
// chunks.  (The lengths themselves are on the device.)  At 8 the walk is no slower
// even if one sequence has nearly all tokens.  Walk and chunks, H_v 32, d 128, bf16,
// in us, by tokens per sequence on average:
//   one long, the others of one token  B 32: 8: 113 and 124, 12: 172 and 126;  B 120: 8: 420 and 377
//   lengths over two decades           B 32: 8: 77 and 120, 16: 127 and 123;   B 120: 8: 243 and 358
//   one sequence                       8: 6 and 17, 64: 25 and 18
bool use_chunks(const gdn_seq_dims& d) { return d.qkv_dtype == GDN_BF16 && d.T > 8 * int64_t(d.B); }

}  // namespace

size_t prefill_ws_bytes(const gdn_seq_dims& d) { return use_chunks(d) ? prep_layout(d).total : 0; }

hipError_t launch_prefill(const SeqArgs& a, hipStream_t stream) {
    if (!use_chunks(a.d)) return launch_prefill_walk(a, stream);
    const PrepLayout l = prep_layout(a.d);
    unsigned char* p = static_cast<unsigned char*>(a.ws);
    ChunkArgs c{a,
                reinterpret_cast<uint4*>(p + l.t),
                reinterpret_cast<uint4*>(p + l.m),
                reinterpret_cast<float*>(p + l.sc),
                reinterpret_cast<int*>(p + l.ordered),
                a.d.T / kC + a.d.B};
    return a.d.d_k == 128 ? launch_chunks<128>(c, stream) : launch_chunks<64>(c, stream);
}

}  // namespace gdn
