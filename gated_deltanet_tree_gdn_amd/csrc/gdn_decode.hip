// gdn_decode.hip -- the delta rule token by token with the state in
// registers: gdn_decode (one token per sequence) and the walk that
// gdn_prefill uses where chunks do not pay.
//
// Lanes share a row of the state in pieces of 4 elements (8 lanes: 128
// contiguous bytes), and a dot product over d_k is a few exchanges between
// them.  S k and S q come from one sweep over the state before the update:
//     u = beta (v - e^g S k),   o = e^g S q + u (k . q),   S <- e^g S + u k^T.

#include "gdn_layer_internal.h"
#include "gdn_layer_util.h"
#include "gdn_mfma.h"

namespace gdn {
namespace {

// Four adjacent elements as loaded.
template <typename T>
struct Four;
template <>
struct Four<uint16_t> {
    uint2 u;
    __device__ __forceinline__ float at(int i) const {
        const uint32_t w = i < 2 ? u.x : u.y;
        return i & 1 ? bf16_hi(w) : bf16_lo(w);
    }
};
template <>
struct Four<float> {
    f32x4 u;
    __device__ __forceinline__ float at(int i) const { return u[i]; }
};

__device__ __forceinline__ float to_float(uint16_t x) { return bf16_lo(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

// L lanes share a row; lane l has N pieces of 4 elements, 4 L apart.
template <int L, int N, typename T>
__device__ __forceinline__ void load_pieces(const T* row, int l, Four<T> (&x)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = *reinterpret_cast<const Four<T>*>(row + 4 * (L * j + l));
}

template <int E, typename T>
__device__ __forceinline__ void unpack(const Four<T> (&x)[E / 4], float (&y)[E]) {
#pragma unroll
    for (int j = 0; j < E; ++j) y[j] = x[j / 4].at(j % 4);
}

template <int L, int E, typename T>
__device__ __forceinline__ void load_row(const T* row, int l, float (&y)[E]) {
    Four<T> x[E / 4];
    load_pieces<L>(row, l, x);
    unpack<E>(x, y);
}

template <int L, int E>
__device__ __forceinline__ void store_row(float* row, int l, const float (&x)[E]) {
#pragma unroll
    for (int j = 0; j < E / 4; ++j)
        *reinterpret_cast<f32x4*>(row + 4 * (L * j + l)) = f32x4{x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
}

template <int E>
__device__ __forceinline__ float dot(const float (&a)[E], const float (&b)[E]) {
    float s0 = a[0] * b[0], s1 = a[1] * b[1];
#pragma unroll
    for (int j = 2; j < E; j += 2) {
        s0 += a[j] * b[j];
        s1 += a[j + 1] * b[j + 1];
    }
    return s0 + s1;
}

// 1 / sqrt(x): the hardware's estimate (1 ulp) after one Newton step.
__device__ __forceinline__ float rsqrt_near(float x) {
    const float r = __builtin_amdgcn_rsqf(x);
    return r + 0.5f * r * fmaf(-x * r, r, 1.0f);
}

// What a token's q and k give besides their directions: their factors (the
// inverse norms where asked for, and q_scale) and k . q, all applied to dot
// products rather than to the vectors.
struct QkScale {
    float rk, rq, kq;
};
template <int L, int E>
__device__ __forceinline__ QkScale qk_scale(const gdn_seq_dims& d, const float (&q)[E], const float (&k)[E]) {
    QkScale s{1.0f, d.q_scale, 0.0f};
    if (d.qk_l2norm) {
        s.rk = rsqrt_near(lane_sum<L>(dot(k, k)) + d.l2_eps);
        s.rq *= rsqrt_near(lane_sum<L>(dot(q, q)) + d.l2_eps);
    }
    s.kq = lane_sum<L>(dot(k, q));
    return s;
}

// One step of a state row: S <- e^g S + u k^T; returns S q.
template <int L, int E>
__device__ __forceinline__ float delta_step(float (&S)[E], const float (&k)[E], const float (&q)[E], const QkScale& f,
                                            float g, float beta, float v) {
    // the hardware's 2^x, off by |g| 2^-24 and an ulp: least where the state stays
    const float alpha = __builtin_amdgcn_exp2f(g * 1.44269504f);
    const float sk = lane_sum<L>(dot(S, k)), sq = lane_sum<L>(dot(S, q));
    const float u = beta * (v - alpha * (f.rk * sk)) * f.rk;
#pragma unroll
    for (int j = 0; j < E; ++j) S[j] = alpha * S[j] + u * k[j];
    return f.rq * (alpha * sq + u * f.kq);
}

// Grid (d_v / 32, H_v, B): a wavefront takes 8 state rows.
// Bound by the states, read and written once: 114 of 120 rows live, H_v 32, d
// 128: 478 MB in 89 us, 5.4 TB/s (a copy of 1 GiB reaches 5.2).  One token alone is
// 4 MB in 3.5 us, most of it latency, over 512 wavefronts.
template <typename T, int DK>
__global__ void __launch_bounds__(256) decode_kernel(SeqArgs a) {
    constexpr int E = DK / 8;
    const gdn_seq_dims& d = a.d;
    const int b = blockIdx.z, h = blockIdx.y, hk = h / (d.H_v / d.H_k);
    const int lane = threadIdx.x & 63, l8 = lane & 7;
    const int row = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 8 + (lane >> 3);
    const int slot = a.slot ? a.slot[b] : b;
    const int64_t bh = int64_t(b) * d.H_v + h;
    if (slot < 0 || slot >= d.n_slots) {
        if (l8 == 0) store1(a.o, d.o_dtype, bh * d.d_v + row, 0.0f);
        return;
    }
    float* S = a.S + ((int64_t(slot) * d.H_v + h) * d.d_v + row) * DK;
    float s[E], q[E], k[E];
    load_row<8>(S, l8, s);
    load_row<8>(static_cast<const T*>(a.q) + b * d.q_stride + int64_t(hk) * DK, l8, q);
    load_row<8>(static_cast<const T*>(a.k) + b * d.k_stride + int64_t(hk) * DK, l8, k);
    const float v = to_float(static_cast<const T*>(a.v)[b * d.v_stride + int64_t(h) * d.d_v + row]);
    const float o = delta_step<8>(s, k, q, qk_scale<8>(d, q, k), a.g[bh], a.beta[bh], v);
    store_row<8>(S, l8, s);
    if (l8 == 0) store1(a.o, d.o_dtype, bh * d.d_v + row, o);
}

// One token as loaded.
template <typename T, int E>
struct Token {
    Four<T> q[E / 4], k[E / 4];
    T v;
    float g, beta;
};

// Grid (d_v L / 256, H_v, B): the tokens of sequence b in order, 64 / L state
// rows per wavefront.  A token takes less time than its loads, so the next kAhead
// are in flight; past the end the last token is loaded again, since a load
// behind a branch would be waited for at the branch's end.
// Bound by instructions, some 80 per token with 4 elements of a row per lane
// (d 64): 0.24 us per token of the longest sequence.
constexpr int kAhead = 4;
template <typename T, int DK, int L>
__global__ void __launch_bounds__(256) walk_kernel(SeqArgs a) {
    constexpr int E = DK / L;
    const gdn_seq_dims& d = a.d;
    const int b = blockIdx.z, h = blockIdx.y, hk = h / (d.H_v / d.H_k);
    const int lane = threadIdx.x & 63, l = lane % L;
    const int row = (blockIdx.x * 4 + (threadIdx.x >> 6)) * (64 / L) + lane / L;
    int64_t t = a.cu[b];
    int64_t end = a.cu[b + 1];
    const bool ok = 0 <= t && t <= end && end <= d.T;
    if (!ok) end = t;
    if (a.seq_status && blockIdx.x == 0 && h == 0 && threadIdx.x == 0) a.seq_status[b] = ok ? GDN_OK : GDN_ERR_SHAPE;
    const int slot = a.slot ? a.slot[b] : b;
    const bool keep = slot >= 0 && slot < d.n_slots;
    float* S = keep ? a.S + ((int64_t(slot) * d.H_v + h) * d.d_v + row) * DK : nullptr;
    float s[E];
    if (keep && (!a.has_state || a.has_state[b] != 0)) {
        load_row<L>(S, l, s);
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) s[j] = 0.0f;
    }
    const T* q = static_cast<const T*>(a.q) + int64_t(hk) * DK;
    const T* k = static_cast<const T*>(a.k) + int64_t(hk) * DK;
    const T* v = static_cast<const T*>(a.v) + int64_t(h) * d.d_v + row;
    if (t < end) {
        Token<T, E> tok[kAhead];
        // the next token to load: running addresses, as products of 64-bit strides
        // would be a third of a token's instructions
        const T *qn = q + t * d.q_stride, *kn = k + t * d.k_stride, *vn = v + t * d.v_stride;
        const float *gn = a.g + t * d.H_v + h, *bn = a.beta + t * d.H_v + h;
        int64_t left = end - t;  // tokens from it on
        auto load = [&](Token<T, E>& x) {
            load_pieces<L>(qn, l, x.q);
            load_pieces<L>(kn, l, x.k);
            x.v = *vn;
            x.g = *gn;
            x.beta = *bn;
            const bool more = --left > 0;
            qn += more ? d.q_stride : 0;
            kn += more ? d.k_stride : 0;
            vn += more ? d.v_stride : 0;
            gn += more ? d.H_v : 0;
            bn += more ? d.H_v : 0;
        };
        auto apply = [&](const Token<T, E>& x) {
            float qc[E], kc[E];
            unpack<E>(x.q, qc);
            unpack<E>(x.k, kc);
            return delta_step<L>(s, kc, qc, qk_scale<L>(d, qc, kc), x.g, x.beta, to_float(x.v));
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load(tok[i]);
        // lane i of a row stores token t + i
        for (; t + kAhead <= end; t += kAhead) {
            float o = 0.0f;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const float x = apply(tok[i]);
                o = l == i ? x : o;
                load(tok[i]);
            }
            if (l < kAhead) store1(a.o, d.o_dtype, ((t + l) * d.H_v + h) * d.d_v + row, o);
        }
#pragma unroll
        for (int i = 0; i < kAhead - 1; ++i)
            if (t + i < end) {
                const float o = apply(tok[i]);
                if (l == 0) store1(a.o, d.o_dtype, ((t + i) * d.H_v + h) * d.d_v + row, o);
            }
    }
    if (keep) store_row<L>(S, l, s);
}

}  // namespace

hipError_t launch_decode(const SeqArgs& a, hipStream_t stream) {
    const bool bf = a.d.qkv_dtype == GDN_BF16;
    const dim3 grid(a.d.d_v / 32, a.d.H_v, a.d.B);
    if (a.d.d_k == 128)
        bf ? decode_kernel<uint16_t, 128><<<grid, 256, 0, stream>>>(a) : decode_kernel<float, 128><<<grid, 256, 0, stream>>>(a);
    else
        bf ? decode_kernel<uint16_t, 64><<<grid, 256, 0, stream>>>(a) : decode_kernel<float, 64><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

template <int L>
static void launch_walk(const SeqArgs& a, hipStream_t stream) {
    const bool bf = a.d.qkv_dtype == GDN_BF16;
    const dim3 grid(a.d.d_v * L / 256, a.d.H_v, a.d.B);
    if (a.d.d_k == 128)
        bf ? walk_kernel<uint16_t, 128, L><<<grid, 256, 0, stream>>>(a)
           : walk_kernel<float, 128, L><<<grid, 256, 0, stream>>>(a);
    else
        bf ? walk_kernel<uint16_t, 64, L><<<grid, 256, 0, stream>>>(a)
           : walk_kernel<float, 64, L><<<grid, 256, 0, stream>>>(a);
}

// 16 lanes to a row halve a wavefront's work per token, which is what a walk
// waits for until the wavefronts crowd each other.  16 and 8 lanes, fp32, H_v
// 32, d 128: 1500 tokens in 1 sequence 495 and 647 us, 500 in 8 120 and 161 us,
// 1500 in 32 294 and 271 us.
hipError_t launch_prefill_walk(const SeqArgs& a, hipStream_t stream) {
    if (int64_t(a.d.B) * a.d.H_v * a.d.d_v <= 32768)
        launch_walk<16>(a, stream);
    else
        launch_walk<8>(a, stream);
    return hipGetLastError();
}

}  // namespace gdn
