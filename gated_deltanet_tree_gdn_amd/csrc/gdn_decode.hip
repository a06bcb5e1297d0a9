// gdn_decode.hip -- the delta rule token by token with the state in
// registers: gdn_decode (one token per sequence) and the walk that
// gdn_prefill uses where chunks do not pay.
//
// Eight lanes share a row of the state (d_k / 8 elements each, in pieces of 4
// so that the eight lanes read 128 contiguous bytes); a wavefront holds 8
// rows, and a dot product over d_k is three exchanges between lanes.  With
// the decayed state S' = e^g S, both S' k and S' q come from one sweep, and
//     u = beta (v - S' k),   o = S' q + u (k . q),   S = S' + u k^T.

#include "gdn_layer_internal.h"
#include "gdn_layer_util.h"

namespace gdn {
namespace {

template <typename T>
__device__ __forceinline__ void load4(const T* p, float* x) {
    if constexpr (sizeof(T) == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
    } else {
        const float4 f = *reinterpret_cast<const float4*>(p);
        x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
    }
}

template <typename T>
__device__ __forceinline__ float to_float(T x) {
    if constexpr (sizeof(T) == 2)
        return __builtin_bit_cast(float, static_cast<uint32_t>(x) << 16);
    else
        return x;
}

// The lane's E = d_k / 8 elements of a row: pieces of 4, 32 apart.
template <int E, typename T>
__device__ __forceinline__ void load_row(const T* row, int l8, float (&x)[E]) {
#pragma unroll
    for (int j = 0; j < E / 4; ++j) load4(row + 32 * j + 4 * l8, x + 4 * j);
}

template <int E>
__device__ __forceinline__ float dot(const float (&a)[E], const float (&b)[E]) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < E; ++j) s[j & 3] += a[j] * b[j];
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// One step of a state row: S <- e^g S + u k^T; returns S q (kq = k . q).
template <int E>
__device__ __forceinline__ float delta_step(float (&S)[E], const float (&k)[E], const float (&q)[E], float alpha,
                                            float beta, float v, float kq) {
#pragma unroll
    for (int j = 0; j < E; ++j) S[j] *= alpha;
    const float sk = lane_sum<8>(dot(S, k)), sq = lane_sum<8>(dot(S, q));
    const float u = beta * (v - sk);
#pragma unroll
    for (int j = 0; j < E; ++j) S[j] += u * k[j];
    return sq + u * kq;
}

// q and k of one token, normalised and scaled as asked; returns k . q.
template <int E>
__device__ __forceinline__ float scale_qk(const gdn_seq_dims& d, float (&q)[E], float (&k)[E]) {
    float rq = d.q_scale;
    if (d.qk_l2norm) {
        const float rk = 1.0f / sqrtf(lane_sum<8>(dot(k, k)) + d.l2_eps);
        rq *= 1.0f / sqrtf(lane_sum<8>(dot(q, q)) + d.l2_eps);
#pragma unroll
        for (int j = 0; j < E; ++j) k[j] *= rk;
    }
#pragma unroll
    for (int j = 0; j < E; ++j) q[j] *= rq;
    return lane_sum<8>(dot(k, q));
}

// Grid (d_v / (32 R), H_v, B): a wavefront takes R groups of 8 state rows.
template <typename T, int DK, int R>
__global__ void __launch_bounds__(256) decode_kernel(SeqArgs a) {
    constexpr int E = DK / 8;
    const gdn_seq_dims& d = a.d;
    const int b = blockIdx.z, h = blockIdx.y, hk = h / (d.H_v / d.H_k);
    const int lane = threadIdx.x & 63, l8 = lane & 7;
    const int row0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 8 * R + (lane >> 3);
    const int slot = a.slot ? a.slot[b] : b;
    const int64_t bh = int64_t(b) * d.H_v + h;
    if (slot < 0 || slot >= d.n_slots) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (l8 == 0) store1(a.o, d.o_dtype, bh * d.d_v + row0 + 8 * r, 0.0f);
        return;
    }
    float* S = a.S + ((int64_t(slot) * d.H_v + h) * d.d_v + row0) * DK;
    float s[R][E];
#pragma unroll
    for (int r = 0; r < R; ++r) load_row<E>(S + int64_t(8 * r) * DK, l8, s[r]);
    float q[E], k[E];
    load_row<E>(static_cast<const T*>(a.q) + b * d.q_stride + int64_t(hk) * DK, l8, q);
    load_row<E>(static_cast<const T*>(a.k) + b * d.k_stride + int64_t(hk) * DK, l8, k);
    const float kq = scale_qk<E>(d, q, k);
    const T* v = static_cast<const T*>(a.v) + b * d.v_stride + int64_t(h) * d.d_v + row0;
    const float alpha = expf(a.g[bh]), beta = a.beta[bh];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float o = delta_step<E>(s[r], k, q, alpha, beta, to_float(v[8 * r]), kq);
#pragma unroll
        for (int j = 0; j < E / 4; ++j)
            *reinterpret_cast<float4*>(S + int64_t(8 * r) * DK + 32 * j + 4 * l8) =
                make_float4(s[r][4 * j], s[r][4 * j + 1], s[r][4 * j + 2], s[r][4 * j + 3]);
        if (l8 == 0) store1(a.o, d.o_dtype, bh * d.d_v + row0 + 8 * r, o);
    }
}

// Grid (d_v / 32, H_v, B): the tokens of sequence b in order, 8 state rows
// per wavefront; the next token's rows are loaded while this one is applied.
template <typename T, int DK>
__global__ void __launch_bounds__(256) walk_kernel(SeqArgs a) {
    constexpr int E = DK / 8;
    const gdn_seq_dims& d = a.d;
    const int b = blockIdx.z, h = blockIdx.y, hk = h / (d.H_v / d.H_k);
    const int lane = threadIdx.x & 63, l8 = lane & 7;
    const int row = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 8 + (lane >> 3);
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
        load_row<E>(S, l8, s);
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) s[j] = 0.0f;
    }
    const T* q = static_cast<const T*>(a.q) + int64_t(hk) * DK;
    const T* k = static_cast<const T*>(a.k) + int64_t(hk) * DK;
    const T* v = static_cast<const T*>(a.v) + int64_t(h) * d.d_v + row;
    float qn[E], kn[E], vn = 0.0f, gn = 0.0f, bn = 0.0f;  // as loaded
    auto load = [&](int64_t n) {
        load_row<E>(q + n * d.q_stride, l8, qn);
        load_row<E>(k + n * d.k_stride, l8, kn);
        vn = to_float(v[n * d.v_stride]);
        gn = a.g[n * d.H_v + h];
        bn = a.beta[n * d.H_v + h];
    };
    if (t < end) load(t);
    for (; t < end; ++t) {
        float qc[E], kc[E];
#pragma unroll
        for (int j = 0; j < E; ++j) {
            qc[j] = qn[j];
            kc[j] = kn[j];
        }
        const float vc = vn, gc = gn, bc = bn;
        if (t + 1 < end) load(t + 1);
        const float kq = scale_qk<E>(d, qc, kc);
        const float o = delta_step<E>(s, kc, qc, expf(gc), bc, vc, kq);
        if (l8 == 0) store1(a.o, d.o_dtype, (t * d.H_v + h) * d.d_v + row, o);
    }
    if (keep) {
#pragma unroll
        for (int j = 0; j < E / 4; ++j)
            *reinterpret_cast<float4*>(S + 32 * j + 4 * l8) =
                make_float4(s[4 * j], s[4 * j + 1], s[4 * j + 2], s[4 * j + 3]);
    }
}

template <typename T, int DK>
void decode_t(const SeqArgs& a, hipStream_t stream) {
    const gdn_seq_dims& d = a.d;
    decode_kernel<T, DK, 1><<<dim3(d.d_v / 32, d.H_v, d.B), 256, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_decode(const SeqArgs& a, hipStream_t stream) {
    const bool bf = a.d.qkv_dtype == GDN_BF16;
    if (a.d.d_k == 128)
        bf ? decode_t<uint16_t, 128>(a, stream) : decode_t<float, 128>(a, stream);
    else
        bf ? decode_t<uint16_t, 64>(a, stream) : decode_t<float, 64>(a, stream);
    return hipGetLastError();
}

hipError_t launch_prefill_walk(const SeqArgs& a, hipStream_t stream) {
    const bool bf = a.d.qkv_dtype == GDN_BF16;
    const dim3 grid(a.d.d_v / 32, a.d.H_v, a.d.B);
    if (a.d.d_k == 128)
        bf ? walk_kernel<uint16_t, 128><<<grid, 256, 0, stream>>>(a) : walk_kernel<float, 128><<<grid, 256, 0, stream>>>(a);
    else
        bf ? walk_kernel<uint16_t, 64><<<grid, 256, 0, stream>>>(a) : walk_kernel<float, 64><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace gdn
