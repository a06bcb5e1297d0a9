// gdn_norm.hip -- the norms around a block: gdn_add_norm and gdn_gated_norm.
//
// Both are one pass over rows held in registers: every input is read once,
// every output written once, sums in fp32 over lanes (and over wavefronts
// through LDS where one row spans several).  Memory-bound: 8191 x 5120, x bf16,
// residual fp32, both norms: 503 MB in 108 us, 4.6 TB/s; gated, 16384 x 32 x 128
// bf16: 403 MB in 70 us, 5.7 TB/s (the last calls' rows are partly in cache; a
// copy of 1 GiB reaches 5.2).  Rows need not start on 16 bytes: pieces of 8
// elements are loaded wherever they start (8191 x 5119: 125 us; one element at a
// time 242 us).

#include "gdn_layer_internal.h"
#include "gdn_layer_util.h"

namespace gdn {
namespace {

__device__ __forceinline__ float inv_rms(float sumsq, float n, float eps) { return 1.0f / sqrtf(sumsq / n + eps); }

// Sum over the NW wavefronts of a workgroup; `part` holds 2 x 16 floats and
// `turn` alternates between calls so that one barrier per sum is enough.
__device__ __forceinline__ float block_sum(float x, float* part, int turn) {
    const int nw = blockDim.x >> 6;
    x = lane_sum<64>(x);
    if (nw == 1) return x;
    float* p = part + 16 * (turn & 1);
    if ((threadIdx.x & 63) == 0) p[threadIdx.x >> 6] = x;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < nw; ++w) s += p[w];
    return s;
}

// The piece of 8 elements at i of a row that has n elements from there on;
// those beyond read as zero and are not written.  Without TAIL n is 8 or more.
template <bool TAIL>
__device__ __forceinline__ void load_piece(const void* p, int dtype, int64_t i, int n, float (&x)[8]) {
    if (!TAIL || n >= 8) {
        load8(p, dtype, i, x);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = e < n ? load1(p, dtype, i + e) : 0.0f;
    }
}
template <bool TAIL>
__device__ __forceinline__ void store_piece(void* p, int dtype, int64_t i, int n, const float (&x)[8]) {
    if (!TAIL || n >= 8) {
        store8(p, dtype, i, x);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) store1(p, dtype, i + e, x[e]);
    }
}

// One row per workgroup, VPT pieces of 8 elements per thread in registers.
// TAIL: D is not a multiple of 8.
template <int VPT, bool TAIL>
__global__ void __launch_bounds__(1024) add_norm_kernel(AddNormArgs a) {
    __shared__ float part[32];
    const gdn_add_norm_dims& d = a.d;
    const int nvec = (d.D + 7) >> 3;
    const int64_t t = block_id();
    if (t >= d.T) return;
    float x[VPT][8], r[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        if (j < nvec) {
            load_piece<TAIL>(a.x, d.x_dtype, t * d.x_stride + 8 * j, d.D - 8 * j, x[i]);
            if (a.res) load_piece<TAIL>(a.res, d.res_dtype, t * d.res_stride + 8 * j, d.D - 8 * j, r[i]);
        }
    }
    if (a.post) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (threadIdx.x + i * blockDim.x < nvec)
#pragma unroll
                for (int e = 0; e < 8; ++e) s += x[i][e] * x[i][e];
        const float inv = inv_rms(block_sum(s, part, 0), d.D, d.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            if (j < nvec) {
                float p[8];
                load_piece<TAIL>(a.post, GDN_F32, 8 * j, d.D - 8 * j, p);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] = x[i][e] * inv * (p[e] + d.weight_offset);
            }
        }
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        if (j < nvec) {
            float c[8];
            if (a.chan) load_piece<TAIL>(a.chan, GDN_F32, 8 * j, d.D - 8 * j, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = a.chan ? c[e] * x[i][e] : x[i][e];
                x[i][e] = a.res ? r[i][e] + d.scale * p : d.scale * p;
                s += x[i][e] * x[i][e];
            }
            if (a.h) store_piece<TAIL>(a.h, d.res_dtype, t * d.h_stride + 8 * j, d.D - 8 * j, x[i]);
        }
    }
    const float inv = inv_rms(block_sum(s, part, 1), d.D, d.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        if (j < nvec) {
            float w[8];
            load_piece<TAIL>(a.w, GDN_F32, 8 * j, d.D - 8 * j, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = x[i][e] * inv * (w[e] + d.weight_offset);
            store_piece<TAIL>(a.y, d.y_dtype, t * d.y_stride + 8 * j, d.D - 8 * j, x[i]);
        }
    }
}

// W lanes of 8 elements per head.  TAIL: d is not a multiple of 8.
template <int W, bool TAIL>
__global__ void __launch_bounds__(256) gated_norm_vec_kernel(GatedNormArgs a) {
    const gdn_gated_norm_dims& d = a.d;
    const int64_t n = int64_t(d.T) * d.H, step = int64_t(gridDim.x) * (256 / W);
    const int e0 = 8 * (threadIdx.x % W);
    const bool in = e0 < d.d;
    float w[8];
    if (in) load_piece<TAIL>(a.w, GDN_F32, e0, d.d - e0, w);
    for (int64_t i = int64_t(blockIdx.x) * (256 / W) + threadIdx.x / W; i < n; i += step) {
        const int64_t t = i / d.H, c = (i - t * d.H) * d.d + e0;
        float o[8], z[8], s = 0.0f;
        if (in) {
            load_piece<TAIL>(a.o, d.o_dtype, t * d.o_stride + c, d.d - e0, o);
            load_piece<TAIL>(a.z, d.z_dtype, t * d.z_stride + c, d.d - e0, z);
#pragma unroll
            for (int e = 0; e < 8; ++e) s += o[e] * o[e];
        }
        const float inv = inv_rms(lane_sum<W>(s), d.d, d.eps);
        if (in) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = o[e] * inv * w[e] * activate(d.gate, z[e]);
            store_piece<TAIL>(a.y, d.y_dtype, t * d.y_stride + c, d.d - e0, o);
        }
    }
}

// Heads wider than 512: one wavefront per head, element by element and o twice, which
// bounds it: 16384 x 4 x 1024 bf16 247 us, 1.6 TB/s; 4096 x 1 x 16384 410 us.
__global__ void __launch_bounds__(256) gated_norm_any_kernel(GatedNormArgs a) {
    const gdn_gated_norm_dims& d = a.d;
    const int64_t n = int64_t(d.T) * d.H, step = int64_t(gridDim.x) * 4;
    const int lane = threadIdx.x & 63;
    for (int64_t i = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); i < n; i += step) {
        const int64_t t = i / d.H, c = (i - t * d.H) * d.d;
        float s = 0.0f;
        for (int e = lane; e < d.d; e += 64) {
            const float o = load1(a.o, d.o_dtype, t * d.o_stride + c + e);
            s += o * o;
        }
        const float inv = inv_rms(lane_sum<64>(s), d.d, d.eps);
        for (int e = lane; e < d.d; e += 64) {
            const float o = load1(a.o, d.o_dtype, t * d.o_stride + c + e);
            const float z = load1(a.z, d.z_dtype, t * d.z_stride + c + e);
            store1(a.y, d.y_dtype, t * d.y_stride + c + e, o * inv * a.w[e] * activate(d.gate, z));
        }
    }
}

}  // namespace

hipError_t launch_add_norm(const AddNormArgs& a, hipStream_t stream) {
    const gdn_add_norm_dims& d = a.d;
    const int nvec = (d.D + 7) / 8;
    auto threads = [&](int vpt) { return ((nvec + vpt - 1) / vpt + 63) / 64 * 64; };
    const bool tail = d.D % 8 != 0;
    if (threads(1) <= 512)
        tail ? add_norm_kernel<1, true><<<grid_of(d.T), threads(1), 0, stream>>>(a)
             : add_norm_kernel<1, false><<<grid_of(d.T), threads(1), 0, stream>>>(a);
    else
        tail ? add_norm_kernel<2, true><<<grid_of(d.T), threads(2), 0, stream>>>(a)
             : add_norm_kernel<2, false><<<grid_of(d.T), threads(2), 0, stream>>>(a);
    return hipGetLastError();
}

template <int W>
static void launch_gated(const GatedNormArgs& a, int64_t groups, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(groups < (1 << 20) ? groups : (1 << 20)));
    if (a.d.d % 8)
        gated_norm_vec_kernel<W, true><<<grid, 256, 0, stream>>>(a);
    else
        gated_norm_vec_kernel<W, false><<<grid, 256, 0, stream>>>(a);
}

hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t stream) {
    const int64_t n = int64_t(a.d.T) * a.d.H;
    const int w = a.d.d;
    if (w <= 64)
        launch_gated<8>(a, (n + 31) / 32, stream);
    else if (w <= 128)
        launch_gated<16>(a, (n + 15) / 16, stream);
    else if (w <= 256)
        launch_gated<32>(a, (n + 7) / 8, stream);
    else if (w <= 512)
        launch_gated<64>(a, (n + 3) / 4, stream);
    else
        gated_norm_any_kernel<<<static_cast<unsigned>((n + 3) / 4 < (1 << 20) ? (n + 3) / 4 : (1 << 20)), 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace gdn
