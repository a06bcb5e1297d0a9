// gdn_norm.hip -- the norms around a block: gdn_add_norm and gdn_gated_norm.
//
// Both are one pass over rows held in registers: every input is read once,
// every output written once, sums in fp32 over lanes (and over wavefronts
// through LDS where one row spans several).  HBM-bound.

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

// One row per workgroup, VPT vectors of 8 elements per thread in registers.
template <int VPT>
__global__ void add_norm_row_kernel(AddNormArgs a) {
    __shared__ float part[32];
    const gdn_add_norm_dims& d = a.d;
    const int nvec = d.D >> 3;
    const int64_t t = blockIdx.x;
    float x[VPT][8], r[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        if (j < nvec) {
            load8(a.x, d.x_dtype, t * d.x_stride + 8 * j, x[i]);
            if (a.res) load8(a.res, d.res_dtype, t * d.res_stride + 8 * j, r[i]);
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
                load8(a.post, GDN_F32, 8 * j, p);
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
            if (a.chan) load8(a.chan, GDN_F32, 8 * j, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = a.chan ? c[e] * x[i][e] : x[i][e];
                x[i][e] = a.res ? r[i][e] + d.scale * p : d.scale * p;
                s += x[i][e] * x[i][e];
            }
            if (a.h) store8(a.h, d.res_dtype, t * d.h_stride + 8 * j, x[i]);
        }
    }
    const float inv = inv_rms(block_sum(s, part, 1), d.D, d.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        if (j < nvec) {
            float w[8];
            load8(a.w, GDN_F32, 8 * j, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = x[i][e] * inv * (w[e] + d.weight_offset);
            store8(a.y, d.y_dtype, t * d.y_stride + 8 * j, x[i]);
        }
    }
}

// Rows of any length and alignment: one row per workgroup, element by
// element, the row kept in LDS as fp32.
__global__ void add_norm_any_kernel(AddNormArgs a) {
    extern __shared__ float row[];
    __shared__ float part[32];
    const gdn_add_norm_dims& d = a.d;
    const int64_t t = blockIdx.x;
    float inv = 1.0f;
    if (a.post) {
        float s = 0.0f;
        for (int j = threadIdx.x; j < d.D; j += blockDim.x) {
            const float x = load1(a.x, d.x_dtype, t * d.x_stride + j);
            row[j] = x;
            s += x * x;
        }
        inv = inv_rms(block_sum(s, part, 0), d.D, d.eps);
    }
    float s = 0.0f;
    for (int j = threadIdx.x; j < d.D; j += blockDim.x) {
        float p = a.post ? row[j] * inv * (a.post[j] + d.weight_offset) : load1(a.x, d.x_dtype, t * d.x_stride + j);
        if (a.chan) p *= a.chan[j];
        const float h = a.res ? load1(a.res, d.res_dtype, t * d.res_stride + j) + d.scale * p : d.scale * p;
        if (a.h) store1(a.h, d.res_dtype, t * d.h_stride + j, h);
        row[j] = h;  // read back by this thread only
        s += h * h;
    }
    inv = inv_rms(block_sum(s, part, 1), d.D, d.eps);
    for (int j = threadIdx.x; j < d.D; j += blockDim.x)
        store1(a.y, d.y_dtype, t * d.y_stride + j, row[j] * inv * (a.w[j] + d.weight_offset));
}

// W lanes of 8 elements per head.
template <int W>
__global__ void __launch_bounds__(256) gated_norm_vec_kernel(GatedNormArgs a) {
    const gdn_gated_norm_dims& d = a.d;
    const int64_t n = int64_t(d.T) * d.H, step = int64_t(gridDim.x) * (256 / W);
    const int e0 = 8 * (threadIdx.x % W);
    const bool in = e0 < d.d;
    float w[8];
    if (in) load8(a.w, GDN_F32, e0, w);
    for (int64_t i = int64_t(blockIdx.x) * (256 / W) + threadIdx.x / W; i < n; i += step) {
        const int64_t t = i / d.H, c = (i - t * d.H) * d.d + e0;
        float o[8], z[8], s = 0.0f;
        if (in) {
            load8(a.o, d.o_dtype, t * d.o_stride + c, o);
            load8(a.z, d.z_dtype, t * d.z_stride + c, z);
#pragma unroll
            for (int e = 0; e < 8; ++e) s += o[e] * o[e];
        }
        const float inv = inv_rms(lane_sum<W>(s), d.d, d.eps);
        if (in) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = o[e] * inv * w[e] * activate(d.gate, z[e]);
            store8(a.y, d.y_dtype, t * d.y_stride + c, o);
        }
    }
}

// Heads of any width and alignment: one wavefront per head.
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

// Rows of 16-byte pieces: the base is aligned, so the stride decides.
bool vec_rows(int64_t stride, int64_t rows, int dtype) { return rows <= 1 || stride * dtype_size(dtype) % 16 == 0; }

}  // namespace

hipError_t launch_add_norm(const AddNormArgs& a, hipStream_t stream) {
    const gdn_add_norm_dims& d = a.d;
    const bool vec = d.D % 8 == 0 && vec_rows(d.x_stride, d.T, d.x_dtype) && vec_rows(d.y_stride, d.T, d.y_dtype) &&
                     (!a.res || vec_rows(d.res_stride, d.T, d.res_dtype)) &&
                     (!a.h || vec_rows(d.h_stride, d.T, d.res_dtype));
    if (!vec) {
        add_norm_any_kernel<<<d.T, 256, d.D * sizeof(float), stream>>>(a);
        return hipGetLastError();
    }
    const int nvec = d.D / 8;
    auto threads = [&](int vpt) { return ((nvec + vpt - 1) / vpt + 63) / 64 * 64; };
    if (threads(1) <= 512)
        add_norm_row_kernel<1><<<d.T, threads(1), 0, stream>>>(a);
    else
        add_norm_row_kernel<2><<<d.T, threads(2), 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t stream) {
    const gdn_gated_norm_dims& d = a.d;
    const int64_t n = int64_t(d.T) * d.H;
    const bool vec = d.d % 8 == 0 && d.d <= 512 && vec_rows(d.o_stride, d.T, d.o_dtype) &&
                     vec_rows(d.z_stride, d.T, d.z_dtype) && vec_rows(d.y_stride, d.T, d.y_dtype);
    auto grid = [&](int per) {
        const int64_t g = (n + per - 1) / per;
        return dim3(static_cast<unsigned>(g < (1 << 20) ? g : (1 << 20)));
    };
    if (!vec)
        gated_norm_any_kernel<<<grid(4), 256, 0, stream>>>(a);
    else if (d.d <= 64)
        gated_norm_vec_kernel<8><<<grid(32), 256, 0, stream>>>(a);
    else if (d.d <= 128)
        gated_norm_vec_kernel<16><<<grid(16), 256, 0, stream>>>(a);
    else if (d.d <= 256)
        gated_norm_vec_kernel<32><<<grid(8), 256, 0, stream>>>(a);
    else
        gated_norm_vec_kernel<64><<<grid(4), 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace gdn
