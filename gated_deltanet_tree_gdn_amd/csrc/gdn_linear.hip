// gdn_linear.hip -- y = residual + scale * act(x w^T + bias) on bf16 MFMA.

#include "gdn_layer_internal.h"
#include "gdn_layer_util.h"
#include "gdn_mfma.h"

namespace gdn {
namespace {

// One output: bias, activation, scale and residual in fp32, rounded once.
__device__ __forceinline__ void put(const LinearArgs& a, int64_t m, int64_t n, float acc) {
    const gdn_linear_dims& d = a.d;
    if (a.bias) acc += a.bias[n];
    acc = d.scale * activate(d.act, acc);
    if (a.res) acc += load1(a.res, d.res_dtype, m * d.res_stride + n);
    store1(a.y, d.y_dtype, m * d.y_stride + n, acc);
}

// 8 elements k .. k + 7 of a row of K, zeros past its end.
template <bool VEC>
__device__ __forceinline__ uint4 load_k8(const uint16_t* row, int k, int K) {
    if constexpr (VEC) {
        return k < K ? *reinterpret_cast<const uint4*>(row + k) : make_uint4(0, 0, 0, 0);
    } else {
        uint32_t u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = k + j < K ? row[k + j] : 0u;
        return make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
    }
}

// 64 x 64 outputs per workgroup, 4 wavefronts of 32 x 32, K in steps of 32.
template <bool VEC>
__global__ void __launch_bounds__(256) linear_tile_kernel(LinearArgs a) {
    __shared__ uint4 xs[64 * 4], ws[64 * 4];
    const gdn_linear_dims& d = a.d;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t m0 = int64_t(blockIdx.y) * 64, n0 = int64_t(blockIdx.x) * 64;
    const int r = tid >> 2, c = tid & 3;
    const int64_t mr = m0 + r < d.M ? m0 + r : d.M - 1, nr = n0 + r < d.N ? n0 + r : d.N - 1;
    const uint16_t* xrow = static_cast<const uint16_t*>(a.x) + mr * d.x_stride;
    const uint16_t* wrow = static_cast<const uint16_t*>(a.w) + nr * d.w_stride;
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    f32x4 acc[2][2] = {};
    for (int k = 0; k < d.K; k += 32) {
        const uint4 xv = load_k8<VEC>(xrow, k + 8 * c, d.K), wv = load_k8<VEC>(wrow, k + 8 * c, d.K);
        __syncthreads();
        xs[r * 4 + (c ^ (r >> 1 & 3))] = xv;
        ws[r * 4 + (c ^ (r >> 1 & 3))] = wv;
        __syncthreads();
        bf16x8 xf[2], wf[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rx = wm + 16 * i + (lane & 15), rw = wn + 16 * i + (lane & 15);
            xf[i] = __builtin_bit_cast(bf16x8, xs[rx * 4 + ((lane >> 4) ^ (rx >> 1 & 3))]);
            wf[i] = __builtin_bit_cast(bf16x8, ws[rw * 4 + ((lane >> 4) ^ (rw >> 1 & 3))]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = mfma(xf[i], wf[j], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t m = m0 + wm + 16 * i + 4 * (lane >> 4) + e, n = n0 + wn + 16 * j + (lane & 15);
                if (m < d.M && n < d.N) put(a, m, n, acc[i][j][e]);
            }
}

}  // namespace

size_t linear_ws_bytes(const gdn_linear_dims&) { return 0; }

hipError_t launch_linear(const LinearArgs& a, hipStream_t stream) {
    const gdn_linear_dims& d = a.d;
    const bool vec = d.K % 8 == 0 && (d.M <= 1 || d.x_stride % 8 == 0) && (d.N <= 1 || d.w_stride % 8 == 0);
    const dim3 grid((d.N + 63) / 64, (d.M + 63) / 64);
    if (vec)
        linear_tile_kernel<true><<<grid, 256, 0, stream>>>(a);
    else
        linear_tile_kernel<false><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace gdn
