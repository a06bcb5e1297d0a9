// gdn_linear.hip -- y = residual + scale * act(x w^T + bias) on bf16 MFMA.
//
// Products run as w x^T: a lane's accumulators are then 4 adjacent outputs of
// one row of y.
//
//  - thin_kernel (M <= 64): the weights straight from memory into operands;
//  - tile_kernel: BM x BN outputs per workgroup, K in steps of 64 through two
//    LDS buffers filled by direct loads while the other one is multiplied.

#include "gdn_layer_internal.h"
#include "gdn_layer_util.h"
#include "gdn_mfma.h"

namespace gdn {
namespace {

constexpr int kBK = 64;  // elements of K per step of the tile kernel: 8 pieces of 16 bytes per row

// Outputs n .. n + E - 1 of row m: bias, activation, scale and residual in
// fp32, rounded once.  VEC (E = 8): all of them exist and rows of y and
// residual are 16-byte aligned.
template <int E, bool VEC>
__device__ __forceinline__ void put(const LinearArgs& a, int64_t m, int n, float (&v)[E]) {
    static_assert(!VEC || E == 8, "");
    const gdn_linear_dims& d = a.d;
    float b[E] = {}, r[E] = {};
    if constexpr (VEC) {
        if (a.bias) load8(a.bias, GDN_F32, n, b);
        if (a.res) load8(a.res, d.res_dtype, m * d.res_stride + n, r);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (n + e < d.N) {
                if (a.bias) b[e] = a.bias[n + e];
                if (a.res) r[e] = load1(a.res, d.res_dtype, m * d.res_stride + n + e);
            }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] += b[e];
    if (d.act == GDN_ACT_GELU) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = activate(GDN_ACT_GELU, v[e]);
    } else if (d.act != GDN_ACT_NONE) {
        const bool silu = d.act == GDN_ACT_SILU;
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = (silu ? v[e] : 1.0f) * sigmoidf(v[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = a.res ? r[e] + d.scale * v[e] : d.scale * v[e];
    if constexpr (VEC) {
        store8(a.y, d.y_dtype, m * d.y_stride + n, v);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (n + e < d.N) store1(a.y, d.y_dtype, m * d.y_stride + n + e, v[e]);
    }
}

// Workgroups go to the 8 XCDs in turn; here each XCD gets a run of
// consecutive tiles, ordered in bands of 8 tile rows, so that the tiles it has
// in flight share rows of x and w in its L2.
__device__ __forceinline__ void tile_of(int id, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int total = tiles_m * tiles_n, q = total / 8, r = total % 8, xcd = id % 8, i = id / 8;
    const int t = xcd * q + min(xcd, r) + i;
    constexpr int kBand = 8;
    const int band = t / (kBand * tiles_n), in = t - band * kBand * tiles_n, rows = min(kBand, tiles_m - band * kBand);
    tm = band * kBand + in % rows;
    tn = in / rows;
}

typedef __attribute__((address_space(3))) void* lds_ptr;
typedef __amdgpu_buffer_rsrc_t rsrc_t;

// 8 elements k .. k + 7 of a row of K, zeros past its end; rows of any alignment.
__device__ __forceinline__ uint4 load_k8(const uint16_t* row, int k, int K) {
    typedef uint32_t u32x4a2 __attribute__((ext_vector_type(4), aligned(2)));
    if (k + 8 <= K) return __builtin_bit_cast(uint4, *reinterpret_cast<const u32x4a2*>(row + k));
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = k + j < K ? row[k + j] : 0u;
    return make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
}

// ROWS rows of x or w by 64 elements of K in LDS: row r's piece p (16 bytes)
// at position p ^ (r & 7), which spreads the 16 rows of a fragment read over
// the banks.  One direct load of a wavefront fills 8 rows (LDS addresses run
// with the lanes), so the permutation is made in the global address.
template <int ROWS, int WAVES>
struct Stage {
    static constexpr int L = ROWS / 8 / WAVES;  // loads per wavefront
    rsrc_t rsrc;
    uint32_t off[L];
    __device__ __forceinline__ void init(const uint16_t* base, int64_t stride, int64_t row0, int64_t rows, int wave,
                                         int lane) {
        const uint16_t* p = base + row0 * stride;
        rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), 0, 0x7fffffff, 0x00027000);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int r = (wave * L + i) * 8 + (lane >> 3);
            const uint32_t row = min(int64_t(r), rows - 1 - row0);
            off[i] = (row * uint32_t(stride) + 8 * ((lane & 7) ^ (r & 7))) * 2;
        }
    }
    __device__ __forceinline__ void load(uint4* lds, int k, int wave) const {
#pragma unroll
        for (int i = 0; i < L; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)(lds + (wave * L + i) * 64), 16, off[i], k * 2, 0, 0);
    }
};

// The same through registers, for rows of any alignment and the end of K.
template <int ROWS, int WAVES>
__device__ __forceinline__ void stage_any(uint4* lds, const uint16_t* base, int64_t stride, int64_t row0, int64_t rows,
                                          int k, int K, int wave, int lane) {
    constexpr int L = ROWS / 8 / WAVES;
    uint4 x[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const int r = (wave * L + i) * 8 + (lane >> 3);
        const int64_t row = min(row0 + r, rows - 1);
        x[i] = load_k8(base + row * stride, k + 8 * ((lane & 7) ^ (r & 7)), K);
    }
#pragma unroll
    for (int i = 0; i < L; ++i) lds[(wave * L + i) * 64 + lane] = x[i];
}

// WM x WN wavefronts, each (BM / WM) x (BN / WN) outputs.
template <int BM, int BN, int WM, int WN, bool DIRECT>
__global__ void __launch_bounds__(64 * WM * WN) tile_kernel(LinearArgs a, int vec_out) {
    constexpr int W = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int kOutRows = TM > 4 ? 64 : TM * 16, kOutLd = TN * 16 + 4;  // epilogue: rows of a wavefront at a time
    constexpr int kStageBytes = (BM + BN) * 8 * 16 * 2, kOutBytes = W * kOutRows * kOutLd * 4;
    __shared__ __align__(16) char lds[kStageBytes > kOutBytes ? kStageBytes : kOutBytes];
    auto xs = [&](int p) { return reinterpret_cast<uint4*>(lds) + p * BM * 8; };
    auto ws = [&](int p) { return reinterpret_cast<uint4*>(lds) + (2 * BM + p * BN) * 8; };
    const gdn_linear_dims& d = a.d;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    int tm, tn;
    tile_of(blockIdx.x, (d.M + BM - 1) / BM, (d.N + BN - 1) / BN, tm, tn);
    const int64_t m0 = int64_t(tm) * BM, n0 = int64_t(tn) * BN;
    const int wm = wave % WM, wn = wave / WM;
    const uint16_t* xp = static_cast<const uint16_t*>(a.x);
    const uint16_t* wp = static_cast<const uint16_t*>(a.w);
    f32x4 acc[TN][TM] = {};
    auto multiply = [&](const uint4* x, const uint4* w) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            bf16x8 xf[TM], wf[TN];
            const int at = (4 * s + g) ^ (col & 7);
#pragma unroll
            for (int i = 0; i < TM; ++i) xf[i] = __builtin_bit_cast(bf16x8, x[((wm * TM + i) * 16 + col) * 8 + at]);
#pragma unroll
            for (int j = 0; j < TN; ++j) wf[j] = __builtin_bit_cast(bf16x8, w[((wn * TN + j) * 16 + col) * 8 + at]);
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i) acc[j][i] = mfma(wf[j], xf[i], acc[j][i]);
        }
    };
    auto any_step = [&](int k) {
        stage_any<BM, W>(xs(0), xp, d.x_stride, m0, d.M, k, d.K, wave, lane);
        stage_any<BN, W>(ws(0), wp, d.w_stride, n0, d.N, k, d.K, wave, lane);
        __syncthreads();
        multiply(xs(0), ws(0));
        __syncthreads();
    };
    if constexpr (DIRECT) {
        const int steps = d.K / kBK;
        if (steps > 0) {
            Stage<BM, W> sx;
            Stage<BN, W> sw;
            sx.init(xp, d.x_stride, m0, d.M, wave, lane);
            sw.init(wp, d.w_stride, n0, d.N, wave, lane);
            sx.load(xs(0), 0, wave);
            sw.load(ws(0), 0, wave);
            __syncthreads();
            for (int t = 0; t < steps; ++t) {
                const int p = t & 1;
                if (t + 1 < steps) {
                    sx.load(xs(p ^ 1), (t + 1) * kBK, wave);
                    sw.load(ws(p ^ 1), (t + 1) * kBK, wave);
                }
                multiply(xs(p), ws(p));
                __syncthreads();
            }
        }
        if (d.K % kBK) any_step(d.K / kBK * kBK);
    } else {
        for (int k = 0; k < d.K; k += kBK) any_step(k);
    }
    // Rows through LDS, so that a lane stores 8 adjacent outputs and the
    // activation's code is not repeated for every register.
    float* out = reinterpret_cast<float*>(lds) + wave * kOutRows * kOutLd;
    constexpr int PER = TN * 16 / 8;  // pieces of 8 outputs per row
#pragma unroll
    for (int half = 0; half < TM * 16 / kOutRows; ++half) {
#pragma unroll
        for (int i = 0; i < kOutRows / 16; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                *reinterpret_cast<f32x4*>(&out[(i * 16 + col) * kOutLd + j * 16 + 4 * g]) =
                    acc[j][half * (kOutRows / 16) + i];
#pragma unroll 1
        for (int e = lane; e < kOutRows * PER; e += 64) {
            const int r = e / PER, c = e % PER * 8;
            const int64_t m = m0 + wm * TM * 16 + half * kOutRows + r, n = n0 + wn * TN * 16 + c;
            float v[8];
            load8(out, GDN_F32, r * kOutLd + c, v);
            if (m < d.M && n < d.N) {
                if (vec_out)
                    put<8, true>(a, m, n, v);
                else
                    put<8, false>(a, m, n, v);
            }
        }
    }
}

// Few rows (M <= 16 MT): the weights are read once, straight into MFMA
// operands, and that read is what bounds it.  A workgroup owns 16 outputs; its
// NW wavefronts take turns at blocks of 128 elements of K and add their sums
// in LDS, in a fixed order.
constexpr int kThinBlock = 128;

template <int MT, int NW, bool VEC>
__global__ void __launch_bounds__(64 * NW) thin_kernel(LinearArgs a) {
    constexpr int L = kThinBlock / 32;
    __shared__ f32x4 part[NW][MT][64];
    const gdn_linear_dims& d = a.d;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int64_t n0 = int64_t(blockIdx.x) * 16;
    const uint16_t* wp = static_cast<const uint16_t*>(a.w) + min(n0 + col, int64_t(d.N) - 1) * d.w_stride + 8 * g;
    const uint16_t* xp[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        xp[i] = static_cast<const uint16_t*>(a.x) + min(16 * i + col, d.M - 1) * d.x_stride + 8 * g;
    uint4 wf[L], xf[MT][L];
    auto load = [&](int k) {
#pragma unroll
        for (int j = 0; j < L; ++j) {
            if constexpr (VEC) {
                const bool in = k + 32 * j + 8 * g < d.K;
                wf[j] = in ? *reinterpret_cast<const uint4*>(wp + k + 32 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    xf[i][j] = in ? *reinterpret_cast<const uint4*>(xp[i] + k + 32 * j) : make_uint4(0, 0, 0, 0);
            } else {
                wf[j] = load_k8(wp, k + 32 * j, d.K - 8 * g);
#pragma unroll
                for (int i = 0; i < MT; ++i) xf[i][j] = load_k8(xp[i], k + 32 * j, d.K - 8 * g);
            }
        }
    };
    f32x4 acc[MT] = {};
    for (int k = wave * kThinBlock; k < d.K; k += NW * kThinBlock) {
        load(k);
#pragma unroll
        for (int j = 0; j < L; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i)
                acc[i] = mfma(__builtin_bit_cast(bf16x8, wf[j]), __builtin_bit_cast(bf16x8, xf[i][j]), acc[i]);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    for (int i = wave; i < MT; i += NW) {
        f32x4 s = part[0][i][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) s += part[w][i][lane];
        const int m = 16 * i + col;
        float v[4] = {s[0], s[1], s[2], s[3]};
        if (m < d.M) put<4, false>(a, m, n0 + 4 * g, v);
    }
}

template <int MT>
void launch_thin(const LinearArgs& a, bool vec, hipStream_t stream) {
    const int grid = (a.d.N + 15) / 16;
    if (vec)
        thin_kernel<MT, 8, true><<<grid, 512, 0, stream>>>(a);
    else
        thin_kernel<MT, 8, false><<<grid, 512, 0, stream>>>(a);
}

}  // namespace

size_t linear_ws_bytes(const gdn_linear_dims&) { return 0; }

hipError_t launch_linear(const LinearArgs& a, hipStream_t stream) {
    const gdn_linear_dims& d = a.d;
    // a tile's rows lie within 2^31 bytes of its first
    const bool direct = d.K % 8 == 0 && (d.M <= 1 || d.x_stride % 8 == 0) && (d.N <= 1 || d.w_stride % 8 == 0) &&
                        d.x_stride < (1 << 21) && d.w_stride < (1 << 21);
    const bool vec_out = d.N % 8 == 0 && (d.M <= 1 || (d.y_stride % 8 == 0 && (!a.res || d.res_stride % 8 == 0)));
    auto tiles = [&](int bm, int bn) { return ((d.M + bm - 1) / bm) * ((d.N + bn - 1) / bn); };
    if (d.M <= 16)
        launch_thin<1>(a, direct, stream);
    else if (d.M <= 32)
        launch_thin<2>(a, direct, stream);
    else if (d.M <= 64)
        launch_thin<4>(a, direct, stream);
    else if (tiles(256, 256) >= 256 && direct)
        tile_kernel<256, 256, 2, 4, true><<<tiles(256, 256), 512, 0, stream>>>(a, vec_out);
    else if (tiles(128, 128) >= 128 && direct)
        tile_kernel<128, 128, 2, 2, true><<<tiles(128, 128), 256, 0, stream>>>(a, vec_out);
    else if (direct)
        tile_kernel<64, 64, 2, 2, true><<<tiles(64, 64), 256, 0, stream>>>(a, vec_out);
    else
        tile_kernel<64, 64, 2, 2, false><<<tiles(64, 64), 256, 0, stream>>>(a, vec_out);
    return hipGetLastError();
}

}  // namespace gdn
