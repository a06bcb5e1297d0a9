// gdn_linear.hip -- y = residual + scale * act(x w^T + bias) on bf16 MFMA.
//
// Products run as w x^T: a lane's accumulators are then 4 adjacent outputs of
// one row of y.
//
//  - thin_kernel (at most 16 rows, few outputs): the weights straight from
//    memory into operands;
//  - tile_kernel: BM x BN outputs per workgroup, K in steps of 64 through LDS
//    buffers filled by direct loads while others are multiplied.
//
// Measured: 1 x 12352 x 4096 18 us with the 101 MB of weights partly in cache, 26 us
// with cold ones (3.9 TB/s); 1 x 4096 x 4096 9.7 us cold (3.5 TB/s);
// 777 x 4096 x 4096 with bias, silu and a residual 40 us (650 TFLOP/s: one round of 224
// tiles of 128 x 128 on 256 CUs, its loads ahead by a step); 16384 x 12352
// x 4096 1350 us (1230 TFLOP/s).  With 256 x 256 tiles LDS carries 256 KiB per
// step (192 read as operands, 64 written by the loads), 2,048 clocks, as many as
// the MFMAs take: the two compete, and the kernel without its loads takes three
// quarters of the time.  Steps of 32 (4% slower), wavefronts of 128 x 128 (spills)
// and wavefronts in opposite phases (7% slower) did not help.

#include <algorithm>
#include <cmath>

#include "gdn_layer_internal.h"
#include "gdn_layer_util.h"
#include "gdn_mfma.h"

namespace gdn {
namespace {

constexpr int kBK = 64;  // elements of K per step of the tile kernel

// Outputs n .. n + E - 1 of row m, those below N: bias, activation, scale and
// residual in fp32, rounded once.
template <int E>
__device__ __forceinline__ void put(const LinearArgs& a, int64_t m, int n, float (&v)[E]) {
    const gdn_linear_dims& d = a.d;
    const bool whole = E == 8 && n + 8 <= d.N;
    float b[E] = {}, r[E] = {};
    if (whole) {
        if constexpr (E == 8) {
            if (a.bias) load8(a.bias, GDN_F32, n, b);
            if (a.res) load8(a.res, d.res_dtype, m * d.res_stride + n, r);
        }
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
    if (whole) {
        if constexpr (E == 8) store8(a.y, d.y_dtype, m * d.y_stride + n, v);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (n + e < d.N) store1(a.y, d.y_dtype, m * d.y_stride + n + e, v[e]);
    }
}

// Tiles of `size` that n rows or outputs (one or more, up to 2^31 - 1) need.
__host__ __device__ constexpr int tiles_of(int n, int size) { return (n - 1) / size + 1; }

// Workgroups go to the 8 XCDs in turn; here each XCD gets a run of
// consecutive tiles, ordered in bands of 8 tile rows, so that the tiles it has
// in flight share rows of x and w in its L2.
__device__ __forceinline__ int xcd_run(int id, int total) {
    const int q = total / 8, r = total % 8, xcd = id % 8;
    return xcd * q + min(xcd, r) + id / 8;
}
__device__ __forceinline__ void tile_at(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
    constexpr int kBand = 8;
    const int band = t / (kBand * tiles_n), in = t - band * kBand * tiles_n, rows = min(kBand, tiles_m - band * kBand);
    tm = band * kBand + in % rows;
    tn = in / rows;
}

typedef __attribute__((address_space(3))) void* lds_ptr;

// 8 elements k .. k + 7 of a row of K, zeros past its end; rows of any alignment.
__device__ __forceinline__ uint4 load_k8(const uint16_t* row, int k, int K) {
    typedef uint32_t u32x4a2 __attribute__((ext_vector_type(4), aligned(2)));
    if (k + 8 <= K) return __builtin_bit_cast(uint4, *reinterpret_cast<const u32x4a2*>(row + k));
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = k + j < K ? row[k + j] : 0u;
    return make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
}

// Direct loads of ROWS rows of x or w by kBK elements of K into LDS.  Piece p
// (16 bytes) of row r sits at position p ^ (r & 7) of its row, which spreads
// the rows of a fragment read over the banks.  One load of a wavefront fills
// 8 rows (LDS addresses run with the lanes), so the permutation is made in the
// global address.
template <int ROWS, int WAVES>
struct Stage {
    static constexpr int L = ROWS / 8 / WAVES;  // loads per wavefront
    const uint16_t* base;  // of the first row
    uint32_t off[L];
    __device__ __forceinline__ void init(const uint16_t* p, int64_t stride, int64_t row0, int64_t rows, int wave,
                                         int lane) {
        base = p + row0 * stride;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int r = (wave * L + i) * 8 + (lane >> 3);
            const uint32_t row = min(int64_t(r), rows - 1 - row0);
            off[i] = (row * uint32_t(stride) + 8 * ((lane & 7) ^ (r & 7))) * 2;
        }
    }
    // Pieces from `pieces` on repeat the last one before: K ends there.
    template <bool TAIL>
    __device__ __forceinline__ void load(uint4* lds, int k, int pieces, int wave, int lane) const {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass rejects the 16-byte form
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base), 0, 0x7fffffff, 0x00027000);
        const uint32_t back = !TAIL ? 0 : max(((lane & 7) ^ (lane >> 3)) - (pieces - 1), 0) * 16;
#pragma unroll
        for (int i = 0; i < L; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)(lds + (wave * L + i) * 64), 16, off[i] - back, k * 2,
                                                     0, 0);
#endif
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

// KG groups of WM x WN wavefronts; a wavefront has (BM / WM) x (BN / WN)
// outputs.  The groups take turns at the steps of K, each through its own NB
// LDS buffers, and add their sums at the end in a fixed order: with few tiles
// that keeps KG times as many loads in flight on a CU.
template <int BM, int BN, int WM, int WN, int KG, int NB>
constexpr int tile_lds_bytes() {
    constexpr int W = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int out = W * (TM > 4 ? 64 : TM * 16) * (TN * 16 + 4) * 4;
    return std::max({KG * (BM + BN) * 8 * NB * 16, out, (KG - 1) * W * TM * TN * 1024});
}

// DIRECT: rows in whole 16-byte pieces; TAIL: K is not a multiple of 64 (looking
// after the last step costs every step 2 to 4 %).
template <int BM, int BN, int WM, int WN, int KG, int NB, bool DIRECT, bool TAIL>
__device__ __forceinline__ void tile(const LinearArgs& a, char* lds, int64_t m0, int64_t n0) {
    constexpr int W = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int kOutRows = TM > 4 ? 64 : TM * 16, kOutLd = TN * 16 + 4;  // epilogue: rows of a wavefront at a time
    constexpr int kGroupPieces = (BM + BN) * 8 * NB;
    const gdn_linear_dims& d = a.d;
    const int lane = threadIdx.x & 63, all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave = all % W, grp = all / W, col = lane & 15, g = lane >> 4;
    auto xs = [&](int p) { return reinterpret_cast<uint4*>(lds) + grp * kGroupPieces + p * BM * 8; };
    auto ws = [&](int p) { return reinterpret_cast<uint4*>(lds) + grp * kGroupPieces + (NB * BM + p * BN) * 8; };
    const int wm = wave % WM, wn = wave / WM;
    const uint16_t* xp = static_cast<const uint16_t*>(a.x);
    const uint16_t* wp = static_cast<const uint16_t*>(a.w);
    f32x4 acc[TN][TM] = {};
    struct Frags {
        bf16x8 x[TM], w[TN];
    };
    auto read = [&](Frags& f, int p, int s) {  // 32 elements of K of buffer p
        const uint4 *x = xs(p), *w = ws(p);
        const int at = (4 * s + g) ^ (col & 7);
#pragma unroll
        for (int i = 0; i < TM; ++i) f.x[i] = __builtin_bit_cast(bf16x8, x[((wm * TM + i) * 16 + col) * 8 + at]);
#pragma unroll
        for (int j = 0; j < TN; ++j) f.w[j] = __builtin_bit_cast(bf16x8, w[((wn * TN + j) * 16 + col) * 8 + at]);
    };
    auto multiply = [&](const Frags& f) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int i = 0; i < TM; ++i) acc[j][i] = mfma(f.w[j], f.x[i], acc[j][i]);
    };
    auto any_step = [&](int k) {  // all groups stage, one multiplies the end of K
        stage_any<BM, W>(xs(0), xp, d.x_stride, m0, d.M, k, d.K, wave, lane);
        stage_any<BN, W>(ws(0), wp, d.w_stride, n0, d.N, k, d.K, wave, lane);
        __syncthreads();
        Frags f;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            read(f, 0, s);
            multiply(f);
        }
        __syncthreads();
    };
    if constexpr (DIRECT) {
        // Whole pieces of 8 elements go through the pipeline; where the last step has
        // fewer than 8 of them, its operands are cleared from there on (both: what the
        // loads bring instead may be infinite).
        const bool whole = !TAIL || d.K % 8 == 0;
        const int steps = TAIL && whole ? (d.K + kBK - 1) / kBK : d.K / kBK;
        const int last = TAIL && whole ? d.K % kBK / 8 : 8;
        auto finish = [&](Frags& f, int t, int s) {
            if (TAIL && t == steps - 1 && 4 * s + g >= last) {
#pragma unroll
                for (int i = 0; i < TM; ++i) f.x[i] = bf16x8{};
#pragma unroll
                for (int j = 0; j < TN; ++j) f.w[j] = bf16x8{};
            }
        };
        if (steps > 0) {
            Stage<BM, W> sx;
            Stage<BN, W> sw;
            sx.init(xp, d.x_stride, m0, d.M, wave, lane);
            sw.init(wp, d.w_stride, n0, d.N, wave, lane);
            // This group's steps are grp, grp + KG, ..; every group goes through as
            // many rounds.  Loads run NB - 1 rounds ahead.
            const int rounds = (steps + KG - 1) / KG;
            auto load = [&](int round) {
                const int t = round * KG + grp, p = round % NB;
                if (t < steps) {
                    const int pieces = t == steps - 1 ? last : 8;
                    sx.template load<TAIL>(xs(p), t * kBK, pieces, wave, lane);
                    sw.template load<TAIL>(ws(p), t * kBK, pieces, wave, lane);
                }
            };
#pragma unroll
            for (int r = 0; r < NB - 1; ++r) load(r);
            loads_barrier<0>();
            constexpr int L = Stage<BM, W>::L + Stage<BN, W>::L;
            if constexpr (NB == 2) {
                for (int r = 0; r < rounds; ++r) {
                    load(r + 1);
                    if (KG == 1 || r * KG + grp < steps) {
                        Frags f;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            read(f, r & 1, s);
                            finish(f, r * KG + grp, s);
                            multiply(f);
                        }
                    }
                    loads_barrier<0>();
                }
            } else {
                // Operands are read half a step ahead, the first of a round before
                // the barrier that ends the round before it: at that barrier the
                // round after next has arrived, that is, only the NB - 3 rounds
                // behind it are outstanding (as long as they were issued by all
                // groups: grp < KG loaded step (r + NB - 1) KG + grp if
                // (r + NB) KG <= steps).  A group whose last round has no step
                // multiplies what is left in its buffer into nothing.
                Frags f0, f1;
                read(f0, 0, 0);
                for (int r = 0, p = 0; r < rounds; ++r) {
                    const int next = p + 1 == NB ? 0 : p + 1;
                    const bool mine = KG == 1 || r * KG + grp < steps;
                    load(r + NB - 1);
                    read(f1, p, 1);
                    __builtin_amdgcn_sched_barrier(0);
                    finish(f0, r * KG + grp, 0);
                    if (mine) multiply(f0);
                    __builtin_amdgcn_sched_barrier(0);
                    read(f0, next, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    finish(f1, r * KG + grp, 1);
                    if (mine) multiply(f1);
                    __builtin_amdgcn_sched_barrier(0);
                    if ((r + NB) * KG <= steps)
                        loads_barrier<(NB - 3) * L, false>();
                    else
                        loads_barrier<0, false>();
                    p = next;
                }
                loads_barrier<0>();
            }
        }
        // the end of K in elements: past it both operands are staged as zeros, so
        // every group but the first adds nothing
        if (TAIL && !whole) any_step(grp == 0 ? d.K / kBK * kBK : d.K);
    } else {
        for (int k = 0; k < d.K; k += kBK * KG) any_step(k + grp * kBK);
    }
    if constexpr (KG > 1) {
        f32x4* sums = reinterpret_cast<f32x4*>(lds);
        if (grp > 0)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    sums[(((grp - 1) * W + wave) * TN * TM + j * TM + i) * 64 + lane] = acc[j][i];
        __syncthreads();
        if (grp == 0)
#pragma unroll
            for (int q = 0; q < KG - 1; ++q)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int i = 0; i < TM; ++i) acc[j][i] += sums[((q * W + wave) * TN * TM + j * TM + i) * 64 + lane];
        __syncthreads();
        if (grp > 0) return;
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
            if (m < d.M && n < d.N) put<8>(a, m, n, v);
        }
    }
}

template <int BM, int BN, int WM, int WN, int KG, int NB, bool DIRECT, bool TAIL>
__global__ void __launch_bounds__(64 * WM * WN * KG) tile_kernel(LinearArgs a) {
    __shared__ __align__(16) char lds[tile_lds_bytes<BM, BN, WM, WN, KG, NB>()];
    const int tiles_m = tiles_of(a.d.M, BM), tiles_n = tiles_of(a.d.N, BN), id = int(block_id());
    if (id >= tiles_m * tiles_n) return;
    int tm, tn;
    tile_at(xcd_run(id, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
    tile<BM, BN, WM, WN, KG, NB, DIRECT, TAIL>(a, lds, int64_t(tm) * BM, int64_t(tn) * BN);
}

// The first `whole` tiles of 256 x 256 as such, the rest in quarters, with two
// groups over K each: what does not fill a round of CUs then takes a third of a
// round for 64 tiles or fewer, two thirds for 128.  In quarters and as another
// round: 4096 x 12352 x 4096 (16 tiles over) 356 and 442 us, 5000 x 4096 x 4096 (64)
// 141 and 163, 6000 x 4096 x 4096 (128) 179 and 182.
template <bool TAIL>
__global__ void __launch_bounds__(512) tile256_kernel(LinearArgs a, int whole) {
    __shared__ __align__(16) char
        lds[std::max(tile_lds_bytes<256, 256, 2, 4, 1, 2>(), tile_lds_bytes<128, 128, 2, 2, 2, 2>())];
    const int tiles_m = tiles_of(a.d.M, 256), tiles_n = tiles_of(a.d.N, 256), id = int(block_id());
    if (id >= whole + 4 * (tiles_m * tiles_n - whole)) return;
    int tm, tn;
    if (id < whole) {
        tile_at(xcd_run(id, whole), tiles_m, tiles_n, tm, tn);
        tile<256, 256, 2, 4, 1, 2, true, TAIL>(a, lds, int64_t(tm) * 256, int64_t(tn) * 256);
    } else {
        const int u = xcd_run(id - whole, 4 * (tiles_m * tiles_n - whole));
        tile_at(whole + (u >> 2), tiles_m, tiles_n, tm, tn);
        const int64_t m0 = int64_t(tm) * 256 + (u & 1) * 128, n0 = int64_t(tn) * 256 + (u >> 1 & 1) * 128;
        if (m0 < a.d.M && n0 < a.d.N) tile<128, 128, 2, 2, 2, 2, true, TAIL>(a, lds, m0, n0);
    }
}

// At most 16 rows: the weights are read once, straight into MFMA operands, and
// that read is what bounds it.  A workgroup owns 16 outputs; its wavefronts take
// turns at blocks of 128 elements of K and add their sums in LDS, in a fixed
// order.
constexpr int kThinBlock = 128, kThinWaves = 8;

template <bool VEC>
__global__ void __launch_bounds__(64 * kThinWaves) thin_kernel(LinearArgs a) {
    constexpr int L = kThinBlock / 32;
    __shared__ f32x4 part[kThinWaves][64];
    const gdn_linear_dims& d = a.d;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int64_t n0 = int64_t(blockIdx.x) * 16;
    const uint16_t* wp = static_cast<const uint16_t*>(a.w) + min(n0 + col, int64_t(d.N) - 1) * d.w_stride + 8 * g;
    const uint16_t* xp = static_cast<const uint16_t*>(a.x) + int64_t(min(col, d.M - 1)) * d.x_stride + 8 * g;
    f32x4 acc = {};
    for (int k = wave * kThinBlock; k < d.K; k += kThinWaves * kThinBlock) {
        uint4 wf[L], xf[L];
#pragma unroll
        for (int j = 0; j < L; ++j) {
            if constexpr (VEC) {
                const bool in = k + 32 * j + 8 * g < d.K;
                wf[j] = in ? *reinterpret_cast<const uint4*>(wp + k + 32 * j) : make_uint4(0, 0, 0, 0);
                xf[j] = in ? *reinterpret_cast<const uint4*>(xp + k + 32 * j) : make_uint4(0, 0, 0, 0);
            } else {
                wf[j] = load_k8(wp, k + 32 * j, d.K - 8 * g);
                xf[j] = load_k8(xp, k + 32 * j, d.K - 8 * g);
            }
        }
#pragma unroll
        for (int j = 0; j < L; ++j)
            acc = mfma(__builtin_bit_cast(bf16x8, wf[j]), __builtin_bit_cast(bf16x8, xf[j]), acc);
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave == 0 && col < d.M) {
#pragma unroll
        for (int w = 1; w < kThinWaves; ++w) acc += part[w][lane];
        float v[4] = {acc[0], acc[1], acc[2], acc[3]};
        put<4>(a, col, n0 + 4 * g, v);
    }
}

void launch_thin(const LinearArgs& a, bool vec, hipStream_t stream) {
    const int grid = (a.d.N + 15) / 16;
    if (vec)
        thin_kernel<true><<<grid, 64 * kThinWaves, 0, stream>>>(a);
    else
        thin_kernel<false><<<grid, 64 * kThinWaves, 0, stream>>>(a);
}

template <int BM, int BN, int WM, int WN, int KG, int NB, bool DIRECT>
void launch_tile(const LinearArgs& a, bool tail, hipStream_t stream) {
    const dim3 grid = grid_of(int64_t(tiles_of(a.d.M, BM)) * tiles_of(a.d.N, BN));
    constexpr int threads = 64 * WM * WN * KG;
    if (DIRECT && tail)
        tile_kernel<BM, BN, WM, WN, KG, NB, DIRECT, DIRECT><<<grid, threads, 0, stream>>>(a);
    else
        tile_kernel<BM, BN, WM, WN, KG, NB, DIRECT, false><<<grid, threads, 0, stream>>>(a);
}

void launch_tile256(const LinearArgs& a, bool tail, int cut, hipStream_t stream) {
    const int whole = tiles_of(a.d.M, 256) * tiles_of(a.d.N, 256) - cut;
    const dim3 grid = grid_of(whole + 4 * int64_t(cut));
    if (tail)
        tile256_kernel<true><<<grid, 512, 0, stream>>>(a, whole);
    else
        tile256_kernel<false><<<grid, 512, 0, stream>>>(a, whole);
}

// Rows of any alignment to rows of 16-byte pieces.
__global__ void __launch_bounds__(256) pack_kernel(const uint16_t* src, int64_t stride, int64_t rows, int K, uint4* dst) {
    const int per = (K + 7) / 8;
    const int64_t n = rows * per, step = int64_t(gridDim.x) * 256;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) {
        const int64_t r = i / per;
        const int k = int(i - r * per) * 8;
        dst[i] = load_k8(src + r * stride, k, K);
    }
}

// Which operand rows do not start on 16 bytes, and whether copying those pays:
// the tile kernel on such rows stages them through registers at 8.8e-9 us per
// multiply-add (8192 x 8192 x 4095: 2411 us) instead of 1.6e-9, a copy costs
// 0.9e-6 us per element, so it pays where M N / (M + N) exceeds about 125.
struct Packing {
    bool x, w;  // not aligned
    bool copy;
};
Packing packing(const gdn_linear_dims& d) {
    Packing p;
    p.x = d.M > 1 && d.x_stride % 8 != 0;
    p.w = d.N > 1 && d.w_stride % 8 != 0;
    p.copy = (p.x || p.w) && d.K > 0 && double(d.M) * d.N > 125.0 * (double(d.M) + d.N);
    return p;
}
size_t packed_bytes(int64_t rows, int K) { return (size_t(rows) * ((size_t(K) + 7) / 8) * 16 + 255) & ~size_t(255); }

void launch_pack(const void* src, int64_t stride, int64_t rows, int K, void* dst, hipStream_t stream) {
    const int64_t blocks = (rows * ((K + 7) / 8) + 255) / 256;
    pack_kernel<<<static_cast<unsigned>(blocks < 8192 ? blocks : 8192), 256, 0, stream>>>(
        static_cast<const uint16_t*>(src), stride, rows, K, static_cast<uint4*>(dst));
}

}  // namespace

size_t linear_ws_bytes(const gdn_linear_dims& d) {
    const Packing p = packing(d);
    return p.copy ? (p.x ? packed_bytes(d.M, d.K) : 0) + (p.w ? packed_bytes(d.N, d.K) : 0) : 0;
}

LinearChoice linear_choice(const gdn_linear_dims& d) {
    const Packing p = packing(d);
    const int64_t packed = (int64_t(d.K) + 7) / 8 * 8;                  // a copied row
    const int K = p.copy && p.x && p.w ? int(packed) : d.K;  // the copies end in zeros
    const bool aligned = p.copy || !(p.x || p.w);
    // direct loads: a tile's rows lie within 2^31 bytes of its first
    auto near = [&](bool copied, int64_t stride) { return (copied ? packed : stride) < (1 << 21); };
    const bool direct = aligned && near(p.copy && p.x, d.x_stride) && near(p.copy && p.w, d.w_stride);
    auto tiles = [&](int64_t t) { return double((d.M + t - 1) / t) * double((d.N + t - 1) / t); };
    // What each kernel takes in us, a part that grows with K and one that does not
    // (start and epilogue), fitted to measurements at K = 256, 1024 and 4096 over M
    // = 64 .. 16384, N = 1024 .. 12352.
    const double k = K / 4096.0, t64 = tiles(64), t128 = tiles(128), t256 = tiles(256);
    // 256 KiB of loads in flight per CU: few tiles
    const double k64two = (2.4 + 15.5 * k) * std::ceil(t64 / 256);
    // two workgroups per CU
    const double k64 = std::max(2.0 + 18.0 * k, (0.005 + 0.0516 * k) * t64);
    // one round of tiles, two groups per CU
    const double k128two = t128 <= 256 ? 7.8 + 34.5 * k : 1e30;
    // two workgroups per CU, rounds of 512 tiles
    const double k128 = std::max(6.5 + 42.0 * k, (6.0 + 59.0 * k) * std::ceil(t128 / 512));
    // fewest bytes through LDS per product; rounds of 256 tiles, and up to half a round
    // of tiles over whole ones in quarters (their start overlaps the end of the round
    // before)
    const double full = std::floor(t256 / 256), over = t256 - 256 * full;
    const bool cut = full > 0 && over > 0 && over <= 128;
    const double part = cut ? 34.5 * k * std::ceil(over / 64) : 11.0 + (75.0 + 25.0 * over / 256) * k;
    const double k256 = 2.0 + (11.0 + 100.0 * k) * full + (over > 0 ? part : 0.0);
    const double best = std::min({k64two, k64, k128two, k128, k256});
    const bool tail = K % kBK != 0;
    // One tile of 16 rows is all that the thin kernel multiplies, and it reads x again for
    // every 16 outputs, which many outputs make dearer than tiles.  Thin and tiles, cold
    // weights, in us: K 4096, N 256: 6.9 and 14.4 (1 row), 9.5 and 14.4 (16 rows); N
    // 8192: 16.6 and 23.2, 23.3 and 23.8; N 10240: 21.2 and 24.5, 31.1 and 24.9; N 12352:
    // 25.7 and 26.3, 38.9 and 26.7.  K 1024, N 8192: 6.1 and 8.8, 8.1 and 9.0; N 12352:
    // 7.9 and 9.2, 11.4 and 9.4.
    if (d.M <= 16 && d.N <= 8192) return {kThin, !aligned || K % 8 != 0, 0};
    if (!direct) return {kTileAny, true, 0};
    if (best == k64two) return {kTile64Two, tail, 0};
    if (best == k64) return {kTile64, tail, 0};
    if (best == k128two) return {kTile128Two, tail, 0};
    if (best == k128) return {kTile128, tail, 0};
    return {kTile256, tail, cut ? int(over) : 0};
}

hipError_t launch_linear(const LinearArgs& args, hipStream_t stream) {
    LinearArgs a = args;
    gdn_linear_dims& d = a.d;
    const LinearChoice c = linear_choice(d);
    const Packing p = packing(d);
    if (p.copy) {
        char* ws = static_cast<char*>(a.ws);
        if (p.x) {
            launch_pack(a.x, d.x_stride, d.M, d.K, ws, stream);
            a.x = ws;
            d.x_stride = (int64_t(d.K) + 7) / 8 * 8;
            ws += packed_bytes(d.M, d.K);
        }
        if (p.w) {
            launch_pack(a.w, d.w_stride, d.N, d.K, ws, stream);
            a.w = ws;
            d.w_stride = (int64_t(d.K) + 7) / 8 * 8;
        }
        if (p.x && p.w) d.K = int(d.x_stride);  // the copies end in zeros
    }
    switch (c.kernel) {
        case kThin: launch_thin(a, !c.tail, stream); break;
        case kTileAny: launch_tile<64, 64, 2, 2, 4, 2, false>(a, false, stream); break;
        case kTile64Two: launch_tile<64, 64, 2, 2, 2, 4, true>(a, c.tail, stream); break;
        case kTile64: launch_tile<64, 64, 2, 2, 1, 4, true>(a, c.tail, stream); break;
        case kTile128Two: launch_tile<128, 128, 2, 2, 2, 2, true>(a, c.tail, stream); break;
        case kTile128: launch_tile<128, 128, 2, 4, 1, 2, true>(a, c.tail, stream); break;
        case kTile256: launch_tile256(a, c.tail, c.cut, stream); break;
    }
    return hipGetLastError();
}

}  // namespace gdn
