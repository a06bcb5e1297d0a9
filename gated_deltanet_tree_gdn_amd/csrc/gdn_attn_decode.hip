// gdn_attn_decode.hip -- softmax attention of one new token per sequence over
// a paged cache.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gdn_attn_internal.h"
#include "gdn_attn_plan.h"
#include "gdn_mfma.h"

namespace gdn {
namespace {

constexpr int kWaves = 4, kStep = 32;  // wavefronts of a workgroup, keys that one takes at a time
constexpr int kUnit = kDecodeUnit;

// Position of the 16-byte piece p of row r of a wavefront's V tile: a
// transposing read takes 32 bytes each of 8 rows at a time, which this spreads
// over all banks.
template <int D>
__device__ __forceinline__ int v_piece(int r, int p) {
    return r * (D / 8) + (p ^ (D >= 128 ? 2 * (r & 7) : 2 * (r >> 1 & 3)));
}

// ---------------------------------------------------------------------------
// A piece of a workgroup's range: some of one sequence's keys, one key head, up
// to 16 of its query heads.  Each wavefront takes a quarter of the keys, 32 at a
// time, with a running maximum and sum of its own; the four are joined at the end.
//   S^T = K Q^T   keys x heads on MFMA: K from memory straight as operand
//   O^T += V^T P  V through the wavefront's LDS rows, read transposed; the
//                 lanes hold P where the product wants it, since the k-slots
//                 of both operands may carry keys in any order
// P goes in as two bf16 (16 bits together), so that only the result is
// rounded to bf16.  What bounds it is memory: a step's loads are under way while
// the step before is worked on, 64 KB or more of each CU.  K goes to the operand
// registers without LDS, since nothing else reads it; steps of 64 keys of 64
// bytes (46 us) were no faster than of 32 (46) and left room for fewer
// wavefronts.  Measured: 96 sequences, 400009 tokens, 32 query and 8 key heads
// of 128, bf16: 309 us, 5.3 TB/s; one of 131071, 16 and 2 heads of 256: 47 us,
// 5.7 TB/s; one of 1531: 11 us, which is a launch and loads that wait for each
// other (length, table, keys); 24 of 200003 tokens, 24 and 4 heads of 64, e4m3:
// 40 us, 2.6 TB/s, as many instructions as bf16 for half the bytes.
// ---------------------------------------------------------------------------
template <int D, bool F8>
struct Step {
    static constexpr int T = kStep / 16;             // tiles of 16 keys
    static constexpr int E = F8 ? 16 : 8;            // elements of a 16-byte piece
    static constexpr int KL = D / (4 * E);           // loads of a K row's quarter
    static constexpr int VL = kStep * D / E / 64;    // loads of the V tile per lane
    static constexpr int VP = D / E;                 // pieces of a V row
    uint4 k[T][KL], v[VL];
    uint32_t ok;  // keys that are there

    static constexpr uint32_t kAll = ~uint32_t(0);

    __device__ __forceinline__ void load(const AttnArgs& a, PageWindow& window, const char* kp, const char* vp,
                                         const int32_t* table, int t0, int end, int lane) {
        constexpr int size = F8 ? 1 : 2;
        const int t = t0 + (lane & (kStep - 1));
        window.cover(table, t0 >> a.page_shift, (min(t0 + kStep, end) - 1) >> a.page_shift, lane);
        const int page = __shfl(window.ids, (min(t, end - 1) >> a.page_shift) - window.first);
        const bool there = t < end && page >= 0 && page < a.cache.n_pages;
        ok = uint32_t(__ballot(there));
        const int row = t & (a.cache.page_size - 1);
        // absent keys read the pool's first row
        const int64_t ko = there ? (page * a.cache.k_page_stride + row * a.cache.k_row_stride) * size : 0;
        const int64_t vo = there ? (page * a.cache.v_page_stride + row * a.cache.v_row_stride) * size : 0;
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const char* p = kp + __shfl(ko, 16 * j + (lane & 15)) + (lane >> 4) * 16;
#pragma unroll
            for (int i = 0; i < KL; ++i) k[j][i] = *reinterpret_cast<const uint4*>(p + i * 64);
        }
#pragma unroll
        for (int i = 0; i < VL; ++i) {
            const int r = (64 * i + lane) / VP;
            v[i] = *reinterpret_cast<const uint4*>(vp + __shfl(vo, r) + lane % VP * 16);
        }
    }

    // V into the wavefront's LDS rows; rows of absent keys are zero.
    __device__ __forceinline__ void store_v(uint4* lds, int lane) const {
#pragma unroll
        for (int i = 0; i < VL; ++i) {
            const int r = (64 * i + lane) / VP, p = lane % VP;
            uint4 x = v[i];
            if (ok != kAll && !(ok >> r & 1)) x = make_uint4(0, 0, 0, 0);
            if constexpr (F8) {
                uint4 lo, hi;
                e4m3_to_bf16(x, lo, hi);
                lds[v_piece<D>(r, 2 * p)] = lo;
                lds[v_piece<D>(r, 2 * p + 1)] = hi;
            } else {
                lds[v_piece<D>(r, p)] = x;
            }
        }
    }
};

// Column of the head's element j of k-slot group g in MFMA number n, as Step loads them.
template <int D, bool F8>
__device__ __forceinline__ int k_column(int n, int g) {
    return F8 ? (n >> 1) * 64 + g * 16 + (n & 1) * 8 : n * 32 + g * 8;
}

template <int D, bool F8>
__global__ __launch_bounds__(kWaves * 64, decode_per_cu(D, F8)) void decode_kernel(AttnArgs a) {
    constexpr int T = kStep / 16;
    __shared__ uint4 vlds[kWaves][kStep * D / 8];  // V by wavefront, then the wavefronts' O in fp32
    __shared__ float ml[kWaves][2][kDecodeRows];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    const float inf = __builtin_inff();
    AttnRange range;
    AttnPlace at;
    if (!attn_begin<kAttnDecode>(a, blockIdx.x, lane, range, at)) return;
    for (int64_t u = range.u; u < range.end;) {
        const int hh = int(quotient(u, range.units)), h = hh / a.head_tiles, head0 = (hh - h * a.head_tiles) * kDecodeRows;
        const int64_t uh = u - hh * range.units;
        attn_next<kAttnDecode>(a, uh, lane, at);
        const AttnSeq& s = at.s;
        const AttnPiece it = attn_piece<kAttnDecode>(a, s, 1, uh - at.first, range.end - u);
        const int rows = min(a.group - head0, kDecodeRows);
        const int64_t q_head = int64_t(h) * a.group + head0;
        constexpr int size = F8 ? 1 : 2;
        const char* kp = static_cast<const char*>(a.cache.k) + h * a.cache.k_head_stride * size;
        const char* vp = static_cast<const char*>(a.cache.v) + h * a.cache.v_head_stride * size;
        const float scale = a.d.scale * kLog2e * (a.cache.k_scale ? a.cache.k_scale[h] : 1.0f);
        const int begin = it.unit * kUnit, end = min(begin + it.units * kUnit, s.keys);
        const int32_t* table = a.table + at.b * a.d.table_stride;

        bf16x8 q[D / 32];
        const uint16_t* qp = a.q + at.b * a.d.q_stride + (q_head + min(col, rows - 1)) * D;
#pragma unroll
        for (int n = 0; n < D / 32; ++n) q[n] = load_frag(qp + k_column<D, F8>(n, g));

        f32x4 o[D / 16];
#pragma unroll
        for (int n = 0; n < D / 16; ++n) o[n] = f32x4{0, 0, 0, 0};
        float m = -inf, l = 0.0f;

        // the piece's steps in four runs of neighbours, so that a wavefront's pages are neighbours too
        const int steps = (end - begin + kStep - 1) / kStep, run = (steps + kWaves - 1) / kWaves;
        int t0 = begin + wave * run * kStep;
        const int stop = __builtin_amdgcn_readfirstlane(min(t0 + run * kStep, end));
        Step<D, F8> cur;
        PageWindow window;
        window.open(end, a.page_shift);
        if (t0 < stop) cur.load(a, window, kp, vp, table, t0, stop, lane);
        for (; t0 < stop; t0 += kStep) {
            cur.store_v(vlds[wave], lane);
            const uint32_t ok = cur.ok;
            f32x4 sc[T];
#pragma unroll
            for (int j = 0; j < T; ++j) {
                sc[j] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < Step<D, F8>::KL; ++i) {
                    if constexpr (F8) {
                        uint4 lo, hi;
                        e4m3_to_bf16(cur.k[j][i], lo, hi);
                        sc[j] = mfma(__builtin_bit_cast(bf16x8, lo), q[2 * i], sc[j]);
                        sc[j] = mfma(__builtin_bit_cast(bf16x8, hi), q[2 * i + 1], sc[j]);
                    } else {
                        sc[j] = mfma(__builtin_bit_cast(bf16x8, cur.k[j][i]), q[i], sc[j]);
                    }
                }
            }
            if (t0 + kStep < stop) cur.load(a, window, kp, vp, table, t0 + kStep, stop, lane);

            float x[4 * T], top = -inf;
#pragma unroll
            for (int j = 0; j < 4 * T; ++j) {
                x[j] = sc[j >> 2][j & 3] * scale;
                if (ok != Step<D, F8>::kAll && !(ok >> (16 * (j >> 2) + 4 * g + (j & 3)) & 1)) x[j] = -inf;
                top = fmaxf(top, x[j]);
            }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float m_new = fmaxf(m, top), base = finite_max(m_new);
            const float keep = exp2_fast(m - base);
            m = m_new;
            l *= keep;
#pragma unroll
            for (int j = 0; j < 4 * T; ++j) {
                x[j] = exp2_fast(x[j] - base);
                l += x[j];
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int n = 0; n < D / 16; ++n) o[n] *= keep;
            bf16x8 hi, lo;
            split8(x, hi, lo);
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                const int r = 4 * g + (col >> 2), p = 2 * n + ((col >> 1) & 1);
                const char* at0 = reinterpret_cast<const char*>(vlds[wave] + v_piece<D>(r, p)) + 8 * (col & 1);
                const char* at1 = reinterpret_cast<const char*>(vlds[wave] + v_piece<D>(r + 16, p)) + 8 * (col & 1);
                const uint2 y0 = read_tr16(lds_address(at0)), y1 = read_tr16(lds_address(at1));
                const bf16x8 vt = __builtin_bit_cast(bf16x8, make_uint4(y0.x, y0.y, y1.x, y1.y));
                o[n] = mfma(vt, lo, mfma(vt, hi, o[n]));
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }

        // the four wavefronts' parts, O as [head][4 elements], pieces permuted over the banks
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (lane < kDecodeRows) {
            ml[wave][0][lane] = m;
            ml[wave][1][lane] = l;
        }
        f32x4* mine = reinterpret_cast<f32x4*>(vlds[wave]);
#pragma unroll
        for (int n = 0; n < D / 16; ++n) mine[col * (D / 4) + ((4 * n + g) ^ (col & 7))] = o[n];
        __syncthreads();
        for (int i = tid; i < rows * (D / 4); i += kWaves * 64) {
            const int r = i / (D / 4), p = i % (D / 4);
            float top = -inf;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) top = fmaxf(top, ml[w][0][r]);
            f32x4 acc{0, 0, 0, 0};
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float f = exp2_fast(ml[w][0][r] - finite_max(top));
                acc += reinterpret_cast<f32x4*>(vlds[w])[r * (D / 4) + (p ^ (r & 7))] * f;
                sum += ml[w][1][r] * f;
            }
            if (it.units < it.all) {
                float* part = part_out(a, 2 * int64_t(range.w) + (u > range.u), kDecodeRows, D);
                reinterpret_cast<f32x4*>(part)[i] = acc;
                if (p == 0) {
                    part[kDecodeRows * D + r] = top;
                    part[kDecodeRows * (D + 1) + r] = sum;
                }
            } else {
                attn_store<D>(a, at.b, h, q_head + r, 4 * p, acc, sum);
            }
        }
        u += it.units;
        if (u < range.end) __syncthreads();  // the next piece overwrites what is joined here
    }
}

template <int D>
hipError_t launch(const AttnArgs& a, const dim3& grid, hipStream_t stream) {
    if (a.cache.dtype == GDN_E4M3)
        decode_kernel<D, true><<<grid, kWaves * 64, 0, stream>>>(a);
    else
        decode_kernel<D, false><<<grid, kWaves * 64, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_decode(const AttnArgs& a, hipStream_t stream) {
    const dim3 grid(attn_grid(a));
    switch (a.cache.d) {
        case 64: return launch<64>(a, grid, stream);
        case 128: return launch<128>(a, grid, stream);
        default: return launch<256>(a, grid, stream);
    }
}

}  // namespace gdn
