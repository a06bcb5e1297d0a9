// gdn_attn_tiles.hip -- softmax attention of many queries per sequence over a
// paged cache: packed prompts and proposal trees.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gdn_attn_internal.h"
#include "gdn_attn_plan.h"

namespace gdn {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kKeys = 64;  // keys of a tile in LDS

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mfma32(const bf16x8& a, const bf16x8& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Positions of the 16-byte piece p of row r in LDS.  K is read 16 rows of one
// piece at a time, V transposed, 4 rows of four adjacent pieces at a time; both
// spread over all banks.
template <int D>
__device__ __forceinline__ int k_piece(int r, int p) {
    return r * (D / 8) + (p ^ (D >= 128 ? r & 15 : r >> 1 & 7));
}
template <int D>
__device__ __forceinline__ int v_piece(int r, int p) {
    return r * (D / 8) + (p ^ (D >= 128 ? 4 * (r & 3) : 4 * (r >> 1 & 1)));
}

template <int D>
struct TileLds {
    uint4 k[2][kKeys * D / 8], v[2][kKeys * D / 8];
};

// A tile's rows on their way from memory to LDS.
template <int D, bool F8>
struct Stage {
    static constexpr int E = F8 ? 16 : 8;                  // elements of a 16-byte piece
    static constexpr int P = D / E;                        // pieces of a row
    static constexpr int L = kKeys * P / kThreads;         // pieces of a thread
    static constexpr int size = F8 ? 1 : 2;
    int page[L];
    uint4 k[L], v[L];

    // Pages of the tile's tokens; -1 where there is none.
    __device__ __forceinline__ void pages(const AttnArgs& a, const int32_t* table, int t0, int end, int tid) {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int t = t0 + (kThreads * i + tid) / P;
            page[i] = -1;
            if (t < end) page[i] = table[t >> a.page_shift];
        }
    }
    __device__ __forceinline__ void load(const AttnArgs& a, const char* kp, const char* vp, int t0, int tid) {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int row = (t0 + (kThreads * i + tid) / P) & (a.cache.page_size - 1);
            k[i] = v[i] = make_uint4(0, 0, 0, 0);
            if (page[i] >= 0 && page[i] < a.cache.n_pages) {
                const int at = tid % P * 16;
                k[i] = *reinterpret_cast<const uint4*>(
                    kp + (page[i] * a.cache.k_page_stride + row * a.cache.k_row_stride) * size + at);
                v[i] = *reinterpret_cast<const uint4*>(
                    vp + (page[i] * a.cache.v_page_stride + row * a.cache.v_row_stride) * size + at);
            }
        }
    }
    // With `check`, returns whether a value among the thread's is not finite.
    __device__ __forceinline__ bool store(uint4* klds, uint4* vlds, int tid, bool check) const {
        bool odd = false;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int r = (kThreads * i + tid) / P, p = tid % P;
            uint4 x[2] = {v[i]};
            if constexpr (F8) {
                uint4 y[2];
                e4m3_to_bf16(k[i], y[0], y[1]);
                klds[k_piece<D>(r, 2 * p)] = y[0];
                klds[k_piece<D>(r, 2 * p + 1)] = y[1];
                e4m3_to_bf16(v[i], x[0], x[1]);
                vlds[v_piece<D>(r, 2 * p)] = x[0];
                vlds[v_piece<D>(r, 2 * p + 1)] = x[1];
            } else {
                klds[k_piece<D>(r, p)] = k[i];
                vlds[v_piece<D>(r, p)] = x[0];
            }
            if (!check) continue;
#pragma unroll
            for (int j = 0; j < (F8 ? 2 : 1); ++j) {
                const uint32_t u[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    odd |= (u[w] & 0x7f80u) == 0x7f80u || (u[w] & 0x7f800000u) == 0x7f800000u;
            }
        }
        return odd;
    }
};

// Bits of the 32 tokens from t0 on that the query may see.
template <AttnKind KIND>
__device__ __forceinline__ uint32_t visible(const AttnArgs& a, const AttnSeq& s, int token, const uint32_t* anc, int t0,
                                            int end) {
    // number of tokens from t0 on that a bound leaves, as bits
    auto below = [&](int bound) {
        const int n = bound - t0;
        return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1;
    };
    if constexpr (KIND == kAttnPrefill) {
        return below(min(s.prefix + token + 1, end));
    } else {
        const int first = t0 - s.prefix;  // node of token t0
        const int W = (a.d.T + 31) >> 5;
        auto word = [&](int w) -> uint32_t {
            if (w < 0) return 0xffffffffu;
            if (w >= W) return 0u;
            uint32_t u = anc[w];
            if (w == W - 1 && (a.d.T & 31)) u &= (1u << (a.d.T & 31)) - 1;
            return u;
        };
        const int w = first >> 5, shift = first & 31;
        uint32_t u = word(w) >> shift;
        if (shift) u |= word(w + 1) << (32 - shift);
        return u & below(end);
    }
}

// V's elements that are not finite, as ones: of kind 0 NaN, 1 +inf, 2 -inf.
__device__ __forceinline__ uint32_t marks_of(uint32_t u, int kind) {
    uint32_t r = 0;
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
        const uint32_t x = u >> h & 0xffff;
        const bool is = kind == 0 ? (x & 0x7fff) > 0x7f80 : x == (kind == 1 ? 0x7f80u : 0xff80u);
        if (is) r |= 0x3f80u << h;
    }
    return r;
}
// V's elements with zeros for those.
__device__ __forceinline__ uint32_t finite_of(uint32_t u) {
    if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
    if ((u & 0x7f800000u) == 0x7f800000u) u &= 0xffffu;
    return u;
}

// ---------------------------------------------------------------------------
// One workgroup: one chunk of one sequence's keys, one key head, 128 rows
// (token, query head of the group); a wavefront has 32 of the rows.  64 keys
// at a time lie in LDS, the next 64 on their way there.
//   S^T = K Q^T    keys x rows on MFMA, Q in registers for the whole chunk
//   O^T += V^T P   V read transposed; the lanes hold P where the product wants it
// The running maximum is raised only where a row's scores pass it by more than
// 2^8: P then stays below 2^8, which costs no precision in floating point, and
// O is rarely rescaled.  P is rounded to bf16 for the product (its sum is not):
// 2^-9 of every weight, as much as the output's own rounding.
// A masked key has P = 0, but 0 times an infinity or NaN of its value would not
// be 0: a tile with masked keys and such values is multiplied with zeros in
// their place, and the rows that do see them get them from products of marks.
// ---------------------------------------------------------------------------
template <AttnKind KIND, int D, bool F8>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void tiles_kernel(AttnArgs a) {
    extern __shared__ uint4 lds_raw[];
    TileLds<D>& lds = *reinterpret_cast<TileLds<D>*>(lds_raw);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int heads = a.cache.H_kv;
    const int64_t wg = block_id(), grid_items = int64_t(gridDim.x) * gridDim.y / heads;
    if (wg >= grid_items * heads) return;
    const int h = int(wg % heads);
    const int c = attn_chunk<KIND>(a, lane);
    constexpr int size = F8 ? 1 : 2;
    const char* kp = static_cast<const char*>(a.cache.k) + h * a.cache.k_head_stride * size;
    const char* vp = static_cast<const char*>(a.cache.v) + h * a.cache.v_head_stride * size;
    const float scale = a.d.scale * kLog2e * (a.cache.k_scale ? a.cache.k_scale[h] : 1.0f);
    const float inf = __builtin_inff();

    AttnItem it;
    for (int64_t item = wg / heads; attn_item<KIND, false>(a, c, item, lane, it); item += grid_items) {
        const AttnSeq s = attn_seq<KIND>(a, it.b);
        const int all_rows = s.n * a.group;
        const int row0 = it.tile * kTileRows, rows = min(kTileRows, all_rows - row0);
        // the last of the tile's tokens sees most
        const int last_token = (row0 + rows - 1) / a.group;
        const int begin = it.chunk * c;
        const int seen = KIND == kAttnPrefill ? min(max(s.prefix + last_token + 1, 0), s.keys) : s.keys;
        const int end = min(begin + c, seen);
        const int chunks = max((seen + c - 1) / c, 1);  // of this tile
        if (it.chunk >= chunks) continue;

        const int my_row = min(row0 + wave * 32 + col, all_rows - 1);
        const int token = my_row / a.group, head = h * a.group + my_row - token * a.group;
        const uint32_t* anc =
            KIND == kAttnVerify ? a.anc + (int64_t(it.b) * s.n + token) * ((a.d.T + 31) >> 5) : nullptr;
        const int32_t* table = a.table + it.b * a.d.table_stride;
        // tokens from here on are masked for some of the tile's rows
        const int open_end = KIND == kAttnPrefill ? s.prefix + row0 / a.group + 1 : s.prefix;

        bool missing = false;  // pages outside the pool
        for (int p = (begin >> a.page_shift) + tid; begin < end && p <= (end - 1) >> a.page_shift; p += kThreads) {
            const int page = table[p];
            missing |= page < 0 || page >= a.cache.n_pages;
        }
        missing = __syncthreads_or(missing);
        auto is_masked = [&](int t0) { return missing || t0 + kKeys > min(open_end, end); };

        bf16x8 q[D / 16];
        const uint16_t* qp = a.q + (s.row0 + token) * a.d.q_stride + int64_t(head) * D + 8 * half;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) q[n] = load_frag(qp + 16 * n);

        f32x16 o[D / 32];
#pragma unroll
        for (int n = 0; n < D / 32; ++n)
#pragma unroll
            for (int j = 0; j < 16; ++j) o[n][j] = 0.0f;
        float m = -inf, l = 0.0f;  // m: what the powers are taken against

        Stage<D, F8> st;
        int odd = 0;
        if (begin < end) {
            st.pages(a, table, begin, end, tid);
            st.load(a, kp, vp, begin, tid);
            st.pages(a, table, begin + kKeys, end, tid);
            odd = __syncthreads_or(st.store(lds.k[0], lds.v[0], tid, is_masked(begin)));
        }
        for (int t0 = begin, buf = 0; t0 < end; t0 += kKeys, buf ^= 1) {
            const bool more = t0 + kKeys < end;
            if (more) {
                st.load(a, kp, vp, t0 + kKeys, tid);
                st.pages(a, table, t0 + 2 * kKeys, end, tid);
            }
            const bool masked = is_masked(t0);
            uint32_t see[2] = {0xffffffffu, 0xffffffffu};
            if (masked) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    see[j] = visible<KIND>(a, s, token, anc, t0 + 32 * j, end);
                    if (missing) {
                        const int t = t0 + 32 * j + col;
                        const int page = t < end ? table[t >> a.page_shift] : -1;
                        see[j] &= uint32_t(__ballot(page >= 0 && page < a.cache.n_pages));
                    }
                }
            }
            if (!masked || __ballot((see[0] | see[1]) != 0)) {
                f32x16 x[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[j][i] = 0.0f;
#pragma unroll
                    for (int n = 0; n < D / 16; ++n)
                        x[j] = mfma32(load_frag(lds.k[buf] + k_piece<D>(32 * j + col, 2 * n + half)), q[n], x[j]);
                }
                // register i of a lane: key 8 (i / 4) + 4 half + i % 4
                float top = -inf;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (masked) {
                        const uint32_t bits = see[j] >> (4 * half);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (!(bits >> (8 * (i >> 2) + (i & 3)) & 1)) x[j][i] = -inf;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) top = fmaxf(top, x[j][i]);
                }
                // a scale of zero makes every visible score zero
                top = fmaxf(top, __shfl_xor(top, 32));
                top = top == -inf ? top : top * scale;
                if (__ballot(top > m + 8.0f)) {
                    const float m_new = fmaxf(m, top), keep = exp2_fast(m - finite_max(m_new));
                    m = m_new;
                    l *= keep;
#pragma unroll
                    for (int n = 0; n < D / 32; ++n) o[n] *= keep;
                }
                const float base = finite_max(m);
                bf16x8 p[4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float y = exp2_fast(fmaf(x[j][i], scale, -base));
                        if (masked && x[j][i] == -inf) y = 0.0f;
                        l += y;
                        p[2 * j + (i >> 3)][i & 7] = static_cast<__bf16>(y);
                    }
                // k-slots 8 half .. 8 half + 7 of product s: keys 16 s + 4 half + {0 .. 3} and 8 more
                const int vr = 4 * half + ((lane & 15) >> 2), vp0 = 2 * (lane >> 4 & 1) + ((lane & 3) >> 1);
                auto v_frag = [&](int n, int k) {
                    const int r = 16 * k + vr, piece = 4 * n + vp0;
                    const char* at0 = reinterpret_cast<const char*>(lds.v[buf] + v_piece<D>(r, piece)) + 8 * (lane & 1);
                    const char* at1 = reinterpret_cast<const char*>(lds.v[buf] + v_piece<D>(r + 8, piece)) + 8 * (lane & 1);
                    const uint2 u = read_tr16(at0), w = read_tr16(at1);
                    return make_uint4(u.x, u.y, w.x, w.y);
                };
                if (!(masked && odd)) {
#pragma unroll
                    for (int n = 0; n < D / 32; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[n] = mfma32(__builtin_bit_cast(bf16x8, v_frag(n, k)), p[k], o[n]);
                } else {
                    bf16x8 one[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int r = 8 * (k & 1) + i;  // register of x[k >> 1]
                            one[k][i] = static_cast<__bf16>(
                                (see[k >> 1] >> (4 * half) >> (8 * (r >> 2) + (r & 3)) & 1) ? 1.0f : 0.0f);
                        }
#pragma unroll
                    for (int n = 0; n < D / 32; ++n) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint4 u = v_frag(n, k);
                            o[n] = mfma32(__builtin_bit_cast(bf16x8, make_uint4(finite_of(u.x), finite_of(u.y), finite_of(u.z),
                                                                                finite_of(u.w))),
                                          p[k], o[n]);
                        }
                        for (int kind = 0; kind < 3; ++kind) {
                            f32x16 count;
#pragma unroll
                            for (int i = 0; i < 16; ++i) count[i] = 0.0f;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint4 u = v_frag(n, k);
                                count = mfma32(__builtin_bit_cast(bf16x8, make_uint4(marks_of(u.x, kind), marks_of(u.y, kind),
                                                                                     marks_of(u.z, kind), marks_of(u.w, kind))),
                                               one[k], count);
                            }
                            const float what = kind == 0 ? __builtin_nanf("") : kind == 1 ? inf : -inf;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (count[i] > 0.0f) o[n][i] += what;
                        }
                    }
                }
            }
            if (more) {
                const bool check = is_masked(t0 + kKeys);
                odd = st.store(lds.k[buf ^ 1], lds.v[buf ^ 1], tid, check);
                if (check)
                    odd = __syncthreads_or(odd);
                else
                    __syncthreads();
            }
        }

        l += __shfl_xor(l, 32);
        if (wave * 32 + col < rows) {
            if (chunks > 1) {
                float* part = part_out(a, it.part + it.chunk, h, kTileRows, D);
                const int r = wave * 32 + col;
#pragma unroll
                for (int n = 0; n < D / 32; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<f32x4*>(part + r * D + 32 * n + 8 * i + 4 * half) =
                            f32x4{o[n][4 * i], o[n][4 * i + 1], o[n][4 * i + 2], o[n][4 * i + 3]};
                if (half == 0) {
                    part[kTileRows * D + r] = m;
                    part[kTileRows * (D + 1) + r] = l;
                }
            } else {
#pragma unroll
                for (int n = 0; n < D / 32; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        attn_store<D>(a, s.row0 + token, h, head, 32 * n + 8 * i + 4 * half,
                                      f32x4{o[n][4 * i], o[n][4 * i + 1], o[n][4 * i + 2], o[n][4 * i + 3]}, l);
            }
        }
        if constexpr (KIND != kAttnPrefill) return;  // the grid has a workgroup for every item
        __syncthreads();
    }
}

template <AttnKind KIND, int D, bool F8>
hipError_t launch_one(const AttnArgs& a, const dim3& grid, hipStream_t stream) {
    const auto kernel = tiles_kernel<KIND, D, F8>;
    constexpr int bytes = sizeof(TileLds<D>);
    if (bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    kernel<<<grid, kThreads, bytes, stream>>>(a);
    return hipGetLastError();
}

template <AttnKind KIND>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
    const int64_t rows = int64_t(a.d.T) * a.group;  // of a tree, or of all prompts
    const int64_t tiles = KIND == kAttnVerify ? a.d.B * ((rows + kTileRows - 1) / kTileRows) : rows / kTileRows + a.d.B;
    const int64_t chunks = ((int64_t(a.d.max_pages) << a.page_shift) + a.min_chunk - 1) / a.min_chunk;
    const dim3 grid = grid_of(std::min(tiles + a.spread, tiles * std::max<int64_t>(chunks, 1)) * a.cache.H_kv);
    const bool f8 = a.cache.dtype == GDN_E4M3;
    switch (a.cache.d) {
        case 64: return f8 ? launch_one<KIND, 64, true>(a, grid, stream) : launch_one<KIND, 64, false>(a, grid, stream);
        case 128: return f8 ? launch_one<KIND, 128, true>(a, grid, stream) : launch_one<KIND, 128, false>(a, grid, stream);
        default: return f8 ? launch_one<KIND, 256, true>(a, grid, stream) : launch_one<KIND, 256, false>(a, grid, stream);
    }
}

}  // namespace

hipError_t launch_attn_tiles(const AttnArgs& a, hipStream_t stream) {
    return a.kind == kAttnVerify ? launch<kAttnVerify>(a, stream) : launch<kAttnPrefill>(a, stream);
}

}  // namespace gdn
