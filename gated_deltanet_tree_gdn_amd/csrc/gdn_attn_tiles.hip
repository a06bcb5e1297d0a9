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

// The 16-byte pieces of a row in LDS are permuted by these.  K is read 16 rows
// of one piece at a time, V transposed, 4 rows of four adjacent pieces at a
// time; both spread over all banks.
template <int D>
__device__ __forceinline__ constexpr int k_xor(int r) {
    return D >= 128 ? r & 15 : r >> 1 & 7;
}
template <int D>
__device__ __forceinline__ constexpr int v_xor(int r) {
    return D >= 128 ? 4 * (r & 3) : 4 * (r >> 1 & 1);
}

// x, but what is computed from it is computed where it stands: the compiler
// would otherwise form it before a loop and keep it in registers throughout.
__device__ __forceinline__ int fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// x = x f + g for accumulators that fill half of a wavefront's 512 registers, in
// place: the other half is what vector instructions can use, and without this
// the compiler moves all of them there and back around every use.
__device__ __forceinline__ void update_acc(f32x16& x, float f, const float (&g)[16]) {
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");  // matrix products may still write x
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float t, y = x[i];
        asm volatile(
            "v_accvgpr_read_b32 %1, %0\n\t"
            "s_nop 1\n\t"
            "v_fma_f32 %1, %1, %2, %3\n\t"
            "s_nop 1\n\t"
            "v_accvgpr_write_b32 %0, %1"
            : "+a"(y), "=&v"(t)
            : "v"(f), "v"(g[i]));
        x[i] = y;
    }
    asm volatile("s_nop 7" ::: "memory");
}

template <int D>
struct TileLds {
    uint4 k[2][kKeys * D / 8], v[2][kKeys * D / 8];
};

// 16 bytes per lane from memory to the 1 KB of LDS at `lds`.  The compiler's own
// forms of these make it wait for all of them before any read of LDS; here what
// has to have arrived is what loads_barrier() waits for.  Nothing else in these
// kernels uses m0.
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void load_to_lds(const i32x4& rsrc, int off, int more, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(off), "s"(rsrc), "s"(more),
                 "s"(lds)
                 : "memory");
}
__device__ __forceinline__ void load_to_lds(const char* at, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(at), "s"(lds) : "memory");
}

// Numbers of the pages from `first` on, one per lane, read from the table 64 at a time.
struct PageWindow {
    int first, ids, last;  // last: the last page that is read at all
    __device__ __forceinline__ void open(int end, int shift) {
        first = 0x7fffffff;
        last = (end - 1) >> shift;
    }
    __device__ __forceinline__ void cover(const int32_t* table, int from, int to, int lane) {
        if (from < first || to >= first + 64) {
            first = from;
            ids = table[min(first + lane, last)];
        }
    }
};

// Rows of K or V on their way from memory to LDS.  Wavefront w brings rows
// 16 w .. 16 w + 15 of a tile.  Rows behind the last token hold what lies there
// in the last page, rows of pages outside the pool what the first page holds;
// both are masked.  bf16 goes straight to LDS (a load fills 64 pieces in the
// order of the lanes, so the permutation of a row's pieces is made in the
// address), e4m3 through registers, where it becomes bf16.
template <int D, bool F8, bool IS_V>
struct Stage {
    static constexpr int P = D / (F8 ? 16 : 8);  // 16-byte pieces of a row
    static constexpr int L = 16 * P / 64;        // loads of a wavefront
    static constexpr int R = 64 / P;             // rows of a load
    static constexpr int size = F8 ? 1 : 2;
    const char* pool;  // of the key head
    int64_t page_stride;
    int row_stride;  // bytes
    PageWindow window;
    int piece, row;  // bytes: the lane's piece of a load's first rows as permuted, and its row
    uint4 x[F8 ? L : 1];

    __device__ __forceinline__ void init(const AttnArgs& a, int h, int end, int lane) {
        const gdn_kv_cache& c = a.cache;
        pool = static_cast<const char*>(IS_V ? c.v : c.k) + h * (IS_V ? c.v_head_stride : c.k_head_stride) * size;
        page_stride = (IS_V ? c.v_page_stride : c.k_page_stride) * size;
        row_stride = int(IS_V ? c.v_row_stride : c.k_row_stride) * size;
        window.open(end, a.page_shift);
        piece = (lane % P ^ perm(lane / P)) << 4;
        row = lane / P * row_stride;
    }
    // of row R j + l that is perm(R j) ^ perm(l)
    __device__ __forceinline__ static constexpr int perm(int r) { return F8 ? 0 : IS_V ? v_xor<D>(r) : k_xor<D>(r); }

    // The loads of a tile: begin(), and then part(0) .. part(L - 1) where a page has 16 rows or more.
    const char* base;
    uint32_t to_lds;
    __device__ __forceinline__ void begin(const AttnArgs& a, const int32_t* table, uint4* lds, int t0, int end, int wave,
                                          int lane) {
        t0 += 16 * wave;
        const int from = min(t0, end - 1) >> a.page_shift, to = min(t0 + 15, end - 1) >> a.page_shift;
        window.cover(table, from, to, lane);
        to_lds = __builtin_amdgcn_readfirstlane(lds_address(lds + 16 * wave * (D / 8)));
        if (a.page_shift >= 4) {  // the 16 rows lie in one page
            piece = fresh(piece);
            int page = __builtin_amdgcn_readlane(window.ids, from - window.first);
            if (page < 0 || page >= a.cache.n_pages) page = 0;
            base = pool + page * page_stride + int64_t(t0 & (a.cache.page_size - 1)) * row_stride;
        } else {
            lane = fresh(lane);
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const int r = (64 * j + lane) / P, t = t0 + r;
                int page = __shfl(window.ids, (min(t, end - 1) >> a.page_shift) - window.first);
                if (page < 0 || page >= a.cache.n_pages) page = 0;
                const char* at = pool + page * page_stride + int64_t(t & (a.cache.page_size - 1)) * row_stride +
                                 ((lane % P ^ perm(r)) << 4);
                if constexpr (F8)
                    x[j] = *reinterpret_cast<const uint4*>(at);
                else
                    load_to_lds(at, to_lds + 1024 * j);
            }
        }
    }
    __device__ __forceinline__ void part(int j) {
        const int off = (piece ^ perm(R * j) << 4) + row, more = R * j * row_stride;
        if constexpr (F8) {
            x[j] = *reinterpret_cast<const uint4*>(base + more + off);
        } else {
            const uint64_t bits = reinterpret_cast<uint64_t>(base);
            load_to_lds(i32x4{int32_t(bits), int32_t(bits >> 32 & 0xffff), 0x7fffffff, 0x00027000}, off, more,
                        to_lds + 1024 * j);
        }
    }
    __device__ __forceinline__ void load(const AttnArgs& a, const int32_t* table, uint4* lds, int t0, int end, int wave,
                                         int lane) {
        begin(a, table, lds, t0, end, wave, lane);
        if (a.page_shift >= 4)
#pragma unroll
            for (int j = 0; j < L; ++j) part(j);
    }
    // e4m3: what load() brought, into LDS as bf16.
    __device__ __forceinline__ void store(uint4* lds, int wave, int lane) const {
        if constexpr (F8) {
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const int r = 16 * wave + (64 * j + lane) / P, p = 2 * (lane % P);
                const int perm_r = IS_V ? v_xor<D>(r) : k_xor<D>(r);
                uint4 lo, hi;
                e4m3_to_bf16(x[j], lo, hi);
                lds[r * (D / 8) + (p ^ perm_r)] = lo;
                lds[r * (D / 8) + (p + 1 ^ perm_r)] = hi;
            }
        }
    }
};

// Whether any of the thread's share of a tile of V is not finite.
template <int D>
__device__ __forceinline__ bool any_odd(const uint4* v, int tid) {
    bool odd = false;
#pragma unroll
    for (int i = 0; i < kKeys * D / 8 / kThreads; ++i) {
        const uint4 x = v[i * kThreads + tid];
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) odd |= (u[w] & 0x7f80u) == 0x7f80u || (u[w] & 0x7f800000u) == 0x7f800000u;
    }
    return odd;
}

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

// A tile of V in LDS, rewritten by the workgroup: kind 0 with zeros for what is
// not finite, else ones where it is NaN (1), +inf (2), -inf (3) and zeros elsewhere.
template <int D>
__device__ __forceinline__ void rewrite(uint4* v, int kind, int tid) {
#pragma unroll 1
    for (int i = tid; i < kKeys * D / 8; i += kThreads) {
        uint4 x = v[i];
        uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t r = 0;
#pragma unroll
            for (int at = 0; at < 32; at += 16) {
                const uint32_t e = u[w] >> at & 0xffff;
                const int is = (e & 0x7f80) != 0x7f80 ? 0 : (e & 0x7f) ? 1 : e == 0x7f80 ? 2 : 3;
                r |= (kind == 0 ? (is ? 0 : e) : is == kind ? 0x3f80u : 0) << at;
            }
            u[w] = r;
        }
        v[i] = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// ---------------------------------------------------------------------------
// A piece of a workgroup's range: some keys of one key head for 128 rows (token,
// query head of the group) of a sequence; a wavefront has 32 of the rows.  64
// keys at a time lie in LDS, the next 64 on their way there.
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
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const AttnPlan plan = attn_plan<KIND>(a, threadIdx.x & 63);
    const int w = attn_range(plan, blockIdx.x);
    const int64_t u0 = w * plan.per, u_end = min(u0 + plan.per, plan.units * a.cache.H_kv);
    const float inf = __builtin_inff();

    AttnPlace at;
    for (int64_t u = u0; u < u_end;) {
        const int tid = fresh(threadIdx.x), lane = tid & 63, col = lane & 31, half = lane >> 5;
        const int h = int(quotient(u, plan.units));
        const int64_t uh = u - h * plan.units;
        if (at.b < 0 || uh < at.first || uh >= at.first + at.count) attn_find<KIND, false>(a, uh, lane, at);
        const AttnSeq s = attn_seq_uniform<KIND>(a, at.b);
        const AttnPiece it = attn_piece<KIND>(a, s, attn_tiles<KIND>(a, s), uh - at.first, u_end - u);
        const bool first = u == u0;
        u += it.units;
        if (it.all == 0) continue;
        const float scale = a.d.scale * kLog2e * (a.cache.k_scale ? a.cache.k_scale[h] : 1.0f);
        const int all_rows = s.n * a.group;
        const int row0 = it.tile * kTileRows, rows = min(kTileRows, all_rows - row0);
        const int begin = it.unit * kKeys;
        const int end = min(begin + it.units * kKeys, attn_seen<KIND>(a, s, it.tile));

        const int my_row = min(row0 + wave * 32 + col, all_rows - 1);
        const int token = my_row / a.group, head = h * a.group + my_row - token * a.group;
        const uint32_t* anc =
            KIND == kAttnVerify ? a.anc + (int64_t(at.b) * s.n + token) * ((a.d.T + 31) >> 5) : nullptr;
        const int32_t* table = a.table + at.b * a.d.table_stride;
        // tokens from here on are masked for some of the tile's rows
        const int open_end = KIND == kAttnPrefill ? s.prefix + row0 / a.group + 1 : s.prefix;

        bool missing = false;  // pages outside the pool
        for (int p = (begin >> a.page_shift) + tid; begin < end && p <= (end - 1) >> a.page_shift; p += kThreads) {
            const int page = table[p];
            missing |= page < 0 || page >= a.cache.n_pages;
        }
        missing = __builtin_amdgcn_readfirstlane(__syncthreads_or(missing));

        bf16x8 q[D / 16];
        const uint16_t* qp = a.q + (s.row0 + token) * a.d.q_stride + int64_t(head) * D + 8 * half;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
            q[n] = load_frag(qp + 16 * n);
            if constexpr (D == 256) asm volatile("" : "+a"(q[n]));  // beside the accumulators
        }

        f32x16 o[D / 32];
#pragma unroll
        for (int n = 0; n < D / 32; ++n)
#pragma unroll
            for (int j = 0; j < 16; ++j) o[n][j] = 0.0f;
        float m = -inf, l = 0.0f;  // m: what the powers are taken against

        // register i of x[j]: key 32 j + 8 (i / 4) + 4 half + i % 4 of the tile, row `col`
        const uint32_t k_row = lds_address(lds.k) + col * (D * 2);
        int k_col = (half ^ k_xor<D>(col)) << 4;
        auto k_frag = [&](int j, int n, int buf) {
            return *reinterpret_cast<const __attribute__((address_space(3))) bf16x8*>(
                k_row + buf * (kKeys * D * 2) + (k_col ^ n << 5) + j * (32 * D * 2));
        };
        // k-slots 8 half .. 8 half + 7 of product k: keys 16 k + 4 half + {0 .. 3} and 8 more, whose rows have the same permutation
        const int vr = 4 * half + ((lane & 15) >> 2);
        const uint32_t v_row = lds_address(lds.v) + vr * (D * 2) + 8 * (lane & 1);
        const int v_col = (2 * (lane >> 4 & 1) + ((lane & 3) >> 1) ^ v_xor<D>(vr)) << 4;
        auto v_frag = [&](int n, int k, int buf) {
            const uint32_t at = v_row + buf * (kKeys * D * 2) + (v_col ^ n << 6) + k * (16 * D * 2);
            const uint2 u = read_tr16(at), w = read_tr16(at + 8 * D * 2);
            return __builtin_bit_cast(bf16x8, make_uint4(u.x, u.y, w.x, w.y));
        };
        const f32x16 zero{};
        // The largest of what x adds to a row, in powers of two.
        auto largest = [&](float top) {
            const auto both = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, top),
                                                               __builtin_bit_cast(uint32_t, top), false, false);
            const uint32_t lo = both[0], hi = both[1];
            top = fmaxf(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
            return top == -inf ? top : top * scale;
        };
        auto raise = [&](float top) {
            if (__ballot(top > m + 8.0f)) {
                const float m_new = fmaxf(m, top), keep = exp2_fast(m - finite_max(m_new));
                m = m_new;
                l *= keep;
#pragma unroll
                for (int n = 0; n < D / 32; ++n) {
                    if constexpr (D == 256)
                        update_acc(o[n], keep, {});
                    else
                        o[n] *= keep;
                }
            }
        };

        if (begin < end) {
            Stage<D, F8, false> sk;
            Stage<D, F8, true> sv;
            sk.init(a, h, end, lane);
            sv.init(a, h, end, lane);
            // V of the tile at t0 and K of the next one are in LDS; those after
            // them may come (K behind the last tile is not used).
            auto arrive = [&](int t0, int buf) {
                if (t0 + kKeys < end) sk.store(lds.k[buf ^ 1], wave, lane);
                sv.store(lds.v[buf], wave, lane);
                loads_barrier<0>();
                if (t0 + kKeys < end) {
                    sk.begin(a, table, lds.k[buf], t0 + 2 * kKeys, end, wave, lane);
                    sv.begin(a, table, lds.v[buf ^ 1], t0 + kKeys, end, wave, lane);
                }
            };
            constexpr int L = Stage<D, F8, true>::L;
            auto part = [&](int i) {
                if (i < L)
                    sk.part(i);
                else
                    sv.part(i - L);
            };
            sk.load(a, table, lds.k[0], begin, end, wave, lane);
            sk.store(lds.k[0], wave, lane);
            loads_barrier<0>();
            if (begin + kKeys < end) sk.load(a, table, lds.k[1], begin + kKeys, end, wave, lane);
            sv.load(a, table, lds.v[0], begin, end, wave, lane);
            constexpr int NQ = D / 8, AHEAD = D == 128 ? 4 : 8;  // products of a tile with K (and with V), operands read ahead
            f32x16 x[2];                          // scores of the tile at t0
#pragma unroll
            for (int i = 0; i < NQ; ++i) x[i & 1] = mfma32(k_frag(i & 1, i >> 1, 0), q[i >> 1], i < 2 ? zero : x[i & 1]);
            int t0 = begin, buf = 0;

            // Tiles that every row sees all of, but the last (pages of fewer than 16
            // rows take the plain loop below for all): the scores of the
            // next tile are formed beside the powers of this one and its maxima
            // beside the products with V, step by step as they stand here.
            const int open = missing || a.page_shift < 4 ? begin : min(max(open_end, begin), end - 1);
            float top = -inf;
#pragma unroll
            for (int i = 0; i < 32; ++i) top = fmaxf(top, x[i >> 4][i & 15]);
            top = largest(top);
            for (; t0 + kKeys <= open; t0 += kKeys, buf ^= 1) {
                arrive(t0, buf);
                k_col = fresh(k_col);
                raise(top);
                const float base = finite_max(m);
                f32x16 y[2];
                bf16x8 f[AHEAD], p[4];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) f[i] = k_frag(i & 1, i >> 1, buf ^ 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    y[i & 1] = mfma32(f[i % AHEAD], q[i >> 1], i < 2 ? zero : y[i & 1]);
                    const int r = i + AHEAD;
                    f[i % AHEAD] = r < NQ ? k_frag(r & 1, r >> 1, buf ^ 1) : v_frag((r - NQ) % (D / 32), (r - NQ) / (D / 32), buf);
                    if (i % (NQ / (2 * L)) == 0) part(i / (NQ / (2 * L)));
#pragma unroll
                    for (int e = i * 32 / NQ; e < (i + 1) * 32 / NQ; ++e) {
                        x[e >> 4][e & 15] = exp2_fast(fmaf(x[e >> 4][e & 15], scale, -base));
                        p[e >> 3][e & 7] = static_cast<__bf16>(x[e >> 4][e & 15]);
                        if (D < 256) l += x[e >> 4][e & 15];
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                top = -inf;
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    o[i % (D / 32)] = mfma32(f[i % AHEAD], p[i / (D / 32)], o[i % (D / 32)]);
                    const int r = i + AHEAD;
                    if (r < NQ) f[i % AHEAD] = v_frag(r % (D / 32), r / (D / 32), buf);
                    if (D == 256) l += x[i >> 4 & 1][i & 15];  // elsewhere x has no registers by now
                    if (i >= NQ / 2) {
#pragma unroll
                        for (int e = (i - NQ / 2) * 64 / NQ; e < (i - NQ / 2 + 1) * 64 / NQ; ++e)
                            top = fmaxf(top, y[e >> 4][e & 15]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                top = largest(top);
                x[0] = y[0];
                x[1] = y[1];
            }
            for (; t0 < end; t0 += kKeys, buf ^= 1) {
                arrive(t0, buf);
                if (t0 + kKeys < end && a.page_shift >= 4)
#pragma unroll
                    for (int i = 0; i < 2 * L; ++i) part(i);
                uint32_t see[2] = {0xffffffffu, 0xffffffffu};
                bool odd = false;
                if (missing || t0 + kKeys > min(open_end, end)) {
                    odd = __builtin_amdgcn_readfirstlane(__syncthreads_or(any_odd<D>(lds.v[buf], tid)));
                    if (odd) {
                        rewrite<D>(lds.v[buf], 0, tid);
                        __syncthreads();
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t bits = visible<KIND>(a, s, token, anc, t0 + 32 * j, end);
                        if (missing) {
                            const int t = t0 + 32 * j + col;
                            const int page = t < end ? table[t >> a.page_shift] : -1;
                            bits &= uint32_t(__ballot(page >= 0 && page < a.cache.n_pages));
                        }
                        see[j] = bits >> (4 * half);
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (!(see[j] >> (8 * (i >> 2) + (i & 3)) & 1)) x[j][i] = -inf;
                top = -inf;
#pragma unroll
                for (int i = 0; i < 32; ++i) top = fmaxf(top, x[i >> 4][i & 15]);
                raise(largest(top));
                const float base = finite_max(m);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    bf16x8 p;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = 8 * (k & 1) + i;
                        float e = exp2_fast(fmaf(x[k >> 1][r], scale, -base));
                        // a scale of zero turns -inf into NaN
                        if (!(see[k >> 1] >> (8 * (r >> 2) + (r & 3)) & 1)) e = 0.0f;
                        l += e;
                        p[i] = static_cast<__bf16>(e);
                    }
#pragma unroll
                    for (int n = 0; n < D / 32; ++n) o[n] = mfma32(v_frag(n, k, buf), p, o[n]);
                }
                if (t0 + kKeys < end) {
#pragma unroll
                    for (int i = 0; i < NQ; ++i)
                        x[i & 1] = mfma32(k_frag(i & 1, i >> 1, buf ^ 1), q[i >> 1], i < 2 ? zero : x[i & 1]);
                }
                if (!odd) continue;
#pragma unroll 1
                for (int kind = 1; kind <= 3; ++kind) {
                    const float what = kind == 1 ? __builtin_nanf("") : kind == 2 ? inf : -inf;
                    __syncthreads();
                    Stage<D, F8, true> again = sv;
                    again.load(a, table, lds.v[buf], t0, end, wave, lane);
                    again.store(lds.v[buf], wave, lane);
                    loads_barrier<0>();
                    rewrite<D>(lds.v[buf], kind, tid);
                    __syncthreads();
#pragma unroll
                    for (int n = 0; n < D / 32; ++n) {
                        f32x16 count;
#pragma unroll
                        for (int i = 0; i < 16; ++i) count[i] = 0.0f;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t bits = see[k >> 1];
                            asm volatile("" : "+v"(bits));  // formed anew each time, to hold no registers for it
                            bf16x8 one;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int r = 8 * (k & 1) + i;
                                one[i] = static_cast<__bf16>((bits >> (8 * (r >> 2) + (r & 3)) & 1) ? 1.0f : 0.0f);
                            }
                            count = mfma32(v_frag(n, k, buf), one, count);
                        }
                        float g[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) g[i] = count[i] > 0.0f ? what : 0.0f;
                        if constexpr (D == 256) {
                            update_acc(o[n], 1.0f, g);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[n][i] += g[i];
                        }
                    }
                }
            }
        }

        l += __shfl_xor(l, 32);
        if (wave * 32 + col < rows) {
            if (it.units < it.all) {
                float* part = part_out(a, 2 * int64_t(w) + (first ? 0 : 1), kTileRows, D);
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
        if (u < u_end) __syncthreads();  // the next piece overwrites LDS
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
    const dim3 grid(a.slots);
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
