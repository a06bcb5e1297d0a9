// gdn_attn_tiles.hip -- softmax attention of many queries per sequence over a
// paged cache: packed prompts and proposal trees.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "gdn_attn_internal.h"
#include "gdn_attn_plan.h"

namespace gdn {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kKeys = kTilesUnit;  // keys of a tile in LDS

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x16 mfma32(const bf16x8& a, const bf16x8& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Rows of K and V in LDS.  A load fills 1 KB in the order of the lanes, a block
// of 512 / D rows; a few bytes after a block, and a permutation of the pieces of
// a row by its place in the block (made in the address that a lane loads from),
// spread over all banks what is read at a time: of K one piece of 16 rows, of V
// four adjacent pieces of 4 rows (transposed).  Both leave constant offsets
// between most reads of a lane.
template <int D, bool IS_V>
struct Layout {
    static constexpr int kRows = 512 / D;                                  // of a block
    static constexpr int kBlock = 1024 + (IS_V ? (D == 256 ? 128 : 0) : (D == 256 ? 32 : 64));
    static constexpr int kTile = kKeys / kRows * kBlock;                   // bytes
    // what the number of a row's piece is xored with: bits 0 and 1 (K), 2 and 3 (V)
    __device__ __forceinline__ static constexpr int perm(int r) {
        return IS_V ? 4 * (D == 256 ? r & 1 : D == 128 ? r & 3 : r >> 1 & 1) : D == 256 ? r & 1 : D == 128 ? r & 3 : r >> 1 & 3;
    }
    __device__ __forceinline__ static constexpr int row(int r) { return r / kRows * kBlock + r % kRows * (D * 2); }
};
template <int D>
struct TileLds {
    static constexpr int kV = 2 * Layout<D, false>::kTile, kBytes = kV + 2 * Layout<D, true>::kTile;
};

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
            "v_fma_f32 %1, %1, %2, %3\n\t"
            "v_accvgpr_write_b32 %0, %1"
            : "+a"(y), "=&v"(t)
            : "v"(f), "v"(g[i]));
        x[i] = y;
    }
    asm volatile("s_nop 7" ::: "memory");
}

// 16 bytes per lane from memory to the 1 KB of LDS at `lds`.  The compiler's own
// forms of these make it wait for all of them before any read of LDS; here what
// has to have arrived is what loads_barrier() waits for.  Nothing else in these
// kernels uses m0.
// A vector memory instruction may read a scalar register no sooner than five wait
// states after a vector instruction wrote it, as one does that brings back a
// spilled register (v_readlane).  The compiler does not look into a statement, so
// the statement itself has them: the move and s_nop 3, of which the load's use of
// m0 needs one.  Two and four loads to a statement, which then share them, are no
// faster (a prompt of 16384, 16 and 2 heads of 256: 2135 us, 2137 and 2155).
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void load_to_lds(const i32x4& rsrc, int off, int more, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(off), "s"(rsrc), "s"(more),
                 "s"(lds)
                 : "memory");
}
__device__ __forceinline__ void load_to_lds(const char* at, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(at), "s"(lds) : "memory");
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ __attribute__((address_space(3))) u32x4* lds_piece(uint32_t at) {
    return reinterpret_cast<__attribute__((address_space(3))) u32x4*>(at);
}

// Rows of K or V on their way from memory to LDS.  Wavefront w brings rows
// 16 w .. 16 w + 15 of a tile.  Rows behind the last token hold what lies there
// in the last page, rows of pages outside the pool what the first page holds;
// both are masked.  bf16 goes straight to LDS, e4m3 through registers, where it
// becomes bf16.
template <int D, bool F8, bool IS_V>
struct Stage {
    using To = Layout<D, IS_V>;
    static constexpr int P = D / (F8 ? 16 : 8);  // 16-byte pieces of a row
    static constexpr int L = 16 * P / 64;        // loads of a wavefront
    static constexpr int R = 64 / P;             // rows of a load
    static constexpr int size = F8 ? 1 : 2;
    const char* pool;  // of the key head
    int64_t page_stride;
    int row_stride;  // bytes
    int off;         // bytes: the lane's piece and row of a load
    const char* base;
    uint32_t to_lds;
    uint4 x[F8 ? L : 1];

    __device__ __forceinline__ void init(const AttnArgs& a, int h, int lane) {
        const gdn_kv_cache& c = a.cache;
        pool = static_cast<const char*>(IS_V ? c.v : c.k) + h * (IS_V ? c.v_head_stride : c.k_head_stride) * size;
        page_stride = (IS_V ? c.v_page_stride : c.k_page_stride) * size;
        row_stride = int(IS_V ? c.v_row_stride : c.k_row_stride) * size;
        off = lane / P * row_stride + ((lane % P ^ (F8 ? 0 : To::perm(lane / P))) << 4);
    }
    // The loads of a tile where a page has 16 rows or more, which so lie in page
    // `page` from row `row` on: at(), and then part(0) .. part(L - 1).
    __device__ __forceinline__ void at(uint32_t lds, int page, int row, int wave) {
        to_lds = lds + 16 / To::kRows * To::kBlock * wave;
        base = pool + page * page_stride + int64_t(row) * row_stride;
    }
    __device__ __forceinline__ void part(int j) {
        const int more = R * j * row_stride;
        if constexpr (F8) {
            x[j] = *reinterpret_cast<const uint4*>(base + more + off);
        } else {
            const uint64_t bits = reinterpret_cast<uint64_t>(base);
            const int lo = __builtin_amdgcn_readfirstlane(int(bits)), hi = __builtin_amdgcn_readfirstlane(int(bits >> 32 & 0xffff));
            load_to_lds(i32x4{lo, hi, 0x7fffffff, 0x00027000}, off, __builtin_amdgcn_readfirstlane(more),
                        __builtin_amdgcn_readfirstlane(to_lds) + To::kBlock * j);
        }
    }
    // The same for smaller pages.
    __device__ __forceinline__ void scattered(const AttnArgs& a, const PageWindow& window, uint32_t lds, int t0, int end,
                                              int wave, int lane) {
        lane = fresh(lane);
        to_lds = lds + 16 / To::kRows * To::kBlock * wave;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int r = R * j + lane / P, t = t0 + 16 * wave + r;
            int page = __shfl(window.ids, (min(t, end - 1) >> a.page_shift) - window.first);
            if (page < 0 || page >= a.cache.n_pages) page = 0;
            const char* from = pool + page * page_stride + int64_t(t & (a.cache.page_size - 1)) * row_stride +
                               ((lane % P ^ (F8 ? 0 : To::perm(r))) << 4);
            if constexpr (F8)
                x[j] = *reinterpret_cast<const uint4*>(from);
            else
                load_to_lds(from, to_lds + To::kBlock * j);
        }
    }
    // e4m3: what the loads brought, into LDS as bf16.
    __device__ __forceinline__ void store(uint32_t lds, int wave, int lane) const {
        if constexpr (F8) {
            lane = fresh(lane);
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const int r = 16 * wave + R * j + lane / P, p = 2 * (lane % P);
                uint4 lo, hi;
                e4m3_to_bf16(x[j], lo, hi);
                *lds_piece(lds + To::row(r) + ((p ^ To::perm(r)) << 4)) = u32x4{lo.x, lo.y, lo.z, lo.w};
                *lds_piece(lds + To::row(r) + ((p + 1 ^ To::perm(r)) << 4)) = u32x4{hi.x, hi.y, hi.z, hi.w};
            }
        }
    }
};

// The two of them, in step: K runs a tile ahead of V, whose pages are then known.
template <int D, bool F8>
struct Loader {
    Stage<D, F8, false> k;
    Stage<D, F8, true> v;
    static constexpr int L = Stage<D, F8, false>::L;
    PageWindow window;  // of K's tiles
    int page, row;      // of K's last tile (pages of 16 rows or more)

    __device__ __forceinline__ void init(const AttnArgs& a, int h, int end, int lane) {
        k.init(a, h, lane);
        v.init(a, h, lane);
        window.open(end, a.page_shift);
    }
    template <bool LARGE = false>
    __device__ __forceinline__ void find(const AttnArgs& a, const int32_t* table, int t0, int end, int wave, int lane) {
        t0 += 16 * wave;
        const int from = min(t0, end - 1) >> a.page_shift, to = min(t0 + 15, end - 1) >> a.page_shift;
        window.cover(table, from, to, lane);
        if (LARGE || a.page_shift >= 4) {
            page = __builtin_amdgcn_readlane(window.ids, from - window.first);
            if (page < 0 || page >= a.cache.n_pages) page = 0;
            row = t0 & (a.cache.page_size - 1);
        }
    }
    // V's tile at t0 and K's at t0 + kKeys: all of it where pages are small,
    // otherwise (and only those with LARGE) the loads follow with k.part() and v.part().
    template <bool LARGE>
    __device__ __forceinline__ void begin(const AttnArgs& a, const int32_t* table, uint32_t k_lds, uint32_t v_lds, int t0,
                                          int end, int wave, int lane) {
        if (LARGE || a.page_shift >= 4) {
            v.at(v_lds, page, row, wave);
            find<LARGE>(a, table, t0 + kKeys, end, wave, lane);
            k.at(k_lds, page, row, wave);
        } else {
            find(a, table, t0, end, wave, lane);
            v.scattered(a, window, v_lds, t0, end, wave, lane);
            find(a, table, t0 + kKeys, end, wave, lane);
            k.scattered(a, window, k_lds, t0 + kKeys, end, wave, lane);
        }
    }
};

// Whether any of the thread's share of a tile of V is not finite.
template <int D>
__device__ __forceinline__ bool any_odd(uint32_t v, int tid) {
    bool odd = false;
#pragma unroll 2
    for (int i = tid; i < kKeys * D / 8; i += kThreads) {
        const u32x4 x = *lds_piece(v + (i >> 6) * Layout<D, true>::kBlock + (i & 63) * 16);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t u = x[w];
            odd |= (u & 0x7f80u) == 0x7f80u || (u & 0x7f800000u) == 0x7f800000u;
        }
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
__device__ __forceinline__ void rewrite(uint32_t v, int kind, int tid) {
#pragma unroll 1
    for (int i = tid; i < kKeys * D / 8; i += kThreads) {
        auto* at = lds_piece(v + (i >> 6) * Layout<D, true>::kBlock + (i & 63) * 16);
        u32x4 x = *at;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t r = 0;
#pragma unroll
            for (int shift = 0; shift < 32; shift += 16) {
                const uint32_t e = x[w] >> shift & 0xffff;
                const int is = (e & 0x7f80) != 0x7f80 ? 0 : (e & 0x7f) ? 1 : e == 0x7f80 ? 2 : 3;
                r |= (kind == 0 ? (is ? 0 : e) : is == kind ? 0x3f80u : 0) << shift;
            }
            x[w] = r;
        }
        *at = x;
    }
}

// ---------------------------------------------------------------------------
// A piece of a workgroup's range: some keys of one key head for a tile of rows
// (token, query head of the group) of a sequence, 32 of them a wavefront's.  64
// keys at a time lie in LDS, the next 64 on their way there.
//   S^T = K Q^T    keys x rows on MFMA, Q in registers for the whole piece
//   O^T += V^T P   V read transposed; the lanes hold P where the product wants it
// The running maximum is raised only where a row's scores pass it by more than
// 2^8: P then stays below 2^8, which costs no precision in floating point, and
// O is rarely rescaled (by rows: what a wavefront's other rows see has no part in
// a row's rounding).  P is rounded to bf16 for the product, at most 2^-8 of a
// weight, as much as the output's own rounding; the sum is that of the rounded
// weights.
// A masked key has P = 0, but 0 times an infinity or NaN of its value would not
// be 0: a tile with masked keys and such values is multiplied with zeros in
// their place, and the rows that do see them get them from products of marks.
// A SIMD has registers for one wavefront (d = 256) or two, and a wavefront issues
// in order, so the main loop stands in the order in which it is to run: beside
// every product what the vector unit can do meanwhile.
// Measured, causal prompts and trees of 64 nodes over 4096 tokens with 16 query
// and 2 key heads: 382 and 457 TFLOP/s (d = 64, bound by the powers: 32 x 64 of
// them per 16 matrix instructions), 626 and 702 (128), 833 and 881 (256); a
// prompt of 16384 with d = 256: 1.04 PFLOP/s, two thirds of what the largest
// library product reaches: the matrix units are busy 48 % of the time, a wavefront
// issues 51 % of its cycles, waits 29 % for barriers and operands and 20 % for its
// turn (16 trees of 128 nodes, heads of 128: 49, 42, 30 and 28 %).
// e4m3 is 0 to 17 % slower, pages of fewer than 16 tokens (whose rows are
// addressed one by one, and which take the plain loop) half as fast.
// ---------------------------------------------------------------------------
template <AttnKind KIND, int D, bool F8>
__global__ __launch_bounds__(kThreads, tiles_per_cu(D)) void tiles_kernel(AttnArgs a) {
    using KL = Layout<D, false>;
    using VL = Layout<D, true>;
    extern __shared__ uint4 lds_raw[];
    const uint32_t lds_k = __builtin_amdgcn_readfirstlane(lds_address(lds_raw)), lds_v = lds_k + TileLds<D>::kV;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const float inf = __builtin_inff();

    AttnRange range;
    AttnPlace at;
    if (!attn_begin<KIND>(a, blockIdx.x, threadIdx.x & 63, range, at)) return;
    for (int64_t u = range.u; u < range.end;) {
        const int tid = fresh(threadIdx.x), lane = tid & 63, col = lane & 31, half = lane >> 5;
        const int h = int(quotient(u, range.units));
        const int64_t uh = u - h * range.units;
        attn_next<KIND>(a, uh, lane, at);
        const AttnSeq s = at.s;
        const AttnPiece it = attn_piece<KIND>(a, s, attn_tiles<KIND>(a, s), uh - at.first, range.end - u);
        const bool first = u == range.u;
        u += it.units;
        if (it.all == 0) continue;
        const float scale = a.d.scale * kLog2e * (a.cache.k_scale ? a.cache.k_scale[h] : 1.0f);
        const int all_rows = s.n * a.group;
        const int row0 = (KIND == kAttnVerify ? range.mate : it.tile) * kTileRows, rows = min(kTileRows, all_rows - row0);
        const int begin = it.unit * kKeys;
        const int end = __builtin_amdgcn_readfirstlane(min(begin + it.units * kKeys, attn_seen<KIND>(a, s, it.tile)));
        const int32_t* table = a.table + at.b * a.d.table_stride;
        // tokens from here on are masked for some of the tile's rows
        const int open_end = KIND == kAttnPrefill ? __builtin_amdgcn_readfirstlane(s.prefix + row0 / a.group + 1) : s.prefix;

        const int row = min(row0 + wave * 32 + col, all_rows - 1), token = row / a.group;
        const int head = h * a.group + row - token * a.group;
        bf16x8 q[D / 16];
        f32x16 o[D / 32];
        float m = -inf, l = 0.0f;  // m: what the powers are taken against
        const uint16_t* qp = a.q + (s.row0 + token) * a.d.q_stride + int64_t(head) * D + 8 * half;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) q[n] = load_frag(qp + 16 * n);
#pragma unroll
        for (int n = 0; n < D / 32; ++n)
#pragma unroll
            for (int j = 0; j < 16; ++j) o[n][j] = 0.0f;

        // Register i of a score x[j]: key 32 j + 8 (i / 4) + 4 half + i % 4 of the tile, row `col` of the wavefront's.
        // K: piece 2 n + half of row 32 j + col; its permutation's higher bit swaps neighbouring n.
        const int k_swap = KL::perm(col) >> 1, k_piece = (half ^ (KL::perm(col) & 1)) << 4;
        const uint32_t k_even = lds_k + KL::row(col) + k_piece + 32 * k_swap, k_odd = k_even - 64 * k_swap;
        auto k_frag = [&](int j, int n, int buf) {
            return *reinterpret_cast<const __attribute__((address_space(3))) bf16x8*>(
                (n & 1 ? k_odd : k_even) + buf * KL::kTile + 32 / KL::kRows * KL::kBlock * j + 32 * n);
        };
        // V: k-slots 8 half .. 8 half + 7 of product k are keys 16 k + 4 half + {0 .. 3} and 8 more, whose rows have the
        // same permutation; it swaps the 64 bytes of product n with those of n ^ v_swap.
        const int vr = 4 * half + ((lane & 15) >> 2), v_swap = VL::perm(vr) >> 2;
        const uint32_t v_row = lds_v + VL::row(vr) + 32 * (lane >> 4 & 1) + 8 * (lane & 3);
        constexpr int VN = D == 128 ? 4 : 2;  // v_swap < VN
        uint32_t v_at[VN];
#pragma unroll
        for (int n = 0; n < VN; ++n) v_at[n] = v_row + 64 * (n ^ v_swap);
        auto v_frag = [&](int n, int k, int buf) {
            const uint32_t from = v_at[n % VN] + buf * VL::kTile + n / VN * VN * 64 + 16 / VL::kRows * VL::kBlock * k;
            const uint2 x = read_tr16(from), y = read_tr16(from + VL::row(8));
            return __builtin_bit_cast(bf16x8, make_uint4(x.x, x.y, y.x, y.y));
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
                const float m_new = top > m + 8.0f ? top : m, keep = exp2_fast(m - finite_max(m_new));
                const bool some = __ballot(m != -inf) != 0;  // that is not zero
                m = m_new;
                if (!some) return;
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
            Loader<D, F8> load;
            constexpr int L = load.L;
            auto rest = [&] {  // of the loads of one tile, at once
                if (a.page_shift < 4) return;
#pragma unroll
                for (int i = 0; i < L; ++i) load.k.part(i);
#pragma unroll
                for (int i = 0; i < L; ++i) load.v.part(i);
            };
            load.init(a, h, end, lane);
            load.find(a, table, begin, end, wave, lane);
            if (a.page_shift >= 4) {
                load.k.at(lds_k, load.page, load.row, wave);
#pragma unroll
                for (int i = 0; i < L; ++i) load.k.part(i);
            } else {
                load.k.scattered(a, load.window, lds_k, begin, end, wave, lane);
            }
            bool missing = false;  // pages outside the pool
            for (int p = (begin >> a.page_shift) + tid; p <= (end - 1) >> a.page_shift; p += kThreads) {
                const int page = table[p];
                missing |= page < 0 || page >= a.cache.n_pages;
            }
            if constexpr (D == 256) {
#pragma unroll
                for (int n = 0; n < D / 16; ++n) asm volatile("" : "+a"(q[n]));  // beside the accumulators
            }
            load.k.store(lds_k, wave, lane);
            wait_count<0>();
            missing = __builtin_amdgcn_readfirstlane(__syncthreads_or(missing));
            // K of the tile behind the last is not used: it repeats what there is
            load.template begin<false>(a, table, lds_k + KL::kTile, lds_v, begin, end, wave, lane);
            rest();
            // K of the tile after t0 and, but for the last PENDING loads, V of that
            // at t0 are in LDS; those after them may come.
            auto arrive = [&](int t0, int buf, auto pending, auto large) {
                load.k.store(lds_k + (buf ^ 1) * KL::kTile, wave, lane);
                load.v.store(lds_v + buf * VL::kTile, wave, lane);
                loads_barrier<pending>();
                if (t0 + kKeys < end)
                    load.template begin<large>(a, table, lds_k + buf * KL::kTile, lds_v + (buf ^ 1) * VL::kTile, t0 + kKeys, end, wave, lane);
            };
            // products of a tile with K, and with V; operands read ahead
            constexpr int NS = D / 8, AHEAD = D == 256 ? 8 : 4;
            f32x16 x[2];  // scores of the tile at t0
            float top = -inf;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const bf16x8 f = k_frag(i & 1, i >> 1, 0);
                x[i & 1] = mfma32(f, q[i >> 1], i < 2 ? zero : x[i & 1]);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) top = fmaxf(top, x[i >> 4][i & 15]);
            top = largest(top);

            // A tile that every row sees all of, and that is not the last: the
            // scores y of the next tile beside the powers of this one's x, and
            // its maxima beside the products with V.  Loads have a whole turn to
            // arrive: K's are issued beside the products with K and waited for
            // before those of the next turn, V's likewise (e4m3, which waits in
            // registers, has V's beside the products with V as well, where x no
            // longer needs them, and stores both at once).
            auto turn = [&](f32x16 (&x)[2], f32x16 (&y)[2], int t0, auto buf) {
                arrive(t0, buf, std::integral_constant<int, F8 ? 0 : L>(), std::true_type());
                bf16x8 f[AHEAD], p[4];
                raise(top);
                const float base = finite_max(m);
                top = -inf;
                // powers that are formed up to step i: 20 of 32 beside K, the others
                // beside the first half of V, in time for the product that wants them
                auto formed = [](int i) { return i <= NS ? i * 20 / NS : i >= NS + NS / 2 ? 32 : 20 + (i - NS) * 24 / NS; };
                auto powers = [&](int i) {
#pragma unroll
                    for (int e = formed(i); e < formed(i + 1); ++e) {
                        p[e >> 3][e & 7] = static_cast<__bf16>(exp2_fast(fmaf(x[e >> 4][e & 15], scale, -base)));
                        if (e & 1) {
                            const bf16x2 two{p[e >> 3][(e & 7) - 1], p[e >> 3][e & 7]}, one{1.0f, 1.0f};
                            l = __builtin_amdgcn_fdot2_f32_bf16(two, one, l, false);
                        }
                    }
                };
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) f[i] = k_frag(i & 1, i >> 1, buf ^ 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    y[i & 1] = mfma32(f[i % AHEAD], q[i >> 1], i < 2 ? zero : y[i & 1]);
                    const int r = i + AHEAD;
                    if (!F8 && r == NS) loads_barrier<L>();  // V is there
                    f[i % AHEAD] = r < NS ? k_frag(r & 1, r >> 1, buf ^ 1) : v_frag((r - NS) % (D / 32), (r - NS) / (D / 32), buf);
                    if (i < L) load.k.part(i);
                    powers(i);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    const int n = i % (D / 32), k = i / (D / 32), r = i + AHEAD;
                    o[n] = mfma32(f[i % AHEAD], p[k], o[n]);
                    if (const int j = F8 ? i - NS / 2 : i; j >= 0 && j < L) load.v.part(j);
                    if (r < NS) f[i % AHEAD] = v_frag(r % (D / 32), r / (D / 32), buf);
                    powers(NS + i);
                    if (i >= NS / 2) {
#pragma unroll
                        for (int e = (i - NS / 2) * 64 / NS; e < (i - NS / 2 + 1) * 64 / NS; ++e)
                            top = fmaxf(top, y[e >> 4][e & 15]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                top = largest(top);
            };
            int t0 = begin, buf = 0;
            // (pages of fewer than 16 rows take the plain loop below for all tiles)
            const int open = missing || a.page_shift < 4 ? begin : min(max(open_end, begin), end - 1);
            {
                f32x16 y[2];
                while (t0 + kKeys <= open) {
                    turn(x, y, t0, std::integral_constant<int, 0>());
                    t0 += kKeys;
                    if (t0 + kKeys > open) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) x[j] = y[j];
                        buf = 1;
                        break;
                    }
                    turn(y, x, t0, std::integral_constant<int, 1>());
                    t0 += kKeys;
                }
            }

            // Other tiles, step by step.
#pragma unroll 1
            for (; t0 < end; t0 += kKeys, buf ^= 1) {
                arrive(t0, buf, std::integral_constant<int, 0>(), std::false_type());
                if (t0 + kKeys < end) rest();
                uint32_t see[2];
                bool odd = false;
                const bool masked = missing || t0 + kKeys > min(open_end, end);
                if (masked) {
                    odd = __builtin_amdgcn_readfirstlane(__syncthreads_or(any_odd<D>(lds_v + buf * VL::kTile, tid)));
                    if (odd) {
                        rewrite<D>(lds_v + buf * VL::kTile, 0, tid);
                        __syncthreads();
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t bits = 0xffffffffu;
                    if (missing) {
                        const int t = t0 + 32 * j + col;
                        const int page = t < end ? table[t >> a.page_shift] : -1;
                        bits = uint32_t(__ballot(page >= 0 && page < a.cache.n_pages));
                    }
                    if (masked)
                        bits &= visible<KIND>(a, s, token,
                                              KIND == kAttnVerify
                                                  ? a.anc + (int64_t(at.b) * s.n + token) * ((a.d.T + 31) >> 5)
                                                  : nullptr,
                                              t0 + 32 * j, end);
                    see[j] = bits >> (4 * half);
                }
                bf16x8 p[4];
                float most = -inf;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    if (!(see[i >> 4] >> (8 * (i >> 2 & 3) + (i & 3)) & 1)) x[i >> 4][i & 15] = -inf;
                    most = fmaxf(most, x[i >> 4][i & 15]);
                }
                raise(largest(most));
                const float base = finite_max(m);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float e = exp2_fast(fmaf(x[i >> 4][i & 15], scale, -base));
                    // a scale of zero turns -inf into NaN
                    if (!(see[i >> 4] >> (8 * (i >> 2 & 3) + (i & 3)) & 1)) e = 0.0f;
                    p[i >> 3][i & 7] = static_cast<__bf16>(e);
                    l += static_cast<float>(p[i >> 3][i & 7]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int n = 0; n < D / 32; ++n) {
                        const bf16x8 f = v_frag(n, k, buf);
                        o[n] = mfma32(f, p[k], o[n]);
                    }
#pragma unroll 1
                for (int kind = 1; odd && kind <= 3; ++kind) {
                    const float what = kind == 1 ? __builtin_nanf("") : kind == 2 ? inf : -inf;
                    const uint32_t to = lds_v + buf * VL::kTile;
                    const int tid = fresh(threadIdx.x), lane = tid & 63;
                    __syncthreads();
                    Loader<D, F8> again = load;
                    again.find(a, table, t0, end, wave, lane);
                    if (a.page_shift >= 4) {
                        again.v.init(a, h, lane);
                        again.v.at(to, again.page, again.row, wave);
#pragma unroll
                        for (int i = 0; i < L; ++i) again.v.part(i);
                    } else {
                        again.v.scattered(a, again.window, to, t0, end, wave, lane);
                    }
                    again.v.store(to, wave, lane);
                    loads_barrier<0>();
                    rewrite<D>(to, kind, tid);
                    __syncthreads();
#pragma unroll
                    for (int n = 0; n < D / 32; ++n) {
                        f32x16 count = zero;
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
                if (t0 + kKeys < end) {
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        const bf16x8 f = k_frag(i & 1, i >> 1, buf ^ 1);
                        x[i & 1] = mfma32(f, q[i >> 1], i < 2 ? zero : x[i & 1]);
                    }
                }
            }
        }

        l += __shfl_xor(l, 32);
        const int r = wave * 32 + col;
        if (r < rows) {
            if (it.units < it.all) {
                // 4 elements of each lane at a time, as they lie in the registers
                float* part = part_out(a, 2 * int64_t(range.w) + (first ? 0 : 1), kTileRows, D);
                f32x4* out = reinterpret_cast<f32x4*>(part) + wave * (D / 4 * 32) + lane;
#pragma unroll
                for (int n = 0; n < D / 32; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        out[(4 * n + i) * 64] = f32x4{o[n][4 * i], o[n][4 * i + 1], o[n][4 * i + 2], o[n][4 * i + 3]};
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
        if (u < range.end) __syncthreads();  // the next piece overwrites LDS
    }
}

template <AttnKind KIND, int D, bool F8>
hipError_t launch_one(const AttnArgs& a, const dim3& grid, hipStream_t stream) {
    const auto kernel = tiles_kernel<KIND, D, F8>;
    constexpr int bytes = TileLds<D>::kBytes;
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
    const dim3 grid(attn_grid(a));
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
