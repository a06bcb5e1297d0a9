// gdn_attn_plan.h -- which keys of which queries a workgroup of the attention
// kernels takes, and where it leaves its part of a result.
//
// The work is numbered in units of some keys of one tile of rows: through the
// tiles of a sequence, the sequences, then the key heads.  Workgroup w takes
// units w per .. (w + 1) per - 1, with per = max(min_units, all / teams), so the
// workgroups that fit the GPU at once (`teams`) have the same work however
// uneven the lengths are, and nothing has to be known on the host.  A range
// covers any number of whole tiles, whose results are final, and at most two
// tiles in part (one where it starts, one where it ends), whose results go to
// parts 2 w and 2 w + 1 of the workspace and are joined by another launch.
//
// In a prompt the last tile sees most keys and the first fewest, so tiles are
// taken in pairs from both ends, and every pair counts the same (the middle one of
// an odd number, too, whose second half is empty).  The tiles of a
// tree all see the same keys: a team of as many workgroups takes them side by
// side, as one unit, so that the keys come from memory once.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gdn_attn_internal.h"
#include "gdn_layer_util.h"
#include "gdn_mfma.h"

namespace gdn {

struct AttnSeq {
    int n;         // query tokens
    int64_t row0;  // first row of q
    int prefix;    // verify: tokens before the tree; prefill: length - n (may be negative)
    int keys;      // tokens of the cache that any of its queries may see
};

template <AttnKind KIND>
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int b) {
    AttnSeq s;
    const int cap = a.d.max_pages << a.page_shift;
    const int len = min(max(a.length[b], 0), cap);
    if constexpr (KIND == kAttnDecode) {
        s.n = 1;
        s.row0 = b;
        s.prefix = len - 1;
        s.keys = len;
    } else if constexpr (KIND == kAttnVerify) {
        s.n = a.d.T;
        s.row0 = int64_t(b) * a.d.T;
        s.prefix = len;
        s.keys = min(len + a.d.T, cap);
    } else {
        const int start = a.cu[b], end = a.cu[b + 1];
        const bool fine = start >= 0 && start <= end && end <= a.d.T;
        s.n = fine ? end - start : 0;
        s.row0 = start;
        s.prefix = len - s.n;
        s.keys = s.n > 0 ? len : 0;
    }
    return s;
}

template <AttnKind KIND>
__device__ __forceinline__ int attn_tiles(const AttnArgs& a, const AttnSeq& s) {
    if constexpr (KIND != kAttnPrefill) return 1;  // a tree: each workgroup of a team has one
    return int((int64_t(s.n) * a.group + a.tile_rows - 1) / a.tile_rows);
}

// Keys that any row of a tile may see.
template <AttnKind KIND>
__device__ __forceinline__ int attn_seen(const AttnArgs& a, const AttnSeq& s, int tile) {
    if constexpr (KIND != kAttnPrefill) return s.keys;
    const int64_t end = min(int64_t(tile + 1) * a.tile_rows, int64_t(s.n) * a.group);  // rows
    return max(min(int(s.prefix + (end - 1) / a.group + 1), s.keys), 0);
}
// A tile's units: at least one, so that rows which see nothing are written.
template <AttnKind KIND>
__device__ __forceinline__ int attn_units(const AttnArgs& a, const AttnSeq& s, int tile) {
    return max((attn_seen<KIND>(a, s, tile) + (1 << a.unit_shift) - 1) >> a.unit_shift, 1);
}
// The units that a pair of tiles counts (prefill: at least those of any pair,
// whose keys sum to 2 prefix + tile_rows (tiles + 1) / group + 2 at most), and
// those of a sequence.
template <AttnKind KIND>
__device__ __forceinline__ int attn_pair(const AttnArgs& a, const AttnSeq& s, int tiles) {
    if constexpr (KIND != kAttnPrefill) return attn_units<KIND>(a, s, 0);
    const int64_t keys = 2 * int64_t(max(s.prefix, 0)) + (int64_t(tiles) + 1) * a.tile_rows / a.group + 2;
    return int(keys >> a.unit_shift) + 2;
}
template <AttnKind KIND>
__device__ __forceinline__ int64_t attn_seq_units(const AttnArgs& a, const AttnSeq& s, int tiles) {
    return int64_t(attn_pair<KIND>(a, s, tiles)) * (KIND == kAttnPrefill ? (tiles + 1) / 2 : tiles);
}

__device__ __forceinline__ int64_t wave_sum64(int64_t x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
    return x;
}
__device__ __forceinline__ int64_t wave_scan64(int64_t x, int lane) {  // inclusive
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    return x;
}
__device__ __forceinline__ int64_t read_lane64(int64_t x, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(x), lane), hi = __builtin_amdgcn_readlane(uint32_t(x >> 32), lane);
    return int64_t(uint64_t(hi) << 32 | lo);
}

// a / b of numbers >= 0 that all lanes agree on; of 32 bits, as most are, it takes a tenth of the instructions.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if ((a | b) >> 32) return a / b;
    return __builtin_amdgcn_readfirstlane(uint32_t(a) / uint32_t(b));
}

// The units of one key head (and head tile), those of a workgroup (team), and
// the number of workgroups (teams) that have any.
struct AttnPlan {
    int64_t units, per;
    int ranges;
};
// A sequence that all lanes agree on, its first unit within the key head, and
// how many it has; and the first of the 64 sequences that it was found among,
// with the units before them.
struct AttnPlace {
    int b = -1, base = 0;
    int64_t first = 0, count = 0, before = 0;
    AttnSeq s;
};
// What a lane knows of 64 sequences in a row.
template <AttnKind KIND>
struct AttnLane {
    AttnSeq s{0, 0, 0, 0};
    int64_t units = 0;
    __device__ __forceinline__ void read(const AttnArgs& a, int b) {
        s = AttnSeq{0, 0, 0, 0};
        units = 0;
        if (b < a.d.B) {
            s = attn_seq<KIND>(a, b);
            units = attn_seq_units<KIND>(a, s, attn_tiles<KIND>(a, s));
        }
    }
};
// The sequence among those from `base` on that holds unit `u` (BY_NUMBER: that
// is sequence u); otherwise the units before the next ones.
template <AttnKind KIND, bool BY_NUMBER>
__device__ __forceinline__ bool attn_find_here(const AttnArgs& a, const AttnLane<KIND>& x, int base, int64_t u, int lane,
                                               int64_t& before, AttnPlace& at) {
    const int64_t end = a.d.B > 1 ? wave_scan64(x.units, lane) : x.units, first = before + end - x.units;
    const uint64_t here = __ballot(BY_NUMBER ? base + lane == u : u >= first && u < first + x.units);
    if (here) {
        const int src = __builtin_ctzll(here);
        at.b = base + src;
        at.base = base;
        at.before = before;
        at.first = read_lane64(first, src);
        at.count = read_lane64(x.units, src);
        at.s.n = __builtin_amdgcn_readlane(x.s.n, src);
        at.s.row0 = read_lane64(x.s.row0, src);
        at.s.prefix = __builtin_amdgcn_readlane(x.s.prefix, src);
        at.s.keys = __builtin_amdgcn_readlane(x.s.keys, src);
        return true;
    }
    before += read_lane64(end, 63);
    return false;
}
template <AttnKind KIND, bool BY_NUMBER>
__device__ __forceinline__ void attn_find(const AttnArgs& a, int base, int64_t before, int64_t u, int lane, AttnPlace& at) {
    for (; base < a.d.B; base += 64) {
        AttnLane<KIND> x;
        x.read(a, base + lane);
        if (attn_find_here<KIND, BY_NUMBER>(a, x, base, u, lane, before, at)) return;
    }
}
// The place of a later unit of the same workgroup, from where the last one was.
template <AttnKind KIND>
__device__ __forceinline__ void attn_next(const AttnArgs& a, int64_t u, int lane, AttnPlace& at) {
    if (u >= at.first && u < at.first + at.count) return;
    const bool on = u >= at.before;  // not in the next key head
    attn_find<KIND, false>(a, on ? at.base : 0, on ? at.before : 0, u, lane, at);
}

// The plan; `x`: what the lanes have read of the first 64 sequences.
template <AttnKind KIND>
__device__ __forceinline__ AttnPlan attn_plan(const AttnArgs& a, int lane, AttnLane<KIND>& x) {
    x.read(a, lane);
    int64_t units = x.units;
#pragma unroll 4
    for (int b = lane + 64; b < a.d.B; b += 64) {
        AttnLane<KIND> y;
        y.read(a, b);
        units += y.units;
    }
    AttnPlan p;
    p.units = read_lane64(a.d.B == 1 ? units : wave_sum64(units), 0);
    const int64_t all = p.units * (a.cache.H_kv * a.head_tiles);
    p.per = max(quotient(all + a.teams - 1, a.teams), int64_t(a.min_units));
    p.ranges = int(quotient(all + p.per - 1, p.per));
    return p;
}

// A workgroup's range, and the place of its first unit.
struct AttnRange {
    int w, team, mate;  // its number, its team and its place there
    int64_t u, end, units;
};
template <AttnKind KIND>
__device__ __forceinline__ bool attn_begin(const AttnArgs& a, int wg, int lane, AttnRange& r, AttnPlace& at) {
    AttnLane<KIND> x;
    const AttnPlan plan = attn_plan<KIND>(a, lane, x);
    r.w = attn_number(plan.ranges * a.team, wg);
    if (r.w < 0) return false;
    r.team = a.team == 1 ? r.w : __builtin_amdgcn_readfirstlane(r.w / a.team);
    r.mate = r.w - r.team * a.team;
    r.units = plan.units;
    r.u = r.team * plan.per;
    r.end = min(r.u + plan.per, plan.units * (a.cache.H_kv * a.head_tiles));
    const int64_t uh = r.u - quotient(r.u, plan.units) * plan.units;
    int64_t before = 0;
    if (!attn_find_here<KIND, false>(a, x, 0, uh, lane, before, at)) attn_find<KIND, false>(a, 64, before, uh, lane, at);
    return true;
}

// A tile, and some of its units.
struct AttnPiece {
    int tile, unit, units, all;  // units from `unit` on, of all the tile's
};
__device__ __forceinline__ AttnPiece uniform(AttnPiece x) {
    x.tile = __builtin_amdgcn_readfirstlane(x.tile);
    x.unit = __builtin_amdgcn_readfirstlane(x.unit);
    x.units = __builtin_amdgcn_readfirstlane(x.units);
    x.all = __builtin_amdgcn_readfirstlane(x.all);
    return x;
}
// What of a sequence lies at its unit `off`, at most `most` units; all == 0: the
// next `units` count nothing (a pair has fewer than it counts).
template <AttnKind KIND>
__device__ __forceinline__ AttnPiece attn_piece(const AttnArgs& a, const AttnSeq& s, int tiles, int64_t off, int64_t most) {
    const int pair = attn_pair<KIND>(a, s, tiles);
    const int p = int(quotient(off, pair));
    AttnPiece x;
    x.unit = int(off - int64_t(p) * pair);
    if constexpr (KIND == kAttnPrefill) {
        x.tile = tiles - 1 - p;
        x.all = attn_units<KIND>(a, s, x.tile);
        if (x.unit >= x.all) {
            x.unit -= x.all;
            x.all = x.tile != p ? attn_units<KIND>(a, s, p) : 0;
            const int last = pair - attn_units<KIND>(a, s, x.tile);
            x.tile = p;
            if (x.unit >= x.all) {
                x.units = int(min(int64_t(last - x.unit), most));
                x.all = 0;
                return uniform(x);
            }
        }
    } else {
        x.tile = p;
        x.all = pair;
    }
    x.units = int(min(int64_t(x.all - x.unit), most));
    return uniform(x);
}
// Part `part` of the workspace: a tile's unnormalised outputs over some of its
// keys (in the order that suits the kernel that writes them), then the running
// maximum (in powers of two) and sum of every row.
__device__ __forceinline__ float* part_out(const AttnArgs& a, int64_t part, int rows, int D) {
    return static_cast<float*>(a.ws) + part * rows * (D + 2);
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

constexpr float kLog2e = 1.4426950408889634f;

// What is above a row's maximum in exponents: zero for rows that have seen
// nothing (a maximum of -inf), so that their powers are 0 and not NaN.
__device__ __forceinline__ float finite_max(float m) { return m == -__builtin_inff() ? 0.0f : m; }

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Elements d0 .. d0 + 3 of query head `head` (of key head h) of row `row`:
// the accumulated values over the sum of the powers, rounded once.
template <int D>
__device__ __forceinline__ void attn_store(const AttnArgs& a, int64_t row, int h, int64_t head, int d0, const f32x4& acc,
                                           float sum) {
    float f = sum == 0.0f ? 0.0f : 1.0f / sum;  // nothing was visible: zero
    if (a.cache.v_scale) f *= a.cache.v_scale[h];
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = acc[j] * f;
    if (a.gate && sum != 0.0f) {
        const uint16_t* z = a.gate + row * a.d.gate_stride + head * a.d.gate_head_stride + d0;
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] *= sigmoidf(__builtin_bit_cast(float, uint32_t(z[j]) << 16));
    }
    *reinterpret_cast<uint2*>(a.o + (row * a.d.H_q + head) * D + d0) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
}

// 16 e4m3 values as bf16 (exact).
__device__ __forceinline__ void e4m3_to_bf16(const uint4& u, uint4& lo, uint4& hi) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t r[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        r[2 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[j], 1.0f, false));
        r[2 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[j], 1.0f, true));
    }
    lo = make_uint4(r[0], r[1], r[2], r[3]);
    hi = make_uint4(r[4], r[5], r[6], r[7]);
}

// Four 16-bit elements of each lane, transposed over groups of 16 lanes: lane
// 4 r + c of a group gives elements 4 c .. 4 c + 3 of row r of a 4 x 16 tile,
// and lane i receives column i.
__device__ __forceinline__ uint2 read_tr16(uint32_t lds) {
    typedef short s16x4v __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         reinterpret_cast<__attribute__((address_space(3))) s16x4v*>(lds)));
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return uint32_t(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)p));
}

}  // namespace gdn
