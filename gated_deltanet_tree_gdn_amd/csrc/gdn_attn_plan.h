// gdn_attn_plan.h -- which keys of which sequence a workgroup of the attention
// kernels takes, and where it leaves its part of the result.
//
// Lengths are on the device, so the division is made there, by every
// wavefront for itself: a tile's work is its sequence's keys, the keys are cut
// into chunks of
//     c = max(min_chunk, sum over tiles of keys / spread)
// (a multiple of min_chunk), and the items (tile, chunk) are numbered through
// the sequences.  That gives at most spread + tiles items of at most c keys,
// however uneven the lengths are, and of those that are one of several chunks
// of their tile at most 2 spread, which is what the workspace has room for.
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

// The same of a sequence that all lanes agree on.
template <AttnKind KIND>
__device__ __forceinline__ AttnSeq attn_seq_uniform(const AttnArgs& a, int b) {
    AttnSeq s = attn_seq<KIND>(a, b);
    s.n = __builtin_amdgcn_readfirstlane(s.n);
    s.row0 = KIND == kAttnPrefill ? __builtin_amdgcn_readfirstlane(int(s.row0)) : s.row0;
    s.prefix = __builtin_amdgcn_readfirstlane(s.prefix);
    s.keys = __builtin_amdgcn_readfirstlane(s.keys);
    return s;
}

template <AttnKind KIND>
__device__ __forceinline__ int attn_tiles(const AttnArgs& a, const AttnSeq& s) {
    if constexpr (KIND == kAttnDecode) return 1;
    return int((int64_t(s.n) * a.group + a.tile_rows - 1) / a.tile_rows);
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

// Keys of a chunk.
template <AttnKind KIND>
__device__ __forceinline__ int attn_chunk(const AttnArgs& a, int lane) {
    int64_t total = 0;
    if (a.d.B == 1) {
        const AttnSeq s = attn_seq<KIND>(a, 0);
        total = int64_t(attn_tiles<KIND>(a, s)) * s.keys;
    } else {
        for (int b = lane; b < a.d.B; b += 64) {
            const AttnSeq s = attn_seq<KIND>(a, b);
            total += int64_t(attn_tiles<KIND>(a, s)) * s.keys;
        }
        total = wave_sum64(total);
    }
    const int64_t c = max((total + a.spread - 1) / a.spread, int64_t(1));
    return __builtin_amdgcn_readfirstlane(int(min((c + a.min_chunk - 1) / a.min_chunk * a.min_chunk, int64_t(1) << 30)));
}

struct AttnItem {
    int b, tile, chunk, chunks;
    int64_t part;  // of the tile's first chunk in the workspace, if chunks > 1
};

// Item `i` (a (tile, chunk), or with TILES a whole tile); false behind the last.
template <AttnKind KIND, bool TILES>
__device__ __forceinline__ bool attn_item(const AttnArgs& a, int c, int64_t i, int lane, AttnItem& it) {
    int64_t items0 = 0, parts0 = 0;
    for (int base = 0; base < a.d.B; base += 64) {
        const int b = base + lane;
        int tiles = 0, chunks = 1;
        if (b < a.d.B) {
            const AttnSeq s = attn_seq<KIND>(a, b);
            tiles = attn_tiles<KIND>(a, s);
            chunks = max((s.keys + c - 1) / c, 1);
        }
        const int64_t items = int64_t(tiles) * (TILES ? 1 : chunks), parts = chunks > 1 ? int64_t(tiles) * chunks : 0;
        int64_t items_end = items, parts_end = parts;
        if (a.d.B > 1) {
            items_end = wave_scan64(items, lane);
            parts_end = wave_scan64(parts, lane);
        }
        const int64_t first = items0 + items_end - items;
        const uint64_t here = __ballot(i >= first && i < first + items);
        if (here) {
            const int src = __builtin_ctzll(here);
            it.b = base + src;
            it.chunks = __builtin_amdgcn_readlane(chunks, src);
            // the item's number within its sequence is below 2^31 (rows and chunks are)
            const uint32_t at = uint32_t(i - read_lane64(first, src));
            it.tile = TILES ? at : at / uint32_t(it.chunks);
            it.chunk = TILES ? 0 : at - it.tile * it.chunks;
            it.part = parts0 + read_lane64(parts_end - parts, src) + int64_t(it.tile) * it.chunks;
            return true;
        }
        items0 += read_lane64(items_end, 63);
        parts0 += read_lane64(parts_end, 63);
    }
    return false;
}

// A tile's parts over chunks of keys: unnormalised outputs, then the running
// maximum (in powers of two) and sum of every row.
__device__ __forceinline__ float* part_out(const AttnArgs& a, int64_t part, int hh, int rows, int D) {
    return static_cast<float*>(a.ws) + (int64_t(hh) * a.part_tiles + part) * rows * (D + 2);
}

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
__device__ __forceinline__ uint2 read_tr16(const void* lds) {
    typedef short s16x4v __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(
        uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4v*)(lds)));
}

}  // namespace gdn
