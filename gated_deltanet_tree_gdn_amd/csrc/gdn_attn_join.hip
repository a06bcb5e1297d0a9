// gdn_attn_join.hip -- what the attention kernels share: the join of tiles whose
// keys were divided, and the verdict on a call's sequences.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gdn_attn_internal.h"
#include "gdn_attn_plan.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// Workgroups that join a tile (or team), whose threads take `pieces` times 4 elements.
__host__ __device__ inline int join_blocks(const AttnArgs& a, int pieces) {
    const int rows = a.group < kDecodeRows ? a.group : kDecodeRows;
    return a.kind == kAttnDecode ? rows : kTileRows * (a.cache.d / 4) / (kThreads * pieces) * a.team;
}

struct Joined {
    f32x4 acc{0, 0, 0, 0};
    float m = -__builtin_inff(), l = 0.0f;
    __device__ __forceinline__ void add(const f32x4& x, float mx, float lx) {
        const float top = fmaxf(m, mx), base = finite_max(top);
        const float f = exp2_fast(m - base), fx = exp2_fast(mx - base);
        acc = acc * f + x * fx;
        l = l * f + lx * fx;
        m = top;
    }
};

// Parts of a tile's rows, joined in the order of the keys.  Where BY_TILE, there
// are workgroups for every tile (which is all of a sequence, as a prompt's are
// not), otherwise for every end of a range within a tile, of which the first
// joins it: whichever are fewer, since each of them has to find its place.
// Single tokens: a workgroup for every row, since there are few and their parts
// may be hundreds; its threads take the parts in turn.  Tiles: every thread has `pieces` pieces of 4 elements, in
// the order in which the parts hold them.  Measured: 4.5 us for a single
// token's two tiles in 12 parts each; by ends of ranges instead of by tiles:
// prompts of 6007 tokens behind 20011, 9 sequences, 410 us instead of 470, all
// in all.
template <AttnKind KIND, int D, bool BY_TILE>
__global__ __launch_bounds__(kThreads) void join_kernel(AttnArgs a, int64_t workgroups, int pieces) {
    constexpr int C = D / 4, K = kThreads / C;  // threads of a row, shares of the parts (single tokens)
    constexpr bool one = KIND == kAttnDecode;
    constexpr int rows_of_part = one ? kDecodeRows : kTileRows;
    __shared__ f32x4 share[one ? K : 1][C];
    __shared__ float share_m[4], share_l[one ? K : 1];
    const int tid = threadIdx.x, lane = tid & 63;
    const int heads = a.cache.H_kv * a.head_tiles;
    const int blocks = join_blocks(a, pieces);
    const int64_t wg = block_id();
    if (wg >= workgroups) return;
    const int block = int(wg % blocks) / a.team, mate = int(wg % blocks) % a.team;
    AttnLane<KIND> x;
    const AttnPlan plan = attn_plan<KIND>(a, lane, x);
    AttnPlace at;
    int hh, t = 0;
    int64_t g0, before = 0;  // g0: the tile's first unit
    if constexpr (BY_TILE) {
        const int b = int(wg / blocks / heads);
        hh = int(wg / blocks % heads);
        if (!attn_find_here<KIND, true>(a, x, 0, b, lane, before, at)) attn_find<KIND, true>(a, 64, before, b, lane, at);
        g0 = hh * plan.units + at.first;
    } else {
        const int64_t w = wg / blocks + 1;
        if (w >= plan.ranges) return;
        const int64_t g = w * plan.per;
        hh = int(quotient(g, plan.units));
        const int64_t uh = g - hh * plan.units;
        if (!attn_find_here<KIND, false>(a, x, 0, uh, lane, before, at)) attn_find<KIND, false>(a, 64, before, uh, lane, at);
        const AttnPiece it = attn_piece<KIND>(a, at.s, attn_tiles<KIND>(a, at.s), uh - at.first, 1);
        if (it.all == 0 || it.unit == 0 || it.unit > plan.per) return;
        t = it.tile;
        g0 = g - it.unit;
    }
    const AttnSeq s = at.s;
    const int h = hh / a.head_tiles;
    const int64_t w0 = quotient(g0, plan.per), w1 = quotient(g0 + attn_units<KIND>(a, s, t) - 1, plan.per);
    const int parts = int(w1 - w0) + 1;
    if (parts == 1) return;
    // the first workgroup either starts with this tile or has it as its last
    auto part = [&](int i) {
        return part_out(a, 2 * ((w0 + i) * a.team + mate) + (i == 0 && g0 != w0 * plan.per), rows_of_part, D);
    };
    if constexpr (one) {
        // maxima first, so that the parts' outputs are loads that wait for nothing but their weights
        const int head0 = (hh - h * a.head_tiles) * kDecodeRows, row = block;
        if (row < a.group - head0) {
            float top = -__builtin_inff();
            for (int i = tid; i < parts; i += kThreads) top = fmaxf(top, part(i)[kDecodeRows * D + row]);
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
            if (lane == 0) share_m[tid >> 6] = top;
            __syncthreads();
            top = finite_max(fmaxf(fmaxf(share_m[0], share_m[1]), fmaxf(share_m[2], share_m[3])));
            const int p = tid % C, k = tid / C;
            f32x4 acc{0, 0, 0, 0};
            float sum = 0.0f;
#pragma unroll 4
            for (int i = k; i < parts; i += K) {
                const float* z = part(i);
                const float f = exp2_fast(z[kDecodeRows * D + row] - top);
                acc += *reinterpret_cast<const f32x4*>(z + row * D + 4 * p) * f;
                sum += z[kDecodeRows * (D + 1) + row] * f;
            }
            share[k][p] = acc;
            if (p == 0) share_l[k] = sum;
            __syncthreads();
            if (k == 0) {
                for (int i = 1; i < K; ++i) {
                    acc += share[i][p];
                    sum += share_l[i];
                }
                attn_store<D>(a, s.row0, h, int64_t(h) * a.group + head0 + row, 4 * p, acc, sum);
            }
        }
    } else {
        const int row0 = (KIND == kAttnVerify ? mate : t) * kTileRows, rows = min(kTileRows, s.n * a.group - row0);
        for (int j = 0; j < pieces; ++j) {
            const int e = (block * pieces + j) * kThreads + tid;  // 32 rows have 32 C pieces
            const int r = e / (32 * C) * 32 + (e & 31), d = e / 64 % (C / 2) * 8 + (e >> 5 & 1) * 4;
            if (r >= rows) continue;
            Joined y;
#pragma unroll 4
            for (int i = 0; i < parts; ++i) {
                const float* z = part(i);
                y.add(reinterpret_cast<const f32x4*>(z)[e], z[kTileRows * D + r], z[kTileRows * (D + 1) + r]);
            }
            const int token = (row0 + r) / a.group;
            attn_store<D>(a, s.row0 + token, h, int64_t(h) * a.group + row0 + r - token * a.group, d, y.acc, y.l);
        }
    }
}

// One workgroup per sequence reads what the attention kernels read of its
// length, its place among the rows and its pages.
__global__ __launch_bounds__(kThreads) void status_kernel(AttnArgs a) {
    const int b = blockIdx.x;
    const int64_t cap = int64_t(a.d.max_pages) << a.page_shift, len = a.length[b];
    int64_t keys = len;
    bool bad = len < 0 || len > cap;
    if (a.kind == kAttnVerify) {
        keys += a.d.T;
        bad |= keys > cap;
    } else if (a.kind == kAttnPrefill) {
        const int start = a.cu[b], end = a.cu[b + 1];
        bad |= start < 0 || start > end || end > a.d.T || end - start > len;
        if (start == end) keys = 0;
    }
    keys = keys < 0 ? 0 : keys < cap ? keys : cap;
    for (int64_t p = threadIdx.x; p << a.page_shift < keys; p += kThreads) {
        const int page = a.table[b * a.d.table_stride + p];
        bad |= page < 0 || page >= a.cache.n_pages;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) a.seq_status[b] = bad ? GDN_ERR_SHAPE : 0;
}

template <AttnKind KIND, bool BY_TILE>
hipError_t launch_join(const AttnArgs& a, int64_t tiles, hipStream_t stream) {
    // half as many workgroups as the GPU has room for, or more: a thread with one piece waits for memory only once, but every
    // workgroup has to find its place (one piece against two: 38 us and 40 us for a tree of 48 nodes behind
    // 2855 tokens, but 448 us and 436 us for prompts of 6007 tokens behind 20011)
    int pieces = 1;
    while (KIND != kAttnDecode && pieces < 8 && tiles * join_blocks(a, 2 * pieces) >= 1024) pieces *= 2;
    const int64_t workgroups = tiles * join_blocks(a, pieces);
    const dim3 grid = grid_of(workgroups);
    switch (a.cache.d) {
        case 64: join_kernel<KIND, 64, BY_TILE><<<grid, kThreads, 0, stream>>>(a, workgroups, pieces); break;
        case 128: join_kernel<KIND, 128, BY_TILE><<<grid, kThreads, 0, stream>>>(a, workgroups, pieces); break;
        default: join_kernel<KIND, 256, BY_TILE><<<grid, kThreads, 0, stream>>>(a, workgroups, pieces); break;
    }
    return hipGetLastError();
}
template <AttnKind KIND>
hipError_t launch_join(const AttnArgs& a, hipStream_t stream) {
    const int64_t tiles = int64_t(a.d.B) * a.cache.H_kv * a.head_tiles, ends = a.teams - 1;
    if constexpr (KIND != kAttnPrefill)  // how many tiles prompts have is not known here
        if (tiles <= ends) return launch_join<KIND, true>(a, tiles, stream);
    return launch_join<KIND, false>(a, ends, stream);
}

}  // namespace

hipError_t launch_attn_join(const AttnArgs& a, hipStream_t stream) {
    return a.kind == kAttnDecode   ? launch_join<kAttnDecode>(a, stream)
           : a.kind == kAttnVerify ? launch_join<kAttnVerify>(a, stream)
                                   : launch_join<kAttnPrefill>(a, stream);
}

hipError_t launch_attn_status(const AttnArgs& a, hipStream_t stream) {
    status_kernel<<<a.d.B, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace gdn
