// gdn_kv.hip -- the paged cache's writers: gdn_kv_append and gdn_kv_commit.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gdn_attn_internal.h"
#include "gdn_layer_util.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 8 floats as e4m3, to nearest even, clamped to the largest finite value;
// infinities and NaN become NaN.
__device__ __forceinline__ uint2 pack_e4m3(const float (&x)[8]) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        y[j] = __builtin_isfinite(x[j]) ? fminf(fmaxf(x[j], -448.0f), 448.0f) : __builtin_nanf("");
    int a = 0, b = 0;
    a = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], a, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], a, true);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], b, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], b, true);
    return make_uint2(a, b);
}

// 8 elements of any alignment as they lie in memory.
struct Raw {
    typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
    u32x4 a, b;
    __device__ __forceinline__ void load(const void* p, int dtype, int64_t i) {
        const char* at = static_cast<const char*>(p) + i * (dtype == GDN_BF16 ? 2 : 4);
        a = *reinterpret_cast<const u32x4u*>(at);
        if (dtype != GDN_BF16) b = *reinterpret_cast<const u32x4u*>(at + 16);
    }
    __device__ __forceinline__ void unpack(int dtype, float (&x)[8]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t u = a[j], v = b[j];
            if (dtype == GDN_BF16) {
                x[2 * j] = bf16_lo(u);
                x[2 * j + 1] = bf16_hi(u);
            } else {
                x[j] = __builtin_bit_cast(float, u);
                x[4 + j] = __builtin_bit_cast(float, v);
            }
        }
    }
};

// ---------------------------------------------------------------------------
// gdn_kv_append.  A head's d elements lie 8 to a lane in d / 8 adjacent lanes,
// so its norm is a sum over lanes, and a pair of neighbours turns within a
// lane; a pair of halves meets through the wavefront's own LDS rows.  Cosines
// and sines of a token are formed once by the first rot / 2 threads of each
// workgroup: the angle position * inv_freq is exact to 2^-53 in fp64, reduced
// there to a fraction of a turn, and from then on fp32 is enough for outputs
// of 8 bits.  A workgroup takes `passes` times 256 / (d / 8) heads of one token;
// the elements of a pass are on their way while the one before (the first:
// while the angles) is worked on.  Memory bounds it: 12289 tokens of 32 + 2 x 8
// heads of 128 into an e4m3 cache take 71 us, 3.9 TB/s; a single token 4 us, a
// launch and loads that wait for each other.
// ---------------------------------------------------------------------------
template <int D>
__global__ __launch_bounds__(kThreads) void append_kernel(KvAppendArgs a, int passes, int groups, int page_shift) {
    constexpr int L = D / 8, PER = kThreads / L;  // lanes of a head, heads of a pass
    __shared__ float cs[128], sn[128];
    __shared__ alignas(16) float rows[kThreads * 8];
    const int tid = threadIdx.x;
    const int64_t wg = block_id();
    const int64_t t = groups == 1 ? wg : wg / groups;
    if (t >= a.d.T) return;
    const int group = int(wg - t * groups);
    const int H_q = a.d.H_q, H_kv = a.cache.H_kv, heads = H_q + 2 * H_kv;
    const int half = a.d.rot >> 1;
    const int e = 8 * (tid % L);

    Raw next;
    auto fetch = [&](int p) {
        const int head = (group * passes + p) * PER + tid / L;
        if (head >= heads) return;
        const bool is_q = head < H_q, is_v = head >= H_q + H_kv;
        const int h = is_q ? head : is_v ? head - H_q - H_kv : head - H_q;
        const void* src = is_q ? a.q : is_v ? a.v : a.k;
        const int64_t ts = is_q ? a.d.q_stride : is_v ? a.d.v_stride : a.d.k_stride;
        const int64_t hs = is_q ? a.d.q_head_stride : is_v ? a.d.v_head_stride : a.d.k_head_stride;
        next.load(src, a.d.in_dtype, t * ts + h * hs + e);
    };
    fetch(0);
    const int32_t slot = a.slot[t];
    if (tid < half) {
        double turn = double(a.position[t]) * double(a.inv_freq[tid]) * 0.15915494309189533577;
        turn -= rint(turn);
        float s, c;
        sincospif(2.0f * float(turn), &s, &c);
        cs[tid] = c;
        sn[tid] = s;
    }
    const bool stored = slot >= 0 && slot < a.cache.n_pages << page_shift;
    const int page = slot >> page_shift, page_row = slot & (a.cache.page_size - 1);
    if (half > 0) __syncthreads();

    float* mine = rows + (tid / L) * D;
    for (int p = 0; p < passes; ++p) {
        const int head = (group * passes + p) * PER + tid / L;
        const bool live = head < heads;
        const bool is_q = head < H_q, is_v = head >= H_q + H_kv;
        const int h = is_q ? head : is_v ? head - H_q - H_kv : head - H_q;
        float x[8] = {};
        if (live) next.unpack(a.d.in_dtype, x);
        if (p + 1 < passes) fetch(p + 1);
        const float* w = is_q ? a.q_weight : is_v ? nullptr : a.k_weight;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += x[j] * x[j];
        sum = lane_sum<L>(sum);
        if (live && w) {
            const float r = 1.0f / sqrtf(sum * (1.0f / D) + a.d.eps);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= r * (w[e + j] + a.d.weight_offset);
        }
        if (half > 0) {
            if (a.d.interleaved) {
                if (live && !is_v && e < a.d.rot) {
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        const int i = (e + j) >> 1;
                        if (i < half) {
                            const float u = x[j], v = x[j + 1];
                            x[j] = u * cs[i] - v * sn[i];
                            x[j + 1] = v * cs[i] + u * sn[i];
                        }
                    }
                }
            } else {
                // the lanes of a head belong to one wavefront, whose LDS accesses are in order
#pragma unroll
                for (int j = 0; j < 8; ++j) mine[e + j] = x[j];
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                if (live && !is_v && e < a.d.rot) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int i = e + j;
                        if (i < half)
                            x[j] = x[j] * cs[i] - mine[i + half] * sn[i];
                        else if (i < a.d.rot)
                            x[j] = x[j] * cs[i - half] + mine[i - half] * sn[i - half];
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
        }
        if (!live) continue;
        if (is_q) {
            store8(a.q_out, GDN_BF16, (t * H_q + h) * int64_t(D) + e, x);
        } else if (stored) {
            const float* scale = is_v ? a.cache.v_scale : a.cache.k_scale;
            if (scale) {
                const float s = scale[h];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] /= s;
            }
            const int64_t at =
                is_v ? page * a.cache.v_page_stride + page_row * a.cache.v_row_stride + h * a.cache.v_head_stride
                     : page * a.cache.k_page_stride + page_row * a.cache.k_row_stride + h * a.cache.k_head_stride;
            char* pool = static_cast<char*>(is_v ? a.cache.v : a.cache.k);
            if (a.cache.dtype == GDN_BF16)
                store8(pool, GDN_BF16, at + e, x);
            else
                *reinterpret_cast<uint2*>(pool + at + e) = pack_e4m3(x);
        }
    }
}

// ---------------------------------------------------------------------------
// gdn_kv_commit.  One workgroup per sequence and cache: the path's nodes are
// ranked by counting bits, then every thread carries its 16-byte pieces of all
// rows down in the path's order.  A row's new place is never behind its old
// one (the j-th node of a path has index j or more), so what a thread
// overwrites it has read before, also with 8 rows in flight.  Latency bounds it:
// 12 caches take 5 us for one sequence and 6 for 32 (path of 8, 13 MB).
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kThreads) void commit_kernel(KvCommitArgs a, int page_shift) {
    __shared__ int32_t from[GDN_ATTN_MAX_N], to[GDN_ATTN_MAX_N];
    __shared__ int bad;
    const int b = blockIdx.x, c = blockIdx.y, tid = threadIdx.x;
    const int N = a.d.N, W = (N + 31) >> 5;
    const int32_t node = a.accepted[b], raw = a.length[b];
    const int64_t cap = int64_t(a.d.max_pages) << page_shift;
    const int64_t len = raw < 0 ? 0 : raw < cap ? raw : cap;
    const bool moves = node >= 0 && node < N;
    if (tid == 0) bad = raw != len;
    __syncthreads();

    const int32_t* table = a.table + b * a.d.table_stride;
    int count = 0, before = 0;
    bool on = false;
    if (moves) {
        const uint32_t* bits = a.anc + (int64_t(b) * N + node) * W;
        for (int w = 0; w < W; ++w) {
            uint32_t u = bits[w];
            if (w == W - 1 && (N & 31)) u &= (1u << (N & 31)) - 1;
            if (w < tid >> 5) before += __popc(u);
            if (w == tid >> 5) {
                before += __popc(u & ((1u << (tid & 31)) - 1));
                on = u >> (tid & 31) & 1;
            }
            count += __popc(u);
        }
    }
    if (on) {
        int32_t at[2];
        const int64_t token[2] = {len + tid, len + before};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            at[i] = -1;
            if (token[i] < cap) {
                const int32_t page = table[token[i] >> page_shift];
                if (page >= 0 && page < a.cache.n_pages)
                    at[i] = int32_t((int64_t(page) << page_shift) + (token[i] & (a.cache.page_size - 1)));
            }
        }
        if (at[0] < 0 || at[1] < 0) {
            bad = 1;  // several threads may write it
            at[0] = at[1];
        }
        from[before] = at[0];
        to[before] = at[1];
    }
    __syncthreads();
    if (tid == 0 && c == 0) {
        if (a.new_length) a.new_length[b] = int32_t(len + count);
        if (a.new_length && a.seq_status)
            a.seq_status[b] = node < -1 || node >= N ? GDN_ERR_ACCEPT : bad ? GDN_ERR_SHAPE : 0;
    }
    if (count == 0) return;

    const int size = a.cache.dtype == GDN_BF16 ? 2 : 1;
    const int pieces = a.cache.d * size / 16, per_side = a.cache.H_kv * pieces;
    // what is listed twice moves once: a path's rows that have moved are not where they were
    const int begin = a.k_moved >> c & 1 ? per_side : 0, end = a.v_moved >> c & 1 ? per_side : 2 * per_side;
    for (int i = begin + tid; i < end; i += kThreads) {
        const bool is_v = i >= per_side;
        const int at = is_v ? i - per_side : i;
        const int64_t page_stride = (is_v ? a.cache.v_page_stride : a.cache.k_page_stride) * size;
        const int64_t row_stride = (is_v ? a.cache.v_row_stride : a.cache.k_row_stride) * size;
        const int64_t head_stride = (is_v ? a.cache.v_head_stride : a.cache.k_head_stride) * size;
        char* pool = static_cast<char*>(is_v ? a.v[c] : a.k[c]) + at / pieces * head_stride + at % pieces * 16;
        auto row = [&](int32_t slot) {
            return reinterpret_cast<u32x4*>(pool + (slot >> page_shift) * page_stride +
                                            (slot & (a.cache.page_size - 1)) * row_stride);
        };
        constexpr int F = 8;
        for (int j0 = 0; j0 < count; j0 += F) {
            u32x4 x[F];
#pragma unroll
            for (int j = 0; j < F; ++j) x[j] = *row(max(from[min(j0 + j, count - 1)], 0));
#pragma unroll
            for (int j = 0; j < F; ++j)
                if (j0 + j < count && from[j0 + j] != to[j0 + j]) *row(to[j0 + j]) = x[j];
        }
    }
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t stream) {
    const int per = kThreads / (a.cache.d / 8);
    const int all = (a.d.H_q + 2 * a.cache.H_kv + per - 1) / per;
    // few tokens: a workgroup for every pass; many: the angles once per token
    const int passes = a.d.T < 1024 ? 1 : all;
    const int groups = (all + passes - 1) / passes;
    const int shift = __builtin_ctz(a.cache.page_size);
    const dim3 grid = grid_of(int64_t(a.d.T) * groups);
    switch (a.cache.d) {
        case 64: append_kernel<64><<<grid, kThreads, 0, stream>>>(a, passes, groups, shift); break;
        case 128: append_kernel<128><<<grid, kThreads, 0, stream>>>(a, passes, groups, shift); break;
        default: append_kernel<256><<<grid, kThreads, 0, stream>>>(a, passes, groups, shift); break;
    }
    return hipGetLastError();
}

hipError_t launch_kv_commit(const KvCommitArgs& a, int n_caches, hipStream_t stream) {
    commit_kernel<<<dim3(a.d.B, n_caches), kThreads, 0, stream>>>(a, __builtin_ctz(a.cache.page_size));
    return hipGetLastError();
}

}  // namespace gdn
