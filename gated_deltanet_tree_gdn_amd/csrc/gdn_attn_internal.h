// gdn_attn_internal.h -- launch interface between the C ABI of gdn_attn.h and
// its kernels, and the division of the keys over workgroups that the
// attention kernels share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "gdn_attn.h"

namespace gdn {

struct KvAppendArgs {
    gdn_kv_append_dims d;
    gdn_kv_cache cache;
    const void* q;
    const void* k;
    const void* v;
    const float* q_weight;
    const float* k_weight;
    const float* inv_freq;
    const int32_t* position;
    const int32_t* slot;
    void* q_out;
};

constexpr int kCommitCaches = 32;  // caches of one launch
struct KvCommitArgs {
    gdn_kv_commit_dims d;
    gdn_kv_cache cache;  // k and v as in the arrays
    void* k[kCommitCaches];
    void* v[kCommitCaches];
    uint32_t k_moved, v_moved;  // bits of caches whose k or v an earlier one has, too
    const uint32_t* anc;
    const int32_t* accepted;
    const int32_t* table;
    const int32_t* length;
    int32_t* new_length;  // NULL in launches after the first
    int32_t* seq_status;
};

enum AttnKind { kAttnDecode, kAttnPrefill, kAttnVerify };

struct AttnArgs {
    gdn_attn_dims d;
    gdn_kv_cache cache;
    const uint16_t* q;
    const int32_t* cu;  // prefill
    const uint32_t* anc;  // verify
    const int32_t* table;
    const int32_t* length;
    const uint16_t* gate;
    uint16_t* o;
    int32_t* seq_status;
    void* ws;
    AttnKind kind;
    int page_shift;
    // Filled by attn_shape():
    int group;       // query heads of a key head
    int tile_rows;   // (token, head of the group) rows of a workgroup
    int head_tiles;  // decode: tiles of 16 heads that the group is cut into, else 1
    int team;        // workgroups side by side: the tiles of a tree, otherwise 1
    int teams;       // that the units are divided over
    int unit_shift;  // keys of a unit, as a power of two
    int min_units;   // of a workgroup
    bool join;       // tiles may be divided
};
constexpr int kDecodeRows = 16, kTileRows = 128;  // rows of a tile
// Workgroups of 4 wavefronts that a CU's registers have room for: what a
// wavefront of the single-token kernel holds goes by the bytes of a key, and the
// fewer those are, the more wavefronts it takes to hide a step's latencies.
constexpr int decode_per_cu(int d, bool e4m3) { return d == 256 ? 1 : d == 128 ? 2 : e4m3 ? 4 : 3; }
constexpr int tiles_per_cu(int d) { return d == 256 ? 1 : 2; }
constexpr int kDecodeUnit = 128, kTilesUnit = 64;  // keys of a unit

// Fills the derived members.
void attn_shape(AttnArgs& a);
size_t attn_ws_bytes(const AttnArgs& a);
int attn_grid(const AttnArgs& a);  // workgroups of the attention kernels

// Which of `all` pieces of work, range times team plus place in the team,
// workgroup `wg` of the grid takes; -1 if none.  Workgroups go to the 8 XCDs in
// turn; each XCD has neighbouring numbers, which share keys, and as many as the
// others, so that what fits the GPU fits every XCD.  With whole teams on an XCD
// some had more than they have room for, or all of a team that is alone: 16 trees
// of 48 nodes behind 6000 tokens, 16 and 2 heads of 256, 175 us, as here 120; one
// of 256 behind 20000, 260 heads of 64 to a key head, 3030 us and 660; 8 of 128
// nodes behind 3000, 50 heads of 128, 220 us and 131.
__host__ __device__ inline int attn_number(int all, int wg) {
    const int each = all >> 3, more = all & 7, xcd = wg & 7, at = wg >> 3;
    return at < each + (xcd < more) ? xcd * each + (xcd < more ? xcd : more) + at : -1;
}

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t stream);
hipError_t launch_kv_commit(const KvCommitArgs& a, int n_caches, hipStream_t stream);
hipError_t launch_attn_decode(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attn_tiles(const AttnArgs& a, hipStream_t stream);
// What the two have in common: the parts of tiles whose keys were divided are
// joined, and seq_status is written.
hipError_t launch_attn_join(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attn_status(const AttnArgs& a, hipStream_t stream);

}  // namespace gdn
