// gdn_attn_shape.cpp -- the sizes of an attention call's division over
// workgroups and of its workspace (host only).

#include <algorithm>
#include <cstdint>

#include "gdn_attn_internal.h"

namespace gdn {

void attn_shape(AttnArgs& a) {
    constexpr int kCu = 256;
    a.page_shift = __builtin_ctz(a.cache.page_size);
    a.group = a.d.H_q / a.cache.H_kv;
    const bool one = a.kind == kAttnDecode;
    a.tile_rows = one ? kDecodeRows : kTileRows;
    a.head_tiles = one ? (a.group + kDecodeRows - 1) / kDecodeRows : 1;
    const int unit = one ? kDecodeUnit : kTilesUnit;
    a.unit_shift = __builtin_ctz(unit);
    // of tiles two or more: a part is as large as four tiles of keys, but with few keys longer ranges leave most of the
    // GPU idle (a tree of 48 nodes behind 2855 tokens: at least 2, 37 us; 3 and 4, 40; 8, 52)
    a.min_units = one ? 1 : 2;
    const int64_t cap = int64_t(a.d.max_pages) << a.page_shift, rows = int64_t(a.d.T) * a.group;
    // what the kernels' registers leave room for at once, and not more than there is work for (prompts may
    // overlap, where cu_seqlens decreases, and each may then have all rows)
    const int64_t tiles = (rows + a.tile_rows - 1) / a.tile_rows;
    auto few = [](int64_t n) { return std::min<int64_t>(n, 1 << 20); };  // enough for all workgroups; the products stay below 2^63
    const int64_t units = few(few((a.kind == kAttnPrefill ? tiles : 1) * a.d.B) * a.cache.H_kv * a.head_tiles) *
                          ((cap + unit - 1) / unit + 2);
    a.team = a.kind == kAttnVerify ? int(std::max<int64_t>(tiles, 1)) : 1;  // no tiles: seq_status only
    a.teams = int(std::max<int64_t>(
        1, std::min<int64_t>(kCu * (one ? decode_per_cu(a.cache.d, a.cache.dtype == GDN_E4M3) : tiles_per_cu(a.cache.d)) / a.team,
                             (units + a.min_units - 1) / a.min_units)));
    a.join = a.teams > 1 && cap > unit;  // otherwise a tile is one unit
}

size_t attn_ws_bytes(const AttnArgs& a) {
    return a.join ? size_t(2 * a.teams) * a.team * a.tile_rows * (a.cache.d + 2) * sizeof(float) : 0;
}

// At most 2^24 - 1: several teams are 512 workgroups or fewer, and one has a place for every 128 rows of a sequence, which
// are fewer than 2^31.
int attn_grid(const AttnArgs& a) { return a.teams * a.team; }

}  // namespace gdn
