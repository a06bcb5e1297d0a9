// attn_sizes_driver.cpp -- drives the host layer of gdn_attn.h with its own
// sizing of workgroups and workspaces and stand-ins for the kernel launchers,
// which look at what they would be launched with (built with sanitizers by
// tests/test_attn_sizes_cpu.py).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>
#include <string>
#include <utility>
#include <vector>

#include "gdn_attn_internal.h"
#include "gdn_internal.h"

extern "C" const char* hipGetErrorString(hipError_t) { return "stand-in error"; }

static std::string last_error;
static int bad, launches, joins;
static size_t given;  // bytes of the call's workspace

static void check(bool fine, const char* what, long long a = 0, long long b = 0, long long c = 0) {
    if (fine) return;
    if (++bad <= 20) std::printf("%s (%lld, %lld, %lld): '%s'\n", what, a, b, c, last_error.c_str());
}

namespace gdn {
void set_last_error(const std::string& msg) { last_error = msg; }
hipError_t launch_kv_append(const KvAppendArgs&, hipStream_t) { return hipSuccess; }
static std::vector<std::pair<void*, void*>> moved;  // what the launches move, null where they do not
hipError_t launch_kv_commit(const KvCommitArgs& a, int n, hipStream_t) {
    for (int i = 0; i < n; ++i) moved.push_back({a.k_moved >> i & 1 ? nullptr : a.k[i], a.v_moved >> i & 1 ? nullptr : a.v[i]});
    return ++launches, hipSuccess;
}
static hipError_t look(const AttnArgs& a) {
    ++launches;
    check(a.teams >= 1 && a.team >= 1 && a.min_units >= 1, "empty division", a.teams, a.team);
    check(a.join == (a.teams > 1 && (int64_t(a.d.max_pages) << a.page_shift) > int64_t(1) << a.unit_shift), "join", a.teams, a.team);
    // two parts for each workgroup of a team, each of the rows' outputs, maxima and sums
    const size_t need = a.join ? size_t(2) * a.teams * a.team * a.tile_rows * (a.cache.d + 2) * 4 : 0;
    check(need <= given, "parts outside the workspace", a.teams, a.team, (long long)given);
    const int64_t rows = int64_t(a.d.T) * a.group, tiles = (rows + a.tile_rows - 1) / a.tile_rows;
    // one dimension of a grid holds fewer than 2^32 threads; a workgroup for every place of every team
    const int64_t grid = attn_grid(a);
    check(grid * 256 < int64_t(1) << 32, "grid", grid, a.teams, a.team);
    check(grid == int64_t(a.teams) * a.team, "workgroups without a place", grid, a.team);
    check(a.team == (a.kind == kAttnVerify ? tiles : 1), "team", a.team, tiles);
    return hipSuccess;
}
hipError_t launch_attn_decode(const AttnArgs& a, hipStream_t) { return look(a); }
hipError_t launch_attn_tiles(const AttnArgs& a, hipStream_t) { return look(a); }
hipError_t launch_attn_join(const AttnArgs& a, hipStream_t) { return ++joins, check(a.join, "join of whole tiles"), hipSuccess; }
hipError_t launch_attn_status(const AttnArgs&, hipStream_t) { return hipSuccess; }
}  // namespace gdn

alignas(256) static unsigned char mem[8192];

static gdn_status verify(const gdn_attn_dims& d, const gdn_kv_cache& c, size_t bytes) {
    void *p = mem, *o = mem + 4096;
    int32_t* i = reinterpret_cast<int32_t*>(mem);
    given = bytes;
    return gdn_attn_verify(&d, &c, p, reinterpret_cast<uint32_t*>(mem), i, i, nullptr, o, nullptr, bytes ? p : nullptr, bytes, nullptr);
}

// The workspace that a tree asks for serves every smaller one.
static void smaller_trees() {
    for (int d : {64, 128, 256})
        for (int group : {1, 4, 7, 64, 130, 300})
            for (int B : {1, 100})
                for (int pages : {5, 40, 4096}) {
                    const gdn_kv_cache c{mem, mem, nullptr, nullptr, 10, 16, 2, d, GDN_BF16, 0, 32 * d, 2 * d, d, 32 * d, 2 * d, d};
                    std::vector<gdn_attn_dims> all;
                    std::vector<size_t> need;
                    for (int T = 1; T <= GDN_ATTN_MAX_N; ++T) {
                        all.push_back({B, T, 2 * group, pages, 0.1f, 0, 2 * group * d, 0, 0, pages});
                        need.push_back(gdn_attn_verify_workspace_bytes(&all.back(), &c));
                    }
                    for (size_t n = 0; n < all.size(); ++n) {
                        check(verify(all[n], c, need[n]) == GDN_OK, "own workspace", d, group, n + 1);
                        size_t least = need[n], last = need[n];
                        for (size_t m = n + 1; m < all.size(); ++m) {
                            if (need[m] == 0 || need[m] == last) continue;
                            last = need[m];
                            check(verify(all[n], c, need[m]) == GDN_OK, "workspace of a larger tree", n + 1, m + 1, group);
                            least = need[m] < least ? need[m] : least;
                        }
                        if (need[n]) {
                            check(3 * least >= 2 * need[n], "far less", d, group, n + 1);
                            check(verify(all[n], c, least - 256) == GDN_ERR_WORKSPACE, "too small", d, group, n + 1);
                            check(verify(all[n], c, 0) == GDN_ERR_WORKSPACE, "missing", d, group, n + 1);
                        }
                    }
                }
}

// The largest sizes that the checks let through.
static void largest() {
    const int most = 0x7fffffff - 255;
    for (int d : {64, 128, 256})
        for (int B : {1, 7, 4000})
            for (int T : {1, 100, 255, GDN_ATTN_MAX_N}) {
                const int heads = std::min(most / (B * T), 1 << 24);
                const gdn_kv_cache c{mem, mem, nullptr, nullptr, 10, 16, 1, d, GDN_BF16, 0, 16 * d, d, d, 16 * d, d, d};
                const gdn_attn_dims v{B, T, heads, 1 << 26, 0.1f, 0, 0, 0, 0, 0};
                const size_t need = gdn_attn_verify_workspace_bytes(&v, &c);
                check(verify(v, c, need) == GDN_OK, "largest tree", B, T, heads);
            }
    // work for every workgroup that there is room for: two parts each
    void *p = mem, *o = mem + 4096;
    int32_t* i = reinterpret_cast<int32_t*>(mem);
    for (int d : {64, 128, 256})
        for (int heads : {1, 8, 65535})
            for (int group : {1, 16, 100}) {
                if (int64_t(heads) * group > 1 << 24) continue;
                const gdn_kv_cache c{mem, mem, nullptr, nullptr, 10, 16, heads, d, GDN_BF16, 0, 16 * d, d, d, 16 * d, d, d};
                gdn_attn_dims a{65535, most / (heads * group), heads * group, 1 << 26, 0.1f, 0, 0, 0, 0, 0};
                const int wide = d == 256 ? 256 : 512, one = d == 64 ? 768 : wide;
                given = gdn_attn_prefill_workspace_bytes(&a, &c);
                check(given == size_t(2) * wide * 128 * (d + 2) * 4, "workspace of prompts", d, heads, group);
                check(gdn_attn_prefill(&a, &c, p, i, i, i, nullptr, o, nullptr, p, given, nullptr) == GDN_OK, "prompts", d, heads, group);
                a.B = std::min(65535, most / (heads * group));
                given = gdn_attn_decode_workspace_bytes(&a, &c);
                check(given == size_t(2) * one * 16 * (d + 2) * 4, "workspace of tokens", d, heads, group);
                a.T = -1;
                check(gdn_attn_decode(&a, &c, p, i, i, nullptr, o, nullptr, p, given, nullptr) == GDN_OK, "tokens", d, heads, group);
            }
}

// What a call of some sizes asks for serves calls of fewer sequences, pages and rows.
static void smaller_calls() {
    void *p = mem, *o = mem + 4096;
    int32_t* i = reinterpret_cast<int32_t*>(mem);
    const int sizes[][3] = {{1, 1, 1}, {1, 9, 7}, {2, 40, 33}, {3, 40, 128}, {17, 300, 160}, {200, 300, 200}, {200, 5000, 256}};  // B, pages, T
    for (int d : {64, 128, 256})
        for (int group : {1, 5, 64})
            for (int dtype : {int(GDN_BF16), int(GDN_E4M3)})
                for (const auto& large : sizes)
                    for (const auto& small : sizes) {
                        if (small[0] > large[0] || small[1] > large[1] || small[2] > large[2]) continue;
                        const gdn_kv_cache c{mem, mem, nullptr, nullptr, 10, 16, 2, d, dtype, 0, 32 * d, 2 * d, d, 32 * d, 2 * d, d};
                        const gdn_attn_dims a{large[0], large[2], 2 * group, large[1], 0.1f, 0, 2 * group * d, 0, 0, large[1]};
                        const gdn_attn_dims b{small[0], small[2], 2 * group, small[1], 0.1f, 0, 2 * group * d, 0, 0, small[1]};
                        given = gdn_attn_decode_workspace_bytes(&a, &c);
                        check(gdn_attn_decode(&b, &c, p, i, i, nullptr, o, nullptr, p, given, nullptr) == GDN_OK, "decode", large[0], small[0]);
                        given = gdn_attn_prefill_workspace_bytes(&a, &c);
                        check(gdn_attn_prefill(&b, &c, p, i, i, i, nullptr, o, nullptr, p, given, nullptr) == GDN_OK, "prefill", large[0], small[0]);
                        given = gdn_attn_verify_workspace_bytes(&a, &c);
                        check(given == 0 || verify(b, c, given) == GDN_OK, "verify", large[0], small[0], group);
                    }
}

// Every number has one workgroup, in grids of that many and more, and no XCD more than an eighth, rounded up.
static void numbers() {
    for (int all = 0; all < 1100; ++all)
        for (int grid : {all, all + 1, all + 13, 1100}) {
            std::vector<int> taken(all), of_xcd(8), last(8, -1);
            for (int wg = 0; wg < grid; ++wg) {
                const int w = gdn::attn_number(all, wg);
                check(w >= -1 && w < all, "number", all, grid, w);
                if (w < 0) continue;
                ++taken[w], ++of_xcd[wg % 8];
                check(last[wg % 8] < 0 || last[wg % 8] == w - 1, "neighbours", all, grid, w);
                last[wg % 8] = w;
            }
            for (int w = 0; w < all; ++w) check(taken[w] == 1, "taken", all, grid, w);
            for (int x = 0; x < 8; ++x) check(of_xcd[x] <= (all + 7) / 8, "too many", all, grid, x);
        }
    const int most = (1 << 24) - 1;
    check(gdn::attn_number(most, most - 1) >= 0 && gdn::attn_number(most, most) == -1, "largest");
    launches = 1;
}

// Of caches that are listed more than once the first moves, in all launches of a call.
static void shared() {
    unsigned char* at = mem;
    int32_t* i = reinterpret_cast<int32_t*>(mem);
    const gdn_kv_cache c{at, at + 16, nullptr, nullptr, 10, 16, 2, 64, GDN_BF16, 0, 2048, 128, 64, 2048, 128, 64};
    std::vector<gdn_kv_cache> all(100, c);
    for (int n = 0; n < 100; ++n) all[n].k = at + 16 * (n % 37), all[n].v = at + 4096 + 16 * (n % 41);
    const gdn_kv_commit_dims m{3, 20, 40, 0, 40};
    check(gdn_kv_commit(&m, all.data(), 100, reinterpret_cast<uint32_t*>(mem), i, i, i, i + 1, nullptr, nullptr) == GDN_OK, "commit");
    check(gdn::moved.size() == 100, "caches", gdn::moved.size());
    for (int n = 0; n < 100; ++n) {
        check(gdn::moved[n].first == (n < 37 ? all[n].k : nullptr), "k", n);
        check(gdn::moved[n].second == (n < 41 ? all[n].v : nullptr), "v", n);
    }
}

int main(int argc, char** argv) {
    const std::string what = argc > 1 ? argv[1] : "";
    if (what == "trees") smaller_trees();
    if (what == "calls") smaller_calls();
    if (what == "largest") largest();
    if (what == "shared") shared();
    if (what == "numbers") numbers();
    if (bad) std::printf("%d failures\n", bad);
    std::printf("%d launches, %d joins\n", launches, joins);
    return bad != 0 || launches == 0;
}
