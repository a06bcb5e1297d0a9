// attn_sizes_driver.cpp -- drives the host layer of gdn_attn.h with its own
// sizing of workgroups and workspaces and stand-ins for the kernel launchers,
// which look at what they would be launched with (built with sanitizers by
// tests/test_attn_sizes_cpu.py).
#include <hip/hip_runtime.h>

#include <cstdio>
#include <string>
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
hipError_t launch_kv_commit(const KvCommitArgs&, int, hipStream_t) { return hipSuccess; }
static hipError_t look(const AttnArgs& a) {
    ++launches;
    check(a.teams >= 1 && a.team >= 1 && a.min_units >= 1, "empty division", a.teams, a.team);
    check(a.join == (a.teams > 1 && (int64_t(a.d.max_pages) << a.page_shift) > int64_t(1) << a.unit_shift), "join", a.teams, a.team);
    // two parts for each workgroup of a team, each of the rows' outputs, maxima and sums
    const size_t need = a.join ? size_t(2) * a.teams * a.team * a.tile_rows * (a.cache.d + 2) * 4 : 0;
    check(need <= given, "parts outside the workspace", a.teams, a.team, (long long)given);
    const int64_t rows = int64_t(a.d.T) * a.group, tiles = (rows + a.tile_rows - 1) / a.tile_rows;
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

int main() {
    smaller_trees();
    if (bad) std::printf("%d failures\n", bad);
    std::printf("%d launches, %d joins\n", launches, joins);
    return bad != 0 || launches == 0 || joins == 0;
}
