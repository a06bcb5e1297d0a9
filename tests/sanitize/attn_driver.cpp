// attn_driver.cpp -- drives the host layer of gdn_attn.h with stand-ins for
// the kernel launchers and the HIP function it uses (built with sanitizers by
// tests/test_attn_cpu.py).
#include <hip/hip_runtime.h>

#include <cstdio>
#include <string>
#include <vector>

#include "gdn_attn_internal.h"
#include "gdn_internal.h"

extern "C" const char* hipGetErrorString(hipError_t) { return "stand-in error"; }

static std::string last_error;
static int launches, joins, verdicts, committed;
static hipError_t outcome = hipSuccess;

namespace gdn {
void set_last_error(const std::string& msg) { last_error = msg; }
void attn_shape(AttnArgs& a) {
    a.join = a.d.max_pages > 8;
    a.tile_rows = 16;
}
size_t attn_ws_bytes(const AttnArgs& a) { return a.join ? 1024 : 0; }
hipError_t launch_kv_append(const KvAppendArgs&, hipStream_t) { return ++launches, outcome; }
hipError_t launch_kv_commit(const KvCommitArgs& a, int n, hipStream_t) {
    for (int i = 0; i < n; ++i) committed += a.k[i] != nullptr && a.v[i] != nullptr;
    return ++launches, outcome;
}
hipError_t launch_attn_decode(const AttnArgs&, hipStream_t) { return ++launches, outcome; }
hipError_t launch_attn_tiles(const AttnArgs&, hipStream_t) { return ++launches, outcome; }
hipError_t launch_attn_join(const AttnArgs&, hipStream_t) { return ++joins, outcome; }
hipError_t launch_attn_status(const AttnArgs&, hipStream_t) { return ++verdicts, outcome; }
}  // namespace gdn

static int bad;
static void expect(gdn_status got, gdn_status want, const char* what) {
    if (got != want || last_error.empty() != (want == GDN_OK)) {
        std::printf("%s: status %d, expected %d, detail '%s'\n", what, got, want, last_error.c_str());
        ++bad;
    }
}

int main() {
    alignas(256) static unsigned char mem[8192];
    void *p = mem, *o = mem + 4096;
    float* f = reinterpret_cast<float*>(mem);
    int32_t* i = reinterpret_cast<int32_t*>(mem);
    int32_t* j = reinterpret_cast<int32_t*>(o);
    uint32_t* u = reinterpret_cast<uint32_t*>(mem);
    gdn_kv_cache c{p, p, f, f, 10, 16, 2, 128, GDN_E4M3, 0, 4096, 256, 128, 4096, 256, 128};
    for (int k = 0; k < 2; ++k) {
        outcome = k ? hipErrorInvalidValue : hipSuccess;
        const gdn_status want = k ? GDN_ERR_HIP : GDN_OK;
        gdn_kv_append_dims a{3, 8, GDN_F32, 64, 1, 1e-6f, 0.0f, 0, 1024, 128, 256, 128, 256, 128};
        expect(gdn_kv_append(&a, &c, p, p, p, f, f, f, i, i, o, nullptr), want, "append");
        gdn_attn_dims d{3, 20, 8, 40, 0.1f, 0, 1024, 1024, 128, 40};
        expect(gdn_attn_decode(&d, &c, p, i, i, p, o, i, p, 1024, nullptr), want, "decode");
        expect(gdn_attn_prefill(&d, &c, p, i, i, i, p, o, i, p, 1024, nullptr), want, "prefill");
        expect(gdn_attn_verify(&d, &c, p, u, i, i, p, o, i, p, 1024, nullptr), want, "verify");
        expect(gdn_attn_decode(&d, &c, p, i, i, p, o, i, p, 1023, nullptr), GDN_ERR_WORKSPACE, "small workspace");
        std::vector<gdn_kv_cache> all(70, c);
        gdn_kv_commit_dims m{3, 20, 40, 0, 40};
        expect(gdn_kv_commit(&m, all.data(), 70, u, i, i, i, j, i, nullptr), want, "commit");
    }
    // a failed launch is followed by no other of its call
    if (launches != 4 + 3 + 4 + 1 || joins != 3 || verdicts != 3 || committed != 70 + 32) ++bad;
    outcome = hipSuccess;
    gdn_attn_dims none{3, 0, 8, 8, 0.1f, 0, 1024, 1024, 128, 40};  // no queries: the verdicts only
    expect(gdn_attn_prefill(&none, &c, nullptr, i, i, i, nullptr, nullptr, i, nullptr, 0, nullptr), GDN_OK, "no rows");
    if (verdicts != 4) ++bad;
    if (gdn_attn_decode_workspace_bytes(nullptr, &c) || gdn_attn_verify_workspace_bytes(&none, nullptr)) ++bad;
    if (bad) std::printf("%d failures (launches %d joins %d verdicts %d committed %d)\n", bad, launches, joins, verdicts, committed);
    return bad != 0;
}
