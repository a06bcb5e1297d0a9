// layer_driver.cpp -- drives the host layer of gdn_layer.h with stand-ins for
// the kernel launchers and the two HIP functions it uses (built with
// sanitizers by tests/test_layer_cpu.py).
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>
#include <string>

#include "gdn_internal.h"
#include "gdn_layer_internal.h"

extern "C" const char* hipGetErrorString(hipError_t) { return "stand-in error"; }

static std::string last_error;
static int launches;
static hipError_t outcome = hipSuccess;

namespace gdn {
void set_last_error(const std::string& msg) { last_error = msg; }
size_t prefill_ws_bytes(const gdn_seq_dims& d) { return 256 * (static_cast<size_t>(d.T) / 64 + d.B); }
size_t linear_ws_bytes(const gdn_linear_dims& d) { return d.K > 1000 ? 512 : 0; }
hipError_t launch_prefill(const SeqArgs&, hipStream_t) { return ++launches, outcome; }
hipError_t launch_decode(const SeqArgs&, hipStream_t) { return ++launches, outcome; }
hipError_t launch_add_norm(const AddNormArgs&, hipStream_t) { return ++launches, outcome; }
hipError_t launch_gated_norm(const GatedNormArgs&, hipStream_t) { return ++launches, outcome; }
hipError_t launch_linear(const LinearArgs&, hipStream_t) { return ++launches, outcome; }
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
    void* p = mem;
    float* f = reinterpret_cast<float*>(mem);
    int32_t* i = reinterpret_cast<int32_t*>(mem);
    gdn_seq_dims s{2, 100, 2, 4, 128, 64, GDN_BF16, GDN_F32, 2, 1, 1.0f, 1e-6f, 256, 256, 256};
    for (int k = 0; k < 2; ++k) {
        outcome = k ? hipErrorInvalidValue : hipSuccess;
        const gdn_status want = k ? GDN_ERR_HIP : GDN_OK;
        expect(gdn_prefill(&s, p, p, p, f, f, i, i, i, f, p, i, p, gdn_prefill_workspace_bytes(&s), nullptr), want, "prefill");
        expect(gdn_decode(&s, p, p, p, f, f, i, f, p, nullptr), want, "decode");
        gdn_add_norm_dims a{3, 100, GDN_BF16, GDN_F32, GDN_BF16, 1.0f, 1e-6f, 0.0f, 100, 100, 100, 100};
        expect(gdn_add_norm(&a, p, p, f, f, f, mem + 256, mem + 512, nullptr), want, "add_norm");
        gdn_gated_norm_dims n{3, 2, 64, GDN_F32, GDN_BF16, GDN_BF16, GDN_ACT_SILU, 1e-6f, 128, 128, 128};
        expect(gdn_gated_norm(&n, p, p, f, mem + 512, nullptr), want, "gated_norm");
        gdn_linear_dims m{3, 5, 2000, GDN_BF16, GDN_BF16, GDN_ACT_GELU, 1.0f, 2000, 2000, 5, 5};
        expect(gdn_linear(&m, p, p, f, p, p, p, 512, nullptr), want, "linear");
        expect(gdn_linear(&m, p, p, f, p, p, nullptr, 0, nullptr), GDN_ERR_WORKSPACE, "linear without workspace");
    }
    if (launches != 10) ++bad;
    s.T = 0;  // no tokens: no token pointers
    outcome = hipSuccess;
    expect(gdn_prefill(&s, nullptr, nullptr, nullptr, nullptr, nullptr, i, nullptr, nullptr, f, nullptr, nullptr, nullptr, 0,
                       nullptr), GDN_OK, "prefill of no tokens");
    expect(gdn_prefill(nullptr, p, p, p, f, f, i, i, i, f, p, i, p, 0, nullptr), GDN_ERR_NULL, "prefill without dims");
    expect(gdn_linear(nullptr, p, p, f, p, p, p, 0, nullptr), GDN_ERR_NULL, "linear without dims");
    std::printf(bad ? "FAILED\n" : "ok\n");
    return bad ? 1 : 0;
}
