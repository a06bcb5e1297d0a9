// gdn_layer_internal.h -- launch interface between the C ABI of gdn_layer.h
// and its kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "gdn_layer.h"

namespace gdn {

struct SeqArgs {
    gdn_seq_dims d;
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const float* beta;
    const int32_t* cu;    // [B + 1] (prefill)
    const int32_t* slot;  // [B] or NULL
    const int32_t* has_state;
    float* S;
    void* o;
    int32_t* seq_status;
    void* ws;
};

struct AddNormArgs {
    gdn_add_norm_dims d;
    const void* x;
    const void* res;
    const float* w;
    const float* post;
    const float* chan;
    void* h;
    void* y;
};

struct GatedNormArgs {
    gdn_gated_norm_dims d;
    const void* o;
    const void* z;
    const float* w;
    void* y;
};

struct LinearArgs {
    gdn_linear_dims d;
    const void* x;
    const void* w;
    const float* bias;
    const void* res;
    void* y;
    void* ws;
};

// The kernel that gdn_linear runs.
enum LinearKernel { kThin, kTileAny, kTile64Two, kTile64, kTile128Two, kTile128, kTile256 };
struct LinearChoice {
    LinearKernel kernel;
    bool tail;  // with the code for ends of K (thin: for rows that are not whole 16-byte pieces)
    int cut;    // tiles of 256 x 256 in quarters
};
LinearChoice linear_choice(const gdn_linear_dims& d);

size_t prefill_ws_bytes(const gdn_seq_dims& d);
size_t linear_ws_bytes(const gdn_linear_dims& d);
hipError_t launch_prefill(const SeqArgs& a, hipStream_t stream);
// Token by token, the state in registers (any dtype).
hipError_t launch_prefill_walk(const SeqArgs& a, hipStream_t stream);
hipError_t launch_decode(const SeqArgs& a, hipStream_t stream);
hipError_t launch_add_norm(const AddNormArgs& a, hipStream_t stream);
hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t stream);
hipError_t launch_linear(const LinearArgs& a, hipStream_t stream);

}  // namespace gdn
