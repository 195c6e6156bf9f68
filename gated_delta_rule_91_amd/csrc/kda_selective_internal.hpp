// kda_selective_internal.hpp -- host-side launch entry points of the short
// convolution and the selective scan.  Arguments were validated by
// kda_selective_api.hip before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

struct ShortConvArgs {
    int64_t B, T, D;
    int64_t n_seq;               // sequences: of a packed batch, or rows
    const int32_t* cu_seqlens;   // or null (uniform rows)
    int taps;
    bool silu;
    const void* x;
    const float* weight;
    const float* bias;           // or null
    const void* state_in;        // or null
    void* out;
    void* state_out;             // or null
    const void* d_out;           // or null
    const void* d_state;         // or null
    void* dx;
    float* dweight;
    float* dbias;                // with bias
    void* d_state_in;            // or null
    float* parts;                // backward: sums over the tokens of a tile
};

struct ShortConvStepArgs {
    int64_t N, D;
    int taps;
    bool silu;
    const void* x;
    const float* weight;
    const float* bias;           // or null
    void* state;
    void* out;
};

struct SelectiveArgs {
    int64_t B, T, D;
    int64_t n_seq;               // sequences: of a packed batch, or rows
    const int32_t* cu_seqlens;   // or null (uniform rows)
    int states;
    const void* x;
    const void* dt;
    const float* A;
    const void* Bm;
    const void* Cm;
    const float* skip;           // or null
    const void* z;               // or null
    const float* dt_bias;        // or null
    const float* state_in;       // or null
    void* out;
    float* state_out;            // or null
    const void* d_out;           // or null
    const float* d_state;        // or null
    void* dx;
    void* ddt;
    float* dA;
    void* dB;
    void* dC;
    float* dskip;                // with skip
    void* dz;                    // with z
    float* ddt_bias;             // with dt_bias
    float* d_state_in;           // or null
    bool keep;                   // forward: leave the states that enter every tile in ws
    char* ws;
};

// Waves that a launch of the convolution, its backward, may not pass.
bool short_conv_fits(const ShortConvArgs& a, bool bf16);
size_t short_conv_backward_workspace_bytes(const ShortConvArgs& a, bool bf16);
hipError_t launch_short_conv(bool bf16, const ShortConvArgs& a, hipStream_t s);
hipError_t launch_short_conv_backward(bool bf16, const ShortConvArgs& a, hipStream_t s);
hipError_t launch_short_conv_step(bool bf16, const ShortConvStepArgs& a, hipStream_t s);

bool selective_scan_fits(const SelectiveArgs& a);
// backward: the workspace of the training pair; else of the prefill alone
size_t selective_scan_workspace_bytes(const SelectiveArgs& a, bool backward);
hipError_t launch_selective_scan(bool bf16, const SelectiveArgs& a, hipStream_t s);
hipError_t launch_selective_scan_backward(bool bf16, const SelectiveArgs& a, hipStream_t s);
hipError_t launch_selective_scan_step(bool bf16, const SelectiveArgs& a, hipStream_t s);

}  // namespace kda
