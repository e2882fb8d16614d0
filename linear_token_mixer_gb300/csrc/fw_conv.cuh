// fw_conv.cuh -- arguments and launchers of the short causal convolution.
#pragma once

#include "fw_decay.cuh"

namespace fw {

struct ConvArgs {
    const void *x;             // [B][H][T][d]
    const float *weight;       // [H][d][W], the last tap on the row itself
    const float *bias;         // [H][d] or NULL (zeros)
    const void *state;         // [B][H][W-1][d], the rows before the first, oldest first, or NULL (zeros)
    const int32_t *lens;       // [B] or NULL (T)
    void *y;                   // [B][H][T][d]
    void *state_out;           // [B][H][W-1][d] or NULL; may be state
    int64_t n_chains, T;
    int H, d, W;
    fw_dtype dtype;
    int silu, zero_rest;
};

struct ConvBwdArgs {
    const void *dy, *x;
    const float *weight, *bias;
    const void *state;
    const int32_t *lens;
    const void *dstate_out;    // gradient of state_out, or NULL (zero)
    void *dx;
    float *dweight, *dbias;    // [H][d][W], [H][d]; NULL: not wanted
    void *dstate;              // gradient of state, or NULL (not wanted)
    int64_t B, T;
    int H, d, W;
    fw_dtype dtype;
    int silu, zero_rest;
    float *ws;
};

struct ConvStepArgs {
    const void *x;             // [n_states][d]
    const float *weight, *bias;
    void *state;               // moved on by one row in place
    void *y;
    int64_t n_states;
    int H, d, W;
    fw_dtype dtype;
    int silu;
};

// Whether the kernels' 32-bit counts hold B H T rows of d channels, and the backward pass's grid a head's groups of them.
bool conv_fits(int64_t B, int64_t H, int64_t T, int64_t d);
bool conv_backward_fits(int64_t H, int64_t d);
size_t conv_workspace(int64_t B, int H, int64_t T, int d, int W);
cudaError_t launch_conv(const ConvArgs &a, cudaStream_t s);
cudaError_t launch_conv_backward(const ConvBwdArgs &a, cudaStream_t s);
cudaError_t launch_conv_step(const ConvStepArgs &a, cudaStream_t s);

}  // namespace fw
