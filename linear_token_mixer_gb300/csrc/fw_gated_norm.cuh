// fw_gated_norm.cuh -- arguments and launchers of the gated norm.
#pragma once

#include "fw_decay.cuh"

namespace fw {

// What both passes read: x, gate, residual [rows][width]; scale, weight, bias [groups][width].
struct GatedIn {
    const void *x, *gate, *residual;          // gate, residual: or NULL
    const float *scale, *weight, *bias;       // or NULL
    int64_t rows;
    int width, groups, inner;                 // group of a row: (row / inner) % groups
    fw_dtype dtype;
    float eps;
    int rms, gate_after;
};

struct GatedArgs {
    GatedIn in;
    void *y, *total;                          // total: or NULL
    float *mean, *rstd;                       // or NULL
};

struct GatedBwdArgs {
    GatedIn in;
    const void *dy, *dtotal;                  // dtotal: or NULL (zero)
    const float *mean, *rstd;                 // mean: NULL with rms
    void *dx, *dgate, *dresidual;             // or NULL (not wanted)
    float *dweight, *dbias, *dscale;          // or NULL (not wanted)
    float *ws;                                // of the three sums, or NULL (none wanted)
};

size_t gated_norm_workspace(int64_t rows, int64_t width, int64_t groups);
cudaError_t launch_gated_norm(const GatedArgs &a, cudaStream_t s);
cudaError_t launch_gated_norm_backward(const GatedBwdArgs &a, cudaStream_t s);

}  // namespace fw
