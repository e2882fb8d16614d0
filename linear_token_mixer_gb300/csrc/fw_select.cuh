// fw_select.cuh -- arguments and launchers of the selective scan: the decayed scan of fw_decay.cuh
// with a step dt for each token and head, g_t = exp(log_decay dt_t), writes times dt_t.
#pragma once

#include "fw_decay.cuh"

namespace fw {

struct GateArgs {
    const void *dt;            // [n_chains][T] (a step: [n_states])
    fw_dtype dt_type;
    const float *log_decay;    // [H]
    const float *dt_bias;      // [H] or NULL
    const float *skip;         // [H] or NULL
    int softplus;
    int G;                     // groups of heads that share a and b: [B][G][T][d]
};

struct SelectArgs {
    ScanArgs scan;             // forward; in_scale 1, no norm
    GateArgs gate;
};

struct SelectStepArgs {
    const void *q, *k, *v;
    float *S;
    void *o;
    int64_t n_states;
    int H, d;
    fw_dtype dtype;
    float scale;
    GateArgs gate;
};

size_t select_workspace(int64_t n_chains, int64_t T, int d, fw_dtype dtype);
cudaError_t launch_select(const SelectArgs &a, cudaStream_t s);
cudaError_t launch_select_step(const SelectStepArgs &a, cudaStream_t s);

// The scans by type (scan.sel formed by the launch before them): tokens of a chunk, bytes of their own
// workspace (scan.ws), and the launch.
int select_chunk_f32();
size_t select_states_f32(int64_t n_chains, int64_t T, int d);
cudaError_t launch_select_f32(const ScanArgs &scan, cudaStream_t s);
int select_chunk_tc();
size_t select_states_tc(int64_t n_chains, int64_t T, int d);
cudaError_t launch_select_tc(const ScanArgs &scan, cudaStream_t s);

// A decay below e^-kReset is zero in fp32: sums of logs are kept finite by it.
constexpr float kReset = 104.f;

// The step of a token.
__device__ __forceinline__ float step_of(const GateArgs &g, int64_t at, int h) {
    float x = g.dt_type == FW_F32 ? static_cast<const float *>(g.dt)[at]
                                  : __bfloat162float(static_cast<const __nv_bfloat16 *>(g.dt)[at]);
    if (g.dt_bias) x += g.dt_bias[h];
    // log(1 + e^x) = max(x, 0) + log(1 + e^-|x|)
    return g.softplus ? fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))) : x;
}

}  // namespace fw
