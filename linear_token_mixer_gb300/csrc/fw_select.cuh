// fw_select.cuh -- arguments and launchers of the selective scan: the decayed scan of fw_decay.cuh
// with a step dt for each token and head, g_t = exp(log_decay dt_t), writes times dt_t.
#pragma once

#include "fw_decay.cuh"

namespace fw {

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

// The scans by type: bytes of the workspace from scan.ws on, and the launch.
size_t select_workspace_f32(int64_t n_chains, int64_t T, int d);
cudaError_t launch_select_f32(const ScanArgs &scan, cudaStream_t s);
size_t select_workspace_tc(int64_t n_chains, int64_t T, int d);
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

// A sum of fp32 values in two terms, hi + lo with |lo| at most half a unit of hi (48 bits; the GPU's 64-bit
// additions are a sixteenth as fast as these four to eight fp32 ones).
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two add(const Two &a, const Two &b) {
    const float s = a.hi + b.hi, t = s - a.hi, e = (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo), hi = s + e;
    return {hi, e - (hi - s)};
}

// A chunk's steps and log decays from its start, C / 32 tokens a lane, one after the other; by a whole warp.  The sums
// are kept in two terms, so that their differences within the chunk lose nothing to their size.
template <int C> struct ChunkLogs {
    static constexpr int PER = C / 32;
    float dt[PER];
    Two c[PER], total;
    // a token's step times its decay to the chunk's end
    __device__ __forceinline__ float weight(int e) const {
        const Two s = add(total, Two{-c[e].hi, -c[e].lo});
        return dt[e] * exp_two(s.hi, s.lo);
    }
    __device__ __forceinline__ float decay() const { return exp_two(total.hi, total.lo); }
};
template <int C>
__device__ __forceinline__ ChunkLogs<C> chunk_logs(const GateArgs &g, int64_t chain, int H, int64_t T, int64_t n, int64_t chunk) {
    constexpr int PER = C / 32;
    ChunkLogs<C> r;
    const int lane = threadIdx.x & 31, h = (int)(chain % H);
    const int64_t first = chunk * C + lane * PER;
    const float rate = g.log_decay[h];
    Two sum{0.f, 0.f};
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const bool on = first + e < n;
        r.dt[e] = on ? step_of(g, chain * T + first + e, h) : 0.f;
        const float x = on ? rate * r.dt[e] : 0.f;
        sum = add(sum, x < -kReset ? Two{-kReset, 0.f} : Two{x, on ? fmaf(rate, r.dt[e], -x) : 0.f});   // (NaN stays)
        r.c[e] = sum;
    }
    Two upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Two x{__shfl_up_sync(~0u, upto.hi, o), __shfl_up_sync(~0u, upto.lo, o)};
        if (lane >= o) upto = add(x, upto);
    }
    r.total = Two{__shfl_sync(~0u, upto.hi, 31), __shfl_sync(~0u, upto.lo, 31)};
    Two before{__shfl_up_sync(~0u, upto.hi, 1), __shfl_up_sync(~0u, upto.lo, 1)};
    if (lane == 0) before = Two{0.f, 0.f};
#pragma unroll
    for (int e = 0; e < PER; ++e) r.c[e] = add(before, r.c[e]);
    return r;
}

}  // namespace fw
