// fw_decay.cuh -- declarations shared by the decayed linear attention kernels.
//
// Forward, and all three gradients, are one scan over the tokens of a chain:
//     out_i = out_scale * ( sum_j g^|i-j| (a_i . b_j) c_j  +  [read of the carried state] )
// over j <= i (forward in time) or j >= i (reverse), with the state X[b-dim][c-dim].  For one
// chunk of n valid rows (local i, j from 0, state X on entry, in time order of processing)
//     forward   out_i += g^(i+1)   X^T a_i,   X' = g^n X + in_scale sum_j g^(n-1-j) b_j c_j^T
//     reverse   out_i += g^(n-1-i) X^T a_i,   X' = g^n X + in_scale sum_j g^(j+1)   b_j c_j^T
// (the reverse scan carries the gradient with respect to the state *before* the token's
// decay, so its final X is dS0).  Only powers g^m with m >= 0 appear.  (The bf16 scans divide within a
// chunk of 128 where 128 |log g| <= 24: the rows' factor g^(i+1) is taken out of the chunk, and
// the scores by g^-(j+1).)
//     o  = scan(q, k, v; X0 = S0)                      out_scale = scale
//     dq = scan(do, v, k; X0 = S0^T)                   out_scale = scale
//     dv = reverse scan(k, q, do; X0 = dS_T)           in_scale  = scale, final X = dS0
//     dk = reverse scan(v, do, q; X0 = dS_T^T)         in_scale  = scale
#pragma once

#include <atomic>

#include "fw_internal.cuh"

namespace fw {

constexpr int kSMs = 152;   // of a GB300: the target of a grid (a workspace's size is asked for without a device)

// Let kernel k use `bytes` of dynamic shared memory: one driver call a device, not one a launch.
// `done` is the kernel's own (a bit for each device).
template <typename K> cudaError_t allow_smem(K k, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

__device__ __forceinline__ void wait_previous_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_grid_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launch k; `overlap`: its blocks may start as soon as the blocks of the grid before it have called
// let_next_grid_start(), and call wait_previous_grid() themselves.
template <typename K, typename... A>
cudaError_t launch_after(K k, dim3 grid, int threads, size_t smem, cudaStream_t stream, bool overlap, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

// Output norm fused into a scan's or a step's epilogue.
struct NormArgs {
    int on;                       // 0: rows stored as they are
    const float *weight, *bias;   // [d] or NULL
    float eps;
};

struct ScanArgs {
    const void *a, *b, *c;    // [n_chains][T][d]
    const float *log_decay;   // [H], chain % H
    const int32_t *lens;      // [B] tokens of each batch row (NULL: T), chain / H
    const float *X0;          // [n_chains][d][d] or NULL (zero)
    float *X_out;             // final state or NULL
    void *out;                // [n_chains][T][d]
    int64_t n_chains, T;
    int H, d;
    fw_dtype dtype;
    int rev;                  // reverse scan
    int x0_trans;             // X0 is stored transposed
    int zero_rest;            // write zeros to the rows of out from lens[b] on
    float in_scale, out_scale;
    NormArgs norm;
    float *ws;                // workspace of this scan
    int *err;
    long long wait_ns;
    int force_timeout;
};

struct DecayStepArgs {
    const void *q, *k, *v;
    const float *log_decay;
    float *S;
    void *o;
    int64_t n_states;
    int H, d;
    fw_dtype dtype;
    float scale;
    NormArgs norm;
};

struct LayerNormArgs {
    const void *x;
    const float *weight, *bias;
    void *y;
    float *mean, *rstd;
    int64_t rows, width;
    fw_dtype dtype;
    float eps;
};

struct LayerNormBwdArgs {
    const void *dy, *x;
    const float *weight, *mean, *rstd;
    void *dx;
    float *dweight, *dbias;
    int64_t rows, width;
    fw_dtype dtype;
    float *ws;
};

// One forward scan, or the three of a backward pass (dq, dv, dk) over chains of the same shape.
// Bytes of workspace of a call, and the launch: s[0].ws is the call's workspace, shared out there.
size_t scan_workspace(int64_t n_chains, int64_t T, int d, fw_dtype dtype, bool backward);
cudaError_t launch_scans(ScanArgs *s, int n, cudaStream_t stream);
cudaError_t launch_decay_step(const DecayStepArgs &a, cudaStream_t s);
cudaError_t launch_layer_norm(const LayerNormArgs &a, cudaStream_t s);
cudaError_t launch_layer_norm_backward(const LayerNormBwdArgs &a, cudaStream_t s);
size_t layer_norm_workspace(int64_t rows, int64_t width);

// Two fp32 operations in one instruction, on pairs.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 halves(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// g^n = exp(n log g).  The product n log g is rounded to fp32; what the rounding
// dropped is recovered by an FMA and multiplied back in, so a large exponent costs no relative
// accuracy.  g^0 = 1 for every g, g = 0 (log g = -inf) included.
__device__ __forceinline__ float decay_pow(float log_g, float n) {
    if (n == 0.f) return 1.f;
    const float x = n * log_g;
    if (x < -150.f) return 0.f;            // below the smallest subnormal
    const float e = fmaf(n, log_g, -x);
    const float p = expf(x);
    return isfinite(p) ? fmaf(p, e, p) : p;   // overflow and NaN as they are
}

// Tokens of a chain: T, or the batch row's length clamped to [0, T].
__device__ __forceinline__ int64_t chain_len(const int32_t *lens, int64_t chain, int H, int64_t T) {
    if (!lens) return T;
    const int64_t n = lens[chain / H];
    return n < 0 ? 0 : n > T ? T : n;
}

}  // namespace fw
