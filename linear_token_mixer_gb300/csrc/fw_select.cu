// fw_select.cu -- selective scan: its form for one token, and the choice of the scan of a prompt.
//
//     dt_t = softplus(dt_raw_t + dt_bias),  g_t = exp(log_decay dt_t),
//     S_t = g_t S_{t-1} + dt_t k_t v_t^T,   o_t = scale S_t^T q_t + skip v_t
//
// A prompt is the chunked scan of fw_scan_tc.cuh (bf16) or fw_decay_f32.cu (fp32) with each chunk's own logs
// (chunk_logs) in place of powers of one decay.
//
// One token: one block a state, the state once through registers, as decay_step_kernel.  Bound by the state's bytes:
// B256 H32 d = 128 bf16 (1.08 GB) 157.9 us, 6.83 TB/s, 101 % of the measured copy rate.
#include "fw_select.cuh"

namespace fw {
namespace {

constexpr int kThreads = 256;

template <int D, typename T>
__global__ void __launch_bounds__(kThreads)
select_step_kernel(SelectStepArgs a) {
    constexpr int TPR = D / 4;             // threads per state row (a float4 each)
    constexpr int RPP = kThreads / TPR;    // rows per pass
    constexpr int NP = D / RPP;
    __shared__ float sq[D], sk[D], sv[D];
    __shared__ float4 part[RPP][TPR];
    const int tid = threadIdx.x, cq = tid % TPR, rg = tid / TPR;
    const int64_t st = blockIdx.x;
    const int h = (int)(st % a.H);
    float4 *S = reinterpret_cast<float4 *>(a.S + st * D * D);
    float4 x[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) x[p] = __ldcs(S + (p * RPP + rg) * TPR + cq);
    const float dt = step_of(a.gate, st, h), rate = a.gate.log_decay[h], x0 = rate * dt;
    const float g = x0 < -kReset ? 0.f : exp_two(x0, fmaf(rate, dt, -x0));
    if (tid < D) {
        const int64_t qk = group_chain(st, a.H, a.gate.G) * D + tid;
        sq[tid] = to_f32(static_cast<const T *>(a.q)[qk]) * a.scale;
        sk[tid] = to_f32(static_cast<const T *>(a.k)[qk]) * dt;
        sv[tid] = to_f32(static_cast<const T *>(a.v)[st * D + tid]);
    }
    __syncthreads();
    const float4 v = reinterpret_cast<const float4 *>(sv)[cq];
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int i = p * RPP + rg;
        const float k = sk[i], q = sq[i];
        x[p].x = fmaf(g, x[p].x, k * v.x);
        x[p].y = fmaf(g, x[p].y, k * v.y);
        x[p].z = fmaf(g, x[p].z, k * v.z);
        x[p].w = fmaf(g, x[p].w, k * v.w);
        o.x = fmaf(x[p].x, q, o.x);
        o.y = fmaf(x[p].y, q, o.y);
        o.z = fmaf(x[p].z, q, o.z);
        o.w = fmaf(x[p].w, q, o.w);
        __stcs(S + i * TPR + cq, x[p]);
    }
    part[rg][cq] = o;
    __syncthreads();
    if (tid < D) {
        float r = 0.f;
#pragma unroll
        for (int g2 = 0; g2 < RPP; ++g2) r += reinterpret_cast<const float *>(part[g2])[tid];
        if (a.gate.skip) r = fmaf(a.gate.skip[h], sv[tid], r);
        static_cast<T *>(a.o)[st * D + tid] = from_f32<T>(r);
    }
}

}  // namespace

size_t select_workspace(int64_t n_chains, int64_t T, int d, fw_dtype dtype) {
    return dtype == FW_BF16 ? select_workspace_tc(n_chains, T, d) : select_workspace_f32(n_chains, T, d);
}

cudaError_t launch_select(const SelectArgs &args, cudaStream_t stream) {
    ScanArgs s = args.scan;
    s.sel.gate = args.gate;
    return s.dtype == FW_BF16 ? launch_select_tc(s, stream) : launch_select_f32(s, stream);
}

cudaError_t launch_select_step(const SelectStepArgs &a, cudaStream_t s) {
    const unsigned grid = (unsigned)a.n_states;
    if (a.dtype == FW_F32) {
        if (a.d == 64) select_step_kernel<64, float><<<grid, kThreads, 0, s>>>(a);
        else select_step_kernel<128, float><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (a.d == 64) select_step_kernel<64, __nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
        else select_step_kernel<128, __nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace fw
