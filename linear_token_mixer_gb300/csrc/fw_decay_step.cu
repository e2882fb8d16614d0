// fw_decay_step.cu -- single-token step of decayed linear attention, one pass over the state:
//     S <- g_h S + k v^T,   o = scale * S^T q   (optionally layer-normed over the head's row).
//
// One block of 256 threads per state, the state streamed once through registers with 16-byte
// loads and stores (evict-first: a decode batch of states is larger than L2 and not reused
// within a step).  Bound by those bytes, 8 d^2 per state: B256 H32 d = 128 bf16 (1.08 GB) 157 us,
// 6.9 TB/s, the measured copy rate.  B1 H16, 16 blocks, is one block's two
// memory round trips and barriers, 5.9 us from a cold cache.
#include "fw_decay.cuh"

namespace fw {
namespace {

constexpr int kThreads = 256;

template <int D, typename T>
__global__ void __launch_bounds__(kThreads)
decay_step_kernel(DecayStepArgs a) {
    constexpr int TPR = D / 4;             // threads per state row (a float4 each)
    constexpr int RPP = kThreads / TPR;    // rows per pass
    constexpr int NP = D / RPP;
    __shared__ float sq[D], sk[D], sv[D];
    __shared__ float4 part[RPP][TPR];
    __shared__ float red[D / 32];
    const int tid = threadIdx.x, cq = tid % TPR, rg = tid / TPR;
    const int64_t st = blockIdx.x;
    float4 *S = reinterpret_cast<float4 *>(a.S + st * D * D);
    float4 x[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) x[p] = __ldcs(S + (p * RPP + rg) * TPR + cq);
    if (tid < D) {
        sq[tid] = to_f32(static_cast<const T *>(a.q)[st * D + tid]) * a.scale;
        sk[tid] = to_f32(static_cast<const T *>(a.k)[st * D + tid]);
        sv[tid] = to_f32(static_cast<const T *>(a.v)[st * D + tid]);
    }
    const float g = decay_pow(a.log_decay[st % a.H], 1.f);
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
    float r = 0.f;
    if (tid < D) {
#pragma unroll
        for (int g2 = 0; g2 < RPP; ++g2) r += reinterpret_cast<const float *>(part[g2])[tid];
    }
    if (a.norm.on) {                       // uniform over the block
        auto row_sum = [&](float z) {      // over the D threads that hold the row
            for (int s = 16; s; s >>= 1) z += __shfl_xor_sync(~0u, z, s);
            if (tid < D && (tid & 31) == 0) red[tid >> 5] = z;
            __syncthreads();
            float t = 0.f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) t += red[e];
            __syncthreads();
            return t;
        };
        const float mean = row_sum(r) / D;
        r = tid < D ? r - mean : 0.f;
        const float rstd = rsqrtf(row_sum(r * r) / D + a.norm.eps);
        r *= rstd;
        if (tid < D) {
            if (a.norm.weight) r *= a.norm.weight[tid];
            if (a.norm.bias) r += a.norm.bias[tid];
        }
    }
    if (tid < D) static_cast<T *>(a.o)[st * D + tid] = from_f32<T>(r);
}

}  // namespace

cudaError_t launch_decay_step(const DecayStepArgs &a, cudaStream_t s) {
    const unsigned grid = (unsigned)a.n_states;
    if (a.dtype == FW_F32) {
        if (a.d == 64) decay_step_kernel<64, float><<<grid, kThreads, 0, s>>>(a);
        else decay_step_kernel<128, float><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (a.d == 64) decay_step_kernel<64, __nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
        else decay_step_kernel<128, __nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace fw
