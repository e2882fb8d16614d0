// fw_decay_simt.cu -- decayed linear attention scans (see fw_decay.cuh) on the CUDA cores,
// parallel over chunks of 64 tokens: every type, d = 64 and 128.
//
//   scan_local    M_c = in_scale sum_j w_j b_j c_j^T of every chunk (one block each)
//   scan_prefix   the short recurrence X' = g^n X + M_c over a chain's chunks, one thread per
//                 four state elements; M_c is replaced by the state on entry to chunk c
//   scan_out      out = rd (A X_c) + (mask . decay . A B^T) C of every chunk (one block each)
//
// All sums in fp32.  A chunk of 64 keeps the 64 x 64 part a little cheaper than the d x d part
// and gives B*H*T/64 blocks, which fills the GPU from a few thousand tokens on.
#include "fw_decay_tc.cuh"

namespace fw {
namespace {

constexpr int C = 64;          // tokens per chunk
constexpr int NT = 256;        // threads per block: 16 row groups x 16 column groups
constexpr int PADP = C + 4;    // row stride of P

struct Scans {
    ScanArgs s[3];
};

template <int D> constexpr int ldt() { return D + 4; }   // row stride of a token tile

// Rows [0, nv) of a 64-row tile as fp32 (rows behind them zero), each times row_w[r].
template <int D, typename T>
__device__ __forceinline__ void load_tile(float *dst, const T *src, int nv, const float *row_w) {
    constexpr int V = 16 / sizeof(T), PR = D / V;
    for (int i = threadIdx.x; i < C * PR; i += NT) {
        const int r = i / PR, c = (i % PR) * V;
        float f[V];
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = 0.f;
        if (r < nv) {
            const uint4 u = *reinterpret_cast<const uint4 *>(src + (int64_t)r * D + c);
            const T *p = reinterpret_cast<const T *>(&u);
            const float w = row_w ? row_w[r] : 1.f;
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = to_f32(p[e]) * w;
        }
#pragma unroll
        for (int e = 0; e < V; e += 4)
            *reinterpret_cast<float4 *>(dst + r * ldt<D>() + c + e) =
                make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    }
}

struct ChunkOf {
    int64_t chain, chunk;
    int nv;            // valid rows
    bool last;         // last chunk in processing order
};

__device__ __forceinline__ ChunkOf chunk_of(const ScanArgs &s, int64_t nch) {
    ChunkOf r;
    r.chain = (int64_t)blockIdx.x / nch;
    r.chunk = (int64_t)blockIdx.x % nch;
    const int64_t n = chain_len(s.lens, r.chain, s.H, s.T);
    const int64_t left = n - r.chunk * C;
    r.nv = left < 0 ? 0 : left > C ? C : (int)left;
    r.last = s.rev ? r.chunk == 0 : (r.chunk + 1) * C >= n;
    return r;
}

template <int D, typename T>
__global__ void __launch_bounds__(NT)
scan_local(const __grid_constant__ Scans all, int64_t nch) {
    extern __shared__ float4 smem4[];
    const ScanArgs &s = all.s[blockIdx.y];
    const ChunkOf k = chunk_of(s, nch);
    if (k.nv == 0 || (k.last && !s.X_out)) return;   // no later chunk and nobody reads the end
    float *sB = reinterpret_cast<float *>(smem4), *sC = sB + C * ldt<D>(), *w = sC + C * ldt<D>();
    const float lg = s.log_decay[k.chain % s.H];
    if (threadIdx.x < C) {
        const int j = threadIdx.x;
        w[j] = s.in_scale * decay_pow(lg, (float)(s.rev ? j + 1 : max(k.nv - 1 - j, 0)));
    }
    __syncthreads();
    const int64_t base = (k.chain * s.T + k.chunk * C) * D;
    load_tile<D>(sB, static_cast<const T *>(s.b) + base, k.nv, w);
    load_tile<D>(sC, static_cast<const T *>(s.c) + base, k.nv, nullptr);
    __syncthreads();
    constexpr int R = D / 16;                        // rows and columns per thread
    const int tr = (threadIdx.x / 16) * R, tc = (threadIdx.x % 16) * 4;
    float acc[R][R] = {};
    for (int j = 0; j < k.nv; ++j) {
        float b[R], c[R];
#pragma unroll
        for (int e = 0; e < R; e += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(sB + j * ldt<D>() + tr + e);
            const float4 y = *reinterpret_cast<const float4 *>(sC + j * ldt<D>() + tc + 16 * e);
            b[e] = x.x; b[e + 1] = x.y; b[e + 2] = x.z; b[e + 3] = x.w;
            c[e] = y.x; c[e + 1] = y.y; c[e + 2] = y.z; c[e + 3] = y.w;
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < R; ++e) acc[i][e] = fmaf(b[i], c[e], acc[i][e]);
    }
    float *M = s.ws + ((int64_t)blockIdx.x * D + tr) * D + tc;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < R; e += 4)
            *reinterpret_cast<float4 *>(M + i * D + 16 * e) =
                make_float4(acc[i][e], acc[i][e + 1], acc[i][e + 2], acc[i][e + 3]);
}

template <int D>
__global__ void __launch_bounds__(128)
scan_prefix(const __grid_constant__ Scans all, int64_t nch) {
    const ScanArgs &s = all.s[blockIdx.y];
    const int64_t idx = (int64_t)blockIdx.x * 128 + threadIdx.x;   // float4 of the states
    constexpr int PER = D * D / 4;
    const int64_t chain = idx / PER;
    if (chain >= s.n_chains) return;
    const int el = (int)(idx % PER) * 4;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (s.X0) {
        const float *X0 = s.X0 + chain * D * D;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[e] = s.x0_trans ? X0[((el + e) % D) * D + (el + e) / D] : X0[el + e];
    }
    const int64_t n = chain_len(s.lens, chain, s.H, s.T);
    const int64_t used = (n + C - 1) / C;
    const float lg = s.log_decay[chain % s.H];
    const float gC = decay_pow(lg, (float)C), gT = decay_pow(lg, (float)(n - (used - 1) * C));
    float *M = s.ws + chain * nch * D * D + el;
    for (int64_t i = 0; i < used; ++i) {
        const int64_t c = s.rev ? used - 1 - i : i;
        float4 *p = reinterpret_cast<float4 *>(M + c * D * D);
        const bool tail = i + 1 == used;
        const float4 m = tail && !s.X_out ? make_float4(0.f, 0.f, 0.f, 0.f) : *p;
        *p = make_float4(x[0], x[1], x[2], x[3]);
        const float g = c == used - 1 ? gT : gC;
        x[0] = fmaf(g, x[0], m.x);
        x[1] = fmaf(g, x[1], m.y);
        x[2] = fmaf(g, x[2], m.z);
        x[3] = fmaf(g, x[3], m.w);
    }
    if (s.X_out)
        *reinterpret_cast<float4 *>(s.X_out + chain * D * D + el) = make_float4(x[0], x[1], x[2], x[3]);
}

// acc[i][e] += sum_k A[row + i][k] B[k][col + e], k < K (a multiple of 4)
template <int RC>
__device__ __forceinline__ void gemm_acc(float (&acc)[4][RC], const float *A, int lda,
                                         const float *B, int ldb, int K) {
    for (int k = 0; k < K; k += 4) {
        float a[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = *reinterpret_cast<const float4 *>(A + i * lda + k);
            a[i][0] = v.x; a[i][1] = v.y; a[i][2] = v.z; a[i][3] = v.w;
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            float b[RC];
#pragma unroll
            for (int e = 0; e < RC; e += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(B + (k + kk) * ldb + 16 * e);
                b[e] = v.x; b[e + 1] = v.y; b[e + 2] = v.z; b[e + 3] = v.w;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < RC; ++e) acc[i][e] = fmaf(a[i][kk], b[e], acc[i][e]);
        }
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(NT)
scan_out(const __grid_constant__ Scans all, int64_t nch) {
    extern __shared__ float4 smem4[];
    const ScanArgs &s = all.s[blockIdx.y];
    const ChunkOf k = chunk_of(s, nch);
    if (k.nv == 0) return;
    float *sA = reinterpret_cast<float *>(smem4), *sB = sA + C * ldt<D>(),
          *sC = sB + C * ldt<D>(), *sX = sC + C * ldt<D>(), *pw = sX + D * D;
    const float lg = s.log_decay[k.chain % s.H];
    if (threadIdx.x <= C) pw[threadIdx.x] = decay_pow(lg, (float)threadIdx.x);
    const int64_t base = (k.chain * s.T + k.chunk * C) * D;
    load_tile<D>(sA, static_cast<const T *>(s.a) + base, k.nv, nullptr);
    load_tile<D>(sB, static_cast<const T *>(s.b) + base, k.nv, nullptr);
    load_tile<D>(sC, static_cast<const T *>(s.c) + base, k.nv, nullptr);
    const float4 *X = reinterpret_cast<const float4 *>(s.ws + (int64_t)blockIdx.x * D * D);
    for (int i = threadIdx.x; i < D * D / 4; i += NT) reinterpret_cast<float4 *>(sX)[i] = X[i];
    __syncthreads();

    // P = mask . decay . A B^T: rows tr.., columns tj + 16 e
    const int tr = (threadIdx.x / 16) * 4, tj = threadIdx.x % 16;
    float p[4][4] = {};
    for (int d = 0; d < D; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = *reinterpret_cast<const float4 *>(sA + (tr + i) * ldt<D>() + d);
            b[i] = *reinterpret_cast<const float4 *>(sB + (tj + 16 * i) * ldt<D>() + d);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[i][e] = fmaf(a[i].x, b[e].x, p[i][e]);
                p[i][e] = fmaf(a[i].y, b[e].y, p[i][e]);
                p[i][e] = fmaf(a[i].z, b[e].z, p[i][e]);
                p[i][e] = fmaf(a[i].w, b[e].w, p[i][e]);
            }
    }
    __syncthreads();                       // B is read: its rows become P
    float *sP = sB;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = tr + i, j = tj + 16 * e, lag = s.rev ? j - r : r - j;
            sP[r * PADP + j] = lag >= 0 && j < k.nv ? p[i][e] * pw[lag] * s.in_scale : 0.f;
        }
    __syncthreads();

    constexpr int RC = D / 16;
    const int tc = tj * 4;                 // columns tc + 16 e .. of groups of four
    float acc[4][RC] = {};
    gemm_acc<RC>(acc, sA + tr * ldt<D>(), ldt<D>(), sX + tc, D, D);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = tr + i;
        const float rd = pw[s.rev ? max(k.nv - 1 - r, 0) : r + 1];
#pragma unroll
        for (int e = 0; e < RC; ++e) acc[i][e] *= rd;
    }
    gemm_acc<RC>(acc, sP + tr * PADP, PADP, sC + tc, ldt<D>(), C);

    T *out = static_cast<T *>(s.out) + base;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int e = 0; e < RC; ++e) acc[i][e] *= s.out_scale;
        if (s.norm.on) {                   // a row is held by 16 neighbouring lanes
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < RC; ++e) sum += acc[i][e];
#pragma unroll
            for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            const float mean = sum / D;
            float var = 0.f;
#pragma unroll
            for (int e = 0; e < RC; ++e) {
                acc[i][e] -= mean;
                var = fmaf(acc[i][e], acc[i][e], var);
            }
#pragma unroll
            for (int o = 8; o; o >>= 1) var += __shfl_xor_sync(~0u, var, o);
            const float rstd = rsqrtf(var / D + s.norm.eps);
#pragma unroll
            for (int e = 0; e < RC; ++e) {
                const int col = tc + 16 * (e & ~3) + (e & 3);
                acc[i][e] *= rstd;
                if (s.norm.weight) acc[i][e] *= s.norm.weight[col];
                if (s.norm.bias) acc[i][e] += s.norm.bias[col];
            }
        }
        if (tr + i < k.nv) {
#pragma unroll
            for (int e = 0; e < RC; ++e)
                out[(int64_t)(tr + i) * D + tc + 16 * (e & ~3) + (e & 3)] = from_f32<T>(acc[i][e]);
        }
    }
}

template <int D, typename T>
cudaError_t launch(const Scans &all, int n, cudaStream_t stream) {
    const ScanArgs &s = all.s[0];
    const int64_t nch = (s.T + C - 1) / C;
    const dim3 grid((unsigned)(s.n_chains * nch), n);
    constexpr int smem_l = (2 * C * ldt<D>() + C) * 4;
    constexpr int smem_o = (3 * C * ldt<D>() + D * D + C + 4) * 4;
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(scan_local<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  smem_l)) != cudaSuccess)
        return e;
    if ((e = cudaFuncSetAttribute(scan_out<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  smem_o)) != cudaSuccess)
        return e;
    scan_local<D, T><<<grid, NT, smem_l, stream>>>(all, nch);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int64_t quads = s.n_chains * (D * D / 4);
    scan_prefix<D><<<dim3((unsigned)((quads + 127) / 128), n), 128, 0, stream>>>(all, nch);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    scan_out<D, T><<<grid, NT, smem_o, stream>>>(all, nch);
    return cudaGetLastError();
}

}  // namespace

size_t scan_workspace(int64_t n_chains, int64_t T, int d, fw_dtype dtype) {
    if (dtype == FW_BF16) return scan_tc_workspace(n_chains, T, d);
    return (size_t)n_chains * (size_t)((T + C - 1) / C) * d * d * sizeof(float);
}

// bf16 rows run on the tensor cores, fp32 rows here.
cudaError_t launch_scans(const ScanArgs *s, int n, cudaStream_t stream) {
    if (s[0].dtype == FW_BF16) {
        for (int i = 0; i < n; ++i) {
            const cudaError_t e = launch_scan_tc(s[i], stream);
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    }
    Scans all{};
    for (int i = 0; i < n; ++i) all.s[i] = s[i];
    return s[0].d == 64 ? launch<64, float>(all, n, stream) : launch<128, float>(all, n, stream);
}

}  // namespace fw
