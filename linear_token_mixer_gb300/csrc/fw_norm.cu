// fw_norm.cu -- layer norm over the last axis, forward and backward:
//     y  = (x - m) r w + b,   m = mean(x),  r = 1 / sqrt(mean((x - m)^2) + eps)
//     dx = r (w dy - mean(w dy) - xh mean(w dy xh)),   xh = (x - m) r
//     dw = sum_rows dy xh,   db = sum_rows dy
//
// Both passes are bound by their rows' bytes: each row is read once into registers (as loaded:
// 16 bytes a thread and vector), the statistics are taken from there (the variance from centred
// values, never as E[x^2] - E[x]^2) and the result is written.  A row is held by ROWT threads:
// a part of a warp for short rows, a warp, or a block.  Widths that are no multiple of 16 bytes
// take the same kernels with one element a load; rows that do not fit the registers of 1024
// threads take the looping kernels, which read the row again for each pass.
//
// The backward kernel's blocks stride over the rows and keep their columns' dw and db in
// registers; every block writes one partial row and a second kernel adds the partial rows in a
// fixed order, so the sums do not depend on the order in which blocks run.
#include "fw_decay.cuh"

namespace fw {
namespace {

constexpr int kBlock = 256;     // block of the part-of-a-warp forms
constexpr int kPartials = 608;  // most partial rows of dw, db (4 blocks for each of 152 SMs)

template <typename T, int VW> struct Vec;
template <typename T> struct Vec<T, 1> { T e[1]; };
template <> struct alignas(16) Vec<float, 4> { float e[4]; };
template <> struct alignas(16) Vec<__nv_bfloat16, 8> { __nv_bfloat16 e[8]; };

// Sum over the ROWT threads of a row; `red` is used by the block form only.
template <int ROWT>
__device__ __forceinline__ float row_sum(float v, float *red) {
    constexpr int W = ROWT < 32 ? ROWT : 32;
#pragma unroll
    for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if constexpr (ROWT > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < ROWT / 32; ++i) v += red[i];
        __syncthreads();
    }
    return v;
}

template <int ROWT>
__device__ __forceinline__ void row_sum2(float &u, float &v, float *red) {
    constexpr int W = ROWT < 32 ? ROWT : 32;
#pragma unroll
    for (int o = W / 2; o; o >>= 1) {
        u += __shfl_xor_sync(~0u, u, o);
        v += __shfl_xor_sync(~0u, v, o);
    }
    if constexpr (ROWT > 32) {
        if ((threadIdx.x & 31) == 0) {
            red[threadIdx.x >> 5] = u;
            red[32 + (threadIdx.x >> 5)] = v;
        }
        __syncthreads();
        u = v = 0.f;
#pragma unroll
        for (int i = 0; i < ROWT / 32; ++i) {
            u += red[i];
            v += red[32 + i];
        }
        __syncthreads();
    }
}

template <int ROWT> constexpr int block_of() { return ROWT <= 32 ? kBlock : ROWT; }

template <typename T, int VW, int ROWT, int VPT>
__global__ void __launch_bounds__(block_of<ROWT>())
ln_fwd(LayerNormArgs a) {
    __shared__ float red[32];
    constexpr int RPB = block_of<ROWT>() / ROWT;
    using V = Vec<T, VW>;
    const int lane = threadIdx.x % ROWT;
    const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / ROWT;
    const bool on = row < a.rows;
    const int W = (int)a.width, nv = W / VW;
    const V *x = reinterpret_cast<const V *>(static_cast<const T *>(a.x) + row * a.width);
    V xv[VPT];
    float sum = 0.f;
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
        const int i = p * ROWT + lane;
        if (on && i < nv) xv[p] = x[i];
        else
#pragma unroll
            for (int e = 0; e < VW; ++e) xv[p].e[e] = from_f32<T>(0.f);
#pragma unroll
        for (int e = 0; e < VW; ++e) sum += to_f32(xv[p].e[e]);
    }
    const float mean = row_sum<ROWT>(sum, red) / W;
    float var = 0.f;
#pragma unroll
    for (int p = 0; p < VPT; ++p)
        if (p * ROWT + lane < nv)
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                const float d = to_f32(xv[p].e[e]) - mean;
                var = fmaf(d, d, var);
            }
    const float rstd = rsqrtf(row_sum<ROWT>(var, red) / W + a.eps);
    if (!on) return;
    V *y = reinterpret_cast<V *>(static_cast<T *>(a.y) + row * a.width);
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
        const int i = p * ROWT + lane;
        if (i >= nv) continue;
        V yv;
#pragma unroll
        for (int e = 0; e < VW; ++e) {
            float f = (to_f32(xv[p].e[e]) - mean) * rstd;
            if (a.weight) f *= a.weight[i * VW + e];
            if (a.bias) f += a.bias[i * VW + e];
            yv.e[e] = from_f32<T>(f);
        }
        y[i] = yv;
    }
    if (lane == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

// Rows wider than the registers of a block: three passes over the row.
template <typename T>
__global__ void __launch_bounds__(1024)
ln_fwd_long(LayerNormArgs a) {
    __shared__ float red[32];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.width;
    T *y = static_cast<T *>(a.y) + row * a.width;
    float sum = 0.f;
    for (int64_t i = threadIdx.x; i < a.width; i += 1024) sum += to_f32(x[i]);
    const float mean = row_sum<1024>(sum, red) / (float)a.width;
    float var = 0.f;
    for (int64_t i = threadIdx.x; i < a.width; i += 1024) {
        const float d = to_f32(x[i]) - mean;
        var = fmaf(d, d, var);
    }
    const float rstd = rsqrtf(row_sum<1024>(var, red) / (float)a.width + a.eps);
    for (int64_t i = threadIdx.x; i < a.width; i += 1024) {
        float f = (to_f32(x[i]) - mean) * rstd;
        if (a.weight) f *= a.weight[i];
        if (a.bias) f += a.bias[i];
        y[i] = from_f32<T>(f);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

template <typename T, int VW, int ROWT, int VPT>
__global__ void __launch_bounds__(block_of<ROWT>())
ln_bwd(LayerNormBwdArgs a) {
    __shared__ float red[64];
    extern __shared__ float sacc[];        // part-of-a-warp forms: [RPB][2][width]
    constexpr int RPB = block_of<ROWT>() / ROWT;
    using V = Vec<T, VW>;
    const int lane = threadIdx.x % ROWT, sub = threadIdx.x / ROWT;
    const int W = (int)a.width, nv = W / VW;
    const bool sums = a.ws != nullptr;
    float w[VPT][VW], dw[VPT][VW], db[VPT][VW];
#pragma unroll
    for (int p = 0; p < VPT; ++p)
#pragma unroll
        for (int e = 0; e < VW; ++e) {
            const int c = (p * ROWT + lane) * VW + e;
            w[p][e] = a.weight && c < W ? a.weight[c] : 1.f;
            dw[p][e] = db[p][e] = 0.f;
        }
    const int64_t stride = (int64_t)gridDim.x * RPB;
    // every thread of the block makes the same number of turns (the row sums synchronise)
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += stride) {
        const int64_t row = r0 + sub;
        const bool on = row < a.rows;
        const V *x = reinterpret_cast<const V *>(static_cast<const T *>(a.x) + row * a.width);
        const V *dy = reinterpret_cast<const V *>(static_cast<const T *>(a.dy) + row * a.width);
        V xv[VPT], gv[VPT];
#pragma unroll
        for (int p = 0; p < VPT; ++p) {
            const int i = p * ROWT + lane;
            if (on && i < nv) {
                xv[p] = x[i];
                gv[p] = dy[i];
            }
        }
        const float mean = on ? a.mean[row] : 0.f, rstd = on ? a.rstd[row] : 0.f;
        float c1 = 0.f, c2 = 0.f;
#pragma unroll
        for (int p = 0; p < VPT; ++p)
            if (on && p * ROWT + lane < nv)
#pragma unroll
                for (int e = 0; e < VW; ++e) {
                    const float g = to_f32(gv[p].e[e]);
                    const float xh = (to_f32(xv[p].e[e]) - mean) * rstd;
                    dw[p][e] = fmaf(g, xh, dw[p][e]);
                    db[p][e] += g;
                    c1 = fmaf(g, w[p][e], c1);
                    c2 = fmaf(g * w[p][e], xh, c2);
                }
        row_sum2<ROWT>(c1, c2, red);
        c1 /= W;
        c2 /= W;
        V *dx = reinterpret_cast<V *>(static_cast<T *>(a.dx) + row * a.width);
#pragma unroll
        for (int p = 0; p < VPT; ++p) {
            const int i = p * ROWT + lane;
            if (!on || i >= nv) continue;
            V o;
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                const float xh = (to_f32(xv[p].e[e]) - mean) * rstd;
                o.e[e] = from_f32<T>(rstd * (to_f32(gv[p].e[e]) * w[p][e] - c1 - xh * c2));
            }
            dx[i] = o;
        }
    }
    if (!sums) return;
    float *part = a.ws + (int64_t)blockIdx.x * 2 * W;
    if constexpr (RPB == 1) {
#pragma unroll
        for (int p = 0; p < VPT; ++p)
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                const int c = (p * ROWT + lane) * VW + e;
                if (c < W) {
                    part[c] = dw[p][e];
                    part[W + c] = db[p][e];
                }
            }
    } else {
#pragma unroll
        for (int p = 0; p < VPT; ++p)
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                const int c = (p * ROWT + lane) * VW + e;
                if (c < W) {
                    sacc[sub * 2 * W + c] = dw[p][e];
                    sacc[sub * 2 * W + W + c] = db[p][e];
                }
            }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * W; c += kBlock) {
            float s = 0.f;
#pragma unroll 4
            for (int i = 0; i < RPB; ++i) s += sacc[i * 2 * W + c];
            part[c] = s;
        }
    }
}

// Rows wider than the registers of a block: dx by passes over the row (no sums) ...
template <typename T>
__global__ void __launch_bounds__(1024)
ln_bwd_long(LayerNormBwdArgs a) {
    __shared__ float red[64];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.width;
    const T *dy = static_cast<const T *>(a.dy) + row * a.width;
    T *dx = static_cast<T *>(a.dx) + row * a.width;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float c1 = 0.f, c2 = 0.f;
    for (int64_t i = threadIdx.x; i < a.width; i += 1024) {
        const float g = to_f32(dy[i]) * (a.weight ? a.weight[i] : 1.f);
        c1 += g;
        c2 = fmaf(g, (to_f32(x[i]) - mean) * rstd, c2);
    }
    row_sum2<1024>(c1, c2, red);
    c1 /= (float)a.width;
    c2 /= (float)a.width;
    for (int64_t i = threadIdx.x; i < a.width; i += 1024) {
        const float g = to_f32(dy[i]) * (a.weight ? a.weight[i] : 1.f);
        dx[i] = from_f32<T>(rstd * (g - c1 - (to_f32(x[i]) - mean) * rstd * c2));
    }
}

// ... and their column sums, one thread a column and block row, before dx is written.
template <typename T>
__global__ void __launch_bounds__(kBlock)
ln_bwd_sums_long(LayerNormBwdArgs a) {
    const int64_t c = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    if (c >= a.width) return;
    float dw = 0.f, db = 0.f;
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float g = to_f32(static_cast<const T *>(a.dy)[r * a.width + c]);
        dw = fmaf(g, (to_f32(static_cast<const T *>(a.x)[r * a.width + c]) - a.mean[r]) * a.rstd[r], dw);
        db += g;
    }
    a.ws[(int64_t)blockIdx.y * 2 * a.width + c] = dw;
    a.ws[(int64_t)blockIdx.y * 2 * a.width + a.width + c] = db;
}

// dw, db = the sum of the partial rows: 32 columns a block, 32 threads a column.
__global__ void __launch_bounds__(1024)
ln_sum_partials(const float *ws, int n, int64_t W, float *dw, float *db) {
    __shared__ float s[32][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x % 32;   // column of [2][W]
    const int y = threadIdx.x / 32;
    float v = 0.f;
    if (c < 2 * W)
        for (int i = y; i < n; i += 32) v += ws[i * 2 * W + c];
    s[y][threadIdx.x % 32] = v;
    __syncthreads();
    v = s[threadIdx.x % 32][y];            // transposed: one warp a column
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    const int64_t cc = (int64_t)blockIdx.x * 32 + y;
    if (threadIdx.x % 32 == 0 && cc < 2 * W) {
        float *dst = cc < W ? dw : db;
        if (dst) dst[cc < W ? cc : cc - W] = v;
    }
}

template <typename T> constexpr int vec_of() { return 16 / (int)sizeof(T); }

template <typename T, int VW, int ROWT, int VPT>
cudaError_t fwd(const LayerNormArgs &a, cudaStream_t s) {
    constexpr int RPB = block_of<ROWT>() / ROWT;
    ln_fwd<T, VW, ROWT, VPT><<<(unsigned)((a.rows + RPB - 1) / RPB), block_of<ROWT>(), 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t forward(const LayerNormArgs &a, cudaStream_t s) {
    constexpr int VW = vec_of<T>();
    const int64_t w = a.width;
    if (w % VW == 0) {
        const int64_t nv = w / VW;
        if (nv <= 4) return fwd<T, VW, 4, 1>(a, s);
        if (nv <= 8) return fwd<T, VW, 8, 1>(a, s);
        if (nv <= 16) return fwd<T, VW, 16, 1>(a, s);
        if (nv <= 32) return fwd<T, VW, 32, 1>(a, s);
        if (nv <= 64) return fwd<T, VW, 32, 2>(a, s);
        if (nv <= 128) return fwd<T, VW, 32, 4>(a, s);
        if (nv <= 256) return fwd<T, VW, 128, 2>(a, s);
        if (nv <= 512) return fwd<T, VW, 256, 2>(a, s);
        if (nv <= 1024) return fwd<T, VW, 256, 4>(a, s);
        if (nv <= 4096) return fwd<T, VW, 1024, 4>(a, s);
    } else {
        if (w <= 32) return fwd<T, 1, 32, 1>(a, s);
        if (w <= 128) return fwd<T, 1, 32, 4>(a, s);
        if (w <= 512) return fwd<T, 1, 32, 16>(a, s);
        if (w <= 2048) return fwd<T, 1, 128, 16>(a, s);
        if (w <= 4096) return fwd<T, 1, 256, 16>(a, s);
        if (w <= 16384) return fwd<T, 1, 1024, 16>(a, s);
    }
    ln_fwd_long<T><<<(unsigned)a.rows, 1024, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t add_partials(const LayerNormBwdArgs &a, int64_t n, cudaStream_t s) {
    if (!a.ws) return cudaSuccess;
    ln_sum_partials<<<(unsigned)((2 * a.width + 31) / 32), 1024, 0, s>>>(a.ws, (int)n, a.width,
                                                                       a.dweight, a.dbias);
    return cudaGetLastError();
}

int64_t partials(int64_t rows) { return rows < kPartials ? rows : kPartials; }

template <typename T, int VW, int ROWT, int VPT>
cudaError_t bwd(const LayerNormBwdArgs &a, cudaStream_t s) {
    constexpr int RPB = block_of<ROWT>() / ROWT;
    const int64_t blocks = (a.rows + RPB - 1) / RPB;
    const int64_t n = blocks < partials(a.rows) ? blocks : partials(a.rows);
    const size_t smem = RPB > 1 ? (size_t)RPB * 2 * a.width * sizeof(float) : 0;
    cudaError_t e;
    if (smem > 48 * 1024 &&
        (e = cudaFuncSetAttribute(ln_bwd<T, VW, ROWT, VPT>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
        return e;
    ln_bwd<T, VW, ROWT, VPT><<<(unsigned)n, block_of<ROWT>(), smem, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return add_partials(a, n, s);
}

template <typename T>
cudaError_t backward(const LayerNormBwdArgs &a, cudaStream_t s) {
    constexpr int VW = vec_of<T>();
    const int64_t w = a.width;
    if (w % VW == 0) {
        const int64_t nv = w / VW;
        if (nv <= 4) return bwd<T, VW, 4, 1>(a, s);
        if (nv <= 8) return bwd<T, VW, 8, 1>(a, s);
        if (nv <= 16) return bwd<T, VW, 16, 1>(a, s);
        if (nv <= 32) return bwd<T, VW, 32, 1>(a, s);
        if (nv <= 64) return bwd<T, VW, 32, 2>(a, s);
        if (nv <= 128) return bwd<T, VW, 128, 1>(a, s);
        if (nv <= 256) return bwd<T, VW, 256, 1>(a, s);
        if (nv <= 512) return bwd<T, VW, 256, 2>(a, s);
        if (nv <= 1024) return bwd<T, VW, 512, 2>(a, s);
        if (nv <= 2048) return bwd<T, VW, 1024, 2>(a, s);
    } else {
        if (w <= 32) return bwd<T, 1, 32, 1>(a, s);
        if (w <= 128) return bwd<T, 1, 32, 4>(a, s);
        if (w <= 1024) return bwd<T, 1, 128, 8>(a, s);
        if (w <= 2048) return bwd<T, 1, 256, 8>(a, s);
        if (w <= 4096) return bwd<T, 1, 512, 8>(a, s);
        if (w <= 8192) return bwd<T, 1, 1024, 8>(a, s);
    }
    cudaError_t e;
    if (a.ws) {
        const int64_t bx = (w + kBlock - 1) / kBlock;
        int64_t by = kPartials / bx;
        by = by < 1 ? 1 : by > partials(a.rows) ? partials(a.rows) : by;
        ln_bwd_sums_long<T><<<dim3((unsigned)bx, (unsigned)by), kBlock, 0, s>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if ((e = add_partials(a, by, s)) != cudaSuccess) return e;
    }
    ln_bwd_long<T><<<(unsigned)a.rows, 1024, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t layer_norm_workspace(int64_t rows, int64_t width) {
    return (size_t)partials(rows) * 2 * (size_t)width * sizeof(float);
}

cudaError_t launch_layer_norm(const LayerNormArgs &a, cudaStream_t s) {
    return a.dtype == FW_F32 ? forward<float>(a, s) : forward<__nv_bfloat16>(a, s);
}

cudaError_t launch_layer_norm_backward(const LayerNormBwdArgs &a, cudaStream_t s) {
    return a.dtype == FW_F32 ? backward<float>(a, s) : backward<__nv_bfloat16>(a, s);
}

}  // namespace fw
