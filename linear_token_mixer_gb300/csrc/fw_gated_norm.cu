// fw_gated_norm.cu -- the norm before a block with its scaled residual sum, and the norm behind a
// mixer with its gate, one kernel for both:
//     u = x + scale residual,   z = gate,   silu(z) = z / (1 + exp(-z))
//     gate before:  s = u silu(z),  y = norm(s) weight + bias
//     gate after:   s = u,          y = (norm(s) weight + bias) silu(z)
//     norm(s) = (s - m) r,   m = mean(s) (rms: 0),   r = 1 / sqrt(mean((s - m)^2) + eps)
// and backwards, with n = norm(s), g = dy weight (gate after: times silu(z)):
//     ds = r (g - mean(g) [rms: 0] - n mean(g n)),   du = ds silu(z) or ds, plus dtotal
//     dx = du,  dresidual = scale du,  dgate = silu'(z) (ds u, or dy (n weight + bias))
//     dweight = sum dy n (gate after: silu(z)),  dbias = sum dy (..),  dscale = sum du residual
//
// Both are bound by their rows' bytes: a row is read once, 16 bytes a thread and vector, and held in
// registers by R threads (a part of a warp, or a block) from its sums to its result; the mean is taken
// first and the squares about it (never E[s^2] - E[s]^2).  Blocks stride over the rows of one group, so that
// a thread keeps its columns' weights and, in the backward pass, its sums: in registers where a row
// takes few vectors a thread, else in shared memory, where each thread has its own columns.  A
// block writes one partial row of sums and a second kernel adds them in a fixed order.
#include "fw_gated_norm.cuh"

namespace fw {
namespace {

template <typename T, int V> struct Raw;
template <> struct Raw<float, 1> { float v; };
template <> struct Raw<float, 4> { float4 v; };
template <> struct Raw<__nv_bfloat16, 1> { __nv_bfloat16 v; };
template <> struct Raw<__nv_bfloat16, 2> { uint32_t v; };
template <> struct Raw<__nv_bfloat16, 8> { uint4 v; };

__device__ __forceinline__ void unpack(uint32_t x, float &a, float &b) {
    a = __uint_as_float(x << 16);
    b = __uint_as_float(x & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ void widen(const Raw<float, 1> &r, float (&x)[1]) { x[0] = r.v; }
__device__ __forceinline__ void widen(const Raw<float, 4> &r, float (&x)[4]) {
    x[0] = r.v.x; x[1] = r.v.y; x[2] = r.v.z; x[3] = r.v.w;
}
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16, 1> &r, float (&x)[1]) { x[0] = __bfloat162float(r.v); }
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16, 2> &r, float (&x)[2]) { unpack(r.v, x[0], x[1]); }
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16, 8> &r, float (&x)[8]) {
    unpack(r.v.x, x[0], x[1]); unpack(r.v.y, x[2], x[3]); unpack(r.v.z, x[4], x[5]); unpack(r.v.w, x[6], x[7]);
}
__device__ __forceinline__ void narrow(Raw<float, 1> &r, const float (&x)[1]) { r.v = x[0]; }
__device__ __forceinline__ void narrow(Raw<float, 4> &r, const float (&x)[4]) { r.v = make_float4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void narrow(Raw<__nv_bfloat16, 1> &r, const float (&x)[1]) { r.v = __float2bfloat16_rn(x[0]); }
__device__ __forceinline__ void narrow(Raw<__nv_bfloat16, 2> &r, const float (&x)[2]) { r.v = pack(x[0], x[1]); }
__device__ __forceinline__ void narrow(Raw<__nv_bfloat16, 8> &r, const float (&x)[8]) {
    r.v = make_uint4(pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]), pack(x[6], x[7]));
}
template <typename T, int V> __device__ __forceinline__ Raw<T, V> load(const void *p, int64_t at) {
    return *reinterpret_cast<const Raw<T, V> *>(static_cast<const T *>(p) + at);
}
template <typename T, int V> __device__ __forceinline__ void store(void *p, int64_t at, const float (&x)[V]) {
    Raw<T, V> r;
    narrow(r, x);
    *reinterpret_cast<Raw<T, V> *>(static_cast<T *>(p) + at) = r;
}
// V floats of a parameter; `other` where it is not given.
template <int V> __device__ __forceinline__ void param(const float *p, int64_t at, float other, float (&x)[V]) {
    if (!p) {
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = other;
    } else if constexpr (V % 4 == 0) {
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            const float4 q = __ldg(reinterpret_cast<const float4 *>(p + at + e));
            x[e] = q.x; x[e + 1] = q.y; x[e + 2] = q.z; x[e + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = __ldg(p + at + e);
    }
}

// 1 / (1 + exp(-z)): for bf16 rows by the fast exponential (a few ulp of fp32, a thousandth of their rounding).
template <typename T> __device__ __forceinline__ float sigmoid(float z) {
    if constexpr (sizeof(T) == 4) return 1.f / (1.f + expf(-z));
    else return __frcp_rn(1.f + __expf(-z));
}

// The sums of N values over the R threads that hold a row, in every one of them.
template <int R, int N> __device__ __forceinline__ void row_sums(float (&z)[N], float *red) {
    constexpr int W = R < 32 ? R : 32;
#pragma unroll
    for (int o = W / 2; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] += __shfl_xor_sync(~0u, z[i], o);
    if constexpr (R > 32) {
        constexpr int NW = R / 32;
        const int warp = threadIdx.x >> 5;
        __syncthreads();                       // the sums before are read
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[i * NW + warp] = z[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            z[i] = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) z[i] += red[i * NW + w];
        }
    }
}

template <int R> constexpr int block_of() { return R <= 32 ? 256 : R; }

__device__ __forceinline__ int64_t row_of(const GatedIn &in, uint32_t group, uint32_t m) {
    if (in.groups == 1) return m;
    return ((int64_t)(m / (uint32_t)in.inner) * in.groups + group) * in.inner + m % (uint32_t)in.inner;
}

// blockIdx.y: the group; blockIdx.x: a share of its rows.
template <typename T, int V, int R, int K>
__global__ void __launch_bounds__(block_of<R>()) gated_kernel(GatedArgs a, uint32_t group_rows) {
    constexpr int RPB = block_of<R>() / R;
    __shared__ float red[R > 32 ? R / 32 : 1];
    const GatedIn &in = a.in;
    const int lane = threadIdx.x % R;
    const float inv = 1.f / (float)in.width;
    const int64_t pat = (int64_t)blockIdx.y * in.width;
    for (uint32_t m0 = blockIdx.x * RPB; m0 < group_rows; m0 += gridDim.x * RPB) {
        const uint32_t m = m0 + threadIdx.x / R;
        const bool live = m < group_rows;
        const int64_t at = row_of(in, blockIdx.y, live ? m : m0) * in.width;
        Raw<T, V> rx[K], rz[K], rr[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * R + lane) * V;
            if (c < in.width) {
                rx[k] = load<T, V>(in.x, at + c);
                if (in.residual) rr[k] = load<T, V>(in.residual, at + c);
                if (in.gate) rz[k] = load<T, V>(in.gate, at + c);
            }
        }
        float s[K][V], sum[1] = {0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * R + lane) * V;
            if (c < in.width) {
                widen(rx[k], s[k]);
                if (in.residual) {
                    float f[V], r[V];
                    param<V>(in.scale, pat + c, 1.f, f);
                    widen(rr[k], r);
#pragma unroll
                    for (int e = 0; e < V; ++e) s[k][e] = fmaf(f[e], r[e], s[k][e]);
                }
                if (a.total && live) store<T, V>(a.total, at + c, s[k]);
                if (in.gate && !in.gate_after) {
                    float z[V];
                    widen(rz[k], z);
#pragma unroll
                    for (int e = 0; e < V; ++e) s[k][e] *= z[e] * sigmoid<T>(z[e]);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) sum[0] += s[k][e];
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) s[k][e] = 0.f;
            }
        }
        float mean = 0.f;
        if (!in.rms) {
            row_sums<R>(sum, red);
            mean = sum[0] * inv;
        }
        sum[0] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if ((k * R + lane) * V < in.width)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    s[k][e] -= mean;
                    sum[0] = fmaf(s[k][e], s[k][e], sum[0]);
                }
        row_sums<R>(sum, red);
        const float rstd = rsqrtf(fmaf(sum[0], inv, in.eps));
        if (!live) continue;                   // (a row of a whole block is always live)
        if (lane == 0) {
            const int64_t row = row_of(in, blockIdx.y, m);
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * R + lane) * V;
            if (c >= in.width) continue;
            float w[V], b[V];
            param<V>(in.weight, pat + c, 1.f, w);
            param<V>(in.bias, pat + c, 0.f, b);
#pragma unroll
            for (int e = 0; e < V; ++e) s[k][e] = fmaf(s[k][e] * rstd, w[e], b[e]);
            if (in.gate && in.gate_after) {
                float z[V];
                widen(rz[k], z);
#pragma unroll
                for (int e = 0; e < V; ++e) s[k][e] *= z[e] * sigmoid<T>(z[e]);
            }
            store<T, V>(a.y, at + c, s[k]);
        }
    }
}

// Sums of a thread's columns over its rows: SM, in shared memory.
template <int K, int V, bool SM> struct Sums {
    float r[SM ? 1 : K][SM ? 1 : V];
    __device__ __forceinline__ void clear(float *) {
        if constexpr (!SM)
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) r[k][e] = 0.f;
    }
    __device__ __forceinline__ void add(float *sm, int k, int c, const float (&x)[V]) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if constexpr (SM) sm[c + e] += x[e];
            else r[k][e] += x[e];
        }
    }
};

template <typename T, int V, int R, int K, bool SM>
__global__ void __launch_bounds__(block_of<R>()) gated_bwd_kernel(GatedBwdArgs a, uint32_t group_rows) {
    constexpr int BLOCK = block_of<R>(), RPB = BLOCK / R;
    static_assert(!SM || RPB == 1, "shared sums need columns that one thread owns");
    extern __shared__ float sm[];              // SM: three rows of sums; else the parts of a block
    __shared__ float red[R > 32 ? 2 * R / 32 : 1];
    const GatedIn &in = a.in;
    const int lane = threadIdx.x % R, width = in.width;
    const float inv = 1.f / (float)width;
    const int64_t pat = (int64_t)blockIdx.y * width;
    Sums<K, V, SM> dw, db, dsc;
    dw.clear(sm);
    db.clear(sm);
    dsc.clear(sm);
    if constexpr (SM) {
        if (a.ws)
            for (int i = threadIdx.x; i < 3 * width; i += BLOCK) sm[i] = 0.f;
        __syncthreads();
    }
    for (uint32_t m0 = blockIdx.x * RPB; m0 < group_rows; m0 += gridDim.x * RPB) {
        const uint32_t m = m0 + threadIdx.x / R;
        const bool live = m < group_rows;
        const int64_t row = row_of(in, blockIdx.y, live ? m : m0), at = row * width;
        Raw<T, V> rx[K], ry[K], rz[K], rr[K], rt[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * R + lane) * V;
            if (c < width) {
                rx[k] = load<T, V>(in.x, at + c);
                ry[k] = load<T, V>(a.dy, at + c);
                if (in.residual) rr[k] = load<T, V>(in.residual, at + c);
                if (in.gate) rz[k] = load<T, V>(in.gate, at + c);
                if (a.dtotal) rt[k] = load<T, V>(a.dtotal, at + c);
            }
        }
        const float mean = in.rms ? 0.f : a.mean[row], rstd = a.rstd[row];
        // n = norm(s) and g of 8 (or 4, 2, 1) columns, u = x + scale residual before them
        auto form = [&](int k, int c, float (&n)[V], float (&g)[V], float (&u)[V], float (&dy)[V]) {
            widen(rx[k], u);
            if (in.residual) {
                float f[V], r[V];
                param<V>(in.scale, pat + c, 1.f, f);
                widen(rr[k], r);
#pragma unroll
                for (int e = 0; e < V; ++e) u[e] = fmaf(f[e], r[e], u[e]);
            }
            widen(ry[k], dy);
            float w[V];
            param<V>(in.weight, pat + c, 1.f, w);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                n[e] = u[e];
                g[e] = dy[e] * w[e];
            }
            if (in.gate) {
                float z[V];
                widen(rz[k], z);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float sl = z[e] * sigmoid<T>(z[e]);
                    if (in.gate_after) g[e] *= sl;
                    else n[e] *= sl;
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) n[e] = (n[e] - mean) * rstd;
        };
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * R + lane) * V;
            if (c < width) {
                float n[V], g[V], u[V], dy[V];
                form(k, c, n, g, u, dy);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    sum[0] += g[e];
                    sum[1] = fmaf(g[e], n[e], sum[1]);
                }
            }
        }
        row_sums<R>(sum, red);
        const float mg = in.rms ? 0.f : sum[0] * inv, mgn = sum[1] * inv;
        if (!live) continue;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * R + lane) * V;
            if (c >= width) continue;
            float n[V], g[V], u[V], dy[V], d[V];
            form(k, c, n, g, u, dy);
#pragma unroll
            for (int e = 0; e < V; ++e) d[e] = rstd * (g[e] - mg - n[e] * mgn);
            if (in.gate) {
                float z[V], dz[V], b[V], w[V];
                widen(rz[k], z);
                if (in.gate_after) {
                    param<V>(in.weight, pat + c, 1.f, w);
                    param<V>(in.bias, pat + c, 0.f, b);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float sg = sigmoid<T>(z[e]), slope = sg * fmaf(z[e], 1.f - sg, 1.f);
                    if (in.gate_after) {
                        dz[e] = dy[e] * fmaf(n[e], w[e], b[e]) * slope;
                        dy[e] *= z[e] * sg;    // of the norm's output
                    } else {
                        dz[e] = d[e] * u[e] * slope;
                        d[e] *= z[e] * sg;
                    }
                }
                if (a.dgate) store<T, V>(a.dgate, at + c, dz);
            }
            if (a.dtotal) {
                float t[V];
                widen(rt[k], t);
#pragma unroll
                for (int e = 0; e < V; ++e) d[e] += t[e];
            }
            if (a.dx) store<T, V>(a.dx, at + c, d);
            if (a.ws) {
                float p[V];
#pragma unroll
                for (int e = 0; e < V; ++e) p[e] = dy[e] * n[e];
                if (a.dweight) dw.add(sm, k, c, p);
                if (a.dbias) db.add(sm + width, k, c, dy);
            }
            if (in.residual) {
                float f[V], r[V];
                param<V>(in.scale, pat + c, 1.f, f);
                widen(rr[k], r);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    r[e] *= d[e];
                    f[e] *= d[e];
                }
                if (a.dresidual) store<T, V>(a.dresidual, at + c, f);
                if (a.ws && a.dscale) dsc.add(sm + 2 * width, k, c, r);
            }
        }
    }
    if (!a.ws) return;
    // [block of the group][group][3][width]
    float *const out = a.ws + ((int64_t)blockIdx.x * in.groups + blockIdx.y) * 3 * width;
    if constexpr (SM) {
        __syncthreads();
        for (int i = threadIdx.x; i < 3 * width; i += BLOCK) out[i] = sm[i];
    } else {
#pragma unroll
        for (int which = 0; which < 3; ++which) {
            const float *given = which == 0 ? a.dweight : which == 1 ? a.dbias : a.dscale;
            if (!given) continue;              // (uniform)
            const auto &acc = which == 0 ? dw : which == 1 ? db : dsc;
            if constexpr (RPB == 1) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int c = (k * R + lane) * V;
                    if (c < width)
#pragma unroll
                        for (int e = 0; e < V; ++e) out[which * width + c + e] = acc.r[k][e];
                }
            } else {                           // the rows that a block holds at once, one after the other
                __syncthreads();
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int c = (k * R + lane) * V;
                    if (c < width)
#pragma unroll
                        for (int e = 0; e < V; ++e) sm[(threadIdx.x / R) * width + c + e] = acc.r[k][e];
                }
                __syncthreads();
                for (int c = threadIdx.x; c < width; c += BLOCK) {
                    float z = 0.f;
#pragma unroll 4
                    for (int p = 0; p < RPB; ++p) z += sm[p * width + c];
                    out[which * width + c] = z;
                }
            }
        }
    }
}

// Sums of the blocks in their order, one column of one of the three a thread.
constexpr int kSumBlock = 128;
__global__ void __launch_bounds__(kSumBlock)
gated_sum_kernel(const float *ws, int slices, int64_t count, int width, float *dweight, float *dbias, float *dscale) {
    wait_previous_grid();
    const int64_t i = (int64_t)blockIdx.x * kSumBlock + threadIdx.x;   // of [groups][3][width]
    if (i >= count) return;
    const int64_t group = i / (3 * width);
    const int which = (int)(i / width % 3), c = (int)(i % width);
    float *const out = which == 0 ? dweight : which == 1 ? dbias : dscale;
    if (!out) return;
    float z = 0.f;
#pragma unroll 8
    for (int s = 0; s < slices; ++s) z += ws[s * count + i];
    out[group * width + c] = z;
}

// Blocks that share the rows of a group.
uint32_t slices_of(int64_t group_rows, int64_t groups, int rows_a_block, int blocks_an_sm) {
    const int64_t most = (group_rows + rows_a_block - 1) / rows_a_block;
    int64_t s = (int64_t)kSMs * blocks_an_sm / groups;
    return (uint32_t)(s < 1 ? 1 : s > most ? most : s);
}
// Blocks an SM: of up to 2048 threads (forward), up to 1024 (backward, whose partial rows are bounded by it).
template <int R> uint32_t forward_slices(const GatedIn &in) {
    return slices_of(in.rows / in.groups, in.groups, block_of<R>() / R, 4 * 2048 / block_of<R>());
}
uint32_t backward_slices(int64_t rows, int64_t groups, int R) {
    const int block = R <= 32 ? 256 : R;
    return slices_of(rows / groups, groups, block / R, 1024 / block);
}

template <typename T, int V, int R, int K> cudaError_t run(const GatedArgs &a, cudaStream_t s) {
    gated_kernel<T, V, R, K><<<dim3(forward_slices<R>(a.in), a.in.groups), block_of<R>(), 0, s>>>(
        a, (uint32_t)(a.in.rows / a.in.groups));
    return cudaGetLastError();
}

template <typename T, int V, int R, int K> cudaError_t run(const GatedBwdArgs &a, cudaStream_t s) {
    constexpr bool SM = R == 512 && K * V >= 16;
    const GatedIn &in = a.in;
    const uint32_t slices = backward_slices(in.rows, in.groups, R);
    const int smem = !a.ws ? 0 : SM ? 3 * in.width * 4 : R <= 32 ? block_of<R>() / R * in.width * 4 : 0;
    auto k = gated_bwd_kernel<T, V, R, K, SM>;
    if (SM) {
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = allow_smem(k, 3 * kGatedWidth * 4, done);
        if (e != cudaSuccess) return e;
    }
    k<<<dim3(slices, in.groups), block_of<R>(), smem, s>>>(a, (uint32_t)(in.rows / in.groups));
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.ws) return e;
    const int64_t count = (int64_t)in.groups * 3 * in.width;
    return launch_after(gated_sum_kernel, dim3((unsigned)((count + kSumBlock - 1) / kSumBlock)), kSumBlock, 0, s, true,
                        (const float *)a.ws, (int)slices, count, in.width, a.dweight, a.dbias, a.dscale);
}

// Threads of a row, by its vectors.
int threads_of(int vectors, bool scalar) {
    if (scalar) return vectors <= 64 ? 32 : vectors <= 256 ? 128 : vectors <= 1024 ? 256 : 512;
    return vectors <= 8 ? 8 : vectors <= 16 ? 16 : vectors <= 64 ? 32 : vectors <= 256 ? 128 : vectors <= 512 ? 256 : 512;
}

// Elements a load: 16 bytes where rows are whole multiples of it, else 4 bytes (bf16 of even width), else one.
int vector_of(int width, fw_dtype dtype) {
    if (dtype == FW_F32) return width % 4 == 0 ? 4 : 1;
    return width % 8 == 0 ? 8 : width % 2 == 0 ? 2 : 1;
}

// R threads a row, each with as few vectors as its width takes.
template <typename T, int V, typename A> cudaError_t by_width(const A &a, cudaStream_t s) {
    const int n = (a.in.width + V - 1) / V;
    if constexpr (V <= 2) {                        // up to 8192 vectors
        if (n <= 32) return run<T, V, 32, 1>(a, s);
        if (n <= 64) return run<T, V, 32, 2>(a, s);
        if (n <= 256) return run<T, V, 128, 2>(a, s);
        if (n <= 1024) return run<T, V, 256, 4>(a, s);
        if (n <= 2048) return run<T, V, 512, 4>(a, s);
        return run<T, V, 512, 16>(a, s);
    } else {                                       // up to 2048 vectors
        if (n <= 8) return run<T, V, 8, 1>(a, s);
        if (n <= 16) return run<T, V, 16, 1>(a, s);
        if (n <= 32) return run<T, V, 32, 1>(a, s);
        if (n <= 64) return run<T, V, 32, 2>(a, s);
        if (n <= 128) return run<T, V, 128, 1>(a, s);
        if (n <= 256) return run<T, V, 128, 2>(a, s);
        if (n <= 512) return run<T, V, 256, 2>(a, s);
        if (n <= 1024) return run<T, V, 512, 2>(a, s);
        if constexpr (V == 4) return run<T, V, 512, 4>(a, s);
        return cudaErrorInvalidValue;              // (8 x 1024 is the widest row)
    }
}

template <typename A> cudaError_t by_type(const A &a, cudaStream_t s) {
    switch (vector_of(a.in.width, a.in.dtype)) {
    case 8: return by_width<__nv_bfloat16, 8>(a, s);
    case 4: return by_width<float, 4>(a, s);
    case 2: return by_width<__nv_bfloat16, 2>(a, s);
    default:
        return a.in.dtype == FW_F32 ? by_width<float, 1>(a, s) : by_width<__nv_bfloat16, 1>(a, s);
    }
}

}  // namespace

size_t gated_norm_workspace(int64_t rows, int64_t width, int64_t groups, fw_dtype dtype) {
    const int V = vector_of((int)width, dtype);
    const int R = threads_of((int)((width + V - 1) / V), V <= 2);
    return (size_t)backward_slices(rows, groups, R) * groups * 3 * width * sizeof(float);
}

cudaError_t launch_gated_norm(const GatedArgs &a, cudaStream_t s) { return by_type(a, s); }
cudaError_t launch_gated_norm_backward(const GatedBwdArgs &a, cudaStream_t s) { return by_type(a, s); }

}  // namespace fw
