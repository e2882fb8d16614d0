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
// Both are bound by their rows' bytes.  A row is read once, by R threads (a part of a warp, or several) with
// eight elements each; the next rows are on their way into shared memory meanwhile (cp.async, each
// thread into slots of its own, so that nothing but the copies has to be waited for), and the backward
// pass reads a row from there twice, which costs fewer registers than keeping it.  The mean is taken first and
// the squares about it (never E[s^2] - E[s]^2).  Blocks stride over the rows of one group, so that a thread keeps
// its columns' weights and, in the backward pass, its sums in registers; a block writes one
// partial row of sums and a second kernel adds them in a fixed order.
#include "fw_gated_norm.cuh"
#include "fw_partial.cuh"

namespace fw {
namespace {

template <typename T, int V> struct Raw;
template <> struct Raw<float, 1> { float v; };
template <> struct Raw<float, 2> { float2 v; };
template <> struct Raw<float, 4> { float4 v; };
template <> struct Raw<__nv_bfloat16, 1> { __nv_bfloat16 v; };
template <> struct Raw<__nv_bfloat16, 2> { uint32_t v; };
template <> struct Raw<__nv_bfloat16, 4> { uint2 v; };
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
__device__ __forceinline__ void widen(const Raw<float, 2> &r, float (&x)[2]) { x[0] = r.v.x; x[1] = r.v.y; }
__device__ __forceinline__ void widen(const Raw<float, 4> &r, float (&x)[4]) {
    x[0] = r.v.x; x[1] = r.v.y; x[2] = r.v.z; x[3] = r.v.w;
}
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16, 1> &r, float (&x)[1]) { x[0] = __bfloat162float(r.v); }
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16, 2> &r, float (&x)[2]) { unpack(r.v, x[0], x[1]); }
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16, 4> &r, float (&x)[4]) {
    unpack(r.v.x, x[0], x[1]); unpack(r.v.y, x[2], x[3]);
}
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16, 8> &r, float (&x)[8]) {
    unpack(r.v.x, x[0], x[1]); unpack(r.v.y, x[2], x[3]); unpack(r.v.z, x[4], x[5]); unpack(r.v.w, x[6], x[7]);
}
__device__ __forceinline__ void narrow(Raw<float, 1> &r, const float (&x)[1]) { r.v = x[0]; }
__device__ __forceinline__ void narrow(Raw<float, 2> &r, const float (&x)[2]) { r.v = make_float2(x[0], x[1]); }
__device__ __forceinline__ void narrow(Raw<float, 4> &r, const float (&x)[4]) { r.v = make_float4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void narrow(Raw<__nv_bfloat16, 1> &r, const float (&x)[1]) { r.v = __float2bfloat16_rn(x[0]); }
__device__ __forceinline__ void narrow(Raw<__nv_bfloat16, 2> &r, const float (&x)[2]) { r.v = pack(x[0], x[1]); }
__device__ __forceinline__ void narrow(Raw<__nv_bfloat16, 4> &r, const float (&x)[4]) {
    r.v = make_uint2(pack(x[0], x[1]), pack(x[2], x[3]));
}
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


constexpr int kEach = 8;                       // elements of a row a thread

template <int R> constexpr int block_of() { return R < 256 ? 256 : R; }

template <int BYTES> __device__ __forceinline__ void copy_async(void *dst, const void *src) {
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest `left` groups of copies have landed.
__device__ __forceinline__ void copies_wait(int left) {
    if (left == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (left == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 2;" ::: "memory");
}

// The sums of N values over the R threads that hold a row, in every one of them.  All threads of the block.
template <int R, int N> __device__ __forceinline__ void row_sums(float (&z)[N], float *red) {
    constexpr int W = R < 32 ? R : 32;
#pragma unroll
    for (int o = W / 2; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] += __shfl_xor_sync(~0u, z[i], o);
    if constexpr (R > 32) {
        constexpr int NW = R / 32, ALL = block_of<R>() / 32;
        const int warp = threadIdx.x >> 5, first = warp / NW * NW;
        __syncthreads();                       // the sums before are read
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[i * ALL + warp] = z[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            z[i] = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) z[i] += red[i * ALL + first + w];
        }
    }
}

__device__ __forceinline__ int64_t row_of(const GatedIn &in, uint32_t group, uint32_t m) {
    if (in.groups == 1) return m;
    return ((int64_t)(m / (uint32_t)in.inner) * in.groups + group) * in.inner + m % (uint32_t)in.inner;
}

// The rows that a thread works on, up to `stages` of them ahead in its slots of shared memory: `n` arrays, K vectors
// each.  (Elements of two bytes are no copy's size: those are read from memory when asked for.)
template <typename T, int V, int R, int N> struct Ahead {
    static constexpr int BYTES = V * (int)sizeof(T), K = kEach / V;
    static constexpr bool COPY = BYTES >= 4;
    const void *src[N];
    Raw<T, V> *slots;
    int stages, width, lane;
    int64_t at;                                // of the row at hand
    int stage = 0;

    __device__ __forceinline__ Raw<T, V> *slot(int s, int a, int k) const {
        return slots + ((s * N + a) * K + k) * block_of<R>() + threadIdx.x;
    }
    __device__ __forceinline__ int column(int k) const { return (k * R + lane) * V; }
    // Copies of a row into a stage, a group of them whether there is a row or not.
    __device__ __forceinline__ void fetch(int s, bool live, int64_t row_at) {
        if constexpr (COPY) {
            if (live)
#pragma unroll
                for (int a = 0; a < N; ++a)
                    if (src[a])
#pragma unroll
                        for (int k = 0; k < K; ++k)
                            if (column(k) < width)
                                copy_async<BYTES>(slot(s, a, k), static_cast<const T *>(src[a]) + row_at + column(k));
            copies_commit();
        }
    }
    __device__ __forceinline__ void get(int a, int k, float (&x)[V]) const {
        if constexpr (COPY) widen(*slot(stage, a, k), x);
        else widen(load<T, V>(src[a], at + column(k)), x);
    }
};

// Walks the rows of a block's share of group blockIdx.y: work(live, row, next row or -1) with the row's
// data in `ahead`.
template <typename T, int V, int R, int N, typename F>
__device__ __forceinline__ void over_rows(Ahead<T, V, R, N> &ahead, const GatedIn &in, uint32_t group_rows, F work) {
    constexpr int RPB = block_of<R>() / R;
    const uint32_t step = gridDim.x * RPB;
    auto fetch = [&](int s, uint32_t m0) {
        const uint32_t m = m0 + threadIdx.x / R;
        const bool live = m0 < group_rows && m < group_rows;
        ahead.fetch(s, live, live ? row_of(in, blockIdx.y, m) * in.width : 0);
    };
    uint32_t m0 = blockIdx.x * RPB, ask = m0;
    for (int s = 0; s < ahead.stages; ++s, ask += step) fetch(s, ask);
    int64_t row = m0 < group_rows ? row_of(in, blockIdx.y, min(m0 + threadIdx.x / R, group_rows - 1)) : 0;
    for (; m0 < group_rows; m0 += step) {
        const bool live = m0 + threadIdx.x / R < group_rows;
        const uint32_t m = m0 + step + threadIdx.x / R;
        const int64_t next = m < group_rows ? row_of(in, blockIdx.y, m) : -1;
        ahead.at = row * in.width;
        if (Ahead<T, V, R, N>::COPY) copies_wait(ahead.stages - 1);
        work(live, row, next);
        fetch(ahead.stage, ask);
        row = next < 0 ? row : next;
        ask += step;
        if (++ahead.stage == ahead.stages) ahead.stage = 0;
    }
    if (Ahead<T, V, R, N>::COPY) copies_wait(0);
}

template <typename T, int V, int R>
__global__ void __launch_bounds__(block_of<R>(), 1) gated_kernel(GatedArgs a, uint32_t group_rows, int stages) {
    constexpr int K = kEach / V, BLOCK = block_of<R>();
    extern __shared__ uint4 slots[];
    __shared__ float red[R > 32 ? BLOCK / 32 : 1];
    const GatedIn &in = a.in;
    Ahead<T, V, R, 3> ahead{{in.x, in.gate, in.residual}, reinterpret_cast<Raw<T, V> *>(slots), stages, in.width,
                            (int)(threadIdx.x % R), 0};
    const float inv = 1.f / (float)in.width;
    const int64_t pat = (int64_t)blockIdx.y * in.width;
    float w[K][V], b[K][V], f[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = ahead.column(k);
        if (c < in.width) {
            param<V>(in.weight, pat + c, 1.f, w[k]);
            param<V>(in.bias, pat + c, 0.f, b[k]);
            param<V>(in.scale, pat + c, 1.f, f[k]);
        }
    }
    over_rows(ahead, in, group_rows, [&](bool live, int64_t row, int64_t) {
        float s[K][V], sum[1] = {0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = ahead.column(k);
            if (live && c < in.width) {
                ahead.get(0, k, s[k]);
                if (in.residual) {
                    float r[V];
                    ahead.get(2, k, r);
#pragma unroll
                    for (int e = 0; e < V; ++e) s[k][e] = fmaf(f[k][e], r[e], s[k][e]);
                }
                if (a.total) store<T, V>(a.total, ahead.at + c, s[k]);
                if (in.gate && !in.gate_after) {
                    float z[V];
                    ahead.get(1, k, z);
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
            if (ahead.column(k) < in.width)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    s[k][e] -= mean;
                    sum[0] = fmaf(s[k][e], s[k][e], sum[0]);
                }
        row_sums<R>(sum, red);
        const float rstd = rsqrtf(fmaf(sum[0], inv, in.eps));
        if (!live) return;
        if (ahead.lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = ahead.column(k);
            if (c >= in.width) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) s[k][e] = fmaf(s[k][e] * rstd, w[k][e], b[k][e]);
            if (in.gate && in.gate_after) {
                float z[V];
                ahead.get(1, k, z);
#pragma unroll
                for (int e = 0; e < V; ++e) s[k][e] *= z[e] * sigmoid<T>(z[e]);
            }
            store<T, V>(a.y, ahead.at + c, s[k]);
        }
    });
}

template <typename T, int V, int R>
__global__ void __launch_bounds__(block_of<R>(), 1) gated_bwd_kernel(GatedBwdArgs a, uint32_t group_rows, int stages) {
    constexpr int K = kEach / V, BLOCK = block_of<R>(), RPB = BLOCK / R;
    extern __shared__ uint4 slots[];
    __shared__ float red[R > 32 ? 2 * BLOCK / 32 : 1];
    const GatedIn &in = a.in;
    Ahead<T, V, R, 5> ahead{{in.x, a.dy, in.gate, in.residual, a.dtotal}, reinterpret_cast<Raw<T, V> *>(slots), stages,
                            in.width, (int)(threadIdx.x % R), 0};
    const int width = in.width;
    const float inv = 1.f / (float)width;
    const int64_t pat = (int64_t)blockIdx.y * width;
    float sums[3][K][V];                       // of dweight, dbias, dscale
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) sums[i][k][e] = 0.f;
    float next_mean = 0.f, next_rstd = 0.f;    // of the next row
    {
        const uint32_t m = blockIdx.x * RPB + threadIdx.x / R;
        if (m < group_rows) {
            const int64_t row = row_of(in, blockIdx.y, m);
            if (!in.rms) next_mean = a.mean[row];
            next_rstd = a.rstd[row];
        }
    }
    over_rows(ahead, in, group_rows, [&](bool live, int64_t row, int64_t next) {
        const float mean = next_mean, rstd = next_rstd;
        if (next >= 0) {
            if (!in.rms) next_mean = a.mean[next];
            next_rstd = a.rstd[next];
        }
        float sg[K][V];                        // sigmoid of the gate
        // n = norm(s), g and u of a vector
        auto form = [&](int k, int c, float (&n)[V], float (&g)[V], float (&u)[V], float (&dy)[V], float (&z)[V]) {
            ahead.get(0, k, u);
            if (in.residual) {
                float f[V], r[V];
                param<V>(in.scale, pat + c, 1.f, f);
                ahead.get(3, k, r);
#pragma unroll
                for (int e = 0; e < V; ++e) u[e] = fmaf(f[e], r[e], u[e]);
            }
            ahead.get(1, k, dy);
            float w[V];
            param<V>(in.weight, pat + c, 1.f, w);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                n[e] = u[e];
                g[e] = dy[e] * w[e];
            }
            if (in.gate) {
                ahead.get(2, k, z);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float act = z[e] * sg[k][e];
                    if (in.gate_after) g[e] *= act;
                    else n[e] *= act;
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) n[e] = (n[e] - mean) * rstd;
        };
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = ahead.column(k);
            if (live && c < width) {
                float n[V], g[V], u[V], dy[V], z[V];
                if (in.gate) {
                    ahead.get(2, k, z);
#pragma unroll
                    for (int e = 0; e < V; ++e) sg[k][e] = sigmoid<T>(z[e]);
                }
                form(k, c, n, g, u, dy, z);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    sum[0] += g[e];
                    sum[1] = fmaf(g[e], n[e], sum[1]);
                }
            }
        }
        row_sums<R>(sum, red);
        const float mg = in.rms ? 0.f : sum[0] * inv, mgn = sum[1] * inv;
        if (!live) return;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = ahead.column(k);
            if (c >= width) continue;
            float n[V], g[V], u[V], dy[V], z[V], d[V];
            form(k, c, n, g, u, dy, z);
#pragma unroll
            for (int e = 0; e < V; ++e) d[e] = rstd * (g[e] - mg - n[e] * mgn);
            if (in.gate) {
                float dz[V];
                if (in.gate_after) {
                    float b[V], w[V];
                    param<V>(in.weight, pat + c, 1.f, w);
                    param<V>(in.bias, pat + c, 0.f, b);
#pragma unroll
                    for (int e = 0; e < V; ++e) dz[e] = dy[e] * fmaf(n[e], w[e], b[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) dz[e] = d[e] * u[e];
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float act = z[e] * sg[k][e];
                    dz[e] *= sg[k][e] * (1.f + z[e] - act);    // silu'
                    if (in.gate_after) dy[e] *= act;           // of the norm's output
                    else d[e] *= act;
                }
                if (a.dgate) store<T, V>(a.dgate, ahead.at + c, dz);
            }
            if (a.dtotal) {
                float t[V];
                ahead.get(4, k, t);
#pragma unroll
                for (int e = 0; e < V; ++e) d[e] += t[e];
            }
            if (a.dx) store<T, V>(a.dx, ahead.at + c, d);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                sums[0][k][e] = fmaf(dy[e], n[e], sums[0][k][e]);
                sums[1][k][e] += dy[e];
            }
            if (in.residual) {
                float f[V], r[V];
                param<V>(in.scale, pat + c, 1.f, f);
                ahead.get(3, k, r);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    sums[2][k][e] = fmaf(r[e], d[e], sums[2][k][e]);
                    f[e] *= d[e];
                }
                if (a.dresidual) store<T, V>(a.dresidual, ahead.at + c, f);
            }
        }
    });
    let_next_grid_start();
    if (!a.ws) return;
    // [block of the group][group][3][width]; the rows that a block holds at once one after the other
    float *const out = a.ws + ((int64_t)blockIdx.x * in.groups + blockIdx.y) * 3 * width;
    float *const part = reinterpret_cast<float *>(slots);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (!(i == 0 ? a.dweight : i == 1 ? a.dbias : a.dscale)) continue;   // (uniform)
        if constexpr (RPB == 1) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (ahead.column(k) < width)
#pragma unroll
                    for (int e = 0; e < V; ++e) out[i * width + ahead.column(k) + e] = sums[i][k][e];
        } else {
            __syncthreads();                   // (the slots are free, or the sums before read)
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) part[(threadIdx.x / R) * (R * kEach) + ahead.column(k) + e] = sums[i][k][e];
            __syncthreads();
            for (int c = threadIdx.x; c < width; c += BLOCK) {
                float z = 0.f;
#pragma unroll 4
                for (int p = 0; p < RPB; ++p) z += part[p * (R * kEach) + c];
                out[i * width + c] = z;
            }
        }
    }
}

// Sums of the blocks in a fixed order.
__global__ void __launch_bounds__(kSumCols * kSumShares)
gated_sum_kernel(const float *ws, int slices, int64_t count, int width, float *dweight, float *dbias, float *dscale) {
    wait_previous_grid();
    sum_slices(ws, slices, count, [&](int64_t i, float z) {               // i: of [groups][3][width]
        const int which = (int)(i / width % 3);
        float *const out = which == 0 ? dweight : which == 1 ? dbias : dscale;
        if (out) out[i / (3 * width) * width + i % width] = z;
    });
}

// Blocks of an SM, of R threads a row.
constexpr int blocks_an_sm(int R) { return R < 512 ? 3 : R < 1024 ? 2 : 1; }

// Blocks that share the rows of a group: what the SMs hold at once, and no more than there are rows for.
uint32_t slices_of(int64_t rows, int64_t groups, int R, int turns) {
    const int64_t group_rows = rows / groups, each = R < 256 ? 256 / R : 1, most = (group_rows + each - 1) / each;
    const int64_t s = (int64_t)kSMs * blocks_an_sm(R) * turns / groups;
    return (uint32_t)(s < 1 ? 1 : s > most ? most : s);
}

// Rows ahead, of `arrays` a block each, that leave room for the blocks of an SM.
template <typename T, int R> int stages_of(int arrays) {
    const int row = arrays * block_of<R>() * kEach * (int)sizeof(T), room = 216 * 1024 / blocks_an_sm(R);
    return row * 3 <= room ? 3 : row * 2 <= room ? 2 : 1;
}

template <typename T, int V, int R> cudaError_t run(const GatedArgs &a, cudaStream_t s) {
    const int stages = stages_of<T, R>(3), smem = stages * 3 * block_of<R>() * kEach * (int)sizeof(T);
    auto k = gated_kernel<T, V, R>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(k, smem, done);
    if (e != cudaSuccess) return e;
    k<<<dim3(slices_of(a.in.rows, a.in.groups, R, 1), a.in.groups), block_of<R>(), smem, s>>>(
        a, (uint32_t)(a.in.rows / a.in.groups), stages);
    return cudaGetLastError();
}

template <typename T, int V, int R> cudaError_t run(const GatedBwdArgs &a, cudaStream_t s) {
    const GatedIn &in = a.in;
    const uint32_t slices = slices_of(in.rows, in.groups, R, 1);
    const int stages = stages_of<T, R>(5), smem = stages * 5 * block_of<R>() * kEach * (int)sizeof(T);
    auto k = gated_bwd_kernel<T, V, R>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(k, smem, done);
    if (e != cudaSuccess) return e;
    k<<<dim3(slices, in.groups), block_of<R>(), smem, s>>>(a, (uint32_t)(in.rows / in.groups), stages);
    if ((e = cudaGetLastError()) != cudaSuccess || !a.ws) return e;
    const int64_t count = (int64_t)in.groups * 3 * in.width;
    return launch_after(gated_sum_kernel, sum_grid(count), kSumCols * kSumShares, 0, s, true, (const float *)a.ws,
                        (int)slices, count, in.width, a.dweight, a.dbias, a.dscale);
}

// Threads of a row.
int threads_of(int width) {
    int R = 8;
    while (R * kEach < width) R *= 2;
    return R;
}

template <typename T, int V, typename A> cudaError_t by_width(const A &a, cudaStream_t s) {
    switch (threads_of(a.in.width)) {
    case 8: return run<T, V, 8>(a, s);
    case 16: return run<T, V, 16>(a, s);
    case 32: return run<T, V, 32>(a, s);
    case 64: return run<T, V, 64>(a, s);
    case 128: return run<T, V, 128>(a, s);
    case 256: return run<T, V, 256>(a, s);
    case 512: return run<T, V, 512>(a, s);
    default:
        // (1024 threads have 64 registers each: a vector of eight at a time is more than they hold)
        return run<T, V == 8 ? 4 : V, 1024>(a, s);
    }
}

// Elements a load: 16 bytes where rows are whole multiples of it, else two (even widths), else one.
template <typename A> cudaError_t by_type(const A &a, cudaStream_t s) {
    const int w = a.in.width;
    if (a.in.dtype == FW_F32)
        return w % 4 == 0 ? by_width<float, 4>(a, s) : w % 2 == 0 ? by_width<float, 2>(a, s) : by_width<float, 1>(a, s);
    return w % 8 == 0 ? by_width<__nv_bfloat16, 8>(a, s)
                      : w % 2 == 0 ? by_width<__nv_bfloat16, 2>(a, s) : by_width<__nv_bfloat16, 1>(a, s);
}

}  // namespace

size_t gated_norm_workspace(int64_t rows, int64_t width, int64_t groups) {
    return (size_t)slices_of(rows, groups, threads_of((int)width), 1) * groups * 3 * width * sizeof(float);
}

cudaError_t launch_gated_norm(const GatedArgs &a, cudaStream_t s) { return by_type(a, s); }
cudaError_t launch_gated_norm_backward(const GatedBwdArgs &a, cudaStream_t s) { return by_type(a, s); }

}  // namespace fw
