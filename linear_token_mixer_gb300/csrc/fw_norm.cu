// fw_norm.cu -- layer norm over the last axis, forward and backward:
//     y  = (x - m) r w + b,   m = mean(x),  r = 1 / sqrt(mean((x - m)^2) + eps)
//     dx = r (w dy - mean(w dy) - xh mean(w dy xh)),   xh = (x - m) r
//     dw = sum_rows dy xh,   db = sum_rows dy
//
// Both passes are bound by their rows' bytes: each row is read once (16 bytes a thread and vector, the
// loads of the next row, or of the next two or three, in flight while this one is worked on) into
// registers, the statistics are taken from there and the result is written.  A row is held by ROWT threads: a
// part of a warp for short rows, a warp, or a block; blocks stride over the rows and keep the
// weights of their columns in registers.  Mean and variance come from one reduction: each thread
// takes the mean and the centred sum of squares of its own values, and pairs are merged by the
// parallel update of Chan, Golub and LeVeque (never E[x^2] - E[x]^2).  Widths that are no multiple
// of 16 bytes take the same kernels with two elements a load, or one; rows that do not fit the registers of
// 1024 threads take the looping kernels, which read the row again for each pass.
//
// Measured (one GB300, 32768 x 2048 bf16): forward 56 us, 4.8 TB/s, 70 % of the measured copy rate;
// backward with its sums 81 us, 5.0 TB/s, 73 %.  What is left is the turn of a row: its reduction is
// a chain of shuffles and a barrier that the few rows of an SM cover only in part.  64 x 2048: 7.3 us and
// 12.4 us, of which a launch is most.
//
// The backward kernel keeps its columns' dw and db in registers too; every block writes one
// partial row and a second kernel adds the partial rows in a fixed order, so the sums do not
// depend on the order in which blocks run.
#include <type_traits>

#include "fw_decay.cuh"

namespace fw {
namespace {

constexpr int kBlock = 256;     // block of the part-of-a-warp forms
constexpr int kPartials = 4 * kSMs;   // most partial rows of dw, db

template <typename T, int VW> struct Vec;
template <typename T> struct Vec<T, 1> { T e[1]; };
template <> struct alignas(16) Vec<float, 4> { float e[4]; };
template <> struct alignas(16) Vec<__nv_bfloat16, 8> { __nv_bfloat16 e[8]; };
template <> struct alignas(8) Vec<float, 2> { float e[2]; };               // even widths
template <> struct alignas(4) Vec<__nv_bfloat16, 2> { __nv_bfloat16 e[2]; };

// fp32 arithmetic on the VW elements of a vector, two in one instruction where there are two.
template <int N> struct Row {   // N values
    float e[N];
};
// a b + c; a scalar stands for N equal values
template <int N> __device__ __forceinline__ Row<N> fma_n(const Row<N> &a, const Row<N> &b, const Row<N> &c) {
    Row<N> d;
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 f = halves(fma2(pair(a.e[i], a.e[i + 1]), pair(b.e[i], b.e[i + 1]), pair(c.e[i], c.e[i + 1])));
            d.e[i] = f.x;
            d.e[i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) d.e[i] = fmaf(a.e[i], b.e[i], c.e[i]);
    }
    return d;
}
template <int N> __device__ __forceinline__ Row<N> all(float x) {
    Row<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.e[i] = x;
    return r;
}
template <int N> __device__ __forceinline__ float total(const Row<N> &a) {
    float t = a.e[0];
#pragma unroll
    for (int i = 1; i < N; ++i) t += a.e[i];
    return t;
}
template <typename T, int N> __device__ __forceinline__ Row<N> widen(const Vec<T, N> &v) {
    Row<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.e[i] = to_f32(v.e[i]);
    return r;
}
template <typename T, int N> __device__ __forceinline__ Vec<T, N> narrow(const Row<N> &a) {
    Vec<T, N> v;
#pragma unroll
    for (int i = 0; i < N; ++i) v.e[i] = from_f32<T>(a.e[i]);
    return v;
}
template <> __device__ __forceinline__ Vec<__nv_bfloat16, 8> narrow(const Row<8> &a) {
    Vec<__nv_bfloat16, 8> v;
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        reinterpret_cast<__nv_bfloat162 *>(v.e)[i / 2] = __floats2bfloat162_rn(a.e[i], a.e[i + 1]);
    return v;
}

// Sum over a block of 1024 threads (looping kernels).
__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += red[i];
    __syncthreads();
    return v;
}

// Sums of two values over the ROWT threads of a row.  The block form takes one barrier: `red`
// (2 x 32 floats for each parity of the turn) is not written again before the next but one.
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
    }
}

// Count, mean and centred sum of squares of a set of values.
struct Moments {
    float n, m, s;
};
__device__ __forceinline__ Moments merge(const Moments &a, const Moments &b) {
    const float n = a.n + b.n, r = n > 0.f ? __fdividef(b.n, n) : 0.f, d = b.m - a.m;
    return {n, fmaf(d, r, a.m), fmaf(d * d, a.n * r, a.s + b.s)};
}
template <int ROWT> __device__ __forceinline__ Moments row_merge(Moments x, Moments *red) {
    constexpr int W = ROWT < 32 ? ROWT : 32;
#pragma unroll
    for (int o = W / 2; o; o >>= 1) {
        const Moments y{__shfl_xor_sync(~0u, x.n, o), __shfl_xor_sync(~0u, x.m, o),
                        __shfl_xor_sync(~0u, x.s, o)};
        // the same order on both sides, so that every thread has the same bits
        x = threadIdx.x & o ? merge(y, x) : merge(x, y);
    }
    if constexpr (ROWT > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
        __syncthreads();
        x = red[0];
#pragma unroll
        for (int i = 1; i < ROWT / 32; ++i) x = merge(x, red[i]);
    }
    return x;
}

template <int ROWT> constexpr int block_of() { return ROWT <= 32 ? kBlock : ROWT; }

// VW floats of weight or bias from column c on (c a multiple of VW).
template <int VW, bool GIVEN> __device__ __forceinline__ Row<VW> load_w(const float *p, int c, float none) {
    Row<VW> w;
    if constexpr (VW >= 4) {
#pragma unroll
        for (int e = 0; e < VW; e += 4) {
            const float4 f = GIVEN || p ? *reinterpret_cast<const float4 *>(p + c + e) : make_float4(none, none, none, none);
            w.e[e] = f.x; w.e[e + 1] = f.y; w.e[e + 2] = f.z; w.e[e + 3] = f.w;
        }
    } else if constexpr (VW == 2) {
        const float2 f = GIVEN || p ? *reinterpret_cast<const float2 *>(p + c) : make_float2(none, none);
        w.e[0] = f.x;
        w.e[1] = f.y;
    } else {
        w.e[0] = GIVEN || p ? p[c] : none;
    }
    return w;
}

// Rows on their way through shared memory, DEPTH - 1 of them behind the one that is worked on: for
// each thread its own PIECES of 16 bytes and two floats of its row.  (With one row ahead, in registers,
// the backward pass had 32 KB an SM in flight, where the memory's latency needs twice that.)
template <int THREADS, int PIECES> struct Ahead {
    static constexpr int STAGE = THREADS * (PIECES * 16 + 8);
    static constexpr int DEPTH = 4 * STAGE * (THREADS < 512 ? 512 / THREADS : 1) <= 160 * 1024 ? 4 : 3;
    static constexpr int BYTES = DEPTH * STAGE;
};
template <int N> __device__ __forceinline__ void copy_async(void *to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
                 "l"(from), "n"(N)
                 : "memory");
}
template <> __device__ __forceinline__ void copy_async<16>(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
                 "l"(from)
                 : "memory");
}
__device__ __forceinline__ void copies_begun() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last N groups have landed (a thread reads its own copies alone).
template <int N> __device__ __forceinline__ void copies_landed() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The forward pass takes its rows that way where a part of a warp holds one: 524288 x 128 bf16 61 us
// in registers, 54 us ahead; rows held by blocks, of which more fit an SM without, 32768 x 2048 56 us
// and 60 us.  (With one vector a thread there is one row, or next to nothing, to read ahead.)
template <typename T, int VW, int ROWT, int VPT> constexpr bool fwd_ahead() {
    return VW * sizeof(T) == 16 && VPT > 1 && ROWT <= 32;
}

// FAST: every thread holds VPT whole vectors of 16 bytes, and weight and bias are given (the checks for
// the other cases are as many instructions as the work).
template <typename T, int VW, int ROWT, int VPT, bool FAST>
__global__ void __launch_bounds__(block_of<ROWT>(), FAST && ROWT <= 512 ? 512 / block_of<ROWT>() : 1)
ln_fwd(LayerNormArgs a) {
    __shared__ Moments red[2][32];
    extern __shared__ float4 dyn[];        // the rows ahead
    constexpr int RPB = block_of<ROWT>() / ROWT, THREADS = block_of<ROWT>();
    constexpr bool ASYNC = fwd_ahead<T, VW, ROWT, VPT>();
    using Q = Ahead<THREADS, VPT>;
    constexpr bool KEEP = VPT * VW <= 16;  // weights in registers, or from L1 for every row
    using V = Vec<T, VW>;
    const int lane = threadIdx.x % ROWT, sub = threadIdx.x / ROWT;
    const int nv = (int)a.width / VW;
    Row<VW> w[KEEP ? VPT : 1], b[KEEP ? VPT : 1];
    if constexpr (KEEP) {
#pragma unroll
        for (int p = 0; p < VPT; ++p)
            if ((FAST || p * ROWT + lane < nv)) {
                w[p] = load_w<VW, FAST>(a.weight, (p * ROWT + lane) * VW, 1.f);
                b[p] = load_w<VW, FAST>(a.bias, (p * ROWT + lane) * VW, 0.f);
            }
    }
    V xv[VPT], nx[VPT];
    auto load = [&](int64_t row, int slot) {
        const V *x = reinterpret_cast<const V *>(static_cast<const T *>(a.x) + row * a.width);
#pragma unroll
        for (int p = 0; p < VPT; ++p)
            if (row < a.rows && (FAST || p * ROWT + lane < nv)) {
                if constexpr (ASYNC) copy_async<16>(dyn + (slot * VPT + p) * THREADS + threadIdx.x, x + p * ROWT + lane);
                else nx[p] = x[p * ROWT + lane];
            }
        if constexpr (ASYNC) copies_begun();
    };
    const int64_t stride = (int64_t)gridDim.x * RPB;
    int turn = 0, slot = 0;
    load((int64_t)blockIdx.x * RPB + sub, 0);
    if constexpr (ASYNC)
#pragma unroll
        for (int i = 1; i < Q::DEPTH - 1; ++i) load((int64_t)blockIdx.x * RPB + sub + i * stride, i);
    // every thread of the block makes the same number of turns (the merge synchronises)
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += stride, turn ^= 1) {
        const int64_t row = r0 + sub;
        const bool on = row < a.rows;
        if constexpr (ASYNC) {
            copies_landed<Q::DEPTH - 2>();
            const V *const at = reinterpret_cast<const V *>(dyn + slot * VPT * THREADS + threadIdx.x);
#pragma unroll
            for (int p = 0; p < VPT; ++p)
                if (on && (FAST || p * ROWT + lane < nv)) xv[p] = at[p * THREADS];
            // over the row before this one
            load(row + (Q::DEPTH - 1) * stride, slot == 0 ? Q::DEPTH - 1 : slot - 1);
            slot = slot == Q::DEPTH - 1 ? 0 : slot + 1;
        } else {
#pragma unroll
            for (int p = 0; p < VPT; ++p) xv[p] = nx[p];
            load(row + stride, 0);
        }
        Moments mo{0.f, 0.f, 0.f};
        Row<VW> acc = all<VW>(0.f);
#pragma unroll
        for (int p = 0; p < VPT; ++p)
            if (on && (FAST || p * ROWT + lane < nv)) {
                mo.n += (float)VW;
                acc = fma_n(widen(xv[p]), all<VW>(1.f), acc);
            }
        mo.m = mo.n > 0.f ? total(acc) / mo.n : 0.f;
        acc = all<VW>(0.f);
#pragma unroll
        for (int p = 0; p < VPT; ++p)
            if (on && (FAST || p * ROWT + lane < nv)) {
                const Row<VW> d = fma_n(widen(xv[p]), all<VW>(1.f), all<VW>(-mo.m));
                acc = fma_n(d, d, acc);
            }
        mo.s = total(acc);
        mo = row_merge<ROWT>(mo, red[turn]);
        if (!on) continue;
        const float mean = mo.m, rstd = rsqrtf(mo.s / (float)a.width + a.eps);
        V *y = reinterpret_cast<V *>(static_cast<T *>(a.y) + row * a.width);
#pragma unroll
        for (int p = 0; p < VPT; ++p) {
            const int i = p * ROWT + lane;
            if (!FAST && i >= nv) continue;
            if constexpr (!KEEP) {
                w[0] = load_w<VW, FAST>(a.weight, i * VW, 1.f);
                b[0] = load_w<VW, FAST>(a.bias, i * VW, 0.f);
            }
            const Row<VW> d = fma_n(widen(xv[p]), all<VW>(1.f), all<VW>(-mean));
            y[i] = narrow<T>(fma_n(fma_n(d, all<VW>(rstd), all<VW>(0.f)), w[KEEP ? p : 0], b[KEEP ? p : 0]));
        }
        if (lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
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
    const float mean = block_sum(sum, red) / (float)a.width;
    float var = 0.f;
    for (int64_t i = threadIdx.x; i < a.width; i += 1024) {
        const float d = to_f32(x[i]) - mean;
        var = fmaf(d, d, var);
    }
    const float rstd = rsqrtf(block_sum(var, red) / (float)a.width + a.eps);
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

template <typename T, int VW, int ROWT, int VPT, bool FAST>
__global__ void __launch_bounds__(block_of<ROWT>(), FAST && ROWT <= 512 ? 512 / block_of<ROWT>() : 1)
ln_bwd(LayerNormBwdArgs a) {
    __shared__ float red[2][64];
    // 16-byte vectors: the rows ahead; then, part-of-a-warp forms: sums [RPB][2][width]
    extern __shared__ float4 dyn[];
    float *const sacc = reinterpret_cast<float *>(dyn);
    constexpr int RPB = block_of<ROWT>() / ROWT, THREADS = block_of<ROWT>();
    constexpr bool ASYNC = VW * sizeof(T) == 16;
    using V = Vec<T, VW>;
    using Q = Ahead<THREADS, 2 * VPT>;
    const int lane = threadIdx.x % ROWT, sub = threadIdx.x / ROWT;
    const int W = (int)a.width, nv = W / VW;
    const bool sums = a.ws != nullptr;
    let_next_grid_start();
    Row<VW> w[VPT], dw[VPT], db[VPT];
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
        w[p] = dw[p] = db[p] = all<VW>(0.f);
        if ((FAST || p * ROWT + lane < nv)) w[p] = load_w<VW, FAST>(a.weight, (p * ROWT + lane) * VW, 1.f);
    }
    V nx[VPT], ng[VPT];
    float nmean = 0.f, nrstd = 0.f;
    float2 *const stats = reinterpret_cast<float2 *>(dyn + Q::DEPTH * 2 * VPT * THREADS);
    auto load = [&](int64_t row, int slot) {
        if (row < a.rows) {
            const V *x = reinterpret_cast<const V *>(static_cast<const T *>(a.x) + row * a.width);
            const V *dy = reinterpret_cast<const V *>(static_cast<const T *>(a.dy) + row * a.width);
            float4 *const to = dyn + slot * 2 * VPT * THREADS + threadIdx.x;
#pragma unroll
            for (int p = 0; p < VPT; ++p)
                if ((FAST || p * ROWT + lane < nv)) {
                    if constexpr (ASYNC) {
                        copy_async<16>(to + p * THREADS, x + p * ROWT + lane);
                        copy_async<16>(to + (VPT + p) * THREADS, dy + p * ROWT + lane);
                    } else {
                        nx[p] = x[p * ROWT + lane];
                        ng[p] = dy[p * ROWT + lane];
                    }
                }
            if constexpr (ASYNC) {
                copy_async<4>(&stats[slot * THREADS + threadIdx.x].x, a.mean + row);
                copy_async<4>(&stats[slot * THREADS + threadIdx.x].y, a.rstd + row);
            } else {
                nmean = a.mean[row];
                nrstd = a.rstd[row];
            }
        }
        if constexpr (ASYNC) copies_begun();
    };
    const int64_t stride = (int64_t)gridDim.x * RPB;
    int turn = 0, slot = 0;
    load((int64_t)blockIdx.x * RPB + sub, 0);
    if constexpr (ASYNC)
#pragma unroll
        for (int i = 1; i < Q::DEPTH - 1; ++i) load((int64_t)blockIdx.x * RPB + sub + i * stride, i);
    // every thread of the block makes the same number of turns (the row sums synchronise)
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += stride, turn ^= 1) {
        const int64_t row = r0 + sub;
        const bool on = row < a.rows;
        if constexpr (ASYNC) {
            copies_landed<Q::DEPTH - 2>();
            const V *const at = reinterpret_cast<const V *>(dyn + slot * 2 * VPT * THREADS + threadIdx.x);
            if (on) {
#pragma unroll
                for (int p = 0; p < VPT; ++p)
                    if (FAST || p * ROWT + lane < nv) {
                        nx[p] = at[p * THREADS];
                        ng[p] = at[(VPT + p) * THREADS];
                    }
                const float2 st = stats[slot * THREADS + threadIdx.x];
                nmean = st.x;
                nrstd = st.y;
            }
            // over the row before this one
            load(row + (Q::DEPTH - 1) * stride, slot == 0 ? Q::DEPTH - 1 : slot - 1);
            slot = slot == Q::DEPTH - 1 ? 0 : slot + 1;
        }
        const float mean = nmean, rstd = nrstd;
        Row<VW> xh[VPT], gw[VPT];
        Row<VW> s1 = all<VW>(0.f), s2 = all<VW>(0.f);
#pragma unroll
        for (int p = 0; p < VPT; ++p)
            if (on && (FAST || p * ROWT + lane < nv)) {
                const Row<VW> g = widen(ng[p]);
                const Row<VW> d = fma_n(widen(nx[p]), all<VW>(1.f), all<VW>(-mean));
                xh[p] = fma_n(d, all<VW>(rstd), all<VW>(0.f));
                gw[p] = fma_n(g, w[p], all<VW>(0.f));
                dw[p] = fma_n(g, xh[p], dw[p]);
                db[p] = fma_n(g, all<VW>(1.f), db[p]);
                s1 = fma_n(gw[p], all<VW>(1.f), s1);
                s2 = fma_n(gw[p], xh[p], s2);
            }
        if constexpr (!ASYNC) load(row + stride, 0);
        float c1 = total(s1), c2 = total(s2);
        row_sum2<ROWT>(c1, c2, red[turn]);
        c1 /= W;
        c2 /= W;
        if (!on) continue;
        V *dx = reinterpret_cast<V *>(static_cast<T *>(a.dx) + row * a.width);
#pragma unroll
        for (int p = 0; p < VPT; ++p) {
            const int i = p * ROWT + lane;
            if (!FAST && i >= nv) continue;
            const Row<VW> t = fma_n(xh[p], all<VW>(-c2), fma_n(gw[p], all<VW>(1.f), all<VW>(-c1)));
            dx[i] = narrow<T>(fma_n(t, all<VW>(rstd), all<VW>(0.f)));
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
                if (FAST || c < W) {
                    part[c] = dw[p].e[e];
                    part[W + c] = db[p].e[e];
                }
            }
    } else {
        if constexpr (ASYNC) {
            copies_landed<0>();
            __syncthreads();               // the sums take the place of the rows
        }
#pragma unroll
        for (int p = 0; p < VPT; ++p)
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                const int c = (p * ROWT + lane) * VW + e;
                if (FAST || c < W) {
                    sacc[sub * 2 * W + c] = dw[p].e[e];
                    sacc[sub * 2 * W + W + c] = db[p].e[e];
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
    c1 = block_sum(c1, red);
    c2 = block_sum(c2, red);
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
    wait_previous_grid();
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

// Blocks of a grid whose blocks stride over the rows: all of them, or what fits the GPU at once.
template <typename K> cudaError_t resident(K k, int threads, size_t smem, int64_t blocks, int64_t *n) {
    int dev = 0, sms = 0, per = 0;
    cudaError_t e;
    *n = blocks;
    if (blocks <= kSMs) return cudaSuccess;   // at most one an SM in any case
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, k, threads, smem)) != cudaSuccess) return e;
    const int64_t most = (int64_t)sms * (per < 1 ? 1 : per);
    if (*n > most) *n = most;
    return cudaSuccess;
}

template <typename T, int VW, int ROWT, int VPT>
cudaError_t fwd(const LayerNormArgs &a, cudaStream_t s) {
    constexpr int RPB = block_of<ROWT>() / ROWT;
    int64_t n;
    constexpr bool whole = VW * sizeof(T) == 16;   // (widths that smaller vectors fill take these)
    const bool fast = whole && a.width == (int64_t)VW * ROWT * VPT && a.weight && a.bias;
    auto k = fast ? ln_fwd<T, VW, ROWT, VPT, whole> : ln_fwd<T, VW, ROWT, VPT, false>;
    constexpr int smem = fwd_ahead<T, VW, ROWT, VPT>() ? Ahead<block_of<ROWT>(), VPT>::BYTES : 0;
    static std::atomic<uint64_t> done[2];
    cudaError_t e;
    if (smem > 48 * 1024 && (e = allow_smem(k, smem, done[fast])) != cudaSuccess) return e;
    if ((e = resident(k, block_of<ROWT>(), smem, (a.rows + RPB - 1) / RPB, &n)) != cudaSuccess) return e;
    k<<<(unsigned)n, block_of<ROWT>(), smem, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t forward(const LayerNormArgs &a, cudaStream_t s) {
    constexpr int VW = vec_of<T>();
    const int64_t w = a.width;
    // few rows: one vector a thread, for the latency; many: four or eight, for the reductions' share
    // of the instructions (32768 x 2048 bf16: two 62 us, four 56 us, eight, for want of registers, 76)
    const bool few = a.rows < 1024;
    if (w % VW == 0) {
        const int64_t nv = w / VW;
        if (few) {
            if (nv <= 32) return fwd<T, VW, 32, 1>(a, s);
            if (nv <= 256) return fwd<T, VW, 256, 1>(a, s);
            if (nv <= 1024) return fwd<T, VW, 1024, 1>(a, s);
        }
        if (nv <= 4) return fwd<T, VW, 4, 1>(a, s);
        if (nv <= 8) return fwd<T, VW, 4, 2>(a, s);
        if (nv <= 16) return fwd<T, VW, 4, 4>(a, s);
        if (nv <= 32) return fwd<T, VW, 8, 4>(a, s);
        if (nv <= 64) return fwd<T, VW, 16, 4>(a, s);
        if (nv <= 128) return fwd<T, VW, 32, 4>(a, s);
        if (nv <= 256) return fwd<T, VW, 64, 4>(a, s);
        if (nv <= 512) return fwd<T, VW, 64, 8>(a, s);
        if (nv <= 1024) return fwd<T, VW, 128, 8>(a, s);
        if (nv <= 4096) return fwd<T, VW, 512, 8>(a, s);
    } else {
        const auto by = [&](auto vw) -> cudaError_t {
            constexpr int V = decltype(vw)::value;
            const int64_t nv = w / V;
            if (nv <= 32) return fwd<T, V, 32, 1>(a, s);
            if (nv <= 128) return fwd<T, V, 32, 4>(a, s);
            if (nv <= 256) return fwd<T, V, 32, 8>(a, s);
            if (nv <= 512) return fwd<T, V, 64, 8>(a, s);
            if (nv <= 1024) return fwd<T, V, 128, 8>(a, s);
            if (nv <= 2048) return fwd<T, V, 256, 8>(a, s);
            if (nv <= 4096) return fwd<T, V, 512, 8>(a, s);
            return fwd<T, V, 1024, 16>(a, s);
        };
        if (w % 2 == 0 && w <= 32768) return by(std::integral_constant<int, 2>{});
        if (w <= 16384) return by(std::integral_constant<int, 1>{});
    }
    ln_fwd_long<T><<<(unsigned)a.rows, 1024, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t add_partials(const LayerNormBwdArgs &a, int64_t n, cudaStream_t s) {
    if (!a.ws) return cudaSuccess;
    return launch_after(ln_sum_partials, dim3((unsigned)((2 * a.width + 31) / 32)), 1024, 0, s, true,
                        (const float *)a.ws, (int)n, a.width, a.dweight, a.dbias);
}

// Partial rows at most, and those of rows wider than the registers of a block, whose columns are many
// blocks already.
int64_t partials(int64_t rows) { return rows < kPartials ? rows : kPartials; }
int64_t partials_long(int64_t rows, int64_t width) {
    const int64_t n = kPartials / ((width + kBlock - 1) / kBlock);
    return n < 1 ? 1 : n < rows ? n : rows;
}
// A row wider than this takes the looping kernels in every type.
constexpr int64_t kWidest = 16384;

template <typename T, int VW, int ROWT, int VPT>
cudaError_t bwd(const LayerNormBwdArgs &a, cudaStream_t s) {
    constexpr int RPB = block_of<ROWT>() / ROWT;
    const int64_t blocks = (a.rows + RPB - 1) / RPB;
    constexpr int ahead = VW * sizeof(T) == 16 ? Ahead<block_of<ROWT>(), 2 * VPT>::BYTES : 0;
    const int sums = RPB > 1 ? RPB * 2 * (int)a.width * (int)sizeof(float) : 0;   // <= 32 KB
    const int smem = ahead > sums ? ahead : sums;
    int64_t n;
    constexpr bool whole = VW * sizeof(T) == 16;
    const bool fast = whole && a.width == (int64_t)VW * ROWT * VPT && a.weight;
    auto k = fast ? ln_bwd<T, VW, ROWT, VPT, whole> : ln_bwd<T, VW, ROWT, VPT, false>;
    static std::atomic<uint64_t> done[2];
    cudaError_t e;
    if (ahead > 48 * 1024 && (e = allow_smem(k, ahead, done[fast])) != cudaSuccess) return e;
    e = resident(k, block_of<ROWT>(), smem, blocks, &n);
    if (e != cudaSuccess) return e;
    if (n > partials(a.rows)) n = partials(a.rows);
    k<<<(unsigned)n, block_of<ROWT>(), smem, s>>>(a);
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
        if (nv <= 8) return bwd<T, VW, 4, 2>(a, s);
        if (nv <= 16) return bwd<T, VW, 8, 2>(a, s);
        if (nv <= 32) return bwd<T, VW, 16, 2>(a, s);
        if (nv <= 64) return bwd<T, VW, 32, 2>(a, s);
        if (nv <= 128) return bwd<T, VW, 64, 2>(a, s);
        if (nv <= 256) return bwd<T, VW, 128, 2>(a, s);
        // sixteen columns a thread: as many as leave its sums in registers in blocks of up to 512 threads
        // (16384 x 2048 fp32: eight 73 us, sixteen 67 us; 32768 x 2048 bf16: sixteen 81 us, 32, for want of
        // registers, 181 us).  Blocks of 1024 have 64 registers a thread, and the widest rows' sums
        // spill there (bf16 588 bytes): the alternative is the looping kernels, which read the rows twice.
        constexpr int V = VW == 4 ? 4 : 2;
        if (nv <= 512) return bwd<T, VW, 512 / V, V>(a, s);
        if (nv <= 1024) return bwd<T, VW, 1024 / V, V>(a, s);
        if (nv <= 2048) return bwd<T, VW, 1024, 2>(a, s);
    } else {
        const auto by = [&](auto vw) -> cudaError_t {
            constexpr int V = decltype(vw)::value;
            const int64_t nv = w / V;
            if (nv <= 32) return bwd<T, V, 32, 1>(a, s);
            if (nv <= 128) return bwd<T, V, 32, 4>(a, s);
            if (nv <= 512) return bwd<T, V, 128, 4>(a, s);
            if (nv <= 1024) return bwd<T, V, 256, 4>(a, s);
            if (nv <= 2048) return bwd<T, V, 512, 4>(a, s);
            if constexpr (V == 1)          // (two elements a load: at most 4096)
                if (nv > 4096) return bwd<T, V, 1024, 8>(a, s);
            return bwd<T, V, 1024, 4>(a, s);
        };
        if (w % 2 == 0 && w <= 8192) return by(std::integral_constant<int, 2>{});
        if (w <= 8192) return by(std::integral_constant<int, 1>{});
    }
    cudaError_t e;
    if (a.ws) {
        const int64_t bx = (w + kBlock - 1) / kBlock, by = partials_long(a.rows, w);
        ln_bwd_sums_long<T><<<dim3((unsigned)bx, (unsigned)by), kBlock, 0, s>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if ((e = add_partials(a, by, s)) != cudaSuccess) return e;
    }
    ln_bwd_long<T><<<(unsigned)a.rows, 1024, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t layer_norm_workspace(int64_t rows, int64_t width) {
    const int64_t n = width > kWidest ? partials_long(rows, width) : partials(rows);
    return (size_t)n * 2 * (size_t)width * sizeof(float);
}

cudaError_t launch_layer_norm(const LayerNormArgs &a, cudaStream_t s) {
    return a.dtype == FW_F32 ? forward<float>(a, s) : forward<__nv_bfloat16>(a, s);
}

cudaError_t launch_layer_norm_backward(const LayerNormBwdArgs &a, cudaStream_t s) {
    return a.dtype == FW_F32 ? backward<float>(a, s) : backward<__nv_bfloat16>(a, s);
}

}  // namespace fw
