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
// its columns' parameters and, in the backward pass, its sums in registers; a block writes one
// partial row of sums and a second kernel adds them in a fixed order.
//
// Measured (one GB300, bf16): 262144 x 128 in 16 groups, rms, gate before: forward 36 us (82 % of the measured copy
// rate), backward 65 us (76 %); 16384 x 2048 with a gate 39 and 79 us, with a scaled residual 45 and 81 us; 4096 x 8192 with a
// gate 47 and 128 us (39 %).  Short rows are bound by instructions, about 28 an element forward (issue slots 76 % busy),
// wide ones by the two barriers of a row's sums.  64 x 2048: 3.5 us of a call of 20.
#include "fw_gated_norm.cuh"

#include <type_traits>

#include "fw_partial.cuh"
#include "fw_rows.cuh"

namespace fw {
namespace {

using namespace fw::rows;

constexpr int kEach = 8;                       // elements of a row a thread

// Blocks of an SM, of R threads a row, forward (80 or 64 registers a thread) and backward (128 or 64).  (Four forward,
// without room for the parameters in registers: 262144 x 128 52 us for 47, 16384 x 2048 69 for 55.)
constexpr int fwd_blocks(int R) { return R < 512 ? 3 : R < 1024 ? 2 : 1; }
constexpr int bwd_blocks(int R) { return R < 512 ? 2 : 1; }
// Elements a thread in the backward pass: where 1024 threads with eight each would have 64 registers, 512 with sixteen, which
// form a row's values again behind its sums instead of holding them (4096 x 8192 with a gate 145 -> 128 us, with a
// scaled residual 178 -> 156).  Single elements are better off with the 1024 (4096 x 8191: 221 us for 291).
constexpr int bwd_each(int R, int V) { return R < 1024 || V == 1 ? kEach : 2 * kEach; }
template <int R> constexpr int block_of() { return R < 256 ? 256 : R; }

// All but the newest `left` groups of copies have landed.
__device__ __forceinline__ void copies_wait(int left) {
    if (left == 0) fw::rows::copies_wait<0>();
    else if (left == 1) fw::rows::copies_wait<1>();
    else fw::rows::copies_wait<2>();
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
        if constexpr (NW <= 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                z[i] = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) z[i] += red[i * ALL + first + w];
            }
        } else {                               // (a warp reads them once, not each thread all of them)
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = red[i * ALL + first + (threadIdx.x & (NW - 1))];
#pragma unroll
            for (int o = NW / 2; o; o >>= 1)
#pragma unroll
                for (int i = 0; i < N; ++i) z[i] += __shfl_xor_sync(~0u, z[i], o);
        }
    }
}

// All threads of a row (and others) are here, and see what the others have written to shared memory.
template <int R> __device__ __forceinline__ void row_barrier() {
    if constexpr (R <= 32) __syncwarp();
    else __syncthreads();
}

// The columns of a thread, in K parts of E elements that are worked on at once, and the rows that it works on, up to
// `stages` of them ahead in shared memory, N arrays each.  V elements a load, in slots of the thread's own; where V is
// one, the two of a part lie R columns apart and the second may be behind the row's end.  bf16 rows of an odd width begin
// at any multiple of two bytes, which is no copy's size: the row's threads copy all 16-byte units that the row touches, for
// one another.  (Outputs may be inputs as well: what a row reads has landed before any of it is written, and of its
// neighbours' elements in its first and last unit nothing is used.  10000 x 1023 with a gate and a residual, forward
// and backward: 25 and 55 us; read from memory when asked for, 57 and 217.)
template <typename T, int V, int R, int N, int C = kEach> struct Ahead {
    static constexpr int E = V > 1 ? V : 2, K = C / E, BYTES = V * (int)sizeof(T), ROW = R * C * (int)sizeof(T);
    static constexpr bool SHARED = BYTES == 2;
    static constexpr int PLACE = block_of<R>() / R * (ROW + (SHARED ? 16 : 0));   // bytes of an array's rows of a block
    const void *src[N];
    char *slots;
    int stages, width, lane;
    int64_t at;                                // of the row at hand
    int stage = 0;

    __device__ __forceinline__ int column(int k, int e = 0) const {
        return V > 1 ? (k * R + lane) * V + e : (k * E + e) * R + lane;
    }
    __device__ __forceinline__ bool has(int k, int e = 0) const { return column(k, e) < width; }
    __device__ __forceinline__ char *array_at(int s, int a) const { return slots + (s * N + a) * PLACE; }
    __device__ __forceinline__ Raw<T, V> *slot(int s, int a, int i) const {
        return reinterpret_cast<Raw<T, V> *>(array_at(s, a)) + i * block_of<R>() + threadIdx.x;
    }
    __device__ __forceinline__ char *row_slot(int s, int a) const {
        return array_at(s, a) + threadIdx.x / R * (ROW + 16);
    }
    // Copies of a row into a stage, a group of them whether there is a row or not.
    __device__ __forceinline__ void fetch(int s, bool live, int64_t row_at) {
        if (live)
#pragma unroll
            for (int a = 0; a < N; ++a) {
                if (!src[a]) continue;
                if constexpr (SHARED) {
                    const int64_t first = row_at * (int)sizeof(T) & ~(int64_t)15;
                    const int bytes = (int)(row_at * (int)sizeof(T) - first) + width * (int)sizeof(T);
                    const char *const from = static_cast<const char *>(src[a]) + first;
                    char *const to = row_slot(s, a);
#pragma unroll
                    for (int i = 0; i <= ROW / 16 / R; ++i) {
                        const int c = (i * R + lane) * 16;
                        if (c < bytes) copy_async_part(to + c, from + c, min(bytes - c, 16));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < C / V; ++i) {
                        const int c = V > 1 ? column(i) : column(i / E, i % E);
                        if (c < width) copy_async<BYTES>(slot(s, a, i), static_cast<const T *>(src[a]) + row_at + c);
                    }
                }
            }
        copies_commit();
    }
    __device__ __forceinline__ Chan<E> get(int a, int k) const {
        if constexpr (V > 1) return widen(*slot(stage, a, k));
        else {
            float x[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (has(k, e)) {
                    if constexpr (SHARED) x[e] = to_f32(reinterpret_cast<const T *>(row_slot(stage, a))[(at & 7) + column(k, e)]);
                    else x[e] = to_f32(slot(stage, a, k * E + e)->v);
                }
            return {{pair(x[0], x[1])}};
        }
    }
    __device__ __forceinline__ void put(void *p, int k, const Chan<E> &x) const {
        T *const to = static_cast<T *>(p) + at;
        if constexpr (V > 1) store<T, V>(to + column(k), x);
        else
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (has(k, e)) to[column(k, e)] = from_f32<T>(element(x, e));
    }
    // A parameter's columns; `other` where it is not given.
    __device__ __forceinline__ Chan<E> of(const float *p, int k, float other) const {
        if constexpr (V > 1) return param<V>(p, column(k), other);
        else {
            float x[2] = {other, other};
            if (p)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (has(k, e)) x[e] = p[column(k, e)];
            return {{pair(x[0], x[1])}};
        }
    }
};

// Every step-th row of group blockIdx.y from the m-th on, without a division or a product a row: m = outer inner + i
// is row (outer groups + group) inner + i.
struct Steps {                                 // from one to the next, and what a turn of `inner` adds
    uint32_t m, i, row, turn;
    int64_t at, turn_at;
    __device__ __forceinline__ Steps(const GatedIn &in, uint32_t step)
        : m(step), i(step % (uint32_t)in.inner),
          row(step / (uint32_t)in.inner * (uint32_t)in.groups * (uint32_t)in.inner + step % (uint32_t)in.inner),
          turn(((uint32_t)in.groups - 1) * (uint32_t)in.inner), at((int64_t)row * in.width), turn_at((int64_t)turn * in.width) {}
};
struct Walk {
    uint32_t m, i, row;
    int64_t at;                                // of the row's first element
    __device__ __forceinline__ Walk(const GatedIn &in, uint32_t first)
        : m(first), i(first % (uint32_t)in.inner),
          row((first / (uint32_t)in.inner * (uint32_t)in.groups + blockIdx.y) * (uint32_t)in.inner + first % (uint32_t)in.inner),
          at((int64_t)row * in.width) {}
    __device__ __forceinline__ void next(const GatedIn &in, const Steps &s) {
        m += s.m;
        i += s.i;
        row += s.row;
        at += s.at;
        if (i >= (uint32_t)in.inner) {
            i -= (uint32_t)in.inner;
            row += s.turn;
            at += s.turn_at;
        }
    }
};

// Walks the rows of a block's share of group blockIdx.y: work(live, row, next row or -1) with the row's
// data in `ahead`.
template <typename T, int V, int R, int N, int C, typename F>
__device__ __forceinline__ void over_rows(Ahead<T, V, R, N, C> &ahead, const GatedIn &in, uint32_t group_rows, F work) {
    constexpr int RPB = block_of<R>() / R;
    const uint32_t step = gridDim.x * RPB;
    const Steps steps(in, step);
    Walk at(in, blockIdx.x * RPB + threadIdx.x / R), ask = at;
    auto fetch = [&](int s) {
        ahead.fetch(s, ask.m < group_rows, ask.at);
        ask.next(in, steps);
    };
    // A stage of the thread's own is filled again as soon as it is read; one that the row's threads share, when all of them
    // are at the next row (with one stage: when all have read it).
    constexpr bool SHARED = Ahead<T, V, R, N, C>::SHARED;
    const int first = ahead.stages - SHARED;
    for (int s = 0; s < first; ++s) fetch(s);
    for (uint32_t m0 = blockIdx.x * RPB; m0 < group_rows; m0 += step) {
        const bool live = at.m < group_rows;
        const uint32_t row = at.row;
        ahead.at = at.at;
        at.next(in, steps);
        if constexpr (SHARED) {
            if (first == 0) {
                row_barrier<R>();
                fetch(0);
            }
            copies_wait(first == 0 ? 0 : first - 1);
            row_barrier<R>();
            if (first > 0) fetch(ahead.stage == 0 ? first : ahead.stage - 1);
        } else {
            copies_wait(first - 1);
        }
        work(live, row, at.m < group_rows ? (int64_t)at.row : (int64_t)-1);
        if constexpr (!SHARED) fetch(ahead.stage);
        if (++ahead.stage == ahead.stages) ahead.stage = 0;
    }
    copies_wait(0);
}

template <typename T, int V, int R>
__global__ void __launch_bounds__(block_of<R>(), fwd_blocks(R)) gated_kernel(GatedArgs a, uint32_t group_rows, int stages) {
    using Rows = Ahead<T, V, R, 3>;
    constexpr int K = Rows::K, E = Rows::E, BLOCK = block_of<R>();
    extern __shared__ uint4 slots[];
    __shared__ float red[R > 32 ? BLOCK / 32 : 1];
    const GatedIn &in = a.in;
    Rows rows{{in.x, in.gate, in.residual}, reinterpret_cast<char *>(slots), stages, in.width, (int)(threadIdx.x % R), 0};
    const float inv = 1.f / (float)in.width;
    const int64_t pat = (int64_t)blockIdx.y * in.width;
    const float *const weight = in.weight ? in.weight + pat : nullptr, *const bias = in.bias ? in.bias + pat : nullptr,
                *const scale = in.scale ? in.scale + pat : nullptr;
    Chan<E> w[K], b[K], f[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (rows.has(k)) {
            w[k] = rows.of(weight, k, 1.f);
            b[k] = rows.of(bias, k, 0.f);
            f[k] = rows.of(scale, k, 1.f);
        }
    over_rows(rows, in, group_rows, [&](bool live, uint32_t row, int64_t) {
        Chan<E> s[K], part = none<E>();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            s[k] = none<E>();
            if (live && rows.has(k)) {
                s[k] = rows.get(0, k);
                if (in.residual) s[k] = fma_n(f[k], rows.get(2, k), s[k]);
                if (a.total) rows.put(a.total, k, s[k]);
                if (in.gate && !in.gate_after) {
                    const Chan<E> z = rows.get(1, k);
                    s[k] = mul_n(s[k], mul_n(z, sigmoid_n<T>(z)));
                }
                part = add_n(part, s[k]);
            }
        }
        float sum[1] = {0.f}, mean = 0.f;
        if (!in.rms) {
            sum[0] = total(part);
            row_sums<R>(sum, red);
            mean = sum[0] * inv;
        }
        part = none<E>();
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (rows.has(k)) {
                if (!in.rms) {
                    s[k] = add_n(s[k], all<E>(-mean));
                    if (V == 1 && !rows.has(k, 1)) s[k].p[0] = pair(halves(s[k].p[0]).x, 0.f);
                }
                part = fma_n(s[k], s[k], part);
            }
        sum[0] = total(part);
        row_sums<R>(sum, red);
        const float rstd = rsqrtf(fmaf(sum[0], inv, in.eps));
        if (!live) return;
        if (rows.lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!rows.has(k)) continue;
            s[k] = fma_n(mul_n(s[k], all<E>(rstd)), w[k], b[k]);
            if (in.gate && in.gate_after) {
                const Chan<E> z = rows.get(1, k);
                s[k] = mul_n(s[k], mul_n(z, sigmoid_n<T>(z)));
            }
            rows.put(a.y, k, s[k]);
        }
    });
}

template <typename T, int V, int R, int C>
__global__ void __launch_bounds__(block_of<R>(), bwd_blocks(R)) gated_bwd_kernel(GatedBwdArgs a, uint32_t group_rows, int stages) {
    using Rows = Ahead<T, V, R, 5, C>;
    constexpr int K = Rows::K, E = Rows::E, BLOCK = block_of<R>(), RPB = BLOCK / R;
    extern __shared__ uint4 slots[];
    __shared__ float red[R > 32 ? 2 * BLOCK / 32 : 1];
    const GatedIn &in = a.in;
    Rows rows{{in.x, a.dy, in.gate, in.residual, a.dtotal}, reinterpret_cast<char *>(slots), stages, in.width,
              (int)(threadIdx.x % R), 0};
    const int width = in.width;
    const float inv = 1.f / (float)width;
    const int64_t pat = (int64_t)blockIdx.y * width;
    const float *const weight = in.weight ? in.weight + pat : nullptr, *const bias = in.bias ? in.bias + pat : nullptr,
                *const scale = in.scale ? in.scale + pat : nullptr;
    Chan<E> sums[3][K];                        // of dweight, dbias, dscale
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k) sums[i][k] = none<E>();
    float next_mean = 0.f, next_rstd = 0.f;    // of the next row
    {
        const Walk first(in, blockIdx.x * RPB + threadIdx.x / R);
        if (first.m < group_rows) {
            if (!in.rms) next_mean = a.mean[first.row];
            next_rstd = a.rstd[first.row];
        }
    }
    // The columns' weights stay in registers, and their scales too but for eight elements a load, for which there is no room.
    constexpr bool HOLD = C == kEach, HOLD_SCALE = HOLD && R < 1024 && V < 8;
    Chan<E> w[K], f[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (rows.has(k)) {
            if constexpr (HOLD) w[k] = rows.of(weight, k, 1.f);
            if constexpr (HOLD_SCALE) f[k] = rows.of(scale, k, 1.f);
        }
    auto weight_of = [&](int k) {
        if constexpr (HOLD) return w[k];
        else return rows.of(weight, k, 1.f);
    };
    auto scale_of = [&](int k) {
        if constexpr (HOLD_SCALE) return f[k];
        else return rows.of(scale, k, 1.f);
    };
    over_rows(rows, in, group_rows, [&](bool live, uint32_t, int64_t next) {
        const float mean = next_mean, rstd = next_rstd;
        if (next >= 0) {
            if (!in.rms) next_mean = a.mean[next];
            next_rstd = a.rstd[next];
        }
        auto sum_of = [&](int k) -> Chan<E> {  // u
            const Chan<E> x = rows.get(0, k);
            return in.residual ? fma_n(scale_of(k), rows.get(3, k), x) : x;
        };
        // n = norm(s), g, and the sigmoid of the gate
        auto part_of = [&](int k, Chan<E> &n, Chan<E> &g, Chan<E> &sg) {
            n = sum_of(k);
            g = mul_n(rows.get(1, k), weight_of(k));
            if (in.gate) {
                const Chan<E> z = rows.get(2, k);
                sg = sigmoid_n<T>(z);
                const Chan<E> act = mul_n(z, sg);
                if (in.gate_after) g = mul_n(g, act);
                else n = mul_n(n, act);
            }
            if (!in.rms) n = add_n(n, all<E>(-mean));
            n = mul_n(n, all<E>(rstd));
        };
        Chan<E> n[K], g[K], sg[K];
        Chan<E> sum_g = none<E>(), sum_gn = none<E>();
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (live && rows.has(k)) {
                part_of(k, n[k], g[k], sg[k]);
                sum_g = add_n(sum_g, g[k]);
                sum_gn = fma_n(g[k], n[k], sum_gn);
            }
        float sum[2] = {total(sum_g), total(sum_gn)};
        row_sums<R>(sum, red);
        if (!live) return;
        const float mg = in.rms ? 0.f : -sum[0] * inv * rstd, mgn = -sum[1] * inv * rstd;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!rows.has(k)) continue;
            if constexpr (!HOLD) part_of(k, n[k], g[k], sg[k]);
            // rstd (g - mean(g) - n mean(g n))
            Chan<E> d = fma_n(n[k], all<E>(mgn), fma_n(g[k], all<E>(rstd), all<E>(mg)));
            Chan<E> dy = rows.get(1, k);
            if (in.gate) {
                const Chan<E> z = rows.get(2, k), act = mul_n(z, sg[k]);
                Chan<E> dz;
                if (in.gate_after) dz = mul_n(dy, fma_n(n[k], weight_of(k), rows.of(bias, k, 0.f)));
                else dz = mul_n(d, sum_of(k));
                dz = mul_n(dz, silu_slope(z, sg[k]));
                if (in.gate_after) dy = mul_n(dy, act);        // of the norm's output
                else d = mul_n(d, act);
                if (a.dgate) rows.put(a.dgate, k, dz);
            }
            if (a.dtotal) d = add_n(d, rows.get(4, k));
            if (a.dx) rows.put(a.dx, k, d);
            sums[0][k] = fma_n(dy, n[k], sums[0][k]);
            sums[1][k] = add_n(sums[1][k], dy);
            if (in.residual) {
                sums[2][k] = fma_n(rows.get(3, k), d, sums[2][k]);
                if (a.dresidual) rows.put(a.dresidual, k, mul_n(d, scale_of(k)));
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
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (rows.has(k, e)) out[i * width + rows.column(k, e)] = element(sums[i][k], e);
        } else {
            __syncthreads();                   // (the slots are free, or the sums before read)
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < E; ++e) part[(threadIdx.x / R) * (R * C) + rows.column(k, e)] = element(sums[i][k], e);
            __syncthreads();
            for (int c = threadIdx.x; c < width; c += BLOCK) {
                float z = 0.f;
#pragma unroll 4
                for (int p = 0; p < RPB; ++p) z += part[p * (R * C) + c];
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

// Blocks that share the rows of a group: what the SMs hold at once, and no more than there are rows for.
uint32_t slices_of(int64_t rows, int64_t groups, int R, int blocks) {
    const int64_t group_rows = rows / groups, each = R < 256 ? 256 / R : 1, most = (group_rows + each - 1) / each;
    const int64_t s = (int64_t)kSMs * blocks / groups;
    return (uint32_t)(s < 1 ? 1 : s > most ? most : s);
}

// Rows ahead, of a block's `bytes` each, that leave room for the blocks of an SM.
int stages_of(int bytes, int blocks) {
    const int room = 216 * 1024 / blocks;
    return bytes * 3 <= room ? 3 : bytes * 2 <= room ? 2 : 1;
}

template <typename T, int V, int R> cudaError_t run(const GatedArgs &a, cudaStream_t s) {
    constexpr int ROW = 3 * Ahead<T, V, R, 3>::PLACE;
    const int stages = stages_of(ROW, fwd_blocks(R)), smem = stages * ROW;
    auto k = gated_kernel<T, V, R>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(k, smem, done);
    if (e != cudaSuccess) return e;
    k<<<dim3(slices_of(a.in.rows, a.in.groups, R, fwd_blocks(R)), a.in.groups), block_of<R>(), smem, s>>>(
        a, (uint32_t)(a.in.rows / a.in.groups), stages);
    return cudaGetLastError();
}

template <typename T, int V, int R0> cudaError_t run(const GatedBwdArgs &a, cudaStream_t s) {
    constexpr int C = bwd_each(R0, V), R = R0 * kEach / C;
    const GatedIn &in = a.in;
    const uint32_t slices = slices_of(in.rows, in.groups, R, bwd_blocks(R));
    constexpr int ROW = 5 * Ahead<T, V, R, 5, C>::PLACE;
    const int stages = stages_of(ROW, bwd_blocks(R)), smem = stages * ROW;
    auto k = gated_bwd_kernel<T, V, R, C>;
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
        // (1024 threads have 64 registers each, and 512 with sixteen elements 128: eight at a time are more than they hold)
        return run<T, V == 8 ? 4 : V, 1024>(a, s);
    }
}

// Elements a load: 16 bytes where rows are whole multiples of it, else two (even widths), else one.
template <typename A> cudaError_t by_type(const A &a, cudaStream_t s) {
    const int w = a.in.width;
    if (a.in.dtype == FW_F32)
        return w % 4 == 0 ? by_width<float, 4>(a, s) : w % 2 == 0 ? by_width<float, 2>(a, s) : by_width<float, 1>(a, s);
    // (Backwards with a residual eight bytes, which leaves room for the scales in registers: 262144 x 128 70 us for 73,
    // 65536 x 512 77 for 95, 16384 x 2048 80 for 98, 8192 x 4096 87 for 103; with a gate too 113 for 123 of 16384 x 2048, but
    // 100 for 98 of 262144 x 128.  Without a residual 81 for 66 of 262144 x 128, 101 for 89 of 8192 x 4096.)
    if (w % 8 == 0)
        return std::is_same_v<A, GatedBwdArgs> && a.in.residual ? by_width<__nv_bfloat16, 4>(a, s)
                                                               : by_width<__nv_bfloat16, 8>(a, s);
    return w % 2 == 0 ? by_width<__nv_bfloat16, 2>(a, s) : by_width<__nv_bfloat16, 1>(a, s);
}

}  // namespace

size_t gated_norm_workspace(int64_t rows, int64_t width, int64_t groups) {
    const int R = threads_of((int)width);
    return (size_t)slices_of(rows, groups, R, bwd_blocks(R)) * groups * 3 * width * sizeof(float);
}

cudaError_t launch_gated_norm(const GatedArgs &a, cudaStream_t s) { return by_type(a, s); }
cudaError_t launch_gated_norm_backward(const GatedBwdArgs &a, cudaStream_t s) { return by_type(a, s); }

}  // namespace fw
