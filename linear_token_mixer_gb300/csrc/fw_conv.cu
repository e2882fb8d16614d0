// fw_conv.cu -- short causal convolution of every channel, W = 2 .. 8 taps, before a mixer:
//     a_t = b + sum_w weight[w] x_{t-W+1+w},   y_t = a_t or a_t / (1 + exp(-a_t)),
// its gradients and its form for one token.  Rows before the first come from a carried state.
//
// All three are bound by their rows' bytes.  A thread holds V channels (16 bytes of a row; 8 in the
// backward pass, which keeps five such rows' worth of registers) and walks a strip of
// tokens with the last W - 1 rows in registers, so that each row is read once but for the W - 1 rows
// before a strip.  The next rows are on their way into shared memory meanwhile (cp.async, each thread into slots of its
// own), three turns of W ahead.
// The backward pass forms a_t again, walks W - 1 tokens past its strip, and writes
//     da_t = dy_t act'(a_t),   dx_{t-W+1} = sum_w weight[w] da_{t-w}
// as t passes; dweight[w] += da_t x_{t-W+1+w} and dbias += da_t stay in registers over all strips
// of a thread, are added up in a block, and a second kernel adds the blocks' in a fixed order.
//
// Measured (one GB300, W = 4 with silu): B8 H16 T2048 d = 128 bf16 forward 23.3 us, 85 % of the measured copy rate;
// backward 44 us, 67 %, with neither the issue slots (54 % busy) nor DRAM (51 %) full: 23 instructions an element (the
// taps three times over, silu and its slope) in 16 warps an SM, whose registers hold taps, sums and windows, and which wait
// for their own results.  fp32: B8 H8 T2048 d = 128 20 and 37 us (99 and 80 %); B4 H8 T1023 d = 65 W = 3 5.5 and 10 us, of
// which launches are most.  One token of B256 H32 d = 128: 6 us behind a call of 13.
#include <type_traits>

#include "fw_conv.cuh"
#include "fw_partial.cuh"
#include "fw_rows.cuh"

namespace fw {
namespace {

using namespace rows;

constexpr int kBlock = 256;
constexpr int kStrip = 256;                   // most tokens of a strip
constexpr int kStripMin = 8;                  // no fewer: only the first strip reads the state (W - 1 <= 7)

// The taps of V channels; element (channel, tap) at w[channel * W + tap].
template <int W, int V> __device__ __forceinline__ void load_taps(Chan<V> (&w)[W], const float *p) {
    float f[V * W];
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V * W; i += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(p + i);
            f[i] = q.x; f[i + 1] = q.y; f[i + 2] = q.z; f[i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * W; ++i) f[i] = p[i];
    }
#pragma unroll
    for (int t = 0; t < W; ++t)
#pragma unroll
        for (int i = 0; i < Chan<V>::N; ++i) w[t].p[i] = pair(f[2 * i * W + t], V > 1 ? f[(2 * i + 1) * W + t] : 0.f);
}
// Rows `t` of a chain, or of the state before it (t < 0); zero without a state.
template <typename T, int V>
__device__ __forceinline__ Chan<V> row_at(const T *x, const T *state, int64_t t, int W, int d) {
    if (t >= 0) return widen(load<T, V>(x + t * d));
    return state ? widen(load<T, V>(state + (t + W - 1) * d)) : none<V>();
}

// The next rows of a strip in shared memory: kStages turns of W rows of N arrays, each thread in slots of its
// own.  (Two bytes are no copy's size: such rows are read from memory when asked for.)
constexpr int kStages = 3;
template <typename T, int V, int W, int N> struct Stage {
    static constexpr int BYTES = V * (int)sizeof(T);
    static constexpr bool COPY = BYTES >= 4;
    uint4 *slots;
    int put = 0, at = 0;
    static constexpr int bytes() { return COPY ? kStages * N * W * kBlock * BYTES : 0; }
    __device__ __forceinline__ Raw<T, V> *slot(int s, int a, int u) const {
        return reinterpret_cast<Raw<T, V> *>(slots) + ((s * N + a) * W + u) * kBlock + threadIdx.x;
    }
    // Rows 0 .. left - 1 of those from `p` on into array a of the stage that is put next; the last array moves on.
    __device__ __forceinline__ void fetch(int a, const T *p, int d, int left) {
        if constexpr (COPY) {
#pragma unroll
            for (int u = 0; u < W; ++u)
                if (u < left) copy_async<BYTES>(slot(put, a, u), p + u * d);
            if (a == N - 1 && ++put == kStages) put = 0;
        }
    }
    __device__ __forceinline__ Chan<V> get(int a, int u, const T *p) const {
        if constexpr (COPY) return widen(*slot(at, a, u));
        else return widen(load<T, V>(p));
    }
    __device__ __forceinline__ void next() {
        if (++at == kStages) at = 0;
    }
};

template <typename T, int V, int W>
__global__ void __launch_bounds__(kBlock, W * V * sizeof(T) <= 64 ? 2 : 1) conv_kernel(ConvArgs a, uint32_t strip, uint32_t strips, uint32_t cols) {
    extern __shared__ uint4 slots[];
    const uint32_t id = blockIdx.x * (uint32_t)kBlock + threadIdx.x;
    const uint32_t s = id / cols, cv = id % cols, st = s % strips;
    const int64_t chain = s / strips;
    if (chain >= a.n_chains) return;
    const int d = a.d, h = (int)(chain % a.H), c0 = (int)cv * V;
    const int n = (int)chain_len(a.lens, chain, a.H, a.T), T_ = (int)a.T;
    const int t0 = (int)(st * strip), t1 = t0 + (int)strip < T_ ? t0 + (int)strip : T_;
    const T *const x = static_cast<const T *>(a.x) + chain * a.T * d + c0;
    const T *const state = a.state ? static_cast<const T *>(a.state) + chain * (W - 1) * d + c0 : nullptr;
    T *const y = static_cast<T *>(a.y) + chain * a.T * d + c0;
    const int end = t1 < n ? t1 : n;
    Chan<V> win[W];                           // the row at t0 + i, and those before it, at i mod W
    if (t0 < end || st == 0) {
#pragma unroll
        for (int i = 1; i < W; ++i) win[i] = row_at<T, V>(x, state, t0 + i - W, W, d);
    }
    if (st == 0 && a.state_out) {             // the last W - 1 of the state's rows and the chain's
        T *const so = static_cast<T *>(a.state_out) + chain * (W - 1) * d + c0;
#pragma unroll
        for (int i = 1; i < W; ++i) {         // (a row of the state is already in win: state_out may be state)
            const int t = n + i - W;
            Chan<V> r = none<V>();
            if (t >= 0) r = widen(load<T, V>(x + (int64_t)t * d));
            else
#pragma unroll
                for (int j = 1; j < W; ++j)
                    if (j == t + W) r = win[j];
            store<T, V>(so + (int64_t)(i - 1) * d, r);
        }
    }
    if (t0 < end) {
        Chan<V> w[W];
        load_taps<W, V>(w, a.weight + ((int64_t)h * d + c0) * W);
        const Chan<V> bias = param<V>(a.bias, (int64_t)h * d + c0, 0.f);
        Stage<T, V, W, 1> in{slots};
        T *to = y + (int64_t)t0 * d;
        int ask = t0;                          // of the rows to fetch
        const T *from = x + (int64_t)t0 * d;
        auto fetch = [&]() {
            in.fetch(0, from, d, end - ask);
            copies_commit();
            from += W * d;
            ask += W;
        };
        auto turn = [&](int t, auto whole) {   // W tokens from t on
#pragma unroll
            for (int u = 0; u < W; ++u) {
                if (!whole.value && t + u >= end) break;
                win[u] = in.get(0, u, x + (int64_t)(t + u) * d);
                Chan<V> r = bias;
#pragma unroll
                for (int i = 0; i < W; ++i) r = fma_n(w[i], win[(u + 1 + i) % W], r);
                if (a.silu) r = mul_n(r, sigmoid_n<T>(r));
                store<T, V>(to + u * d, r);
            }
        };
#pragma unroll
        for (int i = 0; i < kStages; ++i) fetch();
#pragma unroll 1
        for (int t = t0; t < end; t += W, to += W * d) {
            copies_wait<kStages - 1>();
            if (t + W <= end) turn(t, std::true_type{});
            else turn(t, std::false_type{});
            fetch();
            in.next();
        }
        copies_wait<0>();
    }
    if (a.zero_rest)
        for (int t = t0 > n ? t0 : n; t < t1; ++t) store<T, V>(y + (int64_t)t * d, none<V>());
}

// `lanes` (a power of two) of a warp hold the columns of a row, the 32 / lanes parts of it take
// strips of their own.  blockIdx.y: a head's group of columns; blockIdx.x: a share of the head's strips.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kBlock, V > 1 && W > 4 ? 1 : 2)
conv_bwd_kernel(ConvBwdArgs a, uint32_t strip, uint32_t strips, int lanes, uint32_t groups) {
    constexpr int NW = kBlock / 32;
    extern __shared__ uint4 slots[];
    __shared__ float part[NW][32][V * (W + 1)];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cl = lane & (lanes - 1);
    const int h = (int)(blockIdx.y / groups), d = a.d;
    const int c0 = ((int)(blockIdx.y % groups) * lanes + cl) * V;
    const bool mine = c0 < d;
    Chan<V> w[W], dw[W], db = none<V>();
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = dw[i] = none<V>();
    Chan<V> bias = none<V>();
    if (mine) {
        load_taps<W, V>(w, a.weight + ((int64_t)h * d + c0) * W);
        bias = param<V>(a.bias, (int64_t)h * d + c0, 0.f);
    }
    const uint32_t parts = 32u / lanes, step = gridDim.x * NW * parts;
    const uint32_t total = (uint32_t)a.B * strips;
    for (uint32_t m = (blockIdx.x * NW + warp) * parts + lane / lanes; mine && m < total; m += step) {
        const uint32_t b = m / strips, st = m % strips;
        const int64_t chain = (int64_t)b * a.H + h;
        const int n = (int)chain_len(a.lens, chain, a.H, a.T), T_ = (int)a.T;
        const int t0 = (int)(st * strip), t1 = t0 + (int)strip < T_ ? t0 + (int)strip : T_;
        const int end = t1 < n ? t1 : n;
        const int64_t at = chain * a.T * d + c0, sat = chain * (W - 1) * d + c0;
        const T *const x = static_cast<const T *>(a.x) + at, *const dy = static_cast<const T *>(a.dy) + at;
        const T *const state = a.state ? static_cast<const T *>(a.state) + sat : nullptr;
        const T *const dso = a.dstate_out ? static_cast<const T *>(a.dstate_out) + sat : nullptr;
        T *const dx = static_cast<T *>(a.dx) + at, *const ds = a.dstate ? static_cast<T *>(a.dstate) + sat : nullptr;
        if (a.zero_rest)
            for (int t = t0 > n ? t0 : n; t < t1; ++t) store<T, V>(dx + (int64_t)t * d, none<V>());
        if (!(t0 < end || (st == 0 && ds))) continue;
        Chan<V> win[W], da[W];                    // the row at t0 + i, and those before it, at i mod W
#pragma unroll
        for (int i = 1; i < W; ++i) {
            win[i] = row_at<T, V>(x, state, t0 + i - W, W, d);
            da[i] = none<V>();
        }
        Stage<T, V, W, 2> in{slots};
        const T *fx = x + (int64_t)t0 * d, *fy = dy + (int64_t)t0 * d;   // of the rows to fetch
        T *to = dx + (int64_t)(t0 - (W - 1)) * d;                        // where the next row leaves to
        int ask = t0;
        const int stop = (end > t0 ? end : t0) + W - 1;                  // rows up to end - 1 leave at t = end + W - 2
        auto fetch = [&]() {
            const int left = (n < stop ? n : stop) - ask;
            in.fetch(0, fx, d, left);
            in.fetch(1, fy, d, left);
            copies_commit();
            fx += W * d;
            fy += W * d;
            ask += W;
        };
        // W tokens from t on; `whole`: all of them are the strip's, and so are the rows that leave, none of which goes
        // on into the state behind the chain (those leave with t >= n)
        auto turn = [&](int t, auto whole) {
            constexpr bool ALL = decltype(whole)::value;
#pragma unroll
            for (int u = 0; u < W; ++u) {
                if (!ALL && t + u >= stop) break;
                const bool on = ALL || t + u < n;
                win[u] = on ? in.get(0, u, x + (int64_t)(t + u) * d) : none<V>();
                da[u] = on ? in.get(1, u, dy + (int64_t)(t + u) * d) : none<V>();
                if (a.silu) {
                    Chan<V> r = bias;
#pragma unroll
                    for (int i = 0; i < W; ++i) r = fma_n(w[i], win[(u + 1 + i) % W], r);
                    const Chan<V> slope = silu_slope(r, sigmoid_n<T>(r));
                    if (on) da[u] = mul_n(da[u], slope);
                }
                if (ALL || t + u < end) {
#pragma unroll
                    for (int i = 0; i < W; ++i) dw[i] = fma_n(da[u], win[(u + 1 + i) % W], dw[i]);
                    db = add_n(db, da[u]);
                }
                const int s = t + u - (W - 1);                   // the row that leaves
                Chan<V> r = mul_n(w[0], da[u]);
#pragma unroll
                for (int i = 1; i < W; ++i) r = fma_n(w[i], da[(u - i + W) % W], r);
                if (ALL) {
                    store<T, V>(to + u * d, r);
                    continue;
                }
                const int q = s - n + W - 1;                     // its place in the state behind the chain
                if (dso && q >= 0 && q < W - 1 && s < end) r = add_n(r, widen(load<T, V>(dso + q * d)));
                if (s >= t0) {
                    if (s < end) store<T, V>(to + u * d, r);
                } else if (st == 0 && ds && s < 0) {
                    store<T, V>(ds + (s + W - 1) * d, r);
                }
            }
        };
#pragma unroll
        for (int i = 0; i < kStages; ++i) fetch();
#pragma unroll 1
        for (int t = t0; t < stop; t += W, to += W * d) {
            copies_wait<kStages - 1>();
            if (t >= t0 + W - 1 && t + W <= end) turn(t, std::true_type{});
            else turn(t, std::false_type{});
            fetch();
            in.next();
        }
        copies_wait<0>();
    }
    let_next_grid_start();
    if (!a.ws) return;
    // the parts of the warp, then the warps of the block
#pragma unroll
    for (int i = 0; i <= W; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float z = element(i < W ? dw[i] : db, e);
            for (int o = lanes; o < 32; o <<= 1) z += __shfl_xor_sync(~0u, z, o);
            part[warp][lane][e * (W + 1) + i] = z;
        }
    __syncthreads();
    const int used = lanes * V * (W + 1);
    for (int i = threadIdx.x; i < used; i += kBlock) {
        const int l = i / (V * (W + 1)), e = i % (V * (W + 1));
        float z = 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) z += part[k][l][e];
        const int c = ((int)(blockIdx.y % groups) * lanes + l) * V + e / (W + 1);
        if (c < d) a.ws[((int64_t)blockIdx.x * a.H + h) * d * (W + 1) + (int64_t)c * (W + 1) + e % (W + 1)] = z;
    }
}

// The sums of the blocks, in their order.
__global__ void __launch_bounds__(kSumCols * kSumShares)
conv_sum_kernel(const float *ws, int slices, int64_t count, int W, float *dweight, float *dbias) {
    wait_previous_grid();
    sum_slices(ws, slices, count, [&](int64_t i, float z) {
        const int64_t c = i / (W + 1);
        const int e = (int)(i % (W + 1));
        if (e == W) {
            if (dbias) dbias[c] = z;
        } else if (dweight) {
            dweight[c * W + e] = z;
        }
    });
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kBlock) conv_step_kernel(ConvStepArgs a, uint32_t cols) {
    const uint32_t id = blockIdx.x * (uint32_t)kBlock + threadIdx.x;
    const int64_t chain = id / cols;
    if (chain >= a.n_states) return;
    const int d = a.d, h = (int)(chain % a.H), c0 = (int)(id % cols) * V;
    T *const state = static_cast<T *>(a.state) + chain * (W - 1) * d + c0;
    Raw<T, V> row[W];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) row[i] = load<T, V>(state + (int64_t)i * d);
    row[W - 1] = load<T, V>(static_cast<const T *>(a.x) + chain * d + c0);
    Chan<V> w[W];
    load_taps<W, V>(w, a.weight + ((int64_t)h * d + c0) * W);
    Chan<V> r = param<V>(a.bias, (int64_t)h * d + c0, 0.f);
#pragma unroll
    for (int i = 0; i < W; ++i) r = fma_n(w[i], widen(row[i]), r);
    if (a.silu) r = mul_n(r, sigmoid_n<T>(r));
    store<T, V>(static_cast<T *>(a.y) + chain * d + c0, r);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) *reinterpret_cast<Raw<T, V> *>(state + (int64_t)i * d) = row[i + 1];
}

// Tokens of a strip, of chains that are to be cut in about `parts` each: at least kStripMin, at most kStrip (padded
// batches), then in whole multiples of the parts.
uint32_t strip_of(int64_t T, int64_t parts) {
    if (parts < 1) parts = 1;
    int64_t s = (T + parts - 1) / parts;
    if (s > kStrip) {
        parts *= (s + kStrip - 1) / kStrip;
        s = (T + parts - 1) / parts;
    }
    return (uint32_t)(s < kStripMin ? kStripMin : s);
}

// Parts of a chain whose columns all chains' threads hold: what fills the SMs once, with `threads` each (two waves of
// blocks and a few more took 29.5 us where one takes 23.3 for B8 H16 T2048 d = 128), or several times where one part
// each is more than that.
int64_t parts_of(int64_t columns, int threads) {
    const int64_t room = (int64_t)kSMs * threads;
    return columns <= room ? room / columns : columns < 6 * room ? (6 * room + columns - 1) / columns : 1;
}

// Blocks of the backward pass that share a group of a head's columns: two an SM in all, and no more than there are
// strips for; each part of their warps takes one strip, or as many as the others.
struct BwdShape {
    int lanes;
    uint32_t groups, strip, strips, slices;
};
BwdShape bwd_shape(int64_t B, int H, int64_t T, int d, int V) {
    BwdShape r;
    const int cols = (d + V - 1) / V;
    r.lanes = 1;
    while (r.lanes < 32 && r.lanes < cols) r.lanes *= 2;
    r.groups = (uint32_t)((cols + r.lanes - 1) / r.lanes);
    const int64_t y = (int64_t)H * r.groups, each = (kBlock / 32) * (32 / r.lanes);
    int64_t s = 2 * kSMs / y;
    if (s < 1) s = 1;
    r.strip = strip_of(T, s * each / B);
    r.strips = (uint32_t)((T + r.strip - 1) / r.strip);
    const int64_t most = (B * r.strips + each - 1) / each;
    r.slices = (uint32_t)(s > most ? most : s);
    return r;
}

// Channels a thread of the backward pass: 8 bytes of a row, where its alignment allows, beside the taps and their sums.
// (bf16, B8 H16 T2048 d = 128: four channels 45 us with four taps and 77 with eight, two 52 and 88.)
int bwd_vector(int d, fw_dtype dtype) { return dtype == FW_BF16 && d % 4 == 0 ? 4 : d % 2 == 0 ? 2 : 1; }

template <typename T, int V, int W> cudaError_t run(const ConvArgs &a, cudaStream_t s) {
    const int64_t cols = a.d / V;
    const uint32_t strip = strip_of(a.T, parts_of(a.n_chains * cols, V > 2 ? 512 : 1024)), strips = (uint32_t)((a.T + strip - 1) / strip);
    const int64_t n = a.n_chains * strips * cols;
    constexpr int smem = Stage<T, V, W, 1>::bytes();
    auto k = conv_kernel<T, V, W>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(k, smem, done);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)((n + kBlock - 1) / kBlock), kBlock, smem, s>>>(a, strip, strips, (uint32_t)cols);
    return cudaGetLastError();
}

template <typename T, int V, int W> cudaError_t run(const ConvBwdArgs &a, cudaStream_t s) {
    const BwdShape p = bwd_shape(a.B, a.H, a.T, a.d, V);
    constexpr int smem = Stage<T, V, W, 2>::bytes();
    auto k = conv_bwd_kernel<T, V, W>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(k, smem, done);
    if (e != cudaSuccess) return e;
    k<<<dim3(p.slices, a.H * p.groups), kBlock, smem, s>>>(a, p.strip, p.strips, p.lanes, p.groups);
    if ((e = cudaGetLastError()) != cudaSuccess || !a.ws) return e;
    const int64_t count = (int64_t)a.H * a.d * (W + 1);
    return launch_after(conv_sum_kernel, sum_grid(count), kSumCols * kSumShares, 0, s, true,
                        (const float *)a.ws, (int)p.slices, count, W, a.dweight, a.dbias);
}

template <typename T, int V, int W> cudaError_t run(const ConvStepArgs &a, cudaStream_t s) {
    const int64_t cols = a.d / V, n = a.n_states * cols;
    conv_step_kernel<T, V, W><<<(unsigned)((n + kBlock - 1) / kBlock), kBlock, 0, s>>>(a, (uint32_t)cols);
    return cudaGetLastError();
}

template <typename T, int V, typename A> cudaError_t by_taps(const A &a, cudaStream_t s) {
    switch (a.W) {
    case 2: return run<T, V, 2>(a, s);
    case 3: return run<T, V, 3>(a, s);
    case 4: return run<T, V, 4>(a, s);
    case 5: return run<T, V, 5>(a, s);
    case 6: return run<T, V, 6>(a, s);
    case 7: return run<T, V, 7>(a, s);
    default: return run<T, V, 8>(a, s);
    }
}

// 16 bytes of a row a thread where rows are whole multiples of that, else two elements (even d), else one: what the rows'
// alignment allows (forward, bf16, B4 H4 T4096: d = 128 and 130 10 us, 129 16 us; B8 H16 T2048 d = 128 23 us).
template <typename A> cudaError_t by_type(const A &a, cudaStream_t s) {
    if (a.dtype == FW_F32) return a.d % 4 == 0 ? by_taps<float, 4>(a, s) : a.d % 2 == 0 ? by_taps<float, 2>(a, s) : by_taps<float, 1>(a, s);
    if (a.d % 8 == 0) return by_taps<__nv_bfloat16, 8>(a, s);
    return a.d % 2 == 0 ? by_taps<__nv_bfloat16, 2>(a, s) : by_taps<__nv_bfloat16, 1>(a, s);
}

}  // namespace

bool conv_fits(int64_t B, int64_t H, int64_t T, int64_t d) {
    // threads of a call at the shortest strips and one channel each
    const int64_t strips = (T + kStripMin - 1) / kStripMin;
    return T <= INT32_MAX - 4096 && d <= (1 << 24) && B * H <= INT32_MAX / d && B * H * d <= INT32_MAX / strips;
}
bool conv_backward_fits(int64_t H, int64_t d) { return H * ((d + 31) / 32) <= 65535; }   // (the grid's second axis)

size_t conv_workspace(int64_t B, int H, int64_t T, int d, int W) {
    // (of either type)
    const uint32_t a = bwd_shape(B, H, T, d, bwd_vector(d, FW_F32)).slices, b = bwd_shape(B, H, T, d, bwd_vector(d, FW_BF16)).slices;
    return (size_t)(a > b ? a : b) * H * d * (W + 1) * sizeof(float);
}

cudaError_t launch_conv(const ConvArgs &a, cudaStream_t s) { return by_type(a, s); }
cudaError_t launch_conv_step(const ConvStepArgs &a, cudaStream_t s) { return by_type(a, s); }
cudaError_t launch_conv_backward(const ConvBwdArgs &a, cudaStream_t s) {
    const int v = bwd_vector(a.d, a.dtype);
    if (a.dtype == FW_F32) return v == 2 ? by_taps<float, 2>(a, s) : by_taps<float, 1>(a, s);
    if (v == 4) return by_taps<__nv_bfloat16, 4>(a, s);
    return v == 2 ? by_taps<__nv_bfloat16, 2>(a, s) : by_taps<__nv_bfloat16, 1>(a, s);
}

}  // namespace fw
