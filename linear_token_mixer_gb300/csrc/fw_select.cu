// fw_select.cu -- selective scan: the steps and decays of a prompt, and its form for one token.
//
//     dt_t = softplus(dt_raw_t + dt_bias),  g_t = exp(log_decay dt_t),
//     S_t = g_t S_{t-1} + dt_t k_t v_t^T,   o_t = scale S_t^T q_t + skip v_t
//
// A prompt is the chunked scan of fw_decay_tc.cu (bf16) or fw_decay_f32.cu (fp32) with tables in place of
// powers of one decay: select_tables forms, for every chunk of a chain, the running sum of log g to each
// token in two fp32 terms (differences of sums of a chunk lose nothing to their size),
// each token's weight in the chunk's end, and the chunk's decay.  One warp a chunk, 20 bytes a token
// written for the 4 d (bf16) or 8 d that its rows take; the scan's first tiles load meanwhile.
//
// One token: one block a state, the state once through registers, as decay_step_kernel.
#include "fw_select.cuh"

namespace fw {
namespace {

constexpr int kTableBlock = 128;

// A sum of fp32 values in two terms, hi + lo with |lo| at most half a unit of hi (48 bits; the GPU's 64-bit
// additions are a sixteenth as fast as these four to eight fp32 ones).
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two add(const Two &a, const Two &b) {
    const float s = a.hi + b.hi, t = s - a.hi, e = (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo), hi = s + e;
    return {hi, e - (hi - s)};
}

// Where the tables are written (see SelectTables).
struct Tables {
    float2 *c;
    float *dt, *w;
    float4 *chunk, *ends;
    int64_t n_chunks;
};

// TC: in the layout of the bf16 scans; mild_too: chunks may be mild (not with a scale of zero, whose epilogue scales
// A X apart from the rest).
template <int C, bool TC>
__global__ void __launch_bounds__(kTableBlock)
select_tables(GateArgs g, const int32_t *lens, int64_t n_chains, int64_t T, int H, int mild_too, Tables out) {
    constexpr int PER = C / 32;               // tokens of a lane
    let_next_grid_start();
    const int lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * (kTableBlock / 32) + (threadIdx.x >> 5);
    if (id >= n_chains * out.n_chunks) return;
    const int64_t chain = id / out.n_chunks, first = id % out.n_chunks * C + lane * PER;
    const int64_t n = chain_len(lens, chain, H, T);
    const int h = (int)(chain % H);
    const float rate = g.log_decay[h];
    float dt[PER];
    Two c[PER], sum{0.f, 0.f};                // of the logs, to the token
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const bool on = first + e < n;
        dt[e] = on ? step_of(g, chain * T + first + e, h) : 0.f;
        const float x = on ? rate * dt[e] : 0.f;
        sum = add(sum, x < -kReset ? Two{-kReset, 0.f} : Two{x, on ? fmaf(rate, dt[e], -x) : 0.f});   // (NaN stays)
        c[e] = sum;
    }
    Two upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Two x{__shfl_up_sync(~0u, upto.hi, o), __shfl_up_sync(~0u, upto.lo, o)};
        if (lane >= o) upto = add(x, upto);
    }
    const Two total{__shfl_sync(~0u, upto.hi, 31), __shfl_sync(~0u, upto.lo, 31)};
    Two before{__shfl_up_sync(~0u, upto.hi, 1), __shfl_up_sync(~0u, upto.lo, 1)};
    if (lane == 0) before = Two{0.f, 0.f};
    float low = 0.f, high = 0.f;              // the least and the largest sum
    const int64_t at = id * C + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        c[e] = add(before, c[e]);
        low = fminf(low, c[e].hi);
        high = fmaxf(high, c[e].hi);
        const Two s = add(total, Two{-c[e].hi, -c[e].lo});
        const float w = dt[e] * exp_two(s.hi, s.lo);
        if (TC) {
            out.c[at + e] = make_float2(c[e].hi, dt[e]);
            out.w[id * C + weight_place(lane * PER + e)] = w;
        } else {
            out.c[at + e] = make_float2(c[e].hi, c[e].lo);
            out.dt[at + e] = dt[e];
            out.w[at + e] = w;
        }
    }
    if (TC) {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            low = fminf(low, __shfl_xor_sync(~0u, low, o));
            high = fmaxf(high, __shfl_xor_sync(~0u, high, o));
        }
        float end[3];
#pragma unroll
        for (int b = 0; b < 3; ++b) end[b] = __shfl_sync(~0u, c[PER - 1].hi, 32 / PER * (b + 1) - 1);
        if (lane == 0)
            out.ends[id] = make_float4(end[0], end[1], end[2],
                                       mild_too && low >= -kMild && high <= kMild && isfinite(total.hi) ? 1.f : 0.f);
    }
    if (lane == 0) out.chunk[id] = make_float4(exp_two(total.hi, total.lo), total.hi, total.lo, 0.f);
}

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

// Bytes of the tables' parts, each a multiple of 16.
struct TableBytes {
    size_t c, dt, w, chunk, ends;
    size_t all() const { return c + dt + w + chunk + ends; }
};
TableBytes table_bytes(int64_t n_chains, int64_t T, bool tc) {
    const int C = tc ? select_chunk_tc() : select_chunk_f32();
    const size_t chunks = (size_t)n_chains * (size_t)((T + C - 1) / C), tokens = chunks * C;
    return {tokens * sizeof(float2), tc ? 0 : tokens * sizeof(float), tokens * sizeof(float), chunks * sizeof(float4),
            tc ? chunks * sizeof(float4) : 0};
}

}  // namespace

// [tables][the scan's own]
size_t select_workspace(int64_t n_chains, int64_t T, int d, fw_dtype dtype) {
    const bool tc = dtype == FW_BF16;
    return table_bytes(n_chains, T, tc).all() + (tc ? select_states_tc(n_chains, T, d) : select_states_f32(n_chains, T, d));
}

cudaError_t launch_select(const SelectArgs &args, cudaStream_t stream) {
    ScanArgs s = args.scan;
    const bool tc = s.dtype == FW_BF16;
    const int C = tc ? select_chunk_tc() : select_chunk_f32();
    const TableBytes b = table_bytes(s.n_chains, s.T, tc);
    char *p = reinterpret_cast<char *>(s.ws);
    auto part = [&](size_t n) {
        char *const at = p;
        p += n;
        return at;
    };
    Tables t;
    t.c = reinterpret_cast<float2 *>(part(b.c));
    t.dt = reinterpret_cast<float *>(part(b.dt));
    t.w = reinterpret_cast<float *>(part(b.w));
    t.chunk = reinterpret_cast<float4 *>(part(b.chunk));
    t.ends = reinterpret_cast<float4 *>(part(b.ends));
    t.n_chunks = (s.T + C - 1) / C;
    s.ws = reinterpret_cast<float *>(p);
    s.sel = SelectTables{t.c, t.dt, t.w, t.chunk, t.ends, args.gate.skip, t.n_chunks, args.gate.G};
    const int64_t warps = s.n_chains * t.n_chunks;
    const unsigned grid = (unsigned)((warps + kTableBlock / 32 - 1) / (kTableBlock / 32));
    if (tc) select_tables<128, true><<<grid, kTableBlock, 0, stream>>>(args.gate, s.lens, s.n_chains, s.T, s.H, s.out_scale != 0.f, t);
    else select_tables<64, false><<<grid, kTableBlock, 0, stream>>>(args.gate, s.lens, s.n_chains, s.T, s.H, 1, t);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return tc ? launch_select_tc(s, stream) : launch_select_f32(s, stream);
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
