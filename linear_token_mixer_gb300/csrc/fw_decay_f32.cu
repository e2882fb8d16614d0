// fw_decay_f32.cu -- decayed linear attention scans (see fw_decay.cuh) for fp32 rows, d = 64 and
// 128, parallel over chunks of 64 tokens:
//
//   scan_local    M_c = in_scale sum_j w_j b_j c_j^T of every chunk (one block each)
//   scan_prefix   the short recurrence X' = g^n X + M_c over a chain's chunks, a thread for
//                 four elements; M_c is replaced by the state on entry to chunk c
//   scan_out      out = rd (A X_c) + (mask . decay . A B^T) C of every chunk (one block each)
//
// The products run on warp-level tf32 MMAs with every operand split in two (11 + 11 bits):
// a b = a1 b1 + a1 b2 + a2 b1 leaves out 2^-22 relative, so the rows keep fp32's accuracy; sums
// are fp32.  A chunk of 64 keeps the 64 x 64 part no larger than the d x d part and gives
// B*H*T/64 blocks, which is what short batches need to fill the GPU.  The three launches overlap
// their starts (programmatic dependent launch): scan_out loads its rows and forms the masked
// scores before it waits for the states, which it reads straight into the MMAs' operands.  Chains
// of one chunk need no workspace: one launch does both parts (scan_one).
//
// Measured (one GB300): B4 H8 T1000 d = 64 ragged 34 us, B4 H8 T2048 d = 128 171 us (2 % of it the look
// for rows that are not finite), the three scans of a backward pass of B2 H8 T1023 d = 64 45 us.  The short ones are bound by three launches that follow
// each other, the long ones by the split products: scan_out (d = 128) issues in 36 % of its
// cycles, its tensor pipe is busy for 39 %, and its sixteen warps an SM wait for the states' loads and
// for each other's MMAs.
//
// Selective scans (fw_select.cuh) are the same launches; a warp of a block forms the chunk's logs first, in both
// that need them, which is a launch less than tables of them: B4 H8 T1000 d = 64 37 us, B4 H8 T2048 d = 128 184 us.
#include "fw_decay_tc.cuh"
#include "fw_select.cuh"
#include "fw_sm100.cuh"

namespace fw {
namespace {

constexpr int C = 64;          // tokens per chunk

// The third scan's states (dk: sum v do^T) are the second's (dv: sum do v^T) transposed, so the
// second's are formed once and read both ways.
struct Scans {
    ScanArgs s[3];
};
constexpr int kSharing = 2;    // the scan that reads the one before it

// 2 x (D / 32) warps, a 32 x 32 tile of the 64 x D rows each.
template <int D> constexpr int threads() { return 2 * (D / 32) * 32; }
// Row strides that make the MMA fragments' reads free of bank conflicts: 4 (mod 32) where a
// fragment's rows are tile rows, 8 where its k runs along tile rows.
template <int D> constexpr int ld_row() { return D + 4; }
template <int D> constexpr int ld_col() { return D + 8; }

// x = hi + lo: hi rounded to 11 bits, lo what that leaves (exact in fp32; the MMA reads its top 11
// bits, so 2^-22 |x| at most is lost).  An infinity leaves NaN.
__device__ __forceinline__ void split(float x, uint32_t &hi, uint32_t &lo) {
    hi = sm100::f2tf32(x);
    lo = __float_as_uint(x - __uint_as_float(hi));
}

// acc += A B for a warp's 32 x 8 NT tile; element (m, k) of A at a[m * am + k * ak], element (k, n)
// of B at b[k * bk + n * bn].  The MMAs round towards zero: the two small terms are summed on their
// own, so that the large sum is cut a third as often (the d = 128 states summed in one: rows 9.6e-7
// off, apart 7.3e-7, for 2 % of the time).  B is fetched a step ahead: the states come from
// global memory (B4 H8 T2048 d = 128 173 us, then 165 us, with the strides known at compile time).
template <int NT>
__device__ __forceinline__ void gemm(float (&acc)[2][NT][4], const float *a, int am, int ak,
                                     const float *b, int bk, int bn, int K) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    a += g * am + t * ak;
    b += t * bk + g * bn;
    float low[2][NT][4] = {};
    float nb[NT][2];
    auto fetch = [&](int k) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) nb[n][e] = b[(k + 4 * e) * bk + 8 * n * bn];
    };
    fetch(0);
#pragma unroll 2
    for (int k = 0; k < K; k += 8) {
        uint32_t ah[2][4], al[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                split(a[(16 * m + 8 * (e & 1)) * am + (k + 4 * (e >> 1)) * ak], ah[m][e], al[m][e]);
        uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) split(nb[n][e], bh[n][e], bl[n][e]);
        if (k + 8 < K) fetch(k + 8);
        // the three terms one after the other over all tiles: no MMA waits for the one before it
#pragma unroll
        for (int term = 0; term < 3; ++term)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    sm100::mma_tf32_16x8x8(term < 2 ? low[m][n] : acc[m][n], term == 0 ? al[m] : ah[m],
                                           term == 1 ? bl[n] : bh[n]);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][n][e] += low[m][n][e];
}

// Rows [0, nv) of a chunk's 64 x D tile (rows behind them zero), each times row_w[r].
template <int D, int LD>
__device__ __forceinline__ void load_tile(float *dst, const float *src, int nv, const float *row_w) {
    constexpr int PR = D / 4;
#pragma unroll 8
    for (int i = threadIdx.x; i < C * PR; i += threads<D>()) {
        const int r = i / PR, c = (i % PR) * 4;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < nv) {
            f = *reinterpret_cast<const float4 *>(src + (int64_t)r * D + c);
            if (row_w) {
                const float w = row_w[r];
                f.x *= w; f.y *= w; f.z *= w; f.w *= w;
            }
        }
        *reinterpret_cast<float4 *>(dst + r * LD + c) = f;
    }
}

// Zeros to the rows of a chunk behind the sequence's end.
template <int D> __device__ __forceinline__ void zero_rest(const ScanArgs &s, int64_t chain, int64_t chunk, int nv) {
    const int64_t left = s.T - chunk * C;
    const int rows = left < C ? (int)left : C;
    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(s.out) + (chain * s.T + chunk * C) * D);
    for (int i = nv * (D / 4) + threadIdx.x; i < rows * (D / 4); i += threads<D>())
        o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
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

// Where a chunk's rows of a and b begin, given where those of c do.
template <int D, bool SEL> __device__ __forceinline__ int64_t ab_base(const ScanArgs &s, const ChunkOf &k, int64_t base) {
    return SEL ? (group_chain(k.chain, s.H, s.sel.gate.G) * s.T + k.chunk * C) * D : base;
}

// M_c into the workspace; ONE (chains of one chunk): the final state into X_out.  SEL here and below: a
// selective scan, whose weights and decays a warp forms of the chunk's own steps.
template <int D, bool ONE, bool SEL>
__device__ __forceinline__ void local_part(const ScanArgs &s, const ChunkOf &k, float4 *smem4) {
    constexpr int LD = ld_col<D>();
    float *sB = reinterpret_cast<float *>(smem4), *sC = sB + C * LD, *w = sC + C * LD;
    const float lg = SEL ? 0.f : s.log_decay[k.chain % s.H];
    float *const chunk_g = w + C;          // SEL: the chunk's decay
    if (SEL && threadIdx.x < 32) {
        const ChunkLogs<C> logs = chunk_logs<C>(s.sel.gate, k.chain, s.H, s.T, k.chunk * C + k.nv, k.chunk);
#pragma unroll
        for (int e = 0; e < logs.PER; ++e) w[threadIdx.x * logs.PER + e] = logs.weight(e);
        if (threadIdx.x == 0) {
            const float r = logs.decay();
            *chunk_g = r;
            if (!ONE) s.sel.decay[(k.chain * s.sel.n_chunks + k.chunk) * kDecayStride] = r;
        }
    }
    if (!SEL && threadIdx.x < C) {
        const int j = threadIdx.x;
        w[j] = s.in_scale * decay_pow(lg, (float)(s.rev ? j + 1 : max(k.nv - 1 - j, 0)));
    }
    __syncthreads();
    const int64_t base = (k.chain * s.T + k.chunk * C) * D;
    load_tile<D, LD>(sB, static_cast<const float *>(s.b) + ab_base<D, SEL>(s, k, base), k.nv, w);
    load_tile<D, LD>(sC, static_cast<const float *>(s.c) + base, k.nv, nullptr);
    __syncthreads();
    // D x D over 2 x (D / 32) warps: D / 2 rows of X by 32 columns each, 32 rows at a time
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = (warp >> 1) * 32;
    float *M = ONE ? s.X_out + k.chain * D * D : s.ws + (int64_t)blockIdx.x * D * D;
    const float *X0 = ONE && s.X0 ? s.X0 + k.chain * D * D : nullptr;
    const float gn = SEL ? *chunk_g : decay_pow(lg, (float)k.nv);
#pragma unroll 1
    for (int m0 = (warp & 1) * (D / 2), m1 = m0 + D / 2; m0 < m1; m0 += 32) {
        float acc[2][4][4] = {};
        gemm<4>(acc, sB + m0, 1, LD, sC + n0, LD, 1, C);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = m0 + 16 * m + (lane >> 2) + 8 * h, c = n0 + 8 * n + 2 * (lane & 3);
                    float2 v = make_float2(acc[m][n][2 * h], acc[m][n][2 * h + 1]);
                    if (X0) {
                        v.x = fmaf(gn, s.x0_trans ? X0[c * D + r] : X0[r * D + c], v.x);
                        v.y = fmaf(gn, s.x0_trans ? X0[(c + 1) * D + r] : X0[r * D + c + 1], v.y);
                    }
                    *reinterpret_cast<float2 *>(M + r * D + c) = v;
                }
    }
}

template <int D, bool SEL>
__global__ void __launch_bounds__(threads<D>())
scan_local(const __grid_constant__ Scans all, int64_t nch) {
    extern __shared__ float4 smem4[];
    let_next_grid_start();
    const ScanArgs &s = all.s[blockIdx.y];
    const ChunkOf k = chunk_of(s, nch);
    if (k.nv == 0 || (k.last && !s.X_out)) return;   // no later chunk and nobody reads the end
    local_part<D, false, SEL>(s, k, smem4);
}

constexpr int kPrefix = 128;   // threads of a block

// Four elements of a chain's state a thread, eight chunks read ahead of the recurrence (one element a
// thread: B4 H8 T2048 d = 128 196 us in all, then 171 us, B2 H8 T1023 d = 64 backward 46 us, then 44 us).
template <int D, bool SEL>
__global__ void __launch_bounds__(kPrefix)
scan_prefix(const __grid_constant__ Scans all, int64_t nch) {
    const ScanArgs &s = all.s[blockIdx.y];
    constexpr int PER = D * D / 4 / kPrefix;   // blocks of a chain
    const int64_t chain = blockIdx.x / PER;
    const int el = 4 * ((int)(blockIdx.x % PER) * kPrefix + (int)threadIdx.x);
    let_next_grid_start();
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (s.X0) {
        const float *X0 = s.X0 + chain * D * D;
        const int r = el / D, c = el % D;
        x = s.x0_trans ? make_float4(X0[c * D + r], X0[(c + 1) * D + r], X0[(c + 2) * D + r], X0[(c + 3) * D + r])
                       : *reinterpret_cast<const float4 *>(X0 + el);
    }
    const int64_t n = chain_len(s.lens, chain, s.H, s.T);
    const int used = (int)((n + C - 1) / C);
    const float lg = SEL ? 0.f : s.log_decay[chain % s.H];
    const float gC = decay_pow(lg, (float)C), gT = decay_pow(lg, (float)(n - (int64_t)(used - 1) * C));
    // in processing order; the end is nobody's entry, and is left out where it is not asked for
    const int read = s.X_out ? used : used - 1;
    const int64_t step = s.rev ? -(D * D / 4) : D * D / 4;
    float4 *M = reinterpret_cast<float4 *>(s.ws + chain * nch * D * D + el) + (s.rev ? (int64_t)(used - 1) * (D * D / 4) : 0);
    wait_previous_grid();
    constexpr int U = 8;
    for (int i0 = 0; i0 < used; i0 += U, M += U * step) {
        float4 m[U];
#pragma unroll
        for (int u = 0; u < U; ++u) m[u] = i0 + u < read ? M[u * step] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u >= used) break;
            M[u * step] = x;
            const float g = SEL ? s.sel.decay[(chain * nch + i0 + u) * kDecayStride]
                                : (s.rev ? i0 + u == 0 : i0 + u == used - 1) ? gT : gC;
            x.x = fmaf(g, x.x, m[u].x);
            x.y = fmaf(g, x.y, m[u].y);
            x.z = fmaf(g, x.z, m[u].z);
            x.w = fmaf(g, x.w, m[u].w);
        }
    }
    if (s.X_out) *reinterpret_cast<float4 *>(s.X_out + chain * D * D + el) = x;
}

// The output rows of a chunk, from the state at X (element (i, j) at X[i * D + j], or
// X[j * D + i] with `trans`); ONE: known before the launch.
template <int D, bool ONE, bool SEL>
__device__ __forceinline__ void out_part(const ScanArgs &s, const ChunkOf &k, const float *X, const bool trans,
                                         float4 *smem4) {
    constexpr int LR = ld_row<D>(), LC = ld_col<D>(), WN = D / 32, LP = C + 4;
    float *sA = reinterpret_cast<float *>(smem4), *sB = sA + C * LR, *sC = sB + C * LR,
          *pw = sC + C * LC, *red = pw + C + 4;
    int *const first = reinterpret_cast<int *>(red + C * WN);
    float2 *const lc = reinterpret_cast<float2 *>((reinterpret_cast<uintptr_t>(first + D) + 7) & ~(uintptr_t)7);
    if (SEL) {                             // pw: the steps; lc: the logs of the decays
        if (threadIdx.x < 32) {
            const ChunkLogs<C> logs = chunk_logs<C>(s.sel.gate, k.chain, s.H, s.T, k.chunk * C + k.nv, k.chunk);
#pragma unroll
            for (int e = 0; e < logs.PER; ++e) {
                pw[threadIdx.x * logs.PER + e] = logs.dt[e];
                lc[threadIdx.x * logs.PER + e] = make_float2(logs.c[e].hi, logs.c[e].lo);
            }
        }
    } else {
        const float lg = s.log_decay[k.chain % s.H];
        for (int i = threadIdx.x; i <= C; i += threads<D>()) pw[i] = decay_pow(lg, (float)i);
    }
    // the decay from token j, its step among it, to row r >= j; of the state to row r
    const auto lag_of = [&](int r, int j) -> float {
        if (SEL) return pw[j] * exp_two(lc[r].x - lc[j].x, lc[r].y - lc[j].y);
        return pw[s.rev ? j - r : r - j] * s.in_scale;
    };
    const auto entry_of = [&](int r) -> float {
        return SEL ? exp_two(lc[r].x, lc[r].y) : pw[s.rev ? max(k.nv - 1 - r, 0) : r + 1];
    };
    const int64_t base = (k.chain * s.T + k.chunk * C) * D, ab = ab_base<D, SEL>(s, k, base);
    load_tile<D, LR>(sA, static_cast<const float *>(s.a) + ab, k.nv, nullptr);
    load_tile<D, LR>(sB, static_cast<const float *>(s.b) + ab, k.nv, nullptr);
    const float *const c = static_cast<const float *>(s.c) + base;
    load_tile<D, LC>(sC, c, k.nv, nullptr);
    __syncthreads();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int m0 = (warp & 1) * 32, wn = warp >> 1;
    {   // P = mask . decay . A B^T over B's rows: 32 rows by 64 / WN columns a warp
        constexpr int NT = C / WN / 8;
        const int n0 = wn * (C / WN);
        float p[2][NT][4] = {};
        gemm<NT>(p, sA + m0 * LR, LR, 1, sB + n0 * LR, 1, LR, D);
        __syncthreads();                   // B is read
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = m0 + 16 * m + g + 8 * (e >> 1), j = n0 + 8 * n + 2 * t + (e & 1);
                    const int lag = s.rev ? j - r : r - j;
                    sB[r * LP + j] = lag >= 0 && j < k.nv ? p[m][n][e] * lag_of(r, j) : 0.f;
                }
    }
    if (!ONE) wait_previous_grid();        // the states
    __syncthreads();                       // P is written
    const bool zero = !s.X0 && (ONE || (s.rev ? k.nv < C || (k.chunk + 1) * C >= chain_len(s.lens, k.chain, s.H, s.T)
                                              : k.chunk == 0));   // nothing carried in

    const int n0 = wn * 32;
    float acc[2][4][4] = {};
    if (!zero) {
        if (trans) gemm<4>(acc, sA + m0 * LR, LR, 1, X + n0 * D, 1, D, D);
        else gemm<4>(acc, sA + m0 * LR, LR, 1, X + n0, D, 1, D);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = m0 + 16 * m + g + 8 * h;
            const float rd = entry_of(r);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                acc[m][n][2 * h] *= rd;
                acc[m][n][2 * h + 1] *= rd;
            }
        }
    gemm<4>(acc, sB + m0 * LP, LP, 1, sC + n0, LC, 1, C);

#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][n][e] *= s.out_scale;
    // P C reads a value of C that the mask keeps from a row as 0 times it, which is NaN of an infinity or
    // a NaN.  Where a block's rows are not all finite, such values become zero, each column's first in
    // processing order is noted, and the rows are formed once more; those that see one are NaN.
    // (Later chunks have it from the state.)
    float nan = 0.f;                       // 0 while all are finite
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) nan = fmaf(acc[m][n][e], 0.f, nan);
    if (__syncthreads_or(nan != 0.f)) {
        for (int i = threadIdx.x; i < D; i += threads<D>()) first[i] = C;
        __syncthreads();
        for (int i = threadIdx.x; i < k.nv * D; i += threads<D>())
            if (!isfinite(c[i])) {
                atomicMin(first + i % D, s.rev ? C - 1 - i / D : i / D);
                sC[i / D * LC + i % D] = 0.f;
            }
        __syncthreads();
        const auto each = [&](auto f) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        f(acc[m][n][e], m0 + 16 * m + g + 8 * (e >> 1), n0 + 8 * n + 2 * t + (e & 1));
        };
        each([&](float &v, int, int) { v = 0.f; });
        if (!zero)
#pragma unroll 1
            for (int i = 0; i < D; ++i)
                each([&](float &v, int r, int col) { v = fmaf(sA[r * LR + i], trans ? X[col * D + i] : X[i * D + col], v); });
        each([&](float &v, int r, int) { v *= entry_of(r); });
#pragma unroll 1
        for (int j = 0; j < C; ++j)
            each([&](float &v, int r, int col) { v = fmaf(sB[r * LP + j], sC[j * LC + col], v); });
        each([&](float &v, int r, int col) {
            v = first[col] <= (s.rev ? C - 1 - r : r) ? __int_as_float(0x7fffffff) : v * s.out_scale;
        });
    }
    if (SEL && s.sel.gate.skip) {          // (from memory: sC may have lost values that are not finite)
        const float skip = s.sel.gate.skip[k.chain % s.H];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = m0 + 16 * m + g + 8 * h;
                if (r < k.nv)
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const float2 f = *reinterpret_cast<const float2 *>(c + (int64_t)r * D + n0 + 8 * n + 2 * t);
                        acc[m][n][2 * h] = fmaf(skip, f.x, acc[m][n][2 * h]);
                        acc[m][n][2 * h + 1] = fmaf(skip, f.y, acc[m][n][2 * h + 1]);
                    }
            }
    }
    if (!SEL && s.norm.on) {               // a row is held by four lanes of each of WN warps
        auto row_sums = [&](float (&z)[2][2]) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    z[m][h] += __shfl_xor_sync(~0u, z[m][h], 1);
                    z[m][h] += __shfl_xor_sync(~0u, z[m][h], 2);
                    if (t == 0) red[(m0 + 16 * m + g + 8 * h) * WN + wn] = z[m][h];
                }
            __syncthreads();
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    z[m][h] = 0.f;
#pragma unroll
                    for (int w = 0; w < WN; ++w) z[m][h] += red[(m0 + 16 * m + g + 8 * h) * WN + w];
                }
            __syncthreads();
        };
        float z[2][2] = {};
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[m][e >> 1] += acc[m][n][e];
        row_sums(z);
        float v[2][2] = {};
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[m][n][e] -= z[m][e >> 1] / D;
                    v[m][e >> 1] = fmaf(acc[m][n][e], acc[m][n][e], v[m][e >> 1]);
                }
        row_sums(v);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int col = n0 + 8 * n + 2 * t + (e & 1);
                    acc[m][n][e] *= rsqrtf(v[m][e >> 1] / D + s.norm.eps);
                    if (s.norm.weight) acc[m][n][e] *= s.norm.weight[col];
                    if (s.norm.bias) acc[m][n][e] += s.norm.bias[col];
                }
    }
    float *out = static_cast<float *>(s.out) + base;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = m0 + 16 * m + g + 8 * h;
            if (r >= k.nv) continue;
#pragma unroll
            for (int n = 0; n < 4; ++n)
                *reinterpret_cast<float2 *>(out + (int64_t)r * D + n0 + 8 * n + 2 * t) =
                    make_float2(acc[m][n][2 * h], acc[m][n][2 * h + 1]);
        }
}

template <int D, bool SEL>
__global__ void __launch_bounds__(threads<D>(), 2)
scan_out(const __grid_constant__ Scans all, int64_t nch) {
    extern __shared__ float4 smem4[];
    const ScanArgs &s = all.s[blockIdx.y];
    const ChunkOf k = chunk_of(s, nch);
    if (s.zero_rest) zero_rest<D>(s, k.chain, k.chunk, k.nv);
    if (k.nv == 0) {                       // (no block ends before the grids it follows)
        wait_previous_grid();
        return;
    }
    const bool trans = blockIdx.y == kSharing;
    const float *ws = trans ? all.s[kSharing - 1].ws : s.ws;
    out_part<D, false, SEL>(s, k, ws + (int64_t)blockIdx.x * D * D, trans, smem4);
}

// Chains of one chunk: rows (z = 1) and final states (z = 0) at once, or one after the other (one z)
// where X_out is X0, which the rows read.
template <int D, bool SEL>
__global__ void __launch_bounds__(threads<D>())
scan_one(const __grid_constant__ Scans all) {
    extern __shared__ float4 smem4[];
    const ScanArgs &s = all.s[blockIdx.y];
    const ChunkOf k = chunk_of(s, 1);
    const bool both = gridDim.z == 1;
    if (both || blockIdx.z == 1) {
        if (s.zero_rest) zero_rest<D>(s, k.chain, 0, k.nv);
        if (k.nv > 0) out_part<D, true, SEL>(s, k, s.X0 ? s.X0 + k.chain * D * D : nullptr, s.x0_trans, smem4);
    }
    if (both) __syncthreads();
    if (both || blockIdx.z == 0)
        if (s.X_out) local_part<D, true, SEL>(s, k, smem4);
}

template <int D, bool SEL>
cudaError_t launch(const Scans &all, int n, cudaStream_t stream) {
    const ScanArgs &s = all.s[0];
    const int64_t nch = (s.T + C - 1) / C;
    const dim3 grid((unsigned)(s.n_chains * nch), n);
    constexpr int smem_l = (2 * C * ld_col<D>() + C + (SEL ? 1 : 0)) * 4;
    constexpr int smem_o = (2 * C * ld_row<D>() + C * ld_col<D>() + C + 4 + C * (D / 32) + D + (SEL ? 2 * C + 2 : 0)) * 4;
    cudaError_t e;
    if (nch == 1) {
        constexpr int smem = smem_l > smem_o ? smem_l : smem_o;
        static std::atomic<uint64_t> done{0};
        if ((e = allow_smem(scan_one<D, SEL>, smem, done)) != cudaSuccess) return e;
        const bool in_place = s.X_out && s.X_out == s.X0;
        return launch_after(scan_one<D, SEL>, dim3((unsigned)s.n_chains, n, in_place ? 1 : 2), threads<D>(), smem, stream,
                            false, all);
    }
    static std::atomic<uint64_t> local_done{0}, out_done{0};
    if ((e = allow_smem(scan_local<D, SEL>, smem_l, local_done)) != cudaSuccess) return e;
    if ((e = allow_smem(scan_out<D, SEL>, smem_o, out_done)) != cudaSuccess) return e;
    const int states = n < kSharing ? n : kSharing;
    if ((e = launch_after(scan_local<D, SEL>, dim3(grid.x, states), threads<D>(), smem_l, stream, false, all, nch)) !=
        cudaSuccess)
        return e;
    const dim3 gp((unsigned)(s.n_chains * (D * D / 4 / kPrefix)), states);
    if ((e = launch_after(scan_prefix<D, SEL>, gp, kPrefix, 0, stream, true, all, nch)) != cudaSuccess) return e;
    return launch_after(scan_out<D, SEL>, grid, threads<D>(), smem_o, stream, true, all, nch);
}

}  // namespace

// Bytes of the states of every chunk of a scan.
static size_t state_bytes(int64_t n_chains, int64_t T, int d) {
    return (size_t)n_chains * (size_t)((T + C - 1) / C) * d * d * sizeof(float);
}

size_t scan_workspace(int64_t n_chains, int64_t T, int d, fw_dtype dtype, bool backward) {
    if (dtype == FW_BF16) return scan_tc_workspace(n_chains, T, d, backward);
    return T <= C ? 0 : (backward ? kSharing : 1) * state_bytes(n_chains, T, d);
}

// bf16 rows run on the fifth-generation tensor cores, fp32 rows here.
cudaError_t launch_scans(ScanArgs *s, int n, cudaStream_t stream) {
    if (s[0].dtype == FW_BF16) return launch_scans_tc(s, n, stream);
    if (n > 1 && s[0].ws) s[1].ws = s[0].ws + state_bytes(s->n_chains, s->T, s->d) / sizeof(float);   // (the third: none)
    Scans all{};
    for (int i = 0; i < n; ++i) all.s[i] = s[i];
    return s[0].d == 64 ? launch<64, false>(all, n, stream) : launch<128, false>(all, n, stream);
}

// A selective scan: [states][the chunks' decays], neither where a chain is one chunk.
static size_t decay_bytes(int64_t n_chains, int64_t T) {
    return (size_t)n_chains * (size_t)((T + C - 1) / C) * kDecayStride * sizeof(float);
}
size_t select_workspace_f32(int64_t n_chains, int64_t T, int d) {
    return T <= C ? 0 : state_bytes(n_chains, T, d) + decay_bytes(n_chains, T);
}
cudaError_t launch_select_f32(const ScanArgs &scan, cudaStream_t stream) {
    Scans all{};
    ScanArgs &s = all.s[0] = scan;
    s.sel.n_chunks = (s.T + C - 1) / C;
    if (s.T > C) s.sel.decay = s.ws + state_bytes(s.n_chains, s.T, s.d) / sizeof(float);
    return s.d == 64 ? launch<64, true>(all, 1, stream) : launch<128, true>(all, 1, stream);
}

}  // namespace fw
