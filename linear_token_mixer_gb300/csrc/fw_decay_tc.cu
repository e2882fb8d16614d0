// fw_decay_tc.cu -- decayed linear attention scans (see fw_decay.cuh) for bf16 rows on the
// fifth-generation tensor cores, d = 64 and 128, in chunks of 128 tokens.
//
// Per chunk of n valid rows, with the state X on entry (forward; the reverse scan swaps the
// exponents as in fw_decay.cuh):
//     G = A B^T                                     128 x 128 x d
//     P = mask . g^|i-j| . G          (bf16)
//     O = diag(g^(i+1)) (A X) + P C                 128 x d x d, 128 x d x 128
//     X <- g^n X + (diag(w) B)^T C                  d x d x 128, three times
// The last product's left operand is split into three bf16 terms (24 bits of w_j b_j), so the
// fp32 state loses nothing to its operands; P and the copy of X that A reads are rounded to bf16
// once, like the output rows.
//
// One CTA per chain, or per segment of a chain where chains are few, warp-specialised:
//   warp 0       TMA producer: tiles of B, A, C (128 x d, 128-byte swizzle), each released on
//                its own
//   warp 1       MMA issuer of G and P C
//   warp 2       MMA issuer of A X and the state update
//   warp 3       tensor-memory allocation
//   warps 4-7    P: tensor memory -> mask, decay, bf16 -> tensor memory (A operand of P C)
//   warps 8-11   O: scales A X by its row's decay in place before P C accumulates on it, then
//                [output norm,] rounds and stores the rows (one thread a row)
//   warps 12-15  the three terms of (diag(w) B)^T, 32 tokens at a time, into tensor memory
//                (thread = lane = row of X), double-buffered
//   warps 16-19  X: tensor memory -> bf16 shared-memory copy for A X, and X * g^n back
// Tensor memory: G (P over it) 128 columns, O 128, X 128, the split operand 2 x 48.
// Every wait is bounded; on expiry the kernel records an error, the other roles stop at their
// next wait, copies and MMAs in flight are drained, tensor memory is freed and the kernel exits.
#include <cudaTypedefs.h>

#include <mutex>

#include "fw_decay_tc.cuh"
#include "fw_sm100.cuh"

namespace fw {
namespace {
using namespace sm100;

constexpr int C = 128;
constexpr int NTHREADS = 640;
constexpr uint32_t KB = 1024;
constexpr uint32_t HALF = 16 * KB;           // 128 rows x 128 bytes: 64 columns of a tile
constexpr int kSMs = 152;                    // the grid's target (a workspace size needs no device)
constexpr int kMinSegChunks = 4;

constexpr uint32_t COL_G = 0, COL_O = 128, COL_X = 256, COL_K = 384, KBUF = 48;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint64_t kDrainNs = 2000000000ull;

template <int D, bool PRE> struct Lay {
    static constexpr uint32_t TILE = (uint32_t)C * D * 2;
    static constexpr int NT = PRE ? 2 : 3;                       // tiles per stage
    static constexpr int NST = (int)(192 * KB / (TILE * NT));    // 2 (3), d = 64: 4 (6)
    static constexpr uint32_t XB = NST * NT * TILE;              // bf16 copy of X
    static constexpr uint32_t TAB = XB + (uint32_t)D * D * 2;
    static constexpr uint32_t T_PW = TAB, T_PR = T_PW + 132 * 4, T_KW = T_PR + 16 * 4,
                              T_KT = T_KW + 128 * 4, BAR = T_KT + 128 * 4;
    // barriers
    static constexpr int FULL = 0, EMPTY = FULL + NST * NT, GDONE = EMPTY + NST * NT,
                         PRDY = GDONE + 1, QSDONE = PRDY + 1, OSC = QSDONE + 1, PVDONE = OSC + 1,
                         OFREE = PVDONE + 1, XDONE = OFREE + 1, XBRDY = XDONE + 1,
                         XSC = XBRDY + 1, KRDY = XSC + 1, KFREE = KRDY + 2, VZ = KFREE + 2,
                         DRAIN0 = VZ + 1, DRAIN1 = DRAIN0 + 1, NEVER = DRAIN1 + 1,
                         NBAR = NEVER + 1;
    static constexpr uint32_t MISC = BAR + NBAR * 8;
    static constexpr uint32_t BYTES = MISC + 16;
    static constexpr uint32_t ALLOC = BYTES + 1024;
    static_assert(ALLOC <= 227 * KB, "shared memory budget");
};

__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint64_t limit,
                                       volatile int *abort_flag) {
    const uint64_t t0 = globaltimer();
    for (;;) {
        if (mbar_try_wait_sleep(bar, parity, 100000u)) return true;
        if (*abort_flag) return false;
        if (globaltimer() - t0 > limit) return false;
    }
}

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, uint64_t limit,
                                         volatile int *abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    return wait_slow(bar, parity, limit, abort_flag);
}

// Segment `seg` of a chain: its chunks in processing order [first, last) of `total`.
struct Seg {
    int first, last, total;
};
__device__ __forceinline__ Seg seg_of(int64_t n, int seg, int nseg) {
    Seg s;
    s.total = (int)((n + C - 1) / C);
    s.first = (int)((int64_t)seg * s.total / nseg);
    s.last = (int)((int64_t)(seg + 1) * s.total / nseg);
    return s;
}
// Tokens of processing step i of a chain of n tokens in `total` chunks.
template <bool REV> __device__ __forceinline__ int step_tokens(int64_t n, int total, int i) {
    const int c = REV ? total - 1 - i : i;
    return c == total - 1 ? (int)(n - (int64_t)c * C) : C;
}
template <bool REV>
__device__ __forceinline__ int64_t seg_tokens(int64_t n, const Seg &s) {
    if (s.first >= s.last) return 0;
    const int64_t full = (int64_t)(s.last - s.first) * C;
    const bool tail = REV ? s.first == 0 : s.last == s.total;
    return tail ? full - ((int64_t)s.total * C - n) : full;
}

// Four 8x8 b16 matrices, transposed: thread t gets rows 2 (t % 4), +1 of column t / 4.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// 16 lanes x 16 columns: register 2c + h holds lane 8h + t / 4, column 4c + t % 4 of thread t.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ void mul2(float &a0, float &a1, float b0, float b1) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1));
}
__device__ __forceinline__ void sub2(float &a0, float &a1, float b0, float b1) {   // a - b
    asm("{\n\t.reg .b64 x, y, m;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "mov.b64 m, {%4, %4};\n\tfma.rn.f32x2 x, y, m, x;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1), "f"(-1.f));
}

// The upper halves of two fp32 words (bf16, truncated), x0 in the low half.
__device__ __forceinline__ uint32_t top_halves(float x0, float x1) {
    return __byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632);
}
// What that truncation drops of each (exact).
__device__ __forceinline__ void below(float &x0, float &x1) {
    sub2(x0, x1, __uint_as_float(__float_as_uint(x0) & 0xffff0000u),
         __uint_as_float(__float_as_uint(x1) & 0xffff0000u));
}

// PRE: only the state of a segment, from zero (segment 0: from X0), into the workspace.
template <int D, bool REV, bool PRE, bool NORM>
__global__ void __launch_bounds__(NTHREADS, 1)
scan_tc_kernel(const __grid_constant__ CUtensorMap tma, const __grid_constant__ CUtensorMap tmb,
               const __grid_constant__ CUtensorMap tmc, const __grid_constant__ CUtensorMap tmo,
               const ScanArgs a, const int nseg) {
    using L = Lay<D, PRE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int grid_seg = PRE ? nseg - 1 : nseg;
    const int64_t chain = blockIdx.x / grid_seg;
    const int seg = blockIdx.x % grid_seg;
    const int64_t n = chain_len(a.lens, chain, a.H, a.T);
    const Seg sg = seg_of(n, seg, nseg);
    const int nch = sg.last - sg.first;
    const bool final_seg = !PRE && seg == nseg - 1;
    if (nch == 0 && !(final_seg && a.X_out) && !(PRE && seg == 0)) return;
    const uint64_t limit = (uint64_t)a.wait_ns;
    const float lg = a.log_decay[chain % a.H];
    const int x_slots = nseg;                       // workspace: nseg - 1 segment states, X0's copy
    float *const ws = a.ws + chain * x_slots * D * D;

    volatile int *s_abort = reinterpret_cast<volatile int *>(sm + L::MISC);
    volatile uint32_t *s_tmem = reinterpret_cast<volatile uint32_t *>(sm + L::MISC + 4);
    float *const pw = reinterpret_cast<float *>(sm + L::T_PW);   // g^n, n = 0..128
    float *const pr = reinterpret_cast<float *>(sm + L::T_PR);   // g^(15-j) (reverse: g^j), j < 16
    float *const kw = reinterpret_cast<float *>(sm + L::T_KW);   // w_j of a full chunk
    float *const kt = reinterpret_cast<float *>(sm + L::T_KT);   // w_j of the tail chunk
    auto bar = [&](int i) -> uint32_t { return sb + L::BAR + 8u * (uint32_t)i; };
    auto full = [&](int st, int x) -> uint32_t { return bar(L::FULL + st * L::NT + x); };
    auto empty = [&](int st, int x) -> uint32_t { return bar(L::EMPTY + st * L::NT + x); };
    auto tile = [&](int st, int x) -> uint32_t { return sb + (uint32_t)(st * L::NT + x) * L::TILE; };
    constexpr int XB_ = 0, XC = 1, XA = 2;          // tiles of a stage: B, C and (not PRE) A
    auto fail_now = [&]() {
        *s_abort = 1;
        atomicExch(a.err, kDevErrTimeout);
    };
    auto chunk_id = [&](int i) -> int { return REV ? sg.total - 1 - (sg.first + i) : sg.first + i; };
    auto tokens = [&](int i) -> int { return step_tokens<REV>(n, sg.total, sg.first + i); };

    if (tid == 0) {
        for (int i = 0; i < L::NBAR; ++i) {
            uint32_t c = 1;
            const int e = i - L::EMPTY;
            if (e >= 0 && e < L::NST * L::NT)       // B: its readers' four warps (and G); C: the
                c = e % L::NT == XB_ ? (PRE ? 4 : 5)   // update (and P C); A: the O group's warps
                  : e % L::NT == XC ? (PRE ? 1 : 2) : 4;
            if (i == L::PRDY || i == L::OSC || i == L::OFREE || i == L::XBRDY || i == L::XSC ||
                i == L::KRDY || i == L::KRDY + 1 || i == L::VZ)
                c = 4;
            mbar_init(bar(i), c);
        }
        fence_mbar_init();
        *s_abort = 0;
    }
    for (int i = tid; i <= C; i += NTHREADS) pw[i] = decay_pow(lg, (float)i);
    if (tid < 16) pr[tid] = decay_pow(lg, (float)(REV ? tid : 15 - tid));
    if (tid < C) kw[tid] = a.in_scale * decay_pow(lg, (float)(REV ? tid + 1 : C - 1 - tid));
    if (warp == 3) tmem_alloc(sb + L::MISC + 4, TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        if (lane == 0) {
            bool ok = true;
            if (a.force_timeout) ok = wait_bar(bar(L::NEVER), 0, limit, s_abort);
            int issued = 0;                          // tiles, in issue order
            for (int i = 0; i < nch && ok; ++i) {
                const int st = i % L::NST;
                const int y = chunk_id(i) * C;
#pragma unroll
                for (int x0 = 0; x0 < L::NT && ok; ++x0) {
                    const int x = PRE ? x0 : x0 == 0 ? XB_ : x0 == 1 ? XA : XC;
                    if (i >= L::NST) ok = wait_bar(empty(st, x), (uint32_t)(i / L::NST - 1) & 1u, limit, s_abort);
                    if (!ok) break;
                    const CUtensorMap *tm = x == XB_ ? &tmb : x == XC ? &tmc : &tma;
                    mbar_expect_tx(full(st, x), L::TILE);
                    tma_load_3d(tile(st, x), tm, 0, y, (int)chain, full(st, x));
                    if (D == 128) tma_load_3d(tile(st, x) + HALF, tm, 64, y, (int)chain, full(st, x));
                    ++issued;
                }
            }
            if (!ok) fail_now();
            // never leave a copy in flight into this CTA's shared memory
            for (int t = issued > L::NST * L::NT ? issued - L::NST * L::NT : 0; t < issued; ++t) {
                const int i = t / L::NT, x0 = t % L::NT;
                const int x = PRE ? x0 : x0 == 0 ? XB_ : x0 == 1 ? XA : XC;
                mbar_wait(full(i % L::NST, x), (uint32_t)(i / L::NST) & 1u, kDrainNs);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- G, P C
        if (!PRE && lane == 0) {
            bool ok = true;
            for (int i = 0; i < nch; ++i) {
                const int st = i % L::NST;
                const uint32_t ph = (uint32_t)(i / L::NST) & 1u, pi = (uint32_t)i & 1u;
                ok = wait_bar(full(st, XB_), ph, limit, s_abort) &&
                     wait_bar(full(st, XA), ph, limit, s_abort) &&
                     (tokens(i) == C || wait_bar(bar(L::VZ), 0, limit, s_abort)) &&
                     (i == 0 || wait_bar(bar(L::PVDONE), pi ^ 1u, limit, s_abort));
                if (!ok) break;
                tc_fence_after();
                {
                    constexpr uint32_t id = idesc_bf16(128, 128, false, false);
                    const uint64_t da = sdesc_sw128(tile(st, XA), 16, 1024);
                    const uint64_t db = sdesc_sw128(tile(st, XB_), 16, 1024);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t off = ((kk >> 2) * HALF + (kk & 3) * 32u) >> 4;
                        mma_bf16(tmem + COL_G, da + off, db + off, id, kk > 0);
                    }
                    mma_commit(bar(L::GDONE));
                    mma_commit(empty(st, XB_));
                }
                ok = wait_bar(bar(L::PRDY), pi, limit, s_abort) &&
                     wait_bar(full(st, XC), ph, limit, s_abort) &&
                     wait_bar(bar(L::OSC), pi, limit, s_abort);
                if (!ok) break;
                tc_fence_after();
                {
                    constexpr uint32_t id = idesc_bf16(128, D, false, true);
                    const uint64_t dc = sdesc_sw128(tile(st, XC), HALF, 1024);
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk)
                        mma_bf16_ta(tmem + COL_O, tmem + COL_G + 8 * kk, dc + kk * 128, id, 1);
                    mma_commit(bar(L::PVDONE));
                    mma_commit(empty(st, XC));
                }
            }
            if (!ok) fail_now();
            if (nch > 0) {
                mma_commit(bar(L::DRAIN0));
                mbar_wait(bar(L::DRAIN0), 0, kDrainNs);
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---------------------------------------------------------------- A X, state update
        if (lane == 0) {
            bool ok = true;
            for (int i = 0; i < nch; ++i) {
                const int st = i % L::NST;
                const uint32_t ph = (uint32_t)(i / L::NST) & 1u, pi = (uint32_t)i & 1u;
                if (!PRE) {
                    ok = wait_bar(full(st, XA), ph, limit, s_abort) &&
                         wait_bar(bar(L::XBRDY), pi, limit, s_abort) &&
                         (i == 0 || wait_bar(bar(L::OFREE), pi ^ 1u, limit, s_abort));
                    if (!ok) break;
                    tc_fence_after();
                    constexpr uint32_t id = idesc_bf16(128, D, false, true);
                    const uint64_t da = sdesc_sw128(tile(st, XA), 16, 1024);
                    const uint64_t dx = sdesc_sw128(sb + L::XB, HALF, 1024);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_bf16(tmem + COL_O, da + (((kk >> 2) * HALF + (kk & 3) * 32u) >> 4),
                                 dx + kk * 128, id, kk > 0);
                    mma_commit(bar(L::QSDONE));
                }
                ok = wait_bar(full(st, XC), ph, limit, s_abort) &&
                     wait_bar(bar(L::XSC), pi, limit, s_abort);
                for (int u = 0; u < 4 && ok; ++u) {
                    const int b = u & 1;
                    ok = wait_bar(bar(L::KRDY + b), (uint32_t)(2 * i + (u >> 1)) & 1u, limit, s_abort);
                    if (!ok) break;
                    tc_fence_after();
                    constexpr uint32_t id = idesc_bf16(128, D, false, true);
                    const uint64_t dc = sdesc_sw128(tile(st, XC), HALF, 1024);
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                        for (int term = 0; term < 3; ++term)
                            mma_bf16_ta(tmem + COL_X, tmem + COL_K + KBUF * b + 16 * term + 8 * kk,
                                        dc + (2 * u + kk) * 128, id, 1);
                    mma_commit(bar(L::KFREE + b));
                }
                if (!ok) break;
                mma_commit(bar(L::XDONE));
                mma_commit(empty(st, XC));
            }
            if (!ok) fail_now();
            if (nch > 0) {
                mma_commit(bar(L::DRAIN1));
                mbar_wait(bar(L::DRAIN1), 0, kDrainNs);
            }
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // ---------------------------------------------------------------- P
        if (!PRE) {
            const int w = warp & 3, row = w * 32 + lane;
            const uint32_t lb = (uint32_t)(w * 32) << 16;
            bool ok = true;
            for (int i = 0; i < nch; ++i) {
                const int nv = tokens(i);
                ok = __all_sync(~0u, wait_bar(bar(L::GDONE), (uint32_t)i & 1u, limit, s_abort));
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int jb = 0; jb < 8; ++jb) {     // 16 columns j
                    float v[16];
                    uint32_t pk[8];
                    const int blk = jb >> 1;         // against this warp's 32 rows
                    if (REV ? blk < w : blk > w) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) pk[e] = 0u;
                    } else {
                        tmem_ld16(tmem + lb + COL_G + 16 * jb, v);
                        if (blk == w) {              // the diagonal block: one power an element
                            const int lag0 = REV ? 16 * jb - row : row - 16 * jb;
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const int lag = REV ? lag0 + e : lag0 - e;
                                v[e] = lag >= 0 ? v[e] * (a.in_scale * pw[lag < 0 ? 0 : lag]) : 0.f;
                            }
                        } else {                     // g^|i-j| = g^(to the block's edge) g^(in it)
                            const float f = a.in_scale * pw[REV ? 16 * jb - row : row - 16 * jb - 15];
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const float4 u = *reinterpret_cast<const float4 *>(pr + e);
                                mul2(v[e], v[e + 1], f, f);
                                mul2(v[e + 2], v[e + 3], f, f);
                                mul2(v[e], v[e + 1], u.x, u.y);
                                mul2(v[e + 2], v[e + 3], u.z, u.w);
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) pk[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
                    }
                    tmem_st8(tmem + lb + COL_G + 8 * jb, pk);   // over columns already read
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::PRDY));
            }
            if (!ok && lane == 0) fail_now();
        }
    } else if (warp >= 8 && warp < 12) {
        // ---------------------------------------------------------------- O
        if (!PRE) {
            const int w = warp & 3, row = w * 32 + lane;
            const uint32_t lb = (uint32_t)(w * 32) << 16;
            bool ok = true;
            for (int i = 0; i < nch; ++i) {
                const uint32_t pi = (uint32_t)i & 1u;
                const int nv = tokens(i);
                ok = __all_sync(~0u, wait_bar(bar(L::QSDONE), pi, limit, s_abort));
                if (!ok) break;
                tc_fence_after();
                const float rd = pw[REV ? (row < nv ? nv - 1 - row : 0) : row + 1];
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    float v[16];
                    tmem_ld16(tmem + lb + COL_O + c, v);
#pragma unroll
                    for (int e = 0; e < 16; e += 2) mul2(v[e], v[e + 1], rd, rd);
                    tmem_st16(tmem + lb + COL_O + c, v);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::OSC));

                ok = __all_sync(~0u, wait_bar(bar(L::PVDONE), pi, limit, s_abort));
                if (!ok) break;
                tc_fence_after();
                float mean = 0.f, rstd = a.out_scale;
                if (NORM) {                          // a thread holds its whole row
                    float s = 0.f;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float v[32];
                        tmem_ld32(tmem + lb + COL_O + c, v);
#pragma unroll
                        for (int e = 0; e < 32; ++e) s += v[e];
                    }
                    mean = s / D;                    // of the unscaled row
                    s = 0.f;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float v[32];
                        tmem_ld32(tmem + lb + COL_O + c, v);
#pragma unroll
                        for (int e = 0; e < 32; ++e) s = fmaf(v[e] - mean, v[e] - mean, s);
                    }
                    rstd = a.out_scale * rsqrtf(a.out_scale * a.out_scale * (s / D) + a.norm.eps);
                }
                // G and A X have read this chunk's A tile: the rows are staged over it and leave
                // by a tensor store a warp (whole rows), or one by one at a sequence's end
                const bool whole = w * 32 + 32 <= nv;
                const int st = i % L::NST;
                const int64_t row0 = (int64_t)chunk_id(i) * C;
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) +
                                     (chain * a.T + row0 + row) * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    float v[16];
                    tmem_ld16(tmem + lb + COL_O + c, v);
                    if (NORM) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = (v[e] - mean) * rstd;
                        if (a.norm.weight)
#pragma unroll
                            for (int e = 0; e < 16; ++e) v[e] *= __ldg(a.norm.weight + c + e);
                        if (a.norm.bias)
#pragma unroll
                            for (int e = 0; e < 16; ++e) v[e] += __ldg(a.norm.bias + c + e);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) mul2(v[e], v[e + 1], rstd, rstd);
                    }
#pragma unroll
                    for (int e = 0; e < 16; e += 8) {
                        const uint4 o4 = make_uint4(pack_bf16(v[e], v[e + 1]), pack_bf16(v[e + 2], v[e + 3]),
                                                    pack_bf16(v[e + 4], v[e + 5]), pack_bf16(v[e + 6], v[e + 7]));
                        if (whole)
                            st_shared_v4(tile(st, XA) + (uint32_t)(c >> 6) * HALF +
                                             sw128(row, ((uint32_t)(c + e) & 63u) >> 3),
                                         o4.x, o4.y, o4.z, o4.w);
                        else if (row < nv)
                            *reinterpret_cast<uint4 *>(out + c + e) = o4;
                    }
                }
                tc_fence_before();
                if (whole) fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(L::OFREE));
                    if (whole) {
                        const uint32_t src = tile(st, XA) + (uint32_t)w * 4096u;
                        tma_store_3d(&tmo, src, 0, (int)row0 + w * 32, (int)chain);
                        if (D == 128) tma_store_3d(&tmo, src + HALF, 64, (int)row0 + w * 32, (int)chain);
                        bulk_commit();
                        bulk_wait_read0();
                    }
                    mbar_arrive(empty(st, XA));
                }
            }
            if (lane == 0) bulk_wait0();
            if (!ok && lane == 0) fail_now();
        }
    } else if (warp >= 12 && warp < 16) {
        // ---------------------------------------------------------------- (diag(w) B)^T
        const int w = warp & 3;
        const uint32_t lb = (uint32_t)(w * 32) << 16;
        const bool mine = w * 32 < D;
        bool ok = true;
        for (int i = 0; i < nch; ++i) {
            const int st = i % L::NST;
            const uint32_t ph = (uint32_t)(i / L::NST) & 1u;
            const int nv = tokens(i);
            const bool tail = nv < C;
            ok = __all_sync(~0u, wait_bar(full(st, XB_), ph, limit, s_abort));
            if (!ok) break;
            const float *wt = kw;
            if (tail) {
                // rows behind the end may hold anything: those of B and C become zero before any
                // product reads them (and the weights too; every warp writes the same values)
                for (int j = lane; j < C; j += 32)
                    kt[j] = j < nv ? a.in_scale * pw[REV ? j + 1 : nv - 1 - j] : 0.f;
                ok = __all_sync(~0u, wait_bar(full(st, XC), ph, limit, s_abort));
                if (!ok) break;
                for (int j = nv + w; j < C; j += 4)
                    for (int x = lane; x < D / 4; x += 32) {   // D / 8 pieces of B, as many of C
                        const uint32_t y = (uint32_t)x % (D / 8);
                        st_shared_v4(tile(st, x < D / 8 ? XB_ : XC) + (y >> 3) * HALF + sw128(j, y & 7),
                                     0, 0, 0, 0);
                    }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::VZ));
                // each warp reads rows that the others cleared
                ok = __all_sync(~0u, wait_bar(bar(L::VZ), 0, limit, s_abort));
                if (!ok) break;
                wt = kt;
            }
            // ldmatrix x4: matrices (tokens +0, +8) x (rows +0, +8) of X, 16 rows a half-warp
            const uint32_t r8 = (uint32_t)lane & 7u, m = (uint32_t)lane >> 3;
            for (int u = 0; u < 4; ++u) {
                const int b = u & 1;
                const int use = 2 * i + (u >> 1);    // of this buffer
                if (use > 0) ok = __all_sync(~0u, wait_bar(bar(L::KFREE + b), (uint32_t)(use - 1) & 1u, limit, s_abort));
                if (!ok) break;
                tc_fence_after();
                if (mine) {
                    // thread t: tokens 32 u + 8 c + 2 (t % 4), +1 for c = 0..3
                    float2 wv[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        wv[c] = *reinterpret_cast<const float2 *>(wt + 32 * u + 8 * c + 2 * (lane & 3));
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {    // rows w * 32 + 16 h .. +15 of X
                        uint32_t hi[8], mid[8], lo[8];
#pragma unroll
                        for (int t2 = 0; t2 < 2; ++t2) {   // tokens 32 u + 16 t2 .. +15
                            const uint32_t row = 32u * u + 16u * t2 + 8u * (m >> 1) + r8;
                            const uint32_t dd = (uint32_t)w * 32u + 16u * h + 8u * (m & 1u);
                            uint32_t k2[4];          // (tokens 0-7, rows 0-7), (0-7, 8-15), (8-15, 0-7), ..
                            ldmatrix_x4_trans(tile(st, XB_) + (dd >> 6) * HALF + sw128(row, (dd & 63u) >> 3), k2);
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                const int c = 2 * t2 + (z >> 1), o = 2 * c + (z & 1);
                                float x0 = __uint_as_float(k2[z] << 16);
                                float x1 = __uint_as_float(k2[z] & 0xffff0000u);
                                mul2(x0, x1, wv[c].x, wv[c].y);
                                hi[o] = top_halves(x0, x1);
                                below(x0, x1);
                                mid[o] = top_halves(x0, x1);
                                below(x0, x1);
                                lo[o] = top_halves(x0, x1);
                            }
                        }
                        const uint32_t at = tmem + lb + ((uint32_t)(16 * h) << 16) + COL_K + KBUF * b;
                        tmem_st_16x128b_x4(at, hi);
                        tmem_st_16x128b_x4(at + 16, mid);
                        tmem_st_16x128b_x4(at + 32, lo);
                    }
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(L::KRDY + b));
                    if (u == 3) mbar_arrive(empty(st, XB_));
                }
            }
            if (!ok) break;
        }
        if (!ok && lane == 0) fail_now();
    } else if (warp >= 16) {
        // ---------------------------------------------------------------- X
        const int w = warp & 3, d = w * 32 + lane;
        const uint32_t lb = (uint32_t)(w * 32) << 16;
        const bool mine = w * 32 < D;
        const float *X0 = a.X0 ? a.X0 + chain * D * D : nullptr;
        // with S_T = S0 the last segment may finish before another starts: they read a copy
        const bool copy = nseg > 1 && a.X0 && a.X_out == a.X0;
        const float *src0 = !PRE && copy ? ws + (int64_t)(nseg - 1) * D * D : X0;
        bool ok = true;
        // the state on entry, 16 columns at a time
        auto entry = [&](int c, float *v) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.f;
            if (seg == 0) {
                if (src0) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        v[e] = a.x0_trans ? src0[(int64_t)(c + e) * D + d] : src0[(int64_t)d * D + c + e];
                }
            } else if (!PRE) {
                for (int r = 0; r < seg; ++r) {
                    const Seg q = seg_of(n, r, nseg);
                    if (q.first >= q.last && r > 0) continue;
                    const float g = r == 0 ? 0.f : decay_pow(lg, (float)seg_tokens<REV>(n, q));
                    const float *M = ws + (int64_t)r * D * D + d * D + c;
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 m = *reinterpret_cast<const float4 *>(M + e);
                        v[e] = r == 0 ? m.x : fmaf(g, v[e], m.x);
                        v[e + 1] = r == 0 ? m.y : fmaf(g, v[e + 1], m.y);
                        v[e + 2] = r == 0 ? m.z : fmaf(g, v[e + 2], m.z);
                        v[e + 3] = r == 0 ? m.w : fmaf(g, v[e + 3], m.w);
                    }
                }
            }
        };
        float *dst = PRE ? ws + (int64_t)seg * D * D : final_seg ? a.X_out ? a.X_out + chain * D * D : nullptr : nullptr;
        auto put_row = [&](float *base, int c, const float *v) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<float4 *>(base + (int64_t)d * D + c + e) =
                    make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        };
        auto put_copy = [&](int c, const float *v) {   // bf16, rows of X: B operand of A X
#pragma unroll
            for (int e = 0; e < 16; e += 8)
                st_shared_v4(sb + L::XB + (uint32_t)((c + e) >> 6) * ((uint32_t)D * 128u) +
                                 sw128(d, ((uint32_t)(c + e) & 63u) >> 3),
                             pack_bf16(v[e], v[e + 1]), pack_bf16(v[e + 2], v[e + 3]),
                             pack_bf16(v[e + 4], v[e + 5]), pack_bf16(v[e + 6], v[e + 7]));
        };
        if (nch == 0) {                              // no tokens: the state passes through
            if (mine)
                for (int c = 0; c < D; c += 16) {
                    float v[16];
                    entry(c, v);
                    if (dst) put_row(dst, c, v);
                    if (PRE && copy) put_row(ws + (int64_t)(nseg - 1) * D * D, c, v);
                }
        }
        for (int i = 0; i < nch; ++i) {
            const float g = pw[tokens(i)];
            if (i > 0) {
                ok = __all_sync(~0u, wait_bar(bar(L::XDONE), (uint32_t)(i - 1) & 1u, limit, s_abort) &&
                                         (PRE || wait_bar(bar(L::QSDONE), (uint32_t)(i - 1) & 1u, limit, s_abort)));
                if (!ok) break;
                tc_fence_after();
            }
            if (mine) {
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    float v[16];
                    if (i > 0) {
                        tmem_ld16(tmem + lb + COL_X + c, v);
                    } else {
                        entry(c, v);
                        if (PRE && copy) put_row(ws + (int64_t)(nseg - 1) * D * D, c, v);
                    }
                    if (!PRE) put_copy(c, v);
#pragma unroll
                    for (int e = 0; e < 16; e += 2) mul2(v[e], v[e + 1], g, g);
                    tmem_st16(tmem + lb + COL_X + c, v);
                }
                tmem_st_wait();
                tc_fence_before();
                if (!PRE) fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0) {
                if (!PRE) mbar_arrive(bar(L::XBRDY));
                mbar_arrive(bar(L::XSC));
            }
        }
        if (ok && nch > 0 && dst) {
            ok = __all_sync(~0u, wait_bar(bar(L::XDONE), (uint32_t)(nch - 1) & 1u, limit, s_abort));
            if (ok && mine) {
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    float v[16];
                    tmem_ld16(tmem + lb + COL_X + c, v);
                    put_row(dst, c, v);
                }
                tc_fence_before();
            }
        }
        if (!ok && lane == 0) fail_now();
    }

    __syncthreads();
    tc_fence_after();
    if (warp == 3) tmem_dealloc(tmem, TMEM_COLS);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// [n_chains][T][d] bf16 as a 3-D tensor (d, T, chain), boxes of 64 columns and `rows` rows: rows
// behind T read as zero.
bool make_map(CUtensorMap *m, const void *ptr, int64_t T, int64_t nc, int d, int rows = C) {
    auto enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)nc};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)T * d * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)rows, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box,
               es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Segments of each chain: as many as fill the GPU with one CTA an SM, none shorter than
// kMinSegChunks chunks (a segment's state is read back from memory by the ones behind it).
int segments(int64_t n_chains, int64_t T) {
    const int64_t chunks = (T + C - 1) / C;
    int64_t s = kSMs / n_chains;
    if (s > chunks / kMinSegChunks) s = chunks / kMinSegChunks;
    return s < 1 ? 1 : (int)s;
}

template <int D, bool REV>
cudaError_t launch(const ScanArgs &a, cudaStream_t s) {
    CUtensorMap ta, tb, tc, to;
    if (!make_map(&ta, a.a, a.T, a.n_chains, D) || !make_map(&tb, a.b, a.T, a.n_chains, D) ||
        !make_map(&tc, a.c, a.T, a.n_chains, D) || !make_map(&to, a.out, a.T, a.n_chains, D, 32))
        return cudaErrorInvalidValue;
    const int nseg = segments(a.n_chains, a.T);
    cudaError_t e;
    if (nseg > 1) {
        auto k = scan_tc_kernel<D, REV, true, false>;
        constexpr int smem = (int)Lay<D, true>::ALLOC;
        if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
            return e;
        k<<<(unsigned)(a.n_chains * (nseg - 1)), NTHREADS, smem, s>>>(ta, tb, tc, to, a, nseg);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    auto k = a.norm.on ? scan_tc_kernel<D, REV, false, true> : scan_tc_kernel<D, REV, false, false>;
    constexpr int smem = (int)Lay<D, false>::ALLOC;
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
        return e;
    k<<<(unsigned)(a.n_chains * nseg), NTHREADS, smem, s>>>(ta, tb, tc, to, a, nseg);
    return cudaGetLastError();
}

}  // namespace

size_t scan_tc_workspace(int64_t n_chains, int64_t T, int d) {
    const int nseg = segments(n_chains, T);
    return nseg > 1 ? (size_t)n_chains * nseg * d * d * sizeof(float) : 0;
}

cudaError_t launch_scan_tc(const ScanArgs &a, cudaStream_t s) {
    if (a.d == 64) return a.rev ? launch<64, true>(a, s) : launch<64, false>(a, s);
    return a.rev ? launch<128, true>(a, s) : launch<128, false>(a, s);
}

}  // namespace fw
