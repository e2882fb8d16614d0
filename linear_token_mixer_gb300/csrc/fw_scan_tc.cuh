// fw_scan_tc.cuh -- the kernel of the decayed (fw_decay.cuh) and selective (fw_select.cuh) scans for bf16
// rows on the fifth-generation tensor cores, d = 64 and 128, in chunks of 128 tokens.  It is compiled
// for the one by fw_decay_tc.cu and for the other, SEL, by fw_select_tc.cu.
//
// Per chunk of n valid rows, with the state X on entry (forward; the reverse scan swaps the
// exponents as in fw_decay.cuh):
//     G = A B^T                                     128 x 128 x d
//     P = mask . g^|i-j| . G          (bf16)
//     O = diag(g^(i+1)) (A X) + P C                 128 x d x d, 128 x d x 128
//     X <- g^n X + (diag(w) B)^T C                  d x d x 128, three times
// The last product's left operand is split into bf16 terms, each cut towards zero, so that the fp32 state
// loses nothing to its operands: three (less than 2^-23 of w_j b_j is cut) where a state is returned, two
// (less than 2^-15 at most, 7e-6 on average, and always towards zero) where it is only read into bf16
// rows.  (Two terms for chunks of which e^-3.5 or less is left in the returned state, as if every chunk
// wrote as much, left states whose last tokens write little 1e-5 off; without them B8 H16 T4096 d = 128 takes
// 105.7 us for 103.1.)  P and
// the copy of X that A reads are rounded to bf16 once, like the output rows.
//
// One CTA per chain, or per segment of a chain where chains are few, warp-specialised:
//   warp 0       TMA producer: tiles of B, A, C (128 x d, 128-byte swizzle), each released on
//                its own
//   warp 1       MMA issuer of G and P C
//   warp 2       MMA issuer of the state update
//   warp 3       MMA issuer of A X; tensor-memory allocation
//   warps 4-7    P: tensor memory -> mask, decay, bf16 -> tensor memory (A operand of P C)
//   warps 8-11   O: its rows' decay [, output norm], rounded and stored (one thread a row); of a
//                steep head A X is scaled in place before P C accumulates on it
//   warps 12-15, 24-27  the three terms of (diag(w) B)^T, 32 tokens at a time, into tensor
//                memory, a buffer for each four warps (a segment's state alone: 4-11 too)
//   warps 16-23  X, in registers (fp32, half a row a thread): X <- g^n X + the chunk's update,
//                and its bf16 shared-memory copy for A X
// The update of a chunk is summed from zero in tensor memory and added to X by an fp32 FMA: the
// MMAs round towards zero, and X would carry that bias from chunk to chunk.  It also takes the
// MMAs of the update off the state's serial chain (update read -> copy -> A X).
// Measured (one GB300): B8 H16 T4096 d = 128, 128 chains, 545 MB of rows and states: 105.6 us, 5.2
// TB/s, 76 % of the measured copy rate; B1 H32 T32768, four segments a chain: 318 us, of which the
// states of the segments, read again, are a third.  What bounds it is the period of a chunk, 2.8 us (d = 64:
// 2.05 us), in one CTA, and 10 us for its start: at T2048 the tensor pipe is busy for 38 % of the time, the
// issue slots for 38 %, DRAM at 55 %, and the rest is the roles' round trips through tensor memory and barriers.  A second CTA an
// SM would fill it but finds no room: the tiles take 192 KB, G, O and the update 384 columns.
// Tensor memory: G (P over it) 128 columns, O 128, the update 128, the split operand 2 x 48.
// SEL: the decays come from tables in memory (SelectTables), by token and chunk, in place of powers of one; a CTA
// forms those of its chunks before it begins, while the first tiles load.  (A launch of their own: 5 us a call.)  The
// scores of a steep chunk take the product of the decays to and from the end of the block of 32 columns before
// a row's own, each at most 1; those of the diagonal blocks the quotient of the decays from the block's start, or
// where that is below e^-kMild the decay itself.  Whether a chunk is mild goes by its own tables.  skip v is added to a row in
// the epilogue, in fp32, from the tile of C that P C has read, so that it is rounded with the row and never before (on the
// scores' diagonal it was, and skip / scale times the factors there could overflow); calls without it are a kernel of
// their own.  Measured: B8 H16 T4096 d = 128, keys and queries for each head, 128 us (mild chunks 125, steep ones 131;
// 125, 121 and 125 without skip; without SEL 101 and 113), with those of one group 128 us; B16 d = 64 193 us, 187 without
// skip: not its bytes (80 and 43 us at the measured copy rate) but the period of a chunk, 3.4 us.
// What that goes by is all roles' instructions rather than one chain: of 126 us (with skip v on the diagonal) the third term
// of the update was 15, P 23, X 14, a branch that no chunk takes 10, and one warp of nine stalls for instructions (tensor
// pipe 39 % busy, issue slots 47 %, DRAM 44 % at T2048).  B1 H32 T32768 397 us.
// Every wait is bounded; on expiry the kernel records an error, the other roles stop at their
// next wait, copies and MMAs in flight are drained, tensor memory is freed and the kernel exits.
#pragma once

#include <cuda.h>

#include "fw_decay_tc.cuh"
#include "fw_select.cuh"
#include "fw_sm100.cuh"
#include "fw_tma.cuh"

namespace fw {
namespace {
using namespace sm100;

constexpr int C = 128;
constexpr int NTHREADS = 896;
constexpr uint32_t KB = 1024;
constexpr uint32_t HALF = 16 * KB;           // 128 rows x 128 bytes: 64 columns of a tile
// The launches of a call overlap (programmatic dependent launch).  A segment kernel's successor
// waits for it before it begins; a scan that follows an independent one takes the SMs as they come
// free and waits for it only before it ends, so that the last grid to end is the last of all.
constexpr int kWaitFirst = 1, kWaitLast = 2;
constexpr int kMaxRanked = 64;               // batch rows ranked by length (every CTA reads them all)

// Registers a thread: 72 for each of the seven warpgroups at launch; P and O keep them, warps 0-3
// and the split-operand groups hand theirs on to the two groups that hold X.
constexpr int REGS = 72, REGS_W0 = 40, REGS_K = 64, REGS_X = 96;
static_assert(REGS_W0 + 2 * REGS + 2 * REGS_K + 2 * REGS_X <= 7 * REGS, "registers of the launch");
constexpr uint32_t COL_G = 0, COL_O = 128, COL_U = 256, KBUF = 48;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint64_t kDrainNs = 2000000000ull;

template <int D, bool PRE, bool SEL> struct Lay {
    static constexpr uint32_t TILE = (uint32_t)C * D * 2;
    static constexpr int NT = PRE ? 2 : 3;                       // tiles per stage
    // split-operand groups, a tensor-memory buffer each (a state alone leaves room for four)
    static constexpr int KG = PRE ? 4 : 2;
    static constexpr uint32_t COL_K = PRE ? 0 : 384;
    static constexpr int UB = PRE ? 2 : 1;                       // buffers of the update
    static constexpr int NST = (int)(192 * KB / (TILE * NT));    // 2 (3), d = 64: 4 (6)
    static constexpr uint32_t XB = NST * NT * TILE;              // bf16 copy of X
    static constexpr uint32_t TAB = XB + (uint32_t)D * D * 2;
    static constexpr uint32_t T_PW = TAB, T_KW = T_PW + 132 * 4, T_KT = T_KW + 128 * 4;
    // SEL, of the P group: a steep chunk's decays to the ends of blocks (a mild one's from the
    // chunk's start), logs, steps
    static constexpr uint32_t T_SF = TAB, T_SC = T_SF + 192 * 4, T_SD = T_SC + 128 * 4;
    static constexpr uint32_t BAR = !SEL ? T_KT + 128 * 4 : PRE ? TAB : T_SD + 128 * 4;
    // barriers
    static constexpr int FULL = 0, EMPTY = FULL + NST * NT, GDONE = EMPTY + NST * NT,
                         PRDY = GDONE + 1, QSDONE = PRDY + 1, OSC = QSDONE + 1, PVDONE = OSC + 1,
                         OFREE = PVDONE + 1, UDONE = OFREE + 1, XBRDY = UDONE + UB,
                         UFREE = XBRDY + 1, KRDY = UFREE + UB, KFREE = KRDY + KG, VZ = KFREE + KG,
                         DRAIN = VZ + 1, NEVER = DRAIN + 3,
                         NBAR = NEVER + 1;
    static constexpr uint32_t MISC = BAR + NBAR * 8;
    static constexpr uint32_t BYTES = MISC + 16;
    static constexpr uint32_t ALLOC = BYTES + 1024;
    static_assert(ALLOC <= 227 * KB, "shared memory budget");
};

__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint64_t limit,
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

template <int N> __device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
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
template <bool REV>
__device__ __forceinline__ int64_t seg_tokens(int64_t n, const Seg &s) {
    if (s.first >= s.last) return 0;
    const int64_t full = (int64_t)(s.last - s.first) * C;
    const bool tail = REV ? s.first == 0 : s.last == s.total;
    return tail ? full - ((int64_t)s.total * C - n) : full;
}

__device__ __forceinline__ void bar_arrive(int id, int count) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// Four 8x8 b16 matrices, transposed: thread t gets rows 2 (t % 4), +1 of column t / 4.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Sixteen columns of tensor memory into registers that may be read only after tmem_landed().
__device__ __forceinline__ void tmem_fetch16(uint32_t taddr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_landed(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                   "+f"(v[15])::"memory");
}
// do_(v, c) for the columns c = c0, c0 + 16, .. < c1 of this warp's lanes.  (One load at a time:
// seven roles share the instruction cache, and with their loops twice as long, the next load in flight,
// B8 H16 T4096 d = 128 took 107.6 us for 102.5.)
template <typename F> __device__ __forceinline__ void tmem_stream(uint32_t taddr, int c0, int c1, F do_) {
    float v[16];
#pragma unroll 1
    for (int c = c0; c < c1; c += 16) {
        tmem_fetch16(taddr + c, v);
        tmem_landed(v);
        do_(v, c);
    }
}

__device__ __forceinline__ void tmem_ld4(uint32_t taddr, float (&v)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(taddr)
                 : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3])::"memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const float (&v)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3])
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

__device__ __forceinline__ void scale2(float &a0, float &a1, uint64_t b) {
    const float2 f = halves(mul2(pair(a0, a1), b));
    a0 = f.x;
    a1 = f.y;
}

// bf16 (truncated) of a pair, the first in the low half, and what the truncation drops (exact).
__device__ __forceinline__ uint32_t top_halves(uint64_t x) {
    return __byte_perm((uint32_t)x, (uint32_t)(x >> 32), 0x7632);
}
__device__ __forceinline__ uint64_t below(uint64_t x) {
    return fma2(x & 0xffff0000ffff0000ull, pair(-1.f, -1.f), x);
}

// The scans of a launch: one forward, or two reverse ones (dv and dk) over the same rows, whose CTAs
// of a chain are neighbours.  Both read q and do, and the second of them finds the tiles in L2 (B8 H16
// T2048 d = 128 backward 153 us in launches of their own, 151 us).
template <int N> struct Jobs {
    struct {
        CUtensorMap a, b, c, out;
        ScanArgs args;
    } s[N];
};

// SEL: the decay of chunks [first, last) of a chain, by a whole warp.
__device__ __forceinline__ float chunks_decay(const SelectTables &t, int64_t chain, int first, int last) {
    double x = 0.0;
    for (int c = first + (int)(threadIdx.x & 31); c < last; c += 32) {
        x += t.chunk[chain * t.n_chunks + c].y;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    const float hi = (float)x;
    return exp_two(hi, (float)(x - hi));
}

// The state on entry to segment `seg` of `nseg`, element (r, c) of a chain's: X0 (or its copy, which is never
// transposed), or the states of the segments before it added up.  `ws`: the chain's workspace.
template <int D, bool REV>
__device__ __forceinline__ float entry_state(const ScanArgs &a, const ScanArgs &own, const float *ws, int64_t chain,
                                             int64_t n, int seg, int nseg, int r, int c) {
    if (seg == 0) {
        if (!a.X0) return 0.f;
        if (nseg > 1 && own.X_out == a.X0) return ws[(int64_t)(nseg - 1) * D * D + r * D + c];
        const float *X0 = a.X0 + chain * D * D;
        return own.x0_trans ? X0[c * D + r] : X0[r * D + c];
    }
    float x = 0.f;
#pragma unroll 1
    for (int s = 0; s < seg; ++s) {
        const Seg q = seg_of(n, s, nseg);
        if (q.first >= q.last && s > 0) continue;
        x = fmaf(decay_pow(a.log_decay[chain % a.H], (float)seg_tokens<REV>(n, q)), x,
                 ws[(int64_t)s * D * D + r * D + c]);
    }
    return x;
}

// SEL: the tables of a chunk, four tokens a lane; by a whole warp.  Logs are summed within blocks of 32 tokens and over
// the blocks, for the weights from the chunk's end: what counts are short sums, which lose nothing to tokens far off that keep
// nothing (logs of 104 each, 1e4 in a chunk).  Of a chunk that is not mild the sums of a block go on in two terms and are
// rounded once, so that a difference of two is off by a unit of the larger: 1.5e-5 for logs of 200 in a block, 2.5e-4 at
// most (32 tokens that keep nothing).
__device__ __forceinline__ void form_tables(const ScanArgs &a, int64_t chain, int64_t n, int64_t chunk) {
    constexpr int PER = C / 32, LANES = 32 / PER;   // of a block
    const GateArgs &g = a.sel.gate;
    const int lane = threadIdx.x & 31, h = (int)(chain % a.H), place = lane % LANES, block = lane / LANES;
    const int64_t first = chunk * C + lane * PER, id = chain * a.sel.n_chunks + chunk;
    const float rate = g.log_decay[h];
    float dt[PER], x[PER], sum = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const bool on = first + e < n;
        dt[e] = on ? step_of(g, chain * a.T + first + e, h) : 0.f;
        x[e] = on ? rate * dt[e] : 0.f;
        if (x[e] < -kReset) x[e] = -kReset;   // (NaN stays)
        sum += x[e];
    }
    float upto = sum, from = sum;             // of this lane's tokens and those before, and behind, in the block
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
        const float p = __shfl_up_sync(~0u, upto, o, LANES), q = __shfl_down_sync(~0u, from, o, LANES);
        if (place >= o) upto += p;
        if (place < LANES - o) from += q;
    }
    float all[4];                             // of the blocks
#pragma unroll
    for (int b = 0; b < 4; ++b) all[b] = __shfl_sync(~0u, from, LANES * b);
    const float total = all[0] + all[1] + all[2] + all[3];
    float start = 0.f, rest = 0.f;            // of the blocks before, and behind
#pragma unroll
    for (int b = 0; b < 3; ++b) {
        if (block > b) start += all[b];
        if (block < 3 - b) rest += all[3 - b];
    }
    float before = __shfl_up_sync(~0u, upto, 1, LANES), behind = __shfl_down_sync(~0u, from, 1, LANES);
    if (place == 0) before = 0.f;
    if (place == LANES - 1) behind = 0.f;
    float w[PER];
#pragma unroll
    for (int e = PER - 1; e >= 0; --e) {
        w[e] = dt[e] * expf(behind + rest);
        behind += x[e];
    }
    float low = 0.f, high = 0.f, sums[PER];   // from the chunk's start: the least and the largest, and each token's
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        before += x[e];
        sums[e] = start + before;
        low = fminf(low, sums[e]);
        high = fmaxf(high, sums[e]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        low = fminf(low, __shfl_xor_sync(~0u, low, o));
        high = fmaxf(high, __shfl_xor_sync(~0u, high, o));
    }
    const bool one = low >= -kMild && high <= kMild && isfinite(total);
    if (!one) {                               // (the whole warp)
        Two s[PER], all_before{0.f, 0.f};
#pragma unroll
        for (int e = 0; e < PER; ++e) s[e] = add(e ? s[e - 1] : all_before, Two{x[e], 0.f});
        Two t = s[PER - 1];
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) {
            const Two p{__shfl_up_sync(~0u, t.hi, o, LANES), __shfl_up_sync(~0u, t.lo, o, LANES)};
            if (place >= o) t = add(p, t);
        }
        const Two p{__shfl_up_sync(~0u, t.hi, 1, LANES), __shfl_up_sync(~0u, t.lo, 1, LANES)};
        if (place > 0) all_before = p;
#pragma unroll
        for (int e = 0; e < PER; ++e) sums[e] = add(all_before, s[e]).hi;
#pragma unroll
        for (int b = 0; b < 3; ++b) all[b] = __shfl_sync(~0u, sums[PER - 1], LANES * b + LANES - 1);
    }
    float4 *const c = reinterpret_cast<float4 *>(a.sel.c + id * C + lane * PER);
    c[0] = make_float4(sums[0], dt[0], sums[1], dt[1]);
    c[1] = make_float4(sums[2], dt[2], sums[3], dt[3]);
#pragma unroll
    for (int e = 0; e < PER; e += 2)
        *reinterpret_cast<float2 *>(a.sel.w + id * C + weight_place(lane * PER + e)) = make_float2(w[e], w[e + 1]);
    if (lane == 0) {
        a.sel.chunk[id] = make_float2(expf(total), total);
        a.sel.ends[id] = make_float4(all[0], all[1], all[2], one ? 1.f : 0.f);
    }
}

__device__ __forceinline__ bool not_finite(uint32_t bf16x2) {
    return (bf16x2 & 0x7f80u) == 0x7f80u || (bf16x2 & 0x7f800000u) == 0x7f800000u;
}

// The rows of a segment's chunks in which C holds an infinity or a NaN once more, token by token: P C
// reads such a value as 0 times it, which is NaN, also for the rows that the mask keeps from it.  By the 128
// threads of the O group, with the state in shared memory; a thread holds a column or half of one; about 2 us
// a token.  Run only where X is not finite in the end, so that the scan itself pays one look at X a
// CTA, and no time that shows (B8 H16 T4096 d = 128, B16 H16 T4096 d = 64).  Finding such values chunk
// by chunk and clearing them in the tiles before P C took 7 to 12 us of the former.
template <int D, bool REV, bool NORM, bool SEL>
__device__ __forceinline__ void redo_rows(const ScanArgs &a, const ScanArgs &own, const float *ws, float *sm,
                                          int64_t chain, int64_t n, const Seg &sg, int seg, int nseg) {
    constexpr int N = 128, PARTS = N / D, ROWS = D / PARTS;
    const int tid = threadIdx.x & (N - 1), col = tid % D, part = tid / D;
    const __nv_bfloat16 *const A = static_cast<const __nv_bfloat16 *>(own.a),
                        *const B = static_cast<const __nv_bfloat16 *>(own.b),
                        *const Cm = static_cast<const __nv_bfloat16 *>(own.c);
    if ((tid & 31) == 0) bulk_wait0();                           // this warp's rows are written
    auto first_token = [&](int i) -> int64_t { return (int64_t)(REV ? sg.total - 1 - i : i) * C; };
    auto holds = [&](int i) -> bool {                            // by this thread's share of chunk i of C
        const int64_t t0 = first_token(i);
        const int pieces = (n - t0 < C ? (int)(n - t0) : C) * (D / 8);
        const uint4 *const p = reinterpret_cast<const uint4 *>(Cm + (chain * a.T + t0) * D);
        bool found = false;
#pragma unroll 1
        for (int z = tid; z < pieces; z += N) {
            const uint4 q = p[z];
            found = found || not_finite(q.x) || not_finite(q.y) || not_finite(q.z) || not_finite(q.w);
        }
        return found;
    };
    float *const X = sm + part * ROWS * D + col;                // element (r, col) of this part at X[r * D]
#pragma unroll 1
    for (int r = 0; r < ROWS; ++r)
        X[r * D] = SEL && seg > 0 ? 0.f : entry_state<D, REV>(a, own, ws, chain, n, seg, nseg, part * ROWS + r, col);
    if (SEL)
        for (int s = 0; s < seg; ++s) {
            const Seg q = seg_of(n, s, nseg);
            if (q.first >= q.last && s > 0) continue;
            const float g = chunks_decay(a.sel, chain, q.first, q.last);
#pragma unroll 1
            for (int r = 0; r < ROWS; ++r)
                X[r * D] = fmaf(g, X[r * D], ws[(int64_t)s * D * D + (part * ROWS + r) * D + col]);
        }
    bar_arrive(5, 384);                                          // the X group may write X_out
    float *const va = sm + D * D, *const vb = va + D, *const sum = vb + D, *const red = sum + N;
    int *const shared_last = reinterpret_cast<int *>(red);
    if (tid == 0) *shared_last = -1;
    bar_sync(3, N);
    int last = -1;
#pragma unroll 1
    for (int i = sg.first; i < sg.last; ++i)
        if (holds(i)) last = i;
    if (last >= 0) atomicMax(shared_last, last);
    bar_sync(3, N);
    last = min(*shared_last, sg.last - 1);                       // (of a call given up, tiles may still land there)
    float g = SEL ? 1.f : decay_pow(a.log_decay[chain % a.H], 1.f);
    const int64_t ab = SEL ? group_chain(chain, a.H, a.sel.gate.G) : chain;
    for (int i = sg.first; i <= last; ++i) {
        const int64_t t0 = first_token(i);
        const int nv = n - t0 < C ? (int)(n - t0) : C;
        const bool write = bar_or(3, N, holds(i));
        for (int j = 0; j < nv; ++j) {
            const int64_t t = t0 + (REV ? nv - 1 - j : j), row = (chain * a.T + t) * D, abrow = (ab * a.T + t) * D;
            bar_sync(3, N);                                    // the token before is done with
            if (part == 0) {
                va[col] = to_f32(A[abrow + col]);
                vb[col] = to_f32(B[abrow + col]);
            }
            const float value = to_f32(Cm[row + col]);
            float c = a.in_scale * value;
            if (SEL) {
                const int64_t at = (chain * a.sel.n_chunks + i) * C + j;
                const float dt = a.sel.c[at].y;
                g = expf(a.sel.gate.log_decay[chain % a.H] * dt);
                c = dt * value;
            }
            bar_sync(3, N);
            float o = 0.f;
#pragma unroll 2
            for (int r = 0; r < ROWS; ++r) {
                const float b = vb[part * ROWS + r], x = REV ? fmaf(b, c, X[r * D]) : fmaf(g, X[r * D], b * c);
                o = fmaf(va[part * ROWS + r], x, o);
                X[r * D] = REV ? g * x : x;
            }
            if (!write) continue;
            sum[tid] = o;
            bar_sync(3, N);
            o = 0.f;
            for (int s = 0; s < PARTS; ++s) o += sum[s * D + col];
            o *= a.out_scale;
            if (SEL && a.sel.gate.skip) o = fmaf(a.sel.gate.skip[chain % a.H], value, o);
            if (NORM) {
                // every part holds the row, and its N / D copies add up to as many times the sums
                float m[2] = {0.f, 0.f};
#pragma unroll 1
                for (int z = 0; z < 2; ++z) {
                    float y = z == 0 ? o : (o - m[0]) * (o - m[0]);
#pragma unroll 1
                    for (int s = 16; s; s >>= 1) y += __shfl_xor_sync(~0u, y, s);
                    if ((tid & 31) == 0) red[z * 4 + (tid >> 5)] = y;
                    bar_sync(3, N);
                    m[z] = 0.f;
                    for (int w = 0; w < 4; ++w) m[z] += red[z * 4 + w];
                    m[z] *= 1.f / N;
                }
                o = (o - m[0]) * rsqrtf(m[1] + a.norm.eps);
                if (a.norm.weight) o *= a.norm.weight[col];
                if (a.norm.bias) o += a.norm.bias[col];
            }
            if (part == 0) static_cast<__nv_bfloat16 *>(own.out)[row + col] = __float2bfloat16_rn(o);
        }
    }
}

// PRE: only the state of a segment, from zero (segment 0: from X0), into the workspace.  SKIP (with SEL): rows have skip v
// added, in fp32 behind the scan, before they are rounded.
template <int D, bool REV, bool PRE, bool NORM, bool SEL, bool SKIP>
__global__ void __launch_bounds__(NTHREADS, 1)
scan_tc_kernel(const __grid_constant__ Jobs<REV ? 2 : 1> jobs, const int nseg, const int by_length, const int order) {
    using L = Lay<D, PRE, SEL>;
    static_assert(!SEL || !REV, "selective scans run forward");
    static_assert(!SKIP || (SEL && !PRE && !NORM), "skip v is a selective scan's");
    const auto &job = jobs.s[REV ? blockIdx.x & 1 : 0];
    const int block = REV ? blockIdx.x >> 1 : blockIdx.x;
    const ScanArgs &a = jobs.s[0].args, &own = job.args;   // own: a, b, c, out, X_out, x0_trans and ws
    const CUtensorMap &tma = job.a, &tmb = job.b, &tmc = job.c, &tmo = job.out;
    let_next_grid_start();
    if (order & kWaitFirst) wait_previous_grid();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int grid_seg = PRE ? nseg - 1 : nseg;
    int64_t chain = block / grid_seg;
    const int seg = block % grid_seg;
    if (!PRE && by_length) {                        // the longest batch rows' chains start first
        int *row = reinterpret_cast<int *>(sm + L::MISC + 8);
        const int B = (int)(a.n_chains / a.H);
        if (tid < B) {
            const int mine = a.lens[tid];
            int rank = 0;
            for (int b = 0; b < B; ++b) rank += a.lens[b] > mine || (a.lens[b] == mine && b < tid);
            if (rank == (int)(chain / a.H)) *row = tid;
        }
        __syncthreads();
        chain = (int64_t)*row * a.H + chain % a.H;
    }
    const int64_t n = chain_len(a.lens, chain, a.H, a.T);
    const Seg sg = seg_of(n, seg, nseg);
    const int nch = sg.last - sg.first;
    const bool final_seg = !PRE && seg == nseg - 1;
    if (nch == 0 && !(final_seg && (own.X_out || a.zero_rest)) && !(PRE && seg == 0)) {
        if (order & kWaitLast) wait_previous_grid();
        return;
    }
    const uint64_t limit = (uint64_t)a.wait_ns;
    const float lg = SEL ? 0.f : a.log_decay[chain % a.H];
    const int64_t ab_chain = SEL ? group_chain(chain, a.H, a.sel.gate.G) : chain;   // whose rows A and B are
    // Within a chunk of a mild head every quotient of powers of g is at most e^24 = 2.6e10, which
    // leaves the scores and their sums 28 of fp32's and bf16's 38 decimal orders: the rows' decay
    // of a chunk, g^(i+1) (A X + (mask . g^-(j+1) . G) C), is then one factor in the epilogue.
    // Otherwise A X is scaled by its rows' decay on its own and the scores by g^(i-j), and nothing
    // is divided by a power of g.
    const bool mild = fabsf(lg) * C <= 24.f;   // (SEL: by the chunk)
    // SEL: the tables of this segment's chunks, one after the other
    const int64_t tables = SEL ? chain * a.sel.n_chunks + sg.first : 0;
    const int x_slots = nseg;                       // workspace: nseg - 1 segment states, X0's copy
    float *const ws = own.ws + chain * x_slots * D * D;

    volatile int *s_abort = reinterpret_cast<volatile int *>(sm + L::MISC);
    volatile uint32_t *s_tmem = reinterpret_cast<volatile uint32_t *>(sm + L::MISC + 4);
    float *const pw = reinterpret_cast<float *>(sm + L::T_PW);   // g^n, n = 0..128
    float *const kw = reinterpret_cast<float *>(sm + L::T_KW);   // w_j of a full chunk
    float *const kt = reinterpret_cast<float *>(sm + L::T_KT);   // w_j of the tail chunk
    volatile int *const look = reinterpret_cast<volatile int *>(sm + L::MISC + 12);   // X is not finite
    auto bar = [&](int i) -> uint32_t { return sb + L::BAR + 8u * (uint32_t)i; };
    auto full = [&](int st, int x) -> uint32_t { return bar(L::FULL + st * L::NT + x); };
    auto empty = [&](int st, int x) -> uint32_t { return bar(L::EMPTY + st * L::NT + x); };
    auto tile = [&](int st, int x) -> uint32_t { return sb + (uint32_t)(st * L::NT + x) * L::TILE; };
    constexpr int XB_ = 0, XC = 1, XA = 2;          // tiles of a stage: B, C and (not PRE) A
    struct Ring {                                   // stage of a chunk and the phase of its barriers
        int st = 0;
        uint32_t ph = 0;
        __device__ __forceinline__ void next() {
            if (++st == L::NST) {
                st = 0;
                ph ^= 1u;
            }
        }
    };
    auto fail_now = [&]() {
        *s_abort = 1;
        atomicExch(a.err, kDevErrTimeout);
    };
    auto chunk_id = [&](int i) -> int { return REV ? sg.total - 1 - (sg.first + i) : sg.first + i; };
    // The chunk of this segment that a sequence's end cuts short (-1: none), and its tokens.
    const int tail_tokens = (int)(n - (int64_t)(sg.total - 1) * C);
    const int tail_i = tail_tokens == C ? -1 : (REV ? 0 : sg.total - 1) - sg.first;
    auto tokens = [&](int i) -> int { return i == tail_i ? tail_tokens : C; };
    const bool lo3 = own.X_out != nullptr;          // the update takes its third term

    if (tid == 0) {
        for (int i = 0; i < L::NBAR; ++i) {
            uint32_t c = 1;
            const int e = i - L::EMPTY;
            if (e >= 0 && e < L::NST * L::NT)       // B: its readers' warps (and G); C: the
                c = e % L::NT == XB_ ? 4 * L::KG + (PRE ? 0 : 1)   // update (and P C; SKIP: the O group's warps); A: those
                  : e % L::NT == XC ? (PRE ? 1 : SKIP ? 6 : 2) : 4;
            if (i == L::PRDY || i == L::OSC || i == L::OFREE || (i >= L::KRDY && i < L::KFREE)) c = 4;
            if (i == L::VZ) c = 4 * L::KG;
            if (i >= L::XBRDY && i < L::KRDY) c = 8;   // XBRDY, UFREE
            mbar_init(bar(i), c);
        }
        fence_mbar_init();
        *s_abort = 0;
        *look = 0;
    }
    // Warp 0 needs none of what follows: it only announces the barriers, and its first tiles are on
    // their way while the others make the tables and tensor memory ready.
    if (warp == 0) {
        __syncwarp();
        asm volatile("barrier.cta.arrive 1, %0;" ::"n"(NTHREADS) : "memory");
    } else {
        const int j = tid - 32;
        if (SEL) {
            // this segment's tables, unless the launch before has formed them; by all warps that wait for the
            // first tiles
            if (PRE || seg == nseg - 1)
                for (int i = warp - 1; i < nch; i += NTHREADS / 32 - 1) form_tables(a, chain, n, sg.first + i);
        } else if (j <= C) pw[j] = decay_pow(lg, (float)j);
        else if (j <= 2 * C) {
            const int x = j - C - 1;
            kw[x] = a.in_scale * decay_pow(lg, (float)(REV ? x + 1 : C - 1 - x));
        }
        if (warp == 3) tmem_alloc(sb + L::MISC + 4, TMEM_COLS);
        tc_fence_before();
        asm volatile("barrier.cta.sync 1, %0;" ::"n"(NTHREADS) : "memory");
        tc_fence_after();
    }
    const uint32_t tmem = __shfl_sync(~0u, *s_tmem, 0);

    // Every MMA of this warp has finished before it leaves.
    auto drain = [&](bool ok, int which) {
        if (lane == 0) {
            if (!ok) fail_now();
            if (nch > 0) {
                mma_commit(bar(L::DRAIN + which));
                mbar_wait(bar(L::DRAIN + which), 0, kDrainNs);
            }
        }
        __syncwarp();
    };
    if (warp < 4) {
      reg_dec<REGS_W0>();
      if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        if (lane == 0) {
            bool ok = true;
            if (a.force_timeout) ok = wait_bar(bar(L::NEVER), 0, limit, s_abort);
            int issued = 0;                          // tiles, in issue order
            for (int i = 0; i < nch && ok; ++i) {
                const int st = i % L::NST;
                const int y = chunk_id(i) * C;
#pragma unroll 1
                for (int x0 = 0; x0 < L::NT && ok; ++x0) {
                    const int x = PRE ? x0 : x0 == 0 ? XB_ : x0 == 1 ? XA : XC;
                    if (i >= L::NST) ok = wait_bar(empty(st, x), (uint32_t)(i / L::NST - 1) & 1u, limit, s_abort);
                    if (!ok) break;
                    const CUtensorMap *tm = x == XB_ ? &tmb : x == XC ? &tmc : &tma;
                    mbar_expect_tx(full(st, x), L::TILE);
                    const int z = (int)(x == XC ? chain : ab_chain);
                    tma_load_3d(tile(st, x), tm, 0, y, z, full(st, x));
                    if (D == 128) tma_load_3d(tile(st, x) + HALF, tm, 64, y, z, full(st, x));
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
        // (the issuers' loops run warp-uniform, so that addresses stay in uniform registers, and
        // unrolled: an MMA issued from a rolled loop of one lane took about 200 cycles)
        bool ok = true;
        Ring r;
        const uint64_t da0 = sdesc_sw128(tile(0, XA), 16, 1024), db0 = sdesc_sw128(tile(0, XB_), 16, 1024);
        const uint64_t dc0 = sdesc_sw128(tile(0, XC), HALF, 1024);
        uint32_t steep = 0;                          // SEL: steep chunks so far, each a phase of OSC
        const float4 *info = a.sel.ends + tables;    // SEL: whether a chunk is mild, fetched a chunk ahead
        float flag = SEL && !PRE && nch > 0 ? info->w : 0.f;
        for (int i = 0; !PRE && i < nch; ++i, r.next()) {
            const bool one = SEL ? flag != 0.f : mild;
            const uint32_t pi = (uint32_t)i & 1u, off_st = r.st * ((L::NT * L::TILE) >> 4);
            const int st = r.st;
            ok = __all_sync(~0u, wait_bar(full(st, XB_), r.ph, limit, s_abort) &&
                                     wait_bar(full(st, XA), r.ph, limit, s_abort) &&
                                     (i != tail_i || wait_bar(bar(L::VZ), 0, limit, s_abort)) &&
                                     (i == 0 || wait_bar(bar(L::PVDONE), pi ^ 1u, limit, s_abort)));
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
                constexpr uint32_t id = idesc_bf16(128, 128, false, false);
                const uint64_t da = da0 + off_st, db = db0 + off_st;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t off = ((kk >> 2) * HALF + (kk & 3) * 32u) >> 4;
                    mma_bf16(tmem + COL_G, da + off, db + off, id, kk > 0);
                }
                mma_commit(bar(L::GDONE));
                mma_commit(empty(st, XB_));
            }
            __syncwarp();
            if (SEL && i + 1 < nch) flag = (++info)->w;
            ok = __all_sync(~0u, wait_bar(bar(L::PRDY), pi, limit, s_abort) &&
                                     wait_bar(full(st, XC), r.ph, limit, s_abort) &&
                                     wait_bar(bar(one ? L::QSDONE : L::OSC), SEL && !one ? steep & 1u : pi, limit, s_abort));
            steep += !one;
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
                constexpr uint32_t id = idesc_bf16(128, D, false, true);
                const uint64_t dc = dc0 + off_st;
#pragma unroll
                for (int kk = 0; kk < C / 16; ++kk)
                    mma_bf16_ta(tmem + COL_O, tmem + COL_G + 8 * kk, dc + kk * 128, id, 1);
                mma_commit(bar(L::PVDONE));
                mma_commit(empty(st, XC));
            }
            __syncwarp();
        }
        if (!PRE) drain(ok, 0);
      } else if (warp == 2) {
        // ---------------------------------------------------------------- state update
        bool ok = true;
        Ring r;
        const uint64_t dc0 = sdesc_sw128(tile(0, XC), HALF, 1024);
        for (int i = 0; i < nch && ok; ++i, r.next()) {
            const int st = r.st, ub = i % L::UB;
            ok = __all_sync(~0u, wait_bar(full(st, XC), r.ph, limit, s_abort) &&
                                     (i < L::UB || wait_bar(bar(L::UFREE + ub), (uint32_t)(i / L::UB - 1) & 1u, limit, s_abort)));
            const uint64_t dc = dc0 + r.st * ((L::NT * L::TILE) >> 4);
            const uint32_t du = tmem + COL_U + 128 * ub;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int b = u % L::KG;
                ok = ok && __all_sync(~0u, wait_bar(bar(L::KRDY + b), (uint32_t)((4 * i + u) / L::KG) & 1u, limit, s_abort));
                if (!ok) break;
                tc_fence_after();
                if (lane == 0) {
                    constexpr uint32_t id = idesc_bf16(128, D, false, true);
                    const uint32_t ka = tmem + L::COL_K + KBUF * b;
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {         // the small terms first
                        const uint64_t dk = dc + (2 * u + kk) * 128;
                        if (lo3) mma_bf16_ta(du, ka + 32 + 8 * kk, dk, id, u > 0 || kk > 0);
                        mma_bf16_ta(du, ka + 16 + 8 * kk, dk, id, u > 0 || kk > 0 || lo3);
                        mma_bf16_ta(du, ka + 8 * kk, dk, id, 1);
                    }
                    mma_commit(bar(L::KFREE + b));
                    if (u == 3) {
                        mma_commit(bar(L::UDONE + ub));
                        mma_commit(empty(st, XC));
                    }
                }
                __syncwarp();
            }
        }
        drain(ok, 1);
      } else {
        // ---------------------------------------------------------------- A X
        bool ok = true;
        Ring r;
        const uint64_t da0 = sdesc_sw128(tile(0, XA), 16, 1024), dx = sdesc_sw128(sb + L::XB, HALF, 1024);
        for (int i = 0; !PRE && i < nch; ++i, r.next()) {
            const uint32_t pi = (uint32_t)i & 1u;
            ok = __all_sync(~0u, wait_bar(full(r.st, XA), r.ph, limit, s_abort) &&
                                     wait_bar(bar(L::XBRDY), pi, limit, s_abort) &&
                                     (i == 0 || wait_bar(bar(L::OFREE), pi ^ 1u, limit, s_abort)));
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
                constexpr uint32_t id = idesc_bf16(128, D, false, true);
                const uint64_t da = da0 + r.st * ((L::NT * L::TILE) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_bf16(tmem + COL_O, da + (((kk >> 2) * HALF + (kk & 3) * 32u) >> 4),
                             dx + kk * 128, id, kk > 0);
                mma_commit(bar(L::QSDONE));
            }
            __syncwarp();
        }
        if (!PRE) drain(ok, 2);
      }
    } else if (!PRE && warp >= 4 && warp < 8) {
        // ---------------------------------------------------------------- P
        {
            const int w = warp & 3, row = w * 32 + lane;
            const uint32_t lb = (uint32_t)(w * 32) << 16;
            const float sg = REV ? lg : -lg;         // powers from one column to the next
            const float h1 = decay_pow(sg, 1.f), h2 = decay_pow(sg, 2.f), h3 = decay_pow(sg, 3.f),
                        h4 = decay_pow(sg, 4.f), h16 = decay_pow(sg, 16.f);
            float *const sF = reinterpret_cast<float *>(sm + L::T_SF), *const sC = reinterpret_cast<float *>(sm + L::T_SC),
                  *const sD = reinterpret_cast<float *>(sm + L::T_SD);
            // SEL: of the chunk at hand, fetched a chunk ahead: logs of blocks and whether it is mild, the row's
            // log and step
            const float4 *info = a.sel.ends + tables;
            const float2 *at = a.sel.c + tables * C + row;
            float4 ends = {};
            float2 own_row = {};
            if (SEL && nch > 0) {
                ends = *info;
                own_row = *at;
            }
            bool ok = true;
            for (int i = 0; i < nch; ++i) {
                bool one = mild, even = true;
                float in_block = 0.f;                // SEL: log to this row, from its block's start
                if (SEL) {
                    one = ends.w != 0.f;
                    const float dt = own_row.y;
                    bar_sync(6, 128);                // the chunk before is done with (no wait between: it ends)
                    if (one) {
                        sF[row] = dt * __expf(-own_row.x);
                    } else {
                        // to the ends of the blocks of 32 before later rows' own, and of the diagonal block, which is this
                        // warp's own, from its start while its decays are e^-kMild or more, else as they are
                        in_block = own_row.x;
                        even = __all_sync(~0u, fabsf(in_block) <= kMild);
                        float z = (w == 0 ? ends.x : w == 1 ? ends.y : ends.z) - in_block;   // to the block's end
                        if (w < 1) {
                            sF[row] = dt * __expf(z);
                            z += ends.y;
                        }
                        if (w < 2) {
                            sF[32 + row] = dt * __expf(z);
                            z += ends.z;
                        }
                        if (w < 3) sF[96 + row] = dt * __expf(z);
                        sD[row] = even ? dt * __expf(-in_block) : dt;
                        sC[row] = in_block;
                    }
                    if (i + 1 < nch) {
                        ends = *++info;
                        own_row = *(at += C);
                    }
                }
                ok = __all_sync(~0u, wait_bar(bar(L::GDONE), (uint32_t)i & 1u, limit, s_abort));
                if (SEL) ok = !bar_or(7, 128, !ok);  // the tables are written (and all four warps leave together)
                if (!ok) break;
                tc_fence_after();
                // bf16, and on the diagonal blocks of 16 and 32 the mask, over columns already read
                auto put = [&](float (&v)[16], int c) {
                    uint32_t pk[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) pk[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
                    if (c >> 5 == w) {
                        const int d = row - c;       // columns up to (reverse: from) d of this piece
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            if (REV) pk[e] = d <= 2 * e ? pk[e] : d == 2 * e + 1 ? pk[e] & 0xffff0000u : 0u;
                            else pk[e] = d > 2 * e ? pk[e] : d == 2 * e ? pk[e] & 0xffffu : 0u;
                        }
                    }
                    tmem_st8(tmem + lb + COL_G + (c >> 1), pk);
                };
                // the blocks of 32 columns that this warp's 32 rows see, 16 columns a turn
                const int nv = tokens(i);
                const int c0 = REV ? 32 * w : 0, c1 = REV ? C : 32 * w + 32;
                if constexpr (SEL) {
                    // (the rows' own decays are the epilogue's, but for those of a block that is not even)
                    const float *const left = one ? sF : sF + 16 * w * (w - 1);
                    float f = 1.f;                   // the rows' decays to their block, if the epilogue has none
                    if (!even) {
                        f = __expf(in_block);
                        // the diagonal block's decays, in place (a rolled loop: this is rare, and code of the usual
                        // way made longer by it is slower: B16 H16 T4096 d = 64 took 212 us for 191)
#pragma unroll 1
                        for (int c = 32 * w; c < 32 * w + 32; c += 4) {
                            float v[4];
                            tmem_ld4(tmem + lb + COL_G + c, v);
                            const float4 z = *reinterpret_cast<const float4 *>(sC + c);
                            v[0] *= __expf(in_block - z.x);
                            v[1] *= __expf(in_block - z.y);
                            v[2] *= __expf(in_block - z.z);
                            v[3] *= __expf(in_block - z.w);
                            tmem_st4(tmem + lb + COL_G + c, v);
                        }
                        tmem_st_wait();
                    }
                    float v[16];
#pragma unroll 1
                    for (int c = c0; c < c1; c += 16) {
                        tmem_fetch16(tmem + lb + COL_G + c, v);
                        const bool before = c < 32 * w;
                        const float4 *const F = reinterpret_cast<const float4 *>((one || before ? left : sD) + c);
                        const float r = before ? f : 1.f;
                        uint64_t t[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 q = F[e];
                            t[2 * e] = mul2(pair(q.x, q.y), pair(r, r));
                            t[2 * e + 1] = mul2(pair(q.z, q.w), pair(r, r));
                        }
                        tmem_landed(v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) scale2(v[2 * e], v[2 * e + 1], t[e]);
                        put(v, c);
                    }
                } else if (mild) {
                    // column j times g^-(j+1), reverse g^-(n-1-j)
                    float f = a.in_scale * decay_pow(lg, (float)(REV ? c0 + 1 - nv : -1));
                    tmem_stream(tmem + lb + COL_G, c0, c1, [&](float (&v)[16], int c) {
                        uint64_t ta = pair(f, f * h1), tb = pair(f * h2, f * h3);
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            scale2(v[e], v[e + 1], ta);
                            scale2(v[e + 2], v[e + 3], tb);
                            ta = mul2(ta, pair(h4, h4));
                            tb = mul2(tb, pair(h4, h4));
                        }
                        f *= h16;
                        put(v, c);
                    });
                } else {
                    tmem_stream(tmem + lb + COL_G, c0, c1, [&](float (&v)[16], int c) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int lag = REV ? c + e - row : row - c - e;
                            // (behind a sequence's end the power may have overflowed)
                            v[e] *= REV && c + e >= nv ? 0.f : a.in_scale * pw[lag < 0 ? 0 : lag];
                        }
                        put(v, c);
                    });
                }
                const uint32_t none[8] = {};
#pragma unroll 1
                for (int c = REV ? 0 : 32 * w + 32; c < (REV ? 32 * w : C); c += 16)
                    tmem_st8(tmem + lb + COL_G + (c >> 1), none);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::PRDY));
            }
            if (!ok && lane == 0) fail_now();
        }
    } else if (!PRE && warp >= 8 && warp < 12) {
        // ---------------------------------------------------------------- O
        {
            const int w = warp & 3, row = w * 32 + lane;
            const uint32_t lb = (uint32_t)(w * 32) << 16;
            bool ok = true;
            const float4 *info = a.sel.ends + tables; // SEL: as the P group's
            const float2 *at = a.sel.c + tables * C + row;
            float4 ends = {};
            float row_c = 0.f;
            const float skip = SKIP ? a.sel.gate.skip[chain % a.H] : 0.f;
            if (SEL && nch > 0) {
                ends = *info;
                row_c = at->x;
            }
            for (int i = 0; i < nch; ++i) {
                const uint32_t pi = (uint32_t)i & 1u;
                const int nv = tokens(i);
                bool one = mild;
                float rd, last = 1.f;                // the rows' decay of A X, and what of it is P C's too
                if (SEL) {
                    one = ends.w != 0.f;
                    rd = row_c;
                    if (!one) {                      // from the block's start on, where that is the P group's too
                        float before = 0.f;
                        if (w > 0) before += ends.x;
                        if (w > 1) before += ends.y;
                        if (w > 2) before += ends.z;
                        rd = before + row_c;
                        if (__all_sync(~0u, fabsf(row_c) <= kMild)) {
                            rd = before;
                            last = __expf(row_c);
                        }
                    }
                    rd = __expf(rd);
                    if (i + 1 < nch) {
                        ends = *++info;
                        row_c = (at += C)->x;
                    }
                } else {
                    rd = pw[REV ? (row < nv ? nv - 1 - row : 0) : row + 1];
                }
                if (!one) {
                    ok = __all_sync(~0u, wait_bar(bar(L::QSDONE), pi, limit, s_abort));
                    if (!ok) break;
                    tc_fence_after();
                    tmem_stream(tmem + lb + COL_O, 0, D, [&](float (&v)[16], int c) {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) scale2(v[e], v[e + 1], pair(rd, rd));
                        tmem_st16(tmem + lb + COL_O + c, v);
                    });
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(L::OSC));
                    rd = last;
                }
                rd *= a.out_scale;

                ok = __all_sync(~0u, wait_bar(bar(L::PVDONE), pi, limit, s_abort) &&
                                         (!SKIP || wait_bar(full(i % L::NST, XC), (uint32_t)(i / L::NST) & 1u, limit, s_abort)));
                if (!ok) break;
                tc_fence_after();
                float mean = 0.f, rstd = 1.f;
                if (NORM) {                          // a thread holds its whole row
                    // mean and centred sum of squares of 16 values at a time, merged
                    float cnt = 0.f, m2 = 0.f;
                    tmem_stream(tmem + lb + COL_O, 0, D, [&](float (&v)[16], int) {
                        uint64_t x[8], y = 0;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            x[e] = mul2(pair(v[2 * e], v[2 * e + 1]), pair(rd, rd));
                            y = add2(y, x[e]);
                        }
                        float2 f = halves(y);
                        const float t = (f.x + f.y) * (1.f / 16.f);
                        y = 0;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint64_t c = add2(x[e], pair(-t, -t));
                            y = fma2(c, c, y);
                        }
                        f = halves(y);
                        const float r = __fdividef(16.f, cnt + 16.f), dm = t - mean;
                        mean = fmaf(dm, r, mean);
                        m2 += fmaf(dm * dm, cnt * r, f.x + f.y);
                        cnt += 16.f;
                    });
                    rstd = rsqrtf(m2 / D + a.norm.eps);
                }
                const float n1 = rd * rstd, n0 = -mean * rstd;
                // G and A X have read this chunk's A tile: the rows are staged over it and leave
                // by a tensor store a warp (whole rows), or one by one at a sequence's end
                const bool whole = w * 32 + 32 <= nv;
                const int st = i % L::NST;
                const int64_t row0 = (int64_t)chunk_id(i) * C;
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(own.out) +
                                     (chain * a.T + row0 + row) * D;
                const uint32_t to = tile(st, XA) + (uint32_t)(row >> 3) * 1024u + (uint32_t)(row & 7) * 128u;
                // eight columns c + 8 e of the row's place in a tile (SKIP: v is there in C's)
                auto piece = [&](int c, int e) -> uint32_t {
                    return (uint32_t)(c >> 6) * HALF + (((((uint32_t)c & 63u) >> 3) + e ^ ((uint32_t)row & 7u)) << 4);
                };
                tmem_stream(tmem + lb + COL_O, 0, D, [&](float (&v)[16], int c) {
                    if (NORM) {
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const float4 wt = a.norm.weight ? __ldg(reinterpret_cast<const float4 *>(a.norm.weight + c + e))
                                                            : make_float4(1.f, 1.f, 1.f, 1.f);
                            const float4 bs = a.norm.bias ? __ldg(reinterpret_cast<const float4 *>(a.norm.bias + c + e))
                                                          : make_float4(0.f, 0.f, 0.f, 0.f);
                            const float2 lo = halves(fma2(fma2(pair(v[e], v[e + 1]), pair(n1, n1), pair(n0, n0)),
                                                          pair(wt.x, wt.y), pair(bs.x, bs.y)));
                            const float2 hi = halves(fma2(fma2(pair(v[e + 2], v[e + 3]), pair(n1, n1), pair(n0, n0)),
                                                          pair(wt.z, wt.w), pair(bs.z, bs.w)));
                            v[e] = lo.x;
                            v[e + 1] = lo.y;
                            v[e + 2] = hi.x;
                            v[e + 3] = hi.y;
                        }
                    } else if (SKIP) {
#pragma unroll
                        for (int e = 0; e < 16; e += 8) {
                            const uint4 q = ld_shared_v4(to + (tile(st, XC) - tile(st, XA)) + piece(c, e / 8));
                            const uint32_t x[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                const uint64_t own_v = mul2(pair(__uint_as_float(x[z] << 16), __uint_as_float(x[z] & 0xffff0000u)),
                                                            pair(skip, skip));
                                const float2 f = halves(fma2(pair(v[e + 2 * z], v[e + 2 * z + 1]), pair(rd, rd), own_v));
                                v[e + 2 * z] = f.x;
                                v[e + 2 * z + 1] = f.y;
                            }
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) scale2(v[e], v[e + 1], pair(rd, rd));
                    }
                    uint32_t pk[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) pk[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            st_shared_v4(to + piece(c, e), pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
                    } else if (row < nv) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<uint4 *>(out + c + 8 * e) =
                                make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
                    }
                });
                tc_fence_before();
                if (whole) fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(L::OFREE));
                    if (SKIP) mbar_arrive(empty(st, XC));
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
            if (!ok && lane == 0) fail_now();
            if (a.zero_rest && final_seg && ok) {    // rows behind the sequence's end
                uint4 *rest = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(own.out) + (chain * a.T + n) * D);
                const int64_t pieces = (a.T - n) * (D / 8);
                for (int64_t z = tid - 8 * 32; z < pieces; z += 128) rest[z] = make_uint4(0u, 0u, 0u, 0u);
            }
            bar_sync(4, 384);                        // with the X group
            if (*look) redo_rows<D, REV, NORM, SEL>(a, own, ws, reinterpret_cast<float *>(sm), chain, n, sg, seg, nseg);
        }
    } else if (warp < 16 || warp >= 24) {
        // ---------------------------------------------------------------- (diag(w) B)^T
        reg_dec<REGS_K>();
        // the group: warps 12-15 and 24-27, and in a PRE launch 4-11 too
        const int w = warp & 3, b = warp >= 24 ? 1 : warp >= 12 ? 0 : warp >= 8 ? 3 : 2;
        const uint32_t lb = (uint32_t)(w * 32) << 16;
        const bool mine = w * 32 < D;
        bool ok = true;
        Ring r;
        // SEL: the weights of the 32 tokens at hand (thread t has 8 c + 2 (t % 4), +1 for c = 0..3), those of the next
        // on their way behind the last use of these.  A buffer's turns, 32 KG tokens apart, go on from chunk to chunk.
        uint64_t wv[4];
        const float *from = SEL ? a.sel.w + tables * C + 32 * b + 8 * (lane & 3) : nullptr;
        int turns = nch * (4 / L::KG);
        auto fetch_weights = [&]() {
            if (turns-- <= 0) return;
#pragma unroll
            for (int c = 0; c < 4; c += 2) {
                const float4 q = *reinterpret_cast<const float4 *>(from + 2 * c);
                wv[c] = pair(q.x, q.y);
                wv[c + 1] = pair(q.z, q.w);
            }
            from += 32 * L::KG;
        };
        if (SEL) fetch_weights();
        for (int i = 0; i < nch; ++i, r.next()) {
            const int st = r.st;
            const uint32_t ph = r.ph;
            const bool tail = i == tail_i;
            const int nv = tokens(i);
            ok = __all_sync(~0u, wait_bar(full(st, XB_), ph, limit, s_abort));
            if (!ok) break;
            const float *wt = kw;
            if (tail) {
                // rows behind the end may hold anything: those of B and C become zero before any
                // product reads them (and the weights too; every warp writes the same values)
                for (int j = lane; !SEL && j < C; j += 32)
                    kt[j] = j < nv ? a.in_scale * pw[REV ? j + 1 : nv - 1 - j] : 0.f;
                ok = __all_sync(~0u, wait_bar(full(st, XC), ph, limit, s_abort));
                if (!ok) break;
                for (int j = nv + 4 * b + w; j < C; j += 4 * L::KG)
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
                if (!SEL) wt = kt;
            }
            // ldmatrix x4: matrices (tokens +0, +8) x (rows +0, +8) of X, 16 rows a half-warp
            const uint32_t r8 = (uint32_t)lane & 7u, m = (uint32_t)lane >> 3;
            for (int u = b; u < 4; u += L::KG) {
                const int use = (4 * i + u) / L::KG;   // of this buffer
                // thread t: tokens 32 u + 8 c + 2 (t % 4), +1 for c = 0..3
                if (!SEL)
#pragma unroll
                    for (int c = 0; c < 4; ++c) wv[c] = *reinterpret_cast<const uint64_t *>(wt + 32 * u + 8 * c + 2 * (lane & 3));
                uint32_t hi[8], mid[8], lo[8];
                auto form = [&](int h) {             // rows w * 32 + 16 h .. +15 of X
#pragma unroll
                    for (int t2 = 0; t2 < 2; ++t2) { // tokens 32 u + 16 t2 .. +15
                        const uint32_t row = 32u * u + 16u * t2 + 8u * (m >> 1) + r8;
                        const uint32_t dd = (uint32_t)w * 32u + 16u * h + 8u * (m & 1u);
                        uint32_t k2[4];              // (tokens 0-7, rows 0-7), (0-7, 8-15), (8-15, 0-7), ..
                        ldmatrix_x4_trans(tile(st, XB_) + (dd >> 6) * HALF + sw128(row, (dd & 63u) >> 3), k2);
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const int c = 2 * t2 + (z >> 1), o = 2 * c + (z & 1);
                            uint64_t x = mul2(pair(__uint_as_float(k2[z] << 16),
                                                   __uint_as_float(k2[z] & 0xffff0000u)), wv[c]);
                            hi[o] = top_halves(x);
                            x = below(x);
                            mid[o] = top_halves(x);
                            if (lo3) lo[o] = top_halves(below(x));
                        }
                    }
                };
                auto store = [&](int h) {
                    const uint32_t at = tmem + lb + ((uint32_t)(16 * h) << 16) + L::COL_K + KBUF * b;
                    tmem_st_16x128b_x4(at, hi);
                    tmem_st_16x128b_x4(at + 16, mid);
                    if (lo3) tmem_st_16x128b_x4(at + 32, lo);
                };
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    if (mine) form(h);               // the first before the buffer is free
                    if (h == 0) {
                        if (use > 0) ok = __all_sync(~0u, wait_bar(bar(L::KFREE + b), (uint32_t)(use - 1) & 1u, limit, s_abort));
                        if (!ok) break;
                        tc_fence_after();
                    }
                    if (mine) store(h);
                }
                if (!ok) break;
                if (SEL) fetch_weights();
                if (mine) tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(L::KRDY + b));
                    if (u + L::KG >= 4) mbar_arrive(empty(st, XB_));
                }
            }
            if (!ok) break;
        }
        if (!ok && lane == 0) fail_now();
    } else {
        // ---------------------------------------------------------------- X
        reg_inc<REGS_X>();
        constexpr int XC_ = D / 2;                   // columns of a thread
        const int w = warp & 3, d = w * 32 + lane, c0 = ((warp >> 2) & 1) * XC_;
        const uint32_t lb = (uint32_t)(w * 32) << 16;
        const bool mine = w * 32 < D;
        bool ok = true;
        float x[XC_];
#pragma unroll
        for (int e = 0; e < XC_; ++e) x[e] = 0.f;
        if (mine) {                                  // the state on entry
            // with S_T = S0 the last segment may finish before another starts: they read a copy
            const bool copy = nseg > 1 && a.X0 && own.X_out == a.X0;
            float *const x0_copy = ws + (int64_t)(nseg - 1) * D * D;
            if (seg == 0 && a.X0) {
                const float *src = !PRE && copy ? x0_copy : a.X0 + chain * D * D;
                if (own.x0_trans) {
#pragma unroll
                    for (int e = 0; e < XC_; ++e) x[e] = src[(c0 + e) * D + d];
                } else {
#pragma unroll
                    for (int e = 0; e < XC_; e += 4) {
                        const float4 m = *reinterpret_cast<const float4 *>(src + d * D + c0 + e);
                        x[e] = m.x; x[e + 1] = m.y; x[e + 2] = m.z; x[e + 3] = m.w;
                    }
                }
                if (PRE && copy)
#pragma unroll
                    for (int e = 0; e < XC_; ++e) x0_copy[d * D + c0 + e] = x[e];
            }
            if (!PRE && seg > 0) {                   // X <- g^n X + the state of each segment before
#pragma unroll
                for (int e0 = 0; e0 < XC_; e0 += 16) {
#pragma unroll 2
                    for (int r = 0; r < seg; ++r) {
                        const Seg q = seg_of(n, r, nseg);
                        if (q.first >= q.last && r > 0) continue;
                        const float g = SEL ? chunks_decay(a.sel, chain, q.first, q.last)
                                            : decay_pow(lg, (float)seg_tokens<REV>(n, q));
                        const float4 *M = reinterpret_cast<const float4 *>(ws + (int64_t)r * D * D + d * D + c0 + e0);
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const float4 m = M[e / 4];
                            x[e0 + e] = fmaf(g, x[e0 + e], m.x);
                            x[e0 + e + 1] = fmaf(g, x[e0 + e + 1], m.y);
                            x[e0 + e + 2] = fmaf(g, x[e0 + e + 2], m.z);
                            x[e0 + e + 3] = fmaf(g, x[e0 + e + 3], m.w);
                        }
                    }
                }
            }
        }
        auto put_copy = [&](int e0) {                // 16 columns in bf16, rows of X: B operand of A X
#pragma unroll
            for (int e = e0; e < e0 + 16; e += 8)
                st_shared_v4(sb + L::XB + (uint32_t)((c0 + e) >> 6) * ((uint32_t)D * 128u) +
                                 sw128(d, ((uint32_t)(c0 + e) & 63u) >> 3),
                             pack_bf16(x[e], x[e + 1]), pack_bf16(x[e + 2], x[e + 3]),
                             pack_bf16(x[e + 4], x[e + 5]), pack_bf16(x[e + 6], x[e + 7]));
        };
        if (!PRE && nch > 0) {
            if (mine) {
#pragma unroll
                for (int e = 0; e < XC_; e += 16) put_copy(e);
                fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::XBRDY));
        }
        const float2 *info = a.sel.chunk + tables;
        float next_g = SEL && nch > 0 ? info->x : 0.f;   // (fetched a chunk ahead)
        for (int i = 0; i < nch; ++i) {
            const float g = SEL ? next_g : pw[tokens(i)];
            if (SEL && i + 1 < nch) next_g = (++info)->x;
            const bool more = !PRE && i + 1 < nch;
            const int ub = i % L::UB;
            ok = __all_sync(~0u, wait_bar(bar(L::UDONE + ub), (uint32_t)(i / L::UB) & 1u, limit, s_abort) &&
                                     (!more || wait_bar(bar(L::QSDONE), (uint32_t)i & 1u, limit, s_abort)));
            if (!ok) break;
            tc_fence_after();
            if (mine) {
#pragma unroll
                for (int e = 0; e < XC_; e += 16) {
                    float u[16];
                    tmem_ld16(tmem + lb + COL_U + 128 * ub + c0 + e, u);
#pragma unroll
                    for (int z = 0; z < 16; z += 2) {
                        const float2 r = halves(fma2(pair(g, g), pair(x[e + z], x[e + z + 1]), pair(u[z], u[z + 1])));
                        x[e + z] = r.x;
                        x[e + z + 1] = r.y;
                    }
                    if (more) put_copy(e);
                }
                tc_fence_before();
                if (more) fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(L::UFREE + ub));
                if (more) mbar_arrive(bar(L::XBRDY));
            }
        }
        if (!PRE) {
            // A value of C that is not finite has left its column of X without a finite number, in every
            // row, and nothing makes one finite again: 0 times it is NaN.
            uint64_t nan2 = 0;
#pragma unroll
            for (int e = 0; e < XC_; e += 2) nan2 = fma2(pair(x[e], x[e + 1]), 0, nan2);
            const bool bad = bar_or(2, 256, (nan2 & 0x7fffffff7fffffffull) != 0);
            if (bad) *look = 1;
            bar_arrive(4, 384);
            if (bad) bar_sync(5, 384);               // (X_out may be X0, which redone rows begin with)
        }
        float *dst = PRE ? ws + (int64_t)seg * D * D
                         : final_seg && own.X_out ? own.X_out + chain * D * D : nullptr;
        if (ok && mine && dst)
#pragma unroll
            for (int e = 0; e < XC_; e += 4)
                *reinterpret_cast<float4 *>(dst + d * D + c0 + e) =
                    make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        if (!ok && lane == 0) fail_now();
    }

    __syncthreads();
    tc_fence_after();
    if (warp == 3) tmem_dealloc(tmem, TMEM_COLS);
    if (order & kWaitLast) wait_previous_grid();
}

// Times (us) of chains that take one CTA an SM: in one piece a start and so much a chunk; in segments a start with a launch
// more, so much a chunk for states and rows, and what it takes to add up each state before the last.
struct Times {
    double start, chunk, seg_start, seg_chunk, join;
};
// As measured of the decayed scan at d = 128.  (d = 64 takes 2.05 us a chunk; its other terms have not been measured,
// and it takes the same numbers of segments.)
constexpr Times kDecayTimes{0.0, 2.8, 11.0, 4.8, 0.7};

double estimate(const Times &t, int64_t chunks, int s) {
    if (s == 1) return t.start + t.chunk * (double)chunks;
    return t.seg_start + t.seg_chunk * (double)((chunks + s - 1) / s) + t.join * s;
}

// Segments of each chain, at most what fills the GPU with one CTA an SM: those of the least estimated
// time.  (More of them than SMs start one after the other: B1 H32 T32768 in four segments 315 us, in
// nine 333 us.)
int segments(const Times &t, int64_t n_chains, int64_t T) {
    const int64_t chunks = (T + C - 1) / C;
    int best = 1;
    for (int s = 2; s <= kSMs / n_chains && s <= chunks; ++s)
        if (estimate(t, chunks, s) < estimate(t, chunks, best)) best = s;
    return best;
}

// Bytes of a scan's workspace: the states of its segments but the last, and X0's copy.
size_t segment_bytes(int64_t n_chains, int d, int nseg) {
    return nseg > 1 ? (size_t)n_chains * nseg * d * d * sizeof(float) : 0;
}

}  // namespace
}  // namespace fw
