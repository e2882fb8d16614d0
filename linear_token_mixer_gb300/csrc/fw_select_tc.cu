// fw_select_tc.cu -- launches of the selective scan for bf16 rows (the kernel: fw_scan_tc.cuh).
#include "fw_scan_tc.cuh"
#include "fw_select.cuh"

namespace fw {
namespace {

// Measured of this scan (a segment's decay is summed over its chunks' logs for each 16 columns of a state, which is most of
// what joining takes).  Best of all numbers of segments, with that of the decayed scan's times in brackets: d = 128
// H8 T4096 4, 71 us (16, 111); H8 T16384 10, 139 us (19, 164); H16 T2048 4, 55 us (8, 70; in one piece 66); H32
// T32768 4, 395 us (4); d = 64 H8 T4096 8, 43 us (16, 55), H16 T2048 4, 35 us (8, 39).
constexpr Times kTimes128{9.0, 3.4, 11.3, 5.4, 5.7}, kTimes64{5.0, 2.4, 9.0, 3.9, 2.15};
int pieces(int64_t n_chains, int64_t T, int d) { return segments(d == 64 ? kTimes64 : kTimes128, n_chains, T); }

// As the decayed scan's: chains in segments where they are few.
template <int D> cudaError_t launch(const ScanArgs &a, cudaStream_t s) {
    const int nseg = pieces(a.n_chains, a.T, D);
    const int64_t ab = a.n_chains / a.H * a.sel.gate.G;
    Jobs<1> jobs;
    jobs.s[0].args = a;
    if (!make_map(&jobs.s[0].a, a.a, a.T, ab, D, C) || !make_map(&jobs.s[0].b, a.b, a.T, ab, D, C) ||
        !make_map(&jobs.s[0].c, a.c, a.T, a.n_chains, D, C) || !make_map(&jobs.s[0].out, a.out, a.T, a.n_chains, D, 32))
        return cudaErrorInvalidValue;
    cudaError_t e;
    if (nseg > 1) {
        auto k = scan_tc_kernel<D, false, true, false, true, false>;
        constexpr int smem = (int)Lay<D, true, true>::ALLOC;
        static std::atomic<uint64_t> pre_done{0};
        if ((e = allow_smem(k, smem, pre_done)) != cudaSuccess) return e;
        if ((e = launch_after(k, dim3((unsigned)(a.n_chains * (nseg - 1))), NTHREADS, smem, s, false, jobs, nseg, 0, 0)) !=
            cudaSuccess)
            return e;
    }
    constexpr int smem = (int)Lay<D, false, true>::ALLOC;
    const bool skip = a.sel.gate.skip != nullptr;
    auto k = skip ? scan_tc_kernel<D, false, false, false, true, true> : scan_tc_kernel<D, false, false, false, true, false>;
    static std::atomic<uint64_t> done[2];
    if ((e = allow_smem(k, smem, done[skip ? 1 : 0])) != cudaSuccess) return e;
    const int by_length = a.lens && a.n_chains > kSMs && a.n_chains / a.H <= kMaxRanked;
    return launch_after(k, dim3((unsigned)(a.n_chains * nseg)), NTHREADS, smem, s, nseg > 1, jobs, nseg, by_length,
                        nseg > 1 ? kWaitFirst : 0);
}

}  // namespace

// [c][w][ends][chunk][states of segments]: each a multiple of 16 bytes.
static size_t chunks_of(int64_t n_chains, int64_t T) { return (size_t)n_chains * (size_t)((T + C - 1) / C); }
static size_t even(size_t n) { return n + (n & 1); }
size_t select_workspace_tc(int64_t n_chains, int64_t T, int d) {
    const size_t n = chunks_of(n_chains, T);
    return n * (C * (sizeof(float2) + sizeof(float)) + sizeof(float4)) + even(n) * sizeof(float2) +
           segment_bytes(n_chains, d, pieces(n_chains, T, d));
}
cudaError_t launch_select_tc(const ScanArgs &scan, cudaStream_t stream) {
    ScanArgs s = scan;
    const size_t n = chunks_of(s.n_chains, s.T);
    s.sel.n_chunks = (s.T + C - 1) / C;
    s.sel.c = reinterpret_cast<float2 *>(s.ws);
    s.sel.w = reinterpret_cast<float *>(s.sel.c + n * C);
    s.sel.ends = reinterpret_cast<float4 *>(s.sel.w + n * C);
    s.sel.chunk = reinterpret_cast<float2 *>(s.sel.ends + n);
    s.ws = reinterpret_cast<float *>(s.sel.chunk + even(n));
    return s.d == 64 ? launch<64>(s, stream) : launch<128>(s, stream);
}

}  // namespace fw
