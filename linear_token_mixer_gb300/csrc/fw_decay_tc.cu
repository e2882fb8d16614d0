// fw_decay_tc.cu -- launches of the decayed linear attention scans for bf16 rows (the kernel and its
// figures: fw_scan_tc.cuh).
#include "fw_scan_tc.cuh"

namespace fw {
namespace {

// `follows`: behind another scan of the same call.
template <int D, bool REV>
cudaError_t launch(const ScanArgs *scans, int nseg, bool follows, cudaStream_t s) {
    constexpr int N = REV ? 2 : 1;
    Jobs<N> jobs;
    for (int i = 0; i < N; ++i) {
        const ScanArgs &a = scans[i];
        jobs.s[i].args = a;
        if (!make_map(&jobs.s[i].a, a.a, a.T, a.n_chains, D, C) || !make_map(&jobs.s[i].b, a.b, a.T, a.n_chains, D, C) ||
            !make_map(&jobs.s[i].c, a.c, a.T, a.n_chains, D, C) || !make_map(&jobs.s[i].out, a.out, a.T, a.n_chains, D, 32))
            return cudaErrorInvalidValue;
    }
    const ScanArgs &a = scans[0];
    const int64_t ctas = N * a.n_chains;
    cudaError_t e;
    if (nseg > 1) {
        auto k = scan_tc_kernel<D, REV, true, false, false, false>;
        constexpr int smem = (int)Lay<D, true, false>::ALLOC;
        static std::atomic<uint64_t> pre_done{0};
        if ((e = allow_smem(k, smem, pre_done)) != cudaSuccess) return e;
        if ((e = launch_after(k, dim3((unsigned)(ctas * (nseg - 1))), NTHREADS, smem, s, follows, jobs, nseg, 0,
                              follows ? kWaitLast : 0)) != cudaSuccess)
            return e;
    }
    constexpr int smem = (int)Lay<D, false, false>::ALLOC;
    auto k = scan_tc_kernel<D, REV, false, false, false, false>;
    if constexpr (!REV)                             // (an output norm has no backward pass)
        if (a.norm.on) k = scan_tc_kernel<D, REV, false, true, false, false>;
    static std::atomic<uint64_t> done[2];
    if ((e = allow_smem(k, smem, done[a.norm.on ? 1 : 0])) != cudaSuccess) return e;
    // Padded batches of more chains than SMs: the CTAs of the longest rows start first, so that none
    // of them runs alone in the end.
    const int by_length = a.lens && ctas > kSMs && a.n_chains / a.H <= kMaxRanked;
    return launch_after(k, dim3((unsigned)(ctas * nseg)), NTHREADS, smem, s, nseg > 1 || follows, jobs, nseg,
                        by_length, nseg > 1 ? kWaitFirst : follows ? kWaitLast : 0);
}

// Segments of the forward scan of a backward pass, and of its two reverse ones: a launch after the
// other, each in as many as it likes, or all three scans at once in one piece (B1 H32 T8192 d = 128
// one after the other 280 us, at once 181 us; B1 H8 T4096 d = 64, in segments, 64 us).
void segments_backward(int64_t n_chains, int64_t T, int *fwd, int *rev) {
    const int64_t chunks = (T + C - 1) / C;
    *fwd = segments(kDecayTimes, n_chains, T);
    *rev = segments(kDecayTimes, 2 * n_chains, T);
    const double waves = (double)((3 * n_chains + kSMs - 1) / kSMs);
    if (waves * estimate(kDecayTimes, chunks, 1) <= estimate(kDecayTimes, chunks, *fwd) + estimate(kDecayTimes, chunks, *rev)) *fwd = *rev = 1;
}

template <int D> cudaError_t launch_scans_of(ScanArgs *s, int n, cudaStream_t stream) {
    const int64_t nc = s->n_chains;
    if (n == 1) return launch<D, false>(s, segments(kDecayTimes, nc, s->T), false, stream);
    int fwd, rev;
    segments_backward(nc, s->T, &fwd, &rev);
    s[1].ws = s[0].ws + segment_bytes(nc, D, fwd) / sizeof(float);
    s[2].ws = s[1].ws + segment_bytes(nc, D, rev) / sizeof(float);
    const cudaError_t e = launch<D, false>(s, fwd, false, stream);
    return e != cudaSuccess ? e : launch<D, true>(s + 1, rev, true, stream);
}

}  // namespace

size_t scan_tc_workspace(int64_t n_chains, int64_t T, int d, bool backward) {
    if (!backward) return segment_bytes(n_chains, d, segments(kDecayTimes, n_chains, T));
    int fwd, rev;
    segments_backward(n_chains, T, &fwd, &rev);
    return segment_bytes(n_chains, d, fwd) + 2 * segment_bytes(n_chains, d, rev);
}

cudaError_t launch_scans_tc(ScanArgs *s, int n, cudaStream_t stream) {
    return s->d == 64 ? launch_scans_of<64>(s, n, stream) : launch_scans_of<128>(s, n, stream);
}

}  // namespace fw
