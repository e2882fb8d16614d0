// fw_decay_tc.cuh -- the tensor-core form of the decayed scans (bf16 rows).
#pragma once

#include "fw_decay.cuh"

namespace fw {

size_t scan_tc_workspace(int64_t n_chains, int64_t T, int d, bool backward);
// n = 1: a forward scan; n = 3: a forward scan and two reverse ones, as fw_decay_backward orders them.
cudaError_t launch_scans_tc(ScanArgs *s, int n, cudaStream_t stream);

}  // namespace fw
