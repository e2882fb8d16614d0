// fw_decay_tc.cuh -- the tensor-core form of the decayed scans (bf16 rows).
#pragma once

#include "fw_decay.cuh"

namespace fw {

size_t scan_tc_workspace(int64_t n_chains, int64_t T, int d);
// `follows`: behind another scan of the same call, of which it is independent.
cudaError_t launch_scan_tc(const ScanArgs &a, bool follows, cudaStream_t s);

}  // namespace fw
