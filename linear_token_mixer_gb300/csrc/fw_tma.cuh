// fw_tma.cuh -- tensor maps of the kernels that load their rows by TMA.
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace fw {

// [n_chains][T][d] bf16 as a 3-D tensor (d, T, chain), boxes of 64 columns and `rows` rows with the
// 128-byte swizzle; rows behind T read as zero.  False where the driver refuses it.
bool make_map(CUtensorMap *m, const void *ptr, int64_t T, int64_t n_chains, int d, int rows);

}  // namespace fw
