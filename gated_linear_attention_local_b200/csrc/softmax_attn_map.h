// Tensor maps of the attention kernels (internal to libsimplegla.so).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace sgla {

// 3-D TMA map over a [tokens, H, D] tensor, box [box_tokens x box_heads x 128 bytes of
// columns] (64 bf16 or 32 fp32), 128-byte swizzle: the rows (token, head) of a box land as
// consecutive 128-byte rows.
cudaError_t tc_make_map_rows(CUtensorMap *m, const void *ptr, int64_t tokens, int H, int D, int box_heads,
                             int box_tokens, bool f32 = false);

}  // namespace sgla
