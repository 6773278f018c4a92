// Joins the parts of a row whose keys were split: part p has o_p (the softmax over its keys
// alone) and lse_p, and o = sum_p w_p o_p with w_p = exp(lse_p - max) / sum, the same running
// maximum and sum as inside a part.  One warp a row; reads each part once.
#include <math.h>

#include "softmax_attn.h"

namespace sgla {
namespace {

template <typename T>
__global__ void attn_join_kernel(const float *__restrict__ part_o, const float *__restrict__ part_lse, T *__restrict__ o,
                                 int64_t rows, int parts, int D) {
    const int lane = threadIdx.x & 31;
    const int64_t r = blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5);
    if (r >= rows) return;
    float top = -INFINITY;
    for (int p = lane; p < parts; p += 32) top = fmaxf(top, part_lse[p * rows + r]);
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
    for (int p = 0; p < parts; ++p) {
        const float lse = part_lse[p * rows + r];
        if (lse == -INFINITY) continue;  // no key in this part: its o is not written
        const float w = expf(lse - top);
        sum += w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = lane + 32 * e;
            if (c < D) acc[e] = fmaf(w, part_o[(p * rows + r) * D + c], acc[e]);
        }
    }
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int c = lane + 32 * e;
        if (c < D) o[r * D + c] = from_f32<T>(acc[e] * inv);
    }
}

}  // namespace

cudaError_t launch_attn_join(const float *part_o, const float *part_lse, void *o, int64_t rows, int parts, int D,
                             bool bf16, cudaStream_t st) {
    const unsigned grid = (unsigned)((rows + 7) / 8);
    if (bf16)
        attn_join_kernel<<<grid, 256, 0, st>>>(part_o, part_lse, static_cast<__nv_bfloat16 *>(o), rows, parts, D);
    else
        attn_join_kernel<<<grid, 256, 0, st>>>(part_o, part_lse, static_cast<float *>(o), rows, parts, D);
    return cudaGetLastError();
}

}  // namespace sgla
