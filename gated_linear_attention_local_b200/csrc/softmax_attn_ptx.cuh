// PTX that only the attention kernels use, beside tc_ptx.cuh.
#pragma once

#include "tc_ptx.cuh"

namespace sgla {
namespace tc {

// Dynamic work distribution (PTX clusterlaunchcontrol): a running block asks for a block of the
// same grid that has not started yet; if there is one it will never start, and the caller does
// its work.  The 16-byte answer lands at `resp` (16-byte aligned, shared) and completes 16 bytes
// on `bar`.  No further request may follow an answer of "none".
__device__ __forceinline__ void next_block_request(void *resp, uint64_t *bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(resp)),
                 "r"(smem_u32(bar))
                 : "memory");
}
// The block index x of the answer at `resp`, or -1 for none.
__device__ __forceinline__ int next_block_answer(const void *resp) {
    uint32_t got, x;
    asm volatile(
        "{\n .reg .b128 h;\n .reg .pred p;\n .reg .b32 y, z, w;\n mov.b32 %1, 0;\n ld.shared.b128 h, [%2];\n"
        " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n selp.u32 %0, 1, 0, p;\n"
        " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, h;\n}"
        : "=r"(got), "=r"(x)
        : "r"(smem_u32(resp))
        : "memory");
    return got ? (int)x : -1;
}

// Registers of the executing warpgroup (all four warps take part).
template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// named_sync with a vote: true in every thread if x holds in all of them.
__device__ __forceinline__ bool named_all(int id, int count, bool x) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 q, %3, 0;\n bar.red.and.pred p, %1, %2, q;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(r)
                 : "r"(id), "r"(count), "r"((uint32_t)x)
                 : "memory");
    return r != 0;
}

// True in one lane of a converged warp.  A branch on it is known to the compiler to run in
// one lane, so operands that are the same across the warp stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

}  // namespace tc
}  // namespace sgla
