// What the tensor-core kernels of softmax attention share.
#pragma once

#include "softmax_attn_ptx.cuh"
#include "tc_tiles.cuh"

namespace sgla {
namespace {

// Registers a thread of a 384-thread kernel: 168 at launch; its eight row warps take 216, the
// others keep 72 (256 * 216 + 128 * 72 = 64512 = 384 * 168).  With 224 and 56 the product warps spill
// (dk dv of 2 x 4096 tokens, 16 heads on 4: 254 us for 231).
constexpr int kRowRegs = 216, kOtherRegs = 72;
constexpr float kLog2e = 1.4426950408889634f;

// Exponentials on the FMA pipe: with n = round(x), f = x - n, 2^x = 2^n p3(f), p3 the degree-3
// polynomial of least largest relative error on [-1/2, 1/2] (Remez exchange; 7.5e-5, a fiftieth
// of the rounding of p to bf16 that follows).
// (2^x, 2^y) on the FMA pipe for x, y < 128.  2^n is formed as a factor of its own: 0 for n = -127, to
// which lower arguments (-inf among them) are raised, so that what weighs nothing weighs 0.
__device__ __forceinline__ float2 exp2_fma(float2 x) {
    const float2 magic = make_float2(12582912.f, 12582912.f);  // 1.5 * 2^23: the sum's low bits are round(x)
    asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x.x));  // -127, a NaN stays
    asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x.y));
    const float2 t = __fadd2_rn(x, magic);
    const float2 f = __fadd2_rn(x, __fadd2_rn(magic, make_float2(-t.x, -t.y)));
    float2 p = __ffma2_rn(f, make_float2(0.0551716685f, 0.0551716685f), make_float2(0.2426111251f, 0.2426111251f));
    p = __ffma2_rn(p, f, make_float2(0.6932609677f, 0.6932609677f));
    p = __ffma2_rn(p, f, make_float2(0.9999280572f, 0.9999280572f));  // NaN for NaN
    return __fmul2_rn(p, make_float2(__int_as_float((__float_as_int(t.x) << 23) + 0x3f800000),
                                     __int_as_float((__float_as_int(t.y) << 23) + 0x3f800000)));
}

// -lse in units of log2, for p = 2^(sc s - lse): a row whose lse is -inf saw nothing, or only scores
// of -inf, and all its p are 0.
__device__ __forceinline__ float neg_lse(float lse) { return lse == -INFINITY ? -INFINITY : -kLog2e * lse; }

// 32 columns of an output row, the first `left` of them (a multiple of 8), as bf16 to dst.  Every
// lane of a warp stores another row, so an instruction touches 32 lines whatever its width: 32
// bytes at a time where rows are aligned to that (`wide`), else 16.
__device__ __forceinline__ void store_cols32(__nv_bfloat16 *dst, const float (&o)[32], int left, bool wide) {
    uint32_t u[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) u[e] = pack_bf16(o[2 * e], o[2 * e + 1]);
    if (wide) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (16 * e < left) {
                const uint32_t v[8] = {u[8 * e], u[8 * e + 1], u[8 * e + 2], u[8 * e + 3],
                                       u[8 * e + 4], u[8 * e + 5], u[8 * e + 6], u[8 * e + 7]};
                st_global_v8(dst + 16 * e, v);
            }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (8 * e < left)
                *reinterpret_cast<uint4 *>(dst + 8 * e) = make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
    }
}
inline bool wide_rows(const void *p, int D) { return D % 16 == 0 && reinterpret_cast<uintptr_t>(p) % 32 == 0; }

// mbar_wait by all lanes of a warp, with one answer for all: a lane that gave up must not leave the
// others at a warp-wide instruction.
__device__ __forceinline__ bool all_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
}

// A wait that lasts as long as an item, and an item may have any number of tiles (a wait for one tile
// is bounded by itself): gives up when `copies` stood still for the limit, or another thread gave
// up.  IDLE: off the critical path, sleeps in the barrier.
template <bool IDLE>
__device__ __forceinline__ bool item_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, volatile int *copies) {
    auto poll = [&] { return IDLE ? mbar_try_wait_hint(bar, parity, 20000u) : mbar_try_wait(bar, parity); };
    if (poll()) return true;
    uint64_t start = globaltimer_ns();
    int seen = *copies;
    while (true) {
        if (poll()) return true;
        if (*abort_flag) return false;
        if (globaltimer_ns() - start > kWaitLimitNs) {
            const int now = *copies;
            if (now == seen) {
                *abort_flag = 1;
                return false;
            }
            seen = now;
            start = globaltimer_ns();
        }
    }
}

// Work items of a kernel whose grid has a block for every item but whose CTAs stay on their SM: a
// scheduler warp takes over blocks that have not started (clusterlaunchcontrol), describes them
// and hands the description to the other warps.  It asks when the copies of the item in work
// have all been issued: early enough to hide the answer, late enough not to hold an item back
// from SMs that run idle before (asking at the item's start instead: dk dv of 2 x 4096 tokens,
// 1.7 items a CTA, 325 us for 229 us).  Item has int n, the tiles of the item; n < 0: no more.
constexpr int kFeedWarps = 10;  // warps that take items: eight row warps, copies, products
template <typename Item>
struct Feed {
    uint64_t *full, *empty, *want, *next;  // description written, taken, next one wanted, answer arrived
    void *answer;                   // 16 bytes, 16-byte aligned
    Item *item;
    volatile int *abort_flag;
    volatile int *copies;           // changes with every tile copied and every block looked at

    __device__ void init() const {
        *abort_flag = 0;
        *copies = 0;
        mbar_init(full, 1);
        mbar_init(empty, kFeedWarps);
        mbar_init(want, 1);
        mbar_init(next, 1);
    }
    // The next item, by all lanes of a warp; false when there is none.
    __device__ bool take(int &count, Item &it) const {
        if (!__all_sync(0xffffffffu, item_wait<false>(full, count & 1, abort_flag, copies))) return false;
        it = *item;
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(empty);
        ++count;
        return it.n >= 0;
    }
    // The scheduler warp: describe(u, it) fills the item of block u, false if it has nothing to do.
    template <typename F>
    __device__ void run(F describe) const {
        const int lane = threadIdx.x & 31;
        int count = 0;
        bool ok = true;
        auto publish = [&](const Item &it) {
            if (count > 0) ok = __all_sync(0xffffffffu, item_wait<true>(empty, (count - 1) & 1, abort_flag, copies));
            if (ok && lane == 0) {
                *item = it;
                mbar_arrive(full);
            }
            __syncwarp();
            ++count;
        };
        for (int u = blockIdx.x, asked = 0; ok && u >= 0;) {
            Item it;
            *copies = u;  // (blocks without work may come in long runs: that is progress, too)
            if (describe(u, it)) {
                publish(it);
                if (!ok || !(ok = __all_sync(0xffffffffu, item_wait<true>(want, (count - 1) & 1, abort_flag, copies)))) break;
            }
            __syncwarp();
            if (lane == 0) {
                fence_proxy_async_smem();  // the last answer has been read
                mbar_arrive_expect_tx(next, 16);
                next_block_request(answer, next);
            }
            __syncwarp();
            if (!(ok = all_wait(next, asked & 1, abort_flag))) {
                if (lane == 0) mbar_drain(next, asked & 1);  // no answer into shared memory that is given up
                break;
            }
            ++asked;
            u = next_block_answer(answer);
            __syncwarp();
        }
        Item end{};
        end.n = -1;
        if (ok) publish(end);
    }
};

// A ring of N stages: the stage in turn and the parity of its use.
template <int N>
struct Ring {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void step() {
        if (++s == N) {
            s = 0;
            ph ^= 1u;
        }
    }
};

}  // namespace
}  // namespace sgla
