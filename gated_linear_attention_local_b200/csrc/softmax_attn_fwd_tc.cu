// Softmax attention forward on the tensor cores (tcgen05 / TMEM / TMA), bf16 operands.
//
// One CTA takes two tiles of 128 packed rows (row = token * G + g of one key head, R = 128 / G
// tokens a tile) and walks the keys in tiles of 128.  For each tile w of rows and key tile j
//   S_w = Q_w K_j^T            (128 x 128, fp32 in tensor memory)
//   p   = 2^(sc S - m)         one thread a row: maximum and sum need no shuffles
//   O_w += P_w V_j             P_w in bf16 in tensor memory, over S_w's columns
// The two row tiles alternate: while one's 128 threads form p, the tensor cores run the other's
// products.  The tensor pipe executes in issue order, so S_w(j+1) may follow P_w(j) V_j at
// once although it overwrites P_w(j).
//
// The maximum m of a row is only moved (and O, l rescaled, in tensor memory, by the row's own
// thread) when it has grown by more than 2^8: until then p <= 2^8, which fp32 sums and the
// bf16 range (the rounding is relative) carry without loss.
//
// p is rounded to bf16 for the product with V (relative 2^-8, averaged over the keys); its sum
// l, m, S and O are fp32.
//
// Tensor memory (512 columns): S0, S1 [0, 256), O0, O1 [256, 512).
// Shared memory (DP = 128): Q 64 KB, rings of two K and two V tiles 128 KB.
// Warps: 0-3 rows of tile 0, 4-7 rows of tile 1, 8 TMA, 9 MMA (10, 11 fill its warpgroup).
#include <math.h>

#include <algorithm>

#include "softmax_attn.h"
#include "tc_path.h"
#include "tc_ptx.cuh"
#include "tc_tiles.cuh"

namespace sgla {

using namespace tc;

namespace {

constexpr int kFwdThreads = 384;
// Registers a thread: 168 at launch; the row warps take 208, the others keep 80
// (256 * 208 + 128 * 80 = 63488 of 384 * 168 = 64512).
constexpr int kRowRegs = 208, kOtherRegs = 80;
constexpr int kTile = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.f;  // log2 units the maximum may lag behind

template <int DP>
struct FwdCfg {
    static constexpr int NG = DP / 64;               // 64-column groups of a tile
    static constexpr uint32_t T = NG * kRegion;      // one tile, bytes
    static constexpr uint32_t Q0 = 0, K0 = 2 * T, V0 = 4 * T;
    static constexpr uint32_t BARS = 6 * T, MISC = BARS + 20 * 8;
    // at least half of an SM's shared memory: the CTA takes all of its tensor memory
    static constexpr size_t SMEM = MISC + 16 + 1024 > 120 * 1024 ? MISC + 16 + 1024 : 120 * 1024;
    static constexpr uint32_t COL_O = 256;
    static_assert(SMEM <= 232448, "shared memory budget");
};

template <int DP>
__global__ void __launch_bounds__(kFwdThreads, 1)
attn_fwd_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv, AttnArgs a, int R) {
    using C = FwdCfg<DP>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = align1024(smem_raw);
    AttnTile t;
    const int hk = blockIdx.x % a.Hk;
    // heaviest first: a causal sequence's last rows see the most keys
    int64_t slot = gridDim.x / a.Hk - 1 - blockIdx.x / a.Hk;
    if (!a.sq.cu) {
        const int64_t per = gridDim.x / a.Hk / a.N;
        slot = (slot % a.N) * per + slot / a.N;
    }
    if (!attn_locate(a, true, slot, 1, 2 * R, t)) return;
    const int64_t kb = (int64_t)blockIdx.y * a.split, ke = min64(t.tk, kb + a.split);
    // key tiles of each row tile: up to the last key its last row sees
    int nt[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int64_t last = min64(t.row0 + (w + 1) * R, t.tq) - 1;  // last token
        int64_t lim = a.causal ? min64(ke, last + 1 + t.tk - t.tq) : ke;
        if (t.row0 + w * R >= t.tq) lim = 0;
        nt[w] = lim > kb ? (int)((lim - kb + kTile - 1) / kTile) : 0;
    }
    const int n = max(nt[0], nt[1]);

    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::BARS);
    uint64_t *full_q = bars, *full_k = bars + 2, *full_v = bars + 4;   // [2]
    uint64_t *empty_k = bars + 6, *empty_v = bars + 8;                 // [2]
    uint64_t *b_s = bars + 10, *b_p = bars + 12, *b_o = bars + 14;     // [2] per row tile
    uint64_t *b_drain = bars + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + C::MISC + 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int b = 0; b < 12; ++b) mbar_init(&bars[b], 1);
        mbar_init(&b_p[0], 128);
        mbar_init(&b_p[1], 128);
        mbar_init(&b_o[0], 1);
        mbar_init(&b_o[1], 1);
        mbar_init(b_drain, 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 8) {
        // ---------------------------------------------------------------- TMA producer
        setmaxnreg_dec<kOtherRegs>();
        if (lane == 0) {
            const uint32_t qbytes = (uint32_t)(R * a.G) * 128u * C::NG;
            for (int w = 0; w < 2; ++w) {
                if (nt[w] == 0) continue;
                mbar_arrive_expect_tx(&full_q[w], qbytes);
                for (int g = 0; g < C::NG; ++g)
                    tma_load_3d(sm + C::Q0 + w * C::T + g * kRegion, &tq, &full_q[w], 64 * g, hk * a.G,
                                (int)(t.q0 + t.row0 + w * R));
            }
            int j = 0;
            for (; j < n; ++j) {
                const int st = j & 1;
                const uint32_t ph = ((j >> 1) - 1) & 1;
                const int tok = (int)(t.k0 + kb + (int64_t)j * kTile);
                if (j >= 2 && !mbar_wait_idle(&empty_k[st], ph, abort_flag)) break;
                mbar_arrive_expect_tx(&full_k[st], C::T);
                for (int g = 0; g < C::NG; ++g)
                    tma_load_3d(sm + C::K0 + st * C::T + g * kRegion, &tk, &full_k[st], 64 * g, hk, tok);
                if (j >= 2 && !mbar_wait_idle(&empty_v[st], ph, abort_flag)) break;
                mbar_arrive_expect_tx(&full_v[st], C::T);
                for (int g = 0; g < C::NG; ++g)
                    tma_load_3d(sm + C::V0 + st * C::T + g * kRegion, &tv, &full_v[st], 64 * g, hk, tok);
            }
            if (*abort_flag) {  // let the copies in flight land before the CTA exits
                for (int w = 0; w < 2; ++w)
                    if (nt[w]) mbar_drain(&full_q[w], 0);
                for (int i = max(0, j - 2); i <= min(j, n - 1); ++i) mbar_drain(&full_k[i & 1], (i >> 1) & 1);
                for (int i = max(0, j - 2); i < j; ++i) mbar_drain(&full_v[i & 1], (i >> 1) & 1);
            }
        }
    } else if (warp == 9) {
        // ---------------------------------------------------------------- MMA issuer
        setmaxnreg_dec<kOtherRegs>();
        const uint32_t idS = idesc_bf16_f32(128, 128, false, false);
        const int nk = (a.D + 15) / 16;  // 16-column steps of a head (zeros past D)
        const uint32_t idO = idesc_bf16_f32(128, 16 * nk, false, true);
        const uint32_t sbase = smem_u32(sm);
        auto wait = [&](uint64_t *bar, uint32_t ph) { return mbar_wait(bar, ph, abort_flag); };
        auto issue_S = [&](int w, int j) {
            if (lane == 0) {
                const uint32_t qa = sbase + C::Q0 + w * C::T, ka = sbase + C::K0 + (j & 1) * C::T;
                for (int kk = 0; kk < nk; ++kk) {
                    const uint32_t off = (kk >> 2) * kRegion + (kk & 3) * 32;
                    mma_bf16(tmem + w * 128, kdesc(qa + off), kdesc(ka + off), idS, kk > 0 ? 1u : 0u);
                }
                mma_commit(&b_s[w]);
            }
            __syncwarp();
        };
        bool ok = true;
        for (int j = -1; ok && j < n; ++j) {
            const int st = j & 1;
            bool vready = false, kready = false;
            for (int w = 0; ok && w < 2; ++w) {
                if (j >= 0 && j < nt[w]) {
                    if (!vready) {
                        if (!(ok = wait(&full_v[st], (j >> 1) & 1))) break;
                        vready = true;
                        const int64_t valid = t.tk - (kb + (int64_t)j * kTile);
                        if (valid < kTile) {
                            // rows behind the sequence's keys hold its neighbour's data: 0 * NaN must not arise
                            for (int i = lane; i < C::NG * 8 * kTile; i += 32) {
                                const int r = (i >> 3) & (kTile - 1);
                                if (r >= valid)
                                    *reinterpret_cast<uint4 *>(sm + C::V0 + st * C::T + (i >> 10) * kRegion + r * 128 +
                                                               (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                    }
                    if (!(ok = wait(&b_p[w], j & 1))) break;
                    tc_fence_after();
                    if (lane == 0) {
                        const uint32_t va = sbase + C::V0 + st * C::T;
#pragma unroll
                        for (int jj = 0; jj < kTile / 16; ++jj)
                            mma_bf16_tmem_a(tmem + C::COL_O + w * 128, tmem + w * 128 + jj * 8,
                                            sdesc(va + jj * 2048, kRegion, 1024, 2), idO, (j > 0 || jj > 0) ? 1u : 0u);
                        if (j == nt[w] - 1) mma_commit(&b_o[w]);
                    }
                    __syncwarp();
                }
                if (j + 1 < nt[w]) {
                    if (j < 0 && !(ok = wait(&full_q[w], 0))) break;
                    if (!kready) {
                        if (!(ok = wait(&full_k[(j + 1) & 1], ((j + 1) >> 1) & 1))) break;
                        kready = true;
                    }
                    tc_fence_after();
                    issue_S(w, j + 1);
                }
            }
            if (ok && lane == 0) {
                if (j >= 0) mma_commit(&empty_v[st]);
                if (j + 1 < n) mma_commit(&empty_k[(j + 1) & 1]);
            }
            __syncwarp();
        }
        if (lane == 0) {
            mma_commit(b_drain);
            mbar_drain(b_drain, 0);
        }
    } else if (warp < 8) {
        // ---------------------------------------------------------------- softmax: one row a thread
        setmaxnreg_inc<kRowRegs>();
        const int w = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
        const uint32_t cS = tmem + w * 128 + lanes, cO = tmem + C::COL_O + w * 128 + lanes;
        const int tr = r / a.G;
        const int64_t tok = t.row0 + w * R + tr;
        const bool mine = tr < R && tok < t.tq;
        int64_t lim64 = mine ? (a.causal ? min64(ke, tok + 1 + t.tk - t.tq) : ke) : 0;
        const int lim = (int)(lim64 > kb ? lim64 - kb : 0);  // keys of this split that the row sees
        const float sc = a.scale * kLog2e;
        float m = -INFINITY, l = 0.f;  // m in units of S
        bool ok = true;
        for (int j = 0; j < nt[w]; ++j) {
            if (!(ok = mbar_wait(&b_s[w], j & 1, abort_flag))) break;
            tc_fence_after();
            float s[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(cS + 32 * c, s[c]);
            tmem_wait_ld();
            const int left = lim - j * kTile;
            if (__any_sync(0xffffffffu, left < kTile)) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * c + e >= left) s[c][e] = -INFINITY;
            }
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 32; ++e) top = fmaxf(top, s[c][e]);
            // move the maximum when it has grown by more than kGrow (or there was none)
            float f = 1.f;
            if ((top - m) * sc > kGrow) {
                f = fast_exp2((m - top) * sc);  // 0 from m = -inf
                m = top;
            }
            if (__any_sync(0xffffffffu, f != 1.f)) {
                l *= f;
                if (j > 0) {
                    for (int c = 0; c < a.D; c += 32) {
                        float o[32];
                        tmem_ld32(cO + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= f;
                        tmem_st32(cO + c, o);
                    }
                    tmem_wait_st();
                }
            }
            const float ms = m == -INFINITY ? 0.f : m * sc;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t p[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float x = fast_exp2(fmaf(s[c][e], sc, -ms)), y = fast_exp2(fmaf(s[c][e + 1], sc, -ms));
                    sum[(e >> 1) & 3] += x + y;
                    p[e >> 1] = pack_bf16(x, y);
                }
                tmem_st16(cS + 16 * c, p);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&b_p[w]);
        }
        if (ok && nt[w] > 0) ok = mbar_wait(&b_o[w], 0, abort_flag);
        if (ok) {
            tc_fence_after();
            const int64_t row = (t.q0 + tok) * a.H + hk * a.G + (r - tr * a.G);
            const int64_t prow = (int64_t)blockIdx.y * a.part_rows + row;
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN scores stay NaN
            const float lse = l > 0.f ? m * a.scale + log2f(l) * kLn2 : (l == 0.f ? -INFINITY : l);
            if (mine) {
                if (a.part_lse) a.part_lse[prow] = lse;
                else if (a.lse) a.lse[row] = lse;
            }
            for (int c = 0; c < a.D; c += 32) {
                float o[32];
                if (nt[w] > 0) {
                    tmem_ld32(cO + c, o);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = l == 0.f ? 0.f : o[e] * inv;
                if (!mine) continue;
                if (a.part_o) {
                    float4 *dst = reinterpret_cast<float4 *>(a.part_o + prow * a.D + c);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c + 4 * e < a.D)
                            dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                } else {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + row * a.D + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + 8 * e < a.D)
                            dst[e] = make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                                pack_bf16(o[8 * e + 4], o[8 * e + 5]),
                                                pack_bf16(o[8 * e + 6], o[8 * e + 7]));
                }
            }
        } else if (a.status) {
            atomicExch(a.status, kDevTimeout);
        }
    } else {
        setmaxnreg_dec<kOtherRegs>();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int DP>
cudaError_t launch_fwd(const AttnArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, int R,
                       cudaStream_t st) {
    auto kern = attn_fwd_tc_kernel<DP>;
    constexpr size_t smem = FwdCfg<DP>::SMEM;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(attn_slots(a.sq, a.N, 1, 2 * R) * a.Hk), a.nsplit);
    kern<<<grid, kFwdThreads, smem, st>>>(tq, tk, tv, a, R);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_fwd_tc(const AttnArgs &a, cudaStream_t st) {
    const int R = kTile / a.G;
    const int64_t qt = a.sq.cu ? a.sq.T : a.N * a.sq.T, kt = a.sk.cu ? a.sk.T : a.N * a.sk.T;
    CUtensorMap tq, tk, tv;
    cudaError_t e = tc_make_map_rows(&tq, a.q, qt, a.H, a.D, a.G, R);
    if (e != cudaSuccess) return e;
    if (kt > 0) {
        if ((e = tc_make_map_rows(&tk, a.k, kt, a.Hk, a.D, 1, kTile)) != cudaSuccess) return e;
        if ((e = tc_make_map_rows(&tv, a.v, kt, a.Hk, a.D, 1, kTile)) != cudaSuccess) return e;
    } else {
        tk = tv = tq;  // no key anywhere: never used
    }
    return a.D <= 64 ? launch_fwd<64>(a, tq, tk, tv, R, st) : launch_fwd<128>(a, tq, tk, tv, R, st);
}

}  // namespace sgla
