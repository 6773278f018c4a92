// Softmax attention backward on the tensor cores (tcgen05 / TMEM / TMA), bf16 operands.
//
// The probabilities are recomputed, p = 2^(sc s - lse), and with delta_i = sum_d do_id o_id
//   dv_j = sum_i p_ij do_i,  ds_ij = p_ij (do_i . v_j - delta_i),
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i.
// Two kernels, one per output side, so that every sum has one owner and one order (no
// atomics, no fp32 copy of dq in memory); the price is that s, do v and p are formed twice,
// 7 products of the tile instead of 5.
//
// dk, dv: one CTA owns 128 keys of one key head and walks the rows that see them in sub-tiles
// of 64 packed rows (row = token * G + g), two of which are in work at a time:
//   S^T = K Q^T, dP^T = V dO^T   (128 keys x 64 rows, fp32, tensor memory; a thread a key)
//   dV += P^T dO,  dK += dS^T Q  (P^T, dS^T in bf16 over S^T's and dP^T's columns)
// dq: one CTA owns 128 packed rows and walks the keys they see in sub-tiles of 64:
//   S = Q K^T, dP = dO V^T, dQ += dS K   (a thread a row)
// Two warpgroups take the sub-tiles in turn; while one forms p and ds the tensor cores run
// the other's products.  The tensor pipe executes in issue order, so the products of sub-tile
// i + 2 may overwrite the scores' columns right after those that read P and dS of sub-tile i.
//
// P and dS are rounded to bf16 for their products (relative 2^-8 each, averaged over the
// sum); scores, p, ds, lse, delta and every accumulator are fp32.
//
// Tensor memory (512 columns): S 2 x 64, dP 2 x 64, accumulators from column 256.
// Shared memory (DP = 128): the CTA's own two tiles 64 KB, a ring of four sub-tile pairs 128 KB.
// Warps: 0-3 and 4-7 the warpgroups, 8 TMA, 9 MMA.
#include <math.h>

#include <algorithm>

#include "softmax_attn.h"
#include "tc_path.h"
#include "tc_ptx.cuh"
#include "tc_tiles.cuh"

namespace sgla {

using namespace tc;

namespace {

constexpr int kBwdThreads = 320;
constexpr int kTile = 128, kSub = 64, kStages = 4;
constexpr uint32_t kSubRegion = kSub * 128;  // [64 rows x 64 bf16], bytes
constexpr float kLog2e = 1.4426950408889634f;

template <int DP>
struct BwdCfg {
    static constexpr int NG = DP / 64;
    static constexpr uint32_t T = NG * kRegion;      // own tile (128 rows)
    static constexpr uint32_t ST = NG * kSubRegion;  // sub-tile (64 rows)
    static constexpr uint32_t A0 = 0, B0 = T;        // own tiles: K, V (dk dv) or Q, dO (dq)
    static constexpr uint32_t X0 = 2 * T;            // ring: stage s holds X at X0 + 2 s ST, Y one ST further
    static constexpr uint32_t ROWS = X0 + 2 * kStages * ST;  // [2][128] floats: lse, delta of a sub-tile's rows
    static constexpr uint32_t BARS = ROWS + 2 * 128 * 4;
    static constexpr uint32_t MISC = BARS + 24 * 8;
    static constexpr size_t SMEM = MISC + 16 + 1024 > 120 * 1024 ? MISC + 16 + 1024 : 120 * 1024;
    static constexpr uint32_t COL_S = 0, COL_DP = 128, COL_ACC = 256;
    static_assert(SMEM <= 232448, "shared memory budget");
};

struct BwdBars {
    uint64_t *own, *full, *empty, *s, *dp, *p, *ds, *done, *drain;
    __device__ explicit BwdBars(uint64_t *b)
        : own(b), full(b + 1), empty(b + 5), s(b + 9), dp(b + 11), p(b + 13), ds(b + 15), done(b + 17), drain(b + 18) {}
    __device__ void init() const {
        mbar_init(own, 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s[i], 1);
            mbar_init(&dp[i], 1);
            mbar_init(&p[i], 128);
            mbar_init(&ds[i], 128);
        }
        mbar_init(done, 1);
        mbar_init(drain, 1);
    }
};

// Zero rows [from, 64) of a sub-tile pair, by one warp.
template <int NG>
__device__ __forceinline__ void zero_rows(unsigned char *pair, int from, int lane) {
    for (int i = lane; i < 2 * NG * kSub * 8; i += 32)
        if (((i >> 3) & (kSub - 1)) >= from) reinterpret_cast<uint4 *>(pair)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
}

__device__ __forceinline__ void ld64(uint32_t taddr, float (&v)[64]) {
    float x[32], y[32];
    __syncwarp();
    tmem_ld32(taddr, x);
    tmem_ld32(taddr + 32, y);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        v[e] = x[e];
        v[32 + e] = y[e];
    }
}

__device__ __forceinline__ void st64_bf16(uint32_t taddr, const float (&v)[64]) {
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = pack_bf16(v[32 * c + 2 * e], v[32 * c + 2 * e + 1]);
        tmem_st16(taddr + 16 * c, w);
    }
    tmem_wait_st();
}

// Columns [0, D) of this thread's accumulator row times f, as bf16 to dst (zeros with !any).
__device__ __forceinline__ void store_acc(uint32_t taddr, bool any, bool mine, __nv_bfloat16 *dst, int D, float f) {
    __syncwarp();
    for (int c = 0; c < D; c += 32) {
        float o[32];
        if (any) {
            tmem_ld32(taddr + c, o);
            tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = any ? o[e] * f : 0.f;
        if (mine)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + 8 * e < D)
                    *reinterpret_cast<uint4 *>(dst + c + 8 * e) =
                        make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                   pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7]));
        __syncwarp();  // the next tensor memory read is the whole warp's
    }
}

// Producer: the CTA's own tiles, then the ring.  own(bar) and sub(i, dst, bar) issue the copies.
template <int DP, typename Own, typename Sub>
__device__ __forceinline__ void produce(unsigned char *sm, const BwdBars &b, int n, uint32_t own_bytes,
                                        uint32_t sub_bytes, volatile int *abort_flag, Own own, Sub sub) {
    using C = BwdCfg<DP>;
    mbar_arrive_expect_tx(b.own, own_bytes);
    own(b.own);
    int i = 0;
    for (; i < n; ++i) {
        const int st = i % kStages;
        if (i >= kStages && !mbar_wait_idle(&b.empty[st], ((i / kStages) - 1) & 1, abort_flag)) break;
        mbar_arrive_expect_tx(&b.full[st], sub_bytes);
        sub(i, sm + C::X0 + 2 * st * C::ST, &b.full[st]);
    }
    if (*abort_flag) {  // let the copies in flight land before the CTA exits
        mbar_drain(b.own, 0);
        for (int k = max(0, i - kStages); k < i; ++k) mbar_drain(&b.full[k % kStages], (k / kStages) & 1);
    }
}

// ------------------------------------------------------------------------------------ dk, dv
template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
attn_dkdv_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdo,
                    const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, AttnArgs a,
                    int gb, int R) {
    // a sub-tile: R tokens x gb heads (gb = min(G, 64), R = 64 / gb); G > 64 takes several a token
    using C = BwdCfg<DP>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = align1024(smem_raw);
    AttnTile t;
    const int hk = blockIdx.x % a.Hk;
    int64_t slot = blockIdx.x / a.Hk;
    if (!a.sk.cu) {  // the first keys are seen by the most rows: every sequence's first tiles first
        const int64_t per = gridDim.x / a.Hk / a.N;
        slot = (slot % a.N) * per + slot / a.N;
    }
    if (!attn_locate(a, false, slot, 1, kTile, t)) return;
    const int64_t j0 = t.row0, off = t.tk - t.tq;
    const int chunks = (a.G + gb - 1) / gb;
    const int64_t first = a.causal ? max((int64_t)0, j0 - off) : 0;  // first token that sees key j0
    const int64_t b0 = first / R;                                    // its token block
    const int n = first < t.tq ? (int)((t.tq + R - 1) / R - b0) * chunks : 0;
    auto token0 = [&](int i) { return (b0 + i / chunks) * R; };
    // rows of sub-tile i that exist
    auto rows_of = [&](int i) {
        return chunks > 1 ? min(gb, a.G - (i % chunks) * gb) : (int)min64(R, t.tq - token0(i)) * gb;
    };

    const BwdBars b(reinterpret_cast<uint64_t *>(sm + C::BARS));
    float *srow = reinterpret_cast<float *>(sm + C::ROWS);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + C::MISC + 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        b.init();
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (R * gb < kSub)  // rows that no copy writes are operands too
        for (int s = warp; s < kStages; s += kBwdThreads / 32)
            zero_rows<C::NG>(sm + C::X0 + 2 * s * C::ST, R * gb, lane);
    if (warp == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 8) {
        if (lane == 0 && n > 0)
            produce<DP>(
                sm, b, n, 2 * C::T, 2u * C::NG * R * gb * 128, abort_flag,
                [&](uint64_t *bar) {
                    for (int g = 0; g < C::NG; ++g) {
                        tma_load_3d(sm + C::A0 + g * kRegion, &tk, bar, 64 * g, hk, (int)(t.k0 + j0));
                        tma_load_3d(sm + C::B0 + g * kRegion, &tv, bar, 64 * g, hk, (int)(t.k0 + j0));
                    }
                },
                [&](int i, unsigned char *dst, uint64_t *bar) {
                    const int head = hk * a.G + (i % chunks) * gb, tok = (int)(t.q0 + token0(i));
                    for (int g = 0; g < C::NG; ++g) {
                        tma_load_3d(dst + g * kSubRegion, &tq, bar, 64 * g, head, tok);
                        tma_load_3d(dst + C::ST + g * kSubRegion, &tdo, bar, 64 * g, head, tok);
                    }
                });
    } else if (warp == 9) {
        if (n > 0) {
            const uint32_t idS = idesc_bf16_f32(128, kSub, false, false);
            const int nk = (a.D + 15) / 16;
            const uint32_t idA = idesc_bf16_f32(128, 16 * nk, false, true);
            const uint32_t sbase = smem_u32(sm);
            auto wait = [&](uint64_t *bar, uint32_t ph) { return mbar_wait(bar, ph, abort_flag); };
            auto scores = [&](int i) -> bool {
                const int st = i % kStages, buf = i & 1;
                if (!wait(&b.full[st], (i / kStages) & 1)) return false;
                const int rows = rows_of(i);
                if (rows < R * gb) zero_rows<C::NG>(sm + C::X0 + 2 * st * C::ST, rows, lane);
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t x = sbase + C::X0 + 2 * st * C::ST;
                    for (int kk = 0; kk < nk; ++kk)
                        mma_bf16(tmem + C::COL_S + buf * kSub, kdesc(sbase + C::A0 + (kk >> 2) * kRegion + (kk & 3) * 32),
                                 kdesc(x + (kk >> 2) * kSubRegion + (kk & 3) * 32), idS, kk > 0 ? 1u : 0u);
                    mma_commit(&b.s[buf]);
                    for (int kk = 0; kk < nk; ++kk)
                        mma_bf16(tmem + C::COL_DP + buf * kSub, kdesc(sbase + C::B0 + (kk >> 2) * kRegion + (kk & 3) * 32),
                                 kdesc(x + C::ST + (kk >> 2) * kSubRegion + (kk & 3) * 32), idS, kk > 0 ? 1u : 0u);
                    mma_commit(&b.dp[buf]);
                }
                __syncwarp();
                return true;
            };
            auto accumulate = [&](uint32_t acc, uint32_t w, uint32_t x, bool add) {
#pragma unroll
                for (int jj = 0; jj < kSub / 16; ++jj)
                    mma_bf16_tmem_a(tmem + acc, tmem + w + jj * 8, sdesc(x + jj * 2048, kSubRegion, 1024, 2), idA,
                                    (add || jj > 0) ? 1u : 0u);
            };
            bool ok = wait(b.own, 0);
            for (int i = 0; ok && i < min(n, 2); ++i) ok = scores(i);
            for (int i = 0; ok && i < n; ++i) {
                const int st = i % kStages, buf = i & 1;
                const uint32_t x = sbase + C::X0 + 2 * st * C::ST, ph = (i >> 1) & 1;
                if (!(ok = wait(&b.p[buf], ph))) break;
                tc_fence_after();
                if (lane == 0) accumulate(C::COL_ACC, C::COL_S + buf * kSub, x + C::ST, i > 0);
                __syncwarp();
                if (!(ok = wait(&b.ds[buf], ph))) break;
                tc_fence_after();
                if (lane == 0) {
                    accumulate(C::COL_ACC + 128, C::COL_DP + buf * kSub, x, i > 0);
                    mma_commit(&b.empty[st]);
                    if (i == n - 1) mma_commit(b.done);
                }
                __syncwarp();
                if (i + 2 < n) ok = scores(i + 2);
            }
            if (lane == 0) {
                mma_commit(b.drain);
                mbar_drain(b.drain, 0);
            }
        }
    } else {
        const int w = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t cS = tmem + C::COL_S + w * kSub + lanes, cDP = tmem + C::COL_DP + w * kSub + lanes;
        float *my = srow + w * 128;  // [64] lse in log2 units, [64] delta
        const int rr = r & 63, rt = rr / gb, rg = rr - rt * gb;
        // lse (r < 64) or delta (r >= 64) of row rr of sub-tile i
        auto row_value = [&](int i) -> float {
            if (i >= n || rr >= rows_of(i)) return 0.f;
            const int64_t row = (t.q0 + token0(i) + rt) * a.H + hk * a.G + (i % chunks) * gb + rg;
            return r < 64 ? a.lse_in[row] * kLog2e : a.delta[row];
        };
        const float sc = a.scale * kLog2e;
        float next = row_value(w);
        bool ok = true;
        for (int i = w; i < n; i += 2) {
            const uint32_t ph = (i >> 1) & 1;
            named_sync(1 + w, 128);  // the previous sub-tile's rows have been read
            my[r] = next;
            named_sync(1 + w, 128);
            next = row_value(i + 2);
            if (!(ok = mbar_wait(&b.s[w], ph, abort_flag))) break;
            tc_fence_after();
            float p[kSub];
            ld64(cS, p);
            // columns (rows) [lo, hi) see key r
            const int hi = rows_of(i);
            const int64_t lo64 = a.causal ? (j0 + r - off - token0(i)) * gb : 0;
            const int lo = chunks > 1 ? (lo64 > 0 ? kSub : 0) : (int)max((int64_t)0, min64(lo64, kSub));
#pragma unroll
            for (int c = 0; c < kSub; c += 4) {
                const float4 l4 = *reinterpret_cast<const float4 *>(my + c);
                p[c] = fast_exp2(fmaf(p[c], sc, -l4.x));
                p[c + 1] = fast_exp2(fmaf(p[c + 1], sc, -l4.y));
                p[c + 2] = fast_exp2(fmaf(p[c + 2], sc, -l4.z));
                p[c + 3] = fast_exp2(fmaf(p[c + 3], sc, -l4.w));
            }
            const bool masked = __any_sync(0xffffffffu, lo > 0 || hi < kSub);
            if (masked) {
#pragma unroll
                for (int c = 0; c < kSub; ++c)
                    if (c < lo || c >= hi) p[c] = 0.f;
            }
            st64_bf16(cS, p);
            tc_fence_before();
            mbar_arrive(&b.p[w]);
            if (!(ok = mbar_wait(&b.dp[w], ph, abort_flag))) break;
            tc_fence_after();
            float dp[kSub];
            ld64(cDP, dp);
#pragma unroll
            for (int c = 0; c < kSub; c += 4) {
                const float4 d4 = *reinterpret_cast<const float4 *>(my + 64 + c);
                dp[c] = p[c] * (dp[c] - d4.x);
                dp[c + 1] = p[c + 1] * (dp[c + 1] - d4.y);
                dp[c + 2] = p[c + 2] * (dp[c + 2] - d4.z);
                dp[c + 3] = p[c + 3] * (dp[c + 3] - d4.w);
            }
            if (masked) {
#pragma unroll
                for (int c = 0; c < kSub; ++c)
                    if (c < lo || c >= hi) dp[c] = 0.f;
            }
            st64_bf16(cDP, dp);
            tc_fence_before();
            mbar_arrive(&b.ds[w]);
        }
        if (ok && n > 0) ok = mbar_wait(b.done, 0, abort_flag);
        if (ok) {
            tc_fence_after();
            const bool mine = j0 + r < t.tk;
            const int64_t o = ((t.k0 + j0 + r) * a.Hk + hk) * a.D;
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(w == 0 ? a.dv : a.dk) + (mine ? o : 0);
            store_acc(tmem + C::COL_ACC + w * 128 + lanes, n > 0, mine, dst, a.D, w == 0 ? 1.f : a.scale);
        } else if (a.status) {
            atomicExch(a.status, kDevTimeout);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------------------------ dq
template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
attn_dq_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdo,
                  const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, AttnArgs a, int R) {
    using C = BwdCfg<DP>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = align1024(smem_raw);
    AttnTile t;
    const int hk = blockIdx.x % a.Hk;
    int64_t slot = gridDim.x / a.Hk - 1 - blockIdx.x / a.Hk;  // the last rows see the most keys
    if (!a.sq.cu) {
        const int64_t per = gridDim.x / a.Hk / a.N;
        slot = (slot % a.N) * per + slot / a.N;
    }
    if (!attn_locate(a, true, slot, 1, R, t)) return;
    const int64_t last = min64(t.row0 + R, t.tq) - 1;
    const int64_t seen = a.causal ? min64(t.tk, last + 1 + t.tk - t.tq) : t.tk;
    const int n = seen > 0 ? (int)((seen + kSub - 1) / kSub) : 0;

    const BwdBars b(reinterpret_cast<uint64_t *>(sm + C::BARS));
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + C::MISC + 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        b.init();
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
        if (lane == 0 && n > 0)
            produce<DP>(
                sm, b, n, 2u * C::NG * R * a.G * 128, 2 * C::ST, abort_flag,
                [&](uint64_t *bar) {
                    for (int g = 0; g < C::NG; ++g) {
                        tma_load_3d(sm + C::A0 + g * kRegion, &tq, bar, 64 * g, hk * a.G, (int)(t.q0 + t.row0));
                        tma_load_3d(sm + C::B0 + g * kRegion, &tdo, bar, 64 * g, hk * a.G, (int)(t.q0 + t.row0));
                    }
                },
                [&](int i, unsigned char *dst, uint64_t *bar) {
                    const int tok = (int)(t.k0 + (int64_t)i * kSub);
                    for (int g = 0; g < C::NG; ++g) {
                        tma_load_3d(dst + g * kSubRegion, &tk, bar, 64 * g, hk, tok);
                        tma_load_3d(dst + C::ST + g * kSubRegion, &tv, bar, 64 * g, hk, tok);
                    }
                });
    } else if (warp == 9) {
        if (n > 0) {
            const uint32_t idS = idesc_bf16_f32(128, kSub, false, false);
            const int nk = (a.D + 15) / 16;
            const uint32_t idA = idesc_bf16_f32(128, 16 * nk, false, true);
            const uint32_t sbase = smem_u32(sm);
            auto wait = [&](uint64_t *bar, uint32_t ph) { return mbar_wait(bar, ph, abort_flag); };
            auto scores = [&](int i) -> bool {
                const int st = i % kStages, buf = i & 1;
                if (!wait(&b.full[st], (i / kStages) & 1)) return false;
                const int64_t left = t.tk - (int64_t)i * kSub;  // keys behind the sequence are operands too
                if (left < kSub) zero_rows<C::NG>(sm + C::X0 + 2 * st * C::ST, (int)left, lane);
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t x = sbase + C::X0 + 2 * st * C::ST;
                    for (int kk = 0; kk < nk; ++kk)
                        mma_bf16(tmem + C::COL_S + buf * kSub, kdesc(sbase + C::A0 + (kk >> 2) * kRegion + (kk & 3) * 32),
                                 kdesc(x + (kk >> 2) * kSubRegion + (kk & 3) * 32), idS, kk > 0 ? 1u : 0u);
                    mma_commit(&b.s[buf]);
                    for (int kk = 0; kk < nk; ++kk)
                        mma_bf16(tmem + C::COL_DP + buf * kSub, kdesc(sbase + C::B0 + (kk >> 2) * kRegion + (kk & 3) * 32),
                                 kdesc(x + C::ST + (kk >> 2) * kSubRegion + (kk & 3) * 32), idS, kk > 0 ? 1u : 0u);
                    mma_commit(&b.dp[buf]);
                }
                __syncwarp();
                return true;
            };
            bool ok = wait(b.own, 0);
            for (int i = 0; ok && i < min(n, 2); ++i) ok = scores(i);
            for (int i = 0; ok && i < n; ++i) {
                const int st = i % kStages, buf = i & 1;
                if (!(ok = wait(&b.ds[buf], (i >> 1) & 1))) break;
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t x = sbase + C::X0 + 2 * st * C::ST;
#pragma unroll
                    for (int jj = 0; jj < kSub / 16; ++jj)
                        mma_bf16_tmem_a(tmem + C::COL_ACC, tmem + C::COL_DP + buf * kSub + jj * 8,
                                        sdesc(x + jj * 2048, kSubRegion, 1024, 2), idA, (i > 0 || jj > 0) ? 1u : 0u);
                    mma_commit(&b.empty[st]);
                    if (i == n - 1) mma_commit(b.done);
                }
                __syncwarp();
                if (i + 2 < n) ok = scores(i + 2);
            }
            if (lane == 0) {
                mma_commit(b.drain);
                mbar_drain(b.drain, 0);
            }
        }
    } else {
        const int w = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t cS = tmem + C::COL_S + w * kSub + lanes, cDP = tmem + C::COL_DP + w * kSub + lanes;
        const int tr = r / a.G;
        const int64_t tok = t.row0 + tr;
        const bool mine = tr < R && tok < t.tq;
        const int64_t lim64 = mine ? (a.causal ? min64(t.tk, tok + 1 + t.tk - t.tq) : t.tk) : 0;
        const int lim = (int)max((int64_t)0, lim64);
        const int64_t row = mine ? (t.q0 + tok) * a.H + hk * a.G + (r - tr * a.G) : 0;
        const float lse = mine ? a.lse_in[row] * kLog2e : 0.f;
        float delta = mine ? a.delta[row] : 0.f;
        const float sc = a.scale * kLog2e;
        bool ok = true;
        for (int i = w; i < n; i += 2) {
            const uint32_t ph = (i >> 1) & 1;
            if (!(ok = mbar_wait(&b.s[w], ph, abort_flag))) break;
            tc_fence_after();
            float p[kSub];
            ld64(cS, p);
#pragma unroll
            for (int c = 0; c < kSub; ++c) p[c] = fast_exp2(fmaf(p[c], sc, -lse));
            if (!(ok = mbar_wait(&b.dp[w], ph, abort_flag))) break;
            tc_fence_after();
            float dp[kSub];
            ld64(cDP, dp);
            const int left = lim - i * kSub;
            if (i == 0 && __any_sync(0xffffffffu, lim > 0 && lim <= kSub)) {
                // All keys of such a row are here: delta = sum_j p dp in fp32.  The one from o
                // carries o's rounding, which for rows with few keys is the largest error of
                // dq and dk (measured: dq off by 2.5e-3 with it, 2.4e-3 without).
                float x = 0.f;
#pragma unroll
                for (int c = 0; c < kSub; ++c)
                    if (c < lim) x = fmaf(p[c], dp[c], x);
                if (lim > 0 && lim <= kSub) {
                    delta = x;
                    if (mine) a.delta[row] = x;
                }
            }
#pragma unroll
            for (int c = 0; c < kSub; ++c) dp[c] = p[c] * (dp[c] - delta);
            if (__any_sync(0xffffffffu, left < kSub)) {
#pragma unroll
                for (int c = 0; c < kSub; ++c)
                    if (c >= left) dp[c] = 0.f;
            }
            st64_bf16(cDP, dp);
            tc_fence_before();
            mbar_arrive(&b.ds[w]);
        }
        if (ok && n > 0) ok = mbar_wait(b.done, 0, abort_flag);
        if (ok) {
            tc_fence_after();
            if (w == 0)
                store_acc(tmem + C::COL_ACC + lanes, n > 0, mine, static_cast<__nv_bfloat16 *>(a.dq) + row * a.D, a.D,
                          a.scale);
        } else if (a.status) {
            atomicExch(a.status, kDevTimeout);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

struct Maps {
    CUtensorMap q, dout, k, v;
};

// q, dout in boxes of qh heads x qr tokens, k and v in boxes of kr tokens
cudaError_t make_maps(const AttnArgs &a, int qh, int qr, int kr, Maps &m) {
    const int64_t qt = a.sq.cu ? a.sq.T : a.N * a.sq.T, kt = a.sk.cu ? a.sk.T : a.N * a.sk.T;
    cudaError_t e = cudaSuccess;
    if (qt > 0) {
        if ((e = tc_make_map_rows(&m.q, a.q, qt, a.H, a.D, qh, qr)) != cudaSuccess) return e;
        if ((e = tc_make_map_rows(&m.dout, a.dout, qt, a.H, a.D, qh, qr)) != cudaSuccess) return e;
    }
    if (kt > 0) {
        if ((e = tc_make_map_rows(&m.k, a.k, kt, a.Hk, a.D, 1, kr)) != cudaSuccess) return e;
        if ((e = tc_make_map_rows(&m.v, a.v, kt, a.Hk, a.D, 1, kr)) != cudaSuccess) return e;
    }
    if (qt == 0) m.q = m.dout = m.k;  // a side without tokens is never copied
    if (kt == 0) m.k = m.v = m.q;
    return e;
}

template <int DP>
cudaError_t launch_dkdv(const AttnArgs &a, const Maps &m, int gb, int R, cudaStream_t st) {
    auto kern = attn_dkdv_tc_kernel<DP>;
    constexpr size_t smem = BwdCfg<DP>::SMEM;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, smem, done);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(attn_slots(a.sk, a.N, 1, kTile) * a.Hk), kBwdThreads, smem, st>>>(m.q, m.dout, m.k, m.v, a, gb, R);
    return cudaGetLastError();
}

template <int DP>
cudaError_t launch_dq(const AttnArgs &a, const Maps &m, int R, cudaStream_t st) {
    auto kern = attn_dq_tc_kernel<DP>;
    constexpr size_t smem = BwdCfg<DP>::SMEM;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, smem, done);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(attn_slots(a.sq, a.N, 1, R) * a.Hk), kBwdThreads, smem, st>>>(m.q, m.dout, m.k, m.v, a, R);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_bwd_dkdv_tc(const AttnArgs &a, cudaStream_t st) {
    const int gb = std::min(a.G, kSub), R = kSub / gb;
    Maps m;
    const cudaError_t e = make_maps(a, gb, R, kTile, m);
    if (e != cudaSuccess) return e;
    return a.D <= 64 ? launch_dkdv<64>(a, m, gb, R, st) : launch_dkdv<128>(a, m, gb, R, st);
}

cudaError_t launch_attn_bwd_dq_tc(const AttnArgs &a, cudaStream_t st) {
    const int R = kTile / a.G;
    Maps m;
    const cudaError_t e = make_maps(a, a.G, R, kSub, m);
    if (e != cudaSuccess) return e;
    return a.D <= 64 ? launch_dq<64>(a, m, R, st) : launch_dq<128>(a, m, R, st);
}

}  // namespace sgla
