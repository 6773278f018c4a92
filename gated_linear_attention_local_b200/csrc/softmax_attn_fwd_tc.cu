// Softmax attention forward on the tensor cores (tcgen05 / TMEM / TMA), bf16 operands.
//
// A work item is two tiles of 128 packed rows (row = token * G + g of one key head, R = 128 / G
// tokens a tile) against the keys its rows see, in tiles of 128.  For row tile w, key tile j
//   S_w = Q_w K_j^T            (128 x 128, fp32 in tensor memory)
//   p   = 2^(sc S - m)         one thread a row: maximum and sum need no shuffles
//   O_w += P_w V_j             P_w in bf16 in tensor memory, over S_w's columns
// The two row tiles alternate: while one's 128 threads form p, the tensor cores run the other's
// products.  The tensor pipe executes in issue order, so S_w(j+1) may follow P_w(j) V_j at
// once although it overwrites P_w(j).  P_w V_j starts when the first 96 of its 128 keys are
// written.
//
// The grid has a block for every item, heaviest first, and one CTA fits an SM; a scheduler warp
// takes over blocks that have not started (clusterlaunchcontrol), finds their sequence and hands
// out the next item's description while the current one is in work: the copies and first
// products of an item run under the epilogue of the one before, and unequal items even out
// (against a fixed share of the items for each CTA: 8 packed prompts 269 -> 206 us when it came).
//
// Measured (events around the launch, cold L2, less the 5 us that an empty pair of events reads),
// heads of 128, causal: 8192 tokens of 32 heads on 8, 457 us = 1203 TFLOP/s alone (85 % of the
// library's sustained rate; back to back, under the power limit, 535 us = 1028); 8 packed prompts of
// 128 to 4096 tokens, 16 heads on 4, 187 us; 4 x 2048 tokens of 16 heads, 88 us.  What bounds it: the
// chain of a row tile, scores -> probabilities -> P V -> next scores, of which two run side by side.
// Without exponentials, sums and maxima (for timing only, at 436 and 84 us) the first took 399 us
// and the last 79, so the softmax costs a tenth; a tile pair takes some 3000 cycles for the 2048 of
// its products, an item's end 5500.
//
// The maximum m of a row is only moved (and O, l rescaled, in tensor memory, by the row's own
// thread) when it has grown by more than 2^8: until then p <= 2^8, which fp32 sums and the
// bf16 range (the rounding is relative) carry without loss.
//
// Exponentials: 128 x 128 of them take the special-function unit as long as the two products
// take the tensor cores (1024 cycles), so a quarter goes to the FMA pipe instead (softmax_attn_tc.cuh;
// 8192 tokens, when it came: 450 us with none, 447 with a quarter, 453 with three eighths).  A NaN
// among a row's visible scores makes its maximum and so all its p NaN; a score of -inf weighs 0.
//
// p is rounded to bf16 for the product with V (relative 2^-8, averaged over the keys); its sum
// l, m, S and O are fp32.
//
// Tensor memory (512 columns): S0, S1 [0, 256), O0, O1 [256, 512).
// Shared memory (DP = 128): Q 64 KB, rings of two K and two V tiles 128 KB.
// Warps: 0-3 rows of tile 0, 4-7 rows of tile 1, 8 TMA, 9 MMA, 10 scheduler (11 fills up).
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "softmax_attn.h"
#include "softmax_attn_map.h"
#include "softmax_attn_tc.cuh"

namespace sgla {

using namespace tc;

namespace {

constexpr int kFwdThreads = 384;
constexpr int kTile = 128;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.f;  // log2 units the maximum may lag behind
// sc S - m sc in one FMA carries the rounding of m sc, 2^-24 of it, in every p of the row alike.  That
// cancels in o; where it could take p out of range (keys given the lowest value of their type) the
// difference S - m is formed first.
constexpr float kFar = 16777216.f;

// What the roles need to know of a work item; every count fits 32 bits.
struct Item {
    int n;         // key tiles of the item (the larger of nt); < 0: no more items
    int nt[2];     // key tiles of each row tile
    int q_tok;     // first token of row tile 0
    int q_left;    // tokens of the sequence from there on
    int k_tok;     // first key of this split
    int keys;      // keys of this split
    int k_left;    // keys of the sequence from k_tok on
    int shift;     // causal: token x of the item sees keys < x + 1 + shift of this split
    int hk, z;     // key head, split
};

template <int DP>
struct FwdCfg {
    static constexpr int NG = DP / 64;               // 64-column groups of a tile
    static constexpr uint32_t T = NG * kRegion;      // one tile, bytes
    static constexpr uint32_t Q0 = 0, K0 = 2 * T, V0 = 4 * T;
    static constexpr uint32_t BARS = 6 * T, MISC = BARS + 32 * 8, ITEM = MISC + 32;
    // at least half of an SM's shared memory: the CTA takes all of its tensor memory
    static constexpr size_t NEED = ITEM + sizeof(Item) + 1024;
    static constexpr size_t SMEM = NEED > 120 * 1024 ? NEED : 120 * 1024;
    static constexpr uint32_t COL_O = 256;
    static_assert(SMEM <= 232448, "shared memory budget");
};

// The same descriptor, but to the compiler another one for each key tile (0 <= count < 2^30): those
// of both Q tiles, kept across an item's key tiles, would take 32 of the product warp's 72 registers
// (8192 tokens of 32 heads: 454 us for 461).
__device__ __forceinline__ uint64_t fresh(uint64_t desc, int count) { return desc + (uint32_t)(count >> 30); }

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// p of the scores s[0..32) of a row, as bf16 to 16 columns at taddr; their sum onto sum.
template <bool MASKED>
__device__ __forceinline__ void probabilities(const float (&s)[32], float sc, float ms, uint32_t taddr, float2 (&sum)[2]) {
    uint32_t p[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float2 x = __ffma2_rn(make_float2(s[2 * e], s[2 * e + 1]), make_float2(sc, sc), make_float2(-ms, -ms));
        if (!MASKED && (e & 3) == 3) {
            x = exp2_fma(x);
        } else {
            x.x = fast_exp2(x.x);
            x.y = fast_exp2(x.y);
        }
        sum[e & 1] = __fadd2_rn(sum[e & 1], x);
        p[e] = pack_bf16(x.x, x.y);
    }
    tmem_st16(taddr, p);
}

template <int DP, bool PACKED>
__global__ void __launch_bounds__(kFwdThreads, 1)
attn_fwd_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv, AttnArgs a, int R, int slots,
                   bool wide) {
    using C = FwdCfg<DP>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = align1024(smem_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::BARS);
    uint64_t *full_q = bars, *empty_q = bars + 2;                      // [2] per row tile
    uint64_t *full_k = bars + 4, *full_v = bars + 6;                   // [2] stages
    uint64_t *empty_k = bars + 8, *empty_v = bars + 10;                // [2]
    uint64_t *b_s = bars + 12, *b_o = bars + 14;                       // [2] per row tile: S, O complete
    uint64_t *b_pa = bars + 16, *b_pb = bars + 18;                     // [2] first 96, last 32 keys of P written
    uint64_t *b_drain = bars + 23;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + C::MISC + 8);
    const Feed<Item> feed{bars + 20, bars + 21, bars + 22, bars + 24, sm + C::MISC + 16, reinterpret_cast<Item *>(sm + C::ITEM),
                          abort_flag, abort_flag + 1};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int b = 0; b < 16; ++b) mbar_init(&bars[b], 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&b_pa[b], 128);
            mbar_init(&b_pb[b], 128);
        }
        feed.init();
        mbar_init(b_drain, 1);
        mbar_fence_init();
    }
    if (threadIdx.x == 256) {
        prefetch_tmap(&tq);
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
    }
    if (warp == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // (one instruction a warpgroup, ahead of the roles: setmaxnreg is .aligned)
    if (warp >= 8) {
        setmaxnreg_dec<kOtherRegs>();
        if (warp == 10) {
            // ---------------------------------------------------------------- scheduler
            const int per_z = slots * a.Hk;
            AttnOrder order;
            if constexpr (PACKED) order.init(a, 2 * R);
            feed.run([&](int u, Item &it) -> bool {
                it.z = u / per_z;
                const int rest = u - it.z * per_z;
                it.hk = rest % a.Hk;
                AttnTile t;
                if (PACKED && order.on) {
                    if (!order.locate(a, rest / a.Hk, 2 * R, t)) return false;
                } else {
                    // heaviest first: a causal sequence's last rows see the most keys
                    int64_t slot = slots - 1 - rest / a.Hk;
                    if (!PACKED) slot = (slot % a.N) * (slots / a.N) + slot / a.N;
                    if (!attn_locate(a, true, slot, 1, 2 * R, t)) return false;
                }
                const int64_t kb = it.z * a.split, ke = min64(t.tk, kb + a.split);
                it.keys = (int)(ke > kb ? ke - kb : 0);
                it.q_tok = (int)(t.q0 + t.row0);
                it.q_left = (int)(t.tq - t.row0);
                it.k_tok = (int)(t.k0 + kb);
                it.k_left = (int)(t.tk - kb);
                it.shift = (int)max(min64(t.row0 + t.tk - t.tq - kb, (int64_t)INT_MAX - 512), -(int64_t)INT_MAX / 2);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int last = min((w + 1) * R, it.q_left) - 1;  // last token of the row tile
                    const int lim = w * R >= it.q_left ? 0 : (a.causal ? min(it.keys, last + 1 + it.shift) : it.keys);
                    it.nt[w] = lim > 0 ? (lim + kTile - 1) / kTile : 0;
                }
                it.n = max(it.nt[0], it.nt[1]);
                return true;
            });
        } else if (warp == 8) {
            // ---------------------------------------------------------------- TMA producer
            const uint32_t qbytes = (uint32_t)(R * a.G) * 128u * C::NG;
            Item it;
            int ni = 0, kv = 0, nv = 0, nq[2] = {0, 0};
            bool ok = true;
            // One lane waits and copies, the others meet it at the shuffle behind an item's copies: nothing
            // between is warp-wide.  (All lanes in the loop, an elected one copying: 470 -> 478 us at 8192
            // tokens of 32 heads.)  What a product warp that gave up released is not filled again.
            auto wait = [&](uint64_t *bar, uint32_t ph) { return mbar_wait_idle(bar, ph, abort_flag) && !*abort_flag; };
            while (ok && feed.take(ni, it)) {
                if (lane == 0) {
                    auto load_q = [&](int w) {
                        if (it.nt[w] == 0) return true;
                        if (nq[w] > 0 && !wait(&empty_q[w], (nq[w] - 1) & 1)) return false;
                        mbar_arrive_expect_tx(&full_q[w], qbytes);
                        for (int g = 0; g < C::NG; ++g)
                            tma_load_3d(sm + C::Q0 + w * C::T + g * kRegion, &tq, &full_q[w], 64 * g, it.hk * a.G,
                                        it.q_tok + w * R);
                        ++nq[w];
                        return true;
                    };
                    ok = load_q(0);
                    for (int j = 0; ok && j < it.n; ++j) {
                        const int st = kv & 1;
                        const uint32_t ph = ((kv >> 1) - 1) & 1;
                        if (kv >= 2 && !(ok = wait(&empty_k[st], ph))) break;
                        mbar_arrive_expect_tx(&full_k[st], C::T);
                        for (int g = 0; g < C::NG; ++g)
                            tma_load_3d(sm + C::K0 + st * C::T + g * kRegion, &tk, &full_k[st], 64 * g, it.hk,
                                        it.k_tok + j * kTile);
                        ++kv;
                        if (j == 0 && !(ok = load_q(1))) break;
                        if (nv >= 2 && !(ok = wait(&empty_v[st], ph))) break;
                        mbar_arrive_expect_tx(&full_v[st], C::T);
                        for (int g = 0; g < C::NG; ++g)
                            tma_load_3d(sm + C::V0 + st * C::T + g * kRegion, &tv, &full_v[st], 64 * g, it.hk,
                                        it.k_tok + j * kTile);
                        *feed.copies = ++nv;
                    }
                }
                if (lane == 0) mbar_arrive(feed.want);
                ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
            }
            if (lane == 0 && *abort_flag) {  // let the copies in flight land before the CTA exits
                for (int w = 0; w < 2; ++w)
                    if (nq[w] > 0) mbar_drain(&full_q[w], (nq[w] - 1) & 1);
                for (int i = max(0, kv - 2); i < kv; ++i) mbar_drain(&full_k[i & 1], (i >> 1) & 1);
                for (int i = max(0, nv - 2); i < nv; ++i) mbar_drain(&full_v[i & 1], (i >> 1) & 1);
            }
        } else if (warp == 9) {
            // ---------------------------------------------------------------- MMA issuer
            const uint32_t idS = idesc_bf16_f32(128, 128, false, false);
            const int nk = (a.D + 15) / 16;  // 16-column steps of a head (zeros past D)
            const uint32_t idO = idesc_bf16_f32(128, 16 * nk, false, true);
            const uint32_t sbase = smem_u32(sm);
            const uint64_t qd = kdesc(sbase + C::Q0), kd = kdesc(sbase + C::K0);
            const uint64_t vd = sdesc(sbase + C::V0, kRegion, 1024, 2);
            // A wait that gave up (abort is set then) sends no lane another way: the products go on, over
            // whatever is there, to the item's end, where the lanes vote.  (A vote on every wait, all_wait:
            // 446 -> 464 us at 8192 tokens of 32 heads.)
            auto wait = [&](uint64_t *bar, uint32_t ph) { mbar_wait(bar, ph, abort_flag); };
            auto sound = [&] { return __all_sync(0xffffffffu, !*abort_flag); };
            Item it;
            int ni = 0, kv = 0, nq[2] = {0, 0}, np[2] = {0, 0};
            while (sound() && feed.take(ni, it)) {
                // the same in every lane; the reduction leaves them in uniform registers, from which
                // the products' descriptors are formed without a move per operand
                const int nt[2] = {__reduce_max_sync(0xffffffffu, it.nt[0]), __reduce_max_sync(0xffffffffu, it.nt[1])};
                const int n = max(nt[0], nt[1]);
                for (int j = -1; j < n; ++j) {
                    if ((j & 1023) == 1023 && j > 0 && !sound()) break;  // (the rest of a long item)
                    const int c0 = kv + j, c1 = kv + j + 1;  // ring positions of key tiles j and j + 1
                    const uint64_t v0 = desc_at(vd, (c0 & 1) * C::T), k1 = desc_at(kd, (c1 & 1) * C::T);
                    if (j >= 0) {
                        wait(&full_v[c0 & 1], (c0 >> 1) & 1);
                        const int valid = it.k_left - j * kTile;
                        if (valid < kTile) {
                            // rows behind the sequence's keys hold its neighbour's data: 0 * NaN must not arise
                            for (int i = lane; i < C::NG * 8 * kTile; i += 32) {
                                const int r = (i >> 3) & (kTile - 1);
                                if (r >= valid)
                                    *reinterpret_cast<uint4 *>(sm + C::V0 + (c0 & 1) * C::T + (i >> 10) * kRegion + r * 128 +
                                                               (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                    }
                    if (j + 1 < n) wait(&full_k[c1 & 1], (c1 >> 1) & 1);
                    const bool second = j < 0 ? nt[1] > 0 : j < nt[1];  // row tile 1 has products here
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const bool pv = j >= 0 && j < nt[w], more = j + 1 < nt[w];
                        if (pv) {
                            wait(&b_pa[w], np[w] & 1);
                            tc_fence_after();
                            if (elect_one()) {
#pragma unroll
                                for (int jj = 0; jj < 6; ++jj)
                                    mma_bf16_tmem_a(tmem + C::COL_O + w * 128, tmem + w * 128 + jj * 8,
                                                    desc_at(v0, jj * 2048), idO, (j > 0 || jj > 0) ? 1u : 0u);
                            }
                            __syncwarp();
                            wait(&b_pb[w], np[w] & 1);
                            ++np[w];
                        }
                        if (j < 0 && more) {
                            wait(&full_q[w], nq[w] & 1);
                            ++nq[w];
                        }
                        tc_fence_after();
                        // the rest of P V and the next scores without a pause: the pipe holds few products
                        if ((pv || more) && elect_one()) {
                            if (pv) {
#pragma unroll
                                for (int jj = 6; jj < 8; ++jj)
                                    mma_bf16_tmem_a(tmem + C::COL_O + w * 128, tmem + w * 128 + jj * 8,
                                                    desc_at(v0, jj * 2048), idO, 1u);
                                if (!more) mma_commit(&b_o[w]);
                            }
                            if (more) {
                                const uint64_t q1 = fresh(desc_at(qd, w * C::T), c1);
#pragma unroll
                                for (int kk = 0; kk < DP / 16; ++kk)
                                    if (kk < nk)
                                        mma_bf16(tmem + w * 128, desc_at(q1, (kk >> 2) * kRegion + (kk & 3) * 32),
                                                 desc_at(k1, (kk >> 2) * kRegion + (kk & 3) * 32), idS, kk > 0 ? 1u : 0u);
                                mma_commit(&b_s[w]);
                                if (j + 1 == nt[w] - 1) mma_commit(&empty_q[w]);
                            }
                            if (w == 1 || !second) {  // the last products of this pair of tiles
                                if (j >= 0) mma_commit(&empty_v[c0 & 1]);
                                if (j + 1 < n) mma_commit(&empty_k[c1 & 1]);
                            }
                        }
                        __syncwarp();
                    }
                }
                kv += n;
            }
            if (elect_one()) {
                mma_commit(b_drain);
                mbar_drain(b_drain, 0);
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax: one row a thread
        setmaxnreg_inc<kRowRegs>();
        const int w = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
        const uint32_t cS = tmem + w * 128 + lanes, cO = tmem + C::COL_O + w * 128 + lanes;
        const int tr = r / a.G, x = w * R + tr;  // the row's token of the item
        const float sc = a.scale * kLog2e;
        Item it;
        int ni = 0, ns = 0, no = 0;
        bool ok = true;
        while (ok && feed.take(ni, it)) {
            const bool mine = tr < R && x < it.q_left;
            const int n = w == 0 ? it.nt[0] : it.nt[1];
            const int lim = mine ? (a.causal ? min(it.keys, x + 1 + it.shift) : it.keys) : 0;  // keys the row sees
            float m = -INFINITY, l = 0.f;  // m in units of S
            bool far = false;
            for (int j = 0; j < n; ++j, ++ns) {
                if (!(ok = all_wait(&b_s[w], ns & 1, abort_flag))) break;
                tc_fence_after();
                float s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(cS + 32 * c, s[c]);
                tmem_wait_ld();
                const int left = lim - j * kTile;
                const bool masked = __any_sync(0xffffffffu, left < kTile);
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (32 * c + e >= left) s[c][e] = -INFINITY;
                }
                float t4[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) t4[c] = max3_nan(s[c][0], s[c][1], s[c][2]);
#pragma unroll
                for (int e = 3; e + 1 < 32; e += 2)
#pragma unroll
                    for (int c = 0; c < 4; ++c) t4[c] = max3_nan(t4[c], s[c][e], s[c][e + 1]);
                const float top = max3_nan(max3_nan(t4[0], t4[1], s[0][31]), max3_nan(t4[2], t4[3], s[1][31]),
                                           max3_nan(s[2][31], s[3][31], s[3][31]));
                // move the maximum when it has grown by more than kGrow, there was none, or it is NaN
                float f = 1.f;
                if (!((top - m) * sc <= kGrow) && top != -INFINITY) {
                    f = fast_exp2((m - top) * sc);  // 0 from m = -inf
                    m = top;
                }
                __syncwarp();
                if (__any_sync(0xffffffffu, f != 1.f)) {
                    far = __any_sync(0xffffffffu, m != -INFINITY && fabsf(m * sc) > kFar);
                    l *= f;
                    if (j > 0) {
                        for (int c = 0; c < a.D; c += 16) {
                            float o[16];
                            tmem_ld16f(cO + c, o);
                            tmem_wait_ld();
                            uint32_t u[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * f);
                            tmem_st16(cO + c, u);
                        }
                        tmem_wait_st();
                    }
                }
                float ms = m == -INFINITY ? 0.f : m * sc;
                if (far) {
                    const float m0 = m == -INFINITY ? 0.f : m;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[c][e] -= m0;
                    ms = 0.f;
                }
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                auto part = [&](int c) {
                    if (masked) probabilities<true>(s[c], sc, ms, cS + 16 * c, sum);
                    else probabilities<false>(s[c], sc, ms, cS + 16 * c, sum);
                };
                part(0);
                part(1);
                part(2);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&b_pa[w]);
                part(3);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&b_pb[w]);
                const float2 q = __fadd2_rn(sum[0], sum[1]);
                l += q.x + q.y;
            }
            if (!ok) break;
            if (n > 0) {
                if (!(ok = all_wait(&b_o[w], no & 1, abort_flag))) break;
                ++no;
            }
            tc_fence_after();
            const int64_t row = (int64_t)(it.q_tok + x) * a.H + it.hk * a.G + (r - tr * a.G);
            const int64_t prow = (int64_t)it.z * a.part_rows + row;
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN scores stay NaN
            const float lse = l > 0.f ? m * a.scale + log2f(l) * kLn2 : (l == 0.f ? -INFINITY : l);
            if (mine) {
                if (a.part_lse) a.part_lse[prow] = lse;
                else if (a.lse) a.lse[row] = lse;
            }
            for (int c = 0; c < a.D; c += 32) {
                float o[32];
                if (n > 0) {
                    tmem_ld32(cO + c, o);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = l == 0.f ? 0.f : o[e] * inv;
                if (mine && a.part_o) {
                    float4 *dst = reinterpret_cast<float4 *>(a.part_o + prow * a.D + c);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c + 4 * e < a.D)
                            dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                } else if (mine) {
                    store_cols32(static_cast<__nv_bfloat16 *>(a.o) + row * a.D + c, o, a.D - c, wide);
                }
                __syncwarp();  // the next tensor memory read is the whole warp's
            }
            tc_fence_before();  // the next item's first product overwrites O after its P arrives
        }
        if (*abort_flag && a.status) atomicExch(a.status, kDevTimeout);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int DP, bool PACKED>
cudaError_t launch_fwd(const AttnArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, int R,
                       cudaStream_t st) {
    auto kern = attn_fwd_tc_kernel<DP, PACKED>;
    constexpr size_t smem = FwdCfg<DP>::SMEM;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, smem, done);
    if (e != cudaSuccess) return e;
    const int64_t slots = attn_slots(a.sq, a.N, 1, 2 * R), items = slots * a.Hk * a.nsplit;
    if (items >= (int64_t)1 << 31) return cudaErrorInvalidValue;
    kern<<<(unsigned)items, kFwdThreads, smem, st>>>(tq, tk, tv, a, R, (int)slots, wide_rows(a.o, a.D));
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
    if (a.sq.cu)
        return a.D <= 64 ? launch_fwd<64, true>(a, tq, tk, tv, R, st) : launch_fwd<128, true>(a, tq, tk, tv, R, st);
    return a.D <= 64 ? launch_fwd<64, false>(a, tq, tk, tv, R, st) : launch_fwd<128, false>(a, tq, tk, tv, R, st);
}

}  // namespace sgla
