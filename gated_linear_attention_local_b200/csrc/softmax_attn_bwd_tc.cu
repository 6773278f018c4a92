// Softmax attention backward on the tensor cores (tcgen05 / TMEM / TMA), bf16 operands.
//
// The probabilities are recomputed, p = 2^(sc s - lse), and with delta_i = sum_d do_id o_id
//   dv_j = sum_i p_ij do_i,  ds_ij = p_ij (do_i . v_j - delta_i),
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i.
// Two kernels, one per output side, so that every sum has one owner and one order (no
// atomics, no fp32 copy of dq in memory); the price is that s, do v and p are formed twice,
// 7 products of the tile instead of 5.
//
// dk, dv: one CTA owns 128 keys of one key head and walks the rows that see them in tiles of
// 128 packed rows (row = token * G + g, R = 128 / G tokens a tile):
//   S^T = K Q^T, dP^T = V dO^T   (128 keys x 128 rows, fp32, tensor memory; a lane a key)
//   dV += P^T dO,  dK += dS^T Q  (P^T, dS^T in bf16 over S^T's and dP^T's columns)
// issued as dV(i), S(i+1), dK(i), dP(i+1): p of tile i+1 is formed under dK(i) and dP(i+1), ds
// under dV(i+1) and S(i+2), with one buffer each (with heads of 128 tensor memory is full: 4 x 128 columns).
// dq: one CTA owns 128 packed rows and walks the keys they see in tiles of 128:
//   S = Q K^T, dP = dO V^T, dQ += dS K   (a lane a row)
// issued as S(i+1), dP(i+1), dQ(i); dP has two buffers (dS lies over dP).
// Two warpgroups share a tile, 64 of its columns each.  The tensor pipe executes in issue
// order, so a product may overwrite columns that the products issued before it read.
//
// Tiles of 128 x 128 because an M = 128 product of 16 columns costs some 64 cycles for any N
// up to 128: tiles of 64 (tried first) leave half of the tensor rate.
//
// P and dS are rounded to bf16 for their products (relative 2^-8 each, averaged over the
// sum); scores, p, ds, lse, delta and every accumulator are fp32.  A quarter of the
// exponentials runs on the FMA pipe (see softmax_attn_tc.cuh).
//
// The CTAs stay on their SM and take item after item (Feed, softmax_attn_tc.cuh; against a CTA
// an item: the three kernels of packed training 500 -> 427 us when it came): the copies and first
// products of an item run under the stores of the one before.
//
// Measured (events around the launch, cold L2, less the 5 us that an empty pair of events reads):
// 2 x 4096 causal tokens, 16 heads of 128 on 4: dq 187 us, dk dv 231 us (the forward 130); 13 packed
// sequences of up to 2047 tokens, 12 heads of 64: 129 and 164 us (105).  Bound by the chain of a
// tile (scores, p, ds, sums) through one buffer of each in tensor memory (dk dv: it is full for heads
// above 64; up to 64 a quarter of it lies unused); heads of 64 besides by products of 64
// columns, which take as long as 128.
//
// Shared memory (DP = 128): the item's own two tiles 64 KB, rings of three X tiles (Q or K, read
// by the first and the last product of a tile) and two Y tiles (dO or V), 160 KB.
// Warps: 0-7 the warpgroups, 8 TMA, 9 MMA, 10 scheduler (11 fills its warpgroup).
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "softmax_attn.h"
#include "softmax_attn_map.h"
#include "softmax_attn_tc.cuh"

namespace sgla {

using namespace tc;

namespace {

constexpr int kBwdThreads = 384;
constexpr int kTile = 128, kHalf = 64;
constexpr int kStX = 3, kStY = 2;

template <int DP>
struct BwdCfg {
    static constexpr int NG = DP / 64;
    static constexpr uint32_t T = NG * kRegion;      // a tile of 128 rows
    static constexpr uint32_t A0 = 0, B0 = T;        // own tiles: K, V (dk dv) or Q, dO (dq)
    static constexpr uint32_t X0 = 2 * T, Y0 = X0 + kStX * T;
    static constexpr uint32_t ROWS = Y0 + kStY * T;  // [2][128] -lse (log2 units), [128] -delta of a tile's rows
    static constexpr uint32_t BARS = ROWS + 2 * 256 * 4;
    static constexpr uint32_t MISC = BARS + 26 * 8;  // tensor memory address, abort flag, the feed's progress and answer
    static constexpr uint32_t ITEM = MISC + 32;
    // (no slack for alignment: the array is declared with it)
    static constexpr size_t SMEM = ITEM + 64 > 120 * 1024 ? ITEM + 64 : 120 * 1024;
    static constexpr uint32_t COL_S = 0, COL_DP = 128, COL_ACC = 256;  // dk dv: dV, dK; dq: dP's second buffer, dQ
    static_assert(SMEM <= 232448, "shared memory budget");
};

struct BwdBars {
    uint64_t *own, *empty_own, *full_x, *empty_x, *full_y, *empty_y, *s, *sfree, *dp, *p, *ds, *done, *drain, *feed;
    __device__ explicit BwdBars(uint64_t *b)
        : own(b), empty_own(b + 1), full_x(b + 2), empty_x(b + 5), full_y(b + 8), empty_y(b + 10), s(b + 12),
          sfree(b + 13), dp(b + 14), p(b + 16), ds(b + 17), done(b + 19), drain(b + 20), feed(b + 21) {}
    __device__ void init() const {
        mbar_init(own, 1);
        mbar_init(empty_own, 1);
        for (int i = 0; i < kStX; ++i) {
            mbar_init(&full_x[i], 1);
            mbar_init(&empty_x[i], 1);
        }
        for (int i = 0; i < kStY; ++i) {
            mbar_init(&full_y[i], 1);
            mbar_init(&empty_y[i], 1);
        }
        mbar_init(s, 1);
        mbar_init(sfree, 256);
        mbar_init(p, 256);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&dp[i], 1);
            mbar_init(&ds[i], 256);
        }
        mbar_init(done, 1);
        mbar_init(drain, 1);
    }
};

// Zero the rows outside [from, to) of a tile, by one warp.
template <int NG>
__device__ __forceinline__ void zero_outside(unsigned char *tile, int from, int to, int lane) {
    for (int i = lane; i < NG * kTile * 8; i += 32) {
        const int r = (i >> 3) & (kTile - 1);
        if (r < from || r >= to) reinterpret_cast<uint4 *>(tile)[i] = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// Columns [0, D) of this thread's accumulator row times f, as bf16 to dst (zeros with !any; nullptr:
// not stored).
__device__ __forceinline__ void store_acc(uint32_t taddr, bool any, __nv_bfloat16 *dst, int D, float f,
                                          bool wide) {
    __syncwarp();
    for (int c = 0; c < D; c += 32) {
        float o[32];
        if (any) {
            tmem_ld32(taddr + c, o);
            tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = any ? o[e] * f : 0.f;
        if (dst) store_cols32(dst + c, o, D - c, wide);
        __syncwarp();  // the next tensor memory read is the whole warp's
    }
}

__device__ __forceinline__ void ld_pairs(uint32_t taddr, float2 (&v)[32]) {
    float x[32], y[32];
    __syncwarp();
    tmem_ld32(taddr, x);
    tmem_ld32(taddr + 32, y);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        v[e] = make_float2(x[2 * e], x[2 * e + 1]);
        v[16 + e] = make_float2(y[2 * e], y[2 * e + 1]);
    }
}

// The two warps (of the two warpgroups) that share 32 lanes of tensor memory: both have read
// their halves of the columns before either writes over them.
__device__ __forceinline__ void pair_sync(int warp) {
    __syncwarp();
    tc_fence_before();
    named_sync(2 + (warp & 3), 64);
    tc_fence_after();
}

// p = 2^(sc s + nl) of 64 scores (in place); with MASKED only columns [lo, hi) are kept, else a
// quarter of the exponentials goes to the FMA pipe.  nl: one value a column pair.
template <bool MASKED, typename NL>
__device__ __forceinline__ void exp_pass(float2 (&p)[32], float sc, NL nl, int lo, int hi) {
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        float2 x = __ffma2_rn(p[k], make_float2(sc, sc), nl(k));
        if (!MASKED && (k & 3) == 3) {
            x = exp2_fma(x);
        } else {
            x.x = fast_exp2(x.x);
            x.y = fast_exp2(x.y);
        }
        if (MASKED) {
            x.x = (2 * k >= lo && 2 * k < hi) ? x.x : 0.f;
            x.y = (2 * k + 1 >= lo && 2 * k + 1 < hi) ? x.y : 0.f;
        }
        p[k] = x;
    }
}
// ds = p (dp + nd) of 64 columns, into dp; columns outside [lo, hi) are 0 with MASKED (there dp
// may be anything)
template <bool MASKED, typename ND>
__device__ __forceinline__ void ds_pass(const float2 (&p)[32], float2 (&dp)[32], ND nd, int lo, int hi) {
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        float2 x = __fmul2_rn(p[k], __fadd2_rn(dp[k], nd(k)));
        if (MASKED) {
            x.x = (2 * k >= lo && 2 * k < hi) ? x.x : 0.f;
            x.y = (2 * k + 1 >= lo && 2 * k + 1 < hi) ? x.y : 0.f;
        }
        dp[k] = x;
    }
}
// 64 values as bf16 pairs to 32 columns
__device__ __forceinline__ void st64_bf16(uint32_t taddr, const float2 (&v)[32]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = pack_bf16(v[16 * h + e].x, v[16 * h + e].y);
        tmem_st16(taddr + 16 * h, w);
    }
    tmem_wait_st();
}

// Producer, one lane: for every item its own tiles, then X(i), Y(i).  own(it, bar), x(it, i, dst,
// bar), y(...) issue the copies.
template <int DP, typename Item, typename Own, typename X, typename Y>
__device__ __forceinline__ void produce(unsigned char *sm, const BwdBars &b, const Feed<Item> &feed,
                                        uint32_t own_bytes, uint32_t bytes, int lane, Own own, X x, Y y) {
    using C = BwdCfg<DP>;
    volatile int *abort_flag = feed.abort_flag;
    Item it;
    int ni = 0, no = 0, nx = 0, ny = 0;  // items, own tiles, X and Y tiles so far
    Ring<kStX> rx;
    Ring<kStY> ry;
    bool ok = true;
    // (one lane waits and copies, the others meet it at the shuffle behind an item's copies: nothing between
    // is warp-wide; what a product warp that gave up released is not filled again)
    auto wait = [&](uint64_t *bar, uint32_t ph) { return mbar_wait_idle(bar, ph, abort_flag) && !*abort_flag; };
    while (ok && feed.take(ni, it)) {
        if (lane == 0 && it.n > 0) {
            if (no > 0) ok = wait(b.empty_own, (no - 1) & 1);
            if (ok) {
                mbar_arrive_expect_tx(b.own, own_bytes);
                own(it, b.own);
                ++no;
            }
            for (int i = 0; ok && i < it.n; ++i) {
                if (nx >= kStX && !(ok = wait(&b.empty_x[rx.s], rx.ph ^ 1u))) break;
                mbar_arrive_expect_tx(&b.full_x[rx.s], bytes);
                x(it, i, sm + C::X0 + rx.s * C::T, &b.full_x[rx.s]);
                rx.step();
                ++nx;
                if (ny >= kStY && !(ok = wait(&b.empty_y[ry.s], ry.ph ^ 1u))) break;
                mbar_arrive_expect_tx(&b.full_y[ry.s], bytes);
                y(it, i, sm + C::Y0 + ry.s * C::T, &b.full_y[ry.s]);
                ry.step();
                *feed.copies = ++ny;
            }
        }
        if (lane == 0) mbar_arrive(feed.want);
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
    }
    if (lane == 0 && *abort_flag) {  // let the copies in flight land before the CTA exits
        if (no > 0) mbar_drain(b.own, (no - 1) & 1);
        for (int k = max(0, nx - kStX); k < nx; ++k) mbar_drain(&b.full_x[k % kStX], (k / kStX) & 1);
        for (int k = max(0, ny - kStY); k < ny; ++k) mbar_drain(&b.full_y[k % kStY], (k / kStY) & 1);
    }
    __syncwarp();
}

// D (+)= A B over nk 16-column steps, both K-major in shared memory (scores: 128 x 128)
template <int DP>
__device__ __forceinline__ void issue_scores(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id, int nk) {
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk)
        if (kk < nk)
            mma_bf16(d, desc_at(ad, (kk >> 2) * kRegion + (kk & 3) * 32), desc_at(bd, (kk >> 2) * kRegion + (kk & 3) * 32),
                     id, kk > 0 ? 1u : 0u);
}
// D (+)= W X, W (bf16, 128 x 128) in tensor memory, X [128 rows][D] in shared memory
__device__ __forceinline__ void issue_sum(uint32_t d, uint32_t w, uint64_t xd, uint32_t id, bool add) {
#pragma unroll
    for (int jj = 0; jj < kTile / 16; ++jj)
        mma_bf16_tmem_a(d, w + jj * 8, desc_at(xd, jj * 2048), id, (add || jj > 0) ? 1u : 0u);
}

// ------------------------------------------------------------------------------------ dk, dv
struct KvItem {
    int n;       // row tiles that see the item's keys
    int k_tok;   // first key (128 keys of one key head)
    int k_left;  // keys of the sequence from there on
    int q_tok;   // first token of the first row tile
    int q_left;  // tokens of the sequence from there on
    int lead;    // tokens at the head of the first row tile that see none of the keys
    int ahead;   // causal: row c of tile i sees key r iff c >= (ahead + r - i R) G
    int hk;
};

template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
attn_dkdv_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdo,
                    const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, AttnArgs a, int R,
                    int slots, bool wide) {
    using C = BwdCfg<DP>;
    extern __shared__ __align__(1024) unsigned char smem_bwd[];
    unsigned char *sm = smem_bwd;
    const BwdBars b(reinterpret_cast<uint64_t *>(sm + C::BARS));
    float *srow = reinterpret_cast<float *>(sm + C::ROWS);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + C::MISC + 8);
    const Feed<KvItem> feed{b.feed, b.feed + 1, b.feed + 2, b.feed + 3, sm + C::MISC + 16, reinterpret_cast<KvItem *>(sm + C::ITEM),
                            abort_flag, abort_flag + 1};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 256) {
        prefetch_tmap(&tq);
        prefetch_tmap(&tdo);
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
    }
    if (threadIdx.x == 0) {
        b.init();
        feed.init();
        mbar_fence_init();
    }
    if (R * a.G < kTile && warp < kStX + kStY)  // rows that no copy writes are operands too
        zero_outside<C::NG>(sm + C::X0 + warp * C::T, 0, R * a.G, lane);
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
            feed.run([&](int u, KvItem &it) -> bool {
                it.hk = u % a.Hk;
                int64_t slot = u / a.Hk;
                // the first keys are seen by the most rows: every sequence's first tiles first
                if (!a.sk.cu) slot = (slot % a.N) * (slots / a.N) + slot / a.N;
                AttnTile t;
                if (!attn_locate(a, false, slot, 1, kTile, t)) return false;
                const int64_t off = t.tk - t.tq;
                const int64_t first = a.causal ? max((int64_t)0, t.row0 - off) : 0;  // first token that sees the first key
                const int64_t b0 = first / R;                                        // its tile
                it.n = first < t.tq ? (int)((t.tq + R - 1) / R - b0) : 0;
                it.k_tok = (int)(t.k0 + t.row0);
                it.k_left = (int)(t.tk - t.row0);
                it.q_tok = (int)(t.q0 + b0 * R);
                it.q_left = (int)(t.tq - b0 * R);
                it.lead = it.n > 0 ? (int)(first - b0 * R) : 0;
                it.ahead = a.causal ? (int)max(t.row0 - off - b0 * R, -(int64_t)INT_MAX / 2) : -INT_MAX / 2;
                return true;
            });
        } else if (warp == 8) {
            // ---------------------------------------------------------------- TMA producer
            produce<DP>(
                sm, b, feed, 2 * C::T, (uint32_t)(C::NG * R * a.G * 128), lane,
                [&](const KvItem &it, uint64_t *bar) {
                    for (int g = 0; g < C::NG; ++g) {
                        tma_load_3d(sm + C::A0 + g * kRegion, &tk, bar, 64 * g, it.hk, it.k_tok);
                        tma_load_3d(sm + C::B0 + g * kRegion, &tv, bar, 64 * g, it.hk, it.k_tok);
                    }
                },
                [&](const KvItem &it, int i, unsigned char *dst, uint64_t *bar) {
                    for (int g = 0; g < C::NG; ++g)
                        tma_load_3d(dst + g * kRegion, &tq, bar, 64 * g, it.hk * a.G, it.q_tok + i * R);
                },
                [&](const KvItem &it, int i, unsigned char *dst, uint64_t *bar) {
                    for (int g = 0; g < C::NG; ++g)
                        tma_load_3d(dst + g * kRegion, &tdo, bar, 64 * g, it.hk * a.G, it.q_tok + i * R);
                });
        } else if (warp == 9) {
            // ---------------------------------------------------------------- MMA issuer
            const uint32_t idS = idesc_bf16_f32(128, 128, false, false);
            const int nk = (a.D + 15) / 16;
            const uint32_t idA = idesc_bf16_f32(128, 16 * nk, false, true);
            const uint32_t sbase = smem_u32(sm);
            const uint64_t kd = kdesc(sbase + C::A0), vd = kdesc(sbase + C::B0);
            const uint64_t xk = kdesc(sbase + C::X0), yk = kdesc(sbase + C::Y0);
            const uint64_t xm = sdesc(sbase + C::X0, kRegion, 1024, 2), ym = sdesc(sbase + C::Y0, kRegion, 1024, 2);
            auto wait = [&](uint64_t *bar, uint32_t ph) { return all_wait(bar, ph, abort_flag); };
            KvItem it;
            int ni = 0;
            uint32_t own_ph = 0, ph = 0;  // parity of the item's own tiles; of p and ds of the tile in turn
            Ring<kStX> x1, x0;            // X of the scores' tile, of the sums' tile
            Ring<kStY> y1, y0;
            bool ok = true;
            while (ok && feed.take(ni, it)) {
                // the same in every lane; the reduction leaves it in a uniform register
                const int n = __reduce_max_sync(0xffffffffu, it.n);
                if (n == 0) continue;
                // rows of a tile that do not exist, or see none of the keys, are zeroed: 0 * NaN must not arise
                const int whole = it.q_left / R, lead = it.lead * a.G;  // tiles before the first partial one
                auto clean = [&](unsigned char *tile, int i) {
                    if (i >= whole || (i == 0 && lead > 0))
                        zero_outside<C::NG>(tile, i == 0 ? lead : 0, i >= whole ? (it.q_left - i * R) * a.G : kTile, lane);
                };
                if (!(ok = wait(b.own, own_ph))) break;
                own_ph ^= 1u;
                // two blocks of products a tile, each issued without a pause (the pipe holds few
                // products, so a wait between two blocks is time it idles): dV(i) S(i+1), dK(i) dP(i+1)
                for (int i = -1; ok && i < n; ++i) {
                    const bool more = i + 1 < n;
                    if (more) {
                        if (!(ok = wait(&b.full_x[x1.s], x1.ph))) break;
                        clean(sm + C::X0 + x1.s * C::T, i + 1);
                    }
                    if (i >= 0 && !(ok = wait(b.p, ph))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        if (i >= 0) {
                            issue_sum(tmem + C::COL_ACC, tmem + C::COL_S, desc_at(ym, y0.s * C::T), idA, i > 0);
                            mma_commit(&b.empty_y[y0.s]);
                        }
                        if (more) {
                            issue_scores<DP>(tmem + C::COL_S, kd, desc_at(xk, x1.s * C::T), idS, nk);
                            mma_commit(b.s);
                        }
                    }
                    __syncwarp();
                    if (more) {
                        if (!(ok = wait(&b.full_y[y1.s], y1.ph))) break;
                        clean(sm + C::Y0 + y1.s * C::T, i + 1);
                    }
                    if (i >= 0 && !(ok = wait(&b.ds[0], ph))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        if (i >= 0) {
                            issue_sum(tmem + C::COL_ACC + 128, tmem + C::COL_DP, desc_at(xm, x0.s * C::T), idA, i > 0);
                            mma_commit(&b.empty_x[x0.s]);
                            if (!more) mma_commit(b.done);
                        }
                        if (more) {
                            issue_scores<DP>(tmem + C::COL_DP, vd, desc_at(yk, y1.s * C::T), idS, nk);
                            mma_commit(&b.dp[0]);
                            if (i + 1 == n - 1) mma_commit(b.empty_own);
                        }
                    }
                    __syncwarp();
                    if (i >= 0) {
                        y0.step();
                        x0.step();
                        ph ^= 1u;
                    }
                    if (more) {
                        x1.step();
                        y1.step();
                    }
                }
            }
            __syncwarp();
            if (elect_one()) {
                mma_commit(b.drain);
                mbar_drain(b.drain, 0);
            }
        }
    } else {
        // ---------------------------------------------------------------- p, ds and the stores
        setmaxnreg_inc<kRowRegs>();
        const int w = warp >> 2, r = threadIdx.x & 127, c0 = w * kHalf;  // this warpgroup's columns: rows c0 ..
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t cS = tmem + C::COL_S + lanes, cDP = tmem + C::COL_DP + lanes;
        const int rt = r / a.G, rg = r - rt * a.G;
        const float sc = a.scale * kLog2e;
        KvItem it;
        int ni = 0;
        uint32_t tile = 0, done_ph = 0;  // tiles so far, parity of done
        bool ok = true;
        // (all row warps go on or none: a warp that gave up must not leave others at a barrier)
        while (named_all(1, 256, ok && feed.take(ni, it))) {
            const int n = it.n;
            auto rows_of = [&](int i) { return min(R, it.q_left - i * R) * a.G; };
            // -lse (warpgroup 0) or -delta (1) of row r of tile i
            const int64_t row00 = (int64_t)(it.q_tok + rt) * a.H + it.hk * a.G + rg;
            auto row_value = [&](int i) -> float {
                if (i >= n || rt >= R || i * R + rt >= it.q_left) return 0.f;
                const int64_t row = row00 + (int64_t)i * R * a.H;
                return w == 0 ? neg_lse(a.lse_in[row]) : -a.delta[row];
            };
            srow[(tile & 1) * 256 + threadIdx.x] = row_value(0);
            float next = row_value(1);
            // A wait that gave up skips the later ones but none of the barriers: no thread is left behind.
            for (int i = 0; i < n; ++i, ++tile) {
                // this tile's values are written, and those of the one before have been read
                named_sync(1, 256);
                srow[((tile + 1) & 1) * 256 + threadIdx.x] = next;
                next = row_value(i + 2);
                const float4 *l4 = reinterpret_cast<const float4 *>(srow + (tile & 1) * 256 + c0), *d4 = l4 + 32;
                auto nl = [&](int k) {
                    const float4 x = l4[k >> 1];
                    return k & 1 ? make_float2(x.z, x.w) : make_float2(x.x, x.y);
                };
                auto nd = [&](int k) {
                    const float4 x = d4[k >> 1];
                    return k & 1 ? make_float2(x.z, x.w) : make_float2(x.x, x.y);
                };
                const int hi = rows_of(i) - c0;
                const int64_t lo64 = ((int64_t)it.ahead + r - (int64_t)i * R) * a.G;
                const int lo = (int)max((int64_t)0, min64(lo64, kTile)) - c0;
                const bool masked = __any_sync(0xffffffffu, lo > 0 || hi < kHalf);
                ok = ok && mbar_wait(b.s, tile & 1, abort_flag);
                tc_fence_after();
                float2 p[32], dp[32];
                ld_pairs(cS + c0, p);
                if (masked) exp_pass<true>(p, sc, nl, lo, hi);
                else exp_pass<false>(p, sc, nl, lo, hi);
                pair_sync(warp);  // P lies over S
                st64_bf16(cS + c0 / 2, p);
                tc_fence_before();
                mbar_arrive(b.p);
                ok = ok && mbar_wait(&b.dp[0], tile & 1, abort_flag);
                tc_fence_after();
                ld_pairs(cDP + c0, dp);
                if (masked) ds_pass<true>(p, dp, nd, lo, hi);
                else ds_pass<false>(p, dp, nd, lo, hi);
                pair_sync(warp);  // dS lies over dP
                st64_bf16(cDP + c0 / 2, dp);
                tc_fence_before();
                mbar_arrive(&b.ds[0]);
            }
            if (n > 0) {
                ok = ok && mbar_wait(b.done, done_ph, abort_flag);
                done_ph ^= 1u;
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) continue;
            tc_fence_after();
            __nv_bfloat16 *dst = r < it.k_left ? static_cast<__nv_bfloat16 *>(w == 0 ? a.dv : a.dk) +
                                                     ((int64_t)(it.k_tok + r) * a.Hk + it.hk) * a.D
                                               : nullptr;
            store_acc(tmem + C::COL_ACC + w * 128 + lanes, n > 0, dst, a.D, w == 0 ? 1.f : a.scale, wide);
            tc_fence_before();  // the next item's first sums overwrite the accumulators after its P arrives
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

// ------------------------------------------------------------------------------------ dq
struct QItem {
    int n;       // key tiles that the item's rows see
    int q_tok;   // first token
    int q_left;  // tokens of the sequence from there on
    int k_tok;   // first key of the sequence
    int keys;    // its keys
    int shift;   // causal: token x of the item sees keys < x + 1 + shift
    int hk;
};

template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
attn_dq_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdo,
                  const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, AttnArgs a, int R,
                  int slots, bool wide) {
    using C = BwdCfg<DP>;
    extern __shared__ __align__(1024) unsigned char smem_bwd[];
    unsigned char *sm = smem_bwd;
    const BwdBars b(reinterpret_cast<uint64_t *>(sm + C::BARS));
    float *srow = reinterpret_cast<float *>(sm + C::ROWS);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + C::MISC + 8);
    const Feed<QItem> feed{b.feed, b.feed + 1, b.feed + 2, b.feed + 3, sm + C::MISC + 16, reinterpret_cast<QItem *>(sm + C::ITEM),
                           abort_flag, abort_flag + 1};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 256) {
        prefetch_tmap(&tq);
        prefetch_tmap(&tdo);
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
    }
    if (threadIdx.x == 0) {
        b.init();
        feed.init();
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

    // (one instruction a warpgroup, ahead of the roles: setmaxnreg is .aligned)
    if (warp >= 8) {
        setmaxnreg_dec<kOtherRegs>();
        if (warp == 10) {
            // ---------------------------------------------------------------- scheduler
            feed.run([&](int u, QItem &it) -> bool {
                it.hk = u % a.Hk;
                int64_t slot = slots - 1 - u / a.Hk;  // the last rows see the most keys
                if (!a.sq.cu) slot = (slot % a.N) * (slots / a.N) + slot / a.N;
                AttnTile t;
                if (!attn_locate(a, true, slot, 1, R, t)) return false;
                it.q_tok = (int)(t.q0 + t.row0);
                it.q_left = (int)(t.tq - t.row0);
                it.k_tok = (int)t.k0;
                it.keys = (int)t.tk;
                it.shift = (int)max(min64(t.row0 + t.tk - t.tq, INT_MAX - 256), -(int64_t)INT_MAX / 2);
                const int seen = a.causal ? min(it.keys, min(R, it.q_left) + it.shift) : it.keys;
                it.n = seen > 0 ? (seen + kTile - 1) / kTile : 0;
                return true;
            });
        } else if (warp == 8) {
            // ---------------------------------------------------------------- TMA producer
            produce<DP>(
                sm, b, feed, 2u * C::NG * R * a.G * 128, C::T, lane,
                [&](const QItem &it, uint64_t *bar) {
                    for (int g = 0; g < C::NG; ++g) {
                        tma_load_3d(sm + C::A0 + g * kRegion, &tq, bar, 64 * g, it.hk * a.G, it.q_tok);
                        tma_load_3d(sm + C::B0 + g * kRegion, &tdo, bar, 64 * g, it.hk * a.G, it.q_tok);
                    }
                },
                [&](const QItem &it, int i, unsigned char *dst, uint64_t *bar) {
                    for (int g = 0; g < C::NG; ++g)
                        tma_load_3d(dst + g * kRegion, &tk, bar, 64 * g, it.hk, it.k_tok + i * kTile);
                },
                [&](const QItem &it, int i, unsigned char *dst, uint64_t *bar) {
                    for (int g = 0; g < C::NG; ++g)
                        tma_load_3d(dst + g * kRegion, &tv, bar, 64 * g, it.hk, it.k_tok + i * kTile);
                });
        } else if (warp == 9) {
            // ---------------------------------------------------------------- MMA issuer
            const uint32_t idS = idesc_bf16_f32(128, 128, false, false);
            const int nk = (a.D + 15) / 16;
            const uint32_t idA = idesc_bf16_f32(128, 16 * nk, false, true);
            const uint32_t sbase = smem_u32(sm);
            const uint64_t qd = kdesc(sbase + C::A0), dd = kdesc(sbase + C::B0);
            const uint64_t xk = kdesc(sbase + C::X0), yk = kdesc(sbase + C::Y0);
            const uint64_t xm = sdesc(sbase + C::X0, kRegion, 1024, 2);
            // A wait that gave up (abort is set then) sends no lane another way: the products go on, over
            // whatever is there, to the item's end, where the lanes vote.  (A vote on every wait, all_wait:
            // 177 -> 180 us at 2 x 4096 tokens of 16 heads.)
            auto wait = [&](uint64_t *bar, uint32_t ph) { mbar_wait(bar, ph, abort_flag); };
            auto sound = [&] { return __all_sync(0xffffffffu, !*abort_flag); };
            QItem it;
            int ni = 0;
            uint32_t own_ph = 0;
            Ring<kStX> x1, x0;  // K of the scores' tile, of the sum's tile
            Ring<kStY> y1;
            Ring<2> d1, d0;     // dP's buffers, of the scores' tile, of the sum's tile
            uint32_t free_ph = 1;  // parity of S's release by the tile before the scores' tile
            while (sound() && feed.take(ni, it)) {
                const int n = __reduce_max_sync(0xffffffffu, it.n);
                if (n == 0) continue;
                wait(b.own, own_ph);
                own_ph ^= 1u;
                for (int i = -1; i < n; ++i) {
                    if ((i & 1023) == 1023 && i > 0 && !sound()) break;  // (the rest of a long item)
                    if (i + 1 < n) {
                        wait(&b.full_x[x1.s], x1.ph);
                        const int left = it.keys - (i + 1) * kTile;  // keys behind the sequence are operands too
                        if (left < kTile) zero_outside<C::NG>(sm + C::X0 + x1.s * C::T, 0, left, lane);
                        wait(&b.full_y[y1.s], y1.ph);
                        wait(b.sfree, free_ph);  // (the very first passes at once)
                        free_ph ^= 1u;
                        tc_fence_after();
                        if (elect_one()) {
                            issue_scores<DP>(tmem + C::COL_S, qd, desc_at(xk, x1.s * C::T), idS, nk);
                            mma_commit(b.s);
                            issue_scores<DP>(tmem + C::COL_DP + d1.s * 128, dd, desc_at(yk, y1.s * C::T), idS, nk);
                            mma_commit(&b.dp[d1.s]);
                            mma_commit(&b.empty_y[y1.s]);
                            if (i + 1 == n - 1) mma_commit(b.empty_own);
                        }
                        __syncwarp();
                        x1.step();
                        y1.step();
                        d1.step();
                    }
                    if (i >= 0) {
                        wait(&b.ds[d0.s], d0.ph);
                        tc_fence_after();
                        if (elect_one()) {
                            issue_sum(tmem + C::COL_ACC + 128, tmem + C::COL_DP + d0.s * 128, desc_at(xm, x0.s * C::T), idA,
                                      i > 0);
                            mma_commit(&b.empty_x[x0.s]);
                            if (i == n - 1) mma_commit(b.done);
                        }
                        __syncwarp();
                        x0.step();
                        d0.step();
                    }
                }
            }
            __syncwarp();
            if (elect_one()) {
                mma_commit(b.drain);
                mbar_drain(b.drain, 0);
            }
        }
    } else {
        // ---------------------------------------------------------------- delta, p, ds and the stores
        setmaxnreg_inc<kRowRegs>();
        const int w = warp >> 2, r = threadIdx.x & 127, c0 = w * kHalf;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t cS = tmem + C::COL_S + lanes, cDP = tmem + C::COL_DP + lanes;
        const int tr = r / a.G, tg = r - tr * a.G;
        const float sc = a.scale * kLog2e;
        QItem it;
        int ni = 0;
        uint32_t tile = 0, done_ph = 0;
        bool ok = true;
        // (all row warps go on or none: a warp that gave up must not leave others at a barrier)
        while (named_all(1, 256, ok && feed.take(ni, it))) {
            const int n = it.n;
            const bool mine = tr < R && tr < it.q_left;
            const int lim = mine ? max(0, a.causal ? min(it.keys, tr + 1 + it.shift) : it.keys) : 0;
            const int64_t row = mine ? (int64_t)(it.q_tok + tr) * a.H + it.hk * a.G + tg : 0;
            const float nlse = mine ? neg_lse(a.lse_in[row]) : 0.f;
            // delta = sum_d do o: a lane takes a 16-byte piece of a row, a warp 16 rows
            {
                constexpr int PER = DP / 8, NK = 16 * PER / 32;
                const int piece = lane & (PER - 1);
                uint4 g[NK], o[NK];
#pragma unroll
                for (int k = 0; k < NK; ++k) {  // every load first
                    const int rr = warp * 16 + k * (32 / PER) + lane / PER, t = rr / a.G;
                    g[k] = o[k] = make_uint4(0, 0, 0, 0);
                    if (t < R && t < it.q_left && 8 * piece < a.D) {
                        const int64_t at = ((int64_t)(it.q_tok + t) * a.H + it.hk * a.G + rr - t * a.G) * a.D + 8 * piece;
                        g[k] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.dout) + at);
                        o[k] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.o) + at);
                    }
                }
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    const uint32_t gs[4] = {g[k].x, g[k].y, g[k].z, g[k].w}, os[4] = {o[k].x, o[k].y, o[k].z, o[k].w};
                    float x = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&gs[e]));
                        const float2 z = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&os[e]));
                        x = fmaf(y.x, z.x, x);
                        x = fmaf(y.y, z.y, x);
                    }
#pragma unroll
                    for (int d = PER / 2; d >= 1; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                    // (the other half of srow belongs to the item before)
                    if (piece == 0) srow[(ni & 1) * 256 + warp * 16 + k * (32 / PER) + lane / PER] = x;
                }
            }
            named_sync(1, 256);
            float delta = srow[(ni & 1) * 256 + r];
            if (mine && w == 0) a.delta[row] = delta;
            // A wait that gave up skips the later ones but none of the barriers: no thread is left behind.
            for (int i = 0; i < n; ++i, ++tile) {
                const int left = lim - i * kTile - c0;  // of this thread's columns, the first `left` are seen
                const bool masked = __any_sync(0xffffffffu, left < kHalf);
                ok = ok && mbar_wait(b.s, tile & 1, abort_flag);
                tc_fence_after();
                float2 p[32], dp[32];
                ld_pairs(cS + c0, p);
                tc_fence_before();
                mbar_arrive(b.sfree);
                auto nl = [&](int) { return make_float2(nlse, nlse); };
                if (masked) exp_pass<true>(p, sc, nl, 0, left);
                else exp_pass<false>(p, sc, nl, 0, left);
                ok = ok && mbar_wait(&b.dp[tile & 1], (tile >> 1) & 1, abort_flag);
                tc_fence_after();
                ld_pairs(cDP + (tile & 1) * 128 + c0, dp);
                if (i == 0 && w == 0 && __any_sync(0xffffffffu, lim > 0 && lim <= kHalf)) {
                    // All keys of such a row are here: delta = sum_j p dp in fp32.  The one from o
                    // carries o's rounding, which for rows with few keys is the largest error of
                    // dq and dk (measured: dq off by 2.5e-3 with it, 2.4e-3 without).
                    float x = 0.f;
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        if (2 * k < lim) x = fmaf(p[k].x, dp[k].x, x);
                        if (2 * k + 1 < lim) x = fmaf(p[k].y, dp[k].y, x);
                    }
                    if (lim > 0 && lim <= kHalf) {
                        delta = x;
                        a.delta[row] = x;
                    }
                    __syncwarp();
                }
                auto nd = [&](int) { return make_float2(-delta, -delta); };
                if (masked) ds_pass<true>(p, dp, nd, 0, left);
                else ds_pass<false>(p, dp, nd, 0, left);
                pair_sync(warp);  // dS lies over dP
                st64_bf16(cDP + (tile & 1) * 128 + c0 / 2, dp);
                tc_fence_before();
                mbar_arrive(&b.ds[tile & 1]);
            }
            if (n > 0) {
                ok = ok && mbar_wait(b.done, done_ph, abort_flag);
                done_ph ^= 1u;
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) continue;
            tc_fence_after();
            // each warpgroup stores half of the columns
            const int half = a.D > 64 ? 64 : 32, h0 = w == 0 ? 0 : half, h1 = w == 0 ? min(a.D, half) : a.D;
            __nv_bfloat16 *dst = mine ? static_cast<__nv_bfloat16 *>(a.dq) + row * a.D + h0 : nullptr;
            if (h1 > h0) store_acc(tmem + C::COL_ACC + 128 + h0 + lanes, n > 0, dst, h1 - h0, a.scale, wide);
            tc_fence_before();  // the next item's first sum overwrites the accumulator after its dS arrives
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

struct Maps {
    CUtensorMap q, dout, k, v;
};

// boxes: q, dout G heads x R tokens, k and v 128 tokens
cudaError_t make_maps(const AttnArgs &a, int R, Maps &m) {
    const int64_t qt = a.sq.cu ? a.sq.T : a.N * a.sq.T, kt = a.sk.cu ? a.sk.T : a.N * a.sk.T;
    cudaError_t e = cudaSuccess;
    if (qt > 0) {
        if ((e = tc_make_map_rows(&m.q, a.q, qt, a.H, a.D, a.G, R)) != cudaSuccess) return e;
        if ((e = tc_make_map_rows(&m.dout, a.dout, qt, a.H, a.D, a.G, R)) != cudaSuccess) return e;
    }
    if (kt > 0) {
        if ((e = tc_make_map_rows(&m.k, a.k, kt, a.Hk, a.D, 1, kTile)) != cudaSuccess) return e;
        if ((e = tc_make_map_rows(&m.v, a.v, kt, a.Hk, a.D, 1, kTile)) != cudaSuccess) return e;
    }
    if (qt == 0) m.q = m.dout = m.k;  // a side without tokens is never copied
    if (kt == 0) m.k = m.v = m.q;
    return e;
}

template <int DP>
cudaError_t launch_dkdv(const AttnArgs &a, const Maps &m, int R, cudaStream_t st) {
    auto kern = attn_dkdv_tc_kernel<DP>;
    constexpr size_t smem = BwdCfg<DP>::SMEM;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, smem, done);
    if (e != cudaSuccess) return e;
    const int64_t slots = attn_slots(a.sk, a.N, 1, kTile);
    if (slots * a.Hk >= (int64_t)1 << 31) return cudaErrorInvalidValue;
    kern<<<(unsigned)(slots * a.Hk), kBwdThreads, smem, st>>>(m.q, m.dout, m.k, m.v, a, R, (int)slots,
                                                              wide_rows(a.dk, a.D) && wide_rows(a.dv, a.D));
    return cudaGetLastError();
}

template <int DP>
cudaError_t launch_dq(const AttnArgs &a, const Maps &m, int R, cudaStream_t st) {
    auto kern = attn_dq_tc_kernel<DP>;
    constexpr size_t smem = BwdCfg<DP>::SMEM;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, smem, done);
    if (e != cudaSuccess) return e;
    const int64_t slots = attn_slots(a.sq, a.N, 1, R);
    if (slots * a.Hk >= (int64_t)1 << 31) return cudaErrorInvalidValue;
    kern<<<(unsigned)(slots * a.Hk), kBwdThreads, smem, st>>>(m.q, m.dout, m.k, m.v, a, R, (int)slots,
                                                              wide_rows(a.dq, a.D));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_bwd_dkdv_tc(const AttnArgs &a, cudaStream_t st) {
    const int R = kTile / a.G;
    Maps m;
    const cudaError_t e = make_maps(a, R, m);
    if (e != cudaSuccess) return e;
    return a.D <= 64 ? launch_dkdv<64>(a, m, R, st) : launch_dkdv<128>(a, m, R, st);
}

cudaError_t launch_attn_bwd_dq_tc(const AttnArgs &a, cudaStream_t st) {
    const int R = kTile / a.G;
    Maps m;
    const cudaError_t e = make_maps(a, R, m);
    if (e != cudaSuccess) return e;
    return a.D <= 64 ? launch_dq<64>(a, m, R, st) : launch_dq<128>(a, m, R, st);
}

}  // namespace sgla
