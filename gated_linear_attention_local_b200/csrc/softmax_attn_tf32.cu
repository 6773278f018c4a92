// Softmax attention for fp32 operands: forward, dk / dv, dq and the row sums delta.
//
// fp32 products on the tensor cores: x = hi + lo with hi the nearest value of 11 significant
// bits (the tf32 format) and lo the rest (13 bits, of which 11 are kept), and
//   x y = hi hi + hi lo + lo hi  (lo lo, below 2^-22 of the product, is left out),
// three mma.sync m16n8k8 with fp32 sums in place of 8 x 16 x 8 FMAs: the error of a product is
// 2^-21 at most, of the order of an fp32 dot product's own.  (tcgen05 would have to write hi
// and lo as operands of their own to shared memory; these sizes are bound by latency.)
//
// Tiles of 64 packed rows (row = token * G + g) x 64 keys, 256 threads: warp (wr, wc) has 16 of the
// rows and 32 of the keys.  Forward: every warp keeps the running maximum and sum of its rows
// over its keys, and the two halves are joined at the end, so warps only meet to change tiles.
// Backward: p = 2^(s - lse) again, and with delta_i = sum_d do o
//   dv_j = sum_i p_ij do_i,  ds_ij = p_ij (do_i . v_j - delta_i),
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,
// in two passes, one per output side, so that every sum has one owner and one order; there the
// two halves are partial sums, joined at the end.
//
// A cluster of up to 8 CTAs shares a tile where there are fewer tiles than SMs: each takes a part
// of the keys (dk dv: of the rows), and the parts are joined through distributed shared memory
// in a fixed order (2 x 317 queries and 501 keys, 8 heads of 64 on 4: 203 -> 143 us a training pass when it
// came, with two CTAs an SM up to D = 64; now 150, with operands split safely to the ends of their range.
// What is left is latency: four launches, and 2 to 8 tiles a CTA in turn).
//
// The scores' accumulators are the next product's A operand as they stand: columns 2 t and
// 2 t + 1 of an accumulator are taken as k = t and k = t + 4, and the B operand's rows are read in
// that order.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "softmax_attn.h"

namespace sgla {

namespace cg = cooperative_groups;

namespace {

constexpr int kB = 64;  // tile edge
constexpr int kMaxCluster = 8;
constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Row stride (floats) of a [64][DP] tile: stride 4 modulo 32 keeps the fragments' reads, rows g
// and columns t or rows 2 t and columns g, on different banks.
template <int DP>
struct Stride {
    static constexpr int value = DP + 4;
};

struct Split {
    uint32_t hi, lo;
};
__device__ __forceinline__ Split split(float x) {
    // |x| first cut to the largest 11-bit value: rounding would take values above it to infinity, and
    // lo = x - hi to NaN.  (An infinity is then lo's.)
    float cut;
    asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(cut) : "f"(x), "f"(__uint_as_float(0x7f7fe000u)));
    Split s;
    s.hi = (__float_as_uint(cut) + 0x1000u) & 0xffffe000u;
    s.lo = __float_as_uint(x - __uint_as_float(s.hi));
    return s;
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
struct FragA {
    uint32_t hi[4], lo[4];
    __device__ __forceinline__ void set(float x0, float x1, float x2, float x3) {
        const Split s[4] = {split(x0), split(x1), split(x2), split(x3)};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = s[e].hi;
            lo[e] = s[e].lo;
        }
    }
};
__device__ __forceinline__ void mma3(float (&c)[4], const FragA &a, float x0, float x1) {
    const Split b0 = split(x0), b1 = split(x1);
    mma_tf32(c, a.lo, b0.hi, b1.hi);
    mma_tf32(c, a.hi, b0.lo, b1.lo);
    mma_tf32(c, a.hi, b0.hi, b1.hi);
}

__device__ __forceinline__ void copy16(float *dst, const float *src, bool there) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where packed row r of key head hk lies in a [tokens, H, D] tensor.
__device__ __forceinline__ int64_t row_offset(int64_t tok0, int64_t r, int G, int H, int hk) {
    const int64_t t = r / G;
    return (tok0 + t) * H + hk * G + (int)(r - t * G);
}

// Rows [r0, r0 + 64) of one side into a tile, zeros past `rows` and past column D (asynchronous).
template <int DP>
__device__ __forceinline__ void copy_rows(float *tile, const float *src, int64_t tok0, int64_t r0, int64_t rows, int G,
                                          int H, int hk, int D) {
    constexpr int NV = DP / 4;
    for (int i = threadIdx.x; i < kB * NV; i += kThreads) {
        const int r = i / NV, c = (i - r * NV) * 4;
        const bool there = r0 + r < rows && c < D;
        copy16(tile + r * Stride<DP>::value + c,
               there ? src + row_offset(tok0, r0 + r, G, H, hk) * D + c : src, there);
    }
}

// lse in units of log2, for p = 2^(s - lse).  -inf (the row saw nothing, or only scores of -inf): +inf, so
// that all its p are 0.
__device__ __forceinline__ float lse_log2(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

// First key that row r of a sequence must not see (keys [0, limit) are seen).
__device__ __forceinline__ int64_t key_limit(const AttnArgs &a, const AttnTile &t, int64_t r, int64_t k_end) {
    if (r >= t.tq * a.G) return 0;
    return a.causal ? min64(k_end, r / a.G + 1 + t.tk - t.tq) : k_end;
}

// The products' fp32 sums are cut off, not rounded, so a long chain of them drifts (measured: 3e-6
// of the result after some hundred products, 5e-7 in fp32 FMAs).  Chains are therefore kept to
// two steps of 8 (six products) and added up in rounded fp32.
//
// c[n] += A[row0 + .. 16][:] . B[col0 + 8 n + ..][:], both tiles row-major over D
template <int DP>
__device__ __forceinline__ void scores(float (&c)[4][4], const float *A, const float *B, int row0, int col0, int nk,
                                       int lane) {
    constexpr int S = Stride<DP>::value;
    const int g = lane >> 2, t = lane & 3;
    const float *pa = A + (row0 + g) * S + t, *pb = B + (col0 + g) * S + t;
#pragma unroll 2
    for (int k2 = 0; k2 < nk; k2 += 2) {  // (the tiles hold zeros past D)
        FragA a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int k = 8 * (k2 + e);
            a[e].set(pa[k], pa[8 * S + k], pa[k + 4], pa[8 * S + k + 4]);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float x[4] = {};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int k = 8 * (k2 + e);
                mma3(x, a[e], pb[8 * n * S + k], pb[8 * n * S + k + 4]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) c[n][e] += x[e];
        }
    }
}

// o[n] += W X with W the 16 x 32 accumulators w and X the rows row0 .. row0 + 32 of a tile
template <int DP>
__device__ __forceinline__ void weighted(float (&o)[DP / 8][4], const float (&w)[4][4], const float *X, int row0, int nd,
                                         int lane) {
    constexpr int S = Stride<DP>::value;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int k2 = 0; k2 < 4; k2 += 2) {
        FragA a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) a[e].set(w[k2 + e][0], w[k2 + e][2], w[k2 + e][1], w[k2 + e][3]);
        const float *px = X + (row0 + 8 * k2 + 2 * t) * S + g;
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
            if (n < nd) {
                float x[4] = {};
#pragma unroll
                for (int e = 0; e < 2; ++e) mma3(x, a[e], px[8 * e * S + 8 * n], px[8 * e * S + 8 * n + S]);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][e] += x[e];
            }
    }
}

// A warp's 16 x DP accumulators to (or, add: onto those in) rows row0 .. of a tile.
template <int DP>
__device__ __forceinline__ void put_acc(float *tile, const float (&o)[DP / 8][4], int row0, float f0, float f1, bool add,
                                        int lane) {
    constexpr int S = Stride<DP>::value;
    float *p0 = tile + (row0 + (lane >> 2)) * S + 2 * (lane & 3), *p1 = p0 + 8 * S;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
        float2 x = make_float2(o[n][0] * f0, o[n][1] * f0), y = make_float2(o[n][2] * f1, o[n][3] * f1);
        if (add) {
            const float2 u = *reinterpret_cast<float2 *>(p0 + 8 * n), v = *reinterpret_cast<float2 *>(p1 + 8 * n);
            x = make_float2(x.x + u.x, x.y + u.y);
            y = make_float2(y.x + v.x, y.y + v.y);
        }
        *reinterpret_cast<float2 *>(p0 + 8 * n) = x;
        *reinterpret_cast<float2 *>(p1 + 8 * n) = y;
    }
}

// This CTA's part [beg, end) of `tiles` tiles, cut evenly over its cluster.
struct Part {
    int rank, cs;
    int64_t beg, end;
    __device__ Part(int64_t tiles) {
        const cg::cluster_group cluster = cg::this_cluster();
        cs = (int)cluster.num_blocks();
        rank = (int)cluster.block_rank();
        const int64_t per = (tiles + cs - 1) / cs;
        beg = rank * per;
        end = min64(tiles, beg + per);
    }
};
__device__ __forceinline__ void cluster_meet(int cs) {
    if (cs > 1) cg::this_cluster().sync();
    else __syncthreads();
}
// Sum over the cluster of the 4 floats at p of everyone's shared memory, in rank order.
__device__ __forceinline__ float4 cluster_sum(float *p, int cs) {
    const cg::cluster_group cluster = cg::this_cluster();
    float4 x[kMaxCluster], y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
        if (r < cs) x[r] = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(p, r));
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
        if (r < cs) y = make_float4(y.x + x[r].x, y.y + x[r].y, y.z + x[r].z, y.w + x[r].w);
    return y;
}

template <int DP>
__global__ void __launch_bounds__(kThreads, DP <= 64 ? 2 : 1) attn_fwd_tf32_kernel(AttnArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int S = Stride<DP>::value, T = kB * S;
    float *sq = sm, *skv = sq + T;                 // two stages of K, V
    float *sml = skv + 4 * T;                      // [2][64][2] maximum and sum of the halves
    float *sall = sml + 4 * kB;                    // [64][2] of both
    float *sw = sall + 2 * kB;                     // [8][64] weights of the cluster's parts, [64] 1 / sum
    AttnTile t;
    const int hk = blockIdx.y;
    if (!attn_locate(a, true, blockIdx.x / cg::this_cluster().num_blocks(), a.G, kB, t)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wr = warp & 3, wc = warp >> 2;
    const int64_t rows = t.tq * a.G;
    const int64_t kb0 = blockIdx.z * a.split, ke = min64(t.tk, kb0 + a.split);
    const int nk = (a.D + 7) / 8;
    // keys that some row of the tile sees, and this CTA's part of them
    const int64_t seen = key_limit(a, t, min64(t.row0 + kB, rows) - 1, ke);
    const Part part(seen > kb0 ? (seen - kb0 + kB - 1) / kB : 0);
    const int64_t kb = kb0 + part.beg * kB, last = min64(seen, kb0 + part.end * kB);
    int64_t lim[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) lim[h] = key_limit(a, t, t.row0 + 16 * wr + 8 * h + (lane >> 2), ke);
    auto copy_tile = [&](int64_t j0, int st) {
        copy_rows<DP>(skv + 2 * st * T, static_cast<const float *>(a.k), t.k0, j0, t.tk, 1, a.Hk, hk, a.D);
        copy_rows<DP>(skv + (2 * st + 1) * T, static_cast<const float *>(a.v), t.k0, j0, t.tk, 1, a.Hk, hk, a.D);
    };
    copy_rows<DP>(sq, static_cast<const float *>(a.q), t.q0, t.row0, rows, a.G, a.H, hk, a.D);
    if (kb < last) copy_tile(kb, 0);
    copies_commit();
    float o[DP / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    const float sc = a.scale * kLog2e;
    int st = 0;
    for (int64_t j0 = kb; j0 < last; j0 += kB, st ^= 1) {
        if (j0 + kB < last) copy_tile(j0 + kB, st ^ 1);
        copies_commit();
        copies_wait<1>();
        __syncthreads();
        const float *sk = skv + 2 * st * T, *sv = sk + T;
        float s[4][4] = {};
        scores<DP>(s, sq, sk, 16 * wr, 32 * wc, nk, lane);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t left = lim[h] - j0 - 32 * wc - 2 * (lane & 3);
            float top = m[h];
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &x = s[n][2 * h + e];
                    x = 8 * n + e < left ? x * sc : -INFINITY;
                    top = fmaxf(top, x);
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float base = top == -INFINITY ? 0.f : top;
            const float f = exp2f(m[h] - base);  // 0 while nothing was seen
            m[h] = top;
            l[h] *= f;
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &x = s[n][2 * h + e];
                    x = exp2f(x - base);
                    l[h] += x;
                }
#pragma unroll
            for (int n = 0; n < DP / 8; ++n) {
                o[n][2 * h] *= f;
                o[n][2 * h + 1] *= f;
            }
        }
        weighted<DP>(o, s, sv, 32 * wc, nk, lane);
        __syncthreads();  // the stage may be filled again
    }
    copies_wait<0>();
    // the two halves of the keys: their common maximum, the sum, o relative to that maximum
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if ((lane & 3) == 0) {
            float *p = sml + (wc * kB + 16 * wr + 8 * h + (lane >> 2)) * 2;
            p[0] = m[h];
            p[1] = l[h];
        }
    }
    __syncthreads();
    float f[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = 16 * wr + 8 * h + (lane >> 2);
        const float m0 = sml[2 * r], m1 = sml[2 * (kB + r)];
        const float top = fmaxf(m0, m1), base = top == -INFINITY ? 0.f : top;
        f[h] = exp2f(m[h] - base);
        if (wc == 0 && (lane & 3) == 0) {
            sall[2 * r] = top;
            sall[2 * r + 1] = sml[2 * r + 1] * exp2f(m0 - base) + sml[2 * (kB + r) + 1] * exp2f(m1 - base);
        }
    }
    if (wc == 1) put_acc<DP>(sq, o, 16 * wr, f[0], f[1], false, lane);
    __syncthreads();
    if (wc == 0) put_acc<DP>(sq, o, 16 * wr, f[0], f[1], true, lane);
    cluster_meet(part.cs);
    // the parts of the cluster
    const cg::cluster_group cluster = cg::this_cluster();
    if (threadIdx.x < kB) {
        float top = -INFINITY, sum = 0.f;
        for (int c = 0; c < part.cs; ++c) top = fmaxf(top, cluster.map_shared_rank(sall, c)[2 * threadIdx.x]);
        const float base = top == -INFINITY ? 0.f : top;
        for (int c = 0; c < part.cs; ++c) {
            const float *p = cluster.map_shared_rank(sall, c) + 2 * threadIdx.x;
            const float w = exp2f(p[0] - base);
            sw[c * kB + threadIdx.x] = w;
            sum = fmaf(w, p[1], sum);
        }
        sw[kMaxCluster * kB + threadIdx.x] = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);  // NaN scores stay NaN
        const int64_t row = t.row0 + threadIdx.x;
        if (part.rank == 0 && row < rows) {
            const float lse = sum > 0.f ? (base + log2f(sum)) * kLn2 : (sum == 0.f ? -INFINITY : sum);
            const int64_t at = row_offset(t.q0, row, a.G, a.H, hk);
            if (a.part_lse) a.part_lse[blockIdx.z * a.part_rows + at] = lse;
            else if (a.lse) a.lse[at] = lse;
        }
    }
    __syncthreads();
    for (int i = part.rank * kThreads + threadIdx.x; i < kB * (DP / 4); i += part.cs * kThreads) {
        const int r = i / (DP / 4), c = (i - r * (DP / 4)) * 4;
        if (t.row0 + r >= rows || c >= a.D) continue;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < part.cs; ++p) {
            const float4 y = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(sq, p) + r * S + c);
            const float w = sw[p * kB + r];
            x = make_float4(fmaf(w, y.x, x.x), fmaf(w, y.y, x.y), fmaf(w, y.z, x.z), fmaf(w, y.w, x.w));
        }
        const float inv = sw[kMaxCluster * kB + r];
        const int64_t at = row_offset(t.q0, t.row0 + r, a.G, a.H, hk);
        float *dst = a.part_o ? a.part_o + (blockIdx.z * a.part_rows + at) * a.D : static_cast<float *>(a.o) + at * a.D;
        *reinterpret_cast<float4 *>(dst + c) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    }
    cluster_meet(part.cs);  // everyone's shared memory has been read
}

// 64 keys of one key head: dk, dv over every row that sees them.
template <int DP>
__global__ void __launch_bounds__(kThreads, DP <= 64 ? 2 : 1) attn_dkdv_tf32_kernel(AttnArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int S = Stride<DP>::value, T = kB * S;
    float *sk = sm, *sv = sk + T, *sq = sv + T, *sd = sq + T, *srow = sd + T;  // srow: [64] lse (log2 units), [64] delta
    AttnTile t;
    const int hk = blockIdx.y;
    if (!attn_locate(a, false, blockIdx.x / cg::this_cluster().num_blocks(), 1, kB, t)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wr = warp & 3, wc = warp >> 2;
    const int64_t rows = t.tq * a.G, j0 = t.row0;
    const int nk = (a.D + 7) / 8;
    copy_rows<DP>(sk, static_cast<const float *>(a.k), t.k0, j0, t.tk, 1, a.Hk, hk, a.D);
    copy_rows<DP>(sv, static_cast<const float *>(a.v), t.k0, j0, t.tk, 1, a.Hk, hk, a.D);
    // the first row that sees key j0
    const int64_t first = a.causal ? (j0 > t.tk - t.tq ? (j0 - (t.tk - t.tq)) * a.G : 0) : 0;
    const Part part(first < rows ? (rows - first + kB - 1) / kB : 0);
    float dk[DP / 8][4], dv[DP / 8][4];
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) dk[n][e] = dv[n][e] = 0.f;
    const float sc = a.scale * kLog2e;
    for (int64_t i = part.beg; i < part.end; ++i) {
        const int64_t r0 = first + i * kB;
        __syncthreads();
        copy_rows<DP>(sq, static_cast<const float *>(a.q), t.q0, r0, rows, a.G, a.H, hk, a.D);
        copy_rows<DP>(sd, static_cast<const float *>(a.dout), t.q0, r0, rows, a.G, a.H, hk, a.D);
        copies_commit();
        if (threadIdx.x < 2 * kB) {
            const int64_t r = r0 + (threadIdx.x & (kB - 1));
            float x = 0.f;
            if (r < rows) {
                const int64_t at = row_offset(t.q0, r, a.G, a.H, hk);
                x = threadIdx.x < kB ? lse_log2(a.lse_in[at]) : a.delta[at];
            }
            srow[threadIdx.x] = x;
        }
        copies_wait<0>();
        __syncthreads();
        float s[4][4] = {}, dp[4][4] = {};  // rows: keys 16 wr .., columns: rows 32 wc ..
        scores<DP>(s, sk, sq, 16 * wr, 32 * wc, nk, lane);
        scores<DP>(dp, sv, sd, 16 * wr, 32 * wc, nk, lane);
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c = 32 * wc + 8 * n + 2 * (lane & 3) + e;
                const int64_t lim = key_limit(a, t, r0 + c, t.tk) - j0 - 16 * wr - (lane >> 2);
                const float lse = srow[c], delta = srow[kB + c];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool seen = 8 * h < lim;
                    const float p = seen ? exp2f(s[n][2 * h + e] * sc - lse) : 0.f;
                    s[n][2 * h + e] = p;
                    dp[n][2 * h + e] = seen ? p * (dp[n][2 * h + e] - delta) : 0.f;
                }
            }
        weighted<DP>(dv, s, sd, 32 * wc, nk, lane);
        weighted<DP>(dk, dp, sq, 32 * wc, nk, lane);
    }
    copies_wait<0>();
    __syncthreads();
    if (wc == 1) {
        put_acc<DP>(sq, dk, 16 * wr, a.scale, a.scale, false, lane);
        put_acc<DP>(sd, dv, 16 * wr, 1.f, 1.f, false, lane);
    }
    __syncthreads();
    if (wc == 0) {
        put_acc<DP>(sq, dk, 16 * wr, a.scale, a.scale, true, lane);
        put_acc<DP>(sd, dv, 16 * wr, 1.f, 1.f, true, lane);
    }
    cluster_meet(part.cs);
    for (int i = part.rank * kThreads + threadIdx.x; i < kB * (DP / 4); i += part.cs * kThreads) {
        const int r = i / (DP / 4), c = (i - r * (DP / 4)) * 4;
        if (j0 + r >= t.tk || c >= a.D) continue;
        const int64_t off = ((t.k0 + j0 + r) * a.Hk + hk) * a.D + c;
        *reinterpret_cast<float4 *>(static_cast<float *>(a.dk) + off) = cluster_sum(sq + r * S + c, part.cs);
        *reinterpret_cast<float4 *>(static_cast<float *>(a.dv) + off) = cluster_sum(sd + r * S + c, part.cs);
    }
    cluster_meet(part.cs);  // everyone's shared memory has been read
}

// 64 packed rows: dq over every key they see.
template <int DP>
__global__ void __launch_bounds__(kThreads, DP <= 64 ? 2 : 1) attn_dq_tf32_kernel(AttnArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int S = Stride<DP>::value, T = kB * S;
    float *sq = sm, *sd = sq + T, *sk = sd + T, *sv = sk + T;
    AttnTile t;
    const int hk = blockIdx.y;
    if (!attn_locate(a, true, blockIdx.x / cg::this_cluster().num_blocks(), a.G, kB, t)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wr = warp & 3, wc = warp >> 2;
    const int64_t rows = t.tq * a.G;
    const int nk = (a.D + 7) / 8;
    copy_rows<DP>(sq, static_cast<const float *>(a.q), t.q0, t.row0, rows, a.G, a.H, hk, a.D);
    copy_rows<DP>(sd, static_cast<const float *>(a.dout), t.q0, t.row0, rows, a.G, a.H, hk, a.D);
    int64_t lim[2];
    float lse[2], delta[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t r = t.row0 + 16 * wr + 8 * h + (lane >> 2);
        lim[h] = key_limit(a, t, r, t.tk);
        const int64_t at = r < rows ? row_offset(t.q0, r, a.G, a.H, hk) : 0;
        lse[h] = r < rows ? lse_log2(a.lse_in[at]) : 0.f;
        delta[h] = r < rows ? a.delta[at] : 0.f;
    }
    const int64_t seen = key_limit(a, t, min64(t.row0 + kB, rows) - 1, t.tk);
    const Part part(seen > 0 ? (seen + kB - 1) / kB : 0);
    float dq[DP / 8][4];
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) dq[n][e] = 0.f;
    const float sc = a.scale * kLog2e;
    for (int64_t j0 = part.beg * kB; j0 < part.end * kB; j0 += kB) {
        __syncthreads();
        copy_rows<DP>(sk, static_cast<const float *>(a.k), t.k0, j0, t.tk, 1, a.Hk, hk, a.D);
        copy_rows<DP>(sv, static_cast<const float *>(a.v), t.k0, j0, t.tk, 1, a.Hk, hk, a.D);
        copies_commit();
        copies_wait<0>();
        __syncthreads();
        float s[4][4] = {}, dp[4][4] = {};
        scores<DP>(s, sq, sk, 16 * wr, 32 * wc, nk, lane);
        scores<DP>(dp, sd, sv, 16 * wr, 32 * wc, nk, lane);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t left = lim[h] - j0 - 32 * wc - 2 * (lane & 3);
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &x = s[n][2 * h + e];
                    x = 8 * n + e < left ? exp2f(x * sc - lse[h]) * (dp[n][2 * h + e] - delta[h]) : 0.f;
                }
        }
        weighted<DP>(dq, s, sk, 32 * wc, nk, lane);
    }
    copies_wait<0>();
    __syncthreads();
    if (wc == 1) put_acc<DP>(sq, dq, 16 * wr, a.scale, a.scale, false, lane);
    __syncthreads();
    if (wc == 0) put_acc<DP>(sq, dq, 16 * wr, a.scale, a.scale, true, lane);
    cluster_meet(part.cs);
    for (int i = part.rank * kThreads + threadIdx.x; i < kB * (DP / 4); i += part.cs * kThreads) {
        const int r = i / (DP / 4), c = (i - r * (DP / 4)) * 4;
        if (t.row0 + r >= rows || c >= a.D) continue;
        *reinterpret_cast<float4 *>(static_cast<float *>(a.dq) + row_offset(t.q0, t.row0 + r, a.G, a.H, hk) * a.D + c) =
            cluster_sum(sq + r * S + c, part.cs);
    }
    cluster_meet(part.cs);  // everyone's shared memory has been read
}

// One warp a row (token, head): delta = sum_d do o.  HBM bound (reads do and o once).
__global__ void attn_delta_kernel(const float *__restrict__ dout, const float *__restrict__ o, float *__restrict__ delta,
                                  int64_t rows, int D) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t r = blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5); r < rows; r += warps) {
        float acc = 0.f;
        if (4 * lane < D) {  // D is a multiple of 8, at most 128
            const float4 x = *reinterpret_cast<const float4 *>(dout + r * D + 4 * lane);
            const float4 y = *reinterpret_cast<const float4 *>(o + r * D + 4 * lane);
            acc = x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
        }
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, x);
        if (lane == 0) delta[r] = acc;
    }
}

// CTAs a tile: as many as leave every SM at most two, and each at least two tiles of the other
// side (`other` rows or keys, on average).
int cluster_size(int64_t ctas, int64_t other) {
    int cs = 1;
    while (cs < kMaxCluster && ctas * cs * 2 <= 2 * 148 && other >= 4 * kB * cs) cs *= 2;
    return cs;
}

template <typename F>
cudaError_t launch(F kern, dim3 grid, int cs, size_t smem, const AttnArgs &a, cudaStream_t st,
                   std::atomic<uint64_t> &done) {
    if (grid.x == 0) return cudaSuccess;
    const cudaError_t e = allow_smem(kern, smem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid.x * cs, grid.y, grid.z);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

// 0: forward, 1: dk dv, 2: dq
template <int DP>
cudaError_t launch_part(int part, const AttnArgs &a, cudaStream_t st) {
    static std::atomic<uint64_t> done[3];
    const size_t tile = (size_t)kB * Stride<DP>::value;
    const int64_t nq = attn_slots(a.sq, a.N, a.G, kB), nk = attn_slots(a.sk, a.N, 1, kB);
    const int64_t rows = (a.sq.cu ? a.sq.T / a.N : a.sq.T) * a.G, keys = a.sk.cu ? a.sk.T / a.N : a.sk.T;
    if (std::max(nq, nk) >= (int64_t)1 << 28) return cudaErrorInvalidValue;  // times 8 CTAs: past the grid's limit
    const dim3 gq((unsigned)nq, a.Hk, part == 0 ? a.nsplit : 1), gk((unsigned)nk, a.Hk);
    if (part == 0)
        return launch(attn_fwd_tf32_kernel<DP>, gq, cluster_size(nq * a.Hk * a.nsplit, std::min(keys, a.split)),
                      sizeof(float) * (5 * tile + (4 + 2 + kMaxCluster + 1) * kB), a, st, done[0]);
    if (part == 1)
        return launch(attn_dkdv_tf32_kernel<DP>, gk, cluster_size(nk * a.Hk, rows), sizeof(float) * (4 * tile + 2 * kB), a,
                      st, done[1]);
    return launch(attn_dq_tf32_kernel<DP>, gq, cluster_size(nq * a.Hk, keys), sizeof(float) * 4 * tile, a, st, done[2]);
}

// column width of the tiles: D rounded up to a multiple of 32
cudaError_t launch_width(int part, const AttnArgs &a, cudaStream_t st) {
    switch ((a.D + 31) / 32) {
        case 1: return launch_part<32>(part, a, st);
        case 2: return launch_part<64>(part, a, st);
        case 3: return launch_part<96>(part, a, st);
        default: return launch_part<128>(part, a, st);
    }
}

}  // namespace

cudaError_t launch_attn_fwd_tf32(const AttnArgs &a, cudaStream_t st) { return launch_width(0, a, st); }
cudaError_t launch_attn_bwd_dkdv_tf32(const AttnArgs &a, cudaStream_t st) { return launch_width(1, a, st); }
cudaError_t launch_attn_bwd_dq_tf32(const AttnArgs &a, cudaStream_t st) { return launch_width(2, a, st); }

cudaError_t launch_attn_delta(const AttnArgs &a, cudaStream_t st) {
    const int64_t rows = (a.sq.cu ? a.sq.T : a.N * a.sq.T) * a.H;
    if (rows == 0) return cudaSuccess;
    const unsigned grid = (unsigned)std::min<int64_t>((rows + 7) / 8, 148 * 16);
    attn_delta_kernel<<<grid, 256, 0, st>>>(static_cast<const float *>(a.dout), static_cast<const float *>(a.o), a.delta,
                                            rows, a.D);
    return cudaGetLastError();
}

}  // namespace sgla
