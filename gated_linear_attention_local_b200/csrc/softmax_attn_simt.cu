// Softmax attention on the CUDA cores, for fp32 operands: forward, dk / dv, dq and the row
// sums delta.  64 x 64 tiles of scores, 256 threads, a 4 x 4 piece of the tile per thread
// (rows 4 ty + i, columns tx + 16 j), fp32 FMA throughout.
//
// Forward: the running maximum m and sum l of a row (log2 units) live in the registers of the
// 16 threads that share it; o is rescaled by 2^(m_old - m_new) when the maximum moves.
// Backward: the probabilities are recomputed, p = 2^(s - lse); with delta_i = sum_d do o,
//   dv_j = sum_i p_ij do_i,  ds_ij = p_ij (do_i . v_j - delta_i),
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,
// in two passes, one per output side, so that every sum has one owner and one order.
//
// Bound: FFMA issue and shared-memory bandwidth (a 4 x 4 piece reads 8 vectors of 16 bytes
// for 64 FMAs).
#include <math.h>

#include <algorithm>

#include "softmax_attn.h"

namespace sgla {
namespace {

constexpr int kB = 64;            // tile edge
constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Row stride of a [64][DP] tile: 16-byte reads of rows tx + 16 j by 16 threads fall on
// different banks (stride 4 words modulo 32).
template <int DP>
struct Stride {
    static constexpr int value = DP + 4;
};
constexpr int kPS = kB + 4;  // row stride of a [64][64] tile

// Where packed row r of key head hk lies in a [tokens, H, D] tensor.
__device__ __forceinline__ int64_t row_offset(int64_t tok0, int64_t r, int G, int H, int hk) {
    const int64_t t = r / G;
    return (tok0 + t) * H + hk * G + (int)(r - t * G);
}

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

// rows [r0, r0 + 64) of one side into a tile, zeros past `rows` and past column D
template <int DP>
__device__ __forceinline__ void load_rows(float *tile, const float *src, int64_t tok0, int64_t r0, int64_t rows, int G,
                                          int H, int hk, int D) {
    constexpr int NV = DP / 4;
    for (int i = threadIdx.x; i < kB * NV; i += kThreads) {
        const int r = i / NV, c = (i - r * NV) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < rows && c < D)
            x = load4(src + row_offset(tok0, r0 + r, G, H, hk) * D + c);
        *reinterpret_cast<float4 *>(tile + r * Stride<DP>::value + c) = x;
    }
}

// acc[i][j] += A[4 ty + i][:] . B[tx + 16 j][:]
template <int DP>
__device__ __forceinline__ void dot_rows(const float *A, const float *B, int ty, int tx, float (&acc)[4][4]) {
    constexpr int S = Stride<DP>::value;
#pragma unroll 4
    for (int c = 0; c < DP; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(A + (4 * ty + i) * S + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * S + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
                acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
                acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
                acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
            }
    }
}

// acc[i][2 c + e] += sum_s W[4 ty + i][s] X[s][2 tx + 32 c + e]  (W rows of stride kPS)
template <int DP>
__device__ __forceinline__ void mul_rows(const float *W, const float *X, int ty, int tx, float (&acc)[4][DP / 16]) {
    constexpr int S = Stride<DP>::value;
#pragma unroll 2
    for (int s = 0; s < kB; s += 4) {
        float w[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = *reinterpret_cast<const float4 *>(W + (4 * ty + i) * kPS + s);
            w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {
                const float2 x = *reinterpret_cast<const float2 *>(X + (s + e) * S + 2 * tx + 32 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[i][2 * c] = fmaf(w[i][e], x.x, acc[i][2 * c]);
                    acc[i][2 * c + 1] = fmaf(w[i][e], x.y, acc[i][2 * c + 1]);
                }
            }
    }
}

// First key that row r of the tile must not see (keys [0, limit) are seen).
__device__ __forceinline__ int64_t key_limit(const AttnArgs &a, const AttnTile &t, int64_t r, int64_t k_end) {
    if (r >= t.tq * a.G) return 0;
    return a.causal ? min64(k_end, r / a.G + 1 + t.tk - t.tq) : k_end;
}

template <int DP>
__global__ void __launch_bounds__(kThreads) attn_fwd_simt_kernel(AttnArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int S = Stride<DP>::value, NC = DP / 16;
    float *sq = sm, *sk = sq + kB * S, *sv = sk + kB * S, *sp = sv + kB * S;
    AttnTile t;
    const int hk = blockIdx.y;
    if (!attn_locate(a, true, blockIdx.x, a.G, kB, t)) return;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t rows = t.tq * a.G;
    const int64_t kb = blockIdx.z * a.split, ke = min64(t.tk, kb + a.split);
    load_rows<DP>(sq, static_cast<const float *>(a.q), t.q0, t.row0, rows, a.G, a.H, hk, a.D);
    int64_t lim[4];
    int64_t last = 0;  // keys that some row of the tile sees
#pragma unroll
    for (int i = 0; i < 4; ++i) lim[i] = key_limit(a, t, t.row0 + 4 * ty + i, ke);
    last = key_limit(a, t, min64(t.row0 + kB, rows) - 1, ke);
    float m[4], l[4], o[4][NC];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) o[i][c] = 0.f;
    }
    const float sc = a.scale * kLog2e;
    for (int64_t j0 = kb; j0 < last; j0 += kB) {
        __syncthreads();
        load_rows<DP>(sk, static_cast<const float *>(a.k), t.k0, j0, t.tk, 1, a.Hk, hk, a.D);
        load_rows<DP>(sv, static_cast<const float *>(a.v), t.k0, j0, t.tk, 1, a.Hk, hk, a.D);
        __syncthreads();
        float s[4][4] = {};
        dot_rows<DP>(sq, sk, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float top = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = (j0 + tx + 16 * j < lim[i]) ? s[i][j] * sc : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
#pragma unroll
            for (int x = 8; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float base = top == -INFINITY ? 0.f : top;
            const float f = exp2f(m[i] - base);  // 0 while nothing was seen
            m[i] = top;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - base);
                sum += p;
                sp[(4 * ty + i) * kPS + tx + 16 * j] = p;
            }
            l[i] = l[i] * f + sum;
#pragma unroll
            for (int c = 0; c < NC; ++c) o[i][c] *= f;
        }
        __syncthreads();
        mul_rows<DP>(sp, sv, ty, tx, o);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int x = 8; x >= 1; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
        const int64_t r = t.row0 + 4 * ty + i;
        if (r >= rows) continue;
        const int64_t row = row_offset(t.q0, r, a.G, a.H, hk);
        const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
        const float lse = l[i] > 0.f ? (m[i] + log2f(l[i])) * kLn2 : (l[i] == 0.f ? -INFINITY : l[i]);
        const bool nan = !(l[i] >= 0.f);  // NaN scores: NaN, not the zeros of an empty row
        const int64_t pr = (int64_t)blockIdx.z * a.part_rows + row;
        if (a.part_o) {
            if (tx == 0) a.part_lse[pr] = lse;
            if (l[i] == 0.f) continue;  // the join reads no o of an empty part
        } else if (tx == 0 && a.lse) {
            a.lse[row] = lse;
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = 2 * tx + 32 * (c >> 1) + (c & 1);
            if (col >= a.D) continue;
            const float x = nan ? l[i] : o[i][c] * inv;
            if (a.part_o) a.part_o[pr * a.D + col] = x;
            else static_cast<float *>(a.o)[row * a.D + col] = x;
        }
    }
}

// One key tile (64 keys of one key head): dk, dv over every row that sees it.
template <int DP>
__global__ void __launch_bounds__(kThreads) attn_bwd_dkdv_simt_kernel(AttnArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int S = Stride<DP>::value, NC = DP / 16;
    float *sk = sm, *sv = sk + kB * S, *sq = sv + kB * S, *sd = sq + kB * S, *sp = sd + kB * S, *ss = sp + kB * kPS;
    float *slse = ss + kB * kPS, *sdelta = slse + kB;
    AttnTile t;
    const int hk = blockIdx.y;
    if (!attn_locate(a, false, blockIdx.x, 1, kB, t)) return;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t rows = t.tq * a.G, j0 = t.row0;
    load_rows<DP>(sk, static_cast<const float *>(a.k), t.k0, j0, t.tk, 1, a.Hk, hk, a.D);
    load_rows<DP>(sv, static_cast<const float *>(a.v), t.k0, j0, t.tk, 1, a.Hk, hk, a.D);
    // the first row that sees key j0
    const int64_t first = a.causal ? (j0 > t.tk - t.tq ? (j0 - (t.tk - t.tq)) * a.G : 0) : 0;
    float dk[4][NC] = {}, dv[4][NC] = {};
    const float sc = a.scale * kLog2e;
    for (int64_t r0 = first; r0 < rows; r0 += kB) {
        __syncthreads();
        load_rows<DP>(sq, static_cast<const float *>(a.q), t.q0, r0, rows, a.G, a.H, hk, a.D);
        load_rows<DP>(sd, static_cast<const float *>(a.dout), t.q0, r0, rows, a.G, a.H, hk, a.D);
        if (threadIdx.x < kB) {
            const int64_t r = r0 + threadIdx.x;
            const int64_t row = r < rows ? row_offset(t.q0, r, a.G, a.H, hk) : 0;
            slse[threadIdx.x] = r < rows ? a.lse_in[row] * kLog2e : 0.f;
            sdelta[threadIdx.x] = r < rows ? a.delta[row] : 0.f;
        }
        __syncthreads();
        float s[4][4] = {}, dp[4][4] = {};
        dot_rows<DP>(sq, sk, ty, tx, s);
        dot_rows<DP>(sd, sv, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ri = 4 * ty + i;
            const int64_t lim = key_limit(a, t, r0 + ri, t.tk);
            const float lse = slse[ri], delta = sdelta[ri];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = (j0 + tx + 16 * j < lim) ? exp2f(s[i][j] * sc - lse) : 0.f;
                // transposed: row = key, column = query row
                sp[(tx + 16 * j) * kPS + ri] = p;
                ss[(tx + 16 * j) * kPS + ri] = (j0 + tx + 16 * j < lim) ? p * (dp[i][j] - delta) : 0.f;
            }
        }
        __syncthreads();
        mul_rows<DP>(sp, sd, ty, tx, dv);
        mul_rows<DP>(ss, sq, ty, tx, dk);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t j = j0 + 4 * ty + i;
        if (j >= t.tk) continue;
        const int64_t off = ((t.k0 + j) * a.Hk + hk) * a.D;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = 2 * tx + 32 * (c >> 1) + (c & 1);
            if (col >= a.D) continue;
            static_cast<float *>(a.dk)[off + col] = dk[i][c] * a.scale;
            static_cast<float *>(a.dv)[off + col] = dv[i][c];
        }
    }
}

// One query tile: dq over every key its rows see.
template <int DP>
__global__ void __launch_bounds__(kThreads) attn_bwd_dq_simt_kernel(AttnArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int S = Stride<DP>::value, NC = DP / 16;
    float *sq = sm, *sd = sq + kB * S, *sk = sd + kB * S, *sv = sk + kB * S, *ss = sv + kB * S;
    AttnTile t;
    const int hk = blockIdx.y;
    if (!attn_locate(a, true, blockIdx.x, a.G, kB, t)) return;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t rows = t.tq * a.G;
    load_rows<DP>(sq, static_cast<const float *>(a.q), t.q0, t.row0, rows, a.G, a.H, hk, a.D);
    load_rows<DP>(sd, static_cast<const float *>(a.dout), t.q0, t.row0, rows, a.G, a.H, hk, a.D);
    int64_t lim[4];
    float lse[4], delta[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = t.row0 + 4 * ty + i;
        lim[i] = key_limit(a, t, r, t.tk);
        const int64_t row = r < rows ? row_offset(t.q0, r, a.G, a.H, hk) : 0;
        lse[i] = r < rows ? a.lse_in[row] * kLog2e : 0.f;
        delta[i] = r < rows ? a.delta[row] : 0.f;
    }
    const int64_t last = key_limit(a, t, min64(t.row0 + kB, rows) - 1, t.tk);
    float dq[4][NC] = {};
    const float sc = a.scale * kLog2e;
    for (int64_t j0 = 0; j0 < last; j0 += kB) {
        __syncthreads();
        load_rows<DP>(sk, static_cast<const float *>(a.k), t.k0, j0, t.tk, 1, a.Hk, hk, a.D);
        load_rows<DP>(sv, static_cast<const float *>(a.v), t.k0, j0, t.tk, 1, a.Hk, hk, a.D);
        __syncthreads();
        float s[4][4] = {}, dp[4][4] = {};
        dot_rows<DP>(sq, sk, ty, tx, s);
        dot_rows<DP>(sd, sv, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                ss[(4 * ty + i) * kPS + tx + 16 * j] =
                    (j0 + tx + 16 * j < lim[i]) ? exp2f(s[i][j] * sc - lse[i]) * (dp[i][j] - delta[i]) : 0.f;
        __syncthreads();
        mul_rows<DP>(ss, sk, ty, tx, dq);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = t.row0 + 4 * ty + i;
        if (r >= rows) continue;
        const int64_t off = row_offset(t.q0, r, a.G, a.H, hk) * a.D;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = 2 * tx + 32 * (c >> 1) + (c & 1);
            if (col < a.D) static_cast<float *>(a.dq)[off + col] = dq[i][c] * a.scale;
        }
    }
}

// One warp a row (token, head): delta = sum_d do o.  HBM bound (reads do and o once).
__global__ void attn_delta_kernel(const float *__restrict__ dout, const float *__restrict__ o, float *__restrict__ delta,
                                  int64_t rows, int D) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t r = blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5); r < rows; r += warps) {
        float acc = 0.f;
        if (4 * lane < D) {  // D is a multiple of 8, at most 128
            const float4 x = load4(dout + r * D + 4 * lane), y = load4(o + r * D + 4 * lane);
            acc = x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
        }
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, x);
        if (lane == 0) delta[r] = acc;
    }
}

template <int DP>
size_t smem_bytes(int tiles, int squares) {
    return sizeof(float) * ((size_t)tiles * kB * Stride<DP>::value + (size_t)squares * kB * kPS + 2 * kB);
}

template <typename F>
cudaError_t launch(F kern, dim3 grid, size_t smem, const AttnArgs &a, cudaStream_t st) {
    if (grid.x == 0) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<grid, kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

// 0: forward, 1: dk dv, 2: dq
template <int DP>
cudaError_t launch_part(int part, const AttnArgs &a, cudaStream_t st) {
    const dim3 gq((unsigned)attn_slots(a.sq, a.N, a.G, kB), a.Hk, part == 0 ? a.nsplit : 1);
    const dim3 gk((unsigned)attn_slots(a.sk, a.N, 1, kB), a.Hk);
    if (part == 0) return launch(attn_fwd_simt_kernel<DP>, gq, smem_bytes<DP>(3, 1), a, st);
    if (part == 1) return launch(attn_bwd_dkdv_simt_kernel<DP>, gk, smem_bytes<DP>(4, 2), a, st);
    return launch(attn_bwd_dq_simt_kernel<DP>, gq, smem_bytes<DP>(4, 1), a, st);
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

cudaError_t launch_attn_fwd_simt(const AttnArgs &a, cudaStream_t st) {
    return launch_width(0, a, st);
}
cudaError_t launch_attn_bwd_dkdv_simt(const AttnArgs &a, cudaStream_t st) {
    return launch_width(1, a, st);
}
cudaError_t launch_attn_bwd_dq_simt(const AttnArgs &a, cudaStream_t st) {
    return launch_width(2, a, st);
}

cudaError_t launch_attn_delta(const AttnArgs &a, cudaStream_t st) {
    const int64_t rows = (a.sq.cu ? a.sq.T : a.N * a.sq.T) * a.H;
    if (rows == 0) return cudaSuccess;
    const unsigned grid = (unsigned)std::min<int64_t>((rows + 7) / 8, 148 * 16);
    attn_delta_kernel<<<grid, 256, 0, st>>>(static_cast<const float *>(a.dout), static_cast<const float *>(a.o), a.delta,
                                            rows, a.D);
    return cudaGetLastError();
}

}  // namespace sgla
