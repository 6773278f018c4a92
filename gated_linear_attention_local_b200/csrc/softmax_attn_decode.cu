// One token of softmax attention for each of N sequences, at most 16 query heads to a key head.
//
// Bound: HBM (every valid key and value is read once and used by G rows only), so the kernel is
// built around the stream.  A cluster of up to 8 CTAs takes one (sequence, key head) and cuts its
// valid keys evenly (the length is read on the device: no split is empty while others wait);
// each of a CTA's four warps pulls every fourth tile of 16 keys through its own ring of TMA
// copies and keeps its own maximum, sum and output, with no barrier between warps until the end.
// Then all warps of the cluster are joined through distributed shared memory, with the parts of
// a shared prefix (computed before for the whole batch) as further terms, so a step needs one
// launch besides the prefix's.
//   join: o = sum_p w_p o_p / sum_p w_p l_p, w_p = 2^(m_p - max m), parts in a fixed order.
//
// bf16: mma.sync m16n8k16, the G rows padded to 16 (tcgen05 has no tile below 64 rows; the
// products are 1/10 of the time the stream takes).  The scores' accumulators are the second
// product's A operand as they stand.  p is rounded to bf16 for that product.
// fp32: FMA on the CUDA cores; two lanes a key for the scores, a lane four (two) columns of v.
//
// Measured (bf16, 32 heads of 128 on 8; cold L2, less the 5 us that an empty pair of events reads): 128
// caches of up to 4096 tokens (1.08 GB) 170 to 182 us, 91 to 97 % of the measured copy rate; 64 caches
// of up to 512 tokens 26 us behind a prefix, where a CTA's fixed cost (some 5 us) and the join of the
// prefix's parts outweigh the 10 us of the stream.
//
// Keys behind the valid length may hold anything: scores there are -inf, and the value rows of
// the last tile are zeroed in shared memory (0 * NaN must not arise).
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>
#include <utility>

#include "softmax_attn.h"
#include "softmax_attn_map.h"
#include "tc_ptx.cuh"
#include "tc_tiles.cuh"

namespace sgla {

using namespace tc;
namespace cg = cooperative_groups;

namespace {

constexpr int kWarps = 4, kKeys = 16, kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.f;

template <typename T, int DP>
struct DecCfg {
    static constexpr int COLS = 128 / sizeof(T);            // columns of a 128-byte row
    static constexpr int NR = DP / COLS;                    // 128-byte regions of a row
    static constexpr uint32_t REG = kKeys * 128;            // region bytes
    static constexpr uint32_t TILE = NR * REG;              // K or V tile
    static constexpr uint32_t STAGE = 2 * TILE;
    // 24 KB a warp, two CTAs an SM; fp32 with DP = 128 needs 48 KB for three stages
    static constexpr int STAGES = 24576 / STAGE > 3 ? 24576 / STAGE : 3;
    static constexpr uint32_t RING = STAGES * STAGE;        // one warp's ring
    static constexpr uint32_t ML = kWarps * RING;           // [kWarps][16][2]: m, l of the warps
    static constexpr uint32_t QS = ML + kWarps * 16 * 2 * 4;  // fp32: [16][DP] floats q
    static constexpr uint32_t PS = QS + (sizeof(T) == 4 ? 16 * DP * 4 : 0);   // fp32: [kWarps][16][16] p
    static constexpr uint32_t BARS = PS + (sizeof(T) == 4 ? kWarps * 16 * 16 * 4 : 0);
    static constexpr size_t SMEM = BARS + kWarps * STAGES * 8 + 16 + 1024;
    // at the end a warp leaves its output, [16][DP] floats, at the head of its ring; behind those
    // of warps 0 and 1 lie the weights of all parts
    static constexpr uint32_t TAIL = 16 * DP * 4;
    static_assert(TAIL + 16 * 4 * (kMaxCluster * kWarps + kDecodeMaxParts) <= RING, "output and weights fit a ring");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The running softmax and output of one warp over its tiles.  GM: rows kept (fp32 only).
template <typename T, int DP, int GM>
struct Rows;

template <int DP, int GM>
struct Rows<__nv_bfloat16, DP, GM> {
    // lane: rows lane / 4 and lane / 4 + 8; score columns 2 (lane % 4) + {0, 1} of each 8 keys
    uint32_t q[DP / 16][4];
    float o[DP / 8][4];
    float m[2], l[2];

    __device__ void init(const AttnArgs &a, const __nv_bfloat16 *qrow, unsigned char *, int lane) {
        const int r = lane >> 2, c = 2 * (lane & 3);
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = r + 8 * (e & 1), col = 16 * kk + c + 8 * (e >> 1);
                q[kk][e] = (row < a.G && col < a.D) ? *reinterpret_cast<const uint32_t *>(qrow + row * a.D + col) : 0u;
            }
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }

    // one tile of 16 keys, the first `valid` of them seen
    __device__ void tile(const AttnArgs &a, unsigned char *kt, unsigned char *vt, unsigned char *, int valid, float sc,
                         int lane) {
        using C = DecCfg<__nv_bfloat16, DP>;
        float s[2][4] = {};
        {
            const int key = (lane & 7) + ((lane >> 4) << 3);
            const uint32_t base = smem_u32(kt) + key * 128;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
                const int ch = 2 * kk + ((lane >> 3) & 1);
                uint32_t b[4];
                ldsm4(base + (ch >> 3) * C::REG + (((ch ^ key) & 7) << 4), b);
                mma16816(s[0], q[kk], b[0], b[1]);
                mma16816(s[1], q[kk], b[2], b[3]);
            }
        }
        if (valid < kKeys) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (8 * n + 2 * (lane & 3) + (e & 1) >= valid) s[n][e] = -INFINITY;
        }
        float top[2];
        bool grown = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            top[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
            grown |= (top[h] - m[h]) * sc > kGrow;
        }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float to = fmaxf(m[h], top[h]);
                const float f = to == -INFINITY ? 1.f : fast_exp2((m[h] - to) * sc);
                m[h] = to;
                l[h] *= f;
#pragma unroll
                for (int n = 0; n < DP / 8; ++n) {
                    o[n][2 * h] *= f;
                    o[n][2 * h + 1] *= f;
                }
            }
        }
        uint32_t p[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float base = m[h] == -INFINITY ? 0.f : m[h];  // (the difference first: m sc rounds, and may be huge)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float x = fast_exp2((s[n][2 * h] - base) * sc), y = fast_exp2((s[n][2 * h + 1] - base) * sc);
                l[h] += x + y;
                p[2 * n + h] = pack_bf16(x, y);
            }
        }
        {
            const int key = (lane & 7) + ((lane >> 3) & 1) * 8;
            const uint32_t base = smem_u32(vt) + key * 128;
#pragma unroll
            for (int n = 0; n < DP / 16; ++n) {
                const int ch = 2 * n + (lane >> 4);
                uint32_t b[4];
                ldsm4_t(base + (ch >> 3) * C::REG + (((ch ^ key) & 7) << 4), b);
                mma16816(o[2 * n], p, b[0], b[1]);
                mma16816(o[2 * n + 1], p, b[2], b[3]);
            }
        }
    }

    // m (log2 units), l to ml[16][2], o to out[16][DP]
    __device__ void leave(float *out, float *ml, float sc, int lane) {
        const int r = lane >> 2, c = 2 * (lane & 3);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if ((lane & 3) == 0) {
                ml[2 * (r + 8 * h)] = m[h] == -INFINITY ? -INFINITY : m[h] * sc;
                ml[2 * (r + 8 * h) + 1] = l[h];
            }
#pragma unroll
            for (int n = 0; n < DP / 8; ++n)
                *reinterpret_cast<float2 *>(out + (r + 8 * h) * DP + 8 * n + c) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
        }
    }
};

template <int DP, int GM>
struct Rows<float, DP, GM> {
    // scores: lanes key, key + 16 take the even and odd 16-byte chunks of a key; output: a lane
    // CL columns from CL * lane.  m, l: the same in every lane.
    static constexpr int CL = DP / 32;
    float o[GM][CL];
    float m[GM], l[GM];

    __device__ void init(const AttnArgs &a, const float *qrow, unsigned char *qs, int lane) {
        float *q = reinterpret_cast<float *>(qs);  // every warp writes the same values
        for (int i = lane; i < GM * DP; i += 32) {
            const int g = i / DP, c = i - g * DP;
            q[i] = (g < a.G && c < a.D) ? qrow[g * a.D + c] : 0.f;
        }
        __syncwarp();
#pragma unroll
        for (int g = 0; g < GM; ++g) {
            m[g] = -INFINITY;
            l[g] = 0.f;
#pragma unroll
            for (int c = 0; c < CL; ++c) o[g][c] = 0.f;
        }
    }

    __device__ void tile(const AttnArgs &a, unsigned char *kt, unsigned char *vt, unsigned char *qs, int valid, float sc,
                         int lane) {
        using C = DecCfg<float, DP>;
        const float *q = reinterpret_cast<const float *>(qs);
        float *ps = reinterpret_cast<float *>(qs + (C::PS - C::QS)) + (threadIdx.x >> 5) * 256;  // [16 keys][16 rows]
        const int key = lane & 15;
        float s[GM] = {};
#pragma unroll 4
        for (int ch = lane >> 4; ch < DP / 4; ch += 2) {
            const float4 k4 = *reinterpret_cast<const float4 *>(kt + (ch >> 3) * C::REG + key * 128 + (((ch ^ key) & 7) << 4));
#pragma unroll
            for (int g = 0; g < GM; ++g) {
                const float4 q4 = *reinterpret_cast<const float4 *>(q + g * DP + 4 * ch);
                s[g] = fmaf(q4.x, k4.x, s[g]);
                s[g] = fmaf(q4.y, k4.y, s[g]);
                s[g] = fmaf(q4.z, k4.z, s[g]);
                s[g] = fmaf(q4.w, k4.w, s[g]);
            }
        }
        __syncwarp();  // the previous tile's p have been read
#pragma unroll
        for (int g = 0; g < GM; ++g) {
            float x = s[g] + __shfl_xor_sync(0xffffffffu, s[g], 16);
            x = key < valid ? x * sc : -INFINITY;
            float top = x;
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            top = fmaxf(top, m[g]);
            const float base = top == -INFINITY ? 0.f : top;
            const float f = exp2f(m[g] - base);
            m[g] = top;
            const float p = exp2f(x - base);
            float sum = p;
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            l[g] = l[g] * f + sum;
#pragma unroll
            for (int c = 0; c < CL; ++c) o[g][c] *= f;
            if (lane < 16) ps[key * 16 + g] = p;
        }
        __syncwarp();
        const int col = CL * lane, ch = col >> 2;
#pragma unroll 4
        for (int k = 0; k < kKeys; ++k) {
            const unsigned char *v = vt + (ch >> 3) * C::REG + k * 128 + (((ch ^ k) & 7) << 4) + (col & 3) * 4;
            float x[CL];
            if constexpr (CL == 4) {
                const float4 v4 = *reinterpret_cast<const float4 *>(v);
                x[0] = v4.x; x[1] = v4.y; x[2] = v4.z; x[3] = v4.w;
            } else {
                const float2 v2 = *reinterpret_cast<const float2 *>(v);
                x[0] = v2.x; x[1] = v2.y;
            }
#pragma unroll
            for (int g = 0; g < GM; ++g) {
                const float p = ps[k * 16 + g];
#pragma unroll
                for (int c = 0; c < CL; ++c) o[g][c] = fmaf(p, x[c], o[g][c]);
            }
        }
    }

    __device__ void leave(float *out, float *ml, float, int lane) {
#pragma unroll
        for (int g = 0; g < GM; ++g) {
            if (lane == 0) {
                ml[2 * g] = m[g];
                ml[2 * g + 1] = l[g];
            }
#pragma unroll
            for (int c = 0; c < CL; ++c) out[g * DP + CL * lane + c] = o[g][c];
        }
    }
};

template <typename T, int DP, int GM>
__global__ void __launch_bounds__(32 * kWarps)
attn_decode_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, AttnArgs a,
                   int pparts) {
    using C = DecCfg<T, DP>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = align1024(smem_raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int cs = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int64_t unit = blockIdx.x / cs;
    const int hk = (int)(unit % a.Hk);
    const int64_t n = unit / a.Hk;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
    }
    int64_t len = a.sk.len[n];
    if (len < 0 || len > a.sk.T) {  // counts as empty
        if (a.status && threadIdx.x == 0) atomicExch(a.status, kDevBadCuSeqlens);
        len = 0;
    }
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + C::BARS) + warp * C::STAGES;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + C::BARS + kWarps * C::STAGES * 8);
    if (lane == 0)
        for (int s = 0; s < C::STAGES; ++s) mbar_init(&full[s], 1);
    if (threadIdx.x == 0) *abort_flag = 0;
    mbar_fence_init();
    __syncthreads();

    // tiles of 16 keys: [beg, end) for this CTA, every fourth of them for this warp
    const int64_t tiles = (len + kKeys - 1) / kKeys, per = (tiles + cs - 1) / cs;
    const int64_t beg = rank * per, end = min64(tiles, beg + per);
    const int mine = end > beg + warp ? (int)((end - beg - warp + kWarps - 1) / kWarps) : 0;
    unsigned char *ring = sm + warp * C::RING;
    auto copy = [&](int i) {
        const int st = i % C::STAGES;
        const int tok = (int)(n * a.sk.T + (beg + warp + (int64_t)i * kWarps) * kKeys);
        mbar_arrive_expect_tx(&full[st], C::STAGE);
#pragma unroll
        for (int r = 0; r < C::NR; ++r) {
            tma_load_3d(ring + st * C::STAGE + r * C::REG, &tk, &full[st], r * C::COLS, hk, tok);
            tma_load_3d(ring + st * C::STAGE + C::TILE + r * C::REG, &tv, &full[st], r * C::COLS, hk, tok);
        }
    };
    if (lane == 0)
        for (int i = 0; i < min(mine, C::STAGES); ++i) copy(i);
    __syncwarp();
    const float sc = a.scale * kLog2e;
    Rows<T, DP, GM> rows;
    rows.init(a, static_cast<const T *>(a.q) + (n * a.H + hk * a.G) * a.D, sm + C::QS, lane);
    int done = 0;
    for (; done < mine; ++done) {
        const int st = done % C::STAGES;
        // (one answer for all lanes: none is left behind at a warp-wide instruction)
        if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (done / C::STAGES) & 1, abort_flag))) break;
        unsigned char *kt = ring + st * C::STAGE, *vt = kt + C::TILE;
        const int valid = (int)min64(kKeys, len - (beg + warp + (int64_t)done * kWarps) * kKeys);
        if (valid < kKeys) {
            for (int i = lane; i < C::NR * 8 * (kKeys - valid); i += 32) {
                const int r = valid + i / (8 * C::NR), c = i % (8 * C::NR);
                *reinterpret_cast<uint4 *>(vt + (c >> 3) * C::REG + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
        }
        rows.tile(a, kt, vt, sm + C::QS, valid, sc, lane);
        __syncwarp();  // every lane has read the stage
        if (lane == 0 && done + C::STAGES < mine) copy(done + C::STAGES);
        __syncwarp();
    }
    if (done < mine)  // gave up: let the copies in flight land before the ring is reused
        for (int i = done; i < min(mine, done + C::STAGES); ++i) mbar_drain(&full[i % C::STAGES], (i / C::STAGES) & 1);
    __syncwarp();
    float *ml = reinterpret_cast<float *>(sm + C::ML);
    rows.leave(reinterpret_cast<float *>(ring), ml + warp * 32, sc, lane);
    if (cs > 1) cluster.sync();
    else __syncthreads();

    // Join: the warps of the cluster's CTAs, then the prefix's parts.  (log2 maximum, later
    // weight) and l of each part first.
    const int own = cs * kWarps, parts = own + pparts;
    const int64_t row0 = n * a.H + hk * a.G;
    float *pm = reinterpret_cast<float *>(sm + C::TAIL), *pl = reinterpret_cast<float *>(sm + C::RING + C::TAIL);
    for (int i = threadIdx.x; i < parts * a.G; i += 32 * kWarps) {
        const int p = i / a.G, g = i - p * a.G;
        float m, l;
        if (p < own) {
            const float2 x = *reinterpret_cast<const float2 *>(
                cluster.map_shared_rank(ml, p / kWarps) + (p % kWarps) * 32 + 2 * g);
            m = x.x;
            l = x.y;
        } else {
            m = a.part_lse[(p - own) * a.part_rows + row0 + g] * kLog2e;
            l = 1.f;
        }
        pm[p * 16 + g] = m;
        pl[p * 16 + g] = l;
    }
    __syncthreads();
    // one warp a row: its maximum, the parts' weights and 1 / sum
    for (int g = warp; g < a.G; g += kWarps) {
        float top = -INFINITY, l = 0.f;
        for (int p = lane; p < parts; p += 32) top = fmaxf(top, pm[p * 16 + g]);
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float base = top == -INFINITY ? 0.f : top;
        for (int p = lane; p < parts; p += 32) {
            const float f = exp2f(pm[p * 16 + g] - base);
            l = fmaf(f, pl[p * 16 + g], l);
            pm[p * 16 + g] = f;
        }
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        if (lane == 0) pl[g] = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // no key: 0; NaN scores: NaN
    }
    __syncthreads();
    // four columns a thread, the cluster's threads share them; eight loads in flight
    const int quads = a.D / 4;
    for (int i = rank * 32 * kWarps + threadIdx.x; i < a.G * quads; i += cs * 32 * kWarps) {
        const int g = i / quads, d = 4 * (i - g * quads);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p0 = 0; p0 < parts; p0 += 8) {
            float4 x[8];
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int p = p0 + e;
                f[e] = p < parts ? pm[p * 16 + g] : 0.f;
                x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (f[e] == 0.f) continue;  // (a part of the prefix without a key has no o)
                const float *src = p < own ? cluster.map_shared_rank(reinterpret_cast<float *>(sm + (p % kWarps) * C::RING),
                                                                     p / kWarps) + g * DP + d
                                           : a.part_o + ((p - own) * a.part_rows + row0 + g) * a.D + d;
                x[e] = *reinterpret_cast<const float4 *>(src);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                acc.x = fmaf(f[e], x[e].x, acc.x);
                acc.y = fmaf(f[e], x[e].y, acc.y);
                acc.z = fmaf(f[e], x[e].z, acc.z);
                acc.w = fmaf(f[e], x[e].w, acc.w);
            }
        }
        const float inv = pl[g];
        T *dst = static_cast<T *>(a.o) + (row0 + g) * a.D + d;
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        else
            *reinterpret_cast<float4 *>(dst) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
    if (cs > 1) cluster.sync();  // this CTA's shared memory has been read
    if (*abort_flag && a.status && threadIdx.x == 0) atomicExch(a.status, kDevTimeout);
}

template <typename T, int DP, int GM>
cudaError_t launch_rows(const AttnArgs &a, int cs, int pparts, const CUtensorMap &tk, const CUtensorMap &tv,
                        cudaStream_t st) {
    auto kern = attn_decode_kernel<T, DP, GM>;
    constexpr size_t smem = DecCfg<T, DP>::SMEM;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, smem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.N * a.Hk * cs));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tk, tv, a, pparts);
}

template <typename T, int DP>
cudaError_t launch_dec(const AttnArgs &a, int cs, int pparts, cudaStream_t st) {
    CUtensorMap tk, tv;
    constexpr bool f32 = sizeof(T) == 4;
    if (a.sk.T > 0) {
        cudaError_t e = tc_make_map_rows(&tk, a.k, a.N * a.sk.T, a.Hk, a.D, 1, kKeys, f32);
        if (e == cudaSuccess) e = tc_make_map_rows(&tv, a.v, a.N * a.sk.T, a.Hk, a.D, 1, kKeys, f32);
        if (e != cudaSuccess) return e;
    } else {  // no cache at all: never copied
        tk = tv = CUtensorMap{};
    }
    if constexpr (!f32) {
        return launch_rows<T, DP, 16>(a, cs, pparts, tk, tv, st);
    } else {
        if (a.G == 1) return launch_rows<T, DP, 1>(a, cs, pparts, tk, tv, st);
        if (a.G <= 4) return launch_rows<T, DP, 4>(a, cs, pparts, tk, tv, st);
        if (a.G <= 8) return launch_rows<T, DP, 8>(a, cs, pparts, tk, tv, st);
        return launch_rows<T, DP, 16>(a, cs, pparts, tk, tv, st);
    }
}

}  // namespace

cudaError_t launch_attn_decode(const AttnArgs &a, int cs, int pparts, cudaStream_t st) {
    if (a.bf16) return a.D <= 64 ? launch_dec<__nv_bfloat16, 64>(a, cs, pparts, st)
                                 : launch_dec<__nv_bfloat16, 128>(a, cs, pparts, st);
    return a.D <= 64 ? launch_dec<float, 64>(a, cs, pparts, st) : launch_dec<float, 128>(a, cs, pparts, st);
}

}  // namespace sgla
