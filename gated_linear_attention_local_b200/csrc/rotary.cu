// Rotary positions with several axes, applied to q and k in front of a token mixer
// ("relinear -- convert pretrained transformers to linear/hybrid-attention models": the
// layer's _qk_transform rotates q and k; its one-token form is not supported there).
//
// Pair i of the R / 2 rotated pairs of a head turns by theta = p * f_i, with p the token's
// position on the axis of pair i (time, height, width, ... of a patch; one axis for text):
//   (x, y) <- (x cos theta - y sin theta, x sin theta + y cos theta),
// pairs (i, i + R/2) or, interleaved, (2 i, 2 i + 1); columns R .. D-1 pass unchanged.  The
// map is orthogonal, so its gradient is the rotation by -theta.
//
// Precision: theta reaches 10^6 and more, where fp32 holds it to 0.06 only.  The turns
// p * (f_i / 2 pi) are formed in fp64 and reduced to [-1/2, 1/2] there; sine and cosine of
// the reduced angle are fp32.  Products are fp32, rounded once to the operand type.
//
// Bound: HBM (each element read and written once).  cos and sin depend on the token and the
// pair only, so a block first forms those of its tokens once (shared memory) and then streams
// every head of q and k past them in 16-byte vectors, an item (two vectors) a thread at a time
// (two or four items in flight measured slower, 248 and 388 us).  65536 tokens of 32 + 8 heads of
// 128 (1.34 GB): 214 us, 96 % of the measured copy rate.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "common.cuh"
#include "launch_status.h"
#include "simple_gla.h"

namespace sgla {
namespace {

constexpr int kMaxPairs = 256;
constexpr int kRotThreads = 128;

struct RotArgs {
    const void *q, *k;
    void *qo, *ko;
    const int64_t *pos;
    const float *freq;
    int64_t tokens;
    int H, Hk, D, half, A, tpb;  // half = R / 2 pairs, tpb = tokens per block
    float sign;
    uint8_t axis[kMaxPairs];
};

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
    T x[VEC];
};

// STREAM: 16-byte vectors bypass the L2's replacement order (evict first).
template <bool STREAM, typename V>
__device__ __forceinline__ V load_vec(const void *p) {
    if constexpr (STREAM && sizeof(V) == 16) {
        const uint4 u = __ldcs(static_cast<const uint4 *>(p));
        V v;
        memcpy(&v, &u, 16);
        return v;
    } else {
        return *static_cast<const V *>(p);
    }
}
template <bool STREAM, typename V>
__device__ __forceinline__ void store_vec(void *p, const V &v) {
    if constexpr (STREAM && sizeof(V) == 16) {
        uint4 u;
        memcpy(&u, &v, 16);
        __stcs(static_cast<uint4 *>(p), u);
    } else {
        *static_cast<V *>(p) = v;
    }
}

// Items of one head: half layout R/2/VEC items of two vectors (the pairs' first and second
// elements), interleaved R/VEC items of one vector; then (D-R)/VEC vectors that are copied.
template <typename T, int VEC, bool INTER, bool STREAM>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotArgs a) {
    // [tpb][half] cos, sin.  PV pairs belong to an item; they lie two by two, [PV / 2][items][2],
    // so that the lanes of consecutive items read consecutive 16 bytes.
    extern __shared__ __align__(16) float2 cs[];
    constexpr int PV = INTER ? (VEC + 1) / 2 : VEC, PQ = PV >= 2 ? 2 : 1;
    const int rot_items = a.half / PV;
    const int64_t t0 = (int64_t)blockIdx.x * a.tpb;
    const int nt = (int)min64(a.tpb, a.tokens - t0);
    for (int i = threadIdx.x; i < nt * a.half; i += kRotThreads) {
        const int t = i / a.half, p = i - t * a.half;
        double turns = (double)a.pos[(t0 + t) * a.A + a.axis[p]] * ((double)a.freq[p] * 0.15915494309189533577);
        turns -= rint(turns);
        float s, c;
        sincospif(2.f * (float)turns, &s, &c);
        const int e = p % PV;
        cs[t * a.half + ((e / PQ) * rot_items + p / PV) * PQ + e % PQ] = make_float2(c, a.sign * s);
    }
    __syncthreads();
    using V = Vec<T, VEC>;
    const int per_head = rot_items + (a.D - 2 * a.half) / VEC;
    const int heads = a.H + a.Hk, per_token = heads * per_head, total = nt * per_token;
    for (int idx = threadIdx.x; idx < total; idx += kRotThreads) {
        const int tok = idx / per_token, r = idx - tok * per_token, h = r / per_head, item = r - h * per_head;
        const bool isq = h < a.H, rotates = item < rot_items;
        const int col = (INTER || rotates) ? item * VEC : 2 * a.half + (item - rot_items) * VEC;
        const int64_t off = (isq ? (t0 + tok) * a.H + h : (t0 + tok) * a.Hk + (h - a.H)) * a.D + col;
        const T *src = static_cast<const T *>(isq ? a.q : a.k) + off;
        T *dst = static_cast<T *>(isq ? a.qo : a.ko) + off;
        V x = load_vec<STREAM, V>(src), y;
        if (rotates) {
            if constexpr (!INTER) y = load_vec<STREAM, V>(src + a.half);
            float2 w[PV];
#pragma unroll
            for (int e = 0; e < PV; e += PQ) {
                const float2 *c = cs + tok * a.half + ((e / PQ) * rot_items + item) * PQ;
                if constexpr (PQ == 2) {  // PV is even, so is half: 16-byte aligned
                    const float4 q = *reinterpret_cast<const float4 *>(c);
                    w[e] = make_float2(q.x, q.y);
                    w[e + 1] = make_float2(q.z, q.w);
                } else {
                    w[e] = c[0];
                }
            }
            if constexpr (INTER) {
#pragma unroll
                for (int e = 0; e < PV; ++e) {
                    const float p = to_f32(x.x[2 * e]), s = to_f32(x.x[2 * e + 1]);
                    x.x[2 * e] = from_f32<T>(p * w[e].x - s * w[e].y);
                    x.x[2 * e + 1] = from_f32<T>(p * w[e].y + s * w[e].x);
                }
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float p = to_f32(x.x[e]), s = to_f32(y.x[e]);
                    x.x[e] = from_f32<T>(p * w[e].x - s * w[e].y);
                    y.x[e] = from_f32<T>(p * w[e].y + s * w[e].x);
                }
                store_vec<STREAM>(dst + a.half, y);
            }
        }
        store_vec<STREAM>(dst, x);
    }
}

template <typename T, int VEC, bool INTER>
cudaError_t launch_rotary(const RotArgs &a, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.tokens + a.tpb - 1) / a.tpb);
    const size_t smem = (size_t)a.tpb * a.half * sizeof(float2);
    // Tensors that pass twice the L2 (126 MB) gain from the streaming hints (264 -> 214 us at
    // 1.34 GB); smaller ones stay for the kernel that reads them next (36.7 us with, 35.3 without
    // at 168 MB).
    if (2 * a.tokens * (a.H + a.Hk) * a.D * (int64_t)sizeof(T) > ((int64_t)252 << 20))
        rotary_kernel<T, VEC, INTER, true><<<grid, kRotThreads, smem, st>>>(a);
    else
        rotary_kernel<T, VEC, INTER, false><<<grid, kRotThreads, smem, st>>>(a);
    return cudaGetLastError();
}

// The widest vector that divides every run of columns handled together (at most 16 bytes).
// D and R are even, so interleaved pairs always fit vectors of two.
template <typename T>
cudaError_t launch_rotary_vec(const RotArgs &a, bool inter, cudaStream_t st) {
    const int run = inter ? (a.D | (2 * a.half)) : (a.D | a.half);  // common low bits of the column offsets
    constexpr int W = 16 / (int)sizeof(T);
    if (run % W == 0) return inter ? launch_rotary<T, W, true>(a, st) : launch_rotary<T, W, false>(a, st);
    if (W > 4 && run % 4 == 0) return inter ? launch_rotary<T, 4, true>(a, st) : launch_rotary<T, 4, false>(a, st);
    if (run % 2 == 0) return inter ? launch_rotary<T, 2, true>(a, st) : launch_rotary<T, 2, false>(a, st);
    return launch_rotary<T, 1, false>(a, st);
}

}  // namespace
}  // namespace sgla

extern "C" sgla_status multi_axis_rotary(const void *q, const void *k, const int64_t *positions, const float *inv_freq,
                                         const uint8_t *axis_of_pair, void *q_out, void *k_out, int64_t tokens,
                                         int64_t H, int64_t Hk, int64_t D, int64_t R, int64_t A, int interleaved,
                                         int inverse, sgla_dtype dtype, void *stream) {
    using namespace sgla;
    if (tokens < 0 || H < 0 || Hk < 0 || D < 1 || R < 0 || R > D || R % 2 || A < 1)
        return SGLA_ERR_INVALID_ARGUMENT;
    if (dtype != SGLA_BF16 && dtype != SGLA_FP32) return SGLA_ERR_INVALID_ARGUMENT;
    if (D % 2 || R / 2 > kMaxPairs || A > 255 || H + Hk > 65535 || D > 4096 || tokens >= ((int64_t)1 << 31))
        return SGLA_ERR_UNSUPPORTED;
    if (tokens == 0 || H + Hk == 0) return SGLA_OK;
    if ((H > 0 && (!q || !q_out)) || (Hk > 0 && (!k || !k_out)) || (R > 0 && (!positions || !inv_freq || !axis_of_pair)))
        return SGLA_ERR_INVALID_ARGUMENT;
    for (const void *p : {q, k, (const void *)q_out, (const void *)k_out})
        if (reinterpret_cast<uintptr_t>(p) % 16) return SGLA_ERR_INVALID_ARGUMENT;
    if (reinterpret_cast<uintptr_t>(positions) % 8 || reinterpret_cast<uintptr_t>(inv_freq) % 4)
        return SGLA_ERR_INVALID_ARGUMENT;
    RotArgs a{};
    a.q = q; a.k = k; a.qo = q_out; a.ko = k_out; a.pos = positions; a.freq = inv_freq; a.tokens = tokens;
    a.H = (int)H; a.Hk = (int)Hk; a.D = (int)D; a.half = (int)(R / 2); a.A = (int)A;
    a.sign = inverse ? -1.f : 1.f;
    for (int i = 0; i < a.half; ++i) {
        if (axis_of_pair[i] >= A) return SGLA_ERR_INVALID_ARGUMENT;
        a.axis[i] = axis_of_pair[i];
    }
    // four tokens a block once there are enough blocks to fill the GPU that way, else one
    a.tpb = tokens >= 4 * 148 * 4 ? 4 : 1;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    LaunchRecord rec(st);
    return rec.done(dtype == SGLA_BF16 ? launch_rotary_vec<__nv_bfloat16>(a, interleaved != 0, st)
                                       : launch_rotary_vec<float>(a, interleaved != 0, st),
                    "multi_axis_rotary");
}
