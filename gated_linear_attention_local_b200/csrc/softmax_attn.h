// Softmax attention over heads [tokens, H, D] with shared key heads (internal to
// libsimplegla.so): arguments and launchers of the forward, backward and one-token kernels.
//
//   s_ij = scale q_i . k_j for the keys j that row i sees,  p_i = softmax(s_i),
//   o_i = sum_j p_ij v_j,  lse_i = log sum_j exp s_ij.
// Query head h reads key head h / G, G = H / Hk.  A causal row i of a sequence with tq
// queries and tk keys sees j <= i + tk - tq (the last query is aligned with the last key).
// A row that sees nothing has o = 0, lse = -inf and gradients 0.
//
// A tile's rows are "packed rows" r = token * G + g of one key head: the G query heads that
// share a key head are rows of the same tile, so every K and V tile is read once for all of
// them and their dk, dv contributions meet in one accumulator (no atomics, one fixed order).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "common.cuh"

namespace sgla {

// The sequences of a call on one side (queries or keys) of the flattened token axis.
struct AttnSeqs {
    const int64_t *cu;   // packed: device [N+1]; dense: nullptr
    const int64_t *len;  // one-token step: device [N] valid keys of each cache; else nullptr
    int64_t T;           // dense: tokens per sequence; packed: tokens in all
};

struct AttnArgs {
    const void *q, *k, *v;
    void *o;
    float *lse;           // [q tokens, H], natural log
    float scale;
    bool causal, bf16;
    int64_t N;            // sequences
    AttnSeqs sq, sk;
    int H, Hk, G, D;
    int *status;          // optional device word: SGLA_DEVICE_*
    // key splits: split z covers keys [z * split, (z + 1) * split); nullptr parts: one split,
    // o and lse written directly
    int64_t split;
    int nsplit;
    float *part_o;        // [part, q tokens * H, D] o of the split's keys alone
    float *part_lse;      // [part, q tokens * H]
    int64_t part_rows;    // q tokens * H
    // backward (o is only read there)
    const void *dout;
    const float *lse_in;  // [q tokens, H]
    float *delta;         // [q tokens, H] sum_d do o
    void *dq, *dk, *dv;
};

// fp32 (three tf32 products for one)
cudaError_t launch_attn_fwd_tf32(const AttnArgs &a, cudaStream_t st);
cudaError_t launch_attn_bwd_dkdv_tf32(const AttnArgs &a, cudaStream_t st);
cudaError_t launch_attn_bwd_dq_tf32(const AttnArgs &a, cudaStream_t st);
// delta_i = sum_d do_id o_id, one value a row (fp32)
cudaError_t launch_attn_delta(const AttnArgs &a, cudaStream_t st);

// Tensor cores, bf16.  The dq kernel also forms delta, which the dk dv kernel reads.
cudaError_t launch_attn_fwd_tc(const AttnArgs &a, cudaStream_t st);
cudaError_t launch_attn_bwd_dkdv_tc(const AttnArgs &a, cudaStream_t st);
cudaError_t launch_attn_bwd_dq_tc(const AttnArgs &a, cudaStream_t st);
// One query token a sequence (a.sq.T == 1), G <= kDecodeMaxGroup: clusters of cs CTAs a (sequence,
// key head); pparts <= kDecodeMaxParts parts of a prefix (a.part_o, a.part_lse, may
// be 0) join the result.
constexpr int kDecodeMaxGroup = 16, kDecodeMaxParts = 148;
cudaError_t launch_attn_decode(const AttnArgs &a, int cs, int pparts, cudaStream_t st);

// o of `rows` rows from `parts` parts (part_o, part_lse as in AttnArgs)
cudaError_t launch_attn_join(const float *part_o, const float *part_lse, void *o, int64_t rows, int parts, int D,
                             bool bf16, cudaStream_t st);

#ifdef __CUDACC__

// Allow a kernel its dynamic shared memory, once a device (`done`: a bit a device, one word a
// kernel).  Saves a runtime call on every launch.
template <typename F>
cudaError_t allow_smem(F kern, size_t bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// The span of sequence n on one side.  Packed batches have one sequence more than the caller
// gave: index N covers the tokens behind cu[N], which belong to no sequence (their partner
// span is empty, so their outputs are zeros).  False for bounds that are not
// 0 <= start <= end <= T.
__device__ __forceinline__ bool attn_span(const AttnSeqs &s, int64_t N, int64_t n, int64_t &t0, int64_t &len) {
    if (!s.cu) {
        t0 = n * s.T;
        len = s.T;
        if (s.len) {
            len = s.len[n];
            if (len < 0 || len > s.T) return false;
        }
        return true;
    }
    t0 = s.cu[n];
    const int64_t t1 = n < N ? s.cu[n + 1] : s.T;
    len = t1 - t0;
    return t0 >= 0 && t0 <= t1 && t1 <= s.T;
}

// Tiles of a packed batch: sequence n starts at slot floor(cu[n] * mul / div) + n, which
// leaves at least ceil(rows / div) slots for its rows = len * mul and needs no prefix sums;
// a slot past its sequence's rows has nothing to do.  Slots in all: floor(T * mul / div) + N + 1.
struct AttnTile {
    int64_t n;         // sequence
    int64_t q0, tq;    // its queries
    int64_t k0, tk;    // its keys
    int64_t row0;      // first row (own side) of this tile inside the sequence
};

// Fills t for slot `slot` of the side `own` (sq or sk); all 32 lanes of a warp take part
// (uniform result).  False: nothing to do.
__device__ __forceinline__ bool attn_locate(const AttnArgs &a, bool own_q, int64_t slot, int mul, int div,
                                            AttnTile &t) {
    const AttnSeqs &own = own_q ? a.sq : a.sk;
    int64_t first = 0;  // first slot of the sequence
    if (own.cu && a.status && slot < a.N && (threadIdx.x & 31) == 0) {  // every sequence is checked once, found or not
        int64_t s0, n0;
        if (!attn_span(a.sq, a.N, slot, s0, n0) || !attn_span(a.sk, a.N, slot, s0, n0) ||
            (slot == 0 && (a.sq.cu[0] != 0 || a.sk.cu[0] != 0)))
            atomicExch(a.status, kDevBadCuSeqlens);
    }
    if (!own.cu) {
        const int64_t per = (own.T * mul + div - 1) / div;
        t.n = slot / per;
        first = t.n * per;
        if (t.n >= a.N) return false;
    } else {
        // largest n in [0, N] whose first slot is <= slot: 32 probes a level
        const int lane = threadIdx.x & 31;
        int64_t lo = 0, hi = a.N + 1;  // answer in [lo, hi)
        while (hi - lo > 1) {
            const int64_t step = (hi - lo + 31) / 32;
            const int64_t probe = lo + lane * step;
            const bool below = probe < hi && own.cu[probe] * mul / div + probe <= slot;
            const unsigned m = __ballot_sync(0xffffffffu, below);
            const int c = m == 0u ? 0 : 31 - __clz(m);
            const int64_t nlo = lo + c * step;
            hi = min64(hi, nlo + step);
            lo = nlo;
        }
        t.n = lo;
        first = own.cu[lo] * mul / div + lo;
    }
    const bool okq = attn_span(a.sq, a.N, t.n, t.q0, t.tq), okk = attn_span(a.sk, a.N, t.n, t.k0, t.tk);
    if (!okq || !okk) {
        if (a.status) atomicExch(a.status, kDevBadCuSeqlens);
        // a cache whose length is out of range counts as empty; a packed sequence is skipped
        if (!(okq && a.sk.len)) return false;
        t.tk = 0;
    }
    if (t.n >= a.N) {  // behind the last sequence: zeros
        if (own_q) t.tk = 0; else t.tq = 0;
    }
    t.row0 = (slot - first) * div;
    return t.row0 >= 0 && t.row0 < (own_q ? t.tq : t.tk) * mul;
}

// The row tiles of a packed batch of up to kMax - 1 sequences, last ones (which see the most keys)
// first and over all sequences at once, so that no long tile is left for the end: the u-th tile is
// found from the sequences' tile counts, which one warp keeps in registers.  Against sequence by
// sequence: forward of 8 sequences, 16868 tokens in all, 185 -> 178 us.  (The backward kernels
// gained nothing: their items are half as long.)
struct AttnOrder {
    static constexpr int kPer = 8, kMax = 32 * kPer;
    bool on = false;
    int tiles[kPer];  // of sequences lane + 32 i; sequence N: the tokens behind the last

    // By all lanes of a warp; tiles of `div` tokens.
    __device__ __forceinline__ void init(const AttnArgs &a, int div) {
        on = a.sq.cu && a.N < kMax;
        if (!on) return;
        const int lane = threadIdx.x & 31;
        bool bad = a.sq.cu[0] != 0 || a.sk.cu[0] != 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int n = lane + 32 * i;
            tiles[i] = 0;
            int64_t q0, tq, k0, tk;
            if (n > a.N) continue;
            if (attn_span(a.sq, a.N, n, q0, tq) && attn_span(a.sk, a.N, n, k0, tk))
                tiles[i] = (int)((tq + div - 1) / div);
            else
                bad = true;
        }
        if (bad && a.status) atomicExch(a.status, kDevBadCuSeqlens);
        __syncwarp();
    }
    __device__ __forceinline__ int above(int level) const {  // tiles whose index in their sequence is at least level
        int c = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) c += max(tiles[i] - level, 0);
        return __reduce_add_sync(0xffffffffu, c);
    }
    // Tile u in that order; false when there are no more.
    __device__ __forceinline__ bool locate(const AttnArgs &a, int u, int div, AttnTile &t) const {
        int most = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) most = max(most, tiles[i]);
        int lo = 0, hi = __reduce_max_sync(0xffffffffu, most);
        if (u >= above(0)) return false;
        while (hi - lo > 1) {  // above(lo) > u >= above(hi)
            const int mid = lo + (hi - lo) / 2;
            if (above(mid) > u) lo = mid;
            else hi = mid;
        }
        int rank = u - above(lo + 1);  // among the sequences that have a tile `lo`
        t.n = -1;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int lane = threadIdx.x & 31;
            const unsigned m = __ballot_sync(0xffffffffu, tiles[i] > lo);
            const unsigned pick = __ballot_sync(0xffffffffu, tiles[i] > lo && __popc(m & ((1u << lane) - 1)) == rank);
            if (t.n < 0 && pick) t.n = 32 * i + __ffs(pick) - 1;
            rank -= __popc(m);
        }
        if (t.n < 0) return false;
        attn_span(a.sq, a.N, t.n, t.q0, t.tq);
        attn_span(a.sk, a.N, t.n, t.k0, t.tk);
        if (t.n == a.N) t.tk = 0;  // behind the last sequence: zeros
        t.row0 = (int64_t)lo * div;
        return t.row0 < t.tq;
    }
};

__host__ __device__ __forceinline__ int64_t attn_slots(const AttnSeqs &s, int64_t N, int mul, int div) {
    return s.cu ? s.T * mul / div + N + 1 : N * ((s.T * mul + div - 1) / div);
}

#endif

}  // namespace sgla
