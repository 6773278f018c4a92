// Entry points of softmax attention: argument validation, plan, workspace carve-up and
// launch order.  Contracts are in include/simple_gla.h.
#include <math.h>

#include <algorithm>

#include "launch_status.h"
#include "simple_gla.h"
#include "softmax_attn.h"

namespace {

using namespace sgla;

// every token index and difference of two, doubled, fits 32 bits in the kernels
constexpr int64_t kMaxTokens = (int64_t)1 << 30;

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

#define ATTN_LAUNCH(name, call)                       \
    do {                                              \
        LaunchRecord rec_(st);                        \
        const sgla_status s_ = rec_.done(call, name); \
        if (s_ != SGLA_OK) return s_;                 \
    } while (0)

sgla_status check_heads(int64_t H, int64_t Hk, int64_t D, sgla_dtype dtype) {
    if (H < 1 || Hk < 1 || D < 1 || H % Hk) return SGLA_ERR_INVALID_ARGUMENT;
    if (dtype != SGLA_BF16 && dtype != SGLA_FP32) return SGLA_ERR_INVALID_ARGUMENT;
    if (D > 128 || D % 8 || H > 65535 || H / Hk > 128) return SGLA_ERR_UNSUPPORTED;
    return SGLA_OK;
}

float pick_scale(float scale, int64_t D) {
    return (!(scale > 0.f) || isinf(scale)) ? 1.0f / sqrtf((float)D) : scale;
}

sgla_status reset_status(int *device_status, cudaStream_t st) {
    if (!device_status) return SGLA_OK;
    const cudaError_t e = cudaMemsetAsync(device_status, 0, sizeof(int), st);
    return e == cudaSuccess ? SGLA_OK : cuda_failure(e, "status reset");
}

// Checks shared by the forward and the backward; fills the sequence part of a.
sgla_status check_seqs(AttnArgs &a, const int64_t *cu_q, const int64_t *cu_k, int64_t N, int64_t Tq, int64_t Tk,
                       int64_t H, int64_t Hk, int64_t D, sgla_dtype dtype, float scale, int causal,
                       int *device_status, int64_t &q_tokens, int64_t &k_tokens) {
    if (N < 0 || Tq < 0 || Tk < 0 || !cu_q != !cu_k || (cu_q && N < 1)) return SGLA_ERR_INVALID_ARGUMENT;
    const sgla_status s = check_heads(H, Hk, D, dtype);
    if (s != SGLA_OK) return s;
    if (Tq >= kMaxTokens || Tk >= kMaxTokens || N >= kMaxTokens) return SGLA_ERR_UNSUPPORTED;
    q_tokens = cu_q ? Tq : N * Tq;
    k_tokens = cu_k ? Tk : N * Tk;
    if (q_tokens >= kMaxTokens || k_tokens >= kMaxTokens) return SGLA_ERR_UNSUPPORTED;
    if (!aligned(cu_q, 8) || !aligned(cu_k, 8) || !aligned(device_status, 4)) return SGLA_ERR_INVALID_ARGUMENT;
    a.N = N;
    a.sq.cu = cu_q; a.sq.T = Tq;
    a.sk.cu = cu_k; a.sk.T = Tk;
    a.H = (int)H; a.Hk = (int)Hk; a.G = (int)(H / Hk); a.D = (int)D;
    a.bf16 = dtype == SGLA_BF16;
    a.causal = causal != 0;
    a.scale = pick_scale(scale, D);
    a.status = device_status;
    a.split = kMaxTokens;
    a.nsplit = 1;
    return SGLA_OK;
}

cudaError_t launch_fwd(const AttnArgs &a, cudaStream_t st) {
    return a.bf16 ? launch_attn_fwd_tc(a, st) : launch_attn_fwd_tf32(a, st);
}

// The one-token step.  Up to kDecodeMaxGroup query heads a key head the streaming kernel takes
// the caches (clusters of CTAs, joined inside); above, the forward's tiles take them in parts.
// The prefix of all sequences is one sequence of N query tokens for the forward, in parts.
struct DecodePlan {
    sgla_status why = SGLA_ERR_INVALID_ARGUMENT;
    bool stream = true;
    int cluster = 1;                  // CTAs a (sequence, key head) of the streaming kernel
    int64_t split = 0, psplit = 0;    // keys per part of a cache, of the prefix
    int parts = 0, pparts = 0;        // parts of a cache (0: streaming), of the prefix
    bool direct = false;              // one part: no join
    size_t off_lse = 0, bytes = 0;
};

// Keys per part so that `units` work items times the parts come near to `target` CTAs, in
// whole tiles of 128 keys.
int64_t split_keys(int64_t keys, int64_t units, int64_t target) {
    const int64_t parts = std::min<int64_t>(kDecodeMaxParts, std::max<int64_t>(1, target / units));
    return std::max<int64_t>(256, (keys + parts - 1) / parts + 127) / 128 * 128;
}

DecodePlan decode_plan(int64_t N, int64_t S, int64_t P, int64_t H, int64_t Hk, int64_t D, sgla_dtype dtype) {
    DecodePlan p;
    if (N < 0 || S < 0 || P < 0) return p;
    if ((p.why = check_heads(H, Hk, D, dtype)) != SGLA_OK) return p;
    p.why = SGLA_ERR_UNSUPPORTED;
    if (N >= kMaxTokens || S >= kMaxTokens || P >= kMaxTokens || N * std::max<int64_t>(S, H) >= kMaxTokens) return p;
    p.why = SGLA_OK;
    if (N == 0) return p;
    const int64_t G = H / Hk;
    // forward work items of one pass over `tokens` query tokens; one persistent CTA an SM for
    // bf16, two CTAs an SM for fp32
    auto items = [&](int64_t tokens) {
        const int64_t R = 2 * (128 / G);
        return Hk * (dtype == SGLA_BF16 ? (tokens + R - 1) / R : (tokens * G + 63) / 64);
    };
    const int64_t target = dtype == SGLA_BF16 ? 148 : 2 * 148;
    p.stream = G <= kDecodeMaxGroup;
    if (p.stream) {
        // Few units: up to eight CTAs each (one cluster), no more than run at once (two an SM; a
        // second wave would double the time), at least 128 keys each.  Below 37 units that leaves
        // SMs idle however long the cache is: one of 131072 keys takes 187 us on 8 key heads (64
        // CTAs, 82 us at the copy rate) and on one (8 CTAs).  Many: at least four waves, so that
        // unequal lengths even out, at least 512 keys each (a CTA's fixed cost is some 5 us).
        const int64_t units = N * Hk;
        while (p.cluster < 8 && ((units * p.cluster * 2 <= 2 * 148 && S >= 256 * p.cluster) ||
                                 (units > 148 && units * p.cluster < 8 * 148 && S >= 1024 * p.cluster)))
            p.cluster *= 2;
    } else {
        p.split = split_keys(S, N * items(1), target);
        p.parts = (int)std::max<int64_t>(1, (S + p.split - 1) / p.split);
    }
    if (P > 0) {
        p.psplit = split_keys(P, items(N), target);
        p.pparts = (int)((P + p.psplit - 1) / p.psplit);
    }
    p.direct = p.parts + p.pparts <= 1 && P == 0;
    if (!p.direct) {
        const size_t rows = (size_t)(p.parts + p.pparts) * N * H;
        p.off_lse = align_up(rows * D * sizeof(float), 256);
        p.bytes = p.off_lse + align_up(rows * sizeof(float), 256);
    }
    return p;
}

}  // namespace

extern "C" {

sgla_status softmax_attention_fwd(const void *q, const void *k, const void *v, float scale, int causal, void *o,
                                  float *lse, const int64_t *cu_seqlens_q, const int64_t *cu_seqlens_k, int64_t N,
                                  int64_t Tq, int64_t Tk, int64_t H, int64_t Hk, int64_t D, sgla_dtype dtype,
                                  int *device_status, void *stream) {
    AttnArgs a{};
    int64_t q_tokens, k_tokens;
    sgla_status s = check_seqs(a, cu_seqlens_q, cu_seqlens_k, N, Tq, Tk, H, Hk, D, dtype, scale, causal,
                               device_status, q_tokens, k_tokens);
    if (s != SGLA_OK) return s;
    if ((q_tokens > 0 && (!q || !o)) || (k_tokens > 0 && (!k || !v))) return SGLA_ERR_INVALID_ARGUMENT;
    for (const void *p : {q, k, v, (const void *)o})
        if (!aligned(p, 16)) return SGLA_ERR_INVALID_ARGUMENT;
    if (!aligned(lse, 4)) return SGLA_ERR_INVALID_ARGUMENT;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((s = reset_status(device_status, st)) != SGLA_OK) return s;
    if (q_tokens == 0) return SGLA_OK;
    a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
    ATTN_LAUNCH("softmax_attention_fwd", launch_fwd(a, st));
    return SGLA_OK;
}

size_t softmax_attention_bwd_workspace_size(int64_t q_tokens, int64_t H) {
    if (q_tokens < 0 || H < 1 || q_tokens >= kMaxTokens || H > 65535) return 0;
    return align_up(std::max<size_t>(1, (size_t)q_tokens * H * sizeof(float)), 256);
}

sgla_status softmax_attention_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                                  const void *dout, float scale, int causal, void *dq, void *dk, void *dv,
                                  const int64_t *cu_seqlens_q, const int64_t *cu_seqlens_k, int64_t N, int64_t Tq,
                                  int64_t Tk, int64_t H, int64_t Hk, int64_t D, sgla_dtype dtype, int *device_status,
                                  void *workspace, size_t workspace_bytes, void *stream) {
    AttnArgs a{};
    int64_t q_tokens, k_tokens;
    sgla_status s = check_seqs(a, cu_seqlens_q, cu_seqlens_k, N, Tq, Tk, H, Hk, D, dtype, scale, causal,
                               device_status, q_tokens, k_tokens);
    if (s != SGLA_OK) return s;
    if (q_tokens > 0 && (!q || !o || !lse || !dout || !dq)) return SGLA_ERR_INVALID_ARGUMENT;
    if (k_tokens > 0 && (!k || !v || !dk || !dv)) return SGLA_ERR_INVALID_ARGUMENT;
    for (const void *p : {q, k, v, o, dout, (const void *)dq, (const void *)dk, (const void *)dv})
        if (!aligned(p, 16)) return SGLA_ERR_INVALID_ARGUMENT;
    if (!aligned(lse, 4) || !aligned(workspace, 256)) return SGLA_ERR_INVALID_ARGUMENT;
    if (!workspace || workspace_bytes < softmax_attention_bwd_workspace_size(q_tokens, H)) return SGLA_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((s = reset_status(device_status, st)) != SGLA_OK) return s;
    a.q = q; a.k = k; a.v = v; a.dout = dout; a.lse_in = lse; a.delta = static_cast<float *>(workspace);
    a.dq = dq; a.dk = dk; a.dv = dv;
    a.o = const_cast<void *>(o);  // only read
    if (q_tokens > 0 && !a.bf16) ATTN_LAUNCH("softmax_attention_delta", launch_attn_delta(a, st));
    // dq first: for bf16 it forms delta as well
    if (q_tokens > 0)
        ATTN_LAUNCH("softmax_attention_dq", a.bf16 ? launch_attn_bwd_dq_tc(a, st) : launch_attn_bwd_dq_tf32(a, st));
    if (k_tokens > 0)
        ATTN_LAUNCH("softmax_attention_dkdv",
                    a.bf16 ? launch_attn_bwd_dkdv_tc(a, st) : launch_attn_bwd_dkdv_tf32(a, st));
    return SGLA_OK;
}

size_t softmax_attention_decode_workspace_size(int64_t N, int64_t S, int64_t P, int64_t H, int64_t Hk, int64_t D,
                                               sgla_dtype dtype) {
    return decode_plan(N, S, P, H, Hk, D, dtype).bytes;
}

sgla_status softmax_attention_decode_step(const void *q, const void *k_cache, const void *v_cache,
                                          const int64_t *lengths, const void *prefix_k, const void *prefix_v,
                                          float scale, void *o, int64_t N, int64_t S, int64_t P, int64_t H, int64_t Hk,
                                          int64_t D, sgla_dtype dtype, int *device_status, void *workspace,
                                          size_t workspace_bytes, void *stream) {
    const DecodePlan p = decode_plan(N, S, P, H, Hk, D, dtype);
    if (p.why != SGLA_OK) return p.why;
    if (!aligned(device_status, 4) || !aligned(lengths, 8)) return SGLA_ERR_INVALID_ARGUMENT;
    if (N > 0 && (!q || !o || !lengths || (S > 0 && (!k_cache || !v_cache)) || (P > 0 && (!prefix_k || !prefix_v))))
        return SGLA_ERR_INVALID_ARGUMENT;
    for (const void *x : {q, k_cache, v_cache, prefix_k, prefix_v, (const void *)o})
        if (!aligned(x, 16)) return SGLA_ERR_INVALID_ARGUMENT;
    if (p.bytes > 0) {
        if (!workspace || workspace_bytes < p.bytes) return SGLA_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return SGLA_ERR_INVALID_ARGUMENT;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const sgla_status s = reset_status(device_status, st);
    if (s != SGLA_OK || N == 0) return s;
    AttnArgs a{};
    a.q = q; a.o = o;
    a.scale = pick_scale(scale, D);
    a.bf16 = dtype == SGLA_BF16;
    a.H = (int)H; a.Hk = (int)Hk; a.G = (int)(H / Hk); a.D = (int)D;
    a.part_rows = N * H;
    float *part_o = static_cast<float *>(workspace);
    float *part_lse = p.direct ? nullptr : reinterpret_cast<float *>(static_cast<char *>(workspace) + p.off_lse);
    if (P > 0) {  // every query token against the prefix, as one sequence; its parts come first
        a.k = prefix_k; a.v = prefix_v;
        a.N = 1;
        a.sq.T = N;
        a.sk.T = P;
        a.split = p.psplit; a.nsplit = p.pparts;
        a.part_o = part_o;
        a.part_lse = part_lse;
        a.status = device_status;
        ATTN_LAUNCH("softmax_attention_prefix", launch_fwd(a, st));
    }
    a.k = k_cache; a.v = v_cache;
    a.N = N;
    a.sq.T = 1;
    a.sk.T = S; a.sk.len = lengths;
    a.status = device_status;
    if (p.stream) {
        ATTN_LAUNCH("softmax_attention_decode", launch_attn_decode(a, p.cluster, p.pparts, st));
        return SGLA_OK;
    }
    a.split = p.split; a.nsplit = p.parts;
    a.part_o = p.direct ? nullptr : part_o + (int64_t)p.pparts * N * H * D;
    a.part_lse = p.direct ? nullptr : part_lse + (int64_t)p.pparts * N * H;
    ATTN_LAUNCH("softmax_attention_decode", launch_fwd(a, st));
    if (!p.direct)
        ATTN_LAUNCH("softmax_attention_join",
                    launch_attn_join(part_o, part_lse, o, N * H, p.parts + p.pparts, (int)D, a.bf16, st));
    return SGLA_OK;
}

}  // extern "C"
