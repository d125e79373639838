// Linear attention with a decay for each head: the problem description its kernels share.
#pragma once

#include "kda_step.cuh"

namespace kda {

struct LinearArgs {
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;   // elements from token to token
    const float *log_decay;                 // [H] or nullptr
    const float *gate;                      // [tokens][H] or nullptr
    float scale;
    __nv_bfloat16 *out;
    const void *init;                       // [N][H][dim][dim], row v, column k, or nullptr
    void *fin;
    const int32_t *lens;                    // [N] or nullptr
    Tokens tok;
    int H, group, dim;                      // group = heads that share a key head
    unsigned int *err;
};

// Below this a decay is 0 in fp32 (e^-104 < 2^-150) whatever comes after it; clamped there, sums of logarithms stay finite.
constexpr float MIN_LOG_DECAY = -200.0f;

// The logarithm of a token's decay for a head: at most 0 (a positive one is reported and taken as 0), NaN as it is.
__device__ __forceinline__ float log_decay_of(float fixed, float gate, bool &bad)
{
    float a = fixed + gate;
    if (a > 0.0f) {
        bad = true;
        a = 0.0f;
    }
    return a < MIN_LOG_DECAY ? MIN_LOG_DECAY : a;
}
__device__ __forceinline__ float gate_of(const LinearArgs &p, int64_t token, int h) { return p.gate ? p.gate[token * p.H + h] : 0.0f; }

// First token and length of sequence n.
__device__ __forceinline__ void linear_range(const LinearArgs &p, int n, int64_t &bos, int64_t &len, bool &bad)
{
    if (p.tok.cu) {
        bad |= seq_range(p.tok.cu, n, p.tok.N, p.tok.T, bos, len);
        return;
    }
    bos = n * p.tok.T;
    len = p.tok.T;
    if (p.lens) {
        const int64_t x = p.lens[n];
        bad |= x < 0 || x > len;
        len = x < 0 ? 0 : (x > len ? len : x);
    }
}

// How a call runs in chunks: groups of group_chunks chunks of a sequence side by side (groups = 1: none are cut).
struct LinearPlan {
    int64_t group_chunks;
    int groups;               // of a sequence; of the longest there can be with cu_seqlens
    int64_t items, items_before;   // (sequence, group, head), and those whose state a later group starts from (upper bounds)
    float *states;            // what groups add to the state, then the next group's start: [slots][H][dim][dim]  (workspace)
    float2 *decays;           // their decays, as factor and kind: [slots][H]  (workspace)
    kda_dtype_t state_type;
    uint32_t wait_polls;
};

cudaError_t launch_linear_chunks(const LinearArgs &p, const LinearPlan &plan, cudaStream_t stream);
cudaError_t launch_linear_tokens(const LinearArgs &p, kda_dtype_t state, cudaStream_t stream);

}  // namespace kda
