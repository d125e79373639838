// kda_beam_select: log-softmax of the beams' logits, and the K best of a batch entry's beams x vocabulary.
#include "kda_step.cuh"

#include <cfloat>

namespace kda {
namespace {

constexpr int BEAM_THREADS = 512;

struct BeamArgs {
    const void *logits;
    int64_t row_stride;
    const float *beam_scores;
    const uint8_t *finished;
    int eos;
    float *scores;
    int32_t *tokens, *parents;
    int B, W, V, K;
};

__device__ __forceinline__ float load_logit(const float *p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float no_nan(float x) { return x == x ? x : -INFINITY; }

// Order-preserving integer of a float that is not NaN, above the complement of the candidate's index: the larger
// key is the better candidate, ties going to the lower index.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index)
{
    uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);   // -0 and +0 are a tie
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((uint64_t)u << 32) | (0xffffffffu - index);
}
__device__ __forceinline__ float key_value(uint64_t k)
{
    const uint32_t u = (uint32_t)(k >> 32);
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return 0xffffffffu - (uint32_t)k; }

__device__ uint64_t block_max(uint64_t x, uint64_t *sh)
{
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t y = __shfl_xor_sync(0xffffffffu, x, o);
        x = x > y ? x : y;
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0)
        sh[threadIdx.x / 32] = x;
    __syncthreads();
    x = sh[0];
    for (int i = 1; i < BEAM_THREADS / 32; i++)
        x = x > sh[i] ? x : sh[i];
    return x;
}
__device__ float block_sum(float x, float *sh)
{
    for (int o = 16; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0)
        sh[threadIdx.x / 32] = x;
    __syncthreads();
    x = 0.0f;
    for (int i = 0; i < BEAM_THREADS / 32; i++)
        x += sh[i];
    return x;
}

// One CTA per batch entry: the rows' statistics, then K passes that each take the best key below the last one.
template <typename T> __global__ void __launch_bounds__(BEAM_THREADS) kda_beam_kernel(const BeamArgs p)
{
    __shared__ uint64_t shk[BEAM_THREADS / 32];
    __shared__ float shf[BEAM_THREADS / 32], shc[32];
    const int b = blockIdx.x;
    for (int w = 0; w < p.W; w++) {
        const T *row = static_cast<const T *>(p.logits) + ((int64_t)b * p.W + w) * p.row_stride;
        uint64_t best = 0;
        for (int t = threadIdx.x; t < p.V; t += BEAM_THREADS) {
            const uint64_t k = key_of(no_nan(load_logit(row + t)), t);
            best = k > best ? k : best;
        }
        const float m = key_value(block_max(best, shk));
        float sum = 0.0f;
        for (int t = threadIdx.x; t < p.V; t += BEAM_THREADS)
            sum += expf(no_nan(load_logit(row + t)) - m);
        sum = block_sum(sum, shf);
        const float c = (p.beam_scores[b * p.W + w] - m) - logf(sum);
        if (threadIdx.x == 0)
            shc[w] = fabsf(m) <= FLT_MAX ? no_nan(c) : -INFINITY;
    }
    __syncthreads();
    uint64_t last = ~0ull;
    for (int k = 0; k < p.K; k++) {
        uint64_t best = 0;
        for (int w = 0; w < p.W; w++) {
            const T *row = static_cast<const T *>(p.logits) + ((int64_t)b * p.W + w) * p.row_stride;
            const float c = shc[w];
            const bool done = p.finished && p.finished[b * p.W + w];
            for (int t = threadIdx.x; t < p.V; t += BEAM_THREADS) {
                float s = done ? (t == p.eos ? no_nan(p.beam_scores[b * p.W + w]) : -INFINITY)
                               : (c == -INFINITY ? c : no_nan(c + no_nan(load_logit(row + t))));
                const uint64_t x = key_of(s, (uint32_t)w * p.V + t);
                if (x < last && x > best)
                    best = x;
            }
        }
        last = block_max(best, shk);
        if (threadIdx.x == 0) {
            p.scores[b * p.K + k] = key_value(last);
            p.tokens[b * p.K + k] = key_index(last) % p.V;
            p.parents[b * p.K + k] = b * p.W + key_index(last) / p.V;
        }
    }
}

}  // namespace

static kda_status_t check_beam(const void *logits, kda_dtype_t dtype, int64_t row_stride, const float *beam_scores,
                               const uint8_t *finished, int eos, const float *scores, const int32_t *tokens,
                               const int32_t *parents, int B, int W, int V, int K)
{
    if (B < 1 || W < 1 || W > 32 || V < 1 || K < 1 || K > 64 || (int64_t)K > (int64_t)W * V)
        return KDA_ERR_INVALID_ARGUMENT;
    if (V > (1 << 24) || (int64_t)B * W > INT32_MAX || (int64_t)B * K > INT32_MAX)
        return KDA_ERR_UNSUPPORTED;
    if (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_FP32)
        return KDA_ERR_INVALID_ARGUMENT;
    if (!logits || !beam_scores || !scores || !tokens || !parents || row_stride < V)
        return KDA_ERR_INVALID_ARGUMENT;
    if (finished && (eos < 0 || eos >= V))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!is_aligned(logits, dtype == KDA_DTYPE_BF16 ? 2 : 4) || !is_aligned(beam_scores, 4) ||
        !is_aligned(scores, 4) || !is_aligned(tokens, 4) || !is_aligned(parents, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

}  // namespace kda

using namespace kda;

extern "C" size_t kda_beam_select_workspace_size(int B, int W, int V, int K)
{
    return 0;
}

extern "C" kda_status_t kda_beam_select_ws(const void *logits, kda_dtype_t dtype, int64_t row_stride,
                                           const float *beam_scores, const uint8_t *finished, int eos, float *scores,
                                           int32_t *tokens, int32_t *parents, int B, int W, int V, int K,
                                           void *workspace, size_t workspace_bytes, kda_stream_t stream)
{
    const kda_status_t s = check_beam(logits, dtype, row_stride, beam_scores, finished, eos, scores, tokens, parents,
                                      B, W, V, K);
    if (s != KDA_OK)
        return s;
    const BeamArgs p{logits, row_stride, beam_scores, finished, eos, scores, tokens, parents, B, W, V, K};
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == KDA_DTYPE_BF16)
        kda_beam_kernel<__nv_bfloat16><<<B, BEAM_THREADS, 0, st>>>(p);
    else
        kda_beam_kernel<float><<<B, BEAM_THREADS, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_beam_select(const void *logits, kda_dtype_t dtype, int64_t row_stride,
                                        const float *beam_scores, const uint8_t *finished, int eos, float *scores,
                                        int32_t *tokens, int32_t *parents, int B, int W, int V, int K,
                                        kda_stream_t stream)
{
    return kda_beam_select_ws(logits, dtype, row_stride, beam_scores, finished, eos, scores, tokens, parents, B, W, V,
                              K, nullptr, 0, stream);
}
