// kda_verify_drafts: which of a request's drafted tokens the target model's distribution accepts, and the token after them.
//
// Row i of a request's logits is the target's distribution after i drafts, p_i = softmax(l_i / tau).  Draft x_i is
// accepted while u_i q_i(x_i) < p_i(x_i); at the first row r that is not (or the row after the last draft) the token is drawn
// from what the drafts left over, w = max(p_r - q_r, 0), by a race: the largest w_t / E_t with the caller's E_t ~ Exp(1) is
// distributed as w.  (A race needs no running sum over the vocabulary, whose rounding would decide next to every border.)
//
// Two kernels.  Statistics: a CTA takes a chunk of a row, holds it in registers, and writes its maximum m and
// sum_t exp((l_t - m) / tau); every logit is read once, and that is what bounds the call.  Pick: a cluster of CTAs takes a
// request, joins its rows' statistics (each CTA for itself: a few hundred numbers), decides r, and scans row r, the
// draft's row r and the noise, an eighth of the vocabulary a CTA; the best eight meet in shared memory.
#include "kda_step.cuh"

#include <cfloat>
#include <cmath>

namespace kda {
namespace {

constexpr int THREADS = 256;
constexpr int CLUSTER = 8;                  // CTAs of a request in the pick
constexpr int MAX_DRAFTS = 31;
constexpr unsigned FULL = 0xffffffffu;

struct VerifyArgs {
    const void *logits;
    int64_t row_stride;
    const int32_t *drafts;
    const float *probs, *uniform, *noise, *temperature;
    const int32_t *draft_lens;
    int32_t *tokens, *counts;
    int B, K, V;
    int chunk, chunks;
    float2 *stats;               // [B (K + 1)][chunks]: maximum, sum of exponentials (workspace)
    unsigned int *err;
};

// Drafts of request b and its temperature (0: greedy); what breaks the contract is clamped and reported.
__device__ __forceinline__ int drafts_of(const VerifyArgs &p, int b, bool &bad)
{
    if (!p.draft_lens)
        return p.K;
    const int n = p.draft_lens[b];
    bad |= n < 0 || n > p.K;
    return min(max(n, 0), p.K);
}
__device__ __forceinline__ float temperature_of(const VerifyArgs &p, int b, bool &bad)
{
    if (!p.temperature)
        return 1.0f;
    const float t = p.temperature[b];
    if (t >= 0.0f && t <= FLT_MAX)
        return t;
    bad = true;
    return 0.0f;
}

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
// a NaN logit counts as -inf
__device__ __forceinline__ float logit(float x) { return x == x ? x : -INFINITY; }

template <typename T> __device__ __forceinline__ void unpack(const uint4 &y, float *x);
template <> __device__ __forceinline__ void unpack<float>(const uint4 &y, float *x)
{
    x[0] = __uint_as_float(y.x), x[1] = __uint_as_float(y.y), x[2] = __uint_as_float(y.z), x[3] = __uint_as_float(y.w);
}
template <> __device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4 &y, float *x)
{
    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; i++)
        x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
}

__device__ __forceinline__ float block_max(float x, float *sm)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x = fmaxf(x, __shfl_xor_sync(FULL, x, o));
    if ((threadIdx.x & 31) == 0)
        sm[threadIdx.x / 32] = x;
    __syncthreads();
    x = sm[0];
#pragma unroll
    for (int i = 1; i < THREADS / 32; i++)
        x = fmaxf(x, sm[i]);
    return x;
}
__device__ __forceinline__ float block_sum(float x, float *sm)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x += __shfl_xor_sync(FULL, x, o);
    if ((threadIdx.x & 31) == 0)
        sm[threadIdx.x / 32] = x;
    __syncthreads();
    x = sm[0];
#pragma unroll
    for (int i = 1; i < THREADS / 32; i++)
        x += sm[i];
    return x;
}

// log2(e) / tau, kept finite so that a logit at the maximum still gets weight 1 for the smallest tau
__device__ __forceinline__ float exponent_scale(float tau) { return fminf(LOG2E / tau, FLT_MAX); }

// One chunk of one row a CTA: VECS 16-byte vectors a thread.  The row may start anywhere: vectors are cut at 16-byte
// boundaries of memory, and one that reaches over an end of the row is read element by element.
template <typename T, int VECS> __global__ void __launch_bounds__(THREADS) kda_verify_stats_kernel(const VerifyArgs p)
{
    constexpr int E = 16 / sizeof(T);
    __shared__ float sm[2][THREADS / 32];
    const int row = blockIdx.x / p.chunks, c = blockIdx.x % p.chunks, b = row / (p.K + 1);
    const int tid = threadIdx.x;
    stream_order();
    bool bad = false;
    if (row - b * (p.K + 1) > drafts_of(p, b, bad))
        return;                                     // behind the request's last draft
    const float tau = temperature_of(p, b, bad);
    const T *l = static_cast<const T *>(p.logits) + row * p.row_stride;
    const int off = (int)((reinterpret_cast<uintptr_t>(l) & 15) / sizeof(T));
    float x[VECS][E];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VECS; i++) {
        const int at = (c * (THREADS * VECS) + i * THREADS + tid) * E - off;   // first element of the vector
        if (at >= 0 && at + E <= p.V) {
            unpack<T>(__ldcg(reinterpret_cast<const uint4 *>(l + at)), x[i]);
        } else {
#pragma unroll
            for (int e = 0; e < E; e++)
                x[i][e] = at + e >= 0 && at + e < p.V ? as_float(l[at + e]) : -INFINITY;
        }
    }
#pragma unroll
    for (int i = 0; i < VECS; i++)
#pragma unroll
        for (int e = 0; e < E; e++)
            m = fmaxf(m, x[i][e]);                  // (fmaxf leaves NaN out)
    m = block_max(m, sm[0]);
    float s = 0.0f;
    if (tau > 0.0f && m > -INFINITY) {
        const float f = exponent_scale(tau);
#pragma unroll
        for (int i = 0; i < VECS; i++)
#pragma unroll
            for (int e = 0; e < E; e++) {
                const float y = ex2_approx((x[i][e] - m) * f);
                s += y == y ? y : 0.0f;
            }
    }
    s = block_sum(s, sm[1]);
    if (tid == 0)
        p.stats[(int64_t)row * p.chunks + c] = make_float2(m, s);
}

// exp(d / tau) for d <= 0, to about an ulp: the quotient's rounding is put back, and one too small for fp32 is 0.
__device__ __forceinline__ float weight_of(float d, float tau, float inv)
{
    const float x = d * inv;
    if (!(x > -104.0f))
        return 0.0f;
    return expf(x) * (1.0f + fmaf(-x, tau, d) * inv);
}

__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int rank)
{
    uint32_t x;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(x) : "r"(addr), "r"(rank));
    return x;
}

// A cluster a request.
template <typename T> __global__ void __launch_bounds__(THREADS) kda_verify_pick_kernel(const VerifyArgs p)
{
    __shared__ float row_max[MAX_DRAFTS + 1], row_sum[MAX_DRAFTS + 1];
    __shared__ int row_ok[MAX_DRAFTS + 1];
    __shared__ unsigned long long best_of[THREADS / 32], best_cta[2][CLUSTER];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int b = blockIdx.x / CLUSTER, rank = blockIdx.x % CLUSTER;
    stream_order();
    bool bad = false;
    const int L = drafts_of(p, b, bad);
    const float tau = temperature_of(p, b, bad), inv = tau > 0.0f ? fminf(1.0f / tau, FLT_MAX) : 0.0f;
    const T *logits = static_cast<const T *>(p.logits) + (int64_t)b * (p.K + 1) * p.row_stride;
    for (int i = warp; i <= L; i += THREADS / 32) {
        const float2 *st = p.stats + ((int64_t)b * (p.K + 1) + i) * p.chunks;
        float m = -INFINITY, z = 0.0f;
        for (int c = lane; c < p.chunks; c += 32)
            m = fmaxf(m, __ldcg(&st[c].x));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
        if (tau > 0.0f)
            for (int c = lane; c < p.chunks; c += 32) {
                const float2 x = __ldcg(&st[c]);
                z += x.x == -INFINITY ? 0.0f : x.y * weight_of(x.x - m, tau, inv);
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            z += __shfl_xor_sync(FULL, z, o);
        if (lane == 0) {
            bool ok = false;
            if (i < L && fabsf(m) <= FLT_MAX) {
                const int x = p.drafts[b * p.K + i];
                if (x < 0 || x >= p.V) {
                    bad = true;
                } else {
                    const float l = logit(as_float(logits[i * p.row_stride + x]));
                    if (tau > 0.0f) {
                        const float q = p.probs ? p.probs[((int64_t)b * p.K + i) * p.V + x] : 1.0f;
                        ok = p.uniform[b * p.K + i] * q < weight_of(l - m, tau, inv) / z;
                    } else {
                        ok = l == m;
                    }
                }
            }
            row_max[i] = m, row_sum[i] = z, row_ok[i] = ok;
        }
    }
    __syncthreads();
    int r = 0;
    while (r < L && row_ok[r])
        r++;
    const float m = row_max[r], z = row_sum[r];
    const bool alive = fabsf(m) <= FLT_MAX;
    const int x = r < L ? p.drafts[b * p.K + r] : -1;
    const T *l = logits + r * p.row_stride;
    const float *noise = p.noise + (int64_t)b * p.V;
    const float *q = r < L && p.probs ? p.probs + ((int64_t)b * p.K + r) * p.V : nullptr;
    // the best of the race: its value's bits above the complement of its index, so that ties go to the lower one
    unsigned long long best = 0;
    for (int pass = 0; pass < 2; pass++) {
        const int share = (p.V + CLUSTER - 1) / CLUSTER, from = rank * share, to = min(p.V, from + share);
        best = 0;
        if (alive) {
#pragma unroll 4
            for (int t = from + tid; t < to; t += THREADS) {
                const float d = logit(as_float(l[t])) - m;
                float v;
                if (tau > 0.0f) {
                    float w = weight_of(d, tau, inv) / z;
                    if (pass == 0 && r < L)
                        w = q ? w - q[t] : (t == x ? 0.0f : w);
                    v = w > 0.0f ? w / noise[t] : 0.0f;
                } else {
                    v = d == 0.0f ? 1.0f : 0.0f;
                }
                if (v > 0.0f) {
                    const unsigned long long key = ((unsigned long long)__float_as_uint(v) << 32) | (uint32_t)~t;
                    best = key > best ? key : best;
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long y = __shfl_xor_sync(FULL, best, o);
            best = y > best ? y : best;
        }
        if (lane == 0)
            best_of[warp] = best;
        __syncthreads();
        if (tid < CLUSTER) {
            best = best_of[0];
#pragma unroll
            for (int i = 1; i < THREADS / 32; i++)
                best = best_of[i] > best ? best_of[i] : best;
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(in_cta(smem_u32(&best_cta[pass][rank]), tid)), "l"(best) : "memory");
        }
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
        best = 0;
#pragma unroll
        for (int i = 0; i < CLUSTER; i++)
            best = best_cta[pass][i] > best ? best_cta[pass][i] : best;
        if (best != 0 || r == L || !alive)           // the same in every CTA of the cluster
            break;
        // nothing is left over (rounding): the race is run on p itself
    }
    if (rank == 0) {
        const int token = best ? (int)~(uint32_t)best : -1;
        for (int i = tid; i <= p.K; i += THREADS)
            p.tokens[b * (p.K + 1) + i] = i < r ? p.drafts[b * p.K + i] : (i == r ? token : -1);
        if (tid == 0)
            p.counts[b] = r + 1;
    }
    report(p.err, bad && rank == 0, DEVERR_CU_SEQLENS);
}

constexpr int STATS_VECS = 8;       // 16-byte vectors of a thread of the statistics

template <typename T> cudaError_t launch_verify(const VerifyArgs &p, cudaStream_t st)
{
    const cudaError_t e = launch_in_row(kda_verify_stats_kernel<T, STATS_VECS>, (unsigned)(p.chunks * p.B * (p.K + 1)), THREADS, 0, 1, st, p);
    return e != cudaSuccess ? e : launch_in_row(kda_verify_pick_kernel<T>, (unsigned)p.B * CLUSTER, THREADS, 0, CLUSTER, st, p);
}

}  // namespace

// Logits of a chunk; a row that starts off a 16-byte boundary reaches up to 7 further into them.
static int verify_chunk(kda_dtype_t dtype) { return THREADS * STATS_VECS * 16 / (dtype == KDA_DTYPE_BF16 ? 2 : 4); }
static int verify_chunks(kda_dtype_t dtype, int V)
{
    return (V + (dtype == KDA_DTYPE_BF16 ? 7 : 3) + verify_chunk(dtype) - 1) / verify_chunk(dtype);
}
static bool verify_sizes(kda_dtype_t dtype, int B, int K, int V)
{
    return B >= 1 && K >= 0 && V >= 1 && (dtype == KDA_DTYPE_BF16 || dtype == KDA_DTYPE_FP32);
}
static bool verify_fits(kda_dtype_t dtype, int B, int K, int V)
{
    return K <= MAX_DRAFTS && V <= (1 << 24) && (int64_t)B * (K + 1) * verify_chunks(dtype, V) <= INT32_MAX &&
           B <= INT32_MAX / CLUSTER;
}

static kda_status_t check_verify(const void *logits, kda_dtype_t dtype, int64_t row_stride, const int32_t *drafts,
                                 const float *probs, const float *uniform, const float *noise, const float *temperature,
                                 const int32_t *draft_lens, const int32_t *tokens, const int32_t *counts, int B, int K, int V)
{
    if (!verify_sizes(dtype, B, K, V))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!verify_fits(dtype, B, K, V))
        return KDA_ERR_UNSUPPORTED;
    if (!logits || !noise || !tokens || !counts || row_stride < V || (K > 0 && (!drafts || !uniform)))
        return KDA_ERR_INVALID_ARGUMENT;
    const size_t size = dtype == KDA_DTYPE_BF16 ? 2 : 4;
    if (!is_aligned(logits, size))
        return KDA_ERR_INVALID_ARGUMENT;
    const uint64_t rows = (uint64_t)B * (K + 1), n = (uint64_t)B * K * 4;
    const struct {
        const void *p;
        uint64_t bytes;
    } read[] = {{logits, ((rows - 1) * (uint64_t)row_stride + V) * size}, {drafts, n}, {probs, n * V}, {uniform, n},
                {noise, (uint64_t)B * V * 4}, {temperature, (uint64_t)B * 4}, {draft_lens, (uint64_t)B * 4}};
    for (int i = 1; i < 7; i++)
        if (!is_aligned(read[i].p, 4))
            return KDA_ERR_INVALID_ARGUMENT;
    if (!is_aligned(tokens, 4) || !is_aligned(counts, 4) || overlap(tokens, rows * 4, counts, (uint64_t)B * 4))
        return KDA_ERR_INVALID_ARGUMENT;
    for (const auto &r : read)
        if (overlap(tokens, rows * 4, r.p, r.bytes) || overlap(counts, (uint64_t)B * 4, r.p, r.bytes))
            return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

}  // namespace kda

using namespace kda;

extern "C" size_t kda_verify_drafts_workspace_size(kda_dtype_t dtype, int B, int K, int V)
{
    if (!verify_sizes(dtype, B, K, V) || !verify_fits(dtype, B, K, V))
        return 0;
    return (size_t)B * (K + 1) * verify_chunks(dtype, V) * sizeof(float2);
}

extern "C" kda_status_t kda_verify_drafts_ws(const void *logits, kda_dtype_t dtype, int64_t row_stride,
                                             const int32_t *draft_tokens, const float *draft_probs, const float *uniform,
                                             const float *noise, const float *temperature, const int32_t *draft_lens,
                                             int32_t *tokens, int32_t *counts, int B, int K, int V, void *workspace,
                                             size_t workspace_bytes, kda_stream_t stream)
{
    const kda_status_t s = check_verify(logits, dtype, row_stride, draft_tokens, draft_probs, uniform, noise, temperature,
                                        draft_lens, tokens, counts, B, K, V);
    if (s != KDA_OK)
        return s;
    if (!workspace || !is_aligned(workspace, 256) || workspace_bytes < kda_verify_drafts_workspace_size(dtype, B, K, V))
        return KDA_ERR_INVALID_ARGUMENT;
    VerifyArgs p{logits, row_stride, draft_tokens, draft_probs, uniform, noise, temperature, draft_lens, tokens, counts, B, K, V};
    p.chunk = verify_chunk(dtype), p.chunks = verify_chunks(dtype, V);
    p.stats = static_cast<float2 *>(workspace);
    if (step_error_word(&p.err) != cudaSuccess)
        return KDA_ERR_CUDA;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == KDA_DTYPE_BF16 ? launch_verify<__nv_bfloat16>(p, st) : launch_verify<float>(p, st);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_verify_drafts(const void *logits, kda_dtype_t dtype, int64_t row_stride,
                                          const int32_t *draft_tokens, const float *draft_probs, const float *uniform,
                                          const float *noise, const float *temperature, const int32_t *draft_lens,
                                          int32_t *tokens, int32_t *counts, int B, int K, int V, kda_stream_t stream)
{
    const kda_status_t c = check_verify(logits, dtype, row_stride, draft_tokens, draft_probs, uniform, noise, temperature,
                                        draft_lens, tokens, counts, B, K, V);
    if (c != KDA_OK)
        return c;
    const size_t need = kda_verify_drafts_workspace_size(dtype, B, K, V);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    void *ws = nullptr;
    if (pool_alloc(&ws, need, st) != cudaSuccess)
        return KDA_ERR_CUDA;
    kda_status_t s = kda_verify_drafts_ws(logits, dtype, row_stride, draft_tokens, draft_probs, uniform, noise, temperature,
                                          draft_lens, tokens, counts, B, K, V, ws, need, stream);
    if (cudaFreeAsync(ws, st) != cudaSuccess && s == KDA_OK)
        s = KDA_ERR_CUDA;
    return s;
}
