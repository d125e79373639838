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
// draft's row r and the noise, a share of the vocabulary a CTA; the shares' best meet in shared memory.  The race is run on
// (e_t - q_t z) / E_t, z = sum e: no division by z.
//
// Measured (one GPU): 64 requests of 4 drafts, 131072 fp32 logits and the drafts' distributions (235 MB) 43 us, 5.5 TB/s, of which the
// statistics take 30 (5.6 TB/s) and the pick the rest: a cluster waits for its rows' statistics, reads one row, and waits for the shares.
// 128 requests of 3 looked-up drafts, 50257 bf16 logits, 23.3 us; one of 4 drafts, 32001 bf16 logits, 6.2 us: two launches.
#include "kda_step.cuh"

#include <cfloat>
#include <cmath>

namespace kda {
namespace {

constexpr int THREADS = 128;                // of the statistics
constexpr int PICK_THREADS = 512;
constexpr int CLUSTER = 8;                  // CTAs of a request in the pick, at most
constexpr int AHEAD = 8;                    // tokens of a thread whose loads are in flight
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
    int chunks, chunk_vecs;      // chunks of a row, 16-byte vectors of a chunk
    int cluster;                 // CTAs of a request in the pick
    bool first;                  // greedy: a draft that ties for the largest stands only where it is the first of them
    float2 *stats;               // [B (K + 1)][chunks]: maximum, sum of exponentials or (greedy, first) its lowest index  (workspace)
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
__device__ __forceinline__ float given_temperature(const VerifyArgs &p, int b) { return p.temperature ? p.temperature[b] : 1.0f; }
__device__ __forceinline__ float checked_temperature(float t, bool &bad)
{
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

template <typename T> __device__ __forceinline__ uint4 lowest()
{
    const uint32_t w = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;   // -inf
    return make_uint4(w, w, w, w);
}
__device__ __forceinline__ uint32_t word_of(const uint4 &x, int i) { return i == 0 ? x.x : (i == 1 ? x.y : (i == 2 ? x.z : x.w)); }
__device__ __forceinline__ void set_word(uint4 &x, int i, uint32_t w)
{
    x.x = i == 0 ? w : x.x, x.y = i == 1 ? w : x.y, x.z = i == 2 ? w : x.z, x.w = i == 3 ? w : x.w;
}
__device__ __forceinline__ void put(uint4 &x, int e, float v) { set_word(x, e, __float_as_uint(v)); }
__device__ __forceinline__ void put(uint4 &x, int e, __nv_bfloat16 v)
{
    const uint32_t w = word_of(x, e / 2), b = __bfloat16_as_ushort(v);
    set_word(x, e / 2, e & 1 ? (w & 0xffffu) | b << 16 : (w & 0xffff0000u) | b);
}
__device__ __forceinline__ uint32_t bf16_max(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// The largest of a thread's elements
template <typename T, int N> __device__ __forceinline__ float largest(const uint4 (&x)[N])
{
    if constexpr (sizeof(T) == 2) {
        uint32_t m = bf16_max(bf16_max(x[0].x, x[0].y), bf16_max(x[0].z, x[0].w));
#pragma unroll
        for (int i = 1; i < N; i++)
            m = bf16_max(m, bf16_max(bf16_max(x[i].x, x[i].y), bf16_max(x[i].z, x[i].w)));
        return fmaxf(fmaxf(bf16_lo(m), bf16_hi(m)), -INFINITY);
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; i++)
            m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(x[i].x), __uint_as_float(x[i].y)), fmaxf(__uint_as_float(x[i].z), __uint_as_float(x[i].w))));
        return m;
    }
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

__device__ __forceinline__ int block_min(int x, float *sm)
{
    x = __reduce_min_sync(FULL, x);
    if ((threadIdx.x & 31) == 0)
        sm[threadIdx.x / 32] = __int_as_float(x);
    __syncthreads();
    x = __float_as_int(sm[0]);
#pragma unroll
    for (int i = 1; i < THREADS / 32; i++)
        x = min(x, __float_as_int(sm[i]));
    return x;
}

// log2(e) / tau, kept finite so that a logit at the maximum still gets weight 1 for the smallest tau.  One number is enough for the statistics:
// its rounding (2^-23.7 at most, the constant's included) counts times the exponent, which is taken from the chunk's own maximum.  The weights of 4096 or 8192
// tokens matter up to some 8 below it, so a sum is off by 2^-21 at the worst (each chunk a token beside a body 7 below it), by 2^-24
// where one chunk alone has the row's peak.  A second term here: 64 requests of 4 drafts 44.3 us for 43.5.
__device__ __forceinline__ float exponent_scale(float tau) { return fminf(LOG2E / tau, FLT_MAX); }

// One chunk of one row a CTA: at most VECS 16-byte vectors a thread.  The row may start anywhere: vectors are cut at 16-byte
// boundaries of memory, and one that reaches over an end of the row is read element by element.
template <typename T, int VECS> __global__ void __launch_bounds__(THREADS, 8) kda_verify_stats_kernel(const VerifyArgs p)
{
    constexpr int E = 16 / sizeof(T);
    __shared__ float sm[2][THREADS / 32];
    const int row = blockIdx.x / p.chunks, c = blockIdx.x % p.chunks, b = row / (p.K + 1);
    const int tid = threadIdx.x;
    stream_order();
    bool bad = false;
    const float given = given_temperature(p, b);
    if (row - b * (p.K + 1) > drafts_of(p, b, bad))
        return;                                     // behind the request's last draft
    const T *l = static_cast<const T *>(p.logits) + row * p.row_stride;
    const int off = (int)((reinterpret_cast<uintptr_t>(l) & 15) / sizeof(T));
    uint4 x[VECS];                                  // as they lie in memory: half the registers of floats for bf16
#pragma unroll
    for (int i = 0; i < VECS; i++) {
        const int v = i * THREADS + tid, at = (c * p.chunk_vecs + v) * E - off;   // first element of the vector
        const bool mine = v < p.chunk_vecs;
        if (mine && at >= 0 && at + E <= p.V) {
            x[i] = __ldcg(reinterpret_cast<const uint4 *>(l + at));
        } else {
            x[i] = lowest<T>();
            if (mine)
                for (int e = 0; e < E; e++)
                    if (at + e >= 0 && at + e < p.V)
                        put(x[i], e, l[at + e]);
        }
    }
    const float tau = checked_temperature(given, bad);    // (looked at here: the logits' loads do not wait for it)
    float m = largest<T>(x);                        // (NaN left out)
    m = block_max(m, sm[0]);
    float s = 0.0f;
    if (tau > 0.0f && m > -INFINITY) {
        const float f = exponent_scale(tau);
        const f2 f2f = f2_pack(f, f), minus_m = f2_pack(-m, -m), one = f2_pack(1.0f, 1.0f);
        f2 s2 = 0;
#pragma unroll
        for (int i = 0; i < VECS; i++)
        {
            float u[E];
            unpack<T>(x[i], u);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const f2 y = f2_mul(f2_fma(f2_pack(u[e], u[e + 1]), one, minus_m), f2f);
                s2 = f2_fma(f2_pack(ex2_approx(f2_lo(y)), ex2_approx(f2_hi(y))), one, s2);
            }
        }
        s = f2_lo(s2) + f2_hi(s2);
        if (s != s) {                               // a NaN among them (or an infinite maximum): those that are none
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < VECS; i++) {
                float u[E];
                unpack<T>(x[i], u);
#pragma unroll
                for (int e = 0; e < E; e++) {
                    const float y = ex2_approx((u[e] - m) * f);
                    s += y == y ? y : 0.0f;
                }
            }
        }
    }
    if (p.first && tau == 0.0f) {
        int at = INT32_MAX;                         // the lowest index of the maximum
#pragma unroll
        for (int i = VECS - 1; i >= 0; i--) {
            float u[E];
            unpack<T>(x[i], u);
#pragma unroll
            for (int e = E - 1; e >= 0; e--)
                at = u[e] == m ? (c * p.chunk_vecs + i * THREADS + tid) * E - off + e : at;
        }
        s = __int_as_float(block_min(at, sm[1]));
    } else {
        s = block_sum(s, sm[1]);
    }
    if (tid == 0)
        p.stats[(int64_t)row * p.chunks + c] = make_float2(m, s);
}

// exp(d / tau) for d <= 0: the exponent in base 2 as two terms, so that its rounding does not grow with it.  0 for NaN.
struct Exponent {
    float hi, lo;                       // log2(e) / tau
};
__device__ __forceinline__ Exponent exponent_of(float tau)
{
    constexpr float LOG2E_LO = (float)(1.4426950408889634074 - (double)LOG2E);
    const float hi = exponent_scale(tau);
    return Exponent{hi, hi < FLT_MAX ? (fmaf(-hi, tau, LOG2E) + LOG2E_LO) / tau : 0.0f};
}
__device__ __forceinline__ float weight_of(float d, const Exponent &f)
{
    constexpr float LN2 = 0.6931471805599453f;
    const float t = d * f.hi, r = fmaf(d, f.lo, fmaf(d, f.hi, -t)), y = ex2_approx(t);
    return t > -150.0f ? fmaf(y, r * LN2, y) : 0.0f;       // (below that nothing is left, and r is none for -inf)
}

__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int rank)
{
    uint32_t x;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(x) : "r"(addr), "r"(rank));
    return x;
}

// Four neighbouring elements
__device__ __forceinline__ void read_four(const float *p, float *x)
{
    const float4 y = *reinterpret_cast<const float4 *>(p);
    x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
}
__device__ __forceinline__ void read_four(const __nv_bfloat16 *p, float *x)
{
    const uint2 y = *reinterpret_cast<const uint2 *>(p);
    x[0] = bf16_lo(y.x), x[1] = bf16_hi(y.x), x[2] = bf16_lo(y.y), x[3] = bf16_hi(y.y);
}

// A cluster a request.  W neighbouring tokens a thread: 4 where all rows begin on 16 bytes (8 of bf16) and no row ends within four, else 1
// (64 requests of 4 drafts, fp32, statistics included: 44.4 us with 4, 46.8 with 1).  PROBS: the drafts were drawn, not looked up (without
// a kernel of their own these take 24.2 us for 23.3).
template <typename T, int W, bool PROBS> __global__ void __launch_bounds__(PICK_THREADS, 2) kda_verify_pick_kernel(const VerifyArgs p)
{
    __shared__ float row_max[MAX_DRAFTS + 1], row_sum[MAX_DRAFTS + 1];
    __shared__ int row_ok[MAX_DRAFTS + 1];
    __shared__ unsigned long long best_of[PICK_THREADS / 32], best_cta[2][CLUSTER];
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // waited for before anything is sent: every CTA has begun
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int b = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
    const int share = (p.V + p.cluster * W - 1) / (p.cluster * W) * W, from = rank * share, to = min(p.V, from + share);
    const float *noise = p.noise + (int64_t)b * p.V;
    stream_order();
    // the first tokens' noise, which does not depend on what is decided
    auto token = [](int t0, int i) { return t0 + i / W * W * PICK_THREADS + i % W; };   // a thread's i-th
    const int own = from + tid * W;
    float ahead[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; i += W) {
        const int t = token(own, i);
        if constexpr (W == 1)
            ahead[i] = t < to ? noise[t] : -1.0f;
        else if (t < to)
            read_four(noise + t, &ahead[i]);
    }
    // What the rows' tests need, of every row a warp may have: loads that wait for no length and no temperature.
    const T *logits = static_cast<const T *>(p.logits) + (int64_t)b * (p.K + 1) * p.row_stride;
    const float2 *stats = p.stats + (int64_t)b * (p.K + 1) * p.chunks;
    constexpr int WARPS = PICK_THREADS / 32, ROWS = (MAX_DRAFTS + WARPS) / WARPS;
    const float2 none = make_float2(-INFINITY, 0.0f);
    float2 first[ROWS];
    int draft[ROWS];
    float drafted[ROWS], bar[ROWS];                 // the draft's logit, and u q of it
    bool there[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; k++) {
        const int i = warp + k * WARPS;
        draft[k] = i < p.K ? p.drafts[b * p.K + i] : -1;
        bar[k] = i < p.K ? p.uniform[b * p.K + i] : 0.0f;
        first[k] = i <= p.K && lane < p.chunks ? __ldcg(&stats[i * p.chunks + lane]) : none;
    }
#pragma unroll
    for (int k = 0; k < ROWS; k++) {
        const int i = warp + k * WARPS;
        there[k] = draft[k] >= 0 && draft[k] < p.V;
        drafted[k] = there[k] ? logit(as_float(logits[i * p.row_stride + draft[k]])) : -INFINITY;
        if (PROBS && there[k])
            bar[k] *= p.probs[((int64_t)b * p.K + i) * p.V + draft[k]];
    }
    bool bad = false;
    const int L = drafts_of(p, b, bad);
    const float tau = checked_temperature(given_temperature(p, b), bad);
    const bool greedy = tau == 0.0f;
    const Exponent f = exponent_of(greedy ? 1.0f : tau);
#pragma unroll
    for (int k = 0; k < ROWS; k++) {
        const int i = warp + k * WARPS;
        if (i > L)
            break;                                  // (no statistics behind the last draft's)
        const float2 *st = stats + i * p.chunks;
        bad |= i < L && !there[k];
        float m = first[k].x, z = 0.0f;
        for (int c = lane + 32; c < p.chunks; c += 32)
            m = fmaxf(m, __ldcg(&st[c].x));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
        if (!greedy) {
            z = first[k].x == -INFINITY ? 0.0f : first[k].y * weight_of(first[k].x - m, f);
            for (int c = lane + 32; c < p.chunks; c += 32) {
                const float2 x = __ldcg(&st[c]);
                z += x.x == -INFINITY ? 0.0f : x.y * weight_of(x.x - m, f);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            z += __shfl_xor_sync(FULL, z, o);
        if (lane == 0) {
            // a row without a finite maximum, and a draft that cannot be, accept nothing
            const bool can = i < L && there[k] && fabsf(m) <= FLT_MAX && drafted[k] > -INFINITY;
            row_ok[i] = can && (greedy ? drafted[k] == m : bar[k] * z < weight_of(drafted[k] - m, f));
            row_max[i] = m, row_sum[i] = z;
        }
    }
    if (greedy && p.first) {                        // of the largest only the first
        __syncwarp();
#pragma unroll
        for (int k = 0; k < ROWS; k++) {
            const int i = warp + k * WARPS;
            if (i >= L)
                break;
            const float m = row_max[i];
            int lowest = first[k].x == m ? __float_as_int(first[k].y) : INT32_MAX;
            for (int c = lane + 32; c < p.chunks; c += 32) {
                const float2 x = __ldcg(&stats[i * p.chunks + c]);
                lowest = x.x == m ? min(lowest, __float_as_int(x.y)) : lowest;
            }
            lowest = __reduce_min_sync(FULL, lowest);
            if (lane == 0 && draft[k] != lowest)
                row_ok[i] = 0;
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
    const float *q = PROBS && r < L ? p.probs + ((int64_t)b * p.K + r) * p.V : nullptr;
    // the best of the race: its value's bits above the complement of its index, so that ties go to the lower one
    unsigned long long best = 0;
    for (int pass = 0; pass < 2; pass++) {
        float most = 0.0f;
        int at = 0;
        // a thread's tokens in order: the first of equal ones stays
        auto take = [&](float v, int t) {
            if (v > most)
                most = v, at = t;
        };
        auto scan = [&](auto value) {
            for (int t0 = own; t0 < to; t0 += AHEAD * PICK_THREADS) {
                float lt[AHEAD], e[AHEAD], qt[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; i += W) {
                    const int t = token(t0, i);
                    const bool in = t < to;
                    if constexpr (W == 1) {
                        lt[i] = in ? as_float(l[t]) : -INFINITY;
                        e[i] = pass == 0 && t0 == own ? ahead[i] : (in ? noise[t] : -1.0f);
                        qt[i] = in && q && pass == 0 ? q[t] : 0.0f;
                    } else {
#pragma unroll
                        for (int w = i; w < i + W; w++)
                            lt[w] = -INFINITY, e[w] = ahead[w], qt[w] = 0.0f;
                        if (in) {
                            read_four(l + t, &lt[i]);
                            if (pass > 0 || t0 != own)
                                read_four(noise + t, &e[i]);
                            if (q && pass == 0)
                                read_four(q + t, &qt[i]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < AHEAD; i++)
                    take(value(lt[i], e[i], qt[i], token(t0, i)), token(t0, i));
            }
        };
        if (!alive) {
        } else if (greedy) {
            scan([&](float lt, float, float, int) { return lt == m ? 1.0f : 0.0f; });
        } else {
            const int without = q || pass > 0 ? -1 : x;       // a certain draft that was rejected
            scan([&](float lt, float e, float qt, int t) {
                const float w = fmaf(-qt, z, weight_of(lt - m, f));
                return t != without && w > 0.0f ? w * rcp_approx(e) : 0.0f;
            });
        }
        best = most > 0.0f ? ((unsigned long long)__float_as_uint(most) << 32) | (uint32_t)~at : 0ull;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long y = __shfl_xor_sync(FULL, best, o);
            best = y > best ? y : best;
        }
        if (lane == 0)
            best_of[warp] = best;
        __syncthreads();
        if (pass == 0)
            asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        if (tid < p.cluster) {
            best = best_of[0];
#pragma unroll
            for (int i = 1; i < PICK_THREADS / 32; i++)
                best = best_of[i] > best ? best_of[i] : best;
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(in_cta(smem_u32(&best_cta[pass][rank]), tid)), "l"(best) : "memory");
        }
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
        best = 0;
        for (int i = 0; i < p.cluster; i++)
            best = best_cta[pass][i] > best ? best_cta[pass][i] : best;
        if (best != 0 || r == L || !alive)           // the same in every CTA of the cluster
            break;
        // nothing is left over (rounding): the race is run on p itself
    }
    if (rank == 0) {
        const int token = best ? (int)~(uint32_t)best : -1;
        for (int i = tid; i <= p.K; i += PICK_THREADS)
            p.tokens[b * (p.K + 1) + i] = i < r ? p.drafts[b * p.K + i] : (i == r ? token : -1);
        if (tid == 0)
            p.counts[b] = r + 1;
    }
    report(p.err, bad && rank == 0, DEVERR_CU_SEQLENS);
}

// 16-byte vectors of a thread of the statistics: 8, or 2 where that leaves most SMs without a CTA (one request of 5 x 32001 bf16
// logits: 6.3 us, with 8 6.8).
constexpr int VECS_MOST = 8, VECS_FEW = 2;

template <typename T> cudaError_t launch_verify(const VerifyArgs &p, cudaStream_t st)
{
    const unsigned grid = (unsigned)(p.chunks * p.B * (p.K + 1));
    const cudaError_t e = p.chunk_vecs > THREADS * VECS_FEW
                              ? launch_in_row(kda_verify_stats_kernel<T, VECS_MOST>, grid, THREADS, 0, 1, st, p)
                              : launch_in_row(kda_verify_stats_kernel<T, VECS_FEW>, grid, THREADS, 0, 1, st, p);
    if (e != cudaSuccess)
        return e;
    const bool fours = p.V % 4 == 0 && p.row_stride % 4 == 0 && is_aligned(p.logits, 4 * sizeof(T)) && is_aligned(p.probs, 16) &&
                       is_aligned(p.noise, 16);
    const auto kernel = p.probs ? (fours ? kda_verify_pick_kernel<T, 4, true> : kda_verify_pick_kernel<T, 1, true>)
                                : (fours ? kda_verify_pick_kernel<T, 4, false> : kda_verify_pick_kernel<T, 1, false>);
    return launch_in_row(kernel, (unsigned)(p.B * p.cluster), PICK_THREADS, 0, p.cluster, st, p);
}

}  // namespace

// Vectors of a row (one that starts off a 16-byte boundary reaches into one more), its chunks, all of about the same size.
static int verify_vecs(kda_dtype_t dtype, int V)
{
    const int e = dtype == KDA_DTYPE_BF16 ? 8 : 4;
    return (V + 2 * e - 2) / e;
}
static int verify_chunks(kda_dtype_t dtype, int B, int K, int V)
{
    const int vecs = verify_vecs(dtype, V), large = (vecs + THREADS * VECS_MOST - 1) / (THREADS * VECS_MOST);
    return (int64_t)B * (K + 1) * large >= 2 * 152 ? large : (vecs + THREADS * VECS_FEW - 1) / (THREADS * VECS_FEW);
}
static bool verify_sizes(kda_dtype_t dtype, int B, int K, int V)
{
    return B >= 1 && K >= 0 && V >= 1 && (dtype == KDA_DTYPE_BF16 || dtype == KDA_DTYPE_FP32);
}
static bool verify_fits(kda_dtype_t dtype, int B, int K, int V)
{
    return K <= MAX_DRAFTS && V <= (1 << 24) && (int64_t)B * (K + 1) * verify_chunks(dtype, B, K, V) <= INT32_MAX &&
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
    return (size_t)B * (K + 1) * verify_chunks(dtype, B, K, V) * sizeof(float2);
}

extern "C" kda_status_t kda_verify_drafts_opt(const void *logits, kda_dtype_t dtype, int64_t row_stride,
                                              const int32_t *draft_tokens, const float *draft_probs, const float *uniform,
                                              const float *noise, const float *temperature, const int32_t *draft_lens,
                                              int32_t *tokens, int32_t *counts, int B, int K, int V, uint32_t options,
                                              void *workspace, size_t workspace_bytes, kda_stream_t stream)
{
    const kda_status_t s = check_verify(logits, dtype, row_stride, draft_tokens, draft_probs, uniform, noise, temperature,
                                        draft_lens, tokens, counts, B, K, V);
    if (s != KDA_OK)
        return s;
    if (options & ~KDA_VERIFY_FIRST_LARGEST)
        return KDA_ERR_INVALID_ARGUMENT;
    const size_t need = kda_verify_drafts_workspace_size(dtype, B, K, V);
    const bool pool = !workspace && workspace_bytes == 0;
    if (!pool && (!workspace || !is_aligned(workspace, 256) || workspace_bytes < need))
        return KDA_ERR_INVALID_ARGUMENT;
    VerifyArgs p{logits, row_stride, draft_tokens, draft_probs, uniform, noise, temperature, draft_lens, tokens, counts, B, K, V};
    p.chunks = verify_chunks(dtype, B, K, V);
    p.chunk_vecs = (verify_vecs(dtype, V) + p.chunks - 1) / p.chunks;
    // as many CTAs as run at once, two an SM: more of them wait for a place and then for the same chain of loads (128 requests of 3
    // drafts, 50257 bf16 logits, statistics included: 8 CTAs a request 38.6 us, 2 30.1)
    p.cluster = CLUSTER;
    while (p.cluster > 1 && (int64_t)B * p.cluster > 2 * 152)
        p.cluster /= 2;
    p.first = options & KDA_VERIFY_FIRST_LARGEST;
    if (step_error_word(&p.err) != cudaSuccess)
        return KDA_ERR_CUDA;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (pool && pool_alloc(&workspace, need, st) != cudaSuccess)
        return KDA_ERR_CUDA;
    p.stats = static_cast<float2 *>(workspace);
    cudaError_t e = dtype == KDA_DTYPE_BF16 ? launch_verify<__nv_bfloat16>(p, st) : launch_verify<float>(p, st);
    const cudaError_t freed = pool ? cudaFreeAsync(workspace, st) : cudaSuccess;
    return e == cudaSuccess && freed == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_verify_drafts_ws(const void *logits, kda_dtype_t dtype, int64_t row_stride,
                                             const int32_t *draft_tokens, const float *draft_probs, const float *uniform,
                                             const float *noise, const float *temperature, const int32_t *draft_lens,
                                             int32_t *tokens, int32_t *counts, int B, int K, int V, void *workspace,
                                             size_t workspace_bytes, kda_stream_t stream)
{
    // (none at all would be the pool's)
    return kda_verify_drafts_opt(logits, dtype, row_stride, draft_tokens, draft_probs, uniform, noise, temperature, draft_lens,
                                 tokens, counts, B, K, V, 0, workspace, workspace ? workspace_bytes : 1, stream);
}

extern "C" kda_status_t kda_verify_drafts(const void *logits, kda_dtype_t dtype, int64_t row_stride,
                                          const int32_t *draft_tokens, const float *draft_probs, const float *uniform,
                                          const float *noise, const float *temperature, const int32_t *draft_lens,
                                          int32_t *tokens, int32_t *counts, int B, int K, int V, kda_stream_t stream)
{
    return kda_verify_drafts_opt(logits, dtype, row_stride, draft_tokens, draft_probs, uniform, noise, temperature, draft_lens,
                                 tokens, counts, B, K, V, 0, nullptr, 0, stream);
}
