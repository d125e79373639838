// kda_beam_select: log-softmax of the beams' logits, and the K best of a batch entry's beams x vocabulary.
//
// Score of candidate (w, t): fl(c + l[t]), c = (score_w - m) - log sum exp(l - m).  c is known only when the row has
// been read to its end, but fl(c + l) never falls as l rises: so one pass over the logits keeps, for every chunk of a
// row, the chunk's maximum and sum and its K + 1 best logits (kda_beam_chunks_kernel), and a second kernel, one CTA a
// batch entry, turns those few into scores and picks (kda_beam_pick_kernel).  Each logit is read once: the floor.
//
// What the short lists may hide: logits so close that their fp32 scores are equal tie by index and not by logit.  That
// matters only where a chunk's last kept logit reaches the K-th score and a neighbouring logit value has the same score
// too; the pick then goes over all candidates of the entry again (pick_all).
//
// The best of many.  Candidates are 64-bit keys, order-preserving bits of the value above the complement of the index,
// so all are distinct and a tie goes to the lower index.  The n-th best of the thread groups' best keys is a lower
// bound on the n-th best key, and at most n groups have keys from it up: those are gathered in shared memory and each
// ranked by counting the larger ones.
#include "kda_step.cuh"

#include <cfloat>

namespace kda {
namespace {

constexpr int THREADS = 256;
constexpr int CAP = 2048;                 // keys gathered for ranking
constexpr unsigned FULL = 0xffffffffu;

struct BeamArgs {
    const void *logits;
    int64_t row_stride;
    const float *beam_scores;
    const uint8_t *finished;
    int eos;
    float *scores;
    int32_t *tokens, *parents;
    int B, W, V, K;
    int chunks;              // of a row
    float2 *stats;           // [B W][chunks]: maximum, sum of exp(l - maximum)   (workspace)
    uint64_t *lists;         // [B W][chunks][K + 1]: best logits' keys, 0 past the last
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

// A value next to x in T's numbers: above or below (x finite or infinite, not NaN).
__device__ __forceinline__ float neighbour(float x, bool up, bool bf16)
{
    const uint32_t step = bf16 ? 0x10000u : 1u;
    uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);
    if (u == 0)
        return __uint_as_float(up ? step : (0x80000000u | step));
    if (!(u & 0x80000000u))
        u = up ? (u == 0x7f800000u ? u : u + step) : u - step;
    else
        u = up ? u - step : (u == 0xff800000u ? u : u + step);
    return __uint_as_float(u);
}

__device__ uint64_t block_max(uint64_t x, uint64_t *sh)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t y = __shfl_xor_sync(FULL, x, o);
        x = x > y ? x : y;
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0)
        sh[threadIdx.x / 32] = x;
    __syncthreads();
    x = sh[0];
#pragma unroll
    for (int i = 1; i < THREADS / 32; i++)
        x = x > sh[i] ? x : sh[i];
    return x;
}

struct Pick {
    uint64_t group[THREADS / 2];   // best key of each group of threads
    uint64_t cand[CAP];
    uint64_t red[THREADS / 32];
    uint64_t bound;
    int count;
};

// The n-th best of the groups' best keys (1 when fewer than n groups have one: every key is let through).  Groups of
// 4 threads while n <= 32, of 2 up to 65, so that there are twice as many groups as wanted keys and few get through.
__device__ uint64_t group_bound(Pick &sh, uint64_t best, int n)
{
    const int size = n <= 32 ? 4 : 2, groups = THREADS / size;
    uint64_t y = __shfl_xor_sync(FULL, best, 1);
    best = best > y ? best : y;
    y = __shfl_xor_sync(FULL, best, 2);
    if (size == 4)
        best = best > y ? best : y;
    if (threadIdx.x % size == 0)
        sh.group[threadIdx.x / size] = best;
    if (threadIdx.x == 0) {
        sh.bound = 1;
        sh.count = 0;
    }
    __syncthreads();
    if (threadIdx.x < groups) {
        const uint64_t x = sh.group[threadIdx.x];
        int rank = 0;
        const ulonglong2 *g = reinterpret_cast<const ulonglong2 *>(sh.group);
#pragma unroll 8
        for (int i = 0; i < groups / 2; i++) {
            const ulonglong2 v = g[i];
            rank += (v.x > x) + (v.y > x);
        }
        if (x != 0 && rank == n - 1)
            sh.bound = x;
    }
    __syncthreads();
    return sh.bound;
}

// The same on values alone: the n-th best (ties counted) of the groups' best values; below every value when there are
// fewer groups with one.
__device__ float group_bound_value(Pick &sh, float best, int n)
{
    const int size = n <= 32 ? 4 : 2, groups = THREADS / size;
    float *g = reinterpret_cast<float *>(sh.group);
    best = fmaxf(best, __shfl_xor_sync(FULL, best, 1));
    const float y = __shfl_xor_sync(FULL, best, 2);
    if (size == 4)
        best = fmaxf(best, y);
    if (threadIdx.x % size == 0)
        g[threadIdx.x / size] = best;
    uint32_t *lowest = reinterpret_cast<uint32_t *>(&sh.bound);
    if (threadIdx.x == 0) {
        *lowest = FULL;
        sh.count = 0;
    }
    __syncthreads();
    if (threadIdx.x < groups) {
        const float x = g[threadIdx.x];
        int above = 0;
        const float4 *q = reinterpret_cast<const float4 *>(g);
#pragma unroll 8
        for (int i = 0; i < groups / 4; i++) {
            const float4 v = q[i];
            above += (v.x > x) + (v.y > x) + (v.z > x) + (v.w > x);
        }
        // the smallest of the values that fewer than n are above
        const uint32_t u = (uint32_t)(key_of(x, 0) >> 32);
        const uint32_t low = __reduce_min_sync(__activemask(), above < n ? u : FULL);
        if (threadIdx.x % 32 == 0)
            atomicMin(lowest, low);
    }
    __syncthreads();
    return key_value((uint64_t)*lowest << 32);
}

// Ranks the gathered keys (count of them, all distinct) and hands the best n to put(rank, key).
template <typename F> __device__ void rank_gathered(const Pick &sh, int count, int n, F put)
{
    for (int i = threadIdx.x; i < count; i += THREADS) {
        const uint64_t x = sh.cand[i];
        int rank = 0;
        for (int j = 0; j < count; j++)
            rank += sh.cand[j] > x;
        if (rank < n)
            put(rank, x);
    }
}

template <typename T> struct Vec {
    static constexpr int N = 16 / sizeof(T);
};
__device__ __forceinline__ void unpack(const uint4 &x, float *v, const float *)
{
    v[0] = __uint_as_float(x.x), v[1] = __uint_as_float(x.y), v[2] = __uint_as_float(x.z), v[3] = __uint_as_float(x.w);
}
__device__ __forceinline__ void unpack(const uint4 &x, float *v, const __nv_bfloat16 *)
{
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; i++)
        v[2 * i] = bf16_lo(u[i]), v[2 * i + 1] = bf16_hi(u[i]);
}

// The aligned 16 bytes that hold the row's elements from t on (t may be negative): one load where the row covers them,
// else element by element, zeros outside.
__device__ __forceinline__ uint4 load_aligned(const float *l, int t, int V)
{
    if (t >= 0 && t + 4 <= V)
        return __ldcs(reinterpret_cast<const uint4 *>(l + t));
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; e++)
        u[e] = t + e >= 0 && t + e < V ? __float_as_uint(l[t + e]) : 0;
    return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ uint4 load_aligned(const __nv_bfloat16 *l, int t, int V)
{
    if (t >= 0 && t + 8 <= V)
        return __ldcs(reinterpret_cast<const uint4 *>(l + t));
    uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; e++)
        if (t + e >= 0 && t + e < V)
            u[e / 2] |= (uint32_t)reinterpret_cast<const unsigned short *>(l)[t + e] << (16 * (e % 2));
    return make_uint4(u[0], u[1], u[2], u[3]);
}
// The row's 16 bytes from element t on, in a row that lies `off` bytes past a 16-byte boundary: two aligned vectors, the
// second one the next lane's first, shifted together.  By a whole warp, lane i at t + i * (16 / size).
template <typename T> __device__ __forceinline__ uint4 load_shifted(const T *l, int t, int off, int V)
{
    const int back = off / (int)sizeof(T);
    const uint4 a = load_aligned(l, t - back, V);
    if (off == 0)
        return a;
    uint4 b;
    b.x = __shfl_down_sync(FULL, a.x, 1);
    b.y = __shfl_down_sync(FULL, a.y, 1);
    b.z = __shfl_down_sync(FULL, a.z, 1);
    b.w = __shfl_down_sync(FULL, a.w, 1);
    if ((threadIdx.x & 31) == 31)
        b = load_aligned(l, t - back + 16 / (int)sizeof(T), V);
    uint32_t x[5];
    const int words = off / 4;
    if (words == 0)
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x;
    else if (words == 1)
        x[0] = a.y, x[1] = a.z, x[2] = a.w, x[3] = b.x, x[4] = b.y;
    else if (words == 2)
        x[0] = a.z, x[1] = a.w, x[2] = b.x, x[3] = b.y, x[4] = b.z;
    else
        x[0] = a.w, x[1] = b.x, x[2] = b.y, x[3] = b.z, x[4] = b.w;
    if (off & 2)
        return make_uint4(__funnelshift_r(x[0], x[1], 16), __funnelshift_r(x[1], x[2], 16),
                          __funnelshift_r(x[2], x[3], 16), __funnelshift_r(x[3], x[4], 16));
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// One CTA per (chunk, row): PER logits a thread in registers, 16-byte vectors strided over the CTA.  Which thread takes
// which token, and so the order of the sums, does not depend on the row's alignment: equal rows get equal scores.
template <typename T, int PER> __global__ void __launch_bounds__(THREADS, PER > 16 ? 4 : 6) kda_beam_chunks_kernel(const BeamArgs p)
{
    constexpr int N = Vec<T>::N;
    __shared__ __align__(16) Pick sh;
    __shared__ float2 part[THREADS / 32];
    asm volatile("griddepcontrol.launch_dependents;");
    const int64_t row = blockIdx.x / p.chunks;
    const int chunk = (int)(blockIdx.x % p.chunks);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, n = p.K + 1;
    if (p.finished && p.finished[row])
        return;                              // its one candidate needs no logits
    const T *l = static_cast<const T *>(p.logits) + row * p.row_stride;
    const int off = (int)(reinterpret_cast<uintptr_t>(l) & 15);
    const int first = chunk * (THREADS * PER);       // token of the chunk's first element
    const bool whole = first + THREADS * PER <= p.V;
    float v[PER];
#pragma unroll
    for (int i = 0; i < PER / N; i++)
        unpack(load_shifted(l, first + (i * THREADS + tid) * N, off, p.V), v + i * N, l);
    auto token = [&](int i) { return first + ((i / N) * THREADS + tid) * N + i % N; };
    if (!whole) {
#pragma unroll
        for (int i = 0; i < PER; i++)
            v[i] = token(i) < p.V ? v[i] : -INFINITY;
    }
    // maximum and sum of the chunk, warp by warp (fmaxf passes over NaN)
    float best = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; i++)
        best = fmaxf(best, v[i]);
    float m = best;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
    const float mu = fabsf(m) <= FLT_MAX ? m : 0.0f;
    // exp(v - mu) = 2^(v L - c) 2^(c - mu L), c = mu L rounded: the second factor is one for the whole warp
    const float c = mu * LOG2E;
    const f2 scale = f2_pack(LOG2E, LOG2E), shift = f2_pack(-c, -c);
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
        const f2 x = f2_fma(f2_pack(v[i], v[i + 1]), scale, shift);
        s0 += ex2_approx(f2_lo(x));
        s1 += ex2_approx(f2_hi(x));
    }
    float sum = s0 + s1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(FULL, sum, o);
    sum *= ex2_approx(-fmaf(mu, LOG2E, -c));
    if (sum != sum || fabsf(mu) > 1e30f) {   // NaN logits (they count as -inf), or a product past fp32's range
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; i++) {
            v[i] = no_nan(v[i]);
            sum += ex2_approx((v[i] - mu) * LOG2E);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(FULL, sum, o);
    }
    if (lane == 0)
        part[warp] = make_float2(m, sum);

    // In a whole chunk the bound is taken on values alone; a chunk with an end, one whose n-th value is not finite, and
    // one with more ties than can be gathered go by keys.
    bool done = false;
    if (whole) {
        const float bound = group_bound_value(sh, best, n);
        if (fabsf(bound) <= FLT_MAX) {
            if (best >= bound) {
#pragma unroll
                for (int i = 0; i < PER; i++)
                    if (v[i] >= bound) {
                        const int to = atomicAdd(&sh.count, 1);
                        if (to < CAP)
                            sh.cand[to] = key_of(v[i], token(i));
                    }
            }
            __syncthreads();
            done = sh.count <= CAP;
            __syncthreads();
        }
    }
    if (!done) {
        uint64_t key = 0;
#pragma unroll
        for (int i = 0; i < PER; i++) {
            v[i] = no_nan(v[i]);
            const uint64_t x = token(i) < p.V ? key_of(v[i], token(i)) : 0;
            key = x > key ? x : key;
        }
        const uint64_t bound = group_bound(sh, key, n);
        if (key >= bound) {
#pragma unroll
            for (int i = 0; i < PER; i++) {
                const uint64_t x = token(i) < p.V ? key_of(v[i], token(i)) : 0;
                if (x >= bound) {
                    const int to = atomicAdd(&sh.count, 1);
                    if (to < CAP)
                        sh.cand[to] = x;
                }
            }
        }
        __syncthreads();
    }
    const int64_t slot = blockIdx.x;
    uint64_t *list = p.lists + slot * n;
    if (warp == 0) {
        const float2 x = lane < THREADS / 32 ? part[lane] : make_float2(-INFINITY, 0.0f);
        float M = x.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            M = fmaxf(M, __shfl_xor_sync(FULL, M, o));
        float s = fabsf(x.x) <= FLT_MAX ? x.y * expf(x.x - M) : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            s += __shfl_xor_sync(FULL, s, o);
        if (lane == 0)
            p.stats[slot] = make_float2(M, s);
    }
    const int count = sh.count;
    if (count <= CAP) {
        rank_gathered(sh, count, n, [&](int r, uint64_t k) { list[r] = k; });
        for (int r = count + tid; r < n; r += THREADS)
            list[r] = 0;
    } else {
        // more than can be gathered (large values crowded into few threads): one at a time
        uint64_t last = ~0ull;
        for (int r = 0; r < n; r++) {
            uint64_t b = 0;
#pragma unroll
            for (int i = 0; i < PER; i++) {
                const uint64_t x = token(i) < p.V ? key_of(v[i], token(i)) : 0;
                if (x < last && x > b)
                    b = x;
            }
            last = block_max(b, sh.red);
            if (tid == 0)
                list[r] = last;
        }
    }
}

// Score of a candidate whose beam has offset c (-inf: nothing of the beam counts) and logit l.
__device__ __forceinline__ float score_of(float c, float l) { return c == -INFINITY ? c : no_nan(c + l); }

// The K best of all W x V candidates, one pass for each: what the short lists are a shortcut of.
template <typename T> __device__ void pick_all(const BeamArgs &p, int b, const float *c, uint64_t *red)
{
    uint64_t last = ~0ull;
    for (int k = 0; k < p.K; k++) {
        uint64_t best = 0;
        for (int w = 0; w < p.W; w++) {
            const int64_t row = (int64_t)b * p.W + w;
            const T *l = static_cast<const T *>(p.logits) + row * p.row_stride;
            const bool done = p.finished && p.finished[row];
            for (int t = threadIdx.x; t < p.V; t += THREADS) {
                const float s = done ? (t == p.eos ? no_nan(p.beam_scores[row]) : -INFINITY)
                                     : score_of(c[w], no_nan(load_logit(l + t)));
                const uint64_t x = key_of(s, (uint32_t)w * p.V + t);
                if (x < last && x > best)
                    best = x;
            }
        }
        last = block_max(best, red);
        if (threadIdx.x == 0) {
            p.scores[(int64_t)b * p.K + k] = key_value(last);
            p.tokens[(int64_t)b * p.K + k] = key_index(last) % p.V;
            p.parents[(int64_t)b * p.K + k] = b * p.W + key_index(last) / p.V;
        }
    }
}

// One CTA per batch entry.
template <typename T> __global__ void __launch_bounds__(THREADS) kda_beam_pick_kernel(const BeamArgs p)
{
    __shared__ __align__(16) Pick sh;
    __shared__ float c[32];
    __shared__ bool plain[32];             // the beam's candidates come from the lists
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid % 32, n = p.K + 1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int w = tid / 32; w < p.W; w += THREADS / 32) {
        const int64_t row = (int64_t)b * p.W + w;
        const bool done = p.finished && p.finished[row];
        float m = -INFINITY, s = 0.0f;
        if (!done) {
            const float2 *st = p.stats + row * p.chunks;
            for (int i = lane; i < p.chunks; i += 32)
                m = fmaxf(m, st[i].x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
            if (fabsf(m) <= FLT_MAX)
                for (int i = lane; i < p.chunks; i += 32)
                    s += st[i].y * expf(st[i].x - m);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                s += __shfl_xor_sync(FULL, s, o);
        }
        if (lane == 0) {
            c[w] = fabsf(m) <= FLT_MAX ? no_nan((p.beam_scores[row] - m) - logf(s)) : -INFINITY;
            plain[w] = !done && c[w] != -INFINITY;
        }
    }
    __syncthreads();
    // candidate i of beam w: a list entry, or for a beam whose candidates are all but one -inf its first tokens and eos
    const int64_t per = (int64_t)p.chunks * n, total = per * p.W;
    auto candidate = [&](int64_t x) -> uint64_t {
        const int w = (int)(x / per);
        const int64_t i = x % per, row = (int64_t)b * p.W + w;
        if (plain[w]) {
            const uint64_t k = p.lists[row * per + i];
            return k ? key_of(score_of(c[w], key_value(k)), (uint32_t)w * p.V + key_index(k)) : 0;
        }
        const bool done = p.finished && p.finished[row];
        int64_t t = i;
        if (i > p.K || (i == p.K && !(done && p.eos >= p.K)) || (i < p.K && i >= p.V))
            return 0;
        if (i == p.K)
            t = p.eos;
        return key_of(done && t == p.eos ? no_nan(p.beam_scores[row]) : -INFINITY, (uint32_t)w * p.V + (uint32_t)t);
    };
    uint64_t best = 0;
    for (int64_t x = tid; x < total; x += THREADS) {
        const uint64_t k = candidate(x);
        best = k > best ? k : best;
    }
    const uint64_t bound = group_bound(sh, best, p.K);
    if (best >= bound)
        for (int64_t x = tid; x < total; x += THREADS) {
            const uint64_t k = candidate(x);
            if (k >= bound && k) {
                const int to = atomicAdd(&sh.count, 1);
                if (to < CAP)
                    sh.cand[to] = k;
            }
        }
    __syncthreads();
    const int count = sh.count;
    bool again = count > CAP;
    if (!again) {
        // the K-th score, and whether a list may have cut off a logit that has it too
        if (tid == 0)
            sh.bound = 0;
        __syncthreads();
        rank_gathered(sh, count, p.K, [&](int r, uint64_t k) {
            if (r == p.K - 1)
                sh.bound = k;
            p.scores[(int64_t)b * p.K + r] = key_value(k);
            p.tokens[(int64_t)b * p.K + r] = key_index(k) % p.V;
            p.parents[(int64_t)b * p.K + r] = b * p.W + key_index(k) / p.V;
        });
        __syncthreads();
        const float last = key_value(sh.bound);
        for (int x = tid; x < p.W * p.chunks; x += THREADS) {
            const int w = x / p.chunks;
            if (!plain[w])
                continue;
            const uint64_t k = p.lists[((int64_t)b * p.W * p.chunks + x) * n + n - 1];
            if (!k)
                continue;
            const float l = key_value(k);
            if (score_of(c[w], l) == last && (score_of(c[w], neighbour(l, true, sizeof(T) == 2)) == last ||
                                              (l != -INFINITY &&
                                               score_of(c[w], neighbour(l, false, sizeof(T) == 2)) == last)))
                again = true;
        }
    }
    if (__syncthreads_or(again))
        pick_all<T>(p, b, c, sh.red);
}

}  // namespace

// Logits a thread holds.  Many make fewer lists to pick from; few put a small call's logits on more SMs.  See the
// comment at launch_beam for what was measured.
constexpr int PER_LARGE = 32, PER_SMALL = 8;

static int beam_per(int B, int W, int V)
{
    return (int64_t)B * W * ((V + THREADS * PER_LARGE - 1) / (THREADS * PER_LARGE)) >= 152 ? PER_LARGE : PER_SMALL;
}
static int beam_chunks(int B, int W, int V)
{
    const int chunk = THREADS * beam_per(B, W, V);
    return (V + chunk - 1) / chunk;
}

namespace {

template <typename T> cudaError_t launch_beam(const BeamArgs &p, cudaStream_t st)
{
    const unsigned grid = (unsigned)(p.chunks * p.B * p.W);
    if (beam_per(p.B, p.W, p.V) == PER_LARGE)
        kda_beam_chunks_kernel<T, PER_LARGE><<<grid, THREADS, 0, st>>>(p);
    else
        kda_beam_chunks_kernel<T, PER_SMALL><<<grid, THREADS, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.B);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kda_beam_pick_kernel<T>, p);
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
    if ((int64_t)B * W * beam_chunks(B, W, V) > INT32_MAX)
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
    if (B < 1 || W < 1 || W > 32 || V < 1 || V > (1 << 24) || K < 1 || K > 64 || (int64_t)K > (int64_t)W * V ||
        (int64_t)B * W > INT32_MAX)
        return 0;
    return (size_t)B * W * beam_chunks(B, W, V) * (sizeof(float2) + (K + 1) * sizeof(uint64_t));
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
    if (!workspace || !is_aligned(workspace, 256) || workspace_bytes < kda_beam_select_workspace_size(B, W, V, K))
        return KDA_ERR_INVALID_ARGUMENT;
    BeamArgs p{logits, row_stride, beam_scores, finished, eos, scores, tokens, parents, B, W, V, K};
    p.chunks = beam_chunks(B, W, V);
    p.stats = static_cast<float2 *>(workspace);
    p.lists = reinterpret_cast<uint64_t *>(p.stats + (size_t)B * W * p.chunks);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == KDA_DTYPE_BF16 ? launch_beam<__nv_bfloat16>(p, st) : launch_beam<float>(p, st);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_beam_select(const void *logits, kda_dtype_t dtype, int64_t row_stride,
                                        const float *beam_scores, const uint8_t *finished, int eos, float *scores,
                                        int32_t *tokens, int32_t *parents, int B, int W, int V, int K,
                                        kda_stream_t stream)
{
    const kda_status_t c = check_beam(logits, dtype, row_stride, beam_scores, finished, eos, scores, tokens, parents,
                                      B, W, V, K);
    if (c != KDA_OK)
        return c;
    const size_t need = kda_beam_select_workspace_size(B, W, V, K);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    void *ws = nullptr;
    if (pool_alloc(&ws, need, st) != cudaSuccess)
        return KDA_ERR_CUDA;
    kda_status_t s = kda_beam_select_ws(logits, dtype, row_stride, beam_scores, finished, eos, scores, tokens, parents,
                                        B, W, V, K, ws, need, stream);
    if (cudaFreeAsync(ws, st) != cudaSuccess && s == KDA_OK)
        s = KDA_ERR_CUDA;
    return s;
}
