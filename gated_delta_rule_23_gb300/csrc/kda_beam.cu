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

constexpr int THREADS = 256;              // of the chunk kernel
constexpr int PICK_THREADS = 512;
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
    int chunks, span;        // chunks of a row, pieces of a chunk
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

template <int NT> __device__ uint64_t block_max(uint64_t x, uint64_t *sh)
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
    for (int i = 1; i < NT / 32; i++)
        x = x > sh[i] ? x : sh[i];
    return x;
}

struct Pick {
    uint64_t group[128];           // best key of each group of threads
    uint64_t cand[CAP];
    uint64_t red[32];
    uint64_t bound;
    int count;
};

// Groups: twice as many as wanted keys at least, so that few more than the wanted ones get past the bound.
__device__ __forceinline__ int groups_for(int n) { return n <= 32 ? 64 : 128; }

// The n-th best of the groups' best keys; 1 (every key gets through) when fewer than n groups have one.
template <int NT> __device__ uint64_t group_bound(Pick &sh, uint64_t best, int n)
{
    const int groups = groups_for(n), size = NT / groups, lane = threadIdx.x % 32;
    for (int o = 1; o < size; o <<= 1) {
        const uint64_t y = __shfl_xor_sync(FULL, best, o);
        best = best > y ? best : y;
    }
    if (threadIdx.x % size == 0)
        sh.group[threadIdx.x / size] = best;
    if (threadIdx.x == 0) {
        sh.bound = 1;
        sh.count = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x / 32; i < groups; i += NT / 32) {     // a warp ranks a group
        const uint64_t x = sh.group[i];
        int rank = 0;
        for (int j = 0; j < groups; j += 32)
            rank += __popc(__ballot_sync(FULL, sh.group[j + lane] > x));
        if (lane == 0 && x != 0 && rank == n - 1)
            sh.bound = x;
    }
    __syncthreads();
    return sh.bound;
}

// The same on values alone: the n-th best (ties counted) of the groups' best values, -inf when fewer have one.
template <int NT> __device__ float group_bound_value(Pick &sh, float best, int n)
{
    const int groups = groups_for(n), size = NT / groups, lane = threadIdx.x % 32;
    float *g = reinterpret_cast<float *>(sh.group);
    for (int o = 1; o < size; o <<= 1)
        best = fmaxf(best, __shfl_xor_sync(FULL, best, o));
    if (threadIdx.x % size == 0)
        g[threadIdx.x / size] = best;
    uint32_t *lowest = reinterpret_cast<uint32_t *>(&sh.bound);
    if (threadIdx.x == 0) {
        *lowest = FULL;
        sh.count = 0;
    }
    __syncthreads();
    uint32_t low = FULL;
    for (int i = threadIdx.x / 32; i < groups; i += NT / 32) {
        const float x = g[i];
        int above = 0;
        for (int j = 0; j < groups; j += 32)
            above += __popc(__ballot_sync(FULL, g[j + lane] > x));
        // the smallest of the values that fewer than n are above
        if (above < n)
            low = min(low, (uint32_t)(key_of(x, 0) >> 32));
    }
    if (lane == 0)
        atomicMin(lowest, low);
    __syncthreads();
    return key_value((uint64_t)*lowest << 32);
}

// Ranks the gathered keys (count of them, all distinct) and hands the best n to put(rank, key), by one thread each.
template <int NT, typename F> __device__ void rank_gathered(const Pick &sh, int count, int n, F put)
{
    const int lane = threadIdx.x % 32;
    for (int i = threadIdx.x / 32; i < count; i += NT / 32) {      // a warp ranks a key
        const uint64_t x = sh.cand[i];
        int rank = 0;
        for (int j = lane; j < count; j += 32)
            rank += sh.cand[j] > x;
        rank = __reduce_add_sync(FULL, rank);
        if (lane == 0 && rank < n)
            put(rank, x);
    }
}
__device__ __forceinline__ void gather(Pick &sh, uint64_t key)
{
    const int to = atomicAdd(&sh.count, 1);
    if (to < CAP)
        sh.cand[to] = key;
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
// 16 bytes that lie `off` bytes (not 0) past a 16-byte boundary: a holds the aligned 16 bytes they begin in, of lane i of
// a warp at 16 i; the next lane's a is the second half, and lane 31 reads it (element t of the row l on).
template <typename T> __device__ __forceinline__ uint4 shifted(const uint4 &a, const T *l, int t, int off, int V)
{
    uint4 b;
    b.x = __shfl_down_sync(FULL, a.x, 1);
    b.y = __shfl_down_sync(FULL, a.y, 1);
    b.z = __shfl_down_sync(FULL, a.z, 1);
    b.w = __shfl_down_sync(FULL, a.w, 1);
    if ((threadIdx.x & 31) == 31)
        b = load_aligned(l, t, V);
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

// The n best keys of tokens [t0, t1) of a row, whatever they are, straight from memory: the bound on keys, and where more
// than can be gathered lie above it (large values crowded into few threads) one key at a time.
template <typename T>
__device__ __noinline__ void list_by_keys(Pick &sh, const T *l, int t0, int t1, int n, uint64_t *list)
{
    uint64_t best = 0;
    for (int t = t0 + threadIdx.x; t < t1; t += THREADS) {
        const uint64_t x = key_of(no_nan(load_logit(l + t)), t);
        best = x > best ? x : best;
    }
    const uint64_t bound = group_bound<THREADS>(sh, best, n);
    if (best >= bound)
        for (int t = t0 + threadIdx.x; t < t1; t += THREADS) {
            const uint64_t x = key_of(no_nan(load_logit(l + t)), t);
            if (x >= bound)
                gather(sh, x);
        }
    __syncthreads();
    const int count = sh.count;
    if (count <= CAP) {
        rank_gathered<THREADS>(sh, count, n, [&](int r, uint64_t k) { list[r] = k; });
        for (int r = count + threadIdx.x; r < n; r += THREADS)
            list[r] = 0;
        return;
    }
    uint64_t last = ~0ull;
    for (int r = 0; r < n; r++) {
        uint64_t b = 0;
        for (int t = t0 + threadIdx.x; t < t1; t += THREADS) {
            const uint64_t x = key_of(no_nan(load_logit(l + t)), t);
            if (x < last && x > b)
                b = x;
        }
        last = block_max<THREADS>(b, sh.red);
        if (threadIdx.x == 0)
            list[r] = last;
    }
}

// One CTA per (chunk, row); a chunk is p.span pieces of PER x THREADS logits, the next piece's loads in flight while one
// is worked on.  The first piece gives the bound: later ones only compare with it (a piece as good as the first adds
// about K + 1 keys), so there is no barrier between pieces.  Which thread takes which token, and so the order of the
// sums, does not depend on the row's alignment: equal rows get equal scores.
constexpr int MAX_SPAN = 4;

template <typename T, int PER> __global__ void __launch_bounds__(THREADS, PER > 16 ? 2 : 6) kda_beam_chunks_kernel(const BeamArgs p)
{
    constexpr int N = Vec<T>::N, NV = PER / N, PIECE = THREADS * PER;
    __shared__ __align__(16) Pick sh;
    __shared__ float2 part[MAX_SPAN * THREADS / 32];
    asm volatile("griddepcontrol.launch_dependents;");
    const int64_t row = blockIdx.x / p.chunks;
    const int chunk = (int)(blockIdx.x % p.chunks);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, n = p.K + 1;
    if (p.finished && p.finished[row])
        return;                              // its one candidate needs no logits
    const T *l = static_cast<const T *>(p.logits) + row * p.row_stride;
    const int off = (int)(reinterpret_cast<uintptr_t>(l) & 15), back = off / (int)sizeof(T);
    const int t0 = chunk * (PIECE * p.span), t1 = min(p.V, t0 + PIECE * p.span);
    uint4 next[NV];
    auto load = [&](int first) {             // all loads before anything waits for one
        if (first >= back && first + PIECE <= p.V) {
#pragma unroll
            for (int i = 0; i < NV; i++)
                next[i] = __ldcs(reinterpret_cast<const uint4 *>(l + (first + (i * THREADS + tid) * N - back)));
        } else {
#pragma unroll
            for (int i = 0; i < NV; i++)
                next[i] = load_aligned(l, first + (i * THREADS + tid) * N - back, p.V);
        }
    };
    load(t0);
    float bound = -INFINITY;
    bool by_keys = false;
    int pieces = 0;
    for (int first = t0; first < t1; first += PIECE, pieces++) {
        float v[PER];
        if (off) {
#pragma unroll
            for (int i = 0; i < NV; i++)
                next[i] = shifted(next[i], l, first + (i * THREADS + tid) * N - back + N, off, p.V);
        }
#pragma unroll
        for (int i = 0; i < NV; i++)
            unpack(next[i], v + i * N, l);
        if (first + PIECE < t1)
            load(first + PIECE);
        auto token = [&](int i) { return first + ((i / N) * THREADS + tid) * N + i % N; };
        if (first + PIECE > p.V) {
#pragma unroll
            for (int i = 0; i < PER; i++)
                v[i] = token(i) < p.V ? v[i] : -INFINITY;
        }
        // maximum and sum of the piece, warp by warp (fmaxf passes over NaN)
        float best = -INFINITY, top[NV];     // of the thread, and of each of its vectors
#pragma unroll
        for (int i = 0; i < NV; i++) {
            top[i] = v[i * N];
#pragma unroll
            for (int e = 1; e < N; e++)
                top[i] = fmaxf(top[i], v[i * N + e]);
            best = fmaxf(best, top[i]);
        }
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
            for (int i = 0; i < PER; i++)
                sum += ex2_approx((no_nan(v[i]) - mu) * LOG2E);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                sum += __shfl_xor_sync(FULL, sum, o);
        }
        if (lane == 0)
            part[pieces * (THREADS / 32) + warp] = make_float2(m, sum);
        if (first == t0) {
            bound = group_bound_value<THREADS>(sh, best, n);
            by_keys = !(fabsf(bound) <= FLT_MAX);      // too few finite values for a bound
        }
        if (!by_keys && best >= bound) {
#pragma unroll
            for (int i = 0; i < NV; i++) {
                if (!(top[i] >= bound))
                    continue;
#pragma unroll
                for (int e = 0; e < N; e++)
                    if (v[i * N + e] >= bound)
                        gather(sh, key_of(v[i * N + e], token(i * N + e)));
            }
        }
    }
    __syncthreads();
    const int64_t slot = blockIdx.x;
    uint64_t *list = p.lists + slot * n;
    if (warp == 0) {
        const float2 x = lane < pieces * (THREADS / 32) ? part[lane] : make_float2(-INFINITY, 0.0f);
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
    if (by_keys || count > CAP) {            // uniform: many ties, or hardly anything finite
        __syncthreads();
        list_by_keys(sh, l, t0, t1, n, list);
    } else {
        rank_gathered<THREADS>(sh, count, n, [&](int r, uint64_t k) { list[r] = k; });
    }
}
static_assert(MAX_SPAN * THREADS / 32 <= 32, "a warp joins the parts");

// Score of a candidate whose beam has offset c (-inf: nothing of the beam counts) and logit l.
__device__ __forceinline__ float score_of(float c, float l) { return c == -INFINITY ? c : no_nan(c + l); }

// The K best of all W x V candidates, one pass for each: what the short lists are a shortcut of.
template <typename T> __device__ __noinline__ void pick_all(const BeamArgs &p, int b, const float *c, uint64_t *red)
{
    uint64_t last = ~0ull;
    for (int k = 0; k < p.K; k++) {
        uint64_t best = 0;
        for (int w = 0; w < p.W; w++) {
            const int64_t row = (int64_t)b * p.W + w;
            const T *l = static_cast<const T *>(p.logits) + row * p.row_stride;
            const bool done = p.finished && p.finished[row];
            for (int t = threadIdx.x; t < p.V; t += PICK_THREADS) {
                const float s = done ? (t == p.eos ? no_nan(p.beam_scores[row]) : -INFINITY)
                                     : score_of(c[w], no_nan(load_logit(l + t)));
                const uint64_t x = key_of(s, (uint32_t)w * p.V + t);
                if (x < last && x > best)
                    best = x;
            }
        }
        last = block_max<PICK_THREADS>(best, red);
        if (threadIdx.x == 0) {
            p.scores[(int64_t)b * p.K + k] = key_value(last);
            p.tokens[(int64_t)b * p.K + k] = key_index(last) % p.V;
            p.parents[(int64_t)b * p.K + k] = b * p.W + key_index(last) / p.V;
        }
    }
}

// One CTA per batch entry.
template <typename T> __global__ void __launch_bounds__(PICK_THREADS) kda_beam_pick_kernel(const BeamArgs p)
{
    constexpr int HELD = 4;                // candidates a thread keeps in registers
    __shared__ __align__(16) Pick sh;
    __shared__ float c[32], own[32];       // the beams' offsets, and the scores of finished ones
    __shared__ int kind[32];               // 0: candidates from the lists; 1: nothing counts; 2: finished
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid % 32, n = p.K + 1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int w = tid / 32; w < p.W; w += PICK_THREADS / 32) {
        const int64_t row = (int64_t)b * p.W + w;
        const bool done = p.finished && p.finished[row];
        const float score = p.beam_scores[row];
        float m = -INFINITY, s = 0.0f;
        if (!done) {
            const float2 *st = p.stats + row * p.chunks;
            float2 x = lane < p.chunks ? st[lane] : make_float2(-INFINITY, 0.0f);
            m = x.x;
            for (int i = lane + 32; i < p.chunks; i += 32)
                m = fmaxf(m, st[i].x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
            if (fabsf(m) <= FLT_MAX) {
                s = x.y * expf(x.x - m);
                for (int i = lane + 32; i < p.chunks; i += 32) {
                    x = st[i];
                    s += x.y * expf(x.x - m);
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                s += __shfl_xor_sync(FULL, s, o);
        }
        if (lane == 0) {
            const float off = fabsf(m) <= FLT_MAX ? no_nan((score - m) - logf(s)) : -INFINITY;
            c[w] = off;
            own[w] = no_nan(score);
            kind[w] = done ? 2 : (off == -INFINITY ? 1 : 0);
        }
    }
    __syncthreads();
    // candidate i of beam w: a list entry, or for a beam whose candidates are all but one -inf its first tokens and eos
    const uint32_t per = (uint32_t)p.chunks * n, total = per * p.W;
    const uint64_t *lists = p.lists + (int64_t)b * total;
    auto candidate = [&](uint32_t x) -> uint64_t {
        const uint32_t w = x / per, i = x - w * per;
        if (kind[w] == 0) {
            const uint64_t k = lists[x];
            return k ? key_of(score_of(c[w], key_value(k)), w * p.V + key_index(k)) : 0;
        }
        const bool done = kind[w] == 2;
        uint32_t t = i;
        if (i > (uint32_t)p.K || (i == (uint32_t)p.K && !(done && p.eos >= p.K)) ||
            (i < (uint32_t)p.K && i >= (uint32_t)p.V))
            return 0;
        if (i == (uint32_t)p.K)
            t = (uint32_t)p.eos;
        return key_of(done && t == (uint32_t)p.eos ? own[w] : -INFINITY, w * p.V + t);
    };
    uint64_t best = 0, held[HELD];
#pragma unroll
    for (int i = 0; i < HELD; i++) {
        const uint32_t x = i * PICK_THREADS + tid;
        held[i] = x < total ? candidate(x) : 0;
        best = held[i] > best ? held[i] : best;
    }
    for (uint32_t x = HELD * PICK_THREADS + tid; x < total; x += PICK_THREADS) {
        const uint64_t k = candidate(x);
        best = k > best ? k : best;
    }
    const uint64_t bound = group_bound<PICK_THREADS>(sh, best, p.K);
    if (best >= bound) {
#pragma unroll
        for (int i = 0; i < HELD; i++)
            if (held[i] >= bound)
                gather(sh, held[i]);
        for (uint32_t x = HELD * PICK_THREADS + tid; x < total; x += PICK_THREADS) {
            const uint64_t k = candidate(x);
            if (k >= bound)
                gather(sh, k);
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
        rank_gathered<PICK_THREADS>(sh, count, p.K, [&](int r, uint64_t k) {
            if (r == p.K - 1)
                sh.bound = k;
            p.scores[(int64_t)b * p.K + r] = key_value(k);
            p.tokens[(int64_t)b * p.K + r] = key_index(k) % p.V;
            p.parents[(int64_t)b * p.K + r] = b * p.W + key_index(k) / p.V;
        });
        __syncthreads();
        const float last = key_value(sh.bound);
        for (uint32_t x = tid; x < (uint32_t)p.W * p.chunks; x += PICK_THREADS) {
            const uint32_t w = x / p.chunks;
            if (kind[w] != 0)
                continue;
            const uint64_t k = lists[x * n + n - 1];
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

// Logits a thread holds of a piece, and pieces of a chunk.
struct BeamCut {
    int per, span;
};
static BeamCut beam_cut(int B, int W, int V)
{
    const int64_t rows = (int64_t)B * W;
    auto ctas = [&](int chunk) { return rows * ((V + chunk - 1) / chunk); };
    if (ctas(THREADS * 32 * MAX_SPAN) >= 304)
        return {32, MAX_SPAN};
    if (ctas(THREADS * 32) >= 152)
        return {32, 1};
    return {8, 1};
}
static int beam_chunks(int B, int W, int V)
{
    const BeamCut c = beam_cut(B, W, V);
    const int chunk = THREADS * c.per * c.span;
    return (V + chunk - 1) / chunk;
}

namespace {

template <typename T> cudaError_t launch_beam(const BeamArgs &p, cudaStream_t st)
{
    const unsigned grid = (unsigned)(p.chunks * p.B * p.W);
    if (beam_cut(p.B, p.W, p.V).per == 32)
        kda_beam_chunks_kernel<T, 32><<<grid, THREADS, 0, st>>>(p);
    else
        kda_beam_chunks_kernel<T, 8><<<grid, THREADS, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.B);
    cfg.blockDim = dim3(PICK_THREADS);
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
    p.span = beam_cut(B, W, V).span;
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
