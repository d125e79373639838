// kda_beam_select: log-softmax of the beams' logits, and the K best of a batch entry's beams x vocabulary.
//
// Score of candidate (w, t): fl(c + l[t]), c = (score_w - m) - log sum exp(l - m).  c is known only when the row has
// been read to its end, but fl(c + l) never falls as l rises: so one pass over the logits keeps, for every chunk of a
// row, the chunk's maximum and sum and its K + 1 best logits (kda_beam_chunks_kernel), and a second kernel, one CTA a
// batch entry, turns those few into scores and picks (kda_beam_pick_kernel).  Each logit is read once: the floor.
//
// Measured: 32 x 8 rows of 131072 fp32 logits, a tenth of the rows finished and not read (121 MB of 134), 35.7 us, 3.4 TB/s,
// half the measured copy rate: the chunks stream at 55 to 65% of it and all end together, so that their tail (the bound, the few
// threads looked at again) and the pick's chain of latencies (5.5 us) are in nobody's shadow; the fp32 chunk kernel also spills (68
// bytes at the 48 registers of five CTAs an SM).  One request of 4 x 32001 bf16 logits: 9.0 us, both chains.
//
// Chunks that are whole steps of rows on 16 bytes are read by vectors, others one logit at a time in the same order.  No row
// finished, nothing left in L2, us for fp32 | bf16 logits: 131072 (all whole) 43.6 | 27.2, 128256 (the last of three chunks is not) 41.2 |
// 32.5, 151936 45.7 | 37.0, 50304 24.1 | 20.0, 50257 (rows off 16 bytes, none is) 23.0 | 21.9: fp32 loses nothing by it, bf16 up to a
// fifth.
//
// What the short lists may hide: logits so close that their fp32 scores are equal tie by index and not by logit.  That
// matters only where the value a chunk's list was cut off at reaches the K-th score and a neighbouring logit value has
// the same score too; the pick then goes over all candidates of the entry again (pick_all).
//
// The best of many.  Candidates are 64-bit keys, order-preserving bits of the value above the complement of the index,
// so all are distinct and a tie goes to the lower index.  The n-th best of the thread groups' best is a lower bound on
// the n-th best, and at most n groups have candidates from it up: those are gathered, few more than n.
#include "kda_step.cuh"

#include <cfloat>

namespace kda {
namespace {

constexpr int THREADS = 256;              // of the chunk kernel
constexpr int PICK_THREADS = 512;
constexpr int CAP = 2048;                 // keys gathered in shared memory
constexpr int SELECTED = 1024;            // of them from the bound up: K groups of 2048 / 64 or 2048 / 128 keys at most
constexpr int BY_KEYS = 1 << 30;          // in a list's count: the list is the K + 1 best and ends at a logit
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
    int chunks, chunk;       // chunks of a row, tokens of a chunk
    int room;                // keys of a list
    float4 *stats;           // [B W][chunks]: maximum, sum of exp(l - maximum), the value the list was cut off at (NaN:
                             // nowhere), keys in the list (bits)   (workspace)
    uint64_t *lists;         // [B W][chunks][room]: keys of all logits from the cut up, K + 1 at least where there are
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
    uint64_t group[128];           // best of each group of threads
    uint64_t cand[CAP];
    uint64_t red[32];
    uint64_t bound;
    uint32_t lowest;
    int count;
};

// Groups: twice as many as wanted keys at least, so that few more than the wanted ones get past the bound.
__device__ __forceinline__ int groups_for(int n) { return n <= 32 ? 64 : 128; }

// The n-th best of the groups' best keys; 1 (every key gets through) when fewer than n groups have one.
template <int NT, int GROUPS> __device__ __forceinline__ uint64_t group_bound_of(Pick &sh, uint64_t best, int n)
{
    constexpr int SIZE = NT / GROUPS;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int o = 1; o < SIZE; o <<= 1) {
        const uint64_t y = __shfl_xor_sync(FULL, best, o);
        best = best > y ? best : y;
    }
    if (threadIdx.x % SIZE == 0)
        sh.group[threadIdx.x / SIZE] = best;
    if (threadIdx.x == 0)
        sh.bound = 1;
    __syncthreads();
    uint64_t all[GROUPS / 32];
#pragma unroll
    for (int j = 0; j < GROUPS / 32; j++)
        all[j] = sh.group[32 * j + lane];
#pragma unroll
    for (int i = 0; i < GROUPS * 32 / NT; i++) {                   // a warp ranks a group
        const uint64_t x = sh.group[i * (NT / 32) + warp];
        int rank = 0;
#pragma unroll
        for (int j = 0; j < GROUPS / 32; j++)
            rank += __popc(__ballot_sync(FULL, all[j] > x));
        if (lane == 0 && x != 0 && rank == n - 1)
            sh.bound = x;
    }
    __syncthreads();
    return sh.bound;
}
template <int NT> __device__ __forceinline__ uint64_t group_bound(Pick &sh, uint64_t best, int n)
{
    return groups_for(n) == 64 ? group_bound_of<NT, 64>(sh, best, n) : group_bound_of<NT, 128>(sh, best, n);
}

// The same on values alone: the n-th best (ties counted) of the groups' best values, NaN or -inf when fewer groups than n
// have one above -inf.
template <int NT, int GROUPS> __device__ __forceinline__ float group_bound_value_of(Pick &sh, float best, int n)
{
    constexpr int SIZE = NT / GROUPS;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t *g = reinterpret_cast<uint32_t *>(sh.group);
#pragma unroll
    for (int o = 1; o < SIZE; o <<= 1)
        best = fmaxf(best, __shfl_xor_sync(FULL, best, o));
    if (threadIdx.x % SIZE == 0)
        g[threadIdx.x / SIZE] = (uint32_t)(key_of(best, 0) >> 32);
    if (threadIdx.x == 0) {
        sh.count = 0;
        sh.lowest = FULL;
    }
    __syncthreads();
    uint32_t all[GROUPS / 32], low = FULL;
#pragma unroll
    for (int j = 0; j < GROUPS / 32; j++)
        all[j] = g[32 * j + lane];
#pragma unroll
    for (int i = 0; i < GROUPS * 32 / NT; i++) {                   // a warp ranks a group
        const uint32_t x = g[i * (NT / 32) + warp];
        int above = 0;
#pragma unroll
        for (int j = 0; j < GROUPS / 32; j++)
            above += __popc(__ballot_sync(FULL, all[j] > x));
        if (above < n)                                             // the smallest of the values that fewer than n are above
            low = min(low, x);
    }
    if (lane == 0)
        atomicMin(&sh.lowest, low);
    __syncthreads();
    return key_value((uint64_t)sh.lowest << 32);
}
template <int NT> __device__ __forceinline__ float group_bound_value(Pick &sh, float best, int n)
{
    return groups_for(n) == 64 ? group_bound_value_of<NT, 64>(sh, best, n) : group_bound_value_of<NT, 128>(sh, best, n);
}

// Ranks the gathered keys (count of them, all distinct) and hands the best n to put(rank, key), by one thread each.
template <int NT, typename F> __device__ void rank_gathered(const uint64_t *cand, int count, int n, F put)
{
    const int lane = threadIdx.x % 32;
    for (int i = threadIdx.x / 32; i < count; i += NT / 32) {      // a warp ranks a key
        const uint64_t x = cand[i];
        int rank = 0;
        for (int j = lane; j < count; j += 32)
            rank += cand[j] > x;
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
    static constexpr int N = 16 / sizeof(T);        // logits of a 16-byte vector
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
// The two largest of N values (fmaxf and fminf pass over NaN, which can only make lo larger than it is).
template <int N> __device__ __forceinline__ void two_largest(const float *v, float &hi, float &lo)
{
    if constexpr (N == 2) {
        hi = fmaxf(v[0], v[1]);
        lo = fminf(v[0], v[1]);
    } else {
        float h0, l0, h1, l1;
        two_largest<N / 2>(v, h0, l0);
        two_largest<N / 2>(v + N / 2, h1, l1);
        hi = fmaxf(h0, h1);
        lo = fmaxf(fminf(h0, h1), fmaxf(l0, l1));
    }
}

// What a thread keeps of the logits it has seen: the largest, the step it came in and the next largest, and the sum of
// exp(v - ref) as 2^(v L - c), c = ref L rounded; the factor 2^(c - ref L) is put in at the end.  ref follows the maximum
// only in large steps: any of the logits near it serves.
struct Seen {
    float best = -INFINITY, next = -INFINITY, ref = -INFINITY, c = 0.0f, sum = 0.0f;
    int at = 0;
    template <int N> __device__ __forceinline__ void add(const float (&v)[N], int step)
    {
        float m, second;
        two_largest<N>(v, m, second);
        next = fmaxf(next, fmaxf(second, fminf(best, m)));
        at = m > best ? step : at;
        best = fmaxf(best, m);
        if (m > ref + 40.0f && m <= FLT_MAX) {
            const float to = m * LOG2E;
            sum = ref == -INFINITY ? 0.0f : sum * ex2_approx(c - to);
            ref = m;
            c = to;
        }
#pragma unroll
        for (int e = 0; e < N; e++)
            sum += ex2_approx(fmaf(v[e], LOG2E, -c));
    }
};

// Thread i's logits of the tokens [t0, t1): N from t0 + (s THREADS + i) N on for s = 0, 1, ...  DEPTH loads of 16 bytes
// are in flight.  VECTOR: whole steps of a row on a 16-byte boundary; else the same logits in the same order one by one, so
// that the result does not depend on a row's alignment.
template <typename T, bool VECTOR> __device__ __forceinline__ void stream_logits(const T *l, int t0, int t1, Seen &seen)
{
    constexpr int N = Vec<T>::N, STEP = THREADS * N;
    const int steps = (t1 - t0 + STEP - 1) / STEP;
    if constexpr (VECTOR) {
        constexpr int DEPTH = 32 / N;               // bf16 has twice the work a byte
        const uint4 *at = reinterpret_cast<const uint4 *>(l + t0) + threadIdx.x;
        uint4 raw[DEPTH];
#pragma unroll
        for (int d = 0; d < DEPTH; d++)
            if (d < steps)
                raw[d] = at[d * THREADS];
        int s = 0;
        for (; s + 2 * DEPTH <= steps; s += DEPTH) {
            at += DEPTH * THREADS;
#pragma unroll
            for (int d = 0; d < DEPTH; d++) {
                float v[N];
                unpack(raw[d], v, l);
                seen.add(v, s + d);
                raw[d] = at[d * THREADS];
            }
        }
        at += DEPTH * THREADS;
#pragma unroll
        for (int d = 0; d < DEPTH; d++)             // up to DEPTH more steps behind the ones in flight
            if (s + d < steps) {
                float v[N];
                unpack(raw[d], v, l);
                seen.add(v, s + d);
                if (s + DEPTH + d < steps)
                    raw[d] = at[d * THREADS];
            }
#pragma unroll
        for (int d = 0; d < DEPTH; d++)
            if (s + DEPTH + d < steps) {
                float v[N];
                unpack(raw[d], v, l);
                seen.add(v, s + DEPTH + d);
            }
    } else {
        constexpr int FLIGHT = 16 / N;
        float raw[FLIGHT][N];
        int t = t0 + threadIdx.x * N;
        for (int s = 0; s < steps; s += FLIGHT) {
#pragma unroll
            for (int d = 0; d < FLIGHT; d++)
#pragma unroll
                for (int e = 0; e < N; e++) {
                    raw[d][e] = -INFINITY;
                    if (t + d * STEP + e < t1)
                        raw[d][e] = load_logit(l + t + d * STEP + e);
                }
#pragma unroll
            for (int d = 0; d < FLIGHT; d++)
                seen.add(raw[d], s + d);
            t += FLIGHT * STEP;
        }
    }
}

// The n best keys of tokens [t0, t1) of a row, whatever they are, straight from memory: the bound on keys, and where more
// than can be gathered lie above it (large values crowded into few threads) one key at a time.  Zeros past the last.
template <typename T>
__device__ __noinline__ void list_by_keys(Pick &sh, const T *l, int t0, int t1, int n, uint64_t *list)
{
    uint64_t best = 0;
    if (threadIdx.x == 0)
        sh.count = 0;
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
        rank_gathered<THREADS>(sh.cand, count, n, [&](int r, uint64_t k) { list[r] = k; });
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

// One CTA per (chunk, row).  The threads stream through the chunk's logits, with no barrier, and keep their maxima and
// sums.  The maxima then give a bound that about K + 1 logits reach: a thread (of the few) whose maximum does reads that
// one's vector again; where its next largest does too, eight lanes go over all of the thread's logits.
template <typename T> __global__ void __launch_bounds__(THREADS, 5) kda_beam_chunks_kernel(const BeamArgs p)
{
    constexpr int N = Vec<T>::N, STEP = THREADS * N;
    __shared__ __align__(16) Pick sh;
    __shared__ float2 part[THREADS / 32];
    stream_order();
    const int64_t row = blockIdx.x / p.chunks;
    const int chunk = (int)(blockIdx.x % p.chunks);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, n = p.K + 1;
    if (p.finished && p.finished[row])
        return;                              // its one candidate needs no logits
    const T *l = static_cast<const T *>(p.logits) + row * p.row_stride;
    const int t0 = chunk * p.chunk, t1 = min(p.V, t0 + p.chunk);
    Seen seen;
    if ((reinterpret_cast<uintptr_t>(l) & 15) == 0 && (t1 - t0) % STEP == 0)
        stream_logits<T, true>(l, t0, t1, seen);
    else
        stream_logits<T, false>(l, t0, t1, seen);
    const float best = seen.best;
    float m = best;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
    const float mu = fabsf(m) <= FLT_MAX ? m : 0.0f;
    float sum = seen.ref == -INFINITY ? seen.sum
                                      : seen.sum * (ex2_approx(-fmaf(seen.ref, LOG2E, -seen.c)) * ex2_approx((seen.ref - mu) * LOG2E));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(FULL, sum, o);
    if (!(sum <= FLT_MAX) || fabsf(mu) > 1e30f) {  // NaN logits (they count as -inf), or a product past fp32's range
        sum = 0.0f;
        for (int t = t0 + tid * N; t < t1; t += STEP)
            for (int e = 0; e < N && t + e < t1; e++)
                sum += ex2_approx((no_nan(load_logit(l + t + e)) - mu) * LOG2E);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(FULL, sum, o);
    }
    if (lane == 0)
        part[warp] = make_float2(m, sum);
    const float bound = group_bound_value<THREADS>(sh, best, n);
    uint64_t *list = p.lists + (int64_t)blockIdx.x * p.room;
    const bool by_keys = !(fabsf(bound) <= FLT_MAX);       // too few finite values for a bound
    if (!by_keys) {
        constexpr int TURNS = 16 / N;                      // of eight lanes over a thread's vectors, in flight together
        const bool more = seen.next >= bound;
        if (best >= bound && !more) {
            const int t = t0 + (seen.at * THREADS + tid) * N;
            float x[N];
#pragma unroll
            for (int e = 0; e < N; e++)
                x[e] = t + e < t1 ? load_logit(l + t + e) : -INFINITY;
#pragma unroll
            for (int e = 0; e < N; e++)
                if (x[e] >= bound) {
                    const int to = atomicAdd(&sh.count, 1);
                    if (to < p.room)
                        list[to] = key_of(x[e], t + e);
                }
        }
        for (unsigned owners = __ballot_sync(FULL, best >= bound && more); owners;) {
            int of = -1;
#pragma unroll
            for (int k = 0; k < 4; k++)
                if (owners) {
                    if (lane / 8 == k)
                        of = tid - lane + __ffs(owners) - 1;
                    owners &= owners - 1;
                }
            for (int first = t0; first < t1; first += 8 * TURNS * STEP) {
                float x[TURNS][N];
#pragma unroll
                for (int j = 0; j < TURNS; j++)
#pragma unroll
                    for (int e = 0; e < N; e++) {
                        const int t = first + ((lane % 8 + 8 * j) * THREADS + of) * N + e;
                        x[j][e] = -INFINITY;
                        if (of >= 0 && t < t1)
                            x[j][e] = load_logit(l + t);
                    }
#pragma unroll
                for (int j = 0; j < TURNS; j++)
#pragma unroll
                    for (int e = 0; e < N; e++)
                        if (x[j][e] >= bound) {
                            const int to = atomicAdd(&sh.count, 1);
                            if (to < p.room)
                                list[to] = key_of(x[j][e], first + ((lane % 8 + 8 * j) * THREADS + of) * N + e);
                        }
            }
        }
    }
    __syncthreads();
    int count = sh.count;
    float cut = bound;
    if (by_keys || count > p.room) {         // uniform: many ties, or hardly anything finite
        __syncthreads();
        list_by_keys(sh, l, t0, t1, n, list);
        __syncthreads();
        count = min(n, t1 - t0) | BY_KEYS;
        cut = t1 - t0 > n ? key_value(list[n - 1]) : __int_as_float(0x7fffffff);
    }
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
            p.stats[blockIdx.x] = make_float4(M, s, cut, __int_as_float(count));
    }
}

// Score of a candidate whose beam has offset c (-inf: nothing of the beam counts) and logit l.
__device__ __forceinline__ float score_of(float c, float l) { return c == -INFINITY ? c : no_nan(c + l); }

// The K best of all W x V candidates, one pass for each: what the short lists are a shortcut of.  own: the beams' scores, not
// read again from memory, where the entry's new ones may have been written over them.
template <typename T> __device__ __noinline__ void pick_all(const BeamArgs &p, int b, const float *c, const float *own, uint64_t *red)
{
    uint64_t last = ~0ull;
    for (int k = 0; k < p.K; k++) {
        uint64_t best = 0;
        for (int w = 0; w < p.W; w++) {
            const int64_t row = (int64_t)b * p.W + w;
            const T *l = static_cast<const T *>(p.logits) + row * p.row_stride;
            const bool done = p.finished && p.finished[row];
            for (int t = threadIdx.x; t < p.V; t += PICK_THREADS) {
                const float s = done ? (t == p.eos ? own[w] : -INFINITY)
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
    __shared__ __align__(16) Pick sh;
    __shared__ uint64_t sel[SELECTED];     // candidates from the bound up
    uint64_t *const cand = sh.cand;
    __shared__ float c[32], own[32];       // the beams' offsets, and the scores of finished ones
    __shared__ int kind[32];               // 0: candidates from the lists; 1: nothing counts; 2: finished
    __shared__ int selected;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    stream_order();
    if (tid == 0)
        sh.count = selected = 0;
    // The lists' slots, `room` a list and so warp by warp in one list each: the first HELD rounds of them are on their way
    // while the beams' offsets are worked out.
    constexpr int HELD = 4;
    const float4 *stats = p.stats + (int64_t)b * p.W * p.chunks;
    const uint64_t *lists = p.lists + (int64_t)b * p.W * p.chunks * p.room;
    const int64_t slots = (int64_t)p.W * p.chunks * p.room;
    uint64_t raw[HELD];
    int list_of[HELD], have[HELD];
    auto fetch = [&](int64_t from) {
#pragma unroll
        for (int i = 0; i < HELD; i++) {
            const int64_t x = from + i * PICK_THREADS + tid;
            list_of[i] = x < slots ? (int)((uint32_t)x / (uint32_t)p.room) : -1;    // slots < 2^31 (checked on the host)
            raw[i] = x < slots ? lists[x] : 0;
            have[i] = x < slots ? __float_as_int(stats[list_of[i]].w) & ~BY_KEYS : 0;
        }
    };
    fetch(0);
    for (int w = warp; w < p.W; w += PICK_THREADS / 32) {
        const int64_t row = (int64_t)b * p.W + w;
        const bool done = p.finished && p.finished[row];
        const float score = p.beam_scores[row];
        float m = -INFINITY, s = 0.0f;
        if (!done) {
            const float4 *st = p.stats + row * p.chunks;
            float4 x = lane < p.chunks ? st[lane] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
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
    // the candidate of slot j of a list (0: none); a beam whose candidates are all -inf but for a finished one's eos has its
    // first tokens and eos in the slots of its first list
    auto candidate = [&](int64_t from, int i) -> uint64_t {
        const int list = list_of[i];
        if (list < 0)
            return 0;
        const int j = (int)(from + i * PICK_THREADS + tid - (int64_t)list * p.room), w = list / p.chunks;
        if (kind[w] == 0)
            return j < have[i] ? key_of(score_of(c[w], key_value(raw[i])), (uint32_t)w * p.V + key_index(raw[i])) : 0;
        if (list != w * p.chunks)
            return 0;
        const bool eos = kind[w] == 2 && (j < p.K ? j == p.eos : j == p.K && p.eos >= p.K);
        return eos || (j < p.K && j < p.V) ? key_of(eos ? own[w] : -INFINITY, (uint32_t)w * p.V + (eos ? p.eos : j)) : 0;
    };
    uint64_t best = 0;
    for (int64_t from = 0; from < slots; from += HELD * PICK_THREADS) {
        if (from)
            fetch(from);
        uint64_t k[HELD];
        unsigned m[HELD];
        int at = 0;
#pragma unroll
        for (int i = 0; i < HELD; i++) {
            k[i] = candidate(from, i);
            best = k[i] > best ? k[i] : best;
            m[i] = __ballot_sync(FULL, k[i] != 0);
            at += __popc(m[i]);
        }
        if (lane == 0)
            at = atomicAdd(&sh.count, at);
        at = __shfl_sync(FULL, at, 0);
#pragma unroll
        for (int i = 0; i < HELD; i++) {                 // gathered while there is room
            const int to = at + __popc(m[i] & ((1u << lane) - 1));
            if (k[i] != 0 && to < CAP)
                cand[to] = k[i];
            at += __popc(m[i]);
        }
    }
    __syncthreads();
    const int total = sh.count;
    if (total <= CAP) {
        best = 0;
        for (int x = tid; x < total; x += PICK_THREADS)
            best = cand[x] > best ? cand[x] : best;
    }
    const uint64_t bound = group_bound<PICK_THREADS>(sh, best, p.K);
    auto select = [&](uint64_t k) {
        if (k != 0 && k >= bound) {
            const int to = atomicAdd(&selected, 1);
            if (to < SELECTED)
                sel[to] = k;
        }
    };
    if (total <= CAP) {
        for (int x = tid; x < total; x += PICK_THREADS)
            select(cand[x]);
    } else {
        for (int64_t from = 0; from < slots; from += HELD * PICK_THREADS) {
            fetch(from);
#pragma unroll
            for (int i = 0; i < HELD; i++)
                select(candidate(from, i));
        }
    }
    __syncthreads();
    const int count = selected;
    bool again = count > SELECTED;
    if (!again) {
        // the K-th score, and whether a list may have cut off a logit that has it too
        rank_gathered<PICK_THREADS>(sel, count, p.K, [&](int r, uint64_t k) {
            if (r == p.K - 1)
                sh.bound = k;
            p.scores[(int64_t)b * p.K + r] = key_value(k);
            p.tokens[(int64_t)b * p.K + r] = key_index(k) % p.V;
            p.parents[(int64_t)b * p.K + r] = b * p.W + key_index(k) / p.V;
        });
        __syncthreads();
        const float last = key_value(sh.bound);
        for (int x = tid; x < p.W * p.chunks; x += PICK_THREADS) {
            const int w = x / p.chunks;
            if (kind[w] != 0)
                continue;
            // a list by values has every logit from l up; one by keys may have left out equals of its last, l, too.  What was
            // left out is a logit of type T: the neighbours are T's.  (With fp32's for bf16 logits, which often tie, as many as a
            // quarter of the entries of rows in few chunks were picked over all candidates for a logit that bf16 does not have.)
            constexpr bool step16 = sizeof(T) == 2;
            const float l = stats[x].z;
            const bool by_keys = __float_as_int(stats[x].w) & BY_KEYS;
            if (l == l && score_of(c[w], l) == last &&
                ((by_keys && score_of(c[w], neighbour(l, true, step16)) == last) ||
                 (l != -INFINITY && score_of(c[w], neighbour(l, false, step16)) == last)))
                again = true;
        }
    }
    if (__syncthreads_or(again))
        pick_all<T>(p, b, c, own, sh.red);
}

}  // namespace

// Tokens of a chunk: whole steps of 2048 (what the CTA's threads take of bf16 logits at once).  Rows are cut so that the
// chunks are one wave of five CTAs on each of a GB300's 152 SMs (a constant: the workspace's size follows from the sizes alone), but not under 2048 tokens; few and long chunks also leave fewer lists to pick
// from.  32 x 8 rows of 131072 logits, in L2: 32.8 us in 3 chunks a row, 36.8 in 4, 34.4 in 2, 40 in 8.  4 rows of 32001:
// the same with 2048, 4096 and 8192 tokens.
static int beam_chunk(int B, int W, int V)
{
    const int64_t rows = (int64_t)B * W;
    int64_t cut = 5 * 152 / rows;
    cut = rows * cut * 10 < 5 * 152 * 9 ? cut + 1 : cut;       // a wave under nine tenths full is worse than a little over one
    cut = cut < 1 ? 1 : cut;
    const int64_t chunk = (V + cut - 1) / cut;
    return (int)((chunk + 2047) / 2048 * 2048);
}
static int beam_chunks(int B, int W, int V)
{
    const int chunk = beam_chunk(B, W, V);
    return (V + chunk - 1) / chunk;
}
// Keys of a list: some more than K + 1 reach the bound, or tie at it.
static int beam_room(int K) { return (2 * K + 32) / 32 * 32; }

namespace {

template <typename T> cudaError_t launch_beam(const BeamArgs &p, cudaStream_t st)
{
    const unsigned grid = (unsigned)(p.chunks * p.B * p.W);
    const cudaError_t e = launch_in_row(kda_beam_chunks_kernel<T>, grid, THREADS, 0, 1, st, p);
    return e != cudaSuccess ? e : launch_in_row(kda_beam_pick_kernel<T>, p.B, PICK_THREADS, 0, 1, st, p);
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
    if ((int64_t)B * W * beam_chunks(B, W, V) * beam_room(K) > INT32_MAX)
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
    // the outputs overlap neither each other nor an input; scores may be beam_scores where a row of both is one entry's
    const uint64_t rows = (uint64_t)B * W, picks = (uint64_t)B * K * 4;
    const uint64_t read = ((rows - 1) * (uint64_t)row_stride + V) * (dtype == KDA_DTYPE_BF16 ? 2 : 4);
    if (overlap(scores, picks, tokens, picks) || overlap(scores, picks, parents, picks) || overlap(tokens, picks, parents, picks))
        return KDA_ERR_INVALID_ARGUMENT;
    for (const void *out : {static_cast<const void *>(scores), static_cast<const void *>(tokens), static_cast<const void *>(parents)})
        if (overlap(out, picks, logits, read) || overlap(out, picks, finished, rows) ||
            (overlap(out, picks, beam_scores, rows * 4) && !(out == beam_scores && out == scores && K == W)))
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
    return (size_t)B * W * beam_chunks(B, W, V) * (sizeof(float4) + beam_room(K) * sizeof(uint64_t));
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
    p.chunk = beam_chunk(B, W, V);
    p.room = beam_room(K);
    p.stats = static_cast<float4 *>(workspace);
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
