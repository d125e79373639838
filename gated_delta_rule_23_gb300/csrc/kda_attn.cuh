// Windowed attention over the paged cache: the problem description, and the row form of the definition.
#pragma once

#include <cuda.h>

#include "kda_step.cuh"

namespace kda {

struct AttnArgs {
    const __nv_bfloat16 *q;
    int64_t q_stride;
    __nv_bfloat16 *out;
    float *lse;                  // or nullptr
    float scale_log2;            // scale * log2(e): the softmax is taken in base 2
    int window, sinks;
    int hq, group;               // group = query heads of one key head
    PagedCache cache;
    Tokens tok;
    unsigned int *err;
};

// How a call is cut: every (sequence, key head) has group x Q_n query rows, row r being token r / group and head
// r % group of the group (so that heads sharing keys share a tile); rows come in tiles of whole tokens, and the keys a tile needs are
// split `splits` ways, the partial results joined by a cluster's CTAs among themselves, or by a second kernel.
constexpr int ATTN_ROWS = 256;   // query rows of a tile
constexpr int DECODE_ROWS = 16, DECODE_KEYS = 16;   // rows of the decode kernel, keys of its blocks
constexpr int ATTN_CLUSTER = 8;                     // splits that join in a cluster

struct AttnPlan {
    bool decode;            // few query rows: the decode kernel, one item a CTA
    int row_tiles;          // of 16 rows, of a (sequence, key head) (decode kernel)
    bool cluster;           // the splits are a cluster (no workspace, no join kernel)
    int splits;
    int items;              // (row tile, key head, split) items (ragged: an upper bound)
    int granule;            // positions of a cache page that are copied together
    int run;                // tokens of an item
    uint32_t magic;         // ceil(2^20 / group)
    float *part_o;          // [splits][tokens * hq][dim] fp32, unnormalised (workspace)
    float2 *part_ml;        // [splits][tokens * hq]: running maximum (base 2) and sum
    int64_t rows;           // tokens * hq
    uint32_t wait_polls;
    int margin;             // positions that a row's products may take in on either side of what it sees (attn_mend_rows)
};

cudaError_t launch_attn_tiles(const AttnArgs &p, const AttnPlan &plan, cudaStream_t stream);
cudaError_t launch_attn_decode(const AttnArgs &p, const AttnPlan &plan, cudaStream_t stream);
cudaError_t launch_attn_join(const AttnArgs &p, const AttnPlan &plan, cudaStream_t stream);

// A tensor map of the cache as rows [pages * hkv * page][dim], boxes of 64 columns by `rows` rows, 128-byte swizzle.
cudaError_t cache_map(CUtensorMap *map, const void *ptr, const PagedCache &c, int rows);

constexpr int OUTSIDE = INT32_MAX - 4096;   // a row that no cache has: a bulk copy from it gives zeros

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t mbar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(mbar) : "memory");
}
// The same shared-memory address in CTA `rank` of the cluster, and stores there
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int rank)
{
    uint32_t x;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(x) : "r"(addr), "r"(rank));
    return x;
}
__device__ __forceinline__ void store_cluster(uint32_t addr, float2 x)
{
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x.x), "f"(x.y) : "memory");
}
__device__ __forceinline__ void store_cluster(uint32_t addr, float4 x)
{
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w) : "memory");
}
// Every CTA of the cluster comes here, whatever its waits did, so that this wait always ends.
__device__ __forceinline__ void cluster_sync()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
constexpr float LN2 = 0.6931471805599453f;

// Sequence, index within it and length of token t's sequence, by a whole warp; an index outside [0, len) for a token
// that a malformed cu_seqlens gives to nobody.
__device__ __forceinline__ int token_place(const Tokens &tok, int64_t t, int64_t &i, int64_t &len, bool &bad)
{
    if (!tok.cu) {
        len = tok.T;
        const int n = (int)(t / tok.T);
        i = t - (int64_t)n * tok.T;
        return n;
    }
    const int n = seq_of_token(tok.cu, tok.N, t);
    int64_t bos;
    bad |= seq_range(tok.cu, n, tok.N, tok.T, bos, len);
    i = t - bos;
    return n;
}

// One query row (token t of the batch, head h) at position pos, by a whole warp, straight from the definition:
// every visible key in order, with the running maximum m and sum l of the softmax in base 2.  Keys that the row
// does not see are never read.  o is the mean of the values so far, which no finite values carry past fp32's range (their sum
// by the weights does from about 1e38 on).
template <int DIM>
__device__ void attn_row(const AttnArgs &p, int n, int64_t t, int h, int64_t pos, bool &bad)
{
    constexpr int PER = DIM / 32;
    const int lane = threadIdx.x & 31;
    const __nv_bfloat16 *q = p.q + t * p.q_stride + (int64_t)h * DIM + lane * PER;
    const int64_t head = ((int64_t)(h / p.group) << p.cache.page_shift) * DIM;
    float qf[PER], o[PER];
#pragma unroll
    for (int e = 0; e < PER; e++) {
        qf[e] = __bfloat162float(q[e]) * p.scale_log2;
        o[e] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    const int64_t left = pos - p.window + 1;
    for (int64_t j = 0; j <= pos; j++) {
        if (j >= p.sinks && j < left) {
            j = left;
        }
        const int64_t row = cache_row(p.cache, n, j);
        if (row < 0) {
            bad = true;
            continue;
        }
        const __nv_bfloat16 *k = p.cache.k + row + head + lane * PER, *v = p.cache.v + row + head + lane * PER;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < PER; e++)
            s = fmaf(qf[e], __bfloat162float(k[e]), s);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, x);
        const float mn = fmaxf(m, s);
        const float mu = mn == -INFINITY ? 0.0f : mn;
        const float a = exp2f(m - mu), w = exp2f(s - mu);
        const float before = l * a;
        l = before + w;
        const float keep = l == 0.0f ? 1.0f : before / l, take = l == 0.0f ? 0.0f : w / l;
#pragma unroll
        for (int e = 0; e < PER; e++)
            o[e] = fmaf(take, __bfloat162float(v[e]), o[e] * keep);
        m = mn;
    }
    __nv_bfloat16 *out = p.out + (t * p.hq + h) * DIM + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; e++)
        out[e] = __float2bfloat16_rn(l == 0.0f ? 0.0f : o[e]);
    if (p.lse && lane == 0)
        p.lse[t * p.hq + h] = l == 0.0f ? -INFINITY : LN2 * (m + log2f(l));
}

// What of the lane's DIM / 32 columns is not finite: bit e for NaN in column e, bit 4 + e for +infinity, bit 8 + e for -infinity.
template <int DIM> __device__ __forceinline__ unsigned odd_kinds(const uint32_t (&x)[DIM / 64])
{
    unsigned kinds = 0;
#pragma unroll
    for (int e = 0; e < DIM / 32; e++) {
        const uint32_t u = e & 1 ? x[e / 2] >> 16 : x[e / 2] & 0xffffu;
        if ((u & 0x7f80u) == 0x7f80u)
            kinds |= 1u << (e + (u & 0x7fu ? 0 : (u & 0x8000u ? 8 : 4)));
    }
    return kinds;
}
// What of these output kinds the values found do not account for: an infinity takes one of its sign, NaN a NaN or both
// infinities.
__device__ __forceinline__ unsigned unexplained(unsigned kinds, unsigned found)
{
    return kinds & ~(found | (found >> 4 & found >> 8 & 15u));
}
// The kinds of values that are not finite at the positions a..b of sequence n, by a whole warp; it stops when they account for
// all that is wanted (~0u: never).  16 positions at a time, which lie in one page.
template <int DIM>
__device__ unsigned odd_values(const AttnArgs &p, int n, int kvh, int a, int b, unsigned wanted)
{
    constexpr int WORDS = DIM / 64;
    const int lane = threadIdx.x & 31;
    unsigned found = 0;
    for (int j0 = a & -16; j0 <= b; j0 += 16) {
        const int64_t row = cache_row(p.cache, n, j0);
        if (row < 0)
            continue;
        const uint32_t *v = reinterpret_cast<const uint32_t *>(p.cache.v + row + ((int64_t)kvh << p.cache.page_shift) * DIM) + lane * WORDS;
        uint32_t x[16][WORDS];
#pragma unroll
        for (int i = 0; i < 16; i++)
#pragma unroll
            for (int w = 0; w < WORDS; w++)
                x[i][w] = j0 + i >= a && j0 + i <= b ? v[i * (DIM / 2) + w] : 0;
#pragma unroll
        for (int i = 0; i < 16; i++)
            found |= odd_kinds<DIM>(x[i]);
        if (__all_sync(0xffffffffu, unexplained(wanted, found) == 0))
            break;
    }
    return found;
}

// Rows (one a lane, those of the mask `again`) of sequence n and one key head whose softmax sum is finite and whose output,
// which has been stored, is not.  (A sum that is not finite comes from the row's own scores: its output is NaN by
// definition.)  Three things do that: a value that the row sees and that is not finite, and then the output is right; one that
// it does not see and that a tensor-core product took in (0 x infinity); and finite values whose sum passes fp32's range.  So a
// row is left as it is when none of the positions that its products may have taken in and that it does not see holds such a value in
// one of the output's columns that are not finite, and for each of these columns what it sees makes that infinity or that NaN.
// The others are taken again by attn_row.  The products take in what the CTA's other rows see: up to `margin` positions before the row's window and
// behind its own position, and the rest of the sinks' last 32.  All rows are looked at together first.
// Measured with one NaN in a value of the call: 8192 tokens, 96 heads over 8 (1.21 ms without), the NaN in the first tokens
// 1.47 ms, half way 39 ms, nearly all of it attn_row for the tile's rows in front of the NaN; every row by attn_row 320 ms.  A
// decode step of 256 sequences 0.17 to 0.29 ms (0.17 without, 2.0 by attn_row).
// By a whole warp; true when an entry of the page table was out of range.
template <int DIM>
__device__ __noinline__ bool attn_mend_rows(const AttnArgs &p, int n, unsigned again, int t, int h, int pos, int margin)
{
    constexpr unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    bool bad = false;
    __syncwarp();                                    // the rows' stores come before what follows
    const int last = (int)cache_len(p.cache, n, bad) - 1, kvh = __shfl_sync(FULL, h, __ffs(again) - 1) / p.group;
    auto kinds_of = [&](int src) -> unsigned {       // the row's output
        const int64_t at = (int64_t)__shfl_sync(FULL, t, src) * p.hq + __shfl_sync(FULL, h, src);
        const uint32_t *o = reinterpret_cast<const uint32_t *>(p.out + at * DIM) + lane * (DIM / 64);
        uint32_t x[DIM / 64];
#pragma unroll
        for (int w = 0; w < DIM / 64; w++)
            x[w] = o[w];
        return odd_kinds<DIM>(x);
    };
    // rows at positions a..b, whose outputs have these kinds, are right as they are
    auto right = [&](int a, int b, unsigned kinds) -> bool {
        const int gone = b - p.window;               // the last position before b's window
        unsigned hidden = odd_values<DIM>(p, n, kvh, max(max(a - p.window + 1 - margin, p.sinks), 0), gone, ~0u);
        hidden |= odd_values<DIM>(p, n, kvh, a + 1, min(b + margin, last), ~0u);
        hidden |= odd_values<DIM>(p, n, kvh, p.sinks, min(((p.sinks + 31) & -32) - 1, gone), ~0u);
        const unsigned columns = (kinds | kinds >> 4 | kinds >> 8) & 15u;
        if (__any_sync(FULL, ((hidden | hidden >> 4 | hidden >> 8) & columns) != 0))
            return false;
        unsigned seen = odd_values<DIM>(p, n, kvh, 0, min(p.sinks - 1, a), kinds);
        if (__any_sync(FULL, unexplained(kinds, seen) != 0))
            seen |= odd_values<DIM>(p, n, kvh, max(gone + 1, p.sinks), a, unexplained(kinds, seen));
        return __all_sync(FULL, unexplained(kinds, seen) == 0);
    };
    if (again & (again - 1)) {
        int a = INT32_MAX, b = 0;
        unsigned kinds = 0;
        for (unsigned x = again; x; x &= x - 1) {
            const int src = __ffs(x) - 1, at = __shfl_sync(FULL, pos, src);
            a = min(a, at);
            b = max(b, at);
            kinds |= kinds_of(src);
        }
        if (right(a, b, kinds))
            return bad;
    }
    for (; again; again &= again - 1) {
        const int src = __ffs(again) - 1, at = __shfl_sync(FULL, pos, src);
        if (!right(at, at, kinds_of(src)))
            attn_row<DIM>(p, n, __shfl_sync(FULL, t, src), __shfl_sync(FULL, h, src), at, bad);
    }
    return bad;
}

}  // namespace kda
