// kda_window_attn: argument checks and dispatch.
#include "kda_attn.cuh"

#include <cfloat>

namespace kda {
namespace {

constexpr int ROW_THREADS = 256;

// Joins the partial results of a split call:
//   out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s,  M = max m_s.
// PER_ROW warps take a query row, each every PER_ROW-th split, eight splits' loads in flight; the order of the sums is
// fixed.  The lanes read 32 splits' statistics at once.  A row that does not come out finite is taken again from the
// definition (see kda_attn_tiles.cu).
template <int DIM, int PER_ROW>
__global__ void __launch_bounds__(ROW_THREADS) kda_attn_join_kernel(const __grid_constant__ AttnArgs p, const AttnPlan plan)
{
    constexpr int PER = DIM / 32, WARPS = ROW_THREADS / 32, FLIGHT = 8;
    __shared__ float part[WARPS][DIM];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, sub = warp % PER_ROW;
    const int64_t r = (int64_t)blockIdx.x * (WARPS / PER_ROW) + warp / PER_ROW;
    stream_order();
    const bool in = r < plan.rows;
    float m = -INFINITY, l = 0.0f, o[PER];
#pragma unroll
    for (int e = 0; e < PER; e++)
        o[e] = 0.0f;
    if (in) {
        // the statistics, split `lane` and split 32 + lane (there are 64 at most), as weights
        float w2[2] = {-1.0f, -1.0f};
        float2 st[2] = {make_float2(-INFINITY, 0.0f), make_float2(-INFINITY, 0.0f)};
#pragma unroll
        for (int i = 0; i < 2; i++)
            if (32 * i + lane < plan.splits)
                st[i] = plan.part_ml[(32 * i + lane) * plan.rows + r];
        m = fmaxf(st[0].x, st[1].x);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        const float mu = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < 2; i++)
            if (!(st[i].x == -INFINITY && st[i].y == 0.0f)) {      // a split with a visible key
                w2[i] = exp2f(st[i].x - mu);
                l += w2[i] * st[i].y;
            }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1)
            l += __shfl_xor_sync(0xffffffffu, l, x);
        for (int s0 = sub; s0 < plan.splits; s0 += FLIGHT * PER_ROW) {
            float v[FLIGHT][PER];
#pragma unroll
            for (int i = 0; i < FLIGHT; i++) {
                const int s = s0 + i * PER_ROW;
                if (s < plan.splits) {
                    const float *src = plan.part_o + (s * plan.rows + r) * DIM + lane * PER;
#pragma unroll
                    for (int e = 0; e < PER; e++)
                        v[i][e] = src[e];
                }
            }
#pragma unroll
            for (int i = 0; i < FLIGHT; i++) {
                const int s = s0 + i * PER_ROW;
                const float w = __shfl_sync(0xffffffffu, s < 32 ? w2[0] : w2[1], s & 31);
                if (s < plan.splits && !(w < 0.0f))
#pragma unroll
                    for (int e = 0; e < PER; e++)
                        o[e] = fmaf(w, v[i][e], o[e]);
            }
        }
    }
    if (PER_ROW > 1) {
#pragma unroll
        for (int e = 0; e < PER; e++)
            part[warp][lane * PER + e] = o[e];
        __syncthreads();
        if (sub == 0)
#pragma unroll
            for (int i = 1; i < PER_ROW; i++)
#pragma unroll
                for (int e = 0; e < PER; e++)
                    o[e] += part[warp + i][lane * PER + e];
    }
    if (!in || sub)
        return;
    bool finite = true;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    __nv_bfloat16 *out = p.out + r * DIM + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; e++) {
        finite &= fabsf(o[e]) <= FLT_MAX;
        out[e] = __float2bfloat16_rn(l == 0.0f ? 0.0f : o[e] * inv);
    }
    if (p.lse && lane == 0)
        p.lse[r] = l == 0.0f ? -INFINITY : LN2 * (m + log2f(l));
    if (l > 0.0f && l <= FLT_MAX && __any_sync(0xffffffffu, !finite)) {
        const int64_t t = r / p.hq;
        bool bad = false;
        int64_t i, len;
        const int n = token_place(p.tok, t, i, len, bad);
        if (i >= 0 && i < len)
            attn_mend_rows<DIM>(p, n, 1, (int)t, (int)(r % p.hq), (int)(cache_len(p.cache, n, bad) - len + i), plan.margin);
    }
}

kda_status_t check_attn(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
                        const int32_t *block_table, const int32_t *kv_lens, const void *out, const float *lse,
                        float scale, int window, int sinks, const int64_t *cu_seqlens, int N, int64_t T, int Hq,
                        int Hkv, int D, int64_t pages, int page, int max_pages)
{
    const kda_status_t s = check_cache_args(k_cache, v_cache, block_table, kv_lens, cu_seqlens, N, T, Hkv, D, pages,
                                            page, max_pages);
    if (s != KDA_OK)
        return s;
    if (Hq < 1 || Hq % Hkv || window < 1 || sinks < 0)
        return KDA_ERR_INVALID_ARGUMENT;
    if (Hq / Hkv > ATTN_ROWS)
        return KDA_ERR_UNSUPPORTED;
    if (!(scale >= 0.0f) || scale > 3.0e38f)
        return KDA_ERR_UNSUPPORTED;
    const int64_t tokens = cu_seqlens ? T : (int64_t)N * T;
    if (tokens * Hq > INT32_MAX)
        return KDA_ERR_UNSUPPORTED;
    if (tokens == 0)
        return KDA_OK;
    if (!q || !out || !is_aligned(q, 16) || !is_aligned(out, 16) || !is_aligned(lse, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    if (q_stride % 8 || q_stride < (int64_t)Hq * D)
        return KDA_ERR_INVALID_ARGUMENT;
    // rows that are taken again read q after the first out is stored
    const uint64_t rows = (uint64_t)tokens * Hq, read = ((uint64_t)(tokens - 1) * q_stride + (uint64_t)Hq * D) * 2;
    if (overlap(out, rows * D * 2, q, read) || overlap(lse, rows * 4, q, read) || overlap(lse, rows * 4, out, rows * D * 2))
        return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

AttnArgs make_attn(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
                   const int32_t *block_table, const int32_t *kv_lens, void *out, float *lse, float scale, int window,
                   int sinks, const int64_t *cu_seqlens, int N, int64_t T, int Hq, int Hkv, int D, int64_t pages,
                   int page, int max_pages)
{
    AttnArgs p{};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.q_stride = q_stride;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    // never 0, which would make NaN of a masked score's -inf: scores times this are 0 all the same
    p.scale_log2 = fmaxf(scale * LOG2E, FLT_MIN);
    // no position is beyond what the table addresses, so neither need a bound be
    const int cap = max_pages * page;
    p.window = window < cap ? window : cap, p.sinks = sinks < cap ? sinks : cap;
    p.hq = Hq, p.group = Hq / Hkv;
    p.cache = make_cache(k_cache, v_cache, block_table, kv_lens, Hkv, D, pages, page, max_pages);
    p.tok = Tokens{cu_seqlens, T, N};
    return p;
}

// Keys a tile of query rows can need at most.
int64_t most_keys(int window, int sinks, int64_t T, int page, int max_pages)
{
    const int64_t cap = (int64_t)max_pages * page, need = (int64_t)window + sinks + T;
    return need < cap ? need : cap;
}

// The cut of a call (sizes only, so that the workspace is known beforehand).  The keys are split while that still
// adds tiles for idle SMs, two key tiles to a split at least.
AttnPlan make_plan(int window, int sinks, bool varlen, int N, int64_t T, int Hq, int Hkv, int page, int max_pages)
{
    AttnPlan plan{};
    const int group = Hq / Hkv;
    const int64_t tokens = varlen ? T : (int64_t)N * T;
    plan.rows = tokens * Hq;
    plan.wait_polls = wait_limit();
    const int sms = device_sms();
    // The decode kernel: wherever 16 rows hold a key head's queries.  Splits of the keys are a cluster of 8, 4 or 2 CTAs of
    // 128 keys at least (every warp two blocks); with over 8192 keys and room for more than 8 splits they go through memory.
    // 8 splits are taken for up to sms / 16 key heads: clusters of 8 CTAs that fill an SM each leave SMs over, so 16 of them
    // do not run at once (2048 keys: 14.4 us with 8 splits, 10.3 with 4).  4 and 2 splits while each CTA has its SM: 64 key
    // heads gain nothing from a second CTA an SM (512 keys: 9.7 us with 4, 8.6 with 2), 128 lose by it (16.1 with 4,
    // 10.3 with 2 or 1).
    // With more rows, up to the tile kernel's 256, tiles of 16 take it as well while their CTAs run at once and none has
    // over 1152 keys: they read the keys again, out of L2, but fill no 128-key tiles and wait for fewer hand-overs.
    // Measured, 64 heads over 8, decode | tile kernel: 16 tokens of one sequence, window 512: 10.3 | 14.4 us, 2048: 14.6 |
    // 18.4, 4096: 20.6 | 19.0; 16 tokens of four, window 512: 14.4 | 16.5, 1024: 20.5 | 18.6.
    const int64_t row_tiles = (T * group + DECODE_ROWS - 1) / DECODE_ROWS, ctas16 = (int64_t)N * Hkv * row_tiles;
    if (!varlen && (row_tiles == 1 || (row_tiles <= ATTN_ROWS / DECODE_ROWS && ctas16 <= sms))) {
        const int64_t keys = most_keys(window, sinks, T, page, max_pages), most = keys / 128;
        int64_t s = ctas16 > 0 ? 2 * sms / ctas16 : 1;
        s = s < most ? s : most;
        s = s > 64 ? 64 : s;
        plan.cluster = s <= ATTN_CLUSTER || keys <= 1024 * ATTN_CLUSTER;
        if (plan.cluster)
            s = s >= 8 && 16 * ctas16 <= sms ? 8 : (s >= 4 && 4 * ctas16 <= sms ? 4 : (s >= 2 && 2 * ctas16 <= sms ? 2 : 1));
        plan.cluster = plan.cluster && s > 1;
        if (row_tiles == 1 || (s <= ATTN_CLUSTER && keys <= 1152 * s)) {
            plan.decode = true;
            plan.row_tiles = (int)row_tiles;
            plan.granule = DECODE_KEYS;
            plan.margin = DECODE_ROWS + DECODE_KEYS;
            plan.splits = s < 1 ? 1 : (int)s;
            plan.items = (int)(ctas16 * plan.splits);
            return plan;
        }
        plan.cluster = false;
    }
    plan.granule = page < 32 ? page : 32;
    plan.run = ATTN_ROWS / group;
    plan.margin = plan.run + plan.granule;
    plan.magic = ((1u << 20) + group - 1) / group;
    int64_t tiles = varlen ? (T + (int64_t)(plan.run - 1) * N) / plan.run : (int64_t)N * ((T + plan.run - 1) / plan.run);
    if (varlen && tiles > T)
        tiles = T;                        // a tile holds a token at least
    const int64_t ctas = tiles * Hkv;
    const int64_t key_tiles = (most_keys(window, sinks, T < ATTN_ROWS ? T : ATTN_ROWS, page, max_pages) + 127) / 128 + 1;
    int64_t s = ctas > 0 ? sms / ctas : 1;
    s = s < key_tiles / 2 ? s : key_tiles / 2;
    s = s < 1 ? 1 : (s > 64 ? 64 : s);
    // 2, 4 or 8 splits (as above) as a cluster, which joins them in the same launch, unless more splits through memory save
    // over four key tiles of 128, about what the join kernel takes.
    const int64_t c = s >= 8 && 16 * ctas <= sms ? 8 : (s >= 4 ? 4 : (s >= 2 ? 2 : 1));
    plan.cluster = c > 1 && (key_tiles + c - 1) / c <= (key_tiles + s - 1) / s + 4;
    plan.splits = (int)(plan.cluster ? c : s);
    plan.items = (int)(ctas * plan.splits);
    return plan;
}

size_t plan_bytes(const AttnPlan &plan, int dim)
{
    if (plan.splits == 1 || plan.cluster)
        return 0;
    return (size_t)plan.splits * plan.rows * (dim * sizeof(float) + sizeof(float2));
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs &p, const AttnPlan &plan, cudaStream_t st)
{
    // few rows with many splits: all of a CTA's warps take one row
    const bool few = plan.splits > 4 && plan.rows <= 1024;
    const int per_cta = few ? 1 : ROW_THREADS / 32;
    const unsigned grid = (unsigned)((plan.rows + per_cta - 1) / per_cta);
    const auto launch = [&](auto *kernel) { return launch_in_row(kernel, grid, ROW_THREADS, 0, 1, st, p, plan); };
    if (few)
        return p.cache.dim == 128 ? launch(kda_attn_join_kernel<128, 8>) : launch(kda_attn_join_kernel<64, 8>);
    return p.cache.dim == 128 ? launch(kda_attn_join_kernel<128, 1>) : launch(kda_attn_join_kernel<64, 1>);
}

}  // namespace kda

using namespace kda;

extern "C" size_t kda_window_attn_workspace_size(int window, int sinks, int varlen, int N, int64_t T, int Hq, int Hkv,
                                                 int D, int page, int max_pages)
{
    if (window < 1 || sinks < 0 || N < 1 || T < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv || (D != 64 && D != 128) || page < 16 ||
        max_pages < 1 || T > INT32_MAX || (varlen ? T : (int64_t)N * T) > INT32_MAX / Hq ||
        Hq / Hkv > ATTN_ROWS)
        return 0;
    return plan_bytes(make_plan(window, sinks, varlen != 0, N, T, Hq, Hkv, page, max_pages), D);
}

extern "C" kda_status_t kda_window_attn_ws(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
                                           const int32_t *block_table, const int32_t *kv_lens, void *out, float *lse,
                                           float scale, int window, int sinks, const int64_t *cu_seqlens, int N,
                                           int64_t T, int Hq, int Hkv, int D, int64_t pages, int page, int max_pages,
                                           void *workspace, size_t workspace_bytes, kda_stream_t stream)
{
    const kda_status_t s = check_attn(q, q_stride, k_cache, v_cache, block_table, kv_lens, out, lse, scale, window,
                                      sinks, cu_seqlens, N, T, Hq, Hkv, D, pages, page, max_pages);
    if (s != KDA_OK)
        return s;
    const size_t need = kda_window_attn_workspace_size(window, sinks, cu_seqlens != nullptr, N, T, Hq, Hkv, D, page,
                                                       max_pages);
    if (need > 0 && (!workspace || !is_aligned(workspace, 256) || workspace_bytes < need))
        return KDA_ERR_INVALID_ARGUMENT;
    const int64_t tokens = cu_seqlens ? T : (int64_t)N * T;
    if (tokens == 0)
        return KDA_OK;
    AttnArgs p = make_attn(q, q_stride, k_cache, v_cache, block_table, kv_lens, out, lse, scale, window, sinks,
                           cu_seqlens, N, T, Hq, Hkv, D, pages, page, max_pages);
    if (step_error_word(&p.err) != cudaSuccess)
        return KDA_ERR_CUDA;
    AttnPlan plan = make_plan(window, sinks, cu_seqlens != nullptr, N, T, Hq, Hkv, page, max_pages);
    plan.part_o = static_cast<float *>(workspace);
    plan.part_ml = reinterpret_cast<float2 *>(plan.part_o + (size_t)plan.splits * plan.rows * D);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = plan.decode ? launch_attn_decode(p, plan, st) : launch_attn_tiles(p, plan, st);
    if (e == cudaSuccess && plan.splits > 1 && !plan.cluster)
        e = launch_attn_join(p, plan, st);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_window_attn(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
                                        const int32_t *block_table, const int32_t *kv_lens, void *out, float *lse,
                                        float scale, int window, int sinks, const int64_t *cu_seqlens, int N,
                                        int64_t T, int Hq, int Hkv, int D, int64_t pages, int page, int max_pages,
                                        kda_stream_t stream)
{
    const size_t need = kda_window_attn_workspace_size(window, sinks, cu_seqlens != nullptr, N, T, Hq, Hkv, D, page,
                                                       max_pages);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    void *ws = nullptr;
    if (need > 0) {
        // the checks come before the allocation
        const kda_status_t s = check_attn(q, q_stride, k_cache, v_cache, block_table, kv_lens, out, lse, scale,
                                          window, sinks, cu_seqlens, N, T, Hq, Hkv, D, pages, page, max_pages);
        if (s != KDA_OK)
            return s;
        if (pool_alloc(&ws, need, st) != cudaSuccess)
            return KDA_ERR_CUDA;
    }
    kda_status_t s = kda_window_attn_ws(q, q_stride, k_cache, v_cache, block_table, kv_lens, out, lse, scale, window,
                                        sinks, cu_seqlens, N, T, Hq, Hkv, D, pages, page, max_pages, ws, need,
                                        stream);
    if (ws && cudaFreeAsync(ws, st) != cudaSuccess && s == KDA_OK)
        s = KDA_ERR_CUDA;
    return s;
}
