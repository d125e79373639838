// kda_window_attn: argument checks and dispatch.
#include "kda_attn.cuh"

namespace kda {
namespace {

constexpr int ROW_THREADS = 256;

// One warp per query row.
template <int DIM> __global__ void __launch_bounds__(ROW_THREADS) kda_attn_row_kernel(const AttnArgs p, int64_t rows)
{
    const int64_t r = (int64_t)blockIdx.x * (ROW_THREADS / 32) + threadIdx.x / 32;
    if (r >= rows)
        return;
    const int64_t t = r / p.hq;
    const int h = (int)(r % p.hq);
    bool bad = false;
    int n;
    int64_t i, len_q;
    if (p.tok.cu) {
        int64_t bos;
        n = seq_of_token(p.tok.cu, p.tok.N, t);
        bad |= seq_range(p.tok.cu, n, p.tok.N, p.tok.T, bos, len_q);
        i = t - bos;
        if (i < 0 || i >= len_q)
            i = -(int64_t)INT32_MAX - 1;
    } else {
        n = (int)(t / p.tok.T);
        i = t - (int64_t)n * p.tok.T;
        len_q = p.tok.T;
    }
    attn_row<DIM>(p, n, t, h, cache_len(p.cache, n, bad) - len_q + i, bad);
    report(p.err, bad, DEVERR_CU_SEQLENS);
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
    p.scale_log2 = scale * LOG2E;
    p.window = window, p.sinks = sinks;
    p.hq = Hq, p.group = Hq / Hkv;
    p.cache = make_cache(k_cache, v_cache, block_table, kv_lens, Hkv, D, pages, page, max_pages);
    p.tok = Tokens{cu_seqlens, T, N};
    return p;
}

cudaError_t launch_attn(const AttnArgs &p, int64_t tokens, cudaStream_t st)
{
    const int64_t rows = tokens * p.hq;
    const unsigned grid = (unsigned)((rows + ROW_THREADS / 32 - 1) / (ROW_THREADS / 32));
    if (p.cache.dim == 128)
        kda_attn_row_kernel<128><<<grid, ROW_THREADS, 0, st>>>(p, rows);
    else
        kda_attn_row_kernel<64><<<grid, ROW_THREADS, 0, st>>>(p, rows);
    return cudaGetLastError();
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t kda_window_attn_workspace_size(int window, int sinks, int varlen, int N, int64_t T, int Hq, int Hkv,
                                                 int D, int page, int max_pages)
{
    return 0;
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
    return launch_attn(p, tokens, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
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
