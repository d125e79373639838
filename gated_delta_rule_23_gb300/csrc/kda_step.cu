// Host-side helpers shared by the decoder-step operators, and the device word their kernels report in.
#include "kda_step.cuh"

#include <atomic>

__device__ unsigned int g_kda_step_error;   // DEVERR_* bits of the decoder-step kernels (read by kda_device_status)

namespace kda {

cudaError_t step_error_word(unsigned int **word)
{
    static std::atomic<unsigned int *> cache[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    unsigned int *p = cache[dev].load(std::memory_order_acquire);
    if (!p) {
        void *a = nullptr;
        e = cudaGetSymbolAddress(&a, g_kda_step_error);
        if (e != cudaSuccess)
            return e;
        p = static_cast<unsigned int *>(a);
        cache[dev].store(p, std::memory_order_release);
    }
    *word = p;
    return cudaSuccess;
}

cudaError_t step_read_and_clear_error(unsigned int *flag)
{
    cudaError_t e = cudaMemcpyFromSymbol(flag, g_kda_step_error, sizeof *flag);
    if (e == cudaSuccess && *flag) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_kda_step_error, &zero, sizeof zero);
    }
    return e;
}

int device_sms()
{
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 0;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return 0;
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Checks that the cache and token arguments of kda_kv_append and kda_window_attn share (no CUDA calls).
kda_status_t check_cache_args(const void *k_cache, const void *v_cache, const int32_t *block_table,
                              const int32_t *kv_lens, const int64_t *cu_seqlens, int N, int64_t T, int Hkv, int D,
                              int64_t pages, int page, int max_pages)
{
    if (!k_cache || !v_cache || !block_table || !kv_lens || N < 1 || T < 0 || Hkv < 1 || pages < 1 || max_pages < 1)
        return KDA_ERR_INVALID_ARGUMENT;
    if (!is_aligned(k_cache, 16) || !is_aligned(v_cache, 16) || !is_aligned(block_table, 4) ||
        !is_aligned(kv_lens, 4) || !is_aligned(cu_seqlens, 8))
        return KDA_ERR_INVALID_ARGUMENT;
    if (page < 16 || page > 4096 || (page & (page - 1)))
        return KDA_ERR_INVALID_ARGUMENT;
    if (D != 64 && D != 128)
        return KDA_ERR_UNSUPPORTED;
    // cache rows and tokens are 32-bit coordinates of the bulk copies and of the launch grids
    if (pages > INT32_MAX / page || pages * page > INT32_MAX / Hkv || (int64_t)max_pages * page > INT32_MAX - 8192)
        return KDA_ERR_UNSUPPORTED;
    if (T > INT32_MAX || (cu_seqlens ? T : (int64_t)N * T) > INT32_MAX)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace kda
