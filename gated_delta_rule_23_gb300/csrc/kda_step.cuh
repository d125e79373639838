// What the decoder-step kernels (append, windowed attention, beam selection, reorder) share: the paged cache,
// the token bookkeeping, and the word they report malformed device arrays in.
#pragma once

#include "kda_device.cuh"
#include "kda_internal.h"

namespace kda {

struct PagedCache {
    __nv_bfloat16 *k, *v;        // [pages, hkv, page, dim]
    const int32_t *table;        // [N, max_pages]
    const int32_t *lens;         // [N]
    int64_t pages;
    int page_shift, max_pages, hkv, dim;
};

struct Tokens {
    const int64_t *cu;           // cu_seqlens or nullptr
    int64_t T;                   // tokens per sequence (cu == nullptr) or in all
    int N;
};

inline PagedCache make_cache(const void *k, const void *v, const int32_t *table, const int32_t *lens, int hkv, int dim,
                             int64_t pages, int page, int max_pages)
{
    PagedCache c{};
    c.k = static_cast<__nv_bfloat16 *>(const_cast<void *>(k));
    c.v = static_cast<__nv_bfloat16 *>(const_cast<void *>(v));
    c.table = table, c.lens = lens;
    c.pages = pages, c.max_pages = max_pages, c.hkv = hkv, c.dim = dim;
    while ((1 << c.page_shift) < page)
        c.page_shift++;
    return c;
}

// The decoder-step kernels are short and run in a row, so each may be set up while the one before it in its stream ends
// (programmatic dependent launch): stream_order() stands before anything that reads or writes memory, and waits until all
// kernels before are through and their writes to be seen; after it the next kernel may be set up.  What they read may
// be those kernels' output: no read-only (.nc) loads, which need not stay behind the wait.  Calls in a row, launched plainly |
// this way: append of one token 4.1 | 2.8 us, attention of one sequence's step 10.3 | 8.9, beam selection of 4 x 32001
// 12.3 | 9.1, chunks of 509 22.5 | 20.6.
__device__ __forceinline__ void stream_order()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
}
template <typename... P, typename... A>
cudaError_t launch_in_row(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st, const A &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

kda_status_t check_cache_args(const void *k_cache, const void *v_cache, const int32_t *block_table,
                              const int32_t *kv_lens, const int64_t *cu_seqlens, int N, int64_t T, int Hkv, int D,
                              int64_t pages, int page, int max_pages);

// Tokens of the cache that sequence n has, clamped into what its table can address.
__device__ __forceinline__ int64_t cache_len(const PagedCache &c, int n, bool &bad)
{
    const int64_t cap = (int64_t)c.max_pages << c.page_shift;
    const int64_t len = c.lens[n];
    bad |= len < 0 || len > cap;
    return len < 0 ? 0 : (len > cap ? cap : len);
}

// Element offset of (position, head 0) of sequence n in the cache, or -1 when its page id is out of range.
// 64-bit: a cache may hold more than 2^31 elements.
__device__ __forceinline__ int64_t cache_row(const PagedCache &c, int n, int64_t pos)
{
    const int32_t id = c.table[(int64_t)n * c.max_pages + (pos >> c.page_shift)];
    if (id < 0 || id >= c.pages)
        return -1;
    return (((int64_t)id * c.hkv << c.page_shift) + (pos & ((1 << c.page_shift) - 1))) * c.dim;
}

// Sequence of token t (0 <= t < T) of a ragged batch: the last n with cu[n] <= t, by a whole warp (32 entries
// a step; cu is non-decreasing when it is valid, and the result stays in [0, N) when it is not).
__device__ __forceinline__ int seq_of_token(const int64_t *cu, int N, int64_t t)
{
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int base = 0; base < N; base += 32) {
        const bool le = base + lane < N && cu[base + lane] <= t;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        if (m)
            n = base + 31 - __clz(m);
        if (m != 0xffffffffu)
            break;
    }
    return n;
}

__device__ __forceinline__ void report(unsigned int *err, bool bad, unsigned int bit)
{
    if (bad)
        atomicOr(err, bit);
}

}  // namespace kda
