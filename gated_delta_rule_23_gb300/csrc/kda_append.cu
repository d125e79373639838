// kda_kv_append: rotary positions applied to the new queries and keys, keys and values stored in the paged cache.
//
// Per pair (x, y) of a head and the position's angle a_i: (x cos a_i - y sin a_i, y cos a_i + x sin a_i), in fp32 and
// rounded once.  Every element is read once and written once: the floor is the bytes of q, k, v and their copies.
// Measured: 74 us for 8192 ragged tokens of 96 + 2 x 8 heads (472 MB), 6.4 TB/s, 94% of the measured copy rate; 2.8 us for
// one token, 4.8 for 256 (launch latency).
// A thread owns one unit of 16 elements of the head (8 pairs) and walks the token's heads with the unit's 8 cosines
// and sines in registers, so the angles are read once per token and not once per head.
#include "kda_step.cuh"

#include <algorithm>

namespace kda {
namespace {

// CTAs of 128 threads, eight an SM, with the loads of two heads in flight a thread.  8192 tokens of 96 + 2 x 8 heads of 128
// (472 MB), when launches did not overlap yet: 76 us (74 since); four heads in flight 82, one 78; CTAs of 256 threads 79 to 96.
constexpr int APPEND_THREADS = 128, CTAS_PER_SM = 8;
constexpr int FLIGHT = 2;      // heads whose loads a thread has in flight

struct AppendArgs {
    const __nv_bfloat16 *k, *v, *q;
    __nv_bfloat16 *q_out;
    int64_t k_stride, v_stride, q_stride;
    const float *cos, *sin;
    int64_t positions;
    int half, hq;
    PagedCache cache;
    Tokens tok;
    unsigned int *err;
};

struct Vec16 {
    uint4 a, b;   // the unit's two 16-byte vectors
};

__device__ __forceinline__ uint32_t rot_lo(uint32_t x, uint32_t y, const float *c, const float *s)
{
    const __nv_bfloat162 r = __floats2bfloat162_rn(bf16_lo(x) * c[0] - bf16_lo(y) * s[0],
                                                   bf16_hi(x) * c[1] - bf16_hi(y) * s[1]);
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t rot_hi(uint32_t x, uint32_t y, const float *c, const float *s)
{
    const __nv_bfloat162 r = __floats2bfloat162_rn(bf16_lo(y) * c[0] + bf16_lo(x) * s[0],
                                                   bf16_hi(y) * c[1] + bf16_hi(x) * s[1]);
    return *reinterpret_cast<const uint32_t *>(&r);
}
// a word of an interleaved pair: (x, y) in one register
__device__ __forceinline__ uint32_t rot_pair(uint32_t w, float c, float s)
{
    const float x = bf16_lo(w), y = bf16_hi(w);
    const __nv_bfloat162 r = __floats2bfloat162_rn(x * c - y * s, y * c + x * s);
    return *reinterpret_cast<const uint32_t *>(&r);
}

template <bool INTERLEAVED> __device__ __forceinline__ Vec16 rotate(const Vec16 &x, const float *c, const float *s)
{
    Vec16 r;
    if (INTERLEAVED) {
        r.a = make_uint4(rot_pair(x.a.x, c[0], s[0]), rot_pair(x.a.y, c[1], s[1]), rot_pair(x.a.z, c[2], s[2]),
                         rot_pair(x.a.w, c[3], s[3]));
        r.b = make_uint4(rot_pair(x.b.x, c[4], s[4]), rot_pair(x.b.y, c[5], s[5]), rot_pair(x.b.z, c[6], s[6]),
                         rot_pair(x.b.w, c[7], s[7]));
    } else {
        r.a = make_uint4(rot_lo(x.a.x, x.b.x, c, s), rot_lo(x.a.y, x.b.y, c + 2, s + 2),
                         rot_lo(x.a.z, x.b.z, c + 4, s + 4), rot_lo(x.a.w, x.b.w, c + 6, s + 6));
        r.b = make_uint4(rot_hi(x.a.x, x.b.x, c, s), rot_hi(x.a.y, x.b.y, c + 2, s + 2),
                         rot_hi(x.a.z, x.b.z, c + 4, s + 4), rot_hi(x.a.w, x.b.w, c + 6, s + 6));
    }
    return r;
}

// One CTA per token.
template <bool INTERLEAVED> __global__ void __launch_bounds__(APPEND_THREADS, CTAS_PER_SM) kda_append_kernel(const AppendArgs p)
{
    const int64_t t = blockIdx.x;
    const int units = p.cache.dim / 16;
    const int u = threadIdx.x % units, h0 = threadIdx.x / units, hstep = APPEND_THREADS / units;
    bool bad = false;
    int n;
    int64_t i, len_q;
    stream_order();
    if (p.tok.cu) {
        int64_t bos;
        n = seq_of_token(p.tok.cu, p.tok.N, t);
        bad |= seq_range(p.tok.cu, n, p.tok.N, p.tok.T, bos, len_q);
        i = t - bos;
    } else {
        n = (int)(t / p.tok.T);
        i = t - (int64_t)n * p.tok.T;
        len_q = p.tok.T;
    }
    int64_t pos = cache_len(p.cache, n, bad) - len_q + i;
    // a token outside its sequence (malformed cu_seqlens) has no place either
    if (i < 0 || i >= len_q)
        pos = -1;
    if (pos >= ((int64_t)p.cache.max_pages << p.cache.page_shift))
        pos = -1;
    const int64_t row = pos >= 0 ? cache_row(p.cache, n, pos) : -1;
    bad |= pos >= 0 && row < 0;

    // the unit's two vectors: 8 elements from e0, 8 from e1
    const bool turn = p.half > 0 && u < p.half / 8 && pos >= 0;
    const int split = p.half > 0 && u < p.half / 8;
    const int e0 = split ? (INTERLEAVED ? 16 * u : 8 * u) : 16 * u;
    const int e1 = split ? (INTERLEAVED ? 16 * u + 8 : p.half + 8 * u) : 16 * u + 8;
    float c[8], s[8];
    if (turn) {
        bad |= pos >= p.positions;
        const int64_t at = (pos < p.positions ? pos : p.positions - 1) * p.half + 8 * u;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            c[j] = p.cos[at + j];
            s[j] = p.sin[at + j];
        }
    }
    const int total = p.hq + 2 * p.cache.hkv;
    for (int first = h0; first < total; first += FLIGHT * hstep) {
        // all loads before the stores (q_out may be q, so the compiler would keep them in turn)
        Vec16 x[FLIGHT];
        __nv_bfloat16 *dst[FLIGHT];
#pragma unroll
        for (int i = 0; i < FLIGHT; i++) {
            const int h = first + i * hstep;
            const __nv_bfloat16 *src = nullptr;
            dst[i] = nullptr;
            if (h < p.hq) {
                src = p.q + t * p.q_stride + (int64_t)h * p.cache.dim;
                dst[i] = p.q_out + (t * p.hq + h) * p.cache.dim;
            } else if (h < total && row >= 0) {
                const bool is_k = h < p.hq + p.cache.hkv;
                const int g = h - p.hq - (is_k ? 0 : p.cache.hkv);
                src = (is_k ? p.k + t * p.k_stride : p.v + t * p.v_stride) + (int64_t)g * p.cache.dim;
                dst[i] = (is_k ? p.cache.k : p.cache.v) + row + ((int64_t)g << p.cache.page_shift) * p.cache.dim;
            }
            if (src) {
                x[i].a = __ldcs(reinterpret_cast<const uint4 *>(src + e0));
                x[i].b = __ldcs(reinterpret_cast<const uint4 *>(src + e1));
            }
        }
#pragma unroll
        for (int i = 0; i < FLIGHT; i++) {
            if (!dst[i])
                continue;
            if (turn && first + i * hstep < p.hq + p.cache.hkv)
                x[i] = rotate<INTERLEAVED>(x[i], c, s);
            *reinterpret_cast<uint4 *>(dst[i] + e0) = x[i].a;
            *reinterpret_cast<uint4 *>(dst[i] + e1) = x[i].b;
        }
    }
    report(p.err, bad && threadIdx.x == 0, DEVERR_CU_SEQLENS);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status_t kda_kv_append(const void *k, int64_t k_stride, const void *v, int64_t v_stride, void *k_cache,
                                      void *v_cache, const int32_t *block_table, const int32_t *kv_lens,
                                      const float *cos, const float *sin, int rotary, int64_t positions,
                                      int interleaved, const void *q, int64_t q_stride, void *q_out,
                                      const int64_t *cu_seqlens, int N, int64_t T, int Hq, int Hkv, int D,
                                      int64_t pages, int page, int max_pages, kda_stream_t stream)
{
    const kda_status_t s = check_cache_args(k_cache, v_cache, block_table, kv_lens, cu_seqlens, N, T, Hkv, D, pages,
                                            page, max_pages);
    if (s != KDA_OK)
        return s;
    if (Hq < 0 || (Hq > 0) != (q != nullptr) || (Hq > 0) != (q_out != nullptr) || !cos != !sin)
        return KDA_ERR_INVALID_ARGUMENT;
    if (cos && (rotary < 16 || rotary % 16 || rotary > D || positions < 1))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!is_aligned(cos, 16) || !is_aligned(sin, 16))
        return KDA_ERR_INVALID_ARGUMENT;
    const int64_t tokens = cu_seqlens ? T : (int64_t)N * T;
    if (tokens == 0)
        return KDA_OK;
    if (!k || !v || !is_aligned(k, 16) || !is_aligned(v, 16) || !is_aligned(q, 16) || !is_aligned(q_out, 16))
        return KDA_ERR_INVALID_ARGUMENT;
    if (k_stride % 8 || k_stride < (int64_t)Hkv * D || v_stride % 8 || v_stride < (int64_t)Hkv * D ||
        (q && (q_stride % 8 || q_stride < (int64_t)Hq * D)))
        return KDA_ERR_INVALID_ARGUMENT;
    if (q == q_out && q && q_stride != (int64_t)Hq * D)
        return KDA_ERR_INVALID_ARGUMENT;
    // a CTA takes a token: what another token reads is not written, but for q in place
    const uint64_t before = (uint64_t)tokens - 1, turned = (uint64_t)tokens * Hq * D * 2;
    if ((q != q_out && overlap(q_out, turned, q, (before * q_stride + (uint64_t)Hq * D) * 2)) ||
        overlap(q_out, turned, k, (before * k_stride + (uint64_t)Hkv * D) * 2) ||
        overlap(q_out, turned, v, (before * v_stride + (uint64_t)Hkv * D) * 2))
        return KDA_ERR_INVALID_ARGUMENT;
    AppendArgs p{};
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.k_stride = k_stride, p.v_stride = v_stride, p.q_stride = q_stride;
    p.cos = cos, p.sin = sin, p.positions = positions;
    p.half = cos ? rotary / 2 : 0;
    p.hq = Hq;
    p.cache = make_cache(k_cache, v_cache, block_table, kv_lens, Hkv, D, pages, page, max_pages);
    p.tok = Tokens{cu_seqlens, T, N};
    if (step_error_word(&p.err) != cudaSuccess)
        return KDA_ERR_CUDA;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)tokens;
    const cudaError_t e = interleaved ? launch_in_row(kda_append_kernel<true>, grid, APPEND_THREADS, 0, 1, st, p)
                                      : launch_in_row(kda_append_kernel<false>, grid, APPEND_THREADS, 0, 1, st, p);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
