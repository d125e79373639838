// Linear attention token by token: single tokens and short runs.
//
//   S_t = e^(a_t) S_(t-1) + v_t k_t^T  (rows v, columns k, as stored),   o_t = scale S_t q_t
//
// A row of the state needs only its own v and all of k and q, so the rows are dealt out to warps: a warp takes NI rows of
// each of its RPI groups of LPR lanes, a lane E neighbouring columns of them (one 16-byte vector of the state), and the
// state stays in fp32 registers from the first token to the last.  The rows' sums over the lanes go through a butterfly that
// halves the rows a lane holds as it doubles the lanes that a sum covers, NI - 1 shuffles and not NI log2(LPR).
// The state is read once and written once, which is the floor of a single token.
//
// Measured (one GPU): 256 sequences of one token, 96 heads of 128, fp32 states (3.25 GB) 457 us, 7.1 TB/s, the memory's rate; one sequence
// of 32 heads 2.7 us, a launch; 64 sequences of up to 5 tokens, 64 heads over 8, bf16 states 56.4 us, 4.9 TB/s (40.8 at the memory's rate):
// there the tokens' arithmetic on the state takes 33 us of issue slots (two-wide; 80 us in all without).  Rows a warp, bf16: 8 of each lane group
// 56 us, 4 64 (fp32: 16 and 8 take the same).  A gate is only looked at in its turn: at once, its load held up the warp (60.8 us).
#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int THREADS = 128;
constexpr unsigned FULL = 0xffffffffu;

// A 16-byte vector of the state, as pairs for the two-wide fp32 arithmetic (which halves what several tokens a state take).
template <typename STATE> struct Vec;
template <> struct Vec<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ void load(const float *p, f2 (&x)[2])
    {
        const float4 y = __ldcs(reinterpret_cast<const float4 *>(p));
        x[0] = f2_pack(y.x, y.y), x[1] = f2_pack(y.z, y.w);
    }
    static __device__ __forceinline__ void store(float *p, const f2 (&x)[2])
    {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(f2_lo(x[0]), f2_hi(x[0]), f2_lo(x[1]), f2_hi(x[1])));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void load(const __nv_bfloat16 *p, f2 (&x)[4])
    {
        const uint4 y = __ldcs(reinterpret_cast<const uint4 *>(p));
        x[0] = f2_bf16x2(y.x), x[1] = f2_bf16x2(y.y), x[2] = f2_bf16x2(y.z), x[3] = f2_bf16x2(y.w);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const f2 (&x)[4])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __nv_bfloat162 y = __floats2bfloat162_rn(f2_lo(x[i]), f2_hi(x[i]));
            w[i] = *reinterpret_cast<const uint32_t *>(&y);
        }
        __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
    }
};

// E bf16 of a token's head, as words
template <int E> __device__ __forceinline__ void load_bf16(const __nv_bfloat16 *p, uint32_t (&w)[E / 2])
{
    if constexpr (E == 4) {
        const uint2 y = *reinterpret_cast<const uint2 *>(p);
        w[0] = y.x, w[1] = y.y;
    } else {
#pragma unroll
        for (int i = 0; i < E / 8; i++) {
            const uint4 y = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = y.x, w[4 * i + 1] = y.y, w[4 * i + 2] = y.z, w[4 * i + 3] = y.w;
        }
    }
}

// Sums of o[0..CNT) over LANES lanes: on return o[0] is the sum of row `row` (added to), the same in `LANES` lanes at the end.
template <int CNT, int LANES, int NI> __device__ __forceinline__ void sum_rows(float (&o)[NI], int lane, int &row)
{
    if constexpr (LANES > 1) {
        if constexpr (CNT > 1) {
            const bool up = lane & (LANES / 2);
#pragma unroll
            for (int j = 0; j < CNT / 2; j++) {
                const float give = up ? o[j] : o[j + CNT / 2], keep = up ? o[j + CNT / 2] : o[j];
                o[j] = keep + __shfl_xor_sync(FULL, give, LANES / 2);
            }
            row += up ? CNT / 2 : 0;
            sum_rows<CNT / 2, LANES / 2, NI>(o, lane, row);
        } else {
            o[0] += __shfl_xor_sync(FULL, o[0], LANES / 2);
            sum_rows<1, LANES / 2, NI>(o, lane, row);
        }
    }
}

template <int DIM, typename STATE, int NI>
__global__ void __launch_bounds__(THREADS) kda_linear_tokens_kernel(const LinearArgs p)
{
    using V = Vec<STATE>;
    constexpr int E = V::E, LPR = DIM / E, RPI = 32 / LPR, ROWS = NI * RPI, PARTS = DIM / ROWS;
    static_assert(NI <= LPR && NI % 4 == 0, "a lane holds at most one row's sum at the end");
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * (THREADS / 32) + threadIdx.x / 32, pair = w / PARTS;
    if (pair >= (int64_t)p.tok.N * p.H)
        return;
    const int n = (int)(pair / p.H), h = (int)(pair % p.H), c = lane % LPR;
    const int row0 = (int)(w % PARTS) * ROWS + lane / LPR * NI;
    const int64_t at = (pair * DIM + row0) * DIM + c * E;
    stream_order();
    f2 s[NI][E / 2];
#pragma unroll
    for (int i = 0; i < NI; i++) {
        if (p.init) {
            V::load(static_cast<const STATE *>(p.init) + at + (int64_t)i * DIM, s[i]);
        } else {
#pragma unroll
            for (int e = 0; e < E / 2; e++)
                s[i][e] = 0;
        }
    }
    const float fixed = p.log_decay ? p.log_decay[h] : 0.0f;
    const int hk = h / p.group;
    // a token's values are read while the one before it is worked on, and not looked at before their turn
    uint32_t q[E / 2], k[E / 2], v[NI / 2];
    float gate = 0.0f;
    auto read = [&](int64_t t) {
        gate = gate_of(p, t, h);
        load_bf16<E>(p.q + t * p.q_stride + h * DIM + c * E, q);
        load_bf16<E>(p.k + t * p.k_stride + hk * DIM + c * E, k);
        load_bf16<NI>(p.v + t * p.v_stride + hk * DIM + row0, v);
    };
    // the first ones, where it is known which, before the sequence's length is (it may be 0: they are not used then)
    if (!p.tok.cu && p.tok.T > 0)
        read(n * p.tok.T);
    bool bad = false;
    int64_t bos, len;
    linear_range(p, n, bos, len, bad);
    if (p.tok.cu && len > 0)
        read(bos);
    for (int64_t t = bos; t < bos + len; t++) {
        const float decay = expf(log_decay_of(fixed, gate, bad));
        const f2 decay2 = f2_pack(decay, decay);
        f2 q2[E / 2], k2[E / 2];
        float vf[NI], o[NI];
#pragma unroll
        for (int e = 0; e < E / 2; e++)
            q2[e] = f2_bf16x2(q[e]), k2[e] = f2_bf16x2(k[e]);
#pragma unroll
        for (int i = 0; i < NI; i += 2)
            vf[i] = bf16_lo(v[i / 2]), vf[i + 1] = bf16_hi(v[i / 2]);
        if (t + 1 < bos + len)
            read(t + 1);
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const f2 v2 = f2_pack(vf[i], vf[i]);
            f2 sum = 0;
#pragma unroll
            for (int e = 0; e < E / 2; e++) {
                s[i][e] = f2_fma(decay2, s[i][e], f2_mul(v2, k2[e]));
                sum = f2_fma(s[i][e], q2[e], sum);
            }
            o[i] = f2_lo(sum) + f2_hi(sum);
        }
        int row = row0;
        sum_rows<NI, LPR, NI>(o, lane, row);
        if (lane % (LPR / NI) == 0)
            p.out[(t * p.H + h) * DIM + row] = __float2bfloat16_rn(p.scale * o[0]);
    }
    if (p.fin) {
#pragma unroll
        for (int i = 0; i < NI; i++)
            V::store(static_cast<STATE *>(p.fin) + at + (int64_t)i * DIM, s[i]);
    }
    report(p.err, bad && lane == 0, DEVERR_CU_SEQLENS);
}

template <int DIM, typename STATE, int NI> cudaError_t launch(const LinearArgs &p, cudaStream_t st)
{
    constexpr int ROWS = NI * (32 / (DIM / Vec<STATE>::E)), PARTS = DIM / ROWS;
    const int64_t warps = (int64_t)p.tok.N * p.H * PARTS;
    return launch_in_row(kda_linear_tokens_kernel<DIM, STATE, NI>, (unsigned)((warps + THREADS / 32 - 1) / (THREADS / 32)), THREADS,
                         0, 1, st, p);
}

}  // namespace

cudaError_t launch_linear_tokens(const LinearArgs &p, kda_dtype_t state, cudaStream_t st)
{
    if (state == KDA_DTYPE_BF16)
        return p.dim == 128 ? launch<128, __nv_bfloat16, 8>(p, st) : launch<64, __nv_bfloat16, 8>(p, st);
    return p.dim == 128 ? launch<128, float, 16>(p, st) : launch<64, float, 16>(p, st);
}

}  // namespace kda
