// Linear attention in chunks of 64 tokens on the tensor cores.
//
// Within a chunk, with A_i the sum of the logarithms up to token i and S the state before the chunk (rows v, columns k):
//   P = (Q K^T) . e^(A_i - A_j)  (j <= i),   O^T = V^T P^T + e^(A_i) S Q^T,   S <- e^(A_C) S + V^T (e^(A_C - A_j) K).
// All decays are at most 1 by construction: they are exponentials of differences that are never positive, taken from sums in 64
// bits, so a strong decay beside a weak one costs no precision and none is divided by.
//
// The features lie on tensor memory's lanes: O^T and S have a row per v, so that S is the operand of its product straight from tensor
// memory (bf16, written by the threads that hold it) and leaves shared memory's bandwidth, the first bound of such a kernel, to
// the others.  Four products a chunk: Q K^T [64 x 64] (the 64 rows of A above or below are whatever lies next to Q, and their results
// are not read: the alternate chunks' rows come out on lanes 0..63 and 64..127, so that two pairs of warps take turns),
// V^T K~ [D x D], S Q^T and V^T P^T [D x 64].  D = 64 fills the lanes up with a block of zeros.
//
// The state stays in fp32 registers (eight warps): each chunk's V^T K~ comes out of tensor memory and is added there, so the tensor cores'
// own accumulation spans one chunk and what a long sequence adds up is rounded to nearest.  Weak decays are taken as
// S + (expm1(A_C) S + L): a factor next to 1 that is off by half a step in every chunk would drift by 2^-25 a chunk; strong ones as
// e^(A_C) S + L, so that nothing of a state that is forgotten stays behind as rounding.
// K~ = e^(A_C - A_j) K is not a bf16 number: TERMS bf16 terms that add up to it are multiplied with V one after another.
//
// Warps: 0..3 O, scaled and stored; 4..7 K~ and P; 8..15 the state; 16 copies (tensor maps, a ring of three chunks); 17 issue;
// 18 finds the chunks, and works their decays out ahead.  Every role walks one stream of chunks, whatever sequences and heads
// these belong to, so the next sequence's first chunks are under way while the last one's state is stored.
//
// An item is a (sequence, head), or a group of its chunks where there are too few of those for the SMs: then a first launch works
// out what each group adds to the state (its products V^T K~ alone), a small kernel chains the groups' states, and the second
// launch runs all groups side by side.
//
// A token's infinite or NaN v gets P = 0 in the columns of earlier tokens, and 0 x v is NaN in the matrix product: a row of V^T P^T
// that does not come out finite is taken again from P and V in shared memory, token by token (O of earlier tokens stays what it was).
#include "kda_linear.cuh"
#include "kda_tc.cuh"

#include <atomic>
#include <cstddef>

namespace kda {
namespace {

constexpr int THREADS = 608;
constexpr int TMEM_COLS = 512;
constexpr int TM_S1 = 0, TM_O1 = 128, TM_O2 = 192, TM_L = 256, TM_SB = 384;
constexpr int STAGES = 3;
constexpr int ENTRIES = 6;
constexpr int TILE_CB = 64 * 128;            // bytes of 64 tokens x 64 features
constexpr unsigned FULL = 0xffffffffu;
constexpr int MAX_RANKED = 128;              // sequences of a ragged batch that are taken longest first

// S <- e^a S + L.  weak: factor = e^a - 1, else e^a.
struct Decay {
    float factor;
    int weak;
};
__device__ __forceinline__ Decay decay_of(float a)
{
    const bool weak = a > -0.5f;
    return Decay{weak ? expm1f(a) : expf(a), weak};
}
__device__ __forceinline__ float decayed(const Decay &d, float s, float l)
{
    const float x = fmaf(d.factor, s, l);
    return d.weak ? s + x : x;
}

struct alignas(16) Entry {    // one chunk; the tables are read four floats at a time
    float2 logs[64];          // A_i in base 2, as two terms
    float ea[64];             // scale e^(A_i)
    float kf[64];             // e^(A_C - A_j), 0 past the end
    int64_t at_src, at_dst;   // index of the state before and after the chunk's item
    int src, dst;             // and where that is: 0 zeros / nowhere, 1 the call's, 2 a group's
    Decay decay;              // of the whole chunk
    int valid;                // 0: no more chunks
    int first, last;          // of its item
    int tok0, len, h;         // first token, tokens, head
};
static_assert(sizeof(Entry) % 16 == 0 && offsetof(Entry, ea) % 16 == 0 && offsetof(Entry, kf) % 16 == 0, "vector reads");

template <int DIM, int TERMS> struct Shape {
    static constexpr int CB = DIM / 64;
    static constexpr int TILE = CB * TILE_CB;
    static constexpr int STAGE = 3 * TILE;                    // V, Q, K
    static constexpr int KT = STAGES * STAGE;                 // K~: TERMS tiles
    static constexpr int P = KT + TERMS * TILE;               // two of [64 i][64 j]
    static constexpr int ZERO = P + 2 * TILE_CB;              // D = 64: lanes 64 to 127
    static constexpr int ENTRY = ZERO + (DIM == 64 ? TILE_CB : 0);
    static constexpr int BAR = ENTRY + ENTRIES * (int)sizeof(Entry);
    static constexpr int SMEM = 1024 + BAR + 320;
    static_assert(SMEM <= 232448, "a CTA's shared memory");
    static_assert(ENTRY % 16 == 0 && BAR % 8 == 0 && P % 1024 == 0 && KT % 1024 == 0 && ZERO % 1024 == 0, "alignment");
};

// ---------------------------------------------------------------- items
// Item x: (sequence, group, head) with heads innermost, so that neighbours share keys.
struct Item {
    int n, g, h;
    int64_t bos, len;
};

__device__ __forceinline__ int groups_of(const LinearPlan &plan, int64_t len, bool states_only)
{
    const int64_t chunks = (len + 63) / 64;
    const int64_t g = chunks == 0 ? 1 : (chunks + plan.group_chunks - 1) / plan.group_chunks;
    return (int)(states_only ? g - 1 : g);
}

// By a whole warp; false when there is none.  order: sequences longest first, or nullptr.
template <bool STATES_ONLY>
__device__ __forceinline__ bool find_item(const LinearArgs &p, const LinearPlan &plan, const short *order, int x, Item &w, bool &bad)
{
    const int lane = threadIdx.x & 31;
    w.h = x % p.H;
    int y = x / p.H;
    if (!p.tok.cu) {
        const int per = STATES_ONLY ? plan.groups - 1 : plan.groups;
        w.n = y / per;
        w.g = y % per;
        if (w.n >= p.tok.N)
            return false;
        linear_range(p, w.n, w.bos, w.len, bad);
        return w.g < groups_of(plan, w.len, STATES_ONLY);
    }
    int before = 0;
    for (int base = 0; base < p.tok.N; base += 32) {
        const int i = base + lane;
        int64_t bos = 0, len = 0;
        int n = i, count = 0;
        if (i < p.tok.N) {
            n = order ? order[i] : i;
            bad |= seq_range(p.tok.cu, n, p.tok.N, p.tok.T, bos, len);
            count = groups_of(plan, len, STATES_ONLY);
        }
        int sum = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(FULL, sum, o);
            if (lane >= o)
                sum += z;
        }
        const unsigned m = __ballot_sync(FULL, before + sum > y);
        if (m) {
            const int from = __ffs(m) - 1;
            w.n = __shfl_sync(FULL, n, from);
            w.bos = __shfl_sync(FULL, bos, from);
            w.len = __shfl_sync(FULL, len, from);
            w.g = y - (before + __shfl_sync(FULL, sum - count, from));
            return true;
        }
        before += __shfl_sync(FULL, sum, 31);
    }
    return false;
}

// Where a group's state lies in the workspace: distinct for all groups of all sequences, and below group_slots().
__device__ __forceinline__ int64_t slot_of(const LinearArgs &p, const LinearPlan &plan, int n, int64_t bos, int g)
{
    return p.tok.cu ? bos / (64 * (int64_t)plan.group_chunks) + n + g : (int64_t)n * plan.groups + g;
}

// A row of 64-bit halves of the state in registers: COLS columns from `at` on
template <int COLS> __device__ __forceinline__ void load_state(const void *p, kda_dtype_t type, int64_t at, float (&s)[COLS])
{
    if (type == KDA_DTYPE_BF16) {
        const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + at);
#pragma unroll
        for (int i = 0; i < COLS / 8; i++) {
            const uint4 y = x[i];
            const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; e++)
                s[8 * i + 2 * e] = bf16_lo(w[e]), s[8 * i + 2 * e + 1] = bf16_hi(w[e]);
        }
    } else {
        const float4 *x = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
#pragma unroll
        for (int i = 0; i < COLS / 4; i++) {
            const float4 y = x[i];
            s[4 * i] = y.x, s[4 * i + 1] = y.y, s[4 * i + 2] = y.z, s[4 * i + 3] = y.w;
        }
    }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&y);
}
template <int COLS> __device__ __forceinline__ void store_state(void *p, kda_dtype_t type, int64_t at, const float (&s)[COLS])
{
    if (type == KDA_DTYPE_BF16) {
        uint4 *x = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + at);
#pragma unroll
        for (int i = 0; i < COLS / 8; i++)
            x[i] = make_uint4(pack_bf16(s[8 * i], s[8 * i + 1]), pack_bf16(s[8 * i + 2], s[8 * i + 3]),
                              pack_bf16(s[8 * i + 4], s[8 * i + 5]), pack_bf16(s[8 * i + 6], s[8 * i + 7]));
    } else {
        float4 *x = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
#pragma unroll
        for (int i = 0; i < COLS / 4; i++)
            x[i] = make_float4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
    }
}
__device__ __forceinline__ void tmem_put16(uint32_t addr, const uint32_t *u)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 ::"r"(addr), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
                   "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
                 : "memory");
}
__device__ __forceinline__ float tmem_read1(uint32_t addr)
{
    float x;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n tcgen05.wait::ld.sync.aligned;" : "=&f"(x) : "r"(addr) : "memory");
    return x;
}

template <int DIM, int TERMS, bool STATES_ONLY>
__global__ void __launch_bounds__(THREADS, 1)
kda_linear_chunks_kernel(const __grid_constant__ LinearArgs p, const LinearPlan plan, const __grid_constant__ CUtensorMap qmap,
                         const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using S = Shape<DIM, TERMS>;
    constexpr int CB = S::CB;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *const smem = smem_raw + (base - smem_u32(smem_raw));
    Entry *const entries = reinterpret_cast<Entry *>(smem + S::ENTRY);
    const uint32_t bar = base + S::BAR;
    const uint32_t b_full = bar, b_empty = b_full + 8 * STAGES, b_ent = b_empty + 8 * STAGES, b_ent_free = b_ent + 8 * ENTRIES,
                   b_s = b_ent_free + 8 * ENTRIES, b_p = b_s + 16, b_o = b_p + 16, b_sb = b_o + 16, b_pe = b_sb + 16,
                   b_k = b_pe + 16, b_l = b_k + 8, b_l_free = b_l + 8, b_o_free = b_l_free + 8, b_block = b_o_free + 8, b_drain = b_block + 8;
    static_assert(8 * (2 * STAGES + 2 * ENTRIES + 16) <= 320, "barriers");
    __shared__ uint32_t tmem_slot;
    __shared__ uint4 block_answer;
    __shared__ short order[MAX_RANKED];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < STAGES; i++) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, STATES_ONLY ? 1 : 5);   // products, and the epilogue's warps
        }
        for (int i = 0; i < ENTRIES; i++) {
            mbar_init(b_ent + 8 * i, 1);
            mbar_init(b_ent_free + 8 * i, 18);                 // every warp but the one that writes
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(b_s + 8 * i, 1);
            mbar_init(b_p + 8 * i, 2);
            mbar_init(b_o + 8 * i, 1);
            mbar_init(b_sb + 8 * i, 8);
            mbar_init(b_pe + 8 * i, 4);
        }
        mbar_init(b_k, 4);
        mbar_init(b_l, 1);
        mbar_init(b_l_free, 8);
        mbar_init(b_o_free, 4);
        mbar_init(b_block, 1);
        mbar_init(b_drain, 1);
        mbar_fence_init();
    }
    if (warp == 17) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (DIM == 64) {
        for (int i = tid; i < TILE_CB / 16; i += THREADS)
            reinterpret_cast<uint4 *>(smem + S::ZERO)[i] = make_uint4(0, 0, 0, 0);
        fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    stream_order();
    bool timeout = false, bad = false;
    // Waits of a whole warp, which stays converged; once one has given up, the later ones do at once.
    auto wait = [&](uint32_t b, uint32_t parity) -> bool {
        if (__any_sync(FULL, !mbar_wait(b, parity & 1, timeout ? 1 : plan.wait_polls)))
            timeout = true;
        return !timeout;
    };
    // Chunk c of the stream: there when the wait is through and it is valid.
    auto next = [&](uint32_t c) -> bool {
        return wait(b_ent + 8 * (c % ENTRIES), c / ENTRIES) && entries[c % ENTRIES].valid;
    };
    auto arrive = [&](uint32_t b) {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(b);
    };

    if (warp < 4) {
        // ------------------------------------------------------------ O
        const uint32_t quad = (uint32_t)warp << 21;
        const int v = warp * 32 + lane;
        for (uint32_t c = 0; next(c); c++) {
            const Entry &e = entries[c % ENTRIES];
            if (!STATES_ONLY) {
                if (!wait(b_o + 8 * (c & 1), c >> 1))
                    break;
                tc_fence_after();
                const int len = e.len;
                __nv_bfloat16 *out = p.out + ((int64_t)e.tok0 * p.H + e.h) * DIM;
                const int64_t row = (int64_t)p.H * DIM;
                if (warp * 32 < DIM) {
                    uint32_t w[32];                            // pairs of tokens
                    f2 z = 0;                                  // stays 0 while the row of V^T P^T is finite
#pragma unroll
                    for (int half = 0; half < 2; half++) {
                        float x[32], y[32];
                        tmem_read32(tmem + TM_O1 + quad + 32 * half, x);
                        tmem_read32(tmem + TM_O2 + quad + 32 * half, y);
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(&e.ea[32 * half + i]);
                            z = f2_fma(f2_pack(x[i], x[i + 1]), 0, z);
                            z = f2_fma(f2_pack(x[i + 2], x[i + 3]), 0, z);
                            w[16 * half + i / 2] = pack_bf16(fmaf(f.x, y[i], p.scale * x[i]), fmaf(f.y, y[i + 1], p.scale * x[i + 1]));
                            w[16 * half + i / 2 + 1] = pack_bf16(fmaf(f.z, y[i + 2], p.scale * x[i + 2]), fmaf(f.w, y[i + 3], p.scale * x[i + 3]));
                        }
                    }
                    const bool odd = !(f2_lo(z) + f2_hi(z) == 0.0f);
                    if (!__any_sync(FULL, odd)) {
                        tc_fence_before();
                        arrive(b_o_free);
                        // neighbouring lanes swap halves of a pair of tokens: each stores one token's pair of features
                        __nv_bfloat16 *to = out + (v & ~1) + (lane & 1) * row;
                        const uint32_t pick = lane & 1 ? 0x3276 : 0x5410;
#pragma unroll
                        for (int i = 0; i < 32; i++) {
                            const uint32_t y = __shfl_xor_sync(FULL, w[i], 1);
                            if (2 * i + (lane & 1) < len)
                                *reinterpret_cast<uint32_t *>(to + 2 * i * row) = __byte_perm(w[i], y, pick);
                        }
                    } else {
                        // (both are through; waited for here so that this thread sees what they brought)
                        if (!wait(b_full + 8 * (c % STAGES), c / STAGES) || !wait(b_p + 8 * (c & 1), c >> 1))
                            break;
                        const unsigned char *pt = smem + S::P + (c & 1) * TILE_CB;
                        const unsigned char *vt = smem + (c % STAGES) * S::STAGE + (v / 64) * TILE_CB;
                        for (int i = 0; i < len; i++) {
                            float x = tmem_read1(tmem + TM_O1 + quad + i);
                            const float y = tmem_read1(tmem + TM_O2 + quad + i);
                            if (odd) {
                                x = 0.0f;
                                for (int j = 0; j <= i; j++) {
                                    const __nv_bfloat16 a = *reinterpret_cast<const __nv_bfloat16 *>(
                                        pt + i * 128 + (((j / 8) ^ (i & 7)) << 4) + (j % 8) * 2);
                                    const __nv_bfloat16 b = *reinterpret_cast<const __nv_bfloat16 *>(
                                        vt + j * 128 + (((v % 64 / 8) ^ (j & 7)) << 4) + (v % 8) * 2);
                                    x = fmaf(__bfloat162float(a), __bfloat162float(b), x);
                                }
                            }
                            out[i * row + v] = __float2bfloat16_rn(fmaf(e.ea[i], y, p.scale * x));
                        }
                        tc_fence_before();
                        arrive(b_o_free);
                    }
                } else {
                    arrive(b_o_free);
                }
                arrive(b_pe + 8 * (c & 1));
                if (lane == 0)
                    mbar_arrive(b_empty + 8 * (c % STAGES));
            }
            arrive(b_ent_free + 8 * (c % ENTRIES));
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------ K~, P
        const int wp = warp - 4, t = tid - 128;
        for (uint32_t c = 0; next(c); c++) {
            const Entry &e = entries[c % ENTRIES];
            const int st = c % STAGES, len = e.len;
            if (!wait(b_full + 8 * st, c / STAGES) || (c > 0 && !wait(b_l, c - 1)))
                break;
            const unsigned char *kt = smem + st * S::STAGE + 2 * S::TILE;
            constexpr int VECS = 64 * DIM / 8 / 128;           // 16-byte vectors of a thread
#pragma unroll
            for (int m = 0; m < VECS; m++) {
                const int i = t + 128 * m, j = i / (DIM / 8), ch = i % (DIM / 8);
                const int at = (ch / 8) * TILE_CB + j * 128 + (((ch % 8) ^ (j & 7)) << 4);
                const uint4 x = *reinterpret_cast<const uint4 *>(kt + at);
                const float f = e.kf[j];
                const bool live = j < len;
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                uint32_t y[TERMS][4];
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    float a = live ? bf16_lo(w[q]) * f : 0.0f, b = live ? bf16_hi(w[q]) * f : 0.0f;
#pragma unroll
                    for (int r = 0; r < TERMS; r++) {
                        y[r][q] = pack_bf16(a, b);
                        a -= bf16_lo(y[r][q]), b -= bf16_hi(y[r][q]);
                    }
                }
#pragma unroll
                for (int r = 0; r < TERMS; r++)
                    *reinterpret_cast<uint4 *>(smem + S::KT + r * S::TILE + at) = make_uint4(y[r][0], y[r][1], y[r][2], y[r][3]);
            }
            if (len < 64) {                                    // what lies behind the sequence is cleared from V
                unsigned char *vt = smem + st * S::STAGE;
                for (int i = t; i < (64 - len) * 8 * CB; i += 128)
                    *reinterpret_cast<uint4 *>(vt + i / ((64 - len) * 8) * TILE_CB + len * 128 + i % ((64 - len) * 8) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            arrive(b_k);
            if (!STATES_ONLY && (wp >> 1) == (int)(c & 1)) {
                if (!wait(b_s + 8 * (c & 1), c >> 1) || (c >= 2 && !wait(b_pe + 8 * (c & 1), (c >> 1) - 1)))
                    break;
                tc_fence_after();
                const int i = (wp & 1) * 32 + lane;            // token of the row
                unsigned char *pt = smem + S::P + (c & 1) * TILE_CB + i * 128;
                const float2 mine = e.logs[i];
#pragma unroll
                for (int half = 0; half < 2; half++) {
                    uint32_t y[16];
                    if (half > (wp & 1)) {                     // later tokens only
#pragma unroll
                        for (int q = 0; q < 16; q++)
                            y[q] = 0;
                    } else {
                        float s[32];
                        tmem_read32(tmem + TM_S1 + 64 * (c & 1) + ((uint32_t)wp << 21) + 32 * half, s);
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const float4 l = *reinterpret_cast<const float4 *>(&e.logs[32 * half + j]);
                            const float a = s[j] * ex2_approx((mine.x - l.x) + (mine.y - l.y));
                            const float b = s[j + 1] * ex2_approx((mine.x - l.z) + (mine.y - l.w));
                            // bf16, V's type, as the product takes it
                            y[j / 2] = pack_bf16(32 * half + j <= i ? a : 0.0f, 32 * half + j + 1 <= i ? b : 0.0f);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        *reinterpret_cast<uint4 *>(pt + (((4 * half + q) ^ (i & 7)) << 4)) =
                            make_uint4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
                }
                tc_fence_before();
                fence_async_smem();
                arrive(b_p + 8 * (c & 1));
            }
            arrive(b_ent_free + 8 * (c % ENTRIES));
        }
    } else if (warp < 16) {
        // ------------------------------------------------------------ the state
        constexpr int COLS = DIM / 2;
        const int half = (warp - 8) / 4, v = (warp & 3) * 32 + lane;
        const uint32_t quad = (uint32_t)(warp & 3) << 21;
        const bool mine = (warp & 3) * 32 < DIM;
        const uint32_t tm_l = tmem + TM_L + quad + half * COLS, tm_sb = tmem + TM_SB + quad + half * (COLS / 2);
        float s[COLS];
#pragma unroll
        for (int i = 0; i < COLS; i++)
            s[i] = 0.0f;
        // S before chunk c, as the operand of its product
        auto put = [&](uint32_t c) -> bool {
            if (STATES_ONLY)
                return true;
            if (c >= 2 && !wait(b_o + 8 * (c & 1), (c >> 1) - 1))
                return false;
            if (mine) {
                tc_fence_after();
                uint32_t u[COLS / 2];
#pragma unroll
                for (int i = 0; i < COLS; i += 2)
                    u[i / 2] = pack_bf16(s[i], s[i + 1]);
                if constexpr (COLS == 64)
                    tmem_put32(tm_sb + 64 * (c & 1), u);
                else
                    tmem_put16(tm_sb + 64 * (c & 1), u);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
            }
            arrive(b_sb + 8 * (c & 1));
            return true;
        };
        for (uint32_t c = 0; next(c); c++) {
            const Entry &e = entries[c % ENTRIES];
            if (e.first) {
                if (mine && e.src)
                    load_state<COLS>(e.src == 1 ? p.init : plan.states, e.src == 1 ? plan.state_type : KDA_DTYPE_FP32,
                                     (e.at_src * DIM + v) * DIM + half * COLS, s);
                else
#pragma unroll
                    for (int i = 0; i < COLS; i++)
                        s[i] = 0.0f;
                if (!put(c))
                    break;
            }
            if (!wait(b_l, c))
                break;
            if (mine) {
                tc_fence_after();
                const Decay d = e.decay;
#pragma unroll
                for (int i = 0; i < COLS; i += 32) {
                    float l[32];
                    tmem_read32(tm_l + i, l);
#pragma unroll
                    for (int j = 0; j < 32; j++)
                        l[j] = fmaf(d.factor, s[i + j], l[j]);
                    if (d.weak) {
#pragma unroll
                        for (int j = 0; j < 32; j++)
                            s[i + j] += l[j];
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; j++)
                            s[i + j] = l[j];
                    }
                }
                tc_fence_before();
            }
            arrive(b_l_free);
            if (!e.last) {
                if (!put(c + 1))
                    break;
            } else if (mine && e.dst) {
                store_state<COLS>(e.dst == 1 ? p.fin : plan.states, e.dst == 1 ? plan.state_type : KDA_DTYPE_FP32,
                                  (e.at_dst * DIM + v) * DIM + half * COLS, s);
            }
            arrive(b_ent_free + 8 * (c % ENTRIES));
        }
    } else if (warp == 16) {
        // ------------------------------------------------------------ copies
        uint32_t c = 0;
        for (; next(c); c++) {
            const Entry &e = entries[c % ENTRIES];
            const int st = c % STAGES, h = e.h, tok = e.tok0;
            if (c >= STAGES && !wait(b_empty + 8 * st, c / STAGES - 1))
                break;
            if (lane == 0) {
                const uint32_t to = base + st * S::STAGE, b = b_full + 8 * st;
                mbar_expect_tx(b, (STATES_ONLY ? 2 : 3) * S::TILE);
#pragma unroll
                for (int cb = 0; cb < CB; cb++) {
                    tma_load_3d(to + 2 * S::TILE + cb * TILE_CB, &kmap, 64 * cb, h / p.group, tok, b);
                    tma_load_3d(to + cb * TILE_CB, &vmap, 64 * cb, h / p.group, tok, b);
                    if (!STATES_ONLY)
                        tma_load_3d(to + S::TILE + cb * TILE_CB, &qmap, 64 * cb, h, tok, b);
                }
            }
            arrive(b_ent_free + 8 * (c % ENTRIES));
        }
        // no copy is in flight when the CTA leaves, also where the work was given up
        for (uint32_t i = c < STAGES ? 0 : c - STAGES; i < c; i++)
            timeout |= !mbar_wait(b_full + 8 * (i % STAGES), (i / STAGES) & 1);
    } else if (warp == 17) {
        // ------------------------------------------------------------ tensor-core issue
        // The whole warp waits, one elected lane issues from uniform registers.
        const uint32_t id_s = idesc_bf16(128, 64, false), id_o1 = idesc_bf16(128, 64, false) | A_MN,
                       id_l = idesc_bf16(128, DIM, true) | A_MN, id_o2 = idesc_bf16(128, 64, false);
        const uint32_t tm = __shfl_sync(FULL, tmem, 0), lead = elect_one();
        auto scores = [&](uint32_t c) {                        // Q K^T of chunk c
            const uint32_t at = base + (c % STAGES) * S::STAGE;
            const uint32_t a = desc_lo(at + S::TILE - (c & 1) * TILE_CB, 16), b = desc_lo(at + 2 * S::TILE, 16), d = tm + TM_S1 + 64 * (c & 1);
            if (lead && !timeout) {
#pragma unroll
                for (int k = 0; k < DIM / 16; k++) {
                    const uint32_t step = ((k / 4) * TILE_CB + (k % 4) * 32) >> 4;
                    if (k == 0)
                        mma_ss<false>(d, a, b, id_s, 0);
                    else
                        mma_ss<true>(d, a + step, b + step, id_s, 1);
                }
                umma_commit(b_s + 8 * (c & 1));
            }
            __syncwarp();
        };
        bool more = next(0);
        if (more && !STATES_ONLY && wait(b_full, 0)) {
            tc_fence_after();
            scores(0);
        }
        for (uint32_t c = 0; more; c++) {
            const int st = c % STAGES;
            const uint32_t at = base + st * S::STAGE;
            // V as M rows: blocks of 64 features, for D = 64 the second one zeros
            const uint32_t v = desc_lo(at, DIM == 128 ? TILE_CB : S::ZERO - st * S::STAGE);
            if (!wait(b_k, c) || (c > 0 && !wait(b_l_free, c - 1)))
                break;
            tc_fence_after();
            if (lead && !timeout) {
#pragma unroll
                for (int r = TERMS - 1; r >= 0; r--) {         // small terms first
                    const uint32_t b = desc_lo(base + S::KT + r * S::TILE, TILE_CB);
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        if (r == TERMS - 1 && k == 0)
                            mma_ss<false>(tm + TM_L, v, b, id_l, 0);
                        else
                            mma_ss<true>(tm + TM_L, v + k * (2048 >> 4), b + k * (2048 >> 4), id_l, 1);
                    }
                }
                umma_commit(b_l);
                if (STATES_ONLY)
                    umma_commit(b_empty + 8 * st);
            }
            __syncwarp();
            more = next(c + 1);
            if (!STATES_ONLY) {
                if (!wait(b_sb + 8 * (c & 1), c >> 1) || (c > 0 && !wait(b_o_free, c - 1)))
                    break;
                tc_fence_after();
                const uint32_t q = desc_lo(at + S::TILE, 16), sb = tm + TM_SB + 64 * (c & 1);
                if (lead && !timeout) {
#pragma unroll
                    for (int k = 0; k < DIM / 16; k++) {
                        const uint32_t step = ((k / 4) * TILE_CB + (k % 4) * 32) >> 4;
                        if (k == 0)
                            mma_ts<false>(tm + TM_O2, sb, q, id_o2, 0);
                        else
                            mma_ts<true>(tm + TM_O2, sb + 8 * k, q + step, id_o2, 1);
                    }
                }
                __syncwarp();
                if (more) {
                    if (!wait(b_full + 8 * ((c + 1) % STAGES), (c + 1) / STAGES))
                        break;
                    tc_fence_after();
                    scores(c + 1);
                }
                if (!wait(b_p + 8 * (c & 1), c >> 1))
                    break;
                tc_fence_after();
                const uint32_t pd = desc_lo(base + S::P + (c & 1) * TILE_CB, 16);
                if (lead && !timeout) {
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        if (k == 0)
                            mma_ss<false>(tm + TM_O1, v, pd, id_o1, 0);
                        else
                            mma_ss<true>(tm + TM_O1, v + k * (2048 >> 4), pd + k * (32 >> 4), id_o1, 1);
                    }
                    umma_commit(b_o + 8 * (c & 1));
                    umma_commit(b_empty + 8 * st);
                }
                __syncwarp();
            }
            arrive(b_ent_free + 8 * (c % ENTRIES));
        }
        if (lead) {
            // everything issued has to be through before tensor memory is freed
            umma_commit(b_drain);
            timeout |= !mbar_wait(b_drain, 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ chunks and their decays
        const short *ranked = nullptr;
        if (p.tok.cu && p.tok.N <= MAX_RANKED) {
            for (int i = lane; i < p.tok.N; i += 32) {
                int64_t bos, len, x, y;
                seq_range(p.tok.cu, i, p.tok.N, p.tok.T, bos, len);
                int rank = 0;
                for (int j = 0; j < p.tok.N; j++) {
                    seq_range(p.tok.cu, j, p.tok.N, p.tok.T, x, y);
                    rank += y > len || (y == len && j < i);
                }
                order[rank] = (short)i;
            }
            __syncwarp();
            ranked = order;
        }
        const uint32_t answer = smem_u32(&block_answer);
        uint32_t asked = 0, answers = 0, c = 0;
        // The next block of the grid that has not started, taken over when the CTA's own is worked out: CTAs with less to do take more.
        auto next_block = [&]() -> int {
            if (lane == 0) {
                fence_async_smem();                            // the last answer has been read
                mbar_expect_tx(b_block, 16);
                ask_for_block(answer, b_block);
            }
            asked++;
            __syncwarp();
            if (!wait(b_block, answers))
                return -1;
            answers++;
            const int y = take_answer(answer);
            __syncwarp();
            return y;
        };
        auto slot_free = [&]() -> bool { return c < ENTRIES || wait(b_ent_free + 8 * (c % ENTRIES), c / ENTRIES - 1); };
        for (int x = blockIdx.x; x >= 0 && !timeout; x = next_block()) {
            Item w;
            if (!find_item<STATES_ONLY>(p, plan, ranked, x, w, bad))
                continue;
            const int64_t chunks = (w.len + 63) / 64, c0 = (int64_t)w.g * plan.group_chunks;
            const int64_t c1 = c0 + plan.group_chunks < chunks ? c0 + plan.group_chunks : chunks;
            const float fixed = p.log_decay ? p.log_decay[w.h] : 0.0f;
            auto gate = [&](int64_t i) -> float { return i < w.len ? log_decay_of(p, w.bos + i, w.h, fixed, bad) : 0.0f; };
            double total = 0.0;
            float g0 = gate(c0 * 64 + 2 * lane), g1 = gate(c0 * 64 + 2 * lane + 1);
            for (int64_t i = c0; i < c1 || i == c0; i++) {     // (an empty sequence has one chunk of no tokens)
                const double a0 = g0, a1 = g1;
                if (i + 1 < c1)
                    g0 = gate((i + 1) * 64 + 2 * lane), g1 = gate((i + 1) * 64 + 2 * lane + 1);
                double sum = a0 + a1;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double z = __shfl_up_sync(FULL, sum, o);
                    if (lane >= o)
                        sum += z;
                }
                const double all = __shfl_sync(FULL, sum, 31);
                total += all;
                if (!slot_free())
                    break;
                Entry &e = entries[c % ENTRIES];
                const int len = (int)(w.len - i * 64 < 64 ? w.len - i * 64 : 64);
                constexpr double L2E = 1.4426950408889634;
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    const int j = 2 * lane + q;
                    const double a = q ? sum : sum - a1, b = a * L2E;
                    const float hi = (float)b;
                    e.logs[j] = make_float2(hi, (float)(b - hi));
                    e.ea[j] = p.scale * exp2f(hi);
                    e.kf[j] = j < len ? expf((float)(all - a)) : 0.0f;
                }
                if (lane == 0) {
                    e.valid = 1;
                    e.first = i == c0, e.last = i + 1 >= c1;
                    e.tok0 = (int)(w.bos + i * 64), e.len = len, e.h = w.h;
                    e.decay = decay_of((float)all);
                    e.src = w.g > 0 && !STATES_ONLY ? 2 : (!STATES_ONLY && p.init ? 1 : 0);
                    e.at_src = e.src == 2 ? slot_of(p, plan, w.n, w.bos, w.g - 1) * p.H + w.h : (int64_t)w.n * p.H + w.h;
                    e.dst = STATES_ONLY ? 2 : (c1 == chunks && p.fin ? 1 : 0);
                    e.at_dst = STATES_ONLY ? slot_of(p, plan, w.n, w.bos, w.g) * p.H + w.h : (int64_t)w.n * p.H + w.h;
                    const Decay all_of = decay_of((float)total);
                    if (STATES_ONLY && i + 1 >= c1)
                        plan.decays[e.at_dst] = make_float2(all_of.factor, all_of.weak ? 1.0f : 0.0f);
                }
                arrive(b_ent + 8 * (c % ENTRIES));
                c++;
            }
        }
        if (slot_free()) {
            if (lane == 0)
                entries[c % ENTRIES].valid = 0;
            arrive(b_ent + 8 * (c % ENTRIES));
        }
        if (asked > answers)
            timeout |= !mbar_wait(b_block, answers & 1);
    }
    report(p.err, bad, DEVERR_CU_SEQLENS);
    report(p.err, timeout, DEVERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 17)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS));
}

// ---------------------------------------------------------------- groups' start states
// S_0 the call's; what group g adds lies in its slot and is replaced by S_(g+1) = e^(A_g) S_g + it, the state that group g + 1 starts from.
// Four elements a thread, the groups in turn.
__global__ void __launch_bounds__(256) kda_linear_join_kernel(const LinearArgs p, const LinearPlan plan)
{
    const int per = p.dim * p.dim / 4;                         // a multiple of the block
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x, pair = x / per;
    const int n = (int)(pair / p.H), h = (int)(pair % p.H);
    const int64_t at = x % per * 4;
    stream_order();
    bool bad = false;
    int64_t bos, len;
    linear_range(p, n, bos, len, bad);                         // (reported by the kernel before)
    const int groups = groups_of(plan, len, true);
    if (groups <= 0)
        return;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t size = (int64_t)p.dim * p.dim;
    if (p.init) {
        if (plan.state_type == KDA_DTYPE_BF16) {
            const uint2 y = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p.init) + pair * size + at);
            s[0] = bf16_lo(y.x), s[1] = bf16_hi(y.x), s[2] = bf16_lo(y.y), s[3] = bf16_hi(y.y);
        } else {
            const float4 y = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.init) + pair * size + at);
            s[0] = y.x, s[1] = y.y, s[2] = y.z, s[3] = y.w;
        }
    }
    const int64_t first = slot_of(p, plan, n, bos, 0);
#pragma unroll 4
    for (int g = 0; g < groups; g++) {
        const int64_t slot = (first + g) * p.H + h;
        const float2 f = plan.decays[slot];
        const Decay d{f.x, f.y != 0.0f};
        float4 *y = reinterpret_cast<float4 *>(plan.states + slot * size + at);
        const float4 l = *y;
        s[0] = decayed(d, s[0], l.x), s[1] = decayed(d, s[1], l.y), s[2] = decayed(d, s[2], l.z), s[3] = decayed(d, s[3], l.w);
        *y = make_float4(s[0], s[1], s[2], s[3]);
    }
}

// ---------------------------------------------------------------- host
// [tokens][heads][dim] with tokens `stride` elements apart; a box is 64 columns of 64 tokens of a head.
cudaError_t token_map(CUtensorMap *map, const __nv_bfloat16 *ptr, int dim, int heads, int64_t tokens, int64_t stride)
{
    EncodeTiled fn;
    const cudaError_t e = encode_fn(&fn);
    if (e != cudaSuccess)
        return e;
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, 64}, step[3] = {1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16 *>(ptr), dims, strides, box, step,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int DIM, int TERMS, bool STATES_ONLY>
cudaError_t launch(const LinearArgs &p, const LinearPlan &plan, int64_t items, const CUtensorMap *maps, cudaStream_t st)
{
    static std::atomic<uint64_t> ready;      // devices whose kernel attribute is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(ready.load() >> dev & 1)) {
        e = cudaFuncSetAttribute(kda_linear_chunks_kernel<DIM, TERMS, STATES_ONLY>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Shape<DIM, TERMS>::SMEM);
        if (e == cudaSuccess)
            ready.fetch_or(1ull << dev);
    }
    if (e != cudaSuccess)
        return e;
    return launch_in_row(kda_linear_chunks_kernel<DIM, TERMS, STATES_ONLY>, (unsigned)items, THREADS, Shape<DIM, TERMS>::SMEM, 1, st, p,
                         plan, maps[0], maps[1], maps[2]);
}

template <int DIM, int TERMS> cudaError_t launch_all(const LinearArgs &p, const LinearPlan &plan, cudaStream_t st)
{
    CUtensorMap maps[3];
    const int64_t tokens = p.tok.cu ? p.tok.T : p.tok.N * p.tok.T;
    cudaError_t e = token_map(&maps[0], p.q, DIM, p.H, tokens, p.q_stride);
    if (e == cudaSuccess)
        e = token_map(&maps[1], p.k, DIM, p.H / p.group, tokens, p.k_stride);
    if (e == cudaSuccess)
        e = token_map(&maps[2], p.v, DIM, p.H / p.group, tokens, p.v_stride);
    if (e == cudaSuccess && plan.groups > 1) {
        e = launch<DIM, TERMS, true>(p, plan, plan.items_before, maps, st);
        if (e == cudaSuccess)
            e = launch_in_row(kda_linear_join_kernel, (unsigned)((int64_t)p.tok.N * p.H * (DIM * DIM / 4 / 256)), 256, 0, 1, st, p, plan);
    }
    return e != cudaSuccess ? e : launch<DIM, TERMS, false>(p, plan, plan.items, maps, st);
}

}  // namespace

cudaError_t launch_linear_chunks(const LinearArgs &p, const LinearPlan &plan, cudaStream_t st)
{
    const bool exact = plan.state_type == KDA_DTYPE_FP32 && p.fin;
    if (p.dim == 128)
        return exact ? launch_all<128, 2>(p, plan, st) : launch_all<128, 1>(p, plan, st);
    return exact ? launch_all<64, 2>(p, plan, st) : launch_all<64, 1>(p, plan, st);
}

}  // namespace kda
