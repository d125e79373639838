// Linear attention in chunks of 64 tokens on the tensor cores.
//
// Within a chunk, with A_i the sum of the logarithms up to token i and S the state before the chunk (rows v, columns k):
//   P = (Q K^T) . e^(A_i - A_j)  (j <= i),   O^T = V^T P^T + e^(A_i) S Q^T,   S <- e^(A_C) S + (e^(A_C - A_j) V)^T K.
// All decays are at most 1 by construction: they are exponentials of differences that are never positive, taken from sums of two
// terms, so a strong decay beside a weak one costs no precision and none is divided by.
//
// The features lie on tensor memory's lanes: O^T and S have a row per v, so that S and V~ = e^(A_C - A_j) V are operands straight from tensor
// memory (bf16, written by the threads that hold S, and by those that turn V) and leave shared memory's bandwidth, the first bound of
// such a kernel, to the others.  Four products a chunk: Q K^T [64 x 64] (on 16 of each warp's 32 lanes),
// V~^T K [D x D], S Q^T and V^T P^T [D x 64].  D = 64 fills the lanes up with a block of zeros.
//
// The state stays in fp32 registers (eight warps): each chunk's V~^T K comes out of tensor memory and is added there, so the tensor cores'
// own accumulation spans one chunk and what a long sequence adds up is rounded to nearest.  A decay is two numbers, hi S + (lo S + L): a factor
// next to 1 that is off by half a step in every chunk would drift by 2^-25 a chunk.  A state that is forgotten (both 0) leaves nothing behind as
// rounding, and an infinite one stays infinite.
// V~ is not a bf16 number: two bf16 terms that add up to it (to 2^-17) are multiplied with K one after the other.  With
// one, outputs after bf16 states were 2.6e-3 off (norm) and not 2.3e-3, 1.7e-3 of it their own rounding, and a prompt took 3% less:
// what the tensor cores do is not what bounds a chunk.  fp32 states come out 4.1e-6 off (3.1e-6 after a first chunk of 16 tokens; token by token 1e-7).  The other roundings to bf16 are P's, and that of
// the state that a chunk's queries read (outputs are bf16, rounded to 2^-9 of their own).
//
// Warps: 0 copies (tensor maps, a ring of chunks); 1 and 3 issue; 2 finds the chunks, and works their decays out ahead; 4..7 P;
// 8..11 V~; 12..19 the state; 20..23 O, scaled and stored.  Every role walks one stream of chunks, whatever sequences and heads
// these belong to, so the next sequence's first chunks are under way while the last one's state is stored.
//
// Measured (one GPU): 8192 tokens of 96 heads with fp32 states 163 us, 5.0 TB/s (0.74 of the copy rate), of 96 heads of 64 147 us; 12 ragged
// prompts of as many tokens in all 159 to 163 us; 8192 tokens of 64 heads over 8 with gates, two groups a head, 150 us; 32768 tokens of 8 heads, 19
// groups, 91 us; 509 tokens of 14 heads over 2 of 64 14.4 us.  A chunk takes some 2,200 cycles in a (sequence, head)'s chain even where
// nothing else runs, and that is what bounds all but the batches that fill the SMs: O's products into its one place, their issue and the
// barriers, and O on its way out.  Beside it shared memory alone is busy for 1,600 (at 128 bytes a cycle: 48 KB come in, 16 KB are read to be
// turned, 8 KB written for P, the products read 32 + 32 + 16 + 24 KB, O goes out through 32 KB), and the tensor pipe for 70% of
// the time on SMs that have work.
//
// An item is a (sequence, head), or a group of its chunks where there are too few of those for the SMs: then a first launch works
// out what each group adds to the state (its products V~^T K alone), a small kernel chains the groups' states, and the second
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

constexpr int THREADS = 768;                 // six warpgroups
constexpr int TMEM_COLS = 512;
constexpr int TM_S1 = 0, TM_SB = 64, TM_O1 = 128, TM_O2 = 192, TM_L = 256, TM_V = 384;   // columns; two V~, a term 32 each
constexpr int ENTRIES = 6;                   // chunks known ahead (8: 2 us more for ragged prompts, whose last items are taken too early)
constexpr int EARLY = 4;                     // chunks ahead that tiles are brought into L2
constexpr int TILE_CB = 64 * 128;            // bytes of 64 tokens x 64 features
constexpr unsigned FULL = 0xffffffffu;
constexpr int TERMS = 2;                     // bf16 terms of V~
constexpr int MAX_RANKED = 128;              // sequences of a ragged batch that are taken longest first

// A sum of logarithms in base 2 as two terms, good to some 2^-45 of the largest partial sum, without 64-bit arithmetic (whose unit here
// takes longer for a chunk's sums than all else does for the chunk).
struct Sum {
    float hi, lo;
};
__device__ __forceinline__ Sum add(const Sum &a, const Sum &b)
{
    const float s = a.hi + b.hi, x = s - a.hi;
    const float lo = ((a.hi - (s - x)) + (b.hi - x)) + (a.lo + b.lo), hi = s + lo;
    return Sum{hi, lo - (hi - s)};
}
__device__ __forceinline__ float minus(const Sum &a, const Sum &b) { return (a.hi - b.hi) + (a.lo - b.lo); }
constexpr float LOG2E_LO = (float)(1.4426950408889634074 - (double)LOG2E);
__device__ __forceinline__ Sum in_base_2(float a)
{
    const float hi = a * LOG2E;
    return Sum{hi, fmaf(a, LOG2E, -hi) + a * LOG2E_LO};
}

// S <- e^a S + L as hi S + (lo S + L): hi lies just below e^a, and lo is what it leaves off (of a weak decay out of expm1, good to 2^-47).  Both
// products have S's sign, so that an infinite S stays what it is unless e^a is 0.  ZEROS: the state began with zeros, and a strong decay
// is one product (lo = 0): 32768 tokens of 8 heads 91.3 us, without it 92.7; where states are read, a branch between the two forms takes
// longer than the second product (8192 tokens of 96 heads 163.1 us, with it 166.3).
struct Decay {
    float hi, lo;
};
template <bool ZEROS> __device__ __forceinline__ Decay decay_of(const Sum &a)
{
    constexpr float LN2 = 0.6931471805599453f, LN2_LO = (float)(0.69314718055994530942 - (double)LN2);
    const float x = fmaf(a.hi, LN2, fmaf(a.hi, LN2_LO, a.lo * LN2));
    auto below = [](float y) { return __uint_as_float(__float_as_uint(y) - (y > 0.0f)); };
    if (!(x > -0.5f)) {
        const float e = expf(x), hi = ZEROS ? e : below(e);
        return Decay{hi, ZEROS ? 0.0f : e - hi};
    }
    const float less = expm1f(x), hi = below(1.0f + less);
    return Decay{hi, (1.0f - hi) + less};
}
__device__ __forceinline__ float decayed(const Decay &d, float s, float l)
{
    return fmaf(d.hi, s, fmaf(d.lo, s, l));
}

struct alignas(16) Entry {    // one chunk; the tables are read four floats at a time
    float hi[64], lo[64];     // A_i in base 2, as two terms
    float ea[64];             // scale e^(A_i)
    uint32_t f[TERMS][32];    // e^(A_C - A_j) as two bf16 terms, tokens in pairs
    int64_t at_src, at_dst;   // index of the state before and after the chunk's item
    int src, dst;             // and where that is: 0 zeros / nowhere, 1 the call's, 2 a group's
    Decay decay;              // of the whole chunk
    int valid;                // 0: no more chunks
    int first, last;          // of its item
    int tok0, len, h;         // first token, tokens, head
};
static_assert(sizeof(Entry) % 16 == 0 && offsetof(Entry, lo) % 16 == 0 && offsetof(Entry, ea) % 16 == 0, "vector reads");

template <int DIM, bool STATES_ONLY> struct Shape {
    static constexpr int CB = DIM / 64;
    static constexpr int TILE = CB * TILE_CB;
    static constexpr int TILES = STATES_ONLY ? 2 : 3;         // of a chunk: V, K, Q
    static constexpr int STAGE = TILES * TILE;
    static constexpr int STAGES = DIM == 64 ? (STATES_ONLY ? 8 : 6) : (STATES_ONLY ? 6 : 3);
    static constexpr int P = STAGES * STAGE;                  // two of [64 i][64 j]
    static constexpr int OUT = P + (STATES_ONLY ? 0 : 2 * TILE_CB);    // O on its way out
    static constexpr int ZERO = OUT + (STATES_ONLY ? 0 : TILE);        // D = 64: lanes 64 to 127
    static constexpr int ENTRY = ZERO + (DIM == 64 ? TILE_CB : 0);
    static constexpr int BAR = ENTRY + ENTRIES * (int)sizeof(Entry);
    static constexpr int SMEM = 1024 + BAR + 512;
    static_assert(SMEM <= 232448, "a CTA's shared memory");
    static_assert(ENTRY % 16 == 0 && BAR % 8 == 0 && P % 1024 == 0 && ZERO % 1024 == 0, "alignment");
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
    if (plan.groups == 1) {                                    // every sequence is one item
        if (y >= p.tok.N)
            return false;
        w.n = order ? order[y] : y;
        w.g = 0;
        bad |= seq_range(p.tok.cu, w.n, p.tok.N, p.tok.T, w.bos, w.len);
        return true;
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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&y);
}
// COLS columns of a row of the state, in registers as pairs.  A thread has a row of its own, so it moves 32 bytes, a whole sector, at a
// time where the state begins on such a boundary.
__device__ __forceinline__ void load_32(const void *p, bool whole, uint32_t (&w)[8])
{
    if (whole) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(p) : "memory");
    } else {
        const uint4 x = static_cast<const uint4 *>(p)[0], y = static_cast<const uint4 *>(p)[1];
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
    }
}
__device__ __forceinline__ void store_32(void *p, bool whole, const uint32_t (&w)[8])
{
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
    } else {
        static_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
template <int COLS> __device__ __forceinline__ void load_state(const void *p, kda_dtype_t type, int64_t at, f2 (&s)[COLS / 2])
{
    const bool whole = (reinterpret_cast<uintptr_t>(p) & 31) == 0;
    uint32_t w[8];
    if (type == KDA_DTYPE_BF16) {
#pragma unroll
        for (int i = 0; i < COLS / 16; i++) {
            load_32(static_cast<const __nv_bfloat16 *>(p) + at + 16 * i, whole, w);
#pragma unroll
            for (int e = 0; e < 8; e++)
                s[8 * i + e] = f2_bf16x2(w[e]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < COLS / 8; i++) {
            load_32(static_cast<const float *>(p) + at + 8 * i, whole, w);
#pragma unroll
            for (int e = 0; e < 4; e++)
                s[4 * i + e] = f2_pack(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
        }
    }
}
template <int COLS> __device__ __forceinline__ void store_state(void *p, kda_dtype_t type, int64_t at, const f2 (&s)[COLS / 2])
{
    const bool whole = (reinterpret_cast<uintptr_t>(p) & 31) == 0;
    uint32_t w[8];
    if (type == KDA_DTYPE_BF16) {
#pragma unroll
        for (int i = 0; i < COLS / 16; i++) {
#pragma unroll
            for (int e = 0; e < 8; e++)
                w[e] = pack_bf16(f2_lo(s[8 * i + e]), f2_hi(s[8 * i + e]));
            store_32(static_cast<__nv_bfloat16 *>(p) + at + 16 * i, whole, w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < COLS / 8; i++) {
#pragma unroll
            for (int e = 0; e < 4; e++)
                w[2 * e] = __float_as_uint(f2_lo(s[4 * i + e])), w[2 * e + 1] = __float_as_uint(f2_hi(s[4 * i + e]));
            store_32(static_cast<float *>(p) + at + 8 * i, whole, w);
        }
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

__device__ __forceinline__ void tmem_read16(uint32_t addr, float (&s)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
                 " tcgen05.wait::ld.sync.aligned;"
                 : "=&f"(s[0]), "=&f"(s[1]), "=&f"(s[2]), "=&f"(s[3]), "=&f"(s[4]), "=&f"(s[5]), "=&f"(s[6]), "=&f"(s[7]),
                   "=&f"(s[8]), "=&f"(s[9]), "=&f"(s[10]), "=&f"(s[11]), "=&f"(s[12]), "=&f"(s[13]), "=&f"(s[14]), "=&f"(s[15])
                 : "r"(addr) : "memory");
}
__device__ __forceinline__ void prefetch_3d(const CUtensorMap *map, int x, int y, int z)
{
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z) : "memory");
}
// Whether a phase is through, without waiting for it (a try_wait may suspend the thread for some microseconds)
__device__ __forceinline__ bool mbar_test(uint32_t mbar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(done) : "r"(mbar), "r"(parity) : "memory");
    return done;
}
// Pairs of bf16, each result rounded once
__device__ __forceinline__ uint32_t bf16_mul(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16_fma(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// Two factors as two bf16 terms each
__device__ __forceinline__ uint2 two_terms(float f, float g)
{
    const uint32_t a = pack_bf16(f, g);
    return make_uint2(a, pack_bf16(f - bf16_lo(a), g - bf16_hi(a)));
}
// 16 lanes by 16 columns (32 bf16): thread t has columns t % 4, t % 4 + 4, .. of row t / 4 and, in between, of row t / 4 + 8
__device__ __forceinline__ void tmem_put_pairs(uint32_t addr, const uint32_t (&u)[8])
{
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(u[0]), "r"(u[1]),
                 "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]) : "memory");
}
// 16 lanes by 16 columns, laid out for stmatrix: thread t has columns 2 (t % 4) and the next of row t / 4, then of row t / 4 + 8,
// then the same of the next 8 columns.  Two of them at once.
__device__ __forceinline__ void tmem_read_pieces(uint32_t at, float (&s)[8], uint32_t bt, float (&t)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n"
                 " tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n"
                 " tcgen05.wait::ld.sync.aligned;"
                 : "=&f"(s[0]), "=&f"(s[1]), "=&f"(s[2]), "=&f"(s[3]), "=&f"(s[4]), "=&f"(s[5]), "=&f"(s[6]), "=&f"(s[7]),
                   "=&f"(t[0]), "=&f"(t[1]), "=&f"(t[2]), "=&f"(t[3]), "=&f"(t[4]), "=&f"(t[5]), "=&f"(t[6]), "=&f"(t[7])
                 : "r"(at), "r"(bt) : "memory");
}
// The same of lanes 0..15 and 16..31, of all four at once: one wait
__device__ __forceinline__ void tmem_read_pieces(uint32_t at, float (&s)[2][8], uint32_t bt, float (&t)[2][8])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%32];\n"
                 " tcgen05.ld.sync.aligned.16x256b.x2.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%33];\n"
                 " tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%34];\n"
                 " tcgen05.ld.sync.aligned.16x256b.x2.b32 {%24,%25,%26,%27,%28,%29,%30,%31}, [%35];\n"
                 " tcgen05.wait::ld.sync.aligned;"
                 : "=&f"(s[0][0]), "=&f"(s[0][1]), "=&f"(s[0][2]), "=&f"(s[0][3]), "=&f"(s[0][4]), "=&f"(s[0][5]), "=&f"(s[0][6]), "=&f"(s[0][7]),
                   "=&f"(s[1][0]), "=&f"(s[1][1]), "=&f"(s[1][2]), "=&f"(s[1][3]), "=&f"(s[1][4]), "=&f"(s[1][5]), "=&f"(s[1][6]), "=&f"(s[1][7]),
                   "=&f"(t[0][0]), "=&f"(t[0][1]), "=&f"(t[0][2]), "=&f"(t[0][3]), "=&f"(t[0][4]), "=&f"(t[0][5]), "=&f"(t[0][6]), "=&f"(t[0][7]),
                   "=&f"(t[1][0]), "=&f"(t[1][1]), "=&f"(t[1][2]), "=&f"(t[1][3]), "=&f"(t[1][4]), "=&f"(t[1][5]), "=&f"(t[1][6]), "=&f"(t[1][7])
                 : "r"(at), "r"(bt), "r"(at + (1u << 20)), "r"(bt + (1u << 20)) : "memory");
}
__device__ __forceinline__ void stmatrix_x4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void stmatrix_x4_t(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, uint32_t src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(map), "r"(src), "r"(x), "r"(y), "r"(z) : "memory");
}
// The warps that take O out, among themselves.  Whether they go on they decide together: a wait may give up in one of them alone, and a
// barrier that it does not come to would hold the others for ever.
template <int N> __device__ __forceinline__ void out_sync() { asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory"); }
template <int N> __device__ __forceinline__ bool out_agree(bool go)
{
    uint32_t all;
    asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %1, 0; bar.red.and.pred q, 1, %2, p; selp.u32 %0, 1, 0, q; }"
                 : "=r"(all) : "r"((uint32_t)go), "n"(N) : "memory");
    return all;
}
// Tokens 2 q and 2 q + 1 of a pair, as the halves of a word: those at or before the row's (gap = the row's token - 2 q)
__device__ __forceinline__ uint32_t seen_pair(int gap)
{
    uint32_t x;
    asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(x) : "r"(max(16 * (gap + 1), 0)));
    return x;
}
// Registers of a warpgroup's threads from here on.  The kernel starts with 80 a thread, and the six shares add up to six times that.
constexpr int REGS_O = 88, REGS_K = 64, REGS_S = 104, REGS_P = REGS_K, REGS_X = 56;
static_assert(REGS_O + REGS_K + 2 * REGS_S + REGS_P + REGS_X <= 6 * 80, "more than the block was launched with");
template <int N, bool MORE> __device__ __forceinline__ void set_registers()
{
    if (MORE)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int DIM, bool STATES_ONLY>
__global__ void __launch_bounds__(THREADS, 1)
kda_linear_chunks_kernel(const __grid_constant__ LinearArgs p, const LinearPlan plan, const __grid_constant__ CUtensorMap qmap,
                         const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap omap)
{
    using S = Shape<DIM, STATES_ONLY>;
    constexpr int CB = S::CB, STAGES = S::STAGES;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *const smem = smem_raw + (base - smem_u32(smem_raw));
    Entry *const entries = reinterpret_cast<Entry *>(smem + S::ENTRY);
    const uint32_t bar = base + S::BAR;
    const uint32_t b_full = bar, b_empty = b_full + 8 * STAGES, b_ent = b_empty + 8 * STAGES, b_ent_free = b_ent + 8 * ENTRIES,
                   b_s = b_ent_free + 8 * ENTRIES, b_p = b_s + 16, b_o = b_p + 16, b_sb = b_o + 16, b_pe = b_sb + 16,
                   b_k = b_pe + 16, b_l = b_k + 16, b_o2 = b_l + 16, b_block = b_o2 + 8, b_drain = b_block + 8;
    static_assert(8 * (2 * STAGES + 2 * ENTRIES + 21) <= 512, "barriers");
    __shared__ uint32_t tmem_slot;
    __shared__ uint4 block_answer;
    __shared__ short order[MAX_RANKED];
    __shared__ int lengths[MAX_RANKED];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < STAGES; i++) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 1);
        }
        for (int i = 0; i < ENTRIES; i++) {
            mbar_init(b_ent + 8 * i, 1);
            mbar_init(b_ent_free + 8 * i, 23);                 // every warp but the one that writes
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(b_s + 8 * i, 1);
            mbar_init(b_p + 8 * i, 4);
            mbar_init(b_o + 8 * i, 1);
            mbar_init(b_drain + 8 * i, 1);
            mbar_init(b_sb + 8 * i, 12);                       // S stored; O before it read
            mbar_init(b_pe + 8 * i, 4);
            mbar_init(b_k + 8 * i, STATES_ONLY ? 16 : 12);     // V~ stored; the last L read
            mbar_init(b_l + 8 * i, 1);
        }
        mbar_init(b_o2, 1);
        mbar_init(b_block, 1);
        mbar_fence_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    for (int i = tid; i < (STATES_ONLY ? 0 : 2 * TILE_CB / 16); i += THREADS)
        reinterpret_cast<uint4 *>(smem + S::P)[i] = make_uint4(0, 0, 0, 0);
    if (DIM == 64)
        for (int i = tid; i < TILE_CB / 16; i += THREADS)
            reinterpret_cast<uint4 *>(smem + S::ZERO)[i] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
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
      set_registers<REGS_X, false>();
      if (warp == 0) {
        // ------------------------------------------------------------ copies
        uint32_t c = 0;
        for (; next(c); c++) {
            const Entry &e = entries[c % ENTRIES];
            const int st = c % STAGES, h = e.h, tok = e.tok0;
            // a later chunk's tiles, into L2 if it is known by now: they are copied from there in a fraction of the time
            const uint32_t later = (c + EARLY) % ENTRIES;
            if (__all_sync(FULL, mbar_test(b_ent + 8 * later, (c + EARLY) / ENTRIES & 1)) && entries[later].valid &&
                lane < S::TILES * CB) {
                const Entry &f = entries[later];
                const int cb = lane % CB, which = lane / CB;
                prefetch_3d(which == 0 ? &kmap : (which == 1 ? &vmap : &qmap), 64 * cb, which == 2 ? f.h : f.h / p.group, f.tok0);
            }
            if (c >= STAGES && !wait(b_empty + 8 * st, c / STAGES - 1))
                break;
            if (lane == 0) {
                const uint32_t to = base + st * S::STAGE, b = b_full + 8 * st;
                mbar_expect_tx(b, S::STAGE);
#pragma unroll
                for (int cb = 0; cb < CB; cb++) {
                    tma_load_3d(to + S::TILE + cb * TILE_CB, &kmap, 64 * cb, h / p.group, tok, b);
                    tma_load_3d(to + cb * TILE_CB, &vmap, 64 * cb, h / p.group, tok, b);
                    if (!STATES_ONLY)
                        tma_load_3d(to + 2 * S::TILE + cb * TILE_CB, &qmap, 64 * cb, h, tok, b);
                }
            }
            arrive(b_ent_free + 8 * (c % ENTRIES));
        }
        // no copy is in flight when the CTA leaves, also where the work was given up
        for (uint32_t i = c < STAGES ? 0 : c - STAGES; i < c; i++)
            timeout |= !mbar_wait(b_full + 8 * (i % STAGES), (i / STAGES) & 1);
      } else if (warp == 1 || warp == 3) {
        // ------------------------------------------------------------ tensor-core issue
        // Warp 1 the scores, as soon as a chunk's tiles are there; warp 3 the products that wait for other warps' work.  The whole
        // warp waits, one elected lane issues from uniform registers.
        const uint32_t tm = __shfl_sync(FULL, tmem, 0), lead = elect_one();
        if (warp == 1) {
            const uint32_t id_s = idesc_bf16(64, 64, false);
            for (uint32_t c = 0; next(c); c++) {
                const uint32_t at = base + (c % STAGES) * S::STAGE;
                if (!STATES_ONLY) {
                    // where they go, P of the chunk before has been formed from
                    if (!wait(b_full + 8 * (c % STAGES), c / STAGES) || (c > 0 && !wait(b_p + 8 * ((c - 1) & 1), (c - 1) >> 1)))
                        break;
                    tc_fence_after();
                    const uint32_t a = desc_lo(at + 2 * S::TILE, 16), b = desc_lo(at + S::TILE, 16), d = tm + TM_S1;
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
                }
                arrive(b_ent_free + 8 * (c % ENTRIES));
            }
        } else {
            const uint32_t id_l = idesc_bf16(128, DIM, true), id_o2 = idesc_bf16(128, 64, false), id_o1 = id_o2 | A_MN;
            bool more = next(0);
            for (uint32_t c = 0; more; c++) {
                const int st = c % STAGES;
                const uint32_t at = base + st * S::STAGE;
                // V as M rows: blocks of 64 features, for D = 64 the second one zeros
                const uint32_t v = desc_lo(at, DIM == 128 ? TILE_CB : S::ZERO - st * S::STAGE);
                if (!wait(b_k + 8 * (c & 1), c >> 1))          // V~ is there, and the place for the product
                    break;
                tc_fence_after();
                const uint32_t d = tm + TM_L, b = desc_lo(at + S::TILE, TILE_CB);
                if (lead && !timeout) {
#pragma unroll
                    for (int r = TERMS - 1; r >= 0; r--) {     // small terms first
                        const uint32_t a = tm + TM_V + 64 * (c & 1) + 32 * r;
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            if (r == TERMS - 1 && k == 0)
                                mma_ts<false>(d, a, b, id_l, 0);
                            else
                                mma_ts<true>(d, a + 8 * k, b + k * (2048 >> 4), id_l, 1);
                        }
                    }
                    umma_commit(b_l + 8 * (c & 1));
                    if (STATES_ONLY)
                        umma_commit(b_empty + 8 * st);
                }
                __syncwarp();
                // (a wait takes some 200 cycles even where nothing is waited for: these are over while that product runs)
                more = next(c + 1);
                if (!STATES_ONLY) {
                    // P is there, and S, and O of the chunk before is read
                    if (!wait(b_p + 8 * (c & 1), c >> 1) || !wait(b_sb + 8 * (c & 1), c >> 1))
                        break;
                    tc_fence_after();
                    const uint32_t q = desc_lo(at + 2 * S::TILE, 16), sb = tm + TM_SB;
                    if (lead && !timeout) {
#pragma unroll
                        for (int k = 0; k < DIM / 16; k++) {
                            const uint32_t step = ((k / 4) * TILE_CB + (k % 4) * 32) >> 4;
                            if (k == 0)
                                mma_ts<false>(tm + TM_O2, sb, q, id_o2, 0);
                            else
                                mma_ts<true>(tm + TM_O2, sb + 8 * k, q + step, id_o2, 1);
                        }
                        umma_commit(b_o2);
                        const uint32_t pd = desc_lo(base + S::P + (c & 1) * TILE_CB, 16);
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
        }
        if (lead) {
            // everything issued has to be through before tensor memory is freed
            const uint32_t b = b_drain + (warp == 3 ? 8 : 0);
            umma_commit(b);
            timeout |= !mbar_wait(b, 0);
        }
        __syncwarp();
      } else {
        // ------------------------------------------------------------ chunks and their decays
        const short *ranked = nullptr;
        if (p.tok.cu && p.tok.N <= MAX_RANKED) {
            for (int i = lane; i < p.tok.N; i += 32) {
                int64_t bos, len;
                seq_range(p.tok.cu, i, p.tok.N, p.tok.T, bos, len);
                lengths[i] = (int)len;
            }
            __syncwarp();
            for (int i = lane; i < p.tok.N; i += 32) {
                const int len = lengths[i];
                int rank = 0;
#pragma unroll 4
                for (int j = 0; j < p.tok.N; j++)
                    rank += lengths[j] > len || (lengths[j] == len && j < i);
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
        auto slot_free = [&](uint32_t c) -> bool { return c < ENTRIES || wait(b_ent_free + 8 * (c % ENTRIES), c / ENTRIES - 1); };
        for (int x = blockIdx.x; x >= 0 && !timeout; x = next_block()) {
            Item w;
            if (!find_item<STATES_ONLY>(p, plan, ranked, x, w, bad))
                continue;
            const int64_t chunks = (w.len + 63) / 64, c0 = (int64_t)w.g * plan.group_chunks;
            const int64_t c1 = c0 + plan.group_chunks < chunks ? c0 + plan.group_chunks : chunks;
            // The first group's state is read from where the join has put it too: the last group, which writes the final state, perhaps
            // in the same place, does not wait for it.
            const int last_group = groups_of(plan, w.len, true);
            const bool from_slot = !STATES_ONLY && (w.g > 0 || (last_group > 0 && p.init));
            const int src = from_slot ? 2 : (!STATES_ONLY && p.init ? 1 : 0);
            const int dst = STATES_ONLY ? 2 : (c1 == chunks && p.fin ? 1 : 0);
            const int64_t pair = (int64_t)w.n * p.H + w.h;
            const int64_t at_src = src == 2 ? slot_of(p, plan, w.n, w.bos, w.g > 0 ? w.g - 1 : last_group) * p.H + w.h : pair;
            const int64_t at_dst = STATES_ONLY ? slot_of(p, plan, w.n, w.bos, w.g) * p.H + w.h : pair;
            // the state that the item starts from, into L2
            if (src != 0 && lane == 0) {
                const int size = src == 1 && plan.state_type == KDA_DTYPE_BF16 ? 2 : 4;
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const char *>(src == 1 ? p.init : plan.states) +
                             at_src * DIM * DIM * size), "r"(DIM * DIM * size) : "memory");
            }
            const float fixed = p.log_decay ? p.log_decay[w.h] : 0.0f;
            auto gate = [&](int64_t i) -> float { return i < w.len ? gate_of(p, w.bos + i, w.h) : 0.0f; };
            // Two chunks at a time, one by lanes 0..15 and one by the others, four tokens a lane.
            const int half = lane >> 4, j = 4 * (lane & 15);
            Sum total{0.0f, 0.0f};
            float g[4];
#pragma unroll
            for (int q = 0; q < 4; q++)
                g[q] = gate((c0 + half) * 64 + j + q);
            for (int64_t i0 = c0; i0 < c1 || i0 == c0; i0 += 2) {   // (an empty sequence has one chunk of no tokens)
                const int64_t i = i0 + half;
                Sum a[4];
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const Sum x = in_base_2(i * 64 + j + q < w.len ? log_decay_of(fixed, g[q], bad) : 0.0f);
                    a[q] = q > 0 ? add(a[q > 0 ? q - 1 : 0], x) : x;
                }
                if (i0 + 2 < c1) {                             // loaded now and looked at in the next pass
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        g[q] = gate((i + 2) * 64 + j + q);
                }
                Sum sum = a[3];
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) {
                    const Sum z{__shfl_up_sync(FULL, sum.hi, o, 16), __shfl_up_sync(FULL, sum.lo, o, 16)};
                    if ((lane & 15) >= o)
                        sum = add(z, sum);
                }
                Sum before{__shfl_up_sync(FULL, sum.hi, 1, 16), __shfl_up_sync(FULL, sum.lo, 1, 16)};
                if ((lane & 15) == 0)
                    before = Sum{0.0f, 0.0f};
#pragma unroll
                for (int q = 0; q < 3; q++)
                    a[q] = add(before, a[q]);
                a[3] = sum;
                const Sum all{__shfl_sync(FULL, sum.hi, 15, 16), __shfl_sync(FULL, sum.lo, 15, 16)};
                const int count = i0 + 1 < c1 ? 2 : 1;         // (the second may be the next group's first)
                if (STATES_ONLY && half < count)
                    total = add(total, all);                   // every other chunk's
                if (!slot_free(c + count - 1))                 // and the one before, which every warp is through with earlier
                    break;
                Entry &e = entries[(c + half) % ENTRIES];
                if (half < count) {
                    if (!STATES_ONLY) {                        // what P and O want
                        *reinterpret_cast<float4 *>(&e.hi[j]) = make_float4(a[0].hi, a[1].hi, a[2].hi, a[3].hi);
                        *reinterpret_cast<float4 *>(&e.lo[j]) = make_float4(a[0].lo, a[1].lo, a[2].lo, a[3].lo);
                        *reinterpret_cast<float4 *>(&e.ea[j]) = make_float4(p.scale * ex2_approx(a[0].hi), p.scale * ex2_approx(a[1].hi),
                                                                            p.scale * ex2_approx(a[2].hi), p.scale * ex2_approx(a[3].hi));
                    }
                    const uint2 f = two_terms(ex2_approx(minus(all, a[0])), ex2_approx(minus(all, a[1])));
                    const uint2 g = two_terms(ex2_approx(minus(all, a[2])), ex2_approx(minus(all, a[3])));
                    *reinterpret_cast<uint2 *>(&e.f[0][j / 2]) = make_uint2(f.x, g.x);
                    *reinterpret_cast<uint2 *>(&e.f[1][j / 2]) = make_uint2(f.y, g.y);
                    if (j == 0) {
                        const int left = (int)(w.len - i * 64 < 64 ? w.len - i * 64 : 64);
                        e.valid = 1;
                        e.first = i == c0, e.last = i + 1 >= c1;
                        e.tok0 = (int)(w.bos + i * 64), e.len = left, e.h = w.h;
                        e.decay = decay_of<STATES_ONLY>(all);
                        e.src = src, e.at_src = at_src, e.dst = dst, e.at_dst = at_dst;
                    }
                }
                __syncwarp();
                if (lane < count)
                    mbar_arrive(b_ent + 8 * ((c + lane) % ENTRIES));
                c += count;
            }
            if (STATES_ONLY) {
                const Decay d = decay_of<false>(add(total, Sum{__shfl_xor_sync(FULL, total.hi, 16), __shfl_xor_sync(FULL, total.lo, 16)}));
                if (lane == 0)
                    plan.decays[at_dst] = make_float2(d.hi, d.lo);
            }
        }
        if (slot_free(c)) {
            if (lane == 0)
                entries[c % ENTRIES].valid = 0;
            arrive(b_ent + 8 * (c % ENTRIES));
        }
        if (asked > answers)
            timeout |= !mbar_wait(b_block, answers & 1);
      }
    } else if (!STATES_ONLY && warp < 8) {
        // ------------------------------------------------------------ P, 16 tokens a warp
        // In blocks of 16 x 16: a thread has two neighbouring columns of rows t / 4 and t / 4 + 8, twice.  Blocks of later tokens are
        // zeros from the start.
        set_registers<REGS_P, false>();
        const int wp = warp - 4, r0 = 16 * wp + lane / 4, c0 = 2 * (lane & 3);
        const f2 scale = f2_pack(p.scale, p.scale), minus = f2_pack(-1.0f, -1.0f);
        // where this lane's row of a block's four 8 x 8 parts goes: rows 0..7 and 8..15 of its left columns, then of its right ones
        const int row = 16 * wp + (lane & 7) + (lane & 8), right = lane >> 4;
        const uint32_t to = base + S::P + row * 128;
        for (uint32_t c = 0; next(c); c++) {
            const Entry &e = entries[c % ENTRIES];
            {
                const float h0 = e.hi[r0], l0 = e.lo[r0], h1 = e.hi[r0 + 8], l1 = e.lo[r0 + 8];
                if ((c >= 2 && !wait(b_pe + 8 * (c & 1), (c >> 1) - 1)) || !wait(b_s + 8 * (c & 1), c >> 1))
                    break;
                tc_fence_after();
                const uint32_t tm = tmem + TM_S1 + ((uint32_t)wp << 21), pt = to + (c & 1) * TILE_CB;
#pragma unroll 1
                for (int pair = 0; 2 * pair <= wp; pair++) {   // two blocks; the second may be all of later tokens
                    float s[2][8];
                    tmem_read_pieces(tm + 32 * pair, s[0], tm + 32 * pair + 16, s[1]);
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        uint32_t y[4];
#pragma unroll
                        for (int q = 0; q < 2; q++) {          // columns 0..7 and 8..15
                            const int j = 32 * pair + 16 * k + 8 * q + c0;
                            const float2 h = *reinterpret_cast<const float2 *>(&e.hi[j]);
                            const float2 l = *reinterpret_cast<const float2 *>(&e.lo[j]);
                            const f2 hj = f2_pack(h.x, h.y), lj = f2_pack(l.x, l.y);
                            const f2 d0 = f2_add(f2_fma(hj, minus, f2_pack(h0, h0)), f2_fma(lj, minus, f2_pack(l0, l0)));
                            const f2 d1 = f2_add(f2_fma(hj, minus, f2_pack(h1, h1)), f2_fma(lj, minus, f2_pack(l1, l1)));
                            const f2 a = f2_mul(f2_mul(f2_pack(s[k][4 * q], s[k][4 * q + 1]), scale), f2_pack(ex2_approx(f2_lo(d0)), ex2_approx(f2_hi(d0))));
                            const f2 b = f2_mul(f2_mul(f2_pack(s[k][4 * q + 2], s[k][4 * q + 3]), scale), f2_pack(ex2_approx(f2_lo(d1)), ex2_approx(f2_hi(d1))));
                            // bf16, V's type, as the product takes it; later tokens' are cleared, whatever they are
                            y[2 * q] = pack_bf16(f2_lo(a), f2_hi(a)) & seen_pair(r0 - j);
                            y[2 * q + 1] = pack_bf16(f2_lo(b), f2_hi(b)) & seen_pair(r0 + 8 - j);
                        }
                        stmatrix_x4(pt + (((4 * pair + 2 * k + right) ^ (row & 7)) << 4), y[0], y[1], y[2], y[3]);
                    }
                }
                tc_fence_before();
                fence_async_smem();
                arrive(b_p + 8 * (c & 1));
            }
            arrive(b_ent_free + 8 * (c % ENTRIES));
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------ V~
        // From shared memory, turned, into tensor memory: 16 features by 32 tokens at a time.  (Where only states are wanted the warps
        // of P take half of the tokens.)
        set_registers<REGS_K, false>();
        constexpr int THREADS_K = STATES_ONLY ? 256 : 128;
        const int t = tid - (384 - THREADS_K), quad = warp & 3, r = lane & 7;
        const int tok0 = STATES_ONLY && warp < 8 ? 32 : 0, tok1 = STATES_ONLY && warp >= 8 ? 32 : 64;
        for (uint32_t c = 0; next(c); c++) {
            const Entry &e = entries[c % ENTRIES];
            const int st = c % STAGES, len = e.len;
            // V is there, and the product of the chunk before the last is through, whose V~ lies where this one's will
            if ((c >= 2 && !wait(b_l + 8 * (c & 1), (c >> 1) - 1)) || !wait(b_full + 8 * st, c / STAGES))
                break;
            unsigned char *const stage = smem + st * S::STAGE;
            if (len < 64) {
                // What lies behind the sequence is cleared from K, by all, and from V, by the warps that turn it.  (The scores' product may
                // read K meanwhile: what it makes of these rows is masked, whatever it is.)
                for (int i = t; i < (64 - len) * 8 * CB; i += THREADS_K)
                    *reinterpret_cast<uint4 *>(stage + S::TILE + i / ((64 - len) * 8) * TILE_CB + len * 128 + i % ((64 - len) * 8) * 16) =
                        make_uint4(0, 0, 0, 0);
                if (32 * quad < DIM)
                    for (int i = lane; i < 64 * 4; i += 32) {
                        const int tok = i / 4;
                        if (tok >= len && tok >= tok0 && tok < tok1)
                            *reinterpret_cast<uint4 *>(stage + quad / 2 * TILE_CB + tok * 128 + (((quad % 2 * 4 + i % 4) ^ (tok & 7)) << 4)) =
                                make_uint4(0, 0, 0, 0);
                    }
                fence_async_smem();
                __syncwarp();
            }
            if (32 * quad < DIM) {
                tc_fence_after();
                const uint32_t vt = base + st * S::STAGE + quad / 2 * TILE_CB;
#pragma unroll 1
                for (int i = tok0 / 16; i < tok1 / 16; i++) {
                    const int half = i & 1, tok = 32 * (i >> 1);
                    // four blocks of 8 x 8 a load: two of neighbouring features, of 8 tokens and of the next 8
                    const uint32_t from = vt + (tok + (lane >> 4) * 8 + r) * 128 + (((quad % 2 * 4 + 2 * half + (lane >> 3 & 1)) ^ r) << 4);
                    uint32_t w[2][4], y[TERMS][8];
                    ldsm_x4_t(from, w[0]);
                    ldsm_x4_t(from + 16 * 128, w[1]);
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const uint32_t f = e.f[0][tok / 2 + 4 * q + (lane & 3)], g = e.f[1][tok / 2 + 4 * q + (lane & 3)];
#pragma unroll
                        for (int x = 2 * q; x < 2 * q + 2; x++) {
                            // v f1 rounded, and what that left off, which is a bf16 number, with v f2
                            const uint32_t v = w[x / 4][x % 4];
                            y[0][x] = bf16_mul(v, f);
                            y[1][x] = bf16_fma(v, g, bf16_fma(v, f, y[0][x] ^ 0x80008000u));
                        }
                    }
                    const uint32_t to = tmem + TM_V + 64 * (c & 1) + tok / 2 + ((uint32_t)(32 * quad + 16 * half) << 16);
                    tmem_put_pairs(to, y[0]);
                    tmem_put_pairs(to + 32, y[1]);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
            }
            arrive(b_k + 8 * (c & 1));
            if (lane == 0)
                mbar_arrive(b_ent_free + 8 * (c % ENTRIES));
        }
    } else if (warp < 20) {
        // ------------------------------------------------------------ the state
        set_registers<REGS_S, true>();
        constexpr int COLS = DIM / 2;
        const int half = (warp - 12) / 4, v = (warp & 3) * 32 + lane;
        const uint32_t quad = (uint32_t)(warp & 3) << 21;
        const bool mine = (warp & 3) * 32 < DIM;
        const uint32_t tm_l = tmem + TM_L + quad + half * COLS, tm_sb = tmem + TM_SB + quad + half * (COLS / 2);
        f2 s[COLS / 2];
#pragma unroll
        for (int i = 0; i < COLS / 2; i++)
            s[i] = 0;
        if (lane == 0)
            mbar_arrive(b_k);                                  // L is free
        // S before chunk c, as the operand of its product
        auto put = [&](uint32_t c) -> bool {
            if (STATES_ONLY)
                return true;
            if (c > 0 && !wait(b_o2, c - 1))                  // the product with the one before
                return false;
            if (mine) {
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < COLS / 32; k++) {
                    uint32_t u[16];
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        u[i] = pack_bf16(f2_lo(s[16 * k + i]), f2_hi(s[16 * k + i]));
                    tmem_put16(tm_sb + 16 * k, u);
                }
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
                    for (int i = 0; i < COLS / 2; i++)
                        s[i] = 0;
                if (!put(c))
                    break;
            }
            if (!wait(b_l + 8 * (c & 1), c >> 1))
                break;
            if (mine) {
                tc_fence_after();
                const Decay d = e.decay;
                const f2 hi = f2_pack(d.hi, d.hi), lo = f2_pack(d.lo, d.lo);
#pragma unroll
                for (int i = 0; i < COLS; i += 16) {
                    float l[16];
                    tmem_read16(tm_l + i, l);
                    if (STATES_ONLY && d.lo == 0.0f) {
#pragma unroll
                        for (int j = 0; j < 8; j++)
                            s[i / 2 + j] = f2_fma(hi, s[i / 2 + j], f2_pack(l[2 * j], l[2 * j + 1]));
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; j++)
                            s[i / 2 + j] = f2_fma(hi, s[i / 2 + j], f2_fma(lo, s[i / 2 + j], f2_pack(l[2 * j], l[2 * j + 1])));
                    }
                }
                tc_fence_before();
            }
            arrive(b_k + 8 * ((c + 1) & 1));                   // for the next chunk
            if (!e.last) {
                if (!put(c + 1))
                    break;
            } else if (mine && e.dst) {
                store_state<COLS>(e.dst == 1 ? p.fin : plan.states, e.dst == 1 ? plan.state_type : KDA_DTYPE_FP32,
                                  (e.at_dst * DIM + v) * DIM + half * COLS, s);
            }
            arrive(b_ent_free + 8 * (c % ENTRIES));
        }
    } else {
        // ------------------------------------------------------------ O
        set_registers<REGS_O, true>();
        const int ow = warp - 20, t = tid - 640;                // warp and thread of the four
        const uint32_t quad = (uint32_t)ow << 21;
        constexpr int WARPS = DIM / 32;                        // that have features
        // where this lane's row of a piece's four 8 x 8 blocks goes: token (lane & 7) of 8, 8 features
        const int r = lane & 7, block = lane >> 3;
        const uint32_t to = base + S::OUT + (ow >> 1) * TILE_CB + ((block >> 1) * 8 + r) * 128;
        if (lane == 0)
            mbar_arrive(b_sb);                                 // O is free
        const uint32_t to0 = to + ((((ow & 1) * 4 + (block & 1)) ^ r) << 4), to1 = to + ((((ow & 1) * 4 + 2 + (block & 1)) ^ r) << 4);
        for (uint32_t c = 0;; c++) {
            bool go = next(c) && (STATES_ONLY || wait(b_o + 8 * (c & 1), c >> 1));
            if (!STATES_ONLY && ow < WARPS) {
                if (t == 0)
                    bulk_wait_read_all();                      // the last chunk's O has left
                go = out_agree<32 * WARPS>(go);
            }
            if (!go)
                break;
            const Entry &e = entries[c % ENTRIES];
            if (!STATES_ONLY) {
                if (ow < WARPS) {
                    tc_fence_after();
                    const int len = e.len, tok0 = e.tok0, h = e.h;
                    f2 z = 0;                                  // stays 0 while V^T P^T is finite
#pragma unroll 1
                    for (int first = 0; first < 64; first += 16) {
                        const float2 f0 = *reinterpret_cast<const float2 *>(&e.ea[first + 2 * (lane & 3)]);
                        const float2 f1 = *reinterpret_cast<const float2 *>(&e.ea[first + 8 + 2 * (lane & 3)]);
                        const f2 ea[2] = {f2_pack(f0.x, f0.y), f2_pack(f1.x, f1.y)};
                        uint32_t w[2][4];
                        float x[2][8], y[2][8];
                        tmem_read_pieces(tmem + TM_O1 + quad + first, x, tmem + TM_O2 + quad + first, y);
#pragma unroll
                        for (int up = 0; up < 2; up++) {       // lanes 0..15 and 16..31
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                const f2 u = f2_pack(x[up][2 * i], x[up][2 * i + 1]);
                                z = f2_fma(u, 0, z);
                                const f2 o = f2_fma(ea[i / 2], f2_pack(y[up][2 * i], y[up][2 * i + 1]), u);
                                w[up][i] = pack_bf16(f2_lo(o), f2_hi(o));
                            }
                        }
                        stmatrix_x4_t(to0 + first * 128, w[0][0], w[0][1], w[0][2], w[0][3]);
                        stmatrix_x4_t(to1 + first * 128, w[1][0], w[1][1], w[1][2], w[1][3]);
                    }
                    if (__any_sync(FULL, !(f2_lo(z) + f2_hi(z) == 0.0f))) {
                        // (P is through; waited for here so that this thread sees it.  V's place may be another chunk's by now.)
                        wait(b_p + 8 * (c & 1), c >> 1);
                        const int v = ow * 32 + lane;
                        const unsigned char *pt = smem + S::P + (c & 1) * TILE_CB;
                        const __nv_bfloat16 *vt = p.v + (int64_t)tok0 * p.v_stride + h / p.group * DIM + v;
                        for (int i = 0; i < len; i++) {
                            __syncwarp();                      // the reads are the whole warp's
                            float u = tmem_read1(tmem + TM_O1 + quad + i);
                            const float o = tmem_read1(tmem + TM_O2 + quad + i);
                            if (u - u != 0.0f) {
                                u = 0.0f;
                                for (int j = 0; j <= i; j++) {
                                    const __nv_bfloat16 a = *reinterpret_cast<const __nv_bfloat16 *>(
                                        pt + i * 128 + (((j / 8) ^ (i & 7)) << 4) + (j % 8) * 2);
                                    u = fmaf(__bfloat162float(a), __bfloat162float(vt[j * p.v_stride]), u);
                                }
                            }
                            *reinterpret_cast<__nv_bfloat16 *>(smem + S::OUT + (v / 64) * TILE_CB + i * 128 +
                                                               (((v % 64 / 8) ^ (i & 7)) << 4) + (v % 8) * 2) =
                                __float2bfloat16_rn(fmaf(e.ea[i], o, u));
                        }
                        __syncwarp();
                    }
                    tc_fence_before();
                    fence_async_smem();
                    arrive(b_sb + 8 * ((c + 1) & 1));          // for the next chunk
                    arrive(b_pe + 8 * (c & 1));
                    out_sync<32 * WARPS>();
                    if (len == 64) {
                        if (t == 0) {
#pragma unroll
                            for (int cb = 0; cb < CB; cb++)
                                tma_store_3d(&omap, base + S::OUT + cb * TILE_CB, 64 * cb, h, tok0);
                            bulk_commit();
                        }
                    } else {                                   // only the sequence's tokens
                        for (int i = t; i < len * (DIM / 8); i += 32 * WARPS) {
                            const int tok = i / (DIM / 8), ch = i % (DIM / 8);
                            *reinterpret_cast<uint4 *>(p.out + ((int64_t)(tok0 + tok) * p.H + h) * DIM + ch * 8) =
                                *reinterpret_cast<const uint4 *>(smem + S::OUT + (ch / 8) * TILE_CB + tok * 128 + (((ch % 8) ^ (tok & 7)) << 4));
                        }
                    }
                } else {
                    arrive(b_sb + 8 * ((c + 1) & 1));          // for the next chunk
                    arrive(b_pe + 8 * (c & 1));
                }
            }
            arrive(b_ent_free + 8 * (c % ENTRIES));
        }
        if (t == 0)
            bulk_wait_read_all();
    }
    report(p.err, bad, DEVERR_CU_SEQLENS);
    report(p.err, timeout, DEVERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS));
}

// ---------------------------------------------------------------- groups' start states
// S_0 the call's; what group g adds lies in its slot and is replaced by S_(g+1) = e^(A_g) S_g + it, the state that group g + 1 starts from.
// The last group's slot, which no later group starts from, gets S_0.
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
    if (p.init)                                                // the first group's own start, in the last one's slot
        *reinterpret_cast<float4 *>(plan.states + ((first + groups) * p.H + h) * size + at) = make_float4(s[0], s[1], s[2], s[3]);
    // (eight groups' loads before their stores, which the compiler could not tell apart: one group after the other took 13 us for 18
    // groups of 8 heads, 8.5 this way)
    constexpr int AT_ONCE = 8;
    for (int first_g = 0; first_g < groups; first_g += AT_ONCE) {
        float4 l[AT_ONCE];
        float2 f[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; i++)
            if (first_g + i < groups) {
                const int64_t slot = (first + first_g + i) * p.H + h;
                f[i] = plan.decays[slot];
                l[i] = *reinterpret_cast<const float4 *>(plan.states + slot * size + at);
            }
#pragma unroll
        for (int i = 0; i < AT_ONCE; i++)
            if (first_g + i < groups) {
                const Decay d{f[i].x, f[i].y};
                s[0] = decayed(d, s[0], l[i].x), s[1] = decayed(d, s[1], l[i].y), s[2] = decayed(d, s[2], l[i].z), s[3] = decayed(d, s[3], l[i].w);
                *reinterpret_cast<float4 *>(plan.states + ((first + first_g + i) * p.H + h) * size + at) = make_float4(s[0], s[1], s[2], s[3]);
            }
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

template <int DIM, bool STATES_ONLY>
cudaError_t launch(const LinearArgs &p, const LinearPlan &plan, int64_t items, const CUtensorMap *maps, cudaStream_t st)
{
    static std::atomic<uint64_t> ready;      // devices whose kernel attribute is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(ready.load() >> dev & 1)) {
        e = cudaFuncSetAttribute(kda_linear_chunks_kernel<DIM, STATES_ONLY>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Shape<DIM, STATES_ONLY>::SMEM);
        if (e == cudaSuccess)
            ready.fetch_or(1ull << dev);
    }
    if (e != cudaSuccess)
        return e;
    return launch_in_row(kda_linear_chunks_kernel<DIM, STATES_ONLY>, (unsigned)items, THREADS, Shape<DIM, STATES_ONLY>::SMEM, 1, st, p,
                         plan, maps[0], maps[1], maps[2], maps[3]);
}

template <int DIM> cudaError_t launch_all(const LinearArgs &p, const LinearPlan &plan, cudaStream_t st)
{
    CUtensorMap maps[4];
    const int64_t tokens = p.tok.cu ? p.tok.T : p.tok.N * p.tok.T;
    cudaError_t e = token_map(&maps[0], p.q, DIM, p.H, tokens, p.q_stride);
    if (e == cudaSuccess)
        e = token_map(&maps[1], p.k, DIM, p.H / p.group, tokens, p.k_stride);
    if (e == cudaSuccess)
        e = token_map(&maps[2], p.v, DIM, p.H / p.group, tokens, p.v_stride);
    if (e == cudaSuccess)
        e = token_map(&maps[3], p.out, DIM, p.H, tokens, (int64_t)p.H * DIM);
    if (e == cudaSuccess && plan.groups > 1) {
        e = launch<DIM, true>(p, plan, plan.items_before, maps, st);
        if (e == cudaSuccess)
            e = launch_in_row(kda_linear_join_kernel, (unsigned)((int64_t)p.tok.N * p.H * (DIM * DIM / 4 / 256)), 256, 0, 1, st, p, plan);
    }
    return e != cudaSuccess ? e : launch<DIM, false>(p, plan, plan.items, maps, st);
}

}  // namespace

cudaError_t launch_linear_chunks(const LinearArgs &p, const LinearPlan &plan, cudaStream_t st)
{
    return p.dim == 128 ? launch_all<128>(p, plan, st) : launch_all<64>(p, plan, st);
}

}  // namespace kda
