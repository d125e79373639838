// Windowed attention over the paged cache on the tensor cores: 256 query rows a CTA, keys in tiles of 128.
//
// Rows.  An item is a run of 256 / group tokens of a (sequence, key head) with all heads of the group: up to 256 rows (row
// = token * group + head, so heads that share keys share the tile), in two halves of 128.  Keys.  The rows need the sinks
// and the positions from the first row's window on: two ranges of positions, cut into granules of at most 32 positions
// that lie in one page each, and strung together to a list of "virtual" keys; 4 to 8 granules make a key tile, so a few
// sinks cost a granule and not a tile.  Granules past the end are loaded from outside the cache (zeros).
//
// Per half and 64 keys (half a key tile):  S = Q K^T (tcgen05, fp32 in tensor memory);  P = 2^(scale S - m) with one
// thread a row, no shuffles;  O += P V with P (bf16) read from tensor memory where S was.  From the commit of S to the P
// that the issuing warp waits for lie some 2000 cycles of latency even without any arithmetic, against 500 of tensor time
// in a half's S and P V for 64 keys: so a half has two S in tensor memory (2 x 64 columns; O takes 128), and the S after
// next is formed while the softmax works on this one.  (One product for 128 keys reads Q once and not twice, but fills both S, so
// that the softmax waits for it: 1399 us for the 1270 below, 126 for 116.)  An issuing warp's own instructions are the next bound (1150 cycles
// of waits and commits for 64 keys with nothing else to do), hence key tiles of twice that and a warp for each half.
// The running maximum m is moved (and O and l rescaled) only when a row's maximum has grown by more than 2^8: any m
// gives the same quotient, and 2^8 is far from overflow in the fp32 sums.  So a tile's exponentials do not wait for its
// maximum: they are taken with the m at hand while the maximum is formed, and taken again (S still stands; P is stored
// last) in the rare tile that moves m.  A row's first m is 0 when its first keys' maximum is within 2^8 of that either way.
// (Reading S once for the maximum and once more for P there: 137 us for the ragged prompts below.)
//
// Warps 0..3 and 4..7: the halves' softmax and epilogue; warp 8: bulk tensor copies of K and V tiles into a ring; warps 9
// and 10: tensor-core issue for a half each (one thread for both halves spent longer issuing than the tensor cores took:
// 1918 us at 8192 tokens, 96 heads); warp 11: works out the items and brings in their Q.  One CTA an SM walks the (row
// tile, key head, split) items: copies and first S of the next item run while the last one's rows are scaled and stored.
// Where there are fewer items than SMs their keys are split: 2, 4 or 8 splits are a cluster that joins them in the same
// launch, each CTA finishing its share of the rows (two sequences of 509 tokens after 20,011, window 2049, D 64, 14 heads over 2,
// 2 splits: 22.5 us, through memory and a second kernel 28.7; launched as it is now 20.6).
// (When every warp worked out the items for itself and the softmax warps loaded Q, an item of 9 steps spent 13,000 cycles
// between them and 16,000 in them.)
//
// Measured (bf16 rate 1875 TFLOP/s): 8192 tokens, 96 heads over 8, full window, 1.27 ms, 1300 TFLOP/s, 69%; 12 ragged
// prompts of 8192 tokens in all, 64 heads over 8, window 512 and 4 sinks, 116 us.  What bounds it: a step of both halves takes
// 1500 cycles, about what its products take with S in pieces of 64 keys, whose operands both come from shared memory (6 KB
// for 32 cycles of tensor time, against 128 bytes a cycle); the softmax is busy for 870 of them.  Short windows pay the
// 5000 cycles between items and the masked edges besides.
//
// A key that a row does not see gets P = 0.  0 x v is NaN for an infinite or NaN v, and the matrix product has no way
// to skip it: rows past the sequence's end are cleared in shared memory, and an output row that does not come out
// finite is taken again from the definition, key by key, unless what it sees makes it so (attn_mend_rows).
#include "kda_attn.cuh"

#include <atomic>
#include <cfloat>

namespace kda {
namespace {

constexpr int KEYS = 128, SUB = 64;          // keys of a tile, and of a step of the softmax
constexpr int THREADS = 384;                 // three warpgroups
constexpr int HALF = 128;                    // rows of a half
constexpr int TMEM_COLS = 512;
constexpr int TM_S = 0, TM_O = 256;          // columns: two S a half (64 each), O of both halves
constexpr int ITEMS = 4;                      // items worked out ahead
constexpr float RESCALE_AT = 8.0f;           // base-2 growth of the maximum that moves it
constexpr unsigned FULL = 0xffffffffu;

template <int DIM> struct Shape {
    static constexpr int TILE = KEYS * DIM * 2;              // bytes of a K or V tile
    static constexpr int Q = HALF * DIM * 2;                 // of a half's Q
    static constexpr int SLOTS = DIM == 128 ? 4 : 8;         // ring: K0 V0 K1 V1 ...
    static constexpr int STAGE = 32 * 128;                   // a softmax warp's rows on their way out, 128 bytes of each
    static constexpr int OUT = 2 * Q + SLOTS * TILE;         // behind Q and the ring
    static constexpr int BAR = OUT + 8 * STAGE;              // mbarriers last
    static constexpr int SMEM = 1024 + BAR + 768;            // 1024: alignment of the swizzle atoms
    static_assert(SLOTS * TILE >= ATTN_ROWS * DIM * 4, "a cluster's parts of a CTA's rows go where the ring was");
};

struct Tile {             // one item; positions, rows and tokens fit 32 bits (checked on the host)
    int valid;            // 0: no more items
    int n, kvh, split;
    int len;              // tokens of the sequence in the cache
    int tok0;             // first token of the item in the batch
    int pos0;             // its position
    int rows;             // rows of the item, 1..256
    int sink_span;        // virtual keys of the sinks (a multiple of the granule)
    int start;            // position of virtual key sink_span
    int virt;             // virtual keys in all
    int t0, t1;           // key tiles of this split
    int lo[2], hi[2];     // their steps (of SUB keys) that a half needs
};

__device__ __forceinline__ int virt_pos(const Tile &w, int v) { return v < w.sink_span ? v : v - w.sink_span + w.start; }

// r / group for a row r < 256 of an item (plan.magic = ceil(2^20 / group), group <= 256: exact)
__device__ __forceinline__ int token_of(const AttnPlan &plan, int r) { return (int)(((uint32_t)r * plan.magic) >> 20); }

// Works out item x; not valid when there is none (ragged batches have fewer than the bound the grid is made for).  By a
// whole warp.
__device__ __forceinline__ void find_tile(const AttnArgs &p, const AttnPlan &plan, int x, Tile &w, bool &bad)
{
    const int lane = threadIdx.x & 31;
    w.valid = 0;
    if (x >= plan.items)
        return;
    // heaviest first where the work grows along a sequence: the last tiles of all key heads
    w.split = 0;
    if (plan.splits > 1) {
        w.split = x % plan.splits;                  // the splits of an item are neighbours: a cluster
        x /= plan.splits;
    }
    w.kvh = x % p.cache.hkv;
    x /= p.cache.hkv;
    const int run = plan.run;                       // tokens of an item
    int tile = 0, len_q = 0, bos = 0;
    if (p.tok.cu) {
        int before = 0;
        for (int base = 0; base < p.tok.N; base += 32) {
            const int n = base + lane;
            int64_t from = 0, len = 0;
            if (n < p.tok.N)
                bad |= seq_range(p.tok.cu, n, p.tok.N, p.tok.T, from, len);
            const int cnt = ((int)len + run - 1) / run;
            int sum = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(FULL, sum, o);
                if (lane >= o)
                    sum += y;
            }
            const unsigned m = __ballot_sync(FULL, before + sum > x);
            if (m) {
                const int src = __ffs(m) - 1;
                w.n = base + src;
                bos = __shfl_sync(FULL, (int)from, src);
                len_q = __shfl_sync(FULL, (int)len, src);
                tile = x - (before + __shfl_sync(FULL, sum - cnt, src));
                w.valid = 1;
                break;
            }
            before += __shfl_sync(FULL, sum, 31);
        }
        if (!w.valid)
            return;
    } else {
        len_q = (int)p.tok.T;
        const int per = (len_q + run - 1) / run;
        w.n = x % p.tok.N;
        tile = per - 1 - x / p.tok.N;
        bos = w.n * len_q;
        w.valid = 1;
    }
    const int count = min(len_q - tile * run, run);  // tokens of the item
    w.rows = count * p.group;
    w.tok0 = bos + tile * run;
    w.len = (int)cache_len(p.cache, w.n, bad);
    w.pos0 = w.len - len_q + tile * run;
    const int g = plan.granule, p1 = w.pos0 + count - 1;
    w.sink_span = w.start = w.virt = 0;
    if (p1 >= 0) {                                  // else all rows are before the first token
        int lo = max(w.pos0 - p.window + 1, 0) & -g, sink = (p.sinks + g - 1) & -g;
        if (lo <= sink)
            sink = lo = 0;                          // one range
        w.sink_span = sink;
        w.start = lo;
        w.virt = sink + (p1 + 1 - lo);
    }
    const int tiles = (w.virt + KEYS - 1) / KEYS;
    w.t0 = 0;
    w.t1 = tiles;
    if (plan.splits > 1) {
        w.t0 = tiles * w.split / plan.splits;       // at most 2^24 tiles, 64 splits
        w.t1 = tiles * (w.split + 1) / plan.splits;
    }
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int first = h * HALF, last = min(w.rows, first + HALF) - 1;
        const int s0 = 2 * w.t0, s1 = 2 * w.t1;
        w.lo[h] = w.hi[h] = s0;
        if (first > last)
            continue;
        const int a = w.pos0 + token_of(plan, first) - p.window + 1, b = w.pos0 + token_of(plan, last);
        if (b < 0)
            continue;
        // the half's window, in steps; with sinks a half needs the steps from the first on
        const int lo = p.sinks > 0 || a <= w.start ? 0 : (a - w.start) / SUB;
        const int hi = (b - w.start + w.sink_span) / SUB + 1;
        w.lo[h] = min(max(lo, s0), s1);
        w.hi[h] = max(min(max(hi, s0), s1), w.lo[h]);
    }
}

// ---------------------------------------------------------------- tensor cores and copies
// 128-byte swizzled shared-memory matrix descriptors, as their two words.  K-major: groups of 8 rows 1024 bytes apart;
// MN-major: groups of 8 along K 1024 bytes apart, blocks of 64 along MN `lbo` apart.  The high word is the same for all;
// in the low one a step along the operand is an addition, so that the issuing thread spends an instruction or two a
// product (building whole descriptors there cost as much as the products themselves).
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
// (In a cluster a shared-memory address has the CTA's rank above its 18 bits.)
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return ((saddr & 0x3ffff) >> 4) | ((lbo >> 4) << 16); }
// fp32 accumulator, bf16 A and B, A K-major, B K-major or (mn) MN-major
__device__ __forceinline__ constexpr uint32_t idesc_bf16(int M, int N, bool mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}
// D[tmem] (+)= A B^T, A in shared or tensor memory, B in shared memory; ACC: added to D, else as `acc` says
template <bool ACC> __device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, int acc)
{
    if (ACC)
        asm volatile("{\n .reg .pred p;\n .reg .b64 x, y;\n setp.eq.u32 p, 0, 0;\n mov.b64 x, {%1, %4};\n mov.b64 y, {%2, %4};\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}"
                     ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(DESC_HI) : "memory");
    else
        asm volatile("{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n mov.b64 x, {%1, %4};\n mov.b64 y, {%2, %4};\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}"
                     ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(DESC_HI), "r"(acc) : "memory");
}
template <bool ACC> __device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t idesc, int acc)
{
    if (ACC)
        asm volatile("{\n .reg .pred p;\n .reg .b64 y;\n setp.eq.u32 p, 0, 0;\n mov.b64 y, {%2, %4};\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}"
                     ::"r"(d), "r"(a_tmem), "r"(b), "r"(idesc), "r"(DESC_HI) : "memory");
    else
        asm volatile("{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n mov.b64 y, {%2, %4};\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}"
                     ::"r"(d), "r"(a_tmem), "r"(b), "r"(idesc), "r"(DESC_HI), "r"(acc) : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t mbar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(mbar) : "memory");
}

// 32 or 64 columns of the warp's 32 lanes, one row a thread: the load and the wait for it, as one statement so that no register
// is moved or spilled in between.
#define REGS8(k, a, i) k(a[i]), k(a[i + 1]), k(a[i + 2]), k(a[i + 3]), k(a[i + 4]), k(a[i + 5]), k(a[i + 6]), k(a[i + 7])
__device__ __forceinline__ void tmem_read32(uint32_t addr, float (&s)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n tcgen05.wait::ld.sync.aligned;"
                 : REGS8("=&f", s, 0), REGS8("=&f", s, 8), REGS8("=&f", s, 16), REGS8("=&f", s, 24)
                 : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_read64(uint32_t addr, float (&s)[2][32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n"
                 " tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
                 "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n tcgen05.wait::ld.sync.aligned;"
                 : REGS8("=&f", s[0], 0), REGS8("=&f", s[0], 8), REGS8("=&f", s[0], 16), REGS8("=&f", s[0], 24),
                   REGS8("=&f", s[1], 0), REGS8("=&f", s[1], 8), REGS8("=&f", s[1], 16), REGS8("=&f", s[1], 24)
                 : "r"(addr), "r"(addr + 32) : "memory");
}
#undef REGS8
// tcgen05.st of 32 columns without the wait for its completion
__device__ __forceinline__ void tmem_put32(uint32_t addr, const uint32_t (&u)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
                 ::"r"(addr), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
                   "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]),
                   "r"(u[16]), "r"(u[17]), "r"(u[18]), "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]),
                   "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]), "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
                 : "memory");
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b)
{
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t x;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(x));
    return x;
}

// The next block of the grid that has not started, which then never will: asked for, its answer (16 bytes) goes to shared
// memory and completes on the barrier.  take_answer: the block's index, -1 when there was none.
__device__ __forceinline__ void ask_for_block(uint32_t answer, uint32_t mbar)
{
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 ::"r"(answer), "r"(mbar) : "memory");
}
__device__ __forceinline__ int take_answer(uint32_t answer)
{
    int x;
    asm volatile("{\n .reg .b128 a;\n .reg .pred p;\n .reg .b32 y, z, u;\n ld.shared.b128 a, [%1];\n mov.b32 %0, -1;\n"
                 " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n"
                 " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, u}, a;\n}"
                 : "=r"(x) : "r"(answer) : "memory");
    return x;
}

// bits a..b (inclusive, any integers) of a mask of several words, word w; PTX shifts of 32 and more give 0
__device__ __forceinline__ uint32_t range_word(int a, int b, int w)
{
    uint32_t x, y;
    asm("shl.b32 %0, %1, %2;" : "=r"(x) : "r"(FULL), "r"(max(a - 32 * w, 0)));
    asm("shr.u32 %0, %1, %2;" : "=r"(y) : "r"(FULL), "r"(max(31 - (b - 32 * w), 0)));
    return x & y;
}

// CLUSTERED: an item's splits are a cluster, one item a CTA.
template <int DIM, bool CLUSTERED>
__global__ void __launch_bounds__(THREADS, 1)
kda_attn_tiles_kernel(const __grid_constant__ AttnArgs p, const AttnPlan plan, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap)
{
    using S = Shape<DIM>;
    constexpr int CB = DIM / 64;                 // 64-column blocks of a row
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *const smem = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t sm_q = base, sm_ring = base + 2 * S::Q, bar = base + S::BAR;
    const uint32_t b_full = bar, b_empty = bar + 8 * S::SLOTS, b_q = b_empty + 8 * S::SLOTS, b_q_free = b_q + 8,
                   b_s = b_q_free + 8, b_p = b_s + 32, b_o = b_p + 32, b_drain = b_o + 32,  // S, P, P V: [half][buffer]
                   b_item = b_drain + 16, b_item_free = b_item + 8 * ITEMS, b_block = b_item_free + 8 * ITEMS, b_near = b_block + 8;
    __shared__ Tile item_ring[ITEMS];
    __shared__ uint32_t tmem_slot;
    __shared__ uint4 block_answer;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    const int g = plan.granule;
    if (tid == 0) {
        for (int i = 0; i < S::SLOTS; i++) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 2);
        }
        for (int h = 0; h < 2; h++) {
            for (int i = 0; i < 2; i++) {
                mbar_init(b_s + 16 * h + 8 * i, 1);
                mbar_init(b_p + 16 * h + 8 * i, 4);
                mbar_init(b_o + 16 * h + 8 * i, 1);
            }
            mbar_init(b_drain + 8 * h, 1);
        }
        mbar_init(b_q, 1);
        mbar_init(b_block, 1);
        mbar_init(b_near, 1);
        mbar_init(b_q_free, 2);
        for (int i = 0; i < ITEMS; i++) {
            mbar_init(b_item + 8 * i, 1);
            mbar_init(b_item_free + 8 * i, 11);      // every warp but the one that writes
        }
        mbar_fence_init();
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    stream_order();
    bool timeout = false, bad = false, joined = false;
    // Waits of a whole warp: every lane polls and the warp votes, so that it stays converged.  (One lane polling for the
    // others let the compiler keep the warp split behind the wait, and everything after it ran twice: 2420 us instead of
    // 1290 at 8192 tokens, 96 heads.)  Once a wait of the warp has given up, the later ones do at once.
    auto wait = [&](uint32_t b, uint32_t parity) -> bool {
        if (__any_sync(FULL, !mbar_wait(b, parity, timeout ? 1 : plan.wait_polls)))
            timeout = true;
        return !timeout;
    };
    // The i-th item of this CTA, read by a whole warp; false when there is none or the wait gave up.
    auto next_item = [&](int i, Tile &w) -> bool {
        const int slot = i % ITEMS;
        if (!wait(b_item + 8 * slot, (i / ITEMS) & 1))
            return false;
        w = item_ring[slot];
        __syncwarp();
        if (lane == 0)
            mbar_arrive(b_item_free + 8 * slot);
        return w.valid != 0;
    };

    if (warp < 8) {
        // ------------------------------------------------------------ softmax, epilogue
        const int h = warp / 4;
        const uint32_t tm_lane = (uint32_t)(warp & 3) << 21;     // the warp's 32 lanes
        const uint32_t tm_s0 = tmem + TM_S + h * 128 + tm_lane, tm_o = tmem + TM_O + h * 128 + tm_lane;
        int ring = 0;                                            // key tiles of the items before
        // Phases of the two S, and of the P V of an item's last two key tiles, the only ones that are waited for as such: a
        // half's S of tile t + 1 is issued right after its P V of tile t - 1.
        uint32_t s_phase = 0, o_phase = 0;
        Tile w, next;
        bool more = next_item(0, w);
        for (int i = 1; more; i++, w = next) {
            const bool mine = tid < w.rows;
            const int r_tok = mine ? token_of(plan, tid) : 0;
            const int tok = w.tok0 + r_tok, head = w.kvh * p.group + (mine ? tid - r_tok * p.group : 0);
            const int pos = mine ? w.pos0 + r_tok : -1;
            const int lo = h ? w.lo[1] : w.lo[0], hi = h ? w.hi[1] : w.hi[0];
            float m = -INFINITY, l = 0.0f;
            bool any = false;
            for (int t = lo; t < hi; t++) {
                const int v0 = t * SUB;
                // the sequence's end inside the step: what lies behind it in its page is cleared from V (K's scores are
                // masked)
                const int end_v = w.len - w.start + w.sink_span - v0;
                if (end_v > 0 && end_v < SUB && (end_v & (g - 1))) {
                    const int it = 2 * (ring + t / 2 - w.t0) + 1, slot = it % S::SLOTS;
                    if (!wait(b_full + 8 * slot, (it / S::SLOTS) & 1))
                        break;
                    const int count = (g - (end_v & (g - 1))) * 8;       // 16-byte vectors of a column block
                    uint4 *v = reinterpret_cast<uint4 *>(smem + 2 * S::Q + slot * S::TILE) + ((t & 1) * SUB + end_v) * 8;
                    for (int i = tid & (HALF - 1); i < count * CB; i += HALF)
                        v[(i / count) * (KEYS * 8) + i % count] = make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                }
                const int buf = t & 1;
                const uint32_t tm_s = tm_s0 + 64 * buf;
                if (!wait(b_s + 16 * h + 8 * buf, s_phase >> buf & 1))
                    break;
                s_phase ^= 1u << buf;
                tc_fence_after();
                // columns of the tile that the row sees: the window's, and the sinks'
                const int wa = max(pos - p.window + 1, w.start) - w.start + w.sink_span - v0;
                const int wb = pos - w.start + w.sink_span - v0, sb = min(p.sinks, pos + 1) - 1 - v0;
                const bool whole = __all_sync(FULL, wa <= 0 && wb >= SUB - 1);
                auto hide = [&](float (&s)[32], int c) {         // 32 columns from 32 c on
                    if (!whole) {
                        const uint32_t mask = range_word(wa, wb, c) | range_word(-v0, sb, c);
#pragma unroll
                        for (int e = 0; e < 32; e++)
                            s[e] = (mask >> e) & 1 ? s[e] : -INFINITY;
                    }
                };
                auto top_of = [&](const float (&s)[32], float x) {
                    float y = s[0];
#pragma unroll
                    for (int e = 1; e < 32; e += 2) {
                        x = e + 1 < 32 ? fmaxf(x, fmaxf(s[e], s[e + 1])) : fmaxf(x, s[e]);
                    }
                    return fmaxf(x, y);
                };
                float s[2][32];
                uint32_t pk[SUB / 2];
                f2 l0, l1;
                for (;;) {
                    const float mu = m == -INFINITY ? 0.0f : m;
                    const f2 sc = f2_pack(p.scale_log2, p.scale_log2), mm = f2_pack(-mu, -mu);
                    float top = -INFINITY;
                    l0 = l1 = 0;
                    tmem_read64(tm_s, s);
#pragma unroll
                    for (int c = 0; c < SUB / 32; c++) {
                        hide(s[c & 1], c);
                        top = top_of(s[c & 1], top);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const f2 y = f2_fma(f2_pack(s[c & 1][e], s[c & 1][e + 1]), sc, mm);
                            const float a = ex2_approx(f2_lo(y)), b = ex2_approx(f2_hi(y));
                            if (e & 2)
                                l1 = f2_add(l1, f2_pack(a, b));
                            else
                                l0 = f2_add(l0, f2_pack(a, b));
                            // bf16, V's type, as the product takes it: 2^-9 of each P, which leaves the output 2.3e-3 off
                            // (norm) where its own rounding alone leaves 1.6e-3; the sum l is of what P was before
                            const __nv_bfloat162 z = __floats2bfloat162_rn(a, b);
                            pk[16 * c + e / 2] = *reinterpret_cast<const uint32_t *>(&z);
                        }
                    }
                    top *= p.scale_log2;
                    if (m == -INFINITY && fabsf(top) <= RESCALE_AT)
                        m = 0.0f;                                // the row's first keys: what P was formed with will do
                    const bool move = top > m + RESCALE_AT;
                    if (!__any_sync(FULL, move))
                        break;
                    const float a = move ? ex2_approx(m - top) : 1.0f;
                    if (move)
                        m = top;
                    l *= a;
                    if (any) {
                        // the P V before this one has to be through (the ones before it are: this S came after them)
                        const uint32_t other = buf ^ 1;
                        if (!wait(t + 1 < hi ? b_s + 16 * h + 8 * other : b_o + 16 * h + 8 * other,
                                  (t + 1 < hi ? s_phase : o_phase) >> other & 1))
                            break;
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < DIM; c += 32) {
                            float o[32];
                            tmem_read32(tm_o + c, o);
                            uint32_t u[32];
#pragma unroll
                            for (int e = 0; e < 32; e++)
                                u[e] = __float_as_uint(o[e] * a);
                            tmem_put32(tm_o + c, u);
                        }
                    }
                }
                any = true;
                l0 = f2_add(l0, l1);
                l += f2_lo(l0) + f2_hi(l0);
                tmem_put32(tm_s, pk);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(b_p + 16 * h + 8 * buf);
            }
            if (timeout)
                break;
            ring += w.t1 - w.t0;
            // The last P V: those before it are through with it.
            auto last_pv = [&]() -> bool {
                if (any) {
                    const int last_buf = (hi - 1) & 1;
                    o_phase ^= hi - lo > 1 ? 3 : 1u << last_buf;
                    if (!wait(b_o + 16 * h + 8 * last_buf, (o_phase >> last_buf & 1) ^ 1))
                        return false;
                    tc_fence_after();
                }
                return true;
            };
            // A cluster's CTA `split` finishes rows split * per .. of the item; the others send it their O, maximum and sum.
            // They go where its ring and its Q were: every warp of the cluster is through with those at the first barrier.
            const int per = CLUSTERED ? ATTN_ROWS / plan.splits : ATTN_ROWS, owner = tid / per, row = tid % per;
            float own = 1.0f, M = 0.0f;                          // weight of this split's O (below 0: none)
            if constexpr (CLUSTERED) {
                if (!last_pv())
                    break;
                cluster_sync();
                if (owner != w.split) {
                    const int sender = w.split - (w.split > owner);
                    const uint32_t to = in_cta(sm_ring + (sender * (DIM / 4) * per + row) * 16, owner);
                    if (any)
#pragma unroll
                        for (int c = 0; c < DIM; c += 32) {
                            float o[32];
                            tmem_read32(tm_o + c, o);
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                store_cluster(to + (c + e) / 4 * per * 16, make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]));
                        }
                    store_cluster(in_cta(sm_q + (sender * per + row) * 8, owner), make_float2(m, l));
                }
                tc_fence_before();
                cluster_sync();
                joined = true;
                if (owner != w.split)
                    break;
                const float2 *st = reinterpret_cast<const float2 *>(smem) + row;
                const float mine_m = m, mine_l = l;
                for (int i = 0; i < plan.splits - 1; i++)
                    m = fmaxf(m, st[i * per].x);
                M = m == -INFINITY ? 0.0f : m;
                own = mine_m == -INFINITY && mine_l == 0.0f ? -1.0f : ex2_approx(mine_m - M);
                l = own < 0.0f ? 0.0f : own * mine_l;
                for (int i = 0; i < plan.splits - 1; i++) {
                    const float2 x = st[i * per];
                    if (!(x.x == -INFINITY && x.y == 0.0f))
                        l += ex2_approx(x.x - M) * x.y;
                }
            }
            // What of the epilogue needs no O, and the next item, while the last P V runs.
            const int at = mine ? tok * p.hq + head : -1;
            const bool part = !CLUSTERED && plan.splits > 1;
            const float inv = part ? 1.0f : (l == 0.0f ? 0.0f : 1.0f / l);
            const bool blank = __any_sync(FULL, l == 0.0f && !part);         // rows that see nothing: 0
            int out_row[8];                                      // of the rows this lane takes out
#pragma unroll
            for (int k = 0; k < 8; k++)
                out_row[k] = __shfl_sync(FULL, at, 4 * k + lane / 8);
            if (mine && part)
                plan.part_ml[w.split * plan.rows + at] = make_float2(m, l);
            else if (mine && p.lse)
                p.lse[at] = l == 0.0f ? -INFINITY : LN2 * (m + log2f(l));
            more = !CLUSTERED && next_item(i, next);
            if (!CLUSTERED && !last_pv())
                break;
            // Epilogue: the row's thread scales it; 128 bytes of each row at a time go through shared memory (16-byte
            // chunks, swizzled) and out with eight lanes to a row.  (Stored straight by its thread, a row took a line of L1
            // for every 16 bytes: 148 us for ragged 8192 tokens with window 512.)
            const f2 inv2 = f2_pack(inv, inv);
            f2 z0 = 0, z1 = 0;                                   // stay 0 while the row is finite
            unsigned char *const stage = smem + S::OUT + warp * S::STAGE;
            auto put = [&](int chunk, const uint4 &x) {
                *reinterpret_cast<uint4 *>(stage + lane * 128 + ((chunk ^ (lane & 7)) << 4)) = x;
            };
            auto flush = [&](unsigned char *to, int64_t row_bytes) {
                __syncwarp();
                uint4 x[8];
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const int r = 4 * k + lane / 8;
                    x[k] = *reinterpret_cast<const uint4 *>(stage + r * 128 + ((lane % 8 ^ (r & 7)) << 4));
                }
#pragma unroll
                for (int k = 0; k < 8; k++)
                    if (out_row[k] >= 0)
                        *reinterpret_cast<uint4 *>(to + out_row[k] * row_bytes + lane % 8 * 16) = x[k];
                __syncwarp();
            };
#pragma unroll
            for (int c = 0; c < DIM; c += 64) {
                float o[2][32];
                if (any) {
                    tmem_read64(tm_o + c, o);
                } else {
#pragma unroll
                    for (int e = 0; e < 64; e++)
                        o[e / 32][e % 32] = 0.0f;
                }
                if constexpr (CLUSTERED) {
#pragma unroll
                    for (int e = 0; e < 64; e++)
                        o[e / 32][e % 32] = own < 0.0f ? 0.0f : own * o[e / 32][e % 32];
                    for (int i = 0; i < plan.splits - 1; i++) {
                        const float2 x = reinterpret_cast<const float2 *>(smem)[i * per + row];
                        if (x.x == -INFINITY && x.y == 0.0f)     // saw nothing; nor is there an O
                            continue;
                        const float a = ex2_approx(x.x - M);
                        const float4 *y = reinterpret_cast<const float4 *>(smem + 2 * S::Q) + (i * (DIM / 4) + c / 4) * per + row;
#pragma unroll
                        for (int e = 0; e < 64; e += 4) {
                            const float4 z = y[e / 4 * per];
                            float *t = &o[e / 32][e % 32];
                            t[0] = fmaf(a, z.x, t[0]), t[1] = fmaf(a, z.y, t[1]), t[2] = fmaf(a, z.z, t[2]), t[3] = fmaf(a, z.w, t[3]);
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    float &x = o[e / 32][e % 32], &y = o[e / 32][e % 32 + 1];
                    const f2 xy = f2_pack(x, y), q = f2_mul(xy, inv2);
                    if (e & 2)
                        z1 = f2_fma(xy, 0, z1);
                    else
                        z0 = f2_fma(xy, 0, z0);
                    x = f2_lo(q), y = f2_hi(q);
                }
                if (part) {
#pragma unroll
                    for (int i = 0; i < 2; i++) {
#pragma unroll
                        for (int e = 0; e < 8; e++)
                            put(e, make_uint4(__float_as_uint(o[i][4 * e]), __float_as_uint(o[i][4 * e + 1]),
                                              __float_as_uint(o[i][4 * e + 2]), __float_as_uint(o[i][4 * e + 3])));
                        flush(reinterpret_cast<unsigned char *>(plan.part_o + w.split * plan.rows * DIM + c + 32 * i), DIM * 4);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        uint32_t y[4];
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const int i = 8 * e + 2 * j;
                            const __nv_bfloat162 b2 = __floats2bfloat162_rn(o[i / 32][i % 32], o[i / 32][i % 32 + 1]);
                            y[j] = *reinterpret_cast<const uint32_t *>(&b2);
                        }
                        if (blank && l == 0.0f)
                            y[0] = y[1] = y[2] = y[3] = 0;
                        put(e, make_uint4(y[0], y[1], y[2], y[3]));
                    }
                    flush(reinterpret_cast<unsigned char *>(p.out + c), DIM * 2);
                }
            }
            z0 = f2_add(z0, z1);
            const bool finite = f2_lo(z0) + f2_hi(z0) == 0.0f;
            tc_fence_before();                // O is read before the next item's first P lets it be overwritten
            const unsigned again = __ballot_sync(FULL, mine && !finite && l > 0.0f && l <= FLT_MAX && !part);
            if (again)
                bad |= attn_mend_rows<DIM>(p, w.n, again, tok, head, pos, plan.margin);
        }
    } else if (warp == 8) {
        // ------------------------------------------------------------ copies
        const int ng = KEYS / g;
        int issued = 0;
        Tile w;
        for (int i = 0; !timeout && next_item(i, w); i++) {
            if (w.t0 == w.t1 && lane == 0)
                mbar_arrive(b_near);
            for (int t = w.t0; t < w.t1 && !timeout; t++) {
                if (t == w.t1 - 1 && lane == 0)
                    mbar_arrive(b_near);                 // time to look for the next item
                int y = OUTSIDE;
                if (lane < ng) {
                    const int v = t * KEYS + lane * g, j = virt_pos(w, v);
                    if (v < w.virt && j < w.len) {
                        const int32_t id = p.cache.table[(int64_t)w.n * p.cache.max_pages + (j >> p.cache.page_shift)];
                        if (id >= 0 && id < p.cache.pages)
                            y = (int)((((int64_t)id * p.cache.hkv + w.kvh) << p.cache.page_shift) + (j & ((1 << p.cache.page_shift) - 1)));
                        else
                            bad = true;
                    }
                }
#pragma unroll
                for (int kv = 0; kv < 2; kv++) {
                    const int slot = issued % S::SLOTS;
                    if (issued >= S::SLOTS && !wait(b_empty + 8 * slot, (issued / S::SLOTS - 1) & 1))
                        break;
                    if (lane == 0)
                        mbar_expect_tx(b_full + 8 * slot, S::TILE);
                    __syncwarp();
                    if (lane < ng) {
#pragma unroll
                        for (int cb = 0; cb < CB; cb++)
                            tma_load_2d(sm_ring + slot * S::TILE + cb * (KEYS * 128) + lane * g * 128, kv ? &vmap : &kmap,
                                        cb * 64, y, b_full + 8 * slot);
                    }
                    issued++;
                }
            }
        }
        // no copy is in flight when the CTA leaves, also where the work was given up
        for (int it = max(issued - S::SLOTS, 0); it < issued; it++)
            timeout |= !mbar_wait(b_full + 8 * (it % S::SLOTS), (it / S::SLOTS) & 1);
    } else if (warp == 9 || warp == 10) {
        // ------------------------------------------------------------ tensor-core issue, warp 9 for half 0, 10 for half 1
        // The warp walks the items and waits; one elected lane issues.  What an instruction needs (descriptors, addresses) is
        // the same in all lanes and known to be, so that it is formed in uniform registers: issuing from one thread's own
        // registers took some 80 cycles a product.  Once a wait has given up, nothing more is issued.
        const int h = __shfl_sync(FULL, warp, 0) - 9;
        const uint32_t id_s = idesc_bf16(HALF, SUB, false), id_o = idesc_bf16(HALF, DIM, true);
        const uint32_t tm = __shfl_sync(FULL, tmem, 0), lead = elect_one();
        const uint32_t q_lo = desc_lo(sm_q + h * (HALF * 128), 16), k_lo = desc_lo(sm_ring, 16), v_lo = desc_lo(sm_ring, KEYS * 128);
        uint32_t p_phase = 0, q_phase = 0;
        uint32_t ks = 0, kp = 0, vs = 1, vp = 0;                 // next K's and next V's slot, and its phase
        Tile w;
        for (int i = 0; next_item(i, w); i++) {
            const int t0 = w.t0, t1 = w.t1, lo = h ? w.lo[1] : w.lo[0], hi = h ? w.hi[1] : w.hi[0];
            // Every item has a Q, also one whose rows see nothing and one without a step for this half: only when it is there
            // do the halves hand its place back, so that neither the place nor the barrier is taken again under a copy.
            wait(b_q, q_phase);
            q_phase ^= 1;
            // step by step P V of key tile t - 1, then S of tile t into the buffer that P came from
            for (int t = t0; t <= t1; t++) {
                const bool pv = t > t0, sk = t < t1;
                if (pv)
                    wait(b_full + 8 * vs, vp);
#pragma unroll
                for (int buf = 0; buf < 2; buf++) {
                    const int now = 2 * t + buf, old = now - 2;
                    if (pv && old >= lo && old < hi) {
                        wait(b_p + 16 * h + 8 * buf, p_phase >> buf & 1);
                        p_phase ^= 1u << buf;
                        tc_fence_after();
                        const uint32_t b = v_lo + vs * (S::TILE >> 4) + buf * (SUB * 128 >> 4), d = tm + TM_O + h * 128;
                        const uint32_t a = tm + TM_S + h * 128 + 64 * buf;
                        if (lead && !timeout) {
                            mma_ts<false>(d, a, b, id_o, old > lo);
#pragma unroll
                            for (int k = 1; k < SUB / 16; k++)
                                mma_ts<true>(d, a + k * 8, b + k * (2048 >> 4), id_o, 1);
                            if (old + 2 >= hi)
                                umma_commit(b_o + 16 * h + 8 * buf);
                        }
                        __syncwarp();
                    }
                    if (sk && buf == 0)
                        wait(b_full + 8 * ks, kp);
                    if (sk && now >= lo && now < hi) {
                        tc_fence_after();
                        const uint32_t b = k_lo + ks * (S::TILE >> 4) + buf * (SUB * 128 >> 4), d = tm + TM_S + h * 128 + 64 * buf;
                        if (lead && !timeout) {
                            mma_ss<false>(d, q_lo, b, id_s, 0);
#pragma unroll
                            for (int k = 1; k < DIM / 16; k++)
                                mma_ss<true>(d, q_lo + (((k / 4) * (2 * HALF * 128) + (k % 4) * 32) >> 4),
                                             b + (((k / 4) * (KEYS * 128) + (k % 4) * 32) >> 4), id_s, 1);
                            umma_commit(b_s + 16 * h + 8 * buf);
                        }
                        __syncwarp();
                    }
                }
                if (lead && !timeout) {                          // this half is through with V of t - 1 and K of t
                    if (pv)
                        umma_commit(b_empty + 8 * vs);
                    if (sk)
                        umma_commit(b_empty + 8 * ks);
                    if (t == max(t1 - 1, t0))
                        umma_commit(b_q_free);                   // and with Q
                }
                __syncwarp();
                if (pv && (vs += 2) >= S::SLOTS)
                    vs -= S::SLOTS, vp ^= 1;
                if (sk && (ks += 2) >= S::SLOTS)
                    ks -= S::SLOTS, kp ^= 1;
            }
        }
        if (lead) {
            // everything issued has to be through before tensor memory is freed
            umma_commit(b_drain + 8 * h);
            timeout |= !mbar_wait(b_drain + 8 * h, 0);
        }
        __syncwarp();
    } else if (warp == 11) {
        // ------------------------------------------------------------ items and their Q
        // The CTA's own block first, then blocks of the grid that have not started, one when the last key tile of an item is
        // being brought in: CTAs with less to do take more.  Blocks past a ragged batch's items are taken too, so that no CTA
        // starts for them.  (Items dealt out beforehand, 152 apart: 1286 and 121 us for the two calls above, and as much as
        // 133 us in another order; taken an item ahead: 1275 and 121 us.)
        int loaded = 0, x = blockIdx.x;
        uint32_t asked = 0, answers = 0;
        const uint32_t answer = smem_u32(&block_answer);
        auto next_block = [&]() -> int {
            if (lane == 0) {
                fence_async_smem();                      // the last answer has been read
                mbar_expect_tx(b_block, 16);
                ask_for_block(answer, b_block);
            }
            asked++;
            __syncwarp();
            if (!wait(b_block, answers & 1))
                return -1;
            answers++;
            const int y = take_answer(answer);
            __syncwarp();
            return y;
        };
        for (int i = 0;; i++) {
            const int slot = i % ITEMS;
            Tile w;
            w.valid = 0;
            if (i > 0)
                x = !CLUSTERED && wait(b_near, (i - 1) & 1) ? next_block() : -1;
            while (x >= 0) {
                find_tile(p, plan, x, w, bad);
                if (w.valid)
                    break;
                x = CLUSTERED ? -1 : next_block();
            }
            if (i >= ITEMS && !wait(b_item_free + 8 * slot, (i / ITEMS - 1) & 1))
                break;
            if (lane == 0) {
                item_ring[slot] = w;
                mbar_arrive(b_item + 8 * slot);
            }
            if (!w.valid)
                break;
            // Q is free when both halves' last S of the item before is formed
            if (i > 0 && !wait(b_q_free, (i - 1) & 1))
                break;
            if (lane == 0) {
                mbar_expect_tx(b_q, (uint32_t)(CB * 128 * plan.run * p.group));
#pragma unroll
                for (int cb = 0; cb < CB; cb++)
                    tma_load_3d(sm_q + cb * (2 * HALF * 128), &qmap, cb * 64, w.kvh * p.group, w.tok0, b_q);
            }
            loaded++;
        }
        if (loaded > 0)                              // no copy is in flight when the CTA leaves
            timeout |= !mbar_wait(b_q, (loaded - 1) & 1);
        if (asked > answers)
            timeout |= !mbar_wait(b_block, answers & 1);
    }
    if (CLUSTERED && !joined) {                      // the other warps, CTAs without an item, and those that gave up
        cluster_sync();
        cluster_sync();
    }
    report(p.err, bad, DEVERR_CU_SEQLENS);
    report(p.err, timeout, DEVERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 9)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS));
}

// ---------------------------------------------------------------- host
typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encode_fn(EncodeTiled *fn)
{
    static std::atomic<void *> cached;
    void *f = cached.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
        if (e != cudaSuccess)
            return e;
        if (found != cudaDriverEntryPointSuccess || !f)
            return cudaErrorNotSupported;
        cached.store(f, std::memory_order_release);
    }
    *fn = reinterpret_cast<EncodeTiled>(f);
    return cudaSuccess;
}

// Q as [tokens][hq][dim]; a box is 64 columns of an item's tokens and heads.
cudaError_t query_map(CUtensorMap *map, const AttnArgs &p, const AttnPlan &plan)
{
    EncodeTiled fn;
    const cudaError_t e = encode_fn(&fn);
    if (e != cudaSuccess)
        return e;
    const cuuint64_t dims[3] = {(cuuint64_t)p.cache.dim, (cuuint64_t)p.hq, (cuuint64_t)(plan.rows / p.hq)};
    const cuuint64_t strides[2] = {(cuuint64_t)p.cache.dim * 2, (cuuint64_t)p.q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)plan.run}, step[3] = {1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16 *>(p.q), dims, strides, box, step,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int DIM, bool CLUSTERED> cudaError_t launch_tiles(const AttnArgs &p, const AttnPlan &plan, cudaStream_t st)
{
    static std::atomic<uint64_t> ready;      // devices whose kernel attribute is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(ready.load() >> dev & 1)) {
        e = cudaFuncSetAttribute(kda_attn_tiles_kernel<DIM, CLUSTERED>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<DIM>::SMEM);
        if (e == cudaSuccess)
            ready.fetch_or(1ull << dev);
    }
    CUtensorMap kmap, vmap, qmap;
    if (e == cudaSuccess)
        e = cache_map(&kmap, p.cache.k, p.cache, plan.granule);
    if (e == cudaSuccess)
        e = cache_map(&vmap, p.cache.v, p.cache, plan.granule);
    if (e == cudaSuccess)
        e = query_map(&qmap, p, plan);
    if (e != cudaSuccess)
        return e;
    if (plan.items < 1)
        return cudaErrorInvalidValue;
    return launch_in_row(kda_attn_tiles_kernel<DIM, CLUSTERED>, plan.items, THREADS, Shape<DIM>::SMEM, CLUSTERED ? plan.splits : 1,
                         st, p, plan, kmap, vmap, qmap);
}

}  // namespace

// The cache as a matrix of rows [pages * hkv * page][dim]; a box is 64 columns of `rows` rows.
cudaError_t cache_map(CUtensorMap *map, const void *ptr, const PagedCache &c, int rows)
{
    EncodeTiled fn;
    const cudaError_t e = encode_fn(&fn);
    if (e != cudaSuccess)
        return e;
    const int page = 1 << c.page_shift;
    const cuuint64_t dims[2] = {(cuuint64_t)c.dim, (cuuint64_t)c.pages * c.hkv * page};
    const cuuint64_t strides[1] = {(cuuint64_t)c.dim * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)rows}, step[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box, step,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_attn_tiles(const AttnArgs &p, const AttnPlan &plan, cudaStream_t st)
{
    if (plan.cluster)
        return p.cache.dim == 128 ? launch_tiles<128, true>(p, plan, st) : launch_tiles<64, true>(p, plan, st);
    return p.cache.dim == 128 ? launch_tiles<128, false>(p, plan, st) : launch_tiles<64, false>(p, plan, st);
}

}  // namespace kda
