// Windowed attention over the paged cache for few query rows: 16 (tokens x heads of a key head's group) a CTA.
//
// A decode step reads every visible key and value once for a handful of rows: the floor is the cache's bytes at the
// memory's rate, and the arithmetic (16 rows wide on mma.sync) has to stay out of the way.  One CTA takes a (sequence, key
// head) or a split of its keys; each of its 4 or 8 warps works by itself on blocks of 16 keys, every 4th or 8th one, that its lane 0
// brings in with bulk tensor copies into the warp's own ring of shared memory: no barrier of the CTA in the loop, and
// RING x 8 KB in flight a warp.  The warps' results (running maximum, sum, O in fp32) are joined once at the end in shared
// memory.  Up to 8 splits are a cluster, which joins its CTAs' results over distributed shared memory in the same
// launch; more go through memory and the join kernel.  Small calls with more rows are tiles of 16 rows, one a CTA.
//
// Measured: 256 sequences, 64 heads over 8, window 1024 and 16 sinks (1.10 GB), 164 us, 6.70 TB/s, 99% of the measured copy
// rate (the tile kernel: 255 us).  One sequence, 32 heads over 8, window 4096: 8.9 us, a chain of latencies (lengths, page
// table, copies, four blocks a warp, the joins); the CTAs of a cluster send each row's parts to the CTA that finishes it,
// which takes one barrier (2 us less than one CTA that reads the others' parts between two barriers, or than 32 splits with
// a join kernel).
//
// Keys come as in the tile kernel: the sinks' granules, then the window's, 16 positions each, which lie in one page.
// Values that no row of the CTA sees are cleared in shared memory; where the rows differ in what they see (several
// tokens), an output row that does not come out finite is taken again from the definition.
#include "kda_attn.cuh"

#include <atomic>
#include <cfloat>

namespace kda {
namespace {

constexpr int KEYS = DECODE_KEYS, ROWS = DECODE_ROWS, CLUSTER = ATTN_CLUSTER;
constexpr float RESCALE_AT = 8.0f;           // base-2 growth of a maximum that moves it
constexpr unsigned FULL = 0xffffffffu;

// WARPS: 4, two CTAs an SM; 8, one CTA an SM, for calls of fewer CTAs than SMs.
template <int DIM, int WARPS> struct Shape {
    static constexpr int RING = DIM == 128 ? 3 : 6;              // blocks in flight a warp
    static constexpr int BLOCK = KEYS * DIM * 2;                 // bytes of K, and of V
    static constexpr int WARP = RING * 2 * BLOCK;                // a warp's ring
    static constexpr int RECV = WARPS * WARP;                    // what a cluster's CTAs send: ROWS rows of DIM floats
    static constexpr int SMEM = 1024 + RECV + ROWS * DIM * 4;
    static_assert(WARP >= ROWS * DIM * 4, "O of a warp goes where its ring was");
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16-byte chunk c of key `key` in a block of 64-column pieces, 128-byte swizzle
__device__ __forceinline__ uint32_t chunk_at(uint32_t block, int key, int c)
{
    return block + (c / 8) * (KEYS * 128) + key * 128 + (((c & 7) ^ (key & 7)) << 4);
}
// Joins N results (maximum, sum) of a row: their weights, and the row's maximum and sum.  A result without a visible key has
// maximum -inf and sum 0; NaN scores leave a NaN sum.
template <int N> __device__ __forceinline__ void join_stats(const float2 (&st)[N], float (&w)[N], float &M, float &L)
{
    M = -INFINITY;
    L = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++)
        M = fmaxf(M, st[i].x);
    const float mu = M == -INFINITY ? 0.0f : M;
#pragma unroll
    for (int i = 0; i < N; i++) {
        const bool none = st[i].x == -INFINITY && st[i].y == 0.0f;
        w[i] = none ? -1.0f : ex2_approx((st[i].x == -INFINITY ? 0.0f : st[i].x) - mu);
        if (!none)
            L += w[i] * st[i].y;
    }
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&x);
}

template <int DIM, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 8 / WARPS)
kda_attn_decode_kernel(const __grid_constant__ AttnArgs p, const AttnPlan plan, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap)
{
    using S = Shape<DIM, WARPS>;
    constexpr int CB = DIM / 64, KS = DIM / 16, NT = DIM / 8;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t bars[WARPS * S::RING];
    __shared__ float2 stats[WARPS][ROWS], recv_stats[ROWS], recv_failed[CLUSTER];
    if (plan.cluster)                                            // waited for before anything is sent: every CTA has begun
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    if (threadIdx.x == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
    }
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *const smem = smem_raw + (base - smem_u32(smem_raw));
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31, g = lane / 4, t = lane % 4;

    int x = blockIdx.x;
    const int split = x % plan.splits;                           // the splits of an item are neighbours: a cluster
    x /= plan.splits;
    const int row0 = x % plan.row_tiles * ROWS;                  // first of the CTA's rows among those of its key head
    x /= plan.row_tiles;
    const int kvh = x % p.cache.hkv, n = x / p.cache.hkv;
    const int tokens = (int)p.tok.T, rows = min(tokens * p.group - row0, ROWS);
    bool bad = false, timeout = false;
    const uint32_t ring = base + warp * S::WARP, bar = smem_u32(bars + warp * S::RING);
    if (lane == 0) {
        for (int i = 0; i < S::RING; i++)
            mbar_init(bar + 8 * i, 1);
        mbar_fence_init();
    }
    __syncwarp();
    stream_order();
    // Q as the first operand: rows g and g + 8; on its way while the lengths and the page table are read
    uint32_t q[KS][4];
#pragma unroll
    for (int r = 0; r < 2; r++) {
        const int row = g + 8 * r;
        const bool in = row < rows;
        const int tok = in ? (row0 + row) / p.group : 0;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(
            p.q + (int64_t)(n * tokens + tok) * p.q_stride + (kvh * p.group + (in ? (row0 + row) % p.group : 0)) * DIM);
#pragma unroll
        for (int k = 0; k < KS; k++) {
            q[k][r] = in ? src[8 * k + t] : 0;
            q[k][2 + r] = in ? src[8 * k + 4 + t] : 0;
        }
    }
    const int len = (int)cache_len(p.cache, n, bad);
    // positions of the first and the last row's tokens
    const int p0 = len - tokens + row0 / p.group, p1 = len - tokens + (row0 + rows - 1) / p.group;
    int pos[2];
#pragma unroll
    for (int r = 0; r < 2; r++)
        pos[r] = g + 8 * r < rows ? len - tokens + (row0 + g + 8 * r) / p.group : -1;
    // virtual keys: the sinks' granules, then the window's
    int sink = 0, start = 0, virt = 0;
    if (p1 >= 0) {
        start = max(p0 - p.window + 1, 0) & -KEYS;
        sink = (p.sinks + KEYS - 1) & -KEYS;
        if (start <= sink)
            sink = start = 0;
        virt = sink + (p1 + 1 - start);
    }
    const int blocks = (virt + KEYS - 1) / KEYS;
    const int b0 = (int)((int64_t)blocks * split / plan.splits), b1 = (int)((int64_t)blocks * (split + 1) / plan.splits);
    auto position = [&](int b) { return b * KEYS < sink ? b * KEYS : b * KEYS - sink + start; };

    const int mine = b1 - b0 > warp ? (b1 - b0 - warp + WARPS - 1) / WARPS : 0;      // blocks b0 + warp + WARPS i
    auto fetch = [&](int i) {                                    // by lane 0
        const int j = position(b0 + warp + WARPS * i);
        int y = OUTSIDE;
        const int32_t id = p.cache.table[(int64_t)n * p.cache.max_pages + (j >> p.cache.page_shift)];
        if (id >= 0 && id < p.cache.pages)
            y = (int)((((int64_t)id * p.cache.hkv + kvh) << p.cache.page_shift) + (j & ((1 << p.cache.page_shift) - 1)));
        else
            bad = true;
        const uint32_t at = ring + (i % S::RING) * 2 * S::BLOCK, b = bar + 8 * (i % S::RING);
        mbar_expect_tx(b, 2 * S::BLOCK);
#pragma unroll
        for (int c = 0; c < CB; c++) {
            tma_load_2d(at + c * KEYS * 128, &kmap, c * 64, y, b);
            tma_load_2d(at + S::BLOCK + c * KEYS * 128, &vmap, c * 64, y, b);
        }
    };
    if (lane == 0)
        for (int i = 0; i < S::RING && i < mine; i++)
            fetch(i);

    float o[NT][4];
#pragma unroll
    for (int c = 0; c < NT; c++)
        o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    int done = 0;
    for (int i = 0; i < mine; i++) {
        const int slot = i % S::RING, j0 = position(b0 + warp + WARPS * i);
        const uint32_t kb = ring + slot * 2 * S::BLOCK, vb = kb + S::BLOCK;
        if (!mbar_wait(bar + 8 * slot, (i / S::RING) & 1, plan.wait_polls))
            timeout = true;
        if (__any_sync(FULL, timeout)) {
            timeout = true;
            break;
        }
        done = i + 1;
        // S: keys j0 .. j0 + 15 as two tiles of 8
        float s[2][4] = {};
#pragma unroll
        for (int k = 0; k < KS; k++) {
            uint32_t b[4];
            ldsm_x4(chunk_at(kb, (lane / 16) * 8 + lane % 8, 2 * k + (lane / 8) % 2), b);
            mma_bf16(s[0], q[k], b[0], b[1]);
            mma_bf16(s[1], q[k], b[2], b[3]);
        }
        // whole: every row sees every key of the block
        const bool whole = j0 + KEYS - 1 <= p0 && j0 > p1 - p.window;
        if (!whole) {
#pragma unroll
            for (int c = 0; c < 2; c++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int j = j0 + 8 * c + 2 * t + (e & 1), at = pos[e / 2];
                    s[c][e] = j <= at && (j > at - p.window || j < p.sinks) ? s[c][e] : -INFINITY;
                }
            // values that no row sees
            for (int v = lane; v < KEYS * (DIM / 8); v += 32) {
                const int key = v % KEYS, j = j0 + key;
                if (j > p1 || (j <= p0 - p.window && j >= p.sinks)) {
                    const uint32_t z = chunk_at(vb, key, v / KEYS);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(z), "r"(0) : "memory");
                }
            }
            fence_async_smem();                                  // the slot's next copy comes after these
            __syncwarp();
        }
        float top[2];
#pragma unroll
        for (int r = 0; r < 2; r++) {
            top[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
            top[r] = fmaxf(top[r], __shfl_xor_sync(FULL, top[r], 1));
            top[r] = fmaxf(top[r], __shfl_xor_sync(FULL, top[r], 2)) * p.scale_log2;
        }
        const bool move0 = top[0] > m[0] + RESCALE_AT, move1 = top[1] > m[1] + RESCALE_AT;
        if (__any_sync(FULL, move0 || move1)) {                  // also the first block with a visible key
            const float a0 = move0 ? ex2_approx(m[0] - top[0]) : 1.0f, a1 = move1 ? ex2_approx(m[1] - top[1]) : 1.0f;
            m[0] = move0 ? top[0] : m[0];
            m[1] = move1 ? top[1] : m[1];
            l[0] *= a0;
            l[1] *= a1;
#pragma unroll
            for (int c = 0; c < NT; c++) {
                o[c][0] *= a0, o[c][1] *= a0;
                o[c][2] *= a1, o[c][3] *= a1;
            }
        }
        const float mu0 = m[0] == -INFINITY ? 0.0f : m[0], mu1 = m[1] == -INFINITY ? 0.0f : m[1];
#pragma unroll
        for (int c = 0; c < 2; c++) {
            s[c][0] = ex2_approx(fmaf(s[c][0], p.scale_log2, -mu0));
            s[c][1] = ex2_approx(fmaf(s[c][1], p.scale_log2, -mu0));
            s[c][2] = ex2_approx(fmaf(s[c][2], p.scale_log2, -mu1));
            s[c][3] = ex2_approx(fmaf(s[c][3], p.scale_log2, -mu1));
            l[0] += s[c][0] + s[c][1];
            l[1] += s[c][2] + s[c][3];
        }
        // P in bf16, V's type, as the product takes it: 2^-9 of each, which leaves the output 2.3e-3 off (norm) where its own
        // rounding alone leaves 1.65e-3; the sum l is of what P was before
        const uint32_t a[4] = {pack_bf16(s[0][0], s[0][1]), pack_bf16(s[0][2], s[0][3]), pack_bf16(s[1][0], s[1][1]),
                               pack_bf16(s[1][2], s[1][3])};
#pragma unroll
        for (int c = 0; c < NT; c += 2) {
            uint32_t b[4];
            ldsm_x4_t(chunk_at(vb, ((lane / 8) % 2) * 8 + lane % 8, c + lane / 16), b);
            mma_bf16(o[c], a, b[0], b[1]);
            mma_bf16(o[c + 1], a, b[2], b[3]);
        }
        __syncwarp();                                            // all lanes are through with the slot
        if (lane == 0 && i + S::RING < mine)
            fetch(i + S::RING);
    }
    // no copy is in flight when the work was given up
    for (int i = done; i < mine && i < done + S::RING; i++)
        timeout |= !mbar_wait(bar + 8 * (i % S::RING), (i / S::RING) & 1);
    __syncwarp();

    // the warps' results: O where the warp's ring was, row-major
#pragma unroll
    for (int r = 0; r < 2; r++) {
        l[r] += __shfl_xor_sync(FULL, l[r], 1);
        l[r] += __shfl_xor_sync(FULL, l[r], 2);
        if (t == 0)
            stats[warp][g + 8 * r] = make_float2(m[r], l[r]);
    }
    float *const part = reinterpret_cast<float *>(smem + warp * S::WARP);
#pragma unroll
    for (int c = 0; c < NT; c++)
#pragma unroll
        for (int r = 0; r < 2; r++)
            *reinterpret_cast<float2 *>(part + (g + 8 * r) * DIM + ((8 * c + 2 * t) ^ (8 * (g & 3)))) = make_float2(o[c][2 * r], o[c][2 * r + 1]);
    // a row's place in the batch, and its last step: the result, or the split's part of it
    constexpr int PIECES = DIM / 64;                             // float2's a lane has of a row
    auto finish = [&](int row, float M, float L, const float2 (&y)[PIECES], bool whole) {
        const int tok = (row0 + row) / p.group, head = kvh * p.group + (row0 + row) % p.group;
        const int64_t at = (int64_t)(n * tokens + tok) * p.hq + head;
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        bool finite = true;
#pragma unroll
        for (int c = 0; c < PIECES; c++) {
            const int e = 64 * c + 2 * lane;
            finite &= fabsf(y[c].x) <= FLT_MAX && fabsf(y[c].y) <= FLT_MAX;
            if (whole)
                *reinterpret_cast<uint32_t *>(p.out + at * DIM + e) = L == 0.0f ? 0u : pack_bf16(y[c].x * inv, y[c].y * inv);
            else
                *reinterpret_cast<float2 *>(plan.part_o + (split * plan.rows + at) * DIM + e) = y[c];
        }
        if (lane == 0) {
            if (!whole)
                plan.part_ml[split * plan.rows + at] = make_float2(M, L);
            else if (p.lse)
                p.lse[at] = L == 0.0f ? -INFINITY : LN2 * (M + log2f(L));
        }
        if (whole && L > 0.0f && L <= FLT_MAX && __any_sync(FULL, !finite))
            bad |= attn_mend_rows<DIM>(p, n, 1, n * tokens + tok, head, len - tokens + tok, plan.margin);
    };
    bool failed = __syncthreads_or(timeout);
    if (plan.cluster)
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    // Row r of a cluster's item is finished by its CTA r % splits, which the others send their parts of it: place
    // (sender, r / splits) of its receiving area, which is nobody's ring.
    float *const recv = reinterpret_cast<float *>(smem + S::RECV);
    const int places = ROWS / plan.splits;
    if (!failed) {
        for (int row = warp; row < rows; row += WARPS) {         // a warp joins a row
            float2 st[WARPS], y[PIECES];
            float w[WARPS], M, L;
#pragma unroll
            for (int i = 0; i < WARPS; i++)
                st[i] = stats[i][row];
            join_stats(st, w, M, L);
#pragma unroll
            for (int c = 0; c < PIECES; c++) {
                y[c] = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < WARPS; i++) {
                    if (w[i] < 0.0f)
                        continue;
                    const float2 z = *reinterpret_cast<const float2 *>(reinterpret_cast<const float *>(smem + i * S::WARP) +
                                                                       row * DIM + ((64 * c + 2 * lane) ^ (8 * (row & 3))));
                    y[c].x = fmaf(w[i], z.x, y[c].x);
                    y[c].y = fmaf(w[i], z.y, y[c].y);
                }
            }
            if (!plan.cluster) {
                finish(row, M, L, y, plan.splits == 1);
                continue;
            }
            const int to = row % plan.splits, place = split * places + row / plan.splits;
#pragma unroll
            for (int c = 0; c < PIECES; c++)
                store_cluster(in_cta(smem_u32(recv + place * DIM + 64 * c + 2 * lane), to), y[c]);
            if (lane == 0)
                store_cluster(in_cta(smem_u32(&recv_stats[place]), to), make_float2(M, L));
        }
    }
    if (plan.cluster) {
        if (tid < plan.splits)
            store_cluster(in_cta(smem_u32(&recv_failed[split]), tid), make_float2(failed ? 1.0f : 0.0f, 0.0f));
        cluster_sync();
        for (int i = 0; i < plan.splits; i++)
            failed |= recv_failed[i].x != 0.0f;
        for (int k = warp; k < places && !failed; k += WARPS) {
            const int row = split + plan.splits * k;
            if (row >= rows)
                break;
            float2 st[CLUSTER], y[PIECES];
            float w[CLUSTER], M, L;
#pragma unroll
            for (int i = 0; i < CLUSTER; i++)
                st[i] = i < plan.splits ? recv_stats[i * places + k] : make_float2(-INFINITY, 0.0f);
            join_stats(st, w, M, L);
#pragma unroll
            for (int c = 0; c < PIECES; c++) {
                y[c] = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < CLUSTER; i++) {
                    if (i >= plan.splits || w[i] < 0.0f)
                        continue;
                    const float2 z = *reinterpret_cast<const float2 *>(recv + (i * places + k) * DIM + 64 * c + 2 * lane);
                    y[c].x = fmaf(w[i], z.x, y[c].x);
                    y[c].y = fmaf(w[i], z.y, y[c].y);
                }
            }
            finish(row, M, L, y, true);
        }
    }
    report(p.err, bad, DEVERR_CU_SEQLENS);
    report(p.err, timeout, DEVERR_TIMEOUT);
}

template <int DIM, int WARPS> cudaError_t launch_decode_dim(const AttnArgs &p, const AttnPlan &plan, cudaStream_t st)
{
    static std::atomic<uint64_t> ready;      // devices whose kernel attribute is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(ready.load() >> dev & 1)) {
        e = cudaFuncSetAttribute(kda_attn_decode_kernel<DIM, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<DIM, WARPS>::SMEM);
        if (e == cudaSuccess)
            ready.fetch_or(1ull << dev);
    }
    CUtensorMap kmap, vmap;
    if (e == cudaSuccess)
        e = cache_map(&kmap, p.cache.k, p.cache, KEYS);
    if (e == cudaSuccess)
        e = cache_map(&vmap, p.cache.v, p.cache, KEYS);
    if (e != cudaSuccess)
        return e;
    return launch_in_row(kda_attn_decode_kernel<DIM, WARPS>, plan.items, 32 * WARPS, Shape<DIM, WARPS>::SMEM,
                         plan.cluster ? plan.splits : 1, st, p, plan, kmap, vmap);
}

}  // namespace

cudaError_t launch_attn_decode(const AttnArgs &p, const AttnPlan &plan, cudaStream_t st)
{
    if (plan.items <= device_sms())
        return p.cache.dim == 128 ? launch_decode_dim<128, 8>(p, plan, st) : launch_decode_dim<64, 8>(p, plan, st);
    return p.cache.dim == 128 ? launch_decode_dim<128, 4>(p, plan, st) : launch_decode_dim<64, 4>(p, plan, st);
}

}  // namespace kda
