// kda_linear_attn: checks of the arguments, and which kernel a call takes.
#include "kda_linear.cuh"

#include <algorithm>
#include <cmath>

namespace kda {

// Short sequences are evaluated token by token.  A chunk costs the same for 1 token and for 64, about what this many take in the
// other kernel (us, chunks | tokens): one sequence of 32 heads of 128, 16 tokens 9.8 | 7.6, 24 9.9 | 10.1; 8 x 96, 12 tokens 37 | 33, 16
// 37 | 45; 64 x 64, 8 tokens 109 | 101, 12 110 | 144; 32 x 32 of 64, 16 tokens 26 | 16.  With cu_seqlens only the sum is known here.
static bool token_by_token(int N, int64_t T, int H, int D) { return T <= (D == 64 ? 16 : ((int64_t)N * H <= 1024 ? 14 : 8)); }

// The cut of a call into groups (sizes only, so that the workspace is known beforehand), for 152 SMs.  Costs in 10 ns, fitted to what
// was measured: a chunk takes 1.15 us in a (sequence, head)'s chain, however few run; with groups 2.1 us, the pass over K and V
// included, and two launches and the groups' states more.  One chain | groups (us): 8192 tokens of 8 heads 153 | 43, 32 heads over 8 154 | 87,
// 64 over 8 156 | 150, 76 157 | 163; 2048 of 48 45 | 45; 1024 of 8 heads 24.6 | 22.5.
static LinearPlan make_plan(bool varlen, int N, int64_t T, int H)
{
    LinearPlan plan{};
    const int64_t chunks = (T + 63) / 64, pairs = (int64_t)N * H;
    // the longest sequence; of a ragged batch only the sum is known, and twice the mean is taken for it
    const int64_t chain = varlen && N > 1 ? std::min(chunks, 2 * ((chunks + N - 1) / N)) : chunks;
    int64_t cut = 1, best = 650 + 115 * chain;
    for (int64_t g = 2; g * pairs <= 152 && g <= chain; g++) {
        const int64_t cost = 1150 + 210 * ((chain + g - 1) / g) + 30 * g + 5 * g * pairs;
        if (cost < best)
            best = cost, cut = g;
    }
    plan.group_chunks = (chain + cut - 1) / cut;
    plan.groups = (int)((chunks + plan.group_chunks - 1) / std::max<int64_t>(plan.group_chunks, 1));
    if (cut == 1) {
        plan.groups = 1;
        plan.group_chunks = std::max<int64_t>(chunks, 1);
    }
    if (varlen) {
        // every sequence has one group at least, and the cuts of all are no more than one sequence's
        plan.items = (N + (plan.groups > 1 ? T / (64 * plan.group_chunks) : 0)) * H;
        plan.items_before = plan.groups > 1 ? T / (64 * plan.group_chunks) * H : 0;
    } else {
        plan.items = pairs * plan.groups;
        plan.items_before = pairs * (plan.groups - 1);
    }
    return plan;
}
// Slots of groups' states (slot_of is below it).
static int64_t plan_slots(const LinearPlan &plan, bool varlen, int N, int64_t T)
{
    if (plan.groups <= 1)
        return 0;
    return varlen ? T / (64 * plan.group_chunks) + N + 1 : (int64_t)N * plan.groups;
}
static size_t plan_bytes(const LinearPlan &plan, bool varlen, int N, int64_t T, int H, int D)
{
    return (size_t)plan_slots(plan, varlen, N, T) * H * ((size_t)D * D + 2) * sizeof(float);
}

static kda_status_t check_linear(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                 int64_t v_stride, const float *log_decay, const float *gate, float scale, const void *out,
                                 const void *init, const void *fin, kda_dtype_t state, const int32_t *lens,
                                 const int64_t *cu, int N, int64_t T, int H, int Hkv, int D)
{
    if (N < 1 || T < 0 || H < 1 || Hkv < 1 || H % Hkv)
        return KDA_ERR_INVALID_ARGUMENT;
    if ((init || fin) && state != KDA_DTYPE_BF16 && state != KDA_DTYPE_FP32)
        return KDA_ERR_INVALID_ARGUMENT;
    if (lens && cu)
        return KDA_ERR_INVALID_ARGUMENT;
    if (!is_aligned(log_decay, 4) || !is_aligned(gate, 4) || !is_aligned(init, 16) || !is_aligned(fin, 16) ||
        !is_aligned(lens, 4) || !is_aligned(cu, 8))
        return KDA_ERR_INVALID_ARGUMENT;
    if (D != 64 && D != 128)
        return KDA_ERR_UNSUPPORTED;
    if (!std::isfinite(scale))
        return KDA_ERR_UNSUPPORTED;
    // tokens are 32-bit coordinates of the bulk copies; warps of the token kernel (at most 16 a pair) and its grid
    if (T > INT32_MAX || (cu ? T : (int64_t)N * T) > INT32_MAX || (int64_t)N * H > INT32_MAX / 16)
        return KDA_ERR_UNSUPPORTED;
    const uint64_t states = (uint64_t)N * H * D * D * (state == KDA_DTYPE_BF16 ? 2 : 4);
    if (init != fin && overlap(init, states, fin, states))
        return KDA_ERR_INVALID_ARGUMENT;
    if (overlap(fin, states, log_decay, (uint64_t)H * 4) || overlap(fin, states, lens, (uint64_t)N * 4) ||
        overlap(fin, states, cu, (uint64_t)(N + 1) * 8))
        return KDA_ERR_INVALID_ARGUMENT;
    const uint64_t tokens = cu ? (uint64_t)T : (uint64_t)N * T;
    if (tokens == 0)
        return KDA_OK;
    if (!q || !k || !v || !out || !is_aligned(q, 16) || !is_aligned(k, 16) || !is_aligned(v, 16) || !is_aligned(out, 16))
        return KDA_ERR_INVALID_ARGUMENT;
    const int64_t row = (int64_t)H * D, kv_row = (int64_t)Hkv * D;
    if (q_stride % 8 || q_stride < row || k_stride % 8 || k_stride < kv_row || v_stride % 8 || v_stride < kv_row)
        return KDA_ERR_INVALID_ARGUMENT;
    // a head's CTA writes its tokens and its state while others still read theirs
    const uint64_t written = tokens * row * 2;
    const struct {
        const void *p;
        uint64_t bytes;
    } read[] = {{q, ((tokens - 1) * q_stride + row) * 2}, {k, ((tokens - 1) * k_stride + kv_row) * 2},
                {v, ((tokens - 1) * v_stride + kv_row) * 2}, {gate, tokens * H * 4}};
    for (const auto &r : read)
        if (overlap(out, written, r.p, r.bytes) || overlap(fin, states, r.p, r.bytes))
            return KDA_ERR_INVALID_ARGUMENT;
    if (overlap(out, written, fin, states) || overlap(out, written, init, states) || overlap(out, written, log_decay, (uint64_t)H * 4) ||
        overlap(out, written, lens, (uint64_t)N * 4) || overlap(out, written, cu, (uint64_t)(N + 1) * 8))
        return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

}  // namespace kda

using namespace kda;

extern "C" size_t kda_linear_attn_workspace_size(int varlen, int N, int64_t T, int H, int D)
{
    if (N < 1 || T < 0 || H < 1 || (D != 64 && D != 128) || T > INT32_MAX || (varlen ? T : (int64_t)N * T) > INT32_MAX ||
        (int64_t)N * H > INT32_MAX / 16 || token_by_token(N, T, H, D))
        return 0;
    return plan_bytes(make_plan(varlen != 0, N, T, H), varlen != 0, N, T, H, D);
}

extern "C" kda_status_t kda_linear_attn_ws(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                           int64_t v_stride, const float *log_decay, const float *gate, float scale, void *out,
                                           const void *initial_state, void *final_state, kda_dtype_t state_dtype,
                                           const int32_t *lens, const int64_t *cu_seqlens, int N, int64_t T, int H, int Hkv,
                                           int D, void *workspace, size_t workspace_bytes, kda_stream_t stream)
{
    const kda_status_t s = check_linear(q, q_stride, k, k_stride, v, v_stride, log_decay, gate, scale, out, initial_state,
                                        final_state, state_dtype, lens, cu_seqlens, N, T, H, Hkv, D);
    if (s != KDA_OK)
        return s;
    const kda_dtype_t state = initial_state || final_state ? state_dtype : KDA_DTYPE_NONE;
    const size_t need = kda_linear_attn_workspace_size(cu_seqlens != nullptr, N, T, H, D);
    if (need > 0 && (!workspace || !is_aligned(workspace, 256) || workspace_bytes < need))
        return KDA_ERR_INVALID_ARGUMENT;
    LinearArgs p{};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
    p.log_decay = log_decay, p.gate = gate, p.scale = scale;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.init = initial_state, p.fin = final_state;
    p.lens = lens;
    p.tok = Tokens{cu_seqlens, T, N};
    p.H = H, p.group = H / Hkv, p.dim = D;
    if (step_error_word(&p.err) != cudaSuccess)
        return KDA_ERR_CUDA;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (token_by_token(N, T, H, D))
        return launch_linear_tokens(p, state, st) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    LinearPlan plan = make_plan(cu_seqlens != nullptr, N, T, H);
    plan.states = static_cast<float *>(workspace);
    plan.decays = reinterpret_cast<float2 *>(plan.states + plan_slots(plan, cu_seqlens != nullptr, N, T) * H * D * D);
    plan.state_type = state;
    plan.wait_polls = wait_limit();
    return launch_linear_chunks(p, plan, st) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_linear_attn(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                        int64_t v_stride, const float *log_decay, const float *gate, float scale, void *out,
                                        const void *initial_state, void *final_state, kda_dtype_t state_dtype,
                                        const int32_t *lens, const int64_t *cu_seqlens, int N, int64_t T, int H, int Hkv,
                                        int D, kda_stream_t stream)
{
    const kda_status_t c = check_linear(q, q_stride, k, k_stride, v, v_stride, log_decay, gate, scale, out, initial_state,
                                        final_state, state_dtype, lens, cu_seqlens, N, T, H, Hkv, D);
    if (c != KDA_OK)
        return c;
    const size_t need = kda_linear_attn_workspace_size(cu_seqlens != nullptr, N, T, H, D);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    void *ws = nullptr;
    if (need > 0 && pool_alloc(&ws, need, st) != cudaSuccess)
        return KDA_ERR_CUDA;
    kda_status_t s = kda_linear_attn_ws(q, q_stride, k, k_stride, v, v_stride, log_decay, gate, scale, out, initial_state,
                                        final_state, state_dtype, lens, cu_seqlens, N, T, H, Hkv, D, ws, need, stream);
    if (ws && cudaFreeAsync(ws, st) != cudaSuccess && s == KDA_OK)
        s = KDA_ERR_CUDA;
    return s;
}
