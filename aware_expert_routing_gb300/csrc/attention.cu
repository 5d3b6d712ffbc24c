// attention.cu -- attention of a step's tokens (drafted trees, chains, single
// tokens) to a paged cache: moe_tree_attention.
//
// For token i of a request and query head h, over the positions j that it
// sees: s_j = scale q.k_j, out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m).
// The sums run in one pass with the running maximum m: when m grows, the sums
// so far are multiplied by exp(m_old - m_new).
#include "attention.cuh"

namespace moe {

int num_sms();   // api.cu

namespace {

// One block per (token, query head): its warps take positions in turn, a
// lane holds components lane, lane + 32, ..., and the warps' sums are joined
// at the end.
constexpr int kSimpleWarps = 4;

template <typename T>
__global__ void __launch_bounds__(kSimpleWarps * 32) attention_simple_kernel(AttentionArgs a) {
    const int t = blockIdx.x, h = blockIdx.y, kh = h / a.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ float sm[kSimpleWarps], sl[kSimpleWarps], so[kSimpleWarps][MOE_MAX_HEAD_DIM];
    // the token's request: the last r with q_offsets[r] <= t
    int lo = 0, hi = a.R;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.q_offsets[mid] <= t) lo = mid; else hi = mid;
    }
    const int r = lo, t0 = a.q_offsets[r], t1 = a.q_offsets[r + 1], ctx = a.ctx_len[r];
    if (t < t0 || t >= t1) return;
    if (t1 > a.T || ctx < 0 || (long long)ctx + (t1 - t0) > (long long)a.max_pages * a.page_size) {
        if (threadIdx.x == 0) raise_flag(a.flags, kFlagBadIndex);
        return;
    }
    const int n = t1 - t0, i = t - t0;
    constexpr int kPer = MOE_MAX_HEAD_DIM / 32;
    float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
        const int x = lane + 32 * c;
        q[c] = x < a.D ? to_float(((const T*)a.q)[t * a.q_tok + h * a.q_head + x]) : 0.f;
        o[c] = 0.f;
    }
    for (int j = warp; j < ctx + n; j += kSimpleWarps) {
        if (j >= ctx) {
            const int d = j - ctx;
            if (a.mask ? d >= 32 * a.mask_words || !((a.mask[(size_t)t * a.mask_words + d / 32] >> (d & 31)) & 1u) : d > i)
                continue;
        }
        const int page = a.page_table[(size_t)r * a.max_pages + j / a.page_size];
        if (page < 0 || page >= a.n_pages) {
            if (lane == 0) raise_flag(a.flags, kFlagBadIndex);
            continue;
        }
        const size_t row = (((size_t)page * a.kv_heads + kh) * a.page_size + j % a.page_size) * a.D;
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < kPer; ++c)
            if (lane + 32 * c < a.D) s = fmaf(q[c], to_float(((const T*)a.ck)[row + lane + 32 * c]), s);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= a.scale;
        if (s == -INFINITY) continue;   // adds nothing
        const float mn = fmaxf(m, s), old = m == -INFINITY ? 0.f : expf(m - mn), p = expf(s - mn);
        l = l * old + p;
#pragma unroll
        for (int c = 0; c < kPer; ++c)
            if (lane + 32 * c < a.D) o[c] = fmaf(o[c], old, p * to_float(((const T*)a.cv)[row + lane + 32 * c]));
        m = mn;
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int c = 0; c < kPer; ++c) so[warp][lane + 32 * c] = o[c];
    __syncthreads();
    m = -INFINITY;
    for (int w = 0; w < kSimpleWarps; ++w) m = fmaxf(m, sm[w]);
    l = 0.f;
    float f[kSimpleWarps];
    for (int w = 0; w < kSimpleWarps; ++w) {
        f[w] = sl[w] == 0.f ? 0.f : expf(sm[w] - m);
        l += f[w] * sl[w];
    }
    for (int x = threadIdx.x; x < a.D; x += kSimpleWarps * 32) {
        float v = 0.f;
        for (int w = 0; w < kSimpleWarps; ++w) v += f[w] * so[w][x];
        ((T*)a.out)[((size_t)t * a.heads + h) * a.D + x] = from_float<T>(l == 0.f ? 0.f : v / l);
    }
    if (a.lse && threadIdx.x == 0) a.lse[(size_t)t * a.heads + h] = l == 0.f ? -INFINITY : m + logf(l);
}

cudaError_t launch_attention(const AttentionArgs& a, int dtype, cudaStream_t s) {
    if (attention_tc_supported(a, dtype)) return launch_attention_tc(a, num_sms(), s);
    const dim3 grid(a.T, a.heads);
    if (dtype == MOE_DTYPE_BF16) attention_simple_kernel<__nv_bfloat16><<<grid, kSimpleWarps * 32, 0, s>>>(a);
    else attention_simple_kernel<float><<<grid, kSimpleWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

}  // namespace moe

using namespace moe;

namespace {
moe_status check_heads(int T, int heads, const moe_kv_cache* cache) {
    if (T < 0) return report(MOE_ERR_ARG, "T=%d is negative", T);
    if (heads < 1 || heads > kMaxHeads) return report(MOE_ERR_ARG, "heads=%d outside 1..%d", heads, kMaxHeads);
    if ((long long)T * heads > 0x7fffffffLL) return report(MOE_ERR_ARG, "T * heads passes 2^31 - 1");
    if (heads % cache->kv_heads != 0)
        return report(MOE_ERR_ARG, "heads=%d is not a multiple of kv_heads=%d", heads, cache->kv_heads);
    return MOE_OK;
}
}  // namespace

extern "C" {

size_t moe_attention_workspace_bytes(int32_t T, int32_t heads, const moe_kv_cache* cache) {
    if (check_cache(cache, true) != MOE_OK || check_heads(T, heads, cache) != MOE_OK) return 0;
    return attention_layout(T, heads / cache->kv_heads, cache->head_dim).total;
}

moe_status moe_tree_attention(const void* q, const int32_t* q_offsets, const int32_t* ctx_len, const uint32_t* mask,
                              const moe_attention_params* p, const moe_kv_cache* cache, void* out, float* lse,
                              void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    moe_status st = check_cache(cache, true);
    if (st != MOE_OK) return st;
    if (!p) return report(MOE_ERR_ARG, "params is NULL");
    if ((st = check_heads(p->T, p->heads, cache)) != MOE_OK) return st;
    if (mask && p->mask_words < 1) return report(MOE_ERR_ARG, "mask_words=%d must be positive", p->mask_words);
    if (!(p->scale > 0.f) || !(p->scale < INFINITY)) return report(MOE_ERR_ARG, "scale must be positive and finite");
    const size_t need = moe_attention_workspace_bytes(p->T, p->heads, cache);
    if (!workspace || !aligned(workspace, 256)) return report(MOE_ERR_WORKSPACE, "workspace is NULL or not 256-byte aligned");
    if (workspace_bytes < need) return report(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
    if (p->T == 0 || cache->n_requests == 0) return MOE_OK;
    if (!q || !out || !q_offsets || !ctx_len) return report(MOE_ERR_ARG, "a tensor pointer is NULL");
    if (!aligned(q, 16) || !aligned(out, 16)) return report(MOE_ERR_ARG, "q or out is not 16-byte aligned");
    if (!aligned(q_offsets, 4) || !aligned(ctx_len, 4) || !aligned(mask, 4) || !aligned(lse, 4))
        return report(MOE_ERR_ARG, "q_offsets, ctx_len, mask or lse misaligned");
    const int elt = cache->dtype == MOE_DTYPE_BF16 ? 2 : 4;
    if (p->q_tok < 0 || p->q_head < 0 || p->q_tok * elt % 16 != 0 || p->q_head * elt % 16 != 0)
        return report(MOE_ERR_ARG, "distances between tokens and heads must be multiples of 16 bytes, not negative");
    AttentionArgs a{};
    a.q = q; a.q_offsets = q_offsets; a.ctx_len = ctx_len; a.mask = mask;
    a.ck = cache->k; a.cv = cache->v; a.page_table = cache->page_table;
    a.out = out; a.lse = lse; a.flags = &static_cast<WsHeader*>(workspace)->flags;
    a.T = p->T; a.heads = p->heads; a.kv_heads = cache->kv_heads; a.group = p->heads / cache->kv_heads; a.D = cache->head_dim; a.R = cache->n_requests;
    a.n_pages = cache->n_pages; a.page_size = cache->page_size; a.max_pages = cache->max_pages;
    a.mask_words = mask ? p->mask_words : 0;
    a.scale = p->scale; a.q_tok = p->q_tok; a.q_head = p->q_head;
    const AttentionLayout L = attention_layout(p->T, p->heads / cache->kv_heads, cache->head_dim);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    a.total = reinterpret_cast<long long*>(ws + L.plan);
    a.plan = reinterpret_cast<RangeStart*>(ws + L.plan + 16);
    a.ml = reinterpret_cast<float2*>(ws + L.ml);
    a.o = reinterpret_cast<float*>(ws + L.o);
    a.rows = L.rows;
    a.wait_cycles = wait_cycles_now();
    const cudaError_t e = launch_attention(a, cache->dtype, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : report(MOE_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
