// attention.cuh -- what the kernels and entry points around the paged cache
// share (rope.cu, attention.cu).
#pragma once

#include <cstdarg>
#include <cstdio>

#include "common.cuh"

namespace moe {

constexpr int kMaxHeads = 1024;

// Records the thread's last error (api.cu) and returns `status`.
moe_status report_error(moe_status status, const char* message);

inline moe_status report(moe_status status, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return report_error(status, buf);
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The descriptor of a paged cache; attend: its page table is read too.
inline moe_status check_cache(const moe_kv_cache* c, bool attend) {
    if (!c) return report(MOE_ERR_ARG, "cache is NULL");
    if (c->dtype != MOE_DTYPE_BF16 && c->dtype != MOE_DTYPE_F32) return report(MOE_ERR_ARG, "unknown dtype %d", c->dtype);
    if (c->head_dim < 8 || c->head_dim % 8 != 0 || c->head_dim > MOE_MAX_HEAD_DIM)
        return report(MOE_ERR_ARG, "head_dim=%d must be a multiple of 8 in 8..%d", c->head_dim, MOE_MAX_HEAD_DIM);
    if (c->page_size < 1 || c->page_size > MOE_MAX_PAGE)
        return report(MOE_ERR_ARG, "page_size=%d outside 1..%d", c->page_size, MOE_MAX_PAGE);
    if (c->kv_heads < 1 || c->kv_heads > kMaxHeads)
        return report(MOE_ERR_ARG, "kv_heads=%d outside 1..%d", c->kv_heads, kMaxHeads);
    if (c->n_pages < 0) return report(MOE_ERR_ARG, "n_pages=%d is negative", c->n_pages);
    if (c->n_pages > 0 && (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)))
        return report(MOE_ERR_ARG, "the cache's k or v is NULL or not 16-byte aligned");
    if (!attend) return MOE_OK;
    if (c->n_requests < 0 || c->n_requests > MOE_MAX_REQUESTS)
        return report(MOE_ERR_ARG, "n_requests=%d outside 0..%d", c->n_requests, MOE_MAX_REQUESTS);
    if (c->max_pages < 0 || (long long)c->max_pages * c->page_size > (1LL << 30))
        return report(MOE_ERR_ARG, "max_pages=%d is negative, or positions pass 2^30", c->max_pages);
    if (c->n_requests > 0 && c->max_pages > 0 && (!c->page_table || !aligned(c->page_table, 4)))
        return report(MOE_ERR_ARG, "page_table is NULL or misaligned");
    return MOE_OK;
}

// The tensor-core kernel: ranges of work (one per SM of a GB300) and most query
// rows of a unit.  The other kernel: two ranges per SM.
constexpr int kTcRanges = 152, kTcRows = 256;
constexpr int kPlainRanges = 304, kPlainRows = 64;

// Workspace of moe_tree_attention: the flag word's header, the record of each
// range's start, and two partial results a range (of its first and its last
// unit): per row the running maximum (of scores in powers of two) and sum,
// and the unnormalised output.
struct AttentionLayout {
    size_t plan, ml, o, total;
    int rows;
};

struct RangeStart {
    int t0, n;              // the request's tokens
    int h, rt;              // key head and row tile of the unit that the range starts in
    int off, nkt;           // steps into the unit, and the unit's key tiles (0: the range is empty)
    int line_q, line_rem;   // how the line is cut
};

inline AttentionLayout attention_layout(int T, int group, int D, bool tc) {
    AttentionLayout L;
    const long long rows = (long long)T * group;
    const int most = tc ? kTcRows : kPlainRows, ranges = tc ? kTcRanges : kPlainRanges;
    L.rows = (int)(rows < most ? (rows + 31) / 32 * 32 : most);   // whole warps
    size_t o = align256(MOE_ATTENTION_WORKSPACE_MIN);
    L.plan = o; o += align256(sizeof(RangeStart) * ranges);
    L.ml = o;   o += align256(sizeof(float2) * 2 * ranges * (size_t)L.rows);
    L.o = o;    o += align256(sizeof(float) * 2 * ranges * (size_t)L.rows * D);
    L.total = o;
    return L;
}

// Whether the tensor-core kernel (attention_tc.cu) takes a cache: bf16, heads
// of 64 or 128, pages of whole 8-row swizzle atoms that a tile of 128 keys
// holds whole or lies inside of.
inline bool attention_tc_fits(const moe_kv_cache* c) {
    return c->dtype == MOE_DTYPE_BF16 && (c->head_dim == 64 || c->head_dim == 128) && c->page_size % 8 == 0 &&
           (128 % c->page_size == 0 || c->page_size % 128 == 0) &&
           (long long)c->n_pages * c->kv_heads * c->page_size / 8 < 0x7fffffffLL;
}

struct AppendArgs {
    const void *q, *k, *v;
    const float* rope;
    const int32_t* positions;
    const long long* slots;
    void *q_out, *ck, *cv;
    uint32_t* flags;
    int T, heads, kv_heads, D, rot, n_pos, interleaved, page_size;
    long long n_slots;
    long long q_tok, q_head, k_tok, k_head, v_tok, v_head, out_tok, out_head;
};

struct AttentionArgs {
    const void* q;
    const int32_t* q_offsets;
    const int32_t* ctx_len;
    const uint32_t* mask;      // [T][mask_words] or null: causal
    const void *ck, *cv;
    const int32_t* page_table;
    void* out;                 // [T][heads][D]
    float* lse;                // [T][heads] or null
    uint32_t* flags;
    int T, heads, kv_heads, group, D, R, n_pages, page_size, max_pages, mask_words;   // group: heads / kv_heads
    float scale;
    long long q_tok, q_head;
    // the workspace (AttentionLayout)
    RangeStart* plan;          // [ranges]
    float2* ml;                // [2 * ranges][rows]
    float* o;                  // [2 * ranges][rows][D]
    int rows;
    int min_steps;             // fewest steps of a range, on average
    long long wait_cycles;
};

cudaError_t launch_attention_tc(const AttentionArgs& a, int num_sms, cudaStream_t s);

#ifdef __CUDACC__

template <typename T> __device__ __forceinline__ float to_float(T x);
template <> __device__ __forceinline__ float to_float<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

#endif  // __CUDACC__

}  // namespace moe
