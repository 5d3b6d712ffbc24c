// rope.cu -- rotary positions: the table of angles (moe_rope_table) and the
// append of a step's keys and values to a paged cache, with the rotation of
// queries and keys on the way (moe_kv_append).
//
// Position m turns the pair (a, b) of components by the angle m f_i:
//   (a cos - b sin, b cos + a sin),
// so a query's product with a key depends on the distance of their
// positions only.
#include <cmath>

#include "attention.cuh"

namespace moe {

namespace {

// ---- the table ---------------------------------------------------------------
struct RopeArgs {
    double base, factor, low, high, magnitude;   // low, high: YaRN's ramp over the pair index
    int rot, scaling, n_pos;
    float* table;
};

__global__ void rope_table_kernel(RopeArgs a) {
    const int half = a.rot / 2;
    const long long n = (long long)a.n_pos * half;
    for (long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x; t < n; t += (long long)gridDim.x * blockDim.x) {
        const int i = (int)(t % half);
        const long long m = t / half;
        double f = pow(a.base, -2.0 * i / a.rot);
        if (a.scaling == MOE_ROPE_LINEAR) f /= a.factor;
        if (a.scaling == MOE_ROPE_YARN) {
            const double far = fmin(1.0, fmax(0.0, (i - a.low) / (a.high - a.low)));   // 1: interpolated
            f = f / a.factor * far + f * (1.0 - far);
        }
        double sn, cs;
        sincos((double)m * f, &sn, &cs);
        a.table[m * a.rot + i] = (float)(cs * a.magnitude);
        a.table[m * a.rot + half + i] = (float)(sn * a.magnitude);
    }
}

// ---- append -------------------------------------------------------------------
// One block per token, one thread per pair or component.
template <typename T>
__global__ void append_kernel(AppendArgs a) {
    const int t = blockIdx.x;
    const int half = a.rot / 2, D = a.D;
    const int units = half + (D - a.rot);   // pairs, then components that are not rotated
    const float* ang = nullptr;
    if (a.rot > 0) {
        int m = a.positions[t];
        if (m < 0 || m >= a.n_pos) {
            if (threadIdx.x == 0) raise_flag(a.flags, kFlagBadIndex);
            m = m < 0 ? 0 : a.n_pos - 1;
        }
        ang = a.rope + (size_t)m * a.rot;
    }
    const long long slot = a.slots[t];
    const bool keep = slot >= 0 && slot < a.n_slots;
    if (slot >= a.n_slots && threadIdx.x == 0) raise_flag(a.flags, kFlagBadIndex);
    const long long page = keep ? slot / a.page_size : 0;
    const int row = keep ? (int)(slot - page * a.page_size) : 0;
    const int nq = a.q ? a.heads : 0;
    for (int u = threadIdx.x; u < (nq + a.kv_heads) * units; u += blockDim.x) {
        const int h = u / units, c = u - h * units;
        const bool is_q = h < nq;
        const int kh = h - nq;
        const T* src = is_q ? (const T*)a.q + t * a.q_tok + h * a.q_head : (const T*)a.k + t * a.k_tok + kh * a.k_head;
        T* dst = is_q ? (T*)a.q_out + t * a.out_tok + h * a.out_head
                      : (T*)a.ck + ((page * a.kv_heads + kh) * a.page_size + row) * D;
        if (!is_q && !keep) continue;
        if (c < half) {
            const int i0 = a.interleaved ? 2 * c : c, i1 = a.interleaved ? 2 * c + 1 : c + half;
            const float x = to_float(src[i0]), y = to_float(src[i1]), cs = ang[c], sn = ang[half + c];
            dst[i0] = from_float<T>(x * cs - y * sn);
            dst[i1] = from_float<T>(y * cs + x * sn);
        } else {
            dst[c + half] = src[c + half];
        }
    }
    if (!keep) return;
    for (int u = threadIdx.x; u < a.kv_heads * D; u += blockDim.x) {
        const int h = u / D, c = u - h * D;
        ((T*)a.cv)[((page * a.kv_heads + h) * a.page_size + row) * D + c] = ((const T*)a.v)[t * a.v_tok + h * a.v_head + c];
    }
}

cudaError_t launch_append(const AppendArgs& a, int dtype, cudaStream_t s) {
    if (dtype == MOE_DTYPE_BF16) append_kernel<__nv_bfloat16><<<a.T, 256, 0, s>>>(a);
    else append_kernel<float><<<a.T, 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_rope_table(const moe_rope_params* p, int32_t n_pos, float* table, moe_stream_t stream) {
    if (!p) return report(MOE_ERR_ARG, "params is NULL");
    if (p->rot < 2 || p->rot % 2 != 0 || p->rot > MOE_MAX_HEAD_DIM)
        return report(MOE_ERR_ARG, "rot=%d must be even, 2..%d", p->rot, MOE_MAX_HEAD_DIM);
    if (p->scaling < MOE_ROPE_PLAIN || p->scaling > MOE_ROPE_YARN)
        return report(MOE_ERR_ARG, "unknown scaling %d", p->scaling);
    if (!(p->base > 1.0) || !std::isfinite(p->base)) return report(MOE_ERR_ARG, "base=%g must be above 1", p->base);
    const bool scaled = p->scaling != MOE_ROPE_PLAIN;
    if (scaled && (!(p->factor >= 1.0) || !std::isfinite(p->factor)))
        return report(MOE_ERR_ARG, "factor=%g must be at least 1", p->factor);
    if (!std::isfinite(p->magnitude)) return report(MOE_ERR_ARG, "magnitude is not finite");
    if (n_pos < 0) return report(MOE_ERR_ARG, "n_pos=%d is negative", n_pos);
    if (n_pos > 0 && (!table || !aligned(table, 16))) return report(MOE_ERR_ARG, "table is NULL or not 16-byte aligned");
    RopeArgs a{};
    a.base = p->base;
    a.factor = scaled ? p->factor : 1.0;
    a.rot = p->rot;
    a.scaling = p->scaling;
    a.n_pos = n_pos;
    a.table = table;
    a.magnitude = p->magnitude > 0.0 ? p->magnitude : 1.0;
    if (p->scaling == MOE_ROPE_NTK) {
        if (p->rot < 4) return report(MOE_ERR_ARG, "MOE_ROPE_NTK needs rot of 4 or more");
        a.base = p->base * std::pow(p->factor, (double)p->rot / (p->rot - 2));
    }
    if (p->scaling == MOE_ROPE_YARN) {
        if (!(p->original_len > 0.0) || !(p->beta_slow > 0.0) || !(p->beta_fast > p->beta_slow) ||
            !std::isfinite(p->original_len) || !std::isfinite(p->beta_fast))
            return report(MOE_ERR_ARG, "need original_len > 0 and beta_fast > beta_slow > 0");
        // the pair index whose frequency turns `beta` times over original_len:
        // original_len base^(-2 i / rot) = 2 pi beta
        const double two_pi = 6.283185307179586476925;
        auto index = [&](double beta) {
            return p->rot * std::log(p->original_len / (two_pi * beta)) / (2.0 * std::log(p->base));
        };
        a.low = std::fmax(0.0, std::floor(index(p->beta_fast)));
        a.high = std::fmin(p->rot - 1.0, std::ceil(index(p->beta_slow)));
        if (!(a.high > a.low)) a.high = a.low + 0.001;   // no pair in between: a step
        if (!(p->magnitude > 0.0)) a.magnitude = 0.1 * std::log(p->factor) + 1.0;
    }
    if (n_pos == 0) return MOE_OK;
    const long long n = (long long)n_pos * (p->rot / 2);
    const long long blocks = (n + 255) / 256;
    rope_table_kernel<<<(unsigned)(blocks < 152 * 64 ? blocks : 152 * 64), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MOE_OK : report(MOE_ERR_CUDA, "rope table launch: %s", cudaGetErrorString(e));
}

moe_status moe_kv_append(const void* q, const void* k, const void* v, const float* rope, const int32_t* positions,
                         const int64_t* slots, const moe_append_params* p, const moe_kv_cache* cache, void* q_out,
                         void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    moe_status st = check_cache(cache, false);
    if (st != MOE_OK) return st;
    if (!p) return report(MOE_ERR_ARG, "params is NULL");
    if (p->T < 0) return report(MOE_ERR_ARG, "T=%d is negative", p->T);
    const bool has_q = q != nullptr;
    if (has_q != (q_out != nullptr)) return report(MOE_ERR_ARG, "q and q_out must both be given, or neither");
    if (has_q && (p->heads < 1 || p->heads > kMaxHeads)) return report(MOE_ERR_ARG, "heads=%d outside 1..%d", p->heads, kMaxHeads);
    if (p->rot < 0 || p->rot % 2 != 0 || p->rot > cache->head_dim)
        return report(MOE_ERR_ARG, "rot=%d must be even, 0..head_dim=%d", p->rot, cache->head_dim);
    if (p->interleaved != 0 && p->interleaved != 1) return report(MOE_ERR_ARG, "interleaved must be 0 or 1");
    if (workspace_bytes < MOE_ATTENTION_WORKSPACE_MIN || !workspace || !aligned(workspace, 256))
        return report(MOE_ERR_WORKSPACE, "workspace missing, not 256-byte aligned or below %d bytes", MOE_ATTENTION_WORKSPACE_MIN);
    if (p->T == 0) return MOE_OK;
    if (!k || !v || !slots || (p->rot > 0 && (!rope || !positions))) return report(MOE_ERR_ARG, "a tensor pointer is NULL");
    const void* ptrs[] = {q, k, v, rope, q_out};
    for (const void* x : ptrs)
        if (!aligned(x, 16)) return report(MOE_ERR_ARG, "a tensor pointer is not 16-byte aligned");
    if (!aligned(positions, 4) || !aligned(slots, 8)) return report(MOE_ERR_ARG, "positions or slots misaligned");
    if (p->rot > 0 && p->n_pos < 1) return report(MOE_ERR_ARG, "n_pos=%d must be positive", p->n_pos);
    const int elt = cache->dtype == MOE_DTYPE_BF16 ? 2 : 4;
    const int64_t dist[] = {p->k_tok, p->k_head, p->v_tok, p->v_head, has_q ? p->q_tok : 0, has_q ? p->q_head : 0,
                            has_q ? p->out_tok : 0, has_q ? p->out_head : 0};
    for (int64_t x : dist)
        if (x < 0 || x * elt % 16 != 0)
            return report(MOE_ERR_ARG, "distances between tokens and heads must be multiples of 16 bytes, not negative");
    AppendArgs a{};
    a.q = q; a.k = k; a.v = v; a.rope = rope; a.positions = positions;
    a.slots = reinterpret_cast<const long long*>(slots);
    a.q_out = q_out; a.ck = cache->k; a.cv = cache->v;
    a.flags = &static_cast<WsHeader*>(workspace)->flags;
    a.T = p->T; a.heads = has_q ? p->heads : 0; a.kv_heads = cache->kv_heads; a.D = cache->head_dim;
    a.rot = p->rot; a.n_pos = p->n_pos; a.interleaved = p->interleaved; a.page_size = cache->page_size;
    a.n_slots = (long long)cache->n_pages * cache->page_size;
    a.q_tok = p->q_tok; a.q_head = p->q_head; a.k_tok = p->k_tok; a.k_head = p->k_head;
    a.v_tok = p->v_tok; a.v_head = p->v_head; a.out_tok = p->out_tok; a.out_head = p->out_head;
    const cudaError_t e = launch_append(a, cache->dtype, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : report(MOE_ERR_CUDA, "append launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
