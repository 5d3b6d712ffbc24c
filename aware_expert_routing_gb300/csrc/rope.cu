// rope.cu -- rotary positions: the table of angles (moe_rope_table) and the
// append of a step's keys and values to a paged cache, with the rotation of
// queries and keys on the way (moe_kv_append).
//
// Position m turns the pair (a, b) of components by the angle m f_i:
//   (a cos - b sin, b cos + a sin),
// so a query's product with a key depends on the distance of their
// positions only.
#include <cmath>
#include <type_traits>

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
// Bounded by the bytes: queries, keys and values are read once and written once.

struct Place {
    const float* angle;     // the position's cosines, then sines
    bool keep;              // the token's key and value are written
    long long page;
    int row;                // of the page
};

__device__ __forceinline__ Place place_of(const AppendArgs& a, int t, bool report) {
    Place p{};
    if (a.rot > 0) {
        int m = a.positions[t];
        if (m < 0 || m >= a.n_pos) {
            if (report) raise_flag(a.flags, kFlagBadIndex);
            m = m < 0 ? 0 : a.n_pos - 1;
        }
        p.angle = a.rope + (size_t)m * a.rot;
    }
    const long long slot = a.slots[t];
    if (slot >= a.n_slots && report) raise_flag(a.flags, kFlagBadIndex);
    p.keep = slot >= 0 && slot < a.n_slots;
    if (p.keep) {   // slots past 2^32 are rare: the 64-bit division is skipped
        p.page = slot >> 32 ? slot / a.page_size : (long long)((uint32_t)slot / (uint32_t)a.page_size);
        p.row = (int)(slot - p.page * a.page_size);
    }
    return p;
}

// Sixteen bytes of a row as floats, and back.
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ void get(const uint4& u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void get(const uint4& u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Rotations that fall on whole 16-byte words.  A block has one token (and, in
// y, some of its rows: query heads, key heads, value heads); threadIdx.x is
// the place in a row: a word of each half of the rotated part (half layout),
// or a word.  It keeps its cosines and sines for all rows it goes through.
// kMany: small blocks, see kManyTokens.  Registers decide how many words are
// under way: with 84 of them 16000 tokens take 79 us, with 64 67, with 48 60.
template <typename T, bool kPairs, bool kMany>
__global__ void __launch_bounds__(kMany ? 64 : 256, kMany ? 24 : 5) append_kernel(const AppendArgs a) {
    constexpr int N = Vec<T>::kN;
    const int t = blockIdx.x, x = threadIdx.x, nx = blockDim.x, D = a.D;
    const int half = a.rot / 2;
    // half layout: words of one half, then words that are not rotated
    const int turned = kPairs ? a.rot / N : half / N;
    const bool turn = x < turned;
    // the thread's word of a rotated row and its partner, and its words of a value
    const int at = kPairs || turn ? x * N : a.rot + (x - turned) * N, at2 = !kPairs && turn ? at + half : -1;
    const int vat = x * N, vat2 = !kPairs && (x + nx) * N < D ? (x + nx) * N : -1;
    const int rows = a.heads + 2 * a.kv_heads, step = blockDim.y * gridDim.y;
    grid_launch_dependents();
    grid_dependency_wait();

    // The first row is on its way before the token's place and angles are read
    // (two loads one after the other).
    uint4 u, w;
    auto fetch = [&](int r) {
        const bool is_q = r < a.heads, is_v = r >= a.heads + a.kv_heads;
        const int kh = r - a.heads - (is_v ? a.kv_heads : 0);
        const T* src = is_q   ? static_cast<const T*>(a.q) + t * a.q_tok + r * a.q_head
                       : is_v ? static_cast<const T*>(a.v) + t * a.v_tok + kh * a.v_head
                              : static_cast<const T*>(a.k) + t * a.k_tok + kh * a.k_head;
        u = *reinterpret_cast<const uint4*>(src + (is_v ? vat : at));
        if ((is_v ? vat2 : at2) >= 0) w = *reinterpret_cast<const uint4*>(src + (is_v ? vat2 : at2));
    };
    int r = blockIdx.y * blockDim.y + threadIdx.y;
    if (r < rows) fetch(r);
    const Place p = place_of(a, t, x == 0 && threadIdx.y == 0 && blockIdx.y == 0);
    float cs[N], sn[N];
    if (turn) {
        constexpr int M = kPairs ? N / 2 : N;
        const float* c0 = p.angle + x * M;
        if (M % 4 == 0) {
#pragma unroll
            for (int i = 0; i < M; i += 4) {
                const float4 c = *reinterpret_cast<const float4*>(c0 + i), s = *reinterpret_cast<const float4*>(c0 + half + i);
                cs[i] = c.x; cs[i + 1] = c.y; cs[i + 2] = c.z; cs[i + 3] = c.w;
                sn[i] = s.x; sn[i + 1] = s.y; sn[i + 2] = s.z; sn[i + 3] = s.w;
            }
        } else {
            const float2 c = *reinterpret_cast<const float2*>(c0), s = *reinterpret_cast<const float2*>(c0 + half);
            cs[0] = c.x; cs[1] = c.y;
            sn[0] = s.x; sn[1] = s.y;
        }
    }
    const long long page_at = p.page * a.kv_heads;
    for (; r < rows; r += step) {
        const bool is_q = r < a.heads, is_v = r >= a.heads + a.kv_heads;
        const int kh = r - a.heads - (is_v ? a.kv_heads : 0);
        if (is_q || p.keep) {
            T* dst = is_q ? static_cast<T*>(a.q_out) + t * a.out_tok + r * a.out_head
                          : static_cast<T*>(is_v ? a.cv : a.ck) + ((page_at + kh) * a.page_size + p.row) * D;
            if (turn && !is_v) {
                float v[N], o[N];
                Vec<T>::get(u, v);
                if (kPairs) {
#pragma unroll
                    for (int e = 0; e < N; e += 2) {
                        o[e] = v[e] * cs[e / 2] - v[e + 1] * sn[e / 2];
                        o[e + 1] = v[e + 1] * cs[e / 2] + v[e] * sn[e / 2];
                    }
                } else {
                    float b[N], o2[N];
                    Vec<T>::get(w, b);
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        o[e] = v[e] * cs[e] - b[e] * sn[e];
                        o2[e] = b[e] * cs[e] + v[e] * sn[e];
                    }
                    w = Vec<T>::put(o2);
                }
                u = Vec<T>::put(o);
            }
            *reinterpret_cast<uint4*>(dst + (is_v ? vat : at)) = u;
            if ((is_v ? vat2 : at2) >= 0) *reinterpret_cast<uint4*>(dst + (is_v ? vat2 : at2)) = w;
        }
        if (r + step < rows) fetch(r + step);
    }
}

// Any even rotation: one thread per pair or component, in loads of 2 or 4 bytes,
// which bound it.  bf16, 32 + 2 x 4 heads of 80 components: 16000 tokens 146 us
// with 20 of them rotated, against 39 in whole words with all (30 at the copy
// rate); 256 tokens of 64 + 2 x 4 heads 16.8 against 3.4.
template <typename T>
__global__ void append_any_kernel(const AppendArgs a) {
    const int t = blockIdx.x;
    const int half = a.rot / 2, D = a.D;
    const int units = half + (D - a.rot);   // pairs, then components that are not rotated
    grid_launch_dependents();
    grid_dependency_wait();
    const Place p = place_of(a, t, threadIdx.x == 0);
    for (int u = threadIdx.x; u < (a.heads + a.kv_heads) * units; u += blockDim.x) {
        const int h = u / units, c = u - h * units;
        const bool is_q = h < a.heads;
        const int kh = h - a.heads;
        if (!is_q && !p.keep) continue;
        const T* src = is_q ? (const T*)a.q + t * a.q_tok + h * a.q_head : (const T*)a.k + t * a.k_tok + kh * a.k_head;
        T* dst = is_q ? (T*)a.q_out + t * a.out_tok + h * a.out_head
                      : (T*)a.ck + ((p.page * a.kv_heads + kh) * a.page_size + p.row) * D;
        if (c < half) {
            const int i0 = a.interleaved ? 2 * c : c, i1 = a.interleaved ? 2 * c + 1 : c + half;
            const float x = to_float(src[i0]), y = to_float(src[i1]), cs = p.angle[c], sn = p.angle[half + c];
            dst[i0] = from_float<T>(x * cs - y * sn);
            dst[i1] = from_float<T>(y * cs + x * sn);
        } else {
            dst[c + half] = src[c + half];
        }
    }
    if (!p.keep) return;
    for (int u = threadIdx.x; u < a.kv_heads * D; u += blockDim.x) {
        const int h = u / D, c = u - h * D;
        ((T*)a.cv)[((p.page * a.kv_heads + h) * a.page_size + p.row) * D + c] = ((const T*)a.v)[t * a.v_tok + h * a.v_head + c];
    }
}

// Tokens from which blocks are small (64 threads, about five rows each) and
// their number hides the latency; below, more threads share a token.  bf16, 32
// + 2 x 4 heads of 128: 16000 tokens 59.6 (256 threads) against 52.1 us, 6.4
// TB/s; 8000 31.9 / 29.7; 4000 18.2 / 18.3; 256 of 64 + 2 x 4 heads 3.1 / 4.2.
constexpr int kManyTokens = 4000;

template <typename T>
cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
    constexpr int N = Vec<T>::kN;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // whole words: a half of the rotated part (half layout), or all of it
    if (a.interleaved ? a.rot % N != 0 : a.rot / 2 % N != 0) {
        cfg.gridDim = dim3(a.T);
        cfg.blockDim = dim3(256);
        return cudaLaunchKernelEx(&cfg, append_any_kernel<T>, a);
    }
    const bool pairs = a.interleaved || a.rot == 0;
    const int nx = pairs ? a.D / N : a.rot / 2 / N + (a.D - a.rot) / N;
    const int rows = a.heads + 2 * a.kv_heads;
    const bool many = a.T >= kManyTokens && nx <= 64;
    const int most = (many ? 64 : 256) / nx, each = (rows + most - 1) / most;
    const int ny = (rows + each - 1) / each;
    // few tokens: a row per thread, spread over blocks
    cfg.gridDim = dim3(a.T, a.T <= 304 ? each : 1);
    cfg.blockDim = dim3(nx, ny);
    auto launch = [&](auto pair, auto lot) {
        return cudaLaunchKernelEx(&cfg, append_kernel<T, decltype(pair)::value, decltype(lot)::value>, a);
    };
    using Yes = std::true_type;
    using No = std::false_type;
    if (pairs) return many ? launch(Yes{}, Yes{}) : launch(Yes{}, No{});
    return many ? launch(No{}, Yes{}) : launch(No{}, No{});
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
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = cache->dtype == MOE_DTYPE_BF16 ? launch_append<__nv_bfloat16>(a, s) : launch_append<float>(a, s);
    return e == cudaSuccess ? MOE_OK : report(MOE_ERR_CUDA, "append launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
