// append_norm.cu -- appends for models that norm each head of queries and keys
// before the rotation (moe_kv_append_norm), and into a cache of 8-bit numbers
// (moe_kv_append_q8), with the way back (moe_kv_read_q8).
//
// A head's row x becomes x / sqrt(mean(x^2) + eps) * (w + offset), then its
// pairs are rotated as in rope.cu; all in fp32, rounded once.  In 8 bits a
// number is code * scale: the code e4m3 (448 the largest), the scale a power of
// two that a block of consecutive rows of a page and key head share, the
// smallest with which the block's largest component fits.  A power of two costs
// e4m3, a floating format, no accuracy, and a block that has to grow is rescaled
// exactly, but for what falls below the smallest normal code.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cuda_fp16.h>

#include "append.cuh"
#include "pairs.cuh"

namespace moe {

namespace {

// Quotients of slots and blocks without a division, which takes twenty
// instructions, several times a row.  Below 2^31, floor(x / d) = floor(x M / 2^(31 + l))
// with d <= 2^l and M = ceil(2^(31 + l) / d): M d is less than d <= 2^l above
// 2^(31 + l), so x M / 2^(31 + l) less than x / (2^31 d) < 1 / d above x / d.
struct Quotient {
    uint32_t mul, shift, d;
    __device__ __forceinline__ uint32_t small(uint32_t x) const { return d == 1 ? x : __umulhi(x, mul) >> shift; }
    __device__ __forceinline__ long long operator()(long long x) const {   // x >= 0
        return x >> 31 ? x / d : (long long)small((uint32_t)x);
    }
};

Quotient quotient(int d) {
    uint32_t l = 0;
    while ((1u << l) < (uint32_t)d) ++l;
    const uint64_t mul = ((1ull << (31 + l)) + d - 1) / d;   // below 2^32: d > 2^(l - 1)
    return {(uint32_t)mul, l - 1, (uint32_t)d};
}

struct NormArgs {
    AppendArgs a;
    const void *qw, *kw;            // weights, or null: ones
    long long qw_head, kw_head;     // between heads' weights; 0: shared
    int norm;                       // 0: no norm
    float eps, offset;
    float inv_D;
    // the mean's root from the sum: sqrt(D) and D * eps, in two floats each
    float root_hi, root_lo, deps_hi, deps_lo;
    // in 8 bits
    float *ks, *vs;
    int block, nb;                  // rows that share a scale; such blocks of a page
    Quotient by_block, by_nb, by_page;
    int chunk, team_heads;          // tokens in which a thread block looks for blocks, and its heads of keys or values
    int kv_blocks;                  // thread blocks for keys and values, before those for queries
    int split;                      // thread blocks a token's other rows take (0: half of one)
    int G;                          // lanes of a row, a power of two
    int stash;                      // a warp's rounds of rows that wait in shared memory
    int smem_scratch;               // bytes of the kAny rows
};

enum Mode { kHalf = 0, kPairs = 1, kAny = 2 };   // rotation in whole words: halves, pairs; or any

// A lane's two words of a row as pairs of components (word w has those from
// w P on), and the other way.
template <typename T> struct Pairs { static constexpr int P = Vec<T>::kN / 2; };

__device__ __forceinline__ uint64_t as_pair(uint32_t x, uint32_t y) { return pack2(__uint_as_float(x), __uint_as_float(y)); }

__device__ __forceinline__ void widen(const uint4 (&u)[2], uint64_t (&z)[4]) {   // fp32
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        z[2 * w] = as_pair(u[w].x, u[w].y);
        z[2 * w + 1] = as_pair(u[w].z, u[w].w);
    }
}
__device__ __forceinline__ void widen_word(const uint4& u, uint64_t* z) {       // bf16
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = as_pair(w[i] << 16, w[i] & 0xffff0000u);
}
__device__ __forceinline__ void widen(const uint4 (&u)[2], uint64_t (&z)[8]) {
    widen_word(u[0], z);
    widen_word(u[1], z + 4);
}
template <typename T>
__device__ __forceinline__ uint4 narrow(const uint64_t* z) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < Pairs<T>::P; ++i) {
        float x, y;
        unpack2(z[i], x, y);
        if (sizeof(T) == 4) {
            w[(2 * i) & 3] = __float_as_uint(x);
            w[(2 * i + 1) & 3] = __float_as_uint(y);
        } else {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A lane's two words of a row, their first components (-1: none), and the
// rotation's angles for them.
template <typename T, int kMode>
struct Lane {
    static constexpr int N = Vec<T>::kN, P = N / 2;
    int at, at2;
    bool turn;                      // kHalf: the words are rotated with each other
    // kHalf: cosines and sines of the words' pairs of components (i, i + rot / 2),
    // two side by side.  kPairs: of the components' pairs, (c, c) and (-s, s).
    uint64_t cs[kMode == kHalf ? P : kMode == kPairs ? N : 1], sn[kMode == kHalf ? P : kMode == kPairs ? N : 1];
    const float* angle;

    __device__ __forceinline__ Lane(const AppendArgs& a, int x) {
        const int D = a.D;
        if (kMode == kHalf) {
            const int turned = a.rot / 2 / N, rest = (D - a.rot) / N, y = x - turned;
            turn = y < 0;
            at = turn ? x * N : a.rot + y * N;
            at2 = turn ? at + a.rot / 2 : y + (rest + 1) / 2 < rest ? at + (rest + 1) / 2 * N : -1;
            if (!turn && y >= (rest + 1) / 2) at = -1;
        } else {
            const int words = D / N, half = (words + 1) / 2;
            turn = false;
            at = x < half ? x * N : -1;
            at2 = x + half < words && x < half ? (x + half) * N : -1;
        }
        angle = nullptr;
    }
    __device__ __forceinline__ void load_angles(const AppendArgs& a, const float* from) {
        angle = from;
        if (kMode == kAny || !from) return;
        const int half = a.rot / 2;
        if (kMode == kHalf) {
            if (!turn) return;
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                const float4 c = *reinterpret_cast<const float4*>(from + at + 2 * i), s = *reinterpret_cast<const float4*>(from + half + at + 2 * i);
                cs[i] = pack2(c.x, c.y);
                cs[i + 1] = pack2(c.z, c.w);
                sn[i] = pack2(s.x, s.y);
                sn[i + 1] = pack2(s.z, s.w);
            }
        } else {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const int first = w ? at2 : at;
                if (first < 0 || first >= a.rot) continue;
#pragma unroll
                for (int i = 0; i < P; i += 2) {
                    const float2 c = *reinterpret_cast<const float2*>(from + first / 2 + i), s = *reinterpret_cast<const float2*>(from + half + first / 2 + i);
                    cs[w * P + i] = pack2(c.x, c.x);
                    cs[w * P + i + 1] = pack2(c.y, c.y);
                    sn[w * P + i] = pack2(-s.x, s.x);
                    sn[w * P + i + 1] = pack2(-s.y, s.y);
                }
            }
        }
    }
    __device__ __forceinline__ void load(const T* row, uint4 (&u)[2]) const {
        u[0] = u[1] = make_uint4(0, 0, 0, 0);
        if (at >= 0) u[0] = *reinterpret_cast<const uint4*>(row + at);
        if (at2 >= 0) u[1] = *reinterpret_cast<const uint4*>(row + at2);
    }
    __device__ __forceinline__ void store(T* row, const uint4 (&u)[2]) const {
        if (at >= 0) *reinterpret_cast<uint4*>(row + at) = u[0];
        if (at2 >= 0) *reinterpret_cast<uint4*>(row + at2) = u[1];
    }
    __device__ __forceinline__ void store(T* row, const uint64_t (&z)[N]) const {
        if (at >= 0) *reinterpret_cast<uint4*>(row + at) = narrow<T>(z);
        if (at2 >= 0) *reinterpret_cast<uint4*>(row + at2) = narrow<T>(z + P);
    }
    // Whole warp.  kRounded: every product and sum rounded by itself, so that the
    // codes do not depend on what is fused.  scratch: kAny, D floats of this row.
    template <bool kRounded>
    __device__ __forceinline__ void rotate(const AppendArgs& a, uint64_t (&z)[N], float* scratch) const {
        if (a.rot == 0) return;
        if (kMode == kHalf) {
            if (turn)
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const uint64_t x = z[i], y = z[P + i];
                    z[i] = sub2(mul2(x, cs[i]), mul2(y, sn[i]));
                    z[P + i] = kRounded ? add2(mul2(y, cs[i]), mul2(x, sn[i])) : fma2(y, cs[i], mul2(x, sn[i]));
                }
        } else if (kMode == kPairs) {
#pragma unroll
            for (int w = 0; w < 2; ++w)
                if ((w ? at2 : at) >= 0 && (w ? at2 : at) < a.rot)
#pragma unroll
                    for (int i = w * P; i < w * P + P; ++i) {
                        float x, y;
                        unpack2(z[i], x, y);
                        const uint64_t other = mul2(pack2(y, x), sn[i]);
                        z[i] = kRounded ? add2(mul2(z[i], cs[i]), other) : fma2(z[i], cs[i], other);
                    }
        } else {
            // the partner is another lane's: through shared memory
            float q[2 * N];
#pragma unroll
            for (int i = 0; i < N; ++i) unpack2(z[i], q[2 * i], q[2 * i + 1]);
            __syncwarp();
#pragma unroll
            for (int w = 0; w < 2; ++w)
                if ((w ? at2 : at) >= 0)
#pragma unroll
                    for (int e = 0; e < N; ++e) scratch[(w ? at2 : at) + e] = q[w * N + e];
            __syncwarp();
            const int half = a.rot / 2;
#pragma unroll
            for (int w = 0; w < 2; ++w)
                if ((w ? at2 : at) >= 0)
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const int i = (w ? at2 : at) + e;
                        if (i >= a.rot) continue;
                        const bool lower = a.interleaved ? i % 2 == 0 : i < half;
                        const int pair = a.interleaved ? i / 2 : lower ? i : i - half;
                        const float p = scratch[a.interleaved ? i ^ 1 : lower ? i + half : i - half];
                        const float c = angle[pair], t = __fmul_rn(p, angle[half + pair]), x = __fmul_rn(q[w * N + e], c);
                        q[w * N + e] = lower ? __fsub_rn(x, t) : __fadd_rn(x, t);
                    }
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = pack2(q[2 * i], q[2 * i + 1]);
        }
    }
};

// 1 / sqrt(mean of squares + eps) of a row, whose lanes lie side by side.
template <int N>
__device__ __forceinline__ float inverse_root(const NormArgs& n, const uint64_t (&z)[N]) {
    uint64_t s2 = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) s2 = fma2(z[i], z[i], s2);
    float s, t;
    unpack2(s2, s, t);
    s += t;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        if (off < n.G) s += __shfl_xor_sync(0xffffffffu, s, off);
    return rsqrtf(fmaf(s, n.inv_D, n.eps));   // (off by 2 steps of fp32 at most)
}

// The same to the last bit but for rare ties, with sums in two floats: a key's
// code changes by a step of 2^-4 where a last bit decides it, and how many
// lanes a row has should not.
template <int N>
__device__ __forceinline__ float inverse_root_exact(const NormArgs& n, const uint64_t (&z)[N]) {
    auto two_sum2 = [](uint64_t a, uint64_t b, uint64_t& err) {   // Knuth
        const uint64_t s = add2(a, b), bb = sub2(s, a);
        err = add2(sub2(a, sub2(s, bb)), sub2(b, bb));
        return s;
    };
    auto two_sum = [](float a, float b, float& err) {
        const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
        err = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
        return s;
    };
    uint64_t s2 = 0, low2 = 0, err2;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint64_t p = mul2(z[i], z[i]);
        s2 = two_sum2(s2, p, err2);
        // (a bf16's square has 16 bits, and is exact)
        if (N == 4) err2 = add2(err2, fma2(z[i], z[i], sub2(0, p)));
        low2 = add2(low2, err2);
    }
    float s, low, t, err;
    unpack2(s2, s, t);
    s = two_sum(s, t, err);
    unpack2(low2, low, t);
    low = __fadd_rn(__fadd_rn(low, t), err);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        if (off < n.G) {
            const float so = __shfl_xor_sync(0xffffffffu, s, off), lowo = __shfl_xor_sync(0xffffffffu, low, off);
            s = two_sum(s, so, err);
            low = __fadd_rn(__fadd_rn(low, lowo), err);
        }
    s = two_sum(s, n.deps_hi, err);
    if (!(s < INFINITY)) return __frsqrt_rn(s);   // (squares past fp32: 0, as without; NaN)
    low = __fadd_rn(low, __fadd_rn(err, n.deps_lo));
    // y = sqrt(D) (1 + u / 2) r, where u = 1 - (s + low) r^2, by way of s r, about the root
    // of s: r^2 passes fp32 where s is below its smallest normal number (rows of zeros with
    // a tiny eps), and loses bits where s is near its largest.
    const float r = __frsqrt_rn(s), q = __fmul_rn(s, r), qe = __fmaf_rn(s, r, -q);
    float u = __fmaf_rn(-q, r, 1.f);
    u = __fmaf_rn(-qe, r, u);
    u = __fmaf_rn(__fmul_rn(-low, r), r, u);
    const float p = __fmul_rn(r, n.root_hi), pe = __fmaf_rn(r, n.root_hi, -p);
    return __fadd_rn(p, __fmaf_rn(0.5f * u, p, __fmaf_rn(r, n.root_lo, pe)));
}

// x times its row's factor and its weights.
template <typename T, int kMode>
__device__ __forceinline__ void weigh(const Lane<T, kMode>& L, uint64_t (&z)[Vec<T>::kN], float r, const T* weight, float offset) {
    constexpr int N = Vec<T>::kN;
    const uint64_t r2 = pack2(r, r), off2 = pack2(offset, offset);
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = mul2(z[i], r2);
    if (!weight) return;
    uint4 u[2];
    L.load(weight, u);
    uint64_t g[N];
    widen(u, g);
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = mul2(z[i], add2(g[i], off2));
}

// ---- rows that stay in their type -----------------------------------------------
// Bounded by the bytes, and nearly as much by the instructions (two thirds of all
// issue slots): a thread keeps its two words' angles for all rows of the token
// that it goes through, and works on pairs of components.  16000 tokens with 32 + 2
// x 4 heads of 128: 60 us, 5.6 TB/s (50 at the copy rate; fp32 106 of 99); with single
// components and divisions for places 76.
template <typename T, int kMode, bool kCache>
__device__ __forceinline__ void plain_rows(const NormArgs& n, float* scratch, int t, int y, int thread, int threads) {
    constexpr int N = Vec<T>::kN;
    const AppendArgs& a = n.a;
    const int G = n.G, x = thread & (G - 1), g = thread / G, per = threads / G;
    const int rows = kCache ? a.heads + 2 * a.kv_heads : a.heads, step = per * max(n.split, 1);
    Lane<T, kMode> L(a, x);
    uint4 u[2] = {};
    int r = y * per + g;
    const T* src = static_cast<const T*>(a.q) + t * a.q_tok + r * a.q_head;
    const long long src_step = step * a.q_head, out_step = step * a.out_head;
    auto fetch = [&](int to) {
        if (to < a.heads) {
            L.load(src, u);
        } else if (kCache && to < rows) {
            const bool is_v = to >= a.heads + a.kv_heads;
            const int kh = to - a.heads - (is_v ? a.kv_heads : 0);
            L.load(is_v ? static_cast<const T*>(a.v) + t * a.v_tok + kh * a.v_head
                        : static_cast<const T*>(a.k) + t * a.k_tok + kh * a.k_head, u);
        }
        src += src_step;
    };
    // The first row is on its way before the token's place and angles are read
    // (two loads one after the other), each next one while a row is worked on.
    fetch(r);
    const Place p = place_of(a, t, thread == 0 && y == 0);
    L.load_angles(a, p.angle);
    const long long page_at = p.page * a.kv_heads;
    T* out = static_cast<T*>(a.q_out) + t * a.out_tok + r * a.out_head;
    for (int r0 = y * per; r0 < rows; r0 += step, r += step, out += out_step) {   // whole warps together
        const bool is_q = r < a.heads, is_v = kCache && r >= a.heads + a.kv_heads, on = r < rows && (is_q || p.keep);
        const int kh = r - a.heads - (is_v ? a.kv_heads : 0);
        T* dst = out;
        if (kCache && !is_q) dst = static_cast<T*>(is_v ? a.cv : a.ck) + ((page_at + kh) * a.page_size + p.row) * a.D;
        uint64_t z[N];
        widen(u, z);
        if (kCache && on && is_v) L.store(dst, u);
        fetch(r + step);
        if (n.norm) {
            const float f = inverse_root(n, z);
            const T* weight = static_cast<const T*>(is_q ? n.qw : n.kw);
            if (on && !is_v) weigh(L, z, f, weight ? weight + (is_q ? r * n.qw_head : kh * n.kw_head) : nullptr, n.offset);
        }
        L.template rotate<false>(a, z, scratch + g * a.D);
        if (on && !is_v) L.store(dst, z);
    }
}

// ---- 8 bits -----------------------------------------------------------------------

// The smallest power of two s, at least 2^-64, with most <= 448 s.
__device__ __forceinline__ float scale_for(float most) {
    const uint32_t b = __float_as_uint(most);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u);   // 448 = 1.75 * 2^8
    return __uint_as_float((uint32_t)(max(e, -64) + 127) << 23);
}

__device__ __forceinline__ uint32_t code2(float x0, float x1) {   // x0's code in the low byte
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
    return r;
}

__device__ __forceinline__ void values2(uint32_t codes, float& x0, float& x1) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x0 = f.x;
    x1 = f.y;
}

// x / scale: a product where the scale is a power of two, which is the same.
struct Divide {
    float scale, inv;
    bool power;
    __device__ __forceinline__ Divide(float s) {
        scale = s;
        inv = 1.f / s;
        power = (__float_as_uint(s) & 0x7fffffu) == 0;
    }
};

// The codes of a row's words.  wild: components that are not finite may be
// among them; their code is NaN.
template <typename T, int kMode>
__device__ __forceinline__ void store_codes(const Lane<T, kMode>& L, uint8_t* row, const uint64_t (&z)[Vec<T>::kN], const Divide& by,
                                            bool wild) {
    constexpr int N = Vec<T>::kN;
    const uint64_t inv2 = pack2(by.inv, by.inv);
    uint32_t c[N];   // of two components each
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float x, y;
        unpack2(mul2(z[i], inv2), x, y);
        c[i] = code2(x, y);
    }
    if (!by.power || wild)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float x, y;
            unpack2(z[i], x, y);
            c[i] = code2(fabsf(x) < INFINITY ? __fdiv_rn(x, by.scale) : NAN, fabsf(y) < INFINITY ? __fdiv_rn(y, by.scale) : NAN);
        }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int at = w ? L.at2 : L.at, i = w * (N / 2);
        if (at < 0) continue;
        if (N == 8) *reinterpret_cast<uint2*>(row + at) = make_uint2(c[i] | c[i + 1] << 16, c[(i + 2) % N] | c[(i + 3) % N] << 16);
        else *reinterpret_cast<uint32_t*>(row + at) = c[i] | c[i + 1] << 16;
    }
}

constexpr uint32_t kInfBits = 0x7f800000u;

// The largest magnitude's bits; a NaN's are above all.
template <int N>
__device__ __forceinline__ uint32_t most_bits(const uint64_t (&z)[N], bool finite_only) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float x, y;
        unpack2(z[i], x, y);
        if (finite_only) {
            x = fabsf(x) < INFINITY ? x : 0.f;
            y = fabsf(y) < INFINITY ? y : 0.f;
        }
        asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(x), "f"(y));
    }
    return __float_as_uint(m);
}

// Keys and values: a thread block looks for the blocks of rows that begin among
// `chunk` tokens (the token before, skipped ones left out, is in another block)
// and takes each with all its tokens, for one head after the other.  Rows go
// round the warps, 32 / G at a time; between a block's maximum and its codes
// they wait in shared memory, those past a warp's n.stash rounds are read again.
//
// What takes the time is a chain: slots and positions around the chunk; the
// search; rows, angles and the scale; their maximum over the warps; codes.  256
// drafted tokens wait for little else (8.1 us; their bytes would take 1.4).  Of
// a prompt many such chains have to be under way, and each has to be short: with one
// warp for all of a block's rows of one head 16000 tokens took 112 us, with four
// 106, with the search shared by eight heads 93, with one round of rows at a time
// (registers) 81, fewer instructions 74; 48 for the bytes.  The registers that so many
// thread blocks leave do not hold everything: 72 bytes of spill stores and 56 of loads in
// bf16 (240 and 204 for rotations that are not on words).  fp32: 16000 117 us of 92; with a
// scale for every row (bf16) 63.
constexpr int kWarps = 4;
constexpr int kStash = 4;       // rounds of a warp that shared memory holds: 8 KB in bf16
constexpr int kSkipped = 256;   // a token this far behind the last of its block still belongs to it

struct Found {                  // a block: its tokens, and whether its first row is among them
    long long block;
    int t0, count, begun;
};

struct Window {                 // from 32 tokens before the chunk on
    long long slots[96];
    int positions[64];          // from the chunk on
    uint32_t most[2][kWarps];
    Found found;
    uint32_t pad[18];
};
static_assert(sizeof(Window) % 128 == 0, "the stash follows");

template <typename T, int kMode>
__device__ __forceinline__ void block_rows(const NormArgs& n, unsigned char* smem, float* scratch, int unit) {
    constexpr int N = Vec<T>::kN;
    const AppendArgs& a = n.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = n.G, x = lane & (G - 1), g = lane / G, per = 32 / G;
    // heads, keys and values in turn: hv0 .. hv1 - 1
    const int groups = (2 * a.kv_heads + n.team_heads - 1) / n.team_heads, part = unit % groups;
    const int hv0 = part * n.team_heads, hv1 = min(2 * a.kv_heads, hv0 + n.team_heads);
    const int c0 = unit / groups * n.chunk, c1 = c0 + min(n.chunk, a.T - c0);
    Window& W = *reinterpret_cast<Window*>(smem);
    ulonglong2* stash = reinterpret_cast<ulonglong2*>(smem + sizeof(Window)) + (size_t)warp * n.stash * (N / 2) * 32 + lane;
    auto block_of = [&](long long slot) -> long long {   // -1: none
        if (slot < 0 || slot >= a.n_slots) return -1;
        return n.by_block(slot);
    };
    const int tw = c0 - 32 + (int)threadIdx.x;
    const bool in = threadIdx.x < 96 && tw >= 0 && tw < a.T;
    const long long slot_w = in ? a.slots[tw] : -1;
    const int position_w = in && threadIdx.x >= 32 && a.rot > 0 ? a.positions[tw] : 0;
    if (a.heads == 0 && a.rot > 0 && part == 0 && (int)threadIdx.x < c1 - c0) {   // (with queries these are looked at in plain_rows)
        // positions of tokens that write nothing; those of others are looked at with their rows
        const long long slot = a.slots[c0 + threadIdx.x];
        const int m = a.positions[c0 + threadIdx.x];
        if ((slot < 0 || slot >= a.n_slots) && (m < 0 || m >= a.n_pos)) raise_flag(a.flags, kFlagBadIndex);
    }
    if (n.chunk == 1 && n.block > 1 && c0 > 0) {   // most thread blocks find nothing, and make room at once
        const long long mine = block_of(a.slots[c0]);
        if (mine >= 0 && mine == block_of(a.slots[c0 - 1])) return;
    }
    if (threadIdx.x < 96) {
        W.slots[threadIdx.x] = slot_w;
        if (threadIdx.x >= 32) W.positions[threadIdx.x - 32] = position_w;
    }
    __syncthreads();
    // one head's
    bool is_v = false;
    uint8_t* codes = nullptr;
    float* scales = nullptr;
    const T *src = nullptr, *weight = nullptr;
    long long tok = 0;
    int h = 0;
    auto take = [&](int hv) {
        h = hv >> 1;
        is_v = hv & 1;
        codes = static_cast<uint8_t*>(is_v ? a.cv : a.ck) + (size_t)h * a.page_size * a.D;
        scales = (is_v ? n.vs : n.ks) + (size_t)h * n.nb;
        src = static_cast<const T*>(is_v ? a.v : a.k) + h * (is_v ? a.v_head : a.k_head);
        tok = is_v ? a.v_tok : a.k_tok;
        weight = static_cast<const T*>(n.kw);
        if (weight) weight += h * n.kw_head;
    };
    Lane<T, kMode> L(a, x);

    auto slot_at = [&](int t) -> long long {   // -1: past the tokens
        const int i = t - c0 + 32;
        return (unsigned)i < 96u ? W.slots[i] : t < a.T ? a.slots[t] : -1;
    };
    auto finish = [&](int t, bool on, uint64_t (&v)[N]) {   // whole warp: a raw row to what is stored
        if (is_v) return;
        if (a.rot > 0) {
            const int i = t - c0;
            int m = !on ? 0 : (unsigned)i < 64u ? W.positions[i] : a.positions[t];
            if (m < 0 || m >= a.n_pos) {
                if (x == 0 && h == 0) raise_flag(a.flags, kFlagBadIndex);
                m = m < 0 ? 0 : a.n_pos - 1;
            }
            L.load_angles(a, a.rope + (size_t)m * a.rot);
        }
        if (n.norm) weigh(L, v, inverse_root_exact(n, v), weight, n.offset);
        L.template rotate<true>(a, v, scratch + g * a.D);
    };
    auto fetch = [&](int t, bool on, uint4 (&u)[2]) {
        u[0] = u[1] = make_uint4(0, 0, 0, 0);
        if (on) L.load(src + t * tok, u);
    };

    if (n.block == 1) {   // every row has its scale: rows side by side
        for (int i = warp * per; i < n.chunk; i += kWarps * per) {
            const int t = c0 + i + g;
            const long long slot = t < c1 ? slot_at(t) : -1;
            const bool on = slot >= 0 && slot < a.n_slots;
            if (slot >= a.n_slots && x == 0 && part == 0) raise_flag(a.flags, kFlagBadIndex);
            const long long page = on ? n.by_page(slot) : 0;
            const size_t at = (size_t)page * a.kv_heads * a.page_size + (on ? slot - page * a.page_size : 0);
            for (int hv = hv0; hv < hv1; ++hv) {
                take(hv);
                uint4 u[2];
                uint64_t v[N];
                fetch(t, on, u);
                widen(u, v);
                finish(t, on, v);
                auto row_most = [&](bool finite_only) {
                    uint32_t m = most_bits(v, finite_only);
                    for (int off = G >> 1; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
                    return m;
                };
                uint32_t m = row_most(false);
                const bool wild = __any_sync(0xffffffffu, m >= kInfBits);
                if (wild) m = row_most(true);
                if (!on) continue;
                const float scale = scale_for(__uint_as_float(m));
                if (x == 0) scales[at] = scale;
                store_codes(L, codes + at * a.D, v, Divide(scale), wild);
            }
        }
        return;
    }

    // The first warp finds the blocks, one after the other.
    long long mine = -1;
    uint32_t todo = 0, turn = 0;
    if (warp == 0) {
        const int t1 = c0 + lane;
        if (t1 < c1) {
            const long long slot = slot_at(t1);
            mine = block_of(slot);
            if (slot >= a.n_slots && part == 0) raise_flag(a.flags, kFlagBadIndex);
        }
        long long before = -1;
        if (mine >= 0)
            for (int p = t1 - 1; p >= max(0, t1 - kSkipped) && before < 0; --p)
                before = block_of(p >= c0 - 32 ? slot_at(p) : a.slots[p]);
        todo = __ballot_sync(0xffffffffu, mine >= 0 && before != mine);
    }
    for (;;) {
        if (warp == 0) {
            Found f = {0, 0, 0, 0};
            if (todo) {
                const int first = __ffs(todo) - 1;
                todo &= todo - 1;
                f.t0 = c0 + first;
                f.block = __shfl_sync(0xffffffffu, mine, first);
                // the span of its tokens, and whether its first row is among them
                int last = 0;
                for (int base = 0;; base += 32) {
                    const int t = f.t0 + base + lane;
                    const long long slot = slot_at(t), other = block_of(slot);
                    const uint32_t ends = __ballot_sync(0xffffffffu, t >= a.T || (other >= 0 && other != f.block));
                    const uint32_t until = ends ? (1u << (__ffs(ends) - 1)) - 1u : ~0u;
                    const uint32_t ins = __ballot_sync(0xffffffffu, other == f.block) & until;
                    const uint32_t firsts = __ballot_sync(0xffffffffu, other == f.block && slot == f.block * n.block) & until;
                    if (ins) {
                        if (base + __ffs(ins) - 1 - last > kSkipped) break;
                        f.begun |= firsts != 0;
                        last = base + 31 - __clz(ins);
                    }
                    if (ends || base + 32 - last > kSkipped) break;
                }
                f.count = last + 1;
            }
            if (lane == 0) W.found = f;
        }
        __syncthreads();
        const Found found = W.found;
        const long long b = found.block;
        const int t0 = found.t0, count = found.count;
        const bool begun = found.begun != 0;
        if (count == 0) break;
        const long long page = n.by_nb(b);
        const int b0 = (int)(b - page * n.nb) * n.block;              // the block's first row of the page
        const size_t head_at = (size_t)page * a.kv_heads * a.page_size;   // of key head 0
        const size_t scale_at0 = (size_t)page * a.kv_heads * n.nb + (b - page * n.nb);
        auto slot_of = [&](int i) -> long long {   // of the span's token i; -1: skipped
            const long long slot = i < count ? slot_at(t0 + i) : -1;
            return slot < a.n_slots ? slot : -1;
        };
        for (int hv = hv0; hv < hv1; ++hv) {
            take(hv);
            float* scale_at = scales + scale_at0;
            const float old = begun ? 0.f : *scale_at;
            if (!begun)   // the codes that it holds, should it have to grow
                for (long long i = threadIdx.x * 128; i < (long long)n.block * a.D; i += kWarps * 32 * 128)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(codes + (head_at + b0) * a.D + i));

            constexpr int kParts = N / 2;   // a lane's pairs, two at a time
            // The span's rows as they are stored, skipped ones zeros: their maximum,
            // that of what is finite, or, as codes, to the cache.  (One body, since
            // its code is long.)
            uint32_t m = 0;
            bool wild = false;
            float scale = 0.f;
            auto pass = [&](bool store) {
                const Divide by(scale);
                for (int j = 0; (j * kWarps + warp) * per < count; ++j) {   // this warp's rounds
                    const int i = (j * kWarps + warp) * per + g;
                    const long long slot = slot_of(i);
                    ulonglong2* at = stash + j * kParts * 32;
                    uint64_t v[N];
                    if (store && j < n.stash) {
#pragma unroll
                        for (int z = 0; z < kParts; ++z) {
                            const ulonglong2 f = at[z * 32];
                            v[2 * z] = f.x;
                            v[2 * z + 1] = f.y;
                        }
                    } else {
                        uint4 u[2];
                        fetch(t0 + i, slot >= 0, u);
                        widen(u, v);
                        finish(t0 + i, slot >= 0, v);
                    }
                    if (store) {
                        if (slot >= 0) store_codes(L, codes + (head_at + (slot - page * a.page_size)) * a.D, v, by, wild);
                    } else {
                        m = max(m, most_bits(v, wild));
                        if (j < n.stash)
#pragma unroll
                            for (int z = 0; z < kParts; ++z) at[z * 32] = make_ulonglong2(v[2 * z], v[2 * z + 1]);
                    }
                }
            };
            bool store = false;
#pragma unroll 1
            for (;;) {
                pass(store);
                if (store) break;
                m = __reduce_max_sync(0xffffffffu, m);
                uint32_t* most = W.most[turn++ & 1];   // (the other one may still be read)
                if (lane == 0) most[warp] = m;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < kWarps; ++w) m = max(m, most[w]);
                if (!wild && m >= kInfBits) {   // once more, without those
                    wild = true;
                    m = 0;
                    continue;
                }
                const float need = scale_for(__uint_as_float(m));
                scale = old >= need && old < INFINITY ? old : need;
                if (scale != old) {
                    if (threadIdx.x == 0) *scale_at = scale;
                    if (!begun) {
                        // rows that the block holds already (all of them: those that this call writes follow)
                        const float f = old > 0.f && old < INFINITY ? old / scale : 0.f;   // 0: there was no scale, so no values
                        for (long long i = threadIdx.x; i < (long long)n.block * a.D / 16; i += kWarps * 32) {
                            uint4* p = reinterpret_cast<uint4*>(codes + (head_at + b0) * a.D) + i;
                            uint4 c = *p;
                            uint32_t* w = &c.x;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float y[4];
                                values2(w[k] & 0xffffu, y[0], y[1]);
                                values2(w[k] >> 16, y[2], y[3]);
                                w[k] = f == 0.f ? 0u : code2(y[0] * f, y[1] * f) | code2(y[2] * f, y[3] * f) << 16;
                            }
                            *p = c;
                        }
                        __syncthreads();   // before rows are written over them
                    }
                }
                store = true;
            }
        }
    }
}

// Thread blocks on an SM.  6 / 7 (72 registers) / 8: 16000 tokens of a prompt 78.6 / 75.0 /
// 72.2 us, 4000 23.6 / 22.0 / 21.9, 1000 9.9 / 11.0 / 11.8, 256 drafted ones of 16 requests
// 8.9 / 9.5 / 9.9, 1000 single ones 43 / 31 / 31.
constexpr int kBounds = 7;

// kMany: small thread blocks, many on an SM (16000 tokens with 14 of them 61 us, 12 66, 18 68).
template <typename T, int kMode, bool kMany>
__global__ void __launch_bounds__(kMany ? 64 : 256, kMany ? 14 : 2) append_norm_kernel(const NormArgs n) {
    extern __shared__ __align__(128) unsigned char smem[];   // kAny: D floats a row
    grid_launch_dependents();
    grid_dependency_wait();
    const int t = blockIdx.x / n.split;
    plain_rows<T, kMode, true>(n, reinterpret_cast<float*>(smem), t, blockIdx.x - t * n.split, threadIdx.x, blockDim.x);
}

template <typename T, int kMode>
__global__ void __launch_bounds__(32 * kWarps, kBounds) append_q8_kernel(const NormArgs n) {
    extern __shared__ __align__(128) unsigned char smem[];   // kAny: D floats a row; the window, stashes
    float* scratch = reinterpret_cast<float*>(smem);
    grid_launch_dependents();
    grid_dependency_wait();
    int u = blockIdx.x;
    if (u < n.kv_blocks) {
        block_rows<T, kMode>(n, smem + n.smem_scratch, scratch + (size_t)(threadIdx.x >> 5) * (32 / n.G) * n.a.D, u);
        return;
    }
    // Queries: a token's by several thread blocks, or two tokens' by one.
    u -= n.kv_blocks;
    const int threads = n.split > 0 ? 32 * kWarps : 16 * kWarps, thread = threadIdx.x & (threads - 1);
    const int t = n.split > 0 ? u / n.split : 2 * u + (threadIdx.x >= 16 * kWarps), y = n.split > 0 ? u - t * n.split : 0;
    if (t < n.a.T) plain_rows<T, kMode, false>(n, scratch + (threadIdx.x - thread) / n.G * n.a.D, t, y, thread, threads);
}

// A thread block takes up to eight heads' keys or values, which share the search
// for blocks, as long as there are about as many thread blocks as run at once.  Up to
// 8 / 4 / 2 / 1: 16000 tokens 75.0 / 77.6 / 81.8 / 90.1 us, 4000 22.0 / 22.1 / 22.0 / 23.9
// (44.7 with eight whatever their number).
constexpr int kTeamHeads = 8, kTeams = 1000;
// The three forms of the append to a bf16 or fp32 cache: a token's rows spread over thread
// blocks, a row a thread, up to kSpread tokens; a thread block of 256 threads a token; small
// ones from kManyNorm on.  Tokens, spread / 256 threads / small, us:
//   32 + 2 x 4 heads of 128  100 3.1 / 3.3 / 4.9, 128 3.0 / 3.6 / 5.0, 200 4.7 / 3.7 / 5.0,
//                            304 5.0 / 3.6 / 5.0, 400 7.7 / 6.7 / 6.0, 600 10.7 / 7.9 / 7.2,
//                            800 14.4 / 10.7 / 8.2, 1000 17.2 / 13.4 / 8.2, 4000 63 / 43 / 17
//   8 + 2 x 1 of 128         200 2.9 / 2.9 / 3.4, 400 4.5 / 4.5 / 3.6, 800 6.4 / 6.5 / 4.6
//   32 + 2 x 4 of 256        100 3.1 / 3.9 / 7.4, 200 5.8 / 4.9 / 8.6, 400 10.9 / 8.9 / 9.5,
//                            600 15.5 / 9.8 / 11.1, 800 19.8 / 13.3 / 13.1
// (304 tokens are all on the SMs at once in blocks of 256 threads, 400 are not.)  A number
// of tokens alone is a coarse border: between 400 and 800 it costs up to 40 % with few heads.
constexpr int kManyNorm = 800, kSpread = 128;
// The same for the queries beside a cache in 8 bits, where thread blocks for keys and values
// run with them: two tokens a thread block above.  Spread / two, us: single tokens 64 6.0 /
// 7.5, 200 11.3 / 14.1, 304 16.7 / 17.2, 600 28.0 / 27.8, 1000 31.4 / 30.8; of a prompt 200 6.7
// / 6.6, 600 8.4 / 8.5.
constexpr int kSpread8 = 304;

template <typename T, bool kQ8>
cudaError_t launch_append_norm(NormArgs n, cudaStream_t s) {
    constexpr int N = Vec<T>::kN;
    const AppendArgs& a = n.a;
    const bool any = a.interleaved ? a.rot % N != 0 : a.rot / 2 % N != 0;
    const bool half = !any && !a.interleaved && a.rot > 0;
    const int lanes = half ? a.rot / 2 / N + ((a.D - a.rot) / N + 1) / 2 : (a.D / N + 1) / 2;
    n.G = 1;
    while (n.G < lanes) n.G *= 2;
    const bool many = a.T >= kManyNorm;
    const int threads = kQ8 ? 32 * kWarps : many ? 64 : 256, per = threads / n.G;
    const int rows = kQ8 ? a.heads : a.heads + 2 * a.kv_heads, each = (rows + per - 1) / per;
    n.split = a.T <= (kQ8 ? kSpread8 : kSpread) ? (each > 0 ? each : 1) : kQ8 ? 0 : 1;
    n.smem_scratch = any ? (per * a.D * 4 + 127) / 128 * 128 : 0;   // at most 2 N components of 256 threads: 16 KB
    long long blocks = rows <= 0 ? 0 : n.split > 0 ? (long long)a.T * n.split : ((long long)a.T + 1) / 2;
    size_t smem = n.smem_scratch;
    if (kQ8) {
        // Few tokens may lie in a block each, which a search takes one after the other; many
        // are mostly a request's.  A stretch of 1 / 4 / a block's 16 tokens, us: as many requests
        // 256 11.0 / 16.2 / 50, 257 11.0 / 16.1 / 50, 1000 29.0 / 30.8 / 55, 1025 29.7 / 31.3 / 55,
        // 4000 97 / 95 / 108; two tokens a request 1024 24.7 / 22.9 / 35.8, 2048 44 / 42 / 41; eight
        // 512 15.2 / 11.6 / 16.9, 2048 28.9 / 27.6 / 24.1; one request 256 7.6 / 6.0 / 8.0, 1000 24.4
        // / 10.9 / 10.5, 1025 24.5 / 10.9 / 10.6, 4000 32.8 / 29.9 / 21.8.  (What counts is how many
        // blocks begin in a stretch, which the host does not know: single tokens cost up to 1.7
        // times more just past a border.)
        n.chunk = n.block == 1 ? kWarps * (32 / n.G) : a.T <= 256 ? 1 : a.T <= 1024 ? 4 : n.block < 32 ? n.block : 32;
        const long long chunks = ((long long)a.T + n.chunk - 1) / n.chunk;
        n.team_heads = (int)std::max(1LL, std::min((long long)std::min(kTeamHeads, 2 * a.kv_heads), chunks * 2 * a.kv_heads / kTeams));
        const long long units = chunks * ((2 * a.kv_heads + n.team_heads - 1) / n.team_heads);
        if (units > 0x7fffffffLL) return cudaErrorInvalidValue;
        n.kv_blocks = (int)units;
        n.by_block = quotient(n.block);
        n.by_nb = quotient(n.nb);
        n.by_page = quotient(a.page_size);
        blocks += units;
        const int round = kWarps * (32 / n.G), rounds = (std::min(n.block, a.T) + round - 1) / round;
        n.stash = n.block == 1 ? 0 : std::min(rounds, kStash);
        smem += sizeof(Window) + (size_t)kWarps * n.stash * N * 8 * 32;   // below 48 KB
    }
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    auto launch = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, n); };
    if constexpr (kQ8)
        return any ? launch(append_q8_kernel<T, kAny>) : half ? launch(append_q8_kernel<T, kHalf>) : launch(append_q8_kernel<T, kPairs>);
    else if (many)
        return any ? launch(append_norm_kernel<T, kAny, true>) : half ? launch(append_norm_kernel<T, kHalf, true>)
                                                                     : launch(append_norm_kernel<T, kPairs, true>);
    else
        return any ? launch(append_norm_kernel<T, kAny, false>) : half ? launch(append_norm_kernel<T, kHalf, false>)
                                                                      : launch(append_norm_kernel<T, kPairs, false>);
}

// ---- reading back -------------------------------------------------------------------
// Bounded by the bytes: 131000 tokens of 4 heads of 128 take 63 us, 6.4 TB/s (with
// each thread working out its tokens' places 88, two thirds of it instructions), to fp32
// 104 of 100.
// A thread block has some tokens, whose places it works out once; a thread 16 bytes of the result in kReadTokens of them at a time, all of
// whose codes are on their way at once.
struct ReadArgs {
    const uint8_t *ck, *cv;
    const float *ks, *vs;
    const long long* slots;
    void *k, *v;                // one of them may be null
    uint32_t* flags;
    long long n_slots, k_tok, k_head, v_tok, v_head;
    int T, kv_heads, D, page_size, nb, tokens;
    Quotient by_block, by_page;
};

constexpr int kReadTokens = 4;
// A thread block's tokens: sixteen where they are many, else four.  Four / sixteen, us: 4
// key heads of 128 4000 4.6 / 5.5, 16000 10.6 / 11.6, 32000 18.0 / 18.3, 48000 25.6 / 25.3,
// 65000 33.8 / 32.9; to fp32 16000 16.4 / 18.0, 24000 23.2 / 22.3, 65000 58.4 / 53.7; 8 of 256
// 32000 63.5 / 64.4, 48000 93.9 / 92.7; 1 of 128, whose thread blocks are smaller, 4000 2.4 /
// 2.4, 16000 5.8 / 4.6, 32000 8.6 / 7.0, 65000 16.8 / 10.7.
constexpr int kReadMany = 16;
constexpr int kManyRead = 32768;

template <typename T>
__global__ void __launch_bounds__(256) read_q8_kernel(const ReadArgs a) {
    constexpr int N = Vec<T>::kN;
    __shared__ longlong2 place[kReadMany];      // a token's row and scale of key head 0; -1: none
    grid_launch_dependents();
    grid_dependency_wait();
    const int t0 = blockIdx.x * a.tokens, per = a.D / N, words = 2 * a.kv_heads * per;
    if ((int)threadIdx.x < a.tokens) {
        const int t = t0 + threadIdx.x;
        const long long slot = t < a.T ? a.slots[t] : -1;
        longlong2 at = make_longlong2(-1, -1);
        if (slot >= a.n_slots) {
            if (blockIdx.y == 0) raise_flag(a.flags, kFlagBadIndex);
        } else if (slot >= 0) {
            const long long page = a.by_page(slot), head = page * a.kv_heads;
            const int row = (int)(slot - page * a.page_size);
            at.x = (head * a.page_size + row) * a.D;
            at.y = head * a.nb + a.by_block.small((uint32_t)row);
        }
        place[threadIdx.x] = at;
    }
    __syncthreads();
    for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < words * (a.tokens / kReadTokens); i += gridDim.y * blockDim.x) {
        const int part = i / words, u = i - part * words, hv = u / per, at = (u - hv * per) * N;
        const bool is_v = hv >= a.kv_heads;
        const int h = is_v ? hv - a.kv_heads : hv;
        T* out = static_cast<T*>(is_v ? a.v : a.k);
        if (!out) continue;
        const uint8_t* codes = (is_v ? a.cv : a.ck) + (size_t)h * a.page_size * a.D + at;
        const float* scales = (is_v ? a.vs : a.ks) + (size_t)h * a.nb;
        const long long tok = is_v ? a.v_tok : a.k_tok;
        out += (t0 + part * kReadTokens) * tok + h * (is_v ? a.v_head : a.k_head) + at;
        uint2 c[kReadTokens];
        float scale[kReadTokens];
        bool on[kReadTokens];
#pragma unroll
        for (int x = 0; x < kReadTokens; ++x) {
            const longlong2 p = place[part * kReadTokens + x];
            on[x] = p.x >= 0;
            if (!on[x]) continue;
            if (N == 8) c[x] = *reinterpret_cast<const uint2*>(codes + p.x);
            else c[x].x = *reinterpret_cast<const uint32_t*>(codes + p.x);
            scale[x] = scales[p.y];
        }
#pragma unroll
        for (int x = 0; x < kReadTokens; ++x, out += tok) {
            if (!on[x]) continue;
            const uint64_t by = pack2(scale[x], scale[x]);
            uint64_t z[N / 2];
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
                float y0, y1;
                values2((e < 2 ? c[x].x : c[x].y) >> (e & 1) * 16, y0, y1);
                z[e] = mul2(pack2(y0, y1), by);
            }
            *reinterpret_cast<uint4*>(out) = narrow<T>(z);
        }
    }
}

template <typename T>
cudaError_t launch_read(ReadArgs a, cudaStream_t s) {
    const bool many = a.T >= kManyRead;
    a.tokens = many ? kReadMany : kReadTokens;
    const long long words = 2LL * a.kv_heads * (a.D / Vec<T>::kN) * (a.tokens / kReadTokens);
    const int threads = words < 256 ? (int)(words + 31) / 32 * 32 : 256;
    const long long y = many ? 1 : (words + threads - 1) / threads;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)(((long long)a.T + a.tokens - 1) / a.tokens), (unsigned)(y < 64 ? y : 64));
    cfg.blockDim = dim3(threads);
    return cudaLaunchKernelEx(&cfg, read_q8_kernel<T>, a);
}

moe_status fill_norm(const moe_head_norm* p, const AppendArgs& a, NormArgs& n) {
    if (!p) return MOE_OK;
    if (!(p->eps > 0.f) || !(p->eps < INFINITY)) return report(MOE_ERR_ARG, "eps must be positive and finite");
    if (!std::isfinite(p->offset)) return report(MOE_ERR_ARG, "offset is not finite");
    if (p->per_head != 0 && p->per_head != 1) return report(MOE_ERR_ARG, "per_head must be 0 or 1");
    if (!aligned(p->q_weight, 16) || !aligned(p->k_weight, 16)) return report(MOE_ERR_ARG, "a weight is not 16-byte aligned");
    n.norm = 1;
    n.qw = p->q_weight;
    n.kw = p->k_weight;
    n.qw_head = n.kw_head = p->per_head ? a.D : 0;
    n.eps = p->eps;
    n.offset = p->offset;
    n.inv_D = (float)(1.0 / a.D);
    const double root = std::sqrt((double)a.D), deps = (double)p->eps * a.D;
    n.root_hi = (float)root;
    n.root_lo = (float)(root - n.root_hi);
    n.deps_hi = (float)deps;
    n.deps_lo = (float)(deps - n.deps_hi);
    return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_kv_append_norm(const void* q, const void* k, const void* v, const float* rope, const int32_t* positions,
                              const int64_t* slots, const moe_append_params* p, const moe_head_norm* norm,
                              const moe_kv_cache* cache, void* q_out, void* workspace, size_t workspace_bytes,
                              moe_stream_t stream) {
    moe_status st = check_cache(cache, false);
    if (st != MOE_OK) return st;
    if (!norm) return report(MOE_ERR_ARG, "norm is NULL");
    NormArgs n{};
    if ((st = fill_append(q, k, v, rope, positions, slots, p, cache, q_out, workspace, workspace_bytes, n.a)) != MOE_OK) return st;
    const bool bf16 = cache->dtype == MOE_DTYPE_BF16;
    n.a.D = cache->head_dim;
    if ((st = fill_norm(norm, n.a, n)) != MOE_OK || n.a.T == 0) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = bf16 ? launch_append_norm<__nv_bfloat16, false>(n, s) : launch_append_norm<float, false>(n, s);
    return e == cudaSuccess ? MOE_OK : report(MOE_ERR_CUDA, "append launch: %s", cudaGetErrorString(e));
}

moe_status moe_kv_append_q8(const void* q, const void* k, const void* v, const float* rope, const int32_t* positions,
                            const int64_t* slots, const moe_append_params* p, const moe_head_norm* norm,
                            const moe_kv_cache_q8* cache, void* q_out, void* workspace, size_t workspace_bytes,
                            moe_stream_t stream) {
    moe_kv_cache plain;
    moe_status st = check_cache_q8(cache, false, plain);
    if (st != MOE_OK) return st;
    NormArgs n{};
    if ((st = fill_append(q, k, v, rope, positions, slots, p, &plain, q_out, workspace, workspace_bytes, n.a)) != MOE_OK) return st;
    const bool bf16 = cache->dtype == MOE_DTYPE_BF16;
    n.a.D = cache->head_dim;
    if ((st = fill_norm(norm, n.a, n)) != MOE_OK || n.a.T == 0) return st;
    if (norm && !std::isfinite(n.deps_hi)) return report(MOE_ERR_ARG, "eps=%g times head_dim=%d passes fp32", norm->eps, n.a.D);
    n.ks = cache->k_scale;
    n.vs = cache->v_scale;
    n.block = cache->block;
    n.nb = cache->page_size / cache->block;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = bf16 ? launch_append_norm<__nv_bfloat16, true>(n, s) : launch_append_norm<float, true>(n, s);
    return e == cudaSuccess ? MOE_OK : report(MOE_ERR_CUDA, "append launch: %s", cudaGetErrorString(e));
}

moe_status moe_kv_read_q8(const int64_t* slots, const moe_read_params* p, const moe_kv_cache_q8* cache, void* k_out, void* v_out,
                          void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    moe_kv_cache plain;
    moe_status st = check_cache_q8(cache, false, plain);
    if (st != MOE_OK) return st;
    if (!p) return report(MOE_ERR_ARG, "params is NULL");
    if (p->T < 0) return report(MOE_ERR_ARG, "T=%d is negative", p->T);
    if (workspace_bytes < MOE_ATTENTION_WORKSPACE_MIN || !workspace || !aligned(workspace, 256))
        return report(MOE_ERR_WORKSPACE, "workspace missing, not 256-byte aligned or below %d bytes", MOE_ATTENTION_WORKSPACE_MIN);
    if (p->T == 0) return MOE_OK;
    if (!slots || !aligned(slots, 8)) return report(MOE_ERR_ARG, "slots is NULL or misaligned");
    if (!k_out && !v_out) return report(MOE_ERR_ARG, "k_out and v_out are both NULL");
    if (!aligned(k_out, 16) || !aligned(v_out, 16)) return report(MOE_ERR_ARG, "k_out or v_out is not 16-byte aligned");
    const bool bf16 = cache->dtype == MOE_DTYPE_BF16;
    const int64_t dist[] = {k_out ? p->k_tok : 0, k_out ? p->k_head : 0, v_out ? p->v_tok : 0, v_out ? p->v_head : 0};
    for (int64_t x : dist)
        if (x < 0 || x * (bf16 ? 2 : 4) % 16 != 0)
            return report(MOE_ERR_ARG, "distances between tokens and heads must be multiples of 16 bytes, not negative");
    ReadArgs a{};
    a.ck = static_cast<const uint8_t*>(cache->k); a.cv = static_cast<const uint8_t*>(cache->v);
    a.ks = cache->k_scale; a.vs = cache->v_scale;
    a.slots = reinterpret_cast<const long long*>(slots);
    a.k = k_out; a.v = v_out;
    a.flags = &static_cast<WsHeader*>(workspace)->flags;
    a.n_slots = (long long)cache->n_pages * cache->page_size;
    a.k_tok = p->k_tok; a.k_head = p->k_head; a.v_tok = p->v_tok; a.v_head = p->v_head;
    a.T = p->T; a.kv_heads = cache->kv_heads; a.D = cache->head_dim;
    a.page_size = cache->page_size; a.nb = cache->page_size / cache->block;
    a.by_block = quotient(cache->block);
    a.by_page = quotient(cache->page_size);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = bf16 ? launch_read<__nv_bfloat16>(a, s) : launch_read<float>(a, s);
    return e == cudaSuccess ? MOE_OK : report(MOE_ERR_CUDA, "read launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
