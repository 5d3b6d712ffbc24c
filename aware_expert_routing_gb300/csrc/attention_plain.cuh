// attention_plain.cuh -- attention on CUDA cores (attention.cu): fp32, the bf16
// heads and pages that no tensor-core tile is made for, and the same over a cache
// in 8 bits (attention_q8.cu), whose codes are exact in bf16: they become bf16 on
// their way into shared memory, and the scales go into the scores and, with the
// weights, into the products with V.
//
// A cache in 8 bits, 64 single tokens up to 8000 positions with 32 + 4 heads: bf16, heads
// of 80 253 us (the bytes 24), of 192 537 (59), of 256 673 (78), of 128 with pages of 24
// positions 284 (39); fp32, heads of 128 282 (56), and 16 trees of 16 up to 4000 334, of which
// the products take 119 at the FMA rate.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "attention_line.cuh"

namespace moe {

namespace {

constexpr int kPlainCost = 2;   // a unit's own cost, in key tiles

// kC = ceil(D / 64), kR: query rows per thread, kS: shares of a tile's keys.
// 256 threads as kS shares x (16 / kS) x 16: for the scores, thread (z, ty, tx)
// has rows ty kR .. and keys tx, tx + 16, ... of share z; for the products with
// V, the same rows, its share's keys and components 4 tx .. of every 64.  So a
// row's maximum, sum and correction in a share stay with 16 threads (half a
// warp), and shares meet once, at the unit's end.
// Tiles of keys and values arrive by asynchronous copies one tile ahead, in
// the cache's own type; rows are padded by 16 bytes, which puts eight rows'
// 16-byte words in different banks.
struct E4m3 {   // an element of a cache in 8 bits
    uint8_t code;
};
template <typename KT> struct TileOf { using type = KT; };
template <> struct TileOf<E4m3> { using type = __nv_bfloat16; };

template <typename KT, int kC, int kR, int kS>
struct Plain {
    using T = typename TileOf<KT>::type;
    static constexpr bool kQ8 = std::is_same<KT, E4m3>::value;
    static constexpr int kRows = 16 / kS * kR;
    static constexpr int kKeys = kC == 1 || kS == 4 ? 64 : 32;
    static constexpr int kPad = 16 / (int)sizeof(T);
    static_assert(kS == 1 || (kKeys % (16 * kS) == 0 && kS * kRows <= kKeys * (int)sizeof(T) && kS * kRows <= 8 * kKeys),
                  "the shares' sums fit where the tiles were, their maxima in the rows' padding");
    static size_t smem(int D) {
        return 4 * (size_t)kKeys * (D + kPad) * sizeof(T) + (size_t)kRows * (D + 4) * 4 + (size_t)kRows * (kKeys + 4) * 4 +
               2 * kKeys * sizeof(long long) + sizeof(LineStart) + (kQ8 ? 4 * kKeys * sizeof(float) : 0);
    }
};

// Sixteen codes as bf16.
__device__ __forceinline__ void widen(const uint4& c, uint4& lo, uint4& hi) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[i >> 1] >> (i & 1) * 16)));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
        r[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    lo = make_uint4(r[0], r[1], r[2], r[3]);
    hi = make_uint4(r[4], r[5], r[6], r[7]);
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}

// Sixteen bytes of a row.
template <typename T>
struct Word {
    uint32_t u[4];
    __device__ __forceinline__ void load(const T* p) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        u[0] = x.x, u[1] = x.y, u[2] = x.z, u[3] = x.w;
    }
    __device__ __forceinline__ float at(int i) const {
        if (sizeof(T) == 4) return __uint_as_float(u[i & 3]);
        return __uint_as_float(i & 1 ? u[i >> 1] & 0xffff0000u : u[i >> 1] << 16);
    }
};

// T: of the queries and results; KT: of the cache.
template <typename T, typename KT, int kC, int kR, int kS>
__global__ void __launch_bounds__(256, kR * kC >= 16 ? 1 : 2) attention_plain_kernel(const AttentionArgs a) {
    using P = Plain<KT, kC, kR, kS>;
    using TT = typename P::T;
    constexpr bool kQ8 = P::kQ8;
    using Walk = LineWalk<P::kRows, P::kKeys, kPlainCost>;
    constexpr int kRows = P::kRows, kKeys = P::kKeys, kShare = kKeys / kS, kJ = kShare / 16;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const int D = a.D, ld = D + P::kPad, group = a.group;
    TT* ks = reinterpret_cast<TT*>(smem_raw);                    // [2][kKeys][ld]
    TT* vs = ks + 2 * kKeys * ld;
    float* qs = reinterpret_cast<float*>(vs + 2 * kKeys * ld);   // [kRows][D + 4]
    float* ps = qs + kRows * (D + 4);                            // [kRows][kKeys + 4]
    long long* row_at = reinterpret_cast<long long*>(ps + kRows * (kKeys + 4));   // [2][kKeys]: place in the cache, -1: none
    LineStart& S = *reinterpret_cast<LineStart*>(row_at + 2 * kKeys);
    float* ksc = reinterpret_cast<float*>(&S + 1);               // 8 bits: scales of the keys, of the values [2][kKeys]
    float* vsc = ksc + 2 * kKeys;
    const int tid = threadIdx.x, tx = tid & 15, ty = (tid >> 4) % (16 / kS), key0 = (tid >> 4) / (16 / kS) * kShare;
    const float c = a.scale * 1.4426950408889634f;   // scores to powers of two

    prefetch_tables(a);
    grid_launch_dependents();
    grid_dependency_wait();
    find_start<kRows, kKeys, kPlainCost, 256>(a, S);
    __syncthreads();
    Walk W;
    for (bool more = W.start(a, S); more; more = W.next(a)) {
        const int n = W.q.n, ctx = W.q.ctx, len = ctx + n, nrows = W.rows(a), r0 = W.rt * kRows;
        const int32_t* table = a.page_table + (size_t)W.r * a.max_pages;
        auto look = [&](int j) {   // the page of this thread's row of tile j; -2: no row
            const int pos = (W.kt + j) * kKeys + tid;
            return tid < kKeys && pos < len ? table[pos / a.page_size] : -2;
        };
        auto locate = [&](int j, int id) {   // the places of tile j's rows
            if (tid < kKeys) {
                const int pos = (W.kt + j) * kKeys + tid;
                long long at = -1;
                if (id != -2) {
                    if (id < 0 || id >= a.n_pages) raise_flag(a.flags, kFlagBadIndex);
                    else at = (((long long)id * a.kv_heads + W.h) * a.page_size + pos % a.page_size) * D;
                }
                row_at[(j & 1) * kKeys + tid] = at;
                if (kQ8) {
                    const size_t sc = at < 0 ? 0 : (size_t)(((long long)id * a.kv_heads + W.h) * (a.page_size / a.block) + pos % a.page_size / a.block);
                    ksc[(j & 1) * kKeys + tid] = at < 0 ? 0.f : a.k_scale[sc];
                    vsc[(j & 1) * kKeys + tid] = at < 0 ? 0.f : a.v_scale[sc];
                }
            }
        };
        auto fetch = [&](int j) {    // tile j's rows, zeros where there is none
            const int per = D * (int)sizeof(TT) / 16;
            for (int x = tid; x < kKeys * per && !kQ8; x += 256) {
                const int row = x / per, ch = x - row * per;
                const long long at = row_at[(j & 1) * kKeys + row];
                const size_t src = at < 0 ? 0 : (size_t)at + ch * P::kPad;
                const int dst = ((j & 1) * kKeys + row) * ld + ch * P::kPad, bytes = at < 0 ? 0 : 16;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                             ::"r"(smem_u32(ks + dst)), "l"(static_cast<const TT*>(a.ck) + src), "r"(bytes) : "memory");
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                             ::"r"(smem_u32(vs + dst)), "l"(static_cast<const TT*>(a.cv) + src), "r"(bytes) : "memory");
            }
            if (!kQ8) asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // 8 bits: the codes wait in registers while the tile before is worked on.
        constexpr int kCodes = kQ8 ? (kKeys * kC + 63) / 64 : 1;   // 16 codes each, of the keys and of the values
        uint4 kc[kCodes], vc[kCodes];
        auto fetch_codes = [&](int j) {
            const int per = D / 16;
#pragma unroll
            for (int i = 0; i < kCodes; ++i) {
                const int x = tid + 256 * i, row = x / per;
                const long long at = x < kKeys * per ? row_at[(j & 1) * kKeys + row] : -1;
                kc[i] = vc[i] = make_uint4(0, 0, 0, 0);
                if (at < 0) continue;
                kc[i] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.ck) + at + (x - row * per) * 16);
                vc[i] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.cv) + at + (x - row * per) * 16);
            }
        };
        auto store_codes = [&](int j) {
            const int per = D / 16;
#pragma unroll
            for (int i = 0; i < kCodes; ++i) {
                const int x = tid + 256 * i, row = x / per, dst = ((j & 1) * kKeys + row) * ld + (x - row * per) * 16;
                if (x >= kKeys * per) continue;
                uint4 lo, hi;
                widen(kc[i], lo, hi);
                *reinterpret_cast<uint4*>(ks + dst) = lo;
                *reinterpret_cast<uint4*>(ks + dst + 8) = hi;
                widen(vc[i], lo, hi);
                *reinterpret_cast<uint4*>(vs + dst) = lo;
                *reinterpret_cast<uint4*>(vs + dst + 8) = hi;
            }
        };
        locate(0, look(0));
        if (W.nk > 1) locate(1, look(1));
        for (int x = tid; x < kRows * (D / 4); x += 256) {
            const int row = x / (D / 4), ch = x - row * (D / 4), gr = r0 + row;
            float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < nrows)
                q = load4(static_cast<const T*>(a.q) + (W.q.t0 + gr / group) * a.q_tok + (W.h * group + gr % group) * a.q_head + ch * 4);
            *reinterpret_cast<float4*>(qs + row * (D + 4) + ch * 4) = q;
        }
        __syncthreads();
        if (kQ8) {
            fetch_codes(0);
            store_codes(0);
        } else {
            fetch(0);
        }

        float m[kR], l[kR], o[kR][kC][4];
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int y = 0; y < kC; ++y)
#pragma unroll
                for (int z = 0; z < 4; ++z) o[i][y][z] = 0.f;
        }
        for (int j = 0; j < W.nk; ++j) {
            __syncthreads();
            int id = -2;   // the page of the tile after next is on its way during this tile
            if (kQ8) {
                if (j + 1 < W.nk) fetch_codes(j + 1);
                if (j + 2 < W.nk) id = look(j + 2);
            } else if (j + 1 < W.nk) {
                fetch(j + 1);
                if (j + 2 < W.nk) id = look(j + 2);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            if (!kQ8) __syncthreads();
            // ---- scores ----
            float s[kR][kJ];
#pragma unroll
            for (int i = 0; i < kR; ++i)
#pragma unroll
                for (int y = 0; y < kJ; ++y) s[i][y] = 0.f;
            const TT* kt = ks + ((size_t)(j & 1) * kKeys + key0) * ld;
#pragma unroll 2
            for (int d = 0; d < D; d += P::kPad) {
                Word<TT> k[kJ];
#pragma unroll
                for (int y = 0; y < kJ; ++y) k[y].load(kt + (tx + 16 * y) * ld + d);
#pragma unroll
                for (int i = 0; i < kR; ++i)
#pragma unroll
                    for (int z = 0; z < P::kPad; z += 4) {
                        const float4 q = *reinterpret_cast<const float4*>(qs + (ty * kR + i) * (D + 4) + d + z);
#pragma unroll
                        for (int y = 0; y < kJ; ++y)
                            s[i][y] = fmaf(q.x, k[y].at(z), fmaf(q.y, k[y].at(z + 1), fmaf(q.z, k[y].at(z + 2), fmaf(q.w, k[y].at(z + 3), s[i][y]))));
                    }
            }
            const int k0 = (W.kt + j) * kKeys;
            const bool masked = k0 + kKeys > ctx;
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                const int gr = r0 + ty * kR + i, ti = gr / group;
                if (kQ8)
#pragma unroll
                    for (int y = 0; y < kJ; ++y) s[i][y] *= ksc[(j & 1) * kKeys + key0 + tx + 16 * y];
                if (masked) {
#pragma unroll
                    for (int y = 0; y < kJ; ++y) {
                        const int d = k0 + key0 + tx + 16 * y - ctx;   // which drafted token; below 0: context
                        bool seen = d < 0;
                        if (d >= 0 && d < n && ty * kR + i < nrows)
                            seen = a.mask ? d < 32 * a.mask_words &&
                                                ((a.mask[(size_t)(W.q.t0 + ti) * a.mask_words + (d >> 5)] >> (d & 31)) & 1u)
                                          : d <= ti;
                        if (!seen) s[i][y] = -INFINITY;
                    }
                }
                float mt = -INFINITY;
#pragma unroll
                for (int y = 0; y < kJ; ++y) {
                    s[i][y] *= c;
                    mt = fmaxf(mt, s[i][y]);
                }
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
                const float mn = fmaxf(m[i], mt);
                const float f = m[i] == -INFINITY ? 0.f : ex2(m[i] - mn), sub = mn == -INFINITY ? 0.f : mn;
                float sum = 0.f;
#pragma unroll
                for (int y = 0; y < kJ; ++y) {
                    const float p = ex2(s[i][y] - sub);
                    sum += p;
                    // (an unseen value's scale may be anything)
                    ps[(ty * kR + i) * (kKeys + 4) + key0 + tx + 16 * y] =
                        kQ8 ? p == 0.f ? 0.f : p * fmaxf(vsc[(j & 1) * kKeys + key0 + tx + 16 * y], 0x1p-64f) : p;
                }
                l[i] = l[i] * f + sum;   // this thread's keys; the 16 threads' sums meet at the end
                m[i] = mn;
#pragma unroll
                for (int y = 0; y < kC; ++y)
#pragma unroll
                    for (int z = 0; z < 4; ++z) o[i][y][z] *= f;
            }
            __syncwarp();   // a row's P is written and read by the same warp
            // ---- O += P V; where a mask hides a value, it is not multiplied (it may be anything) ----
            const TT* vt = vs + ((size_t)(j & 1) * kKeys + key0) * ld;
            auto product = [&](auto hide) {
#pragma unroll 2
                for (int x = 0; x < kShare; x += 4) {
                    float4 p[kR];
#pragma unroll
                    for (int i = 0; i < kR; ++i) p[i] = *reinterpret_cast<const float4*>(ps + (ty * kR + i) * (kKeys + 4) + key0 + x);
#pragma unroll
                    for (int z = 0; z < 4; ++z)
#pragma unroll
                        for (int y = 0; y < kC; ++y) {
                            if (tx * 4 + 64 * y >= D) continue;
                            const float4 v = load4(vt + (x + z) * ld + tx * 4 + 64 * y);
#pragma unroll
                            for (int i = 0; i < kR; ++i) {
                                const float w = z == 0 ? p[i].x : z == 1 ? p[i].y : z == 2 ? p[i].z : p[i].w;
                                if (decltype(hide)::value && w == 0.f) continue;
                                o[i][y][0] = fmaf(w, v.x, o[i][y][0]);
                                o[i][y][1] = fmaf(w, v.y, o[i][y][1]);
                                o[i][y][2] = fmaf(w, v.z, o[i][y][2]);
                                o[i][y][3] = fmaf(w, v.w, o[i][y][3]);
                            }
                        }
                }
            };
            if (masked) product(std::true_type{});
            else product(std::false_type{});
            if (kQ8) {
                if (j + 1 < W.nk) store_codes(j + 1);
                __syncthreads();   // this tile's scales have been read
            }
            if (j + 2 < W.nk) locate(j + 2, id);
        }
        // ---- the unit's result, or its part ----
        const bool whole = W.nk == W.q.nkt;
        const int slot = 2 * blockIdx.x + (W.first ? 0 : 1);
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
        auto put = [&](int row, int ch, float4 v, float rm, float rl) {   // components 4 ch .. of a row
            const int gr = r0 + row;
            const size_t orow = (size_t)(W.q.t0 + gr / group) * a.heads + W.h * group + gr % group;
            if (whole) store_row(static_cast<T*>(a.out) + orow * D + ch * 4, v, rl);
            else reinterpret_cast<float4*>(a.o)[((size_t)slot * a.rows + (row & ~31)) * (D / 4) + ch * 32 + (row & 31)] = v;
            if (ch == 0) {
                if (!whole) a.ml[(size_t)slot * a.rows + row] = make_float2(rm, rl);
                else if (a.lse) a.lse[orow] = rl == 0.f ? -INFINITY : (rm + log2f(rl)) * 0.6931471805599453f;
            }
        };
        if (kS == 1) {
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                const int row = ty * kR + i;
                if (row >= nrows) continue;
#pragma unroll
                for (int y = 0; y < kC; ++y)
                    if (tx * 4 + 64 * y < D) put(row, tx + 16 * y, make_float4(o[i][y][0], o[i][y][1], o[i][y][2], o[i][y][3]), m[i], l[i]);
            }
        } else {
            // the shares' sums meet where the tiles were: [kS][kRows][D], and
            // behind them their maxima and sums of weights [kS][kRows]
            float* os = reinterpret_cast<float*>(ks);
            float2* mls = reinterpret_cast<float2*>(os + kS * kRows * D);
            const int z = key0 / kShare;
            __syncthreads();   // the last tile's keys and values have been read
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                const int row = z * kRows + ty * kR + i;
#pragma unroll
                for (int y = 0; y < kC; ++y)
                    if (tx * 4 + 64 * y < D)
                        *reinterpret_cast<float4*>(os + row * D + tx * 4 + 64 * y) = make_float4(o[i][y][0], o[i][y][1], o[i][y][2], o[i][y][3]);
                if (tx == 0) mls[row] = make_float2(m[i], l[i]);
            }
            __syncthreads();
            for (int x = tid; x < nrows * (D / 4); x += 256) {
                const int row = x / (D / 4), ch = x - row * (D / 4);
                float rm = -INFINITY, rl = 0.f;
#pragma unroll
                for (int y = 0; y < kS; ++y) rm = fmaxf(rm, mls[y * kRows + row].x);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int y = 0; y < kS; ++y) {
                    const float2 e = mls[y * kRows + row];
                    if (e.y == 0.f) continue;   // saw nothing; a NaN goes on
                    const float f = ex2(e.x - rm);
                    const float4 w = *reinterpret_cast<const float4*>(os + (y * kRows + row) * D + ch * 4);
                    rl = fmaf(f, e.y, rl);
                    v = make_float4(fmaf(f, w.x, v.x), fmaf(f, w.y, v.y), fmaf(f, w.z, v.z), fmaf(f, w.w, v.w));
                }
                put(row, ch, v, rm, rl);
            }
        }
        __syncthreads();   // the next unit overwrites the queries and the tiles
    }
}

template <typename T, typename KT, int kC, int kR, int kS>
cudaError_t launch_plain_t(const AttentionArgs& a, int sms, cudaStream_t s) {
    using P = Plain<KT, kC, kR, kS>;
    const size_t smem = P::smem(a.D);
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        e = cudaFuncSetAttribute(attention_plain_kernel<T, KT, kC, kR, kS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)P::smem(64 * kC));
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    // two blocks per SM where their shared memory allows it
    const int want = sms * (smem <= 113 * 1024 ? 2 : 1), grid = want < kPlainRanges ? want : kPlainRanges;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, attention_plain_kernel<T, KT, kC, kR, kS>, a)) != cudaSuccess) return e;
    if ((long long)a.max_pages * a.page_size <= P::kKeys || grid < 2) return cudaSuccess;   // no unit is cut
    return launch_join<T, 2 * kC, kPlainCost>(a, grid, P::kRows, cfg);
}

template <typename T, typename KT, int kC>
cudaError_t launch_plain_r(const AttentionArgs& a, int rows, int sms, cudaStream_t s) {
    // What bounds units of few rows is the tiles' way from shared memory to the
    // registers: with shares a key serves the unit's rows in fewer warps.  Four
    // shares need tiles of 64 keys, of which two blocks an SM fit up to 4 bytes x
    // 64 components; beyond, two shares, except for up to 4 rows.  64 tokens at up
    // to 4000 positions, one / two / four shares: fp32, 8 rows of 64 components
    // 94.6 / - / 50.6 us, of 128 165 / 107 / 147 (one block an SM), one row of 128
    // 315 / 201 / 167; bf16, 8 rows of 128, pages of 1 373 / 242 / 150.  32 rows in
    // shares (8 a thread) were no faster: 16 trees of 40 79 against 81 us.
    constexpr int kBytes = kC * (int)sizeof(typename TileOf<KT>::type), kS = kBytes <= 4 ? 4 : 2;
    if (rows > 32) return launch_plain_t<T, KT, kC, 4, 1>(a, sms, s);
    if (rows > 16) return launch_plain_t<T, KT, kC, 2, 1>(a, sms, s);
    if (rows > 8) return launch_plain_t<T, KT, kC, kS, kS>(a, sms, s);
    if (rows > 4 || kBytes > 8) return launch_plain_t<T, KT, kC, kS / 2, kS>(a, sms, s);
    return launch_plain_t<T, KT, kC, 1, (kBytes > 8 ? kS : 4)>(a, sms, s);
}

template <typename T, typename KT = T>
cudaError_t launch_plain(const AttentionArgs& a, int sms, cudaStream_t s) {
    if (sms <= 0) return cudaErrorNotSupported;
    // Units of 4 to 64 rows, by the requests' rows a key head on average.
    AttentionArgs b = a;
    const long long mean = ((long long)a.T * a.group + a.R - 1) / a.R;
    b.min_steps = 1;
    const int rows = mean > 64 ? 64 : (int)mean;
    switch ((a.D + 63) / 64) {
        case 1: return launch_plain_r<T, KT, 1>(b, rows, sms, s);
        case 2: return launch_plain_r<T, KT, 2>(b, rows, sms, s);
        case 3: return launch_plain_r<T, KT, 3>(b, rows, sms, s);
        default: return launch_plain_r<T, KT, 4>(b, rows, sms, s);
    }
}

}  // namespace

}  // namespace moe
