// attention_q8.cu -- moe_tree_attention_q8: attention to a cache in 8 bits, on
// the 5th-generation tensor cores for bf16 queries, heads of 64 or 128 and pages
// of 8, 16, 32 or 64 positions or a multiple of 128 (attention_q8_fits); on CUDA
// cores (attention_plain.cuh) else.
//
// The codes go from HBM through shared memory into the tensor cores as they are
// (kind::f8f6f4): half of the bytes, and no pass that widens them.  The other
// operands are made of e4m3 numbers too,
//   q = qs (q0 + q1 / 2^4): qs a power of two for a unit's rows, so that the
//       largest component lies in 224..448; a bf16 component has 8 significant
//       bits, an e4m3 number 4, so two of them hold it exactly (but for what is
//       2^-21 of the unit's largest: half a step of 2^-13, beside 224 at least);
//   w = w0 + w1 / 2^5 + w2 / 2^10: the weights of a tile, scaled so that each row's
//       largest is 2^8: good to 2^-14 of a weight (and 2^-11 before that: they come
//       from f16), or to 2^-28 of the row's largest in the tile.  (Scaled by one bound for the whole
//       context, light weights behind a heavy one, which a long context has many
//       of, kept few bits or none; so each tile's product is added up in registers.
//       Values widened to f16, with f16 weights, cost more shared memory traffic
//       than there is: 455 against 372 us for 256 tokens to 16000.)
// The products are transposed: keys are the rows,
//   S^T = K [q0 | q1]^T       (128 keys x 2 R columns),
//   O^T = V^T [w0 | w1 | w2]  (head_dim x 3 R columns),
// so that the parts stand side by side as columns, each with its own sum, a
// thread has one key, whose scales are two registers, and units of few query rows
// cost few exponentials.  V^T and the weights are read along their other dimension
// (MN-major), as they lie.
//
// With the scales sk, sv of a key and c = scale / ln 2, for every row of a tile:
//   t = c qs sk (q.k) + log2 sv,  m = max t,  w = 2^(t - m + 8),  f = 2^(m - M - 8),
//   l += f sum w / sv,  O += f sum w v;   at the end out = O / l, lse = ln l + M ln 2.
// So a weight carries its value's scale, and what is rounded is small against the
// tile's largest |weight * scale|.  M, a row's reference, is its first tile's m; it
// is moved, and l and O with it, when some m is 2^60 above.
//
// Work, copies, MMA order and partial results are as in attention_tc.cu
// (attention_line.cuh): a line of (request, key head, tile of R rows) cut into
// equal stretches.  Three warps copy keys, values and scales, one issues the MMAs,
// and two warpgroups have the softmax.  These take a unit's tiles in turn, each
// with M, l and O of its own, which meet at the unit's end: a tile's steps wait for
// one another, and two tiles under way cover that.
//
// Requests of more rows go to attention_tc.cu, which widens tiles to bf16: there
// the weights' parts would cost more than the bytes.
//
// Bound by the bytes while a unit has up to 16 rows, by the softmax and the weights'
// parts above.  Measured, heads of 128, 4 key heads: 256 single tokens up to 16000
// positions (2.27 GB) 372 us, 6.1 TB/s (650 in bf16); 64 up to 8000 with a scale for
// every position (275 MB) 56, 4.9 TB/s (89); one token at 1000 10.3, latency as there.
#include <cudaTypedefs.h>

#include <cstddef>

#include "attention_plain.cuh"
#include "tcgen05_tiles.cuh"

namespace moe {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();   // api.cu

namespace {

constexpr int kKeys = 128;          // keys of a tile
constexpr uint32_t kOCol = 256;     // tensor memory: S buffers from 0, O from here
// See attention_line.cuh.  2 / 3 / 4 / 6: 64 tokens to 8000 60.0 / 57.4 / 55.5 / 57.1 us,
// 256 to 16000 369 / 370 / 371 / 374, 64 x 4 to 8000 103 / 102 / 96 / 95 (and, widened in
// attention_tc.cu, 16 trees of 16 36.3 / 37.0 / 37.4 / 38.4).
constexpr int kUnitCost = 4;
constexpr uint32_t kDrainPolls = 1u << 20;   // of the last waits, for work that runs already
constexpr float kNone = -1e30f;     // M of a row that has seen nothing
constexpr float kTop = 8.f;         // log2 of a row's largest weight in a tile (e4m3 ends at 448)
constexpr float kFar = 60.f;        // how far above M a tile's maximum may be
// What e4m3 leaves of a number up to 2^8 is at most 2^3.
constexpr float kPart = 32.f;
constexpr int kScaleStages = 8;

// R: query rows of a unit.
template <int D, int R>
struct Cfg8 {
    static constexpr int kParts = 3;                      // numbers of a weight
    static constexpr int kNS = 2 * R, kNP = kParts * R;   // columns of S and of O
    static constexpr int kThreads = 384;                  // warps: copies of keys, MMAs, scales, copies of values; softmax
    static constexpr int kStage = kKeys * D;              // a tile of keys or of values
    static constexpr int kQTile = kNS * D;
    static constexpr int kPRow = kNP <= 64 ? 64 : 128;    // weights: bytes of a key, a row of the swizzle
    static constexpr int kPTile = kKeys * kPRow;
    static constexpr int kControl = 6144;
    static constexpr int kScales = 2 * kKeys * 4;         // a tile's scales, of keys and of values
    static constexpr int kSmem = 227 * 1024;
    static constexpr int kPairs = (kSmem - 1024 - kControl - kQTile - 2 * kPTile - kScaleStages * kScales) / (2 * kStage);
    static constexpr int kStages = kPairs < 8 ? kPairs : 8;   // of keys, and of values
    static constexpr int kItems = R * D / 16;             // 16 components of a query row
    static constexpr int kQ = (kItems + 255) / 256;
    static_assert(2 * kNS <= 256 && 2 * kNP <= 256 && kNP <= kPRow && kStages >= 3, "tensor memory; rows of weights; a ring");
    static_assert(R * 512 <= 2 * kPTile, "where the warpgroups' sums meet");
};

struct Control8 {
    uint64_t k_full[8], k_empty[8], v_full[8], v_empty[8], sc_full[8], sc_empty[8], q_full, s_full[2], p_full[2], pv_done[2], drained;
    long long wait_cycles;
    LineStart start;
    int abort_flag;
    uint32_t armed[2];         // stages filled, or being filled, so far
    uint32_t tmem_base;
    uint32_t most[8];          // warps' largest query components
    // of each row (by tiles: of the first warpgroup, then of the second)
    alignas(16) float top[4][64];               // a tile's maxima in the four warps
    alignas(16) float shift[64], f[2][64];      // kTop - m; f of the last two tiles
    alignas(16) float grow[64], sum[4][64], factor[64];
    float reference[64];                        // M
    int row_token[2][64], row_out[2][64];     // of two units: the token in its request, the row of `out`
};
static_assert(sizeof(Control8) <= 6144, "control block");

__device__ __forceinline__ bool aborted(Control8& S) { return *(volatile int*)&S.abort_flag != 0; }
__device__ __forceinline__ bool warp_aborted(Control8& S) { return __any_sync(0xffffffffu, aborted(S)); }

// Bounded mbarrier wait; once the CTA has given up every later wait returns
// at once, so the control flow (and every barrier) still completes.
__device__ __forceinline__ void wait_bar(uint64_t* bar, uint32_t parity, Control8& S, uint32_t* flags) {
    if (mbar_try_wait(bar, parity)) return;
    const long long t0 = clock64();
    while (!aborted(S)) {
        if (mbar_try_wait(bar, parity)) return;
        if (clock64() - t0 > S.wait_cycles) {
            *(volatile int*)&S.abort_flag = 1;
            raise_flag(flags, kFlagTimeout);
            return;
        }
    }
}

// Whether any of the barrier's 128 threads says so.
__device__ __forceinline__ bool vote128(uint32_t id, bool x) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.or.pred q, %1, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(r) : "r"(id), "r"((uint32_t)x) : "memory");
    return r != 0;
}

__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// Four codes of w[0..3], in the order of memory, from two pairs in f16, which
// become what the codes leave of them, times kPart (exact in f16).
__device__ __forceinline__ uint32_t codes4(uint32_t& w01, uint32_t& w23, bool rest) {
    uint32_t c;
    asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n cvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n mov.b32 %0, {a, b};\n}"
        : "=r"(c) : "r"(w01), "r"(w23));
    if (rest) {
        uint32_t h01, h23;
        asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
            : "=r"(h01), "=r"(h23) : "r"(c));
        const __half2 k = __float2half2_rn(kPart);
        const __half2 d0 = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&w01), *reinterpret_cast<const __half2*>(&h01)), k);
        const __half2 d1 = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&w23), *reinterpret_cast<const __half2*>(&h23)), k);
        w01 = *reinterpret_cast<const uint32_t*>(&d0);
        w23 = *reinterpret_cast<const uint32_t*>(&d1);
    }
    return c;
}

// Adds up each of kC numbers over the 32 lanes; lane x then has the sum of
// number x / (32 / kC).
template <int kC>
__device__ __forceinline__ float sum_columns(float (&v)[kC]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = kC / 2, off = 16; n > 0; n >>= 1, off >>= 1) {
        const bool up = lane & off;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
        }
    }
    if (kC == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
    return v[0];
}

template <int D, int R>
__global__ void __launch_bounds__(Cfg8<D, R>::kThreads, 1)
attention_q8_kernel(const AttentionArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
    using C = Cfg8<D, R>;
    using Walk = LineWalk<R, kKeys, kUnitCost>;
    constexpr int kC = R;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* ks = smem;                                   // [kStages][kStage]
    unsigned char* vs = ks + C::kStages * C::kStage;            // [kStages][kStage]
    unsigned char* ps = vs + C::kStages * C::kStage;            // [2][kPTile]
    unsigned char* qs = ps + 2 * C::kPTile;                     // [kQTile]
    float* scale_ring = reinterpret_cast<float*>(qs + C::kQTile);   // [kScaleStages][2][kKeys]
    Control8& S = *reinterpret_cast<Control8*>(scale_ring + kScaleStages * 2 * kKeys);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = a.group;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&S.k_full[i], 1);
            mbar_init(&S.k_empty[i], 1);
            mbar_init(&S.v_full[i], 1);
            mbar_init(&S.v_empty[i], 1);
        }
        for (int i = 0; i < kScaleStages; ++i) {
            mbar_init(&S.sc_full[i], 32);
            mbar_init(&S.sc_empty[i], 4);
        }
        mbar_init(&S.q_full, 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.s_full[i], 1);
            mbar_init(&S.p_full[i], 4);
            mbar_init(&S.pv_done[i], 1);
        }
        mbar_init(&S.drained, 1);
        fence_barrier_init();
        S.abort_flag = 0;
        S.armed[0] = S.armed[1] = 0;
        S.wait_cycles = a.wait_cycles;
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
    }
    if (warp == 1) tmem_alloc(&S.tmem_base, 512);
    prefetch_tables(a);
    grid_launch_dependents();   // a kernel that follows may start its prologue; it waits for this grid's end
    grid_dependency_wait();     // lengths, queries and the cache come from preceding kernels

    find_start<R, kKeys, kUnitCost, C::kThreads>(a, S.start);
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tmem = S.tmem_base;
    Walk W;
    const bool any = W.start(a, S.start);

    if (!any) {
        // no work for this CTA
    } else if (warp < 4 && warp != 1) {
        // ---- producers: a warp each for the rings of keys, of values and of scales ----
        // (A warp issues a copy in about 80 cycles; eight pages' keys and values
        // from one took longer than their bytes.)
        uint32_t seq = 0;
        const int page = a.page_size;
        const int per = page < kKeys ? kKeys / page : 1;        // pages of a tile
        const int prow = page < kKeys ? page : kKeys;           // rows of a copy
        const uint32_t bytes = (uint32_t)prow * D;
        const int batch = 32 / per;                             // tiles whose table entries the warp reads at once
        const int my_tile = lane / per, my_page = lane - my_tile * per;
        const int wide = page / kKeys;                          // tiles of a page of more than 128 rows
        // This lane's page of the batch of tiles from j on of a part: is there
        // one, its entry in the table, and its first row in the cache (-1: none).
        auto has = [&](const Walk& U, int j) {
            return my_tile < batch && j + my_tile < U.nk && (U.kt + j + my_tile) * kKeys + my_page * prow < U.q.ctx + U.q.n;
        };
        auto read = [&](const Walk& U, int j) -> int {
            const int t = U.kt + j + my_tile;
            return has(U, j) ? a.page_table[(size_t)U.r * a.max_pages + (page <= kKeys ? t * per + my_page : t / wide)] : 0;
        };
        auto row_of = [&](int id, int j) -> int {
            if (!has(W, j)) return -1;
            if (id < 0 || id >= a.n_pages) {
                raise_flag(a.flags, kFlagBadIndex);
                id = 0;
            }
            const int row = page <= kKeys ? 0 : (W.kt + j + my_tile) % wide * kKeys;
            return (int)(((long long)id * a.kv_heads + W.h) * page + row);
        };
        const bool is_v = warp == 3;
        const CUtensorMap* map = is_v ? &map_v : &map_k;
        unsigned char* ring = is_v ? vs : ks;
        uint64_t *full = is_v ? S.v_full : S.k_full, *empty = is_v ? S.v_empty : S.k_empty;
        auto load = [&](int g) {
            const uint32_t st = seq % C::kStages, ph = (seq / C::kStages) & 1;
            wait_bar(&empty[st], ph ^ 1, S, a.flags);
            ++seq;
            const int n = __popc(__ballot_sync(0xffffffffu, g >= 0));
            if (warp_aborted(S)) return;
            if (lane == 0) {
                mbar_arrive_expect_tx(&full[st], n * bytes);
                S.armed[is_v] = seq;
            }
            __syncwarp();
            if (g >= 0) tma_rows(smem_u32(ring + st * C::kStage) + lane * bytes, map, g, &full[st]);
        };
        // (Read by the softmax's threads, a tile ahead, the scales were what these
        // waited for.)
        ScaleCopy<kScaleStages> scales(a, prow, lane);
        auto load_scales = [&](int cur, int at) {
            wait_bar(&S.sc_empty[scales.stage()], scales.phase() ^ 1, S, a.flags);
            scales.copy(a, cur, at, per, scale_ring, &S.sc_full[scales.stage()]);
        };
        int id0 = read(W, 0), id1 = read(W, batch);
        bool more = true;
        while (more) {
            int at = 0, cur = row_of(id0, 0), nxt = id1;
            Walk N = W;
            for (int j = 0; j < W.nk; ++j) {
                const int t = __shfl_sync(0xffffffffu, cur, min(31, at * per + lane));
                const int g = lane < per ? t : -1;
                if (warp == 2) load_scales(cur, at);
                else load(g);
                if (j == 0) {   // the next part's first entries, while this part is loaded
                    more = N.next(a);
                    if (more) {
                        id0 = read(N, 0);
                        id1 = read(N, batch);
                    }
                }
                if (++at == batch) {
                    at = 0;
                    cur = row_of(nxt, j + 1);
                    nxt = read(W, j + 1 + batch);
                }
            }
            W = N;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 1) {
        // ---- MMA: one warp issues, in the order of the ring ----
        // S: both K-major; O: both MN-major.  Heads of 64: a tile of V^T has 64 rows,
        // the MMA 128: its second 64 are the first again (leading offset 0), and are
        // not looked at.
        constexpr uint32_t idesc_s = umma_idesc_e4m3(128, C::kNS);
        constexpr uint32_t idesc_o = umma_idesc_e4m3(128, C::kNP) | (1u << 15) | (1u << 16);
        constexpr uint64_t swizzle = D == 128 ? 2 : 4;   // 128 or 64 bytes: a row of a tile
        constexpr uint64_t row_desc = (uint64_t)1 << 46 | swizzle << 61 | (uint64_t)(8 * D >> 4) << 32 | 1u << 16;
        constexpr uint64_t v_desc = (uint64_t)1 << 46 | swizzle << 61 | (uint64_t)(8 * D >> 4) << 32 | (D == 128 ? 1u << 16 : 0u);
        constexpr uint64_t p_desc = (uint64_t)1 << 46 | (uint64_t)(C::kPRow == 128 ? 2 : 4) << 61 | (uint64_t)(8 * C::kPRow >> 4) << 32 | 1u << 16;
        const uint32_t ctl = uniform(smem_u32(&S)), k_ring = uniform(smem_u32(ks)), v_ring = uniform(smem_u32(vs)), q0 = uniform(smem_u32(qs)),
                       p0 = uniform(smem_u32(ps)), tm = uniform(tmem);
        uint32_t st = 0, ph = 0, vst = 0, vph = 0;   // next stages of the rings, their phases
        uint32_t tile = 0, seg = 0;                  // key tiles, units
        auto advance = [&](uint32_t& s_, uint32_t& p_) {
            if (++s_ == C::kStages) {
                s_ = 0;
                p_ ^= 1;
            }
        };
        auto issue_s = [&](uint32_t buf) {
            wait_bar(&S.k_full[st], ph, S, a.flags);
            tmem_fence_after_sync();
            const uint32_t kaddr = k_ring + st * C::kStage;
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
                mma8_ss(tm + buf * C::kNS, row_desc | ((kaddr + k * 32) >> 4), row_desc | ((q0 + k * 32) >> 4), idesc_s, k > 0);
            mma_commit(ctl + (uint32_t)offsetof(Control8, s_full) + 8 * buf);
            mma_commit(ctl + (uint32_t)offsetof(Control8, k_empty) + 8 * st);
            advance(st, ph);
        };
        auto issue_pv = [&](uint32_t buf) {
            const uint32_t vaddr = v_ring + vst * C::kStage, paddr = p0 + buf * C::kPTile;
#pragma unroll
            for (int k = 0; k < kKeys / 32; ++k)
                mma8_ss(tm + kOCol + buf * C::kNP, v_desc | ((vaddr + k * 32 * D) >> 4), p_desc | ((paddr + k * 32 * C::kPRow) >> 4), idesc_o, k > 0);
            mma_commit(ctl + (uint32_t)offsetof(Control8, pv_done) + 8 * buf);
            mma_commit(ctl + (uint32_t)offsetof(Control8, v_empty) + 8 * vst);
            advance(vst, vph);
        };
        // Once a wait has given up, all return at once: the loop then runs out on
        // whatever the shared and tensor memory hold, which harms nothing.
        do {
            const int n = uniform(W.nk);
            wait_bar(&S.q_full, seg++ & 1, S, a.flags);
            issue_s(tile & 1);
            for (int j = 0; j < n; ++j) {
                if (j + 1 < n) issue_s((tile + 1) & 1);
                wait_bar(&S.v_full[vst], vph, S, a.flags);
                wait_bar(&S.p_full[tile & 1], (tile >> 1) & 1, S, a.flags);
                tmem_fence_after_sync();
                issue_pv(tile & 1);
                ++tile;
            }
        } while (W.next(a));
    } else {
        // ---- softmax: thread = key = TMEM lane, and component of O ----
        // Tiles alternate between two buffers of S, weights and O.  S of a tile is
        // computed after the product of the last but one, so what finds it complete
        // knows that its buffers of weights and of O have been read.
        const int w = (warp - 4) >> 2, quad = warp & 3, key = quad * 32 + lane;
        const int tid = threadIdx.x - 128;            // among the softmax's threads
        const int wtid = tid & 127;
        const int s0 = w * R;                         // this warpgroup's place among the rows' maxima and sums
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const float c = a.scale * 1.4426950408889634f;   // scores to powers of two
        uint32_t tile = 0, unit = 0;

        // A unit's queries: on their way, then split into two e4m3 numbers.
        uint4 qr[C::kQ][2];
        auto load_q = [&](const Walk& U, int rows) {
#pragma unroll
            for (int i = 0; i < C::kQ; ++i) {
                const int x = tid + i * 256, row = x / (D / 16), ch = x % (D / 16);
                qr[i][0] = qr[i][1] = make_uint4(0, 0, 0, 0);
                if (x >= C::kItems || row >= rows) continue;
                const int gr = U.rt * R + row, tok = gr / group;
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + (U.q.t0 + tok) * a.q_tok +
                                                                  (U.h * group + gr - tok * group) * a.q_head + ch * 16);
                qr[i][0] = src[0];
                qr[i][1] = src[1];
            }
        };
        auto finish_q = [&](const Walk& U, int rows) -> float {   // the unit's qs
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < C::kQ; ++i)
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const uint32_t v = z == 0 ? qr[i][y].x : z == 1 ? qr[i][y].y : z == 2 ? qr[i][y].z : qr[i][y].w;
                        const uint32_t lo = v << 16 & 0x7fffffffu, hi = v & 0x7fff0000u;
                        most = max(most, max(lo < 0x7f800000u ? lo : 0u, hi < 0x7f800000u ? hi : 0u));
                    }
            most = __reduce_max_sync(0xffffffffu, most);
            if (lane == 0) S.most[tid >> 5] = most;
            if (tid < R) {   // the unit's rows; past its own, those of the last
                const int gr = U.rt * R + min(tid, rows - 1), tok = gr / group;
                S.row_token[unit & 1][tid] = tok;
                S.row_out[unit & 1][tid] = (U.q.t0 + tok) * a.heads + U.h * group + gr - tok * group;
            }
            named_barrier(3, 256);
#pragma unroll
            for (int i = 0; i < 8; ++i) most = max(most, S.most[i]);
            // the power of two with most <= 448 of it
            const int e = max((int)(most >> 23) - 127 - 8 + ((most & 0x7fffffu) > 0x600000u), -64);
            const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
            for (int i = 0; i < C::kQ; ++i) {
                const int x = tid + i * 256, row = x / (D / 16), ch = x % (D / 16);
                if (x >= C::kItems) continue;
                uint32_t c0[4], c1[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const uint32_t u0 = y == 0 ? qr[i][0].x : y == 1 ? qr[i][0].z : y == 2 ? qr[i][1].x : qr[i][1].z;
                    const uint32_t u1 = y == 0 ? qr[i][0].y : y == 1 ? qr[i][0].w : y == 2 ? qr[i][1].y : qr[i][1].w;
                    float v[4] = {__uint_as_float(u0 << 16), __uint_as_float(u0 & 0xffff0000u), __uint_as_float(u1 << 16),
                                  __uint_as_float(u1 & 0xffff0000u)};
#pragma unroll
                    for (int z = 0; z < 4; ++z) v[z] = fabsf(v[z]) < INFINITY ? v[z] * inv : NAN;
                    split4(v, 16.f, c0[y], c1[y]);
                }
                // (R is a multiple of 16: both rows have the same place in the swizzle)
                unsigned char* to = qs + row * D + ((D == 128 ? ch ^ (row & 7) : ch ^ (row >> 1 & 3)) << 4);
                *reinterpret_cast<uint4*>(to) = make_uint4(c0[0], c0[1], c0[2], c0[3]);
                *reinterpret_cast<uint4*>(to + R * D) = make_uint4(c1[0], c1[1], c1[2], c1[3]);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.q_full);
            return __uint_as_float((uint32_t)(127 + e) << 23);
        };

        // a warpgroup's first tile of a part
        auto first_of = [&]() -> int { return (int)((tile ^ (uint32_t)w) & 1); };

        int rows = W.rows(a), j0 = first_of();
        load_q(W, rows);
        float qscale = finish_q(W, rows);
        bool more = true;
        while (more) {
            const Walk U = W;
            const int nr = rows, n = U.q.n, j1 = j0;
            const int* row_token = S.row_token[unit & 1];
            const int* row_out = S.row_out[unit & 1];
            const bool whole = U.nk == U.q.nkt;
            const float cq = c * qscale;
            const uint32_t tile0 = tile;
            float l[kC], o[kC];
#pragma unroll
            for (int i = 0; i < kC; ++i) l[i] = o[i] = 0.f;
            float M = kNone;                // of row wtid (threads of a row)
            // Adds the product of this warpgroup's tile t, which is known to be there.
            auto add_o = [&](uint32_t t) {
                const float* f = S.f[t >> 1 & 1] + s0;
#pragma unroll
                for (int i0 = 0; i0 < kC; i0 += 16) {
                    float x[16];
#pragma unroll
                    for (int p = C::kParts - 1; p >= 0; --p) {
                        uint32_t y[16];
                        tmem_ld16(lanes + kOCol + (t & 1) * C::kNP + p * R + i0, y);
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = p == C::kParts - 1 ? __uint_as_float(y[i]) : fmaf(x[i], 1.f / kPart, __uint_as_float(y[i]));
                    }
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 g = *reinterpret_cast<const float4*>(f + i0 + i);
                        o[i0 + i] = fmaf(x[i], g.x, o[i0 + i]);
                        o[i0 + i + 1] = fmaf(x[i + 1], g.y, o[i0 + i + 1]);
                        o[i0 + i + 2] = fmaf(x[i + 2], g.z, o[i0 + i + 2]);
                        o[i0 + i + 3] = fmaf(x[i + 3], g.w, o[i0 + i + 3]);
                    }
                }
            };
            bool pending = false;           // a product that is to be added
            for (int j = j1; j < U.nk; j += 2) {
                tile = tile0 + j;
                const uint32_t buf = tile & 1;
                const int k0 = (U.kt + j) * kKeys, d = k0 + key - U.q.ctx;   // d: which drafted token; below 0: context
                const bool masked = k0 + kKeys > U.q.ctx;
                uint32_t seen = ~0u;
                if (masked && d >= 0) {
                    seen = 0;
                    if (d < n) {
                        if (a.mask) {
                            if (d < 32 * a.mask_words) {
                                const uint32_t* words = a.mask + (size_t)U.q.t0 * a.mask_words + (d >> 5);
#pragma unroll
                                for (int i = 0; i < kC; ++i) seen |= ((words[(size_t)row_token[i] * a.mask_words] >> (d & 31)) & 1u) << i;
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < kC; ++i) seen |= (uint32_t)(d <= row_token[i]) << i;
                        }
                    }
                }
                const uint32_t sst = tile % kScaleStages;
                wait_bar(&S.sc_full[sst], (tile / kScaleStages) & 1, S, a.flags);
                const float sk = scale_ring[sst * 2 * kKeys + key];
                const float sv = fmaxf(scale_ring[sst * 2 * kKeys + kKeys + key], 0x1p-64f);   // (a NaN, of an unseen key, becomes a number)
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.sc_empty[sst]);
                const float lg = __log2f(sv), inv = sv < INFINITY ? ex2(-lg) : 0.f, ca = cq * sk;
                wait_bar(&S.s_full[buf], (tile >> 1) & 1, S, a.flags);
                tmem_fence_after_sync();
                // ---- t, and its maximum in each row ----
                uint64_t u[kC / 2];   // in pairs of rows
                const uint64_t ca2 = pack2(ca, ca), lg2 = pack2(lg, lg), inv2 = pack2(inv, inv), part = pack2(0.0625f, 0.0625f);
#pragma unroll
                for (int i0 = 0; i0 < kC; i0 += 16) {   // (32 at once spilled more)
                    uint32_t h[32];
                    tmem_ld16_two(lanes + buf * C::kNS + i0, lanes + buf * C::kNS + R + i0, h);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        u[i0 / 2 + i] = fma2(fma2(pack2(__uint_as_float(h[16 + 2 * i]), __uint_as_float(h[16 + 2 * i + 1])), part,
                                                  pack2(__uint_as_float(h[2 * i]), __uint_as_float(h[2 * i + 1]))), ca2, lg2);
                }
                if (masked)
#pragma unroll
                    for (int i = 0; i < kC / 2; ++i) {
                        float x, y;
                        unpack2(u[i], x, y);
                        if (!(seen >> (2 * i) & 1u)) x = -INFINITY;
                        if (!(seen >> (2 * i + 1) & 1u)) y = -INFINITY;
                        u[i] = pack2(x, y);
                    }
#pragma unroll
                for (int i = 0; i < kC; i += 4) {
                    float4 t;
                    unpack2(u[i / 2], t.x, t.y);
                    unpack2(u[i / 2 + 1], t.z, t.w);
                    t = make_float4(warp_max(t.x), warp_max(t.y), warp_max(t.z), warp_max(t.w));
                    if (lane == 0) *reinterpret_cast<float4*>(&S.top[quad][s0 + i]) = t;
                }
                named_barrier(1 + w, 128);
                bool far = false;
                const int fbuf = (int)(tile >> 1 & 1);
                if (wtid < kC) {
                    const int i = s0 + wtid;
                    const float m = fmaxf(fmaxf(fmaxf(S.top[0][i], S.top[1][i]), fmaxf(S.top[2][i], S.top[3][i])), kNone);
                    if (j == j1) M = m;
                    far = m > M + kFar;
                    if (far) {
                        S.grow[i] = ex2(M - m);
                        M = m;
                    } else {
                        S.grow[i] = 1.f;
                    }
                    S.shift[i] = kTop - m;
                    S.f[fbuf][i] = ex2(m - M - kTop);
                }
                if (vote128(1 + w, far)) {
                    if (pending) add_o(tile - 2);
                    pending = false;
#pragma unroll
                    for (int i = 0; i < kC; ++i) {
                        l[i] *= S.grow[s0 + i];
                        o[i] *= S.grow[s0 + i];
                    }
                }
                if (masked) {
                    // value rows past the context: zeros past the length (0 times whatever lies there
                    // must be 0), and for those with NaN codes, whose rows become NaN through l
                    const uint32_t vst = tile % C::kStages;
                    wait_bar(&S.v_full[vst], (tile / C::kStages) & 1, S, a.flags);
                    unsigned char* vrow = vs + vst * C::kStage + key * D;
                    uint32_t nan = 0;
                    if (d >= 0 && d < n)
#pragma unroll 4
                        for (int x = 0; x < D / 16; ++x) {   // (in an order that spreads a warp's rows over the banks)
                            const uint4 v = *reinterpret_cast<const uint4*>(vrow + ((x ^ key) & (D / 16 - 1)) * 16);
                            nan |= ((v.x & 0x7f7f7f7fu) + 0x01010101u) | ((v.y & 0x7f7f7f7fu) + 0x01010101u) |
                                   ((v.z & 0x7f7f7f7fu) + 0x01010101u) | ((v.w & 0x7f7f7f7fu) + 0x01010101u);
                        }
                    const bool bad = (nan & 0x80808080u) != 0;
                    if (bad || d >= n)
#pragma unroll 4
                        for (int x = 0; x < D / 16; ++x)
                            *reinterpret_cast<uint4*>(vrow + ((x ^ key) & (D / 16 - 1)) * 16) = make_uint4(0, 0, 0, 0);
                    if (bad)
#pragma unroll
                        for (int i = 0; i < kC; ++i)
                            if (seen >> i & 1u) l[i] = NAN;
                }
                // ---- weights: their sums, and their codes for the product with V ----
                unsigned char* pk = ps + buf * C::kPTile + key * C::kPRow;
                const int pswz = C::kPRow == 128 ? key & 7 : key >> 1 & 3;
#pragma unroll
                for (int i0 = 0; i0 < kC; i0 += 16) {
                    uint32_t c0[4], c1[4], c2[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int i = i0 + 4 * y;
                        const float4 g = *reinterpret_cast<const float4*>(&S.shift[s0 + i]);
                        const float4 f = *reinterpret_cast<const float4*>(&S.f[fbuf][s0 + i]);
                        float x0, x1, x2, x3;
                        unpack2(add2(u[i / 2], pack2(g.x, g.y)), x0, x1);
                        unpack2(add2(u[i / 2 + 1], pack2(g.z, g.w)), x2, x3);
                        x0 = ex2(x0), x1 = ex2(x1), x2 = ex2(x2), x3 = ex2(x3);
                        unpack2(fma2(pack2(x0, x1), mul2(inv2, pack2(f.x, f.y)), pack2(l[i], l[i + 1])), l[i], l[i + 1]);
                        unpack2(fma2(pack2(x2, x3), mul2(inv2, pack2(f.z, f.w)), pack2(l[i + 2], l[i + 3])), l[i + 2], l[i + 3]);
                        uint32_t h01, h23;
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h01) : "f"(x1), "f"(x0));
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h23) : "f"(x3), "f"(x2));
                        c0[y] = codes4(h01, h23, true);
                        c1[y] = codes4(h01, h23, true);
                        c2[y] = codes4(h01, h23, false);
                    }
                    auto put = [&](int part_, const uint32_t (&x)[4]) {
                        *reinterpret_cast<uint4*>(pk + ((((part_ * R + i0) >> 4) ^ pswz) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
                    };
                    put(0, c0);
                    put(1, c1);
                    put(2, c2);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                // the product before this one, while this one's is under way
                if (pending) add_o(tile - 2);
                tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.p_full[buf]);
                pending = true;
            }
            if (pending) {
                wait_bar(&S.pv_done[tile & 1], (tile >> 1) & 1, S, a.flags);
                tmem_fence_after_sync();
                add_o(tile);
            }
            tile = tile0 + U.nk;
            ++unit;
            // ---- the next unit's queries are on their way ----
            more = W.next(a);
            if (more) {
                rows = W.rows(a);
                load_q(W, rows);
                j0 = first_of();
            }
            // ---- the unit's result, or its part ----
            {
                const float sum = sum_columns<kC>(l);
                if (lane % (32 / kC) == 0) S.sum[quad][s0 + lane / (32 / kC)] = sum;
                if (wtid < kC) S.reference[s0 + wtid] = M;
            }
            named_barrier(3, 256);
            const int slot = 2 * blockIdx.x + (U.first ? 0 : 1);
            if (tid < nr) {   // a row: what its sums are to be multiplied by
                auto total = [&](int i) { return (S.sum[0][i] + S.sum[1][i]) + (S.sum[2][i] + S.sum[3][i]); };
                const float L0 = total(tid), L1 = total(R + tid), m0 = S.reference[tid], m1 = S.reference[R + tid], m = fmaxf(m0, m1);
                const float f0 = L0 == 0.f ? 0.f : ex2(m0 - m), f1 = L1 == 0.f ? 0.f : ex2(m1 - m), L = f0 * L0 + f1 * L1;
                if (!whole) a.ml[(size_t)slot * a.rows + tid] = make_float2(L == 0.f ? -INFINITY : m, L);
                else if (a.lse) a.lse[row_out[tid]] = L == 0.f ? -INFINITY : (m + log2f(L)) * 0.6931471805599453f;
                const float r = whole ? 1.f / L : 1.f;
                S.factor[tid] = L == 0.f ? 0.f : f0 * r;
                S.factor[R + tid] = L == 0.f ? 0.f : f1 * r;
            }
            named_barrier(3, 256);
            // each warpgroup hands half of its rows to the other, where the weights were
            constexpr int kHalf = R / 2;
            float* meet = reinterpret_cast<float*>(ps) + key;       // [2][kHalf][128]
#pragma unroll
            for (int i = 0; i < kC; ++i) o[i] = S.factor[s0 + i] == 0.f ? 0.f : o[i] * S.factor[s0 + i];
#pragma unroll
            for (int i = 0; i < kHalf; ++i) meet[(w * kHalf + i) * 128] = w ? o[i] : o[i + kHalf];
            named_barrier(3, 256);
            if (D == 128 || quad < 2) {
                const int e0 = w * kHalf;
#pragma unroll
                for (int i = 0; i < kHalf; ++i) {
                    if (e0 + i >= nr) break;
                    const float x = (w ? o[i + kHalf] : o[i]) + meet[((w ^ 1) * kHalf + i) * 128];
                    if (whole) static_cast<__nv_bfloat16*>(a.out)[(size_t)row_out[e0 + i] * D + key] = __float2bfloat16_rn(x);
                    else a.o[((size_t)slot * a.rows + e0 + i) * D + key] = x;
                }
            }
            tmem_fence_before_sync();
            if (more) qscale = finish_q(W, rows);   // (its barrier: and before a tile overwrites the rows' numbers)
        }
    }
    tmem_fence_before_sync();
    __syncthreads();
    if (aborted(S)) {   // (nobody sets it any more)
        // Copies and products that nobody waited for end before the shared and
        // the tensor memory are released: the last copy into each stage, and a
        // commit behind all MMAs.
        if (warp == 0)
            for (int v = 0; v < 2; ++v)
                for (uint32_t i = S.armed[v] > C::kStages ? S.armed[v] - C::kStages : 0; i < S.armed[v]; ++i)
                    mbar_wait(v ? &S.v_full[i % C::kStages] : &S.k_full[i % C::kStages], (i / C::kStages) & 1, kDrainPolls);
        if (warp == 1) {
            mma_commit(smem_u32(&S.drained));
            mbar_wait(&S.drained, 0, kDrainPolls);
        }
        __syncthreads();
    }
    if (warp == 1) {
        tmem_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, int R>
cudaError_t launch_q8_t(const AttentionArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int grid, cudaStream_t s) {
    using C = Cfg8<D, R>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        e = cudaFuncSetAttribute(attention_q8_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attention_q8_kernel<D, R>, a, mk, mv);
    if (e != cudaSuccess) return e;
    // a unit of one key tile is never cut
    if ((long long)a.max_pages * a.page_size <= kKeys || grid < 2) return cudaSuccess;
    return launch_join<__nv_bfloat16, D / 32, kUnitCost, true>(a, grid, R, cfg);
}

template <int D>
cudaError_t launch_q8_r(const AttentionArgs& a, long long rows, const CUtensorMap& mk, const CUtensorMap& mv, int grid, cudaStream_t s) {
    return rows <= 16 ? launch_q8_t<D, 16>(a, mk, mv, grid, s) : launch_q8_t<D, 32>(a, mk, mv, grid, s);
}

}  // namespace

// Most rows a key head, on average, that this file's kernel takes, in units of 16
// or 32; with more it reads the keys of a request three times.  Here / widened to bf16 /
// a cache in bf16, us: 64 requests of 2 tokens with 8 rows each to 8000 56 / - / 90, of 3 88 /
// 169 / 91, of 4 90 / 166 / 93, of 5 169 / 170 / -, of 6 172 / 171 / 95, of 8 171 / 176 / 96; 16 of
// 2 to 4000 17.8 / - / 23.9, of 3 23.7 / 35.6 / -, of 4 24.7 / 35.0 / 24.0, of 6 34.5 / 36.1 / -,
// of 8 34.8 / 37.0 / 25.7; one of 4 at 65000 33.7 / 46.9 / 37.0, of 8 43.4 / 54.2 / 44.9.  So from 33
// rows on a cache in 8 bits saves memory, and time only over one long context.  (Units of 32
// rows have 154 bytes of spill stores and 108 of loads, those of 16 none with heads of 128.)
constexpr int kFewRows = 64;

cudaError_t launch_attention_q8(const AttentionArgs& a, bool bf16, bool tiles, int sms, cudaStream_t s) {
    if (!tiles) return bf16 ? launch_plain<__nv_bfloat16, E4m3>(a, sms, s) : launch_plain<float, E4m3>(a, sms, s);
    // By the requests' rows a key head on average; T <= R is taken for one token each.
    const long long mean = ((long long)a.T * a.group + a.R - 1) / a.R, few = a.T <= a.R ? a.group : mean;
    if (few > kFewRows) return launch_attention_tc_q8(a, sms, s);
    const auto enc = tensor_map_encoder();
    if (!enc || sms <= 0) return cudaErrorNotSupported;
    const int grid = sms < kTcRanges ? sms : kTcRanges;
    const long long rows = (long long)a.n_pages * a.kv_heads * a.page_size;
    CUtensorMap mk, mv;
    const int box = a.page_size < kKeys ? a.page_size : kKeys;
    if (!encode_rows(&mk, enc, a.ck, a.D, rows, box) || !encode_rows(&mv, enc, a.cv, a.D, rows, box)) return cudaErrorInvalidValue;
    AttentionArgs b = a;
    b.min_steps = 1;
    return a.D == 128 ? launch_q8_r<128>(b, few, mk, mv, grid, s) : launch_q8_r<64>(b, few, mk, mv, grid, s);
}

}  // namespace moe
