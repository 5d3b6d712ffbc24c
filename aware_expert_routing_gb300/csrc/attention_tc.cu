// attention_tc.cu -- moe_tree_attention on the 5th-generation tensor cores:
// bf16 caches with heads of 64 or 128 components and pages of 8, 16, 32 or 64
// positions or a multiple of 128 (attention_tc_fits).
//
// For the query rows of one key head (every drafted token of a request times
// the query heads that share the key head, up to 128 rows a tile), over tiles
// of 128 keys:
//   S = Q K^T;  m' = max(m, rowmax S);  P = exp(scale (S - m'));
//   l = l exp(scale (m - m')) + rowsum P;  O = O exp(scale (m - m')) + P V;
// and at the end O / l.  Keys and values are read once per unit of work, so
// the cache's bytes bound the kernel while a key head has fewer than about
// 250 rows, and the chain from S over the softmax to P V above.  Measured, with
// heads of 128 and 4 key heads, called back to back (from one card to another up
// to 4 % apart): 256 single tokens up to 16000 positions (4.53 GB) 648 to 672 us,
// 6.7 to 7.0 TB/s, as fast as a plain copy; 64 up to 8000 (532 MB) 88 to 89 us,
// 6.0 TB/s, its DRAM reads 1.00 of these bytes; a tree of 64 tokens with 8 query
// heads a key head at 131000 positions 117 to 120 us, 1.17 PFLOP/s; one token at
// 1000 positions 10 us, nearly all of it latency: lengths, table, tile, S, P, O and
// the join one after the other.
//
//   * Work.  A unit is (request, key head, tile of rows); its key tiles follow
//     one another in one line with those of all other units, and each CTA (one
//     per SM) takes an equal stretch of the line, whatever the requests'
//     lengths.  A unit that lies in one stretch is finished there; one that is
//     cut leaves partial (m, l, O) per stretch, which a second kernel adds up
//     in the order of the stretches, so results repeat bit for bit.  (Joining
//     in this kernel, by the CTA that is last to write its part, was slower:
//     one SM reads a unit's parts for 10 to 40 us, and even with two parts its
//     fence and counter take as long as the second launch.)  Lengths are read
//     on the device: nothing depends on the host knowing them.
//   * A producer warp copies pages with TMA into a ring of key and value tiles
//     (8-row swizzle atoms side by side, so that pages of any number of atoms
//     make one operand), one warp issues the MMAs, and one warpgroup per row
//     tile does the softmax from tensor memory, a row a thread.
//   * S sits in two buffers of tensor memory.  With one row tile a unit (up to
//     128 rows) the next tile's S is computed while the softmax works on this
//     one; with two (up to 256 rows) each has a buffer and they take turns, and
//     each tile of keys and values is read once for both.
//   * Units of few rows would leave most of a tile's 128 rows empty and one warp
//     with all exponentials.  There the tile holds the unit's rows four times
//     (up to 16 rows) or twice (up to 64): each copy, or share, has a quarter or
//     half of the keys, its own maximum and sum, P zero elsewhere and its own O,
//     and the shares meet at the unit's end.
//   * P replaces S in tensor memory and is the A operand of P V, in bf16.  With
//     shares it is two bf16 numbers (the weight and what rounding left of it),
//     since with few rows one rounded large weight shows: the result's error is
//     then that of its own rounding alone.  Without shares it is one (off by up to
//     2^-8 of it), which puts the error of some hundred rows at 1.2 to 1.4 times
//     that (two would be 1.00, but, replayed from a graph, 31 against 24 us for 16
//     trees of 16 to 4000, 149 against 112 for a tree of 64 at 131000).
//   * O is corrected only when a row's maximum has grown by more than 8 powers
//     of two since the last correction (P then stays below 2^8, exact in the
//     sums), so almost never after the first tiles.
//   * Drafted positions: a row's mask words become 128 bits per key tile; only
//     tiles that reach past the context look at them.  Value rows past the
//     length are zeroed before the product (0 times whatever lies there must be
//     0), and so are drafted rows that are not finite: rows that see one become
//     NaN through l, the others are not touched.
//
// A cache in 8 bits (moe_tree_attention_q8), for requests of more rows a key head
// than attention_q8.cu takes: the codes are copied as they lie, and two
// warpgroups widen them to bf16 into the ring, one the keys, one the values; the
// rest is as above, without shares.  Half of the bytes come from HBM, but every
// tile costs about 1500 cycles a warpgroup of conversions, which share the issue
// slots with the softmax, and 64 KB written to shared memory and read from it
// besides what the MMAs read.  A tree of 64 at 131000 184 us (0.75 PFLOP/s; 217
// with eight warps on keys and values in turn and one row tile a unit, 202 with
// the keys left in e4m3 and their scales multiplied into S by the softmax; 112 to
// 122 in bf16), 16 trees of 16 to 4000 38.2 (27.5 in bf16; 37.5 with an instruction for
// registers in each of the warps' parts, which a warpgroup may not have), a prompt's
// 2000 tokens at 8000 585 (309), 500 at 32000 366 (204).  With two row tiles a thread's
// registers do not hold everything: 688 bytes of spill stores and 518 of loads (bf16: 4
// and 12) are a part of the issue slots that this costs.
#include <cudaTypedefs.h>

#include <cstddef>

#include "attention_line.cuh"
#include "tcgen05_tiles.cuh"

namespace moe {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();   // api.cu

namespace {

constexpr int kKeys = 128;     // keys per tile
constexpr int kRowsTile = 128; // query rows per tile
constexpr uint32_t kOCol = 256;   // tensor memory: S buffers at 0 and 128, O from here
// See attention_line.cuh.  3 / 4 / 5: 16 trees of 16 to 4000 25.3 / 24.4 / 24.4 us
// (replayed from a graph), 96 pairs of tokens at 127 16.6 / 16.5 / 18.1, 64 tokens
// to 8000 87.7 / 88.3 / 89.0, 38 trees of 12 to 7666 54.1 / 54.7 / 56.4, one token
// at 1000 9.6 / 9.6 / 9.4; 6 and 8 were no better.
constexpr int kUnitCost = 4;
// Polls of the last waits, for copies and products that run already: these end
// within microseconds, and the limit is there for a device that has failed.
constexpr uint32_t kDrainPolls = 1u << 20;
constexpr float kLazy = 8.f;   // powers of two that P may grow before O is corrected

// Whole warp: lane l receives consecutive 32-bit columns of TMEM lane
// (taddr >> 16) + l, from column taddr & 0xffff; complete on return.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63"
        "}, [%64];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
}

// Two weights as bf16, and what that leaves of them as bf16 again.
__device__ __forceinline__ void split2(float p0, float p1, uint32_t& hi, uint32_t& low) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(p0, p1);
    hi = *reinterpret_cast<const uint32_t*>(&p);
    const __nv_bfloat162 r = __floats2bfloat162_rn(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
    low = *reinterpret_cast<const uint32_t*>(&r);
}

// Two components of a result, over the row's sum l (its inverse inv); 0 for an empty row.
__device__ __forceinline__ uint32_t round2(float x, float y, float l, float inv) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(l == 0.f ? 0.f : x * inv, l == 0.f ? 0.f : y * inv);
    return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

// The MMA warp runs its loop as a whole, so that addresses and descriptors
// stay in uniform registers (issued from one thread's branch, every operand of
// every MMA is moved there first: 150 cycles an MMA, measured, against 64 for
// its work); an elected lane issues.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}

// kQ8: a cache in 8 bits, whose tiles further warps widen to bf16.
template <int D, int kTiles, int kShares, bool kQ8>
struct Cfg {
    // warps 0 and 1 copy and issue MMAs, the softmax's warpgroups follow; two
    // of those start at a warpgroup's boundary, so that registers can be moved
    // to them from the first one.  8 bits: warps 0, 2 and 3 copy keys, scales and
    // values, one warpgroup widens keys and one values.
    static constexpr int kFirst = kQ8 ? 12 : kTiles == 1 ? 2 : 4;
    static constexpr int kThreads = 32 * kFirst + 128 * kTiles;
    static constexpr int kBlocks = D / 64;              // 64-component blocks of a head
    static constexpr int kStage = kKeys * D * 2;        // a tile of keys or of values
    static constexpr int kQTile = kRowsTile * D * 2;
    static constexpr int kControl = 2048;
    static constexpr int kSmem = 227 * 1024;
    static constexpr int kSpan = kRowsTile / kShares;   // rows of a tile that a share has
    static constexpr int kRows = kShares == 4 ? 16 : kSpan * kTiles;   // rows of a unit
    // Where shares meet: as many blocks of 32 components at once as there are shares.
    static constexpr int kAtOnce = D / 32 < kShares ? D / 32 : kShares;
    static constexpr int kMeet = kAtOnce * (kShares - 1) * kRows * 128;
    // 8 bits: tiles as they are copied, a ring of keys and one of values; for four
    // tiles the scales, and what the keys' have besides a power of two
    static constexpr int kRaw = kKeys * D, kScaleStages = 4, kScales = kQ8 ? kScaleStages * 3 * kKeys * 4 : 0;
    static constexpr int kRoom = kSmem - 1024 - kControl - kTiles * kQTile - kMeet - kScales;
    // (8 bits, two row tiles: no room for a fourth; one: with three 16 trees of 16 to
    // 4000 take 37.9, with four 37.4 us)
    static constexpr int kStages = !kQ8 ? kRoom / kStage : kTiles == 1 ? 4 : 3;
    static constexpr int kRawRoom = (kRoom - kStages * kStage) / kRaw;
    static constexpr int kValStages = !kQ8 ? 1 : kRawRoom / 2 < 4 ? kRawRoom / 2 : 4;
    static constexpr int kKeyStages = !kQ8 ? 1 : kRawRoom - kValStages < 4 ? kRawRoom - kValStages : 4;
    static constexpr bool kLow = kShares > 1;
    static_assert(kStages <= 16 && (kTiles == 1 || kShares == 1), "barriers; shares of one row tile");
    static_assert(!kQ8 || (kValStages >= 1 && kStages <= kScaleStages), "rings; see odd_part");
};

struct Control {
    uint64_t full[16], empty[16], q_full[2], s_full[2], p_half[2], p_full[2], pv_done[2], drained;
    long long wait_cycles;
    LineStart start;
    int abort_flag;
    uint32_t armed[2];         // stages filled, or being filled, so far (8 bits: of keys, of values)
    uint32_t tmem_base;
    float2 ml[kRowsTile];      // shares' maxima and sums, when they meet
    uint32_t bad[2][2][4];     // per row tile and key tile's parity: keys whose value is not finite
    // 8 bits: keys and values as they are copied, the scales, and of four tiles which
    // keys' scales are no powers of two
    uint64_t raw_full[2][4], raw_empty[2][4], sc_full[4], sc_empty[4];
    alignas(16) uint32_t odd[4][4];
};
static_assert(sizeof(Control) <= 2048, "control block");

__device__ __forceinline__ bool aborted(Control& S) { return *(volatile int*)&S.abort_flag != 0; }

// The same for a whole warp that stays together.
__device__ __forceinline__ bool warp_aborted(Control& S) { return __any_sync(0xffffffffu, aborted(S)); }

// Bounded mbarrier wait; once the CTA has given up every later wait returns
// at once, so the control flow (and every barrier) still completes.
__device__ __forceinline__ void wait_bar(uint64_t* bar, uint32_t parity, Control& S, uint32_t* flags) {
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

// Bits d0 .. d0 + 127 of what token i of n sees among the drafted tokens
// (negative ones are the context): five words, shifted into four.
// mw0 and mw1: the mask's first two words.
__device__ __forceinline__ void seen_bits(const uint32_t* mrow, int words, uint32_t mw0, uint32_t mw1, int i, int n, int d0,
                                          uint32_t (&bits)[4]) {
    const int lim = mrow ? n : min(n, i + 1);
    const int w0 = d0 >> 5;   // rounds down
    uint32_t v[5];
#pragma unroll
    for (int x = 0; x < 5; ++x) {
        const int w = w0 + x;
        v[x] = w < 0 || !mrow ? 0xffffffffu : w == 0 ? mw0 : w == 1 ? mw1 : w < words ? mrow[w] : 0u;
    }
#pragma unroll
    for (int x = 0; x < 5; ++x) {
        const int k = lim - 32 * (w0 + x);
        if (w0 + x >= 0) v[x] = k <= 0 ? 0u : k < 32 ? v[x] & ((1u << k) - 1u) : v[x];
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) bits[x] = __funnelshift_r(v[x], v[x + 1], d0 & 31);
}

template <int D, int kTiles, int kShares, bool kQ8>
__global__ void __launch_bounds__(Cfg<D, kTiles, kShares, kQ8>::kThreads, 1)
attention_tc_kernel(const AttentionArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
    using C = Cfg<D, kTiles, kShares, kQ8>;
    using Walk = LineWalk<C::kRows, kKeys, kUnitCost>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* ring = smem;                                 // [kStages][kStage]
    unsigned char* qs = smem + C::kStages * C::kStage;          // [kTiles][kQTile]
    unsigned char* raw = qs + kTiles * C::kQTile + C::kMeet;    // 8 bits: [kKeyStages][kRaw] of keys, [kValStages][kRaw] of values
    float* scale_ring = reinterpret_cast<float*>(raw + (kQ8 ? (C::kKeyStages + C::kValStages) * C::kRaw : 0));   // [kScaleStages][2][kKeys]
    float* odd_part = scale_ring + C::kScaleStages * 2 * kKeys;                     // keys' scale / its power of two: [kScaleStages][kKeys]
    Control& S = *reinterpret_cast<Control*>(reinterpret_cast<unsigned char*>(scale_ring) + C::kScales);
    // 8 bits: registers; 512 x 128 at launch = 384 x 88 + 128 x 248, or 640 x 96 =
    // 384 x 48 + 256 x 168
    constexpr int kLess = kTiles == 1 ? 88 : 48, kMore = kTiles == 1 ? 248 : 168;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = a.group;
    // rows of row tile w of a unit
    auto rows_of = [&](const Walk& U, int w) { return max(0, min(kRowsTile, U.rows(a) - w * kRowsTile)); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&S.full[i], kQ8 ? 4 : 1);
            mbar_init(&S.empty[i], 1);
        }
        if (kQ8)
            for (int i = 0; i < 4; ++i) {
                mbar_init(&S.raw_full[0][i], 1);
                mbar_init(&S.raw_full[1][i], 1);
                mbar_init(&S.raw_empty[0][i], 4);
                mbar_init(&S.raw_empty[1][i], 4);
                mbar_init(&S.sc_full[i], 32);
                mbar_init(&S.sc_empty[i], 8);
            }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.q_full[i], 4);
            mbar_init(&S.s_full[i], 1);
            mbar_init(&S.p_half[i], 4);
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

    find_start<C::kRows, kKeys, kUnitCost, C::kThreads>(a, S.start);
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tmem = S.tmem_base;
    Walk W;
    const bool any = W.start(a, S.start);

    if (!any) {
        // no work for this CTA
    } else if (warp < C::kFirst) {
        // ---- all but the softmax ----
        // (Registers: one instruction for all warps of a warpgroup, whatever each of them does.)
        if (kQ8 || kTiles == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kQ8 ? kLess : 120));
        if (warp == 0 || (kQ8 && (warp == 2 || warp == 3))) {
            // ---- producer: pages into the ring, in the order in which the MMAs read them ----
            // (8 bits: a warp each for keys, scales and values)
            uint32_t seq = 0;
            const int page = a.page_size;
            const int per = page < kKeys ? kKeys / page : 1;        // pages of a tile
            const int prow = page < kKeys ? page : kKeys;           // rows of a copy
            const uint32_t bytes = (uint32_t)prow * D * (kQ8 ? 1 : 2);
            const int batch = 32 / per;                             // tiles whose table entries the warp reads at once
            const int my_tile = lane / per, my_page = lane - my_tile * per;
            const int wide = page / kKeys;                          // tiles of a page of more than 128 rows
            // This lane's page of the batch of tiles from j on of a part: is there
            // one, its entry in the table, and its first 8-row group in the cache
            // (-1: no page).
            auto has = [&](const Walk& U, int j) {
                return my_tile < batch && j + my_tile < U.nk && (U.kt + j + my_tile) * kKeys + my_page * prow < U.q.ctx + U.q.n;
            };
            auto read = [&](const Walk& U, int j) -> int {
                const int t = U.kt + j + my_tile;
                return has(U, j) ? a.page_table[(size_t)U.r * a.max_pages + (page <= kKeys ? t * per + my_page : t / wide)] : 0;
            };
            auto group_of = [&](int id, int j) -> int {
                if (!has(W, j)) return -1;
                if (id < 0 || id >= a.n_pages) {
                    raise_flag(a.flags, kFlagBadIndex);
                    id = 0;
                }
                const int row = page <= kKeys ? 0 : (W.kt + j + my_tile) % wide * kKeys;
                const long long at = ((long long)id * a.kv_heads + W.h) * page + row;
                return (int)(kQ8 ? at : at / 8);   // 8 bits: the row
            };
            const int vals = kQ8 && warp == 3 ? 1 : 0;
            const uint32_t stages = !kQ8 ? C::kStages : vals ? C::kValStages : C::kKeyStages;
            uint64_t *full = kQ8 ? S.raw_full[vals] : S.full, *empty = kQ8 ? S.raw_empty[vals] : S.empty;
            unsigned char* to = !kQ8 ? ring : raw + vals * C::kKeyStages * C::kRaw;
            auto load = [&](const CUtensorMap* map, int g) {
                const uint32_t st = kQ8 ? seq % stages : seq % C::kStages, ph = (kQ8 ? seq / stages : seq / C::kStages) & 1;
                wait_bar(&empty[st], ph ^ 1, S, a.flags);
                ++seq;
                const int n = __popc(__ballot_sync(0xffffffffu, g >= 0));
                if (warp_aborted(S)) return;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[st], n * bytes);
                    S.armed[vals] = seq;
                }
                __syncwarp();
                if (g < 0) return;
                if (kQ8) tma_rows(smem_u32(to + st * C::kRaw) + lane * bytes, map, g, &full[st]);
                else tma_load_4d(smem_u32(to + st * C::kStage) + lane * bytes, map, 0, 0, 0, g, &full[st]);
            };
            ScaleCopy<C::kScaleStages> scales(a, prow, lane);
            auto load_scales = [&](int cur, int at) {
                wait_bar(&S.sc_empty[scales.stage()], scales.phase() ^ 1, S, a.flags);
                scales.copy(a, cur, at, per, scale_ring, &S.sc_full[scales.stage()]);
            };
            int id0 = read(W, 0), id1 = read(W, batch);
            bool more = true;
            while (more) {
                int g_prev = -1, at = 0, cur = group_of(id0, 0), nxt = id1;
                Walk N = W;
                for (int j = 0; j < W.nk; ++j) {
                    const int t = __shfl_sync(0xffffffffu, cur, min(31, at * per + lane));
                    const int g = lane < per ? t : -1;
                    if (kQ8) {
                        if (warp == 2) load_scales(cur, at);
                        else load(vals ? &map_v : &map_k, g);
                    } else {
                        load(&map_k, g);
                        if (kTiles == 2) load(&map_v, g);
                        else if (j > 0) load(&map_v, g_prev);
                    }
                    if (j == 0) {   // the next part's first entries, while this part is loaded
                        more = N.next(a);
                        if (more) {
                            id0 = read(N, 0);
                            id1 = read(N, batch);
                        }
                    }
                    g_prev = g;
                    if (++at == batch) {
                        at = 0;
                        cur = group_of(nxt, j + 1);
                        nxt = read(W, j + 1 + batch);
                    }
                }
                if (!kQ8 && kTiles == 1) load(&map_v, g_prev);
                W = N;
            }
            if (kQ8) asm volatile("cp.async.wait_all;" ::: "memory");
        } else if (warp == 1) {
            // ---- MMA: one warp issues, in the order of the ring ----
            constexpr uint32_t idesc_s = umma_idesc_bf16(kRowsTile, kKeys);
            constexpr uint32_t idesc_o = umma_idesc_bf16(kRowsTile, D) | (1u << 16);   // V: MN-major
            const uint32_t ctl = uniform(smem_u32(&S)), ring0 = uniform(smem_u32(ring)), q0 = uniform(smem_u32(qs)), tm = uniform(tmem);
            uint32_t st = 0, ph = 0;                        // next stage of the ring, its phase
            uint32_t tile[2] = {0, 0}, seg[2] = {0, 0};     // per row tile: key tiles, units
            // waits for the next stage; its shared memory address
            auto stage_wait = [&](uint32_t s_, uint32_t p_) {
                wait_bar(&S.full[s_], p_, S, a.flags);
                tmem_fence_after_sync();
                return ring0 + s_ * C::kStage;
            };
            auto advance = [&]() {
                if (++st == C::kStages) {
                    st = 0;
                    ph ^= 1;
                }
            };
            // Shared-memory descriptors: a constant part, and the address in the
            // low word.  Q and K are K-major, 8-row groups 1024 and kBlocks * 1024
            // bytes apart.  V is MN-major: swizzle atoms of 8 keys by 64
            // components, 1024 bytes apart along the components (leading offset)
            // and kBlocks * 1024 along the keys (stride offset).
            constexpr uint64_t q_hi = (uint64_t)1 << 46 | (uint64_t)2 << 61 | (uint64_t)(1024 >> 4) << 32 | 1u << 16;
            constexpr uint64_t k_hi = (uint64_t)1 << 46 | (uint64_t)2 << 61 | (uint64_t)(C::kBlocks * 1024 >> 4) << 32 | 1u << 16;
            constexpr uint64_t v_hi = (uint64_t)1 << 46 | (uint64_t)2 << 61 | (uint64_t)(C::kBlocks * 1024 >> 4) << 32 | (1024u >> 4) << 16;
            auto issue_s = [&](int w, uint32_t buf, uint32_t kaddr) {
                const uint32_t qa = (q0 + w * C::kQTile) >> 4, ka = kaddr >> 4, d = tm + buf * 128;
    #pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_ss(d, q_hi | (qa + ((k / 4) * (kRowsTile * 128) + (k % 4) * 32) / 16),
                           k_hi | (ka + ((k / 4) * 1024 + (k % 4) * 32) / 16), idesc_s, k > 0);
                mma_commit(ctl + (uint32_t)offsetof(Control, s_full) + 8 * (buf));
            };
            // The product with V starts with the first 64 keys' P.
            auto issue_pv = [&](int w, uint32_t buf, uint32_t pp, uint32_t vaddr, uint32_t acc) {
                const uint32_t va = vaddr >> 4, d = tm + kOCol + w * D, p = tm + buf * 128;
    #pragma unroll
                for (int k = 0; k < kKeys / 16; ++k) {
                    if (k == kKeys / 32) {
                        wait_bar(&S.p_full[buf], pp, S, a.flags);
                        tmem_fence_after_sync();
                    }
                    const uint32_t pk = p + (k / 4) * 64 + (k % 4) * 8;
                    const uint64_t vk = v_hi | (va + k * 2 * C::kBlocks * 1024 / 16);
                    mma_ts(d, pk, vk, idesc_o, k > 0 ? 1u : acc);
                    if (C::kLow) mma_ts(d, pk + 32, vk, idesc_o, 1u);
                }
                mma_commit(ctl + (uint32_t)offsetof(Control, pv_done) + 8 * (kTiles == 1 ? buf : (uint32_t)w));
            };
            // Once a wait has given up, all return at once: the loop then runs out on
            // whatever the shared and tensor memory hold, which harms nothing.
            // (Leaving it early costs a vote a tile: 3 % for a tree of 64 tokens.)
            do {
                const int nw = uniform(kTiles == 2 && rows_of(W, 1) > 0 ? 2 : 1);
                const int n = uniform(W.nk);
                if (kTiles == 1) {
                    wait_bar(&S.q_full[0], seg[0]++ & 1, S, a.flags);
                    uint32_t kaddr = stage_wait(st, ph);
                    issue_s(0, tile[0] & 1, kaddr);
                    mma_commit(ctl + (uint32_t)offsetof(Control, empty) + 8 * (st));
                    advance();
                    for (int j = 0; j < n; ++j) {
                        if (j + 1 < n) {
                            kaddr = stage_wait(st, ph);
                            issue_s(0, (tile[0] + 1) & 1, kaddr);
                            mma_commit(ctl + (uint32_t)offsetof(Control, empty) + 8 * (st));
                            advance();
                        }
                        const uint32_t buf = tile[0] & 1;
                        const uint32_t pp = (tile[0] >> 1) & 1;
                        wait_bar(&S.p_half[buf], pp, S, a.flags);
                        const uint32_t vaddr = stage_wait(st, ph);
                        issue_pv(0, buf, pp, vaddr, j > 0);
                        mma_commit(ctl + (uint32_t)offsetof(Control, empty) + 8 * (st));
                        advance();
                        ++tile[0];
                    }
                } else {
                    uint32_t kaddr = stage_wait(st, ph);
                    for (int w = 0; w < nw; ++w) {
                        wait_bar(&S.q_full[w], seg[w]++ & 1, S, a.flags);
                        issue_s(w, w, kaddr);
                    }
                    mma_commit(ctl + (uint32_t)offsetof(Control, empty) + 8 * (st));
                    advance();
                    for (int j = 0; j < n; ++j) {
                        const uint32_t v_st = st, v_ph = ph;
                        advance();
                        uint32_t vaddr = 0;
                        for (int w = 0; w < nw; ++w) {
                            const uint32_t pp = tile[w] & 1;
                            wait_bar(&S.p_half[w], pp, S, a.flags);
                            ++tile[w];
                            if (w == 0) vaddr = stage_wait(v_st, v_ph);
                            tmem_fence_after_sync();
                            issue_pv(w, w, pp, vaddr, j > 0);
                            if (w == nw - 1) mma_commit(ctl + (uint32_t)offsetof(Control, empty) + 8 * (v_st));
                            if (j + 1 < n) {
                                if (w == 0) kaddr = stage_wait(st, ph);
                                issue_s(w, w, kaddr);
                                if (w == nw - 1) mma_commit(ctl + (uint32_t)offsetof(Control, empty) + 8 * (st));
                            }
                        }
                        if (j + 1 < n) advance();
                    }
                }
            } while (W.next(a));
        } else if (kQ8 && warp >= 4) {
            // ---- 8 bits: tiles to bf16; a warpgroup the keys, one the values; thread = key ----
            // A code times a power of two is exact in bf16.  What a scale has besides one
            // (which no append writes) is multiplied into the scores for keys; values are
            // rounded to bf16 with it.
            const int v = (warp - 4) / 4, key = threadIdx.x & 127, swz = D == 128 ? key & 7 : key >> 1 & 3;
            const uint32_t stages = v ? C::kValStages : C::kKeyStages;
            const unsigned char* rows = raw + v * C::kKeyStages * C::kRaw + key * D;
            unsigned char* const to = ring + (key >> 3) * (C::kBlocks * 1024) + (key & 7) * 128;
            constexpr int kAtOnce = kTiles == 1 ? D / 16 : 2;   // (few registers)
            uint32_t tile = 0, seq0 = 0;
            do {
                for (int j = 0; j < W.nk; ++j, ++tile) {
                    // (its place in the ring, which the MMAs read in the order K0 K1 V0 K2 V1 ..., with two row tiles K0 V0 K1 V1 ...)
                    const uint32_t seq = seq0 + (kTiles == 2 ? 2 * j + v : v ? j == W.nk - 1 ? 2 * j + 1 : 2 * j + 2 : j == 0 ? 0 : 2 * j - 1);
                    const uint32_t sst = tile % C::kScaleStages, st = seq % C::kStages, rst = tile % stages;
                    wait_bar(&S.sc_full[sst], (tile / C::kScaleStages) & 1, S, a.flags);
                    float f = scale_ring[(sst * 2 + v) * kKeys + key];
                    wait_bar(&S.raw_full[v][rst], (tile / stages) & 1, S, a.flags);
                    const unsigned char* from = rows + rst * C::kRaw;
                    wait_bar(&S.empty[st], ((seq / C::kStages) & 1) ^ 1, S, a.flags);
                    if (v == 0) {
                        // (From here on the softmax of the tile four before has read its own: this
                        // place in the ring was that of a later tile's keys or values, whose product came
                        // after its weights.)
                        const uint32_t bits = __float_as_uint(f);
                        const float p = __uint_as_float(bits & 0xff800000u);
                        const bool odd = (bits & 0x7fffffu) != 0 && p != 0.f && fabsf(p) < INFINITY;
                        odd_part[sst * kKeys + key] = odd ? __uint_as_float((bits & 0x7fffffu) | 0x3f800000u) : 1.f;
                        const uint32_t word = __ballot_sync(0xffffffffu, odd);
                        if (lane == 0) S.odd[sst][warp & 3] = word;
                        f = p;
                    }
    #pragma unroll
                    for (int x0 = 0; x0 < D / 16; x0 += kAtOnce) {
                        uint4 c[kAtOnce];
    #pragma unroll
                        for (int x = 0; x < kAtOnce; ++x) c[x] = *reinterpret_cast<const uint4*>(from + ((x0 + x ^ swz) << 4));
                        if (x0 + kAtOnce == D / 16) {
                            __syncwarp();
                            if (lane == 0) {
                                mbar_arrive(&S.raw_empty[v][rst]);
                                mbar_arrive(&S.sc_empty[sst]);
                            }
                        }
    #pragma unroll
                        for (int x = 0; x < kAtOnce; ++x) {
                            const uint32_t w[4] = {c[x].x, c[x].y, c[x].z, c[x].w};
                            uint32_t y[8];
    #pragma unroll
                            for (int z = 0; z < 8; ++z) y[z] = scaled2(w[z >> 1] >> (z & 1) * 16, f);
                            const int ch = 2 * (x0 + x);   // 16-byte pieces of the row in bf16
                            unsigned char* at = to + st * C::kStage + (ch >> 3) * 1024;
                            *reinterpret_cast<uint4*>(at + (((ch & 7) ^ (key & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                            *reinterpret_cast<uint4*>(at + (((ch & 7) + 1 ^ (key & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.full[st]);
                }
                seq0 += 2 * W.nk;
            } while (W.next(a));
        }
    } else {
        // ---- softmax: warpgroup w owns row tile w, thread = row = TMEM lane ----
        // registers: 384 x 168 at launch = 128 x 120 + 256 x 192
        if (kQ8 || kTiles == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kQ8 ? kMore : 192));
        const int w = (warp - C::kFirst) >> 2, quad = warp & 3;
        // With shares, each holds the unit's rows again, for its own keys of a tile.
        constexpr int kWarps = 4 / kShares;           // of a share
        const int share = kShares == 1 ? 0 : quad / kWarps;
        const int row = kShares == 1 ? quad * 32 + lane : quad % kWarps * 32 + lane;
        const int krow = quad * 32 + lane;            // the key of a tile that this thread looks after
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const int qwarp = (warp - C::kFirst) & 3;     // this warp's share of the query copy
        unsigned char* q_dst = qs + w * C::kQTile;
        const float c = a.scale * 1.4426950408889634f;   // scores to powers of two
        uint32_t seq = 0, tile = 0;
        // The product of this row tile's key tile t is in O.  A wait tells two
        // phases of its barrier apart, so each must find the phase before its
        // own complete.  With one row tile that is only known of t - 2 (its
        // product precedes S of t; t - 1's may still wait for its values), so
        // even and odd tiles have barriers of their own.
        auto wait_pv = [&](uint32_t t) {
            if (kTiles == 1) wait_bar(&S.pv_done[t & 1], (t >> 1) & 1, S, a.flags);
            else wait_bar(&S.pv_done[w], t & 1, S, a.flags);
        };

        // A unit's queries, rows of 128 bytes per 64 components, swizzled:
        // asynchronous copies, then their completion for the MMAs.
        constexpr int kLanes = D / 8;               // lanes per row, 16 bytes each
        constexpr int kPer = 32 / kLanes, kStep = 4 * kPer;   // rows per warp, and of all four at a step
        const int ch = lane % kLanes, qrow = qwarp * kPer + lane / kLanes;
        const uint32_t q_to = smem_u32(q_dst) + (ch >> 3) * (kRowsTile * 128) + qrow * 128 + (((ch & 7) ^ (qrow & 7)) << 4);
        const int step_tok = kStep / group, step_g = kStep - step_tok * group;
        const long long step = step_tok * a.q_tok + step_g * a.q_head, wrap = a.q_tok - group * a.q_head;
        auto copy_q = [&](const Walk& U, int rows) {
            if (qrow >= rows) return;
            const int gr = U.rt * C::kRows + w * kRowsTile + qrow, tok = gr / group;
            int g = gr - tok * group;
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (U.q.t0 + tok) * a.q_tok +
                                       (U.h * group + g) * a.q_head + ch * 8;
            uint32_t to = q_to;
            static_assert(kStep % 8 == 0, "the swizzle is the same at every step");
#pragma unroll 4
            for (int r0 = qrow; r0 < rows; r0 += kStep) {
#pragma unroll
                for (int x = 0; x < kShares; ++x)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + x * C::kSpan * 128), "l"(src) : "memory");
                to += kStep * 128;
                src += step;
                g += step_g;
                if (g >= group) {
                    g -= group;
                    src += wrap;
                }
            }
        };
        auto finish_q = [&]() {
            asm volatile("cp.async.wait_all;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.q_full[w]);
        };

        // The mask words of this row's token in a unit, on their way early.
        uint32_t mw[2];
        auto read_mask = [&](const Walk& U, int rows) {
            mw[0] = mw[1] = 0u;
            if (!a.mask || row >= rows) return;
            const int gr = U.rt * C::kRows + w * kRowsTile + row;
            const uint32_t* mrow = a.mask + (size_t)(U.q.t0 + gr / group) * a.mask_words;
            mw[0] = mrow[0];
            if (a.mask_words > 1) mw[1] = mrow[1];
        };

        int rows = rows_of(W, w);
        if (rows > 0) {
            copy_q(W, rows);
            read_mask(W, rows);
            finish_q();
        }
        bool more = true;
        while (more) {
            const Walk U = W;
            const int nr = rows;
            const int n = U.q.n, len = U.q.ctx + n;
            const bool both = kTiles == 2 && rows_of(U, 1) > 0;
            if (nr == 0) {   // this warpgroup has no rows in the unit
                seq += 2 * U.nk;
                more = W.next(a);
                rows = more ? rows_of(W, w) : 0;
                if (rows > 0) {
                    copy_q(W, rows);
                    read_mask(W, rows);
                    finish_q();
                }
                continue;
            }
            const bool live = row - lane < nr;         // this warp has rows
            const bool valid = row < nr;
            const int gr = U.rt * C::kRows + w * kRowsTile + (valid ? row : 0);
            const int ti = gr / group;                 // token within the request
            const uint32_t* mrow = a.mask ? a.mask + (size_t)(U.q.t0 + ti) * a.mask_words : nullptr;
            const size_t orow = (size_t)(U.q.t0 + ti) * a.heads + U.h * group + (gr - ti * group);
            const bool whole = U.nk == U.q.nkt;
            const int slot = 2 * blockIdx.x + (U.first ? 0 : 1);
            const uint32_t mw0 = mw[0], mw1 = mw[1];
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < U.nk; ++j) {
                const uint32_t buf = kTiles == 1 ? (tile & 1) : (uint32_t)w;
                const uint32_t sph = kTiles == 1 ? (tile >> 1) & 1 : tile & 1;
                const int k0 = (U.kt + j) * kKeys;
                const bool masked = k0 + kKeys > U.q.ctx;
                uint32_t bits[4] = {~0u, ~0u, ~0u, ~0u};
                float poison = 0.f;
                if (masked) seen_bits(mrow, a.mask_words, mw0, mw1, ti, n, k0 - U.q.ctx, bits);
                wait_bar(&S.s_full[buf], sph, S, a.flags);
                tmem_fence_after_sync();
                if (j == U.nk - 1) {   // the queries have been read for the last time: the next unit's, meanwhile
                    more = W.next(a);
                    rows = more ? rows_of(W, w) : 0;
                    copy_q(W, rows);
                    read_mask(W, rows);
                }
                // 8 bits: whether scales of the tile's keys are no powers of two
                const uint32_t sst = (seq / 2 + j) % C::kScaleStages;
                bool odd_k = false;
                if (kQ8) {
                    const uint4 o = *reinterpret_cast<const uint4*>(S.odd[sst]);
                    odd_k = (o.x | o.y | o.z | o.w) != 0;
                }
                constexpr int kWidth = kKeys / kShares;   // a share's keys of a tile
                uint32_t own32[32], own64[64];
                // m for a tile of maximum mt; returns the exponents' offset.
                auto new_max = [&](float mt) {
                    if (j == 0) {
                        m = mt;
                    } else {
                        // (lanes past the unit's rows hold anything, and must not decide)
                        const bool grow = valid && (m == -INFINITY ? mt > -INFINITY : (mt - m) * c > kLazy);
                        if (__any_sync(0xffffffffu, grow)) {
                            // the previous tile's product has to be in O before it is corrected
                            const float mn = fmaxf(m, mt), f = m == -INFINITY ? 0.f : ex2((m - mn) * c);
                            wait_pv(tile - 1);
                            tmem_fence_after_sync();
#pragma unroll 1
                            for (int x = 0; x < D / 32; ++x) {
                                uint32_t o[32];
                                tmem_ld32(lanes + kOCol + w * D + x * 32, o);
#pragma unroll
                                for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                                tmem_st32(lanes + kOCol + w * D + x * 32, o);
                            }
                            l *= f;
                            m = mn;
                        }
                    }
                    return m == -INFINITY ? 0.f : -m * c;
                };
                // The maximum, then P, 64 columns at a time.  With one row
                // tile the row stays in registers between the two; with two
                // (192 registers) it would spill, and S is read twice: 117
                // against 121 us for 1x64 at 131000.  (One tile: 27.6
                // against 28.4 us for 16 trees of 16 to 4000.)
                constexpr bool kHold = kTiles == 1 && !kQ8;   // (8 bits: it would spill)
                constexpr int kTimes = kHold ? 2 : 1;
                uint32_t s[kTimes][64];
                auto load_s = [&](int x) {
                    uint32_t(&h)[64] = s[kHold ? x : 0];
                    tmem_ld64(lanes + buf * 128 + x * 64, h);
                    if (kQ8 && odd_k)
#pragma unroll
                        for (int y = 0; y < 64; ++y) h[y] = __float_as_uint(__uint_as_float(h[y]) * odd_part[sst * kKeys + x * 64 + y]);
                    if (masked) {
                        const uint32_t b0 = x ? bits[2] : bits[0], b1 = x ? bits[3] : bits[1];
#pragma unroll
                        for (int y = 0; y < 64; ++y)
                            if (!(((y < 32 ? b0 : b1) >> (y & 31)) & 1u)) h[y] = 0xff800000u;   // -inf
                    }
                };
                float off = 0.f;
                if (kShares > 1) {
                    if (live) {
                        if (kWidth == 32) tmem_ld32(lanes + buf * 128 + share * 32, own32);
                        else tmem_ld64(lanes + buf * 128 + share * 64, own64);
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        const uint32_t b0 = kWidth == 64 ? (share ? bits[2] : bits[0]) : share < 2 ? (share ? bits[1] : bits[0]) : share == 2 ? bits[2] : bits[3];
                        const uint32_t b1 = share ? bits[3] : bits[1];
#pragma unroll
                        for (int y = 0; y < kWidth; ++y) {
                            uint32_t& v = kWidth == 32 ? own32[y & 31] : own64[y];
                            if (masked && !(((y < 32 ? b0 : b1) >> (y & 31)) & 1u)) v = 0xff800000u;   // -inf
                            mx[y & 3] = fmaxf(mx[y & 3], __uint_as_float(v));
                        }
                        off = new_max(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                    }
                } else if (live) {
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll kTimes
                    for (int x = 0; x < 2; ++x) {
                        load_s(x);
#pragma unroll
                        for (int y = 0; y < 64; ++y) mx[y & 3] = fmaxf(mx[y & 3], __uint_as_float(s[kHold ? x : 0][y]));
                    }
                    const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    off = new_max(mt);
                }
                if (masked) {
                    // value rows past the context: zero those past the length, and those that are not finite
                    const uint32_t vseq = seq + (kTiles == 2 ? 2 * j + 1 : j == U.nk - 1 ? 2 * j + 1 : 2 * j + 2);
                    wait_bar(&S.full[vseq % C::kStages], (vseq / C::kStages) & 1, S, a.flags);
                    unsigned char* vrow = ring + (vseq % C::kStages) * C::kStage + (krow >> 3) * (C::kBlocks * 1024) + (krow & 7) * 128;
                    // (a bf16 of all-ones exponent carries into bit 15 when 0x80 is added)
                    uint32_t top = 0;
                    if (k0 + krow >= U.q.ctx && k0 + krow < len)
#pragma unroll 4
                        for (int x = 0; x < D / 8; ++x) {   // the swizzle's order: no two rows of eight in one bank
                            const uint4 v = *reinterpret_cast<const uint4*>(vrow + (x >> 3) * 1024 + (((x ^ krow) & 7) << 4));
                            top |= ((v.x & 0x7fff7fffu) + 0x00800080u) | ((v.y & 0x7fff7fffu) + 0x00800080u) |
                                   ((v.z & 0x7fff7fffu) + 0x00800080u) | ((v.w & 0x7fff7fffu) + 0x00800080u);
                        }
                    const bool bad = (top & 0x80008000u) != 0;
                    const uint32_t badw = __ballot_sync(0xffffffffu, bad);
                    if (lane == 0) S.bad[w][tile & 1][quad] = badw;   // the other parity may still be read
                    // all have looked before anyone zeroes
                    if (both) named_barrier(1, 256); else named_barrier(2 + w, 128);
                    if (w == 0 && (bad || k0 + krow >= len))
#pragma unroll 4
                        for (int x = 0; x < D / 8; ++x)
                            *reinterpret_cast<uint4*>(vrow + (x >> 3) * 1024 + (((x ^ krow) & 7) << 4)) = make_uint4(0, 0, 0, 0);
                    if (w == 0) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (bits[x] & S.bad[w][tile & 1][x]) poison = NAN;
                }
                if (kShares > 1) {
                    // P of this share's keys, in two bf16 parts; zero where the other shares' keys are
                    if (live) {
                        const uint64_t c2 = pack2(c, c), off2 = pack2(off, off);
                        uint64_t sum[2] = {0, 0};
                        uint32_t hi[32], low[32], none[32];
#pragma unroll
                        for (int y = 0; y < 32; ++y) none[y] = 0;
#pragma unroll
                        for (int y = 0; y < kWidth / 2; ++y) {
                            float p0, p1;
                            unpack2(fma2(pack2(__uint_as_float(kWidth == 32 ? own32[(2 * y) & 31] : own64[2 * y]),
                                               __uint_as_float(kWidth == 32 ? own32[(2 * y + 1) & 31] : own64[2 * y + 1])), c2, off2), p0, p1);
                            p0 = ex2(p0);
                            p1 = ex2(p1);
                            sum[y & 1] = add2(sum[y & 1], pack2(p0, p1));
                            split2(p0, p1, hi[y], low[y]);
                        }
                        const uint32_t at = lanes + buf * 128;
                        if (kWidth == 32) {
                            const uint32_t mine = at + (share >> 1) * 64 + (share & 1) * 16, other = at + (share >> 1) * 64 + (~share & 1) * 16;
                            tmem_st16(mine, hi);
                            tmem_st16(mine + 32, low);
                            tmem_st16(other, none);
                            tmem_st16(other + 32, none);
                            tmem_st32(at + (~share >> 1 & 1) * 64, none);
                            tmem_st32(at + (~share >> 1 & 1) * 64 + 32, none);
                        } else {
                            tmem_st32(at + share * 64, hi);
                            tmem_st32(at + share * 64 + 32, low);
                            tmem_st32(at + (share ^ 1) * 64, none);
                            tmem_st32(at + (share ^ 1) * 64 + 32, none);
                        }
                        tmem_wait_st();
                        float s0, s1;
                        unpack2(add2(sum[0], sum[1]), s0, s1);
                        l += s0 + s1 + poison;
                    }
                    tmem_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&S.p_half[buf]);
                        mbar_arrive(&S.p_full[buf]);
                    }
                } else if (live) {
                    const uint64_t c2 = pack2(c, c), off2 = pack2(off, off);
                    uint64_t sum[2] = {0, 0};
#pragma unroll kTimes
                    for (int x = 0; x < 2; ++x) {
                        if (!kHold) load_s(x);
                        uint32_t(&h)[64] = s[kHold ? x : 0];
#pragma unroll
                        for (int y = 0; y < 32; ++y) {
                            float p0, p1;
                            unpack2(fma2(pack2(__uint_as_float(h[2 * y]), __uint_as_float(h[2 * y + 1])), c2, off2), p0, p1);
                            p0 = ex2(p0);
                            p1 = ex2(p1);
                            sum[y & 1] = add2(sum[y & 1], pack2(p0, p1));
                            const __nv_bfloat162 p = __floats2bfloat162_rn(p0, p1);
                            h[y] = *reinterpret_cast<const uint32_t*>(&p);
                        }
                        tmem_st32(lanes + buf * 128 + x * 64, h);   // over columns of S that have been read
                        tmem_wait_st();
                        tmem_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(x ? &S.p_full[buf] : &S.p_half[buf]);
                    }
                    float s0, s1;
                    unpack2(add2(sum[0], sum[1]), s0, s1);
                    l += s0 + s1 + poison;
                } else {
                    tmem_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&S.p_half[buf]);
                        mbar_arrive(&S.p_full[buf]);
                    }
                }
                ++tile;
            }
            seq += 2 * U.nk;
            if (rows > 0) finish_q();
            // ---- the unit's result, or its part ----
            wait_pv(tile - 1);
            tmem_fence_after_sync();
            if (kShares > 1) {
                // the shares meet, 32 components at a time, each time with another of them
                S.ml[krow] = make_float2(m, l);
                named_barrier(2, 128);
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int x = 0; x < kShares; ++x) M = fmaxf(M, S.ml[x * C::kSpan + row].x);
#pragma unroll
                for (int x = 0; x < kShares; ++x) {
                    const float2 e = S.ml[x * C::kSpan + row];
                    L = fmaf(e.x == -INFINITY ? 0.f : ex2((e.x - M) * c), e.y, L);
                }
                const float f = m == -INFINITY ? 0.f : ex2((m - M) * c), inv = L == 0.f ? 0.f : 1.f / L;
                float4* meet = reinterpret_cast<float4*>(qs + kTiles * C::kQTile) + row;
                float4 v[8];
                auto load_o = [&](int x) {
                    uint32_t o[32];
                    __syncwarp();   // the load is the whole warp's
                    tmem_ld32(lanes + kOCol + x * 32, o);
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        v[y] = make_float4(__uint_as_float(o[4 * y]) * f, __uint_as_float(o[4 * y + 1]) * f,
                                           __uint_as_float(o[4 * y + 2]) * f, __uint_as_float(o[4 * y + 3]) * f);
                };
#pragma unroll 1
                for (int x0 = 0; x0 < D / 32; x0 += C::kAtOnce) {
                    __syncwarp();
                    if (x0 > 0) named_barrier(2, 128);   // the last ones have been read
#pragma unroll 1
                    for (int x = 0; x < C::kAtOnce; ++x) {
                        if (x == share) continue;
                        load_o(x0 + x);
                        if (valid)
#pragma unroll
                            for (int y = 0; y < 8; ++y)
                                meet[((x * (kShares - 1) + (share < x ? share : share - 1)) * 8 + y) * C::kRows] = v[y];
                    }
                    named_barrier(2, 128);
                    if (share >= C::kAtOnce) continue;
                    const int x = x0 + share;
                    load_o(x);
                    if (!valid) continue;
#pragma unroll
                    for (int z = 0; z < kShares - 1; ++z)
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            const float4 e = meet[((share * (kShares - 1) + z) * 8 + y) * C::kRows];
                            v[y] = make_float4(v[y].x + e.x, v[y].y + e.y, v[y].z + e.z, v[y].w + e.w);
                        }
                    if (whole) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + orow * D + x * 32);
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            dst[y] = make_uint4(round2(v[2 * y].x, v[2 * y].y, L, inv), round2(v[2 * y].z, v[2 * y].w, L, inv),
                                                round2(v[2 * y + 1].x, v[2 * y + 1].y, L, inv), round2(v[2 * y + 1].z, v[2 * y + 1].w, L, inv));
                    } else {
                        float4* part = reinterpret_cast<float4*>(a.o) + ((size_t)slot * a.rows + (row - lane)) * (D / 4) + lane;
#pragma unroll
                        for (int y = 0; y < 8; ++y) part[(x * 8 + y) * 32] = v[y];
                    }
                }
                __syncwarp();
                if (valid && share == 0) {
                    if (!whole) a.ml[(size_t)slot * a.rows + row] = make_float2(M * c, L);
                    else if (a.lse) a.lse[orow] = L == 0.f ? -INFINITY : M * a.scale + logf(L);
                }
                tmem_fence_before_sync();   // read before the next unit's product overwrites O
            } else if (live) {
                const size_t prow = (size_t)slot * a.rows + w * kRowsTile + row;
                // 32 rows of a part lie side by side: [D / 4][32] float4
                float4* part = reinterpret_cast<float4*>(a.o) + ((size_t)slot * a.rows + w * kRowsTile + quad * 32) * (D / 4) + lane;
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
                for (int x = 0; x < D / 32; ++x) {   // (rolled: this code runs once or twice, its fetch counts)
                    uint32_t o[32];
                    __syncwarp();   // the load is the whole warp's
                    tmem_ld32(lanes + kOCol + w * D + x * 32, o);
                    if (whole && valid) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + orow * D + x * 32);
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            uint32_t v[4];
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                const __nv_bfloat162 p = __floats2bfloat162_rn(
                                    l == 0.f ? 0.f : __uint_as_float(o[8 * y + 2 * z]) * inv,
                                    l == 0.f ? 0.f : __uint_as_float(o[8 * y + 2 * z + 1]) * inv);
                                v[z] = *reinterpret_cast<const uint32_t*>(&p);
                            }
                            dst[y] = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    } else if (valid) {
#pragma unroll
                        for (int y = 0; y < 8; ++y)
                            part[(x * 8 + y) * 32] = make_float4(__uint_as_float(o[4 * y]), __uint_as_float(o[4 * y + 1]),
                                                                 __uint_as_float(o[4 * y + 2]), __uint_as_float(o[4 * y + 3]));
                    }
                }
                if (valid) {
                    if (!whole) a.ml[prow] = make_float2(m * c, l);
                    else if (a.lse) a.lse[orow] = l == 0.f ? -INFINITY : m * a.scale + logf(l);
                }
                tmem_fence_before_sync();   // read before the next unit's product overwrites O
            }
        }
    }
    tmem_fence_before_sync();
    __syncthreads();
    if (aborted(S)) {   // (nobody sets it any more)
        // Copies and products that nobody waited for end before the shared and
        // the tensor memory are released: the last copy into each stage, and a
        // commit behind all MMAs.
        auto drain = [&](uint64_t* full, uint32_t armed, uint32_t stages) {
            for (uint32_t i = armed > stages ? armed - stages : 0; i < armed; ++i)
                mbar_wait(&full[i % stages], (i / stages) & 1, kDrainPolls);
        };
        if (warp == 0) {
            drain(kQ8 ? S.raw_full[0] : S.full, S.armed[0], kQ8 ? C::kKeyStages : C::kStages);
            if (kQ8) drain(S.raw_full[1], S.armed[1], C::kValStages);
        }
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

// The cache seen as 8-row groups of swizzle atoms: {64 components, 8 rows,
// blocks of 64, groups}; one box is a page's rows of one key head (or 128).
bool encode_cache(CUtensorMap* m, PFN_cuTensorMapEncodeTiled_v12000 enc, const void* base, int D, long long rows, int box_rows) {
    cuuint64_t dims[4] = {64, 8, (cuuint64_t)(D / 64), (cuuint64_t)(rows / 8)};
    cuuint64_t strides[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 16};
    cuuint32_t box[4] = {64, 8, (cuuint32_t)(D / 64), (cuuint32_t)(box_rows / 8)};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int kTiles, int kShares, bool kQ8 = false>
cudaError_t launch_t(const AttentionArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int grid, cudaStream_t s) {
    using C = Cfg<D, kTiles, kShares, kQ8>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        e = cudaFuncSetAttribute(attention_tc_kernel<D, kTiles, kShares, kQ8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
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
    e = cudaLaunchKernelEx(&cfg, attention_tc_kernel<D, kTiles, kShares, kQ8>, a, mk, mv);
    if (e != cudaSuccess) return e;
    // a unit of one key tile is never cut
    if ((long long)a.max_pages * a.page_size <= kKeys || grid < 2) return cudaSuccess;
    return launch_join<__nv_bfloat16, D / 32, kUnitCost>(a, grid, C::kRows, cfg);
}

}  // namespace

cudaError_t launch_attention_tc(const AttentionArgs& a, int sms, cudaStream_t s) {
    const auto enc = tensor_map_encoder();
    if (!enc || sms <= 0) return cudaErrorNotSupported;
    const int grid = sms < kTcRanges ? sms : kTcRanges;
    const long long rows = (long long)a.n_pages * a.kv_heads * a.page_size;
    CUtensorMap mk, mv;
    const int box = a.page_size < kKeys ? a.page_size : kKeys;
    if (!encode_cache(&mk, enc, a.ck, a.D, rows, box) || !encode_cache(&mv, enc, a.cv, a.D, rows, box))
        return cudaErrorInvalidValue;
    // Two row tiles a unit where the requests have more than 128 rows a key
    // head on average: their keys and values are then read once, not twice.
    const bool two = (long long)a.T * a.group > 128LL * a.R;
    // Cutting units of so many rows finer costs more on their parts, which are
    // written and read again (2 requests of 27 x 8 rows at 2276: 1 step 23.0, 2
    // 20.2, 4 21.8, 6 23.5 us; of up to 128 rows no difference).
    AttentionArgs b = a;
    b.min_steps = two ? 2 : 1;
    // Shares by the requests' rows a key head on average, with room for those
    // above it; T <= R is taken for one token each.  (R counts the page table's
    // rows without tokens too: where most are, one request's 64 tokens are cut
    // into units of 16 rows, each of which reads the keys: 94 us against 30 for
    // three such requests at 4000 positions in a table of 256 rows and of 3.)
    // In one process, replayed from a graph, no shares and P in one bf16 / in two
    // / shares and two: 64 tokens to 8000 89.2 / 121.0 / 88.4 us, 256 to 16000 671
    // / 851 / 642, 15 to 5778 16.0 / 18.5 / 14.7, one at 1000 9.6 / 10.2 / 10.1,
    // 38 trees of 12 with 4 heads a key head 55.2 / 70.3 / 55.8.
    const long long all = (long long)a.T * a.group;
    const bool even = a.R == 1;   // the mean is all there is
    const int shares = all <= (even ? 16 : 12) * (long long)a.R || (a.T <= a.R && a.group <= 16)   ? 4
                       : all <= (even ? 64 : 48) * (long long)a.R || (a.T <= a.R && a.group <= 64) ? 2
                                                                                                   : 1;
    if (a.D == 128)
        return two ? launch_t<128, 2, 1>(b, mk, mv, grid, s) : shares == 4 ? launch_t<128, 1, 4>(b, mk, mv, grid, s)
                   : shares == 2 ? launch_t<128, 1, 2>(b, mk, mv, grid, s) : launch_t<128, 1, 1>(b, mk, mv, grid, s);
    return two ? launch_t<64, 2, 1>(b, mk, mv, grid, s) : shares == 4 ? launch_t<64, 1, 4>(b, mk, mv, grid, s)
               : shares == 2 ? launch_t<64, 1, 2>(b, mk, mv, grid, s) : launch_t<64, 1, 1>(b, mk, mv, grid, s);
}

// A cache in 8 bits, for requests of many rows a key head (attention_q8.cu has
// the others).
cudaError_t launch_attention_tc_q8(const AttentionArgs& a, int sms, cudaStream_t s) {
    const auto enc = tensor_map_encoder();
    if (!enc || sms <= 0) return cudaErrorNotSupported;
    const int grid = sms < kTcRanges ? sms : kTcRanges;
    const long long rows = (long long)a.n_pages * a.kv_heads * a.page_size;
    CUtensorMap mk, mv;
    const int box = a.page_size < kKeys ? a.page_size : kKeys;
    if (!encode_rows(&mk, enc, a.ck, a.D, rows, box) || !encode_rows(&mv, enc, a.cv, a.D, rows, box)) return cudaErrorInvalidValue;
    AttentionArgs b = a;
    // As above: a tree of 64 at 131000 takes 180 us with two row tiles, 253 with one.
    const bool two = (long long)a.T * a.group > 128LL * a.R;
    b.min_steps = two ? 2 : 1;
    if (a.D == 128) return two ? launch_t<128, 2, 1, true>(b, mk, mv, grid, s) : launch_t<128, 1, 1, true>(b, mk, mv, grid, s);
    return two ? launch_t<64, 2, 1, true>(b, mk, mv, grid, s) : launch_t<64, 1, 1, true>(b, mk, mv, grid, s);
}

}  // namespace moe
