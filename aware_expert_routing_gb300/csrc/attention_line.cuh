// attention_line.cuh -- how the attention kernels share out their work, and
// the kernel that joins what the shares cut.
//
// A unit of work is (request, key head, tile of query rows).  Its key tiles,
// one step each, and kUnitCost steps for what a unit costs besides (queries,
// first scores, result; some before the tiles, some after them, so that a cut
// close to a unit's end moves to it), follow one another in one line with
// those of all other units, and the line is cut into equal stretches
// ("ranges"), one per CTA.  So ragged lengths balance, one long request is spread over all CTAs,
// and the lengths are read on the device.  A unit that a cut goes through
// leaves partial results (AttentionLayout) in each of its ranges.
#pragma once

#include "attention.cuh"

namespace moe {

namespace {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Of a unit's cost, the steps before its key tiles (all before: 27.5 against
// 27.1 us for 16 trees of 16 to 4000).
__host__ __device__ constexpr int steps_before(int cost) { return cost - cost * 2 / 5; }

// The line of `total` steps in `ranges` equal stretches (the first ones a
// step longer where it does not divide).
struct Line {
    int q, rem;
    __device__ __forceinline__ Line(int total, int ranges) {
        q = ranges > 0 ? total / ranges : 0;
        rem = total - q * ranges;
    }
    __device__ __forceinline__ Line(const RangeStart& s) : q(s.line_q), rem(s.line_rem) {}
    __device__ __forceinline__ int start(int c) const { return q * c + min(c, rem); }
    __device__ __forceinline__ int range_of(int x) const {   // q > 0
        const int cut = rem * (q + 1);
        return x < cut ? x / (q + 1) : rem + (x - cut) / q;
    }
};

struct Request {
    int t0, n, ctx, nrt, nkt;   // n 0: nothing to do
};

template <int kRows, int kKeys>
__device__ __forceinline__ Request load_request(const AttentionArgs& a, int r, bool& bad) {
    Request q;
    q.t0 = a.q_offsets[r];
    const int t1 = a.q_offsets[r + 1];
    q.ctx = a.ctx_len[r];
    q.n = t1 - q.t0;
    bad = q.t0 < 0 || t1 > a.T || t1 < q.t0 ||
          (q.n > 0 && (q.ctx < 0 || (long long)q.ctx + q.n > (long long)a.max_pages * a.page_size));
    if (bad) q.n = 0;
    q.nrt = (int)(((uint32_t)(q.n * a.group) + kRows - 1) / kRows);
    q.nkt = q.n > 0 ? (q.ctx + q.n + kKeys - 1) / kKeys : 0;
    return q;
}

// Where a CTA's range starts (request, unit, steps into the unit) and how long
// it is; in shared memory, written by find_start.
struct LineStart {
    uint2 scan[16];
    int r, t0, n, ctx, nrt, nkt, h, rt, off, left;
};

// A CTA's stretch of the line, one unit (or its part) at a time.
template <int kRows, int kKeys, int kUnitCost>
struct LineWalk {
    Request q;
    int r, h, rt, kt, nk;       // this part: key tiles kt .. kt + nk - 1
    int left;                   // steps after this part
    bool first;                 // the part of the unit in which the stretch starts

    // the part of the current unit from its step `off` on; false: it holds no key tile
    __device__ __forceinline__ bool part(int off) {
        const int take = min(q.nkt + kUnitCost - off, left);
        left -= take;
        constexpr int kBefore = steps_before(kUnitCost);
        kt = min(max(0, off - kBefore), q.nkt);
        nk = min(max(0, off + take - kBefore), q.nkt) - kt;
        return nk > 0;
    }
    __device__ __forceinline__ bool start(const AttentionArgs& a, const LineStart& S) {
        r = S.r;
        q.t0 = S.t0; q.n = S.n; q.ctx = S.ctx; q.nrt = S.nrt; q.nkt = S.nkt;
        h = S.h;
        rt = S.rt;
        left = S.left;
        first = true;
        return left > 0 && (part(S.off) || next(a));
    }
    __device__ __forceinline__ bool next(const AttentionArgs& a) {
        while (left > 0) {
            first = false;
            if (++rt >= q.nrt) {
                rt = 0;
                if (++h >= a.kv_heads) {
                    h = 0;
                    do {
                        if (++r >= a.R) return false;   // not reached: the line ends with a request that has work
                        bool bad;
                        q = load_request<kRows, kKeys>(a, r, bad);
                    } while (q.n == 0);
                }
            }
            if (part(0)) return true;
        }
        return false;
    }
    // query rows of the unit
    __device__ __forceinline__ int rows(const AttentionArgs& a) const { return min(kRows, q.n * a.group - rt * kRows); }
};

// Brings the lengths and the page table towards L2, each CTA a part of them,
// while the kernel before this one ends: they are read one after the other
// once it has.  (A prefetch reads nothing that can go stale: L2 is where the
// other kernel's writes go.)
__device__ __forceinline__ void prefetch_tables(const AttentionArgs& a) {
    const int lane = threadIdx.x & 31;
    auto line = [](const void* p, long long bytes, long long l) {
        if (l * 128 < bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p) + l * 128));
    };
    if (threadIdx.x < 32) {
        line(a.page_table, (long long)a.R * a.max_pages * 4, (long long)blockIdx.x * 32 + lane);
        if (blockIdx.x == 0) {
            line(a.q_offsets, (a.R + 1) * 4LL, lane);
            line(a.ctx_len, a.R * 4LL, lane);
        }
    }
}

// Finds this CTA's range.  All kThreads threads; each adds up a few consecutive
// requests, and the one whose requests hold the range's start writes it down.
// The caller synchronises before S is read.
template <int kRows, int kKeys, int kUnitCost, int kThreads>
__device__ __forceinline__ void find_start(const AttentionArgs& a, LineStart& S) {
    const int per = (a.R + kThreads - 1) / kThreads;
    const int r0 = min(a.R, (int)threadIdx.x * per), r1 = min(a.R, r0 + per);
    long long work = 0;
    Request q0 = {};   // of the first of them
    for (int r = r0; r < r1; ++r) {
        bool bad;
        const Request q = load_request<kRows, kKeys>(a, r, bad);
        if (r == r0) q0 = q;
        if (bad && blockIdx.x == 0) raise_flag(a.flags, kFlagBadIndex);
        work += (long long)q.nrt * (q.nkt + kUnitCost) * a.kv_heads;
    }
    // Places on the line take 31 bits, and so do their sums, modulo 2^32, if the
    // total does: row tiles multiply key tiles, so one long request can have most
    // of the line.  Whether it does is told by a second sum, of 2^16 steps each
    // (rounded down, kThreads times): a longer line (the limit stated at
    // moe_tree_attention) gives no work.
    uint32_t inc = (uint32_t)work;
    const uint32_t thick = __reduce_add_sync(0xffffffffu, (uint32_t)min(work >> 16, 1LL << 20));
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, inc, off);
        if ((int)(threadIdx.x & 31) >= off) inc += t;
    }
    if ((threadIdx.x & 31) == 31) S.scan[threadIdx.x >> 5] = make_uint2(inc, thick);
    __syncthreads();
    uint32_t first = inc - (uint32_t)work, all = 0, all_thick = kThreads;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const uint2 t = S.scan[w];
        if (w < (int)(threadIdx.x >> 5)) first += t.x;
        all += t.x;
        all_thick += t.y;
    }
    const bool over = all_thick > 0x7fff;
    if (over && threadIdx.x == 0 && blockIdx.x == 0) raise_flag(a.flags, kFlagBadIndex);
    const int before = (int)first, total = over ? 0 : (int)all, sum = (int)(uint32_t)work;
    // (no range of a few steps where that makes many parts of many rows)
    const int ranges = min((int)gridDim.x, (total + a.min_steps - 1) / a.min_steps);
    const Line line(total, ranges);
    const int b = line.start(blockIdx.x), e = line.start(blockIdx.x + 1);
    if (threadIdx.x == 0) {
        S.left = (int)blockIdx.x < ranges ? e - b : 0;
        if ((int)blockIdx.x >= ranges) a.plan[blockIdx.x].nkt = 0;   // nothing to join
    }
    if ((int)blockIdx.x < ranges && b >= before && b < before + sum) {   // one thread
        int at = before, r = r0;
        Request q = q0;
        for (;;) {
            const int w = q.nrt * (q.nkt + kUnitCost) * a.kv_heads;
            if (b < at + w) break;
            at += w;
            bool bad;
            q = load_request<kRows, kKeys>(a, ++r, bad);
        }
        const int u = (b - at) / (q.nkt + kUnitCost), off = b - at - u * (q.nkt + kUnitCost);
        S.r = r;
        S.t0 = q.t0; S.n = q.n; S.ctx = q.ctx; S.nrt = q.nrt; S.nkt = q.nkt;
        S.h = u / q.nrt;
        S.rt = u - S.h * q.nrt;
        S.off = off;
        RangeStart rec;
        rec.t0 = q.t0;
        rec.n = q.n;
        rec.h = S.h;
        rec.rt = S.rt;
        rec.off = off;
        rec.nkt = q.nkt;
        rec.line_q = line.q;
        rec.line_rem = line.rem;
        a.plan[blockIdx.x] = rec;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.page_table + (size_t)r * a.max_pages + min(max(0, off - steps_before(kUnitCost)), q.nkt - 1) * kKeys / a.page_size));
    }
}

// Four components of a result: o / l, or zeros where nothing was seen.
__device__ __forceinline__ void store_row(float* dst, float4 o, float l) {
    const float inv = 1.f / l;
    *reinterpret_cast<float4*>(dst) = l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                               : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}
__device__ __forceinline__ void store_row(__nv_bfloat16* dst, float4 o, float l) {
    const float inv = 1.f / l;
    const __nv_bfloat162 p0 = __floats2bfloat162_rn(l == 0.f ? 0.f : o.x * inv, l == 0.f ? 0.f : o.y * inv);
    const __nv_bfloat162 p1 = __floats2bfloat162_rn(l == 0.f ? 0.f : o.z * inv, l == 0.f ? 0.f : o.w * inv);
    *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&p0), *reinterpret_cast<const uint32_t*>(&p1));
}

// Joins the parts of the units that the ranges' ends cut: block x takes the
// unit that range x + 1 starts inside of, unless an earlier range does too.
// A warp holds four rows (lane: row lane % 4, components 4 (lane / 4) and on,
// in steps of 32), and kJoinSplit warps share the parts of the same rows, so
// that few parts take one round of loads; their sums meet in shared memory,
// always in the same order.  Eight warps a block: all on four rows for units of
// few rows, where latency counts, else four on each four of eight.  (16 rows a
// block: 35.1 against 32.7 us for 16 trees of 16 to 4000, fewer of the larger
// blocks are resident.)  kSteps: ceil(D / 32).
constexpr int kJoinWarps = 8;

template <typename T, int kSteps, int kUnitCost, int kJoinSplit>
__global__ void __launch_bounds__(kJoinWarps * 32) attention_join_kernel(const AttentionArgs a, int unit_rows) {
    constexpr int kJoinRows = 4 * kJoinWarps / kJoinSplit;
    const int D = a.D;
    __shared__ float4 so[kJoinWarps][kSteps][32];
    __shared__ float sl[kJoinWarps][32];
    grid_dependency_wait();
    const int c = blockIdx.x + 1;
    const RangeStart rec = a.plan[c];
    if (rec.nkt == 0) return;   // range c is empty
    const Line line(rec);
    auto start = [&](int x) { return line.start(x); };
    // the unit's stretch of the line: its start, its first key tile, its end
    const int u0 = start(c) - rec.off, k0 = u0 + steps_before(kUnitCost), u1 = k0 + rec.nkt;
    if (start(c) <= k0 || start(c) >= u1 || start(c - 1) > k0) return;
    const int group = a.group;
    const int nrows = min(unit_rows, rec.n * group - rec.rt * unit_rows);
    if ((int)blockIdx.y * kJoinRows >= nrows) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, split = warp % kJoinSplit;
    const int row = blockIdx.y * kJoinRows + warp / kJoinSplit * 4 + (lane & 3), ch = lane >> 2;
    const bool valid = row < nrows;
    const int first = c - 1, last = line.range_of(u1 - 1);    // ranges with a part
    const int slot0 = 2 * first + (start(first) >= u0 ? 0 : 1);
    auto slot = [&](int x) { return (size_t)(x == first ? slot0 : 2 * x) * a.rows; };
    // the first part's sums are on their way while the maxima are read
    auto part = [&](int x) {
        return reinterpret_cast<const float4*>(a.o) + (slot(x) + (row & ~31)) * (D / 4) + ch * 32 + (row & 31);
    };
    float4 v[kSteps];
    if (valid && first + split <= last)
#pragma unroll
        for (int y = 0; y < kSteps; ++y)
            if (y * 8 + ch < D / 4) v[y] = part(first + split)[y * 256];
    float mx = -INFINITY;
    if (valid)
        for (int x = first + ch; x <= last; x += 8) mx = fmaxf(mx, a.ml[slot(x) + row].x);
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    float4 o[kSteps];
    float l = 0.f;
#pragma unroll
    for (int y = 0; y < kSteps; ++y) o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (valid) {
#pragma unroll 2
        for (int x = first + split; x <= last; x += kJoinSplit) {
            const float2 ml = a.ml[slot(x) + row];
            const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mx);
            l = fmaf(f, ml.y, l);
#pragma unroll
            for (int y = 0; y < kSteps; ++y) {
                if (y * 8 + ch >= D / 4) continue;
                o[y].x = fmaf(f, v[y].x, o[y].x);
                o[y].y = fmaf(f, v[y].y, o[y].y);
                o[y].z = fmaf(f, v[y].z, o[y].z);
                o[y].w = fmaf(f, v[y].w, o[y].w);
                if (x + kJoinSplit <= last) v[y] = part(x + kJoinSplit)[y * 256];
            }
        }
    }
#pragma unroll
    for (int y = 0; y < kSteps; ++y) so[warp][y][lane] = o[y];
    sl[warp][lane] = l;
    __syncthreads();
    if (split != 0 || !valid) return;
#pragma unroll
    for (int k = 1; k < kJoinSplit; ++k) {
        l += sl[warp + k][lane];
#pragma unroll
        for (int y = 0; y < kSteps; ++y) {
            const float4 v = so[warp + k][y][lane];
            o[y].x += v.x;
            o[y].y += v.y;
            o[y].z += v.z;
            o[y].w += v.w;
        }
    }
    const int gr = rec.rt * unit_rows + row;
    const size_t orow = (size_t)(rec.t0 + gr / group) * a.heads + rec.h * group + gr % group;
#pragma unroll
    for (int y = 0; y < kSteps; ++y)
        if (y * 8 + ch < D / 4) store_row(static_cast<T*>(a.out) + orow * D + y * 32 + ch * 4, o[y], l);
    if (a.lse && ch == 0) a.lse[orow] = l == 0.f ? -INFINITY : (mx + log2f(l)) * 0.6931471805599453f;
}

// Launches the join for a kernel of `ranges` ranges and units of up to
// unit_rows rows (cfg: stream and attributes).
template <typename T, int kSteps, int kUnitCost>
cudaError_t launch_join(const AttentionArgs& a, int ranges, int unit_rows, cudaLaunchConfig_t cfg) {
    const int rows = a.rows < unit_rows ? a.rows : unit_rows;
    const bool few = rows <= 32;
    cfg.gridDim = dim3(ranges - 1, (rows + (few ? 3 : 7)) / (few ? 4 : 8));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.dynamicSmemBytes = 0;
    return few ? cudaLaunchKernelEx(&cfg, attention_join_kernel<T, kSteps, kUnitCost, 8>, a, unit_rows)
               : cudaLaunchKernelEx(&cfg, attention_join_kernel<T, kSteps, kUnitCost, 4>, a, unit_rows);
}

}  // namespace

}  // namespace moe
