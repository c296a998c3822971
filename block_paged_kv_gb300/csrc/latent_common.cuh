// Work items, runs and partials of the attention over latent rows, shared by its
// kernels and the merge.
//
// Item u = (row u / items_per_row, pairs kRows (u % items_per_row) .. of the row's
// (query, head) pairs, query-major).  Its keys are the positions up to its last
// query's, in tiles of kKeys.  The items' tiles in item order form one sequence;
// worker c of n takes units T c / n .. T (c + 1) / n of the T there are, so that
// every worker has the same work whatever the rows' lengths.  Only the first and
// the last piece of a run can cut an item; a cut piece leaves a partial (maximum,
// sum, weighted values) in slot 0 (first piece) or 1 of its worker, which the
// merge kernel joins.
#pragma once

#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

struct LatentItem {
    int32_t r;      // row
    int32_t first;  // position of the row's first query
    int32_t q0;     // its index in q
    int32_t p0;     // the item's first pair of the row's
    int32_t n;      // its pairs (0: the item is empty)
    int32_t hi;     // keys 0 .. hi - 1
    int32_t tiles;
};

template <int kRows, int kKeys>
__device__ __forceinline__ LatentItem latent_item(const LatentParams &p, int32_t u, bool say = false)
{
    LatentItem it;
    it.r = u / p.items_per_row;
    it.p0 = (u - it.r * p.items_per_row) * kRows;
    say = say && it.p0 == 0;
    int32_t L = __ldg(p.seq_lens + it.r), C = 1;
    it.q0 = it.r;
    if (L < 0 || L > p.max_len) {
        if (say) report(p.status, PKV_DEV_BAD_LEN);
        L = L < 0 ? 0 : p.max_len;
    }
    if (p.cu_q_lens != nullptr) {
        const int32_t c0 = __ldg(p.cu_q_lens + it.r), c1 = __ldg(p.cu_q_lens + it.r + 1);
        C = c1 - c0;
        const bool outside = c0 < 0 || C < 0 || c1 > p.num_queries;
        if (outside || C > p.max_q || C > L) {
            if (say) report(p.status, PKV_DEV_BAD_LEN);
            C = outside ? 0 : min(min(C, p.max_q), L);
        }
        it.q0 = c0;
    }
    it.first = L - C;
    it.n = max(0, min(kRows, C * p.heads - it.p0));
    // a decode row of length 0 has a query and no key: one tile, fully masked
    it.hi = it.n > 0 ? max(0, it.first + (it.p0 + it.n - 1) / p.heads + 1) : 0;
    it.tiles = it.n > 0 ? max(1, (it.hi + kKeys - 1) / kKeys) : 0;
    return it;
}

// Keys that a pair's query attends: positions below hi, and of those from `first`
// on (drafts) the mask's alone (all bits set: a chain).
struct LatentRange {
    int32_t hi;
    uint64_t mask;
};
__device__ __forceinline__ LatentRange latent_range(const LatentParams &p, const LatentItem &it, int32_t pair)
{
    LatentRange rg{0, ~0ull};
    if (pair >= it.n) return rg;
    const int32_t i = (it.p0 + pair) / p.heads;  // the row's query
    rg.hi = max(0, it.first + i + 1);
    if (p.tree != nullptr) rg.mask = tree_mask(p.tree, it.q0 + i, i);
    return rg;
}

// What the merge needs of an item that a worker's run begins and does not end.
struct alignas(8) LatentRecord {
    int64_t row;     // its first pair's row of out
    int32_t pieces;  // workers that hold a piece of it, this one first (0: there is no such item)
    int32_t slot;    // this worker's piece's partial slot (the others': 0)
    int32_t pairs;
    int32_t pad;
};
static_assert(sizeof(LatentRecord) == kLatentRecordBytes, "the workspace holds one per worker");

// A worker's run, in units: an item counts its tiles and `over` units before them
// (what a piece costs beside its tiles: queries staged, first products, epilogue).
struct LatentRun {
    int32_t pos, end;  // units still ahead, in the sequence
    int32_t lo;        // item u's first unit
    int32_t u;         // the item that holds pos
    int32_t over;
    int32_t k;         // pieces so far
};
struct LatentPiece {
    LatentItem it;
    int32_t u;
    int32_t t0, n;     // tiles t0 .. t0 + n - 1 of the item
    bool whole;        // all of them
    int32_t slot;      // a cut piece's partial slot
};

// Every thread of the CTA (kThreads of them, at least 128): worker `c`'s run, and the
// record of the item that it begins and does not end; `sm`: kThreads / 32 + 4 words
// of shared memory (64 bits).  An empty run has pos == end.  The runs have `least`
// units at least; where they have `level` tiles or more, items count `over` units
// beside their tiles (`level` > `over`, so that every run holds a tile).
template <int kRows, int kKeys, int kThreads>
__device__ __forceinline__ LatentRun latent_run(const LatentParams &p, int32_t c, int32_t least, int32_t level,
                                                int32_t over, bool record, int64_t *sm)
{
    constexpr int kWarps = kThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t items = p.batch * p.items_per_row;
    // an item's tiles, and (high word) whether it has any
    auto tiles_of = [&](int32_t u, bool say) {
        const int32_t n = u < items ? latent_item<kRows, kKeys>(p, u, say).tiles : 0;
        return static_cast<int64_t>(n) | (n > 0 ? 1ll << 32 : 0ll);
    };
    auto scan = [&](int64_t x) {  // inclusive, over the warp
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        return x;
    };
    // tiles in all; with one pass of items, they are looked up and scanned once
    const bool one = items <= kThreads;
    int64_t mine = 0;
    for (int32_t u = threadIdx.x; u < items; u += kThreads) mine += tiles_of(u, c == 0 && record);
    const int64_t inc0 = scan(mine);
    if (lane == 31) sm[warp] = inc0;
    __syncthreads();
    int64_t all = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sm[w];
        all += sm[w];
    }
    const int32_t tiles = static_cast<int32_t>(all), used = static_cast<int32_t>(all >> 32);
    LatentRun run{0, 0, 0, 0, tiles / level >= p.workers ? over : 0, 0};
    const int32_t T = tiles + run.over * used;
    const int32_t n = min(p.workers, max(1, T / least)), q = T / n, r = T - q * n;
    auto start = [&](int32_t w) { return q * w + r * w / n; };  // T w / n
    if (c < n) {
        run.pos = start(c);
        run.end = start(c + 1);
    }
    auto units = [&](int64_t x) { return static_cast<int32_t>(x) + run.over * static_cast<int32_t>(x >> 32); };
    // items that hold the run's first and last unit: item, first unit; item, first unit, end
    int32_t *found = reinterpret_cast<int32_t *>(sm + kWarps);
    int64_t lo64 = before + inc0 - mine, x64 = mine, base64 = 0;
    for (int32_t base = 0; base < items && run.pos < run.end; base += kThreads) {
        if (!one) {
            x64 = tiles_of(base + threadIdx.x, false);
            const int64_t inc = scan(x64);
            __syncthreads();
            if (lane == 31) sm[warp] = inc;
            __syncthreads();
            lo64 = base64 + inc - x64;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) lo64 += sm[w];
                base64 += sm[w];
            }
        }
        const int32_t lo = units(lo64), hi = units(lo64 + x64);
        if (lo <= run.pos && run.pos < hi) {
            found[0] = base + threadIdx.x;
            found[1] = lo;
        }
        if (lo < run.end && run.end <= hi) {
            found[2] = base + threadIdx.x;
            found[3] = lo;
            found[4] = hi;
        }
        if (!one && units(base64) >= run.end) break;
    }
    __syncthreads();
    if (run.pos < run.end) {
        run.u = found[0];
        run.lo = found[1];
    }
    if (record && threadIdx.x == 96) {  // (of a warp that does not lead)
        // the item at the run's end goes on in later workers, and its first tile is here
        LatentRecord rec{};
        if (run.pos < run.end) {
            const int32_t first = found[3] + run.over, E = found[4];
            if (E > run.end && first >= run.pos && first < run.end) {
                const LatentItem it = latent_item<kRows, kKeys>(p, found[2]);
                rec.pieces = static_cast<int32_t>((static_cast<int64_t>(E) * n + T - 1) / T) - c;  // to the first worker that ends at or past E
                rec.slot = found[2] != found[0] ? 1 : 0;
                rec.pairs = it.n;
                rec.row = static_cast<int64_t>(it.q0) * p.heads + it.p0;
            }
        }
        static_cast<LatentRecord *>(p.rec)[c] = rec;
    }
    return run;
}

// Next piece of the run (false at its end).
template <int kRows, int kKeys>
__device__ __forceinline__ bool latent_next(const LatentParams &p, LatentRun &run, LatentPiece &pc)
{
    while (run.pos < run.end) {
        pc.it = latent_item<kRows, kKeys>(p, run.u);
        const int32_t first = run.lo + run.over, hi = pc.it.tiles > 0 ? first + pc.it.tiles : run.lo;
        const int32_t from = max(run.pos, first), stop = min(hi, run.end);
        pc.u = run.u;
        if (hi <= run.end) {
            ++run.u;
            run.lo = hi;
        }
        run.pos = max(run.pos, stop);
        if (from >= stop) {  // an item without a query, or one whose first tile is the next run's
            if (hi > run.end) run.pos = run.end;
            continue;
        }
        pc.t0 = from - first;
        pc.n = stop - from;
        pc.whole = pc.n == pc.it.tiles;
        pc.slot = run.k == 0 ? 0 : 1;
        ++run.k;
        return true;
    }
    return false;
}

// Partials: value quad d4 of pair i of a piece, and its (maximum, sum).
template <int kRows>
__device__ __forceinline__ float4 *latent_part_o(const LatentParams &p, int32_t worker, int32_t slot)
{
    return reinterpret_cast<float4 *>(p.ws_o) + (static_cast<int64_t>(worker) * 2 + slot) * (p.latent / 4) * kRows;
}
template <int kRows>
__device__ __forceinline__ float2 *latent_part_ml(const LatentParams &p, int32_t worker, int32_t slot)
{
    return reinterpret_cast<float2 *>(p.ws_ml) + (static_cast<int64_t>(worker) * 2 + slot) * kRows;
}

__device__ __forceinline__ int64_t latent_out_row(const LatentParams &p, const LatentItem &it, int32_t pair)
{
    return (static_cast<int64_t>(it.q0) * p.heads + it.p0 + pair) * p.latent;
}

// Joins the pieces of an item cut between workers: worker x's (CTAs (x, ..)).  A
// thread has 16 dims of a pair; nothing but the record comes before the partials, of
// which it has four in flight (one piece after another, each read waiting for the
// last, joined 20 pieces in 20 us).
constexpr int kLatMergeThreads = 256;

template <typename T, int kRows>
__global__ void __launch_bounds__(kLatMergeThreads) latent_merge_kernel(const LatentParams p, const int32_t pairs)
{
    constexpr int kFly = 4;
    pdl_wait();  // the records and partials come from the kernel just before
    pdl_trigger();
    const int32_t c = blockIdx.x, idx = blockIdx.y * kLatMergeThreads + threadIdx.x;
    const LatentRecord rec = static_cast<const LatentRecord *>(p.rec)[c];
    const int32_t pair = idx % pairs, d4 = idx / pairs * 4;  // pairs: of an item, at most
    if (pair >= rec.pairs || d4 * 4 >= p.latent) return;     // (no item: no pairs)
    float M = -INFINITY, l = 0.f;
    float4 acc[4] = {};
    for (int32_t i = 0; i < rec.pieces; i += kFly) {
        float4 v[kFly][4];
        float2 ml[kFly];
#pragma unroll
        for (int j = 0; j < kFly; ++j) {
            ml[j] = make_float2(-INFINITY, 0.f);
            if (i + j >= rec.pieces) continue;
            const int32_t w = c + i + j, slot = i + j == 0 ? rec.slot : 0;
            ml[j] = latent_part_ml<kRows>(p, w, slot)[pair];
            const float4 *o = latent_part_o<kRows>(p, w, slot) + d4 * kRows + pair;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[j][e] = o[e * kRows];
        }
        float mn = M;
#pragma unroll
        for (int j = 0; j < kFly; ++j) mn = fmaxf(mn, ml[j].x);
        if (mn == -INFINITY) continue;  // nothing attended so far
        const float f0 = fast_exp2(M - mn);
        M = mn;
        l *= f0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            acc[e].x *= f0;
            acc[e].y *= f0;
            acc[e].z *= f0;
            acc[e].w *= f0;
        }
#pragma unroll
        for (int j = 0; j < kFly; ++j) {
            if (i + j >= rec.pieces) continue;
            const float f = fast_exp2(ml[j].x - M);
            l = fmaf(f, ml[j].y, l);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[e].x = fmaf(f, v[j][e].x, acc[e].x);
                acc[e].y = fmaf(f, v[j][e].y, acc[e].y);
                acc[e].z = fmaf(f, v[j][e].z, acc[e].z);
                acc[e].w = fmaf(f, v[j][e].w, acc[e].w);
            }
        }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;  // (NaN stays NaN)
    T *out = static_cast<T *>(p.out) + (rec.row + pair) * p.latent + d4 * 4;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            reinterpret_cast<float4 *>(out)[e] =
                make_float4(acc[e].x * inv, acc[e].y * inv, acc[e].z * inv, acc[e].w * inv);
    } else {
        uint32_t v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = pack_bf16x2(acc[e].x * inv, acc[e].y * inv);
            v[2 * e + 1] = pack_bf16x2(acc[e].z * inv, acc[e].w * inv);
        }
        reinterpret_cast<uint4 *>(out)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(out)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

template <typename T, int kRows>
static cudaError_t launch_latent_merge(const LatentParams &p, cudaStream_t stream)
{
    const int32_t pairs = static_cast<int32_t>(std::min<int64_t>(kRows, static_cast<int64_t>(p.max_q) * p.heads));
    const int32_t threads = pairs * (p.latent / 16);
    return launch_pdl(latent_merge_kernel<T, kRows>,
                      dim3(static_cast<unsigned>(p.workers), static_cast<unsigned>((threads + kLatMergeThreads - 1) / kLatMergeThreads)),
                      dim3(kLatMergeThreads), 0, stream, p, pairs);
}

}  // namespace pkv
