// Work items and partials of the attention over latent rows, shared by its kernels
// and the merge.
//
// Item u = (row u / items_per_row, pairs kRows (u % items_per_row) .. of the row's
// (query, head) pairs, query-major).  Its keys are the positions up to its last
// query's, in tiles of kKeys.  The items' tiles are levelled over the workers.
#pragma once

#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "runs.cuh"

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

struct LatentPiece : RunPiece {
    LatentItem it;
};

// Every thread of the CTA: worker `c`'s run, and the record of the item that it
// begins and does not end.
template <int kRows, int kKeys, int kThreads>
__device__ __forceinline__ Run latent_run(const LatentParams &p, int32_t c, int32_t least, int32_t level,
                                          int32_t over, bool record, int64_t *sm)
{
    RunEnd e;
    const Run run = level_run<kThreads>(
        p.batch * p.items_per_row,
        [&](int32_t u, bool say) { return latent_item<kRows, kKeys>(p, u, say && record).tiles; },
        p.workers, c, least, level, over, sm, e);
    if (record && threadIdx.x == 96) {  // (of a warp that does not lead)
        LatentRecord rec{};
        if (e.pieces > 0) {
            const LatentItem it = latent_item<kRows, kKeys>(p, e.u);
            rec.pieces = e.pieces;
            rec.slot = e.slot;
            rec.pairs = it.n;
            rec.row = static_cast<int64_t>(it.q0) * p.heads + it.p0;
        }
        static_cast<LatentRecord *>(p.rec)[c] = rec;
    }
    return run;
}

// Next piece of the run (false at its end).
template <int kRows, int kKeys>
__device__ __forceinline__ bool latent_next(const LatentParams &p, Run &run, LatentPiece &pc)
{
    while (run.pos < run.end) {
        pc.it = latent_item<kRows, kKeys>(p, run.u);
        if (run_step(run, pc.it.tiles, pc)) return true;
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
// thread has 16 dims of a pair; nothing but the record comes before the partials.
constexpr int kLatMergeThreads = 256;

template <typename T, int kRows>
__global__ void __launch_bounds__(kLatMergeThreads) latent_merge_kernel(const LatentParams p, const int32_t pairs)
{
    pdl_wait();  // the records and partials come from the kernel just before
    pdl_trigger();
    const int32_t c = blockIdx.x, idx = blockIdx.y * kLatMergeThreads + threadIdx.x;
    const LatentRecord rec = static_cast<const LatentRecord *>(p.rec)[c];
    const int32_t pair = idx % pairs, d4 = idx / pairs * 4;  // pairs: of an item, at most
    if (pair >= rec.pairs || d4 * 4 >= p.latent) return;     // (no item: no pairs)
    const auto slot = [&](int32_t i) { return i == 0 ? rec.slot : 0; };
    float4 acc[4];
    const float l = join_pieces(
        rec.pieces, kRows,
        [&](int32_t i) -> const float4 * { return latent_part_o<kRows>(p, c + i, slot(i)) + d4 * kRows + pair; },
        [&](int32_t i) { return latent_part_ml<kRows>(p, c + i, slot(i))[pair]; }, acc);
    const float inv = l != 0.f ? 1.f / l : 0.f;  // (NaN stays NaN)
    T *out = static_cast<T *>(p.out) + (rec.row + pair) * p.latent + d4 * 4;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            reinterpret_cast<float4 *>(out)[e] =
                make_float4(acc[e].x * inv, acc[e].y * inv, acc[e].z * inv, acc[e].w * inv);
    } else {
        store_bf16x16(out, acc, inv);
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
