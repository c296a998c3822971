// Levelled runs of work items over a kernel's workers, and the join of the pieces
// that they cut.
//
// The items' tiles in item order form one sequence of T units; worker c of n takes
// units T c / n .. T (c + 1) / n, so that every worker has the same work whatever
// the rows' lengths.  Only the first and the last piece of a run can cut an item; a
// cut piece leaves a partial (maximum, sum, weighted values) in slot 0 (first piece)
// or 1 of its worker, which a merge kernel joins.  Every worker works its run out for
// itself (a plan kernel ahead of the tree attention took 8.6 us, and an exchange of
// counters with the last one to arrive joining the pieces 15 to 20).
#pragma once

#include "pkv_device.cuh"

namespace pkv {

// A worker's run, in units: an item counts its tiles and `over` units before them
// (what a piece costs beside its tiles: queries staged, first products, epilogue).
struct Run {
    int32_t pos, end;  // units still ahead, in the sequence
    int32_t lo;        // item u's first unit
    int32_t u;         // the item that holds pos
    int32_t over;
    int32_t k;         // pieces so far
};

// What a merge needs to know of the item that holds the run's last unit.
struct RunEnd {
    int32_t u;       // the item
    int32_t pieces;  // workers that hold a piece of it, if this run has its first tile and not its last (else 0)
    int32_t slot;    // this worker's piece's slot (the others': 0)
    int32_t tiles;   // tiles in the run
};

constexpr int kRunWords = 7;  // of 4 bytes, beside a 64-bit word a warp

// Every thread of the CTA (kThreads of them): worker `c` of `workers`' run over
// `items` items, item u of tiles_of(u, say) tiles, `say` set for one worker's first
// look; `sm`: kThreads / 32 + (kRunWords + 1) / 2 words of 64 bits in shared memory.
// An empty run has pos == end.  The runs have `least` units at least; where they
// have `level` tiles or more, items count `over` units beside their tiles (`level` >
// `over`, so that every run holds a tile).
template <int kThreads, typename Tiles>
__device__ __forceinline__ Run level_run(int32_t items, const Tiles &tiles_of_item, int32_t workers, int32_t c,
                                         int32_t least, int32_t level, int32_t over, int64_t *sm, RunEnd &e)
{
    constexpr int kWarps = kThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // an item's tiles, and (high word) whether it has any
    auto tiles_of = [&](int32_t u, bool say) {
        const int32_t n = u < items ? tiles_of_item(u, say) : 0;
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
    for (int32_t u = threadIdx.x; u < items; u += kThreads) mine += tiles_of(u, c == 0);
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
    Run run{0, 0, 0, 0, tiles / level >= workers ? over : 0, 0};
    const int32_t T = tiles + run.over * used;
    const int32_t n = min(workers, max(1, T / least)), q = T / n, r = T - q * n;
    auto start = [&](int32_t w) { return q * w + r * w / n; };  // T w / n
    if (c < n) {
        run.pos = start(c);
        run.end = start(c + 1);
    }
    auto units = [&](int64_t x) { return static_cast<int32_t>(x) + run.over * static_cast<int32_t>(x >> 32); };
    // items that hold the run's first and last unit: item, first unit, tiles of the
    // sequence before the unit; the same of the last, and its end
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
        // tiles before a unit of this item
        auto before_unit = [&](int32_t at) { return static_cast<int32_t>(lo64) + max(0, at - lo - run.over); };
        if (lo <= run.pos && run.pos < hi) {
            found[0] = base + threadIdx.x;
            found[1] = lo;
            found[2] = before_unit(run.pos);
        }
        if (lo < run.end && run.end <= hi) {
            found[3] = base + threadIdx.x;
            found[4] = lo;
            found[5] = before_unit(run.end);
            found[6] = hi;
        }
        if (!one && units(base64) >= run.end) break;
    }
    __syncthreads();
    e = RunEnd{0, 0, 0, 0};
    if (run.pos < run.end) {
        run.u = found[0];
        run.lo = found[1];
        e.u = found[3];
        e.tiles = found[5] - found[2];
        // the item at the run's end goes on in later workers, and its first tile is here
        const int32_t first = found[4] + run.over, E = found[6];
        if (E > run.end && first >= run.pos && first < run.end) {
            e.pieces = static_cast<int32_t>((static_cast<int64_t>(E) * n + T - 1) / T) - c;  // to the first worker that ends at or past E
            e.slot = e.u != run.u ? 1 : 0;
        }
    }
    return run;
}

// The run's next piece: tiles t0 .. t0 + n - 1 of item u, which has `tiles` (the
// caller looks them up for run.u: tiles_of(run.u)).
struct RunPiece {
    int32_t u, t0, n;
    bool whole;    // all of its tiles
    int32_t slot;  // a cut piece's partial slot
};

// False: item run.u had no tile of the run, and the walk moved on.
__device__ __forceinline__ bool run_step(Run &run, int32_t tiles, RunPiece &pc)
{
    const int32_t first = run.lo + run.over, hi = tiles > 0 ? first + tiles : run.lo;
    const int32_t from = max(run.pos, first), stop = min(hi, run.end);
    pc.u = run.u;
    if (hi <= run.end) {
        ++run.u;
        run.lo = hi;
    }
    run.pos = max(run.pos, stop);
    if (from >= stop) {  // an item without a query, or one whose first tile is the next run's
        if (hi > run.end) run.pos = run.end;
        return false;
    }
    pc.t0 = from - first;
    pc.n = stop - from;
    pc.whole = pc.n == tiles;
    pc.slot = run.k == 0 ? 0 : 1;
    ++run.k;
    return true;
}

// Joins `pieces` partials: 16 values of a row, piece i's at value(i)[e * stride] (e =
// 0 .. 3), its (maximum, sum) stat(i); four pieces are in flight (one after another,
// each read waiting for the last, joined 20 of them in 20 us).  Returns the sum.
template <typename Value, typename Stat>
__device__ __forceinline__ float join_pieces(int32_t pieces, int32_t stride, const Value &value, const Stat &stat,
                                             float4 (&acc)[4])
{
    constexpr int kFly = 4;
    float M = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int32_t i = 0; i < pieces; i += kFly) {
        float4 v[kFly][4];
        float2 ml[kFly];
#pragma unroll
        for (int j = 0; j < kFly; ++j) {
            ml[j] = make_float2(-INFINITY, 0.f);
            if (i + j >= pieces) continue;
            ml[j] = stat(i + j);
            const float4 *o = value(i + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[j][e] = o[e * stride];
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
            if (ml[j].x == -INFINITY) continue;  // a piece without weight may hold anything
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
    return l;
}

// 16 values as bf16, times f
__device__ __forceinline__ void store_bf16x16(__nv_bfloat16 *out, const float4 (&v)[4], float f)
{
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        w[2 * e] = pack_bf16x2(v[e].x * f, v[e].y * f);
        w[2 * e + 1] = pack_bf16x2(v[e].z * f, v[e].w * f);
    }
    reinterpret_cast<uint4 *>(out)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4 *>(out)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

}  // namespace pkv
