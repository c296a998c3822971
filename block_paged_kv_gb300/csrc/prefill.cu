// Chunked prefill against a paged prefix ("perf.md", gather_kv_for_prefill_chunk:
// a prefill chunk attends its cached prefix through the pages; "paged-cache.md":
// chunk boundaries change the reduction order, not the result).  Query i of a
// row's chunk sits at absolute position p = L - C + i and attends positions
// max(0, p - W + 1) .. p (the whole prefix and the chunk causally for W = 0), and
// with sinks the first S positions beside them.
//
// Tensor-core kernel (bf16 pools; FP8 pools the same kernel with widening),
// work item = (row, kv head, two tiles of 128/G queries).  A tile's 128 M-rows
// are (query, head) pairs of all G q heads of the kv head, and both tiles
// share every K/V tile, so K/V are loaded once per 256 query rows.  QK^T and
// PV are dense contractions and run on the 5th-generation tensor cores:
//   warps 0/2 producers: K and V tiles of 64 keys (4 paged blocks) into
//             4-stage rings (bf16: two 64-dim TMA boxes a block; FP8: bulk
//             copies of the E4M3 blocks into a two-deep staging buffer); a K
//             stage is freed once both S products are computed and the key
//             masks read, a V stage once both P.V products are;
//   warps 1/3 issue tile A's / tile B's tcgen05.mma from one elected lane:
//             S = Q K^T into one of the tile's two S buffers in tensor memory
//             (both operands K-major, 128-byte swizzle), O += P V with P read
//             from tensor memory; per K/V tile j, once K(j+2) has landed and
//             P(j) is stored: P(j).V, then S(j+2) into the buffer that product
//             reads.  Warp 1 also allocates the 512 tensor-memory columns;
//   warps 4-7 / 8-11  softmax of tile A / tile B, concurrently, one M-row per
//             thread: S from tensor memory, causal / window / range mask,
//             running max kept within 2^8 of the true maximum (O is rescaled
//             in tensor memory only when it moves further), P written back
//             over S (bf16: hi + lo terms, 8 columns each per 16 keys, so
//             that P.V carries P to ~2^-17 relative; FP8 pools: one f16
//             term), and the epilogue O / l.  FP8 pools: tile A's warps also
//             widen the staged K tiles to f16, tile B's the V tiles.
// Schedules: one CTA per item while the items fit one wave; more items than
// SMs: one persistent CTA per SM (a whole item, then a run of the remaining
// items' tiles that levels the CTAs, cut pieces merged in the kernel).  A short chunk
// fills tile A only (tile B's warps stay idle, warps whose rows hold no query
// skip the softmax work); on a grid too small for the GPU its key range is
// cut into runs whose fp32 partials prefill_merge_kernel merges.  Drafted trees: a
// levelled run of the items' tiles a CTA, the pieces joined by prefill_tree_merge_kernel.
// f32 kernel: CUDA cores, the same work split with 16 (query, head) pairs per
// CTA, for the fp32 pools.
#include <algorithm>

#include "decode_common.cuh"
#include "runs.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace pf {
constexpr int kD = 128;
constexpr int kRows = 128;                // M of one query tile
constexpr int kQTiles = 2;                // query tiles per CTA, sharing every K/V tile
constexpr int kKeys = 64;                 // keys per K/V tile (4 blocks of 16)
constexpr int kBlocks = kKeys / 16;
constexpr int kQBytes = kRows * 2 * 128;  // one query tile: two 64-dim swizzled regions
constexpr int kKVRegion = kKeys * 128;    // 8 KiB: one 64-dim half of a K/V tile
constexpr int kTileBytes = 2 * kKVRegion; // 16 KiB: a K or a V tile
constexpr int kQOff = 0;
// FP8 pools: the producers stage each tile's E4M3 bytes (4 blocks x 2 KiB)
// by bulk copy, two tiles deep, and widen them into the ring
constexpr int kF8BlockBytes = 16 * kD;                 // one (block, kv head) E4M3 tile
constexpr int kF8StageTile = kBlocks * kF8BlockBytes;  // 8 KiB
constexpr int kSoftmaxWarps = 8;  // 4-7 softmax of query tile A, 8-11 of tile B
constexpr int kSegBytes = 160;    // a softmax warp's segment walk, current and next segment
// kAlt (both warpgroups on one query tile, alternate key tiles): one query tile, and
// for bf16 pools rings of 6 in its place (32 rows of 1024 to 8192 keys x 16 drafts, 32/8
// heads: 112.4 us with 4, 111.2 with 6)
template <bool kF8, bool kAlt = false>
struct Layout {
    static constexpr int kStages = kAlt && !kF8 ? 6 : 4;  // K ring and V ring depth
    static constexpr int kKOff = kQOff + (kAlt ? 1 : kQTiles) * kQBytes;
    static constexpr int kVOff = kKOff + kStages * kTileBytes;
    static constexpr int kStagingOff = kVOff + kStages * kTileBytes;
    static constexpr int kStagingBytes = kF8 ? 2 * 2 * kF8StageTile : 0;  // K and V, 2 deep
    static constexpr int kBarOff = kStagingOff + kStagingBytes;
    // barriers: k_full[4], k_empty[4], v_full[4], v_empty[4], s_full[tile][buf],
    // p_full[tile][buf], pv_done[tile], mma_drain[tile], q_full[tile],
    // o_done[tile], sums (of two, for the alignment), FP8: staged[K/V][2],
    // stg_free[K/V][2]
    static constexpr int kNumBars = 4 * kStages + 4 + 4 + 2 + 2 + 2 + 2 + 2 + (kF8 ? 8 : 0);
    // kmask[kStages], FP8: smask[K/V][2] (blocks loaded of each staging buffer)
    static constexpr int kMaskOff = kBarOff + kNumBars * 8;
    static constexpr int kTmemOff = kMaskOff + ((kStages + 4) * 4 + 15) / 16 * 16;
    static constexpr int kSegOff = kTmemOff + 16;  // per softmax warp: its segment walk
    static constexpr int kBytes = kSegOff + kSoftmaxWarps * kSegBytes;
    static constexpr int kLaunchBytes = kBytes + 1024;
    static_assert(kLaunchBytes <= 227 * 1024, "shared memory of one CTA");
};
// warps: 0 K producer, 1 MMA issue for tile A, 2 V producer, 3 MMA issue for
// tile B;
// 4-7 softmax of query tile A, 8-11 of tile B (one M-row per thread)
constexpr int kThreads = 384;
// tensor memory: S_x[buf] (64 columns each) at 128x + 64buf, O_x at 256 + 128x
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kRescaleLog2 = 8;      // O is rescaled only when the max grows past 2^8
}  // namespace pf

struct PrefillRowInfo {
    int32_t r, g, i0, nq;  // queries i0 .. i0 + nq - 1 of row r's chunk, at positions kv_hi - nq ..
    int32_t q0;            // row of query i0 in q and out
    int32_t kv_lo, kv_hi, s;
    // sinks (kSink): the item's key tiles are numbered from 0 over its nst sink
    // tiles, then the window's; tile v >= nst is key tile v + gap.  Without
    // sinks tiles carry their own number.
    int32_t nst, gap;
};

// the first key tile of an item in its own numbering, and their number
template <bool kSink>
__device__ __forceinline__ int32_t item_first_tile(const PrefillRowInfo &w)
{
    return kSink ? 0 : w.kv_lo / pf::kKeys;
}
__device__ __forceinline__ int32_t item_tiles(const PrefillRowInfo &w)
{
    return w.nst + (w.kv_hi - 1) / pf::kKeys - w.kv_lo / pf::kKeys + 1;
}
template <bool kSink>
__device__ __forceinline__ int32_t key_tile(const PrefillRowInfo &w, int32_t v)
{
    return kSink && v >= w.nst ? v + w.gap : v;
}

// (a call has at most INT32_MAX items)
__device__ __forceinline__ bool prefill_item(const PrefillParams &p, int32_t bid, int qpc,
                                             PrefillRowInfo &w)
{
    w.s = bid % p.kv_splits;
    bid /= p.kv_splits;
    const int32_t qt = bid % p.q_tiles;
    bid /= p.q_tiles;
    w.g = bid % p.hkv;
    w.r = bid / p.hkv;
    const int32_t c0 = __ldg(p.cu_q_lens + w.r), c1 = __ldg(p.cu_q_lens + w.r + 1);
    int32_t C = c1 - c0;
    int32_t L = __ldg(p.seq_lens + w.r);
    const bool report_bad = qt == 0 && w.g == 0;
    if (L < 0 || L > p.max_len) {
        if (report_bad) report(p.status, PKV_DEV_BAD_LEN);
        L = L < 0 ? 0 : p.max_len;
    }
    const bool outside = c0 < 0 || C < 0 || c1 > p.num_queries;
    if (outside || C > p.max_q_len || C > L) {
        if (report_bad) report(p.status, PKV_DEV_BAD_LEN);
        C = outside ? 0 : min(min(C, p.max_q_len), L);
    }
    w.i0 = qt * qpc;
    if (w.i0 >= C) return false;
    w.q0 = c0 + w.i0;
    w.nq = min(qpc, C - w.i0);
    const int32_t p_first = L - C + w.i0;
    w.kv_hi = p_first + w.nq;
    // (a tree's queries may all sit right behind the cached tokens)
    w.kv_lo = p.window > 0 ? max(0, (p.tree != nullptr ? L - C : p_first) - p.window + 1) : 0;
    // tiles wholly before the window's first one that hold sinks
    const int32_t jw = w.kv_lo / pf::kKeys;
    w.nst = p.sinks > 0 ? min((min(p.sinks, w.kv_lo) + pf::kKeys - 1) / pf::kKeys, jw) : 0;
    w.gap = jw - w.nst;
    return true;
}

// Wait by every lane of the warp (false in all lanes if any gave up); reports
// a timeout.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int lane, int32_t *status,
                                          unsigned long long limit_ns)
{
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, limit_ns));
    if (!ok && lane == 0) report(status, PKV_DEV_TIMEOUT);
    return ok;
}

__device__ __forceinline__ bool warp_wait2(uint64_t *bar0, uint32_t parity0, uint64_t *bar1, uint32_t parity1, int lane,
                                           int32_t *status, unsigned long long limit_ns)
{
    const bool ok = __all_sync(0xffffffffu, mbar_wait2(bar0, parity0, bar1, parity1, limit_ns));
    if (!ok && lane == 0) report(status, PKV_DEV_TIMEOUT);
    return ok;
}

// ---------------------------------------------------------------------------
// Segments: the (item, key-tile range) pieces a CTA works through.  An item
// is a (row, kv head, query-tile pair); its key tiles are the 64-key tiles of
// its key range [kv_lo, kv_hi).
//   one CTA per item (sk_ctas == 0): one segment, the item's whole range or,
//     for the key-range runs of a short chunk, one run of it;
//   persistent balanced schedule (sk_ctas = n > 0, fewer than the items),
//     dealt by prefill_sk_plan_kernel: the items' tiles in item order form one
//     sequence of W tiles.  CTA c first runs the c-th item with tiles whole
//     (the CTAs of one (row, kv head) then start together and share its K/V
//     through L2), then a run of consecutive tiles of the rest, item by item.
//     The runs level the CTAs' costs, an item counting kSkItemCost tiles more
//     than it has: with w_c = max(0, level - the c-th item's cost), B the cost
//     of the first n such items and R that of the rest, CTA c's run starts
//     at cost B + R (w_0 + .. + w_(c-1)) / (w_0 + .. + w_(n-1)).  Only the
//     first and the last segment of a run can cut an item; a cut segment
//     writes a partial to slot 0 (first) or 1 (last) of the CTA, and the warp
//     that completes an item's pieces merges them.
//   drafted trees (kTree, sk_ctas > 0): every CTA a levelled run of the items'
//     tiles, none of them dealt whole, the pieces joined by prefill_tree_merge_kernel:
//     its items are few and long, a row's keys read by one of them (bf16, 32/8 heads,
//     4 rows of 8000 keys x 16 drafts: 56.6 us under the schedule above, 39.5 here).
//     An item counts kTreeOver tiles more than it has where runs are long: with 0 in
//     place of 6, 32 rows x 16 drafts 133.7 us against 122.8, with 10, 124.0; runs of
//     fewer than kTreeLeast tiles cost more than they bring (1 row of 1000 keys: 14.2 us
//     with 4, 17.3 with 8, 23.2 with 16).
// ---------------------------------------------------------------------------
struct Seg {
    PrefillRowInfo w;
    int32_t jt0;    // first key tile of the segment (64-key units, the item's numbering)
    int32_t ntile;  // tiles of the segment
    bool whole;     // the item's whole key range
    int32_t slot;   // persistent schedule: partial slot of a cut segment
    int32_t lo, cf, cl;  // persistent schedule: the item's first tile in the sequence,
                         // the first and the last CTA whose runs hold its tiles
};

// persistent schedule: pos .. end are the tiles of the CTA's run still ahead, u the
// item holding tile pos, k the segments returned so far
using SegWalk = Run;

// the plan's arrays: start of CTA c's run (c = n: the end of the sequence), the
// item that holds it, the item CTA c runs whole (-1: none)
__device__ __forceinline__ int32_t sk_run_start(const PrefillParams &p, int32_t c) { return __ldg(p.sk_plan + c); }
__device__ __forceinline__ int32_t sk_run_item(const PrefillParams &p, int32_t c) { return __ldg(p.sk_plan + p.sk_ctas + 1 + c); }
__device__ __forceinline__ int32_t sk_whole_item(const PrefillParams &p, int32_t c) { return __ldg(p.sk_plan + 2 * p.sk_ctas + 1 + c); }

// An item of the persistent schedule as the plan kernel recorded it (one read
// in place of the row's lengths, the prefix sums and the search for the next
// item with tiles, one after another).
struct alignas(16) SkItem {
    PrefillRowInfo w;
    int32_t lo, hi;  // its tiles in the sequence
    int32_t next;    // the next item with tiles
    int32_t cf, cl;  // first and last CTA whose runs hold its tiles
};
static_assert(sizeof(SkItem) == kSkItemBytes, "the workspace holds one per item");

__device__ __forceinline__ SkItem sk_load(const PrefillParams &p, int32_t u)
{
    union {
        SkItem it;
        int4 v[sizeof(SkItem) / 16];
    } r;
    const int4 *src = reinterpret_cast<const int4 *>(p.sk_rec) + static_cast<int64_t>(u) * (sizeof(SkItem) / 16);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(SkItem) / 16); ++i) r.v[i] = __ldg(src + i);
    return r.it;
}

// Next segment of a persistent CTA's run (false at its end).
template <bool kSink>
__device__ __forceinline__ bool sk_next(const PrefillParams &p, int qpc, SegWalk &sw, Seg &sg)
{
    if (sw.pos >= sw.end) return false;
    const SkItem it = sk_load(p, sw.u);
    const int32_t seg_end = min(it.hi, sw.end);
    sg.w = it.w;
    sg.jt0 = item_first_tile<kSink>(sg.w) + (sw.pos - it.lo);
    sg.ntile = seg_end - sw.pos;
    sg.whole = sw.pos == it.lo && seg_end == it.hi;
    sg.slot = sw.k == 0 ? 0 : 1;
    sg.lo = it.lo;
    sg.cf = it.cf;
    sg.cl = it.cl;
    ++sw.k;
    sw.pos = seg_end;
    if (seg_end == it.hi) sw.u = it.next;
    return true;
}

// What the merge needs of an item that a tree's run begins and does not end.
struct alignas(8) TreeRecord {
    int32_t q0, g;   // its first query, kv head
    int32_t rows;    // (query, head) pairs
    int32_t pieces;  // CTAs that hold a piece of it, this one first (0: there is no such item)
    int32_t slot;    // this CTA's piece's partial slot (the others': 0)
    int32_t pad;
};
static_assert(sizeof(TreeRecord) == kTreeRecordBytes, "the workspace holds one per CTA");

__device__ __forceinline__ int32_t tree_tiles(const PrefillParams &p, int32_t u, int qpc, PrefillRowInfo &w)
{
    return prefill_item(p, u, qpc, w) ? item_tiles(w) : 0;
}

// Next segment of a tree's run.
__device__ __forceinline__ bool tree_next(const PrefillParams &p, int qpc, SegWalk &sw, Seg &sg)
{
    RunPiece pc;
    while (sw.pos < sw.end) {
        const int32_t tiles = tree_tiles(p, sw.u, qpc, sg.w);
        if (!run_step(sw, tiles, pc)) continue;
        sg.jt0 = item_first_tile<false>(sg.w) + pc.t0;
        sg.ntile = pc.n;
        sg.whole = pc.whole;
        sg.slot = pc.slot;
        sg.lo = sg.cf = sg.cl = 0;
        return true;
    }
    return false;
}

// A tree's run, its first segment, the run's tiles (every thread of the CTA), and
// the record of the item that it begins and does not end.
constexpr int32_t kTreeLeast = 4, kTreeLevel = 16, kTreeOver = 6;
__device__ __forceinline__ bool tree_first(const PrefillParams &p, int qpc, int64_t *sm, SegWalk &sw, Seg &sg,
                                           int32_t &tiles)
{
    RunEnd e;
    sw = level_run<pf::kThreads>(
        p.sk_items,
        [&](int32_t u, bool) {
            PrefillRowInfo w;
            return tree_tiles(p, u, qpc, w);
        },
        p.sk_ctas, blockIdx.x, kTreeLeast, kTreeLevel, kTreeOver, sm, e);
    tiles = e.tiles;
    if (threadIdx.x == 96) {  // (of a warp that does not lead)
        TreeRecord rec{};
        if (e.pieces > 0) {
            PrefillRowInfo w;
            prefill_item(p, e.u, qpc, w);
            rec.q0 = w.q0;
            rec.g = w.g;
            rec.rows = w.nq * p.group;
            rec.pieces = e.pieces;
            rec.slot = e.slot;
        }
        static_cast<TreeRecord *>(p.sk_rec)[blockIdx.x] = rec;
    }
    return tree_next(p, qpc, sw, sg);
}

// First segment of CTA `cta` (false: nothing to do).  One CTA per item: the
// item (or its key-range run; an empty run sets ntile <= 0).
template <bool kSink>
__device__ __forceinline__ bool seg_first(const PrefillParams &p, int qpc, int32_t c, SegWalk &sw,
                                          Seg &sg)
{
    if (p.sk_ctas > 0) {
        const int32_t whole = sk_whole_item(p, c);
        sw.pos = sk_run_start(p, c);
        sw.end = sk_run_start(p, c + 1);
        sw.k = 0;
        sw.u = sk_run_item(p, c);
        if (whole >= 0) {
            const SkItem it = sk_load(p, whole);
            sg.w = it.w;
            sg.jt0 = item_first_tile<kSink>(sg.w);
            sg.ntile = it.hi - it.lo;
            sg.whole = true;
            sg.slot = 0;
            sg.lo = it.lo;
            sg.cf = sg.cl = 0;
            return true;
        }
        return sk_next<kSink>(p, qpc, sw, sg);
    }
    if (!prefill_item(p, c, qpc, sg.w)) return false;
    sg.jt0 = item_first_tile<kSink>(sg.w);
    sg.ntile = item_tiles(sg.w);
    sg.whole = p.kv_splits <= 1;
    sg.slot = 0;
    sg.lo = sg.cf = sg.cl = 0;
    if (!sg.whole) {
        const int32_t tb = sg.w.s * p.split_tiles;
        sg.ntile = min(sg.ntile, tb + p.split_tiles) - tb;
        sg.jt0 += tb;
    }
    sw.pos = sw.end = 0;  // no further segment
    return true;
}

template <bool kSink, bool kTree = false>
__device__ __forceinline__ bool seg_next(const PrefillParams &p, int qpc, SegWalk &sw, Seg &sg)
{
    if (kTree) return p.sk_ctas > 0 && tree_next(p, qpc, sw, sg);
    return p.sk_ctas > 0 && sk_next<kSink>(p, qpc, sw, sg);
}

// The key tiles of a CTA in order, over its segments (producers).
template <bool kSink, bool kTree>
struct TileCursor {
    SegWalk sw;
    Seg sg;
    int32_t j;  // tile within the segment
    bool valid;
    __device__ __forceinline__ void start(const PrefillParams &p, int qpc, const SegWalk &w0, const Seg &s0)
    {
        sw = w0;
        sg = s0;
        j = 0;
        valid = s0.ntile > 0;
        (void)p;
        (void)qpc;
    }
    __device__ __forceinline__ void advance(const PrefillParams &p, int qpc)
    {
        if (!valid) return;
        if (++j < sg.ntile) return;
        j = 0;
        valid = seg_next<kSink, kTree>(p, qpc, sw, sg);
    }
    __device__ __forceinline__ int32_t kt() const { return key_tile<kSink>(sg.w, sg.jt0 + j); }  // absolute key tile
};

// A softmax warp's 32 rows of a query tile into shared memory (warp wi = 0 .. 7:
// tile wi / 4, rows 32 (wi % 4) ..; row i = (query x*qpt + i/G, head i%G)),
// 128-byte swizzled for the tensor cores.  Sixteen lanes take one row's 256
// bytes, so that a load instruction covers two whole rows.  FP8 pools take f16
// products (bf16 -> f16 is exact inside the f16 range; a magnitude past 65504
// sets PKV_DEV_Q_RANGE); a negative scale is staged as -q (`flip` toggles the
// sign bits), so that the scores the tensor cores produce always take a
// positive factor.  Not inlined: a segment's staging then leaves the registers
// of the softmax loop around it alone.
template <bool kF8>
__device__ __noinline__ void stage_q_rows(const uint4 *q, int32_t hq, int glog,
                                          int qpt, int32_t q0, int32_t nq, int32_t g,
                                          uint32_t flip, int32_t *status, uint8_t *q_s, int wi, int lane)
{
    constexpr int kD = pf::kD, kRows = pf::kRows;
    const int x = wi >> 2, c = lane & 15, first = 32 * (wi & 3) + (lane >> 4);
    const uint4 *src = q + (static_cast<int64_t>(q0) * hq + (g << glog)) * (kD / 8) + c;
    uint8_t *qt_s = q_s + x * pf::kQBytes + (c >> 3) * (kRows * 128);
    uint4 v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int i = first + 2 * k, t = x * qpt + (i >> glog), h = i & ((1 << glog) - 1);
        v[k] = t < nq ? __ldg(src + (static_cast<int64_t>(t) * hq + h) * (kD / 8)) : make_uint4(0, 0, 0, 0);
    }
    bool qbad = false;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int i = first + 2 * k;
        if constexpr (kF8) {
            v[k].x = bf16x2_to_f16x2(v[k].x, qbad);
            v[k].y = bf16x2_to_f16x2(v[k].y, qbad);
            v[k].z = bf16x2_to_f16x2(v[k].z, qbad);
            v[k].w = bf16x2_to_f16x2(v[k].w, qbad);
        }
        v[k].x ^= flip;
        v[k].y ^= flip;
        v[k].z ^= flip;
        v[k].w ^= flip;
        *reinterpret_cast<uint4 *>(qt_s + i * 128 + (((c & 7) ^ (i & 7)) << 4)) = v[k];
    }
    if (qbad) report(status, PKV_DEV_Q_RANGE);
    fence_proxy_async_smem();  // read by the tensor cores (async proxy)
}

// K/V is re-read by the row's other CTAs; a tree that one item covers reads its row's
// pages once.  32 rows x 16 drafts, 32/8 heads, over 1024 to 8192 keys of their own: 112.6
// us with evict_first, 121.0 with evict_normal or evict_last.  Pages that rows share are
// read by each of them, at different times, and it holds there too: a prefix of 1024
// tokens shared by all 32 and up to 7168 of their own 124.3 against 130.0, of 32768
// tokens 738 against 751 (evict_last 753), of 8192 tokens 209.2 against 207.4.
template <bool kTree>
__device__ __forceinline__ uint64_t kv_policy(const PrefillParams &p)
{
    return kTree && p.q_tiles == 1 ? l2_evict_first_policy() : l2_evict_last_policy();
}

// ---------------------------------------------------------------------------
// bf16, tcgen05
// ---------------------------------------------------------------------------
// kSink: a window with sink tokens (their tiles first, then the window's)
// kTree: the queries are a drafted tree's, masked by their ancestors
// kAlt: every chunk fills one query tile at most; tile B's warps then take the
// same rows (their own S and O) and the two alternate over the key tiles, joined in
// the epilogue: a tile's chain (scores, softmax, products) has two tiles' time.  32 rows
// x 16 drafts 111 us, 142 without (32 drafts 133 and 148; FP8 132 and 167, 153 and 191
// before the waits in pairs)
template <bool kF8, bool kSink, bool kTree, bool kAlt>
__global__ void __launch_bounds__(pf::kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const PrefillParams p)
{
    using namespace pf;
    using L = Layout<kF8, kAlt>;
    constexpr int kStages = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *q_s = smem + kQOff;
    uint8_t *k_s = smem + L::kKOff;
    uint8_t *v_s = smem + L::kVOff;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint64_t *k_full = bars, *k_empty = bars + kStages, *v_full = bars + 2 * kStages,
             *v_empty = bars + 3 * kStages;
    uint64_t *s_full = bars + 4 * kStages;      // [tile * 2 + buf]
    uint64_t *p_full = bars + 4 * kStages + 4;  // [tile * 2 + buf]
    uint64_t *pv_done = bars + 4 * kStages + 8; // [tile]
    uint64_t *mma_drain = bars + 4 * kStages + 10;  // [tile]: the issuer's last products
    uint64_t *q_full = bars + 4 * kStages + 12;     // [tile]: a segment's query tile staged
    uint64_t *o_done = bars + 4 * kStages + 14;  // [tile]: a segment's last P.V product
    uint64_t *sums = bars + 4 * kStages + 16;    // kAlt: tile B's maxima and sums of a segment stored
    uint64_t *staged = bars + 4 * kStages + 18;  // FP8: [K/V * 2 + buffer]
    uint64_t *stg_free = bars + 4 * kStages + 22;  // FP8: [K/V * 2 + buffer] widened by the softmax warps
    uint32_t *kmask = reinterpret_cast<uint32_t *>(smem + L::kMaskOff);
    uint32_t *smask = kmask + kStages;  // FP8: [K/V * 2 + buffer] blocks loaded of a staging buffer
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kTmemOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.group;
    const int qpt = kRows / G;  // queries per query tile

    if (!kF8 && threadIdx.x == 0) {
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    pdl_wait();
    pdl_trigger();

    const int qpc = kQTiles * qpt;  // queries per item
    SegWalk sw0;
    Seg seg0;
    int32_t run_tiles = 0;  // kTree: of the CTA's run
    if (kTree && p.sk_ctas > 0) {
        // (the words are the segment walks' once every thread is past the barrier below)
        if (!tree_first(p, qpc, reinterpret_cast<int64_t *>(smem + L::kSegOff), sw0, seg0, run_tiles)) return;
    } else if (!seg_first<kSink>(p, qpc, blockIdx.x, sw0, seg0)) {
        return;
    }
    const bool split = p.kv_splits > 1;  // one CTA per key-range run of a short chunk
    if (split && seg0.ntile <= 0) {
        // an empty run: an empty partial (no weight) for every live row
        const PrefillRowInfo &w = seg0.w;
        if (warp >= 4) {
            const int x = (warp >> 2) - 1, row = 32 * (warp & 3) + lane;
            const int t = x * qpt + row / G;
            if (row < qpt * G && t < w.nq) {
                const size_t pi = ((static_cast<size_t>(w.r) * p.max_q_len + w.i0 + t) * p.hq +
                                   w.g * G + row % G) * p.kv_splits + w.s;
                *reinterpret_cast<float2 *>(p.ws_ml + pi * 2) = make_float2(-INFINITY, 0.f);
            }
        }
        return;
    }
    // query tiles with queries in them: a short chunk (a verify step of a few
    // queries) fills tile A only, and tile B's warps then stay idle; the
    // persistent schedule runs both (its segments' items differ)
    const int nqt = (kAlt || p.sk_ctas > 0 || seg0.w.nq > qpt) ? 2 : 1;
    const int users = kAlt ? 1 : nqt;  // query tiles that read a K/V tile
    // kAlt: tile T is warpgroup T & 1's, as its tile T >> 1
    constexpr int kStep = kAlt ? 2 : 1;
    const auto own = [](int32_t T) { return kAlt ? T >> 1 : T; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            // the S products of the live tiles + their warpgroups' kmask reads
            mbar_init(&k_empty[i], users + users * (kSoftmaxWarps / kQTiles));
            // FP8: one softmax warpgroup widens K into the stages, the other
            // V (tile A's both when it runs alone); bf16: one TMA arrival
            mbar_init(&k_full[i], kF8 ? kSoftmaxWarps / kQTiles : 1);
            mbar_init(&v_full[i], kF8 ? kSoftmaxWarps / kQTiles : 1);
            mbar_init(&v_empty[i], users);  // the live tiles' P.V products
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], kSoftmaxWarps / kQTiles);
        }
        mbar_init(&pv_done[0], 1);
        mbar_init(&pv_done[1], 1);
        mbar_init(&mma_drain[0], 1);
        mbar_init(&mma_drain[1], 1);
        mbar_init(&o_done[0], 1);
        mbar_init(&o_done[1], 1);
        mbar_init(&q_full[0], kSoftmaxWarps / kQTiles);
        // (kAlt: both by tile A's warps, once they have read the last segment's O of
        // both tiles and staged the queries)
        mbar_init(&q_full[1], kSoftmaxWarps / kQTiles);
        mbar_init(&sums[0], kSoftmaxWarps / kQTiles);
        if (kF8) {
            for (int i = 0; i < 4; ++i) mbar_init(&staged[i], 1);
            for (int i = 0; i < 4; ++i) mbar_init(&stg_free[i], kSoftmaxWarps / kQTiles);
        }
        fence_mbar_init();
    }
    if (warp == 1) tc::alloc(tmem_slot, kTmemCols);

    // query tiles: tile x row i = (query t = x * qpt + i / G, head h = i % G);
    // the softmax warps load 32 rows each (a segment's before its first tile)
    // a negative scale: stage -q (sign bits flipped, exact), so that the
    // scores the tensor cores produce always take a positive factor
    const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    const int glog = __ffs(G) - 1;  // G divides the tile's 128 rows
    auto load_q_rows = [&](const PrefillRowInfo &w) {
        stage_q_rows<kF8>(static_cast<const uint4 *>(p.q), p.hq, glog, kAlt ? 0 : qpt, w.q0, w.nq, w.g, flip, p.status, q_s, warp - 4, lane);
    };
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    auto tS = [&](int x, int buf) { return tmem + 128u * static_cast<uint32_t>(x) + 64u * static_cast<uint32_t>(buf); };
    auto tO = [&](int x) { return tmem + 256u + 128u * static_cast<uint32_t>(x); };

    if (warp == 0 || warp == 2) {
        // ------------------------------------------ K (warp 0) / V (warp 2) producer
        // The CTA's key tiles in order over its segments; tile T (a running
        // count) goes to ring stage T % kStages.
        const bool is_k = warp == 0;
        // diagnostic drill: tile 0's loads are never issued (its waits run out)
        auto withheld = [&](int32_t T) { return (p.drill & kDrillWithholdFirst) != 0 && T == 0; };
        uint8_t *ring = is_k ? k_s : v_s;
        uint64_t *full = is_k ? k_full : v_full;
        uint64_t *empty = is_k ? k_empty : v_empty;
        // lane < kBlocks: logical block kt * kBlocks + lane of the cursor's
        // tile, inside the table and the item's key range
        auto in_range_of = [&](const TileCursor<kSink, kTree> &c) {
            const int32_t kb = c.kt() * kBlocks + lane;
            return c.valid && lane < kBlocks && kb < p.width && kb * 16 < c.sg.w.kv_hi &&
                   ((kb + 1) * 16 > c.sg.w.kv_lo || (kSink && kb * 16 < p.sinks));
        };
        auto load_id = [&](const TileCursor<kSink, kTree> &c) {
            return in_range_of(c) ? __ldg(p.tables + static_cast<int64_t>(c.sg.w.r) * p.width +
                                          c.kt() * kBlocks + lane)
                                  : -1;
        };
        if constexpr (kF8) {
            // FP8: tile T's E4M3 blocks are bulk-copied into staging buffer
            // T % 2 (two tiles ahead of the ring), then widened to f16 into
            // the ring stage: K as the bf16 path lays it out (key rows, 64-dim
            // 128-byte-swizzled regions), V transposed (dim rows of the tile's
            // 64 keys, 128-byte swizzled), so that a pair of codes becomes
            // one 4-byte store.  Value columns of keys outside [kv_lo, kv_hi)
            // or of blocks not loaded are written as zeros (stale slots may
            // hold NaN codes).
            const uint64_t policy = kv_policy<kTree>(p);
            const uint8_t *pool = static_cast<const uint8_t *>(is_k ? p.k_pool : p.v_pool);
            uint8_t *stg = smem + L::kStagingOff + (is_k ? 0 : 2) * kF8StageTile;
            uint64_t *stg_bar = staged + (is_k ? 0 : 2);
            int32_t nf = 0;  // tiles 0 .. nf-1 fetched into the staging buffers
            // fetch tile nf at cursor c (block ids read one tile before);
            // whole warp; returns the mask of loaded blocks
            auto fetch = [&](const TileCursor<kSink, kTree> &c, int32_t id) {
                const bool in_range = in_range_of(c);
                const bool good = in_range && static_cast<uint32_t>(id) < static_cast<uint32_t>(p.num_blocks);
                if (is_k && in_range && !good) report(p.status, PKV_DEV_BAD_BLOCK);
                const uint32_t mask = __ballot_sync(0xffffffffu, good) & ((1u << kBlocks) - 1u);
                const int32_t tile = nf++;
                const int sb = tile & 1;
                if (lane == 0) smask[(is_k ? 0 : 2) + sb] = mask;  // published by the arrival below
                if (withheld(tile)) return mask;  // diagnostic drill: never issued
                if (lane == 0) {
                    if (mask == 0)
                        mbar_arrive(&stg_bar[sb]);
                    else
                        mbar_arrive_expect_tx(&stg_bar[sb], __popc(mask) * kF8BlockBytes);
                }
                __syncwarp();
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    const int32_t bid = __shfl_sync(0xffffffffu, id, b);
                    if (((mask >> b) & 1u) && elect_one())
                        bulk_load(stg + sb * kF8StageTile + b * kF8BlockBytes,
                                  pool + (static_cast<int64_t>(bid) * p.hkv + c.sg.w.g) * kF8BlockBytes,
                                  kF8BlockBytes, &stg_bar[sb], policy);
                }
                __syncwarp();
                return mask;
            };
            // bulk copies only, two tiles ahead; the softmax warps widen each
            // tile into the ring and release the staging buffer
            TileCursor<kSink, kTree> cf, ci;
            cf.start(p, qpc, sw0, seg0);
            ci = cf;
            int32_t id_next = load_id(ci);
            ci.advance(p, qpc);
            int32_t T = 0;
            for (; cf.valid; ++T, cf.advance(p, qpc)) {
                const int sb = T & 1;
                if (T >= 2 && !warp_wait(&stg_free[(is_k ? 0 : 2) + sb], ((T >> 1) + 1) & 1, lane, p.status,
                                         p.wait_ns))
                    break;
                fetch(cf, id_next);
                id_next = load_id(ci);
                ci.advance(p, qpc);
            }
            // the copies this warp issued have landed before it leaves
            if (lane == 0)
                for (int32_t t = max(0, T - 2); t < T; ++t)
                    if (!withheld(t)) mbar_wait(&stg_bar[t & 1], (t >> 1) & 1);
            __syncwarp();
        } else {
            const CUtensorMap *map = is_k ? &kmap : &vmap;
            const uint64_t policy = kv_policy<kTree>(p);
            TileCursor<kSink, kTree> cur;
            cur.start(p, qpc, sw0, seg0);
            int32_t T = 0;
            for (; cur.valid; ++T, cur.advance(p, qpc)) {
                const int st = T % kStages;
                if (T >= kStages && !warp_wait(&empty[st], ((T / kStages) + 1) & 1, lane, p.status, p.wait_ns)) break;
                const bool in_range = in_range_of(cur);
                const int32_t id = load_id(cur);
                const bool good = in_range && static_cast<uint32_t>(id) < static_cast<uint32_t>(p.num_blocks);
                if (is_k && in_range && !good) report(p.status, PKV_DEV_BAD_BLOCK);
                const uint32_t mask = __ballot_sync(0xffffffffu, good) & ((1u << kBlocks) - 1u);
                if (is_k && lane == 0) kmask[st] = mask;
                if (withheld(T)) continue;  // diagnostic drill: never issued
                if (lane == 0) {
                    if (mask == 0)
                        mbar_arrive(&full[st]);
                    else
                        mbar_arrive_expect_tx(&full[st], __popc(mask) * 2 * 2048);
                }
                __syncwarp();
                uint8_t *dst = ring + st * kTileBytes;
                const int32_t g = cur.sg.w.g;
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    const int32_t bid = __shfl_sync(0xffffffffu, id, b);
                    if (((mask >> b) & 1u) && elect_one()) {
                        tma_load_4d(dst + b * 2048, map, &full[st], 0, 0, g, bid, policy);
                        tma_load_4d(dst + kKVRegion + b * 2048, map, &full[st], 64, 0, g, bid, policy);
                    }
                }
            }
            // wind-down (a wait ran out) and normal exit alike: the loads of
            // the last ring's worth of tiles have landed before the warp
            // leaves (at a normal exit their consumers saw them land already)
            if (lane == 0)
                for (int32_t t = max(0, T - kStages); t < T; ++t)
                    if (!withheld(t)) mbar_wait(&full[t % kStages], (t / kStages) & 1);
            __syncwarp();
        }
    } else if (warp == 1 || (warp == 3 && nqt == 2)) {
        // ------------------------------------------------------------ MMA issue
        // Warp 1 issues tile A's products, warp 3 tile B's.  Per K/V tile j:
        // P(j).V, then S(j+2) = Q K(j+2)^T into the S buffer that product just
        // read.  With two S buffers a warpgroup finds S(j+1) computed when it
        // finishes P(j).  One thread's products execute in issue order, so a
        // product never overtakes an earlier read of the same columns.
        const int x = warp >> 1;
        // bf16: V is MN-major (key rows); FP8: V^T is K-major (dim rows of keys)
        constexpr uint32_t idS = kF8 ? tc::idesc_f16(kRows, kKeys, 0, 0) : tc::idesc_bf16(kRows, kKeys, 0, 0);
        constexpr uint32_t idO = kF8 ? tc::idesc_f16(kRows, kD, 0, 0) : tc::idesc_bf16(kRows, kD, 0, 1);
        // Descriptors are built once; moving along K (or to the next 16 keys
        // of V) adds the byte offset / 16 to the start-address field, which
        // cannot carry out of it inside shared memory.
        const uint64_t dq = tc::smem_desc(smem_u32(q_s + (kAlt ? 0 : x) * kQBytes), 16, 1024);
        const uint64_t dk = tc::smem_desc(smem_u32(k_s), 16, 1024);
        const uint64_t dv = kF8 ? tc::smem_desc(smem_u32(v_s), 16, 1024)
                                : tc::smem_desc(smem_u32(v_s), kKVRegion, 1024);
        // the B operand of the keys 16kk .. 16kk+15: bf16 key rows 16kk.. (2 KiB
        // on); FP8 32 bytes along each dim row
        constexpr uint64_t kVStep = kF8 ? (32 >> 4) : (2048 >> 4);
        constexpr uint64_t kStageStep = kTileBytes >> 4;
        const uint32_t tO_x = tO(x);
        // The whole warp waits; one elected lane issues a step's products and
        // commits from one straight-line block.
        auto k_landed = [&](int32_t T) {  // K(T) landed (T: the CTA's running tile count)
            return warp_wait(&k_full[T % kStages], (T / kStages) & 1, lane, p.status, p.wait_ns);
        };
        auto s_issue = [&](int32_t T) {  // S(T) = Q K(T)^T
            const uint64_t kd = dk + static_cast<uint64_t>(T % kStages) * kStageStep;
            const uint32_t d = tS(x, own(T) & 1);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                const uint64_t qo = static_cast<uint64_t>(((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4);
                const uint64_t ko = static_cast<uint64_t>(((kk >> 2) * kKVRegion + (kk & 3) * 32) >> 4);
                tc::mma_ss(d, dq + qo, kd + ko, idS, kk > 0 ? 1u : 0u);
            }
            tc::commit(&s_full[x * 2 + (own(T) & 1)]);
            tc::commit(&k_empty[T % kStages]);
        };
        // O += P(T) V(T); V(T) has landed (bf16: the warpgroup checked it before
        // handing P over); a segment's first tile starts O afresh
        auto pv_issue = [&](int32_t T, bool seg_start) {
            const uint64_t vd = dv + static_cast<uint64_t>(T % kStages) * kStageStep;
            const uint32_t a = tS(x, own(T) & 1);
            const uint32_t first = seg_start ? 0u : 1u;
            // bf16: keys 16g..16g+15 hold P hi in S columns 16g..16g+7 and P
            // lo in 16g+8..16g+15 (bf16 pairs); FP8 pools: one f16 term, keys
            // 16g..16g+15 in columns 8g..8g+7
#pragma unroll
            for (int part = 0; part < (kF8 ? 1 : 2); ++part)
#pragma unroll
                for (int kk = 0; kk < kBlocks; ++kk)
                    tc::mma_ts(tO_x, a + (kF8 ? 8 : 16) * kk + 8 * part, vd + kVStep * static_cast<uint64_t>(kk),
                               idO, (part > 0 || kk > 0) ? 1u : first);
            tc::commit(&pv_done[x]);
            tc::commit(&v_empty[T % kStages]);
        };
        SegWalk sw = sw0;
        Seg sg = seg0;
        int32_t T0 = 0;  // the segment's first tile in the running count
        for (int32_t k = 0;; ++k) {
            const int32_t n = sg.ntile;
            // the segment's query tile is staged (the previous segment's
            // products, which read the old one, completed before its epilogue)
            bool ok = warp_wait(&q_full[x], k & 1, lane, p.status, p.wait_ns);
            const int32_t j0 = kAlt ? (T0 ^ x) & 1 : 0;  // its first tile of the segment
            const bool one = j0 < n, two = j0 + kStep < n;
            ok = ok && (!one || k_landed(T0 + j0)) && (!two || k_landed(T0 + j0 + kStep));
            if (ok) {
                tc::fence_after();
                if (elect_one()) {
                    if (one) s_issue(T0 + j0);
                    if (two) s_issue(T0 + j0 + kStep);
                    if (kAlt && !one) tc::commit(&o_done[x]);  // nothing of this segment
                }
                __syncwarp();
            }
            // per tile (kAlt: every other): K(T+2) is waited for first (it landed, or was widened,
            // long before P(T) is ready), so that P(T).V(T) and S(T+2) leave
            // in one block as soon as P(T) is
            for (int32_t j = j0; j < n && ok; j += kStep) {
                const int32_t T = T0 + j, u = own(T);
                const bool more = j + 2 * kStep < n;
                if (more) ok = k_landed(T + 2 * kStep);
                // FP8: V(T) is waited for here (on bf16 pools the softmax warps, which may have
                // rows of it to zero, do: 4 chunks of 512 480 us, 483 with the wait here)
                ok = ok && (kF8 ? warp_wait2(&p_full[x * 2 + (u & 1)], (u >> 1) & 1, &v_full[T % kStages],
                                             (T / kStages) & 1, lane, p.status, p.wait_ns)
                                : warp_wait(&p_full[x * 2 + (u & 1)], (u >> 1) & 1, lane, p.status, p.wait_ns));
                if (!ok) break;
                tc::fence_after();
                if (elect_one()) {
                    pv_issue(T, j == j0);
                    if (j + kStep >= n) tc::commit(&o_done[x]);
                    if (more) s_issue(T + 2 * kStep);
                }
                __syncwarp();
            }
            if (!ok) break;
            T0 += n;
            if (!seg_next<kSink, kTree>(p, qpc, sw, sg)) break;
        }
        // every product this warp issued has completed before the CTA frees
        // tensor memory (after a wait ran out, some may still be running)
        if (elect_one()) tc::commit(&mma_drain[x]);
        __syncwarp();
        mbar_wait(&mma_drain[x], 0);
        __syncwarp();
    } else if (warp >= 4 && (warp < 8 || nqt == 2)) {
        // ------------------------------------------------------------ softmax
        // warpgroup x (warps 4-7: tile A, 8-11: tile B), one M-row per thread:
        // tensor-memory lane quarter warp % 4, the 64 key columns of S
        const int x = (warp >> 2) - 1;
        const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const int row = 32 * (warp & 3) + lane;
        const int t = (kAlt ? 0 : x * qpt) + row / G;
        const uint32_t ox = tO(x) + lane_base;
        // |scale| * log2(e) (q was staged negated for a negative scale), kept
        // away from 0 so that a masked score (-inf) never meets a zero factor
        const float sl = fmaxf(fabsf(p.scale_log2), 1e-30f);
        bool abort = false;
        // FP8: tile A's warpgroup widens K, tile B's V (tile A's both when it
        // runs alone), each 128 threads over a tile's 512 staged chunks: a
        // warp then waits for one staging and one ring barrier per tile, and
        // the two warpgroups need not run in step.  kAlt: each both of its own tiles.
        // K(Tk)'s staged E4M3 chunks, this thread's share, widened to f16
        // into ring stage Tk % kStages (key rows, 64-dim 128-byte-swizzled
        // regions, as the bf16 path lays them out); keys of blocks not loaded
        // are left as they are (their scores are masked).  The stage is free
        // once tile Tk - kStages's S products and mask reads are done.
        const bool do_k = kAlt || nqt == 1 || x == 0, do_v = kAlt || nqt == 1 || x == 1;
        const int wq0 = (threadIdx.x - 128) & (kRows - 1);  // this thread's first chunk
        auto widen_k = [&](int32_t Tk) {
            const int sb = Tk & 1, st = Tk % kStages;
            const bool okw = Tk < kStages ? mbar_wait(&staged[sb], (Tk >> 1) & 1, p.wait_ns)
                                          : mbar_wait2(&staged[sb], (Tk >> 1) & 1, &k_empty[st],
                                                       ((Tk / kStages) + 1) & 1, p.wait_ns);
            if (__any_sync(0xffffffffu, !okw)) return false;
            const uint32_t km = smask[sb];
            if ((kAlt ? row : static_cast<int>(threadIdx.x) - 128) == 0) kmask[st] = km;  // for the score masks of tile Tk
            const uint32_t src = smem_u32(smem + L::kStagingOff + sb * kF8StageTile);
            const uint32_t dst = smem_u32(k_s + st * kTileBytes);
            // A warp takes 32 chunks of one (block, 64-dim group, token half):
            // lane l holds key 8 half + l/4, dims 16kk + 2(l%4) + {0, 1, 8, 9}
            // (kk = 0..3), i.e. the 8x8 matrices (keys) x (dims 16kk + 8h ..
            // + 7) in the fragment order that stmatrix stores as 16-byte rows.
            // Matrix 2kk + h is 16-byte chunk 2kk + h of each key's 128-byte
            // row, swizzled by the key row.
            const int mr = lane & 7, mm = lane >> 3;  // this lane's row address: row mr of matrix mm
            // The four blocks' chunks are read first, so that the reads are in
            // flight together (a block not loaded reads stale bytes, unused).
            const int ch = wq0, grp = ch >> 6, half = (ch >> 5) & 1;  // warp-uniform but for ch % 32
            uint4 q4[kBlocks];
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) q4[b] = lds128(src + b * kF8BlockBytes + ch * 16);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                if (!((km >> b) & 1u)) continue;
                uint32_t f[8];  // f[2kk + h]: matrix (kk, h)
                e4m3x4_to_f16x2x2(q4[b].x, f[0], f[1]);
                e4m3x4_to_f16x2x2(q4[b].y, f[2], f[3]);
                e4m3x4_to_f16x2x2(q4[b].z, f[4], f[5]);
                e4m3x4_to_f16x2x2(q4[b].w, f[6], f[7]);
                const int krow = b * 16 + half * 8 + mr;
                const uint32_t rowa = dst + grp * kKVRegion + krow * 128;
                stsm_x4(rowa + ((mm ^ mr) << 4), f[0], f[1], f[2], f[3]);
                stsm_x4(rowa + (((4 + mm) ^ mr) << 4), f[4], f[5], f[6], f[7]);
            }
            // read by the tensor cores (async proxy); the staging buffer is
            // refilled by bulk copies after these generic-proxy reads
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&k_full[st]);
                mbar_arrive(&stg_free[sb]);
            }
            return true;
        };
        // the CTA's tiles over all its segments
        const int32_t T_total =
            kTree && p.sk_ctas > 0 ? run_tiles
            : p.sk_ctas > 0 ? (seg0.whole && sk_whole_item(p, blockIdx.x) >= 0 ? seg0.ntile : 0) +
                                sk_run_start(p, blockIdx.x + 1) - sk_run_start(p, blockIdx.x)
                          : seg0.ntile;
        if (!kAlt || x == 0) load_q_rows(seg0.w);  // while the producers' first copies are under way
        if constexpr (kF8) {
            for (int32_t Tk = kAlt ? x : 0; do_k && Tk < min(2 * kStep, T_total) && !abort; Tk += kStep)
                if (!widen_k(Tk)) {
                    if (lane == 0) report(p.status, PKV_DEV_TIMEOUT);
                    abort = true;
                }
        }
        // this warp's segment walk, its current segment and the next one live in
        // shared memory (lane 0 writes them): the tile loop keeps its registers
        struct SegSmem {
            SegWalk sw;
            Seg sg[2];  // segment k at k & 1
        };
        static_assert(sizeof(SegSmem) <= kSegBytes, "the per-warp segment slot");
        SegSmem *ss = reinterpret_cast<SegSmem *>(smem + L::kSegOff) + (warp - 4);
        if (lane == 0) {
            ss->sw = sw0;
            ss->sg[0] = seg0;
        }
        __syncwarp();
        int32_t T0 = 0;  // the segment's first tile in the running count
        for (int32_t k = 0; !abort; ++k) {
        const Seg &cs = ss->sg[k & 1];
        const int32_t ntile = cs.ntile, jt0 = cs.jt0;
        const int32_t kv_lo = cs.w.kv_lo, kv_hi = cs.w.kv_hi;
        const int32_t nst = kSink ? cs.w.nst : 0, gap = kSink ? cs.w.gap : 0;
        // the segment's query tile: staged (the first above), then handed to
        // the MMA-issue warp
        if (k > 0 && (!kAlt || x == 0)) load_q_rows(cs.w);
        __syncwarp();
        if (lane == 0 && (!kAlt || x == 0)) {
            mbar_arrive(&q_full[x]);
            if (kAlt) mbar_arrive(&q_full[1]);
        }
        const bool valid_row = row < qpt * G && t < cs.w.nq;
        const int32_t qpos = cs.w.kv_hi - cs.w.nq + t;
        // kTree: positions below `first` hold the cached tokens, the drafts follow
        const int32_t first = cs.w.kv_hi - cs.w.nq - cs.w.i0;
        uint64_t tmask = 0;
        if constexpr (kTree) tmask = valid_row ? tree_mask(p.tree, cs.w.q0 + t, cs.w.i0 + t) : 0ull;
        const int32_t at = kTree ? first + tree_depth(tmask) : qpos;  // where its window ends
        const int32_t qlo = p.window > 0 ? max(0, at - p.window + 1) : 0;
        float m_ref = -INFINITY, l = 0.f;
        const bool warp_live = __any_sync(0xffffffffu, valid_row);
        const int32_t j0 = kAlt ? (T0 ^ x) & 1 : 0;  // this warpgroup's first tile
        for (int32_t jj = j0; jj < ntile; jj += kStep) {
            const int32_t T = T0 + jj, u = own(T);
            const int ks = T % kStages, buf = u & 1;
            const int32_t tbase = (jt0 + jj + (kSink && jt0 + jj >= nst ? gap : 0)) * kKeys;
            const uint32_t sx = tS(x, buf) + lane_base;
            if constexpr (kF8 && !kAlt) {
                if (do_k && T + 2 < T_total && !widen_k(T + 2)) {
                    if (lane == 0) report(p.status, PKV_DEV_TIMEOUT);
                    abort = true;
                    break;
                }
            }
            if (kF8 && do_v) {
                // V(T): this thread's share of the staged E4M3 chunks widened to
                // f16 into ring stage T % kStages, transposed (dim rows of the
                // tile's 64 keys, 128-byte swizzled); value columns of keys
                // outside [kv_lo, kv_hi) or of blocks not loaded as zeros.  The
                // stage is free once both tiles' P.V(T - kStages) completed.
                const int sb = T & 1;
                const bool okw = T < kStages ? mbar_wait(&staged[2 + sb], (T >> 1) & 1, p.wait_ns)
                                             : mbar_wait2(&staged[2 + sb], (T >> 1) & 1, &v_empty[ks],
                                                          ((T / kStages) + 1) & 1, p.wait_ns);
                if (__any_sync(0xffffffffu, !okw)) {
                    if (lane == 0) report(p.status, PKV_DEV_TIMEOUT);
                    abort = true;
                    break;
                }
                const uint32_t vm = smask[2 + sb];
                const uint32_t src = smem_u32(smem + L::kStagingOff + 2 * kF8StageTile + sb * kF8StageTile);
                const uint32_t dst = smem_u32(v_s + ks * kTileBytes);
                const bool vedge = (tbase < kv_lo && !(kSink && tbase + kKeys <= p.sinks)) || tbase + kKeys > kv_hi;
                // A warp takes the 32 chunks of one (block, 32-dim group): lane
                // l holds dim 32g + 8jn + l/4 (jn = 0..3) for keys 16b + 2(l%4)
                // + {0, 1, 8, 9}, i.e. the 8x8 matrices (dims 32g + 8jn .. + 7)
                // x (keys 16b + 8h .. + 7) in stmatrix fragment order.  Matrix
                // (jn, h) is 16-byte chunk 2b + h of each dim row, swizzled by
                // the dim row.
                const int mr = lane & 7, mm = lane >> 3, c = lane & 3;
                const int ch = wq0, g32 = ch >> 5;  // warp-uniform but for ch % 32
                uint4 q4[kBlocks];
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) q4[b] = lds128(src + b * kF8BlockBytes + ch * 16);
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    uint32_t f[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};  // f[2jn + h]: matrix (jn, h)
                    if ((vm >> b) & 1u) {
                        e4m3x4_to_f16x2x2(q4[b].x, f[0], f[1]);
                        e4m3x4_to_f16x2x2(q4[b].y, f[2], f[3]);
                        e4m3x4_to_f16x2x2(q4[b].z, f[4], f[5]);
                        e4m3x4_to_f16x2x2(q4[b].w, f[6], f[7]);
                        if (vedge) {
                            auto live = [&](int k) {
                                const int32_t kp = tbase + b * 16 + k;
                                return (kp >= kv_lo || (kSink && kp < p.sinks)) && kp < kv_hi;
                            };
                            const uint32_t mk0 = (live(2 * c) ? 0x0000ffffu : 0u) | (live(2 * c + 1) ? 0xffff0000u : 0u);
                            const uint32_t mk1 = (live(2 * c + 8) ? 0x0000ffffu : 0u) | (live(2 * c + 9) ? 0xffff0000u : 0u);
#pragma unroll
                            for (int jn = 0; jn < 4; ++jn) {
                                f[2 * jn] &= mk0;
                                f[2 * jn + 1] &= mk1;
                            }
                        }
                    }
                    // row mr of matrix mm: dim 32g + 8(jn0 + mm/2) + mr, chunk 2b + mm%2
                    const uint32_t rowa = dst + (g32 * 32 + (mm >> 1) * 8 + mr) * 128;
                    const uint32_t cx = static_cast<uint32_t>(((2 * b + (mm & 1)) ^ mr) << 4);
                    stsm_x4(rowa + cx, f[0], f[1], f[2], f[3]);
                    stsm_x4(rowa + 16 * 128 + cx, f[4], f[5], f[6], f[7]);
                }
                // read by the tensor cores (async proxy); the staging buffer is
                // refilled by bulk copies after these generic-proxy reads
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&v_full[ks]);
                    mbar_arrive(&stg_free[2 + sb]);
                }
            }
            // (k_full for kmask; on bf16 pools one after the other: together 478 -> 484 us
            // for 4 chunks of 512, on FP8 pools 585 -> 549 with the widening's pairs, and
            // 525 with V's wait in the issuing warp)
            const bool got = kF8 ? mbar_wait2(&s_full[x * 2 + buf], (u >> 1) & 1, &k_full[ks], (T / kStages) & 1, p.wait_ns)
                                 : mbar_wait(&s_full[x * 2 + buf], (u >> 1) & 1, p.wait_ns) &&
                                       mbar_wait(&k_full[ks], (T / kStages) & 1, p.wait_ns);
            if (__any_sync(0xffffffffu, !got)) {
                if (lane == 0) report(p.status, PKV_DEV_TIMEOUT);
                abort = true;
                break;
            }
            const uint32_t mask = kmask[ks];
            __syncwarp();
            if (lane == 0) mbar_arrive(&k_empty[ks]);
            if constexpr (kF8 && kAlt) {  // into the stage that S(T) and the warps' masks have just left
                if (T + 2 * kStep < T_total && !widen_k(T + 2 * kStep)) {
                    if (lane == 0) report(p.status, PKV_DEV_TIMEOUT);
                    abort = true;
                    break;
                }
            }
            tc::fence_after();
            // a warp whose 32 rows hold no query (a short chunk fills only the
            // first rows of the tile) leaves its S rows alone: the P.V product
            // then writes only O rows that are never stored
            if (warp_live) {
                float s[64];
                {
                    uint32_t r0[32], r1[32];
                    tc::ld32(sx, r0);
                    tc::ld32(sx + 32, r1);
                    tc::wait_ld();
    #pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        s[e] = __uint_as_float(r0[e]);
                        s[32 + e] = __uint_as_float(r1[e]);
                    }
                }
                // a tile with any key outside this row's range takes the masked
                // path: key column e is attended iff e - lo is in [0, qpos - qlo]
                // and its block was loaded
                const bool full = mask == (1u << kBlocks) - 1u &&
                                  tbase >= qlo &&
                                  tbase + kKeys - 1 <= (kTree ? first - 1 : qpos) && valid_row;
                if (!full) {
                    // attended columns as bits: the window's from qlo to qpos, the
                    // sinks' up to the query's own, both within loaded blocks
                    const auto below = [](int32_t n) {  // bits 0 .. n-1
                        return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull;
                    };
                    uint64_t bits = below(qpos + 1 - tbase);
                    bits &= kSink ? ~below(qlo - tbase) | below(p.sinks - tbase) : ~below(qlo - tbase);
                    if constexpr (kTree) bits &= tree_bits(tmask, tbase, first);
                    const uint32_t bm = valid_row ? mask : 0u;
                    uint64_t blocks = 0;
    #pragma unroll
                    for (int b = 0; b < kBlocks; ++b) blocks |= ((bm >> b) & 1u) ? 0xFFFFull << (16 * b) : 0ull;
                    bits &= blocks;
                    const uint32_t b0 = static_cast<uint32_t>(bits), b1 = static_cast<uint32_t>(bits >> 32);
    #pragma unroll
                    for (int e = 0; e < 64; ++e) s[e] = (((e < 32 ? b0 : b1) >> (e & 31)) & 1u) ? s[e] : -INFINITY;
                }
                float mt;
                {
                    float m8[8];
    #pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        m8[e] = fmax3(s[e], s[8 + e], s[16 + e]);
                        m8[e] = fmax3(m8[e], s[24 + e], s[32 + e]);
                        m8[e] = fmax3(m8[e], s[40 + e], s[48 + e]);
                        m8[e] = fmaxf(m8[e], s[56 + e]);
                    }
                    mt = fmaxf(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], fmax3(m8[5], m8[6], m8[7]))) * sl;
                }
                // keep the reference max within 2^8 of the running max
                const float new_ref = (mt > m_ref + static_cast<float>(kRescaleLog2)) ? mt : m_ref;
                const float alpha = fast_exp2(m_ref - new_ref);  // 0 from -inf, 1 if unchanged
                const bool resc = new_ref != m_ref && m_ref != -INFINITY;
                if (__any_sync(0xffffffffu, resc)) {
                    // O_x holds P.V up to tile jj-1 once that product completes
                    if (jj > j0) {
                        const bool done = mbar_wait(&pv_done[x], (u - 1) & 1, p.wait_ns);
                        if (__any_sync(0xffffffffu, !done)) {
                            if (lane == 0) report(p.status, PKV_DEV_TIMEOUT);
                            abort = true;
                            break;
                        }
                        tc::fence_after();
                    }
                    const float f = resc ? alpha : 1.f;
    #pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t r32[32];
                        tc::ld32(ox + c * 32, r32);
                        tc::wait_ld();
    #pragma unroll
                        for (int e = 0; e < 32; ++e) r32[e] = __float_as_uint(__uint_as_float(r32[e]) * f);
                        tc::st32(ox + c * 32, r32);
                    }
                    tc::wait_st();
                }
                m_ref = new_ref;
                const float nmu = new_ref == -INFINITY ? 0.f : -new_ref;
                // key pairs in paired fp32 arithmetic: 2^(s * sl - m), the
                // row sum in two paired accumulators
                const uint64_t sl2 = f2_pack(sl, sl), nmu2 = f2_pack(nmu, nmu);
                uint64_t ls2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
                auto p_pair = [&](int k, float &a, float &b) {
                    f2_unpack(f2_fma(f2_pack(s[k], s[k + 1]), sl2, nmu2), a, b);
                    a = fast_exp2(a);
                    b = fast_exp2(b);
                };
                if constexpr (kF8) {
                    // one f16 term: keys 2c, 2c+1 -> column c, in place
    #pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pk[16];
    #pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float a, b;
                            p_pair(32 * h + 2 * e, a, b);
                            ls2[e & 1] = f2_add(ls2[e & 1], f2_pack(a, b));
                            pk[e] = pack_f16x2(a, b);
                        }
                        tc::st16(sx + 16 * h, pk);
                    }
                } else {
                    // group g (16 keys) -> 8 columns of P hi then 8 of P lo
    #pragma unroll
                    for (int g = 0; g < kBlocks; ++g) {
                        uint32_t pk[16];
    #pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float a, b;
                            p_pair(16 * g + 2 * e, a, b);
                            const uint64_t ab = f2_pack(a, b);
                            ls2[e & 1] = f2_add(ls2[e & 1], ab);
                            const uint32_t hi = pack_bf16x2(a, b);
                            pk[e] = hi;
                            float ra, rb;
                            f2_unpack(f2_sub(ab, f2_pack(bf16lo_to_f32(hi), bf16hi_to_f32(hi))), ra, rb);
                            pk[8 + e] = pack_bf16x2(ra, rb);
                        }
                        tc::st16(sx + 16 * g, pk);
                    }
                }
                float l0, l1, l2, l3;
                f2_unpack(ls2[0], l0, l1);
                f2_unpack(ls2[1], l2, l3);
                l = l * (resc ? alpha : 1.f) + ((l0 + l1) + (l2 + l3));
            }
            // bf16: V(jj) must have landed before this tile's P.V is issued.  Value
            // rows of keys outside [kv_lo, kv_hi) or of blocks not loaded hold
            // stale slots (possibly NaN): each warpgroup zeroes them before its
            // own P.V reads them (both write the same zeros, so whichever
            // product runs first reads zeros)
            if constexpr (!kF8) {
                const bool landed = mbar_wait(&v_full[ks], (T / kStages) & 1, p.wait_ns);
                if (__any_sync(0xffffffffu, !landed)) {
                    if (lane == 0) report(p.status, PKV_DEV_TIMEOUT);
                    abort = true;
                    break;
                }
            }
            // (FP8: the issuing warp waits for V, whose columns of those keys are zeros)
            const bool edge = !kF8 && (mask != (1u << kBlocks) - 1u ||
                                       (tbase < kv_lo && !(kSink && tbase + kKeys <= p.sinks)) ||
                                       tbase + kKeys > kv_hi);
            if (edge) {
                // thread row r < 64 zeroes key row r's first 64 dims, r >= 64
                // the second 64 dims of key row r - 64
                const int kr = row & (kKeys - 1), half = row >> 6;
                const int32_t kp = tbase + kr;
                if (!((kp >= kv_lo || (kSink && kp < p.sinks)) && kp < kv_hi && ((mask >> (kr >> 4)) & 1u))) {
                    uint8_t *vs = v_s + ks * kTileBytes + half * kKVRegion + kr * 128;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        *reinterpret_cast<uint4 *>(vs + c * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            tc::wait_st();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[x * 2 + buf]);
        }
        if (abort) break;
        const PrefillRowInfo &w = cs.w;
        if (p.drill & kDrillLate) come_late(20000 + 4000 * (warp & 3));
        // the next segment, read while the last product runs
        bool more = false;
        if (lane == 0) {
            SegWalk sw = ss->sw;
            Seg sg;
            more = seg_next<kSink, kTree>(p, qpc, sw, sg);
            if (more) {
                ss->sw = sw;
                ss->sg[(k + 1) & 1] = sg;
            }
        }
        __syncwarp();
        // epilogue: O / l once the segment's last P.V product is in.  A parity
        // names one phase only while no later one can have completed: o_done
        // completes once a segment, and its next phase needs this warp.
        // pv_done alone cannot tell: a warp that comes late finds the last two
        // products done, where a wait for the first of them never ends
        {
            const int32_t Tl = kAlt ? T0 + j0 + ((ntile - 1 - j0) & ~1) : T0 + ntile - 1;  // its last tile
            bool done = mbar_wait(&o_done[x], k & 1, p.wait_ns);
            if (!kAlt || j0 < ntile) done = done && mbar_wait(&pv_done[x], own(Tl) & 1, p.wait_ns);
            // kAlt: tile B's maximum and sum of every row go to tile A's warps
            // through its S columns (free until the next segment's queries are
            // announced, which tile A's warps take part in), which join the two
            // tiles' O as they read them
            float wa = 1.f, wb = 0.f;
            if constexpr (kTree) m_ref = weight_max(m_ref, l);
            if constexpr (kAlt) {
                const uint32_t hand = tS(1, 0) + lane_base;
                if (x == 1 && !__any_sync(0xffffffffu, !done)) {
                    tc::fence_after();
                    uint32_t ml[16] = {__float_as_uint(m_ref), __float_as_uint(l)};
                    tc::st16(hand, ml);
                    tc::wait_st();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sums[0]);
                } else if (x == 0) {
                    done = done && mbar_wait(&sums[0], k & 1, p.wait_ns) && mbar_wait(&o_done[1], k & 1, p.wait_ns);
                    if (!__any_sync(0xffffffffu, !done)) {
                        tc::fence_after();
                        uint32_t ml[32];
                        tc::ld32(hand, ml);
                        tc::wait_ld();
                        const float mb = __uint_as_float(ml[0]), m = fmaxf(m_ref, mb);
                        wa = m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - m);
                        wb = mb == -INFINITY ? 0.f : fast_exp2(mb - m);
                        l = wa * l + wb * __uint_as_float(ml[1]);
                        m_ref = m;
                    }
                }
            }
            // 32 dims of the row's O, not yet divided (a tile without weight may hold anything)
            const auto load_o = [&](int c, uint32_t (&r32)[32]) {
                tc::ld32(ox + c * 32, r32);
                if constexpr (kAlt) {
                    uint32_t b32[32];
                    tc::ld32(ox + 128 + c * 32, b32);
                    tc::wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float a = wa > 0.f ? wa * __uint_as_float(r32[e]) : 0.f;
                        r32[e] = __float_as_uint(wb > 0.f ? fmaf(wb, __uint_as_float(b32[e]), a) : a);
                    }
                } else {
                    tc::wait_ld();
                }
            };
            if (__any_sync(0xffffffffu, !done)) {
                if (lane == 0) report(p.status, PKV_DEV_TIMEOUT);
                break;
            } else if (kAlt && x == 1) {
                // tile A's warps write the rows
            } else if (p.sk_ctas > 0 && !cs.whole) {
                // a piece of an item cut by this CTA's run: a partial in the
                // CTA's slot (first or last segment), merged afterwards.  Each
                // warp's 32 rows lie dim-group major (float4 d4 of row `lane`
                // at d4 * 32 + lane), so that every access below is 512
                // consecutive bytes a warp (with rows contiguous a merge of two
                // or three pieces took 20 us)
                tc::fence_after();
                const auto piece_at = [&](int32_t c, int32_t slot) {
                    return ((static_cast<size_t>(c) * 2 + slot) * kQTiles + x) * 4 + (warp & 3);
                };
                const size_t own = piece_at(blockIdx.x, cs.slot);
                float4 *dst = reinterpret_cast<float4 *>(p.sk_o) + own * (32 * kD / 4) + lane;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t r32[32];
                    load_o(c, r32);
                    const float vs = kF8 ? p.v_scale : 1.f;
                    if (kTree && !valid_row) continue;  // (a tree's merge reads its rows alone)
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        dst[(c * 8 + v) * 32] = make_float4(__uint_as_float(r32[4 * v]) * vs, __uint_as_float(r32[4 * v + 1]) * vs,
                                                            __uint_as_float(r32[4 * v + 2]) * vs, __uint_as_float(r32[4 * v + 3]) * vs);
                }
                if (!kTree || valid_row)
                    reinterpret_cast<float2 *>(p.sk_ml)[own * 32 + lane] = make_float2(m_ref, l);
                if constexpr (!kTree) {
                // the item's pieces: CTAs cf .. cl; per (query tile, warp) the
                // warp whose piece completes last merges their 32 rows (no
                // waiting: the others published theirs before counting)
                __syncwarp();
                const int32_t cf = cs.cf, cl = cs.cl;
                // CTAs between them may have empty runs
                const auto piece_from = [&](int32_t c) {
                    while (c < cl && sk_run_start(p, c + 1) == sk_run_start(p, c)) ++c;
                    return c;
                };
                int last = 0;
                if (lane == 0) {
                    int others = 0;
                    for (int32_t c = cf; c < cl; ++c) others += sk_run_start(p, c + 1) > sk_run_start(p, c) ? 1 : 0;
                    __threadfence();
                    const int old = atomicAdd(p.sk_count + (cf * 2 + x) * 4 + (warp & 3), 1);
                    last = old == others;
                    if (last) __threadfence();
                }
                last = __shfl_sync(0xffffffffu, last, 0);
                if (last) {
                    // slot 1: the item is not c's first segment
                    const int32_t slot_f = sk_run_start(p, cf) < cs.lo ? 1 : 0;
                    const auto piece = [&](int32_t c) { return piece_at(c, c == cf ? slot_f : 0); };
                    const float2 *ml = reinterpret_cast<const float2 *>(p.sk_ml) + lane;
                    const float4 *po = reinterpret_cast<const float4 *>(p.sk_o) + lane;
                    float M = -INFINITY, lsum = 0.f;
                    for (int32_t c = cf; c <= cl; c = piece_from(c + 1)) M = fmaxf(M, __ldcg(ml + piece(c) * 32).x);
                    // a piece without weight (nothing seen) takes the factor 0
                    const auto weight = [&](float m) { return m == -INFINITY ? 0.f : fast_exp2(m - M); };
                    for (int32_t c = cf; c <= cl; c = piece_from(c + 1)) {
                        const float2 v = __ldcg(ml + piece(c) * 32);
                        lsum = fmaf(weight(v.x), v.y, lsum);
                    }
                    const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out) +
                                 ((static_cast<int64_t>(w.q0) + t) * p.hq +
                                  w.g * G + row % G) * (kD / 8);
                    // 32 dims at a time, two pieces' loads in flight
#pragma unroll 1
                    for (int d0 = 0; d0 < kD; d0 += 32) {
                        float acc[32];
#pragma unroll
                        for (int d = 0; d < 32; ++d) acc[d] = 0.f;
#pragma unroll 1
                        for (int32_t c = cf; c <= cl;) {
                            const int32_t c1 = c < cl ? piece_from(c + 1) : c;  // (the last piece alone: loaded twice)
                            const size_t p0 = piece(c), p1 = piece(c1);
                            float4 o0[8], o1[8];
#pragma unroll
                            for (int v = 0; v < 8; ++v) o0[v] = __ldcg(po + p0 * (32 * kD / 4) + (d0 / 4 + v) * 32);
#pragma unroll
                            for (int v = 0; v < 8; ++v) o1[v] = __ldcg(po + p1 * (32 * kD / 4) + (d0 / 4 + v) * 32);
                            const float w0 = weight(__ldcg(ml + p0 * 32).x);
                            const float w1 = c1 > c ? weight(__ldcg(ml + p1 * 32).x) : 0.f;
                            c = c1 < cl ? piece_from(c1 + 1) : cl + 1;
                            const auto add = [&](float wgt, const float4 (&o)[8]) {
                                if (wgt == 0.f) return;  // (a piece that saw nothing)
#pragma unroll
                                for (int v = 0; v < 8; ++v) {
                                    acc[4 * v] = fmaf(wgt, o[v].x, acc[4 * v]);
                                    acc[4 * v + 1] = fmaf(wgt, o[v].y, acc[4 * v + 1]);
                                    acc[4 * v + 2] = fmaf(wgt, o[v].z, acc[4 * v + 2]);
                                    acc[4 * v + 3] = fmaf(wgt, o[v].w, acc[4 * v + 3]);
                                }
                            };
                            add(w0, o0);
                            add(w1, o1);
                        }
                        if (valid_row) {
#pragma unroll
                            for (int v = 0; v < 4; ++v) {
                                uint4 o;
                                o.x = pack_bf16x2(acc[8 * v + 0] * inv, acc[8 * v + 1] * inv);
                                o.y = pack_bf16x2(acc[8 * v + 2] * inv, acc[8 * v + 3] * inv);
                                o.z = pack_bf16x2(acc[8 * v + 4] * inv, acc[8 * v + 5] * inv);
                                o.w = pack_bf16x2(acc[8 * v + 6] * inv, acc[8 * v + 7] * inv);
                                dst[d0 / 8 + v] = o;
                            }
                        }
                    }
                }
                }
            } else if (split) {
                // a partial: O unnormalised with its reference max and sum
                tc::fence_after();
                const size_t pi = ((static_cast<size_t>(w.r) * p.max_q_len + w.i0 + t) * p.hq +
                                   w.g * G + row % G) * p.kv_splits + w.s;
                float4 *dst = reinterpret_cast<float4 *>(p.ws_o + pi * kD);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t r32[32];
                    load_o(c, r32);
                    if (valid_row) {
                        const float vs = kF8 ? p.v_scale : 1.f;
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            dst[c * 8 + v] = make_float4(__uint_as_float(r32[4 * v]) * vs, __uint_as_float(r32[4 * v + 1]) * vs,
                                                         __uint_as_float(r32[4 * v + 2]) * vs, __uint_as_float(r32[4 * v + 3]) * vs);
                    }
                }
                if (valid_row) *reinterpret_cast<float2 *>(p.ws_ml + pi * 2) = make_float2(m_ref, l);
            } else {
                tc::fence_after();
                // (kTree: NaN stays NaN)
                const float inv = ((kTree ? l != 0.f : l > 0.f) ? 1.f / l : 0.f) * (kF8 ? p.v_scale : 1.f);
                // the warp's rows go through its part of the query tile, which
                // every product of the segment has read: 16-byte chunks
                // swizzled by the row, then whole rows to global memory
                uint8_t *stage = q_s + x * kQBytes + 32 * (warp & 3) * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t r32[32];
                    load_o(c, r32);
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint4 o;
                        o.x = pack_bf16x2(__uint_as_float(r32[8 * v + 0]) * inv, __uint_as_float(r32[8 * v + 1]) * inv);
                        o.y = pack_bf16x2(__uint_as_float(r32[8 * v + 2]) * inv, __uint_as_float(r32[8 * v + 3]) * inv);
                        o.z = pack_bf16x2(__uint_as_float(r32[8 * v + 4]) * inv, __uint_as_float(r32[8 * v + 5]) * inv);
                        o.w = pack_bf16x2(__uint_as_float(r32[8 * v + 6]) * inv, __uint_as_float(r32[8 * v + 7]) * inv);
                        const int ch = c * 4 + v;  // dims 8ch .. 8ch + 7
                        *reinterpret_cast<uint4 *>(stage + (ch >> 3) * (kRows * 128) + lane * 128 +
                                                   (((ch & 7) ^ (lane & 7)) << 4)) = o;
                    }
                }
                __syncwarp();
                const int ch = lane & 15;
                uint4 *dst = reinterpret_cast<uint4 *>(p.out) +
                             (static_cast<int64_t>(w.q0) * p.hq + w.g * G) * (kD / 8) + ch;
#pragma unroll 4
                for (int k = 0; k < 16; ++k) {
                    const int rr = 2 * k + (lane >> 4), i = 32 * (warp & 3) + rr;  // row of the warp, of the tile
                    const int tq = x * qpt + (i >> glog), h = i & (G - 1);
                    const uint4 o = *reinterpret_cast<const uint4 *>(stage + (ch >> 3) * (kRows * 128) + rr * 128 +
                                                                     (((ch & 7) ^ (rr & 7)) << 4));
                    if (tq < w.nq) dst[(static_cast<int64_t>(tq) * p.hq + h) * (kD / 8)] = o;
                }
                __syncwarp();  // the rows are read before the next query tile lands there
            }
        }
        // the next segment: its query tile replaces this one once every
        // product that read it has completed (the waits above)
        tc::fence_before();
        T0 += ntile;
        more = __shfl_sync(0xffffffffu, more, 0);
        __syncwarp();
        if (!more) break;
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after();
        tc::dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// f32, CUDA cores: 16 (query, head) pairs per CTA
// ---------------------------------------------------------------------------
constexpr int kPf32Threads = 128;
constexpr int kPf32Pairs = 16;

__global__ void __launch_bounds__(kPf32Threads) prefill_f32_kernel(const PrefillParams p)
{
    constexpr int NQ = kPf32Pairs;
    extern __shared__ float fsm[];
    const int D = p.head_dim, bs = p.block_size, G = p.group;
    const int qpt = NQ / G;
    float *qs = fsm, *os = qs + NQ * D, *ks = os + NQ * D, *vs = ks + bs * D, *sc = vs + bs * D;
    float *mrow = sc + NQ * bs, *lrow = mrow + NQ, *alpha = lrow + NQ;
    int32_t *phi = reinterpret_cast<int32_t *>(alpha + NQ), *plo = phi + NQ;
    uint64_t *tm = reinterpret_cast<uint64_t *>(plo + NQ);  // drafted trees: the rows' masks (an even word)
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    PrefillRowInfo w;
    if (!prefill_item(p, blockIdx.x, qpt, w)) return;
    const int32_t row0 = w.q0, first = w.kv_hi - w.nq - w.i0;
    if (tid < NQ) {
        const int t = tid / G;
        const bool valid = tid < qpt * G && t < w.nq;
        const int32_t qpos = w.kv_hi - w.nq + t;
        phi[tid] = valid ? qpos + 1 : 0;
        int32_t at = qpos;  // where its window ends
        if (p.tree != nullptr) {
            tm[tid] = valid ? tree_mask(p.tree, w.q0 + t, w.i0 + t) : 0ull;
            at = qpos - (w.i0 + t) + tree_depth(tm[tid]);
        }
        plo[tid] = p.window > 0 ? max(0, at - p.window + 1) : 0;
        mrow[tid] = -INFINITY;
        lrow[tid] = 0.f;
    }
    const float *qg = static_cast<const float *>(p.q);
    for (int i = tid; i < NQ * D; i += kPf32Threads) {
        const int k = i / D, d = i % D, t = k / G, h = k % G;
        const bool valid = k < qpt * G && t < w.nq;
        qs[i] = valid ? qg[(static_cast<int64_t>(row0 + t) * p.hq + w.g * G + h) * D + d] : 0.f;
        os[i] = 0.f;
    }
    __syncthreads();
    const float *kpool = static_cast<const float *>(p.k_pool);
    const float *vpool = static_cast<const float *>(p.v_pool);
    const int32_t *trow = p.tables + static_cast<int64_t>(w.r) * p.width;
    // the sink blocks before the window's first block, then the window's
    const int32_t b_win = w.kv_lo / bs;
    const int32_t nsb = p.sinks > 0 ? min((min(p.sinks, w.kv_lo) + bs - 1) / bs, b_win) : 0;
    const int32_t sink = p.sinks;
    for (int32_t b = nsb > 0 ? 0 : b_win; b * bs < w.kv_hi; b = b + 1 == nsb ? b_win : b + 1) {
        const int32_t blk = b < p.width ? __ldg(trow + b) : -1;
        const bool ok = static_cast<uint32_t>(blk) < static_cast<uint32_t>(p.num_blocks);
        if (!ok && tid == 0) report(p.status, PKV_DEV_BAD_BLOCK);
        if (ok) {
            const int64_t base = (static_cast<int64_t>(blk) * p.hkv + w.g) * bs * D;
            for (int j = tid; j < bs * D; j += kPf32Threads) {
                ks[j] = __ldg(kpool + base + j);
                vs[j] = __ldg(vpool + base + j);
            }
        }
        __syncthreads();
        for (int j = tid; j < NQ * bs; j += kPf32Threads) {
            const int k = j / bs, tt = j % bs;
            const int pos = b * bs + tt;
            float sv = -INFINITY;
            const int dr = pos - first;  // a tree's draft (< 0: a cached token)
            if (ok && (pos >= plo[k] || pos < sink) && pos < phi[k] &&
                (p.tree == nullptr || dr < 0 || ((tm[k] >> dr) & 1u))) {
                float acc = 0.f;
                for (int d = 0; d < D; ++d) acc = fmaf(qs[k * D + d], ks[tt * D + d], acc);
                sv = acc * p.scale_log2;
            }
            sc[j] = sv;
        }
        __syncthreads();
        if (tid < NQ) {
            float mx = -INFINITY;
            for (int tt = 0; tt < bs; ++tt) mx = fmaxf(mx, sc[tid * bs + tt]);
            const float mn = fmaxf(mrow[tid], mx);
            const float mu = mn == -INFINITY ? 0.f : mn;
            const float al = fast_exp2(mrow[tid] - mu);
            float sum = 0.f;
            for (int tt = 0; tt < bs; ++tt) {
                const float e = fast_exp2(sc[tid * bs + tt] - mu);
                sc[tid * bs + tt] = e;
                sum += e;
            }
            lrow[tid] = lrow[tid] * al + sum;
            mrow[tid] = mn;
            alpha[tid] = al;
        }
        __syncthreads();
        for (int j = tid; j < NQ * D; j += kPf32Threads) {
            const int k = j / D, d = j % D;
            float acc = os[j] * alpha[k];
            for (int tt = 0; tt < bs; ++tt) {
                const float wv = sc[k * bs + tt];
                if (wv != 0.f) acc = fmaf(wv, vs[tt * D + d], acc);  // masked slots may hold NaN
            }
            os[j] = acc;
        }
        __syncthreads();
    }
    float *og = static_cast<float *>(p.out);
    for (int j = tid; j < NQ * D; j += kPf32Threads) {
        const int k = j / D, d = j % D, t = k / G, h = k % G;
        if (k >= qpt * G || t >= w.nq) continue;
        const float l = lrow[k];
        og[(static_cast<int64_t>(row0 + t) * p.hq + w.g * G + h) * D + d] = l != 0.f ? os[j] / l : 0.f;  // (NaN stays NaN)
    }
}

// ---------------------------------------------------------------------------
// merge of the key-range runs (bf16, short chunks): one warp per (row, query
// of the chunk, q head).  M = max of the runs' reference maxima; each run is
// weighted by 2^(m_s - M); out = sum w_s O_s / sum w_s l_s.
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 8;

__global__ void __launch_bounds__(kMergeWarps * 32) prefill_merge_kernel(const PrefillParams p)
{
    constexpr int D = pf::kD;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kMergeWarps + warp;
    const int64_t total = static_cast<int64_t>(p.batch) * p.max_q_len * p.hq;
    if (item >= total) return;
    const int32_t h = static_cast<int32_t>(item % p.hq);
    const int64_t ri = item / p.hq;
    const int32_t i = static_cast<int32_t>(ri % p.max_q_len);
    const int32_t r = static_cast<int32_t>(ri / p.max_q_len);
    // the chunk length as the prefill kernel clamps it (call inputs: final
    // before the wait, as the prefill kernel waited on earlier work itself)
    const int32_t c0 = __ldg(p.cu_q_lens + r), c1 = __ldg(p.cu_q_lens + r + 1);
    int32_t C = c1 - c0;
    int32_t L = __ldg(p.seq_lens + r);
    L = L < 0 ? 0 : (L > p.max_len ? p.max_len : L);
    if (c0 < 0 || C < 0 || C > p.max_q_len || C > L)
        C = c0 < 0 || C < 0 ? 0 : min(min(C, p.max_q_len), L);
    if (i >= C) return;
    pdl_wait();  // the partials come from the prefill kernel just before
    const size_t base = ((static_cast<size_t>(r) * p.max_q_len + i) * p.hq + h) * p.kv_splits;
    float M = -INFINITY;
    for (int32_t s = 0; s < p.kv_splits; ++s) M = fmaxf(M, p.ws_ml[(base + s) * 2]);
    float acc[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
    float lsum = 0.f;
    if (M != -INFINITY) {
        for (int32_t s = 0; s < p.kv_splits; ++s) {
            const float2 ml = *reinterpret_cast<const float2 *>(p.ws_ml + (base + s) * 2);
            if (ml.x == -INFINITY) continue;  // an empty run wrote no values
            const float wgt = fast_exp2(ml.x - M);
            lsum = fmaf(wgt, ml.y, lsum);
            const float *src = p.ws_o + (base + s) * D + lane;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(wgt, src[32 * e], acc[e]);
        }
    }
    const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) +
                         (static_cast<size_t>(c0 + i) * p.hq + h) * D + lane;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) out[32 * e] = __float2bfloat16_rn(acc[e] * inv);
}

// Drafted trees: joins the pieces of the item that CTA x's run begins and does not
// end (CTAs (x, ..)); a thread has 16 dims of a (query, head) pair.
constexpr int kTreeMergeThreads = 256;
__global__ void __launch_bounds__(kTreeMergeThreads) prefill_tree_merge_kernel(const PrefillParams p, int32_t rows)
{
    pdl_wait();  // the records and partials come from the kernel just before
    pdl_trigger();
    constexpr int kD = pf::kD;
    const int32_t c = blockIdx.x, idx = blockIdx.y * kTreeMergeThreads + threadIdx.x;
    const TreeRecord rec = static_cast<const TreeRecord *>(p.sk_rec)[c];
    const int32_t row = idx % rows, d4 = idx / rows * 4;  // rows: of an item, at most
    if (row >= rec.rows || d4 * 4 >= kD) return;          // (no item: no rows)
    // a piece's warp of 32 rows
    const auto at = [&](int32_t i) {
        return (static_cast<size_t>(c + i) * 2 + (i == 0 ? rec.slot : 0)) * (pf::kQTiles * 4) + (row >> 5);
    };
    float4 acc[4];
    const float l = join_pieces(
        rec.pieces, 32,
        [&](int32_t i) -> const float4 * {
            return reinterpret_cast<const float4 *>(p.sk_o) + at(i) * (32 * kD / 4) + d4 * 32 + (row & 31);
        },
        [&](int32_t i) { return reinterpret_cast<const float2 *>(p.sk_ml)[at(i) * 32 + (row & 31)]; }, acc);
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) +
                         ((static_cast<int64_t>(rec.q0) + row / p.group) * p.hq + rec.g * p.group + row % p.group) * kD + d4 * 4;
    store_bf16x16(out, acc, l != 0.f ? 1.f / l : 0.f);  // (NaN stays NaN)
}

// ---------------------------------------------------------------------------
// persistent balanced schedule: the plan (the items' records, the CTAs' whole
// items and runs, the cut items' arrival counters zeroed), one CTA
// ---------------------------------------------------------------------------
constexpr int kSkPlanThreads = 1024;
constexpr int kSkMaxCtas = 512;
// What an item costs a CTA beside its tiles, in tiles (its query tile staged, the
// first products, the epilogue: about 7 us against 1.2 a tile), and the fewest
// tiles worth a cut (a piece's partial is written and merged).  Against 0 and 1:
// 8 ragged chunks on FP8 pools (16/4 heads, window 1000) 87.7 -> 73.4 us, 4
// chunks of 512 with a window of 512 61.8 -> 51.0 (bf16), 2 chunks of 4096 with
// one of 4096 470 -> 465; 4 to 8 and 2 to 4 lie within 5 % of each other.
constexpr int32_t kSkItemCost = 6;
constexpr int32_t kSkLeastPiece = 4;
static_assert(kTreeOver <= kSkItemCost, "prefill_sk_counts holds for the runs of trees");

__global__ void __launch_bounds__(kSkPlanThreads) prefill_sk_plan_kernel(const PrefillParams p)
{
    constexpr int kWarps = kSkPlanThreads / 32;
    __shared__ int32_t warp_sum[kWarps], warp_cnt[kWarps], warp_first[kWarps];
    __shared__ int32_t carry, carry_cnt, after, whole_cost;
    __shared__ int32_t whole[kSkMaxCtas], cost[kSkMaxCtas], run[kSkMaxCtas + 1], run_item[kSkMaxCtas];
    __shared__ int32_t run_cost[kSkMaxCtas + 1];  // the runs' starts, each item counted kSkItemCost longer
    pdl_wait();  // lengths may come from the previous kernel on the stream
    pdl_trigger();
    const int qpc = pf::kQTiles * (pf::kRows / p.group);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t ctas = p.sk_ctas;
    SkItem *rec = reinterpret_cast<SkItem *>(p.sk_rec);
    if (threadIdx.x == 0) {
        carry = carry_cnt = 0;
        after = p.sk_items;
    }
    for (int32_t i = threadIdx.x; i < ctas; i += kSkPlanThreads) {
        whole[i] = -1;
        cost[i] = 0;
        run_item[i] = 0;
    }
    for (int32_t i = threadIdx.x; i < ctas * 8; i += kSkPlanThreads) p.sk_count[i] = 0;
    __syncthreads();
    // this thread's item of the first kSkPlanThreads stays in registers, later
    // ones are read back
    int32_t lo0 = 0, hi0 = 0, rank0 = 0;
    for (int32_t base = 0; base < p.sk_items; base += kSkPlanThreads) {
        const int32_t u = base + threadIdx.x;
        int32_t n = 0;
        PrefillRowInfo w;
        if (u < p.sk_items && prefill_item(p, u, qpc, w)) n = item_tiles(w);
        // inclusive scans of the tiles and of the items with tiles: within the
        // warp, then over the warps' sums
        const uint32_t has = __ballot_sync(0xffffffffu, n > 0);
        int32_t v = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += o;
        }
        if (lane == 31) {
            warp_sum[warp] = v;
            warp_cnt[warp] = __popc(has);
        }
        __syncthreads();
        if (warp == 0) {
            int32_t ws = warp_sum[lane], wc = warp_cnt[lane];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t o = __shfl_up_sync(0xffffffffu, ws, d), oc = __shfl_up_sync(0xffffffffu, wc, d);
                if (lane >= d) {
                    ws += o;
                    wc += oc;
                }
            }
            warp_sum[lane] = ws;  // inclusive over the warps
            warp_cnt[lane] = wc;
        }
        __syncthreads();
        const int32_t incl = v + (warp > 0 ? warp_sum[warp - 1] : 0) + carry;
        const int32_t rank = __popc(has & ((1u << lane) - 1u)) + (warp > 0 ? warp_cnt[warp - 1] : 0) + carry_cnt;
        if (u < p.sk_items) {
            if (n > 0) rec[u].w = w;
            rec[u].lo = incl - n;
            rec[u].hi = incl;
            rec[u].next = rank;  // until the next items are known
            if (base == 0) {
                lo0 = incl - n;
                hi0 = incl;
                rank0 = rank;
            }
            if (n > 0 && rank < ctas) {
                whole[rank] = u;
                cost[rank] = n + kSkItemCost;
            }
        }
        __syncthreads();
        if (threadIdx.x == kSkPlanThreads - 1) {
            carry = incl;
            carry_cnt += warp_cnt[kWarps - 1];
        }
        __syncthreads();
    }
    // the runs: the least level at which the CTAs take the cost R that is left
    const int32_t W = carry + carry_cnt * kSkItemCost;
    if (warp == 0) {
        int32_t B = 0, most = 0;
        for (int32_t c = lane; c < ctas; c += 32) {
            B += cost[c];
            most = max(most, cost[c]);
        }
        B = __reduce_add_sync(0xffffffffu, B);
        most = __reduce_max_sync(0xffffffffu, most);
        const int32_t R = W - B;
        // room(level) >= ctas * level - B, with equality while no whole item
        // passes the level: the even level is enough, and exact when it holds
        // every whole item (all costs together stay below 2^31: prefill_sk_counts)
        const auto room = [&](int32_t level) {
            int32_t sum = 0;
            for (int32_t c = lane; c < ctas; c += 32) sum += max(0, level - cost[c]);
            return static_cast<int32_t>(__reduce_add_sync(0xffffffffu, sum));
        };
        int32_t lo = 0, hi = (W + ctas - 1) / ctas;
        if (most <= hi) lo = hi;
        while (lo < hi) {
            const int32_t mid = (lo + hi) >> 1;
            if (room(mid) >= R) hi = mid; else lo = mid + 1;
        }
        int32_t before = 0;  // room of the CTAs before this group of 32
        for (int32_t c0 = 0; c0 < ctas; c0 += 32) {
            const int32_t c = c0 + lane;
            int32_t v = c < ctas ? max(0, lo - cost[c]) : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t o = __shfl_up_sync(0xffffffffu, v, d);
                if (lane >= d) v += o;
            }
            if (c < ctas) run_cost[c + 1] = before + v;
            before += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) {
            run_cost[0] = 0;
            whole_cost = B;
        }
    }
    __syncthreads();
    // the rooms' running sums to costs, in proportion (the last one last)
    const int64_t room_all = run_cost[ctas], R = W - whole_cost;
    __syncthreads();
    for (int32_t c = threadIdx.x; c <= ctas; c += kSkPlanThreads) {
        run_cost[c] = static_cast<int32_t>(whole_cost + (room_all > 0 ? R * run_cost[c] / room_all : 0));
        run[c] = carry;  // a run past the last item
    }
    __syncthreads();
    // the runs' starts in tiles: the item whose cost holds a start places it, on
    // its end where fewer than kSkLeastPiece tiles would lie on one side
    for (int32_t u = threadIdx.x; u < p.sk_items; u += kSkPlanThreads) {  // this thread's own writes above
        const bool mine = u < kSkPlanThreads;
        const int32_t tlo = mine ? lo0 : rec[u].lo, n = (mine ? hi0 : rec[u].hi) - tlo;
        const int32_t clo = tlo + (mine ? rank0 : rec[u].next) * kSkItemCost, chi = clo + n + kSkItemCost;
        if (n == 0 || chi <= run_cost[0]) continue;
        int32_t a = -1, b = ctas + 1;  // the last c with run_cost[c] < clo, the first past it
        while (b - a > 1) {
            const int32_t mid = (a + b) >> 1;
            if (run_cost[mid] < clo) a = mid; else b = mid;
        }
        for (int32_t c = b; c <= ctas && run_cost[c] < chi; ++c) {
            const int32_t at = run_cost[c] - clo;
            run[c] = tlo + (at < kSkLeastPiece ? 0 : n - at < kSkLeastPiece ? n : at);
        }
    }
    __syncthreads();
    // each item's next one with tiles, from the last run of threads to the
    // first; the CTAs that hold its tiles; the item at each run's start
    for (int32_t base = (p.sk_items - 1) / kSkPlanThreads * kSkPlanThreads; base >= 0; base -= kSkPlanThreads) {
        const int32_t u = base + threadIdx.x;
        int32_t lo = 0, hi = 0;
        if (base == 0) {
            lo = lo0;
            hi = hi0;
        } else if (u < p.sk_items) {  // this thread's own writes above
            lo = rec[u].lo;
            hi = rec[u].hi;
        }
        const uint32_t m = __ballot_sync(0xffffffffu, hi > lo);
        if (lane == 0) warp_first[warp] = m != 0 ? base + warp * 32 + __ffs(m) - 1 : -1;
        __syncthreads();
        const uint32_t rest = lane < 31 ? m >> (lane + 1) : 0u;
        int32_t next = rest != 0 ? u + __ffs(rest) : -1;
        for (int i = warp + 1; next < 0 && i < kWarps; ++i) next = warp_first[i];
        if (next < 0) next = after;
        if (u < p.sk_items) {
            int32_t cf = 0, cl = 0;
            if (hi > lo && hi > run[0]) {
                const auto cta_of = [&](int32_t pos) {  // the last c with run[c] <= pos: its run holds pos
                    int32_t a = 0, b = ctas;
                    while (b - a > 1) {
                        const int32_t mid = (a + b) >> 1;
                        if (run[mid] <= pos) a = mid; else b = mid;
                    }
                    return a;
                };
                cf = cta_of(lo);
                cl = cta_of(hi - 1);
                // the runs that start inside this item
                for (int32_t c = run[cf] >= lo ? cf : cf + 1; c <= cl; ++c) run_item[c] = u;
                for (int32_t c = cf; c >= 0 && run[c] >= lo; --c) run_item[c] = u;
            }
            rec[u].next = next;
            rec[u].cf = cf;
            rec[u].cl = cl;
        }
        int32_t first = -1;
        if (threadIdx.x == 0)
            for (int i = 0; first < 0 && i < kWarps; ++i) first = warp_first[i];
        __syncthreads();
        if (threadIdx.x == 0 && first >= 0) after = first;
        __syncthreads();
    }
    for (int32_t c = threadIdx.x; c <= ctas; c += kSkPlanThreads) {
        p.sk_plan[c] = run[c];
        if (c < ctas) {
            p.sk_plan[ctas + 1 + c] = run_item[c];
            p.sk_plan[2 * ctas + 1 + c] = whole[c];
        }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
bool prefill_shape_built(pkv_dtype dtype, int32_t D, int32_t bs, int32_t G)
{
    if (G < 1 || G > 16) return false;
    if (dtype == PKV_BF16 || dtype == PKV_FP8_E4M3) return D == pf::kD && bs == 16 && (pf::kRows % G) == 0;
    return (D == 32 || D == 64 || D == 128 || D == 256) && bs <= 64 && bs * D <= 4096 &&
           (kPf32Pairs % G) == 0;
}

int32_t prefill_queries_per_cta(pkv_dtype dtype, int32_t G)
{
    return dtype != PKV_F32 ? pf::kQTiles * (pf::kRows / G) : kPf32Pairs / G;
}

PrefillSplit prefill_split_plan(int32_t batch, int32_t hq, int32_t hkv, int32_t D, int32_t bs,
                                int32_t max_q_len, int32_t max_seq_len, int32_t window, int32_t sinks,
                                int num_sms)
{
    PrefillSplit sp{1, 0};
    if (hkv <= 0 || hq % hkv != 0 || batch <= 0 || max_q_len <= 0) return sp;
    const int32_t G = hq / hkv;
    if (D != pf::kD || bs != 16 || G < 1 || pf::kRows % G != 0) return sp;
    if (max_q_len > pf::kRows / G) return sp;  // chunks that need both query tiles: no split
    const int64_t ctas = static_cast<int64_t>(batch) * hkv;
    const int64_t keys = window > 0 ? std::min<int64_t>(max_seq_len, static_cast<int64_t>(window) + max_q_len)
                                    : max_seq_len;
    // +1: a CTA's range may start inside a tile
    int64_t tiles = (keys + pf::kKeys - 1) / pf::kKeys + 1;
    if (sinks > 0) tiles += (static_cast<int64_t>(std::min(sinks, max_seq_len)) + pf::kKeys - 1) / pf::kKeys;
    // about four CTAs per SM over the grid, at least 8 tiles (512 keys) per run
    int64_t s = (4ll * std::max(num_sms, 1) + ctas - 1) / ctas;
    s = std::min<int64_t>(s, tiles / 8);
    s = std::max<int64_t>(1, std::min<int64_t>(s, 32));
    if (s == 1) return sp;
    sp.splits = static_cast<int32_t>(s);
    sp.tiles = static_cast<int32_t>((tiles + s - 1) / s);
    return sp;
}

int32_t prefill_sk_ctas(pkv_dtype dtype, int32_t batch, int32_t hq, int32_t hkv, int32_t D, int32_t bs,
                        int32_t max_q_len, int num_sms)
{
    if (dtype == PKV_F32 || hkv <= 0 || hq % hkv != 0 || batch <= 0 || max_q_len <= 0 || num_sms <= 0)
        return 0;
    const int32_t G = hq / hkv;
    if (D != pf::kD || bs != 16 || G < 1 || pf::kRows % G != 0) return 0;
    if (max_q_len <= pf::kRows / G) return 0;  // one query tile: the key-range runs serve it
    const int64_t qpc = static_cast<int64_t>(pf::kQTiles) * (pf::kRows / G);
    const int64_t items = static_cast<int64_t>(batch) * hkv * ((max_q_len + qpc - 1) / qpc);
    // more items than SMs (else one wave of one CTA per item already fits),
    // and a plan the one-CTA plan kernel scans quickly
    if (items <= num_sms || items > 65536 || num_sms > kSkMaxCtas) return 0;
    return num_sms;
}

bool prefill_sk_counts(int32_t items, int32_t max_q_len, int32_t group, int32_t max_len, int32_t window,
                       int32_t sinks)
{
    const int64_t qpc = pf::kQTiles * (pf::kRows / group);
    int64_t tiles = (static_cast<int64_t>(max_len) + pf::kKeys - 1) / pf::kKeys;
    if (window > 0) {
        // the window of the item's first query to its last one, and the sinks' tiles
        const int64_t keys = static_cast<int64_t>(window) - 1 + std::min<int64_t>(qpc, max_q_len);
        tiles = std::min(tiles, (keys + 2 * pf::kKeys - 2) / pf::kKeys +
                                    (static_cast<int64_t>(sinks) + pf::kKeys - 1) / pf::kKeys);
    }
    return items * (tiles + kSkItemCost) <= INT32_MAX - (1 << 20);  // the margin: sums round up per CTA
}

int32_t prefill_tree_ctas(int32_t items, int num_sms) { return items > 0 && items <= 65536 ? num_sms : 0; }

// the records, the pieces' values, their maxima and sums
PrefillTreeWs prefill_tree_ws(int32_t ctas)
{
    const size_t rows = static_cast<size_t>(ctas) * 2 * pf::kQTiles * pf::kRows;
    PrefillTreeWs w{};
    w.o = (static_cast<size_t>(ctas) * kTreeRecordBytes + 255) & ~static_cast<size_t>(255);
    w.ml = w.o + rows * pf::kD * sizeof(float);
    w.bytes = w.ml + rows * 2 * sizeof(float);
    return w;
}

size_t prefill_sk_ws_bytes(int32_t items, int32_t ctas)
{
    if (ctas <= 0) return 0;
    const size_t pre = ((static_cast<size_t>(ctas) * 3 * sizeof(int32_t) + 4 + 255) & ~static_cast<size_t>(255)) +
                       ((static_cast<size_t>(items) * kSkItemBytes + 255) & ~static_cast<size_t>(255)) +
                       ((static_cast<size_t>(ctas) * 8 * sizeof(int32_t) + 255) & ~static_cast<size_t>(255));
    const size_t rows = static_cast<size_t>(ctas) * 2 * pf::kQTiles * pf::kRows;
    const size_t o = (rows * pf::kD * sizeof(float) + 255) & ~static_cast<size_t>(255);
    return pre + o + rows * 2 * sizeof(float);
}

size_t prefill_split_ws_bytes(int32_t batch, int32_t hq, int32_t max_q_len, const PrefillSplit &sp)
{
    if (sp.splits <= 1) return 0;
    const size_t n = static_cast<size_t>(batch) * max_q_len * hq * sp.splits;
    const size_t o = (n * pf::kD * sizeof(float) + 255) & ~static_cast<size_t>(255);
    return o + n * 2 * sizeof(float);
}

template <bool kF8, bool kSink, bool kTree = false, bool kAlt = false>
static cudaError_t launch_prefill_tc(const PrefillParams &p, const CUtensorMap &kmap,
                                    const CUtensorMap &vmap, cudaStream_t stream)
{
    const int64_t ctas = p.sk_ctas > 0 ? p.sk_ctas
                                       : static_cast<int64_t>(p.batch) * p.hkv * p.q_tiles * p.kv_splits;
    if (ctas == 0) return cudaSuccess;
    constexpr int smem = pf::Layout<kF8, kAlt>::kLaunchBytes;
    cudaError_t err = kernel_smem<prefill_kernel<kF8, kSink, kTree, kAlt>>(smem);
    if (err != cudaSuccess) return err;
    prof_begin(PKV_KERNEL_PREFILL, stream);
    if (p.sk_ctas > 0 && !kTree)
        err = launch_pdl(prefill_sk_plan_kernel, dim3(1), dim3(kSkPlanThreads), 0, stream, p);
    if (err == cudaSuccess)
        err = launch_pdl(prefill_kernel<kF8, kSink, kTree, kAlt>, dim3(static_cast<unsigned>(ctas)), dim3(pf::kThreads), smem,
                         stream, kmap, vmap, p);
    if (err == cudaSuccess && p.kv_splits > 1) {
        const int64_t items = static_cast<int64_t>(p.batch) * p.max_q_len * p.hq;
        err = launch_pdl(prefill_merge_kernel,
                         dim3(static_cast<unsigned>((items + kMergeWarps - 1) / kMergeWarps)),
                         dim3(kMergeWarps * 32), 0, stream, p);
    }
    if (kTree && err == cudaSuccess && p.sk_ctas > 0) {
        const int32_t rows = std::min(pf::kQTiles * pf::kRows, p.max_q_len * p.group);
        err = launch_pdl(prefill_tree_merge_kernel,
                         dim3(static_cast<unsigned>(p.sk_ctas),
                              static_cast<unsigned>((rows * (pf::kD / 16) + kTreeMergeThreads - 1) / kTreeMergeThreads)),
                         dim3(kTreeMergeThreads), 0, stream, p, rows);
    }
    prof_end(PKV_KERNEL_PREFILL, stream);
    return err;
}

cudaError_t launch_prefill_bf16(const PrefillParams &p, const CUtensorMap &kmap,
                                const CUtensorMap &vmap, cudaStream_t stream)
{
    if (p.tree != nullptr)
        return p.max_q_len <= pf::kRows / p.group ? launch_prefill_tc<false, false, true, true>(p, kmap, vmap, stream)
                                                  : launch_prefill_tc<false, false, true>(p, kmap, vmap, stream);
    return p.sinks > 0 ? launch_prefill_tc<false, true>(p, kmap, vmap, stream)
                       : launch_prefill_tc<false, false>(p, kmap, vmap, stream);
}

cudaError_t launch_prefill_fp8(const PrefillParams &p, cudaStream_t stream)
{
    const CUtensorMap none{};  // the FP8 producers read the pools by bulk copy
    if (p.tree != nullptr)
        return p.max_q_len <= pf::kRows / p.group ? launch_prefill_tc<true, false, true, true>(p, none, none, stream)
                                                  : launch_prefill_tc<true, false, true>(p, none, none, stream);
    return p.sinks > 0 ? launch_prefill_tc<true, true>(p, none, none, stream)
                       : launch_prefill_tc<true, false>(p, none, none, stream);
}

cudaError_t launch_prefill_f32(const PrefillParams &p, cudaStream_t stream)
{
    const int64_t ctas = static_cast<int64_t>(p.batch) * p.hkv * p.q_tiles;
    if (ctas == 0) return cudaSuccess;
    const int D = p.head_dim, bs = p.block_size, NQ = kPf32Pairs;
    const size_t smem = sizeof(float) * (2 * NQ * D + 2 * bs * D + NQ * bs + 3 * NQ) +
                        sizeof(int32_t) * 2 * NQ + sizeof(uint64_t) * NQ;
    cudaError_t err = cudaFuncSetAttribute(prefill_f32_kernel,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, kF32SmemLimit);
    if (err != cudaSuccess) return err;
    prof_begin(PKV_KERNEL_PREFILL, stream);
    err = launch_pdl(prefill_f32_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kPf32Threads),
                     smem, stream, p);
    prof_end(PKV_KERNEL_PREFILL, stream);
    return err;
}

}  // namespace pkv
