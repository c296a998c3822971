// Attention over latent rows on the 5th-generation tensor cores (bf16 pools,
// latent_dim 256 or 512, rope_dim 64).
//
// Mathematics.  A row [c | k] is key and value at once: s = scale q . [c | k],
// out = softmax(s) c, one pass with a running maximum and sum.  All heads share
// the rows, so 128 (query, head) pairs are the M side of both products and each
// row is read once for all of them.
//
// Layout.  128 pairs x 512 value dims in fp32 are the whole tensor memory of an
// SM, so a pair of CTAs (a cluster) holds an item: CTA c has the c-th half of the
// latent dims, and of the rotary dims, of queries and rows.  Each computes its
// half of the reduction of S for all keys of a tile and all pairs, the halves are
// exchanged through distributed shared memory and added (a + b on one side, b + a
// on the other: the same bits), and each CTA then has the same weights and
// multiplies them with its own half of the values.  No product is computed twice
// and each CTA stages half a row, so that four 64-key tiles fit its shared memory.
//   warps 0, 2   producers: 64-key tiles, one TMA box per (page, 64 dims);
//   warp 1       issues tcgen05.mma from one elected lane: S = Q K^T (Q's latent
//                half in tensor memory, its rotary part in shared memory), then
//                O += P V with P read from tensor memory;
//   warps 4-7    send S: each reads its 32 pairs' half sums and stores them into
//                the peer's shared memory (st.async, counted by an mbarrier there);
//   warps 8-11   softmax, one pair per thread: own half + peer's half, masks, the
//                running maximum kept within 2^8 (O is rescaled in tensor memory
//                only when it moves further), P written over S as two bf16 terms
//                (hi + lo, 2^-17 relative, as in the paged prefill: a single term's
//                2^-9 would be as large as the output's own rounding), epilogue.
// Tensor memory: O 0 .. H-1 (H = latent_dim / 2), S buffers at H and H + 64, Q's
// latent half (bf16 pairs) at H + 128.
//
// Bound: a 64-key tile takes 18 N=64 products (32 cycles each) and 8 N=H products
// (128 cycles at H = 256): about 1600 cycles, as many as the tile's bytes take at
// the HBM rate (both CTAs' 72 KB at 1/76 of the copy rate: 0.82 us).
#include <algorithm>

#include "latent_common.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace lt {
constexpr int kRows = kLatentTcRows;
constexpr int kKeys = 64;
constexpr int kRope = 64;
constexpr int kThreads = 384;
constexpr int kRegion = kKeys * 128;      // 64 dims of a tile: 8 KiB, 128-byte swizzled rows
constexpr float kRescaleLog2 = 8.f;       // O is rescaled only when the max grows past 2^8
constexpr uint32_t kTmemCols = 512;
constexpr int32_t kLeastTiles = 2;        // of a worker's run
// A piece's cost beside its tiles, in tiles, where the runs are long enough to be levelled by it
constexpr int32_t kItemCost = 4, kLevelTiles = 8;
template <int H>  // latent dims of a CTA
struct Layout {
    static constexpr int kRegions = H / 64 + 1;           // its latent dims, then the rotary ones (both halves)
    static constexpr int kStageBytes = kRegions * kRegion;
    static constexpr int kStages = H == 256 ? 4 : 6;
    static constexpr int kQOff = kStages * kStageBytes;   // Q's rotary dims: 128 rows of 128 bytes
    static constexpr int kXOff = kQOff + kRows * 128;     // the peer's half sums: [16 key quads][128 pairs] float4
    static constexpr int kBarOff = kXOff + kKeys * kRows * 4;
    // kv_full, kv_empty [stages], s_full[2], p_full[2], x_full[4], x_free[4], pv_done, o_done, q_full, drain
    static constexpr int kNumBars = 2 * kStages + 4 + 8 + 4;
    static constexpr int kMaskOff = kBarOff + kNumBars * 8;
    static constexpr int kScanOff = (kMaskOff + kStages * 4 + 15) & ~15;
    static constexpr int kTmemOff = kScanOff + (kThreads / 32 + 4) * 8;
    static constexpr int kBytes = kTmemOff + 16;
    static constexpr int kLaunchBytes = kBytes + 1024;
    static_assert(kLaunchBytes <= 227 * 1024, "shared memory of one CTA");
    static constexpr uint32_t kS = H, kQ = H + 128;       // tensor-memory columns
    static_assert(kQ + H / 2 <= kTmemCols, "tensor memory of one CTA");
};
}  // namespace lt

// ---------------------------------------------------------------------------
// cluster
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// the same shared address in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t map_shared(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes into another CTA's shared memory, counted on its mbarrier
__device__ __forceinline__ void st_async(uint32_t addr, uint32_t bar, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
                 : "memory");
}
// Arrive on another CTA's mbarrier without ordering this thread's earlier accesses
// (a release at cluster scope took 1.2 us here): for a buffer whose reads have
// already returned their values.
__device__ __forceinline__ void arrive_remote_relaxed(uint32_t bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// as mbar_wait, ordered after what the other CTA did before it arrived
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, unsigned long long limit_ns)
{
    if (try_wait_cluster(bar, parity)) return true;
    const unsigned long long t0 = globaltimer();
    for (uint32_t it = 1; it < (1u << 26); ++it) {
        if (try_wait_cluster(bar, parity)) return true;
        if ((it & 127u) == 0 && globaltimer() - t0 > limit_ns) return false;
    }
    return false;
}

// Wait by every lane of the warp (false in all lanes if any gave up); reports a timeout.
__device__ __forceinline__ bool lat_wait(uint64_t *bar, uint32_t parity, const LatentParams &p)
{
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, p.wait_ns));
    if (!ok && (threadIdx.x & 31) == 0) report(p.status, PKV_DEV_TIMEOUT);
    return ok;
}
__device__ __forceinline__ bool lat_wait_cluster(uint64_t *bar, uint32_t parity, const LatentParams &p)
{
    const bool ok = __all_sync(0xffffffffu, wait_cluster(bar, parity, p.wait_ns));
    if (!ok && (threadIdx.x & 31) == 0) report(p.status, PKV_DEV_TIMEOUT);
    return ok;
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int32_t c0, int32_t c1,
                                            int32_t c2, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
        : "memory");
}

template <int H>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(lt::kThreads, 1)
    latent_tc_kernel(const __grid_constant__ CUtensorMap map, const LatentParams p)
{
    using namespace lt;
    using L = Layout<H>;
    constexpr int kStages = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint64_t *kv_full = bars, *kv_empty = kv_full + kStages;
    uint64_t *s_full = kv_empty + kStages;  // [buffer]: S's own half computed
    uint64_t *p_full = s_full + 2;          // [buffer]: P stored
    uint64_t *x_full = p_full + 2;          // [warp]: the peer's half has landed, own half read by the sender
    uint64_t *x_free = x_full + 4;          // [warp]: the peer has read what was sent
    uint64_t *pv_done = x_free + 4, *o_done = pv_done + 1, *q_full = o_done + 1, *drain = q_full + 1;
    uint32_t *kmask = reinterpret_cast<uint32_t *>(smem + L::kMaskOff);  // [stage]: pages loaded
    int64_t *scan = reinterpret_cast<int64_t *>(smem + L::kScanOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kTmemOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), peer = rank ^ 1u;
    const int32_t worker = blockIdx.x >> 1;
    const int bs = p.block_size, nb = kKeys / bs;  // pages of a tile
    const uint32_t all_pages = (1u << nb) - 1u;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&map);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&kv_full[i], 2);  // the two producers
            mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&x_full[i], 2);  // armed by the softmax warp; the sender
            mbar_init(&x_free[i], 1);
        }
        mbar_init(pv_done, 1);
        mbar_init(o_done, 1);
        mbar_init(q_full, 8);
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    if (warp == 1) tc::alloc(tmem_slot, kTmemCols);
    tc::fence_before();
    __syncthreads();
    cluster_sync();  // the peer's barriers exist before anything is sent
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tS = tmem + L::kS, tQ = tmem + L::kQ;
    pdl_wait();
    pdl_trigger();
    // (a run without tiles: every role finds no piece)
    const LatentRun run0 = latent_run<kRows, kKeys, kThreads>(p, worker, kLeastTiles, kLevelTiles, kItemCost, rank == 0, scan);

    if (warp == 0 || warp == 2) {
        // ------------------------------------------------------------ producers
        // Tile T (a running count) goes to stage T % kStages; warp 0 brings the
        // first half of its latent regions and the rotary one, warp 2 the rest.
        constexpr int kMine = H / 128;  // latent regions of a producer
        const int first = warp == 0 ? 0 : kMine;
        const uint32_t tile_bytes = static_cast<uint32_t>(kMine + (warp == 0 ? 1 : 0)) * bs * 128;  // of a page
        const uint64_t policy = l2_evict_first_policy();
        auto withheld = [&](int32_t T) { return (p.drill & kDrillWithholdFirst) != 0 && T == 0; };
        LatentRun run = run0;
        LatentPiece pc;
        int32_t T = 0;
        bool ok = true;
        while (ok && latent_next<kRows, kKeys>(p, run, pc)) {
            const int32_t *table = p.tables + static_cast<int64_t>(pc.it.r) * p.width;
            auto page_of = [&](int32_t t, bool &in) {  // lane < nb: page `lane` of tile t
                const int32_t b = t * nb + lane;
                in = lane < nb && t < pc.t0 + pc.n && b < p.width && static_cast<int64_t>(b) * bs < pc.it.hi;
                return in ? __ldg(table + b) : -1;
            };
            bool in;
            int32_t id = page_of(pc.t0, in);
            for (int32_t j = 0; j < pc.n; ++j, ++T) {
                const int st = T % kStages;
                const int32_t cur = id;
                const bool cur_in = in;
                id = page_of(pc.t0 + j + 1, in);
                if (T >= kStages && !(ok = lat_wait(&kv_empty[st], ((T / kStages) + 1) & 1, p))) break;
                const bool good = cur_in && static_cast<uint32_t>(cur) < static_cast<uint32_t>(p.num_blocks);
                if (warp == 0 && rank == 0 && cur_in && !good) report(p.status, PKV_DEV_BAD_BLOCK);
                const uint32_t mask = __ballot_sync(0xffffffffu, good) & all_pages;
                if (warp == 0 && lane == 0) kmask[st] = mask;
                if (withheld(T)) continue;
                if (lane == 0) {
                    if (mask == 0)
                        mbar_arrive(&kv_full[st]);
                    else
                        mbar_arrive_expect_tx(&kv_full[st], __popc(mask) * tile_bytes);
                }
                __syncwarp();
                uint8_t *dst = smem + st * L::kStageBytes;
                for (int b = 0; b < nb; ++b) {
                    const int32_t blk = __shfl_sync(0xffffffffu, cur, b);
                    if (((mask >> b) & 1u) && elect_one()) {
#pragma unroll
                        for (int i = 0; i < kMine; ++i)
                            tma_load_3d(dst + (first + i) * kRegion + b * bs * 128, &map, &kv_full[st],
                                        static_cast<int32_t>(rank) * H + 64 * (first + i), 0, blk, policy);
                        if (warp == 0)
                            tma_load_3d(dst + (H / 64) * kRegion + b * bs * 128, &map, &kv_full[st], 2 * H, 0, blk, policy);
                    }
                    __syncwarp();
                }
            }
        }
        // the last ring's worth of loads has landed before the warp leaves (a
        // barrier counts both producers: waiting for its phase covers this
        // warp's part whenever the other one issued its own)
        if (lane == 0)
            for (int32_t t = max(0, T - kStages); t < T; ++t)
                if (!withheld(t)) mbar_wait(&kv_full[t % kStages], (t / kStages) & 1);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issue
        constexpr uint32_t idS = tc::idesc_bf16(kRows, kKeys, 0, 0);
        constexpr uint32_t idO = tc::idesc_bf16(kRows, H, 0, 1);  // values: MN-major (rows of dims)
        const uint64_t dk = tc::smem_desc(smem_u32(smem), 16, 1024);
        const uint64_t dv = tc::smem_desc(smem_u32(smem), kRegion, 1024);
        const uint64_t dq = tc::smem_desc(smem_u32(smem + L::kQOff), 16, 1024);
        constexpr uint64_t kStageStep = L::kStageBytes >> 4;
        // One elected lane runs the whole role.  A product is issued about as it
        // starts (the queue holds a few), so the waits for the next tile are looked
        // at before a tile's last products: done between two tiles they left the
        // tensor cores idle for 400 cycles each.
        if (elect_one()) {
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (mbar_wait(bar, parity, p.wait_ns)) return true;
                report(p.status, PKV_DEV_TIMEOUT);
                return false;
            };
            auto kv_bar = [&](int32_t T) { return &kv_full[T % kStages]; };
            auto kv_par = [&](int32_t T) { return static_cast<uint32_t>(T / kStages) & 1u; };
            // products first .. last - 1 of S(T)'s H / 16 + 2
            auto s_part = [&](int32_t T, int first, int last) {
                const uint64_t kd = dk + static_cast<uint64_t>(T % kStages) * kStageStep;
                const uint32_t d = tS + 64u * static_cast<uint32_t>(T & 1);
                const uint64_t ro = static_cast<uint64_t>(rank * 64) >> 4;  // this CTA's half of the rotary dims
#pragma unroll
                for (int kk = 0; kk < H / 16 + 2; ++kk) {
                    if (kk < first || kk >= last) continue;
                    if (kk < 2)  // queries in shared memory
                        tc::mma_ss(d, dq + ro + 2 * kk, kd + (((H / 64) * kRegion) >> 4) + ro + 2 * kk, idS, kk > 0 ? 1u : 0u);
                    else
                        tc::mma_ts(d, tQ + 8 * (kk - 2), kd + ((((kk - 2) >> 2) * kRegion + ((kk - 2) & 3) * 32) >> 4), idS, 1u);
                }
            };
            auto pv = [&](int32_t T, bool start) {
                const uint64_t vd = dv + static_cast<uint64_t>(T % kStages) * kStageStep;
                const uint32_t a = tS + 64u * static_cast<uint32_t>(T & 1);
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int kk = 0; kk < kKeys / 16; ++kk)
                        tc::mma_ts(tmem, a + 16 * kk + 8 * part, vd + static_cast<uint64_t>(kk) * (2048 >> 4), idO,
                                   (part > 0 || kk > 0 || !start) ? 1u : 0u);
                tc::commit(pv_done);
                tc::commit(&kv_empty[T % kStages]);
            };
            constexpr int kAll = H / 16 + 2, kLate = 6;
            LatentRun run = run0;
            LatentPiece pc;
            int32_t T0 = 0;
            bool ok = true;
            for (int32_t k = 0; ok && latent_next<kRows, kKeys>(p, run, pc); ++k) {
                const int32_t n = pc.n;
                ok = wait(q_full, k & 1) && wait(kv_bar(T0), kv_par(T0));
                if (!ok) break;
                tc::fence_after();
                s_part(T0, 0, kAll);
                tc::commit(&s_full[T0 & 1]);
                if (n >= 2) {
                    if (!(ok = wait(kv_bar(T0 + 1), kv_par(T0 + 1)))) break;
                    s_part(T0 + 1, 0, kAll);
                    tc::commit(&s_full[(T0 + 1) & 1]);
                }
                bool have_kv = false, have_p = false;  // K/V(T + 2) landed, P(T) stored
                for (int32_t j = 0; j < n; ++j) {
                    const int32_t T = T0 + j;
                    const bool more = j + 2 < n;
                    ok = (!more || have_kv || wait(kv_bar(T + 2), kv_par(T + 2))) && (have_p || wait(&p_full[T & 1], (T >> 1) & 1));
                    if (!ok) break;
                    tc::fence_after();
                    pv(T, j == 0);
                    if (j == n - 1) tc::commit(o_done);
                    if (more) s_part(T + 2, 0, kAll - kLate);
                    have_kv = j + 3 < n && mbar_try_wait(kv_bar(T + 3), kv_par(T + 3));
                    have_p = j + 1 < n && mbar_try_wait(&p_full[(T + 1) & 1], ((T + 1) >> 1) & 1);
                    if (more) {
                        s_part(T + 2, kAll - kLate, kAll);
                        tc::commit(&s_full[T & 1]);
                    }
                }
                T0 += n;
            }
            // every product has completed before tensor memory is freed
            tc::commit(drain);
            mbar_wait(drain, 0);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------ senders (4-7), softmax (8-11)
        const bool soft = warp >= 8;
        const int w = warp & 3, row = 32 * w + lane;
        const uint32_t lane_base = static_cast<uint32_t>(32 * w) << 16;
        // a negative scale: -q is staged (exact), so that scores take a positive factor
        const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
        // kept away from 0 so that a masked score (-inf) never meets a zero factor
        const float sl = fmaxf(fabsf(p.scale_log2), 1e-30f);
        const int W = 2 * H + kRope;
        uint8_t *x_mem = smem + L::kXOff;
        const uint32_t x_own = smem_u32(x_mem) + row * 16;
        const uint32_t x_peer = map_shared(x_own, peer), x_full_peer = map_shared(smem_u32(&x_full[w]), peer);
        const uint32_t x_free_peer = map_shared(smem_u32(&x_free[w]), peer);
        LatentRun run = run0;
        LatentPiece pc;
        int32_t T0 = 0;
        uint32_t xn = 0;  // tiles sent by this warp
        int32_t Tx = 0;   // the tile whose halves the softmax warp waits for next
        bool ok = true;
        for (int32_t k = 0; ok && latent_next<kRows, kKeys>(p, run, pc); ++k) {
            const LatentItem &it = pc.it;
            // Q: this warp's 32 pairs, half of the CTA's dims (the senders the
            // first half); the last piece's products have read the old one
            tc::fence_after();
            {
                const bool live = row < it.n;
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    static_cast<const uint16_t *>(p.q) +
                    (static_cast<int64_t>(it.q0) * p.heads + it.p0 + (live ? row : 0)) * W);
                // H / 2 dims and two chunks of the rotary dims that this CTA
                // multiplies (chunks 4 rank .. 4 rank + 3), all loads in flight at once
                const int h0 = soft ? H / 2 : 0, ch = 4 * static_cast<int>(rank) + (soft ? 2 : 0);
                uint4 v[H / 16 + 2];
#pragma unroll
                for (int i = 0; i < H / 16 + 2; ++i)
                    v[i] = live ? __ldg(src + (i < H / 16 ? (rank * H + h0) / 8 + i : 2 * H / 8 + ch + i - H / 16))
                                : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < H / 16 + 2; ++i) {
                    v[i].x ^= flip;
                    v[i].y ^= flip;
                    v[i].z ^= flip;
                    v[i].w ^= flip;
                }
#pragma unroll
                for (int c = 0; c < H / 16; c += 8) {
                    uint32_t r[32];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        r[4 * i] = v[c + i].x;
                        r[4 * i + 1] = v[c + i].y;
                        r[4 * i + 2] = v[c + i].z;
                        r[4 * i + 3] = v[c + i].w;
                    }
                    tc::st32(tQ + lane_base + h0 / 2 + 4 * c, r);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<uint4 *>(smem + L::kQOff + row * 128 + (((ch + i) ^ (row & 7)) << 4)) = v[H / 16 + i];
                fence_proxy_async_smem();
                tc::wait_st();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            const bool warp_live = 32 * w < it.n;
            if (!soft) {
                for (int32_t j = 0; j < pc.n; ++j) {
                    const int32_t T = T0 + j, buf = T & 1, st = T % kStages, tbase = (pc.t0 + j) * kKeys;
                    // the peer has read the last tile's halves
                    if (warp_live && xn > 0 && !(ok = lat_wait_cluster(&x_free[w], (xn - 1) & 1, p))) break;
                    if (!(ok = lat_wait(&s_full[buf], (T >> 1) & 1, p))) break;
                    tc::fence_after();
                    if (warp_live) {
                        uint32_t r0[32], r1[32];
                        tc::ld32(tS + 64 * buf + lane_base, r0);
                        tc::ld32(tS + 64 * buf + 32 + lane_base, r1);
                        tc::wait_ld();
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            st_async(x_peer + q * (kRows * 16), x_full_peer, r0[4 * q], r0[4 * q + 1], r0[4 * q + 2], r0[4 * q + 3]);
                            st_async(x_peer + (8 + q) * (kRows * 16), x_full_peer, r1[4 * q], r1[4 * q + 1], r1[4 * q + 2], r1[4 * q + 3]);
                        }
                        ++xn;
                    }
                    // value rows of keys past the item's or of pages not loaded
                    // hold stale slots (possibly NaN): thread r zeroes half the
                    // dims of key row r % 64 before the tile's products read them
                    if (!(ok = lat_wait(&kv_full[st], (T / kStages) & 1, p))) break;
                    const uint32_t mask = kmask[st];
                    if (mask != all_pages || tbase + kKeys > it.hi) {
                        const int kr = row & (kKeys - 1);
                        if (tbase + kr >= it.hi || !((mask >> (kr / bs)) & 1u)) {
                            uint8_t *v = smem + st * L::kStageBytes + (row >> 6) * (H / 128) * kRegion + kr * 128;
#pragma unroll
                            for (int i = 0; i < H / 128; ++i)
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                    *reinterpret_cast<uint4 *>(v + i * kRegion + c * 16) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                    }
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x_full[w]);
                }
                T0 += pc.n;
                continue;
            }
            const LatentRange rg = latent_range(p, it, row);
            // keys attended whatever the mask (a pair that is none takes every key: its
            // output is not stored, and its warp keeps to the plain path)
            const int32_t sure = row >= it.n ? INT32_MAX : p.tree != nullptr ? min(rg.hi, it.first) : rg.hi;
            float m_ref = -INFINITY, l = 0.f;
            for (int32_t j = 0; j < pc.n; ++j) {
                const int32_t T = T0 + j, buf = T & 1, st = T % kStages;
                const int32_t tbase = (pc.t0 + j) * kKeys;
                const uint32_t sx = tS + 64 * buf + lane_base;
                // S's own half computed and read by the sender, the peer's half here,
                // stale value rows zeroed: one barrier says it all
                if (lane == 0) {
                    if (warp_live)
                        mbar_arrive_expect_tx(&x_full[w], 32 * kKeys * 4);
                    else
                        mbar_arrive(&x_full[w]);
                }
                if (!(ok = lat_wait_cluster(&x_full[w], T & 1, p))) break;
                Tx = T + 1;
                tc::fence_after();
                const uint32_t mask = kmask[st];
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
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const uint4 v = lds128(x_own + q * (kRows * 16));
                        s[4 * q] += __uint_as_float(v.x);
                        s[4 * q + 1] += __uint_as_float(v.y);
                        s[4 * q + 2] += __uint_as_float(v.z);
                        s[4 * q + 3] += __uint_as_float(v.w);
                    }
                    if (!(mask == all_pages && tbase + kKeys <= sure)) {
                        // attended keys as bits
                        const auto below = [](int32_t n) {  // bits 0 .. n-1
                            return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull;
                        };
                        uint64_t bits = below(rg.hi - tbase);
                        if (p.tree != nullptr) bits &= tree_bits(rg.mask, tbase, it.first);
                        uint64_t pages = 0;
                        for (int b = 0; b < nb; ++b) pages |= ((mask >> b) & 1u) ? below(bs) << (b * bs) : 0ull;
                        bits &= pages;
                        const uint32_t b0 = static_cast<uint32_t>(bits), b1 = static_cast<uint32_t>(bits >> 32);
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            s[e] = (((e < 32 ? b0 : b1) >> (e & 31)) & 1u) ? s[e] : -INFINITY;
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
                    // the reference max stays within 2^8 of the running max
                    const float new_ref = (mt > m_ref + kRescaleLog2) ? mt : m_ref;
                    const float alpha = fast_exp2(m_ref - new_ref);  // 0 from -inf, 1 if unchanged
                    const bool resc = new_ref != m_ref && m_ref != -INFINITY;
                    const bool any = __any_sync(0xffffffffu, resc);
                    // every lane's vote came of values that it has read: the peer
                    // may overwrite them
                    if (lane == 0) arrive_remote_relaxed(x_free_peer);
                    if (any) {
                        // O holds P.V up to tile j-1 once that product completes
                        if (j > 0) {
                            if (!(ok = lat_wait(pv_done, (T - 1) & 1, p))) break;
                            tc::fence_after();
                        }
                        const float f = resc ? alpha : 1.f;
#pragma unroll 1
                        for (int c = 0; c < H; c += 32) {
                            uint32_t r[32];
                            tc::ld32(tmem + lane_base + c, r);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                            tc::st32(tmem + lane_base + c, r);
                        }
                        tc::wait_st();
                    }
                    m_ref = new_ref;
                    const float nmu = new_ref == -INFINITY ? 0.f : -new_ref;
                    const uint64_t sl2 = f2_pack(sl, sl), nmu2 = f2_pack(nmu, nmu);
                    uint64_t ls2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
                    // group g (16 keys) -> 8 columns of P hi then 8 of P lo
#pragma unroll
                    for (int g = 0; g < kKeys / 16; ++g) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float a, b;
                            f2_unpack(f2_fma(f2_pack(s[16 * g + 2 * e], s[16 * g + 2 * e + 1]), sl2, nmu2), a, b);
                            a = fast_exp2(a);
                            b = fast_exp2(b);
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
                    float l0, l1, l2, l3;
                    f2_unpack(ls2[0], l0, l1);
                    f2_unpack(ls2[1], l2, l3);
                    l = l * (resc ? alpha : 1.f) + ((l0 + l1) + (l2 + l3));
                }
                tc::wait_st();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[buf]);
            }
            if (!ok) break;
            T0 += pc.n;
            // epilogue, once the piece's last product is in (a parity names one
            // phase only: o_done completes once a piece, its next needs this warp)
            if (!(ok = lat_wait(o_done, k & 1, p))) break;
            tc::fence_after();
            const bool live = row < it.n;
            if (pc.whole) {
                const float inv = l != 0.f ? 1.f / l : 0.f;  // (NaN stays NaN)
                uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) +
                                                       latent_out_row(p, it, live ? row : 0) + rank * H);
#pragma unroll 1
                for (int c = 0; warp_live && c < H; c += 32) {
                    uint32_t r[32];
                    tc::ld32(tmem + lane_base + c, r);
                    tc::wait_ld();
                    if (!live) continue;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = pack_bf16x2(__uint_as_float(r[8 * i + 2 * e]) * inv,
                                               __uint_as_float(r[8 * i + 2 * e + 1]) * inv);
                        out[c / 8 + i] = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
            } else {
                // a partial: value quads of 32 pairs side by side
                float4 *dst = latent_part_o<kRows>(p, worker, pc.slot) + (rank * H / 4) * kRows + row;
#pragma unroll 1
                for (int c = 0; warp_live && c < H; c += 32) {
                    uint32_t r[32];
                    tc::ld32(tmem + lane_base + c, r);
                    tc::wait_ld();
                    if (!live) continue;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        dst[(c / 4 + i) * kRows] =
                            make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                        __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
                }
                if (rank == 0 && live) latent_part_ml<kRows>(p, worker, pc.slot)[row] = make_float2(m_ref, l);
            }
            tc::fence_before();
        }
        // wind-down after a wait ran out: what the peer may still be sending
        // lands (or the limit passes) before this CTA's shared memory goes
        if (soft && !ok) wait_cluster(&x_full[w], Tx & 1, kWaitLimitNs);
        __syncwarp();
    }
    // both CTAs: nothing is on its way into the other's shared memory any more
    tc::fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) tc::dealloc(tmem, kTmemCols);
}

bool latent_tc_built(pkv_dtype dtype, int32_t latent, int32_t rope, int32_t bs)
{
    return dtype == PKV_BF16 && (latent == 256 || latent == 512) && rope == lt::kRope && (bs == 16 || bs == 32 || bs == 64);
}

template <int H>
static cudaError_t launch(const LatentParams &p, const CUtensorMap &map, cudaStream_t stream)
{
    constexpr int smem = lt::Layout<H>::kLaunchBytes;
    cudaError_t err = cudaFuncSetAttribute(latent_tc_kernel<H>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    prof_begin(PKV_KERNEL_LATENT, stream);
    err = launch_pdl(latent_tc_kernel<H>, dim3(static_cast<unsigned>(2 * p.workers)), dim3(lt::kThreads), smem, stream, map, p);
    if (err == cudaSuccess)
        err = launch_pdl(latent_merge_kernel<__nv_bfloat16, lt::kRows, lt::kKeys>,
                         dim3(static_cast<unsigned>(p.workers), static_cast<unsigned>((p.latent + 63) / 64)),
                         dim3(kLatMergeThreads), 0, stream, p);
    prof_end(PKV_KERNEL_LATENT, stream);
    return err;
}

cudaError_t launch_latent_tc(const LatentParams &p, const CUtensorMap &map, cudaStream_t stream)
{
    return p.latent == 512 ? launch<256>(p, map, stream) : launch<128>(p, map, stream);
}

}  // namespace pkv
