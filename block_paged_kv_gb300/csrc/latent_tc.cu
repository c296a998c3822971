// Attention over latent rows on the 5th-generation tensor cores (bf16 pools,
// latent_dim 256 or 512, rope_dim 64).
//
// Mathematics.  A row [c | k] is key and value at once: s = scale q . [c | k],
// out = softmax(s) c, one pass with a running maximum and sum.  All heads share
// the rows, so 128 (query, head) pairs are the M side of both products and each
// row is read once for all of them.
//
// Layout.  128 pairs x 512 value dims in fp32 are the whole tensor memory of an
// SM, so a pair of CTAs (a cluster) holds an item, and the two products are split
// between them: CTA 0 computes the scores and the softmax, CTA 1 the weighted
// values.  What passes between them is the weights alone, one way, 16 KB a 64-key
// tile through distributed shared memory (which carries about 21 bytes a cycle
// between two SMs here: 800 cycles), so that neither waits for the other within a
// tile.  An item's queries come through CTA 0's ring like two tiles more (read by
// their pairs' threads, 32 rows an instruction, they took 9 us).  Each CTA loads what
// it multiplies, CTA 0 whole rows, CTA 1 their latent part a tile or two later, out of
// L2.
//   both:  warps 0, 2, 3 producers (one issuing thread brings 21 to 25 bytes a cycle
//     whatever its boxes' size, three of them 60), a box of 8 keys each;
//   CTA 0: warp 1 issues S = Q K^T from one lane (Q in tensor memory, three S
//     buffers); warps 4-7 and 8-11 softmax, a thread a pair, the even and the odd
//     tiles: masks, the running maximum kept within 2^8 (handed from tile to tile),
//     weights to CTA 1 (st.async, counted by an mbarrier there);
//   CTA 1: warp 1 issues O += P V (P in shared memory as it came, 8 x 16-byte core
//     matrices); warps 4-11: O rescaled in tensor memory when the maximum moved
//     further, stale value rows zeroed, epilogue, half the dims each.
// (With the dims of both products split instead, each CTA held half of the scores'
// reduction, and exchanging those, 32 KB of fp32 a tile each way, took 1700 cycles
// of a 3100-cycle tile.)
//
// P enters P.V as one bf16 term, and the sums are those of the rounded weights, so
// that a rounding moves a weight against the others but not their sum (2-norm against
// 64 bits 0.0019 to 0.0021; 0.0017, the output's own rounding, with a second term, which
// would double CTA 1's products to 2048 cycles a tile).
//
// Bound: a 64-key tile of 128 pairs takes 36 N=64 products (32 cycles each) on one
// SM beside 8 N=256 ones (128 cycles) on the other, 1152 cycles, and its 72 KB at
// 1/76 of the HBM copy rate 0.82 us, 1600 cycles: HBM, or the tensor cores where the
// rows come from L2 (chunks); and shared memory, at 128 bytes a cycle: 147 KB of rows
// written and read on CTA 0 (1152 cycles), 176 KB with the weights on CTA 1 (1375).
// Measured: 2 chunks of 512 x 16 heads 132 to 135 us (tensor pipe 49 % busy, L2 hits 92 %,
// a tile about 1750 cycles), decode of 32 rows x 128 heads 58.4 us (186 MB from HBM, 3.4
// TB/s; tensor pipe 32 %), of 4 rows x 16 heads 17 us, launches and one chain of
// dependent steps.
#include <algorithm>

#include "latent_common.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace lt {
constexpr int kRows = kLatentTcRows;
constexpr int kKeys = 64;
constexpr int kRope = 64;
constexpr int kThreads = 384;
constexpr int kProducers = 3;             // warps of either CTA
constexpr int kSoftWarps = 8;             // of either CTA: warps 4 .. 11
constexpr int kFins = 3;                  // pieces whose sums may be on their way
constexpr int kSBufs = 3, kPBufs = 2;
// What a tile's softmax waits for, in one barrier: its scores; what the producer wrote
// of it, passed on by the issuing lane; the last tile's reference maximum (four warps).
constexpr int kSArrivals = 1 + 1 + kSoftWarps / 2;
constexpr int kMasks = 16;                // tiles between a producer and the softmax, at most stages + S buffers
constexpr int kPBytes = kRows * kKeys * 2;
constexpr float kRescaleLog2 = 8.f;       // O is rescaled only when the max grows past 2^8
constexpr uint32_t kTmemCols = 512;
// Tiles of a worker's run, at least: 4 rows x 16 heads 16.9 us with 2, 19.4 with 1, 17.7
// with 4.
constexpr int32_t kLeastTiles = 2;
// A piece's cost beside its tiles, in tiles, where the runs are long enough to be
// levelled by it: 16 trees of 1 to 64 drafts 95.5 us with 6, 97.7 with 4, 103.9 with 2,
// 97.2 with 10 (chunks 131.8, 134.2, 132.9, 132.9).
constexpr int32_t kItemCost = 6, kLevelTiles = 8;
template <int NR>  // 64-dim regions of the latent
struct Layout {
    // a tile: [8-key group][region][8 keys][128 bytes], 128-byte swizzled; CTA 0 has
    // the rotary region too
    static constexpr int kGroup0 = (NR + 1) * 1024, kGroup1 = NR * 1024;
    static constexpr int kStages = NR == 8 ? 3 : 5;
    // CTA 0, behind its stages: reference maxima [tile % 2][128], one half's (maximum, sum) [128]
    static constexpr int kMaxOff = kStages * 8 * kGroup0;
    // CTA 1: weights [buffer][8-key chunk][128 pairs][16 bytes]
    static constexpr int kPOff = kStages * 8 * kGroup1;
    static constexpr int kAfter0 = kMaxOff + 4 * kRows * 4, kAfter1 = kPOff + kPBufs * kPBytes;
    static constexpr int kAlphaOff = kAfter0 > kAfter1 ? kAfter0 : kAfter1;  // [buffer][128]: factors of O
    static constexpr int kFinOff = kAlphaOff + kPBufs * kRows * 4;           // [piece % kFins][128]: weight sums
    static constexpr int kBarOff = kFinOff + kFins * kRows * 4;
    // kv_full, kv_empty [stages], s_full, s_free [3], p_full, p_free, p_ready [2], fin_full [3], pv_done, o_done, q_full, l_full, drain, go
    static constexpr int kNumBars = 2 * kStages + 2 * kSBufs + 3 * kPBufs + kFins + 6;
    static constexpr int kMaskOff = kBarOff + kNumBars * 8;
    static constexpr int kScanOff = (kMaskOff + kMasks * 4 + 15) & ~15;  // (of its own: the peer may be sending already)
    static constexpr int kTmemOff = kScanOff + (kThreads / 32 + 4) * 8;
    static constexpr int kBytes = kTmemOff + 16;
    static_assert(kPBufs == 2, "a softmax group keeps to one of the weights' buffers");
    static_assert(kBytes <= 227 * 1024 && kStages + kSBufs <= kMasks, "shared memory of one CTA");
    static constexpr uint32_t kQCols = NR * 32 + 32;  // CTA 0's tensor memory: Q, then the S buffers
    static_assert(kQCols + kSBufs * 64 <= kTmemCols && NR * 64 <= kTmemCols, "tensor memory of one CTA");
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
// 4 bytes likewise
__device__ __forceinline__ void st_async1(uint32_t addr, uint32_t bar, uint32_t a)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr), "r"(a), "r"(bar)
                 : "memory");
}
// Arrive on another CTA's mbarrier without ordering this thread's earlier accesses (a
// release at cluster scope takes 1.2 us).
__device__ __forceinline__ void arrive_remote(uint32_t bar)
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

// v[i] of lane b of a quad (four neighbouring lanes) becomes v[b] of its lane i.
__device__ __forceinline__ void quad_transpose(uint4 (&v)[4], int b)
{
    auto swap = [&](int i, int j, int d) {  // v[i] of the upper lane with v[j] of the lower one
        const bool upper = (b & d) != 0;
        uint4 x = upper ? v[i] : v[j];
        x.x = __shfl_xor_sync(0xffffffffu, x.x, d);
        x.y = __shfl_xor_sync(0xffffffffu, x.y, d);
        x.z = __shfl_xor_sync(0xffffffffu, x.z, d);
        x.w = __shfl_xor_sync(0xffffffffu, x.w, d);
        if (upper) v[i] = x;
        else v[j] = x;
    };
    swap(0, 1, 1);
    swap(2, 3, 1);
    swap(0, 2, 2);
    swap(1, 3, 2);
}

// arrive on the mbarrier of every CTA in `mask` once the products issued so far have completed
__device__ __forceinline__ void commit_to(uint64_t *bar, uint16_t mask)
{
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(mask)
        : "memory");
}

// Shared-memory matrix descriptor without swizzle, K-major: core matrices of 8 rows
// x 16 bytes; lbo between core matrices along K, sbo between those along M.
__device__ __forceinline__ uint64_t smem_desc_plain(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46);
}

// A producer warp (w of three) of CTA kRank.  Ring entry U goes to stage
// U % kStages: in CTA 1 tile T is entry T, in CTA 0 the queries of every piece are two
// entries before its tiles (64 pairs each, laid out as 64 keys are).  Producer w
// brings an entry's 8-row groups w, w + 3, w + 6, and arrives for it also where it has
// none of them: an entry that completed without a producer could be used and freed, and
// its stage's next one too, before that producer looks at the stage, and the parity that
// it waits for would then be two phases old.
template <int NR, int kRank>
__device__ __forceinline__ void latent_produce(const CUtensorMap &map, const CUtensorMap &q_map, const LatentParams &p,
                                               Run run, uint8_t *smem, uint64_t *kv_full, uint64_t *kv_empty,
                                               uint32_t *kmask, int w, int lane)
{
    using namespace lt;
    using L = Layout<NR>;
    constexpr int n = L::kStages, group = kRank == 0 ? L::kGroup0 : L::kGroup1, stage = 8 * group;
    const int bs_log = 31 - __clz(p.block_size), nb = kKeys >> bs_log;  // pages of a tile
    const uint32_t all_pages = (1u << nb) - 1u;
    // CTA 1 is its pair's last reader.  Other pairs may read the rows too, and it holds for
    // them: 2 chunks of 512 x 16 heads 134.9 us (evict_normal 136.8), 32 rows x 128 heads
    // over 32768 shared rows 216.6 (226.5), over 1024 to 8192 of their own 58.5 (59.1).
    const uint64_t policy = kRank == 0 ? l2_evict_normal_policy() : l2_evict_first_policy();
    auto withheld = [&](int32_t U) { return (p.drill & kDrillWithholdFirst) != 0 && U == 0; };
    LatentPiece pc;
    bool ok = true;
    int32_t T = 0, U = 0;
    auto free_stage = [&]() {
        if ((p.drill & kDrillLateProducers) != 0 && w != 0) come_late(5000 * w);
        return U < n || lat_wait(&kv_empty[U % n], ((U / n) + 1) & 1, p);
    };
    auto arm = [&](int32_t groups) {  // this warp's part of an entry
        if (lane != 0) return;
        if (groups == 0)
            mbar_arrive(&kv_full[U % n]);
        else
            mbar_arrive_expect_tx(&kv_full[U % n], groups * group);
    };
    while (ok && latent_next<kRows, kKeys>(p, run, pc)) {
        const int32_t *table = p.tables + static_cast<int64_t>(pc.it.r) * p.width;
        auto page_of = [&](int32_t t, bool &in) {  // lane < nb: page `lane` of tile t
            const int32_t b = t * nb + lane;
            in = lane < nb && t < pc.t0 + pc.n && b < p.width && (static_cast<int64_t>(b) << bs_log) < pc.it.hi;
            return in ? __ldg(table + b) : -1;
        };
        bool in;
        int32_t id = page_of(pc.t0, in);
        if constexpr (kRank == 0) {
            for (int h = 0; h < 2; ++h, ++U) {
                if (!(ok = free_stage())) break;
                const int32_t row = pc.it.q0 * p.heads + pc.it.p0 + 64 * h;
                const int32_t groups = min(max((pc.it.n - 64 * h + 7) / 8, 0), 8);
                if (withheld(U)) continue;
                arm(max(0, groups - w + kProducers - 1) / kProducers);
                __syncwarp();
                uint8_t *dst = smem + (U % n) * stage;
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const int g = w + kProducers * i;
                    if (g < groups && elect_one())
                        tma_load_4d(dst + g * group, &q_map, &kv_full[U % n], 0, row + 8 * g, 0, 0, policy);
                    __syncwarp();
                }
            }
        }
        for (int32_t j = 0; ok && j < pc.n; ++j, ++T) {
            const int32_t cur = id;
            const bool cur_in = in;
            id = page_of(pc.t0 + j + 1, in);
            const bool good = cur_in && static_cast<uint32_t>(cur) < static_cast<uint32_t>(p.num_blocks);
            if (w == 0 && kRank == 0 && cur_in && !good) report(p.status, PKV_DEV_BAD_BLOCK);
            const uint32_t mask = __ballot_sync(0xffffffffu, good) & all_pages;
            if (!(ok = free_stage())) break;
            if (w == 0 && lane == 0) kmask[T % kMasks] = mask;
            if (!withheld(U)) {
                int32_t groups = 0;
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const int g = w + kProducers * i;
                    groups += g < 8 && ((mask >> (g * 8 >> bs_log)) & 1u) ? 1 : 0;
                }
                arm(groups);
                __syncwarp();
                uint8_t *dst = smem + (U % n) * stage;
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const int g = w + kProducers * i, b = ((g & 7) * 8) >> bs_log;
                    const int32_t blk = __shfl_sync(0xffffffffu, cur, b);
                    if (g < 8 && ((mask >> b) & 1u) && elect_one())
                        tma_load_4d(dst + g * group, &map, &kv_full[U % n], 0, g * 8 - (b << bs_log), 0, blk, policy);
                    __syncwarp();
                }
            }
            ++U;
        }
    }
    // what is on its way into this CTA has landed before the warp leaves
    if (lane == 0)
        for (int32_t t = max(0, U - n); t < U; ++t)
            if (!withheld(t)) mbar_wait(&kv_full[t % n], (t / n) & 1);
    __syncwarp();
}

template <int NR>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(lt::kThreads, 1)
    latent_tc_kernel(const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1,
                     const __grid_constant__ CUtensorMap q_map, const LatentParams p)
{
    using namespace lt;
    using L = Layout<NR>;
    constexpr int kStages = L::kStages, R = NR * 64;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint64_t *kv_full = bars, *kv_empty = kv_full + kStages;
    uint64_t *s_full = kv_empty + kStages, *s_free = s_full + kSBufs;   // CTA 0
    uint64_t *p_full = s_free + kSBufs;     // CTA 1: weights landed
    uint64_t *p_free = p_full + kPBufs;     // CTA 0: weights multiplied
    uint64_t *p_ready = p_free + kPBufs;    // CTA 1: O and the value rows ready for them
    uint64_t *fin_full = p_ready + kPBufs;  // CTA 1: a piece's sums landed
    uint64_t *pv_done = fin_full + kFins, *o_done = pv_done + 1;
    uint64_t *q_full = o_done + 1, *l_full = q_full + 1, *drain = l_full + 1, *go = drain + 1;
    uint32_t *kmask = reinterpret_cast<uint32_t *>(smem + L::kMaskOff);  // [tile % kMasks]: pages loaded
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kTmemOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int32_t worker = blockIdx.x >> 1;
    const int bs = p.block_size, nb = kKeys / bs;  // pages of a tile
    const uint32_t all_pages = (1u << nb) - 1u;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(rank == 0 ? &map0 : &map1);
        if (rank == 0) tma_prefetch_desc(&q_map);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&kv_full[i], kProducers);
            mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < kSBufs; ++i) {
            mbar_init(&s_full[i], kSArrivals);
            mbar_init(&s_free[i], kSoftWarps / 2);
        }
        for (int i = 0; i < kPBufs; ++i) {
            mbar_init(&p_full[i], 1);
            mbar_init(&p_free[i], 1);
            mbar_init(&p_ready[i], kSoftWarps);
        }
        for (int i = 0; i < kFins; ++i) mbar_init(&fin_full[i], 1);
        mbar_init(pv_done, 1);
        mbar_init(o_done, 1);
        mbar_init(q_full, kSoftWarps);
        mbar_init(l_full, kSoftWarps / 2);
        mbar_init(drain, 1);
        mbar_init(go, 1);
        fence_mbar_init();
    }
    if (warp == 1) tc::alloc(tmem_slot, kTmemCols);
    tc::fence_before();
    __syncthreads();
    cluster_sync();  // the peer's barriers exist before anything is sent
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tS = tmem + L::kQCols;
    pdl_wait();
    pdl_trigger();
    // (a run without tiles: every role finds no piece)
    const Run run0 = latent_run<kRows, kKeys, kThreads>(p, worker, kLeastTiles, kLevelTiles, kItemCost, rank == 0,
                                                              reinterpret_cast<int64_t *>(smem + L::kScanOff));
    Run run = run0;
    LatentPiece pc;
    bool ok = true;

    if (warp == 0 || warp == 2 || warp == 3) {
        // ------------------------------------------------------------ producers
        const int w = warp == 0 ? 0 : warp - 1;
        if (rank == 0)
            latent_produce<NR, 0>(map0, q_map, p, run0, smem, kv_full, kv_empty, kmask, w, lane);
        else if (run0.pos >= run0.end || lat_wait(go, 0, p))  // the queries come first
            latent_produce<NR, 1>(map1, q_map, p, run0, smem, kv_full, kv_empty, kmask, w, lane);
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        // One elected lane runs the whole role: a product is issued about as it
        // starts (the queue holds a few).
        if (elect_one()) {
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (mbar_wait(bar, parity, p.wait_ns)) return true;
                report(p.status, PKV_DEV_TIMEOUT);
                return false;
            };
            int32_t T = 0, U = 0;
            if (rank == 0) {
                constexpr uint32_t idS = tc::idesc_bf16(kRows, kKeys, 0, 0);
                const uint64_t dk = tc::smem_desc(smem_u32(smem), 16, L::kGroup0);
                // The next tile's waits are looked at before a tile's last products:
                // done between two tiles they left the tensor cores idle.
                constexpr int kAll = (NR + 1) * 4, kLate = 8;
                auto products = [&](int32_t tile, int32_t entry, int first, int last) {
                    const uint64_t kd = dk + static_cast<uint64_t>(entry % kStages) * (8 * L::kGroup0 >> 4);
                    const uint32_t d = tS + 64u * static_cast<uint32_t>(tile % kSBufs);
#pragma unroll
                    for (int kk = 0; kk < kAll; ++kk)
                        if (kk >= first && kk < last)
                            tc::mma_ts(d, tmem + 8 * kk, kd + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), idS, kk > 0 ? 1u : 0u);
                };
                for (int32_t k = 0; ok && latent_next<kRows, kKeys>(p, run, pc); ++k) {
                    ok = wait(q_full, k & 1);
                    if (!ok) break;
                    if (k == 0) arrive_remote(map_shared(smem_u32(go), 1));
                    for (int h = 0; h < 2; ++h, ++U) mbar_arrive(&kv_empty[U % kStages]);  // in tensor memory now
                    bool have_kv = false, have_s = false;  // this tile's rows landed, its S buffer free
                    for (int32_t j = 0; j < pc.n; ++j, ++T, ++U) {
                        const int buf = T % kSBufs;
                        ok = (have_kv || wait(&kv_full[U % kStages], (U / kStages) & 1)) &&
                             (have_s || T < kSBufs || wait(&s_free[buf], ((T / kSBufs) + 1) & 1));
                        if (!ok) break;
                        // what the producer wrote of the tile, passed on
                        // (and what the first tile has no predecessor for)
                        for (int i = 1 + (T == 0 ? kSoftWarps / 2 : 0); i > 0; --i) mbar_arrive(&s_full[buf]);
                        tc::fence_after();
                        products(T, U, 0, kAll - kLate);
                        have_kv = j + 1 < pc.n && mbar_test(&kv_full[(U + 1) % kStages], ((U + 1) / kStages) & 1);
                        have_s = j + 1 < pc.n && T + 1 >= kSBufs && mbar_test(&s_free[(T + 1) % kSBufs], (((T + 1) / kSBufs) + 1) & 1);
                        products(T, U, kAll - kLate, kAll);
                        tc::commit(&s_full[buf]);
                        tc::commit(&kv_empty[U % kStages]);
                    }
                }
            } else {
                constexpr int N = R < 256 ? R : 256;
                constexpr uint32_t idO = tc::idesc_bf16(kRows, N, 0, 1);  // values: MN-major (rows of dims)
                const uint64_t dv = tc::smem_desc(smem_u32(smem), 1024, L::kGroup1);
                const uint64_t dp = smem_desc_plain(smem_u32(smem + L::kPOff), kRows * 16, 128);
                while (ok && latent_next<kRows, kKeys>(p, run, pc)) {
                    for (int32_t j = 0; j < pc.n; ++j, ++T) {
                        const int st = T % kStages, buf = T % kPBufs;
                        ok = wait(&p_ready[buf], (T / kPBufs) & 1) && wait(&kv_full[st], (T / kStages) & 1);
                        if (!ok) break;
                        tc::fence_after();
                        const uint64_t vd = dv + static_cast<uint64_t>(st) * (8 * L::kGroup1 >> 4);
                        const uint64_t pd = dp + static_cast<uint64_t>(buf) * (kPBytes >> 4);
#pragma unroll
                        for (int kk = 0; kk < kKeys / 16; ++kk)
#pragma unroll
                            for (int n = 0; n < R / N; ++n)
                                tc::mma_ss(tmem + n * N, pd + kk * ((2 * kRows * 16) >> 4),
                                           vd + ((kk * 2 * L::kGroup1 + n * (N / 64) * 1024) >> 4), idO, (j > 0 || kk > 0) ? 1u : 0u);
                        tc::commit(pv_done);
                        tc::commit(&kv_empty[st]);
                        commit_to(&p_free[buf], 1);  // CTA 0's
                        if (j == pc.n - 1) tc::commit(o_done);
                    }
                }
            }
            // every product has completed before tensor memory is freed
            tc::commit(drain);
            mbar_wait(drain, 0);
        }
        __syncwarp();
    } else if (warp >= 4 && rank == 0) {
        // ------------------------------------------------------------ softmax
        // group g = 0 (warps 4-7) takes the even tiles, g = 1 (warps 8-11) the odd ones
        const int g = (warp >> 2) - 1, w = warp & 3, row = 32 * w + lane;
        const uint32_t lane_base = static_cast<uint32_t>(32 * w) << 16;
        // a negative scale: -q is staged (exact), so that scores take a positive factor
        const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
        // kept away from 0 so that a masked score (-inf) never meets a zero factor
        const float sl = fmaxf(fabsf(p.scale_log2), 1e-30f);
        float *refs = reinterpret_cast<float *>(smem + L::kMaxOff);                       // [T % 2][128]
        float2 *sums = reinterpret_cast<float2 *>(smem + L::kMaxOff + 2 * kRows * 4);     // [128]
        const uint32_t p_peer = map_shared(smem_u32(smem + L::kPOff), 1) + row * 16;
        const uint32_t alpha_peer = map_shared(smem_u32(smem + L::kAlphaOff), 1) + row * 4;
        const uint32_t fin_peer = map_shared(smem_u32(smem + L::kFinOff), 1) + row * 4;
        const uint32_t p_full_peer = map_shared(smem_u32(p_full), 1), fin_full_peer = map_shared(smem_u32(fin_full), 1);
        int32_t T0 = 0, sent = 0;  // one past the last tile whose weights this warp sent
        for (int32_t k = 0; ok && latent_next<kRows, kKeys>(p, run, pc); ++k) {
            const LatentItem &it = pc.it;
            // Q into tensor memory: this warp's 32 pairs, half of their dims (the last
            // piece's products have read the old one: this warp saw its last scores)
            {
                const int32_t U = T0 + 2 * k + (w >> 1);  // its ring entry
                if (!(ok = lat_wait(&kv_full[U % kStages], (U / kStages) & 1, p))) break;
                tc::fence_after();
                const bool live = row < it.n;
                const uint32_t src = smem_u32(smem + (U % kStages) * 8 * L::kGroup0) + ((row & 63) >> 3) * L::kGroup0 + (row & 7) * 128;
                constexpr int kVecs = (R + kRope) / 16;  // 16-byte vectors of a half
                static_assert(kVecs % 4 == 0, "stored four at a time");
#pragma unroll
                for (int c = 0; c < kVecs; c += 4) {
                    uint32_t r[16];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int v = g * kVecs + c + e;
                        uint4 x = lds128(src + (v >> 3) * 1024 + (((v & 7) ^ (row & 7)) << 4));
                        if (!live) x = make_uint4(0, 0, 0, 0);
                        r[4 * e] = x.x ^ flip;
                        r[4 * e + 1] = x.y ^ flip;
                        r[4 * e + 2] = x.z ^ flip;
                        r[4 * e + 3] = x.w ^ flip;
                    }
                    tc::st16(tmem + lane_base + (g * kVecs + c) * 4, r);
                }
                fence_proxy_async_smem();  // read before the stage is loaded again
                tc::wait_st();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            const bool warp_live = 32 * w < it.n;
            const LatentRange rg = latent_range(p, it, row);
            // keys attended whatever the mask (a pair that is none takes every key: its
            // output is not stored, and its warp keeps to the plain path)
            const int32_t sure = row >= it.n ? INT32_MAX : p.tree != nullptr ? min(rg.hi, it.first) : rg.hi;
            const int32_t end = T0 + pc.n;
            float m_ref = -INFINITY, l = 0.f;  // of this group's tiles: l in units of 2^m_ref
            for (int32_t T = T0 + ((T0 ^ g) & 1); T < end; T += 2) {
                const int buf = T % kSBufs, pb = T & 1;
                const int32_t tbase = (pc.t0 + T - T0) * kKeys;
                if (!(ok = lat_wait_cluster(&s_full[buf], (T / kSBufs) & 1, p))) break;
                const uint32_t mask = kmask[T % kMasks];
                if (!warp_live) {
                    if (lane == 0) {
                        mbar_arrive(&s_free[buf]);
                        mbar_arrive(&s_full[(T + 1) % kSBufs]);
                    }
                    continue;
                }
                tc::fence_after();
                float s[64];
                {
                    uint32_t r0[32], r1[32];
                    tc::ld32(tS + 64 * buf + lane_base, r0);
                    tc::ld32(tS + 64 * buf + 32 + lane_base, r1);
                    tc::wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        s[e] = __uint_as_float(r0[e]);
                        s[32 + e] = __uint_as_float(r1[e]);
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_free[buf]);
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
                // the reference max stays within 2^8 of the running max
                const float last_ref = T > T0 ? refs[(1 - pb) * kRows + row] : -INFINITY;
                const float new_ref = (mt > last_ref + kRescaleLog2) ? mt : last_ref;
                refs[pb * kRows + row] = new_ref;
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_full[(T + 1) % kSBufs]);  // the next tile's group may take it
                const float alpha = new_ref != last_ref && last_ref != -INFINITY ? fast_exp2(last_ref - new_ref) : 1.f;
                if (new_ref != m_ref) l *= fast_exp2(m_ref - new_ref);  // (0 from -inf)
                m_ref = new_ref;
                const float nmu = new_ref == -INFINITY ? 0.f : -new_ref;
                const uint64_t sl2 = f2_pack(sl, sl), nmu2 = f2_pack(nmu, nmu);
                uint64_t ls2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
                uint32_t pk[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    float a, b;
                    f2_unpack(f2_fma(f2_pack(s[2 * e], s[2 * e + 1]), sl2, nmu2), a, b);
                    pk[e] = pack_bf16x2(fast_exp2(a), fast_exp2(b));
                    ls2[e & 1] = f2_add(ls2[e & 1], f2_pack(bf16lo_to_f32(pk[e]), bf16hi_to_f32(pk[e])));
                }
                // off to CTA 1 once the buffer's last weights are multiplied (waited for
                // here and not before the scores are read: the way from those products
                // through a softmax to these took two tiles' time)
                if (T >= kPBufs && !(ok = lat_wait_cluster(&p_free[pb], ((T / kPBufs) + 1) & 1, p))) break;
                const uint32_t bar = p_full_peer + 8 * pb, dst = p_peer + pb * kPBytes;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    st_async(dst + i * (kRows * 16), bar, pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                st_async1(alpha_peer + pb * (kRows * 4), bar, __float_as_uint(alpha));
                sent = T + 1;
                float l0, l1, l2, l3;
                f2_unpack(ls2[0], l0, l1);
                f2_unpack(ls2[1], l2, l3);
                l += (l0 + l1) + (l2 + l3);
            }
            if (!ok) break;
            const int32_t Tl = end - 1;
            if ((Tl & 1) != g) {
                // the other group has the piece's last tile: this group's sums go to it
                sums[row] = make_float2(m_ref, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(l_full);
                if (!(ok = lat_wait_cluster(&s_full[Tl % kSBufs], (Tl / kSBufs) & 1, p))) break;  // Q has been read
            } else {
                if (!(ok = lat_wait(l_full, k & 1, p))) break;
                const float2 o = sums[row];
                l += o.x == m_ref ? o.y : o.y * fast_exp2(o.x - m_ref);  // (0 from -inf)
                if (!pc.whole) {
                    if (row < it.n) latent_part_ml<kRows>(p, worker, pc.slot)[row] = make_float2(weight_max(m_ref, l), l);
                } else if (warp_live) {
                    // (CTA 1 has read the sums of kFins pieces ago: the last weights went
                    // after the products of the tile two before, hence after the
                    // epilogue before that tile's piece)
                    st_async1(fin_peer + (k % kFins) * (kRows * 4), fin_full_peer + 8 * (k % kFins), __float_as_uint(l));
                }
            }
            T0 = end;
        }
        // CTA 1's last arrivals have come (a group's first warp has pairs in every piece)
        if (ok && w == 0 && sent > 0) lat_wait_cluster(&p_free[(sent - 1) % kPBufs], ((sent - 1) / kPBufs) & 1, p);
    } else if (warp >= 4) {
        // ------------------------------------------------------------ values (CTA 1)
        const int half = (warp >> 2) - 1, w = warp & 3, row = 32 * w + lane;
        const uint32_t lane_base = static_cast<uint32_t>(32 * w) << 16;
        const uint32_t ox = tmem + lane_base + half * (R / 2);
        const float *alphas = reinterpret_cast<const float *>(smem + L::kAlphaOff);
        const float *fins = reinterpret_cast<const float *>(smem + L::kFinOff);
        const int tid = threadIdx.x - 128;
        const bool arms = warp == 4 && lane == 0;
        int32_t T = 0, Tp = 0;   // Tp: the tile whose weights are waited for next
        uint32_t fin_phase = 0;  // bit b: parity of fin_full[b]'s next phase
        for (int32_t k = 0; ok && latent_next<kRows, kKeys>(p, run, pc); ++k) {
            const LatentItem &it = pc.it;
            const uint32_t live_warps = static_cast<uint32_t>((it.n + 31) / 32);
            const bool warp_live = 32 * w < it.n, live = row < it.n;
            for (int32_t j = 0; j < pc.n; ++j, ++T) {
                const int st = T % kStages, pb = T % kPBufs;
                const int32_t tbase = (pc.t0 + j) * kKeys;
                if (arms) mbar_arrive_expect_tx(&p_full[pb], live_warps * (32 * kKeys * 2 + 32 * 4));
                ok = lat_wait(&kv_full[st], (T / kStages) & 1, p);
                // value rows of keys past the item's or of pages not loaded hold stale
                // slots (possibly NaN): zeroed before the tile's products read them
                if (ok) {
                    const uint32_t mask = kmask[T % kMasks];
                    if (mask != all_pages || tbase + kKeys > it.hi) {
                        const int kr = tid & (kKeys - 1), quarter = tid >> 6;
                        if (tbase + kr >= it.hi || !((mask >> (kr / bs)) & 1u)) {
                            uint8_t *v = smem + st * 8 * L::kGroup1 + (kr >> 3) * L::kGroup1 + quarter * (NR / 4) * 1024 + (kr & 7) * 128;
#pragma unroll
                            for (int i = 0; i < NR / 4; ++i)
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                    *reinterpret_cast<uint4 *>(v + i * 1024 + c * 16) = make_uint4(0, 0, 0, 0);
                        }
                    }
                }
                ok = ok && lat_wait_cluster(&p_full[pb], (T / kPBufs) & 1, p);
                if (!ok) break;
                Tp = T + 1;
                const float alpha = warp_live ? alphas[pb * kRows + row] : 1.f;
                if (j > 0 && __any_sync(0xffffffffu, live && alpha != 1.f)) {
                    // O holds P.V up to the last tile once that product completes
                    if (!(ok = lat_wait(pv_done, (T - 1) & 1, p))) break;
                    tc::fence_after();
#pragma unroll 1
                    for (int c = 0; c < R / 2; c += 32) {
                        uint32_t r[32];
                        tc::ld32(ox + c, r);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
                        tc::st32(ox + c, r);
                    }
                    tc::wait_st();
                }
                fence_proxy_async_smem();  // the weights and zeroed rows, before the tensor cores read them
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[pb]);
            }
            if (!ok) break;
            // epilogue, once the piece's last product is in (a parity names one
            // phase only: o_done completes once a piece, its next needs this warp)
            const int fb = k % kFins;
            if (pc.whole && arms) mbar_arrive_expect_tx(&fin_full[fb], live_warps * 128);
            ok = lat_wait(o_done, k & 1, p);
            if (ok && pc.whole) ok = lat_wait_cluster(&fin_full[fb], (fin_phase >> fb) & 1, p);
            if (!ok) break;
            if (pc.whole) fin_phase ^= 1u << fb;
            tc::fence_after();
            if (pc.whole) {
                const float l = live ? fins[fb * kRows + row] : 0.f;
                const float inv = l != 0.f ? 1.f / l : 0.f;  // (NaN stays NaN)
                // a thread's 64 bytes change places with those of its three neighbours, so
                // that a store covers 64 bytes of 8 pairs and not 16 of 32
                const int first = 32 * w + (lane & ~3), b = lane & 3;
                uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + latent_out_row(p, it, first) +
                                                       half * (R / 2)) + b;
#pragma unroll 1
                for (int c = 0; warp_live && c < R / 2; c += 32) {
                    uint32_t r[32];
                    tc::ld32(ox + c, r);
                    tc::wait_ld();
                    uint4 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[e] = pack_bf16x2(__uint_as_float(r[8 * i + 2 * e]) * inv,
                                               __uint_as_float(r[8 * i + 2 * e + 1]) * inv);
                        v[i] = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                    quad_transpose(v, b);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (first + i < it.n) out[i * (R / 8) + c / 8] = v[i];
                }
            } else {
                // a partial: value quads of 32 pairs side by side
                float4 *dst = latent_part_o<kRows>(p, worker, pc.slot) + (half * (R / 8)) * kRows + row;
#pragma unroll 1
                for (int c = 0; warp_live && c < R / 2; c += 32) {
                    uint32_t r[32];
                    tc::ld32(ox + c, r);
                    tc::wait_ld();
                    if (!live) continue;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        dst[(c / 4 + i) * kRows] =
                            make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                        __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
                }
            }
            tc::fence_before();
        }
        // wind-down after a wait ran out: what CTA 0 may still be sending lands (or the
        // limit passes) before this CTA's shared memory goes
        if (!ok)
            for (int32_t t = Tp; t < Tp + kPBufs; ++t) wait_cluster(&p_full[t % kPBufs], (t / kPBufs) & 1, kWaitLimitNs);
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

template <int NR>
static cudaError_t launch(const LatentParams &p, const CUtensorMap &map0, const CUtensorMap &map1, const CUtensorMap &q_map,
                          cudaStream_t stream)
{
    constexpr int smem = lt::Layout<NR>::kBytes;
    cudaError_t err = kernel_smem<latent_tc_kernel<NR>>(smem);
    if (err != cudaSuccess) return err;
    prof_begin(PKV_KERNEL_LATENT, stream);
    err = launch_pdl(latent_tc_kernel<NR>, dim3(static_cast<unsigned>(2 * p.workers)), dim3(lt::kThreads), smem, stream, map0,
                     map1, q_map, p);
    if (err == cudaSuccess)
        err = launch_latent_merge<__nv_bfloat16, lt::kRows>(p, stream);
    prof_end(PKV_KERNEL_LATENT, stream);
    return err;
}

cudaError_t launch_latent_tc(const LatentParams &p, const CUtensorMap &map0, const CUtensorMap &map1, const CUtensorMap &q_map,
                          cudaStream_t stream)
{
    return p.latent == 512 ? launch<8>(p, map0, map1, q_map, stream) : launch<4>(p, map0, map1, q_map, stream);
}

}  // namespace pkv
