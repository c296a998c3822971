// C ABI entry points: argument checks, the split plan, TMA descriptors and
// kernel launches.  Everything here runs on the host; nothing allocates
// device memory and nothing synchronises the stream.
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>
#include <vector>

#include <cudaTypedefs.h>

#include "pkv.h"
#include "pkv_internal.h"


using namespace pkv;

namespace {

std::atomic<int32_t> g_split_override{0};
// diagnostic drill (pkv_set_wait_drill): data-wait limit and flags
std::atomic<uint64_t> g_drill_wait_ns{kWaitLimitNs};
std::atomic<uint32_t> g_drill_flags{0};

// ---------------------------------------------------------------------------
// launch counting and optional per-kind event timing
// ---------------------------------------------------------------------------
std::atomic<int64_t> g_launches{0};
std::atomic<uint32_t> g_prof_mask{0};
struct ProfRecord {
    int kind;
    cudaEvent_t start, stop;
};
std::mutex g_prof_mu;
std::vector<ProfRecord> g_prof_records;
std::vector<cudaEvent_t> g_prof_free;
cudaEvent_t g_prof_pending[PKV_KERNEL_KINDS] = {};
constexpr size_t kMaxProfRecords = 65536;

cudaEvent_t take_event()
{
    if (!g_prof_free.empty()) {
        cudaEvent_t e = g_prof_free.back();
        g_prof_free.pop_back();
        return e;
    }
    cudaEvent_t e = nullptr;
    if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
    return e;
}

int num_sms_current()
{
    // per-device cache; host threads may call concurrently
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64) {
        const int c = cache[dev].load(std::memory_order_relaxed);
        if (c > 0) return c;
    }
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool valid_pool(const pkv_pool *pool)
{
    if (pool == nullptr || pool->k == nullptr || pool->v == nullptr) return false;
    if (pool->num_blocks <= 0 || pool->block_size <= 0 || pool->num_kv_heads <= 0 ||
        pool->head_dim <= 0)
        return false;
    if (pool->dtype != PKV_F32 && pool->dtype != PKV_BF16 && pool->dtype != PKV_FP8_E4M3)
        return false;
    if (pool->dtype == PKV_FP8_E4M3 &&
        (!(std::isfinite(pool->k_scale) && pool->k_scale > 0.f) ||
         !(std::isfinite(pool->v_scale) && pool->v_scale > 0.f)))
        return false;
    return aligned16(pool->k) && aligned16(pool->v);
}

// FP8 pools have one tile layout: 16-token blocks, head_dim a multiple of 64
bool fp8_shape_built(const pkv_pool *pool)
{
    return pool->block_size == 16 &&
           (pool->head_dim == 64 || pool->head_dim == 128 || pool->head_dim == 256);
}

// Element type of queries and outputs: bf16 beside FP8 pools, else the pool's own.
pkv_dtype out_dtype(pkv_dtype t) { return t == PKV_FP8_E4M3 ? PKV_BF16 : t; }

int elem_bytes(pkv_dtype t) { return t == PKV_FP8_E4M3 ? 1 : (t == PKV_BF16 ? 2 : 4); }

// Which decode shapes are built.
bool decode_shape_built(pkv_dtype dtype, int32_t D, int32_t bs, int32_t G)
{
    if (G < 1 || G > 16) return false;
    if (dtype == PKV_BF16 || dtype == PKV_FP8_E4M3)
        return bs == 16 && (D == 64 || D == 128 || D == 256);
    return (D == 32 || D == 64 || D == 128 || D == 256) && bs <= 64 && bs * D <= 4096;
}

// The most blocks a row's key range can have.
int64_t plan_blocks(int32_t max_len, int32_t bs, int32_t window, int32_t sinks)
{
    int64_t n = ceil_div64(max_len, bs);
    if (window > 0) n = std::min<int64_t>(n, ceil_div64(window, bs) + 1 + ceil_div64(sinks, bs));
    return std::max<int64_t>(n, 1);
}

// How a plan cuts its rows: split sizes come to about `target` CTAs and at least
// `least` blocks.
struct SplitRule {
    bool few;  // fewer (row, kv head) pairs than SMs
    int64_t target, least;
};

SplitRule split_rule(int64_t pairs, int num_sms)
{
    const bool few = pairs < num_sms;
    return {few, static_cast<int64_t>(std::max(num_sms, 1)) * (few ? 2 : 9), few ? 4 : 8};
}

// The split plan: a pure function of the sizes and the SM count.
DecodePlan make_plan(int32_t batch, int32_t hq, int32_t hkv, int32_t D, int32_t bs,
                     int32_t max_len, int32_t window, const pkv_prefix_desc *prefix,
                     pkv_dtype dtype, int num_sms, int32_t sinks = 0)
{
    DecodePlan pl{};
    const int32_t G = hq / hkv;
    const int64_t nblk_max = plan_blocks(max_len, bs, window, sinks);
    const int64_t tiles_ub = static_cast<int64_t>(batch) * nblk_max * hkv;
    // Split size over the upper bound of (block, kv head) tiles, a multiple of
    // the consumer warp count.  Many (row, kv head) pairs: about nine CTAs
    // per SM (three waves of three resident CTAs), so that rows of unequal
    // length even out, and at least 8 blocks per split (measured on 32 rows of
    // 1-8k tokens: 96 blocks per split beat 64, 72, 80, 108 and 128, for one
    // query per row and for four).  Fewer pairs than SMs (a few long rows):
    // two CTAs per SM, one wave, since each CTA pays a fixed start-up cost
    // and the merge reads every partial; at least 4 blocks per split.
    const SplitRule rule = split_rule(static_cast<int64_t>(batch) * hkv, num_sms);
    const bool few = rule.few;
    int64_t C = ceil_div64(tiles_ub, rule.target);
    C = std::max<int64_t>(C, rule.least);
    C = ceil_div64(C, kDecodeWarps) * kDecodeWarps;
    const int32_t ov = g_split_override.load();
    if (ov > 0) C = ov;
    pl.split_blocks = static_cast<int32_t>(C);
    pl.few = few ? 1 : 0;
    pl.n_suffix_splits = static_cast<int32_t>(ceil_div64(nblk_max, C));
    pl.prefix_split_blocks = 8;
    pl.n_prefix_splits = 0;
    pl.prefix_chunks = 0;
    pl.n_prefix_ctas = 0;
    if (prefix != nullptr && prefix->num_groups > 0 && prefix->max_prefix_blocks > 0) {
        // The prefix cut (blocks per prefix split) is sized for a nominal 64
        // (row, head) pairs per CTA (32 at head_dim 256), about one CTA per SM
        // at that size, whatever the dtype, so that the workspace size does
        // not depend on the dtype.  The row chunks then follow the kernel: the
        // bf16 and FP8 kernels take four warp tiles of 8 pairs (G <= 8) or 16
        // per CTA, so at G <= 8 the prefix CTAs come to about two per SM; the
        // f32 kernel takes 16 pairs per CTA.
        const int64_t rows_pairs = static_cast<int64_t>(prefix->max_group_rows) * G;
        const int64_t pairs_bf16 = D == 256 ? kPrefixPairsPerCta / 2 : kPrefixPairsPerCta;
        const int64_t chunks_bf16 = ceil_div64(rows_pairs, pairs_bf16);
        int64_t Cp = ceil_div64(static_cast<int64_t>(prefix->max_prefix_blocks) * hkv *
                                    prefix->num_groups * chunks_bf16,
                                std::max(num_sms, 1));
        Cp = std::min<int64_t>(std::max<int64_t>(Cp, 4), 64);
        int64_t chunks = ceil_div64(rows_pairs, kF32Rows);
        if (dtype != PKV_F32)
            chunks = ceil_div64(rows_pairs, static_cast<int64_t>(kDecodeWarps) * 8 * query_ntiles(G));
        pl.prefix_split_blocks = static_cast<int32_t>(Cp);
        pl.n_prefix_splits = static_cast<int32_t>(ceil_div64(prefix->max_prefix_blocks, Cp));
        pl.prefix_chunks = static_cast<int32_t>(chunks);
        pl.prefix_max = prefix->max_prefix_blocks;
        pl.n_prefix_ctas = static_cast<int64_t>(pl.n_prefix_splits) * hkv * prefix->num_groups * chunks;
    }
    pl.nslot = pl.n_prefix_splits + pl.n_suffix_splits;
    pl.n_suffix_ctas = static_cast<int64_t>(pl.n_suffix_splits) * hkv * batch;
    // The cooperative kernel (its warps share every block) for long runs, or
    // for a grid under half the SMs; runs of 16 blocks over a full grid
    // (4 rows x 2048 tokens) were faster on the many-row kernel (17.4 against
    // 18.9 us per call), runs of 28 (4 rows x 32768) and the 4-block runs of a
    // 512-token window slower (35.9 against 33.4, 15.4 against 12.6 us).
    pl.coop = few && (C >= 24 || 2 * pl.n_suffix_ctas < num_sms) ? 1 : 0;
    return pl;
}

size_t ws_o_bytes(int32_t batch, int32_t hq, int32_t D, const DecodePlan &pl)
{
    const size_t b = static_cast<size_t>(batch) * hq * pl.nslot * D * sizeof(float);
    return (b + 255) & ~static_cast<size_t>(255);
}

size_t ws_total_bytes(int32_t batch, int32_t hq, int32_t D, const DecodePlan &pl)
{
    return ws_o_bytes(batch, hq, D, pl) + static_cast<size_t>(batch) * hq * pl.nslot * 2 * sizeof(float);
}

// Bytes to report for calls of these sizes: enough for every plan over lengths
// up to max_len.  A call plans with its own bound (its table may hold less than
// max_len), and a shorter row can take more splits than a longer one, as the
// split size moves in steps: 76 blocks in splits of 12 are 7, 72 in splits of 8
// are 9.  A plan of n blocks has splits of C >= max(least, n * pairs / target), so
// at most min(ceil(n / least), ceil(target / pairs)) of them.
size_t ws_query_bytes(int32_t batch, int32_t hq, int32_t hkv, int32_t D, int32_t bs, int32_t max_len,
                      int32_t window, const pkv_prefix_desc *prefix, int32_t sinks, int32_t queries = 1)
{
    const int sms = num_sms_current();
    DecodePlan pl = make_plan(batch, hq, hkv, D, bs, max_len, window, prefix, PKV_BF16, sms, sinks);
    const int64_t pairs = static_cast<int64_t>(batch) * hkv;
    if (pairs > 0 && g_split_override.load() == 0) {
        const SplitRule rule = split_rule(pairs, sms);
        pl.n_suffix_splits = static_cast<int32_t>(
            std::min(ceil_div64(plan_blocks(max_len, bs, window, sinks), rule.least), ceil_div64(rule.target, pairs)));
        pl.nslot = pl.n_prefix_splits + pl.n_suffix_splits;
    }
    return ws_total_bytes(batch * queries, hq, D, pl);
}

bool valid_prefix(const pkv_prefix_desc *prefix, int32_t batch, int32_t width)
{
    if (prefix == nullptr || prefix->num_groups == 0) return true;
    if (prefix->num_groups < 0 || prefix->num_groups > batch) return false;
    if (prefix->group_of_row == nullptr || prefix->prefix_blocks == nullptr) return false;
    if (prefix->max_group_rows < 1 || prefix->max_group_rows > batch) return false;
    if (prefix->max_prefix_blocks < 0 || prefix->max_prefix_blocks > width) return false;
    return true;
}

// ---------------------------------------------------------------------------
// TMA descriptors
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

bool encode_fn_ready()
{
    std::call_once(g_encode_once, [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return g_encode != nullptr;
}

// 4-D map over a bf16 pool [num_blocks][hkv][bs][D], box 64 dims x bs slots,
// 128-byte swizzle.
bool encode_pool_map(CUtensorMap *map, void *base, const pkv_pool &pool)
{
    const cuuint64_t D = pool.head_dim, bs = pool.block_size, hkv = pool.num_kv_heads;
    cuuint64_t dims[4] = {D, bs, hkv, static_cast<cuuint64_t>(pool.num_blocks)};
    cuuint64_t strides[3] = {D * 2, bs * D * 2, hkv * bs * D * 2};
    cuuint32_t box[4] = {64, static_cast<cuuint32_t>(bs), 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box,
                                estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// 5-D view of the same pool for whole-tile boxes: (64 dims, slot, 64-dim
// region, kv head, block), box (64, bs, D/64, 1, 1).  The region stride (128 B)
// is smaller than the slot stride: the box walks dims, then slots, then
// regions, so a (block, kv head) tile lands region by region, each region
// [bs][64] with the 128-byte swizzle, in one load.
bool encode_pool_map_tile(CUtensorMap *map, void *base, const pkv_pool &pool)
{
    const cuuint64_t D = pool.head_dim, bs = pool.block_size, hkv = pool.num_kv_heads;
    cuuint64_t dims[5] = {64, bs, D / 64, hkv, static_cast<cuuint64_t>(pool.num_blocks)};
    cuuint64_t strides[4] = {D * 2, 128, bs * D * 2, hkv * bs * D * 2};
    cuuint32_t box[5] = {64, static_cast<cuuint32_t>(bs), static_cast<cuuint32_t>(D / 64), 1, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, base, dims, strides, box,
                                estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// Validation and parameters of one decode call (no launch).  batch == 0
// returns PKV_OK with nothing filled.
pkv_status decode_setup(const void *q, int32_t num_q_heads, const pkv_pool *pool,
                        const int32_t *block_tables, int32_t max_blocks_per_seq,
                        const int32_t *seq_lens, int32_t batch, int32_t max_seq_len,
                        int32_t window, float scale, void *out, void *workspace, size_t ws_bytes,
                        const pkv_prefix_desc *prefix, int32_t *dev_status, DecodeParams *pp,
                        int32_t sinks = 0)
{
    if (!valid_pool(pool) || batch < 0 || num_q_heads <= 0 || max_seq_len < 0 || window < 0 ||
        sinks < 0 || !std::isfinite(scale))
        return PKV_ERR_INVALID_ARG;
    if (window == 0) sinks = 0;  // full attention sees every position
    if (num_q_heads % pool->num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    if (batch == 0) return PKV_OK;
    if (q == nullptr || out == nullptr || block_tables == nullptr || seq_lens == nullptr ||
        max_blocks_per_seq <= 0 || !aligned16(q) || !aligned16(out))
        return PKV_ERR_INVALID_ARG;
    if (!valid_prefix(prefix, batch, max_blocks_per_seq)) return PKV_ERR_INVALID_ARG;
    const bool use_prefix = prefix != nullptr && prefix->num_groups > 0;
    if (use_prefix && window != 0) return PKV_ERR_UNSUPPORTED;
    const int32_t G = num_q_heads / pool->num_kv_heads;
    if (!decode_shape_built(pool->dtype, pool->head_dim, pool->block_size, G))
        return PKV_ERR_UNSUPPORTED;
    const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * pool->block_size;
    const int32_t max_len = static_cast<int32_t>(std::min<int64_t>(max_seq_len, cap));

    const DecodePlan pl = make_plan(batch, num_q_heads, pool->num_kv_heads, pool->head_dim,
                                    pool->block_size, max_len, window,
                                    use_prefix ? prefix : nullptr, pool->dtype, num_sms_current(), sinks);
    if (pl.n_suffix_ctas > INT32_MAX || pl.n_prefix_ctas > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    const size_t need = ws_total_bytes(batch, num_q_heads, pool->head_dim, pl);
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        ws_bytes < need)
        return PKV_ERR_WORKSPACE;

    DecodeParams &p = *pp;
    p = DecodeParams{};
    p.q = q;
    p.out = out;
    p.k_pool = pool->k;
    p.v_pool = pool->v;
    p.tables = block_tables;
    p.seq_lens = seq_lens;
    p.group_of_row = use_prefix ? prefix->group_of_row : nullptr;
    p.prefix_blocks = use_prefix ? prefix->prefix_blocks : nullptr;
    p.num_groups = use_prefix ? prefix->num_groups : 0;
    p.ws_o = static_cast<float *>(workspace);
    p.ws_ml = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                        ws_o_bytes(batch, num_q_heads, pool->head_dim, pl));
    p.status = dev_status;
    p.cu_q_lens = nullptr;  // one query per row
    p.max_q = 1;
    p.batch = batch;
    p.hq = num_q_heads;
    p.hkv = pool->num_kv_heads;
    p.group = G;
    p.head_dim = pool->head_dim;
    p.block_size = pool->block_size;
    p.width = max_blocks_per_seq;
    p.num_blocks = pool->num_blocks;
    p.max_len = max_len;
    p.window = window;
    p.sinks = sinks;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.v_scale = 1.f;
    if (pool->dtype == PKV_FP8_E4M3) {
        p.scale_log2 *= pool->k_scale;
        p.v_scale = pool->v_scale;
    }
    drill_settings(&p.wait_ns, &p.drill);
    p.plan = pl;
    return PKV_OK;
}

// One validated decode call's launches: the split kernel of its pool type, then the merge.
pkv_status decode_launch(const DecodeParams &p, const pkv_pool *pool, pkv_stream_t stream)
{
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t err;
    if (pool->dtype == PKV_FP8_E4M3) {
        err = launch_decode_fp8(p, st);
    } else if (pool->dtype == PKV_BF16) {
        if (!encode_fn_ready()) return PKV_ERR_CUDA;
        CUtensorMap kmap, vmap;
        if (!encode_pool_map_tile(&kmap, pool->k, *pool) ||
            !encode_pool_map_tile(&vmap, pool->v, *pool))
            return PKV_ERR_UNSUPPORTED;
        err = launch_decode_bf16(p, kmap, vmap, st);
    } else {
        err = launch_decode_f32(p, st);
    }
    if (err != cudaSuccess) return PKV_ERR_CUDA;
    err = launch_decode_combine(p, out_dtype(pool->dtype), st);
    return err == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status decode_call(const void *q, int32_t num_q_heads, const pkv_pool *pool,
                       const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *seq_lens,
                       int32_t batch, int32_t max_seq_len, int32_t window, int32_t sinks, float scale,
                       void *out, void *workspace, size_t ws_bytes, const pkv_prefix_desc *prefix,
                       int32_t *dev_status, pkv_stream_t stream)
{
    DecodeParams p{};
    const pkv_status stt = decode_setup(q, num_q_heads, pool, block_tables, max_blocks_per_seq,
                                        seq_lens, batch, max_seq_len, window, scale, out,
                                        workspace, ws_bytes, prefix, dev_status, &p, sinks);
    return stt != PKV_OK || batch == 0 ? stt : decode_launch(p, pool, stream);
}

// Groups of one fused call must share what fixes the kernel instantiation.
bool groups_compatible(const pkv_decode_group *groups, int32_t n)
{
    const pkv_pool &p0 = groups[0].pool;
    for (int32_t i = 1; i < n; ++i) {
        const pkv_pool &pi = groups[i].pool;
        if (pi.dtype != p0.dtype || pi.head_dim != p0.head_dim || pi.block_size != p0.block_size ||
            pi.num_kv_heads != p0.num_kv_heads)
            return false;
    }
    return true;
}

}  // namespace

namespace pkv {

void drill_settings(uint64_t *wait_ns, uint32_t *flags)
{
    *wait_ns = g_drill_wait_ns.load();
    *flags = g_drill_flags.load();
}

void prof_begin(int kind, cudaStream_t stream)
{
    g_launches.fetch_add(1);
    if (!(g_prof_mask.load() & (1u << kind))) return;
    std::lock_guard<std::mutex> lk(g_prof_mu);
    if (g_prof_records.size() >= kMaxProfRecords) return;
    cudaEvent_t e = take_event();
    if (e != nullptr && cudaEventRecord(e, stream) == cudaSuccess) g_prof_pending[kind] = e;
}

void prof_end(int kind, cudaStream_t stream)
{
    if (!(g_prof_mask.load() & (1u << kind))) return;
    std::lock_guard<std::mutex> lk(g_prof_mu);
    cudaEvent_t s = g_prof_pending[kind];
    g_prof_pending[kind] = nullptr;
    if (s == nullptr) return;
    cudaEvent_t e = take_event();
    if (e != nullptr && cudaEventRecord(e, stream) == cudaSuccess)
        g_prof_records.push_back({kind, s, e});
    else
        g_prof_free.push_back(s);
}

}  // namespace pkv

extern "C" {

pkv_status pkv_set_wait_drill(uint64_t wait_limit_ns, uint32_t flags)
{
    if ((flags & ~static_cast<uint32_t>(PKV_DRILL_WITHHOLD_FIRST_LOAD | PKV_DRILL_LATE_CONSUMERS |
                                        PKV_DRILL_LATE_PRODUCERS)) != 0)
        return PKV_ERR_INVALID_ARG;
    g_drill_wait_ns.store(wait_limit_ns == 0 ? kWaitLimitNs
                                             : std::min<uint64_t>(wait_limit_ns, kWaitLimitNs));
    g_drill_flags.store(flags);
    return PKV_OK;
}

pkv_status pkv_profile_enable(uint32_t kind_mask)
{
    std::lock_guard<std::mutex> lk(g_prof_mu);
    for (auto &r : g_prof_records) {
        g_prof_free.push_back(r.start);
        g_prof_free.push_back(r.stop);
    }
    g_prof_records.clear();
    for (auto &e : g_prof_pending) {
        if (e != nullptr) g_prof_free.push_back(e);
        e = nullptr;
    }
    g_prof_mask.store(kind_mask);
    return PKV_OK;
}

pkv_status pkv_profile_mask(uint32_t kind_mask)
{
    g_prof_mask.store(kind_mask);
    return PKV_OK;
}

pkv_status pkv_profile_read(int32_t kind, int64_t *launches, double *total_ms)
{
    if (kind < 0 || kind >= PKV_KERNEL_KINDS || launches == nullptr || total_ms == nullptr)
        return PKV_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lk(g_prof_mu);
    int64_t n = 0;
    double ms = 0.0;
    for (const auto &r : g_prof_records) {
        if (r.kind != kind) continue;
        float t = 0.f;
        if (cudaEventSynchronize(r.stop) != cudaSuccess ||
            cudaEventElapsedTime(&t, r.start, r.stop) != cudaSuccess)
            return PKV_ERR_CUDA;
        ++n;
        ms += t;
    }
    *launches = n;
    *total_ms = ms;
    return PKV_OK;
}

pkv_status pkv_profile_times(int32_t kind, float *ms_out, int64_t cap, int64_t *launches)
{
    if (kind < 0 || kind >= PKV_KERNEL_KINDS || launches == nullptr || cap < 0 ||
        (cap > 0 && ms_out == nullptr))
        return PKV_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lk(g_prof_mu);
    int64_t n = 0;
    for (const auto &r : g_prof_records) {
        if (r.kind != kind) continue;
        float t = 0.f;
        if (cudaEventSynchronize(r.stop) != cudaSuccess ||
            cudaEventElapsedTime(&t, r.start, r.stop) != cudaSuccess)
            return PKV_ERR_CUDA;
        if (n < cap) ms_out[n] = t;
        ++n;
    }
    *launches = n;
    return PKV_OK;
}

int64_t pkv_launch_count(void) { return g_launches.load(); }


const char *pkv_version(void) { return "pkv 0.1 (sm_103a)"; }

const char *pkv_status_string(pkv_status s)
{
    switch (s) {
    case PKV_OK: return "ok";
    case PKV_ERR_INVALID_ARG: return "invalid argument";
    case PKV_ERR_UNSUPPORTED: return "unsupported dtype/shape combination";
    case PKV_ERR_CUDA: return "CUDA error";
    case PKV_ERR_WORKSPACE: return "workspace too small or misaligned";
    case PKV_ERR_OUT_OF_BLOCKS: return "block pool exhausted at its maximum size (or the block to go on in has expired)";
    case PKV_ERR_HOST_MEMORY: return "out of host memory";
    }
    return "unknown status";
}

int32_t pkv_set_decode_split_blocks(int32_t blocks_per_split)
{
    return g_split_override.exchange(blocks_per_split > 0 ? blocks_per_split : 0);
}

pkv_status paged_kv_append(const pkv_pool *pool, const int32_t *slot_mapping, int32_t num_tokens,
                           const void *k_new, const void *v_new, int32_t *dev_status,
                           pkv_stream_t stream)
{
    if (!valid_pool(pool) || num_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (slot_mapping == nullptr || k_new == nullptr || v_new == nullptr) return PKV_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new)) return PKV_ERR_INVALID_ARG;
    if (pool->dtype == PKV_FP8_E4M3) {
        if (!fp8_shape_built(pool)) return PKV_ERR_UNSUPPORTED;
        if (static_cast<int64_t>(pool->num_blocks) * pool->block_size > INT32_MAX)
            return PKV_ERR_UNSUPPORTED;
        AppendParams p{};
        p.k_pool = pool->k;
        p.v_pool = pool->v;
        p.k_new = k_new;
        p.v_new = v_new;
        p.slot_mapping = slot_mapping;
        p.status = dev_status;
        p.num_tokens = num_tokens;
        p.hkv = pool->num_kv_heads;
        p.block_size = pool->block_size;
        p.num_slots = pool->num_blocks * pool->block_size;
        p.head_dim = pool->head_dim;
        p.k_scale = pool->k_scale;
        p.v_scale = pool->v_scale;
        return launch_append_fp8(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
                   ? PKV_OK
                   : PKV_ERR_CUDA;
    }
    const int64_t row_bytes = static_cast<int64_t>(pool->head_dim) * elem_bytes(pool->dtype);
    if (row_bytes % 16 != 0) return PKV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(pool->num_blocks) * pool->block_size > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    AppendParams p{};
    p.k_pool = pool->k;
    p.v_pool = pool->v;
    p.k_new = k_new;
    p.v_new = v_new;
    p.slot_mapping = slot_mapping;
    p.status = dev_status;
    p.num_tokens = num_tokens;
    p.hkv = pool->num_kv_heads;
    p.block_size = pool->block_size;
    p.vecs_per_row = static_cast<int32_t>(row_bytes / 16);
    p.num_slots = pool->num_blocks * pool->block_size;
    return launch_append(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PKV_OK
                                                                                  : PKV_ERR_CUDA;
}

int32_t pkv_decode_plan(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                        int32_t block_size, int32_t max_seq_len, int32_t window,
                        int32_t *blocks_per_split_out)
{
    if (batch < 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 || head_dim <= 0 ||
        block_size <= 0 || max_seq_len < 0 || window < 0)
        return -1;
    const DecodePlan pl = make_plan(batch, num_q_heads, num_kv_heads, head_dim, block_size,
                                    max_seq_len, window, nullptr, PKV_BF16, num_sms_current());
    if (blocks_per_split_out) *blocks_per_split_out = pl.split_blocks;
    return pl.n_suffix_splits;
}

size_t paged_decode_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                   int32_t head_dim, int32_t block_size, int32_t max_seq_len,
                                   int32_t window, const pkv_prefix_desc *prefix)
{
    if (batch < 0 || num_kv_heads <= 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        head_dim <= 0 || block_size <= 0 || max_seq_len < 0 || window < 0)
        return 0;
    // the f32, bf16 and FP8 plans differ only in how many CTAs cover a
    // prefix group's rows, which does not change the slot count: the size
    // holds for every pool dtype
    return ws_query_bytes(batch, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len, window,
                          prefix, 0);
}

pkv_status paged_decode_attention(const void *q, int32_t num_q_heads, const pkv_pool *pool,
                                  const int32_t *block_tables, int32_t max_blocks_per_seq,
                                  const int32_t *seq_lens, int32_t batch, int32_t max_seq_len,
                                  int32_t window, float scale, void *out, void *workspace,
                                  size_t ws_bytes, const pkv_prefix_desc *prefix,
                                  int32_t *dev_status, pkv_stream_t stream)
{
    return decode_call(q, num_q_heads, pool, block_tables, max_blocks_per_seq, seq_lens, batch,
                       max_seq_len, window, 0, scale, out, workspace, ws_bytes, prefix, dev_status,
                       stream);
}

size_t paged_decode_sinks_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t block_size, int32_t max_seq_len,
                                         int32_t window, int32_t sinks)
{
    if (batch < 0 || num_kv_heads <= 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        head_dim <= 0 || block_size <= 0 || max_seq_len < 0 || window < 0 || sinks < 0)
        return 0;
    return ws_query_bytes(batch, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len, window,
                          nullptr, window > 0 ? sinks : 0);
}

pkv_status paged_decode_attention_sinks(const void *q, int32_t num_q_heads, const pkv_pool *pool,
                                        const int32_t *block_tables, int32_t max_blocks_per_seq,
                                        const int32_t *seq_lens, int32_t batch, int32_t max_seq_len,
                                        int32_t window, int32_t sinks, float scale, void *out,
                                        void *workspace, size_t ws_bytes, int32_t *dev_status,
                                        pkv_stream_t stream)
{
    return decode_call(q, num_q_heads, pool, block_tables, max_blocks_per_seq, seq_lens, batch,
                       max_seq_len, window, sinks, scale, out, workspace, ws_bytes, nullptr,
                       dev_status, stream);
}

size_t paged_decode_groups_sinks_workspace_size(const pkv_decode_group *groups, const int32_t *sinks,
                                                int32_t n_groups, int32_t batch, int32_t num_q_heads)
{
    if (groups == nullptr || n_groups < 1 || n_groups > PKV_MAX_DECODE_GROUPS || batch < 0)
        return 0;
    size_t total = 0;
    for (int32_t i = 0; i < n_groups; ++i) {
        const pkv_decode_group &g = groups[i];
        const size_t one = paged_decode_sinks_workspace_size(
            batch, num_q_heads, g.pool.num_kv_heads, g.pool.head_dim, g.pool.block_size,
            g.max_seq_len, g.window, sinks != nullptr ? sinks[i] : 0);
        if (one == 0) return 0;
        total += (one + 255) & ~static_cast<size_t>(255);
    }
    return total;
}

size_t paged_decode_groups_workspace_size(const pkv_decode_group *groups, int32_t n_groups,
                                          int32_t batch, int32_t num_q_heads)
{
    return paged_decode_groups_sinks_workspace_size(groups, nullptr, n_groups, batch, num_q_heads);
}

pkv_status paged_decode_attention_groups_sinks(const pkv_decode_group *groups, const int32_t *sinks,
                                               int32_t n_groups, int32_t batch, int32_t num_q_heads,
                                               void *workspace, size_t ws_bytes, int32_t *dev_status,
                                               pkv_stream_t stream)
{
    if (groups == nullptr || n_groups < 1 || n_groups > PKV_MAX_DECODE_GROUPS || batch < 0 ||
        num_q_heads <= 0)
        return PKV_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n_groups; ++i)
        if (!valid_pool(&groups[i].pool) || (sinks != nullptr && sinks[i] < 0)) return PKV_ERR_INVALID_ARG;
    if (!groups_compatible(groups, n_groups)) return PKV_ERR_INVALID_ARG;
    const pkv_dtype dt = groups[0].pool.dtype;
    if (dt == PKV_F32) return PKV_ERR_UNSUPPORTED;  // the CUDA-core f32 kernel runs per call
    if (batch == 0) return PKV_OK;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        ws_bytes < paged_decode_groups_sinks_workspace_size(groups, sinks, n_groups, batch, num_q_heads))
        return PKV_ERR_WORKSPACE;
    if (dt == PKV_BF16 && !encode_fn_ready()) return PKV_ERR_CUDA;

    // groups without sinks share the launches; one with sinks gets its own call's
    GroupedDecode gd{};
    DecodeParams own[PKV_MAX_DECODE_GROUPS];
    const pkv_pool *own_pool[PKV_MAX_DECODE_GROUPS];
    int32_t n_own = 0;
    char *ws = static_cast<char *>(workspace);
    size_t left = ws_bytes;
    int64_t ctas = 0;
    for (int32_t i = 0; i < n_groups; ++i) {
        const pkv_decode_group &g = groups[i];
        DecodeParams p{};
        const pkv_status stt = decode_setup(g.q, num_q_heads, &g.pool, g.block_tables,
                                            g.max_blocks_per_seq, g.seq_lens, batch, g.max_seq_len,
                                            g.window, g.scale, g.out, ws, left, nullptr,
                                            dev_status, &p, sinks != nullptr ? sinks[i] : 0);
        if (stt != PKV_OK) return stt;
        const size_t used = (ws_total_bytes(batch, num_q_heads, g.pool.head_dim, p.plan) + 255) &
                            ~static_cast<size_t>(255);
        ws += used;
        left -= used;
        if (p.sinks > 0) {
            own[n_own] = p;
            own_pool[n_own++] = &g.pool;
            continue;
        }
        const int32_t j = gd.n++;
        gd.g[j] = p;
        ctas += p.plan.n_prefix_ctas + p.plan.n_suffix_ctas;
        gd.cta_end[j] = ctas;
        if (dt == PKV_BF16 && (!encode_pool_map_tile(&gd.kmap[j], g.pool.k, g.pool) ||
                               !encode_pool_map_tile(&gd.vmap[j], g.pool.v, g.pool)))
            return PKV_ERR_UNSUPPORTED;
    }
    if (ctas > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    if (gd.n > 0) {
        cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
        cudaError_t err = dt == PKV_FP8_E4M3 ? launch_decode_fp8_grouped(gd, st)
                                             : launch_decode_bf16_grouped(gd, st);
        if (err != cudaSuccess) return PKV_ERR_CUDA;
        err = launch_decode_combine_grouped(gd, out_dtype(dt), st);
        if (err != cudaSuccess) return PKV_ERR_CUDA;
    }
    for (int32_t i = 0; i < n_own; ++i) {
        const pkv_status stt = decode_launch(own[i], own_pool[i], stream);
        if (stt != PKV_OK) return stt;
    }
    return PKV_OK;
}

pkv_status paged_decode_attention_groups(const pkv_decode_group *groups, int32_t n_groups,
                                         int32_t batch, int32_t num_q_heads, void *workspace,
                                         size_t ws_bytes, int32_t *dev_status, pkv_stream_t stream)
{
    return paged_decode_attention_groups_sinks(groups, nullptr, n_groups, batch, num_q_heads, workspace,
                                               ws_bytes, dev_status, stream);
}

}  // extern "C"

namespace {

// Chunks whose (query, head) pairs of a kv head fit one 16-row decode tile
// (verify steps of a few queries) run on the split-KV decode kernel.
bool verify_on_decode(int32_t G, int32_t D, int32_t bs, int32_t max_q_len)
{
    return max_q_len >= 1 && static_cast<int64_t>(G) * max_q_len <= 16 &&
           decode_shape_built(PKV_BF16, D, bs, G);
}

// Queries of a row that a split item of a drafted tree takes: its 16 rows.
int32_t tree_chunk(int32_t G, int32_t max_q_len) { return std::min(max_q_len, std::max(1, 16 / G)); }

// Drafted trees on the split-KV decode kernel: those of 16 rows, and every one of
// a head_dim that the tensor-core prefill is not built for.  32 trees over 1024 to
// 8192 keys, 32/8 heads of 128: 4 drafts (16 rows) 110 us here, 119 on the tensor-core
// kernel (FP8 91 and 144; one row of 1000 keys 11.3 and 13.3); 5 drafts 167 and 118, 16
// drafts 316 and 111 (FP8 314 and 132).
bool tree_on_decode(int32_t G, int32_t D, int32_t bs, int32_t max_q_len)
{
    return decode_shape_built(PKV_BF16, D, bs, G) &&
           (static_cast<int64_t>(G) * max_q_len <= 16 || !prefill_shape_built(PKV_BF16, D, bs, G));
}

// Items of the tensor-core prefill: (row, kv head, query-tile pair).
int32_t prefill_items(int32_t batch, int32_t hq, int32_t hkv, int32_t max_q_len)
{
    if (hkv <= 0 || hq % hkv != 0) return 0;
    const int32_t qpc = prefill_queries_per_cta(PKV_BF16, hq / hkv);
    const int64_t n = static_cast<int64_t>(batch) * hkv * ((max_q_len + qpc - 1) / qpc);
    return n > INT32_MAX ? 0 : static_cast<int32_t>(n);
}

// The decode plan for a verify step: the key range of a row spans its
// queries' windows.
int32_t verify_window(int32_t window, int32_t max_q_len)
{
    return window > 0 ? static_cast<int32_t>(std::min<int64_t>(static_cast<int64_t>(window) + max_q_len - 1, INT32_MAX))
                      : 0;
}

DecodePlan verify_plan(int32_t batch, int32_t hq, int32_t hkv, int32_t D, int32_t bs,
                       int32_t max_len, int32_t window, int32_t max_q_len, int32_t sinks)
{
    return make_plan(batch, hq, hkv, D, bs, max_len, verify_window(window, max_q_len), nullptr, PKV_BF16,
                     num_sms_current(), sinks);
}

// Bytes of one prefill call's workspace (sinks count with a window only).
size_t prefill_ws(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                  int32_t block_size, int32_t max_q_len, int32_t max_seq_len, int32_t window, int32_t sinks)
{
    if (batch <= 0 || num_kv_heads <= 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        max_q_len <= 0 || max_seq_len < 0 || window < 0 || sinks < 0)
        return 0;
    if (window == 0) sinks = 0;
    // scratch only for short bf16 chunks: the decode kernel's split partials
    // (a few queries per row), or the prefill kernel's key-range runs
    const int32_t G = num_q_heads / num_kv_heads;
    if (verify_on_decode(G, head_dim, block_size, max_q_len))
        return ws_query_bytes(batch, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len,
                              verify_window(window, max_q_len), nullptr, sinks, max_q_len);
    const int sms = num_sms_current();
    const PrefillSplit sp = prefill_split_plan(batch, num_q_heads, num_kv_heads, head_dim, block_size,
                                               max_q_len, max_seq_len, window, sinks, sms);
    const int32_t sk = prefill_sk_ctas(PKV_BF16, batch, num_q_heads, num_kv_heads, head_dim, block_size,
                                       max_q_len, sms);
    return std::max(prefill_split_ws_bytes(batch, num_q_heads, max_q_len, sp),
                    prefill_sk_ws_bytes(prefill_items(batch, num_q_heads, num_kv_heads, max_q_len), sk));
}

}  // namespace

extern "C" {

size_t paged_prefill_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                    int32_t head_dim, int32_t block_size, int32_t max_q_len,
                                    int32_t max_seq_len, int32_t window)
{
    return prefill_ws(batch, num_q_heads, num_kv_heads, head_dim, block_size, max_q_len, max_seq_len,
                      window, 0);
}

size_t paged_prefill_sinks_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                          int32_t head_dim, int32_t block_size, int32_t max_q_len,
                                          int32_t max_seq_len, int32_t window, int32_t sinks)
{
    return prefill_ws(batch, num_q_heads, num_kv_heads, head_dim, block_size, max_q_len, max_seq_len,
                      window, sinks);
}

}  // extern "C"

namespace {

pkv_status prefill_call(const void *q, const int32_t *cu_q_lens, int32_t num_q_heads, const pkv_pool *pool,
                        const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *seq_lens,
                        int32_t batch, int32_t max_q_len, int32_t max_seq_len, int32_t window,
                        int32_t sinks, float scale, void *out, void *workspace, size_t ws_bytes,
                        int32_t *dev_status, pkv_stream_t stream, const uint64_t *tree = nullptr,
                        int32_t num_queries = INT32_MAX)
{
    if (!valid_pool(pool) || batch < 0 || num_q_heads <= 0 || max_q_len < 0 || max_seq_len < 0 ||
        window < 0 || sinks < 0 || !std::isfinite(scale))
        return PKV_ERR_INVALID_ARG;
    if (window == 0) sinks = 0;  // full attention sees every position
    if (num_q_heads % pool->num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    if (batch == 0 || max_q_len == 0) return PKV_OK;
    if (q == nullptr || out == nullptr || cu_q_lens == nullptr || block_tables == nullptr ||
        seq_lens == nullptr || max_blocks_per_seq <= 0 || !aligned16(q) || !aligned16(out))
        return PKV_ERR_INVALID_ARG;
    const int32_t G = num_q_heads / pool->num_kv_heads;
    const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * pool->block_size;
    if (pool->dtype != PKV_F32 &&
        (tree != nullptr ? tree_on_decode(G, pool->head_dim, pool->block_size, max_q_len)
                         : verify_on_decode(G, pool->head_dim, pool->block_size, max_q_len))) {
        // a few queries per row: the split-KV decode kernel with (query, head)
        // M-rows, then its merge
        const int32_t max_len = static_cast<int32_t>(std::min<int64_t>(max_seq_len, cap));
        DecodePlan pl = verify_plan(batch, num_q_heads, pool->num_kv_heads, pool->head_dim,
                                    pool->block_size, max_len, window, max_q_len, sinks);
        const int32_t q_chunk = tree != nullptr ? tree_chunk(G, max_q_len) : max_q_len;
        const int32_t q_chunks = (max_q_len + q_chunk - 1) / q_chunk;
        pl.n_suffix_ctas *= q_chunks;
        if (pl.n_suffix_ctas > INT32_MAX) return PKV_ERR_UNSUPPORTED;
        const int32_t prow = batch * max_q_len;
        const size_t need = ws_total_bytes(prow, num_q_heads, pool->head_dim, pl);
        if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
            ws_bytes < need)
            return PKV_ERR_WORKSPACE;
        DecodeParams d{};
        d.q = q;
        d.out = out;
        d.k_pool = pool->k;
        d.v_pool = pool->v;
        d.tables = block_tables;
        d.seq_lens = seq_lens;
        d.group_of_row = nullptr;
        d.prefix_blocks = nullptr;
        d.num_groups = 0;
        d.ws_o = static_cast<float *>(workspace);
        d.ws_ml = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                            ws_o_bytes(prow, num_q_heads, pool->head_dim, pl));
        d.status = dev_status;
        d.cu_q_lens = cu_q_lens;
        d.max_q = max_q_len;
        d.batch = batch;
        d.hq = num_q_heads;
        d.hkv = pool->num_kv_heads;
        d.group = G;
        d.head_dim = pool->head_dim;
        d.block_size = pool->block_size;
        d.width = max_blocks_per_seq;
        d.num_blocks = pool->num_blocks;
        d.max_len = max_len;
        d.window = window;
        d.sinks = sinks;
        d.tree = tree;
        d.q_chunk = q_chunk;
        d.q_chunks = q_chunks;
        d.num_queries = num_queries;
        d.scale_log2 = scale * 1.4426950408889634f;
        d.v_scale = 1.f;
        drill_settings(&d.wait_ns, &d.drill);
        d.plan = pl;
        cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
        cudaError_t err;
        if (pool->dtype == PKV_FP8_E4M3) {
            d.scale_log2 *= pool->k_scale;
            d.v_scale = pool->v_scale;
            err = tree != nullptr ? launch_tree_fp8(d, st) : launch_decode_fp8(d, st);
        } else {
            if (!encode_fn_ready()) return PKV_ERR_CUDA;
            CUtensorMap kmap, vmap;
            if (!encode_pool_map_tile(&kmap, pool->k, *pool) ||
                !encode_pool_map_tile(&vmap, pool->v, *pool))
                return PKV_ERR_UNSUPPORTED;
            err = tree != nullptr ? launch_tree_bf16(d, kmap, vmap, st) : launch_decode_bf16(d, kmap, vmap, st);
        }
        if (err == cudaSuccess) err = launch_decode_combine(d, out_dtype(pool->dtype), st);
        return err == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
    }
    if (!prefill_shape_built(pool->dtype, pool->head_dim, pool->block_size, G))
        return PKV_ERR_UNSUPPORTED;
    PrefillParams p{};
    p.q = q;
    p.out = out;
    p.k_pool = pool->k;
    p.v_pool = pool->v;
    p.cu_q_lens = cu_q_lens;
    p.tables = block_tables;
    p.seq_lens = seq_lens;
    p.status = dev_status;
    p.batch = batch;
    p.hq = num_q_heads;
    p.hkv = pool->num_kv_heads;
    p.group = G;
    p.head_dim = pool->head_dim;
    p.block_size = pool->block_size;
    p.width = max_blocks_per_seq;
    p.num_blocks = pool->num_blocks;
    p.max_len = static_cast<int32_t>(std::min<int64_t>(max_seq_len, cap));
    p.max_q_len = max_q_len;
    p.window = window;
    p.sinks = sinks;
    p.tree = tree;
    p.num_queries = num_queries;
    const int32_t qpt = prefill_queries_per_cta(pool->dtype, G);
    p.q_tiles = static_cast<int32_t>(ceil_div64(max_q_len, qpt));
    p.kv_splits = 1;
    p.split_tiles = 0;
    if (pool->dtype != PKV_F32 && tree == nullptr) {
        const PrefillSplit sp = prefill_split_plan(batch, num_q_heads, pool->num_kv_heads,
                                                   pool->head_dim, pool->block_size, max_q_len,
                                                   p.max_len, window, sinks, num_sms_current());
        if (sp.splits > 1) {
            const size_t need = prefill_split_ws_bytes(batch, num_q_heads, max_q_len, sp);
            if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
                ws_bytes < need)
                return PKV_ERR_WORKSPACE;
            p.kv_splits = sp.splits;
            p.split_tiles = sp.tiles;
            const size_t n = static_cast<size_t>(batch) * max_q_len * num_q_heads * sp.splits;
            p.ws_o = static_cast<float *>(workspace);
            p.ws_ml = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                                ((n * pool->head_dim * sizeof(float) + 255) &
                                                 ~static_cast<size_t>(255)));
        }
    }
    p.scale_log2 = scale * 1.4426950408889634f;
    p.v_scale = 1.f;
    if (pool->dtype == PKV_FP8_E4M3) {
        p.scale_log2 *= pool->k_scale;
        p.v_scale = pool->v_scale;
    }
    drill_settings(&p.wait_ns, &p.drill);
    p.sk_ctas = 0;
    p.sk_items = 0;
    if (pool->dtype != PKV_F32 && tree != nullptr) {
        const int32_t items = prefill_items(batch, num_q_heads, pool->num_kv_heads, max_q_len);
        const int32_t ctas = prefill_tree_ctas(items, num_sms_current());
        if (ctas > 0 && prefill_sk_counts(items, max_q_len, G, p.max_len, verify_window(window, max_q_len), 0)) {
            const PrefillTreeWs w = prefill_tree_ws(ctas);
            if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || ws_bytes < w.bytes)
                return PKV_ERR_WORKSPACE;
            char *ws = static_cast<char *>(workspace);
            p.sk_ctas = ctas;
            p.sk_items = items;
            p.sk_rec = ws;
            p.sk_o = reinterpret_cast<float *>(ws + w.o);
            p.sk_ml = reinterpret_cast<float *>(ws + w.ml);
        }
    } else if (pool->dtype != PKV_F32 && p.kv_splits == 1) {
        const int32_t sk = prefill_sk_ctas(pool->dtype, batch, num_q_heads, pool->num_kv_heads,
                                           pool->head_dim, pool->block_size, max_q_len, num_sms_current());
        const int32_t items = sk > 0 ? prefill_items(batch, num_q_heads, pool->num_kv_heads, max_q_len) : 0;
        if (sk > 0 && prefill_sk_counts(items, max_q_len, G, p.max_len, window, sinks)) {
            if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
                ws_bytes < prefill_sk_ws_bytes(items, sk))
                return PKV_ERR_WORKSPACE;
            p.sk_ctas = sk;
            p.sk_items = items;
            char *ws = static_cast<char *>(workspace);
            p.sk_plan = reinterpret_cast<int32_t *>(ws);
            ws += (static_cast<size_t>(sk) * 3 * sizeof(int32_t) + 4 + 255) & ~static_cast<size_t>(255);
            p.sk_rec = ws;
            ws += (static_cast<size_t>(items) * kSkItemBytes + 255) & ~static_cast<size_t>(255);
            p.sk_count = reinterpret_cast<int32_t *>(ws);
            ws += (static_cast<size_t>(sk) * 8 * sizeof(int32_t) + 255) & ~static_cast<size_t>(255);
            p.sk_o = reinterpret_cast<float *>(ws);
            const size_t rows = static_cast<size_t>(sk) * 2 * 256;
            ws += (rows * 128 * sizeof(float) + 255) & ~static_cast<size_t>(255);
            p.sk_ml = reinterpret_cast<float *>(ws);
        }
    }
    if (static_cast<int64_t>(batch) * p.hkv * p.q_tiles * p.kv_splits > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t err;
    if (pool->dtype == PKV_FP8_E4M3) {
        err = launch_prefill_fp8(p, st);
    } else if (pool->dtype == PKV_BF16) {
        if (!encode_fn_ready()) return PKV_ERR_CUDA;
        CUtensorMap kmap, vmap;
        if (!encode_pool_map(&kmap, pool->k, *pool) || !encode_pool_map(&vmap, pool->v, *pool))
            return PKV_ERR_UNSUPPORTED;
        err = launch_prefill_bf16(p, kmap, vmap, st);
    } else {
        err = launch_prefill_f32(p, st);
    }
    return err == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

extern "C" {

pkv_status paged_prefill_chunk_attention(const void *q, const int32_t *cu_q_lens,
                                         int32_t num_q_heads, const pkv_pool *pool,
                                         const int32_t *block_tables, int32_t max_blocks_per_seq,
                                         const int32_t *seq_lens, int32_t batch, int32_t max_q_len,
                                         int32_t max_seq_len, int32_t window, float scale,
                                         void *out, void *workspace, size_t ws_bytes,
                                         int32_t *dev_status, pkv_stream_t stream)
{
    return prefill_call(q, cu_q_lens, num_q_heads, pool, block_tables, max_blocks_per_seq, seq_lens, batch,
                        max_q_len, max_seq_len, window, 0, scale, out, workspace, ws_bytes, dev_status,
                        stream);
}

pkv_status paged_prefill_chunk_attention_sinks(
    const void *q, const int32_t *cu_q_lens, int32_t num_q_heads, const pkv_pool *pool,
    const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t batch,
    int32_t max_q_len, int32_t max_seq_len, int32_t window, int32_t sinks, float scale, void *out,
    void *workspace, size_t ws_bytes, int32_t *dev_status, pkv_stream_t stream)
{
    return prefill_call(q, cu_q_lens, num_q_heads, pool, block_tables, max_blocks_per_seq, seq_lens, batch,
                        max_q_len, max_seq_len, window, sinks, scale, out, workspace, ws_bytes, dev_status,
                        stream);
}

}  // extern "C"

namespace {

// A row operand of the rotary append: aligned, tokens at least a token's rows
// apart, strides in whole 16-byte vectors.
bool rope_rows_ok(const void *ptr, int64_t stride, int64_t row_elems, int eb)
{
    return ptr != nullptr && aligned16(ptr) && stride >= row_elems && stride <= (INT64_MAX >> 8) &&
           (stride * eb) % 16 == 0;
}

}  // namespace

extern "C" {

pkv_status pkv_rope_init(pkv_rope *rope, int32_t rotary_dim, const double *inv_freq, int32_t num_axes,
                         const int32_t *axis_of_pair, int32_t interleaved, float factor)
{
    if (rope == nullptr || inv_freq == nullptr || rotary_dim < 2 || rotary_dim % 2 != 0 ||
        rotary_dim > 2 * PKV_ROPE_MAX_PAIRS || num_axes < 1 || num_axes > PKV_ROPE_MAX_AXES ||
        !std::isfinite(factor))
        return PKV_ERR_INVALID_ARG;
    pkv_rope r{};
    for (int32_t i = 0; i < rotary_dim / 2; ++i) {
        const int32_t a = axis_of_pair != nullptr ? axis_of_pair[i] : 0;
        if (!std::isfinite(inv_freq[i]) || a < 0 || a >= num_axes) return PKV_ERR_INVALID_ARG;
        r.axis[i] = static_cast<uint8_t>(a);
        // |f| / 2 pi as a double t and its error e (1 / 2 pi carried as two
        // doubles), whole turns dropped, then rounded to fractions of 2^64
        constexpr double kInv2PiHi = 0.15915494309189535, kInv2PiLo = -9.839338337591243e-18;
        const double f = std::fabs(inv_freq[i]), t = f * kInv2PiHi;
        const double e = std::fma(f, kInv2PiHi, -t) + f * kInv2PiLo;
        const double f64 = std::ldexp(t - std::floor(t), 64), whole = std::floor(f64);  // exact, < 2^64
        const double e64 = std::nearbyint(std::ldexp(e - std::nearbyint(e), 64) + (f64 - whole));  // |.| <= 2^63
        constexpr double kHalf = 9223372036854775808.0;  // 2^63: half a turn, either way
        uint64_t bits = static_cast<uint64_t>(whole);
        bits += std::fabs(e64) >= kHalf ? (1ull << 63) : static_cast<uint64_t>(static_cast<int64_t>(e64));
        r.freq[i] = inv_freq[i] < 0 ? 0 - bits : bits;
    }
    r.rotary_dim = rotary_dim;
    r.num_axes = num_axes;
    r.interleaved = interleaved != 0 ? 1 : 0;
    r.factor = factor;
    *rope = r;
    return PKV_OK;
}

pkv_status paged_kv_append_rope(const pkv_pool *pool, const int32_t *slot_mapping, int32_t num_tokens,
                                const void *q, int64_t q_stride, int32_t num_q_heads, const void *k_new,
                                int64_t k_stride, const void *v_new, int64_t v_stride,
                                const int32_t *positions, int64_t pos_stride, const pkv_rope *rope,
                                void *q_out, int64_t q_out_stride, int32_t *dev_status, pkv_stream_t stream)
{
    if (!valid_pool(pool) || num_tokens < 0 || num_q_heads < 0 || rope == nullptr) return PKV_ERR_INVALID_ARG;
    const int32_t rd = rope->rotary_dim;
    if (rd < 2 || rd % 2 != 0 || rd > pool->head_dim || rd > 2 * PKV_ROPE_MAX_PAIRS || rope->num_axes < 1 ||
        rope->num_axes > PKV_ROPE_MAX_AXES || !std::isfinite(rope->factor))
        return PKV_ERR_INVALID_ARG;
    for (int32_t i = 0; i < rd / 2; ++i)
        if (rope->axis[i] >= rope->num_axes) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    const int eb = elem_bytes(out_dtype(pool->dtype));
    const int64_t q_row = static_cast<int64_t>(num_q_heads) * pool->head_dim;
    const int64_t kv_row = static_cast<int64_t>(pool->num_kv_heads) * pool->head_dim;
    if (slot_mapping == nullptr || positions == nullptr ||
        (rope->num_axes > 1 && pos_stride != 0 && pos_stride < num_tokens) ||  // 0: one row for every axis
        !rope_rows_ok(k_new, k_stride, kv_row, eb) || !rope_rows_ok(v_new, v_stride, kv_row, eb))
        return PKV_ERR_INVALID_ARG;
    if (num_q_heads > 0 &&
        (!rope_rows_ok(q, q_stride, q_row, eb) || !rope_rows_ok(q_out, q_out_stride, q_row, eb)))
        return PKV_ERR_INVALID_ARG;
    if ((static_cast<int64_t>(pool->head_dim) * eb) % 16 != 0 || rd % (pool->dtype == PKV_F32 ? 8 : 16) != 0)
        return PKV_ERR_UNSUPPORTED;
    if (pool->dtype == PKV_FP8_E4M3 && !fp8_shape_built(pool)) return PKV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(pool->num_blocks) * pool->block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    // units of a row (rotated vector pairs and copied vectors): a CTA's threads hold a row at least
    if (static_cast<int64_t>(pool->head_dim) * eb / 16 - rd * eb / 32 > 256) return PKV_ERR_UNSUPPORTED;
    RopeParams p{};
    p.q = q;
    p.k_new = k_new;
    p.v_new = v_new;
    p.q_out = q_out;
    p.k_pool = pool->k;
    p.v_pool = pool->v;
    p.slot_mapping = slot_mapping;
    p.positions = positions;
    p.status = dev_status;
    p.q_stride = q_stride * eb / 16;
    p.k_stride = k_stride * eb / 16;
    p.v_stride = v_stride * eb / 16;
    p.q_out_stride = q_out_stride * eb / 16;
    p.pos_stride = pos_stride;
    p.num_tokens = num_tokens;
    p.hq = num_q_heads;
    p.hkv = pool->num_kv_heads;
    p.block_size = pool->block_size;
    p.head_dim = pool->head_dim;
    p.num_slots = pool->num_blocks * pool->block_size;
    p.rotary_dim = rd;
    p.interleaved = rope->interleaved;
    p.num_axes = rope->num_axes;
    p.factor = rope->factor;
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    std::memcpy(p.freq, rope->freq, sizeof(uint64_t) * (rd / 2));
    std::memcpy(p.axis, rope->axis, rd / 2);
    return launch_append_rope(p, pool->dtype, num_sms_current(), reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

pkv_status paged_copy_blocks(const pkv_pool *src, const pkv_pool *dst, int32_t n_pools,
                             const int32_t *src_blocks, const int32_t *dst_blocks, int32_t n,
                             int32_t *dev_status, pkv_stream_t stream)
{
    if (src == nullptr || n_pools < 0 || n < 0) return PKV_ERR_INVALID_ARG;
    if (dst == nullptr) dst = src;
    for (int32_t l = 0; l < n_pools; ++l) {
        const pkv_pool &a = src[l], &b = dst[l], &f = src[0];
        if (!valid_pool(&a) || !valid_pool(&b)) return PKV_ERR_INVALID_ARG;
        for (const pkv_pool *x : {&a, &b})
            if (x->dtype != f.dtype || x->block_size != f.block_size || x->num_kv_heads != f.num_kv_heads ||
                x->head_dim != f.head_dim)
                return PKV_ERR_INVALID_ARG;
    }
    if (n_pools == 0 || n == 0) return PKV_OK;
    if (src_blocks == nullptr || dst_blocks == nullptr) return PKV_ERR_INVALID_ARG;
    const int64_t row_bytes = static_cast<int64_t>(src[0].head_dim) * elem_bytes(src[0].dtype);
    const int64_t page_bytes = row_bytes * src[0].block_size * src[0].num_kv_heads;
    if (page_bytes % 16 != 0) return PKV_ERR_UNSUPPORTED;
    for (int32_t l0 = 0; l0 < n_pools; l0 += PKV_MAX_COPY_POOLS) {
        const int32_t nl = std::min(n_pools - l0, PKV_MAX_COPY_POOLS);
        CopyParams p{};
        p.src_blocks = src_blocks;
        p.dst_blocks = dst_blocks;
        p.status = dev_status;
        p.page_vecs = page_bytes / 16;
        p.n = n;
        p.n_tensors = 2 * nl;
        for (int32_t l = 0; l < nl; ++l) {
            p.src[2 * l] = src[l0 + l].k;
            p.src[2 * l + 1] = src[l0 + l].v;
            p.dst[2 * l] = dst[l0 + l].k;
            p.dst[2 * l + 1] = dst[l0 + l].v;
            p.src_num_blocks[l] = src[l0 + l].num_blocks;
            p.dst_num_blocks[l] = dst[l0 + l].num_blocks;
        }
        if (launch_copy_blocks(p, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

}  // extern "C"

namespace {

// One launch's tensors (at most kCommitTensors); new_seq_lens: of the call's first launch alone.
pkv_status commit_call(CommitParams &p, void *const *base, const int32_t *num_blocks, int32_t n_tensors, bool fp8,
                       const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *seq_lens,
                       const int32_t *cu_q_lens, int32_t batch, const int32_t *path, int32_t max_path,
                       const int32_t *path_lens, int32_t *new_seq_lens, int32_t *dev_status, pkv_stream_t stream)
{
    p.tables = block_tables;
    p.seq_lens = seq_lens;
    p.cu_q_lens = cu_q_lens;
    p.path = path;
    p.path_lens = path_lens;
    p.new_lens = new_seq_lens;
    p.status = dev_status;
    p.batch = batch;
    p.width = max_blocks_per_seq;
    p.max_path = max_path;
    p.n_tensors = n_tensors;
    for (int32_t z = 0; z < n_tensors; ++z) {
        p.base[z] = base[z];
        p.num_blocks[z] = num_blocks[z];
    }
    // a thread's index over the tensors' rows has 32 bits
    if (static_cast<int64_t>(p.heads) * p.row_vecs > (1 << 30) / n_tensors) return PKV_ERR_UNSUPPORTED;
    return launch_commit(p, fp8, num_sms_current(), reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

bool commit_args_ok(const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *seq_lens,
                    const int32_t *cu_q_lens, const int32_t *path, int32_t max_path, const int32_t *path_lens,
                    const int32_t *new_seq_lens)
{
    return block_tables != nullptr && max_blocks_per_seq > 0 && seq_lens != nullptr && cu_q_lens != nullptr &&
           path != nullptr && max_path >= 1 && max_path <= PKV_MAX_TREE && path_lens != nullptr &&
           new_seq_lens != nullptr && new_seq_lens != seq_lens && new_seq_lens != path_lens;
}

bool valid_latent_pool(const pkv_latent_pool *pool)
{
    return pool != nullptr && pool->data != nullptr && aligned16(pool->data) && pool->num_blocks > 0 &&
           pool->block_size > 0 && pool->latent_dim > 0 && pool->rope_dim > 0 &&
           (pool->dtype == PKV_F32 || pool->dtype == PKV_BF16 || pool->dtype == PKV_FP8_E4M3);
}

constexpr int32_t kCommitPools = PKV_MAX_COPY_POOLS;  // of one launch

// rows cut from a wider tensor: aligned, whole 16-byte vectors apart
bool cut_rows_ok(const void *ptr, int64_t stride, int64_t least, int eb)
{
    return ptr != nullptr && aligned16(ptr) && stride >= least && stride <= (1ll << 31) && (stride * eb) % 16 == 0;
}

bool latent_shape_built(pkv_dtype dtype, int32_t latent, int32_t rope, int32_t bs)
{
    return dtype != PKV_FP8_E4M3 && latent % 16 == 0 && latent <= 512 && rope % 16 == 0 && rope <= 128 && bs <= 64;
}

// Maps over a latent pool [num_blocks][bs][row]: a 4-D view (64 dims, slot, 64-dim
// region, block), box of 8 slots of the row's first `regions` regions, 128-byte
// swizzle, so that a box lands region by region, 1 KiB each.
bool encode_latent_map(CUtensorMap *map, const pkv_latent_pool &pool, int32_t regions)
{
    const cuuint64_t W = static_cast<cuuint64_t>(pool.latent_dim) + pool.rope_dim, bs = pool.block_size;
    const cuuint64_t dims[4] = {64, bs, static_cast<cuuint64_t>(regions), static_cast<cuuint64_t>(pool.num_blocks)};
    const cuuint64_t strides[3] = {W * 2, 128, bs * W * 2};
    const cuuint32_t box[4] = {64, 8, static_cast<cuuint32_t>(regions), 1}, one[4] = {1, 1, 1, 1};
    return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pool.data, dims, strides, box, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workers and pairs of an item for these sizes on the current device.
struct LatentPlan {
    int32_t workers, rows;
};
LatentPlan latent_plan(pkv_dtype dtype, int32_t latent, int32_t rope, int32_t bs, int num_sms)
{
    const int sms = std::max(num_sms, 1);
    if (latent_tc_built(dtype, latent, rope, bs)) return {std::max(sms / 2, 1), kLatentTcRows};
    return {2 * sms, kLatentSimpleRows};
}

size_t latent_ws_bytes(const LatentPlan &pl, int32_t latent)
{
    const size_t pieces = static_cast<size_t>(pl.workers) * 2 * pl.rows;
    const auto up = [](size_t b) { return (b + 255) & ~static_cast<size_t>(255); };
    return up(pieces * latent * sizeof(float)) + up(pieces * 2 * sizeof(float)) +
           static_cast<size_t>(pl.workers) * kLatentRecordBytes;
}

}  // namespace

extern "C" {

size_t paged_tree_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                 int32_t block_size, int32_t max_q_len, int32_t max_seq_len, int32_t window)
{
    if (batch <= 0 || num_kv_heads <= 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads != 0 || max_q_len <= 0 ||
        max_q_len > PKV_MAX_TREE || max_seq_len < 0 || window < 0 || head_dim <= 0 || block_size <= 0)
        return 0;
    // enough for every smaller max_q_len too, some of which run on the other kernel
    const int32_t G = num_q_heads / num_kv_heads;
    size_t bytes = 0;
    if (decode_shape_built(PKV_BF16, head_dim, block_size, G)) {
        const int32_t n = tree_on_decode(G, head_dim, block_size, max_q_len) ? max_q_len : 16 / G;
        bytes = ws_query_bytes(batch, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len,
                               verify_window(window, n), nullptr, 0, n);
    }
    if (G * static_cast<int64_t>(max_q_len) > 16 && prefill_shape_built(PKV_BF16, head_dim, block_size, G)) {
        const int32_t items = prefill_items(batch, num_q_heads, num_kv_heads, 1);
        const int32_t ctas = prefill_tree_ctas(items, num_sms_current());
        if (ctas > 0) bytes = std::max(bytes, prefill_tree_ws(ctas).bytes);
    }
    return bytes;
}

pkv_status paged_tree_attention(const void *q, const int32_t *cu_q_lens, const uint64_t *tree_masks,
                                int32_t num_q_heads, const pkv_pool *pool, const int32_t *block_tables,
                                int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t batch,
                                int32_t max_q_len, int32_t max_seq_len, int32_t window, float scale, void *out,
                                void *workspace, size_t ws_bytes, int32_t *dev_status, pkv_stream_t stream)
{
    return paged_tree_attention_queries(q, INT32_MAX, cu_q_lens, tree_masks, num_q_heads, pool, block_tables,
                                        max_blocks_per_seq, seq_lens, batch, max_q_len, max_seq_len, window, scale, out,
                                        workspace, ws_bytes, dev_status, stream);
}

pkv_status paged_tree_attention_queries(const void *q, int32_t num_queries, const int32_t *cu_q_lens,
                                        const uint64_t *tree_masks, int32_t num_q_heads, const pkv_pool *pool,
                                        const int32_t *block_tables, int32_t max_blocks_per_seq,
                                        const int32_t *seq_lens, int32_t batch, int32_t max_q_len, int32_t max_seq_len,
                                        int32_t window, float scale, void *out, void *workspace, size_t ws_bytes,
                                        int32_t *dev_status, pkv_stream_t stream)
{
    if (num_queries < 0 || max_q_len > PKV_MAX_TREE) return PKV_ERR_INVALID_ARG;
    if (num_queries == 0) max_q_len = std::min(max_q_len, 0);
    if (batch > 0 && max_q_len > 0 && tree_masks == nullptr) return PKV_ERR_INVALID_ARG;
    if (window > 0 && window < max_q_len) return PKV_ERR_UNSUPPORTED;
    // (a call without rows or queries launches nothing)
    return prefill_call(q, cu_q_lens, num_q_heads, pool, block_tables, max_blocks_per_seq, seq_lens, batch, max_q_len,
                        max_seq_len, window, 0, scale, out, workspace, ws_bytes, dev_status, stream, tree_masks,
                        num_queries);
}

pkv_status paged_tree_commit(const pkv_pool *pools, int32_t n_pools, const int32_t *block_tables,
                             int32_t max_blocks_per_seq, const int32_t *seq_lens, const int32_t *cu_q_lens,
                             int32_t batch, const int32_t *path, int32_t max_path, const int32_t *path_lens,
                             int32_t *new_seq_lens, int32_t *dev_status, pkv_stream_t stream)
{
    if (pools == nullptr || n_pools < 1 || batch < 0) return PKV_ERR_INVALID_ARG;
    const pkv_pool &f = pools[0];
    for (int32_t l = 0; l < n_pools; ++l)
        if (!valid_pool(&pools[l]) || pools[l].dtype != f.dtype || pools[l].block_size != f.block_size ||
            pools[l].num_kv_heads != f.num_kv_heads || pools[l].head_dim != f.head_dim)
            return PKV_ERR_INVALID_ARG;
    if (batch == 0) return PKV_OK;
    if (!commit_args_ok(block_tables, max_blocks_per_seq, seq_lens, cu_q_lens, path, max_path, path_lens, new_seq_lens))
        return PKV_ERR_INVALID_ARG;
    const bool fp8 = f.dtype == PKV_FP8_E4M3;
    const int64_t row_bytes = static_cast<int64_t>(f.head_dim) * elem_bytes(f.dtype);
    if (row_bytes % 16 != 0 || (fp8 && !fp8_shape_built(&f)) || row_bytes / 16 * f.num_kv_heads > INT32_MAX / PKV_MAX_TREE)
        return PKV_ERR_UNSUPPORTED;
    for (int32_t l0 = 0; l0 < n_pools; l0 += kCommitPools) {
        const int32_t nl = std::min(n_pools - l0, kCommitPools);
        void *base[2 * kCommitPools];
        int32_t blocks[2 * kCommitPools];
        for (int32_t l = 0; l < nl; ++l) {
            base[2 * l] = pools[l0 + l].k;
            base[2 * l + 1] = pools[l0 + l].v;
            blocks[2 * l] = blocks[2 * l + 1] = pools[l0 + l].num_blocks;
        }
        CommitParams p{};
        p.block_size = f.block_size;
        p.heads = f.num_kv_heads;
        p.row_vecs = static_cast<int32_t>(row_bytes / 16);
        const pkv_status st = commit_call(p, base, blocks, 2 * nl, fp8, block_tables, max_blocks_per_seq, seq_lens,
                                          cu_q_lens, batch, path, max_path, path_lens, l0 == 0 ? new_seq_lens : nullptr,
                                          dev_status, stream);
        if (st != PKV_OK) return st;
    }
    return PKV_OK;
}

pkv_status paged_latent_tree_commit(const pkv_latent_pool *pools, int32_t n_pools, const int32_t *block_tables,
                                    int32_t max_blocks_per_seq, const int32_t *seq_lens, const int32_t *cu_q_lens,
                                    int32_t batch, const int32_t *path, int32_t max_path, const int32_t *path_lens,
                                    int32_t *new_seq_lens, int32_t *dev_status, pkv_stream_t stream)
{
    if (pools == nullptr || n_pools < 1 || batch < 0) return PKV_ERR_INVALID_ARG;
    const pkv_latent_pool &f = pools[0];
    for (int32_t l = 0; l < n_pools; ++l)
        if (!valid_latent_pool(&pools[l]) || pools[l].dtype != f.dtype || pools[l].block_size != f.block_size ||
            pools[l].latent_dim != f.latent_dim || pools[l].rope_dim != f.rope_dim)
            return PKV_ERR_INVALID_ARG;
    if (batch == 0) return PKV_OK;
    if (!commit_args_ok(block_tables, max_blocks_per_seq, seq_lens, cu_q_lens, path, max_path, path_lens, new_seq_lens))
        return PKV_ERR_INVALID_ARG;
    const int64_t row_bytes = (static_cast<int64_t>(f.latent_dim) + f.rope_dim) * elem_bytes(f.dtype);
    if (f.dtype == PKV_FP8_E4M3 || row_bytes % 16 != 0 || row_bytes / 16 > INT32_MAX / PKV_MAX_TREE)
        return PKV_ERR_UNSUPPORTED;
    for (int32_t l0 = 0; l0 < n_pools; l0 += kCommitTensors) {
        const int32_t nl = std::min(n_pools - l0, kCommitTensors);
        void *base[kCommitTensors];
        int32_t blocks[kCommitTensors];
        for (int32_t l = 0; l < nl; ++l) {
            base[l] = pools[l0 + l].data;
            blocks[l] = pools[l0 + l].num_blocks;
        }
        CommitParams p{};
        p.block_size = f.block_size;
        p.heads = 1;
        p.row_vecs = static_cast<int32_t>(row_bytes / 16);
        const pkv_status st = commit_call(p, base, blocks, nl, false, block_tables, max_blocks_per_seq, seq_lens,
                                          cu_q_lens, batch, path, max_path, path_lens, l0 == 0 ? new_seq_lens : nullptr,
                                          dev_status, stream);
        if (st != PKV_OK) return st;
    }
    return PKV_OK;
}

pkv_status paged_latent_append(const pkv_latent_pool *pool, const int32_t *slot_mapping, int32_t num_tokens,
                               const void *latent_new, int64_t latent_stride, const void *k_rope_new,
                               int64_t k_rope_stride, const void *norm_weight, float norm_eps, const void *q_rope,
                               int64_t q_stride, int64_t q_head_stride, int32_t num_q_heads, const int32_t *positions,
                               int64_t pos_stride, const pkv_rope *rope, void *q_rope_out, int64_t q_out_stride,
                               int64_t q_out_head_stride, int32_t *dev_status, pkv_stream_t stream)
{
    if (!valid_latent_pool(pool) || num_tokens < 0 || num_q_heads < 0 || rope == nullptr ||
        !(norm_eps >= 0.f && std::isfinite(norm_eps)))
        return PKV_ERR_INVALID_ARG;
    const int32_t rd = rope->rotary_dim;
    if (rd < 2 || rd % 2 != 0 || rd > 2 * PKV_ROPE_MAX_PAIRS || rd != pool->rope_dim || rope->num_axes < 1 ||
        rope->num_axes > PKV_ROPE_MAX_AXES || !std::isfinite(rope->factor))
        return PKV_ERR_INVALID_ARG;
    for (int32_t i = 0; i < rd / 2; ++i)
        if (rope->axis[i] >= rope->num_axes) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    const int eb = elem_bytes(pool->dtype);
    if (slot_mapping == nullptr || positions == nullptr || !aligned16(norm_weight) ||
        (rope->num_axes > 1 && pos_stride != 0 && pos_stride < num_tokens) ||  // 0: one row for every axis
        !cut_rows_ok(latent_new, latent_stride, pool->latent_dim, eb) ||
        !cut_rows_ok(k_rope_new, k_rope_stride, rd, eb))
        return PKV_ERR_INVALID_ARG;
    if (num_q_heads > 0 &&
        (!cut_rows_ok(q_rope, q_stride, 0, eb) || !cut_rows_ok(q_rope, q_head_stride, rd, eb) ||
         !cut_rows_ok(q_rope_out, q_out_stride, 0, eb) || !cut_rows_ok(q_rope_out, q_out_head_stride, rd, eb) ||
         (num_tokens > 1 && (q_stride < (num_q_heads - 1) * q_head_stride + rd ||
                             q_out_stride < (num_q_heads - 1) * q_out_head_stride + rd)) ||
         (q_rope == q_rope_out && (q_head_stride != q_out_head_stride || (num_tokens > 1 && q_stride != q_out_stride)))))
        return PKV_ERR_INVALID_ARG;
    if (pool->dtype == PKV_FP8_E4M3 || pool->latent_dim % 16 != 0 || pool->latent_dim > 512 ||
        rd % (pool->dtype == PKV_F32 ? 8 : 16) != 0 ||
        static_cast<int64_t>(pool->num_blocks) * pool->block_size > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    LatentAppendParams p{};
    p.c_new = latent_new;
    p.k_new = k_rope_new;
    p.q = q_rope;
    p.norm_weight = norm_weight;
    p.pool = pool->data;
    p.q_out = q_rope_out;
    p.slot_mapping = slot_mapping;
    p.positions = positions;
    p.status = dev_status;
    p.c_stride = latent_stride * eb / 16;
    p.k_stride = k_rope_stride * eb / 16;
    p.q_stride = q_stride * eb / 16;
    p.q_head_stride = q_head_stride * eb / 16;
    p.q_out_stride = q_out_stride * eb / 16;
    p.q_out_head_stride = q_out_head_stride * eb / 16;
    p.pos_stride = pos_stride;
    p.num_tokens = num_tokens;
    p.heads = num_q_heads;
    p.num_slots = pool->num_blocks * pool->block_size;
    p.c_vecs = pool->latent_dim * eb / 16;
    p.row_vecs = (pool->latent_dim + rd) * eb / 16;
    p.rotary_dim = rd;
    p.interleaved = rope->interleaved;
    p.num_axes = rope->num_axes;
    p.factor = rope->factor;
    p.eps = norm_eps;
    std::memcpy(p.freq, rope->freq, sizeof(uint64_t) * (rd / 2));
    std::memcpy(p.axis, rope->axis, rd / 2);
    return launch_latent_append(p, pool->dtype, num_sms_current(), reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

size_t paged_latent_workspace_size(int32_t batch, int32_t num_q_heads, int32_t latent_dim, int32_t rope_dim,
                                   int32_t block_size, int32_t max_q_len, int32_t max_seq_len)
{
    if (batch < 0 || num_q_heads <= 0 || latent_dim <= 0 || rope_dim <= 0 || block_size <= 0 || max_q_len <= 0 ||
        max_seq_len < 0)
        return 0;
    // the same for every type and length
    const int sms = num_sms_current();
    return std::max(latent_ws_bytes(latent_plan(PKV_F32, latent_dim, rope_dim, block_size, sms), latent_dim),
                    latent_ws_bytes(latent_plan(PKV_BF16, latent_dim, rope_dim, block_size, sms), latent_dim));
}

pkv_status paged_latent_attention(const void *q, int32_t num_queries, const int32_t *cu_q_lens,
                                  const uint64_t *tree_masks, int32_t num_q_heads, const pkv_latent_pool *pool, const int32_t *block_tables,
                                  int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t batch,
                                  int32_t max_q_len, int32_t max_seq_len, float scale, void *out, void *workspace,
                                  size_t ws_bytes, int32_t *dev_status, pkv_stream_t stream)
{
    if (!valid_latent_pool(pool) || num_q_heads <= 0 || num_queries < 0 || batch < 0 || max_q_len < 0 || max_seq_len < 0 ||
        !std::isfinite(scale) || (cu_q_lens == nullptr && (max_q_len != 1 || num_queries != batch)) ||
        (tree_masks != nullptr && (cu_q_lens == nullptr || max_q_len > PKV_MAX_TREE)))
        return PKV_ERR_INVALID_ARG;
    if (batch == 0 || max_q_len == 0 || num_queries == 0) return PKV_OK;
    if (q == nullptr || out == nullptr || block_tables == nullptr || seq_lens == nullptr || max_blocks_per_seq <= 0 ||
        !aligned16(q) || !aligned16(out))
        return PKV_ERR_INVALID_ARG;
    if (!latent_shape_built(pool->dtype, pool->latent_dim, pool->rope_dim, pool->block_size)) return PKV_ERR_UNSUPPORTED;
    const LatentPlan pl = latent_plan(pool->dtype, pool->latent_dim, pool->rope_dim, pool->block_size, num_sms_current());
    const int64_t per_row = ceil_div64(static_cast<int64_t>(max_q_len) * num_q_heads, pl.rows);
    const int64_t max_len = std::min<int64_t>(max_seq_len, static_cast<int64_t>(max_blocks_per_seq) * pool->block_size);
    // the runs' sums are 32 bits: key tiles of all items, and some beside them
    const int64_t item_tiles = max_len / (pl.rows == kLatentTcRows ? 64 : 16) + 8;
    if (static_cast<int64_t>(max_q_len) * num_q_heads > INT32_MAX / 2 || per_row > INT32_MAX / item_tiles / batch ||
        static_cast<int64_t>(num_queries) * num_q_heads > INT32_MAX / 2)
        return PKV_ERR_UNSUPPORTED;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        ws_bytes < latent_ws_bytes(pl, pool->latent_dim))
        return PKV_ERR_WORKSPACE;
    LatentParams p{};
    p.q = q;
    p.out = out;
    p.pool = pool->data;
    p.tables = block_tables;
    p.seq_lens = seq_lens;
    p.cu_q_lens = cu_q_lens;
    p.tree = tree_masks;
    p.status = dev_status;
    p.batch = batch;
    p.heads = num_q_heads;
    p.latent = pool->latent_dim;
    p.rope = pool->rope_dim;
    p.block_size = pool->block_size;
    p.width = max_blocks_per_seq;
    p.num_blocks = pool->num_blocks;
    p.max_len = static_cast<int32_t>(max_len);
    p.max_q = max_q_len;
    p.num_queries = num_queries;
    p.items_per_row = static_cast<int32_t>(per_row);
    p.workers = pl.workers;
    const size_t pieces = static_cast<size_t>(pl.workers) * 2 * pl.rows;
    char *ws = static_cast<char *>(workspace);
    p.ws_o = reinterpret_cast<float *>(ws);
    ws += (pieces * p.latent * sizeof(float) + 255) & ~static_cast<size_t>(255);
    p.ws_ml = reinterpret_cast<float *>(ws);
    ws += (pieces * 2 * sizeof(float) + 255) & ~static_cast<size_t>(255);
    p.rec = ws;
    p.scale_log2 = scale * 1.4426950408889634f;
    drill_settings(&p.wait_ns, &p.drill);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!latent_tc_built(pool->dtype, p.latent, p.rope, p.block_size))
        return launch_latent_simple(p, pool->dtype, st) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
    if (!encode_fn_ready()) return PKV_ERR_CUDA;
    CUtensorMap map0, map1, q_map;  // whole rows, their latent parts, the queries as pages of one
    const pkv_latent_pool queries = {const_cast<void *>(q), 1, num_queries * num_q_heads, p.latent, p.rope, PKV_BF16};
    if (!encode_latent_map(&map0, *pool, (p.latent + p.rope) / 64) || !encode_latent_map(&map1, *pool, p.latent / 64) ||
        !encode_latent_map(&q_map, queries, (p.latent + p.rope) / 64))
        return PKV_ERR_UNSUPPORTED;
    return launch_latent_tc(p, map0, map1, q_map, st) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // extern "C"
