// Internal host/device interface between the C ABI layer (api.cu) and the
// kernel translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <utility>

#include "pkv.h"

namespace pkv {

// Upper bound on any pipeline wait; a wait that runs past it reports
// PKV_DEV_TIMEOUT and the kernel winds down instead of spinning on.  The
// kernels' data waits take their limit from the launch parameters (this value
// unless a diagnostic drill shortens it); the waits of a wind-down, for copies
// a CTA issued itself, always take this one.
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

// Diagnostic drill flag carried by the launch parameters (pkv_set_wait_drill):
// the first load of every pipeline is never issued, so that the wait for it
// runs out with nothing in flight on its barrier.
constexpr uint32_t kDrillWithholdFirst = PKV_DRILL_WITHHOLD_FIRST_LOAD;

// Diagnostic drill flag: the softmax warps of the tensor-core prefill let 20 us
// or more pass between handing over a segment's last weights and looking for its
// output, long after the tensor cores have finished it.
constexpr uint32_t kDrillLate = PKV_DRILL_LATE_CONSUMERS;

// Diagnostic drill flag: two of the three producer warps of the latent attention look
// at every ring entry 5 and 10 us late.
constexpr uint32_t kDrillLateProducers = PKV_DRILL_LATE_PRODUCERS;

struct AppendParams {
    void *k_pool;
    void *v_pool;
    const void *k_new;
    const void *v_new;
    const int32_t *slot_mapping;
    int32_t *status;
    int32_t num_tokens;
    int32_t hkv;
    int32_t block_size;
    int32_t vecs_per_row;  // head_dim * elem_bytes / 16 (bf16/f32 pools)
    int32_t num_slots;     // num_blocks * block_size
    int32_t head_dim;      // FP8 pools: bf16 rows are quantized with these scales
    float k_scale, v_scale;
    int32_t heads_per_warp;  // FP8: kv heads one warp quantizes for a token (divides hkv)
};

// Rotary append: strides in 16-byte vectors between tokens; the descriptor's
// tables travel in the launch parameters.
constexpr int kRopeMaxPairs = PKV_ROPE_MAX_PAIRS;
constexpr int kRopeMaxTokens = 16;  // tokens of a CTA
struct RopeParams {
    const void *q, *k_new, *v_new;
    void *q_out, *k_pool, *v_pool;
    const int32_t *slot_mapping;
    const int32_t *positions;  // [axes][pos_stride]
    int32_t *status;
    int64_t q_stride, k_stride, v_stride, q_out_stride, pos_stride;
    int32_t num_tokens, hq, hkv, block_size, head_dim, num_slots;
    int32_t rotary_dim, interleaved, num_axes;
    int32_t tokens_per_cta, rows_per_cta;  // set by the launch
    float factor, k_scale, v_scale;
    uint64_t freq[kRopeMaxPairs];
    uint8_t axis[kRopeMaxPairs];
};

// Page copies of up to PKV_MAX_COPY_POOLS pools; tensor 2l is pool l's K, 2l + 1 its V.
struct CopyParams {
    const int32_t *src_blocks, *dst_blocks;
    int32_t *status;
    int64_t page_vecs;  // 16-byte vectors of one block (all kv heads) of one tensor
    int32_t n, n_tensors;
    const void *src[2 * PKV_MAX_COPY_POOLS];
    void *dst[2 * PKV_MAX_COPY_POOLS];
    int32_t src_num_blocks[PKV_MAX_COPY_POOLS];
    int32_t dst_num_blocks[PKV_MAX_COPY_POOLS];
};

// The accepted paths' rows moved behind the cached tokens, in up to
// kCommitTensors tensors (K and V of a pool, or a latent pool each).
constexpr int kCommitTensors = 2 * PKV_MAX_COPY_POOLS;
struct CommitParams {
    const int32_t *tables, *seq_lens, *cu_q_lens, *path, *path_lens;
    int32_t *new_lens;  // nullptr: not wanted (later launches of a call)
    int32_t *status;
    int32_t batch, width, max_path, block_size, heads;
    int32_t row_vecs;   // 16-byte vectors of one head's row (FP8: of one head's codes)
    int32_t n_tensors;
    void *base[kCommitTensors];
    int32_t num_blocks[kCommitTensors];
};

// Latent append: strides in 16-byte vectors; the rotary tables as in RopeParams.
struct LatentAppendParams {
    const void *c_new, *k_new, *q, *norm_weight;
    void *pool, *q_out;
    const int32_t *slot_mapping;
    const int32_t *positions;
    int32_t *status;
    int64_t c_stride, k_stride, q_stride, q_head_stride, q_out_stride, q_out_head_stride, pos_stride;
    int32_t num_tokens, heads, num_slots;
    int32_t c_vecs, row_vecs;  // vectors of the latent part and of a whole row
    int32_t rotary_dim, interleaved, num_axes;
    int32_t tokens_per_cta;    // set by the launch
    float factor, eps;
    uint64_t freq[kRopeMaxPairs];
    uint8_t axis[kRopeMaxPairs];
};

// Attention over latent rows.  The (query, head) pairs of a row's queries are
// cut into items of `rows` pairs, each over the row's keys up to its last
// query's; the items' key tiles in item order form one sequence, of which every
// worker takes an equal run.
struct LatentParams {
    const void *q;
    void *out;
    const void *pool;
    const int32_t *tables;
    const int32_t *seq_lens;
    const int32_t *cu_q_lens;  // nullptr: one query per row
    const uint64_t *tree;      // nullptr: chains
    int32_t *status;
    int32_t batch, heads, latent, rope, block_size, width, num_blocks;
    int32_t max_len, max_q, num_queries;
    int32_t items_per_row;     // item bound of a row: ceil(max_q * heads / pairs of an item)
    int32_t workers;
    float *ws_o;    // [workers][2][latent / 4][pairs of an item][4] unnormalised weighted values
    float *ws_ml;   // [workers][2][pairs of an item][2]: reference max (log2 units), weight sum
    void *rec;      // [workers] records of kLatentRecordBytes: the item that a run begins and does not end
    float scale_log2;
    uint64_t wait_ns;
    uint32_t drill;
};
constexpr int kLatentRecordBytes = 24;
constexpr int kTreeRecordBytes = 24;
constexpr int kLatentSimpleRows = 16;  // pairs of an item: CUDA-core kernel
constexpr int kLatentTcRows = 128;     // tensor-core kernel

// Split plan of one decode call.  A row's key range [lo, L) covers the blocks
// b_first .. b_end-1; split s of the row's suffix covers blocks
// b_first + s*split_blocks .. (capped at b_end).  Rows of a shared-prefix
// group start their suffix at the group's prefix_blocks, and the prefix is cut
// into runs of prefix_split_blocks read once for the whole group.
struct DecodePlan {
    int32_t split_blocks;         // C
    int32_t n_suffix_splits;      // splits per row (upper bound)
    int32_t prefix_split_blocks;  // Cp
    int32_t n_prefix_splits;      // prefix splits per group (upper bound); 0 = no prefix path
    int32_t nslot;                // partial slots per (row, q head) = n_prefix + n_suffix
    int32_t prefix_chunks;        // CTAs per (group, kv head, prefix split) over its rows
    int32_t prefix_max;           // prefix lengths are clamped to this (<= table width)
    int32_t few;                  // rows x kv heads < SMs: a few long rows, about two CTAs per SM
    int32_t coop;                 // few, and runs long enough (or a grid small enough) for the
                                  // cooperative kernel (bf16, one query per row, G <= 8)
    int64_t n_prefix_ctas;
    int64_t n_suffix_ctas;
};

struct DecodeParams {
    const void *q;
    void *out;
    const void *k_pool;  // read directly by the f32 and FP8 kernels; bf16 goes through TMA maps
    const void *v_pool;
    const int32_t *tables;
    const int32_t *seq_lens;
    const int32_t *group_of_row;   // nullptr when there is no prefix path
    const int32_t *prefix_blocks;
    float *ws_o;   // [batch * max_q][hq][nslot][head_dim] unnormalised weighted values
    float *ws_ml;  // [batch * max_q][hq][nslot][2]: running max (log2 units) and weight sum
    int32_t *status;
    // several queries per row (a speculative-verify step; bf16 only): row r
    // owns the packed queries cu_q_lens[r] .. cu_q_lens[r+1]-1 at the last
    // positions of its length, causally.  nullptr: one query per row (decode)
    const int32_t *cu_q_lens;
    int32_t max_q;  // queries per row, upper bound (1 for decode)
    int32_t batch, hq, hkv, group, head_dim, block_size, width, num_blocks;
    int32_t max_len;   // min(max_seq_len, width * block_size): lengths are clamped to it
    int32_t window;
    int32_t sinks;     // with a window: the first positions that stay visible (0 = none)
    // drafted trees: bit j of tree[i] = the packed query i attends its row's
    // draft j (nullptr: chains).  A split item then takes q_chunk of a row's
    // queries, q_chunks of them a row
    const uint64_t *tree;
    int32_t q_chunk, q_chunks;
    int32_t num_queries;  // with cu_q_lens: rows whose queries lie past them are left out
    int32_t num_groups;
    float scale_log2;  // scale * log2(e) (* k_scale for FP8): scores are kept in base-2 units
    float v_scale;     // FP8: applied to each partial's weighted values
    uint64_t wait_ns;  // limit of the pipeline's data waits (kWaitLimitNs unless a drill)
    uint32_t drill;    // diagnostic drill flags (kDrillWithholdFirst); 0 normally
    DecodePlan plan;
};

// Several decode calls fused into one split launch and one merge launch.
constexpr int kMaxDecodeGroups = 4;
struct GroupedDecode {
    CUtensorMap kmap[kMaxDecodeGroups];  // bf16 pools (unused for FP8)
    CUtensorMap vmap[kMaxDecodeGroups];
    DecodeParams g[kMaxDecodeGroups];
    int64_t cta_end[kMaxDecodeGroups];   // split CTAs of groups 0..i (cumulative)
    int64_t item_end[kMaxDecodeGroups];  // merge CTAs of groups 0..i (cumulative)
    int32_t n;
};

// A kernel's launch attributes on the current device: `smem` bytes of dynamic shared
// memory (the same at every call) and, with `carveout`, the largest carveout for it.
// Set once per device: a call for each costs 0.2 us.
template <auto kKernel>
cudaError_t kernel_smem(int smem, bool carveout = false)
{
    static std::atomic<uint64_t> devices{0};  // a bit each
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if ((devices.load(std::memory_order_relaxed) & bit) != 0) return cudaSuccess;
    err = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err == cudaSuccess && carveout)
        err = cudaFuncSetAttribute(kKernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (err == cudaSuccess) devices.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

// Launch with programmatic stream serialization (PDL): the kernel may be
// scheduled while the previous kernel on the stream drains; it calls
// pdl_wait() before touching global memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args &&...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Launch bookkeeping (api.cu): every kernel launch is counted; launches of
// kinds enabled by pkv_profile_enable are bracketed by CUDA events.
void prof_begin(int kind, cudaStream_t stream);
void prof_end(int kind, cudaStream_t stream);

constexpr int kSkItemBytes = 64;  // one item's record of the persistent schedule

struct PrefillParams {
    const void *q;
    void *out;
    const void *k_pool;  // used by the f32 kernel; the bf16 kernel reads via TMA
    const void *v_pool;
    const int32_t *cu_q_lens;
    const int32_t *tables;
    const int32_t *seq_lens;
    int32_t *status;
    int32_t batch, hq, hkv, group, head_dim, block_size, width, num_blocks;
    int32_t max_len;    // min(max_seq_len, width * block_size)
    int32_t max_q_len;
    int32_t num_queries;  // rows whose queries lie past them are left out
    int32_t window;
    int32_t sinks;      // with a window: the first positions that stay visible (0 = none)
    const uint64_t *tree;  // drafted trees: bit j of tree[i] = the packed query i attends its row's draft j
    int32_t q_tiles;    // CTAs per (row, kv head): ceil(max_q_len / queries per CTA)
    // key-range split (bf16, short chunks only; 1 = none): each (row, kv head,
    // query tile) is cut into kv_splits runs of split_tiles 64-key tiles whose
    // fp32 partials a merge kernel combines
    int32_t kv_splits;
    int32_t split_tiles;
    float *ws_o;   // [batch][max_q_len][hq][kv_splits][128] unnormalised weighted values
    float *ws_ml;  // [batch][max_q_len][hq][kv_splits][2]: reference max (log2 units), weight sum
    // persistent balanced schedule (0 = off): sk_ctas CTAs take
    // level runs of the (item, 64-key tile) sequence of the sk_items items
    // (row, kv head, query-tile pair); a run that cuts an item writes a
    // partial to one of its CTA's two slots
    int32_t sk_ctas, sk_items;
    int32_t *sk_plan;    // written by the plan kernel: starts of the CTAs' runs [sk_ctas + 1], the items
                         // there [sk_ctas], the CTAs' whole items [sk_ctas]
    void *sk_rec;        // [sk_items] records of kSkItemBytes (written by the plan kernel); drafted
                         // trees: [sk_ctas] of kTreeRecordBytes (no plan, no counters)
    int32_t *sk_count;   // [sk_ctas][2 query tiles][4 warps]: pieces done of the item cut
                         // after the CTA's first tile (zeroed by the plan kernel)
    float *sk_o;         // [sk_ctas][2][2 query tiles][4 warps][32 dim groups][32 rows][4] unnormalised weighted values
    float *sk_ml;        // [sk_ctas][2][2 query tiles][4 warps][32 rows][2]: reference max (log2 units), weight sum
    float scale_log2;  // scale * log2(e) (* k_scale for FP8 pools)
    float v_scale;     // FP8 pools: applied to the weighted values
    uint64_t wait_ns;  // limit of the pipeline's data waits (kWaitLimitNs unless a drill)
    uint32_t drill;    // diagnostic drill flags (kDrillWithholdFirst); 0 normally
};

// The current diagnostic drill (pkv_set_wait_drill): the data-wait limit and
// the flags every decode / prefill launch carries.
void drill_settings(uint64_t *wait_ns, uint32_t *flags);

// Dynamic shared memory the f32 kernels may ask for (every built shape needs
// less).  Set as one value whatever the call's shape: with each call's own size,
// a second host thread's call could lower the limit between another's setting it
// and its launch, which then failed.
constexpr int kF32SmemLimit = 227 * 1024;

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream);
cudaError_t launch_append_fp8(const AppendParams &p, cudaStream_t stream);
cudaError_t launch_append_rope(const RopeParams &p, pkv_dtype dtype, int num_sms, cudaStream_t stream);
cudaError_t launch_copy_blocks(const CopyParams &p, cudaStream_t stream);
cudaError_t launch_commit(const CommitParams &p, bool fp8, int num_sms, cudaStream_t stream);
cudaError_t launch_latent_append(const LatentAppendParams &p, pkv_dtype dtype, int num_sms, cudaStream_t stream);
bool latent_tc_built(pkv_dtype dtype, int32_t latent, int32_t rope, int32_t bs);
cudaError_t launch_latent_tc(const LatentParams &p, const CUtensorMap &map0, const CUtensorMap &map1, const CUtensorMap &q_map,
                             cudaStream_t stream);
cudaError_t launch_latent_simple(const LatentParams &p, pkv_dtype dtype, cudaStream_t stream);
bool prefill_shape_built(pkv_dtype dtype, int32_t D, int32_t bs, int32_t G);
int32_t prefill_queries_per_cta(pkv_dtype dtype, int32_t G);
// Key-range split of the bf16 prefill for short chunks (all of a row's
// queries in one query tile) on grids too small to fill the GPU: runs per
// (row, kv head) and 64-key tiles per run; {1, 0} = no split.
struct PrefillSplit {
    int32_t splits, tiles;
};
PrefillSplit prefill_split_plan(int32_t batch, int32_t hq, int32_t hkv, int32_t D, int32_t bs,
                                int32_t max_q_len, int32_t max_seq_len, int32_t window,
                                int32_t sinks, int num_sms);
size_t prefill_split_ws_bytes(int32_t batch, int32_t hq, int32_t max_q_len, const PrefillSplit &sp);
// The persistent balanced schedule of the tensor-core prefill: the CTA count
// (0 = off: the grid then holds one CTA per item) and its workspace.
int32_t prefill_sk_ctas(pkv_dtype dtype, int32_t batch, int32_t hq, int32_t hkv, int32_t D,
                        int32_t bs, int32_t max_q_len, int num_sms);
// Drafted trees: CTAs of the levelled runs over the items (0: one CTA an item), and
// their workspace (offsets of the pieces' values and of their maxima and sums).
int32_t prefill_tree_ctas(int32_t items, int num_sms);
struct PrefillTreeWs {
    size_t o, ml, bytes;
};
PrefillTreeWs prefill_tree_ws(int32_t ctas);
size_t prefill_sk_ws_bytes(int32_t items, int32_t ctas);
// Whether the plan's 32-bit sums hold items of up to max_len keys (else the call
// takes one CTA per item; past 65536 items of two million keys, say).
bool prefill_sk_counts(int32_t items, int32_t max_q_len, int32_t group, int32_t max_len, int32_t window,
                       int32_t sinks);
cudaError_t launch_prefill_bf16(const PrefillParams &p, const CUtensorMap &kmap,
                                const CUtensorMap &vmap, cudaStream_t stream);
cudaError_t launch_prefill_f32(const PrefillParams &p, cudaStream_t stream);
cudaError_t launch_prefill_fp8(const PrefillParams &p, cudaStream_t stream);

// bf16 pools: TMA + mbarrier pipeline, mma.sync tiles.  kmap/vmap: 5-D tensor
// maps (64 dims, slot, 64-dim region, kv head, block), whole-tile boxes, 128B swizzle.
cudaError_t launch_decode_bf16(const DecodeParams &p, const CUtensorMap &kmap,
                               const CUtensorMap &vmap, cudaStream_t stream);
// drafted trees (p.tree, p.q_chunk) on the same kernel
cudaError_t launch_tree_bf16(const DecodeParams &p, const CUtensorMap &kmap, const CUtensorMap &vmap,
                             cudaStream_t stream);
cudaError_t launch_tree_fp8(const DecodeParams &p, cudaStream_t stream);
// f32 pools: CUDA-core kernel.
cudaError_t launch_decode_f32(const DecodeParams &p, cudaStream_t stream);
cudaError_t launch_decode_fp8(const DecodeParams &p, cudaStream_t stream);
// grouped launches (decode only: one query per row, no prefix path); the
// merge covers every group with the same kernel shape
cudaError_t launch_decode_bf16_grouped(const GroupedDecode &gd, cudaStream_t stream);
cudaError_t launch_decode_fp8_grouped(const GroupedDecode &gd, cudaStream_t stream);
cudaError_t launch_decode_combine_grouped(GroupedDecode &gd, pkv_dtype out_dtype, cudaStream_t stream);
// merge of the split partials into out (dtype of q)
cudaError_t launch_decode_combine(const DecodeParams &p, pkv_dtype dtype, cudaStream_t stream);

// Warps per decode CTA: a split CTA's warps share one query tile and take its
// blocks in turn; a shared-prefix CTA holds one tile of (row, head) pairs per
// warp.  The prefix cut (the prefix blocks per split) is sized as if a CTA
// held 64 pairs (32 at head_dim 256), whatever the dtype, so that the
// workspace size does not depend on it.
constexpr int kDecodeWarps = 4;
constexpr int kPrefixPairsPerCta = 64;  // head_dim <= 128 (32 for head_dim 256)

// bf16 / FP8 decode: query rows sit on the N side of the products in n-tiles
// of 8; a split item's rows (the G heads, or G x queries of a verify step)
// need this many, and so does each warp's tile of a prefix item (8 x that
// many (row, head) pairs per warp)
inline int query_ntiles(int64_t rows) { return rows > 8 ? 2 : 1; }
// query rows per CTA of the f32 kernel
constexpr int kF32Rows = 16;

}  // namespace pkv
