// Drafted trees on the split-KV decode kernel (decode_kernel.cuh): the queries of
// a row's drafts, each behind the cached tokens and its own ancestors, bf16 and
// FP8 pools.  A split item holds up to 16 (query, head) rows; the items of a
// larger tree's further queries lie side by side and share their blocks through
// L2.  Bound: HBM for up to 16 rows (32 trees of 4 drafts over 1024 to 8192 keys, 32/8
// heads of 128: 107 to 110 us, 0.80 of the copy rate; FP8 91 us), the L2's re-reads above
// (16 trees of 32 over such keys, 8/2 heads of 64: 67 us).
#include "decode_kernel.cuh"

namespace pkv {

template <bool kF8>
static cudaError_t launch_tree(const DecodeParams &p, const CUtensorMap &kmap, const CUtensorMap &vmap,
                               cudaStream_t stream)
{
    const bool two = query_ntiles(static_cast<int64_t>(p.group) * p.q_chunk) == 2;
#define PKV_TREE_LAUNCH(DIM)                                                                  \
    return two ? launch_split<DIM, true, kF8, 2, false, true>(p, kmap, vmap, stream)          \
               : launch_split<DIM, true, kF8, 1, false, true>(p, kmap, vmap, stream)
    switch (p.head_dim) {
    case 64: PKV_TREE_LAUNCH(64);
    case 128: PKV_TREE_LAUNCH(128);
    case 256: PKV_TREE_LAUNCH(256);
    default: return cudaErrorInvalidValue;
    }
#undef PKV_TREE_LAUNCH
}

cudaError_t launch_tree_bf16(const DecodeParams &p, const CUtensorMap &kmap, const CUtensorMap &vmap,
                             cudaStream_t stream)
{
    return launch_tree<false>(p, kmap, vmap, stream);
}

cudaError_t launch_tree_fp8(const DecodeParams &p, cudaStream_t stream)
{
    const CUtensorMap none{};  // FP8 tiles arrive by bulk copy
    return launch_tree<true>(p, none, none, stream);
}

}  // namespace pkv
