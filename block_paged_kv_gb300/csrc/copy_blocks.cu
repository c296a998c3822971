// Page copies: pool[l][dst_i] = pool[l][src_i] for the K and V pools of several
// layers in one launch (a fork's partial page, a rollback, a compaction).
//
// Bound: HBM, every page read once and written once.  A page (all kv heads of
// one block) is one contiguous run in every pool, so a copy is a plain stream;
// a CTA moves one chunk of one page of one pool, 16 bytes per thread and step
// with four loads in flight.
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;

// CTA (x, y, z): chunk x of pair y of tensor z (K and V of pool z / 2)
__global__ void __launch_bounds__(kCopyThreads) copy_blocks_kernel(const __grid_constant__ CopyParams p)
{
    pdl_wait();
    pdl_trigger();
    const int32_t tensor = blockIdx.z;
    const uint4 *sbase = static_cast<const uint4 *>(p.src[tensor]);
    uint4 *dbase = static_cast<uint4 *>(p.dst[tensor]);
    for (int32_t i = blockIdx.y; i < p.n; i += gridDim.y) {
        const int32_t s = __ldg(p.src_blocks + i), d = __ldg(p.dst_blocks + i);
        if (s < 0 || d < 0) continue;
        if (s >= p.src_num_blocks[tensor >> 1] || d >= p.dst_num_blocks[tensor >> 1]) {
            if (threadIdx.x == 0 && blockIdx.x == 0) report(p.status, PKV_DEV_BAD_BLOCK);
            continue;
        }
        const uint4 *src = sbase + s * p.page_vecs;
        uint4 *dst = dbase + d * p.page_vecs;
        if (src == dst) continue;
        const int64_t step = static_cast<int64_t>(gridDim.x) * kCopyThreads * kCopyUnroll;
        for (int64_t v0 = static_cast<int64_t>(blockIdx.x) * kCopyThreads * kCopyUnroll; v0 < p.page_vecs; v0 += step) {
            uint4 x[kCopyUnroll];
#pragma unroll
            for (int u = 0; u < kCopyUnroll; ++u) {
                const int64_t v = v0 + u * kCopyThreads + threadIdx.x;
                if (v < p.page_vecs) x[u] = __ldcs(src + v);
            }
#pragma unroll
            for (int u = 0; u < kCopyUnroll; ++u) {
                const int64_t v = v0 + u * kCopyThreads + threadIdx.x;
                if (v < p.page_vecs) __stcs(dst + v, x[u]);
            }
        }
    }
}

cudaError_t launch_copy_blocks(const CopyParams &p, cudaStream_t stream)
{
    const int64_t chunk = static_cast<int64_t>(kCopyThreads) * kCopyUnroll;
    const unsigned gx = static_cast<unsigned>(std::min<int64_t>((p.page_vecs + chunk - 1) / chunk, 1 << 16));
    const unsigned gy = static_cast<unsigned>(std::min<int32_t>(p.n, 65535));
    prof_begin(PKV_KERNEL_COPY, stream);
    const cudaError_t err =
        launch_pdl(copy_blocks_kernel, dim3(gx, gy, static_cast<unsigned>(p.n_tensors)), dim3(kCopyThreads), 0, stream, p);
    prof_end(PKV_KERNEL_COPY, stream);
    return err;
}

}  // namespace pkv
