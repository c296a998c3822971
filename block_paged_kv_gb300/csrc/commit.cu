// The accepted path of a drafted tree moved behind the cached tokens: for every
// row and every pool, the row of position n + i becomes that of position
// n + path[i] (n = the tokens before the drafts).
//
// A path ascends (path[i] >= i), so that tokens moved in order never write what a
// later one reads; within a pass the reads of all threads come before the first
// write.  Bound: the chain of dependent loads (lengths, path, table, rows), and
// HBM for many layers: a CTA resolves its row's path once and walks several
// tensors with it.
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kCommitThreads = 256;
constexpr int kCommitUnroll = 4;

// The row's moves, resolved: source and destination (block, offset) of each.
struct CommitMoves {
    int32_t n;
    int32_t src_blk[PKV_MAX_TREE], dst_blk[PKV_MAX_TREE];
    int32_t src_off[PKV_MAX_TREE], dst_off[PKV_MAX_TREE];
};

// Every thread of the CTA; ends in a barrier.
__device__ __forceinline__ void commit_resolve(const CommitParams &p, int32_t r, bool report_bad, CommitMoves &m)
{
    const int32_t L = __ldg(p.seq_lens + r);
    const int32_t C = __ldg(p.cu_q_lens + r + 1) - __ldg(p.cu_q_lens + r);
    const int32_t len = __ldg(p.path_lens + r);
    const int64_t cap = static_cast<int64_t>(p.width) * p.block_size;
    const bool sizes = L >= 0 && L <= cap && C >= 0 && C <= L;
    bool bad = !sizes || len < 0 || len > min(min(C, p.max_path), PKV_MAX_TREE);
    int32_t a = -1;
    const int32_t i = threadIdx.x;
    if (!bad && i < len) {
        a = __ldg(p.path + static_cast<int64_t>(r) * p.max_path + i);
        const int32_t before = i > 0 ? __ldg(p.path + static_cast<int64_t>(r) * p.max_path + i - 1) : -1;
        if (a <= before || a >= C) bad = true;  // (ascending: a >= i)
    }
    bad = __syncthreads_or(bad);
    const int32_t n = L - C;
    if (threadIdx.x == 0 && report_bad) {
        if (bad) report(p.status, sizes ? PKV_DEV_BAD_PATH : PKV_DEV_BAD_LEN);
        if (p.new_lens != nullptr) p.new_lens[r] = bad ? max(sizes ? n : L, 0) : n + len;
    }
    // tokens that lie in place already drop out; the others keep their order
    const bool moves = !bad && i < len && a != i;
    int32_t sb = -1, db = -1, so = 0, dof = 0;
    if (moves) {
        const int32_t *row = p.tables + static_cast<int64_t>(r) * p.width;
        const int32_t s = n + a, d = n + i;
        sb = __ldg(row + s / p.block_size);
        db = __ldg(row + d / p.block_size);
        so = s % p.block_size;
        dof = d % p.block_size;
    }
    // PKV_MAX_TREE tokens: the first two warps
    __shared__ uint32_t lower;
    const uint32_t votes = __ballot_sync(0xffffffffu, moves);
    if (threadIdx.x == 0) lower = votes;
    __syncthreads();
    if (moves) {
        const int32_t k = (i >= 32 ? __popc(lower) : 0) + __popc(votes & ((1u << (i & 31)) - 1u));
        m.src_blk[k] = sb;
        m.dst_blk[k] = db;
        m.src_off[k] = so;
        m.dst_off[k] = dof;
    }
    const int32_t total = __syncthreads_count(moves);
    if (threadIdx.x == 0) m.n = total;
    __syncthreads();
}

// 16-byte vector v of head h's row at (block, offset): its index in the tensor.
// FP8 K tiles hold a token's 64 dims as 64 consecutive bytes.
template <bool kF8>
__device__ __forceinline__ int64_t commit_vec(const CommitParams &p, int32_t blk, int32_t off, int32_t h, int32_t v)
{
    const int64_t tile = static_cast<int64_t>(blk) * p.heads + h;
    if constexpr (kF8) return tile * 16 * p.row_vecs + (v >> 2) * 64 + (off >> 3) * 32 + (off & 7) * 4 + (v & 3);
    return (tile * p.block_size + off) * p.row_vecs + v;
}

// CTA (x, y): row y, tensors x * tensors_per_cta ..
template <bool kF8>
__global__ void __launch_bounds__(kCommitThreads) commit_kernel(const __grid_constant__ CommitParams p)
{
    __shared__ CommitMoves m;
    pdl_wait();
    pdl_trigger();
    const int32_t z0 = blockIdx.x * p.tensors_per_cta, z1 = min(z0 + p.tensors_per_cta, p.n_tensors);
    for (int32_t r = blockIdx.y; r < p.batch; r += gridDim.y) {
        commit_resolve(p, r, blockIdx.x == 0, m);
        const int32_t per_token = p.heads * p.row_vecs, n = m.n * per_token;
        for (int32_t z = z0; z < z1; ++z) {
            const int32_t nb = p.num_blocks[z];
            uint8_t *base = static_cast<uint8_t *>(p.base[z]);
            const bool fp8_v = kF8 && (z & 1) != 0;
            // token by token in order, a pass of kCommitUnroll vectors a thread
            for (int32_t w0 = 0; w0 < n; w0 += kCommitThreads * kCommitUnroll) {
                uint4 x[kCommitUnroll];
                int64_t at[kCommitUnroll];
#pragma unroll
                for (int u = 0; u < kCommitUnroll; ++u) {
                    const int32_t w = w0 + u * kCommitThreads + threadIdx.x;
                    at[u] = -1;
                    if (w >= n) continue;
                    const int32_t k = w / per_token, e = w - k * per_token;
                    const int32_t h = e / p.row_vecs, v = e - h * p.row_vecs;
                    const int32_t sb = m.src_blk[k], db = m.dst_blk[k];
                    if (static_cast<uint32_t>(sb) >= static_cast<uint32_t>(nb) ||
                        static_cast<uint32_t>(db) >= static_cast<uint32_t>(nb)) {
                        if (e == 0) report(p.status, PKV_DEV_BAD_BLOCK);
                        continue;
                    }
                    if (!fp8_v) {
                        x[u] = reinterpret_cast<const uint4 *>(base)[commit_vec<kF8>(p, sb, m.src_off[k], h, v)];
                        at[u] = commit_vec<kF8>(p, db, m.dst_off[k], h, v);
                        continue;
                    }
                    // FP8 V tiles: a 16-byte chunk holds one dim of four tokens
                    // over four 8-dim steps; v = (32-dim group, dim class pair):
                    // this thread moves the token's 16 codes of two chunks
                    const int32_t st = m.src_off[k], dt = m.dst_off[k];
                    const int32_t c = (v >> 1) * 32 + (v & 1) * 16;  // first chunk of four dim classes
                    const int64_t tile_s = (static_cast<int64_t>(sb) * p.heads + h) * 16 * p.row_vecs;
                    const int64_t tile_d = (static_cast<int64_t>(db) * p.heads + h) * 16 * p.row_vecs;
                    const int sh = 8 * ((st & 1) + 2 * (st >> 3));
                    uint32_t b[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {  // dim classes 4 (v & 1) + j
                        const uint4 q = reinterpret_cast<const uint4 *>(base)[tile_s + c + 4 * j + ((st & 7) >> 1)];
                        b[j] = ((q.x >> sh) & 255u) | (((q.y >> sh) & 255u) << 8) | (((q.z >> sh) & 255u) << 16) |
                               (((q.w >> sh) & 255u) << 24);
                    }
                    x[u] = make_uint4(b[0], b[1], b[2], b[3]);
                    at[u] = (tile_d + c + ((dt & 7) >> 1)) * 16 + (dt & 1) + 2 * (dt >> 3);  // in bytes
                }
                __syncthreads();  // every read of the pass before its writes
#pragma unroll
                for (int u = 0; u < kCommitUnroll; ++u) {
                    if (at[u] < 0) continue;
                    if (!fp8_v) {
                        reinterpret_cast<uint4 *>(base)[at[u]] = x[u];
                        continue;
                    }
                    const uint32_t b[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int s = 0; s < 4; ++s) base[at[u] + j * 64 + s * 4] = static_cast<uint8_t>(b[j] >> (8 * s));
                }
                __syncthreads();  // the next pass may read what this one's neighbours wrote around
            }
        }
        __syncthreads();  // m is about to be overwritten
    }
}

cudaError_t launch_commit(const CommitParams &p_in, bool fp8, int num_sms, cudaStream_t stream)
{
    CommitParams p = p_in;
    const int64_t rows = std::min<int32_t>(p.batch, 65535);
    // about six CTAs an SM
    const int64_t want = std::max<int64_t>(1, 6ll * std::max(num_sms, 1) / rows);
    p.tensors_per_cta = static_cast<int32_t>((p.n_tensors + want - 1) / want);
    const unsigned gx = static_cast<unsigned>((p.n_tensors + p.tensors_per_cta - 1) / p.tensors_per_cta);
    prof_begin(PKV_KERNEL_COPY, stream);
    const dim3 grid(gx, static_cast<unsigned>(rows));
    const cudaError_t err = fp8 ? launch_pdl(commit_kernel<true>, grid, dim3(kCommitThreads), 0, stream, p)
                                : launch_pdl(commit_kernel<false>, grid, dim3(kCommitThreads), 0, stream, p);
    prof_end(PKV_KERNEL_COPY, stream);
    return err;
}

}  // namespace pkv
