// The accepted path of a drafted tree moved behind the cached tokens: for every
// row and every pool, the row of position n + i becomes that of position
// n + path[i] (n = the tokens before the drafts).
//
// A path ascends (path[i] >= i), so that tokens moved in order never write what a
// later one reads.  Bound: the chain of dependent loads (lengths, path, table, rows):
// 2.1 us for 4 rows and two layers, 7.2 for 64 rows and 32 layers (24 MB, 3.5 us of
// HBM) in rows of 256 bytes.
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kCommitThreads = 256;
// 64 rows, 32 layers, 8 heads of 128 dims (24 MB moved): 16 CTAs an SM 7.2 us, 8 8.2, 6
// 9.9, 24 7.2; two tokens in flight 7.0, eight 9.1 (registers).  Passes of a CTA over
// tokens and tensors, every read before its writes (a barrier), took 16.1, most of it
// divisions.
constexpr int kCommitFly = 4;    // tokens of a thread in flight
constexpr int kCommitCtas = 16;  // CTAs an SM

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

// CTA (x, y): row y.  A thread takes 16 bytes of a token's row in one tensor (of all
// tensors' rows those from its index on, a grid's width apart) and moves them for one
// token after another, kCommitFly in flight: nobody else touches them, so nothing is
// waited for.
template <bool kF8>
__global__ void __launch_bounds__(kCommitThreads) commit_kernel(const __grid_constant__ CommitParams p)
{
    __shared__ CommitMoves m;
    pdl_wait();
    pdl_trigger();
    const int32_t per_token = p.heads * p.row_vecs, all = p.n_tensors * per_token;  // (2^30 at most: commit_call checks)
    for (int32_t r = blockIdx.y; r < p.batch; r += gridDim.y) {
        commit_resolve(p, r, blockIdx.x == 0, m);
        const int32_t n = m.n;
        for (int32_t w = blockIdx.x * kCommitThreads + threadIdx.x; n > 0 && w < all; w += gridDim.x * kCommitThreads) {
            const int32_t z = w / per_token, e = w - z * per_token;
            const int32_t h = e / p.row_vecs, v = e - h * p.row_vecs;
            const uint32_t nb = static_cast<uint32_t>(p.num_blocks[z]);
            uint8_t *base = static_cast<uint8_t *>(p.base[z]);
            const bool fp8_v = kF8 && (z & 1) != 0;
            for (int32_t k0 = 0; k0 < n; k0 += kCommitFly) {
                uint4 x[kCommitFly];
                int64_t at[kCommitFly];
#pragma unroll
                for (int u = 0; u < kCommitFly; ++u) {
                    const int32_t k = k0 + u;
                    at[u] = -1;
                    if (k >= n) continue;
                    const int32_t sb = m.src_blk[k], db = m.dst_blk[k];
                    if (static_cast<uint32_t>(sb) >= nb || static_cast<uint32_t>(db) >= nb) {
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
#pragma unroll
                for (int u = 0; u < kCommitFly; ++u) {
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
            }
        }
        __syncthreads();  // m is about to be overwritten
    }
}

cudaError_t launch_commit(const CommitParams &p, bool fp8, int num_sms, cudaStream_t stream)
{
    const int64_t rows = std::min<int32_t>(p.batch, 65535);
    const int64_t all = static_cast<int64_t>(p.n_tensors) * p.heads * p.row_vecs;
    const unsigned gx = static_cast<unsigned>(
        std::max<int64_t>(1, std::min<int64_t>((all + kCommitThreads - 1) / kCommitThreads,
                                               static_cast<int64_t>(kCommitCtas) * std::max(num_sms, 1) / rows)));
    prof_begin(PKV_KERNEL_COPY, stream);
    const dim3 grid(gx, static_cast<unsigned>(rows));
    const cudaError_t err = fp8 ? launch_pdl(commit_kernel<true>, grid, dim3(kCommitThreads), 0, stream, p)
                                : launch_pdl(commit_kernel<false>, grid, dim3(kCommitThreads), 0, stream, p);
    prof_end(PKV_KERNEL_COPY, stream);
    return err;
}

}  // namespace pkv
