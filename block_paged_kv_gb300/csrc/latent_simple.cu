// Attention over latent rows on CUDA cores: f32 pools, and the shapes that the
// tensor-core kernel is not built for.  A CTA holds 16 (query, head) pairs of a
// row and walks its keys 16 at a time:
//   s = scale q . [c | k],  out = softmax(s) c
// with one pass over the rows (running maximum and sum; the weighted values in
// registers, a thread 1/16 of a pair's dims).  Bound: shared-memory reads of the
// products' operands: 8 rows of 2048 x 16 heads 73 us in f32 (512 + 64 dims, 0.5 TB/s),
// 43 in bf16 (128 + 32 dims); 2 chunks of 64 in f32 762.
#include "latent_common.cuh"

namespace pkv {

namespace ls {
constexpr int kRows = kLatentSimpleRows, kKeys = 16, kThreads = 256;
constexpr int kMaxD = 32;  // values of a thread: latent <= 512
}  // namespace ls

template <typename T>
__device__ __forceinline__ void load4(const T *src, float (&x)[4])
{
    if constexpr (sizeof(T) == 4) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(src));
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src));
        x[0] = bf16lo_to_f32(v.x);
        x[1] = bf16hi_to_f32(v.x);
        x[2] = bf16lo_to_f32(v.y);
        x[3] = bf16hi_to_f32(v.y);
    }
}

template <typename T>
__global__ void __launch_bounds__(ls::kThreads) latent_simple_kernel(const LatentParams p)
{
    using namespace ls;
    extern __shared__ float fsm[];
    __shared__ int64_t scan[kThreads / 32 + 4];
    __shared__ float sc[kRows][kKeys + 1];
    const int W = p.latent + p.rope, WS = W + 4;  // padded: 16 rows' quads hit distinct banks
    float *qs = fsm, *ks = fsm + kRows * WS;
    const int tid = threadIdx.x, pair = tid >> 4, sub = tid & 15;
    pdl_wait();
    pdl_trigger();
    Run run = latent_run<kRows, kKeys, kThreads>(p, blockIdx.x, 4, 8, 0, true, scan);
    LatentPiece pc;
    while (latent_next<kRows, kKeys>(p, run, pc)) {
        const LatentItem &it = pc.it;
        __syncthreads();
        const T *q = static_cast<const T *>(p.q) + (static_cast<int64_t>(it.q0) * p.heads + it.p0) * W;
        for (int i = tid * 4; i < kRows * W; i += kThreads * 4) {
            const int k = i / W, d = i - k * W;
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            if (k < it.n) load4(q + i, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) qs[k * WS + d + e] = x[e];
        }
        const LatentRange rg = latent_range(p, it, pair);
        float o[kMaxD], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int e = 0; e < kMaxD; ++e) o[e] = 0.f;
        const int32_t *table = p.tables + static_cast<int64_t>(it.r) * p.width;
        for (int32_t t = pc.t0; t < pc.t0 + pc.n; ++t) {
            const int32_t p0 = t * kKeys;
            __syncthreads();  // q staged; the last tile's rows are read
            for (int i = tid * 4; i < kKeys * W; i += kThreads * 4) {
                const int k = i / W, d = i - k * W;
                const int32_t pos = p0 + k, b = pos / p.block_size;
                float x[4] = {0.f, 0.f, 0.f, 0.f};
                if (pos < it.hi) {
                    const int32_t blk = b < p.width ? __ldg(table + b) : -1;
                    if (static_cast<uint32_t>(blk) < static_cast<uint32_t>(p.num_blocks))
                        load4(static_cast<const T *>(p.pool) +
                                  (static_cast<int64_t>(blk) * p.block_size + (pos - b * p.block_size)) * W + d, x);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) ks[k * WS + d + e] = x[e];
            }
            // does this thread's key take part: position p0 + sub, pair `pair`
            const int32_t pos = p0 + sub;
            bool seen = pos < rg.hi;
            if (pos < it.hi) {
                const int32_t b = pos / p.block_size;
                const int32_t blk = b < p.width ? __ldg(table + b) : -1;
                if (static_cast<uint32_t>(blk) >= static_cast<uint32_t>(p.num_blocks)) {
                    seen = false;
                    if (pair == 0) report(p.status, PKV_DEV_BAD_BLOCK);
                }
            }
            const int32_t dr = pos - it.first;
            if (p.tree != nullptr && dr >= 0) seen = seen && ((rg.mask >> (dr & 63)) & 1u);
            __syncthreads();
            float acc = 0.f;
            const float4 *qr = reinterpret_cast<const float4 *>(qs + pair * WS);
            const float4 *kr = reinterpret_cast<const float4 *>(ks + sub * WS);
            for (int d = 0; d < W / 4; ++d) {
                const float4 a = qr[d], b = kr[d];
                acc = fmaf(a.x, b.x, acc);
                acc = fmaf(a.y, b.y, acc);
                acc = fmaf(a.z, b.z, acc);
                acc = fmaf(a.w, b.w, acc);
            }
            const float s = seen ? acc * p.scale_log2 : -INFINITY;
            // the pair's 16 keys lie in 16 neighbouring lanes
            float mx = s;
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
            const float al = fast_exp2(m - mu), e = fast_exp2(s - mu);
            float sum = e;
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            l = l * al + sum;
            m = mn;
            sc[pair][sub] = e;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kMaxD; ++i)
                if (i * 16 < p.latent) o[i] *= al;
            for (int k = 0; k < kKeys; ++k) {
                const float wv = sc[pair][k];
                if (wv == 0.f) continue;  // masked slots may hold NaN
                const float *v = ks + k * WS + sub;
#pragma unroll
                for (int i = 0; i < kMaxD; ++i)
                    if (i * 16 < p.latent) o[i] = fmaf(wv, v[i * 16], o[i]);
            }
            __syncwarp();
        }
        if (pair >= it.n) continue;
        if (pc.whole) {
            const float inv = l != 0.f ? 1.f / l : 0.f;  // (NaN stays NaN)
            T *out = static_cast<T *>(p.out) + latent_out_row(p, it, pair) + sub;
#pragma unroll
            for (int i = 0; i < kMaxD; ++i)
                if (i * 16 < p.latent) {
                    if constexpr (sizeof(T) == 4) out[i * 16] = o[i] * inv;
                    else out[i * 16] = __float2bfloat16_rn(o[i] * inv);
                }
        } else {
            float *part = reinterpret_cast<float *>(latent_part_o<kRows>(p, blockIdx.x, pc.slot));
#pragma unroll
            for (int i = 0; i < kMaxD; ++i)
                if (i * 16 < p.latent) {
                    const int d = sub + i * 16;
                    part[((d >> 2) * kRows + pair) * 4 + (d & 3)] = o[i];
                }
            if (sub == 0) latent_part_ml<kRows>(p, blockIdx.x, pc.slot)[pair] = make_float2(weight_max(m, l), l);
        }
    }
}

template <typename T>
static cudaError_t launch(const LatentParams &p, cudaStream_t stream)
{
    const size_t smem = static_cast<size_t>(2) * ls::kRows * (p.latent + p.rope + 4) * sizeof(float);
    cudaError_t err = kernel_smem<latent_simple_kernel<T>>(100 * 1024);
    if (err != cudaSuccess) return err;
    prof_begin(PKV_KERNEL_LATENT, stream);
    err = launch_pdl(latent_simple_kernel<T>, dim3(static_cast<unsigned>(p.workers)), dim3(ls::kThreads), smem, stream, p);
    if (err == cudaSuccess)
        err = launch_latent_merge<T, ls::kRows>(p, stream);
    prof_end(PKV_KERNEL_LATENT, stream);
    return err;
}

cudaError_t launch_latent_simple(const LatentParams &p, pkv_dtype dtype, cudaStream_t stream)
{
    return dtype == PKV_F32 ? launch<float>(p, stream) : launch<__nv_bfloat16>(p, stream);
}

}  // namespace pkv
