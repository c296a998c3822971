// Latent append: one row a token in the latent pool, [c' | k'], with
//   c' = weight * c / sqrt(mean(c^2) + eps)   (or c as it is)
//   k' = the shared key rotated by the token's position,
// and the queries' rotary parts rotated by it.  Angles as in append_rope.cu;
// sums and products in fp32, one rounding to the row's type.
//
// Bound: HBM (every row read once and written once), launch latency for a decode
// step (32 tokens of 16 heads: 3.1 us).  A CTA takes a few tokens: their sines and
// cosines go to shared memory once and serve all heads; a warp normalises a token's
// latent, which it holds in registers between the sum and the product.
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "rope_device.cuh"

namespace pkv {

// 16384 tokens of 128 heads, 512 + 64 dims, bf16 (575 MB): 8 tokens of a CTA at most
// 101.6 us (5.7 TB/s), 16 109.1, 4 108.3; with two rows of a thread in flight 104.4,
// eight 104.6, one 115.5
constexpr int kLatAppTokens = 8;
constexpr int kLatAppBatch = 4;
constexpr int kLatMaxVecs = 4;     // latent vectors of a lane

template <bool kF32, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) latent_append_kernel(const __grid_constant__ LatentAppendParams p)
{
    using V = RopeVec<kF32>;
    constexpr int E = V::kE;
    __shared__ __align__(16) float cs[2 * kLatAppTokens * kRopeMaxPairs];
    __shared__ int32_t pos[PKV_ROPE_MAX_AXES * kRopeTabTokens];
    pdl_wait();
    pdl_trigger();
    RopeTab tab{cs, cs + kLatAppTokens * kRopeMaxPairs, pos, p.rotary_dim / 2};
    const int32_t t0 = blockIdx.x * p.tokens_per_cta, nt = min(p.tokens_per_cta, p.num_tokens - t0);
    tab.begin(p, t0, nt);
    auto row_of = [&](int32_t t, bool say) {  // the token's row in the pool, -1: not stored
        const int32_t slot = __ldg(p.slot_mapping + t);
        if (static_cast<uint32_t>(slot) < static_cast<uint32_t>(p.num_slots)) return static_cast<int64_t>(slot) * p.row_vecs;
        if (say && slot >= 0) report(p.status, PKV_DEV_BAD_SLOT);
        return static_cast<int64_t>(-1);
    };
    // the latents: a warp per token, the loads before the table is filled
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.y == 0) {
        for (int32_t tt = warp; tt < nt; tt += kRopeThreads / 32) {
            const int64_t at = row_of(t0 + tt, lane == 0);
            if (at < 0) continue;
            const uint4 *src = static_cast<const uint4 *>(p.c_new) + p.c_stride * (t0 + tt);
            uint4 *dst = static_cast<uint4 *>(p.pool) + at;
            uint4 x[kLatMaxVecs];
#pragma unroll
            for (int i = 0; i < kLatMaxVecs; ++i)
                if (lane + 32 * i < p.c_vecs) x[i] = __ldcs(src + lane + 32 * i);
            if (p.norm_weight != nullptr) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < kLatMaxVecs; ++i)
                    if (lane + 32 * i < p.c_vecs) {
                        float f[E];
                        V::unpack(x[i], f);
#pragma unroll
                        for (int e = 0; e < E; ++e) sum = fmaf(f[e], f[e], sum);
                    }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const float rs = rsqrtf(sum / static_cast<float>(p.c_vecs * E) + p.eps);
#pragma unroll
                for (int i = 0; i < kLatMaxVecs; ++i)
                    if (lane + 32 * i < p.c_vecs) {
                        float f[E], w[E];
                        V::unpack(x[i], f);
                        V::unpack(__ldg(static_cast<const uint4 *>(p.norm_weight) + lane + 32 * i), w);
#pragma unroll
                        for (int e = 0; e < E; ++e) f[e] = f[e] * rs * w[e];
                        x[i] = V::pack(f);
                    }
            }
#pragma unroll
            for (int i = 0; i < kLatMaxVecs; ++i)
                if (lane + 32 * i < p.c_vecs) dst[lane + 32 * i] = x[i];
        }
    }
    tab.fill(p, nt);
    // the rotated rows: `heads` of q, then the shared key; a thread keeps to one
    // vector pair and one token and walks the rows
    const int nrot = p.rotary_dim / (2 * E);
    const int lanes = kRopeThreads / nrot, ng = min(static_cast<int>(nt), lanes), phases = lanes / ng;
    const int u = threadIdx.x % nrot, r_in = threadIdx.x / nrot, ph = r_in / ng;
    if (ph >= phases) return;
    const int32_t step = phases * gridDim.y, first = ph * gridDim.y + blockIdx.y;
    for (int32_t tt = r_in - ph * ng; tt < nt; tt += ng) {
        const int32_t t = t0 + tt;
        const uint4 *qs = static_cast<const uint4 *>(p.q) + p.q_stride * t + u;
        uint4 *qd = static_cast<uint4 *>(p.q_out) + p.q_out_stride * t + u;
        RopeUnit<kF32, kInter> unit;
        unit.load(tab, tt, u, nrot);
        for (int32_t base = first; base <= p.heads; base += step * kLatAppBatch) {
            uint4 a[kLatAppBatch], b[kLatAppBatch];
#pragma unroll
            for (int j = 0; j < kLatAppBatch; ++j) {
                const int32_t h = base + j * step;
                if (h > p.heads) continue;
                const uint4 *src = h < p.heads ? qs + p.q_head_stride * h
                                               : static_cast<const uint4 *>(p.k_new) + p.k_stride * t + u;
                a[j] = __ldcs(src);
                b[j] = __ldcs(src + nrot);
            }
#pragma unroll
            for (int j = 0; j < kLatAppBatch; ++j) {
                const int32_t h = base + j * step;
                if (h > p.heads) continue;
                uint4 *dst = qd + p.q_out_head_stride * h;
                if (h == p.heads) {
                    const int64_t at = row_of(t, false);
                    if (at < 0) continue;
                    dst = static_cast<uint4 *>(p.pool) + at + p.c_vecs + u;
                }
                unit.rotate(a[j], b[j]);
                dst[0] = a[j];
                dst[nrot] = b[j];
            }
        }
    }
}

cudaError_t launch_latent_append(const LatentAppendParams &p_in, pkv_dtype dtype, int num_sms, cudaStream_t stream)
{
    LatentAppendParams p = p_in;
    const int sms = std::max(num_sms, 1);
    // a call of few tokens: one token a CTA, its heads over several CTAs; many
    // tokens: about eight CTAs an SM
    int tpc = 1;
    while (tpc < kLatAppTokens && static_cast<int64_t>(p.num_tokens) > 8ll * sms * tpc) tpc *= 2;
    p.tokens_per_cta = tpc;
    const unsigned gx = static_cast<unsigned>((p.num_tokens + tpc - 1) / tpc);
    const int nrot = p.rotary_dim * (dtype == PKV_F32 ? 4 : 2) / 32;
    const int passes = (p.heads + 1) * nrot * tpc / (kRopeThreads * kLatAppBatch);  // of a CTA alone
    const unsigned gy = static_cast<unsigned>(
        std::max<int64_t>(1, std::min<int64_t>(passes + 1, 4ll * sms / std::max(1u, gx))));
    prof_begin(PKV_KERNEL_APPEND, stream);
    const dim3 grid(gx, gy), block(kRopeThreads);
    cudaError_t err;
    if (dtype == PKV_F32)
        err = p.interleaved ? launch_pdl(latent_append_kernel<true, true>, grid, block, 0, stream, p)
                            : launch_pdl(latent_append_kernel<true, false>, grid, block, 0, stream, p);
    else
        err = p.interleaved ? launch_pdl(latent_append_kernel<false, true>, grid, block, 0, stream, p)
                            : launch_pdl(latent_append_kernel<false, false>, grid, block, 0, stream, p);
    prof_end(PKV_KERNEL_APPEND, stream);
    return err;
}

}  // namespace pkv
