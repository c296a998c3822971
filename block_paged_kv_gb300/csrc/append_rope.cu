// Rotary positions and append in one pass: q and k rows are rotated by their
// tokens' positions, the rotated k rows and the v rows land in their pool
// slots, the rotated q rows in q_out.
//
// Mathematics.  Pair i of the rotary_dim / 2 pairs turns by pos[axis(i)] * f_i
// radians.  The angle is kept in turns: F_i = f_i / 2 pi mod 1 as a 64-bit
// fixed-point fraction, so that pos * F_i mod 2^64 is the angle's exact
// remainder after whole turns - one integer product, no loss at far positions
// (a float32 product loses every digit of the angle near position 2^24) - and
// sincospif takes it from there without a range reduction of its own.
//   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin     (fp32, one rounding to the row's type)
// with (x1, x2) the dims (i, i + rotary_dim / 2), or (2i, 2i + 1) interleaved.
//
// Bound: HBM (every row read once and written once), launch latency for a
// decode step.  A CTA's sines and cosines (rotary_dim / 2 per token) go to
// shared memory once and serve all its heads; a thread keeps to one vector
// pair of the head and walks the heads with it.
#include <algorithm>

#include "e4m3_quant.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ float2 rope_cos_sin(int32_t pos, uint64_t freq, float factor)
{
    // signed turns * 2^64 in [-2^63, 2^63): half turns = that * 2^-63
    const int64_t a = static_cast<int64_t>(static_cast<uint64_t>(static_cast<int64_t>(pos)) * freq);
    float s, c;
    sincospif(__ll2float_rn(a) * 0x1p-63f, &s, &c);
    return make_float2(c * factor, s * factor);
}

// One rotated element: x its own value, xp its partner's, sn the sine with the
// sign of the element's side (- for the first of a pair).  The same two
// operations wherever an element is rotated, so that every path of a type
// stores the same bits.
__device__ __forceinline__ float rope_elem(float x, float xp, float c, float sn)
{
    return __fmaf_rn(x, c, __fmul_rn(xp, sn));
}

// sines and cosines of tokens t0 .. t0 + nt - 1 into cs[nt][rotary_dim / 2]
__device__ __forceinline__ void rope_table(const RopeParams &p, float2 *cs, int32_t t0, int32_t nt)
{
    const int n = p.rotary_dim / 2;
    for (int i = threadIdx.x; i < nt * n; i += blockDim.x) {
        const int tt = i / n, k = i - tt * n;
        const int32_t pos = __ldg(p.positions + p.pos_stride * p.axis[k] + t0 + tt);
        cs[i] = rope_cos_sin(pos, p.freq[k], p.factor);
    }
}

template <bool kF32>
struct RopeVec {
    static constexpr int kE = kF32 ? 4 : 8;  // elements of a 16-byte vector
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&x)[kE])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kF32) {
                x[i] = __uint_as_float(w[i]);
            } else {
                x[2 * i] = bf16lo_to_f32(w[i]);
                x[2 * i + 1] = bf16hi_to_f32(w[i]);
            }
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[kE])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kF32)
                w[i] = __float_as_uint(x[i]);
            else
                w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// A thread's share of a row: unit u < rotary_dim / 2E is the vectors u and
// u + rotary_dim / 2E (halves: element e of the one is paired with element e of
// the other; interleaved: neighbours within each), later units one vector each
// of the dims past rotary_dim.
template <bool kF32, bool kInter>
__device__ __forceinline__ void rope_unit(uint4 &a, uint4 &b, const float2 *cs, int u, int nrot)
{
    using V = RopeVec<kF32>;
    constexpr int E = V::kE;
    float x[E], y[E], ox[E], oy[E];
    V::unpack(a, x);
    V::unpack(b, y);
    if constexpr (kInter) {
        const float2 *c0 = cs + u * (E / 2), *c1 = cs + (u + nrot) * (E / 2);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 f = c0[e / 2], g = c1[e / 2];
            ox[e] = rope_elem(x[e], x[e + 1], f.x, -f.y);
            ox[e + 1] = rope_elem(x[e + 1], x[e], f.x, f.y);
            oy[e] = rope_elem(y[e], y[e + 1], g.x, -g.y);
            oy[e + 1] = rope_elem(y[e + 1], y[e], g.x, g.y);
        }
    } else {
        const float2 *c0 = cs + u * E;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float2 f = c0[e];
            ox[e] = rope_elem(x[e], y[e], f.x, -f.y);
            oy[e] = rope_elem(y[e], x[e], f.x, f.y);
        }
    }
    a = V::pack(ox);
    b = V::pack(oy);
}

// Rows row0 .. row1 - 1 of token t: q heads first, then k, then v (FP8 pools:
// q only).
template <bool kF32, bool kInter>
__device__ __forceinline__ void rope_rows(const RopeParams &p, const float2 *cs, int32_t t, int32_t row0,
                                          int32_t row1, int32_t slot)
{
    constexpr int E = RopeVec<kF32>::kE;
    const int vpr = p.head_dim / E, nrot = p.rotary_dim / (2 * E);
    const int units = nrot + (vpr - 2 * nrot);
    const int u = threadIdx.x % units, rstep = blockDim.x / units;
    const int r_in = threadIdx.x / units;
    if (r_in >= rstep) return;
    const bool rot = u < nrot;
    const int va = rot ? u : nrot + u;  // copy unit u: vector 2 nrot + (u - nrot)
    const int32_t blk = slot >= 0 ? slot / p.block_size : 0;
    const int32_t off = slot >= 0 ? slot - blk * p.block_size : 0;
    for (int32_t row = row0 + r_in; row < row1; row += rstep) {
        const uint4 *src;
        uint4 *dst;
        bool turn = rot;
        if (row < p.hq) {
            src = static_cast<const uint4 *>(p.q) + p.q_stride * t + static_cast<int64_t>(row) * vpr;
            dst = static_cast<uint4 *>(p.q_out) + p.q_out_stride * t + static_cast<int64_t>(row) * vpr;
        } else {
            if (slot < 0) break;  // k and v rows of a skipped token
            const bool is_v = row >= p.hq + p.hkv;
            const int32_t h = row - p.hq - (is_v ? p.hkv : 0);
            src = (is_v ? static_cast<const uint4 *>(p.v_new) + p.v_stride * t
                        : static_cast<const uint4 *>(p.k_new) + p.k_stride * t) +
                  static_cast<int64_t>(h) * vpr;
            dst = static_cast<uint4 *>(is_v ? p.v_pool : p.k_pool) +
                  ((static_cast<int64_t>(blk) * p.hkv + h) * p.block_size + off) * vpr;
            turn = rot && !is_v;
        }
        uint4 a = __ldcs(src + va);
        if (rot) {
            uint4 b = __ldcs(src + va + nrot);
            if (turn) rope_unit<kF32, kInter>(a, b, cs, u, nrot);
            dst[va + nrot] = b;
        }
        dst[va] = a;
    }
}

// The slot of token t, -1 when its K/V are skipped (negative, or past the
// pool: reported).
__device__ __forceinline__ int32_t rope_slot(const RopeParams &p, int32_t t)
{
    const int32_t slot = __ldg(p.slot_mapping + t);
    if (slot >= p.num_slots) {
        if (threadIdx.x == 0 && blockIdx.y == 0) report(p.status, PKV_DEV_BAD_SLOT);
        return -1;
    }
    return slot;
}

// CTA (x, y): tokens x * tokens_per_cta .., rows y * rows_per_cta ..
template <bool kF32, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) append_rope_kernel(const __grid_constant__ RopeParams p)
{
    __shared__ float2 cs[kRopeMaxTokens * kRopeMaxPairs];
    pdl_wait();
    pdl_trigger();
    const int32_t t0 = blockIdx.x * p.tokens_per_cta;
    const int32_t nt = min(p.tokens_per_cta, p.num_tokens - t0);
    rope_table(p, cs, t0, nt);
    __syncthreads();
    const int32_t row0 = blockIdx.y * p.rows_per_cta;
    const int32_t row1 = min(row0 + p.rows_per_cta, p.hq + 2 * p.hkv);
    for (int32_t tt = 0; tt < nt; ++tt)
        rope_rows<kF32, kInter>(p, cs + tt * (p.rotary_dim / 2), t0 + tt, row0, row1, rope_slot(p, t0 + tt));
}

// ---------------------------------------------------------------------------
// FP8 pools
// ---------------------------------------------------------------------------
// dims d, d + 1 (d even) of a bf16 k row, rotated, as floats
template <bool kInter>
__device__ __forceinline__ float2 rope_bf16_pair(const RopeParams &p, const uint32_t *row, int d, const float2 *cs)
{
    const uint32_t x = __ldg(row + d / 2);
    const float x0 = bf16lo_to_f32(x), x1 = bf16hi_to_f32(x);
    if (d >= p.rotary_dim) return make_float2(x0, x1);
    if constexpr (kInter) {
        const float2 f = cs[d / 2];
        return make_float2(rope_elem(x0, x1, f.x, -f.y), rope_elem(x1, x0, f.x, f.y));
    } else {
        const int h = p.rotary_dim / 2;
        const bool first = d < h;
        const uint32_t y = __ldg(row + (first ? d + h : d - h) / 2);
        const int i = first ? d : d - h;
        const float2 f = cs[i], g = cs[i + 1];
        return make_float2(rope_elem(x0, bf16lo_to_f32(y), f.x, first ? -f.y : f.y),
                           rope_elem(x1, bf16hi_to_f32(y), g.x, first ? -g.y : g.y));
    }
}

__device__ __forceinline__ uint32_t quant4f(float2 a, float2 b, float s, float r)
{
    return static_cast<uint32_t>(f32x2_to_e4m3x2(e4m3_quotient(a.x, s, r), e4m3_quotient(a.y, s, r))) |
           (static_cast<uint32_t>(f32x2_to_e4m3x2(e4m3_quotient(b.x, s, r), e4m3_quotient(b.y, s, r))) << 16);
}

// K and V rows of token t, kv head h, by one warp: 4-byte words of the K tile
// (dims d0, d0 + 1, d0 + 8, d0 + 9 of the token), the V tile's bytes one by one
// (it is token-minor).  The rotated k goes to E4M3 from fp32, without a
// rounding to bf16 between.
template <bool kInter>
__device__ __forceinline__ void rope_fp8_head(const RopeParams &p, const float2 *cs, int32_t t, int32_t h,
                                              int32_t slot, int lane)
{
    const int D = p.head_dim, off = slot & 15;
    const int64_t tile = (static_cast<int64_t>(slot >> 4) * p.hkv + h) * (16 * D);
    uint8_t *kt = static_cast<uint8_t *>(p.k_pool) + tile, *vt = static_cast<uint8_t *>(p.v_pool) + tile;
    const uint32_t *krow = reinterpret_cast<const uint32_t *>(static_cast<const uint4 *>(p.k_new) + p.k_stride * t) +
                           h * (D / 2);
    const uint32_t *vrow = reinterpret_cast<const uint32_t *>(static_cast<const uint4 *>(p.v_new) + p.v_stride * t) +
                           h * (D / 2);
    const float kr = __frcp_rn(p.k_scale), vr = __frcp_rn(p.v_scale);
    const int cv = (off & 7) >> 1, jv = (off & 1) + 2 * (off >> 3);
    for (int w = lane; w < D / 4; w += 32) {
        const int kk = w & 3, c = (w >> 2) & 3, grp = w >> 4;
        const int d0 = grp * 64 + kk * 16 + 2 * c;
        *reinterpret_cast<uint32_t *>(kt + grp * 1024 + (off >> 3) * 512 + ((off & 7) * 4 + c) * 16 + kk * 4) =
            quant4f(rope_bf16_pair<kInter>(p, krow, d0, cs), rope_bf16_pair<kInter>(p, krow, d0 + 8, cs),
                    p.k_scale, kr);
        const uint32_t vc = quant4(__ldg(vrow + d0 / 2), __ldg(vrow + d0 / 2 + 4), p.v_scale, vr);
        const int vd[4] = {d0, d0 + 1, d0 + 8, d0 + 9};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = vd[j];
            vt[(d >> 5) * 512 + ((d & 7) * 4 + cv) * 16 + ((d & 31) >> 3) * 4 + jv] =
                static_cast<uint8_t>(vc >> (8 * j));
        }
    }
}

// rows: the q heads, then the kv heads (a kv head's K and V count as one row)
template <bool kInter>
__global__ void __launch_bounds__(kRopeThreads) append_rope_fp8_kernel(const __grid_constant__ RopeParams p)
{
    __shared__ float2 cs[kRopeMaxTokens * kRopeMaxPairs];
    pdl_wait();
    pdl_trigger();
    const int32_t t0 = blockIdx.x * p.tokens_per_cta;
    const int32_t nt = min(p.tokens_per_cta, p.num_tokens - t0);
    rope_table(p, cs, t0, nt);
    __syncthreads();
    const int32_t row0 = blockIdx.y * p.rows_per_cta;
    const int32_t row1 = min(row0 + p.rows_per_cta, p.hq + p.hkv);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int32_t tt = 0; tt < nt; ++tt) {
        const int32_t slot = rope_slot(p, t0 + tt);
        const float2 *c = cs + tt * (p.rotary_dim / 2);
        rope_rows<false, kInter>(p, c, t0 + tt, row0, min(row1, p.hq), slot);
        if (slot < 0) continue;
        for (int32_t row = max(row0, p.hq) + warp; row < row1; row += kRopeThreads / 32)
            rope_fp8_head<kInter>(p, c, t0 + tt, row - p.hq, slot, lane);
    }
}

cudaError_t launch_append_rope(const RopeParams &params, pkv_dtype dtype, int num_sms, cudaStream_t stream)
{
    RopeParams p = params;
    const int32_t rows = p.hq + (dtype == PKV_FP8_E4M3 ? 1 : 2) * p.hkv;
    // as many tokens per CTA as give a sine and cosine to every thread, while
    // that leaves two CTAs per SM; the rows of a few tokens are dealt to
    // several CTAs
    p.tokens_per_cta = 1;
    while (p.tokens_per_cta < kRopeMaxTokens && p.tokens_per_cta * p.rotary_dim / 2 < kRopeThreads &&
           p.num_tokens / (2 * p.tokens_per_cta) >= 2 * num_sms)
        p.tokens_per_cta *= 2;
    const int32_t gx = (p.num_tokens - 1) / p.tokens_per_cta + 1;
    int32_t gy = std::max(1, std::min((2 * num_sms - 1) / gx + 1, (rows + 7) / 8));
    p.rows_per_cta = (rows + gy - 1) / gy;
    gy = (rows + p.rows_per_cta - 1) / p.rows_per_cta;
    void (*kern)(RopeParams) =
        dtype == PKV_FP8_E4M3 ? (p.interleaved ? append_rope_fp8_kernel<true> : append_rope_fp8_kernel<false>)
        : dtype == PKV_F32    ? (p.interleaved ? append_rope_kernel<true, true> : append_rope_kernel<true, false>)
                              : (p.interleaved ? append_rope_kernel<false, true> : append_rope_kernel<false, false>);
    prof_begin(PKV_KERNEL_APPEND, stream);
    const cudaError_t err = launch_pdl(kern, dim3(gx, gy), dim3(kRopeThreads), 0, stream, p);
    prof_end(PKV_KERNEL_APPEND, stream);
    return err;
}

}  // namespace pkv
