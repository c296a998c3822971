// Rotary building blocks shared by the appends: cosines and sines of a CTA's
// tokens in shared memory, and the rotation of a row's vector pairs (the angle in
// turns as a 64-bit fraction: see append_rope.cu).
#pragma once

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kRopeThreads = 256;
constexpr int kRopeTabTokens = 32;  // tokens a CTA's table can hold
static_assert(PKV_ROPE_MAX_AXES * kRopeTabTokens <= kRopeThreads && kRopeMaxTokens <= kRopeTabTokens, "one position a thread");

__device__ __forceinline__ float2 rope_cos_sin(int32_t pos, uint64_t freq, float factor)
{
    // the high word of pos * freq mod 2^64, as signed turns * 2^32 (dropping the
    // low word costs 2^-32 turns): half turns = that * 2^-31
    const uint32_t u = static_cast<uint32_t>(pos), lo = static_cast<uint32_t>(freq), hi = static_cast<uint32_t>(freq >> 32);
    const uint32_t a = __umulhi(u, lo) + u * hi - (pos < 0 ? lo : 0u);
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(a)) * 0x1p-31f, &s, &c);
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

// The descriptor's tables are read by generic loads: lanes read neighbouring
// entries, which the constant port would serve one address at a time.
template <typename T>
__device__ __forceinline__ const T *generic_address(const T *q)
{
    asm("" : "+l"(q));
    return q;
}

// Cosines and sines of a CTA's tokens in shared memory, a row of `stride`
// floats each per token (16-byte aligned rows).  A thread keeps to one pair of
// the rotary_dim / 2; its frequency, its axis and a position are read by
// begin(), so that they and the first rows are in flight together, and fill()
// computes without touching global memory (a position read per entry, after
// its axis, made a window of 16 tokens wait 14 us).
struct RopeTab {
    float *c, *s;
    int32_t *pos;  // [kRopeMaxAxes][kRopeTabTokens]
    int stride;
    uint64_t freq;
    int32_t axis, my_pos;
    // P: launch parameters with the descriptor's tables and the positions
    template <typename P>
    __device__ __forceinline__ void begin(const P &p, int32_t t0, int32_t nt)
    {
        const int n = p.rotary_dim / 2, k = threadIdx.x % n;
        freq = generic_address(p.freq)[k];
        axis = generic_address(p.axis)[k];
        const int ax = threadIdx.x / kRopeTabTokens, tt = threadIdx.x % kRopeTabTokens;
        my_pos = ax < p.num_axes && tt < nt ? __ldg(p.positions + p.pos_stride * ax + t0 + tt) : 0;
    }
    // every thread of the CTA; ends in a barrier
    template <typename P>
    __device__ __forceinline__ void fill(const P &p, int32_t nt) const
    {
        if (threadIdx.x < PKV_ROPE_MAX_AXES * kRopeTabTokens) pos[threadIdx.x] = my_pos;
        __syncthreads();
        const int n = p.rotary_dim / 2, k = threadIdx.x % n, step = kRopeThreads / n;
        const int32_t *ps = pos + axis * kRopeTabTokens;
        if (threadIdx.x < step * n)
            for (int tt = threadIdx.x / n; tt < nt; tt += step) {
                const float2 v = rope_cos_sin(ps[tt], freq, p.factor);
                c[tt * stride + k] = v.x;
                s[tt * stride + k] = v.y;
            }
        __syncthreads();
    }
};

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

// A thread's share of a row: unit u < nrot = rotary_dim / 2E is the vectors u and
// u + nrot (halves: element e of the one is paired with element e of the other;
// interleaved: neighbours within each), later units one vector each of the
// dims past rotary_dim.  The unit's cosines and sines stay in registers.
template <bool kF32, bool kInter>
struct RopeUnit {
    using V = RopeVec<kF32>;
    static constexpr int E = V::kE;
    float c[E], s[E];  // interleaved: the first vector's E / 2 pairs, then the second's
    __device__ __forceinline__ void load(const RopeTab &tab, int tt, int u, int nrot)
    {
#pragma unroll
        for (int i = 0; i < E; i += kInter ? E / 2 : 4) {
            const int k = kInter ? (i == 0 ? u : u + nrot) * (E / 2) : u * E + i;
            const float *pc = tab.c + tt * tab.stride + k, *ps = tab.s + tt * tab.stride + k;
#pragma unroll
            for (int j = 0; j < (kInter ? E / 2 : 4); j += 2) {
                const float2 vc = *reinterpret_cast<const float2 *>(pc + j), vs = *reinterpret_cast<const float2 *>(ps + j);
                c[i + j] = vc.x;
                c[i + j + 1] = vc.y;
                s[i + j] = vs.x;
                s[i + j + 1] = vs.y;
            }
        }
    }
    __device__ __forceinline__ void rotate(uint4 &a, uint4 &b) const
    {
        float x[E], y[E], ox[E], oy[E];
        V::unpack(a, x);
        V::unpack(b, y);
        if constexpr (kInter) {
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                ox[e] = rope_elem(x[e], x[e + 1], c[e / 2], -s[e / 2]);
                ox[e + 1] = rope_elem(x[e + 1], x[e], c[e / 2], s[e / 2]);
                oy[e] = rope_elem(y[e], y[e + 1], c[(E + e) / 2], -s[(E + e) / 2]);
                oy[e + 1] = rope_elem(y[e + 1], y[e], c[(E + e) / 2], s[(E + e) / 2]);
            }
        } else {
            // two pairs an instruction (each lane rounded as rope_elem's)
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const uint64_t x2 = f2_pack(x[e], x[e + 1]), y2 = f2_pack(y[e], y[e + 1]);
                const uint64_t c2 = f2_pack(c[e], c[e + 1]), s2 = f2_pack(s[e], s[e + 1]);
                f2_unpack(f2_fma(x2, c2, f2_mul(y2, f2_pack(-s[e], -s[e + 1]))), ox[e], ox[e + 1]);
                f2_unpack(f2_fma(y2, c2, f2_mul(x2, s2)), oy[e], oy[e + 1]);
            }
        }
        a = V::pack(ox);
        b = V::pack(oy);
    }
};

}  // namespace pkv
