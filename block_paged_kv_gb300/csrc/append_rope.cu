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
#include "rope_device.cuh"

namespace pkv {

// Rows row0 .. row1 - 1 (q heads first, then k, then v; FP8 pools: q only) of
// tokens t0 .. t0 + nt - 1.  A thread keeps to one unit of the head and one
// token and walks the rows, kRopeBatch at a time: all loads of a batch are
// issued before any is used, those of the first before `table` (which fills
// the CTA's cosines and sines and ends in a barrier) is called.
constexpr int kRopeBatch = 2;

template <bool kF32, bool kInter, typename Table>
__device__ __forceinline__ void rope_rows(const RopeParams &p, const RopeTab &tab, int32_t t0, int32_t nt,
                                          int32_t row0, int32_t row1, Table table)
{
    constexpr int E = RopeVec<kF32>::kE;
    const int vpr = p.head_dim / E, nrot = p.rotary_dim / (2 * E), units = vpr - nrot;
    const int lanes = blockDim.x / units;  // (token, row phase) pairs of a pass
    const int ng = min(static_cast<int>(nt), lanes), phases = lanes / ng;
    const int u = threadIdx.x % units, r_in = threadIdx.x / units;
    const int ph = r_in / ng;
    const bool rot = u < nrot;
    const int va = rot ? u : nrot + u;  // copy unit u: vector 2 nrot + (u - nrot)
    bool first = true;
    for (int32_t tt = r_in - ph * ng; first || tt < nt; tt += ng) {
        const bool live = ph < phases && tt < nt;
        const int32_t t = t0 + (live ? tt : 0);
        const uint4 *qs = static_cast<const uint4 *>(p.q) + p.q_stride * t + va;
        const uint4 *ks = static_cast<const uint4 *>(p.k_new) + p.k_stride * t + va;
        const uint4 *vs = static_cast<const uint4 *>(p.v_new) + p.v_stride * t + va;
        uint4 *qd = static_cast<uint4 *>(p.q_out) + p.q_out_stride * t + va;
        int64_t at = -1;  // the token's vectors in its page, -1: not stored
        if (row1 > p.hq) {
            const int32_t slot = __ldg(p.slot_mapping + t);
            if (static_cast<uint32_t>(slot) < static_cast<uint32_t>(p.num_slots)) {
                const int32_t blk = slot / p.block_size;
                at = (static_cast<int64_t>(blk) * p.hkv * p.block_size + (slot - blk * p.block_size)) * vpr + va;
            } else if (live && slot >= 0) {
                report(p.status, PKV_DEV_BAD_SLOT);
            }
        }
        RopeUnit<kF32, kInter> unit;
        bool have = false;
        const int32_t end = !live ? row0 : at < 0 ? min(row1, p.hq) : row1;
        for (int32_t base = row0 + ph; first || base < end; base += phases * kRopeBatch) {
            uint4 a[kRopeBatch], b[kRopeBatch];
#pragma unroll
            for (int j = 0; j < kRopeBatch; ++j) {
                const int32_t row = base + j * phases;
                if (row >= end) continue;
                const uint4 *src = row < p.hq           ? qs + row * vpr
                                   : row < p.hq + p.hkv ? ks + (row - p.hq) * vpr
                                                        : vs + (row - p.hq - p.hkv) * vpr;
                a[j] = __ldcs(src);
                if (rot) b[j] = __ldcs(src + nrot);
            }
            if (first) table();
            first = false;
            if (!have && rot) unit.load(tab, live ? tt : 0, u, nrot);
            have = true;
#pragma unroll
            for (int j = 0; j < kRopeBatch; ++j) {
                const int32_t row = base + j * phases;
                if (row >= end) continue;
                uint4 *dst = qd + row * vpr;
                if (row >= p.hq) {
                    const bool is_v = row >= p.hq + p.hkv;
                    dst = static_cast<uint4 *>(is_v ? p.v_pool : p.k_pool) + at +
                          static_cast<int64_t>(row - p.hq - (is_v ? p.hkv : 0)) * p.block_size * vpr;
                }
                if (rot) {
                    if (row < p.hq + p.hkv) unit.rotate(a[j], b[j]);
                    dst[nrot] = b[j];
                }
                dst[0] = a[j];
            }
        }
    }
}

// CTA (x, y): tokens x * tokens_per_cta .., rows y * rows_per_cta ..
template <bool kF32, bool kInter>
__global__ void __launch_bounds__(kRopeThreads, 4) append_rope_kernel(const __grid_constant__ RopeParams p)
{
    __shared__ __align__(16) float cs[2 * kRopeMaxTokens * kRopeMaxPairs];
    __shared__ int32_t pos[PKV_ROPE_MAX_AXES * kRopeTabTokens];
    pdl_wait();
    pdl_trigger();
    RopeTab tab{cs, cs + kRopeMaxTokens * kRopeMaxPairs, pos, p.rotary_dim / 2};
    const int32_t t0 = blockIdx.x * p.tokens_per_cta, nt = min(p.tokens_per_cta, p.num_tokens - t0);
    tab.begin(p, t0, nt);
    const int32_t row0 = blockIdx.y * p.rows_per_cta;
    rope_rows<kF32, kInter>(p, tab, t0, nt, row0, min(row0 + p.rows_per_cta, p.hq + 2 * p.hkv), [&]() { tab.fill(p, nt); });
}

// ---------------------------------------------------------------------------
// FP8 pools
// ---------------------------------------------------------------------------
// Dims d, d + 1 (d even) of a bf16 k row, rotated, as floats; word(i) is the
// row's dims 2i, 2i + 1; c, s the token's cosines and sines.
template <bool kInter, typename Word>
__device__ __forceinline__ float2 rope_bf16_pair(const RopeParams &p, const Word &word, int d, const float *c,
                                                 const float *s)
{
    const uint32_t x = word(d / 2);
    const float x0 = bf16lo_to_f32(x), x1 = bf16hi_to_f32(x);
    if (d >= p.rotary_dim) return make_float2(x0, x1);
    if constexpr (kInter) {
        const float fc = c[d / 2], fs = s[d / 2];
        return make_float2(rope_elem(x0, x1, fc, -fs), rope_elem(x1, x0, fc, fs));
    } else {
        const int h = p.rotary_dim / 2;
        const bool first = d < h;
        const uint32_t y = word((first ? d + h : d - h) / 2);
        const int i = first ? d : d - h;
        const float2 fc = *reinterpret_cast<const float2 *>(c + i), fs = *reinterpret_cast<const float2 *>(s + i);
        return make_float2(rope_elem(x0, bf16lo_to_f32(y), fc.x, first ? -fs.x : fs.x),
                           rope_elem(x1, bf16hi_to_f32(y), fc.y, first ? -fs.y : fs.y));
    }
}

__device__ __forceinline__ uint32_t quant4f(float2 a, float2 b, float s, float r)
{
    return static_cast<uint32_t>(f32x2_to_e4m3x2(e4m3_quotient(a.x, s, r), e4m3_quotient(a.y, s, r))) |
           (static_cast<uint32_t>(f32x2_to_e4m3x2(e4m3_quotient(b.x, s, r), e4m3_quotient(b.y, s, r))) << 16);
}

// K and V rows of token t, kv heads h0 .. h0 + nh - 1 (nh <= H), by one warp:
// 4-byte words of the K tile (dims d0, d0 + 1, d0 + 8, d0 + 9 of the token), the
// V tile's bytes one by one (it is token-minor).  The rotated k goes to E4M3
// from fp32, without a rounding to bf16 between.  All heads' loads come before
// the first store, so that they are in flight together.
template <bool kInter, int H>
__device__ __forceinline__ void rope_fp8_heads(const RopeParams &p, const float *cs, const float *sn, int32_t t,
                                               int32_t h0, int32_t nh, int32_t slot, int lane)
{
    const int D = p.head_dim, off = slot & 15;
    const int64_t tile = (static_cast<int64_t>(slot >> 4) * p.hkv + h0) * (16 * D);
    uint8_t *kt = static_cast<uint8_t *>(p.k_pool) + tile, *vt = static_cast<uint8_t *>(p.v_pool) + tile;
    const uint32_t *krow = reinterpret_cast<const uint32_t *>(static_cast<const uint4 *>(p.k_new) + p.k_stride * t) +
                           h0 * (D / 2);
    const uint32_t *vrow = reinterpret_cast<const uint32_t *>(static_cast<const uint4 *>(p.v_new) + p.v_stride * t) +
                           h0 * (D / 2);
    const float kr = __frcp_rn(p.k_scale), vr = __frcp_rn(p.v_scale);
    const int cv = (off & 7) >> 1, jv = (off & 1) + 2 * (off >> 3);
    for (int w = lane; w < D / 4; w += 32) {
        const int kk = w & 3, c = (w >> 2) & 3, grp = w >> 4;
        const int d0 = grp * 64 + kk * 16 + 2 * c;
        uint32_t kc[H], vc[H];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            if (h >= nh) continue;
            const uint32_t *kh = krow + h * (D / 2), *vh = vrow + h * (D / 2);
            const auto word = [&](int i) { return __ldg(kh + i); };
            kc[h] = quant4f(rope_bf16_pair<kInter>(p, word, d0, cs, sn), rope_bf16_pair<kInter>(p, word, d0 + 8, cs, sn),
                            p.k_scale, kr);
            vc[h] = quant4(__ldg(vh + d0 / 2), __ldg(vh + d0 / 2 + 4), p.v_scale, vr);
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            if (h >= nh) continue;
            *reinterpret_cast<uint32_t *>(kt + h * (16 * D) + grp * 1024 + (off >> 3) * 512 + ((off & 7) * 4 + c) * 16 +
                                          kk * 4) = kc[h];
            const int vd[4] = {d0, d0 + 1, d0 + 8, d0 + 9};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d = vd[j];
                vt[h * (16 * D) + (d >> 5) * 512 + ((d & 7) * 4 + cv) * 16 + ((d & 31) >> 3) * 4 + jv] =
                    static_cast<uint8_t>(vc[h] >> (8 * j));
            }
        }
    }
}

// The slot of token t if its K and V are stored, else -1 (one past the pool is reported).
__device__ __forceinline__ int32_t rope_slot(const RopeParams &p, int32_t t)
{
    const int32_t slot = __ldg(p.slot_mapping + t);
    if (slot >= p.num_slots) {
        if ((threadIdx.x & 31) == 0) report(p.status, PKV_DEV_BAD_SLOT);
        return -1;
    }
    return slot;
}

// A few tokens: CTA (x, y) as above, rows: the q heads, then the kv heads (a kv
// head's K and V count as one row, done by one warp).
template <bool kInter>
__global__ void __launch_bounds__(kRopeThreads) append_rope_fp8_kernel(const __grid_constant__ RopeParams p)
{
    __shared__ __align__(16) float cs[2 * kRopeMaxTokens * kRopeMaxPairs];
    __shared__ int32_t pos[PKV_ROPE_MAX_AXES * kRopeTabTokens];
    pdl_wait();
    pdl_trigger();
    RopeTab tab{cs, cs + kRopeMaxTokens * kRopeMaxPairs, pos, p.rotary_dim / 2};
    const int32_t t0 = blockIdx.x * p.tokens_per_cta, nt = min(p.tokens_per_cta, p.num_tokens - t0);
    tab.begin(p, t0, nt);
    const int32_t row0 = blockIdx.y * p.rows_per_cta;
    const int32_t row1 = min(row0 + p.rows_per_cta, p.hq + p.hkv);
    rope_rows<false, kInter>(p, tab, t0, nt, row0, min(row1, p.hq), [&]() { tab.fill(p, nt); });
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int32_t tt = 0; tt < nt; ++tt) {
        const int32_t slot = rope_slot(p, t0 + tt);
        if (slot < 0) continue;
        for (int32_t row = max(row0, p.hq) + warp; row < row1; row += kRopeThreads / 32)
            rope_fp8_heads<kInter, 1>(p, tab.c + tt * tab.stride, tab.s + tt * tab.stride, t0 + tt, row - p.hq, 1, slot,
                                      lane);
    }
}

// Many tokens: CTA (x, y) takes the window of 16 tokens x and the kv heads
// y * kHG .. (with their share of the q heads).  A block that receives its 16
// tokens in order from this call has its first token, the lead, in one window
// (two leads are 16 tokens apart); that window's CTA stages the block's bf16 K
// and V rows in shared memory and writes whole tiles: each thread forms 16-byte
// chunks in the tiles' byte order (a K chunk: one token, 16 dims; a V chunk: one
// dim of four tokens over four 8-dim steps) and stores them coalesced, where
// the byte-wise V stores of the per-token path write 32-byte sectors 32 times.
// Tokens of other blocks take that path.  The q rows are rotated while the
// staged rows arrive.
template <int D>
struct RopeWin {
    static constexpr int kHG = 512 / D;             // kv heads of a CTA
    static constexpr int kRowB = 2 * D + 16;        // padded bytes of a staged row: the reads hit distinct banks
    static constexpr int kTensorB = kHG * 16 * kRowB;
    static constexpr int kTabRows = 31;             // tokens t0 .. t0 + 30: the window's and a late lead's block
    // a row of the table: 8 tokens' 8-byte reads of 4 lanes fall into distinct banks
    __host__ __device__ static constexpr int tab_stride(int rotary_dim) { return rotary_dim / 2 + 8; }
    static int smem(int rotary_dim) { return 2 * kTensorB + kTabRows * tab_stride(rotary_dim) * 8; }
};

template <int D, bool kInter>
__global__ void __launch_bounds__(kRopeThreads, 3) append_rope_fp8_window_kernel(const __grid_constant__ RopeParams p)
{
    using W = RopeWin<D>;
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ int32_t s_lead, s_slot[16];
    const int stride = W::tab_stride(p.rotary_dim);
    float *cs = reinterpret_cast<float *>(sm + 2 * W::kTensorB);
    __shared__ int32_t pos[PKV_ROPE_MAX_AXES * kRopeTabTokens];
    RopeTab tab{cs, cs + W::kTabRows * stride, pos, stride};
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t t0 = blockIdx.x * 16, nt = min(16, p.num_tokens - t0);
    const int32_t h0 = blockIdx.y * W::kHG, nh = min(W::kHG, p.hkv - h0);
    tab.begin(p, t0, min(W::kTabRows, p.num_tokens - t0));
    // thread (i, j) checks token i's block: is its j-th slot written by the
    // j-th token from its first on?  A token whose block is whole and begins
    // with it is the window's lead.
    if (threadIdx.x == 0) s_lead = -1;
    __syncthreads();
    {
        const int32_t tw = t0 + (threadIdx.x >> 4), j = threadIdx.x & 15;
        int32_t s0 = -1;
        bool ok = false;
        if (tw < p.num_tokens) {
            s0 = __ldg(p.slot_mapping + tw);
            const int32_t u = tw - (s0 & 15) + j;
            ok = static_cast<uint32_t>(s0) < static_cast<uint32_t>(p.num_slots) && u >= 0 && u < p.num_tokens &&
                 __ldg(p.slot_mapping + u) == (s0 & ~15) + j;
        }
        const uint32_t m = __ballot_sync(0xffffffffu, ok);
        const bool whole = ((m >> (lane & 16)) & 0xFFFFu) == 0xFFFFu;
        if (j == 0) {
            s_slot[threadIdx.x >> 4] = whole ? -1 : s0;  // left to the per-token path
            if (whole && (s0 & 15) == 0) s_lead = tw;
        }
    }
    __syncthreads();
    const int32_t lead = s_lead;
    if (lead >= 0) {  // the block's K and V rows, 16 bytes per asynchronous copy
        constexpr int kRowChunks = D / 8;
        for (int q = threadIdx.x; q < 2 * W::kHG * 16 * kRowChunks; q += kRopeThreads) {
            const int col = q % kRowChunks, hh = (q / kRowChunks) % W::kHG;
            const int tok = (q / (kRowChunks * W::kHG)) % 16, tensor = q / (kRowChunks * W::kHG * 16);
            if (hh >= nh) continue;
            const uint4 *src = (tensor ? static_cast<const uint4 *>(p.v_new) + p.v_stride * (lead + tok)
                                       : static_cast<const uint4 *>(p.k_new) + p.k_stride * (lead + tok)) +
                               (h0 + hh) * kRowChunks + col;
            const uint32_t dst = smem_u32(sm + tensor * W::kTensorB + (hh * 16 + tok) * W::kRowB + col * 16);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    const int32_t covered = lead >= 0 ? max(lead + 16 - t0, nt) : nt;  // the table's tokens: <= 31, within the call
    const int32_t per_y = (p.hq + gridDim.y - 1) / gridDim.y;
    const int32_t row0 = min(static_cast<int32_t>(blockIdx.y) * per_y, p.hq), row1 = min(row0 + per_y, p.hq);
    rope_rows<false, kInter>(p, tab, t0, nt, row0, row1, [&]() { tab.fill(p, covered); });
    if (lead >= 0) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        const int32_t blk = __ldg(p.slot_mapping + lead) >> 4;
        const float ks = p.k_scale, vs = p.v_scale, kr = __frcp_rn(ks), vr = __frcp_rn(vs);
        // per head: D items of one K chunk (or D/2 of two), then D/2 items of two
        // V chunks (dims n and n + 1 share their 4-byte shared-memory reads).
        // Two K chunks at once where a pair's dims lie whole 64-dim groups apart:
        // chunk r < D/2 and its partner's share their rows, cosines and sines.
        const bool both = !kInter && D >= 128 && p.rotary_dim == D;
        const int k_items = both ? D / 2 : D, items = k_items + D / 2;
        for (int q = threadIdx.x; q < nh * items; q += kRopeThreads) {
            const int hh = q / items, r = q - hh * items;
            const int64_t tile = (static_cast<int64_t>(blk) * p.hkv + h0 + hh) * (16 * D);
            if (r < k_items) {
                // byte 16c of the K tile: c = grp*64 + half*32 + t8*4 + cc; token
                // half*8 + t8, words kk: dims grp*64 + 16kk + 2cc + {0, 1, 8, 9}
                const int grp = r >> 6, tok = ((r >> 5) & 1) * 8 + ((r >> 2) & 7), cc = r & 3;
                const uint32_t row = smem_u32(sm + (hh * 16 + tok) * W::kRowB);
                const float *c = tab.c + (lead - t0 + tok) * stride, *sn = tab.s + (lead - t0 + tok) * stride;
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.k_pool) + tile) + r;
                uint32_t w4[4];
                if (both) {
                    uint32_t z4[4];
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        float2 y1[2], y2[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int d = grp * 64 + kk * 16 + 2 * cc + 8 * e;
                            const uint32_t xw = lds32(row + 2 * d), yw = lds32(row + 2 * d + D);
                            const float2 fc = *reinterpret_cast<const float2 *>(c + d);
                            const float2 fs = *reinterpret_cast<const float2 *>(sn + d);
                            const uint64_t x = f2_pack(bf16lo_to_f32(xw), bf16hi_to_f32(xw));
                            const uint64_t y = f2_pack(bf16lo_to_f32(yw), bf16hi_to_f32(yw));
                            const uint64_t fc2 = f2_pack(fc.x, fc.y);
                            f2_unpack(f2_fma(x, fc2, f2_mul(y, f2_pack(-fs.x, -fs.y))), y1[e].x, y1[e].y);
                            f2_unpack(f2_fma(y, fc2, f2_mul(x, f2_pack(fs.x, fs.y))), y2[e].x, y2[e].y);
                        }
                        w4[kk] = quant4f(y1[0], y1[1], ks, kr);
                        z4[kk] = quant4f(y2[0], y2[1], ks, kr);
                    }
                    __stcs(dst + D / 2, make_uint4(z4[0], z4[1], z4[2], z4[3]));
                } else {
                    const auto word = [&](int i) { return lds32(row + 4 * i); };
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const int d0 = grp * 64 + kk * 16 + 2 * cc;
                        w4[kk] = quant4f(rope_bf16_pair<kInter>(p, word, d0, c, sn),
                                         rope_bf16_pair<kInter>(p, word, d0 + 8, c, sn), ks, kr);
                    }
                }
                __stcs(dst, make_uint4(w4[0], w4[1], w4[2], w4[3]));
            } else {
                // bytes 16c and 16(c + 4) of the V tile, c = g32*32 + n*4 + cq, n
                // even: words jn of chunk c hold dim g32*32 + 8jn + n of tokens
                // 2cq, 2cq + 1, 2cq + 8, 2cq + 9, those of chunk c + 4 dim + 1
                const int v = r - k_items;
                const int g32 = v >> 4, n = ((v >> 2) & 3) * 2, cq = v & 3;
                const uint32_t vb = smem_u32(sm + W::kTensorB + (hh * 16 + 2 * cq) * W::kRowB);
                uint32_t w0[4], w1[4];
#pragma unroll
                for (int jn = 0; jn < 4; ++jn) {
                    const uint32_t at = vb + (g32 * 32 + jn * 8 + n) * 2;
                    const uint32_t x0 = lds32(at), x1 = lds32(at + W::kRowB);
                    const uint32_t x8 = lds32(at + 8 * W::kRowB), x9 = lds32(at + 9 * W::kRowB);
                    w0[jn] = quant4(__byte_perm(x0, x1, 0x5410), __byte_perm(x8, x9, 0x5410), vs, vr);
                    w1[jn] = quant4(__byte_perm(x0, x1, 0x7632), __byte_perm(x8, x9, 0x7632), vs, vr);
                }
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.v_pool) + tile) + g32 * 32 + n * 4 + cq;
                __stcs(dst, make_uint4(w0[0], w0[1], w0[2], w0[3]));
                __stcs(dst + 4, make_uint4(w1[0], w1[1], w1[2], w1[3]));
            }
        }
    }
    // tokens whose block is not whole: four kv heads of a token at a time per warp
    constexpr int kH = W::kHG < 4 ? W::kHG : 4;
    const int groups = (nh + kH - 1) / kH;
    for (int32_t i = warp; i < nt * groups; i += kRopeThreads / 32) {
        const int32_t tt = i / groups, h = (i - tt * groups) * kH, slot = s_slot[tt];
        if (slot < 0) continue;
        if (slot >= p.num_slots) {
            if (lane == 0) report(p.status, PKV_DEV_BAD_SLOT);
            continue;
        }
        rope_fp8_heads<kInter, kH>(p, tab.c + tt * stride, tab.s + tt * stride, t0 + tt, h0 + h, min(nh - h, kH), slot,
                                   lane);
    }
}

template <int D, bool kInter>
static cudaError_t launch_rope_window(const RopeParams &p, cudaStream_t stream)
{
    using W = RopeWin<D>;
    auto kern = append_rope_fp8_window_kernel<D, kInter>;
    const int smem = W::smem(p.rotary_dim);
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, W::smem(2 * kRopeMaxPairs));
    if (err != cudaSuccess) return err;
    return launch_pdl(kern, dim3((p.num_tokens + 15) / 16, (p.hkv + W::kHG - 1) / W::kHG), dim3(kRopeThreads), smem,
                      stream, p);
}

// Calls of at least this many tokens into FP8 pools write whole tiles (measured
// with 32 q and 8 kv heads of 128 dims, per token against windows: 512 tokens
// 8.9 against 13.3 us, 1024 13.7 against 14.5, 2048 25 against 20, 8192 89 against 48:
// they cross a little above it).  Other head counts and sizes were not measured.
constexpr int32_t kRopeWindowTokens = 1024;

cudaError_t launch_append_rope(const RopeParams &params, pkv_dtype dtype, int num_sms, cudaStream_t stream)
{
    RopeParams p = params;
    prof_begin(PKV_KERNEL_APPEND, stream);
    cudaError_t err;
    if (dtype == PKV_FP8_E4M3 && p.num_tokens >= kRopeWindowTokens) {
        err = p.head_dim == 64    ? (p.interleaved ? launch_rope_window<64, true>(p, stream)
                                                   : launch_rope_window<64, false>(p, stream))
              : p.head_dim == 128 ? (p.interleaved ? launch_rope_window<128, true>(p, stream)
                                                   : launch_rope_window<128, false>(p, stream))
                                  : (p.interleaved ? launch_rope_window<256, true>(p, stream)
                                                   : launch_rope_window<256, false>(p, stream));
    } else {
        const int32_t rows = p.hq + (dtype == PKV_FP8_E4M3 ? 1 : 2) * p.hkv;
        const int32_t vec = dtype == PKV_F32 ? 4 : 8;
        const int32_t units = p.head_dim / vec - p.rotary_dim / (2 * vec);
        // as many tokens per CTA as its threads can take at once, while that
        // leaves three CTAs per SM, or one where more tokens only put idle
        // threads to work (few heads); the rows of a few tokens are dealt to
        // several CTAs.  32 q and 8 kv heads of 128 dims, 2048 bf16 tokens:
        // 12.0 us with 4 tokens per CTA, 13.3 with 2; 8192: 38.9 us = 5.2 TB/s.
        const int32_t lanes = kRopeThreads / units;
        p.tokens_per_cta = 1;
        for (int32_t n = 2; n <= std::min(kRopeMaxTokens, lanes); n *= 2)
            if (p.num_tokens / n >= 3 * num_sms || (n * rows <= 2 * lanes && p.num_tokens / n >= num_sms))
                p.tokens_per_cta = n;
        const int32_t gx = (p.num_tokens - 1) / p.tokens_per_cta + 1;
        int32_t gy = std::max(1, std::min((2 * num_sms - 1) / gx + 1, (rows + 7) / 8));
        p.rows_per_cta = (rows + gy - 1) / gy;
        gy = (rows + p.rows_per_cta - 1) / p.rows_per_cta;
        void (*kern)(RopeParams) =
            dtype == PKV_FP8_E4M3 ? (p.interleaved ? append_rope_fp8_kernel<true> : append_rope_fp8_kernel<false>)
            : dtype == PKV_F32    ? (p.interleaved ? append_rope_kernel<true, true> : append_rope_kernel<true, false>)
                                  : (p.interleaved ? append_rope_kernel<false, true> : append_rope_kernel<false, false>);
        err = launch_pdl(kern, dim3(gx, gy), dim3(kRopeThreads), 0, stream, p);
    }
    prof_end(PKV_KERNEL_APPEND, stream);
    return err;
}

}  // namespace pkv
