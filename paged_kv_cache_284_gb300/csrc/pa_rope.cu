// pa_rope.cu -- rotary positions with several axes, fused with the cache write
// (the embedding comes before reshape_and_cache; "vLLM中如何实现大模型推理加速
// 技术？": position_id counts from the hit, so positions are an input).
//
// Pair i of a head, (a, b), is turned by t = position * inv_freq[i]:
//   a' = f (a cos t - b sin t),  b' = f (b cos t + a sin t).
// The angle is only wanted modulo one turn.  inv_freq / 2 pi is held as a
// 64-bit binary fraction of a turn, and position * fraction in wrapping 64-bit
// integers IS that product modulo one turn: exact for every int32 position,
// negative ones too, with a step of 2^-64 turns (2^-33 after the largest
// position).  Its top 32 bits, as a signed fraction x in [-1/2, 1/2) of a
// turn, give cos and sin through sincospif(2 x).
//
// The work is HBM traffic: q, k and v read once, q_out and the cache rows
// written once.  A warp takes one token (or a run of its heads): its lanes
// turn each frequency once, two per lane, share cos and sin through shared
// memory, and then each lane keeps the 8 frequencies of "its" 16 elements of a
// head in registers while it walks over the heads, kBatch of them loaded
// ahead.  The frequencies' fractions stay in registers from token to token.
#include <algorithm>

#include <cuda_fp8.h>

#include "pa_internal.cuh"

namespace pa {

namespace {

// inv_freq / 2 pi modulo one turn as a 64-bit fraction, in integers (the
// FP64 pipe is narrow here): the mantissa m in [2^63, 2^64) times 1 / 2 pi =
// C 2^-66 keeps its upper 64 bits, more than the double itself holds.
__device__ __forceinline__ uint64_t turn_fraction(double inv_freq) {
    const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(inv_freq));
    const int e = static_cast<int>((bits >> 52) & 0x7ff);
    if (e == 0) return 0;  // zero and subnormal
    // |inv_freq| = m * 2^(e - 1023 - 63), 1 / 2 pi = C * 2^-66 with C in [2^63, 2^64)
    const uint64_t m = (bits << 11) | (1ull << 63);
    const uint64_t C = 0xA2F9836E4E441529ull;
    // hi * 2^64 ~ m * C, so the turns are hi * 2^(e - 1023 - 63 - 66 + 64); the
    // fraction is the turns times 2^64, its bits above 2^64 being whole turns
    const uint64_t hi = __umul64hi(m, C);
    const int shift = e - 1023 - 63 - 66 + 64 + 64;  // 0 at e = 1024
    const uint64_t f = shift >= 64 || shift <= -64 ? 0 : shift >= 0 ? hi << shift : hi >> -shift;
    return (bits >> 63) ? 0 - f : f;
}

// cos and sin, times f, of `position` * (the angle per position as a
// fraction of a turn).
__device__ __forceinline__ float2 turn_cos_sin(int position, uint64_t fraction, float f) {
    const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(position)) * fraction;
    const float x = static_cast<float>(static_cast<int32_t>(t >> 32)) * (1.f / 2147483648.f);
    float s, c;
    sincospif(x, &s, &c);  // x = twice the signed fraction
    return make_float2(c * f, s * f);
}

__device__ __forceinline__ float bf16_at(const uint4 &v, int i) {
    const uint32_t w = reinterpret_cast<const uint32_t *>(&v)[i >> 1];
    return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
}

__device__ __forceinline__ uint4 pack8_bf16(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// Eight elements to e4m3 codes of x / s: the rounding of the cache write.
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float s) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(
                   make_float2(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s)),
                   __NV_SATFINITE, __NV_E4M3) &
               0xFFFFu;
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

}  // namespace

// Heads loaded ahead by a lane (two 16-byte pieces each).
constexpr int kBatch = 4;
constexpr int kRopeWarps = 4;
constexpr int kMaxFreqs = 64;  // head_dim 128

// ADJ: pairs of neighbours, else pairs across the two halves of the rotated
// part.  A lane holds two 16-byte pieces of a head: 8 pairs, or 16 elements to
// be copied (ADJ: 4 pairs or 8 elements each).
template <bool FP8, bool ADJ>
__global__ void __launch_bounds__(32 * kRopeWarps, 4) rope_write_kernel(const RopeParams p) {
    __shared__ float2 s_cs[kRopeWarps][kMaxFreqs];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int half = p.rot_dim / 2;
    pdl_wait();
    pdl_trigger();
    // this lane's two frequencies and where their positions are
    uint64_t frac[2] = {0, 0};
    const int32_t *pos[2] = {p.positions, p.positions};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int f = lane + 32 * i;
        if (f >= half) continue;
        frac[i] = turn_fraction(__ldg(p.inv_freq + f));
        int a = p.axis ? __ldg(p.axis + f) : 0;
        if (a < 0 || a >= p.num_axes) {
            flag_status(p.status, PA_DEV_BAD_METADATA);
            a = min(max(a, 0), p.num_axes - 1);
        }
        pos[i] += static_cast<int64_t>(a) * p.num_tokens;
    }
    const int units = p.head_dim / 16;  // lanes per head: 4 or 8
    const int u = lane % units, slot = lane / units, per_iter = 32 / units;
    // Element offsets of the lane's two pieces in a head, chosen so that
    // neighbouring lanes hold neighbouring pieces: the two halves of the
    // rotated part and of the rest, or (neighbours paired) of the head.
    const int rot = p.rot_dim, rot_units = rot / 16;
    const int e0 = ADJ || u < rot_units ? u * 8 : rot + (u - rot_units) * 8;
    const int e1 = e0 + (ADJ ? p.head_dim / 2 : u < rot_units ? half : (p.head_dim - rot) / 2);
    const bool rot0 = e0 < rot, rot1 = e1 < rot;
    // first frequency of each piece (a half layout's two pieces share theirs)
    const int f0 = ADJ ? e0 / 2 : e0, f1 = ADJ ? e1 / 2 : 0;
    const int heads = p.num_q_heads + 2 * p.num_kv_heads;
    const int64_t items = static_cast<int64_t>(p.num_tokens) * p.parts;
    float2(&cs_of)[kMaxFreqs] = s_cs[warp];

    for (int64_t item = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp; item < items;
         item += static_cast<int64_t>(gridDim.x) * kRopeWarps) {
        const int64_t t = p.parts == 1 ? item : item / p.parts;
        const int part = static_cast<int>(item - t * p.parts);
        const int h_end = min(heads, (part + 1) * p.part_heads);
        const int ps0 = lane < half ? __ldg(pos[0] + t) : 0;
        const int ps1 = lane + 32 < half ? __ldg(pos[1] + t) : 0;
        const int64_t sl = __ldg(p.slots + t);
        bool stored = sl >= 0;
        if (sl >= p.num_slots) {
            stored = false;
            if (part == 0 && lane == 0) flag_status(p.status, PA_DEV_BAD_SLOT);
        }
        const int s32 = stored ? static_cast<int>(sl) : 0;  // a pool has < 2^31 rows
        const int blk = s32 / p.block_size, off = s32 - blk * p.block_size;
        float2 cs[8];
        bool have_cs = false;
        for (int h0 = part * p.part_heads + slot; h0 - slot < h_end; h0 += kBatch * per_iter) {
            uint4 x0[kBatch], x1[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int hd = h0 + i * per_iter;
                const __nv_bfloat16 *src;
                if (hd < p.num_q_heads)
                    src = p.q + t * p.q_stride + hd * p.head_dim;
                else if (hd < p.num_q_heads + p.num_kv_heads)
                    src = p.k + t * p.k_stride + (hd - p.num_q_heads) * p.head_dim;
                else
                    src = p.v + t * p.v_stride + (hd - p.num_q_heads - p.num_kv_heads) * p.head_dim;
                if (hd < h_end && (stored || hd < p.num_q_heads)) {
                    x0[i] = __ldcs(reinterpret_cast<const uint4 *>(src + e0));
                    x1[i] = __ldcs(reinterpret_cast<const uint4 *>(src + e1));
                }
            }
            if (!have_cs) {
                // turn the token's frequencies while the heads are on their way
                have_cs = true;
                __syncwarp();
                if (lane < half) cs_of[lane] = turn_cos_sin(ps0, frac[0], p.attn_factor);
                if (lane + 32 < half) cs_of[lane + 32] = turn_cos_sin(ps1, frac[1], p.attn_factor);
                __syncwarp();
                if (rot0) {
#pragma unroll
                    for (int j = 0; j < (ADJ ? 4 : 8); ++j) cs[j] = cs_of[f0 + j];
                }
                if (ADJ && rot1) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) cs[4 + j] = cs_of[f1 + j];
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int hd = h0 + i * per_iter;
                const bool is_q = hd < p.num_q_heads;
                if (hd >= h_end || !(stored || is_q)) continue;
                const bool is_v = hd >= p.num_q_heads + p.num_kv_heads;
                float a[8], b[8];  // the two pieces
                const bool turn0 = rot0 && !is_v, turn1 = rot1 && !is_v;
                if (turn0 || (FP8 && !is_q)) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        a[j] = bf16_at(x0[i], j);
                        b[j] = bf16_at(x1[i], j);
                    }
                }
                if (turn0) {
                    if constexpr (ADJ) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float y = a[2 * j];
                            a[2 * j] = y * cs[j].x - a[2 * j + 1] * cs[j].y;
                            a[2 * j + 1] = a[2 * j + 1] * cs[j].x + y * cs[j].y;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float y = a[j];
                            a[j] = y * cs[j].x - b[j] * cs[j].y;
                            b[j] = b[j] * cs[j].x + y * cs[j].y;
                        }
                    }
                }
                if (ADJ && turn1) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float y = b[2 * j];
                        b[2 * j] = y * cs[4 + j].x - b[2 * j + 1] * cs[4 + j].y;
                        b[2 * j + 1] = b[2 * j + 1] * cs[4 + j].x + y * cs[4 + j].y;
                    }
                }
                // bf16 pieces that are not turned are stored as they came
                if (turn0 && (is_q || !FP8)) x0[i] = pack8_bf16(a);
                if ((ADJ ? turn1 : turn0) && (is_q || !FP8)) x1[i] = pack8_bf16(b);
                if (is_q) {
                    __nv_bfloat16 *dst = p.q_out + (t * p.num_q_heads + hd) * p.head_dim;
                    __stcs(reinterpret_cast<uint4 *>(dst + e0), x0[i]);
                    __stcs(reinterpret_cast<uint4 *>(dst + e1), x1[i]);
                    continue;
                }
                const int h = hd - p.num_q_heads - (is_v ? p.num_kv_heads : 0);
                const int64_t row =
                    (static_cast<int64_t>(blk) * p.num_kv_heads + h) * p.block_size + off;
                if constexpr (FP8) {
                    const float sc = __ldg((is_v ? p.v_scale : p.k_scale) + h);
                    uint8_t *dst =
                        static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache) + row * p.head_dim;
                    __stcs(reinterpret_cast<uint2 *>(dst + e0), pack8_e4m3(a, sc));
                    __stcs(reinterpret_cast<uint2 *>(dst + e1), pack8_e4m3(b, sc));
                } else {
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(is_v ? p.v_cache : p.k_cache) +
                                         row * p.head_dim;
                    __stcs(reinterpret_cast<uint4 *>(dst + e0), x0[i]);
                    __stcs(reinterpret_cast<uint4 *>(dst + e1), x1[i]);
                }
            }
        }
    }
}

int launch_rope_write(RopeParams p, int sms, cudaStream_t s) {
    if (p.num_tokens == 0) return PA_OK;
    // Few tokens: a token's heads are dealt to several warps, down to one
    // batch step each, so that a small step fills the SMs and has no loop.
    const int heads = p.num_q_heads + 2 * p.num_kv_heads;
    const int per_iter = 32 / (p.head_dim / 16);
    const int iters = (heads + per_iter - 1) / per_iter;
    const int64_t want = static_cast<int64_t>(sms) * 4 * kRopeWarps;
    const int64_t split = std::min<int64_t>(iters, (want + p.num_tokens - 1) / p.num_tokens);
    p.part_heads = static_cast<int>((iters + split - 1) / split) * per_iter;
    p.parts = (heads + p.part_heads - 1) / p.part_heads;
    const int64_t warps = static_cast<int64_t>(p.num_tokens) * p.parts;
    const int64_t blocks = std::min<int64_t>((warps + kRopeWarps - 1) / kRopeWarps,
                                             static_cast<int64_t>(sms) * 4);
    PdlLaunch l(static_cast<unsigned>(blocks), 32 * kRopeWarps, 0, s);
    const cudaError_t e = p.fp8 ? (p.adjacent ? launch_kernel(l, rope_write_kernel<true, true>, p)
                                              : launch_kernel(l, rope_write_kernel<true, false>, p))
                                : (p.adjacent ? launch_kernel(l, rope_write_kernel<false, true>, p)
                                              : launch_kernel(l, rope_write_kernel<false, false>, p));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
