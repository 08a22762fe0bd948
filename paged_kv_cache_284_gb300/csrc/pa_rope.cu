// pa_rope.cu -- rotary positions with several axes, fused with the cache write
// (the embedding comes before reshape_and_cache; "vLLM中如何实现大模型推理加速
// 技术？": position_id counts from the hit, so positions are an input).
//
// Pair i of a head, (a, b), is turned by t = position * inv_freq[i]:
//   a' = f (a cos t - b sin t),  b' = f (b cos t + a sin t).
// The angle is only wanted modulo one turn.  inv_freq / 2 pi is held as a
// 64-bit binary fraction of a turn, and position * fraction in wrapping 64-bit
// integers IS that product modulo one turn, for every int32 position, negative
// ones too; the fraction itself is good to 2^-64 max(1, inv_freq) turns, the
// product to 2^31 times that for the farthest position.  Its top 32 bits, as a signed fraction x in [-1/2, 1/2) of a
// turn, give cos and sin through sincospif(2 x).
//
// The work is HBM traffic: q, k and v read once, q_out and the cache rows
// written once.  All tokens' heads (q, k, v of a token in turn) form one line
// of steps, a step being the 4 or 8 heads that a warp turns at a time; every
// warp takes an equal run of it, in items of up to kItemSteps steps of one
// token.  Bulk copies bring the rows of the items ahead into the warp's own
// ring in shared memory, so that bytes in flight cost no registers; the lanes
// turn each frequency once per item, two per lane, and share cos and sin
// through shared memory; then each lane keeps the frequencies of its 16
// elements of a head in registers while it walks over the heads.
// 4096 tokens of 32 + 8 + 8 heads, three axes, bf16 (101 MB): 18.3 us, 5.5 TB/s,
// 0.82 of the measured copy bandwidth; 16384 tokens into an e4m3 pool (369 MB)
// 66.2 us, 0.83; 8 tokens 3.5 us, most of it the launch.  A block per token with
// plain loads took 21-26 and 79-106 us.
#include <algorithm>

#include <cuda_fp8.h>

#include "pa_long.cuh"

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

// Pieces as four packed pairs of fp32 (elements 2 i and 2 i + 1): the two-wide
// multiply and FMA of this architecture halve the rotation's and the
// quantisation's instructions.
__device__ __forceinline__ void unpack8(const uint4 &v, uint64_t (&x)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack8_bf16(const uint64_t (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        f2_unpack(x[i], lo, hi);
        w[i] = pack_bf16x2(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// a b + c rounded down.  A remainder is exact in any rounding; rounded down, an
// exact zero is -0, and -0 added to a zero leaves that zero its sign.
__device__ __forceinline__ uint64_t f2_fma_down(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// A cache row's scale s and r = 1 / s (rounded to nearest).
struct Scale {
    float s, r;
    bool plain;  // s is far from the ends of fp32's range
};
__device__ __forceinline__ Scale make_scale(float s) {
    return {s, __frcp_rn(s), s > 0x1p-60f && s < 0x1p60f};
}
// Eight elements to e4m3 codes of x / s, the rounding of the cache write: x / s
// correctly rounded wherever its code depends on it.  The quotient x r, then
// twice the remainder step of P. Markstein ("Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990): the result is the
// rounded quotient when r is the rounded reciprocal and the quotient before is
// within one unit in the last place.  Quotients past 512 (infinities, whose
// remainder is no number) go the plain way; those whose remainder is subnormal
// have the code of zero, signed as x is; so has -0 (f2_fma_down); NaN stays NaN.
__device__ __forceinline__ uint2 pack8_e4m3(const uint64_t (&x)[4], const Scale &sc) {
    const uint64_t r2 = f2_pack(sc.r, sc.r), s2 = f2_pack(-sc.s, -sc.s);
    uint64_t q[4];
    float lo[4], hi[4], most = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i] = f2_mul(x[i], r2);
        f2_unpack(q[i], lo[i], hi[i]);
        most = max3(most, fabsf(lo[i]), fabsf(hi[i]));
    }
    if (sc.plain && most < 512.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            q[i] = f2_fma(f2_fma_down(q[i], s2, x[i]), r2, q[i]);
            q[i] = f2_fma(f2_fma_down(q[i], s2, x[i]), r2, q[i]);
            f2_unpack(q[i], lo[i], hi[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f2_unpack(x[i], lo[i], hi[i]);
            lo[i] = __fdiv_rn(lo[i], sc.s);
            hi[i] = __fdiv_rn(hi[i], sc.s);
        }
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(lo[i], hi[i]), __NV_SATFINITE, __NV_E4M3) &
               0xFFFFu;
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

}  // namespace

constexpr int kRopeWarps = 8;
constexpr int kRopeCtas = 2;   // per SM
// Steps of an item and entries of a warp's ring.  us per call, 4096 tokens bf16 /
// 16384 tokens e4m3: 6 x 2 19.5 / 65.0, 4 x 2 20.0 / 64.7, 12 x 2 (one block
// per SM) 23.0 / 74.7, 3 x 3 20.5 / 63.5.
constexpr int kItemSteps = 6;
constexpr int kRing = 2;
constexpr int kMaxFreqs = 64;  // head_dim 128
constexpr int kStepBytes = 1024;  // a step's rows: 32 lanes x 2 pieces of 16 bytes
constexpr int kEntryBytes = kItemSteps * kStepBytes;
// [warps][ring] rows, [warps][kMaxFreqs] cos, then sin, [warps][ring] barriers
constexpr int kRopeSmem =
    kRopeWarps * (kRing * (kEntryBytes + static_cast<int>(sizeof(uint64_t))) +
                  kMaxFreqs * static_cast<int>(sizeof(float2)));

// A place in a warp's run of the line: step `step` of token t, `left` steps in all.
struct Cursor {
    int64_t t;
    int step;
    int64_t left;
    __device__ __forceinline__ int item(int steps) const {  // steps of the item here
        return static_cast<int>(min(static_cast<int64_t>(min(kItemSteps, steps - step)), left));
    }
    __device__ __forceinline__ void advance(int n, int steps) {
        left -= n;
        step += n;
        if (step == steps) {
            step = 0;
            ++t;
        }
    }
};

// ADJ: pairs of neighbours, else pairs across the two halves of the rotated
// part.  A lane holds two 16-byte pieces of a head: 8 pairs, or 16 elements to
// be copied (ADJ: 4 pairs or 8 elements each).
template <bool FP8, bool ADJ>
__global__ void __launch_bounds__(32 * kRopeWarps, kRopeCtas)
    rope_write_kernel(const RopeParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int half = p.rot_dim / 2;
    uint8_t *ring = smem + warp * kRing * kEntryBytes;
    float *cos_of = reinterpret_cast<float *>(smem + kRopeWarps * kRing * kEntryBytes) +
                    warp * 2 * kMaxFreqs;
    float *sin_of = cos_of + kMaxFreqs;
    uint64_t *full = reinterpret_cast<uint64_t *>(
                         smem + kRopeWarps * (kRing * kEntryBytes +
                                              kMaxFreqs * static_cast<int>(sizeof(float2)))) +
                     warp * kRing;
    if (lane == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_wait();
    pdl_trigger();
    const int units = p.head_dim / 16;  // lanes per head: 4 or 8
    const int per_step = 32 / units;    // heads of a step
    const int first_k = p.num_q_heads, first_v = first_k + p.num_kv_heads;
    const int heads = first_v + p.num_kv_heads;
    const int steps = (heads + per_step - 1) / per_step;  // of a token
    // this warp's run: an equal share of num_tokens * steps
    const int64_t total = static_cast<int64_t>(p.num_tokens) * steps;
    const int runs = static_cast<int>(gridDim.x) * kRopeWarps;
    const int me = static_cast<int>(blockIdx.x) * kRopeWarps + warp;
    Cursor at;
    if (total < (1ll << 31)) {
        const unsigned all = static_cast<unsigned>(total), share = all / runs, more = all - share * runs;
        const unsigned begin = me * share + min(static_cast<unsigned>(me), more);
        at.left = share + (static_cast<unsigned>(me) < more ? 1 : 0);
        at.t = begin / steps;
        at.step = static_cast<int>(begin - static_cast<unsigned>(at.t) * steps);
    } else {
        const int64_t share = total / runs, more = total - share * runs;
        const int64_t begin = me * share + min(static_cast<int64_t>(me), more);
        at.left = share + (me < more ? 1 : 0);
        at.t = begin / steps;
        at.step = static_cast<int>(begin - at.t * steps);
    }

    // read once: first to leave L2 (4096 tokens: 19.3 -> 18.3 us)
    const uint64_t policy = evict_first_policy();
    // Brings an item's rows into ring entry `e` (lane 0): up to three runs of
    // heads; a token that is not stored needs q alone.
    const bool stall = p.test_stall && me == 0;
    auto fetch = [&](const Cursor &c, int n, int e) {
        if (stall && e > 0) return;
        const int h0 = c.step * per_step, h1 = min(heads, h0 + n * per_step);
        const int64_t sl = h1 > first_k ? __ldg(p.slots + c.t) : 0;
        const bool stored = sl >= 0 && sl < p.num_slots;
        uint8_t *dst = ring + e * kEntryBytes;
        const int d2 = p.head_dim * 2;  // bytes of a head
        const int end = stored ? h1 : min(h1, first_k);
        mbar_arrive_expect_tx(&full[e], static_cast<uint32_t>(max(0, end - h0) * d2));
        auto run = [&](const __nv_bfloat16 *src, int64_t stride, int a, int b) {
            const int lo = max(a, h0), hi = min(b, end);
            if (lo < hi)
                bulk_load(dst + (lo - h0) * d2, src + c.t * stride + (lo - a) * p.head_dim,
                          static_cast<uint32_t>((hi - lo) * d2), &full[e], policy);
        };
        run(p.q, p.q_stride, 0, first_k);
        run(p.k, p.k_stride, first_k, first_v);
        run(p.v, p.v_stride, first_v, heads);
    };
    Cursor ahead = at;  // the next item to fetch
    for (int i = 0; i < kRing - 1 && ahead.left > 0; ++i) {
        const int n = ahead.item(steps);
        if (lane == 0) fetch(ahead, n, i);
        ahead.advance(n, steps);
    }

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
    const int u = lane % units, slot = lane / units;
    // Element offsets of the lane's two pieces in a head, chosen so that
    // neighbouring lanes hold neighbouring pieces: the two halves of the
    // rotated part and of the rest, or (neighbours paired) of the head.
    const int rot = p.rot_dim, rot_units = rot / 16;
    const int e0 = ADJ || u < rot_units ? u * 8 : rot + (u - rot_units) * 8;
    const int e1 = e0 + (ADJ ? p.head_dim / 2 : u < rot_units ? half : (p.head_dim - rot) / 2);
    const bool rot0 = e0 < rot, rot1 = e1 < rot;
    // first frequency of each piece (a half layout's two pieces share theirs)
    const int f0 = ADJ ? e0 / 2 : e0, f1 = ADJ ? e1 / 2 : 0;

    uint32_t k = 0;  // items done
    volatile int gave_up = 0;
    while (at.left > 0) {
        const int64_t t = at.t;
        const int n = at.item(steps), e = static_cast<int>(k % kRing);
        const int h0 = at.step * per_step, h1 = min(heads, h0 + n * per_step);
        const int ps0 = lane < half ? __ldg(pos[0] + t) : 0;
        const int ps1 = lane + 32 < half ? __ldg(pos[1] + t) : 0;
        const int64_t sl = __ldg(p.slots + t);
        // (every lane is done with that entry: an item ends with a barrier)
        if (ahead.left > 0) {
            const int m = ahead.item(steps);
            if (lane == 0) fetch(ahead, m, static_cast<int>((k + kRing - 1) % kRing));
            ahead.advance(m, steps);
        }
        const bool stored = sl >= 0 && sl < p.num_slots;
        if (sl >= p.num_slots && at.step == 0 && lane == 0)
            flag_status(p.status, PA_DEV_BAD_SLOT);
        const int s32 = stored ? static_cast<int>(sl) : 0;  // a pool has < 2^31 rows
        const int blk = s32 / p.block_size, off = s32 - blk * p.block_size;
        if (h0 < first_v) {
            if (lane < half) {
                const float2 cs = turn_cos_sin(ps0, frac[0], p.attn_factor);
                cos_of[lane] = cs.x;
                sin_of[lane] = cs.y;
            }
            if (lane + 32 < half) {
                const float2 cs = turn_cos_sin(ps1, frac[1], p.attn_factor);
                cos_of[lane + 32] = cs.x;
                sin_of[lane + 32] = cs.y;
            }
        }
        __syncwarp();
        // Packed: half layout, frequencies f0 + 2 i, + 1: (c, c'), (s, s') and
        // (-s, -s'); neighbours, frequency i of each piece: (c, c) and (-s, s).
        uint64_t cc[8], ss[8];
        if constexpr (ADJ) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool turn = j < 4 ? rot0 : rot1;
                const int f = turn ? (j < 4 ? f0 + j : f1 + j - 4) : 0;
                const float c = cos_of[f], sn = sin_of[f];
                cc[j] = f2_pack(c, c);
                ss[j] = f2_pack(-sn, sn);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int f = rot0 ? f0 + 2 * j : 0;
                const float2 c = *reinterpret_cast<const float2 *>(cos_of + f);
                const float2 sn = *reinterpret_cast<const float2 *>(sin_of + f);
                cc[j] = f2_pack(c.x, c.y);
                ss[j] = f2_pack(sn.x, sn.y);
                ss[4 + j] = f2_pack(-sn.x, -sn.y);
            }
        }
        if (!warp_mbar_wait(&full[e], (k / kRing) & 1, &gave_up)) {
            if (lane == 0) {
                flag_status(p.status, PA_DEV_WAIT_TIMEOUT);
                // let copies already in flight land before the CTA exits
                for (int i = 0; i < kRing; ++i) mbar_drain(&full[(k + i) % kRing], ((k + i) / kRing) & 1);
            }
            break;
        }
        const __nv_bfloat16 *row =
            reinterpret_cast<const __nv_bfloat16 *>(ring + e * kEntryBytes);
        const int end = stored ? h1 : min(h1, first_k);
        for (int hd = h0 + slot; hd < end; hd += per_step) {
            const __nv_bfloat16 *src = row + (hd - h0) * p.head_dim;
            uint4 x0 = *reinterpret_cast<const uint4 *>(src + e0);
            uint4 x1 = *reinterpret_cast<const uint4 *>(src + e1);
            const bool is_q = hd < first_k, is_v = hd >= first_v;
            uint64_t a[4], b[4];  // the two pieces
            const bool turn0 = rot0 && !is_v, turn1 = rot1 && !is_v;
            if (turn0 || (FP8 && !is_q)) unpack8(x0, a);
            if ((ADJ ? turn1 : turn0) || (FP8 && !is_q)) unpack8(x1, b);
            if constexpr (ADJ) {
                auto turn = [](uint64_t &x, uint64_t c, uint64_t sn) {
                    float lo, hi;
                    f2_unpack(x, lo, hi);
                    x = f2_fma(f2_pack(hi, lo), sn, f2_mul(x, c));
                };
                if (turn0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) turn(a[j], cc[j], ss[j]);
                }
                if (turn1) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) turn(b[j], cc[4 + j], ss[4 + j]);
                }
            } else if (turn0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint64_t y = a[j];
                    a[j] = f2_fma(b[j], ss[4 + j], f2_mul(y, cc[j]));
                    b[j] = f2_fma(y, ss[j], f2_mul(b[j], cc[j]));
                }
            }
            // bf16 pieces that are not turned are stored as they came
            if (turn0 && (is_q || !FP8)) x0 = pack8_bf16(a);
            if ((ADJ ? turn1 : turn0) && (is_q || !FP8)) x1 = pack8_bf16(b);
            if (is_q) {
                __nv_bfloat16 *dst = p.q_out + (t * p.num_q_heads + hd) * p.head_dim;
                __stcs(reinterpret_cast<uint4 *>(dst + e0), x0);
                __stcs(reinterpret_cast<uint4 *>(dst + e1), x1);
                continue;
            }
            const int h = hd - (is_v ? first_v : first_k);
            const int64_t at = (static_cast<int64_t>(blk) * p.num_kv_heads + h) * p.block_size + off;
            void *cache = is_v ? p.v_cache : p.k_cache;
            if constexpr (FP8) {
                const Scale sc = make_scale(__ldg((is_v ? p.v_scale : p.k_scale) + h));
                uint8_t *dst = static_cast<uint8_t *>(cache) + at * p.head_dim;
                __stcs(reinterpret_cast<uint2 *>(dst + e0), pack8_e4m3(a, sc));
                __stcs(reinterpret_cast<uint2 *>(dst + e1), pack8_e4m3(b, sc));
            } else {
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(cache) + at * p.head_dim;
                __stcs(reinterpret_cast<uint4 *>(dst + e0), x0);
                __stcs(reinterpret_cast<uint4 *>(dst + e1), x1);
            }
        }
        at.advance(n, steps);
        ++k;
        __syncwarp();
    }
}

template <bool FP8, bool ADJ>
static int launch(const RopeParams &p, unsigned blocks, cudaStream_t s) {
    static PerDeviceOnce once;
    if (once_per_device(once, [] {
            return cudaFuncSetAttribute(rope_write_kernel<FP8, ADJ>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, kRopeSmem);
        }) != PA_OK)
        return PA_ERR_CUDA;
    PdlLaunch l(blocks, 32 * kRopeWarps, kRopeSmem, s);
    return launch_kernel(l, rope_write_kernel<FP8, ADJ>, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int launch_rope_write(const RopeParams &p, int sms, cudaStream_t s) {
    if (p.num_tokens == 0) return PA_OK;
    const int per_step = 32 / (p.head_dim / 16);
    const int64_t steps = (p.num_q_heads + 2 * p.num_kv_heads + per_step - 1) / per_step;
    const int64_t blocks = std::min<int64_t>((p.num_tokens * steps + kRopeWarps - 1) / kRopeWarps,
                                             static_cast<int64_t>(sms) * kRopeCtas);
    const unsigned g = static_cast<unsigned>(blocks);
    if (p.fp8) return p.adjacent ? launch<true, true>(p, g, s) : launch<true, false>(p, g, s);
    return p.adjacent ? launch<false, true>(p, g, s) : launch<false, false>(p, g, s);
}

}  // namespace pa
