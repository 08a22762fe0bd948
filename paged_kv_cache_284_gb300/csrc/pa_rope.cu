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
#include <cuda_fp8.h>

#include "pa_internal.cuh"

namespace pa {

namespace {

__device__ __forceinline__ uint64_t turn_fraction(double inv_freq) {
    const double turns = inv_freq * 0.15915494309189533577;  // 1 / 2 pi
    return static_cast<uint64_t>((turns - floor(turns)) * 18446744073709551616.0);
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

// One thread per (token, head, 8 elements): heads 0..Hq-1 are q's, then k's,
// then v's.
__global__ void __launch_bounds__(256) rope_write_kernel(const RopeParams p) {
    pdl_wait();
    pdl_trigger();
    const int heads = p.num_q_heads + 2 * p.num_kv_heads;
    const int pieces = p.head_dim / 8;
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int64_t per_token = static_cast<int64_t>(heads) * pieces;
    const int64_t t = idx / per_token;
    if (t >= p.num_tokens) return;
    const int rem = static_cast<int>(idx - t * per_token);
    const int head = rem / pieces, piece = rem - head * pieces;
    const bool is_q = head < p.num_q_heads;
    const bool is_k = !is_q && head < p.num_q_heads + p.num_kv_heads;
    const int h = is_q ? head : head - p.num_q_heads - (is_k ? 0 : p.num_kv_heads);
    int64_t row = 0;
    if (!is_q) {
        const int64_t s = __ldg(p.slots + t);
        if (s < 0) return;
        const int64_t blk = s / p.block_size;
        if (blk >= p.num_blocks) {
            flag_status(p.status, PA_DEV_BAD_SLOT);
            return;
        }
        row = (blk * p.num_kv_heads + h) * p.block_size + (s - blk * p.block_size);
    }
    const __nv_bfloat16 *src = (is_q   ? p.q + t * p.q_stride
                                : is_k ? p.k + t * p.k_stride
                                       : p.v + t * p.v_stride) +
                               static_cast<int64_t>(h) * p.head_dim;
    const uint4 mine = *reinterpret_cast<const uint4 *>(src + piece * 8);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = bf16_at(mine, i);
    if ((is_q || is_k) && piece * 8 < p.rot_dim) {
        const int half = p.rot_dim / 2;
        auto cs_of = [&](int f) {
            int a = p.axis ? __ldg(p.axis + f) : 0;
            if (a < 0 || a >= p.num_axes) {
                flag_status(p.status, PA_DEV_BAD_METADATA);
                a = min(max(a, 0), p.num_axes - 1);
            }
            return turn_cos_sin(__ldg(p.positions + static_cast<int64_t>(a) * p.num_tokens + t),
                                turn_fraction(__ldg(p.inv_freq + f)), p.attn_factor);
        };
        if (p.adjacent) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 cs = cs_of(piece * 4 + i);
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = a * cs.x - b * cs.y;
                x[2 * i + 1] = b * cs.x + a * cs.y;
            }
        } else {
            const bool second = piece * 8 >= half;
            const uint4 other =
                *reinterpret_cast<const uint4 *>(src + (second ? piece * 8 - half : piece * 8 + half));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 cs = cs_of(piece * 8 + i - (second ? half : 0));
                const float y = bf16_at(other, i);
                x[i] = second ? x[i] * cs.x + y * cs.y : x[i] * cs.x - y * cs.y;
            }
        }
    }
    if (is_q) {
        *reinterpret_cast<uint4 *>(p.q_out + (t * p.num_q_heads + h) * p.head_dim + piece * 8) =
            pack8_bf16(x);
        return;
    }
    void *cache = is_k ? p.k_cache : p.v_cache;
    if (p.fp8)
        static_cast<uint2 *>(cache)[row * pieces + piece] =
            pack8_e4m3(x, __ldg((is_k ? p.k_scale : p.v_scale) + h));
    else
        static_cast<uint4 *>(cache)[row * pieces + piece] = pack8_bf16(x);
}

int launch_rope_write(const RopeParams &p, cudaStream_t s) {
    if (p.num_tokens == 0) return PA_OK;
    const int64_t work = static_cast<int64_t>(p.num_tokens) *
                         (p.num_q_heads + 2 * p.num_kv_heads) * (p.head_dim / 8);
    PdlLaunch l(static_cast<unsigned>((work + 255) / 256), 256, 0, s);
    return launch_kernel(l, rope_write_kernel, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
