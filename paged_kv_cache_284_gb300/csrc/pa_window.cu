// pa_window.cu -- attention with a sliding window and sinks over the paged
// pool: row at position p sees key j <= p with j > p - window or j < sinks.
//
// One warp per (query token, q head): lanes across the head dimension, the
// keys one after the other, with the running maximum and sum of the softmax.
#include <cuda_fp8.h>

#include "pa_internal.cuh"

namespace pa {

template <int D, bool FP8>
__global__ void __launch_bounds__(128) window_kernel(const WindowParams p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int t = static_cast<int>(w / p.num_q_heads), hq = static_cast<int>(w % p.num_q_heads);
    if (t >= p.num_q_tokens) return;
    // the request of this token: the last whose first token is not behind it
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(p.qsl + mid) <= t) lo = mid; else hi = mid - 1;
    }
    const int b = lo, q0 = __ldg(p.qsl + b), q1 = __ldg(p.qsl + b + 1);
    const int ctx = __ldg(p.ctx + b), len = __ldg(p.seq_lens + b);
    if (q0 < 0 || q1 < q0 || q1 > p.num_q_tokens || ctx < 0 || len != ctx + q1 - q0) {
        flag_status(p.status, PA_DEV_BAD_METADATA);
        return;
    }
    if (t < q0 || t >= q1) return;
    const int pos = ctx + t - q0;
    const int h = hq / p.group;
    constexpr int E = D / 32;
    float q[E], o[E], m = -INFINITY, l = 0.f;
    const int64_t row = static_cast<int64_t>(t) * p.num_q_heads + hq;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(p.q[row * D + lane * E + e]);
        o[e] = 0.f;
    }
    const float sl2 = p.scale_log2 * (FP8 ? __ldg(p.k_scale + h) : 1.f);
    const int first = max(0, pos - p.window + 1);
    auto elem = [&](const void *cache, int64_t i) {
        if constexpr (FP8)
            return static_cast<float>(static_cast<const __nv_fp8_e4m3 *>(cache)[i]);
        else
            return __bfloat162float(static_cast<const __nv_bfloat16 *>(cache)[i]);
    };
    for (int j = 0; j <= pos; ++j) {
        if (j >= p.sinks && j < first) j = first;
        int col = j / p.block_size;
        if (col >= p.bt_stride) {
            flag_status(p.status, PA_DEV_BAD_METADATA);
            col = p.bt_stride - 1;
        }
        int blk = __ldg(p.block_tables + static_cast<int64_t>(b) * p.bt_stride + col);
        if (blk < 0 || blk >= p.num_blocks) {
            flag_status(p.status, PA_DEV_BAD_BLOCK);
            blk = min(max(blk, 0), p.num_blocks - 1);
        }
        const int64_t base =
            ((static_cast<int64_t>(blk) * p.num_kv_heads + h) * p.block_size + j % p.block_size) *
                D + lane * E;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += q[e] * elem(p.k_cache, base + e);
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
        s *= sl2;
        const float nm = fmaxf(m, s), a = exp2f(m - nm), w1 = exp2f(s - nm);
        l = l * a + w1;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * a + w1 * elem(p.v_cache, base + e);
        m = nm;
    }
    const float inv = (FP8 ? __ldg(p.v_scale + h) : 1.f) / l;
#pragma unroll
    for (int e = 0; e < E; ++e) p.out[row * D + lane * E + e] = __float2bfloat16(o[e] * inv);
    if (p.lse && lane == 0) p.lse[row] = (m + log2f(l)) * 0.69314718055994530942f;
}

int launch_window(const WindowParams &p, int head_dim, bool fp8, cudaStream_t s) {
    const int64_t warps = static_cast<int64_t>(p.num_q_tokens) * p.num_q_heads;
    PdlLaunch l(static_cast<unsigned>((warps + 3) / 4), 128, 0, s);
    const cudaError_t e = fp8               ? launch_kernel(l, window_kernel<128, true>, p)
                          : head_dim == 128 ? launch_kernel(l, window_kernel<128, false>, p)
                                            : launch_kernel(l, window_kernel<64, false>, p);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
