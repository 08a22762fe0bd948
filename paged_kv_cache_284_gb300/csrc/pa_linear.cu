// pa_linear.cu -- linear attention with a decay per head: the recurrent form.
//   S_t = e^(g_t) S_(t-1) + k_t v_t^T,   o_t = scale q_t S_t
// A state S (head_dim x head_dim, fp32) belongs to a request and a kv head; the group's
// query heads read the same one.
//
// A CTA holds COLS columns of one state in registers (columns do not depend on each other)
// and takes the request's tokens in turn, a block of them at a time in shared memory: each
// thread has four columns of R rows, and a sum over the rows goes through shared memory, with one
// barrier for four query heads of a token.
// Bound for single tokens: HBM, each state read and written once.  256 requests of 8 kv heads of
// 128: 48.5 us a call for 270 MB, 5.6 TB/s, of which the prompts' grid beside it, which finds none,
// is one.  A warp to eight columns, with the sums over the rows in it and no barrier, took 58 us
// where this form took 47, since its 32-byte pieces of rows take HBM's pages badly; and 64 x 5 tokens
// 31 us instead of 27, where the sums' steps, not the barriers, are what is waited for.
#include <algorithm>

#include "pa_internal.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeadBatch = 4;  // query heads summed at once
constexpr int kQRows = 32;     // query rows (tokens x heads) in shared memory
constexpr int kTokens = 8;     // tokens of a block

template <int D, int COLS>
struct StepGeom {
    static constexpr int kLanes = COLS / 4;                 // lanes of a row, four columns each
    static constexpr int kSub = 32 / kLanes;                // rows side by side in a warp
    static constexpr int kRows = D / (kWarps * kSub);       // rows of a thread
    static_assert(kRows >= 1, "rows");
};

// R consecutive bf16 values of shared memory
template <int R>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *src, float (&v)[R]) {
    static_assert(R == 2 || R % 8 == 0 || R == 4, "vector loads");
    constexpr int W = R / 2;  // words
    uint32_t w[W];
    if constexpr (R == 2) {
        w[0] = *reinterpret_cast<const uint32_t *>(src);
    } else if constexpr (R == 4) {
        const uint2 x = *reinterpret_cast<const uint2 *>(src);
        w[0] = x.x, w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(src + 2 * i);
            w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
        }
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

}  // namespace

template <int D, int COLS>
__device__ __forceinline__ void step_job(const LinearParams &p) {
    using G = StepGeom<D, COLS>;
    constexpr int R = G::kRows, kSlices = D / COLS;
    __shared__ __align__(16) __nv_bfloat16 s_q[kQRows][D], s_k[kTokens][D], s_v[kTokens][COLS];
    __shared__ float s_keep[kTokens];
    __shared__ __align__(16) float s_part[2][kWarps][kHeadBatch][COLS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // From the last request to the first: batches commonly have their single tokens first, and
    // what takes longer had better not start last (192 requests of 1 token and 32 of 5 in this
    // order 46.7 us, from the first 49.5; 32 of 5 and 192 of 1 50.1 and 46.6).
    const int index = static_cast<int>(gridDim.x) - 1 - static_cast<int>(blockIdx.x);
    const int slice = index % kSlices, job = index / kSlices;
    const int b = job / p.num_kv_heads, h = job - b * p.num_kv_heads;
    const int col = (lane % G::kLanes) * 4, row0 = (warp * G::kSub + lane / G::kLanes) * R;
    const int t0 = __ldg(p.qsl + b), n = __ldg(p.qsl + b + 1) - t0;
    int in = __ldg(p.state_in + b), to = __ldg(p.state_out + b);
    if (n < 0 || t0 < 0 || t0 > p.num_tokens - n) {
        if (tid == 0) flag_status(p.status, PA_DEV_BAD_METADATA);
        return;
    }
    if (n > p.max_rows) return;
    unsigned flags = 0;
    if (in >= p.num_slots) flags |= PA_DEV_BAD_SLOT, in = -1;
    if (to >= p.num_slots) flags |= PA_DEV_BAD_SLOT, to = -1;
    if (flags && tid == 0) flag_status(p.status, flags);
    if (n == 0 && (to < 0 || to == in)) return;

    const int64_t state_size = static_cast<int64_t>(p.num_kv_heads) * D * D;
    const int64_t place = static_cast<int64_t>(h) * D * D + static_cast<int64_t>(row0) * D +
                          slice * COLS + col;
    uint64_t s[R][2];  // four columns of a row
    const float *src = p.state + in * state_size + place;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float4 x = in >= 0 ? __ldcs(reinterpret_cast<const float4 *>(src + i * D))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
        s[i][0] = f2_pack(x.x, x.y);
        s[i][1] = f2_pack(x.z, x.w);
    }

    // 16-byte pieces of `rows` rows of `len` elements
    auto fetch = [&](__nv_bfloat16 *dst, const __nv_bfloat16 *src, int64_t stride, int rows, int len) {
        const int pieces = len / 8;
        for (int i = tid; i < rows * pieces; i += kThreads) {
            const int r = i / pieces, c = i - r * pieces;
            *reinterpret_cast<uint4 *>(dst + r * len + c * 8) =
                *reinterpret_cast<const uint4 *>(src + r * stride + c * 8);
        }
    };
    const int block = max(1, min(kTokens, kQRows / p.group));
    int buf = 0;
    for (int t = t0; t < t0 + n; t += block) {
        const int m = min(block, t0 + n - t);
        if (t > t0) __syncthreads();
        fetch(&s_k[0][0], p.k + t * p.k_stride + h * D, p.k_stride, m, D);
        fetch(&s_v[0][0], p.v + t * p.v_stride + h * D + slice * COLS, p.v_stride, m, COLS);
        if (tid < m) {
            // a positive or NaN logarithm counts as 0, so that no state grows by its decay
            const float g = __ldg(p.decay + static_cast<int64_t>(t + tid) * p.decay_stride + h);
            s_keep[tid] = expf(g < 0.f ? g : 0.f);
        }
        // (groups of more than kQRows heads: one token, several turns)
        for (int g0 = 0; g0 < p.group; g0 += kQRows) {
            const int heads = min(kQRows, p.group - g0);
            if (g0 > 0) __syncthreads();
            for (int i = 0; i < m; ++i)
                fetch(&s_q[i * heads][0], p.q + (t + i) * p.q_stride + (h * p.group + g0) * D, D,
                      heads, D);
            __syncthreads();
            for (int i = 0; i < m; ++i) {
                if (g0 == 0) {
                    const uint64_t keep = f2_pack(s_keep[i], s_keep[i]);
                    const uint2 raw = *reinterpret_cast<const uint2 *>(&s_v[i][col]);
                    const uint64_t v0 = f2_pack(__uint_as_float(raw.x << 16),
                                             __uint_as_float(raw.x & 0xFFFF0000u));
                    const uint64_t v1 = f2_pack(__uint_as_float(raw.y << 16),
                                             __uint_as_float(raw.y & 0xFFFF0000u));
                    float k[R];
                    load_row<R>(&s_k[i][row0], k);
#pragma unroll
                    for (int x = 0; x < R; ++x) {
                        const uint64_t kk = f2_pack(k[x], k[x]);
                        s[x][0] = f2_fma(keep, s[x][0], f2_mul(kk, v0));
                        s[x][1] = f2_fma(keep, s[x][1], f2_mul(kk, v1));
                    }
                }
                for (int j0 = 0; j0 < heads; j0 += kHeadBatch) {
                    const int some = min(kHeadBatch, heads - j0);
                    for (int j = 0; j < some; ++j) {
                        uint64_t o0 = f2_pack(0.f, 0.f), o1 = o0;
                        float q[R];
                        load_row<R>(&s_q[i * heads + j0 + j][row0], q);
#pragma unroll
                        for (int x = 0; x < R; ++x) {
                            const uint64_t y = f2_pack(q[x], q[x]);
                            o0 = f2_fma(y, s[x][0], o0);
                            o1 = f2_fma(y, s[x][1], o1);
                        }
                        float4 o;
                        f2_unpack(o0, o.x, o.y);
                        f2_unpack(o1, o.z, o.w);
#pragma unroll
                        for (int x = G::kLanes; x < 32; x <<= 1) {
                            o.x += __shfl_xor_sync(0xffffffffu, o.x, x);
                            o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
                            o.z += __shfl_xor_sync(0xffffffffu, o.z, x);
                            o.w += __shfl_xor_sync(0xffffffffu, o.w, x);
                        }
                        if (lane < G::kLanes)
                            *reinterpret_cast<float4 *>(&s_part[buf][warp][j][col]) = o;
                    }
                    __syncthreads();
                    // (the next sums go to the other buffer, and meet this one's readers at its
                    // barrier)
                    for (int y = tid; y < some * (COLS / 2); y += kThreads) {
                        const int j = y / (COLS / 2), c = y % (COLS / 2) * 2;
                        float2 o = make_float2(0.f, 0.f);
#pragma unroll
                        for (int w = 0; w < kWarps; ++w) {
                            const float2 x = *reinterpret_cast<const float2 *>(&s_part[buf][w][j][c]);
                            o.x += x.x;
                            o.y += x.y;
                        }
                        *reinterpret_cast<uint32_t *>(
                            p.out + (static_cast<int64_t>(t + i) * p.num_q_heads + h * p.group + g0 +
                                     j0 + j) * D + slice * COLS + c) =
                            pack_bf16x2(o.x * p.scale, o.y * p.scale);
                    }
                    buf ^= 1;
                }
            }
        }
    }
    if (to < 0) return;
    float *dst = p.state + to * state_size + place;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float4 x;
        f2_unpack(s[i][0], x.x, x.y);
        f2_unpack(s[i][1], x.z, x.w);
        __stcs(reinterpret_cast<float4 *>(dst + i * D), x);
    }
}

template <int D, int COLS>
__global__ void __launch_bounds__(kThreads) linear_step_kernel(const LinearParams p) {
    // Beside the prompt kernel, which has waited for whatever wrote the inputs, there is nothing
    // to wait for: its rows and slots are others.  This grid still ends after that one, so that
    // what follows comes after both: its last block waits (waiting blocks would hold the SMs
    // that the prompts leave free: 8 x 512 prompt tokens, 192 single ones and 32 x 5 then take
    // 4 us more).
    if (!p.overlap) pdl_wait();
    pdl_trigger();
    step_job<D, COLS>(p);
    if (p.overlap && blockIdx.x == gridDim.x - 1) pdl_wait();
}


namespace {

template <int D, int COLS>
int launch(const LinearParams &p, cudaStream_t s) {
    const int64_t ctas = static_cast<int64_t>(p.num_seqs) * p.num_kv_heads * (D / COLS);
    PdlLaunch l(static_cast<unsigned>(ctas), kThreads, 0, s);
    return launch_kernel(l, linear_step_kernel<D, COLS>, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

int launch_linear_step(const LinearParams &p, int head_dim, cudaStream_t s) {
    return head_dim == 128 ? launch<128, 64>(p, s) : launch<64, 32>(p, s);
}

}  // namespace pa
