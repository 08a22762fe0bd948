// pa_linear.cu -- linear attention with a decay per head: the recurrent form.
//   S_t = e^(g_t) S_(t-1) + k_t v_t^T,   o_t = scale q_t S_t
// A state S (head_dim x head_dim, fp32) belongs to a request and a kv head; the group's
// query heads read the same one.
//
// A CTA holds COLS columns of one state in registers (columns do not depend on each other)
// and takes the request's tokens in turn: k and q of a token in shared memory, each thread
// four columns of R rows, then a sum over the rows through shared memory.
// Bound for single tokens: HBM, each state read and written once.
#include <algorithm>

#include "pa_internal.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeadBatch = 4;  // query heads summed at once

template <int D, int COLS>
struct StepGeom {
    static constexpr int kLanes = COLS / 4;                 // lanes of a row, four columns each
    static constexpr int kSub = 32 / kLanes;                // rows side by side in a warp
    static constexpr int kRows = D / (kWarps * kSub);       // rows of a thread
    static_assert(kRows >= 1, "rows");
};

}  // namespace

template <int D, int COLS>
__device__ __forceinline__ void step_job(const LinearParams &p) {
    using G = StepGeom<D, COLS>;
    constexpr int R = G::kRows, kSlices = D / COLS;
    __shared__ float s_q[kHeadBatch][D], s_k[D], s_v[COLS];
    __shared__ float s_part[kWarps][kHeadBatch][COLS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slice = blockIdx.x % kSlices, job = blockIdx.x / kSlices;
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
    float4 s[R];
    const float *src = p.state + in * state_size + place;
#pragma unroll
    for (int i = 0; i < R; ++i)
        s[i] = in >= 0 ? *reinterpret_cast<const float4 *>(src + i * D)
                       : make_float4(0.f, 0.f, 0.f, 0.f);

    for (int t = t0; t < t0 + n; ++t) {
        const __nv_bfloat16 *kt = p.k + t * p.k_stride + h * D;
        const __nv_bfloat16 *vt = p.v + t * p.v_stride + h * D + slice * COLS;
        for (int i = tid; i < D; i += kThreads) s_k[i] = __bfloat162float(kt[i]);
        for (int i = tid; i < COLS; i += kThreads) s_v[i] = __bfloat162float(vt[i]);
        // a positive or NaN logarithm counts as 0, so that no state grows by its decay
        const float g = __ldg(p.decay + static_cast<int64_t>(t) * p.decay_stride + h);
        const float keep = expf(g < 0.f ? g : 0.f);
        for (int g0 = 0; g0 < p.group; g0 += kHeadBatch) {
            const int heads = min(kHeadBatch, p.group - g0);
            const __nv_bfloat16 *qt = p.q + t * p.q_stride + (h * p.group + g0) * D;
            for (int i = tid; i < heads * D; i += kThreads)
                s_q[i / D][i % D] = __bfloat162float(qt[i]);
            __syncthreads();
            if (g0 == 0) {
                const float4 v = *reinterpret_cast<const float4 *>(s_v + col);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float k = s_k[row0 + i];
                    s[i].x = fmaf(keep, s[i].x, k * v.x);
                    s[i].y = fmaf(keep, s[i].y, k * v.y);
                    s[i].z = fmaf(keep, s[i].z, k * v.z);
                    s[i].w = fmaf(keep, s[i].w, k * v.w);
                }
            }
            for (int j = 0; j < heads; ++j) {
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float q = s_q[j][row0 + i];
                    o.x = fmaf(q, s[i].x, o.x);
                    o.y = fmaf(q, s[i].y, o.y);
                    o.z = fmaf(q, s[i].z, o.z);
                    o.w = fmaf(q, s[i].w, o.w);
                }
#pragma unroll
                for (int x = G::kLanes; x < 32; x <<= 1) {
                    o.x += __shfl_xor_sync(0xffffffffu, o.x, x);
                    o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
                    o.z += __shfl_xor_sync(0xffffffffu, o.z, x);
                    o.w += __shfl_xor_sync(0xffffffffu, o.w, x);
                }
                if (lane < G::kLanes) *reinterpret_cast<float4 *>(&s_part[warp][j][col]) = o;
            }
            __syncthreads();
            for (int i = tid; i < heads * COLS; i += kThreads) {
                const int j = i / COLS, c = i % COLS;
                float o = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) o += s_part[w][j][c];
                p.out[(static_cast<int64_t>(t) * p.num_q_heads + h * p.group + g0 + j) * D +
                      slice * COLS + c] = __float2bfloat16(o * p.scale);
            }
        }
    }
    if (to < 0) return;
    float *dst = p.state + to * state_size + place;
#pragma unroll
    for (int i = 0; i < R; ++i) *reinterpret_cast<float4 *>(dst + i * D) = s[i];
}

template <int D, int COLS>
__global__ void __launch_bounds__(kThreads) linear_step_kernel(const LinearParams p) {
    // Beside the prompt kernel, which has waited for whatever wrote the inputs, there is nothing
    // to wait for: its rows and slots are others.  This grid then ends after that one, so that
    // what follows comes after both.
    if (!p.overlap) pdl_wait();
    pdl_trigger();
    step_job<D, COLS>(p);
    if (p.overlap) pdl_wait();
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
