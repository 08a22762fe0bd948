// pa_window.cu -- a windowed step in one kernel: no plan, no work lists, no second
// grid.
//
// The host bounds the step's pieces (of at most 16 rows of a request) and launches a
// cluster of 1 to 8 CTAs for each (piece, kv head), or, where there are many and they
// are short, a warp.  Each CTA finds its piece by a scan over the requests; the cluster's warps take the piece's visible 16-key chunks
// in turn, each through a TMA ring of its own that it refills the moment it has
// consumed a slot (no producer, no block barrier in the loop); at the end every
// warp leaves its rows' maximum, sum and unnormalised output in shared memory,
// and the cluster's CTAs fold them from there, a slice of the rows' columns each:
//   M = max m_w,  out = sum 2^(m_w - M) o_w / sum 2^(m_w - M) l_w.
//
// Bound: with few jobs by the chain launch, metadata, block ids, first chunk, fold:
// 5.6 us for one token at window 128, where plan, split-KV grid and their hand-over
// take 11.5; 24 verify requests 7.8 (20.6).  With many jobs by HBM: 64 decode requests
// (8 kv heads, d = 128, window 1024 + 4 sinks, 268 MB) 49.7 us, of which the stream
// takes 40 at the copy bandwidth and the part-filled second round of CTAs most of the
// rest; 56 requests, which run as one round, 41 us.  The split-KV kernel (pa_short.cu),
// whose CTAs are fed stage by stage by a producer warp, takes 67.6 us for the 64.
// A persistent kernel of such warps fed by the plan's list took 60.4 us: the plan
// (7 us) and the way from it to the first chunk (4 us) cost more than the rounds.
#include "pa_short.cuh"

namespace pa {

namespace {

// A piece of a request, for one kv head.  Keys, positions and chunks are packed
// (see KeySpan).
struct Work {
    int b, h, q_count, sink_chunks, gap;
    int key_end, chunks;
    int tok0, ctx;
};

template <int D, bool FP8, int PER_SM>
struct DirectGeom {
    static constexpr int kHalves = FP8 ? 1 : D / 64;
    static constexpr int kBoxBytes = kChunkKeys * 128;
    static constexpr int kHalfBytes = kHalves * kBoxBytes;
    static constexpr int kSlotBytes = 2 * kHalfBytes;
    // a warp's ring: 24 KB with two CTAs per SM, 16 KB with three
    static constexpr int kSlots = (PER_SM == 2 ? 24576 : 16384) / kSlotBytes;
    static constexpr int kRingBytes = kSlots * kSlotBytes;
    static constexpr int kThreads = 32 * kDirectWarps;
    // after the rings: the barriers, maximum and sum of each warp's rows, the
    // piece (each warp's), the requests' scan
    static constexpr int kOffBar = kDirectWarps * kRingBytes;
    static constexpr int kOffRows = kOffBar + kDirectWarps * kSlots * 8;
    static constexpr int kOffWork = kOffRows + kDirectWarps * kDirectRows * 8;
    static constexpr int kOffScan = kOffWork + kDirectWarps * static_cast<int>(sizeof(Work));
    static constexpr int kSmemBytes = kOffScan + 4 * kDirectWarps;
    static_assert(kOffBar % 1024 == 0 && kOffRows % 8 == 0 && kOffWork % alignof(Work) == 0 &&
                      kOffScan % 4 == 0,
                  "alignment");
    static_assert(kDirectRows * D * 4 <= kRingBytes, "a warp's state takes its ring's place");
};

// Block-table entry of chunk c, loaded raw (0 past the item's chunks); an
// out-of-range table column is clamped and flagged.
__device__ __forceinline__ int chunk_block(const ShortParams &p, const Work &w, int c) {
    if (c >= w.chunks) return 0;
    int col = unpacked_key(c * kChunkKeys, w.sink_chunks, w.gap) / p.block_size;
    if (col >= p.bt_stride) {
        flag_status(p.status, PA_DEV_BAD_METADATA);
        col = p.bt_stride - 1;
    }
    return __ldg(p.block_tables + static_cast<int64_t>(w.b) * p.bt_stride + col);
}
// Cache row of that chunk's first key; an out-of-range block id is clamped and
// flagged.
__device__ __forceinline__ int chunk_row(const ShortParams &p, const Work &w, int c, int blk) {
    if (c >= w.chunks) return 0;
    if (blk < 0 || blk >= p.num_blocks) {
        flag_status(p.status, PA_DEV_BAD_BLOCK);
        blk = min(max(blk, 0), p.num_blocks - 1);
    }
    return (blk * p.num_kv_heads + w.h) * p.block_size +
           unpacked_key(c * kChunkKeys, w.sink_chunks, w.gap) % p.block_size;
}

// The item's query rows as MMA fragments, its masks and an empty state.
template <int D, bool FP8>
__device__ __forceinline__ void begin_item(Consumer<D> &cs, const ShortParams &p, const Work &w,
                                           int lane) {
    constexpr int NT = D / 8, KS = D / 16;
    const int g = lane >> 2, t = lane & 3;
    cs.h = w.h;
    cs.tok0 = w.tok0;
    cs.ctx = w.ctx;
    cs.key_end = w.key_end;
    cs.R = w.q_count * p.group;
    cs.sl2 = FP8 ? p.scale_log2 * __ldg(p.k_scale + w.h) : p.scale_log2;
    cs.sinks = p.win.sinks;
    cs.low_first = cs.ctx - p.win.window + 1;
    cs.low_last = cs.low_first + w.q_count - 1;
    // this lane's rows: g and g + 8
    const int i0 = g / p.group, i1 = (g + 8) / p.group;
    cs.limit0 = g < cs.R ? cs.ctx + i0 : -1;
    cs.limit1 = g + 8 < cs.R ? cs.ctx + i1 : -1;
    cs.low0 = cs.low_first + i0;
    cs.low1 = cs.low_first + i1;
    auto row = [&](int r) {
        return r < cs.R ? p.q + (static_cast<int64_t>(cs.tok0 + r / p.group) * p.num_q_heads +
                                 cs.h * p.group + r % p.group) * D
                        : nullptr;
    };
    const __nv_bfloat16 *q0 = row(g), *q1 = row(g + 8);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        if constexpr (FP8) {
            // dims 16 ks + 4 t .. + 3, as the e4m3 K fragments hold them
            const uint2 z = make_uint2(0u, 0u);
            const uint2 x0 = q0 ? __ldg(reinterpret_cast<const uint2 *>(q0) + ks * 4 + t) : z;
            const uint2 x1 = q1 ? __ldg(reinterpret_cast<const uint2 *>(q1) + ks * 4 + t) : z;
            cs.qa[ks][0] = bf16x2_to_f16x2(x0.x);
            cs.qa[ks][1] = bf16x2_to_f16x2(x1.x);
            cs.qa[ks][2] = bf16x2_to_f16x2(x0.y);
            cs.qa[ks][3] = bf16x2_to_f16x2(x1.y);
        } else {
            const uint32_t *w0 = reinterpret_cast<const uint32_t *>(q0);
            const uint32_t *w1 = reinterpret_cast<const uint32_t *>(q1);
            const int at = ks * 8 + t;  // 32-bit word of dims 16 ks + 2 t
            cs.qa[ks][0] = w0 ? __ldg(w0 + at) : 0u;
            cs.qa[ks][1] = w1 ? __ldg(w1 + at) : 0u;
            cs.qa[ks][2] = w0 ? __ldg(w0 + at + 4) : 0u;
            cs.qa[ks][3] = w1 ? __ldg(w1 + at + 4) : 0u;
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) cs.o[nt][e] = 0.f;
    cs.m0 = cs.m1 = -INFINITY;
    cs.l0 = cs.l1 = 0.f;
}

}  // namespace

// ALONE: a warp per job, else a cluster of CTAs.
template <int D, bool FP8, int PER_SM, bool ALONE>
__global__ void __launch_bounds__(DirectGeom<D, FP8, PER_SM>::kThreads, PER_SM)
    window_direct_kernel(const ShortParams p, const __grid_constant__ CUtensorMap tmk,
                        const __grid_constant__ CUtensorMap tmv, const DirectParams dp) {
    using G = DirectGeom<D, FP8, PER_SM>;
    constexpr int NS = G::kSlots;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t *ring = smem + warp * G::kRingBytes;
    float2 *rows = reinterpret_cast<float2 *>(smem + G::kOffRows);
    Work *works = reinterpret_cast<Work *>(smem + G::kOffWork);
    int *scan = reinterpret_cast<int *>(smem + G::kOffScan);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + G::kOffBar) + warp * NS;
    // the CTA's jobs: the cluster's, or one for each warp
    const int size = ALONE ? 1 : dp.cluster, rank = static_cast<int>(blockIdx.x) % size;
    const int first_job = static_cast<int>(blockIdx.x) / size * (ALONE ? kDirectWarps : 1);
    if (lane == 0) {
        for (int i = 0; i < NS; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
        if (warp == 0) {
            tma_prefetch_desc(&tmk);
            tma_prefetch_desc(&tmv);
        }
    }
    if (tid < kDirectWarps) works[tid] = Work{};
    pdl_wait();
    pdl_trigger();

    // thread t: requests t * each .., their pieces and the pieces before them
    const int each = (p.num_seqs + G::kThreads - 1) / G::kThreads;
    const int b_end = min(p.num_seqs, (tid + 1) * each);
    auto pieces_of = [&](int b, int &q0, int &n, int &ctx) {
        q0 = __ldg(p.qsl + b);
        ctx = __ldg(p.ctx + b);
        const int q1 = __ldg(p.qsl + b + 1), len = __ldg(p.seq_lens + b);
        n = q1 - q0;
        if (n < 0 || ctx < 0 || len > dp.max_keys || len != ctx + n || q0 < 0 ||
            q1 > p.num_q_tokens) {
            if (blockIdx.x == 0) flag_status(p.status, PA_DEV_BAD_METADATA);
            n = 0;
        }
        if (static_cast<int64_t>(n) * p.group > dp.max_rows) return 0;
        return (n + dp.piece_tokens - 1) / dp.piece_tokens;
    };
    int pieces = 0, q0 = 0, n = 0, ctx = 0;
    for (int b = tid * each; b < b_end; ++b) pieces += pieces_of(b, q0, n, ctx);
    int incl = pieces;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int before = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += before;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int total = 0, first = incl - pieces;
#pragma unroll
    for (int w = 0; w < kDirectWarps; ++w) {
        if (w < warp) first += scan[w];
        total += scan[w];
    }
    if (total > dp.max_pieces) {  // requests that overlap: none runs
        if (blockIdx.x == 0 && tid == 0) flag_status(p.status, PA_DEV_PLAN_OVERFLOW);
        return;
    }
    if (first_job / p.num_kv_heads >= total) return;  // (all of a cluster's CTAs)
    for (int k = 0; k < (ALONE ? kDirectWarps : 1); ++k) {
        const int piece = (first_job + k) / p.num_kv_heads;
        if (piece < first || piece >= first + pieces) continue;  // none, or another thread's
        int b = tid * each, at = first;
        if (each > 1)
            for (;; ++b) {
                const int of_b = pieces_of(b, q0, n, ctx);
                if (piece < at + of_b) break;
                at += of_b;
            }
        const int begin = (piece - at) * dp.piece_tokens;
        const int count = min(dp.piece_tokens, n - begin);
        const KeySpan ks = key_span(p.win, ctx + begin, ctx + begin + count);
        Work *work = works + k;
        work->b = b;
        work->q_count = count;
        work->sink_chunks = ks.sink_chunks;
        work->gap = ks.gap;
        work->h = (first_job + k) - piece * p.num_kv_heads;
        work->key_end = ks.keys;
        work->chunks = (ks.keys + kChunkKeys - 1) / kChunkKeys;
        work->tok0 = q0 + begin;
        work->ctx = ctx + begin - ks.gap * kChunkKeys;
    }
    __syncthreads();

    // this warp's chunks: worker, worker + workers, ...; lane l holds the TMA
    // row of the (base + l)-th, and the raw block id of the 32 after those
    const Work &w = works[ALONE ? warp : 0];
    const int workers = ALONE ? 1 : size * kDirectWarps;
    const int worker = ALONE ? 0 : rank * kDirectWarps + warp;
    const int mine = w.chunks > worker ? (w.chunks - worker + workers - 1) / workers : 0;
    auto nth = [&](int i) { return i < mine ? worker + i * workers : w.chunks; };
    int row_of = chunk_row(p, w, nth(lane), chunk_block(p, w, nth(lane)));
    int later = chunk_block(p, w, nth(32 + lane));
    const bool stall = p.test_stall && blockIdx.x == 0 && warp == 0;
    int issued = 0;
    auto issue = [&]() {
        if (issued == mine || (stall && issued > 0)) return;
        if (issued > 0 && issued % 32 == 0) {
            row_of = chunk_row(p, w, nth(issued + lane), later);
            later = chunk_block(p, w, nth(issued + 32 + lane));
        }
        const int row = __shfl_sync(0xffffffffu, row_of, issued % 32);
        const int slot = issued % NS;
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], G::kSlotBytes);
        __syncwarp();
        if (lane < 2 * G::kHalves)
            tma_load_2d(ring + slot * G::kSlotBytes + lane * G::kBoxBytes,
                        lane < G::kHalves ? &tmk : &tmv, lane % G::kHalves * 64, row, &full[slot]);
        ++issued;
    };
    for (int i = 0; i < NS; ++i) issue();

    Consumer<D> cs;
    begin_item<D, FP8>(cs, p, w, lane);
    int gave_up = 0, done = 0;
    for (; done < mine; ++done) {
        const int slot = done % NS;
        if (!warp_mbar_wait_spin(&full[slot], (done / NS) & 1, &gave_up)) break;
        const uint32_t kb = smem_u32(ring + slot * G::kSlotBytes), vb = kb + G::kHalfBytes;
        const int key0 = (worker + done * workers) * kChunkKeys, end = key0 + kChunkKeys;
        if (end <= cs.key_end && end - 1 <= cs.ctx && cs.all_in_window(key0))
            row_chunk<D, FP8, false, true>(cs, kb, vb, key0, lane);
        else
            row_chunk<D, FP8, true, true>(cs, kb, vb, key0, lane);
        __syncwarp();  // every lane has read the slot that is refilled now
        issue();
    }
    if (done < mine) {
        if (lane == 0) {
            flag_status(p.status, PA_DEV_WAIT_TIMEOUT);
            for (int k = done; k < issued; ++k) mbar_drain(&full[k % NS], (k / NS) & 1);
        }
        __syncwarp();
    }

    // the warp's rows: maxima and sums, and unnormalised outputs in its ring
    const int g = lane >> 2, t = lane & 3;
    const float l0 = quad_sum(cs.l0), l1 = quad_sum(cs.l1);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int r = g + 8 * half;
        if (r >= cs.R) continue;
        if (t == 0)
            rows[warp * kDirectRows + r] = half ? make_float2(cs.m1, l1) : make_float2(cs.m0, l0);
        float *o = reinterpret_cast<float *>(ring) + r * D;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            if constexpr (FP8) {
                // the even and the odd tile of 16 dims hold pairs' halves
                const int cc = i >> 1, e = i & 1;
                *reinterpret_cast<float2 *>(o + cc * 16 + 4 * t + 2 * e) =
                    make_float2(cs.o[2 * cc][2 * half + e], cs.o[2 * cc + 1][2 * half + e]);
            } else {
                *reinterpret_cast<float2 *>(o + i * 8 + 2 * t) =
                    make_float2(cs.o[i][2 * half], cs.o[i][2 * half + 1]);
            }
        }
    }
    if (ALONE)
        __syncwarp();
    else
        cluster_sync();
    // Fold: four columns of a row per thread, the CTAs of the cluster in turn (a warp
    // alone: its own state)
    const float vsc = FP8 ? __ldg(p.v_scale + w.h) : 1.f;
    const int stride = ALONE ? 32 : size * G::kThreads;
    for (int i = ALONE ? lane : rank * G::kThreads + tid; i < cs.R * (D / 4); i += stride) {
        const int r = i / (D / 4), e4 = i - r * (D / 4);
        float M = -INFINITY, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < size; ++c) {
            float2 ml[kDirectWarps];
            float4 v[kDirectWarps];
            float most = M;
#pragma unroll
            for (int k = 0; k < kDirectWarps; ++k) {
                const bool with = !ALONE || k == warp;
                ml[k] = with ? ld_cluster_f2(&rows[k * kDirectRows + r], c)
                             : make_float2(-INFINITY, 0.f);
                v[k] = with ? ld_cluster_f4(smem + k * G::kRingBytes + (r * D + 4 * e4) * 4, c)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
                most = fmaxf(most, ml[k].x);
            }
            if (most == -INFINITY) continue;
            const float a = fast_exp2(M - most);
            M = most;
            sum *= a;
            acc.x *= a;
            acc.y *= a;
            acc.z *= a;
            acc.w *= a;
#pragma unroll
            for (int k = 0; k < kDirectWarps; ++k) {
                const float e = fast_exp2(ml[k].x - M);
                sum += e * ml[k].y;
                acc.x += e * v[k].x;
                acc.y += e * v[k].y;
                acc.z += e * v[k].z;
                acc.w += e * v[k].w;
            }
        }
        const float inv = sum > 0.f ? vsc / sum : 0.f;
        const int64_t row = static_cast<int64_t>(w.tok0 + r / p.group) * p.num_q_heads +
                            w.h * p.group + r % p.group;
        uint2 out;
        out.x = pack_bf16x2(acc.x * inv, acc.y * inv);
        out.y = pack_bf16x2(acc.z * inv, acc.w * inv);
        reinterpret_cast<uint2 *>(p.out + row * D)[e4] = out;
        if (e4 == 0 && p.lse) p.lse[row] = sum > 0.f ? (M + __log2f(sum)) * kLn2 : -INFINITY;
    }
    if (!ALONE) cluster_sync();  // the others have read this CTA's states
}

namespace {

template <int D, bool FP8, int PER_SM, bool ALONE>
int launch_direct(const ShortParams &p, const CUtensorMap &tk, const CUtensorMap &tv,
                 const DirectParams &dp, cudaStream_t s) {
    using G = DirectGeom<D, FP8, PER_SM>;
    static PerDeviceOnce once;
    if (once_per_device(once, [] {
            return cudaFuncSetAttribute(window_direct_kernel<D, FP8, PER_SM, ALONE>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        G::kSmemBytes);
        }) != PA_OK)
        return PA_ERR_CUDA;
    const int jobs = dp.max_pieces * p.num_kv_heads;
    const int grid = ALONE ? (jobs + kDirectWarps - 1) / kDirectWarps : jobs * dp.cluster;
    PdlLaunch l(grid, G::kThreads, G::kSmemBytes, s);
    if (dp.cluster > 1) l.set_cluster(dp.cluster);
    return launch_kernel(l, window_direct_kernel<D, FP8, PER_SM, ALONE>, p, tk, tv, dp) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

template <int D, bool FP8>
int launch_direct(const ShortParams &p, const CUtensorMap &tk, const CUtensorMap &tv,
                  const DirectParams &dp, cudaStream_t s) {
    if (dp.cluster == 0)
        return dp.per_sm == 2 ? launch_direct<D, FP8, 2, true>(p, tk, tv, dp, s)
                              : launch_direct<D, FP8, 3, true>(p, tk, tv, dp, s);
    return dp.per_sm == 2 ? launch_direct<D, FP8, 2, false>(p, tk, tv, dp, s)
                          : launch_direct<D, FP8, 3, false>(p, tk, tv, dp, s);
}

}  // namespace

int launch_window_direct(const ShortParams &p, const CUtensorMap &tk, const CUtensorMap &tv,
                        const DirectParams &dp, int head_dim, bool fp8, cudaStream_t s) {
    if (fp8) return launch_direct<128, true>(p, tk, tv, dp, s);
    return head_dim == 128 ? launch_direct<128, false>(p, tk, tv, dp, s)
                           : launch_direct<64, false>(p, tk, tv, dp, s);
}

}  // namespace pa
