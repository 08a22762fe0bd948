// pa_window.cu -- windowed attention for large bf16 decode batches: query rows in
// pieces of at most 16 and enough jobs (a piece, for one kv head) to give every
// warp of the GPU work of its own.
//
// The split-KV kernel (pa_short.cu) spreads a job's chunks over the four warps
// of a CTA, fed by a producer warp; a chunk's slot is free again when the
// slowest warp has let go of its stage and the producer has noticed, so a CTA
// moves a 32 KB stage in ~1.4 us however fast memory is, and windows make the
// jobs equally long, 1.7 rounds of them for 304 CTAs.  Here a warp is a worker:
//  * it takes a work item (a range of packed chunks of a job) from the plan's
//    list, longest first, and streams its 16-key chunks through a ring of its
//    own: lane l holds the TMA row of chunk l of the current 32, the first lanes
//    issue a chunk's boxes, and the warp itself refills a slot the moment it has
//    consumed it;
//  * the ring runs on into the next item, whose record, block ids and
//    positions were fetched one dependent step per chunk beforehand;
//  * nothing is shared between warps, so there are no block barriers, an item
//    ends without a merge, and a split item's partial state is folded by the
//    last of its workers while the others stream on.
// Twelve warps with two 8 KB slots each (four of 4 KB for head_dim 64) fill an
// SM's shared memory at 168 registers a thread.  64 decode requests, window
// 1024 + 4 sinks, 8 kv heads, d = 128: 64-65 us with 12 x 2, 10 x 2, 9 x 3 or
// 8 x 3 alike (before the two steps below), and 12 x 2 is ahead where the SMs
// are shared with prompt chunks (213.5 us; 9 x 3 227, 8 x 3 222).
// Bound: HBM.  Of 60.4 us (268 MB, 40.4 us at the copy bandwidth) the stream
// itself takes 40; the plan takes 7 before it (less 2.7 us of stream, see
// warm_l2), the way from the plan to the first chunk 4, the fold and the next
// kernel's start the rest.
#include "pa_short.cuh"

namespace pa {

namespace {

// A work item, in its warp's shared memory.  Keys, positions and chunks are
// packed (see KeySpan).
struct Work {
    ShortItem it;
    int h, key_end, c0, c1;  // its chunks are [c0, c1)
    int tok0, ctx;
};
constexpr int kWarmBytes = 32 << 20;
constexpr int kItemWords = sizeof(ShortItem) / 4;

template <int D>
struct RowsGeom {
    static constexpr int kHalves = D / 64;             // boxes of a chunk of K (or V)
    static constexpr int kBoxBytes = kChunkKeys * 128;
    static constexpr int kHalfBytes = kHalves * kBoxBytes;  // a chunk of K (or V)
    static constexpr int kSlotBytes = 2 * kHalfBytes;       // 8 KB, or 4 KB (head_dim 64)
    static constexpr int kWarps = 12;
    static constexpr int kSlots = 16384 / kSlotBytes;
    static constexpr int kThreads = 32 * kWarps;
    // a warp's ring and its two items; after all warps', their barriers
    static constexpr int kWarpBytes = kSlots * kSlotBytes + 2 * static_cast<int>(sizeof(Work));
    static constexpr int kSmemBytes = kWarps * (kWarpBytes + 8 * kSlots);
    static_assert(sizeof(Work) % 16 == 0 && alignof(Work) <= 16, "items behind the rings");
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

// The record's words, one per lane, become an item.
__device__ __forceinline__ void put_record(const ShortParams &p, Work &w, uint32_t word, int lane) {
    if (lane < kItemWords) reinterpret_cast<uint32_t *>(&w.it)[lane] = word;
    __syncwarp();
    if (lane == 0) {
        w.h = w.it.counter % p.num_kv_heads;
        w.key_end = min(w.it.stage_end * kStageKeys, w.it.seq_len);
        w.c0 = w.it.stage_begin * kStageChunks;
        w.c1 = (w.key_end + kChunkKeys - 1) / kChunkKeys;
    }
    __syncwarp();
}
__device__ __forceinline__ uint32_t record_word(const ShortParams &p, int idx, int lane) {
    return lane < kItemWords
               ? *(reinterpret_cast<const volatile uint32_t *>(p.items + idx) + lane)
               : 0u;
}

// Block-table entry of chunk c, loaded raw (0 past the item's chunks); an
// out-of-range table column is clamped and flagged.
__device__ __forceinline__ int chunk_block(const ShortParams &p, const Work &w, int c) {
    if (c >= w.c1) return 0;
    int col = unpacked_key(c * kChunkKeys, w.it.sink_chunks, w.it.gap) / p.block_size;
    if (col >= p.bt_stride) {
        flag_status(p.status, PA_DEV_BAD_METADATA);
        col = p.bt_stride - 1;
    }
    return __ldg(p.block_tables + static_cast<int64_t>(w.it.b) * p.bt_stride + col);
}
// Cache row of that chunk's first key; an out-of-range block id is clamped and
// flagged.
__device__ __forceinline__ int chunk_row(const ShortParams &p, const Work &w, int c, int blk) {
    if (c >= w.c1) return 0;
    if (blk < 0 || blk >= p.num_blocks) {
        flag_status(p.status, PA_DEV_BAD_BLOCK);
        blk = min(max(blk, 0), p.num_blocks - 1);
    }
    return (blk * p.num_kv_heads + w.h) * p.block_size +
           unpacked_key(c * kChunkKeys, w.it.sink_chunks, w.it.gap) % p.block_size;
}

// While the plan is made: L2 prefetch of the first visible chunks of every
// (request, kv head) pair, as many as kWarmBytes allow, by the worker that the
// pair's number names.  (The planner waited for everything before it in the
// stream and then let this grid start, so metadata and pool are final.)
// Metadata and table entries that the plan will refuse or flag are passed over.
// 61.0 us with 24 or 48 MB, 63.8 without (64 decode requests, window 1024).
template <int D>
__device__ void warm_l2(const ShortParams &p, int worker, int workers, int lane) {
    constexpr int kBytes = RowsGeom<D>::kHalfBytes;  // a chunk of K: consecutive
    const int pairs = p.num_seqs * p.num_kv_heads;
    const int limit = min(32, kWarmBytes / (2 * kBytes) / pairs);
    for (int i = worker; i < pairs; i += workers) {
        const int b = i / p.num_kv_heads, h = i - b * p.num_kv_heads;
        const int n = __ldg(p.qsl + b + 1) - __ldg(p.qsl + b), ctx = __ldg(p.ctx + b);
        if (n <= 0 || n > kShortMaxRows / p.group || ctx < 0 || ctx + n != __ldg(p.seq_lens + b))
            continue;
        const KeySpan ks = key_span(p.win, ctx, ctx + n);
        int row = -1;  // lane l: chunk l's first cache row
        if (lane < limit && lane * kChunkKeys < ks.keys) {
            const int key = unpacked_key(lane * kChunkKeys, ks.sink_chunks, ks.gap);
            const int col = key / p.block_size;
            if (col < p.bt_stride) {
                const int blk = __ldg(p.block_tables + static_cast<int64_t>(b) * p.bt_stride + col);
                if (blk >= 0 && blk < p.num_blocks)
                    row = (blk * p.num_kv_heads + h) * p.block_size + key % p.block_size;
            }
        }
        for (int c = 0; c < limit; ++c) {
            const int r = __shfl_sync(0xffffffffu, row, c);
            if (r < 0) continue;
            const int64_t at = static_cast<int64_t>(r) * (kBytes / kChunkKeys);
            for (int e = lane * 128; e < kBytes; e += 32 * 128) {
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.k_pool + at + e));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.v_pool + at + e));
            }
        }
    }
}

// The item's query rows as MMA fragments, its masks and an empty state.
template <int D>
__device__ __forceinline__ void begin_item(Consumer<D> &cs, const ShortParams &p, const Work &w,
                                           int lane) {
    constexpr int NT = D / 8, KS = D / 16;
    const int g = lane >> 2, t = lane & 3;
    cs.h = w.h;
    cs.tok0 = w.tok0;
    cs.ctx = w.ctx;
    cs.key_end = w.key_end;
    cs.R = w.it.q_count * p.group;
    cs.sl2 = p.scale_log2;
    cs.sinks = p.win.sinks;
    cs.low_first = cs.ctx - p.win.window + 1;
    cs.low_last = cs.low_first + w.it.q_count - 1;
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
    const uint32_t *q0 = reinterpret_cast<const uint32_t *>(row(g));
    const uint32_t *q1 = reinterpret_cast<const uint32_t *>(row(g + 8));
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        const int at = ks * 8 + t;  // 32-bit word of dims 16 ks + 2 t
        cs.qa[ks][0] = q0 ? __ldg(q0 + at) : 0u;
        cs.qa[ks][1] = q1 ? __ldg(q1 + at) : 0u;
        cs.qa[ks][2] = q0 ? __ldg(q0 + at + 4) : 0u;
        cs.qa[ks][3] = q1 ? __ldg(q1 + at + 4) : 0u;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) cs.o[nt][e] = 0.f;
    cs.m0 = cs.m1 = -INFINITY;
    cs.l0 = cs.l1 = 0.f;
}

// The item's rows: output, or partial state of a split, and the fold by the
// last split's worker.
template <int D>
__device__ __forceinline__ void end_item(Consumer<D> &cs, const ShortParams &p, const Work &w,
                                         int lane) {
    const int g = lane >> 2, t = lane & 3;
    const float l0 = quad_sum(cs.l0), l1 = quad_sum(cs.l1);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int r = g + 8 * half;
        if (r >= cs.R) continue;
        const float l = half ? l1 : l0, m = half ? cs.m1 : cs.m0;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const float lse_v = l > 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
        const int64_t row = static_cast<int64_t>(cs.tok0 + r / p.group) * p.num_q_heads +
                            cs.h * p.group + r % p.group;
        const bool whole = w.it.nsplit == 1;
        uint32_t *out = reinterpret_cast<uint32_t *>(p.out + row * D);
        float *part = p.partial_o + static_cast<int64_t>(w.it.partial_base + r) * D;
#pragma unroll
        for (int nt = 0; nt < D / 8; ++nt) {
            const float x = cs.o[nt][2 * half] * inv, y = cs.o[nt][2 * half + 1] * inv;
            if (whole)
                out[nt * 4 + t] = pack_bf16x2(x, y);
            else
                __stcg(reinterpret_cast<float2 *>(part + nt * 8 + 2 * t), make_float2(x, y));
        }
        if (t == 0) {
            if (!whole)
                __stcg(p.partial_lse + w.it.partial_base + r, lse_v);
            else if (p.lse)
                p.lse[row] = lse_v;
        }
    }
    if (w.it.nsplit == 1) return;
    // one lane's acquire-release counter update publishes the warp's partial
    // state (ordered before it by the warp barrier) and, if it is the last,
    // makes the others' visible
    __syncwarp();
    int last = 0;
    if (lane == 0) last = atomic_add_acq_rel_gpu(p.counters + w.it.counter, 1) == w.it.nsplit - 1;
    if (!__shfl_sync(0xffffffffu, last, 0)) return;
    const int base = w.it.partial_base - w.it.split * cs.R;
    for (int i = lane; i < cs.R * (D / 4); i += 32) {
        const int r = i / (D / 4), e4 = i - r * (D / 4);
        const int64_t row = static_cast<int64_t>(cs.tok0 + r / p.group) * p.num_q_heads +
                            cs.h * p.group + r % p.group;
        const float *pl = p.partial_lse + base + r;
        const float4 *po = reinterpret_cast<const float4 *>(
                               p.partial_o + static_cast<int64_t>(base + r) * D) + e4;
        const int64_t stride = static_cast<int64_t>(cs.R) * (D / 4);
        // running maximum and sum over the splits, kFoldBatch at a time
        float M = -INFINITY, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s0 = 0; s0 < w.it.nsplit; s0 += kFoldBatch) {
            float lv[kFoldBatch];
            float4 v[kFoldBatch];
            float most = M;
#pragma unroll
            for (int j = 0; j < kFoldBatch; ++j) {
                const bool in = s0 + j < w.it.nsplit;
                lv[j] = in ? __ldcg(pl + (s0 + j) * cs.R) : -INFINITY;
                v[j] = in ? __ldcg(po + (s0 + j) * stride) : make_float4(0.f, 0.f, 0.f, 0.f);
                most = fmaxf(most, lv[j]);
            }
            if (most == -INFINITY) continue;
            const float a = __expf(M - most);
            M = most;
            sum *= a;
            acc.x *= a;
            acc.y *= a;
            acc.z *= a;
            acc.w *= a;
#pragma unroll
            for (int j = 0; j < kFoldBatch; ++j) {
                const float e = __expf(lv[j] - M);
                sum += e;
                acc.x += e * v[j].x;
                acc.y += e * v[j].y;
                acc.z += e * v[j].z;
                acc.w += e * v[j].w;
            }
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        uint2 o;
        o.x = pack_bf16x2(acc.x * inv, acc.y * inv);
        o.y = pack_bf16x2(acc.z * inv, acc.w * inv);
        reinterpret_cast<uint2 *>(p.out + row * D)[e4] = o;
        if (e4 == 0 && p.lse) p.lse[row] = sum > 0.f ? M + __logf(sum) : -INFINITY;
    }
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(RowsGeom<D>::kThreads, 1)
    window_rows_kernel(const ShortParams p, const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv) {
    using G = RowsGeom<D>;
    constexpr int NS = G::kSlots;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *ring = smem + warp * NS * G::kSlotBytes;
    Work *works = reinterpret_cast<Work *>(smem + G::kWarps * NS * G::kSlotBytes) + 2 * warp;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + G::kWarps * G::kWarpBytes) + warp * NS;
    if (lane == 0) {
        for (int i = 0; i < NS; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
        if (warp == 0) {
            tma_prefetch_desc(&tmk);
            tma_prefetch_desc(&tmv);
        }
    }
    __syncwarp();
    // Before the plan is ready: prefetches, and a pass over an item without rows,
    // which brings the kernel's instructions into the caches (65.1 -> 63.8 us for
    // 64 decode requests; dry is opaque, so that the pass is not compiled as a
    // copy of its own).  After the step's first tensor-core grid, which waited for the plan,
    // there is nothing to wait for.
    int dry;
    asm volatile("mov.u32 %0, 1;" : "=r"(dry));
    if (!p.no_start_wait)
        warm_l2<D>(p, warp * static_cast<int>(gridDim.x) + blockIdx.x,
                        static_cast<int>(gridDim.x) * G::kWarps, lane);
    Work *cur = works, *nxt = works + 1;
    if (lane == 0) {
        *cur = Work{};
        cur->it.nsplit = 1;
        // a chunk without masks (window permitting) and one with
        cur->c1 = p.no_start_wait ? 0 : 2;
        cur->ctx = kChunkKeys - 1;
        cur->key_end = 2 * kChunkKeys - 1;
    }
    __syncwarp();

    // When the grid starts at once, worker w starts with item w (one warp of
    // every SM before the next warp); beside a tensor-core grid CTAs start as
    // SMs free up and every item comes from the counter.
    const int first_static = p.no_start_wait ? 0 : static_cast<int>(gridDim.x) * G::kWarps;
    // test hook: the first worker waits for chunks that it never asks for
    const bool stall = p.test_stall && blockIdx.x == 0 && warp == 0;
    int num_items = 0;
    // The issue side: next chunk `ic` of the item being issued (*cur, or *nxt
    // once on_next), TMA rows of its chunks ibase + lane, raw block ids of the
    // 32 chunks after those.
    bool on_next = false;
    int ic = 0, ic_end = 0, ibase = 0, irow = 0, iblk = 0;
    uint32_t issued = 0, consumed = 0;
    // the next item: 0 not asked for, 1 claimed, 2 its record is on its way, 3 its
    // positions and block ids are, 4 ready, 5 there is none
    int stage = p.no_start_wait ? 0 : 1, nxt_blk = 0;
    int word = warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    auto advance_next = [&]() {
        if (stage == 0) {
            if (lane == 0) word = atomicAdd(&p.hdr->short_next, 1) + first_static;
            stage = 1;
        } else if (stage == 1) {
            const int at = __shfl_sync(0xffffffffu, word, 0);
            stage = at < num_items ? 2 : 5;
            if (stage == 2) word = static_cast<int>(record_word(p, at, lane));
        } else if (stage == 2) {
            put_record(p, *nxt, static_cast<uint32_t>(word), lane);
            nxt_blk = chunk_block(p, *nxt, nxt->c0 + lane);
            if (lane < 2) word = __ldg((lane ? p.ctx : p.qsl) + nxt->it.b);
            stage = 3;
        } else if (stage == 3) {
            if (lane == 0) nxt->tok0 = word + nxt->it.q_begin;
            if (lane == 1) nxt->ctx = word + nxt->it.q_begin - nxt->it.gap * kChunkKeys;
            __syncwarp();
            prefetch_item_q<D>(p, nxt->tok0, nxt->h, nxt->it.q_count, lane);
            stage = 4;
        }
    };
    auto issue = [&]() {
        if (stall && issued > 0) return;
        if (ic == ic_end) {
            if (on_next || stage != 4) return;
            on_next = true;
            ic = ibase = nxt->c0;
            ic_end = nxt->c1;
            irow = chunk_row(p, *nxt, ic + lane, nxt_blk);
            iblk = chunk_block(p, *nxt, ibase + 32 + lane);
            if (ic == ic_end) return;
        } else if (ic == ibase + 32) {
            const Work &w = on_next ? *nxt : *cur;
            ibase = ic;
            irow = chunk_row(p, w, ic + lane, iblk);
            iblk = chunk_block(p, w, ibase + 32 + lane);
        }
        const int row = __shfl_sync(0xffffffffu, irow, ic - ibase);
        const int slot = issued % NS;
        uint8_t *dst = ring + slot * G::kSlotBytes;
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], G::kSlotBytes);
        __syncwarp();
        if (lane < 2 * G::kHalves) {
            const int hf = lane % G::kHalves;
            tma_load_2d(dst + lane * G::kBoxBytes, lane < G::kHalves ? &tmk : &tmv, hf * 64, row,
                        &full[slot]);
        }
        ++ic;
        ++issued;
    };
    volatile int gave_up = 0;
    Consumer<D> cs;
    while (true) {
        begin_item<D>(cs, p, *cur, lane);
        int c = cur->c0;
        const int c1 = cur->c1;
        bool ok = true;
        while (c < c1) {
            const int slot = consumed % NS;
            ok = dry || warp_mbar_wait_spin(&full[slot], (consumed / NS) & 1, &gave_up);
            if (!ok) break;
            const uint32_t kb = smem_u32(ring + slot * G::kSlotBytes), vb = kb + G::kHalfBytes;
            const int key0 = c * kChunkKeys, end = key0 + kChunkKeys;
            // no key needs a mask or a zeroed V row?
            if (end <= cs.key_end && end - 1 <= cs.ctx && cs.all_in_window(key0))
                row_chunk<D, false, false, true>(cs, kb, vb, key0, lane);
            else
                row_chunk<D, false, true, true>(cs, kb, vb, key0, lane);
            __syncwarp();  // every lane has read the slot that is refilled now
            ++c;
            if (dry) continue;
            ++consumed;
            // ask for the next item a few chunks before this one is all issued
            if (!on_next && (stage > 0 ? stage < 4 : ic_end - ic <= 6)) advance_next();
            issue();
        }
        if (!ok) break;
        end_item<D>(cs, p, *cur, lane);
        if (dry) {
            if (!p.no_start_wait) pdl_wait();
            pdl_trigger();
            num_items = *reinterpret_cast<volatile int *>(&p.hdr->num_short_items);
            dry = 0;
        }
        while (stage < 4) advance_next();
        if (stage == 5) break;
        if (!on_next) issue();  // (switches to nxt)
        __syncwarp();  // *cur is read no more
        Work *const done = cur;
        cur = nxt;
        nxt = done;
        on_next = false;
        stage = 0;
        for (int i = issued - consumed; i < NS && ic < ic_end; ++i) issue();
    }
    if (gave_up) {
        if (lane == 0) {
            flag_status(p.status, PA_DEV_WAIT_TIMEOUT);
            // let copies already in flight land before the CTA exits
            for (uint32_t k = consumed; k < issued; ++k)
                mbar_drain(&full[k % NS], (k / NS) & 1);
        }
        __syncwarp();
    }
}

namespace {

template <int D>
int launch(const ShortParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int grid,
           cudaStream_t s) {
    using G = RowsGeom<D>;
    static PerDeviceOnce once;
    if (once_per_device(once, [] {
            return cudaFuncSetAttribute(window_rows_kernel<D>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        G::kSmemBytes);
        }) != PA_OK)
        return PA_ERR_CUDA;
    PdlLaunch l(grid, G::kThreads, G::kSmemBytes, s);
    return launch_kernel(l, window_rows_kernel<D>, p, tk, tv) == cudaSuccess ? PA_OK
                                                                                  : PA_ERR_CUDA;
}

}  // namespace

int window_rows_workers_per_sm(int head_dim) {
    return head_dim == 128 ? RowsGeom<128>::kWarps : RowsGeom<64>::kWarps;
}

int launch_window_rows(const ShortParams &p, const CUtensorMap &tk, const CUtensorMap &tv,
                       int head_dim, int grid, cudaStream_t s) {
    return head_dim == 128 ? launch<128>(p, tk, tv, grid, s) : launch<64>(p, tk, tv, grid, s);
}

}  // namespace pa
