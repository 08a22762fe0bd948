// pa_long.cuh -- what the two tensor-core attention kernels share: work items
// and their schedule, the block-table gathering producer, and packed fp32
// arithmetic.  pa_long.cu holds the plain kernel (causal steps and the cascade
// prefix pass), pa_long_window.cu the windowed one.
#pragma once

#include "pa_internal.cuh"

namespace pa {

namespace {

constexpr int kKStages = 2;  // K is released as soon as Q K^T has read it
constexpr int kVStages = 3;  // V is held until its P V
constexpr int kLongWarps = 12;

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRescaleThreshold = 8.0f;

// Shared-memory sizes of the operands' tiles.
template <int D>
struct LongTiles {
    static constexpr int kHalves = D / 64;
    static constexpr int kHalfBytes = 128 * 128;            // 128 rows x 128 B
    static constexpr int kQBytes = kHalves * kHalfBytes;    // Q tile
    static constexpr int kKVBytes = kHalves * kHalfBytes;   // one K (or V) tile of 128 keys
};

// The lowest n bits set, n clamped to 0 .. 64.
__device__ __forceinline__ uint64_t low_bits(int n) {
    return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;
}

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return warp_mbar_wait(bar, parity, abort);
}

// Packed pairs of fp32 (one 64-bit register pair) for the two-wide FMA / add
// of this architecture, and the three-input maximum: the softmax warps are
// bound by instruction issue, so each score costs half an FMA, half an add,
// half a conversion, half a maximum and one exponential.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Everything one role needs to know about a work item.
struct Item {
    int b, h, tok0, nvalid, pos0, key_begin, key_end, causal, nsplit, split;
    int pair, partial_base, nt;
    int sink_chunks, gap;      // windowed step
    int block_sinks, block_gap;  // windowed step on staged blocks (BlockSpan)
};

template <bool WIN>
__device__ __forceinline__ Item decode_item(const LongParams &p, int idx) {
    Item it{};
    const int TQ = p.q_tile_tokens;
    if (!p.prefix_mode) {
        const int rec = idx / p.num_kv_heads;
        const LongItem li = load_record(p.items, rec);
        it.b = li.b;
        it.h = idx - rec * p.num_kv_heads;
        const int q0 = __ldg(p.qsl + li.b);
        const int n = __ldg(p.qsl + li.b + 1) - q0;
        it.tok0 = q0 + li.q_tile * TQ;
        it.nvalid = min(TQ, n - li.q_tile * TQ);
        it.pos0 = __ldg(p.ctx + li.b) + li.q_tile * TQ;
        it.key_begin = li.key_begin;
        it.key_end = li.key_end;
        it.causal = 1;
        it.nsplit = 1;
        if constexpr (WIN) {
            // positions in packed keys from here on
            if (p.stage_base) {
                const int ctx = it.pos0 - li.q_tile * TQ;
                const BlockSpan bsp = block_span(p.win, ctx, ctx + n, p.block_size);
                it.block_sinks = bsp.sink_blocks;
                it.block_gap = bsp.gap;
            }
            it.sink_chunks = li.sink_chunks;
            it.gap = li.gap;
            it.pos0 -= li.gap * kChunkKeys;
        }
    } else {
        it.split = idx % p.prefix_nsplit;
        const int qt = (idx / p.prefix_nsplit) % p.prefix_q_tiles;
        it.h = idx / (p.prefix_nsplit * p.prefix_q_tiles);
        it.nsplit = p.prefix_nsplit;
        it.tok0 = qt * TQ;
        it.nvalid = min(TQ, p.num_q_tokens - it.tok0);
        it.key_begin = it.split * p.prefix_split_keys;
        it.key_end = min(p.prefix_len, it.key_begin + p.prefix_split_keys);
        it.pair = it.h * p.prefix_q_tiles + qt;
        it.partial_base = it.pair * it.nsplit * kLongRows;
    }
    const int span = it.key_end - it.key_begin;
    it.nt = span > 0 ? (span + kLongKeys - 1) / kLongKeys : 0;
    return it;
}

// Item a CTA takes in round k: items are sorted longest first, and the CTAs
// take them in serpentine order (left to right, then right to left), which
// keeps the per-CTA totals close to a longest-processing-time schedule.
__device__ __forceinline__ int serpentine_item(int round) {
    const int g = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
    return round * g + ((round & 1) ? g - 1 - c : c);
}

// Dynamic schedule (p.dynamic): warp 0 -- the K producer, which runs ahead
// of every other role -- takes item indices from the step's counter, shared
// by every launch of the step, and publishes them in order in a shared
// memory queue; every other warp reads them back in the same order.  A
// CTA that starts late therefore simply takes fewer items.
constexpr int kItemQueue = 64;
constexpr int kSchedDone = -1, kSchedAbort = -2;
struct Sched {
    int *idx;            // [kItemQueue]
    volatile int *pub;   // items published
    volatile int *cons;  // [kLongWarps] items read per warp
};

__device__ __forceinline__ bool sched_spin(bool (*ready)(const Sched &, int), const Sched &sc,
                                           int k, volatile int *abort) {
    if (ready(sc, k)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (ready(sc, k)) return true;
        if (*abort) return false;
        if (global_timer_ns() - t0 > kWaitTimeoutNs) {
            *abort = 1;
            return false;
        }
    }
}
__device__ bool sched_published(const Sched &sc, int k) { return *sc.pub > k; }
__device__ bool sched_slot_free(const Sched &sc, int k) {
    for (int w = 1; w < kLongWarps; ++w)
        if (sc.cons[w] <= k - kItemQueue) return false;
    return true;
}

// Item of round k of this role, or kSchedDone / kSchedAbort.  One thread of
// the warp calls it (a whole-warp role broadcasts the result).
__device__ __forceinline__ int sched_take(const LongParams &p, const Sched &sc, int n_items,
                                          int k, int warp, volatile int *abort) {
    if (!p.dynamic) {
        if (k * static_cast<int>(gridDim.x) >= n_items) return kSchedDone;
        const int idx = serpentine_item(k);
        return idx < n_items ? idx : kSchedDone;
    }
    const int slot = k % kItemQueue;
    int idx;
    if (warp == 0) {
        if (k >= kItemQueue && !sched_spin(sched_slot_free, sc, k, abort)) return kSchedAbort;
        idx = atomicAdd(&p.hdr->long_next, 1);
        if (idx >= n_items) idx = kSchedDone;
        sc.idx[slot] = idx;
        __threadfence_block();
        *sc.pub = k + 1;
    } else {
        if (!sched_spin(sched_published, sc, k, abort)) return kSchedAbort;
        __threadfence_block();
        idx = reinterpret_cast<volatile int *>(sc.idx)[slot];
        sc.cons[warp] = k + 1;
    }
    return idx;
}

__device__ __forceinline__ int num_items(const LongParams &p) {
    if (p.prefix_mode) return p.num_kv_heads * p.prefix_q_tiles * p.prefix_nsplit;
    return *reinterpret_cast<volatile int *>(&p.hdr->num_long_items);
}

// Producer loop of the K warp (which also loads Q) and of the V warp: gathers one 128-key tile per step into its ring.
template <int D, int NS, bool WIN>
__device__ void produce(const LongParams &p, const Sched &sc, const CUtensorMap *tm, uint8_t *ring,
                        uint64_t *full, uint64_t *empty, uint64_t *q_full, uint64_t *q_empty,
                        bool load_q, const CUtensorMap *tmq, uint8_t *sQ,
                        volatile int *abort_flag) {
    using G = LongTiles<D>;
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int n_items = num_items(p);
    uint32_t t = 0;        // tiles issued by this warp so far (all items)
    uint32_t k_item = 0;   // items (with keys) started so far
    bool ok = true;
    for (int round = 0; ok; ++round) {
        int idx = 0;
        if (lane == 0) idx = sched_take(p, sc, n_items, round, warp, abort_flag);
        idx = __shfl_sync(0xffffffffu, idx, 0);
        if (idx == kSchedDone) break;
        if (idx == kSchedAbort) {
            ok = false;
            break;
        }
        const Item it = decode_item<WIN>(p, idx);
        if (it.nt == 0) continue;
        if (load_q) {
            if (k_item > 0 && !warp_wait(q_empty, (k_item - 1) & 1, abort_flag)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(q_full,
                                      static_cast<uint32_t>(G::kHalves * 128 * p.group *
                                                            p.q_tile_tokens));
                for (int hf = 0; hf < G::kHalves; ++hf)
                    tma_load_3d(sQ + hf * G::kHalfBytes, tmq, hf * 64, it.h * p.group, it.tok0,
                                q_full);
            }
        }
        ++k_item;
        const int *bt = p.block_tables + static_cast<int64_t>(it.b) * p.bt_stride;
        int my_row = p.kv_rows;
        for (int j = 0; j < it.nt; ++j, ++t) {
            if ((j & 3) == 0) {
                // rows of the next 32 chunks (4 tiles), one per lane; chunks
                // past key_end are read fully out of bounds -> zeros
                int key0 = it.key_begin + (j * 8 + lane) * kChunkKeys;
                my_row = p.kv_rows;
                if (key0 < it.key_end) {
                    if constexpr (WIN) key0 = unpacked_key(key0, it.sink_chunks, it.gap);
                    int col = key0 / p.block_size;
                    if (p.bt_stride > 0 && col >= p.bt_stride) {
                        flag_status(p.status, PA_DEV_BAD_METADATA);
                        col = p.bt_stride - 1;
                    }
                    // fp8 pool: block col of a staged request is its staging block
                    // (a windowed step stages its visible blocks)
                    int blk;
                    if (p.stage_base) {
                        blk = __ldcg(p.stage_base + it.b) + col;
                        if constexpr (WIN)
                            if (col >= it.block_sinks) blk -= it.block_gap;
                    } else {
                        blk = __ldg(bt + col);
                    }
                    if (blk < 0 || blk >= p.num_blocks) {
                        flag_status(p.status, PA_DEV_BAD_BLOCK);
                        blk = min(max(blk, 0), p.num_blocks - 1);
                    }
                    my_row = (blk * p.num_kv_heads + it.h) * p.block_size + key0 % p.block_size;
                }
            }
            const int slot = t % NS;
            if (t >= NS && !warp_wait(&empty[slot], ((t / NS) - 1) & 1, abort_flag)) {
                ok = false;
                break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&full[slot], static_cast<uint32_t>(G::kKVBytes));
            __syncwarp();
            const int c = lane & 7;
            const int row = __shfl_sync(0xffffffffu, my_row, (j & 3) * 8 + c);
            if (lane < 8) {
#pragma unroll
                for (int hf = 0; hf < G::kHalves; ++hf)
                    tma_load_2d(ring + slot * G::kKVBytes + hf * G::kHalfBytes + c * 2048, tm,
                                hf * 64, row, &full[slot]);
            }
            __syncwarp();
        }
    }
    if (*abort_flag && lane == 0) {
        // let copies already in flight land before the CTA exits
        for (uint32_t k = (t > NS ? t - NS : 0); k < t; ++k) mbar_drain(&full[k % NS], (k / NS) & 1);
    }
}

}  // namespace

}  // namespace pa
