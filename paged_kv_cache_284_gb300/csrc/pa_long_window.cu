// pa_long_window.cu -- tensor-core attention of a windowed step's long requests
// (prompt chunks under a sliding window with sinks): the row at position p
// sees key j <= p if j > p - window or j < sinks.
//
// Work items, packed visible chunks and operands are those of the plain kernel
// (pa_long.cu): 128-row query tiles (128 / group tokens x group heads), 128-key
// K and V tiles gathered by TMA through the block table, S = Q K^T and O += P V
// on tcgen05 with S, P and O in TMEM.  What differs is who does the softmax.
// There, all eight softmax warps work on one key tile at a time, two threads
// to a row; every wait of a tile's chain (scores, the halves' maxima, P) idles
// all of them, and a key tile takes ~2300 cycles against 1024 of MMA.  Here
//  * two groups of four warps take the key tiles in turn, one thread to a row,
//    so one group's waits lie beside the other's arithmetic; each group has its
//    own S and its own P in TMEM, and a row's scores are read in two halves so
//    that 168 registers hold them;
//  * both groups share one accumulator O, so they must agree on each row's
//    reference (the running maximum its exponents are taken against).  A tile's
//    reference is the tile before's unless the tile's maximum exceeds it by
//    2^8 (then O is rescaled), and is handed from tile to tile through shared
//    memory as soon as the tile's maximum is known, long before its P is.
//    Sums are kept per group, each against the reference it last used, and
//    added at the item's end;
//  * items are decoded once, by the K producer, and read by every role from a
//    queue in shared memory; the group that has an item's last tile writes its
//    output while the other begins the next item;
//  * K and V rings are three tiles deep, and Q K^T and P V are issued by two
//    warps (an elected lane of each): a 128 x 128 x 128 group of MMAs takes
//    700-800 cycles by itself and 512 beside the other warp's; one issuing thread
//    for both was slower (616 us against 487 on the case below).
// Two chunks of 4096 tokens, window 4096 + 16 sinks, 32 q / 8 kv heads, d = 128, 552
// GFLOP of visible pairs: 473 us, 1167 TFLOP/s, 0.61 of the measured bf16 rate (565 us
// in the plain kernel's form).  Bound: the chain of a key tile (scores, maximum,
// exponentials, P V) at ~1900 cycles for two tiles in flight, against 1024 of MMA;
// a third S tile with P written over S left too few registers and columns to win.
#include "pa_long.cuh"

namespace pa {

namespace {

// warps: 0 K (+Q) loads, 1 Q K^T issuer (+TMEM allocation), 2 V loads, 3 P V
// issuer, 4-7 softmax of even tiles, 8-11 of odd ones
constexpr int kWarpQK = 1, kWarpV = 2, kWarpPV = 3, kFirstSoftmax = 4;
constexpr int kGroupWarps = 4;
// Key tiles of K (and of V) in shared memory.  A K tile lands ~3000 cycles after
// its copies are issued, under load.
constexpr int kRing = 3;

// A work item as every role needs it (positions and keys packed).
struct alignas(16) WinItem {
    int b, h, tok0, nvalid;         // query tokens [tok0, tok0 + nvalid), kv head h
    int pos0, key_end, nt;          // first position, end of the keys, key tiles (0: no more items)
    int sink_chunks, gap;           // KeySpan
    int block_sinks, block_gap, pad;  // BlockSpan of the request (staged blocks)
};
static_assert(sizeof(WinItem) == 48, "queue entry");
constexpr int kQueue = 8;

template <int D>
struct WinGeom {
    static constexpr int kHalves = D / 64;
    static constexpr int kHalfBytes = 128 * 128;            // 128 rows x 128 B
    static constexpr int kQBytes = kHalves * kHalfBytes;    // Q tile
    static constexpr int kKVBytes = kHalves * kHalfBytes;   // one K (or V) tile of 128 keys
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kQBytes;
    static constexpr int kOffV = kOffK + kRing * kKVBytes;
    static constexpr int kOffBar = kOffV + kRing * kKVBytes;
    static constexpr int kOffCtl = kOffBar + 336;
    // items published by the K producer, their count, and how many each warp has read
    static constexpr int kOffQueue = kOffCtl + 32;
    static constexpr int kOffRead = kOffQueue + kQueue * static_cast<int>(sizeof(WinItem));
    // per row: references by tile parity [2][128], sums by item parity [2][128]
    static constexpr int kOffRef = kOffRead + 64;
    static constexpr int kOffSum = kOffRef + 2 * 128 * 4;
    static constexpr int kSmemRaw = kOffSum + 2 * 128 * 4;
    // at least 116 KiB so that one CTA owns an SM (and its 512 TMEM columns)
    static constexpr int kSmemBytes = kSmemRaw > 116 * 1024 ? kSmemRaw : 116 * 1024;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
    // TMEM columns: S0 | S1 (fp32 scores) | O (fp32) | P0 | P1 (bf16 pairs)
    static constexpr uint32_t kTmemCols = 512;
    static constexpr int kColO = 2 * kLongKeys, kColP = 3 * kLongKeys;
    static_assert(kColO + D <= kColP, "TMEM");
};

struct Bars {
    uint64_t q_full, q_empty;
    uint64_t k_full[kRing], k_empty[kRing];
    uint64_t v_full[kRing], v_empty[kRing];
    // by tile parity, that is, by group
    uint64_t s_full[2], s_free[2];  // scores of a tile written / read (4 warps)
    uint64_t p_full[2], pv_done[2]; // P of a tile written (4 warps) / its P V finished
    uint64_t ref[4][2];         // reference of a tile published, by row quarter and tile parity
    uint64_t sums[2][4];        // the other group's sums of an item left, by item parity and quarter
    uint64_t o_free, drain, drain_pv;
};
static_assert(sizeof(Bars) <= 336, "barrier area");

// A step without a plan (p.own_seqs > 0, at most a warp's lanes of requests): lane b
// holds request b and the tiles up to and with it; a short request has none.
struct OwnPlan {
    int q0, n, ctx, tiles, incl, total;
};
__device__ __forceinline__ OwnPlan own_plan(const LongParams &p) {
    const int lane = threadIdx.x & 31;
    OwnPlan o{};
    if (lane < p.own_seqs) {
        o.q0 = __ldg(p.qsl + lane);
        const int q1 = __ldg(p.qsl + lane + 1), len = __ldg(p.seq_lens + lane);
        o.ctx = p.ctx ? __ldg(p.ctx + lane) : len;  // (cross attention)
        o.n = q1 - o.q0;
        // (a request that the short rows' kernel flags is skipped here too)
        const bool bad = o.n < 0 || o.ctx < 0 || len > p.own_max_keys ||
                         (p.ctx && len != o.ctx + o.n) || o.q0 < 0 || q1 > p.num_q_tokens;
        if (bad) o.n = 0;
        if (o.n * p.group > kShortMaxRows)
            o.tiles = (o.n + p.q_tile_tokens - 1) / p.q_tile_tokens;
    }
    // requests that overlap: none runs
    long long tokens = o.n;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) tokens += __shfl_xor_sync(0xffffffffu, tokens, i);
    if (tokens > p.num_q_tokens) {
        if (blockIdx.x == 0 && threadIdx.x == 0) flag_status(p.status, PA_DEV_PLAN_OVERFLOW);
        o.tiles = 0;
    }
    o.incl = o.tiles;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
        const int before = __shfl_up_sync(0xffffffffu, o.incl, i);
        if (lane >= i) o.incl += before;
    }
    o.total = __shfl_sync(0xffffffffu, o.incl, 31);
    return o;
}
// Its tile `t`, with the request's first row, tokens and context.
__device__ __forceinline__ LongItem own_tile(const LongParams &p, const OwnPlan &o, int t, int &q0,
                                             int &n, int &ctx) {
    const int excl = o.incl - o.tiles;
    const unsigned owner = __ballot_sync(0xffffffffu, excl <= t && t < o.incl);
    const int src = __ffs(owner) - 1;
    q0 = __shfl_sync(0xffffffffu, o.q0, src);
    n = __shfl_sync(0xffffffffu, o.n, src);
    ctx = __shfl_sync(0xffffffffu, o.ctx, src);
    LongItem it{};
    it.b = src;
    it.q_tile = t - __shfl_sync(0xffffffffu, excl, src);
    const int first = it.q_tile * p.q_tile_tokens;
    const KeySpan ks = p.ctx
                           ? key_span(p.win, ctx + first, ctx + min(n, first + p.q_tile_tokens))
                           : key_span(p.win, ctx, ctx);
    it.key_end = ks.keys;
    it.sink_chunks = ks.sink_chunks;
    it.gap = ks.gap;
    return it;
}

// Items in order, one reader per warp.  Warp 0, which runs ahead of every other
// role, takes an item's index -- from the step's counter, shared by every
// launch of the step (p.dynamic), so that a CTA that starts late takes fewer;
// else in serpentine order over the CTAs -- decodes it once and publishes it, so
// that no other role starts an item with a chain of global loads (measured:
// ~1500 cycles of each softmax group's time per item).
struct Queue {
    WinItem *items;
    volatile int *published;
    volatile int *read;  // [kLongWarps]
    volatile int *abort;
};
template <typename Ready>
__device__ __forceinline__ bool queue_spin(const Queue &q, Ready ready) {
    if (ready()) return true;
    const uint64_t t0 = global_timer_ns();
    while (!ready()) {
        if (*q.abort) return false;
        if (global_timer_ns() - t0 > kWaitTimeoutNs) {
            *q.abort = 1;
            return false;
        }
    }
    return true;
}
// Warp 0, all lanes: takes, publishes and returns item k.
__device__ __forceinline__ WinItem queue_next(const LongParams &p, const Queue &q, int n_items,
                                              const OwnPlan &own, int k) {
    const int lane = threadIdx.x & 31;
    int idx = 0;
    if (lane == 0) {
        if (p.dynamic) {
            idx = atomicAdd(&p.hdr->long_next, 1);
        } else {
            const int g = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
            idx = k * g + ((k & 1) ? g - 1 - c : c);
        }
    }
    idx = __shfl_sync(0xffffffffu, idx, 0);
    WinItem it{};
    if (idx < n_items) {
        const int rec = idx / p.num_kv_heads, TQ = p.q_tile_tokens;
        LongItem li;
        int q0, n, ctx;
        if (p.own_seqs > 0) {  // a request's last tiles, which may see more, first
            li = own_tile(p, own, own.total - 1 - rec, q0, n, ctx);
        } else {
            li = load_record(p.items, rec);
            q0 = __ldg(p.qsl + li.b);
            n = __ldg(p.qsl + li.b + 1) - q0;
            ctx = p.ctx ? __ldg(p.ctx + li.b) : __ldg(p.seq_lens + li.b);
        }
        it.b = li.b;
        it.h = idx - rec * p.num_kv_heads;
        it.tok0 = q0 + li.q_tile * TQ;
        it.nvalid = min(TQ, n - li.q_tile * TQ);
        // (cross attention: behind all keys, which may be none: then one tile of zeros)
        it.pos0 = p.ctx ? ctx + li.q_tile * TQ - li.gap * kChunkKeys : ctx;
        it.key_end = li.key_end;
        it.nt = max(1, (li.key_end + kLongKeys - 1) / kLongKeys);
        it.sink_chunks = li.sink_chunks;
        it.gap = li.gap;
        if (p.stage_base) {
            const BlockSpan bsp = block_span(p.win, ctx, p.ctx ? ctx + n : ctx, p.block_size);
            it.block_sinks = bsp.sink_blocks;
            it.block_gap = bsp.gap;
        }
    }
    if (lane == 0) {
        // entry k % kQueue is free once every warp has read item k - kQueue
        const bool ok = k < kQueue || queue_spin(q, [&] {
            for (int w = 1; w < kLongWarps; ++w)
                if (q.read[w] <= k - kQueue) return false;
            return true;
        });
        if (ok) {
            q.items[k % kQueue] = it;
            __threadfence_block();
            *q.published = k + 1;
        }
    }
    if (__any_sync(0xffffffffu, *q.abort)) it.nt = 0;
    return it;
}
// Any other warp, all lanes: item k (nt = 0: no more, or aborted).
__device__ __forceinline__ WinItem queue_item(const Queue &q, int warp, int k) {
    const int lane = threadIdx.x & 31;
    int ok = 1;
    if (lane == 0) ok = queue_spin(q, [&] { return *q.published > k; }) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    WinItem it{};
    if (ok) {
        __threadfence_block();
        const volatile int *src = reinterpret_cast<const volatile int *>(q.items + k % kQueue);
        int *dst = reinterpret_cast<int *>(&it);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(WinItem) / sizeof(int)); ++i) dst[i] = src[i];
    }
    __syncwarp();
    if (lane == 0) q.read[warp] = k + 1;
    return it;
}

// Loads of the K warp (which also takes the items and loads Q) and of the V
// warp: gathers one 128-key tile per step into its ring, eight 16-key chunks
// through the block table.
template <int D>
__device__ void produce(const LongParams &p, const Queue &q, int n_items, const OwnPlan &own,
                        const CUtensorMap *tm, uint8_t *ring, uint64_t *full, uint64_t *empty, Bars *bars,
                        const CUtensorMap *tmq, uint8_t *sQ, int warp) {
    using G = WinGeom<D>;
    const int lane = threadIdx.x & 31;
    uint32_t t = 0;  // tiles issued so far (all items)
    bool ok = true;
    for (int k = 0; ok; ++k) {
        const WinItem it = tmq ? queue_next(p, q, n_items, own, k) : queue_item(q, warp, k);
        if (it.nt == 0) break;
        if (tmq) {
            if (k > 0 && !warp_wait(&bars->q_empty, (k - 1) & 1, q.abort)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars->q_full, static_cast<uint32_t>(
                                                         G::kHalves * 128 * p.group *
                                                         p.q_tile_tokens));
                for (int hf = 0; hf < G::kHalves; ++hf)
                    tma_load_3d(sQ + hf * G::kHalfBytes, tmq, hf * 64, it.h * p.group, it.tok0,
                                &bars->q_full);
            }
        }
        const int *bt = p.block_tables + static_cast<int64_t>(it.b) * p.bt_stride;
        int my_row = p.kv_rows;
        for (int j = 0; j < it.nt; ++j, ++t) {
            if ((j & 3) == 0) {
                // rows of the next 32 chunks (4 tiles), one per lane; chunks
                // past key_end are read fully out of bounds -> zeros
                int key0 = (j * 8 + lane) * kChunkKeys;
                my_row = p.kv_rows;
                if (key0 < it.key_end) {
                    key0 = unpacked_key(key0, it.sink_chunks, it.gap);
                    int col = key0 / p.block_size;
                    if (col >= p.bt_stride) {
                        flag_status(p.status, PA_DEV_BAD_METADATA);
                        col = p.bt_stride - 1;
                    }
                    // fp8 pool: a request's visible blocks in their order are
                    // its staging blocks
                    int blk = p.stage_base ? __ldcg(p.stage_base + it.b) + col -
                                                 (col >= it.block_sinks ? it.block_gap : 0)
                                           : __ldg(bt + col);
                    if (blk < 0 || blk >= p.num_blocks) {
                        flag_status(p.status, PA_DEV_BAD_BLOCK);
                        blk = min(max(blk, 0), p.num_blocks - 1);
                    }
                    my_row = (blk * p.num_kv_heads + it.h) * p.block_size + key0 % p.block_size;
                }
            }
            const int slot = t % kRing;
            if (t >= kRing && !warp_wait(&empty[slot], (t / kRing - 1) & 1, q.abort)) {
                ok = false;
                break;
            }
            // test hook: stop after the first tile, as a producer would whose wait
            // had run out
            if (p.test_stall && tmq && blockIdx.x == 0 && t == 1) {
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
    if (*q.abort && lane == 0) {
        // let copies already in flight land before the CTA exits
        for (uint32_t i = (t > kRing ? t - kRing : 0); i < t; ++i)
            mbar_drain(&full[i % kRing], (i / kRing) & 1);
    }
}

// True for one lane of the warp, whose lanes all call this together.  That lane issues the MMAs:
// it waits, issues and commits in a branch of its own, and the others wait for it at the vote
// behind an item.  So no lane but the issuing one runs between a barrier and the MMAs, and no
// operand depends on lanes having met again after each has polled a barrier for itself (as they
// had to when all lanes ran the loop and the MMAs were predicated; that took 488 us on the case
// above).  With `lane == 0` in the place of the election it takes 547: the compiler then looks for
// the operands of more than one lane.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e != 0;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(32 * kLongWarps, 1)
    long_window_kernel(const LongParams p, const __grid_constant__ CUtensorMap tmq,
                       const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv) {
    using G = WinGeom<D>;
    constexpr int KS = D / 16;
    // (swizzled tiles: the three rings leave no room to align them by hand)
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars *bars = reinterpret_cast<Bars *>(smem + G::kOffBar);
    int *ctl = reinterpret_cast<int *>(smem + G::kOffCtl);
    volatile int *abort_flag = ctl;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ctl + 4);

    // (a shuffled warp index is uniform to the compiler, and so is what follows it)
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    if (p.wait_start) {
        pdl_wait();     // the plan (and any staging copy) first
        pdl_trigger();  // then the split-KV grid may take the other SMs
    }
    // (without a plan: the short rows' grid, which lets this one start, waited for
    // whatever wrote the metadata)
    OwnPlan own{};
    if (p.own_seqs > 0) own = own_plan(p);
    const int n_items = p.own_seqs > 0
                            ? own.total * p.num_kv_heads
                            : *reinterpret_cast<volatile int *>(&p.hdr->num_long_items);
    if (!p.first_done && static_cast<int>(blockIdx.x) >= n_items) {
        pdl_wait();  // complete only after the grid this one overlaps
        return;
    }
    Queue queue;
    queue.items = reinterpret_cast<WinItem *>(smem + G::kOffQueue);
    queue.published = reinterpret_cast<int *>(smem + G::kOffRead);
    queue.read = queue.published + 1;
    queue.abort = abort_flag;

    // ---- setup ----------------------------------------------------------------
    if (threadIdx.x == 0) {
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_empty, 1);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&bars->k_full[i], 1);
            mbar_init(&bars->k_empty[i], 1);
            mbar_init(&bars->v_full[i], 1);
            mbar_init(&bars->v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->s_free[i], kGroupWarps);
            mbar_init(&bars->p_full[i], kGroupWarps);
            mbar_init(&bars->pv_done[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars->ref[i][0], 1);
            mbar_init(&bars->ref[i][1], 1);
            mbar_init(&bars->sums[0][i], 1);
            mbar_init(&bars->sums[1][i], 1);
        }
        mbar_init(&bars->o_free, kGroupWarps);
        mbar_init(&bars->drain, 1);
        mbar_init(&bars->drain_pv, 1);
        ctl[0] = 0;
        *queue.published = 0;
        for (int w = 0; w < kLongWarps; ++w) queue.read[w] = 0;
        fence_mbar_init();
    }
    if (warp == kWarpQK) tmem_alloc(tmem_slot, G::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    uint8_t *sQ = smem + G::kOffQ;
    uint8_t *sK = smem + G::kOffK;
    uint8_t *sV = smem + G::kOffV;

    if (warp == 0) {
        // ============================ K (and Q) loads ============================
        if (lane == 0) {
            tma_prefetch_desc(&tmq);
            tma_prefetch_desc(&tmk);
        }
        produce<D>(p, queue, n_items, own, &tmk, sK, bars->k_full, bars->k_empty, bars, &tmq, sQ, warp);
    } else if (warp == kWarpV) {
        // ============================ V loads ============================
        if (lane == 0) tma_prefetch_desc(&tmv);
        produce<D>(p, queue, n_items, own, &tmv, sV, bars->v_full, bars->v_empty, bars, nullptr, nullptr,
                   warp);
    } else if (warp == kWarpQK) {
        // ============================ Q K^T issuer ============================
        // A tile's scores wait for its K tile and for the scores two tiles back
        // to have been read.
        constexpr uint32_t idesc_qk = idesc_bf16_f32(kLongRows, kLongKeys, 0);
        const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t k_desc = smem_desc_sw128(smem_u32(sK), 16, 1024);
        const bool mine = elect_one();
        uint32_t t = 0, k_item = 0;
        bool ok = true;
        for (; ok; ++k_item) {
            const int nt = __shfl_sync(0xffffffffu, queue_item(queue, warp, k_item).nt, 0);
            if (nt == 0) break;
            if (mine) {
                ok = mbar_wait(&bars->q_full, k_item & 1, abort_flag);
                int j = 0;
                for (; ok && j < nt; ++j) {
                    const uint32_t tt = t + j;
                    const int ks = tt % kRing;
                    const int sb = tt & 1;
                    ok = mbar_wait(&bars->k_full[ks], (tt / kRing) & 1, abort_flag) &&
                         (tt < 2 || mbar_wait(&bars->s_free[sb], ((tt - 2) >> 1) & 1, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t kd = k_desc + static_cast<uint32_t>(ks * (G::kKVBytes >> 4));
#pragma unroll
                    for (int kk = 0; kk < KS; ++kk) {
                        constexpr int kHalf16 = G::kHalfBytes >> 4;
                        const int off = (kk >> 2) * kHalf16 + (kk & 3) * 2;  // 16-byte units
                        tc_mma(tmem + sb * kLongKeys, q_desc + off, kd + off, idesc_qk,
                               kk > 0 ? 1u : 0u);
                    }
                    tc_commit(&bars->s_full[sb]);
                    tc_commit(&bars->k_empty[ks]);
                    if (j == nt - 1) tc_commit(&bars->q_empty);
                }
                if (p.tile_counter) atomicAdd(p.tile_counter, static_cast<unsigned long long>(j));
            }
            ok = __all_sync(0xffffffffu, ok);
            t += nt;
        }
        if (mine && (!ok || *abort_flag)) {
            // let every MMA already issued finish before TMEM is released
            tc_commit(&bars->drain);
            mbar_drain(&bars->drain, 0);
        }
        __syncwarp();
    } else if (warp == kWarpPV) {
        // ============================ P V issuer ============================
        // A tile's P V waits for its P, its V tile and, at the start of an item,
        // for the previous item's epilogue to read O.
        constexpr uint32_t idesc_pv = idesc_bf16_f32(kLongRows, D, 1);
        const uint64_t v_desc = smem_desc_sw128(smem_u32(sV), G::kHalfBytes, 1024);
        const bool mine = elect_one();
        uint32_t t = 0, k_item = 0;
        bool ok = true;
        for (; ok; ++k_item) {
            const int nt = __shfl_sync(0xffffffffu, queue_item(queue, warp, k_item).nt, 0);
            if (nt == 0) break;
            if (mine) {
                for (int j = 0; j < nt; ++j) {
                    const uint32_t tt = t + j;
                    const int sb = tt & 1;
                    const int vs = tt % kRing;
                    ok = (j > 0 || k_item == 0 ||
                          mbar_wait(&bars->o_free, (k_item - 1) & 1, abort_flag)) &&
                         mbar_wait(&bars->v_full[vs], (tt / kRing) & 1, abort_flag) &&
                         mbar_wait(&bars->p_full[sb], (tt >> 1) & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t vd = v_desc + static_cast<uint32_t>(vs * (G::kKVBytes >> 4));
                    // P (bf16) of this tile: row r in TMEM lane r, key k in column k / 2
                    const uint32_t pcol = tmem + G::kColP + sb * (kLongKeys / 2);
#pragma unroll
                    for (int kk = 0; kk < kLongKeys / 16; ++kk)
                        tc_mma_ts(tmem + G::kColO, pcol + kk * 8, vd + kk * (2048 >> 4), idesc_pv,
                                  (j > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(&bars->pv_done[sb]);
                    tc_commit(&bars->v_empty[vs]);
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            t += nt;
        }
        if (mine && (!ok || *abort_flag)) {
            tc_commit(&bars->drain_pv);
            mbar_drain(&bars->drain_pv, 0);
        }
        __syncwarp();
    } else {
        // ============================ softmax + epilogue ============================
        const int wq = warp & 3;  // TMEM lane quarter of this warp
        const int grp = (warp - kFirstSoftmax) / kGroupWarps;
        const int r = wq * 32 + lane;
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const int ttok = r / p.group;
        const int jh = r - ttok * p.group;
        float *refs = reinterpret_cast<float *>(smem + G::kOffRef) + r;  // [parity * 128]
        float *sums = reinterpret_cast<float *>(smem + G::kOffSum) + r;  // [item parity * 128]
        uint32_t t = 0, k_item = 0;
        bool ok = true;
        for (; ok; ++k_item) {
            const WinItem it = queue_item(queue, warp, k_item);
            if (it.nt == 0) break;
            const bool row_valid = ttok < it.nvalid && r < p.q_tile_tokens * p.group;
            // (packed keys) this row's last key, and the first row's lowest key
            // behind the sinks
            const int row_limit = it.pos0 + ttok;
            const int low_first = it.pos0 - p.win.window + 1;
            // scores in log2 units; an fp8 pool's K scale folds in here
            const float sl2 = p.k_scale ? p.scale_log2 * __ldg(p.k_scale + it.h) : p.scale_log2;
            float ref = -INFINITY, l = 0.f;  // this group's sum, against `ref`
            float before = -INFINITY;        // the reference of the tile before the last one done
            for (int j = (t & 1) == static_cast<uint32_t>(grp) ? 0 : 1; j < it.nt; j += 2) {
                const uint32_t tt = t + j;
                const int kb = j * kLongKeys;
                if (!warp_mbar_wait_spin(&bars->s_full[grp], (tt >> 1) & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                // The row's 128 scores, 64 at a time: keys 64..127 for their
                // maximum, keys 0..63, and later keys 64..127 again.
                uint32_t s0[32], s1[32];
                const uint32_t sa = t_lane + grp * kLongKeys;
                // Tiles that hold a key some row does not see are masked; bit i:
                // key at + i is below the causal limit, and a sink or at or past
                // this row's low.
                const bool need_mask =
                    kb + kLongKeys - 1 > it.pos0 || kb + kLongKeys > it.key_end ||
                    (kb < low_first + it.nvalid - 1 && kb + kLongKeys > p.win.sinks);
                auto mask = [&](int at) {
                    const uint64_t seen = low_bits(min(row_limit, it.key_end - 1) + 1 - at) &
                                          (low_bits(p.win.sinks - at) |
                                           ~low_bits(row_limit - p.win.window + 1 - at));
                    const uint32_t lo = static_cast<uint32_t>(seen);
                    const uint32_t hi = static_cast<uint32_t>(seen >> 32);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (!(lo & (1u << i))) s0[i] = __float_as_uint(-INFINITY);
                        if (!(hi & (1u << i))) s1[i] = __float_as_uint(-INFINITY);
                    }
                };
                float mx = -INFINITY;
                auto row_max = [&]() {
                    float mx0 = mx, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        mx0 = max3(mx0, __uint_as_float(s0[i]), __uint_as_float(s0[i + 1]));
                        mx1 = max3(mx1, __uint_as_float(s0[16 + i]), __uint_as_float(s0[17 + i]));
                        mx2 = max3(mx2, __uint_as_float(s1[i]), __uint_as_float(s1[i + 1]));
                        mx3 = max3(mx3, __uint_as_float(s1[16 + i]), __uint_as_float(s1[17 + i]));
                    }
                    mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
                };
                tmem_ld32(sa + 64, s0);
                tmem_ld32(sa + 96, s1);
                tmem_wait_ld();
                if (need_mask) mask(kb + 64);
                row_max();
                tmem_ld32(sa, s0);
                tmem_ld32(sa + 32, s1);
                tmem_wait_ld();
                if (need_mask) mask(kb);
                row_max();
                // the reference: the tile before's, unless this tile exceeds it
                before = -INFINITY;
                if (tt > 0) {
                    if (!warp_mbar_wait_spin(&bars->ref[wq][(tt - 1) & 1], ((tt - 1) >> 1) & 1, abort_flag)) { ok = false; break; }
                    if (j > 0) before = *reinterpret_cast<volatile float *>(refs + ((tt - 1) & 1) * 128);
                }
                const float mxs = mx * sl2;  // scale > 0: max commutes with it
                const bool up = mxs > before + kRescaleThreshold || (before == -INFINITY && mxs > -INFINITY);
                const float now = up ? mxs : before;
                *reinterpret_cast<volatile float *>(refs + (tt & 1) * 128) = now;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->ref[wq][tt & 1]);
                if (ref != now) {
                    l = ref == -INFINITY ? 0.f : l * fast_exp2(ref - now);
                    ref = now;
                }
                const float neg_ref = now == -INFINITY ? 0.f : -now;
                // P row r (bf16 pairs: an MMA's operands have one type, and V is bf16; the
                // sums above take the unrounded values), in four pieces so that a piece's store lies
                // beside the next one's exponentials; the P V that used this
                // buffer two tiles ago must be done
                if (tt >= 2 && !warp_mbar_wait_spin(&bars->pv_done[grp], ((tt - 2) >> 1) & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                const uint64_t sc2 = f2_pack(sl2, sl2);
                const uint64_t nr2 = f2_pack(neg_ref, neg_ref);
                uint64_t acc0 = f2_pack(0.f, 0.f), acc1 = acc0;
                auto exps = [&](const uint32_t (&sv)[32], uint32_t dst) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        float a0, a1, a2, a3;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])),
                                         sc2, nr2), a0, a1);
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[2 * i + 2]), __uint_as_float(sv[2 * i + 3])),
                                         sc2, nr2), a2, a3);
                        a0 = fast_exp2(a0);
                        a1 = fast_exp2(a1);
                        a2 = fast_exp2(a2);
                        a3 = fast_exp2(a3);
                        acc0 = f2_add(acc0, f2_pack(a0, a1));
                        acc1 = f2_add(acc1, f2_pack(a2, a3));
                        pk[i] = pack_bf16x2(a0, a1);
                        pk[i + 1] = pack_bf16x2(a2, a3);
                    }
                    tmem_st16(dst, pk);
                };
                const uint32_t pdst = t_lane + G::kColP + grp * (kLongKeys / 2);
                exps(s0, pdst);
                tmem_ld32(sa + 64, s0);
                exps(s1, pdst + 16);
                tmem_ld32(sa + 96, s1);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->s_free[grp]);
                if (need_mask) mask(kb + 64);
                exps(s0, pdst + 32);
                exps(s1, pdst + 48);
                float sum0, sum1, sum2, sum3;
                f2_unpack(acc0, sum0, sum1);
                f2_unpack(acc1, sum2, sum3);
                l += (sum0 + sum1) + (sum2 + sum3);
                // O is rescaled in place where the reference moved: the previous
                // tile's P V must be done, this tile's has not begun
                const float alpha = up && before != -INFINITY ? fast_exp2(before - now) : 1.f;
                if (j >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    if (!warp_mbar_wait_spin(&bars->pv_done[(tt - 1) & 1], ((tt - 1) >> 1) & 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll
                    for (int qd = 0; qd < D / 32; ++qd) {
                        tmem_ld32(t_lane + G::kColO + qd * 32, s0);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            s0[i] = __float_as_uint(__uint_as_float(s0[i]) * alpha);
                        tmem_st32(t_lane + G::kColO + qd * 32, s0);
                    }
                }
                // V rows that no row of the tile sees may hold anything and are
                // zeroed before a zero probability meets them: past the item's
                // keys (the rest of their chunk), and between the sinks and the
                // first row's window (at most 30 keys that share chunks with
                // visible ones)
                bool zeroed = false;
                auto zero_rows = [&](int z0, int z1) -> bool {
                    if (z0 >= z1) return true;
                    zeroed = true;
                    const int vs = tt % kRing;
                    if (!warp_mbar_wait_spin(&bars->v_full[vs], (tt / kRing) & 1, abort_flag)) return false;
                    const int pieces = (z1 - z0) * 8 * G::kHalves;  // 16-byte pieces
                    for (int q = r; q < pieces; q += 32 * kGroupWarps) {
                        const int hf = q / ((z1 - z0) * 8);
                        const int rem = q - hf * (z1 - z0) * 8;
                        *reinterpret_cast<uint4 *>(sV + vs * G::kKVBytes + hf * G::kHalfBytes +
                                                   (z0 + rem / 8) * 128 + (rem % 8) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    return true;
                };
                const int tail = it.key_end - kb;
                if (!zero_rows(max(p.win.sinks - kb, 0), min(low_first - kb, kLongKeys)) ||
                    !zero_rows(tail, min(kLongKeys, (tail + 15) & ~15))) {
                    ok = false;
                    break;
                }
                __syncwarp();  // (lanes zero different numbers of pieces)
                tmem_wait_st();
                if (zeroed) fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->p_full[grp]);
            }

            if (!ok) break;
            // ---- epilogue ----
            // The group of the item's last tile writes the output; the other
            // leaves its sum (against the last tile's `before`) and goes on to
            // the next item, whose first tile is its own.
            const uint32_t last = t + it.nt - 1;
            float *left = sums + (k_item & 1) * 128;
            uint64_t *sums_bar = &bars->sums[k_item & 1][wq];
            t += it.nt;
            if ((last & 1) != static_cast<uint32_t>(grp)) {
                *reinterpret_cast<volatile float *>(left) = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(sums_bar);
                continue;
            }
            ok = warp_mbar_wait_spin(sums_bar, (k_item >> 1) & 1, abort_flag);
            if (ok && before != -INFINITY)
                l += *reinterpret_cast<volatile float *>(left) * fast_exp2(before - ref);
            if (ok) ok = warp_mbar_wait_spin(&bars->pv_done[last & 1], (last >> 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            // an fp8 pool's V scale multiplies the output
            const float vsc = p.v_scale ? __ldg(p.v_scale + it.h) : 1.f;
            const float inv = l > 0.f ? vsc / l : 0.f;
            const int64_t orow = static_cast<int64_t>(it.tok0 + ttok) * p.num_q_heads +
                                 it.h * p.group + jh;
            uint4 *dst = reinterpret_cast<uint4 *>(p.out + orow * D);
#pragma unroll
            for (int qd = 0; qd < D / 32; ++qd) {
                uint32_t raw[32];
                __syncwarp();  // (lanes without a row have not written the piece before)
                tmem_ld32(t_lane + G::kColO + qd * 32, raw);
                tmem_wait_ld();
                if (qd == D / 32 - 1) {
                    // O has been read: the next item's first P V may overwrite it
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->o_free);
                }
                if (!row_valid) continue;
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) {
                    uint4 w;
                    w.x = pack_bf16x2(__uint_as_float(raw[v4 * 8 + 0]) * inv, __uint_as_float(raw[v4 * 8 + 1]) * inv);
                    w.y = pack_bf16x2(__uint_as_float(raw[v4 * 8 + 2]) * inv, __uint_as_float(raw[v4 * 8 + 3]) * inv);
                    w.z = pack_bf16x2(__uint_as_float(raw[v4 * 8 + 4]) * inv, __uint_as_float(raw[v4 * 8 + 5]) * inv);
                    w.w = pack_bf16x2(__uint_as_float(raw[v4 * 8 + 6]) * inv, __uint_as_float(raw[v4 * 8 + 7]) * inv);
                    dst[qd * 4 + v4] = w;
                }
            }
            if (row_valid && p.lse)
                p.lse[orow] = l > 0.f ? (ref + __log2f(l)) * kLn2 : -INFINITY;
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (after the barrier: thread 0's warp may be done long before another's wait runs out)
    if (*abort_flag && threadIdx.x == 0) flag_status(p.status, PA_DEV_WAIT_TIMEOUT);
    if (warp == kWarpQK) tmem_dealloc(tmem, G::kTmemCols);
    // with overlap_prev: this grid completes only after the split-KV grid it
    // overlapped, so later work on the stream is still ordered after both
    pdl_wait();
    if (p.first_done && threadIdx.x == 0) {
        if (p.first_ctas < 0) {
            // a first launch of the step: count this CTA done (its outputs first)
            __threadfence();
            atomicAdd(p.first_done, 1);
        } else {
            // the last launch: complete only after every CTA of the first one
            const uint64_t t0 = global_timer_ns();
            while (*reinterpret_cast<volatile int *>(p.first_done) < p.first_ctas) {
                if (global_timer_ns() - t0 > kWaitTimeoutNs) {
                    flag_status(p.status, PA_DEV_WAIT_TIMEOUT);
                    break;
                }
            }
            __threadfence();
        }
    }
}

template <int D>
static int launch(const LongParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                  const CUtensorMap &tv, int grid, cudaStream_t s) {
    static PerDeviceOnce once;
    if (once_per_device(once, [] {
            return cudaFuncSetAttribute(long_window_kernel<D>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        WinGeom<D>::kSmemBytes);
        }) != PA_OK)
        return PA_ERR_CUDA;
    const bool pdl = p.overlap_prev != 0 || p.wait_start != 0;
    PdlLaunch l(grid, 32 * kLongWarps, WinGeom<D>::kSmemBytes, s, pdl);
    return launch_kernel(l, long_window_kernel<D>, p, tq, tk, tv) == cudaSuccess ? PA_OK
                                                                                 : PA_ERR_CUDA;
}

// grid: an upper bound on the number of items; at most one CTA per SM is launched.
int launch_long_window(const LongParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                       const CUtensorMap &tv, int head_dim, int grid, int sms, cudaStream_t s) {
    grid = grid < sms ? grid : sms;
    if (grid <= 0) return PA_OK;
    return head_dim == 128 ? launch<128>(p, tq, tk, tv, grid, s)
                           : launch<64>(p, tq, tk, tv, grid, s);
}

}  // namespace pa
