// pa_linear_prompt.cu -- linear attention with a decay per head: prompts, in chunks of 64
// tokens on tcgen05.
//
// With G_i the sum of the logarithms of a chunk's decays up to and with token i, S the state
// before the chunk and L the chunk's last token,
//   o_i  = scale (e^(G_i) q_i S + sum_(j <= i) e^(G_i - G_j) (q_i k_j) v_j)
//   S'   = e^(G_L) S + sum_j (e^(G_L - G_j) k_j) v_j^T
// Every exponent is at most 0.  Columns of S and of o do not depend on each other, so a CTA
// has 64 of them (a slice), for one request and kv head, and walks along the request:
//   scores  Q K^T            M = 64 tokens x 2 query heads of the group (1: half the rows idle)
//   inside  P V              P = the scores times e^(G_i - G_j), masked, over them in TMEM
//   before  Q S              S in bf16, in shared memory
//   update  (K e^(G_L - G))^T V, M = the state's rows
// Roles: warp 0 loads, warp 1 issues the MMAs, warps 4-7 make P and write the outputs (one
// thread a row), warps 8-15 weigh K and keep the state: 32 fp32 values of a thread.
//
// Roundings.  P and the S that Q meets are rounded to bf16, as an MMA's operands must be; both
// go into an output of bf16.  The state itself is a result in fp32 that later chunks build on,
// so the weighed K is taken as a sum of two bf16 numbers (rest below 2^-16 of it) and the
// update's products accumulate in fp32.  With head_dim 64 the two parts are the two halves of
// an M = 128 MMA, and their states are kept apart until the end.
//
// A cluster of up to 8 CTAs shares a request when there are fewer of them than SMs: each rank
// takes a run of chunks, first makes its run's own update from K and V alone, then the ranks
// pass these on through distributed shared memory, so that each knows the state before its
// run, and then goes through its run for the outputs.
#include <algorithm>

#include "pa_internal.cuh"

namespace pa {

namespace {

constexpr int kC = kLinearChunk;
constexpr int kSlice = 64;   // state columns of a CTA
constexpr int kRows = 128;   // rows of a query tile, and of a state's MMA
constexpr int kThreads = 512;
constexpr int kWarpMma = 1, kFirstOut = 4, kFirstState = 8;
constexpr int kOutWarps = 4, kStateWarps = 8;
constexpr int kRing = 3;     // chunks of K and V in shared memory
constexpr int kQueue = 4;
// Logarithms (base 2) below this are as good as none: what they multiply is 0 in fp32.
constexpr float kLeastLog = -150.f;

template <int D>
struct Geom {
    static constexpr int kHalves = D / 64;
    static constexpr int kQHalf = kRows * 128, kKHalf = kC * 128;
    static constexpr int kQBytes = kHalves * kQHalf;
    static constexpr int kKBytes = kHalves * kKHalf, kVBytes = kKHalf;
    static constexpr int kStageBytes = kKBytes + kVBytes;
    static constexpr int kSBytes = kRows * 128;  // bf16 state: 128 rows x 64 columns
    static constexpr int kOffQ = 0;              // [2]
    static constexpr int kOffKV = kOffQ + 2 * kQBytes;
    static constexpr int kOffKt = kOffKV + kRing * kStageBytes;  // weighed K: first parts, rests
    static constexpr int kOffS = kOffKt + 2 * kKBytes;           // [2]
    static constexpr int kOffBar = kOffS + 2 * kSBytes;
    static constexpr int kOffG = kOffBar + 256;                  // [2][kC] sums of logarithms
    static constexpr int kOffCtl = kOffG + 2 * kC * 4;
    static constexpr int kSmemRaw = kOffCtl + 512 + (kThreads + 1) * 4;
    // one CTA per SM: its TMEM columns are all taken
    static constexpr int kSmemBytes = kSmemRaw > 116 * 1024 ? kSmemRaw : 116 * 1024;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
    static_assert(kOffBar % 1024 == 0, "alignment");
    // TMEM columns: scores [2], outputs (before | inside) [2], update
    static constexpr uint32_t kTmemCols = 512;
    static constexpr int kColO = 2 * kC, kColU = kColO + 2 * 2 * kSlice;
    static_assert(kColU + kSlice <= 512, "TMEM");
};

struct Bars {
    uint64_t kv_full[kRing], kv_empty[kRing];
    uint64_t q_full[2], q_empty[2];
    uint64_t kt_full[2], u_full;       // weighed K of a chunk there / its update done
    uint64_t s_full[2], s_empty[2];    // state before a chunk in shared memory / read
    uint64_t sc_full[2], p_full[2];    // scores of a tile / its P
    uint64_t o_full[2], o_empty[2];
    uint64_t drain;
};
static_assert(sizeof(Bars) <= 256, "barrier area");

// One request, kv head and slice, and this rank's run of chunks.
struct alignas(16) Item {
    int t0, n, h, slice;       // n = 0: no more items
    int c_begin, c_end, chunks;
    int in, to, pad[3];
};
static_assert(sizeof(Item) == 48, "queue entry");

struct Ctl {
    int abort, published, read[kThreads / 32];
    uint32_t tmem;
    int pad;
    Item items[kQueue];
    float decay;  // of this rank's run, log2 (read by the cluster)
};
static_assert(sizeof(Ctl) <= 512, "control area");

// The queue's waits do not look at the abort flag: after a wait of the pipeline has run out every
// warp goes on through the items without their work, so that the barriers of the block and of
// the cluster are met all the same.
constexpr uint64_t kQueueTimeoutNs = 5 * kWaitTimeoutNs;
template <typename Ready>
__device__ __forceinline__ bool spin(volatile int *abort, Ready ready) {
    if (ready()) return true;
    const uint64_t t0 = global_timer_ns();
    while (!ready())
        if (global_timer_ns() - t0 > kQueueTimeoutNs) {
            *abort = 1;
            return false;
        }
    return true;
}

// A request's tokens; 0 for one that the recurrent form has, or that is wrong (flagged there).
__device__ __forceinline__ int long_tokens(const LinearParams &p, int b, int &t0) {
    t0 = __ldg(p.qsl + b);
    const int n = __ldg(p.qsl + b + 1) - t0;
    const bool bad = n < 0 || t0 < 0 || t0 > p.num_tokens - n;
    return bad || n <= p.max_rows ? 0 : n;
}

// The k-th item of this cluster, by all lanes of warp 0: long request number idx / (heads *
// slices), found from the threads' counts of long requests before theirs (count[]).
template <int D>
__device__ Item find_item(const LinearParams &p, const int *count, int k, int rank, int size) {
    const int lane = threadIdx.x & 31;
    const int per = p.num_kv_heads * (D / kSlice);
    const int64_t idx = static_cast<int64_t>(k) * (gridDim.x / size) + blockIdx.x / size;
    const int64_t which = idx / per;
    Item it{};
    if (which >= count[kThreads]) return it;
    const int want = static_cast<int>(which), in = static_cast<int>(idx - which * per);
    // the thread whose requests hold it: count[owner] <= want < count[owner + 1]
    unsigned m = __ballot_sync(0xffffffffu, count[lane * (kThreads / 32)] <= want);
    const int group = (31 - __clz(m)) * (kThreads / 32);
    m = __ballot_sync(0xffffffffu, lane < kThreads / 32 && count[group + lane % (kThreads / 32)] <= want);
    const int owner = group + 31 - __clz(m);
    const int each = (p.num_seqs + kThreads - 1) / kThreads;
    int left = want - count[owner];
    for (int b0 = owner * each;; b0 += 32) {  // (the count says that it is there)
        const int b = b0 + lane;
        int t0 = 0;
        const int n = b < min(p.num_seqs, (owner + 1) * each) ? long_tokens(p, b, t0) : 0;
        const unsigned longs = __ballot_sync(0xffffffffu, n > 0);
        if (left < __popc(longs)) {
            // the lane with `left` long requests before it
            const bool mine = n > 0 && __popc(longs & ((1u << lane) - 1)) == left;
            const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
            it.n = __shfl_sync(0xffffffffu, n, src);
            it.t0 = __shfl_sync(0xffffffffu, t0, src);
            const int found = b0 + src;
            it.in = __ldg(p.state_in + found);
            it.to = __ldg(p.state_out + found);
            break;
        }
        left -= __popc(longs);
        if (b0 + 32 >= p.num_seqs) return it;
    }
    it.h = in / (D / kSlice);
    it.slice = in - it.h * (D / kSlice);
    unsigned flags = 0;
    if (it.in >= p.num_slots) it.in = -1, flags = PA_DEV_BAD_SLOT;
    if (it.to >= p.num_slots) it.to = -1, flags = PA_DEV_BAD_SLOT;
    if (flags && lane == 0) flag_status(p.status, flags);
    it.chunks = (it.n + kC - 1) / kC;
    const int run = (it.chunks + size - 1) / size;
    it.c_begin = min(it.chunks, rank * run);
    it.c_end = min(it.chunks, it.c_begin + run);
    return it;
}

// Any other warp, all lanes: item k.
__device__ __forceinline__ Item queue_item(Ctl *ctl, int warp, int k) {
    const int lane = threadIdx.x & 31;
    volatile int *published = &ctl->published;
    int ok = 1;
    if (lane == 0) ok = spin(&ctl->abort, [&] { return *published > k; }) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    Item it{};
    if (ok) {
        __threadfence_block();
        const volatile int *src = reinterpret_cast<const volatile int *>(ctl->items + k % kQueue);
        int *dst = reinterpret_cast<int *>(&it);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(Item) / sizeof(int)); ++i) dst[i] = src[i];
    }
    __syncwarp();
    if (lane == 0) *reinterpret_cast<volatile int *>(&ctl->read[warp]) = k + 1;
    return it;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    linear_prompt_kernel(const LinearParams p, const __grid_constant__ CUtensorMap tmq,
                         const __grid_constant__ CUtensorMap tmk,
                         const __grid_constant__ CUtensorMap tmv, int size) {
    using G = Geom<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars *bars = reinterpret_cast<Bars *>(smem + G::kOffBar);
    float *s_g = reinterpret_cast<float *>(smem + G::kOffG);
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + G::kOffCtl);
    int *count = reinterpret_cast<int *>(smem + G::kOffCtl + 512);
    volatile int *abort_flag = &ctl->abort;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31, tid = threadIdx.x;
    const int rank = static_cast<int>(blockIdx.x) % size;
    const int tiles = (p.group + p.heads_per_tile - 1) / p.heads_per_tile;

    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&bars->kv_full[i], 1);
            mbar_init(&bars->kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->q_full[i], 1);
            mbar_init(&bars->q_empty[i], 1);
            mbar_init(&bars->kt_full[i], kStateWarps);
            mbar_init(&bars->s_full[i], kStateWarps);
            mbar_init(&bars->s_empty[i], 1);
            mbar_init(&bars->sc_full[i], 1);
            mbar_init(&bars->p_full[i], kOutWarps);
            mbar_init(&bars->o_full[i], 1);
            mbar_init(&bars->o_empty[i], kOutWarps);
        }
        mbar_init(&bars->u_full, 1);
        mbar_init(&bars->drain, 1);
        ctl->abort = 0;
        ctl->published = 0;
        for (int w = 0; w < kThreads / 32; ++w) ctl->read[w] = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    if (warp == kWarpMma) tmem_alloc(&ctl->tmem, G::kTmemCols);
    tc_fence_before();
    pdl_wait();
    pdl_trigger();
    // long requests before each thread's
    {
        const int each = (p.num_seqs + kThreads - 1) / kThreads;
        int longs = 0, t0;
        for (int b = min(p.num_seqs, tid * each); b < min(p.num_seqs, (tid + 1) * each); ++b)
            longs += long_tokens(p, b, t0) > 0;
        int incl = longs;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int before = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += before;
        }
        if (lane == 31) reinterpret_cast<int *>(s_g)[warp] = incl;
        __syncthreads();
        int base = 0;
        for (int w = 0; w < warp; ++w) base += reinterpret_cast<int *>(s_g)[w];
        count[tid + 1] = base + incl;
        if (tid == 0) count[0] = 0;
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem, 0);
    uint8_t *sQ = smem + G::kOffQ, *sKV = smem + G::kOffKV, *sKt = smem + G::kOffKt,
            *sS = smem + G::kOffS;

    if (warp == 0) {
        // ============================ loads ============================
        uint32_t c = 0, t = 0;  // chunks and tiles loaded
        bool ok = true;
        auto load_kv = [&](const Item &it, int i) {
            const int st = c % kRing;
            if (ok && c >= kRing) ok = warp_mbar_wait(&bars->kv_empty[st], (c / kRing - 1) & 1, abort_flag);
            // test hook: stop after the first chunk, as if a wait had run out
            if (p.test_stall && blockIdx.x == 0 && c == 1) ok = false;
            if (!ok) return;
            if (lane == 0) {
                uint8_t *dst = sKV + st * G::kStageBytes;
                mbar_arrive_expect_tx(&bars->kv_full[st], G::kStageBytes);
                for (int hf = 0; hf < G::kHalves; ++hf)
                    tma_load_3d(dst + hf * G::kKHalf, &tmk, hf * 64, it.h, it.t0 + i * kC,
                                &bars->kv_full[st]);
                tma_load_3d(dst + G::kKBytes, &tmv, it.slice * kSlice, it.h, it.t0 + i * kC,
                            &bars->kv_full[st]);
            }
            __syncwarp();
            ++c;
        };
        for (int k = 0;; ++k) {
            Item it = find_item<D>(p, count, k, rank, size);
            if (lane == 0) {
                const bool free = k < kQueue || spin(&ctl->abort, [&] {
                                      for (int w = 1; w < kThreads / 32; ++w)
                                          if (*reinterpret_cast<volatile int *>(&ctl->read[w]) <= k - kQueue)
                                              return false;
                                      return true;
                                  });
                if (free) {
                    ctl->items[k % kQueue] = it;
                    __threadfence_block();
                    *reinterpret_cast<volatile int *>(&ctl->published) = k + 1;
                }
            }
            __syncwarp();
            if (it.n == 0) break;
            if (size > 1) {
                if (it.c_end < it.chunks)
                    for (int i = it.c_begin; ok && i < it.c_end; ++i) load_kv(it, i);
                cluster_sync();
                cluster_sync();
            }
            for (int i = it.c_begin; ok && i < it.c_end; ++i) {
                load_kv(it, i);
                for (int j = 0; ok && j < tiles; ++j, ++t) {
                    const int st = t & 1;
                    if (t >= 2) ok = warp_mbar_wait(&bars->q_empty[st], ((t >> 1) - 1) & 1, abort_flag);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bars->q_full[st],
                                              G::kHalves * kC * p.heads_per_tile * 128);
                        for (int hf = 0; hf < G::kHalves; ++hf)
                            tma_load_3d(sQ + st * G::kQBytes + hf * G::kQHalf, &tmq, hf * 64,
                                        it.h * p.group + j * p.heads_per_tile, it.t0 + i * kC,
                                        &bars->q_full[st]);
                    }
                    __syncwarp();
                }
            }
        }
        if (*abort_flag && lane == 0) {
            // copies in flight land before the CTA exits
            for (uint32_t i = c > kRing ? c - kRing : 0; i < c; ++i)
                mbar_drain(&bars->kv_full[i % kRing], (i / kRing) & 1);
            for (uint32_t i = t > 2 ? t - 2 : 0; i < t; ++i) mbar_drain(&bars->q_full[i & 1], (i >> 1) & 1);
        }
    } else if (warp == kWarpMma) {
        // ============================ MMAs ============================
        constexpr uint32_t idesc_qk = idesc_bf16_f32(kRows, kC, 0);
        constexpr uint32_t idesc_v = idesc_bf16_f32(kRows, kSlice, 1);
        constexpr uint32_t idesc_kv = idesc_bf16_f32(kRows, kSlice, 1, 1);
        const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t k_desc = smem_desc_sw128(smem_u32(sKV), 16, 1024);
        const uint64_t v_desc = smem_desc_sw128(smem_u32(sKV) + G::kKBytes, G::kKHalf, 1024);
        const uint64_t kt_desc = smem_desc_sw128(smem_u32(sKt), G::kKHalf, 1024);
        const uint64_t s_desc = smem_desc_sw128(smem_u32(sS), G::kKHalf, 1024);
        const uint32_t elected = elect_one();
        uint32_t c = 0, u = 0, s = 0, t = 0;  // chunks of the ring, updates, states, tiles
        bool ok = true;
        // (one lane may find a barrier complete and another that the CTA has given up)
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            ok = __all_sync(0xffffffffu, ok && mbar_wait(bar, parity, abort_flag));
            return ok;
        };
        auto update = [&](uint32_t chunk) {
            if (!wait(&bars->kt_full[u & 1], (u >> 1) & 1)) return;
            tc_fence_after();
            const uint32_t st = (chunk % kRing) * (G::kStageBytes >> 4);
            // head_dim 128: first parts, then rests; 64: both at once, as the halves of M
            if (elected) {
#pragma unroll
            for (int part = 0; part < G::kHalves; ++part)
#pragma unroll
                for (int kk = 0; kk < kC / 16; ++kk)
                    tc_mma(tmem + G::kColU,
                           kt_desc + ((part * G::kKBytes + kk * 2048) >> 4),
                           v_desc + st + (kk * 2048 >> 4), idesc_kv, part + kk > 0 ? 1u : 0u);
            tc_commit(&bars->u_full);
            }
            __syncwarp();
            ++u;
        };
        for (int k = 0;; ++k) {
            const Item it = queue_item(ctl, warp, k);
            const int n = __shfl_sync(0xffffffffu, it.n, 0);
            if (n == 0) break;
            const int c_begin = __shfl_sync(0xffffffffu, it.c_begin, 0);
            const int c_end = __shfl_sync(0xffffffffu, it.c_end, 0);
            if (size > 1) {
                if (c_end < __shfl_sync(0xffffffffu, it.chunks, 0))
                    for (int i = c_begin; ok && i < c_end; ++i, ++c) {
                        if (!wait(&bars->kv_full[c % kRing], (c / kRing) & 1)) break;
                        update(c);
                        if (ok && elected) tc_commit(&bars->kv_empty[c % kRing]);
                        __syncwarp();
                    }
                cluster_sync();
                cluster_sync();
            }
            // scores of a tile: the first of a chunk waits for the chunk too
            auto scores = [&](uint32_t chunk, uint32_t tile, bool first) {
                if (first && !wait(&bars->kv_full[chunk % kRing], (chunk / kRing) & 1)) return;
                if (!wait(&bars->q_full[tile & 1], (tile >> 1) & 1)) return;
                tc_fence_after();
                const uint64_t qd = q_desc + (tile & 1) * (G::kQBytes >> 4);
                const uint64_t kd = k_desc + (chunk % kRing) * (G::kStageBytes >> 4);
                if (elected) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc_mma(tmem + (tile & 1) * kC,
                           qd + (kk >> 2) * (G::kQHalf >> 4) + (kk & 3) * 2,
                           kd + (kk >> 2) * (G::kKHalf >> 4) + (kk & 3) * 2, idesc_qk,
                           kk > 0 ? 1u : 0u);
                tc_commit(&bars->sc_full[tile & 1]);
                }
                __syncwarp();
            };
            const int total = (c_end - c_begin) * tiles;
            int j = 0;  // tile of the chunk
            if (ok && total > 0) scores(c, t, true);
            for (int i = 0; ok && i < total; ++i, ++t) {
                if (j == 0) {
                    update(c);
                    if (!ok || !wait(&bars->s_full[s & 1], (s >> 1) & 1)) break;
                }
                if (t >= 2 && !wait(&bars->o_empty[t & 1], ((t >> 1) - 1) & 1)) break;
                tc_fence_after();
                const uint32_t o = tmem + G::kColO + (t & 1) * (2 * kSlice);
                const uint64_t qd = q_desc + (t & 1) * (G::kQBytes >> 4);
                const uint64_t sd = s_desc + (s & 1) * (G::kSBytes >> 4);
                const bool last = j == tiles - 1;
                if (elected) {
#pragma unroll
                for (int kk = 0; kk < kRows / 16; ++kk) {
                    const int qk = kk % (D / 16);
                    tc_mma(o, qd + (qk >> 2) * (G::kQHalf >> 4) + (qk & 3) * 2,
                           sd + (kk * 2048 >> 4), idesc_v, kk > 0 ? 1u : 0u);
                }
                tc_commit(&bars->q_empty[t & 1]);
                if (last) tc_commit(&bars->s_empty[s & 1]);
                }
                __syncwarp();
                if (i + 1 < total) scores(last ? c + 1 : c, t + 1, last);
                if (!ok || !wait(&bars->p_full[t & 1], (t >> 1) & 1)) break;
                tc_fence_after();
                const uint64_t vd = v_desc + (c % kRing) * (G::kStageBytes >> 4);
                if (elected) {
#pragma unroll
                for (int kk = 0; kk < kC / 16; ++kk)
                    tc_mma_ts(o + kSlice, tmem + (t & 1) * kC + kk * 8,
                           vd + (kk * 2048 >> 4), idesc_v, kk > 0 ? 1u : 0u);
                tc_commit(&bars->o_full[t & 1]);
                if (last) tc_commit(&bars->kv_empty[c % kRing]);
                }
                __syncwarp();
                j = last ? 0 : j + 1;
                if (last) {
                    ++c;
                    ++s;
                }
            }
        }
        if (__any_sync(0xffffffffu, !ok || *abort_flag)) {
            // MMAs already issued finish before TMEM is released
            if (elected) tc_commit(&bars->drain);
            __syncwarp();
            mbar_drain(&bars->drain, 0);
        }
    } else if (warp >= kFirstOut && warp < kFirstOut + kOutWarps) {
        // ============================ P and outputs ============================
        const int wq = warp & 3, r = wq * 32 + lane;
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const int tok = r / p.heads_per_tile, head = r - tok * p.heads_per_tile;
        uint32_t t = 0, u = 0;  // tiles, updates seen
        bool ok = true;
        for (int k = 0;; ++k) {
            const Item it = queue_item(ctl, warp, k);
            if (it.n == 0) break;
            if (size > 1) {
                if (it.c_end < it.chunks) u += it.c_end - it.c_begin;
                cluster_sync();
                cluster_sync();
            }
            const int total = (it.c_end - it.c_begin) * tiles;
            float grow = 0.f, grow_before = 0.f;  // e^(G_i) of this tile's row, and the last one's
            int i = it.c_begin, j = 0, i_before = 0, j_before = 0;
            for (int m = 0; ok && m <= total; ++m) {
                if (m < total) {
                    const uint32_t tt = t + m;
                    // (the chunk's sums of logarithms are there with its weighed K)
                    if (j == 0) {
                        ok = warp_mbar_wait_spin(&bars->kt_full[u & 1], (u >> 1) & 1, abort_flag);
                        ++u;
                    }
                    ok = ok && warp_mbar_wait_spin(&bars->sc_full[tt & 1], (tt >> 1) & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const float *g = s_g + ((u - 1) & 1) * kC;
                    const float gi = tok < kC ? g[tok] : 0.f;
                    const uint32_t sa = t_lane + (tt & 1) * kC;
                    uint32_t s0[32], s1[32], pk[32];
                    tmem_ld32(sa, s0);
                    tmem_ld32(sa + 32, s1);
                    tmem_wait_ld();
                    auto weigh = [&](const uint32_t (&sv)[32], int at, uint32_t *dst) {
#pragma unroll
                        for (int x = 0; x < 32; x += 4) {
                            const float4 gj = *reinterpret_cast<const float4 *>(g + at + x);
                            const float e0 = fast_exp2(gi - gj.x), e1 = fast_exp2(gi - gj.y),
                                        e2 = fast_exp2(gi - gj.z), e3 = fast_exp2(gi - gj.w);
                            const int lim = tok - at - x;  // last visible token of the four
                            const float a = lim >= 0 ? __uint_as_float(sv[x]) * e0 : 0.f;
                            const float b = lim >= 1 ? __uint_as_float(sv[x + 1]) * e1 : 0.f;
                            const float c = lim >= 2 ? __uint_as_float(sv[x + 2]) * e2 : 0.f;
                            const float d = lim >= 3 ? __uint_as_float(sv[x + 3]) * e3 : 0.f;
                            dst[x / 2] = pack_bf16x2(a, b);
                            dst[x / 2 + 1] = pack_bf16x2(c, d);
                        }
                    };
                    weigh(s0, 0, pk);
                    weigh(s1, 32, pk + 16);
                    tmem_st32(sa, pk);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->p_full[tt & 1]);
                    grow_before = grow;
                    grow = fast_exp2(gi);
                }
                if (m > 0) {
                    const uint32_t tt = t + m - 1;
                    ok = warp_mbar_wait_spin(&bars->o_full[tt & 1], (tt >> 1) & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const float before = (m < total ? grow_before : grow) * p.scale;
                    const int token = i_before * kC + tok, hq = j_before * p.heads_per_tile + head;
                    const bool valid = tok < kC && token < it.n && hq < p.group;
                    uint4 *dst = reinterpret_cast<uint4 *>(
                        p.out + (static_cast<int64_t>(it.t0 + token) * p.num_q_heads +
                                 it.h * p.group + hq) * D + it.slice * kSlice);
                    const uint32_t oa = t_lane + G::kColO + (tt & 1) * (2 * kSlice);
#pragma unroll
                    for (int half = 0; half < kSlice / 32; ++half) {
                        uint32_t a[32], b[32];
                        __syncwarp();
                        tmem_ld32(oa + half * 32, a);
                        tmem_ld32(oa + kSlice + half * 32, b);
                        tmem_wait_ld();
                        if (half == kSlice / 32 - 1) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bars->o_empty[tt & 1]);
                        }
                        if (!valid) continue;
                        auto sum = [&](int x) {
                            return pack_bf16x2(
                                fmaf(before, __uint_as_float(a[x]), p.scale * __uint_as_float(b[x])),
                                fmaf(before, __uint_as_float(a[x + 1]),
                                     p.scale * __uint_as_float(b[x + 1])));
                        };
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            dst[half * 4 + x] = make_uint4(sum(x * 8), sum(x * 8 + 2), sum(x * 8 + 4),
                                                           sum(x * 8 + 6));
                    }
                    __syncwarp();
                }
                i_before = i;
                j_before = j;
                if (++j == tiles) j = 0, ++i;
            }
            t += total;
        }
    } else if (warp >= kFirstState) {
        // ============================ K's weights, the state ============================
        const int sw = warp - kFirstState, wq = warp & 3, half = sw >> 2;
        const int r = wq * 32 + lane;       // row of the update's MMA, 32 of its columns
        const int dk = D == 128 ? r : r % 64;
        const bool rest = D == 64 && r >= 64;  // the state of the rests of K
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        float s[32];
        uint32_t c = 0, u = 0, w = 0;  // chunks of the ring, updates, states written
        bool ok = true;
        float total = 0.f;  // log2 decay of the chunks gone through

        // the state in bf16, for the MMA that follows
        auto give_state = [&]() {
            if (ok && w >= 2) ok = warp_mbar_wait_spin(&bars->s_empty[w & 1], ((w >> 1) - 1) & 1, abort_flag);
            if (!ok) return;
            uint8_t *dst = sS + (w & 1) * G::kSBytes;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *reinterpret_cast<uint4 *>(dst + sw128_offset(r, half * 4 + x)) = make_uint4(
                    pack_bf16x2(s[8 * x], s[8 * x + 1]), pack_bf16x2(s[8 * x + 2], s[8 * x + 3]),
                    pack_bf16x2(s[8 * x + 4], s[8 * x + 5]), pack_bf16x2(s[8 * x + 6], s[8 * x + 7]));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->s_full[w & 1]);
            ++w;
        };
        // logarithm (base 2) of the decay of token i of the request
        auto log_of = [&](const Item &it, int i) {
            if (i >= it.n) return 0.f;
            const float g = __ldg(p.decay + static_cast<int64_t>(it.t0 + i) * p.decay_stride + it.h);
            return g < 0.f ? fmaxf(g * 1.4426950408889634f, kLeastLog) : 0.f;
        };
        // One chunk: weighs K, then takes the update in.  g0, g1: the logarithms of tokens
        // 2 lane and 2 lane + 1, and the next chunk's afterwards.
        auto chunk = [&](const Item &it, int i, float &g0, float &g1, bool more) {
            // sums up to each token, and of those behind it (each without a difference, so
            // that a small one keeps its digits beside large ones)
            float up = g0 + g1, down = up;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float a = __shfl_up_sync(0xffffffffu, up, o);
                const float b = __shfl_down_sync(0xffffffffu, down, o);
                if (lane >= o) up += a;
                if (lane + o < 32) down += b;
            }
            const float all = __shfl_sync(0xffffffffu, up, 31);
            float up0 = __shfl_up_sync(0xffffffffu, up, 1), down1 = __shfl_down_sync(0xffffffffu, down, 1);
            if (lane == 0) up0 = 0.f;
            if (lane == 31) down1 = 0.f;
            up0 += g0;
            const float w0 = exp2f(down1 + g1), w1 = exp2f(down1);
            if (p.decay_stride == 0 && (i + 1) * kC <= it.n) {
                // (one logarithm for all: exact multiples)
                up0 = (2 * lane + 1) * g0;
                up = (2 * lane + 2) * g0;
            }
            if (sw == 0)
                *reinterpret_cast<float2 *>(s_g + (u & 1) * kC + 2 * lane) = make_float2(up0, up);
            const float keep = exp2f(all);
            total += all;
            const int at = (i + 1) * kC + 2 * lane;
            if (more) {
                g0 = log_of(it, at);
                g1 = log_of(it, at + 1);
            }
            const int st = c % kRing;
            ok = ok && warp_mbar_wait_spin(&bars->kv_full[st], (c / kRing) & 1, abort_flag);
            if (!ok) return;
            const uint8_t *k = sKV + st * G::kStageBytes;
            const int valid = min(kC, it.n - i * kC);
            // eight lanes to a row of 64 elements
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int row = sw * 8 + x * 4 + lane / 8;
                const int src = row >> 1;  // the lane that has its weight
                const float wa = __shfl_sync(0xffffffffu, w0, src), wb = __shfl_sync(0xffffffffu, w1, src);
                const float wt = row & 1 ? wb : wa;
#pragma unroll
                for (int hf = 0; hf < G::kHalves; ++hf) {
                    const uint32_t off = hf * G::kKHalf + sw128_offset(row, lane % 8);
                    const uint4 in = *reinterpret_cast<const uint4 *>(k + off);
                    uint4 a = make_uint4(0, 0, 0, 0), b = a;
                    auto part = [&](uint32_t pair, uint32_t &first, uint32_t &more_) {
                        const float lo = __uint_as_float(pair << 16) * wt;
                        const float hi = __uint_as_float(pair & 0xFFFF0000u) * wt;
                        first = pack_bf16x2(lo, hi);
                        more_ = pack_bf16x2(lo - __uint_as_float(first << 16),
                                            hi - __uint_as_float(first & 0xFFFF0000u));
                    };
                    if (row < valid) {
                        part(in.x, a.x, b.x);
                        part(in.y, a.y, b.y);
                        part(in.z, a.z, b.z);
                        part(in.w, a.w, b.w);
                    }
                    *reinterpret_cast<uint4 *>(sKt + off) = a;
                    *reinterpret_cast<uint4 *>(sKt + G::kKBytes + off) = b;
                }
                // rows behind the request are another's, or padding: whatever stands there,
                // it does not reach a sum
                if (row >= valid)
                    *reinterpret_cast<uint4 *>(sKV + st * G::kStageBytes + G::kKBytes +
                                               sw128_offset(row, lane % 8)) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->kt_full[u & 1]);
            ++c;
            ok = warp_mbar_wait_spin(&bars->u_full, u & 1, abort_flag);
            ++u;
            if (!ok) return;
            tc_fence_after();
            uint32_t up_[32];
            tmem_ld32(t_lane + G::kColU + half * 32, up_);
            tmem_wait_ld();
            tc_fence_before();
#pragma unroll
            for (int x = 0; x < 32; ++x) s[x] = fmaf(keep, s[x], __uint_as_float(up_[x]));
        };
        for (int k = 0;; ++k) {
            const Item it = queue_item(ctl, warp, k);
            if (it.n == 0) break;
            const int64_t place = static_cast<int64_t>(it.h) * D * D + static_cast<int64_t>(dk) * D +
                                  it.slice * kSlice + half * 32;
            const int64_t state_size = static_cast<int64_t>(p.num_kv_heads) * D * D;
            const int at0 = it.c_begin * kC + 2 * lane;
            float g0, g1;
            if (size > 1) {
                total = 0.f;
#pragma unroll
                for (int x = 0; x < 32; ++x) s[x] = 0.f;
                if (it.c_end < it.chunks) {
                    g0 = log_of(it, at0);
                    g1 = log_of(it, at0 + 1);
                    for (int i = it.c_begin; ok && i < it.c_end; ++i)
                        chunk(it, i, g0, g1, i + 1 < it.c_end);
                    // (the MMAs of the item before have read both states)
                    for (int x = 0; ok && x < 2; ++x)
                        if (w > static_cast<uint32_t>(x)) {
                            const uint32_t last = w - 1 - x;
                            ok = warp_mbar_wait_spin(&bars->s_empty[last & 1], (last >> 1) & 1, abort_flag);
                        }
                    float *mine = reinterpret_cast<float *>(sS) + (half * 32) * kRows + r;
#pragma unroll
                    for (int x = 0; x < 32; ++x) mine[x * kRows] = s[x];
                    if (sw == 0 && lane == 0) ctl->decay = total;
                }
                cluster_sync();
            }
            g0 = log_of(it, at0);
            g1 = log_of(it, at0 + 1);
            const float4 *src = reinterpret_cast<const float4 *>(p.state + it.in * state_size + place);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const float4 v = it.in >= 0 && !rest ? src[x] : make_float4(0.f, 0.f, 0.f, 0.f);
                s[4 * x] = v.x;
                s[4 * x + 1] = v.y;
                s[4 * x + 2] = v.z;
                s[4 * x + 3] = v.w;
            }
            if (size > 1) {
                if (it.c_begin < it.c_end)
                    for (int other = 0; other < rank; ++other) {
                        const float keep = exp2f(ld_cluster_f1(&ctl->decay, other));
                        const float *theirs = reinterpret_cast<float *>(sS) + (half * 32) * kRows + r;
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            s[x] = fmaf(keep, s[x], ld_cluster_f1(theirs + x * kRows, other));
                    }
                cluster_sync();
            }
            if (it.c_begin < it.c_end) give_state();
            for (int i = it.c_begin; ok && i < it.c_end; ++i) {
                chunk(it, i, g0, g1, i + 1 < it.c_end);
                if (i + 1 < it.c_end) give_state();
            }
            if (D == 64) {
                // the rests' state joins the first parts'
                float *other = reinterpret_cast<float *>(sKt) + (half * 32) * 64 + dk;
                named_bar_sync(1, 32 * kStateWarps);
                if (rest)
#pragma unroll
                    for (int x = 0; x < 32; ++x) other[x * 64] = s[x];
                named_bar_sync(1, 32 * kStateWarps);
                if (!rest)
#pragma unroll
                    for (int x = 0; x < 32; ++x) s[x] += other[x * 64];
                named_bar_sync(1, 32 * kStateWarps);
            }
            if (ok && !rest && it.to >= 0 && it.c_begin < it.c_end && it.c_end == it.chunks) {
                float4 *dst = reinterpret_cast<float4 *>(p.state + it.to * state_size + place);
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    dst[x] = make_float4(s[4 * x], s[4 * x + 1], s[4 * x + 2], s[4 * x + 3]);
            }
        }
    } else if (size > 1) {
        // (warps without a part in it: the cluster's barriers take every thread)
        for (int k = 0;; ++k) {
            if (queue_item(ctl, warp, k).n == 0) break;
            cluster_sync();
            cluster_sync();
        }
    } else {
        for (int k = 0; queue_item(ctl, warp, k).n != 0; ++k) {}
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*abort_flag && tid == 0) flag_status(p.status, PA_DEV_WAIT_TIMEOUT);
    if (warp == kWarpMma) tmem_dealloc(tmem, G::kTmemCols);
}

namespace {

template <int D>
int launch(const LinearParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
           const CUtensorMap &tv, int sms, cudaStream_t s) {
    static PerDeviceOnce once;
    if (once_per_device(once, [] {
            return cudaFuncSetAttribute(linear_prompt_kernel<D>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        Geom<D>::kSmemBytes);
        }) != PA_OK)
        return PA_ERR_CUDA;
    // the most requests that can be long, and their items
    const int64_t longs = std::min<int64_t>(p.num_seqs, p.num_tokens / (p.max_rows + 1));
    const int64_t items = longs * p.num_kv_heads * (D / kSlice);
    if (items == 0) return PA_OK;
    int size = 1;
    while (size < kDirectMaxCluster && 2 * size * items <= sms && 2 * size * 2 * kC <= p.num_tokens)
        size *= 2;
    const int clusters = static_cast<int>(std::min<int64_t>(items, sms / size));
    PdlLaunch l(clusters * size, kThreads, Geom<D>::kSmemBytes, s);
    if (size > 1) l.set_cluster(size);
    return launch_kernel(l, linear_prompt_kernel<D>, p, tq, tk, tv, size) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace

int launch_linear_prompt(const LinearParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                         const CUtensorMap &tv, int head_dim, int sms, cudaStream_t s) {
    return head_dim == 128 ? launch<128>(p, tq, tk, tv, sms, s) : launch<64>(p, tq, tk, tv, sms, s);
}

}  // namespace pa
