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
//    so one group's waits lie beside the other's arithmetic;
//  * S is a ring of three TMEM tiles and P overwrites the S tile it came from,
//    so the scores of up to two later tiles are ready when a group wants one;
//  * both groups share one accumulator O, so they must agree on each row's
//    reference (the running maximum its exponents are taken against).  A tile's
//    reference is the tile before's unless the tile's maximum exceeds it by
//    2^8 (then O is rescaled), and is handed from tile to tile through shared
//    memory as soon as the tile's maximum is known, long before its P is.
//    Sums are kept per group, each against the reference it last used, and
//    added at the item's end.
// Shared memory traffic is what bounds it then: Q and K tiles read by Q K^T,
// V by P V, both written by TMA, 160 KB per key tile at 128 B a cycle = 1280
// cycles.
#include "pa_long.cuh"

namespace pa {

namespace {

// warps: 0 K (+Q) loads, 1 Q K^T issuer (+TMEM allocation), 2 V loads, 3 P V
// issuer, 4-7 softmax of even tiles, 8-11 of odd ones
constexpr int kWarpQK = 1, kWarpV = 2, kWarpPV = 3, kFirstSoftmax = 4;
constexpr int kGroupWarps = 4;
constexpr int kSTiles = 3;

template <int D>
struct WinGeom : LongTiles<D> {
    using T = LongTiles<D>;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + T::kQBytes;
    static constexpr int kOffV = kOffK + kKStages * T::kKVBytes;
    static constexpr int kOffBar = kOffV + kVStages * T::kKVBytes;
    static constexpr int kOffCtl = kOffBar + 384;
    // per row: references by tile parity [2][128], sums [item parity][group][128]
    static constexpr int kOffRef = kOffCtl + 128;
    static constexpr int kOffSum = kOffRef + 2 * 128 * 4;
    static constexpr int kOffQueue = kOffSum + 2 * 2 * 128 * 4;
    static constexpr int kSmemRaw = kOffQueue + 512 + 1024;
    // at least 116 KiB so that one CTA owns an SM (and its 512 TMEM columns)
    static constexpr int kSmemBytes = kSmemRaw > 116 * 1024 ? kSmemRaw : 116 * 1024;
    // TMEM columns: S0 | S1 | S2 (fp32, P in the first half of each) | O (fp32)
    static constexpr uint32_t kTmemCols = 512;
    static constexpr int kColO = kSTiles * kLongKeys;
    static_assert(kColO + D <= 512, "TMEM");
};

struct Bars {
    uint64_t q_full, q_empty;
    uint64_t k_full[kKStages], k_empty[kKStages];
    uint64_t v_full[kVStages], v_empty[kVStages];
    uint64_t s_full[kSTiles];   // scores of a tile written
    uint64_t p_full[kSTiles];   // P of a tile written (4 warps)
    uint64_t pv_done[kSTiles];  // P V of a tile finished: its S tile is free
    uint64_t ref[4][2];         // reference of a tile published, by row quarter and tile parity
    uint64_t sums[4];           // both groups' sums of an item written, by row quarter
    uint64_t o_free, drain, drain_pv;
};
static_assert(sizeof(Bars) <= 384, "barrier area");

}  // namespace

template <int D>
__global__ void __launch_bounds__(32 * kLongWarps, 1)
    long_window_kernel(const LongParams p, const __grid_constant__ CUtensorMap tmq,
                       const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv) {
    using G = WinGeom<D>;
    constexpr int KS = D / 16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Bars *bars = reinterpret_cast<Bars *>(smem + G::kOffBar);
    int *ctl = reinterpret_cast<int *>(smem + G::kOffCtl);
    volatile int *abort_flag = ctl;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ctl + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (p.wait_start) {
        pdl_wait();     // the plan (and any staging copy) first
        pdl_trigger();  // then the split-KV grid may take the other SMs
    }
    const int n_items = num_items(p);
    if (!p.dynamic && static_cast<int>(blockIdx.x) >= n_items) {
        pdl_wait();  // complete only after the grid this one overlaps
        return;
    }
    int *qmem = reinterpret_cast<int *>(smem + G::kOffQueue);
    Sched sched;
    sched.idx = qmem;
    sched.pub = qmem + kItemQueue;
    sched.cons = qmem + kItemQueue + 1;

    // ---- setup ----------------------------------------------------------------
    if (threadIdx.x == 0) {
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_empty, 1);
        for (int i = 0; i < kKStages; ++i) {
            mbar_init(&bars->k_full[i], 1);
            mbar_init(&bars->k_empty[i], 1);
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(&bars->v_full[i], 1);
            mbar_init(&bars->v_empty[i], 1);
        }
        for (int i = 0; i < kSTiles; ++i) {
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_full[i], kGroupWarps);
            mbar_init(&bars->pv_done[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars->ref[i][0], 1);
            mbar_init(&bars->ref[i][1], 1);
            mbar_init(&bars->sums[i], 2);
        }
        mbar_init(&bars->o_free, 2 * kGroupWarps);
        mbar_init(&bars->drain, 1);
        mbar_init(&bars->drain_pv, 1);
        ctl[0] = 0;
        *sched.pub = 0;
        for (int w = 0; w < kLongWarps; ++w) sched.cons[w] = 0;
        fence_mbar_init();
    }
    if (warp == kWarpQK) tmem_alloc(tmem_slot, G::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    uint8_t *sQ = smem + G::kOffQ;
    uint8_t *sK = smem + G::kOffK;
    uint8_t *sV = smem + G::kOffV;

    if (warp == 0) {
        // ============================ K (and Q) loads ============================
        if (lane == 0) {
            tma_prefetch_desc(&tmq);
            tma_prefetch_desc(&tmk);
        }
        produce<D, kKStages, true>(p, sched, &tmk, sK, bars->k_full, bars->k_empty, &bars->q_full,
                                   &bars->q_empty, true, &tmq, sQ, abort_flag);
    } else if (warp == kWarpV) {
        // ============================ V loads ============================
        if (lane == 0) tma_prefetch_desc(&tmv);
        produce<D, kVStages, true>(p, sched, &tmv, sV, bars->v_full, bars->v_empty, nullptr, nullptr,
                                   false, nullptr, nullptr, abort_flag);
    } else if (warp == kWarpQK) {
        // ============================ Q K^T issuer ============================
        // A tile's scores wait for its K tile and for the P V three tiles back,
        // which read P from the same S tile.
        if (lane == 0) {
            constexpr uint32_t idesc_qk = idesc_bf16_f32(kLongRows, kLongKeys, 0);
            const uint32_t q_addr = smem_u32(sQ), k_addr = smem_u32(sK);
            uint32_t t = 0, k_item = 0;
            bool ok = true;
            for (int round = 0; ok; ++round) {
                const int idx = sched_take(p, sched, n_items, round, warp, abort_flag);
                if (idx == kSchedDone) break;
                if (idx == kSchedAbort) {
                    ok = false;
                    break;
                }
                const Item it = decode_item<true>(p, idx);
                if (it.nt == 0) continue;
                if (!mbar_wait(&bars->q_full, k_item & 1, abort_flag)) { ok = false; break; }
                int j = 0;
                for (; j < it.nt; ++j) {
                    const uint32_t tt = t + j;
                    const int ks = tt % kKStages;
                    const int sb = tt % kSTiles;
                    if (!mbar_wait(&bars->k_full[ks], (tt / kKStages) & 1, abort_flag)) { ok = false; break; }
                    if (tt >= kSTiles &&
                        !mbar_wait(&bars->pv_done[sb], (tt / kSTiles - 1) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t kb = k_addr + ks * G::kKVBytes;
#pragma unroll
                    for (int kk = 0; kk < KS; ++kk) {
                        const uint64_t ad = smem_desc_sw128(
                            q_addr + (kk >> 2) * G::kHalfBytes + (kk & 3) * 32, 16, 1024);
                        const uint64_t bd = smem_desc_sw128(
                            kb + (kk >> 2) * G::kHalfBytes + (kk & 3) * 32, 16, 1024);
                        tc_mma(tmem + sb * kLongKeys, ad, bd, idesc_qk, kk > 0 ? 1u : 0u);
                    }
                    tc_commit(&bars->k_empty[ks]);
                    tc_commit(&bars->s_full[sb]);
                    if (j == it.nt - 1) tc_commit(&bars->q_empty);
                }
                if (p.tile_counter) atomicAdd(p.tile_counter, static_cast<unsigned long long>(j));
                t += it.nt;
                ++k_item;
            }
            if (!ok) {
                // let every MMA already issued finish before TMEM is released
                tc_commit(&bars->drain);
                mbar_drain(&bars->drain, 0);
            }
        }
    } else if (warp == kWarpPV) {
        // ============================ P V issuer ============================
        // A tile's P V waits for its P, its V tile and, at the start of an item,
        // for the previous item's epilogue to read O.
        if (lane == 0) {
            constexpr uint32_t idesc_pv = idesc_bf16_f32(kLongRows, D, 1);
            const uint32_t v_addr = smem_u32(sV);
            uint32_t t = 0, k_item = 0;
            bool ok = true;
            for (int round = 0; ok; ++round) {
                const int idx = sched_take(p, sched, n_items, round, warp, abort_flag);
                if (idx == kSchedDone) break;
                if (idx == kSchedAbort) {
                    ok = false;
                    break;
                }
                const Item it = decode_item<true>(p, idx);
                if (it.nt == 0) continue;
                for (int j = 0; j < it.nt; ++j) {
                    const uint32_t tt = t + j;
                    const int sb = tt % kSTiles;
                    if (!mbar_wait(&bars->p_full[sb], (tt / kSTiles) & 1, abort_flag)) { ok = false; break; }
                    if (j == 0 && k_item > 0 &&
                        !mbar_wait(&bars->o_free, (k_item - 1) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const int vs = tt % kVStages;
                    if (!mbar_wait(&bars->v_full[vs], (tt / kVStages) & 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t vbase = v_addr + vs * G::kKVBytes;
                    // P (bf16) of this tile: row r in TMEM lane r, key k in column k / 2
                    const uint32_t pcol = tmem + sb * kLongKeys;
#pragma unroll
                    for (int kk = 0; kk < kLongKeys / 16; ++kk) {
                        const uint64_t bd = smem_desc_sw128(vbase + kk * 2048, G::kHalfBytes, 1024);
                        tc_mma_ts(tmem + G::kColO, pcol + kk * 8, bd, idesc_pv,
                                  (j > 0 || kk > 0) ? 1u : 0u);
                    }
                    tc_commit(&bars->v_empty[vs]);
                    tc_commit(&bars->pv_done[sb]);
                }
                t += it.nt;
                ++k_item;
            }
            if (!ok) {
                tc_commit(&bars->drain_pv);
                mbar_drain(&bars->drain_pv, 0);
            }
        }
    } else {
        // ============================ softmax + epilogue ============================
        const int wq = warp & 3;  // TMEM lane quarter of this warp
        const int grp = (warp - kFirstSoftmax) / kGroupWarps;
        const int r = wq * 32 + lane;
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const int ttok = r / p.group;
        const int jh = r - ttok * p.group;
        float *refs = reinterpret_cast<float *>(smem + G::kOffRef) + r;  // [parity * 128]
        float *sums = reinterpret_cast<float *>(smem + G::kOffSum) + r;  // [(parity * 2 + grp) * 128]
        uint32_t t = 0, k_item = 0;
        bool ok = true;
        for (int round = 0; ok; ++round) {
            int idx = 0;
            if (lane == 0) idx = sched_take(p, sched, n_items, round, warp, abort_flag);
            idx = __shfl_sync(0xffffffffu, idx, 0);
            if (idx == kSchedDone) break;
            if (idx == kSchedAbort) {
                ok = false;
                break;
            }
            const Item it = decode_item<true>(p, idx);
            if (it.nt == 0) continue;
            const bool row_valid = ttok < it.nvalid && r < p.q_tile_tokens * p.group;
            // (packed keys) this row's last key, and the first row's lowest key
            // behind the sinks
            const int row_limit = it.pos0 + ttok;
            const int low_first = it.pos0 - p.win.window + 1;
            // scores in log2 units; an fp8 pool's K scale folds in here
            const float sl2 = p.k_scale ? p.scale_log2 * __ldg(p.k_scale + it.h) : p.scale_log2;
            float ref = -INFINITY, l = 0.f;  // this group's sum, against `ref`
            for (int j = (t & 1) == static_cast<uint32_t>(grp) ? 0 : 1; j < it.nt; j += 2) {
                const uint32_t tt = t + j;
                const int sb = tt % kSTiles;
                const int kb = j * kLongKeys;
                // keys kb + i visible to this row, bit i: below the causal
                // limit, and a sink or at or past the row's low.  Only tiles
                // that hold a key some row does not see are masked.
                const bool need_mask = kb + kLongKeys - 1 > it.pos0 || kb + kLongKeys > it.key_end ||
                                       (kb < low_first + it.nvalid - 1 &&
                                        kb + kLongKeys > p.win.sinks);
                auto seen_from = [&](int at) {
                    return low_bits(min(row_limit, it.key_end - 1) + 1 - at) &
                           (low_bits(p.win.sinks - at) |
                            ~low_bits(row_limit - p.win.window + 1 - at));
                };
                if (!warp_wait(&bars->s_full[sb], (tt / kSTiles) & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                const uint32_t sa = t_lane + sb * kLongKeys;
                // the row's maximum: keys 64..127 first, keys 0..63 stay in registers
                uint32_t s0[32], s1[32];
                float mx = -INFINITY;
                auto mask = [&](uint64_t seen) {
                    const uint32_t lo = static_cast<uint32_t>(seen);
                    const uint32_t hi = static_cast<uint32_t>(seen >> 32);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (!(lo & (1u << i))) s0[i] = __float_as_uint(-INFINITY);
                        if (!(hi & (1u << i))) s1[i] = __float_as_uint(-INFINITY);
                    }
                };
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
                if (need_mask) mask(seen_from(kb + 64));
                row_max();
                tmem_ld32(sa, s0);
                tmem_ld32(sa + 32, s1);
                tmem_wait_ld();
                if (need_mask) mask(seen_from(kb));
                row_max();
                // the reference: the tile before's, unless this tile exceeds it
                float before = -INFINITY;
                if (tt > 0) {
                    if (!warp_wait(&bars->ref[wq][(tt - 1) & 1], ((tt - 1) >> 1) & 1, abort_flag)) { ok = false; break; }
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
                // P row r (bf16 pairs) over the S tile's first 64 columns: 32
                // keys take 16 columns, so a piece only covers scores read before
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
                exps(s0, sa);
                exps(s1, sa + 16);
                tmem_ld32(sa + 64, s0);
                tmem_ld32(sa + 96, s1);
                tmem_wait_ld();
                if (need_mask) mask(seen_from(kb + 64));
                exps(s0, sa + 32);
                exps(s1, sa + 48);
                float sum0, sum1, sum2, sum3;
                f2_unpack(acc0, sum0, sum1);
                f2_unpack(acc1, sum2, sum3);
                l += (sum0 + sum1) + (sum2 + sum3);
                // O is rescaled in place where the reference moved: the previous
                // tile's P V must be done, this tile's has not begun
                const float alpha = up && before != -INFINITY ? fast_exp2(before - now) : 1.f;
                if (j >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    const uint32_t prev = tt - 1;
                    if (!warp_wait(&bars->pv_done[prev % kSTiles], (prev / kSTiles) & 1, abort_flag)) { ok = false; break; }
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
                    const int vs = tt % kVStages;
                    if (!warp_wait(&bars->v_full[vs], (tt / kVStages) & 1, abort_flag)) return false;
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
                tmem_wait_st();
                if (zeroed) fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->p_full[sb]);
            }

            // ---- epilogue: this group's half of the output columns ----
            const uint32_t last = t + it.nt - 1;
            float final_ref = -INFINITY;
            if (ok) ok = warp_wait(&bars->ref[wq][last & 1], (last >> 1) & 1, abort_flag);
            if (ok) {
                final_ref = *reinterpret_cast<volatile float *>(refs + (last & 1) * 128);
                if (ref != final_ref) l = ref == -INFINITY ? 0.f : l * fast_exp2(ref - final_ref);
                float *slot = sums + (k_item & 1) * 256;
                *reinterpret_cast<volatile float *>(slot + grp * 128) = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->sums[wq]);
                ok = warp_wait(&bars->sums[wq], k_item & 1, abort_flag);
                if (ok) l += *reinterpret_cast<volatile float *>(slot + (1 - grp) * 128);
            }
            if (ok) ok = warp_wait(&bars->pv_done[last % kSTiles], (last / kSTiles) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            // an fp8 pool's V scale multiplies the output
            const float vsc = p.v_scale ? __ldg(p.v_scale + it.h) : 1.f;
            const float inv = l > 0.f ? vsc / l : 0.f;
            const int64_t orow = static_cast<int64_t>(it.tok0 + ttok) * p.num_q_heads +
                                 it.h * p.group + jh;
#pragma unroll
            for (int qd = 0; qd < D / 64; ++qd) {
                const int col = grp * (D / 2) + qd * 32;
                uint32_t raw[32];
                tmem_ld32(t_lane + G::kColO + col, raw);
                tmem_wait_ld();
                if (!row_valid) continue;
                uint4 *dst = reinterpret_cast<uint4 *>(p.out + orow * D + col);
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) {
                    uint4 w;
                    w.x = pack_bf16x2(__uint_as_float(raw[v4 * 8 + 0]) * inv, __uint_as_float(raw[v4 * 8 + 1]) * inv);
                    w.y = pack_bf16x2(__uint_as_float(raw[v4 * 8 + 2]) * inv, __uint_as_float(raw[v4 * 8 + 3]) * inv);
                    w.z = pack_bf16x2(__uint_as_float(raw[v4 * 8 + 4]) * inv, __uint_as_float(raw[v4 * 8 + 5]) * inv);
                    w.w = pack_bf16x2(__uint_as_float(raw[v4 * 8 + 6]) * inv, __uint_as_float(raw[v4 * 8 + 7]) * inv);
                    dst[v4] = w;
                }
            }
            // O has been read: the next item's first P V may overwrite it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->o_free);
            if (row_valid && grp == 0 && p.lse)
                p.lse[orow] = l > 0.f ? (final_ref + __log2f(l)) * kLn2 : -INFINITY;
            t += it.nt;
            ++k_item;
        }
    }

    if (*abort_flag && threadIdx.x == 0) flag_status(p.status, PA_DEV_WAIT_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
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
