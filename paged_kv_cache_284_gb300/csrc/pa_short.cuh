// pa_short.cuh -- the arithmetic of the memory-bound attention kernels on one
// 16-key chunk of K and V in shared memory, shared by the split-KV kernel
// (pa_short.cu) and the one-kernel windowed step (pa_window.cu).
#pragma once

#include "pa_internal.cuh"

namespace pa {

namespace {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: lazy max update
constexpr int kFoldBatch = 8;              // splits loaded together by the fold
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// Keep the lower / upper bf16 of a packed pair.
__device__ __forceinline__ uint32_t keep_pair(uint32_t v, bool lo, bool hi) {
    return (lo ? (v & 0xFFFFu) : 0u) | (hi ? (v & 0xFFFF0000u) : 0u);
}

template <int D>
struct Consumer {
    static constexpr int NT = D / 8;   // 8-wide output column tiles
    static constexpr int KS = D / 16;  // 16-deep k steps over the head dim

    // item-wide
    int b, h, tok0, ctx, key_end, R, KQ, rt, kq, nsplit, split, partial_base, counter;
    float sl2, vsc;  // score scale (log2 units) and value scale
    bool swapped;    // fp8 pool, R <= 8: S^T = K Q^T and O^T = V^T P^T
    bool active;
    // Windowed step (packed keys): rows see keys below `sinks` and from their
    // own low0 / low1 on; low_first and low_last are the first and the last
    // row's.  A key in [sinks, low_first) is seen by no row.
    int sinks, low0, low1, low_first, low_last;
    // keys key .. key + 15 are below no row's window (or all are sinks)
    __device__ __forceinline__ bool all_in_window(int key) const {
        return key >= low_last || key + kChunkKeys <= sinks;
    }
    __device__ __forceinline__ bool in_window(int key, int low) const {
        return key < sinks || key >= low;
    }
    // some row sees it, causal limits aside: V rows of other keys may hold
    // anything and are zeroed
    __device__ __forceinline__ bool live(int key) const {
        return key < key_end && in_window(key, low_first);
    }
    // per thread: rows g and g+8 of this warp's 16-row tile
    int limit0, limit1;
    uint32_t qa[KS][4];
    float o[NT][4];
    float m0, m1, l0, l1;
};

// L1 prefetch of an item's query rows (q_count tokens x the group's heads,
// each token's group one contiguous run of group * D bf16), by the producer
// lanes right after the item's first stage is issued: the consumers load
// them as mma fragments when that stage lands, and find them in L1.
template <int D>
__device__ __forceinline__ void prefetch_item_q(const ShortParams &p, int tok0, int h,
                                                int q_count, int lane) {
    const int seg = p.group * D * 2;     // bytes of one token's group
    const int lines = (seg + 127) / 128 + 1;  // a run may straddle one more line
    for (int i = lane; i < q_count * lines; i += 32) {
        const int t = i / lines, l = i - t * lines;
        const char *run = reinterpret_cast<const char *>(
            p.q + (static_cast<int64_t>(tok0 + t) * p.num_q_heads + h * p.group) * D);
        const char *a = run + min(l * 128, seg - 1);
        asm volatile("prefetch.global.L1 [%0];" ::"l"(a));
    }
}

// NC (1 or 2) 16-key chunks of an fp8 item with at most 8 rows, operands
// swapped; two chunks are interleaved so their dependency chains overlap.
// Lane (g = lane/4, t = lane%4) holds scores of keys g, g+8 for rows 2t,
// 2t+1, and O^T tile cc's elements (dim 16cc+2g | 16cc+2g+1) x (row 2t |
// 2t+1): cs.o[cc][0] = (row 2t, dim 16cc+2g), [1] = (2t+1, 16cc+2g),
// [2] = (2t, 16cc+2g+1), [3] = (2t+1, 16cc+2g+1).  CHECK = false: every
// key of the chunks is below the item's end and visible to every row (the
// caller checked), so the masks and the V-tail zeroing are compiled out.
template <int D, int NC, bool CHECK, bool WIN>
__device__ __forceinline__ void swapped_chunks(Consumer<D> &cs, const uint32_t (&kb)[NC],
                                               const uint32_t (&vb)[NC], const int (&key0)[NC],
                                               int lane) {
    constexpr int KS = D / 16;
    const int g = lane >> 2, t = lane & 3, mi = lane >> 3;
    // S^T = K Q^T, two accumulators per chunk (even / odd k-steps)
    float st[NC][2][4];
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) st[n][h][e] = 0.f;
#pragma unroll
    for (int ks2 = 0; ks2 < KS / 2; ++ks2) {
        // matrices: keys 0-7 | 8-15 of k-step 2ks2, then of 2ks2+1
        const int key = (mi & 1) * 8 + (lane & 7);
        const int col = ks2 * 2 + (mi >> 1);
        uint32_t r[NC][4];
#pragma unroll
        for (int n = 0; n < NC; ++n)
            ldsm_x4(kb[n] + sw128_offset(key, col), r[n][0], r[n][1], r[n][2], r[n][3]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_f16x2x2(r[n][2 * h], a0, a2);      // key g:   dims 4t,4t+1 | 4t+2,4t+3
                e4m3x4_to_f16x2x2(r[n][2 * h + 1], a1, a3);  // key g+8
                const int ks = ks2 * 2 + h;
                mma_f16_16816(st[n][h], a0, a1, a2, a3, cs.qa[ks][0], cs.qa[ks][1]);
            }
    }
    float s[NC][4];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        const bool need_mask =
            CHECK && ((key0[n] + kChunkKeys - 1 > cs.ctx) || (key0[n] + kChunkKeys > cs.key_end) ||
                      (WIN && !cs.all_in_window(key0[n])));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[n][e] = (st[n][0][e] + st[n][1][e]) * cs.sl2;
            if (need_mask) {
                const int key = key0[n] + g + (e >> 1) * 8;
                const int lim = (e & 1) ? cs.limit1 : cs.limit0;
                if (key > lim || key >= cs.key_end ||
                    (WIN && !cs.in_window(key, (e & 1) ? cs.low1 : cs.low0)))
                    s[n][e] = -INFINITY;
            }
        }
    }
    // lazy max: reduce over the 8 lanes of a row only when needed
    float la = -INFINITY, lb = -INFINITY;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        la = fmaxf(la, fmaxf(s[n][0], s[n][2]));
        lb = fmaxf(lb, fmaxf(s[n][1], s[n][3]));
    }
    const bool ua = la > cs.m0 + kRescaleThreshold || (cs.m0 == -INFINITY && la > -INFINITY);
    const bool ub = lb > cs.m1 + kRescaleThreshold || (cs.m1 == -INFINITY && lb > -INFINITY);
    if (__any_sync(0xffffffffu, ua || ub)) {
        float ma = la, mb = lb;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, o));
            mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
        }
        const bool up0 = ma > cs.m0 + kRescaleThreshold || (cs.m0 == -INFINITY && ma > -INFINITY);
        const bool up1 = mb > cs.m1 + kRescaleThreshold || (cs.m1 == -INFINITY && mb > -INFINITY);
        const float a0 = up0 ? (cs.m0 == -INFINITY ? 0.f : fast_exp2(cs.m0 - ma)) : 1.f;
        const float a1 = up1 ? (cs.m1 == -INFINITY ? 0.f : fast_exp2(cs.m1 - mb)) : 1.f;
        if (up0) cs.m0 = ma;
        if (up1) cs.m1 = mb;
        cs.l0 *= a0;
        cs.l1 *= a1;
#pragma unroll
        for (int cc = 0; cc < D / 16; ++cc) {
            cs.o[cc][0] *= a0;
            cs.o[cc][2] *= a0;
            cs.o[cc][1] *= a1;
            cs.o[cc][3] *= a1;
        }
    }
    const float ref0 = cs.m0 == -INFINITY ? 0.f : cs.m0;
    const float ref1 = cs.m1 == -INFINITY ? 0.f : cs.m1;
    // P^T fragments (key g | g+8) x (rows 2t, 2t+1) -> P fragments of row g
    uint32_t pb0[NC], pb1[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        const float p0 = fast_exp2(s[n][0] - ref0), p1 = fast_exp2(s[n][1] - ref1);
        const float p2 = fast_exp2(s[n][2] - ref0), p3 = fast_exp2(s[n][3] - ref1);
        cs.l0 += p0 + p2;
        cs.l1 += p1 + p3;
        pb0[n] = movmatrix_trans(pack_f16x2(p0, p1));
        pb1[n] = movmatrix_trans(pack_f16x2(p2, p3));
    }
    // O^T += V^T P^T; V rows past the item's keys are zeroed in the fragments
    bool tail[NC], k0[NC], k1[NC], k8[NC], k9[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        const int nvalid = cs.key_end - key0[n];
        tail[n] = CHECK && nvalid < kChunkKeys;
        k0[n] = 2 * t < nvalid;
        k1[n] = 2 * t + 1 < nvalid;
        k8[n] = 2 * t + 8 < nvalid;
        k9[n] = 2 * t + 9 < nvalid;
        if constexpr (WIN && CHECK) {
            tail[n] = tail[n] || !cs.all_in_window(key0[n]);
            k0[n] = cs.live(key0[n] + 2 * t);
            k1[n] = cs.live(key0[n] + 2 * t + 1);
            k8[n] = cs.live(key0[n] + 2 * t + 8);
            k9[n] = cs.live(key0[n] + 2 * t + 9);
        }
    }
#pragma unroll
    for (int c2 = 0; c2 < D / 32; ++c2) {
        // matrices: keys 0-7 | 8-15 of dim group 2c2, then of 2c2+1; lane:
        // keys 2t, 2t+1 x dims 2g, 2g+1 of the group
        const int key = (mi & 1) * 8 + (lane & 7);
        const int col = c2 * 2 + (mi >> 1);
        uint32_t r[NC][4];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            ldsm_x4_t(vb[n] + sw128_offset(key, col), r[n][0], r[n][1], r[n][2], r[n][3]);
            if (tail[n]) {
                r[n][0] = keep_pair(r[n][0], k0[n], k1[n]);
                r[n][2] = keep_pair(r[n][2], k0[n], k1[n]);
                r[n][1] = keep_pair(r[n][1], k8[n], k9[n]);
                r[n][3] = keep_pair(r[n][3], k8[n], k9[n]);
            }
        }
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t a0, a1, a2, a3;
                // low halves: dim 16cc+2g (A row g), high: 16cc+2g+1 (A row g+8)
                e4m3x4_to_f16x2x2(byte_perm(r[n][2 * h], 0x3120u), a0, a1);
                e4m3x4_to_f16x2x2(byte_perm(r[n][2 * h + 1], 0x3120u), a2, a3);
                mma_f16_16816(cs.o[2 * c2 + h], a0, a1, a2, a3, pb0[n], pb1[n]);
            }
    }
}

// One 16-key chunk of K (at kb) and V (at vb) for this warp's 16-row tile: S = Q
// K^T and O += P V on mma.sync with an online softmax.  CHECK = false: every key
// of the chunk is below the item's end and visible to every row (the caller
// checked), so that the masks and the V-tail zeroing are compiled out.
template <int D, bool FP8, bool CHECK, bool WIN>
__device__ __forceinline__ void row_chunk(Consumer<D> &cs, uint32_t kb, uint32_t vb, int key0,
                                          int lane) {
    constexpr int NT = D / 8, KS = D / 16;
    constexpr int kBoxBytes = kChunkKeys * 128;
    const int t = lane & 3, mi = lane >> 3;
    float sacc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sacc[i][e] = 0.f;
    if constexpr (FP8) {
#pragma unroll
        for (int ks2 = 0; ks2 < KS / 2; ++ks2) {
            // matrices: keys 0-7 | 8-15 of k-step 2ks2, then of 2ks2+1
            const int key = (mi & 1) * 8 + (lane & 7);
            const int col = ks2 * 2 + (mi >> 1);
            uint32_t r[4];
            ldsm_x4(kb + sw128_offset(key, col), r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int ks = ks2 * 2 + (m >> 1);
                uint32_t b0, b1;
                e4m3x4_to_f16x2x2(r[m], b0, b1);
                mma_f16_16816(sacc[m & 1], cs.qa[ks][0], cs.qa[ks][1], cs.qa[ks][2],
                              cs.qa[ks][3], b0, b1);
            }
        }
    } else {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int key = (mi >> 1) * 8 + (lane & 7);
            const int col = (ks & 3) * 2 + (mi & 1);
            uint32_t b0, b1, b2, b3;
            ldsm_x4(kb + (ks >> 2) * kBoxBytes + sw128_offset(key, col), b0, b1,
                    b2, b3);
            mma_bf16_16816(sacc[0], cs.qa[ks][0], cs.qa[ks][1], cs.qa[ks][2],
                           cs.qa[ks][3], b0, b1);
            mma_bf16_16816(sacc[1], cs.qa[ks][0], cs.qa[ks][1], cs.qa[ks][2],
                           cs.qa[ks][3], b2, b3);
        }
    }
    // scale to log2 units and mask (causal limit per row, item key range)
    const bool need_mask = CHECK && ((key0 + kChunkKeys - 1 > cs.ctx) ||
                                     (key0 + kChunkKeys > cs.key_end) ||
                                     (WIN && !cs.all_in_window(key0)));
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float s = sacc[nt][e] * cs.sl2;
            if (need_mask) {
                const int key = key0 + nt * 8 + 2 * t + (e & 1);
                const int lim = (e < 2) ? cs.limit0 : cs.limit1;
                if (key > lim || key >= cs.key_end ||
                    (WIN && !cs.in_window(key, (e < 2) ? cs.low0 : cs.low1)))
                    s = -INFINITY;
            }
            sacc[nt][e] = s;
        }
    float mx0 = fmaxf(fmaxf(sacc[0][0], sacc[0][1]), fmaxf(sacc[1][0], sacc[1][1]));
    float mx1 = fmaxf(fmaxf(sacc[0][2], sacc[0][3]), fmaxf(sacc[1][2], sacc[1][3]));
    mx0 = quad_max(mx0);
    mx1 = quad_max(mx1);
    const bool up0 = mx0 > cs.m0 + kRescaleThreshold || (cs.m0 == -INFINITY && mx0 > -INFINITY);
    const bool up1 = mx1 > cs.m1 + kRescaleThreshold || (cs.m1 == -INFINITY && mx1 > -INFINITY);
    if (__any_sync(0xffffffffu, up0 || up1)) {
        const float nm0 = up0 ? mx0 : cs.m0;
        const float nm1 = up1 ? mx1 : cs.m1;
        const float a0 = up0 ? (cs.m0 == -INFINITY ? 0.f : fast_exp2(cs.m0 - nm0)) : 1.f;
        const float a1 = up1 ? (cs.m1 == -INFINITY ? 0.f : fast_exp2(cs.m1 - nm1)) : 1.f;
        cs.m0 = nm0;
        cs.m1 = nm1;
        cs.l0 *= a0;
        cs.l1 *= a1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            cs.o[nt][0] *= a0;
            cs.o[nt][1] *= a0;
            cs.o[nt][2] *= a1;
            cs.o[nt][3] *= a1;
        }
    }
    const float ref0 = cs.m0 == -INFINITY ? 0.f : cs.m0;
    const float ref1 = cs.m1 == -INFINITY ? 0.f : cs.m1;
    float pr[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
        pr[nt][0] = fast_exp2(sacc[nt][0] - ref0);
        pr[nt][1] = fast_exp2(sacc[nt][1] - ref0);
        pr[nt][2] = fast_exp2(sacc[nt][2] - ref1);
        pr[nt][3] = fast_exp2(sacc[nt][3] - ref1);
    }
    // The probabilities are rounded once, to the type that V has in the MMA: bf16, or f16 for
    // decoded e4m3 codes (they are at most 2^kRescaleThreshold).  The sums take them
    // unrounded.  A bf16 pool's output is off by 0.0021-0.0023 of its size for it, where
    // rounding the output alone costs 0.0017; an e4m3 pool's by 0.0017.
    cs.l0 += pr[0][0] + pr[0][1] + pr[1][0] + pr[1][1];
    cs.l1 += pr[0][2] + pr[0][3] + pr[1][2] + pr[1][3];
    const uint32_t pa0 = FP8 ? pack_f16x2(pr[0][0], pr[0][1]) : pack_bf16x2(pr[0][0], pr[0][1]);
    const uint32_t pa1 = FP8 ? pack_f16x2(pr[0][2], pr[0][3]) : pack_bf16x2(pr[0][2], pr[0][3]);
    const uint32_t pa2 = FP8 ? pack_f16x2(pr[1][0], pr[1][1]) : pack_bf16x2(pr[1][0], pr[1][1]);
    const uint32_t pa3 = FP8 ? pack_f16x2(pr[1][2], pr[1][3]) : pack_bf16x2(pr[1][2], pr[1][3]);
    // V rows past the item's keys may hold anything (even NaN):
    // zero them in the fragments of a partially valid chunk.
    const int nvalid = cs.key_end - key0;
    bool tail = CHECK && nvalid < kChunkKeys;
    bool k0 = 2 * t < nvalid, k1 = 2 * t + 1 < nvalid;
    bool k8 = 2 * t + 8 < nvalid, k9 = 2 * t + 9 < nvalid;
    if constexpr (WIN && CHECK) {
        tail = tail || !cs.all_in_window(key0);
        k0 = cs.live(key0 + 2 * t);
        k1 = cs.live(key0 + 2 * t + 1);
        k8 = cs.live(key0 + 2 * t + 8);
        k9 = cs.live(key0 + 2 * t + 9);
    }
    if constexpr (FP8) {
#pragma unroll
        for (int c2 = 0; c2 < D / 32; ++c2) {
            // matrices: keys 0-7 | 8-15 of dim group 2c2, then of 2c2+1;
            // lane: keys 2t, 2t+1 x dims 2j, 2j+1 (j = lane / 4)
            const int key = (mi & 1) * 8 + (lane & 7);
            const int col = c2 * 2 + (mi >> 1);
            uint32_t r[4];
            ldsm_x4_t(vb + sw128_offset(key, col), r[0], r[1], r[2], r[3]);
            if (tail) {
                r[0] = keep_pair(r[0], k0, k1);
                r[2] = keep_pair(r[2], k0, k1);
                r[1] = keep_pair(r[1], k8, k9);
                r[3] = keep_pair(r[3], k8, k9);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) r[m] = byte_perm(r[m], 0x3120u);
            // low halves: dim 2j (even tile), high halves: dim 2j+1 (odd tile)
#pragma unroll
            for (int gsub = 0; gsub < 2; ++gsub) {
                // keys 0-7 (b0) and 8-15 (b1) of the even and odd tile
                uint32_t e0, o0, e1, o1;
                e4m3x4_to_f16x2x2(r[2 * gsub], e0, o0);
                e4m3x4_to_f16x2x2(r[2 * gsub + 1], e1, o1);
                mma_f16_16816(cs.o[4 * c2 + 2 * gsub], pa0, pa1, pa2, pa3, e0, e1);
                mma_f16_16816(cs.o[4 * c2 + 2 * gsub + 1], pa0, pa1, pa2, pa3, o0, o1);
            }
        }
    } else {
#pragma unroll
        for (int dp = 0; dp < KS; ++dp) {
            const int key = (mi & 1) * 8 + (lane & 7);
            const int col = (dp & 3) * 2 + (mi >> 1);
            uint32_t v0, v1, v2, v3;
            ldsm_x4_t(vb + (dp >> 2) * kBoxBytes + sw128_offset(key, col), v0, v1,
                      v2, v3);
            if (tail) {
                v0 = keep_pair(v0, k0, k1);
                v2 = keep_pair(v2, k0, k1);
                v1 = keep_pair(v1, k8, k9);
                v3 = keep_pair(v3, k8, k9);
            }
            mma_bf16_16816(cs.o[2 * dp], pa0, pa1, pa2, pa3, v0, v1);
            mma_bf16_16816(cs.o[2 * dp + 1], pa0, pa1, pa2, pa3, v2, v3);
        }
    }
}

}  // namespace

}  // namespace pa
