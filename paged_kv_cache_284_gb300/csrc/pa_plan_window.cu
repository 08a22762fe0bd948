// pa_plan_window.cu -- device-side planner of a windowed step.
//
// Like the plain planner (pa_plan.cu) it turns the step's metadata into the two
// kernels' work lists without a host round trip, over the packed visible
// chunks of each request (KeySpan), longest first.  Windows bound the lengths,
// so with many requests most split-KV jobs (a piece, for one kv head) are
// equally long, and taking whole jobs leaves CTAs idle in the last round.  So
//  * with more jobs than CTAs, whole jobs go first and the pieces that make up
//    the last kTailStages stages per CTA are cut into splits of kTailSplit
//    stages, which the CTAs pull as they come free;
//  * with fewer jobs than CTAs, every job is cut so that all splits run in one
//    round.
// One CTA; latency is all that counts.  Every list is written by one thread
// per record (splits, tensor-core tiles), so that one long request is not
// planned by one thread.
#include "pa_internal.cuh"

namespace pa {

namespace {

constexpr int kT = 512;
constexpr int kWarps = kT / 32;
constexpr int kTableInSmem = 1024;
#ifndef TAIL_STAGES
#define TAIL_STAGES 0
#define TAIL_SPLIT 4
#endif
constexpr int kTailStages = TAIL_STAGES;
constexpr int kTailSplit = TAIL_SPLIT;

// Exclusive prefix of v over the block; *total = the block's sum.
struct Sums {
    long long a, b;
    int c, d;
};
__device__ __forceinline__ Sums operator+(const Sums &x, const Sums &y) {
    return {x.a + y.a, x.b + y.b, x.c + y.c, x.d + y.d};
}
__device__ __forceinline__ Sums operator-(const Sums &x, const Sums &y) {
    return {x.a - y.a, x.b - y.b, x.c - y.c, x.d - y.d};
}
__device__ __forceinline__ Sums warp_inclusive(Sums x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums n = {__shfl_up_sync(0xffffffffu, x.a, o), __shfl_up_sync(0xffffffffu, x.b, o),
                        __shfl_up_sync(0xffffffffu, x.c, o), __shfl_up_sync(0xffffffffu, x.d, o)};
        if (lane >= o) x = x + n;
    }
    return x;
}
__device__ Sums block_scan(const Sums &v, Sums *tmp, Sums *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Sums incl = warp_inclusive(v);
    if (lane == 31) tmp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const Sums mine = lane < kWarps ? tmp[lane] : Sums{0, 0, 0, 0};
        const Sums w = warp_inclusive(mine);
        if (lane < kWarps) tmp[lane] = w - mine;
        if (lane == kWarps - 1) tmp[kWarps] = w;
    }
    __syncthreads();
    const Sums base = tmp[warp];
    *total = tmp[kWarps];
    __syncthreads();
    return base + incl - v;
}

__device__ int block_max(int v, int *tmp) {
    const int m = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(v)));
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = m;
    __syncthreads();
    int r = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) r = max(r, tmp[i]);
    __syncthreads();
    return r;
}

struct Req {
    int n, ctx;
    int pieces, qtiles;  // split-KV pieces or tensor-core tiles
};

__device__ __forceinline__ Req load_req(const PlanParams &p, int b) {
    Req r{};
    const int q0 = p.qsl[b], q1 = p.qsl[b + 1], len = p.seq_lens[b];
    r.n = q1 - q0;
    r.ctx = p.ctx[b];
    if (r.n < 0 || r.ctx < 0 || len > p.max_keys || len != r.ctx + r.n || q0 < 0 ||
        q1 > p.num_q_tokens) {
        flag_status(p.status, PA_DEV_BAD_METADATA);
        r.n = 0;
    }
    return r;
}
// Which kernel a (valid) request runs on, and in how many pieces or tiles.
__device__ __forceinline__ void classify(const PlanParams &p, Req &r, int b) {
    if (r.n <= 0) return;
    bool is_short = static_cast<long long>(r.n) * p.group <= p.short_max_rows;
    // fp8 pool: a long request without a staging copy runs as pieces
    if (p.fp8 && !is_short && !(p.stage_cap > 0 && p.stage_base[b] >= 0)) is_short = true;
    if (is_short)
        r.pieces = (r.n + p.piece_tokens - 1) / p.piece_tokens;
    else
        r.qtiles = (r.n + p.q_tile_tokens - 1) / p.q_tile_tokens;
}

__device__ __forceinline__ WindowPiece piece_of(const PlanParams &p, const Req &r, int b, int i) {
    WindowPiece w{};
    w.b = b;
    w.q_begin = i * p.piece_tokens;
    w.q_count = min(p.piece_tokens, r.n - w.q_begin);
    const KeySpan ks = key_span(p.win, r.ctx + w.q_begin, r.ctx + w.q_begin + w.q_count);
    w.keys = ks.keys;
    w.sink_chunks = ks.sink_chunks;
    w.gap = ks.gap;
    w.stages = (ks.keys + kStageKeys - 1) / kStageKeys;
    return w;
}

__device__ __forceinline__ unsigned long long udiv(unsigned long long a, unsigned long long b) {
    return ((a | b) >> 32) ? a / b
                           : static_cast<unsigned>(a) / static_cast<unsigned>(b);
}

// Sort bin of an item of `len` stages or tiles: bin 0 holds the longest; a bin
// holds 2^shift consecutive lengths.
__device__ __forceinline__ int bin_shift(int longest) {
    int shift = 0;
    while ((longest >> shift) >= kT) ++shift;
    return shift;
}
__device__ __forceinline__ int len_bin(int len, int shift) {
    return kT - 1 - min(len >> shift, kT - 1);
}
// atomicAdd(&bins[bin], 1) by the active lanes of a warp, one atomic per bin.
__device__ __forceinline__ int bin_slot(int *bins, int bin) {
    const unsigned same = __match_any_sync(__activemask(), bin);
    const int leader = __ffs(same) - 1, lane = threadIdx.x & 31;
    int at = 0;
    if (lane == leader) at = atomicAdd(&bins[bin], __popc(same));
    return __shfl_sync(same, at, leader) + __popc(same & ((1u << lane) - 1));
}

}  // namespace

__global__ void __launch_bounds__(kT) plan_window_kernel(const PlanParams p) {
    __shared__ Sums tmps[kWarps + 1];
    __shared__ int tmpi[kWarps];
    __shared__ int bins[kT];
    // splits (one head) before each piece; tiles before each long request
    __shared__ int s_off[kTableInSmem], s_loff[kTableInSmem];
    __shared__ int s_overflow;
    const int tid = threadIdx.x;
    const int hkv = p.num_kv_heads;
    // the metadata (and the workspace) may belong to the previous kernel
    pdl_wait();
    pdl_trigger();
    if (tid == 0) s_overflow = 0;
    bins[tid] = 0;
    // request tid's metadata is read once; the others' again in each pass
    const Req mine = tid < p.num_seqs ? load_req(p, tid) : Req{};
    auto req = [&](int b) { return b == tid ? mine : b < p.num_seqs ? load_req(p, b) : Req{}; };

    // 0. fp8 pool with a staging area: long requests get consecutive bf16
    // staging blocks for their visible blocks, in request order while they fit
    int staged = 0;
    long long staged_blocks = 0;
    if (p.fp8 && p.stage_cap > 0) {
        long long cand = 0;
        for (int b0 = 0; b0 < p.num_seqs; b0 += kT) {
            const int b = b0 + tid;
            const Req r = req(b);
            int cnt = 0;
            if (r.n > 0 && static_cast<long long>(r.n) * p.group > p.short_max_rows)
                cnt = (r.ctx + r.n + p.block_size - 1) / p.block_size -
                      block_span(p.win, r.ctx, r.ctx + r.n, p.block_size).gap;
            Sums tot;
            const long long base = cand + block_scan({cnt, 0, 0, 0}, tmps, &tot).a;
            cand += tot.a;
            const bool fits = cnt > 0 && base + cnt <= p.stage_cap;
            const Sums at = block_scan({fits ? cnt : 0, 0, fits ? 1 : 0, 0}, tmps, &tot);
            if (b < p.num_seqs) p.stage_base[b] = fits ? static_cast<int>(base) : -1;
            if (fits) p.stage_list[staged + at.c] = b;
            staged += tot.c;
            staged_blocks += tot.a;
        }
    }

    // 1. tables: the pieces, with the stages before each, from the front;
    // the long requests, with the tiles before each, from the back
    Sums base{0, 0, 0, 0};  // stages (one head), tiles, pieces, long requests
    int max_stages = 0;
    for (int b0 = 0; b0 < p.num_seqs; b0 += kT) {
        const int b = b0 + tid;
        Req r = req(b);
        classify(p, r, b);
        long long sum = 0;
        for (int i = 0; i < r.pieces; ++i) {
            const int st = piece_of(p, r, b, i).stages;
            sum += st;
            max_stages = max(max_stages, st);
        }
        Sums tot;
        const Sums off =
            base + block_scan({sum, r.qtiles, r.pieces, r.qtiles > 0 ? 1 : 0}, tmps, &tot);
        base = base + tot;
        if (base.c + base.d > p.max_pieces || base.b * hkv > p.max_long) {
            if (tid == 0) s_overflow = 1;
            break;  // uniform: the totals are block-wide
        }
        long long at = off.a;
        for (int i = 0; i < r.pieces; ++i) {
            WindowPiece w = piece_of(p, r, b, i);
            w.before = at;
            at += w.stages;
            p.pieces[off.c + i] = w;
        }
        if (r.qtiles > 0) {
            WindowPiece w{};
            w.b = b;
            w.q_count = r.n;
            w.keys = r.ctx;
            w.before = off.b;
            p.pieces[p.max_pieces - 1 - off.d] = w;
            if (off.d < kTableInSmem) s_loff[off.d] = static_cast<int>(off.b);
        }
    }
    max_stages = block_max(max_stages, tmpi);  // (its barriers publish the tables)
    const int P = base.c, n_long = base.d;
    const long long J = static_cast<long long>(P) * hkv;  // jobs
    const long long total = base.a * hkv;                 // stages
    const int n_tiles = static_cast<int>(base.b);
    const long long C = max(1, p.num_ctas);

    // 2. splits per piece -------------------------------------------------------
    // More jobs than CTAs: pieces whose work lies in the last kTailStages
    // stages per CTA are cut by kTailSplit, the others stay whole.  Else all
    // by sp: total / (C - J / 2) stages a split usually gives at most C splits
    // (half a split of rounding per job), total / (C - J) always does.
    // Partial states that do not fit double the split.
    long long tail = J > C ? C * kTailStages : total;
    int sp = kTailSplit;
    if (J > 0 && J <= C)
        sp = static_cast<int>(max(static_cast<long long>(kMinSplitStages),
                                  static_cast<long long>(udiv(total + C - J / 2 - 1, C - J / 2))));
    auto splits_of = [&](const WindowPiece &w, long long stages_before) {
        return (base.a - stages_before) * hkv <= tail ? (w.stages + sp - 1) / sp : 1;
    };
    long long items = 0, rows = 0;
    for (int tries = 0; !s_overflow && P > 0; ++tries) {
        Sums sum{0, 0, 0, 0};
        for (int i = tid; i < P; i += kT) {
            const WindowPiece w = p.pieces[i];
            const int ns = splits_of(w, w.before);
            sum.a += ns;
            if (ns > 1) sum.b += static_cast<long long>(ns) * w.q_count * p.group;
        }
        Sums tot;
        (void)block_scan(sum, tmps, &tot);
        items = tot.a * hkv;
        rows = tot.b * hkv;
        if (sp >= max_stages ||
            (rows <= p.cap_rows && items <= p.max_short && (J > C || items <= C)))
            break;
        sp = tries == 0 && J < C
                 ? max(sp, static_cast<int>(min(static_cast<long long>(max_stages),
                                                static_cast<long long>(udiv(total + C - J - 1, C - J)))))
                 : min(max_stages, 2 * sp);
    }
    const bool fits = !s_overflow && J <= p.num_counters && items <= p.max_short &&
                      rows <= p.cap_rows;

    // 3. split-KV records, longest first (counting sort on the stages).  A
    // piece cuts its stages into splits that differ by at most one stage; its
    // splits of one length take consecutive records of their bin.
    if (fits && P > 0) {
        const int shift = bin_shift(max_stages);
        for (int i = tid; i < P; i += kT) {
            const WindowPiece w = p.pieces[i];
            const int ns = splits_of(w, w.before);
            const int q = w.stages / ns, extra = w.stages - q * ns;
            if (extra > 0) atomicAdd(&bins[len_bin(q + 1, shift)], extra * hkv);
            atomicAdd(&bins[len_bin(q, shift)], (ns - extra) * hkv);
        }
        __syncthreads();
        Sums tot;
        const int bin_at = block_scan({0, 0, bins[tid], 0}, tmps, &tot).c;
        bins[tid] = bin_at;
        __syncthreads();
        Sums run{0, 0, 0, 0};
        for (int i0 = 0; i0 < P; i0 += kT) {
            const int i = i0 + tid;
            WindowPiece w{};
            int ns = 0;
            if (i < P) {
                w = p.pieces[i];
                ns = splits_of(w, w.before);
            }
            const Sums at =
                run + block_scan({ns > 1 ? static_cast<long long>(ns) * w.q_count * p.group : 0, 0,
                                  ns, 0}, tmps, &tot);
            run = run + tot;
            if (i >= P) continue;
            const int q = w.stages / ns, extra = w.stages - q * ns;
            w.splits = ns;
            w.rows = static_cast<int>(at.a) * hkv;
            w.slot_hi = extra > 0 ? atomicAdd(&bins[len_bin(q + 1, shift)], extra * hkv) : 0;
            w.slot_lo = atomicAdd(&bins[len_bin(q, shift)], (ns - extra) * hkv);
            w.before = at.c;
            p.pieces[i] = w;
            if (i < kTableInSmem) s_off[i] = at.c;
        }
        __syncthreads();
        for (long long j = tid; j < items; j += kT) {
            int lo = 0, hi = P - 1;  // the piece: the last that starts at or before j
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                const long long before = mid < kTableInSmem ? s_off[mid] : p.pieces[mid].before;
                if (before * hkv <= j) lo = mid; else hi = mid - 1;
            }
            const WindowPiece w = p.pieces[lo];
            const int in = static_cast<int>(j - w.before * hkv);
            const int h = in / w.splits, s = in - h * w.splits;
            const int q = w.stages / w.splits, extra = w.stages - q * w.splits;
            const int R = w.q_count * p.group;
            ShortItem it;
            it.b = w.b;
            it.split = s;
            it.nsplit = w.splits;
            it.stage_begin = s * q + min(s, extra);
            it.stage_end = it.stage_begin + q + (s < extra ? 1 : 0);
            it.partial_base = w.splits > 1 ? w.rows + in * R : 0;
            it.q_begin = w.q_begin;
            it.q_count = w.q_count;
            it.counter = lo * hkv + h;
            it.seq_len = w.keys;
            it.sink_chunks = w.sink_chunks;
            it.gap = w.gap;
            store_record(p.short_items,
                         s < extra ? w.slot_hi + h * extra + s
                                   : w.slot_lo + h * (w.splits - extra) + (s - extra),
                         it);
        }
    }

    // 4. tensor-core tiles, longest key range first
    if (fits && n_tiles > 0) {
        auto tile = [&](int t, LongItem &it) {
            int lo = 0, hi = n_long - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                const long long before =
                    mid < kTableInSmem ? s_loff[mid] : p.pieces[p.max_pieces - 1 - mid].before;
                if (before <= t) lo = mid; else hi = mid - 1;
            }
            const WindowPiece w = p.pieces[p.max_pieces - 1 - lo];
            it = LongItem{};
            it.b = w.b;
            it.q_tile = t - static_cast<int>(w.before);
            const int first = w.keys + it.q_tile * p.q_tile_tokens;
            const KeySpan ks = key_span(p.win, first,
                                        min(w.keys + w.q_count, first + p.q_tile_tokens));
            it.key_end = ks.keys;
            it.sink_chunks = ks.sink_chunks;
            it.gap = ks.gap;
            return (ks.keys + kLongKeys - 1) / kLongKeys;
        };
        __syncthreads();
        bins[tid] = 0;
        LongItem first_item;
        int longest = 0, first_len = 0;
        for (int t = tid; t < n_tiles; t += kT) {
            LongItem it;
            const int len = tile(t, it);
            longest = max(longest, len);
            if (t == tid) {
                first_item = it;
                first_len = len;
            }
        }
        const int shift = bin_shift(block_max(longest, tmpi));
        for (int t = tid; t < n_tiles; t += kT) {
            LongItem it;
            const int len = t == tid ? first_len : tile(t, it);
            (void)bin_slot(bins, len_bin(len, shift));
        }
        __syncthreads();
        Sums tot;
        const int bin_at = block_scan({0, 0, bins[tid], 0}, tmps, &tot).c;
        bins[tid] = bin_at;
        __syncthreads();
        for (int t = tid; t < n_tiles; t += kT) {
            LongItem it = first_item;
            const int len = t == tid ? first_len : tile(t, it);
            store_record(p.long_items, bin_slot(bins, len_bin(len, shift)), it);
        }
    }

    // 5. counters and header ----------------------------------------------------
    for (int i = tid; i < p.num_counters && i < J; i += kT) p.counters[i] = 0;
    __syncthreads();
    if (tid == 0) {
        // a work list that did not fit is never run partially: no items at all
        if (!fits) flag_status(p.status, PA_DEV_PLAN_OVERFLOW);
        p.hdr->num_short_items = fits ? static_cast<int>(items) : 0;
        p.hdr->num_long_items = fits ? n_tiles * hkv : 0;
        p.hdr->short_next = 0;
        p.hdr->long_next = 0;
        p.hdr->split_stages = sp;
        p.hdr->partial_rows = fits ? static_cast<int>(rows) : 0;
        p.hdr->num_staged = fits ? staged : 0;
        p.hdr->staged_blocks = fits ? static_cast<int>(staged_blocks) : 0;
        p.hdr->first_done = 0;
    }
}

int launch_plan_window(const PlanParams &p, cudaStream_t s) {
    PdlLaunch l(1, kT, 0, s);
    return launch_kernel(l, plan_window_kernel, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
