// pa_plan_window.cu -- device-side planner of a windowed step.
//
// Like the plain planner (pa_plan.cu) it turns the step's metadata into the two
// kernels' work lists without a host round trip, over the packed visible
// chunks of each request (KeySpan), longest first.  Windows bound the lengths:
//  * with more split-KV jobs (a piece, for one kv head) than CTAs every job
//    stays whole.  Cutting the last ones finer, or the whole line of work into
//    equal runs of stages per CTA, balances better on paper and was slower
//    (512 jobs of 17 stages: 70.6 us whole, 71.9 / 76.9 / 87.3 us with the
//    last 4 / 8 / 16 stages per CTA cut by 4, 74.9 us in equal runs): a split
//    costs its CTA about three stages' time;
//  * with fewer jobs than CTAs, every job is cut so that all splits run in one
//    round.
// One CTA; latency is all that counts.  Every list is written by one thread
// per record (splits, tensor-core tiles), so that one long request is not
// planned by one thread, and the tables stay in shared memory.
#include "pa_internal.cuh"

namespace pa {

namespace {

constexpr int kT = 512;
constexpr int kWarps = kT / 32;
constexpr int kTableInSmem = 768;

struct Sums {
    int a, b, c;
};
__device__ __forceinline__ Sums operator+(const Sums &x, const Sums &y) {
    return {x.a + y.a, x.b + y.b, x.c + y.c};
}
__device__ __forceinline__ Sums operator-(const Sums &x, const Sums &y) {
    return {x.a - y.a, x.b - y.b, x.c - y.c};
}
__device__ __forceinline__ Sums warp_inclusive(Sums x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums n = {__shfl_up_sync(0xffffffffu, x.a, o), __shfl_up_sync(0xffffffffu, x.b, o),
                        __shfl_up_sync(0xffffffffu, x.c, o)};
        if (lane >= o) x = x + n;
    }
    return x;
}
// Exclusive prefix of v over the block; *total = the block's sum.  (Two
// barriers; the caller has one between two uses of tmp.)
__device__ Sums block_scan(const Sums &v, Sums *tmp, Sums *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Sums incl = warp_inclusive(v);
    if (lane == 31) tmp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const Sums mine = lane < kWarps ? tmp[lane] : Sums{0, 0, 0};
        const Sums w = warp_inclusive(mine);
        __syncwarp();
        if (lane < kWarps) tmp[lane] = w - mine;
        if (lane == kWarps - 1) tmp[kWarps] = w;
    }
    __syncthreads();
    const Sums base = tmp[warp];
    *total = tmp[kWarps];
    return base + incl - v;
}

struct Req {
    int n, ctx;
    int pieces, qtiles;  // split-KV pieces or tensor-core tiles
};

__device__ __forceinline__ Req load_req(const PlanParams &p, int b) {
    Req r{};
    const int q0 = __ldg(p.qsl + b), q1 = __ldg(p.qsl + b + 1), len = __ldg(p.seq_lens + b);
    r.n = q1 - q0;
    r.ctx = __ldg(p.ctx + b);
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

// Sort bin of an item of `len` stages or tiles: bin 0 holds the longest; a bin
// holds 2^shift consecutive lengths.
__device__ __forceinline__ int bin_shift(int longest) {
    const int bits = 32 - __clz(longest / kT);  // longest >> bits < kT
    return longest < kT ? 0 : bits;
}
__device__ __forceinline__ int len_bin(int len, int shift) {
    return kT - 1 - min(len >> shift, kT - 1);
}
// atomicAdd(&bins[bin], n) by the active lanes of a warp, one atomic per bin;
// returns where this lane's n start.
__device__ __forceinline__ int bin_take(int *bins, int bin, int n) {
    const unsigned same = __match_any_sync(__activemask(), bin);
    const int leader = __ffs(same) - 1, lane = threadIdx.x & 31;
    int at = 0;
    if (lane == leader) at = atomicAdd(&bins[bin], __popc(same) * n);
    return __shfl_sync(same, at, leader) + __popc(same & ((1u << lane) - 1)) * n;
}

}  // namespace

__global__ void __launch_bounds__(kT) plan_window_kernel(const PlanParams p) {
    __shared__ Sums tmp_a[kWarps + 1], tmp_b[kWarps + 1], tmp_c[kWarps + 1];
    __shared__ int bins[kT], tile_bins[kT];
    __shared__ int s_max_stages, s_max_tiles;
    __shared__ float s_stages;
    __shared__ long long s_blocks[kWarps];
    __shared__ WindowPiece s_table[kTableInSmem];
    const int tid = threadIdx.x;
    const int hkv = p.num_kv_heads;
    if (tid == 0) {
        s_max_stages = s_max_tiles = 0;
        s_stages = 0.f;
    }
    bins[tid] = tile_bins[tid] = 0;
    // the pieces from the front, the long requests from the back
    const int table_size = p.max_pieces;
    WindowPiece *table = table_size <= kTableInSmem ? s_table : p.pieces;
    // the metadata (and the workspace) may belong to the previous kernel
    pdl_wait();
    pdl_trigger();
    // request tid's metadata is read once; the others' again in each pass
    const Req mine = tid < p.num_seqs ? load_req(p, tid) : Req{};
    auto req = [&](int b) { return b == tid ? mine : b < p.num_seqs ? load_req(p, b) : Req{}; };
    for (int i = tid; i < p.num_counters; i += kT) p.counters[i] = 0;

    // 0. fp8 pool with a staging area: long requests get consecutive bf16
    // staging blocks for their visible blocks, in request order while they fit
    int staged = 0, staged_blocks = 0;
    if (p.fp8 && p.stage_cap > 0) {
        int cand = 0;
        bool full = false;
        for (int b0 = 0; b0 < p.num_seqs; b0 += kT) {
            const int b = b0 + tid;
            const Req r = req(b);
            int cnt = 0;
            if (!full && r.n > 0 && static_cast<long long>(r.n) * p.group > p.short_max_rows)
                cnt = min(p.stage_cap + 1,
                          (r.ctx + r.n + p.block_size - 1) / p.block_size -
                              block_span(p.win, r.ctx, r.ctx + r.n, p.block_size).gap);
            // blocks before this request, in 64 bits (2^28 blocks a request)
            long long before = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long n = __shfl_up_sync(0xffffffffu, before, o);
                if ((tid & 31) >= o) before += n;
            }
            if ((tid & 31) == 31) s_blocks[tid >> 5] = before;
            __syncthreads();
            long long base = cand + before - cnt, all = cand;
            for (int w = 0; w < kWarps; ++w) {
                if (w < (tid >> 5)) base += s_blocks[w];
                all += s_blocks[w];
            }
            const bool fits = cnt > 0 && base + cnt <= p.stage_cap;
            Sums tot;
            const Sums at = block_scan({fits ? cnt : 0, fits ? 1 : 0, 0}, tmp_b, &tot);
            if (b < p.num_seqs) p.stage_base[b] = fits ? static_cast<int>(base) : -1;
            if (fits) p.stage_list[staged + at.b] = b;
            staged += tot.b;
            staged_blocks += tot.a;
            full = all > p.stage_cap;  // no later request fits
            cand = full ? 0 : static_cast<int>(all);
            __syncthreads();
        }
    }

    // 1. tables: the pieces from the front, the long requests (q_count = tokens,
    // keys = context, before = tiles before it) from the back
    Sums base{0, 0, 0};  // pieces, tiles, long requests
    bool overflow = false;
    int max_stages = 0;
    float stages = 0.f;
    for (int b0 = 0; b0 < p.num_seqs; b0 += kT) {
        const int b = b0 + tid;
        Req r = req(b);
        classify(p, r, b);
        if (b0 > 0) __syncthreads();
        Sums tot;
        const Sums off = base + block_scan({r.pieces, r.qtiles, r.qtiles > 0 ? 1 : 0}, tmp_a, &tot);
        base = base + tot;
        if (base.a + base.c > table_size || static_cast<long long>(base.b) * hkv > p.max_long) {
            overflow = true;  // uniform: the totals are block-wide
            break;
        }
        for (int i = 0; i < r.pieces; ++i) {
            const WindowPiece w = piece_of(p, r, b, i);
            stages += static_cast<float>(w.stages);
            max_stages = max(max_stages, w.stages);
            table[off.a + i] = w;
        }
        if (r.qtiles > 0) {
            WindowPiece w{};
            w.b = b;
            w.q_count = r.n;
            w.keys = r.ctx;
            w.before = off.b;
            table[table_size - 1 - off.c] = w;
        }
    }
    max_stages = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(max_stages)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) stages += __shfl_xor_sync(0xffffffffu, stages, o);
    if ((tid & 31) == 0 && max_stages > 0) {
        atomicMax(&s_max_stages, max_stages);
        atomicAdd(&s_stages, stages);
    }
    __syncthreads();  // the tables too
    max_stages = s_max_stages;
    const int P = base.a, n_long = base.c, n_tiles = base.b;
    const int J = overflow ? 0 : P * hkv;  // jobs (at most num_counters, see below)
    const int C = max(1, p.num_ctas);

    // 2. splits per piece: one, or with at most as many jobs as CTAs
    // ceil(stages / sp).  total / (C - J / 2) stages a split usually gives at
    // most C splits (half a split of rounding per job), total / (C - J) always
    // does.  Partial states that do not fit double the split.  (The total in
    // fp32: it only steers the cut.)
    int sp = max(1, max_stages);
    int items = J, rows = 0;
    if (J > 0 && J <= C && max_stages > kMinSplitStages) {
        const float total = s_stages * static_cast<float>(hkv);
        auto size = [&](int d) {
            return max(kMinSplitStages,
                       static_cast<int>(fminf(ceilf(total / static_cast<float>(max(1, d))),
                                              static_cast<float>(max_stages))));
        };
        sp = size(C - J / 2);
        for (int tries = 0;; ++tries) {
            Sums sum{0, 0, 0};
            for (int i = tid; i < P; i += kT) {
                const int ns = (table[i].stages + sp - 1) / sp;
                sum.a += min(ns, C + 1);
                if (ns > 1) sum.b += min(ns, C + 1) * table[i].q_count * p.group;
            }
            Sums tot;
            (void)block_scan(sum, tmp_b, &tot);
            __syncthreads();
            items = tot.a * hkv;
            rows = tot.b * hkv;
            if (sp >= max_stages || (items <= C && items <= p.max_short && rows <= p.cap_rows)) break;
            sp = tries == 0 && J < C ? max(sp, size(C - J)) : min(max_stages, 2 * sp);
        }
    }
    const bool split = sp < max_stages;
    if (!split) {
        items = J;
        rows = 0;
    }
    const bool fits = !overflow && static_cast<long long>(P) * hkv <= p.num_counters &&
                      items <= p.max_short;

    // 3. split-KV records, longest first (counting sort on the stages).  A
    // piece cuts its stages into splits that differ by at most one stage; its
    // splits of one length take consecutive records of their bin.
    if (fits && P > 0) {
        const int shift = bin_shift(max_stages);
        for (int i = tid; i < P; i += kT) {
            const int st = table[i].stages, ns = split ? (st + sp - 1) / sp : 1;
            const int q = st / ns, extra = st - q * ns;
            if (extra > 0) atomicAdd(&bins[len_bin(q + 1, shift)], extra * hkv);
            atomicAdd(&bins[len_bin(q, shift)], (ns - extra) * hkv);
        }
        __syncthreads();
        Sums tot;
        const int bin_at = block_scan({bins[tid], 0, 0}, tmp_c, &tot).a;
        bins[tid] = bin_at;
        __syncthreads();
        Sums run{0, 0, 0};
        for (int i0 = 0; i0 < P; i0 += kT) {
            const int i = i0 + tid;
            int ns = 0, q = 0, extra = 0, need = 0;
            if (i < P) {
                const int st = table[i].stages;
                ns = split ? (st + sp - 1) / sp : 1;
                q = st / ns;
                extra = st - q * ns;
                need = ns > 1 ? ns * table[i].q_count * p.group : 0;
            }
            Sums at{i, 0, 0};
            if (split) {  // (one split each: the splits before piece i are i)
                if (i0 > 0) __syncthreads();
                at = run + block_scan({ns, need, 0}, tmp_a, &tot);
                run = run + tot;
            }
            if (i >= P) continue;
            table[i].splits = ns;
            table[i].rows = at.b * hkv;
            table[i].slot_hi =
                extra > 0 ? atomicAdd(&bins[len_bin(q + 1, shift)], extra * hkv) : 0;
            table[i].slot_lo = atomicAdd(&bins[len_bin(q, shift)], (ns - extra) * hkv);
            table[i].before = at.a;
        }
        __syncthreads();
        // a warp writes a run of consecutive items: it looks its first one's
        // piece up and walks on from there
        const int run_len = (items + kWarps - 1) / kWarps, run_begin = (tid >> 5) * run_len;
        const int run_end = min(items, run_begin + run_len);
        int lo = 0;
        if (split) {
            int hi = P - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (table[mid].before * hkv <= run_begin) lo = mid; else hi = mid - 1;
            }
        }
        for (int j = run_begin + (tid & 31); j < run_end; j += 32) {
            // the piece: the last that starts at or before j
            if (split)
                while (lo + 1 < P && table[lo + 1].before * hkv <= j) ++lo;
            else
                lo = static_cast<unsigned>(j) / static_cast<unsigned>(hkv);
            const WindowPiece w = table[lo];
            const int in = j - w.before * hkv;
            const int h = static_cast<unsigned>(in) / static_cast<unsigned>(w.splits);
            const int s = in - h * w.splits;
            const int q = static_cast<unsigned>(w.stages) / static_cast<unsigned>(w.splits);
            const int extra = w.stages - q * w.splits;
            ShortItem it;
            it.b = w.b;
            it.split = s;
            it.nsplit = w.splits;
            it.stage_begin = s * q + min(s, extra);
            it.stage_end = it.stage_begin + q + (s < extra ? 1 : 0);
            it.partial_base = w.splits > 1 ? w.rows + in * w.q_count * p.group : 0;
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
                if (table[table_size - 1 - mid].before <= t) lo = mid; else hi = mid - 1;
            }
            const WindowPiece w = table[table_size - 1 - lo];
            it = LongItem{};
            it.b = w.b;
            it.q_tile = t - w.before;
            const int first = w.keys + it.q_tile * p.q_tile_tokens;
            const KeySpan ks = key_span(p.win, first,
                                        min(w.keys + w.q_count, first + p.q_tile_tokens));
            it.key_end = ks.keys;
            it.sink_chunks = ks.sink_chunks;
            it.gap = ks.gap;
            return (ks.keys + kLongKeys - 1) / kLongKeys;
        };
        LongItem first_item{};
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
        longest = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(longest)));
        if ((tid & 31) == 0 && longest > 0) atomicMax(&s_max_tiles, longest);
        __syncthreads();
        const int shift = bin_shift(s_max_tiles);
        for (int t = tid; t < n_tiles; t += kT) {
            LongItem it;
            (void)bin_take(tile_bins, len_bin(t == tid ? first_len : tile(t, it), shift), 1);
        }
        __syncthreads();
        Sums tot;
        const int bin_at = block_scan({tile_bins[tid], 0, 0}, tmp_b, &tot).a;
        tile_bins[tid] = bin_at;
        __syncthreads();
        for (int t = tid; t < n_tiles; t += kT) {
            LongItem it = first_item;
            const int len = t == tid ? first_len : tile(t, it);
            store_record(p.long_items, bin_take(tile_bins, len_bin(len, shift), 1), it);
        }
    }

    // 5. header -----------------------------------------------------------------
    if (tid == 0) {
        // a work list that did not fit is never run partially: no items at all
        if (!fits) flag_status(p.status, PA_DEV_PLAN_OVERFLOW);
        p.hdr->num_short_items = fits ? items : 0;
        p.hdr->num_long_items = fits ? n_tiles * hkv : 0;
        p.hdr->short_next = 0;
        p.hdr->long_next = 0;
        p.hdr->split_stages = sp;
        p.hdr->partial_rows = fits ? rows : 0;
        p.hdr->num_staged = fits ? staged : 0;
        p.hdr->staged_blocks = fits ? staged_blocks : 0;
        p.hdr->first_done = 0;
    }
}

int launch_plan_window(const PlanParams &p, cudaStream_t s) {
    PdlLaunch l(1, kT, 0, s);
    return launch_kernel(l, plan_window_kernel, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
