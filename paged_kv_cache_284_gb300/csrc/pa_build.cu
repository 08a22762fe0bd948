// pa_build.cu -- a step's metadata from the requests' lengths, on the GPU: query starts,
// lengths, slots and positions, blocks taken from a free list for the new tokens and given
// back by finished rows ("11. 推理加速(一):vLLM 原理", §11.2: a block is allocated when the
// tokens reach it; §11.5: a decode step is dominated by fixed per-step costs, of which the
// host's tables and their upload are one).
//
// With n_b new tokens behind c_b cached ones, row b needs ceil((c_b + n_b) / bs) - ceil(c_b /
// bs) new blocks; its first token and its first new block are the sums of n and of these over
// the rows before it.  Everything else follows from the two sums for each token on its own:
// its row (the last one that starts at or before it, found by halving), its position, the
// table column, and the block -- an old one from the table, a new one from the list.
//
// Bound: latency (launch, lengths, scan, table entry; the bytes of 65536 tokens are 0.2 us of
// HBM time).  Every CTA scans all rows for itself, so that no sum crosses CTAs.  Up to
// kWholeTokens one CTA does the whole step (64 decode rows: 3.4 us).  Above, the tokens have a
// grid of their own, a token to a thread, and a cluster of 8 beside it has the rows: it counts
// the entries of finished rows, a warp to a row, passes the counts round through distributed
// shared memory, gives the blocks back, and after the tokens' kernel has ended writes what the
// call may change in place (lengths, the list's state).  4500 tokens of 256 rows, 12 of them
// done: 7.9 us, 9.0 as one kernel of 8 CTAs; 140000 tokens of 1024 rows, 64 done: 10.3 us, 32.6
// so.  Decode rows: 300 take 3.9 us whole and 5.3 split, 1000 8.8 and 8.7, 2000 11.7 and 9.7.
// (The look at each id that is taken came after these: 0.2 us whole, 0.3 and 0.9 split.)
#include <algorithm>

#include "pa_internal.cuh"

namespace pa {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kWholeTokens = kThreads;

struct Sums {
    long long tokens, blocks;
    int done;  // rows
};
__device__ __forceinline__ Sums operator+(const Sums &a, const Sums &b) {
    return {a.tokens + b.tokens, a.blocks + b.blocks, a.done + b.done};
}
__device__ __forceinline__ Sums shfl_up(const Sums &s, int o) {
    return {__shfl_up_sync(0xffffffffu, s.tokens, o), __shfl_up_sync(0xffffffffu, s.blocks, o),
            __shfl_up_sync(0xffffffffu, s.done, o)};
}

// A row of the batch as the call found it.
struct Row {
    int n, ctx, have, need;  // new and cached tokens, blocks owned and wanted
    bool done, bad;
};
__device__ __forceinline__ Row load_row(const BuildParams &p, int b) {
    Row r{};
    const int q = p.query_lens[b], c = p.cached_lens[b];
    r.done = q < 0;
    r.n = max(q, 0);
    r.ctx = c;
    r.bad = c < 0 || static_cast<long long>(c) + r.n > p.max_keys;
    if (r.bad) {
        r.n = 0;
        r.ctx = max(0, min(c, p.max_keys));
    }
    r.have = (r.ctx + p.block_size - 1) / p.block_size;
    r.need = (r.ctx + r.n + p.block_size - 1) / p.block_size - r.have;
    return r;
}

// The last row that starts at or before t (start[] does not decrease, start[0] = 0 <= t): rows
// without tokens start where the next one does and are passed over.
__device__ __forceinline__ int row_of(const int *start, int rows, int t) {
    int lo = 0;
    for (int step = 1 << (31 - __clz(rows)); step > 0; step >>= 1)
        if (lo + step < rows && start[lo + step] <= t) lo += step;
    return lo;
}

// Calls f with a table row's first n entries, 32 at a time (-1 behind the last), by a whole
// warp; eight loads in flight, whose latency is what a row costs.
template <typename F>
__device__ __forceinline__ void for_entries(const int32_t *row, int n, F f) {
    const int lane = threadIdx.x & 31;
    for (int col0 = 0; col0 < n; col0 += 256) {
        int entry[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int col = col0 + 32 * i + lane;
            entry[i] = col < n ? row[col] : -1;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) f(entry[i]);
    }
}

// What a launch does: the whole step (one CTA), its tokens (any grid), or the rest (one cluster).
enum Part { kWhole, kTokens, kRows };

}  // namespace

template <Part PART>
__global__ void __launch_bounds__(kThreads) build_step_kernel(const BuildParams p) {
    // [5][num_seqs]: first token, cached tokens, first new block; the rows that are done and
    // how many blocks each gives back
    extern __shared__ int row_info[];
    __shared__ Sums warp_sums[kWarps];
    __shared__ int warp_given[kWarps];
    __shared__ int list_is_bad;  // an id that is none of the pool's was taken from it
    int *start = row_info, *ctx_of = row_info + p.num_seqs, *block_of = ctx_of + p.num_seqs,
        *done_rows = block_of + p.num_seqs, *gives = done_rows + p.num_seqs;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x, size = gridDim.x;
    if (PART == kRows) cluster_arrive_relaxed();
    // kRows: the tokens' kernel has let this one start after its own wait, so what came before
    // is there; only the outputs that may be inputs wait for its end
    if (PART != kRows) {
        pdl_wait();
        pdl_trigger();
    }
    const int head = p.free_state[0], count = p.free_state[1];
    if (tid == 0) list_is_bad = 0;

    // 1. sums over the rows: thread t has rows t * each ..
    const int each = (p.num_seqs + kThreads - 1) / kThreads;
    const int b0 = min(p.num_seqs, tid * each), b1 = min(p.num_seqs, b0 + each);
    Sums mine{0, 0, 0};
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        const Row r = load_row(p, b);
        bad |= r.bad;
        mine = mine + Sums{r.n, r.need, r.done};
    }
    Sums incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums before = shfl_up(incl, o);
        if (lane >= o) incl = incl + before;
    }
    if (lane == 31) warp_sums[warp] = incl;
    bad = head < 0 || head >= p.capacity || count < 0 || count > p.capacity || bad;
    bad = __syncthreads_or(bad);
    if (warp == 0) {
        Sums w = lane < kWarps ? warp_sums[lane] : Sums{0, 0, 0};
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sums before = shfl_up(w, o);
            if (lane >= o) w = w + before;
        }
        if (lane < kWarps) warp_sums[lane] = w;
    }
    __syncthreads();
    const Sums total = warp_sums[kWarps - 1];
    const Sums base = warp > 0 ? warp_sums[warp - 1] : Sums{0, 0, 0};
    // all or nothing: a step that does not fit leaves the rows, the tables and the list as
    // they are, and its metadata holds no token
    bad |= total.tokens > p.num_tokens;
    const long long missing = bad ? 0 : max(0ll, total.blocks - count);
    const bool good = !bad && missing == 0;
    if (PART != kTokens && rank == 0 && tid == 0 && !good)
        flag_status(p.status, bad ? PA_DEV_BAD_METADATA : PA_DEV_NO_BLOCKS);
    {
        // (sums of a step that does not fit may pass 32 bits and are not used)
        Sums at = base + Sums{incl.tokens - mine.tokens, incl.blocks - mine.blocks,
                              incl.done - mine.done};
        for (int b = b0; b < b1; ++b) {
            const Row r = load_row(p, b);
            start[b] = good ? static_cast<int>(at.tokens) : 0;
            ctx_of[b] = r.ctx;
            block_of[b] = good ? static_cast<int>(at.blocks) : 0;
            if (r.done) done_rows[at.done] = b;
            at = at + Sums{r.n, r.need, r.done};
        }
    }
    __syncthreads();
    const int tokens = good ? static_cast<int>(total.tokens) : 0;
    const int taken = good ? static_cast<int>(total.blocks) : 0;

    // 2. slots and positions; the first token of a new block enters it in the table
    for (int64_t i = static_cast<int64_t>(rank) * kThreads + tid; PART != kRows && i < p.num_tokens;
         i += static_cast<int64_t>(size) * kThreads) {
        const int t = static_cast<int>(i);
        int64_t slot = -1;
        int pos = 0;
        if (t < tokens) {
            const int b = row_of(start, p.num_seqs, t);
            const int c = ctx_of[b];
            pos = c + t - start[b];
            const int col = pos / p.block_size, have = (c + p.block_size - 1) / p.block_size;
            int32_t *entry = p.block_tables + static_cast<int64_t>(b) * p.max_blocks + col;
            int blk;
            if (col < have) {
                blk = *entry;
            } else {
                int64_t at = static_cast<int64_t>(head) + block_of[b] + (col - have);
                if (at >= p.capacity) at -= p.capacity;
                blk = p.free_blocks[at];
            }
            const bool ok = blk >= 0 && blk < p.num_blocks;
            if (!ok) {
                flag_status(p.status, PA_DEV_BAD_BLOCK);
                if (col >= have) list_is_bad = 1;
            }
            if (col >= have && pos % p.block_size == 0)
                *entry = ok ? blk : min(max(blk, 0), p.num_blocks - 1);
            slot = ok ? static_cast<int64_t>(blk) * p.block_size + pos % p.block_size : -1;
        }
        p.slot_mapping[t] = slot;
        p.positions[t] = pos;
    }

    // 3. the blocks of finished rows to the list's tail, rows and columns in order; entries
    // that were given back before (negative) are passed over.  The tail lies behind all that
    // was free, so nothing taken above is overwritten.
    if (PART == kTokens) return;
    int given = 0;
    if (PART == kRows) {
        // (the tokens' grid looks at the ids that it takes, but has nobody to tell)
        bool bad_id = false;
#pragma unroll 4
        for (int64_t i = tid; rank == 0 && i < taken; i += kThreads) {
            const int64_t at = head + i;
            const int blk = p.free_blocks[at >= p.capacity ? at - p.capacity : at];
            bad_id |= blk < 0 || blk >= p.num_blocks;
        }
        if (bad_id) list_is_bad = 1;
        cluster_wait();  // every CTA runs: its shared memory may be written
    }
    if (total.done > 0 && good) {
        // entries of a row, one warp of the cluster each
        for (int d = rank * kWarps + warp; d < total.done; d += size * kWarps) {
            const int b = done_rows[d];
            int live = 0;
            for_entries(p.block_tables + static_cast<int64_t>(b) * p.max_blocks,
                        (ctx_of[b] + p.block_size - 1) / p.block_size,
                        [&](int blk) { live += blk >= 0 && blk < p.num_blocks; });
            live = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(live)));
            if (PART == kRows) {
                if (lane < size) st_cluster(gives + d, lane, live);
            } else if (lane == 0) {
                gives[d] = live;
            }
        }
        if (PART == kRows)
            cluster_sync();
        else
            __syncthreads();
        const int d_each = (total.done + kThreads - 1) / kThreads;
        const int d0 = min(total.done, tid * d_each), d1 = min(total.done, d0 + d_each);
        int sum = 0;
        for (int d = d0; d < d1; ++d) sum += gives[d];
        int run = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int before = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += before;
        }
        if (lane == 31) warp_given[warp] = run;
        __syncthreads();
        int at = run - sum;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += warp_given[w];
            given += warp_given[w];
        }
        for (int d = d0; d < d1; ++d) {
            const int n = gives[d];
            gives[d] = at;
            at += n;
        }
        __syncthreads();
        const int room = p.capacity - count;
        for (int d = rank * kWarps + warp; d < total.done; d += size * kWarps) {
            const int b = done_rows[d];
            int next = gives[d];
            for_entries(p.block_tables + static_cast<int64_t>(b) * p.max_blocks,
                        (ctx_of[b] + p.block_size - 1) / p.block_size, [&](int blk) {
                            if (blk >= p.num_blocks) flag_status(p.status, PA_DEV_BAD_BLOCK);
                            const bool live = blk >= 0 && blk < p.num_blocks;
                            const unsigned lives = __ballot_sync(0xffffffffu, live);
                            const int place = next + __popc(lives & ((1u << lane) - 1));
                            if (live && place < room) {
                                int64_t to = static_cast<int64_t>(head) + count + place;
                                if (to >= p.capacity) to -= p.capacity;
                                p.free_blocks[to] = blk;
                            }
                            next += __popc(lives);
                        });
        }
        if (given > room) {  // more blocks than the list holds: one was in it twice
            if (rank == 0 && tid == 0) flag_status(p.status, PA_DEV_BAD_METADATA);
            given = room;
        }
    }

    // 4. the rows' lengths and the list's state, which may be the call's inputs: after every
    // CTA has read them
    if (PART == kRows) {
        pdl_wait();
        pdl_trigger();
        cluster_sync();
    } else {
        __syncthreads();
    }
    if (rank != 0) return;
    for (int b = b0; b < b1; ++b) {
        const Row r = load_row(p, b);
        // (a row whose cached length is out of range is handed on as it is)
        const int c = good && r.done ? 0 : p.cached_lens[b];
        p.query_start_loc[b] = start[b];
        p.context_lens[b] = c;
        p.seq_lens[b] = c + (good ? r.n : 0);
    }
    if (tid == 0) {
        p.query_start_loc[p.num_seqs] = tokens;
        int64_t h = static_cast<int64_t>(head) + taken;
        if (h >= p.capacity) h -= p.capacity;
        // The row's table has a block of another row's or of the list's from now on, and would
        // write there with its next token: a head out of range has later calls refused.
        p.free_state_out[0] = !good ? head : static_cast<int>(list_is_bad ? -1 - h : h);
        p.free_state_out[1] = count - taken + given;
        p.free_state_out[2] = static_cast<int>(min(missing, 0x7fffffffll));
        p.free_state_out[3] = 0;
    }
}

namespace {
template <Part PART>
int launch(const BuildParams &p, int ctas, cudaStream_t s) {
    static PerDeviceOnce once;
    if (once_per_device(once, [] {
            return cudaFuncSetAttribute(build_step_kernel<PART>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        5 * 4 * kBuildMaxSeqs);
        }) != PA_OK)
        return PA_ERR_CUDA;
    PdlLaunch l(ctas, kThreads, 5 * sizeof(int) * p.num_seqs, s);
    if (PART == kRows) l.set_cluster(ctas);
    return launch_kernel(l, build_step_kernel<PART>, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
}  // namespace

int launch_build_step(const BuildParams &p, cudaStream_t s) {
    if (p.num_tokens <= kWholeTokens) return launch<kWhole>(p, 1, s);
    const int64_t ctas = (static_cast<int64_t>(p.num_tokens) + kThreads - 1) / kThreads;
    const int rc = launch<kTokens>(p, static_cast<int>(std::min<int64_t>(p.sms, ctas)), s);
    return rc != PA_OK ? rc : launch<kRows>(p, kDirectMaxCluster, s);
}

}  // namespace pa
