// pa_linear_prompt.cu -- linear attention with a decay per head: prompts, in chunks of 64 or 128
// tokens on tcgen05.
//
// With G_i the sum of the logarithms of a chunk's decays up to and with token i, S the state
// before the chunk and L the chunk's last token,
//   o_i  = scale (e^(G_i) q_i S + sum_(j <= i) e^(G_i - G_j) (q_i k_j) v_j)
//   S'   = e^(G_L) S + sum_j k_j (e^(G_L - G_j) v_j)^T
// No exponent is above 0, but for the rounding of the sums in it.  Columns of S and of o do not
// depend on each other, so a CTA has 64 of them (a slice), for one request and kv head, and walks
// along the request:
//   scores  Q K^T            M = 64 tokens x 2 query heads of the group, or 128 x 1
//   inside  P V              P = the scores times e^(G_i - G_j), masked, over them in TMEM
//   before  Q S              S in bf16, in shared memory
//   update  K^T (e^(G_L - G) V), M = the state's rows
// Roles: warp 0 loads; a thread each of warps 1-3 and 25 issues updates, scores, "before" and
// "inside"; warps 4-11, two groups that take the tiles in turn, make P and write the outputs
// (one thread a row); warps 12-15 weigh V; warps 16-23 keep the state, 32 fp32 values of a
// thread; warp 24 sums the logarithms.  So the chain from one chunk's state to the next (update,
// sum, rounding) and the chain of the weighed V run beside each other and beside the outputs.
//
// Bound: the path between shared memory, the tensor cores' operands and L1 (128 bytes a cycle),
// and what the schedulers issue; not HBM or the tensor pipe.  2 x 8192 tokens of 32 kv heads of
// 128 take 170 us, where HBM alone would need 80 (95 on the 128 SMs that have a slice).  Of the
// 5200 cycles of 128 tokens, that path carries the MMAs' operands for 2000, copies, weighed V and
// states for 1300, and the stores, a sector from each row, for 500.  Leaving a role's work out
// saves about its share, whichever it is: no stores 20 us, no weights and a third of the updates'
// MMAs 30, no states 20.  What that led to:
//  - where a group is one head, chunks of 128 tokens, whose tiles fill the MMA's 128 rows: 193 us
//    with chunks of 64 and half the rows idle (216 before the idle rows took turns)
//  - outputs by 32 bytes of a lane: 190 us by 16
//  - chunks of 64: two of the three parts of the weighed V in one MMA, into columns of their own
//    (2 x 8192 of 64 / 32 heads 200 us, 207 with an MMA to each and two buffers for the update);
//    chunks of 128 have these columns for a second "before" (173 us, 181)
//  - the warps of the states and outputs wait for the table, not for the weighed V (P V does: V is
//    weighed by then, and holds nothing any more that is no number)
//  - packed fp32 arithmetic, waits that sleep on the barrier, roles dealt to the schedulers by
//    what they issue
//  - loops over 16 columns stay loops, and only the MMAs of 64 of a dimension are unrolled: the
//    code of all roles has to fit the instruction cache (109 KB of it: 349 us when 72 KB took
//    215; the weighing by two rows of a lane instead of one: 172 us, and 229 instead of 209 with
//    64 / 32 heads), and a burst of one thread's MMAs holds up the others' (all unrolled: 20 %
//    more).  An MMA of 128 x 64 x 16 takes the pipe 47 cycles, from one thread or from four
//  - without a cluster a kernel of its own, that has no exchange: 8 us less
//  - left out: more chunks of K and V or more query tiles in shared memory, K and V given back one
//    by one, eight warps for the weights, two threads for the updates: none gained
// P's weights: within 16 tokens exponentials, from one run of 16 to a later one products of a
// factor of the row's and one of the column's.
//
// Roundings.  P and the S that Q meets are rounded to bf16, as an MMA's operands must be; both
// go into an output of bf16.  The state itself is a result in fp32 that later chunks build on,
// so the weighed V is taken as a sum of three bf16 numbers, which holds all its digits, and the
// update's products accumulate in fp32.
//
// A cluster of up to 8 CTAs shares a request when there are fewer of them than SMs: each rank
// takes a run of chunks, first makes its run's own update from K and V alone, then the ranks
// pass these on through distributed shared memory, so that each knows the state before its
// run, and then goes through its run for the outputs.
#include <algorithm>

#include "pa_internal.cuh"

namespace pa {

namespace {

constexpr int kSlice = 64;   // state columns of a CTA
constexpr int kRows = 128;   // rows of a query tile, and of a state's MMA
constexpr int kWarpKV = 1, kWarpQK = 2, kWarpQS = 3, kFirstOut = 4, kFirstWeigh = 12,
              kFirstState = 16;
constexpr int kMmaWarps = 4, kGroupWarps = 4, kWeighWarps = 4, kStateWarps = 8;
// (a warp is on the SM's quarter of its number modulo 4: each has as much to issue)
constexpr int kWarpScan = kFirstState + kStateWarps, kWarpPV = kWarpScan + 1;
constexpr int kWarps = kWarpPV + 1, kThreads = 32 * kWarps;
constexpr int kQueue = 4;
constexpr int kTables = 8;   // chunks whose sums of logarithms are kept
constexpr int kVtBars = 8;   // more than weighed V can be ahead of whoever looks at its barrier
constexpr int kPart = 64;    // tokens of a buffer of weighed V
constexpr int kParts = 3;    // bf16 numbers whose sum is a weighed element of V
// Logarithms (base 2) below this are as good as none: what they multiply is 0 in fp32.
constexpr float kLeastLog = -150.f;

// Of a chunk's tokens, in runs of 16 (logarithms base 2): the sums in their run up to and with
// each; e^ of what lies between a token and the end of its run, and of what lies behind it in the
// chunk; between[r][x], the sum of the runs x .. r - 1 (0 from x = r on); the chunk's sum.  Only
// tokens of one run meet in a difference of sums, which keeps the digits that 16 logarithms leave:
// in sums from the chunk's start a cleared token (-150) takes digits from all weights behind it,
// 64 of them up to 0.002 of a weight (2 x 8192 tokens of 32 heads took 168.5 us so and take 169,
// 64 / 32 heads 203 and 209).
template <int C>
struct alignas(16) Table {
    static constexpr int kRuns = C / 16;
    float sum[C], tail[C], weight[C], between[kRuns][kRuns];
    float all, pad[3];
};

// Pairs of fp32, in packed arithmetic.
__device__ __forceinline__ uint64_t f2_twice(float v) { return f2_pack(v, v); }
__device__ __forceinline__ uint64_t f2_words(uint32_t lo, uint32_t hi) {
    return f2_pack(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint32_t f2_bf16x2(uint64_t v) {
    float lo, hi;
    f2_unpack(v, lo, hi);
    return pack_bf16x2(lo, hi);
}

// Two of bf16, with 0 for what is no finite number.
__device__ __forceinline__ uint32_t finite2(uint32_t v) {
    return ((v & 0x7F80u) == 0x7F80u ? 0u : v & 0xFFFFu) |
           ((v & 0x7F800000u) == 0x7F800000u ? 0u : v & 0xFFFF0000u);
}

// 32 aligned bytes: a whole sector from each lane
__device__ __forceinline__ void store32(uint4 *dst, const uint4 &lo, const uint4 &hi) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(lo.x),
                 "r"(lo.y), "r"(lo.z), "r"(lo.w), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
                 : "memory");
}

// A chunk is 64 tokens beside tiles of two heads, 128 beside tiles of one.
template <int D, int C>
struct Geom {
    static constexpr int kHeads = kRows / C;  // of a tile
    static constexpr int kRing = C == 64 ? 3 : 2;   // chunks of K and V in shared memory
    static constexpr int kQBufs = C == 64 ? 2 : 1;  // query tiles
    static constexpr int kFills = C / kPart;        // buffers of weighed V that a chunk fills
    static constexpr int kHalves = D / 64;
    static constexpr int kQHalf = kRows * 128, kKHalf = C * 128;
    static constexpr int kQBytes = kHalves * kQHalf;
    static constexpr int kKBytes = kHalves * kKHalf, kVBytes = kKHalf;
    static constexpr int kStageBytes = kKBytes + kVBytes;
    static constexpr int kSBytes = kRows * 128;  // bf16 state: 128 rows x 64 columns
    static constexpr int kOffQ = 0;              // [kQBufs]
    static constexpr int kOffKV = kOffQ + kQBufs * kQBytes;
    static constexpr int kOffVt = kOffKV + kRing * kStageBytes;  // weighed V, part after part [2]
    static constexpr int kVtBytes = kPart * 128;
    static constexpr int kOffS = kOffVt + 2 * kParts * kVtBytes;  // [2]
    static constexpr int kOffBar = kOffS + 2 * kSBytes;
    static constexpr int kOffTab = kOffBar + 416;                // [kTables]
    static constexpr int kOffCtl = kOffTab + kTables * static_cast<int>(sizeof(Table<C>));
    static constexpr int kSmemRaw = kOffCtl + 512 + (kThreads + 1) * 4;
    // one CTA per SM: its TMEM columns are all taken
    static constexpr int kSmemBytes = kSmemRaw > 116 * 1024 ? kSmemRaw : 116 * 1024;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
    static_assert(kOffBar % 1024 == 0, "alignment");
    // TMEM columns: scores [2], "before" [2], "inside" [kInsides], update (64: of the first part of
    // the weighed V | of the others)
    static constexpr uint32_t kTmemCols = 512;
    static constexpr int kInsides = C == 64 ? 2 : 1, kUpdates = C == 64 ? 2 : 1;
    static constexpr int kColB = 2 * C, kColI = kColB + 2 * kSlice, kColU = kColI + kInsides * kSlice;
    static_assert(kColU + kUpdates * kSlice <= 512, "TMEM");
};

struct Bars {
    uint64_t kv_full[3], kv_empty[3];
    uint64_t q_full[2], q_empty[2];
    // table of a chunk there, weighed V of 64 tokens there / read; an update done / read
    uint64_t tab_full[kVtBars], vt_full[kVtBars], vt_empty[2], u_full, u_empty;
    uint64_t s_full[2], s_empty[2];    // state before a chunk in shared memory / read
    uint64_t sc_full[2], p_full[2];    // scores of a tile / its P
    uint64_t o_full[2], o_empty[2];
    uint64_t drain[kMmaWarps];
};
static_assert(sizeof(Bars) <= 416, "barrier area");
static_assert(kWarpKV < kMmaWarps && kWarpQK < kMmaWarps && kWarpQS < kMmaWarps, "drain[]");

// One request, kv head and slice, and this rank's run of chunks.
struct alignas(16) Item {
    int t0, n, h, slice;       // n = 0: no more items
    int c_begin, c_end, chunks;
    int in, to, pad[3];
};
static_assert(sizeof(Item) == 48, "queue entry");

struct Ctl {
    int abort, published, read[kWarps];
    int odd;      // V held an infinity or a NaN
    uint32_t tmem;
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
template <int D, int C>
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
    m = __ballot_sync(0xffffffffu,
                      lane < kThreads / 32 && count[group + lane % (kThreads / 32)] <= want);
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
    it.chunks = (it.n + C - 1) / C;
    const int run = (it.chunks + size - 1) / size;
    it.c_begin = min(it.chunks, rank * run);
    it.c_end = min(it.chunks, it.c_begin + run);
    return it;
}

// Outputs behind an infinity or a NaN of V in the same chunk, by all warps of a CTA that has seen
// one, when all its outputs are written.  P has zeros for earlier tokens, which P V would turn into
// NaN; so V's element is 0 there, and here its column's outputs become NaN from its token on to the
// end of the chunk.  (Later chunks have it from the state, whose update meets V as it is.)  At the
// kernel's end it costs the roles neither registers nor instruction cache: among the outputs, or as
// a function that is called, it cost 6 to 13 %.
template <int D, int C>
__device__ __forceinline__ void late_columns(const LinearParams &p, int rank, int size) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = p.num_kv_heads * (D / kSlice);
    // this cluster's items, as find_item has them
    int64_t longs = 0, idx = blockIdx.x / size;  // long requests before b, next item
#pragma unroll 1
    for (int b = 0; b < p.num_seqs; ++b) {
        int t0;
        const int n = long_tokens(p, b, t0);
        if (n == 0) continue;
        const int chunks = (n + C - 1) / C, run = (chunks + size - 1) / size;
        ++longs;
#pragma unroll 1
        for (; idx < longs * per; idx += gridDim.x / size) {
            const int in = static_cast<int>(idx % per), h = in / (D / kSlice);
            const int col = in % (D / kSlice) * kSlice + 2 * lane;  // and the next one
#pragma unroll 1
            for (int i = rank * run + warp; i < min(chunks, (rank + 1) * run); i += kWarps) {
                bool lo = false, hi = false;
#pragma unroll 1
                for (int t = i * C; t < min(n, (i + 1) * C); ++t) {
                    const uint32_t v = *reinterpret_cast<const uint32_t *>(
                        p.v + (t0 + t) * p.v_stride + h * D + col);
                    lo |= (v & 0x7F80u) == 0x7F80u;
                    hi |= (v & 0x7F800000u) == 0x7F800000u;
                    if (!lo && !hi) continue;
                    unsigned short *out = reinterpret_cast<unsigned short *>(p.out) +
                        (static_cast<int64_t>(t0 + t) * p.num_q_heads + h * p.group) * D + col;
#pragma unroll 1
                    for (int j = 0; j < p.group; ++j, out += D) {
                        if (lo) out[0] = 0x7FFF;
                        if (hi) out[1] = 0x7FFF;
                    }
                }
            }
        }
    }
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
    __syncwarp();
    return it;
}

}  // namespace

template <int D, int C, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 1)
    linear_prompt_kernel(const LinearParams p, const __grid_constant__ CUtensorMap tmq,
                         const __grid_constant__ CUtensorMap tmk,
                         const __grid_constant__ CUtensorMap tmv, int ranks) {
    using G = Geom<D, C>;
    constexpr int kRing = G::kRing;
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars *bars = reinterpret_cast<Bars *>(smem + G::kOffBar);
    Table<C> *tables = reinterpret_cast<Table<C> *>(smem + G::kOffTab);
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + G::kOffCtl);
    int *count = reinterpret_cast<int *>(smem + G::kOffCtl + 512);
    volatile int *abort_flag = &ctl->abort;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31, tid = threadIdx.x;
    const int size = CLUSTER ? ranks : 1;
    const int rank = CLUSTER ? static_cast<int>(blockIdx.x) % size : 0;
    const int tiles = (p.group + G::kHeads - 1) / G::kHeads;

    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&bars->kv_full[i], 1);
            mbar_init(&bars->kv_empty[i], kMmaWarps);
        }
        mbar_init(&bars->u_full, 1);
        mbar_init(&bars->u_empty, kStateWarps);
        for (int i = 0; i < kMmaWarps; ++i) mbar_init(&bars->drain[i], 1);
        for (int i = 0; i < kVtBars; ++i) {
            mbar_init(&bars->tab_full[i], 1);
            mbar_init(&bars->vt_full[i], kWeighWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->q_full[i], 1);
            mbar_init(&bars->q_empty[i], 2);  // by Q K^T and Q S
            mbar_init(&bars->vt_empty[i], 1);
            mbar_init(&bars->s_full[i], kStateWarps);
            mbar_init(&bars->s_empty[i], 1);
            mbar_init(&bars->sc_full[i], 1);
            mbar_init(&bars->p_full[i], kGroupWarps);
            mbar_init(&bars->o_full[i], 2);  // by Q S and P V
            mbar_init(&bars->o_empty[i], kGroupWarps);
        }
        ctl->abort = 0;
        ctl->odd = 0;
        ctl->published = 0;
        for (int w = 0; w < kWarps; ++w) ctl->read[w] = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    if (warp == kWarpQK) tmem_alloc(&ctl->tmem, G::kTmemCols);
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
        if (lane == 31) reinterpret_cast<int *>(tables)[warp] = incl;
        __syncthreads();
        int base = 0;
        for (int w = 0; w < warp; ++w) base += reinterpret_cast<int *>(tables)[w];
        count[tid + 1] = base + incl;
        if (tid == 0) count[0] = 0;
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem, 0);
    uint8_t *sQ = smem + G::kOffQ, *sKV = smem + G::kOffKV, *sVt = smem + G::kOffVt,
            *sS = smem + G::kOffS;

    if (warp == 0) {
        // ============================ loads ============================
        uint32_t c = 0, t = 0;  // chunks and tiles loaded
        bool ok = true;
        auto load_kv = [&](const Item &it, int i) {
            const int st = c % kRing;
            if (ok && c >= kRing)
                ok = warp_mbar_wait_small(&bars->kv_empty[st], (c / kRing - 1) & 1, abort_flag);
            // test hook: stop after the first chunk, as if a wait had run out
            if (p.test_stall && blockIdx.x == 0 && c == 1) ok = false;
            if (!ok) return;
            if (lane == 0) {
                uint8_t *dst = sKV + st * G::kStageBytes;
                mbar_arrive_expect_tx(&bars->kv_full[st], G::kStageBytes);
                for (int hf = 0; hf < G::kHalves; ++hf)
                    tma_load_3d(dst + hf * G::kKHalf, &tmk, hf * 64, it.h, it.t0 + i * C,
                                &bars->kv_full[st]);
                tma_load_3d(dst + G::kKBytes, &tmv, it.slice * kSlice, it.h, it.t0 + i * C,
                            &bars->kv_full[st]);
            }
            __syncwarp();
            ++c;
        };
        for (int k = 0;; ++k) {
            Item it = find_item<D, C>(p, count, k, rank, size);
            if (lane == 0) {
                const bool free = k < kQueue || spin(&ctl->abort, [&] {
                                      for (int w = 1; w < kWarps; ++w)
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
#pragma unroll 1
            for (int outputs = size > 1 ? 0 : 1; outputs < 2; ++outputs) {
                const int end = outputs || it.c_end < it.chunks ? it.c_end : it.c_begin;
#pragma unroll 1
                for (int i = it.c_begin; ok && i < end; ++i) {
                    load_kv(it, i);
                    if (!outputs) continue;
#pragma unroll 1
                    for (int j = 0; ok && j < tiles; ++j, ++t) {
                        const int st = t % G::kQBufs;
                        if (t >= G::kQBufs)
                            ok = warp_mbar_wait_small(&bars->q_empty[st], (t / G::kQBufs - 1) & 1, abort_flag);
                        if (!ok) break;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&bars->q_full[st], G::kQBytes);
                            for (int hf = 0; hf < G::kHalves; ++hf)
                                tma_load_3d(sQ + st * G::kQBytes + hf * G::kQHalf, &tmq, hf * 64,
                                            it.h * p.group + j * G::kHeads, it.t0 + i * C,
                                            &bars->q_full[st]);
                        }
                        __syncwarp();
                    }
                }
                if (!outputs) {
                    cluster_sync();
                    cluster_sync();
                }
            }
        }
        if (*abort_flag && lane == 0) {
            // copies in flight land before the CTA exits
            for (uint32_t i = c > kRing ? c - kRing : 0; i < c; ++i)
                mbar_drain(&bars->kv_full[i % kRing], (i / kRing) & 1);
            for (uint32_t i = t > G::kQBufs ? t - G::kQBufs : 0; i < t; ++i)
                mbar_drain(&bars->q_full[i % G::kQBufs], (i / G::kQBufs) & 1);
        }
    } else if (warp < kFirstOut || warp == kWarpPV) {
        // ============================ MMAs ============================
        // A thread of four warps each, so that none stands behind another's wait or issue (an MMA
        // takes its thread 100 to 200 cycles, four at a time): the scores, the updates, Q S, and
        // P V.  (One thread, not a warp with an elected lane's predicate: operands in a warp's
        // uniform registers are no longer its own when a wait has taken the lanes apart.  A commit
        // was seen to arrive twice, and worse.)
        constexpr uint32_t idesc_qk = idesc_bf16_f32(kRows, C, 0);
        constexpr uint32_t idesc_v = idesc_bf16_f32(kRows, kSlice, 1);
        constexpr uint32_t idesc_kv = idesc_bf16_f32(kRows, kSlice, 1, 1);
        constexpr uint32_t idesc_kv2 = idesc_bf16_f32(kRows, 2 * kSlice, 1, 1);
        const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t k_desc = smem_desc_sw128(smem_u32(sKV), 16, 1024);
        // K with its tokens as the summed dimension (head_dim 64: the second half of M is V, and
        // those rows of the update are not read)
        const uint64_t kt_desc = smem_desc_sw128(smem_u32(sKV), G::kKHalf, 1024);
        const uint64_t v_desc = smem_desc_sw128(smem_u32(sKV) + G::kKBytes, G::kKHalf, 1024);
        const uint64_t vt_desc = smem_desc_sw128(smem_u32(sVt), G::kVtBytes, 1024);
        const uint64_t s_desc = smem_desc_sw128(smem_u32(sS), G::kKHalf, 1024);
        uint32_t c = 0, u = 0, s = 0, t = 0;  // chunks of the ring, updates, states, tiles
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            ok = ok && mbar_wait_small(bar, parity, abort_flag);
            return ok;
        };
        auto wait_chunk = [&]() { return wait(&bars->kv_full[c % kRing], (c / kRing) & 1); };
        // the last of a chunk's weighed V (and with it zeros behind the request)
        auto wait_weighed = [&](uint32_t u) {
            const uint32_t w = u * G::kFills + G::kFills - 1;
            return wait(&bars->vt_full[w % kVtBars], (w / kVtBars) & 1);
        };
        auto update = [&]() {
            if (u >= 1 && !wait(&bars->u_empty, (u - 1) & 1)) return;
            const uint32_t d = tmem + G::kColU;
            uint64_t kd = kt_desc + (c % kRing) * (G::kStageBytes >> 4);
#pragma unroll 1
            for (uint32_t w = u * G::kFills; w < (u + 1) * G::kFills; ++w) {
                if (!wait(&bars->vt_full[w % kVtBars], (w / kVtBars) & 1)) return;
                tc_fence_after();
                const uint64_t vd = vt_desc + (w & 1) * (kParts * G::kVtBytes >> 4);
                const uint32_t more = w > u * G::kFills ? 1u : 0u;
                if constexpr (G::kUpdates == 2) {
#pragma unroll
                    for (int kk = 0; kk < kPart / 16; ++kk) {
                        tc_mma(d, kd + kk * (2048 >> 4), vd + kk * (2048 >> 4), idesc_kv2,
                               kk > 0 ? 1u : more);
                        tc_mma(d + kSlice, kd + kk * (2048 >> 4),
                               vd + (2 * G::kVtBytes >> 4) + kk * (2048 >> 4), idesc_kv, 1u);
                    }
                } else {
#pragma unroll 1
                    for (int part = 0; part < kParts; ++part)
#pragma unroll
                        for (int kk = 0; kk < kPart / 16; ++kk)
                            tc_mma(d, kd + kk * (2048 >> 4),
                                   vd + part * (G::kVtBytes >> 4) + kk * (2048 >> 4), idesc_kv,
                                   part + kk > 0 ? 1u : more);
                }
                kd += kPart * 128 >> 4;
                tc_commit(&bars->vt_empty[w & 1]);
            }
            tc_commit(&bars->u_full);
            ++u;
        };
        // Q by K or by S for the tiles of a chunk (one code for both): B's descriptor, and its
        // steps from 16 of the summed dimension to the next and from 64 to the next; the barrier
        // of two tiles ago says that D's columns are free
        auto by_q = [&](uint64_t b_desc, uint32_t step, uint32_t step64, uint32_t d, uint32_t d_next,
                        uint32_t idesc, uint64_t *before, uint64_t *after) {
#pragma unroll 1
            for (int j = 0; j < tiles; ++j, ++t) {
                const uint32_t b = t & 1, slot = t % G::kQBufs;
                if (!wait(&bars->q_full[slot], (t / G::kQBufs) & 1) ||
                    (t >= 2 && !wait(&before[b], ((t >> 1) - 1) & 1)))
                    return;
                tc_fence_after();
                const uint64_t qd = q_desc + slot * (G::kQBytes >> 4);
#pragma unroll 1
                for (int hf = 0; hf < G::kHalves; ++hf)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma(d + b * d_next, qd + hf * (G::kQHalf >> 4) + kk * 2,
                               b_desc + hf * step64 + kk * step, idesc, hf + kk > 0 ? 1u : 0u);
                tc_commit(&after[b]);
                tc_commit(&bars->q_empty[slot]);
            }
        };
        auto inside = [&]() {
#pragma unroll 1
            for (int j = 0; j < tiles; ++j, ++t) {
                const uint32_t b = t & 1, turn = (t >> 1) & 1;
                // (P is there after the outputs of two tiles ago have been read)
                if (!wait(&bars->p_full[b], turn) ||
                    (G::kInsides == 1 && t >= 1 && !wait(&bars->o_empty[b ^ 1], ((t - 1) >> 1) & 1)))
                    return;
                tc_fence_after();
                const uint64_t vd = v_desc + (c % kRing) * (G::kStageBytes >> 4);
#pragma unroll
                for (int kk = 0; kk < C / 16; ++kk)
                    tc_mma_ts(tmem + G::kColI + b % G::kInsides * kSlice, tmem + b * C + kk * 8,
                              vd + (kk * 2048 >> 4), idesc_v, kk > 0 ? 1u : 0u);
                tc_commit(&bars->o_full[b]);
            }
        };
        for (int k = 0;; ++k) {
            const Item it = queue_item(ctl, warp, k);
            if (it.n == 0) break;
            // the rank's chunks, first for their updates alone where others build on them
#pragma unroll 1
            for (int outputs = size > 1 ? 0 : 1; outputs < 2; ++outputs) {
                if (lane == 0 && (outputs || it.c_end < it.chunks))
#pragma unroll 1
                    for (int i = it.c_begin; ok && i < it.c_end && wait_chunk(); ++i, ++c) {
                        if (warp == kWarpKV) update();
                        // (V's weighing zeroes rows behind the request, and what is no number)
                        if (warp == kWarpPV) {
                            wait_weighed(u);
                            ++u;
                        }
                        if (ok && outputs && warp != kWarpKV) {
                            const bool qs = warp == kWarpQS;
                            if (qs) wait(&bars->s_full[s & 1], (s >> 1) & 1);
                            if (warp == kWarpPV)
                                inside();
                            else if (ok)
                                // (Q K^T: the columns hold P of two tiles ago until its P V is done)
                                by_q(qs ? s_desc + (s & 1) * (G::kSBytes >> 4)
                                        : k_desc + (c % kRing) * (G::kStageBytes >> 4),
                                     qs ? 2048 >> 4 : 2, qs ? 8192 >> 4 : G::kKHalf >> 4,
                                     tmem + (qs ? G::kColB : 0), qs ? kSlice : C,
                                     qs ? idesc_v : idesc_qk, qs ? bars->o_empty : bars->o_full,
                                     qs ? bars->o_full : bars->sc_full);
                            if (qs && ok) {
                                tc_commit(&bars->s_empty[s & 1]);
                                ++s;
                            }
                        }
                        if (ok) tc_commit(&bars->kv_empty[c % kRing]);
                    }
                __syncwarp();
                if (!outputs) {
                    cluster_sync();
                    cluster_sync();
                }
            }
        }
        if (lane == 0 && (!ok || *abort_flag)) {
            // MMAs already issued finish before TMEM is released
            uint64_t *drain = &bars->drain[warp == kWarpPV ? 0 : warp];
            tc_commit(drain);
            mbar_drain(drain, 0);
        }
        __syncwarp();
    } else if (warp < kFirstWeigh) {
        // ============================ P and outputs ============================
        const int wq = warp & 3;
        const uint32_t grp = (warp - kFirstOut) / kGroupWarps;  // takes tiles of this parity
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const uint32_t sa = t_lane + grp * C, oa = t_lane + G::kColB + grp * kSlice,
                       ia = t_lane + G::kColI + grp % G::kInsides * kSlice;
        const int tok = (wq * 32 + lane) / G::kHeads, head = (wq * 32 + lane) % G::kHeads;
        // the runs of 16 tokens that the warp's rows lie in
        const int first_run = wq * 32 / G::kHeads / 16, last_run = (wq * 32 + 31) / G::kHeads / 16;
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        uint32_t t = 0, u = 0;  // tiles, updates up to this item
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
            int i = it.c_begin, j = 0;  // chunk, tile of the chunk
#pragma unroll 1
            for (int m = 0; ok && m < total; ++m) {
                const uint32_t tt = t + m;
                if ((tt & 1) == grp) {
                    const uint32_t turn = (tt >> 1) & 1, uu = u + (i - it.c_begin);
                    ok = warp_mbar_wait_small(&bars->tab_full[uu % kVtBars], (uu / kVtBars) & 1, abort_flag) &&
                         warp_mbar_wait_small(&bars->sc_full[grp], turn, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const Table<C> &tab = tables[uu % kTables];
                    // the sum up to the row's token from its run's start, and from first_run's
                    const float gi = tab.sum[tok], *const between = tab.between[tok / 16];
                    const float gi_first = gi + between[first_run];
#pragma unroll 1
                    for (int run = 0; run < C / 16; ++run) {
                        uint32_t pk[8];
#pragma unroll
                        for (int x = 0; x < 8; ++x) pk[x] = 0u;
                        if (run <= last_run) {
                            uint32_t v[16];
                            tmem_ld16(sa + run * 16, v);
                            if (run < first_run) {
                                // e^(G_i - G_j) by way of the run's last token
                                const uint64_t row = f2_twice(fast_exp2(gi + between[run + 1]));
                                tmem_wait_ld();
#pragma unroll
                                for (int x = 0; x < 16; x += 4) {
                                    const float4 f =
                                        *reinterpret_cast<const float4 *>(tab.tail + run * 16 + x);
                                    auto w = [&](int e, float f0, float f1) {
                                        return f2_bf16x2(f2_mul(f2_mul(f2_words(v[x + e], v[x + e + 1]), row),
                                                                f2_pack(f0, f1)));
                                    };
                                    pk[x / 2] = w(0, f.x, f.y);
                                    pk[x / 2 + 1] = w(2, f.z, f.w);
                                }
                            } else {
                                const int lim = tok - run * 16;  // its last visible column
                                const float from_run =
                                    G::kHeads == 1 && run == first_run ? gi_first : gi;
                                const uint64_t minus = f2_twice(-1.f);
                                tmem_wait_ld();
#pragma unroll
                                for (int x = 0; x < 16; x += 4) {
                                    const float4 g =
                                        *reinterpret_cast<const float4 *>(tab.sum + run * 16 + x);
                                    auto w = [&](int e, float g0, float g1) {
                                        float a, b;
                                        f2_unpack(f2_fma(f2_pack(g0, g1), minus, f2_twice(from_run)), a, b);
                                        f2_unpack(f2_mul(f2_words(v[x + e], v[x + e + 1]),
                                                         f2_pack(fast_exp2(a), fast_exp2(b))), a, b);
                                        return pack_bf16x2(x + e <= lim ? a : 0.f,
                                                           x + e + 1 <= lim ? b : 0.f);
                                    };
                                    pk[x / 2] = w(0, g.x, g.y);
                                    pk[x / 2 + 1] = w(2, g.z, g.w);
                                }
                            }
                        }
                        // (over scores that have been read: a run's P takes half their columns)
                        tmem_st8(sa + run * 8, pk);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->p_full[grp]);

                    ok = warp_mbar_wait_small(&bars->o_full[grp], turn, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t before = f2_twice(fast_exp2(gi + between[0]) * p.scale);
                    const uint64_t scale = f2_twice(p.scale);
                    const int token = i * C + tok, hq = j * G::kHeads + head;
                    const bool valid = token < it.n && hq < p.group;
                    uint4 *dst = reinterpret_cast<uint4 *>(
                        p.out + (static_cast<int64_t>(it.t0 + token) * p.num_q_heads +
                                 it.h * p.group + hq) * D + it.slice * kSlice);
#pragma unroll 1
                    for (int part = 0; part < kSlice / 16; ++part) {
                        uint32_t a[16], b[16];
                        __syncwarp();
                        tmem_ld16(oa + part * 16, a);
                        tmem_ld16(ia + part * 16, b);
                        tmem_wait_ld();
                        auto sum = [&](int x) {
                            return f2_bf16x2(f2_fma(before, f2_words(a[x], a[x + 1]),
                                                    f2_mul(scale, f2_words(b[x], b[x + 1]))));
                        };
                        if (valid) {
                            const uint4 lo = make_uint4(sum(0), sum(2), sum(4), sum(6));
                            const uint4 hi = make_uint4(sum(8), sum(10), sum(12), sum(14));
                            if (wide) {
                                store32(dst + part * 2, lo, hi);
                            } else {
                                dst[part * 2] = lo;
                                dst[part * 2 + 1] = hi;
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->o_empty[grp]);
                }
                if (++j == tiles) j = 0, ++i;
            }
            t += total;
            u += it.c_end - it.c_begin;
        }
    } else if (warp < kFirstState) {
        // ============================ V's weights ============================
        const int vw = warp - kFirstWeigh;
        uint32_t w = 0;  // buffers filled
        bool ok = true;
        for (int k = 0;; ++k) {
            const Item it = queue_item(ctl, warp, k);
            if (it.n == 0) break;
#pragma unroll 1
            for (int outputs = size > 1 ? 0 : 1; outputs < 2; ++outputs) {
                const int c_last = outputs || it.c_end < it.chunks ? it.c_end : it.c_begin;
#pragma unroll 1
                for (uint32_t f = 0; ok && f < (c_last - it.c_begin) * G::kFills; ++f, ++w) {
                    const uint32_t u = w / G::kFills;
                    const int st = u % kRing, i = it.c_begin + f / G::kFills;
                    // the chunk is here, and the MMAs of two fills ago have read theirs
                    ok = warp_mbar_wait_small(&bars->kv_full[st], (u / kRing) & 1, abort_flag) &&
                         warp_mbar_wait_small(&bars->tab_full[u % kVtBars], (u / kVtBars) & 1, abort_flag) &&
                         (w < 2 ||
                          warp_mbar_wait_small(&bars->vt_empty[w & 1], ((w >> 1) - 1) & 1, abort_flag));
                    if (!ok) break;
                    const uint32_t half = w % G::kFills * (kPart * 128);
                    uint8_t *k_tile = sKV + st * G::kStageBytes + half, *v = k_tile + G::kKBytes;
                    uint8_t *vt = sVt + (w & 1) * (kParts * G::kVtBytes);
                    const float *weight = tables[u % kTables].weight + w % G::kFills * kPart;
                    const int valid = it.n - i * C - w % G::kFills * kPart;
                    uint32_t rests = 0;
                    // eight lanes to a row of 64 elements
#pragma unroll 1
                    for (int x = 0; x < kPart / (4 * kWeighWarps); ++x) {
                        const int row = vw * (kPart / kWeighWarps) + x * 4 + lane / 8;
                        const uint32_t off = sw128_offset(row, lane % 8);
                        const uint64_t wt = f2_twice(weight[row]);
                        uint4 in = *reinterpret_cast<const uint4 *>(v + off);
                        // rows behind the request are another's, or padding: whatever stands
                        // there does not reach a sum
                        if (row >= valid) {
                            in = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4 *>(v + off) = in;
#pragma unroll
                            for (int hf = 0; hf < G::kHalves; ++hf)
                                *reinterpret_cast<uint4 *>(k_tile + hf * G::kKHalf + off) = in;
                        }
                        uint4 part[kParts];
                        const uint64_t minus = f2_twice(-1.f);
                        auto two = [](uint32_t pair) {
                            return f2_pack(__uint_as_float(pair << 16),
                                           __uint_as_float(pair & 0xFFFF0000u));
                        };
                        auto split = [&](uint32_t pair, uint32_t &p0, uint32_t &p1, uint32_t &p2) {
                            uint64_t y = f2_mul(two(pair), wt);
                            p0 = f2_bf16x2(y);
                            y = f2_fma(two(p0), minus, y);
                            p1 = f2_bf16x2(y);
                            p2 = f2_bf16x2(f2_fma(two(p1), minus, y));
                        };
                        split(in.x, part[0].x, part[1].x, part[2].x);
                        split(in.y, part[0].y, part[1].y, part[2].y);
                        split(in.z, part[0].z, part[1].z, part[2].z);
                        split(in.w, part[0].w, part[1].w, part[2].w);
                        // (the rest of an infinity or a NaN is a NaN)
                        rests |= part[2].x | part[2].y;
                        rests |= part[2].z | part[2].w;
#pragma unroll
                        for (int n = 0; n < kParts; ++n)
                            *reinterpret_cast<uint4 *>(vt + n * G::kVtBytes + off) = part[n];
                    }
                    if (__builtin_expect(finite2(rests) != rests, 0)) {
                        // There may be one (the rests of values from 2^17 on, or-ed, can look like
                        // it too): P V meets a 0 in its place, see late_columns.
#pragma unroll 1
                        for (int x = 0; x < kPart / (4 * kWeighWarps); ++x) {
                            const int row = vw * (kPart / kWeighWarps) + x * 4 + lane / 8;
                            uint32_t *at = reinterpret_cast<uint32_t *>(v + sw128_offset(row, lane % 8));
#pragma unroll 1
                            for (int e = 0; e < 4; ++e)
                                if (finite2(at[e]) != at[e]) {
                                    at[e] = finite2(at[e]);
                                    ctl->odd = 1;
                                }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->vt_full[w % kVtBars]);
                }
                if (!outputs) {
                    cluster_sync();
                    cluster_sync();
                }
            }
        }
    } else if (warp == kWarpScan) {
        // ============================ sums of logarithms ============================
        constexpr int T = C / 32;  // tokens of a lane
        constexpr int kLanes = 16 / T, kRuns = Table<C>::kRuns;  // lanes of a run
        constexpr int kPairs = (kRuns * kRuns + 31) / 32;        // of between[][] to a lane
        const int at = lane % kLanes;
        // 1 where a run belongs to those behind the lane's, to its pair, else 0
        float in_after[kRuns], in_pair[kPairs][kRuns];
#pragma unroll
        for (int x = 0; x < kRuns; ++x) {
            in_after[x] = x > lane / kLanes ? 1.f : 0.f;
#pragma unroll
            for (int y = 0; y < kPairs; ++y) {
                const int e = lane + 32 * y;
                in_pair[y][x] = x >= e % kRuns && x < e / kRuns ? 1.f : 0.f;
            }
        }
        uint32_t c = 0;
        bool ok = true;
        // logarithm (base 2) of the decay of token i of the request
        auto log_of = [&](const Item &it, int i) {
            if (i >= it.n) return 0.f;
            const float g = __ldg(p.decay + static_cast<int64_t>(it.t0 + i) * p.decay_stride + it.h);
            return g < 0.f ? fmaxf(g * 1.4426950408889634f, kLeastLog) : 0.f;
        };
        for (int k = 0;; ++k) {
            const Item it = queue_item(ctl, warp, k);
            if (it.n == 0) break;
#pragma unroll 1
            for (int outputs = size > 1 ? 0 : 1; outputs < 2; ++outputs) {
                const int c_last = outputs || it.c_end < it.chunks ? it.c_end : it.c_begin;
                float g[T] = {}, next[T] = {};
#pragma unroll 1
                for (int i = it.c_begin - 1; ok && i < c_last; ++i) {
#pragma unroll
                    for (int x = 0; x < T; ++x) {
                        g[x] = next[x];
                        if (i + 1 < c_last) next[x] = log_of(it, (i + 1) * C + T * lane + x);  // a chunk ahead
                    }
                    if (i < it.c_begin) continue;
                    // sums in the run up to each token (T to a lane), and of those behind it (each
                    // without a difference, so that a small one keeps its digits beside large ones)
                    float up = g[0];
#pragma unroll
                    for (int x = 1; x < T; ++x) up += g[x];
                    float down = up;
#pragma unroll
                    for (int o = 1; o < kLanes; o <<= 1) {
                        const float a = __shfl_up_sync(0xffffffffu, up, o);
                        const float b = __shfl_down_sync(0xffffffffu, down, o);
                        if (at >= o) up += a;
                        if (at + o < kLanes) down += b;
                    }
                    float sum[T], behind[T];
                    sum[0] = __shfl_up_sync(0xffffffffu, up, 1);
                    behind[T - 1] = __shfl_down_sync(0xffffffffu, down, 1);
                    if (at == 0) sum[0] = 0.f;
                    if (at == kLanes - 1) behind[T - 1] = 0.f;
                    sum[0] += g[0];
#pragma unroll
                    for (int x = 1; x < T; ++x) {
                        sum[x] = sum[x - 1] + g[x];
                        behind[T - 1 - x] = behind[T - x] + g[T - x];
                    }
                    // of whole runs: all, those behind the lane's, and its pairs of between[][]
                    float all = 0.f, after = 0.f, pair[kPairs] = {};
#pragma unroll
                    for (int x = 0; x < kRuns; ++x) {
                        const float run = __shfl_sync(0xffffffffu, sum[T - 1], x * kLanes + kLanes - 1);
                        all += run;
                        after = fmaf(run, in_after[x], after);
#pragma unroll
                        for (int y = 0; y < kPairs; ++y) pair[y] = fmaf(run, in_pair[y][x], pair[y]);
                    }
                    float weight[T];
#pragma unroll
                    for (int x = 0; x < T; ++x) weight[x] = exp2f(behind[x] + after);
                    // (the chunk that had this place in the ring is through its MMAs: who still reads
                    // a table is at most two further behind)
                    ok = c < kRing ||
                         warp_mbar_wait_small(&bars->kv_empty[c % kRing], (c / kRing - 1) & 1, abort_flag);
                    if (!ok) break;
                    Table<C> &tab = tables[c % kTables];
#pragma unroll
                    for (int x = 0; x < T; x += 2) {
                        const int t = T * lane + x;
                        *reinterpret_cast<float2 *>(tab.sum + t) = make_float2(sum[x], sum[x + 1]);
                        *reinterpret_cast<float2 *>(tab.tail + t) =
                            make_float2(fast_exp2(behind[x]), fast_exp2(behind[x + 1]));
                        *reinterpret_cast<float2 *>(tab.weight + t) = make_float2(weight[x], weight[x + 1]);
                    }
#pragma unroll
                    for (int y = 0; y < kPairs; ++y)
                        if (lane + 32 * y < kRuns * kRuns) (&tab.between[0][0])[lane + 32 * y] = pair[y];
                    if (lane == 31) tab.all = all;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->tab_full[c % kVtBars]);
                    ++c;
                }
                if (!outputs) {
                    cluster_sync();
                    cluster_sync();
                }
            }
        }
    } else {
        // ============================ the state ============================
        const int sw = warp - kFirstState, wq = warp & 3, half = sw >> 2;
        const int r = wq * 32 + lane;       // row of the update's MMA, 32 of its columns
        const bool real = r < D;  // (head_dim 64: the MMA's other rows go along unread)
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        uint64_t s[16];  // pairs of columns
        uint32_t u = 0, w = 0;  // updates, states written
        bool ok = true;
        float total = 0.f;  // log2 decay of the chunks gone through

        // the state in bf16, for the MMA that follows
        auto give_state = [&]() {
            if (w >= 2) ok = warp_mbar_wait_small(&bars->s_empty[w & 1], ((w >> 1) - 1) & 1, abort_flag);
            if (!ok) return;
            uint8_t *dst = sS + (w & 1) * G::kSBytes;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *reinterpret_cast<uint4 *>(dst + sw128_offset(r, half * 4 + x)) =
                    make_uint4(f2_bf16x2(s[4 * x]), f2_bf16x2(s[4 * x + 1]),
                               f2_bf16x2(s[4 * x + 2]), f2_bf16x2(s[4 * x + 3]));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->s_full[w & 1]);
            ++w;
        };
        // takes a chunk's update in
        auto update = [&]() {
            ok = warp_mbar_wait_small(&bars->u_full, u & 1, abort_flag) &&
                 warp_mbar_wait_small(&bars->tab_full[u % kVtBars], (u / kVtBars) & 1, abort_flag);
            if (!ok) return;
            tc_fence_after();
            const float all = tables[u % kTables].all;
            const uint64_t keep = f2_twice(exp2f(all));
#pragma unroll
            for (int part = 0; part < 2 * G::kUpdates; ++part) {
                constexpr int K = G::kUpdates;
                uint32_t up[16];
                tmem_ld16(t_lane + G::kColU + part % K * kSlice + half * 32 + part / K * 16, up);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    uint64_t &y = s[part / K * 8 + x];
                    const uint64_t z = f2_words(up[2 * x], up[2 * x + 1]);
                    y = part % K ? f2_add(y, z) : f2_fma(keep, y, z);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->u_empty);
            ++u;
            total += all;
        };
        for (int k = 0;; ++k) {
            const Item it = queue_item(ctl, warp, k);
            if (it.n == 0) break;
            const int64_t place = static_cast<int64_t>(it.h) * D * D + static_cast<int64_t>(r) * D +
                                  it.slice * kSlice + half * 32;
            const int64_t state_size = static_cast<int64_t>(p.num_kv_heads) * D * D;
            float *exchange = reinterpret_cast<float *>(sS) + (half * 32) * kRows + r;
#pragma unroll 1
            for (int outputs = size > 1 ? 0 : 1; outputs < 2; ++outputs) {
                // the state before the run: the request's, and the ranks' before this one; for
                // the updates alone none
                total = 0.f;
                const float4 *src =
                    reinterpret_cast<const float4 *>(p.state + it.in * state_size + place);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const float4 v = outputs && it.in >= 0 && real ? src[x]
                                                                   : make_float4(0.f, 0.f, 0.f, 0.f);
                    s[2 * x] = f2_pack(v.x, v.y);
                    s[2 * x + 1] = f2_pack(v.z, v.w);
                }
                if (outputs && size > 1) {
                    if (it.c_begin < it.c_end)
#pragma unroll 1
                        for (int other = 0; other < rank; ++other) {
                            const uint64_t keep = f2_twice(exp2f(ld_cluster_f1(&ctl->decay, other)));
                            const uint32_t theirs = cluster_addr(exchange, other);
#pragma unroll
                            for (int x = 0; x < 16; ++x)
                                s[x] = f2_fma(keep, s[x],
                                              f2_pack(ld_cluster_at(theirs + 2 * x * kRows * 4),
                                                      ld_cluster_at(theirs + (2 * x + 1) * kRows * 4)));
                        }
                    cluster_sync();
                }
                const int c_last = outputs || it.c_end < it.chunks ? it.c_end : it.c_begin;
#pragma unroll 1
                for (int i = it.c_begin; ok && i < c_last; ++i) {
                    if (outputs) give_state();
                    if (ok) update();
                }
                if (!outputs) {
                    if (c_last > it.c_begin) {
                        // (the MMAs of the item before have read both states)
                        for (uint32_t x = 0; ok && x < 2; ++x)
                            if (w > x) {
                                const uint32_t last = w - 1 - x;
                                ok = warp_mbar_wait_small(&bars->s_empty[last & 1], (last >> 1) & 1,
                                                          abort_flag);
                            }
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            f2_unpack(s[x], exchange[2 * x * kRows], exchange[(2 * x + 1) * kRows]);
                        if (sw == 0 && lane == 0) ctl->decay = total;
                    }
                    cluster_sync();
                }
            }
            if (it.c_begin == it.c_end || it.c_end < it.chunks) continue;
            // the last rank has the state behind the request
            if (ok && real && it.to >= 0) {
                float4 *dst = reinterpret_cast<float4 *>(p.state + it.to * state_size + place);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    float4 v;
                    f2_unpack(s[2 * x], v.x, v.y);
                    f2_unpack(s[2 * x + 1], v.z, v.w);
                    dst[x] = v;
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*abort_flag && tid == 0) flag_status(p.status, PA_DEV_WAIT_TIMEOUT);
    if (warp == kWarpQK) tmem_dealloc(tmem, G::kTmemCols);
    if (ctl->odd && !*abort_flag) late_columns<D, C>(p, rank, size);
}

namespace {

template <int D, int C, bool CLUSTER>
int launch(const LinearParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
           const CUtensorMap &tv, int clusters, int size, cudaStream_t s) {
    static PerDeviceOnce once;
    if (once_per_device(once, [] {
            return cudaFuncSetAttribute(linear_prompt_kernel<D, C, CLUSTER>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        Geom<D, C>::kSmemBytes);
        }) != PA_OK)
        return PA_ERR_CUDA;
    PdlLaunch l(clusters * size, kThreads, Geom<D, C>::kSmemBytes, s);
    if (CLUSTER) l.set_cluster(size);
    return launch_kernel(l, linear_prompt_kernel<D, C, CLUSTER>, p, tq, tk, tv, size) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

template <int D, int C>
int launch(const LinearParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
           const CUtensorMap &tv, int sms, cudaStream_t s) {
    // the most requests that can be long, and their items (at least one of each: the caller has
    // more than max_rows tokens and a request)
    const int64_t tokens = p.num_tokens;
    const int64_t longs = std::min<int64_t>(p.num_seqs, tokens / (p.max_rows + 1));
    const int64_t items = longs * p.num_kv_heads * (D / kSlice);
    // the largest cluster whose ranks have two chunks and whose items run at once (152 SMs hold 76
    // clusters of 2, 36 of 4 and 15 of 8: a ninth of the SMs belongs to none of 8)
    int size = 1;
    while (size < kDirectMaxCluster && 2 * size * 2 * C <= tokens &&
           2 * size * items <= (size < 4 ? sms * 18 / 19 : sms * 15 / 19))
        size *= 2;
    // Which requests are long is known on the GPU only, so the two forms' SMs are shared out by
    // what T tokens and B states would take: reading and writing a state counts as 24 tokens of a
    // prompt.  (Measured apart an SM takes 35 to 46 times a token's time for it, with 32 kv heads,
    // either head_dim and groups of 1, 2 and 4 heads, so neither enters.  Counted as 24 / 40, us: 8 x
    // 512 tokens beside 224 short rows of 32 / 8 heads 78.9 / 77.6, of 16 / 16 126 / 124, of 32 / 8
    // heads of 64 34.2 / 33.8; 32 x 40 beside 80, of 32 / 8 41.3 / 42.3, of 16 / 16 76 / 80, of 6 / 6 of
    // 64 15.7 / 16.7.)  256 single tokens, without any prompt: 47.6 us, 60 with a prompt CTA on
    // every SM.
    // Above kLinearFewRows tokens on average some request is likely to be long, and all may be, of
    // one short chunk each, which takes as long as a full one: tokens count four times then.  8 x 512
    // tokens among 224 requests of 1 and 5 take 75.7 / 79.2 / 80.5 us with tokens counted once, four
    // and eight times, 64 requests of 16 96 / 58 / 49, 128 of 32 137 / 96 / 91.
    constexpr int64_t kStateTokens = 24;
    const int64_t work = tokens > int64_t{kLinearFewRows} * p.num_seqs ? 4 * tokens : tokens;
    const int share = static_cast<int>(sms * work / (work + kStateTokens * p.num_seqs));
    const int clusters = static_cast<int>(std::min<int64_t>(items, std::max(1, share / size)));
    return size > 1 ? launch<D, C, true>(p, tq, tk, tv, clusters, size, s)
                    : launch<D, C, false>(p, tq, tk, tv, clusters, 1, s);
}

}  // namespace

int launch_linear_prompt(const LinearParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                         const CUtensorMap &tv, int head_dim, int sms, cudaStream_t s) {
    if (p.chunk == 64)
        return head_dim == 128 ? launch<128, 64>(p, tq, tk, tv, sms, s)
                               : launch<64, 64>(p, tq, tk, tv, sms, s);
    return head_dim == 128 ? launch<128, 128>(p, tq, tk, tv, sms, s)
                           : launch<64, 128>(p, tq, tk, tv, sms, s);
}

}  // namespace pa
