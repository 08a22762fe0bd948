// pa_api.cu -- the C ABI of libpa (declared in include/pa.h): argument checks,
// TMA tensor maps, workspace layout and the launch sequence of one step.
// Every step of the path runs in this library's kernels; nothing here
// computes on the host beyond integer bookkeeping.
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <algorithm>
#include <atomic>
#include <mutex>
#include <vector>

#include "pa_internal.cuh"

using namespace pa;

// Per-device status word (PA_DEV_* bits).  Host code passes its device
// address to the kernels; pa_read_device_status reads it back.
__device__ unsigned int g_pa_status;

namespace {

thread_local char g_err[256] = "";

int fail(int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return code;
}

constexpr int kMaxDevices = 64;

struct DeviceInfo {
    bool ready = false;
    int sms = 0;
    int short_ctas_per_sm[2][3] = {};  // [windowed][bf16 head_dim 64, bf16 128, fp8 128]
    unsigned *status = nullptr;
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

int device_info(DeviceInfo **out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return fail(PA_ERR_CUDA, "no current CUDA device");
    std::lock_guard<std::mutex> lock(g_dev_mu);
    DeviceInfo &d = g_dev[dev];
    if (!d.ready) {
        void *sym = nullptr;
        if (cudaGetSymbolAddress(&sym, g_pa_status) != cudaSuccess)
            return fail(PA_ERR_CUDA, "cudaGetSymbolAddress(status) failed");
        d.status = static_cast<unsigned *>(sym);
        if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return fail(PA_ERR_CUDA, "cannot query SM count");
        for (int w = 0; w < 2; ++w) {
            d.short_ctas_per_sm[w][0] = short_max_ctas_per_sm(64, false, w != 0);
            d.short_ctas_per_sm[w][1] = short_max_ctas_per_sm(128, false, w != 0);
            d.short_ctas_per_sm[w][2] = short_max_ctas_per_sm(128, true, w != 0);
        }
        d.ready = true;
    }
    *out = &d;
    return PA_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// 2-D view of one cache array: rows = (block, kv head, offset) flattened,
// head_dim columns; boxes of 16 rows x 128 bytes (64 bf16 or 128 e4m3
// columns), 128-byte swizzle.
int make_kv_map(CUtensorMap *m, void *base, int64_t rows, int head_dim, bool fp8) {
    auto fn = encode_fn();
    if (!fn) return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
    const int esize = fp8 ? 1 : 2;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(head_dim) * esize};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / esize), static_cast<cuuint32_t>(kChunkKeys)};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                    base, dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PA_OK : fail(PA_ERR_CUDA, "KV tensor map encode failed (%d)", (int)r);
}

// 3-D view of q [tokens][q heads][head_dim]; a box is 64 dims x group heads x
// tile tokens, i.e. the 128 (token, head) rows of one tensor-core tile.
int make_q_map(CUtensorMap *m, const void *q, int tokens, int heads, int head_dim, int group,
               int tile_tokens) {
    auto fn = encode_fn();
    if (!fn) return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(heads),
                          static_cast<cuuint64_t>(tokens > 0 ? tokens : 1)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_dim) * 2,
                             static_cast<cuuint64_t>(heads) * head_dim * 2};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(tile_tokens)};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides,
                    box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PA_OK : fail(PA_ERR_CUDA, "Q tensor map encode failed (%d)", (int)r);
}

std::atomic<unsigned long long> g_launches{0};
std::atomic<int> g_test_stall{PA_TEST_STALL_NONE};  // pa_set_test_stall
std::atomic<uint64_t *> g_tile_counter{nullptr};     // pa_set_tile_counter

// Profiling hook state (pa_set_profile_events).
void *g_prof[4][2] = {};
std::mutex g_prof_mu;

struct ProfScope {
    int which;
    cudaStream_t s;
    void *end;
    ProfScope(int w, cudaStream_t st) : which(w), s(st), end(nullptr) {
        void *start;
        {
            std::lock_guard<std::mutex> lock(g_prof_mu);
            start = g_prof[w][0];
            end = g_prof[w][1];
        }
        if (start) cudaEventRecord(static_cast<cudaEvent_t>(start), s);
    }
    ~ProfScope() {
        if (end) cudaEventRecord(static_cast<cudaEvent_t>(end), s);
    }
};

// Fewest query tokens for which a step runs its split-KV and tensor-core
// kernels side by side (below it they run one after the other).
constexpr int kSideBySideMinTokens = 512;
// In a windowed step the short rows' work is bounded too: with fewer chunks than
// this, if every request were a decode row, there is nothing for the extra grids
// to overlap.  32 q / 8 kv heads, side by side / one after the other: a chunk of
// 1024 tokens at window 128 29 / 21 us, at window 4096 76 / 72; 4 chunks of 512 and
// 72 decode and verify rows 50 / 46 us at window 16 (2.4 k chunks), 60 / 65 at 128
// (6.7 k), 227 / 291 at 4096.  8 / 2 heads, the same rows: 43 / 38 us at window 512
// (5.3 k), 94 / 99 at 4096 (39 k).
constexpr int64_t kSideBySideMinChunks = 6144;

// A windowed bf16 step of at most this many requests needs no plan (see run_step): the
// tensor-core kernel finds the tiles itself (a lane per request), and CTAs are launched
// for all pieces that its requests might have as short rows.  32 q / 8 kv heads, without
// / with a plan: one chunk of 256 tokens at window 128 11.0 / 14.4 us, of 1024 at window
// 1024 31.8 / 34.3.  With 32 requests, most of them verify rows, the CTAs without a piece
// cost more than the plan (29.6 / 25.4).
constexpr int kOwnPlanMaxSeqs = 8;
static_assert(kOwnPlanMaxSeqs <= 32, "a lane per request");
// More tiles gain more from the plan's counter: 3 chunks of 2048 tokens, 8 kv heads, window
// 512 (1536 tiles) 104 us without a plan, 100 with; one of 1024 (256 tiles) 25 / 28.
constexpr int kOwnPlanTilesPerSm = 6;

// A windowed step of groups of at most 16 runs as one kernel (window_direct_kernel)
// in place of the plan and the planned kernels (times: one kernel / planned)
//  * whatever its requests are, when its pieces (of 16 rows), kv heads and windows
//    bound its work to kDirectAnyChunks chunks on at most kDirectJobsPerSm jobs per
//    SM, or its jobs fill one round and its work kDirectRoundChunks: a lone token at
//    window 128 5.7 / 11.5 us, 24 verify requests 7.8 / 20.6.  e4m3 pools, whose
//    prompts are staged as bf16 first: 128 tokens of 32 q / 8 kv heads at window 512
//    14.1 / 23.3, 512 tokens of 8 / 2 heads at window 1024 20.5 / 25.6.  In bf16
//    steps of few requests the other form has no plan either (see run_step) and the
//    bounds are closer: 64 tokens (136 jobs) at window 1024 16.2 / 17.6, 128 (264 jobs)
//    at window 128 10.6 / 10.9 and at 512 15.4 / 14.1, 256 (520 jobs) at window 16
//    14.8 / 10.5; at head_dim 64 128 tokens at window 512 11.3 / 12.5;
//  * beyond that when it has few rows, or on average no more than a piece's per
//    request (or two pieces', of little work): a chunk of 64 tokens at window 4096
//    33 / 40 us, but of 128 57 / 41; 16 verify requests of 20 rows at window 1024 16 /
//    23.  Decode, 8 kv heads, d = 128: 16 requests at window 1024 18 / 28 us, 64 50 /
//    68, 256 at window 700 126 / 155 and at 128 40 / 73;
//  * on e4m3 pools, where decoding the codes bounds both, the latter only while there
//    is little to decode: 32 requests at window 2048 36 / 43 us, 64 at 4096 115 / 107.
// The averages are over all requests, empty ones too, so that a long chunk among many
// decode rows or empty slots goes along, in pieces of 16 rows: 192 decode rows and a chunk
// of 512 at window 128 51 / 67 us, at 1024 177 / 161, at 4096 576 / 498; a chunk of 4096
// tokens in a batch padded to 1024 requests 125 / 59, 358 / 95 and 1150 / 248.
constexpr int64_t kDirectAnyChunks = 4096;
constexpr int64_t kDirectAnyChunksE4m3 = 6144;
constexpr int64_t kDirectJobsPerSm = 7;
constexpr int64_t kDirectRoundChunks = 16384;
constexpr int64_t kDirectAnyRows = 256;
constexpr int64_t kDirectE4m3Chunks = 65536;

// ... and short rows alone (no request can be long) leave it when their windows are long
// and they are few: a job gets 8 CTAs at most, while the plan's splits take every SM, with a
// fold that grows with the rows.  More chunks a job than kDirectLongPerRow times a request's
// rows, and than kDirectLongPerJob times the jobs, go there.  d = 128, one kernel / planned,
// bf16: one job of 4 rows at 8192 keys 19 / 21 us, 16384 30 / 27, 32768 51 / 37, 131072 179 /
// 71; 8 jobs at 16384 31 / 32, 32768 53 / 44, 131072 181 / 99; 16 jobs at 32768 57 / 60, 65536
// 105 / 99; 32 at 65536 165 / 169.  One job of 8 rows at 32768 52 / 60, 131072 180 / 108; two of
// 16 at 65536 96 / 111, 131072 182 / 121.  e4m3: one job of 4 rows at 16384 29 / 27, 131072 178 /
// 66; 16 jobs at 16384 34 / 33, 65536 114 / 68; 32 at 32768 64 / 67.  (A table wider than its
// requests' contexts counts in full: the host does not know the lengths.)
constexpr int64_t kDirectLongPerRow = 256;
constexpr int64_t kDirectLongPerJob = 192;
constexpr int64_t kDirectLongPerJobE4m3 = 64;

// True while per-kernel profiling events are set: the step then launches its
// kernels one after the other so that each event pair times one kernel.
bool profiling_active() {
    std::lock_guard<std::mutex> lock(g_prof_mu);
    return g_prof[PA_KERNEL_SPLIT_KV][0] || g_prof[PA_KERNEL_TENSOR_CORE][0];
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int q_tile_tokens(int group) { return group <= kLongRows ? kLongRows / group : 0; }

// Query tokens per split-KV piece (a piece fills at most kShortMaxRows rows),
// and a bound on the pieces of a step with these sizes.
int piece_tokens_for(int group, int rows = kShortMaxRows) {
    return std::max(1, rows / std::max(1, group));
}
int pieces_bound(int num_seqs, int num_q_tokens, int group, int rows = kShortMaxRows) {
    const int pt = piece_tokens_for(group, rows);
    return num_seqs + (num_q_tokens + pt - 1) / pt;
}

// prefix_rows > 0: room for the cascade prefix pass's split states;
// with_extra: room for cascade decode's fp32 suffix state ([T*Hq] rows).
WsLayout make_layout(int num_seqs, int num_q_tokens, int num_q_heads, int num_kv_heads,
                     int head_dim, int prefix_rows, bool with_extra) {
    WsLayout L{};
    const int group = num_q_heads / num_kv_heads;
    const int tq = q_tile_tokens(group);
    const int pieces = pieces_bound(num_seqs, num_q_tokens, group);
    L.max_short = num_kv_heads * (num_seqs * 8 + pieces) + 4096;
    L.max_long = num_kv_heads * ((num_q_tokens + tq - 1) / tq + num_seqs);
    L.cap_rows = L.max_short * 4;
    L.num_counters = num_kv_heads * std::max(1, pieces);
    size_t off = 0;
    L.header = off;
    off = align256(off + sizeof(PlanHeader));
    L.counters = off;
    off = align256(off + sizeof(int) * static_cast<size_t>(L.num_counters));
    L.short_items = off;
    off = align256(off + sizeof(ShortItem) * static_cast<size_t>(L.max_short));
    L.long_items = off;
    off = align256(off + sizeof(LongItem) * static_cast<size_t>(L.max_long));
    L.partial_o = off;
    off = align256(off + sizeof(float) * static_cast<size_t>(L.cap_rows) * head_dim);
    L.partial_lse = off;
    off = align256(off + sizeof(float) * static_cast<size_t>(L.cap_rows));
    L.stage_base = off;
    off = align256(off + sizeof(int) * static_cast<size_t>(num_seqs > 0 ? num_seqs : 1));
    L.stage_list = off;
    off = align256(off + sizeof(int) * static_cast<size_t>(num_seqs > 0 ? num_seqs : 1));
    if (with_extra) {
        const size_t rows = static_cast<size_t>(num_q_tokens) * num_q_heads;
        L.extra_o = off;
        off = align256(off + sizeof(float) * rows * head_dim);
        L.extra_lse = off;
        off = align256(off + sizeof(float) * rows);
    }
    if (prefix_rows > 0) {
        L.prefix_o = off;
        off = align256(off + sizeof(float) * static_cast<size_t>(prefix_rows) * head_dim);
        L.prefix_lse = off;
        off = align256(off + sizeof(float) * static_cast<size_t>(prefix_rows));
    }
    L.total = off;
    return L;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// need_scales: false for calls that move codes without their values.
int check_kv(const pa_kv_desc *kv, bool need_scales = true) {
    if (!kv) return fail(PA_ERR_INVALID_ARG, "kv descriptor is NULL");
    if (!kv->k_cache || !kv->v_cache) return fail(PA_ERR_INVALID_ARG, "cache pointer is NULL");
    if (!aligned(kv->k_cache, 16) || !aligned(kv->v_cache, 16))
        return fail(PA_ERR_INVALID_ARG, "cache pointers must be 16-byte aligned");
    if (kv->num_blocks <= 0 || kv->num_kv_heads <= 0)
        return fail(PA_ERR_INVALID_ARG, "num_blocks and num_kv_heads must be positive");
    if (kv->head_dim != 64 && kv->head_dim != 128)
        return fail(PA_ERR_UNSUPPORTED, "head_dim %d not built (64 or 128)", kv->head_dim);
    if (kv->block_size <= 0 || kv->block_size % 16 != 0 || kv->block_size > 256)
        return fail(PA_ERR_UNSUPPORTED, "block_size %d: need a multiple of 16, at most 256",
                    kv->block_size);
    if (kv->reserved != 0) return fail(PA_ERR_INVALID_ARG, "pa_kv_desc.reserved must be 0");
    if (kv->kv_dtype == PA_KV_FP8_E4M3) {
        if (kv->head_dim != 128)
            return fail(PA_ERR_UNSUPPORTED, "fp8 KV pool: head_dim %d not built (128)", kv->head_dim);
        if (need_scales &&
            (!kv->k_scale || !kv->v_scale || !aligned(kv->k_scale, 4) || !aligned(kv->v_scale, 4)))
            return fail(PA_ERR_INVALID_ARG, "fp8 KV pool needs 4-byte aligned k_scale and v_scale");
    } else if (kv->kv_dtype != PA_KV_BF16) {
        return fail(PA_ERR_UNSUPPORTED, "kv_dtype %d unknown", kv->kv_dtype);
    }
    const int64_t rows = static_cast<int64_t>(kv->num_blocks) * kv->num_kv_heads * kv->block_size;
    if (rows >= (static_cast<int64_t>(1) << 31) - 256)
        return fail(PA_ERR_UNSUPPORTED, "pool too large: %lld cache rows", (long long)rows);
    return PA_OK;
}

int check_heads(const pa_kv_desc *kv, int num_q_heads) {
    if (num_q_heads <= 0 || num_q_heads % kv->num_kv_heads != 0)
        return fail(PA_ERR_INVALID_ARG, "num_q_heads %d is not a multiple of num_kv_heads %d",
                    num_q_heads, kv->num_kv_heads);
    const int group = num_q_heads / kv->num_kv_heads;
    if (group > kLongRows || group > 255)
        return fail(PA_ERR_UNSUPPORTED, "group size %d too large", group);
    return PA_OK;
}

int64_t kv_rows(const pa_kv_desc *kv) {
    return static_cast<int64_t>(kv->num_blocks) * kv->num_kv_heads * kv->block_size;
}

struct StepMaps {
    CUtensorMap q, k, v;
};

// bf16 staging copy of the long requests' blocks of an fp8 pool: the part of
// the caller's workspace beyond the step's own layout (cap blocks for K and
// for V, [cap][Hkv][bs][d] each).
struct Staging {
    int cap = 0;
    void *k = nullptr, *v = nullptr;
    CUtensorMap tk, tv;
};

size_t stage_block_bytes(const pa_kv_desc *kv) {
    return static_cast<size_t>(kv->num_kv_heads) * kv->block_size * kv->head_dim * 2;
}

// Carves the staging area out of workspace bytes [used, total).
int make_staging(Staging *st, const pa_kv_desc *kv, uint8_t *ws, size_t used, size_t total) {
    st->cap = 0;
    if (kv->kv_dtype != PA_KV_FP8_E4M3 || !ws) return PA_OK;
    const size_t start = align256(used);
    const size_t blk = stage_block_bytes(kv);
    if (total < start + 512 + 2 * blk) return PA_OK;
    size_t cap = (total - start - 512) / (2 * blk);
    const size_t max_rows = (static_cast<size_t>(1) << 31) - 256;
    cap = std::min(cap, max_rows / (static_cast<size_t>(kv->num_kv_heads) * kv->block_size));
    cap = std::min<size_t>(cap, 1u << 28);
    st->cap = static_cast<int>(cap);
    st->k = ws + start;
    st->v = ws + start + align256(cap * blk);
    const int64_t rows = static_cast<int64_t>(cap) * kv->num_kv_heads * kv->block_size;
    int rc = make_kv_map(&st->tk, st->k, rows, kv->head_dim, false);
    if (rc == PA_OK) rc = make_kv_map(&st->tv, st->v, rows, kv->head_dim, false);
    return rc;
}

// Cascade decode on an e4m3 pool: the shared prefix decoded to bf16 for the
// tensor-core prefix pass, in the workspace beyond the call's own layout:
// the identity block list ident[k] = k (n int32), then n staging blocks of K
// and of V.  n = 0: a bf16 pool or an empty prefix (nothing staged).
struct PrefixStage {
    int n = 0;
    int32_t *ident = nullptr;
    Staging stg;
};

size_t prefix_stage_bytes(int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                          int32_t prefix_len) {
    const int64_t n = (static_cast<int64_t>(prefix_len) + block_size - 1) / block_size;
    if (n == 0) return 0;
    const size_t blk = static_cast<size_t>(num_kv_heads) * block_size * head_dim * 2;
    return align256(sizeof(int32_t) * static_cast<size_t>(n)) +
           2 * align256(static_cast<size_t>(n) * blk) + 768;
}

int make_prefix_stage(PrefixStage *ps, const pa_kv_desc *kv, int32_t prefix_len, uint8_t *ws,
                      size_t used, size_t total) {
    ps->n = 0;
    if (kv->kv_dtype != PA_KV_FP8_E4M3 || prefix_len == 0) return PA_OK;
    const int n = static_cast<int>((static_cast<int64_t>(prefix_len) + kv->block_size - 1) /
                                   kv->block_size);
    const size_t start = align256(used);
    const size_t need =
        start + prefix_stage_bytes(kv->num_kv_heads, kv->head_dim, kv->block_size, prefix_len);
    if (total < need)
        return fail(PA_ERR_WORKSPACE,
                    "an e4m3 pool's shared prefix is decoded to bf16 in the workspace: it needs "
                    "%zu bytes (pa_cascade_workspace_size + pa_cascade_fp8_staging_bytes), got %zu",
                    need, total);
    ps->ident = reinterpret_cast<int32_t *>(ws + start);
    int rc = make_staging(&ps->stg, kv, ws, start + align256(sizeof(int32_t) * n), total);
    if (rc != PA_OK) return fail(rc, "prefix staging map failed");
    if (ps->stg.cap < n) return fail(PA_ERR_WORKSPACE, "prefix staging area too small");
    ps->n = n;
    return PA_OK;
}

// Decodes the prefix into the staging area (a launch on `s`) and points the
// prefix pass at it: the identity list, the staging blocks and the pool's
// scales.  The pass's K and V tensor maps become *tk and *tv.
int stage_prefix(const PrefixStage &ps, const pa_kv_desc *kv, const int32_t *prefix_blocks,
                 LongParams *lp, const CUtensorMap **tk, const CUtensorMap **tv,
                 DeviceInfo *dev, cudaStream_t s) {
    if (ps.n == 0) return PA_OK;
    const int rc = launch_stage_prefix_fp8(kv, prefix_blocks, ps.n, ps.ident, ps.stg.k,
                                           ps.stg.v, dev->status, 2 * dev->sms, s);
    if (rc != PA_OK) return fail(rc, "prefix staging launch failed");
    lp->block_tables = ps.ident;
    lp->num_blocks = ps.stg.cap;
    lp->kv_rows = ps.stg.cap * kv->num_kv_heads * kv->block_size;
    lp->k_scale = kv->k_scale;
    lp->v_scale = kv->v_scale;
    *tk = &ps.stg.tk;
    *tv = &ps.stg.tv;
    return PA_OK;
}

// need_q: only the tensor-core kernel reads q through a map
int make_maps(StepMaps *m, const void *q, const pa_kv_desc *kv, int tokens, int heads,
              bool need_q = true) {
    const int group = heads / kv->num_kv_heads;
    const bool fp8 = kv->kv_dtype == PA_KV_FP8_E4M3;
    int rc = make_kv_map(&m->k, kv->k_cache, kv_rows(kv), kv->head_dim, fp8);
    if (rc == PA_OK) rc = make_kv_map(&m->v, kv->v_cache, kv_rows(kv), kv->head_dim, fp8);
    if (rc == PA_OK && need_q)
        rc = make_q_map(&m->q, q, tokens, heads, kv->head_dim, group, q_tile_tokens(group));
    return rc;
}

int prefix_plan(int T, int prefix_len, int num_kv_heads, int group, int sms, int *q_tiles,
                int *nsplit, int *split_keys) {
    const int tq = q_tile_tokens(group);
    *q_tiles = (T + tq - 1) / tq;
    const int tiles = (prefix_len + kLongKeys - 1) / kLongKeys;
    const int pairs = num_kv_heads * *q_tiles;
    // the prefix kernel is persistent (one CTA per SM): split the key range so
    // that every (kv head, query tile, split) item gets an SM of its own
    int ns = std::max(1, sms / std::max(1, pairs));
    ns = std::max(1, std::min(ns, std::min(64, tiles)));
    const int per = std::max(1, (tiles + ns - 1) / ns);  // KV tiles per split (an empty prefix: 1)
    *split_keys = per * kLongKeys;
    *nsplit = (prefix_len + *split_keys - 1) / *split_keys;
    if (*nsplit < 1) *nsplit = 1;
    return PA_OK;
}

// Parameters of the shared-prefix ("multi-query") pass: items are (kv head,
// query tile, key split), implicit in the index; split states go to
// (split_o, split_lse) at row (pair * nsplit + split) * 128 + r.
LongParams prefix_params(const pa_kv_desc *kv, const int32_t *prefix_blocks, int32_t prefix_len,
                         int32_t T, int32_t Hq, float scale, int q_tiles, int nsplit,
                         int split_keys, float *split_o, float *split_lse, DeviceInfo *dev) {
    const int group = Hq / kv->num_kv_heads;
    LongParams lp{};
    lp.block_tables = prefix_blocks;
    lp.bt_stride = 0;
    lp.num_q_tokens = T;
    lp.num_q_heads = Hq;
    lp.num_kv_heads = kv->num_kv_heads;
    lp.group = group;
    lp.q_tile_tokens = q_tile_tokens(group);
    lp.block_size = kv->block_size;
    lp.num_blocks = kv->num_blocks;
    lp.kv_rows = static_cast<int>(kv_rows(kv));
    lp.scale_log2 = scale * 1.4426950408889634f;
    lp.prefix_mode = 1;
    lp.prefix_len = prefix_len;
    lp.prefix_nsplit = nsplit;
    lp.prefix_split_keys = split_keys;
    lp.prefix_q_tiles = q_tiles;
    lp.partial_o = split_o;
    lp.partial_lse = split_lse;
    lp.status = dev->status;
    return lp;
}

// Cascade decode: the shared prefix and where its states and the suffix
// states live in the workspace.
struct CascadeArgs {
    const int32_t *prefix_blocks;
    int32_t prefix_len;
    const PrefixStage *ps;  // an e4m3 pool's prefix, decoded to bf16 (ps->n = 0: none)
    float *prefix_o, *prefix_lse;  // prefix split states
    float *suffix_o, *suffix_lse;  // suffix state per row, fp32
};

// The step's new K/V rows, for the call that writes them and attends.
struct NewRows {
    const void *k, *v;
    const int64_t *slots;
    int32_t num_tokens;
};

// Checks of pa_write_kv's arguments; num_tokens == 0 needs no pointers.
int check_new_rows(const NewRows &nr) {
    if (nr.num_tokens < 0) return fail(PA_ERR_INVALID_ARG, "num_tokens < 0");
    if (nr.num_tokens == 0) return PA_OK;
    if (!nr.k || !nr.v || !nr.slots) return fail(PA_ERR_INVALID_ARG, "NULL input");
    if (!aligned(nr.k, 16) || !aligned(nr.v, 16))
        return fail(PA_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
    return PA_OK;
}

// Longest block table of a windowed call, in keys (int32 arithmetic on keys
// then never overflows), and most axes of a rotary embedding.
constexpr int64_t kMaxWindowKeys = static_cast<int64_t>(1) << 30;
constexpr int kMaxRopeAxes = 8;

int check_window(int32_t window, int32_t num_sinks, float scale) {
    if (window < 1) return fail(PA_ERR_INVALID_ARG, "window %d: need at least 1", window);
    if (num_sinks < 0) return fail(PA_ERR_INVALID_ARG, "num_sinks < 0");
    if (!(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f))
        return fail(PA_ERR_INVALID_ARG, "scale must be positive and finite");
    return PA_OK;
}

// Most chunks that `tokens` consecutive rows see: their sinks' and their windows' (cut
// anywhere), at most a whole table's.
int64_t seen_chunks(const WindowArgs &win, int tokens, int max_blocks, int block_size) {
    const int64_t table = static_cast<int64_t>(max_blocks) * block_size / kChunkKeys;
    const int64_t seen = (static_cast<int64_t>(win.sinks) + kChunkKeys - 1) / kChunkKeys +
                         (static_cast<int64_t>(win.window) + tokens) / kChunkKeys + 2;
    return std::min(table, seen);
}

// The one-kernel form's warps per job (one, or all of 1, 2, 4 or 8 CTAs) and CTAs per SM:
// the fewest rounds times a CTA's time, from what was measured in units of a chunk of
// one warp (0.67 us): 7 for its start and fold, half a unit more per CTA of a cluster
// and 10 for warps on their own, and a chunk half as long again for each further CTA on
// the SM.  (8 jobs at window 1024: 15.9, 11.8, 9.7 and 9.3 us with 1, 2, 4 and 8 CTAs; at
// window 64 6.1, 5.9, 6.6 and 7.6; 384 jobs at window 1024 36 us with three CTAs per SM,
// one round, and 47 with two; 1024 jobs at window 128 21 us with a warp each, 29 with a
// CTA.)
void direct_shape(int64_t jobs, int64_t chunks, int sms, DirectParams *dp) {
    int64_t best = -1;
    for (int per = 2; per <= 3; ++per)
        for (int c = 0; c <= (per == 2 ? kDirectMaxCluster : kDirectMaxCluster / 2);
             c = c == 0 ? 1 : 2 * c) {
            const int64_t warps = c == 0 ? 1 : kDirectWarps * c;
            const int64_t per_warp = (chunks + warps - 1) / warps;
            const int64_t ctas = (jobs * warps + kDirectWarps - 1) / kDirectWarps;
            const int64_t slots = static_cast<int64_t>(per) * sms;
            const int64_t on_sm = std::min<int64_t>(per, (ctas + sms - 1) / sms);
            const int64_t start = c == 0 ? 20 : c == 1 ? 14 : 14 + c;  // half units
            const int64_t time = (ctas + slots - 1) / slots * (per_warp * (on_sm + 1) + start);
            if (best < 0 || time < best) {
                best = time;
                dp->cluster = c;
                dp->per_sm = per;
            }
        }
}

// Whether a windowed step is one for the one-kernel form, and its launch.
bool direct_step(const WindowArgs &win, int num_seqs, int T, const pa_kv_desc *kv, int group,
                 int max_blocks, int sms, DirectParams *dp) {
    if (group > kDirectRows || num_seqs > kDirectMaxSeqs) return false;
    dp->piece_tokens = piece_tokens_for(group, kDirectRows);
    dp->max_pieces = std::min(T, pieces_bound(num_seqs, T, group, kDirectRows));
    dp->max_keys = max_blocks * kv->block_size;
    const int64_t chunks = seen_chunks(win, dp->piece_tokens, max_blocks, kv->block_size);
    const int64_t jobs = static_cast<int64_t>(dp->max_pieces) * kv->num_kv_heads;
    const int64_t rows = static_cast<int64_t>(T) * group;
    const bool e4m3 = kv->kv_dtype == PA_KV_FP8_E4M3;
    const int64_t work = jobs * chunks;
    if (rows <= kShortMaxRows &&
        chunks > std::max(kDirectLongPerRow * ((rows + num_seqs - 1) / num_seqs),
                          (e4m3 ? kDirectLongPerJobE4m3 : kDirectLongPerJob) * num_seqs *
                              kv->num_kv_heads))
        return false;
    bool any;
    if (!e4m3 && num_seqs <= kOwnPlanMaxSeqs)
        any = jobs <= sms ? work <= kDirectRoundChunks
                          : kv->head_dim == 64 ? jobs <= 3 * sms && work <= 2 * kDirectAnyChunks
                                               : jobs <= 2 * sms && 4 * work <= 3 * kDirectAnyChunks;
    else if (work <= (e4m3 ? kDirectAnyChunksE4m3 : kDirectAnyChunks))
        any = jobs <= kDirectJobsPerSm * sms;
    else
        any = jobs <= 2 * sms && work <= (e4m3 ? 2 : 1) * kDirectRoundChunks;
    const bool few = rows <= kDirectAnyRows || rows <= static_cast<int64_t>(num_seqs) * kDirectRows ||
                     (rows <= 2 * static_cast<int64_t>(num_seqs) * kDirectRows &&
                      work <= 2 * kDirectRoundChunks);
    if (!any && !(few && (!e4m3 || work <= kDirectE4m3Chunks))) return false;
    dp->max_rows = 0x7fffffff;
    direct_shape(jobs, chunks, sms, dp);
    return true;
}

// Runs the planner, the split-KV kernel and the tensor-core kernel of one
// step on `s`.  With `casc` (cascade decode, all rows short) the step is
// the unique-suffix pass, run side by side with the shared-prefix pass.
// With `fresh`, the step's new rows are written into the cache first.  With
// `win` the step is windowed (no cascade): the windowed forms of the plan and
// of both kernels run.
int run_step(const void *q, const pa_kv_desc *kv, const int32_t *block_tables, int32_t max_blocks,
             const int32_t *qsl, const int32_t *ctx, const int32_t *seq_lens, int32_t num_seqs,
             int32_t T, int32_t Hq, float scale, void *out, float *lse, uint8_t *ws,
             const WsLayout &L, int short_max_rows, int split_keys, const CascadeArgs *casc,
             bool forbid_long, const StepMaps &maps, const Staging &stg, DeviceInfo *dev,
             cudaStream_t s, const NewRows *fresh = nullptr, const WindowArgs *win = nullptr) {
    const int D = kv->head_dim;
    const int group = Hq / kv->num_kv_heads;
    const int tq = q_tile_tokens(group);
    PlanHeader *hdr = reinterpret_cast<PlanHeader *>(ws + L.header);

    PlanParams pp{};
    pp.qsl = qsl;
    pp.ctx = ctx;
    pp.seq_lens = seq_lens;
    pp.num_seqs = num_seqs;
    pp.num_q_tokens = T;
    pp.num_kv_heads = kv->num_kv_heads;
    pp.group = group;
    pp.q_tile_tokens = tq;
    // An fp8 pool runs short rows on the split-KV kernel; long requests run on
    // the tensor-core kernel over a bf16 staging copy while staging blocks
    // last, and as split-KV pieces of piece_tokens query tokens otherwise
    // (all of them when the workspace has no staging area).
    const bool fp8 = kv->kv_dtype == PA_KV_FP8_E4M3;
    const bool staged = fp8 && stg.cap > 0;
    if (fp8 && !staged) forbid_long = true;
    pp.short_max_rows = forbid_long ? 0x7fffffff : short_max_rows;
    pp.piece_tokens = std::max(1, std::min(pp.short_max_rows, kShortMaxRows) / group);
    pp.fp8 = fp8 ? 1 : 0;
    pp.stage_cap = staged ? stg.cap : 0;
    pp.block_size = kv->block_size;
    pp.stage_base = staged ? reinterpret_cast<int *>(ws + L.stage_base) : nullptr;
    pp.stage_list = staged ? reinterpret_cast<int *>(ws + L.stage_list) : nullptr;
    pp.split_stages = split_keys / kStageKeys;
    const int short_grid =
        dev->sms * dev->short_ctas_per_sm[win ? 1 : 0][fp8 ? 2 : (D == 128 ? 1 : 0)];
    pp.target_items = kSplitItemsPerCta * short_grid;
    pp.num_ctas = short_grid;
    pp.hdr = hdr;
    pp.short_items = reinterpret_cast<ShortItem *>(ws + L.short_items);
    pp.long_items = reinterpret_cast<LongItem *>(ws + L.long_items);
    pp.counters = reinterpret_cast<int *>(ws + L.counters);
    pp.max_short = L.max_short;
    pp.max_long = L.max_long;
    pp.cap_rows = L.cap_rows;
    pp.num_counters = L.num_counters;
    pp.status = dev->status;
    // a long request has q_len * group > short_max_rows, so there are at
    // most T / (short_max_rows / group + 1) of them
    const int min_long_tokens = short_max_rows / group + 1;
    const int max_long_reqs =
        forbid_long ? 0 : std::min(num_seqs, T / std::max(1, min_long_tokens));
    bool side_by_side = max_long_reqs > 0 && T >= kSideBySideMinTokens && !profiling_active();
    if (win && static_cast<int64_t>(num_seqs) * kv->num_kv_heads *
                       seen_chunks(*win, 1, max_blocks, kv->block_size) <
                   kSideBySideMinChunks)
        side_by_side = false;
    if (win) {
        // the windowed planner keeps its table at the end of the partial states
        pp.win = *win;
        pp.max_keys = max_blocks * kv->block_size;
        pp.max_pieces = pieces_bound(num_seqs, T, group);
        const size_t row = sizeof(float) * D;
        const int piece_rows = static_cast<int>(
            (sizeof(WindowPiece) * static_cast<size_t>(pp.max_pieces) + row - 1) / row);
        pp.cap_rows -= piece_rows;
        pp.pieces = reinterpret_cast<WindowPiece *>(ws + L.partial_o + row * pp.cap_rows);
    }
    ShortParams sp{};
    sp.q = static_cast<const __nv_bfloat16 *>(q);
    sp.out = static_cast<__nv_bfloat16 *>(out);
    sp.lse = lse;
    sp.block_tables = block_tables;
    sp.bt_stride = max_blocks;
    sp.qsl = qsl;
    sp.ctx = ctx;
    sp.seq_lens = seq_lens;
    sp.num_q_heads = Hq;
    sp.num_kv_heads = kv->num_kv_heads;
    sp.group = group;
    sp.block_size = kv->block_size;
    sp.num_blocks = kv->num_blocks;
    sp.kv_rows = static_cast<int>(kv_rows(kv));
    sp.scale_log2 = scale * 1.4426950408889634f;
    sp.hdr = hdr;
    sp.items = pp.short_items;
    sp.counters = pp.counters;
    sp.partial_o = reinterpret_cast<float *>(ws + L.partial_o);
    sp.partial_lse = reinterpret_cast<float *>(ws + L.partial_lse);
    sp.out_f32 = nullptr;
    sp.k_scale = fp8 ? kv->k_scale : nullptr;
    sp.v_scale = fp8 ? kv->v_scale : nullptr;
    sp.status = dev->status;
    sp.num_seqs = num_seqs;
    sp.num_q_tokens = T;
    sp.max_items = L.max_short;
    sp.claim_ahead = kClaimAheadStages;
    if (win) sp.win = *win;
    const int stall = g_test_stall.load(std::memory_order_relaxed);
    sp.test_stall = stall == PA_TEST_STALL_SPLIT_KV ? 1 : 0;

    int rc = PA_OK;
    if (fresh && fresh->num_tokens > 0) {
        // The step's new rows first, as pa_write_kv does: its kernel runs as a
        // programmatic dependent ahead of the planner and is off the step's
        // critical path.  (Writing them from copy blocks in the planner's
        // grid measured no faster on an 8-request decode step and slower on
        // large ones.)
        ProfScope prof(PA_KERNEL_WRITE_KV, s);
        rc = launch_write_kv(fresh->k, fresh->v, fresh->slots, fresh->num_tokens, kv, dev->status,
                             s);
        if (rc != PA_OK) return fail(rc, "write_kv launch failed");
    }

    DirectParams direct{};
    if (win && direct_step(*win, num_seqs, T, kv, group, max_blocks, dev->sms, &direct)) {
        ProfScope prof(PA_KERNEL_SPLIT_KV, s);
        rc = launch_window_direct(sp, maps.k, maps.v, direct, D, fp8, s);
        return rc == PA_OK ? PA_OK : fail(rc, "window kernel launch failed: %s",
                                          cudaGetErrorString(cudaGetLastError()));
    }
    // A windowed step of few requests whose kernels run one after the other needs no
    // plan either: its short rows run in the one-kernel form, and the tensor-core
    // kernel finds the long requests' tiles itself.
    const bool own_plans = win && !fp8 && group <= kDirectRows && num_seqs <= kOwnPlanMaxSeqs &&
                           max_long_reqs > 0 && !side_by_side &&
                           kv->num_kv_heads * ((T + tq - 1) / tq) <= kOwnPlanTilesPerSm * dev->sms;
    if (own_plans) {
        const int per_request = (kShortMaxRows / group + direct.piece_tokens - 1) / direct.piece_tokens;
        direct.max_pieces = std::min(direct.max_pieces, num_seqs * per_request);
        direct.max_rows = kShortMaxRows;
        direct_shape(static_cast<int64_t>(num_seqs) * kv->num_kv_heads,
                     seen_chunks(*win, direct.piece_tokens, max_blocks, kv->block_size), dev->sms,
                     &direct);
        ProfScope prof(PA_KERNEL_SPLIT_KV, s);
        rc = launch_window_direct(sp, maps.k, maps.v, direct, D, fp8, s);
        if (rc != PA_OK)
            return fail(rc, "window kernel launch failed: %s", cudaGetErrorString(cudaGetLastError()));
    }
    if (!own_plans) {
        ProfScope prof(PA_KERNEL_PLAN, s);
        rc = win ? launch_plan_window(pp, s) : launch_plan(pp, s);
    }
    if (rc != PA_OK) return fail(rc, "plan launch failed");
    if (staged) {
        rc = launch_stage_fp8(kv, block_tables, max_blocks, hdr, pp.stage_base, pp.stage_list,
                              stg.k, stg.v, dev->status, 2 * dev->sms, s, ctx, seq_lens, win);
        if (rc != PA_OK) return fail(rc, "fp8 staging copy launch failed");
    }

    if (casc) {
        // Cascade decode ([AI] §02.1): the shared-prefix pass (tensor cores,
        // compute-heavy, each prefix tile read once per 128 query rows) and
        // the unique-suffix pass (split-KV, HBM-bound) have disjoint inputs,
        // so they run side by side like the two halves of a mixed step: a
        // first prefix grid waits for the plan and lets the split-KV grid in
        // on the other SMs; a second prefix grid takes SMs over as split-KV
        // CTAs finish (both pull prefix items from the step's counter) and
        // completes after both.  The split-KV grid writes
        // each row's suffix state in fp32; the fold kernel merges it with the
        // prefix split states into out and lse.
        // The prefix pass's items are cut for one round on about 36 % of the
        // SMs (the first grid takes them all); the split-KV grid streams the
        // suffixes on the rest.  Measured on 64 requests x an 8192-token
        // prefix, us per call by share: 28 % 73.9 (too few splits), 32 %
        // 63.4, 36 % 63.1-63.5, 42 % 64.6, 48 % 64.5, 54 % 67.4.
        int q_tiles, nsplit, split_keys_p;
        const int prefix_sms = std::max(1, (dev->sms * 36 + 50) / 100);
        prefix_plan(T, casc->prefix_len, kv->num_kv_heads, group, prefix_sms, &q_tiles, &nsplit,
                    &split_keys_p);
        LongParams cp = prefix_params(kv, casc->prefix_blocks, casc->prefix_len, T, Hq, scale,
                                      q_tiles, nsplit, split_keys_p, casc->prefix_o,
                                      casc->prefix_lse, dev);
        // an e4m3 pool: the prefix decoded to bf16 first (after the plan; the
        // first prefix grid waits for it)
        const CUtensorMap *ptk = &maps.k, *ptv = &maps.v;
        rc = stage_prefix(*casc->ps, kv, casc->prefix_blocks, &cp, &ptk, &ptv, dev, s);
        if (rc != PA_OK) return rc;
        cp.hdr = hdr;
        cp.states_only = 1;
        cp.dynamic = 1;
        cp.first_done = &hdr->first_done;
        const int n_prefix = kv->num_kv_heads * q_tiles * nsplit;
        const int g1 = std::min(dev->sms, n_prefix);
        LongParams c1 = cp;
        c1.wait_start = 1;
        c1.first_ctas = -1;
        rc = launch_long(c1, maps.q, *ptk, *ptv, D, g1, s);
        if (rc != PA_OK) return fail(rc, "prefix kernel launch failed: %s",
                                     cudaGetErrorString(cudaGetLastError()));
        sp.no_start_wait = 1;
        sp.test_stall = 0;
        sp.out_f32 = casc->suffix_o;
        sp.lse = casc->suffix_lse;
        rc = launch_short(sp, maps.k, maps.v, D, fp8, win != nullptr, short_grid, s);
        if (rc != PA_OK) return fail(rc, "split-KV kernel launch failed: %s",
                                     cudaGetErrorString(cudaGetLastError()));
        LongParams c2 = cp;
        c2.overlap_prev = 1;
        c2.first_ctas = g1;
        rc = launch_long(c2, maps.q, *ptk, *ptv, D, n_prefix, s);
        if (rc != PA_OK) return fail(rc, "prefix kernel launch failed: %s",
                                     cudaGetErrorString(cudaGetLastError()));
        PrefixFoldParams f{};
        f.partial_o = casc->prefix_o;
        f.partial_lse = casc->prefix_lse;
        f.extra_o = casc->suffix_o;
        f.extra_lse = casc->suffix_lse;
        f.nsplit = nsplit;
        f.q_tiles = q_tiles;
        f.pairs = kv->num_kv_heads * q_tiles;
        f.group = group;
        f.q_tile_tokens = tq;
        f.num_q_tokens = T;
        f.num_q_heads = Hq;
        f.out = static_cast<__nv_bfloat16 *>(out);
        f.out_f32 = nullptr;
        f.lse = lse;
        rc = launch_prefix_fold(f, D, s);
        return rc == PA_OK ? PA_OK : fail(rc, "cascade fold launch failed");
    }

    LongParams lp{};
    int long_grid = 0;
    if (max_long_reqs > 0) {
        lp.out = sp.out;
        lp.lse = lse;
        lp.out_f32 = nullptr;
        lp.block_tables = block_tables;
        lp.bt_stride = max_blocks;
        lp.qsl = qsl;
        lp.ctx = ctx;
        lp.seq_lens = seq_lens;
        lp.num_q_tokens = T;
        lp.num_q_heads = Hq;
        lp.num_kv_heads = kv->num_kv_heads;
        lp.group = group;
        lp.q_tile_tokens = tq;
        lp.block_size = kv->block_size;
        lp.num_blocks = kv->num_blocks;
        lp.kv_rows = sp.kv_rows;
        lp.scale_log2 = sp.scale_log2;
        lp.prefix_mode = 0;
        if (win) lp.win = *win;
        lp.test_stall = stall == PA_TEST_STALL_TENSOR_CORE ? 1 : 0;
        if (own_plans) {
            lp.own_seqs = num_seqs;
            lp.own_max_keys = direct.max_keys;
        }
        lp.hdr = hdr;
        lp.items = pp.long_items;
        lp.partial_o = sp.partial_o;
        lp.partial_lse = sp.partial_lse;
        lp.status = dev->status;
        lp.tile_counter = reinterpret_cast<unsigned long long *>(
            g_tile_counter.load(std::memory_order_relaxed));
        if (staged) {
            lp.stage_base = pp.stage_base;
            lp.k_scale = kv->k_scale;
            lp.v_scale = kv->v_scale;
            lp.num_blocks = stg.cap;
            lp.kv_rows = stg.cap * kv->num_kv_heads * kv->block_size;
        }
        long_grid = std::min(kv->num_kv_heads * ((T + tq - 1) / tq + max_long_reqs), L.max_long);
    }
    const CUtensorMap &lk = staged ? stg.tk : maps.k;
    const CUtensorMap &lv = staged ? stg.tv : maps.v;
    auto tensor_core = [&](const LongParams &params, int grid) {
        return win ? launch_long_window(params, maps.q, lk, lv, D, grid, dev->sms, s)
                   : launch_long(params, maps.q, lk, lv, D, grid, s);
    };

    if (side_by_side) {
        // The HBM-bound split-KV kernel and the tensor-core kernel run side by
        // side: a first tensor-core grid takes part of the SMs (it waits
        // for the plan, then lets the next grid in), the split-KV grid fills
        // the others, and a second tensor-core grid takes SMs over as
        // split-KV CTAs finish.  Both tensor-core grids pull items, longest
        // first, from the step's counter; the second completes only after
        // the first and after the split-KV grid.  A step of few tokens has
        // little or no tensor-core work: there the two extra launches would
        // only add latency, and the kernels run one after the other.
        LongParams l1 = lp;
        l1.dynamic = 1;
        l1.wait_start = 1;
        l1.first_done = &hdr->first_done;
        l1.first_ctas = -1;
        // share of the SMs measured best on the mixed step: two fifths beside
        // the HBM-bound bf16 split-KV kernel (60 of 152 SMs: 767.9 us per step,
        // against 769.6 with 56, 773.4 with 64 and 785.4 with 50); a tenth
        // beside the fp8 one, whose rate follows its SM count (707.3 us, 710.1
        // with an eighth)
        const int g1 = std::min(std::max(1, fp8 ? dev->sms / 10 : dev->sms * 2 / 5), long_grid);
        rc = tensor_core(l1, g1);
        if (rc != PA_OK) return fail(rc, "tensor-core kernel launch failed: %s",
                                     cudaGetErrorString(cudaGetLastError()));
        sp.no_start_wait = 1;
        sp.claim_ahead = 0;
        sp.test_stall = 0;
        rc = launch_short(sp, maps.k, maps.v, D, fp8, win != nullptr, short_grid, s);
        if (rc != PA_OK) return fail(rc, "split-KV kernel launch failed: %s",
                                     cudaGetErrorString(cudaGetLastError()));
        LongParams l2 = lp;
        l2.dynamic = 1;
        l2.overlap_prev = 1;
        l2.first_done = &hdr->first_done;
        // the test hook waits for one CTA that the first grid never had
        l2.first_ctas = g1 + (stall == PA_TEST_STALL_LAST_GRID ? 1 : 0);
        rc = tensor_core(l2, long_grid);
        if (rc != PA_OK) return fail(rc, "tensor-core kernel launch failed: %s",
                                     cudaGetErrorString(cudaGetLastError()));
        return PA_OK;
    }

    if (!own_plans) {
        ProfScope prof(PA_KERNEL_SPLIT_KV, s);
        rc = launch_short(sp, maps.k, maps.v, D, fp8, win != nullptr, short_grid, s);
    }
    if (rc != PA_OK) return fail(rc, "split-KV kernel launch failed: %s",
                                 cudaGetErrorString(cudaGetLastError()));
    if (max_long_reqs > 0) {
        // the split-KV kernel was launched just before: the tensor-core grid
        // may take over SMs as split-KV CTAs finish (its rows are disjoint)
        lp.overlap_prev = short_grid > 0 ? 1 : 0;
        // (many windowed items: from the step's counter, see pa_long_window.cu)
        lp.dynamic = win && !own_plans && long_grid > 2 * dev->sms ? 1 : 0;
        {
            ProfScope prof(PA_KERNEL_TENSOR_CORE, s);
            rc = tensor_core(lp, long_grid);
        }
        if (rc != PA_OK) return fail(rc, "tensor-core kernel launch failed: %s",
                                     cudaGetErrorString(cudaGetLastError()));
    }
    return PA_OK;
}

int common_checks(const void *q, const pa_kv_desc *kv, int32_t num_q_tokens, int32_t num_q_heads,
                  float scale, const void *out, const void *workspace) {
    int rc = check_kv(kv);
    if (rc != PA_OK) return rc;
    rc = check_heads(kv, num_q_heads);
    if (rc != PA_OK) return rc;
    if (num_q_tokens < 0) return fail(PA_ERR_INVALID_ARG, "num_q_tokens < 0");
    if (num_q_tokens > 0 && (!q || !out)) return fail(PA_ERR_INVALID_ARG, "q or out is NULL");
    if (!aligned(q, 16) || !aligned(out, 16))
        return fail(PA_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
    if (!std::isfinite(scale)) return fail(PA_ERR_INVALID_ARG, "scale is not finite");
    if (kv->kv_dtype == PA_KV_FP8_E4M3 && num_q_heads / kv->num_kv_heads > kShortMaxRows)
        return fail(PA_ERR_UNSUPPORTED, "fp8 KV pool: group size above %d not built",
                    kShortMaxRows);
    if (workspace && !aligned(workspace, 256))
        return fail(PA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    return PA_OK;
}

int run_prefix(const void *q, const pa_kv_desc *kv, const int32_t *prefix_blocks, int32_t prefix_len,
               int32_t T, int32_t Hq, float scale, void *out, float *lse, uint8_t *ws,
               const WsLayout &L, const StepMaps &maps, const PrefixStage &ps, DeviceInfo *dev,
               cudaStream_t s) {
    const int group = Hq / kv->num_kv_heads;
    int q_tiles, nsplit, split_keys;
    prefix_plan(T, prefix_len, kv->num_kv_heads, group, dev->sms, &q_tiles, &nsplit, &split_keys);
    // a split prefix leaves its split states to the fold kernel, which runs
    // the fold of a (kv head, query tile) on many SMs
    LongParams lp = prefix_params(kv, prefix_blocks, prefix_len, T, Hq, scale, q_tiles, nsplit,
                                  split_keys, reinterpret_cast<float *>(ws + L.prefix_o),
                                  reinterpret_cast<float *>(ws + L.prefix_lse), dev);
    lp.out = static_cast<__nv_bfloat16 *>(out);
    lp.lse = lse;
    const CUtensorMap *tk = &maps.k, *tv = &maps.v;
    int rc = stage_prefix(ps, kv, prefix_blocks, &lp, &tk, &tv, dev, s);
    if (rc != PA_OK) return rc;
    const int grid = kv->num_kv_heads * q_tiles * nsplit;
    rc = launch_long(lp, maps.q, *tk, *tv, kv->head_dim, grid, s);
    if (rc != PA_OK) return fail(rc, "prefix kernel launch failed");
    if (nsplit > 1) {
        PrefixFoldParams f{};
        f.partial_o = lp.partial_o;
        f.partial_lse = lp.partial_lse;
        f.nsplit = nsplit;
        f.q_tiles = q_tiles;
        f.pairs = kv->num_kv_heads * q_tiles;
        f.group = group;
        f.q_tile_tokens = lp.q_tile_tokens;
        f.num_q_tokens = T;
        f.num_q_heads = Hq;
        f.out = static_cast<__nv_bfloat16 *>(out);
        f.lse = lse;
        rc = launch_prefix_fold(f, kv->head_dim, s);
        if (rc != PA_OK) return fail(rc, "prefix fold launch failed");
    }
    return PA_OK;
}

int prefix_partial_rows(int T, int prefix_len, int num_kv_heads, int group) {
    int q_tiles, nsplit, split_keys;
    // the split count never exceeds 64, whatever the SM count
    prefix_plan(T, prefix_len, num_kv_heads, group, 1 << 20, &q_tiles, &nsplit, &split_keys);
    return num_kv_heads * q_tiles * nsplit * kLongRows;
}

}  // namespace

namespace pa {

void count_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

// Attention for one step inside a caller-provided scratch region of fixed
// size (used by the entry point that never allocates).  The work lists get
// the smallest capacity that always fits (one split per request and kv
// head, plus room for extra splits); whatever space is left holds split-KV
// partial states, and the planner picks split sizes that fit it.
int attention_in_fixed_workspace(const void *q, const pa_kv_desc *kv,
                                 const int32_t *block_tables, int32_t max_blocks_per_seq,
                                 const int32_t *query_start_loc, const int32_t *context_lens,
                                 const int32_t *seq_lens, int32_t num_seqs, int32_t num_q_tokens,
                                 int32_t num_q_heads, float scale, void *out, float *lse,
                                 void *scratch, size_t scratch_bytes, cudaStream_t s) {
    g_err[0] = 0;
    int rc = common_checks(q, kv, num_q_tokens, num_q_heads, scale, out, scratch);
    if (rc != PA_OK) return rc;
    if (num_seqs < 0) return fail(PA_ERR_INVALID_ARG, "num_seqs < 0");
    if (num_seqs == 0 || num_q_tokens == 0) return PA_OK;
    if (!block_tables || !query_start_loc || !context_lens || !seq_lens)
        return fail(PA_ERR_INVALID_ARG, "metadata pointer is NULL");
    if (max_blocks_per_seq <= 0) return fail(PA_ERR_INVALID_ARG, "max_blocks_per_seq <= 0");
    const int hkv = kv->num_kv_heads, D = kv->head_dim;
    const int tq = q_tile_tokens(num_q_heads / hkv);
    WsLayout L{};
    const int pieces = pieces_bound(num_seqs, num_q_tokens, num_q_heads / hkv);
    L.max_short = hkv * pieces + 4096;
    L.max_long = hkv * ((num_q_tokens + tq - 1) / tq + num_seqs);
    L.num_counters = hkv * pieces;
    size_t off = 0;
    L.header = off;
    off = align256(off + sizeof(PlanHeader));
    L.counters = off;
    off = align256(off + sizeof(int) * static_cast<size_t>(L.num_counters));
    L.short_items = off;
    off = align256(off + sizeof(ShortItem) * static_cast<size_t>(L.max_short));
    L.long_items = off;
    off = align256(off + sizeof(LongItem) * static_cast<size_t>(L.max_long));
    const size_t fixed = off + 512;  // + alignment of the two partial arrays
    if (fixed > scratch_bytes)
        return fail(PA_ERR_WORKSPACE,
                    "step too large for the fixed scratch: its work lists need %zu bytes, "
                    "the scratch holds %zu", fixed, scratch_bytes);
    const size_t rows = (scratch_bytes - fixed) / (sizeof(float) * (static_cast<size_t>(D) + 1));
    L.cap_rows = static_cast<int>(std::min<size_t>(rows, 1u << 24));
    L.partial_o = off;
    off = align256(off + sizeof(float) * static_cast<size_t>(L.cap_rows) * D);
    L.partial_lse = off;
    off = align256(off + sizeof(float) * static_cast<size_t>(L.cap_rows));
    L.total = off;
    if (L.total > scratch_bytes) return fail(PA_ERR_WORKSPACE, "scratch layout overflow");
    DeviceInfo *dev;
    if ((rc = device_info(&dev)) != PA_OK) return rc;
    StepMaps maps;
    if ((rc = make_maps(&maps, q, kv, num_q_tokens, num_q_heads)) != PA_OK) return rc;
    return run_step(q, kv, block_tables, max_blocks_per_seq, query_start_loc, context_lens,
                    seq_lens, num_seqs, num_q_tokens, num_q_heads, scale, out, lse,
                    static_cast<uint8_t *>(scratch), L, kShortMaxRows, 0, nullptr, false, maps,
                    Staging(), dev, s);
}

int set_error_message(int code, const char *msg) { return fail(code, "%s", msg); }

}  // namespace pa

extern "C" {

const char *pa_last_error_message(void) { return g_err; }

const char *pa_status_string(int code) {
    switch (code) {
    case PA_OK: return "PA_OK";
    case PA_ERR_INVALID_ARG: return "PA_ERR_INVALID_ARG";
    case PA_ERR_UNSUPPORTED: return "PA_ERR_UNSUPPORTED";
    case PA_ERR_WORKSPACE: return "PA_ERR_WORKSPACE";
    case PA_ERR_CUDA: return "PA_ERR_CUDA";
    case PA_ERR_BAD_METADATA: return "PA_ERR_BAD_METADATA";
    default: return "PA_ERR_UNKNOWN";
    }
}

int pa_write_kv(const void *k, const void *v, const int64_t *slot_mapping, int32_t num_tokens,
                const pa_kv_desc *kv, void *stream) {
    g_err[0] = 0;
    int rc = check_kv(kv);
    if (rc != PA_OK) return rc;
    if ((rc = check_new_rows(NewRows{k, v, slot_mapping, num_tokens})) != PA_OK) return rc;
    if (num_tokens == 0) return PA_OK;
    DeviceInfo *dev;
    if ((rc = device_info(&dev)) != PA_OK) return rc;
    {
        ProfScope prof(PA_KERNEL_WRITE_KV, static_cast<cudaStream_t>(stream));
        rc = launch_write_kv(k, v, slot_mapping, num_tokens, kv, dev->status,
                             static_cast<cudaStream_t>(stream));
    }
    return rc == PA_OK ? PA_OK : fail(rc, "write_kv launch failed");
}

size_t pa_attention_workspace_size(int32_t num_seqs, int32_t num_q_tokens, int32_t num_q_heads,
                                   int32_t num_kv_heads, int32_t head_dim) {
    if (num_seqs < 0 || num_q_tokens < 0 || num_kv_heads <= 0 || num_q_heads <= 0 ||
        num_q_heads % num_kv_heads != 0 || (head_dim != 64 && head_dim != 128))
        return 0;
    return make_layout(num_seqs, num_q_tokens, num_q_heads, num_kv_heads, head_dim, 0, false).total;
}

}  // extern "C"

namespace {

// pa_attention_ex, with `fresh` the write of the step's new rows first, with
// `win` a windowed step.
int attention_entry(const void *q, const pa_kv_desc *kv, const int32_t *block_tables,
                    int32_t max_blocks_per_seq, const int32_t *query_start_loc,
                    const int32_t *context_lens, const int32_t *seq_lens, int32_t num_seqs,
                    int32_t num_q_tokens, int32_t num_q_heads, float scale, void *out, float *lse,
                    void *workspace, size_t workspace_bytes, int32_t short_q_max_rows,
                    int32_t split_keys, cudaStream_t stream, const NewRows *fresh,
                    const WindowArgs *win = nullptr) {
    g_err[0] = 0;
    int rc = common_checks(q, kv, num_q_tokens, num_q_heads, scale, out, workspace);
    if (rc != PA_OK) return rc;
    if (num_seqs < 0) return fail(PA_ERR_INVALID_ARG, "num_seqs < 0");
    if (short_q_max_rows < -1 || short_q_max_rows > kShortMaxRows)
        return fail(PA_ERR_INVALID_ARG, "short_q_max_rows must be -1 or in [0, %d]", kShortMaxRows);
    if (split_keys < 0 || split_keys % kStageKeys != 0)
        return fail(PA_ERR_INVALID_ARG, "split_keys must be 0 or a multiple of %d", kStageKeys);
    if (fresh && (rc = check_new_rows(*fresh)) != PA_OK) return rc;
    if (num_seqs == 0 || num_q_tokens == 0) {
        // nothing to attend: the write alone, as pa_write_kv
        if (!fresh || fresh->num_tokens == 0) return PA_OK;
        DeviceInfo *dev;
        if ((rc = device_info(&dev)) != PA_OK) return rc;
        ProfScope prof(PA_KERNEL_WRITE_KV, stream);
        rc = launch_write_kv(fresh->k, fresh->v, fresh->slots, fresh->num_tokens, kv, dev->status,
                             stream);
        return rc == PA_OK ? PA_OK : fail(rc, "write_kv launch failed");
    }
    if (!block_tables || !query_start_loc || !context_lens || !seq_lens)
        return fail(PA_ERR_INVALID_ARG, "metadata pointer is NULL");
    if (max_blocks_per_seq <= 0) return fail(PA_ERR_INVALID_ARG, "max_blocks_per_seq <= 0");
    if (win && static_cast<int64_t>(max_blocks_per_seq) * kv->block_size > kMaxWindowKeys)
        return fail(PA_ERR_UNSUPPORTED, "block tables of more than 2^30 tokens per request");
    const WsLayout L = make_layout(num_seqs, num_q_tokens, num_q_heads, kv->num_kv_heads,
                                   kv->head_dim, 0, false);
    if (!workspace || workspace_bytes < L.total)
        return fail(PA_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", L.total,
                    workspace_bytes);
    DeviceInfo *dev;
    if ((rc = device_info(&dev)) != PA_OK) return rc;
    StepMaps maps;
    // (a windowed step of few tokens has no long request: see run_step)
    const bool any_long =
        !win || num_q_tokens > kShortMaxRows / (num_q_heads / kv->num_kv_heads);
    if ((rc = make_maps(&maps, q, kv, num_q_tokens, num_q_heads, any_long)) != PA_OK) return rc;
    // an fp8 pool stages long requests in the workspace beyond the layout
    Staging stg;
    if ((rc = make_staging(&stg, kv, static_cast<uint8_t *>(workspace), L.total, workspace_bytes)) !=
        PA_OK)
        return rc;
    return run_step(q, kv, block_tables, max_blocks_per_seq, query_start_loc, context_lens,
                    seq_lens, num_seqs, num_q_tokens, num_q_heads, scale, out, lse,
                    static_cast<uint8_t *>(workspace), L,
                    short_q_max_rows < 0 ? kShortMaxRows : short_q_max_rows, split_keys, nullptr,
                    false, maps, stg, dev, stream, fresh, win);
}

}  // namespace

extern "C" {

int pa_attention_ex(const void *q, const pa_kv_desc *kv, const int32_t *block_tables,
                    int32_t max_blocks_per_seq, const int32_t *query_start_loc,
                    const int32_t *context_lens, const int32_t *seq_lens, int32_t num_seqs,
                    int32_t num_q_tokens, int32_t num_q_heads, float scale, void *out, float *lse,
                    void *workspace, size_t workspace_bytes, int32_t short_q_max_rows,
                    int32_t split_keys, void *stream) {
    return attention_entry(q, kv, block_tables, max_blocks_per_seq, query_start_loc,
                               context_lens, seq_lens, num_seqs, num_q_tokens, num_q_heads, scale,
                               out, lse, workspace, workspace_bytes, short_q_max_rows, split_keys,
                               static_cast<cudaStream_t>(stream), nullptr);
}

int pa_write_kv_attention(const void *k, const void *v, const int64_t *slot_mapping,
                          int32_t num_new_tokens, const void *q, const pa_kv_desc *kv,
                          const int32_t *block_tables, int32_t max_blocks_per_seq,
                          const int32_t *query_start_loc, const int32_t *context_lens,
                          const int32_t *seq_lens, int32_t num_seqs, int32_t num_q_tokens,
                          int32_t num_q_heads, float scale, void *out, float *lse,
                          void *workspace, size_t workspace_bytes, void *stream) {
    const NewRows fresh{k, v, slot_mapping, num_new_tokens};
    return attention_entry(q, kv, block_tables, max_blocks_per_seq, query_start_loc,
                               context_lens, seq_lens, num_seqs, num_q_tokens, num_q_heads, scale,
                               out, lse, workspace, workspace_bytes, -1, 0,
                               static_cast<cudaStream_t>(stream), &fresh);
}



size_t pa_fp8_staging_bytes(int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                            int64_t num_blocks) {
    if (num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks < 0) return 0;
    const size_t blk = static_cast<size_t>(num_kv_heads) * block_size * head_dim * 2;
    return 2 * align256(static_cast<size_t>(num_blocks) * blk) + 768;
}

int pa_attention(const void *q, const pa_kv_desc *kv, const int32_t *block_tables,
                 int32_t max_blocks_per_seq, const int32_t *query_start_loc,
                 const int32_t *context_lens, const int32_t *seq_lens, int32_t num_seqs,
                 int32_t num_q_tokens, int32_t num_q_heads, float scale, void *out, float *lse,
                 void *workspace, size_t workspace_bytes, void *stream) {
    return pa_attention_ex(q, kv, block_tables, max_blocks_per_seq, query_start_loc, context_lens,
                           seq_lens, num_seqs, num_q_tokens, num_q_heads, scale, out, lse,
                           workspace, workspace_bytes, -1, 0, stream);
}

int pa_window_attention(const void *q, const pa_kv_desc *kv, const int32_t *block_tables,
                        int32_t max_blocks_per_seq, const int32_t *query_start_loc,
                        const int32_t *context_lens, const int32_t *seq_lens, int32_t num_seqs,
                        int32_t num_q_tokens, int32_t num_q_heads, float scale, int32_t window,
                        int32_t num_sinks, void *out, float *lse, void *workspace,
                        size_t workspace_bytes, void *stream) {
    g_err[0] = 0;
    const int rc = check_window(window, num_sinks, scale);
    if (rc != PA_OK) return rc;
    // a request has at most 2^30 keys: more window or sinks see no more of it
    const int32_t most = static_cast<int32_t>(kMaxWindowKeys);
    const WindowArgs win{std::min(window, most), std::min(num_sinks, most)};
    return attention_entry(q, kv, block_tables, max_blocks_per_seq, query_start_loc, context_lens,
                           seq_lens, num_seqs, num_q_tokens, num_q_heads, scale, out, lse,
                           workspace, workspace_bytes, -1, 0, static_cast<cudaStream_t>(stream),
                           nullptr, &win);
}

int pa_rope_write_kv(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                     const void *v, int64_t v_stride, const int32_t *positions,
                     const pa_rope_desc *rope, const int64_t *slot_mapping, int32_t num_tokens,
                     int32_t num_q_heads, const pa_kv_desc *kv, void *q_out, void *stream) {
    g_err[0] = 0;
    int rc = check_kv(kv);
    if (rc != PA_OK) return rc;
    if ((rc = check_new_rows(NewRows{k, v, slot_mapping, num_tokens})) != PA_OK) return rc;
    if (!rope || !rope->inv_freq) return fail(PA_ERR_INVALID_ARG, "rope descriptor or inv_freq is NULL");
    if (rope->rot_dim < 16 || rope->rot_dim % 16 != 0 || rope->rot_dim > kv->head_dim)
        return fail(PA_ERR_UNSUPPORTED, "rot_dim %d: need a multiple of 16, at most head_dim %d",
                    rope->rot_dim, kv->head_dim);
    if (rope->num_axes < 1 || rope->num_axes > kMaxRopeAxes)
        return fail(PA_ERR_UNSUPPORTED, "num_axes %d: need 1 .. %d", rope->num_axes, kMaxRopeAxes);
    if (rope->adjacent != 0 && rope->adjacent != 1)
        return fail(PA_ERR_INVALID_ARG, "pa_rope_desc.adjacent must be 0 or 1");
    if (!std::isfinite(rope->attn_factor))
        return fail(PA_ERR_INVALID_ARG, "attn_factor is not finite");
    if (num_q_heads < 0) return fail(PA_ERR_INVALID_ARG, "num_q_heads < 0");
    if (num_tokens == 0) return PA_OK;
    if (!positions) return fail(PA_ERR_INVALID_ARG, "positions is NULL");
    if (!aligned(positions, 4) || !aligned(slot_mapping, 8) || !aligned(rope->inv_freq, 8) ||
        !aligned(rope->axis, 4))
        return fail(PA_ERR_INVALID_ARG, "positions, axis, inv_freq or slot_mapping is misaligned");
    if (num_q_heads > 0) {
        if (!q || !q_out) return fail(PA_ERR_INVALID_ARG, "q or q_out is NULL");
        if (!aligned(q, 16) || !aligned(q_out, 16))
            return fail(PA_ERR_INVALID_ARG, "q and q_out must be 16-byte aligned");
    }
    const int64_t d = kv->head_dim;
    const int64_t stride[3] = {num_q_heads > 0 ? q_stride : 0, k_stride, v_stride};
    const int64_t least[3] = {num_q_heads * d, kv->num_kv_heads * d, kv->num_kv_heads * d};
    for (int i = 0; i < 3; ++i)
        if (stride[i] % 8 != 0 || (num_tokens > 1 && stride[i] < least[i]))
            return fail(PA_ERR_INVALID_ARG,
                        "%c_stride %lld: need a multiple of 8 that holds a token's heads", "qkv"[i],
                        (long long)stride[i]);
    if (num_q_heads > 0 && q == q_out && q_stride != least[0] && num_tokens > 1)
        return fail(PA_ERR_INVALID_ARG, "q rotated in place must be contiguous");
    DeviceInfo *dev;
    if ((rc = device_info(&dev)) != PA_OK) return rc;
    RopeParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.positions = positions;
    p.inv_freq = rope->inv_freq;
    p.axis = rope->axis;
    p.slots = slot_mapping;
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.k_cache = kv->k_cache;
    p.v_cache = kv->v_cache;
    p.fp8 = kv->kv_dtype == PA_KV_FP8_E4M3 ? 1 : 0;
    p.k_scale = kv->k_scale;
    p.v_scale = kv->v_scale;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = kv->num_kv_heads;
    p.head_dim = kv->head_dim;
    p.block_size = kv->block_size;
    p.num_slots = static_cast<int64_t>(kv->num_blocks) * kv->block_size;
    p.rot_dim = rope->rot_dim;
    p.num_axes = rope->num_axes;
    p.adjacent = rope->adjacent;
    p.attn_factor = rope->attn_factor;
    p.test_stall = g_test_stall.load(std::memory_order_relaxed) == PA_TEST_STALL_ROPE ? 1 : 0;
    p.status = dev->status;
    rc = launch_rope_write(p, dev->sms, static_cast<cudaStream_t>(stream));
    return rc == PA_OK ? PA_OK : fail(rc, "rope_write_kv launch failed");
}

int pa_copy_blocks(const pa_kv_desc *kv, int32_t num_layers, const int32_t *pairs,
                   int32_t num_pairs, void *stream) {
    g_err[0] = 0;
    if (num_layers < 0 || num_pairs < 0)
        return fail(PA_ERR_INVALID_ARG, "num_layers or num_pairs < 0");
    if (num_layers > 0 && !kv) return fail(PA_ERR_INVALID_ARG, "kv descriptors are NULL");
    for (int l = 0; l < num_layers; ++l) {
        const int rc = check_kv(&kv[l], false);
        if (rc != PA_OK) return rc;
        if (kv[l].num_blocks != kv->num_blocks || kv[l].block_size != kv->block_size ||
            kv[l].num_kv_heads != kv->num_kv_heads || kv[l].head_dim != kv->head_dim ||
            kv[l].kv_dtype != kv->kv_dtype)
            return fail(PA_ERR_INVALID_ARG, "layer %d's pool differs from layer 0's in its geometry",
                        l);
    }
    if (num_layers == 0 || num_pairs == 0) return PA_OK;
    if (!pairs) return fail(PA_ERR_INVALID_ARG, "pairs is NULL");
    if (!aligned(pairs, 8)) return fail(PA_ERR_INVALID_ARG, "pairs must be 8-byte aligned");
    DeviceInfo *dev;
    int rc = device_info(&dev);
    if (rc != PA_OK) return rc;
    rc = launch_copy_blocks(kv, num_layers, pairs, num_pairs, dev->sms, dev->status,
                            static_cast<cudaStream_t>(stream));
    return rc == PA_OK ? PA_OK : fail(rc, "copy_blocks launch failed");
}

int pa_validate_copies(const int32_t *pairs, int32_t num_pairs, int32_t num_blocks) {
    g_err[0] = 0;
    if (num_pairs < 0 || num_blocks <= 0 || (num_pairs > 0 && !pairs))
        return fail(PA_ERR_INVALID_ARG, "bad sizes");
    try {
        std::vector<uint8_t> role(static_cast<size_t>(num_blocks), 0);  // 1: a src, 2: a dst
        for (int pass = 0; pass < 2; ++pass)
            for (int i = 0; i < num_pairs; ++i) {
                const int32_t src = pairs[2 * i], dst = pairs[2 * i + 1];
                if (src < 0 || dst < 0 || src == dst) continue;
                if (src >= num_blocks || dst >= num_blocks)
                    return fail(PA_ERR_BAD_METADATA, "pair %d (%d, %d) outside the pool", i, src,
                                dst);
                if (pass == 0) {
                    role[static_cast<size_t>(src)] = 1;
                    continue;
                }
                uint8_t &r = role[static_cast<size_t>(dst)];
                if (r) return fail(PA_ERR_BAD_METADATA, "block %d is written by pair %d and %s", dst,
                                   i, r == 1 ? "read by another" : "written by another");
                r = 2;
            }
    } catch (...) {
        return fail(PA_ERR_INVALID_ARG, "out of host memory");
    }
    return PA_OK;
}

int pa_merge_states(const void *o_a, const float *lse_a, const void *o_b, const float *lse_b,
                    int32_t n, int32_t num_heads, int32_t head_dim, void *out, float *lse_out,
                    void *stream) {
    g_err[0] = 0;
    if (n < 0 || num_heads <= 0) return fail(PA_ERR_INVALID_ARG, "bad n / num_heads");
    if (head_dim <= 0 || head_dim % 8 != 0)
        return fail(PA_ERR_UNSUPPORTED, "head_dim must be a positive multiple of 8");
    if (n == 0) return PA_OK;
    if (!o_a || !o_b || !lse_a || !lse_b || !out) return fail(PA_ERR_INVALID_ARG, "NULL input");
    if (!aligned(o_a, 16) || !aligned(o_b, 16) || !aligned(out, 16))
        return fail(PA_ERR_INVALID_ARG, "o_a, o_b and out must be 16-byte aligned");
    const int rc = launch_merge(o_a, lse_a, o_b, lse_b, n, num_heads, head_dim, out, lse_out,
                                static_cast<cudaStream_t>(stream));
    return rc == PA_OK ? PA_OK : fail(rc, "merge launch failed");
}

size_t pa_cascade_workspace_size(int32_t num_seqs, int32_t num_q_tokens, int32_t num_q_heads,
                                 int32_t num_kv_heads, int32_t head_dim, int32_t prefix_len) {
    if (num_seqs < 0 || num_q_tokens < 0 || num_kv_heads <= 0 || num_q_heads <= 0 ||
        num_q_heads % num_kv_heads != 0 || (head_dim != 64 && head_dim != 128) || prefix_len < 0)
        return 0;
    const int group = num_q_heads / num_kv_heads;
    const int rows = prefix_partial_rows(num_q_tokens, prefix_len, num_kv_heads, group);
    return make_layout(num_seqs, num_q_tokens, num_q_heads, num_kv_heads, head_dim, rows, true)
        .total;
}

int pa_prefix_attention(const void *q, const pa_kv_desc *kv, const int32_t *prefix_blocks,
                        int32_t prefix_len, int32_t num_q_tokens, int32_t num_q_heads,
                        float scale, void *out, float *lse, void *workspace,
                        size_t workspace_bytes, void *stream) {
    g_err[0] = 0;
    int rc = common_checks(q, kv, num_q_tokens, num_q_heads, scale, out, workspace);
    if (rc != PA_OK) return rc;
    if (prefix_len < 0) return fail(PA_ERR_INVALID_ARG, "prefix_len < 0");
    if (prefix_len > 0 && !prefix_blocks) return fail(PA_ERR_INVALID_ARG, "prefix_blocks is NULL");
    if (num_q_tokens == 0) return PA_OK;
    const int group = num_q_heads / kv->num_kv_heads;
    const WsLayout L = make_layout(1, num_q_tokens, num_q_heads, kv->num_kv_heads, kv->head_dim,
                                   prefix_partial_rows(num_q_tokens, prefix_len, kv->num_kv_heads,
                                                       group),
                                   true);
    if (!workspace || workspace_bytes < L.total)
        return fail(PA_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", L.total,
                    workspace_bytes);
    PrefixStage ps;
    if ((rc = make_prefix_stage(&ps, kv, prefix_len, static_cast<uint8_t *>(workspace), L.total,
                                workspace_bytes)) != PA_OK)
        return rc;
    DeviceInfo *dev;
    if ((rc = device_info(&dev)) != PA_OK) return rc;
    StepMaps maps;
    if ((rc = make_maps(&maps, q, kv, num_q_tokens, num_q_heads)) != PA_OK) return rc;
    return run_prefix(q, kv, prefix_blocks, prefix_len, num_q_tokens, num_q_heads, scale, out,
                      lse, static_cast<uint8_t *>(workspace), L, maps, ps, dev,
                      static_cast<cudaStream_t>(stream));
}

int pa_cascade_decode(const void *q, const pa_kv_desc *kv, const int32_t *prefix_blocks,
                      int32_t prefix_len, const int32_t *block_tables,
                      int32_t max_blocks_per_seq, const int32_t *query_start_loc,
                      const int32_t *context_lens, const int32_t *seq_lens, int32_t num_seqs,
                      int32_t num_q_tokens, int32_t num_q_heads, float scale, void *out,
                      float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    g_err[0] = 0;
    int rc = common_checks(q, kv, num_q_tokens, num_q_heads, scale, out, workspace);
    if (rc != PA_OK) return rc;
    if (num_q_heads / kv->num_kv_heads > kShortMaxRows)
        return fail(PA_ERR_UNSUPPORTED, "cascade decode: group size above %d not built",
                    kShortMaxRows);
    if (num_seqs < 0 || prefix_len < 0) return fail(PA_ERR_INVALID_ARG, "negative size");
    if (prefix_len > 0 && !prefix_blocks) return fail(PA_ERR_INVALID_ARG, "prefix_blocks is NULL");
    if (num_seqs == 0 || num_q_tokens == 0) return PA_OK;
    if (!block_tables || !query_start_loc || !context_lens || !seq_lens)
        return fail(PA_ERR_INVALID_ARG, "metadata pointer is NULL");
    if (max_blocks_per_seq <= 0) return fail(PA_ERR_INVALID_ARG, "max_blocks_per_seq <= 0");
    const int group = num_q_heads / kv->num_kv_heads;
    const WsLayout L = make_layout(num_seqs, num_q_tokens, num_q_heads, kv->num_kv_heads,
                                   kv->head_dim,
                                   prefix_partial_rows(num_q_tokens, prefix_len, kv->num_kv_heads,
                                                       group),
                                   true);
    if (!workspace || workspace_bytes < L.total)
        return fail(PA_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", L.total,
                    workspace_bytes);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    PrefixStage ps;
    if ((rc = make_prefix_stage(&ps, kv, prefix_len, ws, L.total, workspace_bytes)) != PA_OK)
        return rc;
    DeviceInfo *dev;
    if ((rc = device_info(&dev)) != PA_OK) return rc;
    StepMaps maps;
    if ((rc = make_maps(&maps, q, kv, num_q_tokens, num_q_heads)) != PA_OK) return rc;
    CascadeArgs casc;
    casc.prefix_blocks = prefix_blocks;
    casc.prefix_len = prefix_len;
    casc.ps = &ps;
    casc.prefix_o = reinterpret_cast<float *>(ws + L.prefix_o);
    casc.prefix_lse = reinterpret_cast<float *>(ws + L.prefix_lse);
    casc.suffix_o = reinterpret_cast<float *>(ws + L.extra_o);
    casc.suffix_lse = reinterpret_cast<float *>(ws + L.extra_lse);
    return run_step(q, kv, block_tables, max_blocks_per_seq, query_start_loc, context_lens,
                    seq_lens, num_seqs, num_q_tokens, num_q_heads, scale, out, lse, ws, L,
                    kShortMaxRows, 0, &casc, true, maps, Staging(), dev,
                    static_cast<cudaStream_t>(stream));
}

size_t pa_cascade_fp8_staging_bytes(int32_t num_kv_heads, int32_t head_dim,
                                    int32_t block_size, int32_t prefix_len) {
    if (num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || prefix_len < 0) return 0;
    return prefix_stage_bytes(num_kv_heads, head_dim, block_size, prefix_len);
}

// pa_validate_metadata; with window > 0 only the blocks of which some row of
// the request sees a key are looked at.
static int validate_metadata(const int32_t *block_tables, int32_t max_blocks_per_seq,
                             const int32_t *query_start_loc, const int32_t *context_lens,
                             const int32_t *seq_lens, int32_t num_seqs, int32_t num_q_tokens,
                             int32_t window, int32_t num_sinks, const int64_t *slot_mapping,
                             int32_t num_blocks, int32_t block_size) {
    g_err[0] = 0;
    if (num_seqs < 0 || num_q_tokens < 0 || block_size <= 0 || num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARG, "bad sizes");
    if (num_seqs > 0 && (!block_tables || !query_start_loc || !context_lens || !seq_lens))
        return fail(PA_ERR_INVALID_ARG, "metadata pointer is NULL");
    if (num_seqs > 0 && query_start_loc[0] != 0)
        return fail(PA_ERR_BAD_METADATA, "query_start_loc[0] = %d, expected 0", query_start_loc[0]);
    for (int b = 0; b < num_seqs; ++b) {
        const int n = query_start_loc[b + 1] - query_start_loc[b];
        if (n < 0) return fail(PA_ERR_BAD_METADATA, "query_start_loc decreases at %d", b);
        if (context_lens[b] < 0) return fail(PA_ERR_BAD_METADATA, "context_lens[%d] < 0", b);
        if (seq_lens[b] != context_lens[b] + n)
            return fail(PA_ERR_BAD_METADATA, "seq_lens[%d]=%d != context %d + q_len %d", b,
                        seq_lens[b], context_lens[b], n);
        const int64_t nblk = (static_cast<int64_t>(seq_lens[b]) + block_size - 1) / block_size;
        if (nblk > max_blocks_per_seq)
            return fail(PA_ERR_BAD_METADATA, "request %d needs %lld blocks > max_blocks_per_seq",
                        b, (long long)nblk);
        if (window > 0 && n == 0) continue;
        // blocks [hide_from, hide_to) lie between the sinks and the first row's window
        const int64_t hide_from = (static_cast<int64_t>(num_sinks) + block_size - 1) / block_size;
        const int64_t seen = static_cast<int64_t>(context_lens[b]) - window + 1;
        const int64_t hide_to = window > 0 && seen > 0 ? seen / block_size : 0;
        for (int64_t j = 0; j < nblk; ++j) {
            if (j >= hide_from && j < hide_to) continue;
            const int32_t blk = block_tables[static_cast<int64_t>(b) * max_blocks_per_seq + j];
            if (blk < 0 || blk >= num_blocks)
                return fail(PA_ERR_BAD_METADATA, "block_tables[%d][%lld] = %d out of range", b,
                            (long long)j, blk);
        }
    }
    if (num_seqs > 0 && query_start_loc[num_seqs] > num_q_tokens)
        return fail(PA_ERR_BAD_METADATA, "query_start_loc[num_seqs] = %d > num_q_tokens %d",
                    query_start_loc[num_seqs], num_q_tokens);
    if (slot_mapping && num_q_tokens > 0) {
        const int64_t nslots = static_cast<int64_t>(num_blocks) * block_size;
        // duplicates: mark slots in a bitmap
        std::vector<uint8_t> seen(static_cast<size_t>((nslots + 7) / 8), 0);
        for (int t = 0; t < num_q_tokens; ++t) {
            const int64_t s = slot_mapping[t];
            if (s < 0) continue;
            if (s >= nslots) return fail(PA_ERR_BAD_METADATA, "slot_mapping[%d] = %lld outside pool", t, (long long)s);
            uint8_t &byte = seen[static_cast<size_t>(s >> 3)];
            const uint8_t bit = static_cast<uint8_t>(1u << (s & 7));
            if (byte & bit) return fail(PA_ERR_BAD_METADATA, "slot %lld used twice", (long long)s);
            byte |= bit;
        }
    }
    return PA_OK;
}

int pa_validate_metadata(const int32_t *block_tables, int32_t max_blocks_per_seq,
                         const int32_t *query_start_loc, const int32_t *context_lens,
                         const int32_t *seq_lens, int32_t num_seqs, int32_t num_q_tokens,
                         const int64_t *slot_mapping, int32_t num_blocks, int32_t block_size) {
    return validate_metadata(block_tables, max_blocks_per_seq, query_start_loc, context_lens,
                             seq_lens, num_seqs, num_q_tokens, 0, 0, slot_mapping, num_blocks,
                             block_size);
}

int pa_validate_window_metadata(const int32_t *block_tables, int32_t max_blocks_per_seq,
                                const int32_t *query_start_loc, const int32_t *context_lens,
                                const int32_t *seq_lens, int32_t num_seqs, int32_t num_q_tokens,
                                int32_t window, int32_t num_sinks, const int64_t *slot_mapping,
                                int32_t num_blocks, int32_t block_size) {
    g_err[0] = 0;
    if (window < 1 || num_sinks < 0) return fail(PA_ERR_INVALID_ARG, "bad window or num_sinks");
    return validate_metadata(block_tables, max_blocks_per_seq, query_start_loc, context_lens,
                             seq_lens, num_seqs, num_q_tokens, window, num_sinks, slot_mapping,
                             num_blocks, block_size);
}

int pa_set_profile_events(int32_t which, void *start_event, void *end_event) {
    g_err[0] = 0;
    if (which < 0 || which > 3) return fail(PA_ERR_INVALID_ARG, "unknown kernel id %d", which);
    std::lock_guard<std::mutex> lock(g_prof_mu);
    g_prof[which][0] = start_event;
    g_prof[which][1] = end_event;
    return PA_OK;
}

int pa_set_tile_counter(uint64_t *counter) {
    g_err[0] = 0;
    if (counter && !aligned(counter, 8))
        return fail(PA_ERR_INVALID_ARG, "tile counter must be 8-byte aligned");
    g_tile_counter.store(counter, std::memory_order_relaxed);
    return PA_OK;
}

int pa_set_test_stall(int32_t which) {
    g_err[0] = 0;
    if (which < PA_TEST_STALL_NONE || which > PA_TEST_STALL_ROPE)
        return fail(PA_ERR_INVALID_ARG, "unknown test stall %d", which);
    g_test_stall.store(which, std::memory_order_relaxed);
    return PA_OK;
}

int pa_read_device_status(uint32_t *status, int clear, void *stream) {
    g_err[0] = 0;
    if (!status) return fail(PA_ERR_INVALID_ARG, "status is NULL");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) return fail(PA_ERR_CUDA, "stream sync failed");
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_pa_status, sizeof v) != cudaSuccess)
        return fail(PA_ERR_CUDA, "status read failed");
    *status = v;
    if (clear) {
        const unsigned zero = 0;
        if (cudaMemcpyToSymbol(g_pa_status, &zero, sizeof zero) != cudaSuccess)
            return fail(PA_ERR_CUDA, "status clear failed");
    }
    return PA_OK;
}

uint64_t pa_kernel_launches(void) { return g_launches.load(std::memory_order_relaxed); }

}  // extern "C"
