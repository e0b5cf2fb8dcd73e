// Cutting the cached tokens of long requests down to those with the most attention weight, and giving pages
// back to the free list.
//
// Eviction, per (request, KV head): of n weights between the sink and the recent tokens the m largest are
// kept, equal ones the earlier first.  A cluster of CTAs shares the places in contiguous slices:
//   1. each weight becomes a 32-bit key that orders as the weights do; three rounds of a histogram (11, 11, 10
//      bits from the top; every CTA adds the cluster's histograms up through shared memory of the
//      others) find the key of the m-th largest and how many equal ones are kept;
//   2. each warp counts its keys above and at that key, learns the counts before its own from the others,
//      and writes its kept places in order;
//   3. keys, values and weights move down in windows: every CTA has its tokens of the window copied to shared
//      memory, a window ahead, the cluster meets, every CTA writes.  A token never moves up, so a
//      write hits only places whose tokens this window or an earlier one has read.
// Bound by HBM where there are many requests: the weights are read once (they stay in shared memory), every moved
// token read and written once; by the trips to memory and the meetings (about ten in a row, then one a window) where
// there are few.  Steps, of 32 requests of up to 12,000 tokens cut to 4,096 and of one of 128K cut to 16K in e4m3: windows
// of registers without copies ahead, histograms read one count at a time 427 and 122 us; copies ahead, 16 bytes of a histogram at
// a time 213 and 90; places by warps instead of block-wide scans, weights 16 bytes at a time, and a meeting that waits for no
// stores (each thread's would have to reach L2 first) 156 and 82; key and value of a token by the same threads 124 and 65; pages
// looked up a window before they are used 113 and 52. (Bulk copies of a row each instead, a thread per token: 258 and 148.)
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "fm_paged.h"
#include "fm_ptx.cuh"

namespace cg = cooperative_groups;

namespace fm {
namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kBins = 2048;
constexpr int kHeld = 16384;            // keys of a CTA that stay in shared memory (64 KB); more are read again
constexpr int kLoads = 4;               // groups of four weights of a thread in flight
constexpr int kMoves = 2, kStages = 2;  // tokens of a thread per window; windows in shared memory
constexpr int kStageBytes = kMoves * kEvictThreads * 32;
constexpr int kEvictBytes = 3 * kBins * 4 + kHeld * 4;
static_assert(kStages * (kStageBytes + kMoves * (kEvictThreads / 4) * 4) <= kEvictBytes, "the windows fit where the keys were");   // 4 pieces a row at least

struct EvictArgs {
    uint8_t *kv[2];
    int64_t page[2], head[2], tok[2];   // bytes
    const int32_t *lens, *table;
    float *weights;
    int32_t *kept, *new_lens, *status;
    int64_t max_tokens;                 // of a request
    int32_t max_pages, num_pages, page_size, Hkv;
    int32_t pieces;                     // of 16 bytes in a row
    int32_t piece_shift;                // log2 of them
    int32_t page_shift;                 // log2 of the page size, -1 if it is no power of two
    int32_t budget, recent, sink;
};

// The order of the weights as that of unsigned integers: larger weights larger, both zeros the same, NaN on top.
__device__ __forceinline__ uint32_t order_of(float w)
{
    if (w != w) return 0xffffffffu;
    const uint32_t b = __float_as_uint(w + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Sums of x over the block's threads before this one, and over all of them.
__device__ __forceinline__ int block_before(int x, int *total, int *sh)
{
    const int lane = lane_id(), warp = threadIdx.x >> 5;
    int y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    if (lane == 31) sh[warp] = y;
    __syncthreads();
    int w = lane < kEvictWarps ? sh[lane] : 0;
#pragma unroll
    for (int o = 1; o < kEvictWarps; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += z;
    }
    *total = __shfl_sync(0xffffffffu, w, kEvictWarps - 1);
    const int before = warp > 0 ? __shfl_sync(0xffffffffu, w, max(warp - 1, 0)) : 0;
    __syncthreads();
    return before + y - x;
}

// Adds a CTA's counts of keys by digit to those of the cluster, of which each CTA holds its share of the digits.  (Every CTA reading
// the counts of all the others instead takes 2 us a round for 1, with eight of them.)
template <int C, int BINS>
__device__ __forceinline__ void share_counts(const cg::cluster_group &cl, const int *hist, int *shared)
{
    if (C == 1) return;
    __syncthreads();
    for (int i = threadIdx.x; i < BINS; i += kEvictThreads) {
        const int x = hist[i];
        if (x) atomicAdd(cl.map_shared_rank(shared + i % (BINS / C), i / (BINS / C)), x);
    }
}

// Finds, among the cluster's counts, the digit of the need-th largest key; *need becomes its rank
// among the keys of that digit.  Thread t looks at the t-th PER digits from the top.
template <int C, int BINS>
__device__ __forceinline__ int digit_of(const cg::cluster_group &cl, int *hist, int *shared, int *need, int *s_warp, int *s_found)
{
    constexpr int PER = BINS / kEvictThreads;
    static_assert((PER == 4 || PER == 2) && BINS / C % PER == 0, "digits of a thread");
    using V = typename std::conditional<PER == 4, int4, int2>::type;
    const int at = BINS / PER - 1 - threadIdx.x, owner = at * PER / (BINS / C);
    int count[PER] = {};
    {
        const V v = *reinterpret_cast<const V *>(C > 1 ? cl.map_shared_rank(shared + at * PER - owner * (BINS / C), owner) : hist + at * PER);
        count[0] = v.x;
        count[1] = v.y;
        if constexpr (PER == 4) {
            count[2] = v.z;
            count[3] = v.w;
        }
    }
    int sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += count[i];
    int total, before = block_before(sum, &total, s_warp);
    if (before < *need && before + sum >= *need) {
#pragma unroll
        for (int i = PER - 1; i >= 0; --i) {
            if (before < *need && before + count[i] >= *need) {
                s_found[0] = at * PER + i;
                s_found[1] = *need - before;
            }
            before += count[i];
        }
    }
    __syncthreads();
    *need = s_found[1];
    const int digit = s_found[0];
    __syncthreads();
    return digit;
}

template <int C>
__global__ void __launch_bounds__(kEvictThreads, 2) fm_paged_evict_kernel(const EvictArgs a)
{
    // The histograms and the keys, later the tokens on their way.
    extern __shared__ __align__(16) uint8_t smem[];
    int (*s_hist)[kBins] = reinterpret_cast<int (*)[kBins]>(smem);
    uint4 *s_key = reinterpret_cast<uint4 *>(smem + 3 * kBins * 4);             // [kHeld / 4]
    float *s_moved = reinterpret_cast<float *>(smem + kStages * kStageBytes);    // [kStages][kMoves][tokens of a step]
    __shared__ int s_warp[kEvictWarps];
    __shared__ int s_bad, s_found[2];
    __shared__ int2 s_count[kEvictWarps];
    __shared__ __align__(16) int s_shared[3][C > 1 ? kBins / C : 4];
    const cg::cluster_group cl = cg::this_cluster();
    auto meet = [&]() {
        if (C > 1) cl.sync();
        else __syncthreads();
    };
    const int cta = C > 1 ? (int)cl.block_rank() : 0, tid = threadIdx.x;
    const int64_t unit = blockIdx.x / (unsigned)C;
    const int r = (int)(unit / a.Hkv), h = (int)(unit - (int64_t)r * a.Hkv);
    const int len = a.lens[r];
    const bool in_range = len >= 0 && len <= a.max_tokens;
    int32_t *kept = a.kept + unit * a.budget;
    const int32_t *table = a.table + (int64_t)r * a.max_pages;
    auto leave = [&](int32_t code) {
        for (int i = cta * kEvictThreads + tid; i < a.budget; i += C * kEvictThreads) kept[i] = -1;
        if (cta == 0 && tid == 0) {
            if (code != FM_OK) set_status(a.status, code);
            if (h == 0) a.new_lens[r] = len;
        }
    };
    if (!in_range || len <= a.budget) {             // the whole cluster
        leave(in_range ? FM_OK : FM_ERR_LENGTHS);
        return;
    }
    const int lo = a.sink, hi = len - a.recent, m = a.budget - a.recent - a.sink;    // m of the places [lo, hi)
    // The places in groups of four that share a page and 16 bytes of weights; each warp of the cluster has
    // consecutive ones, and its lanes next to one another.
    const int g_lo = lo >> 2, groups = m > 0 ? ((hi + 3) >> 2) - g_lo : 0;
    const int per_warp = ((groups + C * kEvictWarps - 1) / (C * kEvictWarps) + 31) & ~31, per_cta = per_warp * kEvictWarps;
    const int warp = tid >> 5, lane = lane_id();
    const int own = warp * per_warp;                                                // the warp's first group of the CTA
    const int64_t head_weights = (int64_t)h * a.page_size, page_weights = (int64_t)a.Hkv * a.page_size;
    auto page_of = [&](int p) { return a.page_shift >= 0 ? p >> a.page_shift : p / a.page_size; };
    // Keys of the CTA's groups i, i + 32, ..: their loads are in flight together.  A place that is none of [lo, hi) has
    // key 0, which no weight has; so has a page outside the pool, whose request is then left alone.
    auto keys_of = [&](int i, uint4 (&key)[kLoads]) {
        int page[kLoads], in[kLoads];
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int64_t g = (int64_t)g_lo + (int64_t)cta * per_cta + i + 32 * q;
            page[q] = -1;
            if (4 * g >= hi) continue;
            const int p = (int)(4 * g), b = page_of(p);
            in[q] = p - b * a.page_size;
            page[q] = __ldg(table + b);
        }
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            key[q] = make_uint4(0u, 0u, 0u, 0u);
            if ((unsigned)page[q] >= (unsigned)a.num_pages) continue;
            const float4 w = *reinterpret_cast<const float4 *>(a.weights + page[q] * page_weights + head_weights + in[q]);
            const int p = (int)(4 * ((int64_t)g_lo + (int64_t)cta * per_cta + i + 32 * q));
            if (p >= lo) key[q].x = order_of(w.x);
            if (p + 1 >= lo && p + 1 < hi) key[q].y = order_of(w.y);
            if (p + 2 >= lo && p + 2 < hi) key[q].z = order_of(w.z);
            if (p + 3 >= lo && p + 3 < hi) key[q].w = order_of(w.w);
        }
    };
    // f(group, its keys) of the warp's groups, all lanes together.
    auto each = [&](auto f) {
        for (int i0 = 0; i0 < per_warp; i0 += 32 * kLoads) {
            uint4 key[kLoads];
            if (per_cta > kHeld / 4) {
                keys_of(own + i0 + lane, key);
            } else {
#pragma unroll
                for (int q = 0; q < kLoads; ++q) key[q] = i0 + 32 * q < per_warp ? s_key[own + i0 + 32 * q + lane] : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int q = 0; q < kLoads; ++q)
                if (i0 + 32 * q < per_warp) f(own + i0 + 32 * q + lane, key[q]);
        }
    };

    if (m > 0)
        for (int i = tid; i < 3 * kBins / 4; i += kEvictThreads) reinterpret_cast<int4 *>(s_hist)[i] = make_int4(0, 0, 0, 0);
    if (C > 1 && m > 0)
        for (int i = tid; i < 3 * kBins / C; i += kEvictThreads) s_shared[0][i] = 0;
    if (tid == 0) s_bad = 0;
    meet();                                         // every CTA's counts are zero
    // Every page of the request is one of the pool's, or the request is left alone.
    const int pages = page_of(len - 1) + 1;
    for (int b = cta * kEvictThreads + tid; b < pages; b += C * kEvictThreads)
        if ((unsigned)__ldg(table + b) >= (unsigned)a.num_pages) s_bad = 1;
    for (int i0 = 0; m > 0 && i0 < per_warp; i0 += 32 * kLoads) {
        uint4 key[kLoads];
        keys_of(own + i0 + lane, key);
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            if (i0 + 32 * q >= per_warp) break;
            if (per_cta <= kHeld / 4) s_key[own + i0 + 32 * q + lane] = key[q];
            const uint32_t k[4] = {key[q].x, key[q].y, key[q].z, key[q].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k[j]) atomicAdd(&s_hist[0][k[j] >> 21], 1);
        }
    }
    if (m > 0) share_counts<C, kBins>(cl, s_hist[0], s_shared[0]);
    meet();
    bool bad = false;
#pragma unroll
    for (int c = 0; c < C; ++c) bad |= *(C > 1 ? cl.map_shared_rank(&s_bad, c) : &s_bad) != 0;
    if (bad) {
        meet();                                     // the others have read this CTA's flag
        leave(FM_ERR_PAGES);
        return;
    }

    // The key of the m-th largest, from the top bits down: `prefix` its bits so far, `need` the keys
    // with that prefix that are kept.
    if (m > 0) {
        int need = m;
        uint32_t prefix = (uint32_t)digit_of<C, kBins>(cl, s_hist[0], s_shared[0], &need, s_warp, s_found);
        each([&](int, const uint4 &key) {
            const uint32_t k[4] = {key.x, key.y, key.z, key.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k[j] >> 21 == prefix && k[j]) atomicAdd(&s_hist[1][(k[j] >> 10) & 2047], 1);
        });
        share_counts<C, kBins>(cl, s_hist[1], s_shared[1]);
        meet();
        prefix = prefix << 11 | (uint32_t)digit_of<C, kBins>(cl, s_hist[1], s_shared[1], &need, s_warp, s_found);
        each([&](int, const uint4 &key) {
            const uint32_t k[4] = {key.x, key.y, key.z, key.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k[j] >> 10 == prefix && k[j]) atomicAdd(&s_hist[2][k[j] & 1023], 1);
        });
        share_counts<C, 1024>(cl, s_hist[2], s_shared[2]);
        meet();
        prefix = prefix << 10 | (uint32_t)digit_of<C, 1024>(cl, s_hist[2], s_shared[2], &need, s_warp, s_found);
        // How many of the warp's keys lie above that key and at it, and how many of the warps and CTAs before.
        int above = 0, at = 0;
        each([&](int, const uint4 &key) {
            above += (key.x > prefix) + (key.y > prefix) + (key.z > prefix) + (key.w > prefix);
            at += (key.x == prefix) + (key.y == prefix) + (key.z == prefix) + (key.w == prefix);
        });
        above = __reduce_add_sync(0xffffffffu, above);
        at = __reduce_add_sync(0xffffffffu, at);
        if (lane == 0) s_count[warp] = make_int2(above, at);
        meet();
        above = at = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {               // lane w: warp w of CTA c
            int2 v = make_int2(0, 0);
            if (lane < kEvictWarps && (c < cta || (c == cta && lane < warp))) v = (C > 1 ? cl.map_shared_rank(&s_count[0], c) : s_count)[lane];
            above += v.x;
            at += v.y;
        }
        int run_above = __reduce_add_sync(0xffffffffu, above), run_at = __reduce_add_sync(0xffffffffu, at);
        each([&](int i, const uint4 &key) {
            const uint32_t k[4] = {key.x, key.y, key.z, key.w};
            int count = 0;                          // above | at << 16: 128 of a step at most
#pragma unroll
            for (int j = 0; j < 4; ++j) count += (k[j] > prefix ? 1 : 0) + (k[j] == prefix ? 1 << 16 : 0);
            int upto = count;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            int ups = run_above + ((upto - count) & 0xffff), eqs = run_at + ((upto - count) >> 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (k[j] > prefix || (k[j] == prefix && eqs < need))
                    kept[a.sink + ups + min(eqs, need)] = (int)(4 * ((int64_t)g_lo + (int64_t)cta * per_cta + i)) + j;
                ups += k[j] > prefix;
                eqs += k[j] == prefix;
            }
            const int total = __shfl_sync(0xffffffffu, upto, 31);
            run_above += total & 0xffff;
            run_at += total >> 16;
        });
    }
    for (int i = cta * kEvictThreads + tid; i < a.sink; i += C * kEvictThreads) kept[i] = i;
    for (int i = cta * kEvictThreads + tid; i < a.recent; i += C * kEvictThreads) kept[a.budget - a.recent + i] = len - a.recent + i;
    if (cta == 0 && tid == 0 && h == 0) a.new_lens[r] = a.budget;
    meet();                                          // the kept places are visible to the cluster

    // Windows of kMoves tokens a thread, of each of which it moves 16 bytes of the key and of the value, kStages - 1 of them on
    // their way to shared memory while one is written.
    const int tokens = kEvictThreads >> a.piece_shift, mate = tid >> a.piece_shift;      // tokens of a step of the CTA
    const int piece = tid & (a.pieces - 1);
    const int64_t col_k = (int64_t)h * a.head[0] + piece * 16, col_v = (int64_t)h * a.head[1] + piece * 16;
    const int window = tokens * kMoves * C, j0 = a.sink + cta * tokens * kMoves + mate;
    const int windows = (a.budget - a.sink + window - 1) / window;
    auto sources = [&](int w, int (&from)[kMoves]) {
#pragma unroll
        for (int i = 0; i < kMoves; ++i) {
            const int64_t j = (int64_t)w * window + j0 + i * tokens;
            from[i] = w < windows && j < a.budget ? __ldcg(kept + j) : -1;
        }
    };
    // Pages of places (those that are none: -1), and of the window's own tokens: looked up a window before they are used.
    auto pages_of = [&](const int (&at)[kMoves], int (&page)[kMoves]) {
#pragma unroll
        for (int i = 0; i < kMoves; ++i) page[i] = at[i] >= 0 ? __ldg(table + page_of(at[i])) : 0;
    };
    auto targets = [&](int w, int (&page)[kMoves]) {
        int at[kMoves];
#pragma unroll
        for (int i = 0; i < kMoves; ++i) {
            const int64_t j = (int64_t)w * window + j0 + i * tokens;
            at[i] = w < windows && j < a.budget ? (int)j : -1;
        }
        pages_of(at, page);
    };
    // Starts the loads of window w; a bit for each token that moves.
    auto start = [&](int w, const int (&from)[kMoves], const int (&pages)[kMoves]) {
        unsigned moves = 0;
        uint8_t *stage = smem + (w % kStages) * kStageBytes;
#pragma unroll
        for (int i = 0; i < kMoves; ++i) {
            if (from[i] < 0 || from[i] == w * window + j0 + i * tokens) continue;
            moves |= 1u << i;
            const int in = from[i] - page_of(from[i]) * a.page_size;
            const int64_t page = pages[i];
            copy_async16(stage + (i * 2 * kEvictThreads + tid) * 16, a.kv[0] + page * a.page[0] + in * a.tok[0] + col_k);
            copy_async16(stage + ((i * 2 + 1) * kEvictThreads + tid) * 16, a.kv[1] + page * a.page[1] + in * a.tok[1] + col_v);
            if (piece == 0) copy_async4(s_moved + ((w % kStages) * kMoves + i) * tokens + mate, a.weights + page * page_weights + head_weights + in);
        }
        copy_async_commit();
        return moves;
    };
    unsigned moves[kStages] = {};
    int from[kMoves], next[kMoves], from_page[kMoves], to_page[kMoves];
#pragma unroll
    for (int w = 0; w < kStages - 1; ++w) {
        sources(w, from);
        pages_of(from, from_page);
        moves[w] = start(w, from, from_page);
    }
    sources(kStages - 1, from);
    sources(kStages, next);
    pages_of(from, from_page);
    targets(0, to_page);
    for (int w = 0; w < windows; ++w) {
        copy_async_wait<kStages - 2>();
        if (C > 1) cluster_arrive_relaxed();               // this thread has read its sources of the window
        moves[kStages - 1] = start(w + kStages - 1, from, from_page);
        int page_now[kMoves];
#pragma unroll
        for (int i = 0; i < kMoves; ++i) {
            page_now[i] = to_page[i];
            from[i] = next[i];
        }
        pages_of(from, from_page);
        targets(w + 1, to_page);
        sources(w + kStages + 1, next);
        if (C > 1) cluster_wait();                   // and every other
        else __syncthreads();
        const uint8_t *stage = smem + (w % kStages) * kStageBytes;
#pragma unroll
        for (int i = 0; i < kMoves; ++i) {
            if (!(moves[0] >> i & 1u)) continue;
            const int j = w * window + j0 + i * tokens;
            const int in = j - page_of(j) * a.page_size;
            const int64_t page = page_now[i];
            *reinterpret_cast<uint4 *>(a.kv[0] + page * a.page[0] + in * a.tok[0] + col_k) = *reinterpret_cast<const uint4 *>(stage + (i * 2 * kEvictThreads + tid) * 16);
            *reinterpret_cast<uint4 *>(a.kv[1] + page * a.page[1] + in * a.tok[1] + col_v) = *reinterpret_cast<const uint4 *>(stage + ((i * 2 + 1) * kEvictThreads + tid) * 16);
            if (piece == 0) a.weights[page * page_weights + head_weights + in] = s_moved[((w % kStages) * kMoves + i) * tokens + mate];
        }
#pragma unroll
        for (int i = 0; i + 1 < kStages; ++i) moves[i] = moves[i + 1];
    }
    copy_async_wait<0>();
}

// ---- release ---------------------------------------------------------------------------
// One CTA: lengths to page counts and their sums, the pages looked at, then handed back: all or none.
// Latency-bound: three dependent reads (lengths, table, head) around a block scan.
constexpr int kReleaseThreads = 512;
static_assert(kReleaseThreads == kEvictThreads, "block_before");

struct ReleaseArgs {
    const int32_t *held, *lens, *table;
    int32_t *free_pages;
    const int32_t *free_head;
    int32_t *free_next, *seq, *status;
    int64_t max_tokens;
    int32_t R, max_pages, num_pages, page_size, n_free;
};

__global__ void __launch_bounds__(kReleaseThreads) fm_paged_release_kernel(const ReleaseArgs a)
{
    extern __shared__ int32_t s_off[];      // [R] pages before request r
    int32_t *s_first = s_off + a.R;         // [R] its first page to give back
    __shared__ int s_warp[kEvictWarps];
    const int tid = threadIdx.x;
    const int32_t head = a.free_pages ? *a.free_head : 0;
    bool bad = false;
    int64_t run = 0;
    for (int r0 = 0; r0 < a.R; r0 += kReleaseThreads) {
        const int r = r0 + tid;
        int count = 0;
        if (r < a.R) {
            const int64_t held = a.held[r], len = a.lens[r];
            if (len < 0 || len > held || held > a.max_tokens) {
                bad = true;
            } else {
                const int64_t want = (len + a.page_size - 1) / a.page_size;
                count = (int)((held + a.page_size - 1) / a.page_size - want);
                s_first[r] = (int)want;
            }
        }
        // A request has 2^27 pages at most, a block of them more than 31 bits hold: in two parts.
        int total_lo, total_hi;
        const int lo = block_before(count & 4095, &total_lo, s_warp), hi = block_before(count >> 12, &total_hi, s_warp);
        if (r < a.R) s_off[r] = (int)min(run + ((int64_t)hi << 12) + lo, (int64_t)INT32_MAX);    // (past the list's length nothing is given back)
        run += ((int64_t)total_hi << 12) + total_lo;
    }
    int32_t err = FM_OK;
    if (__syncthreads_or(bad)) err = FM_ERR_LENGTHS;
    else if (a.free_pages && (head < 0 || head > a.n_free || run > head)) err = FM_ERR_PAGES;
    int n = err == FM_OK && a.free_pages ? (int)run : 0;
    bad = false;
    for (int x = tid; x < n; x += kReleaseThreads) {
        const int r = last_at_most(s_off, a.R, x);
        bad |= (unsigned)a.table[(int64_t)r * a.max_pages + s_first[r] + x - s_off[r]] >= (unsigned)a.num_pages;
    }
    if (__syncthreads_or(bad)) err = FM_ERR_PAGES;
    if (err != FM_OK) n = 0;
    for (int x = tid; x < n; x += kReleaseThreads) {
        const int r = last_at_most(s_off, a.R, x);
        a.free_pages[head - n + x] = a.table[(int64_t)r * a.max_pages + s_first[r] + x - s_off[r]];
    }
    const int32_t *now = err == FM_OK ? a.lens : a.held;
    for (int r = tid; r < a.R; r += kReleaseThreads) a.seq[r] = now[r];
    if (tid == 0) {
        if (a.free_pages) *a.free_next = head - n;
        if (err != FM_OK) set_status(a.status, err);
    }
}

template <int C>
fm_status launch_evict(const EvictArgs &a, int64_t units, cudaStream_t stream)
{
    static std::atomic<uint8_t> done[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FM_ERR_CUDA;
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(fm_paged_evict_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictBytes) != cudaSuccess) return FM_ERR_CUDA;
        done[dev].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(units * C));
    cfg.blockDim = dim3(kEvictThreads);
    cfg.dynamicSmemBytes = kEvictBytes;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fm_paged_evict_kernel<C>, a) == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

}  // namespace
}  // namespace fm

using namespace fm;

extern "C" {

fm_status fm_paged_evict(const fm_paged_cache *cache, int requests, int max_pages, const int32_t *lens, const int32_t *block_table,
                         float *weights, int budget, int recent, int sink, int32_t *kept, int32_t *new_lens, int32_t *dev_status,
                         fm_stream_t stream)
{
    fm_status st = check_cache(cache);
    if (st != FM_OK) return st;
    if (requests <= 0 || max_pages <= 0 || budget <= 0 || recent < 0 || sink < 0 || (int64_t)recent + sink > budget) return FM_ERR_INVALID_ARG;
    if (!aligned4(lens) || !aligned4(block_table) || !aligned16(weights) || !aligned4(kept) || !aligned4(new_lens) || !aligned4(dev_status) ||
        lens == new_lens)
        return FM_ERR_INVALID_ARG;
    if (requests > kMaxRequests || (int64_t)max_pages * cache->page_size > (int64_t)0x7fffffff - 2 * kMaxPage) return FM_ERR_UNSUPPORTED;
    if ((st = device_ok()) != FM_OK) return st;
    const int64_t esz = cache->dtype == FM_DT_E4M3 ? 1 : 2;
    EvictArgs a{};
    a.kv[0] = (uint8_t *)cache->k, a.kv[1] = (uint8_t *)cache->v;
    a.page[0] = cache->k_page * esz, a.page[1] = cache->v_page * esz;
    a.head[0] = cache->k_head * esz, a.head[1] = cache->v_head * esz;
    a.tok[0] = cache->k_tok * esz, a.tok[1] = cache->v_tok * esz;
    a.lens = lens;
    a.table = block_table;
    a.weights = weights;
    a.kept = kept;
    a.new_lens = new_lens;
    a.status = dev_status;
    a.max_tokens = (int64_t)max_pages * cache->page_size;
    a.max_pages = max_pages;
    a.num_pages = cache->num_pages;
    a.page_size = cache->page_size;
    a.Hkv = cache->Hkv;
    a.pieces = (int)(cache->d * esz / 16);
    for (a.piece_shift = 0; 1 << a.piece_shift < a.pieces; ++a.piece_shift) {}
    a.budget = budget;
    a.recent = recent;
    a.sink = sink;
    a.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (a.page_size == 1 << i) a.page_shift = i;
    const int64_t units = (int64_t)requests * cache->Hkv;
    cudaStream_t cs = (cudaStream_t)stream;
    ProfScope ps(kKPagedEvict, stream);
    // CTAs per unit by the number of units, at measured crossovers: the lengths are on the device.  More CTAs shorten a unit's
    // chain of loads, fewer leave room for more units at once (two CTAs a SM) and meet at less cost.  us with 1, 2, 4 and 8 a unit:
    //   12,000 tokens each to 4,096: 16 units 109, 57, 37, 39; 64 109, 72, 68, 84; 65 109, 72, 70, 82; 76 111, 78, 98, 100;
    //     304 254, 252, 268, 326; 305 303, 266, 268, 326; 512 395, 397, 424, 532
    //   spread below 12,000 (what is not cut leaves at once): 16 units 109, 55, 37, 29; 17 109, 57, 37, 37; 64 109, 55, 55, 39; 65 109, 57, 57, 45;
    //     160 109, 94, 74, 90; 256 180, 104, 117, 125; 384 176, 113, 123, 143; 512 182, 197, 182, 219
    //   2,000 each to 1,000: 17 units 35, 27, 23, 23; 64 35, 29, 29, 45; 76 35, 31, 45, 57; 152 41, 45, 70, 96; 304 70, 84, 115, 174
    // The rule is at the best of the four or within a fifth of it where all units are cut, and within 1.6 where few are.
    if (units <= 16) return launch_evict<8>(a, units, cs);
    if (units <= 64) return launch_evict<4>(a, units, cs);
    return units <= 304 ? launch_evict<2>(a, units, cs) : launch_evict<1>(a, units, cs);
}

fm_status fm_paged_release(int requests, int max_pages, int num_pages, int page_size, const int32_t *held, const int32_t *lens,
                           const int32_t *block_table, int32_t *free_pages, int n_free, const int32_t *free_head, int32_t *free_next,
                           int32_t *seq_lens, int32_t *dev_status, fm_stream_t stream)
{
    if (requests <= 0 || max_pages <= 0 || num_pages <= 0 || page_size <= 0) return FM_ERR_INVALID_ARG;
    if (!aligned4(held) || !aligned4(lens) || !aligned4(block_table) || !aligned4(seq_lens) || !aligned4(dev_status)) return FM_ERR_INVALID_ARG;
    if (free_pages && (((uintptr_t)free_pages & 3u) || n_free < 0 || !aligned4(free_head) || !aligned4(free_next))) return FM_ERR_INVALID_ARG;
    if (requests > kMaxRequests || page_size % kPageGranule != 0 || page_size > kMaxPage ||
        (int64_t)max_pages * page_size > (int64_t)0x7fffffff - 2 * kMaxPage)
        return FM_ERR_UNSUPPORTED;
    const fm_status st = device_ok();
    if (st != FM_OK) return st;
    ReleaseArgs a{};
    a.held = held;
    a.lens = lens;
    a.table = block_table;
    a.free_pages = free_pages;
    a.free_head = free_head;
    a.free_next = free_next;
    a.seq = seq_lens;
    a.status = dev_status;
    a.max_tokens = (int64_t)max_pages * page_size;
    a.R = requests;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.n_free = n_free;
    static std::atomic<uint8_t> done[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FM_ERR_CUDA;
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(fm_paged_release_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRequests * 8) != cudaSuccess)
            return FM_ERR_CUDA;
        done[dev].store(1, std::memory_order_release);
    }
    ProfScope ps(kKPagedRelease, stream);
    fm_paged_release_kernel<<<1, kReleaseThreads, (size_t)requests * 8, (cudaStream_t)stream>>>(a);
    return cudaPeekAtLastError() == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

}  // extern "C"
