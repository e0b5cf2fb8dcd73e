// Cutting the cached tokens of long requests down to those with the most attention weight, and giving pages
// back to the free list.
//
// Eviction, per (request, KV head): of n weights between the sink and the recent tokens the m largest are
// kept, equal ones the earlier first.  A cluster of CTAs shares the places in contiguous slices:
//   1. each weight becomes a 32-bit key that orders as the weights do; three rounds of a histogram (11, 11, 10
//      bits from the top; every CTA adds the cluster's histograms up through shared memory of the
//      others) find the key of the m-th largest and how many equal ones are kept;
//   2. each CTA counts its keys above and at that key, learns the counts before its slice from the others,
//      and writes its kept places in order;
//   3. keys, values and weights move down in windows: every CTA reads its tokens of the
//      window into registers, the cluster meets, every CTA writes.  A token never moves up, so a
//      write hits only places whose tokens this window or an earlier one has read.
// Bound by HBM where there are many requests: the weights are read once (slices stay in shared memory), every moved
// token read and written once; by the trips to memory (about eight in a row, then two a window) where there are few.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>

#include <cmath>

#include "fm_paged.h"
#include "fm_ptx.cuh"

namespace cg = cooperative_groups;

namespace fm {
namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictCluster = 8;        // portable cluster size
constexpr int kBins = 2048;
constexpr int kHeld = 12288;            // keys of a slice that stay in shared memory (48 KB); longer slices are read again
constexpr int kMoves = 8;               // pieces of 16 bytes of a thread per window

struct EvictArgs {
    uint8_t *kv[2];
    int64_t page[2], head[2], tok[2];   // bytes
    const int32_t *lens, *table;
    float *weights;
    int32_t *kept, *new_lens, *status;
    int64_t max_tokens;                 // of a request
    int32_t max_pages, num_pages, page_size, Hkv;
    int32_t pieces;                     // of 16 bytes in a row
    int32_t piece_shift;                // log2 of the pieces of a token's key and value
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

__global__ void __launch_bounds__(kEvictThreads, 2) fm_paged_evict_kernel(const EvictArgs a)
{
    extern __shared__ __align__(16) uint32_t s_key[];       // [kHeld]
    __shared__ int s_hist[3][kBins];
    __shared__ int s_warp[kEvictWarps];
    __shared__ int s_bad, s_bin, s_need, s_count[2];
    cg::cluster_group cl = cg::this_cluster();
    const int ctas = (int)cl.num_blocks(), cta = (int)cl.block_rank(), tid = threadIdx.x;
    const int64_t unit = blockIdx.x / (unsigned)ctas;
    const int r = (int)(unit / a.Hkv), h = (int)(unit - (int64_t)r * a.Hkv);
    const int len = a.lens[r];
    const bool in_range = len >= 0 && len <= a.max_tokens;
    int32_t *kept = a.kept + unit * a.budget;
    const int32_t *table = a.table + (int64_t)r * a.max_pages;
    auto leave = [&](int32_t code) {
        for (int i = cta * kEvictThreads + tid; i < a.budget; i += ctas * kEvictThreads) kept[i] = -1;
        if (cta == 0 && tid == 0) {
            if (code != FM_OK) set_status(a.status, code);
            if (h == 0) a.new_lens[r] = len;
        }
    };
    if (!in_range || len <= a.budget) {             // the whole cluster
        leave(in_range ? FM_OK : FM_ERR_LENGTHS);
        return;
    }
    const int n = len - a.recent - a.sink, m = a.budget - a.recent - a.sink;        // m of n; m < n
    const int slice = (n + ctas - 1) / ctas;
    const int first = min(cta * slice, n), mine = min(slice, n - first);            // places sink + first ..
    const float *weights = a.weights + (int64_t)h * a.page_size;
    const int64_t page_weights = (int64_t)a.Hkv * a.page_size;
    auto weight_at = [&](int i) {
        const int p = a.sink + first + i, b = p / a.page_size;
        const int page = __ldg(table + b);
        return (unsigned)page < (unsigned)a.num_pages ? weights + page * page_weights + (p - b * a.page_size) : nullptr;
    };
    auto key_of = [&](int i) -> uint32_t {
        if (i < kHeld) return s_key[i];
        const float *w = weight_at(i);
        return w ? order_of(*w) : 0u;
    };

    for (int i = tid; i < 3 * kBins; i += kEvictThreads) s_hist[0][i] = 0;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    // Every page of the request is one of the pool's, or the request is left alone.
    const int pages = (int)(((int64_t)len + a.page_size - 1) / a.page_size);
    for (int b = cta * kEvictThreads + tid; b < pages; b += ctas * kEvictThreads)
        if ((unsigned)__ldg(table + b) >= (unsigned)a.num_pages) s_bad = 1;
    if (m > 0) {
        for (int i = tid; i < mine; i += kEvictThreads) {
            const float *w = weight_at(i);
            const uint32_t key = w ? order_of(*w) : 0u;
            if (i < kHeld) s_key[i] = key;
            atomicAdd(&s_hist[0][key >> 21], 1);
        }
    }
    cl.sync();
    bool bad = false;
    for (int c = 0; c < ctas; ++c) bad |= *cl.map_shared_rank(&s_bad, c) != 0;
    if (bad) {
        cl.sync();                                  // the others have read this CTA's flag
        leave(FM_ERR_PAGES);
        return;
    }

    // The key of the m-th largest, from the top bits down: `prefix` its bits so far, `need` the keys
    // with that prefix that are kept.
    uint32_t prefix = 0;
    int need = m;
    if (m > 0) {
#pragma unroll 1
        for (int round = 0; round < 3; ++round) {
            const int shift = round == 0 ? 21 : round == 1 ? 10 : 0, bins = round == 2 ? 1024 : kBins;
            if (round > 0) {
                const int above = round == 1 ? 21 : 10;
                for (int i = tid; i < mine; i += kEvictThreads) {
                    const uint32_t key = key_of(i);
                    if (key >> above == prefix) atomicAdd(&s_hist[round][(key >> shift) & (bins - 1)], 1);
                }
                cl.sync();
            }
            // Thread t's bins are the t-th group from the top.
            const int per = bins / kEvictThreads;
            int sum = 0;
            for (int c = 0; c < ctas; ++c) {
                const int *hist = cl.map_shared_rank(&s_hist[round][0], c);
                for (int j = 0; j < per; ++j) sum += hist[bins - 1 - (tid * per + j)];
            }
            int total;
            int before = block_before(sum, &total, s_warp);
            if (before < need && before + sum >= need) {
                for (int j = 0; j < per; ++j) {
                    const int bin = bins - 1 - (tid * per + j);
                    int x = 0;
                    for (int c = 0; c < ctas; ++c) x += cl.map_shared_rank(&s_hist[round][0], c)[bin];
                    if (before + x >= need) {
                        s_bin = bin;
                        s_need = need - before;
                        break;
                    }
                    before += x;
                }
            }
            __syncthreads();
            prefix = prefix << (round == 2 ? 10 : 11) | (uint32_t)s_bin;
            need = s_need;
            __syncthreads();
        }
        // How many of the slice lie above the key and at it.
        int above = 0, at = 0;
        for (int i = tid; i < mine; i += kEvictThreads) {
            const uint32_t key = key_of(i);
            above += key > prefix;
            at += key == prefix;
        }
        int total_above, total_at;
        block_before(above, &total_above, s_warp);
        block_before(at, &total_at, s_warp);
        if (tid == 0) {
            s_count[0] = total_above;
            s_count[1] = total_at;
        }
        cl.sync();
        int run_above = 0, run_at = 0;
        for (int c = 0; c < cta; ++c) {
            run_above += cl.map_shared_rank(&s_count[0], c)[0];
            run_at += cl.map_shared_rank(&s_count[0], c)[1];
        }
        for (int i0 = 0; i0 < mine; i0 += kEvictThreads) {
            const int i = i0 + tid;
            const uint32_t key = i < mine ? key_of(i) : 0u;
            const bool up = i < mine && key > prefix, eq = i < mine && key == prefix;
            int total;
            const int before = block_before((up ? 1 : 0) | (eq ? 1 << 16 : 0), &total, s_warp);    // at most 512 of each
            const int ups = run_above + (before & 0xffff), eqs = run_at + (before >> 16);
            if (up || (eq && eqs < need)) kept[a.sink + ups + min(eqs, need)] = a.sink + first + i;
            run_above += total & 0xffff;
            run_at += total >> 16;
        }
    }
    for (int i = cta * kEvictThreads + tid; i < a.sink; i += ctas * kEvictThreads) kept[i] = i;
    for (int i = cta * kEvictThreads + tid; i < a.recent; i += ctas * kEvictThreads) kept[a.budget - a.recent + i] = len - a.recent + i;
    if (cta == 0 && tid == 0 && h == 0) a.new_lens[r] = a.budget;
    cl.sync();                                      // the kept places are visible to the cluster

    // Windows of kMoves pieces a thread.
    const int per_token = 1 << a.piece_shift, tokens = kEvictThreads >> a.piece_shift;      // tokens of a step of the CTA
    const int piece = tid & (per_token - 1), which = piece >= a.pieces ? 1 : 0;
    const int64_t col = (int64_t)h * a.head[which] + (int64_t)(piece - which * a.pieces) * 16;
    const int window = tokens * kMoves * ctas;
    for (int w0 = a.sink; w0 < a.budget; w0 += window) {
        const int j0 = w0 + cta * tokens * kMoves + (tid >> a.piece_shift);
        uint4 x[kMoves];
        float w[kMoves];
        int from[kMoves];
#pragma unroll
        for (int i = 0; i < kMoves; ++i) {
            const int j = j0 + i * tokens;
            from[i] = j < a.budget ? __ldcg(kept + j) : j;
        }
#pragma unroll
        for (int i = 0; i < kMoves; ++i) {
            const int j = j0 + i * tokens;
            if (j >= a.budget || from[i] == j) continue;
            const int b = from[i] / a.page_size;
            const int64_t page = __ldg(table + b), in = from[i] - b * a.page_size;
            x[i] = __ldcg(reinterpret_cast<const uint4 *>(a.kv[which] + page * a.page[which] + in * a.tok[which] + col));
            if (piece == 0) w[i] = __ldcg(weights + page * page_weights + in);
        }
        cl.sync();
#pragma unroll
        for (int i = 0; i < kMoves; ++i) {
            const int j = j0 + i * tokens;
            if (j >= a.budget || from[i] == j) continue;
            const int b = j / a.page_size;
            const int64_t page = __ldg(table + b), in = j - b * a.page_size;
            *reinterpret_cast<uint4 *>(a.kv[which] + page * a.page[which] + in * a.tok[which] + col) = x[i];
            if (piece == 0) a.weights[(int64_t)h * a.page_size + page * page_weights + in] = w[i];
        }
    }
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
    if (!aligned4(lens) || !aligned4(block_table) || !aligned4(weights) || !aligned4(kept) || !aligned4(new_lens) || !aligned4(dev_status) ||
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
    for (a.piece_shift = 0; 1 << a.piece_shift < 2 * a.pieces; ++a.piece_shift) {}
    a.budget = budget;
    a.recent = recent;
    a.sink = sink;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((int64_t)requests * cache->Hkv * kEvictCluster));
    cfg.blockDim = dim3(kEvictThreads);
    cfg.dynamicSmemBytes = kHeld * 4;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kEvictCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    static std::atomic<uint8_t> done[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FM_ERR_CUDA;
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(fm_paged_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeld * 4) != cudaSuccess) return FM_ERR_CUDA;
        done[dev].store(1, std::memory_order_release);
    }
    ProfScope ps(kKPagedEvict, stream);
    return cudaLaunchKernelEx(&cfg, fm_paged_evict_kernel, a) == cudaSuccess ? FM_OK : FM_ERR_CUDA;
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
