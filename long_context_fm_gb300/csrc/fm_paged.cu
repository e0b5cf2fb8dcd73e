// Paged key/value cache: the step's planner (block tables, slot map, positions
// and the attention's work list from request lengths), the append of new keys
// and values, and the C entry points of both and of the attention.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "fm_paged.h"
#include "fm_ptx.cuh"

namespace cg = cooperative_groups;

namespace fm {

// ---- planner -------------------------------------------------------------------
// One cluster: every CTA scans the request lengths for itself (they are few
// next to the tokens) and writes its share of the tokens' slots and of the
// new table entries; CTA 0 also writes what there is once per request.  The
// cluster barrier at the end lets the lengths and the free-list head be
// advanced in place.  Latency-bound: two dependent reads (lengths, then a table
// entry or a free page) around one block scan.
constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanCluster = 8;         // portable cluster size
constexpr int kPlanTokensPerCta = 4096; // above this many rows of q the planner runs as a cluster

struct PlanArgs {
    PagedShape s;
    PagedLayout L;
    const int32_t *ctx, *n_new, *free_pages, *free_head;
    int32_t n_free;
    int32_t *table, *free_next, *seq, *cu, *pos;
    int64_t *slots;
    uint8_t *plan;
    int32_t *status;
};


// What the planner adds up over the requests.  Tokens and pages saturate: a sum that
// reaches the bound does not fit anyway.
constexpr uint32_t kSumMax = 1u << 30;
struct PlanSums {
    uint32_t tokens, pages;
    uint32_t entries;       // few-rows entries | many-rows entries << 16 (kMaxRequests fits)
    int64_t few_tiles, units;
    __device__ __forceinline__ void add(const PlanSums &o)
    {
        tokens = min(tokens + o.tokens, kSumMax);
        pages = min(pages + o.pages, kSumMax);
        entries += o.entries;
        few_tiles += o.few_tiles;
        units += o.units;
    }
    __device__ __forceinline__ PlanSums up(int o) const
    {
        return PlanSums{__shfl_up_sync(0xffffffffu, tokens, o), __shfl_up_sync(0xffffffffu, pages, o),
                        __shfl_up_sync(0xffffffffu, entries, o), __shfl_up_sync(0xffffffffu, few_tiles, o),
                        __shfl_up_sync(0xffffffffu, units, o)};
    }
};

// Sums before this thread's (every thread of the block calls), and of the block.
__device__ __forceinline__ void block_scan(const PlanSums &mine, PlanSums *before, PlanSums *total, PlanSums *sh)
{
    const int lane = lane_id(), warp = threadIdx.x >> 5;
    PlanSums x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const PlanSums y = x.up(o);
        if (lane >= o) x.add(y);
    }
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    PlanSums w = lane < kPlanWarps ? sh[lane] : PlanSums{};     // every warp scans the warps' sums
#pragma unroll
    for (int o = 1; o < kPlanWarps; o <<= 1) {
        const PlanSums y = w.up(o);
        if (lane >= o) w.add(y);
    }
    auto from = [&](const PlanSums &p, int l) {
        return PlanSums{__shfl_sync(0xffffffffu, p.tokens, l), __shfl_sync(0xffffffffu, p.pages, l), __shfl_sync(0xffffffffu, p.entries, l),
                        __shfl_sync(0xffffffffu, p.few_tiles, l), __shfl_sync(0xffffffffu, p.units, l)};
    };
    *total = from(w, kPlanWarps - 1);
    *before = from(w, max(warp - 1, 0));
    if (warp == 0) *before = PlanSums{};
    const PlanSums y = x.up(1);
    if (lane > 0) before->add(y);
    __syncthreads();
}

// Index of the last of n non-decreasing values that is <= x (a[0] = 0 <= x).
template <class T>
__device__ __forceinline__ int last_at_most(const T *a, int n, T x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Pieces per many-rows unit (called by a full warp): the number whose pieces are done
// first, at a cost of `tiles` plus about eight tiles each (the pipeline's start, the
// epilogue and the partial sums, measured): in one round when they fit on the
// CTAs, else in the mean share of a CTA and one piece more.  16 units of 240 tiles:
// 9 pieces 53 us, 19 pieces 62, 29 pieces 66; 264 units of up to 240 tiles: whole
// 363 us, halves 304.
__device__ __forceinline__ int split_of(int64_t units, int64_t tiles)
{
    if (units == 0 || units > kMaxSplitUnits) return 1;
    const float n = (float)tiles / (float)units, u = (float)units;
    const int most = (int)min((int64_t)kMaxPieces / units, tiles / units / 2);
    float best = INFINITY;
    int at = 1;
    for (int x = 1 + lane_id(); x <= max(most, 1); x += 32) {
        const float len = n / (float)x + 8.f, pieces = u * (float)x;
        const float t = pieces <= (float)kPagedCtas ? len : pieces * len / (float)kPagedCtas + len;
        if (t < best) {
            best = t;
            at = x;
        }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float t = __shfl_xor_sync(0xffffffffu, best, o);
        const int x = __shfl_xor_sync(0xffffffffu, at, o);
        if (t < best || (t == best && x < at)) {
            best = t;
            at = x;
        }
    }
    return at;
}

__global__ void __launch_bounds__(kPlanThreads, 1) paged_plan_kernel(const PlanArgs a)
{
    extern __shared__ __align__(16) uint8_t plan_smem[];
    __shared__ PlanSums sh[kPlanWarps];
    __shared__ unsigned long long sh_tiles;
    __shared__ int32_t s_key[kPlanThreads], s_units[kPlanThreads];
    __shared__ int32_t s_warp[kPlanWarps];
    const PagedShape &s = a.s;
    const int tid = threadIdx.x, ctas = gridDim.x, cta = blockIdx.x;
    int64_t *s_tiles = reinterpret_cast<int64_t *>(plan_smem);             // [R + 1] tiles before few-rows entry i
    int32_t *s_cu = reinterpret_cast<int32_t *>(s_tiles + s.R + 1);        // [R] tokens before request r
    int32_t *s_off = s_cu + s.R;                                           // [R] pages handed out before request r
    int32_t *s_ctx = s_off + s.R;                                          // [R] tokens cached
    uint8_t *s_rows = reinterpret_cast<uint8_t *>(s_ctx + s.R);            // [R] rows of few-rows entry i
    const int G = s.Hq / s.Hkv;
    const int64_t max_keys = (int64_t)s.max_pages * s.page_size;
    PagedEntry *few = reinterpret_cast<PagedEntry *>(a.plan + a.L.off_few);
    int64_t *few_cum = reinterpret_cast<int64_t *>(a.plan + a.L.off_few_cum);
    PagedEntry *many = reinterpret_cast<PagedEntry *>(a.plan + a.L.off_many);
    int32_t *many_cum = reinterpret_cast<int32_t *>(a.plan + a.L.off_many_cum);
    const int tpt = 128 / G;                 // tokens of a many-rows unit
    const int32_t head = a.free_pages ? *a.free_head : 0;

    PlanSums run{};
    int64_t many_tiles = 0;                  // of this thread's requests, about
    bool bad = false;
    if (tid == 0) sh_tiles = 0;
    for (int r0 = 0; r0 < s.R; r0 += kPlanThreads) {
        const int r = r0 + tid;
        int ctx = 0, n = 0;
        if (r < s.R) {
            ctx = a.ctx[r];
            n = a.n_new[r];
            if (ctx < 0 || n < 0 || n > s.max_q || (int64_t)ctx + n > max_keys) {
                bad = true;
                ctx = n = 0;
            }
        }
        const bool is_few = n > 0 && n * G <= kFewRows;       // n <= 2^24, G <= 32
        const bool is_many = n > 0 && !is_few;
        PlanSums v{};
        v.tokens = n;
        v.pages = (ctx + n + s.page_size - 1) / s.page_size - (ctx + s.page_size - 1) / s.page_size;
        v.entries = (is_few ? 1u : 0u) | (is_many ? 1u << 16 : 0u);
        if (is_few) v.few_tiles = (int64_t)key_range(ctx, ctx + n - 1, s.window, s.sink).n * s.Hkv;
        if (is_many) {
            v.units = (int64_t)((n + tpt - 1) / tpt) * s.Hkv;
            // The units' mean length lies between the first one's and the last one's.
            many_tiles += v.units * (key_range(ctx, ctx + min(n, tpt) - 1, s.window, s.sink).n +
                                     key_range(ctx + (n - 1) / tpt * tpt, ctx + n - 1, s.window, s.sink).n) / 2;
        }
        PlanSums before, total;
        block_scan(v, &before, &total, sh);
        before.add(run);
        if (r < s.R) {
            s_cu[r] = (int32_t)before.tokens;
            s_off[r] = (int32_t)before.pages;
            s_ctx[r] = ctx;
            if (is_few) {
                const int e = (int)(before.entries & 0xffffu);
                s_tiles[e] = before.few_tiles;
                s_rows[e] = (uint8_t)(n * G);
                if (cta == 0) {
                    few[e] = PagedEntry{r, (int32_t)before.tokens, n, ctx};
                    few_cum[e] = before.few_tiles;
                }
            }
            if (is_many && cta == 0) {
                const int e = (int)(before.entries >> 16);
                many[e] = PagedEntry{r, (int32_t)before.tokens, n, ctx};
                many_cum[e] = (int32_t)before.units;
            }
        }
        run.add(total);
    }
    if (cta == 0 && many_tiles > 0) atomicAdd(&sh_tiles, (unsigned long long)many_tiles);
    // Every CTA comes to the same verdict.  A plan that fails hands out nothing
    // and is empty: no slot, no row of attention.  (Tiles of the few-rows list are counted in
    // 31 bits from here on; units fit them: at least 104 rows each of 2^36, and one
    // per request and KV head.)
    int32_t err = FM_OK;
    if (__syncthreads_or(bad) || run.tokens > (uint32_t)s.T || run.few_tiles > INT32_MAX) err = FM_ERR_LENGTHS;
    else if (a.free_pages && (head < 0 || head > a.n_free || run.pages > (uint32_t)(a.n_free - head))) err = FM_ERR_PAGES;
    if (err != FM_OK && cta == 0 && tid == 0) set_status(a.status, err);
    const int total = err == FM_OK ? (int)run.tokens : 0;
    const int handed = err == FM_OK && a.free_pages ? (int)run.pages : 0;
    const int n_few = err == FM_OK ? (int)(run.entries & 0xffffu) : 0;
    const int64_t W = err == FM_OK ? run.few_tiles : 0;

    // Slots and positions, four tokens of a thread at a time: the pages' loads are
    // in flight together.
    const int stride = ctas * kPlanThreads;
    for (int t0 = cta * kPlanThreads + tid; t0 < s.T; t0 += 4 * stride) {
        int p[4], in[4], page[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + i * stride;
            p[i] = page[i] = -1;
            in[i] = 0;
            if (t < total) {
                const int r = last_at_most(s_cu, s.R, t), ctx = s_ctx[r];
                p[i] = ctx + t - s_cu[r];
                const int b = p[i] / s.page_size, have = (ctx + s.page_size - 1) / s.page_size;
                in[i] = p[i] - b * s.page_size;
                // Page b of the request, as the step leaves the table.
                page[i] = (a.free_pages && b >= have) ? a.free_pages[head + s_off[r] + b - have] : a.table[(int64_t)r * s.max_pages + b];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + i * stride;
            if (t >= s.T) break;
            int64_t slot = -1;
            if (t < total) {
                if (page[i] >= 0 && page[i] < s.num_pages) slot = (int64_t)page[i] * s.page_size + in[i];
                else set_status(a.status, FM_ERR_PAGES);
            }
            a.slots[t] = slot;
            if (a.pos) a.pos[t] = p[i];
        }
    }
    for (int x = cta * kPlanThreads + tid; x < handed; x += stride) {
        const int r = last_at_most(s_off, s.R, x);
        const int have = (s_ctx[r] + s.page_size - 1) / s.page_size;
        a.table[(int64_t)r * s.max_pages + have + x - s_off[r]] = a.free_pages[head + x];
    }
    if (cta == 0) {
        // Many-rows entries, the longest keys first (up to a block of them; beyond that
        // there are units enough to fill the gaps): the CTAs claim in this order.
        const int n_many = err == FM_OK ? (int)(run.entries >> 16) : 0;
        if (n_many > 1 && n_many <= kPlanThreads) {
            __syncthreads();
            PagedEntry en{};
            if (tid < n_many) en = many[tid];
            s_key[tid] = tid < n_many ? en.ctx + en.n : 0;
            __syncthreads();
            int rank = 0;
            if (tid < n_many) {
                for (int i = 0; i < n_many; ++i) rank += s_key[i] > s_key[tid] || (s_key[i] == s_key[tid] && i < tid) ? 1 : 0;
                s_units[rank] = (en.n + tpt - 1) / tpt * s.Hkv;
                many[rank] = en;
            }
            __syncthreads();
            const int u = tid < n_many ? s_units[tid] : 0;      // the sum fits 31 bits (checked above)
            int x = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane_id() >= o) x += y;
            }
            if (lane_id() == 31) s_warp[tid >> 5] = x;
            __syncthreads();
            for (int w = 0; w < tid >> 5; ++w) x += s_warp[w];
            if (tid < n_many) many_cum[tid] = x - u;
        }
        // (A CTA per tile at least: two or four tiles each were slower, 7.7 and 7.6 for 7.2 us
        // with two short requests, 6.7 and 10.3 for 4.9 with one.)
        const int ctas_few = (int)(W < kPagedCtas ? W : kPagedCtas);
        const int splits = tid < 32 ? split_of(run.units, (int64_t)sh_tiles) : 1;
        if (tid == 0) {
            PagedHeader h{};
            h.magic = kPagedMagic;
            h.s = s;
            h.n_few = n_few;
            h.ctas_few = ctas_few;
            h.tiles_few = W;
            h.rows = total;
            h.n_many = n_many;
            h.units_many = err == FM_OK ? (int)run.units : 0;
            h.splits_many = h.units_many > 0 ? splits : 1;
            *reinterpret_cast<PagedHeader *>(a.plan) = h;
            few_cum[n_few] = W;
            if (h.n_many > 0) many_cum[h.n_many] = h.units_many;
            *reinterpret_cast<uint32_t *>(a.plan + a.L.off_claim) = 0u;
            a.cu[s.R] = total;
        }
        for (int r = tid; r < s.R; r += kPlanThreads) a.cu[r] = err == FM_OK ? s_cu[r] : 0;
        for (int i = tid; i < kPagedCtas; i += kPlanThreads) {
            PagedStart st{};
            if (i < ctas_few) {
                const int64_t x = share_begin(W, ctas_few, i);
                const int e = last_at_most(s_tiles, n_few, x);
                const int64_t next = e + 1 < n_few ? s_tiles[e + 1] : W;
                const int n = (int)((next - s_tiles[e]) / s.Hkv), y = (int)(x - s_tiles[e]);
                st.e = e;
                st.h = y / n;
                st.x = y % n;
                st.count = (int)(share_begin(W, ctas_few, i + 1) - x);
                st.ent = few[e];        // written by this CTA, before the barrier above
                st.cum = s_tiles[e];
                for (int y = e; y < n_few && s_tiles[y] < x + st.count; ++y) st.rows = max(st.rows, (int)s_rows[y]);
            }
            reinterpret_cast<PagedStart *>(a.plan + a.L.off_start)[i] = st;
            reinterpret_cast<uint32_t *>(a.plan + a.L.off_count)[i] = 0u;
        }
    }
    // Every CTA has read the lengths and the head: they may be advanced in place.
    if (ctas > 1) cg::this_cluster().sync();
    else __syncthreads();
    if (cta == 0) {
        for (int r = tid; r < s.R; r += kPlanThreads) {
            const int ctx = a.ctx[r];
            a.seq[r] = err == FM_OK ? ctx + a.n_new[r] : ctx;
        }
        if (tid == 0 && a.free_next) *a.free_next = head + handed;
    }
}

// ---- append -----------------------------------------------------------------------
// cache[slot] = x, one piece of 16 bytes of the cache of K and of V per thread: bound by
// the bytes (10,111 tokens of 8 heads: bf16 9.4 us on what L2 holds, 16.4 a call on what it does not;
// 11,112 to e4m3 13.3 and 18.4; two or four pieces in flight per thread were slower, bf16 9.1 to 10.4 and,
// then with plain divisions, e4m3 15.1 to 16.7 for 14.4).
// e4m3: code = e4m3(x / descale), the quotient in fp32, nearest even, saturating:
// the quantizer's rule.
constexpr int kAppendThreads = 256;

struct AppendArgs {
    const uint8_t *k, *v;                        // bf16; strides in bytes
    int64_t k_tok, k_head, v_tok, v_head;
    uint8_t *kc, *vc;
    int64_t kc_page, kc_head, kc_tok, vc_page, vc_head, vc_tok;
    const int64_t *slots;
    const float *k_descale, *v_descale;
    int64_t n_slots;                             // num_pages * page_size
    int32_t page_size, T, block_tokens;
    int32_t per_tok, per_row;                    // pieces of a token, of a row
    uint64_t tok_magic, row_magic;               // 2^40 / per_tok and / per_row, rounded up
    int32_t *status;
};

// Correctly rounded quotients by one divisor, from its correctly rounded
// reciprocal and one correction (Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990: q = x r, q + (x - q d) r): three instructions
// each.  A divisor outside [2^-80, 2^80], where the remainder could underflow,
// divides.
struct Divisor {
    float d, r;
    bool plain;
    __device__ __forceinline__ explicit Divisor(float x) : d(x), r(1.f / x), plain(!(x >= 8.271806e-25f && x <= 1.2089258e24f)) {}
    __device__ __forceinline__ float operator()(float x) const
    {
        if (plain) return x / d;
        const float q = x * r, c = fmaf(fmaf(-q, d, x), r, q);
        return fabsf(q) == INFINITY ? q : copysignf(c, q);      // (the correction loses the sign of a zero)
    }
};
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w, const Divisor &ds)
{
    return pack_e4m3x2(ds(__uint_as_float(w << 16)), ds(__uint_as_float(w & 0xffff0000u)));
}
__device__ __forceinline__ uint4 e4m3_piece(const uint4 &x, const uint4 &y, const Divisor &ds)
{
    return make_uint4(e4m3_pair(x.x, ds) | e4m3_pair(x.y, ds) << 16, e4m3_pair(x.z, ds) | e4m3_pair(x.w, ds) << 16,
                      e4m3_pair(y.x, ds) | e4m3_pair(y.y, ds) << 16, e4m3_pair(y.z, ds) | e4m3_pair(y.w, ds) << 16);
}

template <bool FP8>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const AppendArgs a)
{
    constexpr int IN = FP8 ? 2 : 1;              // 16-byte loads of a piece
    const int t0 = blockIdx.x * a.block_tokens;
    const int pieces = min(a.block_tokens, a.T - t0) * a.per_tok;
    const Divisor kd(FP8 ? *a.k_descale : 1.f), vd(FP8 ? *a.v_descale : 1.f);
    for (int j = threadIdx.x; j < pieces; j += kAppendThreads) {      // once, unless a token has more pieces than that
        const int t = (int)(((uint64_t)j * a.tok_magic) >> 40), in = j - t * a.per_tok;
        const int h = (int)(((uint64_t)in * a.row_magic) >> 40), ch = in - h * a.per_row;
        const int64_t slot = a.slots[t0 + t];
        if (slot < 0) continue;
        if (slot >= a.n_slots) {
            set_status(a.status, FM_ERR_PAGES);
            continue;
        }
        const uint4 *kp = reinterpret_cast<const uint4 *>(a.k + (int64_t)(t0 + t) * a.k_tok + (int64_t)h * a.k_head + ch * (16 * IN));
        const uint4 *vp = reinterpret_cast<const uint4 *>(a.v + (int64_t)(t0 + t) * a.v_tok + (int64_t)h * a.v_head + ch * (16 * IN));
        const uint4 k0 = __ldg(kp), v0 = __ldg(vp);
        const uint4 k1 = FP8 ? __ldg(kp + 1) : k0, v1 = FP8 ? __ldg(vp + 1) : v0;
        const int64_t page = slot <= INT32_MAX ? (int64_t)((uint32_t)slot / (uint32_t)a.page_size) : slot / a.page_size;
        const int64_t at = slot - page * a.page_size;
        *reinterpret_cast<uint4 *>(a.kc + page * a.kc_page + h * a.kc_head + at * a.kc_tok + ch * 16) = FP8 ? e4m3_piece(k0, k1, kd) : k0;
        *reinterpret_cast<uint4 *>(a.vc + page * a.vc_page + h * a.vc_head + at * a.vc_tok + ch * 16) = FP8 ? e4m3_piece(v0, v1, vd) : v0;
    }
}

}  // namespace fm

using namespace fm;

namespace {

bool aligned16(const void *p) { return p && ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void *p) { return p && ((uintptr_t)p & 3u) == 0; }

// Sizes of a step; *out gets them in the library's own form.
fm_status check_step(const fm_paged_step *p, PagedShape *out)
{
    if (!p) return FM_ERR_INVALID_ARG;
    if (p->requests <= 0 || p->max_tokens <= 0 || p->max_q <= 0 || p->max_pages <= 0 || p->num_pages <= 0 || p->page_size <= 0 ||
        p->Hq <= 0 || p->Hkv <= 0 || p->window < 0 || p->sink < 0)
        return FM_ERR_INVALID_ARG;
    if (p->max_q > p->max_tokens || p->Hq % p->Hkv != 0) return FM_ERR_INVALID_ARG;
    if (p->d != 64 && p->d != 128) return FM_ERR_UNSUPPORTED;
    if (p->requests > kMaxRequests || p->max_tokens > (1 << 24) || p->page_size % kPageGranule != 0 || p->page_size > kMaxPage ||
        p->Hq > 4096 || p->Hq / p->Hkv > kFewRows)
        return FM_ERR_UNSUPPORTED;
    // Positions are int32, and so are a page's and a tile's last key behind them.
    if ((int64_t)p->max_pages * p->page_size > (int64_t)0x7fffffff - 2 * kMaxPage) return FM_ERR_UNSUPPORTED;
    if (p->window > (1 << 30) || p->sink > (1 << 30)) return FM_ERR_UNSUPPORTED;
    *out = PagedShape{p->requests, p->max_tokens, p->max_q, p->max_pages, p->num_pages, p->page_size, p->Hq, p->Hkv, p->d,
                      p->window, p->window > 0 ? p->sink : 0};     // (no window: every key is attended anyway)
    return FM_OK;
}

// Pages, strides and descales of a cache; alignment of 16 bytes everywhere.
fm_status check_cache(const fm_paged_cache *c)
{
    if (!c || !aligned16(c->k) || !aligned16(c->v)) return FM_ERR_INVALID_ARG;
    if (c->num_pages <= 0 || c->page_size <= 0 || c->Hkv <= 0) return FM_ERR_INVALID_ARG;
    if (c->Hkv > 4096) return FM_ERR_UNSUPPORTED;
    if (c->dtype != FM_DT_BF16 && c->dtype != FM_DT_E4M3) return FM_ERR_INVALID_ARG;
    if (c->d != 64 && c->d != 128) return FM_ERR_UNSUPPORTED;
    if (c->page_size % kPageGranule != 0 || c->page_size > kMaxPage) return FM_ERR_UNSUPPORTED;
    const int esz = c->dtype == FM_DT_E4M3 ? 1 : 2;
    const int64_t st[6] = {c->k_page, c->k_head, c->k_tok, c->v_page, c->v_head, c->v_tok};
    for (int64_t x : st)
        if (x <= 0 || (x * esz) % 16 != 0 || x > ((int64_t)1 << 38)) return FM_ERR_INVALID_ARG;
    if (c->k_tok < c->d || c->v_tok < c->d) return FM_ERR_INVALID_ARG;
    if (esz == 1 && (!aligned4(c->k_descale) || !aligned4(c->v_descale))) return FM_ERR_INVALID_ARG;
    return FM_OK;
}

// Rows of bf16 read 16 bytes at a time: token and head strides in elements.
bool rows_ok(const void *p, int64_t tok, int64_t head)
{
    return aligned16(p) && tok > 0 && head > 0 && tok % 8 == 0 && head % 8 == 0 && tok <= ((int64_t)1 << 38) &&
           head <= ((int64_t)1 << 38);
}

fm_status device_ok()
{
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return FM_ERR_CUDA;
    static std::atomic<int8_t> known[kMaxDevices];
    if (dev >= kMaxDevices) return FM_ERR_UNSUPPORTED;
    int8_t k = known[dev].load(std::memory_order_acquire);
    if (k == 0) {
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return FM_ERR_CUDA;
        k = (major == 10 && minor == 3) ? 1 : 2;
        if (k == 1 && cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           kMaxRequests * 21 + 16) != cudaSuccess)
            return FM_ERR_CUDA;
        known[dev].store(k, std::memory_order_release);
    }
    return k == 1 ? FM_OK : FM_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

size_t fm_paged_plan_bytes(const fm_paged_step *step)
{
    PagedShape s;
    return check_step(step, &s) == FM_OK ? (size_t)paged_layout(s).total : 0;
}

fm_status fm_paged_plan(const fm_paged_step *step, const int32_t *ctx_lens, const int32_t *q_lens, int32_t *block_table,
                        const int32_t *free_pages, int n_free, const int32_t *free_head, int32_t *free_next,
                        int32_t *seq_lens, int32_t *cu_q, int64_t *slots, int32_t *positions, void *plan, size_t plan_bytes,
                        int32_t *dev_status, fm_stream_t stream)
{
    PlanArgs a{};
    const fm_status st = check_step(step, &a.s);
    if (st != FM_OK) return st;
    if (!aligned4(ctx_lens) || !aligned4(q_lens) || !aligned4(block_table) || !aligned4(seq_lens) || !aligned4(cu_q) ||
        !slots || ((uintptr_t)slots & 7u) || ((uintptr_t)positions & 3u) || !aligned4(dev_status))
        return FM_ERR_INVALID_ARG;
    if (free_pages && (((uintptr_t)free_pages & 3u) || n_free < 0 || !aligned4(free_head) || !aligned4(free_next)))
        return FM_ERR_INVALID_ARG;
    a.L = paged_layout(a.s);
    if (!plan || ((uintptr_t)plan & 255u) || plan_bytes < (size_t)a.L.total) return FM_ERR_WORKSPACE;
    const fm_status dv = device_ok();
    if (dv != FM_OK) return dv;
    a.ctx = ctx_lens;
    a.n_new = q_lens;
    a.table = block_table;
    a.free_pages = free_pages;
    a.n_free = n_free;
    a.free_head = free_head;
    a.free_next = free_pages ? free_next : nullptr;
    a.seq = seq_lens;
    a.cu = cu_q;
    a.slots = slots;
    a.pos = positions;
    a.plan = (uint8_t *)plan;
    a.status = dev_status;
    const int ctas = a.s.T > kPlanTokensPerCta ? kPlanCluster : 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = (size_t)a.s.R * 21 + 16;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    ProfScope ps(kKPagedPlan, stream);
    return cudaLaunchKernelEx(&cfg, paged_plan_kernel, a) == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

fm_status fm_paged_append(const void *k, int64_t k_tok, int64_t k_head, const void *v, int64_t v_tok, int64_t v_head,
                          const int64_t *slots, int T, const fm_paged_cache *cache, int32_t *dev_status, fm_stream_t stream)
{
    const fm_status st = check_cache(cache);
    if (st != FM_OK) return st;
    if (T < 0 || T > (1 << 24) || !rows_ok(k, k_tok, k_head) || !rows_ok(v, v_tok, v_head) || !slots ||
        ((uintptr_t)slots & 7u) || !aligned4(dev_status))
        return FM_ERR_INVALID_ARG;
    const fm_status dv = device_ok();
    if (dv != FM_OK) return dv;
    if (T == 0) return FM_OK;
    const bool fp8 = cache->dtype == FM_DT_E4M3;
    const int64_t esz = fp8 ? 1 : 2;
    AppendArgs a{};
    a.k = (const uint8_t *)k;
    a.v = (const uint8_t *)v;
    a.k_tok = k_tok * 2;
    a.k_head = k_head * 2;
    a.v_tok = v_tok * 2;
    a.v_head = v_head * 2;
    a.kc = (uint8_t *)cache->k;
    a.vc = (uint8_t *)cache->v;
    a.kc_page = cache->k_page * esz;
    a.kc_head = cache->k_head * esz;
    a.kc_tok = cache->k_tok * esz;
    a.vc_page = cache->v_page * esz;
    a.vc_head = cache->v_head * esz;
    a.vc_tok = cache->v_tok * esz;
    a.slots = slots;
    a.k_descale = cache->k_descale;
    a.v_descale = cache->v_descale;
    a.n_slots = (int64_t)cache->num_pages * cache->page_size;
    a.page_size = cache->page_size;
    a.T = T;
    a.per_row = (int)(cache->d * esz / 16);
    a.per_tok = cache->Hkv * a.per_row;
    a.block_tokens = a.per_tok < kAppendThreads ? kAppendThreads / a.per_tok : 1;
    a.tok_magic = ((uint64_t)1 << 40) / a.per_tok + 1;
    a.row_magic = ((uint64_t)1 << 40) / a.per_row + 1;
    a.status = dev_status;
    const int blocks = (T + a.block_tokens - 1) / a.block_tokens;
    ProfScope ps(kKPagedAppend, stream);
    if (fp8) paged_append_kernel<true><<<blocks, kAppendThreads, 0, (cudaStream_t)stream>>>(a);
    else paged_append_kernel<false><<<blocks, kAppendThreads, 0, (cudaStream_t)stream>>>(a);
    return cudaPeekAtLastError() == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

fm_status fm_attn_paged(const fm_paged_step *step, const void *q, int64_t q_tok, int64_t q_head, int rows,
                        const fm_paged_cache *cache, const int32_t *block_table, void *plan, size_t plan_bytes, float scale, void *o, int o_dtype,
                        float *lse, int32_t *dev_status, fm_stream_t stream)
{
    PagedArgs a{};
    fm_status st = check_step(step, &a.s);
    if (st != FM_OK) return st;
    if ((st = check_cache(cache)) != FM_OK) return st;
    if (cache->num_pages != a.s.num_pages || cache->page_size != a.s.page_size || cache->Hkv != a.s.Hkv || cache->d != a.s.d)
        return FM_ERR_INVALID_ARG;
    if (rows < 0 || !rows_ok(q, q_tok, q_head) || !aligned16(o) || !aligned4(lse) || !aligned4(block_table) || !aligned4(dev_status))
        return FM_ERR_INVALID_ARG;
    if (o_dtype != FM_DT_BF16 && o_dtype != FM_DT_F32) return FM_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return FM_ERR_INVALID_ARG;
    a.L = paged_layout(a.s);
    if (!plan || ((uintptr_t)plan & 255u) || plan_bytes < (size_t)a.L.total) return FM_ERR_WORKSPACE;
    if ((st = device_ok()) != FM_OK) return st;
    const bool fp8 = cache->dtype == FM_DT_E4M3;
    const int64_t esz = fp8 ? 1 : 2;
    a.plan = (uint8_t *)plan;
    a.table = block_table;
    a.q = (const uint8_t *)q;
    a.q_tok = q_tok * 2;
    a.q_head = q_head * 2;
    a.k_descale = cache->k_descale;
    a.v_descale = cache->v_descale;
    a.o = o;
    a.lse = lse;
    a.status = dev_status;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.o_f32 = o_dtype == FM_DT_F32;
    a.rows = rows;
    a.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (a.s.page_size == 1 << i) a.page_shift = i;
    const int G = a.s.Hq / a.s.Hkv;
    const uint64_t d = a.s.d, kt = cache->k_tok * esz, kh = cache->k_head * esz, kp = cache->k_page * esz, vt = cache->v_tok * esz,
                   vh = cache->v_head * esz, vp = cache->v_page * esz;
    const uint64_t pages = a.s.num_pages, page = a.s.page_size, heads = a.s.Hkv;
    // Boxes of consecutive keys of one page, a power of two of them.
    int box_keys = kPageGranule;
    while (box_keys < kKeyTile && a.s.page_size % (2 * box_keys) == 0) box_keys *= 2;
    if ((int64_t)a.s.max_q * G > kFewRows) {
        // Some request may have many rows.  Q boxes: the query heads of a KV head times
        // as many tokens as make 128 rows.
        CUtensorMap tq, tk, tv;
        const uint64_t qd[3] = {d, (uint64_t)a.s.Hq, (uint64_t)(rows > 0 ? rows : 1)};
        const uint64_t qs[2] = {(uint64_t)a.q_head, (uint64_t)a.q_tok};
        const uint32_t qb[3] = {64, (uint32_t)G, (uint32_t)(128 / G)};
        const uint64_t cd[4] = {d, page, heads, pages};
        const uint64_t ks[3] = {kt, kh, kp}, vs[3] = {vt, vh, vp};
        const uint32_t cb[4] = {fp8 ? (uint32_t)a.s.d : 64u, (uint32_t)box_keys, 1, 1};
        if (!make_tmap_strided(&tq, q, false, 3, qd, qs, qb, 128) || !make_tmap_strided(&tk, cache->k, fp8, 4, cd, ks, cb, fp8 ? a.s.d : 128) ||
            !make_tmap_strided(&tv, cache->v, fp8, 4, cd, vs, cb, fp8 ? 0 : 128))
            return FM_ERR_CUDA;
        wait_test_args(kKPagedChunk, &a.wait_limit, &a.withhold);
        if ((st = fm_paged_chunk_launch(tq, tk, tv, a, box_keys, fp8, (cudaStream_t)stream)) != FM_OK) return st;
    }
    // Rows of 128 bytes (bf16, d = 128: two of them, as a
    // dimension of its own) or of 64 bytes (e4m3, d = 64).
    const uint64_t wide = fp8 ? d : 64;
    const uint32_t halves = (uint32_t)(d / wide);
    CUtensorMap tk, tv;
    const uint64_t cd[5] = {wide, page, halves, heads, pages};
    const uint64_t ks[4] = {kt, 128, kh, kp}, vs[4] = {vt, 128, vh, vp};
    const uint32_t cb[5] = {(uint32_t)wide, (uint32_t)box_keys, halves, 1, 1};
    const int swizzle = (int)(wide * esz);
    if (!make_tmap_strided(&tk, cache->k, fp8, 5, cd, ks, cb, swizzle) || !make_tmap_strided(&tv, cache->v, fp8, 5, cd, vs, cb, swizzle))
        return FM_ERR_CUDA;
    wait_test_args(kKPagedDecode, &a.wait_limit, &a.withhold);
    return fm_paged_decode_launch(tk, tv, a, box_keys, fp8, (cudaStream_t)stream);
}

}  // extern "C"
