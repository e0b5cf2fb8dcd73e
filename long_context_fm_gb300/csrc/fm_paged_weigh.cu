// Attention weight that the cached keys of a step's requests receive:
//
//   weights[key] (+)= sum over rows and query heads that attend the key of exp2(scale log2(e) q.k - log2(e) lse)
//
// The scores are computed with the keys as the rows of the product: S = K Q^T, so that a TMEM lane, and with it a thread,
// holds one key and all its columns are summed in the thread: no exchange, no atomics among threads, one fixed
// order.  Two kernels, as the attention has: requests of at most kFewRows rows (new tokens x query heads per KV
// head), where K is read once and little is computed, and those with more, which are matrix work.
//
// Few rows: bound by HBM (K once): 96 requests of one token over up to 16,000 keys, 32 / 8 heads, 159 us (6.4 TB/s), 64 of up
// to three over e4m3 73 us (5.3 TB/s).  Key tiles (128 keys) of all (request, KV head) units lie end to end and are cut into
// equal shares, as the plan has them for the attention.  Rows are 16 or 32 columns of the product.  A tile of codes takes
// as little as 700 cycles of HBM, so each step that one thread or warp does for every tile (loads, products, sums) is done by
// two on alternate tiles: with one of each the e4m3 batch took 92 us, with the products and sums alone doubled 91.
//   warps 0, 11 walk the share, look pages up (a batch of tiles at a time), TMA of K, alternate tiles (ring of 128 to 192 KB)
//   warps 1, 10 one thread each issues K Q^T of every second tile (1: TMEM)
//   warps 2-5   even tiles, thread = key: exponentials, sum, one add or store to the key's weight;  warps 6-9  odd ones
//   warps 12-15 Q and lse of the next units to shared memory (e4m3 caches: Q as two e4m3 terms, so that K is used as it is)
//
// Many rows: a unit is two key tiles of a (request, KV head), whose K stays in shared memory while the row tiles (128
// rows: the query heads of the KV head times as many tokens as fit) that attend them stream through, each multiplied by
// both.  Per pair of tiles 512 cycles of products (128 x 128 x 128) beside 512 of exponentials (32 a cycle and SM): both
// about even, and each key tile has its own issuing thread, two score buffers and a warpgroup for each of them.  4,178 tokens
// over up to 16K keys: 316 to 336 us (1,410 to 1,500 TFLOP/s, by the clock that the power leaves); while an SM has work the tensor pipe
// and the exponentials are busy 70 % of the time each (a warp's waits and loads from TMEM are what is between).
// One key tile a unit, one issuing thread and two warpgroups took 455 us (a row tile's products waited for their own
// barriers), two issuing threads 457 (Q's arrival), two key tiles a unit 439 (the sums' latency), four warpgroups 350, units cut
// along the rows 327, the next scores on their way while some are summed and the masked case apart 318.  Not
// kept: four issuing threads (375), K as the TMEM operand with three score buffers (375: the buffers come free too late), two
// warpgroups that hold all 128 scores of a row tile (380).
//   warp 0      claims units (longest first), TMA of K
//   warps 1, 19 one thread each issues K Q^T of one of the key tiles (1: TMEM)
//   warps 2-5, 6-9    first key tile, even and odd row tiles, thread = key;  warps 10-13, 14-17  second one
//   warp 18     TMA of Q, lse of the row tiles
//   warps 20-23 e4m3 caches only: K to bf16, exactly, once per unit
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <type_traits>

#include "fm_paged.h"
#include "fm_ptx.cuh"

namespace fm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct WeighArgs {
    PagedArgs p;
    float *weights;                 // [num_pages, Hkv, page_size]
    const float *lse;               // [rows, Hq]
    int box_keys;
};

// Place of key j of request r in the pool of weights (head 0), or -1 where no page of the pool holds it.
__device__ __forceinline__ int64_t weight_place(const PagedArgs &a, int r, int j)
{
    const PagedShape &s = a.s;
    const int b = a.page_shift >= 0 ? j >> a.page_shift : j / s.page_size, in = j - b * s.page_size;
    const int page = __ldg(a.table + (int64_t)r * s.max_pages + b);
    return (unsigned)page < (unsigned)s.num_pages ? (int64_t)page * s.Hkv * s.page_size + in : -1;
}

// A key's sum to its weight: added, or the first one of a key that this step brought.
__device__ __forceinline__ void put(float *at, float sum, bool fresh)
{
    if (fresh) *at = sum;
    else red_add_f32(at, sum);
}

// ---- pieces of the many rows ------------------------------------------------------------
// A unit (two key tiles of a request's KV head) whose row tiles are many is cut into pieces along them, so that the CTAs
// end together: pieces of about an eighth of a CTA's share, four row tiles at least.  Their sums go to the plan's workspace and
// the kernel of the few rows, which follows, adds them up in their order.  (504 units of up to 128 row tiles: whole
// 350 us, in thirds 327; one KV head of 2,000 tokens over 4,000 keys, 16 units, 115 and 29.)
struct ManyPieces {
    int len;                // row tiles of a piece
    int tpt;                // tokens of a row tile
    int64_t units, pieces;  // of all entries
    __device__ __forceinline__ int64_t units_of(const PagedShape &s, const PagedEntry &en) const
    {
        return (int64_t)((key_range(en.ctx, en.ctx + en.n - 1, s.window, s.sink).n + 1) / 2) * s.Hkv;
    }
    __device__ __forceinline__ int tiles_of(const PagedEntry &en) const { return (en.n + tpt - 1) / tpt; }
    __device__ __forceinline__ int parts_of(const PagedEntry &en) const { return (tiles_of(en) + len - 1) / len; }
};

// Room for the pieces' sums behind that of the exchange within a CTA (floats of the workspace).
constexpr int64_t kExchange = (int64_t)kPagedCtas * 4 * 128;

// Called by a full warp; the same in every CTA.
__device__ __forceinline__ ManyPieces many_pieces(const PagedArgs &a, const PagedHeader *hd, int tpt)
{
    const PagedEntry *list = reinterpret_cast<const PagedEntry *>(a.plan + a.L.off_many);
    const PagedShape &s = a.s;
    auto sum = [](int64_t x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x;
    };
    const int n = hd->n_many, lane = lane_id();
    ManyPieces m{1, tpt, 0, 0};
    // The lane's first entry is all that it has, most often: once read.
    const PagedEntry first = list[min(lane, n - 1)];
    const int64_t u0 = lane < n ? m.units_of(s, first) : 0;
    const int t0 = m.tiles_of(first);
    int64_t tiles = u0 * t0;
    m.units = u0;
    for (int i = lane + 32; i < n; i += 32) {
        const int64_t u = m.units_of(s, list[i]);
        m.units += u;
        tiles += u * m.tiles_of(list[i]);
    }
    tiles = sum(tiles);
    m.units = sum(m.units);
    m.len = (int)min(max(tiles / (8 * kPagedCtas), (int64_t)4), (int64_t)1 << 24);
    if (!__any_sync(0xffffffffu, lane < n && t0 > m.len) && n <= 32) {
        m.pieces = m.units;                         // nothing to cut
        return m;
    }
    for (int go = 0; go < 2; ++go) {
        m.pieces = u0 * ((t0 + m.len - 1) / m.len);
        for (int i = lane + 32; i < n; i += 32) m.pieces += m.units_of(s, list[i]) * m.parts_of(list[i]);
        m.pieces = sum(m.pieces);
        if ((m.pieces + 1) * 256 + kExchange <= (int64_t)kMaxPieces * 128 * s.d) break;
        m.len = 1 << 24;                            // no room: whole units
    }
    return m;
}

// ---- few rows ------------------------------------------------------------------------

template <int D, bool FP8>
struct FewCfg {
    static constexpr int kThreads = 512;
    static constexpr int kTile = 128 * D * (FP8 ? 1 : 2);
    static constexpr int kSt = kTile == 32768 ? 6 : kTile == 16384 ? 8 : 16;    // 192 or 128 KB in flight
    static constexpr int kSBuf = 4, kQSlots = 3, kRing = 8;
    // Who takes every second tile meets a stage in every phase or in none: with an odd number it would see a phase that another
    // one was to wait for, and take the parity of the one before it for its own.
    static_assert(kSt % 2 == 0 && kSBuf % 2 == 0, "stages that alternate");
    static constexpr int kQBox = kFewRows * 128;                  // 32 rows of 128 bytes
    static constexpr int kQTerm = kFewRows * D;                   // e4m3: from the first term to the second
    static constexpr int kQBytes = kFewRows * D * 2;
    static constexpr int kQ = kSt * kTile;
    static constexpr int kCol = kQ + kQSlots * kQBytes;           // float [kQSlots][2][32]: score factor and -log2(e) lse of the rows
    static constexpr int kUnit = kCol + kQSlots * 2 * kFewRows * 4;   // int [kRing][8]
    static constexpr int kBar = kUnit + kRing * 8 * 4;
    enum { B_KF = 0, B_KE = B_KF + kSt, B_SF = B_KE + kSt, B_SE = B_SF + kSBuf, B_QF = B_SE + kSBuf, B_QE = B_QF + kQSlots,
           B_UF = B_QE + kQSlots, B_UE = B_UF + kRing, B_DRAIN = B_UE + kRing, B_COUNT };
    static constexpr int kMisc = kBar + B_COUNT * 8;
    static constexpr int kBytes = kMisc + 64;
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

// A stretch of a (request, KV head)'s tiles.
struct FewUnit {
    int n;                  // tiles; -1: no more
    int r, h, tok0, ntok, ctx;
    int x0;                 // its first tile in the request's range
};

template <int D, bool FP8>
__global__ void __launch_bounds__(FewCfg<D, FP8>::kThreads, 1)
    fm_paged_weigh_few_kernel(const __grid_constant__ CUtensorMap tk, const WeighArgs w)
{
    using C = FewCfg<D, FP8>;
    constexpr int NBOX = FP8 ? 1 : D / 64;
    extern __shared__ __align__(1024) uint8_t smem[];
    float *sCol = reinterpret_cast<float *>(smem + C::kCol);
    volatile int *sUnit = reinterpret_cast<volatile int *>(smem + C::kUnit);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBar);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::kMisc);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + C::kMisc + 4);
    const PagedArgs &a = w.p;
    const PagedShape &s = a.s;
    const PagedHeader *hd = reinterpret_cast<const PagedHeader *>(a.plan);
    const int warp = warp_id(), lane = lane_id();
    if (!paged_plan_fits(hd, s) || hd->rows > a.rows || (smem_u32(smem) & 1023u) != 0) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            set_status(a.status, !paged_plan_fits(hd, s) ? FM_ERR_PLAN_MISMATCH : hd->rows > a.rows ? FM_ERR_LENGTHS : FM_ERR_UNSUPPORTED);
        return;
    }
    if (hd->n_many > 0 && hd->weigh_len > 0) {
        // The pieces of the many rows' units, whose kernel is over: a thread per key.
        const ManyPieces mp{hd->weigh_len, 128 / (s.Hq / s.Hkv), 0, 0};
        const PagedEntry *list = reinterpret_cast<const PagedEntry *>(a.plan + a.L.off_many);
        const float *ws = reinterpret_cast<const float *>(a.plan + a.L.off_many_o) + kExchange;
        int64_t cum = 0;
        for (int e0 = 0; e0 < hd->n_many; e0 += 32) {
            const int i = e0 + lane;
            const int64_t mine = i < hd->n_many ? mp.units_of(s, list[i]) * mp.parts_of(list[i]) : 0;
            int64_t upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            unsigned cut = __ballot_sync(0xffffffffu, i < hd->n_many && mp.parts_of(list[min(i, hd->n_many - 1)]) > 1);
            while (cut) {
                const int l = __ffs(cut) - 1;
                cut &= cut - 1;
                const PagedEntry en = list[e0 + l];
                const int64_t first = cum + __shfl_sync(0xffffffffu, upto - mine, l);
                const int parts = mp.parts_of(en);
                const int64_t units = mp.units_of(s, en);
                const KeyRange kr = key_range(en.ctx, en.ctx + en.n - 1, s.window, s.sink);
                for (int64_t u = blockIdx.x * 2 + (threadIdx.x >> 8); u < units; u += gridDim.x * 2) {
                    const int x = 2 * (int)(u / s.Hkv) + (threadIdx.x >> 7 & 1);
                    if (x >= kr.n) continue;
                    const int j = kr.tile(x) * kKeyTile + (threadIdx.x & 127);
                    if (j >= en.ctx + en.n || !(s.window == 0 || j > en.ctx - s.window || j < s.sink)) continue;
                    const float *from = ws + (first + u * parts) * 256 + (threadIdx.x & 255);
                    float sum = 0.f;
                    for (int p = 0; p < parts; ++p) sum += ld_cg(from + (int64_t)p * 256);
                    const int64_t at = weight_place(a, en.r, j);
                    if (at >= 0) put(w.weights + at + (u % s.Hkv) * s.page_size, sum, j >= en.ctx);
                }
            }
            cum += __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    if ((int)blockIdx.x >= hd->ctas_few) return;
    if (warp == 0 && lane == 0) {
        *abort = 0;
        for (int i = 0; i < C::kSt; ++i) {
            mbar_init(&bars[C::B_KF + i], 1);
            mbar_init(&bars[C::B_KE + i], 1);
        }
        for (int i = 0; i < C::kSBuf; ++i) {
            mbar_init(&bars[C::B_SF + i], 1);
            mbar_init(&bars[C::B_SE + i], 4);
        }
        for (int i = 0; i < C::kQSlots; ++i) {
            mbar_init(&bars[C::B_QF + i], 4);
            mbar_init(&bars[C::B_QE + i], 10);
        }
        for (int i = 0; i < C::kRing; ++i) {
            mbar_init(&bars[C::B_UF + i], 1);
            mbar_init(&bars[C::B_UE + i], 15);
        }
        mbar_init(&bars[C::B_DRAIN], 2);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, 128);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const int G = s.Hq / s.Hkv;
    // a.wait_limit is for the thread that waits for K and for the drains; the other warps leave by the flag.
    constexpr long long lim = kWaitLimitCycles;
    auto read_unit = [&](int k) -> FewUnit {
        const int slot = k % C::kRing;
        FewUnit u{-1};
        if (!warp_wait(&bars[C::B_UF + slot], (k / C::kRing) & 1, abort, a.status, lim)) return u;
        const volatile int *p = sUnit + slot * 8;
        u = FewUnit{p[0], p[1], p[2], p[3], p[4], p[5], p[6]};
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[C::B_UE + slot]);
        return u;
    };
    auto range_of = [&](int ctx, int n) { return key_range(ctx, ctx + n - 1, s.window, s.sink); };

    if (warp == 0 || warp == 11) {
        // -------------------------------------------- the share's units (warp 0); K, every second tile each
        const int mine = warp == 0 ? 0 : 1;
        const PagedEntry *list = reinterpret_cast<const PagedEntry *>(a.plan + a.L.off_few);
        const PagedStart st0 = reinterpret_cast<const PagedStart *>(a.plan + a.L.off_start)[blockIdx.x];
        int left = st0.count, e = st0.e, h = st0.h, x = st0.x;
        PagedEntry en = st0.ent, en_next = list[min(e + 1, hd->n_few - 1)];
        bool run = true;
        // Cuts unit k off the share, and tells the others.
        auto next_unit = [&](int k) -> FewUnit {
            FewUnit u{-1};
            if (left > 0) {
                const int n = min(left, range_of(en.ctx, en.n).n - x);
                u = FewUnit{n, en.r, h, en.tok0, en.n, en.ctx, x};
                left -= n;
                x = 0;
                if (++h == s.Hkv) {
                    h = 0;
                    ++e;
                    en = en_next;
                    en_next = list[min(e + 1, hd->n_few - 1)];
                }
            }
            const int slot = k % C::kRing;
            if (k >= C::kRing && !warp_wait(&bars[C::B_UE + slot], ((k / C::kRing) - 1) & 1, abort, a.status, lim)) {
                run = false;
                return FewUnit{-1};
            }
            if (lane == 0) {
                const int f[7] = {u.n, u.r, u.h, u.tok0, u.ntok, u.ctx, u.x0};
#pragma unroll
                for (int i = 0; i < 7; ++i) sUnit[slot * 8 + i] = f[i];
                mbar_arrive(&bars[C::B_UF + slot]);
            }
            __syncwarp();
            return u;
        };
        auto unit = [&](int k) { return mine == 0 ? next_unit(k) : read_unit(k); };
        const int nb = kKeyTile / w.box_keys, batch = 32 / nb;     // boxes of a tile; tiles whose pages one look finds
        const int my_tile = lane / nb, my_box = lane - my_tile * nb;
        // Page and place in it of the lane's box of the unit's tile t0 + my_tile.
        struct Box {
            int page, in;
        };
        auto look_up = [&](const FewUnit &u, int t0) -> Box {
            const int t = t0 + my_tile;
            if (t >= u.n) return Box{s.num_pages, 0};
            const KeyRange kr = range_of(u.ctx, u.ntok);
            const int j = kr.tile(u.x0 + t) * kKeyTile + my_box * w.box_keys;
            const int b = a.page_shift >= 0 ? j >> a.page_shift : j / s.page_size, b0 = b * s.page_size;
            Box box{s.num_pages, j - b0};               // a page that no row needs arrives as zeros
            if (j < kr.hi && (b0 + s.page_size > kr.lo || b0 < s.sink)) {
                const int page = __ldg(a.table + (int64_t)u.r * s.max_pages + b);
                if ((unsigned)page < (unsigned)s.num_pages) box.page = page;
                else set_status(a.status, FM_ERR_PAGES);
            }
            return box;
        };
        int g = 0;
        unsigned loaded = 0;            // stages that this warp has loaded
        FewUnit u = unit(0);
        Box box = look_up(u, 0);
        // A unit ahead: the pages of its first tiles are on their way while this one's tiles are loaded.
        for (int k = 0; run && u.n >= 0; ++k) {
            const FewUnit un = unit(k + 1);
            const Box box_next = look_up(un, 0);
            for (int t0 = 0; run && t0 < u.n; t0 += batch) {
                const Box now = box;
                if (t0 + batch < u.n) box = look_up(u, t0 + batch);
                for (int t = t0; t < min(t0 + batch, u.n); ++t, ++g) {
                    if ((g & 1) != mine) continue;
                    const int st = g % C::kSt;
                    if (g >= C::kSt && !warp_wait(&bars[C::B_KE + st], ((g / C::kSt) - 1) & 1, abort, a.status, lim)) {
                        run = false;
                        break;
                    }
                    uint64_t *bar = &bars[C::B_KF + st];
                    // Wait test: one byte more than comes.
                    if (lane == 0) mbar_arrive_expect_tx(bar, C::kTile + (a.withhold && blockIdx.x == 0 && g == 1 ? 1 : 0));
                    loaded |= 1u << st;
                    __syncwarp();
                    if (t - t0 == my_tile) {
                        uint8_t *tile = smem + st * C::kTile;
#pragma unroll
                        for (int half = 0; half < NBOX; ++half)
                            tma_load_4d(tile + half * (128 * 128) + my_box * w.box_keys * (FP8 ? D : 128), &tk, bar, half * 64, now.in, u.h, now.page);
                    }
                    __syncwarp();
                }
            }
            u = un;
            box = box_next;
        }
        // After an abort: copies in flight end before the CTA leaves (the last load of a stage is that of its last tile before g).
        if (lane == 0 && *abort)
            for (int st = 0; st < C::kSt; ++st)
                if (loaded >> st & 1) {
                    const int last = g - 1 - ((g - 1 - st) % C::kSt + C::kSt) % C::kSt;
                    mbar_wait_drain(&bars[C::B_KF + st], (last / C::kSt) & 1, a.status, a.wait_limit);
                }
    } else if (warp == 1 || warp == 10) {
        // -------------------------------------------- K Q^T, every second tile
        const int mine = warp == 1 ? 0 : 1;
        auto desc = [&](uint8_t *p) {             // K-major rows of 128 bytes, or of 64 (e4m3, d = 64)
            return FP8 && D == 64 ? sdesc_sw64(smem_u32(p), 16, 512) : sdesc_sw128(smem_u32(p), 16, 1024);
        };
        int g = 0;
        bool run = true;
        for (int k = 0; run; ++k) {
            const FewUnit u = read_unit(k);
            if (u.n < 0) break;
            if (lane == 0) {
                const int cols = u.ntok * G <= 16 ? 16 : 32, qs = k % C::kQSlots;
                const uint32_t id = FP8 ? idesc_e4m3(128, cols) : idesc_bf16(128, cols, false, false);
                run = mbar_wait(&bars[C::B_QF + qs], (k / C::kQSlots) & 1, abort, a.status, lim);
                const uint64_t dQ = desc(smem + C::kQ + qs * C::kQBytes);
                for (int t = 0; run && t < u.n; ++t, ++g) {
                    if ((g & 1) != mine) continue;
                    const int st = g % C::kSt, sb = g % C::kSBuf;
                    if (!mbar_wait(&bars[C::B_KF + st], (g / C::kSt) & 1, abort, a.status, a.wait_limit) ||
                        (g >= C::kSBuf && !mbar_wait(&bars[C::B_SE + sb], ((g / C::kSBuf) - 1) & 1, abort, a.status, lim))) {
                        run = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t dK = desc(smem + st * C::kTile);
                    if (FP8) {
#pragma unroll
                        for (int term = 0; term < 2; ++term)
#pragma unroll
                            for (int kk = 0; kk < D / 32; ++kk)
                                mma_ss_e4m3(tmem + sb * 32, sdesc_add(dK, kk * 32), sdesc_add(dQ, term * C::kQTerm + kk * 32), id, term + kk > 0);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_ss(tmem + sb * 32, sdesc_add(dK, (kk >> 2) * (128 * 128) + (kk & 3) * 32),
                                   sdesc_add(dQ, (kk >> 2) * C::kQBox + (kk & 3) * 32), id, kk > 0);
                    }
                    tc_commit(&bars[C::B_SF + sb]);
                    tc_commit(&bars[C::B_KE + st]);
                }
                if (run) tc_commit(&bars[C::B_QE + qs]);
            }
            run = __shfl_sync(0xffffffffu, run, 0);
        }
        if (lane == 0) {
            tc_commit(&bars[C::B_DRAIN]);
            mbar_wait_drain(&bars[C::B_DRAIN], 0, a.status, a.wait_limit);
        }
    } else if (warp < 10) {
        // -------------------------------------------- exponentials and sums, every second tile
        const int mine = warp < 6 ? 0 : 1;
        const int key = (warp & 3) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        int g = 0;
        bool run = true;
        for (int k = 0; run; ++k) {
            const FewUnit u = read_unit(k);
            if (u.n < 0) break;
            const int qs = k % C::kQSlots, rows = u.ntok * G;
            if (!warp_wait(&bars[C::B_QF + qs], (k / C::kQSlots) & 1, abort, a.status, lim)) break;
            const float *fac = sCol + qs * 2 * kFewRows, *off = fac + kFewRows;
            const KeyRange kr = range_of(u.ctx, u.ntok);
            for (int t = 0; t < u.n; ++t, ++g) {
                if ((g & 1) != mine) continue;
                const int sb = g % C::kSBuf;
                const int j = kr.tile(u.x0 + t) * kKeyTile + key;
                // Rows that attend the key: tokens at its place or behind it, within the window.
                const int first = max(0, j - u.ctx), last = s.window > 0 && j >= s.sink ? min(u.ntok, j - u.ctx + s.window) : u.ntok;
                const uint32_t mask = first < last ? row_bits32(first * G, last * G) : 0u;
                const int64_t at = mask ? weight_place(a, u.r, j) : -1;      // on its way while the product is
                if (!warp_wait(&bars[C::B_SF + sb], (g / C::kSBuf) & 1, abort, a.status, lim)) {
                    run = false;
                    break;
                }
                tc_fence_after();
                float sum = 0.f;
                auto add = [&](const uint32_t *v, int c0, int n) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        if (c >= n) break;
                        const float p = ex2(fmaf(__uint_as_float(v[c]), FP8 ? fac[c0 + c] : a.scale_log2, off[c0 + c]));
                        sum += mask >> (c0 + c) & 1 ? p : 0.f;
                    }
                };
                const uint32_t tS = tmem + sb * 32 + lane_off;
                if (rows <= 8) {
                    uint32_t v[8];
                    tmem_ld8(tS, v);
                    tmem_ld_wait();
                    tmem_reg_fence(v);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[C::B_SE + sb]);
                    add(v, 0, 8);
                } else if (rows <= 16) {
                    uint32_t v[16];
                    tmem_ld16(tS, v);
                    tmem_ld_wait();
                    tmem_reg_fence(v);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[C::B_SE + sb]);
                    add(v, 0, 16);
                } else {
                    uint32_t v[32];
                    tmem_ld32(tS, v);
                    tmem_ld_wait();
                    tmem_reg_fence(v);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[C::B_SE + sb]);
                    add(v, 0, 32);
                }
                if (at >= 0) put(w.weights + at + (int64_t)u.h * s.page_size, sum, j >= u.ctx);
            }
            __syncwarp();
            if (run && lane == 0) mbar_arrive(&bars[C::B_QE + qs]);
        }
    } else if (warp >= 12) {
        // -------------------------------------------- Q and lse
        constexpr int LPR = D / 8, RPI = 32 / LPR, STEPS = kFewRows / RPI / 4;      // lanes per row, rows per step of a warp, its steps
        const int mate = warp - 12, l = lane % LPR, r_in = lane / LPR;
        const float scale = a.scale_log2 * (FP8 ? *a.k_descale : 1.f);
        for (int k = 0;; ++k) {
            const FewUnit u = read_unit(k);
            if (u.n < 0) break;
            const int qs = k % C::kQSlots, rows = u.ntok * G;
            uint4 x[STEPS];
            float z[STEPS];
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int row = (mate * STEPS + i) * RPI + r_in, t = row / G, hq = u.h * G + row - t * G;
                x[i] = make_uint4(0, 0, 0, 0);
                z[i] = 0.f;
                if (row < rows) {
                    x[i] = *reinterpret_cast<const uint4 *>(a.q + (int64_t)(u.tok0 + t) * a.q_tok + (int64_t)hq * a.q_head + l * 16);
                    if (l == 0) z[i] = w.lse[(int64_t)(u.tok0 + t) * s.Hq + hq];
                }
            }
            if (k >= C::kQSlots && !warp_wait(&bars[C::B_QE + qs], ((k / C::kQSlots) - 1) & 1, abort, a.status, lim)) break;
            uint8_t *q = smem + C::kQ + qs * C::kQBytes;
            float *fac = sCol + qs * 2 * kFewRows, *off = fac + kFewRows;
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int row = (mate * STEPS + i) * RPI + r_in;
                float f = 1.f;
                if (FP8) {
                    const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    float amax = 0.f;
#pragma unroll
                    for (int y = 0; y < 4; ++y) amax = fmax3(amax, fabsf(__uint_as_float(v[y] << 16)), fabsf(__uint_as_float(v[y] & 0xffff0000u)));
#pragma unroll
                    for (int y = 1; y < LPR; y <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, y));
                    // An infinite element makes the row NaN (it would saturate).
                    f = amax == INFINITY ? __uint_as_float(0x7fc00000u) : row_factor(amax, 7);
                    uint32_t hi[2] = {0u, 0u}, lw[2] = {0u, 0u};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const float q0 = __uint_as_float(v[y] << 16) * f, q1 = __uint_as_float(v[y] & 0xffff0000u) * f;
                        const uint32_t h = pack_e4m3x2(q0, q1);
                        float h0, h1;
                        unpack_f16x2(f16x2_of_e4m3(h), h0, h1);
                        hi[y >> 1] |= h << (16 * (y & 1));
                        lw[y >> 1] |= pack_e4m3x2(q0 - h0, q1 - h1) << (16 * (y & 1));
                    }
                    const uint32_t at = D == 128 ? row * 128 + (((l >> 1) ^ (row & 7)) << 4) : row * 64 + (((l >> 1) ^ ((row >> 1) & 3)) << 4);
                    uint8_t *p = q + at + (l & 1) * 8;
                    *reinterpret_cast<uint2 *>(p) = make_uint2(hi[0], hi[1]);
                    *reinterpret_cast<uint2 *>(p + C::kQTerm) = make_uint2(lw[0], lw[1]);
                } else {
                    st_shared_v4(q + (l >> 3) * C::kQBox + row * 128 + (((l & 7) ^ (row & 7)) << 4), x[i]);
                }
                if (l == 0) {
                    fac[row] = scale / f;
                    off[row] = -z[i] * kLog2e;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[C::B_QF + qs]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 128);
    }
}

// ---- many rows ------------------------------------------------------------------------

template <int D, bool FP8>
struct ManyCfg {
    static constexpr int kThreads = FP8 ? 768 : 640;
    static constexpr int kBox = 128 * 128, kTile = 128 * D * 2, kRaw = 128 * D;
    // bf16: K of two units. e4m3: K of one unit, and of the next as it comes.
    static constexpr int kKBuf = FP8 ? 1 : 2, kQSt = D == 64 ? 6 : FP8 ? 4 : 3, kLSt = 4, kRing = 4;
    static constexpr int kK = 0;                                  // [kKBuf][2 key tiles]
    static constexpr int kQ = kK + kKBuf * 2 * kTile;
    static constexpr int kRawK = kQ + kQSt * kTile;               // e4m3: [2 key tiles]
    static constexpr int kLse = kRawK + (FP8 ? 2 * kRaw : 0);     // float [kLSt][128]
    static constexpr int kUnit = kLse + kLSt * 128 * 4;           // int [kRing][kInts]
    static constexpr int kInts = 12;
    static constexpr int kBar = kUnit + kRing * kInts * 4;
    enum { B_KF = 0, B_KE = B_KF + kKBuf, B_RF = B_KE + kKBuf, B_RE, B_QF, B_QE = B_QF + kQSt, B_SF = B_QE + kQSt, B_SE = B_SF + 4,
           B_LF = B_SE + 4, B_LE = B_LF + kLSt, B_XF = B_LE + kLSt, B_XE = B_XF + 4, B_UF = B_XE + 4, B_UE = B_UF + kRing, B_DRAIN = B_UE + kRing, B_COUNT };
    static constexpr int kMisc = kBar + B_COUNT * 8;
    // Over 114 KB, so that one CTA with all of TMEM is resident per SM.
    static constexpr int kBytes = kMisc + 64 > 120 * 1024 ? kMisc + 64 : 120 * 1024;
    static_assert(kBytes <= 227 * 1024 && kBar % 8 == 0, "shared memory");
    static constexpr int kReaders = 19 + (FP8 ? 4 : 0);
    static_assert(kLSt % 2 == 0, "alternate row tiles meet alternate places");
};

// Two key tiles and the row tiles that attend one of them.
struct ManyUnit {
    int n;                  // row tiles; -1: no more
    int r, h, tok0, ntok, ctx;
    int t0;                 // first row tile
    int kb[2];              // first key of either tile (the second one may lie behind the request: no row attends it)
    int piece;              // where the sums go in the workspace; -1: to the weights
};

// PAD: the last columns of a row tile that may be empty, 0, 8 or 24, where K may hold infinities (bf16).  Columns that no token fills (128
// is no multiple of the query heads of a KV head) are rows of zeros, which have no score beside such a key; the tokens' rows may have
// scored it at -infinity, a weight of nothing.  So these columns are masked, in a kernel of its own: chunks of 4,096 tokens of 28 / 4
// heads 294 -> 297 us (with the last 32 305, the sum looked at and taken again 311), of 28 / 1, with 24 columns, 320 -> 338.
// An e4m3 code is finite, or no number for every row.
template <int D, bool FP8, int PAD>
__global__ void __launch_bounds__(ManyCfg<D, FP8>::kThreads, 1)
    fm_paged_weigh_many_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk, const WeighArgs w)
{
    using C = ManyCfg<D, FP8>;
    constexpr int NBOX = D / 64;
    extern __shared__ __align__(1024) uint8_t smem[];
    float *sLse = reinterpret_cast<float *>(smem + C::kLse);
    volatile int *sUnit = reinterpret_cast<volatile int *>(smem + C::kUnit);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBar);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::kMisc);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + C::kMisc + 4);
    const PagedArgs &a = w.p;
    const PagedShape &s = a.s;
    const PagedHeader *hd = reinterpret_cast<const PagedHeader *>(a.plan);
    const int warp = warp_id(), lane = lane_id();
    // The same verdict in every CTA: none claims a unit of a plan that does not fit.
    if (!paged_plan_fits(hd, s) || hd->rows > a.rows || (smem_u32(smem) & 1023u) != 0) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            set_status(a.status, !paged_plan_fits(hd, s) ? FM_ERR_PLAN_MISMATCH : hd->rows > a.rows ? FM_ERR_LENGTHS : FM_ERR_UNSUPPORTED);
        return;
    }
    if (hd->n_many == 0) return;
    const int G = s.Hq / s.Hkv, tpt = 128 / G;      // tokens of a row tile
    if (warp == 0 && lane == 0) {
        *abort = 0;
        for (int i = 0; i < C::kKBuf; ++i) {
            mbar_init(&bars[C::B_KF + i], FP8 ? 4 : 1);
            mbar_init(&bars[C::B_KE + i], 2);
        }
        mbar_init(&bars[C::B_RF], 1);
        mbar_init(&bars[C::B_RE], 4);
        for (int i = 0; i < C::kQSt; ++i) {
            mbar_init(&bars[C::B_QF + i], 1);
            mbar_init(&bars[C::B_QE + i], 2);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars[C::B_SF + i], 1);
            mbar_init(&bars[C::B_SE + i], 4);
            mbar_init(&bars[C::B_XF + i], 4);
            mbar_init(&bars[C::B_XE + i], 4);
        }
        for (int i = 0; i < C::kLSt; ++i) {
            mbar_init(&bars[C::B_LF + i], 1);
            mbar_init(&bars[C::B_LE + i], 8);
        }
        for (int i = 0; i < C::kRing; ++i) {
            mbar_init(&bars[C::B_UF + i], 1);
            mbar_init(&bars[C::B_UE + i], C::kReaders);
        }
        mbar_init(&bars[C::B_DRAIN], 2);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    // Rows of a row tile that no token fills (128 is no multiple of G) are zeros for good: TMA writes the others alone.
    const int filled = G * tpt;
    for (int i = threadIdx.x; i < C::kQSt * NBOX * (128 - filled) * 8; i += C::kThreads) {
        const int ch = i & 7, row = (i >> 3) % (128 - filled), box = (i >> 3) / (128 - filled);
        st_shared_v4(smem + C::kQ + box * C::kBox + (filled + row) * 128 + ch * 16, make_uint4(0, 0, 0, 0));
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    constexpr long long lim = kWaitLimitCycles;
    auto read_unit = [&](int k) -> ManyUnit {
        const int slot = k % C::kRing;
        ManyUnit u{-1};
        if (!warp_wait(&bars[C::B_UF + slot], (k / C::kRing) & 1, abort, a.status, lim)) return u;
        const volatile int *p = sUnit + slot * C::kInts;
        u = ManyUnit{p[0], p[1], p[2], p[3], p[4], p[5], p[6], {p[7], p[8]}, p[9]};
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[C::B_UE + slot]);
        return u;
    };

    if (warp == 0) {
        // -------------------------------------------- claims; K
        const PagedEntry *list = reinterpret_cast<const PagedEntry *>(a.plan + a.L.off_many);
        unsigned *claim = reinterpret_cast<unsigned *>(a.plan + a.L.off_claim);
        const ManyPieces mp = many_pieces(a, hd, tpt);
        if (blockIdx.x == 0 && lane == 0) reinterpret_cast<PagedHeader *>(a.plan)->weigh_len = mp.pieces > mp.units ? mp.len : 0;
        const bool fits = mp.pieces < (int64_t)1 << 31;
        if (!fits && blockIdx.x == 0 && lane == 0) set_status(a.status, FM_ERR_LENGTHS);
        const unsigned n_claims = fits ? (unsigned)mp.pieces : 0u;
        int e = 0;
        int64_t cum = 0;            // pieces before entry e
        PagedEntry en = list[0];
        int64_t units = mp.units_of(s, en);
        int parts = mp.parts_of(en);
        const int nb = kKeyTile / w.box_keys;
        bool run = true;
        int started = 0;            // loads of K
        for (int k = 0;; ++k) {
            ManyUnit u{-1};
            while (n_claims > 0) {
                unsigned c = 0;
                // Every CTA claims once past the end: the counter comes back to 0 by itself.
                if (lane == 0) c = atomicInc(claim, n_claims + gridDim.x - 1);
                c = __shfl_sync(0xffffffffu, c, 0);
                if (c >= n_claims) break;
                // Claims only grow, so the entry is at or behind the last one.
                while ((int64_t)c >= cum + units * parts) {
                    const int i = e + lane;
                    const int64_t mine = i < hd->n_many ? mp.units_of(s, list[i]) * mp.parts_of(list[i]) : 0;
                    int64_t upto = mine;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
                        if (lane >= o) upto += y;
                    }
                    const int past = __popc(__ballot_sync(0xffffffffu, cum + upto <= (int64_t)c));     // entries that end before the claim
                    const int64_t gone = __shfl_sync(0xffffffffu, upto, max(past - 1, 0));
                    if (past > 0) cum += gone;
                    e += past;
                    en = list[min(e, hd->n_many - 1)];
                    units = mp.units_of(s, en);
                    parts = mp.parts_of(en);
                }
                const int local = (int)((int64_t)c - cum), part = local % parts, unit = local / parts, x = unit / s.Hkv;
                const KeyRange kr = key_range(en.ctx, en.ctx + en.n - 1, s.window, s.sink);
                u = ManyUnit{0, en.r, unit - x * s.Hkv, en.tok0, en.n, en.ctx, 0, {0, 0}, parts > 1 ? (int)c : -1};
                // Row tiles [t0, t1) attend the unit: from the first token at its first key's place on, until the last within a
                // window of its last key.
                int t1 = 0;
                u.t0 = INT32_MAX;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    u.kb[y] = 2 * x + y < kr.n ? kr.tile(2 * x + y) * kKeyTile : (kr.hi + kKeyTile - 1) / kKeyTile * kKeyTile;
                    if (2 * x + y >= kr.n) continue;
                    u.t0 = min(u.t0, max(0, u.kb[y] - en.ctx) / tpt);
                    int last = (en.n + tpt - 1) / tpt;
                    if (s.window > 0 && u.kb[y] >= s.sink) last = min(last, max(u.kb[y] - en.ctx + kKeyTile - 2 + s.window + tpt, 0) / tpt);
                    t1 = max(t1, last);
                }
                // The piece's share of them, which may be empty (its sums are then zeros).
                const int n = max(t1 - u.t0, 0), t_first = (int)((int64_t)n * part / parts);
                u.n = (int)((int64_t)n * (part + 1) / parts) - t_first;
                u.t0 += t_first;
                break;
            }
            // The tiles' pages, looked up before the waits: lane i the box i of the two tiles.
            int page = s.num_pages, in = 0;
            if (u.n > 0 && lane < 2 * nb) {
                const KeyRange kr = key_range(u.ctx, u.ctx + u.ntok - 1, s.window, s.sink);
                const int j = (lane < nb ? u.kb[0] + lane * w.box_keys : u.kb[1] + (lane - nb) * w.box_keys);
                const int b = a.page_shift >= 0 ? j >> a.page_shift : j / s.page_size, b0 = b * s.page_size;
                in = j - b0;
                if (j < kr.hi && (b0 + s.page_size > kr.lo || b0 < s.sink)) {
                    const int p = __ldg(a.table + (int64_t)u.r * s.max_pages + b);
                    if ((unsigned)p < (unsigned)s.num_pages) page = p;
                    else set_status(a.status, FM_ERR_PAGES);
                }
            }
            const int slot = k % C::kRing, ks = k % C::kKBuf;
            if (k >= C::kRing && !warp_wait(&bars[C::B_UE + slot], ((k / C::kRing) - 1) & 1, abort, a.status, lim)) run = false;
            if (!run) break;
            if (lane == 0) {
                const int f[10] = {u.n, u.r, u.h, u.tok0, u.ntok, u.ctx, u.t0, u.kb[0], u.kb[1], u.piece};
#pragma unroll
                for (int i = 0; i < 10; ++i) sUnit[slot * C::kInts + i] = f[i];
                mbar_arrive(&bars[C::B_UF + slot]);
            }
            __syncwarp();
            if (u.n < 0) break;
            // Where the tiles go is free again: the codes converted, or K multiplied.
            if (FP8 ? k >= 1 && !warp_wait(&bars[C::B_RE], (k - 1) & 1, abort, a.status, lim)
                    : k >= C::kKBuf && !warp_wait(&bars[C::B_KE + ks], (k / C::kKBuf - 1) & 1, abort, a.status, lim))
                break;
            uint64_t *bar = &bars[FP8 ? C::B_RF : C::B_KF + ks];
            // Wait test: one byte more than comes.
            if (lane == 0) mbar_arrive_expect_tx(bar, 2 * (FP8 ? C::kRaw : C::kTile) + a.withhold);
            ++started;
            __syncwarp();
            if (lane < 2 * nb) {
                const int y = lane < nb ? 0 : 1, box = lane - y * nb;
                if (FP8) {
                    tma_load_4d(smem + C::kRawK + y * C::kRaw + box * w.box_keys * D, &tk, bar, 0, in, u.h, page);
                } else {
#pragma unroll
                    for (int half = 0; half < NBOX; ++half)
                        tma_load_4d(smem + C::kK + (ks * 2 + y) * C::kTile + half * C::kBox + box * w.box_keys * 128, &tk, bar, half * 64, in, u.h, page);
                }
            }
            __syncwarp();
        }
        if (lane == 0 && *abort) {
            if (FP8 && started > 0) mbar_wait_drain(&bars[C::B_RF], (started - 1) & 1, a.status, a.wait_limit);
            for (int i = max(started - C::kKBuf, 0); !FP8 && i < started; ++i)
                mbar_wait_drain(&bars[C::B_KF + i % C::kKBuf], (i / C::kKBuf) & 1, a.status, a.wait_limit);
        }
    } else if (warp == 1 || warp == 19) {
        // -------------------------------------------- K Q^T of one of the key tiles
        constexpr uint32_t id = idesc_bf16(128, 128, false, false);
        const int mine = warp == 1 ? 0 : 1;
        int g = 0;
        bool run = true;
        for (int k = 0; run; ++k) {
            const ManyUnit u = read_unit(k);
            if (u.n < 0) break;
            if (lane == 0) {
                const int ks = k % C::kKBuf;
                run = mbar_wait(&bars[C::B_KF + ks], (k / C::kKBuf) & 1, abort, a.status, a.wait_limit);
                const uint64_t dK = sdesc_sw128(smem_u32(smem + C::kK + (ks * 2 + mine) * C::kTile), 16, 1024);
                for (int t = 0; run && t < u.n; ++t, ++g) {
                    const int st = g % C::kQSt, sb = 2 * mine + (g & 1);
                    if (!mbar_wait(&bars[C::B_QF + st], (g / C::kQSt) & 1, abort, a.status, a.wait_limit) ||
                        (g >= 2 && !mbar_wait(&bars[C::B_SE + sb], ((g >> 1) - 1) & 1, abort, a.status, a.wait_limit))) {
                        run = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t dQ = sdesc_sw128(smem_u32(smem + C::kQ + st * C::kTile), 16, 1024);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::kBox + (kk & 3) * 32;
                        mma_ss(tmem + sb * 128, sdesc_add(dK, off), sdesc_add(dQ, off), id, kk > 0);
                    }
                    tc_commit(&bars[C::B_SF + sb]);
                    tc_commit(&bars[C::B_QE + st]);
                }
                if (run) tc_commit(&bars[C::B_KE + ks]);
            }
            run = __shfl_sync(0xffffffffu, run, 0);
        }
        if (lane == 0) {
            tc_commit(&bars[C::B_DRAIN]);
            mbar_wait_drain(&bars[C::B_DRAIN], 0, a.status, a.wait_limit);
        }
    } else if (warp < 18) {
        // -------------------------------------------- exponentials and sums: of one of the key tiles, alternate row tiles
        const int mine = warp < 10 ? 0 : 1, turn = (warp - 2) >> 2 & 1;
        const int key = (warp & 3) * 32 + lane, sb = 2 * mine + turn;
        const uint32_t tS = tmem + sb * 128 + ((uint32_t)((warp & 3) * 32) << 16);
        const float scale = a.scale_log2 * (FP8 ? *a.k_descale : 1.f);
        const uint64_t sc2 = f2_pack(scale, scale);
        // Where the odd row tiles' sums go to those of the even ones: in the plan's workspace, for shared memory is full; by unit and
        // key tile in turn.
        float *part = reinterpret_cast<float *>(a.plan + a.L.off_many_o) + ((int64_t)blockIdx.x * 4 + mine) * 128 + key;
        float *ws = reinterpret_cast<float *>(a.plan + a.L.off_many_o) + kExchange + mine * 128 + key;     // of pieces
        int g = 0;
        bool run = true;
        for (int k = 0; run; ++k) {
            const ManyUnit u = read_unit(k);
            if (u.n < 0) break;
            const int kb = mine ? u.kb[1] : u.kb[0], j = kb + key, seq = u.ctx + u.ntok;
            const bool some = j < seq && (s.window == 0 || j > u.ctx - s.window || j < s.sink);     // attended by some row
            int64_t at = -1;
            if (turn == 0 && some) at = weight_place(a, u.r, j);
            float sum = 0.f;
            for (int t = 0; t < u.n; ++t, ++g) {
                if ((g & 1) != turn) continue;
                const int ls = g % C::kLSt;
                const int tok = (u.t0 + t) * tpt, pos = u.ctx + tok, ntok = min(tpt, u.ntok - tok);
                // Free of the mask: every row behind every key, within every window.
                const bool full = kb + kKeyTile - 1 <= pos && ntok == tpt && (s.window == 0 || kb > pos + tpt - 1 - s.window || kb + kKeyTile <= s.sink);
                if (!warp_wait(&bars[C::B_LF + ls], (g / C::kLSt) & 1, abort, a.status, lim) ||
                    !warp_wait(&bars[C::B_SF + sb], (g >> 1) & 1, abort, a.status, lim)) {
                    run = false;
                    break;
                }
                tc_fence_after();
                int lo = 0, hi = 128;               // the row tile's columns that attend the key
                bool any = true;
                if (!full) {
                    lo = some ? min(max(j - pos, 0), 128) * G : 128;
                    hi = (s.window > 0 && j >= s.sink ? min(max(j - pos + s.window, 0), ntok) : ntok) * G;
                    any = __any_sync(0xffffffffu, lo < hi);
                }
                const float4 *z = reinterpret_cast<const float4 *>(sLse + ls * 128);
                uint64_t sum2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
                // (The mask is put over the exponents: a row that does not attend the key gives it nothing, whatever its lse.)  `first`:
                // the group of four columns from which on it is looked at.
                auto add = [&](const uint32_t (&x)[32], const float4 *off, uint32_t keep, auto first) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 o = off[i];
                        float e[4];
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1])), sc2, f2_pack(o.x, o.y)), e[0], e[1]);
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3])), sc2, f2_pack(o.z, o.w)), e[2], e[3]);
                        if (i >= decltype(first)::value) {
#pragma unroll
                            for (int y = 0; y < 4; ++y) e[y] = keep >> (4 * i + y) & 1 ? e[y] : -INFINITY;
                        }
                        sum2[0] = f2_add(sum2[0], f2_pack(ex2(e[0]), ex2(e[1])));
                        sum2[1] = f2_add(sum2[1], f2_pack(ex2(e[2]), ex2(e[3])));
                    }
                };
                auto release = [&]() {              // every score is in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[C::B_SE + sb]);
                };
                if (full) {
                    uint32_t x[2][32];              // the next ones on their way
                    tmem_ld32(tS, x[0]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        tmem_ld_wait();
                        tmem_reg_fence(x[c & 1]);
                        if (c < 3) tmem_ld32(tS + 32 * (c + 1), x[(c + 1) & 1]);
                        else release();
                        if (c < 3) add(x[c & 1], z + c * 8, 0u, std::integral_constant<int, 8>{});
                        else add(x[c & 1], z + c * 8, row_bits32(0, filled - 96), std::integral_constant<int, 8 - PAD / 4>{});
                    }
                } else if (any) {
                    // (Rolled up: unrolled beside the other one it costs 5 % of the whole, in registers and instruction fetches.)
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t x[32];
                        tmem_ld32(tS + 32 * c, x);
                        tmem_ld_wait();
                        tmem_reg_fence(x);
                        if (c == 3) release();
                        add(x, z + c * 8, row_bits32(lo - 32 * c, hi - 32 * c), std::integral_constant<int, 0>{});
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    if (!any) mbar_arrive(&bars[C::B_SE + sb]);
                    mbar_arrive(&bars[C::B_LE + ls]);
                }
                float s0, s1;
                f2_unpack(f2_add(sum2[0], sum2[1]), s0, s1);
                sum += s0 + s1;
            }
            if (!run) break;
            const int x = 2 * mine + (k & 1);
            float *to = part + (k & 1) * 256;
            if (turn == 1) {
                if (k >= 2 && !warp_wait(&bars[C::B_XE + x], ((k >> 1) - 1) & 1, abort, a.status, lim)) break;
                __stcg(to, sum);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[C::B_XF + x]);
            } else {
                if (!warp_wait(&bars[C::B_XF + x], (k >> 1) & 1, abort, a.status, lim)) break;
                sum += ld_cg(to);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[C::B_XE + x]);
                if (u.piece >= 0) __stcg(ws + (int64_t)u.piece * 256, sum);
                else if (at >= 0) put(w.weights + at + (int64_t)u.h * s.page_size, sum, j >= u.ctx);
            }
        }
    } else if (warp == 18) {
        // -------------------------------------------- Q and lse of the row tiles
        int tk[4], at[4];                   // token of a row tile's row (past any step's rows where none fills it), and its place from the tile's first
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = lane + 32 * i;
            tk[i] = c < filled ? c / G : 1 << 30;
            at[i] = c < filled ? tk[i] * s.Hq + c % G : 0;
        }
        int g = 0;
        bool run = true;
        for (int k = 0; run; ++k) {
            const ManyUnit u = read_unit(k);
            if (u.n < 0) break;
            float z[4];
            auto fetch = [&](int t) {
                const int tok = (u.t0 + t) * tpt;
                const float *p = w.lse + (int64_t)(u.tok0 + tok) * s.Hq + u.h * G;
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = tok + tk[i] < u.ntok ? __ldg(p + at[i]) : INFINITY;
            };
            fetch(0);
            for (int t = 0; t < u.n; ++t, ++g) {
                const int st = g % C::kQSt, ls = g % C::kLSt;
                if (g >= C::kQSt && !warp_wait(&bars[C::B_QE + st], ((g / C::kQSt) - 1) & 1, abort, a.status, lim)) {
                    run = false;
                    break;
                }
                if (lane == 0) {
                    uint64_t *bar = &bars[C::B_QF + st];
                    mbar_arrive_expect_tx(bar, (uint32_t)(filled * D * 2));
#pragma unroll
                    for (int x = 0; x < NBOX; ++x)
                        tma_load_3d(smem + C::kQ + st * C::kTile + x * C::kBox, &tq, bar, x * 64, u.h * G, u.tok0 + (u.t0 + t) * tpt);
                }
                __syncwarp();
                float now[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) now[i] = -z[i] * kLog2e;
                if (t + 1 < u.n) fetch(t + 1);
                if (g >= C::kLSt && !warp_wait(&bars[C::B_LE + ls], ((g / C::kLSt) - 1) & 1, abort, a.status, lim)) {
                    ++g;
                    run = false;
                    break;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) sLse[ls * 128 + lane + 32 * i] = now[i];
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[C::B_LF + ls]);
            }
        }
        if (lane == 0 && *abort)
            for (int i = (g > C::kQSt ? g - C::kQSt : 0); i < g; ++i)
                mbar_wait_drain(&bars[C::B_QF + i % C::kQSt], (i / C::kQSt) & 1, a.status, a.wait_limit);
    } else if (FP8) {
        // -------------------------------------------- K to bf16
        const int mate = warp & 3;
        constexpr int LPR = D / 8, RPI = 32 / LPR;        // lanes per row, rows per step of a warp
        const int l = lane % LPR, r_in = lane / LPR;
        auto bf16x2 = [](uint32_t x) {
            float lo, hi;
            unpack_f16x2(f16x2_of_e4m3(x), lo, hi);
            return pack_bf16x2(lo, hi);
        };
        for (int k = 0;; ++k) {
            const ManyUnit u = read_unit(k);
            if (u.n < 0) break;
            if (!warp_wait(&bars[C::B_RF], k & 1, abort, a.status, lim)) break;
            if (k >= 1 && !warp_wait(&bars[C::B_KE], (k - 1) & 1, abort, a.status, lim)) break;
            const uint8_t *raw = smem + C::kRawK;
#pragma unroll 4
            for (int i = mate; i < 256 / RPI; i += 4) {
                const int line = i * RPI + r_in, row = line & 127;
                const uint2 x = *reinterpret_cast<const uint2 *>(raw + line * D + l * 8);
                uint8_t *tile = smem + C::kK + (line >> 7) * C::kTile;
                st_shared_v4(tile + (l >> 3) * C::kBox + row * 128 + (((l & 7) ^ (row & 7)) << 4),
                             make_uint4(bf16x2(x.x), bf16x2(x.x >> 16), bf16x2(x.y), bf16x2(x.y >> 16)));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars[C::B_KF]);
                mbar_arrive(&bars[C::B_RE]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Opts a kernel into its shared memory, once per device.
template <class K>
fm_status ready(K kernel, int bytes, std::atomic<uint8_t> *done)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FM_ERR_CUDA;
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return FM_ERR_CUDA;
        done[dev].store(1, std::memory_order_release);
    }
    return FM_OK;
}

template <int D, bool FP8>
fm_status launch_few(const CUtensorMap &tk, const WeighArgs &w, cudaStream_t stream)
{
    using C = FewCfg<D, FP8>;
    static std::atomic<uint8_t> done[kMaxDevices];
    const fm_status st = ready(fm_paged_weigh_few_kernel<D, FP8>, C::kBytes, done);
    if (st != FM_OK) return st;
    ProfScope ps(kKPagedWeighFew, stream);
    fm_paged_weigh_few_kernel<D, FP8><<<kPagedCtas, C::kThreads, C::kBytes, stream>>>(tk, w);
    return cudaPeekAtLastError() == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

template <int D, bool FP8, int PAD>
fm_status launch_many(const CUtensorMap &tq, const CUtensorMap &tk, const WeighArgs &w, cudaStream_t stream)
{
    using C = ManyCfg<D, FP8>;
    static std::atomic<uint8_t> done[kMaxDevices];
    const fm_status st = ready(fm_paged_weigh_many_kernel<D, FP8, PAD>, C::kBytes, done);
    if (st != FM_OK) return st;
    ProfScope ps(kKPagedWeighMany, stream);
    fm_paged_weigh_many_kernel<D, FP8, PAD><<<kPagedCtas, C::kThreads, C::kBytes, stream>>>(tq, tk, w);
    return cudaPeekAtLastError() == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

}  // namespace
}  // namespace fm

using namespace fm;

extern "C" fm_status fm_paged_weights(const fm_paged_step *step, const void *q, int64_t q_tok, int64_t q_head, int rows,
                                      const fm_paged_cache *cache, const int32_t *block_table, void *plan, size_t plan_bytes, float scale,
                                      const float *lse, float *weights, int32_t *dev_status, fm_stream_t stream)
{
    WeighArgs w{};
    PagedArgs &a = w.p;
    fm_status st = check_step(step, &a.s);
    if (st != FM_OK) return st;
    if ((st = check_cache(cache)) != FM_OK) return st;
    if (cache->num_pages != a.s.num_pages || cache->page_size != a.s.page_size || cache->Hkv != a.s.Hkv || cache->d != a.s.d)
        return FM_ERR_INVALID_ARG;
    if (rows < 0 || !rows_ok(q, q_tok, q_head) || !aligned4(lse) || !aligned16(weights) || !aligned4(block_table) || !aligned4(dev_status))
        return FM_ERR_INVALID_ARG;
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
    a.status = dev_status;
    a.scale_log2 = scale * kLog2e;
    a.rows = rows;
    a.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (a.s.page_size == 1 << i) a.page_shift = i;
    w.lse = lse;
    w.weights = weights;
    // Boxes of consecutive keys of one page, a power of two of them.
    w.box_keys = kPageGranule;
    while (w.box_keys < kKeyTile && a.s.page_size % (2 * w.box_keys) == 0) w.box_keys *= 2;
    const int G = a.s.Hq / a.s.Hkv;
    const bool d128 = a.s.d == 128;
    const uint64_t cd[4] = {(uint64_t)a.s.d, (uint64_t)a.s.page_size, (uint64_t)a.s.Hkv, (uint64_t)a.s.num_pages};
    const uint64_t ks[3] = {(uint64_t)(cache->k_tok * esz), (uint64_t)(cache->k_head * esz), (uint64_t)(cache->k_page * esz)};
    const uint32_t cb[4] = {fp8 ? (uint32_t)a.s.d : 64u, (uint32_t)w.box_keys, 1, 1};
    cudaStream_t cs = (cudaStream_t)stream;
    CUtensorMap tq, tk;
    if ((int64_t)a.s.max_q * G > kFewRows) {            // some request may have many rows
        const uint64_t qd[3] = {(uint64_t)a.s.d, (uint64_t)a.s.Hq, (uint64_t)(rows > 0 ? rows : 1)};
        const uint64_t qs[2] = {(uint64_t)a.q_head, (uint64_t)a.q_tok};
        const uint32_t qb[3] = {64, (uint32_t)G, (uint32_t)(128 / G)};
        if (!make_tmap_strided(&tq, q, false, 3, qd, qs, qb, 128) || !make_tmap_strided(&tk, cache->k, fp8, 4, cd, ks, cb, fp8 ? 0 : 128))
            return FM_ERR_CUDA;
        wait_test_args(kKPagedWeighMany, &a.wait_limit, &a.withhold);
        const int empty = 128 % G;          // 24 at most, with 26 heads
        if (fp8) st = d128 ? launch_many<128, true, 0>(tq, tk, w, cs) : launch_many<64, true, 0>(tq, tk, w, cs);
        else if (empty == 0) st = d128 ? launch_many<128, false, 0>(tq, tk, w, cs) : launch_many<64, false, 0>(tq, tk, w, cs);
        else if (empty <= 8) st = d128 ? launch_many<128, false, 8>(tq, tk, w, cs) : launch_many<64, false, 8>(tq, tk, w, cs);
        else st = d128 ? launch_many<128, false, 24>(tq, tk, w, cs) : launch_many<64, false, 24>(tq, tk, w, cs);
        if (st != FM_OK) return st;
    }
    if (!make_tmap_strided(&tk, cache->k, fp8, 4, cd, ks, cb, fp8 ? a.s.d : 128)) return FM_ERR_CUDA;
    wait_test_args(kKPagedWeighFew, &a.wait_limit, &a.withhold);
    if (d128) return fp8 ? launch_few<128, true>(tk, w, cs) : launch_few<128, false>(tk, w, cs);
    return fp8 ? launch_few<64, true>(tk, w, cs) : launch_few<64, false>(tk, w, cs);
}
