// Attention of many new tokens over a paged cache (prompt chunks), on tcgen05:
// requests with more than kFewRows rows (new tokens x query heads per KV head).
//
//   o_row = sum_j p_j v_j / sum_j p_j,  p_j = exp2(s_j - m),  s_j = scale log2(e) q_row . k_j
//
// The structure of the masked forward kernel: a unit is 128 rows of one
// (request, KV head) — the query heads that share the KV head times as many tokens as
// fit, so K and V are read once for all of them — against the key tiles (128
// keys) that some row attends; S = Q K^T in TMEM (three buffers), softmax by two
// warpgroups on alternate tiles, P back to TMEM as the operand of O += P V, the
// running maximum handed from tile to tile and raised lazily.  Bound by the
// tensor pipe and the exponentials at long chunks.
//   warp 0      claims units, TMA of Q and K (a box of consecutive keys of one
//               page per lane; the lane looks its page up itself)
//   warp 1      TMEM; one thread issues Q K^T
//   warps 2-5   softmax of even tiles, thread = row
//   warps 6-9   softmax of odd tiles
//   warp 10     TMA of V
//   warp 11     one thread issues P V
//   warps 12-15 e4m3 caches only: Q to e4m3 terms, V to fp16, in shared memory
// e4m3 caches: K is multiplied as it is (kind::f8f6f4, twice the rate of 16 bits) by Q as
// two e4m3 terms of four bits each, which together hold bf16's eight: after a
// power of two per row that puts its largest element in [128, 256), and which the
// score factor takes back, elements down to 2^-9 of it are exact and smaller
// ones are off by at most 2^-17 of it.  V becomes fp16, exactly, because P needs
// more bits than e4m3 has.
// P: bf16 caches one bf16 term for 16-bit outputs, two (hi + lo) for fp32
// outputs; e4m3 caches fp16 terms likewise, lifted by 2^kLift.  A second term doubles
// the second product and the softmax's packing: 4,178 tokens over up to 16K keys 0.59 ms with one,
// 1.03 with two, for 2.3e-3 of relative error in place of the bf16 output's own 1.7e-3.
//
// The mask is arithmetic: a row at position p attends keys j <= p, j > p -
// window or j < sink, so a tile is either free of it or compared element by
// element against three numbers per row.  Keys outside the request are never
// part of a product: masked scores are replaced, V rows behind the last token
// are zeroed in shared memory (0 x NaN), pages that no row needs arrive as zeros.
//
// Few units (a short chunk over a long cache) are split along the keys into
// pieces, whose partial sums the kernel behind this one adds up in their order, with
// every SM (one CTA, the last to arrive, reads 64 KB a part at about 30 bytes a
// cycle: 60 us and more for 29 parts).
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "fm_paged.h"
#include "fm_ptx.cuh"

namespace fm {
namespace {

constexpr int kSBuf = 3, kMaxSt = 4, kRing = 4, kUnitInts = 16;

enum {
    B_Q = 0, B_QR,                                   // Q ready; Q landed (e4m3: before its conversion)
    B_KF, B_KE = B_KF + kMaxSt,                      // K stage ready / free
    B_VF = B_KE + kMaxSt, B_VE = B_VF + kMaxSt, B_VR = B_VE + kMaxSt,   // V stage ready / free / landed, but not ready
    B_S = B_VR + kMaxSt, B_P = B_S + kSBuf, B_PB = B_P + kSBuf, B_O = B_PB + kSBuf,
    B_QE = B_O + kSBuf, B_OE, B_UF, B_UE = B_UF + kRing, B_DRAIN = B_UE + kRing,
    B_COUNT
};

template <int D, bool FP8>
struct ChunkCfg {
    static constexpr int kThreads = FP8 ? 512 : 384;
    // Registers: softmax warps take what the others give back; the sum is the launch's total.
    static constexpr int kRegsLaunch = FP8 ? 128 : 168, kRegsSoftmax = FP8 ? (D == 64 ? 200 : 216) : 224, kRegsOther = FP8 ? (D == 64 ? 56 : 40) : 56;
    static_assert(8 * 32 * kRegsSoftmax + (kThreads - 256) * kRegsOther <= kThreads * kRegsLaunch, "register split");
    static constexpr int kBox = 128 * 128;                     // 128 rows of 128 bytes (64 values of 16 bits)
    static constexpr int kTile = 128 * D * 2;                  // 16-bit Q or V
    static constexpr int kRaw = 128 * D;                       // 8-bit K or V
    static constexpr int kKTile = FP8 ? kRaw : kTile;
    static constexpr int kKSt = FP8 ? 4 : 3, kVSt = FP8 ? 3 : 2;
    static constexpr uint32_t kTerm = FP8 ? kRaw : 0;          // from Q's first e4m3 term to its second
    // e4m3, d = 128: a raw row of 128 bytes lands where the V row's second half will be
    // (and Q's terms replace Q), so it is overwritten by its own expansion alone.
    // d = 64: beside the stages.
    static constexpr bool kInside = D == 128;
    static constexpr int kQ = 0;
    static constexpr int kK = kTile;
    static constexpr int kV = kK + kKSt * kKTile;
    static constexpr int kRawV = kV + kVSt * kTile;
    static constexpr int kRawQ = kRawV + (FP8 && !kInside ? kVSt * kRaw : 0);
    static constexpr int kOst = kRawQ + (FP8 && !kInside ? kTile : 0);   // [8 warps][32 rows][64 bytes]
    static constexpr int kMax = kOst + 8 * 2048;               // float [2][2][128]
    static constexpr int kSum = kMax + 2 * 2 * 128 * 4;        // float [2][2][128]
    static constexpr int kChain = kSum + 2 * 2 * 128 * 4;      // float [128]
    // float [kRing][128]: 1 / factor of Q rows.  As long as the units' ring: the softmax may still
    // be at the end of a short unit when Q of the one after the next is converted, but has
    // released the entry that a new unit takes.
    static constexpr int kQf = kChain + 128 * 4;
    static constexpr int kUnit = kQf + kRing * 128 * 4;        // int [kRing][kUnitInts]
    static constexpr int kFlag = kUnit + kRing * kUnitInts * 4;   // int [2][8]
    static constexpr int kBar = kFlag + 16 * 4;
    static constexpr int kMisc = kBar + B_COUNT * 8;
    // Over 114 KB, so that one CTA with all of TMEM is resident per SM.
    static constexpr int kBytes = kMisc + 64 > 120 * 1024 ? kMisc + 64 : 120 * 1024;
    static_assert(kBytes <= 227 * 1024, "shared memory of the chunk kernel");
    static constexpr int kReaders = 11 + (FP8 ? 4 : 0);        // warps that read a claimed unit
};

// A claimed piece of a unit, and its place in a ring entry.
enum { U_N, U_R, U_H, U_TOK0, U_NTOK, U_POS0, U_SEQ, U_X0, U_NS, U_FIRST, U_LO, U_HI, U_U, U_PART, U_PARTS };
struct Unit {
    int n;              // tiles of the piece; -1: no more
    int r, h;           // request, KV head
    int tok0, ntok;     // rows of q, o, lse: first, and how many tokens
    int pos0, seq;      // position of the first, tokens of the request with the new ones
    int x0;             // the piece's first tile in the unit's range
    int ns, first, lo, hi;
    int u, part, parts;
};

}  // namespace

template <int D, bool FP8, bool TWO>
__global__ void __launch_bounds__(ChunkCfg<D, FP8>::kThreads, 1)
    fm_paged_chunk_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                          const __grid_constant__ CUtensorMap tv, const PagedArgs a, const int box_keys)
{
    using C = ChunkCfg<D, FP8>;
    constexpr float kLazy = FP8 ? 8.f : 32.f;     // fp16 P stays <= 2^(8 + kLift); bf16 P may grow to 2^32
    constexpr float kUp = FP8 ? kLift : 0.f;
    constexpr int NBOX = D / 64;                  // 128-byte boxes of a 16-bit row
    constexpr int kKSt = C::kKSt, kVSt = C::kVSt;
    extern __shared__ __align__(1024) uint8_t smem[];
    float *sMax = reinterpret_cast<float *>(smem + C::kMax);
    float *sSum = reinterpret_cast<float *>(smem + C::kSum);
    volatile float *sChain = reinterpret_cast<volatile float *>(smem + C::kChain);
    volatile float *sQf = reinterpret_cast<volatile float *>(smem + C::kQf);
    volatile int *sUnit = reinterpret_cast<volatile int *>(smem + C::kUnit);
    volatile int *sFlag = reinterpret_cast<volatile int *>(smem + C::kFlag);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBar);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::kMisc);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + C::kMisc + 4);

    const int warp = warp_id(), lane = lane_id();
    grid_launch_dependents();           // the few-rows kernel takes over SM by SM
    const PagedShape &s = a.s;
    const PagedHeader *hd = reinterpret_cast<const PagedHeader *>(a.plan);
    // The same verdict in every CTA: none claims a unit of a plan that does not fit.
    if (!paged_plan_fits(hd, s) || hd->rows > a.rows || (smem_u32(smem) & 1023u) != 0) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            set_status(a.status, !paged_plan_fits(hd, s) ? FM_ERR_PLAN_MISMATCH : hd->rows > a.rows ? FM_ERR_LENGTHS : FM_ERR_UNSUPPORTED);
        return;
    }
    const int n_units = hd->units_many, splits = hd->splits_many;
    if (n_units == 0) return;
    const unsigned n_claims = (unsigned)n_units * (unsigned)splits;

    if (warp == 0 && lane == 0) {
        *abort = 0;
        mbar_init(&bars[B_Q], FP8 ? 4 : 1);
        mbar_init(&bars[B_QR], 1);
        for (int i = 0; i < kKSt; ++i) {
            mbar_init(&bars[B_KF + i], 1);
            mbar_init(&bars[B_KE + i], 1);
        }
        for (int i = 0; i < kVSt; ++i) {
            mbar_init(&bars[B_VF + i], FP8 ? 4 : 1);
            mbar_init(&bars[B_VR + i], 1);
            mbar_init(&bars[B_VE + i], 1);
        }
        for (int i = 0; i < kSBuf; ++i) {
            mbar_init(&bars[B_S + i], 1);
            mbar_init(&bars[B_P + i], 128);
            mbar_init(&bars[B_PB + i], 128);
            mbar_init(&bars[B_O + i], 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&bars[B_UF + i], 1);
            mbar_init(&bars[B_UE + i], C::kReaders);
        }
        mbar_init(&bars[B_QE], 1);
        mbar_init(&bars[B_OE], 256);
        mbar_init(&bars[B_DRAIN], 2);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    const int G = s.Hq / s.Hkv, tpt = 128 / G;      // tokens of a unit
    // a.wait_limit is for the warp that waits for K and for the drains: in the other warps' waits it
    // costs 1 to 2 % (they leave by the flag).
    constexpr long long lim = kWaitLimitCycles;

    auto read_unit = [&](int k, Unit &u) -> bool {
        const int slot = k % kRing;
        if (!warp_wait(&bars[B_UF + slot], (k / kRing) & 1, abort, a.status, lim)) return false;
        const volatile int *p = sUnit + slot * kUnitInts;
        u = Unit{p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], p[10], p[11], p[12], p[13], p[14]};
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_UE + slot]);
        return u.n >= 0;
    };
    // The same for warps that need no more than the number of tiles.
    auto read_tiles = [&](int k) -> int {
        const int slot = k % kRing;
        if (!warp_wait(&bars[B_UF + slot], (k / kRing) & 1, abort, a.status, lim)) return -1;
        const int n = sUnit[slot * kUnitInts];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_UE + slot]);
        return n;
    };
    auto key_base = [&](const Unit &u, int t) {
        const int x = u.x0 + t;
        return (x < u.ns ? x : u.first + x - u.ns) * kKeyTile;
    };
    const int nb = kKeyTile / box_keys;         // boxes of a tile; lane i looks up the page of box i
    // Number of the page that holds the lane's box of the unit's tile at kb, as the
    // table has it; not `need` when no row of the unit needs the page (it arrives as
    // zeros; any number may stand in a table, so none of them can say that).  The page as a whole
    // decides: one that is partly attended is held.
    struct Page {
        int at;
        bool need;
    };
    auto look_up = [&](const Unit &u, int kb) -> Page {
        const int j = kb + lane * box_keys;
        const int b = a.page_shift >= 0 ? j >> a.page_shift : j / s.page_size, b0 = b * s.page_size;
        if (lane >= nb || j >= u.hi || (b0 + s.page_size <= u.lo && b0 >= s.sink)) return Page{0, false};
        return Page{__ldg(a.table + (int64_t)u.r * s.max_pages + b), true};
    };
    // Starts a tile's boxes, one per lane (all lanes call).
    auto load_boxes = [&](const CUtensorMap *map, uint8_t *tile, uint64_t *bar, const Unit &u, int kb, const Page &pg) {
        int page = pg.at;
        if (!pg.need || page < 0 || page >= s.num_pages) {
            if (pg.need) set_status(a.status, FM_ERR_PAGES);
            page = s.num_pages;                 // outside the pool: zeros
        }
        const int in0 = a.page_shift >= 0 ? kb & (s.page_size - 1) : kb % s.page_size;
        if (lane >= nb) return;
        int in = in0 + lane * box_keys;         // past a page's end in the following ones
        in = a.page_shift >= 0 ? in & (s.page_size - 1) : in % s.page_size;
        if (FP8) {
            tma_load_4d(tile + lane * box_keys * D, map, bar, 0, in, u.h, page);
        } else {
#pragma unroll
            for (int half = 0; half < NBOX; ++half)
                tma_load_4d(tile + half * C::kBox + lane * box_keys * 128, map, bar, half * 64, in, u.h, page);
        }
    };
    auto k_tile = [&](int st) { return smem + C::kK + st * C::kKTile; };
    auto v_tile = [&](int st) { return smem + C::kV + st * C::kTile; };
    auto v_raw = [&](int st) { return C::kInside ? v_tile(st) + C::kBox : smem + C::kRawV + st * C::kRaw; };
    uint8_t *q_raw = smem + (FP8 && !C::kInside ? C::kRawQ : C::kQ);

    if (warp == 0) {
        warp_regs_dec<C::kRegsOther>();
        // -------------------------------------------- claims, Q and K
        const PagedEntry *list = reinterpret_cast<const PagedEntry *>(a.plan + a.L.off_many);
        const int32_t *cum = reinterpret_cast<const int32_t *>(a.plan + a.L.off_many_cum);
        unsigned *claim = reinterpret_cast<unsigned *>(a.plan + a.L.off_claim);
        int e = 0;
        // Claims the next piece into ring entry k.  The entry of the unit after the
        // one in work is filled early, so that the claim's trips to memory are over
        // when its loads are due.
        auto publish = [&](int k) -> bool {
            Unit u{};
            while (true) {
                unsigned c = 0;
                // Every CTA claims once past the end: the counter comes back to 0 by itself.
                if (lane == 0) c = atomicInc(claim, n_claims + gridDim.x - 1);
                c = __shfl_sync(0xffffffffu, c, 0);
                u.n = -1;
                if (c >= n_claims) break;
                u.u = (int)(c / (unsigned)splits);
                u.part = (int)(c - (unsigned)u.u * (unsigned)splits);
                // Claims only grow, so the entry is at or behind the last one.
                while (true) {
                    const int i = e + 1 + lane;
                    const unsigned past = __ballot_sync(0xffffffffu, i <= hd->n_many && cum[i] <= u.u);
                    e += __popc(past);
                    if (past != 0xffffffffu) break;
                }
                const PagedEntry en = list[e];
                const int nqt = (en.n + tpt - 1) / tpt, local = u.u - cum[e];
                u.r = en.r;
                u.h = local / nqt;
                const int qt = nqt - 1 - (local - u.h * nqt);     // longest first
                u.tok0 = en.tok0 + qt * tpt;
                u.ntok = min(tpt, en.n - qt * tpt);
                u.pos0 = en.ctx + qt * tpt;
                u.seq = en.ctx + en.n;
                const KeyRange kr = key_range(u.pos0, u.pos0 + u.ntok - 1, s.window, s.sink);
                u.ns = kr.ns;
                u.first = kr.first;
                u.lo = kr.lo;
                u.hi = kr.hi;
                u.parts = min(splits, kr.n);
                if (u.part >= u.parts) continue;                  // fewer tiles than pieces
                u.x0 = (int)((int64_t)kr.n * u.part / u.parts);
                u.n = (int)((int64_t)kr.n * (u.part + 1) / u.parts) - u.x0;
                break;
            }
            const int slot = k % kRing;
            if (k >= kRing && !warp_wait(&bars[B_UE + slot], ((k / kRing) - 1) & 1, abort, a.status, lim)) return false;
            if (lane == 0) {
                const int w[15] = {u.n, u.r, u.h, u.tok0, u.ntok, u.pos0, u.seq, u.x0, u.ns, u.first, u.lo, u.hi, u.u, u.part, u.parts};
#pragma unroll
                for (int i = 0; i < 15; ++i) sUnit[slot * kUnitInts + i] = w[i];
                mbar_arrive(&bars[B_UF + slot]);
            }
            __syncwarp();
            return true;
        };
        int g = 0, nq = 0;
        bool run = publish(0);
        for (int k = 0; run; ++k) {
            const volatile int *p = sUnit + (k % kRing) * kUnitInts;
            const Unit u{p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], p[10], p[11], p[12], p[13], p[14]};
            if (u.n < 0) break;
            Page page = look_up(u, key_base(u, 0));
            if (nq > 0 && !warp_wait(&bars[B_QE], (nq - 1) & 1, abort, a.status, lim)) break;
            if (lane == 0) {
                uint64_t *qb = &bars[FP8 ? B_QR : B_Q];
                mbar_arrive_expect_tx(qb, (uint32_t)(G * tpt * D * 2));
#pragma unroll
                for (int x = 0; x < NBOX; ++x) tma_load_3d(q_raw + x * C::kBox, &tq, qb, x * 64, u.h * G, u.tok0);
            }
            ++nq;
            for (int t = 0; t < u.n; ++t, ++g) {
                const int st = g % kKSt;
                const int kb = key_base(u, t);
                const Page pg = page;
                if (t + 1 < u.n) page = look_up(u, key_base(u, t + 1));
                if (g >= kKSt && !warp_wait(&bars[B_KE + st], ((g / kKSt) - 1) & 1, abort, a.status, lim)) {
                    run = false;
                    break;
                }
                uint64_t *bar = &bars[B_KF + st];
                // Wait test: one byte more than comes.  (A load left out by the first CTA alone: 0.6 %.)
                if (lane == 0) mbar_arrive_expect_tx(bar, C::kKTile + a.withhold);
                __syncwarp();
                load_boxes(&tk, k_tile(st), bar, u, kb, pg);
                __syncwarp();
            }
            if (run && !publish(k + 1)) run = false;
        }
        // After an abort: copies in flight end before the CTA leaves.
        if (lane == 0 && *abort) {
            if (nq > 0) mbar_wait_drain(&bars[FP8 ? B_QR : B_Q], (nq - 1) & 1, a.status, a.wait_limit);
            for (int i = (g > kKSt ? g - kKSt : 0); i < g; ++i)
                mbar_wait_drain(&bars[B_KF + i % kKSt], (i / kKSt) & 1, a.status, a.wait_limit);
        }
    } else if (warp == 10) {
        warp_regs_dec<C::kRegsOther>();
        // -------------------------------------------- V
        int g = 0;
        unsigned phase = 0, ragged_last = 0;     // per stage: parity of B_VR, whether it had the last load
        bool run = true;
        Unit u;
        for (int k = 0; run; ++k) {
            if (!read_unit(k, u)) break;
            Page page = look_up(u, key_base(u, 0));
            for (int t = 0; t < u.n; ++t, ++g) {
                const int st = g % kVSt;
                const int kb = key_base(u, t);
                const Page pg = page;
                if (t + 1 < u.n) page = look_up(u, key_base(u, t + 1));
                if (g >= kVSt && !warp_wait(&bars[B_VE + st], ((g / kVSt) - 1) & 1, abort, a.status, lim)) {
                    run = false;
                    break;
                }
                // A bf16 tile with the request's end in it lands on B_VR, and is
                // released once its rows behind the last token are zero.
                const bool ragged = kb + kKeyTile > u.seq;
                uint64_t *bar = &bars[(FP8 || ragged ? B_VR : B_VF) + st];
                if (lane == 0) mbar_arrive_expect_tx(bar, FP8 ? C::kRaw : C::kTile);
                __syncwarp();
                uint8_t *tile = v_tile(st);
                load_boxes(&tv, FP8 ? v_raw(st) : tile, bar, u, kb, pg);
                __syncwarp();
                const unsigned bit = 1u << st;
                ragged_last = ragged ? ragged_last | bit : ragged_last & ~bit;
                if (!FP8 && ragged) {
                    // B_VR of a stage counts its ragged tiles alone.
                    if (!warp_wait(bar, (phase & bit) ? 1 : 0, abort, a.status, lim)) {
                        ++g;
                        run = false;
                        break;
                    }
                    phase ^= bit;
                    const int r0 = u.seq - kb;
                    for (int i = r0 * 8 * NBOX + lane; i < 128 * 8 * NBOX; i += 32) {
                        const int row = i / (8 * NBOX), ch = i % (8 * NBOX);
                        st_shared_v4(tile + (ch >> 3) * C::kBox + row * 128 + (ch & 7) * 16, make_uint4(0, 0, 0, 0));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[B_VF + st]);
                }
            }
        }
        if (lane == 0 && *abort)
            for (int i = (g > kVSt ? g - kVSt : 0); i < g; ++i) {
                const int st = i % kVSt;
                if (FP8) mbar_wait_drain(&bars[B_VR + st], (i / kVSt) & 1, a.status, a.wait_limit);
                else if (!((ragged_last >> st) & 1)) mbar_wait_drain(&bars[B_VF + st], (i / kVSt) & 1, a.status, a.wait_limit);
                else if (i == g - 1 && !run) mbar_wait_drain(&bars[B_VR + st], (phase >> st) & 1, a.status, a.wait_limit);
            }
    } else if (warp == 1) {
        warp_regs_dec<C::kRegsOther>();
        // -------------------------------------------- Q K^T
        constexpr uint32_t id = FP8 ? idesc_e4m3(128, 128) : idesc_bf16(128, 128, false, false);
        auto desc = [&](uint8_t *p) {             // K-major rows of 128 bytes, or of 64 (e4m3, d = 64)
            return FP8 && D == 64 ? sdesc_sw64(smem_u32(p), 16, 512) : sdesc_sw128(smem_u32(p), 16, 1024);
        };
        const uint64_t dQ = desc(smem + C::kQ);
        int g = 0, nq = 0;
        bool run = true;
        for (int k = 0; run; ++k) {
            const int n = read_tiles(k);
            if (n < 0) break;
            if (lane == 0) {
                run = mbar_wait(&bars[B_Q], nq & 1, abort, a.status, a.wait_limit);
                for (int t = 0; run && t < n; ++t, ++g) {
                    const int st = g % kKSt, sb = g % kSBuf;
                    // The score buffer's previous tile, g - 3, has been through P V.
                    if (!mbar_wait(&bars[B_KF + st], (g / kKSt) & 1, abort, a.status, a.wait_limit) ||
                        (g >= kSBuf && !mbar_wait(&bars[B_O + sb], ((g - kSBuf) / kSBuf) & 1, abort, a.status, a.wait_limit))) {
                        run = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t dK = desc(k_tile(st));
                    if (FP8) {
#pragma unroll
                        for (int term = 0; term < 2; ++term)
#pragma unroll
                            for (int kk = 0; kk < D / 32; ++kk)   // K = 32 bytes per instruction
                                mma_ss_e4m3(tmem + sb * 128, sdesc_add(dQ, term * C::kTerm + kk * 32), sdesc_add(dK, kk * 32), id, term + kk > 0);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = (kk >> 2) * C::kBox + (kk & 3) * 32;
                            mma_ss(tmem + sb * 128, sdesc_add(dQ, off), sdesc_add(dK, off), id, kk > 0);
                        }
                    }
                    tc_commit(&bars[B_S + sb]);
                    tc_commit(&bars[B_KE + st]);
                }
                if (run) tc_commit(&bars[B_QE]);      // Q is free once these products are done
            }
            ++nq;
            run = __shfl_sync(0xffffffffu, run, 0);
        }
        if (lane == 0) {
            tc_commit(&bars[B_DRAIN]);
            mbar_wait_drain(&bars[B_DRAIN], 0, a.status, a.wait_limit);
        }
    } else if (warp == 11) {
        warp_regs_dec<C::kRegsOther>();
        // -------------------------------------------- O += P V
        constexpr uint32_t id = FP8 ? idesc_f16(128, D, true) : idesc_bf16(128, D, false, true);
        const uint32_t tO = tmem + 384;
        int g = 0, nu = 0;
        bool run = true;
        for (int k = 0; run; ++k) {
            const int n = read_tiles(k);
            if (n < 0) break;
            if (lane == 0) {
                // The unit's first product overwrites O: the last epilogue has read it.
                if (nu > 0) run = mbar_wait(&bars[B_OE], (nu - 1) & 1, abort, a.status, lim);
                for (int t = 0; run && t < n; ++t, ++g) {
                    const int st = g % kVSt, sb = g % kSBuf;
                    if (!mbar_wait(&bars[B_VF + st], (g / kVSt) & 1, abort, a.status, lim) ||
                        !mbar_wait(&bars[B_P + sb], (g / kSBuf) & 1, abort, a.status, lim)) {
                        run = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t dV = sdesc_sw128(smem_u32(smem + C::kV + st * C::kTile), C::kBox, 1024);
                    // In two halves over the keys: the softmax releases P in two.
                    auto half = [&](int h) {
#pragma unroll
                        for (int part = 0; part < (TWO ? 2 : 1); ++part)
#pragma unroll
                            for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
                                mma_ts(tO, tmem + sb * 128 + part * 64 + kk * 8, sdesc_add(dV, kk * 2048), id, t > 0 || part > 0 || kk > 0);
                    };
                    half(0);
                    if (!mbar_wait(&bars[B_PB + sb], (g / kSBuf) & 1, abort, a.status, lim)) {
                        run = false;
                        break;
                    }
                    tc_fence_after();
                    half(1);
                    tc_commit(&bars[B_O + sb]);
                    tc_commit(&bars[B_VE + st]);
                }
            }
            ++nu;
            run = __shfl_sync(0xffffffffu, run, 0);
        }
        if (lane == 0) {
            tc_commit(&bars[B_DRAIN]);
            mbar_wait_drain(&bars[B_DRAIN], 0, a.status, a.wait_limit);
        }
    } else if (FP8 && warp >= 12) {
        warp_regs_dec<C::kRegsOther>();
        // -------------------------------------------- conversions
        // Four warps, each every fourth group of rows.  A row is read by d / 8 lanes,
        // 8 values each: of V they become one 16-byte chunk of the swizzled operand (no
        // bank conflict either way), of Q eight bytes of either term.
        const int mate = warp & 3;
        constexpr int LPR = D / 8, RPI = 32 / LPR;        // lanes per row, rows per warp step
        constexpr int BATCH = 8;                          // steps whose loads are in flight together
        const int l = lane % LPR, r_in = lane / LPR;
        int g = 0, nq = 0;
        bool run = true;
        Unit u;
        for (int k = 0; run; ++k) {
            if (!read_unit(k, u)) break;
            if (!warp_wait(&bars[B_QR], nq & 1, abort, a.status, lim)) break;
            // Two steps' rows at a time: their chains of loads, maxima and roundings overlap.
            constexpr int QB = 2;
            for (int i0 = mate * QB; i0 < 128 / RPI; i0 += 4 * QB) {
                uint4 x[QB];
                float amax[QB];
#pragma unroll
                for (int b = 0; b < QB; ++b) {
                    const int row = (i0 + b) * RPI + r_in;
                    x[b] = *reinterpret_cast<const uint4 *>(q_raw + (l >> 3) * C::kBox + row * 128 + (((l & 7) ^ (row & 7)) << 4));
                }
#pragma unroll
                for (int b = 0; b < QB; ++b) {
                    const uint32_t w[4] = {x[b].x, x[b].y, x[b].z, x[b].w};
                    amax[b] = 0.f;
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        amax[b] = fmax3(amax[b], fabsf(__uint_as_float(w[y] << 16)), fabsf(__uint_as_float(w[y] & 0xffff0000u)));
                }
#pragma unroll
                for (int y = 1; y < LPR; y <<= 1)
#pragma unroll
                    for (int b = 0; b < QB; ++b) amax[b] = fmaxf(amax[b], __shfl_xor_sync(0xffffffffu, amax[b], y));   // the rows' lanes have read them
#pragma unroll
                for (int b = 0; b < QB; ++b) {
                    const int row = (i0 + b) * RPI + r_in;
                    const uint32_t w[4] = {x[b].x, x[b].y, x[b].z, x[b].w};
                    // An infinite element makes the row NaN (it would saturate).
                    const float f = amax[b] == INFINITY ? __uint_as_float(0x7fc00000u) : row_factor(amax[b], 7);
                    uint32_t hi[2] = {0u, 0u}, lw[2] = {0u, 0u};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const float q0 = __uint_as_float(w[y] << 16) * f, q1 = __uint_as_float(w[y] & 0xffff0000u) * f;
                        const uint32_t h = pack_e4m3x2(q0, q1);
                        float h0, h1;
                        unpack_f16x2(f16x2_of_e4m3(h), h0, h1);
                        hi[y >> 1] |= h << (16 * (y & 1));
                        lw[y >> 1] |= pack_e4m3x2(q0 - h0, q1 - h1) << (16 * (y & 1));
                    }
                    const uint32_t at = D == 128 ? row * 128 + (((l >> 1) ^ (row & 7)) << 4) : row * 64 + (((l >> 1) ^ ((row >> 1) & 3)) << 4);
                    uint8_t *p = smem + C::kQ + at + (l & 1) * 8;
                    *reinterpret_cast<uint2 *>(p) = make_uint2(hi[0], hi[1]);
                    *reinterpret_cast<uint2 *>(p + C::kTerm) = make_uint2(lw[0], lw[1]);
                    if (l == 0) sQf[(nq % kRing) * 128 + row] = 1.f / f;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_Q]);
            ++nq;
            for (int t = 0; t < u.n; ++t, ++g) {
                const int st = g % kVSt;
                if (!warp_wait(&bars[B_VR + st], (g / kVSt) & 1, abort, a.status, lim)) {
                    run = false;
                    break;
                }
                const uint8_t *raw = v_raw(st);
                uint8_t *tile = v_tile(st);
                const int rows = u.seq - key_base(u, t);  // V behind the last token: zeros
                for (int i0 = mate * BATCH; i0 < 128 / RPI; i0 += 4 * BATCH) {
                    uint2 x[BATCH];
#pragma unroll
                    for (int b = 0; b < BATCH; ++b) x[b] = *reinterpret_cast<const uint2 *>(raw + ((i0 + b) * RPI + r_in) * D + l * 8);
                    __syncwarp();                         // the rows' lanes have read them
#pragma unroll
                    for (int b = 0; b < BATCH; ++b) {
                        const int row = (i0 + b) * RPI + r_in;
                        if (row >= rows) x[b] = make_uint2(0, 0);
                        st_shared_v4(tile + (l >> 3) * C::kBox + row * 128 + (((l & 7) ^ (row & 7)) << 4),
                                     make_uint4(f16x2_of_e4m3(x[b].x), f16x2_of_e4m3(x[b].x >> 16), f16x2_of_e4m3(x[b].y),
                                                f16x2_of_e4m3(x[b].y >> 16)));
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_VF + st]);
            }
        }
    } else if (warp >= 10) {
        warp_regs_dec<C::kRegsOther>();     // idle warps too: the softmax warps' increase waits for every share
    } else {
        warp_regs_inc<C::kRegsSoftmax>();
        // -------------------------------------------- softmax
        const int w = warp < 6 ? 0 : 1;                   // warpgroup: the tiles g with g & 1 == w
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;              // row of the unit = TMEM lane
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tO = tmem + 384;
        constexpr int OC = D / 2;                         // output columns that this warpgroup stores
        const float scale = a.scale_log2 * (FP8 ? *a.k_descale : 1.f), vds = FP8 ? *a.v_descale : 1.f;
        const int tk = row / G, gh = row - tk * G;        // token and head of the row
        // False for the whole warp once a wait gave up: it still reaches every
        // named barrier, so that the other warpgroup is never left waiting.
        bool live = true;
        auto wait_pv = [&](int k) {
            live = live && warp_wait(&bars[B_O + k % kSBuf], (k / kSBuf) & 1, abort, a.status, lim);
        };
        int g = 0, nu = 0;
        for (int k = 0;; ++k) {
            // The unit's numbers stay in the ring (a broadcast load each where they
            // are used, instead of registers); the entry is released at the unit's end.
            const volatile int *un = sUnit + (k % kRing) * kUnitInts;
            const bool here = warp_wait(&bars[B_UF + k % kRing], (k / kRing) & 1, abort, a.status, lim);
            const int n = here ? un[U_N] : -1;
            if (lane == 0) sFlag[(k & 1) * 8 + (warp - 2)] = n >= 0 ? 1 : 0;
            named_bar_sync(1, 256);
            int all = sFlag[(k & 1) * 8];
#pragma unroll
            for (int q = 1; q < 8; ++q) all &= sFlag[(k & 1) * 8 + q];
            if (!all) break;
            const int pos = un[U_POS0] + tk;
            const int lo = (s.window > 0 && pos >= s.window) ? pos - s.window + 1 : 0;
            float m = -INFINITY, l = 0.f, sl2 = scale;
            const int g0 = g;
            for (int t = (w - g0) & 1; t < n; t += 2) {
                const int gt = g0 + t, sb = gt % kSBuf;
                const int x = un[U_X0] + t, ns = un[U_NS];
                const int kb = (x < ns ? x : un[U_FIRST] + x - ns) * kKeyTile;
                // Free of the mask: behind no row's position, before no row's window.
                const bool full = kb + kKeyTile - 1 <= un[U_POS0] &&
                                  (s.window == 0 || kb > un[U_POS0] + un[U_NTOK] - 1 - s.window || kb + kKeyTile <= s.sink);
                const uint32_t tS = tmem + sb * 128;
                live = live && warp_wait(&bars[B_S + sb], (gt / kSBuf) & 1, abort, a.status, lim);
                uint32_t sv[128];
                float mx = -INFINITY;
                if (live) {
                    tc_fence_after();
                    if (FP8) sl2 = scale * sQf[(nu % kRing) * 128 + row];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        tmem_ld32(tS + lane_off + c * 32, reinterpret_cast<uint32_t (&)[32]>(sv[c * 32]));
                    tmem_ld_wait();
                    tmem_reg_fence(sv);
                    if (!full) {
                        // The row's keys of the tile as 128 bits.
                        uint32_t keep[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int b0 = kb + 32 * c;
                            keep[c] = row_bits32(lo - b0, pos + 1 - b0) | row_bits32(0, min(s.sink, pos + 1) - b0);
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (__any_sync(0xffffffffu, keep[c] != 0xffffffffu)) {    // 32 keys that every row keeps take no select
#pragma unroll
                                for (int i = 0; i < 32; ++i) sv[32 * c + i] = (keep[c] & (1u << i)) ? sv[32 * c + i] : 0xff800000u;
                            }
                    }
                    float mx4[4] = {__uint_as_float(sv[0]), __uint_as_float(sv[1]), __uint_as_float(sv[2]), __uint_as_float(sv[3])};
#pragma unroll
                    for (int i = 0; i < 62; ++i)
                        mx4[i & 3] = fmax3(mx4[i & 3], __uint_as_float(sv[4 + 2 * i]), __uint_as_float(sv[5 + 2 * i]));
                    mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
                }
                // The maximum in force passes from the owner of tile t - 1 to t's and on.
                float m_prev = -INFINITY;
                if (t > 0) {
                    named_bar_sync(2 + (1 - w), 256);
                    m_prev = sChain[row];
                }
                const float m_new = (mx > m_prev + kLazy) ? mx : m_prev;
                if (t + 1 < n) {
                    sChain[row] = m_new;
                    named_bar_arrive(2 + w, 256);
                }
                if (!live) continue;
                if (__any_sync(0xffffffffu, t > 0 && m_new != m_prev)) {
                    const float alpha = (m_new != m_prev) ? ex2(m_prev - m_new) : 1.f;
                    wait_pv(gt - 1);
                    if (!live) continue;
                    tc_fence_after();
#pragma unroll
                    for (int cc = 0; cc < D / 16; ++cc) {
                        uint32_t ov[16];
                        tmem_ld16(tO + lane_off + cc * 16, ov);
                        tmem_ld_wait();
                        tmem_reg_fence(ov);
#pragma unroll
                        for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                        tmem_st16(tO + lane_off + cc * 16, ov);
                    }
                }
                const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
                const uint64_t sc2 = f2_pack(sl2, sl2), nm2 = f2_pack(kUp - m_use, kUp - m_use);
                uint64_t sum2 = f2_pack(0.f, 0.f);
#pragma unroll
                for (int hh = 0; hh < 4; ++hh) {
                    uint32_t hi[16], lw[16];
#pragma unroll
                    for (int cc = 0; cc < 16; ++cc) {
                        float x0, x1;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[hh * 32 + 2 * cc]), __uint_as_float(sv[hh * 32 + 2 * cc + 1])), sc2, nm2),
                                  x0, x1);
                        const float p0 = ex2(x0), p1 = ex2(x1);
                        sum2 = f2_add(sum2, f2_pack(p0, p1));
                        hi[cc] = FP8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
                        if (TWO) {
                            if (FP8) {
                                float u0, u1;
                                unpack_f16x2(hi[cc], u0, u1);
                                lw[cc] = pack_f16x2(p0 - u0, p1 - u1);
                            } else {
                                lw[cc] = pack_bf16x2(p0 - __uint_as_float(hi[cc] << 16), p1 - __uint_as_float(hi[cc] & 0xffff0000u));
                            }
                        }
                    }
                    tmem_st16(tS + lane_off + hh * 16, hi);
                    if (TWO) tmem_st16(tS + lane_off + 64 + hh * 16, lw);
                    if (hh == 1) {
                        tmem_st_wait();
                        tc_fence_before();
                        mbar_arrive(&bars[B_P + sb]);
                    }
                }
                float s0, s1;
                f2_unpack(sum2, s0, s1);
                l = (m == m_new ? l : l * ex2(m - m_new)) + (s0 + s1);
                m = m_new;
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bars[B_PB + sb]);
            }
            g = g0 + n;
            // ---------------------------------------- epilogue
            const int su = nu & 1;
            sSum[(su * 2 + w) * 128 + row] = l;
            sMax[(su * 2 + w) * 128 + row] = m;
            named_bar_sync(1, 256);
            wait_pv(g - 1);
            uint32_t ov[OC];
            float lt = 0.f, mf = -INFINITY;
            const bool valid = tk < un[U_NTOK] && tk < tpt;
            if (live) {
                tc_fence_after();
                const float m0 = sMax[(su * 2) * 128 + row], m1 = sMax[(su * 2 + 1) * 128 + row];
                const float l0 = sSum[(su * 2) * 128 + row], l1 = sSum[(su * 2 + 1) * 128 + row];
                mf = fmaxf(m0, m1);
                lt = (l0 != 0.f ? l0 * ex2(m0 - mf) : 0.f) + (l1 != 0.f ? l1 * ex2(m1 - mf) : 0.f);
                mf -= kUp;
#pragma unroll
                for (int cc = 0; cc < OC / 32; ++cc)
                    tmem_ld32(tO + lane_off + w * OC + cc * 32, reinterpret_cast<uint32_t (&)[32]>(ov[cc * 32]));
                tmem_ld_wait();
                tmem_reg_fence(ov);
                tc_fence_before();
            }
            mbar_arrive(&bars[B_OE]);       // O is free for the next unit's first product (after an abort nothing reads it)
            const int parts = un[U_PARTS];
            if (parts > 1) {
                // Partial sums of the piece, for the few-rows kernel behind this one to
                // add up: column-major in groups of four, so that the lanes (rows)
                // write next to one another.
                float4 *po = reinterpret_cast<float4 *>(a.plan + a.L.off_many_o);
                float *pml = reinterpret_cast<float *>(a.plan + a.L.off_many_ml);
                if (live && valid) {
                    const int64_t slot = (int64_t)un[U_U] * splits + un[U_PART];
#pragma unroll
                    for (int c4 = 0; c4 < OC / 4; ++c4)
                        __stcg(po + (slot * (D / 4) + w * (OC / 4) + c4) * 128 + row,
                               make_float4(__uint_as_float(ov[4 * c4]), __uint_as_float(ov[4 * c4 + 1]), __uint_as_float(ov[4 * c4 + 2]),
                                           __uint_as_float(ov[4 * c4 + 3])));
                    if (w == 0) {
                        __stcg(pml + slot * 256 + row, mf);
                        __stcg(pml + slot * 256 + 128 + row, lt);
                    }
                }
            } else if (live) {
                const float inv = lt != 0.f ? vds / lt : 0.f;
                // Through shared memory, 32 rows of 64 bytes at a time, so that four
                // lanes write a row's 64 bytes; rows behind the unit's tokens are left out.
                uint8_t *stg = smem + C::kOst + (warp - 2) * 2048;
                int64_t at[4];
                unsigned mine4 = 0;
                const int64_t at0 = (int64_t)un[U_TOK0] * s.Hq + un[U_H] * G;
#pragma unroll
                for (int i = 0; i < 4; ++i) {       // row i * 8 + lane / 4 of the warp: its lane knows the place
                    at[i] = (at0 + __shfl_sync(0xffffffffu, tk * s.Hq + gh, i * 8 + (lane >> 2))) * D + w * OC;
                    mine4 |= __shfl_sync(0xffffffffu, valid ? 1 : 0, i * 8 + (lane >> 2)) ? 1u << i : 0u;
                }
                auto stage = [&](const uint4 (&pk)[4], int col_bytes, int esz) {
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 4; ++q) st_shared_v4(stg + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4), pk[q]);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int x = i * 8 + (lane >> 2), q = lane & 3;
                        const uint4 v = *reinterpret_cast<const uint4 *>(stg + x * 64 + ((q ^ ((x >> 1) & 3)) << 4));
                        if ((mine4 >> i) & 1)
                            *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(a.o) + at[i] * esz + col_bytes + q * 16) = v;
                    }
                };
                if (a.o_f32) {
#pragma unroll
                    for (int c = 0; c < OC / 16; ++c) {
                        uint4 pk[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t *oc = ov + c * 16 + 4 * q;
                            pk[q] = make_uint4(__float_as_uint(__uint_as_float(oc[0]) * inv), __float_as_uint(__uint_as_float(oc[1]) * inv),
                                               __float_as_uint(__uint_as_float(oc[2]) * inv), __float_as_uint(__uint_as_float(oc[3]) * inv));
                        }
                        stage(pk, c * 64, 4);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < OC / 32; ++c) {
                        uint4 pk[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t *oc = ov + c * 32 + 8 * q;
                            pk[q] = make_uint4(pack_bf16x2(__uint_as_float(oc[0]) * inv, __uint_as_float(oc[1]) * inv),
                                               pack_bf16x2(__uint_as_float(oc[2]) * inv, __uint_as_float(oc[3]) * inv),
                                               pack_bf16x2(__uint_as_float(oc[4]) * inv, __uint_as_float(oc[5]) * inv),
                                               pack_bf16x2(__uint_as_float(oc[6]) * inv, __uint_as_float(oc[7]) * inv));
                        }
                        stage(pk, c * 64, 2);
                    }
                }
                if (w == 0 && valid) a.lse[(int64_t)(un[U_TOK0] + tk) * s.Hq + un[U_H] * G + gh] = row_lse(mf, lt);
            }
            ++nu;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_UE + k % kRing]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace fm

using namespace fm;

namespace {

template <int D, bool FP8, bool TWO>
fm_status launch(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const PagedArgs &a, int box_keys,
                 cudaStream_t stream)
{
    using C = ChunkCfg<D, FP8>;
    static std::atomic<uint8_t> done[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FM_ERR_CUDA;
    if (!done[dev].load(std::memory_order_acquire)) {
        // The register split adds up to the launch's registers only if the
        // kernel was compiled to that many per thread.
        cudaFuncAttributes fa{};
        if (cudaFuncGetAttributes(&fa, fm_paged_chunk_kernel<D, FP8, TWO>) != cudaSuccess || fa.numRegs != C::kRegsLaunch)
            return FM_ERR_CUDA;
        if (cudaFuncSetAttribute(fm_paged_chunk_kernel<D, FP8, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes) !=
            cudaSuccess)
            return FM_ERR_CUDA;
        done[dev].store(1, std::memory_order_release);
    }
    ProfScope ps(kKPagedChunk, stream);
    fm_paged_chunk_kernel<D, FP8, TWO><<<kPagedCtas, C::kThreads, C::kBytes, stream>>>(tq, tk, tv, a, box_keys);
    return cudaPeekAtLastError() == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

template <int D>
fm_status launch_as(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const PagedArgs &a, int box_keys, bool e4m3,
                    cudaStream_t stream)
{
    if (e4m3)
        return a.o_f32 ? launch<D, true, true>(tq, tk, tv, a, box_keys, stream) : launch<D, true, false>(tq, tk, tv, a, box_keys, stream);
    return a.o_f32 ? launch<D, false, true>(tq, tk, tv, a, box_keys, stream) : launch<D, false, false>(tq, tk, tv, a, box_keys, stream);
}

}  // namespace

fm_status fm_paged_chunk_launch(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const PagedArgs &a, int box_keys,
                                bool e4m3, cudaStream_t stream)
{
    return a.s.d == 128 ? launch_as<128>(tq, tk, tv, a, box_keys, e4m3, stream) : launch_as<64>(tq, tk, tv, a, box_keys, e4m3, stream);
}
