// Attention of few new tokens over a paged cache (decoding steps): requests
// whose new tokens times the query heads per KV head make at most kFewRows
// rows.
//
//   o_row = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale q_row . k_j
//
// over the keys j that the row attends, one pass over K and V with the running
// maximum and sum per row.  Bound by reading K and V once from HBM: at 8 rows
// the work is 8 FLOPs per byte, so the products run on warp-level matrix
// instructions straight from registers (a 16-row operand; a 128-row tcgen05
// operand would be padding), and everything is arranged around the loads.
//
// Work: the key tiles (128 keys) of every (request, KV head) in a row, cut
// into equal shares for the persistent CTAs, so ragged lengths and few
// requests balance alike.  A unit (request, KV head) that crosses a border is
// finished by the CTA that arrives last at it, which adds the partial results
// in the order of the CTAs: the result does not depend on who is last.
//
// Four warps load whole tiles by TMA, boxes of up to 128 consecutive keys of a page,
// through a ring of 192 KB; eight compute, each on 16 or 32 keys of a tile with a
// running maximum and sum of its own, so that they meet only when a unit ends.  (With
// every warp loading its own 16 keys the loads' bookkeeping and the boxes' start, about
// 130 cycles each, bounded it: 96 ragged requests of up to 16K tokens 0.320 ms, now
// 0.287, 6.88 TB/s; per-thread copies before that 0.374.)  Fragment
// layouts: the head-dim order of the score product is free as long as Q and K agree, the
// order of keys as long as P and V do, and the order of output columns altogether, so K
// and V fragments are read with 16-byte shared loads in an order that meets no bank
// conflict under TMA's swizzle, and V is transposed by byte permutes of two keys'
// registers.  e4m3 caches halve the bytes but not the products: 64 requests of one or two
// tokens 0.123 ms, 5.9 TB/s, where the loads alone take 0.117 and the products alone 0.123.  A
// unit's end is what stands between the two (the ring of loads fills up meanwhile): it is
// one exchange between the warps, with the next unit's Q on its way (0.138 before).
// For 8 rows, Q K in e4m3 instructions (half the products) was no faster, for more rows
// slower; so were twelve computing warps.
//
// P enters the second product as two 16-bit terms (hi + lo, about 16
// significant bits), so that the rounding of a 16-bit output is the only one
// that counts, and as three when the output is fp32.  With at most 8 rows the low
// terms use the 8 idle rows of the 16-row operand, and are free.  e4m3 caches
// take P as fp16 (11 bits a term; one term for 16-bit outputs of more rows), lifted by
// 2^kLift: e4m3 values are exact in fp16, and so is Q after a power-of-two factor per row
// that puts its largest element in [2^14, 2^15).
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "fm_paged.h"
#include "fm_ptx.cuh"

namespace fm {
namespace {

constexpr float kBand = 8.f;   // lazy rescale: P stays <= 2^8 (2^(8 + kLift) over e4m3), sums are rescaled when a maximum grows by more

constexpr int kWarps = 8;              // that compute; a warpgroup behind them has the one that loads
constexpr int kThreads = (kWarps + 4) * 32;
// Registers: the loading warpgroup gives its share to the others.
constexpr int kLaunchRegs = 168, kRegsCompute = 232, kRegsLoad = 40;
static_assert(kWarps * 32 * kRegsCompute + 128 * kRegsLoad <= kThreads * kLaunchRegs, "register split");
constexpr int kSumBar = 1;             // named barrier of the computing warps

template <int D, bool FP8, int ROWS>
struct DecodeCfg {
    static constexpr int kRow = D * (FP8 ? 1 : 2);          // bytes of a key's row
    // 16-key groups that a warp takes at a time.  Two where a row has 128 bytes or
    // fewer and the registers allow it: more independent products per step; every
    // other tile then belongs to one half of the warps.
    static constexpr int kSub = (kRow == 256 || ROWS == 32) ? 1 : 2;
    static constexpr int kStage = 2 * kKeyTile * kRow;      // a tile: K boxes, then V boxes
    static constexpr int kStages = 192 * 1024 / kStage < 8 ? 192 * 1024 / kStage : 8;
    static constexpr int kPieces = ROWS == 8 && D == 64 ? 4 : 8;     // that a warp leaves at a time when a unit ends
    static constexpr int kRed = kStages * kStage;           // float4 [warps][pieces][32 lanes]; Q of 32 rows between units
    static constexpr int kMl = kRed + kWarps * kPieces * 32 * 16;   // float [warps][2][kFewRows]
    static constexpr int kBar = kMl + kWarps * 2 * kFewRows * 4;    // mbarrier [2][stages]: loaded, read
    static constexpr int kMisc = kBar + 2 * kStages * 8;
    static constexpr int kBytes = kMisc + 32;                       // int [8]: flags, abort, a split unit's first CTA and their number
    static_assert(kBytes <= 227 * 1024, "shared memory of the few-rows kernel");
    static_assert(kPagedCtas * ROWS * 4 <= kMl - kRed, "weights of a split unit's parts");
    static_assert(ROWS != 32 || kFewRows * (D * 2 + 4) <= kMl - kRed, "Q of 32 rows");
};

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// c (16 x 8 fp32) += a (16 x 16) b (16 x 8)
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    if (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Order of keys and columns.  Column n of the score fragment is key
// key_of(n) of its group of eight, and column n of the output fragment is piece
// piece_of(n) of the head dim: the lanes of a shared-load phase then hit eight
// different bank groups under the 128-byte swizzle (chunk ^ row & 7).  Rows of 64
// bytes (e4m3, d = 64; 64-byte swizzle) keep V free of conflicts and K at two ways.
template <bool NARROW>
__host__ __device__ constexpr int key_of(int n)
{
    return NARROW ? ((n >> 1) & 1) | ((n >> 2) << 2) | ((n & 1) << 1) : (n >> 1) | ((n & 1) << 2);
}
template <bool NARROW>
__host__ __device__ constexpr int piece_of(int n)
{
    return NARROW ? n : (n >> 1) | ((n & 1) << 2);
}
// Byte offset of 16-byte chunk ch of key row `row` (0-15) in a 16-row box.
template <bool NARROW>
__device__ __forceinline__ uint32_t chunk_at(int row, int ch)
{
    return NARROW ? (uint32_t)(row * 64 + ((ch ^ ((row >> 1) & 3)) << 4)) : (uint32_t)(row * 128 + ((ch ^ (row & 7)) << 4));
}

// A walk over the CTA's share of the list.
struct Cursor {
    int e, h, x;          // entry, KV head, tile of the entry's range
    PagedEntry ent;
    int64_t cum;          // tiles before the entry
    KeyRange kr;
};

}  // namespace

// Adds up the parts of the many-rows kernel's split units, in their order.  A warp
// takes 32 rows (a lane each) and eight columns of a unit: the parts' loads of a
// batch are all started before the first is used.  (Called by the computing warps.)
template <int D>
__device__ __forceinline__ void add_parts(const PagedArgs &a, const PagedHeader *hd, float vds)
{
    constexpr int COLS = D / 8, BP = 8;
    const PagedShape &s = a.s;
    const PagedEntry *list = reinterpret_cast<const PagedEntry *>(a.plan + a.L.off_many);
    const int32_t *cum = reinterpret_cast<const int32_t *>(a.plan + a.L.off_many_cum);
    const float *ml = reinterpret_cast<const float *>(a.plan + a.L.off_many_ml);
    const float4 *po = reinterpret_cast<const float4 *>(a.plan + a.L.off_many_o);
    const int G = s.Hq / s.Hkv, tpt = 128 / G, splits = hd->splits_many;
    const int items = hd->units_many * 4 * COLS;
    for (int it = blockIdx.x * kWarps + warp_id(); it < items; it += gridDim.x * kWarps) {
        const int u = it / (4 * COLS), rest = it - u * (4 * COLS), row = rest / COLS * 32 + lane_id(), c8 = rest % COLS;
        int e = 0;
        while (e + 1 < hd->n_many && cum[e + 1] <= u) ++e;
        const PagedEntry en = list[e];
        const int nqt = (en.n + tpt - 1) / tpt, local = u - cum[e], h = local / nqt, qt = nqt - 1 - (local - h * nqt);
        const int ntok = min(tpt, en.n - qt * tpt), tk = row / G;
        const int parts = min(splits, key_range(en.ctx + qt * tpt, en.ctx + qt * tpt + ntok - 1, s.window, s.sink).n);
        if (parts == 1 || tk >= ntok) continue;
        const float *m = ml + (int64_t)u * splits * 256 + row;
        float mx = -INFINITY, sum = 0.f;
        for (int p0 = 0; p0 < parts; p0 += BP) {
            float y[BP], z[BP], top = mx;
#pragma unroll
            for (int i = 0; i < BP; ++i) {
                y[i] = ld_cg(m + min(p0 + i, parts - 1) * 256);
                z[i] = p0 + i < parts ? ld_cg(m + (p0 + i) * 256 + 128) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < BP; ++i) top = fmaxf(top, y[i]);
            const float mu = top == -INFINITY ? 0.f : top;
            sum *= ex2(mx - mu);
#pragma unroll
            for (int i = 0; i < BP; ++i) sum += ex2(y[i] - mu) * z[i];
            mx = top;
        }
        const float mu = mx == -INFINITY ? 0.f : mx, inv = sum != 0.f ? vds / sum : 0.f;
        const float4 *pc = po + ((int64_t)u * splits * (D / 4) + c8 * 2) * 128 + row;
        float x[8] = {};
        for (int p0 = 0; p0 < parts; p0 += BP) {
            float y[BP];
            float4 v[BP][2];
#pragma unroll
            for (int i = 0; i < BP; ++i) {
                const int p = min(p0 + i, parts - 1);
                y[i] = ld_cg(m + p * 256);
                v[i][0] = ld_cg(pc + (int64_t)p * (D / 4) * 128);
                v[i][1] = ld_cg(pc + (int64_t)p * (D / 4) * 128 + 128);
            }
#pragma unroll
            for (int i = 0; i < BP; ++i) {
                const float w = p0 + i < parts ? ex2(y[i] - mu) : 0.f;
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    x[4 * z] += w * v[i][z].x;
                    x[4 * z + 1] += w * v[i][z].y;
                    x[4 * z + 2] += w * v[i][z].z;
                    x[4 * z + 3] += w * v[i][z].w;
                }
            }
        }
        const int64_t at = (int64_t)(en.tok0 + qt * tpt + tk) * s.Hq + h * G + (row - tk * G);
        if (c8 == 0) a.lse[at] = row_lse(mx, sum);
        if (a.o_f32) {
            float4 *o = reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.o) + at * D + c8 * 8);
            o[0] = make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
            o[1] = make_float4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
        } else {
            *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(a.o) + at * D + c8 * 8) =
                make_uint4(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv), pack_bf16x2(x[4] * inv, x[5] * inv),
                           pack_bf16x2(x[6] * inv, x[7] * inv));
        }
    }
}

// A CTA's share.  ROWS: 8, 16 or 32 rows of a unit at most; TERMS: 16-bit terms of P.
template <int D, bool FP8, int ROWS, int TERMS>
__device__ __forceinline__ void walk_share(const CUtensorMap &tk, const CUtensorMap &tv, const PagedArgs &a, const int box_keys,
                                           const PagedHeader *hd, const PagedStart &start, uint8_t *smem)
{
    using C = DecodeCfg<D, FP8, ROWS>;
    constexpr int ST = C::kStages, SUB = C::kSub;
    constexpr int WPT = kWarps / SUB;       // warps of a tile
    constexpr bool NARROW = C::kRow == 64;
    constexpr int MT = ROWS == 32 ? 2 : 1;  // 16-row blocks
    constexpr int NR = ROWS == 8 ? 1 : 2;   // rows of a block per thread
    constexpr int KS = D / 16;              // score product: k-steps
    constexpr int NT = D / 8;               // output product: 8-column tiles
    constexpr int NP = NT / 8;              // groups of 8 tiles
    constexpr float kUp = FP8 ? kLift : 0.f;
    const int warp = warp_id(), lane = lane_id();
    const int g = lane >> 2, c = lane & 3;
    const int kg = key_of<NARROW>(g), ka = key_of<NARROW>(2 * c), kb2 = key_of<NARROW>(2 * c + 1);
    const PagedShape &s = a.s;
    const int ctas = hd->ctas_few;
    const int64_t W = hd->tiles_few;
    int left = start.count;                 // tiles to compute

    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBar), *empty = full + ST;
    volatile int *abort = reinterpret_cast<volatile int *>(smem + C::kMisc + 4);
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 4);         // the loading warps
            mbar_init(&empty[i], WPT);
        }
        *abort = 0;
        fence_barrier_init();
    }
    __syncthreads();

    const PagedEntry *list = reinterpret_cast<const PagedEntry *>(a.plan + a.L.off_few);
    const int64_t *cum = reinterpret_cast<const int64_t *>(a.plan + a.L.off_few_cum);
    const int G = s.Hq / s.Hkv;
    auto enter = [&](Cursor &u) {
        const int4 v = *reinterpret_cast<const int4 *>(list + u.e);
        u.ent = PagedEntry{v.x, v.y, v.z, v.w};
        u.cum = cum[u.e];
        u.kr = key_range(v.w, v.w + v.z - 1, s.window, s.sink);
    };
    // Next tile of the walk; true when it begins another unit.
    auto advance = [&](Cursor &u, bool more) -> bool {
        if (++u.x < u.kr.n) return false;
        u.x = 0;
        if (++u.h == s.Hkv) {
            u.h = 0;
            ++u.e;
            if (more) enter(u);
        }
        return true;
    };

    Cursor cu{start.e, start.h, start.x, start.ent, start.cum, key_range(start.ent.ctx, start.ent.ctx + start.ent.n - 1, s.window, s.sink)};
    // A tile's boxes of box_keys consecutive keys of one page: [128-byte box of a
    // row][key][128 bytes] each.  Some: a row attends one of the n keys from j on.
    const int n_box = kKeyTile / box_keys;
    auto some = [&](int j, int n) { return j < cu.kr.hi && !(j + n <= cu.kr.lo && j >= s.sink); };

    if (warp >= kWarps) {
        warp_regs_dec<kRegsLoad>();
        // ------------------------------------------------ loads
        // Warps 0 and 1 of the group load the even and the odd boxes of K, 2 and 3
        // those of V, a lane each with its own page, looked up a tile ahead.  (One
        // warp alone starts its boxes one after the other, about 130 cycles each:
        // 16-token pages of e4m3, 0.160 ms where four warps need 0.136.)
        const int part = warp - kWarps, bx = (part & 1) + 2 * lane;
        const bool mine = bx < n_box;
        const CUtensorMap *map = part < 2 ? &tk : &tv;
        const uint32_t box_bytes = (uint32_t)box_keys * C::kRow;
        // Page of the lane's box of the tile at the cursor; *need: some row attends one of its keys.
        // (Any number may stand in a table, so none of them can mark a box that is not needed.)
        auto look_up = [&](bool *need) -> int {
            const int j = cu.kr.tile(cu.x) * kKeyTile + bx * box_keys;
            *need = mine && some(j, box_keys);
            if (!*need) return 0;
            return __ldg(a.table + (int64_t)cu.ent.r * s.max_pages + (a.page_shift >= 0 ? j >> a.page_shift : j / s.page_size));
        };
        const int withheld = a.withhold && blockIdx.x == 0 ? 1 : -1;      // test hook
        bool next_need;
        int next = look_up(&next_need), t = 0;
        for (; t < left; ++t) {
            const int st = t % ST;
            int page = next;
            const bool need = next_need;
            const int j = cu.kr.tile(cu.x) * kKeyTile + bx * box_keys, h = cu.h;
            advance(cu, t + 1 < left);
            if (t + 1 < left) next = look_up(&next_need);
            if (t >= ST && !warp_wait(&empty[st], ((t / ST) - 1) & 1, abort, a.status, a.wait_limit)) break;
            if (t == withheld) continue;
            const unsigned used = __ballot_sync(0xffffffffu, need);
            if (lane == 0) {
                if (used) mbar_arrive_expect_tx(&full[st], __popc(used) * box_bytes);
                else mbar_arrive(&full[st]);
            }
            __syncwarp();
            if (need) {
                if (page < 0 || page >= s.num_pages) {
                    set_status(a.status, FM_ERR_PAGES);
                    page = s.num_pages;         // outside the pool: arrives as zeros
                }
                const int in = a.page_shift >= 0 ? j & (s.page_size - 1) : j % s.page_size;
                tma_load_5d(smem + st * C::kStage + ((part >> 1) * n_box + bx) * box_bytes, map, &full[st], 0, in, 0, h, page);
            }
        }
        // After a wait that ran out: the copies end before the CTA leaves.
        if (*abort && lane == 0)
            for (int i = max(t - ST, 0); i < t; ++i) mbar_wait_drain(&full[i % ST], (i / ST) & 1, a.status, a.wait_limit);
        grid_wait_before();
        return;
    }
    warp_regs_inc<kRegsCompute>();
    // This warp's keys of a tile, 16 SUB of them, and where they lie in a stage.
    const int turn = warp / WPT;            // with SUB = 2: takes the even or the odd tiles of the walk
    const int key0 = (warp % WPT) * (16 * SUB);
    const uint32_t half_box = (uint32_t)box_keys * 128;     // from a row's first 128 bytes to its second

    uint32_t qf[MT == 1 ? KS : 1][4];       // one 16-row block: Q fragments in registers
    float qs[MT][NR];                       // score factor of rows g, g + 8 (softmax scale, log2 e, descale, Q's own factor)
    int pos[MT][NR];                        // position of rows g, g + 8 of each block
    float m[MT][NR], l[MT][NR];             // maxima less kUp, sums
    float oa[MT][NT][4];
    uint8_t *sq = smem + C::kRed;           // two blocks: Q in shared memory between units
    const float kds = FP8 ? *a.k_descale : 1.f, vds = FP8 ? *a.v_descale : 1.f;

    // Q rows of a unit, in up to 16 rows: thread c of a row holds the dims that it reads of K (see
    // the product below).
    uint4 qw[MT == 1 ? NR : 1][D / 32];
    auto fetch_q = [&](const Cursor &u) {
#pragma unroll
        for (int hf = 0; hf < NR; ++hf) {
            const int row = hf * 8 + g, tk = row / G;
            const bool in = tk < u.ent.n;
            const uint8_t *qp = a.q + (int64_t)(u.ent.tok0 + (in ? tk : 0)) * a.q_tok + (int64_t)(u.h * G + (in ? row - tk * G : 0)) * a.q_head;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int ch = FP8 ? (c + 4 * (i >> 1)) * 2 + (i & 1) : c + 4 * i;
                qw[MT == 1 ? hf : 0][i] = make_uint4(0, 0, 0, 0);
                if (in) qw[MT == 1 ? hf : 0][i] = *reinterpret_cast<const uint4 *>(qp + ch * 16);
            }
        }
    };
    auto begin_unit = [&]() {
        const int nrows = cu.ent.n * G;
#pragma unroll
        for (int b = 0; b < MT; ++b)
#pragma unroll
            for (int hf = 0; hf < NR; ++hf) {
                const int row = b * 16 + hf * 8 + g;
                const bool in = row < nrows;
                const int tk = in ? row / G : 0;
                pos[b][hf] = in ? cu.ent.ctx + tk : -1;
                m[b][hf] = -INFINITY;
                l[b][hf] = 0.f;
                if (MT == 1) {
                    float amax = 0.f;
                    uint32_t w[KS][2];
#pragma unroll
                    for (int i = 0; i < KS / 2; ++i) {
                        const uint4 &v = qw[MT == 1 ? hf : 0][i];
                        w[2 * i][0] = v.x;
                        w[2 * i][1] = v.y;
                        w[2 * i + 1][0] = v.z;
                        w[2 * i + 1][1] = v.w;
                    }
                    float f = 1.f;
                    if (FP8) {
#pragma unroll
                        for (int i = 0; i < KS; ++i)
#pragma unroll
                            for (int y = 0; y < 2; ++y)
                                amax = fmax3(amax, fabsf(__uint_as_float(w[i][y] << 16)), fabsf(__uint_as_float(w[i][y] & 0xffff0000u)));
                        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                        f = row_factor(amax, 14);
#pragma unroll
                        for (int i = 0; i < KS; ++i)
#pragma unroll
                            for (int y = 0; y < 2; ++y)
                                w[i][y] = pack_f16x2(__uint_as_float(w[i][y] << 16) * f, __uint_as_float(w[i][y] & 0xffff0000u) * f);
                    }
                    qs[b][hf] = a.scale_log2 * kds / f;
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        qf[MT == 1 ? i : 0][hf] = w[i][0];
                        qf[MT == 1 ? i : 0][2 + hf] = w[i][1];
                        if (NR == 1) qf[MT == 1 ? i : 0][1] = qf[MT == 1 ? i : 0][3] = 0u;
                    }
                }
            }
#pragma unroll
        for (int b = 0; b < MT; ++b)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int y = 0; y < 4; ++y) oa[b][t][y] = 0.f;
        if (MT == 2) {
            // Q of up to 32 rows to shared memory: eight threads a row, as bf16
            // or as scaled fp16 (the factor kept behind the rows).
            const int row = threadIdx.x >> 3, part = threadIdx.x & 7;
            const bool in = row < nrows;
            const int tk = in ? row / G : 0;
            const uint8_t *qp = a.q + (int64_t)(cu.ent.tok0 + tk) * a.q_tok + (int64_t)(cu.h * G + (in ? row - tk * G : 0)) * a.q_head;
            uint32_t w[D / 16];
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (in) v = *reinterpret_cast<const uint4 *>(qp + (part * (D / 64) + i) * 16);
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
            float f = 1.f;
            if (FP8) {
                float amax = 0.f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    amax = fmax3(amax, fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u)));
#pragma unroll
                for (int y = 1; y < 8; y <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, y));
                f = row_factor(amax, 14);
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    w[i] = pack_f16x2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
            }
            named_bar_sync(kSumBar, kWarps * 32);                    // the previous unit's use of the space is over
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const int ch = part * (D / 64) + i;
                *reinterpret_cast<uint4 *>(sq + row * D * 2 + ((ch ^ (FP8 ? (row & 1) : ((row & 1) << 2))) << 4)) =
                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            }
            if (part == 0) *reinterpret_cast<float *>(sq + kFewRows * D * 2 + row * 4) = f;
            named_bar_sync(kSumBar, kWarps * 32);
#pragma unroll
            for (int b = 0; b < MT; ++b)
#pragma unroll
                for (int hf = 0; hf < NR; ++hf)
                    qs[b][hf] = a.scale_log2 * kds / *reinterpret_cast<const float *>(sq + kFewRows * D * 2 + (b * 16 + hf * 8 + g) * 4);
        }
    };

    const int bid = blockIdx.x;
    float4 *red = reinterpret_cast<float4 *>(smem + C::kRed);
    float *sml = reinterpret_cast<float *>(smem + C::kMl);
    volatile int *flag = reinterpret_cast<volatile int *>(smem + C::kMisc);
    float *ws_o = reinterpret_cast<float *>(a.plan + a.L.off_few_o);
    float *ws_ml = reinterpret_cast<float *>(a.plan + a.L.off_few_ml);

    auto store4 = [&](const PagedEntry &en, int h, int row, int dim, float4 v, float inv) {
        const int tk = row / G;
        const int64_t at = ((int64_t)(en.tok0 + tk) * s.Hq + h * G + (row - tk * G)) * D + dim;
        if (a.o_f32)
            *reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.o) + at) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        else
            *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(a.o) + at) =
                make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
    };
    auto store_lse = [&](const PagedEntry &en, int h, int row, float mx, float sum) {
        const int tk = row / G;
        a.lse[(int64_t)(en.tok0 + tk) * s.Hq + h * G + (row - tk * G)] = row_lse(mx, sum);
    };
    // Pieces of the unit's output that a thread handles in the sums below: rows
    // 8 (z >> 2) + g, columns of 4 in the order of the fragments.
    auto dim_of = [&](int np, int z) {
        const int cc = piece_of<NARROW>(2 * c + ((z >> 1) & 1)), jq = (z & 1) * 4;
        return (FP8 && D == 128) ? 16 * cc + 8 * np + jq : 64 * np + 8 * cc + jq;
    };
    // Whether the unit at the cursor begins in this CTA's share, and whether it ends there too.
    auto begins = [&]() { return cu.e != start.e || cu.h != start.h || start.x == 0; };
    // Sums the unit over the warps and writes its rows, or this CTA's partial result of
    // them: every warp leaves its maxima, sums and output in shared memory, eight pieces
    // of the output at a time, and then adds one piece up.  (5 us a unit when it took an
    // exchange more for the maxima, twice the passes, and a fence and an atomic for a split
    // unit in the middle of the walk: 64 requests of one or two tokens over e4m3 0.138 ms, 0.132 so.)
    constexpr int ZP = 4 * NR * (NR == 1 ? NP : 1);         // pieces of a pass
    static_assert(ZP <= C::kPieces && ZP <= kWarps, "pieces of a pass");
    auto end_unit = [&]() {
        const PagedEntry en = cu.ent;
        const int h = cu.h, nrows = en.n * G;
        const bool first = begins(), whole = first && cu.x + 1 == cu.kr.n;
        // Slot of a partial result: 2 c + 1 when the unit begins in this CTA's share, 2 c when it comes in from the left.
        const int slot = 2 * bid + (first ? 1 : 0);
        if (NR == 1) {                  // the low terms' products stand in the idle rows
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                oa[0][t][0] += oa[0][t][2];
                oa[0][t][1] += oa[0][t][3];
            }
        }
#pragma unroll
        for (int b = 0; b < MT; ++b)
#pragma unroll
            for (int hf = 0; hf < NR; ++hf) {
                l[b][hf] += __shfl_xor_sync(0xffffffffu, l[b][hf], 1);
                l[b][hf] += __shfl_xor_sync(0xffffffffu, l[b][hf], 2);
            }
#pragma unroll
        for (int b = 0; b < MT; ++b)
#pragma unroll
            for (int pass = 0; pass < (NR == 1 ? 1 : NP); ++pass) {
                named_bar_sync(kSumBar, kWarps * 32);           // what was there has been read
                if (b == 0 && pass == 0 && c == 0)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int hf = 0; hf < NR; ++hf) {
                            sml[(warp * 2) * kFewRows + i * 16 + hf * 8 + g] = m[i][hf];
                            sml[(warp * 2 + 1) * kFewRows + i * 16 + hf * 8 + g] = l[i][hf];
                        }
                // piece z = (row half or group of 8 tiles, column half, 4 of 8 tiles)
#pragma unroll
                for (int z = 0; z < ZP; ++z) {
                    const int hf = NR == 1 ? 0 : z >> 2, np = NR == 1 ? z >> 2 : pass;
                    const int y = 2 * hf + ((z >> 1) & 1), t = np * 8 + (z & 1) * 4;
                    if (b * 16 + hf * 8 < nrows)
                        red[(warp * ZP + z) * 32 + lane] = make_float4(oa[b][t][y], oa[b][t + 1][y], oa[b][t + 2][y], oa[b][t + 3][y]);
                }
                named_bar_sync(kSumBar, kWarps * 32);
                const int z = warp, hf = NR == 1 ? 0 : z >> 2, np = NR == 1 ? z >> 2 : pass, row = b * 16 + hf * 8 + g;
                if (z < ZP && row < nrows) {
                    float f[kWarps], mx = -INFINITY, sum = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        f[w] = sml[(w * 2) * kFewRows + row];
                        mx = fmaxf(mx, f[w]);
                    }
                    const float mu = mx == -INFINITY ? 0.f : mx;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        f[w] = ex2(f[w] - mu);
                        sum += sml[(w * 2 + 1) * kFewRows + row] * f[w];
                        const float4 u = red[(w * ZP + z) * 32 + lane];
                        v.x += u.x * f[w];
                        v.y += u.y * f[w];
                        v.z += u.z * f[w];
                        v.w += u.w * f[w];
                    }
                    if (whole) store4(en, h, row, dim_of(np, z), v, sum != 0.f ? vds / sum : 0.f);
                    else __stcg(reinterpret_cast<float4 *>(ws_o + ((int64_t)slot * kFewRows + row) * D + dim_of(np, z)), v);
                    if (c == 0 && np == 0 && (z & 3) == 0) {
                        if (whole) {
                            store_lse(en, h, row, mx, sum);
                        } else {
                            __stcg(ws_ml + (int64_t)slot * 2 * kFewRows + row, mx);
                            __stcg(ws_ml + (int64_t)slot * 2 * kFewRows + kFewRows + row, sum);
                        }
                    }
                }
            }
    };
    // After the walk: the units that began before this share or go on behind it, the
    // share's first and last at most.  The last of a unit's CTAs adds the partial results
    // up, in the CTAs' order.  (At the cursor: the share's last unit.)
    auto join_units = [&]() {
        const bool first = begins(), last_cut = !(first && cu.x + 1 == cu.kr.n);
        const bool one = cu.e == start.e && cu.h == start.h;    // the share lies in one unit
        const bool first_cut = start.x > 0 && !one;             // (a first unit that goes on is the last one, too)
        if (!first_cut && !last_cut) return;
        // (The share's first entry is read again: in registers it would be there all the way.)
        const PagedStart *again = reinterpret_cast<const PagedStart *>(a.plan + a.L.off_start) + bid;
        const int4 e0 = __ldcg(reinterpret_cast<const int4 *>(&again->ent));       // r, tok0, n, ctx
        const int64_t cum0 = __ldcg(reinterpret_cast<const long long *>(&again->cum));
        const KeyRange kr0 = key_range(e0.w, e0.w + e0.z - 1, s.window, s.sink);
        // The unit's CTAs, from the first one (tiles [ub, ub + n) of the list), beside the flags.
        const int who = threadIdx.x == 0 ? 0 : threadIdx.x == 32 ? 1 : -1;
        int from = 0, more = 0;
        if (who >= 0) {
            const int64_t ub = who == 0 ? cum0 + (int64_t)start.h * kr0.n : cu.cum + (int64_t)cu.h * cu.kr.n;
            from = share_owner(W, ctas, ub);
            more = share_owner(W, ctas, ub + (who == 0 ? kr0.n : cu.kr.n) - 1) - from;
            flag[4 + who] = from;
            flag[6 + who] = more + 1;
        }
        __threadfence();
        named_bar_sync(kSumBar, kWarps * 32);
        if (who >= 0) {
            int mine = 0;
            if (who == 0 ? first_cut : last_cut) {
                unsigned *cnt = reinterpret_cast<unsigned *>(a.plan + a.L.off_count) + from;
                mine = atomicInc(cnt, (unsigned)more) == (unsigned)more ? 1 : 0;        // returns to 0 by itself
                __threadfence();
            }
            flag[2 * who] = mine;
        }
        named_bar_sync(kSumBar, kWarps * 32);
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            if (!flag[2 * i]) continue;
            const PagedEntry en{0, i == 0 ? e0.y : cu.ent.tok0, i == 0 ? e0.z : cu.ent.n, 0};
            const int h = i == 0 ? start.h : cu.h, nrows = en.n * G, c_first = flag[4 + i], parts = flag[6 + i];
            float *wt = reinterpret_cast<float *>(red);             // [part][row] weights
            auto slot_of = [&](int p) { return (int64_t)(2 * (c_first + p) + (p == 0 ? 1 : 0)); };
            for (int row = warp; row < nrows; row += kWarps) {
                // A lane holds up to five parts (kPagedCtas of them at most).
                constexpr int PL = (kPagedCtas + 31) / 32;
                float y[PL], z[PL], mx = -INFINITY, sum = 0.f;
#pragma unroll
                for (int x = 0; x < PL; ++x) {
                    const int p = lane + 32 * x;
                    y[x] = p < parts ? ld_cg(ws_ml + slot_of(p) * 2 * kFewRows + row) : -INFINITY;
                    z[x] = p < parts ? ld_cg(ws_ml + slot_of(p) * 2 * kFewRows + kFewRows + row) : 0.f;
                }
#pragma unroll
                for (int x = 0; x < PL; ++x) mx = fmaxf(mx, y[x]);
#pragma unroll
                for (int x = 1; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                const float mu = mx == -INFINITY ? 0.f : mx;
#pragma unroll
                for (int x = 0; x < PL; ++x) {
                    const float w = ex2(y[x] - mu);
                    if (lane + 32 * x < parts) wt[(lane + 32 * x) * ROWS + row] = w;
                    sum += w * z[x];
                }
#pragma unroll
                for (int x = 1; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                if (lane == 0) {
                    store_lse(en, h, row, mx, sum);
                    sml[row] = sum != 0.f ? vds / sum : 0.f;
                }
            }
            named_bar_sync(kSumBar, kWarps * 32);
            for (int x = threadIdx.x; x < nrows * (D / 4); x += kWarps * 32) {
                const int row = x / (D / 4), dim = (x % (D / 4)) * 4;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                constexpr int BP = 8;               // parts in flight: loads first, uses after
                for (int p0 = 0; p0 < parts; p0 += BP) {
                    float4 u[BP];
#pragma unroll
                    for (int y = 0; y < BP; ++y)
                        u[y] = ld_cg(reinterpret_cast<const float4 *>(ws_o + (slot_of(min(p0 + y, parts - 1)) * kFewRows + row) * D + dim));
#pragma unroll
                    for (int y = 0; y < BP; ++y) {
                        const float w = p0 + y < parts ? wt[(p0 + y) * ROWS + row] : 0.f;
                        v.x += u[y].x * w;
                        v.y += u[y].y * w;
                        v.z += u[y].z * w;
                        v.w += u[y].w * w;
                    }
                }
                store4(en, h, row, dim, v, sml[row]);
            }
            named_bar_sync(kSumBar, kWarps * 32);
        }
    };

    // ---- the walk -------------------------------------------------------------
    if (MT == 1) fetch_q(cu);
    begin_unit();
    // Byte offsets of this thread's fragments in a stage.
    uint32_t group[SUB], k_at[2], v_at[2];  // groups of 16 keys; K: even and odd load of a box; V: keys ka and kb2
#pragma unroll
    for (int i = 0; i < SUB; ++i) {
        const int j = key0 + 16 * i;
        group[i] = (uint32_t)(j / box_keys * box_keys * C::kRow + j % box_keys * (NARROW ? 64 : 128));
    }
    k_at[0] = chunk_at<NARROW>(kg, c);
    k_at[1] = NARROW ? 0 : chunk_at<NARROW>(kg, c + 4);
    constexpr uint32_t V0 = kKeyTile * C::kRow;             // V behind K
    v_at[0] = V0 + (NARROW ? chunk_at<NARROW>(ka, g >> 1) + (g & 1) * 8 : chunk_at<NARROW>(ka, piece_of<NARROW>(g)));
    v_at[1] = V0 + (NARROW ? chunk_at<NARROW>(kb2, g >> 1) + (g & 1) * 8 : chunk_at<NARROW>(kb2, piece_of<NARROW>(g)));
    constexpr uint32_t ROW8 = NARROW ? 512 : 1024;          // eight rows further
    int st = 0, step = 0;
    uint32_t phase = 0;
    while (true) {
        const int kw = cu.kr.tile(cu.x) * kKeyTile + key0;
        // A wait that ran out has set the status: the walk goes on, so that every
        // barrier is reached, and what it writes does not count.
        if (step % SUB == turn) warp_wait(&full[st], phase, abort, a.status, a.wait_limit);
        if (step % SUB == turn && some(kw, 16 * SUB)) {
            const uint32_t base = smem_u32(smem) + st * C::kStage;
            const bool whole = kw + 16 * SUB <= cu.kr.hi && (kw >= cu.kr.lo || kw + 16 * SUB <= s.sink);
            if (!whole) {
                // V of keys that no row attends becomes zero: what a page holds behind
                // the last token (or the stage from before) reaches no product (0 x NaN).
                constexpr int CH = C::kRow / 16;
#pragma unroll
                for (int q = 0; q < SUB; ++q)
                    for (int i = lane; i < 16 * CH; i += 32) {
                        const int row = i / CH, ch = i % CH, j = kw + 16 * q + row;
                        if (j >= cu.kr.hi || (j < cu.kr.lo && j >= s.sink))
                            st_shared_v4(smem + st * C::kStage + V0 + group[q] + (ch >> 3) * half_box + chunk_at<NARROW>(row, ch & 7),
                                         make_uint4(0, 0, 0, 0));
                    }
                fence_proxy_async_smem();       // before a later tile's copy into the stage
                __syncwarp();
            }
            float sc[MT][2 * SUB][4];
#pragma unroll
            for (int b = 0; b < MT; ++b)
#pragma unroll
                for (int nt = 0; nt < 2 * SUB; ++nt)
#pragma unroll
                    for (int y = 0; y < 4; ++y) sc[b][nt][y] = 0.f;
            // Scores: 16 bytes of a key per thread and load are two k-steps of
            // bf16 (words 0, 1 and 2, 3) or four of e4m3 (one word each).
#pragma unroll
            for (int i = 0; i < C::kRow / 64; ++i) {
                constexpr int PER = FP8 ? 4 : 2;
                uint32_t qa[MT][PER][4];
#pragma unroll
                for (int b = 0; b < MT; ++b) {
                    if (MT == 1) {
#pragma unroll
                        for (int y = 0; y < PER; ++y)
#pragma unroll
                            for (int z = 0; z < 4; ++z) qa[b][y][z] = qf[MT == 1 ? i * PER + y : 0][z];
                    } else {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const int row = b * 16 + hf * 8 + g;
                            const uint32_t qb = smem_u32(sq) + row * D * 2;
#pragma unroll
                            for (int y = 0; y < PER / 2; ++y) {
                                const int ch = FP8 ? (c + 4 * i) * 2 + y : c + 4 * i;
                                const uint4 v = lds128(qb + ((ch ^ (FP8 ? (row & 1) : ((row & 1) << 2))) << 4));
                                qa[b][2 * y][hf] = v.x;
                                qa[b][2 * y][2 + hf] = v.y;
                                qa[b][2 * y + 1][hf] = v.z;
                                qa[b][2 * y + 1][2 + hf] = v.w;
                            }
                        }
                    }
                }
#pragma unroll
                for (int nt = 0; nt < 2 * SUB; ++nt) {
                    const uint4 kv = lds128(base + group[nt >> 1] + k_at[i & 1] + (i >> 1) * half_box + (nt & 1) * ROW8);
                    const uint32_t w[4] = {kv.x, kv.y, kv.z, kv.w};
#pragma unroll
                    for (int y = 0; y < PER; ++y) {
                        const uint32_t b0 = FP8 ? f16x2_of_e4m3(w[y]) : w[(2 * y) & 3];
                        const uint32_t b1 = FP8 ? f16x2_of_e4m3(w[y] >> 16) : w[(2 * y + 1) & 3];
#pragma unroll
                        for (int b = 0; b < MT; ++b)
                            mma16816<FP8>(sc[b][nt], qa[b][y][0], qa[b][y][1], qa[b][y][2], qa[b][y][3], b0, b1);
                    }
                }
            }
            // Scaled, and masked where some row does not attend some of the keys.
            const bool edge = kw + 16 * SUB - 1 > cu.ent.ctx ||
                              (s.window > 0 && kw <= cu.ent.ctx + cu.ent.n - 1 - s.window && kw + 16 * SUB > s.sink);
#pragma unroll
            for (int b = 0; b < MT; ++b)
#pragma unroll
                for (int nt = 0; nt < 2 * SUB; ++nt)
#pragma unroll
                    for (int y = 0; y < 2 * NR; ++y) sc[b][nt][y] *= qs[b][y >> 1];
            if (edge) {
#pragma unroll
                for (int b = 0; b < MT; ++b)
#pragma unroll
                    for (int nt = 0; nt < 2 * SUB; ++nt)
#pragma unroll
                        for (int y = 0; y < 2 * NR; ++y) {
                            const int j = kw + nt * 8 + ((y & 1) ? kb2 : ka), p = pos[b][y >> 1];
                            if (!(j <= p && (s.window == 0 || j > p - s.window || j < s.sink))) sc[b][nt][y] = -INFINITY;
                        }
            }
            // Running maxima, raised lazily: only when a score exceeds one by more
            // than the band do the lanes of a row agree on a new one.
            auto row_max = [&](int b, int hf) {
                float x = fmaxf(sc[b][0][2 * hf], sc[b][0][2 * hf + 1]);
#pragma unroll
                for (int nt = 1; nt < 2 * SUB; ++nt) x = fmax3(x, sc[b][nt][2 * hf], sc[b][nt][2 * hf + 1]);
                return x;
            };
            bool raise = false;
#pragma unroll
            for (int b = 0; b < MT; ++b)
#pragma unroll
                for (int hf = 0; hf < NR; ++hf)
                    raise = raise || row_max(b, hf) > m[b][hf] + (kBand + kUp);
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int b = 0; b < MT; ++b)
#pragma unroll
                    for (int hf = 0; hf < NR; ++hf) {
                        float x = row_max(b, hf);
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2)) - kUp;
                        if (x > m[b][hf]) {
                            const float f = ex2(m[b][hf] - x);
                            m[b][hf] = x;
                            l[b][hf] *= f;
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                oa[b][t][2 * hf] *= f;
                                oa[b][t][2 * hf + 1] *= f;
                                if (NR == 1) {
                                    oa[b][t][2] *= f;
                                    oa[b][t][3] *= f;
                                }
                            }
                        }
                    }
            }
            // P and its sums, as fragments: pt[term][key half][row half].
            uint32_t pt[MT][TERMS][2 * SUB][NR];
#pragma unroll
            for (int b = 0; b < MT; ++b)
#pragma unroll
                for (int hf = 0; hf < NR; ++hf) {
                    const float mu = m[b][hf] == -INFINITY ? 0.f : m[b][hf];
#pragma unroll
                    for (int nt = 0; nt < 2 * SUB; ++nt) {
                        float p0 = ex2(sc[b][nt][2 * hf] - mu), p1 = ex2(sc[b][nt][2 * hf + 1] - mu);
                        l[b][hf] += p0 + p1;
#pragma unroll
                        for (int y = 0; y < TERMS; ++y) {
                            const uint32_t hi = FP8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
                            pt[b][y][nt][hf] = hi;
                            if (y + 1 < TERMS) {
                                float u0 = __uint_as_float(hi << 16), u1 = __uint_as_float(hi & 0xffff0000u);
                                if (FP8) unpack_f16x2(hi, u0, u1);
                                p0 -= u0;
                                p1 -= u1;
                            }
                        }
                    }
                }
            // O += P V: the thread's two key pairs, columns as dim_of() says.
            auto pv = [&](int q, int t, uint32_t b0, uint32_t b1) {
#pragma unroll
                for (int b = 0; b < MT; ++b) {
                    if (NR == 1) {
                        // Rows 0-7 the first term, rows 8-15 the second; then the third.
                        mma16816<FP8>(oa[b][t], pt[b][0][2 * q][0], TERMS > 1 ? pt[b][1 % TERMS][2 * q][0] : 0u, pt[b][0][2 * q + 1][0],
                                      TERMS > 1 ? pt[b][1 % TERMS][2 * q + 1][0] : 0u, b0, b1);
                        if (TERMS > 2)
                            mma16816<FP8>(oa[b][t], 0u, pt[b][2 % TERMS][2 * q][0], 0u, pt[b][2 % TERMS][2 * q + 1][0], b0, b1);
                    } else {
#pragma unroll
                        for (int y = 0; y < TERMS; ++y)
                            mma16816<FP8>(oa[b][t], pt[b][y][2 * q][0], pt[b][y][2 * q][NR - 1], pt[b][y][2 * q + 1][0],
                                          pt[b][y][2 * q + 1][NR - 1], b0, b1);
                    }
                }
            };
#pragma unroll
            for (int q = 0; q < SUB; ++q) {
                const uint32_t vq = base + group[q];
                if (!FP8) {
#pragma unroll
                    for (int np = 0; np < NP; ++np) {
                        uint32_t w[4][4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint4 v = lds128(vq + v_at[r & 1] + np * half_box + (r >> 1) * ROW8);
                            w[r][0] = v.x;
                            w[r][1] = v.y;
                            w[r][2] = v.z;
                            w[r][3] = v.w;
                        }
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            pv(q, np * 8 + 2 * x, __byte_perm(w[0][x], w[1][x], 0x5410), __byte_perm(w[2][x], w[3][x], 0x5410));
                            pv(q, np * 8 + 2 * x + 1, __byte_perm(w[0][x], w[1][x], 0x7632), __byte_perm(w[2][x], w[3][x], 0x7632));
                        }
                    }
                } else {
                    constexpr int WD = D / 32;      // words of e4m3 per key and thread
                    uint32_t w[4][WD];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint32_t at = vq + v_at[r & 1] + (r >> 1) * ROW8;
                        if (WD == 4) {
                            const uint4 v = lds128(at);
                            w[r][0] = v.x;
                            w[r][1] = v.y;
                            w[r][2 % WD] = v.z;
                            w[r][3 % WD] = v.w;
                        } else {
                            const uint2 v = lds64(at);
                            w[r][0] = v.x;
                            w[r][1] = v.y;
                        }
                    }
                    // The bytes of two keys are paired before they are expanded.
#pragma unroll
                    for (int x = 0; x < WD; ++x) {
                        const uint32_t lo01 = __byte_perm(w[0][x], w[1][x], 0x5140), hi01 = __byte_perm(w[0][x], w[1][x], 0x7362);
                        const uint32_t lo23 = __byte_perm(w[2][x], w[3][x], 0x5140), hi23 = __byte_perm(w[2][x], w[3][x], 0x7362);
                        pv(q, 4 * x, f16x2_of_e4m3(lo01), f16x2_of_e4m3(lo23));
                        pv(q, 4 * x + 1, f16x2_of_e4m3(lo01 >> 16), f16x2_of_e4m3(lo23 >> 16));
                        pv(q, 4 * x + 2, f16x2_of_e4m3(hi01), f16x2_of_e4m3(hi23));
                        pv(q, 4 * x + 3, f16x2_of_e4m3(hi01 >> 16), f16x2_of_e4m3(hi23 >> 16));
                    }
                }
            }
        }
        if (step % SUB == turn) {
            __syncwarp();               // every lane has read the stage
            if (lane == 0) mbar_arrive(&empty[st]);
        }
        if (++st == ST) {
            st = 0;
            phase ^= 1;
        }
        ++step;
        --left;
        const bool last_of_unit = cu.x + 1 == cu.kr.n || left == 0;
        if (!last_of_unit) {
            ++cu.x;
            continue;
        }
        // The next unit's Q is on its way while this one ends (more rows lack the registers).
        Cursor next = cu;
        if (left > 0) {
            advance(next, true);
            if (NR == 1) fetch_q(next);
        }
        end_unit();
        if (left == 0) break;
        cu = next;
        if (MT == 1 && NR == 2) fetch_q(cu);
        begin_unit();
    }
    join_units();
    // The many-rows kernel may still run on other SMs (see the launch).
    grid_wait_before();
    if (hd->splits_many > 1) add_parts<D>(a, hd, vds);
}

// 16-bit terms of P (see above).
FM_HD constexpr int terms_of(bool fp8, int rows, bool f32) { return fp8 ? (rows == 8 || f32 ? 2 : 1) : (f32 ? 3 : 2); }

// RMAX: rows that a request of the step can have at most, 8, 16 or 32.
template <int D, bool FP8, bool F32, int RMAX>
__global__ void __launch_bounds__(kThreads, 1)
    fm_paged_decode_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const PagedArgs a,
                           const int box_keys)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    const PagedHeader *hd = reinterpret_cast<const PagedHeader *>(a.plan);
    const PagedStart start = reinterpret_cast<const PagedStart *>(a.plan + a.L.off_start)[blockIdx.x];   // used if the plan fits
    if (!paged_plan_fits(hd, a.s)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, FM_ERR_PLAN_MISMATCH);
        grid_wait_before();
        return;
    }
    if (hd->rows > a.rows) {            // more rows than the caller's tensors have
        if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, FM_ERR_LENGTHS);
        grid_wait_before();
        return;
    }
    // No CTA ends before the many-rows kernel, which may still run on other SMs (see the launch), so
    // that whatever comes behind this kernel comes behind both; its parts are added up
    // after the few rows.
    if ((int)blockIdx.x >= hd->ctas_few) {
        grid_wait_before();
        if (hd->splits_many > 1 && warp_id() < kWarps) add_parts<D>(a, hd, FP8 ? *a.v_descale : 1.f);
        return;
    }
    // By the rows that the units of this CTA's share have at most (parts of a unit fit together
    // whichever way they are computed): a step that could have 32 rows seldom has.  64
    // requests of one token and four heads per KV head in a step of up to 512: bf16 437 us as
    // 32 rows, 364 as 8; e4m3 361 and 216.  16 rows in such a step: e4m3 104 and 78.
    if (RMAX > 16 && start.rows > 16) {
        walk_share<D, FP8, 32, terms_of(FP8, 32, F32)>(tk, tv, a, box_keys, hd, start, smem);
        return;
    }
    if (RMAX > 8 && start.rows > 8) {
        walk_share<D, FP8, 16, terms_of(FP8, 16, F32)>(tk, tv, a, box_keys, hd, start, smem);
        return;
    }
    walk_share<D, FP8, 8, terms_of(FP8, 8, F32)>(tk, tv, a, box_keys, hd, start, smem);
}

}  // namespace fm

using namespace fm;

namespace {

template <int D, bool FP8, bool F32, int RMAX>
fm_status launch(const CUtensorMap &tk, const CUtensorMap &tv, const PagedArgs &a, int box_keys, cudaStream_t stream)
{
    constexpr int smem = DecodeCfg<D, FP8, RMAX>::kBytes;
    static_assert(DecodeCfg<D, FP8, 8>::kBytes <= smem && (RMAX < 32 || DecodeCfg<D, FP8, 16>::kBytes <= smem), "shared memory of either way");
    static std::atomic<uint8_t> done[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FM_ERR_CUDA;
    if (!done[dev].load(std::memory_order_acquire)) {
        // The register split adds up to the launch's registers only if the
        // kernel was compiled to that many per thread.
        cudaFuncAttributes fa{};
        if (cudaFuncGetAttributes(&fa, fm_paged_decode_kernel<D, FP8, F32, RMAX>) != cudaSuccess || fa.numRegs != kLaunchRegs)
            return FM_ERR_CUDA;
        if (cudaFuncSetAttribute(fm_paged_decode_kernel<D, FP8, F32, RMAX>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return FM_ERR_CUDA;
        done[dev].store(1, std::memory_order_release);
    }
    // Behind a many-rows launch this one may start before it ends: its CTAs need a whole
    // SM's shared memory, so each comes when the SM's own CTA of that kernel has left.
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kPagedCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = (int64_t)a.s.max_q * (a.s.Hq / a.s.Hkv) > kFewRows ? 1 : 0;
    ProfScope ps(kKPagedDecode, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fm_paged_decode_kernel<D, FP8, F32, RMAX>, tk, tv, a, box_keys);
    return e == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

// By the rows that a request of the step can have at most: a kernel with fewer ways in it is
// faster where they are enough (when they were separated: 8 rows
// alone 295 us, beside the others 301; 32 rows alone 252, beside the others 258; today 241).
template <int D, bool FP8>
fm_status launch_rows(const CUtensorMap &tk, const CUtensorMap &tv, const PagedArgs &a, int box_keys, cudaStream_t stream)
{
    const int64_t rows = (int64_t)a.s.max_q * (a.s.Hq / a.s.Hkv);
    if (a.o_f32)                        // (8 rows of e4m3 take two terms for either output)
        return rows <= 8 ? launch<D, FP8, !FP8, 8>(tk, tv, a, box_keys, stream)
                         : rows <= 16 ? launch<D, FP8, true, 16>(tk, tv, a, box_keys, stream) : launch<D, FP8, true, 32>(tk, tv, a, box_keys, stream);
    return rows <= 8 ? launch<D, FP8, false, 8>(tk, tv, a, box_keys, stream)
                     : rows <= 16 ? launch<D, FP8, false, 16>(tk, tv, a, box_keys, stream) : launch<D, FP8, false, 32>(tk, tv, a, box_keys, stream);
}

}  // namespace

fm_status fm_paged_decode_launch(const CUtensorMap &tk, const CUtensorMap &tv, const PagedArgs &a, int box_keys, bool e4m3,
                                 cudaStream_t stream)
{
    if (a.s.d == 128) return e4m3 ? launch_rows<128, true>(tk, tv, a, box_keys, stream) : launch_rows<128, false>(tk, tv, a, box_keys, stream);
    return e4m3 ? launch_rows<64, true>(tk, tv, a, box_keys, stream) : launch_rows<64, false>(tk, tv, a, box_keys, stream);
}
