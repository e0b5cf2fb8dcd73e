// Internal definitions of the paged-cache operators: the layout of a step's
// plan buffer and the key ranges that the planner and the kernels share.
#pragma once

#include <cuda.h>

#include <cmath>

#include "fm_internal.h"

namespace fm {

constexpr uint32_t kPagedMagic = 0x464D5047u;   // "FMPG"
constexpr int kKeyTile = 128;                   // keys per tile of work, a multiple of every page granule
constexpr int kPageGranule = 16;                // page sizes are multiples of this: 16 aligned keys share a page
constexpr int kMaxPage = 1 << 16;               // tokens of a page at most
constexpr int kFewRows = 32;                    // (new tokens x query heads per KV head) up to which a request is "few rows"
constexpr int kPagedCtas = 152;                 // CTAs of the persistent attention kernels (no CTA waits for another)
constexpr int kMaxRequests = 8192;
constexpr int kMaxSplitUnits = 2 * kPagedCtas;  // many-rows units that are still split along the keys
constexpr int kMaxPieces = 4 * kPagedCtas;      // pieces they are split into at most

struct PagedShape {
    int32_t R, T, max_q, max_pages, num_pages, page_size, Hq, Hkv, d, window, sink;
};

// First 256 bytes of a plan, written by the planner.
struct PagedHeader {
    uint32_t magic;
    PagedShape s;
    int32_t n_few;        // entries of the few-rows list
    int32_t ctas_few;     // CTAs that share its tiles (0: none)
    int64_t tiles_few;    // key tiles of the list, over all KV heads
    int32_t rows;         // rows of q: new tokens of all requests
    int32_t n_many;       // entries of the many-rows list
    int32_t units_many;   // its units (request, KV head, query tile)
    int32_t splits_many;  // pieces per unit along the keys (1: whole units)
    int32_t pad[44];
};
static_assert(sizeof(PagedHeader) == 256, "plan header size");

// One request of an attention work list.
struct PagedEntry {
    int32_t r, tok0, n, ctx;   // request, its first row of q, new tokens, tokens cached before them
};

// Where a CTA's share of the few-rows list begins: all that its first loads need, so that
// they wait for one read of the plan and one of the block table.
struct PagedStart {
    int32_t e, h, x, count;    // entry, KV head, tile of the entry's range; tiles of the share
    PagedEntry ent;            // the entry
    int64_t cum;               // tiles before it
    int32_t rows;              // rows of the share's units at most
    int32_t pad;
};
static_assert(sizeof(PagedStart) == 48, "start record size");

struct PagedLayout {
    int64_t off_few;       // PagedEntry [R]
    int64_t off_few_cum;   // int64 [R + 1]  tiles before entry i, over all KV heads
    int64_t off_start;     // PagedStart [kPagedCtas]
    int64_t off_count;     // uint32 [kPagedCtas]  arrivals at the split unit that begins in CTA c
    int64_t off_few_o;     // fp32 [2 kPagedCtas][kFewRows][d]  unnormalised partial outputs
    int64_t off_few_ml;    // fp32 [2 kPagedCtas][2][kFewRows]  their row maxima (base 2) and sums
    int64_t off_many;      // PagedEntry [R]
    int64_t off_many_cum;  // int32 [R + 1]  units before entry i
    int64_t off_claim;     // uint32  next piece to claim
    int64_t off_many_o;    // fp32 [kMaxPieces][d / 4][128][4]  unnormalised partial outputs
    int64_t off_many_ml;   // fp32 [kMaxPieces][2][128]
    int64_t total;
};

inline PagedLayout paged_layout(const PagedShape &s)
{
    PagedLayout L;
    int64_t off = 256;
    L.off_few = off;      off = align256(off + (int64_t)s.R * 16);
    L.off_few_cum = off;  off = align256(off + ((int64_t)s.R + 1) * 8);
    L.off_start = off;    off = align256(off + kPagedCtas * 48);
    L.off_count = off;    off = align256(off + kPagedCtas * 4);
    L.off_few_o = off;    off = align256(off + (int64_t)2 * kPagedCtas * kFewRows * s.d * 4);
    L.off_few_ml = off;   off = align256(off + (int64_t)2 * kPagedCtas * 2 * kFewRows * 4);
    const bool many = (int64_t)s.max_q * (s.Hq / s.Hkv) > kFewRows;   // else no request can have many rows
    L.off_many = off;       off = align256(off + (many ? (int64_t)s.R * 16 : 0));
    L.off_many_cum = off;   off = align256(off + (many ? ((int64_t)s.R + 1) * 4 : 0));
    L.off_claim = off;      off = align256(off + 4);
    L.off_many_o = off;     off = align256(off + (many ? (int64_t)kMaxPieces * 128 * s.d * 4 : 0));
    L.off_many_ml = off;    off = align256(off + (many ? (int64_t)kMaxPieces * 2 * 128 * 4 : 0));
    L.total = off;
    return L;
}

// Keys that the rows at positions [p0, p1] of a request attend: j < hi and
// (j >= lo or j < sink), with j <= p for the row at p, and j > p - window or
// j < sink when there is a window.  As key tiles: tile x of n stands for key
// tile x while x < ns (the sink), else for first + x - ns.
struct KeyRange {
    int lo, hi;
    int ns, first, n;
    FM_HD int tile(int x) const { return x < ns ? x : first + x - ns; }
};

FM_HD KeyRange key_range(int p0, int p1, int window, int sink)
{
    KeyRange k;
    k.hi = p1 + 1;
    k.lo = (window > 0 && p0 >= window) ? p0 - window + 1 : 0;
    if (sink >= k.lo) k.lo = 0;
    k.first = k.lo / kKeyTile;
    const int s = (sink + kKeyTile - 1) / kKeyTile;
    k.ns = k.lo > 0 ? (s < k.first ? s : k.first) : 0;
    k.n = k.ns + (k.hi + kKeyTile - 1) / kKeyTile - k.first;
    return k;
}

// Tiles [share_begin(c), share_begin(c + 1)) of n belong to CTA c of ctas;
// tile x belongs to CTA share_owner(x).
FM_HD int64_t share_begin(int64_t n, int ctas, int64_t c) { return c * n / ctas; }
FM_HD int share_owner(int64_t n, int ctas, int64_t x) { return (int)(((x + 1) * ctas - 1) / n); }

#if defined(__CUDACC__)
__device__ __forceinline__ bool paged_plan_fits(const PagedHeader *h, const PagedShape &s)
{
    const PagedShape &p = h->s;
    return h->magic == kPagedMagic && p.R == s.R && p.T == s.T && p.max_q == s.max_q && p.max_pages == s.max_pages &&
           p.num_pages == s.num_pages && p.page_size == s.page_size && p.Hq == s.Hq && p.Hkv == s.Hkv && p.d == s.d &&
           p.window == s.window && p.sink == s.sink;
}

// Power of two that puts a row's largest element amax in [2^top, 2^(top + 1));
// 1 when the row is zero or not finite.  Q beside e4m3 keys: exact in fewer
// exponents than bf16 has once the row is scaled, and taken back in the score
// factor.
__device__ __forceinline__ float row_factor(float amax, int top)
{
    if (!(amax > 0.f) || amax == INFINITY) return 1.f;
    const int ex = (int)(__float_as_uint(amax) >> 23) - 127;
    return __uint_as_float((uint32_t)(min(top - ex, 100) + 127) << 23);
}

// P beside e4m3 values enters its product as fp16, whose steps end at 2^-24: it is held
// as 2^kLift exp2(s - m), so that with the lazy maximum's 2^8 it stays below fp16's
// 65504 and a weight of 2^-32 of the row's largest still counts half a step (without
// the lift 2^-25: a key 18 nats above 100,000 others lost them all, 0.15 % of the
// output).  Sums are of the lifted P, and the maxima that belong to them are less kLift.
constexpr float kLift = 7.f;

// Natural log-sum-exp of a row from its maximum (base 2) and sum.
__device__ __forceinline__ float row_lse(float mx, float sum)
{
    return sum > 0.f ? (mx + log2f(sum)) * 0.69314718055994531f : (sum == 0.f ? -INFINITY : sum);
}
#endif

// Arguments of the attention kernels (everything but TMA descriptors).
struct PagedArgs {
    PagedShape s;
    PagedLayout L;
    uint8_t *plan;
    const int32_t *table;
    const uint8_t *q;               // bf16
    int64_t q_tok, q_head;          // strides in bytes, as all of these
    const float *k_descale, *v_descale;   // e4m3 cache: one float each
    void *o;                        // [rows, Hq, d]
    float *lse;                     // [rows, Hq]
    int32_t *status;
    float scale_log2;
    int o_f32;
    int rows;                       // rows that q, o and lse have
    int page_shift;                 // log2 of the page size, -1 if it is no power of two
    long long wait_limit;           // cycles after which a wait gives up
    int withhold;                   // wait test, 0 or 1: the first CTA leaves its second tile out (few rows), K's loads never end (many rows)
};

// Tensor map of bf16 or 8-bit data with any strides (bytes, of dimensions 1 and
// up), zero fill outside, swizzle of 128, 64 or 0 bytes (fm_api.cu).
bool make_tmap_strided(CUtensorMap *map, const void *base, bool u8, int rank, const uint64_t *dims, const uint64_t *strides,
                       const uint32_t *box, int swizzle);

}  // namespace fm

// Launchers of the few-rows kernel (fm_paged_decode.cu) and of the many-rows
// kernel (fm_paged_chunk.cu); box_keys: consecutive keys of one TMA box.
fm_status fm_paged_decode_launch(const CUtensorMap &tk, const CUtensorMap &tv, const fm::PagedArgs &a, int box_keys,
                                 bool e4m3, cudaStream_t stream);
fm_status fm_paged_chunk_launch(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const fm::PagedArgs &a,
                                int box_keys, bool e4m3, cudaStream_t stream);
