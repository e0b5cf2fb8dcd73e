// Verification of drafted tokens: per request, the drafts that the target keeps and the token behind them.
//
//   row i: keep t = tokens[i + 1] if u_i q(t) < p(t), until the first refusal;
//   then the smallest x with sum_(y <= x) w(y) > u sum w,  w = max(p - q, 0), or p where all are kept.
//
// One row of p and one of q are read per request, by a cluster of CTAs that share the vocabulary in contiguous
// slices, so that a few requests are spread over the SMs.  Bound by a chain, not by bytes or terms: lengths, tokens,
// their probabilities, a vote, the row's first load, its sums, a meeting, the search (64 requests of up to five rows over
// 131,072 tokens, fp32 or bf16, with or without the drafts' probabilities: 10 to 2.5 us of bytes, 20 to 21 us each, the
// release of the pages among them).  A token at a border has to come out the same however the sums are added up,
// which 24 bits do not give over 100,000 terms, and 64-bit units take far too long here (two results a cycle and SM: with
// them in the search alone, 64 requests over 131,072 tokens took 51 us for 17, two over 32,000 21 for 7): every sum is
// held in a pair of floats, with the exact error of each addition and difference (Knuth's two-sum, Dekker's fast one for a
// larger minus a smaller), about 48 bits.  Every CTA of 512 is resident at once (64 registers, 4 a SM).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cmath>

#include "fm_paged.h"
#include "fm_ptx.cuh"

namespace cg = cooperative_groups;

namespace fm {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCluster = 8;
constexpr int kSegments = 256;          // of a CTA's slice at most
constexpr int kLoads = 2;               // loads of 8 tokens of a lane in flight, of p and of q
constexpr int kSegment = 512;           // tokens of a segment at least: 32 lanes and as many loads

struct VerifyArgs {
    const uint8_t *target, *draft;      // bytes; draft may be null
    int64_t target_row, draft_row;      // bytes
    const int32_t *tokens, *cu, *seq;
    const float *u_accept, *u_sample;
    int32_t *out, *n_out, *new_lens, *status;
    int32_t V, rows, R;
    int32_t slice, segment;             // tokens of a CTA and of a segment (multiples of 8)
    int32_t wide;                       // rows may be read 16 bytes at a time
};

template <class T>
__device__ __forceinline__ float prob(const uint8_t *row, int64_t i);
template <>
__device__ __forceinline__ float prob<float>(const uint8_t *row, int64_t i) { return __ldg(reinterpret_cast<const float *>(row) + i); }
template <>
__device__ __forceinline__ float prob<uint16_t>(const uint8_t *row, int64_t i)
{
    return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t *>(row) + i) << 16);
}

// Eight probabilities from place i on (those at or behind `end` as zeros).
template <class T>
__device__ __forceinline__ void probs8(const uint8_t *row, int64_t i, int64_t end, bool wide, float (&x)[8])
{
    if (wide && i + 8 <= end) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(row + i * 4)), b = __ldg(reinterpret_cast<const float4 *>(row + i * 4) + 1);
            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        } else {
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(row + i * 2));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) x[2 * j] = __uint_as_float(w[j] << 16), x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = i + j < end ? prob<T>(row, i + j) : 0.f;
    }
}

// A sum in two floats: hi + lo, with the rounding error of every addition to hi kept in lo.
struct Pair {
    float hi, lo;
    __device__ __forceinline__ void add(float x, float more)
    {
        const float s = hi + x, b = s - hi;
        lo += ((hi - (s - b)) + (x - b)) + more;
        hi = s;
    }
    __device__ __forceinline__ void add(const Pair &o) { add(o.hi, o.lo); }
    // lo below half a step of hi, so that pairs compare.
    __device__ __forceinline__ Pair whole() const
    {
        const float s = hi + lo;
        return Pair{s, lo - (s - hi)};
    }
    __device__ __forceinline__ bool above(const Pair &o) const { return (hi - o.hi) + (lo - o.lo) > 0.f; }      // (both whole; exact where they are near)
    __device__ __forceinline__ Pair from(int lane) const { return Pair{__shfl_sync(0xffffffffu, hi, lane), __shfl_sync(0xffffffffu, lo, lane)}; }
    // Sum over the lanes up to this one.
    __device__ __forceinline__ Pair upto() const
    {
        Pair s = *this;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Pair y{__shfl_up_sync(0xffffffffu, s.hi, o), __shfl_up_sync(0xffffffffu, s.lo, o)};
            if (lane_id() >= o) s.add(y);
        }
        return s;
    }
};

// The weights of a request's draw.
struct Row {
    const uint8_t *p, *q;       // q null: p alone
    int hot;                    // the token whose weight is zero (drafts taken with certainty), or -1
};

// Weight of a token: x in two floats, exactly.
__device__ __forceinline__ Pair weight_of(const Row &w, float p, float q, int64_t i)
{
    Pair x{p, 0.f};
    if (w.q) {
        x.hi = p - q;
        x.lo = (p - x.hi) - q;                  // exact where p > q
    }
    if (i == w.hot || (!(x.hi > 0.f) && x.hi == x.hi)) x = Pair{0.f, 0.f};
    return x;
}

// Sum of a segment's weights, the same in every lane.
template <class T>
__device__ __forceinline__ Pair segment_sum(const Row &w, int64_t begin, int64_t end, bool wide)
{
    Pair s[2] = {{0.f, 0.f}, {0.f, 0.f}};
    for (int64_t i0 = begin + lane_id() * 8; i0 < end; i0 += 32 * 8 * kLoads) {
        float p[kLoads][8], q[kLoads][8];
#pragma unroll
        for (int l = 0; l < kLoads; ++l) probs8<T>(w.p, i0 + l * 256, end, wide, p[l]);
        if (w.q) {
#pragma unroll
            for (int l = 0; l < kLoads; ++l) probs8<T>(w.q, i0 + l * 256, end, wide, q[l]);
        }
#pragma unroll
        for (int l = 0; l < kLoads; ++l)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j & 1].add(weight_of(w, p[l][j], q[l][j], i0 + l * 256 + j));
    }
    s[0].add(s[1]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) s[0].add(Pair{__shfl_xor_sync(0xffffffffu, s[0].hi, o), __shfl_xor_sync(0xffffffffu, s[0].lo, o)});
    return s[0].whole();
}

template <class T>
__global__ void __launch_bounds__(kVerifyThreads, 4) fm_verify_kernel(const VerifyArgs a)
{
    __shared__ Pair s_seg[kSegments];
    __shared__ Pair s_total[2];             // of the weights, of p alone (where they are zero)
    __shared__ int s_row;
    cg::cluster_group cl = cg::this_cluster();
    const int ctas = (int)cl.num_blocks(), cta = (int)cl.block_rank(), tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
    const int r = blockIdx.x / ctas;
    int begin = a.cu[r], end = a.cu[r + 1];
    const bool fits = begin >= 0 && begin <= end && end <= a.rows;
    const int n = fits ? end - begin : 0;
    if (n == 0) {                           // the whole cluster
        if (cta == 0 && tid == 0) {
            if (!fits) set_status(a.status, FM_ERR_LENGTHS);
            a.n_out[r] = 0;
            a.new_lens[r] = a.seq[r];
        }
        return;
    }
    // The row of the first refusal; every CTA looks for itself.
    if (warp == 0) {
        int row = n - 1;
        bool odd = false;
        for (int i0 = 0; i0 < n - 1; i0 += 32) {
            const int i = i0 + lane;
            bool no = false;
            if (i < n - 1) {
                const int t = a.tokens[begin + i + 1];
                const bool known = t >= 0 && t < a.V;
                no = true;
                if (known) {
                    const double p = prob<T>(a.target + (begin + i) * a.target_row, t);
                    const double q = a.draft ? (double)prob<T>(a.draft + (begin + i) * a.draft_row, t) : 1.0;
                    no = !((double)a.u_accept[begin + i] * q < p);
                }
                odd = !known;
            }
            const unsigned bits = __ballot_sync(0xffffffffu, no);
            if (bits) {
                row = i0 + __ffs(bits) - 1;
                odd = odd && i == row;
                break;
            }
        }
        if (odd && cta == 0) set_status(a.status, FM_ERR_PROBS);
        if (lane == 0) s_row = row;
    }
    __syncthreads();
    const int kept = s_row;
    const int64_t row = begin + kept;
    Row w{a.target + row * a.target_row, nullptr, -1};
    if (kept < n - 1) {
        if (a.draft) w.q = a.draft + row * a.draft_row;
        else w.hot = a.tokens[row + 1];
    }
    const int64_t v0 = min((int64_t)cta * a.slice, (int64_t)a.V), v1 = min(v0 + a.slice, (int64_t)a.V);
    const int segments = (int)((v1 - v0 + a.segment - 1) / a.segment);
    Pair total{0.f, 0.f}, before{0.f, 0.f}, want{0.f, 0.f};
    int owner = -1;                         // the CTA whose slice holds the border
    // Once, and a second time with p alone where the weights are all zero.
    for (int go = 0; go < 2; ++go) {
        for (int x = warp; x < segments; x += kVerifyWarps) {
            const int64_t b = v0 + (int64_t)x * a.segment;
            const Pair t = segment_sum<T>(w, b, min(b + a.segment, v1), a.wide);
            if (lane == 0) s_seg[x] = t;
        }
        __syncthreads();
        if (warp == 0) {
            Pair t{0.f, 0.f};
            for (int x = lane; x < segments; x += 32) t.add(s_seg[x]);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) t.add(Pair{__shfl_xor_sync(0xffffffffu, t.hi, o), __shfl_xor_sync(0xffffffffu, t.lo, o)});
            if (lane == 0) s_total[go] = t.whole();
        }
        cl.sync();
        // Lane c: the slice of CTA c.  (The last one with any weight, if rounding or a number outside [0, 1) leaves the
        // border behind all.)
        Pair part{0.f, 0.f};
        if (lane < ctas) part = *cl.map_shared_rank(&s_total[go], lane);
        const Pair upto = part.upto();
        total = upto.whole().from(31);
        const float u = __ldg(a.u_sample + r);
        want.hi = u * total.hi;
        want.lo = fmaf(u, total.hi, -want.hi) + u * total.lo;
        want = want.whole();
        const unsigned past = __ballot_sync(0xffffffffu, part.hi > 0.f && upto.whole().above(want)), any = __ballot_sync(0xffffffffu, part.hi > 0.f);
        owner = past ? __ffs(past) - 1 : any ? 31 - __clz(any) : -1;
        before = owner > 0 ? upto.from(max(owner - 1, 0)) : Pair{0.f, 0.f};
        if (total.hi != 0.f || (!w.q && w.hot < 0)) break;
        w.q = nullptr;
        w.hot = -1;
    }
    const bool usable = total.hi > 0.f && total.hi < INFINITY && owner >= 0;
    if (cta == 0) {
        for (int i = tid; i < n; i += kVerifyThreads)
            if (i != kept) a.out[begin + i] = i < kept ? a.tokens[begin + i + 1] : -1;
        if (tid == 0) {
            a.n_out[r] = kept + 1;
            a.new_lens[r] = a.seq[r] - n + kept + 1;
            if (!usable) {
                a.out[row] = -1;
                set_status(a.status, FM_ERR_PROBS);
            }
        }
    }
    if (usable && cta == owner && warp == 0) {
        // The segment that holds the border, then the token, a warp's width at a time.
        Pair run = before;
        int seg = 0;
        bool found = false;
        for (int x0 = 0; x0 < segments && !found; x0 += 32) {
            const Pair mine = x0 + lane < segments ? s_seg[x0 + lane] : Pair{0.f, 0.f};
            Pair upto = mine.upto();
            upto.add(run);
            const unsigned past = __ballot_sync(0xffffffffu, mine.hi > 0.f && upto.whole().above(want)), any = __ballot_sync(0xffffffffu, mine.hi > 0.f);
            const int at = past ? __ffs(past) - 1 : any ? 31 - __clz(any) : -1;
            found = past != 0;
            if (at >= 0) {
                seg = x0 + at;
                const Pair b = upto.from(max(at - 1, 0));
                before = at > 0 ? b : run;
            }
            run = upto.from(31);
        }
        const int64_t b = v0 + (int64_t)seg * a.segment, e = min(b + a.segment, v1);
        int64_t token = b;
        run = before;
        found = false;
        for (int64_t i0 = b; i0 < e && !found; i0 += 256) {
            const int64_t i = i0 + lane * 8;
            float p[8], q[8];
            probs8<T>(w.p, i, e, a.wide, p);
            if (w.q) probs8<T>(w.q, i, e, a.wide, q);
            Pair x[8], sum{0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = weight_of(w, p[j], q[j], i + j);
                sum.add(x[j]);
            }
            const Pair upto = sum.upto();
            Pair here{__shfl_up_sync(0xffffffffu, upto.hi, 1), __shfl_up_sync(0xffffffffu, upto.lo, 1)};
            if (lane == 0) here = Pair{0.f, 0.f};
            here.add(run);
            int first = -1, last = -1;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                here.add(x[j]);
                if (x[j].hi > 0.f) {
                    last = j;
                    if (first < 0 && here.whole().above(want)) first = j;
                }
            }
            const unsigned past = __ballot_sync(0xffffffffu, first >= 0), any = __ballot_sync(0xffffffffu, last >= 0);
            found = past != 0;
            if (any) {
                const int at = past ? __ffs(past) - 1 : 31 - __clz(any);
                token = i0 + at * 8 + __shfl_sync(0xffffffffu, past ? first : last, at);
            }
            run.add(upto.from(31));
        }
        if (lane == 0) a.out[row] = (int)token;
    }
    cl.sync();                              // the others have read this CTA's sums
}

}  // namespace
}  // namespace fm

using namespace fm;

extern "C" fm_status fm_verify_drafts(const void *target, int64_t target_row, const void *draft, int64_t draft_row, int dtype, int V, int rows,
                                      const int32_t *tokens, const float *u_accept, const float *u_sample, const int32_t *cu_q,
                                      const int32_t *seq_lens, int requests, int32_t *out, int32_t *n_out, int32_t *new_lens,
                                      int32_t *dev_status, fm_stream_t stream)
{
    if (dtype != FM_DT_BF16 && dtype != FM_DT_F32) return FM_ERR_INVALID_ARG;
    const int64_t esz = dtype == FM_DT_F32 ? 4 : 2;
    if (requests <= 0 || rows < 0 || V <= 0 || (uintptr_t)target % esz || (uintptr_t)draft % esz) return FM_ERR_INVALID_ARG;
    if (target_row < V || (draft && draft_row < V) || target_row > ((int64_t)1 << 38) || draft_row > ((int64_t)1 << 38)) return FM_ERR_INVALID_ARG;
    // (A step without rows has no place for them.)
    if (rows > 0 && (!target || !aligned4(tokens) || !aligned4(u_accept) || !aligned4(out))) return FM_ERR_INVALID_ARG;
    if (!aligned4(u_sample) || !aligned4(cu_q) || !aligned4(seq_lens) || !aligned4(n_out) || !aligned4(new_lens) || !aligned4(dev_status))
        return FM_ERR_INVALID_ARG;
    if (requests > kMaxRequests || rows > (1 << 24) || V > (1 << 24)) return FM_ERR_UNSUPPORTED;
    const fm_status st = device_ok();
    if (st != FM_OK) return st;
    VerifyArgs a{};
    a.target = (const uint8_t *)target;
    a.draft = (const uint8_t *)draft;
    a.target_row = target_row * esz;
    a.draft_row = draft_row * esz;
    a.tokens = tokens;
    a.cu = cu_q;
    a.seq = seq_lens;
    a.u_accept = u_accept;
    a.u_sample = u_sample;
    a.out = out;
    a.n_out = n_out;
    a.new_lens = new_lens;
    a.status = dev_status;
    a.V = V;
    a.rows = rows;
    a.R = requests;
    int ctas = 1;
    while (ctas < kVerifyCluster && V > 2048 * ctas) ctas *= 2;
    a.slice = ((V + ctas - 1) / ctas + 7) / 8 * 8;
    a.segment = kSegment * ((a.slice + kSegment * kSegments - 1) / (kSegment * kSegments));
    a.wide = aligned16(target) && a.target_row % 16 == 0 && (!draft || (aligned16(draft) && a.draft_row % 16 == 0));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(requests * ctas));
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    ProfScope ps(kKVerify, stream);
    const cudaError_t e = esz == 4 ? cudaLaunchKernelEx(&cfg, fm_verify_kernel<float>, a) : cudaLaunchKernelEx(&cfg, fm_verify_kernel<uint16_t>, a);
    return e == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}
