// Rotary positions: the frequency table (host), the turning of a training batch's queries or keys and of
// their gradients, and of a serving step's rows on their way into the paged cache.
//
//   a' = m (a cos phi - b sin phi),  b' = m (b cos phi + a sin phi),  phi = p theta_i;  back: phi -> -phi.
//
// An angle matters modulo a turn, so theta_i / 2 pi is held as a 64-bit fraction f of a turn and
// p f is taken modulo 2^64 by the multiplication itself, exactly, and its upper 32 bits used.  f comes from doubles, off by
// under 2^-54.5 turns, which p multiplies: with the cut to 32 bits the angle is within 2^-30 turns below 2^24 positions, and
// within 2^-23 at the last int32 (p theta_i in fp32 is off by 2^-4 radians, 2^-7 turns, at 1M).
//
// A thread owns four pairs (eight elements) of a token, has their sine and cosine in
// registers, and walks heads with four loads of 16 bytes in flight: they are computed once per
// token and pair, whatever the number of heads.  Bound by HBM: each element is read and written once.
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "fm_paged.h"
#include "fm_ptx.cuh"

namespace fm {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kInFlight = 4;        // heads whose loads are in flight together

struct Turn {
    float c[4], s[4];
};

// m cos and m sin of pairs 4u .. 4u + 3 at position pos.
__device__ __forceinline__ Turn turn_of(const uint64_t *turns, int u, int pos, float m, bool inverse)
{
    const ulonglong2 x = __ldg(reinterpret_cast<const ulonglong2 *>(turns) + 2 * u), y = __ldg(reinterpret_cast<const ulonglong2 *>(turns) + 2 * u + 1);
    const uint64_t f[4] = {x.x, x.y, y.x, y.y};
    Turn t;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // In 2^-32 turns: the nearest quarter, taken off as an integer, and what is left, which 24 bits hold to 2^-28 turns.
        const uint32_t a = (uint32_t)((f[i] * (uint64_t)(uint32_t)pos) >> 32), quarter = (a + (1u << 29)) >> 30;
        float s, c;
        sincospif((float)(int32_t)(a - (quarter << 30)) * 0x1p-31f, &s, &c);
        t.c[i] = (quarter & 1 ? s : c) * ((quarter + 1) & 2 ? -m : m);
        t.s[i] = (quarter & 1 ? c : s) * (((quarter & 2) != 0) != inverse ? -m : m);
    }
    return t;
}

__device__ __forceinline__ void turn(const Turn &t, float (&a)[4], float (&b)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = a[i] * t.c[i] - b[i] * t.s[i];
        b[i] = b[i] * t.c[i] + a[i] * t.s[i];
        a[i] = x;
    }
}

// Eight elements of a row as two groups of four, lo and hi: of a turned unit the a and b
// of the halves form, else neighbours in memory.
struct Bf8 {
    uint2 lo, hi;
};
struct F8 {
    float4 lo, hi;
};
template <class T>
using Raw = typename std::conditional<sizeof(T) == 2, Bf8, F8>::type;

template <class T>
__device__ __forceinline__ Raw<T> load8(const uint8_t *row, int at_lo, int at_hi)
{
    using V = decltype(Raw<T>::lo);
    Raw<T> r;
    r.lo = *reinterpret_cast<const V *>(row + at_lo * (int)sizeof(T));
    r.hi = *reinterpret_cast<const V *>(row + at_hi * (int)sizeof(T));
    return r;
}
__device__ __forceinline__ void values(const Bf8 &r, float (&x)[8])
{
    const uint32_t w[4] = {r.lo.x, r.lo.y, r.hi.x, r.hi.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void values(const F8 &r, float (&x)[8])
{
    x[0] = r.lo.x, x[1] = r.lo.y, x[2] = r.lo.z, x[3] = r.lo.w;
    x[4] = r.hi.x, x[5] = r.hi.y, x[6] = r.hi.z, x[7] = r.hi.w;
}
__device__ __forceinline__ void of_values(const float (&x)[8], Bf8 &r)
{
    r.lo = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    r.hi = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void of_values(const float (&x)[8], F8 &r)
{
    r.lo = make_float4(x[0], x[1], x[2], x[3]);
    r.hi = make_float4(x[4], x[5], x[6], x[7]);
}
template <class T>
__device__ __forceinline__ void store8(uint8_t *row, int at_lo, int at_hi, const Raw<T> &r)
{
    using V = decltype(Raw<T>::lo);
    *reinterpret_cast<V *>(row + at_lo * (int)sizeof(T)) = r.lo;
    *reinterpret_cast<V *>(row + at_hi * (int)sizeof(T)) = r.hi;
}

// The unit's eight values turned, as they lie in memory.
template <bool INTER>
__device__ __forceinline__ void turn8(const Turn &t, float (&x)[8])
{
    float a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = INTER ? x[2 * i] : x[i];
        b[i] = INTER ? x[2 * i + 1] : x[4 + i];
    }
    turn(t, a, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (INTER) x[2 * i] = a[i], x[2 * i + 1] = b[i];
        else x[i] = a[i], x[4 + i] = b[i];
    }
}

struct RopeArgs {
    const uint8_t *x;
    uint8_t *y;
    int64_t x_batch, x_head, x_tok, y_batch, y_head, y_tok;     // bytes
    const int32_t *pos;
    int64_t pos_batch;
    const uint64_t *turns;
    float m;
    int32_t N, H, heads;            // heads per thread
    int32_t units, shift;           // units that are turned; log2 of the units of a row
    int32_t inverse, in_place;
};

// (float4 stands for fp32, uint16_t for bf16 elements: types of 4 and 2 bytes.)
template <class IN, class OUT, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) fm_rope_kernel(const RopeArgs a)
{
    const int u = threadIdx.x & ((1 << a.shift) - 1);
    const int64_t n = (int64_t)blockIdx.x * (kRopeThreads >> a.shift) + (threadIdx.x >> a.shift);
    if (n >= a.N) return;
    const int pos = __ldg(a.pos + blockIdx.z * a.pos_batch + n);
    const bool turned = u < a.units;
    if (pos < 0 || (!turned && a.in_place)) return;
    Turn t;
    if (turned) t = turn_of(a.turns, u, pos, a.m, a.inverse);
    const int lo = turned && !INTER ? 4 * u : 8 * u, hi = turned && !INTER ? 4 * (a.units + u) : 8 * u + 4;
    const int h0 = blockIdx.y * a.heads, h1 = min(h0 + a.heads, a.H);
    const uint8_t *x = a.x + blockIdx.z * a.x_batch + n * a.x_tok + h0 * a.x_head;
    uint8_t *y = a.y + blockIdx.z * a.y_batch + n * a.y_tok + h0 * a.y_head;
    for (int h = h0; h < h1; h += kInFlight) {
        Raw<IN> r[kInFlight];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i)
            if (h + i < h1) r[i] = load8<IN>(x + i * a.x_head, lo, hi);
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            if (h + i >= h1) break;
            if constexpr (sizeof(IN) == sizeof(OUT)) {
                if (!turned) {          // the same bits
                    store8<OUT>(y + i * a.y_head, lo, hi, r[i]);
                    continue;
                }
            }
            float v[8];
            values(r[i], v);
            if (turned) turn8<INTER>(t, v);
            Raw<OUT> w;
            of_values(v, w);
            store8<OUT>(y + i * a.y_head, lo, hi, w);
        }
        x += kInFlight * a.x_head;
        y += kInFlight * a.y_head;
    }
}

struct AppendRopeArgs {
    const uint8_t *in[3];                        // q, k, v: bf16; strides in bytes
    int64_t tok[3], head[3];
    uint8_t *out[3];                             // q's rows, the caches of K and V
    int64_t q_tok, kv_page[2], kv_tok[2], out_head[3];
    const int64_t *slots;
    const int32_t *pos;
    const uint64_t *turns;
    const float *descale[2];
    float m;
    int64_t n_slots;
    int32_t page_size, T, Hq, Hkv;
    int32_t rows;                                // rows of a token (Hq + 2 Hkv) per thread
    int32_t units, shift, q_in_place;
    int32_t *status;
};

// Rows of a token in one line: its query heads, its key heads, its value heads.  (Held to 64 registers, four blocks a SM: 48 us
// for 69 with the 80 that it would take, chunks of 10,000 rows to an e4m3 cache, although 64 bytes are spilled there.)
template <bool FP8, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 4) fm_paged_append_rope_kernel(const AppendRopeArgs a)
{
    const int u = threadIdx.x & ((1 << a.shift) - 1);
    const int64_t t = (int64_t)blockIdx.x * (kRopeThreads >> a.shift) + (threadIdx.x >> a.shift);
    if (t >= a.T) return;
    const int r0 = blockIdx.y * a.rows, r1 = min(r0 + a.rows, a.Hq + 2 * a.Hkv);
    const int pos = __ldg(a.pos + t);
    const int64_t slot = r1 > a.Hq ? __ldg(a.slots + t) : -1;
    if (pos < 0) return;
    const bool turned = u < a.units;
    const bool inside = slot >= 0 && slot < a.n_slots;
    if (slot >= a.n_slots) set_status(a.status, FM_ERR_PAGES);
    int64_t at[2] = {0, 0};
    if (inside) {
        const int64_t page = slot <= INT32_MAX ? (int64_t)((uint32_t)slot / (uint32_t)a.page_size) : slot / a.page_size;
        const int64_t in = slot - page * a.page_size;
        at[0] = page * a.kv_page[0] + in * a.kv_tok[0];
        at[1] = page * a.kv_page[1] + in * a.kv_tok[1];
    }
    const int lo = turned && !INTER ? 4 * u : 8 * u, hi = turned && !INTER ? 4 * (a.units + u) : 8 * u + 4;
    Turn ang;
    if (turned && r0 < a.Hq + a.Hkv) ang = turn_of(a.turns, u, pos, a.m, false);
    // Heads [h0, h1) of q (kind 0), k (1) or v (2).
    auto heads = [&](auto kind_of, int h0, int h1) {
        constexpr int K = decltype(kind_of)::value;
        const bool tu = turned && K < 2;
        if (h0 >= h1 || (K > 0 && !inside) || (K == 0 && !turned && a.q_in_place)) return;
        const int l = K == 2 ? 8 * u : lo, g = K == 2 ? 8 * u + 4 : hi;
        const Divisor ds(K > 0 && FP8 ? __ldg(a.descale[K > 0 ? K - 1 : 0]) : 1.f);
        const int64_t step_in = a.head[K], step_out = a.out_head[K];
        const uint8_t *x = a.in[K] + t * a.tok[K] + h0 * step_in;
        uint8_t *y = a.out[K] + (K == 0 ? t * a.q_tok : at[K > 0 ? K - 1 : 0]) + h0 * step_out;
        for (int h = h0; h < h1; h += kInFlight) {
            Bf8 r[kInFlight];
#pragma unroll
            for (int i = 0; i < kInFlight; ++i)
                if (h + i < h1) r[i] = load8<uint16_t>(x + i * step_in, l, g);
#pragma unroll
            for (int i = 0; i < kInFlight; ++i) {
                if (h + i >= h1) break;
                float v[8];
                values(r[i], v);
                if (tu) turn8<INTER>(ang, v);
                if constexpr (K > 0 && FP8) {
                    uint32_t w[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        w[j] = pack_e4m3x2(ds(v[4 * j]), ds(v[4 * j + 1])) | pack_e4m3x2(ds(v[4 * j + 2]), ds(v[4 * j + 3])) << 16;
                    *reinterpret_cast<uint32_t *>(y + i * step_out + l) = w[0];
                    *reinterpret_cast<uint32_t *>(y + i * step_out + g) = w[1];
                } else {
                    Bf8 w = r[i];               // the same bits where nothing turns
                    if (tu) of_values(v, w);
                    store8<uint16_t>(y + i * step_out, l, g, w);
                }
            }
            x += kInFlight * step_in;
            y += kInFlight * step_out;
        }
    };
    heads(std::integral_constant<int, 0>{}, r0, min(r1, a.Hq));
    heads(std::integral_constant<int, 1>{}, max(r0 - a.Hq, 0), min(r1 - a.Hq, a.Hkv));
    heads(std::integral_constant<int, 2>{}, max(r0 - a.Hq - a.Hkv, 0), r1 - a.Hq - a.Hkv);
}

bool rotary_ok(const fm_rotary *r) { return r && aligned16(r->turns) && r->rot > 0 && std::isfinite(r->magnitude); }

// Whether no two rows of d elements share memory: going up the strides, each is at least what lies below it.
bool rows_apart(int dims, const int64_t *stride, const int *size, int d)
{
    int64_t below = d;
    for (unsigned done = 0; done != (1u << dims) - 1u;) {
        int least = -1;
        for (int i = 0; i < dims; ++i)
            if (!(done >> i & 1u) && (least < 0 || stride[i] < stride[least])) least = i;
        done |= 1u << least;
        if (size[least] <= 1) continue;
        if (stride[least] < below) return false;
        below = stride[least] * (size[least] - 1) + below;
    }
    return true;
}

template <class IN, class OUT>
void launch_rope(const RopeArgs &a, bool inter, dim3 grid, cudaStream_t st)
{
    if (inter) fm_rope_kernel<IN, OUT, true><<<grid, kRopeThreads, 0, st>>>(a);
    else fm_rope_kernel<IN, OUT, false><<<grid, kRopeThreads, 0, st>>>(a);
}

// Rows per thread: as many as share a thread's sines (at most `most`), but no more than
// leave the device `blocks` blocks.
int rows_per_thread(int64_t token_blocks, int rows, int most)
{
    int n = most;
    while (n > 1 && token_blocks * ((rows + n - 1) / n) < 4 * kPagedCtas) n >>= 1;
    return n;
}

}  // namespace
}  // namespace fm

using namespace fm;

extern "C" {

fm_status fm_rotary_table(const fm_rotary_spec *s, uint64_t *turns, float *magnitude)
{
    if (!s || !turns || !magnitude || s->rot < 2 || s->rot > 128 || s->rot % 2) return FM_ERR_INVALID_ARG;
    if (!(s->base > 1.0) || !std::isfinite(s->base)) return FM_ERR_INVALID_ARG;
    if (s->scaling < FM_ROPE_PLAIN || s->scaling > FM_ROPE_YARN) return FM_ERR_INVALID_ARG;
    const double f = s->scaling == FM_ROPE_PLAIN ? 1.0 : s->factor;
    if (!(f >= 1.0) || !std::isfinite(f)) return FM_ERR_INVALID_ARG;
    const bool yarn = s->scaling == FM_ROPE_YARN;
    if (yarn && (!(s->original > 0.0) || !(s->slow >= 0.0) || !(s->fast > s->slow) || !std::isfinite(s->original) || !std::isfinite(s->fast)))
        return FM_ERR_INVALID_ARG;
    if (s->scaling == FM_ROPE_NTK && s->rot == 2) return FM_ERR_INVALID_ARG;
    double base = s->base;
    if (s->scaling == FM_ROPE_NTK) base *= std::pow(f, (double)s->rot / (s->rot - 2));
    if (!std::isfinite(base)) return FM_ERR_INVALID_ARG;
    for (int i = 0; i < s->rot / 2; ++i) {
        const double theta = std::pow(base, -2.0 * i / s->rot), turn = theta / 6.283185307179586476925287;   // radians and turns per position
        double scaled = turn;
        if (s->scaling == FM_ROPE_LINEAR) scaled = turn / f;
        if (yarn) {
            double g = (s->original * turn - s->slow) / (s->fast - s->slow);
            g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
            scaled = turn * (g + (1.0 - g) / f);
        }
        turns[i] = (uint64_t)std::ldexp(scaled, 64);        // scaled <= 1 / 2 pi
    }
    *magnitude = yarn ? (float)(0.1 * std::log(f) + 1.0) : 1.f;
    return FM_OK;
}

fm_status fm_rope(const void *x, int x_dtype, fm_strides xs, const int32_t *positions, int64_t pos_batch, int B, int H, int N, int d,
                  const fm_rotary *rotary, int inverse, void *y, int y_dtype, fm_strides ys, fm_stream_t stream)
{
    fm_status st = check_shapes(B, H, N, d);
    if (st != FM_OK) return st;
    if (!rotary_ok(rotary) || !aligned16(x) || !aligned16(y) || !aligned4(positions) || pos_batch < 0) return FM_ERR_INVALID_ARG;
    if ((x_dtype != FM_DT_BF16 && x_dtype != FM_DT_F32) || (y_dtype != FM_DT_BF16 && y_dtype != FM_DT_F32)) return FM_ERR_INVALID_ARG;
    if (rotary->rot > d || rotary->rot % 8) return FM_ERR_UNSUPPORTED;
    const int xe = x_dtype == FM_DT_F32 ? 4 : 2, ye = y_dtype == FM_DT_F32 ? 4 : 2;
    for (int64_t s : {xs.batch, xs.head, xs.tok})
        if (s < 0 || s * xe % 16 || s > ((int64_t)1 << 40)) return FM_ERR_INVALID_ARG;
    for (int64_t s : {ys.batch, ys.head, ys.tok})
        if (s < 0 || s * ye % 16 || s > ((int64_t)1 << 40)) return FM_ERR_INVALID_ARG;
    const int64_t strides[3] = {ys.batch, ys.head, ys.tok};
    const int sizes[3] = {B, H, N};
    if (!rows_apart(3, strides, sizes, d)) return FM_ERR_INVALID_ARG;
    if (x == y && (x_dtype != y_dtype || xs.batch != ys.batch || xs.head != ys.head || xs.tok != ys.tok)) return FM_ERR_INVALID_ARG;
    if ((st = device_ok()) != FM_OK) return st;
    RopeArgs a{};
    a.x = (const uint8_t *)x;
    a.y = (uint8_t *)y;
    a.x_batch = xs.batch * xe, a.x_head = xs.head * xe, a.x_tok = xs.tok * xe;
    a.y_batch = ys.batch * ye, a.y_head = ys.head * ye, a.y_tok = ys.tok * ye;
    a.pos = positions;
    a.pos_batch = pos_batch;
    a.turns = rotary->turns;
    a.m = rotary->magnitude;
    a.N = N;
    a.H = H;
    a.units = rotary->rot / 8;
    a.shift = d == 128 ? 4 : 3;
    a.inverse = inverse != 0;
    a.in_place = x == y;
    const int64_t tiles = (N + (kRopeThreads >> a.shift) - 1) / (kRopeThreads >> a.shift);
    a.heads = rows_per_thread(tiles * B, H, 8);
    while ((H + a.heads - 1) / a.heads > 65535) a.heads *= 2;
    const dim3 grid((unsigned)tiles, (unsigned)((H + a.heads - 1) / a.heads), (unsigned)B);
    const bool inter = rotary->interleaved != 0;
    ProfScope ps(kKRope, stream);
    if (xe == 2 && ye == 2) launch_rope<uint16_t, uint16_t>(a, inter, grid, (cudaStream_t)stream);
    else if (xe == 2) launch_rope<uint16_t, float>(a, inter, grid, (cudaStream_t)stream);
    else if (ye == 2) launch_rope<float, uint16_t>(a, inter, grid, (cudaStream_t)stream);
    else launch_rope<float, float>(a, inter, grid, (cudaStream_t)stream);
    return cudaPeekAtLastError() == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

fm_status fm_paged_append_rope(const void *q, int64_t q_tok, int64_t q_head, int Hq, const void *k, int64_t k_tok, int64_t k_head,
                               const void *v, int64_t v_tok, int64_t v_head, const int64_t *slots, const int32_t *positions, int T,
                               const fm_rotary *rotary, const fm_paged_cache *cache, void *q_out, int64_t qo_tok, int64_t qo_head,
                               int32_t *dev_status, fm_stream_t stream)
{
    fm_status st = check_cache(cache);
    if (st != FM_OK) return st;
    if (T < 0 || T > (1 << 24) || Hq <= 0 || !rows_ok(q, q_tok, q_head) || !rows_ok(k, k_tok, k_head) || !rows_ok(v, v_tok, v_head) ||
        !rows_ok(q_out, qo_tok, qo_head) || !slots || ((uintptr_t)slots & 7u) || !aligned4(positions) || !aligned4(dev_status) || !rotary_ok(rotary))
        return FM_ERR_INVALID_ARG;
    if (Hq > 4096 || rotary->rot > cache->d || rotary->rot % 8) return FM_ERR_UNSUPPORTED;
    const int64_t strides[2] = {qo_tok, qo_head};
    const int sizes[2] = {T, Hq};
    if (!rows_apart(2, strides, sizes, cache->d)) return FM_ERR_INVALID_ARG;
    if (q == q_out && (q_tok != qo_tok || q_head != qo_head)) return FM_ERR_INVALID_ARG;
    if ((st = device_ok()) != FM_OK) return st;
    if (T == 0) return FM_OK;
    const bool fp8 = cache->dtype == FM_DT_E4M3;
    const int64_t esz = fp8 ? 1 : 2;
    AppendRopeArgs a{};
    a.in[0] = (const uint8_t *)q, a.in[1] = (const uint8_t *)k, a.in[2] = (const uint8_t *)v;
    a.tok[0] = q_tok * 2, a.tok[1] = k_tok * 2, a.tok[2] = v_tok * 2;
    a.head[0] = q_head * 2, a.head[1] = k_head * 2, a.head[2] = v_head * 2;
    a.out[0] = (uint8_t *)q_out, a.out[1] = (uint8_t *)cache->k, a.out[2] = (uint8_t *)cache->v;
    a.q_tok = qo_tok * 2;
    a.out_head[0] = qo_head * 2, a.out_head[1] = cache->k_head * esz, a.out_head[2] = cache->v_head * esz;
    a.kv_page[0] = cache->k_page * esz, a.kv_page[1] = cache->v_page * esz;
    a.kv_tok[0] = cache->k_tok * esz, a.kv_tok[1] = cache->v_tok * esz;
    a.slots = slots;
    a.pos = positions;
    a.turns = rotary->turns;
    a.descale[0] = cache->k_descale, a.descale[1] = cache->v_descale;
    a.m = rotary->magnitude;
    a.n_slots = (int64_t)cache->num_pages * cache->page_size;
    a.page_size = cache->page_size;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = cache->Hkv;
    a.units = rotary->rot / 8;
    a.shift = cache->d == 128 ? 4 : 3;
    a.q_in_place = q == q_out;
    a.status = dev_status;
    const int per = kRopeThreads >> a.shift, rows = Hq + 2 * cache->Hkv;
    const int64_t tiles = (T + per - 1) / per;
    a.rows = rows_per_thread(tiles, rows, 8);
    const dim3 grid((unsigned)tiles, (unsigned)((rows + a.rows - 1) / a.rows));
    ProfScope ps(kKPagedAppendRope, stream);
    const bool inter = rotary->interleaved != 0;
    cudaStream_t cs = (cudaStream_t)stream;
    if (fp8 && inter) fm_paged_append_rope_kernel<true, true><<<grid, kRopeThreads, 0, cs>>>(a);
    else if (fp8) fm_paged_append_rope_kernel<true, false><<<grid, kRopeThreads, 0, cs>>>(a);
    else if (inter) fm_paged_append_rope_kernel<false, true><<<grid, kRopeThreads, 0, cs>>>(a);
    else fm_paged_append_rope_kernel<false, false><<<grid, kRopeThreads, 0, cs>>>(a);
    return cudaPeekAtLastError() == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

}  // extern "C"
