// Attention weight that the cached keys of a step's requests receive:
//
//   weights[key] (+)= sum over rows and query heads that attend the key of exp(scale q.k - lse)
//
// The plain form: a block of 128 keys of a (request, KV head), thread = key, K as fp32 in shared memory, the rows that
// attend them one after the other.  Bound by shared-memory reads (one per product).
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "fm_paged.h"
#include "fm_ptx.cuh"

namespace fm {
namespace {

struct WeighArgs {
    PagedArgs p;
    const uint8_t *k;
    int64_t k_page, k_head, k_tok;      // bytes
    float *weights;
    const float *lse;
};

template <int D, bool FP8>
__global__ void __launch_bounds__(128) fm_paged_weigh_kernel(const WeighArgs w)
{
    extern __shared__ float sh[];       // [128][D + 1] keys, [D] a query
    float *s_q = sh + 128 * (D + 1);
    const PagedArgs &a = w.p;
    const PagedShape &s = a.s;
    const PagedHeader *hd = reinterpret_cast<const PagedHeader *>(a.plan);
    if (!paged_plan_fits(hd, s) || hd->rows > a.rows) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, !paged_plan_fits(hd, s) ? FM_ERR_PLAN_MISMATCH : FM_ERR_LENGTHS);
        return;
    }
    const int G = s.Hq / s.Hkv, tid = threadIdx.x;
    const float kd = FP8 ? *a.k_descale : 1.f;
    int64_t base = 0;
    for (int list = 0; list < 2; ++list) {
        const PagedEntry *entries = reinterpret_cast<const PagedEntry *>(a.plan + (list ? a.L.off_many : a.L.off_few));
        for (int e = 0; e < (list ? hd->n_many : hd->n_few); ++e) {
            const PagedEntry en = entries[e];
            const KeyRange kr = key_range(en.ctx, en.ctx + en.n - 1, s.window, s.sink);
            const int64_t units = (int64_t)kr.n * s.Hkv;
            for (int64_t u = (blockIdx.x + gridDim.x - base % gridDim.x) % gridDim.x; u < units; u += gridDim.x) {
                const int h = (int)(u / kr.n), j = kr.tile((int)(u - (int64_t)h * kr.n)) * kKeyTile + tid;
                const int b = j / s.page_size, in = j - b * s.page_size;
                const bool any = j < en.ctx + en.n && (s.window == 0 || j > en.ctx - s.window || j < s.sink);
                int page = any ? a.table[(int64_t)en.r * s.max_pages + b] : -1;
                if (any && (unsigned)page >= (unsigned)s.num_pages) {
                    set_status(a.status, FM_ERR_PAGES);
                    page = -1;
                }
                __syncthreads();
                if (page >= 0) {
                    const uint8_t *row = w.k + page * w.k_page + h * w.k_head + in * w.k_tok;
                    for (int c = 0; c < D; ++c) {
                        float x, y;
                        if (FP8) unpack_f16x2(f16x2_of_e4m3(row[c]), x, y);
                        else x = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(row)[c] << 16);
                        sh[tid * (D + 1) + c] = x * kd;
                    }
                }
                float sum = 0.f;
                for (int i = 0; i < en.n * G; ++i) {
                    const int t = i / G, hq = h * G + i % G;
                    __syncthreads();
                    for (int c = tid; c < D; c += 128)
                        s_q[c] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(a.q + (en.tok0 + t) * a.q_tok + hq * a.q_head)[c] << 16);
                    __syncthreads();
                    const int p = en.ctx + t;
                    if (page < 0 || j > p || !(s.window == 0 || j > p - s.window || j < s.sink)) continue;
                    float x = 0.f;
                    for (int c = 0; c < D; ++c) x += s_q[c] * sh[tid * (D + 1) + c];
                    sum += exp2f(x * a.scale_log2 - w.lse[(int64_t)(en.tok0 + t) * s.Hq + hq] * 1.4426950408889634f);
                }
                if (page < 0) continue;
                float *at = w.weights + ((int64_t)page * s.Hkv + h) * s.page_size + in;
                if (j < en.ctx) red_add_f32(at, sum);
                else *at = sum;
            }
            base += units;
        }
    }
}

template <int D, bool FP8>
fm_status launch(const WeighArgs &w, cudaStream_t stream)
{
    constexpr int kBytes = (128 * (D + 1) + D) * 4;
    static std::atomic<uint8_t> done[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FM_ERR_CUDA;
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(fm_paged_weigh_kernel<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes) != cudaSuccess) return FM_ERR_CUDA;
        done[dev].store(1, std::memory_order_release);
    }
    ProfScope ps(kKPagedWeighFew, stream);
    fm_paged_weigh_kernel<D, FP8><<<kPagedCtas * 3, 128, kBytes, stream>>>(w);
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
    if (rows < 0 || !rows_ok(q, q_tok, q_head) || !aligned4(lse) || !aligned4(weights) || !aligned4(block_table) || !aligned4(dev_status))
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
    a.scale_log2 = scale * 1.4426950408889634f;
    a.rows = rows;
    w.lse = lse;
    w.weights = weights;
    w.k = (const uint8_t *)cache->k;
    w.k_page = cache->k_page * esz, w.k_head = cache->k_head * esz, w.k_tok = cache->k_tok * esz;
    cudaStream_t cs = (cudaStream_t)stream;
    if (a.s.d == 128) return fp8 ? launch<128, true>(w, cs) : launch<128, false>(w, cs);
    return fp8 ? launch<64, true>(w, cs) : launch<64, false>(w, cs);
}
