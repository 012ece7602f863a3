// spec_filter.cu -- host layer and C ABI of filtered sampling and filtered
// logits: argument checks, launch shapes.  Nothing here allocates,
// synchronises or keeps state between calls.
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/specverify.h"
#include "sv_filter.cuh"

namespace sv {
namespace {

sv_status check_rows(const void* logits, sv_dtype dtype, const float* temperature, const int32_t* top_k, const float* top_p,
                     const float* min_p, int32_t B, int32_t S, int32_t V, FilterArgs* a)
{
    if (B < 0 || S < 1 || V < 1 || (dtype != SV_DTYPE_F32 && dtype != SV_DTYPE_BF16))
        return SV_ERR_INVALID_ARG;
    if (V > sv_max_vocab(dtype) || (long long)B * S > 0x3fffffffLL)
        return SV_ERR_UNSUPPORTED;
    if (B == 0)
        return SV_OK;
    if (!logits || !temperature || ((uintptr_t)logits & (dtype == SV_DTYPE_BF16 ? 1 : 3)) ||
        (((uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p | (uintptr_t)min_p) & 3))
        return SV_ERR_INVALID_ARG;
    a->logits = logits;
    a->temperature = temperature;
    a->top_k = top_k;
    a->top_p = top_p;
    a->min_p = min_p;
    a->has_k = top_k != nullptr;
    a->has_p = top_p != nullptr;
    a->has_m = min_p != nullptr;
    a->B = B;
    a->S = S;
    a->V = V;
    return SV_OK;
}

// CTAs a row is spread over: one for each SM at most while the rows alone are
// fewer, 56 KB or more each; of long rows half that each, once half the SMs do.
// More and smaller parts read faster and then wait for one another more often.
// By this rule and by others: one row of 128256 bf16, top-p alone, 26 us by eight CTAs, 28
// by four, 32 by one; 16 rows of 151936 fp32 57 by eight, 47 by four, 62 by two, 86 by one;
// 37 rows of 50257 bf16 22 by one, 26 by two; 145 rows of 32003 fp32 35 and 45; 256 rows
// of 151936 fp32 154 and 182.
int row_ctas(long long rows, long long row_bytes, int nsm)
{
    int C = 1;
    while (C < kClusterMost && ((rows * 2 * C <= nsm && row_bytes / C >= (112 << 10)) ||
                                (C > 1 && rows * 4 * C <= nsm && row_bytes / C >= (56 << 10))))
        C *= 2;
    return C;
}

template <typename T, bool DRAW, int NT> cudaError_t launch(FilterArgs& a, cudaStream_t st)
{
    int dev = 0, nsm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    static std::atomic<unsigned long long> ready{0};   // devices whose limit has been raised
    if (dev >= 64 || !((ready.load(std::memory_order_relaxed) >> dev) & 1)) {
        e = cudaFuncSetAttribute(sv_filter_kernel<T, DRAW, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)filter_smem_bytes<NT>(kGroupsMost<NT>));
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    const long long rows = (long long)a.B * a.S;
    a.C = row_ctas(rows, (long long)a.V * sizeof(T), nsm);
    const int vectors = a.V / Elem<T>::E / a.C + 1, per = kGroup * NT;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(rows * a.C));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = filter_smem_bytes<NT>((vectors + per - 1) / per);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)a.C;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = a.C > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, sv_filter_kernel<T, DRAW, NT>, a);
}

template <bool DRAW> sv_status launch_rows(FilterArgs& a, sv_dtype dtype, cudaStream_t st)
{
    const bool small = a.V <= kShortMost;
    cudaError_t e;
    if (dtype == SV_DTYPE_BF16)
        e = small ? launch<__nv_bfloat16, DRAW, kShortThreads>(a, st) : launch<__nv_bfloat16, DRAW, kThreadsOf<__nv_bfloat16>>(a, st);
    else
        e = small ? launch<float, DRAW, kShortThreads>(a, st) : launch<float, DRAW, kThreadsOf<float>>(a, st);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace
}  // namespace sv

extern "C" {

sv_status spec_sample_filtered(const void* logits, sv_dtype dtype, const float* uniforms, const float* temperature,
                               const int32_t* top_k, const float* top_p, const float* min_p, int32_t B, int32_t V,
                               int32_t* out_tokens, float* out_prob, int32_t* out_kept, cudaStream_t stream)
{
    sv::FilterArgs a{};
    const sv_status st = sv::check_rows(logits, dtype, temperature, top_k, top_p, min_p, B, 1, V, &a);
    if (st != SV_OK || B == 0)
        return st;
    if (!uniforms || !out_tokens || (((uintptr_t)uniforms | (uintptr_t)out_tokens | (uintptr_t)out_prob | (uintptr_t)out_kept) & 3))
        return SV_ERR_INVALID_ARG;
    a.uniforms = uniforms;
    a.out_tokens = out_tokens;
    a.out_prob = out_prob;
    a.out_kept = out_kept;
    a.has_prob = out_prob != nullptr;
    a.has_kept = out_kept != nullptr;
    return sv::launch_rows<true>(a, dtype, stream);
}

sv_status spec_filter_logits(const void* logits, sv_dtype dtype, const float* temperature, const int32_t* top_k,
                             const float* top_p, const float* min_p, int32_t B, int32_t S, const int32_t* n_rows, int32_t V,
                             void* out, int32_t* out_kept, cudaStream_t stream)
{
    sv::FilterArgs a{};
    const sv_status st = sv::check_rows(logits, dtype, temperature, top_k, top_p, min_p, B, S, V, &a);
    if (st != SV_OK || B == 0)
        return st;
    const size_t elem = dtype == SV_DTYPE_BF16 ? 2 : 4, bytes = (size_t)B * S * V * elem;
    const uintptr_t x = (uintptr_t)logits, y = (uintptr_t)out;
    if (!out || y % elem || (((uintptr_t)n_rows | (uintptr_t)out_kept) & 3) || (x != y && x < y + bytes && y < x + bytes))
        return SV_ERR_INVALID_ARG;
    a.out = out;
    a.n_rows = n_rows;
    a.out_kept = out_kept;
    a.has_n = n_rows != nullptr;
    a.has_kept = out_kept != nullptr;
    a.same_phase = (x & 15) == (y & 15);
    return sv::launch_rows<false>(a, dtype, stream);
}

}  // extern "C"
