// spec_pages.cu -- host layer and C ABI of the page operators: argument checks
// and launch shapes.  Nothing here allocates, synchronises or keeps state
// between calls.
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/specverify.h"
#include "sv_pages.cuh"

namespace sv {
namespace {

constexpr int kClusterMost = 8;
constexpr int kBlocksMost = 152;

sv_status check_pool(const sv_kv_pool* p, const int32_t* kv_len, int32_t* held_out, int32_t* free_count_out, uint32_t* errors,
                     PoolArgs* a)
{
    if (!p || p->B < 0 || p->max_pages < 1 || p->capacity < 0)
        return SV_ERR_INVALID_ARG;
    if (p->page_size < 8 || p->page_size > 1024 || (p->page_size & (p->page_size - 1)) ||
        (long long)p->max_pages * p->page_size > 0x7fff0000LL)
        return SV_ERR_UNSUPPORTED;
    if (p->B == 0)
        return SV_OK;
    if (!p->page_table || !p->held || !p->free_pages || !p->free_count || !kv_len || !held_out || !free_count_out)
        return SV_ERR_INVALID_ARG;
    if (((uintptr_t)p->page_table | (uintptr_t)p->held | (uintptr_t)p->free_pages | (uintptr_t)p->free_count | (uintptr_t)kv_len |
         (uintptr_t)held_out | (uintptr_t)free_count_out | (uintptr_t)errors) & 3)
        return SV_ERR_INVALID_ARG;
    a->table = p->page_table;
    a->kv_len = kv_len;
    a->held = p->held;
    a->stack = p->free_pages;
    a->free_count = p->free_count;
    a->held_out = held_out;
    a->free_out = free_count_out;
    a->err = errors;
    a->has_err = errors != nullptr;
    a->B = p->B;
    a->max_pages = p->max_pages;
    a->page_shift = __builtin_ctz(p->page_size);
    a->capacity = p->capacity;
    return SV_OK;
}

// One cluster while `items` (pages and slots) are few, else up to a block an SM,
// with the in-place updates in a launch of their own.
template <typename K> sv_status launch_pages(K kernel, PoolArgs a, long long items, cudaStream_t st)
{
    const long long per = 4 * kPageThreads;
    int blocks = (int)std::min<long long>(kBlocksMost, std::max<long long>(1, (items + per - 1) / per));
    const bool in_place = a.held_out == a.held || a.free_out == a.free_count;
    a.work = 1;
    a.clustered = in_place && blocks > 1 && blocks <= kClusterMost;
    a.update = !in_place || blocks <= kClusterMost;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kPageThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)blocks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = a.clustered ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess)
        return SV_ERR_CUDA;
    if (!a.update) {
        a.work = 0;
        a.update = 1;
        kernel<<<1, kPageThreads, 0, st>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace
}  // namespace sv

extern "C" {

sv_status spec_kv_reserve(const sv_kv_pool* pool, const int32_t* kv_len, const int32_t* n_new, const int32_t* row_start, int32_t S,
                          int32_t rows, int32_t* held_out, int32_t* free_count_out, int64_t* slots, uint32_t* errors,
                          cudaStream_t stream)
{
    sv::PoolArgs a{};
    const sv_status st = sv::check_pool(pool, kv_len, held_out, free_count_out, errors, &a);
    if (st != SV_OK)
        return st;
    const bool packed = row_start != nullptr;
    if (packed ? (n_new != nullptr || rows < 0) : (S < 0 || (long long)pool->B * S != rows))
        return SV_ERR_INVALID_ARG;
    if (pool->B == 0)
        return SV_OK;
    if ((((uintptr_t)n_new | (uintptr_t)row_start) & 3) || ((uintptr_t)slots & 7))
        return SV_ERR_INVALID_ARG;
    a.n_new = n_new;
    a.row_start = row_start;
    a.slots = reinterpret_cast<long long*>(slots);
    a.S = S;
    a.rows = rows;
    a.has_n = n_new != nullptr;
    a.packed = packed;
    a.has_slots = slots != nullptr;
    a.slots16 = ((uintptr_t)slots & 15) == 0;
    // By fours and one by one: 2000003 rows 13.3 and 19.9 us, 131072 6.8 and 9.4, 15360 6.7
    // and 9.2, 4000 6.5 and 6.8, 1000 6.4 and 5.5.  (Fours would pay from some 4000 rows on.)
    a.each = rows >= 1 << 17 ? 4 : 1;
    const long long pages = rows / pool->page_size + pool->B;   // about: what the tokens need
    return sv::launch_pages(sv::sv_reserve_kernel, a, pages + (slots ? rows : 0), stream);
}

sv_status spec_kv_release(const sv_kv_pool* pool, const int32_t* kv_len, int32_t* held_out, int32_t* free_count_out,
                          uint32_t* errors, cudaStream_t stream)
{
    sv::PoolArgs a{};
    const sv_status st = sv::check_pool(pool, kv_len, held_out, free_count_out, errors, &a);
    if (st != SV_OK || pool->B == 0)
        return st;
    return sv::launch_pages(sv::sv_release_kernel, a, (long long)pool->B * pool->max_pages / 8, stream);
}

}  // extern "C"
