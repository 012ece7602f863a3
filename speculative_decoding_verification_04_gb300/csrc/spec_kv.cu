// spec_kv.cu -- host layer and C ABI of the paged key/value cache and the
// attention over it: argument checks, launch shapes.  Nothing here allocates,
// synchronises or keeps state between calls.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "../../include/specverify.h"
#include "sv_attention.cuh"

namespace sv {
namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Positions of a sequence: the kernels' positions are ints, and step past a
// sequence's end by up to 32 pages of the largest size.
constexpr long long kMaxPositions = 0x7fff0000LL;

// The cache description, checked.  Row counts stay below 2^31 so that a row
// is an int coordinate; byte offsets are 64-bit everywhere.
sv_status check_cache(const sv_kv_cache* c, bool need_table, KvCache* out)
{
    if (!c || !c->k || !c->v || (need_table && !c->page_table) ||
        (c->format != SV_KV_BF16 && c->format != SV_KV_E4M3))
        return SV_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->n_kv_heads < 1 || c->layers < 1 || c->max_pages < 1)
        return SV_ERR_INVALID_ARG;
    if (c->format == SV_KV_E4M3 ? (!c->k_scale || !c->v_scale) : (c->k_scale || c->v_scale))
        return SV_ERR_INVALID_ARG;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale) ||
        ((uintptr_t)c->page_table & 3))
        return SV_ERR_INVALID_ARG;
    if (c->head_dim < 64 || c->head_dim > 256 || c->head_dim % 16 || c->page_size < 8 || c->page_size > 1024 ||
        (c->page_size & (c->page_size - 1)))
        return SV_ERR_UNSUPPORTED;
    if ((long long)c->num_pages * c->n_kv_heads * c->page_size > 0x7fffffffLL ||
        (long long)c->max_pages * c->page_size > kMaxPositions)
        return SV_ERR_UNSUPPORTED;
    out->k = static_cast<unsigned char*>(c->k);
    out->v = static_cast<unsigned char*>(c->v);
    out->k_scale = c->k_scale;
    out->v_scale = c->v_scale;
    out->table = c->page_table;
    out->max_pages = c->max_pages;
    out->layers = c->layers;
    out->num_pages = c->num_pages;
    out->Hkv = c->n_kv_heads;
    out->D = c->head_dim;
    out->page_shift = __builtin_ctz(c->page_size);
    return SV_OK;
}

sv_status launched(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

// Warps a token's work of `passes` warp passes is spread over: all of them
// while the tokens alone leave the GPU's SMs short of warps, one per six
// passes once there are plenty (a warp's token lookup is then shared by them:
// 16411 prompt tokens take 81.8 us, 84.8 with one per four).
int warps_per_token(int passes, long long tokens)
{
    const long long want = 152 * 16;
    const int most = std::max(1, passes), least = std::max(1, (passes + 5) / 6);
    const long long w = tokens > 0 ? (want + tokens - 1) / tokens : most;
    return (int)std::min<long long>(most, std::max<long long>(least, w));
}

template <typename T, bool E4M3>
cudaError_t launch_append(AppendArgs& a, cudaStream_t st)
{
    const int units = a.c.D / 16, lpr = units <= 4 ? 4 : units <= 8 ? 8 : 16;
    const int heads = (a.has_q ? a.Hq : 0) + 2 * a.c.Hkv, rpw = 32 / lpr;
    const int wpt = std::min(8, warps_per_token((heads + rpw - 1) / rpw, a.rows)), tpb = 8 / wpt;
    const dim3 block(32, wpt, tpb);
    const unsigned grid = (unsigned)((a.rows + tpb - 1) / tpb);
    if (lpr == 4)
        sv_append_kernel<T, 4, E4M3><<<grid, block, 0, st>>>(a);
    else if (lpr == 8)
        sv_append_kernel<T, 8, E4M3><<<grid, block, 0, st>>>(a);
    else
        sv_append_kernel<T, 16, E4M3><<<grid, block, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T, bool E4M3>
cudaError_t launch_read(ReadArgs& a, cudaStream_t st)
{
    const int units = 2 * a.c.Hkv * (a.c.D / 16);
    a.wpt = warps_per_token((units + 31) / 32, a.rows);
    const long long warps = (long long)a.rows * a.wpt;
    sv_read_kernel<T, E4M3><<<(unsigned)((warps + 7) / 8), 256, 0, st>>>(a);
    return cudaGetLastError();
}

// --- attention -------------------------------------------------------------
constexpr int kSmemMax = 232448;   // dynamic shared memory a CTA may have

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor map encoder (the library does not link the driver).
EncodeTiled tensor_map_encoder()
{
    static std::atomic<void*> found{nullptr};
    void* f = found.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            return nullptr;
        found.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

// Rows of one tensor of the cache: [num_pages * Hkv * page_size][head_dim].
bool cache_map(CUtensorMap* m, void* base, const AttnArgs& a, bool e4m3)
{
    const EncodeTiled encode = tensor_map_encoder();
    if (!encode)
        return false;
    const int elem = e4m3 ? 1 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)a.c.D, ((cuuint64_t)a.c.num_pages * a.c.Hkv) << a.c.page_shift};
    const cuuint64_t strides[1] = {(cuuint64_t)a.c.D * elem};
    const cuuint32_t box[2] = {(cuuint32_t)(e4m3 ? 128 : 64), (cuuint32_t)a.box_rows}, ones[2] = {1, 1};
    return encode(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides,
                  box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries: [B * Nmax][Hq][D], a box being one row group.
bool query_map(CUtensorMap* m, const AttnArgs& a)
{
    const EncodeTiled encode = tensor_map_encoder();
    if (!encode)
        return false;
    const cuuint64_t dims[3] = {(cuuint64_t)a.c.D, (cuuint64_t)a.Hq, (cuuint64_t)a.B * a.Nmax};
    const cuuint64_t strides[2] = {(cuuint64_t)a.c.D * 2, (cuuint64_t)(a.B * (long long)a.Nmax > 1 ? a.q_stride : (long long)a.Hq * a.c.D) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.heads, (cuuint32_t)a.nodes}, ones[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(a.q), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a key head's rows (Nmax nodes by G query heads) are spread over groups of
// at most `most`: whole nodes while a node's heads fit, evenly.
struct RowGroups {
    int nodes, heads, head_blocks, groups, rows;
};

RowGroups attention_rows(int Nmax, int G, int most)
{
    RowGroups r;
    r.head_blocks = (G + most - 1) / most;
    r.heads = (G + r.head_blocks - 1) / r.head_blocks;
    const int fit = std::max(1, most / r.heads), blocks = (Nmax + fit - 1) / fit;
    r.nodes = (Nmax + blocks - 1) / blocks;
    r.groups = blocks * r.head_blocks;
    r.rows = r.nodes * r.heads;
    return r;
}

size_t attention_part_bytes(int rows, int D) { return (size_t)2 * kAttnMaxCtas * rows * (D + 2) * 4; }

template <int NT, int NWG, bool E4M3>
cudaError_t launch_attention(AttnArgs& a, const CUtensorMap (&m)[3], int dev, int nsm, cudaStream_t st)
{
    constexpr int N = NT * NWG;
    const int q_bytes = E4M3 ? 3 * N * 128 * a.nd : N * 128 * ((a.c.D + 63) / 64);
    const int fixed = (int)sizeof(AttnShared) + (N + 63) / 64 * kHalfBytes + q_bytes;
    int room = kSmemMax - fixed;
    const int operand = a.c.D <= 64 ? kHalfBytes : 2 * kHalfBytes;   // a bf16 chunk of 128 columns
    if (E4M3) {
        a.conv = 2;
        a.conv_bytes = operand;
        a.k_bytes = a.v_bytes = kHalfBytes;
        room -= a.conv * a.conv_bytes;
    } else {
        a.conv = a.conv_bytes = 0;
        a.k_bytes = a.v_bytes = operand;
    }
    const int slots = std::min(2 * kMaxSlots, room / a.k_bytes);
    a.kslots = slots / 2;
    a.vslots = slots - a.kslots;
    const int smem = fixed + slots * a.k_bytes + a.conv * a.conv_bytes;
    static std::atomic<unsigned long long> ready{0};   // devices whose limit has been raised
    if (dev >= 64 || !((ready.load(std::memory_order_relaxed) >> dev) & 1)) {
        const cudaError_t e = cudaFuncSetAttribute(sv_attention_kernel<NT, NWG, E4M3>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
        if (e != cudaSuccess)
            return e;
        // the warpgroups share out what the block is launched with: with fewer registers they would wait for ever
        cudaFuncAttributes fa;
        const cudaError_t e2 = cudaFuncGetAttributes(&fa, sv_attention_kernel<NT, NWG, E4M3>);
        if (e2 != cudaSuccess || fa.numRegs != kAttnRegs)
            return e2 != cudaSuccess ? e2 : cudaErrorInvalidConfiguration;
        if (dev < 64)
            ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    const int ctas = std::min(nsm, kAttnMaxCtas);
    sv_attention_kernel<NT, NWG, E4M3><<<ctas, kAttnThreads, smem, st>>>(a, m[0], m[1], m[2]);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    // a page table of one tile: no item can be cut
    if (((long long)a.c.max_pages << a.c.page_shift) <= kTile)
        return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)((a.rows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sv_attention_combine, a, ctas);
}

template <bool E4M3>
cudaError_t launch_attention_rows(AttnArgs& a, const CUtensorMap (&m)[3], int dev, int nsm, cudaStream_t st)
{
    if (a.rows <= 16)
        return launch_attention<16, 1, E4M3>(a, m, dev, nsm, st);
    switch ((a.rows + 15) / 16) {
    case 2: return launch_attention<16, 2, E4M3>(a, m, dev, nsm, st);
    case 3: return launch_attention<24, 2, E4M3>(a, m, dev, nsm, st);
    case 4: return launch_attention<32, 2, E4M3>(a, m, dev, nsm, st);
    case 5: return launch_attention<40, 2, E4M3>(a, m, dev, nsm, st);
    case 6: return launch_attention<48, 2, E4M3>(a, m, dev, nsm, st);
    default: return launch_attention<64, 2, E4M3>(a, m, dev, nsm, st);
    }
}

}  // namespace
}  // namespace sv

extern "C" {

sv_status spec_kv_append(const sv_kv_cache* cache, const sv_kv_tokens* x, const int32_t* kv_len,
                         uint32_t* errors, cudaStream_t stream)
{
    if (!x)
        return SV_ERR_INVALID_ARG;
    sv::AppendArgs a{};
    sv_status st = sv::check_cache(cache, x->rows > 0, &a.c);
    if (st != SV_OK)
        return st;
    const bool packed = x->row_start != nullptr;
    if ((x->dtype != SV_DTYPE_F32 && x->dtype != SV_DTYPE_BF16) || x->B < 0 || x->rows < 0 ||
        (!packed && (x->S < 0 || (long long)x->B * x->S != x->rows)))
        return SV_ERR_INVALID_ARG;
    if (x->rows == 0)
        return SV_OK;
    const int s = x->dtype == SV_DTYPE_BF16 ? 2 : 4, D = cache->head_dim;
    if (x->B < 1 || !x->k || !x->v || !kv_len || (x->q && (!x->q_out || x->n_heads < 1)) ||
        (packed && (x->parent || x->n_new)) || (x->parent && x->S > SV_K_MAX))
        return SV_ERR_INVALID_ARG;
    if (x->cos_sin && (x->rotary_dim < 16 || x->rotary_dim > D || x->rotary_dim % 16 || x->max_positions < 1))
        return SV_ERR_INVALID_ARG;
    if (!(x->eps >= 0.0f))
        return SV_ERR_INVALID_ARG;
    const void* vec[] = {x->q, x->k, x->v, x->q_norm, x->k_norm, x->cos_sin, x->q_out};
    for (const void* p : vec)
        if (!sv::aligned16(p))
            return SV_ERR_INVALID_ARG;
    const void* word[] = {x->parent, x->n_new, x->row_start, kv_len, errors};
    for (const void* p : word)
        if ((uintptr_t)p & 3)
            return SV_ERR_INVALID_ARG;
    if ((x->q && (x->q_stride * s) % 16) || (x->k_stride * s) % 16 || (x->v_stride * s) % 16)
        return SV_ERR_INVALID_ARG;
    if (x->q && (const void*)x->q_out == x->q && x->q_stride != (long long)x->n_heads * D)
        return SV_ERR_INVALID_ARG;
    if (x->n_heads > (1 << 16) || cache->n_kv_heads > (1 << 16) ||
        (long long)x->rows * (x->n_heads + 2 * cache->n_kv_heads) > 0x3fffffffLL)
        return SV_ERR_UNSUPPORTED;
    a.q = x->q;
    a.k = x->k;
    a.v = x->v;
    a.q_stride = x->q_stride;
    a.k_stride = x->k_stride;
    a.v_stride = x->v_stride;
    a.q_norm = x->q_norm;
    a.k_norm = x->k_norm;
    a.cos_sin = x->cos_sin;
    a.parent = x->parent;
    a.n_new = x->n_new;
    a.row_start = x->row_start;
    a.kv_len = kv_len;
    a.q_out = x->q_out;
    a.err = errors;
    a.has_q = x->q != nullptr;
    a.has_qn = x->q_norm != nullptr;
    a.has_kn = x->k_norm != nullptr;
    a.has_rot = x->cos_sin != nullptr;
    a.has_parent = x->parent != nullptr;
    a.has_n = x->n_new != nullptr;
    a.packed = packed;
    a.has_err = errors != nullptr;
    a.Hq = x->n_heads;
    a.B = x->B;
    a.S = x->S;
    a.rows = x->rows;
    a.max_positions = x->max_positions;
    a.rot = x->rotary_dim;
    a.interleaved = x->interleaved != 0;
    a.eps = x->eps;
    const bool e4m3 = cache->format == SV_KV_E4M3;
    if (x->dtype == SV_DTYPE_BF16)
        return sv::launched(e4m3 ? sv::launch_append<__nv_bfloat16, true>(a, stream)
                                 : sv::launch_append<__nv_bfloat16, false>(a, stream));
    return sv::launched(e4m3 ? sv::launch_append<float, true>(a, stream) : sv::launch_append<float, false>(a, stream));
}

size_t sv_attention_workspace_size(int32_t Nmax, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim)
{
    if (Nmax < 1 || Nmax > sv::kNodeMax || n_kv_heads < 1 || n_heads < n_kv_heads || n_heads % n_kv_heads ||
        head_dim < 64 || head_dim > 256 || head_dim % 16)
        return 0;
    // the format is not known here: 128-row groups are never smaller than 64-row ones
    const int rows = sv::attention_rows(Nmax, n_heads / n_kv_heads, sv::attn_rows_max(false, head_dim)).rows;
    return (sv::kAttnMaxCtas * 8 + sv::attention_part_bytes(rows, head_dim) + 255) / 256 * 256;
}

sv_status spec_tree_attention(const sv_kv_cache* cache, const int32_t* kv_len, const int32_t* n_nodes,
                              const int32_t* parent, const void* q, int64_t q_stride, sv_dtype dtype,
                              int32_t n_heads, int32_t B, int32_t Nmax, float scale, void* out,
                              uint32_t* errors, void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    return spec_tree_attention_ex(cache, kv_len, n_nodes, parent, q, q_stride, dtype, n_heads, B, Nmax, scale, out, errors,
                                  workspace, workspace_bytes, 0, stream);
}

sv_status spec_tree_attention_ex(const sv_kv_cache* cache, const int32_t* kv_len, const int32_t* n_nodes,
                                 const int32_t* parent, const void* q, int64_t q_stride, sv_dtype dtype,
                                 int32_t n_heads, int32_t B, int32_t Nmax, float scale, void* out,
                                 uint32_t* errors, void* workspace, size_t workspace_bytes, uint32_t expire_waits,
                                 cudaStream_t stream)
{
    sv::AttnArgs a{};
    sv_status st = sv::check_cache(cache, B > 0, &a.c);
    if (st != SV_OK)
        return st;
    if (B < 0 || Nmax < 1 || Nmax > sv::kNodeMax || n_heads < 1 || n_heads % cache->n_kv_heads || expire_waits >> sv::kAttnWaits ||
        (dtype != SV_DTYPE_F32 && dtype != SV_DTYPE_BF16) || !(scale > -3e38f && scale < 3e38f))
        return SV_ERR_INVALID_ARG;
    if (dtype != SV_DTYPE_BF16)
        return SV_ERR_UNSUPPORTED;
    if (B == 0)
        return SV_OK;
    if (!kv_len || !q || !out || !sv::aligned16(q) || !sv::aligned16(out) || q_stride % 8 ||
        ((long long)B * Nmax > 1 && q_stride < (long long)n_heads * cache->head_dim) ||
        (((uintptr_t)kv_len | (uintptr_t)n_nodes | (uintptr_t)parent | (uintptr_t)errors) & 3))
        return SV_ERR_INVALID_ARG;
    if ((long long)B * Nmax * n_heads > 0x3fffffffLL)
        return SV_ERR_UNSUPPORTED;
    if (!workspace || ((uintptr_t)workspace & 255) ||
        workspace_bytes < sv_attention_workspace_size(Nmax, n_heads, cache->n_kv_heads, cache->head_dim))
        return SV_ERR_NO_MEMORY;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_stride = q_stride;
    a.kv_len = kv_len;
    a.n_nodes = n_nodes;
    a.parent = parent;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.err = errors;
    a.has_n = n_nodes != nullptr;
    a.has_parent = parent != nullptr;
    a.has_err = errors != nullptr;
    a.Hq = n_heads;
    a.B = B;
    a.Nmax = Nmax;
    a.scale_log2 = scale * 1.44269504088896341f;
    a.hold = expire_waits;
    a.limit = expire_waits ? 1u << 14 : sv::kWaitSpins;
    a.G = n_heads / cache->n_kv_heads;
    const bool e4m3 = cache->format == SV_KV_E4M3;
    const sv::RowGroups rg = sv::attention_rows(Nmax, a.G, sv::attn_rows_max(e4m3, cache->head_dim));
    a.nodes = rg.nodes;
    a.heads = rg.heads;
    a.head_blocks = rg.head_blocks;
    a.groups = rg.groups;
    a.rows = rg.rows;
    a.nd = cache->head_dim > 128 ? 2 : 1;
    a.box_rows = std::min(cache->page_size, e4m3 ? sv::kTile : sv::kQuarter);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    a.part_o = reinterpret_cast<float*>(ws);
    ws += (size_t)2 * sv::kAttnMaxCtas * a.rows * cache->head_dim * 4;
    a.part_ml = reinterpret_cast<float*>(ws);
    ws += (size_t)2 * sv::kAttnMaxCtas * a.rows * 2 * 4;
    a.meta = reinterpret_cast<int*>(ws);
    int dev = 0, nsm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return SV_ERR_CUDA;
    CUtensorMap m[3];
    if (!sv::cache_map(&m[0], a.c.k, a, e4m3) || !sv::cache_map(&m[1], a.c.v, a, e4m3) ||
        (e4m3 ? (m[2] = m[0], false) : !sv::query_map(&m[2], a)))
        return SV_ERR_CUDA;
    return sv::launched(e4m3 ? sv::launch_attention_rows<true>(a, m, dev, nsm, stream)
                             : sv::launch_attention_rows<false>(a, m, dev, nsm, stream));
}

sv_status spec_kv_commit(const sv_kv_cache* cache, const int32_t* kv_len, const int32_t* out_path,
                         const int32_t* out_len, int32_t B, int32_t Nmax, int32_t* kv_len_out,
                         uint32_t* errors, cudaStream_t stream)
{
    sv::CommitArgs a{};
    sv_status st = sv::check_cache(cache, B > 0, &a.c);
    if (st != SV_OK)
        return st;
    if (B < 0 || Nmax < 1 || Nmax > sv::kNodeMax)
        return SV_ERR_INVALID_ARG;
    if (B == 0)
        return SV_OK;
    if (!kv_len || !out_path || !out_len || !kv_len_out ||
        (((uintptr_t)kv_len | (uintptr_t)out_path | (uintptr_t)out_len | (uintptr_t)kv_len_out | (uintptr_t)errors) & 3))
        return SV_ERR_INVALID_ARG;
    if (cache->layers > 65535)
        return SV_ERR_UNSUPPORTED;
    a.kv_len = kv_len;
    a.path = out_path;
    a.len = out_len;
    a.kv_len_out = kv_len_out;
    a.err = errors;
    a.layer_rows = (long long)cache->num_pages * cache->n_kv_heads * cache->page_size;
    a.elem = cache->format == SV_KV_E4M3 ? 1 : 2;
    a.Nmax = Nmax;
    a.has_err = errors != nullptr;
    a.in_place = kv_len_out == kv_len;
    sv::sv_commit_kernel<<<dim3((unsigned)B, (unsigned)cache->layers), 128, 0, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess)
        return SV_ERR_CUDA;
    if (a.in_place)
        sv::sv_commit_len_kernel<<<(unsigned)((B + 7) / 8), 256, 0, stream>>>(a, B);
    return sv::launched(cudaGetLastError());
}

sv_status spec_kv_read(const sv_kv_cache* cache, const int32_t* start, const int32_t* row_start, int32_t B,
                       int32_t rows, sv_dtype dtype, void* k_out, void* v_out, uint32_t* errors,
                       cudaStream_t stream)
{
    sv::ReadArgs a{};
    sv_status st = sv::check_cache(cache, rows > 0, &a.c);
    if (st != SV_OK)
        return st;
    if (B < 0 || rows < 0 || (dtype != SV_DTYPE_F32 && dtype != SV_DTYPE_BF16))
        return SV_ERR_INVALID_ARG;
    if (rows == 0)
        return SV_OK;
    if (B < 1 || !start || !row_start || !k_out || !v_out || !sv::aligned16(k_out) || !sv::aligned16(v_out) ||
        (((uintptr_t)start | (uintptr_t)row_start | (uintptr_t)errors) & 3))
        return SV_ERR_INVALID_ARG;
    if (cache->n_kv_heads > (1 << 16) || (long long)rows * cache->n_kv_heads > 0x3fffffffLL)
        return SV_ERR_UNSUPPORTED;
    a.start = start;
    a.row_start = row_start;
    a.k_out = k_out;
    a.v_out = v_out;
    a.err = errors;
    a.B = B;
    a.rows = rows;
    a.has_err = errors != nullptr;
    const bool e4m3 = cache->format == SV_KV_E4M3;
    if (dtype == SV_DTYPE_BF16)
        return sv::launched(e4m3 ? sv::launch_read<__nv_bfloat16, true>(a, stream)
                                 : sv::launch_read<__nv_bfloat16, false>(a, stream));
    return sv::launched(e4m3 ? sv::launch_read<float, true>(a, stream) : sv::launch_read<float, false>(a, stream));
}

}  // extern "C"
