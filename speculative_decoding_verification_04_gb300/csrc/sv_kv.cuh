// sv_kv.cuh -- the paged key/value cache: writing new tokens into it (norms,
// rotation and quantisation in the same pass), moving a verified path, and
// reading ranges back.
//
// All three move each byte once and compute little, so what bounds them is
// memory bandwidth for many tokens and the chain of dependent loads (length,
// page, row) for few.  A lane holds 16 elements of a head's row in two chunks
// of 8, so that both elements of every rotated pair are its own and a row's
// sums take log2(head_dim / 16) shuffles.
#pragma once

#include <cuda_fp8.h>

#include "sv_common.cuh"

namespace sv {

constexpr int kNodeMax = 32;   // one lane, or one bit, per node

struct KvCache {
    unsigned char* k;
    unsigned char* v;
    float* k_scale;
    float* v_scale;
    const int32_t* table;   // [B][max_pages]
    int max_pages;
    int layers, num_pages, Hkv, D;
    int page_shift;         // page_size = 1 << page_shift
};

// Row index (one row: one position of one head) of head 0 at (page, slot);
// head h is h << page_shift rows further.
__device__ __forceinline__ long long kv_row(const KvCache& c, int page, int pos)
{
    return (((long long)page * c.Hkv) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// The page holding position pos of sequence b, or -1 where the table's entry
// is none; pos has been checked against the table's width.
__device__ __forceinline__ int kv_page(const KvCache& c, int b, int pos)
{
    const int p = __ldg(c.table + (long long)b * c.max_pages + (pos >> c.page_shift));
    return (unsigned)p < (unsigned)c.num_pages ? p : -1;
}

__device__ __forceinline__ bool kv_span_ok(const KvCache& c, int base, int n)
{
    return base >= 0 && n >= 0 && (long long)base + n <= ((long long)c.max_pages << c.page_shift);
}

// The warp's view of a tree of n <= 32 nodes: lane l gets node l's parent (the
// root's is -1); false where a parent is not an earlier node.  par == nullptr
// (has == false) is the chain.
__device__ __forceinline__ bool tree_parents(const int32_t* par, bool has, int n, int lane, int& p)
{
    p = lane - 1;
    if (has && lane > 0 && lane < n)
        p = __ldg(par + lane);
    const bool bad = lane > 0 && lane < n && (p < 0 || p >= lane);
    return !__any_sync(kFull, bad);
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
struct AppendArgs {
    KvCache c;
    const void* q;
    const void* k;
    const void* v;
    long long q_stride, k_stride, v_stride;   // elements between tokens
    const void* q_norm;
    const void* k_norm;
    const float* cos_sin;
    const int32_t* parent;
    const int32_t* n_new;
    const int32_t* row_start;
    const int32_t* kv_len;
    void* q_out;
    uint32_t* err;
    int has_q, has_qn, has_kn, has_rot, has_parent, has_n, packed, has_err;
    int Hq, B, S, rows, max_positions, rot, interleaved;
    float eps;
};

// Where token t goes, the same in every lane of the warp.
struct TokenPlace {
    int page;    // -1: not stored
    int pos;     // slot position in the cache
    int angle;   // row of the rotation table
    int state;   // 0 stored, 1 no token (its query is zeros), 2 unusable (NaN)
};

__device__ __forceinline__ TokenPlace token_place(const AppendArgs& a, int t, int lane)
{
    TokenPlace r{-1, 0, 0, 0};
    int b, i, n;
    if (a.packed) {
        // the sequence whose rows hold t: 32 splits of the range a step
        int lo = 0, hi = a.B;   // row_start[lo] <= t < row_start[hi]
        const int first = __ldg(a.row_start), end = __ldg(a.row_start + a.B);
        if (t < first || t >= end) {
            r.state = 1;
            return r;
        }
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) >> 5;
            const int at = min(lo + (lane + 1) * step, hi);
            const unsigned m = __ballot_sync(kFull, at < hi && __ldg(a.row_start + at) <= t);
            const int c = __popc(m);   // ascending row starts: the first c splits are at or below t
            const int nlo = lo + c * step;
            hi = min(nlo + step, hi);
            lo = min(nlo, hi - 1);
        }
        b = lo;
        const int r0 = __ldg(a.row_start + b), r1 = __ldg(a.row_start + b + 1);
        i = t - r0;
        n = r1 - r0;
        if (t < r0 || t >= r1 || r0 < max(first, 0) || r1 > end) {   // row_start does not ascend
            r.state = 2;
            return r;
        }
    } else {
        b = t / a.S;
        i = t - b * a.S;
        n = a.has_n ? __ldg(a.n_new + b) : a.S;
        if (n < 0 || n > a.S) {
            r.state = 2;
            return r;
        }
    }
    const int base = __ldg(a.kv_len + b);
    int depth = i;
    if (a.has_parent) {
        // (the whole row, so that it does not wait for the count)
        const int p = lane > 0 && lane < a.S ? __ldg(a.parent + (long long)b * a.S + lane) : lane - 1;
        const bool ok = !__any_sync(kFull, lane > 0 && lane < n && (p < 0 || p >= lane));
        depth = 0;
        for (int at = i; ok && i < n && at > 0 && depth < kNodeMax; ++depth)
            at = __shfl_sync(kFull, p, at);
        if (!ok)
            n = -1;   // malformed: as a bad length
    }
    if (n < 0 || !kv_span_ok(a.c, base, n)) {
        r.state = 2;
        return r;
    }
    if (i >= n) {
        r.state = 1;
        return r;
    }
    r.pos = base + i;
    r.angle = base + depth;
    r.page = kv_page(a.c, b, r.pos);
    if (r.page < 0 || (a.has_rot && r.angle >= a.max_positions))
        r.state = 2;
    return r;
}

// Whether, among this thread's starts, one is negative or above the next: the
// threads of a launch (of `threads` a block, this one the `tid`th) share out all
// starts, those that no row leads to among them.  Blocks past the starts' number
// do nothing (without that, 16411 prompt tokens take 84 us instead of 82).
__device__ __forceinline__ bool starts_unusable(const int32_t* row_start, int B, int threads, int tid)
{
    bool bad = false;
    long long b = (long long)blockIdx.x * threads;
    if (b < B)
#pragma unroll 1
        for (b += tid; b < B; b += (long long)gridDim.x * threads) {
            const int s = __ldg(row_start + b);
            bad |= s < 0 || s > __ldg(row_start + b + 1);
        }
    return bad;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <typename T> struct Row16;   // 16 elements in two chunks of 8

template <> struct Row16<__nv_bfloat16> {
    uint4 w[2];
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int c0, int c1)
    {
        w[0] = __ldg(reinterpret_cast<const uint4*>(p + 8 * c0));
        w[1] = __ldg(reinterpret_cast<const uint4*>(p + 8 * c1));
    }
    __device__ __forceinline__ void get(float (&x)[16]) const
    {
        float y[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            Elem<__nv_bfloat16>::unpack(w[h], y);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[8 * h + j] = y[j];
        }
    }
};

template <> struct Row16<float> {
    float4 w[4];
    __device__ __forceinline__ void load(const float* p, int c0, int c1)
    {
        w[0] = __ldg(reinterpret_cast<const float4*>(p + 8 * c0));
        w[1] = __ldg(reinterpret_cast<const float4*>(p + 8 * c0 + 4));
        w[2] = __ldg(reinterpret_cast<const float4*>(p + 8 * c1));
        w[3] = __ldg(reinterpret_cast<const float4*>(p + 8 * c1 + 4));
    }
    __device__ __forceinline__ void get(float (&x)[16]) const
    {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            x[4 * h] = w[h].x;
            x[4 * h + 1] = w[h].y;
            x[4 * h + 2] = w[h].z;
            x[4 * h + 3] = w[h].w;
        }
    }
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint4 bf16_chunk(const float* x)
{
    return make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
}

__device__ __forceinline__ void store_chunk(__nv_bfloat16* p, const float* x)
{
    *reinterpret_cast<uint4*>(p) = bf16_chunk(x);
}

__device__ __forceinline__ void store_chunk(float* p, const float* x)
{
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ uint32_t e4m3_quad(const float* x)
{
    uint32_t y;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(y) : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]));
    return y;
}

//   y = x rsqrt(mean(x^2) + eps) w;  (a, c) -> (a cos - c sin, c cos + a sin);
//   e4m3: scale = max(amax |y| / 448, 2^-100), stored y / scale.
// One pass: each element is read and written once.  On a GB300, 16411 prompt
// tokens of 32 + 8 + 8 heads of 128 (bf16) take 82 us a call, 0.75 of the
// copy rate (61.7 us); issue slots are 62 % busy, DRAM 57 %.  256 trees of 15
// nodes written to e4m3 take 22.6 us on the GPU (13.3): the lookups' three
// dependent loads, and 960 blocks on 456 places, two waves and a tenth.  8
// single tokens take 3 us on the GPU.
//
// LPR lanes hold a head's row: 16 elements each, the lanes from D / 16 on none
// (D = 80, 96, 112 of LPR 8; 144 ... 240 of LPR 16).  A warp holds 32 / LPR
// rows at a time; the next are on their way to registers while it works and
// the two passes after them to L2, and the first are asked for before the
// token's place is looked up (three loads that depend on one another).  With
// rows loaded when they are needed the 16411 tokens took 104 us.  At three
// blocks an SM (80 registers) bf16 rows spill 20 to 24 bytes, fp32 rows 64 to 72.
template <typename T, int LPR, bool E4M3>
__global__ void __launch_bounds__(256, 3) sv_append_kernel(const __grid_constant__ AppendArgs a)
{
    // a block is tpb tokens of wpt warps each
    const int lane = threadIdx.x, sub = threadIdx.y, wpt = blockDim.y;
    const int t = blockIdx.x * blockDim.z + threadIdx.z;
    if (a.packed && starts_unusable(a.row_start, a.B, 32 * wpt * blockDim.z, (threadIdx.z * wpt + sub) * 32 + lane) && a.has_err)
        atomicOr(a.err, kErrCache);
    if (t >= a.rows)
        return;
    constexpr int RPW = 32 / LPR;
    const int c = lane % LPR, D = a.c.D;
    const int Hk = a.c.Hkv, Hq = a.has_q ? a.Hq : 0, H = Hq + 2 * Hk;
    const bool live = c < D / 16;
    // the lane's two chunks of 8: a rotated pair's two elements are both its own
    const bool turn = a.has_rot && c < a.rot / 16;
    const int c0 = turn && !a.interleaved ? c : 2 * c;
    const int c1 = turn && !a.interleaved ? c + a.rot / 16 : 2 * c + 1;

    // the rows that the lane's part of pass r0 lies in: queries, keys, values
    const T* const q = static_cast<const T*>(a.q) + t * a.q_stride;
    const T* const k = static_cast<const T*>(a.k) + t * a.k_stride;
    const T* const v = static_cast<const T*>(a.v) + t * a.v_stride;
    auto at = [&](int r) -> const T* {
        return r >= H || !live ? nullptr : r < Hq ? q + r * D : r < Hq + Hk ? k + (r - Hq) * D : v + (r - Hq - Hk) * D;
    };
    auto load = [&](int r, Row16<T>& w) {
        if (const T* const x = at(r))
            w.load(x, c0, c1);
    };
    Row16<T> now{};
    int r = sub * RPW + lane / LPR;
    load(r, now);
    // the three passes after it, into L2 (registers to hold them would cost a third of the warps): the first lane
    // of each 128 bytes asks
#pragma unroll
    for (int j = 1; j < 4; ++j) {
        const T* const x = at(r + j * wpt * RPW);
        if (x && c % (128 / (16 * (int)sizeof(T))) == 0)
            prefetch_l2(x + 16 * c);
    }
    const TokenPlace pl = token_place(a, t, lane);
    if (pl.state == 2 && a.has_err && sub == 0 && lane == 0)
        atomicOr(a.err, kErrCache);
    const bool placed = pl.state == 0;

    // cosines and sines of the lane's eight pairs, two by two
    uint64_t cs[4], sn[4];
    if (turn && placed) {
        const float* x = a.cos_sin + (long long)pl.angle * a.rot + 8 * c;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 u = __ldg(reinterpret_cast<const float4*>(x) + j);
            const float4 w = __ldg(reinterpret_cast<const float4*>(x + a.rot / 2) + j);
            cs[2 * j] = f2_pack(u.x, u.y), cs[2 * j + 1] = f2_pack(u.z, u.w);
            sn[2 * j] = f2_pack(w.x, w.y), sn[2 * j + 1] = f2_pack(w.z, w.w);
        }
    }
    for (int r0 = sub * RPW; r0 < H; r0 += wpt * RPW, r += wpt * RPW) {   // uniform in the warp: the shuffles need every lane
        const int kind = r < Hq ? 0 : r < Hq + Hk ? 1 : 2;
        const bool act = r < H && live, here = act && placed;
        float x[16];
        now.get(x);
        load(r + wpt * RPW, now);
        if (!here) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                x[j] = 0.0f;
        }
        uint64_t y[8];   // two by two
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = f2_pack(x[2 * j], x[2 * j + 1]);
        if (a.has_qn | a.has_kn) {
            uint64_t s2 = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s2 = f2_fma(y[j], y[j], s2);
            float ss, other;
            f2_unpack(s2, ss, other);
            ss += other;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1)
                ss += __shfl_xor_sync(kFull, ss, o);
            if (here && (kind == 0 ? a.has_qn : kind == 1 ? a.has_kn : false)) {
                Row16<T> n;
                n.load(static_cast<const T*>(kind == 0 ? a.q_norm : a.k_norm), c0, c1);
                float g[16];
                n.get(g);
                const float inv = rsqrtf(ss / (float)D + a.eps);
                const uint64_t i2 = f2_pack(inv, inv);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = f2_mul(f2_mul(y[j], i2), f2_pack(g[2 * j], g[2 * j + 1]));
            }
        }
        if (turn && kind < 2 && placed) {
            if (a.interleaved) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float c2[2], s2[2], u, w;
                    f2_unpack(cs[j / 2], c2[0], c2[1]);
                    f2_unpack(sn[j / 2], s2[0], s2[1]);
                    f2_unpack(y[j], u, w);
                    y[j] = f2_pack(u * c2[j & 1] - w * s2[j & 1], w * c2[j & 1] + u * s2[j & 1]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint64_t u = y[j], z = y[4 + j];
                    y[j] = f2_sub(f2_mul(u, cs[j]), f2_mul(z, sn[j]));
                    y[4 + j] = f2_fma(u, sn[j], f2_mul(z, cs[j]));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f2_unpack(y[j], x[2 * j], x[2 * j + 1]);
        if (kind == 0 && act) {
            if (pl.state == 2) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    x[j] = NAN;
            }
            T* dst = static_cast<T*>(a.q_out) + ((long long)t * a.Hq + r) * D;
            store_chunk(dst + 8 * c0, x);
            store_chunk(dst + 8 * c1, x + 8);
        }
        const int h = kind == 1 ? r - Hq : r - Hq - Hk;
        const long long row = kv_row(a.c, pl.page, pl.pos) + ((long long)h << a.c.page_shift);
        if (E4M3 && __any_sync(kFull, kind > 0 && act)) {
            // one scale a row: its largest magnitude becomes 448; the floor keeps it finite for rows of (nearly) zeros
            uint32_t m = 0;   // (magnitudes order as integers, NaN above infinity)
#pragma unroll
            for (int j = 0; j < 16; ++j)
                m = max(m, __float_as_uint(x[j]) & 0x7fffffffu);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1)
                m = max(m, __shfl_xor_sync(kFull, m, o));
            if (kind > 0 && here) {
                float step = __uint_as_float(m) / 448.0f;
                step = step < 0x1p-100f ? 0x1p-100f : step;
                // x / step, rounded as a division is (the quotient by the reciprocal and its remainder's correction,
                // Markstein 1990), so that the stored value depends on the row alone
                const float inv = __frcp_rn(step);
                const uint64_t i2 = f2_pack(inv, inv), n2 = f2_pack(-step, -step);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint64_t z = f2_pack(x[2 * j], x[2 * j + 1]), u = f2_mul(z, i2);
                    f2_unpack(f2_fma(f2_fma(u, n2, z), i2, u), x[2 * j], x[2 * j + 1]);
                }
                unsigned char* dst = (kind == 1 ? a.c.k : a.c.v) + row * D;
                *reinterpret_cast<uint2*>(dst + 8 * c0) = make_uint2(e4m3_quad(x), e4m3_quad(x + 4));
                *reinterpret_cast<uint2*>(dst + 8 * c1) = make_uint2(e4m3_quad(x + 8), e4m3_quad(x + 12));
                if (c == 0)
                    (kind == 1 ? a.c.k_scale : a.c.v_scale)[row] = step;
            }
        }
        if (!E4M3 && kind > 0 && here) {
            __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(kind == 1 ? a.c.k : a.c.v) + row * D;
            store_chunk(dst + 8 * c0, x);
            store_chunk(dst + 8 * c1, x + 8);
        }
    }
}

// ---------------------------------------------------------------------------
// read: x scale, rounded once.  Bound by HBM where there is much to read:
// 100003 rows of 8 heads of 128 from e4m3 to bf16 take 118 us on a GB300, 0.79
// of the copy rate (93 us).
// ---------------------------------------------------------------------------
struct ReadArgs {
    KvCache c;
    const int32_t* start;
    const int32_t* row_start;
    void* k_out;
    void* v_out;
    uint32_t* err;
    int B, rows, has_err;
    int wpt;   // warps a row's heads are spread over
};

template <typename T, bool E4M3>
__global__ void __launch_bounds__(256) sv_read_kernel(const __grid_constant__ ReadArgs a)
{
    const int lane = threadIdx.x & 31;
    const int gw = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int t = gw / a.wpt;
    if (starts_unusable(a.row_start, a.B, 256, threadIdx.x) && a.has_err)
        atomicOr(a.err, kErrCache);
    if (t >= a.rows)
        return;
    const int sub = gw - t * a.wpt;
    // the append's place of a packed token, with `start` in place of the length
    AppendArgs p;
    p.c = a.c;
    p.packed = 1;
    p.row_start = a.row_start;
    p.kv_len = a.start;
    p.B = a.B;
    p.has_parent = p.has_rot = 0;
    const TokenPlace pl = token_place(p, t, lane);
    if (pl.state == 2 && a.has_err && sub == 0 && lane == 0)
        atomicOr(a.err, kErrCache);
    const int D = a.c.D, per = D / 16, units = 2 * a.c.Hkv * per;   // 16 elements a unit
    const long long row0 = pl.state == 0 ? kv_row(a.c, pl.page, pl.pos) : 0;
    for (int u = sub * 32 + lane; u < units; u += a.wpt * 32) {
        const int hh = u / per, e = (u - hh * per) * 16;
        const bool isv = hh >= a.c.Hkv;
        const int h = isv ? hh - a.c.Hkv : hh;
        const long long row = row0 + ((long long)h << a.c.page_shift);
        float x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            x[j] = pl.state == 2 ? NAN : 0.0f;
        if (pl.state == 0) {
            const unsigned char* base = isv ? a.c.v : a.c.k;
            if (E4M3) {
                const uint4 w = *reinterpret_cast<const uint4*>(base + row * D + e);
                const float s = (isv ? a.c.v_scale : a.c.k_scale)[row];
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(ww[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
                    const float2 f = __half22float2(__half2(hr));
                    x[2 * j] = f.x * s;
                    x[2 * j + 1] = f.y * s;
                }
            } else {
                Row16<__nv_bfloat16> w;
                w.load(reinterpret_cast<const __nv_bfloat16*>(base) + row * D + e, 0, 1);
                w.get(x);
            }
        }
        T* dst = static_cast<T*>(isv ? a.v_out : a.k_out) + ((long long)t * a.c.Hkv + h) * D + e;
        store_chunk(dst, x);
        store_chunk(dst + 8, x + 8);
    }
}

// ---------------------------------------------------------------------------
// commit
// ---------------------------------------------------------------------------
struct CommitArgs {
    KvCache c;
    const int32_t* kv_len;
    const int32_t* path;
    const int32_t* len;
    int32_t* kv_len_out;
    uint32_t* err;
    long long layer_rows;   // rows of one layer
    int elem;               // bytes of an element
    int Nmax, has_err, in_place;
};

// The new length of sequence b, the same in every lane; lane i < its kept
// count gets the rows of move i.  -1: unusable.
__device__ __forceinline__ int commit_moves(const CommitArgs& a, int b, int lane, int& kept, long long& src,
                                            long long& dst)
{
    kept = __ldg(a.len + b);
    const int base = a.kv_len[b];   // the last launch of an in-place call writes it
    src = dst = 0;
    if (kept == -1) {
        kept = 0;
        return base;
    }
    bool bad = kept < 0 || kept >= a.Nmax || !kv_span_ok(a.c, base, 1 + max(kept, 0));
    if (!bad) {
        const int node = lane < kept ? __ldg(a.path + (long long)b * a.Nmax + lane) : 0;
        const int before = __shfl_up_sync(kFull, node, 1);
        bool wrong = false;
        if (lane < kept) {
            wrong = node >= a.Nmax || node <= (lane ? before : 0) || !kv_span_ok(a.c, base, node + 1);
            if (!wrong) {
                const int ps = kv_page(a.c, b, base + node), pd = kv_page(a.c, b, base + 1 + lane);
                wrong = ps < 0 || pd < 0;
                src = kv_row(a.c, ps, base + node);
                dst = kv_row(a.c, pd, base + 1 + lane);
            }
        }
        bad = __any_sync(kFull, wrong);
    }
    if (bad) {
        kept = 0;
        return -1;
    }
    return base + 1 + kept;
}

// Latency bounds it: length, path, pages, then rows, each waiting for the one
// before.  32 layers of 256 trees take 10.5 us on a GB300 (the bytes 10.4), two
// layers of four 3.3 us.
// One block per (sequence, layer).  A thread takes one 16-byte column of a
// head's rows through all moves in order: path[i] > i strictly ascends, so a
// move writes only rows that no later move reads.
__global__ void __launch_bounds__(128) sv_commit_kernel(const __grid_constant__ CommitArgs a)
{
    __shared__ long long s_src[kNodeMax], s_dst[kNodeMax];
    __shared__ int s_kept;
    const int b = blockIdx.x, layer = blockIdx.y;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int kept;
        long long src, dst;
        const int now = commit_moves(a, b, lane, kept, src, dst);
        s_src[lane] = src;
        s_dst[lane] = dst;
        if (lane == 0) {
            s_kept = kept;
            if (layer == 0) {
                if (now < 0 && a.has_err)
                    atomicOr(a.err, kErrCache);
                if (!a.in_place)
                    a.kv_len_out[b] = now < 0 ? a.kv_len[b] : now;
            }
        }
    }
    __syncthreads();
    const int kept = s_kept;
    if (kept == 0)
        return;
    const bool e4m3 = a.elem == 1;
    const long long lrow = layer * a.layer_rows;
    const int cols = a.c.D * a.elem / 16, per = 2 * a.c.Hkv * cols, total = per + (e4m3 ? 2 * a.c.Hkv : 0);
    const long long pitch = (long long)a.c.D * a.elem;
    for (int u = threadIdx.x; u < total; u += blockDim.x) {
        if (u < per) {
            const int hh = u / cols, col = u - hh * cols;
            const bool isv = hh >= a.c.Hkv;
            const int h = isv ? hh - a.c.Hkv : hh;
            unsigned char* base = (isv ? a.c.v : a.c.k) + (lrow + ((long long)h << a.c.page_shift)) * pitch + 16 * col;
            for (int i = 0; i < kept; ++i)
                if (s_src[i] != s_dst[i])
                    *reinterpret_cast<uint4*>(base + s_dst[i] * pitch) =
                        *reinterpret_cast<const uint4*>(base + s_src[i] * pitch);
        } else {
            const int hh = u - per;
            const bool isv = hh >= a.c.Hkv;
            float* base = (isv ? a.c.v_scale : a.c.k_scale) + lrow +
                          ((long long)(isv ? hh - a.c.Hkv : hh) << a.c.page_shift);
            for (int i = 0; i < kept; ++i)
                base[s_dst[i]] = base[s_src[i]];
        }
    }
}

// The lengths of an in-place call, after every block above has read them.
__global__ void __launch_bounds__(256) sv_commit_len_kernel(const __grid_constant__ CommitArgs a, int B)
{
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (b >= B)
        return;
    int kept;
    long long src, dst;
    const int now = commit_moves(a, b, lane, kept, src, dst);
    if (lane == 0 && now >= 0)
        a.kv_len_out[b] = now;
}

}  // namespace sv
