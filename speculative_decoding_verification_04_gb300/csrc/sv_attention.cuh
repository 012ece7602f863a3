// sv_attention.cuh -- attention of tree nodes over the paged cache.
//
//   out[n] = sum_j softmax_j(scale q_n . k_j) v_j
// over the context's positions and node n's ancestors (itself included).
//
// One block per (sequence, node, query head): its warps take every fourth
// position with a running maximum and sum each, joined at the end.
#pragma once

#include "sv_kv.cuh"

namespace sv {

constexpr int kAttnMaxCtas = 160;

struct AttnArgs {
    KvCache c;
    const __nv_bfloat16* q;
    long long q_stride;      // elements between tokens
    const int32_t* kv_len;
    const int32_t* n_nodes;
    const int32_t* parent;
    __nv_bfloat16* out;
    uint32_t* err;
    int has_n, has_parent, has_err;
    int Hq, B, Nmax;
    float scale_log2;        // scale * log2(e)
};

template <bool E4M3>
__global__ void __launch_bounds__(128) sv_attention_kernel(const __grid_constant__ AttnArgs a)
{
    constexpr int kW = 4, kE = 8;   // warps; elements a lane holds (32 apart)
    __shared__ float s_m[kW], s_l[kW], s_o[kW][256];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, D = a.c.D;
    const int h = blockIdx.x % a.Hq, n = (blockIdx.x / a.Hq) % a.Nmax, b = blockIdx.x / a.Hq / a.Nmax;
    const int nn = a.has_n ? __ldg(a.n_nodes + b) : a.Nmax, base = __ldg(a.kv_len + b);
    __nv_bfloat16* out = a.out + (((long long)b * a.Nmax + n) * a.Hq + h) * D;
    int par;
    bool ok = nn >= 0 && nn <= a.Nmax && kv_span_ok(a.c, base, nn);
    ok = tree_parents(a.parent + (long long)b * a.Nmax, a.has_parent, ok ? nn : 0, lane, par) && ok;
    unsigned anc = 0;
    for (int at = n, d = 0; ok && n < nn && at >= 0 && d <= kNodeMax; ++d) {
        anc |= 1u << at;
        at = __shfl_sync(kFull, par, at);
    }
    float m = -1e30f, l = 0.0f, q[kE], o[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        const int d = lane + 32 * e;
        o[e] = 0.0f;
        q[e] = d < D ? Elem<__nv_bfloat16>::load(a.q + ((long long)b * a.Nmax + n) * a.q_stride + (long long)h * D + d) : 0.0f;
    }
    const int hk = h / (a.Hq / a.c.Hkv), end = ok && n < nn ? base + nn : 0;
    for (int j = w; j < end; j += kW) {
        if (j >= base && !((anc >> (j - base)) & 1u))
            continue;
        const int page = kv_page(a.c, b, j);
        if (page < 0) {
            ok = false;
            break;
        }
        const long long row = kv_row(a.c, page, j) + ((long long)hk << a.c.page_shift);
        float s = 0.0f, v[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const int d = lane + 32 * e;
            v[e] = 0.0f;
            if (d < D) {
                float k;
                if (E4M3) {
                    k = (float)*reinterpret_cast<const __nv_fp8_e4m3*>(a.c.k + row * D + d) * a.c.k_scale[row];
                    v[e] = (float)*reinterpret_cast<const __nv_fp8_e4m3*>(a.c.v + row * D + d) * a.c.v_scale[row];
                } else {
                    k = Elem<__nv_bfloat16>::load(reinterpret_cast<const __nv_bfloat16*>(a.c.k) + row * D + d);
                    v[e] = Elem<__nv_bfloat16>::load(reinterpret_cast<const __nv_bfloat16*>(a.c.v) + row * D + d);
                }
                s = fmaf(q[e], k, s);
            }
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1)
            s += __shfl_xor_sync(kFull, s, x);
        s *= a.scale_log2;
        const float top = max_nan(m, s), f = ex2_approx(m - top), p = ex2_approx(s - top);
        m = top;
        l = l * f + p;
#pragma unroll
        for (int e = 0; e < kE; ++e)
            o[e] = o[e] * f + p * v[e];
    }
    if (lane == 0) {
        s_m[w] = m;
        s_l[w] = l;
    }
#pragma unroll
    for (int e = 0; e < kE; ++e)
        s_o[w][lane + 32 * e] = o[e];
    ok = __syncthreads_and(ok);
    if (!ok && a.has_err && threadIdx.x == 0)
        atomicOr(a.err, kErrCache);
    float top = s_m[0];
    for (int i = 1; i < kW; ++i)
        top = max_nan(top, s_m[i]);
    float f[kW], sum = 0.0f;
    for (int i = 0; i < kW; ++i) {
        f[i] = ex2_approx(s_m[i] - top);
        sum += f[i] * s_l[i];
    }
    for (int d = threadIdx.x; d < D; d += blockDim.x) {
        float x = 0.0f;
        for (int i = 0; i < kW; ++i)
            x += f[i] * s_o[i][d];
        x = !ok ? NAN : n < nn ? x / sum : 0.0f;
        out[d] = __float2bfloat16_rn(x);
    }
}

}  // namespace sv
