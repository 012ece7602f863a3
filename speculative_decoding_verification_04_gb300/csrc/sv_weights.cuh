// sv_weights.cuh -- softmax weights as whole numbers: exp((l - m) / T) in units
// of 2^-62, for sums that do not depend on their order and comparisons of them
// that are exact.
//
// A filter's border is where a cumulative mass C crosses p Z.  With sums of
// relative error e it moves by e Z / w tokens of weight w, so that fp32 sums
// (e near 1e-7) over a row whose tokens weigh 1e-5 of it each would misplace
// one border in a hundred.  Whole numbers add without rounding, in any order.
#pragma once

#include "sv_common.cuh"

namespace sv {

typedef unsigned __int128 u128;

constexpr uint64_t kOne62 = 1ull << 62;

// 2^64 times 2^-(2^i / 64), i = 0 .. 5: one half's repeated square roots
__constant__ const uint64_t kRoots[6] = {0xfd3e0c0cf486c175ull, 0xfa83b2db722a033aull, 0xf5257d152486cc2cull,
                                         0xeac0c6e7dd24392full, 0xd744fccad69d6af4ull, 0xb504f333f9de6484ull};

// 2^(62 - j / 64): the product of the roots that j's bits name
__device__ __forceinline__ uint64_t root_power(int j)
{
    uint64_t t = kOne62;
#pragma unroll
    for (int i = 0; i < 6; ++i)
        if (j >> i & 1)
            t = __umul64hi(t, kRoots[i]);
    return t;
}

// fp32 values in an order of unsigned integers (-0 counts as +0).
__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

constexpr uint32_t kKeyNegInf = 0x007fffffu;
constexpr uint32_t kKeyPosInf = 0xff800000u;

// What the weights of one row are made with: x = (m - l) log2(e) / T in units
// of 2^-48 from products with a constant split in two floats (each product is
// exact with its remainder, so x is good to about 2^-42 at |l| log2(e) / T up
// to 2^6, to 2^-36 at 2^12); rows beyond that take differences in 64 bits.
struct RowScale {
    float ch, cl;       // log2(e) / T
    float m, T;
    float least;        // logits below it weigh nothing (less than 2^-64)
    long long top;      // m log2(e) / T, units of 2^-48
    bool cold;
};

__device__ __forceinline__ long long scaled48(float l, float ch, float cl)
{
    const float t = __fmul_rn(l, ch);
    const float e = __fmaf_rn(l, cl, __fmaf_rn(l, ch, -t));
    // t = n + f, |f| <= 1/2, and f in steps of 2^-24, the rest with e in steps of
    // 2^-48 (|e| < 2^-10): conversions to 32 bits, which are fast
    const float n = rintf(t), f = (t - n) * 16777216.0f, a = rintf(f);
    const float b = fmaf(e, 16777216.0f, f - a) * 16777216.0f;   // (below 2^39: as two)
    const float b1 = rintf(b * 5.9604644775390625e-8f);
    return ((long long)(int)n << 48) + ((long long)((int)a + (int)b1) << 24) + (long long)(int)rintf(fmaf(b1, -16777216.0f, b));
}

__device__ __forceinline__ RowScale row_scale(float m, float T)
{
    RowScale r;
    r.ch = __fdiv_rn(1.44269502162933349609375f, T);   // log2(e) is this and 1.92596e-8
    r.cl = __fdiv_rn(__fmaf_rn(-r.ch, T, 1.44269502162933349609375f) + 1.92596299112661746887e-8f, T);
    r.m = m;
    r.T = T;
    r.cold = !(fabsf(m) * r.ch < 4096.0f) || T > 1e30f;   // (the constant's second part would be subnormal)
    r.least = fmaxf(m - 70.0f * T, -3.4028234e38f);
    r.top = r.cold ? 0 : scaled48(m, r.ch, r.cl);
    return r;
}

// 2^-x in units of 2^-62, x >= 0 in units of 2^-48.  2^-x = 2^-n 2^(-j / 64) e^-y
// with y = ln 2 times the rest, below 1/64; e^-y by its series, the terms from
// the third on (below 2^-22) in fp32.  Good to 2^-45 of itself and half a unit.
__device__ __forceinline__ uint64_t exp2_neg(uint64_t x, const uint64_t* roots)
{
    const int n = (int)min((unsigned long long)(x >> 48), 63ull);
    if (n > 62)
        return 0;
    const int j = (int)(x >> 42) & 63;
    const uint64_t y = __umul64hi((x & ((1ull << 42) - 1)) << 16, 0xb17217f7d1cf79acull);   // 2^64 ln 2
    const float f = (float)(y >> 32) * 2.3283064365386963e-10f;
    const float c = f * f * f * (1.0f / 6 - f * (1.0f / 24 - f * (1.0f / 120)));
    const uint64_t q = y - (__umul64hi(y, y) >> 1) + ((uint64_t)(uint32_t)(c * 1.8014398509481984e16f) << 10);   // 1 - e^-y; c < 2^-22, in 2^-54
    const uint64_t w = roots[j] - __umul64hi(roots[j], q);
    return n ? ((w >> (n - 1)) + 1) >> 1 : w;
}

// The weight of logit l <= m (no NaN).
__device__ __forceinline__ uint64_t weight62(float l, const RowScale& r, const uint64_t* roots)
{
    if (l < r.least || l == -INFINITY)
        return 0;
    long long x;
    if (r.cold) {
        const double d = ((double)r.m - (double)l) * (1.4426950408889634 / (double)r.T);
        x = d < 64.0 ? (long long)(d * 281474976710656.0) : 64ll << 48;
    } else {
        x = r.top - scaled48(l, r.ch, r.cl);
    }
    return exp2_neg((uint64_t)(x > 0 ? x : 0), roots);
}

// ceil(p z) and floor(p z) of an fp32 share p in [0, 1] of a whole number
// z < 2^96, exactly: p is a whole number of 24 bits times a power of two.
__device__ __forceinline__ u128 share_of(float p, u128 z, bool up)
{
    const uint32_t b = __float_as_uint(p);
    const int e = (int)(b >> 23);
    const uint32_t a = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
    const int s = 150 - (e ? e : 1);
    const u128 n = z * a;
    if (s > 126)
        return up && n != 0 ? 1 : 0;
    return up ? (n + (((u128)1 << s) - 1)) >> s : n >> s;
}

// The same of a whole number below 2^64.
__device__ __forceinline__ uint64_t share_of(float p, uint64_t z, bool up)
{
    return (uint64_t)share_of(p, (u128)z, up);
}

// w / z as the nearest fp32 (but for one case in 2^20), z < 2^96: a quotient of
// the leading bits, and a correction by the rest.
__device__ __forceinline__ float quotient(uint64_t w, u128 z)
{
    const uint64_t over = (uint64_t)(z >> 64);
    const int down = over ? 64 - __clzll(over) : 0;
    const uint64_t y = (uint64_t)(z >> down);
    const float wh = __ull2float_rz(w), yh = __ull2float_rz(y);
    const float wl = (float)(w - (uint64_t)wh), yl = (float)(y - (uint64_t)yh);
    const float q = __fdiv_rn(wh, yh);
    return (q + __fdiv_rn(__fmaf_rn(-q, yl, __fmaf_rn(-q, yh, wh) + wl), yh)) * __int_as_float((127 - down) << 23);
}

}  // namespace sv
