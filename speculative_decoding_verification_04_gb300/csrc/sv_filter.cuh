// sv_filter.cuh -- min-p, top-k and top-p over rows of logits: the kept set, a
// draw from it, and the row with the rest at -inf.
//
// Order a row's tokens by logit, the largest first, equal ones by index.  Each
// filter keeps a prefix of that order, and so does their sequence; a prefix is
// named by its last token (key, index).  A draw is the end of a prefix too: of
// the shortest one whose mass is above u Z.  So everything is one question:
// where does a prefix reach a given count or mass?
#pragma once

#include "sv_weights.cuh"

namespace sv {

struct FilterArgs {
    const void* logits;      // [B * S][V]
    void* out;               // the same, filter only
    const float* uniforms;   // draw only
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const int32_t* n_rows;
    int32_t* out_tokens;
    float* out_prob;
    int32_t* out_kept;
    int B, S, V;
    int has_k, has_p, has_m, has_n, has_prob, has_kept;
    int same_phase;          // out's rows have the 16-byte phase of logits' rows
};

constexpr int kFilterThreads = 512;

// A row as its 16-byte vectors and the elements before and after them.
template <typename T> struct RowSpan {
    const T* p;
    int V, head, nvec;
    __device__ RowSpan(const T* row, int V_) : p(row), V(V_)
    {
        const int phase = (int)(((uintptr_t)row & 15) / sizeof(T));
        head = min(V, phase ? Elem<T>::E - phase : 0);
        nvec = (V - head) / Elem<T>::E;
    }
    // f(value, index) for every element, spread over the block's threads
    template <typename F> __device__ __forceinline__ void each(F&& f) const
    {
        constexpr int E = Elem<T>::E;
        const uint4* v = reinterpret_cast<const uint4*>(p + head);
        for (int i = threadIdx.x; i < nvec; i += kFilterThreads) {
            float x[E];
            Elem<T>::unpack(__ldg(v + i), x);
#pragma unroll
            for (int k = 0; k < E; ++k)
                f(x[k], head + i * E + k);
        }
        const int rest = V - nvec * E;   // head and tail
        if ((int)threadIdx.x < rest) {
            const int i = (int)threadIdx.x < head ? threadIdx.x : nvec * E + threadIdx.x;
            f(Elem<T>::load(p + i), i);
        }
    }
};

struct FilterShared {
    uint64_t roots[64];
    u128 part[kFilterThreads / 32];
    u128 sum;
};

__device__ __forceinline__ u128 shfl_down128(u128 v, int o)
{
    const unsigned long long lo = __shfl_down_sync(kFull, (unsigned long long)v, o);
    const unsigned long long hi = __shfl_down_sync(kFull, (unsigned long long)(v >> 64), o);
    return ((u128)hi << 64) | lo;
}

__device__ __forceinline__ u128 block_sum(u128 v, FilterShared& s)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += shfl_down128(v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        s.part[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        u128 t = 0;
        for (int w = 0; w < kFilterThreads / 32; ++w)
            t += s.part[w];
        s.sum = t;
    }
    __syncthreads();
    return s.sum;
}

// The last token of a prefix of the order.
struct Prefix {
    uint32_t key;
    int index;
};

// The sum over a prefix of 1 (kCount) or of the weights.
template <bool kCount, typename T>
__device__ u128 prefix_sum(const RowSpan<T>& row, Prefix p, const RowScale& sc, FilterShared& s)
{
    u128 a = 0;
    row.each([&](float x, int i) {
        const uint32_t k = key_of(x);
        if (k > p.key || (k == p.key && i <= p.index))
            a += kCount ? 1 : weight62(x, sc, s.roots);
    });
    return block_sum(a, s);
}

// The shortest prefix within `most` that sums to `goal` (which `most` does).
template <bool kCount, typename T>
__device__ Prefix prefix_reaching(const RowSpan<T>& row, u128 goal, Prefix most, uint32_t top, const RowScale& sc, FilterShared& s)
{
    uint32_t lo = most.key, hi = top;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        if (prefix_sum<kCount>(row, Prefix{mid, INT_MAX}, sc, s) >= goal)
            lo = mid;
        else
            hi = mid - 1;
    }
    const u128 above = lo == 0xffffffffu ? 0 : prefix_sum<kCount>(row, Prefix{lo + 1, INT_MAX}, sc, s);
    int a = 0, b = most.key == lo ? min(most.index, row.V - 1) : row.V - 1;
    const u128 each = kCount ? 1 : weight62(value_of(lo), sc, s.roots);
    while (a < b) {
        const int mid = a + (b - a) / 2;
        int n = 0;
        row.each([&](float x, int i) { n += key_of(x) == lo && i <= mid; });
        if (above + block_sum((u128)n, s) * each >= goal)
            b = mid;
        else
            a = mid + 1;
    }
    return Prefix{lo, a};
}

template <typename T, bool DRAW>
__global__ void __launch_bounds__(kFilterThreads) sv_filter_kernel(FilterArgs a)
{
    __shared__ FilterShared s;
    const long long r = blockIdx.x;
    const int b = (int)(r / a.S), i = (int)(r % a.S), V = a.V;
    if (!DRAW && a.has_n && i >= a.n_rows[b]) {   // no row: its logits and outputs stay
        if (threadIdx.x == 0 && a.has_kept)
            a.out_kept[r] = 0;
        return;
    }
    if (threadIdx.x < 64)
        s.roots[threadIdx.x] = root_power(threadIdx.x);
    const float T_ = a.temperature[b];
    const int k = a.has_k ? a.top_k[b] : 0;
    const float p = a.has_p ? a.top_p[b] : 1.0f, mp = a.has_m ? a.min_p[b] : 0.0f;
    const float u = DRAW && T_ != 0.0f ? a.uniforms[r] : 0.0f;
    const RowSpan<T> row(static_cast<const T*>(a.logits) + r * V, V);
    // the largest key; a NaN's key is above +inf's or below -inf's
    uint32_t top = 0, bottom = 0xffffffffu;
    row.each([&](float x, int) {
        const uint32_t key = key_of(x);
        top = max(top, key);
        bottom = min(bottom, key);
    });
    top = __reduce_max_sync(kFull, top);
    bottom = __reduce_min_sync(kFull, bottom);
    __shared__ uint32_t s_top, s_bottom;
    if (threadIdx.x == 0) {
        s_top = 0;
        s_bottom = 0xffffffffu;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        atomicMax(&s_top, top);
        atomicMin(&s_bottom, bottom);
    }
    __syncthreads();
    top = s_top;
    bottom = s_bottom;
    const bool usable = bottom >= kKeyNegInf && top < kKeyPosInf && top > kKeyNegInf && temperature_usable(T_) && k >= 0 &&
                        p >= 0.0f && p <= 1.0f && mp >= 0.0f && mp <= 1.0f && u >= 0.0f && u < 1.0f;
    Prefix end{kKeyNegInf + 1, INT_MAX};
    u128 mass = 0;
    RowScale sc{};
    if (usable && T_ == 0.0f) {
        end = prefix_reaching<true>(row, 1, Prefix{top, INT_MAX}, top, sc, s);
    } else if (usable) {
        const float m = value_of(top);
        sc = row_scale(m, T_);
        if (mp > 0.0f) {
            const double t = (double)m + (double)T_ * log((double)mp);
            float least = (float)fmax(t, -3.4028234e38);
            if ((double)least < t)
                least = value_of(key_of(least) + 1);
            end.key = max(end.key, key_of(least));
        }
        if (k > 0 && prefix_sum<true>(row, end, sc, s) > (u128)k)
            end = prefix_reaching<true>(row, (u128)k, end, top, sc, s);
        if (p < 1.0f || DRAW)
            mass = prefix_sum<false>(row, end, sc, s);
        if (p < 1.0f) {
            const u128 goal = share_of(p, mass, true);
            end = prefix_reaching<false>(row, goal > 1 ? goal : 1, end, top, sc, s);
            if (DRAW)
                mass = prefix_sum<false>(row, end, sc, s);
        }
    }
    int kept = -1;
    if (usable && a.has_kept)
        kept = (int)prefix_sum<true>(row, end, sc, s);
    if (threadIdx.x == 0 && a.has_kept)
        a.out_kept[r] = kept;
    if (DRAW) {
        int token = -1;
        float prob = __int_as_float(0x7fc00000);
        if (usable && T_ == 0.0f) {
            token = end.index;
            prob = 1.0f;
        } else if (usable) {
            const Prefix at = prefix_reaching<false>(row, share_of(u, mass, false) + 1, end, top, sc, s);
            token = at.index;
            prob = (float)((double)weight62(value_of(at.key), sc, s.roots) / (double)mass);
        }
        if (threadIdx.x == 0) {
            a.out_tokens[r] = token;
            if (a.has_prob)
                a.out_prob[r] = prob;
        }
        return;
    }
    T* out = static_cast<T*>(a.out) + r * V;
    for (int j = threadIdx.x; j < V; j += kFilterThreads) {
        const T x = static_cast<const T*>(a.logits)[r * V + j];
        const uint32_t key = key_of((float)x);
        const bool keep = key > end.key || (key == end.key && j <= end.index);
        out[j] = !usable ? T(__int_as_float(0x7fc00000)) : keep ? x : T(-INFINITY);
    }
}

}  // namespace sv
