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
    int C;                   // CTAs a row is spread over (its cluster)
    int same_phase;          // out's rows have the 16-byte phase of logits' rows
};


constexpr int kFilterThreads = 512;
constexpr int kFilterWarps = kFilterThreads / 32;
constexpr int kGroup = 8;          // vectors of a thread whose maximum is kept
constexpr int kGroupsMost = 24;    // sv_max_vocab on one CTA
constexpr int kList = 2048;        // tokens sorted at a time
constexpr int kBoundMost = 384;    // thread maxima a top-k bound may count down
constexpr int kBinShift = 6;       // 64 bins an octave of weights
constexpr int kBins = 64 << kBinShift;
constexpr uint32_t kCarryBits = 12;   // of a bin's upper word; its count above (V < 2^20)

// What rank 0 of a row's cluster asks of all its CTAs next.
enum : int { kCmdEnd = 0, kCmdGather = 1, kCmdWrite = 2, kCmdRecount = 3 };

struct Command {
    int op;
    int from, to, also;    // kCmdGather: bins from .. to, and bin `also`
    uint32_t key;          // kCmdWrite, kCmdRecount: the kept prefix's last token
    int index;
};

struct FilterShared {
    union {
        struct {
            uint32_t lo[kBins], hi[kBins];
        } bin;
        float group[kGroupsMost][kFilterThreads];
    };
    uint64_t list[kList];
    uint64_t roots[64];
    u128 part[kFilterWarps];
    u128 sum, found_mass;
    Command cmd;
    RowScale scale;
    uint32_t least_key;    // min-p's border
    float max_of[kFilterWarps];
    float top;             // this CTA's largest logit
    uint32_t bound;        // this CTA's lower bound for the top-k
    int count;             // entries of this CTA's list
    int first;             // lowest index of the largest logit
    int found, found_r;
};

// ---------------------------------------------------------------------------
// the row, the block and the cluster
// ---------------------------------------------------------------------------

// A CTA's part of a row: a range of its 16-byte vectors, and for rank 0 the
// elements before and after them.  Plain loads throughout: the filtered row may
// be written where the row is.
template <typename T> struct RowSpan {
    static constexpr int E = Elem<T>::E;
    const T* p;
    int V, head, nvec, v0, v1;
    __device__ RowSpan(const T* row, int V_, int rank, int C) : p(row), V(V_)
    {
        const int phase = (int)(((uintptr_t)row & 15) / sizeof(T));
        head = min(V, phase ? E - phase : 0);
        nvec = (V - head) / E;
        v0 = (int)((long long)nvec * rank / C);
        v1 = (int)((long long)nvec * (rank + 1) / C);
        rest = rank == 0 ? V - nvec * E : 0;
    }
    int rest;
    __device__ __forceinline__ const uint4* vec() const { return reinterpret_cast<const uint4*>(p + head); }
    // the index of this thread's element outside the vectors, or -1
    __device__ __forceinline__ int lone() const
    {
        const int t = threadIdx.x;
        return t < rest ? (t < head ? t : nvec * E + t) : -1;
    }
    // f(values, index of the first) for every vector, four loads in flight
    template <typename F> __device__ __forceinline__ void vectors(F&& f) const
    {
        const uint4* v = vec();
        for (int i0 = v0 + threadIdx.x; i0 < v1; i0 += 4 * kFilterThreads) {
            uint4 w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i0 + u * kFilterThreads < v1)
                    w[u] = v[i0 + u * kFilterThreads];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i0 + u * kFilterThreads < v1) {
                    float x[E];
                    Elem<T>::unpack(w[u], x);
                    f(x, head + (i0 + u * kFilterThreads) * E);
                }
        }
    }
    // f(value, index) for every element
    template <typename F> __device__ __forceinline__ void each(F&& f) const
    {
        vectors([&](const float (&x)[E], int i) {
#pragma unroll
            for (int k = 0; k < E; ++k)
                f(x[k], i + k);
        });
        const int i = lone();
        if (i >= 0)
            f((float)p[i], i);
    }
};

__device__ __forceinline__ uint32_t ld_rank(const void* p, int rank)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(smem_addr(p), rank)) : "memory");
    return v;
}

__device__ __forceinline__ uint64_t ld_rank64(const void* p, int rank)
{
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(map_to_rank(smem_addr(p), rank)) : "memory");
    return v;
}

__device__ __forceinline__ void row_sync(int C)
{
    if (C > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
}

__device__ __forceinline__ u128 shfl_up128(u128 v, int o)
{
    const unsigned long long lo = __shfl_up_sync(kFull, (unsigned long long)v, o);
    const unsigned long long hi = __shfl_up_sync(kFull, (unsigned long long)(v >> 64), o);
    return ((u128)hi << 64) | lo;
}

// Exclusive prefix sum over the block; `total` gets the whole.
__device__ __forceinline__ u128 block_scan(u128 v, FilterShared& s, u128& total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    u128 x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u128 y = shfl_up128(x, o);
        if (lane >= o)
            x += y;
    }
    __syncthreads();
    if (lane == 31)
        s.part[w] = x;
    __syncthreads();
    u128 before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kFilterWarps; ++i) {
        const u128 q = s.part[i];
        if (i < w)
            before += q;
        all += q;
    }
    total = all;
    return before + x - v;
}

__device__ __forceinline__ u128 block_sum(u128 v, FilterShared& s)
{
    u128 t;
    block_scan(v, s, t);
    return t;
}

// The last token of a prefix of the order.
struct Prefix {
    uint32_t key;
    int index;
    __device__ __forceinline__ bool has(uint32_t k, int i) const { return k > key || (k == key && i <= index); }
};

// ---------------------------------------------------------------------------
// Any row: bisection (one CTA).  Tens of passes over the row; it takes rows whose
// border lies among more equal or nearly equal logits than a list holds, and
// rows of nearly no temperature.
// ---------------------------------------------------------------------------

// The sum over a prefix of 1 (kCount) or of the weights.
template <bool kCount, typename T>
__device__ u128 prefix_sum(const RowSpan<T>& row, Prefix p, const RowScale& sc, FilterShared& s)
{
    u128 a = 0;
    row.each([&](float x, int i) {
        if (p.has(key_of(x), i))
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
        const uint32_t mid = lo + (hi - lo) / 2 + 1;
        if (prefix_sum<kCount>(row, Prefix{mid, INT_MAX}, sc, s) >= goal)
            lo = mid;
        else
            hi = mid - 1;
    }
    const u128 above = prefix_sum<kCount>(row, Prefix{lo + 1, INT_MAX}, sc, s);
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

// ---------------------------------------------------------------------------
// the result of a row
// ---------------------------------------------------------------------------
struct Settings {
    float T, p, min_p, u;
    int k;
};

// A row's numbers.  (64-bit floating point runs at a hundredth of the fp32
// rate: one thread's at most, never a block's.)
template <bool DRAW>
__device__ __forceinline__ void put_row(const FilterArgs& a, long long r, int kept, int token = -1, uint64_t weight = 0, u128 mass = 0)
{
    if (threadIdx.x == 0) {
        if (a.has_kept)
            a.out_kept[r] = kept;
        if (DRAW) {
            a.out_tokens[r] = token;
            if (a.has_prob)
                a.out_prob[r] = token < 0 ? __int_as_float(0x7fc00000) : (float)((double)weight / (double)mass);
        }
    }
}

// This CTA's part of the filtered row: what the prefix holds, -inf for the rest.
template <typename T> struct Bits;
template <> struct Bits<float> {
    typedef uint32_t type;
    static constexpr uint32_t ninf = 0xff800000u, nan = 0x7fc00000u;
};
template <> struct Bits<__nv_bfloat16> {
    typedef unsigned short type;
    static constexpr unsigned short ninf = 0xff80u, nan = 0x7fc0u;
};

template <typename T>
__device__ __forceinline__ void write_row(const RowSpan<T>& row, T* out, bool same_phase, Prefix end)
{
    typedef typename Bits<T>::type U;
    constexpr int E = Elem<T>::E;
    const float kv = value_of(end.key);
    U* o = reinterpret_cast<U*>(out);
    const U* x = reinterpret_cast<const U*>(row.p);
    if (same_phase) {
        const uint4* v = row.vec();
        uint4* ov = reinterpret_cast<uint4*>(o + row.head);
        for (int i0 = row.v0 + threadIdx.x; i0 < row.v1; i0 += 4 * kFilterThreads) {
            uint4 w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i0 + u * kFilterThreads < row.v1)
                    w[u] = v[i0 + u * kFilterThreads];   // (out may be the row)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + u * kFilterThreads;
                if (i < row.v1) {
                    float f[E];
                    Elem<T>::unpack(w[u], f);
                    union {
                        uint4 v;
                        U e[E];
                    } y;
                    y.v = w[u];
#pragma unroll
                    for (int k = 0; k < E; ++k)
                        if (!(f[k] > kv || (f[k] == kv && row.head + i * E + k <= end.index)))
                            y.e[k] = Bits<T>::ninf;
                    ov[i] = y.v;
                }
            }
        }
    } else {
        for (int j = row.head + row.v0 * E + threadIdx.x; j < row.head + row.v1 * E; j += kFilterThreads) {
            const float f = (float)row.p[j];
            o[j] = f > kv || (f == kv && j <= end.index) ? x[j] : Bits<T>::ninf;
        }
    }
    const int j = row.lone();
    if (j >= 0) {
        const float f = (float)row.p[j];
        o[j] = f > kv || (f == kv && j <= end.index) ? x[j] : Bits<T>::ninf;
    }
}

template <typename T>
__device__ __forceinline__ void fill_row(const RowSpan<T>& row, T* out, bool same_phase, typename Bits<T>::type what)
{
    typedef typename Bits<T>::type U;
    constexpr int E = Elem<T>::E;
    U* o = reinterpret_cast<U*>(out);
    if (same_phase) {
        const uint32_t w = sizeof(T) == 4 ? (uint32_t)what : (uint32_t)what * 0x10001u;
        uint4* ov = reinterpret_cast<uint4*>(o + row.head);
        for (int i = row.v0 + threadIdx.x; i < row.v1; i += kFilterThreads)
            ov[i] = make_uint4(w, w, w, w);
    } else {
        for (int j = row.head + row.v0 * E + threadIdx.x; j < row.head + row.v1 * E; j += kFilterThreads)
            o[j] = what;
    }
    const int j = row.lone();
    if (j >= 0)
        o[j] = what;
}

// The lowest logit that min-p keeps: the least float at or above m + T ln(min_p).
__device__ __forceinline__ uint32_t min_p_key(float m, double t_log)
{
    const double t = (double)m + t_log;
    const float least = (float)fmax(t, -3.4028234663852886e38);
    return (double)least < t ? key_of(least) + 1 : key_of(least);
}

// By bisection, rank 0 alone.
template <typename T, bool DRAW>
__device__ __noinline__ void whole_row(const FilterArgs& a, long long r, const Settings& g, float m, Prefix end, const RowScale& sc, FilterShared& s)
{
    const RowSpan<T> row(static_cast<const T*>(a.logits) + r * a.V, a.V, 0, 1);
    const uint32_t top = key_of(m);
    u128 mass = 0;
    if (g.k > 0 && prefix_sum<true>(row, end, sc, s) > (u128)g.k)
        end = prefix_reaching<true>(row, (u128)g.k, end, top, sc, s);
    if (g.p < 1.0f || DRAW)
        mass = prefix_sum<false>(row, end, sc, s);
    if (g.p < 1.0f) {
        const u128 goal = share_of(g.p, mass, true);
        end = prefix_reaching<false>(row, goal > 1 ? goal : 1, end, top, sc, s);
        if (DRAW)
            mass = prefix_sum<false>(row, end, sc, s);
    }
    const int kept = a.has_kept ? (int)prefix_sum<true>(row, end, sc, s) : 0;
    if (DRAW) {
        const Prefix at = prefix_reaching<false>(row, share_of(g.u, mass, false) + 1, end, top, sc, s);
        put_row<DRAW>(a, r, kept, at.index, weight62(value_of(at.key), sc, s.roots), mass);
    } else {
        put_row<DRAW>(a, r, kept);
        write_row(row, static_cast<T*>(a.out) + r * a.V, a.same_phase, end);
    }
}

// ---------------------------------------------------------------------------
// Few candidates: the list
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t entry_of(uint32_t key, int index) { return ((uint64_t)key << 32) | (0xffffffffu - (uint32_t)index); }
__device__ __forceinline__ uint32_t entry_key(uint64_t e) { return (uint32_t)(e >> 32); }
__device__ __forceinline__ int entry_index(uint64_t e) { return (int)(0xffffffffu - (uint32_t)e); }

__device__ __forceinline__ void append(FilterShared& s, uint32_t key, int index)
{
    const int at = atomicAdd(&s.count, 1);
    if (at < kList)
        s.list[at] = entry_of(key, index);
}

// The lists of the cluster's CTAs one after the other in rank 0's; the total,
// which every CTA learns (above kList: nothing is copied).  Ends the phase that
// reads other CTAs' lists only with the next row_sync.
__device__ __forceinline__ int collect(FilterShared& s, int rank, int C)
{
    row_sync(C);
    int total = s.count;
    if (C > 1) {
        total = 0;
        int before = 0;
        for (int c = 0; c < C; ++c) {
            const int n = (int)ld_rank(&s.count, c);
            before = total;
            total += n;
            if (rank == 0 && c > 0 && total <= kList)
                for (int i = threadIdx.x; i < n; i += kFilterThreads)
                    s.list[before + i] = ld_rank64(&s.list[i], c);
        }
        __syncthreads();
    }
    return total;
}

// Sorts list[0 .. n), the largest first.
__device__ __forceinline__ void sort_list(FilterShared& s, int n)
{
    const int t = threadIdx.x;
    if (n <= kFilterThreads) {   // each entry counts those before it
        const uint64_t e = t < n ? s.list[t] : 0;
        int r = 0;
        if (t < n)
            for (int j = 0; j < n; ++j)
                r += s.list[j] > e;
        __syncthreads();
        if (t < n)
            s.list[r] = e;
    } else {
        int size = 1024;
        while (size < n)
            size *= 2;
        for (int i = n + t; i < size; i += kFilterThreads)
            s.list[i] = 0;
        for (int k = 2; k <= size; k <<= 1)
            for (int j = k >> 1; j > 0; j >>= 1) {
                __syncthreads();
                for (int i = t; i < size / 2; i += kFilterThreads) {
                    const int x = 2 * i - (i & (j - 1)), y = x + j;
                    const uint64_t p = s.list[x], q = s.list[y];
                    if ((p < q) == ((x & k) == 0)) {
                        s.list[x] = q;
                        s.list[y] = p;
                    }
                }
            }
    }
    __syncthreads();
}

// A thread's entries of the sorted list, and the mass before each of its own.
struct ListPart {
    int r0, n;                         // ranks r0 .. r0 + n - 1
    uint64_t w[kList / kFilterThreads];
    u128 before;                       // mass of the ranks below r0
};

__device__ __forceinline__ ListPart weigh_list(FilterShared& s, int n, const RowScale& sc, u128& total)
{
    ListPart q;
    const int per = (n + kFilterThreads - 1) / kFilterThreads;
    q.r0 = min(n, (int)threadIdx.x * per);
    q.n = min(n, q.r0 + per) - q.r0;
    u128 sum = 0;
#pragma unroll
    for (int i = 0; i < kList / kFilterThreads; ++i) {
        q.w[i] = i < q.n ? weight62(value_of(entry_key(s.list[q.r0 + i])), sc, s.roots) : 0;
        sum += q.w[i];
    }
    q.before = block_scan(sum, s, total);
    return q;
}

// The first rank of lo .. hi - 1 whose cumulative mass, counted from rank lo on
// and with `base` before it, reaches goal (hi - 1 if none does); its mass in
// `mass`.
__device__ __forceinline__ int rank_reaching(const ListPart& q, int lo, int hi, u128 base, u128 goal, FilterShared& s, u128& mass)
{
    __syncthreads();
    if (threadIdx.x == 0) {
        s.found_r = lo;
        s.sum = 0;
    }
    __syncthreads();
    u128 c = q.before;
    if (lo > 0) {   // what is before rank lo
#pragma unroll
        for (int i = 0; i < kList / kFilterThreads; ++i) {
            if (i < q.n && q.r0 + i == lo)
                s.sum = c;
            c += q.w[i];
        }
    }
    __syncthreads();
    const u128 skip = s.sum;
    c = q.before;
#pragma unroll
    for (int i = 0; i < kList / kFilterThreads; ++i) {
        const int r = q.r0 + i;
        const u128 was = c;
        c += q.w[i];
        if (i < q.n && r >= lo && r < hi) {
            const bool reached = base + (c - skip) >= goal, before = r > lo && base + (was - skip) >= goal;
            if ((reached && !before) || (r == hi - 1 && !reached)) {
                s.found_r = r;
                s.found_mass = base + (c - skip);
            }
        }
    }
    __syncthreads();
    mass = s.found_mass;
    return s.found_r;
}

// ---------------------------------------------------------------------------
// Any number of candidates: bins of weight
// ---------------------------------------------------------------------------
// A bin holds the tokens whose l log2(e) / T rounds to the same 64th; it sums
// 2^f - 1 of the remainders f, in units of 2^-29, and counts.  Bin 0 holds the
// largest logit.  The last bin holds whatever weighs less than 2^-63 too; its
// mass does not count.
constexpr float kMagicBin = 196608.0f;       // 1.5 * 2^17: adding it rounds to 64ths
constexpr float kMagicSum = 0.0234375f;      // 1.5 * 2^-6: adding it rounds to 2^-29

struct BinScale {
    float ch, cl, least;   // least: below it, the last bin
    uint32_t ref;          // the bits of the largest logit's rounded product
};

__device__ __forceinline__ BinScale bin_scale(float m, float T, const RowScale& sc)
{
    BinScale b;
    b.ch = sc.ch;
    b.cl = sc.cl;
    b.ref = __float_as_uint(__fadd_rn(__fmul_rn(m, sc.ch), kMagicBin));
    b.least = fmaxf(m - 44.6f * T, -3.4028234e38f);   // (64.3 octaves)
    return b;
}

__device__ __forceinline__ int bin_of(float l, const BinScale& b)
{
    const uint32_t x = b.ref - __float_as_uint(__fadd_rn(__fmul_rn(fmaxf(l, b.least), b.ch), kMagicBin));
    return (int)min(x, (uint32_t)kBins - 1);
}

__device__ __forceinline__ void bin_add(FilterShared& s, uint32_t x, uint32_t q)
{
    const uint32_t i = min(x, (uint32_t)kBins - 1);
    const uint32_t old = atomicAdd(&s.bin.lo[i], q);
    atomicAdd(&s.bin.hi[i], (1u << kCarryBits) + (old + q < old ? 1u : 0u));
}

// Two tokens; `in` says which of them count.
__device__ __forceinline__ void bin_pair(FilterShared& s, float l0, float l1, bool in0, bool in1, const BinScale& b)
{
    const uint64_t L = f2_pack(fmaxf(l0, b.least), fmaxf(l1, b.least));
    const uint64_t nt = f2_mul(L, f2_pack(-b.ch, -b.ch));
    const uint64_t e = f2_fma(L, f2_pack(b.cl, b.cl), f2_fma(L, f2_pack(b.ch, b.ch), nt));
    const uint64_t at = f2_sub(f2_pack(kMagicBin, kMagicBin), nt);
    const uint64_t f = f2_sub(e, f2_add(nt, f2_sub(at, f2_pack(kMagicBin, kMagicBin))));
    // 2^f - 1, |f| < 2^-7 + 2^-11: ln 2 f + (ln 2 f)^2 / 2 + (ln 2 f)^3 / 6, the next term below 2^-35
    const uint64_t g = f2_fma(f, f2_fma(f, f2_pack(0.05550411f, 0.05550411f), f2_pack(0.24022651f, 0.24022651f)), f2_pack(0.69314718f, 0.69314718f));
    const uint64_t q = f2_fma(f, g, f2_pack(kMagicSum, kMagicSum));
    const uint32_t unit = 0x3c800000u;   // 2^-6: q's bits less these are (2^f - 1 + 2^-7) 2^29
    if (in0)
        bin_add(s, b.ref - (uint32_t)at, (uint32_t)q - unit);
    if (in1)
        bin_add(s, b.ref - (uint32_t)(at >> 32), (uint32_t)(q >> 32) - unit);
}

__device__ __forceinline__ uint32_t bin_count(const FilterShared& s, int i) { return s.bin.hi[i] >> kCarryBits; }

// The mass of bin i in units of 2^-62, weights relative to 2^(1/64) times bin 0's centre.
__device__ __forceinline__ u128 bin_mass(const FilterShared& s, int i)
{
    if (i == kBins - 1)
        return 0;
    const uint32_t hi = s.bin.hi[i], n = hi >> kCarryBits;
    if (n == 0)
        return 0;
    const uint64_t sum = (((uint64_t)(hi & ((1u << kCarryBits) - 1)) << 32) | s.bin.lo[i]) + ((uint64_t)n << 29) - ((uint64_t)n << 22);
    return ((u128)sum * s.roots[(i + 1) & 63]) >> (29 + ((i + 1) >> 6));
}

// The bin where a running sum over all bins (counts, or masses) reaches `goal`;
// what is before the bin in `before`.  kBins if it is not reached.
template <bool kCount>
__device__ __forceinline__ int bin_reaching(FilterShared& s, u128 goal, u128& before, u128& total)
{
    constexpr int per = kBins / kFilterThreads;
    const int i0 = threadIdx.x * per;
    u128 v = 0;
    for (int i = 0; i < per; ++i)
        v += kCount ? bin_count(s, i0 + i) : bin_mass(s, i0 + i);
    u128 c = block_scan(v, s, total);
    __syncthreads();
    if (threadIdx.x == 0)
        s.found = kBins;
    __syncthreads();
    if (c < goal && goal <= c + v)
        for (int i = 0; i < per; ++i) {
            const u128 x = kCount ? bin_count(s, i0 + i) : bin_mass(s, i0 + i);
            if (goal <= c + x) {
                s.found = i0 + i;
                s.found_mass = c;
                break;
            }
            c += x;
        }
    __syncthreads();
    before = s.found_mass;
    return s.found;
}

// All of the cluster's bins in rank 0's.
__device__ __forceinline__ void merge_bins(FilterShared& s, int rank, int C)
{
    row_sync(C);
    if (C == 1)
        return;
    const int per = (kBins + C - 1) / C, i0 = rank * per, i1 = min(kBins, i0 + per);
    for (int i = i0 + threadIdx.x; i < i1; i += kFilterThreads) {
        uint64_t lo = 0;
        uint32_t hi = 0;
        for (int c = 0; c < C; ++c) {
            lo += ld_rank(&s.bin.lo[i], c);
            hi += ld_rank(&s.bin.hi[i], c);
        }
        s.bin.lo[i] = (uint32_t)lo;
        s.bin.hi[i] = hi + (uint32_t)(lo >> 32);
    }
    row_sync(C);
    if (rank == 0) {
        for (int i = per + threadIdx.x; i < kBins; i += kFilterThreads) {
            const int c = i / per;
            s.bin.lo[i] = ld_rank(&s.bin.lo[i], c);
            s.bin.hi[i] = ld_rank(&s.bin.hi[i], c);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <typename T, bool DRAW>
__global__ void __launch_bounds__(kFilterThreads, 2) sv_filter_kernel(FilterArgs a)
{
    extern __shared__ __align__(16) unsigned char filter_smem[];
    FilterShared& s = *reinterpret_cast<FilterShared*>(filter_smem);
    constexpr int E = Elem<T>::E;
    const int C = a.C, t = threadIdx.x, V = a.V;
    const int rank = C > 1 ? (int)cluster_ctarank() : 0;
    const long long r = blockIdx.x / (unsigned)C;
    const int b = (int)(r / a.S), nth = (int)(r % a.S);
    if (!DRAW && a.has_n && nth >= a.n_rows[b]) {   // no row: its logits and outputs stay
        if (rank == 0 && t == 0 && a.has_kept)
            a.out_kept[r] = 0;
        return;
    }
    Settings g;
    g.T = a.temperature[b];
    g.k = a.has_k ? a.top_k[b] : 0;
    g.p = a.has_p ? a.top_p[b] : 1.0f;
    g.min_p = a.has_m ? a.min_p[b] : 0.0f;
    g.u = DRAW && g.T != 0.0f ? a.uniforms[r] : 0.0f;
    const bool greedy = g.T == 0.0f;
    const bool good = temperature_usable(g.T) && g.k >= 0 && g.p >= 0.0f && g.p <= 1.0f && g.min_p >= 0.0f && g.min_p <= 1.0f &&
                      g.u >= 0.0f && g.u < 1.0f;
    const T* logits = static_cast<const T*>(a.logits) + r * V;
    T* out = static_cast<T*>(a.out) + (DRAW ? 0 : r * V);
    const RowSpan<T> row(logits, V, rank, C);

    double t_log = 0.0;   // thread 0's: what of the row's constants does not need its maximum
    if (t == 0 && good && !greedy) {
        s.scale = row_scale(g.T);
        if (g.min_p > 0.0f)
            t_log = (double)g.T * log((double)g.min_p);
    }

    // 1. The maxima of the row, of each thread, and of each thread's groups of
    // vectors: the one pass that has to read everything from memory.
    const int groups = (row.v1 - row.v0 + kGroup * kFilterThreads - 1) / (kGroup * kFilterThreads);
    float mine = -INFINITY;
    for (int n = 0; n < groups; ++n) {
        const int i0 = row.v0 + n * kGroup * kFilterThreads + t;
        uint4 w[kGroup];
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            const uint32_t none = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
            w[u] = make_uint4(none, none, none, none);
            if (i0 + u * kFilterThreads < row.v1)
                w[u] = row.vec()[i0 + u * kFilterThreads];
        }
        float top;
        if (sizeof(T) == 4) {
            top = -INFINITY;
#pragma unroll
            for (int u = 0; u < kGroup; ++u) {
                top = max3_nan(top, __uint_as_float(w[u].x), __uint_as_float(w[u].y));
                top = max3_nan(top, __uint_as_float(w[u].z), __uint_as_float(w[u].w));
            }
        } else {
            uint32_t x = 0xff80ff80u;
#pragma unroll
            for (int u = 0; u < kGroup; ++u)
                x = bmax2_nan(bmax2_nan(bmax2_nan(x, w[u].x), w[u].y), bmax2_nan(w[u].z, w[u].w));
            top = max_nan(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
        }
        s.group[n][t] = top;
        mine = max_nan(mine, top);
    }
    const int lone = row.lone();
    const float lone_x = lone >= 0 ? (float)logits[lone] : -INFINITY;
    mine = max_nan(mine, lone_x);
    if (t < 64)
        s.roots[t] = root_power(t);
    if (t == 0) {
        s.count = 0;
        s.first = INT_MAX;
    }
    const float warp_top = warp_max_nan(mine);
    if ((t & 31) == 0)
        s.max_of[t >> 5] = warp_top;
    __syncthreads();
    float m = s.max_of[0];
#pragma unroll
    for (int i = 1; i < kFilterWarps; ++i)
        m = max_nan(m, s.max_of[i]);

    // 2. With top-k, a logit that at least k of the row reach: in each of C CTAs
    // the k / C-th of the threads' maxima (about), the lowest of these.
    const int share = (g.k + C - 1) / C;
    const bool bounded = !greedy && g.k > 0 && share <= kBoundMost;
    uint32_t bound = 0;
    if (bounded) {
        const uint32_t key = key_of(mine);
        uint32_t lo = 0, hi = m < INFINITY ? key_of(m) : 0;   // (a NaN or +inf: no token will come of it)
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2 + 1;
            const int n = __syncthreads_count(key >= mid);
            if (n >= share) {
                lo = mid;
                if (n <= share + share / 4 + 4)
                    break;
            } else {
                hi = mid - 1;
            }
        }
        bound = lo;
    }
    if (C > 1) {
        if (t == 0) {
            s.top = m;
            s.bound = bound;
        }
        row_sync(C);
        for (int c = 0; c < C; ++c) {
            m = max_nan(m, __uint_as_float(ld_rank(&s.top, c)));
            bound = min(bound, ld_rank(&s.bound, c));
        }
    }

    const bool usable = good && m > -INFINITY && m < INFINITY;
    if (!usable) {
        if (rank == 0)
            put_row<DRAW>(a, r, -1);
        if (!DRAW)
            fill_row(row, out, a.same_phase, Bits<T>::nan);
        row_sync(C);
        return;
    }
    const uint32_t top_key = key_of(m);
    if (greedy) {
        for (int n = 0; n < groups; ++n)
            if (s.group[n][t] == m)
                for (int u = 0; u < kGroup; ++u) {
                    const int i = row.v0 + (n * kGroup + u) * kFilterThreads + t;
                    if (i < row.v1) {
                        float x[E];
                        Elem<T>::unpack(row.vec()[i], x);
#pragma unroll
                        for (int k = E - 1; k >= 0; --k)
                            if (x[k] == m)
                                atomicMin(&s.first, row.head + i * E + k);
                    }
                }
        if (lone >= 0 && lone_x == m)
            atomicMin(&s.first, lone);
        row_sync(C);
        int first = s.first;
        for (int c = 1; c < C; ++c)
            first = min(first, (int)ld_rank(&s.first, c == rank ? 0 : c));
        if (rank == 0)
            put_row<DRAW>(a, r, 1, first, 1, 1);
        row_sync(C);
        if (!DRAW)
            write_row(row, out, a.same_phase, Prefix{top_key, first});
        return;
    }

    if (t == 0) {
        s.scale.at(m, g.T);
        s.least_key = max(kKeyNegInf + 1, g.min_p > 0.0f ? min_p_key(m, t_log) : 0u);
    }
    __syncthreads();
    Prefix end{s.least_key, INT_MAX};
    RowScale sc = s.scale;

    // 3. Few candidates (a top-k bound, min-p, or a short row): they are read
    // again, by the groups that hold one, sorted and weighed.
    if (bounded || g.min_p > 0.0f || V <= kList) {
        const uint32_t cut = max(end.key, bound);
        const float cv = value_of(cut);
        for (int n = 0; n < groups; ++n)
            if (s.group[n][t] >= cv)
                for (int u = 0; u < kGroup; ++u) {
                    const int i = row.v0 + (n * kGroup + u) * kFilterThreads + t;
                    if (i < row.v1) {
                        float x[E];
                        Elem<T>::unpack(row.vec()[i], x);
#pragma unroll
                        for (int k = 0; k < E; ++k)
                            if (x[k] >= cv)
                                append(s, key_of(x[k]), row.head + i * E + k);
                    }
                }
        if (lone >= 0 && lone_x >= cv)
            append(s, key_of(lone_x), lone);
        int n = collect(s, rank, C);
        if (n <= kList) {
            if (!DRAW)
                fill_row(row, out, a.same_phase, Bits<T>::ninf);
            row_sync(C);   // lists have been read; all of out is -inf
            if (rank != 0)
                return;
            sort_list(s, n);
            if (g.k > 0)
                n = min(n, g.k);
            u128 mass = 0;
            ListPart q;
            if (DRAW || g.p < 1.0f)
                q = weigh_list(s, n, sc, mass);
            if (g.p < 1.0f) {
                const u128 goal = share_of(g.p, mass, true);
                n = rank_reaching(q, 0, n, 0, goal > 1 ? goal : 1, s, mass) + 1;
            }
            if (DRAW) {
                u128 to;
                const int at = rank_reaching(q, 0, n, 0, share_of(g.u, mass, false) + 1, s, to);
                const uint64_t e = s.list[at];
                put_row<DRAW>(a, r, n, entry_index(e), weight62(value_of(entry_key(e)), sc, s.roots), mass);
            } else {
                put_row<DRAW>(a, r, n);
                for (int i = t; i < n; i += kFilterThreads) {
                    const int j = entry_index(s.list[i]);
                    out[j] = (T)value_of(entry_key(s.list[i]));
                }
            }
            return;
        }
        row_sync(C);   // too many (every CTA has read the counts): the bins take them
    }

    // 4. Nothing but min-p, if that: every token above its border stays.
    if (!DRAW && g.p >= 1.0f && g.k == 0) {
        int n = 0;
        const float least = value_of(end.key);
        row.each([&](float x, int) { n += x >= least; });
        const int all = (int)block_sum((u128)n, s);
        if (t == 0)
            s.count = all;
        row_sync(C);
        int total = 0;
        for (int c = 0; c < C; ++c)
            total += C > 1 ? (int)ld_rank(&s.count, c) : all;
        if (rank == 0)
            put_row<DRAW>(a, r, total);
        row_sync(C);
        write_row(row, out, a.same_phase, end);
        return;
    }

    // 5. The bins.
    if (sc.cold) {
        if (rank == 0)
            whole_row<T, DRAW>(a, r, g, m, end, s.scale, s);
        row_sync(C);
        return;
    }
    const BinScale bs = bin_scale(m, g.T, sc);
    sc.top = ((long long)(int)(bs.ref - __float_as_uint(kMagicBin)) + 1) * (1ll << (48 - kBinShift));   // as the bins' masses
    int k = g.k;
    for (;;) {
        __syncthreads();
        for (int i = t; i < kBins; i += kFilterThreads)
            s.bin.lo[i] = s.bin.hi[i] = 0;
        __syncthreads();
        const float least = value_of(end.key);
        const bool all = end.index == INT_MAX;
        row.vectors([&](const float (&x)[E], int i) {
#pragma unroll
            for (int j = 0; j < E; j += 2)
                bin_pair(s, x[j], x[j + 1], x[j] > least || (x[j] == least && (all || i + j <= end.index)),
                         x[j + 1] > least || (x[j + 1] == least && (all || i + j + 1 <= end.index)), bs);
        });
        if (lone >= 0)
            bin_pair(s, lone_x, lone_x, lone_x > least || (lone_x == least && lone <= end.index), false, bs);
        merge_bins(s, rank, C);
        bool again = false;
        Prefix stop{0, 0};
        int stage = 0;   // rank 0's: what the gathered list is for
        int kept = 0, last = 0, first_bin = 0, n_first = 0, listed = 0;
        u128 above = 0, above_first = 0, total = 0, mass = 0, goal = 0;
        for (;;) {
            if (rank == 0) {
                Command c{kCmdEnd, 0, 0, -1, 0, 0};
                bool give_up = false;
                if (stage == 0) {
                    u128 n_all, before;
                    const int bk = bin_reaching<true>(s, k > 0 ? (u128)k : ~(u128)0, before, n_all);
                    if (k > 0 && (u128)k < n_all) {   // top-k first: its last token
                        stage = 1;
                        kept = k - (int)before;
                        c.op = kCmdGather;
                        c.from = c.to = c.also = bk;
                        give_up = bin_count(s, bk) > kList;
                    } else {
                        kept = (int)n_all;
                        u128 none;
                        bin_reaching<false>(s, ~(u128)0, none, total);
                        mass = total;
                        stage = 2;
                        if (g.p < 1.0f) {
                            goal = share_of(g.p, total, true);
                            goal = goal > 1 ? goal : 1;
                            last = bin_reaching<false>(s, goal, above, none);
                            // the draw's point lies between u times the goal and that plus u times a token of the last bin
                            int d0 = last, d1 = last;
                            above_first = above;
                            if (DRAW) {
                                u128 x;
                                d0 = bin_reaching<false>(s, share_of(g.u, goal, false) + 1, above_first, none);
                                const u128 one = ((u128)s.roots[last & 63] >> (last >> 6)) + (total >> 24);
                                d1 = bin_reaching<false>(s, share_of(g.u, goal + one, false) + 1, x, none);
                                d0 = min(d0, last);
                                d1 = max(d0, min(d1, last));
                            }
                            int n = 0, nl = 0;
                            for (int i = d0 + t; i <= d1; i += kFilterThreads)
                                n += (int)bin_count(s, i);
                            n_first = (int)block_sum((u128)n, s);
                            nl = d1 < last ? (int)bin_count(s, last) : 0;
                            c.op = kCmdGather;
                            c.from = d0;
                            c.to = d1;
                            c.also = last;
                            first_bin = d0;
                            if (n_first + nl > kList) {   // not both at once: the last bin first
                                stage = 3;
                                c.from = c.to = last;
                                first_bin = last;
                                above_first = above;
                                n_first = (int)bin_count(s, last);
                                give_up = n_first > kList;
                            }
                            n = 0;
                            for (int i = t; i < last; i += kFilterThreads)
                                n += (int)bin_count(s, i);
                            kept = (int)block_sum((u128)n, s);
                        } else if (!DRAW) {   // top-k reaches past the last token
                            put_row<DRAW>(a, r, kept);
                            c.op = kCmdWrite;
                            c.key = end.key;
                            c.index = end.index;
                        } else {
                            stage = 4;
                            first_bin = bin_reaching<false>(s, share_of(g.u, total, false) + 1, above_first, none);
                            c.op = kCmdGather;
                            c.from = c.to = c.also = first_bin;
                            give_up = bin_count(s, first_bin) > kList;
                        }
                    }
                } else if (stage == 1) {
                    sort_list(s, listed);
                    const uint64_t e = s.list[kept - 1];
                    c.op = kCmdRecount;
                    c.key = entry_key(e);
                    c.index = entry_index(e);
                } else {
                    const int n = listed;
                    u128 sum;
                    sort_list(s, n);
                    const ListPart q = weigh_list(s, n, sc, sum);
                    bool draw_now = DRAW;
                    int hi = n;
                    u128 at_mass;
                    if (stage == 2 || stage == 3) {
                        // the last bin's tokens are the list's last ones, or all of a range that ends with it
                        const int nl = (int)bin_count(s, last), lo = n - nl;
                        u128 own = 0;
                        rank_reaching(q, lo, n, 0, ~(u128)0, s, own);
                        goal = share_of(g.p, total - bin_mass(s, last) + own, true);   // with that bin's exact mass
                        goal = goal > 1 ? goal : 1;
                        const int end_r = rank_reaching(q, lo, n, above, goal, s, mass);
                        kept += end_r - lo + 1;
                        stop = Prefix{entry_key(s.list[end_r]), entry_index(s.list[end_r])};
                        hi = end_r + 1;
                        if (!DRAW) {
                            put_row<DRAW>(a, r, kept);
                            c.op = kCmdWrite;
                            c.key = stop.key;
                            c.index = stop.index;
                        } else if (stage == 3 && share_of(g.u, mass, false) + 1 <= above) {   // the draw is in a bin before
                            draw_now = false;
                            stage = 4;
                            u128 none;
                            first_bin = bin_reaching<false>(s, share_of(g.u, mass, false) + 1, above_first, none);
                            c.op = kCmdGather;
                            c.from = c.to = c.also = first_bin;
                            give_up = bin_count(s, first_bin) > kList;
                        } else if (stage == 2 && first_bin < last && share_of(g.u, mass, false) + 1 > above) {
                            // the point is in the last bin after all
                            const int at = rank_reaching(q, lo, hi, above, share_of(g.u, mass, false) + 1, s, at_mass);
                            const uint64_t e = s.list[at];
                            put_row<DRAW>(a, r, kept, entry_index(e), weight62(value_of(entry_key(e)), sc, s.roots), mass);
                            draw_now = false;
                        } else if (stage == 2 && first_bin < last) {
                            hi = n_first < lo ? n_first : lo;
                            hi = hi > 0 ? hi : 1;
                        }
                    }
                    if (draw_now) {
                        const int at = rank_reaching(q, 0, hi, above_first, share_of(g.u, mass, false) + 1, s, at_mass);
                        const uint64_t e = s.list[at];
                        put_row<DRAW>(a, r, kept, entry_index(e), weight62(value_of(entry_key(e)), sc, s.roots), mass);
                    }
                }
                if (give_up) {
                    Settings rest = g;
                    rest.k = k;
                    c = Command{kCmdEnd, 0, 0, -1, 0, 0};
                    whole_row<T, DRAW>(a, r, rest, m, end, s.scale, s);
                }
                __syncthreads();
                if (t == 0) {
                    s.cmd = c;
                    s.count = 0;
                }
            } else if (t == 0) {
                s.count = 0;
            }
            row_sync(C);
            const int op = C > 1 ? (int)ld_rank(&s.cmd.op, 0) : s.cmd.op;
            if (op == kCmdEnd)
                break;
            if (op == kCmdGather) {
                const int from = C > 1 ? (int)ld_rank(&s.cmd.from, 0) : s.cmd.from, to = C > 1 ? (int)ld_rank(&s.cmd.to, 0) : s.cmd.to;
                const int also = C > 1 ? (int)ld_rank(&s.cmd.also, 0) : s.cmd.also;
                row.each([&](float x, int i) {
                    const int n = bin_of(x, bs);
                    if (((n >= from && n <= to) || n == also) && end.has(key_of(x), i))
                        append(s, key_of(x), i);
                });
                listed = collect(s, rank, C);
                row_sync(C);   // the lists have been read
                continue;
            }
            stop.key = C > 1 ? ld_rank(&s.cmd.key, 0) : s.cmd.key;
            stop.index = C > 1 ? (int)ld_rank(&s.cmd.index, 0) : s.cmd.index;
            if (op == kCmdWrite) {
                row_sync(C);
                write_row(row, out, a.same_phase, stop);
                return;
            }
            again = true;   // kCmdRecount
            end = stop;
            break;
        }
        row_sync(C);
        if (!again)
            return;
        if (!DRAW && g.p >= 1.0f) {   // top-k was all there was
            if (rank == 0)
                put_row<DRAW>(a, r, k);
            write_row(row, out, a.same_phase, end);
            return;
        }
        k = 0;
    }
}

}  // namespace sv
