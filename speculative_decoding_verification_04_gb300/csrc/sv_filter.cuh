// sv_filter.cuh -- min-p, top-k and top-p over rows of logits: the kept set, a
// draw from it, and the row with the rest at -inf.
//
// Order a row's tokens by logit, the largest first, equal ones by index.  Each
// filter keeps a prefix of that order, and so does their sequence; a prefix is
// named by its last token (key, index).  A draw is the end of a prefix too: of
// the shortest one whose mass is above u Z.  So everything is one question:
// where does a prefix reach a given count or mass?
//
// Four ways to the answer, by a row's settings:
//  - a list (top-k up to 128 or 256 a CTA, min-p, short rows): the row's one pass
//    from memory keeps the maxima of each thread and of its groups of four vectors;
//    the k-th largest of the threads' maxima bounds the k-th largest logit, the
//    few groups above it are read again, and what passes is sorted and weighed.
//    Bounded by the bytes for many rows: 1024 rows of 128256 bf16 draw by top-k 50
//    in 59 us (4.4 TB/s, 0.66 of the copy rate), 900 are filtered in 86 (5.4 TB/s
//    read and written, 0.80); by the chain of steps for one row (9 us).
//  - levels (bf16 where every token counts): the one pass counts how often each
//    of 8192 values occurs, an atomic a token; weights times counts are the sums.
//    1024 rows of 128256 draw in 141 us (1.9 TB/s): what bounds it is the atomics
//    in shared memory, some ten cycles for each warp's.
//  - bins (fp32 where every token counts): sums by weight, and the border's bins
//    read once more.  256 rows of 151936 draw in 154 us (1.0 TB/s of the one pass
//    that has to be): bounded by two atomics a token, the arithmetic of the
//    remainders, and three sweeps of rows that L2 does not hold all of.
//  - bisection, for what none of these settles: right for any row and slow, 2 to 11
//    ms for one of them (which ones stands there).
// All four compare whole numbers, so that none depends on the order of its sums.
// How finely they count: sums of a list in 2^-52 of the largest weight, of levels in
// 2^-42 of the largest of 32 neighbouring values, of bins in 2^-29 of the bin's own
// weight, of bisection in 2^-62 of the largest weight.
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

// Threads a row: 256 for bf16 (three blocks an SM), 512 for fp32 (two).  What a row
// costs beside its bytes is a chain of short steps (maxima, bound, candidates, sums,
// the crossing), which more threads shorten and more rows at a time hide.  By 256 and
// by 512: 1024 rows of 128256 bf16 with top-p 141 and 165 us, with top-k 50 59 and 67;
// 256 rows of 151936 fp32 with top-p 159 and 154 us, 64 rows 81 and 68.  A fourth block
// an SM leaves L1, through which the loads in flight pass, 28 KB: top-k 50 64 us for
// 59, 900 filtered rows 104 for 86, top-p 139 for 141.
template <typename T> constexpr int kThreadsOf = sizeof(T) == 2 ? 256 : 512;
template <typename T> constexpr int kBlocksOf = sizeof(T) == 2 ? 3 : 2;
// Rows of at most kShortMost tokens, all of them in the list: 128 threads, eight blocks
// an SM without the sums' shared memory.  By these and by 512 threads: 7680 rows of 1000
// fp32 filtered by top-p 207 and 487 us, 600 rows of 300 drawn 18 and 29, one row of 300
// 12 and 10.
constexpr int kShortThreads = 128, kShortBlocks = 8, kShortMost = 8 * kShortThreads;
constexpr int kClusterMost = 8;
constexpr int kGroup = 4;          // vectors of a thread whose maximum is kept (1024 rows, top-k 50: 59 us; by eights 65)
constexpr int kList = 2048;        // tokens sorted at a time
constexpr int kBins = 4096;
constexpr int kBinShift = 6;       // 64 bins an octave of weights
template <int NT> constexpr int kBinsEach = kBins / NT;
constexpr int kLevelsSide = 4097;   // bf16 magnitudes: 2^-24 (and below) to 2^8 one by one, from 2^8
constexpr int kLevels = 2 * kLevelsSide;
template <int NT> constexpr int kLevelsEach = 4096 * 2 / NT;
template <int NT> constexpr int kGroupsMost = 50 * 512 / NT;   // sv_max_vocab on one CTA
constexpr int kFewKept = 512;      // kept tokens that are all listed
constexpr uint32_t kCarryBits = 12;   // of a bin's upper word; its count above (V < 2^20)

// What rank 0 of a row's cluster asks of all its CTAs next.
enum : int { kCmdEnd = 0, kCmdGather = 1, kCmdWrite = 2, kCmdRecount = 3 };

struct alignas(16) Command {
    int op;
    int from, to, also;    // kCmdGather: bins from .. to, and bin `also`
    uint32_t key;          // kCmdWrite: the kept prefix's last token; kCmdRecount: top-k's
    int index;
    int pad;
    float value;           // kCmdGather of bf16 levels: the logit
};

// A value among whose tokens a running sum reaches a goal.
struct LevelAt {
    float value;
    uint64_t weight;        // of one of its tokens, in units of 2^-62
    int n, n_before;        // its tokens, and those before them
    u128 before, mass;      // the mass before them, and theirs in the sums
};

struct BinAt {
    int bin, n_before;     // a bin, and what is before it
    u128 before;
};

template <int NT> struct FilterShared {
    alignas(16) uint64_t list[kList];
    uint64_t roots[64];
    u128 part[NT / 32];
    u128 found_mass;
    RowScale scale;
    LevelAt level_at;
    BinAt bin_at;
    uint64_t part64[NT / 32], found64, found_ratio;
    uint32_t steps[kBinsEach<NT>];   // 2^31 times 2^(-j / 64)
    Command cmd;
    uint32_t warp_top[NT / 32], warp_low[NT / 32];
    int warp_count[2][NT / 32];
    uint32_t peer_top[kClusterMost], peer_bound[kClusterMost];   // what each CTA of the cluster found
    int peer_kept[kClusterMost];
    uint32_t least_key;    // min-p's border
    int count;             // rank 0: entries of the list
    int hits;              // groups that hold a candidate
    int first;             // lowest index of the largest logit
    int found, found_count, found_at;
    int top_level;         // the maximum's place among the levels, the largest first
    // the maxima of each thread's groups (as many as the row has) and behind them the
    // groups that hold a candidate (`hit`, kList of them), then the bins
    union alignas(16) {
        struct {
            uint32_t lo[kBins], hi[kBins];
        } bin;
        uint32_t level[kLevels];
        float group[kGroupsMost<NT>][NT];
    };
};

// Shared memory for rows of `groups` groups a CTA.
template <int NT> constexpr size_t filter_smem_bytes(int groups)
{
    const size_t g = (size_t)groups * NT * 4 + kList * sizeof(uint16_t);
    const size_t b = NT == kShortThreads ? 0 : ((size_t)kLevels * 4 + 15) / 16 * 16;   // (more than the bins)
    return sizeof(FilterShared<NT>) - sizeof(float) * kGroupsMost<NT> * NT + (g > b ? g : b);
}

// ---------------------------------------------------------------------------
// the row, the block and the cluster
// ---------------------------------------------------------------------------

// A row's vector, past L1 (no use of it there: 1024 rows of 128256 bf16 with top-p
// draw in 141 us, 148 by plain loads).  Not through the read-only path: the filtered
// row may be written where the row is.
__device__ __forceinline__ uint4 ld_row(const uint4* p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// N of a thread's vectors, at i, i + stride, ...; zeros for those past the end.
template <int N> struct Vectors {
    uint4 w[N];
    __device__ __forceinline__ void load(const uint4* v, int i, int end, int stride)
    {
#pragma unroll
        for (int u = 0; u < N; ++u)
            w[u] = i + u * stride < end ? ld_row(v + i + u * stride) : make_uint4(0, 0, 0, 0);
    }
};

// f(vector, its place, whether there) for the vectors at first + threadIdx.x,
// + stride, ... below `end`, by whole warps; four are on their way while four are
// worked on.  kRolled: f is in the code once, for longer ones: code that runs a
// few times a row comes from L2, and costs more than the moves do.
template <bool kRolled, typename F>
__device__ __forceinline__ void each_vector(const uint4* v, int first, int end, int stride, F&& f)
{
    const int t = threadIdx.x;
    Vectors<4> next;
    next.load(v, first + t, end, stride);
#pragma unroll 1
    for (int i = first + t; i - t < end; i += 4 * stride) {
        Vectors<4> now = next;
        next.load(v, i + 4 * stride, end, stride);
        if (kRolled) {
#pragma unroll 1
            for (int u = 0; u < 4; ++u) {
                f(now.w[0], i + u * stride, i + u * stride < end);
                now.w[0] = now.w[1];
                now.w[1] = now.w[2];
                now.w[2] = now.w[3];
            }
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                f(now.w[u], i + u * stride, i + u * stride < end);
        }
    }
}

// A CTA's part of a row: a range of its 16-byte vectors, and for rank 0 the
// elements before and after them.
template <typename T> struct RowSpan {
    static constexpr int E = Elem<T>::E;
    const T* p;
    int V, head, nvec, v0, v1, rest;
    __device__ RowSpan(const T* row, int V_, int rank, int C) : p(row), V(V_)
    {
        const int phase = (int)(((uintptr_t)row & 15) / sizeof(T));
        head = min(V, phase ? E - phase : 0);
        nvec = (V - head) / E;
        v0 = (int)((long long)nvec * rank / C);
        v1 = (int)((long long)nvec * (rank + 1) / C);
        rest = rank == 0 ? V - nvec * E : 0;
    }
    __device__ __forceinline__ const uint4* vec() const { return reinterpret_cast<const uint4*>(p + head); }
    // the index of this thread's element outside the vectors, or -1
    __device__ __forceinline__ int lone() const
    {
        const int t = threadIdx.x;
        return t < rest ? (t < head ? t : nvec * E + t) : -1;
    }
    // f(values, index of the first) for every vector.
    template <typename F> __device__ __forceinline__ void vectors(F&& f) const
    {
        each_vector<true>(vec(), v0, v1, (int)blockDim.x, [&](const uint4& w, int i, bool there) {
            float x[E];
            Elem<T>::unpack(w, x);
            if (there)
                f(x, head + i * E);
        });
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

__device__ __forceinline__ uint4 ld_rank128(const void* p, int rank)
{
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(map_to_rank(smem_addr(p), rank)) : "memory");
    return v;
}

__device__ __forceinline__ void st_rank(void* p, int rank, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_rank(smem_addr(p), rank)), "r"(v) : "memory");
}

__device__ __forceinline__ void st_rank64(void* p, int rank, uint64_t v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(map_to_rank(smem_addr(p), rank)), "l"(v) : "memory");
}

__device__ __forceinline__ void row_sync(int C)
{
    if (C > 1) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
}

// A CTA's shared memory may be reached from its cluster once it has started: every
// CTA says so as it begins, and waits for the others before its first store to one
// of them, behind its pass over the row.  Relaxed: no data goes with it (one row of
// 128256 bf16 with top-k 50 takes 9.0 us, 9.5 by an arrival that releases).
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }

__device__ __forceinline__ void peers_announce(int C)
{
    if (C > 1) {
        __syncwarp();
        cluster_arrive_relaxed();
    }
}

__device__ __forceinline__ void peers_started(int C)
{
    if (C > 1) {
        __syncwarp();
        cluster_wait();
    }
}

__device__ __forceinline__ u128 shfl_up128(u128 v, int o)
{
    const unsigned long long lo = __shfl_up_sync(kFull, (unsigned long long)v, o);
    const unsigned long long hi = __shfl_up_sync(kFull, (unsigned long long)(v >> 64), o);
    return ((u128)hi << 64) | lo;
}

// Exclusive prefix sum over the block; `total` gets the whole.
template <int NT> __device__ __noinline__ u128 block_scan(u128 v, FilterShared<NT>& s, u128& total)
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
    for (int i = 0; i < NT / 32; ++i) {
        const u128 q = s.part[i];
        if (i < w)
            before += q;
        all += q;
    }
    total = all;
    return before + x - v;
}

template <int NT> __device__ __forceinline__ u128 block_sum(u128 v, FilterShared<NT>& s)
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
// rows of nearly no temperature.  Which ones, what one of them and many of them take,
// and in brackets what a sort in torch operations takes for the same:
//  - |m| / T of 2839 and more, with top-p or no filter.  128256 bf16, T = 0.01, a
//    largest logit of 30: 1.7 ms, 1024 rows 6.4 (0.7 and 22).
//  - fewer than k logits over a finite mask.  128256 bf16, ten tokens over -1e4,
//    top-k 50: 2.8 ms, 1024 rows 13 (0.8 and 22).
//  - fp32 rows with more than 2048 tokens in the bin (T ln 2 / 64 wide) of the border
//    or of the draw.  151936 normal logits of deviation 0.5 with top-p 0.9, T = 3: a
//    draw 11 ms, a filtered row 5.4; 256 rows 17 and 8.7 (0.7 and 7).  Such draws from
//    T = 1.5 on, filtered rows from T = 3; at T = 1, 256 rows take 0.22 and 0.19 ms.
// ---------------------------------------------------------------------------

// The sum over a prefix of 1 (kCount) or of the weights.
template <bool kCount, typename T, int NT>
__device__ u128 prefix_sum(const RowSpan<T>& row, Prefix p, FilterShared<NT>& s)
{
    u128 a = 0;
    row.each([&](float x, int i) {
        if (p.has(key_of(x), i))
            a += kCount ? 1 : weight62(x, s.scale, s.roots);
    });
    return block_sum(a, s);
}

// The shortest prefix within `most` that sums to `goal` (which `most` does).
template <bool kCount, typename T, int NT>
__device__ Prefix prefix_reaching(const RowSpan<T>& row, u128 goal, Prefix most, uint32_t top, FilterShared<NT>& s)
{
    uint32_t lo = most.key, hi = top;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2 + 1;
        if (prefix_sum<kCount>(row, Prefix{mid, INT_MAX}, s) >= goal)
            lo = mid;
        else
            hi = mid - 1;
    }
    const u128 above = prefix_sum<kCount>(row, Prefix{lo + 1, INT_MAX}, s);
    int a = 0, b = most.key == lo ? min(most.index, row.V - 1) : row.V - 1;
    const u128 each = kCount ? 1 : weight62(value_of(lo), s.scale, s.roots);
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

// The index of the n-th logit (from 1) that equals x.
template <typename T, int NT> __device__ __noinline__ int index_of_nth(const RowSpan<T>& row, float x, int n, FilterShared<NT>& s)
{
    int a = 0, b = row.V - 1;
    while (a < b) {
        const int mid = a + (b - a) / 2;
        int here = 0;
        row.each([&](float y, int i) { here += y == x && i <= mid; });
        if (block_sum((u128)(uint32_t)here, s) >= (u128)(uint32_t)n)
            b = mid;
        else
            a = mid + 1;
    }
    return a;
}

// ---------------------------------------------------------------------------
// the result of a row
// ---------------------------------------------------------------------------
struct Settings {
    float T, p, min_p, u;
    int k;
};

// A row's numbers, by one thread.
template <bool DRAW>
__device__ __forceinline__ void put_row(const FilterArgs& a, long long r, int kept, int token = -1, uint64_t weight = 1, u128 mass = 1)
{
    if (a.has_kept)
        a.out_kept[r] = kept;
    if (DRAW) {
        a.out_tokens[r] = token;
        if (a.has_prob)
            a.out_prob[r] = token < 0 ? __int_as_float(0x7fc00000) : quotient(weight, mass);
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

// Returns how many this thread kept.
template <typename T>
__device__ __noinline__ int write_row(const RowSpan<T> row, T* out, bool same_phase, Prefix end)
{
    int n = 0;
    typedef typename Bits<T>::type U;
    constexpr int E = Elem<T>::E;
    const float kv = value_of(end.key);
    U* o = reinterpret_cast<U*>(out);
    const U* x = reinterpret_cast<const U*>(row.p);
    // (a thread's vectors are its own: fetched before any of them is written, where out is the row)
    each_vector<false>(row.vec(), row.v0, row.v1, (int)blockDim.x, [&](const uint4& w, int i, bool there) {
        if (!there)
            return;
        float f[E];
        Elem<T>::unpack(w, f);
        union {
            uint4 v;
            U e[E];
        } y;
        y.v = w;
        const int left = end.index - (row.head + i * E);   // ties up to this one stay
#pragma unroll
        for (int k = 0; k < E; ++k)
            if (f[k] > kv || (f[k] == kv && k <= left))
                ++n;
            else
                y.e[k] = Bits<T>::ninf;
        if (same_phase) {
            __stcs(reinterpret_cast<uint4*>(o + row.head) + i, y.v);
        } else {
#pragma unroll
            for (int k = 0; k < E; ++k)
                o[row.head + i * E + k] = y.e[k];
        }
    });
    const int j = row.lone();
    if (j >= 0) {
        const float f = (float)row.p[j];
        const bool keep = f > kv || (f == kv && j <= end.index);
        o[j] = keep ? x[j] : Bits<T>::ninf;
        n += keep;
    }
    return n;
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
        for (int i = row.v0 + threadIdx.x; i < row.v1; i += (int)blockDim.x)
            __stcs(ov + i, make_uint4(w, w, w, w));
    } else {
        for (int j = row.head + row.v0 * E + threadIdx.x; j < row.head + row.v1 * E; j += (int)blockDim.x)
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
template <typename T, bool DRAW, int NT>
__device__ __noinline__ void whole_row(const FilterArgs& a, long long r, const Settings& g, float m, Prefix end, FilterShared<NT>& s)
{
    const RowSpan<T> row(static_cast<const T*>(a.logits) + r * a.V, a.V, 0, 1);
    const uint32_t top = key_of(m);
    u128 mass = 0;
    if (g.k > 0 && prefix_sum<true>(row, end, s) > (u128)g.k)
        end = prefix_reaching<true>(row, (u128)g.k, end, top, s);
    if (g.p < 1.0f || DRAW)
        mass = prefix_sum<false>(row, end, s);
    if (g.p < 1.0f) {
        const u128 goal = share_of(g.p, mass, true);
        end = prefix_reaching<false>(row, goal > 1 ? goal : 1, end, top, s);
        if (DRAW)
            mass = prefix_sum<false>(row, end, s);
    }
    const int kept = a.has_kept ? (int)prefix_sum<true>(row, end, s) : 0;
    if (DRAW) {
        const Prefix at = prefix_reaching<false>(row, share_of(g.u, mass, false) + 1, end, top, s);
        if (threadIdx.x == 0)
            put_row<DRAW>(a, r, kept, at.index, weight62(value_of(at.key), s.scale, s.roots), mass);
    } else {
        if (threadIdx.x == 0)
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

// Into rank 0's list.
template <int NT> __device__ __noinline__ void append(FilterShared<NT>& s, int C, uint32_t key, int index, int n = 1)
{
    if (C == 1) {
        const int at = atomicAdd(&s.count, n);
        if (at < kList)
            s.list[at] = entry_of(key, index);
    } else {
        int at;
        asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(at) : "r"(map_to_rank(smem_addr(&s.count), 0)), "r"(n) : "memory");
        if (at < kList)
            st_rank64(&s.list[at], 0, entry_of(key, index));
    }
}

// Room in rank 0's list for each lane's n entries, by all lanes of a warp: one
// atomic a warp.  The place of the lane's first.
template <int NT> __device__ __forceinline__ int list_room(FilterShared<NT>& s, int C, int n)
{
    const int lane = threadIdx.x & 31;
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, upto, o);
        if (lane >= o)
            upto += y;
    }
    int at = 0;
    if (lane == 31) {
        if (C == 1)
            at = atomicAdd(&s.count, upto);
        else
            asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(at) : "r"(map_to_rank(smem_addr(&s.count), 0)), "r"(upto) : "memory");
    }
    return __shfl_sync(kFull, at, 31) + upto - n;
}

template <int NT> __device__ __forceinline__ void list_put(FilterShared<NT>& s, int C, int at, uint64_t e)
{
    if (at >= kList)
        return;
    if (C == 1)
        s.list[at] = e;
    else
        st_rank64(&s.list[at], 0, e);
}

// The marked logits of N vectors (bit u E + j: logit j of vector u, which is at
// place(u)) into rank 0's list, by all lanes of a warp.
template <typename T, int N, typename P, int NT>
__device__ __forceinline__ void append_marked(const RowSpan<T>& row, FilterShared<NT>& s, int C, uint32_t marks, const uint4 (&w)[N], P&& place)
{
    constexpr int E = Elem<T>::E;
    if (!__any_sync(kFull, marks))
        return;
    int at = list_room(s, C, __popc(marks));
#pragma unroll
    for (int u = 0; u < N; ++u) {
        float x[E];
        Elem<T>::unpack(w[u], x);
        if (marks >> (u * E) & ((1u << E) - 1))
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (marks >> (u * E + j) & 1)
                    list_put(s, C, at++, entry_of(key_of(x[j]), row.head + place(u) * E + j));
    }
    __syncwarp();
}

// The logits of a CTA's part that mark(vector, its place) marks (E bits), into
// rank 0's list.  kOneKey: all of them are the key `key`.
template <bool kOneKey, typename T, typename M, int NT>
__device__ __forceinline__ void gather(const RowSpan<T>& row, FilterShared<NT>& s, int C, uint32_t key, M&& mark)
{
    constexpr int E = Elem<T>::E;
    const int t = threadIdx.x;
    Vectors<4> next;
    next.load(row.vec(), row.v0 + t, row.v1, NT);
#pragma unroll 1
    for (int i = row.v0 + t; i - t < row.v1; i += 4 * NT) {
        const Vectors<4> now = next;
        next.load(row.vec(), i + 4 * NT, row.v1, NT);
        uint32_t marks = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i + u * NT < row.v1)
                marks |= mark(now.w[u], i + u * NT) << (u * E);
        __syncwarp();
        if (!kOneKey) {
            append_marked(row, s, C, marks, now.w, [&](int u) { return i + u * NT; });
        } else if (__any_sync(kFull, marks)) {
            int at = list_room(s, C, __popc(marks));
            for (; marks; marks &= marks - 1) {
                const int bit = __ffs(marks) - 1;
                list_put(s, C, at++, entry_of(key, row.head + (i + bit / E * NT) * E + bit % E));
            }
            __syncwarp();
        }
    }
}

// f(values, index of the first) for the vectors of the groups that reach `least`:
// the groups are listed, then read by all threads, a vector each.  What f returns
// marks the values that go into rank 0's list.
template <typename T, typename F, int NT>
__device__ __forceinline__ void each_hit(const RowSpan<T>& row, int groups, float least, int C, FilterShared<NT>& s, F&& f)
{
    constexpr int E = Elem<T>::E;
    const int t = threadIdx.x;
    uint16_t* hit = reinterpret_cast<uint16_t*>(s.group[groups]);
    for (int n = 0; n < groups; ++n)
        if (s.group[n][t] >= least) {
            const int at = atomicAdd(&s.hits, 1);
            if (at < kList)
                hit[at] = (uint16_t)(n * NT + t);
        }
    __syncthreads();
    const int n = min(s.hits, kList) * kGroup;
    auto place = [&](int j) {   // the vector of item j, or -1
        if (j >= n)
            return -1;
        const int h = hit[j / kGroup], i = row.v0 + (h / NT * kGroup + j % kGroup) * NT + h % NT;
        return i < row.v1 ? i : -1;
    };
#pragma unroll 1
    for (int j = t; j - t < n; j += 2 * NT) {
        int i[2] = {place(j), place(j + NT)};
        uint4 w[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
            w[u] = i[u] >= 0 ? row.vec()[i[u]] : make_uint4(0, 0, 0, 0);
        uint32_t marks = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (i[u] >= 0) {
                float x[E];
                Elem<T>::unpack(w[u], x);
                marks |= f(x, row.head + i[u] * E) << (u * E);
            }
        __syncwarp();
        append_marked(row, s, C, marks, w, [&](int u) { return u ? i[1] : i[0]; });
    }
}

// Sorts list[0 .. n), the largest first.
template <int NT> __device__ __noinline__ void sort_list(FilterShared<NT>& s, int n)
{
    const int t = threadIdx.x;
    if (n <= NT) {   // each entry counts those before it, by one thread or up to eight
        const int g = n <= NT / 8 ? 8 : n <= NT / 4 ? 4 : n <= NT / 2 ? 2 : 1, i = t / g, each = ((n + g - 1) / g + 1) & ~1;
        const uint64_t e = i < n ? s.list[i] : 0;
        const int j0 = min(n, t % g * each), j1 = min(n, j0 + each);   // (j0 even, or at the end)
        const ulonglong2* pairs = reinterpret_cast<const ulonglong2*>(s.list);
        int r = 0, j = j0 / 2;
#pragma unroll 4
        for (; j < j1 / 2; ++j) {
            const ulonglong2 p = pairs[j];
            r += (p.x > e) + (p.y > e);
        }
        if ((j1 & 1) && j1 > j0)
            r += s.list[j1 - 1] > e;
        for (int o = 1; o < g; o <<= 1)
            r += __shfl_xor_sync(kFull, r, o);
        __syncthreads();
        if (i < n && t % g == 0)
            s.list[r] = e;
    } else {   // bitonic, kEach neighbours a thread: three of four steps need registers and shuffles alone
        constexpr int kEach = NT == kShortThreads ? 8 : kList / NT;
        int size = 2 * NT;
        while (size < n)
            size *= 2;
        const int i0 = t * kEach;
        uint64_t e[kEach];
#pragma unroll
        for (int x = 0; x < kEach; ++x)
            e[x] = i0 + x < n ? s.list[i0 + x] : 0;
        // of a pair: the larger one where the run of k descends and this is its first, or neither
        auto pick = [](uint64_t a, uint64_t b, bool larger) { return (a > b) == larger ? a : b; };
#pragma unroll 1
        for (int k = 2; k <= size; k <<= 1) {
            int j = k >> 1;
#pragma unroll 1
            for (; j >= 32 * kEach; j >>= 1) {
                __syncthreads();
#pragma unroll
                for (int x = 0; x < kEach; ++x)
                    s.list[x * NT + t] = e[x];
                __syncthreads();
#pragma unroll
                for (int x = 0; x < kEach; ++x)
                    e[x] = pick(e[x], s.list[x * NT + (t ^ (j / kEach))], ((i0 & k) == 0) == ((i0 & j) == 0));
            }
#pragma unroll 1
            for (; j >= kEach; j >>= 1)
#pragma unroll
                for (int x = 0; x < kEach; ++x)
                    e[x] = pick(e[x], __shfl_xor_sync(kFull, (unsigned long long)e[x], j / kEach), ((i0 & k) == 0) == ((i0 & j) == 0));
#pragma unroll
            for (int y = kEach / 2; y > 0; y >>= 1)
                if (y <= j)
#pragma unroll
                    for (int x = 0; x < kEach; ++x)
                        if (!(x & y)) {
                            const uint64_t a = e[x], b = e[x | y];
                            const bool swap = (a < b) == (((i0 | x) & k) == 0);
                            e[x] = swap ? b : a;
                            e[x | y] = swap ? a : b;
                        }
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kEach; ++x)
            s.list[i0 + x] = e[x];
    }
    __syncthreads();
}

template <int NT> __device__ __noinline__ uint64_t entry_weight(const FilterShared<NT>& s, int r)
{
    return weight62(value_of(entry_key(s.list[r])), s.scale, s.roots);
}

// Sums over the list are in units of 2^-52: 2048 weights fit 64 bits, and what
// their rounding moves stays below a thousandth of a token of weight 2^-32.
__device__ __forceinline__ uint64_t weight52(uint64_t w62) { return (w62 + 512) >> 10; }

template <int NT>
__device__ __noinline__ uint64_t list_weight(const FilterShared<NT>& s, int r) { return weight52(entry_weight(s, r)); }

// Exclusive prefix sum over the block; `total` gets the whole.
template <int NT> __device__ __noinline__ uint64_t block_scan(uint64_t v, FilterShared<NT>& s, uint64_t& total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    uint64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(kFull, (unsigned long long)x, o);
        if (lane >= o)
            x += y;
    }
    __syncthreads();
    if (lane == 31)
        s.part64[w] = x;
    __syncthreads();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        const uint64_t q = s.part64[i];
        if (i < w)
            before += q;
        all += q;
    }
    total = all;
    return before + x - v;
}

// The mass of the sorted list's ranks lo .. hi - 1, a block's worth at a time;
// `first` is the weight of rank lo + threadIdx.x (0 from hi on).
template <int NT> __device__ __noinline__ uint64_t list_mass(FilterShared<NT>& s, int lo, int hi, uint64_t first)
{
    uint64_t sum = first, total;
    for (int r = lo + NT + (int)threadIdx.x; r < hi; r += NT)
        sum += list_weight(s, r);
    block_scan(sum, s, total);
    return total;
}

// The first rank of lo .. hi - 1 whose cumulative mass, counted from rank lo on,
// reaches goal (hi - 1 if none does); its mass in `mass`.
template <int NT>
__device__ __noinline__ int list_reaching(FilterShared<NT>& s, int lo, int hi, uint64_t first, uint64_t goal, uint64_t& mass)
{
    uint64_t base = 0;
    for (int r0 = lo;; r0 += NT) {
        const int r = r0 + (int)threadIdx.x;
        const uint64_t w = r0 == lo ? first : r < hi ? list_weight(s, r) : 0;
        uint64_t total;
        const uint64_t c = base + block_scan(w, s, total);
        base += total;
        if (base < goal && r0 + NT < hi)
            continue;
        if (r < hi && (base >= goal ? (c < goal || r == lo) && c + w >= goal : r == hi - 1)) {
            s.found = r;
            s.found64 = c + w;
        }
        __syncthreads();
        mass = s.found64;
        return s.found;
    }
}

// ---------------------------------------------------------------------------
// Any number of candidates: bins of weight
// ---------------------------------------------------------------------------
// A bin holds the tokens whose l log2(e) / T rounds to the same 64th; it sums
// 2^f - 1 of the remainders f, in units of 2^-29, and counts.  Bin 0 holds the
// largest logit.  The last bin holds whatever weighs less than 2^-63 too; its
// mass does not count.  Weights are relative to a bin's width above bin 0's centre.
// (Bins for the tokens near the border alone, found from an eighth of the row, the
// rest summed on the way, took 174 us where this took 159, 256 rows of 151936.)
constexpr float kBinStep = 0.015625f;
constexpr float kBinMagic = 196608.0f;   // 1.5 * 2^23 steps: adding it rounds to steps

struct BinScale {
    float ch, cl, least;   // least: logits below it count as it
    float unit;            // the centre of the bin before the first, in octaves
    uint32_t ref;          // the bits of the largest logit's rounded product
};

__device__ __forceinline__ BinScale bin_scale(const RowScale& sc)
{
    BinScale b;
    b.ch = sc.ch;
    b.cl = sc.cl;
    const float at = __fadd_rn(__fmul_rn(sc.m, sc.ch), kBinMagic);
    b.ref = __float_as_uint(at);
    b.unit = (at - kBinMagic) + kBinStep;
    b.least = fmaxf(sc.m - 44.6f * sc.T, -3.4028234e38f);   // 64.3 octaves: no weight
    return b;
}

__device__ __forceinline__ int bin_of(float l, const BinScale& b)
{
    const uint32_t x = b.ref - __float_as_uint(__fadd_rn(__fmul_rn(fmaxf(l, b.least), b.ch), kBinMagic));
    return (int)min(x, (uint32_t)kBins - 1);
}

// (Predicated rather than branched around: most lanes of a warp are out, in every
// warp some are in.)
template <int NT> __device__ __forceinline__ void bin_add(FilterShared<NT>& s, uint32_t i, uint32_t q, bool in)
{
    const uint32_t lo = smem_addr(&s.bin.lo[i]);
    uint32_t old = 0;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t@p atom.shared.add.u32 %0, [%1], %2;\n\t}"
                 : "+r"(old) : "r"(lo), "r"(q), "r"((uint32_t)in) : "memory");
    const uint32_t more = (1u << kCarryBits) + (old + q < old ? 1u : 0u);
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p red.shared.add.u32 [%0], %1;\n\t}"
                 ::"r"(lo + (uint32_t)sizeof(s.bin.lo)), "r"(more), "r"((uint32_t)in) : "memory");
}

// Two tokens of at least b.least, the packed pair L; `in` says which of them count.
template <int NT>
__device__ __forceinline__ void bin_pair(FilterShared<NT>& s, uint64_t L, bool in0, bool in1, const BinScale& b)
{
    const uint64_t magic = f2_pack(kBinMagic, kBinMagic), nt = f2_mul(L, f2_pack(-b.ch, -b.ch));
    const uint64_t e = f2_fma(L, f2_pack(b.cl, b.cl), f2_fma(L, f2_pack(b.ch, b.ch), nt));
    const uint64_t at = f2_sub(magic, nt);
    const uint64_t f = f2_sub(e, f2_add(nt, f2_sub(at, magic)));
    // 2^f - 1, |f| < 2^-7 + 2^-11: ln 2 f + (ln 2 f)^2 / 2 + (ln 2 f)^3 / 6, the next term below
    // 2^-35; adding one and a half steps rounds it to 2^-29
    const uint64_t g = f2_fma(f, f2_fma(f, f2_pack(0.05550411f, 0.05550411f), f2_pack(0.24022651f, 0.24022651f)), f2_pack(0.69314718f, 0.69314718f));
    const uint64_t q = f2_fma(f, g, f2_pack(1.5f * kBinStep, 1.5f * kBinStep));
    const uint32_t unit = 0x3c800000u;   // one step: q's bits less these are (2^f - 1) 2^29 + 2^22
    bin_add(s, min(b.ref - (uint32_t)at, (uint32_t)kBins - 1), (uint32_t)q - unit, in0);
    bin_add(s, min(b.ref - (uint32_t)(at >> 32), (uint32_t)kBins - 1), (uint32_t)(q >> 32) - unit, in1);
}

template <int NT>
__device__ __forceinline__ uint32_t bin_count(const FilterShared<NT>& s, int i) { return s.bin.hi[i] >> kCarryBits; }

// Bin i's share of its thread's bins: the sum of its weights over the weight of
// the thread's first bin's centre, in units of 2^-29.
template <int NT> __device__ __forceinline__ uint64_t bin_part(const FilterShared<NT>& s, int i)
{
    const uint32_t hi = s.bin.hi[i], n = hi >> kCarryBits;
    const uint64_t sum = (((uint64_t)(hi & ((1u << kCarryBits) - 1)) << 32) | s.bin.lo[i]) + ((uint64_t)n << 29) - ((uint64_t)n << 22);
    const uint64_t f = i == kBins - 1 ? 0 : s.steps[i % kBinsEach<NT>];
    return ((sum & 0xffffffffu) * f >> 31) + ((sum >> 32) * f << 1);
}

// The weight that multiplies the parts of thread t's bins.
template <int NT> __device__ __forceinline__ uint64_t part_weight(const FilterShared<NT>& s, int t)
{
    return exp2_neg((uint64_t)(t * kBinsEach<NT> + 1) << (48 - kBinShift), s.roots);
}

__device__ __forceinline__ u128 part_mass(uint64_t part, uint64_t weight) { return ((u128)part * weight) >> 29; }

// A thread's bins (kBinsEach of them), and what is before them; masses in units of 2^-62.
struct BinPart {
    u128 before, own;
    int n_before, n_own;
};

template <int NT> __device__ __noinline__ BinPart scan_bins(FilterShared<NT>& s, u128& mass, int& count)
{
    BinPart q;
    const int t = threadIdx.x;
    if (t < kBinsEach<NT>)
        s.steps[t] = (uint32_t)(exp2_neg((uint64_t)t << (48 - kBinShift), s.roots) >> 31);
    __syncthreads();
    uint64_t part = 0;
    q.n_own = 0;
#pragma unroll 4
    for (int i = 0; i < kBinsEach<NT>; ++i) {
        const int j = t * kBinsEach<NT> + ((i + t) & (kBinsEach<NT> - 1));   // (lanes on different banks)
        part += bin_part(s, j);
        q.n_own += (int)bin_count(s, j);
    }
    q.own = part ? part_mass(part, part_weight(s, t)) : 0;
    // the count in the low bits of one sum with the mass: masses are below 2^83
    u128 total;
    const u128 both = block_scan((q.own << 24) | (u128)(uint32_t)q.n_own, s, total);
    q.before = both >> 24;
    q.n_before = (int)((uint32_t)both & 0xffffffu);
    mass = total >> 24;
    count = (int)((uint32_t)total & 0xffffffu);
    return q;
}

template <int NT> __device__ __forceinline__ u128 bin_mass(const FilterShared<NT>& s, int i)
{
    return part_mass(bin_part(s, i), part_weight(s, i / kBinsEach<NT>));
}

// Where in the bins of thread s.found: one warp, a bin a lane.
template <bool kCount, int NT> __device__ __noinline__ void bin_within(FilterShared<NT>& s, u128 goal)
{
    const int lane = threadIdx.x, i = s.found * kBinsEach<NT> + (lane & (kBinsEach<NT> - 1));
    const uint64_t weight = part_weight(s, s.found), own = lane < kBinsEach<NT> ? bin_part(s, i) : 0;
    const int n_own = lane < kBinsEach<NT> ? (int)bin_count(s, i) : 0;
    uint64_t x = own;
    int n = n_own;
#pragma unroll
    for (int o = 1; o < kBinsEach<NT>; o <<= 1) {
        const uint64_t y = __shfl_up_sync(kFull, (unsigned long long)x, o);
        const int z = __shfl_up_sync(kFull, n, o);
        if (lane >= o) {
            x += y;
            n += z;
        }
    }
    const u128 base = s.found_mass, from = base + part_mass(x - own, weight);
    const bool here = lane < kBinsEach<NT> && (kCount ? (u128)(uint32_t)(s.found_count + n) : base + part_mass(x, weight)) >= goal;
    const int l = max(0, __ffs(__ballot_sync(kFull, here)) - 1);
    BinAt r;
    r.bin = s.found * kBinsEach<NT> + l;
    r.before = ((u128)__shfl_sync(kFull, (unsigned long long)(from >> 64), l) << 64) | __shfl_sync(kFull, (unsigned long long)from, l);
    r.n_before = s.found_count + __shfl_sync(kFull, n - n_own, l);
    if (lane == 0)
        s.bin_at = r;
}

// The bin where the running sum over all bins, of counts or of masses, reaches
// `goal` (which all of them do).
template <bool kCount, int NT> __device__ __noinline__ BinAt bin_reaching(const BinPart& q, FilterShared<NT>& s, u128 goal)
{
    __syncthreads();
    if (threadIdx.x == 0)
        s.found = 0;
    __syncthreads();
    const u128 c = kCount ? (u128)(uint32_t)q.n_before : q.before, v = kCount ? (u128)(uint32_t)q.n_own : q.own;
    if (c < goal && goal <= c + v) {
        s.found = threadIdx.x;
        s.found_count = q.n_before;
        s.found_mass = q.before;
    }
    __syncthreads();
    if (threadIdx.x < 32)
        bin_within<kCount>(s, goal);
    __syncthreads();
    return s.bin_at;
}

// What rank 0 asks for, behind a row_sync.
template <int NT> __device__ __forceinline__ Command command_of(const FilterShared<NT>& s, int C)
{
    if (C == 1)
        return s.cmd;
    const uint4 x = ld_rank128(&s.cmd, 0), y = ld_rank128(reinterpret_cast<const char*>(&s.cmd) + 16, 0);
    return Command{(int)x.x, (int)x.y, (int)x.z, (int)x.w, y.x, (int)y.y, (int)y.z, __uint_as_float(y.w)};
}

// All of the cluster's bins in rank 0's.
template <int NT> __device__ __noinline__ void merge_bins(FilterShared<NT>& s, int rank, int C)
{
    row_sync(C);
    if (C == 1)
        return;
    const int per = kBins / C, i0 = rank * per, t = threadIdx.x;   // (C is a power of two)
    for (int i = i0 + 4 * t; i < i0 + per; i += 4 * NT) {
        uint64_t lo[4] = {0, 0, 0, 0};
        uint32_t hi[4] = {0, 0, 0, 0};
#pragma unroll 2
        for (int c = 0; c < C; ++c) {
            const uint4 x = ld_rank128(&s.bin.lo[i], c), y = ld_rank128(&s.bin.hi[i], c);
            lo[0] += x.x, lo[1] += x.y, lo[2] += x.z, lo[3] += x.w;
            hi[0] += y.x, hi[1] += y.y, hi[2] += y.z, hi[3] += y.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s.bin.lo[i + j] = (uint32_t)lo[j];
            s.bin.hi[i + j] = hi[j] + (uint32_t)(lo[j] >> 32);
        }
    }
    row_sync(C);
    if (rank == 0) {
#pragma unroll 4
        for (int i = per + 4 * t; i < kBins; i += 4 * NT) {
            const int c = i / per;
            *reinterpret_cast<uint4*>(&s.bin.lo[i]) = ld_rank128(&s.bin.lo[i], c);
            *reinterpret_cast<uint4*>(&s.bin.hi[i]) = ld_rank128(&s.bin.hi[i], c);
        }
        __syncthreads();
    }
}

// A CTA's part of the row, as far as it is in the prefix, into its bins.
template <typename T, int NT>
__device__ __noinline__ void fill_bins(const RowSpan<T> row, Prefix end, const BinScale b, FilterShared<NT>& s)
{
    constexpr int E = Elem<T>::E;
    __syncthreads();
    for (int i = 4 * threadIdx.x; i < kBins; i += 4 * NT)
        *reinterpret_cast<uint4*>(&s.bin.lo[i]) = *reinterpret_cast<uint4*>(&s.bin.hi[i]) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    const float least = value_of(end.key);
    each_vector<true>(row.vec(), row.v0, row.v1, NT, [&](const uint4& w, int i, bool there) {
        float x[E];
        Elem<T>::unpack(w, x);
        const int left = there ? end.index - (row.head + i * E) : -1;   // ties up to this one count
        const float above = there ? least : INFINITY;
#pragma unroll
        for (int j = 0; j < E; j += 2)
            bin_pair(s, f2_pack(fmaxf(x[j], b.least), fmaxf(x[j + 1], b.least)), x[j] > above || (x[j] == above && j <= left),
                     x[j + 1] > above || (x[j + 1] == above && j + 1 <= left), b);
    });
    const int lone = row.lone();
    if (lone >= 0) {
        const float x = (float)row.p[lone], y = fmaxf(x, b.least);
        bin_pair(s, f2_pack(y, y), end.has(key_of(x), lone), false, b);
    }
}

// The lowest logit of bin i or one before it: near where the bin's border should
// be, by bisection (bin_of does not increase with the logit).
__device__ __noinline__ float bin_floor(int i, float m, const BinScale& b)
{
    if (i >= kBins - 1)
        return -INFINITY;
    const float at = (b.unit - ((float)i + 1.5f) * kBinStep) / b.ch, wide = 2.0f * kBinStep / b.ch;
    uint32_t lo = key_of(fmaxf(at - wide, -3.4028234e38f)), hi = key_of(fminf(at + wide, m));   // bin_of(lo) > i >= bin_of(hi)
    while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (bin_of(value_of(mid), b) <= i)
            hi = mid;
        else
            lo = mid;
    }
    return value_of(hi);
}

// The tokens of the prefix that are in bins from .. to, or in `also`.
template <typename T, int NT>
__device__ __noinline__ void gather_bins(const RowSpan<T> row, int from, int to, int also, Prefix end, const BinScale b, int C,
                                         FilterShared<NT>& s)
{
    constexpr int E = Elem<T>::E;
    const float m = s.scale.m;
    // [low, top) and [low2, top2), the four borders at once
    float border = 0.0f;
    const int lane = threadIdx.x & 31, of = lane == 0 ? to : lane == 1 ? from - 1 : lane == 2 ? also : also - 1;
    if (lane < 4)
        border = of < 0 ? INFINITY : bin_floor(of, m, b);
    const float low = fmaxf(__shfl_sync(kFull, border, 0), value_of(end.key)), top = __shfl_sync(kFull, border, 1);
    const float low2 = fmaxf(__shfl_sync(kFull, border, 2), value_of(end.key)), top2 = __shfl_sync(kFull, border, 3);
    const float least = value_of(end.key);
    const bool both = also < from || also > to, ties = end.index != INT_MAX;
    auto in = [&](float x, int i) {
        return ((x >= low && x < top) || (both && x >= low2 && x < top2)) && (x > least || (x == least && i <= end.index));
    };
    gather<false>(row, s, C, 0, [&](const uint4& w, int i) {
        float x[E];
        Elem<T>::unpack(w, x);
        uint32_t marks = 0;
#pragma unroll
        for (int j = 0; j < E; ++j)
            marks |= x[j] >= low && x[j] < top ? 1u << j : 0u;
        if (both)
#pragma unroll
            for (int j = 0; j < E; ++j)
                marks |= x[j] >= low2 && x[j] < top2 ? 1u << j : 0u;
        if (ties && marks)
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (!in(x[j], row.head + i * E + j))
                    marks &= ~(1u << j);
        return marks;
    });
    const int lone = row.lone();
    if (lone >= 0 && in((float)row.p[lone], lone))
        append(s, C, key_of((float)row.p[lone]), lone);
}

template <typename T, bool DRAW, int NT>
__device__ __noinline__ void binned_row(const FilterArgs& a, long long r, const Settings& g, const RowSpan<T>& row, int rank, Prefix end,
                                        FilterShared<NT>& s)
{
    const int C = a.C, t = threadIdx.x;
    T* out = static_cast<T*>(a.out) + (DRAW ? 0 : r * a.V);
    int k = g.k;
    const BinScale bs = bin_scale(s.scale);
    for (;;) {
        fill_bins(row, end, bs, s);
        if (t == 0)   // the list's weights as the bins' masses (read behind the next barriers)
            s.scale.top = ((long long)(int)(bs.ref - __float_as_uint(kBinMagic)) + 1) * (1ll << (48 - kBinShift));
        merge_bins(s, rank, C);
        bool again = false;
        int stage = 0;   // rank 0's: what the gathered list is for
        int kept = 0, last = 0, lo_first = 0, n_last = 0;
        u128 above = 0, above_first = 0, total = 0, mass = 0;
        BinPart part{};
        for (;;) {
            if (rank == 0) {
                Command c{kCmdEnd, 0, 0, -1, 0, 0, 0, 0.0f};
                bool give_up = false;
                if (stage == 0) {
                    int n_all;
                    part = scan_bins(s, total, n_all);
                    if (k > 0 && k < n_all) {   // top-k first: its last token
                        const BinAt at = bin_reaching<true>(part, s, (u128)(uint32_t)k);
                        stage = 1;
                        kept = k - at.n_before;
                        c.op = kCmdGather;
                        c.from = c.to = c.also = at.bin;
                        give_up = bin_count(s, at.bin) > kList;
                    } else if (g.p < 1.0f) {
                        stage = 2;
                        const u128 share = share_of(g.p, total, true), goal = share > 1 ? share : 1;
                        const BinAt end_at = bin_reaching<false>(part, s, goal);
                        last = end_at.bin;
                        above = above_first = end_at.before;
                        kept = end_at.n_before;
                        n_last = (int)bin_count(s, last);
                        give_up = n_last > kList;
                        c.op = kCmdGather;
                        c.from = c.to = c.also = last;
                        if (DRAW && kept + n_last <= kFewKept) {   // all of them
                            c.from = 0;
                            above_first = 0;
                        } else if (DRAW) {   // and the bins the draw is in, if the kept mass is the goal or little more
                            const BinAt at = bin_reaching<false>(part, s, share_of(g.u, goal, false) + 1);
                            const int to = min(at.bin + 1, last);
                            if (at.bin < last && (int)bin_count(s, at.bin) + (int)bin_count(s, to) + n_last <= kList) {
                                c.from = at.bin;
                                c.to = to;
                                above_first = at.before;
                            }
                        }
                        lo_first = c.from;
                    } else if (!DRAW) {   // top-k reaches past the last token
                        if (t == 0)
                            put_row<DRAW>(a, r, n_all);
                        c.op = kCmdWrite;
                        c.key = end.key;
                        c.index = end.index;
                    } else {
                        kept = n_all;
                        mass = total;
                        const BinAt at = bin_reaching<false>(part, s, share_of(g.u, total, false) + 1);
                        stage = 4;
                        above_first = at.before;
                        c.op = kCmdGather;
                        c.from = c.to = c.also = at.bin;
                        give_up = bin_count(s, at.bin) > kList;
                    }
                } else {
                    const int n = s.count;
                    sort_list(s, n);
                    if (stage == 1) {
                        const uint64_t e = s.list[kept - 1];
                        c.op = kCmdRecount;
                        c.key = entry_key(e);
                        c.index = entry_index(e);
                    } else {
                        uint64_t w = 0, to;
                        int lo = 0, hi = n;   // where the draw is looked for
                        auto after = [](u128 goal, u128 base) {   // what of a goal is left to the list
                            const u128 d = goal > base ? goal - base : 1;
                            return (uint64_t)((d + 1023) >> 10);
                        };
                        bool draw_now = DRAW, sure = stage == 4;
                        if (stage == 2) {
                            const int from = n - n_last;   // the last bin's tokens
                            w = from + t < n ? list_weight(s, from + t) : 0;
                            const u128 own = (u128)list_mass(s, from, n, w) << 10;
                            // the goal again, with that bin's mass by its tokens
                            const u128 goal = share_of(g.p, total - bin_mass(s, last) + own, true);
                            const int end_r = list_reaching(s, from, n, w, after(goal, above), to);
                            mass = above + ((u128)to << 10);
                            kept += end_r - from + 1;
                            if (!DRAW) {
                                if (t == 0)
                                    put_row<DRAW>(a, r, kept);
                                c.op = kCmdWrite;
                                c.key = entry_key(s.list[end_r]);
                                c.index = entry_index(s.list[end_r]);
                            } else if (share_of(g.u, mass, false) + 1 > above) {   // the draw is in the last bin
                                lo = from;
                                hi = end_r + 1;
                                sure = true;
                                above_first = above;
                            } else {                                               // in a bin before it
                                hi = from;
                                draw_now = lo_first < last;
                            }
                        }
                        int at = 0;
                        if (draw_now) {
                            const uint64_t want = after(share_of(g.u, mass, false) + 1, above_first);
                            w = lo + t < hi ? list_weight(s, lo + t) : 0;
                            at = list_reaching(s, lo, hi, w, want, to);
                            draw_now = to >= want || sure;
                        }
                        if (draw_now) {
                            if (t == 0)
                                put_row<DRAW>(a, r, kept, entry_index(s.list[at]), entry_weight(s, at), mass);
                        } else if (DRAW) {   // not in the bins that are here
                            const BinAt b = bin_reaching<false>(part, s, share_of(g.u, mass, false) + 1);
                            stage = 4;
                            above_first = b.before;
                            c.op = kCmdGather;
                            c.from = c.to = c.also = b.bin;
                            give_up = bin_count(s, b.bin) > kList;
                        }
                    }
                }
                if (give_up) {
                    Settings left = g;
                    left.k = k;
                    c = Command{kCmdEnd, 0, 0, -1, 0, 0, 0, 0.0f};
                    whole_row<T, DRAW>(a, r, left, s.scale.m, end, s);
                }
                __syncthreads();
                if (t == 0) {
                    s.cmd = c;
                    s.count = 0;
                }
            }
            row_sync(C);
            const Command c = command_of(s, C);
            if (c.op == kCmdEnd)
                break;
            if (c.op == kCmdGather) {
                gather_bins(row, c.from, c.to, c.also, end, bs, C, s);
                row_sync(C);
                continue;
            }
            if (c.op == kCmdWrite) {
                write_row(row, out, a.same_phase, Prefix{c.key, c.index});
                break;
            }
            again = true;   // kCmdRecount
            end = Prefix{c.key, c.index};
            break;
        }
        if (!again)
            return;
        row_sync(C);   // the bins and the command have been read
        if (!DRAW && g.p >= 1.0f) {   // top-k was all there was
            if (rank == 0 && t == 0)
                put_row<DRAW>(a, r, k);
            write_row(row, out, a.same_phase, end);
            return;
        }
        k = 0;
    }
}

// ---------------------------------------------------------------------------
// bf16 rows where every token counts: how often each value occurs
// ---------------------------------------------------------------------------
// 8192 values (both signs, 32 octaves of 128) are counted one by one, in the one
// pass over the row; their weights times their counts are the exact sums, and a
// border lies inside one value's tokens.  An atomic a token, where bins of fp32
// logits take two and the arithmetic of the remainders.
__device__ __forceinline__ uint64_t times62(uint64_t f, uint64_t g) { return __umul64hi(f, g) << 2; }

constexpr float kLeastLevel = 5.9604644775390625e-8f;   // 2^-24

struct LevelScale {
    uint64_t first, ratio;   // the weight of the thread's first value up to the maximum, and from one value to the next
    int at;                  // which of its values that first one is
};

// Thread t's values: kLevelsEach of them in descending order, all of one octave.
template <int NT> __device__ __forceinline__ float level_value(int t, int j)
{
    const int o = t * kLevelsEach<NT> + j;
    return o < 4096 ? __uint_as_float((uint32_t)(13183 + 4096 - o) << 16) : __uint_as_float(((uint32_t)(13184 + o - 4096) << 16) | 0x80000000u);
}

template <int NT> __device__ __forceinline__ uint32_t level_count(const FilterShared<NT>& s, int t, int j)
{
    const int o = t * kLevelsEach<NT> + j;
    return s.level[o < 4096 ? 4095 - o : kLevelsSide + o - 4096];
}

template <int NT> __device__ __forceinline__ LevelScale level_scale(const FilterShared<NT>& s, int t)
{
    LevelScale l;
    l.at = max(0, min(s.top_level - t * kLevelsEach<NT>, kLevelsEach<NT> - 1));
    const float value = level_value<NT>(t, l.at), step = level_value<NT>(t, 0) - level_value<NT>(t, 1);
    l.first = value > s.scale.m ? 0 : weight62(value, s.scale, s.roots);   // (all above the maximum: none there)
    l.ratio = step * s.scale.ch > 63.0f ? 0 : exp2_neg((uint64_t)scaled48(step, s.scale.ch, s.scale.cl), s.roots);
    return l;
}

// f^n, n < 32, in units of 2^-62.
__device__ __forceinline__ uint64_t power62(uint64_t f, int n)
{
    uint64_t y = kOne62;
#pragma unroll
    for (int b = 0; b < 5; ++b) {
        if (n >> b & 1)
            y = times62(y, f);
        f = times62(f, f);
    }
    return y;
}

// Parts are in units of 2^-42 of a thread's first weight: those of 2^20 tokens fit 64
// bits, and what the rounding of 2^17 tokens moves is 2^-25 of the largest one's weight.
__device__ __forceinline__ uint64_t part42(uint64_t f) { return (f + (1u << 19)) >> 20; }

__device__ __forceinline__ u128 level_mass(uint64_t part, uint64_t first) { return ((u128)part * first) >> 42; }

struct LevelPart : BinPart {
    LevelScale scale;
};

template <int NT> __device__ __noinline__ LevelPart scan_levels(FilterShared<NT>& s, u128& mass, int& count)
{
    LevelPart q;
    const int t = threadIdx.x, lane = t & 31;
    q.scale = level_scale(s, t);
    uint64_t part = 0, f = power62(q.scale.ratio, max(0, (lane & (kLevelsEach<NT> - 1)) - q.scale.at));
    q.n_own = 0;
#pragma unroll 4
    for (int j = 0; j < kLevelsEach<NT>; ++j) {   // (each lane from another value on: other banks)
        const int i = (j + lane) & (kLevelsEach<NT> - 1);
        const uint32_t n = level_count(s, t, i);
        q.n_own += (int)n;
        part += n * part42(f);   // (nothing above the maximum: n is 0 before `at`)
        f = i == kLevelsEach<NT> - 1 || i < q.scale.at ? kOne62 : times62(f, q.scale.ratio);
    }
    q.own = level_mass(part, q.scale.first);
    u128 total;
    const u128 both = block_scan((q.own << 24) | (u128)(uint32_t)q.n_own, s, total);
    q.before = both >> 24;
    q.n_before = (int)((uint32_t)both & 0xffffffu);
    mass = total >> 24;
    count = (int)((uint32_t)total & 0xffffffu);
    return q;
}

// Where in the values of thread s.found: one warp, a value a lane.
template <bool kCount, int NT> __device__ __noinline__ void level_within(FilterShared<NT>& s, u128 goal)
{
    const int lane = threadIdx.x;
    const LevelScale l{s.found64, s.found_ratio, s.found_at};
    const uint64_t f = power62(l.ratio, max(0, lane - l.at));
    const int n_own = lane < kLevelsEach<NT> ? (int)level_count(s, s.found, lane) : 0;
    uint64_t x = n_own * part42(f);
    const uint64_t own = x;
    int n = n_own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(kFull, (unsigned long long)x, o);
        const int z = __shfl_up_sync(kFull, n, o);
        if (lane >= o) {
            x += y;
            n += z;
        }
    }
    const u128 from = s.found_mass + level_mass(x - own, l.first);
    const bool here = (kCount ? (u128)(uint32_t)(s.found_count + n) : s.found_mass + level_mass(x, l.first)) >= goal;
    // (the sums above went through other roundings of the powers: a goal may lie between)
    const uint32_t at = __ballot_sync(kFull, here), some = __ballot_sync(kFull, n_own > 0);
    const int i = at ? __ffs(at) - 1 : 31 - __clz(some | 1u);
    LevelAt r;
    r.value = level_value<NT>(s.found, i);
    r.weight = weight62(r.value, s.scale, s.roots);
    r.n = __shfl_sync(kFull, n_own, i);
    r.n_before = s.found_count + __shfl_sync(kFull, n - n_own, i);
    r.before = ((u128)__shfl_sync(kFull, (unsigned long long)(from >> 64), i) << 64) | __shfl_sync(kFull, (unsigned long long)from, i);
    const u128 to = s.found_mass + level_mass(x, l.first) - from;
    r.mass = ((u128)__shfl_sync(kFull, (unsigned long long)(to >> 64), i) << 64) | __shfl_sync(kFull, (unsigned long long)to, i);
    if (lane == 0)
        s.level_at = r;
}

// The value among whose tokens the running count, or mass, reaches goal (which
// the row does).
template <bool kCount, int NT> __device__ __noinline__ LevelAt level_reaching(const LevelPart& q, FilterShared<NT>& s, u128 goal)
{
    __syncthreads();
    if (threadIdx.x == 0)
        s.found = 0;
    __syncthreads();
    const u128 c = kCount ? (u128)(uint32_t)q.n_before : q.before, v = kCount ? (u128)(uint32_t)q.n_own : q.own;
    if (c < goal && goal <= c + v) {
        s.found = threadIdx.x;
        s.found_count = q.n_before;
        s.found_mass = q.before;
        s.found64 = q.scale.first;
        s.found_ratio = q.scale.ratio;
        s.found_at = q.scale.at;
    }
    __syncthreads();
    if (threadIdx.x < 32)
        level_within<kCount>(s, goal);
    __syncthreads();
    return s.level_at;
}

// How many tokens of weight w (at least one, at most n) reach a mass.
__device__ __forceinline__ int tokens_for(u128 mass, uint64_t w, int n)
{
    if (w == 0 || mass >= (u128)w * (uint32_t)n)
        return n;
    const uint64_t over = (uint64_t)(mass >> 64);
    const int down = over ? 64 - __clzll(over) : 0;
    int j = max(1, (int)__fdividef((float)(uint64_t)(mass >> down), (float)(w >> down)));   // within 2^-20 of itself
    j = min(j, n);
    while ((u128)w * (uint32_t)j < mass)
        ++j;
    while (j > 1 && (u128)w * (uint32_t)(j - 1) >= mass)
        --j;
    return j;
}

// Counts this CTA's part; returns the largest logit (NaN if there is one).
template <int NT> __device__ __noinline__ float count_levels(const RowSpan<__nv_bfloat16> row, FilterShared<NT>& s)
{
    uint32_t top = 0xff80ff80u;
    auto one = [&](uint32_t w, bool both) {
        uint32_t m = w & 0x7fff7fffu;
        asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(0x33803380u));
        asm("min.u16x2 %0, %0, %1;" : "+r"(m) : "r"(0x43804380u));
        const uint32_t i = m - 0x33803380u + ((w >> 15) & 0x00010001u) * (uint32_t)kLevelsSide;
        atomicAdd(&s.level[i & 0xffffu], 1u);
        if (both)
            atomicAdd(&s.level[i >> 16], 1u);
        top = bmax2_nan(top, both ? w : w | 0xff800000u);
    };
    each_vector<false>(row.vec(), row.v0, row.v1, NT, [&](const uint4& w, int, bool there) {
        if (there) {
            one(w.x, true);
            one(w.y, true);
            one(w.z, true);
            one(w.w, true);
        }
    });
    const int lone = row.lone();
    if (lone >= 0)
        one(reinterpret_cast<const unsigned short*>(row.p)[lone], false);
    return max_nan(__uint_as_float(top << 16), __uint_as_float(top & 0xffff0000u));
}

// The tokens of one value into rank 0's list.
template <int NT>
__device__ __noinline__ void gather_level(const RowSpan<__nv_bfloat16> row, float value, int C, FilterShared<NT>& s)
{
    const uint32_t both = (__float_as_uint(value) >> 16) * 0x10001u;
    gather<true>(row, s, C, key_of(value), [&](const uint4& w, int) {   // (no value here is a zero: equal logits are equal bits)
        const uint32_t m = __vcmpeq2(w.x, both) & 0x00020001u, n = __vcmpeq2(w.y, both) & 0x00080004u;
        const uint32_t o = __vcmpeq2(w.z, both) & 0x00200010u, p = __vcmpeq2(w.w, both) & 0x00800040u;
        const uint32_t all = m | n | o | p;
        return (all | all >> 16) & 0xffu;
    });
    const int lone = row.lone();
    if (lone >= 0 && (float)row.p[lone] == value)
        append(s, C, key_of(value), lone);
}

// Logits nearer to zero than 2^-24 are counted with that value, and none of them is
// told from the others.  That changes a weight by up to ch 2^-24 of itself: all of
// them may move the row's mass by 2^-34 of it.  (One row in 130 of 128256 normal
// logits of deviation 2 has such a logit; at T = 0.8 it moves the mass by 2^-44.)
template <int NT> __device__ __noinline__ bool near_zero_close(const FilterShared<NT>& s, u128 total)
{
    const float near = (float)(s.level[0] + s.level[kLevelsSide]) * (float)weight62(kLeastLevel, s.scale, s.roots);
    return near * s.scale.ch <= (float)(uint64_t)(total >> 20) * 1024.0f;   // 2^(24 - 34 + 20)
}

// False: some logits are not among the values (or not finite): to be done
// another way.  Waits for the cluster's CTAs to have started (peers_started).
template <bool DRAW, int NT>
__device__ __noinline__ bool levels_row(const FilterArgs& a, long long r, const Settings& g, const RowSpan<__nv_bfloat16>& row, int rank,
                                        FilterShared<NT>& s)
{
    typedef __nv_bfloat16 T;
    const int C = a.C, t = threadIdx.x;
    __syncthreads();
    for (int i = t; i < kLevels; i += NT)
        s.level[i] = 0;
    __syncthreads();
    const uint32_t key = __reduce_max_sync(kFull, key_of(count_levels(row, s)));
    if ((t & 31) == 0)
        s.warp_top[t >> 5] = key;
    __syncthreads();
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i)
        top = max(top, s.warp_top[i]);
    if (C > 1) {
        peers_started(C);
        if (t < C)
            st_rank(&s.peer_top[rank], t, top);
        row_sync(C);
        for (int c = 0; c < C; ++c)
            top = max(top, s.peer_top[c]);
        const int per = (kLevels + C - 1) / C, i0 = rank * per, i1 = min(kLevels, i0 + per);
        for (int i = i0 + t; i < i1; i += NT) {
            uint32_t n = 0;
#pragma unroll 4
            for (int c = 0; c < C; ++c)
                n += ld_rank(&s.level[i], c);
            s.level[i] = n;
        }
        row_sync(C);
        if (rank == 0) {
#pragma unroll 4
            for (int i = per + t; i < kLevels; i += NT)
                s.level[i] = ld_rank(&s.level[i], i / per);
            __syncthreads();
        }
    }
    // rank 0's: `stage` says what its list is for
    int stage = 0, kept = 0, nth = 0;
    LevelAt at{};
    u128 mass = 0;
    for (;;) {
        if (rank == 0) {
            Command c{kCmdEnd, 0, 0, -1, 0, 0, 0, 0.0f};
            int index = -1;   // of the nth token of at.value, where it is known
            if (stage == 0) {
                const float m = value_of(top);
                const uint32_t low = s.level[2 * kLevelsSide - 1];
                const bool fit = top > kKeyNegInf && top < kKeyPosInf && m < 256.0f && m > -256.0f && fabsf(m) >= kLeastLevel;
                if (t == 0 && fit) {
                    const int bits = (int)(__float_as_uint(m) >> 16);
                    s.top_level = bits >> 15 ? 4096 + (bits & 0x7fff) - 13184 : 13183 + 4096 - bits;
                    s.scale = row_scale(m, g.T);
                }
                __syncthreads();
                // Logits below -256 have to weigh nothing, and their number is not known.
                const bool able = fit && !s.scale.cold && (low == 0 || ((m + 256.0f) * s.scale.ch > 64.0f && g.k == 0 && g.p < 1.0f)) &&
                                  s.scale.ch < 256.0f;
                if (!able) {
                    c.op = kCmdRecount;
                } else {
                    int n_all;
                    u128 total;
                    const LevelPart part = scan_levels(s, total, n_all);
                    const bool close = s.level[0] + s.level[kLevelsSide] == 0 || near_zero_close(s, total);
                    bool cut = false;   // whether the prefix ends inside the row
                    kept = n_all;
                    mass = total;
                    if (g.k > 0 && g.k < n_all) {
                        at = level_reaching<true>(part, s, (u128)(uint32_t)g.k);
                        kept = g.k;
                        nth = g.k - at.n_before;
                        mass = at.before + (u128)at.weight * (uint32_t)nth;
                        cut = true;
                    }
                    if (g.p < 1.0f) {
                        u128 goal = share_of(g.p, mass, true);
                        goal = goal > 1 ? goal : 1;
                        const bool in_last = cut && goal > at.before;   // among the tokens that top-k cut
                        int most = nth;
                        if (!in_last) {
                            const u128 all = mass;
                            at = level_reaching<false>(part, s, goal);
                            most = at.n;
                            // the goal again, that value's mass by its tokens
                            const u128 own = (u128)at.weight * (uint32_t)at.n;
                            goal = share_of(g.p, all - at.mass + own, true);
                            goal = goal > 1 ? goal : 1;
                        }
                        nth = tokens_for(goal > at.before ? goal - at.before : 1, at.weight, most);
                        kept = at.n_before + nth;
                        mass = at.before + (u128)at.weight * (uint32_t)nth;
                        cut = true;
                    }
                    if (DRAW) {
                        const u128 point = share_of(g.u, mass, false) + 1;
                        if (!cut || point <= at.before) {
                            at = level_reaching<false>(part, s, point);
                            nth = at.n;
                        }
                        nth = tokens_for(point > at.before ? point - at.before : 1, at.weight, nth);
                    }
                    if (!close || fabsf(at.value) == kLeastLevel) {
                        c.op = kCmdRecount;
                    } else if (!DRAW && (!cut || nth == at.n)) {   // whole values
                        stage = 2;
                        index = INT_MAX;
                        if (!cut)
                            at.value = -3.4028234663852886e38f;
                    } else if (at.n <= kList) {
                        stage = 1;
                        c.op = kCmdGather;
                        c.value = at.value;
                    } else {
                        stage = 2;
                        index = index_of_nth(RowSpan<T>(row.p, row.V, 0, 1), at.value, nth, s);
                    }
                }
            } else {
                sort_list(s, s.count);
                index = entry_index(s.list[nth - 1]);
                stage = 2;
            }
            if (stage == 2) {
                if (t == 0)
                    put_row<DRAW>(a, r, kept, index, at.weight, mass);
                if (!DRAW) {
                    c.op = kCmdWrite;
                    c.key = key_of(at.value);
                    c.index = index;
                }
            }
            __syncthreads();
            if (t == 0) {
                s.cmd = c;
                s.count = 0;
            }
        }
        row_sync(C);
        const Command c = command_of(s, C);
        if (c.op == kCmdGather) {
            gather_level(row, c.value, C, s);
            row_sync(C);
            continue;
        }
        if (c.op == kCmdWrite)
            write_row(row, static_cast<T*>(a.out) + r * a.V, a.same_phase, Prefix{c.key, c.index});
        row_sync(C);   // the command has been read
        return c.op != kCmdRecount;
    }
}

// A row that no filter touches, in the one pass that has to read it anyway; if it
// turns out unusable, NaN over it.  Waits as levels_row does.
template <typename T, int NT>
__device__ __noinline__ void copy_row(const FilterArgs& a, long long r, const RowSpan<T> row, int rank, FilterShared<NT>& s)
{
    typedef typename Bits<T>::type U;
    constexpr int E = Elem<T>::E;
    const int C = a.C, t = threadIdx.x;
    T* out = static_cast<T*>(a.out) + r * a.V;
    U* o = reinterpret_cast<U*>(out);
    float top = -INFINITY;
    int n = 0;
    each_vector<false>(row.vec(), row.v0, row.v1, NT, [&](const uint4& w, int i, bool there) {
        if (!there)
            return;
        float x[E];
        Elem<T>::unpack(w, x);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            top = max_nan(top, x[j]);
            n += x[j] > -INFINITY;
        }
        if (a.same_phase) {
            __stcs(reinterpret_cast<uint4*>(o + row.head) + i, w);
        } else {
            union {
                uint4 v;
                U e[E];
            } y;
            y.v = w;
#pragma unroll
            for (int j = 0; j < E; ++j)
                o[row.head + i * E + j] = y.e[j];
        }
    });
    const int lone = row.lone();
    if (lone >= 0) {
        const float x = (float)row.p[lone];
        top = max_nan(top, x);
        n += x > -INFINITY;
        o[lone] = reinterpret_cast<const U*>(row.p)[lone];
    }
    const uint32_t key = __reduce_max_sync(kFull, key_of(top));
    if ((t & 31) == 0)
        s.warp_top[t >> 5] = key;
    const int own = (int)block_sum((u128)(uint32_t)n, s);   // (a barrier behind warp_top)
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i)
        most = max(most, s.warp_top[i]);
    int all = own;
    if (C > 1) {
        peers_started(C);
        if (t < C) {
            st_rank(&s.peer_top[rank], t, most);
            st_rank(&s.peer_kept[rank], t, (uint32_t)own);
        }
        row_sync(C);
        all = 0;
        for (int c = 0; c < C; ++c) {
            most = max(most, s.peer_top[c]);
            all += s.peer_kept[c];
        }
    }
    const bool usable = most > kKeyNegInf && most < kKeyPosInf;
    if (rank == 0 && t == 0)
        put_row<false>(a, r, usable ? all : -1);
    if (!usable)
        fill_row(row, out, a.same_phase, Bits<T>::nan);
}

// Rows whose candidates, the tokens up to `end`, no list holds.
template <typename T, bool DRAW, int NT>
__device__ __forceinline__ void many_candidates(const FilterArgs& a, long long r, const Settings& g, const RowSpan<T>& row, int rank, Prefix end,
                                                FilterShared<NT>& s)
{
    const int C = a.C, t = threadIdx.x;
    T* out = static_cast<T*>(a.out) + (DRAW ? 0 : r * a.V);
    // Nothing but min-p, if that: every token above its border stays.
    if (!DRAW && g.p >= 1.0f && g.k == 0) {
        const int all = (int)block_sum((u128)(uint32_t)write_row(row, out, a.same_phase, end), s);
        if (C > 1) {
            if (t == 0)
                st_rank(&s.peer_kept[rank], 0, (uint32_t)all);
            row_sync(C);
        }
        int total = all;
        for (int c = 1; c < C; ++c)
            total += s.peer_kept[c];
        if (rank == 0 && t == 0)
            put_row<DRAW>(a, r, total);
        return;
    }

    if (s.scale.cold) {
        if (rank == 0)
            whole_row<T, DRAW>(a, r, g, s.scale.m, end, s);
        return;
    }
    binned_row<T, DRAW>(a, r, g, row, rank, end, s);
    row_sync(C);
}

// ---------------------------------------------------------------------------
// the kernel: a row a cluster
// ---------------------------------------------------------------------------
template <typename T, bool DRAW, int NT>
__global__ void __launch_bounds__(NT, NT == kShortThreads ? kShortBlocks : kBlocksOf<T>) sv_filter_kernel(FilterArgs a)
{
    extern __shared__ __align__(16) unsigned char filter_smem[];
    FilterShared<NT>& s = *reinterpret_cast<FilterShared<NT>*>(filter_smem);
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
    if (g.k >= V)
        g.k = 0;   // (all of the row)
    g.p = a.has_p ? a.top_p[b] : 1.0f;
    g.min_p = a.has_m ? a.min_p[b] : 0.0f;
    g.u = DRAW && g.T != 0.0f ? a.uniforms[r] : 0.0f;
    const bool greedy = g.T == 0.0f;
    const bool good = temperature_usable(g.T) && (greedy || (g.k >= 0 && g.p >= 0.0f && g.p <= 1.0f && g.min_p >= 0.0f && g.min_p <= 1.0f &&
                                                             g.u >= 0.0f && g.u < 1.0f));
    const T* logits = static_cast<const T*>(a.logits) + r * V;
    T* out = static_cast<T*>(a.out) + (DRAW ? 0 : r * V);
    const RowSpan<T> row(logits, V, rank, C);

    if (t < 64)
        s.roots[t] = root_power(t);
    if (t == 0) {
        s.count = 0;
        s.hits = 0;
        s.first = INT_MAX;
    }
    peers_announce(C);
    bool started = false;
    const int groups = (row.v1 - row.v0 + kGroup * NT - 1) / (kGroup * NT);
    // How a top-k is bounded: by the threads' maxima, or with a larger share of them
    // by the groups'; not where too many would pass.
    const int share = (g.k + C - 1) / C;
    const bool by_thread = share <= NT / 2;
    const bool bounded = !greedy && g.k > 0 && (by_thread || (share <= groups * (NT / 2) && g.k <= kList / 2));
    // bf16 rows where every token counts, or nearly: 1024 rows of 128256 with top-k 250
    // take 101 us by the bound and 132 by levels, with top-k 500 125 and 133, with 700
    // 139 and 133, with 1000 164 and 133.  (Between 256 and 600 the bound would be the
    // faster one for these; where the row is spread over CTAs k is shared among them.)
    if constexpr (sizeof(T) == 2 && NT != kShortThreads)
        if (good && !greedy && g.min_p == 0.0f && V > kList && (g.k == 0 ? DRAW || g.p < 1.0f : share > NT || !bounded)) {
            if (levels_row<DRAW>(a, r, g, row, rank, s))
                return;
            started = true;   // (it has waited)
        }

    if (!DRAW && good && !greedy && g.min_p == 0.0f && g.p >= 1.0f && g.k == 0) {
        copy_row<T>(a, r, row, rank, s);
        return;
    }

    double t_log = 0.0;   // one thread's: 64-bit floating point runs at a hundredth of the fp32 rate
    if (t == NT - 32 && good && !greedy && g.min_p > 0.0f)
        t_log = (double)g.T * log((double)g.min_p);

    // 1. The maxima of the row, of each thread, and of each thread's groups of
    // vectors: the one pass that has to read everything from memory.
    float mine = -INFINITY;
    for (int n = 0; n < groups; ++n) {
        const int i0 = row.v0 + n * kGroup * NT + t;
        uint4 w[kGroup];
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            const uint32_t none = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
            w[u] = make_uint4(none, none, none, none);
            if (i0 + u * NT < row.v1)
                w[u] = ld_row(row.vec() + i0 + u * NT);
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
    const uint32_t own_key = key_of(mine);
    {
        const uint32_t top = __reduce_max_sync(kFull, own_key), low = __reduce_min_sync(kFull, own_key);
        if ((t & 31) == 0) {
            s.warp_top[t >> 5] = top;
            s.warp_low[t >> 5] = low;
        }
    }
    __syncthreads();
    uint32_t top_key = 0, low_key = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        top_key = max(top_key, s.warp_top[i]);
        low_key = min(low_key, s.warp_low[i]);
    }

    // 2. With top-k, a logit that at least k of the row reach: in each of C CTAs
    // the k / C-th (or a few after it) of the threads' or the groups' maxima, and
    // the lowest of these.  (A k of which the row has no finite logits leaves them all.)
    uint32_t bound = 0;
    if (bounded && top_key < kKeyPosInf) {   // (a NaN or +inf: no token will come of it)
        uint32_t lo = by_thread ? low_key : 0, hi = top_key;
        for (int turn = 0; lo < hi; turn ^= 1) {
            const uint32_t mid = lo + (hi - lo) / 2 + 1;
            int n = own_key >= mid;
            if (!by_thread) {
                const float pivot = value_of(mid);
                n = 0;
                for (int i = 0; i < groups; ++i)
                    n += s.group[i][t] >= pivot;
            }
            n = __reduce_add_sync(kFull, n);
            if ((t & 31) == 0)
                s.warp_count[turn][t >> 5] = n;
            __syncthreads();
            n = 0;
#pragma unroll
            for (int i = 0; i < NT / 32; ++i)
                n += s.warp_count[turn][i];
            if (n >= share) {
                lo = mid;
                if (n <= share + share / 4 + (C > 1 ? 1 : 8))
                    break;
            } else {
                hi = mid - 1;
            }
        }
        bound = lo;
    }
    if (C > 1) {
        if (!started)
            peers_started(C);
        if (t < C) {
            st_rank(&s.peer_top[rank], t, top_key);
            st_rank(&s.peer_bound[rank], t, bound);
        }
        row_sync(C);
        for (int c = 0; c < C; ++c) {
            top_key = max(top_key, s.peer_top[c]);
            bound = min(bound, s.peer_bound[c]);
        }
    }

    if (!good || top_key <= kKeyNegInf || top_key >= kKeyPosInf) {
        if (rank == 0 && t == 0)
            put_row<DRAW>(a, r, -1);
        if (!DRAW)
            fill_row(row, out, a.same_phase, Bits<T>::nan);
        return;
    }
    const float m = value_of(top_key);
    if (greedy) {
        each_hit(row, groups, m, C, s, [&](const float (&x)[E], int i) {
#pragma unroll
            for (int k = E - 1; k >= 0; --k)
                if (x[k] == m)
                    atomicMin(&s.first, i + k);
            return 0u;
        });
        // (more hits than the list of them holds: by all threads' groups)
        if (s.hits > kList)
            row.each([&](float x, int i) {
                if (x == m)
                    atomicMin(&s.first, i);
            });
        if (lone >= 0 && lone_x == m)
            atomicMin(&s.first, lone);
        row_sync(C);
        int first = s.first;
        for (int c = 0; c < C; ++c)
            if (c != rank)
                first = min(first, (int)ld_rank(&s.first, c));
        if (rank == 0 && t == 0)
            put_row<DRAW>(a, r, 1, first);
        if (!DRAW)
            fill_row(row, out, a.same_phase, Bits<T>::ninf);
        row_sync(C);
        if (!DRAW && rank == 0 && t == 0)
            out[first] = (T)m;
        return;
    }

    Prefix end{kKeyNegInf + 1, INT_MAX};
    if (t == 0)
        s.scale = row_scale(m, g.T);
    if (t == NT - 32 && g.min_p > 0.0f)
        s.least_key = min_p_key(m, t_log);
    __syncthreads();
    if (g.min_p > 0.0f)
        end.key = max(end.key, s.least_key);

    // 3. Few candidates (a top-k bound, min-p, or a short row): they are read
    // again, by the groups that hold one, sorted and weighed.
    if (bounded || g.min_p > 0.0f || V <= kList) {
        const uint32_t cut = max(end.key, bound);
        const float cv = value_of(cut);
        each_hit(row, groups, cv, C, s, [&](const float (&x)[E], int) {
            uint32_t marks = 0;
#pragma unroll
            for (int k = 0; k < E; ++k)
                marks |= x[k] >= cv ? 1u << k : 0u;
            return marks;
        });
        if (lone >= 0 && lone_x >= cv)
            append(s, C, key_of(lone_x), lone);
        if (t == 0 && s.hits > kList)   // (each holds a candidate)
            append(s, C, 0, 0, kList + 1);
        row_sync(C);
        int n = C > 1 && rank != 0 ? (int)ld_rank(&s.count, 0) : s.count;
        if (n <= kList) {
            if (!DRAW)
                fill_row(row, out, a.same_phase, Bits<T>::ninf);
            if (C > 1) {   // the count has been read, and this part of out is -inf
                __syncwarp();
                if (DRAW)
                    cluster_arrive_relaxed();
                else
                    cluster_arrive();
                if (rank != 0) {
                    cluster_wait();
                    return;
                }
            }
            sort_list(s, n);
            if (g.k > 0)
                n = min(n, g.k);
            uint64_t mass = 0, w = 0;
            if (n <= NT) {   // a rank a thread: one sum answers both questions
                if (DRAW || g.p < 1.0f) {
                    const uint64_t w62 = t < n ? entry_weight(s, t) : 0;
                    w = weight52(w62);
                    const uint64_t c = block_scan(w, s, mass);
                    if (g.p < 1.0f) {
                        const uint64_t share = share_of(g.p, mass, true), goal = share > 1 ? share : 1;
                        if (c < goal && c + w >= goal) {
                            s.found = t;
                            s.found64 = c + w;
                        }
                        __syncthreads();
                        n = s.found + 1;
                        mass = s.found64;
                    }
                    if (DRAW) {
                        const uint64_t goal = share_of(g.u, mass, false) + 1;
                        if (c < goal && c + w >= goal)
                            put_row<DRAW>(a, r, n, entry_index(s.list[t]), w62, (u128)mass << 10);
                    }
                }
                if (!DRAW && t == 0)
                    put_row<DRAW>(a, r, n);
            } else {
                if (DRAW || g.p < 1.0f) {
                    w = list_weight(s, t);
                    mass = list_mass(s, 0, n, w);
                }
                if (g.p < 1.0f) {
                    const uint64_t goal = share_of(g.p, mass, true);
                    n = list_reaching(s, 0, n, w, goal > 1 ? goal : 1, mass) + 1;
                    w = t < n ? w : 0;
                }
                uint64_t to;
                const int at = DRAW ? list_reaching(s, 0, n, w, share_of(g.u, mass, false) + 1, to) : 0;
                if (t == 0)
                    put_row<DRAW>(a, r, n, entry_index(s.list[at]), entry_weight(s, at), (u128)mass << 10);
            }
            __syncwarp();
            if (C > 1)
                cluster_wait();
            else
                __syncthreads();
            if (!DRAW)
                for (int i = t; i < n; i += NT)
                    out[entry_index(s.list[i])] = (T)value_of(entry_key(s.list[i]));
            return;
        }
        if constexpr (NT == kShortThreads)   // (V <= kShortMost: they have been listed)
            return;
        row_sync(C);   // too many (every CTA has read the count): the bins take them
        if (t == 0)
            s.count = 0;
    }
    if constexpr (NT != kShortThreads)
        many_candidates<T, DRAW>(a, r, g, row, rank, end, s);
}

}  // namespace sv
