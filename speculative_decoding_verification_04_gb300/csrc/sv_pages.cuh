// sv_pages.cuh -- the pages of the paged cache: from a stack of free ones into
// the sequences' page tables, the slots of new tokens, and back.
//
// Which pages a sequence gets follows from a prefix sum over the sequences'
// requests alone, so every block computes that sum itself (12 bytes a
// sequence, from L2) and then writes its share of pages and slots; no block
// waits for another's results.  What may be updated in place (the held counts
// and the stack's height) is written once every block has read it: behind a
// cluster barrier while one cluster is enough for the call, by a second kernel
// otherwise.
#pragma once

#include "sv_common.cuh"

namespace sv {

constexpr int kPageThreads = 1024;         // and sequences worked on at a time
constexpr uint32_t kErrPages = 8u;         // bit 3: the stack holds too few pages

struct PoolArgs {
    int32_t* table;            // [B][max_pages]
    const int32_t* kv_len;
    const int32_t* n_new;
    const int32_t* row_start;
    const int32_t* held;
    int32_t* stack;            // [capacity]
    const int32_t* free_count;
    int32_t* held_out;
    int32_t* free_out;
    long long* slots;
    uint32_t* err;
    int B, S, rows, max_pages, page_shift, capacity;
    int has_n, packed, has_slots, has_err;
    int slots16;               // slots is 16-byte aligned
    int each;                  // slots a thread writes at a time: 1 or 4
    int update;                // write held_out and free_out
    int work;                  // write pages and slots
    int clustered;             // the grid is one cluster
};

struct PageShared {
    long long before[kPageThreads + 1];   // pages asked for by the chunk's earlier sequences
    int len[kPageThreads], held[kPageThreads], count[kPageThreads];   // count: new tokens, -1: none granted
    int first[kPageThreads + 1];          // packed rows
    long long part[kPageThreads / 32];
};

// Exclusive prefix sum over the block; `total` gets the whole.
__device__ __forceinline__ long long block_scan(long long v, PageShared& s, long long& total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(kFull, x, o);
        if (lane >= o)
            x += y;
    }
    __syncthreads();   // an earlier sum's parts have been read
    if (lane == 31)
        s.part[w] = x;
    __syncthreads();
    if (w == 0) {
        long long p = lane < kPageThreads / 32 ? s.part[lane] : 0;
#pragma unroll
        for (int o = 1; o < kPageThreads / 32; o <<= 1) {
            const long long y = __shfl_up_sync(kFull, p, o);
            if (lane >= o)
                p += y;
        }
        if (lane < kPageThreads / 32)
            s.part[lane] = p;
    }
    __syncthreads();
    total = s.part[kPageThreads / 32 - 1];
    return x - v + (w ? s.part[w - 1] : 0);
}

// The last i in [0, n) with v[i] <= x; v[0] <= x.
template <typename V> __device__ __forceinline__ int last_at_most(const V* v, int n, V x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// f(r) for every n-th row of [from, to), from the me-th on.  Rows are counted in 64
// bits: up to 2^31 - 1 of them and a step of up to 152 blocks pass 32.
template <typename F> __host__ __device__ __forceinline__ void every(long long from, long long to, unsigned me, unsigned n, F&& f)
{
    for (long long r = from + me; r < to; r += n)
        f(r);
}

__device__ __forceinline__ int pages_for(long long positions, int shift)
{
    return (int)((positions + (1 << shift) - 1) >> shift);
}

// How many packed rows lie between two starts; -1 where they do not ascend from 0 or
// more (starts may be any numbers: what their difference wraps to says nothing).
__host__ __device__ __forceinline__ int packed_count(int start, int next)
{
    return start < 0 || next < start ? -1 : next - start;
}

// What sequence b asks for (count 0 past the last one).
struct Request {
    int len, held, count, first;
};

__device__ __forceinline__ Request load_request(const PoolArgs& a, int b)
{
    Request q{0, 0, 0, 0};
    if (b < a.B) {
        q.len = a.kv_len[b];
        q.held = a.held[b];
        q.count = a.has_n ? a.n_new[b] : a.S;
        if (a.packed) {
            q.first = a.row_start[b];
            q.count = packed_count(q.first, a.row_start[b + 1]);
        }
    }
    return q;
}

__global__ void __launch_bounds__(kPageThreads) sv_reserve_kernel(PoolArgs a)
{
    __shared__ PageShared s;
    const int t = threadIdx.x;
    const unsigned nthr = gridDim.x * kPageThreads, me = blockIdx.x * kPageThreads + t;
    const bool first_block = blockIdx.x == 0;
    // the loads that need no other's result, before anything waits: what is left is
    // the chain length, page, slot
    Request q = load_request(a, t);
    const int avail = *a.free_count;
    const int row0 = a.packed ? a.row_start[0] : 0, row1 = a.packed ? a.row_start[a.B] : 0;
    uint32_t err = 0;
    bool bad = avail < 0 || avail > a.capacity || (a.packed && (row0 < 0 || row1 > a.rows || q.count < 0));
    if (a.packed)   // starts that do not ascend: no row could be told whose it is
        for (int b = t + kPageThreads; b < a.B; b += kPageThreads)
            bad |= packed_count(a.row_start[b], a.row_start[b + 1]) < 0;
    const bool all_bad = __syncthreads_or(bad) != 0;
    if (all_bad)
        err |= kErrCache;
    if (a.work && a.has_slots && a.packed) {   // rows of no sequence
        auto none = [&](long long r) { a.slots[r] = -1; };
        every(0, all_bad ? a.rows : row0, me, nthr, none);
        every(all_bad ? a.rows : row1, a.rows, me, nthr, none);
    }
    long long asked = 0, took = 0;   // by the sequences before this chunk
    for (int b0 = 0; b0 < a.B; b0 += kPageThreads) {
        const int b = b0 + t, nb = min(kPageThreads, a.B - b0);
        if (b0 > 0)
            q = load_request(a, b);
        const int len = q.len, held = q.held, count = q.count;
        long long want = 0;
        bool ok = false;
        if (t < nb) {
            s.first[t] = q.first;
            if (a.packed && t == nb - 1)
                s.first[nb] = q.first + count;
            ok = !all_bad && len >= 0 && count >= 0 && (a.packed || count <= a.S) && held >= 0 && held <= a.max_pages &&
                 (long long)len + count <= ((long long)a.max_pages << a.page_shift);
            if (ok)
                want = max(0, pages_for((long long)len + count, a.page_shift) - held);
            else
                err |= kErrCache;
        }
        if (a.clustered) {   // every block has read what the first one may write
            __syncwarp();    // (the barrier is for whole warps; the last sequences' lanes have just parted)
            cluster_arrive();
            cluster_wait();
        }
        long long total;
        const long long before = block_scan(want, s, total);
        const bool granted = ok && (want == 0 || asked + before + want <= avail);
        if (ok && !granted)
            err |= kErrPages;
        if (t < nb) {
            s.before[t] = before;
            s.len[t] = len;
            s.held[t] = held;
            s.count[t] = granted ? count : -1;
            if (a.update && first_block)
                a.held_out[b] = granted ? held + (int)want : held;
        }
        if (t == 0)
            s.before[nb] = total;
        __syncthreads();
        if (a.work) {
            for (long long j = me; j < total; j += nthr) {
                const int i = last_at_most(s.before, nb, j);
                const bool granted = s.count[i] >= 0;
                const int page = granted ? a.stack[avail - 1 - (asked + j)] : -1;
                if (granted && page < 0)
                    err |= kErrCache;
                a.table[(long long)(b0 + i) * a.max_pages + s.held[i] + (int)(j - s.before[i])] = page;
            }
            if (!a.has_slots && a.has_err)   // (slots look at every page that new tokens go to; without them, a warp a sequence)
                for (long long i = me >> 5; i < nb; i += nthr >> 5) {
                    if (s.count[i] <= 0)
                        continue;
                    const int first = s.len[i] >> a.page_shift;
                    const int end = min(s.held[i], pages_for((long long)s.len[i] + s.count[i], a.page_shift));
                    for (int pg = first + (t & 31); pg < end; pg += 32)
                        if (a.table[(b0 + i) * a.max_pages + pg] < 0)
                            err |= kErrCache;
                }
            if (a.has_slots && !(a.packed && all_bad)) {
                const long long r0 = a.packed ? s.first[0] : (long long)b0 * a.S;
                const long long r1 = a.packed ? s.first[nb] : (long long)(b0 + nb) * a.S;
                // a token a thread, or four from a multiple of four on where there are many: one
                // search, stores of 16 bytes
                const int each = a.each;
                for (long long r = r0 / each * each + (long long)each * me; r < r1; r += (long long)each * nthr) {
                    const long long x = max(r, r0), to = min(r + each, r1);
                    int i = a.packed ? last_at_most(s.first, nb, (int)x) : (int)(x / a.S) - b0;
                    int n = a.packed ? (int)x - s.first[i] : (int)(x - (long long)(b0 + i) * a.S);
                    long long slot[4] = {-1, -1, -1, -1};
                    int at_page = -1, page = -1;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        if (r + u >= to)
                            break;
                        if (r + u < x)
                            continue;
                        while (a.packed ? (int)(r + u) >= s.first[i + 1] : n >= a.S) {
                            ++i;
                            n = 0;
                            at_page = -1;
                        }
                        if (n < s.count[i]) {
                            const int pos = s.len[i] + n, pg = pos >> a.page_shift;
                            if (pg != at_page) {
                                at_page = pg;
                                page = pg < s.held[i] ? a.table[(long long)(b0 + i) * a.max_pages + pg]
                                                      : a.stack[avail - 1 - (asked + s.before[i] + pg - s.held[i])];
                            }
                            if (page >= 0)
                                slot[u] = ((long long)page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
                            else
                                err |= kErrCache;
                        }
                        ++n;
                    }
                    if (each == 4 && a.slots16 && r >= r0 && r + 4 <= r1) {
                        longlong2* out = reinterpret_cast<longlong2*>(a.slots + r);
                        out[0] = make_longlong2(slot[0], slot[1]);
                        out[1] = make_longlong2(slot[2], slot[3]);
                    } else {
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            if (r + u >= x && r + u < to)
                                a.slots[r + u] = slot[u];
                    }
                }
            }
        }
        if (a.update && first_block) {
            long long chunk_took;
            block_scan(granted ? want : 0, s, chunk_took);
            took += chunk_took;
        }
        asked += total;
        __syncthreads();
    }
    if (a.update && first_block && t == 0)
        *a.free_out = all_bad ? avail : (int)(avail - took);
    if (err && a.has_err && a.work)
        atomicOr(a.err, err);
}

__global__ void __launch_bounds__(kPageThreads) sv_release_kernel(PoolArgs a)
{
    __shared__ PageShared s;
    const int t = threadIdx.x;
    const unsigned nthr = gridDim.x * kPageThreads, me = blockIdx.x * kPageThreads + t;
    const bool first_block = blockIdx.x == 0;
    const int free_ = *a.free_count;
    uint32_t err = 0;
    // pages sequence b gives back; -1: its lengths cannot be used
    auto spare = [&](int b, int& keep) {
        const int len = a.kv_len[b], held = a.held[b];
        keep = pages_for(len, a.page_shift);
        return len < 0 || held < 0 || held > a.max_pages || keep > held ? -1 : held - keep;
    };
    long long mine = 0, all;
#pragma unroll 4
    for (int b = t; b < a.B; b += kPageThreads) {
        int keep;
        mine += max(0, spare(b, keep));
    }
    block_scan(mine, s, all);
    const bool all_bad = free_ < 0 || free_ > a.capacity || free_ + all > a.capacity;
    if (all_bad)
        err |= kErrCache;
    long long done = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPageThreads) {
        const int b = b0 + t, nb = min(kPageThreads, a.B - b0);
        int keep = 0, n = 0;
        if (t < nb) {
            n = spare(b, keep);
            if (n < 0)
                err |= kErrCache;
            s.held[t] = a.held[b];
            if (n < 0 || all_bad) {
                n = 0;
                keep = s.held[t];
            }
            s.len[t] = keep;
        }
        if (a.clustered) {
            __syncwarp();
            cluster_arrive();
            cluster_wait();
        }
        long long total;
        const long long before = block_scan(n, s, total);
        if (t < nb) {
            s.before[t] = before;
            if (a.update && first_block)
                a.held_out[b] = keep;
        }
        if (t == 0)
            s.before[nb] = total;
        __syncthreads();
        if (a.work)
            for (long long j = me; j < total; j += nthr) {
                const int i = last_at_most(s.before, nb, j);
                const int page = a.table[(long long)(b0 + i) * a.max_pages + s.len[i] + (int)(j - s.before[i])];
                if (page < 0)
                    err |= kErrCache;
                a.stack[free_ + all - 1 - (done + j)] = page;
            }
        done += total;
        __syncthreads();
    }
    if (a.update && first_block && t == 0)
        *a.free_out = all_bad ? free_ : (int)(free_ + all);
    if (err && a.has_err && a.work)
        atomicOr(a.err, err);
}

}  // namespace sv
