// sv_attention.cuh -- attention of tree nodes over the paged cache.
//
//   out[n] = sum_j softmax_j(scale q_n . k_j) v_j
// over the context's positions and node n's ancestors (itself included).
//
// The query rows that share a key head (nodes x query heads of its group, at
// most 128 to a CTA) are few beside the positions, so both products put the
// long side on the tensor core's 128 lanes:
//   S^T [128 positions x rows] = K_tile Q^T        (K and Q as they lie)
//   O^T [head_dim x rows]     += V_tile^T P^T      (V and P with positions as k)
// A thread of the softmax then owns one position of a tile and half of the
// rows: the e4m3 cache's scales are one multiplier a thread, the exponentials
// cost what the rows cost (no padding to 128), and the tree mask is one bit a
// row.  The price is that a row's maximum runs across threads, so it is not
// kept: weights are exp2(score - reference) with a reference a row that moves
// only when some score lies too far above it (a vote a tile).
//  * bf16 caches: references start at zero and stay there while scores are
//    within 2^+-24 of them; bf16 weights and fp32 sums keep their relative
//    precision at any such distance, so this is the softmax's value to rounding.
//  * e4m3 caches: weights are fp16 (below), so references are the maxima of the
//    first tile and move when a score is 2^8 above; a largest weight near 2^6
//    leaves fp16's floor (2^-25) at 2^-31 of it.
//
// An e4m3 cache's keys go to the tensor core as they are: each query element
// is split into an e4m3 and two e5m2 terms, which hold a bf16's eight bits
// exactly (to 2^-25 of the largest element that it is scaled with: the row
// group's, or the row's own where magnitudes spread by 2^8 or more), and the
// three products add up in the same accumulator.  Its values become fp16 in shared
// memory (one instruction a pair; 8-bit weights would need three terms and
// more range); their scales join the scores' exponents, so that weight times
// scale is what fp16 holds.
//
// Warps: 0-7 softmax (two warpgroups), 8 and 10 the issue of the first and the
// second product, 11 what an item needs before its first tile (tree masks).
//  * bf16: 9 loads the queries, 12-15 a quarter of each tile's keys and values
//    (a TMA copy of a page holds its warp for about 130 cycles, so one warp
//    cannot load small pages as fast as memory delivers them: on an earlier
//    form of the kernel 256 trees at pages of 16 took 371 us, 275 with four).
//  * e4m3: 9 loads the keys and 11 the values, 12-15 make the queries' terms
//    and convert a quarter of the values each (on an earlier form, with
//    converting warps that load as well, 64 chains took 118 us instead of 102).
// Tiles run through them in one stream across items.
//
// Measured on a GB300, a call (8 key heads of 128, 32 query heads):
//  * 256 trees of 15 nodes over 100-1500 positions, bf16, pages of 16: 173 us,
//    0.80 of the copy rate; HBM bounds it (914 MB read, nothing twice).
//  * 64 chains of 9 over 200-3000 positions, e4m3: 104-110 us (bytes 34 us); what a
//    tile takes from its load over conversion, products and softmax.
//  * 2 x 32 nodes over 100-120 thousand positions, e4m3: 199-207 us, 600 TFLOP/s;
//    tensor pipe 36 % and issue slots 38 % busy.
//  * one token over 700 positions: 11.7 us on the GPU, latency.
//
// Work is (sequence, key head, row group) items of 128-position tiles, laid
// end to end and cut into runs of equal cost, one to a CTA (an item costs its
// tiles and kItemCost more).  An item cut by a run's end leaves partial sums in
// the workspace, which sv_attention_combine joins.
#pragma once

#include "sv_kv.cuh"
#include "sv_tcgen05.cuh"

namespace sv {

constexpr int kAttnMaxCtas = 160;
constexpr int kTile = 128;                 // positions a tile
constexpr int kHalfBytes = kTile * 128;    // 128 swizzled rows of 128 bytes
// log2 of a weight at its row's reference, and of the largest before that moves
template <bool E4M3> constexpr float kAtRef = E4M3 ? 6.0f : 0.0f;
template <bool E4M3> constexpr float kLazy = E4M3 ? 14.0f : 24.0f;
constexpr int kMaxSlots = 8;
// What an item's start and end cost, in tiles.  Measured with 4, 2, 1 and 0: 256
// trees 173, 176, 187, 204 us; odd sizes (heads of 80) 52, 57, 61, 67; 64 chains 108,
// 114, 122, 132.  Wider heads were not measured: their tiles cost more, so that
// less would do there.
constexpr int kItemCost = 4;
constexpr int kQuarter = kTile / 4;        // positions a loading warp takes care of
// Query rows a CTA: 128, but 64 where the three 8-bit terms of wider heads'
// queries would leave the loads no room.
__host__ __device__ constexpr int attn_rows_max(bool e4m3, int D) { return e4m3 && D > 128 ? 64 : 128; }

// What the waits inside a CTA wait for (there, or free again): queries, slots of
// keys, values and converted values, what an item's rows need, scores, weights,
// sums.
enum AttnWait : int {
    kQFull, kQEmpty, kKFull, kKEmpty, kVFull, kVEmpty, kCFull, kCEmpty, kInfoFull, kInfoEmpty, kSFull, kSEmpty, kPFull, kOFull, kAttnWaits
};
static_assert(kAttnWaits == SV_ATTENTION_WAITS, "the header lists them");

struct AttnArgs {
    KvCache c;
    const __nv_bfloat16* q;
    long long q_stride;      // elements between tokens
    const int32_t* kv_len;
    const int32_t* n_nodes;
    const int32_t* parent;
    __nv_bfloat16* out;
    uint32_t* err;
    float* part_o;           // [2 CTAs][rows][D]
    float* part_ml;          // [2 CTAs][rows][2]
    int* meta;               // [CTAs][2]: the item a CTA begins / continues without ending it alone
    int has_n, has_parent, has_err;
    int Hq, G, B, Nmax;
    // row groups of a key head: blocks of `nodes` nodes by blocks of `heads` of
    // its query heads; rows = nodes * heads, row r being head r % heads of node
    // r / heads of the block
    int nodes, heads, head_blocks, groups, rows;
    int nd;                  // 128-wide chunks of head_dim
    int kslots, vslots, conv;         // ring sizes
    int k_bytes, v_bytes, conv_bytes; // of one slot
    int box_rows;            // rows of one TMA box (a page, or a tile)
    float scale_log2;        // scale * log2(e)
    uint32_t limit;          // polls before a wait gives up
    uint32_t hold;           // kinds of barriers (bits) made to lack an arrival
};

// Row r of group g: its node (of the sequence) and query head (of the key
// head's), false past either.
__device__ __forceinline__ bool attn_row(const AttnArgs& a, int g, int r, int& node, int& head)
{
    const int nb = g / a.head_blocks, n = r / a.heads;
    node = nb * a.nodes + n;
    head = (g - nb * a.head_blocks) * a.heads + r - n * a.heads;
    return r < a.rows && node < a.Nmax && head < a.G;
}

// One sequence's lengths; tiles >= 1 so that every output row has an item.
struct SeqLens {
    int ctx, nn, len, tiles;
    bool ok;
};

__device__ __forceinline__ SeqLens seq_lens(const AttnArgs& a, int b)
{
    SeqLens s;
    s.nn = a.has_n ? __ldg(a.n_nodes + b) : a.Nmax;
    s.ctx = __ldg(a.kv_len + b);
    const bool nodes = s.nn >= 0 && s.nn <= a.Nmax;
    s.ok = nodes && kv_span_ok(a.c, s.ctx, s.nn);
    s.len = s.ok && s.nn > 0 ? s.ctx + s.nn : 0;
    s.nn = nodes ? s.nn : a.Nmax;   // rows to report on
    s.tiles = max(1, (s.len + kTile - 1) / kTile);
    return s;
}

// A CTA's run of tiles, an item (or a part of one) at a time.  The items of
// no position are passed over but for the role that writes their rows.
struct Run {
    long long left;
    int b, h, g, tile;   // sequence, key head, row group; the tile after the part
    SeqLens s;
    // the current part
    int t0, t1;

    __device__ __forceinline__ bool next(const AttnArgs& a, bool empty_too = false)
    {
        do {
            if (left <= 0)
                return false;
            if (tile == s.tiles) {
                tile = 0;
                if (++g == a.groups) {
                    g = 0;
                    if (++h == a.c.Hkv) {
                        h = 0;
                        s = seq_lens(a, ++b);
                    }
                }
            }
            t0 = tile;
            t1 = (int)min((long long)s.tiles, t0 + left);
            left -= t1 - t0;
            tile = t1;
        } while (s.len == 0 && !empty_too);
        return true;
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == s.tiles; }
};

// The same a tile at a time.
struct Tiles {
    Run run;
    int j;          // the tile
    bool more;      // there is one

    __device__ __forceinline__ void start(const AttnArgs& a, const Run& r)
    {
        run = r;
        more = run.next(a);
        j = run.t0;
    }
    __device__ __forceinline__ void step(const AttnArgs& a)
    {
        if (++j == run.t1) {
            more = run.next(a);
            j = run.t0;
        }
    }
    __device__ __forceinline__ int valid() const { return min(kTile, run.s.len - j * kTile); }
};

// What an item's rows need to know, prepared while the one before is worked on.
struct alignas(16) ItemInfo {
    unsigned anc[128];     // the rows' ancestor bits (0: no row)
    int row_out[128];      // where their results go (-1: nowhere)
    unsigned poison;       // nodes whose values are not finite (or have a negative scale)
    unsigned bad;          // malformed tree, unusable page
};

struct AttnShared {
    uint64_t kfull[kMaxSlots], kempty[kMaxSlots];  // K slots
    uint64_t vfull[kMaxSlots], vempty[kMaxSlots];  // V slots
    uint64_t cfull[2], cempty[2];                  // converted V slots (e4m3)
    uint64_t q_full, q_empty, info_full[2], info_empty[2];
    uint64_t s_full[2], s_empty[2], p_full, o_full, drain[2];
    uint32_t fills[2][4];                          // slots of keys (values) that warps 12 .. 15 have asked for (bf16)
    long long t_begin, t_end, sum[16];
    uint32_t tmem;
    uint32_t limit;                                // polls a wait may take; zero once one has given up
    int b, h, g, tile, active;
    SeqLens first;                                 // the first sequence's lengths
    int unset[2];
    uint32_t top[4], low[4];
    uint32_t row_top[128];
    int q_spread[4];                               // by item: the rows have powers of two of their own,
    alignas(16) float q_row[4][128];               // these, over their group's
    float q_unscale[4];                            // undoes the queries' power of two (e4m3), by item: the first
                                                   // product runs at most two ahead of the softmax
    alignas(16) float negm[128];                   // minus the rows' references
    float scratch[2][5 * 64];
    ItemInfo info[2];
};

// The dynamic shared memory.  Every role derives its own pointers (through a
// zero the compiler does not see): shared ones would hold registers in all of
// them, and the roles have few.
struct AttnLayout {
    unsigned char *k, *v, *c, *p, *q;   // K, V, converted V slots; P; Q (bf16, or three 8-bit terms)
    AttnShared* sh;
    int q_part;                         // bytes of one 8-bit term of Q
};

template <int N, bool E4M3>
__device__ __forceinline__ AttnLayout attn_layout(const AttnArgs& a, unsigned char* smem)
{
    int zero;
    asm volatile("mov.u32 %0, 0;" : "=r"(zero));
    AttnLayout L;
    L.k = smem + zero;
    L.v = L.k + a.kslots * a.k_bytes;
    L.c = L.v + a.vslots * a.v_bytes;
    L.p = L.c + (E4M3 ? a.conv * a.conv_bytes : 0);
    L.q = L.p + (N + 63) / 64 * kHalfBytes;
    L.q_part = N * 128 * a.nd;
    L.sh = reinterpret_cast<AttnShared*>(L.q + (E4M3 ? 3 * L.q_part : N * 128 * ((a.c.D + 63) / 64)));
    return L;
}

__device__ __forceinline__ Run run_of(const AttnShared& shared)
{
    const volatile AttnShared& sh = shared;
    Run r;
    r.left = sh.active ? sh.t_end - sh.t_begin : 0;
    r.b = sh.active ? sh.b : 0;
    r.h = sh.h;
    r.g = sh.g;
    r.tile = sh.tile;
    r.t0 = r.t1 = 0;
    r.s.ctx = sh.first.ctx;
    r.s.nn = sh.first.nn;
    r.s.len = sh.first.len;
    r.s.tiles = sh.first.tiles;
    r.s.ok = sh.first.ok;
    return r;
}

// A wait that ends, of a whole warp and alike in all its lanes: on a timeout
// the CTA's limit becomes zero, so that every later wait gives up too (after a
// poll that fails).  A warp whose wait gave up issues and arrives at nothing any
// more: what the others still wait for is there when their waits pass.  The
// warps that own named barriers run on (they all reach the same ones), the
// others stop.
__device__ __forceinline__ bool cta_wait(AttnShared& sh, uint64_t* bar, uint32_t parity)
{
    const uint32_t addr = smem_addr(bar);
    volatile uint32_t* const limit = &sh.limit;
    // (never unrolled: the kernel has some forty of these, and its code has to stay in the instruction caches)
#pragma unroll 1
    for (uint32_t i = 1; !__all_sync(kFull, mbar_try_wait(addr, parity)); ++i)
        if (i >= *limit) {   // (one load of the converged warp)
            *limit = 0;
            return false;
        }
    return true;
}

// A role's last wait, for its own copies and products in flight: they land
// before the CTA's memory is given back, whoever gave up.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity)
{
    const uint32_t addr = smem_addr(bar);
#pragma unroll 1
    for (uint32_t i = 0; i < kWaitSpins && !mbar_try_wait(addr, parity); ++i)
        ;
}

// Ring position: slot index and the parity its next wait takes.
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step(int n)
    {
        if (++slot == n) {
            slot = 0;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ void back(int n)
    {
        if (slot == 0) {
            slot = n;
            phase ^= 1;
        }
        --slot;
    }
};

// One lane: the arrival that a barrier was made to lack, once a wait has given up.
__device__ __forceinline__ void make_up(AttnShared& sh, uint64_t* bar)
{
#pragma unroll 1
    for (uint32_t i = 0; i < kWaitSpins && *reinterpret_cast<volatile uint32_t*>(&sh.limit); ++i)
        __nanosleep(500);
    mbar_arrive(smem_addr(bar));
}

// The last copies into each slot of a ring that has been filled `fills` times,
// `r` standing at the next.  `held`: the slots' barriers lack an arrival (none
// has been filled twice then), which one lane makes up for.
__device__ __forceinline__ void drain_ring(AttnShared& sh, uint64_t* full, Ring r, int slots, uint32_t fills, bool held)
{
#pragma unroll 1
    for (uint32_t n = min(fills, (uint32_t)slots); n > 0; --n) {
        r.back(slots);
        if (held)
            make_up(sh, &full[r.slot]);
        drain_wait(&full[r.slot], r.phase);
    }
}

// Four e4m3 values as fp16, exactly (NaN as NaN).
__device__ __forceinline__ uint2 e4m3_to_f16(uint32_t w)
{
    uint2 y;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(y.x), "=r"(y.y) : "r"(w));
    return y;
}

__device__ __forceinline__ uint32_t f16_pair(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ bool bf16_pair_nonfinite(uint32_t w)
{
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// The e4m3 NaNs are the bytes 0x7f and 0xff (there is no infinity): adding one
// to the low seven bits carries into the eighth there alone.
__device__ __forceinline__ bool chunk_nan_e4m3(uint4 w)
{
    constexpr uint32_t low = 0x7f7f7f7fu, one = 0x01010101u;
    return ((((w.x & low) + one) | ((w.y & low) + one) | ((w.z & low) + one) | ((w.w & low) + one)) & 0x80808080u) != 0;
}

__device__ __forceinline__ bool chunk_nonfinite(uint4 w, bool e4m3)
{
    return e4m3 ? chunk_nan_e4m3(w)
                : bf16_pair_nonfinite(w.x) || bf16_pair_nonfinite(w.y) || bf16_pair_nonfinite(w.z) || bf16_pair_nonfinite(w.w);
}

// Two query elements (scaled so that the group's largest is below 256) as an
// e4m3 and two e5m2 terms each.  The differences are exact in fp16 (down to
// 2^-24).  NaN stays NaN; an infinity, which the conversions would saturate,
// is made one by the difference with itself.
__device__ __forceinline__ void split_q(float x0, float x1, uint32_t& h, uint32_t& m, uint32_t& l)
{
    const uint64_t z = f2_pack(x0, x1);
    f2_unpack(f2_add(z, f2_sub(z, z)), x0, x1);
    const __half2 x = __floats2half2_rn(x0, x1);
    h = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(x), __NV_SATFINITE, __NV_E4M3);
    const __half2 r = __hsub2(x, __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h, __NV_E4M3)));
    m = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(r), __NV_SATFINITE, __NV_E5M2);
    const __half2 r2 = __hsub2(r, __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)m, __NV_E5M2)));
    l = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(r2), __NV_SATFINITE, __NV_E5M2);
}

// One lane: the products of a K slot (bf16, or e4m3 with the three terms of
// Q).  `steps`: 32-byte steps of the contraction in this slot.  Descriptors
// differ by constants in their low words.
template <int N, bool E4M3>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t k, uint32_t q, uint32_t q_part, int steps, bool add)
{
    const uint32_t ka = tc_desc_lo(k, 16), qb = tc_desc_lo(q, 16);
    if (E4M3) {
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const uint32_t id = tc_idesc(128, N, 0, p > 0, false, false), qp = qb + p * (q_part >> 4);
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (s < steps)
                    tc_mma_f8(d, tc_desc(ka + 2 * s), tc_desc(qp + 2 * s), id, add || p + s > 0);
        }
    } else {
        constexpr uint32_t id = tc_idesc(128, N, 1, 1, false, false);
#pragma unroll
        for (int s = 0; s < 8; ++s)
            if (s < steps)
                tc_mma_16(d, tc_desc(ka + (s >> 2) * (kHalfBytes / 16) + (s & 3) * 2),
                            tc_desc(qb + (s >> 2) * (N * 128 / 16) + (s & 3) * 2), id, add || s > 0);
    }
}

// One lane: a V slot (bf16, or fp16 from e4m3) times P.  `steps`: 16-position
// steps.
template <int N, bool E4M3>
__device__ __forceinline__ void mma_values(uint32_t d, uint32_t v, uint32_t p, uint32_t lbo, int steps, bool add)
{
    constexpr uint32_t id = tc_idesc(128, N, E4M3 ? 0 : 1, E4M3 ? 0 : 1, true, true);
    const uint32_t va = tc_desc_lo(v, lbo), pb = tc_desc_lo(p, kHalfBytes);
#pragma unroll
    for (int s = 0; s < 8; ++s)
        if (s < steps)
            tc_mma_16(d, tc_desc(va + s * (2048 / 16)), tc_desc(pb + s * (2048 / 16)), id, add || s > 0);
}

// The rare step of the softmax, by the warpgroup's 128 threads: rows whose
// scores lie too far from their references get new ones (their maxima over
// this tile), and the sums in TMEM are rescaled.  In bf16 each row goes by its
// own scores, so that its rounding does not depend on the rows beside it.  In
// e4m3, where moves are frequent, all rows that have risen move at once (two
// sequences of 110 thousand positions: 200 us, 233 with a move a row on an
// earlier form).  scratch[0 .. NT) then holds
// the factors of what was summed so far, [NT .. 2 NT) how far references rose.
template <int NT, bool E4M3>
__device__ __forceinline__ void move_references(float* scratch, float* negm, int* unset_flag, uint32_t s_at, uint32_t o_at,
                                                int o_chunks, int o_pitch, float mult, float add, unsigned long long seen, int t, int bar)
{
    const int lane = t & 31, warp = t >> 5;
#pragma unroll 1
    for (int c = 0; c < NT; c += 8) {
        float s[8], keep = 0.0f;
        tmem_ld8(s_at + c, s);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float x = warp_redux_max((seen >> (c + k)) & 1 ? fmaf(s[k], mult, negm[c + k] + add) : -INFINITY);
            keep = lane == k ? x : keep;
        }
        if (lane < 8)
            scratch[warp * NT + c + lane] = keep;
    }
    bar_sync(bar, 128);
    bool unset = false;
    if (t < NT) {
        const float x = fmaxf(fmaxf(scratch[t], scratch[NT + t]), fmaxf(scratch[2 * NT + t], scratch[3 * NT + t]));
        float f = 1.0f, delta = 0.0f;
        // +0 marks a row that has no reference yet: nothing is in its sums
        const float old = negm[t];
        if (__float_as_uint(old) == 0u) {
            unset = x == -INFINITY;
            delta = unset || (!E4M3 && fabsf(x) <= kLazy<E4M3>) ? 0.0f : x - kAtRef<E4M3>;
        } else if (x > (E4M3 ? kAtRef<E4M3> : kLazy<E4M3>)) {
            delta = x - kAtRef<E4M3>;
            f = ex2_approx(-delta);
        }
        if (!unset) {
            const float now = old - delta;
            negm[t] = __float_as_uint(now) == 0u ? -0.0f : now;
        }
        scratch[t] = f;
        scratch[NT + t] = delta;
    }
    unset = bar_any(bar, 128, unset);
    if (t == 0)
        *unset_flag = unset;
#pragma unroll 1
    for (int i = 0; i < o_chunks; ++i)
#pragma unroll 1
        for (int c = 0; c < NT; c += 8) {
            float o[8];
            tmem_ld8(o_at + i * o_pitch + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 8; ++k)
                o[k] *= scratch[c + k];
            tmem_st8(o_at + i * o_pitch + c, o);
        }
    tmem_wait_st();
}

// A thread's scores brought to one scale, where they are: for the rare items
// whose queries spread widely.
template <int NT>
__device__ __forceinline__ void scale_rows(uint32_t s_at, const float* by)
{
#pragma unroll 1
    for (int c = 0; c < NT; c += 8) {
        float s[8];
        tmem_ld8(s_at + c, s);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s[k] *= by[c + k];
        tmem_st8(s_at + c, s);
    }
    tmem_wait_st();
}

// Weights exp2(s) of a position, rounded once into P, and their sums.
//  * bf16: a weight's rounding (a bf16 unit of 2^-8) averages out over the
//    positions.  ROUNDED sums take what P holds, so that the rounding of a
//    weight that dominates its row cancels; that costs three instructions a
//    pair, which the launches of few rows have to spare.
//  * e4m3: s holds the value's scale too; the sums take it back (unscale).
template <int NT, bool E4M3, bool ROUNDED>
__device__ __forceinline__ void weigh(const float (&s)[NT], float unscale, uint64_t (&l2)[NT / 2], unsigned char* p_row, int at, int t)
{
    const uint64_t u2 = f2_pack(unscale, unscale);
#pragma unroll
    for (int i = 0; i < NT / 8; ++i) {
        uint32_t x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float lo = ex2_approx(s[8 * i + 2 * k]), hi = ex2_approx(s[8 * i + 2 * k + 1]);
            uint64_t& l = l2[4 * i + k];
            if (E4M3) {
                l = f2_fma(f2_pack(lo, hi), u2, l);
                x[k] = f16_pair(lo, hi);
            } else {
                x[k] = bf16_pair(lo, hi);
                l = f2_add(l, ROUNDED ? f2_pack(__uint_as_float(x[k] << 16), __uint_as_float(x[k] & 0xffff0000u)) : f2_pack(lo, hi));
            }
        }
        // P: rows of 64 of the CTA's N columns a position, swizzled
        *reinterpret_cast<uint4*>(p_row + ((at + i) >> 3) * kHalfBytes + ((((at + i) ^ t) & 7) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
    }
}

// A thread's element of NT rows of O: out(row's place, element, row's factor).
template <int NT, typename F>
__device__ __forceinline__ void store_rows(uint32_t o_at, const int* row_out, const float* fin, int d, int D, F out)
{
#pragma unroll 1
    for (int i = 0; i < NT; i += 8) {
        float o[8];
        tmem_ld8(o_at + i, o);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
            const int4 at = *reinterpret_cast<const int4*>(row_out + i + k);
            const float4 f = *reinterpret_cast<const float4*>(fin + i + k);
            if (d < D) {
                if (at.x >= 0)
                    out(at.x, o[k], f.x);
                if (at.y >= 0)
                    out(at.y, o[k + 1], f.y);
                if (at.z >= 0)
                    out(at.z, o[k + 2], f.z);
                if (at.w >= 0)
                    out(at.w, o[k + 3], f.w);
            }
        }
    }
}

// Loads that stay where they are written (a plain one sinks to its first use,
// an iteration later, and takes its latency there).
__device__ __forceinline__ int load_now(const int* p)
{
    int x;
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(x) : "l"(p));
    return x;
}

__device__ __forceinline__ float load_now(const float* p)
{
    float x;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(x) : "l"(p));
    return x;
}

// The page table's entry for position pos of sequence b, as it is.
__device__ __forceinline__ int page_entry(const AttnArgs& a, int b, int pos)
{
    return load_now(a.c.table + (long long)b * a.c.max_pages + (pos >> a.c.page_shift));
}

// The boxes of `count` positions of a tile from `first` on: lane l's is where
// its page starts, or nowhere.
struct Boxes {
    int page, pos, h;

    // asks for the pages (the entries are looked at by row(), a tile later)
    __device__ __forceinline__ void ask(const AttnArgs& a, const Tiles& x, int first, int count, int lane)
    {
        pos = x.j * kTile + first + lane * a.box_rows;
        h = x.run.h;
        page = -1;
        if (x.more && lane * a.box_rows < count && pos < x.run.s.len)
            page = page_entry(a, x.run.b, pos);
    }
    // its first row, -1 where the box holds no position (or its page is unusable)
    __device__ __forceinline__ int row(const AttnArgs& a) const
    {
        return (unsigned)page < (unsigned)a.c.num_pages ? (int)kv_row(a.c, page, pos) + (h << a.c.page_shift) : -1;
    }
};

// One warp: chunk c of such boxes into a slot's rows at dst.
template <bool E4M3>
__device__ __forceinline__ void load_boxes(const AttnArgs& a, uint32_t dst, uint32_t bar, const CUtensorMap* map, int c, int row, int lane)
{
    const uint32_t step = a.box_rows * 128;
    const bool two = !E4M3 && a.c.D - 128 * c > 64;
    const unsigned have = __ballot_sync(kFull, row >= 0);
    if (lane == 0)
        mbar_arrive_expect_tx(bar, __popc(have) * step * (two ? 2 : 1));
    __syncwarp();
    if (row >= 0) {
        tma_load_2d(dst + lane * step, map, 128 * c, row, bar);
        if (two)
            tma_load_2d(dst + kHalfBytes + lane * step, map, 128 * c + 64, row, bar);
    }
    __syncwarp();
}

// One warp: what item number `items` of the CTA's run needs to know of its rows.
template <int N, bool E4M3>
__device__ __forceinline__ bool prepare_item(const AttnArgs& a, AttnShared& sh, const Run& run, uint32_t items, int lane)
{
    ItemInfo& info = sh.info[items & 1];
    const int h = run.h, g = run.g, nn = run.s.nn, ctx = run.s.ctx;
    const int part = 2 * blockIdx.x + (run.t0 > 0 ? 0 : 1);
    int par;
    const bool tree = tree_parents(a.parent + (long long)run.b * a.Nmax, a.has_parent, nn, lane, par);
    // lane n: node n and its ancestors
    unsigned anc = lane < nn ? 1u << lane : 0u;
    {
        int at = lane < nn && tree ? par : -1;
        while (__any_sync(kFull, at >= 0)) {   // parents are earlier nodes: at most 31 steps
            if (at >= 0)
                anc |= 1u << at;
            const int up = __shfl_sync(kFull, par, max(at, 0));
            at = at >= 0 ? up : -1;
        }
        if (!tree && lane < nn)
            anc = ~0u;   // (a malformed tree's rows end as NaN, whatever they see)
    }
    // the part's pages; its nodes' values
    bool bad = !tree;
    const int p1 = min(run.t1 * kTile, run.s.len);
#pragma unroll 1
    for (int pos = run.t0 * kTile + (lane << a.c.page_shift); pos < p1; pos += 32 << a.c.page_shift)
        bad |= kv_page(a.c, run.b, pos) < 0;
    bad = __any_sync(kFull, bad);
    unsigned poison = 0;
    if (nn > 1 && run.t1 * kTile > ctx) {
        const int bytes = a.c.D * (E4M3 ? 1 : 2);
        // lane m: where node m's row lies
        long long row = -1;
        if (lane < nn && ctx + lane >= run.t0 * kTile && ctx + lane < run.t1 * kTile) {
            const int page = kv_page(a.c, run.b, ctx + lane);
            if (page >= 0)
                row = kv_row(a.c, page, ctx + lane) + ((long long)h << a.c.page_shift);
        }
        if (E4M3 && row >= 0) {   // a negative scale reads as NaN
            const float s = a.c.v_scale[row];
            if (!(s >= 0.0f && s < INFINITY))
                poison = 1u << lane;
        }
        if (row >= 0) {   // a lane reads its node's row, eight pieces in flight
            const uint4* x = reinterpret_cast<const uint4*>(a.c.v + row * bytes);
            bool hit = false;
#pragma unroll 1
            for (int i = 0; i < bytes / 16; i += 8) {
                uint4 y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    y[k] = i + k < bytes / 16 ? __ldg(x + i + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    hit |= chunk_nonfinite(y[k], E4M3);
            }
            if (hit)
                poison = 1u << lane;
        }
        poison = __reduce_or_sync(kFull, poison);
    }
    if (!cta_wait(sh, &sh.info_empty[items & 1], ((items >> 1) & 1) ^ 1))
        return false;
    if (lane == 0) {
        info.poison = poison;
        info.bad = bad;
    }
#pragma unroll 1
    for (int r = lane; r < (N + 31) / 32 * 32; r += 32) {
        int node = 0, head = 0;
        const bool real = r < N && attn_row(a, g, r, node, head);
        const unsigned its = __shfl_sync(kFull, anc, node & 31);
        info.anc[r] = real && node < nn ? its : 0u;
        info.row_out[r] = !real         ? -1
                          : run.whole() ? (run.b * a.Nmax + node) * a.Hq + h * a.G + head
                                        : part * a.rows + r;
    }
    __syncwarp();
    if (lane == 0)
        mbar_arrive(smem_addr(&sh.info_full[items & 1]));
    return true;
}

constexpr int kAttnThreads = 512;
// Registers a thread: the softmax's warpgroups (warps 0 .. 7) hold NT scores and
// NT sums a thread, the issuing warps (8 .. 11) little; a spill costs a loop
// its L2 latency, the caches being shared memory (bf16 spills 32 bytes at 48
// rows a warpgroup and 28 at 64, e4m3 16 at 64, the others none).  The shares
// add up to the launch's.
constexpr int kAttnRegs = 128;       // at launch
template <int NT> constexpr int kRegsSoftmax = NT >= 64 ? 168 : 152;
template <int NT> constexpr int kRegsIssue = NT >= 64 ? 80 : 96;
template <int NT> constexpr int kRegsTiles = 4 * kAttnRegs - kRegsIssue<NT> - 2 * kRegsSoftmax<NT>;

// NT: rows (TMEM columns) a softmax warpgroup handles; NWG: softmax
// warpgroups with rows.
template <int NT, int NWG, bool E4M3>
__global__ void __launch_bounds__(kAttnThreads, 1)
    sv_attention_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_q)
{
    constexpr int kThreads = kAttnThreads, kWarps = kThreads / 32, N = NT * NWG;
    extern __shared__ __align__(1024) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, D = a.c.D;
    {
        const AttnLayout L = attn_layout<N, E4M3>(a, smem);
        AttnShared& sh = *L.sh;
        if (warp == 8) {
            tmem_alloc(smem_addr(&sh.tmem), 512);
        } else if (tid == 9 * 32) {
            sh.limit = a.limit;
            auto init = [&](uint64_t& bar, int count, int kind) { mbar_init(smem_addr(&bar), count + ((a.hold >> kind) & 1)); };
#pragma unroll 1
            for (int i = 0; i < a.kslots; ++i) {
                init(sh.kfull[i], E4M3 ? 1 : 4, kKFull);
                init(sh.kempty[i], 1, kKEmpty);
            }
#pragma unroll 1
            for (int i = 0; i < a.vslots; ++i) {
                init(sh.vfull[i], E4M3 ? 1 : 4, kVFull);
                init(sh.vempty[i], E4M3 ? 4 : 1, kVEmpty);
            }
            for (int i = 0; i < 2; ++i) {
                init(sh.cfull[i], 4, kCFull);
                init(sh.cempty[i], 1, kCEmpty);
                init(sh.s_full[i], 1, kSFull);
                init(sh.s_empty[i], 4 * NWG, kSEmpty);
                init(sh.info_full[i], 1, kInfoFull);
                init(sh.info_empty[i], 4 * NWG, kInfoEmpty);
            }
            init(sh.q_full, 1, kQFull);
            init(sh.q_empty, 1, kQEmpty);
            init(sh.p_full, 4 * NWG, kPFull);
            init(sh.o_full, 1, kOFull);
            mbar_init(smem_addr(&sh.drain[0]), 1);
            mbar_init(smem_addr(&sh.drain[1]), 1);
            fence_mbar_init();
            tma_prefetch_map(&map_k);
            tma_prefetch_map(&map_v);
        }
        // the rows of no query, and the elements past head_dim, stay zeros
#pragma unroll 1
        for (int i = tid; i < (int)(reinterpret_cast<unsigned char*>(L.sh) - L.q) / 16; i += kThreads)
            reinterpret_cast<uint4*>(L.q)[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async();
        // the CTA's run: tiles of all sequences before each thread's share of them
        const int share = (a.B + kThreads - 1) / kThreads, b0 = min(tid * share, a.B), b1 = min(b0 + share, a.B);
        const int per = a.c.Hkv * a.groups;
        long long mine = 0;
#pragma unroll 1
        for (int b = b0; b < b1; ++b)
            mine += (long long)(seq_lens(a, b).tiles + kItemCost) * per;
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(kFull, incl, o);
            if (lane >= o)
                incl += x;
        }
        if (lane == 31)
            sh.sum[warp] = incl;
        __syncthreads();
        long long before = 0, total = 0;
#pragma unroll 1
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp)
                before += sh.sum[w];
            total += sh.sum[w];
        }
        const long long excl = before + incl - mine;
        const int act = (int)min((long long)gridDim.x, total), i = blockIdx.x;
        const long long each = total / act, extra = total - each * act;
        const long long begin = each * i + min((long long)i, extra), end = each * (i + 1) + min((long long)i + 1, extra);
        // the tile that a point of the cost line falls in (a point in an item's fixed cost: its first tile)
        if (b1 > b0)
#pragma unroll 1
            for (int which = 0; which < 2; ++which) {
                const long long point = which ? end : begin;
                if (point < excl || point >= excl + mine) {
                    if (which && point == total && b1 == a.B)
                        sh.t_end = total - (long long)kItemCost * per * a.B;
                    continue;
                }
                long long at = excl;
                int b = b0, cost;
#pragma unroll 1
                for (;; ++b) {
                    cost = seq_lens(a, b).tiles + kItemCost;
                    if (point < at + (long long)cost * per)
                        break;
                    at += (long long)cost * per;
                }
                const int hg = (int)((point - at) / cost);
                const int tile = max(0, (int)(point - at - (long long)hg * cost) - kItemCost);
                const long long t_index = at - (long long)kItemCost * per * b + (long long)hg * (cost - kItemCost) + tile;
                if (which) {
                    sh.t_end = t_index;
                } else {
                    sh.t_begin = t_index;
                    sh.b = b;
                    sh.h = hg / a.groups;
                    sh.g = hg - sh.h * a.groups;
                    sh.tile = tile;
                    sh.first = seq_lens(a, b);
                }
            }
        if (tid == 0) {
            sh.active = i < act;
            a.meta[2 * i] = a.meta[2 * i + 1] = -1;
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }

    // (The register moves stand inside the warpgroups' branches: ptxas budgets
    // what they dominate.)
    if (warp < 8) {
        regs_grow<kRegsSoftmax<NT>>();
        if (warp < 4 * NWG) {
            // --- softmax: one position a thread, NT rows --------------------------
            const AttnLayout L = attn_layout<N, E4M3>(a, smem);
            AttnShared& sh = *L.sh;
            Run run = run_of(sh);
            const int w = warp >> 2, t = tid & 127, bar = 1 + w;
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t tmem = sh.tmem + lanes + w * NT, tmem_o = tmem + 2 * N;   // S (two buffers of N columns), then O
            float* const scratch = sh.scratch[w];
            float* const negm = sh.negm + w * NT;
            uint32_t gt = 0, items = 0;   // tiles, items so far
            constexpr uint32_t kGaveUp = 1u << 31;   // in gt: a wait of this warp gave up (a flag of its own is a spill)
            while (run.next(a, true)) {
                const int ctx = run.s.ctx, nn = run.s.nn, h = run.h;
                const int part = 2 * blockIdx.x + (run.t0 > 0 ? 0 : 1);
                const bool whole = run.whole();
                if (!whole && tid == 0)   // meta[2i]: begun here, meta[2i + 1]: continued here
                    a.meta[part ^ 1] = (run.b * a.c.Hkv + h) * a.groups + run.g;
                bool lost = !run.s.ok;   // the item's rows are NaN
                if (run.s.len != 0) {
                    // pages and scales a tile ahead (e4m3)
                    auto page_of = [&](int j) {
                        const int pos = j * kTile + t;
                        return E4M3 && j < run.t1 && pos < run.s.len ? page_entry(a, run.b, pos) : -1;
                    };
                    auto scales_of = [&](int j, int page, float& k, float& v) {
                        k = v = 0.0f;
                        if (E4M3 && (unsigned)page < (unsigned)a.c.num_pages) {
                            const long long row = kv_row(a.c, page, j * kTile + t) + ((long long)h << a.c.page_shift);
                            k = load_now(a.c.k_scale + row);
                            v = load_now(a.c.v_scale + row);
                        }
                    };
                    float ks, vs, ks_next = 0.0f, vs_next = 0.0f;
                    int page_next = page_of(run.t0);
                    scales_of(run.t0, page_next, ks, vs);
                    page_next = page_of(run.t0 + 1);
                    const ItemInfo& info = sh.info[items & 1];
                    if (t < NT)
                        negm[t] = 0.0f;
                    if (t == 0)
                        sh.unset[w] = 0;
                    bar_sync(bar, 128);
                    float scale_log2 = a.scale_log2;
                    uint64_t l2[NT / 2];  // this thread's share of the rows' sums, in pairs
#pragma unroll
                    for (int i = 0; i < NT / 2; ++i)
                        l2[i] = 0;

#pragma unroll 1
                    for (int j = run.t0; j < run.t1; ++j, ++gt) {
                        const bool first_tile = j == run.t0;
                        if (!cta_wait(sh, &sh.s_full[gt & 1], (gt >> 1) & 1))
                            gt |= kGaveUp;
                        tc_fence_after();
                        const uint32_t s_at = tmem + (gt & 1) * N;
                        if (E4M3 && sh.q_spread[items & 3])
                            scale_rows<NT>(s_at, sh.q_row[items & 3] + w * NT);
                        float s[NT];
#pragma unroll
                        for (int i = 0; i < NT / 16; ++i)
                            tmem_ld16(s_at + 16 * i, s + 16 * i);
                        if (NT % 16)
                            tmem_ld8(s_at + NT - 8, s + NT - 8);
                        float mult = a.scale_log2, add = 0.0f;   // add: log2 of the value's scale
                        if (E4M3) {
                            if (first_tile)
                                scale_log2 = a.scale_log2 * sh.q_unscale[items & 3];
                            // a scale that is not finite marks a row that held something that was not
                            mult = scale_log2 * (isfinite(ks) ? ks : NAN);
                            // (below 2^-100 all of a row's values are zero in the sum; a negative scale is none)
                            add = isfinite(vs) ? __log2f(vs >= 0.0f && vs < 0x1p-100f ? 0x1p-100f : vs) : NAN;
                            scales_of(j + 1, page_next, ks_next, vs_next);
                            page_next = page_of(j + 2);
                        }
                        // scores in powers of two, relative to the rows' references
                        const uint64_t m2 = f2_pack(mult, mult), a2 = f2_pack(add, add);
                        const ulonglong2* nm = reinterpret_cast<const ulonglong2*>(negm);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < NT / 4; ++i) {
                            ulonglong2 x = nm[i];
                            if (E4M3)
                                x = make_ulonglong2(f2_add(x.x, a2), f2_add(x.y, a2));
                            f2_unpack(f2_fma(f2_pack(s[4 * i], s[4 * i + 1]), m2, x.x), s[4 * i], s[4 * i + 1]);
                            f2_unpack(f2_fma(f2_pack(s[4 * i + 2], s[4 * i + 3]), m2, x.y), s[4 * i + 2], s[4 * i + 3]);
                        }
                        // who sees this position: every row in the context, a node's descendants behind it
                        unsigned long long seen = ~0ull;
                        if ((j + 1) * kTile > ctx) {   // the tile holds nodes, or ends the sequence
                            if (!cta_wait(sh, &sh.info_full[items & 1], (items >> 1) & 1))
                                gt |= kGaveUp;
                            const unsigned poison = info.poison;
                            const int m = j * kTile + t - ctx;
                            if (m >= 0) {
                                seen = 0;
                                if (m < nn && !((poison >> m) & 1u)) {
#pragma unroll 1
                                    for (int i = 0; i < NT; ++i)
                                        seen |= (unsigned long long)((info.anc[w * NT + i] >> m) & 1u) << i;
                                } else {   // nothing does: its scales may be anything
                                    add = 0.0f;
                                }
                            }
#pragma unroll
                            for (int i = 0; i < NT; ++i)
                                s[i] = (seen >> i) & 1 ? s[i] : -INFINITY;
                        }
                        // are all scores near enough to the references?
                        float top[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            top[k] = max3(s[4 * k], s[4 * k + 1], fmaxf(s[4 * k + 2], s[4 * k + 3]));
#pragma unroll
                        for (int i = 16; i < NT; i += 2)
                            top[(i >> 1) & 3] = max3(top[(i >> 1) & 3], s[i], s[i + 1]);
                        bool move = bar_any(bar, 128, max3(top[0], top[1], fmaxf(top[2], top[3])) > kLazy<E4M3>) || sh.unset[w];
                        if (first_tile && E4M3) {
                            move = true;
                        } else if (first_tile) {
                            // no reference yet: zero will do if some position's scores are all near enough
                            float low[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                low[k] = min3(s[4 * k], s[4 * k + 1], fminf(s[4 * k + 2], s[4 * k + 3]));
#pragma unroll
                            for (int i = 16; i < NT; i += 2)
                                low[(i >> 1) & 3] = min3(low[(i >> 1) & 3], s[i], s[i + 1]);
                            move = !bar_any(bar, 128, min3(low[0], low[1], fminf(low[2], low[3])) >= -kLazy<E4M3>) || move;
                            if (!move && t < NT)
                                negm[t] = -0.0f;   // (+0 marks a row without a reference)
                        } else {   // the previous tile's product is done with P (and O)
                            if (!cta_wait(sh, &sh.o_full, (gt - 1) & 1))
                                gt |= kGaveUp;
                            tc_fence_after();
                        }
                        if (move) {
                            move_references<NT, E4M3>(scratch, negm, &sh.unset[w], s_at, tmem_o, first_tile ? 0 : a.nd, N, mult, add, seen, t, bar);
#pragma unroll
                            for (int i = 0; i < NT / 4; ++i) {
                                const ulonglong2 f = reinterpret_cast<const ulonglong2*>(scratch)[i];
                                const float4 d = reinterpret_cast<const float4*>(scratch + NT)[i];
                                l2[2 * i] = f2_mul(l2[2 * i], f.x);
                                l2[2 * i + 1] = f2_mul(l2[2 * i + 1], f.y);
                                s[4 * i] -= d.x;
                                s[4 * i + 1] -= d.y;
                                s[4 * i + 2] -= d.z;
                                s[4 * i + 3] -= d.w;
                            }
                            bar_sync(bar, 128);   // the scratch may be written again
                        }
                        weigh<NT, E4M3, NWG == 1>(s, E4M3 ? ex2_approx(-add) : 1.0f, l2, L.p + t * 128, w * (NT / 8), t);
                        tc_fence_before();
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0 && gt < kGaveUp) {
                            mbar_arrive(smem_addr(&sh.s_empty[gt & 1]));
                            mbar_arrive(smem_addr(&sh.p_full));
                        }
                        if (E4M3) {
                            ks = ks_next;
                            vs = vs_next;
                        }
                    }

                    // the rows' sums over the 128 threads, while the last product runs
#pragma unroll
                    for (int i = 0; i < NT / 8; ++i) {
                        // lane c (of 8) ends with column 8 i + c: halve the columns, double the lanes summed
                        float x[8];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            f2_unpack(l2[4 * i + k], x[2 * k], x[2 * k + 1]);
#pragma unroll
                        for (int o = 4; o > 0; o >>= 1)
#pragma unroll
                            for (int k = 0; k < o; ++k) {
                                const bool up = lane & o;
                                const float send = up ? x[k] : x[k + o];
                                const float keep = up ? x[k + o] : x[k];
                                x[k] = keep + __shfl_xor_sync(kFull, send, o);
                            }
                        x[0] += __shfl_xor_sync(kFull, x[0], 8);
                        x[0] += __shfl_xor_sync(kFull, x[0], 16);
                        if (lane < 8)
                            scratch[(warp & 3) * NT + 8 * i + lane] = x[0];
                    }
                    float* const fin = scratch + 4 * NT;
                    if (!cta_wait(sh, &sh.info_full[items & 1], (items >> 1) & 1))
                        gt |= kGaveUp;
                    bar_sync(bar, 128);
                    const bool bad = info.bad;
                    float l = 0.0f;
                    if (t < NT) {
                        const unsigned anc = info.anc[w * NT + t];
                        l = (scratch[t] + scratch[NT + t]) + (scratch[2 * NT + t] + scratch[3 * NT + t]);
                        if (bad || (anc & info.poison))
                            l = NAN;
                        // (anc == 0: no node's row.  A node's sum is zero only where all its scores are -inf: NaN)
                        fin[t] = anc == 0 ? 0.0f : __fdividef(1.0f, l);
                    }
                    if (!cta_wait(sh, &sh.o_full, (gt - 1) & 1))
                        gt |= kGaveUp;
                    tc_fence_after();
                    // After a wait that gave up, the item's last one among them, nothing of the item can be relied on: its
                    // rows are written as NaN below, and reported when the CTA ends.
                    const bool abort = bar_any(bar, 128, *reinterpret_cast<volatile uint32_t*>(&sh.limit) == 0);
                    if (tid == 0 && bad && !abort && a.has_err)
                        atomicOr(a.err, kErrCache);
                    lost |= abort;
                    if (t < NT && !whole && !abort) {
                        const int at = info.row_out[w * NT + t];
                        if (at >= 0)
                            reinterpret_cast<float2*>(a.part_ml)[at] = make_float2(-negm[t], l);
                    }
#pragma unroll 1
                    for (int c = 0; c < a.nd && !abort; ++c) {
                        const int d = 128 * c + t;
                        const int* const row_out = info.row_out + w * NT;
                        if (whole)
                            store_rows<NT>(tmem_o + c * N, row_out, fin, d, D, [&](int at, float x, float f) {
                                a.out[(long long)at * D + d] = __float2bfloat16_rn(f == 0.0f ? 0.0f : x * f);
                            });
                        else
                            store_rows<NT>(tmem_o + c * N, row_out, fin, d, D, [&](int at, float x, float) { a.part_o[(long long)at * D + d] = x; });
                    }
                    tc_fence_before();
                    bar_sync(bar, 128);   // O, the scratch and the item's rows have been read
                    if (lane == 0 && gt < kGaveUp)
                        mbar_arrive(smem_addr(&sh.info_empty[items & 1]));
                    ++items;
                }
                if (run.s.len == 0 || lost) {
                    // no position: zeros; unusable lengths, or a wait that gave up: NaN
                    if (!run.s.ok && tid == 0 && a.has_err)
                        atomicOr(a.err, kErrCache);
#pragma unroll 1
                    for (int r = w * NT + (warp & 3); r < min(a.rows, (w + 1) * NT); r += 4) {
                        int node, head;
                        if (!attn_row(a, run.g, r, node, head))
                            continue;
                        if (!whole && lane < 2)
                            a.part_ml[((long long)part * a.rows + r) * 2 + lane] = NAN;
#pragma unroll 1
                        for (int d = lane; whole && d < D; d += 32)
                            a.out[(((long long)run.b * a.Nmax + node) * a.Hq + h * a.G + head) * D + d] =
                                __float2bfloat16_rn(node < nn && lost ? NAN : 0.0f);
                    }
                }
            }
        }
    } else if (warp >= 12) {
        regs_shrink<kRegsTiles<NT>>();
        // --- tiles: a quarter of the positions a warp ----------------------------------
        const AttnLayout L = attn_layout<N, E4M3>(a, smem);
        AttnShared& sh = *L.sh;
        const int quarter = warp & 3, t = tid - 384, key = t & 7;
        // how far keys and values are asked for ahead of the tile that the loop is at: a slot less than there
        // are, so that the one to be refilled is likely free
        const int k_ahead = max(1, a.kslots / a.nd - 1), v_ahead = max(1, a.vslots / a.nd - 1);
        Tiles k, v;
        k.start(a, run_of(sh));
        v = k;
        Ring rk, rv;
        uint32_t fills_k = 0, fills_v = 0;   // slots asked for (bf16)
        Boxes box_k, box_v;
        box_k.ask(a, k, quarter * kQuarter, kQuarter, lane);
        box_v = box_k;
        auto load_k = [&]() {
            const int now = box_k.row(a);
            k.step(a);
            box_k.ask(a, k, quarter * kQuarter, kQuarter, lane);   // on its way while this tile is asked for
#pragma unroll 1
            for (int c = 0; c < a.nd; ++c) {
                if (!cta_wait(sh, &sh.kempty[rk.slot], rk.phase ^ 1))
                    return false;
                load_boxes<E4M3>(a, smem_addr(L.k) + rk.slot * a.k_bytes + quarter * kQuarter * 128, smem_addr(&sh.kfull[rk.slot]), &map_k, c, now, lane);
                rk.step(a.kslots);
                ++fills_k;
            }
            return true;
        };
        auto load_v = [&]() {
            const int now = box_v.row(a);
            v.step(a);
            box_v.ask(a, v, quarter * kQuarter, kQuarter, lane);
#pragma unroll 1
            for (int c = 0; c < a.nd; ++c) {
                if (!cta_wait(sh, &sh.vempty[rv.slot], rv.phase ^ 1))
                    return false;
                load_boxes<E4M3>(a, smem_addr(L.v) + rv.slot * a.v_bytes + quarter * kQuarter * 128,
                                 smem_addr(&sh.vfull[rv.slot]), &map_v, c, now, lane);
                rv.step(a.vslots);
                ++fills_v;
            }
            return true;
        };
        bool go = true;
        Tiles it;
        it.start(a, run_of(sh));
        uint32_t items = 0;
        Ring r, w;
        // an item's queries, as three 8-bit terms (before its keys' first product): a thread takes one 8-element
        // chunk of every `stride`th row
        const int per = D / 8, stride = 128 / per, row0 = t / per, ch = t - row0 * per;
        auto queries = [&](const Run& x) {
            const int nb = x.g / a.head_blocks, node0 = nb * a.nodes, head0 = (x.g - nb * a.head_blocks) * a.heads;
            const int live = min(a.nodes, x.s.nn - node0), heads = min(a.heads, a.G - head0);
            const uint4* const q = reinterpret_cast<const uint4*>(a.q + ((long long)x.b * a.Nmax + node0) * a.q_stride +
                                                                  (long long)(x.h * a.G + head0) * D) + ch;
            // kRows rows a thread at a time (which is all of up to 64, or 32, rows of 128 elements), zeros where there is
            // no query
            constexpr int kRows = NT >= 64 ? 4 : 8;
            const int turn = kRows * stride;
            uint4 y[kRows];
            auto load_q = [&](int row) {
                int n = row / a.heads, head = row - n * a.heads;
#pragma unroll
                for (int k = 0; k < kRows; ++k) {
                    y[k] = n < live && head < heads && row0 < stride ? __ldg(q + n * (a.q_stride / 8) + head * per) : make_uint4(0, 0, 0, 0);
                    for (head += stride; head >= a.heads; head -= a.heads)
                        ++n;
                }
            };
            // the largest magnitude of eight elements (magnitudes order as integers; what is not finite does not count)
            auto largest = [](uint4 x) {
                const uint32_t z[4] = {x.x, x.y, x.z, x.w};
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t lo = (z[e] << 16) & 0x7fff0000u, hi = z[e] & 0x7fff0000u;
                    m = max(m, max(lo < 0x7f800000u ? lo : 0u, hi < 0x7f800000u ? hi : 0u));
                }
                return m;
            };
            // the exponent of the power of two that brings it to [128, 256)
            auto raise = [](uint32_t m) { return m ? min(max(261 - (int)(m >> 23), 1), 253) : 127; };
            // One power of two for the group; where some eight elements lie 2^8 below its largest (which ordinary
            // queries do not) one for each row, as the terms hold 2^-25 of the largest element that they share it with.
            uint32_t top = 0, low = ~0u;
            bool spread = false;
#pragma unroll 1
            for (;;) {   // (a second pass where spread: one place in the code for both)
#pragma unroll 1
                for (int row = row0; row < a.rows; row += turn) {
                    load_q(row);
#pragma unroll
                    for (int k = 0; k < kRows; ++k) {
                        const uint32_t m = largest(y[k]);
                        top = max(top, m);
                        low = min(low, m - 1u);   // (zeros do not count)
                        if (spread && m)          // (zeros where there is no query)
                            atomicMax(&sh.row_top[row + k * stride], m);
                    }
                }
                if (spread)
                    break;
                top = __reduce_max_sync(kFull, top);
                low = __reduce_min_sync(kFull, low);
                if (lane == 0) {
                    sh.top[warp & 3] = top;
                    sh.low[warp & 3] = low;
                }
                sh.row_top[t] = 0;
                bar_sync(3, 128);
                top = max(max(sh.top[0], sh.top[1]), max(sh.top[2], sh.top[3]));
                low = min(min(sh.low[0], sh.low[1]), min(sh.low[2], sh.low[3]));
                spread = top > (8u << 23) && low < top - (8u << 23);
                if (!spread)
                    break;
            }
            if (spread)
                bar_sync(3, 128);
            const int e = raise(top);
            const float group_scale = __uint_as_float((uint32_t)e << 23);
            auto row_exponent = [&](int row) { return sh.row_top[row] ? min(raise(sh.row_top[row]), e + 126) : e; };
            go = go && cta_wait(sh, &sh.q_empty, (items & 1) ^ 1);
            if (t == 0) {
                sh.q_unscale[items & 3] = __uint_as_float((uint32_t)(254 - e) << 23);
                sh.q_spread[items & 3] = spread;
            }
            if (spread)
                sh.q_row[items & 3][t] = __uint_as_float((uint32_t)(127 + e - row_exponent(t)) << 23);
#pragma unroll 1
            for (int row = row0; go && row < a.rows; row += turn) {
                if (a.rows > turn)
                    load_q(row);
#pragma unroll 1
                for (int k = 0; k < kRows; ++k) {
                    const int at = row + k * stride;
                    if (at >= a.rows || row0 >= stride)
                        break;
                    float scale = group_scale;
                    if (spread)
                        scale = __uint_as_float((uint32_t)row_exponent(at) << 23);
                    float z[8];
                    Elem<__nv_bfloat16>::unpack(y[0], z);
                    uint32_t p[3][4];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        split_q(z[2 * c] * scale, z[2 * c + 1] * scale, p[0][c], p[1][c], p[2][c]);
                    unsigned char* o = L.q + (ch >> 4) * (N * 128) + at * 128 + ((((ch & 15) >> 1) ^ (at & 7)) << 4) + (ch & 1) * 8;
#pragma unroll
                    for (int c = 0; c < 3; ++c)
                        *reinterpret_cast<uint2*>(o + c * L.q_part) = make_uint2(p[c][0] | (p[c][1] << 16), p[c][2] | (p[c][3] << 16));
#pragma unroll
                    for (int c = 0; c < kRows - 1; ++c)   // (rolled, the code being long: the next one to the front)
                        y[c] = y[c + 1];
                }
            }
            fence_proxy_async();
            go = !bar_any(3, 128, !go);   // (also: sh.top may be written again)
            if (t == 0 && go)
                mbar_arrive(smem_addr(&sh.q_full));
            ++items;
        };
        // step g asks for tile g + k_ahead of the keys and g + v_ahead of the values (bf16), or converts the values of
        // tile g (e4m3)
#pragma unroll 1
        for (int g = -max(k_ahead, v_ahead); E4M3 ? it.more : go && (k.more || v.more); ++g) {
            // (e4m3: the warps share a barrier: after a timeout they all run on, doing nothing)
            if (!E4M3 && go && k.more && g >= -k_ahead)
                go = load_k();
            if (E4M3 && (g == -1 || (g >= 0 && it.j == it.run.t1 - 1))) {
                // the first item's queries; the next one's, before this one's last values
                Run x = it.run;
                if (g == -1 || x.next(a))
                    queries(x);
            }
            if (E4M3 && g >= 0) {
                const int valid = it.valid(), rows = (valid + 15) & ~15;
                const int node0 = it.run.s.nn > 1 ? it.run.s.ctx - it.j * kTile : kTile;   // first row of a node
#pragma unroll 1
                for (int c = 0; c < a.nd; ++c) {
                    go = go && cta_wait(sh, &sh.vfull[r.slot], r.phase) && cta_wait(sh, &sh.cempty[w.slot], w.phase ^ 1);
                    const unsigned char* src = L.v + r.slot * a.v_bytes + t * 128;
                    unsigned char* dst = L.c + w.slot * a.conv_bytes + t * 128;
                    const int pieces = min(128, D - 128 * c) / 16;
                    if (go && t < rows) {
#pragma unroll 1
                        for (int i = 0; i < pieces; i += 4) {
                            // four 16-byte pieces at a time, so that their chains overlap (what is past the row is not used)
                            uint4 x[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                x[k] = t < valid ? *reinterpret_cast<const uint4*>(src + (((i + k) ^ key) << 4)) : make_uint4(0, 0, 0, 0);
                            if (t >= node0) {   // a node's values are seen by some rows only (which end as NaN)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    if (chunk_nan_e4m3(x[k]))
                                        x[k] = make_uint4(0, 0, 0, 0);
                            }
                            unsigned char* o = dst + (i >> 2) * kHalfBytes;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint2 y0 = e4m3_to_f16(x[k].x), y1 = e4m3_to_f16(x[k].y), y2 = e4m3_to_f16(x[k].z), y3 = e4m3_to_f16(x[k].w);
                                *reinterpret_cast<uint4*>(o + (((2 * k) ^ key) << 4)) = make_uint4(y0.x, y0.y, y1.x, y1.y);
                                *reinterpret_cast<uint4*>(o + (((2 * k + 1) ^ key) << 4)) = make_uint4(y2.x, y2.y, y3.x, y3.y);
                            }
                        }
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0 && go) {
                        mbar_arrive(smem_addr(&sh.vempty[r.slot]));
                        mbar_arrive(smem_addr(&sh.cfull[w.slot]));
                    }
                    r.step(a.vslots);
                    w.step(a.conv);
                }
                it.step(a);
            }
            if (!E4M3 && go && v.more && g >= -v_ahead)
                go = load_v();
        }
        if (!E4M3) {
            // A warp that gave up before the others has not arrived for slots whose copies they have on their way: it
            // does so now, with no bytes of its own (a warp is behind by at most the ring, so these are the slots'
            // current phases), and all wait for the last copies of each slot.
            if (lane == 0) {
                sh.fills[0][quarter] = fills_k;
                sh.fills[1][quarter] = fills_v;
            }
            bar_sync(3, 128);
            const uint32_t most_k = max(max(sh.fills[0][0], sh.fills[0][1]), max(sh.fills[0][2], sh.fills[0][3]));
            const uint32_t most_v = max(max(sh.fills[1][0], sh.fills[1][1]), max(sh.fills[1][2], sh.fills[1][3]));
#pragma unroll 1
            for (; fills_k < most_k; ++fills_k, rk.step(a.kslots))
                if (lane == 0)
                    mbar_arrive(smem_addr(&sh.kfull[rk.slot]));
#pragma unroll 1
            for (; fills_v < most_v; ++fills_v, rv.step(a.vslots))
                if (lane == 0)
                    mbar_arrive(smem_addr(&sh.vfull[rv.slot]));
            drain_ring(sh, sh.kfull, rk, a.kslots, fills_k, t == 0 && ((a.hold >> kKFull) & 1));
            drain_ring(sh, sh.vfull, rv, a.vslots, fills_v, t == 0 && ((a.hold >> kVFull) & 1));
        }
    } else {
        regs_shrink<kRegsIssue<NT>>();
        const AttnLayout L = attn_layout<N, E4M3>(a, smem);
        AttnShared& sh = *L.sh;
        if (warp == 9) {
            // --- bf16 queries; e4m3 keys ----------------------------------------------------
            Run run = run_of(sh);
            uint32_t items = 0;
            bool go = true;
#pragma unroll 1
            while (!E4M3 && run.next(a)) {
                go = cta_wait(sh, &sh.q_empty, (items & 1) ^ 1);
                if (!go)
                    break;
                ++items;
                if (lane == 0) {
                    const int nb = run.g / a.head_blocks;
                    mbar_arrive_expect_tx(smem_addr(&sh.q_full), a.rows * 128 * ((D + 63) / 64));
#pragma unroll 1
                    for (int c = 0; c < (D + 63) / 64; ++c)
                        tma_load_3d(smem_addr(L.q) + c * (N * 128), &map_q, 64 * c, run.h * a.G + (run.g - nb * a.head_blocks) * a.heads,
                                    run.b * a.Nmax + nb * a.nodes, smem_addr(&sh.q_full));
                }
                __syncwarp();
            }
            if (items) {
                if (lane == 0 && ((a.hold >> kQFull) & 1))
                    make_up(sh, &sh.q_full);
                drain_wait(&sh.q_full, (items - 1) & 1);
            }
            if (E4M3) {
                Tiles k;
                Ring rk;
                Boxes box;
                uint32_t fills = 0;
                k.start(a, run);
                box.ask(a, k, 0, kTile, lane);
#pragma unroll 1
                while (go && k.more) {
                    const int now = box.row(a);
                    k.step(a);
                    box.ask(a, k, 0, kTile, lane);   // on its way while this tile is asked for
#pragma unroll 1
                    for (int c = 0; go && c < a.nd; ++c) {
                        go = cta_wait(sh, &sh.kempty[rk.slot], rk.phase ^ 1);
                        if (!go)
                            break;
                        load_boxes<E4M3>(a, smem_addr(L.k) + rk.slot * a.k_bytes, smem_addr(&sh.kfull[rk.slot]), &map_k, c, now, lane);
                        rk.step(a.kslots);
                        ++fills;
                    }
                }
                drain_ring(sh, sh.kfull, rk, a.kslots, fills, lane == 0 && ((a.hold >> kKFull) & 1));
            }
        } else if (warp == 8) {
            // --- first product -----------------------------------------------------------
            const uint32_t tmem = sh.tmem, k0 = smem_addr(L.k), q0 = smem_addr(L.q);
            Ring rk;
            uint32_t g = 0, items = 0;   // tiles, items so far
            Tiles k;
            bool go = true, issued = false;
            for (k.start(a, run_of(sh)); k.more; k.step(a), ++g) {
                if (k.j == k.run.t0)
                    go = cta_wait(sh, &sh.q_full, items++ & 1);
                go = go && cta_wait(sh, &sh.s_empty[g & 1], ((g >> 1) & 1) ^ 1);
#pragma unroll 1
                for (int c = 0; go && c < a.nd; ++c) {
                    const int width = min(128, D - 128 * c);
                    go = cta_wait(sh, &sh.kfull[rk.slot], rk.phase);
                    if (!go)
                        break;
                    tc_fence_after();
                    if (lane == 0) {
                        mma_scores<N, E4M3>(tmem + (g & 1) * N, k0 + rk.slot * a.k_bytes, q0 + (E4M3 ? c : 2 * c) * (N * 128), L.q_part,
                                            E4M3 ? (width + 31) / 32 : width / 16, c > 0);
                        tc_commit(smem_addr(&sh.kempty[rk.slot]));
                        if (c == a.nd - 1) {
                            tc_commit(smem_addr(&sh.s_full[g & 1]));
                            if (k.j == k.run.t1 - 1)
                                tc_commit(smem_addr(&sh.q_empty));
                        }
                    }
                    __syncwarp();
                    issued = true;
                    rk.step(a.kslots);
                }
                if (!go)
                    break;
            }
            if (issued) {   // products in flight end before the CTA's memory is given back
                if (lane == 0)
                    tc_commit(smem_addr(&sh.drain[0]));
                __syncwarp();
                drain_wait(&sh.drain[0], 0);
            }
        } else if (warp == 10) {
            // --- second product ----------------------------------------------------------
            const uint32_t tmem_o = sh.tmem + 2 * N, p0 = smem_addr(L.p);
            const int ring = E4M3 ? a.conv : a.vslots;
            const uint32_t v0 = smem_addr(E4M3 ? L.c : L.v), v_bytes = E4M3 ? a.conv_bytes : a.v_bytes;
            uint64_t* const full = E4M3 ? sh.cfull : sh.vfull;
            uint64_t* const empty = E4M3 ? sh.cempty : sh.vempty;
            Ring rv;
            uint32_t g = 0, items = 0;
            Tiles v;
            bool go = true;
            bool issued = false;
            for (v.start(a, run_of(sh)); v.more; ++g) {
                const int valid = v.valid(), ksteps = (valid + 15) / 16;
                const bool tail = (v.j + 1) * kTile > v.run.s.ctx;
#pragma unroll 1
                for (int c = 0; go && c < a.nd; ++c) {
                    const int width = min(128, D - 128 * c);
                    go = cta_wait(sh, &full[rv.slot], rv.phase);
                    if (!go)
                        break;
                    if (!E4M3 && tail) {
                        // rows behind the last position may hold anything: zeros instead of 0 * NaN.  A node's
                        // values are seen by some rows only: what is not finite there is zeroed too (the rows
                        // that do see it are set to NaN at the end).
                        unsigned char* x = L.v + rv.slot * a.v_bytes;
                        const int chunks = width > 64 ? 16 : 8;
#pragma unroll 1
                        for (int i = valid * chunks + lane; i < ksteps * 16 * chunks; i += 32) {
                            const int row = i / chunks, ch = i % chunks;
                            *reinterpret_cast<uint4*>(x + (ch >> 3) * kHalfBytes + row * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        go = cta_wait(sh, &sh.info_full[items & 1], (items >> 1) & 1);
                        if (!go)
                            break;
                        const int row = v.run.s.ctx + lane - v.j * kTile;
                        if (((sh.info[items & 1].poison >> lane) & 1u) && row >= 0 && row < kTile)
#pragma unroll 1
                            for (int ch = 0; ch < chunks; ++ch) {
                                uint4* p = reinterpret_cast<uint4*>(x + (ch >> 3) * kHalfBytes + row * 128 + ((ch ^ lane) & 7) * 16);
                                if (chunk_nonfinite(*p, false))
                                    *p = make_uint4(0, 0, 0, 0);
                            }
                        fence_proxy_async();
                        __syncwarp();
                    }
                    if (c == 0) {
                        go = cta_wait(sh, &sh.p_full, g & 1);
                        if (!go)
                            break;
                    }
                    tc_fence_after();
                    if (lane == 0) {
                        mma_values<N, E4M3>(tmem_o + c * N, v0 + rv.slot * v_bytes, p0, width > 64 ? kHalfBytes : 0, ksteps, v.j > v.run.t0);
                        if (c == a.nd - 1)
                            tc_commit(smem_addr(&sh.o_full));
                        tc_commit(smem_addr(&empty[rv.slot]));
                    }
                    __syncwarp();
                    issued = true;
                    rv.step(ring);
                }
                if (!go)
                    break;
                if (v.j == v.run.t1 - 1)
                    ++items;
                v.step(a);
            }
            if (issued) {
                if (lane == 0)
                    tc_commit(smem_addr(&sh.drain[1]));
                __syncwarp();
                drain_wait(&sh.drain[1], 0);
            }
        } else {
            // --- an item's rows; e4m3 values -------------------------------------------------
            Run run = run_of(sh);   // the item to prepare next
            uint32_t items = 0;
            Tiles v;
            Ring rv;
            Boxes box;
            uint32_t fills = 0;
            v.start(a, run);
            if (E4M3)
                box.ask(a, v, 0, kTile, lane);
            bool go = true, busy = true;
            int owed = 1;   // items to prepare: the first, and the next one whenever an item's last values are asked for
#pragma unroll 1
            while (go && busy) {
                busy = false;
                if (E4M3 && v.more) {   // (bf16 values are loaded elsewhere)
                    busy = true;
                    owed += v.j == v.run.t1 - 1;
                    const int now = box.row(a);
                    v.step(a);
                    box.ask(a, v, 0, kTile, lane);   // on its way while this tile is asked for
#pragma unroll 1
                    for (int c = 0; go && c < a.nd; ++c) {
                        go = cta_wait(sh, &sh.vempty[rv.slot], rv.phase ^ 1);
                        if (!go)
                            break;
                        load_boxes<E4M3>(a, smem_addr(L.v) + rv.slot * a.v_bytes, smem_addr(&sh.vfull[rv.slot]), &map_v, c, now, lane);
                        rv.step(a.vslots);
                        ++fills;
                    }
                }
                if (go && (owed > 0 || !E4M3) && run.next(a)) {
                    busy = true;
                    go = prepare_item<N, E4M3>(a, sh, run, items++, lane);
                    --owed;
                }
            }
            drain_ring(sh, sh.vfull, rv, a.vslots, fills, lane == 0 && ((a.hold >> kVFull) & 1));
        }
    }
    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const AttnShared& sh = *attn_layout<N, E4M3>(a, smem).sh;
    if (warp == 8)
        tmem_free(sh.tmem, 512);
    if (tid == 0 && a.has_err && *reinterpret_cast<const volatile uint32_t*>(&sh.limit) == 0)
        atomicOr(a.err, kErrWaitTimeout);
}

// Items cut between CTAs: CTA i's last item, if it does not end it, is joined
// with the parts of the CTAs that go on with it.  A warp takes one row, a lane
// four elements at a time; what bounds it is latency (meta, sums, parts), so
// four parts' loads are in flight at once.
__global__ void __launch_bounds__(256) sv_attention_combine(const __grid_constant__ AttnArgs a, int ctas)
{
    const int i = blockIdx.x, lane = threadIdx.x & 31, D = a.c.D;
    const int row = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
    pdl_wait();
    const int item = a.meta[2 * i];
    if (item < 0 || row >= a.rows)
        return;
    int n = 1;
    for (;;) {   // parts: a ballot of the following CTAs that continue this item
        const int at = i + n + lane;
        const unsigned same = __ballot_sync(kFull, at < ctas && a.meta[2 * min(at, ctas - 1) + 1] == item);
        const int more = same == kFull ? 32 : __ffs(~same) - 1;
        n += more;
        if (more < 32)
            break;
    }
    // part p: CTA i's begun slot, then the continued slots of CTAs i + 1 ...
    auto slot = [&](int p) { return (p == 0 ? 2LL * i + 1 : 2LL * (i + p)) * a.rows + row; };
    auto sums = [&](int p) {
        return p < n ? reinterpret_cast<const float2*>(a.part_ml)[slot(p)] : make_float2(-INFINITY, 0.0f);
    };
    const float2 mine = sums(lane);   // of the first 32 parts
    float m = -INFINITY;
    for (int p = lane; p < n; p += 32) {
        const float2 x = p < 32 ? mine : sums(p);
        if (x.y != 0.0f)
            m = fmaxf(m, x.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    float l = 0.0f, acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        acc[e] = 0.0f;
    const int quads = D / 4;
    for (int p0 = 0; p0 < n; p0 += 32) {
        const float2 x = p0 == 0 ? mine : sums(p0 + lane);
        const float wgt = x.y == 0.0f ? 0.0f : ex2_approx(x.x - m);
        float wl = wgt * x.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            wl += __shfl_xor_sync(kFull, wl, o);
        l += wl;
        const int end = min(n - p0, 32);
        for (int p = 0; p < end; p += 4) {
            float4 y[4][2];
            float wp[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                wp[k] = __shfl_sync(kFull, wgt, (p + k) & 31);
                const float4* o = reinterpret_cast<const float4*>(a.part_o + slot(p0 + p + k) * D);
#pragma unroll
                for (int e = 0; e < 2; ++e)   // (a part without weight may hold what no product has written)
                    y[k][e] = p + k < end && wp[k] != 0.0f && lane + 32 * e < quads ? o[lane + 32 * e] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float w = p + k < end ? wp[k] : 0.0f;
                    acc[4 * e] = fmaf(w, y[k][e].x, acc[4 * e]);
                    acc[4 * e + 1] = fmaf(w, y[k][e].y, acc[4 * e + 1]);
                    acc[4 * e + 2] = fmaf(w, y[k][e].z, acc[4 * e + 2]);
                    acc[4 * e + 3] = fmaf(w, y[k][e].w, acc[4 * e + 3]);
                }
        }
    }
    const int per = a.c.Hkv * a.groups, b = item / per, h = (item - b * per) / a.groups, g = item - (b * a.c.Hkv + h) * a.groups;
    int node, head;
    if (!attn_row(a, g, row, node, head))
        return;
    const int nn = a.has_n ? __ldg(a.n_nodes + b) : a.Nmax;   // (an item of unusable lengths is never cut)
    __nv_bfloat16* out = a.out + (((long long)b * a.Nmax + node) * a.Hq + h * a.G + head) * D;
    const float inv = 1.0f / l;   // (zero only where all of a node's scores are -inf: NaN)
#pragma unroll
    for (int e = 0; e < 2; ++e)
        if (lane + 32 * e < quads) {
            reinterpret_cast<uint2*>(out)[lane + 32 * e] =
                node < nn ? make_uint2(bf16_pair(acc[4 * e] * inv, acc[4 * e + 1] * inv), bf16_pair(acc[4 * e + 2] * inv, acc[4 * e + 3] * inv))
                          : make_uint2(0, 0);
        }
}

}  // namespace sv
