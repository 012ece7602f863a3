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
// A thread of the softmax then owns one position of a tile and every row: the
// e4m3 cache's scales are one multiplier a thread, the exponentials cost what
// the rows cost (no padding to 128), and the tree mask is one bit a row.  The
// price is that a row's maximum runs across threads; it is kept lazily: the
// weights are relative to a running reference that moves only when some score
// exceeds it by more than 2^8 (a vote a tile), so the cross-thread maximum and
// the rescaling of O are rare.
//
// Work is (sequence, key head, row group) items of 128-position tiles, laid
// end to end and cut into equal runs, one to a CTA.  An item cut by a run's
// end leaves partial sums in the workspace, which sv_attention_combine joins.
#pragma once

#include "sv_kv.cuh"
#include "sv_tcgen05.cuh"

namespace sv {

constexpr int kAttnMaxCtas = 160;
constexpr int kTile = 128;                 // positions a tile
constexpr int kRowsMax = 128;              // query rows a CTA
constexpr int kHalfBytes = kTile * 128;    // 128 rows of 64 bf16 elements
constexpr float kLazy = 8.0f;              // log2 of the largest weight before the reference moves
constexpr int kMaxSlots = 12, kMaxConv = 4;

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
    int groups, rows;        // row groups of a key head; rows of one group
    int half;                // rows of the first warpgroup (the second has the rest)
    int nd;                  // 128-wide chunks of head_dim
    int slots, conv;         // ring sizes
    int slot_bytes, conv_bytes;
    int box_rows;            // rows of one TMA box (a page, or a tile)
    int raw_pitch, raw_swizzled;
    float scale_log2;        // scale * log2(e)
};

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

// A CTA's run of tiles, an item (or a part of one) at a time.
struct Run {
    long long left;
    int b, hg, tile;
    SeqLens s;
    // the current part
    int t0, t1;

    __device__ __forceinline__ bool next(const AttnArgs& a)
    {
        if (left <= 0)
            return false;
        if (tile == s.tiles) {
            tile = 0;
            if (++hg == a.c.Hkv * a.groups) {
                hg = 0;
                s = seq_lens(a, ++b);
            }
        }
        t0 = tile;
        t1 = (int)min((long long)s.tiles, t0 + left);
        left -= t1 - t0;
        tile = t1;
        return true;
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == s.tiles; }
};

struct AttnShared {
    uint64_t full[kMaxSlots], empty[kMaxSlots];    // TMA slots
    uint64_t cfull[kMaxConv], cempty[kMaxConv];    // converted slots (e4m3)
    uint64_t q_full[2], s_full[2][2], s_empty[2][2], p_full[2], o_full[2];
    uint64_t drain;
    uint32_t tmem;
    int abort;
    long long t_begin, t_end, sum[14];
    int b, hg, tile, active;
    unsigned poison[2];
    int unset[2];
    alignas(16) float negm[2][64];                 // minus the rows' references
    unsigned anc[2][64];                           // the rows' ancestor bits
};

// A wait that ends: on a timeout every later wait of the CTA gives up too.
// The warps that own named barriers run on regardless (they all reach the
// same ones), the others stop.
__device__ __forceinline__ bool cta_wait(AttnShared& sh, uint64_t* bar, uint32_t parity)
{
    const uint32_t addr = smem_addr(bar);
    for (uint32_t i = 0; i < kWaitSpins; ++i) {
        if (mbar_try_wait(addr, parity))
            return true;
        if ((i & 15) == 15 && *reinterpret_cast<volatile int*>(&sh.abort))
            return false;
    }
    *reinterpret_cast<volatile int*>(&sh.abort) = 1;
    return false;
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
};

// e4m3 bytes to bf16, exactly: the eight bits' exponent and mantissa fields
// land in the bf16's low exponent and high mantissa bits, which is the value
// times 2^-120 (subnormals included); one multiplication restores it.
__device__ __forceinline__ uint32_t bf16x2_scale(uint32_t x)
{
    uint32_t y;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0x7b807b80u));   // 2^120
    return y;
}

// Four e4m3 values as four bf16 in order.
__device__ __forceinline__ uint2 e4m3_to_bf16(uint32_t w)
{
    // bytes 0 and 2 / 1 and 3 in the high bytes of 16-bit lanes
    const uint32_t e = w << 8, s = 0x80008000u, m = 0x07f007f0u;
    const uint32_t even = bf16x2_scale((e & s) | ((e & 0x7f007f00u) >> 4));   // v0, v2
    const uint32_t odd = bf16x2_scale((w & s) | ((w >> 4) & m));              // v1, v3
    return make_uint2(__byte_perm(even, odd, 0x5410), __byte_perm(even, odd, 0x7632));
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

// NaN for the NaN bytes of w, which e4m3_to_bf16 reads as 480.
__device__ __noinline__ uint2 e4m3_keep_nan(uint32_t w, uint2 y)
{
    const uint32_t m = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    y.x |= ((m >> 7) & 1u) * 0x7fffu | ((m >> 15) & 1u) * 0x7fff0000u;
    y.y |= ((m >> 23) & 1u) * 0x7fffu | (m >> 31) * 0x7fff0000u;
    return y;
}

__device__ __forceinline__ bool chunk_nonfinite(uint4 w, bool e4m3)
{
    return e4m3 ? chunk_nan_e4m3(w)
                : bf16_pair_nonfinite(w.x) || bf16_pair_nonfinite(w.y) || bf16_pair_nonfinite(w.z) || bf16_pair_nonfinite(w.w);
}

// NT: rows (TMEM columns) a softmax warpgroup handles; E4M3: four more warps
// convert the cache's bytes to bf16 operands.
template <int NT, bool E4M3>
__global__ void __launch_bounds__(E4M3 ? 448 : 320, 1)
    sv_attention_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v)
{
    constexpr int kThreads = E4M3 ? 448 : 320, kWarps = kThreads / 32;
    extern __shared__ __align__(1024) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, D = a.c.D;
    const int nwg = a.rows > 16 ? 2 : 1;
    // layout: operand slots, P, Q, the small things
    unsigned char* s_raw = smem;                                                    // a.slots * a.slot_bytes
    unsigned char* s_conv = s_raw + (E4M3 ? a.conv * a.conv_bytes : 0);             // e4m3: conv slots first
    if (E4M3) {
        unsigned char* t = s_raw;
        s_raw = s_conv;
        s_conv = t;
    }
    unsigned char* s_p = s_raw + a.slots * a.slot_bytes;
    const int q_bytes = NT * 128 * ((D + 63) / 64);
    unsigned char* s_q = s_p + nwg * kHalfBytes;
    AttnShared& sh = *reinterpret_cast<AttnShared*>(s_q + nwg * q_bytes);

    // --- the CTA's run of tiles --------------------------------------------
    if (warp == 8) {
        tmem_alloc(smem_addr(&sh.tmem), 512);
    } else if (tid == 9 * 32) {
        sh.abort = 0;
        for (int i = 0; i < a.slots; ++i) {
            mbar_init(smem_addr(&sh.full[i]), 1);
            mbar_init(smem_addr(&sh.empty[i]), E4M3 ? 4 : 1);
        }
        for (int i = 0; i < a.conv; ++i) {
            mbar_init(smem_addr(&sh.cfull[i]), 4);
            mbar_init(smem_addr(&sh.cempty[i]), 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(smem_addr(&sh.q_full[w]), 4);
            mbar_init(smem_addr(&sh.p_full[w]), 4);
            mbar_init(smem_addr(&sh.o_full[w]), 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_addr(&sh.s_full[w][i]), 1);
                mbar_init(smem_addr(&sh.s_empty[w][i]), 4);
            }
        }
        mbar_init(smem_addr(&sh.drain), 1);
        fence_mbar_init();
        tma_prefetch_map(&map_k);
        tma_prefetch_map(&map_v);
    }
    {
        // tiles of all sequences before each thread's share of them
        const int share = (a.B + kThreads - 1) / kThreads, b0 = min(tid * share, a.B), b1 = min(b0 + share, a.B);
        const int per = a.c.Hkv * a.groups;
        long long mine = 0;
        for (int b = b0; b < b1; ++b)
            mine += (long long)seq_lens(a, b).tiles * per;
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
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp)
                before += sh.sum[w];
            total += sh.sum[w];
        }
        const long long excl = before + incl - mine;
        const int act = (int)min((long long)gridDim.x, total), i = blockIdx.x;
        const long long begin = total * i / act, end = total * (i + 1) / act;
        if (i < act && begin >= excl && begin < excl + mine) {
            long long at = excl;
            int b = b0;
            for (;; ++b) {
                const long long n = (long long)seq_lens(a, b).tiles * per;
                if (begin < at + n)
                    break;
                at += n;
            }
            const int tiles = seq_lens(a, b).tiles;
            sh.b = b;
            sh.hg = (int)((begin - at) / tiles);
            sh.tile = (int)((begin - at) % tiles);
            sh.t_begin = begin;
            sh.t_end = end;
        }
        if (tid == 0) {
            sh.active = i < act;
            a.meta[2 * i] = a.meta[2 * i + 1] = -1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    Run run;
    run.left = 0;
    run.tile = 0;
    run.s.tiles = -1;
    if (sh.active) {
        run.left = sh.t_end - sh.t_begin;
        run.b = sh.b;
        run.hg = sh.hg;
        run.tile = sh.tile;
        run.s = seq_lens(a, run.b);
    }
    const uint32_t ring_full = smem_addr(sh.full), ring_empty = smem_addr(sh.empty);

    if (warp == 9) {
        // --- TMA producer ----------------------------------------------------
        // Slots are filled in the order the products take them: K(0), then
        // K(j + 1), V(j) for every tile j.
        Ring r;
        int issued = 0;
        const int boxes = kTile / a.box_rows;
        bool go = true;
        while (go && run.next(a)) {
            if (run.s.len == 0)
                continue;
            const int h = run.hg / a.groups;
            for (int step = 0; go && step < 2 * (run.t1 - run.t0); ++step) {
                // steps: K0, K1, V0, K2, V1, ..., K(n-1), V(n-2), V(n-1)
                const int n = run.t1 - run.t0;
                const bool is_k = step == 0 || ((step & 1) && (step + 1) / 2 < n);
                const int j = run.t0 + (step == 0 ? 0 : is_k ? (step + 1) / 2 : step == 2 * n - 1 ? n - 1 : step / 2 - 1);
                const int valid = min(kTile, run.s.len - j * kTile);
                // lane l: the tile's box l
                int row = -1;
                if (lane < boxes && lane * a.box_rows < valid) {
                    const int pos = j * kTile + lane * a.box_rows;
                    const int page = kv_page(a.c, run.b, pos);
                    if (page >= 0)
                        row = (int)kv_row(a.c, page, pos) + (h << a.c.page_shift);
                }
                const unsigned have = __ballot_sync(kFull, row >= 0);
                for (int c = 0; go && c < a.nd; ++c) {
                    go = cta_wait(sh, &sh.empty[r.slot], r.phase ^ 1);
                    if (!go)
                        break;
                    const uint32_t bar = ring_full + 8 * r.slot, dst = smem_addr(s_raw) + r.slot * a.slot_bytes;
                    const int halves = E4M3 ? 1 : min(2, (D - 128 * c + 63) / 64);
                    const int pitch = E4M3 ? a.raw_pitch : 128;
                    if (lane == 0)
                        mbar_arrive_expect_tx(bar, __popc(have) * a.box_rows * pitch * halves);
                    __syncwarp();
                    if (row >= 0)
                        for (int x = 0; x < halves; ++x)
                            tma_load_2d(dst + x * kHalfBytes + lane * a.box_rows * pitch, is_k ? &map_k : &map_v,
                                        128 * c + 64 * x, row, bar);
                    __syncwarp();
                    r.step(a.slots);
                    issued = min(issued + 1, a.slots);
                }
            }
        }
        // copies in flight land before the CTA's memory is given back
        if (!go)
            for (int i = 0; i < issued; ++i) {
                if (r.slot == 0) {
                    r.slot = a.slots;
                    r.phase ^= 1;
                }
                --r.slot;
                mbar_wait_bounded(ring_full + 8 * r.slot, r.phase, kWaitSpins);
            }
    } else if (warp == 8) {
        // --- MMA -------------------------------------------------------------
        Ring r;
        uint32_t item = 0;        // items with keys so far (parity of q_full)
        uint32_t n_tiles = 0;     // tiles so far (parity of p_full, buffer of S)
        const int ring = E4M3 ? a.conv : a.slots;
        uint64_t* const full = E4M3 ? sh.cfull : sh.full;
        const uint32_t op_empty = E4M3 ? smem_addr(sh.cempty) : ring_empty;
        const uint32_t ops = smem_addr(E4M3 ? s_conv : s_raw), op_bytes = E4M3 ? a.conv_bytes : a.slot_bytes;
        const uint32_t q0 = smem_addr(s_q), p0 = smem_addr(s_p);
        constexpr uint32_t kIdS = tc_idesc_bf16(128, NT, false, false), kIdO = tc_idesc_bf16(128, NT, true, true);
        bool go = true;
        while (go && run.next(a)) {
            if (run.s.len == 0)
                continue;
            for (int w = 0; go && w < nwg; ++w)
                go = cta_wait(sh, &sh.q_full[w], item & 1);
            ++item;
            const int n = run.t1 - run.t0;
            for (int step = 0; go && step < 2 * n; ++step) {
                const bool is_k = step == 0 || ((step & 1) && (step + 1) / 2 < n);
                const int jj = step == 0 ? 0 : is_k ? (step + 1) / 2 : step == 2 * n - 1 ? n - 1 : step / 2 - 1;
                const int j = run.t0 + jj;
                const uint32_t g = n_tiles + jj;   // the CTA's tile count
                for (int c = 0; go && c < a.nd; ++c) {
                    go = cta_wait(sh, &full[r.slot], r.phase);
                    if (!go)
                        break;
                    tc_fence_after();
                    const uint32_t base = ops + r.slot * op_bytes;
                    const int width = min(128, D - 128 * c);
                    if (is_k) {
                        for (int w = 0; go && w < nwg; ++w) {
                            if (c == 0) {
                                go = cta_wait(sh, &sh.s_empty[w][g & 1], ((g >> 1) & 1) ^ 1);
                                if (!go)
                                    break;
                                tc_fence_after();
                            }
                            if (lane == 0) {
                                const uint32_t q = q0 + w * q_bytes + 2 * c * (NT * 128), d = tmem + (2 * w + (g & 1)) * NT;
                                for (int s = 0; s < width / 16; ++s)
                                    tc_mma_bf16(d, tc_desc_sw128(base + (s >> 2) * kHalfBytes + (s & 3) * 32, 16, 1024),
                                                tc_desc_sw128(q + (s >> 2) * (NT * 128) + (s & 3) * 32, 16, 1024), kIdS, c + s > 0);
                                if (c == a.nd - 1)
                                    tc_commit(smem_addr(&sh.s_full[w][g & 1]));
                            }
                        }
                    } else {
                        const int valid = min(kTile, run.s.len - j * kTile), ksteps = (valid + 15) / 16;
                        if (!E4M3) {
                            // rows behind the last position may hold anything: zeros instead of 0 * NaN.  A node's
                            // values are seen by some rows only: what is not finite there is zeroed too (the rows
                            // that do see it are set to NaN at the end).
                            unsigned char* v = s_raw + r.slot * a.slot_bytes;
                            bool wrote = false;
                            const int chunks = width > 64 ? 16 : 8;
                            for (int i = valid * chunks + lane; i < ksteps * 16 * chunks; i += 32) {
                                const int row = i / chunks, ch = i % chunks;
                                *reinterpret_cast<uint4*>(v + (ch >> 3) * kHalfBytes + row * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
                                wrote = true;
                            }
                            const int row = run.s.ctx + lane - j * kTile;
                            if (run.s.nn > 1 && lane < run.s.nn && row >= 0 && row < kTile)
                                for (int ch = 0; ch < chunks; ++ch) {
                                    uint4* p = reinterpret_cast<uint4*>(v + (ch >> 3) * kHalfBytes + row * 128 + (ch & 7) * 16);
                                    if (chunk_nonfinite(*p, false)) {
                                        *p = make_uint4(0, 0, 0, 0);
                                        wrote = true;
                                    }
                                }
                            if (wrote)
                                fence_proxy_async();
                            __syncwarp();
                        }
                        for (int w = 0; go && w < nwg; ++w) {
                            if (c == 0) {
                                go = cta_wait(sh, &sh.p_full[w], g & 1);
                                if (!go)
                                    break;
                                tc_fence_after();
                            }
                            if (lane == 0) {
                                const uint32_t p = p0 + w * kHalfBytes, d = tmem + (4 + w * a.nd + c) * NT;
                                const uint32_t lbo = width > 64 ? kHalfBytes : 0;
                                for (int s = 0; s < ksteps; ++s)
                                    tc_mma_bf16(d, tc_desc_sw128(base + s * 2048, lbo, 1024), tc_desc_sw128(p + s * 2048, 0, 1024), kIdO, jj + s > 0);
                                if (c == a.nd - 1)
                                    tc_commit(smem_addr(&sh.o_full[w]));
                            }
                        }
                    }
                    if (lane == 0)
                        tc_commit(op_empty + 8 * r.slot);
                    __syncwarp();
                    r.step(ring);
                }
            }
            n_tiles += n;
        }
        if (!go) {   // products in flight end before TMEM is given back
            if (lane == 0)
                tc_commit(smem_addr(&sh.drain));
            __syncwarp();
            mbar_wait_bounded(smem_addr(&sh.drain), 0, kWaitSpins);
        }
    } else if (E4M3 && warp >= 10) {
        // --- e4m3 bytes to bf16 operands -----------------------------------------
        Ring r, w;
        const int t = tid - 320;
        bool go = true;
        while (go && run.next(a)) {
            if (run.s.len == 0)
                continue;
            const int n = run.t1 - run.t0;
            for (int step = 0; go && step < 2 * n; ++step) {
                const bool is_k = step == 0 || ((step & 1) && (step + 1) / 2 < n);
                const int jj = step == 0 ? 0 : is_k ? (step + 1) / 2 : step == 2 * n - 1 ? n - 1 : step / 2 - 1;
                const int valid = min(kTile, run.s.len - (run.t0 + jj) * kTile), rows = (valid + 15) & ~15;
                const int node0 = run.s.nn > 1 ? run.s.ctx - (run.t0 + jj) * kTile : kTile;   // first row of a node
                for (int c = 0; go && c < a.nd; ++c) {
                    go = cta_wait(sh, &sh.full[r.slot], r.phase) && cta_wait(sh, &sh.cempty[w.slot], w.phase ^ 1);
                    if (!go)
                        break;
                    const unsigned char* src = s_raw + r.slot * a.slot_bytes;
                    unsigned char* dst = s_conv + w.slot * a.conv_bytes;
                    // a thread takes one row: 16 bytes of the row to two 16-byte bf16 chunks at a time; rows of a
                    // warp differ in their swizzle, so neither side's accesses collide
                    if (t < rows) {
                        const int pieces = min(128, D - 128 * c) / 16, key = t & 7;
#pragma unroll 4
                        for (int i = 0; i < pieces; ++i) {
                            uint4 x = make_uint4(0, 0, 0, 0);
                            if (t < valid)
                                x = *reinterpret_cast<const uint4*>(src + t * a.raw_pitch + ((a.raw_swizzled ? i ^ key : i) << 4));
                            const bool nan = chunk_nan_e4m3(x);
                            if (nan && t >= node0 && !is_k)
                                x = make_uint4(0, 0, 0, 0);
                            uint2 y0 = e4m3_to_bf16(x.x), y1 = e4m3_to_bf16(x.y), y2 = e4m3_to_bf16(x.z), y3 = e4m3_to_bf16(x.w);
                            if (nan) {
                                y0 = e4m3_keep_nan(x.x, y0);
                                y1 = e4m3_keep_nan(x.y, y1);
                                y2 = e4m3_keep_nan(x.z, y2);
                                y3 = e4m3_keep_nan(x.w, y3);
                            }
                            unsigned char* o = dst + (i >> 2) * kHalfBytes + t * 128;
                            const int ch = 2 * (i & 3);
                            *reinterpret_cast<uint4*>(o + ((ch ^ key) << 4)) = make_uint4(y0.x, y0.y, y1.x, y1.y);
                            *reinterpret_cast<uint4*>(o + (((ch + 1) ^ key) << 4)) = make_uint4(y2.x, y2.y, y3.x, y3.y);
                        }
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(ring_empty + 8 * r.slot);
                        mbar_arrive(smem_addr(&sh.cfull[w.slot]));
                    }
                    r.step(a.slots);
                    w.step(a.conv);
                }
            }
        }
    } else if (warp < 4 * nwg) {
        // --- softmax: one position a thread, NT rows ------------------------------
        const int w = warp >> 2, t = tid & 127, bar = 1 + w;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        unsigned char* const p_buf = s_p + w * kHalfBytes;
        float* const scratch = reinterpret_cast<float*>(p_buf);   // [4][NT], while no P is in it
        float* const negm = sh.negm[w];
        uint32_t n_tiles = 0;
        while (run.next(a)) {
            const int h = run.hg / a.groups, g = run.hg - h * a.groups;
            const int ctx = run.s.ctx, nn = run.s.nn, len = run.s.len;
            const int part = 2 * blockIdx.x + (run.t0 > 0 ? 0 : 1);
            const int item = run.b * (a.c.Hkv * a.groups) + run.hg;
            if (!run.whole() && t == 0 && w == 0)
                a.meta[part ^ 1] = item;   // meta[2i]: begun here, meta[2i + 1]: continued here
            // row c of this warpgroup: row `w * half + c` of the group
            const int mine = w == 0 ? min(a.half, a.rows) : a.rows - a.half, first = g * a.rows + w * a.half;
            const int total_rows = nn * a.G, all_rows = a.Nmax * a.G;
            if (len == 0) {
                // no position, or unusable lengths: zeros, or NaN
                const float x = run.s.ok ? 0.0f : NAN;
                if (!run.s.ok && t == 0 && w == 0 && a.has_err)
                    atomicOr(a.err, kErrCache);
                for (int i = t; i < mine * D; i += 128) {
                    const int rr = first + i / D, node = rr / a.G;
                    if (rr < all_rows)
                        a.out[(((long long)run.b * a.Nmax + node) * a.Hq + h * a.G + rr - node * a.G) * D + i % D] =
                            __float2bfloat16_rn(node < nn ? x : 0.0f);
                }
                continue;
            }
            // queries to shared memory, swizzled as the product reads them
            {
                const int per = D / 8;
                for (int i = t; i < NT * per; i += 128) {
                    const int row = i / per, ch = i - row * per, rr = first + row;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (row < mine && rr < total_rows) {
                        const int node = rr / a.G;
                        x = __ldg(reinterpret_cast<const uint4*>(a.q + ((long long)run.b * a.Nmax + node) * a.q_stride +
                                                                 (long long)(h * a.G + rr - node * a.G) * D) + ch);
                    }
                    *reinterpret_cast<uint4*>(s_q + w * q_bytes + (ch >> 3) * (NT * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) = x;
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&sh.q_full[w]));
            }
            // the rows' ancestors; nodes whose values are not finite
            bool bad;
            {
                int par;
                bad = !tree_parents(a.parent + (long long)run.b * a.Nmax, a.has_parent, nn, lane, par);
                if (t < 64) {
                    const int rr = first + t;
                    int at = t < mine && rr < total_rows && !bad ? rr / a.G : -1;
                    unsigned anc = 0;
                    for (int d = 0; d < kNodeMax && __any_sync(kFull, at >= 0); ++d) {
                        if (at >= 0)
                            anc |= 1u << at;
                        const int up = __shfl_sync(kFull, par, max(at, 0));
                        at = at >= 0 ? up : -1;
                    }
                    sh.anc[w][t] = anc;
                    if (t < NT)
                        negm[t] = 0.0f;
                }
                if (t == 0) {
                    sh.poison[w] = 0;
                    sh.unset[w] = 1;
                }
                bar_sync(bar, 128);
                if (nn > 1 && run.t1 * kTile > ctx) {
                    const int m = t >> 2, pos = ctx + m, bytes = D * (E4M3 ? 1 : 2);
                    bool hit = false;
                    if (m < nn && pos >= run.t0 * kTile && pos < run.t1 * kTile) {
                        const int page = kv_page(a.c, run.b, pos);
                        if (page >= 0) {
                            const long long row = kv_row(a.c, page, pos) + ((long long)h << a.c.page_shift);
                            const uint4* v = reinterpret_cast<const uint4*>(a.c.v + row * bytes);
                            for (int i = t & 3; i < bytes / 16; i += 4)
                                hit |= chunk_nonfinite(v[i], E4M3);
                            if (E4M3)
                                hit |= !isfinite(a.c.v_scale[row]);
                        }
                    }
                    if (hit)
                        atomicOr(&sh.poison[w], 1u << m);
                    bar_sync(bar, 128);
                }
            }
            const unsigned poison = sh.poison[w];

            uint64_t l2[NT / 2];   // this thread's share of the rows' sums, in pairs
#pragma unroll
            for (int i = 0; i < NT / 2; ++i)
                l2[i] = 0;
            // pages and scales one tile ahead
            int page = -1, page_next = -1;
            float ks = 1.0f, vs = 1.0f, ks_next = 1.0f, vs_next = 1.0f;
            auto page_of = [&](int j) {
                const int pos = j * kTile + t;
                return j < run.t1 && pos < len ? kv_page(a.c, run.b, pos) : 0;
            };
            auto scales_of = [&](int j, int pg, float& k, float& v) {
                if (E4M3) {
                    const int pos = j * kTile + t;
                    k = v = 0.0f;
                    if (j < run.t1 && pos < len && pg >= 0) {
                        const long long row = kv_row(a.c, pg, pos) + ((long long)h << a.c.page_shift);
                        // a scale that is not finite marks a row that held something that was not
                        k = a.c.k_scale[row];
                        v = a.c.v_scale[row];
                        k = isfinite(k) ? k : NAN;
                        v = isfinite(v) ? v : NAN;
                    }
                }
            };
            page = page_of(run.t0);
            scales_of(run.t0, page, ks, vs);
            page_next = page_of(run.t0 + 1);

            for (int j = run.t0; j < run.t1; ++j) {
                const uint32_t gt = n_tiles + (j - run.t0);
                bad |= page < 0;
                scales_of(j + 1, page_next, ks_next, vs_next);
                page = page_next;
                page_next = page_of(j + 2);
                const int pos = j * kTile + t;
                const bool first_tile = j == run.t0;
                const float mult = E4M3 ? a.scale_log2 * ks : a.scale_log2;

                cta_wait(sh, &sh.s_full[w][gt & 1], (gt >> 1) & 1);
                tc_fence_after();
                float s[NT];
#pragma unroll
                for (int i = 0; i < NT / 16; ++i)
                    tmem_ld16(tmem + lanes + (2 * w + (gt & 1)) * NT + 16 * i, s + 16 * i);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&sh.s_empty[w][gt & 1]));

                // scores in powers of two, relative to the rows' references
                float top = -INFINITY;
                {
                    const uint64_t m2 = f2_pack(mult, mult);
                    const ulonglong2* nm = reinterpret_cast<const ulonglong2*>(negm);
#pragma unroll
                    for (int i = 0; i < NT / 4; ++i) {
                        const ulonglong2 x = nm[i];
                        f2_unpack(f2_fma(f2_pack(s[4 * i], s[4 * i + 1]), m2, x.x), s[4 * i], s[4 * i + 1]);
                        f2_unpack(f2_fma(f2_pack(s[4 * i + 2], s[4 * i + 3]), m2, x.y), s[4 * i + 2], s[4 * i + 3]);
                    }
                }
                if ((j + 1) * kTile > ctx) {   // the tile holds nodes, or ends the sequence
                    const int m = pos - ctx;
                    const bool dead = m >= 0 && (m >= nn || ((poison >> (m & 31)) & 1u));
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        if (m >= 0 && (dead || !((sh.anc[w][i] >> (m & 31)) & 1u)))
                            s[i] = -INFINITY;
                    if (dead)
                        vs = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < NT / 2; ++i)
                    top = max3(top, s[2 * i], s[2 * i + 1]);
                const bool moved = bar_any(bar, 128, top > kLazy) || sh.unset[w];
                if (!first_tile) {   // the previous tile's product is done with P (and O)
                    cta_wait(sh, &sh.o_full[w], (gt - 1) & 1);
                    tc_fence_after();
                }
                if (moved) {
                    // the rows' maxima over the 128 positions, and the references moved to them
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const float x = warp_redux_max(s[i]);
                        if (lane == (i & 31))
                            scratch[(warp & 3) * NT + i] = x;
                    }
                    bar_sync(bar, 128);
                    float f = 1.0f, delta = 0.0f;
                    bool unset = false;
                    if (t < NT) {
                        const float x = fmaxf(fmaxf(scratch[t], scratch[NT + t]), fmaxf(scratch[2 * NT + t], scratch[3 * NT + t]));
                        // negm == +0 marks a row without a reference: no score has been seen
                        const float old = negm[t];
                        const bool fresh = __float_as_uint(old) == 0u;
                        if (fresh) {
                            unset = x == -INFINITY;
                            delta = unset ? 0.0f : x;
                        } else if (x > 0.0f) {
                            delta = x;
                            f = ex2_approx(-x);
                        }
                        if (!unset) {
                            const float now = old - delta;
                            negm[t] = __float_as_uint(now) == 0u ? -0.0f : now;
                        }
                    }
                    if (t < NT) {
                        scratch[t] = f;
                        scratch[NT + t] = delta;
                    }
                    unset = bar_any(bar, 128, unset);
                    if (t == 0)
                        sh.unset[w] = unset;
#pragma unroll
                    for (int i = 0; i < NT / 4; ++i) {
                        const float4 d = reinterpret_cast<const float4*>(scratch + NT)[i];
                        const ulonglong2 f4 = reinterpret_cast<const ulonglong2*>(scratch)[i];
                        s[4 * i] -= d.x;
                        s[4 * i + 1] -= d.y;
                        s[4 * i + 2] -= d.z;
                        s[4 * i + 3] -= d.w;
                        l2[2 * i] = f2_mul(l2[2 * i], f4.x);
                        l2[2 * i + 1] = f2_mul(l2[2 * i + 1], f4.y);
                    }
                    if (!first_tile) {
                        for (int c = 0; c < a.nd; ++c)
#pragma unroll
                            for (int i = 0; i < NT / 16; ++i) {
                                float o[16];
                                const uint32_t at = tmem + lanes + (4 + w * a.nd + c) * NT + 16 * i;
                                tmem_ld16(at, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    o[k] *= scratch[16 * i + k];
                                tmem_st16(at, o);
                            }
                        tmem_wait_st();
                    }
                    bar_sync(bar, 128);   // scratch is P again
                }
                // weights: fp32 sums, rounded once to bf16 for the second product (a weight's relative error of
                // 2^-9 averages out over the positions and stays below the result's own rounding)
                {
                    const uint64_t v2 = f2_pack(vs, vs);
#pragma unroll
                    for (int i = 0; i < NT / 8; ++i) {
                        uint32_t x[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float e0 = ex2_approx(s[8 * i + 2 * k]), e1 = ex2_approx(s[8 * i + 2 * k + 1]);
                            uint64_t e = f2_pack(e0, e1);
                            l2[4 * i + k] = f2_add(l2[4 * i + k], e);
                            if (E4M3)
                                e = f2_mul(e, v2);
                            float lo, hi;
                            f2_unpack(e, lo, hi);
                            x[k] = bf16_pair(lo, hi);
                        }
                        *reinterpret_cast<uint4*>(p_buf + t * 128 + ((i ^ (t & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                }
                fence_proxy_async();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&sh.p_full[w]));
                ks = ks_next;
                vs = vs_next;
            }
            n_tiles += run.t1 - run.t0;

            // the rows' sums over the 128 threads, while the last product runs
            float sum[NT / 16];
#pragma unroll
            for (int i = 0; i < NT / 16; ++i) {
                // lane c (of 16) ends with column 16 i + c: halve the columns, double the lanes summed
                float x[16];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    f2_unpack(l2[8 * i + k], x[2 * k], x[2 * k + 1]);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1)
#pragma unroll
                    for (int k = 0; k < o; ++k) {
                        const bool up = lane & o;
                        const float send = up ? x[k] : x[k + o];
                        const float keep = up ? x[k + o] : x[k];
                        x[k] = keep + __shfl_xor_sync(kFull, send, o);
                    }
                sum[i] = x[0] + __shfl_xor_sync(kFull, x[0], 16);
            }
            cta_wait(sh, &sh.o_full[w], (n_tiles - 1) & 1);
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < NT / 16; ++i)
                if (lane < 16)
                    scratch[(warp & 3) * NT + 16 * i + lane] = sum[i];
            bad = bar_any(bar, 128, bad) || *reinterpret_cast<volatile int*>(&sh.abort);
            if (t == 0 && bad && a.has_err)
                atomicOr(a.err, *reinterpret_cast<volatile int*>(&sh.abort) ? kErrWaitTimeout : kErrCache);
            float* const fin = scratch + 4 * NT;
            if (t < NT) {
                float l = (scratch[t] + scratch[NT + t]) + (scratch[2 * NT + t] + scratch[3 * NT + t]);
                if (bad || (sh.anc[w][t] & poison))
                    l = NAN;
                if (run.whole()) {
                    fin[t] = l == 0.0f ? 0.0f : 1.0f / l;
                } else {
                    fin[t] = 1.0f;
                    if (t < mine) {
                        float* ml = a.part_ml + ((long long)part * a.rows + w * a.half + t) * 2;
                        ml[0] = -negm[t];
                        ml[1] = l;
                    }
                }
            }
            bar_sync(bar, 128);
            for (int c = 0; c < a.nd; ++c) {
                const int d = 128 * c + t;
#pragma unroll
                for (int i = 0; i < NT / 16; ++i) {
                    float o[16];
                    tmem_ld16(tmem + lanes + (4 + w * a.nd + c) * NT + 16 * i, o);
                    tmem_wait_ld();
                    if (d < D) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const int row = 16 * i + k, rr = first + row;
                            if (row < mine) {
                                if (run.whole()) {
                                    const int node = rr / a.G;
                                    if (rr < all_rows)
                                        a.out[(((long long)run.b * a.Nmax + node) * a.Hq + h * a.G + rr - node * a.G) * D + d] =
                                            __float2bfloat16_rn(node < nn ? o[k] * fin[row] : 0.0f);
                                } else {
                                    a.part_o[((long long)part * a.rows + w * a.half + row) * D + d] = o[k];
                                }
                            }
                        }
                    }
                }
            }
            tc_fence_before();
            bar_sync(bar, 128);   // O and the scratch are read before the next item's product and P
        }
    }
    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8)
        tmem_free(tmem, 512);
}

// Items cut between CTAs: CTA i's last item, if it does not end it, is joined
// with the parts of the CTAs that go on with it.  A warp takes one row.
__global__ void __launch_bounds__(256) sv_attention_combine(const __grid_constant__ AttnArgs a, int ctas)
{
    pdl_wait();
    const int i = blockIdx.x, lane = threadIdx.x & 31, D = a.c.D;
    const int item = a.meta[2 * i];
    if (item < 0)
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
    const int per = a.c.Hkv * a.groups, b = item / per, hg = item - b * per, h = hg / a.groups, g = hg - h * a.groups;
    const int row = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5), rr = g * a.rows + row;
    if (row >= a.rows || rr >= a.Nmax * a.G)
        return;
    const int node = rr / a.G;
    const SeqLens s = seq_lens(a, b);
    // part p: CTA i's begun slot, then the continued slots of CTAs i + 1 ...
    auto slot = [&](int p) { return p == 0 ? 2LL * i + 1 : 2LL * (i + p); };
    float m = -INFINITY;
    for (int p = lane; p < n; p += 32) {
        const float2 x = *reinterpret_cast<const float2*>(a.part_ml + (slot(p) * a.rows + row) * 2);
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
    for (int p0 = 0; p0 < n; p0 += 32) {
        float wgt = 0.0f, wl = 0.0f;
        if (p0 + lane < n) {
            const float2 x = *reinterpret_cast<const float2*>(a.part_ml + (slot(p0 + lane) * a.rows + row) * 2);
            wgt = x.y == 0.0f ? 0.0f : ex2_approx(x.x - m);
            wl = wgt * x.y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            wl += __shfl_xor_sync(kFull, wl, o);
        l += wl;
        for (int p = p0; p < min(n, p0 + 32); ++p) {
            const float wp = __shfl_sync(kFull, wgt, p - p0);
            const float* o = a.part_o + (slot(p) * a.rows + row) * D;
            if (wp != 0.0f)   // a part without weight may hold what no product has written
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (lane + 32 * e < D)
                        acc[e] = fmaf(wp, o[lane + 32 * e], acc[e]);
        }
    }
    __nv_bfloat16* out = a.out + (((long long)b * a.Nmax + node) * a.Hq + h * a.G + rr - node * a.G) * D;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (lane + 32 * e < D)
            out[lane + 32 * e] = __float2bfloat16_rn(node < s.nn ? acc[e] * inv : 0.0f);
}

}  // namespace sv
