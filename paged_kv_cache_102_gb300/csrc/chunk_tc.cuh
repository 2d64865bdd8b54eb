// Attention of each sequence's new tokens over the paged cache, on the tensor
// cores (tcgen05, accumulators in tensor memory), sm_103a.
//
// Row i of sequence b (n_b = seq_starts[b + 1] - seq_starts[b] new tokens at the
// end of its L_b = context_lens[b] tokens) has position p = L_b - n_b + i and
// sees the tokens j <= p, with a window only those with j > p - window or
// j < sinks:  out = sum_j softmax_j(scale <q, K[j]>) V[j].
//
// Item: (sequence, kv head, 2 TQ consecutive new tokens), TQ = 128 / G: the G
// query heads of a kv head are rows of one product, so that two tiles of 128
// rows share every K and V tile.  Tokens come in tiles of 128, those that some
// row of the item sees; with few items a second grid axis splits their list, and
// a merge kernel joins the partial results.  One item a block, a block an SM.
// Roles:
//  warps 0-3, 4-7  softmax of row tile 0, 1 (a thread a row): scores from tensor
//                  memory, running maximum and sum, weights back to tensor memory
//                  over the scores, at last the output.  The reference maximum
//                  moves only when a row's maximum passes it by 2^8; then (almost
//                  never after the first tile) the thread multiplies its row of O.
//  warp 8          MMA: S_t = Q_t K^T (M = 128 rows, N = 128 tokens), O_t += P_t V
//                  (P from tensor memory, N = head_dim).  Order: S_0(0), S_1(0),
//                  then for each tile i and t: O_t(i), S_t(i + 1).  While one row
//                  tile is in the softmax, the other's products run.
//  warps 9, 10     producers of K and of V: one TMA copy (128-byte swizzle) for
//                  each (block, 64 channels) of a tile, into a ring of stages.
//  warp 11         V tiles that some row sees in part: rows that no row of the
//                  item sees become zeros (what lies there may be anything, and
//                  0 times it must be 0); a number that is not finite among the
//                  others sends the item to the plain loop at the end, since a
//                  weight of 0 would carry it to rows that do not see it.
//  warps 12-15     E4M3 caches: conversion.  The producers copy the codes (one bulk
//                  copy a block) into a ring of their own; these warps write them
//                  as 16-bit elements, exactly, into the ring that the products
//                  read, and do warp 11's work on the way.  One scale per tensor
//                  joins the logits' factor and the output's.  Block scales: the
//                  K producer leaves a tile's scales in shared memory; a logit is
//                  multiplied by its block's K scale, and a weight, for the product
//                  alone, by vs 2^(m - R), R the running maximum of a row's logits
//                  plus log2 |vs|: O is a sum in units of 2^R whose largest term
//                  is about 1, however far apart the scales are.
// Every barrier wait is bounded (kWaitLimitNs); on a timeout the block stops,
// drains its copies and products, frees tensor memory and reports kErrTimeout.
#pragma once

#include "kernels.h"
#include "pkv_tc.cuh"

namespace pkv {

__host__ __device__ constexpr int chunk_threads(int cache) { return is_e4m3(cache) ? 512 : 384; }
constexpr int kChunkTile = 128;       // tokens of a tile
constexpr int kChunkTmemCols = 512;   // two S (128 columns each, P over them), two O
constexpr float kChunkRescale = 8.f;  // log2 by which a maximum may pass the reference

template <int CACHE, int D>
struct ChunkSmem {
    static constexpr bool E8 = is_e4m3(CACHE);
    static constexpr int HALVES = D / 64;
    static constexpr int STG = kChunkTile * D * 2;  // a K or V tile: per 64 channels 128 rows of 128 bytes
    static constexpr int NS = E8 ? (D == 128 ? 3 : 5) : (D == 128 ? 4 : 8);
    // A role that waits for the K or for the V tiles alone sees every use of its stages when their number is even (a
    // parity names a phase only to whom none before it is still open).
    static_assert(E8 || NS % 2 == 0, "K and V tiles in stages of their own");
    static constexpr int CSTG = kChunkTile * D;  // its codes
    static constexpr int NC = E8 ? (D == 128 ? 4 : 6) : 0;
    static_assert(NC % 2 == 0, "the codes too");
    // Scales of a tile: [8] K scales, [8] V scales, [8] log2 |V scale|.  Entry i % SLOTS is written again for
    // tile i + SLOTS, once the codes of K tile use 2 (i + SLOTS) - NC were converted, for which the stage of use
    // 2 (i + SLOTS) - NC - NS >= 2 i + 1 was free: V tile i's, so that softmax(i) was over.
    static constexpr int SLOTS = CACHE == kE4M3B ? (NC + NS + 2) / 2 : 0;
    static constexpr int QT = kChunkTile * D * 2;
    static constexpr int RING = 0;
    static constexpr int Q = NS * STG;
    static constexpr int CODES = Q + 2 * QT;
    static constexpr int SCALES = CODES + NC * CSTG;
    static constexpr int BARS = SCALES + SLOTS * 24 * 4;
    // full, empty, v_ok [NS]; c_full, c_empty [NC]; q_full, s_full[2], p_full[2][2], o_done[2], final
    static constexpr int NBARS = 3 * NS + 2 * NC + 10;
    static constexpr int MISC = BARS + NBARS * 8;
    static constexpr int BYTES = MISC + 64 + 1024;  // room to align the base
    static_assert(BYTES <= 227 * 1024, "shared memory of a block");
};

// What an item covers, known to every thread of its block.
struct ChunkItem {
    int seq, kvh;
    int row0;      // first row of q and out
    int n;         // its new tokens: at most 2 TQ
    int pos0;      // position of the first
    int first_lo;  // the first row's window begins here
    int sink_tiles, win_tile0, i0, i1;  // tiles of the list, and this block's share [i0, i1) of it
};

__device__ __forceinline__ bool chunk_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort_flag) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            atomicOr(err, kErrTimeout);
            return false;
        }
    }
    return true;
}

// The sequence of row slot `slot`: the last b with starts[b] / rows + b <= slot
// (sequence b's slots begin there, and it has at most as many as lie before the
// next one's).  Warp-wide, 32 probes a step.
__device__ __forceinline__ int chunk_find(const int32_t* starts, int num_seqs, int rows, int slot, int lane) {
    int lo = 0, hi = num_seqs;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int b = lo + lane * step;
        const bool at = b < hi && starts[b] / rows + b <= slot;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, at) | 1u);
        lo += k * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

__device__ __forceinline__ int chunk_tile_start(const ChunkItem& it, int i) {
    return (i < it.sink_tiles ? i : i - it.sink_tiles + it.win_tile0) * kChunkTile;
}

// 16 bytes of 16-bit elements: whether one of them is an infinity or a NaN.
template <int ACT>
__device__ __forceinline__ bool any_not_finite(const uint4& u) {
    constexpr uint32_t EXP = ACT == kBF16 ? 0x7f807f80u : 0x7c007c00u;
    const uint32_t top = __vmaxu2(__vmaxu2(u.x & EXP, u.y & EXP), __vmaxu2(u.z & EXP, u.w & EXP));
    return (top & 0xffffu) == (EXP & 0xffffu) || (top >> 16) == (EXP >> 16);
}

// Two floats -> 16-bit pair, `a` in the low half.
template <int ACT>
__device__ __forceinline__ uint32_t pack_act(float a, float b) {
    if constexpr (ACT == kBF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

// max(a, b, c); a NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two binary32 values in a 64-bit register: multiply-add and add of both at once.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 2^a, 2^b for a, b below 127 on the multiply-add pipe, which the exponential
// unit (16 results a cycle and SM) leaves idle: x = n + f, n the nearest whole
// number (found by adding 1.5 * 2^23, which leaves it in the low bits), 2^f by a
// polynomial that is 1 at 0, of the least largest relative error on [-1/2, 1/2],
// and n added to its exponent.  At most 2^-13.2 off for bfloat16 weights, 2^-18.4
// for binary16 ones, whose rounding is 2^-9 and 2^-12.  x counts as -127 below
// that and 2^-127 comes out as 0, so that a masked weight is 0 exactly.  Not for
// NaN (the row's maximum tells of them).
template <int ACT>
__device__ __forceinline__ void exp2_pair(uint64_t x, float& a, float& b) {
    float x0, x1;
    unpair(x, x0, x1);
    x = pair(fmaxf(x0, -127.f), fmaxf(x1, -127.f));
    const uint64_t t = add2(x, pair(12582912.f, 12582912.f));
    const uint64_t f = fma2(add2(t, pair(-12582912.f, -12582912.f)), pair(-1.f, -1.f), x);
    uint64_t y;
    if constexpr (ACT == kBF16) {
        y = fma2(f, pair(0.05500893294811249f, 0.05500893294811249f), pair(0.2422109693288803f, 0.2422109693288803f));
        y = fma2(f, y, pair(0.6932829022407532f, 0.6932829022407532f));
    } else {
        y = fma2(f, pair(0.009582852944731712f, 0.009582852944731712f), pair(0.055906426161527634f, 0.055906426161527634f));
        y = fma2(f, y, pair(0.24024099111557007f, 0.24024099111557007f));
        y = fma2(f, y, pair(0.6931241750717163f, 0.6931241750717163f));
    }
    y = fma2(f, y, pair(1.f, 1.f));
    float t0, t1;
    unpair(t, t0, t1);
    unpair(y, a, b);
    a = __uint_as_float(__float_as_uint(a) + (__float_as_uint(t0) << 23));
    b = __uint_as_float(__float_as_uint(b) + (__float_as_uint(t1) << 23));
}

// One element of a cache, without its scale.
template <int CACHE>
__device__ __forceinline__ float cache_element(const void* base, int64_t i) {
    if constexpr (is_e4m3(CACHE)) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(base)[i], __NV_E4M3);
        return __half2float(*reinterpret_cast<const __half*>(&h));
    } else {
        return act_to_float<CACHE>(static_cast<const uint16_t*>(base)[i]);
    }
}

template <int ACT, int CACHE, int D>
__global__ void __launch_bounds__(chunk_threads(CACHE), 1)
    paged_chunk_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                          const __grid_constant__ CUtensorMap qmap, const ChunkParams p) {
    using S = ChunkSmem<CACHE, D>;
    constexpr bool E8 = S::E8, SCALED = CACHE == kE4M3B;
    constexpr int THREADS = chunk_threads(CACHE);
    constexpr int NS = S::NS, STG = S::STG, HALVES = S::HALVES, HALF = kChunkTile * 128;
    constexpr int NP = E8 ? S::NC : NS;  // stages of the ring that the producers fill
    constexpr uint32_t IDESC_S = tc::idesc_f16(128, kChunkTile, ACT == kBF16, false, false);
    constexpr uint32_t IDESC_O = tc::idesc_f16(128, D, ACT == kBF16, false, true);
    constexpr int O_COL = 2 * kChunkTile;  // first column of O_0; O_1 D further
    asm volatile("griddepcontrol.launch_dependents;");
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* ring = sm + S::RING;
    unsigned char* qbuf = sm + S::Q;
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + S::BARS);
    uint64_t* empty = full + NS;
    uint64_t* v_ok = empty + NS;
    uint64_t* c_full = v_ok + NS;
    uint64_t* c_empty = c_full + S::NC;
    uint64_t* q_full = c_empty + S::NC;
    uint64_t* s_full = q_full + 1;
    uint64_t* p_full = s_full + 2;
    uint64_t* o_done = p_full + 4;
    uint64_t* final_bar = o_done + 2;
    uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(sm + S::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + S::MISC + 4);
    volatile int* plain_flag = reinterpret_cast<volatile int*>(sm + S::MISC + 8);
    int* s_seq = reinterpret_cast<int*>(sm + S::MISC + 12);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.num_q_heads / p.num_kv_heads, TQ = kChunkTile / G, R = 2 * TQ;
    const int slot = (gridDim.x - 1 - blockIdx.x) / p.num_kv_heads;  // later rows, which see more, first
    if (warp == 11) {
        const int b = chunk_find(p.seq_starts, p.num_seqs, R, slot, lane);
        if (lane == 0) *s_seq = b;
        if (blockIdx.x == 0 && blockIdx.y == 0)  // every sequence's rows and length once
            for (int i = lane; i < p.num_seqs; i += 32) {
                const int s0 = p.seq_starts[i], s1 = p.seq_starts[i + 1], L = p.context_lens[i];
                if (s0 < 0 || s1 < s0 || s1 > p.num_tokens || (s1 > s0 && (L < s1 - s0 || L > p.max_blocks_per_seq * p.block_size)))
                    atomicOr(p.err, kErrBadLen);
            }
    } else if (warp == 8) {
        tc::tmem_alloc(tmem_base_smem, kChunkTmemCols);
        tc::tmem_relinquish();
    } else if (threadIdx.x == 9 * 32) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], E8 ? 4 : 1);
            mbar_init(&empty[i], 1);
            mbar_init(&v_ok[i], 1);
        }
        for (int i = 0; i < S::NC; ++i) {
            mbar_init(&c_full[i], 1);
            mbar_init(&c_empty[i], 4);
        }
        mbar_init(q_full, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[2 * t], 4);
            mbar_init(&p_full[2 * t + 1], 4);
            mbar_init(&o_done[t], 1);
        }
        mbar_init(final_bar, 1);
        *abort_flag = 0;
        *plain_flag = 0;
        mbar_init_fence();
        if constexpr (!E8) {
            tc::prefetch_tensormap(&kmap);
            tc::prefetch_tensormap(&vmap);
        }
        tc::prefetch_tensormap(&qmap);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_base_smem;

    ChunkItem it;
    it.seq = *s_seq;
    it.kvh = (gridDim.x - 1 - blockIdx.x) % p.num_kv_heads;
    bool any;
    {
        const int s0 = p.seq_starts[it.seq], s1 = p.seq_starts[it.seq + 1], L = p.context_lens[it.seq];
        const int first = (slot - (s0 / R + it.seq)) * R;  // of the sequence's new tokens
        any = s0 >= 0 && s1 <= p.num_tokens && first >= 0 && first < s1 - s0 && L >= s1 - s0 &&
              L <= p.max_blocks_per_seq * p.block_size;
        it.row0 = s0 + first;
        it.n = min(R, s1 - s0 - first);
        it.pos0 = L - (s1 - s0) + first;
    }
    const int last = it.pos0 + it.n - 1;  // position of the last row
    it.first_lo = p.window ? max(0, it.pos0 - p.window + 1) : 0;
    it.win_tile0 = it.first_lo / kChunkTile;
    it.sink_tiles = min(it.win_tile0, p.sinks / kChunkTile + (p.sinks % kChunkTile != 0));
    const int tiles = last / kChunkTile - it.win_tile0 + 1 + it.sink_tiles;
    it.i0 = static_cast<int>(static_cast<int64_t>(tiles) * blockIdx.y / gridDim.y);
    it.i1 = static_cast<int>(static_cast<int64_t>(tiles) * (blockIdx.y + 1) / gridDim.y);
    const int n_list = any ? it.i1 - it.i0 : 0;
    // row tile t's share of the list: up to the tile of its last row (none without rows)
    auto rows_of = [&](int t) { return max(0, min(TQ, it.n - t * TQ)); };
    auto count_of = [&](int t) {
        const int rows = rows_of(t);
        if (rows == 0) return 0;
        const int end = (it.pos0 + t * TQ + rows - 1) / kChunkTile - it.win_tile0 + 1 + it.sink_tiles;
        return max(0, min(n_list, end - it.i0));
    };
    const int cnt0 = count_of(0), cnt1 = count_of(1);
    const int n_run = max(cnt0, cnt1);
    const uint64_t policy = l2_policy_evict_first();

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        const int t = warp >> 2, row = (warp & 3) * 32 + lane;
        const int cnt = t == 0 ? cnt0 : cnt1;
        const int tok = row / G, g = row - tok * G;  // (rows past TQ * G and past the last token: none)
        const bool mine = tok < rows_of(t);
        const bool live = __any_sync(0xffffffffu, mine);
        const int pos = mine ? it.pos0 + t * TQ + tok : -1;
        const int pos_lo = it.pos0 + t * TQ, pos_hi = pos_lo + rows_of(t) - 1;  // of the row tile
        const uint32_t s_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + t * kChunkTile;
        const uint32_t o_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + O_COL + t * D;
        const float factor = CACHE == kE4M3 ? p.scale_log2 * *p.k_scale : p.scale_log2;
        const float c = SCALED ? 1.f : fmaxf(fabsf(factor), 1e-37f);  // (times -inf: never a NaN, at a factor of 0 either)
        const bool negative = !SCALED && factor < 0.f;
        // reference maximum (log2 units) and sum; block scales: of the logits plus log2 |vs|, the unit of O
        float m = -INFINITY, l = 0.f;
        [[maybe_unused]] float unit = -INFINITY;
        bool ok = true;
        for (int i = 0; i < cnt && ok; ++i) {
            ok = __all_sync(0xffffffffu, chunk_wait(&s_full[t], i & 1, abort_flag, p.err));
            if (!ok) break;
            tc::fence_after_sync();
            if (live) {
                const int start = chunk_tile_start(it, it.i0 + i);
                const bool masked = start + kChunkTile - 1 > pos_lo ||
                                    (p.window != 0 && start <= pos_hi - p.window && start + kChunkTile > p.sinks);
                const int end = pos - start;                         // sees columns up to this one
                const int from = p.window ? end - p.window + 1 : 0;  // and from this one on,
                const int sink = p.sinks - start;                    // or before this one
                [[maybe_unused]] const float* scales =
                    reinterpret_cast<const float*>(sm + S::SCALES) + (SCALED ? (i % max(1, S::SLOTS)) * 24 : 0);
                [[maybe_unused]] const int bshift = p.block_size == 32 ? 1 : 0;  // 16-column groups to blocks
                // 32 scores from column k on, in what `c` makes log2 units (16-bit caches: they are there already)
                auto scores = [&](int k, float* s) {
                    if constexpr (E8) {
                        tc::TmemLd<32>::load(s_addr + k, s);
                        tc::tmem_wait_ld();
                    }
                    if constexpr (SCALED) {
#pragma unroll
                        for (int x = 0; x < 32; x += 16) {
                            const float f = factor * scales[((k + x) >> 4) >> bshift];
#pragma unroll
                            for (int j = 0; j < 16; ++j) s[x + j] *= f;
                        }
                    } else if (negative) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) s[j] = -s[j];
                    }
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (k + j > end || (k + j < from && k + j >= sink)) s[j] = -INFINITY;
                    }
                };
                // 16-bit caches hold a row's scores; the others, with fewer registers a thread, read them twice
                float s[E8 ? 32 : kChunkTile];
                if constexpr (!E8) {
#pragma unroll
                    for (int k = 0; k < kChunkTile; k += 32) tc::TmemLd<32>::load(s_addr + k, s + k);
                    tc::tmem_wait_ld();
                }
                float mx = -INFINITY, tops[8];
                [[maybe_unused]] float mu = -INFINITY;
#pragma unroll
                for (int k = 0; k < kChunkTile; k += 32) {
                    float* x = s + (E8 ? 0 : k);
                    scores(k, x);
#pragma unroll
                    for (int y = 0; y < 32; y += 16) {
                        float top = max3_nan(x[y], x[y + 1], x[y + 2]);
#pragma unroll
                        for (int j = 3; j < 15; j += 2) top = max3_nan(top, x[y + j], x[y + j + 1]);
                        tops[(k + y) / 16] = top = max3_nan(top, x[y + 15], x[y + 15]);
                        if constexpr (SCALED) mu = fmaxf(mu, top + scales[16 + (((k + y) >> 4) >> bshift)]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; j += 2) mx = max3_nan(mx, tops[j], tops[j + 1]);
                mx *= c;
                if (!(mx < INFINITY)) l = NAN;  // an infinite logit or none at all: no weights
                const bool move = mine && mx > m + kChunkRescale;
                const bool turn = SCALED ? mine && mu > unit + kChunkRescale : move;
                if (__any_sync(0xffffffffu, turn && l > 0.f)) {
                    // O holds the tiles before: their products are done, then the row is multiplied
                    ok = __all_sync(0xffffffffu, chunk_wait(&o_done[t], (i - 1) & 1, abort_flag, p.err));
                    if (!ok) break;
                    tc::fence_after_sync();
                    const float f = !turn ? 1.f : SCALED ? fast_exp2(unit - mu) : fast_exp2(m - mx);
#pragma unroll
                    for (int k = 0; k < D; k += 8) {
                        float o[8];
                        tc::TmemLd<8>::load(o_addr + k, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[j] *= f;
                        tc::tmem_st<8>(o_addr + k, o);
                    }
                }
                if (move) {
                    l *= fast_exp2(m - mx);  // (0 times what it is at first)
                    m = mx;
                }
                if (SCALED && turn) unit = mu;
                const float ref = m == -INFINITY ? 0.f : m;  // nothing seen yet: weights of 0
                [[maybe_unused]] const float lift = SCALED && unit != -INFINITY ? fast_exp2(ref - unit) : 0.f;
                uint64_t sum = pair(0.f, 0.f);
                const uint64_t c2 = pair(c, c), ref2 = pair(-ref, -ref);
#pragma unroll
                for (int k = 0; k < kChunkTile; k += 32) {
                    float* x = s + (E8 ? 0 : k);
                    if constexpr (E8) scores(k, x);
                    uint32_t w[16];
#pragma unroll
                    for (int y = 0; y < 32; y += 16) {
                        [[maybe_unused]] float vf = 1.f;
                        if constexpr (SCALED) vf = lift * scales[8 + (((k + y) >> 4) >> bshift)];
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const uint64_t e = fma2(pair(x[y + j], x[y + j + 1]), c2, ref2);
                            float a, b;
                            if (j % 8 == 6) {
                                exp2_pair<ACT>(e, a, b);
                            } else {
                                unpair(e, a, b);
                                a = fast_exp2(a);
                                b = fast_exp2(b);
                            }
                            sum = add2(sum, pair(a, b));
                            if constexpr (SCALED) {
                                a *= vf;
                                b *= vf;
                            }
                            w[(y + j) / 2] = pack_act<ACT>(a, b);
                        }
                    }
                    tc::tmem_st16(s_addr + k / 2, w);
                    if (k == 32) {  // the products over the first 64 tokens may begin
                        tc::tmem_wait_st();
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&p_full[2 * t]);
                    }
                }
                float sum0, sum1;
                unpair(sum, sum0, sum1);
                l += sum0 + sum1;
                tc::tmem_wait_st();
            } else if (lane == 0) {
                mbar_arrive(&p_full[2 * t]);
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * t + 1]);
        }
        if (ok && cnt > 0) {
            ok = __all_sync(0xffffffffu, chunk_wait(&o_done[t], (cnt - 1) & 1, abort_flag, p.err));
            tc::fence_after_sync();
        }
        if (ok && live && any) {
            // what an element of O stands for
            float vmul = 1.f;
            if constexpr (CACHE == kE4M3) vmul = *p.v_scale;
            if constexpr (SCALED) vmul = unit == -INFINITY ? 0.f : fast_exp2(unit - m);
            const int64_t at = it.row0 + t * TQ + tok;
            const int h = it.kvh * G + g;
            if (p.ws_ml != nullptr) {
                const int64_t slot_row = (static_cast<int64_t>(blockIdx.y) * p.num_tokens + at) * p.num_q_heads + h;
                if (mine) reinterpret_cast<float2*>(p.ws_ml)[slot_row] = make_float2(m, l);
#pragma unroll
                for (int k = 0; k < D; k += 16) {
                    float o[16];
                    if (cnt > 0) {
                        tc::TmemLd<16>::load(o_addr + k, o);
                        tc::tmem_wait_ld();
                    }
                    if (mine && cnt > 0) {
                        float4* dst = reinterpret_cast<float4*>(p.ws_o + slot_row * D + k);
#pragma unroll
                        for (int j = 0; j < 4; ++j) dst[j] = make_float4(o[4 * j] * vmul, o[4 * j + 1] * vmul, o[4 * j + 2] * vmul, o[4 * j + 3] * vmul);
                    }
                }
            } else {
                const float inv = vmul / l;
                uint16_t* dst = static_cast<uint16_t*>(p.out) + at * p.out_stride + static_cast<int64_t>(h) * D;
#pragma unroll
                for (int k = 0; k < D; k += 32) {
                    float o[32];
                    tc::TmemLd<32>::load(o_addr + k, o);
                    tc::tmem_wait_ld();
                    if (mine) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8)
                            *reinterpret_cast<uint4*>(dst + k + j) =
                                make_uint4(pack_act<ACT>(o[j] * inv, o[j + 1] * inv), pack_act<ACT>(o[j + 2] * inv, o[j + 3] * inv),
                                           pack_act<ACT>(o[j + 4] * inv, o[j + 5] * inv), pack_act<ACT>(o[j + 6] * inv, o[j + 7] * inv));
                    }
                }
            }
        }
    } else if (warp == 8) {
        // ---------------------------------------------------------------- MMA
        const uint32_t k_base = smem_addr(ring), q_base = smem_addr(qbuf);
        auto mma_s = [&](int t, int stage) {
            const uint32_t a = q_base + t * S::QT, b = k_base + stage * STG;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * HALF + (kk & 3) * 32;
                tc::mma_f16(tmem + t * kChunkTile, tc::desc_sw128(a + off, 16, 1024), tc::desc_sw128(b + off, 16, 1024),
                            IDESC_S, kk > 0);
            }
        };
        auto mma_o = [&](int t, int stage, int half, bool add) {  // over 64 tokens
            const uint32_t b = k_base + stage * STG;
#pragma unroll
            for (int kk = half * 4; kk < half * 4 + 4; ++kk)
                tc::mma_f16_ts(tmem + O_COL + t * D, tmem + t * kChunkTile + kk * 8, tc::desc_sw128(b + kk * 2048, HALF, 1024),
                               IDESC_O, add || half > 0 || kk > 0);
        };
        bool ok = n_run > 0 && __all_sync(0xffffffffu, chunk_wait(q_full, 0, abort_flag, p.err));
        // tile i: K is stage use 2 i, V 2 i + 1
        if (ok) ok = __all_sync(0xffffffffu, chunk_wait(&full[0], 0, abort_flag, p.err));
        if (ok) {
            tc::fence_after_sync();
            if (tc::elect_one()) {
                if (cnt0 > 0) {
                    mma_s(0, 0);
                    tc::commit(&s_full[0]);
                }
                if (cnt1 > 0) {
                    mma_s(1, 0);
                    tc::commit(&s_full[1]);
                }
                tc::commit(&empty[0]);
            }
            __syncwarp();
        }
        for (int i = 0; i < n_run && ok; ++i) {
            const int uv = 2 * i + 1, uk = 2 * i + 2;
            const int sv = uv % NS, sk = uk % NS;
            const bool more = i + 1 < n_run;
            ok = __all_sync(0xffffffffu, E8 ? chunk_wait(&full[sv], (uv / NS) & 1, abort_flag, p.err)
                                            : chunk_wait(&v_ok[i % NS], (i / NS) & 1, abort_flag, p.err));
            if (!ok) break;
            if (more) ok = __all_sync(0xffffffffu, chunk_wait(&full[sk], (uk / NS) & 1, abort_flag, p.err));
            if (!ok) break;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int cnt = t == 0 ? cnt0 : cnt1;
                if (i >= cnt) continue;
                ok = __all_sync(0xffffffffu, chunk_wait(&p_full[2 * t], i & 1, abort_flag, p.err));
                if (!ok) break;
                tc::fence_after_sync();
                if (tc::elect_one()) mma_o(t, sv, 0, i > 0);
                __syncwarp();
                ok = __all_sync(0xffffffffu, chunk_wait(&p_full[2 * t + 1], i & 1, abort_flag, p.err));
                if (!ok) break;
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    mma_o(t, sv, 1, true);
                    tc::commit(&o_done[t]);
                    if (i + 1 < cnt) {
                        mma_s(t, sk);
                        tc::commit(&s_full[t]);
                    }
                }
                __syncwarp();
            }
            if (!ok) break;
            if (tc::elect_one()) {
                tc::commit(&empty[sv]);
                if (more) tc::commit(&empty[sk]);
            }
            __syncwarp();
        }
        // every product issued has completed before tensor memory is freed
        if (tc::elect_one()) {
            tc::commit(final_bar);
            if (!mbar_wait(final_bar, 0)) atomicOr(p.err, kErrTimeout);
        }
        __syncwarp();
    } else if (warp < 11) {
        // ---------------------------------------------------------- producers
        const int v = warp - 9;  // 0: K (and Q), 1: V
        const CUtensorMap* map = v ? &vmap : &kmap;
        if (v == 0 && lane == 0 && n_run > 0) {
            const uint32_t bytes = HALVES * G * TQ * 128;
            mbar_arrive_expect_tx(q_full, ((cnt0 > 0) + (cnt1 > 0)) * bytes);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if ((t == 0 ? cnt0 : cnt1) > 0)
                    for (int h = 0; h < HALVES; ++h)
                        tc::tma_load_3d(qbuf + t * S::QT + h * HALF, &qmap, h * 64, it.kvh * G, it.row0 + t * TQ, q_full, policy);
        }
        const int BS = p.block_size, bpt = kChunkTile / BS;
        const int32_t* table = p.block_tables + static_cast<int64_t>(it.seq) * p.max_blocks_per_seq;
        // block of the tile and 64-channel part of this lane (codes: the whole block)
        constexpr int PARTS = E8 ? 1 : HALVES;
        const int j = lane / PARTS, h = lane % PARTS;
        // the lane's block in tile i: -1 past the last row's tokens, wholly hidden, or outside the pool
        auto entry = [&](int i) {
            if (i >= n_run || j >= bpt) return -1;
            const int t0 = chunk_tile_start(it, it.i0 + i) + j * BS;
            if (t0 > last || (t0 >= p.sinks && t0 + BS <= it.first_lo)) return -1;
            const int phys = table[t0 / BS];
            if (phys < 0 || phys >= p.num_blocks) {
                atomicOr(p.err, kErrBadBlock);
                return -1;
            }
            return phys;
        };
        int phys = entry(0);
        int issued = 0;
        for (int i = 0; i < n_run; ++i) {
            const int use = 2 * i + v, s = use % NP;
            uint64_t* filled = E8 ? &c_full[s] : &full[s];
            const int next = entry(i + 1);
            [[maybe_unused]] float ks = 0.f, vs = 0.f;
            if (SCALED && v == 0 && phys >= 0) {
                const int64_t at = static_cast<int64_t>(phys) * p.num_kv_heads + it.kvh;
                ks = p.k_scale[at];
                vs = p.v_scale[at];
            }
            const unsigned loads = __ballot_sync(0xffffffffu, phys >= 0);
            bool good = true;
            if (lane == 0 && use >= NP)
                good = chunk_wait(E8 ? &c_empty[s] : &empty[s], (use / NP - 1) & 1, abort_flag, p.err);
            if (!__shfl_sync(0xffffffffu, good, 0)) break;
            if constexpr (SCALED) {
                if (v == 0) {
                    if (lane < 8) {
                        float* dst = reinterpret_cast<float*>(sm + S::SCALES) + (i % S::SLOTS) * 24 + lane;
                        dst[0] = ks;
                        dst[8] = vs;
                        dst[16] = fmaxf(__log2f(fabsf(vs)), -100.f);
                    }
                    __syncwarp();  // before the copies' barrier, which the softmax waits on in the end
                }
            }
            if (lane == 0) mbar_arrive_expect_tx(filled, __popc(loads) * (E8 ? BS * D : BS * 128));
            __syncwarp();
            if constexpr (E8) {
                if (phys >= 0)
                    bulk_copy_g2s(sm + S::CODES + s * S::CSTG + j * BS * D,
                                  static_cast<const unsigned char*>(v ? p.v_cache : p.k_cache) +
                                      (static_cast<int64_t>(phys) * p.num_kv_heads + it.kvh) * (BS * D),
                                  BS * D, filled, policy);
            } else if (phys >= 0)
                tc::tma_load_2d(ring + s * STG + h * HALF + j * BS * 128, map, h * 64, (phys * p.num_kv_heads + it.kvh) * BS,
                                &full[s], policy);
            phys = next;
            ++issued;
        }
        // leave only when every copy into this block's shared memory has landed
        if (lane == 0) {
            for (int i = max(0, issued - NP); i < issued; ++i) {
                const int use = 2 * i + v;
                if (use + NP >= 2 * issued && !mbar_wait(E8 ? &c_full[use % NP] : &full[use % NP], (use / NP) & 1))
                    atomicOr(p.err, kErrTimeout);
            }
            if (v == 0 && n_run > 0 && !mbar_wait(q_full, 0)) atomicOr(p.err, kErrTimeout);
        }
        __syncwarp();
    } else if (E8 && warp >= 12) {
        // --------------------------------------------------------- conversion
        // 16 codes a lane and step.  8 neighbouring lanes, which shared memory serves at once, take 64 channels of
        // two tokens (head_dim 128: the other half of the second), so that neither their reads nor their writes,
        // which the swizzle moves by one 16-byte chunk from token to token, meet in a bank.
        if constexpr (E8) {
            for (int u = 0; u < 2 * n_run; ++u) {
                const int cs = u % S::NC, s = u % NS;
                bool good = chunk_wait(&c_full[cs], (u / S::NC) & 1, abort_flag, p.err);
                if (good && u >= NS) good = chunk_wait(&empty[s], (u / NS - 1) & 1, abort_flag, p.err);
                if (!__all_sync(0xffffffffu, good)) break;
                const unsigned char* codes = sm + S::CODES + cs * S::CSTG;
                unsigned char* dst = ring + s * STG;
                const int start = chunk_tile_start(it, it.i0 + (u >> 1));
                const int last_lo = p.window ? max(0, last - p.window + 1) : 0;
                const bool partly = (u & 1) && (start + kChunkTile - 1 > it.pos0 || (start < last_lo && start + kChunkTile > p.sinks));
                bool bad = false;
                constexpr int TOKENS = 32 / (4 * HALVES);  // a warp's step
#pragma unroll 4
                for (int r0 = (warp - 12) * TOKENS; r0 < kChunkTile; r0 += 4 * TOKENS) {
                    const int pair = lane & 15, second = (lane >> 2) & 1;
                    const int r = r0 + (HALVES == 2 ? (lane >> 4) * 2 + second : lane >> 2);
                    const int h = HALVES == 2 ? ((pair >> 3) ^ second) : 0;
                    const int x = (lane & 3) * 2;  // first of two 8-channel chunks of the part
                    uint4 c = *reinterpret_cast<const uint4*>(codes + r * D + h * 64 + x * 8);
                    if (partly) {
                        const int j = start + r;
                        if (j > last || (j < it.first_lo && j >= p.sinks)) c = make_uint4(0u, 0u, 0u, 0u);
                        const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q)  // a code of 0x7f or 0xff
                            bad = bad || __vcmpeq4(cw[q] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
                    }
                    const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
                    uint32_t w[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const uint32_t f = e4m3x2_to_f16x2(static_cast<uint16_t>(cw[q / 2] >> (16 * (q % 2))));
                        if constexpr (ACT == kF16) {
                            w[q] = f;
                        } else {
                            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f));
                            w[q] = pack_act<kBF16>(v.x, v.y);
                        }
                    }
                    unsigned char* row = dst + h * HALF + r * 128;
                    *reinterpret_cast<uint4*>(row + ((x ^ (r & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(row + (((x + 1) ^ (r & 7)) * 16)) = make_uint4(w[4], w[5], w[6], w[7]);
                }
                if (bad) *plain_flag = 1;
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&full[s]);
                    mbar_arrive(&c_empty[cs]);
                }
            }
        }
    } else if (!E8) {
        // ------------------------------------------------------- V tiles' check
        for (int i = 0; i < n_run; ++i) {
            const int use = 2 * i + 1, s = use % NS;
            if (!__all_sync(0xffffffffu, chunk_wait(&full[s], (use / NS) & 1, abort_flag, p.err))) break;
            const int start = chunk_tile_start(it, it.i0 + i);
            const int last_lo = p.window ? max(0, last - p.window + 1) : 0;  // the last row's window begins here
            if (start + kChunkTile - 1 > it.pos0 || (start < last_lo && start + kChunkTile > p.sinks)) {
                constexpr int CH = 8 * HALVES, STEP = 32 / CH;  // 16-byte chunks of a token, tokens of a warp's access
                const int x = lane % CH, r0 = lane / CH;
                unsigned char* vb = ring + s * STG + (x >> 3) * HALF + (x & 7) * 16;
                auto clear = [&](int from, int to) {  // tokens [from, to) of the tile
                    for (int r = min(kChunkTile, max(0, from)) + r0; r < min(kChunkTile, to); r += STEP)
                        *reinterpret_cast<uint4*>(vb + r * 128) = make_uint4(0u, 0u, 0u, 0u);
                };
                auto look = [&](int from, int to) {
                    bool bad = false;
                    to = min(kChunkTile, to);
                    for (int r = min(kChunkTile, max(0, from)) + r0; r < to; r += 8 * STEP) {
                        uint4 u[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y)
                            u[y] = r + y * STEP < to ? *reinterpret_cast<const uint4*>(vb + (r + y * STEP) * 128)
                                                     : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                        for (int y = 0; y < 8; ++y) bad = any_not_finite<ACT>(u[y]) || bad;
                    }
                    if (bad) *plain_flag = 1;
                };
                clear(last + 1 - start, kChunkTile);
                if (p.window) {
                    clear(p.sinks - start, it.first_lo - start);                    // hidden from every row
                    look(max(p.sinks, it.first_lo) - start, last_lo - start);       // from the last ones
                    look(max(it.pos0 + 1, last_lo) - start, last + 1 - start);      // from the first ones
                    look(it.pos0 + 1 - start, min(p.sinks, last + 1) - start);
                } else {
                    look(it.pos0 + 1 - start, last + 1 - start);
                }
                tc::fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_ok[i % NS]);  // (the i-th V tile's, whatever its stage)
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 8) tc::tmem_dealloc(tmem, kChunkTmemCols);

    // A V that is not finite, in a tile that some row sees in part: the item's rows one by one.
    if (*plain_flag != 0 && *abort_flag == 0) {
        constexpr int W = D / 32;
        const int32_t* table = p.block_tables + static_cast<int64_t>(it.seq) * p.max_blocks_per_seq;
        for (int r = warp; r < it.n * G; r += THREADS / 32) {
            const int64_t at = it.row0 + r / G;
            const int pos = it.pos0 + r / G, h = it.kvh * G + r % G;
            const uint16_t* q = static_cast<const uint16_t*>(p.q) + at * p.q_stride + static_cast<int64_t>(h) * D;
            float qf[W], acc[W] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
            for (int x = 0; x < W; ++x) qf[x] = act_to_float<ACT>(q[lane + 32 * x]) * p.scale_log2;
            const float kt = CACHE == kE4M3 ? *p.k_scale : 1.f, vt = CACHE == kE4M3 ? *p.v_scale : 1.f;
            const int lo = p.window ? max(0, pos - p.window + 1) : 0;
            for (int i = it.i0; i < it.i1; ++i) {
                const int start = chunk_tile_start(it, i);
                for (int j = start; j < start + kChunkTile && j <= pos; ++j) {
                    if (j < lo && j >= p.sinks) continue;
                    const int blk = table[j / p.block_size];
                    if (blk < 0 || blk >= p.num_blocks) continue;
                    const int64_t tile = static_cast<int64_t>(blk) * p.num_kv_heads + it.kvh;
                    const int64_t src = (tile * p.block_size + j % p.block_size) * D;
                    float d = 0.f;
#pragma unroll
                    for (int x = 0; x < W; ++x) d = fmaf(qf[x], cache_element<CACHE>(p.k_cache, src + lane + 32 * x), d);
#pragma unroll
                    for (int off = 16; off >= 1; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
                    d *= SCALED ? p.k_scale[tile] : kt;
                    if (d > m) {
                        const float f = fast_exp2(m - d);
                        l *= f;
#pragma unroll
                        for (int x = 0; x < W; ++x) acc[x] *= f;
                        m = d;
                    }
                    const float w = fast_exp2(d - m);
                    l += w;
                    const float wv = w * (SCALED ? p.v_scale[tile] : vt);
#pragma unroll
                    for (int x = 0; x < W; ++x) acc[x] = fmaf(wv, cache_element<CACHE>(p.v_cache, src + lane + 32 * x), acc[x]);
                }
            }
            if (p.ws_ml != nullptr) {
                const int64_t slot_row = (static_cast<int64_t>(blockIdx.y) * p.num_tokens + at) * p.num_q_heads + h;
                if (lane == 0) reinterpret_cast<float2*>(p.ws_ml)[slot_row] = make_float2(m, l);
#pragma unroll
                for (int x = 0; x < W; ++x) p.ws_o[slot_row * D + lane + 32 * x] = acc[x];
            } else {
                uint16_t* dst = static_cast<uint16_t*>(p.out) + at * p.out_stride + static_cast<int64_t>(h) * D;
#pragma unroll
                for (int x = 0; x < W; ++x) dst[lane + 32 * x] = float_to_act<ACT>(acc[x] / l);
            }
        }
    }
}

}  // namespace pkv
