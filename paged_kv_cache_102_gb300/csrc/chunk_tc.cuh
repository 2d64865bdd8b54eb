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
// An item of one row tile (up to TQ tokens: single tokens, drafts) is folded: both
// halves of the machinery below, row tile 0's and 1's, take its rows, one the even
// and one the odd token tiles, each with a maximum, sum and O of its own, which the
// first joins at the end; one's products run under the other's softmax all the same.
// Roles:
//  warps 0-15      softmax: a row of a tile is two threads', 64 tokens each (row
//                  tile (w >> 2) & 1, half w >> 3, rows 32 (w & 3) .. of warp w):
//                  scores from tensor memory, running maximum and sum, weights
//                  back to tensor memory over the scores, at last the output.  The
//                  reference maximum moves only when a maximum passes it by 2^8,
//                  so that the two need no more of each other than a vote; when it
//                  moves (almost never after the first tile) they exchange their
//                  maxima and multiply the row of O, half each.  For binary16
//                  weights the reference lies 2^7 below the maximum: the largest
//                  are 2^7, at most 2^15, and weights keep the type's precision
//                  down to 2^-21 of the largest, below that 2^-32 of it.  (Beside
//                  a first token that has nearly all the weight and a V of nearly
//                  nothing, as such tokens do, the others' weights are the output:
//                  with the maximum itself for a reference those of 2^-21.6 lost 5 %.)
//  warp 19         MMA: S_t = Q_t K^T (M = 128 rows, N = 128 tokens), O_t += P_t V
//                  (P from tensor memory, N = head_dim).  Order: S_0(0), S_1(0),
//                  then for each tile i and t: O_t(i), S_t(i + 1).  While one row
//                  tile is in the softmax, the other's products run.
//  warps 17, 18    producers of K and of V, into a ring of stages: TMA copies (128-byte
//                  swizzle), for K one of each (block, 64 channels) of a tile, for V,
//                  whose products take a block's tokens at a time, one of each block.
//                  The copies of a warp leave one after the other, some 94 cycles
//                  each; sharing K's 16 between the two warps was no faster.
//  warp 16         V tiles that some row sees in part: rows that no row of the
//                  item sees become zeros (what lies there may be anything, and
//                  0 times it must be 0); a number that is not finite among the
//                  others sends the item to the plain loop at the end, since a
//                  weight of 0 would carry it to rows that do not see it.
//  warps 20-23     E4M3 caches: conversion.  The producers copy the codes (one bulk
//                  copy a block) into a ring of their own; these warps, and of a
//                  folded item the softmax warps that have none of its rows, write them
//                  as 16-bit elements, exactly, into the ring that the products
//                  read, and do warp 16's work on the way.  One scale per tensor
//                  joins the logits' factor and the output's.  Block scales: the
//                  K producer leaves a tile's scales in shared memory; a logit is
//                  multiplied by its block's K scale, and a weight, for the product
//                  alone, by vs 2^(m - R), R the running maximum of a row's logits
//                  plus log2 |vs|: O is a sum in units of 2^R whose largest term
//                  is about 1 (binary16: 2^7), however far apart the scales are.
// Measured, head_dim 128: four prompts of up to 4096 tokens, 64 / 8 heads, bfloat16, 499 us, 1.02 PFLOP/s (52 % of a large
// library product's); 509 new tokens behind 32K, 32 / 8 heads, binary16, 244 us, 1.11 PFLOP/s; head_dim 64 a third of that
// (the same exponentials for half the products).  Of each pair of row tiles' 128-token step, 3300 cycles, the products
// are 2048 at the tensor rate, and their operands and the copies take 256 KB of shared memory's 128 bytes a cycle, as long;
// with the exponentials, maxima and sums left out it is 10 % shorter, and no pipe is busy for half of it.  What fills the
// other 1250 cycles was not traced: likely a row tile's chain of scores, weights, O and the next scores, which have one
// buffer.  Products add in float32, so that weights below 2^-24 of an O's size are lost to it.
// Single tokens over 16-bit caches are bound by HBM (1.5 us a tile an SM), over E4M3 ones (1.7 us; block scales 2.0) by
// shared memory, which the products' operands, the conversion and the copies of codes share (224 KB a tile).  A block's
// start and end are some 6 tiles' time.
// Every barrier wait is bounded (kWaitLimitNs); on a timeout the block stops,
// drains its copies and products, frees tensor memory and reports kErrTimeout.
#pragma once

#include <type_traits>

#include "kernels.h"
#include "pkv_tc.cuh"

namespace pkv {

__host__ __device__ constexpr int chunk_threads(int cache) { return is_e4m3(cache) ? 768 : 640; }
constexpr int kChunkTile = 128;       // tokens of a tile
constexpr int kConverters = 16;       // most warps that convert codes
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
    // Scales of a tile: [8] K scales, [8] V scales, [8] log2 |V scale|.  Entry i % SLOTS is written again for tile
    // i + SLOTS, once the codes of K tile i' = i + SLOTS - NC / 2 were converted, as use 2 i' at least 2 i' - 1 of the
    // ring, for which the stage of NS uses before was free; no earlier than V tile i's (use 2 i + 2 at most), so that
    // softmax(i) was over.
    static constexpr int SLOTS = CACHE == kE4M3B ? (NC + NS + 4) / 2 : 0;
    static_assert(CACHE != kE4M3B || 2 * SLOTS >= NC + NS + 3, "scales of a tile in use");
    static constexpr int QT = kChunkTile * D * 2;
    static constexpr int RING = 0;
    static constexpr int Q = NS * STG;
    static constexpr int CODES = Q + 2 * QT;
    static constexpr int SCALES = CODES + NC * CSTG;
    static constexpr int SWAP = SCALES + SLOTS * 24 * 4;  // a value of each row, between its two threads
    static constexpr int BARS = SWAP + 2 * kChunkTile * 4;
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
    int sink_tiles, win_tile0, i0, i1;  // tiles of the list, and this block's share [i0, i1) of it (0, 0: nothing to do)
    int any;       // whether it has rows
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
        __nanosleep(50);  // most warps wait most of the time: their tries take issue slots from the others
    }
    return true;
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(n) : "memory");
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

// Codes are converted in the order in which the products take the tiles: K(0), V(0), K(1), V(1), ..., folded K(0), K(1),
// V(0), K(2), V(1), ..., K(n - 1), V(n - 2), V(n - 1).  The place of a tile in it, and the tile of a place.
__device__ __forceinline__ int chunk_use_k(int i, bool fold) { return fold && i > 0 ? 2 * i - 1 : 2 * i; }
__device__ __forceinline__ int chunk_use_v(int i, int n, bool fold) { return fold && i < n - 1 ? 2 * i + 2 : 2 * i + 1; }
__device__ __forceinline__ void chunk_tile_of(int use, int n, bool fold, int& i, bool& is_v) {
    is_v = fold ? use == 2 * n - 1 || (use > 0 && use % 2 == 0) : use % 2 == 1;
    i = !fold || use == 0 || use == 2 * n - 1 ? use / 2 : is_v ? use / 2 - 1 : (use + 1) / 2;
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

// Whether any of the 64 threads of named barrier `id` says so; a barrier among them.
__device__ __forceinline__ bool pair_any(int id, bool mine) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 64, p;\n\t"
        "selp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(mine ? 1 : 0), "r"(id)
        : "memory");
    return r != 0;
}

// The lowest n bits.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

// max(a, b, c) in one instruction.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
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
    ChunkItem* s_item = reinterpret_cast<ChunkItem*>(sm + S::MISC + 16);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.group, TQ = p.row_tokens, R = 2 * TQ;
    if (warp == 16) {
        // the item: found and worked out once, for the others to read
        const int slot = (gridDim.x - 1 - blockIdx.x) / p.num_kv_heads;  // later rows, which see more, first
        int b, s0, s1, L;
        if (p.num_seqs < 32) {  // one round trip
            const int at = lane <= p.num_seqs ? p.seq_starts[lane] : 0, len = lane < p.num_seqs ? p.context_lens[lane] : 0;
            b = 31 - __clz(__ballot_sync(0xffffffffu, lane < p.num_seqs && at / R + lane <= slot) | 1u);
            s0 = __shfl_sync(0xffffffffu, at, b);
            s1 = __shfl_sync(0xffffffffu, at, b + 1);
            L = __shfl_sync(0xffffffffu, len, b);
        } else {
            b = chunk_find(p.seq_starts, p.num_seqs, R, slot, lane);
            s0 = p.seq_starts[b];
            s1 = p.seq_starts[b + 1];
            L = p.context_lens[b];
        }
        if (lane == 0) {
            const int first = (slot - (s0 / R + b)) * R;  // of the sequence's new tokens
            ChunkItem x;
            x.seq = b;
            x.kvh = (gridDim.x - 1 - blockIdx.x) - slot * p.num_kv_heads;
            x.any = s0 >= 0 && s1 <= p.num_tokens && first >= 0 && first < s1 - s0 && L >= s1 - s0 &&
                    L <= p.max_blocks_per_seq * p.block_size;
            x.row0 = s0 + first;
            x.n = min(R, s1 - s0 - first);
            x.pos0 = L - (s1 - s0) + first;
            x.first_lo = p.window ? max(0, x.pos0 - p.window + 1) : 0;
            x.win_tile0 = x.first_lo / kChunkTile;
            x.sink_tiles = min(x.win_tile0, p.sinks / kChunkTile + (p.sinks % kChunkTile != 0));
            const unsigned tiles = (x.pos0 + x.n - 1) / kChunkTile - x.win_tile0 + 1 + x.sink_tiles;
            x.i0 = x.any ? tiles * blockIdx.y / gridDim.y : 0;  // (at most 2^24 tiles, 32 shares)
            x.i1 = x.any ? tiles * (blockIdx.y + 1) / gridDim.y : 0;
            *s_item = x;
        }
        if (blockIdx.x == 0 && blockIdx.y == 0)  // every sequence's rows and length once
            for (int i = lane; i < p.num_seqs; i += 32) {
                const int s0 = p.seq_starts[i], s1 = p.seq_starts[i + 1], L = p.context_lens[i];
                if (s0 < 0 || s1 < s0 || s1 > p.num_tokens || (s1 > s0 && (L < s1 - s0 || L > p.max_blocks_per_seq * p.block_size)))
                    atomicOr(p.err, kErrBadLen);
            }
    } else if (warp == 19) {
        tc::tmem_alloc(tmem_base_smem, kChunkTmemCols);
        tc::tmem_relinquish();
    } else if (threadIdx.x == 17 * 32) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], E8 ? kConverters : 1);
            mbar_init(&empty[i], 1);
            mbar_init(&v_ok[i], 1);
        }
        for (int i = 0; i < S::NC; ++i) {
            mbar_init(&c_full[i], 1);
            mbar_init(&c_empty[i], kConverters);
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

    const ChunkItem it = *s_item;
    const bool any = it.any;
    const int last = it.pos0 + it.n - 1;  // position of the last row
    const int n_list = it.i1 - it.i0;
    const bool fold = it.n <= TQ;
    // row tile t's first token (folded: both have the same), and its share of the list: up to the tile of its last row
    auto first_of = [&](int t) { return fold ? 0 : t * TQ; };
    auto rows_of = [&](int t) { return min(TQ, it.n - first_of(t)); };
    auto count_of = [&](int t) {
        if (fold) return (n_list + 1 - t) / 2;
        const int rows = rows_of(t);
        const int end = (it.pos0 + t * TQ + rows - 1) / kChunkTile - it.win_tile0 + 1 + it.sink_tiles;
        return max(0, min(n_list, end - it.i0));
    };
    const int cnt0 = count_of(0), cnt1 = count_of(1);
    const int n_run = fold ? n_list : max(cnt0, cnt1);
    const uint64_t policy = l2_policy_evict_normal();  // other row tiles read them too

    // Conversion: warps 20-23, and of a folded item the softmax warps whose 32 rows it has not.
    const int quarters = min(4, (rows_of(0) * G + 31) / 32);
    const bool converter = E8 && (warp >= 20 || (fold && warp < 16 && (warp & 3) >= quarters));
    [[maybe_unused]] const int team = fold ? 4 + 4 * (4 - quarters) : 4;
    [[maybe_unused]] const int index = warp >= 20 ? warp - 20 : 4 + ((warp & 3) - quarters) * 4 + (warp >> 2);

    if (converter) {
        // --------------------------------------------------------- conversion
        // 16 codes a lane and step.  8 neighbouring lanes, which shared memory serves at once, take 64 channels of
        // two tokens (head_dim 128: the other half of the second), so that neither their reads nor their writes,
        // which the swizzle moves by one 16-byte chunk from token to token, meet in a bank.
        if constexpr (E8) {
            // the first one arrives for the warps that are not there
            const uint32_t arrivals = warp == 20 ? 1 + kConverters - team : 1;
            for (int u = 0; u < 2 * n_run; ++u) {
                int tile;
                bool is_v;
                chunk_tile_of(u, n_run, fold, tile, is_v);
                const int code = 2 * tile + is_v, cs = code % S::NC, s = u % NS;
                bool good = chunk_wait(&c_full[cs], (code / S::NC) & 1, abort_flag, p.err);
                if (good && u >= NS) good = chunk_wait(&empty[s], (u / NS - 1) & 1, abort_flag, p.err);
                if (!__all_sync(0xffffffffu, good)) break;
                const unsigned char* codes = sm + S::CODES + cs * S::CSTG;
                unsigned char* dst = ring + s * STG;
                const int start = chunk_tile_start(it, it.i0 + tile);
                const int last_lo = p.window ? max(0, last - p.window + 1) : 0;
                const bool partly = is_v && (start + kChunkTile - 1 > it.pos0 || (start < last_lo && start + kChunkTile > p.sinks));
                constexpr int TOKENS = 32 / (4 * HALVES), GROUPS = kChunkTile / TOKENS;  // tokens of a warp's step, steps
                const int second = (lane >> 2) & 1;
                const int lane_r = HALVES == 2 ? (lane >> 4) * 2 + second : lane >> 2;
                const int h = HALVES == 2 ? ((lane >> 3) & 1) ^ second : 0;
                const int x = (lane & 3) * 2;  // first of two 8-channel chunks of the part
                const unsigned char* src = codes + lane_r * D + h * 64 + x * 8;
                bool bad = false;
                // four steps' codes are read before the first is written; a tile that no row sees in part needs no look
                auto convert = [&](auto look) {
#pragma unroll 1
                    for (int g0 = index; g0 < GROUPS; g0 += 4 * team) {
                        uint4 c[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            if (g0 + y * team < GROUPS)
                                c[y] = *reinterpret_cast<const uint4*>(src + (g0 + y * team) * TOKENS * D);
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            if (g0 + y * team >= GROUPS) break;
                            const int r = (g0 + y * team) * TOKENS + lane_r;
                            if constexpr (decltype(look)::value) {
                                const int j = start + r;
                                if (j > last || (j < it.first_lo && j >= p.sinks)) c[y] = make_uint4(0u, 0u, 0u, 0u);
                                const uint32_t cw[4] = {c[y].x, c[y].y, c[y].z, c[y].w};
#pragma unroll
                                for (int q = 0; q < 4; ++q)  // a code of 0x7f or 0xff
                                    bad = bad || __vcmpeq4(cw[q] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
                            }
                            const uint32_t cw[4] = {c[y].x, c[y].y, c[y].z, c[y].w};
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
                    }
                };
                if (partly) convert(std::true_type{});
                else convert(std::false_type{});
                if constexpr (SCALED)  // a V scale is a factor of weights of 0 too (K's place came first, and its scales)
                    if (partly && lane < 8)
                        bad = bad || !isfinite(reinterpret_cast<const float*>(sm + S::SCALES)[(tile % S::SLOTS) * 24 + 8 + lane]);
                if (bad) *plain_flag = 1;
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_n(&full[s], arrivals);
                    mbar_arrive_n(&c_empty[cs], arrivals);
                }
            }
        }
    } else if (warp < 16) {
        // ------------------------------------------------------------ softmax
        const int t = (warp >> 2) & 1, half = warp >> 3, row = (warp & 3) * 32 + lane;
        const int pair = 1 + (warp & 7);  // named barrier of the two warps of these rows
        const int cnt = t == 0 ? cnt0 : cnt1;
        const int tok = (row * p.inv_group) >> 16, g = row - tok * G;  // (rows past TQ * G and past the last token: none)
        const bool mine = tok < rows_of(t);
        const bool live = __any_sync(0xffffffffu, mine);
        const int pos = mine ? it.pos0 + first_of(t) + tok : -1;
        const int pos_lo = it.pos0 + first_of(t), pos_hi = pos_lo + rows_of(t) - 1;  // of the row tile
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t s_addr = lanes + t * kChunkTile + half * 64;  // this thread's scores, then its weights, packed
        const uint32_t o_addr = lanes + O_COL + t * D + half * (D / 2);
        volatile float* swap = reinterpret_cast<volatile float*>(sm + S::SWAP) + t * kChunkTile + row;
        const float factor = CACHE == kE4M3 ? p.scale_log2 * *p.k_scale : p.scale_log2;
        const float c = SCALED ? 1.f : fmaxf(fabsf(factor), 1e-37f);  // (times -inf: never a NaN, at a factor of 0 either)
        const bool negative = !SCALED && factor < 0.f;
        // reference maximum (log2 units) and this half's sum; block scales: of the logits plus log2 |vs|, the unit of O
        float m = -INFINITY, l = 0.f;
        [[maybe_unused]] float unit = -INFINITY;
        // how far below its maximum the reference (block scales: the unit, by which weights are rounded) is set
        constexpr float LOW = ACT == kF16 ? 7.f : 0.f, LOW_M = SCALED ? 0.f : LOW;
        bool ok = true;
        // Warps without a row have nothing to do; the first one, which has some if any has, arrives for them.
        const uint32_t arrivals = (warp & 3) == 0 ? 1 + 4 - (rows_of(t) * G + 31) / 32 : 1;
        for (int i = 0; live && i < cnt; ++i) {
            ok = __all_sync(0xffffffffu, chunk_wait(&s_full[t], i & 1, abort_flag, p.err));
            tc::fence_after_sync();
            const int tile = fold ? 2 * i + t : i;
            const int start = chunk_tile_start(it, it.i0 + tile) + half * 64;  // this half's first token
            const bool masked = start + 63 > pos_lo || (p.window != 0 && start <= pos_hi - p.window && start + 64 > p.sinks);
            [[maybe_unused]] const float* scales =
                reinterpret_cast<const float*>(sm + S::SCALES) + (SCALED ? (tile % max(1, S::SLOTS)) * 24 : 0);
            [[maybe_unused]] const int block0 = half * 64 / p.block_size, bshift = p.block_size == 32 ? 1 : 0;
            // scores x[0 .. N) from column k on, as loaded, to what `c` makes log2 units
            auto prepare = [&](int k, int n, float* x) {
                if constexpr (SCALED) {
#pragma unroll
                    for (int y = 0; y < n; y += 16) {
                        const float f = factor * scales[block0 + (((k + y) >> 4) >> bshift)];
#pragma unroll
                        for (int j = 0; j < 16; ++j) x[y + j] *= f;
                    }
                } else if (negative) {
#pragma unroll
                    for (int j = 0; j < n; ++j) x[j] = -x[j];
                }
                if (masked) {
                    const int end = pos - start - k;                     // sees columns up to this one
                    const int from = p.window ? end - p.window + 1 : 0;  // and from this one on,
                    const int sink = p.sinks - start - k;                // or before this one
#pragma unroll
                    for (int y = 0; y < n; y += 32) {
                        const uint32_t seen = low_bits(end + 1 - y) & (~low_bits(from - y) | low_bits(sink - y));
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(seen & (1u << j))) x[y + j] = -INFINITY;
                    }
                }
            };
            // 16-bit caches hold a thread's scores; the others, with fewer registers a thread, read them twice
            constexpr int HELD = E8 ? 32 : 64;
            float s[HELD], tops[4];
            [[maybe_unused]] float mu = -INFINITY;
#pragma unroll
            for (int k = 0; k < 64; k += HELD) {
#pragma unroll
                for (int y = 0; y < HELD; y += 32) tc::TmemLd<32>::load(s_addr + k + y, s + y);
                tc::tmem_wait_ld();
                prepare(k, HELD, s);
#pragma unroll
                for (int y = 0; y < HELD; y += 16) {
                    float top = max3(s[y], s[y + 1], s[y + 2]);
#pragma unroll
                    for (int j = 3; j < 15; j += 2) top = max3(top, s[y + j], s[y + j + 1]);
                    tops[(k + y) / 16] = top = fmaxf(top, s[y + 15]);
                    if constexpr (SCALED) mu = fmaxf(mu, top + scales[16 + block0 + (((k + y) >> 4) >> bshift)]);
                }
            }
            float mx = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]) * c;
            const bool past = mine && (mx > m + (LOW_M + kChunkRescale) || (SCALED && mu > unit + (LOW + kChunkRescale)));
            if (pair_any(pair, past || !ok)) {
                // the products of the tiles before are done before the row of O is multiplied
                if (ok && i > 0) {
                    ok = __all_sync(0xffffffffu, chunk_wait(&o_done[t], (i - 1) & 1, abort_flag, p.err));
                    tc::fence_after_sync();
                }
                if (pair_any(pair, !ok)) {  // both leave
                    ok = false;
                    break;
                }
                // the row's maximum, and so its reference, from both threads
                auto agree = [&](float top, float at, float low) {
                    if (half == 1) *swap = top;
                    pair_any(pair, false);
                    float to = at;
                    if (half == 0) {
                        top = fmaxf(top, *swap);
                        if (mine && top > at + (low + kChunkRescale)) to = top - low;
                        *swap = to;
                    }
                    pair_any(pair, false);
                    if (half == 1) to = *swap;
                    return to;
                };
                const float to = agree(mx, m, LOW_M);
                const float down = to == m ? 1.f : fast_exp2(m - to);
                float f = down;
                if constexpr (SCALED) {
                    const float u = agree(mu, unit, LOW);
                    f = u == unit ? 1.f : fast_exp2(unit - u);
                    unit = u;
                }
                l *= down;
                m = to;
                if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
                    for (int k = 0; k < D / 2; k += 8) {
                        float o[8];
                        tc::TmemLd<8>::load(o_addr + k, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[j] *= f;
                        tc::tmem_st<8>(o_addr + k, o);
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                }
                // The product with the first half's weights adds to all of the row, so these are not announced before
                // both halves of it are multiplied.
                if (i > 0) pair_any(pair, false);
            }
            const float ref = m == -INFINITY ? 0.f : m;  // nothing seen yet: weights of 0
            [[maybe_unused]] const float lift = SCALED && unit != -INFINITY ? fast_exp2(ref - unit) : 0.f;
            float sum[4] = {};
#pragma unroll
            for (int k = 0; k < 64; k += 32) {
                float* x = s + (E8 ? 0 : k);
                if constexpr (E8) {
                    tc::TmemLd<32>::load(s_addr + k, x);
                    tc::tmem_wait_ld();
                    prepare(k, 32, x);
                }
                uint32_t w[16];
#pragma unroll
                for (int y = 0; y < 32; y += 16) {
                    [[maybe_unused]] float vf = 1.f;
                    if constexpr (SCALED) vf = lift * scales[8 + block0 + (((k + y) >> 4) >> bshift)];
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        float a = fast_exp2(fmaf(x[y + j], c, -ref));
                        float b = fast_exp2(fmaf(x[y + j + 1], c, -ref));
                        sum[j & 2] += a;
                        sum[(j & 2) + 1] += b;
                        if constexpr (SCALED) {
                            a *= vf;
                            b *= vf;
                        }
                        w[(y + j) / 2] = pack_act<ACT>(a, b);
                    }
                }
                tc::tmem_st16(s_addr + k / 2, w);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_n(&p_full[2 * t + half], arrivals);
        }
        if (live && ok && cnt > 0) {
            ok = __all_sync(0xffffffffu, chunk_wait(&o_done[t], (cnt - 1) & 1, abort_flag, p.err));
            tc::fence_after_sync();
        }
        // folded: both slots' threads of a quarter of the rows (128) go on or stop together
        auto quarter_any = [&](bool say) {
            int r;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.ne.b32 p, %1, 0;\n\t"
                "bar.red.or.pred q, %2, 128, p;\n\t"
                "selp.b32 %0, 1, 0, q;\n\t}"
                : "=r"(r)
                : "r"(say ? 1 : 0), "r"(9 + (warp & 3))
                : "memory");
            return r != 0;
        };
        if (live && any && !(fold ? quarter_any(!ok) : pair_any(pair, !ok))) {
            // the row's sum from both threads
            if (half == 1) *swap = l;
            pair_any(pair, false);
            if (half == 0) *swap = l = l + *swap;
            pair_any(pair, false);
            l = *swap;
            // what an element of O stands for
            float vmul = 1.f;
            if constexpr (CACHE == kE4M3) vmul = *p.v_scale;
            if constexpr (SCALED) vmul = unit == -INFINITY ? 0.f : fast_exp2(unit - m);
            // Folded: slot 1 leaves its maximum, sum and unit; slot 0 reads both slots' O, the same lanes of tensor memory.
            float keep = 1.f, other = 0.f;
            if (fold) {
                float* join = reinterpret_cast<float*>(sm + S::SWAP);  // [m, l], then [vmul]
                quarter_any(false);  // the sums above were read
                if (t == 1 && half == 0) {
                    join[row] = m;
                    join[kChunkTile + row] = l;
                }
                tc::fence_before_sync();
                quarter_any(false);
                tc::fence_after_sync();
                const float m1 = join[row], l1 = join[kChunkTile + row], top = fmaxf(m, m1);
                if constexpr (SCALED) {
                    quarter_any(false);
                    if (t == 1 && half == 0) join[row] = vmul;
                    quarter_any(false);
                    other = join[row];
                } else {
                    other = 1.f;
                }
                if (t == 0) {
                    keep = m == -INFINITY && l == 0.f ? 0.f : fast_exp2(m - top);
                    const float f = m1 == -INFINITY && l1 == 0.f ? 0.f : fast_exp2(m1 - top);
                    l = l * keep + l1 * f;
                    other *= f;
                    m = top;
                }
            }
            // 32 channels of the row from k on, in units of 2^m (per-tensor E4M3: without the scale)
            auto load_o = [&](int k, float* o) {
                tc::TmemLd<32>::load(o_addr + k, o);
                if (fold && cnt1 > 0) {
                    const float f = keep * (CACHE == kE4M3 ? 1.f : vmul);
#pragma unroll
                    for (int x = 0; x < 32; x += 16) {
                        float o1[16];
                        tc::TmemLd<16>::load(o_addr + D + k + x, o1);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[x + j] = o[x + j] * f + o1[j] * other;
                    }
                } else {
                    tc::tmem_wait_ld();
                    if constexpr (SCALED) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] *= vmul;
                    }
                }
            };
            const int64_t at = it.row0 + first_of(t) + tok;
            const int h = it.kvh * G + g;
            const float vt = CACHE == kE4M3 ? vmul : 1.f;
            if (!fold || t == 0) {
                // Rows go out through the row tile's queries' memory, which its last scores have read: 32 rows of 128 bytes
                // a warp and turn, chunks of 16 bytes swizzled by the row; then 8 lanes write 128 bytes of one row (a lane
                // with a row of its own would take 32 lines an instruction).
                unsigned char* stage = qbuf + t * S::QT + (half * 4 + (warp & 3)) * (S::QT / 8);
                static_assert(S::QT / 8 >= 32 * 64, "room for half a turn of each warp");
                constexpr int TURN = S::QT / 8 / 32;  // bytes of a row: 128, or 64 at head_dim 64
                constexpr int CHUNKS = TURN / 16;
                auto put = [&](int x, const uint4& v) {  // chunk x of this thread's row
                    *reinterpret_cast<uint4*>(stage + lane * TURN + ((x ^ (lane & (CHUNKS - 1))) * 16)) = v;
                };
                const int inv_g = p.inv_group;  // (r inv_g) >> 16 = r / G for r < 128, G <= 64
                // the warp's rows, TURN bytes each, to `row_dst(row's index in the item) + offset`
                auto flush = [&](auto row_dst) {
                    __syncwarp();
#pragma unroll
                    for (int y = 0; y < CHUNKS; ++y) {
                        const int r = y * (32 / CHUNKS) + lane / CHUNKS, x = lane % CHUNKS;
                        const int rr = (warp & 3) * 32 + r, rt = (rr * inv_g) >> 16;
                        if (rt < rows_of(t))
                            *reinterpret_cast<uint4*>(row_dst(it.row0 + first_of(t) + rt, it.kvh * G + rr - rt * G) + x * 16) =
                                *reinterpret_cast<const uint4*>(stage + r * TURN + ((x ^ (r & (CHUNKS - 1))) * 16));
                    }
                    __syncwarp();
                };
                if (p.ws_ml != nullptr) {
                    const int64_t share = static_cast<int64_t>(blockIdx.y) * p.num_tokens;
                    if (mine && half == 0) reinterpret_cast<float2*>(p.ws_ml)[(share + at) * p.num_q_heads + h] = make_float2(m, l);
                    if (cnt > 0) {
#pragma unroll
                        for (int k = 0; k < D / 2; k += 32) {
                            float o[32];
                            load_o(k, o);
#pragma unroll
                            for (int y = 0; y < 32; y += TURN / 4) {
#pragma unroll
                                for (int x = 0; x < CHUNKS; ++x)
                                    put(x, make_uint4(__float_as_uint(o[y + 4 * x] * vt), __float_as_uint(o[y + 4 * x + 1] * vt),
                                                      __float_as_uint(o[y + 4 * x + 2] * vt), __float_as_uint(o[y + 4 * x + 3] * vt)));
                                flush([&](int64_t r, int head) {
                                    return reinterpret_cast<unsigned char*>(
                                        p.ws_o + ((share + r) * p.num_q_heads + head) * D + half * (D / 2) + k + y);
                                });
                            }
                        }
                    }
                } else {
                    const float inv = vt / l;
#pragma unroll
                    for (int k = 0; k < D / 2; k += 32) {
                        float o[32];
                        load_o(k, o);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            put((k / 8 + x) % CHUNKS, make_uint4(pack_act<ACT>(o[8 * x] * inv, o[8 * x + 1] * inv),
                                                                 pack_act<ACT>(o[8 * x + 2] * inv, o[8 * x + 3] * inv),
                                                                 pack_act<ACT>(o[8 * x + 4] * inv, o[8 * x + 5] * inv),
                                                                 pack_act<ACT>(o[8 * x + 6] * inv, o[8 * x + 7] * inv)));
                        if ((k + 32) % (TURN / 2) == 0)
                            flush([&](int64_t r, int head) {
                                return reinterpret_cast<unsigned char*>(static_cast<uint16_t*>(p.out) + r * p.out_stride +
                                                                        static_cast<int64_t>(head) * D + half * (D / 2) + (k + 32 - TURN / 2));
                            });
                    }
                }
            }
        }
    } else if (warp == 19) {
        // ---------------------------------------------------------------- MMA
        // Descriptors as words, stepped by additions; one elected lane issues.
        constexpr uint32_t HI = tc::desc_hi_sw128(1024);
        const uint32_t q_lo = tc::desc_start(smem_addr(qbuf)) + tc::desc_lo(16);
        const uint32_t k_lo = tc::desc_start(smem_addr(ring)) + tc::desc_lo(16);
        // V: 16-bit, a block's tokens together, its 64-channel parts v_part apart (the converted tile: as K)
        const uint32_t v_part = E8 ? HALF : p.block_size * 128;
        const uint32_t v_lo = tc::desc_start(smem_addr(ring)) + tc::desc_lo(v_part);
        const uint32_t v_two = E8 || p.block_size == 16 ? 2 * (E8 ? 2048 : 2048 * HALVES) : v_part * HALVES;  // 32 tokens
        const uint32_t v_one = E8 || p.block_size == 32 ? 2048 : 2048 * HALVES;                              // 16 tokens
        auto mma_s = [&](int t, int stage) {
            const uint32_t a = q_lo + (fold ? 0 : t * (S::QT / 16)), b = k_lo + stage * (STG / 16), to = tmem + t * kChunkTile;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * HALF + (kk & 3) * 32) / 16;
                tc::mma_f16_words<HI, HI>(to, a + off, b + off, IDESC_S, kk > 0);
            }
        };
        auto mma_o = [&](int t, int stage, int half, bool add) {  // over 64 tokens
            const uint32_t b = v_lo + stage * (STG / 16) + half * (v_two / 8);
            const uint32_t a = tmem + t * kChunkTile + half * 64, to = tmem + O_COL + t * D;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                tc::mma_f16_ts_words<HI>(to, a + kk * 8, b + (kk >> 1) * (v_two / 16) + (kk & 1) * (v_one / 16), IDESC_O, add || kk > 0);
        };
        bool ok = n_run > 0 && __all_sync(0xffffffffu, chunk_wait(q_full, 0, abort_flag, p.err));
        // K and V of tile i: their stages, and whether they are there
        auto k_use = [&](int i) { return E8 ? chunk_use_k(i, fold) : 2 * i; };
        auto v_use = [&](int i) { return E8 ? chunk_use_v(i, n_run, fold) : 2 * i + 1; };
        auto k_there = [&](int i) {
            const int use = k_use(i);
            return __all_sync(0xffffffffu, chunk_wait(&full[use % NS], (use / NS) & 1, abort_flag, p.err));
        };
        auto v_there = [&](int i) {
            const int use = v_use(i);
            return __all_sync(0xffffffffu, E8 ? chunk_wait(&full[use % NS], (use / NS) & 1, abort_flag, p.err)
                                              : chunk_wait(&v_ok[i % NS], (i / NS) & 1, abort_flag, p.err));
        };
        // O_t += P_t V, the k-th of slot t, half by half as its weights come
        auto product_o = [&](int t, int k, int stage) {
            if (!__all_sync(0xffffffffu, chunk_wait(&p_full[2 * t], k & 1, abort_flag, p.err))) return false;
            tc::fence_after_sync();
            if (tc::elect_one()) mma_o(t, stage, 0, k > 0);
            __syncwarp();
            if (!__all_sync(0xffffffffu, chunk_wait(&p_full[2 * t + 1], k & 1, abort_flag, p.err))) return false;
            tc::fence_after_sync();
            if (tc::elect_one()) {
                mma_o(t, stage, 1, true);
                tc::commit(&o_done[t]);
            }
            __syncwarp();
            return true;
        };
        auto product_s = [&](int t, int stage) {
            if (tc::elect_one()) {
                mma_s(t, stage);
                tc::commit(&s_full[t]);
            }
            __syncwarp();
        };
        auto release = [&](int stage) {
            if (tc::elect_one()) tc::commit(&empty[stage]);
            __syncwarp();
        };
        if (fold) {
            for (int i = 0; i < 2 && i < n_run && ok; ++i) {
                ok = k_there(i);
                if (!ok) break;
                tc::fence_after_sync();
                product_s(i, k_use(i) % NS);
                release(k_use(i) % NS);
            }
            for (int i = 0; i < n_run && ok; ++i) {
                const int t = i & 1;
                ok = v_there(i) && product_o(t, i >> 1, v_use(i) % NS);
                if (!ok) break;
                release(v_use(i) % NS);
                if (i + 2 < n_run) {
                    ok = k_there(i + 2);
                    if (!ok) break;
                    tc::fence_after_sync();
                    product_s(t, k_use(i + 2) % NS);
                    release(k_use(i + 2) % NS);
                }
            }
        } else {
            if (ok) ok = k_there(0);
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
                const int sv = (2 * i + 1) % NS, sk = (2 * i + 2) % NS;
                const bool more = i + 1 < n_run;
                ok = v_there(i) && (!more || k_there(i + 1));
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
        }
        // every product issued has completed before tensor memory is freed
        if (tc::elect_one()) {
            tc::commit(final_bar);
            if (!mbar_wait(final_bar, 0)) atomicOr(p.err, kErrTimeout);
        }
        __syncwarp();
    } else if (warp == 17 || warp == 18) {
        // ---------------------------------------------------------- producers
        const bool second = warp == 18;  // V and Q; else K
        const int BS = p.block_size, bpt = kChunkTile / BS;
        const int32_t* table = p.block_tables + static_cast<int64_t>(it.seq) * p.max_blocks_per_seq;
        // Table entries are asked for two tiles ahead and looked at one tile ahead, so that nothing waits for them (single
        // and drafted tokens, 16 bit: 5 % of the whole call).
        struct Entry {
            int block;
            bool seen;
        };
        auto entry = [&](int i, int j, bool take) {  // of block j of tile i, unless wholly hidden or past the last row's tokens
            const int t0 = chunk_tile_start(it, it.i0 + i) + j * BS;
            const bool seen = take && i < n_run && t0 <= last && (t0 < p.sinks || t0 + BS > it.first_lo);
            return Entry{seen ? table[t0 / BS] : -1, seen};
        };
        auto checked = [&](const Entry& e) {  // -1: none, or outside the pool
            if (e.block >= 0 && e.block < p.num_blocks) return e.block;
            if (e.seen) atomicOr(p.err, kErrBadBlock);
            return -1;
        };
        // this lane's part of a tile: block j, of K channels from 64 kh on (codes: the block)
        const int parts = E8 ? 1 : HALVES;
        const int j = second ? lane : lane / parts, kh = lane % parts;
        const bool take = lane < (second ? bpt : bpt * parts);
        const Entry first = entry(0, j, take);
        Entry ahead = entry(1, j, take);
        int phys = checked(first), issued = 0;
        // its K and V scales, asked for a tile ahead
        auto scales_of = [&](int block) {
            if (!SCALED || second || block < 0) return make_float2(0.f, 0.f);
            const int64_t at = static_cast<int64_t>(block) * p.num_kv_heads + it.kvh;
            return make_float2(p.k_scale[at], p.v_scale[at]);
        };
        [[maybe_unused]] float2 scale = scales_of(phys);
        if (second && lane == 0 && n_run > 0) {
            const uint32_t bytes = HALVES * G * TQ * 128;
            const bool both = !fold && cnt1 > 0;  // (tiles of a share that are all behind row tile 0 leave its queries unused)
            mbar_arrive_expect_tx(q_full, (both ? 2 : 1) * bytes);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (t == 0 || both)
                    for (int h = 0; h < HALVES; ++h)
                        tc::tma_load_3d(qbuf + t * S::QT + h * HALF, &qmap, h * 64, it.kvh * G, it.row0 + t * TQ, q_full, policy);
        }
        for (int i = 0; i < n_run; ++i) {
            const int use = 2 * i + second, next = checked(ahead);
            ahead = entry(i + 2, j, take);
            const int s = use % NP;
            uint64_t* filled = E8 ? &c_full[s] : &full[s];
            [[maybe_unused]] const float2 next_scale = scales_of(next);
            const unsigned loads = __ballot_sync(0xffffffffu, phys >= 0);
            bool good = true;
            if (lane == 0 && use >= NP)
                good = chunk_wait(E8 ? &c_empty[s] : &empty[s], (use / NP - 1) & 1, abort_flag, p.err);
            if (!__shfl_sync(0xffffffffu, good, 0)) break;
            if constexpr (SCALED) {
                if (!second) {
                    if (lane < 8) {
                        float* dst = reinterpret_cast<float*>(sm + S::SCALES) + (i % S::SLOTS) * 24 + lane;
                        dst[0] = scale.x;
                        dst[8] = scale.y;
                        dst[16] = fmaxf(__log2f(fabsf(scale.y)), -100.f);
                    }
                    __syncwarp();  // before the copies' barrier, which the softmax waits on in the end
                }
            }
            if (lane == 0) mbar_arrive_expect_tx(filled, __popc(loads) * (E8 ? BS * D : second ? BS * D * 2 : BS * 128));
            __syncwarp();
            if (phys >= 0) {
                if constexpr (E8) {
                    bulk_copy_g2s(sm + S::CODES + s * S::CSTG + j * BS * D,
                                  static_cast<const unsigned char*>(second ? p.v_cache : p.k_cache) +
                                      (static_cast<int64_t>(phys) * p.num_kv_heads + it.kvh) * (BS * D),
                                  BS * D, filled, policy);
                } else {
                    const int y = (phys * p.num_kv_heads + it.kvh) * BS;
                    if (second) tc::tma_load_3d(ring + s * STG + j * BS * D * 2, &vmap, 0, y, 0, filled, policy);
                    else tc::tma_load_2d(ring + s * STG + kh * HALF + j * BS * 128, &kmap, kh * 64, y, filled, policy);
                }
            }
            phys = next;
            scale = next_scale;
            ++issued;
        }
        // leave only when every copy into this block's shared memory has landed
        if (lane == 0) {
            for (int i = max(0, issued - NP / 2); i < issued; ++i) {
                const int use = 2 * i + second;
                if (!mbar_wait(E8 ? &c_full[use % NP] : &full[use % NP], (use / NP) & 1)) atomicOr(p.err, kErrTimeout);
            }
            if (second && n_run > 0 && !mbar_wait(q_full, 0)) atomicOr(p.err, kErrTimeout);
        }
        __syncwarp();
    } else if (!E8 && warp == 16) {
        // ------------------------------------------------------- V tiles' check
        for (int i = 0; i < n_run; ++i) {
            const int use = 2 * i + 1, s = use % NS;
            if (!__all_sync(0xffffffffu, chunk_wait(&full[s], (use / NS) & 1, abort_flag, p.err))) break;
            const int start = chunk_tile_start(it, it.i0 + i);
            const int last_lo = p.window ? max(0, last - p.window + 1) : 0;  // the last row's window begins here
            if (start + kChunkTile - 1 > it.pos0 || (start < last_lo && start + kChunkTile > p.sinks)) {
                constexpr int CH = 8 * HALVES, STEP = 32 / CH;  // 16-byte chunks of a token, tokens of a warp's access
                const int x = lane % CH, r0 = lane / CH;
                const int bsh = p.block_size == 32 ? 5 : 4, part = p.block_size * 128;
                unsigned char* vb = ring + s * STG + (x >> 3) * part + (x & 7) * 16;
                auto row_at = [&](int r) { return vb + (r >> bsh) * (part * HALVES) + (r & (p.block_size - 1)) * 128; };
                auto clear = [&](int from, int to) {  // tokens [from, to) of the tile
                    for (int r = min(kChunkTile, max(0, from)) + r0; r < min(kChunkTile, to); r += STEP)
                        *reinterpret_cast<uint4*>(row_at(r)) = make_uint4(0u, 0u, 0u, 0u);
                };
                auto look = [&](int from, int to) {
                    bool bad = false;
                    to = min(kChunkTile, to);
                    for (int r = min(kChunkTile, max(0, from)) + r0; r < to; r += 8 * STEP) {
                        uint4 u[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y)
                            u[y] = r + y * STEP < to ? *reinterpret_cast<const uint4*>(row_at(r + y * STEP))
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
    if (warp == 19) tc::tmem_dealloc(tmem, kChunkTmemCols);

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
                for (int y = 0; y < kChunkTile && y <= pos - start; ++y) {
                    const int j = start + y;
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
                    const float w = d == -INFINITY ? 0.f : fast_exp2(d - m);
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
