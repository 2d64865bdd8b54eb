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
// Every barrier wait is bounded (kWaitLimitNs); on a timeout the block stops,
// drains its copies and products, frees tensor memory and reports kErrTimeout.
#pragma once

#include "kernels.h"
#include "pkv_tc.cuh"

namespace pkv {

constexpr int kChunkThreads = 384;
constexpr int kChunkTile = 128;       // tokens of a tile
constexpr int kChunkTmemCols = 512;   // two S (128 columns each, P over them), two O
constexpr float kChunkRescale = 8.f;  // log2 by which a maximum may pass the reference

template <int D>
struct ChunkSmem {
    static constexpr int HALVES = D / 64;
    static constexpr int STG = kChunkTile * D * 2;  // a K or V tile: per 64 channels 128 rows of 128 bytes
    static constexpr int NS = D == 128 ? 5 : 8;
    static constexpr int QT = kChunkTile * D * 2;
    static constexpr int RING = 0;
    static constexpr int Q = NS * STG;
    static constexpr int BARS = Q + 2 * QT;
    static constexpr int NBARS = 3 * NS + 8;  // full, empty, v_ok, q_full, s_full[2], p_full[2], o_done[2], final
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
    bool bad = false;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t e = w[i] & EXP;
        bad = bad || (e & 0xffffu) == (EXP & 0xffffu) || (e >> 16) == (EXP >> 16);
    }
    return bad;
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

template <int ACT, int D>
__global__ void __launch_bounds__(kChunkThreads, 1)
    paged_chunk_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                          const __grid_constant__ CUtensorMap qmap, const ChunkParams p) {
    using S = ChunkSmem<D>;
    constexpr int NS = S::NS, STG = S::STG, HALVES = S::HALVES, HALF = kChunkTile * 128;
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
    uint64_t* q_full = v_ok + NS;
    uint64_t* s_full = q_full + 1;
    uint64_t* p_full = s_full + 2;
    uint64_t* o_done = p_full + 2;
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
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            mbar_init(&v_ok[i], 1);
        }
        mbar_init(q_full, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], 4);
            mbar_init(&o_done[t], 1);
        }
        mbar_init(final_bar, 1);
        *abort_flag = 0;
        *plain_flag = 0;
        mbar_init_fence();
        tc::prefetch_tensormap(&kmap);
        tc::prefetch_tensormap(&vmap);
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
        const float c = fmaxf(fabsf(p.scale_log2), 1e-37f);  // (times -inf: never a NaN, at a scale of 0 either)
        const bool negative = p.scale_log2 < 0.f;
        float m = -INFINITY, l = 0.f;  // reference maximum (log2 units) and sum
        bool ok = true;
        for (int i = 0; i < cnt && ok; ++i) {
            ok = __all_sync(0xffffffffu, chunk_wait(&s_full[t], i & 1, abort_flag, p.err));
            if (!ok) break;
            tc::fence_after_sync();
            if (live) {
                float s[kChunkTile];
#pragma unroll
                for (int k = 0; k < kChunkTile; k += 32) tc::TmemLd<32>::load(s_addr + k, s + k);
                tc::tmem_wait_ld();
                if (negative) {
#pragma unroll
                    for (int k = 0; k < kChunkTile; ++k) s[k] = -s[k];
                }
                const int start = chunk_tile_start(it, it.i0 + i);
                if (start + kChunkTile - 1 > pos_lo ||
                    (p.window != 0 && start <= pos_hi - p.window && start + kChunkTile > p.sinks)) {
                    const int end = pos - start;                            // sees columns up to this one
                    const int from = p.window ? end - p.window + 1 : 0;     // and from this one on,
                    const int sink = p.sinks - start;                       // or before this one
#pragma unroll
                    for (int k = 0; k < kChunkTile; ++k)
                        if (k > end || (k < from && k >= sink)) s[k] = -INFINITY;
                }
                float mx = s[0];
#pragma unroll
                for (int k = 1; k < kChunkTile; ++k) mx = fmaxf(mx, s[k]);
                mx *= c;
                const bool move = mine && mx > m + kChunkRescale;
                if (__any_sync(0xffffffffu, move && l > 0.f)) {
                    // O holds the tiles before: their products are done, then the row is multiplied
                    ok = __all_sync(0xffffffffu, chunk_wait(&o_done[t], (i - 1) & 1, abort_flag, p.err));
                    if (!ok) break;
                    tc::fence_after_sync();
                    const float f = move ? fast_exp2(m - mx) : 1.f;
                    l *= f;
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
                if (move) m = mx;
                const float ref = m == -INFINITY ? 0.f : m;  // nothing seen yet: weights of 0
                float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
                for (int k = 0; k < kChunkTile; k += 64) {
                    uint32_t w[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float a = fast_exp2(fmaf(s[k + 2 * j], c, -ref));
                        const float b = fast_exp2(fmaf(s[k + 2 * j + 1], c, -ref));
                        sum0 += a;
                        sum1 += b;
                        w[j] = pack_act<ACT>(a, b);
                    }
                    tc::tmem_st32(s_addr + k / 2, w);
                }
                l += sum0 + sum1;
                tc::tmem_wait_st();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[t]);
        }
        if (ok && cnt > 0) {
            ok = __all_sync(0xffffffffu, chunk_wait(&o_done[t], (cnt - 1) & 1, abort_flag, p.err));
            tc::fence_after_sync();
        }
        if (ok && live && any) {
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
                        for (int j = 0; j < 4; ++j) dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    }
                }
            } else {
                const float inv = 1.f / l;
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
        auto mma_o = [&](int t, int stage, bool add) {
            const uint32_t b = k_base + stage * STG;
#pragma unroll
            for (int kk = 0; kk < kChunkTile / 16; ++kk)
                tc::mma_f16_ts(tmem + O_COL + t * D, tmem + t * kChunkTile + kk * 8, tc::desc_sw128(b + kk * 2048, HALF, 1024),
                               IDESC_O, add || kk > 0);
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
            ok = __all_sync(0xffffffffu, chunk_wait(&v_ok[i % NS], (i / NS) & 1, abort_flag, p.err));
            if (!ok) break;
            if (more) ok = __all_sync(0xffffffffu, chunk_wait(&full[sk], (uk / NS) & 1, abort_flag, p.err));
            if (!ok) break;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int cnt = t == 0 ? cnt0 : cnt1;
                if (i >= cnt) continue;
                ok = __all_sync(0xffffffffu, chunk_wait(&p_full[t], i & 1, abort_flag, p.err));
                if (!ok) break;
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    mma_o(t, sv, i > 0);
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
        const int j = lane / HALVES, h = lane % HALVES;  // block of the tile and 64-channel part of this lane
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
            const int use = 2 * i + v, s = use % NS;
            const int next = entry(i + 1);
            const unsigned loads = __ballot_sync(0xffffffffu, phys >= 0);
            bool good = true;
            if (lane == 0) {
                if (use >= NS) good = chunk_wait(&empty[s], (use / NS - 1) & 1, abort_flag, p.err);
                if (good) mbar_arrive_expect_tx(&full[s], __popc(loads) * BS * 128);
            }
            if (!__shfl_sync(0xffffffffu, good, 0)) break;
            if (phys >= 0)
                tc::tma_load_2d(ring + s * STG + h * HALF + j * BS * 128, map, h * 64, (phys * p.num_kv_heads + it.kvh) * BS,
                                &full[s], policy);
            phys = next;
            ++issued;
        }
        // leave only when every copy into this block's shared memory has landed
        if (lane == 0) {
            for (int i = max(0, issued - NS); i < issued; ++i) {
                const int use = 2 * i + v;
                if (use + NS >= 2 * issued && !mbar_wait(&full[use % NS], (use / NS) & 1)) atomicOr(p.err, kErrTimeout);
            }
            if (v == 0 && n_run > 0 && !mbar_wait(q_full, 0)) atomicOr(p.err, kErrTimeout);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------- V tiles' check
        for (int i = 0; i < n_run; ++i) {
            const int use = 2 * i + 1, s = use % NS;
            if (!__all_sync(0xffffffffu, chunk_wait(&full[s], (use / NS) & 1, abort_flag, p.err))) break;
            const int start = chunk_tile_start(it, it.i0 + i);
            const int last_lo = p.window ? max(0, last - p.window + 1) : 0;  // the last row's window begins here
            if (start + kChunkTile - 1 > it.pos0 || (start < last_lo && start + kChunkTile > p.sinks)) {
                unsigned char* vb = ring + s * STG;
                bool bad = false;
                // a token's row is HALVES parts of 8 chunks; 4 / HALVES tokens a turn of the warp
                constexpr int CH = 8 * HALVES;
                for (int k = lane; k < kChunkTile * CH; k += 32) {
                    const int r = k / CH, x = k % CH, j = start + r;
                    uint4* at = reinterpret_cast<uint4*>(vb + (x >> 3) * HALF + r * 128 + (x & 7) * 16);
                    if (j > last || (j < it.first_lo && j >= p.sinks)) *at = make_uint4(0u, 0u, 0u, 0u);
                    else bad = bad || any_not_finite<ACT>(*at);
                }
                if (bad) *plain_flag = 1;
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
        const uint16_t *kc = static_cast<const uint16_t*>(p.k_cache), *vc = static_cast<const uint16_t*>(p.v_cache);
        const int32_t* table = p.block_tables + static_cast<int64_t>(it.seq) * p.max_blocks_per_seq;
        for (int r = warp; r < it.n * G; r += kChunkThreads / 32) {
            const int64_t at = it.row0 + r / G;
            const int pos = it.pos0 + r / G, h = it.kvh * G + r % G;
            const uint16_t* q = static_cast<const uint16_t*>(p.q) + at * p.q_stride + static_cast<int64_t>(h) * D;
            float qf[W], acc[W] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
            for (int x = 0; x < W; ++x) qf[x] = act_to_float<ACT>(q[lane + 32 * x]) * p.scale_log2;
            const int lo = p.window ? max(0, pos - p.window + 1) : 0;
            for (int i = it.i0; i < it.i1; ++i) {
                const int start = chunk_tile_start(it, i);
                for (int j = start; j < start + kChunkTile && j <= pos; ++j) {
                    if (j < lo && j >= p.sinks) continue;
                    const int blk = table[j / p.block_size];
                    if (blk < 0 || blk >= p.num_blocks) continue;
                    const int64_t src = ((static_cast<int64_t>(blk) * p.num_kv_heads + it.kvh) * p.block_size + j % p.block_size) * D;
                    float d = 0.f;
#pragma unroll
                    for (int x = 0; x < W; ++x) d = fmaf(qf[x], act_to_float<ACT>(kc[src + lane + 32 * x]), d);
#pragma unroll
                    for (int off = 16; off >= 1; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
                    if (d > m) {
                        const float f = fast_exp2(m - d);
                        l *= f;
#pragma unroll
                        for (int x = 0; x < W; ++x) acc[x] *= f;
                        m = d;
                    }
                    const float w = fast_exp2(d - m);
                    l += w;
#pragma unroll
                    for (int x = 0; x < W; ++x) acc[x] = fmaf(w, act_to_float<ACT>(vc[src + lane + 32 * x]), acc[x]);
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
