// Eviction by accumulated attention weight: which tokens of a sequence stay, and
// their move to the blocks of a smaller table; and the accumulation itself.
//
// Of the L tokens of (sequence b, kv head h) the first `sinks`, the last `recent`
// and of the others those with the largest scores stay, min(L, budget) in all,
// in their order (of equal scores the earliest; a NaN counts least).
//
// evict_select_kernel: one block per (b, h).  The scores become 32-bit keys of
// the same order, kept in shared memory (up to kKeyTokens of them; longer rows
// are read again).  The key of the last token that stays is found by radix, 11
// bits from the top, then 11, then 10: a histogram of the keys that agree so far
// and a scan of it from the top.  Then one ordered pass: a thread looks at 4
// neighbouring tokens, and with g tokens above that key and e equal to it before
// a token, its place is g + min(e, equal ones that stay); g and e come from one
// packed scan.
// A small budget's rows move in the same kernel, by the block that chose them.
// Measured: 4 sequences of 270 tokens, 8 heads of 64, to 256: 8.0 us, a launch and a
// dozen dependent passes over shared memory (a call 12.5, 11 to 13 with the host; two launches
// took 4 more); 16 of 4096 to 8192 tokens, 8 heads of 128, to 2048: selection 13 us, bound by its passes too (a
// block an SM, 128 blocks), the move 43, 268 MB at 6.2 TB/s.
// evict_move_kernel: 16 bytes a thread, kept rows of K and V to their new
// blocks; source and destination blocks differ, so that rows are independent.
#include "kernels.h"
#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kKeyTokens = 48 * 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveHere = 64 * 1024;  // bytes of K that the selecting block moves itself
constexpr int kAddThreads = 256;
constexpr int kAddEach = 2;  // tokens a thread
constexpr int kAddTokens = kAddThreads * kAddEach;

// 32-bit key of the scores' order: NaN 0, then -inf .. +inf (-0 as 0).
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return 0;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive sum over the block of each thread's x, and the total (one sync
// before `totals` may be written again is the caller's).
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* totals, uint32_t& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) totals[warp] = incl;
    __syncthreads();
    const uint32_t t = totals[lane];
    uint32_t ti = t;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, ti, off);
        if (lane >= off) ti += v;
    }
    all = __shfl_sync(0xffffffffu, ti, 31);
    return incl - x + __shfl_sync(0xffffffffu, ti - t, warp);
}

// 16 bytes, chunk c of the row, of kept token `from` to place i; false if a table entry is no block.
__device__ __forceinline__ bool move_chunk(const EvictParams& p, int b, int h, int from, int i, int c, int vecs) {
    const int src = p.block_tables[static_cast<int64_t>(b) * p.max_blocks_per_seq + from / p.block_size];
    const int dst = p.dst_tables[static_cast<int64_t>(b) * p.max_dst_blocks + i / p.block_size];
    if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_blocks) return false;
    const int64_t s = ((static_cast<int64_t>(src) * p.num_kv_heads + h) * p.block_size + from % p.block_size) * vecs + c;
    const int64_t d = ((static_cast<int64_t>(dst) * p.num_kv_heads + h) * p.block_size + i % p.block_size) * vecs + c;
    const uint4 k = static_cast<const uint4*>(p.k_cache)[s], v = static_cast<const uint4*>(p.v_cache)[s];
    static_cast<uint4*>(p.k_cache)[d] = k;
    static_cast<uint4*>(p.v_cache)[d] = v;
    return true;
}

// The selection of one (sequence, kv head): kept tokens, their scores; returns how many stay.
__device__ __forceinline__ int evict_select(const EvictParams& p, int h, int b, uint32_t* keys) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t totals[2][kSelectWarps];
    __shared__ uint32_t s_bin, s_rest;
    const int tid = threadIdx.x;
    const int64_t row = static_cast<int64_t>(b) * p.num_kv_heads + h;
    const float* scores = p.scores + row * p.score_tokens;
    int32_t* kept = p.kept + row * p.budget;
    float* out = p.scores_out + row * p.score_tokens_out;
    int L = p.context_lens[b];
    if (L < 0 || L > static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size || L > p.score_tokens) {
        if (h == 0 && tid == 0) atomicOr(p.err, kErrBadLen);
        L = 0;
    }
    int m = min(L, p.budget);
    if (m > static_cast<int64_t>(p.max_dst_blocks) * p.block_size) {  // no room in the new table
        if (h == 0 && tid == 0) atomicOr(p.err, kErrNoSpace);
        L = m = 0;
    }
    if (h == 0 && tid == 0) p.lens_out[b] = m;
    // (unsigned: a step of the block's threads may pass 2^31 - 1)
    const unsigned budget = p.budget, len = L;
    for (unsigned i = m + tid; i < budget; i += kSelectThreads) kept[i] = -1;
    for (int64_t i = m + tid; i < p.score_tokens_out; i += kSelectThreads) out[i] = 0.f;
    if (L <= p.budget) {
        for (unsigned i = tid; i < len; i += kSelectThreads) {
            kept[i] = i;
            out[i] = scores[i];
        }
        return m;
    }
    // the others compete: [sinks, L - recent)
    const unsigned first = p.sinks, last = L - p.recent;
    const bool cached = L <= kKeyTokens;
    auto key_at = [&](unsigned i) { return cached ? keys[i] : score_key(scores[i]); };
    if (cached)
        for (unsigned i = tid; i < len; i += kSelectThreads) keys[i] = score_key(scores[i]);
    uint32_t rest = p.budget - p.sinks - p.recent;  // of them this many stay
    uint32_t found = 0, mask = 0;
    if (rest == 0) {
        found = 0xffffffffu;  // (no key: a NaN's is 0, +inf's 0xff800000)
    } else {
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
            for (int i = tid; i < kBins; i += kSelectThreads) hist[i] = 0;
            __syncthreads();
            for (unsigned i = first + tid; i < last; i += kSelectThreads) {
                const uint32_t k = key_at(i);
                if ((k & mask) == found) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
            }
            __syncthreads();
            // bins from the top, two a thread
            const int hi = kBins - 1 - 2 * tid;
            const uint32_t c1 = hist[hi], c0 = hist[hi - 1];
            uint32_t all;
            const uint32_t before = block_scan(c0 + c1, totals[pass & 1], all);
            if (before < rest && rest <= before + c0 + c1) {
                const bool upper = rest <= before + c1;
                s_bin = upper ? hi : hi - 1;
                s_rest = rest - before - (upper ? 0 : c1);
            }
            __syncthreads();
            found |= s_bin << shift;
            mask |= static_cast<uint32_t>(bins - 1) << shift;
            rest = s_rest;
        }
    }
    __syncthreads();
    // keys above `found` stay, and the first `rest` equal to it
    uint32_t above = 0, equal = 0;
    for (unsigned base = 0, turn = 0; base < len; base += 4 * kSelectThreads, ++turn) {
        uint32_t flags = 0;  // 2 bits a token: 1 above, 2 equal
        const unsigned i0 = base + 4 * tid;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const unsigned i = i0 + j;
            if (i >= len) continue;
            const bool must = i < first || i >= last;
            const uint32_t k = must ? 0 : key_at(i);
            if (must || k > found) flags |= 1u << (2 * j);
            else if (k == found) flags |= 2u << (2 * j);
        }
        const uint32_t mine = __popc(flags & 0x55u) | (__popc(flags & 0xaau) << 16);
        uint32_t all;
        const uint32_t before = block_scan(mine, totals[turn & 1], all);
        uint32_t g = above + (before & 0xffffu), e = equal + (before >> 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t f = (flags >> (2 * j)) & 3u;
            if (f == 1 || (f == 2 && e < rest)) {
                const uint32_t to = g + min(e, rest);
                kept[to] = i0 + j;
                out[to] = scores[i0 + j];
            }
            g += f == 1;
            e += f == 2;
        }
        above += all & 0xffffu;
        equal += all >> 16;
    }
    return m;
}

template <bool MOVE>
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictParams p) {
    extern __shared__ uint32_t keys[];
    asm volatile("griddepcontrol.launch_dependents;");
    const int h = blockIdx.x, b = blockIdx.y;
    const int m = evict_select(p, h, b, keys);
    if constexpr (MOVE) {
        __syncthreads();  // the list of tokens, written by this block's threads
        const int32_t* kept = p.kept + (static_cast<int64_t>(b) * p.num_kv_heads + h) * p.budget;
        const int vecs = p.row_bytes / 16, shift = 31 - __clz(vecs);
        bool good = true;
#pragma unroll 4
        for (int x = threadIdx.x; x < m * vecs; x += kSelectThreads)
            good = move_chunk(p, b, h, kept[x >> shift], x >> shift, x & (vecs - 1), vecs) && good;
        if (!good) atomicOr(p.err, kErrBadBlock);
    }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
    const int vecs = p.row_bytes / 16;  // 4, 8 or 16
    const int rows = kMoveThreads / vecs;
    const int b = blockIdx.z, h = blockIdx.y;
    const int i = blockIdx.x * rows + threadIdx.x / vecs, c = threadIdx.x % vecs;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (i >= p.budget) return;
    const int from = p.kept[(static_cast<int64_t>(b) * p.num_kv_heads + h) * p.budget + i];
    if (from >= 0 && !move_chunk(p, b, h, from, i, c, vecs)) atomicOr(p.err, kErrBadBlock);
}

// What is left once every partition is there, for 512 tokens of a (sequence, kv
// head) a block: scores += sum over the group's heads of 2^(logit - M) / l, one
// thread for every two tokens, (M, l) the statistics of the head's partitions joined; and a
// share of the output's elements, where there are partitions to join (as the
// merge kernel would: sum_i w_i o_i / l with w_i = l_i 2^(m_i - M)).  Rows with a
// partition that went wrong, statistics (0, 0), leave their scores as they are, all
// do where a block of the tensor-core kernel gave up a wait.  Bound by
// the chain of loads of a block; 1, 2 or 4 tokens a thread: 122.5, 119.5 and
// 120.9 us for the call over 64 sequences of up to 4096 tokens, 64 / 8 heads (the
// decode before it 108 by itself, its K and V 80 at the copy's rate).
template <int ACT, int D>
__global__ void __launch_bounds__(kAddThreads) scored_finish_kernel(const AddWeightsParams p) {
    __shared__ float s_max[8], s_inv[8];
    const int seq = blockIdx.z, kvh = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int L = p.context_lens[seq];
    if (L > p.max_context) L = 0;  // flagged before
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kAddTokens;
    if (first >= L) {
        // Nothing to do here.  Each row's first block waits all the same, so that this grid does not end, and what follows
        // it on the stream begin, while the decode still runs.
        if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const int parts = (L - 1) / p.partition_size + 1;
    const int64_t row = static_cast<int64_t>(seq) * p.num_kv_heads + kvh;
    float before[kAddEach], logit[kAddEach][8];
#pragma unroll
    for (int y = 0; y < kAddEach; ++y) {  // not written by the kernel before
        const int64_t t = first + y * kAddThreads + threadIdx.x;
        before[y] = t < L ? p.scores[row * p.score_tokens + t] : 0.f;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
    for (int y = 0; y < kAddEach; ++y) {
        const int64_t t = first + y * kAddThreads + threadIdx.x;
        const float* x = p.logits + (row * p.logit_tokens + t) * p.group;
        if (p.group % 4 == 0) {  // (a token's logits are together)
            const float4 none = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            const float4 a = t < L ? reinterpret_cast<const float4*>(x)[0] : none;
            const float4 b = t < L && p.group == 8 ? reinterpret_cast<const float4*>(x)[1] : none;
            logit[y][0] = a.x, logit[y][1] = a.y, logit[y][2] = a.z, logit[y][3] = a.w;
            logit[y][4] = b.x, logit[y][5] = b.y, logit[y][6] = b.z, logit[y][7] = b.w;
        } else {
#pragma unroll
            for (int g = 0; g < 8; ++g) logit[y][g] = t < L && g < p.group ? x[g] : -INFINITY;
        }
    }
    const float2* stats = reinterpret_cast<const float2*>(p.ws_ml) + row * p.group * p.max_parts;
    bool wrong = threadIdx.x == 0 && p.failed != nullptr && *p.failed != 0;
    auto is_wrong = [](float2 x) { return x.x == 0.f && x.y == 0.f; };  // (a sum has a term of 1 at least, or 2^-inf ones alone)
    if (warp < p.group) {
        const float2* ml = stats + warp * p.max_parts;
        const float2 mine = lane < parts ? ml[lane] : make_float2(-INFINITY, 0.f);
        wrong = wrong || (lane < parts && is_wrong(mine));
        float M = mine.x;
        for (int i = 32 + lane; i < parts; i += 32) {
            wrong = wrong || is_wrong(ml[i]);
            M = fmaxf(M, ml[i].x);
        }
        M = warp_max(M);
        float l = lane < parts ? mine.y * fast_exp2(mine.x - M) : 0.f;
        for (int i = 32 + lane; i < parts; i += 32) l += ml[i].y * fast_exp2(ml[i].x - M);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        if (lane == 0) {
            s_max[warp] = M;
            s_inv[warp] = 1.f / l;
        }
    }
    wrong = __syncthreads_or(wrong);
#pragma unroll
    for (int y = 0; y < kAddEach; ++y) {
        const int64_t t = first + y * kAddThreads + threadIdx.x;
        if (t >= L || wrong) break;
        float sum = 0.f;
#pragma unroll
        for (int g = 0; g < 8; ++g)
            if (g < p.group) sum += fast_exp2(logit[y][g] - s_max[g]) * s_inv[g];
        p.scores[row * p.score_tokens + t] = before[y] + sum;
    }
    if (parts == 1) return;
    const int blocks = (L - 1) / kAddTokens + 1, each = (p.group * D + blocks - 1) / blocks;
    const int end = min(p.group * D, static_cast<int>(blockIdx.x + 1) * each);
    for (int e = blockIdx.x * each + threadIdx.x; e < end; e += kAddThreads) {
        const int g = e / D, d = e % D;
        const float2* ml = stats + g * p.max_parts;
        const float* o = p.ws_o + (row * p.group + g) * p.max_parts * D + d;
        float acc = 0.f;
#pragma unroll 4
        for (int i = 0; i < parts; ++i) acc = fmaf(ml[i].y * fast_exp2(ml[i].x - s_max[g]), o[static_cast<int64_t>(i) * D], acc);
        static_cast<uint16_t*>(p.out)[(row * p.group + g) * D + d] = float_to_act<ACT>(acc * s_inv[g]);
    }
}

template <class Params>
cudaError_t launch_after(void (*kernel)(const Params), const Params& p, dim3 grid, int threads, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
    static bool configured[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeyTokens * 4);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(evict_select_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeyTokens * 4);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    const int64_t most = static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size;
    const int smem = static_cast<int>((most < kKeyTokens ? most : kKeyTokens) * 4);
    const dim3 heads(p.num_kv_heads, p.num_seqs);
    const int64_t stay = p.budget < most ? p.budget : most;  // tokens of a row that may
    if (stay * p.row_bytes <= kMoveHere) {
        evict_select_kernel<true><<<heads, kSelectThreads, smem, stream>>>(p);
        return cudaGetLastError();
    }
    evict_select_kernel<false><<<heads, kSelectThreads, smem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int rows = kMoveThreads / (p.row_bytes / 16);
    const dim3 grid(static_cast<unsigned>((stay + rows - 1) / rows), p.num_kv_heads, p.num_seqs);
    return launch_after(evict_move_kernel, p, grid, kMoveThreads, stream);
}

cudaError_t launch_scored_finish(const AddWeightsParams& p, int act, int head_dim, cudaStream_t stream) {
    const dim3 grid((p.max_context - 1) / kAddTokens + 1, p.num_kv_heads, p.num_seqs);
    auto kernel = head_dim == 64 ? (act == kBF16 ? scored_finish_kernel<kBF16, 64> : scored_finish_kernel<kF16, 64>)
                                 : (act == kBF16 ? scored_finish_kernel<kBF16, 128> : scored_finish_kernel<kF16, 128>);
    return launch_after(kernel, p, grid, kAddThreads, stream);
}

}  // namespace pkv
