// Block tables, slots and positions of a step's tokens, built on the GPU.
//
// For request b with c_b tokens in the cache and n_b new ones, block size bs:
//   h_b = ceil(c_b / bs) blocks there, t_b = ceil((c_b + n_b) / bs) - h_b to take;
//   seq_starts = exclusive prefix sum of n, block_starts = exclusive prefix sum of t;
//   logical block j >= h_b of b is free_blocks[head + block_starts[b] + j - h_b];
//   token i of b has position c_b + i and slot table[b][pos / bs] * bs + pos % bs.
// This is the order in which the host block manager pops its free list, so
// host and device make the same tables from the same requests.
//
// Nothing here computes; a step costs its launch and, for prompts, the 12
// bytes written per token.  Up to kMaxShared requests: one launch, in which
// every block scans all requests into shared memory (every thread a contiguous
// chunk of them, one block-wide scan of the chunk sums), so that each takes the
// same all-or-nothing decision, the first block writes the per-request outputs
// and each expands its tokens, four neighbours a thread (one binary search over
// the starts, 16-byte stores).  Lengths or a head updated in place would be
// read by one block after another has written them: several blocks then run as
// two launches, as do more requests: one block scans, then tokens expand from
// the outputs.  Measured (GPU time): 64 requests of one token 4.7 us, 64
// prompts of 263 thousand tokens 4.8 us (two launches: 5.4 and 7.5 us).
#include "kernels.h"
#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kScanThreads = 1024;
constexpr int kMaxShared = 2048;  // requests of the one-launch form
constexpr int kExpandThreads = 256;
constexpr int kTokensPerThread = 4;

// The requests' scanned numbers, in the outputs or in shared memory.
struct ScannedOutputs {
    const ExtendParams& p;
    int head0;  // head before this call
    __device__ __forceinline__ explicit ScannedOutputs(const ExtendParams& q)
        : p(q), head0(*q.free_head_out - q.block_starts[q.num_seqs]) {}
    __device__ __forceinline__ int start(int b) const { return p.seq_starts[b]; }
    __device__ __forceinline__ int blocks(int b) const { return p.block_starts[b]; }
    __device__ __forceinline__ int ctx(int b) const { return p.lens_out[b] - p.new_lens[b]; }
};
struct ScannedShared {
    const int *starts, *takes, *lens;
    int head0;
    __device__ __forceinline__ int start(int b) const { return starts[b]; }
    __device__ __forceinline__ int blocks(int b) const { return takes[b]; }
    __device__ __forceinline__ int ctx(int b) const { return lens[b]; }
};

// Four consecutive tokens from t0: slots and positions, and the table entry of
// each new block by the token that is first in it.
template <class Scanned>
__device__ __forceinline__ void expand_tokens(const ExtendParams& p, const Scanned& q, int t0) {
    const int B = p.num_seqs;
    const int total = q.start(B);
    int64_t slots[kTokensPerThread];
    int pos_out[kTokensPerThread];
    int b = 0;
    if (t0 < total) {  // the last request that starts at or before t0 (empty ones before it are passed over)
        int lo = 0, hi = B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (q.start(mid) <= t0) lo = mid;
            else hi = mid;
        }
        b = lo;
    }
#pragma unroll
    for (int i = 0; i < kTokensPerThread; ++i) {
        const int t = t0 + i;
        slots[i] = -1;
        pos_out[i] = -1;
        if (t >= total) continue;
        while (t >= q.start(b + 1)) ++b;
        const int ctx = q.ctx(b);
        const int pos = ctx + (t - q.start(b));
        const int j = pos / p.block_size, off = pos - j * p.block_size;
        const int have = (ctx + p.block_size - 1) / p.block_size;
        int32_t* row = p.block_tables + static_cast<int64_t>(b) * p.max_blocks_per_seq;
        int phys;
        if (j < have) {
            phys = row[j];
        } else {
            phys = p.free_blocks[q.head0 + q.blocks(b) + (j - have)];
            if (off == 0) row[j] = phys;
        }
        pos_out[i] = pos;
        if (phys < 0 || phys >= p.num_blocks) atomicOr(p.err, kErrBadBlock);
        else slots[i] = static_cast<int64_t>(phys) * p.block_size + off;
    }
    if (t0 + kTokensPerThread <= p.num_tokens) {
        *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos_out[0], pos_out[1], pos_out[2], pos_out[3]);
        *reinterpret_cast<longlong2*>(p.slot_mapping + t0) = make_longlong2(slots[0], slots[1]);
        *reinterpret_cast<longlong2*>(p.slot_mapping + t0 + 2) = make_longlong2(slots[2], slots[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kTokensPerThread; ++i) {
            if (t0 + i < p.num_tokens) {
                p.positions[t0 + i] = pos_out[i];
                p.slot_mapping[t0 + i] = slots[i];
            }
        }
    }
}

__device__ __forceinline__ int64_t warp_inclusive_scan(int64_t x, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += v;
    }
    return x;
}

// Scan of the requests by one block of THREADS threads.  visit(b, ctx, starts,
// takes) sees each request with its exclusive sums; returns the step's totals
// and whether it is refused (then the sums are of no use).
struct ScanResult {
    int64_t tokens, blocks;
    int err;
};
template <int THREADS, class Visit>
__device__ __forceinline__ ScanResult scan_requests(const ExtendParams& p, int head, Visit visit) {
    constexpr int WARPS = THREADS / 32;
    __shared__ int64_t s_new[WARPS], s_take[WARPS];
    __shared__ int s_bad;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = p.num_seqs;
    const int chunk = (B + THREADS - 1) / THREADS;
    const int b0 = min(B, tid * chunk), b1 = min(B, b0 + chunk);
    if (tid == 0) s_bad = 0;
    __syncthreads();
    auto blocks_of = [&](int64_t tokens) { return (tokens + p.block_size - 1) / p.block_size; };
    int64_t n_new = 0, n_take = 0;
    int bad = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t c = p.context_lens[b], n = p.new_lens[b];
        if (c < 0 || n < 0 || c + n > static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size) {
            bad = kErrBadLen;
            continue;
        }
        n_new += n;
        n_take += blocks_of(c + n) - blocks_of(c);
    }
    int64_t i_new = warp_inclusive_scan(n_new, lane), i_take = warp_inclusive_scan(n_take, lane);
    if (lane == 31) {
        s_new[warp] = i_new;
        s_take[warp] = i_take;
    }
    if (bad) atomicOr(&s_bad, bad);
    __syncthreads();
    ScanResult r{0, 0, s_bad};
    int64_t run_new = i_new - n_new, run_take = i_take - n_take;
#pragma unroll 8
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) {
            run_new += s_new[w];
            run_take += s_take[w];
        }
        r.tokens += s_new[w];
        r.blocks += s_take[w];
    }
    if (r.tokens > p.num_tokens || head < 0 || head + r.blocks > p.num_free) r.err |= kErrNoSpace;
    for (int b = b0; b < b1; ++b) {
        const int c = p.context_lens[b], n = p.new_lens[b];
        visit(b, c, n, r.err ? 0 : static_cast<int>(run_new), r.err ? 0 : static_cast<int>(run_take));
        if (!r.err) {  // all or nothing: a refused step has no tokens
            run_new += n;
            run_take += blocks_of(static_cast<int64_t>(c) + n) - blocks_of(c);
        }
    }
    return r;
}

// What one thread writes of the totals.
__device__ __forceinline__ void write_totals(const ExtendParams& p, const ScanResult& r, int head) {
    p.seq_starts[p.num_seqs] = r.err ? 0 : static_cast<int>(r.tokens);
    p.block_starts[p.num_seqs] = r.err ? 0 : static_cast<int>(r.blocks);
    *p.free_head_out = r.err ? head : static_cast<int>(head + r.blocks);
    if (r.err) atomicOr(p.err, r.err);
}

// At most kMaxShared requests, one launch.
__global__ void __launch_bounds__(kExpandThreads) extend_kernel(const ExtendParams p) {
    __shared__ int s_starts[kMaxShared + 1], s_takes[kMaxShared + 1], s_lens[kMaxShared];
    const int head = *p.free_head;
    const bool writes = blockIdx.x == 0;
    const ScanResult r = scan_requests<kExpandThreads>(p, head, [&](int b, int c, int n, int start, int take) {
        s_starts[b] = start;
        s_takes[b] = take;
        s_lens[b] = c;
    });
    if (threadIdx.x == 0) {
        s_starts[p.num_seqs] = r.err ? 0 : static_cast<int>(r.tokens);
        s_takes[p.num_seqs] = r.err ? 0 : static_cast<int>(r.blocks);
    }
    __syncthreads();  // and every thread of a lone block has read the lengths and the head
    if (writes) {
        for (int b = threadIdx.x; b < p.num_seqs; b += kExpandThreads) {
            p.seq_starts[b] = s_starts[b];
            p.block_starts[b] = s_takes[b];
            p.lens_out[b] = s_lens[b] + (s_starts[b + 1] - s_starts[b]);
        }
        if (threadIdx.x == 0) write_totals(p, r, head);
    }
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kExpandThreads + threadIdx.x) * kTokensPerThread;
    if (t0 < p.num_tokens) expand_tokens(p, ScannedShared{s_starts, s_takes, s_lens, head}, static_cast<int>(t0));
}

// Any number of requests: one block scans (FUSED: and expands), or a second
// launch expands.
template <bool FUSED>
__global__ void __launch_bounds__(kScanThreads) extend_scan_kernel(const ExtendParams p) {
    const int head = *p.free_head;
    const ScanResult r = scan_requests<kScanThreads>(p, head, [&](int b, int c, int n, int start, int take) {
        p.seq_starts[b] = start;
        p.block_starts[b] = take;
    });
    __syncthreads();  // every thread has read the lengths and the head before they may be updated in place
    for (int b = threadIdx.x; b < p.num_seqs; b += kScanThreads)
        p.lens_out[b] = p.context_lens[b] + (r.err ? 0 : p.new_lens[b]);
    if (threadIdx.x == 0) write_totals(p, r, head);
    if constexpr (FUSED) {
        __syncthreads();
        const ScannedOutputs q(p);
        for (int t0 = threadIdx.x * kTokensPerThread; t0 < p.num_tokens; t0 += kScanThreads * kTokensPerThread)
            expand_tokens(p, q, t0);
    }
}

__global__ void __launch_bounds__(kExpandThreads) extend_expand_kernel(const ExtendParams p) {
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kExpandThreads + threadIdx.x) * kTokensPerThread;
    if (t0 < p.num_tokens) expand_tokens(p, ScannedOutputs(p), static_cast<int>(t0));
}

// Whether two int32 buffers share memory.
bool overlap(const int32_t* a, int64_t na, const int32_t* b, int64_t nb) { return a < b + nb && b < a + na; }

}  // namespace

cudaError_t launch_extend_tables(const ExtendParams& p, cudaStream_t stream) {
    const int per = kExpandThreads * kTokensPerThread;
    const int blocks = p.num_tokens > 0 ? (p.num_tokens - 1) / per + 1 : 1;
    if (p.num_seqs <= kMaxShared &&
        (blocks == 1 || !(overlap(p.lens_out, p.num_seqs, p.context_lens, p.num_seqs) ||
                          overlap(p.lens_out, p.num_seqs, p.new_lens, p.num_seqs) ||
                          overlap(p.free_head_out, 1, p.free_head, 1)))) {
        extend_kernel<<<blocks, kExpandThreads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    if (p.num_tokens <= kScanThreads * kTokensPerThread) {
        extend_scan_kernel<true><<<1, kScanThreads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    extend_scan_kernel<false><<<1, kScanThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    extend_expand_kernel<<<blocks, kExpandThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pkv
