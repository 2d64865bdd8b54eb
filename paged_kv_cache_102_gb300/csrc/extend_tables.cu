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
// Nothing here computes; a step costs its launches and, for prompts, the 12
// bytes written per token.  One block scans the requests (every thread a
// contiguous chunk of them, one block-wide scan of the chunk sums), which
// takes all-or-nothing decisions before anything is written.  Tokens then
// expand in parallel, four neighbours a thread (one binary search over
// seq_starts, 16-byte stores).
#include "kernels.h"
#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kScanThreads = 1024;
constexpr int kExpandThreads = 256;
constexpr int kTokensPerThread = 4;

// Four consecutive tokens from t0: slots and positions, and the table entry of
// each new block by the token that is first in it.
__device__ __forceinline__ void expand_tokens(const ExtendParams& p, int t0) {
    const int B = p.num_seqs;
    const int total = p.seq_starts[B];
    int64_t slots[kTokensPerThread];
    int pos_out[kTokensPerThread];
    int b = 0;
    if (t0 < total) {  // the last request that starts at or before t0 (empty ones before it are passed over)
        int lo = 0, hi = B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.seq_starts[mid] <= t0) lo = mid;
            else hi = mid;
        }
        b = lo;
    }
    const int head0 = *p.free_head_out - p.block_starts[B];  // head before this call
#pragma unroll
    for (int i = 0; i < kTokensPerThread; ++i) {
        const int t = t0 + i;
        slots[i] = -1;
        pos_out[i] = -1;
        if (t >= total) continue;
        while (t >= p.seq_starts[b + 1]) ++b;
        const int ctx = p.lens_out[b] - p.new_lens[b];
        const int pos = ctx + (t - p.seq_starts[b]);
        const int j = pos / p.block_size, off = pos - j * p.block_size;
        const int have = (ctx + p.block_size - 1) / p.block_size;
        int32_t* row = p.block_tables + static_cast<int64_t>(b) * p.max_blocks_per_seq;
        int phys;
        if (j < have) {
            phys = row[j];
        } else {
            phys = p.free_blocks[head0 + p.block_starts[b] + (j - have)];
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

// One block: scan, decide, write the per-request outputs; FUSED: the tokens too.
template <bool FUSED>
__global__ void __launch_bounds__(kScanThreads) extend_scan_kernel(const ExtendParams p) {
    __shared__ int64_t s_new[kScanThreads / 32], s_take[kScanThreads / 32];
    __shared__ int s_bad;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = p.num_seqs;
    const int chunk = (B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(B, tid * chunk), b1 = min(B, b0 + chunk);
    if (tid == 0) s_bad = 0;
    __syncthreads();
    int64_t n_new = 0, n_take = 0;
    int bad = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t c = p.context_lens[b], n = p.new_lens[b];
        if (c < 0 || n < 0 || c + n > static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size) {
            bad = kErrBadLen;
            continue;
        }
        n_new += n;
        n_take += (c + n + p.block_size - 1) / p.block_size - (c + p.block_size - 1) / p.block_size;
    }
    int64_t i_new = warp_inclusive_scan(n_new, lane), i_take = warp_inclusive_scan(n_take, lane);
    if (lane == 31) {
        s_new[warp] = i_new;
        s_take[warp] = i_take;
    }
    if (bad) atomicOr(&s_bad, bad);
    __syncthreads();
    if (warp == 0) {
        const int nw = blockDim.x / 32;
        int64_t a = lane < nw ? s_new[lane] : 0, c = lane < nw ? s_take[lane] : 0;
        a = warp_inclusive_scan(a, lane);
        c = warp_inclusive_scan(c, lane);
        if (lane < nw) {
            s_new[lane] = a;
            s_take[lane] = c;
        }
    }
    __syncthreads();
    const int nw = blockDim.x / 32;
    const int64_t total_new = s_new[nw - 1], total_take = s_take[nw - 1];
    const int head = *p.free_head;
    int err = s_bad;
    if (total_new > p.num_tokens || head < 0 || head + total_take > p.num_free) err |= kErrNoSpace;
    int64_t run_new = i_new - n_new + (warp ? s_new[warp - 1] : 0);
    int64_t run_take = i_take - n_take + (warp ? s_take[warp - 1] : 0);
    for (int b = b0; b < b1; ++b) {
        const int c = p.context_lens[b];
        int n = p.new_lens[b];
        if (err) n = 0;  // all or nothing: a refused step has no tokens
        p.seq_starts[b] = err ? 0 : static_cast<int>(run_new);
        p.block_starts[b] = err ? 0 : static_cast<int>(run_take);
        run_new += n;
        if (!err)
            run_take += (static_cast<int64_t>(c) + n + p.block_size - 1) / p.block_size -
                        (static_cast<int64_t>(c) + p.block_size - 1) / p.block_size;
        p.lens_out[b] = c + n;
    }
    __syncthreads();  // every thread has read the head before it may be updated in place
    if (tid == 0) {
        p.seq_starts[B] = err ? 0 : static_cast<int>(total_new);
        p.block_starts[B] = err ? 0 : static_cast<int>(total_take);
        *p.free_head_out = err ? head : static_cast<int>(head + total_take);
        if (err) atomicOr(p.err, err);
    }
    if constexpr (FUSED) {
        __syncthreads();
        for (int t0 = tid * kTokensPerThread; t0 < p.num_tokens; t0 += blockDim.x * kTokensPerThread)
            expand_tokens(p, t0);
    }
}

__global__ void __launch_bounds__(kExpandThreads) extend_expand_kernel(const ExtendParams p) {
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kExpandThreads + threadIdx.x) * kTokensPerThread;
    if (t0 < p.num_tokens) expand_tokens(p, static_cast<int>(t0));
}

}  // namespace

cudaError_t launch_extend_tables(const ExtendParams& p, cudaStream_t stream) {
    if (p.num_tokens <= kScanThreads * kTokensPerThread) {
        extend_scan_kernel<true><<<1, kScanThreads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    extend_scan_kernel<false><<<1, kScanThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int per = kExpandThreads * kTokensPerThread;
    extend_expand_kernel<<<(p.num_tokens - 1) / per + 1, kExpandThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pkv
