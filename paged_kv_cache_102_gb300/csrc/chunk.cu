// Attention of each sequence's new tokens over the paged cache: the plain kernel.
//
// Row i of sequence b (n_b = seq_starts[b + 1] - seq_starts[b] new tokens at the
// end of its L_b = context_lens[b] tokens) has position p = L_b - n_b + i and
// sees the tokens j <= p, with a window only those with j > p - window or
// j < sinks:  out = sum_j softmax_j(scale <q, K[j]>) V[j].
// One warp per (row, query head), a token at a time, running maximum and sum.
#include "kernels.h"
#include "pkv_device.cuh"

namespace pkv {

namespace {

template <int CACHE>
__device__ __forceinline__ float element(const void* base, int64_t i) {
    if constexpr (is_e4m3(CACHE)) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(base)[i], __NV_E4M3);
        return __half2float(*reinterpret_cast<const __half*>(&h));
    } else {
        return act_to_float<CACHE>(static_cast<const uint16_t*>(base)[i]);
    }
}

template <int ACT, int CACHE, int D>
__global__ void __launch_bounds__(128) paged_chunk_plain_kernel(const ChunkParams p) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int row = static_cast<int>(w / p.num_q_heads), h = static_cast<int>(w % p.num_q_heads);
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.num_seqs; b += 128)
            if (p.seq_starts[b] < 0 || p.seq_starts[b] > p.seq_starts[b + 1] || p.seq_starts[b + 1] > p.num_tokens)
                atomicOr(p.err, kErrBadLen);
    if (row >= p.num_tokens) return;
    int b = 0, hi = p.num_seqs;  // the last b with seq_starts[b] <= row
    while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (p.seq_starts[mid] <= row) b = mid;
        else hi = mid;
    }
    const int s0 = p.seq_starts[b], s1 = p.seq_starts[b + 1];
    if (row < s0 || row >= s1) return;
    const int L = p.context_lens[b], n = s1 - s0;
    if (s1 > p.num_tokens || s0 < 0 || L < n || L > p.max_blocks_per_seq * p.block_size) {
        if (lane == 0) atomicOr(p.err, kErrBadLen);
        return;
    }
    const int pos = L - n + row - s0;
    const int kvh = h / (p.num_q_heads / p.num_kv_heads);
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + row * p.q_stride + static_cast<int64_t>(h) * D;
    float qf[V], acc[V] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) qf[v] = act_to_float<ACT>(q[lane + 32 * v]);
    const int lo = p.window ? max(0, pos - p.window + 1) : 0;
    for (int j = 0; j <= pos; ++j) {
        if (j < lo && j >= p.sinks) j = lo;
        const int blk = p.block_tables[static_cast<int64_t>(b) * p.max_blocks_per_seq + j / p.block_size];
        if (blk < 0 || blk >= p.num_blocks) {
            if (lane == 0) atomicOr(p.err, kErrBadBlock);
            continue;
        }
        const int64_t tile = static_cast<int64_t>(blk) * p.num_kv_heads + kvh;
        const int64_t at = (tile * p.block_size + j % p.block_size) * D;
        float d = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) d = fmaf(qf[v], element<CACHE>(p.k_cache, at + lane + 32 * v), d);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
        float vs = 1.f;
        if (CACHE == kE4M3) d *= *p.k_scale, vs = *p.v_scale;
        if (CACHE == kE4M3B) d *= p.k_scale[tile], vs = p.v_scale[tile];
        d *= p.scale_log2;
        if (d > m) {
            const float f = fast_exp2(m - d);
            l *= f;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] *= f;
            m = d;
        }
        const float w1 = fast_exp2(d - m);
        l += w1;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = fmaf(w1 * vs, element<CACHE>(p.v_cache, at + lane + 32 * v), acc[v]);
    }
    uint16_t* out = static_cast<uint16_t*>(p.out) + row * p.out_stride + static_cast<int64_t>(h) * D;
#pragma unroll
    for (int v = 0; v < V; ++v) out[lane + 32 * v] = float_to_act<ACT>(acc[v] / l);
}

template <int ACT, int CACHE>
cudaError_t launch_dim(const ChunkParams& p, int D, cudaStream_t s) {
    const int64_t warps = static_cast<int64_t>(p.num_tokens) * p.num_q_heads;
    const unsigned grid = static_cast<unsigned>((warps + 3) / 4);
    if (D == 64) paged_chunk_plain_kernel<ACT, CACHE, 64><<<grid, 128, 0, s>>>(p);
    else paged_chunk_plain_kernel<ACT, CACHE, 128><<<grid, 128, 0, s>>>(p);
    return cudaGetLastError();
}

template <int ACT>
cudaError_t launch_cache(const ChunkParams& p, int cache, int D, cudaStream_t s) {
    if (cache == kE4M3) return launch_dim<ACT, kE4M3>(p, D, s);
    if (cache == kE4M3B) return launch_dim<ACT, kE4M3B>(p, D, s);
    return launch_dim<ACT, ACT>(p, D, s);
}

}  // namespace

cudaError_t launch_chunk(const ChunkParams& p, int act, int cache, int head_dim, cudaStream_t s) {
    if (cache == act) return launch_chunk_tc(p, act, head_dim, s);
    return act == kBF16 ? launch_cache<kBF16>(p, cache, head_dim, s) : launch_cache<kF16>(p, cache, head_dim, s);
}

}  // namespace pkv
