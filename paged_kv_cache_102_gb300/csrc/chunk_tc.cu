// Launch of the tensor-core chunk attention and the merge of its shares.
#include "chunk_tc.cuh"
#include "tensor_map.cuh"

#include <algorithm>

namespace pkv {

namespace {

constexpr int kChunkMaxSplits = 32;
constexpr int kMergeThreads = 128;

// A [rows][D] 16-bit matrix in boxes of 64 columns x box_rows rows, 128-byte swizzled.
bool cache_map(CUtensorMap* m, const void* base, int act, int D, uint64_t rows, uint32_t box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), rows};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * 2};
    cuuint32_t box[2] = {64, box_rows}, steps[2] = {1, 1};
    return fn(m, act == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
              const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same in boxes of all D columns, 64 of them after the other (box_rows rows of 128 bytes each).
bool value_map(CUtensorMap* m, const void* base, int act, int D, uint64_t rows, uint32_t box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {64, rows, static_cast<cuuint64_t>(D / 64)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, 128};
    cuuint32_t box[3] = {64, box_rows, static_cast<cuuint32_t>(D / 64)}, steps[3] = {1, 1, 1};
    return fn(m, act == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q as [tokens][heads][D] in boxes of 64 channels x G heads x 128 / G tokens.
bool query_map(CUtensorMap* m, const ChunkParams& p, int act, int D) {
    auto fn = encode_fn();
    if (!fn) return false;
    const int G = p.num_q_heads / p.num_kv_heads;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(p.num_q_heads), static_cast<cuuint64_t>(p.num_tokens)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(p.q_stride) * 2};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(kChunkTile / G)}, steps[3] = {1, 1, 1};
    return fn(m, act == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void*>(p.q), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over the shares of a (row, query head), one warp each.
template <int ACT, int D>
__global__ void __launch_bounds__(kMergeThreads) paged_chunk_merge_kernel(const ChunkParams p) {
    constexpr int W = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * (kMergeThreads / 32) + (threadIdx.x >> 5);
    const int64_t rows = static_cast<int64_t>(p.num_tokens) * p.num_q_heads;
    if (w >= rows) return;
    int64_t row64;
    int h;
    divmod_u(w, p.num_q_heads, row64, h);
    const int row = static_cast<int>(row64);
    int lo = 0, hi = p.num_seqs;  // the row's sequence: the last b with seq_starts[b] <= row
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, b = lo + lane * step;
        const bool at = b < hi && p.seq_starts[b] <= row;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, at) | 1u);
        lo += k * step;
        hi = min(hi, lo + step);
    }
    const int s0 = p.seq_starts[lo], s1 = p.seq_starts[lo + 1], L = p.context_lens[lo];
    // (every row waits, so that this grid does not end, and what follows it on the stream begin, before the one ahead)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // rows of no sequence, or of one that was flagged
    if (s0 < 0 || row < s0 || row >= s1 || s1 > p.num_tokens || L < s1 - s0 || L > p.max_blocks_per_seq * p.block_size) return;
    const float2* ml = reinterpret_cast<const float2*>(p.ws_ml);
    const float2 mine = lane < p.splits ? ml[lane * rows + w] : make_float2(-INFINITY, 0.f);
    const float M = warp_max(mine.x);
    // a share without tokens of this row wrote no sums
    const float f = mine.x == -INFINITY && mine.y == 0.f ? 0.f : fast_exp2(mine.x - M);
    float l = f * mine.y;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    float acc[W] = {};
    for (int s = 0; s < p.splits; ++s) {
        const float fs = __shfl_sync(0xffffffffu, f, s);
        if (fs == 0.f) continue;
        const float* o = p.ws_o + (s * rows + w) * D + lane * W;
#pragma unroll
        for (int x = 0; x < W; ++x) acc[x] = fmaf(fs, o[x], acc[x]);
    }
    uint16_t* dst = static_cast<uint16_t*>(p.out) + row * p.out_stride + static_cast<int64_t>(h) * D + lane * W;
#pragma unroll
    for (int x = 0; x < W; ++x) dst[x] = float_to_act<ACT>(acc[x] / l);
}

template <int ACT, int CACHE, int D>
cudaError_t launch_one(const ChunkParams& p, cudaStream_t s) {
    auto kern = paged_chunk_tc_kernel<ACT, CACHE, D>;
    static bool configured[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkSmem<CACHE, D>::BYTES);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    const uint64_t cache_rows = static_cast<uint64_t>(p.num_blocks) * p.num_kv_heads * p.block_size;
    CUtensorMap km, vm, qm;
    if (!query_map(&qm, p, ACT, D)) return cudaErrorInvalidValue;
    if (is_e4m3(CACHE)) km = vm = qm;  // codes are copied without
    else if (!cache_map(&km, p.k_cache, ACT, D, cache_rows, p.block_size) ||
             !value_map(&vm, p.v_cache, ACT, D, cache_rows, p.block_size))
        return cudaErrorInvalidValue;
    const int R = 2 * (kChunkTile / (p.num_q_heads / p.num_kv_heads));
    const int64_t blocks = (static_cast<int64_t>(p.num_tokens) / R + p.num_seqs) * p.num_kv_heads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    kern<<<dim3(static_cast<unsigned>(blocks), p.splits), chunk_threads(CACHE), ChunkSmem<CACHE, D>::BYTES, s>>>(km, vm, qm, p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.splits == 1) return e;
    const int64_t rows = static_cast<int64_t>(p.num_tokens) * p.num_q_heads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((rows + kMergeThreads / 32 - 1) / (kMergeThreads / 32)));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_chunk_merge_kernel<ACT, D>, p);
}

}  // namespace

// The sequences are taken to be alike, as long as the tables: items of `tiles` token tiles in waves of an SM each, 6
// tiles' time for the start and end of a block, and for the partial results to be written and read.  Measured, us, shares
// 1 / 2 / 3 / 4: 16 sequences of 5 new tokens, 128 items of 1 to 32 tiles, 41.2 / 47.1 / 47.0 / 52.4 (all of 32 tiles 51.6 /
// 65.2 / 72.2 / 78.8); 4 of them, 32 items, 28.9 / 21.7 / 19.9 / 19.2; 509 tokens behind 32K, 64 items of 256 tiles, 443 /
// 238 / 314 / 249; one single token there, 8 items, 235 / 125 / 88 / 70, and 41 with the 19 shares that this takes.
int chunk_splits(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads, int64_t max_context) {
    const int R = 2 * std::max(1, kChunkTile / (num_q_heads / num_kv_heads));
    const int64_t each = (static_cast<int64_t>(num_tokens) + num_seqs - 1) / num_seqs;
    const int64_t items = std::max<int64_t>(1, std::min<int64_t>(num_seqs, num_tokens) * ((each + R - 1) / R) * num_kv_heads);
    const double tiles = static_cast<double>((max_context + kChunkTile - 1) / kChunkTile);
    const double rows = static_cast<double>(num_tokens) * num_q_heads;
    int best = 1;
    double least = 0;
    for (int s = 1; s <= kChunkMaxSplits && (s == 1 || s * 4 <= tiles); ++s) {
        const double waves = static_cast<double>((items * s + 151) / 152);
        const double cost = waves * (tiles / s + 6) + (s > 1 ? 1 + rows * s * 1024 / (6.7e6 * 1.7) : 0);
        if (s == 1 || cost < least) {
            best = s;
            least = cost;
        }
    }
    return best;
}

namespace {

template <int ACT, int CACHE>
cudaError_t by_dim(const ChunkParams& p, int head_dim, cudaStream_t s) {
    return head_dim == 64 ? launch_one<ACT, CACHE, 64>(p, s) : launch_one<ACT, CACHE, 128>(p, s);
}

template <int ACT>
cudaError_t by_cache(const ChunkParams& p, int cache, int head_dim, cudaStream_t s) {
    if (cache == kE4M3) return by_dim<ACT, kE4M3>(p, head_dim, s);
    if (cache == kE4M3B) return by_dim<ACT, kE4M3B>(p, head_dim, s);
    return by_dim<ACT, ACT>(p, head_dim, s);
}

}  // namespace

cudaError_t launch_chunk(const ChunkParams& given, int act, int cache, int head_dim, cudaStream_t s) {
    ChunkParams p = given;
    p.group = p.num_q_heads / p.num_kv_heads;
    p.row_tokens = kChunkTile / p.group;
    p.inv_group = 65536 / p.group + 1;
    return act == kBF16 ? by_cache<kBF16>(p, cache, head_dim, s) : by_cache<kF16>(p, cache, head_dim, s);
}

}  // namespace pkv
