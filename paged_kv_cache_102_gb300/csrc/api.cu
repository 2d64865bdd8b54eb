// C-ABI entry points of libpagedkv.so: argument checks, partition-size
// choice, workspace carving and kernel dispatch.  Declarations and the
// contract of each call are in include/pagedkv.h.
#include <atomic>
#include <algorithm>
#include <cmath>
#include <mutex>
#include <string>

#include "../../include/pagedkv.h"
#include "kernels.h"
#include "pkv_error.h"

// Per-device error word written by the kernels (OR of pkv_device_error_bits).
static __device__ int g_pkv_device_error;

namespace pkv {

namespace {
thread_local std::string t_last_error;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Device address of g_pkv_device_error on the current device.
int* device_error_word() {
    static std::mutex mu;
    static int* addr[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!addr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_pkv_device_error) != cudaSuccess) return nullptr;
        addr[dev] = static_cast<int*>(p);
    }
    return addr[dev];
}

int cuda_fail(const char* where, cudaError_t e) {
    return fail(PKV_ERR_CUDA, std::string(where) + ": " + cudaGetErrorString(e));
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

constexpr int kStageTokens = 32;  // tokens per shared-memory stage of the decode kernel
constexpr int kAutoPartition = 1024;
constexpr int kAutoPartitionGrouped = 512;
constexpr int kScaledLongItems = 2048;
// Grouped shapes with a few hundred (sequence, kv head, partition) items get
// 256-token partitions, so that the persistent grid's CTAs each get several
// to balance.  Below 256 items every CTA has at most about one, and smaller
// partitions only add merge work (QUEST's sparse decode of 8 x 8 rows: 41.0 ->
// 37.1 us at 4096 selected tokens a row, 29.4 -> 28.7 at 2048, 20.6 -> 22.6 at
// 1024 if it were applied there).
constexpr long long kAutoGroupedItemsLow = 256, kAutoGroupedItemsHigh = 1024;
constexpr size_t kWorkspaceHeader = 256;  // work counter of the tensor-core path

std::atomic<int> g_kernel_path{PKV_PATH_AUTO};

}  // namespace

void set_error(const std::string& msg) { t_last_error = msg; }

}  // namespace pkv

using namespace pkv;

extern "C" {

static bool rows_overlap(const void* a, int64_t a_stride, int64_t a_row, const void* b, int64_t b_stride, int64_t b_row,
                         int num_tokens);

const char* pkv_last_error(void) { return t_last_error.c_str(); }

int pkv_version(void) { return 100; }

int pkv_selftest_wait_timeout(int limit_us, void* stream) {
    if (limit_us < 1 || limit_us > 2000000)
        return fail(PKV_ERR_INVALID, "pkv_selftest_wait_timeout: limit_us must be in 1 .. 2,000,000");
    int* err = device_error_word();
    if (!err) return fail(PKV_ERR_CUDA, "pkv_selftest_wait_timeout: cannot resolve the device error word");
    const cudaError_t e =
        launch_selftest_wait(static_cast<uint64_t>(limit_us) * 1000u, err, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail("pkv_selftest_wait_timeout: launch", e);
}

int pkv_set_kernel_path(int path) {
    if (path < PKV_PATH_AUTO || path > PKV_PATH_TENSOR_2CTA) return -1;
    return g_kernel_path.exchange(path);
}

int pkv_device_error(int* bits, int reset, void* stream) {
    if (!bits) return fail(PKV_ERR_INVALID, "pkv_device_error: bits is NULL");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail("pkv_device_error: stream synchronize", e);
    int* word = device_error_word();
    if (!word) return fail(PKV_ERR_CUDA, "pkv_device_error: cannot resolve the device error word");
    e = cudaMemcpy(bits, word, sizeof(int), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail("pkv_device_error: read", e);
    if (reset) {
        e = cudaMemset(word, 0, sizeof(int));
        if (e != cudaSuccess) return cuda_fail("pkv_device_error: reset", e);
    }
    return PKV_OK;
}

int pkv_resolve_partition_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                               int max_blocks_per_seq, int block_size, int partition_size) {
    if (max_blocks_per_seq < 1 || block_size < 1 || num_kv_heads < 1 || num_q_heads < 1) return -1;
    const long long max_ctx = static_cast<long long>(max_blocks_per_seq) * block_size;
    const long long single = (max_ctx + kStageTokens - 1) / kStageTokens * kStageTokens;
    long long P;
    if (partition_size == PKV_PARTITION_SINGLE) {
        P = single;
    } else if (partition_size == PKV_PARTITION_AUTO) {
        // the tensor-core grouped-query kernel holds 512 tokens of scores in tensor
        // memory; the CUDA-core kernel amortises its per-partition work over 1024
        const int G = num_q_heads / num_kv_heads;
        const bool grouped = G >= 4 && (head_dim == 128 || (head_dim == 64 && num_kv_heads % 2 == 0));
        P = grouped ? kAutoPartitionGrouped : kAutoPartition;
        if (grouped) {
            // items: (sequence, kv head, partition), or (sequence, pair of kv heads, partition) at head_dim 64
            const int item_heads = head_dim == 64 ? num_kv_heads / 2 : num_kv_heads;
            auto items = [&](long long p) { return static_cast<long long>(num_seqs) * item_heads * ((max_ctx + p - 1) / p); };
            if (items(P) >= kAutoGroupedItemsLow && items(P) < kAutoGroupedItemsHigh && (P / 2) % block_size == 0)
                P /= 2;
        }
    } else if (partition_size > 0) {
        if (partition_size % kStageTokens != 0 || partition_size % block_size != 0) return -1;
        P = partition_size;
    } else {
        return -1;
    }
    if (P >= single) P = single;
    if (P > 0x7fffffff) return -1;
    return static_cast<int>(P);
}

// Workspace for partitions of P tokens.
static size_t pkv_workspace_size_of(int num_seqs, int num_q_heads, int head_dim, int max_blocks_per_seq, int block_size,
                                    int P) {
    if (P <= 0 || num_seqs <= 0 || num_q_heads <= 0 || head_dim <= 0) return 0;
    const long long max_ctx = static_cast<long long>(max_blocks_per_seq) * block_size;
    const long long parts = (max_ctx + P - 1) / P;
    if (parts <= 1) return kWorkspaceHeader;
    const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads * static_cast<size_t>(parts);
    return kWorkspaceHeader + align_up(rows * 2 * sizeof(float), 256) +
           rows * static_cast<size_t>(head_dim) * sizeof(float);
}

size_t pkv_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                          int max_blocks_per_seq, int block_size, int partition_size) {
    const int P = pkv_resolve_partition_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                                             block_size, partition_size);
    return pkv_workspace_size_of(num_seqs, num_q_heads, head_dim, max_blocks_per_seq, block_size, P);
}

int pkv_scaled_partition_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                              int block_size, int partition_size) {
    if (partition_size != PKV_PARTITION_AUTO)
        return pkv_resolve_partition_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size,
                                          partition_size);
    if (max_blocks_per_seq < 1 || block_size < 1 || num_kv_heads < 1 || num_q_heads < 1) return -1;
    const long long max_ctx = static_cast<long long>(max_blocks_per_seq) * block_size;
    const long long single = (max_ctx + kStageTokens - 1) / kStageTokens * kStageTokens;
    // The tensor-core kernel's segment of 512 tokens whatever the group; 256 for so
    // few items that twice as many still get an SM each.  Measured, 512 / 256 tokens,
    // head_dim 128, one and eight query heads: 32 items 9.9 / 8.6 and 10.8 / 9.5
    // us, 128 items 10.4 / 10.6 and 11.8 / 11.8, 256 items 12.4 / 14.6 and
    // 13.1 / 18.2, 512 items 16.1 / 16.6 and 17.9 / 20.7.  Four segments when there
    // are items enough for every SM all the same; 512 / 2048 tokens, eight query
    // heads, sequences of equal and of ragged lengths: 1024 items 25.8 / 24.8 and
    // 18.0 / 22.4 us, 2048 items 42.1 / 41.4 and 29.9 / 26.0, 4096 items 76.2 / 78.7
    // and 46.7 / 42.8, 4096 items of at most 2048 tokens, ragged, 52.7 / 43.2.
    long long P = kAutoPartitionGrouped;
    const long long items = static_cast<long long>(num_seqs) * num_kv_heads * ((max_ctx + P - 1) / P);
    if (items <= 64 && (P / 2) % block_size == 0) P /= 2;
    else if (items >= kScaledLongItems) P *= 4;
    if (P >= single) P = single;
    return static_cast<int>(P);
}

size_t pkv_scaled_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                                 int block_size, int partition_size) {
    const int P = pkv_scaled_partition_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                                            block_size, partition_size);
    return P <= 0 ? 0 : pkv_workspace_size_of(num_seqs, num_q_heads, head_dim, max_blocks_per_seq, block_size, P);
}

int paged_kv_append(const void* k, const void* v, const int64_t* slot_mapping, int num_tokens, void* k_cache,
                    void* v_cache, int num_blocks, int num_kv_heads, int block_size, int head_dim, int act_dtype,
                    int cache_dtype, const float* k_scale, const float* v_scale, void* stream) {
    if (num_tokens < 0 || num_kv_heads <= 0 || block_size <= 0 || num_blocks <= 0 || head_dim <= 0 ||
        head_dim % 8 != 0)
        return fail(PKV_ERR_INVALID, "paged_kv_append: sizes must be positive and head_dim a multiple of 8");
    if (act_dtype != PKV_F16 && act_dtype != PKV_BF16)
        return fail(PKV_ERR_INVALID, "paged_kv_append: act_dtype must be PKV_F16 or PKV_BF16");
    if (cache_dtype != act_dtype && cache_dtype != PKV_E4M3)
        return fail(PKV_ERR_INVALID, "paged_kv_append: cache_dtype must equal act_dtype or be PKV_E4M3");
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !slot_mapping || !k_cache || !v_cache)
        return fail(PKV_ERR_INVALID, "paged_kv_append: null pointer");
    if (cache_dtype == PKV_E4M3 && (!k_scale || !v_scale))
        return fail(PKV_ERR_INVALID, "paged_kv_append: an E4M3 cache needs k_scale and v_scale");
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(slot_mapping, 8))
        return fail(PKV_ERR_INVALID, "paged_kv_append: buffers must be 16-byte aligned (slot_mapping 8)");
    int* err = device_error_word();
    if (!err) return fail(PKV_ERR_CUDA, "paged_kv_append: cannot resolve the device error word");
    AppendParams p{k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, err,
                   num_tokens, num_kv_heads, head_dim, block_size, num_blocks};
    cudaError_t e = launch_append(p, act_dtype, cache_dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("paged_kv_append: launch", e);
    return PKV_OK;
}

int paged_block_copy(void* k_cache, void* v_cache, const int32_t* src_dst_pairs, int num_pairs, int num_blocks,
                     size_t block_bytes, void* stream) {
    if (num_pairs < 0 || num_blocks <= 0 || block_bytes == 0 || block_bytes % 16 != 0)
        return fail(PKV_ERR_INVALID, "paged_block_copy: num_pairs >= 0, num_blocks > 0, block_bytes a positive multiple of 16");
    if (num_pairs == 0) return PKV_OK;
    if (num_pairs > 65535 * 64) return fail(PKV_ERR_INVALID, "paged_block_copy: too many pairs in one call");
    if (!k_cache || !v_cache || !src_dst_pairs) return fail(PKV_ERR_INVALID, "paged_block_copy: null pointer");
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(src_dst_pairs, 4))
        return fail(PKV_ERR_INVALID, "paged_block_copy: caches must be 16-byte aligned");
    int* err = device_error_word();
    if (!err) return fail(PKV_ERR_CUDA, "paged_block_copy: cannot resolve the device error word");
    CopyParams p{k_cache, v_cache, src_dst_pairs, err, block_bytes, num_blocks, nullptr, nullptr, 0};
    cudaError_t e = launch_block_copy(p, num_pairs, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("paged_block_copy: launch", e);
    return PKV_OK;
}

int paged_block_swap(void* k_cache, void* v_cache, const int32_t* block_ids, int num_ids, int num_blocks,
                     size_t block_bytes, void* staging, int direction, void* stream) {
    if (num_ids < 0 || num_blocks <= 0 || block_bytes == 0 || block_bytes % 16 != 0 ||
        (direction != PKV_SWAP_OUT && direction != PKV_SWAP_IN))
        return fail(PKV_ERR_INVALID, "paged_block_swap: bad sizes or direction");
    if (num_ids == 0) return PKV_OK;
    if (num_ids > 0x7fffffff / 2) return fail(PKV_ERR_INVALID, "paged_block_swap: too many blocks");
    if (!k_cache || !v_cache || !block_ids || !staging) return fail(PKV_ERR_INVALID, "paged_block_swap: null pointer");
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(staging, 16) || !aligned(block_ids, 4))
        return fail(PKV_ERR_INVALID, "paged_block_swap: buffers must be 16-byte aligned");
    cudaPointerAttributes attr{};
    cudaError_t e = cudaPointerGetAttributes(&attr, staging);
    if (e != cudaSuccess) return cuda_fail("paged_block_swap: staging pointer", e);
    if (attr.type == cudaMemoryTypeUnregistered)
        return fail(PKV_ERR_INVALID, "paged_block_swap: staging must be device memory or pinned/registered host memory");
    int* err = device_error_word();
    if (!err) return fail(PKV_ERR_CUDA, "paged_block_swap: cannot resolve the device error word");
    void* dev_staging = attr.type == cudaMemoryTypeHost && attr.devicePointer ? attr.devicePointer : staging;
    SwapParams p{k_cache, v_cache, block_ids, dev_staging, err, block_bytes, num_blocks,
                 direction == PKV_SWAP_OUT ? 1 : 0};
    e = launch_block_swap(p, num_ids, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("paged_block_swap: launch", e);
    return PKV_OK;
}

}  // extern "C"

static size_t pool_bytes(int num_blocks, int num_kv_heads, int block_size, int head_dim, int cache_dtype) {
    return static_cast<size_t>(num_blocks) * num_kv_heads * block_size * head_dim * (cache_dtype == PKV_E4M3 ? 1 : 2);
}

// What the calls with a window or with accumulated weights add to a decode.
struct DecodeExt {
    int window = 0;  // 0: none
    int sinks = 0;
    float* scores = nullptr;
    int64_t score_tokens = 0;
};

// Blocks that a row of max_blocks keeps under a window: those of the first tokens, those that the window may touch.
static int window_blocks(int max_blocks, int block_size, int window, int sinks) {
    if (window <= 0 || sinks < 0 || block_size <= 0) return max_blocks;
    const long long n = (static_cast<long long>(sinks) + block_size - 1) / block_size +
                        (static_cast<long long>(window) + block_size - 2) / block_size + 1;
    return static_cast<int>(std::min<long long>(max_blocks, n));
}

// Partitions of the calls with a window or kept logits.  Under a window most rows are as long as they can be, so
// partitions of equal size (tensor cores: whole tiles of 128) waste none: 1072 tokens in three of 384 instead of 512,
// 512 and 48.  The CUDA-core kernel's 1024 tokens are halved while its blocks would not fill the GPU's SMs (three
// blocks each) twice.
static int ext_partition_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int blocks, int block_size,
                              int partition_size, bool block_scales, bool window) {
    const int P0 = (block_scales ? pkv_scaled_partition_size : pkv_resolve_partition_size)(
        num_seqs, num_q_heads, num_kv_heads, head_dim, blocks, block_size, partition_size);
    if (P0 <= 0 || partition_size != PKV_PARTITION_AUTO) return P0;
    const int64_t ctx = static_cast<int64_t>(blocks) * block_size;
    const int G = num_q_heads / num_kv_heads;
    const bool grouped = block_scales || (G >= 4 && (head_dim == 128 || num_kv_heads % 2 == 0));
    int64_t P = P0;
    if (!grouped)
        while (P > 256 && (P / 2) % block_size == 0 && (P / 2) % kStageTokens == 0 &&
               num_seqs * static_cast<int64_t>(num_kv_heads) * ((ctx + P - 1) / P) < 2 * 456)
            P /= 2;
    if (window && P < ctx) {
        const int64_t parts = (ctx + P - 1) / P, unit = grouped ? 128 : kStageTokens;
        P = std::min<int64_t>(P, ((ctx + parts - 1) / parts + unit - 1) / unit * unit);
    }
    return static_cast<int>(P);
}

// Workspace with kept logits: the statistics of every partition, then as without, then the logits.
struct ScoredLayout {
    size_t ml, o, logits, total;
};
static ScoredLayout scored_layout(int num_seqs, int num_q_heads, int head_dim, long long max_ctx, int P) {
    const size_t parts = static_cast<size_t>((max_ctx + P - 1) / P), heads = static_cast<size_t>(num_seqs) * num_q_heads;
    ScoredLayout w;
    w.ml = kWorkspaceHeader;
    w.o = w.ml + align_up(heads * parts * 2 * sizeof(float), 256);
    w.logits = w.o + (parts > 1 ? align_up(heads * parts * head_dim * sizeof(float), 256) : 0);
    w.total = w.logits + heads * static_cast<size_t>(max_ctx) * sizeof(float);
    return w;
}

extern "C" size_t pkv_window_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                            int max_blocks_per_seq, int block_size, int window, int sinks,
                                            int block_scales, int partition_size) {
    const int n = window_blocks(max_blocks_per_seq, block_size, window, sinks);
    if (num_seqs < 1 || num_q_heads < 1 || num_kv_heads < 1 || n < 1 || block_size < 1 || num_q_heads < num_kv_heads) return 0;
    const int P = ext_partition_size(num_seqs, num_q_heads, num_kv_heads, head_dim, n, block_size, partition_size,
                                     block_scales != 0, true);
    return pkv_workspace_size_of(num_seqs, num_q_heads, head_dim, n, block_size, P);
}

extern "C" size_t pkv_scored_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                            int max_blocks_per_seq, int block_size, int partition_size) {
    if (num_seqs < 1 || num_q_heads < 1 || num_kv_heads < 1 || head_dim < 1 || max_blocks_per_seq < 1 || block_size < 1 ||
        num_q_heads < num_kv_heads)
        return 0;
    const int P = ext_partition_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size,
                                     partition_size, false, false);
    if (P <= 0) return 0;
    return scored_layout(num_seqs, num_q_heads, head_dim, static_cast<long long>(max_blocks_per_seq) * block_size, P).total;
}

static int decode_impl(const char* fn, const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens, int num_seqs,
                       int num_q_heads, int num_kv_heads, int block_size, int head_dim, int num_blocks, float scale,
                       void* out, int act_dtype, int cache_dtype, const float* k_scale, const float* v_scale,
                       int partition_size, void* workspace, size_t workspace_bytes, void* stream, const void* k_new,
                       const void* v_new, const int64_t* new_slots, bool per_kvh_tables = false,
                       bool block_scales = false, const DecodeExt* ext = nullptr) {
    const std::string F(fn);
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
        return fail(PKV_ERR_INVALID, F + ": " + "sizes must be positive");
    if (num_q_heads % num_kv_heads != 0)
        return fail(PKV_ERR_SHAPE, F + ": " + "num_q_heads must be a multiple of num_kv_heads");
    const int G = num_q_heads / num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8)
        return fail(PKV_ERR_INVALID, F + ": " + "query heads per kv head must be 1, 2, 4 or 8");
    if (head_dim != 64 && head_dim != 128)
        return fail(PKV_ERR_INVALID, F + ": " + "head_dim must be 64 or 128");
    if (block_size != 16 && block_size != 32)
        return fail(PKV_ERR_INVALID, F + ": " + "block_size must be 16 or 32");
    if (act_dtype != PKV_F16 && act_dtype != PKV_BF16)
        return fail(PKV_ERR_INVALID, F + ": " + "act_dtype must be PKV_F16 or PKV_BF16");
    if (cache_dtype != act_dtype && cache_dtype != PKV_E4M3)
        return fail(PKV_ERR_INVALID, F + ": " + "cache_dtype must equal act_dtype or be PKV_E4M3");
    if (!std::isfinite(scale)) return fail(PKV_ERR_INVALID, F + ": " + "scale must be finite");
    if (num_seqs == 0) return PKV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out)
        return fail(PKV_ERR_INVALID, F + ": " + "null pointer");
    if (cache_dtype == PKV_E4M3 && (!k_scale || !v_scale))
        return fail(PKV_ERR_INVALID, F + ": " + (block_scales ? "the cache needs k_scales and v_scales"
                                                              : "an E4M3 cache needs k_scale and v_scale"));
    if (block_scales && (!aligned(k_scale, 4) || !aligned(v_scale, 4)))
        return fail(PKV_ERR_INVALID, F + ": " + "k_scales and v_scales must be 4-byte aligned");
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(workspace, 16))
        return fail(PKV_ERR_INVALID, F + ": " + "q, caches, out, workspace must be 16-byte aligned");
    // partitions count the tokens that are left (ext: a window's)
    const int kept_blocks = ext ? window_blocks(max_blocks_per_seq, block_size, ext->window, ext->sinks) : max_blocks_per_seq;
    const int P = ext ? ext_partition_size(num_seqs, num_q_heads, num_kv_heads, head_dim, kept_blocks, block_size,
                                           partition_size, block_scales, ext->window > 0)
                      : (block_scales ? pkv_scaled_partition_size : pkv_resolve_partition_size)(
                            num_seqs, num_q_heads, num_kv_heads, head_dim, kept_blocks, block_size, partition_size);
    if (P <= 0)
        return fail(PKV_ERR_INVALID, F + ": " + "partition_size must be 0, -1 or a positive multiple of 32 and of block_size");
    if (static_cast<long long>(max_blocks_per_seq) * block_size > 0x7fffffffLL)
        return fail(PKV_ERR_INVALID, F + ": " + "table too long");
    const long long max_ctx = static_cast<long long>(kept_blocks) * block_size;
    const bool scored = ext && ext->scores;
    const int max_parts = static_cast<int>((max_ctx + P - 1) / P);
    if (max_parts > 65535 || num_kv_heads > 65535 || num_seqs > 65535)
        return fail(PKV_ERR_INVALID, F + ": " + "grid too large (partitions, kv heads or sequences > 65535)");
    const ScoredLayout layout = scored_layout(num_seqs, num_q_heads, head_dim, max_ctx, P);
    const size_t need = scored ? layout.total
                               : pkv_workspace_size_of(num_seqs, num_q_heads, head_dim, kept_blocks, block_size, P);
    if (!workspace || workspace_bytes < need)
        return fail(PKV_ERR_INVALID, F + ": " + "workspace of " + std::to_string(need) + " bytes required (" +
                                         (scored ? "pkv_scored_workspace_size)" : ext ? "pkv_window_workspace_size)"
                                          : block_scales ? "pkv_scaled_workspace_size)" : "pkv_workspace_size)"));
    if (scored) {  // written, the scores read and written by different blocks
        const auto at = reinterpret_cast<uintptr_t>(ext->scores);
        const size_t B = num_seqs, rows = 2 * B * num_q_heads * head_dim;
        const size_t pool = pool_bytes(num_blocks, num_kv_heads, block_size, head_dim, cache_dtype);
        const uintptr_t end = at + sizeof(float) * B * num_kv_heads * ext->score_tokens;
        const struct { const void* at; size_t bytes; } others[] = {
            {q, rows}, {out, rows}, {context_lens, 4 * B}, {block_tables, 4 * B * max_blocks_per_seq}, {workspace, need},
            {k_cache, pool}, {v_cache, pool}, {k_scale, k_scale ? 4u : 0u}, {v_scale, v_scale ? 4u : 0u}};
        for (const auto& o : others) {
            const auto x = reinterpret_cast<uintptr_t>(o.at);
            if (x < end && at < x + o.bytes) return fail(PKV_ERR_INVALID, F + ": " + "scores must be a buffer of its own");
        }
    }
    int* err = device_error_word();
    if (!err) return fail(PKV_ERR_CUDA, F + ": " + "cannot resolve the device error word");

    DecodeParams p{};
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.out = out;
    const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads * static_cast<size_t>(max_parts);
    char* ws = static_cast<char*>(workspace);
    p.work_counter = reinterpret_cast<int*>(ws);
    p.ws_ml = max_parts > 1 ? reinterpret_cast<float*>(ws + kWorkspaceHeader) : nullptr;
    p.ws_o = max_parts > 1 ? reinterpret_cast<float*>(ws + kWorkspaceHeader + align_up(rows * 2 * sizeof(float), 256))
                           : nullptr;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.err = err;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.num_blocks = num_blocks;
    p.partition_size = P;
    p.max_parts = max_parts;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.k_new = k_new;
    p.v_new = v_new;
    p.new_slots = new_slots;
    if (ext) {
        p.window = ext->window;
        p.sinks = ext->sinks;
    }
    if (scored) {
        p.ws_ml = reinterpret_cast<float*>(ws + layout.ml);
        p.ws_o = max_parts > 1 ? reinterpret_cast<float*>(ws + layout.o) : nullptr;
        p.logits = reinterpret_cast<float*>(ws + layout.logits);
        p.logit_tokens = max_ctx;
    }
    if (per_kvh_tables) {  // tables [B][Hkv][max_blocks], lengths [B][Hkv]
        p.table_seq_stride = static_cast<int64_t>(num_kv_heads) * max_blocks_per_seq;
        p.table_kvh_stride = max_blocks_per_seq;
        p.lens_seq_stride = num_kv_heads;
        p.lens_kvh_stride = 1;
    } else {
        p.table_seq_stride = max_blocks_per_seq;
        p.table_kvh_stride = 0;
        p.lens_seq_stride = 1;
        p.lens_kvh_stride = 0;
    }

    // the kernels' cache kind: E4M3 codes with one scale, or one per (block, kv head)
    const int kind = block_scales ? kCacheE4M3Blocks : cache_dtype;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    const int path = g_kernel_path.load();
    // the tensor-core kernel keeps per-row tables in shared memory: larger
    // batches run as several launches over consecutive sequences
    const int rows_per_seq = per_kvh_tables ? num_kv_heads : 1;
    const bool tc_ok = rows_per_seq <= decode_tc_max_rows() &&
                       decode_tc_supported(head_dim, block_size, G, act_dtype, kind, P, num_kv_heads,
                                           per_kvh_tables);
    if ((path == PKV_PATH_TENSOR || path == PKV_PATH_TENSOR_2CTA) && !tc_ok)
        return fail(PKV_ERR_INVALID, F + ": " + "the tensor-core path needs head_dim 128 (16-bit or E4M3 "
                                     "cache) or 64 (16-bit cache, even kv heads, shared tables), 2/4/8 query "
                                     "heads per kv head and partitions of at most 512 tokens (block-scaled "
                                     "caches: either head_dim, any group and partitions of at most 2^20 tokens)");
    // Block-scaled: short contexts and few rows take the CUDA-core kernel, whose
    // one launch is over in 4 to 8 us where the tensor-core kernel takes 7 to 13
    // (head_dim 128, 128 tokens, us: 5.2 / 7.5 for 16 x 8 rows of one query head,
    // 12.0 / 12.3 for 16 x 32 of two; 8.4 / 7.8 for 16 x 8 of four, where the border
    // could lie lower; from there on the other way: 17.7 / 12.9 for 16 x 32 of four,
    // 22.2 / 20.4 for 64 x 32 of one, and at eight query heads always: 12.7 / 8.7 for
    // 8 rows of 32 tokens).
    const bool small = block_scales && G <= 4 && max_ctx <= 256 &&
                       static_cast<long long>(num_seqs) * num_q_heads <= 1024;
    const bool use_tc = path == PKV_PATH_TENSOR || path == PKV_PATH_TENSOR_2CTA ||
                        (path == PKV_PATH_AUTO && tc_ok && !small && (G >= 4 || block_scales));
    if (use_tc) {
        const int chunk = (ext ? decode_tc_ext_max_rows(head_dim, kind) : decode_tc_max_rows()) / rows_per_seq;
        const size_t act_bytes = 2;
        e = cudaSuccess;
        p.zero_words = 1;
        if (scored) p.failed = p.work_counter + 1;
        for (int s0 = 0; s0 < num_seqs && e == cudaSuccess; s0 += chunk) {
            DecodeParams c = p;
            c.num_seqs = std::min(chunk, num_seqs - s0);
            c.q = static_cast<const char*>(q) + static_cast<size_t>(s0) * num_q_heads * head_dim * act_bytes;
            c.out = static_cast<char*>(out) + static_cast<size_t>(s0) * num_q_heads * head_dim * act_bytes;
            c.block_tables = block_tables + s0 * p.table_seq_stride;
            c.context_lens = context_lens + static_cast<int64_t>(s0) * p.lens_seq_stride;
            if (new_slots) {
                c.k_new = static_cast<const char*>(k_new) + static_cast<size_t>(s0) * num_kv_heads * head_dim * act_bytes;
                c.v_new = static_cast<const char*>(v_new) + static_cast<size_t>(s0) * num_kv_heads * head_dim * act_bytes;
                c.new_slots = new_slots + s0;
            }
            if (max_parts > 1) {
                const size_t hrow0 = static_cast<size_t>(s0) * num_q_heads * max_parts;
                c.ws_ml = p.ws_ml + hrow0 * 2;
                c.ws_o = p.ws_o + hrow0 * head_dim;
            }
            if (scored) {
                c.ws_ml = p.ws_ml + static_cast<size_t>(s0) * num_q_heads * max_parts * 2;
                c.logits = p.logits + static_cast<int64_t>(s0) * num_q_heads * max_ctx;
                c.zero_words = s0 == 0 ? 2 : 1;  // (the launches of a call share `failed`)
            }
            e = ext ? launch_decode_tc_ext(c, act_dtype, kind, head_dim, block_size, G, s)
                    : launch_decode_tc(c, act_dtype, kind, head_dim, block_size, G, path == PKV_PATH_TENSOR ? 0 : 1, s);
        }
    } else if (ext) {
        const bool f16 = act_dtype == PKV_F16;
        auto launch = kind == kCacheE4M3Blocks ? (f16 ? launch_decode_ext_f16_e4m3b : launch_decode_ext_bf16_e4m3b)
                      : kind == PKV_E4M3       ? (f16 ? launch_decode_ext_f16_e4m3 : launch_decode_ext_bf16_e4m3)
                                               : (f16 ? launch_decode_ext_f16_f16 : launch_decode_ext_bf16_bf16);
        e = launch(p, head_dim, block_size, G, s);
    } else if (block_scales)
        e = act_dtype == PKV_F16 ? launch_decode_f16_e4m3b(p, head_dim, block_size, G, s)
                                 : launch_decode_bf16_e4m3b(p, head_dim, block_size, G, s);
    else if (act_dtype == PKV_F16)
        e = cache_dtype == PKV_E4M3 ? launch_decode_f16_e4m3(p, head_dim, block_size, G, s)
                                    : launch_decode_f16_f16(p, head_dim, block_size, G, s);
    else
        e = cache_dtype == PKV_E4M3 ? launch_decode_bf16_e4m3(p, head_dim, block_size, G, s)
                                    : launch_decode_bf16_bf16(p, head_dim, block_size, G, s);
    if (e != cudaSuccess) return cuda_fail((F + ": partition kernel launch").c_str(), e);
    if (max_parts > 1 && !scored) {
        MergeParams m{};
        m.context_lens = context_lens;
        m.num_seqs = num_seqs;
        m.lens_seq_stride = p.lens_seq_stride;
        m.lens_kvh_stride = p.lens_kvh_stride;
        m.group = G;
        m.ws_ml = p.ws_ml;
        m.ws_o = p.ws_o;
        m.out = out;
        m.num_q_heads = num_q_heads;
        m.head_dim = head_dim;
        m.partition_size = P;
        m.max_parts = max_parts;
        m.max_context = max_blocks_per_seq * block_size;
        m.window = p.window;
        m.sinks = p.sinks;
        m.block_size = block_size;
        e = launch_merge(m, act_dtype, s);
        if (e != cudaSuccess) return cuda_fail((F + ": merge kernel launch").c_str(), e);
    }
    if (scored) {
        const AddWeightsParams a{p.logits, p.ws_ml, context_lens, p.failed, ext->scores, p.ws_o, out, ext->score_tokens,
                                 p.logit_tokens, num_seqs, num_kv_heads, G, P, max_parts, static_cast<int>(max_ctx)};
        e = launch_scored_finish(a, act_dtype, head_dim, s);
        if (e != cudaSuccess) return cuda_fail((F + ": weights kernel launch").c_str(), e);
    }
    return PKV_OK;
}

extern "C" {

int paged_attention_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                           int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int num_q_heads,
                           int num_kv_heads, int block_size, int head_dim, int num_blocks, float scale, void* out,
                           int act_dtype, int cache_dtype, const float* k_scale, const float* v_scale,
                           int partition_size, void* workspace, size_t workspace_bytes, void* stream) {
    return decode_impl("paged_attention_decode", q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                       num_seqs, num_q_heads, num_kv_heads, block_size, head_dim, num_blocks, scale, out, act_dtype,
                       cache_dtype, k_scale, v_scale, partition_size, workspace, workspace_bytes, stream, nullptr,
                       nullptr, nullptr);
}

int paged_attention_decode_append(const void* q, const void* k_new, const void* v_new, const int64_t* slot_mapping,
                                  void* k_cache, void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
                                  const int32_t* context_lens, int num_seqs, int num_q_heads, int num_kv_heads,
                                  int block_size, int head_dim, int num_blocks, float scale, void* out, int act_dtype,
                                  int cache_dtype, const float* k_scale, const float* v_scale, int partition_size,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    if (num_seqs > 0 && (!k_new || !v_new || !slot_mapping))
        return fail(PKV_ERR_INVALID, "paged_attention_decode_append: null pointer");
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(slot_mapping, 8))
        return fail(PKV_ERR_INVALID, "paged_attention_decode_append: k_new, v_new must be 16-byte aligned");
    return decode_impl("paged_attention_decode_append", q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                       context_lens, num_seqs, num_q_heads, num_kv_heads, block_size, head_dim, num_blocks, scale, out,
                       act_dtype, cache_dtype, k_scale, v_scale, partition_size, workspace, workspace_bytes, stream,
                       k_new, v_new, slot_mapping);
}


int paged_attention_decode_sparse(const void* q, const void* k_cache, const void* v_cache, const int32_t* sel_tables,
                                  int max_sel_blocks, const int32_t* sel_lens, int num_seqs, int num_q_heads,
                                  int num_kv_heads, int block_size, int head_dim, int num_blocks, float scale,
                                  void* out, int act_dtype, int cache_dtype, const float* k_scale,
                                  const float* v_scale, int partition_size, void* workspace, size_t workspace_bytes,
                                  void* stream) {
    return decode_impl("paged_attention_decode_sparse", q, k_cache, v_cache, sel_tables, max_sel_blocks, sel_lens,
                       num_seqs, num_q_heads, num_kv_heads, block_size, head_dim, num_blocks, scale, out, act_dtype,
                       cache_dtype, k_scale, v_scale, partition_size, workspace, workspace_bytes, stream, nullptr,
                       nullptr, nullptr, true);
}

int paged_attention_decode_scaled(const void* q, const void* k_cache, const void* v_cache, const float* k_scales,
                                  const float* v_scales, const int32_t* block_tables, int max_blocks_per_seq,
                                  const int32_t* context_lens, int num_seqs, int num_q_heads, int num_kv_heads,
                                  int block_size, int head_dim, int num_blocks, float scale, void* out, int act_dtype,
                                  int partition_size, void* workspace, size_t workspace_bytes, void* stream) {
    return decode_impl("paged_attention_decode_scaled", q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                       context_lens, num_seqs, num_q_heads, num_kv_heads, block_size, head_dim, num_blocks, scale, out,
                       act_dtype, PKV_E4M3, k_scales, v_scales, partition_size, workspace, workspace_bytes, stream,
                       nullptr, nullptr, nullptr, false, true);
}

int paged_attention_decode_window(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                                  int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int num_q_heads,
                                  int num_kv_heads, int block_size, int head_dim, int num_blocks, float scale,
                                  int window, int sinks, void* out, int act_dtype, int cache_dtype, const float* k_scale,
                                  const float* v_scale, const float* k_scales, const float* v_scales,
                                  int partition_size, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "paged_attention_decode_window";
    if (window < 1 || sinks < 0)
        return fail(PKV_ERR_INVALID, std::string(fn) + ": window must be positive and sinks not negative");
    const bool blocks = k_scales || v_scales;
    if (blocks && (cache_dtype != PKV_E4M3 || k_scale || v_scale))
        return fail(PKV_ERR_INVALID, std::string(fn) + ": an E4M3 cache has k_scale and v_scale or k_scales and v_scales");
    // no row has more tokens than the tables: more than that of either changes nothing
    const int64_t context = std::max<int64_t>(1, static_cast<int64_t>(max_blocks_per_seq) * block_size);
    DecodeExt ext;
    ext.window = static_cast<int>(std::min<int64_t>(window, context));
    ext.sinks = static_cast<int>(std::min<int64_t>(sinks, context));
    return decode_impl(fn, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, num_q_heads,
                       num_kv_heads, block_size, head_dim, num_blocks, scale, out, act_dtype, cache_dtype,
                       blocks ? k_scales : k_scale, blocks ? v_scales : v_scale, partition_size, workspace,
                       workspace_bytes, stream, nullptr, nullptr, nullptr, false, blocks, &ext);
}

int paged_attention_decode_scored(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                                  int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int num_q_heads,
                                  int num_kv_heads, int block_size, int head_dim, int num_blocks, float scale,
                                  float* scores, int64_t score_tokens, void* out, int act_dtype, int cache_dtype,
                                  const float* k_scale, const float* v_scale, int partition_size, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    const char* fn = "paged_attention_decode_scored";
    if (score_tokens < static_cast<int64_t>(max_blocks_per_seq) * block_size)
        return fail(PKV_ERR_INVALID, std::string(fn) + ": scores need a value for each of a row's max_blocks_per_seq * block_size tokens");
    if (num_seqs > 0 && (!scores || !aligned(scores, 4)))
        return fail(PKV_ERR_INVALID, std::string(fn) + ": scores must be given, 4-byte aligned");
    DecodeExt ext;
    ext.scores = scores;
    ext.score_tokens = score_tokens;
    return decode_impl(fn, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, num_q_heads,
                       num_kv_heads, block_size, head_dim, num_blocks, scale, out, act_dtype, cache_dtype, k_scale,
                       v_scale, partition_size, workspace, workspace_bytes, stream, nullptr, nullptr, nullptr, false,
                       false, &ext);
}

int paged_kv_evict(void* k_cache, void* v_cache, int num_blocks, int num_kv_heads, int block_size, int head_dim,
                   int cache_dtype, const float* scores, int64_t score_tokens, const int32_t* block_tables,
                   int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, const int32_t* dst_tables,
                   int max_dst_blocks, int budget, int recent, int sinks, float* scores_out, int64_t score_tokens_out,
                   int32_t* context_lens_out, int32_t* kept, void* stream) {
    const std::string F("paged_kv_evict: ");
    if (num_blocks <= 0 || num_kv_heads <= 0 || block_size <= 0 || head_dim <= 0 || max_blocks_per_seq <= 0 ||
        max_dst_blocks <= 0 || num_seqs < 0 || score_tokens <= 0 || score_tokens_out <= 0)
        return fail(PKV_ERR_INVALID, F + "sizes must be positive");
    if (cache_dtype != PKV_F16 && cache_dtype != PKV_BF16 && cache_dtype != PKV_E4M3)
        return fail(PKV_ERR_INVALID, F + "cache_dtype must be PKV_F16, PKV_BF16 or PKV_E4M3");
    if (head_dim != 64 && head_dim != 128) return fail(PKV_ERR_INVALID, F + "head_dim must be 64 or 128");
    if (budget <= 0 || recent < 0 || sinks < 0 || static_cast<int64_t>(recent) + sinks > budget)
        return fail(PKV_ERR_INVALID, F + "budget must be positive, recent and sinks not negative and at most budget in all");
    if (static_cast<int64_t>(max_blocks_per_seq) * block_size > 0x7fffffffLL ||
        static_cast<int64_t>(max_dst_blocks) * block_size > 0x7fffffffLL)
        return fail(PKV_ERR_INVALID, F + "table too long");
    if (score_tokens_out < std::min<int64_t>(budget, score_tokens))
        return fail(PKV_ERR_INVALID, F + "scores_out has no room for the tokens that stay");
    if (num_kv_heads > 65535 || num_seqs > 65535) return fail(PKV_ERR_INVALID, F + "grid too large");
    if (num_seqs == 0) return PKV_OK;
    if (!k_cache || !v_cache || !scores || !block_tables || !context_lens || !dst_tables || !scores_out ||
        !context_lens_out || !kept)
        return fail(PKV_ERR_INVALID, F + "null pointer");
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(scores, 4) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4) || !aligned(dst_tables, 4) || !aligned(scores_out, 4) || !aligned(context_lens_out, 4) ||
        !aligned(kept, 4))
        return fail(PKV_ERR_INVALID, F + "caches must be 16-byte aligned (others 4)");
    // what is written (first; the pools too) and read: buffers of their own
    const size_t B = num_seqs, BH = B * num_kv_heads;
    const size_t pool = pool_bytes(num_blocks, num_kv_heads, block_size, head_dim, cache_dtype);
    const struct { const void* at; size_t bytes; } buffers[] = {
        {scores_out, 4 * BH * score_tokens_out}, {context_lens_out, 4 * B}, {kept, 4 * BH * budget},
        {k_cache, pool}, {v_cache, pool}, {scores, 4 * BH * score_tokens}, {context_lens, 4 * B}, {block_tables, 4 * B * max_blocks_per_seq},
        {dst_tables, 4 * B * max_dst_blocks}};
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < 9; ++j) {
            if (i == 3 && j == 4) continue;  // K and V: the caller's pools
            const auto a = reinterpret_cast<uintptr_t>(buffers[i].at), b = reinterpret_cast<uintptr_t>(buffers[j].at);
            if (a < b + buffers[j].bytes && b < a + buffers[i].bytes)
                return fail(PKV_ERR_INVALID, F + "scores_out, context_lens_out, kept and the caches must be buffers of their own");
        }
    int* err = device_error_word();
    if (!err) return fail(PKV_ERR_CUDA, F + "cannot resolve the device error word");
    const EvictParams p{k_cache, v_cache, scores, block_tables, context_lens, dst_tables, scores_out, context_lens_out,
                        kept, err, score_tokens, score_tokens_out, max_blocks_per_seq, max_dst_blocks, num_seqs,
                        num_kv_heads, block_size, num_blocks, head_dim * (cache_dtype == PKV_E4M3 ? 1 : 2), budget,
                        recent, sinks};
    const cudaError_t e = launch_evict(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail("paged_kv_evict: launch", e);
}

size_t pkv_chunk_workspace_size(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                int max_blocks_per_seq, int block_size) {
    if (num_seqs <= 0 || num_tokens <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        max_blocks_per_seq <= 0 || block_size <= 0 || num_q_heads < num_kv_heads)
        return kWorkspaceHeader;
    const int splits = chunk_splits(num_seqs, num_tokens, num_q_heads, num_kv_heads,
                                    static_cast<int64_t>(max_blocks_per_seq) * block_size);
    if (splits == 1) return kWorkspaceHeader;
    const size_t rows = static_cast<size_t>(splits) * num_tokens * num_q_heads;
    return kWorkspaceHeader + align_up(rows * 2 * sizeof(float), 256) + rows * head_dim * sizeof(float);
}

int paged_attention_chunk(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                          const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
                          const int32_t* seq_starts, int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads,
                          int block_size, int head_dim, int num_blocks, float scale, int window, int sinks, void* out,
                          int64_t out_stride, int act_dtype, int cache_dtype, const float* k_scale, const float* v_scale,
                          const float* k_scales, const float* v_scales, void* workspace, size_t workspace_bytes,
                          void* stream) {
    const std::string F("paged_attention_chunk: ");
    if (num_seqs < 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
        return fail(PKV_ERR_INVALID, F + "sizes must be positive (num_seqs and num_tokens may be 0)");
    if (num_q_heads % num_kv_heads != 0)
        return fail(PKV_ERR_SHAPE, F + "num_q_heads must be a multiple of num_kv_heads");
    if (num_q_heads / num_kv_heads > 64) return fail(PKV_ERR_INVALID, F + "at most 64 query heads per kv head");
    if (head_dim != 64 && head_dim != 128) return fail(PKV_ERR_INVALID, F + "head_dim must be 64 or 128");
    if (block_size != 16 && block_size != 32) return fail(PKV_ERR_INVALID, F + "block_size must be 16 or 32");
    if (act_dtype != PKV_F16 && act_dtype != PKV_BF16)
        return fail(PKV_ERR_INVALID, F + "act_dtype must be PKV_F16 or PKV_BF16");
    if (cache_dtype != act_dtype && cache_dtype != PKV_E4M3)
        return fail(PKV_ERR_INVALID, F + "cache_dtype must equal act_dtype or be PKV_E4M3");
    if (!std::isfinite(scale)) return fail(PKV_ERR_INVALID, F + "scale must be finite");
    if (window < 0 || sinks < 0) return fail(PKV_ERR_INVALID, F + "window and sinks must not be negative (window 0: none)");
    const bool blocks = k_scales || v_scales;
    if (blocks && (cache_dtype != PKV_E4M3 || k_scale || v_scale))
        return fail(PKV_ERR_INVALID, F + "an E4M3 cache has k_scale and v_scale or k_scales and v_scales");
    if (cache_dtype == PKV_E4M3 && (blocks ? (!k_scales || !v_scales) : (!k_scale || !v_scale)))
        return fail(PKV_ERR_INVALID, F + "an E4M3 cache needs scales for both K and V");
    if (static_cast<int64_t>(max_blocks_per_seq) * block_size > 0x7fffffffLL)
        return fail(PKV_ERR_INVALID, F + "table too long");
    const int64_t row = static_cast<int64_t>(num_q_heads) * head_dim;
    if (q_stride % 8 != 0 || out_stride % 8 != 0 || (num_tokens > 1 && (q_stride < row || out_stride < row)))
        return fail(PKV_ERR_INVALID, F + "token strides of q and out must be multiples of 8 elements and at least a row");
    if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !seq_starts || !out)
        return fail(PKV_ERR_INVALID, F + "null pointer");
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(workspace, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(seq_starts, 4) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(k_scales, 4) || !aligned(v_scales, 4))
        return fail(PKV_ERR_INVALID, F + "q, caches, out and workspace must be 16-byte aligned (others 4)");
    // a row's output may not be another row's query: rows are done in any order
    if (rows_overlap(out, 2 * out_stride, 2 * row, q, 2 * q_stride, 2 * row, num_tokens))
        return fail(PKV_ERR_INVALID, F + "out shares memory with q");
    const size_t need = pkv_chunk_workspace_size(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim,
                                                 max_blocks_per_seq, block_size);
    if (!workspace || workspace_bytes < need)
        return fail(PKV_ERR_INVALID, F + "workspace of " + std::to_string(need) + " bytes required (pkv_chunk_workspace_size)");
    ChunkParams p{};
    p.q = q;
    p.q_stride = num_tokens > 1 ? q_stride : row;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.seq_starts = seq_starts;
    p.out = out;
    p.out_stride = num_tokens > 1 ? out_stride : row;
    p.k_scale = blocks ? k_scales : k_scale;
    p.v_scale = blocks ? v_scales : v_scale;
    p.err = device_error_word();
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    // no row has more tokens than the tables: a window of as many is none, more first tokens change nothing
    const int64_t context = static_cast<int64_t>(max_blocks_per_seq) * block_size;
    p.window = window < context ? window : 0;
    p.sinks = p.window ? static_cast<int>(std::min<int64_t>(sinks, context)) : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    // a window's tokens alone are shared out (never more shares than the workspace was sized for)
    p.splits = chunk_splits(num_seqs, num_tokens, num_q_heads, num_kv_heads, context);
    if (p.window)
        p.splits = std::min(p.splits, chunk_splits(num_seqs, num_tokens, num_q_heads, num_kv_heads,
                                                   std::min<int64_t>(context, static_cast<int64_t>(p.window) + p.sinks)));
    if (p.splits > 1) {
        char* ws = static_cast<char*>(workspace) + kWorkspaceHeader;
        const size_t rows = static_cast<size_t>(p.splits) * num_tokens * num_q_heads;
        p.ws_ml = reinterpret_cast<float*>(ws);
        p.ws_o = reinterpret_cast<float*>(ws + align_up(rows * 2 * sizeof(float), 256));
    }
    if (!p.err) return fail(PKV_ERR_CUDA, F + "cannot resolve the device error word");
    const cudaError_t e = launch_chunk(p, act_dtype, blocks ? kCacheE4M3Blocks : cache_dtype, head_dim,
                                       static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail("paged_attention_chunk: launch", e);
}

int paged_extend_tables(int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
                        const int32_t* new_lens, int num_seqs, int block_size, const int32_t* free_blocks, int num_free,
                        const int32_t* free_head, int num_blocks, int num_tokens, int64_t* slot_mapping,
                        int32_t* positions, int32_t* seq_starts, int32_t* block_starts, int32_t* context_lens_out,
                        int32_t* free_head_out, void* stream) {
    const std::string F("paged_extend_tables: ");
    if (num_seqs < 0 || max_blocks_per_seq <= 0 || block_size <= 0 || num_free < 0 || num_blocks <= 0 || num_tokens < 0)
        return fail(PKV_ERR_INVALID, F + "sizes must be positive (num_seqs, num_free and num_tokens may be 0)");
    if (static_cast<long long>(max_blocks_per_seq) * block_size > 0x7fffffffLL)
        return fail(PKV_ERR_INVALID, F + "table too long");
    if (num_tokens > 0x7fffffff - 4) return fail(PKV_ERR_INVALID, F + "too many tokens");
    if (!free_head || !seq_starts || !block_starts || !free_head_out)
        return fail(PKV_ERR_INVALID, F + "null pointer");
    if (num_seqs > 0 && (!block_tables || !context_lens || !new_lens || !context_lens_out))
        return fail(PKV_ERR_INVALID, F + "null pointer");
    if ((num_free > 0 && !free_blocks) || (num_tokens > 0 && (!slot_mapping || !positions)))
        return fail(PKV_ERR_INVALID, F + "null pointer");
    // what is written (first) and read: written buffers share memory with no other, but for the two updated in place
    const size_t B = num_seqs, T = num_tokens;
    const struct { const void* at; size_t bytes; } buffers[] = {
        {slot_mapping, 8 * T}, {positions, 4 * T}, {seq_starts, 4 * (B + 1)}, {block_starts, 4 * (B + 1)},
        {block_tables, 4 * B * max_blocks_per_seq}, {context_lens_out, 4 * B}, {free_head_out, 4},
        {context_lens, 4 * B}, {free_head, 4}, {new_lens, 4 * B}, {free_blocks, 4 * static_cast<size_t>(num_free)}};
    for (int i = 0; i < 7; ++i) {
        for (int j = i + 1; j < 11; ++j) {
            const auto a = reinterpret_cast<uintptr_t>(buffers[i].at), b = reinterpret_cast<uintptr_t>(buffers[j].at);
            const bool in_place = (i == 5 && j == 7) || (i == 6 && j == 8);
            if (buffers[i].bytes && buffers[j].bytes && a < b + buffers[j].bytes && b < a + buffers[i].bytes &&
                !(in_place && a == b))
                return fail(PKV_ERR_INVALID, F + "outputs must be buffers of their own (context_lens_out may be "
                                                 "context_lens, free_head_out may be free_head)");
        }
    }
    if (!aligned(slot_mapping, 16) || !aligned(positions, 16))
        return fail(PKV_ERR_INVALID, F + "slot_mapping and positions must be 16-byte aligned");
    if (!aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(new_lens, 4) || !aligned(free_blocks, 4) ||
        !aligned(free_head, 4) || !aligned(seq_starts, 4) || !aligned(block_starts, 4) ||
        !aligned(context_lens_out, 4) || !aligned(free_head_out, 4))
        return fail(PKV_ERR_INVALID, F + "int32 buffers must be 4-byte aligned");
    int* err = device_error_word();
    if (!err) return fail(PKV_ERR_CUDA, F + "cannot resolve the device error word");
    ExtendParams p{block_tables, context_lens, new_lens, free_blocks, free_head, slot_mapping, positions, seq_starts,
                   block_starts, context_lens_out, free_head_out, err, num_seqs, max_blocks_per_seq, block_size,
                   num_free, num_blocks, num_tokens};
    const cudaError_t e = launch_extend_tables(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail("paged_extend_tables: launch", e);
}

// Checks shared by the strided appends; returns PKV_OK or the status to return.
static int append_checks(const std::string& F, const RopeAppendParams& p, int act_dtype) {
    if (p.num_tokens < 0 || p.num_kv_heads <= 0 || p.block_size <= 0 || p.num_blocks <= 0 || p.head_dim <= 0 ||
        p.head_dim % 8 != 0 || p.head_dim > 256 || p.block_size > (1 << 20) || p.num_kv_heads > 65535)
        return fail(PKV_ERR_INVALID, F + "sizes must be positive, head_dim a multiple of 8 up to 256, block_size at most "
                                         "2^20 and num_kv_heads at most 65535");
    if (act_dtype != PKV_F16 && act_dtype != PKV_BF16)
        return fail(PKV_ERR_INVALID, F + "act_dtype must be PKV_F16 or PKV_BF16");
    if (p.k_stride % 8 != 0 || p.v_stride % 8 != 0 || p.k_stride < 0 || p.v_stride < 0)
        return fail(PKV_ERR_INVALID, F + "token strides must be multiples of 8 elements and not negative");
    return PKV_OK;
}

int paged_kv_append_scaled(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           const int64_t* slot_mapping, int num_tokens, void* k_cache, void* v_cache, float* k_scales,
                           float* v_scales, int num_blocks, int num_kv_heads, int block_size, int head_dim,
                           int act_dtype, void* stream) {
    const std::string F("paged_kv_append_scaled: ");
    RopeAppendParams p{};
    p.k = k;
    p.v = v;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.slot_mapping = slot_mapping;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.num_tokens = num_tokens;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    const int c = append_checks(F, p, act_dtype);
    if (c != PKV_OK) return c;
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !slot_mapping || !k_cache || !v_cache || !k_scales || !v_scales)
        return fail(PKV_ERR_INVALID, F + "null pointer");
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(slot_mapping, 8) || !aligned(k_scales, 4) || !aligned(v_scales, 4))
        return fail(PKV_ERR_INVALID, F + "buffers must be 16-byte aligned (slot_mapping 8, scales 4)");
    p.err = device_error_word();
    if (!p.err) return fail(PKV_ERR_CUDA, F + "cannot resolve the device error word");
    const cudaError_t e = launch_rope_append(p, act_dtype, kCacheE4M3Blocks, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail("paged_kv_append_scaled: launch", e);
}

// Whether two sets of num_tokens rows share memory (strides and row lengths in bytes; with different strides:
// whether they may).
static bool rows_overlap(const void* a, int64_t a_stride, int64_t a_row, const void* b, int64_t b_stride, int64_t b_row,
                         int num_tokens) {
    const auto x = reinterpret_cast<intptr_t>(a), y = reinterpret_cast<intptr_t>(b);
    if (x >= y + (num_tokens - 1) * b_stride + b_row || y >= x + (num_tokens - 1) * a_stride + a_row) return false;
    if (a_stride != b_stride || a_stride == 0 || num_tokens == 1) return true;
    const intptr_t d = ((x - y) % a_stride + a_stride) % a_stride;  // a's columns behind b's
    return d < b_row || d + a_row > a_stride;
}

int paged_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                      int64_t v_stride, const int32_t* positions, const int64_t* slot_mapping, int num_tokens,
                      const float* inv_freq, int rotary_dim, int interleaved, float attention_factor, void* q_out,
                      int64_t q_out_stride, void* k_cache, void* v_cache, int num_blocks, int num_q_heads,
                      int num_kv_heads, int block_size, int head_dim, int act_dtype, int cache_dtype,
                      const float* k_scale, const float* v_scale, float* k_scales, float* v_scales, void* stream) {
    const std::string F("paged_rope_append: ");
    RopeAppendParams p{};
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.positions = positions;
    p.slot_mapping = slot_mapping;
    p.inv_freq = inv_freq;
    p.q_out = q_out;
    p.q_out_stride = q_out_stride;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.factor = attention_factor;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.rotary_dim = rotary_dim;
    p.interleaved = interleaved ? 1 : 0;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    const int c = append_checks(F, p, act_dtype);
    if (c != PKV_OK) return c;
    if (num_q_heads < 0 || num_q_heads > 65535)
        return fail(PKV_ERR_INVALID, F + "num_q_heads must be in 0 .. 65535");
    if (rotary_dim <= 0 || rotary_dim % 2 != 0 || rotary_dim > head_dim)
        return fail(PKV_ERR_INVALID, F + "rotary_dim must be even, positive and at most head_dim");
    if (!std::isfinite(attention_factor)) return fail(PKV_ERR_INVALID, F + "attention_factor must be finite");
    if (cache_dtype != act_dtype && cache_dtype != PKV_E4M3)
        return fail(PKV_ERR_INVALID, F + "cache_dtype must equal act_dtype or be PKV_E4M3");
    if (num_q_heads > 0 && (q_stride % 8 != 0 || q_stride < 0 || q_out_stride % 8 != 0 ||
                            (num_tokens > 1 && q_out_stride < static_cast<int64_t>(num_q_heads) * head_dim)))
        return fail(PKV_ERR_INVALID, F + "q token strides must be multiples of 8 elements, and q_out's rows apart");
    if (num_q_heads > 0 && q && q == q_out && num_tokens > 1 && q_stride != q_out_stride)
        return fail(PKV_ERR_INVALID, F + "in place, q and q_out have one stride");
    const bool blocks = k_scales || v_scales;
    if (cache_dtype == PKV_E4M3 && blocks == (k_scale || v_scale))
        return fail(PKV_ERR_INVALID, F + "an E4M3 cache needs either k_scale and v_scale or k_scales and v_scales");
    if (cache_dtype == PKV_E4M3 && (blocks ? (!k_scales || !v_scales) : (!k_scale || !v_scale)))
        return fail(PKV_ERR_INVALID, F + "an E4M3 cache needs scales for both K and V");
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !positions || !slot_mapping || !inv_freq || !k_cache || !v_cache ||
        (num_q_heads > 0 && (!q || !q_out)))
        return fail(PKV_ERR_INVALID, F + "null pointer");
    if (num_q_heads > 0) {
        const int64_t q_row = 2LL * num_q_heads * head_dim, kv_row = 2LL * num_kv_heads * head_dim, qo = 2 * q_out_stride;
        if ((q != q_out && rows_overlap(q_out, qo, q_row, q, 2 * q_stride, q_row, num_tokens)) ||
            rows_overlap(q_out, qo, q_row, k, 2 * k_stride, kv_row, num_tokens) ||
            rows_overlap(q_out, qo, q_row, v, 2 * v_stride, kv_row, num_tokens))
            return fail(PKV_ERR_INVALID, F + "q_out may be q itself, but shares no memory with k, v or other rows of q");
    }
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(slot_mapping, 8) || !aligned(positions, 4) || !aligned(inv_freq, 4) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(k_scales, 4) || !aligned(v_scales, 4))
        return fail(PKV_ERR_INVALID, F + "buffers must be 16-byte aligned (slot_mapping 8; positions, inv_freq, "
                                         "scales 4)");
    p.err = device_error_word();
    if (!p.err) return fail(PKV_ERR_CUDA, F + "cannot resolve the device error word");
    const cudaError_t e = launch_rope_append(p, act_dtype, cache_dtype == PKV_E4M3 && blocks ? kCacheE4M3Blocks : cache_dtype,
                                             static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail("paged_rope_append: launch", e);
}

int paged_block_copy_scaled(void* k_cache, void* v_cache, float* k_scales, float* v_scales,
                            const int32_t* src_dst_pairs, int num_pairs, int num_blocks, int num_kv_heads,
                            size_t block_bytes, void* stream) {
    const std::string F("paged_block_copy_scaled: ");
    if (num_pairs < 0 || num_blocks <= 0 || num_kv_heads <= 0 || block_bytes == 0 || block_bytes % 16 != 0)
        return fail(PKV_ERR_INVALID, F + "num_pairs >= 0, num_blocks and num_kv_heads > 0, block_bytes a positive multiple of 16");
    if (num_pairs == 0) return PKV_OK;
    if (num_pairs > 65535 * 64) return fail(PKV_ERR_INVALID, F + "too many pairs in one call");
    if (!k_cache || !v_cache || !k_scales || !v_scales || !src_dst_pairs) return fail(PKV_ERR_INVALID, F + "null pointer");
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(src_dst_pairs, 4) || !aligned(k_scales, 4) ||
        !aligned(v_scales, 4))
        return fail(PKV_ERR_INVALID, F + "caches must be 16-byte aligned (pairs and scales 4)");
    int* err = device_error_word();
    if (!err) return fail(PKV_ERR_CUDA, F + "cannot resolve the device error word");
    CopyParams p{k_cache, v_cache, src_dst_pairs, err, block_bytes, num_blocks, k_scales, v_scales, num_kv_heads};
    const cudaError_t e = launch_block_copy(p, num_pairs, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail("paged_block_copy_scaled: launch", e);
}

int paged_block_scales_swap(float* k_scales, float* v_scales, const int32_t* block_ids, int num_ids, int num_blocks,
                            int num_kv_heads, float* staging, int direction, void* stream) {
    const std::string F("paged_block_scales_swap: ");
    if (num_ids < 0 || num_blocks <= 0 || num_kv_heads <= 0 || (direction != PKV_SWAP_OUT && direction != PKV_SWAP_IN))
        return fail(PKV_ERR_INVALID, F + "bad sizes or direction");
    if (num_ids == 0) return PKV_OK;
    if (num_ids > 0x7fffffff / 2) return fail(PKV_ERR_INVALID, F + "too many blocks");
    if (!k_scales || !v_scales || !block_ids || !staging) return fail(PKV_ERR_INVALID, F + "null pointer");
    if (!aligned(k_scales, 4) || !aligned(v_scales, 4) || !aligned(staging, 4) || !aligned(block_ids, 4))
        return fail(PKV_ERR_INVALID, F + "buffers must be 4-byte aligned");
    cudaPointerAttributes attr{};
    cudaError_t e = cudaPointerGetAttributes(&attr, staging);
    if (e != cudaSuccess) return cuda_fail("paged_block_scales_swap: staging pointer", e);
    if (attr.type == cudaMemoryTypeUnregistered)
        return fail(PKV_ERR_INVALID, F + "staging must be device memory or pinned/registered host memory");
    int* err = device_error_word();
    if (!err) return fail(PKV_ERR_CUDA, F + "cannot resolve the device error word");
    float* dev_staging = attr.type == cudaMemoryTypeHost && attr.devicePointer
                             ? static_cast<float*>(attr.devicePointer) : staging;
    e = launch_scales_swap(ScalesSwapParams{k_scales, v_scales, block_ids, dev_staging, err, num_ids, num_blocks,
                                            num_kv_heads, direction == PKV_SWAP_OUT ? 1 : 0},
                           static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail("paged_block_scales_swap: launch", e);
}

int quest_block_minmax(const void* k_cache, const int32_t* block_tables, int max_blocks_per_seq,
                       const int32_t* context_lens, int num_seqs, int num_kv_heads, int block_size, int head_dim,
                       int num_blocks, int cache_dtype, int meta_dtype, void* kmeta, void* stream) {
    if (num_seqs < 0 || max_blocks_per_seq <= 0 || num_kv_heads <= 0 || block_size <= 0 || num_blocks <= 0 ||
        head_dim <= 0 || head_dim % 8 != 0)
        return fail(PKV_ERR_INVALID, "quest_block_minmax: sizes must be positive, head_dim a multiple of 8");
    if (meta_dtype != PKV_F16 && meta_dtype != PKV_BF16)
        return fail(PKV_ERR_INVALID, "quest_block_minmax: meta_dtype must be PKV_F16 or PKV_BF16");
    if (cache_dtype != meta_dtype && cache_dtype != PKV_E4M3)
        return fail(PKV_ERR_INVALID, "quest_block_minmax: the cache must be of meta_dtype or PKV_E4M3");
    if (num_seqs == 0) return PKV_OK;
    if (!k_cache || !block_tables || !context_lens || !kmeta) return fail(PKV_ERR_INVALID, "quest_block_minmax: null pointer");
    if (!aligned(k_cache, 16) || !aligned(kmeta, 16)) return fail(PKV_ERR_INVALID, "quest_block_minmax: misaligned");
    int* err = device_error_word();
    if (!err) return fail(PKV_ERR_CUDA, "quest_block_minmax: cannot resolve the device error word");
    QuestMetaParams p{k_cache, block_tables, context_lens, kmeta, err, num_seqs, max_blocks_per_seq, num_kv_heads,
                      block_size, head_dim, num_blocks};
    cudaError_t e = launch_quest_minmax(p, meta_dtype, cache_dtype, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail("quest_block_minmax: launch", e);
}

int quest_append_minmax(const void* k_new, const int64_t* slot_mapping, int num_tokens, int num_kv_heads,
                        int block_size, int head_dim, int num_blocks, int act_dtype, int cache_dtype,
                        const float* k_scale, void* kmeta, void* stream) {
    if (num_tokens < 0 || num_kv_heads <= 0 || block_size <= 0 || num_blocks <= 0 || head_dim <= 0 || head_dim % 8 != 0)
        return fail(PKV_ERR_INVALID, "quest_append_minmax: sizes must be positive, head_dim a multiple of 8");
    if (act_dtype != PKV_F16 && act_dtype != PKV_BF16)
        return fail(PKV_ERR_INVALID, "quest_append_minmax: act_dtype must be PKV_F16 or PKV_BF16");
    if (cache_dtype != act_dtype && cache_dtype != PKV_E4M3)
        return fail(PKV_ERR_INVALID, "quest_append_minmax: the cache must be of act_dtype or PKV_E4M3");
    if (num_tokens == 0) return PKV_OK;
    if (!k_new || !slot_mapping || !kmeta) return fail(PKV_ERR_INVALID, "quest_append_minmax: null pointer");
    if (cache_dtype == PKV_E4M3 && !k_scale)
        return fail(PKV_ERR_INVALID, "quest_append_minmax: an E4M3 cache needs k_scale");
    if (!aligned(k_new, 16) || !aligned(kmeta, 16) || !aligned(slot_mapping, 8))
        return fail(PKV_ERR_INVALID, "quest_append_minmax: misaligned");
    int* err = device_error_word();
    if (!err) return fail(PKV_ERR_CUDA, "quest_append_minmax: cannot resolve the device error word");
    QuestAppendParams p{k_new, slot_mapping, cache_dtype == PKV_E4M3 ? k_scale : nullptr, kmeta, err, num_tokens,
                        num_kv_heads, block_size, head_dim, num_blocks};
    cudaError_t e = launch_quest_append_minmax(p, act_dtype, cache_dtype, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail("quest_append_minmax: launch", e);
}

size_t quest_workspace_size(int num_seqs, int num_kv_heads, int max_blocks_per_seq) {
    if (num_seqs <= 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0) return 0;
    return static_cast<size_t>(num_seqs) * num_kv_heads * max_blocks_per_seq * sizeof(float);
}

int quest_select(const void* q, const void* kmeta, const int32_t* block_tables, int max_blocks_per_seq,
                 const int32_t* context_lens, int num_seqs, int num_q_heads, int num_kv_heads, int block_size,
                 int head_dim, int num_blocks, int act_dtype, int budget_blocks, int32_t* sel_tables, int32_t* sel_lens,
                 void* workspace, size_t workspace_bytes, void* stream) {
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        max_blocks_per_seq <= 0 || block_size <= 0 || num_blocks <= 0 || budget_blocks <= 0)
        return fail(PKV_ERR_INVALID, "quest_select: sizes must be positive, num_q_heads a multiple of num_kv_heads");
    const int G = num_q_heads / num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return fail(PKV_ERR_INVALID, "quest_select: group must be 1, 2, 4 or 8");
    if (head_dim != 64 && head_dim != 128) return fail(PKV_ERR_INVALID, "quest_select: head_dim must be 64 or 128");
    if (act_dtype != PKV_F16 && act_dtype != PKV_BF16)
        return fail(PKV_ERR_INVALID, "quest_select: act_dtype must be PKV_F16 or PKV_BF16");
    if (max_blocks_per_seq > 16384) return fail(PKV_ERR_INVALID, "quest_select: at most 16384 blocks per sequence");
    if (num_seqs == 0) return PKV_OK;
    if (num_seqs > 65535 || num_kv_heads > 65535) return fail(PKV_ERR_INVALID, "quest_select: grid too large");
    if (!q || !kmeta || !block_tables || !context_lens || !sel_tables || !sel_lens)
        return fail(PKV_ERR_INVALID, "quest_select: null pointer");
    if (!aligned(q, 16) || !aligned(kmeta, 16)) return fail(PKV_ERR_INVALID, "quest_select: q and kmeta must be 16-byte aligned");
    const size_t need = quest_workspace_size(num_seqs, num_kv_heads, max_blocks_per_seq);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
        return fail(PKV_ERR_INVALID, "quest_select: workspace of " + std::to_string(need) +
                                         " bytes (16-byte aligned) required (quest_workspace_size)");
    int* err = device_error_word();
    if (!err) return fail(PKV_ERR_CUDA, "quest_select: cannot resolve the device error word");
    QuestSelectParams p{q, kmeta, block_tables, context_lens, sel_tables, sel_lens, static_cast<float*>(workspace),
                        err, num_seqs, num_q_heads, num_kv_heads, block_size, head_dim, num_blocks,
                        max_blocks_per_seq, budget_blocks, /*group_heads: chosen at launch*/ 0};
    cudaError_t e = launch_quest_select(p, act_dtype, G, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail("quest_select: launch", e);
}

}  // extern "C"
