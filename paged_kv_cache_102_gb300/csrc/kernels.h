// Kernel parameter blocks and launchers (host-visible, no device code).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pkv {

constexpr int kMaxDevices = 64;
// Cache kind of the launchers next to the pkv_dtype codes: E4M3 with one scale
// per (block, kv head) (kE4M3B of the kernels).
constexpr int kCacheE4M3Blocks = 3;

struct AppendParams {
    const void* k;
    const void* v;
    const int64_t* slot_mapping;
    void* k_cache;
    void* v_cache;
    const float* k_scale;
    const float* v_scale;
    int* err;
    int num_tokens;
    int num_kv_heads;
    int head_dim;
    int block_size;
    int num_blocks;
};

// Rotary positions and the append of rotated keys (positions == nullptr: no
// rotation and no queries).
struct RopeAppendParams {
    const void* q;
    const void* k;
    const void* v;
    int64_t q_stride;  // elements from one token's row to the next
    int64_t k_stride;
    int64_t v_stride;
    const int32_t* positions;
    const int64_t* slot_mapping;
    const float* inv_freq;  // [rotary_dim / 2]
    void* q_out;
    int64_t q_out_stride;
    void* k_cache;
    void* v_cache;
    const float* k_scale;  // E4M3, one scale per tensor
    const float* v_scale;
    float* k_scales;  // E4M3, [num_blocks][num_kv_heads]
    float* v_scales;
    int* err;
    float factor;  // multiplies cos and sin
    int num_tokens;
    int num_q_heads;
    int num_kv_heads;
    int head_dim;
    int rotary_dim;
    int interleaved;
    int block_size;
    int num_blocks;
};

// Tables, slots and positions of a step's tokens (extend_tables.cu).
struct ExtendParams {
    int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* new_lens;
    const int32_t* free_blocks;
    const int32_t* free_head;
    int64_t* slot_mapping;
    int32_t* positions;
    int32_t* seq_starts;    // [num_seqs + 1]
    int32_t* block_starts;  // [num_seqs + 1]
    int32_t* lens_out;
    int32_t* free_head_out;
    int* err;
    int num_seqs;
    int max_blocks_per_seq;
    int block_size;
    int num_free;
    int num_blocks;
    int num_tokens;
};

struct CopyParams {
    void* k_cache;
    void* v_cache;
    const int32_t* pairs;
    int* err;
    size_t block_bytes;
    int num_blocks;
    float* k_scales;  // [num_blocks][num_kv_heads], copied with the block; null: none
    float* v_scales;
    int num_kv_heads;
};

struct ScalesSwapParams {
    float* k_scales;
    float* v_scales;
    const int32_t* block_ids;
    float* staging;  // [n][2][num_kv_heads]: K then V scales of each listed block
    int* err;
    int n;
    int num_blocks;
    int num_kv_heads;
    int to_staging;
};

struct SwapParams {
    void* k_cache;
    void* v_cache;
    const int32_t* block_ids;
    void* staging;  // [n][2][block_bytes]: K then V of each listed block
    int* err;
    size_t block_bytes;
    int num_blocks;
    int to_staging;  // 1: pools -> staging (swap out), 0: staging -> pools (swap in)
};

struct DecodeParams {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    void* out;
    float* ws_ml;  // [num_seqs][num_q_heads][max_parts][2]: (max in log2 units, sum)
    float* ws_o;   // [num_seqs][num_q_heads][max_parts][head_dim]: normalised partial outputs
    int* work_counter;  // workspace header: next item to claim (tensor-core path), zero at launch
    // fused append (optional): new K/V row of each sequence ([num_seqs][Hkv][D], act dtype) and its
    // slot; the row is the sequence's last context token
    const void* k_new;
    const void* v_new;
    const int64_t* new_slots;
    // table row of (seq, kvh) = block_tables + seq*table_seq_stride + kvh*table_kvh_stride;
    // its length = context_lens[seq*lens_seq_stride + kvh*lens_kvh_stride]
    // (per-sequence tables: max_blocks_per_seq, 0, 1, 0)
    int64_t table_seq_stride;
    int64_t table_kvh_stride;
    int lens_seq_stride;
    int lens_kvh_stride;
    const float* k_scale;  // block-scaled E4M3 cache: [num_blocks][num_kv_heads], else one value
    const float* v_scale;
    int* err;
    int max_blocks_per_seq;
    int num_seqs;
    int num_q_heads;
    int num_kv_heads;
    int num_blocks;
    int partition_size;  // tokens per partition, a multiple of 32 and of the block size
    int max_parts;
    float scale_log2;  // scale * log2(e)
    // the extended kernels (EXT) alone; lengths and partitions count the tokens of windowed_len then
    int window;      // the last `window` tokens and the first `sinks` are seen; 0: all
    int sinks;
    bool one_scale;  // block-scaled kernels: k_scale and v_scale hold one value, every block's
    int* failed;     // tensor cores, kept logits: set to 1 where a block gave up a wait; the word behind work_counter
    int zero_words;  // words at work_counter to zero ahead of the launch
    float* logits;   // [num_seqs][num_kv_heads][logit_tokens][G], in log2 units; null: not kept
    int64_t logit_tokens;
};

// Tokens that a sequence of L keeps when the blocks wholly between its first
// `sinks` tokens and its last `window` ones are left out, so that the others
// are numbered through: token v of the result is token v in the first blocks,
// v + L - windowed_len behind them.  The hidden ones left, inside the blocks at
// either edge, are those with sinks <= v < windowed_len - window; every block
// left has a visible token (it holds a first token, the window's first one, or
// one between that and the last).
#ifdef __CUDACC__
__host__ __device__
#endif
inline int windowed_len(int L, int window, int sinks, int block_size) {
    if (window == 0 || L <= window) return L;
    const int first = sinks / block_size + (sinks % block_size != 0);  // blocks of the first tokens
    const int from = (L - window) / block_size;                        // the window's first block
    return from > first ? L - (from - first) * block_size : L;
}

struct MergeParams {
    const int32_t* context_lens;
    int num_seqs;
    int lens_seq_stride;
    int lens_kvh_stride;
    int group;  // query heads per kv head
    const float* ws_ml;
    const float* ws_o;
    void* out;
    int num_q_heads;
    int head_dim;
    int partition_size;
    int max_parts;
    int max_context;
    int window;  // as in DecodeParams, 0: none
    int sinks;
    int block_size;
};

// scores[seq][kvh][token] += sum over the group's heads of their weights.
struct AddWeightsParams {
    const float* logits;  // [num_seqs][num_kv_heads][logit_tokens][group], log2 units
    const float* ws_ml;   // [num_seqs][num_kv_heads * group][max_parts][2]; (0, 0): the partition went wrong
    const int32_t* context_lens;
    const int* failed;    // not null and not 0: nothing is added
    float* scores;        // [num_seqs][num_kv_heads][score_tokens]
    const float* ws_o;    // [num_seqs][num_kv_heads * group][max_parts][head_dim], where there are several
    void* out;
    int64_t score_tokens;
    int64_t logit_tokens;
    int num_seqs;
    int num_kv_heads;
    int group;
    int partition_size;
    int max_parts;
    int max_context;
};

// The tokens that stay and their move to other blocks (evict.cu).
struct EvictParams {
    void* k_cache;
    void* v_cache;
    const float* scores;  // [num_seqs][num_kv_heads][score_tokens]
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* dst_tables;
    float* scores_out;
    int32_t* lens_out;
    int32_t* kept;  // [num_seqs][num_kv_heads][budget]
    int* err;
    int64_t score_tokens;
    int64_t score_tokens_out;
    int max_blocks_per_seq;
    int max_dst_blocks;
    int num_seqs;
    int num_kv_heads;
    int block_size;
    int num_blocks;
    int row_bytes;  // head_dim elements
    int budget;
    int recent;
    int sinks;
};

// Attention of each sequence's new tokens over the cache (chunk_tc.cuh, chunk_tc.cu).
struct ChunkParams {
    const void* q;
    int64_t q_stride;  // elements from one token's row to the next
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* seq_starts;  // [num_seqs + 1]
    void* out;
    int64_t out_stride;
    const float* k_scale;  // E4M3: one, or with block scales [num_blocks][num_kv_heads]
    const float* v_scale;
    int* err;
    int max_blocks_per_seq;
    int num_seqs;
    int num_tokens;  // rows of q and out
    int num_q_heads;
    int num_kv_heads;
    int block_size;
    int num_blocks;
    int window;  // 0: none
    int sinks;
    float scale_log2;
    int group;       // query heads of a kv head, set by launch_chunk with the two below
    int row_tokens;  // tokens of a row tile: 128 / group
    int inv_group;   // 65536 / group + 1: (r * inv_group) >> 16 = r / group for r < 128, group <= 64
    int splits;   // shares of an item's token tiles, each a block's; 1: none
    float* ws_ml;  // [splits][num_tokens][num_q_heads][2]: (reference maximum in log2 units, sum); null: one share
    float* ws_o;   // [splits][num_tokens][num_q_heads][head_dim]: sums relative to the maximum
};

struct QuestMetaParams {
    const void* k_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    void* kmeta;
    int* err;
    int num_seqs;
    int max_blocks_per_seq;
    int num_kv_heads;
    int block_size;
    int head_dim;
    int num_blocks;
};

struct QuestAppendParams {
    const void* k_new;
    const int64_t* slot_mapping;
    const float* k_scale;  // E4M3 cache only
    void* kmeta;
    int* err;
    int num_tokens;
    int num_kv_heads;
    int block_size;
    int head_dim;
    int num_blocks;
};

struct QuestSelectParams {
    const void* q;
    const void* kmeta;
    const int32_t* block_tables;
    const int32_t* context_lens;
    int32_t* sel_tables;
    int32_t* sel_lens;
    float* bounds;  // workspace [num_seqs][num_kv_heads][max_blocks_per_seq]
    int* err;
    int num_seqs;
    int num_q_heads;
    int num_kv_heads;
    int block_size;
    int head_dim;
    int num_blocks;
    int max_blocks_per_seq;
    int budget_blocks;
    int group_heads;  // kv heads per bound item (set by launch_quest_select)
};

cudaError_t launch_quest_minmax(const QuestMetaParams& p, int meta, int cache, cudaStream_t s);
cudaError_t launch_quest_append_minmax(const QuestAppendParams& p, int act, int cache, cudaStream_t s);
cudaError_t launch_quest_select(const QuestSelectParams& p, int dtype, int G, cudaStream_t s);

cudaError_t launch_rope_append(const RopeAppendParams& p, int act, int cache, cudaStream_t stream);
cudaError_t launch_extend_tables(const ExtendParams& p, cudaStream_t stream);
cudaError_t launch_append(const AppendParams& p, int act, int cache, cudaStream_t stream);
cudaError_t launch_block_copy(const CopyParams& p, int num_pairs, cudaStream_t stream);
cudaError_t launch_block_swap(const SwapParams& p, int n, cudaStream_t stream);
cudaError_t launch_scales_swap(const ScalesSwapParams& p, cudaStream_t stream);
cudaError_t launch_merge(const MergeParams& p, int act, cudaStream_t stream);
cudaError_t launch_selftest_wait(uint64_t limit_ns, int* err, cudaStream_t stream);

// Partition kernel for one (act, cache) pair; returns cudaErrorInvalidValue
// for a (head_dim, block_size, group) it was not built for.
cudaError_t launch_decode_f16_f16(const DecodeParams& p, int D, int BS, int G, cudaStream_t s);
cudaError_t launch_decode_ext_f16_f16(const DecodeParams& p, int D, int BS, int G, cudaStream_t s);
cudaError_t launch_decode_bf16_bf16(const DecodeParams& p, int D, int BS, int G, cudaStream_t s);
cudaError_t launch_decode_ext_bf16_bf16(const DecodeParams& p, int D, int BS, int G, cudaStream_t s);
cudaError_t launch_decode_f16_e4m3(const DecodeParams& p, int D, int BS, int G, cudaStream_t s);
cudaError_t launch_decode_ext_f16_e4m3(const DecodeParams& p, int D, int BS, int G, cudaStream_t s);
cudaError_t launch_decode_bf16_e4m3(const DecodeParams& p, int D, int BS, int G, cudaStream_t s);
cudaError_t launch_decode_ext_bf16_e4m3(const DecodeParams& p, int D, int BS, int G, cudaStream_t s);
cudaError_t launch_decode_f16_e4m3b(const DecodeParams& p, int D, int BS, int G, cudaStream_t s);
cudaError_t launch_decode_ext_f16_e4m3b(const DecodeParams& p, int D, int BS, int G, cudaStream_t s);
cudaError_t launch_decode_bf16_e4m3b(const DecodeParams& p, int D, int BS, int G, cudaStream_t s);
cudaError_t launch_decode_ext_bf16_e4m3b(const DecodeParams& p, int D, int BS, int G, cudaStream_t s);

// Tensor-core grouped-query path (head_dim 128 with a 16-bit or E4M3 cache
// of either scaling, or head_dim 64 with a 16-bit cache, an even kv-head count
// and shared tables, or with a block-scaled cache; group 2/4/8, block-scaled
// also 1; partitions of at most 512 tokens, block-scaled 2^20).  variant 0: one CTA per SM; variant 1:
// two CTAs per SM (block-scaled: always two).
bool decode_tc_supported(int head_dim, int block_size, int group, int act, int cache, int partition_size,
                         int num_kv_heads, bool per_kvh_tables);
int decode_tc_max_rows();  // table rows (sequences, or (sequence, kv head) pairs) of one launch
cudaError_t launch_decode_tc(const DecodeParams& p, int act, int cache, int head_dim, int BS, int G, int variant,
                             cudaStream_t s);
cudaError_t launch_decode_tc_e4m3(const DecodeParams& p, int act, int BS, int G, int variant, cudaStream_t s);
cudaError_t launch_decode_tc_e4m3b(const DecodeParams& p, int act, int BS, int G, cudaStream_t s);
cudaError_t launch_decode_tc_e4m3b_d64(const DecodeParams& p, int act, int BS, int G, cudaStream_t s);
cudaError_t launch_decode_tc_d64(const DecodeParams& p, int act, int BS, int G, int variant, cudaStream_t s);

// The same with a window or kept logits (tables shared by a sequence's kv heads).
int decode_tc_ext_max_rows(int head_dim, int cache);
cudaError_t launch_decode_tc_ext(const DecodeParams& p, int act, int cache, int head_dim, int BS, int G, cudaStream_t s);
cudaError_t launch_decode_tc_ext_e4m3b(const DecodeParams& p, int act, int head_dim, int BS, int G, cudaStream_t s);

// Adds each token's weights, from kept logits and the partitions' statistics, to its scores, and joins the partitions.
cudaError_t launch_scored_finish(const AddWeightsParams& p, int act, int head_dim, cudaStream_t stream);
cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream);
cudaError_t launch_chunk(const ChunkParams& p, int act, int cache, int head_dim, cudaStream_t stream);
// Shares that an item's token tiles are split into (a function of the sizes).
int chunk_splits(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads, int64_t max_context);

}  // namespace pkv
