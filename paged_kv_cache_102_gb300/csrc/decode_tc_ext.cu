// Tensor-core decode with a window or kept logits over 16-bit caches: kernel
// instantiations and their launch (E4M3 caches: decode_tc_ext_e4m3b.cu).  One ring depth each, two CTAs per SM: the API calls
// with at most decode_tc_ext_max_rows sequences, whose tables leave room for it.
// Measured: a window of 1024 and 4 first tokens, 128 sequences of up to 8192, 64 / 8
// heads of 128, bfloat16: 82 us with the merge (8), its K and V 58 at the copy's rate;
// block scales, 64 sequences of 40 heads, each its own: 62 us of 50.  Ramp and tail of
// one launch, as without a window.
#include "decode_tc_host.cuh"

namespace pkv {

int decode_tc_ext_max_rows(int head_dim, int cache) { return head_dim == 64 && !is_e4m3(cache) ? kTcMaxSeqs : kTcExtRows; }

namespace {

template <int ACT>
cudaError_t launch_ext(const DecodeParams& p, const CUtensorMap& km, const CUtensorMap& vm, const CUtensorMap& qm,
                       int head_dim, int BS, int G, cudaStream_t s) {
    return head_dim == 64 ? by_shape<ACT, ACT, 2, true, false, true>(p, km, vm, qm, BS, G, 2, s)
                          : by_shape<ACT, ACT, 3, false, false, true>(p, km, vm, qm, BS, G, 2, s);
}

}  // namespace

cudaError_t launch_decode_tc_ext(const DecodeParams& p, int act, int cache, int head_dim, int BS, int G, cudaStream_t s) {
    if (cache == kE4M3B) return launch_decode_tc_ext_e4m3b(p, act, head_dim, BS, G, s);
    if (cache == kE4M3) {
        // One scale for all: the block-scaled kernel, whose queries and weights enter in three parts, which keep what the
        // outputs can hold.  Two parts, as paged_attention_decode takes, leave 2^-8 of a weight, half a step of bfloat16
        // and eight times that of binary16, and were slower, one segment of 512 tokens an item: a window of 1024 of 128
        // sequences, eight query heads, 64.8 against 50.2 us (binary16 69.0, 50.8), scored, 64 sequences of up to 4096,
        // 90.4 against 74.5 (96.6, 75.9); three sequences of 700 22.5 against 24.1.
        DecodeParams one = p;
        one.one_scale = true;
        return launch_decode_tc_ext_e4m3b(one, act, head_dim, BS, G, s);
    }
    if (head_dim == 64 && p.num_kv_heads % 2 != 0) return cudaErrorInvalidValue;
    const uint64_t cache_rows = static_cast<uint64_t>(p.num_blocks) * p.num_kv_heads * BS;
    CUtensorMap km, vm, qm;
    if (!make_map(&km, p.k_cache, act, cache_rows, BS, head_dim) || !make_map(&vm, p.v_cache, act, cache_rows, BS, head_dim) ||
        !make_map(&qm, p.q, act, static_cast<uint64_t>(p.num_seqs) * p.num_q_heads, G, head_dim))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaMemsetAsync(p.work_counter, 0, sizeof(int) * p.zero_words, s);
    if (e != cudaSuccess) return e;
    return act == kBF16 ? launch_ext<kBF16>(p, km, vm, qm, head_dim, BS, G, s)
                        : launch_ext<kF16>(p, km, vm, qm, head_dim, BS, G, s);
}

}  // namespace pkv
