// Tensor-core grouped-query decode for E4M3 caches with block scales: kernel
// instantiations and their launch (head_dim 128, and head_dim 64 with two
// tokens of a kv head in a tile row).
#include "decode_tc_host.cuh"

namespace pkv {

namespace {

// 16 KB stages; ten at one CTA per SM (variant 0), else five (or four, when
// the per-row tables leave no room) at two CTAs per SM.
template <int ACT, bool HALF>
cudaError_t launch_scaled(const DecodeParams& p, const CUtensorMap& km, const CUtensorMap& vm, int BS, int G,
                          int variant, cudaStream_t s) {
    const int rows = p.table_kvh_stride != 0 ? p.num_seqs * p.num_kv_heads : p.num_seqs;
    const bool five = 2 * (TcSmem<5, kTcStage8, false, true, HALF>::alloc(rows) + 1024) <= kTcSmemPerSm;
    if (variant == 0) return by_shape<ACT, kE4M3B, 10, false, HALF>(p, km, vm, km, BS, G, 1, s);
    if (five) return by_shape<ACT, kE4M3B, 5, false, HALF>(p, km, vm, km, BS, G, 2, s);
    return by_shape<ACT, kE4M3B, 4, false, HALF>(p, km, vm, km, BS, G, 2, s);
}

}  // namespace

cudaError_t launch_decode_tc_e4m3b(const DecodeParams& p, int act, int head_dim, int BS, int G, int variant,
                                   cudaStream_t s) {
    const bool half = head_dim == 64;
    const int box_rows = half ? BS / 2 : BS;
    const uint64_t cache_rows = static_cast<uint64_t>(p.num_blocks) * p.num_kv_heads * box_rows;
    CUtensorMap km, vm;
    if (!make_map8(&km, p.k_cache, cache_rows, box_rows) || !make_map8(&vm, p.v_cache, cache_rows, box_rows))
        return cudaErrorInvalidValue;
    if (half)
        return act == kBF16 ? launch_scaled<kBF16, true>(p, km, vm, BS, G, variant, s)
                            : launch_scaled<kF16, true>(p, km, vm, BS, G, variant, s);
    return act == kBF16 ? launch_scaled<kBF16, false>(p, km, vm, BS, G, variant, s)
                        : launch_scaled<kF16, false>(p, km, vm, BS, G, variant, s);
}

}  // namespace pkv
