// Tensor-core decode with a window or kept logits over E4M3 caches, with block
// scales or (p.one_scale) one for all: kernel instantiations and their launch.
#include "decode_tc_host.cuh"

namespace pkv {

namespace {

// 16 KB stages at two CTAs per SM: five, with the larger P of eight heads four (head_dim 64: three)
template <int ACT, bool HALF, int BS>
cudaError_t launch_ext(const DecodeParams& p, const CUtensorMap& km, const CUtensorMap& vm, int G, cudaStream_t s) {
    constexpr int WIDE = HALF ? 3 : 4;
    if (G == 1) return launch<ACT, kE4M3B, BS, 1, 5, false, HALF, true>(p, km, vm, km, 2, s);
    if (G == 2) return launch<ACT, kE4M3B, BS, 2, 5, false, HALF, true>(p, km, vm, km, 2, s);
    if (G == 4) return launch<ACT, kE4M3B, BS, 4, 5, false, HALF, true>(p, km, vm, km, 2, s);
    if (G == 8) return launch<ACT, kE4M3B, BS, 8, WIDE, false, HALF, true>(p, km, vm, km, 2, s);
    return cudaErrorInvalidValue;
}

template <int ACT, bool HALF>
cudaError_t launch_ext(const DecodeParams& p, const CUtensorMap& km, const CUtensorMap& vm, int BS, int G, cudaStream_t s) {
    return BS == 16 ? launch_ext<ACT, HALF, 16>(p, km, vm, G, s) : launch_ext<ACT, HALF, 32>(p, km, vm, G, s);
}

}  // namespace

cudaError_t launch_decode_tc_ext_e4m3b(const DecodeParams& p, int act, int head_dim, int BS, int G, cudaStream_t s) {
    const int box_rows = head_dim == 64 ? BS / 2 : BS;
    const uint64_t cache_rows = static_cast<uint64_t>(p.num_blocks) * p.num_kv_heads * box_rows;
    CUtensorMap km, vm;
    if (!make_map8(&km, p.k_cache, cache_rows, box_rows) || !make_map8(&vm, p.v_cache, cache_rows, box_rows))
        return cudaErrorInvalidValue;
    if (head_dim == 64)
        return act == kBF16 ? launch_ext<kBF16, true>(p, km, vm, BS, G, s) : launch_ext<kF16, true>(p, km, vm, BS, G, s);
    return act == kBF16 ? launch_ext<kBF16, false>(p, km, vm, BS, G, s) : launch_ext<kF16, false>(p, km, vm, BS, G, s);
}

}  // namespace pkv
