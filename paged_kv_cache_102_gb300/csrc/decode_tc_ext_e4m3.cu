// Tensor-core decode with a window or kept logits over E4M3 caches at head_dim
// 128: kernel instantiations and their launch.
#include "decode_tc_host.cuh"

namespace pkv {

cudaError_t launch_decode_tc_ext_e4m3(const DecodeParams& p, int act, int BS, int G, cudaStream_t s) {
    const uint64_t cache_rows = static_cast<uint64_t>(p.num_blocks) * p.num_kv_heads * BS;
    CUtensorMap km, vm;
    if (!make_map8(&km, p.k_cache, cache_rows, BS) || !make_map8(&vm, p.v_cache, cache_rows, BS))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaMemsetAsync(p.work_counter, 0, sizeof(int), s);
    if (e != cudaSuccess) return e;
    return act == kBF16 ? by_shape<kBF16, kE4M3, 5, false, false, true>(p, km, vm, km, BS, G, 2, s)
                        : by_shape<kF16, kE4M3, 5, false, false, true>(p, km, vm, km, BS, G, 2, s);
}

}  // namespace pkv
