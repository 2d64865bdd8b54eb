// Tensor-core decode for E4M3 caches with block scales at head_dim 64 (two tokens
// of a kv head in a tile row):
// kernel instantiations and their launch.
#include "decode_tc_host.cuh"

namespace pkv {

namespace {

// 16 KB stages at two CTAs per SM: five, or four when the per-row tables (or the
// larger P of eight heads) leave no room, then three.
template <int ACT>
cudaError_t launch_scaled(const DecodeParams& p, const CUtensorMap& km, const CUtensorMap& vm, int BS, int G,
                          cudaStream_t s) {
    const int rows = p.table_kvh_stride != 0 ? p.num_seqs * p.num_kv_heads : p.num_seqs;
    const bool wide = tc_p_columns(kE4M3B, G) == 2;
    auto fits = [](int bytes) { return 2 * (bytes + 1024) <= kTcSmemPerSm; };
    if (wide)
        return fits(TcSmem<4, kTcStage8, false, true, true, 2>::alloc(rows))
                   ? by_shape<ACT, kE4M3B, 4, false, true>(p, km, vm, km, BS, G, 2, s)
                   : by_shape<ACT, kE4M3B, 3, false, true>(p, km, vm, km, BS, G, 2, s);
    return fits(TcSmem<5, kTcStage8, false, true, true>::alloc(rows))
               ? by_shape<ACT, kE4M3B, 5, false, true>(p, km, vm, km, BS, G, 2, s)
               : by_shape<ACT, kE4M3B, 4, false, true>(p, km, vm, km, BS, G, 2, s);
}

}  // namespace

cudaError_t launch_decode_tc_e4m3b_d64(const DecodeParams& p, int act, int BS, int G, cudaStream_t s) {
    const int box_rows = BS / 2;
    const uint64_t cache_rows = static_cast<uint64_t>(p.num_blocks) * p.num_kv_heads * box_rows;
    CUtensorMap km, vm;
    if (!make_map8(&km, p.k_cache, cache_rows, box_rows) || !make_map8(&vm, p.v_cache, cache_rows, box_rows))
        return cudaErrorInvalidValue;
    return act == kBF16 ? launch_scaled<kBF16>(p, km, vm, BS, G, s) : launch_scaled<kF16>(p, km, vm, BS, G, s);
}

}  // namespace pkv
