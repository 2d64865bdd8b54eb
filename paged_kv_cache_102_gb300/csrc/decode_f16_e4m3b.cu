// Paged decode partition kernels: f16 queries/outputs, e4m3 cache with block scales.
#include "pkv_device.cuh"
#define PKV_ACT pkv::kF16
#define PKV_CACHE pkv::kE4M3B
#define PKV_LAUNCH_NAME launch_decode_f16_e4m3b
#include "decode_inst.cuh"
