// CUDA-core decode with a window or kept logits: bf16 activations, e4m3 cache.
#include "pkv_device.cuh"
#define PKV_ACT pkv::kBF16
#define PKV_CACHE pkv::kE4M3
#define PKV_EXT true
#define PKV_LAUNCH_NAME launch_decode_ext_bf16_e4m3
#include "decode_inst.cuh"
