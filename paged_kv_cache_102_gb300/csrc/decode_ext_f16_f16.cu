// CUDA-core decode with a window or kept logits: f16 activations, f16 cache.
#include "pkv_device.cuh"
#define PKV_ACT pkv::kF16
#define PKV_CACHE pkv::kF16
#define PKV_EXT true
#define PKV_LAUNCH_NAME launch_decode_ext_f16_f16
#include "decode_inst.cuh"
