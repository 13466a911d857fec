// The tiled kernels over the FP8 cache.
#include "kv_attention_tiled.h"

namespace nvfp4 {

hipError_t launch_attention_tiled(const AttnArgs& a, int head_dim, bool bf16, hipStream_t stream) {
  return launch_tiled<attn::Cache::Fp8>(a, head_dim, bf16, stream);
}

}  // namespace nvfp4
