// The tiled kernels over the 4-bit cache.
#include "kv_attention_tiled.h"

namespace nvfp4 {

hipError_t launch_attention_tiled_fp4(const AttnArgs& a, int head_dim, bool bf16, hipStream_t stream) {
  return launch_tiled<attn::Cache::Fp4>(a, head_dim, bf16, stream);
}

}  // namespace nvfp4
