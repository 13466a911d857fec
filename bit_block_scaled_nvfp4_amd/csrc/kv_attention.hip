// The streaming kernels over the FP8 cache, and the launch of its attentions.
#include "kv_attention_stream.h"

namespace nvfp4 {

hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, int head_dim, bool bf16,
                            hipStream_t stream) {
  return launch_any<attn::Cache::Fp8>(a, p, head_dim, bf16, stream);
}

}  // namespace nvfp4
