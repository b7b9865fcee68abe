// kvq_attn_e2m1_d64.cu -- the E2M1 attention kernel's instances at head_dim 64.
#include "kvq_attn_e2m1.cuh"

namespace kvq {

cudaError_t launch_attention_e2m1_d64(const AttnArgs &a, bool merge, cudaStream_t stream)
{
    return launch_e2m1_dim<64>(a, merge, stream);
}

}  // namespace kvq
