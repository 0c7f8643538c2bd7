// attn_kvq_d256.cu -- attention over the 4-bit cache, head_dim 256.
#include "attn_kvq.cuh"

namespace wm {

cudaError_t launch_kvq_attn_d256(const KvqAttnParams &p, int n_cta, cudaStream_t stream) {
    return launch_kvq_attn_d<256>(p, n_cta, stream);
}

}  // namespace wm
