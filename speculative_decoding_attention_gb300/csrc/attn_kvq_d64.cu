// attn_kvq_d64.cu -- attention over the 4-bit cache, head_dim 64.
#include "attn_kvq.cuh"

namespace wm {

cudaError_t launch_kvq_attn_d64(const KvqAttnParams &p, int n_cta, cudaStream_t stream) {
    return launch_kvq_attn_d<64>(p, n_cta, stream);
}

}  // namespace wm
