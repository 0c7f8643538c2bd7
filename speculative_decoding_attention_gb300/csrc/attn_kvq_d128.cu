// attn_kvq_d128.cu -- attention over the 4-bit cache, head_dim 128.
#include "attn_kvq.cuh"

namespace wm {

cudaError_t launch_kvq_attn_d128(const KvqAttnParams &p, int n_cta, cudaStream_t stream) {
    return launch_kvq_attn_d<128>(p, n_cta, stream);
}

}  // namespace wm
