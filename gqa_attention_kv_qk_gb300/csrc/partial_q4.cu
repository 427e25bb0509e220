// partial_q4.cu -- the tensor-core partial kernels (partial_tc.cuh) of 4-bit caches.
#include "partial_tc.cuh"

namespace uaa {

cudaError_t launch_partial_q4(const PartialParams& p, const PartialMaps& m, int n_head_tiles, int n_ctas, cudaStream_t s)
{
    return p.first_tokens > 0 ? launch_kv<kKvQ4, true>(p, m, n_head_tiles, n_ctas, s)
                              : launch_kv<kKvQ4, false>(p, m, n_head_tiles, n_ctas, s);
}

}  // namespace uaa
