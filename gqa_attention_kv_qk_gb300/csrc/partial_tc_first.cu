// partial_tc_first.cu -- the tensor-core partial kernels (partial_tc.cuh) of launches
// with first tokens behind a window.
#include "partial_tc.cuh"

namespace uaa {

cudaError_t launch_partial_tc_first(const PartialParams& p, const PartialMaps& m, int kv_dtype, int n_head_tiles,
                                    int n_ctas, cudaStream_t s)
{
    switch (kv_dtype) {
    case UAA_DTYPE_Q8: return launch_kv<kKvQ8, true>(p, m, n_head_tiles, n_ctas, s);
    case UAA_DTYPE_VQ8: return launch_kv<kKvVq8, true>(p, m, n_head_tiles, n_ctas, s);
    default: return launch_kv<kKvBf16, true>(p, m, n_head_tiles, n_ctas, s);
    }
}

}  // namespace uaa
