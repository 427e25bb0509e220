// partial_tc.cu -- the tensor-core partial kernels (partial_tc.cuh) of launches
// without first tokens behind a window, and the choice among all of them.
#include "partial_tc.cuh"

namespace uaa {
namespace {

int kv_kind(int kv_dtype)
{
    if (kv_dtype == UAA_DTYPE_Q4) return kKvQ4;
    return kv_dtype == UAA_DTYPE_Q8 ? kKvQ8 : (kv_dtype == UAA_DTYPE_VQ8 ? kKvVq8 : kKvBf16);
}

template <int KV>
int keys_per_stage_kv(int D, int nht)
{
    switch (D) {
    case 64: return (nht == 2 ? KeyGroups<64, KV, 2>::kMG : KeyGroups<64, KV>::kMG) * kTileKeys;
    case 128: return (nht == 2 ? KeyGroups<128, KV, 2>::kMG : KeyGroups<128, KV>::kMG) * kTileKeys;
    default: return KeyGroups<256, KV>::kMG * kTileKeys;
    }
}

}  // namespace

int partial_tc_keys_per_stage(int D, int kv_dtype, int nht)
{
    switch (kv_kind(kv_dtype)) {
    case kKvQ4: return keys_per_stage_kv<kKvQ4>(D, nht);
    case kKvQ8: return keys_per_stage_kv<kKvQ8>(D, nht);
    case kKvVq8: return keys_per_stage_kv<kKvVq8>(D, nht);
    default: return keys_per_stage_kv<kKvBf16>(D, nht);
    }
}

int partial_tc_ctas_per_sm(int D, int kv_dtype, int nht) { return ctas_per_sm(D, kv_kind(kv_dtype), nht); }

size_t partial_tc_smem_bytes(int D, int kv_dtype, int n_head_tiles)
{
    switch (kv_kind(kv_dtype)) {
    case kKvQ4: return smem_bytes_kv<kKvQ4>(D, n_head_tiles);
    case kKvQ8: return smem_bytes_kv<kKvQ8>(D, n_head_tiles);
    case kKvVq8: return smem_bytes_kv<kKvVq8>(D, n_head_tiles);
    default: return smem_bytes_kv<kKvBf16>(D, n_head_tiles);
    }
}

cudaError_t launch_partial_tc(const PartialParams& p, const PartialMaps& m, int kv_dtype, int n_head_tiles,
                              int n_ctas, cudaStream_t s)
{
    if (kv_dtype == UAA_DTYPE_Q4) return launch_partial_q4(p, m, n_head_tiles, n_ctas, s);
    if (p.first_tokens > 0) return launch_partial_tc_first(p, m, kv_dtype, n_head_tiles, n_ctas, s);
    switch (kv_kind(kv_dtype)) {
    case kKvQ8: return launch_kv<kKvQ8, false>(p, m, n_head_tiles, n_ctas, s);
    case kKvVq8: return launch_kv<kKvVq8, false>(p, m, n_head_tiles, n_ctas, s);
    default: return launch_kv<kKvBf16, false>(p, m, n_head_tiles, n_ctas, s);
    }
}

}  // namespace uaa
