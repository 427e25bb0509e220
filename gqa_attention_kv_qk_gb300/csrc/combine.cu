// combine.cu -- step 3 of the decode step: log-sum-exp merge of the records of
// units that the stream-K partition cut between CTAs, with the per-head sink.
//
// One CTA per unit (sequence, kv head, group of (token, head) query rows: the
// query heads of the kv head for a decode step). A unit that lies inside one
// CTA's range was written by the partial kernel already and is skipped. For a
// cut unit with records (o_c normalised, e_c the log2-sum-exp of the final
// logits) from its owner CTAs, and the sink logit z_h of each head (llamay
// "Models and formats", "Architectures": a per-head sink in the softmax
// denominator):
//   M   = max(max_c e_c, z_h log2 e)
//   out = sum_c o_c 2^(e_c - M) / (sum_c 2^(e_c - M) + 2^(z_h log2 e - M))
// which is the full softmax over every visible key with the sink's mass in the
// denominator only. A sequence with no visible key gets zeros.
//
// Every range is non-empty, so the owners of a cut unit's stages are exactly the
// ranges cA .. cB, which the partial kernel leaves per unit (UnitOwners in
// internal.cuh). The record weights are formed per
// head from one parallel round of loads; every thread then loads all records'
// rows for four output elements before it adds any of them. The CTA has a
// thread per four output elements of a unit (128 to 512 threads), so a unit of
// up to 16 rows of 128 dims is merged in one round of loads: the merge is a
// chain of dependent loads, not a stream of bytes.
#include "internal.cuh"

namespace uaa {
namespace {

constexpr int kCombineMinThreads = 128;
constexpr int kCombineMaxThreads = 512;
constexpr int kRecBatch = 4;     // records loaded together per output element

// D, HC (query rows per unit: 8, 16 or 24) are template arguments: divisions by them at
// run time were most of the code, and a kernel of a few microseconds that runs cold
// pays for every line of it (5 us for a one-sequence step's combine, of 14).
template <int D, int HC>
__global__ void __launch_bounds__(kCombineMaxThreads) combine_kernel(const CombineParams p)
{
    extern __shared__ float wts[];  // [R][HC]: record log2-sum-exp, then weights
    grid_dependency_wait();         // the partial kernel's records are complete
    allow_dependent_launch();
    if (blockIdx.x == gridDim.x - 1) {     // the extra CTA: the partial kernel's range balance
        if (p.bal.header && threadIdx.x < 32) rebalance(p.bal, p.P, threadIdx.x);
        return;
    }

    // the unit's first and last owner, left by the partial kernel (cleared for the next launch)
    unsigned* own = p.owners + 2 * static_cast<size_t>(blockIdx.x);
    const uint2 fl = *reinterpret_cast<const uint2*>(own);
    const unsigned first = fl.x, last = fl.y;
    const int units = p.Hkv * p.head_groups;
    const int b = blockIdx.x / units, u = blockIdx.x - b * units;
    const int kvh = u / p.head_groups, hg = u - kvh * p.head_groups;
    const int r0 = hg * HC;                      // the unit's first query row (query_row)
    const int nh = min(HC, p.q_len * p.G - r0);  // its query rows
    const int tid = threadIdx.x, nthr = blockDim.x;
    __syncthreads();  // every thread has read the pair
    if (tid == 0) *reinterpret_cast<uint2*>(own) = make_uint2(0u, 0u);
    const int cA = static_cast<int>(first & 0x7fffffffu) - 1, cB = static_cast<int>(last) - 1;
    const bool empty = first == 0u || last == 0u;  // no visible key: zeros
    if (!empty && cA == cB) return;                // a whole unit: the partial kernel wrote it
    if (!empty && (cA < 0 || cB < cA || cB >= p.P)) {  // owner words no range of this launch wrote: not read further
        if (tid == 0) atomicOr(p.status, UAA_DEVFLAG_TIMEOUT);
        return;
    }
    const bool first_is_slot0 = (first & 0x80000000u) != 0u;
    const int R = empty ? 0 : cB - cA + 1;  // the unit's records: owners cA .. cB

    for (int i = tid; i < R * HC; i += nthr)
        if (i % HC < nh) wts[i] = p.rec_lse[static_cast<size_t>(record_of(cA + i / HC, cA, first_is_slot0)) * HC + i % HC];
    __syncthreads();
    for (int hc = tid; hc < nh && !empty; hc += nthr) {
        const float z = p.sink ? p.sink[kvh * p.G + (r0 + hc) % p.G] * kLog2e : -INFINITY;
        float M = z;
#pragma unroll 4
        for (int r = 0; r < R; ++r) M = fmaxf(M, wts[r * HC + hc]);
        float den = 0.f;
        if (M != -INFINITY) {
            den = p.sink ? exp2f(z - M) : 0.f;
#pragma unroll 1
            for (int r = 0; r < R; ++r) {
                const float e = wts[r * HC + hc];
                const float w = e == -INFINITY ? 0.f : exp2f(e - M);
                wts[r * HC + hc] = w;
                den += w;
            }
        }
        const float inv = den > 0.f ? 1.f / den : 0.f;
#pragma unroll 1
        for (int r = 0; r < R; ++r) wts[r * HC + hc] = M == -INFINITY ? 0.f : wts[r * HC + hc] * inv;
    }
    __syncthreads();
    // four neighbouring elements of a row per thread
#pragma unroll 1
    for (int i = tid; i < nh * (D / 4); i += nthr) {
        const int hc = i / (D / 4), d = 4 * (i % (D / 4));
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int r1 = 0; r1 < R; r1 += kRecBatch) {
            float4 v[kRecBatch];
#pragma unroll
            for (int r = 0; r < kRecBatch; ++r) {
                v[r] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r1 + r < R) {
                    const int rec = record_of(cA + r1 + r, cA, first_is_slot0);
                    v[r] = *reinterpret_cast<const float4*>(p.rec_o + (static_cast<size_t>(rec) * HC + hc) * D + d);
                }
            }
#pragma unroll
            for (int r = 0; r < kRecBatch; ++r)
                if (r1 + r < R) {
                    const float w = wts[(r1 + r) * HC + hc];
                    acc[0] = fmaf(w, v[r].x, acc[0]);
                    acc[1] = fmaf(w, v[r].y, acc[1]);
                    acc[2] = fmaf(w, v[r].z, acc[2]);
                    acc[3] = fmaf(w, v[r].w, acc[3]);
                }
        }
        const size_t at = query_row(b, r0 + hc, kvh, p.G, p.Hq, p.q_len) * D + d;
        if (p.out_dtype == UAA_DTYPE_F32) {
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[0], acc[1]), hi = __floats2bfloat162_rn(acc[2], acc[3]);
            uint2 w;
            memcpy(&w.x, &lo, 4);
            memcpy(&w.y, &hi, 4);
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) = w;
        }
    }
}

template <int D, int HC>
cudaError_t launch_combine_of(const CombineParams& p, cudaStream_t s)
{
    // one CTA per unit, and one that rebalances the partial kernel's ranges; a
    // thread per four output elements of a unit's rows, in whole warps
    const long long blocks = static_cast<long long>(p.B) * p.Hkv * p.head_groups + 1;
    if (blocks == 1) return cudaSuccess;
    const int rows = HC < p.q_len * p.G ? HC : p.q_len * p.G;
    int threads = (rows * D / 4 + 31) / 32 * 32;
    threads = threads < kCombineMinThreads ? kCombineMinThreads : (threads > kCombineMaxThreads ? kCombineMaxThreads : threads);
    // weights for up to every range's record of a unit
    const size_t smem = static_cast<size_t>(p.P) * HC * 4;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(combine_kernel<D, HC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(combine_kernel<D, HC>, dim3(static_cast<unsigned>(blocks)), dim3(threads), smem, s, p);
}

}  // namespace

cudaError_t launch_combine(const CombineParams& p, cudaStream_t s)
{
    if (p.heads_per_cta == 8) {
        switch (p.D) {
        case 64: return launch_combine_of<64, 8>(p, s);
        case 128: return launch_combine_of<128, 8>(p, s);
        case 256: return launch_combine_of<256, 8>(p, s);
        default: return cudaErrorInvalidValue;
        }
    }
    if (p.heads_per_cta == 24) return p.D == 64 ? launch_combine_of<64, 24>(p, s) : cudaErrorInvalidValue;
    if (p.heads_per_cta != 16) return cudaErrorInvalidValue;
    switch (p.D) {
    case 64: return launch_combine_of<64, 16>(p, s);
    case 128: return launch_combine_of<128, 16>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace uaa
