// append.cuh -- arithmetic and stores of the append kernels that hold 16 elements of a head
// row per thread (append.cu, packed_append.cu).
#pragma once

#include "internal.cuh"

namespace uaa {
namespace {

__device__ __forceinline__ void store8_f32(float* dst, const float (&y)[8], float scale)
{
    reinterpret_cast<float4*>(dst)[0] = make_float4(y[0] * scale, y[1] * scale, y[2] * scale, y[3] * scale);
    reinterpret_cast<float4*>(dst)[1] = make_float4(y[4] * scale, y[5] * scale, y[6] * scale, y[7] * scale);
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    uint32_t u;
    memcpy(&u, &h, 4);
    return u;
}

__device__ __forceinline__ void store8_bf16(void* dst, const float (&y)[8])
{
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(bf16x2_bits(y[0], y[1]), bf16x2_bits(y[2], y[3]), bf16x2_bits(y[4], y[5]), bf16x2_bits(y[6], y[7]));
}

__device__ __forceinline__ void store8_codes(int8_t* dst, const float (&y)[8], float s)
{
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(vq8_code(y[i], s))) << (8 * (i & 3));
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
}

// The 4-bit codes of 8 values with scale s.
__device__ __forceinline__ uint32_t q4_word(const float (&y)[8], float s)
{
    uint32_t w = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= q4_nibble(y[i], s) << (4 * i);
    return w;
}

// Sum / maximum over the U lanes that hold one head row (aligned groups of U lanes).
template <int U>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = U / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int U>
__device__ __forceinline__ float group_max(float v)
{
#pragma unroll
    for (int o = U / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

}  // namespace
}  // namespace uaa
