// cache_rows.cu -- rows on their way into and out of a cache outside a step's
// attention: the 4-bit quantiser that fills a cache from existing values, the
// reader that gives cached rows back as values, and the widening of a 4-bit cache's
// visible rows to fp16 for a prefill chunk. All stream: each value is read once and
// written once, a thread takes 16 (quantise) or 8 (read) neighbouring values with
// 16-byte accesses, and HBM is the bound for anything beyond a few hundred rows.
#include "internal.cuh"

namespace uaa {
namespace {

constexpr int kRowThreads = 256;

template <typename T>
__device__ __forceinline__ void load16(const T* src, float (&x)[16])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 a = reinterpret_cast<const float4*>(src)[i];
            x[4 * i] = a.x, x[4 * i + 1] = a.y, x[4 * i + 2] = a.z, x[4 * i + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 a = reinterpret_cast<const uint4*>(src)[i];
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
    }
}

// Half a group per thread: two neighbouring lanes share a group's maximum.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) q4_quantize_kernel(const T* x, int64_t n_halves, uint2* codes,
                                                                  __half* scales)
{
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRowThreads;
    // every lane of a warp runs the same number of rounds (the pair's exchange)
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kRowThreads; i0 < n_halves; i0 += step) {
        const int64_t i = i0 + threadIdx.x;
        const bool in = i < n_halves;  // n_halves is even: a pair is in or out as a whole
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0.f;
        if (in) load16(x + 16 * i, v);
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(v[j]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const __half s = q4_scale(m);
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j >> 3] |= q4_nibble(v[j], __half2float(s)) << (4 * (j & 7));
        if (in) {
            codes[i] = make_uint2(w[0], w[1]);
            if (!(i & 1)) scales[i >> 1] = s;
        }
    }
}

__device__ __forceinline__ void store8(void* out, int dtype, size_t at, const float (&x)[8])
{
    if (dtype == UAA_DTYPE_F32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            memcpy(&w[i], &h, 4);
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Values 8 e .. 8 e + 7 of cache row `row` (element type: 4 fp32, 2 bf16, 1 int8
// codes with one fp32 scale, 0 4-bit codes with an fp16 scale per 32).
__device__ __forceinline__ void load8_row(const void* cache, const float* scale, int type, size_t row, int D, int e,
                                          float (&x)[8])
{
    const size_t at = row * D + 8 * e;
    if (type == 4) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(cache) + at);
        const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(cache) + at + 4);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else if (type == 2) {
        const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(cache) + at);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    } else if (type == 1) {
        const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const int8_t*>(cache) + at);
        const float s = scale[row];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = static_cast<float>(static_cast<int8_t>((j < 4 ? a.x : a.y) >> (8 * (j & 3)))) * s;
    } else {
        const uint32_t a = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(cache) + at / 2);
        const float s = __half2float(reinterpret_cast<const __half*>(scale)[at / 32]);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (static_cast<float>((a >> (4 * j)) & 15u) - 8.f) * s;
    }
}

// A thread per 8 values of a row [b][t][kvh] of the keys (blockIdx.y 0) or values.
__global__ void __launch_bounds__(kRowThreads) cache_read_kernel(const ReadParams p)
{
    grid_dependency_wait();  // the step that appended the rows is complete
    const bool is_v = blockIdx.y == 1;
    void* out = is_v ? p.v_out : p.k_out;
    const int units = p.D / 8;
    const int64_t total = static_cast<int64_t>(p.B) * p.n * p.Hkv * units;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
    if (!out || i >= total) return;
    const int e = static_cast<int>(i % units);
    const int64_t r = i / units;
    const int h = static_cast<int>(r % p.Hkv);
    const int64_t bt = r / p.Hkv;
    const int b = static_cast<int>(bt / p.n), t = static_cast<int>(bt - static_cast<int64_t>(b) * p.n);
    const int64_t pos = static_cast<int64_t>(p.start ? p.start[b] : 0) + t;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    long long row = -1;
    if (pos >= 0 && pos < p.cap) row = cache_row(p.pages, p.Hkv, p.cap, b, h, static_cast<int>(pos));
    const int type = p.kv_dtype == UAA_DTYPE_F32   ? 4
                     : p.kv_dtype == UAA_DTYPE_Q4  ? 0
                     : p.kv_dtype == UAA_DTYPE_Q8 || (p.kv_dtype == UAA_DTYPE_VQ8 && is_v) ? 1
                                                                                          : 2;
    if (row >= 0)
        load8_row(is_v ? p.v_cache : p.k_cache, is_v ? p.v_scale : p.k_scale, type, static_cast<size_t>(row), p.D, e, x);
    store8(out, p.out_dtype, static_cast<size_t>(i) * 8, x);
}

// A CTA per 64 rows of (sequence, kv head), keys (blockIdx.z 0) or values: a thread
// takes 16 values (8 bytes of codes) at a time. Rows in 128-row blocks (the prefill
// kernel's) that no token of the chunk sees are left alone; in the others rows that
// none sees, or without a page, are zeros.
constexpr int kWidenRows = 64;

__global__ void __launch_bounds__(kRowThreads) widen_q4_kernel(const WidenParams p)
{
    grid_dependency_wait();  // the append's rows and lengths are complete
    const int row0 = blockIdx.x * kWidenRows;
    const int bh = blockIdx.y, b = bh / p.Hkv, h = bh - b * p.Hkv;
    const bool is_v = blockIdx.z == 1;
    const int n = p.seq_lens[b];
    if (n > p.row_cap) {  // longer than the caller's bound: the prefill kernel leaves zero rows
        if (blockIdx.x == 0 && h == 0 && !is_v && threadIdx.x == 0 && n <= p.cap)
            atomicOr(p.status, UAA_DEVFLAG_LEN_HINT);
        return;
    }
    if (n < p.q_len || row0 >= n) return;
    const Keys keys = key_range(n, p.window, p.first_tokens);  // the chunk's union
    const int block = row0 / kPrefillKeys * kPrefillKeys;
    if (block + kPrefillKeys <= keys.lo && block >= keys.first) return;
    const void* cache = is_v ? p.v_cache : p.k_cache;
    const __half* scale = reinterpret_cast<const __half*>(is_v ? p.v_scale : p.k_scale);
    __half* out = static_cast<__half*>(is_v ? p.v_out : p.k_out) + static_cast<size_t>(bh) * p.row_cap * p.D;
    const int per_row = p.D / 16;
    for (int i = threadIdx.x; i < kWidenRows * per_row; i += kRowThreads) {
        const int r = row0 + i / per_row, e = i % per_row;
        if (r >= n) break;
        const bool seen = r < keys.first || r >= keys.lo;
        const long long row = seen ? cache_row(p.pages, p.Hkv, p.cap, p.b_off + b, h, r) : -1;
        uint2 c = make_uint2(0x88888888u, 0x88888888u);  // code 0
        __half2 s = __half2half2(__float2half_rn(0.f));
        if (row >= 0) {
            c = reinterpret_cast<const uint2*>(cache)[row * per_row + e];
            s = __half2half2(scale[row * (p.D / 32) + e / 2]);
        } else if (seen && e == 0) {
            atomicOr(p.status, UAA_DEVFLAG_PAGE);
        }
        // byte j (codes 2 j and 2 j + 1) in both halves of a word; the low nibble of the
        // lower half as 1024 + u, the high nibble of the upper one as 64 + u, less 1032 and
        // 72: the codes, exactly; times the scale (3 bits times 8), exactly
        const uint32_t exponents = 0x54006400u + (static_cast<uint32_t>(p.D) >> 16);  // not a literal: one and-or
        const __half2 off = __halves2half2(__float2half_rn(1032.f), __float2half_rn(72.f));
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t u = __byte_perm(j < 4 ? c.x : c.y, 0, 0x0101 * (j & 3) | 0x4040);
            const uint32_t t = (u & 0x00F0000Fu) | exponents;
            __half2 v;
            memcpy(&v, &t, 4);
            const __half2 x = __hmul2(__hsub2(v, off), s);
            memcpy(&w[j], &x, 4);
        }
        uint4* o = reinterpret_cast<uint4*>(out + static_cast<size_t>(r) * p.D + 16 * e);
        o[0] = make_uint4(w[0], w[1], w[2], w[3]);
        o[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

}  // namespace

cudaError_t launch_widen_q4(const WidenParams& p, cudaStream_t s)
{
    if (p.B == 0) return cudaSuccess;
    if (static_cast<long long>(p.B) * p.Hkv > 65535) return cudaErrorInvalidConfiguration;
    return launch_dependent(widen_q4_kernel,
                            dim3(static_cast<unsigned>((p.row_cap + kWidenRows - 1) / kWidenRows),
                                 static_cast<unsigned>(p.B * p.Hkv), 2),
                            dim3(kRowThreads), 0, s, p);
}

cudaError_t launch_q4_quantize(const void* x, int dtype, int64_t n_rows, int D, uint8_t* codes, __half* scales,
                               cudaStream_t s)
{
    const int64_t n_halves = n_rows * (D / 16);
    const int64_t blocks64 = (n_halves + kRowThreads - 1) / kRowThreads;
    const unsigned blocks = static_cast<unsigned>(blocks64 < (1 << 20) ? blocks64 : 1 << 20);
    if (dtype == UAA_DTYPE_F32)
        q4_quantize_kernel<<<blocks, kRowThreads, 0, s>>>(static_cast<const float*>(x), n_halves,
                                                          reinterpret_cast<uint2*>(codes), scales);
    else
        q4_quantize_kernel<<<blocks, kRowThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(x), n_halves,
                                                          reinterpret_cast<uint2*>(codes), scales);
    return cudaGetLastError();
}

cudaError_t launch_cache_read(const ReadParams& p, cudaStream_t s)
{
    const int64_t total = static_cast<int64_t>(p.B) * p.n * p.Hkv * (p.D / 8);
    const int64_t blocks = (total + kRowThreads - 1) / kRowThreads;
    if (blocks > 2147483647LL) return cudaErrorInvalidConfiguration;
    return launch_dependent(cache_read_kernel, dim3(static_cast<unsigned>(blocks), 2), dim3(kRowThreads), 0, s, p);
}

}  // namespace uaa
