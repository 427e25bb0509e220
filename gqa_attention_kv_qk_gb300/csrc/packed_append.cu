// packed_append.cu -- the append of a packed batch: per-head RMSNorm, the rotation at each
// row's own positions (one axis or several), k and v rows into their slots, rotated q rows
// out. It streams: q, k and v rows are read once, q rows leave as fp32, k and v rows as the
// cache holds them; HBM is the bound (for rows read and written in whole 32-byte sectors),
// instruction issue next.
//
// A CTA takes up to 8 neighbouring rows of the packed tensors (whose tokens may lie at
// strides of their own), a warp one token's head rows, or a share of them where there are
// fewer tokens than warps. A thread holds 16 elements of a head row, as two runs of 8 at e0
// and e1: NeoX pairs element e0 + j with e1 + j, otherwise the runs are contiguous; D / 16
// threads make a row. So a lane's places in a row, its 8 pairs' (cos, sin) and the token's slot
// are the same for every chunk of rows (finding them anew for each was half of 516
// instructions a chunk). The next chunk's loads are on their way while one is worked on. The
// angles are reduced in 64-bit integers by steps from the host (rope_cos_sin_two).
//
// bf16 keys: cos, sin and a norm's factor are sums of two floats and the products exact, so that
// the fp32 result is the nearest float to the exact one, or now and then its neighbour,
// which is then rounded to bf16. Everything else takes norm and rotation in plain fp32. 16,200
// normed tokens of 32 + 2 x 8 heads of 128 take 113 us (32 KiB a token: 4.7 TB/s), 8,191 tokens without
// a norm 60 us (4.5 TB/s); with keys in plain fp32 too, whose bf16 rows then differ in one of some
// 10^4 elements, the former took 105. The steps of equal lengths recompute in fp64 what lies near a
// rounding boundary: the fp64 unit took 130 us of 236 here.
#include "append.cuh"
#include "schedule.cuh"

namespace uaa {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowTokens = 8;     // tokens per CTA at most

// 32 bytes in one store (addresses of whole rows' runs of 8 floats are 32-byte aligned
// where the tensor's base is).
__device__ __forceinline__ void store8_wide(float* dst, const float (&y)[8], float s)
{
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(y[0] * s), "f"(y[1] * s),
                 "f"(y[2] * s), "f"(y[3] * s), "f"(y[4] * s), "f"(y[5] * s), "f"(y[6] * s), "f"(y[7] * s)
                 : "memory");
}

// Eight elements as loaded, and as fp32.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* src)
    {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
    }
    __device__ __forceinline__ float at(int j) const
    {
        const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
        if constexpr (sizeof(T) == 4) return __uint_as_float(u[j]);
        return __uint_as_float(j & 1 ? u[j >> 1] & 0xffff0000u : u[j >> 1] << 16);
    }
};

// cos and sin of pos * theta'_p times mscale as sums of two floats each (c, s) and what they lack
// (c_lo, s_lo), within 2^-27. The angle in units of pi is the low 64 bits of pos * g (angle_step);
// less the nearest multiple of 1/2 it is within 1/4, x = pi times that as two floats, and the Taylor
// series are summed with their first terms exact: sin x = x + x^3 (-1/6 + ..), whose second part is
// below 0.08 and so off by 2^-27 in fp32, and cos x = 1 - x^2 / 2 + x^4 (1/24 - ..).
__device__ __forceinline__ float4 rope_cos_sin_two(int pos, unsigned long long g, float mscale)
{
    constexpr float kPi = 3.14159265358979323846f, kPiLo = static_cast<float>(3.14159265358979323846 - static_cast<double>(kPi));
    const unsigned long long t = static_cast<unsigned long long>(pos) * g;
    const int quarter = static_cast<int>((t + (1ull << 61)) >> 62);
    const long long r = static_cast<long long>(t - (static_cast<unsigned long long>(quarter) << 62));
    const float r0 = __ll2float_rn(r);
    const float rh = r0 * 0x1p-63f, rl = __ll2float_rn(r - __float2ll_rn(r0)) * 0x1p-63f;
    const float x = __fmul_rn(rh, kPi), xl = fmaf(rh, kPi, -x) + fmaf(rh, kPiLo, rl * kPi);
    const float z = __fmul_rn(x, x), zl = fmaf(x, x, -z) + 2.f * x * xl;
    float ps = fmaf(z, -1.f / 39916800.f, 1.f / 362880.f);
    ps = fmaf(z, ps, -1.f / 5040.f);
    ps = fmaf(z, ps, 1.f / 120.f);
    ps = fmaf(z, ps, -1.f / 6.f);
    float pc = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
    pc = fmaf(z, pc, -1.f / 720.f);
    pc = fmaf(z, pc, 1.f / 24.f);
    const float s_rest = fmaf(x * z, ps, fmaf(-0.5f * z, xl, xl));
    const float sn = __fadd_rn(x, s_rest), sl = __fsub_rn(s_rest, __fsub_rn(sn, x));
    const float w = -0.5f * z, c0 = __fadd_rn(1.f, w);
    const float c_rest = __fsub_rn(w, __fsub_rn(c0, 1.f)) + fmaf(z * z, pc, -0.5f * zl);
    const float cn = __fadd_rn(c0, c_rest), cl = __fsub_rn(c_rest, __fsub_rn(cn, c0));
    // turned by the quarters
    const bool odd = quarter & 1;
    const float a = odd ? sn : cn, al = odd ? sl : cl, b = odd ? cn : sn, bl = odd ? cl : sl;
    const float fa = ((quarter + 1) & 2 ? -mscale : mscale), fb = (quarter & 2 ? -mscale : mscale);
    const float c = __fmul_rn(a, fa), s = __fmul_rn(b, fb);
    return make_float4(c, s, fmaf(a, fa, -c) + al * fa, fmaf(b, fb, -s) + bl * fb);
}

// a + b as the nearest float and what it lacks.
__device__ __forceinline__ float2 sum_two(float a, float b)
{
    const float sum = __fadd_rn(a, b), bb = __fsub_rn(sum, a);
    return make_float2(sum, __fadd_rn(__fsub_rn(a, __fsub_rn(sum, bb)), __fsub_rn(b, bb)));
}

// a c - b s as the nearest float (nearly always), every operand a sum of two (x: the float, y: what it
// lacks). A sum that is infinite, of infinite operands or past the largest float, stays so: what it
// lacks is no number then.
__device__ __forceinline__ float dot_two(float2 a, float2 b, float2 c, float2 s)
{
    const float p = __fmul_rn(a.x, c.x), q = -__fmul_rn(b.x, s.x);
    const float2 sum = sum_two(p, q);
    const float rest = (fmaf(a.x, c.x, -p) - fmaf(b.x, s.x, q)) + fmaf(a.x, c.y, -b.x * s.y) + fmaf(a.y, c.x, -b.y * s.x);
    return isinf(sum.x) ? sum.x : sum.x + (sum.y + rest);
}

// Q4: a 4-bit cache. NORM: q and k rows are normed. Template arguments, as they cost the
// others registers and instructions of every chunk.
template <int D, typename T, bool Q4, bool NORM>
__global__ void __launch_bounds__(kRowThreads, NORM || sizeof(T) == 4 ? 3 : 4)
append_rows_kernel(const AppendParams p, const ScheduleParams sched)
{
    constexpr int HALF = D / 2;
    constexpr int U = D / 16;   // threads per head row
    constexpr int R = 32 / U;   // rows of a chunk
    __shared__ float2 cs[kRowTokens * HALF], cs_lo[kRowTokens * HALF];
    __shared__ float nw[NORM ? 2 * D : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    if (sched.header && blockIdx.x == gridDim.x - 1) {  // the attention's work list
        __shared__ __align__(8) int scratch[kScheduleWords];
        build_schedule(sched, scratch);
        return;
    }
    // warp w takes token w % TPS of the CTA's, every (8 / TPS)-th of its chunks: R rows of q, k or v
    const int TPS = p.tokens_per_cta;  // 1, 2, 4 or 8
    const int t0 = blockIdx.x * TPS, nt = min(TPS, p.pk.n_tokens - t0);
    const int tok = warp % TPS, part = warp / TPS, parts = kRowThreads / 32 / TPS;
    const int t = t0 + tok;
    const bool neox = p.style == UAA_ROPE_NEOX;
    const int nqc = (p.Hq + R - 1) / R, nkc = (p.Hkv + R - 1) / R;
    int n_chunks = tok < nt ? nqc + 2 * nkc : 0;
    const int u = lane & (U - 1), rl = lane / U;
    // a lane's elements of a q or k row, and of a v row (two neighbouring runs)
    const bool rot = neox && 8 * u < p.half_rot;
    const int e0 = neox ? (rot ? 8 * u : 2 * p.half_rot + 16 * (u - p.half_rot / 8)) : 16 * u;
    const int e1 = rot ? e0 + p.half_rot : e0 + 8;
    auto load = [&](int c, Raw8<T>& a, Raw8<T>& b) {
        const int kind = c < nqc ? 0 : c < nqc + nkc ? 1 : 2;
        const int head = (c - (kind == 0 ? 0 : kind == 1 ? nqc : nqc + nkc)) * R + rl;
        if (head >= (kind == 0 ? p.Hq : p.Hkv)) return;
        const T* src = static_cast<const T*>(kind == 0 ? p.q : kind == 1 ? p.k_new : p.v_new) +
                       static_cast<size_t>(t) * (kind == 0 ? p.pk.q_stride : kind == 1 ? p.pk.k_stride : p.pk.v_stride) + head * D;
        a.load(src + (kind < 2 ? e0 : 16 * u));
        b.load(src + (kind < 2 ? e1 : 16 * u + 8));
    };
    Raw8<T> ra{}, rb{};
    int c = part;
    if (c < n_chunks) load(c, ra, rb);
    const int seq = tok < nt ? p.pk.token_seq[t] : -1;
    const long long slot_at = tok < nt ? p.pk.slots[t] : -1;

    // the tables, while the first loads are on their way
    if constexpr (NORM)
        for (int i = tid; i < 2 * D; i += kRowThreads) nw[i] = (i < D ? p.q_norm_w[i] : p.k_norm_w[i - D]) + p.norm_offset;
    auto pair_pos = [&](int r, int pp) {  // the position that turns pair pp of packed row r
        return p.pk.axis_pos ? p.pk.axis_pos[static_cast<size_t>(p.pk.pair_axis[pp]) * p.pk.n_tokens + r] : p.pk.positions[r];
    };
    for (int i = tid; i < nt * HALF; i += kRowThreads) {
        const int pp = i & (HALF - 1);
        const float4 v = pp < p.half_rot ? rope_cos_sin_two(pair_pos(t0 + i / HALF, pp), p.pk.angle_step[pp], p.mscale)
                                         : make_float4(1.f, 0.f, 0.f, 0.f);
        cs[i] = make_float2(v.x, v.y);
        cs_lo[i] = make_float2(v.z, v.w);
    }
    __syncthreads();
    if (seq < 0) n_chunks = 0;  // behind the last request

    float* const q_to = p.q_prime ? p.q_prime : p.q_rot_out;
    const bool wide_q = (reinterpret_cast<uintptr_t>(q_to) & 31u) == 0;
    const float2* const cst = cs + tok * HALF + 8 * u;  // this lane's 8 pairs
    const int n_rot = min(max(p.half_rot - 8 * u, 0), 8);  // how many of them turn
    auto norm = [&](float (&x0)[8], float (&x1)[8], const float* w) {
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s0 = fmaf(x0[j], x0[j], s0);
            s1 = fmaf(x1[j], x1[j], s1);
        }
        const float mean = group_sum<U>(s0 + s1) * (1.f / D) + p.eps, r0 = rsqrtf(mean);
        // a Newton step: rsqrtf is off by 2 ulp, and every element of the row by the same
        const float inv = r0 > 0.f ? fmaf(0.5f * r0, fmaf(-(mean * r0), r0, 1.f), r0) : r0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x0[j] = x0[j] * inv * w[e0 + j];
            x1[j] = x1[j] * inv * w[e1 + j];
        }
    };
    auto turn = [&](float (&x0)[8], float (&x1)[8]) {
        if (neox) {
            if (rot) {
#pragma unroll
                for (int j = 0; j < 8; ++j) rope_rotate(x0[j], x1[j], cst[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j < n_rot) rope_rotate(x0[2 * j], x0[2 * j + 1], cst[j]);
                if (j + 4 < n_rot) rope_rotate(x1[2 * j], x1[2 * j + 1], cst[j + 4]);
            }
        }
    };
    // Keys that are rounded to bf16: norm and rotation as if exact, rounded to fp32 once. l0, l1:
    // what the normed elements lack.
    auto norm_exact = [&](float (&x0)[8], float (&x1)[8], float (&l0)[8], float (&l1)[8], const float* w) {
        float2 sum = make_float2(0.f, 0.f);
        auto add = [&](float x) {
            const float q = __fmul_rn(x, x);
            const float2 t = sum_two(sum.x, q);
            sum = make_float2(t.x, sum.y + t.y + (sizeof(T) == 4 ? fmaf(x, x, -q) : 0.f));  // (bf16: exact squares)
        };
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            add(x0[j]);
            add(x1[j]);
        }
#pragma unroll
        for (int o = U / 2; o > 0; o >>= 1) {
            const float h = __shfl_xor_sync(0xffffffffu, sum.x, o), l = __shfl_xor_sync(0xffffffffu, sum.y, o);
            const float2 t = sum_two(sum.x, h);
            sum = make_float2(t.x, t.y + sum.y + l);
        }
        const float2 t = sum_two(sum.x * (1.f / D), p.eps);
        const float m = t.x, ml = fmaf(sum.y, 1.f / D, t.y), r = rsqrtf(m);
        // a Newton step from rsqrtf, whose end is kept apart
        const float mr = __fmul_rn(m, r), mrl = fmaf(m, r, -mr) + ml * r;
        const float rl = r > 0.f ? 0.5f * r * (fmaf(-mr, r, 1.f) - mrl * r) : 0.f;
        auto scale = [&](float& x, float& l, float g) {
            const float a = __fmul_rn(x, g), al = fmaf(x, g, -a), y = __fmul_rn(a, r);
            l = fmaf(a, r, -y) + fmaf(a, rl, al * r);
            x = y;
        };
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            scale(x0[j], l0[j], w[e0 + j]);
            scale(x1[j], l1[j], w[e1 + j]);
        }
    };
    auto turn_exact = [&](float (&x0)[8], float (&x1)[8], const float (&l0)[8], const float (&l1)[8]) {
        const float2* const lo = cs_lo + tok * HALF + 8 * u;
        auto pair = [&](float& a, float& b, float al, float bl, int j) {
            const float2 h = cst[j], l = lo[j], c = make_float2(h.x, l.x), s = make_float2(h.y, l.y);
            const float2 at = make_float2(a, al), bt = make_float2(b, bl);
            a = dot_two(at, bt, c, s);
            b = dot_two(bt, at, c, make_float2(-s.x, -s.y));
        };
        if (neox) {
            if (rot) {
#pragma unroll
                for (int j = 0; j < 8; ++j) pair(x0[j], x1[j], l0[j], l1[j], j);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j < n_rot) pair(x0[2 * j], x0[2 * j + 1], l0[2 * j], l0[2 * j + 1], j);
                if (j + 4 < n_rot) pair(x1[2 * j], x1[2 * j + 1], l1[2 * j], l1[2 * j + 1], j + 4);
            }
        }
    };
    const bool bf16_keys = !Q4 && (p.kv_dtype == UAA_DTYPE_BF16 || p.kv_dtype == UAA_DTYPE_VQ8);
    for (; c < n_chunks; c += parts) {
        const Raw8<T> a = ra, b = rb;
        if (c + parts < n_chunks) load(c + parts, ra, rb);
        float x0[8], x1[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x0[j] = a.at(j);
            x1[j] = b.at(j);
        }
        if (c < nqc) {  // ------------------------------------------------ q rows (the warp's branch)
            const int head = c * R + rl;
            if constexpr (NORM) norm(x0, x1, nw);
            turn(x0, x1);
            const float scale = p.q_prime ? p.qscale : 1.f;
            if (head < p.Hq) {
                float* to = q_to + (static_cast<size_t>(t) * p.Hq + head) * D;
                if (wide_q) {
                    store8_wide(to + e0, x0, scale);
                    store8_wide(to + e1, x1, scale);
                } else {
                    store8_f32(to + e0, x0, scale);
                    store8_f32(to + e1, x1, scale);
                }
            }
            continue;
        }
        const bool is_k = c < nqc + nkc;
        const int head = (c - (is_k ? nqc : nqc + nkc)) * R + rl;
        long long crow = -1;
        if (head < p.Hkv && slot_at >= 0) {
            crow = slot_row(p.pages, p.Hkv, p.cap, p.pk.batch, head, slot_at);
            if (crow < 0 && u == 0) atomicOr(p.status, UAA_DEVFLAG_PAGE);
        }
        const bool stores = crow >= 0;
        const int f0 = is_k ? e0 : 16 * u, f1 = is_k ? e1 : 16 * u + 8;
        if (is_k) {
            if (bf16_keys) {
                float l0[8] = {}, l1[8] = {};
                if constexpr (NORM) norm_exact(x0, x1, l0, l1, nw + D);
                turn_exact(x0, x1, l0, l1);
            } else {
                if constexpr (NORM) norm(x0, x1, nw + D);
                turn(x0, x1);
            }
        }
        void* cache = is_k ? p.k_cache : p.v_cache;
        float* scales = is_k ? p.k_scale : p.v_scale;
        const size_t slot = static_cast<size_t>(crow) * D;
        if (Q4) {
            // 4-bit groups of 32 dims: each run of 8 with those of the 4 neighbouring threads (NeoX
            // halves), or both runs with those of the next thread
            float g0 = 0.f, g1 = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                g0 = fmaxf(g0, fabsf(x0[j]));
                g1 = fmaxf(g1, fabsf(x1[j]));
            }
            const bool halves = is_k && rot;
            if (!halves) g0 = g1 = fmaxf(g0, g1);
            g0 = fmaxf(g0, __shfl_xor_sync(0xffffffffu, g0, 1));
            g1 = fmaxf(g1, __shfl_xor_sync(0xffffffffu, g1, 1));
            const float h0 = __shfl_xor_sync(0xffffffffu, g0, 2), h1 = __shfl_xor_sync(0xffffffffu, g1, 2);
            if (halves) {
                g0 = fmaxf(g0, h0);
                g1 = fmaxf(g1, h1);
            }
            if (stores) {
                const __half s0 = q4_scale(g0), s1 = q4_scale(g1);
                uint8_t* codes = static_cast<uint8_t*>(cache) + slot / 2;
                __half* sc = reinterpret_cast<__half*>(scales) + slot / 32;
                *reinterpret_cast<uint32_t*>(codes + f0 / 2) = q4_word(x0, __half2float(s0));
                *reinterpret_cast<uint32_t*>(codes + f1 / 2) = q4_word(x1, __half2float(s1));
                if (f0 % 32 == 0) sc[f0 / 32] = s0;
                if (f1 % 32 == 0) sc[f1 / 32] = s1;
            }
        } else if (p.kv_dtype == UAA_DTYPE_Q8 || (!is_k && p.kv_dtype == UAA_DTYPE_VQ8)) {
            float amax = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fmaxf(fabsf(x0[j]), fabsf(x1[j])));
            const float s = vq8_scale(group_max<U>(amax));
            if (stores) {
                int8_t* codes = static_cast<int8_t*>(cache) + slot;
                store8_codes(codes + f0, x0, s);
                store8_codes(codes + f1, x1, s);
                if (u == 0) scales[crow] = s;
            }
        } else if (stores && p.kv_dtype == UAA_DTYPE_F32) {
            store8_f32(static_cast<float*>(cache) + slot + f0, x0, 1.f);
            store8_f32(static_cast<float*>(cache) + slot + f1, x1, 1.f);
        } else if (stores) {
            store8_bf16(static_cast<__nv_bfloat16*>(cache) + slot + f0, x0);
            store8_bf16(static_cast<__nv_bfloat16*>(cache) + slot + f1, x1);
        }
    }
    if (blockIdx.x == 0)  // nothing in this launch reads the lengths
        for (int i = tid; i < p.pk.batch; i += kRowThreads)
            if (p.pk.kv_ends[i] >= 0) p.seq_lens[i] = p.pk.kv_ends[i];
}

template <int D, typename T>
cudaError_t launch_rows(const AppendParams& p, const ScheduleParams& list, dim3 grid, cudaStream_t s)
{
    const bool q4 = p.kv_dtype == UAA_DTYPE_Q4;
    if (p.qk_norm)
        return q4 ? launch_dependent(append_rows_kernel<D, T, true, true>, grid, dim3(kRowThreads), 0, s, p, list)
                  : launch_dependent(append_rows_kernel<D, T, false, true>, grid, dim3(kRowThreads), 0, s, p, list);
    return q4 ? launch_dependent(append_rows_kernel<D, T, true, false>, grid, dim3(kRowThreads), 0, s, p, list)
              : launch_dependent(append_rows_kernel<D, T, false, false>, grid, dim3(kRowThreads), 0, s, p, list);
}

}  // namespace

// Tokens per CTA: eight where there are enough for every SM to have a few CTAs, fewer below
// (a step of a few tokens is latency-bound).
cudaError_t launch_append_packed(const AppendParams& p, const ScheduleParams* sched, int n_sm, cudaStream_t s)
{
    // runs of 8 elements pair up (and groups of 32 dims lie within neighbouring threads) only
    // for these; other partial rotations take a warp per row
    if (p.style == UAA_ROPE_NEOX && p.half_rot % (p.kv_dtype == UAA_DTYPE_Q4 ? 32 : 8) != 0)
        return launch_append_packed_rows(p, sched, n_sm, s);
    AppendParams q = p;
    int tps = kRowTokens;
    while (tps > 1 && p.pk.n_tokens / tps < 3 * n_sm) tps /= 2;
    q.tokens_per_cta = tps;
    const long long ctas = (p.pk.n_tokens + q.tokens_per_cta - 1) / q.tokens_per_cta + (sched ? 1 : 0);
    const ScheduleParams list = sched ? *sched : ScheduleParams{};
    const dim3 grid(static_cast<unsigned>(ctas));
    const bool f32 = p.io_dtype == UAA_DTYPE_F32;
    switch (p.D) {
    case 64: return f32 ? launch_rows<64, float>(q, list, grid, s) : launch_rows<64, __nv_bfloat16>(q, list, grid, s);
    case 128: return f32 ? launch_rows<128, float>(q, list, grid, s) : launch_rows<128, __nv_bfloat16>(q, list, grid, s);
    case 256: return f32 ? launch_rows<256, float>(q, list, grid, s) : launch_rows<256, __nv_bfloat16>(q, list, grid, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace uaa
