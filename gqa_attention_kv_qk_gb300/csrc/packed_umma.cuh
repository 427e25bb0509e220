// packed_umma.cuh -- attention of a packed batch over a bf16, vq8 or q8 cache (contiguous or
// paged, head_dim 64 or 128) on the 5th-generation tensor cores (tcgen05), single tokens and
// chunks of prompts in one launch.
//
// Work: the list of schedule.cuh, taken item by item from a counter by one CTA per SM. An
// item is a row pair (up to 2 x 128 (token, head) rows of one request and kv head) and a
// run of 128-key blocks. Two tiles of 128 rows are in flight, each with S, P and O in
// tensor memory and a warpgroup of its own (a thread per row: no exchange between
// threads), so that the tensor core multiplies for one while the other is in its softmax:
//   - more than 128 rows: the tiles are the pair's two halves; a key block serves both;
//   - up to 128 rows (decodes, drafts; every item of an 8-bit cache): both tiles hold the same
//     rows and take the key blocks in turn, and are merged at the end (both tiles' O are lanes
//     of the same threads, so only maxima and sums pass through shared memory).
// Step s of an item (tile s % 2):
//   S (128 x 128, fp32) = Q . K^T, Q rows in shared memory (K-major, 128-byte swizzle);
//   softmax: the running maximum m is raised only where a logit exceeds it by more than
//     2^8 (the final division cancels m); P = exp2(S - m) over S's columns as two bf16 parts,
//     and the row's sum of the weights before they are split;
//   O (128 x D, fp32) += P . V, P from tensor memory.
// The MMA lane issues S of step s + 2 right after P . V of step s (they share columns and
// run in order), while the other tile's softmax runs; an item's first S beside the epilogue of
// the item before.
//
// 8-bit caches: S of q8 is multiplied by the key's scale, P by the value's (in fp32, before it
// is rounded), and int8 codes are exact as bf16, so the MMAs are the same. The codes land in
// stages; the warps that bring q' widen them into the ring's tiles.
//
// Rounding: q' enters as bf16 hi + lo parts (2^-16 relative), two MMAs each, so that logits
// of any size keep their last bits. The weights (8-bit caches: times the value's scale) enter as
// bf16 hi + lo parts too (hi truncated, the rest rounded to nearest: 2^-15 relative), two MMAs
// each, as in the steps of equal lengths. One part, 2^-8 at most, would be the largest error of a
// bf16 output beside its own rounding (0.0020 to 0.0024 relative to 64 bits against 0.0017), for 843
// instead of 1,002 us for the two chunks below.
//
// What bounds it. Decodes: the cache's bytes (64 requests of up to 16,000 tokens, head_dim
// 128: 343 us, 6.2 TB/s). Long prompts: the chain of a tile's step, softmax -> P . V -> S (8,191
// tokens at once 660 us, 833 TFLOP/s; two chunks of 1,000 behind 20,000 to 32,000 cached 1,002
// us; q' and P in two parts make twice those operations in MMAs). In that chain instruction
// fetch weighed most: with the weights in a loop of 32 columns and mask and softcap in one of 16,
// against all 128 unrolled, chunks went from 881 to 842 us, a mixed batch from 332 to 304 and
// 8-bit drafts from 115 to 87 (the weights in one part then). Short items: their own latency.
//
// Warps (512 threads): 0 and 3 TMA (keys and values, through one ring in the order of their
// first use), 1 MMA issue and TMEM, 2 takes items from the
// list, 4-7 and 8-11 softmax and rows of the two tiles, 12-15 bring the next item's q'
// rows into shared memory and widen codes. setmaxnreg moves registers to the softmax warps:
// 64 x 128 x 2 + 192 x 128 x 2 = 65,536 = 512 threads x the 128 they were launched with.
// Every wait is bounded: one that gives up sets UAA_DEVFLAG_TIMEOUT and its warp leaves;
// the CTA still drains its copies and MMAs and frees its tensor memory.
#pragma once

#include <type_traits>

#include "schedule.cuh"

#include "ptx.cuh"

namespace uaa {
namespace {

constexpr int kPkThreads = 512;
constexpr int kPkItems = 4;       // slots for items that some warp has yet to read
constexpr int kPkClaim = 256;     // 256 at head_dim 64: four blocks left to load when the next item is claimed, 128: two
constexpr uint32_t kPkTmemCols = 512;  // S / P of tile x at 128 x, O at 256 + 128 x
constexpr long long kGraceCycles = 4000000;  // 2 ms
constexpr int kPkBf16 = 0, kPkVq8 = 1, kPkQ8 = 2;  // caches

// Shared memory: tiles of 128 rows. q' takes tiles 0 and 1 (hi, lo of tile 0's rows), and 2
// and 3 for a second tile of rows; keys and values a ring of the others, which at head_dim
// 128 has tiles 2 and 3 as well (slots 3 and 4) while an item has one tile of rows.
// 8-bit caches: items have one tile of rows (kPackedRows8). Codes land in stages of their own,
// with their scales behind them, and are widened into the ring's tiles; each ring slot has
// room for its block's scales.
template <int D, int KV>
struct PkShape {
    static constexpr bool kCodes = KV != kPkBf16;
    static constexpr int kTile = 128 * D * 2;
    static constexpr int kQTiles = kCodes ? 2 : 4;
    static constexpr int kTiles = kCodes ? (D == 128 ? 5 : 10) : D == 128 ? 7 : 12;
    static constexpr int kRing = kCodes ? kTiles - 2 : D == 128 ? 5 : 8;  // slots of an item of one tile of rows
    static constexpr int kRingTwo = kCodes ? kRing : D == 128 ? 3 : 8;    // and of two
    static constexpr int kStages = kCodes ? (D == 128 ? 3 : 6) : 0;
    static constexpr int kStage = 128 * D + 1024;               // codes, value scales, key scales
    // Warps that widen a tile: two at head_dim 64, which take tiles in turn with the other two, each
    // pair with half of the stages; all four at 128, where there is no room for four stages.
    static constexpr int kTeams = D == 64 ? 2 : 1, kWideners = 4 / kTeams;
    static constexpr int kTeamStages = kStages / kTeams;
    static_assert(kTeamStages * kTeams == kStages, "stages by team");
    static __device__ __forceinline__ int stage(int t)          // of the t-th tile of codes
    {
        return kCodes ? t % kTeams * kTeamStages + t / kTeams % kTeamStages : 0;
    }
    static constexpr int kScales = kCodes ? 1024 : 0;           // of a ring slot: value scales, key scales
    static constexpr int kOffStage = kTiles * kTile;
    static constexpr int kOffScales = kOffStage + kStages * kStage;
    static constexpr int kOffBar = kOffScales + kRing * kScales;  // 512 bytes
    static constexpr int kOffItems = kOffBar + 512;
    static constexpr int kOffMl = kOffItems + kPkItems * 64;    // (m, l) of tile 1: 128 float2
    static constexpr int kOffLast = kOffMl + 1024;              // per tile: this was a cut pair's last piece
    static constexpr int kSmemBytes = 1024 + kOffLast + 16;
    static_assert(kSmemBytes <= 232448, "shared memory of the packed kernel");
    static_assert(16 * kRing + 16 * kPkItems + 16 * kStages + 160 <= 512, "barrier area");
};

// An item as the warps see it.
struct PkItem {
    int flags;             // 1: an item (0: the list has ended), 2: the tiles are two halves of the rows
    int b, kvh;
    int r0, rows;          // the pair's first row and its rows
    int row0, L, blk0, n;  // first packed row of the request, tokens cached, first block, blocks
    int n_f, kb0, first;   // the pair's key runs (PairKeys)
    int lo, pieces, group, rec;
};
static_assert(sizeof(PkItem) == 64, "an item");

__device__ __forceinline__ uint32_t pk_pack(float lo, float hi)
{
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// The key and value ring as every warp counts it: loads go to slots in turn (of the item's
// ring); ph has each slot's parity of uses so far.
template <int D, int KV>
struct PkRing {
    using SH = PkShape<D, KV>;
    int at, size;
    uint32_t ph;

    __device__ __forceinline__ void begin(bool two)
    {
        size = two ? SH::kRingTwo : SH::kRing;
        if (SH::kRingTwo < SH::kRing && at >= size) at = 0;
    }
    __device__ __forceinline__ uint32_t parity() const { return ph >> at & 1u; }  // of the next load
    __device__ __forceinline__ int take()
    {
        const int s = at;
        ph ^= 1u << s;
        at = s + 1 == size ? 0 : s + 1;
        return s;
    }
    // slot and parity of the load k loads on
    __device__ __forceinline__ int slot(int k) const { return (at + k) % size; }
    __device__ __forceinline__ uint32_t parity(int k) const { return (ph >> slot(k) ^ static_cast<uint32_t>(k / size)) & 1u; }
    __device__ __forceinline__ void skip(int n)
    {
        const int whole = n / size, rest = n - whole * size;
        if (whole & 1) ph ^= (1u << size) - 1u;
        for (int k = 0; k < rest; ++k) take();
    }
    static __device__ __forceinline__ uint32_t tile(int slot)  // byte offset of a slot
    {
        return (SH::kRingTwo < SH::kRing && slot >= SH::kRingTwo ? slot - SH::kRingTwo + 2 : slot + SH::kQTiles) * SH::kTile;
    }
};

// An item's loads go in the order of first use: K0 V0 K1 V1 .., or K0 K1 V0 K2 V1 .. where the
// tiles take blocks in turn. The indexes of block j's keys and values among them (n blocks).
__device__ __forceinline__ int key_load(bool two, int j) { return two ? 2 * j : (j == 0 ? 0 : 2 * j - 1); }
__device__ __forceinline__ int value_load(bool two, int j, int n) { return two ? 2 * j + 1 : (j == n - 1 ? 2 * n - 1 : 2 * j + 2); }

// N columns of this thread's lane, N a multiple of 32.
template <int N>
__device__ __forceinline__ void ld_cols(uint32_t taddr, float (&v)[N])
{
#pragma unroll
    for (int c = 0; c < N; c += 32)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
            "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
            : "=f"(v[c + 0]), "=f"(v[c + 1]), "=f"(v[c + 2]), "=f"(v[c + 3]), "=f"(v[c + 4]), "=f"(v[c + 5]),
              "=f"(v[c + 6]), "=f"(v[c + 7]), "=f"(v[c + 8]), "=f"(v[c + 9]), "=f"(v[c + 10]), "=f"(v[c + 11]),
              "=f"(v[c + 12]), "=f"(v[c + 13]), "=f"(v[c + 14]), "=f"(v[c + 15]), "=f"(v[c + 16]),
              "=f"(v[c + 17]), "=f"(v[c + 18]), "=f"(v[c + 19]), "=f"(v[c + 20]), "=f"(v[c + 21]),
              "=f"(v[c + 22]), "=f"(v[c + 23]), "=f"(v[c + 24]), "=f"(v[c + 25]), "=f"(v[c + 26]),
              "=f"(v[c + 27]), "=f"(v[c + 28]), "=f"(v[c + 29]), "=f"(v[c + 30]), "=f"(v[c + 31])
            : "r"(taddr + c)
            : "memory");
    ptx::tmem_wait_ld();
}

// Parts of P of keys 16 k2 .. + 15: 32 keys' parts take those keys' columns of S.
__device__ __forceinline__ constexpr int p_col(int k2, int part) { return 32 * (k2 >> 1) + 8 * (k2 & 1) + 16 * part; }

template <int R>
__device__ __forceinline__ void set_max_regs_inc()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void set_max_regs_dec()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// The low n of 32 bits.
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// Whether a work list's entry lies within this batch, its cache and its workspace.
template <int ROWS>
__device__ __forceinline__ bool list_holds(const PackedUmmaParams& p, const PackedEntry& e)
{
    const int n = e.pieces >> 16, c = e.pieces & 0xffff;
    if (e.b < 0 || e.b >= p.B || e.T <= 0 || e.row0 < 0 || e.T > p.n_tokens - e.row0 || e.rp < 0) return false;
    if (e.rp >= (e.T * p.G + ROWS - 1) / ROWS || (e.end >= 0 && (e.end < e.T || e.end > p.cap)) || c >= n) return false;
    if (n <= 1) return true;
    const long long rows = static_cast<long long>(n) * p.Hkv * min(ROWS, e.T * p.G - e.rp * ROWS);
    return e.rec >= 0 && e.rec + rows <= p.max_rec_rows && e.group >= 0 && (e.group + 1LL) * 2 * p.Hkv <= p.max_counters;
}

// Half of S = Q . K^T (from k-step FROM on), both parts of q' on each chunk of K in turn
// (the tensor core takes a B chunk twice in a row faster than two different ones).
// Descriptors move by their address field alone.
template <int D, int FROM>
__device__ __forceinline__ void issue_qk(uint32_t lead, uint32_t t_s, uint64_t qd, uint64_t kd, uint32_t idesc)
{
#pragma unroll
    for (int kk = FROM; kk < FROM + D / 32; ++kk) {
        const uint32_t off = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4;
#pragma unroll
        for (int part = 0; part < 2; ++part)
            ptx::umma_bf16_lead(lead, t_s, qd + ((part * 128 * D * 2) >> 4) + off, kd + off, idesc, part | kk);
    }
}

// Half of O += P . V: keys 16 FROM .. + 63, both parts of P on each chunk of V.
template <int FROM>
__device__ __forceinline__ void issue_pv(uint32_t lead, uint32_t t_o, uint32_t t_p, uint64_t vd, uint32_t idesc, uint32_t more)
{
#pragma unroll
    for (int k2 = FROM; k2 < FROM + 4; ++k2)
#pragma unroll
        for (int part = 0; part < 2; ++part)
            ptx::umma_bf16_ts_lead(lead, t_o, t_p + p_col(k2, part), vd + ((k2 * 2048) >> 4), idesc,
                                   (part > 0 || k2 > FROM) ? 1u : more);
}

// Rows rr0 + quad, + 4, .. below rr0 + n of a cut pair from its pieces' records, the sink
// in the denominator: a warp takes RU rows at a time and PB pieces of each, a lane D / 32
// neighbouring dims, so that RU x PB loads are on their way together (one row and 8 pieces at a
// time kept a pair of 27 pieces for 200 us and more: the records are read at L2's latency).
template <int D, bool F32, int RU, int PB>
__device__ __forceinline__ void merge_rows(const PackedUmmaParams& p, const PkItem& it, int rr0, int n, int n_pieces, int quad, int lane)
{
    constexpr int E = D / 32;
    const size_t step = static_cast<size_t>(p.Hkv) * it.rows;  // rows between pieces
    for (int k0 = quad; k0 < n; k0 += 4 * RU) {
        size_t first[RU];
        float M[RU], z[RU], den[RU], acc[RU][E];
        int hq[RU], t[RU];
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            const int rr = rr0 + min(k0 + 4 * u, n - 1), R = it.r0 + rr;
            t[u] = R / p.G;
            hq[u] = it.kvh * p.G + (R - t[u] * p.G);
            first[u] = static_cast<size_t>(it.rec) + static_cast<size_t>(it.kvh) * it.rows + rr;
            z[u] = p.sink ? p.sink[hq[u]] * kLog2e : -INFINITY;
            M[u] = lane < n_pieces ? __ldcg(p.rec_lse + first[u] + lane * step) : -INFINITY;
            for (int c = lane + 32; c < n_pieces; c += 32) M[u] = fmaxf(M[u], __ldcg(p.rec_lse + first[u] + c * step));
        }
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            M[u] = fmaxf(warp_max(M[u]), z[u]);
            den[u] = z[u] == -INFINITY ? 0.f : ptx::ex2(z[u] - M[u]);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[u][e] = 0.f;
        }
        for (int c0 = 0; c0 < n_pieces; c0 += PB) {
            float v[RU][PB][E], w[RU][PB];
#pragma unroll
            for (int u = 0; u < RU; ++u)
#pragma unroll
                for (int c = 0; c < PB; ++c) {
                    const bool in = c0 + c < n_pieces;
                    const size_t at = first[u] + (in ? c0 + c : c0) * step;
                    w[u][c] = in ? __ldcg(p.rec_lse + at) : -INFINITY;
                    const float* from = p.rec_o + at * D + E * lane;
                    if constexpr (E == 4) {
                        const float4 a = __ldcg(reinterpret_cast<const float4*>(from));
                        v[u][c][0] = a.x, v[u][c][1] = a.y, v[u][c][2] = a.z, v[u][c][3] = a.w;
                    } else {
                        const float2 a = __ldcg(reinterpret_cast<const float2*>(from));
                        v[u][c][0] = a.x, v[u][c][1] = a.y;
                    }
                }
#pragma unroll
            for (int u = 0; u < RU; ++u)
#pragma unroll
                for (int c = 0; c < PB; ++c) {
                    const float f = w[u][c] == -INFINITY ? 0.f : ptx::ex2(w[u][c] - M[u]);
                    den[u] += f;
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[u][e] = f != 0.f ? fmaf(f, v[u][c][e], acc[u][e]) : acc[u][e];
                }
        }
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            if (k0 + 4 * u >= n) break;
            const float inv = den[u] > 0.f ? 1.f / den[u] : den[u] == 0.f ? 0.f : den[u];  // (a NaN stays one)
            const size_t to = (static_cast<size_t>(it.row0 + t[u]) * p.Hq + hq[u]) * D + E * lane;
            if (F32) {
#pragma unroll
                for (int e = 0; e < E; ++e) static_cast<float*>(p.out)[to + e] = acc[u][e] * inv;
            } else {
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + to + e) =
                        pk_pack(acc[u][e] * inv, acc[u][e + 1] * inv);
            }
        }
    }
}

// Four int8 codes as two words of bf16 pairs: 128 + the low seven bits, less 128 or, where the
// sign bit stands, 256 (0x4300 is 128 as bf16, 0x4380 is 256), each exact.
__device__ __forceinline__ void widen8(uint32_t codes, uint32_t& w0, uint32_t& w1)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t x = __byte_perm(codes, 0u, h ? 0x4342 : 0x4140);
        const uint32_t a = (x & 0x007f007fu) | 0x43004300u, b = (x & 0x00800080u) | 0x43004300u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
        (h ? w1 : w0) = *reinterpret_cast<const uint32_t*>(&d);
    }
}

// Sixteen codes of a row to its place in a swizzled tile of bf16 (group: of the row's sixteens).
__device__ __forceinline__ void store_widened(uint32_t tile, int row, int group, const uint4& c)
{
    const uint32_t at = tile + (group >> 2) * (kPackedKeys * 128) + row * 128, u = 2 * (group & 3);
    uint32_t o[8];
    widen8(c.x, o[0], o[1]);
    widen8(c.y, o[2], o[3]);
    widen8(c.z, o[4], o[5]);
    widen8(c.w, o[6], o[7]);
    ptx::st_shared_v4(at + ((u ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
    ptx::st_shared_v4(at + (((u + 1) ^ (row & 7)) << 4), o[4], o[5], o[6], o[7]);
}

// (not inlined: the softmax's registers need not make room for it)
template <int D, bool F32>
__device__ __noinline__ void merge_pieces(const PackedUmmaParams& p, const PkItem& it, int rr0, int n, int n_pieces, int quad, int lane)
{
    if (n <= 4) merge_rows<D, F32, 1, 16>(p, it, rr0, n, n_pieces, quad, lane);
    else merge_rows<D, F32, 4, 4>(p, it, rr0, n, n_pieces, quad, lane);
}

// F32: fp32 outputs
template <int D, int KV, bool F32>
__global__ void __launch_bounds__(kPkThreads, 1)
packed_umma_kernel(const __grid_constant__ PackedMaps tm, const PackedUmmaParams p)
{
    using SH = PkShape<D, KV>;
    constexpr bool kCodes = SH::kCodes, kKeyCodes = KV == kPkQ8;
    constexpr int kRows = kCodes ? kPackedRows8 : kPackedRows;  // of an item at most
    constexpr int NR = SH::kRing;
    constexpr uint32_t kIdS = ptx::umma_idesc_bf16(128, kPackedKeys, false, false);
    constexpr uint32_t kIdO = ptx::umma_idesc_bf16(128, D, false, true);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw);
    const uint32_t qsm = base, bars = base + SH::kOffBar;
    const uint32_t bar_full = bars, bar_empty = bars + 8 * NR;
    const uint32_t bar_ifull = bars + 16 * NR, bar_iempty = bar_ifull + 8 * kPkItems;
    const uint32_t bar_qfull = bar_iempty + 8 * kPkItems, bar_qfree = bar_qfull + 8;
    const uint32_t bar_s = bar_qfree + 8;       // [2] S of a tile's step (MMA commit)
    const uint32_t bar_p = bar_s + 16;          // [2] P of it (a lane per warp)
    const uint32_t bar_o = bar_p + 16;          // [2] the item's O of a tile (MMA commit)
    const uint32_t bar_ofree = bar_o + 16;      // O of both tiles read (8 arrivals)
    const uint32_t bar_ml = bar_ofree + 8;      // tile 1's maxima and sums, for the merge (a lane per warp)
    const uint32_t bar_mlfree = bar_ml + 8;     // and that they were read
    const uint32_t bar_rec = bar_mlfree + 8;    // [2] a cut pair's records written (a lane per warp)
    const uint32_t bar_last = bar_rec + 16;     // [2] whether they were the last
    const uint32_t bar_idone = bar_last + 16;   // an item's last P . V (MMA commit)
    const uint32_t bar_qtwo = bar_idone + 8;    // as bar_qfree, for items of two tiles of rows
    const uint32_t bar_claim = bar_qtwo + 8;    // an item's loads are nearly all issued: the next may be taken
    const uint32_t bar_drain = bar_claim + 8;
    const uint32_t bar_sfull = bar_drain + 8;   // [stages] codes have landed
    const uint32_t bar_sempty = bar_sfull + 8 * SH::kStages;  // and were read (a lane per widening warp)
    const uint32_t tmem_slot = bar_sempty + 8 * SH::kStages;
    const uint32_t failed = base + SH::kOffLast + 12;  // a wait gave up
    const uint32_t q_count = base + SH::kOffLast + 8;  // items of two tiles whose S MMAs are done (the TMA warps')
    volatile PkItem* items = reinterpret_cast<volatile PkItem*>(base_ptr + SH::kOffItems);
    float2* ml = reinterpret_cast<float2*>(base_ptr + SH::kOffMl);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NR; ++s) {
            ptx::mbar_init(bar_full + 8 * s, kCodes ? 4 : 1);  // (by the widening warps, or a TMA lane for all)
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        for (int s = 0; s < kPkItems; ++s) {
            ptx::mbar_init(bar_ifull + 8 * s, 1);
            ptx::mbar_init(bar_iempty + 8 * s, 15);  // 2 TMA, MMA, 8 softmax warps, 4 q' warps
        }
        ptx::mbar_init(bar_qfull, 4);
        ptx::mbar_init(bar_qfree, 1);
        for (int x = 0; x < 2; ++x) {
            ptx::mbar_init(bar_s + 8 * x, 1);
            ptx::mbar_init(bar_p + 8 * x, 4);
            ptx::mbar_init(bar_o + 8 * x, 1);
        }
        for (int x = 0; x < 2; ++x) {
            ptx::mbar_init(bar_rec + 8 * x, 4);
            ptx::mbar_init(bar_last + 8 * x, 1);
        }
        ptx::mbar_init(bar_ofree, 8);
        ptx::mbar_init(bar_ml, 4);
        ptx::mbar_init(bar_mlfree, 4);
        ptx::mbar_init(bar_idone, 1);
        ptx::mbar_init(bar_qtwo, 1);
        ptx::mbar_init(bar_claim, 1);
        ptx::flag_set(q_count, 0u);
        ptx::flag_set(failed, 0u);
        ptx::mbar_init(bar_drain, 1);
        for (int s = 0; s < SH::kStages; ++s) {
            ptx::mbar_init(bar_sfull + 8 * s, 1);
            ptx::mbar_init(bar_sempty + 8 * s, SH::kWideners);
        }
        ptx::fence_barrier_init();
        ptx::prefetch_tensormap(&tm.k);
        ptx::prefetch_tensormap(&tm.v);
    }
    if (warp == 1) {
        ptx::tmem_alloc(tmem_slot, kPkTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    grid_dependency_wait();  // the append's rows, q' and the work list are complete
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(base_ptr + SH::kOffBar + (tmem_slot - bars));

    auto give_up = [&]() {
        atomicOr(p.status, UAA_DEVFLAG_TIMEOUT);
        ptx::flag_set(failed, 1u);
    };
    // the i-th item, as every warp takes it (false: a wait gave up)
    auto take_item = [&](int i, PkItem& it) {
        const int slot = i % kPkItems;
        if (!ptx::mbar_wait(bar_ifull + 8 * slot, (i / kPkItems) & 1, kWaitLimitCycles)) return false;
        const volatile int* from = reinterpret_cast<const volatile int*>(items + slot);
        int* to = reinterpret_cast<int*>(&it);
#pragma unroll
        for (int k = 0; k < 16; ++k) to[k] = from[k];
        return true;
    };
    auto drop_item = [&](int i) {  // this warp (or lane) has read the item
        ptx::mbar_arrive(bar_iempty + 8 * (i % kPkItems));
    };

    if (warp < 4) {
        set_max_regs_dec<64>();
        if (warp == 0 || warp == 3) {
            // ------------------------------------------------------------ TMA
            // Warp 0 loads the keys, warp 3 the values; both count every load through the ring. A
            // lane per page of a block looks its entry up a block ahead. Codes go to the stages in
            // turn, from one warp: warp 3 where values alone are codes, warp 0 (both) where keys are too.
            const bool is_v = warp == 3;
            const bool paged = p.pages.table != nullptr;
            const int box = paged ? min(1 << p.pages.shift, kPackedKeys) : kPackedKeys;
            const int n_sub = kPackedKeys / box;
            const uint64_t once = ptx::l2_evict_first_policy();
            PkRing<D, KV> ring{};
            uint32_t used = 0, last = 0;  // slots that held a copy, and the parity of each one's last
            int coded = 0;               // tiles of codes so far
            uint32_t stage_ph = 0, staged = 0;  // parity of each stage's uses so far; stages used
            // one block's codes (of keys, or of values with the block's scales) into the next stage
            auto load_codes = [&](bool keys, bool mine, long long row, uint32_t n) {
                const int s = SH::stage(coded++);
                const uint32_t par = stage_ph >> s & 1u, bar = bar_sfull + 8 * s;
                bool there = true;
                if (lane == 0) there = ptx::mbar_wait(bar_sempty + 8 * s, par ^ 1u, kWaitLimitCycles);
                if (!__shfl_sync(0xffffffffu, there, 0)) return false;
                stage_ph ^= 1u << s;
                staged |= 1u << s;
                const int bytes = box * (keys ? D : D + (kKeyCodes ? 8 : 4));
                if (lane == 0) ptx::mbar_arrive_expect_tx(bar, n * bytes);
                __syncwarp();
                if (mine) {
                    const uint32_t st = base + SH::kOffStage + s * SH::kStage;
                    const int y = row < 0 ? -box : static_cast<int>(row);  // an entry that is no page reads as zeros
                    ptx::tma_load_2d_hint(st + lane * box * D, keys ? &tm.k : &tm.v, 0, y, bar, once);
                    if (!keys) {
                        // the scales lie by page (or sequence) and kv head
                        const int per = paged ? 1 << p.pages.shift : p.cap;
                        const int sy = row < 0 ? -1 : static_cast<int>(row / per), sx = row < 0 ? 0 : static_cast<int>(row % per);
                        ptx::tma_load_2d_hint(st + 128 * D + lane * box * 4, &tm.vs, sx, sy, bar, once);
                        if (kKeyCodes) ptx::tma_load_2d_hint(st + 128 * D + 512 + lane * box * 4, &tm.ks, sx, sy, bar, once);
                    }
                }
                return true;
            };
            auto count_load = [&]() {
                const uint32_t par = ring.parity();
                const int s = ring.take();
                used |= 1u << s;
                last = (last & ~(1u << s)) | par << s;
                return s;
            };
            int twos = 0;                // earlier items of two tiles of rows
            bool q_there = false;        // the last one's q' rows may still lie where slots kRingTwo .. are
            bool ok = true;
            for (int i = 0; ok; ++i) {
                PkItem it;
                ok = take_item(i, it);
                if (ok) {
                    __syncwarp();
                    if (lane == 0) drop_item(i);
                }
                if (!ok || !(it.flags & 1)) break;
                const bool two = !kCodes && (it.flags & 2);
                const int hi = it.L + (it.r0 + it.rows - 1) / p.G + 1;
                // the next item is claimed late, so that the CTAs that are done first take what is left,
                // and early enough for its loads to follow this one's (by the keys' warp)
                const int claim_at = max(0, it.n - kPkClaim / D);
                if (it.n == 0) {
                    if (!is_v && lane == 0) ptx::mbar_arrive(bar_claim);
                    continue;
                }
                if (kKeyCodes && is_v) continue;  // (warp 0 loads both)
                ring.begin(two);
                // this lane's page of block j, where any of its keys is visible: its table entry, looked
                // up a block ahead (nothing waits for it before it is used)
                auto key_of = [&](int j, bool& mine) {
                    const int blk = it.blk0 + j;
                    const bool in_first = blk < it.n_f;
                    const int key0 = (in_first ? blk : it.kb0 + blk - it.n_f) * kPackedKeys;
                    const int run_lo = in_first ? 0 : it.lo, run_hi = in_first ? it.first : hi;
                    const int ku = key0 + lane * box;
                    mine = j < it.n && lane < n_sub && ku < run_hi && ku + box > run_lo;
                    return ku;
                };
                const int* const entries = p.pages.table + static_cast<size_t>(it.b) * p.pages.per_seq;
                bool mine_next;
                int key_next = key_of(0, mine_next), entry_next = 0;
                if (paged && mine_next) entry_next = __ldg(entries + (key_next >> p.pages.shift));
                bool mine_last = false;  // (of the block before)
                long long row_last = 0;
                uint32_t n_last = 0;
                int k = 0;  // loads of the item so far, in the order of first use
                for (int j = 0; j < it.n; ++j) {
                    const bool mine = mine_next;
                    const int key = key_next, entry = entry_next;
                    if (j + 1 < it.n) {
                        key_next = key_of(j + 1, mine_next);
                        if (paged && mine_next) entry_next = __ldg(entries + (key_next >> p.pages.shift));
                    }
                    // its first cache row, or -1 where the entry is no page
                    long long row = (static_cast<long long>(it.b) * p.Hkv + it.kvh) * p.cap + key;
                    if (paged)
                        row = entry < 0 || entry >= p.pages.n_pages
                                  ? -1
                                  : (((static_cast<long long>(entry) * p.Hkv + it.kvh) << p.pages.shift) | (key & ((1 << p.pages.shift) - 1)));
                    if (mine && row < 0) atomicOr(p.status, UAA_DEVFLAG_PAGE);
                    if (!is_v && lane == 0 && j == claim_at) ptx::mbar_arrive(bar_claim);
                    // The q' rows of an item of two tiles lie where slots kRingTwo .. are until its S
                    // MMAs are done. The keys' warp waits for that once for each such item, before a
                    // following one of one tile loads anything, or one of two its last block (a wait
                    // tells a phase of a barrier from the one before it, not from one two phases on),
                    // and counts them for the values' warp.
                    if (kCodes && (kKeyCodes || is_v)) {
                        const uint32_t n_in = __popc(__ballot_sync(0xffffffffu, mine));
                        if (!kKeyCodes) {
                            ok = load_codes(false, mine, row, n_in);
                        } else {  // K0, K1 V0, K2 V1, ..
                            if (j > 0) ok = load_codes(true, mine, row, n_in) && load_codes(false, mine_last, row_last, n_last);
                            else ok = load_codes(true, mine, row, n_in);
                            if (ok && j == it.n - 1) ok = load_codes(false, mine, row, n_in);
                            mine_last = mine, row_last = row, n_last = n_in;
                        }
                        if (!ok) break;
                        continue;
                    }
                    if (q_there && (is_v ? !two : j == (two ? it.n - 1 : 0))) {
                        if (is_v) {
                            const long long since = clock64();
                            while (static_cast<int>(ptx::flag_get(q_count)) < twos && (ok = clock64() - since < kWaitLimitCycles))
                                __nanosleep(64);
                        } else {
                            ok = ptx::mbar_wait(bar_qtwo, (twos - 1) & 1, kWaitLimitCycles);
                        }
                        __threadfence_block();
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        if (!is_v && lane == 0) ptx::flag_set(q_count, static_cast<uint32_t>(twos));
                        q_there = false;
                    }
                    const int at = is_v ? value_load(two, j, it.n) : key_load(two, j);
                    for (; k < at; ++k) count_load();  // the other warp's
                    const uint32_t par = ring.parity();
                    const int s = count_load();
                    ++k;
                    if (lane == 0) ok = ptx::mbar_wait(bar_empty + 8 * s, par ^ 1u, kWaitLimitCycles);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    const uint32_t bar = bar_full + 8 * s;
                    const int n = __popc(__ballot_sync(0xffffffffu, mine));
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(bar, n * box * D * 2);
                        if (kCodes) ptx::mbar_arrive_n(bar, 3);
                    }
                    __syncwarp();
                    if (mine) {
                        const uint32_t st = base + PkRing<D, KV>::tile(s) + lane * box * 128;
                        const int y = row < 0 ? -box : static_cast<int>(row);  // an entry that is no page reads as zeros
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) {
                            if (two)  // other row pairs read the same tiles from L2
                                ptx::tma_load_2d(st + c * (kPackedKeys * 128), is_v ? &tm.v : &tm.k, c * 64, y, bar);
                            else
                                ptx::tma_load_2d_hint(st + c * (kPackedKeys * 128), is_v ? &tm.v : &tm.k, c * 64, y, bar, once);
                        }
                    }
                }
                if (!ok) break;
                if (!kCodes || (!kKeyCodes && !is_v))
                    for (; k < 2 * it.n; ++k) count_load();
                if (two) {
                    q_there = true;
                    ++twos;
                }
            }
            if (!ok && lane == 0) give_up();
            // every issued copy lands before the CTA may exit: each slot's (and stage's) last one
            if (!is_v && !kKeyCodes && lane == 0)
                for (int s = 0; s < NR; ++s)
                    if ((used >> s & 1u) && !ptx::mbar_wait(bar_full + 8 * s, last >> s & 1u, kWaitLimitCycles)) {
                        give_up();
                        break;
                    }
            if (lane == 0)
                for (int s = 0; s < SH::kStages; ++s)
                    if ((staged >> s & 1u) && !ptx::mbar_wait(bar_sfull + 8 * s, (stage_ph >> s & 1u) ^ 1u, kWaitLimitCycles)) {
                        give_up();
                        break;
                    }
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issue
            // The warp stays converged and one lane issues (umma_bf16_lead). A step's key and
            // value tiles are waited for before its P, so that nothing stands between the
            // softmax's end and the next MMAs.
            const uint32_t lead = ptx::elect_one();
            bool ok = true;
            PkRing<D, KV> ring{};
            int busy = 0;                // earlier items with steps
            int steps0 = 0, steps1 = 0;  // earlier steps of each tile
            for (int i = 0; ok; ++i) {
                PkItem it;
                ok = __all_sync(0xffffffffu, take_item(i, it));
                if (!ok) break;
                if (lane == 0) drop_item(i);
                if (!(it.flags & 1)) break;
                const int n = __shfl_sync(0xffffffffu, it.n, 0);
                if (n == 0) continue;
                const bool two = !kCodes && (__shfl_sync(0xffffffffu, it.flags, 0) & 2);
                const int n_steps = two ? 2 * n : n;
                ring.begin(two);
                auto free_tile = [&](int slot) { ptx::umma_commit_lead(lead, bar_empty + 8 * slot); };
                ok = ptx::mbar_wait(bar_qfull, busy & 1, kWaitLimitCycles);
                int ks = 0, vs = 0;   // slots of the step's key and value tile
                bool v_here = false;  // the next value tile was seen to have landed
                uint32_t v_par = 0;
                uint64_t vd = 0;
                // (after a failed wait the item's other MMAs are issued without waiting: results mean
                // nothing by then, and every place they touch is this CTA's)
                auto step = [&](int s, auto X) {
                    constexpr int x = decltype(X)::value;
                    const bool has_pv = s >= 2 && s - 2 < n_steps, has_s = s < n_steps;  // P . V of step s - 2, then S of step s
                    const bool fresh = !two || x == 0, done = !two || x == 1;  // the tiles' first, last use
                    // A step's tiles are looked for between MMAs, where the tensor core has work
                    // meanwhile, and waited for only when they are needed (a tile may need a slot
                    // that the MMAs between free).
                    bool k_here = !fresh;
                    uint32_t k_par = 0;
                    uint64_t kd = 0;
                    auto look_for_k = [&]() {
                        if (fresh && has_s) {
                            k_par = ring.parity();
                            ks = ring.take();
                            k_here = ptx::mbar_try_wait(bar_full + 8 * ks, k_par);
                        }
                        kd = ptx::umma_desc(base + PkRing<D, KV>::tile(ks), 16, 1024);
                    };
                    if (has_pv) {
                        // O of the item before has been read (its first S MMAs run beside that)
                        if (s == 2 && busy > 0) ok = ok && ptx::mbar_wait(bar_ofree, (busy - 1) & 1, kWaitLimitCycles);
                        ok = ok && ptx::mbar_wait(bar_p + 8 * x, ((x ? steps1 : steps0) + ((s - 2) >> 1)) & 1, kWaitLimitCycles);
                        if (fresh && !v_here) ok = ok && ptx::mbar_wait(bar_full + 8 * vs, v_par, kWaitLimitCycles);
                        __syncwarp();
                        ptx::tc_fence_after();
                        issue_pv<0>(lead, tmem + 256 + 128 * x, tmem + 128 * x, vd, kIdO, s >= 4);  // (4: O has a step's sum)
                        look_for_k();
                        issue_pv<4>(lead, tmem + 256 + 128 * x, tmem + 128 * x, vd, kIdO, 1u);
                        if (done) free_tile(vs);
                        if (s >= n_steps) ptx::umma_commit_lead(lead, bar_o + 8 * x);
                        if (s == n_steps + 1) ptx::umma_commit_lead(lead, bar_idone);
                    } else {
                        look_for_k();
                    }
                    // the next step's value tile, before the last S MMAs
                    auto next_v = [&]() {
                        if (done && s >= 1 && s - 1 < n_steps) {
                            v_par = ring.parity();
                            vs = ring.take();
                            v_here = ptx::mbar_try_wait(bar_full + 8 * vs, v_par);
                            vd = ptx::umma_desc(base + PkRing<D, KV>::tile(vs), kPackedKeys * 128, 1024);
                        }
                    };
                    if (has_s) {
                        if (!k_here) ok = ok && ptx::mbar_wait(bar_full + 8 * ks, k_par, kWaitLimitCycles);
                        __syncwarp();
                        ptx::tc_fence_after();
                        const uint64_t qd = ptx::umma_desc(qsm + (two ? 2 * x : 0) * SH::kTile, 16, 1024);
                        const int k_slot = ks;
                        issue_qk<D, 0>(lead, tmem + 128 * x, qd, kd, kIdS);
                        next_v();
                        issue_qk<D, D / 32>(lead, tmem + 128 * x, qd, kd, kIdS);
                        ptx::umma_commit_lead(lead, bar_s + 8 * x);
                        if (done) free_tile(k_slot);
                        if (s == n_steps - 1) {  // the q' rows may be replaced
                            ptx::umma_commit_lead(lead, bar_qfree);
                            if (two) ptx::umma_commit_lead(lead, bar_qtwo);
                        }
                    } else {
                        next_v();
                    }
                };
                for (int s = 0; s < n_steps + 2; s += 2) {
                    step(s, std::integral_constant<int, 0>{});
                    if (s + 1 < n_steps + 2) step(s + 1, std::integral_constant<int, 1>{});
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                steps0 += two ? n : (n + 1) / 2;
                steps1 += two ? n : n / 2;
                ++busy;
            }
            if (!ok && lane == 0) give_up();
            // every MMA issued has completed before TMEM is freed
            __syncwarp();
            ptx::umma_commit_lead(lead, bar_drain);
            if (!ptx::mbar_wait(bar_drain, 0, kWaitLimitCycles)) give_up();
        } else if (warp == 2) {
            // ------------------------------------------------------------ items
            if (lane == 0) {
                const unsigned n_items = min(*p.entries_n, static_cast<unsigned>(p.max_entries)) * static_cast<unsigned>(p.Hkv);
                for (int i = 0;; ++i) {
                    const int slot = i % kPkItems;
                    bool ok = i == 0 || ptx::mbar_wait(bar_claim, (i - 1) & 1, kWaitLimitCycles);
                    if (ok && i >= kPkItems) ok = ptx::mbar_wait(bar_iempty + 8 * slot, ((i / kPkItems) - 1) & 1, kWaitLimitCycles);
                    if (!ok) {
                        give_up();
                        break;
                    }
                    const unsigned w = i == 0 ? blockIdx.x : atomicAdd(p.next, 1u);
                    PkItem it{};
                    if (w < n_items) {
                        const PackedEntry e = p.entries[w / p.Hkv];
                        it.kvh = static_cast<int>(w % p.Hkv);
                        it.flags = 1;
                        it.pieces = 1 << 16;
                        // (an entry of another batch's list, or of none, names nothing outside this one's)
                        if (list_holds<kRows>(p, e)) {
                            it.r0 = e.rp * kRows;
                            it.rows = min(kRows, e.T * p.G - it.r0);
                            it.flags = !kCodes && it.rows > 128 ? 3 : 1;
                            it.b = e.b;
                            it.row0 = e.row0;
                            it.L = e.end - e.T;
                            it.pieces = e.pieces;
                            it.rec = e.rec;
                            it.group = e.group;
                            if (e.end >= 0) {
                                const PairKeys k = pair_keys(it.r0, it.rows, p.G, it.L, p.window, p.first_tokens);
                                const int n = e.pieces >> 16, c = e.pieces & 0xffff;
                                it.blk0 = static_cast<int>(static_cast<long long>(k.n_blocks) * c / n);
                                it.n = static_cast<int>(static_cast<long long>(k.n_blocks) * (c + 1) / n) - it.blk0;
                                it.n_f = k.n_f;
                                it.kb0 = k.kb0;
                                it.first = k.first;
                                it.lo = k.lo;
                            }
                        }
                    }
                    const int* from = reinterpret_cast<const int*>(&it);
                    volatile int* to = reinterpret_cast<volatile int*>(items + slot);
#pragma unroll
                    for (int k = 0; k < 16; ++k) to[k] = from[k];
                    ptx::mbar_arrive(bar_ifull + 8 * slot);
                    if (w >= n_items) {
                        // the last CTA to come here starts the list over, for another attention by it
                        if (atomicAdd(p.next + 2, 1u) == gridDim.x - 1) {
                            p.next[0] = gridDim.x;
                            p.next[2] = 0u;
                        }
                        break;
                    }
                }
            }
        }
    } else if (warp < 12) {
        set_max_regs_inc<192>();
        // ---------------------------------------------------------------- softmax and rows of tile x
        const int x = (warp - 4) >> 2, quad = warp & 3;
        const int r = 32 * quad + lane;  // this thread's row of the tile, and TMEM lane
        const uint32_t lane_addr = static_cast<uint32_t>(32 * quad) << 16;
        const uint32_t t_s = tmem + lane_addr + 128 * x;
        bool ok = true;
        PkRing<D, KV> ring{};
        int steps = 0;                       // earlier steps of this tile
        int items_with[2] = {0, 0};          // earlier items with steps of each tile
        int merges = 0, cuts = 0;            // earlier items of up to 128 rows; pieces of cut pairs (of this tile)
        for (int i = 0; ok; ++i) {
            PkItem it;
            ok = take_item(i, it);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) drop_item(i);
            if (!(it.flags & 1)) break;
            const bool two = !kCodes && (it.flags & 2);
            const int rr = (two ? 128 * x : 0) + r;  // row of the pair
            const int R = it.r0 + rr;                // row of the request's kv head
            const bool row_ok = rr < it.rows;
            const int warp_row = (two ? 128 * x : 0) + 32 * quad;  // the warp's first row of the pair
            const bool warp_ok = warp_row < it.rows;
            const int tok = R / p.G;
            const int kmax = it.L + tok;
            const int kmin = p.window > 0 ? kmax - p.window + 1 : INT_MIN;
            const int hi = it.L + (it.r0 + it.rows - 1) / p.G + 1;  // the pair's last visible key + 1
            // keys that every row of the warp sees: up to its first row's position, from its last row's window on
            const int all_hi = it.L + (it.r0 + warp_row) / p.G;
            const int all_lo = p.window > 0 ? it.L + (it.r0 + min(warp_row + 31, it.rows - 1)) / p.G - p.window + 1 : INT_MIN;
            const int n_mine = two ? it.n : (it.n + 1 - x) / 2;
            if (it.n > 0) ring.begin(two);
            const float sink_z = p.sink && (it.pieces >> 16) == 1 && row_ok ? p.sink[it.kvh * p.G + (R - tok * p.G)] * kLog2e : -INFINITY;
            float m = -INFINITY, l = 0.f;
            for (int c = 0; c < n_mine && ok; ++c) {
                const int j = two ? c : 2 * c + x;
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_s + 8 * x, (steps + c) & 1, kWaitLimitCycles));
                if (!ok) break;
                ptx::tc_fence_after();
                const int blk = it.blk0 + j;
                const bool in_first = blk < it.n_f;
                const int key0 = (in_first ? blk : it.kb0 + blk - it.n_f) * kPackedKeys;
                // value rows that no row of the pair sees (unused slots, absent pages, what lies
                // behind the window) may hold anything, NaN included: zero them once they have
                // landed, as P is 0 there (tile 0's warps where both tiles use the block)
                const int keep = (in_first ? it.first : hi) - key0, skip = in_first ? 0 : it.lo - key0;
                if (!kCodes && (keep < kPackedKeys || skip > 0) && (!two || x == 0)) {
                    const int vl = value_load(two, j, it.n);
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_full + 8 * ring.slot(vl), ring.parity(vl), kWaitLimitCycles));
                    if (!ok) break;
                    const uint32_t vt = base + PkRing<D, KV>::tile(ring.slot(vl));
                    const int head = max(skip, 0), tail = min(keep, kPackedKeys);
                    const int n_chunks = (head + kPackedKeys - tail) * (D / 8);
                    for (int q = 32 * quad + lane; q < n_chunks; q += 128) {
                        const int z = q / (D / 8), ch = q % (D / 8);
                        const int row = z < head ? z : tail + z - head;
                        ptx::st_shared_v4(vt + (ch >> 3) * (kPackedKeys * 128) + row * 128 + (ch & 7) * 16, 0u, 0u, 0u, 0u);
                    }
                    ptx::fence_proxy_async();  // visible to the tensor core
                }
                // (8-bit: the widening warps have zeroed them, and the scales are there with the values)
                uint32_t sc_at = 0;
                if (kCodes) {
                    const int vl = value_load(false, j, it.n);
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_full + 8 * ring.slot(vl), ring.parity(vl), kWaitLimitCycles));
                    if (!ok) break;
                    sc_at = base + SH::kOffScales + ring.slot(vl) * SH::kScales;
                }
                // The columns are read twice, for the maximum at once and for the weights in a loop of
                // 32: with all 128 kept in registers and the weights unrolled, the warps spent more time
                // waiting for instructions than on anything else (ten warps at work at once, spread over
                // more code than the nearest cache holds).
                if (warp_ok) {
                    // (a missing row's values mean nothing: it asks for no mask and no maximum)
                    const bool masked = !(key0 + kPackedKeys - 1 <= all_hi && (in_first ? key0 + kPackedKeys <= it.first : key0 >= all_lo));
                    // keys below i_f are among the first tokens: visible in their own blocks, or
                    // where there is one run (not in the window's first block, which may hold
                    // them once more)
                    const int i_f = in_first || it.n_f == 0 ? p.first_tokens - key0 : 0;
                    const int i_lo = p.window > 0 ? (in_first ? 128 : kmin - key0) : 0;
                    const int i_hi = kmax - key0;
                    // Mask and softcap in a loop of 16 of their own, written back, so that the loops
                    // below are the same few instructions for every block: inline and unrolled, the mask
                    // of a decode's last block alone took 4 us, most of it instruction fetch.
                    const bool pre = masked || p.softcap_log2e > 0.f;
                    if (pre) {
#pragma unroll 1
                        for (int h = 0; h < 128; h += 16) {
                            uint32_t o[16];
                            ptx::tmem_ld16(t_s + h, o);
                            ptx::tmem_wait_ld();
                            const uint32_t seen = masked ? bits_below(i_hi + 1 - h) & (~bits_below(i_lo - h) | bits_below(i_f - h)) : ~0u;
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                float x = __uint_as_float(o[k]);
                                if (kKeyCodes) x *= ptx::ld_shared_f32(sc_at + 512 + 4 * (h + k));
                                if (p.softcap_log2e > 0.f) x = tanhf(x) * p.softcap_log2e;
                                o[k] = seen >> k & 1u ? __float_as_uint(x) : 0xff800000u;  // -inf
                            }
                            ptx::tmem_st16(t_s + h, o);
                        }
                        ptx::tmem_wait_st();
                    }
                    float mx;
                    {
                        float v[128];
                        ld_cols(t_s, v);
                        if (kKeyCodes && !pre) {  // S is in units of the keys' scales
#pragma unroll
                            for (int k = 0; k < 128; k += 4) {
                                const float4 c4 = ptx::ld_shared_f4(sc_at + 512 + 4 * k);
                                v[k] *= c4.x, v[k + 1] *= c4.y, v[k + 2] *= c4.z, v[k + 3] *= c4.w;
                            }
#pragma unroll
                            for (int c0 = 0; c0 < 128; c0 += 16) {
                                uint32_t o[16];
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(v[c0 + k]);
                                ptx::tmem_st16(t_s + c0, o);
                            }
                            ptx::tmem_wait_st();
                        }
                        float t[8];
#pragma unroll
                        for (int a = 0; a < 8; ++a) t[a] = fmaxf(v[a], v[a + 8]);
#pragma unroll
                        for (int a = 16; a < 128; a += 16)
#pragma unroll
                            for (int e = 0; e < 8; ++e) t[e] = ptx::max3(t[e], v[a + e], v[a + 8 + e]);
                        mx = fmaxf(ptx::max3(ptx::max3(t[0], t[1], t[2]), t[3], t[4]), ptx::max3(t[5], t[6], t[7]));
                    }
                    const bool raise = row_ok && mx > m + 8.f;
                    if (__any_sync(0xffffffffu, raise)) {
                        const float f = raise ? ptx::ex2(m - mx) : 1.f;  // 0 while m = -inf
                        if (c > 0 && __any_sync(0xffffffffu, raise && m != -INFINITY)) {
                            // (S of this step follows P . V of the one before: O is complete so far)
#pragma unroll 1
                            for (int d = 0; d < D; d += 16) {
                                uint32_t o[16];
                                ptx::tmem_ld16(tmem + lane_addr + 256 + 128 * x + d, o);
                                ptx::tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                                ptx::tmem_st16(tmem + lane_addr + 256 + 128 * x + d, o);
                            }
                        }
                        if (raise) {
                            l *= f;
                            m = mx;
                        }
                    }
                    const float mu = m == -INFINITY ? 0.f : m;
                    const float2 nmu = make_float2(-mu, -mu);
                    float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll 1
                    for (int h = 0; h < 128; h += 32) {
                        float v[32];
                        ld_cols(t_s + h, v);
                        uint32_t hh[16], lo16[16];
                        float4 vs4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float2 a = ptx::add_f32x2(make_float2(v[2 * k], v[2 * k + 1]), nmu);
                            float e0 = ptx::ex2(a.x), e1 = ptx::ex2(a.y);
                            const float2 e = make_float2(e0, e1);
                            if (kCodes) {  // the codes' weight: the value's times its scale
                                if (!(k & 1)) vs4 = ptx::ld_shared_f4(sc_at + 4 * (h + 2 * k));
                                e0 *= k & 1 ? vs4.z : vs4.x;
                                e1 *= k & 1 ? vs4.w : vs4.y;
                            }
                            const uint32_t b0 = __float_as_uint(e0) & 0xffff0000u, b1 = __float_as_uint(e1) & 0xffff0000u;
                            hh[k] = __byte_perm(b0, b1, 0x7632);
                            const float2 rest = ptx::add_f32x2(make_float2(e0, e1), make_float2(-__uint_as_float(b0), -__uint_as_float(b1)));
                            lo16[k] = pk_pack(rest.x, rest.y);
                            if (k & 1) s1 = ptx::add_f32x2(s1, e);
                            else s0 = ptx::add_f32x2(s0, e);
                        }
                        ptx::tmem_st16(t_s + h, hh);
                        ptx::tmem_st16(t_s + h + 16, lo16);
                    }
                    l += (s0.x + s0.y) + (s1.x + s1.y);
                    ptx::tmem_wait_st();
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar_p + 8 * x);
            }
            if (!ok) break;

            // ------------------------------------------------------------ the item's rows
            // one tile's rows, or the merge of both tiles' (by tile 0's warps)
            float m1 = -INFINITY, l1 = 0.f;
            if (!two && x == 1) {
                if (merges > 0) ok = ptx::mbar_wait(bar_mlfree, (merges - 1) & 1, kWaitLimitCycles);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ml[r] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar_ml);
            } else if (!two) {
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_ml, merges & 1, kWaitLimitCycles));
                if (!ok) break;
                const float2 a = ml[r];
                m1 = a.x;
                l1 = a.y;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar_mlfree);
            }
            const int n_pieces = it.pieces >> 16;
            if (two || x == 0) {
                const bool has0 = n_mine > 0, has1 = !two && it.n > 1;  // O of this tile, of tile 1
                if (has0) ok = ptx::mbar_wait(bar_o + 8 * x, items_with[x] & 1, kWaitLimitCycles);
                if (has1) ok = ok && ptx::mbar_wait(bar_o + 8, items_with[1] & 1, kWaitLimitCycles);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ptx::tc_fence_after();
                if (warp_ok) {
                    const int t = tok, hq = it.kvh * p.G + (R - t * p.G);
                    const float z = sink_z;
                    const float M = fmaxf(fmaxf(m, m1), z);
                    float f0 = 0.f, f1 = 0.f, lse = -INFINITY;
                    if (M != -INFINITY) {
                        const float w0 = m == -INFINITY ? 0.f : ptx::ex2(m - M), w1 = m1 == -INFINITY ? 0.f : ptx::ex2(m1 - M);
                        const float den = l * w0 + l1 * w1 + (z == -INFINITY ? 0.f : ptx::ex2(z - M));
                        f0 = w0 / den;
                        f1 = w1 / den;
                        lse = M + log2f(den);
                    }
                    float* rec = nullptr;
                    if (n_pieces > 1) {
                        const int c = it.pieces & 0xffff;
                        const size_t at = static_cast<size_t>(it.rec) + (static_cast<size_t>(c) * p.Hkv + it.kvh) * it.rows + rr;
                        rec = p.rec_o + at * D;
                        if (row_ok) p.rec_lse[at] = lse;
                    }
                    const size_t out_row = (static_cast<size_t>(it.row0 + t) * p.Hq + hq) * D;
#pragma unroll 1
                    for (int d = 0; d < D; d += 16) {
                        float o[16];
                        {
                            uint32_t a[16], b[16];
                            if (has0) ptx::tmem_ld16(tmem + lane_addr + 256 + 128 * x + d, a);
                            if (has1) ptx::tmem_ld16(tmem + lane_addr + 384 + d, b);
                            if (has0) ptx::tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                o[k] = has0 && f0 != 0.f ? __uint_as_float(a[k]) * f0 : 0.f;
                                if (has1 && f1 != 0.f) o[k] = fmaf(__uint_as_float(b[k]), f1, o[k]);
                            }
                        }
                        if (!row_ok) continue;
                        if (rec || F32) {
                            float4* to = reinterpret_cast<float4*>((rec ? rec : static_cast<float*>(p.out) + out_row) + d);
#pragma unroll
                            for (int k = 0; k < 4; ++k) to[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                        } else {
                            uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + out_row + d);
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                to[k] = make_uint4(pk_pack(o[8 * k], o[8 * k + 1]), pk_pack(o[8 * k + 2], o[8 * k + 3]),
                                                   pk_pack(o[8 * k + 4], o[8 * k + 5]), pk_pack(o[8 * k + 6], o[8 * k + 7]));
                        }
                    }
                }
                ptx::tc_fence_before();
            }
            // O may be overwritten: each tile's warps count in for what they have read, tile 0's for
            // both tiles where they merged them (tile 1's may be an item ahead by then)
            __syncwarp();
            if (it.n > 0 && lane == 0 && (two || x == 0)) ptx::mbar_arrive_n(bar_ofree, two ? 1 : 2);

            // the last piece of a cut pair to finish merges the records, in the pieces' order
            if (n_pieces > 1 && (two || x == 0)) {
                __threadfence();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar_rec + 8 * x);
                volatile int* last = reinterpret_cast<volatile int*>(base_ptr + SH::kOffLast) + x;
                if (r == 0) {
                    ok = ptx::mbar_wait(bar_rec + 8 * x, cuts & 1, kWaitLimitCycles);
                    unsigned* count = p.counters + (static_cast<size_t>(it.group) * p.Hkv + it.kvh) * 2 + x;
                    __threadfence();
                    const bool is_last = ok && atomicAdd(count, 1u) == static_cast<unsigned>(n_pieces) - 1u;
                    if (is_last) *count = 0u;  // for another attention by the same list
                    __threadfence();
                    *last = is_last;
                    ptx::mbar_arrive(bar_last + 8 * x);
                }
                ok = __all_sync(0xffffffffu, ok && ptx::mbar_wait(bar_last + 8 * x, cuts & 1, kWaitLimitCycles));
                if (!ok) break;
                if (*last) merge_pieces<D, F32>(p, it, two ? 128 * x : 0, two ? min(128, it.rows - 128 * x) : it.rows, n_pieces, quad, lane);
                ++cuts;
            }
            if (!two) ++merges;
            if (it.n > 0) ring.skip(2 * it.n);
            steps += n_mine;
            if (it.n > 0) ++items_with[0];
            if (it.n > (two ? 0 : 1)) ++items_with[1];
        }
        if (!ok && lane == 0) give_up();
    } else {
        set_max_regs_dec<64>();
        // ---------------------------------------------------------------- q' rows
        // A warp takes every fourth row, a lane D / 32 neighbouring dims; the first 32 rows'
        // loads are out before the item before has let go of the slots.
        constexpr int E = D / 32;
        const int w = warp - 12;
        bool ok = true;
        int busy = 0;
        bool was_two = false;
        PkRing<D, KV> ring{};
        int coded = 0;           // tiles of codes so far (of all teams)
        uint32_t stage_ph = 0;   // parity of the uses so far of the team's stages
        ring.begin(false);
        for (int i = 0; ok; ++i) {
            PkItem it;
            ok = take_item(i, it);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) drop_item(i);
            if (!(it.flags & 1)) break;
            if (it.n == 0) continue;
            const bool two = !kCodes && (it.flags & 2);
            // the rows' tiles are free once the S MMAs of the item before are done; a second tile's
            // may still hold its values before the last P . V
            const bool wait_pv = SH::kRingTwo < SH::kRing && two && !was_two;
            for (int b0 = 0; b0 < it.rows; b0 += 32) {
                float q[8][E];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int rr = b0 + 4 * k + w;
#pragma unroll
                    for (int e = 0; e < E; ++e) q[k][e] = 0.f;
                    if (rr < it.rows) {
                        const int R = it.r0 + rr, t = R / p.G;
                        const float* from = p.q_prime + (static_cast<size_t>(it.row0 + t) * p.Hq + it.kvh * p.G + (R - t * p.G)) * D + E * lane;
                        if constexpr (E == 4) {
                            const float4 a = *reinterpret_cast<const float4*>(from);
                            q[k][0] = a.x, q[k][1] = a.y, q[k][2] = a.z, q[k][3] = a.w;
                        } else {
                            const float2 a = *reinterpret_cast<const float2*>(from);
                            q[k][0] = a.x, q[k][1] = a.y;
                        }
                    }
                }
                if (b0 == 0 && busy > 0) {
                    ok = ptx::mbar_wait(bar_qfree, (busy - 1) & 1, kWaitLimitCycles);
                    if (ok && wait_pv) ok = ptx::mbar_wait(bar_idone, (busy - 1) & 1, kWaitLimitCycles);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int rr = b0 + 4 * k + w;
                    if (rr >= it.rows) continue;
                    const int row = rr & 127, d = E * lane;
                    uint8_t* to = base_ptr + (rr >> 7) * 2 * SH::kTile + (d >> 6) * (128 * 128) + row * 128 +
                                  ((((d & 63) >> 3) ^ (row & 7)) << 4) + (d & 7) * 2;
                    uint32_t hi[E / 2], lo[E / 2];
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        hi[e] = pk_pack(q[k][2 * e], q[k][2 * e + 1]);
                        lo[e] = pk_pack(q[k][2 * e] - __uint_as_float(hi[e] << 16),
                                        q[k][2 * e + 1] - __uint_as_float(hi[e] & 0xffff0000u));
                    }
                    if constexpr (E == 4) {
                        *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
                        *reinterpret_cast<uint2*>(to + SH::kTile) = make_uint2(lo[0], lo[1]);
                    } else {
                        *reinterpret_cast<uint32_t*>(to) = hi[0];
                        *reinterpret_cast<uint32_t*>(to + SH::kTile) = lo[0];
                    }
                }
            }
            if (!ok) break;
            ptx::fence_proxy_async();  // visible to the tensor core
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_qfull);
            was_two = two;
            ++busy;
            if (kCodes) {
                // The item's codes, widened to bf16 (exact) into the ring's tiles in the order of first
                // use. At head_dim 64 two warps take a tile, in turn with the other two: its waits, loads
                // and fences are as long as its arithmetic. 16 codes of a row per thread and turn, neighbouring rows taking other halves
                // at head_dim 128, so that neither the loads nor the swizzled stores share banks.
                const int hi = it.L + (it.r0 + it.rows - 1) / p.G + 1;
                constexpr int kRowStep = 8 * SH::kWideners;  // rows of a turn
                const int tid = 32 * (w % SH::kWideners) + lane, rt = tid >> 2;
                for (int k = 0; k < 2 * it.n && ok; ++k) {
                    const bool is_key = k == 0 || ((k & 1) && k != 2 * it.n - 1);
                    const uint32_t par = ring.parity();
                    const int s = ring.take();
                    if (is_key && !kKeyCodes) continue;
                    const int t = coded++;
                    if (t % SH::kTeams != w / SH::kWideners) continue;
                    const int sg = SH::stage(t);
                    const uint32_t stage_par = stage_ph >> sg & 1u;
                    stage_ph ^= 1u << sg;
                    const int j = is_key ? (k + 1) / 2 : k == 2 * it.n - 1 ? it.n - 1 : (k - 2) / 2;
                    const int blk = it.blk0 + j;
                    const bool in_first = blk < it.n_f;
                    const int key0 = (in_first ? blk : it.kb0 + blk - it.n_f) * kPackedKeys;
                    // rows that no row of the pair sees may hold anything: zeros, and scales of zero
                    const int keep = is_key ? kPackedKeys : (in_first ? it.first : hi) - key0, skip = is_key || in_first ? 0 : it.lo - key0;
                    const bool whole = keep >= kPackedKeys && skip <= 0;
                    ok = ptx::mbar_wait(bar_sfull + 8 * sg, stage_par, kWaitLimitCycles) &&
                         ptx::mbar_wait(bar_empty + 8 * s, par ^ 1u, kWaitLimitCycles);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint32_t st = base + SH::kOffStage + sg * SH::kStage, to = base + PkRing<D, KV>::tile(s);
                    constexpr int kTurns = 128 / kRowStep * (D / 64), kAhead = 4;
#pragma unroll 1
                    for (int q0 = 0; q0 < kTurns; q0 += kAhead) {
                        uint4 c[kAhead];
                        int row[kAhead], group[kAhead];
#pragma unroll
                        for (int q = 0; q < kAhead; ++q) {
                            row[q] = D == 64 ? kRowStep * (q0 + q) + rt : kRowStep * ((q0 + q) >> 1) + rt;
                            group[q] = D == 64 ? tid & 3 : (tid & 3) + 4 * ((q & 1) ^ (rt & 1));
                            c[q] = ptx::ld_shared_v4(st + row[q] * D + 16 * group[q]);
                        }
                        if (!whole)
#pragma unroll
                            for (int q = 0; q < kAhead; ++q)
                                if (row[q] < skip || row[q] >= keep) c[q] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                        for (int q = 0; q < kAhead; ++q) store_widened(to, row[q], group[q], c[q]);
                    }
                    if (!is_key) {
#pragma unroll
                        for (int key = tid; key < kPackedKeys; key += 32 * SH::kWideners) {
                            const bool in = key >= skip && key < keep;
                            const uint32_t sc = base + SH::kOffScales + s * SH::kScales + 4 * key;
                            const float vs = ptx::ld_shared_f32(st + 128 * D + 4 * key);
                            ptx::st_shared_f32(sc, in ? vs : 0.f);
                            if (kKeyCodes) {
                                const float ks = ptx::ld_shared_f32(st + 128 * D + 512 + 4 * key);
                                ptx::st_shared_f32(sc + 512, in ? ks : 0.f);
                            }
                        }
                    }
                    ptx::fence_proxy_async();  // visible to the tensor core
                    __syncwarp();
                    if (lane == 0) {
                        ptx::mbar_arrive(bar_sempty + 8 * sg);
                        ptx::mbar_arrive_n(bar_full + 8 * s, SH::kTeams);
                    }
                }
            }
        }
        if (!ok && lane == 0) give_up();
    }

    // TMEM is freed by the warp that allocated it, after every reader and the MMAs are done
    ptx::tc_fence_before();
    __syncthreads();
    if (ptx::flag_get(failed))  // the barriers' phases mean little then: copies in flight have this long to land
        for (const long long since = clock64(); clock64() - since < kGraceCycles;) __nanosleep(1000);
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kPkTmemCols);
    }
}

template <int D, int KV, bool F32>
cudaError_t launch_pk(const PackedUmmaParams& p, const PackedMaps& maps, int n_sm, cudaStream_t s)
{
    using SH = PkShape<D, KV>;
    auto kern = packed_umma_kernel<D, KV, F32>;
    static int configured_device_mask = 0;  // bit per device that has the smem attribute set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 31 || !(configured_device_mask & (1 << dev))) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SH::kSmemBytes);
        if (e != cudaSuccess) return e;
        if (dev < 31) configured_device_mask |= 1 << dev;
    }
    return launch_dependent(kern, dim3(n_sm), dim3(kPkThreads), SH::kSmemBytes, s, maps, p);
}

}  // namespace
}  // namespace uaa
