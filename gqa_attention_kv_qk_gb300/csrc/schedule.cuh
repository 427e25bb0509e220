// schedule.cuh -- the work list of the packed attention kernel (packed_umma.cuh), built
// by one CTA of the append's launch from the plan's arrays.
//
// The (token, head) rows of a kv head of request b (row r: token r / G, head r % G) are
// cut into row pairs, 2 x 128 rows that read the same keys (128 over 8-bit caches). A row pair's cost is its
// 128-key blocks and a constant. Pairs are listed by falling cost (16 classes), so that
// CTAs that take entries from a counter end at about the same time; with n_sm CTAs, the
// pairs beyond the last full round of n_sm (all of them where there are fewer), and any
// pair that costs more than an even share of everything, are cut along the keys into
// pieces, whose records the last one to finish merges. What is cut, and where, depends on
// the lengths alone: results do not depend on the order in which CTAs run.
#pragma once

#include "internal.cuh"

namespace uaa {

// The key blocks that rows [r0, r0 + n) of a request see: [0, first) in n_f blocks, then
// [lo, hi) from block kb0.
struct PairKeys {
    int n_blocks, n_f, kb0, first, lo, hi;
};

__device__ __forceinline__ PairKeys pair_keys(int r0, int n, int G, int L, int window, int first_tokens)
{
    PairKeys k;
    k.hi = L + (r0 + n - 1) / G + 1;
    const int lo_w = window > 0 ? max(0, L + r0 / G + 1 - window) : 0;
    k.first = lo_w > first_tokens ? first_tokens : 0;
    k.lo = lo_w > first_tokens ? lo_w : 0;
    k.n_f = (k.first + kPackedKeys - 1) / kPackedKeys;
    k.kb0 = k.lo / kPackedKeys;
    k.n_blocks = k.n_f + (k.hi + kPackedKeys - 1) / kPackedKeys - k.kb0;
    return k;
}

namespace {

constexpr int kCostClasses = 16;
constexpr int kCostFixed = 2;      // an item's start and end, in key blocks
constexpr int kMinPieceBlocks = 2;
constexpr int kMinGuided = 6;
constexpr int kSplitTries = 8;
// Requests, and pairs, whose arrays lie in shared memory (others: the workspace's).
constexpr int kScheduleFit = 512;
// shared words that build_schedule needs
constexpr int kScheduleWords = 32 * (2 + kSplitTries) + 32 * kCostClasses + kCostClasses + 8 + 3 * kScheduleFit + 4 + 3 * kScheduleFit;

struct PairOf {
    int b, rp, T, end, row0;
    int cost;
};

// Where the requests' arrays are read: shared memory or global.
struct Requests {
    const int* first;   // first pair of each
    const int* starts;  // q_starts
    const int* ends;    // kv_ends
};

// Pair i of the batch: its request (by the pairs' prefix) and cost.
__device__ __forceinline__ PairOf pair_of(const ScheduleParams& s, const Requests& q, int i)
{
    int lo = 0, hi = s.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q.first[mid] <= i) lo = mid;
        else hi = mid;
    }
    PairOf p;
    p.b = lo;
    p.rp = i - q.first[lo];
    p.row0 = q.starts[lo];
    p.T = q.starts[lo + 1] - p.row0;
    p.end = q.ends[lo];
    if (p.end > s.cap || p.end < p.T) p.end = -1;  // not a plan's
    p.cost = 1;
    if (p.end >= 0) {
        const int r0 = p.rp * s.pair_rows;
        p.cost = kCostFixed + pair_keys(r0, min(s.pair_rows, p.T * s.G - r0), s.G, p.end - p.T, s.window, s.first_tokens).n_blocks;
    }
    return p;
}

__device__ __forceinline__ int rows_of(const ScheduleParams& s, const PairOf& p)
{
    return min(s.pair_rows, p.T * s.G - p.rp * s.pair_rows);
}

// N sums over the CTA, or with MAX the last of them a maximum (every thread gets them; buf: 32 N words).
template <int N, bool MAX>
__device__ __forceinline__ void cta_reduce(int (&v)[N], int* buf)
{
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const int y = __shfl_xor_sync(0xffffffffu, v[k], o);
            v[k] = MAX && k == N - 1 ? max(v[k], y) : v[k] + y;
        }
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) buf[32 * k + (threadIdx.x >> 5)] = v[k];
    __syncthreads();
    const int n_warps = static_cast<int>(blockDim.x >> 5);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = buf[32 * k];
        for (int w = 1; w < n_warps; ++w) v[k] = MAX && k == N - 1 ? max(v[k], buf[32 * k + w]) : v[k] + buf[32 * k + w];
    }
}

// Exclusive prefix over the CTA's threads and the total (buf: 33 words).
__device__ __forceinline__ int cta_prefix(int v, int* buf, int& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) buf[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
        if (w < warp) before += buf[w];
        total += buf[w];
    }
    return before + x - v;
}

// Pieces of at most `size` cost units for a pair of this cost and these rows (no more
// than whose records are merged in a few microseconds).
__device__ __forceinline__ int pieces_of(int cost, int size, int rows)
{
    const int n = (cost - kCostFixed + size - 1) / size;
    return max(1, min(min(n, (cost - kCostFixed) / kMinPieceBlocks), kMergeRows / rows));
}

// One CTA of whole warps; sm: kScheduleWords words of shared memory, 8-byte aligned. A step
// of few requests waits for this (its rows are done in 3 us), so the arrays are in shared
// memory where they fit: the append of 64 decodes 15 us with them in L2, 12 us so.
__device__ void build_schedule(const ScheduleParams& s, int* sm)
{
    int2* order_s = reinterpret_cast<int2*>(sm);              // [kScheduleFit]
    int* costs_s = sm + 2 * kScheduleFit;                     // [kScheduleFit]
    int* first_s = costs_s + kScheduleFit;                    // [kScheduleFit]
    int* starts_s = first_s + kScheduleFit;                   // [kScheduleFit + 1]
    int* ends_s = starts_s + kScheduleFit + 4;                // [kScheduleFit]
    int* buf = ends_s + kScheduleFit;                         // 32 (2 + tries)
    int* counts = buf + 32 * (2 + kSplitTries);               // [warps][classes]
    int* class_at = counts + 32 * kCostClasses;               // [classes] next rank
    const int tid = threadIdx.x, nthr = blockDim.x, warp = tid >> 5, lane = tid & 31, n_warps = nthr >> 5;

    const bool few = s.B <= kScheduleFit;
    Requests q;
    if (few) {
        for (int b = tid; b <= s.B; b += nthr) {
            starts_s[b] = s.q_starts[b];
            if (b < s.B) ends_s[b] = s.kv_ends[b];
        }
        if (tid < kCostClasses) class_at[tid] = 0;
        __syncthreads();
        q = Requests{first_s, starts_s, ends_s};
    } else {
        if (tid < kCostClasses) class_at[tid] = 0;
        q = Requests{s.pair_first, s.q_starts, s.kv_ends};
    }
    int* const first = few ? first_s : s.pair_first;

    // the pairs of each request
    int n_pairs = 0;
    for (int b0 = 0; b0 < s.B; b0 += nthr) {
        const int b = b0 + tid;
        const int row0 = b < s.B ? q.starts[b] : 0;
        int T = b < s.B ? q.starts[b + 1] - row0 : 0;
        if (row0 < 0 || row0 > s.n_tokens - T) T = 0;  // not a plan's
        const int n = T > 0 ? (T * s.G + s.pair_rows - 1) / s.pair_rows : 0;
        int total;
        const int at = n_pairs + cta_prefix(n, buf, total);
        if (b < s.B) first[b] = at;
        n_pairs += total;
    }
    n_pairs = min(n_pairs, s.max_pairs);  // (the caller's arrays hold every plan of n_tokens rows)
    const bool small = n_pairs <= kScheduleFit;
    int* const costs = small ? costs_s : s.costs;
    int2* const order = small ? order_s : s.order;
    __syncthreads();

    // total and largest cost, and how many pairs of each class there are
    int sums[2] = {0, 0};
    for (int i = tid; i < n_pairs; i += nthr) {
        const int c = pair_of(s, q, i).cost;
        costs[i] = c;
        sums[0] += c;
        sums[1] = max(sums[1], c);
    }
    cta_reduce<2, true>(sums, buf);
    const int all = sums[0], top = sums[1];
    auto class_of = [&](int cost) { return kCostClasses - 1 - static_cast<int>(static_cast<long long>(cost) * kCostClasses / (top + 1)); };
    for (int i = tid; i < n_pairs; i += nthr) atomicAdd(&class_at[class_of(costs[i])], 1);
    __syncthreads();
    if (tid == 0) {
        int at = 0;
        for (int c = 0; c < kCostClasses; ++c) {
            const int n = class_at[c];
            class_at[c] = at;
            at += n;
        }
    }
    __syncthreads();
    // the pairs in order of (class, index)
    for (int i0 = 0; i0 < n_pairs; i0 += nthr) {
        const int i = i0 + tid;
        const int cost = i < n_pairs ? costs[i] : 0;
        const int mine = i < n_pairs ? class_of(cost) : -1;
        int before = 0;
#pragma unroll
        for (int c = 0; c < kCostClasses; ++c) {
            const unsigned m = __ballot_sync(0xffffffffu, mine == c);
            if (mine == c) before = __popc(m & ((1u << lane) - 1u));
            if (lane == 0) counts[warp * kCostClasses + c] = __popc(m);
        }
        __syncthreads();
        if (mine >= 0) {
            int rank = class_at[mine] + before;
            for (int w = 0; w < warp; ++w) rank += counts[w * kCostClasses + mine];
            order[rank] = make_int2(i, cost);
        }
        __syncthreads();
        if (tid < kCostClasses)
            for (int w = 0; w < n_warps; ++w) class_at[tid] += counts[w * kCostClasses + tid];
        __syncthreads();
    }

    // whole rounds of n_sm items, and the pairs beyond them
    const long long items = static_cast<long long>(n_pairs) * s.Hkv;
    const int whole = static_cast<int>(items / s.n_sm * s.n_sm / s.Hkv);
    const int share = static_cast<int>((static_cast<long long>(all) * s.Hkv + s.n_sm - 1) / s.n_sm);
    // The beyond-pairs' pieces. After whole rounds the CTAs come at different times: each pair
    // is cut into pieces of half an even share of what is left from it on, so that the last
    // ones are small. Without whole rounds: the size, of some around an even share, whose
    // pieces should end first (one round: with the largest piece; several: a piece after an even share).
    int tails[1] = {0};
    for (int r = whole + tid; r < n_pairs; r += nthr) tails[0] += order[r].y;
    cta_reduce<1, false>(tails, buf);
    const int tail = tails[0];
    int size = 0;
    if (whole == 0) {
        const int even = max(kMinPieceBlocks, static_cast<int>((static_cast<long long>(tail) * s.Hkv + s.n_sm - 1) / s.n_sm));
        const int tenths[kSplitTries] = {10, 11, 13, 16, 25, 6, 4, 2};
        int sizes[kSplitTries], n[kSplitTries];
#pragma unroll
        for (int k = 0; k < kSplitTries; ++k) {
            sizes[k] = max(kMinPieceBlocks, static_cast<int>(static_cast<long long>(even) * tenths[k] / 10));
            n[k] = 0;
        }
        for (int r = tid; r < n_pairs; r += nthr) {
            const int c = order[r].y, rows = rows_of(s, pair_of(s, q, order[r].x));
#pragma unroll
            for (int k = 0; k < kSplitTries; ++k) n[k] += pieces_of(c, sizes[k], rows);
        }
        cta_reduce<kSplitTries, false>(n, buf);
        float best = 0.f;
#pragma unroll
        for (int k = 0; k < kSplitTries; ++k) {
            const float pieces = static_cast<float>(n[k]) * s.Hkv, work = static_cast<float>(tail) * s.Hkv;
            const float each = work / fmaxf(pieces, 1.f);
            const float t = pieces <= s.n_sm ? each + kCostFixed : (work + kCostFixed * pieces) / s.n_sm + each;
            if (k == 0 || t < best) {
                best = t;
                size = sizes[k];
            }
        }
    }

    // the entries, with the places in the records and the counters of what is cut (a pair
    // whose records, counters or entries would not fit stays whole; each pair after it keeps
    // room for one entry, max_entries being max_pairs at least)
    int n_entries = 0, n_rec = 0, n_groups = 0, before = 0;  // (before: cost of the beyond-pairs so far)
    for (int r0 = 0; r0 < n_pairs; r0 += nthr) {
        const int r = r0 + tid;
        PairOf p{};
        int n = 0, rows = 0, n_tail;
        const int at_tail = before + cta_prefix(r >= whole && r < n_pairs ? order[r].y : 0, buf, n_tail);
        before += n_tail;
        if (r < n_pairs) {
            p = pair_of(s, q, order[r].x);
            rows = rows_of(s, p);
            n = 1;
            const int left = static_cast<int>(static_cast<long long>(tail - at_tail) * s.Hkv / (2 * s.n_sm));
            if (p.end >= 0 && r >= whole) n = pieces_of(p.cost, whole > 0 ? max(kMinGuided, left) : size, rows);
            else if (p.end >= 0 && p.cost > share) n = pieces_of(p.cost, max(kMinPieceBlocks, (share + 1) / 2), rows);
        }
        const long long want = n > 1 ? static_cast<long long>(n) * s.Hkv * rows : 0;
        int n_take, n_cut, n_all;
        const int rec = n_rec + cta_prefix(static_cast<int>(min(want, static_cast<long long>(s.max_rec_rows) + 1)), buf, n_take);
        const int group = n_groups + cta_prefix(n > 1 ? 1 : 0, buf, n_cut);
        if (rec + want > s.max_rec_rows || (group + 1) * 2 * s.Hkv > s.max_counters) n = min(n, 1);
        int at = n_entries + cta_prefix(n, buf, n_all);
        if (n_entries + n_all > s.max_entries - max(0, n_pairs - r0 - nthr)) {  // (the same for all threads)
            if (at + n > s.max_entries - (n_pairs - 1 - r)) n = min(n, 1);
            at = n_entries + cta_prefix(n, buf, n_all);
        }
        for (int k = 0; k < n; ++k)
            s.entries[at + k] = PackedEntry{p.b, p.rp, k | n << 16, group, p.row0, p.T, p.end, rec};
        if (n > 1)
            for (int h = 0; h < 2 * s.Hkv; ++h) s.counters[group * 2 * s.Hkv + h] = 0u;
        n_entries += n_all;
        n_rec = min(n_rec + n_take, s.max_rec_rows + 1);
        n_groups += n_cut;
    }
    if (tid == 0) {
        s.header[0] = static_cast<unsigned>(s.n_sm);                  // the next item after each CTA's first
        s.header[2] = 0u;                                             // CTAs that came to the list's end
        s.header[1] = static_cast<unsigned>(n_entries);               // entries
    }
}

}  // namespace
}  // namespace uaa
