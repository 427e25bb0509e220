// pages.cu -- the pages of a paged cache: branching sequences (fork, reserve),
// giving pages back (trim) and closing the holes they leave (compact), on the
// block table and a reference count per page; and the copies that these ask of
// every layer's pools.
//
// page_refs[p] is the number of table entries that name page p (plus whatever the
// caller pins); 0 is a free page. There is no free list: the free pages are the
// zeros of page_refs in ascending order, so every result is a function of the
// state alone, whatever order CTAs run in (the counts are integer atomics, whose
// order does not matter).
//
// The bookkeeping reads and writes the table and the counts once or twice, some
// hundred kilobytes: it is bound by launches and dependent loads. fork and trim
// are a thread per table entry; reserve and compact rank pages in order, which one
// CTA does by scanning (1,024 threads take 16 Ki pages a round). The copy is bound
// by HBM: pages are contiguous, CTAs take 16 KB pieces of them round robin.
#include "internal.cuh"

namespace uaa {
namespace {

constexpr int kPageThreads = 256;
constexpr int kScanThreads = 1024;
constexpr int kScanPer = 16;  // pages per thread and round of a scan, as four 16-byte loads

__device__ __forceinline__ bool is_page(const PageParams& p, int e) { return e >= 0 && e < p.n_pages; }

// A table entry that is neither a page nor absent (-1) is flagged and left alone.
__device__ __forceinline__ void check_entry(const PageParams& p, int e)
{
    if (e < -1 || e >= p.n_pages) atomicOr(p.status, UAA_DEVFLAG_PAGE);
}

// A copy that follows finds nothing to do.
__device__ __forceinline__ void no_moves(const PageParams& p) { p.counts[0] = 0; }

// ---------------------------------------------------------------- fork
// Row b takes row parents[b] as it was before the call (-1: no pages, length 0).
// First every new row into the workspace, with the counts; then the rows back. The
// moves of an operator before this one are void (no_moves): its pages may be others'
// now.
__global__ void __launch_bounds__(kPageThreads) fork_gather_kernel(const PageParams p, const int* parents)
{
    grid_dependency_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kPageThreads + threadIdx.x;
    if (i >= static_cast<int64_t>(p.B) * p.per_seq) return;
    if (i == 0) no_moves(p);
    const int b = static_cast<int>(i / p.per_seq), l = static_cast<int>(i - static_cast<int64_t>(b) * p.per_seq);
    int par = parents[b];
    if (par < -1 || par >= p.B) {
        if (l == 0) atomicOr(p.status, UAA_DEVFLAG_PAGE);
        par = b;
    }
    const int old = p.table[i];
    const int now = par < 0 ? -1 : p.table[static_cast<int64_t>(par) * p.per_seq + l];
    if (l == 0) p.lens_tmp[b] = par < 0 ? 0 : p.seq_lens[par];
    p.table_tmp[i] = now;
    if (par == b) return;
    check_entry(p, old);
    if (is_page(p, old)) atomicSub(p.refs + old, 1);
    if (is_page(p, now)) atomicAdd(p.refs + now, 1);
}

__global__ void __launch_bounds__(kPageThreads) fork_scatter_kernel(const PageParams p)
{
    grid_dependency_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kPageThreads + threadIdx.x;
    if (i < static_cast<int64_t>(p.B) * p.per_seq) p.table[i] = p.table_tmp[i];
    if (i < p.B) p.seq_lens[i] = p.lens_tmp[i];
}

// A table of up to kForkEntries entries in one launch: one CTA holds all new rows in
// registers before it writes any (2.5 us for the two launches, 1.6 for this one).
constexpr int kForkThreads = 1024, kForkPer = 8;
constexpr int kForkEntries = kForkThreads * kForkPer;

__global__ void __launch_bounds__(kForkThreads) fork_small_kernel(const PageParams p, const int* parents)
{
    grid_dependency_wait();
    const int n = p.B * p.per_seq;
    if (threadIdx.x == 0) no_moves(p);
    int now[kForkPer], len[kForkPer];
#pragma unroll
    for (int k = 0; k < kForkPer; ++k) {
        const int i = k * kForkThreads + threadIdx.x;
        if (i >= n) break;
        const int b = i / p.per_seq, l = i - b * p.per_seq;
        int par = parents[b];
        if (par < -1 || par >= p.B) {
            if (l == 0) atomicOr(p.status, UAA_DEVFLAG_PAGE);
            par = b;
        }
        const int old = p.table[i];
        now[k] = par < 0 ? -1 : p.table[par * p.per_seq + l];
        len[k] = l == 0 ? (par < 0 ? 0 : p.seq_lens[par]) : -1;
        if (par == b) continue;
        check_entry(p, old);
        if (is_page(p, old)) atomicSub(p.refs + old, 1);
        if (is_page(p, now[k])) atomicAdd(p.refs + now[k], 1);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kForkPer; ++k) {
        const int i = k * kForkThreads + threadIdx.x;
        if (i >= n) break;
        p.table[i] = now[k];
        if (i % p.per_seq == 0) p.seq_lens[i / p.per_seq] = len[k];
    }
}

// ---------------------------------------------------------------- trim
// Pages whose positions no later token sees (behind the window of the token that
// comes next, and past the first tokens) leave the table.
__global__ void __launch_bounds__(kPageThreads) trim_kernel(const PageParams p, int window, int first_tokens)
{
    grid_dependency_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kPageThreads + threadIdx.x;
    if (i >= static_cast<int64_t>(p.B) * p.per_seq) return;
    if (i == 0) no_moves(p);
    const int b = static_cast<int>(i / p.per_seq), l = static_cast<int>(i - static_cast<int64_t>(b) * p.per_seq);
    const int64_t at = static_cast<int64_t>(l) * p.page_size;
    const int e = p.table[i];
    check_entry(p, e);
    if (!is_page(p, e)) return;
    if (at < first_tokens || at + p.page_size > static_cast<int64_t>(p.seq_lens[b]) - window + 1) return;
    p.table[i] = -1;
    atomicSub(p.refs + e, 1);
}

// ---------------------------------------------------------------- scans of one CTA

// Exclusive prefix of v over the CTA's threads, and the total (buf: 33 ints; every
// thread takes part; buf may be reused after the next __syncthreads).
__device__ __forceinline__ int block_prefix(int v, int* buf, int& total)
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
    if (warp == 0) {
        const int w = lane < kScanThreads / 32 ? buf[lane] : 0;
        int s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        buf[lane] = s - w;
        if (lane == 31) buf[32] = s;
    }
    __syncthreads();
    total = buf[32];
    return buf[warp] + x - v;
}

// The counts of pages i0 .. i0 + kScanPer - 1 (pages past the end count as held: 1).
__device__ __forceinline__ void load_refs(const PageParams& p, int64_t i0, int (&r)[kScanPer])
{
    if (i0 + kScanPer <= p.n_pages) {
#pragma unroll
        for (int k = 0; k < kScanPer / 4; ++k) {
            const int4 a = reinterpret_cast<const int4*>(p.refs + i0)[k];
            r[4 * k] = a.x, r[4 * k + 1] = a.y, r[4 * k + 2] = a.z, r[4 * k + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < kScanPer; ++k) r[k] = i0 + k < p.n_pages ? p.refs[i0 + k] : 1;
    }
}

// ---------------------------------------------------------------- reserve
// Pages of its own for every sequence's next q_len tokens. A request is a table
// entry (b, l) of those positions that is absent, or whose page others hold too
// (where all holders ask, the last of them in (b, l) order keeps it). Requests in
// (b, l) order take the free pages in ascending order. All of them, or none.
//
// Requests are enumerated as (b, k), k < per: logical page seq_lens[b] / ps + k.
struct Request {
    bool wanted, held;
    int at;    // table index
    int e;     // its entry
    int L;
    int l;
};

__device__ __forceinline__ Request request_of(const PageParams& p, int64_t i, int per, int q_len)
{
    Request r{};
    const int b = static_cast<int>(i / per), k = static_cast<int>(i - static_cast<int64_t>(b) * per);
    if (b >= p.B) return r;
    r.L = p.seq_lens[b];
    const int64_t end = static_cast<int64_t>(r.L) + q_len;
    if (r.L < 0 || end > static_cast<int64_t>(p.per_seq) * p.page_size) return r;  // the step does not append it
    r.l = r.L / p.page_size + k;
    if (r.l > (end - 1) / p.page_size) return r;
    r.at = b * p.per_seq + r.l;
    r.e = p.table[r.at];
    r.held = is_page(p, r.e);
    r.wanted = r.held || r.e == -1;
    return r;
}

__device__ __forceinline__ bool stays(const PageParams& p, const Request& r)
{
    const int n = __ldcg(p.refs + r.e);
    return n <= 1 || (n == __ldcg(p.asked + r.e) && __ldcg(p.last + r.e) == r.at + 1);
}

// Up to a request per thread (most steps): each is read once and kept in registers,
// the first pages' counts are on their way meanwhile, and the free pages go through
// shared memory: four dependent round trips to memory.
__global__ void __launch_bounds__(kScanThreads) reserve_small_kernel(const PageParams p, int q_len)
{
    __shared__ int buf[33];
    __shared__ int list[kScanThreads];
    grid_dependency_wait();
    const int tid = threadIdx.x;
    const int per = (q_len - 1) / p.page_size + 2;  // logical pages that q_len positions can touch
    int cnt[kScanPer];
    load_refs(p, static_cast<int64_t>(tid) * kScanPer, cnt);
    const Request r = request_of(p, tid, per, q_len);
    if (!r.wanted && r.e != 0) check_entry(p, r.e);
    const bool held = r.wanted && r.held;
    if (held) {
        atomicAdd(p.asked + r.e, 1);
        atomicMax(p.last + r.e, r.at + 1);
    }
    __threadfence();
    __syncthreads();
    const bool take = r.wanted && !(held && stays(p, r));
    const bool copy = take && held && static_cast<int64_t>(r.l) * p.page_size < r.L;
    int both;  // takes, and copies in the upper half (at most 1,024 each)
    const int rank2 = block_prefix((take ? 1 : 0) | (copy ? 1 << 16 : 0), buf, both);
    const int takes = both & 0xffff, rank = rank2 & 0xffff, c = rank2 >> 16;
    int found = 0;
    for (int64_t i0 = 0; i0 < p.n_pages && found < takes; i0 += kScanThreads * kScanPer) {
        if (i0) load_refs(p, i0 + static_cast<int64_t>(tid) * kScanPer, cnt);
        int n = 0;
#pragma unroll
        for (int k = 0; k < kScanPer; ++k) n += cnt[k] == 0;
        int total;
        int at = found + block_prefix(n, buf, total);
#pragma unroll
        for (int k = 0; k < kScanPer; ++k)
            if (cnt[k] == 0) {
                if (at < takes) list[at] = static_cast<int>(i0) + tid * kScanPer + k;
                ++at;
            }
        found += total;
    }
    __syncthreads();  // the list; and every decision is made
    const bool enough = found >= takes;
    if (take && enough) {
        const int page = list[rank];
        p.table[r.at] = page;
        p.refs[page] = 1;
        if (held) atomicSub(p.refs + r.e, 1);
        if (copy) {
            p.moves[2 * c] = r.e;
            p.moves[2 * c + 1] = page;
        }
    }
    if (held) {
        p.asked[r.e] = 0;
        p.last[r.e] = 0;
    }
    if (tid == 0) {
        p.counts[0] = enough ? both >> 16 : 0;
        p.counts[2] = takes;
        if (!enough) atomicOr(p.status, UAA_DEVFLAG_POOL);
    }
}

__global__ void __launch_bounds__(kScanThreads) reserve_kernel(const PageParams p, int q_len)
{
    __shared__ int buf[33];
    grid_dependency_wait();
    const int tid = threadIdx.x;
    const int per = (q_len - 1) / p.page_size + 2;  // logical pages that q_len positions can touch
    const int64_t n_req = static_cast<int64_t>(p.B) * per;

    // who asks for which held page (asked and last are zero between calls)
    for (int64_t i = tid; i < n_req; i += kScanThreads) {
        const Request r = request_of(p, i, per, q_len);
        if (!r.wanted) {
            if (r.e != 0 && !r.held) check_entry(p, r.e);
            continue;
        }
        if (r.held) {
            atomicAdd(p.asked + r.e, 1);
            atomicMax(p.last + r.e, r.at + 1);
        }
    }
    __threadfence();
    __syncthreads();

    // how many take a page
    int mine = 0, takes;
    for (int64_t i = tid; i < n_req; i += kScanThreads) {
        const Request r = request_of(p, i, per, q_len);
        mine += r.wanted && !(r.held && stays(p, r));
    }
    block_prefix(mine, buf, takes);

    // the free pages of lowest index, as many as are asked for
    int found = 0;
    for (int64_t i0 = 0; i0 < p.n_pages && found < takes; i0 += kScanThreads * kScanPer) {
        int r[kScanPer];
        load_refs(p, i0 + static_cast<int64_t>(tid) * kScanPer, r);
        int n = 0;
#pragma unroll
        for (int k = 0; k < kScanPer; ++k) n += r[k] == 0;
        int total;
        int rank = found + block_prefix(n, buf, total);
#pragma unroll
        for (int k = 0; k < kScanPer; ++k)
            if (r[k] == 0) {
                if (rank < takes) p.list[rank] = static_cast<int>(i0) + tid * kScanPer + k;
                ++rank;
            }
        found += total;
    }
    __syncthreads();
    const bool enough = found >= takes;

    // the new entries, and the pages to copy (those with rows before the new tokens).
    // stays() reads counts and marks of held pages, which nothing changes in this loop:
    // the counts set here are those of free pages, and the pages given up are listed in
    // table_tmp and taken off their counts after it.
    int given = 0, copies = 0;
    for (int64_t i0 = 0; i0 < n_req; i0 += kScanThreads) {
        const Request r = request_of(p, i0 + tid, per, q_len);
        const bool take = r.wanted && !(r.held && stays(p, r));
        int n_take, n_copy;
        const int rank = given + block_prefix(take, buf, n_take);
        const bool copy = take && r.held && static_cast<int64_t>(r.l) * p.page_size < r.L;
        const int c = copies + block_prefix(copy, buf, n_copy);
        if (take && enough) {
            const int page = p.list[rank];
            p.table[r.at] = page;
            p.table_tmp[rank] = r.held ? r.e : -1;  // the page given up, taken off its count at the end
            p.refs[page] = 1;
            if (copy) {
                p.moves[2 * c] = r.e;
                p.moves[2 * c + 1] = page;
            }
        }
        if (r.held && !enough) {  // nothing changes: the marks go
            p.asked[r.e] = 0;
            p.last[r.e] = 0;
        }
        given += n_take;
        copies += n_copy;
    }
    __syncthreads();
    if (enough) {
        for (int i = tid; i < given; i += kScanThreads) {
            const int e = p.table_tmp[i];
            if (e < 0) continue;
            atomicSub(p.refs + e, 1);
            p.asked[e] = 0;
            p.last[e] = 0;
        }
        // requests that kept their page
        for (int64_t i = tid; i < n_req; i += kScanThreads) {
            const Request r = request_of(p, i, per, q_len);
            if (!r.held) continue;
            p.asked[r.e] = 0;
            p.last[r.e] = 0;
        }
    }
    if (tid == 0) {
        p.counts[0] = enough ? copies : 0;
        p.counts[2] = takes;
        if (!enough) atomicOr(p.status, UAA_DEVFLAG_POOL);
    }
}

// ---------------------------------------------------------------- compact
// The i-th held page at or past the number of held pages moves to the i-th free
// page before it. One CTA ranks the pages and writes the moves, the new counts and
// the map from old to new pages; the grid that follows renames the table's entries.
__global__ void __launch_bounds__(kScanThreads) compact_kernel(const PageParams p)
{
    __shared__ int buf[33];
    grid_dependency_wait();
    const int tid = threadIdx.x;
    int r[kScanPer];
    int mine = 0, live;
    for (int64_t i0 = 0; i0 < p.n_pages; i0 += kScanThreads * kScanPer) {
        load_refs(p, i0 + static_cast<int64_t>(tid) * kScanPer, r);
#pragma unroll
        for (int k = 0; k < kScanPer; ++k) mine += r[k] != 0 && i0 + static_cast<int64_t>(tid) * kScanPer + k < p.n_pages;
    }
    block_prefix(mine, buf, live);
    int holes = 0, movers = 0;
    for (int64_t i0 = 0; i0 < p.n_pages; i0 += kScanThreads * kScanPer) {
        const int64_t first = i0 + static_cast<int64_t>(tid) * kScanPer;
        if (p.n_pages > kScanThreads * kScanPer) load_refs(p, first, r);  // else they are the ones just counted
        int nh = 0, nm = 0;
#pragma unroll
        for (int k = 0; k < kScanPer; ++k) {
            if (first + k < p.n_pages) {
                nh += r[k] == 0 && first + k < live;
                nm += r[k] != 0 && first + k >= live;
            }
        }
        int th, tm;
        int h = holes + block_prefix(nh, buf, th);
        int m = movers + block_prefix(nm, buf, tm);
        int to[kScanPer];
#pragma unroll
        for (int k = 0; k < kScanPer; ++k) {
            const int page = static_cast<int>(first) + k;
            to[k] = r[k] != 0 && page < live ? page : -1;
            if (first + k >= p.n_pages) continue;
            if (r[k] == 0 && page < live) p.moves[2 * h++ + 1] = page;
            if (r[k] != 0 && page >= live) p.moves[2 * m++] = page;
        }
        if (first + kScanPer <= p.n_pages) {
#pragma unroll
            for (int k = 0; k < kScanPer / 4; ++k)
                reinterpret_cast<int4*>(p.map + first)[k] = make_int4(to[4 * k], to[4 * k + 1], to[4 * k + 2], to[4 * k + 3]);
        } else {
#pragma unroll
            for (int k = 0; k < kScanPer; ++k)
                if (first + k < p.n_pages) p.map[first + k] = to[k];
        }
        holes += th;
        movers += tm;
    }
    __threadfence_block();
    __syncthreads();
    for (int i = tid; i < movers; i += kScanThreads) {  // as many holes as movers
        const int2 mv = reinterpret_cast<const int2*>(p.moves)[i];
        const int n = p.refs[mv.x];
        p.map[mv.x] = mv.y;
        p.refs[mv.y] = n;
        p.refs[mv.x] = 0;
    }
    if (tid == 0) {
        p.counts[0] = movers;
        p.counts[1] = live;
    }
}

__global__ void __launch_bounds__(kPageThreads) rename_kernel(const PageParams p)
{
    grid_dependency_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kPageThreads + threadIdx.x;
    if (i >= static_cast<int64_t>(p.B) * p.per_seq) return;
    const int e = p.table[i];
    check_entry(p, e);
    if (!is_page(p, e)) return;
    const int to = p.map[e];
    if (to < 0)
        atomicOr(p.status, UAA_DEVFLAG_PAGE);  // an entry whose page has no count
    else if (to != e)
        p.table[i] = to;
}

// ---------------------------------------------------------------- copy
// The listed pages of every pool, src to dst. CTAs take pieces of kPiece bytes
// round robin over (move, pool, piece).
constexpr int kCopyThreads = 256;
constexpr int kPiece = kCopyThreads * 16 * 4;

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const PageParams p, const PagePools pools)
{
    grid_dependency_wait();
    const int n = p.counts[0];
    const int64_t total = static_cast<int64_t>(min(max(n, 0), p.n_pages)) * pools.pieces;
    for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
        const int m = static_cast<int>(w / pools.pieces);
        int piece = static_cast<int>(w - static_cast<int64_t>(m) * pools.pieces), k = 0;
        while (piece >= pools.pool_pieces[k]) piece -= pools.pool_pieces[k++];
        const int src = p.moves[2 * m], dst = p.moves[2 * m + 1];
        if (!is_page(p, src) || !is_page(p, dst)) {
            if (threadIdx.x == 0) atomicOr(p.status, UAA_DEVFLAG_PAGE);
            continue;
        }
        const int64_t bytes = pools.bytes[k], off = static_cast<int64_t>(piece) * kPiece;
        const char* from = pools.base[k] + src * bytes;
        char* to = pools.base[k] + dst * bytes;
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t at = off + (j * kCopyThreads + threadIdx.x) * 16;
            if (at < bytes) v[j] = __ldcs(reinterpret_cast<const uint4*>(from + at));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t at = off + (j * kCopyThreads + threadIdx.x) * 16;
            if (at < bytes) __stcs(reinterpret_cast<uint4*>(to + at), v[j]);
        }
    }
}

dim3 entries_grid(const PageParams& p)
{
    const int64_t n = static_cast<int64_t>(p.B) * p.per_seq;
    return dim3(static_cast<unsigned>((n + kPageThreads - 1) / kPageThreads));
}

}  // namespace

cudaError_t launch_pages_fork(const PageParams& p, const int* parents, cudaStream_t s)
{
    if (static_cast<int64_t>(p.B) * p.per_seq <= kForkEntries)
        return launch_dependent(fork_small_kernel, dim3(1), dim3(kForkThreads), 0, s, p, parents);
    const cudaError_t e = launch_dependent(fork_gather_kernel, entries_grid(p), dim3(kPageThreads), 0, s, p, parents);
    if (e != cudaSuccess) return e;
    return launch_dependent(fork_scatter_kernel, entries_grid(p), dim3(kPageThreads), 0, s, p);
}

cudaError_t launch_pages_trim(const PageParams& p, int window, int first_tokens, cudaStream_t s)
{
    return launch_dependent(trim_kernel, entries_grid(p), dim3(kPageThreads), 0, s, p, window, first_tokens);
}

cudaError_t launch_pages_reserve(const PageParams& p, int q_len, cudaStream_t s)
{
    const int64_t n_req = static_cast<int64_t>(p.B) * ((q_len - 1) / p.page_size + 2);
    auto* kern = n_req <= kScanThreads ? reserve_small_kernel : reserve_kernel;
    return launch_dependent(kern, dim3(1), dim3(kScanThreads), 0, s, p, q_len);
}

cudaError_t launch_pages_compact(const PageParams& p, cudaStream_t s)
{
    const cudaError_t e = launch_dependent(compact_kernel, dim3(1), dim3(kScanThreads), 0, s, p);
    if (e != cudaSuccess || p.B == 0) return e;
    return launch_dependent(rename_kernel, entries_grid(p), dim3(kPageThreads), 0, s, p);
}

cudaError_t launch_pages_copy(const PageParams& p, const PagePools& in, int n_sm, cudaStream_t s)
{
    PagePools pools = in;
    pools.pieces = 0;
    for (int k = 0; k < pools.n; ++k) {
        const int64_t n = (pools.bytes[k] + kPiece - 1) / kPiece;
        if (pools.pieces + n > (1 << 30)) return cudaErrorInvalidValue;
        pools.pool_pieces[k] = static_cast<int>(n);
        pools.pieces += static_cast<int>(n);
    }
    return launch_dependent(copy_pages_kernel, dim3(8 * n_sm), dim3(kCopyThreads), 0, s, p, pools);
}

}  // namespace uaa
