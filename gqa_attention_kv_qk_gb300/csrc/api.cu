// api.cu -- the C ABI of libuaa: descriptor validation (typed refusals that name
// the fact, the Model support matrix page's "Conformance CLI" convention), the
// split geometry, workspace layout, TMA descriptors and the kernel launches.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <mutex>

#include "internal.cuh"

namespace {

thread_local char g_err[512] = "";

uaa_status fail(uaa_status st, const char* fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return st;
}

uaa_status cuda_fail(cudaError_t e, const char* what)
{
    return fail(UAA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

#define UAA_TRY(expr)                          \
    do {                                       \
        const uaa_status st_ = (expr);         \
        if (st_ != UAA_OK) return st_;         \
    } while (0)

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// ---------------------------------------------------------------- descriptor checks

uaa_status check_desc(const uaa_attn_desc* d)
{
    if (!d) return fail(UAA_ERR_INVALID_ARGUMENT, "desc is NULL");
    if (d->n_kv_heads <= 0) return fail(UAA_ERR_UNSUPPORTED, "n_kv_heads=%d is not positive", d->n_kv_heads);
    if (d->n_q_heads <= 0 || d->n_q_heads % d->n_kv_heads != 0)
        return fail(UAA_ERR_UNSUPPORTED,
                    "n_q_heads=%d is not a positive multiple of n_kv_heads=%d (integral GQA ratio required)",
                    d->n_q_heads, d->n_kv_heads);
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
        return fail(UAA_ERR_UNSUPPORTED, "head_dim=%d is not supported (supported: {64, 128, 256})",
                    d->head_dim);
    if (!(d->scale >= 0.f) || !isfinite(d->scale))
        return fail(UAA_ERR_UNSUPPORTED, "scale=%g is not a finite value >= 0", (double)d->scale);
    const uaa_rope_params& r = d->rope;
    if (r.style != UAA_ROPE_NEOX && r.style != UAA_ROPE_INTERLEAVED)
        return fail(UAA_ERR_UNSUPPORTED, "rope.style=%d is not NEOX (0) or INTERLEAVED (1)", r.style);
    if (!(r.theta > 0.0) || !isfinite(r.theta))
        return fail(UAA_ERR_UNSUPPORTED, "rope.theta=%g is not a finite value > 0", r.theta);
    if (r.scaling == UAA_ROPE_SCALING_LLAMA3) {
        if (!(r.factor >= 1.0) || !(r.low_freq_factor > 0.0) || !(r.high_freq_factor > r.low_freq_factor) ||
            r.original_max_pos <= 0)
            return fail(UAA_ERR_UNSUPPORTED,
                        "llama3 rope scaling needs factor>=1, 0<low_freq_factor<high_freq_factor, "
                        "original_max_pos>0 (got %g, %g, %g, %d)",
                        r.factor, r.low_freq_factor, r.high_freq_factor, r.original_max_pos);
    } else if (r.scaling == UAA_ROPE_SCALING_YARN) {
        if (!(r.factor > 0.0) || r.original_max_pos <= 0 || !(r.beta_slow > 0.0) || !(r.beta_fast > r.beta_slow))
            return fail(UAA_ERR_UNSUPPORTED,
                        "yarn rope scaling needs factor>0, original_max_pos>0, beta_fast>beta_slow>0 "
                        "(got %g, %d, %g, %g)",
                        r.factor, r.original_max_pos, r.beta_fast, r.beta_slow);
    } else if (r.scaling == UAA_ROPE_SCALING_LINEAR) {
        if (!(r.factor > 0.0) || !isfinite(r.factor))
            return fail(UAA_ERR_UNSUPPORTED, "linear rope scaling needs a finite factor>0 (got %g)", r.factor);
    } else if (r.scaling != UAA_ROPE_SCALING_NONE) {
        return fail(UAA_ERR_UNSUPPORTED, "rope.scaling=%d is not supported (none, llama3, yarn, linear)",
                    r.scaling);
    }
    if (d->rotary_dim != 0 && (d->rotary_dim < 2 || d->rotary_dim > d->head_dim || d->rotary_dim % 2 != 0))
        return fail(UAA_ERR_UNSUPPORTED, "rotary_dim=%d is not 0 or an even value in [2, head_dim=%d]",
                    d->rotary_dim, d->head_dim);
    if (d->norm_offset != 0 && d->norm_offset != 1)
        return fail(UAA_ERR_UNSUPPORTED, "norm_offset=%d is not 0 or 1", d->norm_offset);
    if (d->reproducible != 0 && d->reproducible != 1)
        return fail(UAA_ERR_UNSUPPORTED, "reproducible=%d is not 0 or 1", d->reproducible);
    if (d->qk_norm != 0 && d->qk_norm != 1)
        return fail(UAA_ERR_UNSUPPORTED, "qk_norm=%d is not 0 or 1", d->qk_norm);
    if (d->qk_norm && (!(d->norm_eps >= 0.f) || !isfinite(d->norm_eps)))
        return fail(UAA_ERR_UNSUPPORTED, "norm_eps=%g is not a finite value >= 0", (double)d->norm_eps);
    if (d->window < 0) return fail(UAA_ERR_UNSUPPORTED, "window=%d is negative", d->window);
    if (d->first_tokens < 0) return fail(UAA_ERR_UNSUPPORTED, "first_tokens=%d is negative", d->first_tokens);
    if (!(d->softcap >= 0.f) || !isfinite(d->softcap))
        return fail(UAA_ERR_UNSUPPORTED, "softcap=%g is not a finite value >= 0", (double)d->softcap);
    if (d->has_sink != 0 && d->has_sink != 1)
        return fail(UAA_ERR_UNSUPPORTED, "has_sink=%d is not 0 or 1", d->has_sink);
    if (d->kv_dtype != UAA_DTYPE_F32 && d->kv_dtype != UAA_DTYPE_BF16 && d->kv_dtype != UAA_DTYPE_VQ8 &&
        d->kv_dtype != UAA_DTYPE_Q8 && d->kv_dtype != UAA_DTYPE_Q4)
        return fail(UAA_ERR_UNSUPPORTED, "kv_dtype=%d is not F32, BF16, VQ8, Q8 or Q4", d->kv_dtype);
    if (d->io_dtype != UAA_DTYPE_F32 && d->io_dtype != UAA_DTYPE_BF16)
        return fail(UAA_ERR_UNSUPPORTED, "io_dtype=%d is not F32 or BF16", d->io_dtype);
    if (d->out_dtype != UAA_DTYPE_F32 && d->out_dtype != UAA_DTYPE_BF16)
        return fail(UAA_ERR_UNSUPPORTED, "out_dtype=%d is not F32 or BF16", d->out_dtype);
    return UAA_OK;
}

// ---------------------------------------------------------------- split geometry

// Tokens per sequence one step takes at most (a prefill chunk).
constexpr int kMaxQLen = 1024;

// Workspace that a prefill chunk over a 4-bit cache takes for widened rows, at most
// (more only where one sequence needs it).
constexpr size_t kDenseBytes = (size_t)512 << 20;

struct Plan {
    int G;
    int q_len;           // tokens per sequence (1: decode)
    int kernel;          // 0 CUDA-core, 1 tensor-core
    int heads_per_cta;   // query rows of one unit ((token, head) pairs; heads for a decode step)
    int head_groups;     // units per kv head
    int n_head_tiles;    // 8-head column tiles of the tensor-core kernel
    int mg;              // 64-key tiles per ring stage
    int n_ctas;          // P: persistent CTAs of the partial kernel
    int slice;           // sequences per partial launch
    int n_slices;
    int per_sm;          // resident CTAs per SM
    int prefill;         // a contiguous or 4-bit cache takes the query-tiled prefill kernel (no combine)
    int dense_rows;      // 4-bit caches there: rows per (sequence, kv head) widened in the workspace,
    int dense_batch;     // for so many sequences at a time (0 rows: other caches)
    size_t off_status, off_counts, off_qrot, off_prefix, off_rec_lse, off_rec_o, off_ranges, off_owners, off_balance, off_dense, total;
    size_t prefix_stride, rec_lse_stride, rec_o_stride, ranges_stride, owners_stride;  // bytes per slice
};

int device_sm_count()
{
    static int cache[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    if (dev < 64 && cache[dev] > 0) return cache[dev];
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
    if (dev < 64) cache[dev] = n;
    return n;
}

// Range-balance state of the tensor-core kernel (BalanceState), at a fixed
// offset after the status word so that it survives changes of batch: header |
// claim[P] (uint64) | rate[P] | weight[P] | cumw[P + 1], each part 256-byte
// aligned.
size_t balance_bytes(int P)
{
    return 256 + align256((size_t)P * 8) + 2 * align256((size_t)P * 4) + align256(((size_t)P + 1) * 4);
}

uaa::BalanceState balance_of(void* ws, const Plan& pl)
{
    char* b = static_cast<char*>(ws) + pl.off_balance;
    const size_t P = (size_t)pl.n_ctas;
    uaa::BalanceState r;
    r.header = reinterpret_cast<unsigned*>(b);
    r.claim = reinterpret_cast<unsigned long long*>(b + 256);
    r.rate = reinterpret_cast<float*>(b + 256 + align256(P * 8));
    r.weight = reinterpret_cast<float*>(b + 256 + align256(P * 8) + align256(P * 4));
    r.cumw = reinterpret_cast<unsigned*>(b + 256 + align256(P * 8) + 2 * align256(P * 4));
    return r;
}

// Geometry of a step. The partial kernels are persistent: P = SMs x resident CTAs
// (4 for the CUDA-core kernel, 2 for the tensor-core kernel, 1 at head_dim 256 or
// with two column tiles),
// each attending one contiguous range of all units' key stages (the stream-K
// partition in internal.cuh), so the split needs no length bound. Batches above
// kMaxSliceBatch sequences are cut into slices (one partial + combine launch each)
// because a CTA keeps the slice's stage prefix in shared memory.
uaa_status make_plan(const uaa_attn_desc* d, int batch, int q_len, int max_len, int n_sm, Plan* pl)
{
    UAA_TRY(check_desc(d));
    if (batch < 0) return fail(UAA_ERR_INVALID_ARGUMENT, "batch=%d is negative", batch);
    if (max_len < 0) return fail(UAA_ERR_INVALID_ARGUMENT, "max_seq_len=%d is negative", max_len);
    if (n_sm <= 0) return fail(UAA_ERR_INVALID_ARGUMENT, "SM count %d is not positive", n_sm);
    if (q_len < 0 || q_len > kMaxQLen)
        return fail(UAA_ERR_UNSUPPORTED, "q_len=%d is not in [0, %d]", q_len, kMaxQLen);
    Plan p{};
    p.G = d->n_q_heads / d->n_kv_heads;
    p.q_len = q_len > 1 ? q_len : 1;
    p.kernel = d->kv_dtype == UAA_DTYPE_F32 ? 0 : 1;
    // a unit's query rows are the (token, head) pairs of one kv head: q_len G of them
    const int rows = p.q_len * p.G;
    if (p.kernel == 0 || d->head_dim == 256 || rows <= 8) {
        p.heads_per_cta = 8;
        p.n_head_tiles = 1;
    } else {
        p.heads_per_cta = 16;
        p.n_head_tiles = 2;
    }
    // a 4-bit cache's codes are widened once per unit: three tiles where they make fewer
    // units and their state fits two CTAs per SM (head_dim 64)
    if (d->kv_dtype == UAA_DTYPE_Q4 && d->head_dim == 64 && (rows + 23) / 24 < (rows + 15) / 16) {
        p.heads_per_cta = 24;
        p.n_head_tiles = 3;
    }
    p.head_groups = (rows + p.heads_per_cta - 1) / p.heads_per_cta;
    p.mg = p.kernel == 1 ? uaa::partial_tc_keys_per_stage(d->head_dim, d->kv_dtype, p.n_head_tiles) / uaa::kTileKeys : 1;
    p.per_sm = p.kernel == 0 ? 4 : uaa::partial_tc_ctas_per_sm(d->head_dim, d->kv_dtype, p.n_head_tiles);
    p.n_ctas = n_sm * p.per_sm;
    // long chunks on contiguous bf16 caches and on 4-bit caches: whole 128-row blocks of
    // (token, head) rows per CTA, each streaming its keys once (the partial kernel's units
    // hold 8 to 24 rows)
    p.prefill = p.kernel == 1 && (d->kv_dtype == UAA_DTYPE_BF16 || d->kv_dtype == UAA_DTYPE_Q4) &&
                (d->head_dim == 64 || d->head_dim == 128) && rows >= uaa::kPrefillRows;
    p.slice = batch < uaa::kMaxSliceBatch ? (batch > 0 ? batch : 1) : uaa::kMaxSliceBatch;
    p.n_slices = batch > 0 ? (batch + p.slice - 1) / p.slice : 0;

    const size_t B = (size_t)(batch > 0 ? batch : 0), Hq = d->n_q_heads, D = d->head_dim;
    const size_t HC = (size_t)p.heads_per_cta, P = (size_t)p.n_ctas;
    p.prefix_stride = align256(((size_t)p.slice + 1) * 4);
    p.rec_lse_stride = align256(2 * P * HC * 4);
    p.rec_o_stride = align256(2 * P * HC * D * 4);
    p.ranges_stride = align256((P + 1) * 8);
    p.owners_stride = align256((size_t)p.slice * d->n_kv_heads * p.head_groups * 8);
    p.off_status = 0;
    p.off_balance = 256;
    // The splits' counters of the fp32 one-launch step (one per unit, at most P of its
    // grid: f32_step_splits) are zero between launches, so no other geometry's arrays may
    // reach them: they and what lies before them have places that depend on n_sm alone.
    const int max_ctas = 4 * n_sm;
    p.off_counts = p.off_balance + balance_bytes(max_ctas);
    p.off_qrot = p.off_counts + align256((size_t)max_ctas * 4);
    p.off_prefix = p.off_qrot + align256(B * p.q_len * Hq * D * 4);
    p.off_rec_lse = p.off_prefix + p.n_slices * p.prefix_stride;
    p.off_rec_o = p.off_rec_lse + p.n_slices * p.rec_lse_stride;
    p.off_ranges = p.off_rec_o + p.n_slices * p.rec_o_stride;
    p.off_owners = p.off_ranges + p.n_slices * p.ranges_stride;
    p.total = p.off_owners + p.n_slices * p.owners_stride;
    if (p.prefill && d->kv_dtype == UAA_DTYPE_Q4) {
        // the visible rows of as many sequences as kDenseBytes hold (one at least),
        // widened to fp16: keys, then values
        const long long rows_max = 2147483647LL - 2 * uaa::kTileKeys;
        const long long per_head = ((long long)max_len + p.q_len + 63) / 64 * 64;
        if (per_head * d->n_kv_heads > rows_max)
            return fail(UAA_ERR_UNSUPPORTED, "(max_seq_len + q_len) * n_kv_heads=%lld exceeds 2^31 cache rows",
                        per_head * d->n_kv_heads);
        const size_t per_seq = (size_t)per_head * d->n_kv_heads * D * 4;
        const size_t whole = B * per_seq, limit = per_seq > kDenseBytes ? per_seq : kDenseBytes;
        const size_t dense = whole < limit ? whole : limit;
        long long nb = per_seq ? (long long)(dense / per_seq) : 0;
        const long long by_grid = 65535 / d->n_kv_heads, by_rows = rows_max / (per_head * d->n_kv_heads);
        if (nb > by_grid) nb = by_grid;
        if (nb > by_rows) nb = by_rows;
        if (B > 0 && nb < 1)
            return fail(UAA_ERR_UNSUPPORTED, "n_kv_heads=%d is above 65535 for a chunk over a 4-bit cache",
                        d->n_kv_heads);
        p.dense_rows = (int)per_head;
        p.dense_batch = (int)nb;
        p.off_dense = align256(p.total);
        p.total = p.off_dense + dense;
    }
    *pl = p;
    return UAA_OK;
}

// Bytes of a workspace that serves steps of q_len tokens and every shorter one: a
// shorter step may need more (24-row units over a 4-bit cache, where a longer one
// takes 16-row units). 0 on refused facts.
size_t workspace_bytes(const uaa_attn_desc* d, int batch, int q_len, int max_len, int n_sm)
{
    size_t bytes = 0;
    for (int t = q_len; t >= (q_len > 1 ? 1 : q_len); --t) {  // the longest first: its refusal is the caller's
        Plan pl{};
        if (make_plan(d, batch, t, max_len, n_sm, &pl) != UAA_OK) return 0;
        if (pl.total > bytes) bytes = pl.total;
    }
    return bytes;
}

// The facts of a step's caches: their geometry, and the pointers that hold them.
uaa_status check_cache_shape(const uaa_attn_desc* d, const uaa_step_args* a)
{
    // a ring stage that holds a sequence's last key reaches past it (two tiles; four over
    // a 4-bit cache), and positions are 32-bit
    const bool long_stage = d->kv_dtype == UAA_DTYPE_Q4 || d->first_tokens > 0;
    const long long rows_max = 2147483647LL - (long_stage ? 8 : 2) * uaa::kTileKeys;
    if (long_stage && a->cache_capacity > rows_max)
        return fail(UAA_ERR_UNSUPPORTED, "cache_capacity=%d is above %lld, the largest of a 4-bit cache or with first_tokens",
                    a->cache_capacity, rows_max);
    if (a->block_table) {
        const int ps = a->page_size;
        if (ps < 16 || ps > 4096 || (ps & (ps - 1)) != 0)
            return fail(UAA_ERR_UNSUPPORTED, "page_size=%d is not a power of two in [16, 4096]", ps);
        // a page's scales are one TMA box of a stage; its shared-memory destination
        // (4 bytes per key, or D / 16 for q4) must start on 128 bytes
        if (ps < 32 && d->kv_dtype != UAA_DTYPE_F32 && d->kv_dtype != UAA_DTYPE_BF16)
            return fail(UAA_ERR_UNSUPPORTED, "page_size=%d is below 32, the smallest page of a vq8 / q8 / q4 cache", ps);
        if (a->pages_per_seq <= 0 || (long long)a->pages_per_seq * ps != a->cache_capacity)
            return fail(UAA_ERR_INVALID_ARGUMENT,
                        "cache_capacity=%d is not pages_per_seq=%d x page_size=%d", a->cache_capacity,
                        a->pages_per_seq, ps);
        if (a->n_pages <= 0) return fail(UAA_ERR_INVALID_ARGUMENT, "n_pages=%d is not positive", a->n_pages);
        if ((long long)a->n_pages * d->n_kv_heads * ps > rows_max)
            return fail(UAA_ERR_UNSUPPORTED, "n_pages*n_kv_heads*page_size=%lld exceeds 2^31 cache rows",
                        (long long)a->n_pages * d->n_kv_heads * ps);
        if (!aligned16(a->block_table)) return fail(UAA_ERR_INVALID_ARGUMENT, "block_table is not 16-byte aligned");
    } else if ((long long)a->batch * d->n_kv_heads * a->cache_capacity > rows_max) {
        return fail(UAA_ERR_UNSUPPORTED, "batch*n_kv_heads*cache_capacity=%lld exceeds 2^31 cache rows",
                    (long long)a->batch * d->n_kv_heads * a->cache_capacity);
    }
    return UAA_OK;
}

bool scaled_values(const uaa_attn_desc* d)
{
    return d->kv_dtype == UAA_DTYPE_VQ8 || d->kv_dtype == UAA_DTYPE_Q8 || d->kv_dtype == UAA_DTYPE_Q4;
}

bool scaled_keys(const uaa_attn_desc* d) { return d->kv_dtype == UAA_DTYPE_Q8 || d->kv_dtype == UAA_DTYPE_Q4; }

// A call that only reads the caches (uaa_cache_read).
uaa_status check_cache(const uaa_attn_desc* d, const uaa_step_args* a)
{
    if (!a) return fail(UAA_ERR_INVALID_ARGUMENT, "args is NULL");
    if (a->batch < 0) return fail(UAA_ERR_INVALID_ARGUMENT, "batch=%d is negative", a->batch);
    if (a->cache_capacity <= 0 || a->cache_capacity % 4 != 0)
        return fail(UAA_ERR_INVALID_ARGUMENT, "cache_capacity=%d is not a positive multiple of 4", a->cache_capacity);
    UAA_TRY(check_cache_shape(d, a));
    const struct {
        const void* p;
        const char* name;
        bool needed;
    } ptrs[] = {{a->k_cache, "k_cache", true},
                {a->v_cache, "v_cache", true},
                {a->v_scale, "v_scale", scaled_values(d)},
                {a->k_scale, "k_scale", scaled_keys(d)}};
    for (auto& e : ptrs) {
        if (e.needed && !e.p && a->batch > 0) return fail(UAA_ERR_INVALID_ARGUMENT, "%s is NULL", e.name);
        if (e.p && !aligned16(e.p)) return fail(UAA_ERR_INVALID_ARGUMENT, "%s is not 16-byte aligned", e.name);
    }
    return UAA_OK;
}

uaa_status check_args(const uaa_attn_desc* d, const uaa_step_args* a, const uaa_workspace* ws, bool need_io)
{
    if (!a) return fail(UAA_ERR_INVALID_ARGUMENT, "args is NULL");
    if (!ws || !ws->ptr) return fail(UAA_ERR_INVALID_ARGUMENT, "workspace is NULL");
    if (!aligned16(ws->ptr)) return fail(UAA_ERR_INVALID_ARGUMENT, "workspace is not 16-byte aligned");
    if (a->batch < 0) return fail(UAA_ERR_INVALID_ARGUMENT, "batch=%d is negative", a->batch);
    if (a->max_seq_len < 0) return fail(UAA_ERR_INVALID_ARGUMENT, "max_seq_len=%d is negative", a->max_seq_len);
    if (a->cache_capacity <= 0 || a->cache_capacity % 4 != 0)
        return fail(UAA_ERR_INVALID_ARGUMENT, "cache_capacity=%d is not a positive multiple of 4",
                    a->cache_capacity);
    const int q_len = a->q_len > 1 ? a->q_len : 1;
    if ((long long)a->max_seq_len + q_len > a->cache_capacity)
        return fail(UAA_ERR_CAPACITY, "max_seq_len=%d + %d new token(s) does not fit cache_capacity=%d",
                    a->max_seq_len, q_len, a->cache_capacity);
    UAA_TRY(check_cache_shape(d, a));
    struct {
        const void* p;
        const char* name;
        bool needed;
    } ptrs[] = {
        {a->q, "q", need_io},
        {a->k_new, "k_new", need_io},
        {a->v_new, "v_new", need_io},
        {a->k_cache, "k_cache", true},
        {a->v_cache, "v_cache", true},
        {a->seq_lens, "seq_lens", true},
        {a->out, "out", true},
        {a->v_scale, "v_scale", scaled_values(d)},
        {a->k_scale, "k_scale", scaled_keys(d)},
        {a->q_norm_w, "q_norm_w", need_io && d->qk_norm},
        {a->k_norm_w, "k_norm_w", need_io && d->qk_norm},
        {a->sink, "sink", d->has_sink != 0},
    };
    for (auto& e : ptrs) {
        if (e.needed && !e.p && a->batch > 0)  // a batch of 0 reads and writes nothing
            return fail(d->has_sink && !strcmp(e.name, "sink") ? UAA_ERR_UNSUPPORTED : UAA_ERR_INVALID_ARGUMENT,
                        "%s is NULL%s", e.name,
                        !strcmp(e.name, "sink") ? " while has_sink=1" : "");
        if (e.p && !aligned16(e.p)) return fail(UAA_ERR_INVALID_ARGUMENT, "%s is not 16-byte aligned", e.name);
    }
    if (a->q_rot && !aligned16(a->q_rot)) return fail(UAA_ERR_INVALID_ARGUMENT, "q_rot is not 16-byte aligned");
    return UAA_OK;
}

// The partial kernels count a slice's key stages over all its units in 32 bits.
uaa_status check_stages(const uaa_attn_desc* d, const uaa_step_args* a, const Plan& pl)
{
    if (pl.prefill && (!a->block_table || pl.dense_rows > 0)) return UAA_OK;  // not theirs (takes_prefill)
    long long keys = (long long)a->max_seq_len + pl.q_len;
    if (d->window > 0) {  // two runs, each with a stage more where it starts inside one
        const long long seen = (long long)d->window + pl.q_len - 1 + d->first_tokens;
        keys = keys < seen ? keys : seen;
    }
    const long long stages = keys / (uaa::kTileKeys * pl.mg) + 3;
    const double all = (double)stages * pl.slice * d->n_kv_heads * pl.head_groups;
    if (a->batch > 0 && all > 2147483647.0)
        return fail(UAA_ERR_UNSUPPORTED,
                    "max_seq_len=%d, q_len=%d: %.3g key stages over %d sequences exceed 2^31 (split the batch or the tokens)",
                    a->max_seq_len, pl.q_len, all, pl.slice);
    return UAA_OK;
}

uaa_status prepare(const uaa_attn_desc* d, const uaa_step_args* a, const uaa_workspace* ws, bool need_io,
                   Plan* pl)
{
    UAA_TRY(check_desc(d));
    UAA_TRY(check_args(d, a, ws, need_io));
    const int n_sm = device_sm_count();
    UAA_TRY(make_plan(d, a->batch, a->q_len, a->max_seq_len, n_sm > 0 ? n_sm : 1, pl));
    UAA_TRY(check_stages(d, a, *pl));
    if (n_sm <= 0) return fail(UAA_ERR_CUDA, "no CUDA device: the SM count query failed");
    if (ws->bytes < pl->total)
        return fail(UAA_ERR_INVALID_ARGUMENT, "workspace has %zu bytes, the step needs %zu", ws->bytes,
                    pl->total);
    return UAA_OK;
}

// The partition covers the union of the rows' windows: the first token's window
// starts q_len - 1 keys before the last one's. A window that no position reaches
// (2^31 keys with the chunk) is none.
int partition_window(const uaa_attn_desc* d, const Plan& pl)
{
    const long long w = (long long)d->window + pl.q_len - 1;
    return d->window > 0 && w <= 2147483647LL ? (int)w : 0;
}

// The keys that stay visible behind the window; without a window every key is.
int first_tokens(const uaa_attn_desc* d) { return d->window > 0 ? d->first_tokens : 0; }

float softmax_scale(const uaa_attn_desc* d)
{
    return d->scale > 0.f ? d->scale : 1.0f / sqrtf((float)d->head_dim);
}

// The prescale of the rotated q rows: logits come out in the log2 domain
// (scale log2 e), or as s / c when a softcap c applies tanh to them first.
// The paging of a step's caches (KvPages in internal.cuh).
uaa::KvPages pages_of(const uaa_step_args* a)
{
    uaa::KvPages pg{};
    if (a->block_table) {
        pg.table = a->block_table;
        int shift = 0;
        while ((1 << shift) < a->page_size) ++shift;
        pg.shift = shift;
        pg.per_seq = a->pages_per_seq;
        pg.n_pages = a->n_pages;
    }
    return pg;
}

float qscale(const uaa_attn_desc* d)
{
    const float scale = softmax_scale(d);
    return d->softcap > 0.f ? scale / d->softcap : scale * uaa::kLog2e;
}

// Rotary frequencies theta'_p / pi in fp64 and the cos/sin multiplier: plain
// base^(-2p/R) over the R rotated dims; llama3 wavelength interpolation; YaRN
// ramp over the pair index between the pairs whose wavelength fits beta_fast /
// beta_slow times into the original context; linear division by the factor
// (huggingface_decoder_completeness.md, P0.2 and P1.5; YaRN as published).
// Entries of pairs beyond R/2 stay 0 (those pairs are not rotated).
int rotary_dims(const uaa_attn_desc* d) { return d->rotary_dim > 0 ? d->rotary_dim : d->head_dim; }

void make_rope_table(const uaa_attn_desc* d, double* inv_freq_over_pi, double* mscale)
{
    const int D = rotary_dims(d);
    for (int i = 0; i < d->head_dim / 2; ++i) inv_freq_over_pi[i] = 0.0;
    const double pi = 3.14159265358979323846;
    const uaa_rope_params& r = d->rope;
    double ms = 1.0;
    double lo = 0.0, hi = 0.0;
    if (r.scaling == UAA_ROPE_SCALING_YARN) {
        const double ln_base = log(r.theta);
        lo = D * log(r.original_max_pos / (2.0 * pi * r.beta_fast)) / (2.0 * ln_base);
        hi = D * log(r.original_max_pos / (2.0 * pi * r.beta_slow)) / (2.0 * ln_base);
        ms = r.attn_factor > 0.0 ? r.attn_factor : (r.factor > 1.0 ? 1.0 + 0.1 * log(r.factor) : 1.0);
    }
    for (int i = 0; i < D / 2; ++i) {
        const double f = pow(r.theta, -(2.0 * i) / D);
        double g = f;
        if (r.scaling == UAA_ROPE_SCALING_LLAMA3) {
            const double wl = 2.0 * pi / f;
            const double wl_keep = r.original_max_pos / r.high_freq_factor;
            const double wl_div = r.original_max_pos / r.low_freq_factor;
            if (wl > wl_div) {
                g = f / r.factor;
            } else if (wl >= wl_keep) {
                const double t = (r.original_max_pos / wl - r.low_freq_factor) /
                                 (r.high_freq_factor - r.low_freq_factor);
                g = t * f + (1.0 - t) * f / r.factor;
            }
        } else if (r.scaling == UAA_ROPE_SCALING_YARN) {
            double ramp = hi > lo ? (i - lo) / (hi - lo) : (i >= lo ? 1.0 : 0.0);
            ramp = ramp < 0.0 ? 0.0 : (ramp > 1.0 ? 1.0 : ramp);
            g = ramp * (f / r.factor) + (1.0 - ramp) * f;
        } else if (r.scaling == UAA_ROPE_SCALING_LINEAR) {
            g = f / r.factor;
        }
        inv_freq_over_pi[i] = g / pi;
    }
    *mscale = ms;
}

// The table of the descriptor, kept from the thread's last call with the same rotary
// facts (64 pow take longer than a launch).
void rope_table(const uaa_attn_desc* d, double* inv_freq_over_pi, float* mscale, double* mscale64 = nullptr)
{
    struct Kept {
        bool valid;
        int head_dim, rotary_dim;
        uaa_rope_params rope;
        double table[uaa::kMaxHeadDim / 2], mscale;
    };
    static thread_local Kept k = {};
    const uaa_rope_params &a = k.rope, &b = d->rope;
    if (!k.valid || k.head_dim != d->head_dim || k.rotary_dim != d->rotary_dim || a.theta != b.theta ||
        a.scaling != b.scaling || a.factor != b.factor || a.low_freq_factor != b.low_freq_factor ||
        a.high_freq_factor != b.high_freq_factor || a.original_max_pos != b.original_max_pos ||
        a.beta_fast != b.beta_fast || a.beta_slow != b.beta_slow || a.attn_factor != b.attn_factor) {
        make_rope_table(d, k.table, &k.mscale);
        k.head_dim = d->head_dim;
        k.rotary_dim = d->rotary_dim;
        k.rope = d->rope;
        k.valid = true;
    }
    memcpy(inv_freq_over_pi, k.table, sizeof(double) * (d->head_dim / 2));
    *mscale = (float)k.mscale;
    if (mscale64) *mscale64 = k.mscale;
}

// ---------------------------------------------------------------- TMA descriptors

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

uaa_status encode_2d(CUtensorMap* tm, CUtensorMapDataType dt, void* ptr, uint64_t inner, uint64_t rows,
                     uint64_t row_bytes, uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle sw,
                     const char* what)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return fail(UAA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t dims[2] = {inner, rows};
    const cuuint64_t strides[1] = {row_bytes};
    const cuuint32_t box[2] = {box_inner, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(tm, dt, 2, ptr, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(UAA_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed with %d", what, (int)r);
    return UAA_OK;
}

// ---------------------------------------------------------------- the three launches

uaa_status run_append(const uaa_attn_desc* d, const uaa_step_args* a, const uaa_workspace* ws, const Plan& pl,
                      cudaStream_t s)
{
    if (a->batch == 0) return UAA_OK;
    uaa::AppendParams p{};
    p.B = a->batch;
    p.Hq = d->n_q_heads;
    p.Hkv = d->n_kv_heads;
    p.D = d->head_dim;
    p.q_len = pl.q_len;
    {  // tokens per CTA: one for short steps (parallelism), up to 16 once the grid has ~4 CTAs per SM anyway
        const int n_sm = device_sm_count();
        const long long tokens = (long long)a->batch * pl.q_len;
        long long tpc = n_sm > 0 ? tokens / (4LL * n_sm) : 1;
        p.tokens_per_cta = (int)(tpc < 1 ? 1 : (tpc > 16 ? 16 : tpc));
    }
    p.cap = a->cache_capacity;
    p.max_len = a->max_seq_len;
    p.style = d->rope.style;
    p.half_rot = rotary_dims(d) / 2;
    p.qk_norm = d->qk_norm;
    p.eps = d->norm_eps;
    p.norm_offset = d->norm_offset ? 1.f : 0.f;
    p.qscale = qscale(d);
    p.io_dtype = d->io_dtype;
    p.kv_dtype = d->kv_dtype;
    p.q = a->q;
    p.k_new = a->k_new;
    p.v_new = a->v_new;
    p.q_norm_w = a->q_norm_w;
    p.k_norm_w = a->k_norm_w;
    p.k_cache = a->k_cache;
    p.v_cache = a->v_cache;
    p.v_scale = a->v_scale;
    p.k_scale = a->k_scale;
    p.pages = pages_of(a);
    p.seq_lens = a->seq_lens;
    char* w = static_cast<char*>(ws->ptr);
    p.q_prime = reinterpret_cast<float*>(w + pl.off_qrot);
    p.q_rot_out = a->q_rot;
    p.status = reinterpret_cast<unsigned*>(w + pl.off_status);
    rope_table(d, p.inv_freq_over_pi, &p.mscale, &p.mscale64);
    const cudaError_t e = uaa::launch_append(p, s);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "append kernel launch");
}

// The query-tiled prefill kernel takes step 2 of this call (and step 3 has nothing to do).
bool takes_prefill(const uaa_step_args* a, const Plan& pl)
{
    return pl.prefill && (!a->block_table || pl.dense_rows > 0);
}

// A prefill chunk over a 4-bit cache: the rows that it sees widened to fp16, then the
// prefill kernel on them, as many sequences at a time as the workspace holds.
uaa_status run_prefill_q4(const uaa_attn_desc* d, const uaa_step_args* a, const uaa_workspace* ws, const Plan& pl,
                          cudaStream_t s)
{
    char* w = static_cast<char*>(ws->ptr);
    const uint64_t D = d->head_dim;
    const size_t q_rows = (size_t)pl.q_len * d->n_q_heads * D;
    const size_t out_elem = d->out_dtype == UAA_DTYPE_F32 ? 4 : 2;
    for (int b0 = 0; b0 < a->batch; b0 += pl.dense_batch) {
        const int nb = a->batch - b0 < pl.dense_batch ? a->batch - b0 : pl.dense_batch;
        const uint64_t rows = (uint64_t)nb * d->n_kv_heads * pl.dense_rows;
        uaa::WidenParams wp{};
        wp.B = nb;
        wp.Hkv = d->n_kv_heads;
        wp.D = d->head_dim;
        wp.cap = a->cache_capacity;
        wp.row_cap = pl.dense_rows;
        wp.b_off = b0;
        wp.q_len = pl.q_len;
        wp.window = partition_window(d, pl);
        wp.first_tokens = first_tokens(d);
        wp.seq_lens = a->seq_lens + b0;
        wp.k_cache = a->k_cache;
        wp.v_cache = a->v_cache;
        wp.k_scale = a->k_scale;
        wp.v_scale = a->v_scale;
        wp.pages = pages_of(a);
        if (!a->block_table) wp.pages.table = nullptr;
        wp.k_out = w + pl.off_dense;
        wp.v_out = w + pl.off_dense + rows * D * 2;
        wp.status = reinterpret_cast<unsigned*>(w + pl.off_status);
        cudaError_t e = uaa::launch_widen_q4(wp, s);
        if (e != cudaSuccess) return cuda_fail(e, "4-bit widening kernel launch");
        CUtensorMap tk, tv;
        UAA_TRY(encode_2d(&tk, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, wp.k_out, D, rows, D * 2, 64,
                          (uint32_t)uaa::kPrefillKeys, CU_TENSOR_MAP_SWIZZLE_128B, "widened keys"));
        UAA_TRY(encode_2d(&tv, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, wp.v_out, D, rows, D * 2, 64,
                          (uint32_t)uaa::kPrefillKeys, CU_TENSOR_MAP_SWIZZLE_128B, "widened values"));
        uaa::PrefillParams p{};
        p.B = nb;
        p.Hq = d->n_q_heads;
        p.Hkv = d->n_kv_heads;
        p.D = d->head_dim;
        p.G = pl.G;
        p.q_len = pl.q_len;
        p.cap = a->cache_capacity;
        p.row_cap = pl.dense_rows;
        p.window = d->window;
        p.first_tokens = first_tokens(d);
        p.softcap_log2e = d->softcap > 0.f ? d->softcap * uaa::kLog2e : 0.f;
        p.q_prime = reinterpret_cast<const float*>(w + pl.off_qrot) + b0 * q_rows;
        p.seq_lens = a->seq_lens + b0;
        p.sink = d->has_sink ? a->sink : nullptr;
        p.out = static_cast<char*>(a->out) + b0 * q_rows * out_elem;
        p.out_dtype = d->out_dtype;
        p.status = reinterpret_cast<unsigned*>(w + pl.off_status);
        e = uaa::launch_prefill_umma(p, tk, tv, s);
        if (e != cudaSuccess) return cuda_fail(e, "prefill kernel launch");
    }
    return UAA_OK;
}

uaa_status run_prefill(const uaa_attn_desc* d, const uaa_step_args* a, const uaa_workspace* ws, const Plan& pl,
                       cudaStream_t s)
{
    char* w = static_cast<char*>(ws->ptr);
    const uint64_t D = d->head_dim;
    if (pl.dense_rows > 0) return run_prefill_q4(d, a, ws, pl, s);
    const uint64_t rows = (uint64_t)a->batch * d->n_kv_heads * a->cache_capacity;
    CUtensorMap tk, tv;
    UAA_TRY(encode_2d(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a->k_cache, D, rows, D * 2, 64,
                      (uint32_t)uaa::kPrefillKeys, CU_TENSOR_MAP_SWIZZLE_128B, "k_cache"));
    UAA_TRY(encode_2d(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a->v_cache, D, rows, D * 2, 64,
                      (uint32_t)uaa::kPrefillKeys, CU_TENSOR_MAP_SWIZZLE_128B, "v_cache"));
    uaa::PrefillParams p{};
    p.B = a->batch;
    p.Hq = d->n_q_heads;
    p.Hkv = d->n_kv_heads;
    p.D = d->head_dim;
    p.G = pl.G;
    p.q_len = pl.q_len;
    p.cap = a->cache_capacity;
    p.window = d->window;
    p.first_tokens = first_tokens(d);
    p.softcap_log2e = d->softcap > 0.f ? d->softcap * uaa::kLog2e : 0.f;
    p.q_prime = reinterpret_cast<const float*>(w + pl.off_qrot);
    p.seq_lens = a->seq_lens;
    p.sink = d->has_sink ? a->sink : nullptr;
    p.out = a->out;
    p.out_dtype = d->out_dtype;
    p.status = reinterpret_cast<unsigned*>(w + pl.off_status);
    const cudaError_t e = uaa::launch_prefill_umma(p, tk, tv, s);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "prefill kernel launch");
}

// The tensor maps of the tensor-core partial kernel over a step's caches.
uaa_status partial_maps(const uaa_attn_desc* d, const uaa_step_args* a, int n_head_tiles, uaa::PartialMaps* maps)
{
    const size_t D = d->head_dim;
    // contiguous caches: one box of a whole stage per row kind (and a second set of
    // 64-key boxes for units' partial last stages); paged caches: the pools, and one
    // box per page-aligned sub-tile of min(64, page_size) keys
    const bool paged = a->block_table != nullptr;
    const uint64_t rows = paged ? (uint64_t)a->n_pages * d->n_kv_heads * a->page_size
                                : (uint64_t)a->batch * d->n_kv_heads * a->cache_capacity;
    const uint32_t tk_rows =
        paged ? (uint32_t)(a->page_size < uaa::kTileKeys ? a->page_size : uaa::kTileKeys)
              : (uint32_t)uaa::partial_tc_keys_per_stage(d->head_dim, d->kv_dtype, n_head_tiles);  // box height
    const uint64_t heads = paged ? (uint64_t)a->n_pages * d->n_kv_heads : (uint64_t)a->batch * d->n_kv_heads;
    const uint64_t scale_inner = paged ? (uint64_t)a->page_size : (uint64_t)a->cache_capacity;
    // int8 codes: boxes of box_rows x min(D, 128) bytes, swizzled like the bf16 boxes so
    // the kernel's ldmatrix reads on them are free of bank conflicts; scales: one
    // box_rows-float box per stage
    const uint32_t code_box = D > 128 ? 128u : (uint32_t)D;
    const CUtensorMapSwizzle code_sw = D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    auto encode_set = [&](uint32_t box_rows, CUtensorMap& tk, CUtensorMap& tv, CUtensorMap& ts,
                          CUtensorMap& tks) -> uaa_status {
        if (d->kv_dtype == UAA_DTYPE_Q4) {
            // rows of D / 2 code bytes in one box each; a key's D / 32 fp16 scales as one
            // element of 4 or 8 bytes (two of 8 at head_dim 256)
            const CUtensorMapSwizzle sw = D == 64    ? CU_TENSOR_MAP_SWIZZLE_32B
                                          : D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                     : CU_TENSOR_MAP_SWIZZLE_128B;
            const CUtensorMapDataType st = D == 64 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_FLOAT64;
            const uint64_t per_key = D == 256 ? 2 : 1, row = scale_inner * (D / 16);
            UAA_TRY(encode_2d(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, a->k_cache, D / 2, rows, D / 2, (uint32_t)D / 2,
                              box_rows, sw, "k_cache 4-bit codes"));
            UAA_TRY(encode_2d(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, a->v_cache, D / 2, rows, D / 2, (uint32_t)D / 2,
                              box_rows, sw, "v_cache 4-bit codes"));
            UAA_TRY(encode_2d(&tks, st, a->k_scale, scale_inner * per_key, heads, row, box_rows * (uint32_t)per_key,
                              1, CU_TENSOR_MAP_SWIZZLE_NONE, "k_scale"));
            return encode_2d(&ts, st, a->v_scale, scale_inner * per_key, heads, row, box_rows * (uint32_t)per_key, 1,
                             CU_TENSOR_MAP_SWIZZLE_NONE, "v_scale");
        }
        if (d->kv_dtype == UAA_DTYPE_Q8) {
            UAA_TRY(encode_2d(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, a->k_cache, D, rows, D, code_box, box_rows,
                              code_sw, "k_cache codes"));
            UAA_TRY(encode_2d(&tks, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a->k_scale, scale_inner, heads,
                              scale_inner * 4, box_rows, 1, CU_TENSOR_MAP_SWIZZLE_NONE, "k_scale"));
        } else {
            UAA_TRY(encode_2d(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a->k_cache, D, rows, D * 2, 64, box_rows,
                              CU_TENSOR_MAP_SWIZZLE_128B, "k_cache"));
        }
        if (d->kv_dtype == UAA_DTYPE_VQ8 || d->kv_dtype == UAA_DTYPE_Q8) {
            UAA_TRY(encode_2d(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, a->v_cache, D, rows, D, code_box, box_rows,
                              code_sw, "v_cache codes"));
            UAA_TRY(encode_2d(&ts, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a->v_scale, scale_inner, heads,
                              scale_inner * 4, box_rows, 1, CU_TENSOR_MAP_SWIZZLE_NONE, "v_scale"));
        } else {
            UAA_TRY(encode_2d(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a->v_cache, D, rows, D * 2, 64, box_rows,
                              CU_TENSOR_MAP_SWIZZLE_128B, "v_cache"));
            ts = tv;  // unused by the bf16 kernel
        }
        if (d->kv_dtype != UAA_DTYPE_Q8) tks = ts;  // unused without key codes
        return UAA_OK;
    };
    UAA_TRY(encode_set(tk_rows, maps->k, maps->v, maps->s, maps->ks));
    if (!paged && tk_rows > (uint32_t)uaa::kTileKeys) {
        UAA_TRY(encode_set((uint32_t)uaa::kTileKeys, maps->kt, maps->vt, maps->st, maps->kst));
    } else {  // never used: every stage is one 64-key tile, or the pool boxes are sub-tiles already
        maps->kt = maps->k;
        maps->vt = maps->v;
        maps->st = maps->s;
        maps->kst = maps->ks;
    }
    return UAA_OK;
}

// fused: the tensor-core kernel also performs the append (steps 1 and 2 in one launch).
uaa_status run_partial(const uaa_attn_desc* d, const uaa_step_args* a, const uaa_workspace* ws, const Plan& pl,
                       cudaStream_t s, bool fused = false)
{
    if (a->batch == 0) return UAA_OK;
    if (takes_prefill(a, pl)) return run_prefill(d, a, ws, pl, s);
    char* w = static_cast<char*>(ws->ptr);
    const size_t D = d->head_dim, Hq = d->n_q_heads;
    const size_t out_elem = d->out_dtype == UAA_DTYPE_F32 ? 4 : 2;
    uaa::PartialMaps maps{};
    if (pl.kernel == 1) UAA_TRY(partial_maps(d, a, pl.n_head_tiles, &maps));
    for (int sl = 0; sl < pl.n_slices; ++sl) {
        const int b0 = sl * pl.slice;
        const int nb = a->batch - b0 < pl.slice ? a->batch - b0 : pl.slice;
        uaa::PartialParams p{};
        p.B = nb;
        p.Hq = d->n_q_heads;
        p.Hkv = d->n_kv_heads;
        p.D = d->head_dim;
        p.G = pl.G;
        p.b_off = b0;
        p.heads_per_cta = pl.heads_per_cta;
        p.head_groups = pl.head_groups;
        p.cap = a->cache_capacity;
        p.q_len = pl.q_len;
        p.attn_window = d->window;
        p.window = partition_window(d, pl);
        p.first_tokens = first_tokens(d);
        p.mg = pl.mg;
        p.softcap_log2e = d->softcap > 0.f ? d->softcap * uaa::kLog2e : 0.f;
        p.q_prime = reinterpret_cast<const float*>(w + pl.off_qrot) + (size_t)b0 * pl.q_len * Hq * D;
        p.k_cache = a->k_cache;
        p.v_cache = a->v_cache;
        p.v_scale = a->v_scale;
        p.k_scale = a->k_scale;
        p.pages = pages_of(a);
        p.seq_lens = a->seq_lens + b0;
        p.prefix = reinterpret_cast<int*>(w + pl.off_prefix + sl * pl.prefix_stride);
        p.ranges = reinterpret_cast<long long*>(w + pl.off_ranges + sl * pl.ranges_stride);
        p.owners = reinterpret_cast<unsigned*>(w + pl.off_owners + sl * pl.owners_stride);
        if (pl.kernel == 1) {
            p.bal = balance_of(w, pl);
            p.slice = sl;
            p.per_sm = pl.per_sm;
            p.uniform = d->reproducible;
        }
        p.rec_lse = reinterpret_cast<float*>(w + pl.off_rec_lse + sl * pl.rec_lse_stride);
        p.rec_o = reinterpret_cast<float*>(w + pl.off_rec_o + sl * pl.rec_o_stride);
        p.sink = d->has_sink ? a->sink : nullptr;
        p.out = static_cast<char*>(a->out) + (size_t)b0 * pl.q_len * Hq * D * out_elem;
        p.out_dtype = d->out_dtype;
        p.status = reinterpret_cast<unsigned*>(w + pl.off_status);
        if (fused) {
            const size_t io_elem = d->io_dtype == UAA_DTYPE_F32 ? 4 : 2;
            const size_t Hkv = d->n_kv_heads;
            p.fused = 1;
            p.max_len = a->max_seq_len;
            p.arrivals = reinterpret_cast<unsigned*>(w + pl.off_status) + 1;
            p.q = static_cast<const char*>(a->q) + (size_t)b0 * Hq * D * io_elem;  // one token per sequence
            p.k_new = static_cast<const char*>(a->k_new) + (size_t)b0 * Hkv * D * io_elem;
            p.v_new = static_cast<const char*>(a->v_new) + (size_t)b0 * Hkv * D * io_elem;
            p.io_dtype = d->io_dtype;
            p.kv_dtype = d->kv_dtype;
            p.style = d->rope.style;
            p.half_rot = rotary_dims(d) / 2;
            p.qk_norm = d->qk_norm;
            p.eps = d->norm_eps;
            p.norm_offset = d->norm_offset ? 1.f : 0.f;
            p.qscale = qscale(d);
            p.q_norm_w = a->q_norm_w;
            p.k_norm_w = a->k_norm_w;
            p.q_rot_out = a->q_rot ? a->q_rot + (size_t)b0 * Hq * D : nullptr;
            rope_table(d, p.inv_freq_over_pi, &p.mscale, &p.mscale64);
        }
        const cudaError_t e = pl.kernel == 0
                                  ? uaa::launch_partial_simt(p, pl.n_ctas, s)
                                  : uaa::launch_partial_tc(p, maps, d->kv_dtype, pl.n_head_tiles, pl.n_ctas, s);
        if (e != cudaSuccess) return cuda_fail(e, "partial kernel launch");
    }
    return UAA_OK;
}

uaa_status run_combine(const uaa_attn_desc* d, const uaa_step_args* a, const uaa_workspace* ws, const Plan& pl,
                       cudaStream_t s)
{
    if (a->batch == 0) return UAA_OK;
    if (takes_prefill(a, pl)) return UAA_OK;  // the prefill kernel wrote the output rows
    char* w = static_cast<char*>(ws->ptr);
    const size_t D = d->head_dim, Hq = d->n_q_heads;
    const size_t out_elem = d->out_dtype == UAA_DTYPE_F32 ? 4 : 2;
    for (int sl = 0; sl < pl.n_slices; ++sl) {
        const int b0 = sl * pl.slice;
        const int nb = a->batch - b0 < pl.slice ? a->batch - b0 : pl.slice;
        uaa::CombineParams p{};
        p.B = nb;
        p.Hq = d->n_q_heads;
        p.Hkv = d->n_kv_heads;
        p.D = d->head_dim;
        p.G = pl.G;
        p.heads_per_cta = pl.heads_per_cta;
        p.head_groups = pl.head_groups;
        p.q_len = pl.q_len;
        p.window = partition_window(d, pl);
        p.mg = pl.mg;
        p.P = pl.n_ctas;
        p.out_dtype = d->out_dtype;
        p.sink = d->has_sink ? a->sink : nullptr;
        p.seq_lens = a->seq_lens + b0;
        p.prefix = reinterpret_cast<const int*>(w + pl.off_prefix + sl * pl.prefix_stride);
        p.ranges = reinterpret_cast<const long long*>(w + pl.off_ranges + sl * pl.ranges_stride);
        p.owners = reinterpret_cast<unsigned*>(w + pl.off_owners + sl * pl.owners_stride);
        if (pl.kernel == 1) p.bal = balance_of(w, pl);
        p.rec_lse = reinterpret_cast<const float*>(w + pl.off_rec_lse + sl * pl.rec_lse_stride);
        p.rec_o = reinterpret_cast<const float*>(w + pl.off_rec_o + sl * pl.rec_o_stride);
        p.out = static_cast<char*>(a->out) + (size_t)b0 * pl.q_len * Hq * D * out_elem;
        p.status = reinterpret_cast<unsigned*>(w + pl.off_status);
        const cudaError_t e = uaa::launch_combine(p, s);
        if (e != cudaSuccess) return cuda_fail(e, "combine kernel launch");
    }
    return UAA_OK;
}

// The whole step: the fp32 one-launch kernel where it applies, else steps 1 and
// 2 (fused for the tensor-core kernel) and the combine.
uaa_status run_step(const uaa_attn_desc* d, const uaa_step_args* a, const uaa_workspace* ws, const Plan& pl,
                    cudaStream_t s);

// Keys per split of the fp32 one-launch step.
constexpr int kF32SplitKeys = 512;

// Splits per unit of the fp32 one-launch step (step_f32.cu), or 0 when the step
// takes the three-kernel path: it serves fp32 caches with one token per
// sequence in a single batch slice whose split records fit the slice's 2P.
int f32_step_splits(const uaa_attn_desc* d, const uaa_step_args* a, const Plan& pl)
{
    if (pl.kernel != 0 || pl.q_len != 1 || pl.n_slices != 1) return 0;
    const long long S = ((long long)a->max_seq_len + kF32SplitKeys) / kF32SplitKeys;  // keys: max_seq_len + 1
    const long long recs = (long long)a->batch * d->n_kv_heads * pl.head_groups * S;
    if (S > 1 && recs > 2LL * pl.n_ctas) return 0;
    return (int)S;
}

uaa_status run_step_f32(const uaa_attn_desc* d, const uaa_step_args* a, const uaa_workspace* ws, const Plan& pl,
                        int splits, cudaStream_t s)
{
    if (a->batch == 0) return UAA_OK;
    char* w = static_cast<char*>(ws->ptr);
    uaa::StepF32Params p{};
    p.B = a->batch;
    p.Hq = d->n_q_heads;
    p.Hkv = d->n_kv_heads;
    p.D = d->head_dim;
    p.G = pl.G;
    p.head_groups = pl.head_groups;
    p.cap = a->cache_capacity;
    p.max_len = a->max_seq_len;
    p.window = d->window;
    p.first_tokens = first_tokens(d);
    p.splits = splits;
    p.split_keys = kF32SplitKeys;
    p.style = d->rope.style;
    p.half_rot = rotary_dims(d) / 2;
    p.qk_norm = d->qk_norm;
    p.eps = d->norm_eps;
    p.norm_offset = d->norm_offset ? 1.f : 0.f;
    p.qscale = qscale(d);
    p.softcap_log2e = d->softcap > 0.f ? d->softcap * uaa::kLog2e : 0.f;
    p.io_dtype = d->io_dtype;
    p.out_dtype = d->out_dtype;
    p.q = a->q;
    p.k_new = a->k_new;
    p.v_new = a->v_new;
    p.q_norm_w = a->q_norm_w;
    p.k_norm_w = a->k_norm_w;
    p.sink = d->has_sink ? a->sink : nullptr;
    p.k_cache = static_cast<float*>(a->k_cache);
    p.v_cache = static_cast<float*>(a->v_cache);
    p.pages = pages_of(a);
    p.seq_lens = a->seq_lens;
    p.out = a->out;
    p.q_rot_out = a->q_rot;
    p.rec_o = reinterpret_cast<float*>(w + pl.off_rec_o);
    p.rec_lse = reinterpret_cast<float*>(w + pl.off_rec_lse);
    p.unit_count = reinterpret_cast<unsigned*>(w + pl.off_counts);
    p.arrivals = reinterpret_cast<unsigned*>(w + pl.off_status) + 1;
    p.status = reinterpret_cast<unsigned*>(w + pl.off_status);
    rope_table(d, p.inv_freq_over_pi, &p.mscale);
    const cudaError_t e = uaa::launch_step_f32(p, s);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "fp32 step kernel launch");
}

// Steps 1 and 2: one fused launch for the tensor-core kernel, append then
// partial for the fp32 kernel.
uaa_status run_append_partial(const uaa_attn_desc* d, const uaa_step_args* a, const uaa_workspace* ws,
                              const Plan& pl, cudaStream_t s)
{
    // one token per sequence; a chunk's append runs first, a warp per head row (a fused
    // kernel that staged a chunk's rows itself measured slower: its prep warp's
    // start-of-segment work is not hidden at one CTA per SM)
    if (pl.kernel == 1 && pl.q_len == 1) return run_partial(d, a, ws, pl, s, true);
    UAA_TRY(run_append(d, a, ws, pl, s));
    return run_partial(d, a, ws, pl, s);
}

uaa_status run_step(const uaa_attn_desc* d, const uaa_step_args* a, const uaa_workspace* ws, const Plan& pl,
                    cudaStream_t s)
{
    const int splits = f32_step_splits(d, a, pl);
    if (splits > 0) return run_step_f32(d, a, ws, pl, splits, s);
    UAA_TRY(run_append_partial(d, a, ws, pl, s));
    return run_combine(d, a, ws, pl, s);
}

// ---------------------------------------------------------------- packed batches

constexpr int kMaxAxes = 4;

// Geometry of a packed step: its workspace keeps the places of the status word, the
// range balance and the fp32 step's counters (make_plan); the q' rows follow.
struct PackedGeo {
    int G;
    int umma;                // the tcgen05 kernel (packed_umma.cuh): bf16, vq8 and q8 caches at head_dim 64 and 128
    int partial;             // the partial kernel and combine: 4-bit caches, head_dim 256; 8-bit ones with few rows (kPackedFewRows)
    Plan pl;                 // its geometry
    size_t off_ranges, off_owners, off_part_o, off_part_lse;
    uaa::ScheduleParams list;  // its work list's sizes
    size_t off_status, off_qrot, off_header, off_entries, off_counters, off_first, off_costs, off_order, off_rec_o, off_rec_lse;
    size_t total;
};

// Record rows of what the packed kernel cuts along the keys. A cut pair i of r_i rows in n_i pieces
// has r_i n_i <= kMergeRows records for each kv head, and so all have at most
// sum sqrt(kMergeRows r_i n_i) <= sqrt(kMergeRows R E), of R rows and E pieces together. E was below
// 4.1 n_sm / Hkv where records were many (12,000 random batches); a pair without room stays whole, and
// so do those beyond kPackedRecRows. 64 rows of 32 / 8 heads: 60 thousand records, 30 MiB at
// head_dim 128, of which 13 were the most that was asked for.
constexpr int kPackedRecRows = 320 << 10;
constexpr int kPackedRecCutsPerSm = 5;

// Entries of its work list beyond one for each row pair, per SM and over the kv heads. The
// list (schedule.cuh) cuts the last m pairs, less than n_sm / Hkv + 1, at half an even share of what
// is left from each on: of equal pairs, the one with k left takes 2 n_sm / (Hkv k) pieces, so that
// all take 2 n_sm / Hkv (1 + 1/2 + .. + 1/m). For one kv head and 152 SMs that is 11 n_sm; 10.0 were
// the most of 6,000 random batches.
constexpr int kPackedCutsPerSm = 16;

// Over 8-bit caches: query rows per kv head, where the caller bounds a request's tokens, up to
// which the partial kernel takes the batch. Its warps widen codes in registers as they multiply,
// but each unit of rows reads the cache anew. 64 requests of up to 8,000 tokens, vq8, head_dim 64 /
// 128: 8 rows 89 / 149 us against 165 / 246 of the tcgen05 kernel, 16 rows 149 / 220 against 169 /
// 246, 24 rows 185 / 271 against 171 / 250, 48 rows 271 / 409 against 181 / 254.
constexpr int kPackedFewRows = 16;

uaa_status packed_geometry(const uaa_attn_desc* d, int batch, int n_tokens, int q_len, int n_sm, PackedGeo* g)
{
    // units of 8 rows where single tokens have no more, of 16 (24) where a request is known to bring more
    Plan& pl = g->pl;
    const int T = q_len < 1 ? 1 : (q_len < 16 ? q_len : 16);
    UAA_TRY(make_plan(d, 0, T, 0, n_sm, &pl));
    if (batch < 0) return fail(UAA_ERR_INVALID_ARGUMENT, "batch=%d is negative", batch);
    if (n_tokens < 0) return fail(UAA_ERR_INVALID_ARGUMENT, "n_tokens=%d is negative", n_tokens);
    if (d->n_kv_heads > 65535) return fail(UAA_ERR_UNSUPPORTED, "n_kv_heads=%d is above 65535 for a packed batch", d->n_kv_heads);
    g->G = pl.G;
    g->off_status = pl.off_status;
    g->off_qrot = pl.off_qrot;
    g->total = g->off_qrot + align256((size_t)n_tokens * d->n_q_heads * d->head_dim * 4);
    const bool codes = d->kv_dtype == UAA_DTYPE_VQ8 || d->kv_dtype == UAA_DTYPE_Q8;
    g->umma = (d->kv_dtype == UAA_DTYPE_BF16 || codes) && (d->head_dim == 64 || d->head_dim == 128);
    g->partial = d->kv_dtype != UAA_DTYPE_F32 && (!g->umma || codes);
    if (g->umma) {
        const int pair_rows = codes ? uaa::kPackedRows8 : uaa::kPackedRows;
        const long long pairs = (long long)n_tokens * pl.G / pair_rows + (n_tokens < batch ? n_tokens : batch) + 1;
        const long long cuts = (long long)kPackedCutsPerSm * n_sm / d->n_kv_heads + 16;
        const long long items = (pairs + cuts) * d->n_kv_heads;
        if (items > 2147483647LL || (long long)n_tokens * pl.G > 2147483647LL)
            return fail(UAA_ERR_UNSUPPORTED, "n_tokens=%d: %lld work items exceed 2^31", n_tokens, items);
        uaa::ScheduleParams& l = g->list;
        l.n_sm = n_sm;
        l.n_tokens = n_tokens;
        l.pair_rows = pair_rows;
        l.max_pairs = (int)pairs;
        l.max_entries = (int)(pairs + cuts);
        const double rec = d->n_kv_heads * ceil(sqrt((double)uaa::kMergeRows * n_tokens * pl.G *
                                                     ((double)kPackedRecCutsPerSm * n_sm / d->n_kv_heads + 16)));
        l.max_rec_rows = rec < kPackedRecRows ? (int)rec : kPackedRecRows;
        l.max_counters = 4 * n_sm + 16 * d->n_kv_heads;
        size_t at = g->total;
        auto take = [&at](size_t bytes) {
            const size_t here = at;
            at += align256(bytes);
            return here;
        };
        g->off_header = take(256);
        g->off_entries = take((size_t)l.max_entries * sizeof(uaa::PackedEntry));
        g->off_counters = take((size_t)l.max_counters * 4);
        g->off_first = take(((size_t)batch + 1) * 4);
        g->off_costs = take((size_t)pairs * 4);
        g->off_order = take((size_t)pairs * 8);
        g->off_rec_lse = take((size_t)l.max_rec_rows * 4);
        g->off_rec_o = take((size_t)l.max_rec_rows * d->head_dim * 4);
        g->total = at;
    }
    if (g->partial) {  // (behind the list, whose places q_len does not move)
        pl.slice = batch < uaa::kMaxSliceBatch ? (batch > 0 ? batch : 1) : uaa::kMaxSliceBatch;
        const size_t P = (size_t)pl.n_ctas, HC = (size_t)pl.heads_per_cta;
        const size_t units = (size_t)n_tokens * uaa::packed_units(pl.G, pl.heads_per_cta) * d->n_kv_heads;
        if (units > 2147483646u) {
            g->partial = 0;
            return g->umma ? UAA_OK : fail(UAA_ERR_UNSUPPORTED, "n_tokens=%d: %zu units exceed 2^31", n_tokens, units);
        }
        g->off_ranges = g->total;
        g->off_owners = g->off_ranges + align256((P + 1) * 8);
        g->off_part_lse = g->off_owners + align256(units * 8);
        g->off_part_o = g->off_part_lse + align256(2 * P * HC * 4);
        g->total = g->off_part_o + align256(2 * P * HC * d->head_dim * 4);
    }
    return UAA_OK;
}

struct NamedPtr {
    const void* p;
    const char* name;
    bool needed;
};

uaa_status check_ptrs(const NamedPtr* ptrs, size_t n)
{
    for (size_t i = 0; i < n; ++i) {
        if (ptrs[i].needed && !ptrs[i].p) return fail(UAA_ERR_INVALID_ARGUMENT, "%s is NULL", ptrs[i].name);
        if (ptrs[i].p && !aligned16(ptrs[i].p))
            return fail(UAA_ERR_INVALID_ARGUMENT, "%s is not 16-byte aligned", ptrs[i].name);
    }
    return UAA_OK;
}

uaa_status check_plan_arrays(const uaa_packed_plan* p, bool need_lens)
{
    if (!p) return fail(UAA_ERR_INVALID_ARGUMENT, "plan is NULL");
    if (p->batch < 0) return fail(UAA_ERR_INVALID_ARGUMENT, "plan.batch=%d is negative", p->batch);
    if (p->n_tokens < 0 || p->n_tokens > (1 << 30))
        return fail(UAA_ERR_UNSUPPORTED, "n_tokens=%d is not in [0, 2^30]", p->n_tokens);
    const bool any = p->batch > 0, rows = p->n_tokens > 0;
    const NamedPtr ptrs[] = {{p->q_lens, "q_lens", any && need_lens}, {p->q_starts, "q_starts", any || rows},
                             {p->kv_ends, "kv_ends", any},           {p->token_seq, "token_seq", rows},
                             {p->positions, "positions", rows},      {p->slots, "slots", rows}};
    return check_ptrs(ptrs, sizeof ptrs / sizeof *ptrs);
}

void plan_arrays(const uaa_packed_plan* p, uaa::PlanParams* out)
{
    out->n_tokens = p->n_tokens;
    out->q_lens = p->q_lens;
    out->q_starts = p->q_starts;
    out->kv_ends = p->kv_ends;
    out->token_seq = p->token_seq;
    out->positions = p->positions;
    out->slots = reinterpret_cast<long long*>(p->slots);
}

// Key stages of a packed batch's units at most: the partial kernel counts them in 32 bits.
double packed_stages(const uaa_attn_desc* d, const uaa_packed_args* a, const PackedGeo& g)
{
    long long keys = a->step.cache_capacity;
    if (d->window > 0) {
        const long long seen = (long long)d->window + a->plan.n_tokens + d->first_tokens;
        keys = keys < seen ? keys : seen;
    }
    const double stages = (double)(keys / (uaa::kTileKeys * g.pl.mg) + 3);
    return stages * (((double)a->plan.n_tokens * g.G / g.pl.heads_per_cta + a->step.batch) * d->n_kv_heads);
}

// Whether the partial kernel takes the batch's attention.
bool takes_packed_partial(const uaa_attn_desc* d, const uaa_packed_args* a, const PackedGeo& g)
{
    if (!g.partial || !g.umma) return g.partial;
    return a->step.q_len > 0 && a->step.q_len <= kPackedFewRows / g.G && packed_stages(d, a, g) <= 2147483647.0;
}

uaa_status check_packed_stages(const uaa_attn_desc* d, const uaa_packed_args* a, const PackedGeo& g)
{
    if (!g.partial || g.umma || packed_stages(d, a, g) <= 2147483647.0) return UAA_OK;
    return fail(UAA_ERR_UNSUPPORTED, "cache_capacity=%d, n_tokens=%d: %.3g key stages exceed 2^31 (split the batch)",
                a->step.cache_capacity, a->plan.n_tokens, packed_stages(d, a, g));
}

uaa_status check_packed(const uaa_attn_desc* d, const uaa_packed_args* a, const uaa_workspace* ws, bool need_io,
                        bool need_out, PackedGeo* g)
{
    UAA_TRY(check_desc(d));
    if (!a) return fail(UAA_ERR_INVALID_ARGUMENT, "args is NULL");
    const uaa_step_args* st = &a->step;
    UAA_TRY(check_cache(d, st));
    UAA_TRY(check_plan_arrays(&a->plan, false));
    if (a->plan.batch != st->batch)
        return fail(UAA_ERR_INVALID_ARGUMENT, "plan.batch=%d is not the step's batch=%d", a->plan.batch, st->batch);
    if (st->q_len < 0) return fail(UAA_ERR_INVALID_ARGUMENT, "q_len=%d is negative", st->q_len);
    if (!ws || !ws->ptr) return fail(UAA_ERR_INVALID_ARGUMENT, "workspace is NULL");
    if (!aligned16(ws->ptr)) return fail(UAA_ERR_INVALID_ARGUMENT, "workspace is not 16-byte aligned");
    if (need_io && (a->n_axes < 0 || a->n_axes > kMaxAxes))
        return fail(UAA_ERR_UNSUPPORTED, "n_axes=%d is not in [0, %d]", a->n_axes, kMaxAxes);
    const bool any = st->batch > 0 && a->plan.n_tokens > 0;
    const NamedPtr ptrs[] = {{st->q, "q", any && need_io},
                             {st->k_new, "k_new", any && need_io},
                             {st->v_new, "v_new", any && need_io},
                             {st->seq_lens, "seq_lens", st->batch > 0 && need_io},
                             {st->out, "out", any && need_out},
                             {st->q_norm_w, "q_norm_w", any && need_io && d->qk_norm},
                             {st->k_norm_w, "k_norm_w", any && need_io && d->qk_norm},
                             {st->sink, "sink", any && need_out && d->has_sink},
                             {st->q_rot, "q_rot", false},
                             {a->axis_positions, "axis_positions", any && need_io && a->n_axes > 0}};
    UAA_TRY(check_ptrs(ptrs, sizeof ptrs / sizeof *ptrs));
    if (need_io) {
        const long long align = d->io_dtype == UAA_DTYPE_F32 ? 4 : 8;
        const struct {
            long long stride;
            int heads;
            const char* name;
        } strides[] = {{a->q_stride, d->n_q_heads, "q_stride"},
                       {a->k_stride, d->n_kv_heads, "k_stride"},
                       {a->v_stride, d->n_kv_heads, "v_stride"}};
        for (auto& e : strides)
            if (e.stride != 0 && (e.stride < (long long)e.heads * d->head_dim || e.stride % align != 0))
                return fail(UAA_ERR_UNSUPPORTED, "%s=%lld is not a multiple of %lld elements holding a token's %d heads",
                            e.name, e.stride, align, e.heads);
        for (int p = 0; a->n_axes > 0 && p < rotary_dims(d) / 2; ++p)
            if (a->pair_axis[p] >= a->n_axes)
                return fail(UAA_ERR_UNSUPPORTED, "pair_axis[%d]=%d is not below n_axes=%d", p, a->pair_axis[p], a->n_axes);
    }
    const int n_sm = device_sm_count();
    UAA_TRY(packed_geometry(d, st->batch, a->plan.n_tokens, st->q_len, n_sm > 0 ? n_sm : 1, g));
    UAA_TRY(check_packed_stages(d, a, *g));
    if (n_sm <= 0) return fail(UAA_ERR_CUDA, "no CUDA device: the SM count query failed");
    if (ws->bytes < g->total)
        return fail(UAA_ERR_INVALID_ARGUMENT, "workspace has %zu bytes, the packed step needs %zu", ws->bytes, g->total);
    return UAA_OK;
}

uaa_status run_packed_append(const uaa_attn_desc* d, const uaa_packed_args* a, const uaa_workspace* ws,
                             const PackedGeo& g, cudaStream_t s)
{
    if (a->step.batch == 0 || a->plan.n_tokens == 0) return UAA_OK;
    const uaa_step_args* st = &a->step;
    uaa::AppendParams p{};
    p.B = st->batch;
    p.Hq = d->n_q_heads;
    p.Hkv = d->n_kv_heads;
    p.D = d->head_dim;
    p.cap = st->cache_capacity;
    p.style = d->rope.style;
    p.half_rot = rotary_dims(d) / 2;
    p.qk_norm = d->qk_norm;
    p.eps = d->norm_eps;
    p.norm_offset = d->norm_offset ? 1.f : 0.f;
    p.qscale = qscale(d);
    p.io_dtype = d->io_dtype;
    p.kv_dtype = d->kv_dtype;
    p.q = st->q;
    p.k_new = st->k_new;
    p.v_new = st->v_new;
    p.q_norm_w = st->q_norm_w;
    p.k_norm_w = st->k_norm_w;
    p.k_cache = st->k_cache;
    p.v_cache = st->v_cache;
    p.v_scale = st->v_scale;
    p.k_scale = st->k_scale;
    p.pages = pages_of(st);
    p.seq_lens = st->seq_lens;
    char* w = static_cast<char*>(ws->ptr);
    p.q_prime = st->q_rot ? nullptr : reinterpret_cast<float*>(w + g.off_qrot);
    p.q_rot_out = st->q_rot;
    p.status = reinterpret_cast<unsigned*>(w + g.off_status);
    rope_table(d, p.inv_freq_over_pi, &p.mscale, &p.mscale64);
    uaa::PackedRows& k = p.pk;
    k.n_tokens = a->plan.n_tokens;
    k.batch = st->batch;
    k.token_seq = a->plan.token_seq;
    k.positions = a->plan.positions;
    k.slots = reinterpret_cast<const long long*>(a->plan.slots);
    k.kv_ends = a->plan.kv_ends;
    k.axis_pos = a->n_axes > 0 ? a->axis_positions : nullptr;
    k.q_stride = a->q_stride ? a->q_stride : (long long)d->n_q_heads * d->head_dim;
    k.k_stride = a->k_stride ? a->k_stride : (long long)d->n_kv_heads * d->head_dim;
    k.v_stride = a->v_stride ? a->v_stride : (long long)d->n_kv_heads * d->head_dim;
    for (int i = 0; i < d->head_dim / 2; ++i)
        k.angle_step[i] = (unsigned long long)llrint(ldexp(fmod(p.inv_freq_over_pi[i], 2.0), 62)) << 1;
    if (a->n_axes > 0) memcpy(k.pair_axis, a->pair_axis, rotary_dims(d) / 2);  // (pairs that pass unchanged: axis 0)
    uaa::ScheduleParams l = g.list;
    if (g.umma && !st->q_rot) {
        l.B = st->batch;
        l.G = g.G;
        l.Hkv = d->n_kv_heads;
        l.cap = st->cache_capacity;
        l.window = d->window;
        l.first_tokens = first_tokens(d);
        l.q_starts = a->plan.q_starts;
        l.kv_ends = a->plan.kv_ends;
        l.header = reinterpret_cast<unsigned*>(w + g.off_header);
        l.entries = reinterpret_cast<uaa::PackedEntry*>(w + g.off_entries);
        l.counters = reinterpret_cast<unsigned*>(w + g.off_counters);
        l.pair_first = reinterpret_cast<int*>(w + g.off_first);
        l.costs = reinterpret_cast<int*>(w + g.off_costs);
        l.order = reinterpret_cast<int2*>(w + g.off_order);
    }
    const cudaError_t e = uaa::launch_append_packed(p, l.header ? &l : nullptr, device_sm_count(), s);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "packed append kernel launch");
}

// The partial kernel and the combine over a packed batch, slice by slice.
uaa_status run_packed_partial(const uaa_attn_desc* d, const uaa_packed_args* a, const uaa_workspace* ws, const PackedGeo& g,
                              cudaStream_t s)
{
    const uaa_step_args* st = &a->step;
    char* w = static_cast<char*>(ws->ptr);
    uaa::PartialMaps maps{};
    UAA_TRY(partial_maps(d, st, g.pl.n_head_tiles, &maps));
    for (int b0 = 0; b0 < st->batch; b0 += g.pl.slice) {
        uaa::PartialParams p{};
        p.B = st->batch - b0 < g.pl.slice ? st->batch - b0 : g.pl.slice;
        p.Hq = d->n_q_heads;
        p.Hkv = d->n_kv_heads;
        p.D = d->head_dim;
        p.G = g.G;
        p.b_off = b0;
        p.heads_per_cta = g.pl.heads_per_cta;
        p.cap = st->cache_capacity;
        p.q_len = 1;
        p.attn_window = d->window;
        p.first_tokens = first_tokens(d);
        p.mg = g.pl.mg;
        p.softcap_log2e = d->softcap > 0.f ? d->softcap * uaa::kLog2e : 0.f;
        p.q_prime = reinterpret_cast<const float*>(w + g.off_qrot);
        p.k_cache = st->k_cache;
        p.v_cache = st->v_cache;
        p.v_scale = st->v_scale;
        p.k_scale = st->k_scale;
        p.pages = pages_of(st);
        p.seq_lens = const_cast<int32_t*>(a->plan.kv_ends) + b0;  // read only
        p.q_starts = a->plan.q_starts + b0;
        p.ranges = reinterpret_cast<long long*>(w + g.off_ranges);
        p.owners = reinterpret_cast<unsigned*>(w + g.off_owners);
        p.bal = balance_of(w, g.pl);
        p.per_sm = g.pl.per_sm;
        p.uniform = d->reproducible;
        p.rec_lse = reinterpret_cast<float*>(w + g.off_part_lse);
        p.rec_o = reinterpret_cast<float*>(w + g.off_part_o);
        p.sink = d->has_sink ? st->sink : nullptr;
        p.out = st->out;
        p.out_dtype = d->out_dtype;
        p.status = reinterpret_cast<unsigned*>(w + g.off_status);
        cudaError_t e = uaa::launch_partial_packed(p, maps, d->kv_dtype, g.pl.n_head_tiles, g.pl.n_ctas, s);
        if (e != cudaSuccess) return cuda_fail(e, "packed partial kernel launch");
        uaa::CombineParams c{};
        c.B = p.B;
        c.Hq = p.Hq;
        c.Hkv = p.Hkv;
        c.D = p.D;
        c.G = p.G;
        c.heads_per_cta = p.heads_per_cta;
        c.q_len = st->q_len > 0 && st->q_len < 16 ? st->q_len : 16;  // (sizes the CTAs)
        c.P = g.pl.n_ctas;
        c.out_dtype = p.out_dtype;
        c.sink = p.sink;
        c.owners = p.owners;
        c.bal = p.bal;
        c.rec_lse = p.rec_lse;
        c.rec_o = p.rec_o;
        c.out = p.out;
        c.status = p.status;
        c.q_starts = a->plan.q_starts;
        c.token_seq = a->plan.token_seq;
        c.n_tokens = a->plan.n_tokens;
        c.b_off = b0;
        e = uaa::launch_combine(c, s);
        if (e != cudaSuccess) return cuda_fail(e, "packed combine kernel launch");
    }
    return UAA_OK;
}

uaa_status run_packed_attn(const uaa_attn_desc* d, const uaa_packed_args* a, const uaa_workspace* ws,
                           const PackedGeo& g, cudaStream_t s)
{
    if (a->step.batch == 0 || a->plan.n_tokens == 0) return UAA_OK;
    const uaa_step_args* st = &a->step;
    char* w = static_cast<char*>(ws->ptr);
    if (takes_packed_partial(d, a, g)) return run_packed_partial(d, a, ws, g, s);
    if (g.umma) {
        const uint64_t D = d->head_dim;
        const uint64_t rows = st->block_table ? (uint64_t)st->n_pages * d->n_kv_heads * st->page_size
                                              : (uint64_t)st->batch * d->n_kv_heads * st->cache_capacity;
        const uint32_t box = st->block_table && st->page_size < uaa::kPackedKeys ? (uint32_t)st->page_size
                                                                                 : (uint32_t)uaa::kPackedKeys;
        uaa::PackedMaps maps;
        auto values = [&](CUtensorMap* m, const void* at, const char* name) {
            return encode_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, const_cast<void*>(at), D, rows, D * 2, 64, box, CU_TENSOR_MAP_SWIZZLE_128B, name);
        };
        auto codes = [&](CUtensorMap* m, const void* at, const char* name) {
            return encode_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<void*>(at), D, rows, D, (uint32_t)D, box, CU_TENSOR_MAP_SWIZZLE_NONE, name);
        };
        auto scales = [&](CUtensorMap* m, const void* at, const char* name) {
            const uint64_t per = st->block_table ? st->page_size : st->cache_capacity;
            return encode_2d(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, const_cast<void*>(at), per, rows / per, per * 4, box, 1,
                             CU_TENSOR_MAP_SWIZZLE_NONE, name);
        };
        if (d->kv_dtype == UAA_DTYPE_Q8) UAA_TRY(codes(&maps.k, st->k_cache, "k_cache codes"));
        else UAA_TRY(values(&maps.k, st->k_cache, "k_cache"));
        if (d->kv_dtype == UAA_DTYPE_BF16) UAA_TRY(values(&maps.v, st->v_cache, "v_cache"));
        else UAA_TRY(codes(&maps.v, st->v_cache, "v_cache codes"));
        maps.vs = maps.v;  // (unused without value codes, key codes)
        if (d->kv_dtype != UAA_DTYPE_BF16) UAA_TRY(scales(&maps.vs, st->v_scale, "v_scale"));
        maps.ks = maps.vs;
        if (d->kv_dtype == UAA_DTYPE_Q8) UAA_TRY(scales(&maps.ks, st->k_scale, "k_scale"));
        uaa::PackedUmmaParams p{};
        p.B = st->batch;
        p.n_tokens = a->plan.n_tokens;
        p.max_entries = g.list.max_entries;
        p.max_rec_rows = g.list.max_rec_rows;
        p.max_counters = g.list.max_counters;
        p.Hq = d->n_q_heads;
        p.Hkv = d->n_kv_heads;
        p.G = g.G;
        p.cap = st->cache_capacity;
        p.window = d->window;
        p.first_tokens = first_tokens(d);
        p.softcap_log2e = d->softcap > 0.f ? d->softcap * uaa::kLog2e : 0.f;
        p.q_prime = reinterpret_cast<const float*>(w + g.off_qrot);
        p.pages = pages_of(st);
        p.sink = d->has_sink ? st->sink : nullptr;
        p.out = st->out;
        p.out_dtype = d->out_dtype;
        p.next = reinterpret_cast<unsigned*>(w + g.off_header);
        p.entries_n = p.next + 1;
        p.entries = reinterpret_cast<const uaa::PackedEntry*>(w + g.off_entries);
        p.counters = reinterpret_cast<unsigned*>(w + g.off_counters);
        p.rec_o = reinterpret_cast<float*>(w + g.off_rec_o);
        p.rec_lse = reinterpret_cast<float*>(w + g.off_rec_lse);
        p.status = reinterpret_cast<unsigned*>(w + g.off_status);
        const cudaError_t e = uaa::launch_packed_umma(p, d->head_dim, d->kv_dtype, maps, device_sm_count(), s);
        return e == cudaSuccess ? UAA_OK : cuda_fail(e, "packed attention kernel launch");
    }
    uaa::PackedParams p{};
    p.B = st->batch;
    p.Hq = d->n_q_heads;
    p.Hkv = d->n_kv_heads;
    p.D = d->head_dim;
    p.G = g.G;
    p.n_tokens = a->plan.n_tokens;
    p.cap = st->cache_capacity;
    p.window = d->window;
    p.first_tokens = first_tokens(d);
    p.softcap_log2e = d->softcap > 0.f ? d->softcap * uaa::kLog2e : 0.f;
    p.out_dtype = d->out_dtype;
    p.q_prime = reinterpret_cast<const float*>(w + g.off_qrot);
    p.q_starts = a->plan.q_starts;
    p.kv_ends = a->plan.kv_ends;
    p.token_seq = a->plan.token_seq;
    p.k_cache = st->k_cache;
    p.v_cache = st->v_cache;
    p.pages = pages_of(st);
    p.sink = d->has_sink ? st->sink : nullptr;
    p.out = st->out;
    p.status = reinterpret_cast<unsigned*>(w + g.off_status);
    const cudaError_t e = uaa::launch_packed_simt(p, s);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "packed attention kernel launch");
}

// ---------------------------------------------------------------- pages of a cache

// Workspace of the page operators: status word | a copy of the table | of the
// lengths | a list of free pages | per page: requests, the last of them, its map.
struct PageLayout {
    size_t table, lens, list, asked, last, map, total;
};

uaa_status page_layout(int batch, int per_seq, int n_pages, PageLayout* lay)
{
    if (batch < 0) return fail(UAA_ERR_INVALID_ARGUMENT, "batch=%d is negative", batch);
    if (per_seq <= 0) return fail(UAA_ERR_INVALID_ARGUMENT, "pages_per_seq=%d is not positive", per_seq);
    if (n_pages <= 0) return fail(UAA_ERR_INVALID_ARGUMENT, "n_pages=%d is not positive", n_pages);
    if ((long long)batch * per_seq > (1LL << 30) || n_pages > (1 << 30))
        return fail(UAA_ERR_UNSUPPORTED, "batch*pages_per_seq=%lld or n_pages=%d exceeds 2^30", (long long)batch * per_seq,
                    n_pages);
    const size_t entries = align256((size_t)batch * per_seq * 4), pages = align256((size_t)n_pages * 4);
    lay->table = 256;
    lay->lens = lay->table + entries;
    lay->list = lay->lens + align256((size_t)batch * 4);
    lay->asked = lay->list + entries;
    lay->last = lay->asked + pages;
    lay->map = lay->last + pages;
    lay->total = lay->map + pages;
    return UAA_OK;
}

uaa_status page_params(const uaa_page_args* a, const uaa_workspace* ws, uaa::PageParams* p)
{
    if (!a) return fail(UAA_ERR_INVALID_ARGUMENT, "args is NULL");
    if (!ws || !ws->ptr) return fail(UAA_ERR_INVALID_ARGUMENT, "workspace is NULL");
    if (!aligned16(ws->ptr)) return fail(UAA_ERR_INVALID_ARGUMENT, "workspace is not 16-byte aligned");
    if (a->page_size < 16 || a->page_size > 4096 || (a->page_size & (a->page_size - 1)) != 0)
        return fail(UAA_ERR_UNSUPPORTED, "page_size=%d is not a power of two in [16, 4096]", a->page_size);
    PageLayout lay;
    UAA_TRY(page_layout(a->batch, a->pages_per_seq, a->n_pages, &lay));
    if ((long long)a->pages_per_seq * a->page_size > 2147483647LL)
        return fail(UAA_ERR_UNSUPPORTED, "pages_per_seq=%d x page_size=%d exceeds 2^31 positions", a->pages_per_seq,
                    a->page_size);
    if (ws->bytes < lay.total)
        return fail(UAA_ERR_INVALID_ARGUMENT, "workspace has %zu bytes, the page operators need %zu", ws->bytes,
                    lay.total);
    const struct {
        const void* q;
        const char* name;
        bool needed;
    } ptrs[] = {{a->block_table, "block_table", a->batch > 0},
                {a->seq_lens, "seq_lens", a->batch > 0},
                {a->page_refs, "page_refs", true},
                {a->moves, "moves", true},
                {a->counts, "counts", true}};
    for (auto& e : ptrs) {
        if (e.needed && !e.q) return fail(UAA_ERR_INVALID_ARGUMENT, "%s is NULL", e.name);
        if (e.q && !aligned16(e.q)) return fail(UAA_ERR_INVALID_ARGUMENT, "%s is not 16-byte aligned", e.name);
    }
    char* w = static_cast<char*>(ws->ptr);
    p->B = a->batch;
    p->per_seq = a->pages_per_seq;
    p->page_size = a->page_size;
    p->n_pages = a->n_pages;
    p->table = a->block_table;
    p->seq_lens = a->seq_lens;
    p->refs = a->page_refs;
    p->moves = a->moves;
    p->counts = a->counts;
    p->status = reinterpret_cast<unsigned*>(w);
    p->table_tmp = reinterpret_cast<int*>(w + lay.table);
    p->lens_tmp = reinterpret_cast<int*>(w + lay.lens);
    p->list = reinterpret_cast<int*>(w + lay.list);
    p->asked = reinterpret_cast<int*>(w + lay.asked);
    p->last = reinterpret_cast<int*>(w + lay.last);
    p->map = reinterpret_cast<int*>(w + lay.map);
    return UAA_OK;
}

}  // namespace

// ---------------------------------------------------------------- exported C ABI

extern "C" {

uaa_status uaa_rope_qk_norm_append(const uaa_attn_desc* desc, const uaa_step_args* args, const uaa_workspace* ws,
                                   cudaStream_t stream)
{
    Plan pl{};
    UAA_TRY(prepare(desc, args, ws, true, &pl));
    return run_append(desc, args, ws, pl, stream);
}

uaa_status uaa_decode_attn_partial(const uaa_attn_desc* desc, const uaa_step_args* args, const uaa_workspace* ws,
                                   cudaStream_t stream)
{
    Plan pl{};
    UAA_TRY(prepare(desc, args, ws, false, &pl));
    return run_partial(desc, args, ws, pl, stream);
}

uaa_status uaa_decode_attn_combine(const uaa_attn_desc* desc, const uaa_step_args* args, const uaa_workspace* ws,
                                   cudaStream_t stream)
{
    Plan pl{};
    UAA_TRY(prepare(desc, args, ws, false, &pl));
    return run_combine(desc, args, ws, pl, stream);
}

uaa_status uaa_decode_attn_append_partial(const uaa_attn_desc* desc, const uaa_step_args* args,
                                          const uaa_workspace* ws, cudaStream_t stream)
{
    Plan pl{};
    UAA_TRY(prepare(desc, args, ws, true, &pl));
    return run_append_partial(desc, args, ws, pl, stream);
}

uaa_status uaa_decode_attn(const uaa_attn_desc* desc, const uaa_step_args* args, const uaa_workspace* ws,
                           cudaStream_t stream)
{
    Plan pl{};
    UAA_TRY(prepare(desc, args, ws, true, &pl));
    return run_step(desc, args, ws, pl, stream);
}

size_t uaa_workspace_size(const uaa_attn_desc* desc, int32_t batch, int32_t max_seq_len, int32_t n_sm,
                          int32_t q_len)
{
    if (n_sm <= 0) n_sm = device_sm_count();
    return workspace_bytes(desc, batch, q_len, max_seq_len, n_sm);
}

int32_t uaa_num_splits(const uaa_attn_desc* desc, int32_t batch, int32_t max_seq_len, int32_t n_sm, int32_t q_len)
{
    Plan pl{};
    if (n_sm <= 0) n_sm = device_sm_count();
    if (make_plan(desc, batch, q_len, max_seq_len, n_sm, &pl) != UAA_OK) return 0;
    return pl.n_ctas;
}

uaa_status uaa_get_workspace_layout(const uaa_attn_desc* desc, int32_t batch, int32_t max_seq_len, int32_t n_sm,
                                    int32_t q_len, uaa_workspace_layout* layout)
{
    if (!layout) return fail(UAA_ERR_INVALID_ARGUMENT, "layout is NULL");
    Plan pl{};
    if (n_sm <= 0) n_sm = device_sm_count();
    UAA_TRY(make_plan(desc, batch, q_len, max_seq_len, n_sm, &pl));
    layout->n_ctas = pl.n_ctas;
    layout->stage_keys = pl.mg * uaa::kTileKeys;
    layout->heads_per_cta = pl.heads_per_cta;
    layout->kernel = pl.prefill ? 2 : pl.kernel;
    layout->n_slices = pl.n_slices;
    layout->slice_batch = pl.slice;
    {
        uaa_step_args a{};
        a.batch = batch;
        a.max_seq_len = max_seq_len;
        layout->step_splits = f32_step_splits(desc, &a, pl);
        layout->step_kernels = batch == 0 ? 0
                               : layout->step_splits > 0 ? 1
                               : pl.dense_rows > 0 ? 1 + 2 * ((batch + pl.dense_batch - 1) / pl.dense_batch)
                               : pl.prefill ? 2
                               : (pl.kernel == 1 && pl.q_len == 1) ? 2 * pl.n_slices
                                                                   : 1 + 2 * pl.n_slices;
    }
    layout->status_offset = pl.off_status;
    layout->q_rot_offset = pl.off_qrot;
    layout->prefix_offset = pl.off_prefix;
    layout->rec_lse_offset = pl.off_rec_lse;
    layout->rec_o_offset = pl.off_rec_o;
    layout->prefix_stride = pl.prefix_stride;
    layout->rec_lse_stride = pl.rec_lse_stride;
    layout->rec_o_stride = pl.rec_o_stride;
    layout->ranges_offset = pl.off_ranges;
    layout->ranges_stride = pl.ranges_stride;
    layout->owners_offset = pl.off_owners;
    layout->owners_stride = pl.owners_stride;
    layout->balance_offset = pl.off_balance;
    layout->total_bytes = workspace_bytes(desc, batch, q_len, max_seq_len, n_sm);
    return UAA_OK;
}

uaa_status uaa_vq8_quantize(const void* v, int32_t v_dtype, int64_t n_rows, int32_t head_dim, int8_t* codes,
                            float* scales, cudaStream_t stream)
{
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return fail(UAA_ERR_UNSUPPORTED, "head_dim=%d is not supported (supported: {64, 128, 256})", head_dim);
    if (v_dtype != UAA_DTYPE_F32 && v_dtype != UAA_DTYPE_BF16)
        return fail(UAA_ERR_UNSUPPORTED, "v_dtype=%d is not F32 or BF16", v_dtype);
    if (n_rows < 0) return fail(UAA_ERR_INVALID_ARGUMENT, "n_rows=%lld is negative", (long long)n_rows);
    if (n_rows == 0) return UAA_OK;
    if (!v || !codes || !scales) return fail(UAA_ERR_INVALID_ARGUMENT, "a vq8_quantize pointer is NULL");
    if (!aligned16(v) || !aligned16(codes) || !aligned16(scales))
        return fail(UAA_ERR_INVALID_ARGUMENT, "vq8_quantize pointers must be 16-byte aligned");
    const cudaError_t e = uaa::launch_vq8_quantize(v, v_dtype, n_rows, head_dim, codes, scales, stream);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "vq8 quantize kernel launch");
}

uaa_status uaa_q4_quantize(const void* x, int32_t x_dtype, int64_t n_rows, int32_t head_dim, uint8_t* codes,
                           void* scales, cudaStream_t stream)
{
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return fail(UAA_ERR_UNSUPPORTED, "head_dim=%d is not supported (supported: {64, 128, 256})", head_dim);
    if (x_dtype != UAA_DTYPE_F32 && x_dtype != UAA_DTYPE_BF16)
        return fail(UAA_ERR_UNSUPPORTED, "x_dtype=%d is not F32 or BF16", x_dtype);
    if (n_rows < 0) return fail(UAA_ERR_INVALID_ARGUMENT, "n_rows=%lld is negative", (long long)n_rows);
    if (n_rows > (1LL << 55)) return fail(UAA_ERR_UNSUPPORTED, "n_rows=%lld is above 2^55", (long long)n_rows);
    if (n_rows == 0) return UAA_OK;
    if (!x || !codes || !scales) return fail(UAA_ERR_INVALID_ARGUMENT, "a q4_quantize pointer is NULL");
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales))
        return fail(UAA_ERR_INVALID_ARGUMENT, "q4_quantize pointers must be 16-byte aligned");
    const cudaError_t e =
        uaa::launch_q4_quantize(x, x_dtype, n_rows, head_dim, codes, static_cast<__half*>(scales), stream);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "q4 quantize kernel launch");
}

uaa_status uaa_cache_read(const uaa_attn_desc* desc, const uaa_step_args* args, const int32_t* start, int32_t n_rows,
                          void* k_out, void* v_out, cudaStream_t stream)
{
    UAA_TRY(check_desc(desc));
    UAA_TRY(check_cache(desc, args));
    if (n_rows < 0) return fail(UAA_ERR_INVALID_ARGUMENT, "n_rows=%d is negative", n_rows);
    if (!aligned16(k_out) || !aligned16(v_out))
        return fail(UAA_ERR_INVALID_ARGUMENT, "cache_read outputs must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(start) & 3u) return fail(UAA_ERR_INVALID_ARGUMENT, "start is not 4-byte aligned");
    if (args->batch == 0 || n_rows == 0 || (!k_out && !v_out)) return UAA_OK;
    uaa::ReadParams p{};
    p.B = args->batch;
    p.Hkv = desc->n_kv_heads;
    p.D = desc->head_dim;
    p.cap = args->cache_capacity;
    p.n = n_rows;
    p.kv_dtype = desc->kv_dtype;
    p.out_dtype = desc->out_dtype;
    p.start = start;
    p.k_cache = args->k_cache;
    p.v_cache = args->v_cache;
    p.k_scale = args->k_scale;
    p.v_scale = args->v_scale;
    p.pages = pages_of(args);
    p.k_out = k_out;
    p.v_out = v_out;
    const cudaError_t e = uaa::launch_cache_read(p, stream);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "cache read kernel launch");
}

size_t uaa_pages_workspace_size(int32_t batch, int32_t pages_per_seq, int32_t n_pages)
{
    PageLayout lay;
    return page_layout(batch, pages_per_seq, n_pages, &lay) == UAA_OK ? lay.total : 0;
}

uaa_status uaa_pages_fork(const uaa_page_args* args, const int32_t* parents, const uaa_workspace* ws,
                          cudaStream_t stream)
{
    uaa::PageParams p;
    UAA_TRY(page_params(args, ws, &p));
    if (p.B == 0) return UAA_OK;
    if (!parents) return fail(UAA_ERR_INVALID_ARGUMENT, "parents is NULL");
    if (reinterpret_cast<uintptr_t>(parents) & 3u)
        return fail(UAA_ERR_INVALID_ARGUMENT, "parents is not 4-byte aligned");
    const cudaError_t e = uaa::launch_pages_fork(p, parents, stream);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "page fork kernel launch");
}

uaa_status uaa_pages_trim(const uaa_page_args* args, int32_t window, int32_t first_tokens, const uaa_workspace* ws,
                          cudaStream_t stream)
{
    uaa::PageParams p;
    UAA_TRY(page_params(args, ws, &p));
    if (window <= 0) return fail(UAA_ERR_UNSUPPORTED, "window=%d is not positive", window);
    if (first_tokens < 0) return fail(UAA_ERR_UNSUPPORTED, "first_tokens=%d is negative", first_tokens);
    if (p.B == 0) return UAA_OK;
    const cudaError_t e = uaa::launch_pages_trim(p, window, first_tokens, stream);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "page trim kernel launch");
}

uaa_status uaa_pages_reserve(const uaa_page_args* args, int32_t q_len, const uaa_workspace* ws, cudaStream_t stream)
{
    uaa::PageParams p;
    UAA_TRY(page_params(args, ws, &p));
    if (q_len < 1 || q_len > kMaxQLen) return fail(UAA_ERR_UNSUPPORTED, "q_len=%d is not in [1, %d]", q_len, kMaxQLen);
    const cudaError_t e = uaa::launch_pages_reserve(p, q_len, stream);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "page reserve kernel launch");
}

uaa_status uaa_pages_compact(const uaa_page_args* args, const uaa_workspace* ws, cudaStream_t stream)
{
    uaa::PageParams p;
    UAA_TRY(page_params(args, ws, &p));
    const cudaError_t e = uaa::launch_pages_compact(p, stream);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "page compact kernel launch");
}

uaa_status uaa_pages_copy(const uaa_page_args* args, void* const* pools, const int64_t* page_bytes, int32_t n_pools,
                          const uaa_workspace* ws, cudaStream_t stream)
{
    uaa::PageParams p;
    UAA_TRY(page_params(args, ws, &p));
    if (n_pools < 0 || n_pools > uaa::kMaxPools)
        return fail(UAA_ERR_UNSUPPORTED, "n_pools=%d is not in [0, %d]", n_pools, uaa::kMaxPools);
    if (n_pools == 0) return UAA_OK;
    if (!pools || !page_bytes) return fail(UAA_ERR_INVALID_ARGUMENT, "pools or page_bytes is NULL");
    uaa::PagePools pp{};
    for (int k = 0; k < n_pools; ++k) {
        if (!pools[k]) return fail(UAA_ERR_INVALID_ARGUMENT, "pools[%d] is NULL", k);
        if (!aligned16(pools[k])) return fail(UAA_ERR_INVALID_ARGUMENT, "pools[%d] is not 16-byte aligned", k);
        if (page_bytes[k] <= 0 || page_bytes[k] % 16 != 0 || page_bytes[k] > (1LL << 31))
            return fail(UAA_ERR_UNSUPPORTED, "page_bytes[%d]=%lld is not a positive multiple of 16 up to 2^31", k,
                        (long long)page_bytes[k]);
        pp.base[k] = static_cast<char*>(pools[k]);
        pp.bytes[k] = page_bytes[k];
    }
    pp.n = n_pools;
    const int n_sm = device_sm_count();
    if (n_sm <= 0) return fail(UAA_ERR_CUDA, "no CUDA device: the SM count query failed");
    const cudaError_t e = uaa::launch_pages_copy(p, pp, n_sm, stream);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "page copy kernel launch");
}

uaa_status uaa_pages_plan(const uaa_page_args* args, const uaa_packed_plan* plan, const uaa_workspace* ws,
                          cudaStream_t stream)
{
    uaa::PlanParams p{};
    UAA_TRY(page_params(args, ws, &p.pg));
    UAA_TRY(check_plan_arrays(plan, true));
    if (plan->batch != args->batch)
        return fail(UAA_ERR_INVALID_ARGUMENT, "plan.batch=%d is not the table's batch=%d", plan->batch, args->batch);
    if (plan->batch == 0 && plan->n_tokens == 0) return UAA_OK;
    if (!p.pg.table) return fail(UAA_ERR_INVALID_ARGUMENT, "block_table is NULL");
    p.cap = args->pages_per_seq * args->page_size;
    plan_arrays(plan, &p);
    const cudaError_t e = uaa::launch_plan(p, stream);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "plan kernel launch");
}

uaa_status uaa_contiguous_plan(const uaa_packed_plan* plan, const int32_t* seq_lens, int32_t cache_capacity,
                               const uaa_workspace* ws, cudaStream_t stream)
{
    UAA_TRY(check_plan_arrays(plan, true));
    if (!ws || !ws->ptr) return fail(UAA_ERR_INVALID_ARGUMENT, "workspace is NULL");
    if (!aligned16(ws->ptr)) return fail(UAA_ERR_INVALID_ARGUMENT, "workspace is not 16-byte aligned");
    if (ws->bytes < 256) return fail(UAA_ERR_INVALID_ARGUMENT, "workspace has %zu bytes, a plan needs 256", ws->bytes);
    if (cache_capacity <= 0) return fail(UAA_ERR_INVALID_ARGUMENT, "cache_capacity=%d is not positive", cache_capacity);
    if (plan->batch == 0 && plan->n_tokens == 0) return UAA_OK;
    if (plan->batch > 0 && !seq_lens) return fail(UAA_ERR_INVALID_ARGUMENT, "seq_lens is NULL");
    if (!aligned16(seq_lens)) return fail(UAA_ERR_INVALID_ARGUMENT, "seq_lens is not 16-byte aligned");
    uaa::PlanParams p{};
    p.pg.B = plan->batch;
    p.pg.seq_lens = const_cast<int32_t*>(seq_lens);  // read only
    p.pg.status = static_cast<unsigned*>(ws->ptr);
    p.cap = cache_capacity;
    plan_arrays(plan, &p);
    const cudaError_t e = uaa::launch_plan(p, stream);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "plan kernel launch");
}

size_t uaa_packed_workspace_size(const uaa_attn_desc* desc, int32_t batch, int32_t n_tokens, int32_t n_sm)
{
    PackedGeo g{};
    if (n_sm <= 0) n_sm = device_sm_count();
    // the most that any q_len takes (units of 8, 16 or 24 rows)
    size_t bytes = 0;
    for (int q_len = 1; q_len <= 16; ++q_len) {
        if (packed_geometry(desc, batch, n_tokens, q_len, n_sm, &g) != UAA_OK) return 0;
        if (g.total > bytes) bytes = g.total;
    }
    return bytes;
}

uaa_status uaa_packed_append(const uaa_attn_desc* desc, const uaa_packed_args* args, const uaa_workspace* ws,
                             cudaStream_t stream)
{
    PackedGeo g{};
    UAA_TRY(check_packed(desc, args, ws, true, false, &g));
    return run_packed_append(desc, args, ws, g, stream);
}

uaa_status uaa_packed_attn(const uaa_attn_desc* desc, const uaa_packed_args* args, const uaa_workspace* ws,
                           cudaStream_t stream)
{
    PackedGeo g{};
    UAA_TRY(check_packed(desc, args, ws, false, true, &g));
    return run_packed_attn(desc, args, ws, g, stream);
}

uaa_status uaa_packed_step(const uaa_attn_desc* desc, const uaa_packed_args* args, const uaa_workspace* ws,
                           cudaStream_t stream)
{
    PackedGeo g{};
    if (args && args->step.q_rot) return fail(UAA_ERR_UNSUPPORTED, "q_rot takes the rows of uaa_packed_append alone");
    UAA_TRY(check_packed(desc, args, ws, true, true, &g));
    UAA_TRY(run_packed_append(desc, args, ws, g, stream));
    return run_packed_attn(desc, args, ws, g, stream);
}

uaa_status uaa_packed_read(const uaa_attn_desc* desc, const uaa_packed_args* args, void* k_out, void* v_out,
                           cudaStream_t stream)
{
    UAA_TRY(check_desc(desc));
    if (!args) return fail(UAA_ERR_INVALID_ARGUMENT, "args is NULL");
    UAA_TRY(check_cache(desc, &args->step));
    UAA_TRY(check_plan_arrays(&args->plan, false));
    if (!aligned16(k_out) || !aligned16(v_out))
        return fail(UAA_ERR_INVALID_ARGUMENT, "packed_read outputs must be 16-byte aligned");
    if (args->plan.n_tokens == 0 || (!k_out && !v_out)) return UAA_OK;
    uaa::ReadParams p{};
    p.B = 1;
    p.batch = args->step.batch;
    p.Hkv = desc->n_kv_heads;
    p.D = desc->head_dim;
    p.cap = args->step.cache_capacity;
    p.n = args->plan.n_tokens;
    p.kv_dtype = desc->kv_dtype;
    p.out_dtype = desc->out_dtype;
    p.slots = reinterpret_cast<const long long*>(args->plan.slots);
    p.k_cache = args->step.k_cache;
    p.v_cache = args->step.v_cache;
    p.k_scale = args->step.k_scale;
    p.v_scale = args->step.v_scale;
    p.pages = pages_of(&args->step);
    p.k_out = k_out;
    p.v_out = v_out;
    const cudaError_t e = uaa::launch_cache_read(p, stream);
    return e == cudaSuccess ? UAA_OK : cuda_fail(e, "packed read kernel launch");
}

uaa_status uaa_device_status(const uaa_workspace* ws, cudaStream_t stream, uint32_t* flags)
{
    if (!ws || !ws->ptr || !flags) return fail(UAA_ERR_INVALID_ARGUMENT, "workspace or flags is NULL");
    uint32_t f = 0;
    cudaError_t e = cudaMemcpyAsync(&f, ws->ptr, sizeof f, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && f) e = cudaMemsetAsync(ws->ptr, 0, sizeof f, stream);
    if (e == cudaSuccess && f) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return cuda_fail(e, "reading the device status word");
    *flags = f;
    if (f)
        return fail(UAA_ERR_DEVICE, "device flags 0x%x:%s%s%s%s%s%s", f, (f & UAA_DEVFLAG_CAPACITY) ? " capacity" : "",
                    (f & UAA_DEVFLAG_LEN_HINT) ? " max_seq_len-exceeded" : "",
                    (f & UAA_DEVFLAG_TIMEOUT) ? " wait-timeout" : "", (f & UAA_DEVFLAG_PAGE) ? " page" : "",
                    (f & UAA_DEVFLAG_POOL) ? " pool-exhausted" : "",
                    (f & UAA_DEVFLAG_TOKENS) ? " more-tokens-than-rows" : "");
    return UAA_OK;
}

const char* uaa_last_error(void) { return g_err; }

const char* uaa_status_string(uaa_status s)
{
    switch (s) {
    case UAA_OK: return "UAA_OK";
    case UAA_ERR_INVALID_ARGUMENT: return "UAA_ERR_INVALID_ARGUMENT";
    case UAA_ERR_UNSUPPORTED: return "UAA_ERR_UNSUPPORTED";
    case UAA_ERR_CAPACITY: return "UAA_ERR_CAPACITY";
    case UAA_ERR_CUDA: return "UAA_ERR_CUDA";
    case UAA_ERR_DEVICE: return "UAA_ERR_DEVICE";
    }
    return "UAA_UNKNOWN_STATUS";
}

int32_t uaa_abi_version(void) { return UAA_ABI_VERSION; }

}  // extern "C"

// ---------------------------------------------------------------- built-in scratch
// For callers that cannot allocate device memory: the workspace of
// uaa_decode_attn_static is this array. In host code the name is only a
// host-side stand-in, so the device address is looked up once per device
// (cudaGetSymbolAddress, device current) and handed to the kernels.
static __device__ __align__(256) unsigned char g_static_scratch[UAA_STATIC_SCRATCH_BYTES];

namespace {

std::mutex g_static_scratch_mu;
void* g_static_scratch_addr[64] = {};
// per device: a call launched the partial kernel but not the combine that frees
// its range slots, so the next call starts the scheduling state over
bool g_static_scratch_dirty[64] = {};

uaa_status static_scratch_address(void** out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= 64) return fail(UAA_ERR_UNSUPPORTED, "device index %d is above 63", dev);
    std::lock_guard<std::mutex> lock(g_static_scratch_mu);
    if (!g_static_scratch_addr[dev]) {
        void* p = nullptr;
        e = cudaGetSymbolAddress(&p, g_static_scratch);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress of the built-in scratch");
        g_static_scratch_addr[dev] = p;
    }
    *out = g_static_scratch_addr[dev];
    return UAA_OK;
}

}  // namespace

extern "C" uaa_status uaa_decode_attn_static(const uaa_attn_desc* desc, const uaa_step_args* args,
                                             cudaStream_t stream)
{
    UAA_TRY(check_desc(desc));
    if (!args) return fail(UAA_ERR_INVALID_ARGUMENT, "args is NULL");
    const int n_sm = device_sm_count();
    if (n_sm <= 0) return fail(UAA_ERR_CUDA, "no CUDA device: the SM count query failed");
    Plan pl{};
    UAA_TRY(make_plan(desc, args->batch, args->q_len, args->max_seq_len, n_sm, &pl));
    if (pl.total > (size_t)UAA_STATIC_SCRATCH_BYTES)
        return fail(UAA_ERR_INVALID_ARGUMENT,
                    "this step needs %zu bytes of scratch; the built-in scratch of uaa_decode_attn_static "
                    "holds %zu bytes (pass a workspace to uaa_decode_attn instead)",
                    pl.total, (size_t)UAA_STATIC_SCRATCH_BYTES);
    void* scratch = nullptr;
    UAA_TRY(static_scratch_address(&scratch));
    const uaa_workspace ws{scratch, (size_t)UAA_STATIC_SCRATCH_BYTES};
    UAA_TRY(check_args(desc, args, &ws, true));
    UAA_TRY(check_stages(desc, args, pl));
    if (args->batch == 0) return UAA_OK;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    // Every call starts from a clear status word and arrival counter (the first 8
    // bytes: a launch whose bounded wait gave up may leave the counter short of
    // its wrap). After a call that launched the partial kernel without its
    // combine, the range slots stay claimed: clear the balance state too.
    const size_t clear = g_static_scratch_dirty[dev] ? pl.off_qrot : 2 * sizeof(uint32_t);
    e = cudaMemsetAsync(static_cast<char*>(scratch) + pl.off_status, 0, clear, stream);
    if (e != cudaSuccess) return cuda_fail(e, "clearing the built-in scratch state");
    g_static_scratch_dirty[dev] = true;
    UAA_TRY(run_step(desc, args, &ws, pl, stream));
    g_static_scratch_dirty[dev] = false;
    return UAA_OK;
}
