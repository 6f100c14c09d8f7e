// Host side of the paged key/value cache and the attention over it (k_kv.h,
// k_attend.h): argument checks, launch shapes.
#include "w4a4.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <numeric>

#include "abi.h"
#include "common.h"
#include "k_attend.h"
#include "k_kv.h"

using namespace w4a4;

namespace {

constexpr int64_t kMaxSeqs = 65536, kMaxHeads = 8192, kMax31 = (int64_t{1} << 31) - 1;
constexpr double kLog2e = 1.4426950408889634;
constexpr int64_t kMaxTokens = int64_t{1} << 30;  // of a sequence: block ends stay within 31 bits

inline bool known(w4a4_dtype t) { return t == W4A4_DTYPE_F32 || t == W4A4_DTYPE_F16 || t == W4A4_DTYPE_BF16; }
inline bool known16(w4a4_dtype t) { return t == W4A4_DTYPE_F16 || t == W4A4_DTYPE_BF16; }
inline int64_t size_of(w4a4_dtype t) { return t == W4A4_DTYPE_F32 ? 4 : 2; }

inline bool geometry_valid(int64_t pages, int64_t page, int64_t heads, int64_t dim) {
    return pages >= 0 && pages <= kMax31 && page > 0 && page <= kMaxTokens && page % KV_BLOCK == 0 && heads > 0 && heads <= kMaxHeads &&
           (dim == 64 || dim == 128 || dim == 256) && pages * heads <= kMax31 && pages * heads * (page / KV_BLOCK) <= kMax31;
}

// Sizes of a call, before anything is known of its pointers.
bool sizes_valid(const w4a4_kv_cache *c, const w4a4_kv_batch *s) {
    return c && s && geometry_valid(c->pages, c->page, c->heads, c->dim) && s->seqs >= 0 && s->seqs <= kMaxSeqs && s->rows >= 0 &&
           s->rows <= kMaxRows && s->pages_per_seq >= 0 && s->pages_per_seq <= kMaxTokens / c->page && s->ld >= s->pages_per_seq &&
           s->ld <= kMax31;
}
inline bool no_work(const w4a4_kv_batch *s) { return s->rows == 0 || s->seqs == 0; }

// The pointers of a call with work to do.
w4a4_status check_batch(const w4a4_kv_cache *c, const w4a4_kv_batch *s) {
    if (!s->starts || !s->lens || (s->pages_per_seq && !s->pages) || (c->pages && (!c->codes || !c->scales))) return W4A4_ERR_INVALID_VALUE;
    if (!aligned(s->starts, 4) || !aligned(s->lens, 4) || !aligned(s->pages, 4) || !aligned(c->codes, 16) || !aligned(c->scales, 2))
        return W4A4_ERR_MISALIGNED;
    return W4A4_OK;
}

// Inputs: strides that are not negative and reach no further than 2^62 elements.
bool strides_valid(const w4a4_head_rows *x) {
    constexpr int64_t most = int64_t{1} << 40;
    return x->row_stride >= 0 && x->row_stride <= most && x->head_stride >= 0 && x->head_stride <= most;
}
// Outputs: rows within a head's, or heads within a row's, and none over another.
bool apart(const w4a4_head_rows *x, int64_t rows, int64_t heads, int64_t dim) {
    if (!strides_valid(x)) return false;
    const int64_t r = rows > 1 ? x->row_stride : 0, h = heads > 1 ? x->head_stride : 0;
    if ((rows > 1 && r < dim) || (heads > 1 && h < dim)) return false;
    return rows <= 1 || heads <= 1 || r >= (heads - 1) * h + dim || h >= (rows - 1) * r + dim;
}

KvPool pool_of(const w4a4_kv_cache *c) {
    return KvPool{static_cast<uint8_t *>(c->codes), c->scales, (int32_t)c->pages, (int32_t)c->heads, (int32_t)(c->page / KV_BLOCK)};
}
KvBatch batch_of(const w4a4_kv_batch *s) {
    return KvBatch{s->pages, s->starts, s->lens, s->ld, (int32_t)s->pages_per_seq, (int32_t)s->seqs, (int32_t)s->rows};
}
// At least the blocks that a batch's rows reach: one row reaches one, a second may
// reach another, and each 32 more one more.
int64_t block_bound(const w4a4_kv_batch *s) {
    const int64_t some = std::min(s->seqs, s->rows), more = s->rows - some;
    return some + std::min(more, some) + std::max<int64_t>(more - some, 0) / KV_BLOCK;
}

template <class F>
void with_dim(int64_t dim, F f) {
    if (dim == 64) f(std::integral_constant<int, 64>{});
    else if (dim == 128) f(std::integral_constant<int, 128>{});
    else f(std::integral_constant<int, 256>{});
}

// How attention runs for these sizes.
struct Plan {
    int rows;         // of a tile
    int waves;        // of a tile's rows, in a workgroup of many rows; 0: few rows, streamed
    int64_t tiles;    // of all sequences, at most
    int64_t workers;  // few rows: 0, a workgroup a tile and head, or the workgroups that share all
    int64_t splits;   // many rows: workgroups that share a tile's tokens
    int64_t slots(int64_t heads) const { return waves ? (splits > 1 ? tiles * heads * splits : 0) : 2 * workers; }
};
// Tiles of all sequences, at most: n rows of `group` heads have at most (n group +
// tile - g) / tile, g the largest common divisor.
int64_t tile_bound(int64_t rows, int64_t seqs, int64_t group, int64_t tile) {
    return (rows * group + std::min(rows, seqs) * (tile - std::gcd(group, tile))) / tile;
}
Plan plan_of(int64_t rows, int64_t seqs, int64_t q_heads, int64_t heads, int64_t dim, int64_t tokens) {
    const int64_t group = q_heads / heads;
    Plan p{};
    if (rows * group <= 32 * seqs) {
        p.rows = rows * group <= 16 * seqs ? 16 : 32, p.splits = 1;
        p.tiles = tile_bound(rows, seqs, group, p.rows);
        const int64_t steps = (tokens + STREAM_PAIR - 1) / STREAM_PAIR, tasks = p.tiles * heads;
        // A workgroup a tile and head, or all steps shared evenly and joined (us).  Measured:
        // a wave's step 1.3 us at D = 256, 0.9 at 128, 0.6 at 64; 5 TB/s with all CUs at work;
        // start and end 8, or 13 with a join, and 0.03 a task joined.  Sequences of other
        // lengths than the longest cost the first kind more than this knows: 14 us or less is
        // taken as it is, and a quarter more than the second, up to 512 tasks.  With those the
        // CUs have more than one each and even out by themselves: 66 sequences of up to 8192
        // tokens (8 heads of 256) 218 us, shared 243; 160 (8 of 64) 144 and 211; 50 of up to
        // 16384 (8 of 128), 400 tasks, 177 shared.
        const double bytes_us = (double)(std::min(rows, seqs) * tokens * heads * 2 * dim) / 5e6;
        const double step_us = (dim == 256 ? 1.3 : dim == 128 ? 0.9 : 0.6) * (p.rows == 32 ? 1.6 : 1.0);
        const double rounds = (double)((tasks + 256 * (512 / dim) - 1) / (256 * (512 / dim)));
        const double whole = 8 + std::max(rounds * std::ceil((double)steps / STREAM_WAVES) * step_us, bytes_us);
        const double shared = 13 + bytes_us + 0.03 * (double)tasks;
        if (steps > STREAM_LEAST && whole > 14 && shared < (tasks >= 512 ? 1.0 : 1.25) * whole)
            p.workers = std::min<int64_t>(STREAM_WORKERS, tasks * (steps / STREAM_LEAST + 1));
        return p;
    }
    // The waves of a workgroup over rows or over tokens, and tiles whole or split: the
    // least of what the rounds of workgroups would take (us), by a workgroup's start and
    // end and its waves' blocks of tokens, and what the partial sums would, written and read.
    // Measured: a block with all CUs at work 1.9 us at D = 256 and 1.2 at 128, two waves a
    // SIMD, 0.85 and with two workgroups a CU 1.45 at 64, an eighth more where four waves
    // take four blocks in turns; start and end 13, joining 4 and 0.45 a split.
    double best = 1e30;
    const double blocks = (double)((tokens + KV_BLOCK - 1) / KV_BLOCK);
    const int64_t slots = dim == 64 ? 512 : 256;
    for (int waves = 8; waves >= 2; waves /= 2) {
        const int64_t tiles = tile_bound(rows, seqs, group, 32 * waves), tasks = tiles * heads;
        for (int64_t splits = 1; splits <= SPLITS_MOST; splits++) {
            if (splits > 1 && (tasks * splits > 1024 || blocks < 4 * (double)splits)) break;
            const int64_t all = tasks * splits;
            const double block = (dim == 256 ? 1.9 : dim == 128 ? 1.2 : all > 256 ? 1.45 : 0.85) * (waves == 2 ? 1.13 : 1.0);
            double us = (double)((all + slots - 1) / slots) * (13 + std::ceil(blocks / (double)splits * waves / 8) * block);
            if (splits > 1) us += 4 + 0.45 * (double)splits + (double)(all * 32 * waves * dim * 8) / 8e6;
            if (us < best) best = us, p = Plan{32 * waves, waves, tiles, 0, splits};
        }
    }
    return p;
}
size_t part_bytes(const Plan &p, int64_t heads, int64_t dim) { return (size_t)(p.slots(heads) * p.rows * dim * 4); }
size_t ml_bytes(const Plan &p, int64_t heads) { return (size_t)(p.slots(heads) * p.rows * 8); }
size_t workspace_of(const Plan &p, int64_t heads, int64_t dim) {
    return p.slots(heads) ? up256_bytes(part_bytes(p, heads, dim)) + up256_bytes(ml_bytes(p, heads)) : 0;
}

// With a window a tile's rows see fewer tokens; the workspace is as the sizes alone have it.
Plan plan_of(int64_t rows, int64_t seqs, int64_t q_heads, int64_t heads, int64_t dim, int64_t tokens, int64_t window) {
    const Plan all = plan_of(rows, seqs, q_heads, heads, dim, tokens);
    if (!window || window >= tokens) return all;
    const Plan less = plan_of(rows, seqs, q_heads, heads, dim, std::min(tokens, window + 3 * KV_BLOCK));
    return workspace_of(less, heads, dim) <= workspace_of(all, heads, dim) ? less : all;
}
bool plan_sizes_valid(int64_t rows, int64_t seqs, int64_t q_heads, int64_t heads, int64_t dim, int64_t tokens) {
    return rows >= 0 && rows <= kMaxRows && seqs >= 0 && seqs <= kMaxSeqs && geometry_valid(0, KV_BLOCK, heads, dim) && q_heads >= heads &&
           q_heads <= kMaxHeads && q_heads % heads == 0 && tokens >= 0 && tokens <= kMaxTokens;
}

template <int D, bool BF16, int NR>
void launch_stream(const AttendArgs &a, const Plan &p, hipStream_t s) {
    const unsigned tasks = (unsigned)(p.tiles * a.pool.heads);
    attend_stream_kernel<D, BF16, NR><<<p.workers ? (unsigned)p.workers : tasks, 64 * STREAM_WAVES, 0, s>>>(a);
    if (p.workers) attend_join_kernel<D, 16 * NR><<<dim3(tasks, 16 * NR), 64 * STREAM_WAVES, 0, s>>>(a);
}
template <int D, bool BF16, int RW>
void launch_tile(const AttendArgs &a, const Plan &p, hipStream_t s) {
    using C = AttTile<D, RW>;
    const unsigned tasks = (unsigned)(p.tiles * a.pool.heads);
    attend_tile_kernel<C, BF16><<<tasks * (unsigned)p.splits, C::THREADS, 0, s>>>(a);
    if (p.splits > 8) attend_splits_kernel<D, C::ROWS, 4><<<dim3(tasks, C::ROWS), 256, 0, s>>>(a);
    else if (p.splits > 1) attend_splits_kernel<D, C::ROWS, 1><<<dim3(tasks, C::ROWS / 4), 256, 0, s>>>(a);
}
template <int D, bool BF16>
void launch_attend(const AttendArgs &a, const Plan &p, hipStream_t s) {
    switch (p.waves) {
    case 0: return p.rows == 16 ? launch_stream<D, BF16, 1>(a, p, s) : launch_stream<D, BF16, 2>(a, p, s);
    case 2: return launch_tile<D, BF16, 2>(a, p, s);
    case 4: return launch_tile<D, BF16, 4>(a, p, s);
    default: return launch_tile<D, BF16, 8>(a, p, s);
    }
}

}  // namespace

extern "C" {

size_t w4a4_kv_cache_code_bytes(int64_t pages, int64_t page, int64_t heads, int64_t dim) {
    return geometry_valid(pages, page, heads, dim) ? (size_t)(pages * heads * page * 2 * dim) : 0;
}

size_t w4a4_kv_cache_scale_bytes(int64_t pages, int64_t page, int64_t heads, int64_t dim) {
    return geometry_valid(pages, page, heads, dim) ? (size_t)(pages * heads * (page / KV_BLOCK) * 2) : 0;
}

w4a4_status w4a4_append_kv(w4a4_dtype dt, const w4a4_head_rows *k, const w4a4_head_rows *v, const w4a4_head_rows *q,
                           int64_t q_heads, const w4a4_head_rows *q_out, w4a4_dtype odt, const float *q_weight,
                           const float *k_weight, double eps, const w4a4_rope *rope, const w4a4_kv_cache *cache,
                           const w4a4_kv_batch *batch, void *stream) {
    const bool queries = q && q->data;
    if (!known(dt) || (queries && !known16(odt))) return W4A4_ERR_UNSUPPORTED_DTYPE;
    if (!sizes_valid(cache, batch) || !k || !v || q_heads < 0 || q_heads > kMaxHeads) return W4A4_ERR_INVALID_VALUE;
    const int64_t rows = batch->rows, dim = cache->dim;
    if (queries != (q_out && q_out->data) || !strides_valid(k) || !strides_valid(v)) return W4A4_ERR_INVALID_VALUE;
    if (queries && (q_heads == 0 || !strides_valid(q) || !apart(q_out, rows, q_heads, dim))) return W4A4_ERR_INVALID_VALUE;
    // in place: the same elements only
    if (queries && q->data == q_out->data &&
        (odt != dt || (rows > 1 && q->row_stride != q_out->row_stride) || (q_heads > 1 && q->head_stride != q_out->head_stride)))
        return W4A4_ERR_INVALID_VALUE;
    if ((q_weight || k_weight) && (!(eps > 0.0) || !std::isfinite(eps))) return W4A4_ERR_INVALID_VALUE;
    if (rope) {
        if (rope->width <= 0 || rope->width > dim || rope->width % 16 || rope->table_rows < 0 || rope->table_rows > kMax31 ||
            (rope->axes && (!rope->positions || rope->n_axes > 256)) || (rope->positions && rope->n_axes < 1) || (!rope->axes && rope->n_axes > 1) ||
            (rope->positions && rope->axes && rope->n_axes > 1 && rope->ld < rows) || rope->ld < 0)
            return W4A4_ERR_INVALID_VALUE;
    }
    const int64_t blocks = block_bound(batch) * cache->heads, threads = kv_threads((int)dim);
    if (blocks > kMax31 || !grid_fits(blocks * threads + rows * ((q_heads * dim / 8 + 63) / 64 * 64) + threads)) return W4A4_ERR_INVALID_VALUE;
    if (no_work(batch)) return W4A4_OK;
    if (!k->data || !v->data || (rope && !rope->table && rope->table_rows)) return W4A4_ERR_INVALID_VALUE;
    const w4a4_status st = check_batch(cache, batch);
    if (st != W4A4_OK) return st;
    if (!aligned(k->data, size_of(dt)) || !aligned(v->data, size_of(dt)) || (queries && (!aligned(q->data, size_of(dt)) || !aligned(q_out->data, 2))) ||
        !aligned(q_weight, 4) || !aligned(k_weight, 4) || (rope && (!aligned(rope->table, 4) || !aligned(rope->positions, 4))))
        return W4A4_ERR_MISALIGNED;

    AppendArgs a{};
    a.k = static_cast<const uint8_t *>(k->data), a.k_row = k->row_stride, a.k_head = k->head_stride;
    a.v = static_cast<const uint8_t *>(v->data), a.v_row = v->row_stride, a.v_head = v->head_stride;
    if (queries) {
        a.q = static_cast<const uint8_t *>(q->data), a.q_row = q->row_stride, a.q_head = q->head_stride;
        a.q_out = static_cast<uint8_t *>(q_out->data), a.o_row = q_out->row_stride, a.o_head = q_out->head_stride;
    }
    a.q_weight = q_weight, a.k_weight = k_weight, a.eps = eps, a.dt = dt, a.odt = odt, a.q_heads = queries ? (int32_t)q_heads : 0;
    if (rope) {
        a.rope = rope->table, a.rope_rows = (int32_t)rope->table_rows, a.half = (int32_t)(rope->width / 2);
        a.positions = rope->positions, a.ld_positions = rope->ld, a.axes = rope->axes, a.n_axes = (int32_t)rope->n_axes;
        a.interleaved = rope->interleaved != 0;
    }
    a.pool = pool_of(cache), a.batch = batch_of(batch), a.kv_groups = (int32_t)blocks;
    // heads of a wave: steps of 512 / dim, as many as leave every CU 8 waves
    const int64_t step = 512 / dim, steps = queries ? (q_heads + step - 1) / step : 0;
    const int64_t passes = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(steps, 8), rows * steps / 2048));
    const int64_t tasks = rows * ((steps + passes - 1) / passes);
    a.q_passes = (int32_t)passes;
    const unsigned grid = (unsigned)(blocks + (tasks * 64 + threads - 1) / threads);
    with_dim(dim, [&](auto d) { append_kernel<decltype(d)::value><<<grid, (unsigned)threads, 0, as_stream(stream)>>>(a); });
    return hip_status("append_kernel");
}

w4a4_status w4a4_read_kv(const w4a4_kv_cache *cache, const w4a4_kv_batch *batch, w4a4_dtype dt, const w4a4_head_rows *k,
                         const w4a4_head_rows *v, void *stream) {
    if (!known(dt)) return W4A4_ERR_UNSUPPORTED_DTYPE;
    if (!sizes_valid(cache, batch) || !k || !v) return W4A4_ERR_INVALID_VALUE;
    if (!apart(k, batch->rows, cache->heads, cache->dim) || !apart(v, batch->rows, cache->heads, cache->dim)) return W4A4_ERR_INVALID_VALUE;
    const int64_t blocks = block_bound(batch) * cache->heads;
    const int64_t threads = kv_threads((int)cache->dim);
    if (blocks > kMax31 || !grid_fits(blocks * threads)) return W4A4_ERR_INVALID_VALUE;
    if (no_work(batch)) return W4A4_OK;
    if (!k->data || !v->data) return W4A4_ERR_INVALID_VALUE;
    const w4a4_status st = check_batch(cache, batch);
    if (st != W4A4_OK) return st;
    if (!aligned(k->data, size_of(dt)) || !aligned(v->data, size_of(dt))) return W4A4_ERR_MISALIGNED;
    const KvReadArgs a{pool_of(cache), batch_of(batch), static_cast<uint8_t *>(k->data), static_cast<uint8_t *>(v->data),
                       k->row_stride, k->head_stride, v->row_stride, v->head_stride, dt};
    with_dim(cache->dim, [&](auto d) { read_kv_kernel<decltype(d)::value><<<(unsigned)blocks, (unsigned)threads, 0, as_stream(stream)>>>(a); });
    return hip_status("read_kv_kernel");
}

size_t w4a4_attention_kv_workspace_bytes(int64_t rows, int64_t seqs, int64_t q_heads, int64_t heads, int64_t dim,
                                         int64_t tokens) {
    if (!plan_sizes_valid(rows, seqs, q_heads, heads, dim, tokens) || rows == 0 || seqs == 0) return 0;
    return workspace_of(plan_of(rows, seqs, q_heads, heads, dim, tokens), heads, dim);
}

size_t w4a4_attention_kv_plan(int64_t rows, int64_t seqs, int64_t q_heads, int64_t heads, int64_t dim, int64_t tokens,
                              int64_t window, char *text, size_t bytes) {
    if (!text) bytes = 0;
    if (bytes) text[0] = 0;
    if (!plan_sizes_valid(rows, seqs, q_heads, heads, dim, tokens) || window < 0 || rows == 0 || seqs == 0) return 0;
    const Plan p = plan_of(rows, seqs, q_heads, heads, dim, tokens, window);
    int len;
    if (p.waves && p.splits > 1) len = std::snprintf(text, bytes, "tile %d split %d", p.rows, (int)p.splits);
    else if (p.workers) len = std::snprintf(text, bytes, "stream %d shared %d", p.rows, (int)p.workers);
    else len = std::snprintf(text, bytes, "%s %d", p.waves ? "tile" : "stream", p.rows);
    return (size_t)len;
}

w4a4_status w4a4_attention_kv(const w4a4_head_rows *q, w4a4_dtype dt, int64_t q_heads, const w4a4_head_rows *out,
                              w4a4_dtype odt, float *lse, int64_t ld_lse, double scale, int causal, int64_t window,
                              const w4a4_kv_cache *cache, const w4a4_kv_batch *batch, void *workspace,
                              size_t workspace_bytes, void *stream) {
    if (!known16(dt) || !known16(odt)) return W4A4_ERR_UNSUPPORTED_DTYPE;
    if (!sizes_valid(cache, batch) || !q || !out || q_heads < cache->heads || q_heads > kMaxHeads || q_heads % cache->heads)
        return W4A4_ERR_INVALID_VALUE;
    const int64_t rows = batch->rows, dim = cache->dim;
    if (!(scale > 0.0) || !std::isfinite((float)(scale * kLog2e)) || window < 0 || !strides_valid(q) || !apart(out, rows, q_heads, dim) ||
        (lse && ld_lse < q_heads))
        return W4A4_ERR_INVALID_VALUE;
    if (q->data && q->data == out->data &&
        (odt != dt || (rows > 1 && q->row_stride != out->row_stride) || (q_heads > 1 && q->head_stride != out->head_stride)))
        return W4A4_ERR_INVALID_VALUE;
    const int64_t tokens = batch->pages_per_seq * cache->page, heads = cache->heads;
    const int64_t some_rows = std::max<int64_t>(rows, 1), some_seqs = std::max<int64_t>(batch->seqs, 1);
    const Plan p = plan_of(some_rows, some_seqs, q_heads, heads, dim, tokens, window);
    if (p.tiles > kMax31 / heads || !grid_fits(p.tiles * heads * p.splits * 512)) return W4A4_ERR_INVALID_VALUE;
    if (no_work(batch)) return W4A4_OK;
    if (!q->data || !out->data) return W4A4_ERR_INVALID_VALUE;
    const size_t need = workspace_of(plan_of(rows, batch->seqs, q_heads, heads, dim, tokens), heads, dim);
    if (need && !workspace) return W4A4_ERR_INVALID_VALUE;
    const w4a4_status st = check_batch(cache, batch);
    if (st != W4A4_OK) return st;
    if (!aligned(q->data, 2) || !aligned(out->data, 2) || !aligned(lse, 4) || (need && !aligned(workspace, 256))) return W4A4_ERR_MISALIGNED;
    if (workspace_bytes < need) return W4A4_ERR_WORKSPACE_TOO_SMALL;

    AttendArgs a{};
    a.q = static_cast<const uint8_t *>(q->data), a.q_row = q->row_stride, a.q_head = q->head_stride;
    a.out = static_cast<uint8_t *>(out->data), a.o_row = out->row_stride, a.o_head = out->head_stride;
    a.lse = lse, a.lse_row = ld_lse, a.scale_log2 = (float)(scale * kLog2e);
    a.heads = (int32_t)q_heads, a.group = (int32_t)(q_heads / cache->heads), a.causal = causal != 0;
    a.window = (int32_t)std::min<int64_t>(window, kMax31), a.odt = odt;
    a.pool = pool_of(cache), a.batch = batch_of(batch);
    if (!cache->pages) a.batch.per_seq = 0;  // no block at all: none may stand in for one that a sequence lacks
    a.part = static_cast<float *>(workspace), a.tile_bound = (int32_t)p.tiles;
    a.workers = (int32_t)p.workers, a.splits = (int32_t)p.splits;
    if (p.slots(heads)) a.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + up256_bytes(part_bytes(p, heads, dim)));
    hipStream_t s = as_stream(stream);
    with_dim(dim, [&](auto d) {
        constexpr int D = decltype(d)::value;
        dt == W4A4_DTYPE_BF16 ? launch_attend<D, true>(a, p, s) : launch_attend<D, false>(a, p, s);
    });
    return hip_status("attend_kernel");
}

}  // extern "C"
