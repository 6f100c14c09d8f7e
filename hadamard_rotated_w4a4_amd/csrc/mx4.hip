// Host side of the MXFP4 product (k_mx4.h): argument checks, launch shapes.
#include "w4a4.h"

#include <algorithm>
#include <cstdint>
#include <cstdio>

#include "abi.h"
#include "common.h"
#include "k_mx4.h"

using namespace w4a4;

extern "C" {

size_t w4a4_mx4_packed_bytes(int64_t n, int64_t k) {
    if (n < 0 || k < 0 || k % QK || !within_bounds(0, n, k)) return 0;
    return (size_t)mx4_packed_bytes(n, k);
}

w4a4_status w4a4_repack_mx4(const uint8_t *codes, const uint8_t *scales, int64_t n, int64_t k, void *packed,
                            void *stream) {
    if (n < 0 || k < 0 || !within_bounds(0, n, k)) return W4A4_ERR_INVALID_VALUE;
    if (k % QK) return W4A4_ERR_K_NOT_MULTIPLE_OF_32;
    if (n == 0 || k == 0) return W4A4_OK;
    if (!codes || !scales || !packed) return W4A4_ERR_INVALID_VALUE;
    const int64_t threads = padded_n(n) / TILE_N * mx4_rec_stages(k) * 64;
    if (!grid_fits(threads + 256)) return W4A4_ERR_INVALID_VALUE;
    if (!aligned(codes, 16) || !aligned(scales, 8) || !aligned(packed, 16)) return W4A4_ERR_MISALIGNED;
    repack_mx4_kernel<<<blocks_for(threads, 256), 256, 0, as_stream(stream)>>>(codes, scales, n, k,
                                                                              static_cast<uint8_t *>(packed));
    return hip_status("repack_mx4_kernel");
}

}  // extern "C"

namespace {

// The streaming kernels: up to 16, 32 or 64 rows a block, waves, records in
// flight, LDS share in KB.  Measured: 16 rows, 8 waves for K up to 5120 and 16 past
// it, where the two cross at every width tried (weights from memory, us with 8 and
// 16 waves: 1024 columns 4.3 and 4.4 at K 4096, 4.7 and 4.7 at 5120, 6.2 and 5.4 at
// 7168; 5120 columns 5.7 and 5.8, 6.7 and 6.6, 9.2 and 8.0; 17408 columns 11.3 and
// 11.7, 14.0 and 13.7, 18.1 and 17.5); 32 rows, 16 waves with a CU's whole LDS while every
// column tile has a CU (5120 x 8192 8.2 us against 10.2), else 8 (17408 x 5120
// 13.7 us against 16.5).
using Stream16 = Mx4Stream<16, 8, 2, 52>;
using Stream16LongK = Mx4Stream<16, 16, 2, 78>;
using Stream32 = Mx4Stream<32, 8, 2, 53>;
using Stream32Few = Mx4Stream<32, 16, 2, 144>;
using Stream64Few = Mx4Stream<64, 16, 1, 144>;
constexpr int64_t kPlanCus = 256;  // the plans are pure functions of the sizes: the workspace's size depends on them

template <class C>
void launch_stream(const Mx4Args &a, hipStream_t s) {
    const dim3 grid((unsigned)(padded_n(a.n) / TILE_N), (unsigned)((a.m + C::ROWS - 1) / C::ROWS));
    gemm_mx4_stream_kernel<C><<<grid, C::NT, mx4_stream_lds<C>(a.k), s>>>(a);
}
// m past 32 streams only while every (block of 64 rows, column tile) has a CU of
// its own: then it needs no records of the rows and no second launch (64 x
// 1024 x 5120 7.0 us against 12.5 tiled, 64 x 5120 x 17408 23 against 29), but
// with several workgroups on a CU the tiles' reuse wins (64 x 17408 x 5120 21
// against 16).
bool streams(int64_t m, int64_t n) { return m <= 32 || (m + 63) / 64 * (padded_n(n) / TILE_N) <= kPlanCus; }
struct StreamShape {
    int rows, waves;
    void (*launch)(const Mx4Args &, hipStream_t);
};
template <class C>
constexpr StreamShape stream_shape() {
    return StreamShape{C::ROWS, C::WAVES, launch_stream<C>};
}
StreamShape stream_plan(int64_t m, int64_t n, int64_t k) {
    if (m > 32) return stream_shape<Stream64Few>();
    if (m > 16) return padded_n(n) / TILE_N <= kPlanCus ? stream_shape<Stream32Few>() : stream_shape<Stream32>();
    return k > 5120 ? stream_shape<Stream16LongK>() : stream_shape<Stream16>();
}

// Tile shapes of the tiled product.
using T64x64 = Mx4Cfg<2, 2, 1, 1, 2, 3>;
using T64x128 = Mx4Cfg<2, 4, 1, 1, 2, 3>;
using T128x128 = Mx4Cfg<2, 4, 2, 1, 1, 4>;
using T160x128 = Mx4Cfg<5, 2, 1, 2, 1, 4>;
using T256x192 = Mx4Cfg<4, 2, 2, 3, 1, 4>;
using T256x256 = Mx4Cfg<4, 2, 2, 4, 1, 4>;

template <class C>
void launch_tile(const Mx4Args &a, hipStream_t s) {
    const int64_t tiles = (a.m + C::BM - 1) / C::BM * a.columns * a.splits;
    gemm_mx4_tile_kernel<C><<<(unsigned)tiles, C::NT, 0, s>>>(a);
}

// What the plan knows of a shape: its size, how many workgroups a CU holds (the
// LDS rings decide, but for 160 x 128: two of its rings fit, and its registers
// leave 4 waves a SIMD where two workgroups of 10 waves need 5), and the measured
// time of one stage (128 of K), in us, of a workgroup on an otherwise idle chip
// and of a full round.
struct TileShape {
    int64_t bm, bn, per_cu;
    double alone, full;
    void (*launch)(const Mx4Args &, hipStream_t);
};
template <class C>
constexpr TileShape shape(int64_t per_cu, double alone, double full) {
    return TileShape{C::BM, C::BN, per_cu, alone, full, launch_tile<C>};
}
const TileShape kShapes[] = {shape<T64x64>(3, 0.15, 0.36), shape<T64x128>(2, 0.21, 0.50), shape<T128x128>(2, 0.40, 0.80),
                             shape<T160x128>(1, 0.34, 0.56), shape<T256x192>(1, 0.74, 1.00),
                             shape<T256x256>(1, 0.86, 1.30)};

// Modelled time of one launch: rounds of resident workgroups; a partial round
// lies between the two times by how much of the chip it fills.
double tiles_time(const TileShape &t, int64_t tiles, double stages) {
    const int64_t slots = kPlanCus * t.per_cu, whole = tiles / slots, left = tiles % slots;
    const double last = left == 0 ? 0.0 : t.alone + (t.full - t.alone) * (double)left / (double)slots;
    return ((double)whole * t.full + last) * stages;
}

// The tiled product's launches: shape `a` over the first `columns` of its
// column tiles with `splits` K splits, then shape `b` over the rest (none: -1).
// The least modelled time wins.  Both sides, measured: 302 x 5120 x 17408 64 x 64
// 35.0 us, three splits of 160 x 128 35.5, 64 x 64 in two splits 43.2; 140 x 10240
// x 17408 three splits of 160 x 128 39.0, 64 x 128 41.0, 64 x 64 43.1; 512 x 34816
// x 5120 one round of 256 x 256 and the rest in 64 x 64 68 us, all in 256 x 192
// 78; 200 x 17408 x 17408 three splits of 256 x 256 71.8, whole 128 x 128 88.4;
// 2048 x 5120 x 5120 256 x 192 44.2.  Over 14 sizes the choice was 6 % slower than
// the best of the shapes and splits tried on average, 22 % at worst (100 x 17408 x
// 17408); K below about 1024 is where it errs most (up to 15 %).
struct TilePlan {
    int a, b;
    int64_t columns, splits;
};
TilePlan tile_plan(int64_t m, int64_t n, int64_t k) {
    constexpr double kLaunch = 2.5;  // us: a further launch, its start and its outputs' tail
    const double stages = (double)mx4_stages(k);
    TilePlan best{0, -1, 0, 1};
    double best_time = 1e30;
    auto take = [&](double time, TilePlan p) {
        if (time < best_time) best = p, best_time = time;
    };
    for (int i = 0; i < (int)(sizeof kShapes / sizeof kShapes[0]); i++) {
        const TileShape &t = kShapes[i];
        const int64_t rows = (m + t.bm - 1) / t.bm, cols = (n + t.bn - 1) / t.bn;
        take(tiles_time(t, rows * cols, stages), TilePlan{i, -1, cols, 1});
        // K splits: their partial sums (4 bytes, written and read) at 4 TB/s
        for (int64_t s = 2; s <= 8 && stages >= 8.0 * s; s++)
            take(tiles_time(t, rows * cols * s, (double)((mx4_stages(k) + s - 1) / s)) + kLaunch + 8e-6 * s * m * n / 4.0,
                 TilePlan{i, -1, cols, s});
        // whole rounds of this shape, the rest in another
        const int64_t slots = kPlanCus * t.per_cu, first = rows * cols / slots * slots / rows;
        if (first == 0 || first == cols) continue;
        for (int j = 0; j < i; j++) {
            const TileShape &u = kShapes[j];
            const int64_t rest = (m + u.bm - 1) / u.bm * ((n - first * t.bn + u.bn - 1) / u.bn);
            take(tiles_time(t, rows * first, stages) + tiles_time(u, rest, stages) + kLaunch, TilePlan{i, j, first, 1});
        }
    }
    return best;
}

}  // namespace

extern "C" {

size_t w4a4_gemm_mx4_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (m < 0 || n < 0 || k < 0 || k % QK || n == 0 || k == 0 || !within_bounds(m, n, k) || streams(m, n)) return 0;
    const TilePlan p = tile_plan(m, n, k);  // the rows as records, then the splits' partial sums
    return up256_bytes(mx4_packed_bytes(m, k)) + (p.splits > 1 ? up256_bytes(p.splits * m * n * 4) : 0);
}

size_t w4a4_gemm_mx4_plan(int64_t m, int64_t n, int64_t k, char *text, size_t bytes) {
    if (!text) bytes = 0;
    if (bytes) text[0] = 0;
    if (m <= 0 || n <= 0 || k <= 0 || k % QK || !within_bounds(m, n, k)) return 0;
    int len;
    if (streams(m, n)) {
        const StreamShape c = stream_plan(m, n, k);
        len = std::snprintf(text, bytes, "stream %dx%d", c.rows, c.waves);
    } else {
        const TilePlan p = tile_plan(m, n, k);
        const TileShape &a = kShapes[p.a], &b = kShapes[p.b < 0 ? 0 : p.b];
        if (p.b >= 0) len = std::snprintf(text, bytes, "tile %dx%d + %dx%d", (int)a.bm, (int)a.bn, (int)b.bm, (int)b.bn);
        else if (p.splits > 1) len = std::snprintf(text, bytes, "tile %dx%d split %d", (int)a.bm, (int)a.bn, (int)p.splits);
        else len = std::snprintf(text, bytes, "tile %dx%d", (int)a.bm, (int)a.bn);
    }
    return (size_t)len;
}

w4a4_status w4a4_gemm_mx4(const void *packed_w, const uint8_t *codes, const uint8_t *scales, void *y, w4a4_dtype ydt,
                          int64_t m, int64_t n, int64_t k, int64_t ldy, void *workspace, size_t workspace_bytes,
                          void *stream) {
    if (ydt != W4A4_DTYPE_F32 && ydt != W4A4_DTYPE_F16 && ydt != W4A4_DTYPE_BF16) return W4A4_ERR_UNSUPPORTED_DTYPE;
    if (m < 0 || n < 0 || k < 0 || ldy < n || !within_bounds(m, n, k)) return W4A4_ERR_INVALID_VALUE;
    if (k % QK) return W4A4_ERR_K_NOT_MULTIPLE_OF_32;
    if (m == 0 || n == 0) return W4A4_OK;
    if (!y) return W4A4_ERR_INVALID_VALUE;
    if (!aligned(y, ydt == W4A4_DTYPE_F32 ? 4 : 2)) return W4A4_ERR_MISALIGNED;
    hipStream_t s = as_stream(stream);
    if ((m + 127) / 128 * ((n + 127) / 128) >= (int64_t{1} << 20)) return W4A4_ERR_INVALID_VALUE;
    if (k == 0) {  // empty sum
        zero_typed_kernel<<<(unsigned)std::min<int64_t>((m * n + 255) / 256, 1 << 16), 256, 0, s>>>(
            static_cast<uint8_t *>(y), ydt, m, n, ldy);
        return hip_status("zero_typed_kernel");
    }
    if (!packed_w || !codes || !scales) return W4A4_ERR_INVALID_VALUE;
    if (!aligned(packed_w, 16) || !aligned(codes, 16) || !aligned(scales, 8)) return W4A4_ERR_MISALIGNED;
    const size_t need = w4a4_gemm_mx4_workspace_bytes(m, n, k);
    if (need) {
        if (!workspace) return W4A4_ERR_INVALID_VALUE;
        if (!aligned(workspace, 256)) return W4A4_ERR_MISALIGNED;
        if (workspace_bytes < need) return W4A4_ERR_WORKSPACE_TOO_SMALL;
    }
    Mx4Args a{};
    a.packed = static_cast<const uint8_t *>(packed_w);
    a.codes = codes;
    a.scales = scales;
    a.rows = static_cast<const uint8_t *>(workspace);
    a.y = static_cast<uint8_t *>(y);
    a.m = m;
    a.n = n;
    a.k = k;
    a.ldy = ldy;
    a.dt = ydt;
    a.splits = 1;
    if (streams(m, n)) {
        stream_plan(m, n, k).launch(a, s);
        return hip_status("gemm_mx4_stream_kernel");
    }
    const w4a4_status st = w4a4_repack_mx4(codes, scales, m, k, workspace, stream);
    if (st != W4A4_OK) return st;
    const TilePlan p = tile_plan(m, n, k);
    a.columns = p.columns;
    a.splits = p.splits;
    a.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + up256_bytes(mx4_packed_bytes(m, k)));
    kShapes[p.a].launch(a, s);
    if (p.splits > 1) mx4_reduce_kernel<<<blocks_for(m * n, 256), 256, 0, s>>>(a);
    if (p.b >= 0) {
        const TileShape &u = kShapes[p.b];
        a.first = p.columns * kShapes[p.a].bn / TILE_N;
        a.columns = (n - a.first * TILE_N + u.bn - 1) / u.bn;
        u.launch(a, s);
    }
    return hip_status("gemm_mx4_tile_kernel");
}

}  // extern "C"
