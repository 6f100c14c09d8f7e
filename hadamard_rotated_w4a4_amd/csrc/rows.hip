// Host side of the producers of quantised rows (k_rows.h): argument checks,
// launch shapes.
#include "w4a4.h"

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "abi.h"
#include "common.h"
#include "k_rows.h"

using namespace w4a4;

static_assert(W4A4_ACT_INT4 == FMT_INT4 && W4A4_ACT_INT4_SMALL == FMT_INT4_SMALL && W4A4_ACT_INT8 == FMT_INT8 &&
              W4A4_ACT_MX4 == FMT_MX4 && W4A4_ACT_MX4_H32 == FMT_MX4_H32, "the kernels' formats are the ABI's");
static_assert(W4A4_DTYPE_F32 == ROW_F32 && W4A4_DTYPE_F16 == ROW_F16 && W4A4_DTYPE_BF16 == ROW_BF16, "and its types");
static_assert(W4A4_GLU_SILU == GLU_SILU && W4A4_GLU_GELU_TANH == GLU_GELU_TANH, "and its activations");

namespace {

inline bool known(w4a4_dtype t) { return t == W4A4_DTYPE_F32 || t == W4A4_DTYPE_F16 || t == W4A4_DTYPE_BF16; }
inline int64_t size_of(w4a4_dtype t) { return t == W4A4_DTYPE_F32 ? 4 : 2; }
inline bool known_format(int f) { return f >= FMT_INT4 && f <= FMT_MX4_H32; }
// what the size queries take: beyond it no call does, and a size may not fit 64 bits
inline bool sizes_valid(int f, int64_t m, int64_t k) {
    return known_format(f) && m >= 0 && m <= kMaxN && k >= 0 && k <= kMaxK && k % QK == 0;
}
inline bool is_mx4(int f) { return f == FMT_MX4 || f == FMT_MX4_H32; }

// The quantised outputs of a producer: sizes known to be >= 0 and in bounds,
// work to do.
w4a4_status check_outputs(int fmt, const RowsOut &o, size_t act_bytes) {
    if (!o.codes || !o.scales) return W4A4_ERR_INVALID_VALUE;
    if (o.act && is_mx4(fmt)) return W4A4_ERR_INVALID_VALUE;  // MXFP4 rows are their own operand
    if (fmt == FMT_INT4_SMALL && (o.m > SMA_ROWS || !o.act)) return W4A4_ERR_INVALID_VALUE;
    if (!aligned(o.codes, 16) || !aligned(o.scales, is_mx4(fmt) ? 8 : 4) || (o.act && !aligned(o.act, 256)))
        return W4A4_ERR_MISALIGNED;
    if (o.act && act_bytes < w4a4_act_format_operand_bytes(static_cast<w4a4_act_format>(fmt), o.m, o.k))
        return W4A4_ERR_WORKSPACE_TOO_SMALL;
    return W4A4_OK;
}

}  // namespace

extern "C" {

size_t w4a4_mx4_scale_stride(int64_t k) {
    if (k < 0 || k % QK || k > kMaxK) return 0;
    return (size_t)mx4_stride(k);
}

size_t w4a4_act_format_code_bytes(w4a4_act_format fmt, int64_t m, int64_t k) {
    if (!sizes_valid(fmt, m, k)) return 0;
    return (size_t)(fmt == W4A4_ACT_INT8 ? m * k : m * (k / 2));
}

size_t w4a4_act_format_scale_bytes(w4a4_act_format fmt, int64_t m, int64_t k) {
    if (!sizes_valid(fmt, m, k)) return 0;
    return (size_t)(is_mx4(fmt) ? m * mx4_stride(k) : m * (k / QK) * 4);
}

size_t w4a4_act_format_operand_bytes(w4a4_act_format fmt, int64_t m, int64_t k) {
    if (!sizes_valid(fmt, m, k)) return 0;
    switch (fmt) {
    case W4A4_ACT_INT4: return w4a4_act_operand_bytes(m, k);
    case W4A4_ACT_INT4_SMALL: return w4a4_small_act_operand_bytes(m, k);
    case W4A4_ACT_INT8: return w4a4_act8_operand_bytes(m, k);
    default: return 0;
    }
}

w4a4_status w4a4_quantize_mx4(const void *x, w4a4_dtype dt, int64_t m, int64_t k, int64_t ldx, int rotate,
                              uint8_t *codes, uint8_t *scales, void *stream) {
    if (!known(dt)) return W4A4_ERR_UNSUPPORTED_DTYPE;
    if (m < 0 || k < 0 || ldx < k || m > kMaxN || k > kMaxK) return W4A4_ERR_INVALID_VALUE;
    if (k % QK) return W4A4_ERR_K_NOT_MULTIPLE_OF_32;
    if (m == 0 || k == 0) return W4A4_OK;
    if (!x) return W4A4_ERR_INVALID_VALUE;
    const int fmt = rotate ? FMT_MX4_H32 : FMT_MX4;
    PlainArgs a{static_cast<const uint8_t *>(x), ldx, dt, row_blocks(mx4_stride(k)),
                 RowsOut{codes, scales, nullptr, m, k}};
    const int64_t threads = m * mx4_stride(k) * 4;
    if (!grid_fits(threads + ROWS_THREADS)) return W4A4_ERR_INVALID_VALUE;
    const w4a4_status st = check_outputs(fmt, a.out, 0);
    if (st != W4A4_OK) return st;
    if (!aligned(x, size_of(dt))) return W4A4_ERR_MISALIGNED;
    const unsigned grid = blocks_for(threads, ROWS_THREADS);
    hipStream_t s = as_stream(stream);
    if (rotate) quantise_rows_kernel<FMT_MX4_H32><<<grid, ROWS_THREADS, 0, s>>>(a);
    else quantise_rows_kernel<FMT_MX4><<<grid, ROWS_THREADS, 0, s>>>(a);
    return hip_status("quantise_rows_kernel");
}

w4a4_status w4a4_dequantize_act(w4a4_act_format fmt, const void *codes, const void *scales, int64_t m, int64_t k,
                                void *y, w4a4_dtype dt, int64_t ldy, void *stream) {
    if (!known_format(fmt)) return W4A4_ERR_INVALID_VALUE;
    if (!known(dt)) return W4A4_ERR_UNSUPPORTED_DTYPE;
    if (m < 0 || k < 0 || ldy < k || m > kMaxN || k > kMaxK) return W4A4_ERR_INVALID_VALUE;
    if (k % QK) return W4A4_ERR_K_NOT_MULTIPLE_OF_32;
    if (m == 0 || k == 0) return W4A4_OK;
    if (!codes || !scales || !y) return W4A4_ERR_INVALID_VALUE;
    const int64_t threads = m * (k / QK) * 4;
    if (!grid_fits(threads + ROWS_THREADS)) return W4A4_ERR_INVALID_VALUE;
    if (!aligned(codes, 16) || !aligned(scales, is_mx4(fmt) ? 8 : 4) || !aligned(y, size_of(dt)))
        return W4A4_ERR_MISALIGNED;
    const ReadArgs a{static_cast<const uint8_t *>(codes), scales, static_cast<uint8_t *>(y), m, k, ldy, dt,
                     row_blocks(k / QK)};
    const unsigned grid = blocks_for(threads, ROWS_THREADS);
    hipStream_t s = as_stream(stream);
    switch (fmt) {
    case W4A4_ACT_INT8: read_rows_kernel<FMT_INT8><<<grid, ROWS_THREADS, 0, s>>>(a); break;
    case W4A4_ACT_INT4:
    case W4A4_ACT_INT4_SMALL: read_rows_kernel<FMT_INT4><<<grid, ROWS_THREADS, 0, s>>>(a); break;
    default: read_rows_kernel<FMT_MX4><<<grid, ROWS_THREADS, 0, s>>>(a); break;
    }
    return hip_status("read_rows_kernel");
}

}  // extern "C"

namespace {

template <int FMT>
void launch_glu(const GluArgs &a, hipStream_t s) {
    const int64_t rows = rows_covered(FMT, a.out.act != nullptr, a.out.m);
    const int64_t blocks = blocks_covered(FMT, a.out.act != nullptr, a.out.k);
    if constexpr (FMT != FMT_MX4 && FMT != FMT_MX4_H32) {
        if (a.out.act) {
            const dim3 grid((unsigned)((blocks + RQ_BLOCKS - 1) / RQ_BLOCKS), (unsigned)((rows + 31) / 32));
            glu_rows_kernel<FMT, true><<<grid, ROWS_THREADS, 0, s>>>(a);
            return;
        }
    }
    if constexpr (FMT != FMT_INT4_SMALL)  // always has its operand
        glu_rows_kernel<FMT, false><<<blocks_for(rows * blocks * 4, ROWS_THREADS), ROWS_THREADS, 0, s>>>(a);
}

template <int FMT, int CHUNKS>
void launch_norm_chunks(const NormArgs &a, int64_t rows, int64_t threads, hipStream_t s) {
    norm_rows_kernel<FMT, CHUNKS><<<(unsigned)rows, (unsigned)threads, 0, s>>>(a, a.out.act != nullptr);
}
// A row's pieces of 8 elements over a workgroup's threads, in 1, 2 or 4 pieces
// each; rows past 32768 walk twice.  Few rows wait for one row's chain of loads,
// sum and stores: as many threads as a workgroup holds (1 x 5120 3.6 us against
// 4.2 with at most 512).  With two rows a CU and more, rows up to 16384 go to at
// most 512 threads, so that several workgroups share a CU (to int8, from memory:
// 2048 x 16384 64 us against 76 with up to 1024, 512 x 16384 22.0 against 23.4).
// Rows that 1024 threads hold in one piece each do not gain from that: 512 x 5120
// 10.4 us against 9.5, 2048 x 5120 25.1 against 24.0, 2048 x 2048 the same.
template <int FMT>
void launch_norm(const NormArgs &a, hipStream_t s) {
    const int64_t rows = rows_covered(FMT, a.out.act != nullptr, a.out.m);
    const int64_t pieces = blocks_covered(FMT, a.out.act != nullptr, a.out.k) * 4;
    const int64_t most = rows >= 512 && pieces <= 4 * 512 ? 512 : 1024;
    const int64_t chunks = pieces <= most ? 1 : pieces <= 2 * most ? 2 : pieces <= 4 * most ? 4 : 0;
    const int64_t threads = chunks ? ((pieces + chunks - 1) / chunks + 63) / 64 * 64 : 1024;
    switch (chunks) {
    case 1: return launch_norm_chunks<FMT, 1>(a, rows, threads, s);
    case 2: return launch_norm_chunks<FMT, 2>(a, rows, threads, s);
    case 4: return launch_norm_chunks<FMT, 4>(a, rows, threads, s);
    default: return launch_norm_chunks<FMT, 0>(a, rows, threads, s);
    }
}

}  // namespace

extern "C" {

w4a4_status w4a4_glu_quantize(const void *gate, const void *up, w4a4_dtype dt, int64_t m, int64_t k, int64_t ldg,
                              int64_t ldu, w4a4_glu_act act, w4a4_act_format fmt, void *codes, void *scales,
                              void *operand, size_t operand_bytes, void *stream) {
    if (!known(dt)) return W4A4_ERR_UNSUPPORTED_DTYPE;
    if (!known_format(fmt) || (act != W4A4_GLU_SILU && act != W4A4_GLU_GELU_TANH)) return W4A4_ERR_INVALID_VALUE;
    if (m < 0 || k < 0 || ldg < k || ldu < k || !within_bounds(m, 0, k)) return W4A4_ERR_INVALID_VALUE;
    if (k % QK) return W4A4_ERR_K_NOT_MULTIPLE_OF_32;
    if (m == 0 || k == 0) return W4A4_OK;
    if (!gate || !up) return W4A4_ERR_INVALID_VALUE;
    const GluArgs a{static_cast<const uint8_t *>(gate), static_cast<const uint8_t *>(up), ldg, ldu, dt, act,
                    row_blocks(blocks_covered(fmt, operand, k)),
                    RowsOut{static_cast<uint8_t *>(codes), scales, static_cast<uint8_t *>(operand), m, k}};
    if (!grid_fits(rows_covered(fmt, operand, m) * blocks_covered(fmt, operand, k) * 4 + ROWS_THREADS))
        return W4A4_ERR_INVALID_VALUE;
    const w4a4_status st = check_outputs(fmt, a.out, operand_bytes);
    if (st != W4A4_OK) return st;
    if (!aligned(gate, size_of(dt)) || !aligned(up, size_of(dt))) return W4A4_ERR_MISALIGNED;
    hipStream_t s = as_stream(stream);
    switch (fmt) {
    case W4A4_ACT_INT4: launch_glu<FMT_INT4>(a, s); break;
    case W4A4_ACT_INT4_SMALL: launch_glu<FMT_INT4_SMALL>(a, s); break;
    case W4A4_ACT_INT8: launch_glu<FMT_INT8>(a, s); break;
    case W4A4_ACT_MX4: launch_glu<FMT_MX4>(a, s); break;
    case W4A4_ACT_MX4_H32: launch_glu<FMT_MX4_H32>(a, s); break;
    }
    return hip_status("glu_rows_kernel");
}

w4a4_status w4a4_rms_norm_quantize(const void *x, w4a4_dtype xdt, int64_t ldx, const void *residual, w4a4_dtype rdt,
                                   int64_t ldr, const float *weight, double eps, int64_t m, int64_t k, void *h,
                                   int64_t ldh, w4a4_act_format fmt, void *codes, void *scales, void *operand,
                                   size_t operand_bytes, void *stream) {
    if (!known(xdt) || !known(rdt)) return W4A4_ERR_UNSUPPORTED_DTYPE;
    if (!known_format(fmt) || !(eps > 0.0) || !std::isfinite(eps)) return W4A4_ERR_INVALID_VALUE;
    if (m < 0 || k < 0 || ldx < k || (residual && ldr < k) || (h && ldh < k) || !within_bounds(m, 0, k))
        return W4A4_ERR_INVALID_VALUE;
    if (k % QK) return W4A4_ERR_K_NOT_MULTIPLE_OF_32;
    if (m == 0 || k == 0) return W4A4_OK;
    if (!x) return W4A4_ERR_INVALID_VALUE;
    // in place: the same elements only (one row has no stride)
    if ((h == x && (xdt != rdt || (m > 1 && ldh != ldx))) || (h && h == residual && m > 1 && ldh != ldr))
        return W4A4_ERR_INVALID_VALUE;
    const NormArgs a{static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(residual), weight,
                     static_cast<uint8_t *>(h), ldx, ldr, ldh, eps, 1.0 / (double)k, xdt, rdt,
                     RowsOut{static_cast<uint8_t *>(codes), scales, static_cast<uint8_t *>(operand), m, k}};
    if (!grid_fits(rows_covered(fmt, operand, m) * 1024)) return W4A4_ERR_INVALID_VALUE;
    const w4a4_status st = check_outputs(fmt, a.out, operand_bytes);
    if (st != W4A4_OK) return st;
    if (!aligned(x, size_of(xdt)) || !aligned(residual, size_of(rdt)) || !aligned(h, size_of(rdt)) || !aligned(weight, 4))
        return W4A4_ERR_MISALIGNED;
    hipStream_t s = as_stream(stream);
    switch (fmt) {
    case W4A4_ACT_INT4: launch_norm<FMT_INT4>(a, s); break;
    case W4A4_ACT_INT4_SMALL: launch_norm<FMT_INT4_SMALL>(a, s); break;
    case W4A4_ACT_INT8: launch_norm<FMT_INT8>(a, s); break;
    case W4A4_ACT_MX4: launch_norm<FMT_MX4>(a, s); break;
    case W4A4_ACT_MX4_H32: launch_norm<FMT_MX4_H32>(a, s); break;
    }
    return hip_status("norm_rows_kernel");
}

}  // extern "C"
