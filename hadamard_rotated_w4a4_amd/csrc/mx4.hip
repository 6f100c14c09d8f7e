// Host side of the MXFP4 product (k_mx4.h): argument checks, launch shapes.
#include "w4a4.h"

#include <algorithm>
#include <cstdint>

#include "abi.h"
#include "common.h"
#include "k_mx4.h"

using namespace w4a4;

extern "C" {

size_t w4a4_mx4_packed_bytes(int64_t n, int64_t k) {
    if (n < 0 || k < 0 || k % QK) return 0;
    return (size_t)mx4_packed_bytes(n, k);
}

w4a4_status w4a4_repack_mx4(const uint8_t *codes, const uint8_t *scales, int64_t n, int64_t k, void *packed,
                            void *stream) {
    if (n < 0 || k < 0 || !within_bounds(0, n, k)) return W4A4_ERR_INVALID_VALUE;
    if (k % QK) return W4A4_ERR_K_NOT_MULTIPLE_OF_32;
    if (n == 0 || k == 0) return W4A4_OK;
    if (!codes || !scales || !packed) return W4A4_ERR_INVALID_VALUE;
    const int64_t threads = padded_n(n) / TILE_N * mx4_groups(k) * 64;
    if (!grid_fits(threads + 256)) return W4A4_ERR_INVALID_VALUE;
    if (!aligned(codes, 16) || !aligned(scales, 8) || !aligned(packed, 16)) return W4A4_ERR_MISALIGNED;
    repack_mx4_kernel<<<blocks_for(threads, 256), 256, 0, as_stream(stream)>>>(codes, scales, n, k,
                                                                              static_cast<uint8_t *>(packed));
    return hip_status("repack_mx4_kernel");
}

size_t w4a4_gemm_mx4_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    (void)m, (void)n, (void)k;
    return 0;
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
    const int64_t tiles = padded_n(n) / TILE_N;
    const dim3 grid((unsigned)((tiles + MX4_WAVES - 1) / MX4_WAVES), (unsigned)((m + 31) / 32));
    if (!grid_fits((int64_t)grid.x * grid.y * 64 * MX4_WAVES)) return W4A4_ERR_INVALID_VALUE;
    if (k == 0) {  // empty sum
        zero_typed_kernel<<<(unsigned)std::min<int64_t>((m * n + 255) / 256, 1 << 16), 256, 0, s>>>(
            static_cast<uint8_t *>(y), ydt, m, n, ldy);
        return hip_status("zero_typed_kernel");
    }
    if (!packed_w || !codes || !scales) return W4A4_ERR_INVALID_VALUE;
    if (!aligned(packed_w, 16) || !aligned(codes, 16) || !aligned(scales, 8)) return W4A4_ERR_MISALIGNED;
    (void)workspace, (void)workspace_bytes;
    gemm_mx4_kernel<<<grid, 64 * MX4_WAVES, 0, s>>>(Mx4Args{static_cast<const uint8_t *>(packed_w), codes, scales,
                                                           static_cast<uint8_t *>(y), m, n, k, ldy, ydt});
    return hip_status("gemm_mx4_kernel");
}

}  // extern "C"
