// MXFP4 product: y[i][j] = sum_b 2^(ea[i][b] + ew[j][b]) sum_t a[i][t] w[j][t],
// both sides FP4 E2M1 codes with one E8M0 scale per 32 elements of K.
//
// The matrix cores take both operands as they are:
// v_mfma_scale_f32_32x32x64_f8f6f4 (formats 4, 4) multiplies 32 rows by 32
// columns over 64 elements of K, a lane holding 32 consecutive elements of one
// row or column (16 bytes) and the scale byte of that block, and adds into
// fp32.  So a block needs no work beyond the instruction: no widening, no
// scale product, no epilogue per block, which is what bounds the Q4_0 product.
//
// Weight records (written once by repack_mx4_kernel): [n / 32 tiles][K groups
// of 256][4352 B], in the instruction's lane order.  Lane l = 32 h + c of
// instruction p (0..3) of a group takes block 4 h + p of column c:
//   bytes [0, 4096)     lane l's 16 code bytes for instruction p at 1024 p + 16 l;
//   bytes [4096, 4352)  lane l's scale bytes of blocks 4 h .. 4 h + 3 at
//                       4096 + 4 l; instruction p selects byte p.
// Columns past n and blocks past k / 32 hold zero codes and scale byte 127:
// FP4 has no NaN or infinity, so they add exact zeros whatever finite value
// the other side holds there.
#pragma once

#include "common.h"
#include "k_rows.h"

namespace w4a4 {

typedef int mx4_v8i __attribute__((ext_vector_type(8)));
constexpr int MX4_REC = 4352;
constexpr int MX4_SCALE_OFF = 4096;
constexpr int MX4_GROUP_BYTES = MX4_GROUP * QK / 2;  // code bytes of a row per K group
__host__ __device__ inline int64_t mx4_groups(int64_t k) { return mx4_stride(k) / MX4_GROUP; }
__host__ __device__ inline int64_t mx4_packed_bytes(int64_t n, int64_t k) {
    return padded_n(n) / TILE_N * mx4_groups(k) * MX4_REC;
}

// One thread per (tile, group, lane).
__global__ __launch_bounds__(256) void repack_mx4_kernel(const uint8_t *__restrict__ codes,
                                                         const uint8_t *__restrict__ scales, int64_t n, int64_t k,
                                                         uint8_t *__restrict__ packed) {
    const int64_t groups = mx4_groups(k), nb = k / QK;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= padded_n(n) / TILE_N * groups * 64) return;
    const int lane = (int)(i & 63), h = lane >> 5;
    const int64_t rec = i >> 6, tile = rec / groups, grp = rec % groups, col = tile * TILE_N + (lane & 31);
    uint32_t sc = 0;
    for (int p = 0; p < 4; p++) {
        const int64_t b = grp * MX4_GROUP + 4 * h + p;
        uint4 c = make_uint4(0, 0, 0, 0);
        uint32_t s = 127;
        if (col < n && b < nb) {
            c = *reinterpret_cast<const uint4 *>(codes + col * (k / 2) + b * 16);
            s = scales[col * mx4_stride(k) + b];
        }
        *reinterpret_cast<uint4 *>(packed + rec * MX4_REC + 1024 * p + 16 * lane) = c;
        sc |= s << (8 * p);
    }
    *reinterpret_cast<uint32_t *>(packed + rec * MX4_REC + MX4_SCALE_OFF + 4 * lane) = sc;
}

// An FP4 operand (four dwords) as the v8i the builtin takes; the instruction
// reads four registers for FP4.
__device__ __forceinline__ mx4_v8i mx4_operand(v4u c) {
    const v4i v = {(int)c.x, (int)c.y, (int)c.z, (int)c.w};
    return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}
// acc += instruction P of a group (P picks the scale byte on both sides).
template <int P>
__device__ __forceinline__ v16f mx4_mfma(v4u a, v4u b, v16f acc, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx4_operand(a), mx4_operand(b), acc, 4, 4, P, (int)sa, P,
                                                           (int)sb);
}

struct Mx4Args {
    const uint8_t *packed, *codes, *scales;
    uint8_t *y;
    int64_t m, n, k, ldy;  // ldy: elements
    int dt;
};

// One output of type dt.
__device__ __forceinline__ void mx4_store(uint8_t *y, int dt, int64_t i, float v) {
    if (dt == ROW_F32) reinterpret_cast<float *>(y)[i] = v;
    else reinterpret_cast<uint16_t *>(y)[i] = dt == ROW_F16 ? f16_bits(v) : bf16_bits(v);
}

// A wave per 32 x 32 outputs over the whole of K, operands straight from
// global memory.
constexpr int MX4_WAVES = 4;
__global__ __launch_bounds__(64 * MX4_WAVES) void gemm_mx4_kernel(Mx4Args a) {
    const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
    const int64_t tile = (int64_t)blockIdx.x * MX4_WAVES + (threadIdx.x >> 6);
    if (tile >= padded_n(a.n) / TILE_N) return;
    const int64_t groups = mx4_groups(a.k), nb = a.k / QK;
    const int64_t row0 = (int64_t)blockIdx.y * 32, row = min(row0 + r, a.m - 1);
    const uint8_t *arow = a.codes + row * (a.k / 2), *srow = a.scales + row * mx4_stride(a.k);
    v16f acc = {};
    for (int64_t g = 0; g < groups; g++) {
        const uint8_t *rec = a.packed + (tile * groups + g) * MX4_REC;
        v4u av[4], bv[4];
        uint32_t sa = 0;
#pragma unroll
        for (int p = 0; p < 4; p++) {
            const int64_t b = g * MX4_GROUP + 4 * h + p;
            bv[p] = *reinterpret_cast<const v4u *>(rec + 1024 * p + 16 * lane);
            av[p] = *reinterpret_cast<const v4u *>(arow + min(b, nb - 1) * 16);
            sa |= (b < nb ? (uint32_t)srow[b] : 127u) << (8 * p);
        }
        const uint32_t sb = *reinterpret_cast<const uint32_t *>(rec + MX4_SCALE_OFF + 4 * lane);
        acc = mx4_mfma<0>(av[0], bv[0], acc, sa, sb);
        acc = mx4_mfma<1>(av[1], bv[1], acc, sa, sb);
        acc = mx4_mfma<2>(av[2], bv[2], acc, sa, sb);
        acc = mx4_mfma<3>(av[3], bv[3], acc, sa, sb);
    }
    const int64_t col = tile * TILE_N + r;
#pragma unroll
    for (int v = 0; v < 16; v++) {
        const int64_t i = row0 + mfma32_row(v, lane);
        if (i < a.m && col < a.n) mx4_store(a.y, a.dt, i * a.ldy + col, acc[v]);
    }
}

// y[0..m)[0..n) = 0 (k == 0: an empty sum).
__global__ void zero_typed_kernel(uint8_t *y, int dt, int64_t m, int64_t n, int64_t ldy) {
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < m * n; i += stride)
        mx4_store(y, dt, (i / n) * ldy + i % n, 0.0f);
}

}  // namespace w4a4
