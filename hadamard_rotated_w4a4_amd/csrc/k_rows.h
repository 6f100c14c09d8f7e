// Producers of quantised activation rows, and the rows read back.
//
// Every product here reads rows of 32-element blocks in one of these formats
// (w4a4_act_format): int4 or int8 codes of the rotated block with one fp32
// scale, or MXFP4 (the OCP Microscaling format: FP4 E2M1 codes with one E8M0
// power-of-two scale), rotated or not.  The kernels below write them straight
// from what makes the rows: a residual addition and RMS norm, a gated
// activation, or a plain matrix (MXFP4; k_rotq.h has the int4 and int8 forms).
//
// Codes depend on every rounding before them, so each is defined by a fixed
// sequence of roundings.  Where an exact value is an unordered sum (the row's
// sum of squares) or a transcendental function (the gated activation), it is
// evaluated in fp64 (the sum to about 2^-50, the function to within 2^-40) and
// rounded once to fp32: a launch shape that takes the sum in another order gives
// another last place of the root for less than one row in 2^26, and the same codes
// for all others.  fp64 multiply-adds issue at the fp32 rate on this part: the norm's
// are hidden behind its loads, the gated activation's are two fifths of its
// instructions.
//
// A block is held by a quad of lanes (lane L: elements 8L .. 8L + 7), as in
// the quantiser.
#pragma once

#include "common.h"
#include "k_rotq.h"

namespace w4a4 {

constexpr int ROW_F32 = 0, ROW_F16 = 1, ROW_BF16 = 2;  // w4a4_dtype
constexpr int FMT_INT4 = 0, FMT_INT4_SMALL = 1, FMT_INT8 = 2, FMT_MX4 = 3, FMT_MX4_H32 = 4;  // w4a4_act_format

// MXFP4 rows: scale bytes per row (whole groups of 8 blocks: 256 elements of
// K; the bytes past k / 32 are written as 127 and never read as scales).
constexpr int MX4_GROUP = 8;
__host__ __device__ inline int64_t mx4_stride(int64_t k) { return (k / QK + MX4_GROUP - 1) / MX4_GROUP * MX4_GROUP; }

struct RowsOut {
    uint8_t *codes;
    void *scales;
    uint8_t *act;  // operand records (int4, int8), the record-ordered operand (int4_small), or null
    int64_t m, k;
};

// Eight elements of a row, as loaded: 16 bytes of a 2-byte type, 32 of fp32.
// Loading and converting are apart so that a thread can have every load of its
// row in flight before it waits for the first.
struct Raw8 {
    v4u lo, hi;
};
// 16 bytes an instruction whatever the alignment of the rows: the hardware takes
// any element-aligned address.
typedef v4u v4u_any __attribute__((aligned(2)));
__device__ __forceinline__ Raw8 load_raw8(const uint8_t *p, int dt) {
    Raw8 x;
    x.lo = *reinterpret_cast<const v4u_any *>(p);
    if (dt == ROW_F32) x.hi = *reinterpret_cast<const v4u_any *>(p + 16);
    return x;
}
__device__ __forceinline__ void to_f32(const Raw8 &x, int dt, float v[8]) {
    if (dt == ROW_F32) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[i] = __uint_as_float(x.lo[i]);
            v[4 + i] = __uint_as_float(x.hi[i]);
        }
    } else if (dt == ROW_F16) {
#pragma unroll
        for (int i = 0; i < 4; i++) halves_to_float(x.lo[i], v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(x.lo[i] << 16);
            v[2 * i + 1] = __uint_as_float(x.lo[i] & 0xFFFF0000u);
        }
    }
}
__device__ __forceinline__ int row_size(int dt) { return dt == ROW_F32 ? 4 : 2; }

// fp32 -> 16-bit types, to nearest even.
__device__ __forceinline__ uint16_t f16_bits(float x) { return __half_as_ushort(__float2half_rn(x)); }
__device__ __forceinline__ uint16_t bf16_bits(float x) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x)); }

// v rounded to type dt.
__device__ __forceinline__ void round_row8(int dt, float v[8]) {
    if (dt == ROW_F16) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = __half2float(__ushort_as_half(f16_bits(v[i])));
    } else if (dt == ROW_BF16) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = __uint_as_float((uint32_t)bf16_bits(v[i]) << 16);
    }
}

// Eight values rounded to type dt at byte address p (element-aligned).
__device__ __forceinline__ void store_row8(uint8_t *p, int dt, const float v[8]) {
    v4u lo, hi;
    if (dt == ROW_F32) {
#pragma unroll
        for (int i = 0; i < 4; i++) lo[i] = __float_as_uint(v[i]), hi[i] = __float_as_uint(v[4 + i]);
        reinterpret_cast<v4u_any *>(p)[1] = hi;
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint16_t a = dt == ROW_F16 ? f16_bits(v[2 * i]) : bf16_bits(v[2 * i]);
            const uint16_t b = dt == ROW_F16 ? f16_bits(v[2 * i + 1]) : bf16_bits(v[2 * i + 1]);
            lo[i] = (uint32_t)a | (uint32_t)b << 16;
        }
    }
    *reinterpret_cast<v4u_any *>(p) = lo;
}

// One block as MXFP4: e = floor(log2 max|v|) - 2 (at least -127), the codes
// E2M1(v 2^-e) to nearest even, magnitudes of 6 and more saturating at 6, the
// scale byte e + 127.  A block that holds an infinity or NaN gets byte 255
// (the format's NaN) and zero codes; a zero block byte 0.  Returns this lane's
// eight codes, element 8L + i in bits 4i .. 4i + 3.
__device__ __forceinline__ uint32_t mx4_quantise(const float v[8], uint32_t &byte) {
    uint32_t top = 0;  // |v| as integers: the same order, NaN and infinity on top
#pragma unroll
    for (int t = 0; t < 8; t++) top = max(top, __float_as_uint(v[t]) & 0x7FFFFFFFu);
    top = max(top, quad_u32<QP_XOR1>(top));
    top = max(top, quad_u32<QP_XOR2>(top));
    const int E = (int)(top >> 23);  // biased exponent; 0 for subnormals
    byte = E == 255 ? 255u : (uint32_t)max(E - 2, 0);
    const int sh = 127 - (int)byte;
    float u[8];
#pragma unroll
    for (int t = 0; t < 8; t++)  // exact (the scale is a power of two); in (-8, 8) before the clamp
        u[t] = __builtin_amdgcn_fmed3f(ldexpf(v[t], sh), -6.0f, 6.0f);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[0], u[1], 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[2], u[3], 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[4], u[5], 1.0f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[6], u[7], 1.0f, 3);
    return E == 255 ? 0u : c;
}

// The values v of one (row, block), held by a quad, quantised and written in
// format FMT: public codes and scales for rows below m and blocks below k / 32,
// padding scale bytes (MXFP4) and operand records as the format has them.
// Every lane of the quad must take part.
template <int FMT>
__device__ __forceinline__ void emit_block(float v[8], int L, int64_t row, int64_t b, const RowsOut &o) {
    if constexpr (FMT == FMT_MX4 || FMT == FMT_MX4_H32) {
        if constexpr (FMT == FMT_MX4_H32) {
            fwht32_quad(v, L);
#pragma unroll
            for (int t = 0; t < 8; t++) v[t] = __fmul_rn(v[t], kInvSqrt32f);
        }
        uint32_t byte;
        const uint32_t c = mx4_quantise(v, byte);
        if (row < o.m) {
            const bool live = b < o.k / QK;
            if (live) reinterpret_cast<uint32_t *>(o.codes + row * (o.k / 2) + b * 16)[L] = c;
            if (L == 0 && b < mx4_stride(o.k))
                static_cast<uint8_t *>(o.scales)[row * mx4_stride(o.k) + b] = (uint8_t)(live ? byte : 127u);
        }
    } else {
        constexpr int QMAX = FMT == FMT_INT8 ? 127 : 7;
        int q[8];
        float s;
        quantise_values<QMAX, true, true>(v, L, q, s);
        store_quantised<QMAX>(q, s, L, row, b, o.m, o.k, o.codes, static_cast<float *>(o.scales),
                              FMT == FMT_INT4_SMALL ? nullptr : o.act, FMT == FMT_INT4_SMALL ? o.act : nullptr);
    }
}

// Rows and blocks that a format's outputs cover, padding included.
__host__ __device__ inline int64_t rows_covered(int fmt, bool act, int64_t m) {
    return !act ? m : fmt == FMT_INT4_SMALL ? SMA_ROWS : (m + 31) / 32 * 32;
}
__host__ __device__ inline int64_t blocks_covered(int fmt, bool act, int64_t k) {
    if (fmt == FMT_MX4 || fmt == FMT_MX4_H32) return mx4_stride(k);
    return !act ? k / QK : fmt == FMT_INT4_SMALL ? sq_quads(k) * SQ_BLOCKS : mx_blocks(k);
}

// Which (row, block) a quad of the element-wise kernels takes.  TILED (outputs
// with operand records): as the quantiser, a workgroup covers 32 rows x 2
// blocks, so that the records are written in runs.  Otherwise consecutive
// quads take consecutive blocks of a row: every load and store is contiguous.
constexpr int ROWS_THREADS = 256;
// Blocks per row with ceil(2^64 / n), so that a quad's row is one high product:
// exact for quads below 2^32 (the error, below n, times 2^32 is below 2^64 / n
// as n < 2^20).
struct RowBlocks {
    uint32_t n;
    uint64_t magic;  // 0 for n == 1
};
inline RowBlocks row_blocks(int64_t n) { return RowBlocks{(uint32_t)n, n > 1 ? ~0ull / (uint64_t)n + 1 : 0}; }
template <bool TILED>
__device__ __forceinline__ void block_of_quad(RowBlocks blocks, int64_t &row, int64_t &b) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if constexpr (TILED) {
        b = (int64_t)blockIdx.x * RQ_BLOCKS + (wave >> 1);
        row = (int64_t)blockIdx.y * 32 + (wave & 1) * 16 + (lane >> 2);
    } else {
        const uint32_t i = blockIdx.x * (ROWS_THREADS / 4) + (tid >> 2);  // below 2^30 (the launch is below 2^32 threads)
        const uint32_t q = blocks.magic ? (uint32_t)__umul64hi(i, blocks.magic) : i;
        row = q;
        b = i - q * blocks.n;
    }
}

// ---------------------------------------------------------------------------
// Plain rows to MXFP4.  Bound by memory: one pass, every byte once.  17408 x 5120
// fp32 73 us, 5.5 TB/s; 512 x 5120 fp16 3.4 us, of which a launch that does
// nothing takes about 2.
// ---------------------------------------------------------------------------
struct PlainArgs {
    const uint8_t *x;
    int64_t ld;  // elements
    int dt;
    RowBlocks blocks;
    RowsOut out;
};
template <int FMT>
__global__ __launch_bounds__(ROWS_THREADS) void quantise_rows_kernel(PlainArgs a) {
    int64_t row, b;
    block_of_quad<false>(a.blocks, row, b);
    const int L = threadIdx.x & 3;
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (row < a.out.m && b < a.out.k / QK)
        to_f32(load_raw8(a.x + (row * a.ld + b * QK + 8 * L) * row_size(a.dt), a.dt), a.dt, v);
    emit_block<FMT>(v, L, row, b, a.out);
}

// ---------------------------------------------------------------------------
// Gated activation: v = fl32(act(g) u), act in fp64.  Bound by vector issue: 65
// instructions an element for 302 x 17408 fp16 to int8, 5,174 a SIMD, which at 4
// cycles of 2.4 GHz are 8.6 of its 11.6 us (27.1 MB, 2.3 TB/s).  8192 x 768 fp32 to
// int4 13.2 us (54.4 MB, 4.1 TB/s), 16 x 17408 3.2 us.  With operand records 302 x
// 17408 takes 17.0 us to int8 (40.2 MB, 7,260 instructions) and 13.9 to int4.
// ---------------------------------------------------------------------------
constexpr int GLU_SILU = 0, GLU_GELU_TANH = 1;  // w4a4_glu_act

// act(g) u in fp64 to within 2^-40, rounded once to fp32: silu(g) = g s(g) with
// s(z) = 1 / (1 + e^-z); the tanh form of gelu, g (1 + tanh w) / 2 with w =
// sqrt(2 / pi) (g + 0.044715 g^3), is g s(2 w).
//
// e^t: t = n ln 2 + r, |r| <= ln 2 / 2 (n from the low bits of t log2 e + 1.5
// 2^52; n times the error of ln 2 in fp64 is below 2^-44); e^r by the degree 9
// interpolant at the Chebyshev nodes of the interval (2^-45.5); n into the
// exponent.  The quotient: the hardware reciprocal x of d, off by e = 1 - d x
// (about 2^-23), corrected as x (1 + e + e^2).  g is clamped for the exponential
// only, where fp64 would overflow past it (t within +-700: the result is u times
// g or 0 in fp32 there; a gate of minus infinity stays infinite).  About 22 fp64
// operations an element.
__device__ __forceinline__ float gated(float gate, float up, int act) {
    constexpr double kMagic = 0x1.8p52;
    double t;
    if (act == GLU_GELU_TANH) {
        const double c = fminf(fmaxf(gate, -21.0f), 21.0f);
        t = c * fma(c * c, -1.5957691216057308 * 0.044715, -1.5957691216057308);  // -2 w, within +-695
    } else {
        t = -(double)fminf(fmaxf(gate, -700.0f), 700.0f);
    }
    const double s = fma(t, 0x1.71547652b82fep+0, kMagic), n = s - kMagic;
    const double r = fma(n, -0x1.62e42fefa39efp-1, t);
    double p = 0x1.72ea9fa1a615ep-19;
    p = fma(p, r, 0x1.a17dbfc6c99d6p-16);
    p = fma(p, r, 0x1.a0198b67fb9ecp-13);
    p = fma(p, r, 0x1.6c162be1ccf47p-10);
    p = fma(p, r, 0x1.11111126c1431p-7);
    p = fma(p, r, 0x1.55555588a2487p-5);
    p = fma(p, r, 0x1.555555554f71ap-3);
    p = fma(p, r, 0x1.ffffffffe75d7p-2);
    p = fma(p, r, 0x1.000000000000bp+0);
    p = fma(p, r, 0x1.000000000003dp+0);
    const uint64_t bits = __builtin_bit_cast(uint64_t, p);  // in (0.7, 1.42); n within +-1010
    const uint32_t lo = (uint32_t)__builtin_bit_cast(uint64_t, s);  // n as an integer
    const double d = 1.0 + __builtin_bit_cast(double, (uint64_t)((uint32_t)(bits >> 32) + (lo << 20)) << 32 | (uint32_t)bits);
    const double x = __builtin_amdgcn_rcp(d), e = fma(-d, x, 1.0);
    // the quotient corrected before the product (gate up is exact): an infinite
    // gate or up stays infinite
    return (float)((double)gate * (double)up * fma(x, fma(e, e, e), x));
}

struct GluArgs {
    const uint8_t *gate, *up;
    int64_t ldg, ldu;  // elements
    int dt, act;
    RowBlocks blocks;
    RowsOut out;
};
template <int FMT, bool TILED>
__global__ __launch_bounds__(ROWS_THREADS) void glu_rows_kernel(GluArgs a) {
    int64_t row, b;
    block_of_quad<TILED>(a.blocks, row, b);
    const int L = threadIdx.x & 3, esz = row_size(a.dt);
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (row < a.out.m && b < a.out.k / QK) {
        float g[8], u[8];
        const Raw8 rg = load_raw8(a.gate + (row * a.ldg + b * QK + 8 * L) * esz, a.dt);
        const Raw8 ru = load_raw8(a.up + (row * a.ldu + b * QK + 8 * L) * esz, a.dt);
        to_f32(rg, a.dt, g);
        to_f32(ru, a.dt, u);
#pragma unroll
        for (int t = 0; t < 8; t++) v[t] = gated(g[t], u[t], a.act);
    }
    emit_block<FMT>(v, L, row, b, a.out);
}

// ---------------------------------------------------------------------------
// Residual addition + RMS norm: h = r(x + residual), the sum of h^2 in fp64
// (each square exact), rstd = fl32((sum / k + eps)^(-1/2)), v = fl32(fl32(h
// rstd) weight).
//
// One workgroup per row: its threads hold the row in registers, CHUNKS pieces
// of 8 elements each, between the sum and the quantising; CHUNKS = 0 walks a
// longer row twice, reading h (or the inputs, when h is not written) again.
// With operand records, the 32 rows of a tile go to workgroups of one XCD
// (they are dealt round-robin), whose L2 joins their 8-byte pieces of a record
// to whole lines: 512 x 5120 to int8 with its records writes 13.43 MB, the outputs'
// own bytes (10.3 us).
//
// Few rows are bound by one chain of latencies, load -> sum over the workgroup ->
// quantise -> store (1 x 5120 3.3 us), 512 x 5120 to int8 (9.3 us, 24.2 MB, 2.6 TB/s)
// by a launch and one burst of reads followed by one of writes, all its workgroups
// being resident together; many rows by memory (2048 x 5120 20.4 us, 4.7 TB/s).
// ---------------------------------------------------------------------------
struct NormArgs {
    const uint8_t *x, *residual;  // residual may be null
    const float *weight;          // may be null: ones
    uint8_t *h;                   // may be null, or x or residual itself
    int64_t ldx, ldr, ldh;        // elements
    double eps, inv_k;
    int xdt, rdt;
    RowsOut out;
};

// Sum over the wave, in a fixed order, in every lane: DPP shifts within rows
// of 16 lanes and two row broadcasts bring it to lane 63.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_f64(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double shifted_sum(double x) {  // lane 15 of each row of 16 gets the row's sum
    x += dpp_f64<0x111, 0xF>(x);  // row_shr:1
    x += dpp_f64<0x112, 0xF>(x);  // row_shr:2
    x += dpp_f64<0x114, 0xF>(x);  // row_shr:4
    x += dpp_f64<0x118, 0xF>(x);  // row_shr:8
    return x;
}
__device__ __forceinline__ double row_sum(double x) { return lane_f64(shifted_sum(x), 15); }  // of the first row
__device__ __forceinline__ double wave_sum(double x) {
    x = shifted_sum(x);
    x += dpp_f64<0x142, 0xA>(x);  // row_bcast:15 into rows 1 and 3
    x += dpp_f64<0x143, 0xC>(x);  // row_bcast:31 into rows 2 and 3
    return lane_f64(x, 63);
}

// What this lane loads for 8 elements at column c of the row, and h of them.
struct NormRaw {
    Raw8 x, r, w;
};
__device__ __forceinline__ NormRaw norm_load8(const NormArgs &a, int64_t row, int64_t c, bool weight) {
    NormRaw n;
    n.x = load_raw8(a.x + (row * a.ldx + c) * row_size(a.xdt), a.xdt);
    if (a.residual) n.r = load_raw8(a.residual + (row * a.ldr + c) * row_size(a.rdt), a.rdt);
    if (weight && a.weight) n.w = load_raw8(reinterpret_cast<const uint8_t *>(a.weight + c), ROW_F32);
    return n;
}
__device__ __forceinline__ void norm_h8(const NormArgs &a, const NormRaw &n, float v[8]) {
    to_f32(n.x, a.xdt, v);
    if (a.residual) {
        float r[8];
        to_f32(n.r, a.rdt, r);
#pragma unroll
        for (int t = 0; t < 8; t++) v[t] = __fadd_rn(v[t], r[t]);
    }
    round_row8(a.rdt, v);
}
__device__ __forceinline__ void norm_scale8(const NormArgs &a, const Raw8 &weight, float rstd, float v[8]) {
#pragma unroll
    for (int t = 0; t < 8; t++) v[t] = __fmul_rn(v[t], rstd);
    if (a.weight) {
        float w[8];
        to_f32(weight, ROW_F32, w);
#pragma unroll
        for (int t = 0; t < 8; t++) v[t] = __fmul_rn(v[t], w[t]);
    }
}
__device__ __forceinline__ void norm_store8(const NormArgs &a, int64_t row, int64_t c, const float v[8]) {
    if (a.h) store_row8(a.h + (row * a.ldh + c) * row_size(a.rdt), a.rdt, v);
}
__device__ __forceinline__ void zero8(float v[8]) {
#pragma unroll
    for (int t = 0; t < 8; t++) v[t] = 0.0f;
}
// 1 / sqrt(x) in fp64: the hardware root y, off by e = 1 - x y^2 (about 2^-23),
// corrected as y (1 + e / 2 + 3 e^2 / 8).  At infinity y is 0 and e would be NaN:
// an infinity in a row makes its root 0.
__device__ __forceinline__ double rsqrt64(double x) {
    const double y = __builtin_amdgcn_rsq(x), e = y == 0.0 ? 0.0 : fma(-(x * y), y, 1.0);
    return fma(y * e, fma(0.375, e, 0.5), y);
}

template <int FMT, int CHUNKS>
__global__ __launch_bounds__(1024) void norm_rows_kernel(NormArgs a, bool act) {
    __shared__ double part[16];
    const int tid = threadIdx.x, L = tid & 3, quads = blockDim.x / 4, waves = blockDim.x / 64;
    const int64_t k = a.out.k, nb = k / QK, blocks = blocks_covered(FMT, act, k);
    int64_t row = blockIdx.x;
    if (act && FMT != FMT_INT4_SMALL) {
        const int64_t tiles = gridDim.x / 32, group = row / 256, in = row % 256;
        const int64_t width = min((int64_t)8, tiles - group * 8);
        row = (group * 8 + in % width) * 32 + in / width;
    }
    const bool live = row < a.out.m;

    constexpr int HELD = CHUNKS ? CHUNKS : 1;
    float v[HELD][8];
    NormRaw raw[HELD];
    double sum = 0.0;
    if (live) {
        if constexpr (CHUNKS > 0) {
            // every load of the row, the weights' too, before the first wait
#pragma unroll
            for (int i = 0; i < CHUNKS; i++) {
                const int64_t b = i * quads + (tid >> 2);
                if (b < nb) raw[i] = norm_load8(a, row, b * QK + 8 * L, true);
            }
#pragma unroll
            for (int i = 0; i < CHUNKS; i++) {
                const int64_t b = i * quads + (tid >> 2);
                if (b < nb) {
                    norm_h8(a, raw[i], v[i]);
                    norm_store8(a, row, b * QK + 8 * L, v[i]);
#pragma unroll
                    for (int t = 0; t < 8; t++) sum = fma((double)v[i][t], (double)v[i][t], sum);
                }
            }
        } else {
            for (int64_t b = tid >> 2; b < nb; b += quads) {
                norm_h8(a, norm_load8(a, row, b * QK + 8 * L, false), v[0]);
                norm_store8(a, row, b * QK + 8 * L, v[0]);
#pragma unroll
                for (int t = 0; t < 8; t++) sum = fma((double)v[0][t], (double)v[0][t], sum);
            }
        }
    }
    sum = wave_sum(sum);
    if ((tid & 63) == 0) part[tid >> 6] = sum;
    __syncthreads();
    // the waves' sums, one to a lane, in a fixed order (rows of 16 lanes hold the same)
    sum = (tid & 15) < waves ? part[tid & 15] : 0.0;
    sum = row_sum(sum);
    const float rstd = (float)rsqrt64(fma(sum, a.inv_k, a.eps));

    if constexpr (CHUNKS > 0) {
#pragma unroll
        for (int i = 0; i < CHUNKS; i++) {
            const int64_t b = i * quads + (tid >> 2);
            if (b >= blocks) continue;  // uniform per quad
            if (live && b < nb) norm_scale8(a, raw[i].w, rstd, v[i]);
            else zero8(v[i]);
            emit_block<FMT>(v[i], L, row, b, a.out);
        }
    } else {
        for (int64_t b = tid >> 2; b < blocks; b += quads) {
            if (live && b < nb) {
                const int64_t c = b * QK + 8 * L;
                raw[0] = norm_load8(a, row, c, true);
                // this thread's own stores above, when h is written (it may be x or residual itself)
                if (a.h) to_f32(load_raw8(a.h + (row * a.ldh + c) * row_size(a.rdt), a.rdt), a.rdt, v[0]);
                else norm_h8(a, raw[0], v[0]);
                norm_scale8(a, raw[0].w, rstd, v[0]);
            } else {
                zero8(v[0]);
            }
            emit_block<FMT>(v[0], L, row, b, a.out);
        }
    }
}

// ---------------------------------------------------------------------------
// Quantised rows read back: y = fl(q s) in type dt (MXFP4 values are exact in
// fp32 and bf16; a block whose scale byte is 255 reads as NaN).  Bound by memory:
// 17408 x 5120 MXFP4 to bf16 52 us, 4.4 TB/s; 302 x 17408 int8 to fp16 3.5 us.
// ---------------------------------------------------------------------------
struct ReadArgs {
    const uint8_t *codes;
    const void *scales;
    uint8_t *y;
    int64_t m, k, ld;  // ld: elements
    int dt;
    RowBlocks blocks;
};
template <int FMT>
__global__ __launch_bounds__(ROWS_THREADS) void read_rows_kernel(ReadArgs a) {
    const int64_t nb = a.k / QK;
    int64_t row, b;
    block_of_quad<false>(a.blocks, row, b);
    if (row >= a.m) return;
    const int L = threadIdx.x & 3;
    float v[8];
    if constexpr (FMT == FMT_MX4 || FMT == FMT_MX4_H32) {
        const uint32_t c = reinterpret_cast<const uint32_t *>(a.codes + row * (a.k / 2) + b * 16)[L];
        const int byte = static_cast<const uint8_t *>(a.scales)[row * mx4_stride(a.k) + b];
#pragma unroll
        for (int t = 0; t < 8; t++) {
            const uint32_t q = c >> (4 * t) & 15u;
            const float twice = (float)(0xC8643210u >> (4 * (q & 7u)) & 15u);  // 2 |E2M1|: 0 1 2 3 4 6 8 12
            const float x = ldexpf(q & 8u ? -twice : twice, byte - 128);
            v[t] = byte == 255 ? __uint_as_float(0x7FC00000u) : x;
        }
    } else {
        const float s = static_cast<const float *>(a.scales)[row * nb + b];
        if constexpr (FMT == FMT_INT8) {
            const uint2 w = *reinterpret_cast<const uint2 *>(a.codes + row * a.k + b * QK + 8 * L);
#pragma unroll
            for (int t = 0; t < 8; t++) v[t] = __fmul_rn((float)(int8_t)((t < 4 ? w.x : w.y) >> (8 * (t & 3))), s);
        } else {  // byte j: element j low, element j + 16 high
            const uint2 w = *reinterpret_cast<const uint2 *>(a.codes + row * (a.k / 2) + b * 16 + 8 * (L & 1));
            const int up = L < 2 ? 4 : 0;  // bring the nibble to the top of its byte
#pragma unroll
            for (int t = 0; t < 8; t++) {
                const uint32_t byte = (t < 4 ? w.x : w.y) >> (8 * (t & 3)) & 255u;
                v[t] = __fmul_rn((float)((int8_t)(byte << up) >> 4), s);
            }
        }
    }
    store_row8(a.y + (row * a.ld + b * QK + 8 * L) * row_size(a.dt), a.dt, v);
}

}  // namespace w4a4
