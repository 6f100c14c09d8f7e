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
// K is walked in stages of 128 (4 blocks, two instructions): in instruction j
// of a stage, lane half h = l / 32 takes block 2 j + h.  The four scale bytes
// of a row's stage are one dword; shifted right by 8 h, its bytes 0 and 2 are
// the scales of the lane's two blocks.
//
// Records (written by repack_mx4_kernel: once for the weights, per call for the
// rows of a tiled product): [32-row tiles][stages, K padded to 256][2176 B], in
// the instruction's lane order:
//   bytes [0, 2048)     lane l's 16 code bytes for instruction j at 1024 j + 16 l;
//   bytes [2048, 2176)  row (column) c's four scale bytes at 2048 + 4 c.
// Rows past the matrix and blocks past k / 32 hold zero codes and scale byte
// 127: FP4 has no NaN or infinity, so they add exact zeros whatever codes the
// other side holds there (a reader of plain rows replaces the scale bytes past
// k / 32 by 127).
#pragma once

#include <type_traits>

#include "common.h"
#include "k_rows.h"

namespace w4a4 {

typedef int mx4_v8i __attribute__((ext_vector_type(8)));
constexpr int MX4_REC = 2176;
constexpr int MX4_SCALE_OFF = 2048;
constexpr int MX4_BLOCKS = 4;                      // blocks per stage
constexpr int MX4_ROW_BYTES = MX4_BLOCKS * QK / 2;  // code bytes of a row per stage
__host__ __device__ inline int64_t mx4_rec_stages(int64_t k) { return mx4_stride(k) / MX4_BLOCKS; }  // stored
__host__ __device__ inline int64_t mx4_stages(int64_t k) { return (k / QK + MX4_BLOCKS - 1) / MX4_BLOCKS; }  // to compute
__host__ __device__ inline int64_t mx4_packed_bytes(int64_t n, int64_t k) {
    return padded_n(n) / TILE_N * mx4_rec_stages(k) * MX4_REC;
}

// One thread per (tile, stage, lane).  Bound by memory for weights (5120 x 17408
// 19.4 us, 95 MB, 4.9 TB/s) and by a launch's latency for rows (302 x 17408 4.2 us,
// 512 x 5120 3.6).
__global__ __launch_bounds__(256) void repack_mx4_kernel(const uint8_t *__restrict__ codes,
                                                         const uint8_t *__restrict__ scales, int64_t n, int64_t k,
                                                         uint8_t *__restrict__ packed) {
    const int64_t stages = mx4_rec_stages(k), nb = k / QK;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= padded_n(n) / TILE_N * stages * 64) return;
    const int lane = (int)(i & 63), h = lane >> 5;
    const int64_t rec = i >> 6, tile = rec / stages, t = rec % stages, col = tile * TILE_N + (lane & 31);
    uint8_t *out = packed + rec * MX4_REC;
    for (int j = 0; j < 2; j++) {
        const int64_t b = t * MX4_BLOCKS + 2 * j + h;
        uint4 c = make_uint4(0, 0, 0, 0);
        uint8_t s = 127;
        if (col < n && b < nb) {
            c = *reinterpret_cast<const uint4 *>(codes + col * (k / 2) + b * 16);
            s = scales[col * mx4_stride(k) + b];
        }
        *reinterpret_cast<uint4 *>(out + 1024 * j + 16 * lane) = c;
        out[MX4_SCALE_OFF + 4 * (lane & 31) + 2 * j + h] = s;
    }
}

// An FP4 operand (four dwords) as the v8i the builtin takes; the instruction
// reads four registers for FP4.
__device__ __forceinline__ mx4_v8i mx4_operand(v4u c) {
    const v4i v = {(int)c.x, (int)c.y, (int)c.z, (int)c.w};
    return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}
// acc += instruction J of a stage; sa, sb: the lanes' scale dwords, shifted.
template <int J>
__device__ __forceinline__ v16f mx4_mfma(v4u a, v4u b, v16f acc, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx4_operand(a), mx4_operand(b), acc, 4, 4, 2 * J, (int)sa,
                                                           2 * J, (int)sb);
}
// The scale bytes of stage t with those of blocks past nb replaced by 127.
__device__ __forceinline__ uint32_t mx4_live_scales(uint32_t s, int64_t t, int64_t nb) {
    const int live = (int)min(nb - t * MX4_BLOCKS, (int64_t)MX4_BLOCKS);  // 1..4 for a stage that is computed
    const uint32_t keep = 0xFFFFFFFFu >> (8 * (MX4_BLOCKS - live));
    return (s & keep) | (0x7F7F7F7Fu & ~keep);
}

struct Mx4Args {
    const uint8_t *packed, *codes, *scales;
    const uint8_t *rows;  // the activation rows as records (tiled product)
    uint8_t *y;
    int64_t m, n, k, ldy;  // ldy: elements
    int dt;
    int64_t first;    // tiled product: first 32-column tile (the columns before it are another launch's)
    int64_t columns;  // and how many of the kernel's own column tiles
    int64_t splits;   // K splits of every tile (1: stored to y)
    float *partial;   // splits > 1: [splits][m][n] partial sums
};

// One output of type dt.
__device__ __forceinline__ void mx4_store(uint8_t *y, int dt, int64_t i, float v) {
    if (dt == ROW_F32) reinterpret_cast<float *>(y)[i] = v;
    else reinterpret_cast<uint16_t *>(y)[i] = dt == ROW_F16 ? f16_bits(v) : bf16_bits(v);
}

// ---------------------------------------------------------------------------
// Tiled product (both sides as records): WM x WN waves, each owning TM x TN
// tiles of 32 x 32.  The records go through a ring of NS slots of KS stages in
// LDS, filled by direct global-to-LDS loads NS - 1 slots ahead of the one
// computed; one barrier per slot.
//
// A slot is filled in units of 1 KB, one load instruction each and dealt to the
// waves in turn: unit 2 (KS t + u) + j is the codes of instruction j of stage u
// of tile t (row tiles first, then column tiles), the units after those the
// scale bytes, 128 of a tile's stage to every 8 lanes.  In LDS unit i lies at
// 1024 i.  A load instruction occupies the CU's address path for about 16
// cycles whatever its width, and a wave waits while it is busy: so scales are
// gathered into whole units, and a wave issues its loads one by one between
// its MFMAs, not at the barrier.
//
// What bounds it: a 256 x 256 tile's slot holds 1024 matrix-core cycles a SIMD and
// 770 cycles of LDS reads, and takes 1.04 us where a launch fills the chip, 0.75
// with zero codes: random codes draw so much power that the clock falls from 2.4 to
// 1.9 GHz (512 x 32768 x 5120, one full round: 54 us back to back, 3.2 PFLOP/s, 50
// with the chip idle before it; 41 with zero codes).  About 12 us of that are the
// start, the first loads and the output's way to memory, which the one round leaves
// in the open.  Small tiles wait for LDS reads, the loads' writes there and
// barriers: 302 x 5120 x 17408 spends 30.6 us in 64 x 64 tiles, 18 % of it in
// matrix instructions, and 4.2 in the rows' records.
//
// Tried and slower or no faster: the rows read in place instead of from records
// (302 x 5120 x 17408 47.7 us against 38.9 with the same tiles: their 64- and
// 128-byte pieces cost the address path what the records save); the weights
// straight to registers (the same time, with a deeper chain of latencies); rings
// of more slots; two groups of waves on halves of K.
// ---------------------------------------------------------------------------
template <int WM_, int WN_, int TM_, int TN_, int KS_, int NS_>
struct Mx4Cfg {
    static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_, KS = KS_, NS = NS_;
    static_assert(KS == 1 || KS == 2, "the records hold whole slots: K padded to 256");
    static constexpr int WAVES = WM * WN, NT = 64 * WAVES;
    static constexpr int RT = WM * TM, CT = WN * TN, BM = 32 * RT, BN = 32 * CT;
    static constexpr int PIECES = (RT + CT) * KS;                 // tile stages in a slot
    static constexpr int CODE_UNITS = 2 * PIECES, UNITS = CODE_UNITS + (PIECES + 7) / 8;
    static constexpr int SLOT = 1024 * UNITS;                     // bytes
    static constexpr int LOADS = (UNITS + WAVES - 1) / WAVES;     // of a slot, per wave: this many for the first
    static constexpr int FULL = UNITS - (LOADS - 1) * WAVES;      // FULL waves, one less for the others
    // Loads and waits decided inside asm blocks, so that a slot is one scheduling
    // region: its MFMAs issue ahead of its waits, behind the next slot's LDS reads.
    // 64 x 64 tiles gain most (302 x 5120 x 17408 34.4 us against 38.5, 128 x 128
    // 512 x 34816 x 5120 78 against 81).  Not for 8 tiles of 32 x 32 a wave, whose
    // registers then spill (512 x 32768 x 5120 131 us against 63).
    static constexpr bool STRAIGHT = TM * TN <= 6;
    static_assert(NS >= 3 && NS * SLOT <= 160 * 1024, "the ring fits the LDS");
    static_assert(2048 * TN * WAVES <= NS * SLOT, "so does a row of 16-bit output tiles per wave");
};

// One global-to-LDS load of 16 bytes per lane: the 16 bytes at lane l's p land
// at LDS byte address lds + 16 l (lds is uniform).  A load that reads M0 needs one
// wait state after the write (the compiler sees neither in here).
__device__ __forceinline__ void mx4_load16(const uint8_t *p, uint32_t lds) {
    uint32_t m0;  // written
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : "={m0}"(m0) : "v"(p), "s"(lds) : "memory");
}
// The same, if on (uniform); see Mx4Cfg::STRAIGHT.
__device__ __forceinline__ void mx4_load16(const uint8_t *p, uint32_t lds, int on) {
    uint32_t m0;
    asm volatile(
        "s_cmp_eq_u32 %3, 0\n\ts_cbranch_scc1 1f\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off\n1:"
        : "={m0}"(m0)
        : "v"(p), "s"(lds), "s"(__builtin_amdgcn_readfirstlane(on))
        : "memory", "scc");
}
// Until at most A (which = 0), B (which = 1) or no vector loads are in flight.
template <int A, int B>
__device__ __forceinline__ void mx4_wait(int which) {
    asm volatile(
        "s_cmp_eq_u32 %2, 0\n\ts_cbranch_scc0 1f\n\ts_waitcnt vmcnt(%0)\n\ts_branch 3f\n1:\n\ts_cmp_eq_u32 %2, 1\n\t"
        "s_cbranch_scc0 2f\n\ts_waitcnt vmcnt(%1)\n\ts_branch 3f\n2:\n\ts_waitcnt vmcnt(0)\n3:" ::"n"(A),
        "n"(B), "s"(__builtin_amdgcn_readfirstlane(which))
        : "memory", "scc");
}
// Until this wave's LDS reads have returned, in a form that the compiler counts
// (it would wait for them again at their first use, and for later ones with them).
__device__ __forceinline__ void mx4_wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }
template <class T>
__device__ __forceinline__ T mx4_lds(const uint8_t *p) {
    return *reinterpret_cast<const volatile __attribute__((address_space(3))) T *>(
        (const __attribute__((address_space(3))) uint8_t *)p);
}
// Tile of workgroup id, XCD-aware: workgroups are dealt to the 8 XCDs
// round-robin, so ids x, x + 8, ... share an L2; the row tiles of a column
// tile take ids x + 8 y and read its weights from HBM about once.
__device__ __forceinline__ void mx4_tile_of(uint32_t id, uint32_t nx, uint32_t ny, uint32_t &bx, uint32_t &by) {
    const uint32_t group = id / (8 * ny), in = id % (8 * ny), width = min(8u, nx - group * 8);
    bx = group * 8 + in % width;
    by = in / width;
}

template <class C>
__global__ __launch_bounds__(C::NT) void gemm_mx4_tile_kernel(Mx4Args a) {
    __shared__ __align__(1024) uint8_t smem[C::NS * C::SLOT];
    constexpr int RT = C::RT, CT = C::CT, TM = C::TM, TN = C::TN, KS = C::KS, NS = C::NS, STEPS = 2 * KS, L = C::LOADS;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / C::WN, wn = wave % C::WN, h = lane >> 5, r = lane & 31;
    const int64_t rec_stages = mx4_rec_stages(a.k);
    const uint32_t slots = (uint32_t)(mx4_stages(a.k) + KS - 1) / KS;  // of K: at most 2^17
    const int64_t rtiles = padded_n(a.m) / TILE_N, ctiles = padded_n(a.n) / TILE_N;

    // 32-bit index arithmetic: a 64-bit division takes hundreds of cycles, and the
    // few here are ahead of the first load
    uint32_t id = blockIdx.x, z = 0, bx, by;
    const uint32_t splits = (uint32_t)a.splits;
    if (splits > 1) {
        z = id % splits;
        id /= splits;
    }
    mx4_tile_of(id, (uint32_t)a.columns, (uint32_t)((a.m + C::BM - 1) / C::BM), bx, by);
    const int64_t rt0 = (int64_t)by * RT, ct0 = a.first + (int64_t)bx * CT;
    const uint32_t lo = z * slots / splits;
    const int nst = (int)((z + 1) * slots / splits - lo);

    // ---- this wave's loads: units wave, wave + WAVES, ...  Tiles past the
    // matrix are clamped (their outputs are not stored).
    const uint32_t smem_base = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)smem;
    const bool full = wave < C::FULL;
    const uint8_t *src[L];
#pragma unroll
    for (int d = 0; d < L; d++) {
        const int i = wave + C::WAVES * d;
        // the lane's tile stage, and its 16 bytes of that record
        const int piece = i < C::CODE_UNITS ? i >> 1 : min((i - C::CODE_UNITS) * 8 + (lane >> 3), C::PIECES - 1);
        const int at = i < C::CODE_UNITS ? (i & 1) * 1024 + lane * 16 : MX4_SCALE_OFF + (lane & 7) * 16;
        const int t = min(piece / KS, RT + CT - 1), u = piece % KS;
        const uint8_t *side = t < RT ? a.rows : a.packed;
        const int64_t tile = t < RT ? min(rt0 + t, rtiles - 1) : min(ct0 + t - RT, ctiles - 1);
        src[d] = side + (tile * rec_stages + (int64_t)lo * KS + u) * MX4_REC + at;
    }
    // load d of the next slot not yet asked for, into ring slot `into`, if on (sure: it is)
    auto load = [&](int d, int into, auto sure, int on) {
        const uint32_t lds = __builtin_amdgcn_readfirstlane(smem_base + into * C::SLOT + (wave + C::WAVES * d) * 1024);
        const bool every = d < L - 1 || C::FULL == C::WAVES;  // every wave has this load
        if constexpr (C::STRAIGHT) {
            if (every && decltype(sure)::value) mx4_load16(src[d], lds);
            else mx4_load16(src[d], lds, every || full ? on : 0);
        } else if (on && (every || full)) {
            mx4_load16(src[d], lds);
        }
        src[d] += KS * MX4_REC;
    };
    // Until this wave's LDS reads are back and at most n slots' loads are in flight
    // (on = 0: none), and the other waves are there.
    auto wait = [&](auto n, int on) {
        constexpr int A = decltype(n)::value * L, B = decltype(n)::value * (L - 1);
        if constexpr (C::STRAIGHT) {
            mx4_wait_lds();
            mx4_wait<A, B>(!on ? 2 : full ? 0 : 1);
        } else if (!on) {
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        } else if (full) {
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(A) : "memory");
        } else {
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(B) : "memory");
        }
        __builtin_amdgcn_s_barrier();
    };

    v16f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++)
#pragma unroll
            for (int v = 0; v < 16; v++) acc[i][j][v] = 0.0f;

    // A slot's fragments are all read into registers one slot ahead: while the
    // MFMAs of slot s run, those of slot s + 1 arrive.  At the barrier between
    // them slot s + 1's reads have returned, so its place in the ring is free for
    // slot s + 1 + NS, and slot s + 2 has landed.  A wave thus waits for one LDS
    // round trip a slot, behind a slot's MFMAs.
    struct Fragments {
        v4u a[STEPS][TM], b[STEPS][TN];
        uint32_t sa[KS][TM], sb[KS][TN];
    };
    auto read = [&](int s, Fragments &f) {
        const uint8_t *p = smem + (s % NS) * C::SLOT;
        const uint8_t *sc = p + C::CODE_UNITS * 1024 + 4 * r;
        p += lane * 16;
#pragma unroll
        for (int u = 0; u < KS; u++) {
#pragma unroll
            for (int i = 0; i < TN; i++) f.sb[u][i] = mx4_lds<uint32_t>(sc + ((RT + wn * TN + i) * KS + u) * 128);
#pragma unroll
            for (int i = 0; i < TM; i++) f.sa[u][i] = mx4_lds<uint32_t>(sc + ((wm * TM + i) * KS + u) * 128);
        }
#pragma unroll
        for (int q = 0; q < STEPS; q++) {
#pragma unroll
            for (int i = 0; i < TN; i++) f.b[q][i] = mx4_lds<v4u>(p + (RT + wn * TN + i) * KS * 2048 + q * 1024);
#pragma unroll
            for (int i = 0; i < TM; i++) f.a[q][i] = mx4_lds<v4u>(p + (wm * TM + i) * KS * 2048 + q * 1024);
        }
    };
    // Slot s from cur, slot s + 1 into next, loads of slot s + NS (sure: there is one).
    auto slot = [&](auto sure, int s, Fragments &cur, Fragments &next) {
        const int more = decltype(sure)::value || s + NS < nst;
        const int into = s % NS;
        read(min(s + 1, nst - 1), next);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < STEPS; q++) {
            uint32_t sa[TM], sb[TN];  // bytes 0 and 2 of the shifted dword are the lane's
#pragma unroll
            for (int i = 0; i < TM; i++) sa[i] = cur.sa[q >> 1][i] >> (8 * h);
#pragma unroll
            for (int i = 0; i < TN; i++) sb[i] = cur.sb[q >> 1][i] >> (8 * h);
#pragma unroll
            for (int i = 0; i < TM; i++)
#pragma unroll
                for (int j = 0; j < TN; j++) {
                    acc[i][j] = (q & 1) ? mx4_mfma<1>(cur.a[q][i], cur.b[q][j], acc[i][j], sa[i], sb[j])
                                        : mx4_mfma<0>(cur.a[q][i], cur.b[q][j], acc[i][j], sa[i], sb[j]);
                    // the next loads, spread over the slot's MFMAs
                    constexpr int SPREAD = STEPS * TM * TN;
                    const int x = (q * TM + i) * TN + j;
#pragma unroll
                    for (int d = 0; d < L; d++)
                        if (d >= x * L / SPREAD && d < (x + 1) * L / SPREAD) load(d, into, sure, more);
                    __builtin_amdgcn_sched_barrier(0);
                }
        }
        wait(std::integral_constant<int, NS - 2>{}, more);
    };
#pragma unroll
    for (int s = 0; s < NS; s++)
#pragma unroll
        for (int d = 0; d < L; d++) load(d, s, std::false_type{}, s < nst);
    wait(std::integral_constant<int, NS - 1>{}, nst >= NS);
    Fragments even, odd;
    read(0, even);
    wait(std::integral_constant<int, NS - 2>{}, nst >= NS);
    int s = 0;
    if constexpr (C::STRAIGHT) {
        for (; s + NS + 1 < nst; s += 2) {
            slot(std::true_type{}, s, even, odd);
            slot(std::true_type{}, s + 1, odd, even);
        }
    }
    for (;;) {
        slot(std::false_type{}, s, even, odd);
        if (++s == nst) break;
        slot(std::false_type{}, s, odd, even);
        if (++s == nst) break;
    }
    __syncthreads();

    // ---- outputs.  A 32 x 32 tile's registers hold 32 columns of two rows per
    // register: 128 contiguous bytes a row in fp32, stored as they are.  16-bit
    // outputs go through the wave's own part of the LDS, a row of tiles at a time,
    // and leave as 16 bytes per lane, 64 TN contiguous bytes a row.
    if (a.dt == ROW_F32 || a.splits > 1) {
        float *out = a.splits > 1 ? a.partial + z * a.m * a.n : reinterpret_cast<float *>(a.y);
        const int64_t ld = a.splits > 1 ? a.n : a.ldy;
#pragma unroll
        for (int i = 0; i < TM; i++)
#pragma unroll
            for (int j = 0; j < TN; j++) {
                const int64_t row = (rt0 + wm * TM + i) * TILE_N, col = (ct0 + wn * TN + j) * TILE_N;
                float *p = out + row * ld + col + (4 * h * ld + r);  // register v: row v % 4 + 8 (v / 4) + 4 h, column r
                if (row + 32 <= a.m && col + 32 <= a.n) {
#pragma unroll
                    for (int v = 0; v < 16; v++) p[(v % 4 + 8 * (v / 4)) * ld] = acc[i][j][v];
                } else if (col + r < a.n) {
#pragma unroll
                    for (int v = 0; v < 16; v++)
                        if (row + mfma32_row(v, lane) < a.m) p[(v % 4 + 8 * (v / 4)) * ld] = acc[i][j][v];
                }
            }
        return;
    }
    const int64_t col0 = (ct0 + wn * TN) * TILE_N;
    uint16_t *y = reinterpret_cast<uint16_t *>(a.y);
    constexpr int PIECES = TN * 4;  // of 16 bytes in a row
    uint16_t *mine = reinterpret_cast<uint16_t *>(smem) + wave * TN * 1024;
#pragma unroll
    for (int i = 0; i < TM; i++) {
#pragma unroll
        for (int j = 0; j < TN; j++)
#pragma unroll
            for (int v = 0; v < 16; v++)
                mine[mfma32_row(v, lane) * (TN * 32) + j * 32 + r] =
                    a.dt == ROW_F16 ? f16_bits(acc[i][j][v]) : bf16_bits(acc[i][j][v]);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wave's own writes, read below by other lanes of it
#pragma unroll
        for (int q = 0; q < 32 * PIECES / 64; q++) {
            const int lr = (q * 64 + lane) / PIECES, lc = (q * 64 + lane) % PIECES * 8;
            const int64_t row = (rt0 + wm * TM + i) * 32 + lr, col = col0 + lc;
            const v4u u = *reinterpret_cast<const v4u *>(mine + lr * (TN * 32) + lc);
            if (row >= a.m) continue;
            if (col + 8 <= a.n) {
                *reinterpret_cast<v4u_any *>(y + row * a.ldy + col) = u;
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    if (col + e < a.n) y[row * a.ldy + col + e] = (uint16_t)(u[e >> 1] >> (16 * (e & 1)));
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// y = the splits' partial sums added in ascending order (the order is fixed: the
// same inputs give the same bits).  140 x 10240, three splits: 5.7 us, 22.9 MB.
__global__ __launch_bounds__(256) void mx4_reduce_kernel(Mx4Args a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.m * a.n) return;
    float s = a.partial[i];
    for (int64_t z = 1; z < a.splits; z++) s += a.partial[z * a.m * a.n + i];
    mx4_store(a.y, a.dt, (i / a.n) * a.ldy + i % a.n, s);
}

// ---------------------------------------------------------------------------
// Few rows: the weights are streamed straight into registers, once per block of
// ROWS rows.
//
// Bound by the weights' way from memory: 16 x 17408 x 5120 11.2 us, 48.9 MB, 4.4
// TB/s (9.8 at best; a copy reaches 5.15); 1 x 1024 x 5120, 32 workgroups and 2.8 MB,
// 3.7 us of launch and load latency.  With fewer column tiles than CUs, or a K of
// several chunks, less: 16 x 5120 x 17408 11.0 us, 64 x 5120 x 17408 23.3.
//
// A workgroup takes one 32-column tile (blockIdx.x) of one block of rows
// (blockIdx.y) over the whole of K; its waves take the stages round-robin, each
// with its next DEPTH records in flight, and their sums meet in LDS, added in wave
// order.  The rows' codes and scales are staged
// in LDS, CHUNK stages at a time (the LDS bounds how many workgroups share a
// CU), the codes by direct loads issued before the weights': a row's four
// 16-byte chunks of a stage lie at chunk ^ f(row), so that reading one chunk of
// 16 or 32 rows spreads over all banks, and a load still takes 64 contiguous
// bytes a row.  With ROWS = 16 the matrix instruction's other 16 rows read the
// same ones (their outputs are dropped).
// ---------------------------------------------------------------------------
__device__ __forceinline__ int mx4_swizzle(int row) { return ((row >> 1) ^ (row >> 2)) & 3; }

template <int ROWS_, int WAVES_, int DEPTH_, int CHUNK_KB_>
struct Mx4Stream {
    static constexpr int ROWS = ROWS_, WAVES = WAVES_, DEPTH = DEPTH_, NT = 64 * WAVES;
    static constexpr int TM = ROWS > 32 ? ROWS / 32 : 1;  // row tiles
    static constexpr int STAGE = ROWS * (MX4_ROW_BYTES + 4);  // LDS bytes of a stage: codes, then scales
    // what fits in the LDS share, in whole turns of the rings
    static constexpr int CHUNK = CHUNK_KB_ * 1024 / STAGE / (WAVES * DEPTH) * (WAVES * DEPTH);
    static_assert(CHUNK > 0, "one turn of the rings at least");
};
template <class C>
__host__ inline size_t mx4_stream_lds(int64_t k) {
    const int64_t st = mx4_stages(k);
    const size_t staged = (size_t)((st < C::CHUNK ? st : C::CHUNK) * C::STAGE), red = (size_t)C::WAVES * C::ROWS * 32 * 4;
    return staged > red ? staged : red;
}

template <class C>
__global__ __launch_bounds__(C::NT) void gemm_mx4_stream_kernel(Mx4Args a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int ROWS = C::ROWS, WAVES = C::WAVES, DEPTH = C::DEPTH, CHUNK = C::CHUNK, TM = C::TM;
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, r = lane & 31, ar = ROWS < 32 ? r % ROWS : r;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t nb = a.k / QK, tile = blockIdx.x, row0 = (int64_t)blockIdx.y * ROWS, stride = mx4_stride(a.k);
    const int stages = (int)mx4_stages(a.k);
    const uint8_t *rec = a.packed + tile * mx4_rec_stages(a.k) * MX4_REC;
    const uint32_t smem_base = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)smem;

    // codes of stages t0 .. t0 + cnt - 1: 1 KB (16 rows of a stage) a load
    auto stage_codes = [&](int t0, int cnt) {
        const int row = lane >> 2, chunk = (lane & 3) ^ mx4_swizzle(row);  // f has period 16
        for (int i = wave; i < cnt * (ROWS / 16); i += WAVES) {
            const int64_t b = min((int64_t)(t0 + i / (ROWS / 16)) * MX4_BLOCKS + chunk, nb - 1);
            const int64_t src = min(row0 + i % (ROWS / 16) * 16 + row, a.m - 1);
            mx4_load16(a.codes + src * (a.k / 2) + b * 16, __builtin_amdgcn_readfirstlane(smem_base + i * 1024));
        }
    };
    // their scales, by way of registers
    constexpr int HELD = (CHUNK * ROWS + C::NT - 1) / C::NT;
    uint32_t held[HELD];
    auto load_scales = [&](int t0, int cnt) {
#pragma unroll
        for (int j = 0; j < HELD; j++) {
            const int i = min(tid + j * C::NT, cnt * ROWS - 1), t = i / ROWS, row = i % ROWS;
            held[j] = *reinterpret_cast<const uint32_t *>(a.scales + min(row0 + row, a.m - 1) * stride +
                                                          (int64_t)(t0 + t) * MX4_BLOCKS);
        }
    };
    // Until the chunk's scales are there and with them its codes, whose loads are
    // older and return in order.  The compiler counts the loads behind them (the
    // weights' at the start, which stay in flight).
    auto wait_rows = [&] {
#pragma unroll
        for (int j = 0; j < HELD; j++) asm volatile("" ::"v"(held[j]) : "memory");
    };
    auto store_scales = [&](int t0, int cnt) {
        uint32_t *scl = reinterpret_cast<uint32_t *>(smem + cnt * ROWS * MX4_ROW_BYTES);
#pragma unroll
        for (int j = 0; j < HELD; j++) {
            const int i = tid + j * C::NT;
            if (i < cnt * ROWS) scl[i] = mx4_live_scales(held[j], t0 + i / ROWS, nb);
        }
    };
    // this wave's stages: wave, wave + WAVES, ...; past the end the last one
    // again (not computed), so that every wave has the same loads in flight
    struct Rec { v4u c0, c1; uint32_t s; } ring[DEPTH];
    auto load = [&](int t, Rec &R) {
        const uint8_t *p = rec + (int64_t)min(t, stages - 1) * MX4_REC;
        R.c0 = *reinterpret_cast<const v4u *>(p + 16 * lane);
        R.c1 = *reinterpret_cast<const v4u *>(p + 1024 + 16 * lane);
        R.s = *reinterpret_cast<const uint32_t *>(p + MX4_SCALE_OFF + 4 * r);
    };

    const int first = min(CHUNK, stages);
    stage_codes(0, first);
    load_scales(0, first);
    asm volatile("" ::: "memory");  // in this order: the wait for the rows leaves the weights in flight
#pragma unroll
    for (int d = 0; d < DEPTH; d++) load(wave + WAVES * d, ring[d]);

    v16f acc[TM];
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int v = 0; v < 16; v++) acc[i][v] = 0.0f;
    const int sw = mx4_swizzle(ar);
    wait_rows();
    for (int t0 = 0; t0 < stages; t0 += CHUNK) {
        const int cnt = min(CHUNK, stages - t0);
        if (t0) {
            __syncthreads();  // every wave is done with the last chunk
            stage_codes(t0, cnt);
            load_scales(t0, cnt);
            wait_rows();
        }
        store_scales(t0, cnt);
        __syncthreads();
        const uint8_t *scl = smem + cnt * ROWS * MX4_ROW_BYTES;
        for (int t = t0 + wave; t < t0 + cnt; t += WAVES * DEPTH) {
#pragma unroll
            for (int d = 0; d < DEPTH; d++) {
                const int u = t + WAVES * d;
                if (u < t0 + cnt) {
                    const uint8_t *p = smem + (u - t0) * ROWS * MX4_ROW_BYTES + ar * MX4_ROW_BYTES;
                    v4u x0[TM], x1[TM];
                    uint32_t sa[TM];
#pragma unroll
                    for (int i = 0; i < TM; i++) {
                        x0[i] = mx4_lds<v4u>(p + i * 32 * MX4_ROW_BYTES + (h ^ sw) * 16);
                        x1[i] = mx4_lds<v4u>(p + i * 32 * MX4_ROW_BYTES + ((2 + h) ^ sw) * 16);
                        sa[i] = mx4_lds<uint32_t>(scl + ((u - t0) * ROWS + i * 32 + ar) * 4) >> (8 * h);
                    }
                    const uint32_t sb = ring[d].s >> (8 * h);
#pragma unroll
                    for (int i = 0; i < TM; i++) {
                        acc[i] = mx4_mfma<0>(x0[i], ring[d].c0, acc[i], sa[i], sb);
                        acc[i] = mx4_mfma<1>(x1[i], ring[d].c1, acc[i], sa[i], sb);
                    }
                    load(u + WAVES * DEPTH, ring[d]);
                }
            }
        }
    }
    __syncthreads();
    // sums of the waves: [wave][row][column]
    float *red = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int v = 0; v < ROWS / 2; v++) red[(wave * ROWS + (v >> 4) * 32 + mfma32_row(v & 15, lane)) * 32 + r] = acc[v >> 4][v & 15];
    __syncthreads();
    for (int i = tid; i < ROWS * 32; i += C::NT) {
        const int64_t row = row0 + i / 32, col = tile * TILE_N + i % 32;
        float s = red[i];
#pragma unroll
        for (int w = 1; w < WAVES; w++) s += red[w * ROWS * 32 + i];
        if (row < a.m && col < a.n) mx4_store(a.y, a.dt, row * a.ldy + col, s);
    }
}

// y[0..m)[0..n) = 0 (k == 0: an empty sum).
__global__ void zero_typed_kernel(uint8_t *y, int dt, int64_t m, int64_t n, int64_t ldy) {
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < m * n; i += stride)
        mx4_store(y, dt, (i / n) * ldy + i % n, 0.0f);
}

}  // namespace w4a4
