// The paged key/value cache in 8 bits: its layout, the rows of new tokens
// written into it (with the RMS norm and the rotary positions of their heads on
// the way), and tokens read back.
//
// A page holds a whole number of blocks of 32 tokens for each key/value head;
// the pool is [pages][heads][blocks of a page] blocks of 64 D bytes, D the width
// of a head: the keys' codes, then the values', OCP E4M3 both.  A block has two
// power-of-two scales (E8M0 bytes), one for its keys and one for its values: code c
// stands for c 2^(byte - 127).  Codes lie as the matrix cores read them, so that a
// wave's 16-byte loads are contiguous and none of a block has to move between lanes:
//   keys    [D / 32][2][32 tokens][16]: bytes 1024 c + 512 h + 16 t + j, channel
//           32 c + 16 h + j of token t;
//   values  [D / 32][2][32 channels][16]: token 16 i + 8 q + 4 h + r of channel
//           32 c + d at byte 1024 c + 512 h + 16 d + 8 q + 4 i + r.  A 32 x 32
//           product of keys and queries leaves tokens 8 j + 4 h + r in lane half h:
//           the same 16 tokens, as the next product wants them.
//
// A block's scale is the least power of two that holds its largest value, and
// grows when a later token needs it: the codes of the tokens before are then
// rounded again on the coarser grid, which is exact but for values below
// 2^-6 of a code.  (A grid of 8-bit integers would lose half a step every time.)
//
// What bounds these kernels.  Many tokens (8 prompts of up to 1023 tokens, 32 + 2 x 4 heads of
// 128, three axes, 94 MB): 31 us, 3.0 TB/s, where a copy reaches 4.9 and the queries copied
// alone take 19; vector instructions (norm, rotation, codes) issue for half of the time, and
// waves wait for their loads for half of theirs: neither alone.  A prompt of 512 (10 us) has
// a fifth of its time in vector instructions: the chain below, in 68 workgroups for its
// blocks.  A decode step is the chain of dependent loads: lengths, page, scale (one token
// 5.8 us, 64 sequences' 6.0; the norm's sum and the table's row cost 1 us each of it).
#pragma once

#include "common.h"
#include "k_rows.h"

namespace w4a4 {

constexpr int KV_BLOCK = 32;     // tokens of a block
// Threads of a workgroup of the kernels here: 32 tokens of a head's rows, 8 channels
// a thread, in one or two steps.
__host__ __device__ constexpr int kv_threads(int dim) { return dim == 256 ? 512 : 256; }

typedef float v2f __attribute__((ext_vector_type(2)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

struct KvPool {
    uint8_t *codes, *scales;
    int32_t pages, heads, per_page;  // per_page: blocks of a page
};
struct KvBatch {
    const int32_t *pages, *starts, *lens;
    int64_t ld;                     // of pages
    int32_t per_seq, seqs, tokens;  // per_seq: pages of a sequence
};

// A sequence: its first row, its rows, and its tokens with them.  Whatever the
// arrays hold, rows lie in [0, tokens) and tokens in its pages.
struct KvSeq {
    int row, n, len;
    __device__ __forceinline__ int first() const { return len - n; }  // token of its first row (< 0: more rows than tokens)
};
__device__ __forceinline__ KvSeq kv_seq(const KvBatch &s, int page_tokens, int b) {
    const int lo = min(max(s.starts[b], 0), s.tokens), hi = min(max(s.starts[b + 1], lo), s.tokens);
    return KvSeq{lo, hi - lo, (int)min((int64_t)max(s.lens[b], 0), (int64_t)s.per_seq * page_tokens)};
}

// Where block `blk` of a sequence lies for one head, in blocks of the pool; -1
// where the sequence has no page there.
__device__ __forceinline__ int kv_block(const KvPool &p, const KvBatch &s, int b, int head, int blk) {
    const int slot = blk / p.per_page, page = s.pages[b * s.ld + slot];
    return (uint32_t)page < (uint32_t)p.pages ? (page * p.heads + head) * p.per_page + (blk - slot * p.per_page) : -1;
}

// x of another lane by a DPP pattern (no LDS round trip, as __shfl has); 0 where
// the pattern has no lane, or ROWS leaves a row of 16 out.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ int32_t dpp_of(int32_t x) {
    return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xF, true);
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ int64_t dpp_of(int64_t x) {
    return (int64_t)((uint64_t)(uint32_t)dpp_of<CTRL, ROWS>((int32_t)(x >> 32)) << 32 | (uint32_t)dpp_of<CTRL, ROWS>((int32_t)x));
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp_of(double x) {
    return __builtin_bit_cast(double, dpp_of<CTRL, ROWS>(__builtin_bit_cast(int64_t, x)));
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp_of(float x) {
    return __builtin_bit_cast(float, dpp_of<CTRL, ROWS>(__builtin_bit_cast(int32_t, x)));
}
constexpr int DPP_SHR1 = 0x111, DPP_SHR2 = 0x112, DPP_SHR4 = 0x114, DPP_SHR8 = 0x118, DPP_BCAST15 = 0x142, DPP_BCAST31 = 0x143,
              DPP_XOR1 = 0xB1, DPP_XOR2 = 0x4E, DPP_MIRROR8 = 0x141, DPP_MIRROR16 = 0x140;
// Inclusive sum over the wave's lanes.
template <class T>
__device__ __forceinline__ T wave_scan(T x) {
    x += dpp_of<DPP_SHR1>(x);
    x += dpp_of<DPP_SHR2>(x);
    x += dpp_of<DPP_SHR4>(x);
    x += dpp_of<DPP_SHR8>(x);
    x += dpp_of<DPP_BCAST15, 0xA>(x);
    return x + dpp_of<DPP_BCAST31, 0xC>(x);
}
// x over the lanes l and l ^ 16, or l ^ 32: f of both.
template <class F>
__device__ __forceinline__ uint32_t swap16(uint32_t x, F f) {
    const auto y = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return f(y[0], y[1]);
}
template <class F>
__device__ __forceinline__ uint32_t swap32(uint32_t x, F f) {
    const auto y = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return f(y[0], y[1]);
}
// The sum over a row's LANES lanes (8, 16 or 32), the same in each.
template <int LANES>
__device__ __forceinline__ double lanes_sum(double x) {
    x += dpp_of<DPP_XOR1>(x);
    x += dpp_of<DPP_XOR2>(x);
    x += dpp_of<DPP_MIRROR8>(x);  // a quad's lanes hold the same: as good as l ^ 4
    if constexpr (LANES > 8) x += dpp_of<DPP_MIRROR16>(x);
    if constexpr (LANES > 16) {
        const uint64_t u = __builtin_bit_cast(uint64_t, x);
        const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
        x = __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]) + __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
    }
    return x;
}
// The largest of the wave's lanes, in each.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    auto larger = [](uint32_t a, uint32_t b) { return max(a, b); };
    x = max(x, (uint32_t)dpp_of<DPP_XOR1>((int32_t)x));
    x = max(x, (uint32_t)dpp_of<DPP_XOR2>((int32_t)x));
    x = max(x, (uint32_t)dpp_of<DPP_MIRROR8>((int32_t)x));
    x = max(x, (uint32_t)dpp_of<DPP_MIRROR16>((int32_t)x));
    return swap32(swap16(x, larger), larger);
}
__device__ __forceinline__ int32_t wave_pick(int32_t x, int lane) { return __builtin_amdgcn_readlane(x, lane); }
__device__ __forceinline__ int64_t wave_pick(int64_t x, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)x, lane), hi = __builtin_amdgcn_readlane((int)(x >> 32), lane);
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// The sequence that holds item `id` (uniform) when sequence b has weight(b)
// items, and the item's number in it (in id); -1 past the last.  Every wave for
// itself: 64 sequences a step, no barrier.
template <class T, class F>
__device__ __forceinline__ int kv_find(int seqs, T &id, int lane, F weight) {
    if (seqs == 1) return id < weight(0) ? 0 : -1;
    for (int base = 0; base < seqs; base += 64) {
        const T w = base + lane < seqs ? weight(base + lane) : 0;
        const T sum = wave_scan(w), total = wave_pick(sum, 63);
        if (id < total) {
            const int at = __builtin_ctzll(__ballot(sum > id));
            id -= wave_pick(sum, at) - wave_pick(w, at);
            return base + at;
        }
        id -= total;
    }
    return -1;
}

// Blocks that the tokens [first, len) of a sequence reach.
__device__ __forceinline__ int kv_first_block(const KvSeq &s) { return max(s.first(), 0) / KV_BLOCK; }
__device__ __forceinline__ int kv_blocks(const KvSeq &s) {
    return s.n > 0 && s.len > 0 ? (s.len - 1) / KV_BLOCK - kv_first_block(s) + 1 : 0;
}

// The exponent of a block whose largest magnitude has these bits: the least
// e >= -127 with it at most 448 2^e.
__device__ __forceinline__ int kv_exponent(uint32_t top) {
    return max((int)(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0), -127);
}

// Two values |x| <= 448 as E4M3, to nearest even, in the low or high half of w.
template <bool HIGH>
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w, float a, float b) {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)w, HIGH);
}
__device__ __forceinline__ uint32_t e4m3_quad(float a, float b, float c, float d) {
    return e4m3_pair<true>(e4m3_pair<false>(0, a, b), c, d);
}
__device__ __forceinline__ void e4m3_values(uint32_t w, float v[4]) {
    const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    v[0] = lo.x, v[1] = lo.y, v[2] = hi.x, v[3] = hi.y;
}
// Four codes on a grid 2^shift as coarse.
__device__ __forceinline__ uint32_t e4m3_coarser(uint32_t w, int shift) {
    float v[4];
    e4m3_values(w, v);
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = ldexpf(v[i], -shift);
    return e4m3_quad(v[0], v[1], v[2], v[3]);
}
// Four codes, of which `keep` (bytes 00 or FF) come from a and the rest from b.
__device__ __forceinline__ uint32_t bytes_of(uint32_t keep, uint32_t a, uint32_t b) { return (a & keep) | (b & ~keep); }

// Bytes of the dword (q, i) of a value piece of half h (see the layout) whose
// tokens lie in [lo, hi): FF, else 00.
__device__ __forceinline__ uint32_t kv_token_bytes(int q, int i, int h, int lo, int hi) {
    const int t = 16 * i + 8 * q + 4 * h;
    const int a = min(max(lo - t, 0), 4), b = min(max(hi - t, 0), 4);  // bytes a .. b - 1
    return (uint32_t)((0xFFFFFFFFull >> (32 - 8 * b)) & ~(0xFFFFFFFFull >> (32 - 8 * a)));
}

struct AppendArgs {
    const uint8_t *q, *k, *v;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;  // strides, in elements
    const float *q_weight, *k_weight;
    double eps;
    const float *rope;  // [positions][half] cosines, [half] sines
    const int32_t *positions;
    int64_t ld_positions;
    const uint8_t *axes;
    int32_t rope_rows, half, n_axes, interleaved;
    uint8_t *q_out;
    int64_t o_row, o_head;
    int32_t dt, odt, q_heads, q_passes;
    int32_t kv_groups;  // workgroups of keys and values, before those of queries
    KvPool pool;
    KvBatch batch;
};

// The cosines and sines that turn channels d .. d + 7 of a head of a row at
// token `index` of its sequence: pair d + i (halves) or d / 2 + i, i < 4
// (interleaved).  Positions outside the table give NaN; channels that are not
// turned nothing.
struct Turn {
    v4u c[2], s[2];
};
typedef v4u v4u_word __attribute__((aligned(4)));
__device__ __forceinline__ void rope_turn(const AppendArgs &a, int row, int index, int d, Turn &t) {
    if (d >= 2 * a.half) return;
    const int pair = a.interleaved ? d / 2 : d >= a.half ? d - a.half : d;
    constexpr uint32_t bad = 0x7FC00000u;
    int axis = 0;
    bool mixed = false;  // pairs of more than one axis among this lane's
    if (a.axes) {
        axis = a.axes[pair];
#pragma unroll
        for (int i = 1; i < 8; i++)
            if (i < 4 || !a.interleaved) mixed |= a.axes[pair + i] != axis;
    }
    if (!mixed) {
        const int at = !a.positions ? index : axis < a.n_axes ? a.positions[axis * a.ld_positions + row] : -1;
        const bool in = (uint32_t)at < (uint32_t)a.rope_rows;
        const float *p = a.rope + (in ? (int64_t)at * 2 * a.half : 0) + pair;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (i && a.interleaved) continue;
            t.c[i] = in ? reinterpret_cast<const v4u_word *>(p)[i] : v4u{bad, bad, bad, bad};
            t.s[i] = in ? reinterpret_cast<const v4u_word *>(p + a.half)[i] : v4u{bad, bad, bad, bad};
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
        if (i >= 4 && a.interleaved) continue;
        const int of = a.axes[pair + i], at = of < a.n_axes ? a.positions[of * a.ld_positions + row] : -1;
        const bool in = (uint32_t)at < (uint32_t)a.rope_rows;
        const float *p = a.rope + (in ? (int64_t)at * 2 * a.half : 0) + pair + i;
        t.c[i / 4][i % 4] = in ? __float_as_uint(p[0]) : bad, t.s[i / 4][i % 4] = in ? __float_as_uint(p[a.half]) : bad;
    }
}

// A head's row is held by D / 8 consecutive lanes of a wave, a lane channels d ..
// d + 7.  Its RMS norm when there is a weight, as in w4a4_rms_norm_quantize (fp64
// sum and root, one rounding), then its leading 2 half channels turned in pairs,
// one fp32 operation at a time; the other channels of a lane's pairs, halves
// apart, come from the lane that holds them.  Every lane of the wave takes part.
template <int D>
__device__ __forceinline__ void head_row(const AppendArgs &a, const Raw8 &raw, const float *weight, const float w[8], const Turn &t,
                                         int d, float v[8]) {
    to_f32(raw, a.dt, v);
    if (weight) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < 8; i++) sum = fma((double)v[i], (double)v[i], sum);
        const float root = (float)rsqrt64(fma(lanes_sum<D / 8>(sum), 1.0 / D, a.eps));
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = v[i] * root * w[i];
    }
    if (!a.half) return;
    auto c = [&](int i) { return __uint_as_float(t.c[i / 4][i % 4]); };
    auto s = [&](int i) { return __uint_as_float(t.s[i / 4][i % 4]); };
    if (a.interleaved) {
        if (d >= 2 * a.half) return;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float p = v[2 * i], r = v[2 * i + 1];
            v[2 * i] = p * c(i) - r * s(i);
            v[2 * i + 1] = r * c(i) + p * s(i);
        }
        return;
    }
    const int mate = ((threadIdx.x & 63) + (d < a.half ? a.half / 8 : -a.half / 8)) & 63;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; i++) y[i] = __shfl(v[i], mate);
    if (d >= 2 * a.half) return;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float ys = y[i] * s(i);
        v[i] = v[i] * c(i) + (d < a.half ? -ys : ys);
    }
}
__device__ __forceinline__ void load_weight(const float *weight, int d, float w[8]) {
    if (!weight) return;
#pragma unroll
    for (int i = 0; i < 8; i++) w[i] = weight[d + i];
}

// Sequence of a row (uniform): the last that begins at or before it; -1 for rows
// outside every sequence.
__device__ __forceinline__ int seq_of_row(const KvBatch &s, int row, int lane) {
    int before = 0;
    for (int base = 0; base <= s.seqs; base += 64)
        before += __builtin_popcountll(__ballot(base + lane <= s.seqs && s.starts[min(base + lane, s.seqs)] <= row));
    return before == 0 || before > s.seqs ? -1 : before - 1;
}

template <int D>
constexpr int kv_pitch() { return D / 8 * 16; }  // LDS bytes of one channel residue, below

// Where token t's byte of channel d lies in LDS: value pieces of 16 bytes (one
// channel and half) ordered by channel residue mod 8, so that the lanes of a row
// (8 channels each) touch consecutive pieces.
template <int D>
__device__ __forceinline__ int kv_lds_piece(int d, int h) { return (h * 8 + d % 8) * kv_pitch<D>() + d / 8 * 16; }
__device__ __forceinline__ int kv_piece_byte(int t) { return (t >> 3 & 1) * 8 + (t >> 4) * 4 + (t & 3); }

// One block of one head for a workgroup: the rows of new tokens that fall in it.
// Every load of its rows is asked for before the page is waited for.
template <int D>
__device__ __forceinline__ void append_block(const AppendArgs &a, int id, uint8_t *smem) {
    constexpr int THREADS = kv_threads(D), LANES = D / 8, ROWS = THREADS / LANES, PASSES = KV_BLOCK / ROWS;
    const int tid = threadIdx.x, lane = tid & 63, page_tokens = a.pool.per_page * KV_BLOCK;
    const int head = id % a.pool.heads;
    int32_t slot = id / a.pool.heads;
    const int b = kv_find(a.batch.seqs, slot, lane, [&](int i) { return kv_blocks(kv_seq(a.batch, page_tokens, i)); });
    if (b < 0) return;
    const KvSeq s = kv_seq(a.batch, page_tokens, b);
    const int blk = kv_first_block(s) + slot, t0 = blk * KV_BLOCK;
    const int kept = max(s.first() - t0, 0), lo = kept, hi = min(s.len - t0, KV_BLOCK);  // new tokens lo .. hi - 1

    const int d = tid % LANES * 8, r0 = tid / LANES, size = row_size(a.dt);
    Raw8 raw[PASSES] = {}, vraw[PASSES] = {};
    Turn turn[PASSES] = {};
    float weight[8] = {};
#pragma unroll
    for (int p = 0; p < PASSES; p++) {
        const int t = r0 + p * ROWS, index = t0 + t;
        if (t < lo || t >= hi) continue;
        const int64_t row = s.row + (index - s.first());
        raw[p] = load_raw8(a.k + (row * a.k_row + head * a.k_head + d) * size, a.dt);
        vraw[p] = load_raw8(a.v + (row * a.v_row + head * a.v_head + d) * size, a.dt);
        rope_turn(a, (int)row, index, d, turn[p]);
    }
    load_weight(a.k_weight, d, weight);
    const int at = kv_block(a.pool, a.batch, b, head, blk);
    if (at < 0) return;
    uint8_t *codes = a.pool.codes + (int64_t)at * (64 * D);
    uint16_t *scale = reinterpret_cast<uint16_t *>(a.pool.scales) + at;
    int was = kept ? *scale : 0;

    float k[PASSES][8], v[PASSES][8];
    bool lost[PASSES];
    uint32_t ktop = 0, vtop = 0;
#pragma unroll
    for (int p = 0; p < PASSES; p++) {
        const int t = r0 + p * ROWS;
        const bool live = t >= lo && t < hi;
        lost[p] = false;
        if (p * ROWS >= hi || (p + 1) * ROWS <= lo) continue;  // uniform
        head_row<D>(a, raw[p], a.k_weight, weight, turn[p], d, k[p]);
        to_f32(vraw[p], a.dt, v[p]);
        uint32_t kt = 0, vt = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            kt = max(kt, __float_as_uint(k[p][i]) & 0x7FFFFFFFu);
            vt = max(vt, __float_as_uint(v[p][i]) & 0x7FFFFFFFu);
        }
        // a token with a NaN or an infinity: known to all lanes of its row
        const uint64_t bad = __ballot(live && max(kt, vt) >= 0x7F800000u);
        lost[p] = (bad >> (lane / LANES * LANES) & ((1ull << LANES) - 1)) != 0;
        if (live && !lost[p]) ktop = max(ktop, kt), vtop = max(vtop, vt);
    }
    ktop = wave_max(ktop), vtop = wave_max(vtop);
    uint32_t *tops = reinterpret_cast<uint32_t *>(smem + 32 * D);  // [waves][2]
    if (lane == 0) tops[tid / 64 * 2] = ktop, tops[tid / 64 * 2 + 1] = vtop;
    asm volatile("" : "+v"(was));  // every wave has read the old scales before one writes the new
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; w++) ktop = max(ktop, tops[2 * w]), vtop = max(vtop, tops[2 * w + 1]);
    const int kwas = (was & 255) - 127, vwas = (was >> 8) - 127;
    const int ke = kept ? max(kv_exponent(ktop), kwas) : kv_exponent(ktop);
    const int ve = kept ? max(kv_exponent(vtop), vwas) : kv_exponent(vtop);
    if (tid == 0) *scale = (uint16_t)((ke + 127) | (ve + 127) << 8);

    // Few new values and no new grid: their bytes alone.  Otherwise the block's
    // pieces of 16 tokens are written whole, with the bytes of the others read: 16
    // stores of D / 8 lanes for a token's bytes, against two reads and writes of
    // all 2 D pieces.
    const bool bytes = hi - lo <= 2 && !(kept && ve > vwas);
    uint8_t *values = codes + 32 * D;
#pragma unroll
    for (int p = 0; p < PASSES; p++) {
        const int t = r0 + p * ROWS;
        if (t < lo || t >= hi) continue;
        v2u kc = {0x7F7F7F7Fu, 0x7F7F7F7Fu}, vc = {0u, 0u};
        if (!lost[p]) {
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const float *x = k[p] + 4 * i, *y = v[p] + 4 * i;
                kc[i] = e4m3_quad(ldexpf(x[0], -ke), ldexpf(x[1], -ke), ldexpf(x[2], -ke), ldexpf(x[3], -ke));
                vc[i] = e4m3_quad(ldexpf(y[0], -ve), ldexpf(y[1], -ve), ldexpf(y[2], -ve), ldexpf(y[3], -ve));
            }
        }
        *reinterpret_cast<v2u *>(codes + d / 16 * 512 + t * 16 + d % 16) = kc;
        const int h = t >> 2 & 1, byte = kv_piece_byte(t);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint8_t c = (uint8_t)(vc[i / 4] >> (i % 4 * 8));
            if (bytes) values[(d + i) / 32 * 1024 + h * 512 + (d + i) % 32 * 16 + byte] = c;
            else smem[kv_lds_piece<D>(d + i, h) + byte] = c;
        }
    }
    if (kept && ke > kwas) {  // the tokens before, on the coarser grid
        for (int u = tid; u < 2 * D; u += THREADS) {
            if (u % 32 >= kept) continue;
            v4u *p = reinterpret_cast<v4u *>(codes) + u;
            v4u x = *p;
#pragma unroll
            for (int i = 0; i < 4; i++) x[i] = e4m3_coarser(x[i], ke - kwas);
            *p = x;
        }
    }
    if (bytes) return;  // uniform
    __syncthreads();
    const bool grown = kept && ve > vwas, whole = hi - lo == KV_BLOCK;
    for (int u = tid; u < 2 * D; u += THREADS) {
        const int h = u / 32 % 2, c = u / 64 * 32 + u % 32;
        v4u *p = reinterpret_cast<v4u *>(values) + u;
        v4u x = *reinterpret_cast<const v4u *>(smem + kv_lds_piece<D>(c, h));
        if (!whole) {
            const v4u old = *p;
#pragma unroll
            for (int i = 0; i < 4; i++) {  // dword 2 q + i
                const int q = i >> 1, j = i & 1;
                uint32_t o = old[i];
                if (grown) o = bytes_of(kv_token_bytes(q, j, h, 0, kept), e4m3_coarser(o, ve - vwas), o);
                x[i] = bytes_of(kv_token_bytes(q, j, h, lo, hi), x[i], o);
            }
        }
        *p = x;
    }
}

// The queries of a row: D / 8 lanes a head, a wave's heads from one row, so that
// cosines, sines and weights are loaded once for a.q_passes steps of 64 / LANES
// heads (5156 rows of 32 heads of 128: 99 us before that and without loads ahead, 46 with
// both, 31 with the pairs exchanged between lanes and one table row a lane).
template <int D>
__device__ __forceinline__ void append_queries(const AppendArgs &a, int id) {
    constexpr int LANES = D / 8, HEADS = 64 / LANES, AHEAD = 4;
    const int lane = threadIdx.x & 63, per = HEADS * a.q_passes, groups = (a.q_heads + per - 1) / per;
    const int64_t task = (int64_t)id * (kv_threads(D) / 64) + threadIdx.x / 64;
    const int row = __builtin_amdgcn_readfirstlane((int)(task / groups)), head0 = (int)(task % groups) * per + lane / LANES;
    if (row >= a.batch.tokens) return;
    const int d = lane % LANES * 8, size = row_size(a.dt), end = min(a.q_heads, head0 - lane / LANES + per);
    const uint8_t *src = a.q + ((int64_t)row * a.q_row + d) * size;
    Raw8 raw[AHEAD] = {};
    auto load = [&](int h, Raw8 &x) {
        if (h < end) x = load_raw8(src + h * a.q_head * size, a.dt);
    };
#pragma unroll
    for (int i = 0; i < AHEAD; i++) load(head0 + i * HEADS, raw[i]);
    float weight[8] = {};
    load_weight(a.q_weight, d, weight);
    const int b = seq_of_row(a.batch, row, lane);
    if (b < 0) return;
    Turn turn = {};
    if (a.half) {
        int index = 0;
        if (!a.positions) {
            const KvSeq s = kv_seq(a.batch, a.pool.per_page * KV_BLOCK, b);
            index = s.first() + (row - s.row);
        }
        rope_turn(a, row, index, d, turn);
    }
    uint8_t *dst = a.q_out + ((int64_t)row * a.o_row + d) * 2;
    for (int h = head0; h - lane / LANES < end; h += AHEAD * HEADS) {
#pragma unroll
        for (int i = 0; i < AHEAD; i++) {
            const int at = h + i * HEADS;
            float x[8];
            head_row<D>(a, raw[i], a.q_weight, weight, turn, d, x);
            if (at < end) store_row8(dst + (int64_t)at * a.o_head * 2, a.odt, x);
            load(at + AHEAD * HEADS, raw[i]);
        }
    }
}

template <int D>
__global__ __launch_bounds__(kv_threads(D)) void append_kernel(AppendArgs a) {
    __shared__ __align__(16) uint8_t smem[32 * D + kv_threads(D) / 8];
    if ((int)blockIdx.x < a.kv_groups) append_block<D>(a, (int)blockIdx.x, smem);
    else append_queries<D>(a, (int)blockIdx.x - a.kv_groups);
}

struct KvReadArgs {
    KvPool pool;
    KvBatch batch;
    uint8_t *k, *v;
    int64_t k_row, k_head, v_row, v_head;
    int32_t dt;
};

// A batch's last rows' keys and values: one block of one head a workgroup.
// Tokens without a page, or before a sequence's first, read as zeros.
template <int D>
__global__ __launch_bounds__(kv_threads(D)) void read_kv_kernel(KvReadArgs a) {
    constexpr int THREADS = kv_threads(D), LANES = D / 8, ROWS = THREADS / LANES, PASSES = KV_BLOCK / ROWS;
    __shared__ __align__(16) uint8_t smem[32 * D];
    const int tid = threadIdx.x, lane = tid & 63, page_tokens = a.pool.per_page * KV_BLOCK;
    const int head = (int)(blockIdx.x % a.pool.heads);
    int32_t slot = (int)(blockIdx.x / a.pool.heads);
    // rows before the first token count as blocks of their own, ahead of the others
    auto lead = [](const KvSeq &s) { return (max(-s.first(), 0) + KV_BLOCK - 1) / KV_BLOCK; };
    const int b = kv_find(a.batch.seqs, slot, lane, [&](int i) {
        const KvSeq s = kv_seq(a.batch, page_tokens, i);
        return lead(s) + kv_blocks(s);
    });
    if (b < 0) return;
    const KvSeq s = kv_seq(a.batch, page_tokens, b);
    const int t0 = (kv_first_block(s) + slot - lead(s)) * KV_BLOCK;  // negative: rows without a token
    const int at = t0 < 0 ? -1 : kv_block(a.pool, a.batch, b, head, t0 / KV_BLOCK);
    const uint8_t *codes = a.pool.codes + (int64_t)max(at, 0) * (64 * D);
    int ke = 0, ve = 0;
    if (at >= 0) {
        const int e = reinterpret_cast<const uint16_t *>(a.pool.scales)[at];
        ke = (e & 255) - 127, ve = (e >> 8) - 127;
        for (int u = tid; u < 2 * D; u += THREADS)
            *reinterpret_cast<v4u *>(smem + kv_lds_piece<D>(u / 64 * 32 + u % 32, u / 32 % 2)) =
                reinterpret_cast<const v4u *>(codes + 32 * D)[u];
    }
    __syncthreads();
    const int d = tid % LANES * 8;
#pragma unroll
    for (int p = 0; p < PASSES; p++) {
        const int t = tid / LANES + p * ROWS, index = t0 + t;
        if (index < s.first() || index >= (t0 < 0 ? 0 : s.len)) continue;
        const int64_t row = s.row + (index - s.first());
        float x[8] = {}, y[8] = {};
        if (at >= 0) {
            const v2u kc = *reinterpret_cast<const v2u *>(codes + d / 16 * 512 + t * 16 + d % 16);
            uint32_t vc[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; i++)
                vc[i / 4] |= (uint32_t)smem[kv_lds_piece<D>(d + i, t >> 2 & 1) + kv_piece_byte(t)] << (i % 4 * 8);
            e4m3_values(kc.x, x), e4m3_values(kc.y, x + 4), e4m3_values(vc[0], y), e4m3_values(vc[1], y + 4);
#pragma unroll
            for (int i = 0; i < 8; i++) x[i] = ldexpf(x[i], ke), y[i] = ldexpf(y[i], ve);
        }
        const int size = row_size(a.dt);
        store_row8(a.k + (row * a.k_row + head * a.k_head + d) * size, a.dt, x);
        store_row8(a.v + (row * a.v_row + head * a.v_head + d) * size, a.dt, y);
    }
}

}  // namespace w4a4
