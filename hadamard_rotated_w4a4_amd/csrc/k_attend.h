// Attention over the paged 8-bit key/value cache (k_kv.h).
//
//   s_rj = scale sum_d q_rd k_jd,  p_rj = e^(s_rj - m_r),  o_r = sum_j p_rj v_j / sum_j p_rj
//
// over the tokens j that row r sees, in one pass: running maximum m and sum in
// fp32, 16 products in 16 bits an fp32 accumulator.  Keys become the queries' type
// (fp16 or bf16; an E4M3 code is exact in both) and values fp16 by the conversion
// instruction, two a lane.  The keys' scale goes into the factor of the exponent.
// p is rounded to fp16 (11 bits, as the output's own type or better), and summed as
// rounded, so that a row's weights add up to one.  The values' scale goes into the
// weights then, relative to a power of two of each row, 2^E (below), and 2^E at the end:
// exact but below 2^-14.  (Applied by the values' conversion it would be one E for all
// rows of a wave, and one that not all of them may see.)
//
// One row of 131072 tokens (24 heads over 4 of 256, 268 MB) takes 58 us, 4.6 TB/s; 32
// sequences of up to 16384 (48 over 8 of 128, 683 MB) 133, 5.1 TB/s: memory, where a
// copy reaches 4.9.  512 rows of 32768 tokens take 375 to 411 us (with the card's clock),
// 1.0 to 1.1 PFLOP/s, at D = 256, and of 8192 151, 660 TFLOP/s, at D = 128, where a large
// product reaches 1200.  A block's 32 x 32 scores cost a wave the same 90 vector instructions
// and 16 exponentials whatever D, and its keys and values D / 2 conversions, beside D / 8
// products, and these hardly overlap: at D = 128 the vector units are 40 % and the matrix
// cores 24 % busy (192 workgroups; 53 and 32 % on the CUs that have one), at D = 64 71 and
// 28 %, at D = 256 50 and 42 %.
//
// m is raised only where a tile's maximum passes it by over RAISE: accumulators are
// rescaled seldom.  Weights carry a factor 2^LIFT: at most 2^(LIFT + RAISE) < 65504,
// and full precision down to 2^-(14 + LIFT) of the nominal maximum.
#pragma once

#include <type_traits>

#include "common.h"
#include "k_kv.h"

namespace w4a4 {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr float ATT_RAISE = 8.0f, ATT_LIFT = 6.0f;  // powers of two
// A row's exponents t f - m + LIFT come from one fused step up to this |m - LIFT|: what m's
// rounding took is then 2^-4 at most.  From |m| of 2^24 on it would carry weights over
// fp16's range, or all of a row's below it; past this bound products are rounded as m
// was, and m is taken from them before LIFT comes to it: the largest is 2^LIFT exactly.
constexpr float ATT_FAR = 1048576.0f;

// Scores are the products' sums t times f = 2^k scale log2(e), k their keys' exponent.  Where
// f itself is no normal number, 2^k and the rest come one after the other: the scores may
// be ordinary for all that, and a factor of 0 is no mask (0 times -infinity).
__device__ __forceinline__ bool att_normal(float f) { return f >= 1.17549435e-38f && f < INFINITY; }

// Weighted values are summed in units of 2^E, E whole, of each row.  What a block adds is
// of the size of its value scale 2^e times its largest weight, and E follows the largest
// size of what the row has seen (where m rises, all before get smaller), and not the
// largest scale: beside one whose weights are almost nothing, others would lose their
// bits.  Weights of a scale up to 2^ABOVE over the unit are multiplied by the ratio, as those
// below it; further ones get it in the exponent, and are summed for themselves.  E stays
// where it is up to SPARE over what it could be, so that blocks of nearly one scale raise
// it seldom.  A weight times its scale is off by 2^-24 of the largest size at most:
// fp16's half step, 2^-25, times 2^ABOVE, 2^(SPARE + 1), over 2^LIFT.  (Sums are joined by
// fp32 factors, which end at 2^-126: weights below 2^(RAISE - 126) may be lost with them.)
constexpr float ATT_ABOVE = 4.0f, ATT_SPARE = 2.0f, ATT_NEVER = -2000.0f;
constexpr float ATT_UNSEEN = 1000.0f;  // E of a row that has seen nothing
// x <= 0, an exponent, up to the next whole number; NaN (neither has seen anything) as NEVER.
__device__ __forceinline__ float att_whole(float x) { return ceilf(fmaxf(x, ATT_NEVER)); }
// The least E for a block of scale 2^e and largest score top, and where E may stay if it holds m.
__device__ __forceinline__ float att_size(float E, float e, float top, float m) {
    return fmaxf(e + att_whole(fminf(top - m, 0.0f)), top >= m && E <= e + ATT_SPARE ? E : ATT_NEVER);
}

struct AttendArgs {
    const uint8_t *q;
    uint8_t *out;
    float *lse;
    int64_t q_row, q_head, o_row, o_head, lse_row;  // in elements
    float scale_log2;                               // of the scores, times log2(e)
    int32_t heads, group;                           // query heads; of them for one key/value head
    int32_t causal, window, odt;
    KvPool pool;
    KvBatch batch;
    // partial results: [slots][rows of a tile][D] weighted means, then [slots][rows][2] maxima and sums
    float *part, *part_ml;
    int32_t splits;      // workgroups that share a tile's tokens (many rows)
    int32_t workers;     // workgroups that share all tiles' tokens evenly; 0: one workgroup a tile and head
    int32_t tile_bound;  // at least the tiles of the batch
};

// Two dwords of codes (8 values) as a 16-bit operand, times the power of two s.
template <bool BF16>
__device__ __forceinline__ v4u widen_e4m3(uint32_t lo, uint32_t hi, float s) {
    if constexpr (BF16) {
        const v2b a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, 1);
        const v2b c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, 0), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, 1);
        return v4u{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                   __builtin_bit_cast(uint32_t, d)};
    } else {
        const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, s, 1);
        const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, s, 0), d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, s, 1);
        return v4u{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                   __builtin_bit_cast(uint32_t, d)};
    }
}
template <bool BF16>
__device__ __forceinline__ v4f mfma_16x16x32(v4u a, v4u b, v4f c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Two fp32 values as fp16, to nearest even.
__device__ __forceinline__ uint32_t f16_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2h));
}
// Two fp16 values times f; 2^e, e whole.
__device__ __forceinline__ uint32_t scale_pair(uint32_t x, _Float16 f) { return __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, x) * v2h{f, f}); }
__device__ __forceinline__ _Float16 half_power(float e) { return (_Float16)ldexpf(1.0f, (int)e); }
// c + the sum of two fp16 values, times f.
__device__ __forceinline__ float add_pair(uint32_t x, _Float16 f, float c) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(v2h, x), v2h{f, f}, c, false);
}

// x over the lanes l and l ^ 32; l and l ^ 16; l, l ^ 16, l ^ 32 and l ^ 48.
template <class F>
__device__ __forceinline__ float over_halves(float x, F f) {
    const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return f(__uint_as_float(y[0]), __uint_as_float(y[1]));
}
template <class F>
__device__ __forceinline__ float over_pairs(float x, F f) {
    const auto y = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return f(__uint_as_float(y[0]), __uint_as_float(y[1]));
}
template <class F>
__device__ __forceinline__ float over_groups(float x, F f) {
    return over_halves(over_pairs(x, f), f);
}
struct Larger {
    __device__ __forceinline__ float operator()(float x, float y) const { return fmaxf(x, y); }
};
struct Sum {
    __device__ __forceinline__ float operator()(float x, float y) const { return x + y; }
};

// The wave's lanes' largest (NaN passed over), and their sum in a fixed order, in each.
__device__ __forceinline__ float wave_larger(float x) {
    x = fmaxf(x, dpp_of<DPP_XOR1>(x));
    x = fmaxf(x, dpp_of<DPP_XOR2>(x));
    x = fmaxf(x, dpp_of<DPP_MIRROR8>(x));
    return over_groups(fmaxf(x, dpp_of<DPP_MIRROR16>(x)), Larger{});
}
__device__ __forceinline__ float wave_sum32(float x) {
    x += dpp_of<DPP_XOR1>(x);
    x += dpp_of<DPP_XOR2>(x);
    x += dpp_of<DPP_MIRROR8>(x);
    return over_groups(x + dpp_of<DPP_MIRROR16>(x), Sum{});
}

// The tokens that rows [r0, r1) of a sequence's head group see: [lo, hi), in
// tokens; hi <= lo: none.
struct Span {
    int lo, hi;
};
__device__ __forceinline__ Span span_of(const AttendArgs &a, const KvSeq &s, int r0, int r1) {
    const int first = s.first() + r0 / a.group, last = s.first() + (r1 - 1) / a.group;
    const int64_t low = a.window ? (int64_t)first - a.window + 1 : 0;
    return Span{(int)(low > 0 ? low : 0), a.causal ? min(s.len, last + 1) : s.len};
}

// What sums of weighted values are multiplied with: the weights' sum, inverse; 0 for
// a row that sees nothing.  Before the values' own exponent, so that no product on the
// way is larger than the values are.
__device__ __forceinline__ float inverse(float total) { return total == 0.0f ? 0.0f : 1.0f / total; }

// Where a row's result goes.
struct RowOut {
    uint8_t *out;
    int odt;
    __device__ __forceinline__ void store(int d, v4f y) const {  // four channels
        uint32_t w[2];
#pragma unroll
        for (int x = 0; x < 2; x++) {
            const float lo = y[2 * x], hi = y[2 * x + 1];
            w[x] = odt == ROW_F16 ? f16_pair(lo, hi) : __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{lo, hi}), v2b));
        }
        typedef v2u v2u_any __attribute__((aligned(2)));
        *reinterpret_cast<v2u_any *>(out + d * 2) = v2u{w[0], w[1]};
    }
};
// Weights that sum to `total` stand on maximum m (a power of two, above LIFT).
__device__ __forceinline__ RowOut row_out(const AttendArgs &a, int row0, int r, int head, float m, float total, bool lse) {
    const int i = r / a.group, h = head * a.group + (r - i * a.group);
    if (lse && a.lse)
        a.lse[(int64_t)(row0 + i) * a.lse_row + h] =
            total == 0.0f ? -INFINITY : (m - ATT_LIFT + __builtin_amdgcn_logf(total)) * 0.693147180559945309f;
    return RowOut{a.out + ((int64_t)(row0 + i) * a.o_row + (int64_t)h * a.o_head) * 2, a.odt};
}

// Tiles of R rows of a sequence, for one head.
template <int R>
__device__ __forceinline__ int tiles_of(const AttendArgs &a, const KvSeq &s) {
    return (int)(((int64_t)s.n * a.group + R - 1) / R);
}

// ---------------------------------------------------------------------------
// Few rows: a wave streams the cache from memory into its registers
// ---------------------------------------------------------------------------

constexpr int STREAM_WAVES = 4, STREAM_PAIR = 2 * KV_BLOCK;  // a step of a wave: two blocks
constexpr int STREAM_LEAST = 8;                              // steps of a worker, at least
constexpr int STREAM_WORKERS = 256;                          // at most: a thread each where they are joined

// The steps from a tile's first token that it sees to the last.
__device__ __forceinline__ int steps_over(const Span &x) { return x.hi <= x.lo ? 0 : (x.hi + STREAM_PAIR - 1) / STREAM_PAIR - x.lo / STREAM_PAIR; }
// Steps that count for a tile of a sequence of n > 0 rows: one number for all of them,
// at least what each takes, so that any can be found without the others (a prompt of 512
// rows beside 255 single ones, 8 x 8 heads of 128, shared: 700 us, and 2130 where every
// workgroup and row summed the tiles before its own; its 4000 tasks are not shared
// any more, 452).
template <int R>
__device__ __forceinline__ int steps_each(const AttendArgs &a, const KvSeq &s) {
    int steps = steps_over(span_of(a, s, 0, s.n * a.group));
    if (a.window && a.causal) steps = (int)min((int64_t)steps, ((int64_t)a.window + (R - 1) / a.group + STREAM_PAIR) / STREAM_PAIR + 1);
    return max(steps, 1);  // a tile without tokens writes zeros
}
template <int R>
__device__ __forceinline__ int64_t steps_of(const AttendArgs &a, const KvSeq &s) {
    return s.n > 0 ? (int64_t)tiles_of<R>(a, s) * steps_each<R>(a, s) : 0;
}
template <int R>
__device__ __forceinline__ int64_t all_steps(const AttendArgs &a, int page_tokens, int lane) {
    int64_t mine = 0;
    for (int b = lane; b < a.batch.seqs; b += 64) mine += steps_of<R>(a, kv_seq(a.batch, page_tokens, b));
    return wave_pick(wave_scan(mine), 63) * a.pool.heads;
}
// Workers in use, and where worker w begins among all steps.
__device__ __forceinline__ int64_t workers_used(int64_t steps, int workers) {
    const int64_t most = (steps + STREAM_LEAST - 1) / STREAM_LEAST;
    return most < workers ? most : workers;
}

// R = 16 NR rows (one head group's) of one sequence against its tokens, 64 a step:
// S^T = K Q^T by 16 x 16 x 32 products, whose rows are chosen such that lane group
// g holds the tokens of block g / 2 and half g % 2 as the value pieces have them.
// A wave asks for a step's 128 D bytes at once, 16 contiguous bytes a lane: with 4 waves
// a CU 128 KB in flight at D = 256, and no faster with 8 or 16.  Short sequences are a
// chain of latencies (lengths, page, codes, two steps, the waves' sums): 300 tokens 8.6 us.
template <int D, bool BF16, int NR>
__global__ __launch_bounds__(64 * STREAM_WAVES) void attend_stream_kernel(AttendArgs a) {
    constexpr int R = 16 * NR, J = D / 64, C = D / 32, PITCH = D + 4;
    __shared__ __align__(16) float sums[STREAM_WAVES * R * PITCH];
    __shared__ float mls[STREAM_WAVES][R][2];
    __shared__ float es[STREAM_WAVES][R];
    __shared__ __align__(16) v4f stats[R];  // of all waves: maximum, sum, its inverse, exponent
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int t16 = lane & 15, g = lane >> 4, page_tokens = a.pool.per_page * KV_BLOCK, heads = a.pool.heads;

    // where this workgroup begins, and how many steps it has
    int b, head, tile, step;
    int64_t left;
    if (a.workers) {
        const int64_t all = all_steps<R>(a, page_tokens, lane), used = workers_used(all, a.workers);
        const int64_t w = blockIdx.x;
        if (w >= used) return;
        int64_t at = all * w / used;
        left = all * (w + 1) / used - at;
        b = kv_find(a.batch.seqs, at, lane, [&](int i) { return steps_of<R>(a, kv_seq(a.batch, page_tokens, i)) * heads; });
        if (b < 0) return;
        const KvSeq s = kv_seq(a.batch, page_tokens, b);
        const int64_t of_head = steps_of<R>(a, s), of_tile = steps_each<R>(a, s);
        head = (int)(at / of_head);
        at -= head * of_head;
        tile = (int)(at / of_tile);
        step = (int)(at - tile * of_tile);
    } else {
        int32_t id = (int32_t)(blockIdx.x / heads);
        head = (int)(blockIdx.x % heads), step = 0, left = int64_t{1} << 40;
        b = kv_find(a.batch.seqs, id, lane, [&](int i) { return tiles_of<R>(a, kv_seq(a.batch, page_tokens, i)); });
        if (b < 0) return;
        tile = id;
    }

    for (;;) {
        const KvSeq s = kv_seq(a.batch, page_tokens, b);
        const int rows = (int)min((int64_t)R, (int64_t)s.n * a.group - (int64_t)tile * R);
        const Span span = span_of(a, s, tile * R, tile * R + rows);
        const int steps = steps_each<R>(a, s), stop = (int)min((int64_t)steps, step + left), pair0 = span.lo / STREAM_PAIR;
        const int some = min(stop, steps_over(span));  // of them, up to here there are tokens

        // the queries, and what each row sees
        v4u q[NR][J][2];
        int row_lo[NR], row_hi[NR];
#pragma unroll
        for (int n = 0; n < NR; n++) {
            const int r = tile * R + 16 * n + t16;
            const bool live = 16 * n + t16 < rows;
            const int i = live ? r / a.group : 0, h = live ? r - i * a.group : 0;
            const uint8_t *p = a.q + ((int64_t)(s.row + i) * a.q_row + (int64_t)(head * a.group + h) * a.q_head) * 2;
#pragma unroll
            for (int j = 0; j < J; j++)
#pragma unroll
                for (int k = 0; k < 2; k++)
                    q[n][j][k] = live ? *reinterpret_cast<const v4u_any *>(p + (64 * j + 16 * g + 8 * k) * 2) : v4u{0, 0, 0, 0};
            const Span x = span_of(a, s, live ? r : tile * R, (live ? r : tile * R) + 1);
            row_lo[n] = x.lo, row_hi[n] = live ? x.hi : 0;
        }
        // tokens in here are seen by every live row
        const int every_lo = span_of(a, s, tile * R + rows - 1, tile * R + rows).lo;
        const int every_hi = span_of(a, s, tile * R, tile * R + 1).hi;

        float m[NR], l[NR];
        v4f o[NR][C][2];
        float E[NR];
#pragma unroll
        for (int n = 0; n < NR; n++) {
            m[n] = -INFINITY, l[n] = 0.0f, E[n] = ATT_UNSEEN;
#pragma unroll
            for (int c = 0; c < C; c++) o[n][c][0] = o[n][c][1] = v4f{0, 0, 0, 0};
        }

        // lane 2 k + x: block x of this wave's step k of the next 32
        int held_block = 0, held_scale = 0;
        int k = 32;
        const int begin = step + wave;
        for (int u = begin; u < some; u += STREAM_WAVES, k++) {
            if (k == 32) {
                k = 0;
                const int blk = 2 * (pair0 + u + (lane >> 1) * STREAM_WAVES) + (lane & 1);
                held_block = (int64_t)blk * KV_BLOCK < s.len ? kv_block(a.pool, a.batch, b, head, blk) : -1;
                held_scale = held_block >= 0 ? reinterpret_cast<const uint16_t *>(a.pool.scales)[held_block] : 0;
            }
            const int b0 = wave_pick(held_block, 2 * k), b1 = wave_pick(held_block, 2 * k + 1);
            const int s0 = wave_pick(held_scale, 2 * k), s1 = wave_pick(held_scale, 2 * k + 1);
            const uint8_t *p0 = a.pool.codes + (int64_t)max(b0, 0) * (64 * D), *p1 = a.pool.codes + (int64_t)max(b1, 0) * (64 * D);
            const uint8_t *kp = (t16 & 8 ? p1 : p0) + (g >> 1) * 1024 + (g & 1) * 512 + (t16 & 7) * 16;
            const uint8_t *vp = (g & 2 ? p1 : p0) + 32 * D + (g & 1) * 512 + t16 * 16;
            v4u kr[4][J], vr[C][2];
#pragma unroll
            for (int x = 0; x < 4; x++)
#pragma unroll
                for (int j = 0; j < J; j++) kr[x][j] = *reinterpret_cast<const v4u *>(kp + j * 2048 + x * 128);
#pragma unroll
            for (int c = 0; c < C; c++)
#pragma unroll
                for (int x = 0; x < 2; x++) vr[c][x] = *reinterpret_cast<const v4u *>(vp + c * 1024 + x * 256);

            const int mine = g & 2 ? s1 : s0, token = (pair0 + u) * STREAM_PAIR + (g & 2 ? 32 : 0) + (g & 1) * 4;
            const bool have = (g & 2 ? b1 : b0) >= 0;
            float f = ldexpf(a.scale_log2, (mine & 255) - 127);

            // subtile x = 2 i + q holds tokens 16 i + 8 q + 4 h + r
            v4f st[NR][4];
#pragma unroll
            for (int x = 0; x < 4; x++) {
#pragma unroll
                for (int n = 0; n < NR; n++) st[n][x] = v4f{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < J; j++) {
                    const v4u k0 = widen_e4m3<BF16>(kr[x][j][0], kr[x][j][1], 1.0f), k1 = widen_e4m3<BF16>(kr[x][j][2], kr[x][j][3], 1.0f);
#pragma unroll
                    for (int n = 0; n < NR; n++) {
                        st[n][x] = mfma_16x16x32<BF16>(k0, q[n][j][0], st[n][x]);
                        st[n][x] = mfma_16x16x32<BF16>(k1, q[n][j][1], st[n][x]);
                    }
                }
            }
            const int tokens0 = (pair0 + u) * STREAM_PAIR;
            const bool whole = b0 >= 0 && b1 >= 0 && tokens0 + STREAM_PAIR <= s.len;
            if (!whole || tokens0 < every_lo || tokens0 + STREAM_PAIR > every_hi || __ballot(!att_normal(f)) != 0) {
                const bool apart = !att_normal(f);
#pragma unroll
                for (int n = 0; n < NR; n++)
#pragma unroll
                    for (int x = 0; x < 4; x++)
#pragma unroll
                        for (int r = 0; r < 4; r++) {
                            const int t = token + 8 * x + r;
                            if (apart) st[n][x][r] = ldexpf(st[n][x][r], (mine & 255) - 127) * a.scale_log2;
                            if (!have || t < row_lo[n] || t >= row_hi[n]) st[n][x][r] = -INFINITY;
                        }
                f = apart ? 1.0f : f;
            }
            if (!whole) {  // nothing but zeros where there is no token
                const int t0 = tokens0 + (g & 2 ? 32 : 0), in = have ? min(max(s.len - t0, 0), KV_BLOCK) : 0;
#pragma unroll
                for (int x = 0; x < 4; x++) {
                    const uint32_t mask = kv_token_bytes(x >> 1, x & 1, g & 1, 0, in);
#pragma unroll
                    for (int c = 0; c < C; c++) vr[c][0][x] &= mask, vr[c][1][x] &= mask;
                }
            }

            const float e = have ? (float)((mine >> 8) - 127) : ATT_NEVER;  // of this lane's tokens' values
            float top[NR], own_top[NR];  // of the step's two blocks, and of this lane's
            bool raise = false;
#pragma unroll
            for (int n = 0; n < NR; n++) {
                float t = st[n][0][0];
#pragma unroll
                for (int x = 0; x < 4; x++)
#pragma unroll
                    for (int r = 0; r < 4; r++) t = fmaxf(t, st[n][x][r]);
                t = over_pairs(t * f, Larger{});
                own_top[n] = t, top[n] = over_halves(t, Larger{});
                raise |= top[n] - m[n] > ATT_RAISE || (E[n] < e && t - m[n] > E[n] - e);
            }
            if (__ballot(raise) != 0) {
#pragma unroll
                for (int n = 0; n < NR; n++) {
                    const bool up = top[n] - m[n] > ATT_RAISE;
                    const float fall = up ? m[n] - top[n] : 0.0f, was = E[n];
                    if (up) m[n] = top[n];
                    E[n] = fmaxf(E[n] + att_whole(fall), over_halves(att_size(E[n], e, own_top[n], m[n]), Larger{}));
                    const float beta = __builtin_amdgcn_exp2f(fall + (was - E[n]));
                    l[n] *= __builtin_amdgcn_exp2f(fall);
#pragma unroll
                    for (int c = 0; c < C; c++)
#pragma unroll
                        for (int x = 0; x < 2; x++)
#pragma unroll
                            for (int r = 0; r < 4; r++) o[n][c][x][r] *= beta;
                }
            }
            uint32_t p[NR][4][2];
#pragma unroll
            for (int n = 0; n < NR; n++) {
                float base = (m[n] > -INFINITY ? m[n] : 0.0f) - ATT_LIFT, by = f;
                float shift = e - E[n];
                _Float16 counted = (_Float16)1.0f;
                if (__ballot(fabsf(base) > ATT_FAR || shift > ATT_ABOVE) != 0) {
                    const bool far = fabsf(base) > ATT_FAR;
#pragma unroll
                    for (int x = 0; x < 4; x++)
#pragma unroll
                        for (int r = 0; r < 4; r++) st[n][x][r] = far ? st[n][x][r] * f - m[n] : st[n][x][r];
                    base = far ? -ATT_LIFT : base, by = far ? 1.0f : by;
                    if (shift > ATT_ABOVE) {
#pragma unroll
                        for (int x = 0; x < 4; x++)
#pragma unroll
                            for (int r = 0; r < 4; r++) l[n] += __builtin_amdgcn_exp2f(__builtin_fmaf(st[n][x][r], by, -base));
                        base -= shift, shift = 0.0f, counted = (_Float16)0.0f;
                    }
                }
                const _Float16 unit = half_power(shift);
#pragma unroll
                for (int x = 0; x < 4; x++)
#pragma unroll
                    for (int r = 0; r < 2; r++) {
                        p[n][x][r] = f16_pair(__builtin_amdgcn_exp2f(__builtin_fmaf(st[n][x][2 * r], by, -base)),
                                              __builtin_amdgcn_exp2f(__builtin_fmaf(st[n][x][2 * r + 1], by, -base)));
                        l[n] = add_pair(p[n][x][r], counted, l[n]);
                        p[n][x][r] = scale_pair(p[n][x][r], unit);
                    }
            }
#pragma unroll
            for (int c = 0; c < C; c++)
#pragma unroll
                for (int x = 0; x < 2; x++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const v4u v = widen_e4m3<false>(vr[c][x][i], vr[c][x][2 + i], 1.0f);
#pragma unroll
                        for (int n = 0; n < NR; n++)
                            o[n][c][x] = mfma_16x16x32<false>(
                                v, v4u{p[n][2 * i][0], p[n][2 * i][1], p[n][2 * i + 1][0], p[n][2 * i + 1][1]}, o[n][c][x]);
                    }
        }

        // the waves' sums, on the largest of their maxima
        const bool done = step == 0 && stop == steps;
#pragma unroll
        for (int n = 0; n < NR; n++) {
            l[n] = over_groups(l[n], Sum{});
            if (g == 0) mls[wave][16 * n + t16][0] = m[n], mls[wave][16 * n + t16][1] = l[n], es[wave][16 * n + t16] = E[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NR; n++) {
            float M = -INFINITY, top = 2 * ATT_NEVER, total = 0.0f;
#pragma unroll
            for (int w = 0; w < STREAM_WAVES; w++) M = fmaxf(M, mls[w][16 * n + t16][0]);
#pragma unroll
            for (int w = 0; w < STREAM_WAVES; w++) {
                const float below = mls[w][16 * n + t16][0] - M;  // NaN where a wave has seen nothing
                top = fmaxf(top, es[w][16 * n + t16] + att_whole(below));
                total += mls[w][16 * n + t16][0] > -INFINITY ? __builtin_amdgcn_exp2f(below) * mls[w][16 * n + t16][1] : mls[w][16 * n + t16][1];
            }
            if (wave == 0 && g == 0) stats[16 * n + t16] = v4f{M, total, inverse(total), top};
            const float alpha = m[n] > -INFINITY ? __builtin_amdgcn_exp2f(m[n] - M + (E[n] - top)) : 0.0f;
            if (16 * n + t16 < rows) {
#pragma unroll
                for (int c = 0; c < C; c++)
#pragma unroll
                    for (int x = 0; x < 2; x++) {
                        v4f y = o[n][c][x];
#pragma unroll
                        for (int r = 0; r < 4; r++) y[r] *= alpha;
                        *reinterpret_cast<v4f *>(sums + (wave * R + 16 * n + t16) * PITCH + 32 * c + 16 * x + 4 * g) = y;
                    }
            }
        }
        __syncthreads();
        const int64_t slot = 2 * (int64_t)blockIdx.x + (step == 0 ? 1 : 0);  // of a tile begun here, or before
        for (int at = tid; at < rows * (D / 4); at += 64 * STREAM_WAVES) {
            const int r = at / (D / 4), d = at % (D / 4) * 4;
            const v4f of = stats[r];
            const float M = of[0], total = of[1];
            v4f y = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < STREAM_WAVES; w++) y += *reinterpret_cast<const v4f *>(sums + (w * R + r) * PITCH + d);
#pragma unroll
            for (int i = 0; i < 4; i++) y[i] = ldexpf(y[i] * of[2], (int)of[3]);
            if (!done) {
                *reinterpret_cast<v4f *>(a.part + (slot * R + r) * D + d) = y;
                if (d == 0) a.part_ml[(slot * R + r) * 2] = M, a.part_ml[(slot * R + r) * 2 + 1] = total;
                continue;
            }
            row_out(a, s.row, tile * R + r, head, M, total, d == 0).store(d, y);
        }
        left -= stop - step;
        if (left <= 0 || !a.workers) return;
        // the next tile, head, sequence
        step = 0;
        if (++tile == tiles_of<R>(a, s)) {
            tile = 0;
            if (++head == heads) {
                head = 0;
                do b++;
                while (b < a.batch.seqs && kv_seq(a.batch, page_tokens, b).n == 0);
                if (b >= a.batch.seqs) return;
            }
        }
        __syncthreads();
    }
}

// One row of a tile whose tokens several workers had: their sums joined, always
// in the workers' order.
template <int D, int R>
__global__ __launch_bounds__(64 * STREAM_WAVES) void attend_join_kernel(AttendArgs a) {
    __shared__ v4f sums[1024 / D][D / 4];
    __shared__ float weights[STREAM_WAVES], tops[STREAM_WAVES], factors[STREAM_WORKERS];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int page_tokens = a.pool.per_page * KV_BLOCK, heads = a.pool.heads, row = (int)blockIdx.y;
    int32_t tile = (int32_t)(blockIdx.x / heads);
    const int head = (int)(blockIdx.x % heads);
    const int b = kv_find(a.batch.seqs, tile, lane, [&](int i) { return tiles_of<R>(a, kv_seq(a.batch, page_tokens, i)); });
    if (b < 0) return;
    const KvSeq s = kv_seq(a.batch, page_tokens, b);
    if (row >= (int64_t)s.n * a.group - (int64_t)tile * R) return;
    int64_t before = 0, own = 0, all = 0;  // steps of the sequences before, of this one, of all: for one head
    for (int i = lane; i < a.batch.seqs; i += 64) {
        const int64_t n = steps_of<R>(a, kv_seq(a.batch, page_tokens, i));
        all += n;
        if (i < b) before += n;
        if (i == b) own += n;
    }
    all = wave_pick(wave_scan(all), 63) * heads;
    before = wave_pick(wave_scan(before), 63) * heads;
    own = wave_pick(wave_scan(own), 63);
    int64_t begin = before + head * own;
    begin += (int64_t)tile * steps_each<R>(a, s);
    const int64_t end = begin + steps_each<R>(a, s), used = workers_used(all, a.workers);
    const int w0 = (int)(((begin + 1) * used - 1) / all), w1 = (int)((end * used - 1) / all);
    if (w0 == w1) return;  // written by its only worker

    auto slot = [&](int w) { return (int64_t)(2 * w + (w == w0 ? 1 : 0)) * R + row; };
    const int count = w1 - w0 + 1;  // at most STREAM_WORKERS
    v2f ml = {-INFINITY, 0.0f};
    if (tid < count) ml = *reinterpret_cast<const v2f *>(a.part_ml + slot(w0 + tid) * 2);
    float m = wave_larger(ml.x);
    if (lane == 0) tops[wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    const float f = ml.x > -INFINITY ? __builtin_amdgcn_exp2f(ml.x - m) : 1.0f;
    float total = wave_sum32(tid < count ? f * ml.y : 0.0f);
    if (lane == 0) weights[wave] = total;
    __syncthreads();
    total = (weights[0] + weights[1]) + (weights[2] + weights[3]);
    if (tid < count) factors[tid] = f * ml.y * inverse(total);
    __syncthreads();
    // 4 channels a lane: a load of a wave holds 256 / D workers' rows
    constexpr int LANES = D / 4, SIDE = 256 / LANES;
    const int d = tid % LANES * 4, side = tid / LANES;
    v4f y = {0, 0, 0, 0};
#pragma unroll 8
    for (int i = side; i < count; i += SIDE) y += factors[i] * *reinterpret_cast<const v4f *>(a.part + slot(w0 + i) * D + d);
    sums[side][tid % LANES] = y;
    __syncthreads();
    if (tid >= LANES) return;
#pragma unroll
    for (int i = 1; i < SIDE; i++) y += sums[i][tid];
    row_out(a, s.row, tile * R + row, head, m, total, tid == 0).store(d, y);
}

// ---------------------------------------------------------------------------
// Many rows: a workgroup's waves share the cache's blocks through LDS
// ---------------------------------------------------------------------------

__device__ __forceinline__ v16f mfma_32x32x16_f16(v4u a, v4u b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}
template <bool BF16>
__device__ __forceinline__ v16f mfma_32x32x16(v4u a, v4u b, v16f c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
    else return mfma_32x32x16_f16(a, b, c);
}

// 16 bytes a lane from p + at (p uniform) to LDS byte address lds + 16 lane
// (uniform), without passing registers; counted by vmcnt, unseen by the compiler.
__device__ __forceinline__ void att_load16(const uint8_t *p, uint32_t at, uint32_t lds) {
    uint32_t m0;  // written; the load that reads it needs one wait state
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" : "={m0}"(m0) : "v"(at), "s"(p), "s"(lds) : "memory");
}

// What holds a workgroup here: blocks come to LDS as 8-bit codes by direct loads (2
// a wave and block at D = 256), so that 8 waves share each; a wave converts what it
// reads.  Converted once, in LDS, they would be twice the reads, as long as the products
// take.  Measured at D = 256, two waves a SIMD, cycles a block: keys 1050 and values 1050
// (the matrix cores' 512 each, for both waves), softmax 820, loads, barrier and loop 600;
// the two waves' products hardly meet the other's softmax.  Half a turn apart by barriers
// (one multiplies while the other exponentiates) it was slower, 505 us against 428: a wave
// alone issues a vector instruction every 7 to 8 cycles.  64 rows a wave (D = 64, 128)
// changed nothing, nor did reads further ahead.
//
// RW waves of 32 rows each, times TW that take turns at a stage's blocks.
template <int D_, int RW_>
struct AttTile {
    static constexpr int D = D_, RW = RW_, WAVES = 8, TW = WAVES / RW, ROWS = 32 * RW, THREADS = 64 * WAVES;
    static constexpr int EU_WAVES = D == 64 ? 4 : 2;  // a SIMD's waves: what the registers are held to
    static constexpr int BLOCK_BYTES = 64 * D;
    static constexpr int SB = D == 256 ? (TW > 2 ? TW : 2) : (TW > 4 ? TW : 4);  // blocks of a stage
    static constexpr int RING = SB * BLOCK_BYTES > 49152 ? 2 : 3;                // stages in LDS
    static constexpr int LOADS = SB * BLOCK_BYTES / 1024 / WAVES;                // of a wave and stage
    static constexpr int STAGE_BYTES = SB * BLOCK_BYTES, RING_BYTES = RING * STAGE_BYTES;
    static constexpr int JOIN_BYTES = TW > 1 ? 4 * 32 * D * 4 + WAVES * 64 * 12 : 0;  // half of the waves' sums, maxima and exponents
    static constexpr int LDS = RING_BYTES > JOIN_BYTES ? RING_BYTES : JOIN_BYTES;
    static_assert(SB % TW == 0 && 64 % SB == 0 && LOADS >= 1 && LOADS * WAVES * 1024 == SB * BLOCK_BYTES && LDS <= 163840, "");
};

template <int N>
__device__ __forceinline__ void att_wait() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// The order of N pieces' reads, conversions and products: two reads ahead, and
// each product's conversions while the one before runs.
template <int N>
__device__ __forceinline__ void att_interleave() {
    constexpr int READ = 0x100, VALU = 0x2, MFMA = 0x8, AHEAD = 2;
    __builtin_amdgcn_sched_group_barrier(READ, AHEAD, 0);
#pragma unroll
    for (int c = 0; c < N; c++) {
        __builtin_amdgcn_sched_group_barrier(VALU, 4, 0);
        __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
        __builtin_amdgcn_sched_group_barrier(VALU, 4, 0);
        if (c + AHEAD < N) __builtin_amdgcn_sched_group_barrier(READ, 1, 0);
        __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
    }
}

template <class C, bool BF16>
__global__ __launch_bounds__(C::THREADS, C::EU_WAVES) void attend_tile_kernel(AttendArgs a) {
    constexpr int D = C::D, N = D / 32;
    __shared__ __align__(1024) uint8_t smem[C::LDS];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int rw = wave % C::RW, tw = wave / C::RW, col = lane & 31, h = lane >> 5;
    const int page_tokens = a.pool.per_page * KV_BLOCK, heads = a.pool.heads;

    // splits and heads first, so that workgroups of one XCD share keys and values;
    // the last tiles, which see most, first
    const int split = (int)(blockIdx.x % a.splits), task = (int)(blockIdx.x / a.splits), head = task % heads;
    const int order = a.tile_bound - 1 - task / heads;
    int32_t tile = order;
    const int b = kv_find(a.batch.seqs, tile, lane, [&](int i) { return tiles_of<C::ROWS>(a, kv_seq(a.batch, page_tokens, i)); });
    if (b < 0) return;
    const KvSeq s = kv_seq(a.batch, page_tokens, b);
    const int all_rows = (int)((int64_t)s.n * a.group), row0 = tile * C::ROWS, rows = min(C::ROWS, all_rows - row0);
    const Span span = span_of(a, s, row0, row0 + rows);
    const int first_block = span.lo / KV_BLOCK, blocks_all = span.hi <= span.lo ? 0 : (span.hi - 1) / KV_BLOCK + 1 - first_block;
    const int stages_all = (blocks_all + C::SB - 1) / C::SB;
    const int begin = (int)((int64_t)stages_all * split / a.splits), stages = __builtin_amdgcn_readfirstlane((int)((int64_t)stages_all * (split + 1) / a.splits) - begin);
    const int block0 = __builtin_amdgcn_readfirstlane(first_block + begin * C::SB), blocks = __builtin_amdgcn_readfirstlane(min(stages * C::SB, blocks_all - begin * C::SB));

    // this wave's rows, and what they see: each its own [row_lo, row_hi), one of them
    // [wspan.lo, wspan.hi), all [every_lo, every_hi)
    const int wrow0 = row0 + 32 * rw, wrows = min(max(rows - 32 * rw, 0), 32);
    const Span wspan = wrows ? span_of(a, s, wrow0, wrow0 + wrows) : Span{0, 0};
    const int every_lo = wrows ? span_of(a, s, wrow0 + wrows - 1, wrow0 + wrows).lo : 0;
    const int every_hi = wrows ? span_of(a, s, wrow0, wrow0 + 1).hi : 0;

    // lane i, for block i of 64 of this workgroup's: where it lies, and its scales (16
    // bits, and EDGE where not every row sees all of it or its factor is not normal), or -1 where this wave has
    // nothing to do.  One read of a lane a block then, not a dozen scalar operations.
    constexpr int EDGE = 1 << 16;
    int held_block = -1, held_info = -1, held_chunk = 0;
    uint32_t held_lo = 0, held_hi = 0;
    auto fetch_block = [&](int chunk) {
        const int rel = chunk * 64 + lane;
        held_chunk = chunk;
        held_block = rel < blocks ? kv_block(a.pool, a.batch, b, head, block0 + rel) : -1;
        const uint64_t at = reinterpret_cast<uint64_t>(a.pool.codes) + (uint64_t)max(held_block, 0) * C::BLOCK_BYTES;
        held_lo = (uint32_t)at, held_hi = (uint32_t)(at >> 32);
    };
    auto fetch_info = [&] {
        const int token = (block0 + held_chunk * 64 + lane) * KV_BLOCK;
        const bool some = held_block >= 0 && token + KV_BLOCK > wspan.lo && token < wspan.hi;
        held_info = some ? reinterpret_cast<const uint16_t *>(a.pool.scales)[held_block] : -1;
        if (some && (token < every_lo || token + KV_BLOCK > every_hi || !att_normal(ldexpf(a.scale_log2, (held_info & 255) - 127)))) held_info |= EDGE;
    };
    fetch_block(0);  // first: all that follows waits for the pages

    const bool live = col < wrows;
    const int r = live ? wrow0 + col : row0, qi = r / a.group;
    v4u q[N][2];
    {
        const uint8_t *p = a.q + ((int64_t)(s.row + qi) * a.q_row + (int64_t)(head * a.group + r - qi * a.group) * a.q_head) * 2;
#pragma unroll
        for (int c = 0; c < N; c++)
#pragma unroll
            for (int i = 0; i < 2; i++) q[c][i] = *reinterpret_cast<const v4u_any *>(p + (32 * c + 16 * h + 8 * i) * 2);
    }
    const Span mine = span_of(a, s, r, r + 1);
    const int row_lo = mine.lo, row_hi = live ? mine.hi : 0;

    // This wave's i-th load of a stage: unit (KB) wave + 8 i of its blocks.  at: the
    // stage's first block in the held 64; into: its place in LDS.
    const uint32_t ring = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)smem;
    constexpr int PIECES = D / 16;  // of a block
    const uint32_t lane_at = (wave % PIECES) * 1024 + lane * 16;
    auto load = [&](int at, uint32_t into, int i) {
        const int block = at + (wave + i * C::WAVES) / PIECES;
        const uint64_t p = (uint64_t)(uint32_t)wave_pick((int)held_hi, block) << 32 | (uint32_t)wave_pick((int)held_lo, block);
        att_load16(reinterpret_cast<const uint8_t *>(p), lane_at + i * C::WAVES % PIECES * 1024, into + wave * 1024 + i * (C::WAVES * 1024));
    };

    float m = -INFINITY, l = 0.0f;
    float E = ATT_UNSEEN;
    v16f o[N];
#pragma unroll
    for (int c = 0; c < N; c++) o[c] = v16f{};

    if (stages > 0) {
#pragma unroll
        for (int i = 0; i < C::LOADS; i++) load(0, ring, i);
    }
    fetch_info();
    // the queries here once, or the compiler waits for them in the loop, and with them
    // for the loads that it does not see
#pragma unroll
    for (int c = 0; c < N; c++) asm volatile("" : "+v"(q[c][0]), "+v"(q[c][1]), "+v"(held_info));
#pragma unroll
    for (int st = 1; st < C::RING - 1; st++) {
        if (st >= stages) break;
#pragma unroll
        for (int i = 0; i < C::LOADS; i++) load(st * C::SB, ring + st * C::STAGE_BYTES, i);
    }
    int info = held_info, from = 0, to = C::RING - 1;  // the stage's blocks, its place, and that of the next to ask for
    const int tail = __builtin_amdgcn_readfirstlane(s.len / KV_BLOCK - block0);               // the block with the sequence's end, of this workgroup's
    for (int st = 0; st < stages; st++) {
        if (C::RING > 2 && st + 1 < stages) att_wait<(C::RING - 2) * C::LOADS>();
        else att_wait<0>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");  // no read of the stage moves up
        const int first = st * C::SB, next = first + (C::RING - 1) * C::SB;  // blocks
        const bool more = st + C::RING - 1 < stages;  // a stage to ask for, while this one is worked on
        if ((first & 63) == 0 && st) info = held_info;
        if (more && (next & 63) == 0) {
            fetch_block(next / 64), fetch_info();
            asm volatile("" : "+v"(held_info));  // waited for here, and not every stage
        }
        uint8_t *stage = smem + from * C::STAGE_BYTES;
        // no value but zero where there is no token: once a sequence, in its last stage
        if (tail < first + C::SB) {
            for (int u = tid; u < C::SB * 2 * D; u += C::THREADS) {
                const int j = u / (2 * D), x = u % (2 * D), in = s.len - (block0 + first + j) * KV_BLOCK;
                if (in >= KV_BLOCK) continue;
                v4u *piece = reinterpret_cast<v4u *>(stage + j * C::BLOCK_BYTES + 32 * D) + x;
                v4u y = *piece;
#pragma unroll
                for (int i = 0; i < 4; i++) y[i] &= kv_token_bytes(i >> 1, i & 1, x / 32 % 2, 0, in);
                *piece = y;
            }
            __syncthreads();
        }
        const uint32_t into = ring + to * C::STAGE_BYTES;
        // as if neither were known: a turn taken out of the loop moves every sum between registers
        int j = tw, step = C::TW;
        asm("" : "+s"(j), "+s"(step));
#pragma unroll 1
        for (int turn = 0; j < C::SB; j += step, turn++) {
            int scale = wave_pick(info, (first & 63) + j);
            asm volatile("" : "+s"(scale));  // nor this (the second test below is a part of the same: -1 says it all)
            // a turn's share of the loads, in two parts: all at once they wait for each other
            auto ask = [&](auto part) {
                constexpr int SHARE = (C::LOADS * C::TW + C::SB - 1) / C::SB, LO = part ? (SHARE + 1) / 2 : 0, HI = part ? SHARE : (SHARE + 1) / 2;
#pragma unroll
                for (int i = LO; i < HI; i++)
                    if (more && turn * SHARE + i < C::LOADS) load(next & 63, into, turn * SHARE + i);
            };
            ask(std::integral_constant<int, 0>{});
            const bool some = scale >= 0 && (block0 + first + j) * KV_BLOCK < wspan.hi;
            if (!some) {
                ask(std::integral_constant<int, 1>{});
                continue;
            }
            const uint8_t *p = stage + j * C::BLOCK_BYTES + lane * 16;
            v16f t = {};
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int c = 0; c < N; c++) {
                const v4u x = *reinterpret_cast<const v4u *>(p + c * 1024);
                t = mfma_32x32x16<BF16>(widen_e4m3<BF16>(x[0], x[1], 1.0f), q[c][0], t);
                t = mfma_32x32x16<BF16>(widen_e4m3<BF16>(x[2], x[3], 1.0f), q[c][1], t);
            }
            att_interleave<N>();
            __builtin_amdgcn_sched_barrier(0);
            ask(std::integral_constant<int, 1>{});
            float f = ldexpf(a.scale_log2, (scale & 255) - 127);
            if (scale & EDGE) {
                if (!att_normal(f)) {
#pragma unroll
                    for (int v = 0; v < 16; v++) t[v] = ldexpf(t[v], (scale & 255) - 127) * a.scale_log2;
                    f = 1.0f;
                }
                const int token = (block0 + first + j) * KV_BLOCK;
#pragma unroll
                for (int v = 0; v < 16; v++) {
                    const int at = token + mfma32_row(v, lane);
                    if (at < row_lo || at >= row_hi) t[v] = -INFINITY;
                }
            }
            float top = t[0];
#pragma unroll
            for (int v = 1; v < 16; v++) top = fmaxf(top, t[v]);
            top = over_halves(top * f, Larger{});
            const bool up = top - m > ATT_RAISE;
            const float e = (float)((scale >> 8 & 255) - 127);
            const bool grow = E < e && top - m > E - e;  // of what the row sees
            if (__ballot(up || grow) != 0) {
                const float fall = up ? m - top : 0.0f, was = E;
                if (up) m = top;
                E = fmaxf(E + att_whole(fall), att_size(E, e, top, m));
                const float beta = __builtin_amdgcn_exp2f(fall + (was - E));
                l *= __builtin_amdgcn_exp2f(fall);
#pragma unroll
                for (int c = 0; c < N; c++)
#pragma unroll
                    for (int v = 0; v < 16; v++) o[c][v] *= beta;
            }
            float base = (m > -INFINITY ? m : 0.0f) - ATT_LIFT, by = f;
            float shift = e - E;
            _Float16 counted = (_Float16)1.0f;
            if (__ballot(fabsf(base) > ATT_FAR || shift > ATT_ABOVE) != 0) {
                const bool far = fabsf(base) > ATT_FAR;
#pragma unroll
                for (int v = 0; v < 16; v++) t[v] = far ? t[v] * f - m : t[v];
                base = far ? -ATT_LIFT : base, by = far ? 1.0f : by;
                if (shift > ATT_ABOVE) {
#pragma unroll
                    for (int v = 0; v < 16; v++) l += __builtin_amdgcn_exp2f(__builtin_fmaf(t[v], by, -base));
                    base -= shift, shift = 0.0f, counted = (_Float16)0.0f;
                }
            }
            const _Float16 unit = half_power(shift);
            v4u w[2];
#pragma unroll
            for (int v = 0; v < 8; v++) {
                const uint32_t x = f16_pair(__builtin_amdgcn_exp2f(__builtin_fmaf(t[2 * v], by, -base)),
                                            __builtin_amdgcn_exp2f(__builtin_fmaf(t[2 * v + 1], by, -base)));
                w[v / 4][v % 4] = scale_pair(x, unit);
                l = add_pair(x, counted, l);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int c = 0; c < N; c++) {
                const v4u x = *reinterpret_cast<const v4u *>(p + 32 * D + c * 1024);
                o[c] = mfma_32x32x16_f16(widen_e4m3<false>(x[0], x[2], 1.0f), w[0], o[c]);
                o[c] = mfma_32x32x16_f16(widen_e4m3<false>(x[1], x[3], 1.0f), w[1], o[c]);
            }
            att_interleave<N>();
            __builtin_amdgcn_sched_barrier(0);
        }
        from = from + 1 == C::RING ? 0 : from + 1, to = to + 1 == C::RING ? 0 : to + 1;
    }

    // The waves of the same rows: each pair exchanges halves of its channels, until a
    // wave has 4 N / TW quads of channels, from quad `base` on, of all.
    l = over_halves(l, Sum{});
    constexpr int QUADS = 4 * N / C::TW;
    int base = 0;
    if constexpr (C::TW > 1) {
        v4f *sums = reinterpret_cast<v4f *>(smem);  // [wave][quad][64 lanes]
        v2f *mls = reinterpret_cast<v2f *>(smem + 4 * 32 * D * 4);
        float *es = reinterpret_cast<float *>(smem + 4 * 32 * D * 4 + C::WAVES * 64 * 8);
        auto quad = [&](int z) { return v4f{o[z / 4][z % 4 * 4], o[z / 4][z % 4 * 4 + 1], o[z / 4][z % 4 * 4 + 2], o[z / 4][z % 4 * 4 + 3]}; };
#pragma unroll
        for (int half = C::TW / 2, n = 2 * N; half > 0; half /= 2, n /= 2) {  // n: quads kept, and given
            const bool upper = (tw & half) != 0;
            const int other = wave ^ (half * C::RW);
            __syncthreads();
            mls[wave * 64 + lane] = v2f{m, l};
            es[wave * 64 + lane] = E;
            if (upper) {
#pragma unroll
                for (int z = 0; z < n; z++) sums[(wave * n + z) * 64 + lane] = quad(z);
            } else {
#pragma unroll
                for (int z = 0; z < n; z++) sums[(wave * n + z) * 64 + lane] = quad(n + z);
            }
            __syncthreads();
            const v2f ml = mls[other * 64 + lane];
            const float mb = fmaxf(m, ml.x);
            const float e = es[other * 64 + lane], eb = fmaxf(E + att_whole(m - mb), e + att_whole(ml.x - mb));
            const float own = m > -INFINITY ? __builtin_amdgcn_exp2f(m - mb) : 1.0f, theirs = ml.x > -INFINITY ? __builtin_amdgcn_exp2f(ml.x - mb) : 1.0f;
            const float fo = m > -INFINITY ? __builtin_amdgcn_exp2f(m - mb + (E - eb)) : 1.0f;
            const float fe = ml.x > -INFINITY ? __builtin_amdgcn_exp2f(ml.x - mb + (e - eb)) : 1.0f;
            l = l * own + ml.y * theirs, m = mb, E = eb;
            if (upper) base += n;
#pragma unroll
            for (int z = 0; z < n; z++) {
                const v4f x = upper ? quad(n + z) : quad(z), y = sums[(other * n + z) * 64 + lane];
#pragma unroll
                for (int i = 0; i < 4; i++) o[z / 4][z % 4 * 4 + i] = x[i] * fo + y[i] * fe;
            }
        }
    }
    if (!live) return;
    const int64_t slot = ((int64_t)(order * heads + head) * a.splits + split) * C::ROWS + 32 * rw + col;
    const bool first = tw == 0 && h == 0;
    if (a.splits > 1) {
        if (first) a.part_ml[slot * 2] = m, a.part_ml[slot * 2 + 1] = l;
        if (m == -INFINITY && l == 0.0f) return;  // nothing seen: never read
    }
    const RowOut out = row_out(a, s.row, r, head, m, l, first && a.splits == 1);
    const float inv = inverse(l);
#pragma unroll
    for (int z = 0; z < QUADS; z++) {
        v4f y;
#pragma unroll
        for (int i = 0; i < 4; i++) y[i] = ldexpf(o[z / 4][z % 4 * 4 + i] * inv, (int)E);
        const int d = (base + z) * 8 + 4 * h;
        if (a.splits > 1) *reinterpret_cast<v4f *>(a.part + slot * D + d) = y;
        else out.store(d, y);
    }
}

constexpr int SPLITS_MOST = 32;

// The rows of a tile that `splits` workgroups had the tokens of, WAVES waves a row:
// one where the splits are few, four where the loads of many would follow each
// other (16 splits of 96 rows: 4.7 us against 8.4).
template <int D, int ROWS, int WAVES>
__global__ __launch_bounds__(256) void attend_splits_kernel(AttendArgs a) {
    constexpr int LANES = D / 4, SIDE = 64 * WAVES / LANES, ROW_THREADS = 64 * WAVES, TOGETHER = 4 / WAVES;
    __shared__ float factors[4][SPLITS_MOST];
    __shared__ v4f sums[TOGETHER][SIDE][LANES];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), of = wave / WAVES;
    const int page_tokens = a.pool.per_page * KV_BLOCK, heads = a.pool.heads;
    const int order = (int)(blockIdx.x / heads), head = (int)(blockIdx.x % heads);
    int32_t tile = order;
    const int b = kv_find(a.batch.seqs, tile, lane, [&](int i) { return tiles_of<ROWS>(a, kv_seq(a.batch, page_tokens, i)); });
    if (b < 0) return;
    const KvSeq s = kv_seq(a.batch, page_tokens, b);
    const int rows = (int)min((int64_t)ROWS, (int64_t)s.n * a.group - (int64_t)tile * ROWS);
    if ((int)blockIdx.y * TOGETHER >= rows) return;
    const int row = min((int)blockIdx.y * TOGETHER + of, rows - 1);  // the last again, where there are no more
    const int64_t slot0 = (int64_t)(order * heads + head) * a.splits * ROWS + row;
    const v2f own = lane < a.splits ? *reinterpret_cast<const v2f *>(a.part_ml + (slot0 + (int64_t)lane * ROWS) * 2) : v2f{-INFINITY, 0.0f};
    const float m = wave_larger(own.x), f = own.x > -INFINITY ? __builtin_amdgcn_exp2f(own.x - m) : 1.0f;
    const float total = wave_sum32(f * own.y);
    // a split without tokens wrote no sums: whatever lies there is not taken
    if (lane < a.splits) factors[wave][lane] = own.x > -INFINITY || own.y != 0.0f ? f * own.y * inverse(total) : -1.0f;
    __syncthreads();
    const int at = threadIdx.x % ROW_THREADS, d = at % LANES * 4, side = at / LANES;
    v4f y = {0, 0, 0, 0};
#pragma unroll 8
    for (int i = side; i < a.splits; i += SIDE) {
        const v4f x = *reinterpret_cast<const v4f *>(a.part + (slot0 + (int64_t)i * ROWS) * D + d);
        const float fi = factors[wave][i];
        y = fi != -1.0f ? y + fi * x : y;
    }
    sums[of][side][at % LANES] = y;
    __syncthreads();
    if (side) return;
#pragma unroll
    for (int i = 1; i < SIDE; i++) y += sums[of][i][at];
    row_out(a, s.row, tile * ROWS + row, head, m, total, d == 0).store(d, y);
}

}  // namespace w4a4
